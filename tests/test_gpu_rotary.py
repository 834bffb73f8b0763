"""Rotary positions and per-head q/k norms against their formulas in 64 bits.

Tolerances.  The kernels compute in fp32 (unit roundoff u = 2^-24) and round
once.  A rotated element is two products and a sum of cosines and sines that
are within 4 u of theirs: 8 u of its pair's size; the norm's factor adds the
error of a sum of squares (a tree of at most 16 + 8 terms a lane and 5
levels) and of rsqrt: 32 u.  64 u of the size of the terms covers both
passes.  bf16 outputs add half a unit in the last place, at most 2^-8 of the
value.  A gain's gradient is a sum of fp32 terms in a fixed order: its error
is at most u times the longest chain of additions times the sum of the
terms' sizes; no chain is longer than the number of terms plus 64."""

import ctypes

import pytest
import torch

from adamw_optimizer_step_gb300 import _binding as B
from adamw_optimizer_step_gb300 import layers

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    from adamw_optimizer_step_gb300 import build
    build.build()
    B.lib()


def pairs_of(spec):
    """Index pairs (first, second) of the rotated elements."""
    o, r = spec.opts.offset, spec.rot_dim
    if spec.opts.layout == B.GBO_ROPE_HALF:
        a = torch.arange(r // 2) + o
        return a, a + r // 2
    a = 2 * torch.arange(r // 2) + o
    return a, a + 1


def turn64(x, pos, spec, sign=1.0):
    """x (batch, seq, heads, dim) in 64 bits, rotated; with the size of each element's terms."""
    x = x.double().cpu()
    f = torch.tensor(spec.frequencies, dtype=torch.float64)
    ang = (pos.double().cpu()[..., None] * f)[:, :, None]
    c, s = ang.cos() * spec.opts.magnitude, sign * ang.sin() * spec.opts.magnitude
    a, b = pairs_of(spec)
    y, size = x.clone(), x.abs().clone()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    both = (x[..., a].abs() + x[..., b].abs()) * max(1.0, spec.opts.magnitude)
    size[..., a], size[..., b] = both, both
    return y, size


def turn_size(size, spec):
    """Sizes of the terms of a rotated vector whose elements have sizes `size`."""
    a, b = pairs_of(spec)
    out = size.clone()
    both = (size[..., a] + size[..., b]) * max(1.0, spec.opts.magnitude)
    out[..., a], out[..., b] = both, both
    return out


def near(got, want, size, dtype):
    got = got.double().cpu()
    tol = 64 * U * size + (2.0 ** -8 * want.abs() if dtype == torch.bfloat16 else 0.0) + 1e-30
    assert torch.all((got - want).abs() <= tol), float(((got - want).abs() - tol).max())


def heads(gen, shape, dtype):
    return torch.randn(shape, generator=gen).to(dtype).cuda()


CASES = [
    # dim, rot, offset, layout, scaling, batch, seq, heads, dtype
    (128, 128, 0, "half", None, 2, 37, 5, torch.bfloat16),
    (128, 128, 0, "half", None, 2, 37, 5, torch.float32),
    (64, 64, 0, "interleaved", dict(kind="linear", factor=4.0), 1, 130, 3, torch.bfloat16),
    (192, 64, 128, "interleaved", dict(kind="yarn", factor=8.0, trained=4096.0, fast=32.0, slow=1.0), 1, 33, 4,
     torch.bfloat16),
    (192, 64, 128, "half", dict(kind="wavelength", factor=8.0, trained=8192.0, fast=4.0, slow=1.0), 3, 5, 2,
     torch.float32),
    (512, 512, 0, "half", dict(kind="ntk", factor=2.0), 1, 9, 2, torch.bfloat16),
    (512, 256, 128, "interleaved", None, 1, 9, 2, torch.float32),
    (72, 36, 4, "interleaved", None, 2, 11, 3, torch.float32),  # 8-byte chunks
    (72, 72, 0, "half", None, 2, 11, 3, torch.bfloat16),        # 8-byte chunks
    (72, 36, 36, "interleaved", None, 1, 70, 3, torch.bfloat16),  # 4-byte chunks
    (72, 72, 0, "interleaved", None, 1, 9, 2, torch.float32),
    (76, 20, 8, "half", None, 1, 9, 2, torch.bfloat16),         # 4-byte chunks, an odd number of them copied
    (504, 500, 4, "half", None, 1, 5, 2, torch.bfloat16),       # 4-byte chunks, several a lane
    (508, 508, 0, "interleaved", None, 1, 5, 2, torch.float32),
    (80, 20, 60, "half", None, 1, 7, 1, torch.bfloat16),
    (40, 24, 8, "half", None, 2, 3, 2, torch.bfloat16),     # an odd number of copied chunks
    (7, 2, 3, "half", None, 1, 5, 3, torch.bfloat16),       # odd head
    (1, 0, 0, "half", None, 1, 4, 2, torch.float32),        # nothing to rotate
    (511, 510, 1, "interleaved", None, 1, 3, 2, torch.float32),
    (128, 128, 0, "half", None, 1, 1, 20, torch.bfloat16),  # one token
]


@pytest.mark.parametrize("dim,rot,offset,layout,scaling,batch,seq,nh,dtype", CASES)
def test_rotary_and_inverse(dim, rot, offset, layout, scaling, batch, seq, nh, dtype):
    gen = torch.Generator().manual_seed(dim + seq)
    spec = layers.RotarySpec(dim, rot_dim=rot, offset=offset, layout=layout, scaling=scaling)
    x = heads(gen, (batch, seq, nh, dim), dtype)
    pos = torch.randint(-50, 100000, (batch, seq), generator=gen).cuda()
    near(layers.rotary(x, pos, spec), *turn64(x, pos, spec), dtype)
    near(layers.rotary(x, pos, spec, inverse=True), *turn64(x, pos, spec, -1.0), dtype)
    # in place, on 32-bit positions
    y = x.clone()
    layers.rotary(y, pos.int(), spec, out=y)
    assert torch.equal(y, layers.rotary(x, pos, spec))


@pytest.mark.parametrize("dim,rot,offset,layout,scaling,batch,seq,nh,dtype", CASES)
def test_norm_rotary_and_gradients(dim, rot, offset, layout, scaling, batch, seq, nh, dtype):
    gen = torch.Generator().manual_seed(2 * dim + seq)
    spec = layers.RotarySpec(dim, rot_dim=rot, offset=offset, layout=layout, scaling=scaling)
    eps = 1e-5
    nk = max(1, nh // 2)
    tensors = []
    for count in (nh, nk):
        x = heads(gen, (batch, seq, count, dim), dtype)
        dy = heads(gen, (batch, seq, count, dim), dtype)
        gain = (1 + 0.3 * torch.randn(dim, generator=gen)).cuda()
        tensors.append((x, dy, gain))
    (q, dq, gq), (k, dk, gk) = tensors
    pos = torch.randint(0, 5000, (batch, seq), generator=gen).cuda()
    out = layers.qk_norm_rotary(q, k, gq, gk, pos, spec, eps=eps)
    grads = layers.qk_norm_rotary_backward(dq, dk, q, k, gq, gk, pos, spec, eps=eps)
    for n, (x, dy, gain) in enumerate(tensors):
        X, g = x.double().cpu(), gain.double().cpu()
        rho = (X.square().mean(-1, keepdim=True) + eps).rsqrt()
        normed = X * rho * g
        want, _ = turn64(normed, pos, spec)
        near(out[n], want, turn_size(normed.abs(), spec), dtype)
        e, esize = turn64(dy, pos, spec, -1.0)
        u, w, wsize = X * rho, e * g, esize * g.abs()
        mean, msize = (w * u).mean(-1, keepdim=True), (wsize * u.abs()).mean(-1, keepdim=True)
        near(grads[n], rho * (w - u * mean), rho * (wsize + u.abs() * msize), dtype)
        terms = x.numel() // dim
        dg, dgsize = (e * u).sum((0, 1, 2)), (esize * u.abs()).sum((0, 1, 2))
        assert torch.all((grads[2 + n].double().cpu() - dg).abs() <= (terms + 64 + 64) * U * dgsize + 1e-30)


def test_many_tokens_share_a_block():
    """Enough tokens that a group walks over several heads and a block over
    several rounds; dgain is the same bits twice."""
    gen = torch.Generator().manual_seed(5)
    spec = layers.RotarySpec(64)
    q, k = heads(gen, (2, 4099, 12, 64), torch.bfloat16), heads(gen, (2, 4099, 5, 64), torch.bfloat16)
    dq, dk = heads(gen, q.shape, torch.bfloat16), heads(gen, k.shape, torch.bfloat16)
    g = torch.ones(64, device="cuda")
    pos = torch.arange(4099, device="cuda")
    yq, yk = layers.qk_norm_rotary(q, k, g, g, pos, spec, eps=1e-6)
    for x, y in ((q, yq), (k, yk)):
        X = x.double().cpu()
        normed = X * (X.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
        near(y, turn64(normed, pos[None].expand(2, -1), spec)[0], turn_size(normed.abs(), spec), torch.bfloat16)
    a = layers.qk_norm_rotary_backward(dq, dk, q, k, g, g, pos, spec)
    b = layers.qk_norm_rotary_backward(dq, dk, q, k, g, g, pos, spec)
    for s, t in zip(a, b):
        assert torch.equal(s, t)
    for x, dy, dx, dg in ((q, dq, a[0], a[2]), (k, dk, a[1], a[3])):
        X = x.double().cpu()
        rho = (X.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
        e, esize = turn64(dy, pos[None].expand(2, -1), spec, -1.0)
        u = X * rho
        near(dx, rho * (e - u * (e * u).mean(-1, keepdim=True)),
             rho * (esize + u.abs() * (esize * u.abs()).mean(-1, keepdim=True)), torch.bfloat16)
        terms = x.numel() // 64
        assert torch.all((dg.double().cpu() - (e * u).sum((0, 1, 2))).abs()
                         <= (terms + 128) * U * (esize * u.abs()).sum((0, 1, 2)))


def test_gradient_against_differences():
    """Directional differences of the 64-bit formula match the gradients' inner products."""
    gen = torch.Generator().manual_seed(9)
    spec = layers.RotarySpec(32, rot_dim=16, offset=8, layout="interleaved")
    q, dq = heads(gen, (1, 6, 2, 32), torch.float32), heads(gen, (1, 6, 2, 32), torch.float32)
    gain = (1 + 0.3 * torch.randn(32, generator=gen)).cuda()
    pos = torch.arange(6)[None].cuda()
    dx, _, dg, _ = layers.qk_norm_rotary_backward(dq, dq, q, q, gain, gain, pos, spec, eps=1e-6)

    def objective(X, g):
        y, _ = turn64(X * (X.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * g, pos, spec)
        return (y * dq.double().cpu()).sum()

    X, g, h = q.double().cpu(), gain.double().cpu(), 1e-5
    dirx, dirg = torch.randn(X.shape, generator=gen).double(), torch.randn(32, generator=gen).double()
    numx = (objective(X + h * dirx, g) - objective(X - h * dirx, g)) / (2 * h)
    numg = (objective(X, g + h * dirg) - objective(X, g - h * dirg)) / (2 * h)
    # the differences' own error: h^2 times third derivatives, ~1e-9 here
    assert abs(numx - (dx.double().cpu() * dirx).sum()) <= 1e-5 * dx.norm().item() * dirx.norm()
    assert abs(numg - (dg.double().cpu() * dirg).sum()) <= 1e-5 * dg.norm().item() * dirg.norm()


def test_long_positions_are_exact():
    """The angle keeps its accuracy far beyond 2^24 and 2^31 (positions that fp32 does
    not hold), and for negative positions."""
    spec = layers.RotarySpec(16, frequencies=[0.5, 0.25, 1.0, 0.125, 0.0625, 2.0 ** -10, 1e-3, 0.3])
    x = torch.randn(1, 5, 1, 16, device="cuda")
    values = [2 ** 24 + 1, 2 ** 31 + 3, 2 ** 40 + 12345, -(2 ** 33) - 7, -1]
    pos = torch.tensor([values], device="cuda")
    got = layers.rotary(x, pos, spec).double().cpu()
    X = x.double().cpu()
    for s, t in enumerate(values):
        for j, f in enumerate(spec.frequencies):
            # the reduction in exact rationals: the 64-bit turn has the rounding of f / 2 pi to a
            # double (2^-53 relative) times t
            from fractions import Fraction
            import math
            turns = Fraction(t) * Fraction(f / (2 * math.pi))
            frac = float(turns - math.floor(turns))
            c, sn = math.cos(2 * math.pi * frac), math.sin(2 * math.pi * frac)
            a, b = X[0, s, 0, j].item(), X[0, s, 0, j + 8].item()
            assert abs(got[0, s, 0, j].item() - (a * c - b * sn)) <= 64 * U * (abs(a) + abs(b))
            assert abs(got[0, s, 0, j + 8].item() - (a * sn + b * c)) <= 64 * U * (abs(a) + abs(b))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_and_layouts(dtype):
    """Slices of a fused projection, (batch, heads, seq, dim) storage, a base off
    its 16-byte boundary, and positions shared by the batch: the same bits as
    contiguous tensors."""
    gen = torch.Generator().manual_seed(3)
    spec = layers.RotarySpec(64)
    gain = torch.ones(64, device="cuda")
    qkv = heads(gen, (2, 19, 7, 64), dtype)
    pos = torch.arange(19, device="cuda")
    q, k = qkv[:, :, :4], qkv[:, :, 4:6]
    a = layers.qk_norm_rotary(q, k, gain, gain, pos, spec)
    b = layers.qk_norm_rotary(q.contiguous(), k.contiguous(), gain, gain, pos[None].expand(2, 19), spec)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    swapped = q.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(layers.rotary(swapped, pos, spec), layers.rotary(q.contiguous(), pos, spec))
    for off in (1, 2, 4):  # an element, 4 or 8 bytes, 8 or 16 bytes behind a 16-byte boundary
        odd = torch.empty(q.numel() + off, dtype=dtype, device="cuda")[off:].view(q.shape)
        odd.copy_(q)
        near(layers.rotary(odd, pos, spec), *turn64(q, pos[None].expand(2, 19), spec), dtype)
        got = layers.qk_norm_rotary(odd, k, gain, gain, pos, spec)[0]
        assert torch.allclose(got.float(), a[0].float(), rtol=2.0 ** -7 if dtype == torch.bfloat16 else 1e-5, atol=1e-6)
    # the start as a number
    assert torch.equal(layers.rotary(q, 11, spec), layers.rotary(q, pos + 11, spec))


def test_empty_and_zero_rows():
    spec = layers.RotarySpec(64)
    g = torch.ones(64, device="cuda")
    empty = torch.empty(2, 0, 3, 64, device="cuda")
    assert layers.rotary(empty, 0, spec).shape == empty.shape
    dq, dk, dgq, dgk = layers.qk_norm_rotary_backward(empty, empty, empty, empty, g, g, 0, spec)
    assert torch.all(dgq == 0) and torch.all(dgk == 0)
    # a head of zeros: finite with eps > 0
    z = torch.zeros(1, 2, 1, 64, device="cuda")
    yq, _ = layers.qk_norm_rotary(z, z, g, g, 0, spec, eps=1e-6)
    assert torch.all(yq == 0)
    dq, _, dgq, _ = layers.qk_norm_rotary_backward(torch.ones_like(z), torch.ones_like(z), z, z, g, g, 0, spec, eps=1e-6)
    assert torch.isfinite(dq).all() and torch.all(dgq == 0)


def test_nan_stays_in_its_head():
    spec = layers.RotarySpec(64)
    x = torch.randn(1, 3, 2, 64, device="cuda")
    x[0, 1, 0, 5] = float("nan")
    g = torch.ones(64, device="cuda")
    y, _ = layers.qk_norm_rotary(x, x, g, g, 0, spec)
    assert torch.isnan(y[0, 1, 0]).all()
    y[0, 1, 0] = 0
    assert torch.isfinite(y).all()


def test_stream_and_graph():
    """On a stream of the caller's, and captured once and replayed on new data."""
    spec = layers.RotarySpec(128)
    x = torch.randn(1, 64, 4, 128, device="cuda", dtype=torch.bfloat16)
    pos = torch.arange(64, device="cuda")
    want = layers.rotary(x, pos, spec)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = torch.empty_like(x)
    B.gbo_rope_forward([dict(x=x, y=y)], spec.opts, pos, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layers.rotary(x, pos, spec, out=y)
    x.copy_(torch.randn_like(x))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, layers.rotary(x, pos, spec))


def test_autograd():
    spec = layers.RotarySpec(32)
    x = torch.randn(1, 8, 2, 32, device="cuda", requires_grad=True)
    y = layers.rotary_autograd(x, 3, spec)
    dy = torch.randn_like(y)
    y.backward(dy)
    assert torch.equal(x.grad, layers.rotary(dy, 3, spec, inverse=True))
    q, k = (torch.randn(1, 8, n, 32, device="cuda", requires_grad=True) for n in (2, 1))
    gq, gk = (torch.ones(32, device="cuda", requires_grad=True) for _ in range(2))
    yq, yk = layers.qk_norm_rotary_autograd(q, k, gq, gk, 0, spec)
    (yq.square().sum() + yk.sum()).backward()
    want = layers.qk_norm_rotary_backward(2 * yq.detach(), torch.ones_like(yk), q.detach(), k.detach(), gq.detach(),
                                          gk.detach(), 0, spec)
    for got, w in zip((q.grad, k.grad, gq.grad, gk.grad), want):
        assert torch.equal(got, w)


def test_workspace_refused_when_small():
    spec = layers.RotarySpec(32)
    x = torch.randn(1, 8, 2, 32, device="cuda")
    g = torch.ones(32, device="cuda")
    table = [dict(x=x, dy=x, y=torch.empty_like(x), gain=g, dgain=torch.empty_like(g), norm=True)]
    need = B.gbo_rope_workspace_bytes(table, spec.opts)
    assert need > 0
    for ws in (None, torch.empty(need - 4, dtype=torch.uint8, device="cuda")):
        with pytest.raises(B.GboError) as e:
            B.gbo_rope_backward(table, spec.opts, 0, ws)
        assert e.value.code == -6
    assert ctypes.sizeof(B.RopeTensor) == B.gbo_struct_size(8)


def test_scratch_of_one_gain_among_other_heads():
    """One spec, a gain of the queries alone, and keys of fewer heads than the call
    before: the scratch is sized for this call's heads, not the last one's."""
    spec = layers.RotarySpec(64)
    gq = torch.ones(64, device="cuda")
    for kv in (16, 4, 1, 8):
        q, k = torch.randn(1, 900, 4, 64, device="cuda"), torch.randn(1, 900, kv, 64, device="cuda")
        dq, dk, dgq, dgk = layers.qk_norm_rotary_backward(q, k, q, k, gq, None, 0, spec)
        alone = layers.RotarySpec(64)
        want = layers.qk_norm_rotary_backward(q, k, q, k, gq, None, 0, alone)
        assert dgk is None and torch.equal(dgq, want[2])
        assert torch.equal(dq, want[0]) and torch.equal(dk, want[1])


def test_positions_changed_before_the_backward_pass_are_noticed():
    spec = layers.RotarySpec(32)
    q, k = (torch.randn(1, 8, n, 32, device="cuda", requires_grad=True) for n in (2, 1))
    pos = torch.arange(8, device="cuda")
    y = layers.rotary_autograd(q, pos, spec)
    yq, yk = layers.qk_norm_rotary_autograd(q, k, None, None, pos, spec)
    y.sum().backward(retain_graph=True)  # unchanged: taken
    pos += 1
    with pytest.raises(RuntimeError):
        y.sum().backward()
    with pytest.raises(RuntimeError):
        (yq.sum() + yk.sum()).backward()


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last tokens come out as in a call of their own."""
    seq, nh, dim = 140000, 120, 128
    assert seq * nh * dim > 2 ** 31
    spec = layers.RotarySpec(dim)
    x = torch.empty(1, seq, nh, dim, dtype=torch.bfloat16, device="cuda")
    x[:, :, 0] = 1.0
    x[:, :, 1:].copy_(torch.randn(1, 1, nh - 1, dim, device="cuda"))
    x[:, -9:].copy_(torch.randn(1, 9, nh, dim, device="cuda"))
    tail, k = x[:, -9:].clone(), torch.ones(1, seq, 1, dim, dtype=torch.bfloat16, device="cuda")
    start = 5
    y = layers.rotary(x, start, spec)
    assert torch.equal(y[:, -9:], layers.rotary(tail, start + seq - 9, spec))
    gain = torch.linspace(0.5, 1.5, dim, device="cuda")
    y, _ = layers.qk_norm_rotary(x, k, gain, None, start, spec)
    assert torch.equal(y[:, -9:], layers.qk_norm_rotary(tail, k[:, -9:], gain, None, start + seq - 9, spec)[0])
    dx = layers.qk_norm_rotary_backward(y, k, x, k, gain, None, start, spec)[0]
    want = layers.qk_norm_rotary_backward(y[:, -9:].clone(), k[:, -9:], tail, k[:, -9:], gain, None, start + seq - 9, spec)[0]
    assert torch.equal(dx[:, -9:], want)
