"""The residual update, its gradients and dropout against the formulas in 64 bits.

Tolerances, u = 2^-24, all of sizes (the same formula with every term's absolute
value).  A mean square over d elements is off by at most (d / 2 + 4) u of it, so a
norm's factor by (d / 4 + 6) u; a mean of products by (d + 4) u of its size.  The
sigmoid is off by (8 + 2 |a|) u of it (the exponential's argument and result), as is
its slope.  With a handful of multiplications on top, values are off by c u of their
size, c = 2 d + 64 + 8 max |a|, a sum over n rows by c + n.  A bf16 output adds 2^-8
of its value, an fp32 one u."""

import numpy as np
import pytest
import torch

from adamw_optimizer_step_gb300 import _binding as B
from adamw_optimizer_step_gb300 import layers

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    from adamw_optimizer_step_gb300 import build
    build.build()
    B.lib()


def draws(count, seed, offset):
    """The generator's 16-bit draws on the host, in Python's integers."""
    out, low = [], 0xFFFFFFFF
    for i in range((count + 7) // 8):
        a, b, c, d = i & low, i >> 32, offset & low, offset >> 32
        k0, k1 = seed & low, seed >> 32
        for _ in range(10):
            u, v = 0xD2511F53 * a, 0xCD9E8D57 * c
            a, b, c, d = (v >> 32) ^ b ^ k0, v & low, (u >> 32) ^ d ^ k1, u & low
            k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
        for w in (a, b, c, d):
            out += [w & 0xFFFF, w >> 16]
    return np.array(out[:count])


def mask_of(shape, p, seed, offset):
    limit = round(65536 * p)
    keep = draws(int(np.prod(shape)), seed % (1 << 64), offset % (1 << 64)) >= limit
    return torch.tensor(keep.reshape(shape) * (65536.0 / (65536 - limit)), dtype=torch.float64, device="cuda")


def test_the_generator_is_the_published_one():
    """Known answers of Philox 4x32-10: counter and key of zeros, of ones, of pi's digits."""
    assert [int(draws(8, 0, 0)[2 * k] + (draws(8, 0, 0)[2 * k + 1] << 16)) for k in range(4)] == [
        0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    # the kernel's element 0 under that key: draw 0xe8d5 is below 0.95 of 65536, not below 0.9
    one = torch.ones(8, device="cuda")
    for p, kept in ((0.95, 0), (0.9, 1)):
        assert bool(layers.dropout(one, p, 0)[0] != 0) == bool(kept)


@pytest.mark.parametrize("shape", [(1,), (7,), (8,), (9,), (33, 31), (5, 3, 16), (300, 65)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("p,seed,offset", [(0.5, 1, 0), (0.1, -1, 3), (0.0, 5, 5), (1.0 - 2.0 ** -16, 2 ** 63, 2 ** 40 + 1)])
def test_dropout(shape, dtype, p, seed, offset):
    x = torch.randn(shape, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    m = mask_of(shape, p, seed, offset)
    want = x.double() * m
    for s in (seed, torch.tensor([seed - (1 << 64) if seed >= 1 << 63 else seed], device="cuda")):
        y = layers.dropout(x, p, s, offset=offset)
        assert torch.equal(y != 0, (m != 0) & (x != 0))
        assert ((y.double() - want).abs() <= (2.0 ** -8 if dtype == BF16 else 4 * U) * want.abs()).all()
    z = x.clone()
    assert layers.dropout(z, p, seed, offset=offset, out=z) is z and torch.equal(z, y)


def test_dropout_of_strided_rows_and_misaligned_ones():
    base = torch.randn(40, 50, device="cuda")
    x = base[:, 3:34]
    y = layers.dropout(x, 0.3, 9)
    assert torch.equal(y, layers.dropout(x.contiguous(), 0.3, 9))
    out = torch.full((40, 50), 7.0, device="cuda")
    layers.dropout(x, 0.3, 9, out=out[:, 3:34])
    assert torch.equal(out[:, 3:34], y) and (out[:, :3] == 7).all() and (out[:, 34:] == 7).all()
    flat = torch.randn(1001, device="cuda")[1:]
    assert torch.equal(layers.dropout(flat, 0.3, 9), layers.dropout(flat.clone(), 0.3, 9))


def test_dropout_of_many_elements_and_its_gradient():
    x = torch.ones(3000, 1000, device="cuda", requires_grad=True)
    y = layers.dropout_autograd(x, 0.25, 123, offset=1)
    share = float((y != 0).double().mean())
    assert abs(share - 0.75) < 6 * (0.75 * 0.25 / 3e6) ** 0.5
    y.sum().backward()
    assert torch.equal(x.grad, y.detach())
    assert float((layers.dropout(x.detach(), 0.25, 123, offset=2) != y).double().mean()) > 0.3


def test_dropout_past_32_bits():
    """The counter of an element past 2^32, and of an offset past it."""
    n = (1 << 32) + 24
    x = torch.ones(n, dtype=BF16, device="cuda")
    y = layers.dropout(x, 0.5, 77, out=x)
    tail = y[-16:].cpu().double()

    def block(i):
        low, out = 0xFFFFFFFF, []
        a, b, c, d, k0, k1 = i & low, i >> 32, 0, 0, 77, 0
        for _ in range(10):
            u, v = 0xD2511F53 * a, 0xCD9E8D57 * c
            a, b, c, d = (v >> 32) ^ b ^ k0, v & low, (u >> 32) ^ d ^ k1, u & low
            k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
        for w in (a, b, c, d):
            out += [w & 0xFFFF, w >> 16]
        return out

    want = [2.0 * (d >= 32768) for i in ((n - 16) // 8, (n - 8) // 8) for d in block(i)]
    assert tail.tolist() == want
    del x, y


# ---------------------------------------------------------------------------
# residual update

class Case:
    """Inputs, and outputs and gradients in 64 bits with their sizes."""

    def __init__(self, n, d, xt=BF16, bt=BF16, post=True, pre=True, gate=None, kind="sigmoid", scale="vector", p=0.0, gains=True,
                 seed=0, eps=1e-6):
        g = torch.Generator().manual_seed(seed)
        made = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.n, self.d = n, d
        self.x, self.block = made(n, d).to(xt).cuda(), (0.5 * made(n, d)).to(bt).cuda()
        self.gate = None if gate is None else (2 * made(n, 1 if gate == "row" else d)).to(bt).cuda()
        self.scale = {None: None, "one": 0.3 + made(1), "vector": 0.3 + 0.2 * made(d)}[scale]
        self.scale = None if self.scale is None else self.scale.cuda()
        self.post_gain = (1 + 0.3 * made(d)).cuda() if post and gains else None
        self.pre_gain = (1 + 0.3 * made(d)).cuda() if pre and gains else None
        self.dx_out, self.dh = made(n, d).to(xt).cuda(), made(n, d).to(bt).cuda() if pre else None
        self.post, self.pre, self.p, self.seed, self.offset, self.eps, self.kind = post, pre, p, 3 * seed + 1, 7, eps, kind
        self.m = mask_of((n, d), p, self.seed, self.offset) if p else torch.ones(n, d, dtype=torch.float64, device="cuda")
        self.c = (2 * d + 64 + (8 * float(self.gate.float().abs().max()) if gate and n else 0)) * U

    def kw(self):
        return dict(post_norm=self.post, pre_norm=self.pre, post_gain=self.post_gain, pre_gain=self.pre_gain, gate=self.gate,
                    gate_kind=self.kind, scale=self.scale, dropout=self.p, seed=self.seed, offset=self.offset, eps=self.eps)

    def pieces(self):
        D = lambda t, other=1.0: other if t is None else t.double()  # noqa: E731
        o = self.block.double()
        ro = 1 / (o.square().mean(-1, keepdim=True) + self.eps).sqrt() if self.post else 1.0
        v = o * ro
        a = D(self.gate)
        if self.gate is None:
            f, slope = 1.0, 0.0
        elif self.kind == "sigmoid":
            f = torch.sigmoid(a)
            slope = f * torch.sigmoid(-a)
        else:
            f, slope = a, torch.ones_like(a)
        return o, ro, v, f, slope, D(self.scale), D(self.post_gain), D(self.pre_gain)

    def forward(self):
        """{name: (value, size)}"""
        o, ro, v, f, _, s, gp, gq = self.pieces()
        part = s * f * self.m * v * gp
        x, size = self.x.double() + part, self.x.double().abs() + part.abs()
        out = dict(x=(x, size))
        if self.pre:
            r = 1 / (x.square().mean(-1, keepdim=True) + self.eps).sqrt()
            out["h"] = (x * r * gq, (size * r * gq).abs() + (x * r * gq).abs() * (size.square().mean(-1, keepdim=True) * r ** 2))
        return out

    def backward(self, x_new, dx_out=True):
        o, ro, v, f, slope, s, gp, gq = self.pieces()
        g = self.dx_out.double() if dx_out else torch.zeros_like(self.m)
        size, out = g.abs(), {}
        if self.pre:
            x, dh = x_new.double(), self.dh.double()
            r = 1 / (x.square().mean(-1, keepdim=True) + self.eps).sqrt()
            nrm, w = x * r, dh * gq
            out["dpre_gain"] = ((dh * nrm).sum(0), (dh * nrm).abs().sum(0))
            g = g + r * (w - nrm * (w * nrm).mean(-1, keepdim=True))
            size = size + r * (w.abs() + nrm.abs() * (w * nrm).abs().mean(-1, keepdim=True))
        out["dx"] = (g, size)
        gm, sm = g * self.m, size * self.m
        t, ts = gm * f * v * gp, (sm * f * v * gp).abs()
        if self.scale is not None:
            one = self.scale.numel() == 1
            out["dscale"] = (t.sum().view(1), ts.sum().view(1)) if one else (t.sum(0), ts.sum(0))
        if self.gate is not None:
            t, ts = gm * s * v * gp * slope, (sm * s * v * gp * slope).abs()
            row = self.gate.shape[1] == 1
            out["dgate"] = (t.sum(1, keepdim=True), ts.sum(1, keepdim=True)) if row else (t, ts)
        du, dus = gm * s * f, (sm * s * f).abs()
        if self.post_gain is not None:
            out["dpost_gain"] = ((du * v).sum(0), (dus * v).abs().sum(0))
        if self.post:
            w, ws = du * gp, dus * torch.as_tensor(gp).abs()
            du = ro * (w - v * (w * v).mean(-1, keepdim=True))
            dus = ro * (ws + v.abs() * (ws * v).abs().mean(-1, keepdim=True))
        out["dblock"] = (du, dus)
        return {k: z for k, z in out.items() if k != "dpre_gain" or self.pre_gain is not None}

    def near(self, got, want, what):
        value, size = want
        assert got.shape == value.shape and torch.isfinite(got).all(), what
        c = self.c + (self.n * U if what in ("dscale", "dpost_gain", "dpre_gain") else 0)
        if what == "dscale" and got.numel() == 1 and self.d > 1:
            c += self.d * U
        tol = c * size + (2.0 ** -8 if got.dtype == BF16 else U) * (value.abs() + c * size) + 1e-30
        off = ((got.double() - value).abs() - tol).max() if got.numel() else torch.tensor(0.0)
        assert off <= 0, (what, float(off))

    def check(self, **more):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        x_new, h = layers.residual_norm(self.x, self.block, dev_status=status, **self.kw())
        want = self.forward()
        self.near(x_new, want["x"], "x")
        assert (h is None) == (not self.pre)
        if self.pre:
            self.near(h, want["h"], "h")
        grads = layers.residual_norm_backward(self.dx_out, self.dh, x_new, self.block, dev_status=status, **self.kw())
        want = self.backward(x_new)
        assert {k for k, t in grads.items() if t is not None} == set(want)
        for k, z in want.items():
            self.near(grads[k], z, k)
        assert int(status.item()) == 0
        return x_new, h, grads


TYPES = [(BF16, BF16), (F32, BF16), (F32, F32)]
# widths below a warp's groups, of one chunk, odd ones, of every way through the kernels:
# groups within a warp, direct rows, the ring with one and two chunks a thread
WIDTHS = [1, 5, 8, 24, 72, 100, 256, 509, 512, 520, 1031, 2048, 2056, 4104, 5000, 8192, 8200, 16384]


@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(x)[6:] for x in t))
@pytest.mark.parametrize("d", WIDTHS)
def test_widths(d, types):
    n = 37 if d < 4000 else 5
    Case(n, d, *types, gate="element", p=0.25 if d < 600 else 0.0, seed=d).check()
    Case(n, d, *types, gate="row", kind="linear", scale="one", seed=d + 1).check()


# rows of single elements through the ring (from 505 elements to 8192) with one and two
# chunks a thread, and rows that no ring has room for, with chunks and single elements
ODD_AND_WIDE = [505, 513, 1030, 2051, 4097, 6001, 8191, 8193, 12288, 12291, 16383]


@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(x)[6:] for x in t))
@pytest.mark.parametrize("d", ODD_AND_WIDE)
def test_odd_and_wide_rows(d, types):
    Case(5, d, *types, gate="element", p=0.25, seed=d).check()
    Case(400 if d < 3000 else 3, d, *types, gate="row", scale="one", seed=d + 1).check()
    Case(4, d, *types, post=False, scale=None, seed=d + 2).check()
    Case(4, d, *types, pre=False, p=0.1, seed=d + 3).check()


@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(x)[6:] for x in t))
@pytest.mark.parametrize("d,stride", [(1024, 1024), (1023, 1023), (1027, 1030), (4104, 4109)])
@pytest.mark.parametrize("n", [1, 2, 9])
def test_rows_that_start_and_end_anywhere(n, d, stride, types):
    """Tensors that start and end inside a 16-byte block, with NaN around and between their rows."""
    c = Case(n, d, *types, gate="element", p=0.1, seed=n)
    at = [0]

    def placed(t):
        at[0] += 1
        flat = torch.full((at[0] + (n - 1) * stride + d + 9,), float("nan"), dtype=t.dtype, device="cuda")
        out = flat[at[0]:at[0] + (n - 1) * stride + d].as_strided((n, d), (stride, 1))
        out.copy_(t)
        return out

    for name in ("x", "block", "gate", "dx_out", "dh"):
        setattr(c, name, placed(getattr(c, name)))
    x, _, _ = c.check()
    want = c.backward(x)
    got = layers.residual_norm_backward(c.dx_out, c.dh, placed(x), c.block, **c.kw())
    for k, z in want.items():
        c.near(got[k], z, k)


@pytest.mark.parametrize("d", [64, 77, 1024])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("gate", [None, "row", "element"])
@pytest.mark.parametrize("scale", [None, "one", "vector"])
def test_every_combination(d, post, pre, gate, scale):
    Case(21, d, post=post, pre=pre, gate=gate, scale=scale, kind="linear" if d == 77 else "sigmoid", gains=d != 64, p=0.1,
         seed=2).check()


@pytest.mark.parametrize("n", [1, 2, 3, 33, 1000, 5000])
@pytest.mark.parametrize("d", [16, 520])
def test_numbers_of_rows(n, d):
    Case(n, d, F32, F32, gate="element", seed=n).check()


def test_the_norm_alone():
    for d in (8, 100, 1024):
        c = Case(19, d, post=False, seed=3)
        x, h = layers.residual_norm(c.x, pre_gain=c.pre_gain)
        assert x is c.x
        r = 1 / (c.x.double().square().mean(-1, keepdim=True) + 1e-6).sqrt()
        want = c.x.double() * r * c.pre_gain.double()
        c.near(h, (want, want.abs()), "h")
        g = layers.residual_norm_backward(None, c.dh, c.x, pre_gain=c.pre_gain)
        assert {k for k, t in g.items() if t is not None} == {"dx", "dpre_gain"}
        nrm, w = c.x.double() * r, c.dh.double() * c.pre_gain.double()
        mean = (w * nrm).mean(-1, keepdim=True)
        c.near(g["dx"], (r * (w - nrm * mean), r * (w.abs() + nrm.abs() * (w * nrm).abs().mean(-1, keepdim=True))), "dx")
        c.near(g["dpre_gain"], ((c.dh.double() * nrm).sum(0), (c.dh.double() * nrm).abs().sum(0)), "dpre_gain")


def test_dropout_here_is_dropout_alone():
    """One update with dropout, and the same from dropout's own call: the same elements."""
    for d in (40, 77, 2048):
        c = Case(11, d, F32, F32, post=False, pre=False, scale=None, p=0.5, seed=4)
        x, _ = layers.residual_norm(torch.zeros_like(c.x), c.block, **c.kw())
        assert torch.equal(x, layers.dropout(c.block, 0.5, c.seed, offset=c.offset))


def test_extremes():
    """Gates far out (nothing overflows, slopes do not cancel), rows of zeros, a NaN that stays
    in its row."""
    c = Case(8, 1024, F32, F32, gate="element", seed=5)
    c.gate[0] = 200.0
    c.gate[1] = -200.0
    c.gate[2] = 20.0
    c.gate[3] = -20.0
    c.c = (2 * 1024 + 64 + 8 * 200) * U
    c.block[4] = 0
    c.x[5] = 0
    c.block[5] = 0
    x, h, grads = c.check()
    clean = [t.clone() for t in (x, h, grads["dx"], grads["dblock"])]
    c.block[6, 3] = float("nan")
    x, h = layers.residual_norm(c.x, c.block, **c.kw())
    g = layers.residual_norm_backward(c.dx_out, c.dh, clean[0], c.block, **c.kw())
    others = [0, 1, 2, 3, 4, 5, 7]
    for a, b in zip((x, h, g["dx"], g["dblock"]), clean):
        assert torch.equal(a[others], b[others])
    assert torch.isnan(x[6]).any() and torch.isnan(h[6]).all()


@pytest.mark.parametrize("d", [64, 1024, 1027])
def test_strides_and_in_place(d):
    c = Case(13, d, gate="element", seed=6)
    x, h, grads = c.check()
    wide = lambda t: torch.nn.functional.pad(t, (8, 16))[:, 8:8 + d]  # noqa: E731
    kw = c.kw()
    kw["gate"] = wide(c.gate)
    x2, h2 = layers.residual_norm(wide(c.x), wide(c.block), **kw)
    # other strides may take another path through the kernels: the same values to their rounding
    want = c.forward()
    c.near(x2, want["x"], "x")
    c.near(h2, want["h"], "h")
    z = c.x.clone()
    y, h3 = layers.residual_norm(z, c.block, x_out=z, **c.kw())
    assert y.data_ptr() == z.data_ptr() and torch.equal(z, x) and torch.equal(h3, h)
    g = layers.residual_norm_backward(wide(c.dx_out), wide(c.dh), wide(x), wide(c.block), **kw)
    for k, t in c.backward(x).items():
        c.near(g[k], t, k)
    x4, h4 = layers.residual_norm(c.x.view(1, 13, 1, d), c.block.view(1, 13, 1, d), **dict(c.kw(), gate=c.gate.view(1, 13, 1, d)))
    assert x4.shape == (1, 13, 1, d) and torch.equal(x4.view(13, d), x) and torch.equal(h4.view(13, d), h)


def test_results_repeat_bit_for_bit():
    for d in (72, 2048):
        c = Case(3000, d, gate="element", p=0.1 if d == 72 else 0.0, seed=7)
        x, h = layers.residual_norm(c.x, c.block, **c.kw())
        first = layers.residual_norm_backward(c.dx_out, c.dh, x, c.block, **c.kw())
        for _ in range(3):
            g = layers.residual_norm_backward(c.dx_out, c.dh, x, c.block, **c.kw())
            assert all(torch.equal(g[k], first[k]) for k in first)


def test_gradients_against_differences():
    """sum dx_out x' + dh h by differences of the formula in 64 bits, for each input."""
    c = Case(9, 40, F32, F32, gate="element", p=0.2, seed=8)
    x_new, h, grads = c.check()
    gen = torch.Generator().manual_seed(1)
    for name, field in (("dx", "x"), ("dblock", "block"), ("dgate", "gate"), ("dscale", "scale"), ("dpost_gain", "post_gain"),
                        ("dpre_gain", "pre_gain")):
        t = getattr(c, field)
        step = torch.randn(t.shape, generator=gen).cuda().double()

        def objective(e):
            setattr(c, field, t.double() + e * step)
            f = c.forward()
            setattr(c, field, t)
            return float((f["x"][0] * c.dx_out.double()).sum() + (f["h"][0] * c.dh.double()).sum())

        slope = (objective(1e-5) - objective(-1e-5)) / 2e-5
        got = float((grads[name].double() * step).sum())
        size = float((c.backward(x_new)[name][1] * step.abs()).sum())
        assert abs(got - slope) <= (c.c + 2 * U + c.n * U) * size + 1e-7 * abs(slope) + 1e-8, (name, got, slope)


def test_autograd():
    c = Case(30, 96, F32, BF16, gate="row", p=0.3, seed=9)
    leaves = [t.requires_grad_() for t in (c.x, c.block, c.gate, c.scale, c.post_gain, c.pre_gain)]
    seed = torch.tensor([c.seed], device="cuda")
    kw = dict(c.kw(), seed=seed)
    x, h = layers.residual_norm_autograd(c.x, c.block, **kw)
    torch.autograd.backward((x, h), (c.dx_out, c.dh))
    for t, name in zip(leaves, ("dx", "dblock", "dgate", "dscale", "dpost_gain", "dpre_gain")):
        assert t.grad.shape == t.shape and t.grad.dtype == t.dtype
        c.near(t.grad, c.backward(x.detach())[name], name)
    # only h, only x', expanded gradients
    for which in (0, 1):
        for t in leaves:
            t.grad = None
        out = layers.residual_norm_autograd(c.x, c.block, **kw)
        out[which].sum().backward()
        c.dx_out, c.dh = torch.ones_like(c.dx_out), torch.ones_like(c.dh)
        if which == 0:
            pre, gain, c.pre, c.pre_gain = c.pre, c.pre_gain, False, None
            c.near(leaves[0].grad, c.backward(x.detach())["dx"], "dx")
            c.near(leaves[1].grad, c.backward(x.detach())["dblock"], "dblock")
            assert leaves[5].grad is None
            c.pre, c.pre_gain = pre, gain
        else:
            c.near(leaves[0].grad, c.backward(x.detach(), dx_out=False)["dx"], "dx")
            c.near(leaves[5].grad, c.backward(x.detach(), dx_out=False)["dpre_gain"], "dpre_gain")
    # a seed that changes before the backward pass is noticed
    x, h = layers.residual_norm_autograd(c.x, c.block, **kw)
    seed += 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        h.sum().backward()
    # the norm alone
    y, h = layers.residual_norm_autograd(c.x, pre_gain=c.pre_gain)
    assert y is c.x
    h.sum().backward()
    assert torch.isfinite(c.x.grad).all()


def test_stream_and_graph():
    """Captured with the seed on the device: each replay draws with the seed it finds."""
    c = Case(50, 1024, gate="element", p=0.5, seed=10)
    seed = torch.tensor([c.seed], device="cuda")
    kw = dict(c.kw(), seed=seed)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x, h = layers.residual_norm(c.x, c.block, **kw)
        g = layers.residual_norm_backward(c.dx_out, c.dh, x, c.block, **kw)
        y = layers.dropout(c.x, 0.5, seed)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gx, gh = layers.residual_norm(c.x, c.block, **kw)
        gg = layers.residual_norm_backward(c.dx_out, c.dh, gx, c.block, **kw)
        gy = layers.dropout(c.x, 0.5, seed)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(gx, x) and torch.equal(gh, h) and torch.equal(gy, y) and all(torch.equal(gg[k], g[k]) for k in g)
    seed += 5
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(gy, layers.dropout(c.x, 0.5, c.seed + 5)) and not torch.equal(gy, y)
    c.seed += 5
    c.m = mask_of((50, 1024), 0.5, c.seed, c.offset)
    for k, t in c.backward(gx).items():
        c.near(gg[k], t, k)


def test_nothing_to_do():
    c = Case(0, 64, gate="element", seed=11)
    x, h = layers.residual_norm(c.x, c.block, **c.kw())
    g = layers.residual_norm_backward(c.dx_out, c.dh, x, c.block, **c.kw())
    assert x.shape == h.shape == (0, 64) and not g["dpre_gain"].any() and not g["dscale"].any()
    assert layers.dropout(torch.empty(0, 5, device="cuda"), 0.5, 1).shape == (0, 5)
    assert layers.dropout(torch.empty(3, 0, device="cuda"), 0.5, 1).shape == (3, 0)


def test_offsets_past_32_bits():
    """Rows that begin past 2^31 elements."""
    step, n = 1 << 25, 66
    flat = torch.empty(step * n, dtype=BF16, device="cuda")
    for d in (1024, 100):
        c = Case(n, d, gate="element", seed=12)
        block = flat.as_strided((n, d), (step, 1))
        block.copy_(c.block)
        x, h = layers.residual_norm(c.x, block, **c.kw())
        want = c.forward()
        c.near(x, want["x"], "x")
        c.near(h, want["h"], "h")
        g = layers.residual_norm_backward(c.dx_out, c.dh, x, block, **c.kw())
        for k, t in c.backward(x).items():
            c.near(g[k], t, k)
    del flat


def test_workspace_refused_when_small():
    c = Case(40, 128, seed=13)
    x, h = layers.residual_norm(c.x, c.block, **c.kw())
    args = B.residual_args(x, c.block, **{k: v for k, v in c.kw().items()})
    need = B.gbo_residual_workspace_bytes(40, 128, 1)
    out = torch.empty(128, device="cuda")
    for ws in (None, torch.empty(need - 1, dtype=torch.uint8, device="cuda"), torch.empty(need + 8, dtype=torch.uint8, device="cuda")[8:]):
        with pytest.raises(B.GboError, match="workspace"):
            B.gbo_residual_backward(args, ws, (40, 128), BF16, BF16, dx_out=c.dx_out, dh=c.dh, dpre_gain=out)


def test_tensors_of_another_device_are_refused(monkeypatch):
    """Where the current device is another one than the tensors' (here: as the binding sees it)."""
    c = Case(4, 64)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    for call in (lambda: layers.residual_norm(c.x, c.block, **c.kw()), lambda: layers.dropout(c.x, 0.5, 1),
                 lambda: layers.residual_norm_backward(c.dx_out, c.dh, c.x, c.block, **c.kw())):
        with pytest.raises(ValueError, match="on the current device"):
            call()


@pytest.mark.parametrize("d", [64, 77, 1023, 1024, 6144, 8199, 12288])
@pytest.mark.parametrize("post", [True, False])
def test_outputs_in_the_places_of_inputs(d, post):
    """x' over x and h over the block's output; dx over dx_out and dblock over dh: the same bits."""
    c = Case(700 if d < 2000 else 5, d, gate="element", post=post, seed=9)
    x, h = layers.residual_norm(c.x, c.block, **c.kw())
    want = layers.residual_norm_backward(c.dx_out, c.dh, x, c.block, **c.kw())
    shape = (c.n, d)
    args = B.residual_args(c.x, c.block, **c.kw())
    x_in, block_in = c.x.clone(), c.block.clone()
    B.gbo_residual_forward(args, c.x, c.block, shape, BF16, BF16)
    assert torch.equal(c.x, x) and torch.equal(c.block, h)
    c.x, c.block = x_in, block_in
    args = B.residual_args(x, c.block, **c.kw())
    sums = {k: torch.empty_like(want[k]) for k in ("dscale", "dpost_gain", "dpre_gain") if want[k] is not None}
    ws = torch.empty(B.gbo_residual_workspace_bytes(c.n, d, len(sums)), dtype=torch.uint8, device="cuda")
    dgate = torch.empty_like(c.gate)
    B.gbo_residual_backward(args, ws, shape, BF16, BF16, dx_out=c.dx_out, dh=c.dh, dx=c.dx_out, dblock=c.dh, dgate=dgate, **sums)
    assert torch.equal(c.dx_out, want["dx"]) and torch.equal(c.dh, want["dblock"]) and torch.equal(dgate, want["dgate"])
    for k, t in sums.items():
        assert torch.equal(t, want[k])
