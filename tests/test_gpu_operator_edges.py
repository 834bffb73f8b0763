"""Corners of the rotary and cross-entropy operators that need a GPU: memory of the loss
in autograd, frequencies of either sign at long positions, in-place norms,
tables of three and four tensors, sweeps of rows over pieces of the vocabulary.

Tolerances are those of test_gpu_rotary.py and test_gpu_xent.py, derived there; where
another one is taken its reason stands beside it."""

import math
from fractions import Fraction

import pytest
import torch

from adamw_optimizer_step_gb300 import _binding as B
from adamw_optimizer_step_gb300 import layers
from tests.test_gpu_xent import U, Want, close, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from adamw_optimizer_step_gb300 import build
    build.build()
    B.lib()


# ---------------------------------------------------------------------------
# memory of the loss in autograd

# small tensors of a call (lse, totals, the mean, upstream)
SLACK = 1 << 16


def peak_of(call):
    """Bytes that the call asks for at its peak and holds afterwards, and what it returns.
    (The blocks that torch hands out for them may be up to 1 MB larger each.)"""
    held = lambda which: torch.cuda.memory_stats()["requested_bytes.all." + which]  # noqa: E731
    torch.cuda.synchronize()
    base = held("current")
    torch.cuda.reset_peak_memory_stats()
    kept = call()
    torch.cuda.synchronize()
    return held("peak") - base, held("current") - base, kept


def test_memory_of_the_loss():
    """Without gradients: the workspace of the losses alone, and the same losses.  With
    them: one workspace from the forward to the backward pass, given back after it
    although the loss is still held."""
    n, v, d = 500, 20011, 512
    H, W, y = inputs(n, v, d, 7, ignored=0.1)
    small, large = (B.gbo_xent_workspace_bytes(n, v, d, grad) for grad in (False, True))
    assert large > small + 2 * n * v  # the logits are kept
    H.requires_grad_()
    W.requires_grad_()
    want = Want(H.detach(), W.detach(), y)
    layers.linear_cross_entropy_loss(H, W, y)  # (first-call set-up is no part of it)
    with torch.no_grad():
        peak, _, loss = peak_of(lambda: layers.linear_cross_entropy_loss(H, W, y))
    assert peak <= small + SLACK
    close(loss, want.total / want.weight, want.total_tol / want.weight, torch.float32)

    def step():
        loss = layers.linear_cross_entropy_loss(H, W, y)
        loss.backward()
        return loss

    grads = 2 * (n + v) * d
    peak, left, loss = peak_of(step)
    assert large <= peak <= large + grads + SLACK
    assert left <= grads + SLACK and loss.grad_fn is not None


# ---------------------------------------------------------------------------
# angles

# more digits than any rational here needs
PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


@pytest.mark.parametrize("sign", [1, -1])
def test_angles_keep_their_bound(sign):
    """Against rationals with 80 digits of pi: beside the rounding of the pass (64 u of the
    pair, see test_gpu_rotary.py) the angle is off by at most |t| (2^-52 |f| + 2^-61), the
    bound that gbo.h states, for frequencies of either sign."""
    freq = [sign * f for f in (1.0, 0.3, 1e-2, 1e-3, 1e-4, 1e-8, 2.0 ** -40, 17.5)]
    spec = layers.RotarySpec(16, frequencies=freq)
    x = torch.randn(1, 6, 1, 16, generator=torch.Generator().manual_seed(4)).cuda()
    values = [1, 2 ** 24 + 1, 2 ** 31 + 3, 2 ** 40 + 12345, -(2 ** 33) - 7, 2 ** 52 + 1]
    got = layers.rotary(x, torch.tensor([values], device="cuda"), spec).double().cpu()
    for s, t in enumerate(values):
        for j, f in enumerate(freq):
            turns = Fraction(t) * Fraction(f) / (2 * PI)
            angle = 2 * math.pi * float(turns - math.floor(turns))
            c, sn = math.cos(angle), math.sin(angle)
            a, b = x[0, s, 0, j].item(), x[0, s, 0, j + 8].item()
            tol = (64 * U + abs(t) * (2.0 ** -52 * abs(f) + 2.0 ** -61)) * (abs(a) + abs(b))
            assert abs(got[0, s, 0, j].item() - (a * c - b * sn)) <= tol, (t, f)
            assert abs(got[0, s, 0, j + 8].item() - (a * sn + b * c)) <= tol, (t, f)


# ---------------------------------------------------------------------------
# rotary: in place with a norm, three and four tensors

def rotary_inputs(counts, dim, dtype, seed, batch=2, seq=67):
    gen = torch.Generator().manual_seed(seed)
    made = lambda *shape: torch.randn(*shape, generator=gen)  # noqa: E731
    return [(made(batch, seq, h, dim).to(dtype).cuda(), made(batch, seq, h, dim).to(dtype).cuda(),
             (1 + 0.3 * made(dim)).cuda()) for h in counts]


def backward(table, spec):
    ws = torch.empty(max(16, B.gbo_rope_workspace_bytes(table, spec.opts)), dtype=torch.uint8, device="cuda")
    B.gbo_rope_backward(table, spec.with_eps(1e-6), 11, ws)


# chunks of 16, 8 and 4 bytes and of one element
@pytest.mark.parametrize("dim,rot,offset", [(128, 64, 32), (72, 36, 4), (76, 20, 8), (7, 2, 3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place_with_a_norm(dim, rot, offset, dtype):
    """The output in the input's place, the input's gradient in the gradient's: the same bits."""
    spec = layers.RotarySpec(dim, rot_dim=rot, offset=offset)
    (x, dy, gain), = rotary_inputs((9,), dim, dtype, dim)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    B.gbo_rope_forward([dict(x=x, y=y, gain=gain, norm=True)], spec.with_eps(1e-6), 11)
    dgain, again = torch.empty_like(gain), torch.empty_like(gain)
    backward([dict(x=x, dy=dy, y=dx, gain=gain, dgain=dgain, norm=True)], spec)
    backward([dict(x=x, dy=dy, y=dy, gain=gain, dgain=again, norm=True)], spec)
    assert torch.equal(dy, dx) and torch.equal(again, dgain)
    B.gbo_rope_forward([dict(x=x, y=x, gain=gain, norm=True)], spec.with_eps(1e-6), 11)
    assert torch.equal(x, y)


@pytest.mark.parametrize("counts", [(6, 2, 1), (6, 2, 1, 3), (5, 0, 2, 1)])
@pytest.mark.parametrize("norm", [False, True])
def test_three_and_four_tensors(counts, norm):
    """Each tensor of a table as in a call of its own (its heads do not meet the others');
    the gains' gradients, whose order of summation depends on the table, by their bound."""
    spec = layers.RotarySpec(64, rot_dim=32, offset=16, layout="interleaved")
    tensors = rotary_inputs(counts, 64, torch.bfloat16, sum(counts))
    extra = (lambda gain: dict(gain=gain, norm=True)) if norm else (lambda gain: {})
    ys, dxs = [torch.empty_like(t[0]) for t in tensors], [torch.empty_like(t[0]) for t in tensors]
    B.gbo_rope_forward([dict(x=x, y=y, **extra(g)) for (x, _, g), y in zip(tensors, ys)], spec.with_eps(1e-6), 11)
    dgains = [torch.full((64,), float("nan"), device="cuda") for _ in tensors]
    table = [dict(x=x, dy=dy, y=dx, **extra(g)) for (x, dy, g), dx in zip(tensors, dxs)]
    if norm:
        for e, dg in zip(table, dgains):
            e["dgain"] = dg
        backward(table, spec)
    else:
        for e in table:
            del e["x"]
        B.gbo_rope_backward(table, spec.opts, 11)
    for (x, dy, gain), y, dx, dg in zip(tensors, ys, dxs, dgains):
        want, want_dx, one = torch.empty_like(x), torch.empty_like(x), torch.empty_like(gain)
        B.gbo_rope_forward([dict(x=x, y=want, **extra(gain))], spec.with_eps(1e-6), 11)
        assert torch.equal(y, want)
        if norm:
            backward([dict(x=x, dy=dy, y=want_dx, dgain=one, **extra(gain))], spec)
            # two sums of the same fp32 terms e_j u_j: either is off by at most (terms + 128) u of
            # the terms' sizes, which are within the pair's |dy| times |u|
            u = x.double() * (x.double().square().mean(-1, keepdim=True) + 1e-6).rsqrt()
            e = dy.double().abs()
            e[..., 16:48] = (e[..., 16:48:2] + e[..., 17:48:2]).repeat_interleave(2, -1)
            terms = x.numel() // 64
            assert torch.all((dg.double() - one.double()).abs()
                             <= 2 * (terms + 128) * U * (e * u.abs()).sum((0, 1, 2)) + 1e-30)
        else:
            B.gbo_rope_backward([dict(dy=dy, y=want_dx)], spec.opts, 11)
        assert torch.equal(dx, want_dx)


# ---------------------------------------------------------------------------
# cross entropy: sweeps of rows, pieces of the vocabulary, cuts of dH's axis

def schedule(n, v, d, piece_tiles):
    """(bytes, columns of a piece, pieces, cuts of dH's axis, columns of a cut) of a call whose
    pieces are `piece_tiles` tiles of 256 columns at most: the arithmetic of the
    workspace, which the tests below check against its size."""
    up = lambda x, m: (x + m - 1) // m * m  # noqa: E731
    rows = up(max(n, 1), 256)
    size = [up(x, 1024) for x in (16, 4 * rows // 256) + 6 * (4 * rows,) + (2 * rows * up(d, 64),)]
    part = 8 * rows * max(-(-v // 128), 1024 if n <= 32 else 0)
    pieces = -(-v // (256 * piece_tiles))
    piece = up(-(-v // pieces), 256)
    pieces = -(-v // piece)
    d_tiles, kit, dw_kit = -(-d // 256), -(-piece // 128), rows // 128
    share = max(1, (rows // 256 * d_tiles * kit + piece // 256 * d_tiles * (max(dw_kit, 5) + 1)) // 76)
    cut = -(-kit // min(16, max(1, kit // 8), -(-2 * kit // share)))
    cuts = -(-kit // cut)
    size.append(up(4 * cuts * rows * d, 1024) if pieces > 1 or cuts > 1 else 0)
    size.append(up(max(part, 2 * rows * (piece + 64)), 1024))
    return sum(size), piece, pieces, cuts, 128 * cut


def check_pieces(n, v, d, piece_tiles, seed):
    nbytes, piece, pieces, cuts, cut = schedule(n, v, d, piece_tiles)
    assert B.gbo_xent_workspace_bytes(n, v, d, True, nbytes) == nbytes < B.gbo_xent_workspace_bytes(n, v, d, True)
    H, W, y = inputs(n, v, d, seed, ignored=0.02)
    for k, edge in enumerate(e for c in range(1, pieces) for e in (c * piece - 1, c * piece)):
        y[3 * k] = edge  # labels on both sides of every seam
    y[0], y[-1] = 0, v - 1
    want = Want(H, W, y, z=1e-3)
    dh, dw = torch.full_like(H, float("nan")), torch.full_like(W, float("nan"))
    loss, _, _ = layers.linear_cross_entropy_grad(H, W, y, z_loss=1e-3, dh=dh, dw=dw, workspace_cap=nbytes)
    close(loss, want.loss, want.loss_tol, torch.float32)
    close(dh, want.dh, want.dh_tol, torch.bfloat16)
    close(dw, want.dw, want.dw_tol, torch.bfloat16)
    return piece, pieces, cuts, cut


def test_sweeps_of_rows_over_pieces_of_the_vocabulary():
    """More rows than one sweep takes (8192), three pieces and more."""
    _, pieces, _, _ = check_pieces(8500, 1030, 72, 1, 62)
    assert pieces >= 3


def test_a_last_piece_that_ends_before_the_last_cut():
    """Nine pieces, dH's axis cut in two: the last piece's 412 columns end before the second
    cut begins, and the sums over the pieces before it stay."""
    v = 82 * 256 - 100
    piece, pieces, cuts, cut = check_pieces(100, v, 64, 10, 63)
    assert pieces == 9 and cuts == 2 and v - (pieces - 1) * piece <= cut
