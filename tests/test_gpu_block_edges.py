"""Attention, the residual update and dropout at the edges of what their arguments allow:
no rows, an eps of zero, strides of any kind, a caller's context.  Values are compared as in
tests/test_gpu_residual.py, whose tolerances hold here."""

import ctypes
import threading

import pytest
import torch

from adamw_optimizer_step_gb300 import _binding as B
from adamw_optimizer_step_gb300 import layers
from tests.test_gpu_residual import BF16, F32, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from adamw_optimizer_step_gb300 import build
    build.build()
    B.lib()


@pytest.mark.parametrize("d", [64, 505, 1024, 8192, 8200])
@pytest.mark.parametrize("scale", [None, "one", "vector"])
def test_gradients_of_no_rows(d, scale):
    """Tensors of no rows, without a norm behind the update: sums of nothing are 0."""
    c = Case(0, d, pre=False, gate="element", scale=scale)
    x, h = layers.residual_norm(c.x, c.block, **c.kw())
    g = layers.residual_norm_backward(c.dx_out, None, x, c.block, **c.kw())
    assert h is None and x.shape == g["dx"].shape == g["dblock"].shape == g["dgate"].shape == (0, d)
    assert not g["dpost_gain"].any() and (scale is None or not g["dscale"].any())


@pytest.mark.parametrize("types", [(BF16, BF16), (F32, BF16), (F32, F32)], ids=lambda t: "-".join(str(x)[6:] for x in t))
@pytest.mark.parametrize("n", [1, 3, 37])
@pytest.mark.parametrize("d", [5, 64, 128, 200, 2048, 8200])
def test_eps_of_zero(d, n, types):
    """Rows of numbers that are not 0 have a norm without an eps; the rows that a warp of
    several does not have (32 / threads of them, widths up to 128) reach no sum."""
    for gate in (None, "row", "element"):
        Case(n, d, *types, gate=gate, eps=0.0, seed=d + n).check()


def test_dropout_of_any_strides():
    """Transposed and expanded tensors, of two axes as of three: the bits of their copies."""
    base = torch.randn(24, 40, device="cuda")
    for t in (base.T, base[:, ::2], base[:1].expand(24, 40), base[:, :1].expand(24, 40), base[:, 3:4], base[:, :1].T):
        want = layers.dropout(t.contiguous(), 0.4, 5)
        assert torch.equal(layers.dropout(t, 0.4, 5), want)
        assert torch.equal(layers.dropout(t[None], 0.4, 5), want[None])
        out = torch.full((t.shape[0], t.shape[1] + 3), 7.0, device="cuda")
        layers.dropout(t, 0.4, 5, out=out[:, :t.shape[1]])
        assert torch.equal(out[:, :t.shape[1]], want) and (out[:, t.shape[1]:] == 7).all()
    x = base.T.requires_grad_()
    y = layers.dropout_autograd(x, 0.4, 5)
    y.backward(torch.ones_like(y))
    assert torch.equal(x.grad, layers.dropout(torch.ones_like(y), 0.4, 5))


def test_a_callers_context_stays_current():
    """A thread with a driver context of its own: a call of attention (of no sequences, so nothing
    runs in it) leaves it current."""
    driver = ctypes.CDLL("libcuda.so.1")
    torch.zeros(1, device="cuda")
    args = B.AttnArgs(batch=0, sq=4, sk=4, q_heads=1, k_heads=1, dk=64, dv=64, causal=1, dtype=B.GBO_BF16, scale=1.0)
    seen = []

    def call():
        mine, now, device = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_int()
        seen.append(driver.cuDeviceGet(ctypes.byref(device), 0))
        seen.append(driver.cuCtxCreate_v2(ctypes.byref(mine), 0, device))
        seen.append(B.lib().gbo_attn_forward(ctypes.byref(args), None, None, None, None, 0, None, None))
        seen.append(driver.cuCtxGetCurrent(ctypes.byref(now)))
        seen.append(now.value == mine.value)
        seen.append(driver.cuCtxDestroy_v2(mine))

    t = threading.Thread(target=call)
    t.start()
    t.join()
    assert seen == [0, 0, 0, 0, True, 0]
    assert torch.equal(layers.dropout(torch.ones(8, device="cuda"), 0.0, 1), torch.ones(8, device="cuda"))


def test_a_training_pass_captured():
    """Both passes of a block in autograd, captured into a graph with the seed on the device: replays have
    the bits of the eager pass, on the values and with the seed that they find."""
    gen = torch.Generator().manual_seed(3)
    made = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    b, s, hq, hk, d = 2, 150, 4, 2, 64
    x, block, qkv = (made(b, s, hq * d).to(BF16).cuda(), made(b, s, hq * d).to(BF16).cuda(),
                     made(b, s, hq + 2 * hk, d).to(BF16).cuda())
    gain = (1 + 0.3 * made(hq * d)).cuda()
    leaves = [t.requires_grad_() for t in (x, block, qkv, gain)]
    seed, lengths = torch.tensor([5], device="cuda"), torch.tensor([150, 90], dtype=torch.int32, device="cuda")

    def both():
        y = layers.attention_autograd(*qkv.split((hq, hk, hk), dim=2), q_lengths=lengths, k_lengths=lengths)
        z, h = layers.residual_norm_autograd(x, block + y.flatten(2), post_norm=True, post_gain=gain, pre_gain=gain, dropout=0.25, seed=seed)
        out = layers.dropout_autograd(h, 0.5, seed, offset=1)
        return (out, *torch.autograd.grad((z.float() + out.float().square()).sum(), leaves))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = [t.clone() for t in both()]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, w) for a, w in zip(got, first))
    with torch.no_grad():
        seed += 1
        qkv.copy_(qkv.flip(1))
        lengths.copy_(lengths.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in got]
    assert all(torch.equal(a, w) for a, w in zip(replayed, both())) and not torch.equal(replayed[0], first[0])


def test_two_residual_calls_at_once():
    """Two streams at the same time, each with partial sums of its own: the bits of the calls alone."""
    cases = [Case(3000, d, gate="element", seed=d) for d in (72, 1024)]
    alone = []
    for c in cases:
        x, h = layers.residual_norm(c.x, c.block, **c.kw())
        alone.append((x, h, layers.residual_norm_backward(c.dx_out, c.dh, x, c.block, **c.kw())))
    streams = [torch.cuda.Stream() for _ in cases]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(10):
        for n, (c, st) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(st):
                x, h = layers.residual_norm(c.x, c.block, **c.kw())
                got[n].append((x, h, layers.residual_norm_backward(c.dx_out, c.dh, x, c.block, **c.kw())))
    torch.cuda.synchronize()
    for n, (x, h, g) in enumerate(alone):
        for x1, h1, g1 in got[n]:
            assert torch.equal(x1, x) and torch.equal(h1, h) and all(torch.equal(g1[k], g[k]) for k in g)


def test_what_the_gradients_need_is_asked_for():
    """Without the forward's lse, its output or the gradient of that: the library's refusal."""
    q = torch.zeros(1, 4, 2, 64, dtype=BF16, device="cuda")
    y, lse = layers.attention(q, q, q, return_lse=True)
    for dy, out, sums, what in ((y, y, None, "lse"), (None, y, lse, "NULL"), (y, None, lse, "NULL")):
        with pytest.raises(B.GboError, match=what):
            layers.attention_backward(dy, q, q, q, out, sums)
