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
