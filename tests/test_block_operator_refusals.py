"""Host-side behaviour of attention, the residual update and dropout: what they
refuse, workspace sizes, autograd's constants.  No GPU needed: every refusal comes
before the device is touched, and the fake addresses are never dereferenced."""

import ctypes

import pytest
import torch

from adamw_optimizer_step_gb300 import _binding as B
from adamw_optimizer_step_gb300 import build as build_mod
from adamw_optimizer_step_gb300 import layers

FAKE = 1 << 20
INVALID, SHAPE, DTYPE, WORKSPACE = -1, -2, -5, -6
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return B.lib()


# ---------------------------------------------------------------------------
# attention

def attn_args(**kw):
    a = B.AttnArgs()
    o = dict(q=FAKE, k=2 * FAKE, v=3 * FAKE, batch=2, sq=64, sk=64, window=0, q_heads=4, k_heads=2, dk=64, dv=64,
             n_documents=0, causal=1, dtype=B.GBO_BF16, scale=0.125)
    strides = dict(q_stride=(64 * 256, 256, 64), k_stride=(64 * 128, 128, 64), v_stride=(64 * 128, 128, 64))
    o.update({k: v for k, v in kw.items() if k not in strides})
    strides.update({k: v for k, v in kw.items() if k in strides})
    for k, v in o.items():
        setattr(a, k, v)
    for k, v in strides.items():
        getattr(a, k)[:] = v
    return a


STRIDE = (ctypes.c_int64 * 3)(64 * 256, 256, 64)


def attn_forward(L, a, y=4 * FAKE, stride=STRIDE, lse=None):
    return L.gbo_attn_forward(ctypes.byref(a) if a is not None else None, y, stride, lse, None, 0, None, None)


@pytest.mark.parametrize("args,code", [
    (dict(dtype=B.GBO_F32), DTYPE), (dict(batch=-1), SHAPE), (dict(sq=-1), SHAPE), (dict(sk=(1 << 30) + 1), SHAPE),
    (dict(q_heads=3), SHAPE), (dict(k_heads=0), SHAPE), (dict(q_heads=1), SHAPE), (dict(dk=0), SHAPE),
    (dict(dk=12), SHAPE), (dict(dk=200), SHAPE), (dict(dv=136), SHAPE), (dict(dv=4), SHAPE),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(causal=2), INVALID), (dict(window=-1), INVALID),
    (dict(window=8, causal=0), INVALID), (dict(q_lengths=FAKE + 2), INVALID), (dict(k_lengths=FAKE + 1), INVALID),
    (dict(documents=FAKE), INVALID), (dict(documents=FAKE, n_documents=3), INVALID),
    (dict(documents=FAKE, n_documents=3, batch=1, sk=65), INVALID),
    (dict(documents=FAKE, n_documents=3, batch=1, k_lengths=FAKE), INVALID), (dict(n_documents=2), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=FAKE + 8), INVALID),
    (dict(q_stride=(64 * 256, 256, 60)), INVALID), (dict(k_stride=(0, 128, 64)), INVALID),
    (dict(v_stride=(-64, 128, 64)), INVALID), (dict(q_stride=(1 << 39, 256, 64)), INVALID),
])
def test_attention_arguments_refused(L, args, code):
    assert attn_forward(L, attn_args(**args)) == code, L.gbo_last_error()


def test_attention_outputs_refused(L):
    assert attn_forward(L, None) == INVALID
    assert attn_forward(L, attn_args(), y=None) == INVALID
    assert attn_forward(L, attn_args(), stride=None) == INVALID
    assert attn_forward(L, attn_args(), y=FAKE + 4) == INVALID
    assert attn_forward(L, attn_args(), lse=FAKE + 2) == INVALID
    a = attn_args()
    assert L.gbo_attn_backward(ctypes.byref(a), None, None, 0, None, None) == INVALID
    g = B.AttnGrads()
    assert L.gbo_attn_backward(ctypes.byref(a), ctypes.byref(g), None, 0, None, None) == INVALID  # no dy
    g.dy, g.y = FAKE, 2 * FAKE
    g.dy_stride[:] = g.y_stride[:] = STRIDE[:]
    assert L.gbo_attn_backward(ctypes.byref(a), ctypes.byref(g), None, 0, None, None) == INVALID  # no lse
    g.lse = FAKE + 2
    assert L.gbo_attn_backward(ctypes.byref(a), ctypes.byref(g), None, 0, None, None) == INVALID
    g.lse, g.dq = FAKE, FAKE + 8
    g.dq_stride[:] = STRIDE[:]
    assert L.gbo_attn_backward(ctypes.byref(a), ctypes.byref(g), None, 0, None, None) == INVALID


def test_attention_workspace_of_refused_arguments(L):
    assert L.gbo_attn_forward_workspace_bytes(None) == 0
    assert L.gbo_attn_backward_workspace_bytes(ctypes.byref(attn_args(dk=12))) == 0
    assert L.gbo_attn_backward_workspace_bytes(ctypes.byref(attn_args())) == 2 * 64 * 4 * 8


def test_attention_binding_refuses():
    q, k = torch.zeros(2, 5, 4, 64, dtype=BF16), torch.zeros(2, 7, 2, 64, dtype=BF16)
    with pytest.raises(TypeError, match="bfloat16"):
        B.attn_args(q.float(), k, k)
    with pytest.raises(ValueError, match="batch, seq, heads, dim"):
        B.attn_args(q[0], k, k)
    with pytest.raises(ValueError, match="k must be"):
        B.attn_args(q, k[:1], k)
    with pytest.raises(ValueError, match="v must be"):
        B.attn_args(q, k, k[:, :3])
    with pytest.raises(ValueError, match="consecutive"):
        B.attn_args(q.transpose(1, 3).contiguous().transpose(1, 3), k, k)
    with pytest.raises(ValueError, match="CUDA"):
        B.attn_args(q, k, k)


def test_index_tensors_are_int32():
    for bad in (torch.zeros(2, dtype=torch.int64), torch.zeros(3, dtype=torch.int32), torch.zeros(2, 1, dtype=torch.int32)):
        with pytest.raises(ValueError, match="q_lengths"):
            B._attn_index(bad, 2, "q_lengths")
    with pytest.raises(ValueError, match="CUDA"):
        B._attn_index(torch.zeros(2, dtype=torch.int32), 2, "q_lengths")
    assert B._attn_index(None, 2, "q_lengths") == 0


# ---------------------------------------------------------------------------
# residual update, dropout

def res_args(**kw):
    a = B.ResidualArgs()
    o = dict(x=FAKE, block=2 * FAKE, n=4, d=64, x_stride=64, block_stride=64, gate_stride=64, x_dtype=B.GBO_BF16,
             block_dtype=B.GBO_BF16, has_block=1, post_norm=1, pre_norm=1, gate_sigmoid=1, eps=1e-6)
    o.update(kw)
    for k, v in o.items():
        setattr(a, k, v)
    return a


def res_forward(L, a, x_out=3 * FAKE, xs=64, h=4 * FAKE, hs=64):
    return L.gbo_residual_forward(ctypes.byref(a) if a is not None else None, x_out, xs, h, hs, None, None)


@pytest.mark.parametrize("args,code", [
    (dict(x_dtype=7), DTYPE), (dict(block_dtype=B.GBO_F32), DTYPE), (dict(n=-1), SHAPE), (dict(d=0), SHAPE),
    (dict(d=16385), SHAPE), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(post_norm=2), INVALID),
    (dict(gate_mode=3), INVALID), (dict(scale_mode=5), INVALID), (dict(dropout=1.0), INVALID), (dict(dropout=-0.1), INVALID),
    (dict(dropout=1.0 - 2.0 ** -18), INVALID), (dict(dropout=float("nan")), INVALID), (dict(dev_seed=FAKE + 4), INVALID),
    (dict(gate_mode=1), INVALID), (dict(gate=FAKE), INVALID), (dict(scale_mode=1), INVALID), (dict(scale=FAKE), INVALID),
    (dict(post_gain=FAKE, post_norm=0), INVALID), (dict(pre_gain=FAKE, pre_norm=0), INVALID),
    (dict(pre_gain=FAKE + 2), INVALID), (dict(has_block=0), INVALID),
    (dict(has_block=0, block=None, post_norm=0, pre_norm=0), INVALID),
    (dict(has_block=0, block=None, post_norm=0, dropout=0.5), INVALID), (dict(block=None), INVALID),
    (dict(block_stride=63), INVALID), (dict(x=None), INVALID), (dict(x=FAKE + 1), INVALID),
    (dict(gate_mode=1, gate=FAKE, gate_stride=8), INVALID),
])
def test_residual_arguments_refused(L, args, code):
    assert res_forward(L, res_args(**args)) == code, L.gbo_last_error()


def test_residual_outputs_refused(L):
    assert res_forward(L, None) == INVALID
    assert res_forward(L, res_args(), x_out=None) == INVALID
    assert res_forward(L, res_args(), h=None) == INVALID
    assert res_forward(L, res_args(), hs=32) == INVALID
    assert res_forward(L, res_args(pre_norm=0)) == INVALID  # h without pre_norm
    assert res_forward(L, res_args(has_block=0, block=None, post_norm=0)) == INVALID  # x_out without a block

    def backward(a, **kw):
        g = B.ResidualGrads()
        for k, v in dict(dict(dx_out=FAKE, dh=2 * FAKE, dx=3 * FAKE, dx_out_stride=64, dh_stride=64, dx_stride=64), **kw).items():
            setattr(g, k, v)
        return L.gbo_residual_backward(ctypes.byref(a), ctypes.byref(g), None, 0, None, None)

    assert L.gbo_residual_backward(ctypes.byref(res_args()), None, None, 0, None, None) == INVALID
    assert backward(res_args(), dpre_gain=FAKE) == INVALID   # no pre_gain to have one
    assert backward(res_args(), dscale=FAKE) == INVALID
    assert backward(res_args(), dgate=FAKE, dgate_stride=64) == INVALID
    assert backward(res_args(pre_norm=0)) == INVALID         # dh without pre_norm
    assert backward(res_args(), dh=None) == INVALID
    assert backward(res_args(pre_norm=0), dh=None, dx_out=None) == INVALID
    assert backward(res_args(), dx_stride=8) == INVALID
    assert backward(res_args(pre_gain=FAKE), dpre_gain=FAKE + 1) == INVALID


@pytest.mark.parametrize("call,code", [
    (dict(dtype=5), DTYPE), (dict(n=-1), SHAPE), (dict(n=1 << 62), SHAPE), (dict(p=1.0), INVALID), (dict(p=-0.5), INVALID),
    (dict(p=float("nan")), INVALID), (dict(x=None), INVALID), (dict(y=FAKE + 1), INVALID), (dict(x_stride=4), INVALID),
    (dict(dev_seed=FAKE + 4), INVALID),
])
def test_dropout_refused(L, call, code):
    o = dict(x=FAKE, x_stride=8, y=2 * FAKE, y_stride=8, n=4, d=8, dtype=B.GBO_BF16, p=0.5, seed=1, offset=0, dev_seed=None)
    o.update(call)
    assert L.gbo_dropout(*o.values(), None) == code, L.gbo_last_error()


def test_residual_binding_refuses():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="gate_kind"):
        B.residual_args(x, None, gate_kind="tanh")
    with pytest.raises(ValueError, match="CUDA"):
        B.residual_args(x, None)
    with pytest.raises(ValueError, match="seed"):
        B._seed_of(torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="seed"):
        B._seed_of(torch.zeros(2, dtype=torch.int64))
    assert B._seed_of(-1) == ((1 << 64) - 1, 0)
    with pytest.raises(TypeError):
        B.gbo_dropout(x, x.to(BF16), 0.5, 1)


def test_constants_that_require_a_gradient_are_refused():
    c = torch.tensor(0.5, requires_grad=True)
    x = torch.zeros(1, 2, 1, 8, dtype=BF16)
    with pytest.raises(ValueError, match="scale"):
        layers.attention_autograd(x, x, x, scale=c)
    with pytest.raises(ValueError, match="dropout"):
        layers.residual_norm_autograd(x[0, :, 0], x[0, :, 0], dropout=c)
    with pytest.raises(ValueError, match="eps"):
        layers.residual_norm_autograd(x[0, :, 0], x[0, :, 0], eps=c)
    with pytest.raises(ValueError, match="p has"):
        layers.dropout_autograd(x, c, 1)
    with pytest.raises(ValueError, match="norm alone"):
        layers.residual_norm_autograd(x[0, :, 0], dropout=0.5)


def test_expanded_gradients_become_rows_of_their_own():
    t = torch.zeros(2, 3, 4, 16, dtype=BF16)
    assert layers._aligned_heads(t) is t
    for odd in (torch.zeros(1, dtype=BF16).expand(2, 3, 4, 16), t[..., 4:12], t.transpose(2, 3)[:, :, :8].transpose(2, 3)[:, :, :, ::2]):
        c = layers._aligned_heads(odd)
        assert c.shape == odd.shape and c.is_contiguous() and c is not odd
    part = torch.zeros(2, 3, 12, 16, dtype=BF16)[:, :, 4:8]
    assert layers._aligned_heads(part) is part
