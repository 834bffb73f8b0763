"""Host-side behaviour of the rotary and cross-entropy entry points: what they
refuse, frequencies, workspace sizes.  No GPU needed: every refusal comes
before the device is touched, and the fake addresses are never dereferenced."""

import ctypes
import math

import pytest
import torch

from adamw_optimizer_step_gb300 import _binding as B
from adamw_optimizer_step_gb300 import build as build_mod
from adamw_optimizer_step_gb300 import layers

FAKE = 1 << 20
INVALID, SHAPE, DTYPE, WORKSPACE = -1, -2, -5, -6


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return B.lib()


# ---------------------------------------------------------------------------
# rotary

def rope_opts(**kw):
    f = (ctypes.c_double * 64)(*([0.5] * 64))
    o = dict(head_dim=128, rot_dim=128, offset=0, layout=B.GBO_ROPE_HALF, freq=f, magnitude=1.0, eps=1e-6)
    o.update(kw)
    freq = ctypes.cast(o["freq"], ctypes.POINTER(ctypes.c_double)) if o["freq"] is not None else None
    return B.RopeOpts(o["head_dim"], o["rot_dim"], o["offset"], o["layout"], freq, o["magnitude"], o["eps"]), f


def rope_tensor(**kw):
    t = B.RopeTensor()
    o = dict(x=FAKE, y=2 * FAKE, heads=4, dtype=B.GBO_BF16, norm=1)
    o.update(kw)
    for k, v in o.items():
        setattr(t, k, v)
    for s in (t.x_stride, t.dy_stride, t.y_stride):
        s[0], s[1], s[2] = 4096, 512, 128
    return t


def rope_call(L, tensors, opts, back=False, batch=1, seq=8, n=None, pos=None, ws=None, nbytes=0):
    arr = (B.RopeTensor * max(1, len(tensors)))(*tensors)
    n = len(tensors) if n is None else n
    p = ctypes.byref(pos) if pos is not None else None
    o = ctypes.byref(opts) if opts is not None else None
    if back:
        return L.gbo_rope_backward(arr, n, o, batch, seq, p, ws, nbytes, None)
    return L.gbo_rope_forward(arr, n, o, batch, seq, p, None)


@pytest.mark.parametrize("opts,code", [
    (dict(head_dim=0), SHAPE), (dict(head_dim=513), SHAPE), (dict(rot_dim=127), SHAPE), (dict(rot_dim=-2), SHAPE),
    (dict(offset=1), SHAPE), (dict(offset=-1), SHAPE), (dict(head_dim=64), SHAPE), (dict(layout=2), INVALID),
    (dict(freq=None), INVALID), (dict(freq=(ctypes.c_double * 64)(*([float("nan")] * 64))), INVALID),
    (dict(magnitude=float("inf")), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
])
def test_rotary_options_refused(L, opts, code):
    o, keep = rope_opts(**opts)
    assert rope_call(L, [rope_tensor()], o) == code and L.gbo_last_error()


@pytest.mark.parametrize("tensor,back,code", [
    (dict(x=None), False, INVALID), (dict(y=None), False, INVALID), (dict(x=FAKE + 1), False, INVALID),
    (dict(dtype=7), False, DTYPE), (dict(heads=-1), False, SHAPE), (dict(norm=2), False, INVALID),
    (dict(norm=0, gain=FAKE), False, INVALID), (dict(gain=FAKE + 2), False, INVALID),
    (dict(dy=FAKE), False, INVALID), (dict(dgain=FAKE), False, INVALID),
    (dict(dy=None), True, INVALID), (dict(dy=FAKE, norm=0, x=None, dgain=FAKE), True, INVALID),
    (dict(dy=FAKE, x=None), True, INVALID),
])
def test_rotary_tensors_refused(L, tensor, back, code):
    o, keep = rope_opts()
    assert rope_call(L, [rope_tensor(**tensor)], o, back) == code and L.gbo_last_error()


def test_rotary_tables_refused(L):
    o, keep = rope_opts()
    t = rope_tensor()
    assert rope_call(L, [t] * 4, o, n=5) == INVALID
    assert rope_call(L, [t], o, n=-1) == INVALID
    assert rope_call(L, [t], None) == INVALID
    assert rope_call(L, [t], o, batch=-1) == SHAPE and rope_call(L, [t], o, seq=-1) == SHAPE
    assert rope_call(L, [t], o, batch=1 << 40, seq=1 << 40) == SHAPE
    assert rope_call(L, [t, rope_tensor(dtype=B.GBO_F32)], o) == DTYPE
    assert rope_call(L, [t, rope_tensor(norm=0)], o) == INVALID
    assert rope_call(L, [t], o, pos=B.RopePositions(FAKE, 0, 1, 0, B.GBO_F32, 0)) == DTYPE
    assert rope_call(L, [t], o, pos=B.RopePositions(FAKE + 4, 0, 1, 0, B.GBO_I64, 0)) == INVALID


def test_binding_refuses():
    spec = layers.RotarySpec(64)
    x = torch.zeros(1, 2, 3, 64)
    with pytest.raises(ValueError):
        layers.rotary(x, 0, spec)  # not on a GPU
    with pytest.raises(ValueError):
        layers.rotary(x[0], 0, spec)  # three axes
    with pytest.raises(ValueError):
        layers.rotary(x[..., :32], 0, spec)  # another head size
    with pytest.raises(TypeError):
        layers.rotary(x.half(), 0, spec)
    with pytest.raises(ValueError):
        layers.RotarySpec(64, layout="thirds")
    with pytest.raises(ValueError):
        layers.RotarySpec(64, scaling=dict(kind="cubic"))
    with pytest.raises(ValueError):
        layers.RotarySpec(64, frequencies=[1.0])
    with pytest.raises(B.GboError):
        layers.RotarySpec(64, rot_dim=63)
    with pytest.raises(ValueError):
        layers.linear_cross_entropy(torch.zeros(2, 8).bfloat16(), torch.zeros(4, 8).bfloat16(), torch.zeros(2).long())
    with pytest.raises(ValueError):
        layers.linear_cross_entropy_grad(torch.zeros(2, 8).bfloat16(), torch.zeros(4, 8).bfloat16(),
                                         torch.zeros(2).long())


# ---------------------------------------------------------------------------
# frequencies

def test_frequencies(L):
    """Each scaling against its definition, element by element."""
    r, base, factor, trained = 64, 10000.0, 8.0, 4096.0
    plain = [base ** (-2 * j / r) for j in range(r // 2)]

    def freqs(**s):
        spec = layers.RotarySpec(r, base=base, scaling=s or None)
        return spec.frequencies, spec.magnitude

    def same(a, b):
        assert len(a) == len(b) and all(abs(x - y) <= 1e-14 * abs(y) for x, y in zip(a, b))

    same(freqs()[0], plain)
    same(freqs(kind="none")[0], plain)
    same(freqs(kind="linear", factor=factor)[0], [f / factor for f in plain])
    stretched = base * factor ** (r / (r - 2))
    f, m = freqs(kind="ntk", factor=factor)
    assert m == 1.0 and all(abs(x - stretched ** (-2 * j / r)) <= 1e-13 * x for j, x in enumerate(f))
    # the slowest frequency is the plain one divided by the factor, the fastest unchanged
    assert abs(f[0] - 1.0) < 1e-15 and abs(f[-1] - plain[-1] / factor) < 1e-12 * f[-1]
    f, m = freqs(kind="yarn", factor=factor, trained=trained, fast=32.0, slow=1.0)
    assert abs(m - (0.1 * math.log(factor) + 1)) < 1e-6
    turns = [trained * x / (2 * math.pi) for x in plain]
    low = max(math.floor(r * math.log(trained / (32 * 2 * math.pi)) / (2 * math.log(base))), 0)
    high = min(math.ceil(r * math.log(trained / (2 * math.pi)) / (2 * math.log(base))), r - 1)
    for j, x in enumerate(f):
        w = min(max((j - low) / (high - low), 0.0), 1.0)
        assert abs(x - plain[j] * ((1 - w) + w / factor)) <= 1e-13 * x
        if j <= low:
            assert turns[j] >= 31 or j == low
    f, m = freqs(kind="wavelength", factor=factor, trained=trained, fast=4.0, slow=1.0)
    assert m == 1.0
    for j, x in enumerate(f):
        if turns[j] >= 4:
            assert x == plain[j]
        elif turns[j] <= 1:
            assert abs(x - plain[j] / factor) <= 1e-15 * x
        else:
            w = (turns[j] - 1) / 3
            assert abs(x - plain[j] * (w + (1 - w) / factor)) <= 1e-13 * x


@pytest.mark.parametrize("rot,base,scaling,code", [
    (0, 1e4, None, SHAPE), (63, 1e4, None, SHAPE), (514, 1e4, None, SHAPE), (64, 0.0, None, INVALID),
    (64, float("inf"), None, INVALID), (64, 1e4, (9, 0, 1.0, 0, 0, 0), INVALID),
    (64, 1e4, (B.GBO_ROPE_SCALE_LINEAR, 0, 0.0, 0, 0, 0), INVALID), (2, 1e4, (B.GBO_ROPE_SCALE_NTK, 0, 2.0, 0, 0, 0), SHAPE),
    (64, 1e4, (B.GBO_ROPE_SCALE_YARN, 0, 2.0, 0.0, 32.0, 1.0), INVALID),
    (64, 1e4, (B.GBO_ROPE_SCALE_YARN, 0, 2.0, 4096.0, 1.0, 1.0), INVALID),
    (64, 1.0, (B.GBO_ROPE_SCALE_YARN, 0, 2.0, 4096.0, 32.0, 1.0), INVALID),
    (64, 1e4, (B.GBO_ROPE_SCALE_WAVELENGTH, 0, 2.0, 4096.0, 4.0, 0.0), INVALID),
])
def test_frequencies_refused(L, rot, base, scaling, code):
    with pytest.raises(B.GboError) as e:
        B.gbo_rope_frequencies(rot, base, B.RopeScaling(*scaling) if scaling else None)
    assert e.value.code == code


# ---------------------------------------------------------------------------
# cross entropy

def xent_args(**kw):
    a = B.XentArgs(FAKE, 2 * FAKE, 3 * FAKE, None, None, 16, 1000, 64, 64, 64, 1.0, 0.0, B.GBO_I64, 1, 0, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def xent_grads(**kw):
    g = B.XentGrads(4 * FAKE, 5 * FAKE, 64, 64, B.GBO_BF16, B.GBO_F32, 0, 0)
    for k, v in kw.items():
        setattr(g, k, v)
    return g


@pytest.mark.parametrize("args,code", [
    (dict(n=-1), SHAPE), (dict(n=(1 << 30) + 1), SHAPE), (dict(v=0), SHAPE), (dict(d=0), SHAPE), (dict(d=60), SHAPE),
    (dict(h_stride=63), SHAPE), (dict(w_stride=63), SHAPE), (dict(w_stride=68), SHAPE), (dict(w=None), INVALID),
    (dict(w=FAKE + 2), INVALID), (dict(h=None), INVALID), (dict(h=FAKE + 1), INVALID), (dict(labels=None), INVALID),
    (dict(labels=FAKE + 4), INVALID), (dict(label_dtype=B.GBO_F32), DTYPE), (dict(row_weight=FAKE + 1), INVALID),
    (dict(upstream=FAKE + 2), INVALID), (dict(logit_scale=float("nan")), INVALID), (dict(z_loss=float("inf")), INVALID),
    (dict(mean=2), INVALID), (dict(keep=-1), INVALID),
])
def test_cross_entropy_arguments_refused(L, args, code):
    a = xent_args(**args)
    ws = ctypes.c_void_p(FAKE)
    assert L.gbo_xent_forward(ctypes.byref(a), FAKE, FAKE, FAKE, ws, 1 << 30, None, None) == code
    g = xent_grads()
    assert L.gbo_xent_grad(ctypes.byref(a), FAKE, FAKE, FAKE, ctypes.byref(g), ws, 1 << 30, None, None) == code
    assert L.gbo_last_error()


@pytest.mark.parametrize("grads,code", [
    (dict(dh=None, dw=None), INVALID), (dict(dh_dtype=5), DTYPE), (dict(dw_dtype=-1), DTYPE), (dict(dh_stride=63), SHAPE),
    (dict(dw_stride=8), SHAPE), (dict(dh=FAKE + 1), INVALID), (dict(dw=FAKE + 2), INVALID), (dict(accumulate_dw=2), INVALID),
])
def test_cross_entropy_gradients_refused(L, grads, code):
    a, g, ws = xent_args(), xent_grads(**grads), ctypes.c_void_p(FAKE)
    assert L.gbo_xent_grad(ctypes.byref(a), FAKE, None, None, ctypes.byref(g), ws, 1 << 30, None, None) == code
    assert L.gbo_xent_backward(ctypes.byref(a), FAKE, ctypes.byref(g), ws, 1 << 30, None, None) == code


def test_cross_entropy_null_and_misaligned(L):
    a, g, ws = xent_args(), xent_grads(), ctypes.c_void_p(FAKE)
    assert L.gbo_xent_forward(None, FAKE, None, None, ws, 1 << 30, None, None) == INVALID
    assert L.gbo_xent_grad(ctypes.byref(a), FAKE, None, None, None, ws, 1 << 30, None, None) == INVALID
    assert L.gbo_xent_backward(ctypes.byref(a), None, ctypes.byref(g), ws, 1 << 30, None, None) == INVALID
    assert L.gbo_xent_forward(ctypes.byref(a), FAKE + 1, None, None, ws, 1 << 30, None, None) == INVALID


def test_cross_entropy_workspace_sizes():
    size = B.gbo_xent_workspace_bytes
    # losses alone: a copy of the rows and 8 bytes per row and 128 columns
    n, v, d = 8192, 128000, 2048
    forward = size(n, v, d)
    assert 2 * n * d + 8 * n * v // 128 <= forward <= 1.02 * (2 * n * d + 8 * n * v // 128)
    # gradients: 2 bytes a logit, kept whole up to 8 GiB
    assert size(n, v, d, True) >= forward + 2 * n * v
    # more rows: pieces of at most 2 GiB (beside the row copy, the fp32 sums and statistics)
    n = 65536
    big = size(n, v, d, True)
    assert big < (2 << 30) + 2 * n * d + 4 * n * d + 256 * n + 8 * n * v // 128
    # a cap is kept to, and the least one is a piece of 256 columns
    for cap in (1 << 30, 1 << 31, 1 << 32, 1 << 34):
        got = size(n, v, d, True, cap)
        assert 0 <= got <= cap
    assert size(n, v, d, True, 1 << 35) > 2 * n * v > size(n, v, d, True, 1 << 33) > 0
    assert size(64, 1000, 64, True, 1000) == 0
    for bad in ((-1, 10, 8), (4, 0, 8), (4, 10, 12), (4, 10, 0)):
        assert size(*bad) == 0


def test_a_spec_can_be_copied_and_saved(L):
    import copy
    import pickle
    spec = layers.RotarySpec(64, 32, 16, "interleaved", 1e6,
                             scaling=dict(kind="yarn", factor=4.0, trained=4096, fast=32, slow=1))
    for other in (copy.deepcopy(spec), pickle.loads(pickle.dumps(spec))):
        assert other.frequencies == spec.frequencies and other.opts.magnitude == spec.opts.magnitude
        assert (other.opts.offset, other.opts.layout, other.rot_dim) == (16, B.GBO_ROPE_INTERLEAVED, 32)
        assert ctypes.addressof(other.opts.freq.contents) != ctypes.addressof(spec.opts.freq.contents)
