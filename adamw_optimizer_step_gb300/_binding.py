"""ctypes binding of libgbo.so: argument marshalling only.

Every function here has the name of the C entry point it calls (see
``include/gbo.h``), turns torch tensors into device pointers and Python
numbers into C scalars, and raises :class:`GboError` on a non-zero status.
All arithmetic runs in the library's CUDA kernels; there is no fallback.
"""

import ctypes
import functools
import os
import struct

import torch

from . import build as _build

GBO_OK = 0
GBO_F32 = 0
GBO_BF16 = 1
GBO_NS_BF16 = 0
GBO_NS_F32 = 1
GBO_ROUTE_AUTO = 0
GBO_ROUTE_X = 1
GBO_ROUTE_GRAM = 2
GBO_STATUS_NONFINITE = 1
GBO_STATUS_TIMEOUT = 2
GBO_STATUS_BAD_LABEL = 4
GBO_I32 = 16
GBO_I64 = 17
GBO_ROPE_HALF = 0
GBO_ROPE_INTERLEAVED = 1
GBO_ROPE_SCALE_NONE = 0
GBO_ROPE_SCALE_LINEAR = 1
GBO_ROPE_SCALE_NTK = 2
GBO_ROPE_SCALE_YARN = 3
GBO_ROPE_SCALE_WAVELENGTH = 4
GBO_ROPE_MAX_TENSORS = 4
GBO_MAX_VIEW_DIMS = 6
GBO_N_PHASES = 6
PHASE_NAMES = ("momentum", "gram", "product", "square", "rows", "final")

c_void_p, c_int32, c_int64, c_float, c_size_t = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                                                 ctypes.c_float, ctypes.c_size_t)


class GboError(RuntimeError):
    def __init__(self, code, message):
        super().__init__("libgbo error %d: %s" % (code, message))
        self.code = code


class MuonDesc(ctypes.Structure):
    _fields_ = [("w", c_void_p), ("g", c_void_p), ("mom", c_void_p), ("row_v", c_void_p),
                ("rows", c_int64), ("cols", c_int64), ("view", c_int64 * GBO_MAX_VIEW_DIMS),
                ("w_dtype", c_int32), ("g_dtype", c_int32), ("view_ndim", c_int32),
                ("n_split", c_int32), ("split_off", c_int32), ("lr_mult", c_float), ("wd", c_float),
                ("reserved", c_int32)]


class MuonOpts(ctypes.Structure):
    _fields_ = [("abc", ctypes.POINTER(c_float)), ("mu", c_float), ("beta2", c_float),
                ("eps", c_float), ("nesterov", c_int32), ("ns_steps", c_int32),
                ("abc_per_step", c_int32), ("precision", c_int32), ("normuon", c_int32),
                ("route", c_int32), ("rms_target", c_float), ("reserved", c_int32),
                ("workspace_cap", c_int64)]


class Tensor(ctypes.Structure):
    _fields_ = [("ptr", c_void_p), ("numel", c_int64), ("dtype", c_int32), ("reserved", c_int32)]


class AdamWDesc(ctypes.Structure):
    _fields_ = [("p", c_void_p), ("g", c_void_p), ("m", c_void_p), ("v", c_void_p),
                ("numel", c_int64), ("g_dtype", c_int32), ("reserved", c_int32)]


class AdamWOpts(ctypes.Structure):
    _fields_ = [("lr", c_float), ("beta1", c_float), ("beta2", c_float), ("eps", c_float),
                ("weight_decay", c_float), ("step", c_int32), ("dev_step", c_void_p)]


class PlanInfo(ctypes.Structure):
    _fields_ = [("n_weights", c_int64), ("n_active", c_int64), ("n_matrices", c_int64),
                ("n_shape_classes", c_int64), ("muon_params", c_int64), ("ns_flops", ctypes.c_double),
                ("ns_flops_executed", ctypes.c_double), ("launches_per_step", c_int64),
                ("n_gram_route", c_int64), ("n_mom_fused", c_int64)]


class RopeScaling(ctypes.Structure):
    _fields_ = [("kind", c_int32), ("reserved", c_int32), ("factor", ctypes.c_double),
                ("trained", ctypes.c_double), ("fast", ctypes.c_double), ("slow", ctypes.c_double)]


class RopeOpts(ctypes.Structure):
    _fields_ = [("head_dim", c_int32), ("rot_dim", c_int32), ("offset", c_int32), ("layout", c_int32),
                ("freq", ctypes.POINTER(ctypes.c_double)), ("magnitude", c_float), ("eps", c_float)]


class RopeTensor(ctypes.Structure):
    _fields_ = [("x", c_void_p), ("dy", c_void_p), ("y", c_void_p), ("gain", c_void_p), ("dgain", c_void_p),
                ("x_stride", c_int64 * 3), ("dy_stride", c_int64 * 3), ("y_stride", c_int64 * 3),
                ("heads", c_int32), ("dtype", c_int32), ("norm", c_int32), ("reserved", c_int32)]


class RopePositions(ctypes.Structure):
    _fields_ = [("ptr", c_void_p), ("stride_b", c_int64), ("stride_s", c_int64), ("start", c_int64),
                ("dtype", c_int32), ("reserved", c_int32)]


class XentArgs(ctypes.Structure):
    _fields_ = [("h", c_void_p), ("w", c_void_p), ("labels", c_void_p), ("row_weight", c_void_p),
                ("upstream", c_void_p), ("n", c_int64), ("v", c_int64), ("d", c_int64), ("h_stride", c_int64),
                ("w_stride", c_int64), ("logit_scale", c_float), ("z_loss", c_float), ("label_dtype", c_int32),
                ("mean", c_int32), ("keep", c_int32), ("reserved", c_int32)]


class XentGrads(ctypes.Structure):
    _fields_ = [("dh", c_void_p), ("dw", c_void_p), ("dh_stride", c_int64), ("dw_stride", c_int64),
                ("dh_dtype", c_int32), ("dw_dtype", c_int32), ("accumulate_dw", c_int32), ("reserved", c_int32)]


_STRUCTS = (MuonDesc, MuonOpts, Tensor, AdamWDesc, AdamWOpts, PlanInfo, RopeScaling, RopeOpts, RopeTensor,
            RopePositions, XentArgs, XentGrads)
_lib = None


def library_path():
    return _build.LIB_PATH


def lib():
    """Load libgbo.so (built by ``adamw_optimizer_step_gb300.build.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise ImportError("libgbo.so is not built (%s); run adamw_optimizer_step_gb300.build.build()" % path)
    L = ctypes.CDLL(path)
    sig = {
        "gbo_muon_plan_create": (c_int32, [ctypes.POINTER(MuonDesc), c_int32, ctypes.POINTER(c_int64),
                                           c_int32, ctypes.POINTER(MuonOpts), ctypes.POINTER(c_void_p)]),
        "gbo_muon_plan_destroy": (None, [c_void_p]),
        "gbo_muon_workspace_bytes": (c_size_t, [c_void_p]),
        "gbo_desc_hash": (ctypes.c_uint64, [c_void_p]),
        "gbo_muon_step": (c_int32, [c_void_p, c_float, c_void_p, c_size_t, c_void_p, c_void_p, c_void_p]),
        "gbo_normuon_rownorm": (c_int32, [c_void_p, c_int64, c_int64, c_void_p, c_void_p, c_int32, c_float,
                                          c_float, c_float, c_float, c_float, c_void_p, c_void_p]),
        "gbo_clip_norm_workspace_bytes": (c_size_t, []),
        "gbo_clip_norm": (c_int32, [ctypes.POINTER(Tensor), c_int32, c_float, c_void_p, c_void_p, c_void_p,
                                    c_void_p, c_size_t, c_void_p]),
        "gbo_h2d_copy": (c_int32, [c_void_p, c_void_p, ctypes.c_int64, c_int32, c_void_p]),
        "gbo_muon_plan_set_free_sms": (c_int32, [c_void_p, c_int32]),
        "gbo_clip_norm_noalloc": (c_int32, [ctypes.POINTER(Tensor), c_int32, c_float, c_void_p, c_void_p,
                                            c_void_p, c_void_p]),
        "gbo_adamw_step": (c_int32, [ctypes.POINTER(AdamWDesc), c_int32, ctypes.POINTER(AdamWOpts), c_void_p,
                                     c_void_p, c_void_p]),
        "gbo_rope_frequencies": (c_int32, [c_int32, ctypes.c_double, ctypes.POINTER(RopeScaling),
                                           ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)]),
        "gbo_rope_workspace_bytes": (c_size_t, [c_void_p, c_int32, ctypes.POINTER(RopeOpts)]),
        "gbo_rope_forward": (c_int32, [c_void_p, c_int32, ctypes.POINTER(RopeOpts), c_int64, c_int64, c_void_p,
                                       c_void_p]),
        "gbo_rope_backward": (c_int32, [c_void_p, c_int32, ctypes.POINTER(RopeOpts), c_int64, c_int64, c_void_p,
                                        c_void_p, c_size_t, c_void_p]),
        "gbo_xent_workspace_bytes": (c_size_t, [c_int64, c_int64, c_int64, c_int32, c_int64]),
        "gbo_xent_forward": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                                       c_void_p, c_void_p]),
        "gbo_xent_backward": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p,
                                        c_size_t, c_void_p, c_void_p]),
        "gbo_xent_grad": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                    c_void_p, c_size_t, c_void_p, c_void_p]),
        "gbo_testing_wait_timeout": (c_int32, [c_void_p, ctypes.c_uint32, c_void_p]),
        "gbo_testing_set_small_chain": (c_int32, [c_int32]),
        "gbo_testing_set_fused_gram": (c_int32, [c_int32]),
        "gbo_testing_set_fused_momentum": (c_int32, [c_int32]),
        "gbo_testing_set_tail_split": (c_int32, [c_int32]),
        "gbo_testing_set_momentum_stream": (c_int32, [c_int32]),
        "gbo_testing_pair_residency": (c_int32, []),
        "gbo_testing_set_pdl": (c_int32, [c_int32]),
        "gbo_last_error": (ctypes.c_char_p, []),
        "gbo_abi_version": (c_int32, []),
        "gbo_struct_size": (c_size_t, [c_int32]),
        "gbo_launch_count": (ctypes.c_uint64, []),
        "gbo_muon_plan_info": (c_int32, [c_void_p, ctypes.POINTER(PlanInfo)]),
        "gbo_muon_plan_desc_flops": (c_int32, [c_void_p, ctypes.POINTER(ctypes.c_double), c_int32]),
        "gbo_muon_plan_set_timing": (c_int32, [c_void_p, c_int32]),
        "gbo_muon_plan_set_stats": (c_int32, [c_void_p, c_void_p]),
        "gbo_muon_plan_set_event": (c_int32, [c_void_p, c_int32, c_void_p]),
        "gbo_muon_plan_phase_times": (c_int32, [c_void_p, ctypes.POINTER(c_float), ctypes.POINTER(c_int64),
                                                c_int32]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    for i, S in enumerate(_STRUCTS):
        if L.gbo_struct_size(i) != ctypes.sizeof(S):
            raise ImportError("ABI mismatch for %s: C %d bytes, Python %d" %
                              (S.__name__, L.gbo_struct_size(i), ctypes.sizeof(S)))
    _lib = L
    return L


def _check(code):
    if code != GBO_OK:
        raise GboError(code, lib().gbo_last_error().decode())


def _dtype(t):
    if t.dtype == torch.float32:
        return GBO_F32
    if t.dtype == torch.bfloat16:
        return GBO_BF16
    raise TypeError("tensor dtype must be float32 or bfloat16, got %s" % t.dtype)


def _dev_ptr(t, what, allow_host=False):
    if t is None:
        return None
    if not t.is_cuda and not allow_host:
        raise ValueError("%s must be a CUDA tensor" % what)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)
    return t.data_ptr()


def _current_stream():
    """Torch's current stream on the current device, as a handle."""
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


if not (hasattr(torch._C, "_cuda_getCurrentRawStream") and hasattr(torch._C, "_cuda_getDevice")):
    # without torch's direct accessors: through a Stream object, a few microseconds slower
    def _current_stream():  # noqa: F811
        return torch.cuda.current_stream().cuda_stream


def _stream(stream):
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ---------------------------------------------------------------------------
# Muon

class MuonPlan:
    """Owns a ``gbo_plan*`` and keeps the tensors it points to alive."""

    def __init__(self, handle, keepalive, n_descs=0):
        self.handle = handle
        self._keep = keepalive
        self.n_descs = n_descs

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.gbo_muon_plan_destroy(self.handle)
            self.handle = None


def muon_desc_table(entries, allow_host=False):
    """Marshal Muon weights into a ``gbo_muon_desc`` array and a split pool.

    Each entry is a dict with ``w`` (rows x cols, float32/bfloat16), ``g``
    (same shape, or None to skip), ``mom`` (float32), optional ``row_v``
    (float32, rows), ``view`` (tuple), ``split`` (tuple), ``lr_mult``, ``wd``.
    ``allow_host``: accept host tensors, for a plan that is only queried
    (plan creation never dereferences the pointers; such a plan must never
    be stepped).
    """
    arr = (MuonDesc * len(entries))()
    pool = []
    keep = []
    for d, e in zip(arr, entries):
        w, g, mom, rv = e["w"], e.get("g"), e.get("mom"), e.get("row_v")
        if w.dim() != 2:
            raise ValueError("Muon weights are 2-D")
        d.w = _dev_ptr(w, "w", allow_host)
        d.g = _dev_ptr(g, "g", allow_host)
        d.mom = _dev_ptr(mom, "mom", allow_host)
        d.row_v = _dev_ptr(rv, "row_v", allow_host)
        d.rows, d.cols = w.shape
        d.w_dtype = _dtype(w)
        d.g_dtype = _dtype(g) if g is not None else d.w_dtype
        view = e.get("view")
        if view is not None:
            if len(view) > GBO_MAX_VIEW_DIMS:
                raise ValueError("view has more than %d axes" % GBO_MAX_VIEW_DIMS)
            d.view_ndim = len(view)
            for k, s in enumerate(view):
                d.view[k] = int(s)
        split = e.get("split")
        if split is not None:
            d.n_split = len(split)
            d.split_off = len(pool)
            pool += [int(s) for s in split]
        d.lr_mult = float(e.get("lr_mult", 1.0))
        d.wd = float(e.get("wd", 0.0))
        keep += [w, g, mom, rv]
    return arr, pool, keep


def gbo_muon_plan_create(entries, *, abc=(1.5, -0.5, 0.0), ns_steps=5, mu=0.95, nesterov=True,
                         precision=GBO_NS_BF16, normuon=False, beta2=0.95, eps=1e-8, route=GBO_ROUTE_AUTO,
                         rms_target=0.0, workspace_cap=0, _query_only=False):
    """Validate a Muon table and build a plan (``abc``: one triple or one per step;
    ``route``: GBO_ROUTE_AUTO, GBO_ROUTE_X or GBO_ROUTE_GRAM; ``rms_target`` > 0
    with NorMuon: each matrix's update is scaled to that RMS; ``workspace_cap``
    > 0: the step runs the table in groups whose workspace fits the cap)."""
    L = lib()
    arr, pool, keep = muon_desc_table(entries, allow_host=_query_only)
    flat = []
    for t in ([abc] if len(abc) and not hasattr(abc[0], "__len__") else abc):
        flat += [float(x) for x in t]
    per_step = len(flat) > 3
    cabc = (c_float * len(flat))(*flat)
    opts = MuonOpts(ctypes.cast(cabc, ctypes.POINTER(c_float)), mu, beta2, eps, int(bool(nesterov)),
                    int(ns_steps), int(per_step), int(precision), int(bool(normuon)), int(route),
                    float(rms_target), 0, int(workspace_cap))
    cpool = (c_int64 * max(1, len(pool)))(*pool)
    out = c_void_p()
    _check(L.gbo_muon_plan_create(arr, len(entries), cpool, len(pool), ctypes.byref(opts), ctypes.byref(out)))
    return MuonPlan(out.value, keep, len(entries))


def gbo_muon_plan_destroy(plan):
    if plan.handle:
        lib().gbo_muon_plan_destroy(plan.handle)
        plan.handle = None


def gbo_muon_workspace_bytes(plan):
    return int(lib().gbo_muon_workspace_bytes(plan.handle))


def gbo_desc_hash(plan):
    return int(lib().gbo_desc_hash(plan.handle))


def gbo_muon_plan_info(plan):
    info = PlanInfo()
    _check(lib().gbo_muon_plan_info(plan.handle, ctypes.byref(info)))
    return {k: getattr(info, k) for k, _ in PlanInfo._fields_}


def muon_desc_flops(entries, **opts):
    """Executed Newton-Schulz FLOPs per step of every entry (host or device
    tensors), from a plan built only to be queried and then dropped."""
    plan = gbo_muon_plan_create(entries, _query_only=True, **opts)
    try:
        return gbo_muon_plan_desc_flops(plan)
    finally:
        gbo_muon_plan_destroy(plan)


def gbo_muon_plan_desc_flops(plan):
    """Executed Newton-Schulz FLOPs per step of every descriptor, in table order."""
    n = plan.n_descs
    out = (ctypes.c_double * max(1, n))()
    _check(lib().gbo_muon_plan_desc_flops(plan.handle, out, n))
    return [float(out[i]) for i in range(n)]


def gbo_muon_step(plan, lr, workspace, dbg_update=None, dev_status=None, stream=None):
    """One Muon step on ``stream`` (default: torch's current stream)."""
    ws = _dev_ptr(workspace, "workspace") if workspace is not None else None
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().gbo_muon_step(plan.handle, float(lr), ws, nbytes, _dev_ptr(dbg_update, "dbg_update"),
                               _dev_ptr(dev_status, "dev_status"), _stream(stream)))


def gbo_muon_plan_set_free_sms(plan, n):
    """Leave ``n`` SMs free of the plan's persistent Newton-Schulz kernels in
    later steps (for gbo_h2d_copy with ``n`` blocks on another stream)."""
    _check(lib().gbo_muon_plan_set_free_sms(plan.handle, int(n)))


def gbo_muon_plan_set_stats(plan, stats):
    """Per-matrix norms from later steps: ``stats`` is a float32 CUDA tensor of
    2 * n_matrices values (||D||_F, ||U||_F per matrix, table order), or None
    to stop."""
    if stats is not None and (stats.dtype != torch.float32 or stats.numel() < 2 * plan_matrices(plan)):
        raise ValueError("stats must be float32 with 2 values per matrix")
    plan._stats = stats  # kept alive while the plan writes to it
    _check(lib().gbo_muon_plan_set_stats(plan.handle, _dev_ptr(stats, "stats")))


def plan_matrices(plan):
    return gbo_muon_plan_info(plan)["n_matrices"]


def gbo_muon_plan_set_timing(plan, enable=True):
    _check(lib().gbo_muon_plan_set_timing(plan.handle, int(bool(enable))))


def gbo_muon_plan_set_event(plan, phase, event):
    """Record ``event`` (a torch.cuda.Event, or None to stop) after ``phase``
    (0 = momentum) of every later step, on the step's stream."""
    handle = None
    if event is not None:
        if not event.cuda_event:  # torch creates the CUDA event on first use
            event.record()
        handle = event.cuda_event
    _check(lib().gbo_muon_plan_set_event(plan.handle, int(phase), handle))
    plan._event = event  # keep it alive while the plan records it


def gbo_muon_plan_phase_times(plan):
    ms = (c_float * GBO_N_PHASES)()
    n = (c_int64 * GBO_N_PHASES)()
    _check(lib().gbo_muon_plan_phase_times(plan.handle, ms, n, GBO_N_PHASES))
    return {name: (float(ms[i]), int(n[i])) for i, name in enumerate(PHASE_NAMES)}


def gbo_normuon_rownorm(O, row_v, w, *, beta2, eps, scale, lr, wd=0.0, dbg_update=None, stream=None):
    rows, cols = O.shape
    if O.dtype != torch.float32:
        raise TypeError("O must be float32")
    _check(lib().gbo_normuon_rownorm(_dev_ptr(O, "O"), rows, cols, _dev_ptr(row_v, "row_v"), _dev_ptr(w, "w"),
                                     _dtype(w), float(beta2), float(eps), float(scale), float(lr), float(wd),
                                     _dev_ptr(dbg_update, "dbg_update"), _stream(stream)))


# ---------------------------------------------------------------------------
# AdamW

def gbo_clip_norm_workspace_bytes():
    return int(lib().gbo_clip_norm_workspace_bytes())


def gbo_clip_norm(grads, max_norm, total_norm, coef, workspace, dev_status=None, stream=None):
    """Global norm of ``grads`` into ``total_norm`` and the clip factor into ``coef``."""
    arr = (Tensor * max(1, len(grads)))()
    for d, g in zip(arr, grads):
        d.ptr = _dev_ptr(g, "grad")
        d.numel = g.numel()
        d.dtype = _dtype(g)
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib().gbo_clip_norm(arr, len(grads), float(max_norm), _dev_ptr(total_norm, "total_norm"),
                               _dev_ptr(coef, "coef"), _dev_ptr(dev_status, "dev_status"),
                               _dev_ptr(workspace, "workspace"), nbytes, _stream(stream)))


def gbo_clip_norm_noalloc(grads, max_norm, total_norm, coef, dev_status=None, stream=None):
    """gbo_clip_norm without a workspace: the library's fixed device scratch
    is used, so nothing is allocated (for callers that cannot allocate)."""
    arr = (Tensor * max(1, len(grads)))()
    for d, g in zip(arr, grads):
        d.ptr = _dev_ptr(g, "grad")
        d.numel = g.numel()
        d.dtype = _dtype(g)
    _check(lib().gbo_clip_norm_noalloc(arr, len(grads), float(max_norm), _dev_ptr(total_norm, "total_norm"),
                                       _dev_ptr(coef, "coef"), _dev_ptr(dev_status, "dev_status"),
                                       _stream(stream)))


def gbo_h2d_copy(dst, src, blocks=0, stream=None):
    """Copy the page-locked host tensor ``src`` into the device tensor
    ``dst`` (both contiguous, the same number of bytes) with the library's
    copy kernel (``blocks`` SMs; 0: all), asynchronously on ``stream``."""
    if not (dst.is_cuda and dst.is_contiguous()):
        raise ValueError("dst must be a contiguous CUDA tensor")
    if src.is_cuda or not src.is_contiguous():
        raise ValueError("src must be a contiguous host tensor")
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nbytes:
        raise ValueError("dst and src differ in size")
    _check(lib().gbo_h2d_copy(ctypes.c_void_p(dst.data_ptr()), ctypes.c_void_p(src.data_ptr()), nbytes,
                              int(blocks), _stream(stream)))


def gbo_adamw_step(params, *, lr, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0, step=1,
                   coef=None, dev_status=None, stream=None, dev_step=None):
    """AdamW on ``params``: a list of (p, g, m, v) tensors (p, m, v float32).
    ``dev_step``: an int32 CUDA tensor holding t, read when the kernel runs
    (for CUDA graph replay), instead of the host ``step``."""
    arr = (AdamWDesc * max(1, len(params)))()
    for d, (p, g, m, v) in zip(arr, params):
        for t, nm in ((p, "p"), (m, "m"), (v, "v")):
            if t.dtype != torch.float32:
                raise TypeError("%s must be float32" % nm)
        d.p, d.g, d.m, d.v = (_dev_ptr(p, "p"), _dev_ptr(g, "g"), _dev_ptr(m, "m"), _dev_ptr(v, "v"))
        d.numel = p.numel()
        d.g_dtype = _dtype(g)
    if dev_step is not None and dev_step.dtype != torch.int32:
        raise TypeError("dev_step must be int32")
    opts = AdamWOpts(lr, beta1, beta2, eps, weight_decay, int(step), _dev_ptr(dev_step, "dev_step"))
    _check(lib().gbo_adamw_step(arr, len(params), ctypes.byref(opts), _dev_ptr(coef, "coef"),
                                _dev_ptr(dev_status, "dev_status"), _stream(stream)))


# ---------------------------------------------------------------------------
# rotary positions and q/k norms, cross entropy of the tied classifier

def gbo_rope_frequencies(rot_dim, base=10000.0, scaling=None):
    """(frequencies, magnitude) of a rotation; ``scaling``: a RopeScaling or None."""
    freq = (ctypes.c_double * max(1, int(rot_dim) // 2))()
    magnitude = ctypes.c_double()
    _check(lib().gbo_rope_frequencies(int(rot_dim), float(base), ctypes.byref(scaling) if scaling else None, freq,
                                      ctypes.byref(magnitude)))
    return freq, magnitude.value


# The tables of the rotary calls are packed by struct (the layouts of RopeTensor
# and RopePositions): a call while answering takes microseconds on the GPU,
# and filling ctypes fields one by one takes longer than that.
_PACK_ROPE_TENSOR = struct.Struct("@5P9q4i").pack
_PACK_ROPE_POSITIONS = struct.Struct("@P3q2i").pack
_ZERO3 = (0, 0, 0)
_ELEMENT = {torch.float32: GBO_F32, torch.bfloat16: GBO_BF16}
_INDEX = {torch.int32: GBO_I32, torch.int64: GBO_I64}


def _heads_of(t, what, shape, dtype):
    """Strides of a (batch, seq, heads, dim) tensor whose head elements are consecutive."""
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError("x, dy and y differ in shape or dtype")
    s = t.stride()
    if s[3] != 1 and shape[3] > 1:
        raise ValueError("the elements of a head of %s must be consecutive" % what)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % what)
    return s[:3]


def _rope_gain(t, what, dim):
    if t is None:
        return 0
    if t.dtype != torch.float32 or t.numel() != dim:
        raise ValueError("%s must be %d float32 values" % (what, dim))
    return _dev_ptr(t, what)


def _rope_table(tensors, opts, positions):
    """Marshal a list of dicts with ``x``, ``y`` (and ``dy``, ``gain``, ``dgain``,
    ``norm``) into a table; returns it with the batch, the length and the positions."""
    dim = opts.head_dim
    batch = seq = 0
    table = b""
    for n, e in enumerate(tensors):
        y, get = e["y"], e.get
        x, dy = get("x"), get("dy")
        shape = y.shape
        if len(shape) != 4 or shape[3] != dim:
            raise ValueError("(batch, seq, heads, %d) is wanted, got %s" % (dim, tuple(shape)))
        if n == 0:
            batch, seq = shape[0], shape[1]
        elif batch != shape[0] or seq != shape[1]:
            raise ValueError("the tensors of one call have the same batch and length")
        dtype = y.dtype
        if dtype not in _ELEMENT:
            raise TypeError("tensor dtype must be float32 or bfloat16, got %s" % dtype)
        table += _PACK_ROPE_TENSOR(
            0 if x is None else x.data_ptr(), 0 if dy is None else dy.data_ptr(), y.data_ptr(),
            _rope_gain(get("gain"), "gain", dim), _rope_gain(get("dgain"), "dgain", dim),
            *(_ZERO3 if x is None else _heads_of(x, "x", shape, dtype)),
            *(_ZERO3 if dy is None else _heads_of(dy, "dy", shape, dtype)), *_heads_of(y, "y", shape, dtype), shape[2],
            _ELEMENT[dtype], 1 if get("norm") else 0, 0)
    if isinstance(positions, int):
        return table, batch, seq, _PACK_ROPE_POSITIONS(0, 0, 0, positions, GBO_I64, 0)
    index = _INDEX.get(positions.dtype)
    if index is None:
        raise TypeError("positions must be int32 or int64")
    if not positions.is_cuda:
        raise ValueError("positions must be a CUDA tensor")
    shape, stride = positions.shape, positions.stride()
    if len(shape) == 1:
        shape, stride = (1, shape[0]), (0, stride[0])
    if len(shape) != 2 or shape[1] != seq or (shape[0] != 1 and shape[0] != batch):
        raise ValueError("positions must be (seq,), (1, seq) or (batch, seq)")
    return table, batch, seq, _PACK_ROPE_POSITIONS(positions.data_ptr(), stride[0] if shape[0] == batch else 0,
                                                   stride[1], 0, index, 0)


def gbo_rope_forward(tensors, opts, positions, stream=None):
    """Rotate tensors (dicts with ``x``, ``y`` of (batch, seq, heads, dim), and
    ``norm``, ``gain``) in one launch.  ``positions``: an integer tensor (seq,)
    or (batch, seq), or the first position."""
    table, batch, seq, pos = _rope_table(tensors, opts, positions)
    _check(lib().gbo_rope_forward(table, len(tensors), ctypes.byref(opts), batch, seq, pos, _stream(stream)))


def gbo_rope_workspace_bytes(tensors, opts):
    table = b"".join(_PACK_ROPE_TENSOR(0, 0, 0, 0, 0 if e.get("dgain") is None else 4, *_ZERO3, *_ZERO3, *_ZERO3,
                                       e["dy"].shape[2], 0, 1, 0) for e in tensors)
    return int(lib().gbo_rope_workspace_bytes(table, len(tensors), ctypes.byref(opts)))


def gbo_rope_backward(tensors, opts, positions, workspace=None, stream=None):
    """Gradients: dicts with ``dy``, ``y`` (receives the input's gradient) and,
    with a norm, ``x``, ``gain`` and ``dgain``."""
    table, batch, seq, pos = _rope_table(tensors, opts, positions)
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().gbo_rope_backward(table, len(tensors), ctypes.byref(opts), batch, seq, pos,
                                   _dev_ptr(workspace, "workspace"), nbytes, _stream(stream)))


@functools.lru_cache(maxsize=256)
def gbo_xent_workspace_bytes(n, v, d, grad=False, cap=0):
    return int(lib().gbo_xent_workspace_bytes(int(n), int(v), int(d), int(bool(grad)), int(cap)))


_PACK_XENT_ARGS = struct.Struct("@5P5q2f4i").pack     # XentArgs
_PACK_XENT_GRADS = struct.Struct("@2P2q4i").pack      # XentGrads


def _rows_of(t, what, shape=None):
    """Row stride of a two-dimensional CUDA tensor with consecutive row elements."""
    s = t.shape
    if len(s) != 2 or (shape is not None and s != shape):
        raise ValueError("%s must be two-dimensional%s" % (what, "" if shape is None else " %s" % (tuple(shape),)))
    stride = t.stride()
    if stride[1] != 1 and s[1] > 1:
        raise ValueError("the row elements of %s must be consecutive" % what)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % what)
    return stride[0] if s[0] > 1 else s[1]  # (of one row any stride will do)


def _xent_args(h, w, labels, row_weight, upstream, logit_scale, z_loss, mean, keep=False):
    """The packed arguments and the number of rows."""
    h_stride, w_stride = _rows_of(h, "h"), _rows_of(w, "w")
    if h.dtype != torch.bfloat16 or w.dtype != torch.bfloat16:
        raise TypeError("h and w must be bfloat16")
    n, d = h.shape
    v, dw = w.shape
    if d != dw:
        raise ValueError("h and w differ in width")
    index = _INDEX.get(labels.dtype)
    if index is None:
        raise TypeError("labels must be int32 or int64")
    if labels.numel() != n:
        raise ValueError("one label per row of h")
    weight = _out_f32(row_weight, n, "row_weight") or 0
    up = _out_f32(upstream, 1, "upstream") or 0
    return _PACK_XENT_ARGS(h.data_ptr(), w.data_ptr(), _dev_ptr(labels, "labels"), weight, up, n, v, d, h_stride, w_stride,
                           logit_scale, z_loss, index, 1 if mean else 0, 1 if keep else 0, 0), n


def _xent_grads(dh, dw, h, w, accumulate_dw):
    dh_ptr = dw_ptr = dh_stride = dw_stride = 0
    dh_type = dw_type = GBO_BF16
    if dh is not None:
        dh_stride, dh_ptr, dh_type = _rows_of(dh, "dh", h.shape), dh.data_ptr(), _dtype(dh)
    if dw is not None:
        dw_stride, dw_ptr, dw_type = _rows_of(dw, "dw", w.shape), dw.data_ptr(), _dtype(dw)
    return _PACK_XENT_GRADS(dh_ptr, dw_ptr, dh_stride, dw_stride, dh_type, dw_type, 1 if accumulate_dw else 0, 0)


def _out_f32(t, count, what):
    if t is not None and (t.dtype != torch.float32 or t.numel() != count):
        raise ValueError("%s must be %d float32 values" % (what, count))
    return _dev_ptr(t, what)


def gbo_xent_forward(h, w, labels, workspace, *, loss=None, lse=None, totals=None, row_weight=None, logit_scale=1.0,
                     z_loss=0.0, keep=False, dev_status=None, stream=None):
    """Cross entropy of each row of ``h`` @ ``w``.T against ``labels`` into ``loss``,
    ``lse`` (n) and ``totals`` (2), whichever are given.  ``keep``: leave the logits
    in the workspace (of ``grad`` size) for gbo_xent_backward."""
    a, n = _xent_args(h, w, labels, row_weight, None, logit_scale, z_loss, True, keep)
    _check(lib().gbo_xent_forward(a, _out_f32(loss, n, "loss"), _out_f32(lse, n, "lse"),
                                  _out_f32(totals, 2, "totals"), _dev_ptr(workspace, "workspace"),
                                  workspace.numel() * workspace.element_size(), _dev_ptr(dev_status, "dev_status"),
                                  _stream(stream)))


def gbo_xent_backward(h, w, labels, lse, workspace, *, dh=None, dw=None, accumulate_dw=False, row_weight=None,
                      upstream=None, mean=True, logit_scale=1.0, z_loss=0.0, keep=False, dev_status=None, stream=None):
    """Gradients into ``dh`` and ``dw`` from the forward's ``lse`` (``keep``: and the
    logits that a forward with ``keep`` left in this workspace)."""
    a, n = _xent_args(h, w, labels, row_weight, upstream, logit_scale, z_loss, mean, keep)
    g = _xent_grads(dh, dw, h, w, accumulate_dw)
    _check(lib().gbo_xent_backward(a, _out_f32(lse, n, "lse"), g,
                                   _dev_ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(),
                                   _dev_ptr(dev_status, "dev_status"), _stream(stream)))


def gbo_xent_grad(h, w, labels, workspace, *, loss=None, lse=None, totals=None, dh=None, dw=None,
                  accumulate_dw=False, row_weight=None, upstream=None, mean=True, logit_scale=1.0, z_loss=0.0,
                  dev_status=None, stream=None):
    """Losses and gradients in one call."""
    a, n = _xent_args(h, w, labels, row_weight, upstream, logit_scale, z_loss, mean)
    g = _xent_grads(dh, dw, h, w, accumulate_dw)
    _check(lib().gbo_xent_grad(a, _out_f32(loss, n, "loss"), _out_f32(lse, n, "lse"),
                               _out_f32(totals, 2, "totals"), g, _dev_ptr(workspace, "workspace"),
                               workspace.numel() * workspace.element_size(), _dev_ptr(dev_status, "dev_status"),
                               _stream(stream)))


# ---------------------------------------------------------------------------
# diagnostics

def gbo_last_error():
    return lib().gbo_last_error().decode()


def gbo_abi_version():
    return int(lib().gbo_abi_version())


def gbo_struct_size(which):
    return int(lib().gbo_struct_size(which))


def gbo_testing_set_small_chain(enable):
    """Whether plans created from now on run the Gram route's p x p
    iterations of matrices with p <= 192 (bf16) in one on-chip chain launch.
    Returns the previous setting."""
    return bool(lib().gbo_testing_set_small_chain(1 if enable else 0))


def gbo_testing_set_fused_gram(enable):
    """Whether plans created from now on run the Gram of the chain's wide
    matrices with p <= 128 inside the chain launch (X_0 streamed through
    shared memory) rather than as a launch of its own.  Returns the previous
    setting."""
    return bool(lib().gbo_testing_set_fused_gram(1 if enable else 0))


def gbo_testing_set_fused_momentum(enable):
    """Whether plans created from now on run the momentum pass of the chain's
    wide p <= 128 matrices with bf16 gradients inside the chain launch (G and
    B streamed through shared memory) rather than in the momentum kernel
    (the default).  Returns the previous setting."""
    return bool(lib().gbo_testing_set_fused_momentum(1 if enable else 0))


def gbo_testing_set_tail_split(enable):
    """Whether launches of the bf16 CTA-pair kernel from now on run a last
    wave of at most half the resident pairs as 256 x 128 half tiles (the
    default).  Returns the previous setting."""
    return bool(lib().gbo_testing_set_tail_split(1 if enable else 0))


def gbo_testing_set_momentum_stream(enable):
    """Whether momentum passes from now on stream their tiles through shared
    memory where the plan allows it (the default) or take the register
    kernel; the results are bitwise the same.  Returns the previous
    setting."""
    return bool(lib().gbo_testing_set_momentum_stream(1 if enable else 0))


def gbo_testing_pair_residency():
    """CTA pairs of the bf16 Newton-Schulz kernel the current device holds at
    once (its pair launches' persistent grid)."""
    return int(lib().gbo_testing_pair_residency())


def gbo_testing_set_pdl(mode):
    """When launches from now on carry the programmatic-dependent-launch
    attribute: 0 never, 1 always, 2 (the default) in CUDA graph capture only.
    Returns the previous mode."""
    return int(lib().gbo_testing_set_pdl(int(mode)))


def gbo_testing_wait_timeout(dev_status, limit_us, stream=None):
    """Test hook: the GEMM's bounded wait on a barrier nothing arrives on."""
    _check(lib().gbo_testing_wait_timeout(_dev_ptr(dev_status, "dev_status"), int(limit_us), _stream(stream)))


def gbo_launch_count():
    return int(lib().gbo_launch_count())
