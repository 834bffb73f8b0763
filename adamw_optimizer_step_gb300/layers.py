"""Torch-facing calls of the operators around the optimizer step: rotary
positions, per-head q/k norms with rotation, and the tied classifier's cross
entropy with its gradients.

Each allocates its outputs and scratch with torch's allocator and makes one
library call, on torch's current stream (under ``torch.cuda.stream(s)`` both the
memory and the work belong to ``s``; the binding's functions take a stream and
the caller's buffers).  No call waits for the GPU, so what is found there is told
in ``dev_status`` alone, a CUDA int32 of the caller's that the cross entropy ORs
its ``GBO_STATUS_*`` bits into: without one, a label outside the vocabulary
leaves its row out and a wait that ran out (``GBO_STATUS_TIMEOUT``, outputs invalid)
goes unnoticed.  ``rotary_autograd``, ``qk_norm_rotary_autograd``
and ``linear_cross_entropy_loss`` are the same operators inside autograd, so
that ``loss.backward()`` leaves the gradients that
:class:`~.routing.HybridOptimizer` steps.

Heads are (batch, seq, heads, dim) tensors whose last axis is contiguous; any
other strides are taken as they are (slices of a fused projection, or a
transposed (batch, heads, seq, dim) tensor).  Positions are an integer tensor
(seq,) or (batch, seq), or an int, the first position.
"""

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import _binding as B

LAYOUTS = {"half": B.GBO_ROPE_HALF, "interleaved": B.GBO_ROPE_INTERLEAVED}
SCALINGS = {"none": B.GBO_ROPE_SCALE_NONE, "linear": B.GBO_ROPE_SCALE_LINEAR, "ntk": B.GBO_ROPE_SCALE_NTK,
            "yarn": B.GBO_ROPE_SCALE_YARN, "wavelength": B.GBO_ROPE_SCALE_WAVELENGTH}


class RotarySpec:
    """A rotation's layout and frequencies, built once and kept by the model.

    ``rot_dim`` elements from ``offset`` on are rotated (default: the whole
    head).  ``scaling``: None, or a dict with ``kind`` ("linear", "ntk", "yarn",
    "wavelength") and its ``factor``, ``trained`` (length), ``fast``, ``slow``
    (turns); see ``gbo_rope_scaling``.  ``frequencies``: radians per position,
    instead of base and scaling.
    """

    def __init__(self, head_dim, rot_dim=None, offset=0, layout="half", base=10000.0, scaling=None, frequencies=None,
                 magnitude=1.0):
        self._made_of = (head_dim, rot_dim, offset, layout, base, scaling, frequencies, magnitude)
        self.head_dim = int(head_dim)
        self.rot_dim = self.head_dim - int(offset) if rot_dim is None else int(rot_dim)
        if layout not in LAYOUTS:
            raise ValueError("layout must be one of %s" % ", ".join(sorted(LAYOUTS)))
        if frequencies is not None:
            if scaling is not None or len(frequencies) != self.rot_dim // 2:
                raise ValueError("one frequency per pair, and no scaling beside them")
            self._freq = (ctypes.c_double * max(1, len(frequencies)))(*[float(f) for f in frequencies])
            self.magnitude = float(magnitude)
        elif self.rot_dim == 0:
            self._freq, self.magnitude = (ctypes.c_double * 1)(), 1.0
        else:
            s = None
            if scaling is not None:
                if scaling.get("kind") not in SCALINGS:
                    raise ValueError("scaling kind must be one of %s" % ", ".join(sorted(SCALINGS)))
                s = B.RopeScaling(SCALINGS[scaling["kind"]], 0, *(float(scaling.get(k, 0.0)) for k in
                                                                  ("factor", "trained", "fast", "slow")))
            self._freq, self.magnitude = B.gbo_rope_frequencies(self.rot_dim, base, s)
        self.opts = B.RopeOpts(self.head_dim, self.rot_dim, int(offset), LAYOUTS[layout],
                               ctypes.cast(self._freq, ctypes.POINTER(ctypes.c_double)), self.magnitude, 0.0)
        self._eps, self._scratch = {}, {}  # options by eps, scratch sizes by heads

    def __reduce__(self):  # a model that holds one can be copied and saved
        return RotarySpec, self._made_of

    @property
    def frequencies(self):
        return [self._freq[j] for j in range(self.rot_dim // 2)]

    def with_eps(self, eps):
        """The options with the norm's eps (the same frequencies)."""
        eps = float(eps)  # a tensor's value, not the tensor, is the key
        o = self._eps.get(eps)
        if o is None:
            o = self.opts
            o = self._eps[eps] = B.RopeOpts(o.head_dim, o.rot_dim, o.offset, o.layout, o.freq, o.magnitude, eps)
        return o

    def backward_workspace(self, table):
        """Scratch bytes of the gains' gradients for a table's numbers of heads (and its device)."""
        key = (table[0]["dy"].device, *((e["dy"].shape[2], e["dgain"] is not None) for e in table))
        need = self._scratch.get(key)
        if need is None:
            need = self._scratch[key] = max(16, B.gbo_rope_workspace_bytes(table, self.opts))
        return need


_like = torch.empty_like


def rotary(x, positions, spec, *, inverse=False, out=None):
    """``x`` rotated (``inverse``: turned back, which is the rotation's gradient).
    ``out`` may be ``x``."""
    y = _like(x) if out is None else out
    if inverse:
        B.gbo_rope_backward([dict(dy=x, y=y)], spec.opts, positions)
    else:
        B.gbo_rope_forward([dict(x=x, y=y)], spec.opts, positions)
    return y


def qk_norm_rotary(q, k, q_gain, k_gain, positions, spec, *, eps=1e-6):
    """Queries and keys normed per head (root mean square, gain of head_dim float32
    values or None) and rotated, in one launch."""
    yq, yk = _like(q), _like(k)
    B.gbo_rope_forward([dict(x=q, y=yq, gain=q_gain, norm=True), dict(x=k, y=yk, gain=k_gain, norm=True)],
                       spec.with_eps(eps), positions)
    return yq, yk


def qk_norm_rotary_backward(dq_out, dk_out, q, k, q_gain, k_gain, positions, spec, *, eps=1e-6):
    """Gradients of :func:`qk_norm_rotary` by q, k and the gains (None where the gain is)."""
    dq, dk = _like(q), _like(k)
    dgq = torch.empty_like(q_gain) if q_gain is not None else None
    dgk = torch.empty_like(k_gain) if k_gain is not None else None
    table = [dict(x=q, dy=dq_out, y=dq, gain=q_gain, dgain=dgq, norm=True),
             dict(x=k, dy=dk_out, y=dk, gain=k_gain, dgain=dgk, norm=True)]
    opts = spec.with_eps(eps)
    ws = torch.empty(spec.backward_workspace(table), dtype=torch.uint8, device=q.device)
    B.gbo_rope_backward(table, opts, positions, ws)
    return dq, dk, dgq, dgk


def linear_cross_entropy(h, w, labels, *, z_loss=0.0, logit_scale=1.0, lse=None, totals=None, row_weight=None,
                         dev_status=None):
    """Loss of each row of ``h`` (n x d, bf16) against ``labels`` under the classifier
    ``w`` (v x d, bf16); rows with negative labels are left out (loss 0)."""
    n, d = h.shape
    loss = torch.empty(n, dtype=torch.float32, device=h.device)
    ws = torch.empty(B.gbo_xent_workspace_bytes(n, w.shape[0], d), dtype=torch.uint8, device=h.device)
    B.gbo_xent_forward(h, w, labels, ws, loss=loss, lse=lse, totals=totals, row_weight=row_weight,
                       logit_scale=logit_scale, z_loss=z_loss, dev_status=dev_status)
    return loss


def linear_cross_entropy_grad(h, w, labels, *, z_loss=0.0, logit_scale=1.0, mean=True, row_weight=None, upstream=None,
                              dh=None, dw=None, accumulate_dw=False, totals=None, workspace_cap=0, dev_status=None):
    """(losses, dh, dw): the losses of :func:`linear_cross_entropy` and the gradients
    of their (weighted) mean, or sum with ``mean=False``, by ``h`` and ``w``, in one
    call.  ``dh``, ``dw``: buffers to write (bf16 or float32; with ``accumulate_dw``
    dw is added to).  ``workspace_cap``: bytes of scratch at most (more pieces of the
    vocabulary).  Without a cap the logits are kept in 16 bits, up to 8 GiB; see
    ``gbo_xent_workspace_bytes``."""
    n, d = h.shape
    loss = torch.empty(n, dtype=torch.float32, device=h.device)
    dh = _like(h) if dh is None else dh
    dw = _like(w) if dw is None else dw
    ws = torch.empty(B.gbo_xent_workspace_bytes(n, w.shape[0], d, True, workspace_cap), dtype=torch.uint8,
                     device=h.device)
    B.gbo_xent_grad(h, w, labels, ws, loss=loss, totals=totals, dh=dh, dw=dw, accumulate_dw=accumulate_dw,
                    row_weight=row_weight, upstream=upstream, mean=mean, logit_scale=logit_scale, z_loss=z_loss,
                    dev_status=dev_status)
    return loss, dh, dw


# ---------------------------------------------------------------------------
# autograd

def _rows(t):
    """``t`` with consecutive last-axis elements (autograd hands over expanded gradients)."""
    return t if t.stride(-1) == 1 or t.shape[-1] == 1 else t.contiguous()


def _constant(value, what):
    """Refuse a tensor whose gradient the caller waits for and would not get."""
    if isinstance(value, torch.Tensor) and value.requires_grad and torch.is_grad_enabled():
        raise ValueError("%s has no gradient here: detach it" % what)


def _save_positions(ctx, positions, *tensors):
    """Saved as a tensor, so that autograd notices positions that change before the
    backward pass; an int is kept beside it."""
    ctx.start = positions if isinstance(positions, int) else None
    ctx.save_for_backward(None if ctx.start is not None else positions, *tensors)


def _saved_positions(ctx):
    positions, *tensors = ctx.saved_tensors
    return (positions if ctx.start is None else ctx.start, *tensors)


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, positions, spec):
        ctx.spec = spec
        _save_positions(ctx, positions)
        return rotary(x, positions, spec)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        return rotary(_rows(dy), _saved_positions(ctx)[0], ctx.spec, inverse=True), None, None


class _QkNormRotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_gain, k_gain, positions, spec, eps):
        ctx.rest = (spec, eps)
        _save_positions(ctx, positions, q, k, q_gain, k_gain)
        return qk_norm_rotary(q, k, q_gain, k_gain, positions, spec, eps=eps)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        spec, eps = ctx.rest
        positions, *saved = _saved_positions(ctx)
        grads = qk_norm_rotary_backward(_rows(dq), _rows(dk), *saved, positions, spec, eps=eps)
        return (*grads, None, None, None)


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, w, labels, row_weight, z_loss, logit_scale, workspace_cap, dev_status, grad):
        n, d = h.shape
        wb = w.to(torch.bfloat16)
        lse = torch.empty(n, dtype=torch.float32, device=h.device)
        totals = torch.empty(2, dtype=torch.float32, device=h.device)
        ws = torch.empty(B.gbo_xent_workspace_bytes(n, w.shape[0], d, grad, workspace_cap), dtype=torch.uint8,
                         device=h.device)
        B.gbo_xent_forward(h, wb, labels, ws, lse=lse, totals=totals, row_weight=row_weight, logit_scale=logit_scale,
                           z_loss=z_loss, keep=grad, dev_status=dev_status)
        ctx.save_for_backward(h, wb, labels, row_weight, lse)
        ctx.rest = (z_loss, logit_scale, workspace_cap, w.dtype, ws, dev_status)
        return torch.where(totals[1] != 0, totals[0] / totals[1], torch.zeros_like(totals[0]))

    @staticmethod
    @once_differentiable
    def backward(ctx, up):
        h, w, labels, row_weight, lse = ctx.saved_tensors
        z_loss, logit_scale, workspace_cap, w_dtype, ws, dev_status = ctx.rest
        keep = ws is not None
        # the first pass uses the kept logits up; another one (retain_graph) forms them again
        ctx.rest = (z_loss, logit_scale, workspace_cap, w_dtype, None, dev_status)
        if not keep:
            ws = torch.empty(B.gbo_xent_workspace_bytes(h.shape[0], *w.shape, True, workspace_cap), dtype=torch.uint8,
                             device=h.device)
        dh = _like(h) if ctx.needs_input_grad[0] else None
        dw = torch.empty(w.shape, dtype=w_dtype, device=w.device) if ctx.needs_input_grad[1] else None
        B.gbo_xent_backward(h, w, labels, lse, ws, dh=dh, dw=dw, row_weight=row_weight,
                            upstream=up.float().reshape(1), logit_scale=logit_scale, z_loss=z_loss, keep=keep,
                            dev_status=dev_status)
        return dh, dw, None, None, None, None, None, None, None


def rotary_autograd(x, positions, spec):
    """:func:`rotary` with its gradient."""
    return _Rotary.apply(x, positions, spec)


def qk_norm_rotary_autograd(q, k, q_gain, k_gain, positions, spec, eps=1e-6):
    """:func:`qk_norm_rotary` with its gradients by q, k and the gains."""
    _constant(eps, "eps")
    return _QkNormRotary.apply(q, k, q_gain, k_gain, positions, spec, float(eps))


def linear_cross_entropy_loss(h, w, labels, row_weight=None, z_loss=0.0, logit_scale=1.0, workspace_cap=0,
                              dev_status=None):
    """Mean loss over the rows that count, with its gradients by ``h`` (bf16) and ``w``
    (bf16, or a float32 master table, which is cast for the products and gets a
    float32 gradient).  Between the passes the workspace (``workspace_cap``) keeps the
    logits in 16 bits where it has room for them; under ``torch.no_grad()``, or when neither
    requires a gradient, it is that of :func:`linear_cross_entropy`.  ``dev_status``: a
    CUDA int32 for the status bits of both passes.  ``row_weight``, ``z_loss`` and
    ``logit_scale`` are constants: refused when they require a gradient."""
    _constant(row_weight, "row_weight")
    _constant(z_loss, "z_loss")
    _constant(logit_scale, "logit_scale")
    # (within apply grad mode is off, and ctx.needs_input_grad says what requires a gradient
    # whether or not a backward pass can follow)
    grad = torch.is_grad_enabled() and (h.requires_grad or w.requires_grad)
    return _LinearCrossEntropy.apply(h, w, labels, row_weight, float(z_loss), float(logit_scale), workspace_cap,
                                     dev_status, grad)
