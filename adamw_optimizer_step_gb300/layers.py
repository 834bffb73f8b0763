"""Torch-facing calls of the operators around the optimizer step: rotary
positions, per-head q/k norms with rotation, attention, the residual update with
the norms around it, dropout, and the tied classifier's cross entropy, each with
its gradients.

Each allocates its outputs and scratch with torch's allocator and makes one
library call, on torch's current stream (under ``torch.cuda.stream(s)`` both the
memory and the work belong to ``s``; the binding's functions take a stream and
the caller's buffers).  No call waits for the GPU, so what is found there is told
in ``dev_status`` alone, a CUDA int32 of the caller's that the cross entropy,
attention and the residual update OR their ``GBO_STATUS_*`` bits into: without one,
a label outside the vocabulary leaves its row out and a wait that ran out
(``GBO_STATUS_TIMEOUT``, outputs invalid) goes unnoticed.  ``rotary_autograd``,
``qk_norm_rotary_autograd``, ``attention_autograd``, ``residual_norm_autograd``,
``dropout_autograd`` and ``linear_cross_entropy_loss`` are the same operators inside
autograd, so that ``loss.backward()`` leaves the gradients that
:class:`~.routing.HybridOptimizer` steps.  A captured backward pass must find no graph of an
eager one alive that accumulates into the same leaves (torch would leave the capture for
that one's stream).

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
# attention

def attention(q, k, v, *, causal=True, window=0, scale=None, q_lengths=None, k_lengths=None, documents=None, out=None,
              return_lse=False, dev_status=None):
    """Softmax attention of ``q`` (batch, sq, q_heads, dk) over ``k`` and ``v`` (batch,
    sk, k_heads, dk and dv), all bfloat16: a training batch, a prompt, or single
    tokens (sq = 1) over a cache.  ``q_heads`` is a multiple of ``k_heads``.

    ``causal``: the last query of a sequence sees all its keys, each one before it
    a key less; ``window`` > 0: only the last ``window`` of these.  ``q_lengths``,
    ``k_lengths``: int32 CUDA tensors (batch), what each sequence of a padded batch,
    or its cache, holds.  ``documents``: int32 CUDA tensor, the first tokens of
    sequences packed into one row and the end of the last.  ``scale``: of the
    scores, 1 / sqrt(dk) by default.  Queries that see nothing get 0.

    With ``return_lse`` also the log of each row's sum (batch, sq, q_heads), which
    :func:`attention_backward` takes."""
    args = B.attn_args(q, k, v, causal=causal, window=window, scale=scale, q_lengths=q_lengths, k_lengths=k_lengths,
                       documents=documents)
    shape = q.shape
    if out is not None:
        y = out
    else:
        y = _like(q) if shape[3] == v.shape[3] else q.new_empty((*shape[:3], v.shape[3]))
    lse = torch.empty(shape[:3], dtype=torch.float32, device=q.device) if return_lse else None
    need = B.gbo_attn_forward_workspace_bytes(args)
    ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    B.gbo_attn_forward(args, q, v, y, ws, lse=lse, dev_status=dev_status)
    return (y, lse) if return_lse else y


def attention_backward(dy, q, k, v, y, lse, *, causal=True, window=0, scale=None, q_lengths=None, k_lengths=None,
                       documents=None, wanted=(True, True, True), dev_status=None):
    """Gradients of :func:`attention` by q, k and v (None where not ``wanted``) from its
    output ``y``, its ``lse`` and the gradient ``dy``; the same masks as there."""
    args = B.attn_args(q, k, v, causal=causal, window=window, scale=scale, q_lengths=q_lengths, k_lengths=k_lengths,
                       documents=documents)
    dq, dk, dv = _like(q) if wanted[0] else None, _like(k) if wanted[1] else None, _like(v) if wanted[2] else None
    need = B.gbo_attn_backward_workspace_bytes(args)
    ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    B.gbo_attn_backward(args, q, k, v, dy, y, lse, ws, dq=dq, dk=dk, dv=dv, dev_status=dev_status)
    return dq, dk, dv


# ---------------------------------------------------------------------------
# the residual update between two blocks, dropout

def _flat(t):
    """Rows of the last axis, as a two-dimensional view where strides allow it."""
    return t if t is None or t.dim() == 2 else t.reshape(-1, t.shape[-1])


def residual_norm(x, block=None, *, post_norm=False, pre_norm=True, post_gain=None, pre_gain=None, gate=None,
                  gate_kind="sigmoid", scale=None, dropout=0.0, seed=0, offset=0, eps=1e-6, x_out=None,
                  dev_status=None):
    """(x', h): the residual stream ``x`` (..., d) after a block's output ``block``, and
    the next block's input, in one pass:

        u = block, normed with ``post_norm`` (root mean square, times ``post_gain``)
        x' = x + scale * gate * dropout(u);  h = x' normed with ``pre_norm``, times ``pre_gain``

    ``gate``: (..., d) or (..., 1), through a sigmoid or (``gate_kind="linear"``) as it
    is; ``scale``: float32, one value or d; gains: float32, d, or None for ones.
    ``dropout``: its probability, drawn from ``seed`` (an int, or a CUDA int64 tensor
    that is read when the kernel runs) and ``offset``, see ``gbo_residual_args``.
    ``block=None``: the norm alone, and x' is ``x``.  ``x`` and ``block`` are bfloat16 or
    float32, ``block`` bfloat16 where ``x`` is; ``h`` has the dtype of ``block``.
    ``x_out`` (with a block's output) may be ``x``.  Without ``pre_norm`` h is None."""
    if block is None and x_out is not None:
        raise ValueError("x_out without a block's output: the stream stays as it is")
    flat = x.dim() == 2
    x2, b2, g2 = (x, block, gate) if flat else (_flat(x), _flat(block), _flat(gate))
    bt = x.dtype if block is None else block.dtype
    args = B.residual_args(x2, b2, post_norm=post_norm, pre_norm=pre_norm, post_gain=post_gain, pre_gain=pre_gain,
                           gate=g2, gate_kind=gate_kind, scale=scale, dropout=dropout, seed=seed, offset=offset, eps=eps)
    shape = x2.shape
    if block is None:
        xo = None
    else:
        xo = _like(x2) if x_out is None else x_out if flat else x_out.view(shape)
    h = _like(x2, dtype=bt) if pre_norm else None
    B.gbo_residual_forward(args, xo, h, shape, x.dtype, bt, dev_status)
    if flat:
        return x if xo is None else xo, h
    return x if xo is None else xo.view(x.shape), None if h is None else h.view(x.shape)


def residual_norm_backward(dx_out, dh, x_new, block=None, *, post_norm=False, pre_norm=True, post_gain=None,
                           pre_gain=None, gate=None, gate_kind="sigmoid", scale=None, dropout=0.0, seed=0, offset=0,
                           eps=1e-6, wanted=("dx", "dblock", "dgate", "dscale", "dpost_gain", "dpre_gain"), dev_status=None):
    """Gradients of :func:`residual_norm` from those of x' (``dx_out``, None for none) and
    of h (``dh``), the updated stream ``x_new`` and the block's output: a dict with
    ``dx``, ``dblock``, ``dgate``, ``dscale``, ``dpost_gain`` and ``dpre_gain`` (None for
    what was not given or is not ``wanted``)."""
    flat = x_new.dim() == 2
    x2, b2, g2, dx2, dh2 = ((x_new, block, gate, dx_out, dh) if flat else
                            (_flat(x_new), _flat(block), _flat(gate), _flat(dx_out), _flat(dh)))
    bt = x_new.dtype if block is None else block.dtype
    args = B.residual_args(x2, b2, post_norm=post_norm, pre_norm=pre_norm, post_gain=post_gain, pre_gain=pre_gain,
                           gate=g2, gate_kind=gate_kind, scale=scale, dropout=dropout, seed=seed, offset=offset, eps=eps)
    like = {"dx": x2, "dblock": b2, "dgate": g2, "dscale": scale, "dpost_gain": post_gain, "dpre_gain": pre_gain}
    out = {k: _like(t) if t is not None and k in wanted else None for k, t in like.items()}
    sums = (out["dscale"] is not None) + (out["dpost_gain"] is not None) + (out["dpre_gain"] is not None)
    shape, ws = x2.shape, None
    if sums:
        ws = torch.empty(B._residual_workspace(*shape, sums, x2.device), dtype=torch.uint8, device=x2.device)
    B.gbo_residual_backward(args, ws, shape, x_new.dtype, bt, dx_out=dx2, dh=dh2, dev_status=dev_status, **out)
    if not flat:
        for k, t in (("dx", x_new), ("dblock", block), ("dgate", gate)):
            if out[k] is not None:
                out[k] = out[k].view(t.shape)
    return out


def dropout(x, p, seed, *, offset=0, out=None):
    """``x`` with elements dropped with probability ``p`` (a multiple of 2^-16) and the
    others divided by the share kept.  Which ones follows from ``seed`` (an int, or a
    CUDA int64 tensor that is read when the kernel runs), ``offset`` and an element's
    place alone: no mask is kept, and the same call on a gradient is the gradient.  Rows
    of a two-dimensional ``x`` may lie apart; other strides are copied together first."""
    flat = x.dim() == 2
    rows = x if flat else x.reshape(1, -1)  # (a view where it can be, with any stride)
    (n, d), (by, apart) = rows.shape, rows.stride()
    if (apart != 1 and d > 1) or (by < d and n > 1):
        rows = rows.contiguous()
    if flat:
        y = _like(rows) if out is None else out
        B.gbo_dropout(rows, y, p, seed, offset)
        return y
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device) if out is None else out
    B.gbo_dropout(rows, y.view(1, -1), p, seed, offset)
    return y


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


def _aligned_heads(t):
    """``t`` as attention takes it: consecutive head elements, positive strides of whole
    16-byte pieces (autograd hands over expanded gradients and slices of any place)."""
    s, n = t.stride(), t.shape
    ok = s[3] == 1 and t.data_ptr() % 16 == 0 and all(n[i] <= 1 or (s[i] > 0 and s[i] % 8 == 0) for i in range(3))
    return t if ok else t.clone(memory_format=torch.contiguous_format)


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, q_lengths, k_lengths, documents, causal, window, scale, dev_status):
        mask = dict(causal=causal, window=window, scale=scale)
        y, lse = attention(q, k, v, q_lengths=q_lengths, k_lengths=k_lengths, documents=documents, return_lse=True,
                           dev_status=dev_status, **mask)
        ctx.rest = (mask, dev_status)
        ctx.save_for_backward(q, k, v, y, lse, q_lengths, k_lengths, documents)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        q, k, v, y, lse, q_lengths, k_lengths, documents = ctx.saved_tensors
        mask, dev_status = ctx.rest
        grads = attention_backward(_aligned_heads(dy), q, k, v, y, lse, q_lengths=q_lengths, k_lengths=k_lengths,
                                   documents=documents, wanted=ctx.needs_input_grad[:3], dev_status=dev_status, **mask)
        return (*grads, None, None, None, None, None, None, None)


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, block, gate, scale, post_gain, pre_gain, seed, rest):
        ctx.set_materialize_grads(False)
        x_new, h = residual_norm(x, block, gate=gate, scale=scale, post_gain=post_gain, pre_gain=pre_gain, seed=seed,
                                 **rest)
        ctx.rest = rest
        ctx.host_seed = None if isinstance(seed, torch.Tensor) else seed
        ctx.save_for_backward(x_new, block, gate, scale, post_gain, pre_gain, seed if ctx.host_seed is None else None)
        return x_new, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dx_out, dh):
        if dx_out is None and dh is None:
            return (None,) * 8
        x_new, block, gate, scale, post_gain, pre_gain, seed = ctx.saved_tensors
        rest = dict(ctx.rest, seed=seed if ctx.host_seed is None else ctx.host_seed)
        names = ("dx", "dblock", "dgate", "dscale", "dpost_gain", "dpre_gain")
        wanted = [n for n, need in zip(names, ctx.needs_input_grad) if need]
        if dh is None:  # nothing comes through the norm behind the update
            rest["pre_norm"], pre_gain = False, None
        d = x_new.shape[-1]
        rows = lambda t: None if t is None else _rows(_flat(t))  # noqa: E731
        dx_out, dh = (t if t is None or t.stride(0) >= d else t.contiguous() for t in (rows(dx_out), rows(dh)))
        g = residual_norm_backward(dx_out, dh, x_new, block, gate=gate, scale=scale, post_gain=post_gain,
                                   pre_gain=pre_gain, wanted=wanted, **rest)
        return (*(g[n] for n in names), None, None)


class _Norm(torch.autograd.Function):
    """The norm alone: the residual update without a block."""

    @staticmethod
    def forward(ctx, x, gain, eps, dev_status):
        ctx.rest = dict(eps=eps, dev_status=dev_status)
        ctx.save_for_backward(x, gain)
        return residual_norm(x, pre_gain=gain, **ctx.rest)[1]

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        x, gain = ctx.saved_tensors
        wanted = [n for n, need in zip(("dx", "dpre_gain"), ctx.needs_input_grad) if need]
        dh = _rows(_flat(dh))
        dh = dh if dh.stride(0) >= x.shape[-1] else dh.contiguous()
        g = residual_norm_backward(None, dh, x, pre_gain=gain, wanted=wanted, **ctx.rest)
        return g["dx"], g["dpre_gain"], None, None


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, p, seed, offset):
        ctx.rest = (p, offset)
        ctx.host_seed = None if isinstance(seed, torch.Tensor) else seed
        ctx.save_for_backward(seed if ctx.host_seed is None else None)
        return dropout(x, p, seed, offset=offset)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        p, offset = ctx.rest
        seed = ctx.saved_tensors[0] if ctx.host_seed is None else ctx.host_seed
        return dropout(dy.contiguous(), p, seed, offset=offset), None, None, None


def attention_autograd(q, k, v, *, causal=True, window=0, scale=None, q_lengths=None, k_lengths=None, documents=None,
                       dev_status=None):
    """:func:`attention` with its gradients by q, k and v.  ``scale`` is a constant."""
    _constant(scale, "scale")
    return _Attention.apply(q, k, v, q_lengths, k_lengths, documents, bool(causal), int(window),
                            None if scale is None else float(scale), dev_status)


def residual_norm_autograd(x, block=None, *, post_norm=False, pre_norm=True, post_gain=None, pre_gain=None, gate=None,
                           gate_kind="sigmoid", scale=None, dropout=0.0, seed=0, offset=0, eps=1e-6, dev_status=None):
    """:func:`residual_norm` with its gradients by the stream, the block's output, the gate,
    the scale and the gains.  Between the passes x' is kept, and no mask; ``dropout`` and
    ``eps`` are constants."""
    _constant(dropout, "dropout")
    _constant(eps, "eps")
    if block is None:
        if post_norm or not pre_norm or gate is not None or scale is not None or post_gain is not None or float(dropout):
            raise ValueError("without a block's output there is the norm alone")
        return x, _Norm.apply(x, pre_gain, float(eps), dev_status)
    rest = dict(post_norm=bool(post_norm), pre_norm=bool(pre_norm), gate_kind=gate_kind, dropout=float(dropout),
                offset=int(offset), eps=float(eps), dev_status=dev_status)
    return _ResidualNorm.apply(x, block, gate, scale, post_gain, pre_gain, seed, rest)


def dropout_autograd(x, p, seed, *, offset=0):
    """:func:`dropout` with its gradient (the same elements, drawn again)."""
    _constant(p, "p")
    return _Dropout.apply(x, float(p), seed, int(offset))


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
