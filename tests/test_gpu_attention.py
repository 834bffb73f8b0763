"""Attention and its gradients against the formulas in 64 bits.

Tolerances, u = 2^-24.  A score is a sum of dk products of bf16 values (exact in
fp32) accumulated in fp32 by the tensor core: off by at most D = 2 dk u sum |q k|
scale (2: its own order and rounding of partial sums).  A probability inherits
e = D + 64 u (|s| + |lse| + 1) relative (its exponent's rounding and the
exponential), and is rounded to bf16 (2^-8 of it) as an operand of a product,
unrounded in the sum.  A product of K terms accumulated in fp32 adds 2 K u of the sum
of the terms' sizes, a bf16 output 2^-8 of its value.  So, sums over keys j,
    y    sum p (2^-8 + e + 2 K u) |v| + |y| (max e + K u)
    lse  max e + (K + 64) u (|lse| + 1)
Gradients take p = exp(s - lse), relative e' = e + tol(lse), the rounded y in
D_i = dy_i y_i, off by d = sum |dy| (tol(y) + 2^-8 |y| + 2 dv u |y|), and dP, off
by E = 2 dv u sum |dy v|:
    ds   p (E + d) + |ds| (e' + 2^-8 (1 + 2^-7)) + 8 u p (|dP| + |D|)
    dq   scale (sum tol(ds) |k| + 2 K u sum |ds k|), dk likewise over rows and heads
    dv   sum p (2^-8 + e' + 2 K u) |dy|
Bounds are summed as sizes, so they are far from what rounding does on average, and
near enough to see a wrong key, row or head."""

import math

import pytest
import torch

from adamw_optimizer_step_gb300 import _binding as B
from adamw_optimizer_step_gb300 import layers

pytestmark = pytest.mark.gpu
U, R = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def built():
    from adamw_optimizer_step_gb300 import build
    build.build()
    B.lib()


def heads(gen, batch, seq, h, d, size=1.0):
    return (size * torch.randn(batch, seq, h, d, generator=gen)).to(torch.bfloat16).cuda()


def inputs(batch, sq, sk, hq, hk, dk, dv, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return (heads(gen, batch, sq, hq, dk, 1.2), heads(gen, batch, sk, hk, dk, 1.2), heads(gen, batch, sk, hk, dv, 0.7),
            heads(gen, batch, sq, hq, dv))


def seen_by(batch, sq, sk, causal=True, window=0, q_lengths=None, k_lengths=None, documents=None):
    """Which keys each query sees, from the definition."""
    lq = torch.full((batch,), sq) if q_lengths is None else q_lengths.cpu().long().clamp(0, sq)
    lk = torch.full((batch,), sk) if k_lengths is None else k_lengths.cpu().long().clamp(0, sk)
    i, j = torch.arange(sq)[None, :, None], torch.arange(sk)[None, None, :]
    lq, lk = lq[:, None, None], lk[:, None, None]
    m = (i < lq) & (j < lk)
    if causal:
        m &= j <= i + lk - lq
    if window:
        m &= j > i + lk - lq - window
    if documents is not None:
        d = documents.cpu().long()
        doc = torch.searchsorted(d, torch.arange(sk), right=True) - 1
        doc = torch.where((doc >= 0) & (doc < len(d) - 1), doc, torch.full_like(doc, -1))
        m &= (doc[None, :, None] == doc[None, None, :]) & (doc >= 0)[None, :, None]
    return m.cuda()


class Want:
    def __init__(self, q, k, v, dy=None, scale=None, **mask):
        b, sq, hq, dk = q.shape
        sk, hk, dv = v.shape[1:]
        g = hq // hk
        scale = dk ** -0.5 if scale is None else scale
        seen = seen_by(b, sq, sk, **mask)[:, None, None]
        Q = q.double().view(b, sq, hk, g, dk).permute(0, 2, 3, 1, 4)
        K, V = k.double().transpose(1, 2)[:, :, None], v.double().transpose(1, 2)[:, :, None]
        # what nothing sees may hold anything
        K = torch.where(seen.any(3)[..., None], K, 0.0)
        V = torch.where(seen.any(3)[..., None], V, 0.0)
        Q = torch.where(seen.any(4)[..., None], Q, 0.0)
        s = scale * (Q @ K.transpose(-1, -2))
        D = 2 * dk * U * scale * (Q.abs() @ K.abs().transpose(-1, -2))
        s = s.masked_fill(~seen, -math.inf)
        lse = torch.logsumexp(s, -1, keepdim=True) if sk else torch.full_like(Q[..., :1], -math.inf)
        dead = torch.isinf(lse)
        p = torch.where(seen & ~dead, torch.exp(s - torch.where(dead, 0.0, lse)), 0.0)
        fin = lambda t: torch.where(torch.isfinite(t), t, 0.0)  # noqa: E731
        e = torch.where(seen, D + 64 * U * (fin(s).abs() + fin(lse).abs() + 1), 0.0)
        top = e.amax(-1, keepdim=True) if sk else torch.zeros_like(lse)
        y = p @ V
        ty = (p * (R + e + 2 * sk * U)) @ V.abs() + y.abs() * (top + sk * U)
        tl = top + (sk + 64) * U * (fin(lse).abs() + 1)
        rows = lambda t: t.permute(0, 3, 1, 2, 4).reshape(b, sq, hq, -1)  # noqa: E731
        self.y, self.ty, self.lse, self.tl = rows(y), rows(ty), rows(lse)[..., 0], rows(tl)[..., 0]
        if dy is None:
            return
        G = torch.where(seen.any(4)[..., None], dy.double().view(b, sq, hk, g, dv).permute(0, 2, 3, 1, 4), 0.0)
        dP = G @ V.transpose(-1, -2)
        Di = (G * y).sum(-1, keepdim=True)
        tD = (G.abs() * (ty + R * (y.abs() + ty) + 2 * dv * U * y.abs())).sum(-1, keepdim=True)
        E = 2 * dv * U * (G.abs() @ V.abs().transpose(-1, -2))
        ds = p * (dP - Di)
        ep = e + tl
        tds = p * (E + tD) + ds.abs() * (ep + R * (1 + 2.0 ** -7)) + 8 * U * p * (dP.abs() + Di.abs())
        keys = lambda t: t.sum(2).transpose(1, 2)  # noqa: E731
        self.dq = rows(scale * (ds @ K))
        self.tdq = rows(scale * (tds @ K.abs() + 2 * sk * U * (ds.abs() @ K.abs())))
        n = sq * g
        self.dk = keys(scale * (ds.transpose(-1, -2) @ Q))
        self.tdk = keys(scale * ((tds + 2 * n * U * ds.abs()).transpose(-1, -2) @ Q.abs()))
        self.dv = keys(p.transpose(-1, -2) @ G)
        self.tdv = keys((p * (R + ep + 2 * n * U)).transpose(-1, -2) @ G.abs())


def near(got, want, tol, what):
    assert got.shape == want.shape and torch.isfinite(got).all(), what
    off = (got.double() - want).abs() - (tol * (1 + 2.0 ** -6) + R * want.abs() + 1e-30)
    assert off.numel() == 0 or off.max() <= 0, (what, float(off.max()), float((got.double() - want).abs().max()))


def check(q, k, v, dy=None, scale=None, **mask):
    w = Want(q, k, v, dy, scale, **mask)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, lse = layers.attention(q, k, v, scale=scale, return_lse=True, dev_status=status, **mask)
    near(y, w.y, w.ty, "y")
    dead = torch.isinf(w.lse)
    assert torch.equal(torch.isinf(lse) & (lse < 0), dead)
    assert ((lse.double() - w.lse).abs()[~dead] <= w.tl[~dead]).all()
    assert (y[dead] == 0).all()
    grads = None
    if dy is not None:
        grads = layers.attention_backward(dy, q, k, v, y, lse, scale=scale, dev_status=status, **mask)
        for name, got in zip(("dq", "dk", "dv"), grads):
            near(got, getattr(w, name), getattr(w, "t" + name), name)
        assert (grads[0][dead] == 0).all()
    assert int(status.item()) == 0
    return y, lse, grads


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# sizes of queries and keys, query and key heads, head dims: one tile and many, odd
# ones, shared heads in blocks of 1, 2, 4 and 32, one of each place of a tile's border
SHAPES = [
    (1, 1, 1, 1, 1, 8, 8), (1, 128, 128, 1, 1, 64, 64), (2, 129, 129, 2, 1, 64, 32), (1, 300, 300, 6, 2, 72, 72),
    (2, 48, 48, 4, 2, 32, 32), (1, 257, 257, 4, 4, 128, 128), (2, 200, 200, 8, 2, 128, 64), (1, 140, 140, 3, 1, 96, 96),
    (1, 130, 130, 2, 2, 192, 128), (2, 333, 333, 4, 1, 136, 120), (1, 70, 70, 64, 2, 80, 80), (1, 40, 40, 5, 1, 184, 16),
    (3, 65, 65, 2, 2, 16, 128),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_training(shape, causal):
    q, k, v, dy = inputs(*shape)
    check(q, k, v, dy, causal=causal)


@pytest.mark.parametrize("sq,sk", [(100, 300), (300, 100), (1, 500), (40, 41), (129, 1), (33, 0)])
@pytest.mark.parametrize("causal", [True, False])
def test_other_numbers_of_queries_than_keys(sq, sk, causal):
    """With more queries than keys the first ones see nothing under a causal mask."""
    q, k, v, dy = inputs(2, sq, sk, 4, 2, 64, 64, seed=1)
    check(q, k, v, dy, causal=causal)


@pytest.mark.parametrize("window", [1, 2, 63, 128, 200, 1000])
def test_window(window):
    q, k, v, dy = inputs(2, 300, 300, 4, 2, 64, 64, seed=2)
    check(q, k, v, dy, window=window)
    q, k, v, dy = inputs(1, 90, 400, 2, 1, 128, 128, seed=2)
    check(q, k, v, dy, window=window)


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_lengths_with_anything_behind_them(dims, causal):
    """Padding holds NaN and infinities; lengths of nothing, of one, of all, past the end, and
    more queries than keys."""
    q, k, v, dy = inputs(7, 150, 170, 4, 2, *dims, seed=3)
    lq, lk = ints(150, 1, 60, 0, 129, 500, 100), ints(170, 1, 128, 50, 0, 500, 40)
    for t, n in ((q, lq), (dy, lq), (k, lk), (v, lk)):
        for b in range(7):
            t[b, int(n[b]):] = float("nan") if b % 2 else float("inf")
    check(q, k, v, dy, causal=causal, q_lengths=lq, k_lengths=lk)
    check(q, k, v, dy, causal=True, window=20, q_lengths=lq, k_lengths=lk)


def test_negative_lengths_count_as_nothing():
    q, k, v, dy = inputs(2, 40, 40, 2, 1, 64, 64, seed=4)
    y, lse, grads = check(q, k, v, dy, q_lengths=ints(-3, 40), k_lengths=ints(40, -1))
    assert not y.any() and not any(g.any() for g in grads)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("starts", [(0, 300), (0, 1, 2, 130, 131, 300), (0, 0, 150, 150, 150, 260), (7, 130, 290),
                                    tuple(range(0, 270, 6)), tuple(range(0, 301, 1)), (0, 40, 300, 300)], ids=lambda s: len(s))
def test_documents(starts, causal):
    """Empty documents, documents of one token, more than a warp holds, tokens before the
    first and behind the last (which hold NaN)."""
    q, k, v, dy = inputs(1, 300, 300, 4, 2, 64, 64, seed=5)
    for t in (q, k, v, dy):
        t[:, :starts[0]] = float("nan")
        t[:, starts[-1]:] = float("nan")
    check(q, k, v, dy, causal=causal, documents=ints(*starts))
    if causal:
        check(q, k, v, dy, window=17, documents=ints(*starts))


@pytest.mark.parametrize("sq,hq,hk,dk,dv,sk", [(1, 4, 2, 32, 32, 48), (1, 16, 1, 128, 128, 5000), (1, 8, 8, 64, 64, 700),
                                               (3, 10, 2, 72, 40, 333), (16, 1, 1, 192, 128, 1030), (2, 14, 2, 128, 128, 64),
                                               (1, 32, 1, 128, 128, 3000), (1, 3, 1, 192, 128, 65), (4, 4, 1, 8, 8, 63)])
def test_few_queries_over_a_cache(sq, hq, hk, dk, dv, sk):
    """Single tokens and a few of them, rows of a key head at most sixteen and more; caches
    of different fill with NaN behind it; keys split over many blocks."""
    q, k, v, _ = inputs(5, sq, sk, hq, hk, dk, dv, seed=6)
    n = ints(sk, max(0, sk - 1), sk // 2, min(sk, 1), 0)
    for b in range(5):
        k[b, int(n[b]):] = float("nan")
        v[b, int(n[b]):] = float("inf")
    check(q, k, v, k_lengths=n)
    check(q, k, v, k_lengths=n, window=min(40, sk))
    check(q, k, v, k_lengths=n, causal=False)


def test_keys_split_over_blocks():
    """A chunk of a prompt against a long cache: parts joined, some of them with nothing."""
    q, k, v, _ = inputs(1, 64, 6000, 4, 2, 64, 64, seed=7)
    args = B.attn_args(q, k, v)
    assert B.gbo_attn_forward_workspace_bytes(args) > 0
    check(q, k, v)
    check(q, k, v, k_lengths=ints(300))
    check(q, k, v, window=100)
    q, k, v, _ = inputs(1, 70, 4000, 2, 1, 192, 128, seed=7)
    check(q, k, v)


def test_tokens_one_at_a_time_give_the_prompts_rows():
    """A prompt as one call and the same tokens one by one over a growing cache: the same rows,
    both within their bound of the formulas."""
    q, k, v, _ = inputs(2, 70, 70, 8, 2, 64, 64, seed=8)
    w = Want(q, k, v)
    for t in range(70):
        y = layers.attention(q[:, t:t + 1], k, v, k_lengths=torch.full((2,), t + 1, dtype=torch.int32, device="cuda"))
        near(y, w.y[:, t:t + 1], w.ty[:, t:t + 1], t)


@pytest.mark.parametrize("scale", [1e-3, 0.3, 3.0])
def test_scale_and_large_scores(scale):
    """Scores of hundreds: the running maximum moves by much more than its threshold."""
    q, k, v, dy = inputs(1, 200, 300, 2, 1, 64, 64, seed=9)
    k[:, 100:110] *= 8
    k[:, 290:] *= 20
    check(q, k, v, dy, scale=scale, causal=False)


def test_strides():
    """Slices of a fused projection, a (batch, heads, seq, dim) layout, outputs of any stride
    whose neighbours stay as they were."""
    gen = torch.Generator().manual_seed(10)
    qkv = heads(gen, 2, 150, 8, 64)
    q, k, v = qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:]
    dy = heads(gen, 2, 4, 150, 64).transpose(1, 2)
    check(q, k, v, dy)
    w = Want(q, k, v)
    for rows in (150, 3):  # tiles, and the kernel for few rows
        big = torch.full((2, 150, 9, 96), 7.0, dtype=torch.bfloat16, device="cuda")
        out = big[:, :rows, 2:6, 16:80]
        assert layers.attention(q[:, 150 - rows:], k, v, out=out) is out
        near(out, w.y[:, 150 - rows:], w.ty[:, 150 - rows:], "out")
        out.fill_(7.0)
        assert (big == 7.0).all()
    with pytest.raises(B.GboError, match="strides"):
        layers.attention(q, k[:, :1].expand(-1, 150, -1, -1), v)
    with pytest.raises(B.GboError, match="aligned"):
        layers.attention(qkv[:, :, :4, 4:60], k[..., :56], v)


@pytest.mark.parametrize("sq", [1, 64])
def test_offsets_past_32_bits(sq):
    """A cache whose last tokens lie past 2^31 elements, and 2^32 bytes."""
    step, sk = 1 << 17, 20000
    flat = torch.empty(step * sk, dtype=torch.bfloat16, device="cuda")
    assert flat.numel() > 1 << 31
    gen = torch.Generator().manual_seed(11)
    k, v = (flat.as_strided((1, sk, 2, 64), (0, step, 64, 1), at) for at in (0, 128))
    for t in (k, v):
        t.copy_(heads(gen, 1, sk, 2, 64))
    q = heads(gen, 1, sq, 4, 64)
    for window in (0, 500):
        check(q, k, v, window=window)
    del flat


def test_results_repeat_bit_for_bit():
    q, k, v, dy = inputs(2, 500, 500, 8, 2, 128, 128, seed=12)
    first = None
    for _ in range(5):
        y, lse = layers.attention(q, k, v, return_lse=True)
        all_of = (y, lse, *layers.attention_backward(dy, q, k, v, y, lse))
        if first is None:
            first = all_of
        assert all(torch.equal(a, b) for a, b in zip(first, all_of))


def test_each_gradient_alone():
    q, k, v, dy = inputs(1, 150, 150, 2, 1, 64, 64, seed=13)
    y, lse = layers.attention(q, k, v, return_lse=True)
    whole = layers.attention_backward(dy, q, k, v, y, lse)
    for n in range(3):
        wanted = tuple(m == n for m in range(3))
        part = layers.attention_backward(dy, q, k, v, y, lse, wanted=wanted)
        assert [g is not None for g in part] == list(wanted) and torch.equal(part[n], whole[n])
    assert layers.attention_backward(dy, q, k, v, y, lse, wanted=(False,) * 3) == (None,) * 3


def test_nothing_to_do():
    for b, sq, sk in ((0, 5, 5), (2, 0, 7), (2, 7, 0), (2, 0, 0)):
        q, k, v, dy = inputs(b, sq, sk, 2, 1, 64, 64)
        y, lse = layers.attention(q, k, v, return_lse=True)
        grads = layers.attention_backward(dy, q, k, v, y, lse)
        assert y.shape == dy.shape and not y.any() and not any(g.any() for g in grads)


def test_a_row_that_is_not_finite_stays_alone():
    """A NaN in a query reaches its own row, and the keys that the row sees."""
    q, k, v, dy = inputs(1, 200, 200, 2, 1, 64, 64, seed=14)
    clean = layers.attention(q, k, v)
    q[0, 77, 1] = float("nan")
    y = layers.attention(q, k, v)
    assert torch.isnan(y[0, 77, 1]).all()
    y[0, 77, 1] = clean[0, 77, 1]
    assert torch.equal(y, clean)


def test_gradients_against_differences():
    """The objective sum dy . y by differences of the formula in 64 bits, along a direction."""
    q, k, v, dy = inputs(1, 60, 60, 4, 2, 32, 32, seed=15)
    y, lse = layers.attention(q, k, v, return_lse=True)
    grads = layers.attention_backward(dy, q, k, v, y, lse)
    w = Want(q, k, v, dy)
    gen = torch.Generator().manual_seed(1)
    for n, (t, name) in enumerate(((q, "q"), (k, "k"), (v, "v"))):
        step = torch.randn(t.shape, generator=gen).cuda().double()

        def objective(h):
            args = [x.double() for x in (q, k, v)]
            args[n] = args[n] + h * step
            return (Want(*args).y * dy.double()).sum()

        slope = float((objective(1e-5) - objective(-1e-5)) / 2e-5)
        tol = float(((getattr(w, "td" + name) + R * getattr(w, "d" + name).abs()) * step.abs()).sum())
        got = float((grads[n].double() * step).sum())
        assert abs(got - slope) <= tol + 1e-6 * abs(slope), (name, got, slope, tol)


def test_autograd():
    q, k, v, dy = (t.requires_grad_() for t in inputs(2, 100, 100, 4, 2, 64, 64, seed=16))
    lq = ints(100, 60)
    y = layers.attention_autograd(q, k, v, q_lengths=lq, k_lengths=lq)
    y.backward(dy)
    w = Want(q.detach(), k.detach(), v.detach(), dy.detach(), q_lengths=lq, k_lengths=lq)
    for name, t in (("dq", q), ("dk", k), ("dv", v)):
        near(t.grad, getattr(w, name), getattr(w, "t" + name), name)
    # an expanded gradient, and only one of the three wanted
    k2 = k.detach().requires_grad_()
    layers.attention_autograd(q.detach(), k2, v.detach()).sum().backward()
    w = Want(q.detach(), k.detach(), v.detach(), torch.ones_like(dy))
    near(k2.grad, w.dk, w.tdk, "dk")
    # lengths that change before the backward pass are noticed
    y = layers.attention_autograd(q, k, v, k_lengths=lq)
    lq.fill_(3)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    y = layers.attention_autograd(q, k, v)
    (g,) = torch.autograd.grad(y.float().square().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_on_a_thread_of_its_own():
    """A thread whose first call into CUDA is the operator's."""
    import threading
    q, k, v, dy = inputs(1, 130, 130, 2, 1, 64, 64, seed=16)
    y, lse = layers.attention(q, k, v, return_lse=True)
    grads = layers.attention_backward(dy, q, k, v, y, lse)
    torch.cuda.synchronize()
    for call, want in ((lambda: (layers.attention(q, k, v),), (y,)),
                       (lambda: layers.attention_backward(dy, q, k, v, y, lse), grads)):
        got = []
        t = threading.Thread(target=lambda: got.append(call()))
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert got and all(torch.equal(a, b) for a, b in zip(got[0], want))


def test_stream_and_graph():
    """On a side stream, and captured: a replay takes the lengths and values it finds."""
    q, k, v, dy = inputs(2, 130, 600, 4, 2, 64, 64, seed=17)
    n = ints(600, 333)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y, lse = layers.attention(q, k, v, k_lengths=n, return_lse=True)
        grads = layers.attention_backward(dy, q, k, v, y, lse, k_lengths=n)
        tok = layers.attention(q[:, :1], k, v, k_lengths=n)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gy, glse = layers.attention(q, k, v, k_lengths=n, return_lse=True)
        ggrads = layers.attention_backward(dy, q, k, v, gy, glse, k_lengths=n)
        gtok = layers.attention(q[:, :1], k, v, k_lengths=n)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((y, lse, tok, *grads), (gy, glse, gtok, *ggrads)):
        assert torch.equal(a, b)
    n.copy_(ints(50, 600))
    q.copy_(q.flip(1))
    graph.replay()
    w = Want(q, k, v, dy, k_lengths=n)
    near(gy, w.y, w.ty, "y")
    for name, t in zip(("dq", "dk", "dv"), ggrads):
        near(t, getattr(w, name), getattr(w, "t" + name), name)
    w = Want(q[:, :1], k, v, k_lengths=n)
    near(gtok, w.y, w.ty, "token")


def test_two_calls_at_once():
    """Two streams at the same time, each with parts and statistics of its own."""
    sets = [inputs(1, 64, 3000, 4, 2, 64, 64, seed=s) for s in (18, 19)]
    alone = [layers.attention(*s[:3]) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(10):
        for n, (s, st) in enumerate(zip(sets, streams)):
            with torch.cuda.stream(st):
                y, lse = layers.attention(*s[:3], return_lse=True)
                got[n].append((y, layers.attention_backward(s[3], *s[:3], y, lse)))
    torch.cuda.synchronize()
    for n in range(2):
        for y, g in got[n]:
            assert torch.equal(y, alone[n]) and all(torch.equal(a, b) for a, b in zip(g, got[n][0][1]))


def test_workspace_refused_when_small():
    q, k, v, dy = inputs(1, 64, 6000, 4, 2, 64, 64)
    args = B.attn_args(q, k, v)
    y = torch.empty_like(q)
    need = B.gbo_attn_forward_workspace_bytes(args)
    for ws in (None, torch.empty(need - 1, dtype=torch.uint8, device="cuda"),
               torch.empty(need + 8, dtype=torch.uint8, device="cuda")[8:]):
        with pytest.raises(B.GboError, match="workspace"):
            B.gbo_attn_forward(args, q, v, y, ws)
    lse = torch.zeros(1, 64, 4, device="cuda")
    for ws in (None, torch.empty(B.gbo_attn_backward_workspace_bytes(args) - 1, dtype=torch.uint8, device="cuda")):
        with pytest.raises(B.GboError, match="workspace"):
            B.gbo_attn_backward(args, q, k, v, dy, y, lse, ws, dq=torch.empty_like(q))


def test_sequences_of_a_batch_are_the_sequences_alone():
    """Many tiles a CTA's place could be mistaken in, some that see nothing: the same bits as of two sequences alone."""
    g = torch.Generator(device="cuda").manual_seed(11)
    made = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    b, s, h = 6, 500, 30
    q, k, v, dy = made(b, s, h, 192), made(b, s, h, 192), made(b, s, h, 128), made(b, s, h, 128)
    lengths = torch.tensor([500, 1, 0, 257, 128, 499], dtype=torch.int32, device="cuda")
    for causal in (True, False):
        mask = dict(causal=causal, q_lengths=lengths, k_lengths=lengths)
        y, lse = layers.attention(q, k, v, return_lse=True, **mask)
        grads = layers.attention_backward(dy, q, k, v, y, lse, **mask)
        for i in range(0, b, 2):
            part = slice(i, i + 2)
            one = dict(causal=causal, q_lengths=lengths[part], k_lengths=lengths[part])
            yi, li = layers.attention(q[part], k[part], v[part], return_lse=True, **one)
            assert torch.equal(yi, y[part]) and torch.equal(li, lse[part])
            gi = layers.attention_backward(dy[part], q[part], k[part], v[part], yi, li, **one)
            for got, want in zip(gi, grads):
                assert torch.equal(got, want[part])


def test_tensors_of_another_device_are_refused(monkeypatch):
    """Where the current device is another one than the tensors' (here: as the binding sees it)."""
    q, k, v = (torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    y, lse = layers.attention(q, k, v, return_lse=True)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    for call in (lambda: layers.attention(q, k, v), lambda: layers.attention_backward(y, q, k, v, y, lse)):
        with pytest.raises(ValueError, match="on the current device"):
            call()


@pytest.mark.parametrize("dims", [(8, 8, 4, 4), (16, 8, 2, 1), (24, 16, 6, 2)])
@pytest.mark.parametrize("window", [1, 0])
def test_rows_of_one_key_take_no_error_from_the_rounded_output(dims, window):
    """A query that sees one key: P is 1, dS = P (dy . v - D) is 0.  Sums of dk and dv products are off by at most
    2^-23 a product of |q| |k| and |dy| |v| (truncated sums), P by as much of the exponent s = scale log2(e) q . k and
    16 more steps, so |dS| <= 2^-23 (dk + dv + 16) (1 + |s|) |dy| |v|.  D from y in bf16 would be off by some
    2^-10 |dy| |v| / sqrt(dv)."""
    dk, dv, hq, hk = dims
    q, k, v, dy = inputs(3, 200, 200, hq, hk, dk, dv, seed=dk)
    y, lse = layers.attention(q, k, v, return_lse=True, window=window)
    dq, dk_, _ = layers.attention_backward(dy, q, k, v, y, lse, window=window)
    rows = 200 if window else 1  # without a window the first query alone sees one key
    norm = lambda t: t.double().norm(dim=-1)  # noqa: E731
    shared = lambda t: norm(t).repeat_interleave(hq // hk, 2)  # noqa: E731
    ds = 2.0 ** -23 * (dk + dv + 16) * (1 + 1.4427 * dk ** -0.5 * norm(q) * shared(k)) * norm(dy) * shared(v) * dk ** -0.5
    assert (norm(dq)[:, :rows] <= (1 + 2.0 ** -8) * (ds * shared(k))[:, :rows]).all()
    if window:
        tol = (ds * norm(q)).view(3, 200, hk, hq // hk).sum(-1)
        assert (norm(dk_) <= (1 + 2.0 ** -7) * tol).all()


@pytest.mark.parametrize("shape", [(2, 16, 16), (1, 40, 17), (3, 5, 300), (2, 33, 33)])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_on_either_side_of_few_keys(shape, causal):
    """Rows that see a handful of keys, and more, of ragged sequences and documents, in heads of every kind."""
    b, sq, sk = shape
    for dk, dv, hq, hk in ((64, 64, 4, 2), (192, 128, 3, 3), (136, 72, 6, 1)):
        q, k, v, dy = inputs(b, sq, sk, hq, hk, dk, dv, seed=sq)
        lengths = dict(q_lengths=ints(*[max(0, sq - 7 * i) for i in range(b)]), k_lengths=ints(*[max(1, sk - 9 * i) for i in range(b)]))
        check(q, k, v, dy, causal=causal, **lengths)
        if b == 1:
            continue
        check(q, k, v, dy, causal=True, window=11)
    q, k, v, dy = inputs(1, 90, 90, 4, 2, 64, 64, seed=3)
    check(q, k, v, dy, causal=causal, documents=ints(2, 3, 3, 19, 36, 80))
