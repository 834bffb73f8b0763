"""Cross entropy of the classifier and its gradients against the formulas in 64 bits.

Tolerances.  A logit is a sum of d products of bf16 values (exact in fp32)
accumulated in fp32: it is off by at most D = 2 d u sum_k |h_k w_k|, u =
2^-24 (2: the tensor core's own order and rounding of partial sums).  Then
lse is off by at most the largest D of its row plus the error of the
exponentials and of their sum, at most 64 u (|lse| + 1), and so is the
logit taken from it.  The gradient of a logit, P, is rounded to bf16, at most
2^-8 of it, and inherits 2 (D + 64 u (|lse| + 1)) of its softmax part; logits
that are kept between the passes are rounded to steps of 2^-9 bits, which
moves the softmax part by at most 2^-10 ln 2 < 2^-10 of it.
The products accumulate K terms in fp32: 2 K u of the sum of the terms'
sizes.  A bf16 output adds 2^-8 of its value, an fp32 one u."""

import pytest
import torch

from adamw_optimizer_step_gb300 import _binding as B
from adamw_optimizer_step_gb300 import layers

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    from adamw_optimizer_step_gb300 import build
    build.build()
    B.lib()


def inputs(n, v, d, seed, ignored=0.0, lean=6.0, dtype=torch.int64):
    g = torch.Generator().manual_seed(seed)
    W = torch.randn(v, d, generator=g) / d ** 0.5
    y = torch.randint(0, v, (n,), generator=g)
    H = torch.randn(n, d, generator=g) + lean * torch.rand(n, 1, generator=g) * W[y]
    y = torch.where(torch.rand(n, generator=g) < ignored, torch.full_like(y, -100), y)
    return H.to(torch.bfloat16).cuda(), W.to(torch.bfloat16).cuda(), y.to(dtype).cuda()


class Want:
    """Losses and gradients in 64 bits, with how far fp32 work may be off."""

    def __init__(self, H, W, y, weight=None, z=0.0, scale=1.0, mean=True, upstream=1.0):
        H, W, y = H.double().cpu(), W.double().cpu(), y.long().cpu()
        n, d = H.shape
        v = W.shape[0]
        w = torch.ones(n, dtype=torch.float64) if weight is None else weight.double().cpu()
        w = torch.where((y >= 0) & (y < v), w, torch.zeros_like(w))
        use = w != 0
        H = torch.where(use[:, None], H, torch.zeros_like(H))
        at = y.clamp(0, v - 1)
        L = scale * (H @ W.T)
        D = 2 * d * U * abs(scale) * (H.abs() @ W.abs().T)
        self.lse = torch.logsumexp(L, 1)
        dl = D.max(1).values + 64 * U * (self.lse.abs() + 1)
        rows = torch.arange(n)
        self.loss = torch.where(use, self.lse - L[rows, at] + z * self.lse ** 2, torch.zeros(n).double())
        self.loss_tol = dl + D[rows, at] + 64 * U * (self.lse.abs() + 1) + 2 * abs(z) * self.lse.abs() * dl
        self.total, self.weight = (w * self.loss).sum(), w.sum()
        self.total_tol = (w.abs() * (self.loss_tol + (n + 64) * U * self.loss.abs())).sum()
        soft = torch.softmax(L, 1) * (1 + 2 * z * self.lse)[:, None]
        hot = torch.zeros_like(L)
        hot[rows, at] = 1.0
        g = upstream / (self.weight if mean and use.any() else 1.0) * scale
        P = w[:, None] * (soft - hot)
        dP = 2.0 ** -8 * P.abs() + w.abs()[:, None] * soft.abs() * (2 * (D + dl[:, None]) + 2.0 ** -10)
        self.dh, self.dw = g * (P @ W), g * (P.T @ H)
        self.dh_tol = abs(g) * (dP @ W.abs() + 2 * v * U * (P.abs() @ W.abs()))
        self.dw_tol = abs(g) * (dP.T @ H.abs() + 2 * max(n, 1) * U * (P.abs().T @ H.abs()))
        self.use = use


def close(got, want, tol, dtype):
    rounding = (2.0 ** -8 if dtype == torch.bfloat16 else 2 * U) * want.abs()
    off = (got.double().cpu() - want).abs() - (tol * (1 + 2.0 ** -7) + rounding + 1e-30)
    assert torch.isfinite(got).all() and off.max() <= 0, float(off.max())


SHAPES = [(1, 1, 8), (1, 300, 64), (5, 257, 72), (130, 256, 128), (300, 1000, 64), (257, 2049, 136), (513, 130, 264),
          (64, 5003, 512), (32, 20011, 136), (17, 4099, 72)]


@pytest.mark.parametrize("n,v,d", SHAPES)
def test_losses(n, v, d):
    H, W, y = inputs(n, v, d, n + v, ignored=0.2 if n > 1 else 0.0)
    lse, totals = torch.empty(n, device="cuda"), torch.empty(2, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss = layers.linear_cross_entropy(H, W, y, z_loss=1e-3, lse=lse, totals=totals, dev_status=status)
    want = Want(H, W, y, z=1e-3)
    close(loss, want.loss, want.loss_tol, torch.float32)
    close(lse, torch.where(want.use, want.lse, torch.zeros_like(want.lse)), want.loss_tol, torch.float32)
    close(totals[0], want.total, want.total_tol, torch.float32)
    assert totals[1].item() == want.weight.item() and status.item() == 0


@pytest.mark.parametrize("n,v,d", SHAPES)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_gradients(n, v, d, out):
    H, W, y = inputs(n, v, d, 3 * n + v, ignored=0.3 if n > 1 else 0.0, dtype=torch.int32)
    dh, dw = (torch.full(t.shape, float("nan"), dtype=out, device="cuda") for t in (H, W))
    loss, _, _ = layers.linear_cross_entropy_grad(H, W, y, z_loss=1e-3, dh=dh, dw=dw)
    want = Want(H, W, y, z=1e-3)
    close(loss, want.loss, want.loss_tol, torch.float32)
    close(dh, want.dh, want.dh_tol, out)
    close(dw, want.dw, want.dw_tol, out)


def test_weights_scale_sum_and_upstream():
    H, W, y = inputs(200, 700, 64, 11, ignored=0.1)
    g = torch.Generator().manual_seed(1)
    weight = torch.rand(200, generator=g).cuda() * 2
    weight[::7] = 0  # left out, like a negative label
    up = torch.tensor([0.37], device="cuda")
    totals = torch.empty(2, device="cuda")
    for mean in (True, False):
        _, dh, dw = layers.linear_cross_entropy_grad(H, W, y, logit_scale=0.5, row_weight=weight, upstream=up,
                                                     mean=mean, totals=totals)
        want = Want(H, W, y, weight=weight, scale=0.5, mean=mean, upstream=0.37)
        close(dh, want.dh, want.dh_tol, torch.bfloat16)
        close(dw, want.dw, want.dw_tol, torch.bfloat16)
        close(totals[0], want.total, want.total_tol, torch.float32)


def smallest_cap(n, v, d):
    lo, hi = 0, B.gbo_xent_workspace_bytes(n, v, d, True)
    while hi - lo > 1024:
        mid = (lo + hi) // 2
        lo, hi = (lo, mid) if B.gbo_xent_workspace_bytes(n, v, d, True, mid) else (mid, hi)
    return hi


def test_pieces_of_the_vocabulary():
    """Workspaces that hold 256 columns, some, and all of the vocabulary: the losses
    and, as long as the logits are formed again, dW are the same bit for bit (each row
    of dW is one product); everything is within its tolerance."""
    H, W, y = inputs(300, 3001, 128, 21)
    want = Want(H, W, y)
    full = layers.linear_cross_entropy_grad(H, W, y)
    least, most = smallest_cap(300, 3001, 128), B.gbo_xent_workspace_bytes(300, 3001, 128, True)
    sizes, first = set(), None
    for cap in (least, (3 * least + most) // 4, (least + most) // 2, most - 1024):
        sizes.add(B.gbo_xent_workspace_bytes(300, 3001, 128, True, cap))
        got = layers.linear_cross_entropy_grad(H, W, y, workspace_cap=cap)
        first = first or got
        assert torch.equal(got[0], full[0]) and torch.equal(got[2], first[2])
        close(got[1], want.dh, want.dh_tol, torch.bfloat16)
        close(got[2], want.dw, want.dw_tol, torch.bfloat16)
    assert len(sizes) >= 3 and max(sizes) < most
    assert B.gbo_xent_workspace_bytes(300, 3001, 128, True, least // 2) == 0


@pytest.mark.parametrize("d", [64, 520])
def test_kept_logits_out_of_range(d):
    """A few rows whose largest logit is more than 64 bits above their label's, among
    others: their tiles are formed again; the rest is kept (of wide rows)."""
    H, W, y = inputs(700, 900, d, 23)
    H[300:310] *= 60
    H[650] *= 100
    want = Want(H, W, y)
    assert (want.loss > 50).sum() >= 3
    loss, dh, dw = layers.linear_cross_entropy_grad(H, W, y)
    close(loss, want.loss, want.loss_tol, torch.float32)
    close(dh, want.dh, want.dh_tol, torch.bfloat16)
    close(dw, want.dw, want.dw_tol, torch.bfloat16)
    again = layers.linear_cross_entropy_grad(H, W, y)
    assert torch.equal(again[1], dh) and torch.equal(again[2], dw)


def test_few_rows_cut_the_long_axis():
    """A long vocabulary and few rows: dH's sum over the vocabulary is cut and joined."""
    for n in (1, 40, 300):
        H, W, y = inputs(n, 20011, 72, 71 + n, ignored=0.1 if n > 1 else 0.0)
        want = Want(H, W, y)
        for out in (torch.float32, torch.bfloat16):
            dh, dw = torch.empty(H.shape, dtype=out, device="cuda"), torch.empty(W.shape, dtype=out, device="cuda")
            layers.linear_cross_entropy_grad(H, W, y, dh=dh, dw=dw)
            close(dh, want.dh, want.dh_tol, out)
            close(dw, want.dw, want.dw_tol, out)
        cap = smallest_cap(n, 20011, 72)
        _, dh, dw = layers.linear_cross_entropy_grad(H, W, y, workspace_cap=2 * cap)
        close(dh, want.dh, want.dh_tol, torch.bfloat16)


def test_accumulate_and_one_gradient_alone():
    H, W, y = inputs(100, 600, 64, 31)
    _, dh, dw = layers.linear_cross_entropy_grad(H, W, y, dw=torch.empty(600, 64, device="cuda"))
    for dtype in (torch.float32, torch.bfloat16):
        base = torch.randn(600, 64, device="cuda").to(dtype)
        into = base.clone()
        layers.linear_cross_entropy_grad(H, W, y, dw=into, accumulate_dw=True)
        assert torch.equal(into, (base.float() + dw).to(dtype))
    lse = torch.empty(100, device="cuda")
    layers.linear_cross_entropy(H, W, y, lse=lse)
    ws = torch.empty(B.gbo_xent_workspace_bytes(100, 600, 64, True), dtype=torch.uint8, device="cuda")
    for which in ("dh", "dw"):
        into = torch.empty_like(H if which == "dh" else W)
        B.gbo_xent_backward(H, W, y, lse, ws, **{which: into})
        # the row's lse in bits is rounded on its way through fp32: P may differ by a bf16 rounding
        want = Want(H, W, y)
        close(into, getattr(want, which), getattr(want, which + "_tol"), torch.bfloat16)


def test_rows_left_out():
    """Rows that are left out hold NaN and infinities: nothing of them reaches
    a loss or a gradient.  A label outside the vocabulary is one of them, and is told."""
    H, W, y = inputs(300, 500, 64, 41, ignored=0.4)
    out = y < 0
    H[out] = float("nan")
    H[torch.nonzero(out)[0]] = float("inf")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, dh, dw = layers.linear_cross_entropy_grad(H, W, y, dev_status=status)
    want = Want(torch.where(out[:, None], torch.zeros_like(H), H), W, y)
    close(loss, want.loss, want.loss_tol, torch.float32)
    close(dh, want.dh, want.dh_tol, torch.bfloat16)
    close(dw, want.dw, want.dw_tol, torch.bfloat16)
    assert torch.all(loss[out] == 0) and torch.all(dh[out] == 0) and status.item() == 0
    y2 = y.clone()
    y2[out] = 500
    loss2, dh2, dw2 = layers.linear_cross_entropy_grad(H, W, y2, dev_status=status)
    assert torch.equal(loss2, loss) and torch.equal(dh2, dh) and torch.equal(dw2, dw)
    assert status.item() == B.GBO_STATUS_BAD_LABEL


def test_no_row_counts():
    H, W, y = inputs(300, 500, 64, 43)
    y.fill_(-1)
    totals = torch.full((2,), 7.0, device="cuda")
    loss, dh, dw = layers.linear_cross_entropy_grad(H, W, y, totals=totals)
    assert torch.all(loss == 0) and torch.all(dh == 0) and torch.all(dw == 0) and torch.all(totals == 0)
    base = torch.randn(500, 64, device="cuda")
    into = base.clone()
    layers.linear_cross_entropy_grad(H, W, y, dw=into, accumulate_dw=True)
    assert torch.equal(into, base)
    # no rows at all
    loss, dh, dw = layers.linear_cross_entropy_grad(H[:0], W, y[:0])
    assert loss.shape == (0,) and dh.shape == (0, 64) and torch.all(dw == 0)
    assert layers.linear_cross_entropy(H[:0], W, y[:0]).shape == (0,)


def test_large_logits():
    """Logits in the hundreds: one softmax entry takes all, others vanish."""
    H, W, y = inputs(64, 700, 64, 47, lean=0.0)
    H, W = H * 30, W * 4
    loss, dh, dw = layers.linear_cross_entropy_grad(H, W, y)
    want = Want(H, W, y)
    assert want.loss.max() > 200
    close(loss, want.loss, want.loss_tol, torch.float32)
    close(dh, want.dh, want.dh_tol, torch.bfloat16)
    close(dw, want.dw, want.dw_tol, torch.bfloat16)


def test_not_finite_is_told():
    H, W, y = inputs(40, 300, 64, 49)
    H[3, 5] = float("nan")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss = layers.linear_cross_entropy(H, W, y, dev_status=status)
    assert status.item() == B.GBO_STATUS_NONFINITE and torch.isnan(loss[3])
    loss[3] = 0
    assert torch.isfinite(loss).all()


def test_strided_and_misaligned_rows():
    """H and the gradients as slices of wider buffers, H off its 16-byte boundary: the same bits."""
    H, W, y = inputs(130, 400, 72, 51)
    loss, dh, dw = layers.linear_cross_entropy_grad(H, W, y)
    wide = torch.zeros(130, 101, dtype=torch.bfloat16, device="cuda")
    wide[:, 5:77] = H
    Wide = torch.zeros(400, 88, dtype=torch.bfloat16, device="cuda")
    Wide[:, 8:80] = W
    oh = torch.zeros(130, 75, dtype=torch.bfloat16, device="cuda")
    ow = torch.zeros(400, 99, dtype=torch.bfloat16, device="cuda")
    got = layers.linear_cross_entropy_grad(wide[:, 5:77], Wide[:, 8:80], y, dh=oh[:, 3:75], dw=ow[:, 1:73])
    assert torch.equal(got[0], loss) and torch.equal(oh[:, 3:75], dh) and torch.equal(ow[:, 1:73], dw)
    assert torch.all(oh[:, :3] == 0) and torch.all(ow[:, 73:] == 0) and torch.all(ow[:, 0] == 0)
    # slices whose rows are 16-byte aligned, and added to where they are not
    ow = torch.full((400, 88), 3.0, dtype=torch.bfloat16, device="cuda")
    got = layers.linear_cross_entropy_grad(H, W, y, dw=ow[:, 8:80])
    assert torch.equal(ow[:, 8:80], dw) and torch.all(ow[:, :8] == 3) and torch.all(ow[:, 80:] == 3)
    _, _, dw32 = layers.linear_cross_entropy_grad(H, W, y, dw=torch.empty(400, 72, device="cuda"))
    for width, first in ((96, 4), (75, 1)):
        ow = torch.full((400, width), 3.0, device="cuda")
        layers.linear_cross_entropy_grad(H, W, y, dw=ow[:, first:first + 72], accumulate_dw=True)
        assert torch.equal(ow[:, first:first + 72], 3.0 + dw32)
        assert torch.all(ow[:, :first] == 3) and torch.all(ow[:, first + 72:] == 3)


def test_gradient_against_differences():
    """Directional differences of the 64-bit loss match the gradients' inner products,
    within the gradients' tolerance."""
    H, W, y = inputs(24, 90, 32, 53)
    want = Want(H, W, y, z=1e-3)
    dh, dw = torch.empty(24, 32, device="cuda"), torch.empty(90, 32, device="cuda")
    layers.linear_cross_entropy_grad(H, W, y, z_loss=1e-3, dh=dh, dw=dw)
    g = torch.Generator().manual_seed(2)
    a, b = torch.randn(24, 32, generator=g).double(), torch.randn(90, 32, generator=g).double()

    def objective(t):
        L = (H.double().cpu() + t * a) @ (W.double().cpu() + t * b).T
        lse = torch.logsumexp(L, 1)
        return (lse - L[torch.arange(24), y.cpu()] + 1e-3 * lse ** 2).mean()

    h = 1e-5
    num = (objective(h) - objective(-h)) / (2 * h)
    got = (dh.double().cpu() * a).sum() + (dw.double().cpu() * b).sum()
    tol = (want.dh_tol * a.abs()).sum() + (want.dw_tol * b.abs()).sum() + 1e-7
    assert abs(num - got) <= tol


@pytest.mark.parametrize("d", [64, 520])
@pytest.mark.parametrize("cap", ["keep", "pieces"])
def test_autograd_matches_the_formula(cap, d):
    """Logits kept from the forward pass, or formed again; bf16 weights and a float32
    master table, whose gradient is float32."""
    H, W, y = inputs(96, 1333, d, 57, ignored=0.1)
    want = Want(H, W, y, z=1e-3, upstream=3.0)
    cap = 0 if cap == "keep" else smallest_cap(96, 1333, d)
    for master in (False, True):
        Hg, Wg = H.clone().requires_grad_(), (W.float() if master else W.clone()).requires_grad_()
        loss = layers.linear_cross_entropy_loss(Hg, Wg, y, z_loss=1e-3, workspace_cap=cap)
        (3.0 * loss).backward()
        close(loss.detach(), want.total / want.weight, want.total_tol / want.weight, torch.float32)
        close(Hg.grad, want.dh, want.dh_tol, torch.bfloat16)
        close(Wg.grad, want.dw, want.dw_tol, Wg.dtype)


@pytest.mark.parametrize("d", [72, 520])
def test_kept_logits_between_two_calls(d):
    """forward with keep, then backward on its workspace: the gradients of one call,
    among them of tiles that are out of the kept range; other kernels in between."""
    H, W, y = inputs(600, 1100, d, 58, ignored=0.1)
    H[300:310] *= 100
    want = Want(H, W, y)
    assert (want.loss > 50).any()
    ws = torch.empty(B.gbo_xent_workspace_bytes(600, 1100, d, True), dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty(600, device="cuda"), torch.empty(600, device="cuda")
    B.gbo_xent_forward(H, W, y, ws, loss=loss, lse=lse, keep=True)
    layers.linear_cross_entropy(W, H, torch.zeros(1100, dtype=torch.long, device="cuda"))
    dh, dw = torch.empty_like(H), torch.empty_like(W)
    B.gbo_xent_backward(H, W, y, lse, ws, dh=dh, dw=dw, keep=True)
    close(loss, want.loss, want.loss_tol, torch.float32)
    close(dh, want.dh, want.dh_tol, torch.bfloat16)
    close(dw, want.dw, want.dw_tol, torch.bfloat16)


def test_repeatable_on_a_stream_and_in_a_graph():
    H, W, y = inputs(700, 1500, 136, 59, ignored=0.2)
    first = layers.linear_cross_entropy_grad(H, W, y)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = layers.linear_cross_entropy_grad(H, W, y)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(first, second):
        assert torch.equal(a, b)
    loss, dh, dw = (torch.empty_like(t) for t in first)
    ws = torch.empty(B.gbo_xent_workspace_bytes(700, 1500, 136, True), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.gbo_xent_grad(H, W, y, ws, loss=loss, dh=dh, dw=dw)
    y[:100] = -1  # fewer rows count in the replay than in the capture
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((loss, dh, dw), layers.linear_cross_entropy_grad(H, W, y)):
        assert torch.equal(a, b)


def test_large_tile_sweep():
    """More than one sweep of 8192 rows, several pieces, against the 64-bit formula."""
    H, W, y = inputs(8500, 1030, 72, 61, ignored=0.01)
    want = Want(H, W, y)
    loss, dh, dw = layers.linear_cross_entropy_grad(H, W, y)
    close(loss, want.loss, want.loss_tol, torch.float32)
    close(dh, want.dh, want.dh_tol, torch.bfloat16)
    close(dw, want.dw, want.dw_tol, torch.bfloat16)


@pytest.mark.parametrize("ignored", [0.0, 0.4])
def test_many_rows_in_one_and_in_two_calls(ignored):
    """Thousands of rows with tiles among them that are out of the kept range, all of
    them counting or a part, in one call and in a kept pair of calls."""
    H, W, y = inputs(6500, 777, 72, 67, ignored=ignored)
    H[1000:1003] *= 100
    H[4000] *= 100
    want = Want(H, W, y)
    assert (want.loss > 50).any()
    loss, dh, dw = layers.linear_cross_entropy_grad(H, W, y)
    lse, ws = torch.empty(6500, device="cuda"), torch.empty(B.gbo_xent_workspace_bytes(6500, 777, 72, True),
                                                            dtype=torch.uint8, device="cuda")
    totals = torch.empty(2, device="cuda")
    B.gbo_xent_forward(H, W, y, ws, lse=lse, totals=totals, keep=True)
    dh2, dw2 = torch.empty_like(H), torch.empty_like(W)
    B.gbo_xent_backward(H, W, y, lse, ws, dh=dh2, dw=dw2, keep=True)
    close(loss, want.loss, want.loss_tol, torch.float32)
    close(totals[0], want.total, want.total_tol, torch.float32)
    for a, b in ((dh, dw), (dh2, dw2)):
        close(a, want.dh, want.dh_tol, torch.bfloat16)
        close(b, want.dw, want.dw_tol, torch.bfloat16)


@pytest.mark.parametrize("n", [2, 5, 31, 32, 33])
def test_few_rows_among_rows_left_out(n):
    """Losses of few rows (those that count are fewer still), statistics of runs of the
    vocabulary that end inside a tile; repeated with the same bits."""
    H, W, y = inputs(n, 5003, 200, 80 + n, ignored=0.4)
    want = Want(H, W, y)
    loss = layers.linear_cross_entropy(H, W, y)
    close(loss, want.loss, want.loss_tol, torch.float32)
    assert torch.equal(loss, layers.linear_cross_entropy(H, W, y))
    W[-7:] = 0
    W[-7:, 0] = -float("inf")  # logits of -inf where h_0 > 0: no part in the sum
    H[:, 0] = H[:, 0].abs() + 1
    y = torch.where(y >= 4990, y - 4990, y)
    loss = layers.linear_cross_entropy(H, W, y)
    want = Want(H, W[:-7], y)
    close(loss, want.loss, want.loss_tol, torch.float32)


@pytest.mark.parametrize("n,v,d", [(1, 40009, 72), (16, 58369, 64), (3, 38913, 200), (17, 40009, 1000), (32, 60001, 680)])
def test_few_rows_of_large_tables(n, v, d):
    """Tables of several tiles an SM, whose last rows are cut in runs that end anywhere."""
    H, W, y = inputs(n, v, d, v + n, ignored=0.2 if n > 3 else 0.0)
    y[-1] = v - 1
    want = Want(H, W, y)
    lse, totals = torch.empty(n, device="cuda"), torch.empty(2, device="cuda")
    loss = layers.linear_cross_entropy(H, W, y, lse=lse, totals=totals)
    close(loss, want.loss, want.loss_tol, torch.float32)
    close(lse, torch.where(want.use, want.lse, torch.zeros_like(want.lse)), want.loss_tol, torch.float32)
    close(totals[0], want.total, want.total_tol, torch.float32)


def test_weights_that_sum_to_zero():
    """The mean over weights +1 and -1: the loss and its gradients are 0, not inf."""
    H, W, y = inputs(2, 300, 64, 71)
    weight = torch.tensor([1.0, -1.0], device="cuda")
    Hg, Wg = H.clone().requires_grad_(), W.clone().requires_grad_()
    loss = layers.linear_cross_entropy_loss(Hg, Wg, y, weight)
    loss.backward()
    assert loss.item() == 0
    assert torch.equal(Hg.grad, torch.zeros_like(H)) and torch.equal(Wg.grad, torch.zeros_like(W))


@pytest.mark.parametrize("d", [64, 512])
@pytest.mark.parametrize("cap", ["keep", "pieces"])
def test_two_backward_passes(cap, d):
    """retain_graph: the second pass has no kept logits, and the same gradients by its own
    bounds; a gradient of a gradient is refused."""
    H, W, y = inputs(70, 900, d, 72, ignored=0.1)
    want = Want(H, W, y)
    cap = 0 if cap == "keep" else smallest_cap(70, 900, d)
    Hg, Wg = H.clone().requires_grad_(), W.clone().requires_grad_()
    loss = layers.linear_cross_entropy_loss(Hg, Wg, y, workspace_cap=cap)
    for _ in range(2):
        dh, dw = torch.autograd.grad(loss, (Hg, Wg), retain_graph=True)
        close(dh, want.dh, want.dh_tol, torch.bfloat16)
        close(dw, want.dw, want.dw_tol, torch.bfloat16)
    dh, = torch.autograd.grad(loss, Hg, create_graph=True)
    with pytest.raises(RuntimeError):
        dh.float().sum().backward()


def test_status_and_single_rows_through_autograd():
    """A label outside the vocabulary is told; one row of h and of w, slices whose strides
    belong to wider tensors of an odd width."""
    H, W, y = inputs(5, 300, 64, 73)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    layers.linear_cross_entropy_loss(H, W, y, dev_status=status)
    assert status.item() == 0
    y[2] = 300
    layers.linear_cross_entropy_loss(H, W, y, dev_status=status)
    assert status.item() == 4
    wide = torch.zeros(3, 65, dtype=torch.bfloat16, device="cuda")
    wide[:1, :64] = H[:1]
    one = wide[:1, :64]
    loss, dh, dw = layers.linear_cross_entropy_grad(one, one, torch.zeros(1, dtype=torch.int64, device="cuda"))
    # one class: its probability is 1, the loss and the gradients 0 (P off by the bound of lse)
    want = Want(one, one, torch.zeros(1, dtype=torch.int64))
    close(loss, want.loss, want.loss_tol, torch.float32)
    close(dh, want.dh, want.dh_tol, torch.bfloat16)
    close(dw, want.dw, want.dw_tol, torch.bfloat16)


def test_many_wide_rows_in_one_and_in_two_calls():
    """The same with rows wide enough for kept logits; rows that are out of the kept range
    have the class of their smallest logit as their label."""
    H, W, y = inputs(6500, 777, 520, 68, ignored=0.2)
    for r in (1000, 1002, 4000):
        H[r] *= 100
        y[r] = (W.double() @ H[r].double()).argmin()
    want = Want(H, W, y)
    assert (want.loss[[1000, 1002, 4000]] > 64).all()
    loss, dh, dw = layers.linear_cross_entropy_grad(H, W, y)
    lse, ws = torch.empty(6500, device="cuda"), torch.empty(B.gbo_xent_workspace_bytes(6500, 777, 520, True),
                                                            dtype=torch.uint8, device="cuda")
    B.gbo_xent_forward(H, W, y, ws, lse=lse, keep=True)
    dh2, dw2 = torch.empty_like(H), torch.empty_like(W)
    B.gbo_xent_backward(H, W, y, lse, ws, dh=dh2, dw=dw2, keep=True)
    close(loss, want.loss, want.loss_tol, torch.float32)
    for a, b in ((dh, dw), (dh2, dw2)):
        close(a, want.dh, want.dh_tol, torch.bfloat16)
        close(b, want.dw, want.dw_tol, torch.bfloat16)


def test_offsets_past_32_bits():
    """More than 2^31 elements of W, of dW and of kept logits: losses and dH of sampled
    rows, and dW of sampled classes, the last ones among them."""
    n, v, d = 2100, 1050000, 2056
    assert v * d > 2 ** 31 and n * v > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(91)
    W = torch.empty(v, d, dtype=torch.bfloat16, device="cuda")
    for a in range(0, v, 131072):
        W[a:a + 131072] = torch.randn(min(131072, v - a), d, generator=g, device="cuda") / d ** 0.5
    y = torch.randint(0, v, (n,), generator=g, device="cuda")
    y[-1], y[0], y[7] = v - 1, 0, -1
    H = (torch.randn(n, d, generator=g, device="cuda") + 6 * W[y.clamp(min=0)].float()).bfloat16()
    cap = 16 << 30
    assert B.gbo_xent_workspace_bytes(n, v, d, True, cap) > 2 * n * v
    lse = torch.empty(n, device="cuda")
    ws = torch.empty(B.gbo_xent_workspace_bytes(n, v, d, True, cap), dtype=torch.uint8, device="cuda")
    loss, dh, dw = torch.empty(n, device="cuda"), torch.empty_like(H), torch.empty_like(W)
    B.gbo_xent_grad(H, W, y, ws, loss=loss, lse=lse, dh=dh, dw=dw)
    del ws
    rows = torch.tensor([0, 6, 1031, n - 1], device="cuda")
    Hr = H[rows].double()
    L = torch.cat([Hr @ W[a:a + 65536].double().T for a in range(0, v, 65536)], 1)
    size = torch.cat([Hr.abs() @ W[a:a + 65536].double().abs().T for a in range(0, v, 65536)], 1)
    D, want_lse = 2 * d * U * size, torch.logsumexp(L, 1)
    dl = D.max(1).values + 64 * U * (want_lse.abs() + 1)
    at, pick = torch.arange(4, device="cuda"), y[rows]
    want = want_lse - L[at, pick]
    tol = dl + D[at, pick] + 64 * U * (want_lse.abs() + 1)
    assert torch.all((loss[rows].double() - want).abs() <= tol + 2 * U * want.abs())
    gain = 1.0 / (n - 1)
    soft = torch.softmax(L, 1)
    P = soft.clone()
    P[at, pick] -= 1
    dP = 2.0 ** -8 * P.abs() + soft * (2 * (D + dl[:, None]) + 2.0 ** -10)
    parts = [(P[:, a:a + 65536] @ w, dP[:, a:a + 65536] @ w.abs(), P[:, a:a + 65536].abs() @ w.abs())
             for a in range(0, v, 65536) for w in (W[a:a + 65536].double(),)]
    want, off, terms = (sum(p[k] for p in parts) for k in range(3))
    tol = gain * (off + 2 * v * U * terms)
    assert torch.all((dh[rows].double() - gain * want).abs() <= tol * (1 + 2.0 ** -7) + 2.0 ** -8 * (gain * want).abs())
    assert not dh[7].any() and loss[7] == 0
    classes = torch.tensor([0, 1, 524287, 1048575, 1048576, v - 2, v - 1], device="cuda")
    use, Hd, Wc = (y >= 0)[:, None], H.double(), W[classes].double()
    Lc = Hd @ Wc.T
    D = 2 * d * U * (Hd.abs() @ Wc.abs().T)
    soft = torch.where(use, (Lc - lse.double()[:, None]).exp(), 0.0)
    P = soft - (y[:, None] == classes).double()
    # (lse is the kernel's, within 64 u (|lse| + 1) and the largest D of its row)
    dP = 2.0 ** -8 * P.abs() + soft * (2 * (D + dl.max() + 64 * U * (lse.double().abs() + 1)[:, None]) + 2.0 ** -10)
    want, tol = gain * (P.T @ Hd), gain * (dP.T @ Hd.abs() + 2 * n * U * (P.abs().T @ Hd.abs()))
    assert torch.all((dw[classes].double() - want).abs() <= tol * (1 + 2.0 ** -7) + 2.0 ** -8 * want.abs())
