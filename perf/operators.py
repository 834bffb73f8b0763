"""Cases of the operators that surround the optimizer step in training and
scoring: the tied classifier's cross entropy with its gradient, and the
rotation of queries and keys, alone and with their per-head norm.

Each case's inputs are made on the GPU from a seed.  With ``own`` false,
``run`` computes the operator from elementary torch operations in 32 bits,
rounded once at the end; with ``own`` true it calls the framework.
``exact`` computes the same outputs in 64 bits.

Notation.  Cross entropy: hidden rows H (n x d), classifier W (v x d, the tied
embedding), labels y (negative: the row is left out),

    l = H W^T,  lse_i = log sum_j exp l_ij,  loss_i = lse_i - l_iy + z lse_i^2,
    L = mean of loss_i over the rows that count,  dH = dL/dH,  dW = dL/dW.

Rotation: the pair (a, b) at frequency f_j and position t becomes
m (a cos(t f_j) - b sin(t f_j), a sin(t f_j) + b cos(t f_j)).
"""

import math

import torch

own = False

BF16, F32 = "bf16", "f32"
DTYPES = {BF16: torch.bfloat16, F32: torch.float32}
EPS = 1e-6


def listed():
    return [
        # the 128000 x 2048 tied embedding's loss and gradients for one micro-batch
        dict(name="xent_train_128000x2048", op="xent_train", n=8192, v=128000, d=2048, ignored=0.0, z=1e-4),
        # the 32000 x 4096 embedding, prompts left out of the loss
        dict(name="xent_train_32000x4096", op="xent_train", n=4096, v=32000, d=4096, ignored=0.4, z=0.0),
        # odd rows and an odd vocabulary
        dict(name="xent_train_ragged", op="xent_train", n=777, v=32003, d=1032, ignored=0.1, z=1e-4),
        # the 1000 x 64 embedding of the small correctness set: latency
        dict(name="xent_train_1000x64", op="xent_train", n=64, v=1000, d=64, ignored=0.2, z=0.0),
        # evaluation: losses alone, the 128256 x 2048 embedding
        dict(name="xent_eval_128256x2048", op="xent_eval", n=4096, v=128256, d=2048, ignored=0.0, z=0.0),
        # scoring one token while answering
        dict(name="xent_score_one_token", op="xent_eval", n=1, v=128000, d=2048, ignored=0.0, z=0.0),
        # q/k norms (gains of 128) with rotation on a fused projection's output, training length
        dict(name="qk_norm_rotary_train", op="qk_fwd", batch=4, seq=8192, hq=16, hk=4, dim=128, rot=128, offset=0,
             layout="half", scaling="none", dtype=BF16, start=0, longest=8192),
        # ... and its backward pass
        dict(name="qk_norm_rotary_backward", op="qk_bwd", batch=4, seq=8192, hq=16, hk=4, dim=128, rot=128, offset=0,
             layout="half", scaling="none", dtype=BF16, start=0, longest=8192),
        # ... and one token of each of eight sequences while answering, far into a long context
        dict(name="qk_norm_rotary_one_token", op="qk_fwd", batch=8, seq=1, hq=16, hk=4, dim=128, rot=128, offset=0,
             layout="half", scaling="wavelength", dtype=BF16, start=100000, longest=131072),
        # odd sizes in 32 bits, half of a head of 72 rotated
        dict(name="qk_norm_rotary_backward_f32", op="qk_bwd", batch=3, seq=341, hq=3, hk=1, dim=72, rot=36, offset=4,
             layout="interleaved", scaling="none", dtype=F32, start=7, longest=1024),
        # 32 heads of 128 + 64, the last 64 rotated in pairs, context stretched
        dict(name="rotary_192_of_64", op="rotary", batch=2, seq=16384, hq=32, hk=0, dim=192, rot=64, offset=128,
             layout="interleaved", scaling="yarn", dtype=BF16, start=0, longest=65536),
        # the gradient of a rotation in 32 bits
        dict(name="rotary_inverse_f32", op="rotary_inverse", batch=1, seq=4099, hq=8, hk=0, dim=128, rot=128, offset=0,
             layout="half", scaling="linear", dtype=F32, start=0, longest=8192),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["xent_train", "xent_train", "xent_eval", "qk_fwd", "qk_bwd", "rotary", "rotary_inverse"])
    if kind.startswith("xent"):
        while True:
            c = dict(op=kind, n=_log_int(rng, 1, 8192), v=_log_int(rng, 200, 131072), d=8 * _log_int(rng, 4, 512),
                     ignored=rng.choice([0.0, 0.0, 0.1, 0.5]), z=rng.choice([0.0, 1e-4]))
            if c["n"] * c["v"] * c["d"] <= 8192 * 128000 * 2048:
                return c
    dim = rng.choice([64, 72, 80, 96, 128, 128, 192, 256])
    rot = rng.choice([dim, dim, 2 * (dim // 4), 32])
    hq = rng.choice([1, 3, 8, 16, 32])
    seq = _log_int(rng, 1, 16384)
    longest = max(2048, 2 * seq)
    return dict(op=kind, batch=rng.choice([1, 1, 2, 3]), seq=seq, hq=hq,
                hk=rng.choice([1, max(1, hq // 4), hq]) if kind.startswith("qk") else 0, dim=dim, rot=rot,
                offset=rng.choice([0, dim - rot]), layout=rng.choice(["half", "interleaved"]),
                scaling=rng.choice(["none", "linear", "ntk", "yarn", "wavelength"]),
                dtype=rng.choice([BF16, BF16, F32]), start=rng.randrange(longest - seq), longest=longest)


# ---------------------------------------------------------------------------
# frequencies of a rotation, in 64 bits

BASE, FACTOR = 10000.0, 4.0


def _frequencies(case):
    """(frequencies, factor on cos and sin) of the case's scaling; the context
    was trained at an eighth of its longest position."""
    r, trained = case["rot"], case["longest"] / 8.0
    f = [BASE ** (-2.0 * j / r) for j in range(r // 2)]
    kind = case["scaling"]
    if kind == "linear":
        return [x / FACTOR for x in f], 1.0
    if kind == "ntk":
        base = BASE * FACTOR ** (r / (r - 2.0))
        return [base ** (-2.0 * j / r) for j in range(r // 2)], 1.0
    if kind == "yarn":
        # index at which a frequency turns `turns` times over the trained context
        at = lambda turns: r * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(BASE))  # noqa: E731
        low, high = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), r - 1)
        ramp = [min(max((j - low) / max(high - low, 1e-3), 0.0), 1.0) for j in range(r // 2)]
        return [x * (1 - w) + x / FACTOR * w for x, w in zip(f, ramp)], 0.1 * math.log(FACTOR) + 1.0
    if kind == "wavelength":
        out = []
        for x in f:
            turns = trained * x / (2 * math.pi)
            keep = min(max((turns - 1.0) / (4.0 - 1.0), 0.0), 1.0)
            out.append(x * keep + x / FACTOR * (1 - keep))
        return out, 1.0
    return f, 1.0


def _spec(case):
    """The framework's handle for the case's rotation, which a program keeps."""
    from adamw_optimizer_step_gb300 import layers
    scaling = None
    if case["scaling"] in ("linear", "ntk"):
        scaling = dict(kind=case["scaling"], factor=FACTOR)
    elif case["scaling"] == "yarn":
        scaling = dict(kind="yarn", factor=FACTOR, trained=case["longest"] / 8.0, fast=32.0, slow=1.0)
    elif case["scaling"] == "wavelength":
        scaling = dict(kind="wavelength", factor=FACTOR, trained=case["longest"] / 8.0, fast=4.0, slow=1.0)
    return layers.RotarySpec(case["dim"], rot_dim=case["rot"], offset=case["offset"], layout=case["layout"],
                             base=BASE, scaling=scaling)


# ---------------------------------------------------------------------------
# inputs

def _xent_inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    n, v, d = case["n"], case["v"], case["d"]
    W = torch.randn(v, d, generator=g, device="cuda").mul_(0.02)
    # frequent tokens first, as in a vocabulary ordered by rank
    u = torch.rand(n, generator=g, device="cuda")
    y = (torch.exp(u * math.log(v + 1.0)) - 1.0).long().clamp_(0, v - 1)
    # normed hidden rows that lean to their label's row, some of them strongly
    H = torch.randn(n, d, generator=g, device="cuda")
    lean = torch.rand(n, 1, generator=g, device="cuda") * 14.0
    at = W[y]
    H += lean * at / at.norm(dim=1, keepdim=True).clamp_min(1e-9)
    skip = torch.rand(n, generator=g, device="cuda") < case["ignored"]
    return H.to(torch.bfloat16), W.to(torch.bfloat16), torch.where(skip, torch.full_like(y, -100), y)


def _rot_inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    b, s, hq, hk, dim = case["batch"], case["seq"], case["hq"], case["hk"], case["dim"]
    dt = DTYPES[case["dtype"]]
    made = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    # queries, keys and values as one projection writes them
    qkv = made(b, s, hq + 2 * hk, dim).mul_(0.7).to(dt)
    dq, dk = made(b, s, hq, dim).to(dt), made(b, s, hk, dim).to(dt)
    gq, gk = (1.0 + 0.2 * made(dim) for _ in range(2))
    # each sequence starts at a place of its own
    starts = torch.randint(0, case["longest"] - case["start"] - s + 1, (b, 1), generator=g, device="cuda")
    pos = case["start"] + starts + torch.arange(s, device="cuda")
    return qkv[:, :, :hq], qkv[:, :, hq:hq + hk], dq, dk, gq, gk, pos


def prepare(case, seed):
    if case["op"].startswith("xent"):
        H, W, y = _xent_inputs(case, seed)
        return dict(case=case, H=H, W=W, y=y)
    q, k, dq, dk, gq, gk, pos = _rot_inputs(case, seed)
    f, m = _frequencies(case)
    # tables of cosines and sines for every position, which a program keeps
    t = torch.arange(case["longest"], device="cuda", dtype=torch.float64)[:, None] * torch.tensor(
        f, device="cuda", dtype=torch.float64)
    state = dict(case=case, q=q, k=k, dq=dq, dk=dk, gq=gq, gk=gk, pos=pos, cos=(t.cos() * m).float(),
                 sin=(t.sin() * m).float())
    if own:
        state["spec"] = _spec(case)
    return state


# ---------------------------------------------------------------------------
# plain forms, in 32 bits

def _plain_xent(s):
    c, H, W, y = s["case"], s["H"].float(), s["W"].float(), s["y"]
    valid = y >= 0
    at = y.clamp_min(0)[:, None]
    logits = H @ W.t()
    top = logits.amax(dim=1, keepdim=True)
    e = torch.exp(logits - top)
    total = e.sum(dim=1, keepdim=True)
    lse = top + torch.log(total)
    loss = lse - logits.gather(1, at) + c["z"] * lse * lse
    loss = torch.where(valid, loss[:, 0], torch.zeros_like(loss[:, 0]))
    if c["op"] == "xent_eval":
        return dict(loss=loss)
    g = valid.float()[:, None] / valid.sum().clamp_min(1).float()
    P = e / total * (1.0 + 2.0 * c["z"] * lse)
    P.scatter_add_(1, at, torch.full_like(lse, -1.0))
    P *= g
    return dict(loss=loss, dh=(P @ W).to(torch.bfloat16), dw=(P.t() @ H).to(torch.bfloat16))


def _turn(x, cos, sin, c):
    """x (batch, seq, heads, dim) in 32 bits, rotated."""
    o, r = c["offset"], c["rot"]
    part = x[..., o:o + r]
    if c["layout"] == "half":
        a, b = part[..., :r // 2], part[..., r // 2:]
    else:
        a, b = part[..., 0::2], part[..., 1::2]
    u, v = a * cos - b * sin, a * sin + b * cos
    turned = torch.cat((u, v), dim=-1) if c["layout"] == "half" else torch.stack((u, v), dim=-1).flatten(-2)
    return torch.cat((x[..., :o], turned, x[..., o + r:]), dim=-1)


def _plain_rot(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    cos, sin = s["cos"][s["pos"]][:, :, None], s["sin"][s["pos"]][:, :, None]
    if c["op"] == "rotary":
        return dict(y=_turn(s["q"].float(), cos, sin, c).to(dt))
    if c["op"] == "rotary_inverse":
        return dict(y=_turn(s["q"].float(), cos, -sin, c).to(dt))
    unit = lambda x: x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS)  # noqa: E731
    if c["op"] == "qk_fwd":
        return dict(q=_turn(unit(s["q"].float()) * s["gq"], cos, sin, c).to(dt),
                    k=_turn(unit(s["k"].float()) * s["gk"], cos, sin, c).to(dt))

    def back(dy, x, gain):
        e, x = _turn(dy.float(), cos, -sin, c), x.float()
        rho = torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS)
        u, ge = x * rho, gain * e
        return (rho * (ge - u * (ge * u).mean(dim=-1, keepdim=True))).to(dt), (e * u).sum(dim=(0, 1, 2))

    dq, dgq = back(s["dq"], s["q"], s["gq"])
    dk, dgk = back(s["dk"], s["k"], s["gk"])
    return dict(dq=dq, dk=dk, dgq=dgq, dgk=dgk)


def _own(s):
    from adamw_optimizer_step_gb300 import layers
    c = s["case"]
    if c["op"] == "xent_eval":
        return dict(loss=layers.linear_cross_entropy(s["H"], s["W"], s["y"], z_loss=c["z"]))
    if c["op"] == "xent_train":
        loss, dh, dw = layers.linear_cross_entropy_grad(s["H"], s["W"], s["y"], z_loss=c["z"])
        return dict(loss=loss, dh=dh, dw=dw)
    if c["op"] == "rotary":
        return dict(y=layers.rotary(s["q"], s["pos"], s["spec"]))
    if c["op"] == "rotary_inverse":
        return dict(y=layers.rotary(s["q"], s["pos"], s["spec"], inverse=True))
    if c["op"] == "qk_fwd":
        q, k = layers.qk_norm_rotary(s["q"], s["k"], s["gq"], s["gk"], s["pos"], s["spec"], eps=EPS)
        return dict(q=q, k=k)
    dq, dk, dgq, dgk = layers.qk_norm_rotary_backward(s["dq"], s["dk"], s["q"], s["k"], s["gq"], s["gk"], s["pos"],
                                                      s["spec"], eps=EPS)
    return dict(dq=dq, dk=dk, dgq=dgq, dgk=dgk)


def run(state):
    if own:
        return _own(state)
    return _plain_xent(state) if state["case"]["op"].startswith("xent") else _plain_rot(state)


def work(case):
    """Inputs read once, outputs written once, and the products that cannot be
    left out: the logits, and for the gradients one product each."""
    if case["op"].startswith("xent"):
        n, v, d = case["n"], case["v"], case["d"]
        train = case["op"] == "xent_train"
        rows = n * (1.0 - case["ignored"])  # the rows that count
        return dict(bytes=2.0 * d * (rows + v + (n + v if train else 0)) + 12.0 * n,
                    flops=(6.0 if train else 2.0) * rows * v * d)
    tokens, heads, dim = case["batch"] * case["seq"], case["hq"] + case["hk"], case["dim"]
    size = 2 if case["dtype"] == BF16 else 4
    x = float(tokens) * heads * dim
    back = case["op"] == "qk_bwd"
    gains = 8.0 * dim * (2 if back else 1) if case["hk"] else 0.0
    return dict(bytes=(3 if back else 2) * size * x + 8.0 * tokens + gains,
                flops=x * {"rotary": 3, "rotary_inverse": 3, "qk_fwd": 8, "qk_bwd": 16}[case["op"]])


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_xent(case, seed):
    H, W, y = _xent_inputs(case, seed)
    H, W = H.double(), W.double()
    n, train = case["n"], case["op"] == "xent_train"
    count = max(1, int((y >= 0).sum()))
    loss = torch.zeros(n, device="cuda", dtype=torch.float64)
    dh, dw = torch.zeros_like(H) if train else None, torch.zeros_like(W) if train else None
    for r0 in range(0, n, 1024):  # rows at a time, so that the logits fit
        rows = torch.arange(r0, min(n, r0 + 1024), device="cuda")
        rows = rows[y[rows] >= 0]
        if not rows.numel():
            continue
        L = H[rows] @ W.T
        lse = torch.logsumexp(L, dim=1)
        loss[rows] = lse - L[torch.arange(len(rows), device="cuda"), y[rows]] + case["z"] * lse ** 2
        if train:
            P = torch.softmax(L, dim=1) * (1 + 2 * case["z"] * lse)[:, None]
            P[torch.arange(len(rows), device="cuda"), y[rows]] -= 1.0
            dh[rows] = P @ W / count
            dw += P.T @ H[rows] / count
    return dict(loss=loss, dh=dh, dw=dw) if train else dict(loss=loss)


def exact(case, seed):
    if case["op"].startswith("xent"):
        return _exact_xent(case, seed)
    q, k, dq, dk, gq, gk, pos = _rot_inputs(case, seed)
    f, m = _frequencies(case)
    # the pair as a complex number, turned by multiplication
    angle = pos.double()[..., None] * torch.tensor(f, device="cuda", dtype=torch.float64)
    turn = torch.polar(torch.full_like(angle, m), angle)[:, :, None]
    o, r = case["offset"], case["rot"]

    def rotate(x, by):
        y = x.double().clone()
        part = y[..., o:o + r]
        pairs = part.unflatten(-1, (2, r // 2)).transpose(-1, -2) if case["layout"] == "half" else part.unflatten(
            -1, (r // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * by)
        y[..., o:o + r] = (z.transpose(-1, -2) if case["layout"] == "half" else z).flatten(-2)
        return y

    if case["op"] == "rotary":
        return dict(y=rotate(q, turn))
    if case["op"] == "rotary_inverse":
        return dict(y=rotate(q, turn.conj()))

    def normed(x, gain):
        x = x.double()
        return x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * gain.double()

    if case["op"] == "qk_fwd":
        return dict(q=rotate(normed(q, gq), turn), k=rotate(normed(k, gk), turn))

    def gradient(dy, x, gain):
        """From the derivative of x / root: dx = (w - x (w . x) / (dim root^2)) / root with w = gain e."""
        e, x = rotate(dy, turn.conj()), x.double()
        root = (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
        w = gain.double() * e
        dx = (w - x * (w * x).sum(-1, keepdim=True) / (case["dim"] * root ** 2)) / root
        return dx, torch.einsum("bshd,bshd->d", e, x / root)

    (a, c), (b, d) = gradient(dq, q, gq), gradient(dk, k, gk)
    return dict(dq=a, dk=b, dgq=c, dgk=d)
