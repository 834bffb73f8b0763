"""Cases of the operators of a block around its projections: attention with its
gradients and its form for single tokens, the residual update between two
blocks with the norms on either side of it, and dropout.

Each case's inputs are made on the GPU from a seed.  With ``own`` false,
``run`` computes the operator from elementary torch operations in 32 bits,
rounded once at the end; with ``own`` true it calls the framework.
``exact`` computes the same outputs in 64 bits.

Attention.  Queries (batch, sq, hq, dk), keys (batch, sk, hk, dk), values
(batch, sk, hk, dv); query head h reads key head h // (hq / hk).  Query i of a
sequence with lq queries and lk keys sees the keys j < lk with

    j <= i + lk - lq                     (causal: the last query sees all keys)
    j >  i + lk - lq - window            (window > 0)
    start(i) <= j < end(i)               (documents: those of i's document)

and y_i = sum_j softmax_j(scale q_i k_j) v_j; 0 where nothing is seen.

Residual update of rows of d elements, with rho(x) = 1 / sqrt(mean x^2 + eps):

    u  = block rho(block) post_gain      (or block itself)
    x' = x + scale gate(a) drop(u)       (gate: sigmoid, or a itself)
    h  = x' rho(x') pre_gain

Dropout.  Element e takes 16 bits of the counter generator of Salmon, Moraes,
Dror and Shaw ("Parallel random numbers: as easy as 1, 2, 3", 4 x 32 bits, ten
rounds) under the key `seed` at the counter (e // 8, offset): bits 16 (e % 2) of
word (e % 8) // 2.  Values below round(65536 p) drop it; what is kept is
divided by the share kept.
"""

import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "f32"
DTYPES = {BF16: torch.bfloat16, F32: torch.float32}
EPS = 1e-6


def _attn(name, op, batch, sq, sk, hq, hk, dk, dv, causal=True, window=0, spread=0.0, documents=0):
    return dict(name=name, op=op, batch=batch, sq=sq, sk=sk, hq=hq, hk=hk, dk=dk, dv=dv, causal=causal, window=window,
                spread=spread, documents=documents)


def listed():
    return [
        # 16 query and 4 key heads of 128 (2048 and 512 wide projections), training length, both passes
        _attn("attention_train_8192", "train", 2, 8192, 8192, 16, 4, 128, 128),
        # 32 heads of 128 + 64 for the scores and 128 for the values, a padded batch
        _attn("attention_train_192_padded", "train", 6, 777, 777, 32, 32, 192, 128, spread=0.8),
        # documents packed into one row
        _attn("attention_train_documents", "train", 1, 8192, 8192, 16, 4, 128, 128, documents=13),
        # the small example's batch: latency
        _attn("attention_train_48", "train", 16, 48, 48, 4, 2, 32, 32),
        # a chunk of a prompt against what the cache holds
        _attn("attention_chunk_of_prompt", "forward", 1, 512, 32768, 16, 4, 128, 128),
        # one token of each of eight sequences over caches of different fill
        _attn("attention_token_65536", "forward", 8, 1, 65536, 16, 4, 128, 128, spread=0.5),
        # ... and of one short one: latency
        _attn("attention_token_48", "forward", 1, 1, 48, 4, 2, 32, 32),
        # between two blocks in training: norm after, learned scale, norm before the next
        dict(name="residual_norm_32768x2048", op="residual", n=32768, d=2048, post=True, pre=True, gate="none",
             scale="vector", p=0.0, x=BF16, b=BF16),
        # ... its gradients, with a gate and dropout
        dict(name="residual_norm_backward_32768x2048", op="residual_back", n=32768, d=2048, post=True, pre=True,
             gate="sigmoid", scale="vector", p=0.1, x=BF16, b=BF16),
        # ... one token of eight sequences while answering, the stream held in 32 bits
        dict(name="residual_norm_8x2048", op="residual", n=8, d=2048, post=True, pre=True, gate="none",
             scale="vector", p=0.0, x=F32, b=BF16),
        # dropout of a block's output
        dict(name="dropout_32768x2048", op="dropout", n=32768, d=2048, p=0.1, x=BF16),
        # odd sizes in 32 bits
        dict(name="dropout_1023x1031", op="dropout", n=1023, d=1031, p=0.5, x=F32),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["train", "train", "forward", "token", "residual", "residual_back", "dropout"])
    if kind in ("train", "forward", "token"):
        while True:
            dk, dv = rng.choice([(32, 32), (64, 64), (72, 72), (80, 80), (96, 96), (128, 128), (128, 128), (192, 128)])
            hk = rng.choice([1, 2, 4, 8])
            hq = hk * rng.choice([1, 2, 3, 4, 8])
            sk = _log_int(rng, 1, 65536 if kind == "token" else 16384)
            sq = sk if kind == "train" else 1 if kind == "token" else _log_int(rng, 1, sk)
            batch = rng.choice([1, 1, 2, 3, 6])
            documents = rng.choice([0, 0, 2, 7]) if kind == "train" and batch == 1 and sk >= 8 else 0
            c = _attn(None, "forward" if kind == "token" else kind, batch, sq, sk, hq, hk, dk, dv,
                      causal=kind == "token" or rng.random() < 0.7, documents=documents,
                      window=rng.choice([0, 0, 0, _log_int(rng, 1, 2 * sk)]),
                      spread=0.0 if documents else rng.choice([0.0, 0.0, 0.5, 1.0]))
            del c["name"]
            c["causal"] = c["causal"] or c["window"] > 0
            # (no more scores, and no more operations on them, than the largest listed case)
            if batch * hq * sq * sk <= 2 * 16 * 8192 * 8192 and sq * sk * batch * hq * (dk + dv) <= 2 * 16 * 8192 * 8192 * 256:
                return c
    n, d = _log_int(rng, 1, 32768), _log_int(rng, 8, 8192)
    x = rng.choice([BF16, BF16, F32])
    while n * d > 32768 * 2048:
        n //= 2
    if kind == "dropout":
        return dict(op=kind, n=n, d=d, p=rng.choice([0.05, 0.1, 0.5]), x=x)
    return dict(op=kind, n=n, d=d - d % rng.choice([1, 2, 8, 8]), post=rng.random() < 0.7, pre=rng.random() < 0.8,
                gate=rng.choice(["none", "none", "sigmoid", "linear", "row"]), scale=rng.choice(["none", "one", "vector"]),
                p=rng.choice([0.0, 0.0, 0.1]), x=x, b=rng.choice([x, BF16]))


# ---------------------------------------------------------------------------
# what a case's masks are: lengths and documents follow from the case alone

def _lengths(c):
    """Keys of each sequence, from all of them down by ``spread``; the queries are the
    last ones of their sequence."""
    lk = [int(round(c["sk"] * (1.0 - c["spread"] * b / max(1, c["batch"] - 1)))) for b in range(c["batch"])]
    return [min(c["sq"], n) for n in lk], lk


def _starts(c):
    """First tokens of the documents (uneven lengths) and the end of the last."""
    at = sorted(set(int(c["sk"] * (i / c["documents"]) ** 1.5) for i in range(c["documents"])))
    return at + [c["sk"] - c["sk"] // 50]  # a little padding behind the last


def _bounds(c):
    """Keys [low, high) that each query of each sequence sees (batch x sq, integers)."""
    lq, lk = (np.array(v)[:, None] for v in _lengths(c))
    i = np.arange(c["sq"])[None, :]
    at = i + lk - lq
    high = np.minimum(lk, at + 1) if c["causal"] else np.broadcast_to(lk, at.shape)
    low = np.maximum(0, at - c["window"] + 1) if c["window"] else np.zeros_like(at)
    if c["documents"]:
        s = np.array(_starts(c))
        doc = np.searchsorted(s, i, side="right") - 1
        inside = doc < len(s) - 1
        first, last = s[np.minimum(doc, len(s) - 1)], s[np.minimum(doc + 1, len(s) - 1)]
        low, high = np.maximum(low, first), np.where(inside, np.minimum(high, last), 0)
    high = np.where(i < lq, np.maximum(high, low), low)
    return low, high


# ---------------------------------------------------------------------------
# inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return lambda *shape: torch.randn(*shape, generator=g, device="cuda")


def _attn_inputs(c, seed):
    made = _generator(seed)
    # normed and rotated queries and keys, values as their projection leaves them
    q = (1.2 * made(c["batch"], c["sq"], c["hq"], c["dk"])).to(torch.bfloat16)
    k = (1.2 * made(c["batch"], c["sk"], c["hk"], c["dk"])).to(torch.bfloat16)
    v = (0.7 * made(c["batch"], c["sk"], c["hk"], c["dv"])).to(torch.bfloat16)
    dy = made(c["batch"], c["sq"], c["hq"], c["dv"]).to(torch.bfloat16) if c["op"] == "train" else None
    return q, k, v, dy


def _rows_inputs(c, seed):
    made = _generator(seed)
    n, d, xt = c["n"], c["d"], DTYPES[c["x"]]
    s = dict(x=made(n, d).to(xt), seed=1000003 * int(seed) + 17, offset=5)
    if c["op"] == "dropout":
        return s
    bt = DTYPES[c["b"]]
    s["block"] = (0.5 * made(n, d)).to(bt)
    s["gate"] = None if c["gate"] == "none" else made(n, 1 if c["gate"] == "row" else d).to(bt)
    s["scale"] = None if c["scale"] == "none" else 0.3 + 0.1 * made(1 if c["scale"] == "one" else d)
    s["post_gain"] = 1.0 + 0.2 * made(d) if c["post"] else None
    s["pre_gain"] = 1.0 + 0.2 * made(d) if c["pre"] else None
    if c["op"] == "residual_back":
        s["dx"] = made(n, d).to(xt)
        s["dh"] = made(n, d).to(bt) if c["pre"] else None
    return s


def prepare(case, seed):
    if case["op"] not in ("train", "forward"):
        return dict(case=case, **_rows_inputs(case, seed))
    q, k, v, dy = _attn_inputs(case, seed)
    ints = lambda a: torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    lq, lk = _lengths(case)
    ragged = case["spread"] > 0
    low, high = _bounds(case)
    return dict(case=case, q=q, k=k, v=v, dy=dy, q_lengths=ints(lq) if ragged else None,
                k_lengths=ints(lk) if ragged else None, documents=ints(_starts(case)) if case["documents"] else None,
                low=ints(low), high=ints(high))


# ---------------------------------------------------------------------------
# plain forms, in 32 bits

def _plain_attention(s):
    c = s["case"]
    b, sq, sk, hq, hk, dk, dv = (c[n] for n in ("batch", "sq", "sk", "hq", "hk", "dk", "dv"))
    q = s["q"].float().view(b, sq, hk, hq // hk, dk).permute(0, 2, 3, 1, 4)
    k, v = (t.float().transpose(1, 2)[:, :, None] for t in (s["k"], s["v"]))
    j = torch.arange(sk, device="cuda")
    seen = ((j >= s["low"][..., None]) & (j < s["high"][..., None]))[:, None, None]
    score = (q @ k.transpose(-1, -2)) * dk ** -0.5
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(dim=-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)  # (nothing seen: any number)
    P = torch.exp(score.sub_(top))
    P /= P.sum(dim=-1, keepdim=True).clamp_min(1e-37)
    y = P @ v
    back = lambda t: t.permute(0, 3, 1, 2, 4).reshape(b, t.shape[3], -1, t.shape[4]).to(torch.bfloat16)  # noqa: E731
    if c["op"] == "forward":
        return dict(y=back(y))
    dy = s["dy"].float().view(b, sq, hk, hq // hk, dv).permute(0, 2, 3, 1, 4)
    ds = dy @ v.transpose(-1, -2)
    ds -= (dy * y).sum(dim=-1, keepdim=True)
    ds *= P
    ds *= dk ** -0.5
    return dict(y=back(y), dq=back(ds @ k), dk=back((ds.transpose(-1, -2) @ q).sum(dim=2, keepdim=True)),
                dv=back((P.transpose(-1, -2) @ dy).sum(dim=2, keepdim=True)))


def _keep(count, p, seed, offset):
    """Which of `count` elements are kept, and the share kept: the generator on
    int64 values (their products wrap, as 64-bit ones do)."""
    low = 0xFFFFFFFF
    i = torch.arange((count + 7) // 8, device="cuda", dtype=torch.int64)
    a, b = i & low, i >> 32
    c, d = torch.full_like(i, offset & low), torch.full_like(i, offset >> 32 & low)
    k0, k1 = seed & low, seed >> 32 & low
    for _ in range(10):
        u, v = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = (v >> 32 & low) ^ b ^ k0, v & low, (u >> 32 & low) ^ d ^ k1, u & low
        k0, k1 = k0 + 0x9E3779B9 & low, k1 + 0xBB67AE85 & low
    bits = torch.stack((a & 0xFFFF, a >> 16, b & 0xFFFF, b >> 16, c & 0xFFFF, c >> 16, d & 0xFFFF, d >> 16), dim=1)
    limit = round(65536 * p)
    return bits.view(-1)[:count] >= limit, 1.0 - limit / 65536.0


def _plain_drop(u, s):
    if s["case"]["p"] == 0.0:
        return u, None
    keep, share = _keep(u.numel(), s["case"]["p"], s["seed"], s["offset"])
    m = keep.view(u.shape).float() / share
    return u * m, m


def _gate(c, a):
    return torch.sigmoid(a.float()) if c["gate"] == "sigmoid" else a.float()


def _plain_residual(s):
    c = s["case"]
    rho = lambda t: torch.rsqrt(t.square().mean(dim=-1, keepdim=True) + EPS)  # noqa: E731
    xt, bt = DTYPES[c["x"]], DTYPES[c["b"]]
    o = s["block"].float()
    r = rho(o) if c["post"] else None
    u = o * r * s["post_gain"] if c["post"] else o
    scale = 1.0 if s["scale"] is None else s["scale"]
    gate = 1.0 if s["gate"] is None else _gate(c, s["gate"])
    u, mask = _plain_drop(u, s)
    if c["op"] == "residual":
        x = s["x"].float() + scale * gate * u
        out = dict(x=x.to(xt))
        if c["pre"]:
            out["h"] = (x * rho(x) * s["pre_gain"]).to(bt)
        return out
    x, g, out = s["x"].float(), s["dx"].float(), {}  # x: the updated one
    if c["pre"]:
        t = rho(x)
        dh, n = s["dh"].float(), x * t
        w = dh * s["pre_gain"]
        g = g + t * (w - n * (w * n).mean(dim=-1, keepdim=True))
        out["dpre_gain"] = (dh * n).sum(dim=0)
    out["dx"] = g.to(xt)
    if s["scale"] is not None:
        ds = g * gate * u
        out["dscale"] = ds.sum(dim=0) if c["scale"] == "vector" else ds.sum().view(1)
    if s["gate"] is not None:
        da = g * scale * u * (gate * (1.0 - gate) if c["gate"] == "sigmoid" else 1.0)
        out["dgate"] = (da.sum(dim=-1, keepdim=True) if c["gate"] == "row" else da).to(bt)
    du = g * scale * gate
    if mask is not None:
        du = du * mask
    if c["post"]:
        n = o * r
        out["dpost_gain"] = (du * n).sum(dim=0)
        w = du * s["post_gain"]
        du = r * (w - n * (w * n).mean(dim=-1, keepdim=True))
    out["dblock"] = du.to(bt)
    return out


def _own(s):
    from adamw_optimizer_step_gb300 import layers
    c = s["case"]
    if c["op"] in ("train", "forward"):
        mask = dict(causal=c["causal"], window=c["window"], q_lengths=s["q_lengths"], k_lengths=s["k_lengths"],
                    documents=s["documents"])
        if c["op"] == "forward":
            return dict(y=layers.attention(s["q"], s["k"], s["v"], **mask))
        y, lse = layers.attention(s["q"], s["k"], s["v"], return_lse=True, **mask)
        dq, dk, dv = layers.attention_backward(s["dy"], s["q"], s["k"], s["v"], y, lse, **mask)
        return dict(y=y, dq=dq, dk=dk, dv=dv)
    if c["op"] == "dropout":
        return dict(y=layers.dropout(s["x"], c["p"], s["seed"], offset=s["offset"]))
    rest = dict(post_norm=c["post"], pre_norm=c["pre"], post_gain=s["post_gain"], pre_gain=s["pre_gain"], gate=s["gate"],
                gate_kind="sigmoid" if c["gate"] == "sigmoid" else "linear", scale=s["scale"], dropout=c["p"],
                seed=s["seed"], offset=s["offset"], eps=EPS)
    if c["op"] == "residual":
        x, h = layers.residual_norm(s["x"], s["block"], **rest)
        return dict(x=x, h=h) if c["pre"] else dict(x=x)
    grads = layers.residual_norm_backward(s["dx"], s["dh"], s["x"], s["block"], **rest)
    return {name: t for name, t in grads.items() if t is not None}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op in ("train", "forward"):
        return _plain_attention(state)
    if op == "dropout":
        return dict(y=_plain_drop(state["x"].float(), state)[0].to(state["x"].dtype))
    return _plain_residual(state)


def work(case):
    """Inputs read once, outputs written once; of attention the products of the
    pairs of a query and a key that it sees (gradients: the scores once more,
    and a product each for dP, dV, dQ and dK)."""
    c = case
    if c["op"] in ("train", "forward"):
        low, high = _bounds(c)
        pairs = float((high - low).sum()) * c["hq"]
        lq, lk = (float(sum(v)) for v in _lengths(c))
        queries, keys = lq * c["hq"] * (c["dk"] + c["dv"]), lk * c["hk"] * (c["dk"] + c["dv"])
        if c["op"] == "forward":
            return dict(bytes=2.0 * (queries + keys), flops=2.0 * pairs * (c["dk"] + c["dv"]))
        # read q, k, v, dy; written y, dq, dk, dv
        return dict(bytes=2.0 * (2 * queries + 2 * keys), flops=pairs * (8.0 * c["dk"] + 6.0 * c["dv"]))
    size = {BF16: 2.0, F32: 4.0}
    elements, x = float(c["n"]) * c["d"], size[c["x"]]
    if c["op"] == "dropout":
        return dict(bytes=2 * x * elements, flops=30.0 * elements)
    b, gate = size[c["b"]], 0.0 if c["gate"] == "none" else 1.0 / c["d"] if c["gate"] == "row" else 1.0
    tables = 4.0 * (c["post"] * c["d"] + c["pre"] * c["d"] + {"none": 0, "one": 1, "vector": c["d"]}[c["scale"]])
    if c["op"] == "residual":
        return dict(bytes=elements * (2 * x + b * (1 + c["pre"] + gate)) + tables, flops=12.0 * elements)
    # x' is needed for its norm alone, the block's output only where something multiplies it
    reads_x, reads_o = c["pre"], c["post"] or c["gate"] != "none" or c["scale"] != "none"
    return dict(bytes=elements * (x * (2 + reads_x) + b * (1 + c["pre"] + reads_o + 2 * gate)) + 2 * tables,
                flops=30.0 * elements)


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_attention(c, seed):
    q, k, v, dy = (None if t is None else t.double() for t in _attn_inputs(c, seed))
    low, high = (torch.as_tensor(np.ascontiguousarray(t), device="cuda") for t in _bounds(c))
    j = torch.arange(c["sk"], device="cuda")
    group, beta = c["hq"] // c["hk"], 1.0 / math.sqrt(c["dk"])
    y = torch.zeros(c["batch"], c["sq"], c["hq"], c["dv"], dtype=torch.float64, device="cuda")
    train = c["op"] == "train"
    gq, gk, gv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for b in range(c["batch"]):
        for i0 in range(0, c["sq"], 2048):  # rows and heads at a time, so that the scores fit
            rows = slice(i0, min(c["sq"], i0 + 2048))
            first, last = int(low[b, rows].min()), int(high[b, rows].max())
            if last <= first:
                continue
            keys = slice(first, last)
            hidden = (j[keys] < low[b, rows, None]) | (j[keys] >= high[b, rows, None])
            blank = hidden.all(dim=1)
            for h in range(c["hq"]):
                A, K, V = q[b, rows, h], k[b, keys, h // group], v[b, keys, h // group]
                t = (beta * (A @ K.T)).masked_fill(hidden, -math.inf)
                p = torch.softmax(t, dim=1)
                p[blank] = 0.0
                y[b, rows, h] = p @ V
                if train:
                    D = dy[b, rows, h]
                    gv[b, keys, h // group] += p.T @ D
                    e = D @ V.T
                    e = beta * p * (e - torch.einsum("ij,ij->i", p, e)[:, None])
                    gq[b, rows, h] = e @ K
                    gk[b, keys, h // group] += e.T @ A
    return dict(y=y, dq=gq, dk=gk, dv=gv) if train else dict(y=y)


def _exact_mask(c, s):
    """1 / share where an element is kept, 0 where it is dropped, on the host in unsigned integers."""
    shape = s["x"].shape
    if c["p"] == 0.0:
        return torch.ones(shape, dtype=torch.float64, device="cuda")
    count = s["x"].numel()
    half, word = np.uint64(32), np.uint64(0xFFFFFFFF)
    x = np.zeros((4, -(-count // 8)), dtype=np.uint64)
    x[0] = np.arange(x.shape[1], dtype=np.uint64)
    x[2] = np.uint64(s["offset"])
    key = [s["seed"] % 2 ** 32, s["seed"] // 2 ** 32]
    for r in range(10):
        left, right = np.uint64(0xD2511F53) * x[0], np.uint64(0xCD9E8D57) * x[2]
        ka, kb = (np.uint64((key[n] + r * w) % 2 ** 32) for n, w in enumerate((0x9E3779B9, 0xBB67AE85)))
        x = np.stack(((right >> half) ^ x[1] ^ ka, right & word, (left >> half) ^ x[3] ^ kb, left & word))
    halves = x.T.astype("<u4").copy().view("<u2").reshape(-1)[:count]  # low half of each word first
    cut = int(math.floor(65536 * c["p"] + 0.5))
    kept = torch.as_tensor((halves.astype(np.int32) >= cut), device="cuda")
    return kept.view(shape).double() * (65536.0 / (65536 - cut))


def _exact_rows(c, seed):
    s = _rows_inputs(c, seed)
    m = _exact_mask(c, s)
    if c["op"] == "dropout":
        return dict(y=s["x"].double() * m)
    wide = lambda t, other=1.0: other if t is None else t.double()  # noqa: E731
    x, o, gain_after, gain_before = wide(s["x"]), wide(s["block"]), wide(s["post_gain"]), wide(s["pre_gain"])
    beta, a = wide(s["scale"]), wide(s["gate"])
    root = lambda t: (torch.einsum("ij,ij->i", t, t) / c["d"] + EPS).sqrt()[:, None]  # noqa: E731
    gate = 1.0 / (1.0 + torch.exp(-a)) if c["gate"] == "sigmoid" else a
    unit = o / root(o) if c["post"] else o
    if c["op"] == "residual":
        x = x + beta * gate * m * (unit * gain_after)
        return dict(x=x, h=x / root(x) * gain_before) if c["pre"] else dict(x=x)

    def through(w, t):
        """Gradient of t / root(t) against w."""
        r = root(t)
        return (w - t * (torch.einsum("ij,ij->i", w, t)[:, None] / (c["d"] * r ** 2))) / r

    g, out = s["dx"].double(), {}
    if c["pre"]:
        dh = s["dh"].double()
        out["dpre_gain"] = torch.einsum("ij,ij->j", dh, x / root(x))
        g = g + through(dh * gain_before, x)
    out["dx"] = g
    gm = g * m
    if s["scale"] is not None:
        t = gm * gate * unit * gain_after
        out["dscale"] = t.sum(dim=0) if c["scale"] == "vector" else t.sum().reshape(1)
    if s["gate"] is not None:
        t = gm * beta * unit * gain_after * (torch.exp(-a) * gate * gate if c["gate"] == "sigmoid" else 1.0)
        out["dgate"] = t.sum(dim=1, keepdim=True) if c["gate"] == "row" else t
    du = gm * beta * gate
    if c["post"]:
        out["dpost_gain"] = torch.einsum("ij,ij->j", du, unit)
        du = through(du * gain_after, o)
    out["dblock"] = du
    return out


def exact(case, seed):
    if case["op"] not in ("train", "forward"):
        return _exact_rows(case, seed)
    # the largest: about 2 x 16 x 8192 x 8192 x 128 x 14 operations in 64 bits
    return _exact_attention(case, seed)
