"""Gradients of attention where rows see 64 keys or fewer, and values lie close together.

dS = P (dP - D) is a difference there: with v = c + w, c the same for every key and large, dP and
D are both near dy . c, and D from the output, which is rounded to bf16, would be off by up to
2^-8 sum |dy| |c| (c = 64, so y is off by up to 0.25 an element and D by some 0.14 sqrt(dv), while
dP - D is about sqrt(dv)).  D from the same p and dP as dS itself is not.

Tolerances, as in tests/test_gpu_attention.py but for D's own: with u = 2^-24, a score off by
2 dk u scale sum |q k|, p by e' = that + 64 u (|s| + |lse| + 1) and as much again of the forward's lse
(and (n + 64) u (|lse| + 1) of its sum), dP by E = 2 dv u sum |dy v|, so
    D    sum p (E + e' |dP|) + 2 n u sum p |dP|
    ds   p (E + tol(D)) + |ds| (e' + 2^-8 (1 + 2^-7)) + 8 u p (|dP| + |D|) + e' p (|dP| + |D|)
    dq   scale (sum tol(ds) |k| + 2 n u sum |ds k|) + 2^-8 |dq|, dk likewise over rows and heads."""

import math

import pytest
import torch

from adamw_optimizer_step_gb300 import _binding as B
from adamw_optimizer_step_gb300 import layers
from tests.test_gpu_attention import ints, seen_by

pytestmark = pytest.mark.gpu
U, R = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def built():
    from adamw_optimizer_step_gb300 import build
    build.build()
    B.lib()


def check(batch, sq, sk, hq, hk, dk, dv, seed=0, **mask):
    gen = torch.Generator().manual_seed(seed)
    made = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    q, k = (made(batch, n, h, dk).to(torch.bfloat16).cuda() for n, h in ((sq, hq), (sk, hk)))
    # 64 and a few halves: exact in bf16
    v = (64 + (2 * made(batch, sk, hk, dv)).round() / 2).to(torch.bfloat16).cuda()
    dy = made(batch, sq, hq, dv).to(torch.bfloat16).cuda()
    seen = seen_by(batch, sq, sk, **mask)[:, None, None]
    n = seen.sum(-1)
    dy[(n[:, 0, 0] > 64)] = 0  # (rows that see more say nothing here)
    g, scale = hq // hk, dk ** -0.5
    Q = q.double().view(batch, sq, hk, g, dk).permute(0, 2, 3, 1, 4)
    G = dy.double().view(batch, sq, hk, g, dv).permute(0, 2, 3, 1, 4)
    K, V = k.double().transpose(1, 2)[:, :, None], v.double().transpose(1, 2)[:, :, None]
    s = (scale * (Q @ K.transpose(-1, -2))).masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1, keepdim=True)
    p = torch.where(seen & ~torch.isinf(lse), torch.exp(s - torch.where(torch.isinf(lse), 0.0, lse)), 0.0)
    fin = lambda t: torch.where(torch.isfinite(t), t, 0.0).abs()  # noqa: E731
    e = 2 * dk * U * scale * (Q.abs() @ K.abs().transpose(-1, -2)) + 64 * U * (fin(s) + fin(lse) + 1)
    e = torch.where(seen, e, 0.0)
    e = e + e.amax(-1, keepdim=True) + (sk + 64) * U * (fin(lse) + 1)
    dP, E = G @ V.transpose(-1, -2), 2 * dv * U * (G.abs() @ V.abs().transpose(-1, -2))
    D = (p * dP).sum(-1, keepdim=True)
    tD = (p * (E + (e + 2 * sk * U) * dP.abs())).sum(-1, keepdim=True)
    ds = p * (dP - D)
    tds = p * (E + tD) + ds.abs() * (e + R * (1 + 2.0 ** -7)) + (8 * U + e) * p * (dP.abs() + D.abs())
    rows = lambda t: t.permute(0, 3, 1, 2, 4).reshape(batch, sq, hq, -1)  # noqa: E731
    keys = lambda t: t.sum(2).transpose(1, 2)  # noqa: E731
    m = sq * g
    want = dict(dq=(rows(scale * (ds @ K)), rows(scale * (tds @ K.abs() + 2 * sk * U * (ds.abs() @ K.abs())))),
                dk=(keys(scale * (ds.transpose(-1, -2) @ Q)),
                    keys(scale * ((tds + 2 * m * U * ds.abs()).transpose(-1, -2) @ Q.abs()))))
    y, lse32 = layers.attention(q, k, v, return_lse=True, **mask)
    got = dict(zip(("dq", "dk", "dv"), layers.attention_backward(dy, q, k, v, y, lse32, **mask)))
    for name, (value, tol) in want.items():
        off = (got[name].double() - value).abs() - tol * (1 + 2.0 ** -6) - R * value.abs() - 1e-30
        assert torch.isfinite(got[name]).all() and float(off.max()) <= 0, (name, float(off.max()), float(tol.max()))


HEADS = [(4, 2, 64, 64), (3, 3, 192, 128), (16, 1, 32, 32), (5, 1, 136, 72), (2, 1, 8, 8), (40, 1, 96, 128)]


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("tokens", [2, 9, 33, 64, 65, 150])
def test_first_tokens_of_a_sequence(heads, tokens):
    check(2, tokens, tokens, *heads, seed=tokens)
    if tokens <= 64:
        check(2, tokens, tokens, *heads, seed=tokens, causal=False)


@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_windows_documents_and_lengths(heads):
    for window in (9, 40, 64):
        check(1, 200, 200, *heads, window=window, seed=window)
        check(2, 70, 130, *heads, window=window, seed=window)
    check(1, 300, 300, *heads, documents=ints(0, 20, 84, 84, 150, 290), seed=1)
    check(1, 300, 300, *heads, documents=ints(0, 20, 84, 150, 290), causal=False, seed=2)
    check(1, 300, 300, *heads, documents=ints(*range(3, 290, 11)), seed=3)
    check(1, 900, 900, *heads, documents=ints(0, 17, 500, 530, 890), seed=3)  # (few documents among many tokens)
    lengths = ints(150, 64, 20)
    check(3, 150, 150, *heads, causal=False, k_lengths=lengths, seed=4)
    check(3, 150, 150, *heads, q_lengths=lengths, k_lengths=lengths, seed=5)
    check(3, 100, 40, *heads, q_lengths=ints(100, 30, 7), seed=6)
