"""A small language model trained with the hybrid optimizer and the operators
around it, then asked for tokens one at a time.

    python examples/tied_lm.py [--steps 60]

Per block: a fused projection gives queries, keys and values; the q/k norms
(their gains on the AdamW path) and the rotation are one call each way; the
loss of the tied embedding (AdamW, float32) is one call each way.  The
projections step on the Muon path.  Sequences count upwards from a random
token with a random step, so what comes next is learnable in a few dozen steps.
"""

import argparse
import os
import sys

import torch
import torch.nn as nn
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from adamw_optimizer_step_gb300 import layers  # noqa: E402
from adamw_optimizer_step_gb300.routing import Block, HybridOptimizer, Layout, STANDARD_LAYOUTS  # noqa: E402

VOCAB, WIDTH, HEADS, KV_HEADS, DIM, FFN, BLOCKS = 512, 128, 4, 2, 32, 256, 2


class Attention(nn.Module):
    def __init__(self, spec):
        super().__init__()
        self.spec = spec
        self.heads = HEADS + 2 * KV_HEADS
        self.qkv = nn.Linear(WIDTH, self.heads * DIM, bias=False, dtype=torch.bfloat16)
        self.out = nn.Linear(HEADS * DIM, WIDTH, bias=False, dtype=torch.bfloat16)
        self.q_norm, self.k_norm = nn.RMSNorm(DIM), nn.RMSNorm(DIM)

    def forward(self, x, positions, cache=None):
        b, s, _ = x.shape
        heads = self.qkv(x).view(b, s, self.heads, DIM)
        q, k, v = heads.split((HEADS, KV_HEADS, KV_HEADS), dim=2)
        if torch.is_grad_enabled():
            q, k = layers.qk_norm_rotary_autograd(q, k, self.q_norm.weight, self.k_norm.weight, positions, self.spec)
        else:
            q, k = layers.qk_norm_rotary(q, k, self.q_norm.weight, self.k_norm.weight, positions, self.spec)
        if cache is not None:  # one token at a time: keys and values of the earlier ones
            cache.append((k, v))
            k, v = (torch.cat(t, dim=1) for t in zip(*cache))
        q, k, v = (t.float().transpose(1, 2) for t in (q, k, v))
        k, v = (t.repeat_interleave(HEADS // KV_HEADS, dim=1) for t in (k, v))
        score = q @ k.transpose(-1, -2) / DIM ** 0.5
        if cache is None:
            score = score.masked_fill(torch.ones(s, s, dtype=torch.bool, device=x.device).triu(1), float("-inf"))
        y = (score.softmax(-1) @ v).transpose(1, 2).reshape(b, s, HEADS * DIM)
        return self.out(y.to(torch.bfloat16))


class Layer(nn.Module):
    def __init__(self, spec):
        super().__init__()
        self.intermediate_size = FFN
        self.norm1, self.norm2 = nn.RMSNorm(WIDTH), nn.RMSNorm(WIDTH)
        self.attention = Attention(spec)
        self.gate_up_proj = nn.Linear(WIDTH, 2 * FFN, bias=False, dtype=torch.bfloat16)
        self.down = nn.Linear(FFN, WIDTH, bias=False, dtype=torch.bfloat16)

    def forward(self, x, positions, cache=None):
        x = x + self.attention(self.norm1(x.float()).to(torch.bfloat16), positions, cache)
        gate, up = self.gate_up_proj(self.norm2(x.float()).to(torch.bfloat16)).chunk(2, dim=-1)
        return x + self.down(F.silu(gate) * up)


class TiedLM(nn.Module):
    def __init__(self):
        super().__init__()
        spec = layers.RotarySpec(DIM, scaling=dict(kind="yarn", factor=4.0, trained=64.0, fast=32.0, slow=1.0))
        self.embedding = nn.Embedding(VOCAB, WIDTH)
        nn.init.normal_(self.embedding.weight, std=0.05)
        self.layers = nn.ModuleList(Layer(spec) for _ in range(BLOCKS))
        self.norm = nn.RMSNorm(WIDTH)

    def hidden(self, tokens, positions, caches=None):
        x = self.embedding(tokens).to(torch.bfloat16)
        for n, layer in enumerate(self.layers):
            x = layer(x, positions, None if caches is None else caches[n])
        return self.norm(x.float()).to(torch.bfloat16)

    def loss(self, tokens, labels):
        h = self.hidden(tokens, torch.arange(tokens.shape[1], device=tokens.device))
        return layers.linear_cross_entropy_loss(h.flatten(0, 1), self.embedding.weight, labels.flatten(), z_loss=1e-4)


def batch(generator, size=16, length=48):
    start = torch.randint(0, VOCAB, (size, 1), generator=generator)
    step = torch.randint(1, 4, (size, 1), generator=generator)
    tokens = ((start + step * torch.arange(length + 1)) % VOCAB).cuda()
    labels = tokens[:, 1:].clone()
    labels[:, :2] = -100  # the first two tokens say what the step is: no loss there
    return tokens[:, :-1], labels


def train(steps, seed=0):
    torch.manual_seed(seed)
    generator = torch.Generator().manual_seed(seed)
    model = TiedLM().cuda()
    # every head of the fused projection is a matrix of its own for Muon
    heads = Layout("qkv", ("heads",), lambda f, lin: (Block(lin.out_features, view=(f.heads, DIM, lin.in_features)),))
    opt = HybridOptimizer(model, muon_lr=0.02, adamw_lr=3e-3, layouts=STANDARD_LAYOUTS + (heads,))
    losses = []
    for _ in range(steps):
        loss = model.loss(*batch(generator))
        for p in model.parameters():
            p.grad = None
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    assert int(opt.status.item()) == 0
    return model, [float(x) for x in losses]


@torch.no_grad()
def answer(model, prompt, count):
    """Greedy continuation of one prompt, a token at a time over the kept keys
    and values, and the model's loss on each token it gives."""
    caches = [[] for _ in model.layers]
    tokens, losses = list(prompt), []
    table = model.embedding.weight.to(torch.bfloat16)
    for t in range(len(prompt) + count - 1):
        at = torch.tensor([[tokens[t]]], device="cuda")
        h = model.hidden(at, t, caches)[:, 0]
        if t + 1 >= len(prompt):
            tokens.append(int((h.float() @ table.float().T).argmax()))
        losses.append(float(layers.linear_cross_entropy(h, table, torch.tensor([tokens[t + 1]], device="cuda"))))
    return tokens, losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=120)
    a = ap.parse_args()
    trained, curve = train(a.steps)
    print("loss %.3f -> %.3f in %d steps" % (curve[0], curve[-1], a.steps))
    out, nll = answer(trained, [7, 9, 11, 13], 12)
    print("answer", out, "mean loss %.3f" % (sum(nll[3:]) / len(nll[3:])))
