"""The example model runs the operators and the optimizer together: its loss
falls, its single-token path gives what its whole-sequence path gives."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from adamw_optimizer_step_gb300 import build, _binding as B
    build.build()
    B.lib()


def test_example_trains_and_answers():
    from examples import tied_lm
    model, losses = tied_lm.train(40)
    # a uniform guess costs ln 512 = 6.2; the step of the sequence is learnt
    # within a few dozen steps
    assert losses[0] > 5.0 and losses[-1] < 0.7 * losses[0]
    tokens, nll = tied_lm.answer(model, [7, 9, 11, 13], 8)
    assert len(tokens) == 12 and len(nll) == 11
    # the same losses from one pass over the whole sequence; both compute in
    # bf16 between fp32 norms, in other orders of summation
    t = torch.tensor([tokens], device="cuda")
    with torch.no_grad():
        h = model.hidden(t[:, :-1], torch.arange(11, device="cuda"))
        table = model.embedding.weight.to(torch.bfloat16)
        whole = tied_lm.layers.linear_cross_entropy(h[0], table, t[0, 1:])
    assert torch.allclose(whole.cpu(), torch.tensor(nll), atol=0.15)


def test_example_gradients_match_plain_autograd():
    """Gradients of the whole example by its own operators against the same model with
    their formulas written in torch (float32 where the operators are)."""
    from examples import tied_lm
    from adamw_optimizer_step_gb300 import layers
    torch.manual_seed(3)
    model = tied_lm.TiedLM().cuda()
    tokens, labels = tied_lm.batch(torch.Generator().manual_seed(1), size=4, length=24)
    model.loss(tokens, labels).backward()
    ours = {n: p.grad.float().clone() for n, p in model.named_parameters()}
    for p in model.parameters():
        p.grad = None

    def plain_qk(q, k, gq, gk, pos, spec, eps=1e-6):
        out = []
        for x, g in ((q, gq), (k, gk)):
            x = x.float()
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * g
            f = torch.tensor(spec.frequencies, device=x.device, dtype=torch.float64)
            ang = (pos.double()[:, None] * f)[None, :, None]
            c, s = (ang.cos() * spec.magnitude).float(), (ang.sin() * spec.magnitude).float()
            a, b = x.chunk(2, dim=-1)
            out.append(torch.cat((a * c - b * s, a * s + b * c), -1).to(torch.bfloat16))
        return out

    def plain_loss(h, w, y, row_weight=None, z_loss=0.0, logit_scale=1.0, workspace_cap=0):
        logits = h.float() @ w.to(torch.bfloat16).float().T
        lse = torch.logsumexp(logits, -1)
        use = y >= 0
        loss = lse - logits.gather(1, y.clamp_min(0)[:, None])[:, 0] + z_loss * lse ** 2
        return loss[use].mean()

    kept = layers.qk_norm_rotary_autograd, layers.linear_cross_entropy_loss
    layers.qk_norm_rotary_autograd, layers.linear_cross_entropy_loss = plain_qk, plain_loss
    try:
        model.loss(tokens, labels).backward()
    finally:
        layers.qk_norm_rotary_autograd, layers.linear_cross_entropy_loss = kept
    for n, p in model.named_parameters():
        # both backward passes run through bf16 activations (2^-8 an element, a
        # dozen roundings on the longest path)
        off = (ours[n] - p.grad.float()).norm() / p.grad.float().norm()
        assert off <= 12 * 2.0 ** -8, (n, float(off))
