"""Corners of the rotary and cross-entropy operators that need a GPU: memory of the loss
in autograd, frequencies of either sign at long positions.

Tolerances are those of test_gpu_rotary.py and test_gpu_xent.py, derived there; where
another one is taken its reason stands beside it."""

import math
from fractions import Fraction

import pytest
import torch

from adamw_optimizer_step_gb300 import _binding as B
from adamw_optimizer_step_gb300 import layers
from tests.test_gpu_xent import U, Want, close, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from adamw_optimizer_step_gb300 import build
    build.build()
    B.lib()


# ---------------------------------------------------------------------------
# memory of the loss in autograd

# small tensors of a call (lse, totals, the mean, upstream)
SLACK = 1 << 16


def peak_of(call):
    """Bytes that the call asks for at its peak and holds afterwards, and what it returns.
    (The blocks that torch hands out for them may be up to 1 MB larger each.)"""
    held = lambda which: torch.cuda.memory_stats()["requested_bytes.all." + which]  # noqa: E731
    torch.cuda.synchronize()
    base = held("current")
    torch.cuda.reset_peak_memory_stats()
    kept = call()
    torch.cuda.synchronize()
    return held("peak") - base, held("current") - base, kept


def test_memory_of_the_loss():
    """Without gradients: the workspace of the losses alone, and the same losses.  With
    them: one workspace from the forward to the backward pass, given back after it
    although the loss is still held."""
    n, v, d = 500, 20011, 512
    H, W, y = inputs(n, v, d, 7, ignored=0.1)
    small, large = (B.gbo_xent_workspace_bytes(n, v, d, grad) for grad in (False, True))
    assert large > small + 2 * n * v  # the logits are kept
    H.requires_grad_()
    W.requires_grad_()
    want = Want(H.detach(), W.detach(), y)
    layers.linear_cross_entropy_loss(H, W, y)  # (first-call set-up is no part of it)
    with torch.no_grad():
        peak, _, loss = peak_of(lambda: layers.linear_cross_entropy_loss(H, W, y))
    assert peak <= small + SLACK
    close(loss, want.total / want.weight, want.total_tol / want.weight, torch.float32)

    def step():
        loss = layers.linear_cross_entropy_loss(H, W, y)
        loss.backward()
        return loss

    grads = 2 * (n + v) * d
    peak, left, loss = peak_of(step)
    assert large <= peak <= large + grads + SLACK
    assert left <= grads + SLACK and loss.grad_fn is not None


# ---------------------------------------------------------------------------
# angles

# more digits than any rational here needs
PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


@pytest.mark.parametrize("sign", [1, -1])
def test_angles_keep_their_bound(sign):
    """Against rationals with 80 digits of pi: beside the rounding of the pass (64 u of the
    pair, see test_gpu_rotary.py) the angle is off by at most |t| (2^-52 |f| + 2^-61), the
    bound that gbo.h states, for frequencies of either sign."""
    freq = [sign * f for f in (1.0, 0.3, 1e-2, 1e-3, 1e-4, 1e-8, 2.0 ** -40, 17.5)]
    spec = layers.RotarySpec(16, frequencies=freq)
    x = torch.randn(1, 6, 1, 16, generator=torch.Generator().manual_seed(4)).cuda()
    values = [1, 2 ** 24 + 1, 2 ** 31 + 3, 2 ** 40 + 12345, -(2 ** 33) - 7, 2 ** 52 + 1]
    got = layers.rotary(x, torch.tensor([values], device="cuda"), spec).double().cpu()
    for s, t in enumerate(values):
        for j, f in enumerate(freq):
            turns = Fraction(t) * Fraction(f) / (2 * PI)
            angle = 2 * math.pi * float(turns - math.floor(turns))
            c, sn = math.cos(angle), math.sin(angle)
            a, b = x[0, s, 0, j].item(), x[0, s, 0, j + 8].item()
            tol = (64 * U + abs(t) * (2.0 ** -52 * abs(f) + 2.0 ** -61)) * (abs(a) + abs(b))
            assert abs(got[0, s, 0, j].item() - (a * c - b * sn)) <= tol, (t, f)
            assert abs(got[0, s, 0, j + 8].item() - (a * sn + b * c)) <= tol, (t, f)
