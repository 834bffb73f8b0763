"""What the loss's autograd form does with its arguments, on the CPU: the library
calls are replaced by recorders."""

import pytest
import torch

from adamw_optimizer_step_gb300 import _binding as B
from adamw_optimizer_step_gb300 import layers


@pytest.fixture
def calls(monkeypatch):
    """Records the library calls of the loss instead of making them."""
    made = []

    def forward(h, w, labels, workspace, *, lse, totals, keep, **rest):
        made.append(dict(keep=keep, bytes=workspace.numel()))
        totals.copy_(torch.tensor([6.0, 2.0]))

    def backward(h, w, labels, lse, workspace, *, dh, dw, **rest):
        made.append(dict(keep=rest["keep"], bytes=workspace.numel()))
        for t in (dh, dw):
            if t is not None:
                t.fill_(0.5)

    monkeypatch.setattr(B, "gbo_xent_forward", forward)
    monkeypatch.setattr(B, "gbo_xent_backward", backward)
    monkeypatch.setattr(B, "gbo_xent_workspace_bytes", lambda n, v, d, grad=False, cap=0: 2000 if grad else 1000)
    return made


def inputs():
    return (torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(6, 8, dtype=torch.bfloat16),
            torch.zeros(4, dtype=torch.int64))


@pytest.mark.parametrize("name", ["row_weight", "z_loss", "logit_scale"])
def test_constants_that_require_a_gradient_are_refused(calls, name):
    """The loss has gradients by h and w alone: a weight or a scale that waits for one is
    told, not left without."""
    h, w, y = inputs()
    value = torch.ones(4) if name == "row_weight" else torch.tensor(1.0)
    with pytest.raises(ValueError, match=name):
        layers.linear_cross_entropy_loss(h.requires_grad_(), w, y, **{name: value.clone().requires_grad_()})
    assert not calls
    layers.linear_cross_entropy_loss(h, w, y, **{name: value}).backward()
    assert len(calls) == 2
    with torch.no_grad():  # nothing waits for a gradient here
        layers.linear_cross_entropy_loss(h, w, y, **{name: value.clone().requires_grad_()})


def test_the_norms_eps_is_a_constant_too():
    q = torch.zeros(1, 2, 1, 8)
    with pytest.raises(ValueError, match="eps"):
        layers.qk_norm_rotary_autograd(q, q, None, None, 0, layers.RotarySpec(8),
                                       eps=torch.tensor(1e-6, requires_grad=True))


def test_without_gradients_the_loss_takes_the_losses_own_path(calls):
    """Under no_grad and inference_mode nothing is kept for a backward pass: the workspace
    of the losses alone, although the table requires a gradient."""
    h, w, y = inputs()
    w.requires_grad_()
    for off in (torch.no_grad, torch.inference_mode):
        with off():
            loss = layers.linear_cross_entropy_loss(h, w, y)
        assert calls.pop() == dict(keep=False, bytes=1000) and loss.item() == 3.0 and not calls
    with torch.no_grad(), torch.enable_grad():
        layers.linear_cross_entropy_loss(h, w, y)
    assert calls.pop() == dict(keep=True, bytes=2000)
    layers.linear_cross_entropy_loss(h, w.detach(), y)  # nothing requires a gradient
    assert calls.pop() == dict(keep=False, bytes=1000)


def test_constants_given_as_tensors_are_read_when_the_call_is_made(calls, monkeypatch):
    """A tensor that changes afterwards changes neither an options record made earlier nor
    the backward pass, and its next value is taken."""
    spec, eps = layers.RotarySpec(8), torch.tensor(1e-3)
    assert abs(spec.with_eps(eps).eps - 1e-3) < 1e-9
    eps.fill_(1e-5)
    assert abs(spec.with_eps(eps).eps - 1e-5) < 1e-11
    assert spec.with_eps(1e-3) is spec.with_eps(torch.tensor(1e-3, dtype=torch.float64))

    given = []
    wrapped = {name: getattr(B, name) for name in ("gbo_xent_forward", "gbo_xent_backward")}
    for name, call in wrapped.items():
        monkeypatch.setattr(B, name, lambda *a, call=call, **k: (given.append((k["z_loss"], k["logit_scale"])),
                                                                call(*a, **k)))
    h, w, y = inputs()
    z, scale = torch.tensor(0.25), torch.tensor(0.5)
    loss = layers.linear_cross_entropy_loss(h.requires_grad_(), w, y, z_loss=z, logit_scale=scale)
    z.fill_(7.0), scale.fill_(7.0)
    loss.backward()
    assert given == [(0.25, 0.5)] * 2
