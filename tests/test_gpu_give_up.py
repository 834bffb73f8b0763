"""Waits of the operators' kernels that run out, made to on the device without a fault: with
a short limit, on a copy that never starts, in kernels of those waits alone."""

import time

import pytest
import torch

from adamw_optimizer_step_gb300 import _binding as B
from adamw_optimizer_step_gb300 import layers

pytestmark = pytest.mark.gpu
LIMIT_US = 20000


@pytest.fixture(scope="module", autouse=True)
def built():
    from adamw_optimizer_step_gb300 import build
    build.build()
    B.lib()


def still_works():
    x = torch.ones(4, 1024, device="cuda")
    assert torch.equal(layers.residual_norm(x, x, pre_norm=False)[0], x + x)


@pytest.mark.parametrize("n,lost", [(8, -1), (2, -1), (8, 4), (8, 0), (3, 2), (8, 7), (64, 30), (1, 0)])
def test_a_rows_copy_that_does_not_land(n, lost):
    """The rows before it arrive; from its wait on no copy is started; those under way have
    landed when the kernel ends.  Stages: three."""
    rows = torch.arange(n, dtype=torch.int32, device="cuda").add(100).repeat_interleave(256).view(n, 256)
    found = torch.full((n + 2,), -7, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    B.gbo_testing_ring_give_up(rows, lost, found, status, LIMIT_US)
    torch.cuda.synchronize()
    took = time.perf_counter() - t0
    got = found.tolist()
    good = n if lost < 0 else lost
    assert got[:n] == [100 + r for r in range(good)] + [-1] * (n - good)
    # a row is asked for behind the join of the one two rows before it (three in the beginning)
    asked = n if lost < 0 else min(n, max(3, lost + 2))
    assert got[n] == asked
    last = {k % 3: k for k in range(max(0, asked - 3), asked)}  # each stage's last row
    assert got[n + 1] == sum(1 << s for s, k in last.items() if k != lost)
    if lost < 0:
        assert int(status) == 0
    else:
        assert int(status) == B.GBO_STATUS_TIMEOUT
        # one limit for the row, one for the last look at its stage
        assert 0.9e-6 * LIMIT_US < took < 0.5
    still_works()


@pytest.mark.parametrize("first", [0, 1, 2])
def test_attentions_waits_give_up_together(first):
    """The one with the short limit raises the flag, the others (two seconds) see it; the ring's
    tiles have landed, the cleaned one among them, when the kernel ends."""
    gen = torch.Generator().manual_seed(first)
    tokens = torch.randn(64, 64, generator=gen).to(torch.bfloat16).cuda()
    words = tokens.view(torch.int32)
    found = torch.full((10,), -7, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.gbo_testing_attn_give_up(tokens, first, found, status, LIMIT_US)
    got = found.tolist()
    assert int(status) == B.GBO_STATUS_TIMEOUT
    assert got[:3] == [0, 0, 0]
    assert all(0.9 * LIMIT_US < t < 50 * LIMIT_US for t in got[3:6]), got  # (half of their own)
    assert got[6] == 3 and got[7] == int(words[0, 0]) and got[8] == int(words[32 + 8, 0]) and got[9] == 0
    still_works()


def test_refused():
    rows = torch.zeros(2, 256, dtype=torch.int32, device="cuda")
    found, status = (torch.zeros(k, dtype=torch.int32, device="cuda") for k in (4, 1))
    for lost, limit in ((2, 10), (-2, 10), (0, 0), (0, 10 ** 7)):
        with pytest.raises(B.GboError):
            B.gbo_testing_ring_give_up(rows, lost, found, status, limit)
    tokens, found = torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(10, dtype=torch.int32, device="cuda")
    for first, limit in ((3, 10), (-1, 10), (0, 0), (0, 50001)):
        with pytest.raises(B.GboError):
            B.gbo_testing_attn_give_up(tokens, first, found, status, limit)
