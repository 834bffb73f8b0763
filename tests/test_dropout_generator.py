"""Dropout's generator against the published known answers of Philox 4x32-10 (the vectors that
come with Salmon, Moraes, Dror and Shaw's own implementation): counters and keys of zeros, of
ones and of pi's digits.  With words of their own in every place, an exchange of two of them
shows, in the generator and in the order in which a seed, an element's number and an offset
become its words."""

import numpy as np
import pytest
import torch

from adamw_optimizer_step_gb300 import layers

LOW = 0xFFFFFFFF
# counter (four words), key (two), answer (four)
KNOWN = [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((LOW,) * 4, (LOW,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
]


def philox(counter, key):
    """Ten rounds, as the paper has them: of each pair of words one is multiplied; the products'
    low halves stay, the high ones go to the other pair with its second word and a word of the key."""
    c, k = list(counter), list(key)
    for _ in range(10):
        p0, p1 = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & LOW, (p0 >> 32) ^ c[3] ^ k[1], p0 & LOW]
        k = [(k[0] + 0x9E3779B9) & LOW, (k[1] + 0xBB67AE85) & LOW]
    return tuple(c)


def draws(seed, eighth, offset):
    """The 16-bit draws of elements 8 eighth .. 8 eighth + 7, as the C header orders words and halves."""
    w = philox((eighth & LOW, eighth >> 32, offset & LOW, offset >> 32), (seed & LOW, seed >> 32))
    return [w[e // 2] >> 16 * (e % 2) & 0xFFFF for e in range(8)]


@pytest.mark.parametrize("counter,key,answer", KNOWN)
def test_known_answers(counter, key, answer):
    assert philox(counter, key) == answer
    seed, eighth, offset = (lo | hi << 32 for lo, hi in (key, counter[:2], counter[2:]))
    assert [lo | hi << 16 for lo, hi in zip(draws(seed, eighth, offset)[::2], draws(seed, eighth, offset)[1::2])] == list(answer)


@pytest.mark.gpu
@pytest.mark.parametrize("seed,offset", [(lo | hi << 32, c[2] | c[3] << 32) for c, (lo, hi), _ in KNOWN] + [(1 << 32, 1), (1, 1 << 32)])
def test_the_kernels_draws(seed, offset):
    """Each draw pinned from both sides: an element is dropped from a probability of one step above its
    draw on, and kept up to the draw itself.  In words that differ, of dropout alone and in the update."""
    from adamw_optimizer_step_gb300 import build
    build.build()
    want = [d for eighth in range(4) for d in draws(seed, eighth, offset)]
    x = torch.ones(32, device="cuda")
    for e in range(32):
        for step, kept in ((0, True), (1, False)):
            p = (want[e] + step) / 65536.0
            if p >= 1.0:
                continue
            y = layers.dropout(x, p, seed, offset=offset)
            assert [v != 0 for v in y.tolist()] == [d >= want[e] + step for d in want]
            assert bool(y[e] != 0) == kept
    # rows of an update draw by the element's number in all of them
    for n, d in ((4, 8), (2, 16), (32, 1)):
        z, _ = layers.residual_norm(torch.zeros(n, d, device="cuda"), x.view(n, d), pre_norm=False, dropout=0.5, seed=seed, offset=offset)
        assert np.array_equal((z != 0).flatten().cpu().numpy(), np.array(want) >= 32768)
