"""``rope_frequencies`` against values worked out by hand from its definition."""

import math

import pytest
import torch

from token_indexed_sparse_b200 import qsa


def _blend(dim, base, factor, kept, divided):
    """Frequencies of the pairs, the share divided by the factor growing from index kept to index divided."""
    out = []
    for i in range(dim // 2):
        share = min(max((i - kept) / (divided - kept), 0.0), 1.0)
        f = base ** (-2.0 * i / dim)
        out.append(f * (1.0 - share) + f / factor * share)
    return torch.tensor(out, dtype=torch.float64)


@pytest.mark.parametrize("dim,base,factor,length,fast,slow,kept,divided", [
    # pairs 10.47 and 22.51 make 32 turns and 1 over 4096 positions
    (64, 1e4, 4.0, 4096, 32.0, 1.0, 10, 23),
    # 23.60 and 39.65 of 64 over 32768 at base 10^6
    (128, 1e6, 8.0, 32768, 32.0, 1.0, 23, 40),
    # 11.31 and 35.39 make 64 turns and 2
    (256, 1e8, 16.0, 2048, 64.0, 2.0, 11, 36),
    # pair 0 makes 15.9 turns only (-1.21): the ramp starts there
    (32, 1e4, 2.0, 100, 32.0, 1.0, 0, 5),
    # a small base: every pair makes more than 32 turns (pair 15 the fewest), all are kept
    (32, 20.0, 2.0, 70000, 32.0, 1.0, 31, 50),
    # the ramp ends behind the last pair, at 15.97 of 8
    (16, 4.0, 2.0, 100, 64.0, 1.0, 0, 16),
])
def test_yarn_by_hand(dim, base, factor, length, fast, slow, kept, divided):
    at = [dim / 2 * math.log(length / (2 * math.pi * n), base) for n in (fast, slow)]
    assert max(math.floor(at[0]), 0) == kept and math.ceil(at[1]) == divided
    f, m = qsa.rope_frequencies(dim, base, scaling="yarn", factor=factor, original_len=length, fast_turns=fast,
                                slow_turns=slow, device="cpu")
    assert torch.allclose(f, _blend(dim, base, factor, kept, divided), rtol=1e-14, atol=0.0)
    assert m == 0.1 * math.log(factor) + 1.0


def test_yarn_pinned():
    f, m = qsa.rope_frequencies(64, 10000.0, scaling="yarn", factor=4.0, device="cpu")
    # 10^(-i / 8): pairs 0 and 10 kept, 13 with 3/13, 16 with 6/13, 23 and 31 whole parts divided by 4
    want = {0: 1.0, 10: 10.0**-1.25, 13: 10.0**-1.625 * (1 - 0.75 * 3 / 13), 16: 0.01 * (1 - 0.75 * 6 / 13),
            23: 10.0**-2.875 / 4, 31: 10.0**-3.875 / 4}
    for i, x in want.items():
        assert abs(f[i].item() - x) <= 1e-14 * x, i
    assert abs(f[16].item() - 0.0065384615384615385) < 1e-16 and abs(m - 1.1386294361119891) < 1e-15


def test_yarn_divides_every_pair_of_a_length_without_a_turn():
    f, _ = qsa.rope_frequencies(32, 10000.0, scaling="yarn", factor=4.0, original_len=4, device="cpu")
    plain, _ = qsa.rope_frequencies(32, 10000.0, device="cpu")
    assert torch.equal(f, plain / 4)
