"""The paged-cache calls at the edges of what their documentation allows, against the
FP64 oracle with its bounds (``oracle.qsa_paged``)."""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch
from test_gpu_cache import DEV, SCALE, _attend, _cache, _check, _routes

from token_indexed_sparse_b200 import qsa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("end", [2**30, 2**30 + 5, 2**31 - 1])
@pytest.mark.parametrize("first", [-3, 0, 90])
def test_a_sequence_whose_rows_go_on_behind_the_batch(end, first):
    # cu_q names rows past T: row t sits at kv_len - (cu_q[1] - t), whatever the offset
    T = 6
    c = _cache([first + T], [T], 16, 1, 70, junk=0.5)
    c["cu_q"] = torch.tensor([0, end], dtype=torch.int32)
    r = _routes(c, 30, 4)
    c["kv_len"] = torch.tensor([min(first + end, 2**31 - 1)], dtype=torch.int32)
    for window, sinks in ((0, 0), (7, 2)):
        _check(c, *_attend(c, window=window, sinks=sinks), window=window, sinks=sinks)
    _check(c, *_attend(c, routes=r), routes=r)


@pytest.mark.parametrize("news", [1, 3, 40])
@pytest.mark.parametrize("W", [5, 400, 2048])
def test_rows_whose_scores_are_all_minus_infinity(news, W):
    # zeros and -inf in every form: one part or several, joined or not, by routes and by position
    c = _cache([2100], [news], 32, 1, 71, junk=0.0)
    c["q"].fill_(1.0)
    c["kp"].fill_(float("-inf"))
    r = torch.arange(W, dtype=torch.int32).expand(news, W).contiguous()
    for kw in (dict(routes=r), dict(), dict(window=W, sinks=3)):
        out, lse = _attend(c, **kw)
        assert (lse == -float("inf")).all() and (out == 0).all(), kw


PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803")


@pytest.mark.parametrize("backward", [False, True])
def test_angles_of_far_positions_and_fast_pairs(backward):
    # angles taken modulo a turn in exact arithmetic; cosine and sine come out by themselves (x = (1, 0), (0, 1))
    f = [1.0, 0.9997, 1.0 / 3.0, 100.3, -12345.678, 1000000.1, 3.0e9 / 7.0, 2.0**40 / 3.0]
    pos = [2**31 - 1, -2**31, 2**30 + 12345, 987654321, 65537, 1, -1, 0]
    x = torch.zeros(len(pos), 2, 256, dtype=torch.bfloat16)
    x[:, 0, :8] = 1.0
    x[:, 1, 8:16] = 1.0
    call = qsa.rope_backward if backward else qsa.rope
    y, _ = call(x.to(DEV), None, torch.tensor(pos, dtype=torch.int32, device=DEV),
                torch.tensor(f, dtype=torch.float64, device=DEV))
    y = y.cpu().double().numpy()
    a = np.array([[float((p * Fraction(v) / (2 * PI)) % 1 * 2 * PI) for v in f] for p in pos])
    c, s = np.cos(a), np.sin(-a if backward else a)
    ref = np.stack([np.concatenate([c, s], 1), np.concatenate([-s, c], 1)], 1)
    # the angle within 2^-25 of a turn (the exact one as a double: 2^-52), two units in the last place of the
    # cosine and sine, one BF16 rounding
    tol = 2 * math.pi * 2.0**-25 + 2.0**-22 + 2.0**-8 * np.abs(ref)
    assert (np.abs(y[..., :16] - ref) <= tol).all()


def test_the_status_word_says_that_no_wait_gave_up():
    c = _cache([900, 20], [30, 1], 32, 1, 72)
    r = _routes(c, 300, 2)
    n = max(qsa.paged_causal_workspace_size(31, 12, 1, 32, c["table"].shape[1]),
            qsa.paged_forward_workspace_size(31, 12, 1, 300, 32, c["table"].shape[1]))
    for kw in (dict(), dict(window=50, sinks=2), dict(routes=r)):
        ws = torch.full((n,), 0xAB, dtype=torch.uint8, device=DEV)
        _check(c, *_attend(c, workspace=ws, **kw), **kw)
        assert qsa.status_word(ws).item() == 0
