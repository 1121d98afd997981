"""The paged-cache calls at the edges of what their documentation allows, against the
FP64 oracle with its bounds (``oracle.qsa_paged``)."""

import pytest
import torch
from test_gpu_cache import DEV, SCALE, _attend, _cache, _check, _routes

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
