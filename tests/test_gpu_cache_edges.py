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
