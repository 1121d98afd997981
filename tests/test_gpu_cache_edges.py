"""The paged-cache calls at the edges of what their documentation allows, against the
FP64 oracle with its bounds (``oracle.qsa_paged``)."""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch
from test_gpu_cache import DEV, SCALE, _attend, _bf, _cache, _check, _gen, _routes

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


def test_inputs_broadcast_over_tokens_or_heads():
    g = _gen(73)
    f, m = qsa.rope_frequencies(64, device=DEV)
    pos = torch.arange(9, dtype=torch.int32, device=DEV) * 1000
    for x in (_bf(g, 1, 12, 256).to(DEV).expand(9, 12, 256), _bf(g, 9, 1, 256).to(DEV).expand(9, 12, 256),
              _bf(g, 1, 1, 256).to(DEV).expand(9, 12, 256)):
        for call in (qsa.rope, qsa.rope_backward):
            y, none = call(x, None, pos, f, mscale=m)
            z, _ = call(x.contiguous(), None, pos, f, mscale=m)
            assert none is None and torch.equal(y, z)
        with pytest.raises(qsa.QSAError) as e:     # rows that lie on one another cannot be written
            qsa.rope(x, None, pos, f, out_q=x)
        assert e.value.status == 1
    c = _cache([40], [9], 16, 1, 74, junk=0.0)
    a, b = ({n: x.to(DEV) for n, x in c.items()} for _ in range(2))
    k = _bf(g, 1, 1, 256).to(DEV).expand(9, 1, 256)
    qsa.cache_append(k, k, a["kp"], a["vp"], a["table"], a["kv_len"], a["cu_q"], inv_freq=f)
    qsa.cache_append(k.contiguous(), k.contiguous(), b["kp"], b["vp"], b["table"], b["kv_len"], b["cu_q"], inv_freq=f)
    assert torch.equal(a["kp"], b["kp"]) and torch.equal(a["vp"], b["vp"])


def test_a_batch_without_any_sequence():
    c = _cache([30, 0, 17], [0, 0, 0], 16, 1, 75, behind=5)
    r = _routes(c, 20, 1)
    for kw in (dict(), dict(window=4, sinks=1), dict(routes=r)):
        out, lse = _attend(c, **kw)
        assert (out == 7.0).all() and (lse == 7.0).all()
    d = {n: x.to(DEV) for n, x in c.items()}
    kp = d["kp"].clone()
    k = torch.ones(5, 1, 256, dtype=torch.bfloat16, device=DEV)
    q = qsa.cache_append(k, k, d["kp"], d["vp"], d["table"], d["kv_len"], d["cu_q"], q=d["q"].clone(),
                         inv_freq=qsa.rope_frequencies(64, device=DEV)[0], out_q=d["q"])
    assert torch.equal(d["kp"].view(torch.int16), kp.view(torch.int16)) and torch.equal(q.cpu(), c["q"])


GUARD = 4096


def _guarded(shape, dtype, raws, fill=None):
    n = int(np.prod(shape)) * torch.tensor([], dtype=dtype).element_size()
    raw = torch.full((GUARD + n + GUARD,), 0xA5, dtype=torch.uint8, device=DEV)
    x = raw[GUARD:GUARD + n].view(dtype).view(shape)
    if fill is not None:
        x.copy_(fill)
    raws.append(raw)
    return x


@pytest.mark.parametrize("lens,news,page,G,W", [([700, 0, 33], [130, 0, 33], 16, 2, 70), ([5000], [1], 64, 1, 2048),
                                                ([90, 2**31 - 1], [3, 5], 32, 1, 17), ([3], [3], 256, 3, 1),
                                                ([260] * 40, [1] * 40, 16, 1, 300)])
def test_nothing_is_written_outside_outputs_workspace_and_named_rows(lens, news, page, G, W):
    c = _cache([min(n, 300) if n > 10**6 else n for n in lens], news, page, G, 76, junk=0.5, lead=2, behind=3)
    r = _routes(c, W, 3)
    c["kv_len"] = torch.tensor(lens, dtype=torch.int32)
    T, H = c["q"].shape[:2]
    raws = []
    q, kp, vp = (_guarded(c[n].shape, torch.bfloat16, raws, c[n]) for n in ("q", "kp", "vp"))
    where = tuple(_guarded(c[n].shape, torch.int32, raws, c[n]) for n in ("table", "kv_len", "cu_q"))
    routes = _guarded(r.shape, torch.int32, raws, r)
    out, oq = (_guarded(q.shape, torch.bfloat16, raws) for _ in range(2))
    lse = _guarded((T, H), torch.float32, raws)
    ok = _guarded((T, G, 256), torch.bfloat16, raws)
    mp = c["table"].shape[1]
    ws = _guarded((qsa.paged_forward_workspace_size(T, H, G, W, page, mp),), torch.uint8, raws)
    qsa.paged_forward(q, kp, vp, routes, *where, SCALE, out=out, lse=lse, workspace=ws)
    ws = _guarded((qsa.paged_causal_workspace_size(T, H, G, page, mp, 40, 3),), torch.uint8, raws)
    qsa.paged_causal(q, kp, vp, *where, SCALE, window=40, sinks=3, out=out, lse=lse, workspace=ws)
    f, _ = qsa.rope_frequencies(256, device=DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    qsa.rope(q, kp.view(-1, G, 256)[:T] if kp.numel() >= T * G * 256 else None, pos, f, out_q=oq,
             out_k=ok if kp.numel() >= T * G * 256 else None)
    qsa.cache_append(ok, ok, kp, vp, *where, q=q, inv_freq=f, out_q=oq)
    torch.cuda.synchronize()
    for raw in raws:
        assert (raw[:GUARD] == 0xA5).all() and (raw[-GUARD:] == 0xA5).all()
