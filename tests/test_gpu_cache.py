"""GPU parity of the paged-cache operators against the FP64 oracle
(``oracle.qsa_paged``): rotary positions and their gradient, the append, and
attention of new tokens over the pages by routes and by position.

Tolerances: a rotation's cosine and sine are within 2^-21 (angle to 1e-7 and
two units in the last place of FP32) and its products and sum within 3 * 2^-24,
so before rounding y is within 2^-20 m (|x1| + |x2|), and the BF16 rounding adds
2^-8 |y|.  Attention: the oracle's elementwise bounds (see ``qsa_paged.attend``).
"""

import numpy as np
import pytest
import torch

from oracle import qsa_paged as P
from token_indexed_sparse_b200 import qsa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SCALE = 1.0 / 16.0


def _n(x):
    return x.detach().cpu().double().numpy()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _bf(g, *shape):
    return torch.randn(*shape, generator=g).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------

def _check_turned(y, x, positions, f, interleaved, m, backward):
    ref = P.rope(x, positions, f, interleaved=interleaved, mscale=m, backward=backward)
    mate = np.abs(P.rope(np.abs(x), np.zeros(len(positions)), f))  # |x|, then its pair's
    n = len(f)
    pair = np.abs(x).copy()
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    pair[..., a], pair[..., b] = mate[..., b], mate[..., a]
    tol = 2.0**-8 * np.abs(ref) + 2.0**-20 * m * (np.abs(x) + pair)
    assert (np.abs(y - ref) <= tol)[..., :2 * n].all()
    assert np.array_equal(y[..., 2 * n:], x[..., 2 * n:])


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,G,rot,m", [(1, 12, 1, 256, 1.0), (7, 24, 2, 64, 1.25), (33, 5, 3, 16, 0.5),
                                         (10, 12, 1, 96, 1.0), (3, 36, 3, 240, 1.1)])
def test_rope(T, H, G, rot, m, interleaved, backward):
    g = _gen(T + rot)
    q, k = _bf(g, T, H, 256), _bf(g, T, G, 256)
    pos = torch.randint(-5, 1 << 20, (T,), generator=g, dtype=torch.int32)
    pos[0] = 2**31 - 1 if T == 7 else 0
    f, _ = qsa.rope_frequencies(rot, 10000.0, device=DEV)
    fn = qsa.rope_backward if backward else qsa.rope
    qo, ko = fn(q.to(DEV), k.to(DEV), pos.to(DEV), f, interleaved=interleaved, mscale=m)
    for y, x in ((qo, q), (ko, k)):
        # position 2^31 - 1 leaves the 64-bit oracle's own angle 2^31 * 2^-53 off: far below the tolerance
        _check_turned(_n(y), _n(x), pos.tolist(), f.cpu().numpy(), interleaved, m, backward)


def test_rope_strided_in_place_and_without_k():
    g = _gen(5)
    T, f = 9, qsa.rope_frequencies(64, device=DEV)[0]
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    qkv = _bf(g, T, 12 + 2, 256).to(DEV)               # one projection: q heads, k, v
    q, k, v = qkv[:, :12], qkv[:, 12:13], qkv[:, 13:].clone()
    ref_q, ref_k = qsa.rope(q.contiguous(), k.contiguous(), pos, f)
    alone, none = qsa.rope(q, None, pos, f)
    assert none is None and torch.equal(alone, ref_q)
    heads_first = q.transpose(0, 1).contiguous().transpose(0, 1)   # [T, H, 256] with heads outermost
    out = torch.empty(12, T, 256, dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    assert torch.equal(qsa.rope(heads_first, None, pos, f, out_q=out)[0], ref_q)
    q2, k2 = qsa.rope(q, k, pos, f, out_q=q, out_k=k)
    assert q2.data_ptr() == q.data_ptr() and torch.equal(q2, ref_q) and torch.equal(k2, ref_k)
    assert torch.equal(qkv[:, 13:], v)


def test_rope_backward_undoes_a_pure_turn_and_matches_differences():
    g = _gen(6)
    T, f = 4, qsa.rope_frequencies(256, device=DEV)[0]
    pos = torch.tensor([0, 3, 500, 131071], dtype=torch.int32, device=DEV)
    # <g, d rope(x) e> by differences of the kernel itself: the map is linear, so a step of 256 in one
    # coordinate gives its column exactly but for the output's rounding
    go = _bf(g, T, 1, 256).to(DEV)
    dx = _n(qsa.rope_backward(go, None, pos, f)[0])
    for i in (0, 5, 127, 128, 200, 255):
        e = torch.zeros(T, 1, 256, dtype=torch.bfloat16, device=DEV)
        e[:, :, i] = 256.0
        d = (_n(qsa.rope(e, None, pos, f)[0]) - _n(qsa.rope(-e, None, pos, f)[0])) / 512.0
        want = (_n(go) * d).sum(-1)
        # two products of |g| <= max, each factor with one BF16 rounding, and dx's own
        tol = 2 * 2.0**-8 * np.abs(_n(go)).max() + 2.0**-8 * np.abs(dx[:, :, i]) + 1e-6
        assert (np.abs(want - dx[:, :, i]) <= tol).all(), i


# ---------------------------------------------------------------------------
# a paged cache
# ---------------------------------------------------------------------------

def _cache(lens, news, page, G, seed, *, spare=3, lead=0, behind=0, max_pages=None, junk=float("nan")):
    """A shuffled cache: dict of CPU tensors.  Pool rows that no sequence holds are `junk`."""
    g = _gen(seed)
    held = [-(-max(n, 0) // page) for n in lens]
    n_pages = sum(held) + spare
    ids = torch.randperm(n_pages, generator=g)
    table = torch.full((len(lens), max_pages or max(held + [1])), -1, dtype=torch.int32)
    kp, vp = (torch.full((n_pages, page, G, 256), junk, dtype=torch.bfloat16) for _ in range(2))
    at = 0
    for b, n in enumerate(lens):
        for i in range(held[b]):
            pg = int(ids[at])
            at += 1
            if i < table.shape[1]:
                table[b, i] = pg
            fill = min(page, n - i * page)
            kp[pg, :fill], vp[pg, :fill] = _bf(g, fill, G, 256), _bf(g, fill, G, 256)
    cu = torch.tensor([lead] + news).cumsum(0).to(torch.int32)
    T = int(cu[-1]) + behind
    return {"q": _bf(g, T, 12 * G, 256), "kp": kp, "vp": vp, "table": table,
            "kv_len": torch.tensor(lens, dtype=torch.int32), "cu_q": cu}


def _attend(c, *, routes=None, window=0, sinks=0, **kw):
    """The GPU call into outputs filled with 7: (out, lse)."""
    d = {n: x.to(DEV) for n, x in c.items()}
    out = torch.full(d["q"].shape, 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(d["q"].shape[:2], 7.0, device=DEV)
    where = (d["table"], d["kv_len"], d["cu_q"])
    if routes is not None:
        return qsa.paged_forward(d["q"], d["kp"], d["vp"], routes.to(DEV), *where, SCALE, out=out, lse=lse, **kw)
    return qsa.paged_causal(d["q"], d["kp"], d["vp"], *where, SCALE, window=window, sinks=sinks, out=out, lse=lse, **kw)


def _check(c, out, lse, *, routes=None, window=0, sinks=0):
    ref, ref_lse, tol, tol_lse = P.attend(
        _n(c["q"]), _n(c["kp"]), _n(c["vp"]), c["table"].numpy(), c["kv_len"].numpy(), c["cu_q"].numpy(), SCALE,
        routes=None if routes is None else routes.numpy(), window=window, sinks=sinks)
    out, lse = _n(out), _n(lse)
    none = np.isnan(ref_lse)  # rows of no sequence
    assert (out[none] == 7.0).all() and (lse[none] == 7.0).all()
    empty = np.isneginf(ref_lse)
    assert (lse[empty] == -np.inf).all() and (out[empty] == 0.0).all()
    rest = ~none & ~empty
    assert (np.abs(lse[rest] - ref_lse[rest]) <= tol_lse[rest]).all()
    err = np.abs(out[rest] - ref[rest])
    assert (err <= tol[rest]).all(), (err / tol[rest]).max()


BATCHES = {
    # lens, news, page, G, more
    "one_token": ([1], [1], 16, 1, {}),
    "one_long": ([5000], [1], 64, 1, {}),
    "decode": ([17, 1, 300, 64, 999, 128], [1] * 6, 16, 2, {}),
    "chunk": ([200], [75], 32, 1, {}),
    "prompt": ([150], [150], 128, 2, {}),
    "ragged": ([33, 0, 700, 130, 16], [5, 0, 41, 130, 1], 64, 1, {"lead": 3, "behind": 9}),
    "idle": ([40, 77, 12], [0, 2, 0], 16, 2, {"behind": 1}),
    "short_table": ([300, 90], [10, 60], 16, 1, {"max_pages": 4}),   # positions past the table have no page
    "short_len": ([3, 40], [8, 4], 16, 1, {}),                        # more new tokens than the cache holds
    "page256": ([513, 256], [20, 3], 256, 1, {}),
    "page1024": ([1500], [9], 1024, 3, {}),
    "negative": ([-3, 40, -2**31], [2, 7, 1], 16, 1, {}),             # a length below zero holds nothing
}


def _routes(c, W, seed):
    """Random IDs: duplicates, invalid ones, empty rows; some rows full of neighbours."""
    g = _gen(seed)
    T = c["q"].shape[0]
    top = int(max(c["kv_len"].max(), 1))
    r = torch.randint(-2, top + 6, (T, W), generator=g, dtype=torch.int32)
    r[::5] = -1
    for t in range(1, T, 3):
        r[t] = torch.arange(W, dtype=torch.int32) + int(torch.randint(0, top, (1,), generator=g))
    r[T // 2, 0] = 2**31 - 1
    return r


@pytest.mark.parametrize("W", [1, 37, 600])
@pytest.mark.parametrize("name", BATCHES)
def test_paged_forward(name, W):
    lens, news, page, G, more = BATCHES[name]
    c = _cache(lens, news, page, G, 11, **more)
    r = _routes(c, W, W)
    _check(c, *_attend(c, routes=r), routes=r)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (13, 4), (64, 130), (200, 1), (2**31 - 1, 2**31 - 1)])
@pytest.mark.parametrize("name", BATCHES)
def test_paged_causal(name, window, sinks):
    lens, news, page, G, more = BATCHES[name]
    c = _cache(lens, news, page, G, 12, **more)
    _check(c, *_attend(c, window=window, sinks=sinks), window=window, sinks=sinks)


@pytest.mark.parametrize("W", [2049, 4097, 9001, 16384])
def test_long_route_rows(W):
    c = _cache([20000, 333], [2, 3], 64, 1, 21)
    r = _routes(c, W, W)
    r[1] = torch.randint(0, 50, (W,), generator=_gen(W), dtype=torch.int32)  # hardly anything but repeats
    r[3] = 7
    _check(c, *_attend(c, routes=r), routes=r)


@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 5)])
def test_items_cut_into_ranges(window, sinks):
    # more key tiles than CTAs, items that end inside ranges and ranges inside items
    c = _cache([2400, 130, 900], [330, 1, 77], 32, 2, 22)
    _check(c, *_attend(c, window=window, sinks=sinks), window=window, sinks=sinks)


def test_many_sequences_most_of_them_short_or_empty():
    # more sequences and query tiles than the planning takes in one batch
    g = _gen(23)
    lens = torch.randint(0, 19, (1100,), generator=g).tolist()
    news = [min(n, int(x)) for n, x in zip(lens, torch.randint(0, 4, (1100,), generator=g))]
    news[40] = lens[40] = 60
    c = _cache(lens, news, 16, 1, 24, lead=1, behind=2)
    _check(c, *_attend(c))
    r = _routes(c, 12, 5)
    _check(c, *_attend(c, routes=r), routes=r)


def test_pools_past_32_bits():
    # rows whose element offsets pass 2^32: pages at the end of 9 GB pools
    page, G = 64, 2
    n_pages = (2**32 // (G * 256) + 4096) // page
    c = _cache([150], [60], page, G, 25)
    d = {n: x.to(DEV) for n, x in c.items()}
    kp, vp = (torch.empty(n_pages, page, G, 256, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    last = torch.arange(n_pages - d["kp"].shape[0], n_pages, device=DEV)
    kp[last], vp[last] = d["kp"], d["vp"]
    table = torch.where(d["table"] >= 0, d["table"] + int(last[0]), -1).to(torch.int32)
    where = (table, d["kv_len"], d["cu_q"])
    out, lse = qsa.paged_causal(d["q"], kp, vp, *where, SCALE)
    _check(c, out, lse)
    r = _routes(c, 40, 6)
    out, lse = qsa.paged_forward(d["q"], kp, vp, r.to(DEV), *where, SCALE)
    _check(c, out, lse, routes=r)
    k, v = _bf(_gen(26), 60, G, 256), _bf(_gen(27), 60, G, 256)
    qsa.cache_append(k.to(DEV), v.to(DEV), kp, vp, *where)
    for t in (0, 37, 59):
        p = 90 + t
        row = (int(table[0, p // page]), p % page)
        assert torch.equal(kp[row].cpu(), k[t]) and torch.equal(vp[row].cpu(), v[t])


@pytest.mark.parametrize("news", [1, 40])
def test_bad_page_ids_hold_nothing(news):
    c = _cache([400], [news], 32, 1, 13)
    c["table"][0, 2], c["table"][0, 7], c["table"][0, 12] = -1, c["kp"].shape[0], 2**31 - 1
    r = _routes(c, 200, 1)
    _check(c, *_attend(c, routes=r), routes=r)
    for window, sinks in ((0, 0), (50, 70)):
        _check(c, *_attend(c, window=window, sinks=sinks), window=window, sinks=sinks)
    c["table"][:] = -1                                  # nothing mapped at all: empty rows
    out, lse = _attend(c)
    assert (lse == -np.inf).all() and (out == 0).all()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("news", [1, 60])
def test_unseen_non_finite_rows_reach_nothing(news, value):
    # rows past kv_len, on unmapped pages, behind the token, outside the window
    c = _cache([300], [news], 32, 1, 14, junk=value)
    j = 300 - news // 2 - 1                              # only the rows from it on see it
    pg, at = int(c["table"][0, j // 32]), j % 32
    c["kp"][pg, at], c["vp"][pg, at] = 1.0, value
    d = 100                                              # seen by no row with the window
    c["kp"][int(c["table"][0, d // 32]), d % 32] = value
    out, lse = _attend(c, window=90, sinks=2)
    p = torch.arange(300 - news, 300)
    sees = ((p >= j) & (p - j < 90)).to(DEV)
    assert torch.isfinite(out[~sees]).all() and torch.isfinite(lse).all()
    assert not torch.isfinite(out[sees]).any()
    c["vp"][pg, at] = 0.0
    clean, _ = _attend(c, window=90, sinks=2)
    assert torch.equal(clean[~sees], out[~sees])         # bit for bit what it is without the value
    r = torch.full((news, 8), -1, dtype=torch.int32)
    r[:, 0], r[:, 1] = 5, 299
    assert all(torch.isfinite(x).all() for x in _attend(c, routes=r))


def test_a_non_finite_value_in_a_cut_item():
    # V of the diagonal's keys, where the item's last tile lies in a range of its own
    c = _cache([3000], [30], 64, 1, 28)
    j = 2985                                             # seen by the last 15 tokens
    c["vp"][int(c["table"][0, j // 64]), j % 64, 0, 5] = float("inf")
    out, lse = _attend(c)
    assert torch.isfinite(lse).all() and torch.isfinite(out[:15]).all()
    assert (out[15:, :, 5] == float("inf")).all()
    out[15:, :, 5] = 0
    assert torch.isfinite(out).all()


def test_large_scores_and_first_keys_that_dominate():
    # scores of several hundred, the largest at the front, in the middle and at the end
    for seed, at in ((1, 0), (2, 250), (3, 511)):
        c = _cache([512], [40], 32, 1, 20 + seed)
        c["kp"][int(c["table"][0, at // 32]), at % 32] *= 24
        c["q"] *= 8
        _check(c, *_attend(c))
        r = torch.arange(512, dtype=torch.int32).expand(40, 512).contiguous()
        _check(c, *_attend(c, routes=r), routes=r)


def test_repeats_bit_for_bit_and_shared_pages():
    c = _cache([900, 900, 650], [1, 1, 30], 16, 2, 15)
    c["table"][1] = c["table"][0]                        # two sequences read the same pages
    a, b = _attend(c), _attend(c)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    _check(c, *a)
    r = _routes(c, 300, 3)
    a, b = _attend(c, routes=r), _attend(c, routes=r)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    _check(c, *a, routes=r)


# ---------------------------------------------------------------------------
# append, and the calls together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("name", BATCHES)
@pytest.mark.parametrize("rot,interleaved", [(0, False), (64, True), (256, False)])
def test_cache_append(name, rot, interleaved):
    lens, news, page, G, more = BATCHES[name]
    c = _cache(lens, news, page, G, 16, junk=3.0, **more)
    T = c["q"].shape[0]
    g = _gen(17)
    k, v = _bf(g, T, G, 256), _bf(g, T, G, 256)
    d = {n: x.to(DEV) for n, x in c.items()}
    where = (d["table"], d["kv_len"], d["cu_q"])
    kw = {}
    if rot:
        f, m = qsa.rope_frequencies(rot, 1e6, scaling="yarn", factor=4.0, device=DEV)
        out_q = torch.full(d["q"].shape, 7.0, dtype=torch.bfloat16, device=DEV)
        kw = dict(q=d["q"], inv_freq=f, interleaved=interleaved, mscale=m, out_q=out_q)
    got_q = qsa.cache_append(k.to(DEV), v.to(DEV), d["kp"], d["vp"], *where, **kw)
    at = [P.place(t, c["kv_len"].tolist(), c["cu_q"].tolist()) for t in range(T)]
    # (a length of -2^31 has positions that rope's int32 cannot name: their q rows are not compared)
    named = torch.tensor([x is not None and x[1] >= -2**31 for x in at], device=DEV)
    pos = torch.tensor([0 if x is None else max(x[1], -2**31) for x in at], dtype=torch.int32, device=DEV)
    k_ref = k
    if rot:  # the same rotation as rope's, bit for bit
        q_ref, k_ref = qsa.rope(d["q"], k.to(DEV), pos, f, interleaved=interleaved, mscale=m)
        k_ref = k_ref.cpu()
        of_none = torch.tensor([x is None for x in at], device=DEV)
        assert (got_q[of_none] == 7.0).all() and torch.equal(got_q[named], q_ref[named])
    else:
        assert got_q is None
    kp, vp = P.append(_n(k_ref), _n(v), _n(c["kp"]), _n(c["vp"]), c["table"].numpy(), c["kv_len"].numpy(),
                      c["cu_q"].numpy())
    assert np.array_equal(_n(d["kp"]), kp) and np.array_equal(_n(d["vp"]), vp)


def test_append_from_a_fused_projection_in_place():
    c = _cache([70, 33], [20, 33], 16, 1, 18, junk=0.0)
    qkv = _bf(_gen(19), 53, 14, 256).to(DEV)
    q, k, v = qkv[:, :12], qkv[:, 12:13], qkv[:, 13:]
    f, _ = qsa.rope_frequencies(128, device=DEV)
    a = {n: x.to(DEV) for n, x in c.items()}
    b = {n: x.clone() for n, x in a.items()}
    want = qsa.cache_append(k.contiguous(), v.contiguous(), a["kp"], a["vp"], a["table"], a["kv_len"], a["cu_q"],
                            q=q.contiguous(), inv_freq=f)
    got = qsa.cache_append(k, v, b["kp"], b["vp"], b["table"], b["kv_len"], b["cu_q"], q=q, inv_freq=f, out_q=q)
    assert got.data_ptr() == qkv.data_ptr() and torch.equal(got, want)
    assert torch.equal(a["kp"], b["kp"]) and torch.equal(a["vp"], b["vp"])


def _step(s):
    """One serving step: append with the rotation, then both attentions."""
    q = qsa.cache_append(s["k"], s["v"], s["kp"], s["vp"], s["table"], s["kv_len"], s["cu_q"], q=s["q"],
                         inv_freq=s["f"])
    cache = (s["kp"], s["vp"])
    where = (s["table"], s["kv_len"], s["cu_q"])
    return (q, *qsa.paged_forward(q, *cache, s["routes"], *where, SCALE, workspace=s["ws"]),
            *qsa.paged_causal(q, *cache, *where, SCALE, window=100, sinks=4, workspace=s["ws"]))


def _serving(lens, news, seed, W=64):
    c = _cache(lens, news, 16, 1, seed, junk=0.0)
    T = c["q"].shape[0]
    g = _gen(seed)
    s = {n: x.to(DEV) for n, x in c.items()}
    s |= {"k": _bf(g, T, 1, 256).to(DEV), "v": _bf(g, T, 1, 256).to(DEV), "routes": _routes(c, W, seed).to(DEV),
          "f": qsa.rope_frequencies(64, device=DEV)[0]}
    n = max(qsa.paged_forward_workspace_size(T, 12, 1, W, 16, c["table"].shape[1]),
            qsa.paged_causal_workspace_size(T, 12, 1, 16, c["table"].shape[1], 100, 4))
    s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    return c, s


def test_a_prompt_in_chunks_then_tokens_is_the_whole_prompt():
    # a sequence of 83 tokens fed as 50 + 30 + 1 + 1 + 1 attends like one call over all of them
    L, parts = 83, [50, 30, 1, 1, 1]
    g = _gen(30)
    q, k, v = _bf(g, L, 12, 256), _bf(g, L, 1, 256), _bf(g, L, 1, 256)
    f, m = qsa.rope_frequencies(256, device=DEV)
    table = torch.tensor([[4, 1, 5, 0, 2, 3]], dtype=torch.int32, device=DEV)

    def feed(parts):
        kp = torch.zeros(6, 16, 1, 256, dtype=torch.bfloat16, device=DEV)
        vp = torch.zeros_like(kp)
        outs, at = [], 0
        for n in parts:
            kv_len = torch.tensor([at + n], dtype=torch.int32, device=DEV)
            cu_q = torch.tensor([0, n], dtype=torch.int32, device=DEV)
            part = [x[at:at + n].to(DEV) for x in (q, k, v)]
            qr = qsa.cache_append(part[1], part[2], kp, vp, table, kv_len, cu_q, q=part[0], inv_freq=f, mscale=m)
            outs.append((qr, *qsa.paged_causal(qr, kp, vp, table, kv_len, cu_q, SCALE)))
            at += n
        return [torch.cat(x) for x in zip(*outs)], kp, vp

    (q1, o1, l1), kp1, vp1 = feed(parts)
    (q2, o2, l2), kp2, vp2 = feed([L])
    assert torch.equal(q1, q2) and torch.equal(kp1, kp2) and torch.equal(vp1, vp2)
    pos = np.arange(L)
    qr = qsa.rope(q.to(DEV), k.to(DEV), torch.arange(L, dtype=torch.int32, device=DEV), f)
    c = {"q": qr[0].cpu(), "kp": kp1.cpu(), "vp": vp1.cpu(), "table": table.cpu(),
         "kv_len": torch.tensor([L], dtype=torch.int32), "cu_q": torch.tensor([0, L], dtype=torch.int32)}
    assert len(pos) == L
    _check(c, o1, l1)
    _check(c, o2, l2)
    # and by routes that name every token up to its own: the contiguous forward's answer
    r = torch.arange(L, dtype=torch.int32).expand(L, L).clone()
    r[r > torch.arange(L)[:, None]] = -1
    out, lse = qsa.paged_forward(qr[0], kp1, vp1, r.to(DEV), table, c["kv_len"].to(DEV), c["cu_q"].to(DEV), SCALE)
    _check(c, out, lse, routes=r)
    ref, ref_lse = qsa.forward(qr[0], qr[1], v.to(DEV), r.to(DEV), SCALE)
    assert torch.allclose(out.float(), ref.float(), atol=2.0**-6) and torch.allclose(lse, ref_lse, atol=1e-4)


def test_captured_steps_that_share_a_workspace_replay():
    c1, s1 = _serving([200, 90, 31], [1, 1, 1], 40)
    c2, s2 = _serving([150], [60], 41)
    if s2["ws"].numel() > s1["ws"].numel():
        s1["ws"] = s2["ws"]
    else:
        s2["ws"] = s1["ws"]
    want = [[x.clone() for x in _step(s)] for s in (s1, s2)]
    side = torch.cuda.Stream()
    graphs, got = [], []
    with torch.cuda.stream(side):
        for s in (s1, s2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                got.append(_step(s))
            graphs.append(g)
        for i in (0, 1, 1, 0):
            s1["ws"].fill_(0xAB)
            graphs[i].replay()
            side.synchronize()
            for a, b in zip(got[i], want[i]):
                assert torch.equal(a, b)
    # new values in the captured inputs (lengths among them) are followed
    s1["kv_len"].copy_(torch.tensor([190, 17, 3], dtype=torch.int32))
    s1["q"].copy_(s1["q"].flip(0))
    graphs[0].replay()
    torch.cuda.synchronize()
    for a, b in zip(got[0], _step(s1)):
        assert torch.equal(a, b)
    assert c1 is not c2


def test_two_streams_at_once():
    _, s1 = _serving([700, 90], [20, 1], 42)
    _, s2 = _serving([650], [1], 43)
    want = [_step(s) for s in (s1, s2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for s, st in zip((s1, s2), streams):
            with torch.cuda.stream(st):
                got.append(_step(s))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_refusals_on_the_device():
    c = _cache([20], [2], 16, 1, 50)
    d = {n: x.to(DEV) for n, x in c.items()}
    where = (d["table"], d["kv_len"], d["cu_q"])
    with pytest.raises(ValueError, match="on cuda"):
        qsa.paged_causal(d["q"], d["kp"], d["vp"], c["table"], *where[1:], SCALE)
    with pytest.raises(qsa.QSAError) as e:
        qsa.paged_causal(d["q"][:, :11].contiguous(), d["kp"], d["vp"], *where, SCALE)
    assert e.value.status == 2
    with pytest.raises(qsa.QSAError) as e:
        qsa.paged_causal(d["q"], d["kp"], d["vp"], *where, SCALE, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.status in (3, 4)
    with pytest.raises(qsa.QSAError) as e:
        qsa.paged_causal(d["q"], d["kp"], d["vp"], *where, SCALE, window=-1)
    assert e.value.status == 1
    odd = torch.zeros(2, 24, 1, 256, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(qsa.QSAError) as e:
        qsa.paged_causal(d["q"], odd, odd, *where, SCALE)
    assert e.value.status == 2


class _Declines:
    """A compiled binding that takes nothing."""

    def __getattr__(self, name):
        return lambda *args: NotImplemented


def test_the_short_and_the_long_way_agree(monkeypatch):
    short = qsa._short_way()
    taken = []

    class Counts:
        def __getattr__(self, name):
            def call(*args):
                r = getattr(short, name)(*args)
                taken.append(r is not NotImplemented)
                return r
            return call

    def everything():
        c, s = _serving([200, 90, 31], [1, 40, 1], 60)
        pos = torch.arange(s["q"].shape[0], dtype=torch.int32, device=DEV)
        got = [*_step(s), s["kp"], s["vp"], *qsa.rope(s["q"], s["k"], pos, s["f"], interleaved=True, mscale=1.5),
               *qsa.rope_backward(s["q"], None, pos, s["f"])[:1]]
        where = (s["table"], s["kv_len"], s["cu_q"])
        assert qsa.cache_append(s["k"], s["v"], s["kp"], s["vp"], *where) is None
        out, lse = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:2], device=DEV)
        a, b = qsa.paged_causal(s["q"], s["kp"], s["vp"], *where, out=out, lse=lse)
        assert a is out and b is lse
        return got + [out, lse, s["kp"], s["vp"]]

    monkeypatch.setattr(qsa, "_short", Counts())
    a = everything()
    assert len(taken) == 7 and all(taken)
    monkeypatch.setattr(qsa, "_short", _Declines())
    b = everything()
    assert len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))
    # what the short way leaves: routes in another layout, q in pieces
    monkeypatch.setattr(qsa, "_short", Counts())
    _, s = _serving([200, 90, 31], [1, 40, 1], 60)
    where = (s["table"], s["kv_len"], s["cu_q"])
    wide = torch.zeros(s["q"].shape[0], 24, 256, dtype=torch.bfloat16, device=DEV)
    wide[:, 6:18] = s["q"]
    r = s["routes"].t().contiguous().t()
    x = qsa.paged_forward(wide[:, 6:18], s["kp"], s["vp"], r, *where)
    y = qsa.paged_forward(s["q"], s["kp"], s["vp"], s["routes"], *where)
    assert taken[-2:] == [False, True] and all(torch.equal(u, v) for u, v in zip(x, y))


def test_refusals_are_the_same_both_ways(monkeypatch):
    c = _cache([20], [2], 16, 1, 50)
    d = {n: x.to(DEV) for n, x in c.items()}
    where = (d["table"], d["kv_len"], d["cu_q"])
    bad = [
        lambda: qsa.paged_causal(d["q"], d["kp"], d["vp"], *where, -1.0),
        lambda: qsa.paged_causal(d["q"], d["kp"], d["vp"], *where, sinks=-2),
        lambda: qsa.paged_causal(d["q"], d["kp"], d["vp"], *where, workspace=d["q"]),
        lambda: qsa.paged_causal(d["q"], d["kp"], d["vp"], *where, out=d["q"][:1]),
        lambda: qsa.paged_forward(d["q"], d["kp"], d["vp"], d["table"].long(), *where),
        lambda: qsa.paged_forward(d["q"], d["kp"].float(), d["vp"], d["table"], *where),
        lambda: qsa.rope(d["q"], None, d["kv_len"], torch.ones(8, dtype=torch.float64, device=DEV)),
        lambda: qsa.rope(d["q"], None, torch.zeros(2, dtype=torch.int32, device=DEV),
                         torch.ones(9, dtype=torch.float64, device=DEV)),
        lambda: qsa.cache_append(d["q"][:, :1], d["q"][:, :1], d["kp"], d["kp"], *where),
        lambda: qsa.cache_append(d["q"][:, :2], d["q"][:, :2], d["kp"], d["vp"], *where),
    ]

    def said(call):
        with pytest.raises(Exception) as e:
            call()
        return type(e.value), str(e.value)

    both = [said(x) for x in bad]
    monkeypatch.setattr(qsa, "_short", _Declines())
    assert [said(x) for x in bad] == both
