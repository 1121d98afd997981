"""Host-side checks of the paged-cache calls: they return before any CUDA work,
so they run without a GPU."""

import ctypes

import pytest
import torch

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from token_indexed_sparse_b200 import build, qsa
    build.build()
    return qsa.library()


def test_rope_refusals(lib):
    def call(q=4096, q_ts=24 * 256, q_hs=256, k=1 << 30, k_ts=256, k_hs=256, qo=1 << 31, qo_ts=24 * 256, qo_hs=256,
             ko=1 << 32, ko_ts=256, ko_hs=256, pos=256, inv=256, T=8, H=24, G=1, rot=64, mscale=1.0):
        return lib.qsa_rope(P(q), q_ts, q_hs, P(k), k_ts, k_hs, P(qo), qo_ts, qo_hs, P(ko), ko_ts, ko_hs, P(pos),
                            P(inv), T, H, G, rot, 0, mscale, 0, None)
    assert call(q=0) == 1 and call(k=0) == 1 and call(qo=0) == 1 and call(ko=0) == 1
    assert call(pos=0) == 1 and call(inv=0) == 1
    assert call(T=0) == 1 and call(H=0) == 1 and call(G=-1) == 1 and call(T=2**30 + 1) == 1
    assert call(T=2**30) == 1                                  # T * heads over 2^31
    assert call(rot=0) == 1 and call(rot=24) == 2 and call(rot=272) == 2
    assert call(mscale=0.0) == 1 and call(mscale=float("nan")) == 1 and call(mscale=float("inf")) == 1
    assert call(q=4104) == 3 and call(q_ts=24 * 256 + 4) == 3 and call(k_hs=252) == 3 and call(inv=260) == 3
    assert call(pos=258) == 3 and call(ko=(1 << 32) + 8) == 3
    assert call(q_ts=-256) == 1 and call(q_ts=1 << 60) == 1
    # outputs: rows that overlap each other, or the input other than in place
    assert call(qo_ts=23 * 256) == 1 and call(qo_hs=128) == 1 and call(qo_ts=0) == 1
    assert call(qo=4096 + 512) == 1 and call(qo=4096, qo_ts=25 * 256) == 1
    assert call(q=1 << 31, q_ts=25 * 256) == 1


def _cache_args(table=256, kv_len=256, cu_q=256, T=8, B=2, n_pages=4, page=16, max_pages=3, H=12, G=1):
    return P(table), P(kv_len), P(cu_q), T, B, n_pages, page, max_pages, H, G


CACHE_REFUSALS = [
    (dict(table=0), 1), (dict(kv_len=0), 1), (dict(cu_q=0), 1), (dict(T=0), 1), (dict(B=0), 1), (dict(n_pages=0), 1),
    (dict(max_pages=0), 1), (dict(page=0), 1), (dict(page=8), 2), (dict(page=24), 2), (dict(n_pages=2**27), 1),
    (dict(max_pages=2**27), 1), (dict(H=13), 2), (dict(H=24), 2), (dict(G=0), 1), (dict(T=2**28), 1),
    (dict(table=258), 3), (dict(kv_len=258), 3), (dict(cu_q=258), 3),
]


@pytest.mark.parametrize("bad,status", CACHE_REFUSALS)
def test_cache_refusals(lib, bad, status):
    c = _cache_args(**bad)
    rows = [P(4096), 256, 256, P(1 << 30), 256, 256, None, 0, 0, None, 0, 0]
    assert lib.qsa_cache_append(*rows, None, 0, 0, 1.0, P(1 << 31), P(1 << 32), *c, None) == status
    assert lib.qsa_paged_forward(P(256), P(256), P(256), P(256), *c, 4, 0.0625, P(256), P(256), P(256), 1 << 40,
                                 None) == status
    assert lib.qsa_paged_causal(P(256), P(256), P(256), *c, 0, 0, 0.0625, P(256), P(256), P(256), 1 << 40,
                                None) == status


def test_append_refusals(lib):
    def call(k=4096, k_ts=256, v=1 << 30, q=None, qo=None, inv=None, rot=64, mscale=1.0, kp=1 << 31, vp=1 << 32):
        rows = [P(k), k_ts, 256, P(v), 256, 256, P(q), 12 * 256, 256, P(qo), 12 * 256, 256]
        return lib.qsa_cache_append(*rows, P(inv), rot, 0, mscale, P(kp), P(vp), *_cache_args(), None)
    assert call(k=0) == 1 and call(v=0) == 1 and call(kp=0) == 1 and call(vp=0) == 1 and call(kp=1 << 32) == 1
    assert call(k=4104) == 3 and call(k_ts=260) == 3 and call(kp=(1 << 31) + 8) == 3
    assert call(q=4096, qo=1 << 33) == 1                       # q without frequencies
    assert call(q=4096, inv=256) == 1                          # no output for q
    assert call(q=4096, qo=4096 + 512, inv=256) == 1           # overlap
    assert call(inv=256, rot=20) == 2 and call(inv=256, mscale=-1.0) == 1


def test_paged_attention_refusals(lib):
    def fwd(q=256, kp=256, vp=256, routes=256, n_sel=4, scale=0.0625, out=256, lse=256, ws=256, n=1 << 40):
        return lib.qsa_paged_forward(P(q), P(kp), P(vp), P(routes), *_cache_args(), n_sel, scale, P(out), P(lse),
                                     P(ws), n, None)
    for name in ("q", "kp", "vp", "routes", "out", "lse", "ws"):
        assert fwd(**{name: 0}) == 1
    assert fwd(n_sel=0) == 1 and fwd(n_sel=16385) == 1 and fwd(scale=0.0) == 1 and fwd(scale=float("nan")) == 1
    assert fwd(q=264) == 3 and fwd(kp=264) == 3 and fwd(out=264) == 3 and fwd(routes=258) == 3 and fwd(lse=258) == 3
    need = lib.qsa_paged_forward_workspace_size(8, 12, 1, 4, 16, 3)
    assert need > 0 and fwd(ws=264) == 3 and fwd(n=need - 1) == 4
    assert lib.qsa_paged_forward_workspace_size(8, 12, 1, 4, 24, 3) == 0

    def causal(q=256, window=0, sinks=0, scale=0.0625, out=256, lse=256, ws=256, n=1 << 40):
        return lib.qsa_paged_causal(P(q), P(256), P(256), *_cache_args(), window, sinks, scale, P(out), P(lse), P(ws),
                                    n, None)
    assert causal(q=0) == 1 and causal(out=0) == 1 and causal(lse=0) == 1 and causal(ws=0) == 1
    assert causal(window=-1) == 1 and causal(sinks=-1) == 1 and causal(scale=-1.0) == 1
    assert causal(scale=float("inf")) == 1 and causal(q=264) == 3 and causal(lse=258) == 3
    need = lib.qsa_paged_causal_workspace_size(8, 12, 1, 16, 3, 0, 0)
    assert need > 0 and causal(n=need - 1) == 4
    assert lib.qsa_paged_causal_workspace_size(8, 12, 1, 16, 3, -1, 0) == 0


def test_binding_refusals(lib):
    from token_indexed_sparse_b200 import qsa
    bf, i32 = torch.bfloat16, torch.int32
    q, k = torch.zeros(4, 12, 256, dtype=bf), torch.zeros(4, 1, 256, dtype=bf)
    pos, f = torch.zeros(4, dtype=i32), torch.ones(8, dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        qsa.rope(q, k, pos, f)
    with pytest.raises(TypeError):
        qsa.rope(q.float(), k, pos, f)
    with pytest.raises(TypeError):
        qsa.rope(q, k, pos.long(), f)
    with pytest.raises(TypeError):
        qsa.rope(q, k, pos, f.float())
    with pytest.raises(ValueError, match="positions"):
        qsa.rope(q, k, pos[:3], f)
    with pytest.raises(ValueError, match="256"):
        qsa.rope(q[..., :128], k, pos, f)
    with pytest.raises(ValueError, match="contiguous dims"):
        qsa.rope(torch.zeros(4, 256, 12, dtype=bf).transpose(1, 2), k, pos, f)
    with pytest.raises(ValueError, match="shape"):
        qsa.rope(q, k, pos, f, out_q=q[:3])
    pages = torch.zeros(3, 16, 1, 256, dtype=bf)
    table, kv_len, cu_q = torch.zeros(2, 3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(3, dtype=i32)
    with pytest.raises(ValueError, match="contiguous"):
        qsa.cache_append(k, k, pages[::2], pages[::2], table, kv_len, cu_q)
    with pytest.raises(ValueError, match="kv_len"):
        qsa.cache_append(k, k, pages, pages, table, kv_len, cu_q[:2])
    with pytest.raises(TypeError):
        qsa.cache_append(k, k, pages, pages, table.long(), kv_len, cu_q)
    with pytest.raises(ValueError, match="inv_freq"):
        qsa.cache_append(k, k, pages, pages, table, kv_len, cu_q, q=q)
    with pytest.raises(ValueError, match="KV heads"):
        qsa.cache_append(torch.zeros(4, 2, 256, dtype=bf), torch.zeros(4, 2, 256, dtype=bf), pages, pages, table,
                         kv_len, cu_q)


def test_rope_frequencies():
    from token_indexed_sparse_b200 import qsa
    f, m = qsa.rope_frequencies(64, 10000.0, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (32,) and m == 1.0
    assert torch.allclose(f, 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32))
    lin, m = qsa.rope_frequencies(64, 10000.0, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(lin, f / 4) and m == 1.0
    y, m = qsa.rope_frequencies(64, 10000.0, scaling="yarn", factor=4.0, original_len=4096, device="cpu")
    turns = 4096 * f / (2 * torch.pi)
    # fast pairs as they were, slow ones divided, no pair outside, never rising
    assert torch.equal(y[turns > 64], f[turns > 64]) and torch.allclose(y[turns < 0.5], f[turns < 0.5] / 4)
    assert ((y <= f) & (y >= f / 4)).all() and (y.diff() < 0).all()
    assert abs(m - 1.1386294361119891) < 1e-12
    for bad in (dict(rotary_dim=24), dict(rotary_dim=272), dict(rotary_dim=64, base=1.0),
                dict(rotary_dim=64, factor=0.5), dict(rotary_dim=64, scaling="other")):
        with pytest.raises(ValueError):
            qsa.rope_frequencies(**{"device": "cpu", **bad})


def test_the_short_way_leaves_what_it_does_not_take(lib):
    # the compiled binding does nothing with what the Python one would convert or refuse
    from token_indexed_sparse_b200 import qsa
    short = qsa._short_way()
    q, pos = torch.zeros(4, 12, 256, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    f = torch.ones(8, dtype=torch.float64)
    for args in ((q, None, pos, f, False, 1.0, None, None, False), (q, q, pos), (1, 2, 3, 4, 5, 6, 7, 8, 9),
                 (q, None, pos, f, False, "one", None, None, False)):
        assert short.rope(*args) is NotImplemented
    assert short.cache_append(*[q] * 12) is NotImplemented and short.paged_forward(*[q] * 11) is NotImplemented
    assert short.paged_causal(*[q] * 12) is NotImplemented and short.paged_causal() is NotImplemented
    with pytest.raises(TypeError):
        short.bind(1, 2)
