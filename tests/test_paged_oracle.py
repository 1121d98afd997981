"""The FP64 oracle of the paged-cache operators, pinned on the CPU: rotations by
complex arithmetic, the gradient by differences, the cache's index arithmetic
by hand, attention by the contiguous oracle and by torch's causal attention."""

import numpy as np
import pytest
import torch

import oracle
from oracle import qsa_paged as P


def _rand(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_a_complex_turn(interleaved):
    x, pos = _rand(1, 5, 3, 32), [0, 1, 7, 100, -3]
    f = 10000.0 ** (-np.arange(8) / 8.0)
    y = P.rope(x, pos, f, interleaved=interleaved, mscale=1.25)
    a, b = (slice(0, 16, 2), slice(1, 16, 2)) if interleaved else (slice(0, 8), slice(8, 16))
    z = (x[..., a] + 1j * x[..., b]) * 1.25 * np.exp(1j * np.outer(pos, f))[:, None]
    assert np.allclose(y[..., a], z.real, atol=1e-12) and np.allclose(y[..., b], z.imag, atol=1e-12)
    assert np.array_equal(y[..., 16:], x[..., 16:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient_by_differences(interleaved):
    x, g, pos, f = _rand(2, 2, 1, 16), _rand(3, 2, 1, 16), [3, 11], np.array([1.0, 0.3, 0.1, 0.01])
    kw = dict(interleaved=interleaved, mscale=0.7)
    dx = P.rope(g, pos, f, backward=True, **kw)
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = 0.5  # the map is linear: differences are exact
        d = (g * (P.rope(x + e, pos, f, **kw) - P.rope(x - e, pos, f, **kw))).sum()
        assert abs(d - dx[i]) < 1e-12


def test_places_and_rows_by_hand():
    kv_len, cu_q = [20, 3, 7], [1, 4, 4, 6]
    assert [P.place(t, kv_len, cu_q) for t in range(8)] == [
        None, (0, 17), (0, 18), (0, 19), (2, 5), (2, 6), None, None]
    table = np.array([[2, 0], [5, -1]])
    assert P.pool_row(0, 0, table, 16, 6) == 32 and P.pool_row(17, 0, table, 16, 6) == 1
    assert P.pool_row(15, 1, table, 16, 6) == 95
    assert P.pool_row(16, 1, table, 16, 6) is None      # no page
    assert P.pool_row(15, 1, table, 16, 5) is None      # page past the pool
    assert P.pool_row(32, 0, table, 16, 6) is None and P.pool_row(-1, 0, table, 16, 6) is None


def test_sets_by_hand():
    assert P.route_set([5, -1, 5, 9, 2, 10, 2**31 - 1], 0, [10]) == [2, 5, 9]
    assert P.causal_set(6, 0, 3, 99) == list(range(7))
    assert P.causal_set(6, 2, 0, 99) == [5, 6]
    assert P.causal_set(6, 2, 3, 99) == [0, 1, 2, 5, 6]
    assert P.causal_set(6, 2, 6, 99) == list(range(7))
    assert P.causal_set(6, 2, 3, 4) == [0, 1, 2]
    assert P.causal_set(-1, 2, 3, 99) == []


def _paged(k, page, seed, spare=2):
    """A contiguous [L, G, D] tensor cut into shuffled pages: (pool, table row)."""
    L, G, D = k.shape
    n = -(-L // page)
    ids = np.random.default_rng(seed).permutation(n + spare)[:n]
    pool = np.full((n + spare, page, G, D), np.nan)
    for i in range(n):
        part = k[i * page:(i + 1) * page]
        pool[ids[i], :len(part)] = part
    return pool, ids[None].astype(np.int32)


def test_routes_over_pages_are_routes_over_the_tensor():
    L, T = 50, 6
    k, v, q = _rand(4, L, 1, 64), _rand(5, L, 1, 64), _rand(6, T, 12, 64)
    routes = np.random.default_rng(7).integers(-3, L + 5, (T, 20)).astype(np.int32)
    routes[2] = -1
    kp, table = _paged(k, 16, 8)
    vp, _ = _paged(v, 16, 8)
    out, lse, _, _ = P.attend(q, kp, vp, table, [L], [0, T], 0.125, routes=routes)
    ref, ref_lse = oracle.forward_dense(q, k, v, routes, 0.125)
    assert np.allclose(out, ref, atol=1e-12)
    assert np.array_equal(np.isfinite(lse), np.isfinite(ref_lse)) and np.isneginf(lse[2]).all()
    fin = np.isfinite(lse)
    assert np.allclose(lse[fin], ref_lse[fin], atol=1e-12)


def test_causal_over_pages_is_causal_attention():
    L, T = 37, 9
    k, v, q = _rand(9, L, 2, 64), _rand(10, L, 2, 64), _rand(11, T, 24, 64)
    kp, table = _paged(k, 16, 12)
    vp, _ = _paged(v, 16, 12)
    out, _, _, _ = P.attend(q, kp, vp, table, [L], [0, T], 0.125)
    f = lambda x: torch.from_numpy(x).transpose(0, 1)[None]  # noqa: E731
    mask = torch.arange(L)[None] <= torch.arange(L - T, L)[:, None]
    ref = torch.nn.functional.scaled_dot_product_attention(f(q), f(np.repeat(k, 12, 1)), f(np.repeat(v, 12, 1)),
                                                           attn_mask=mask, scale=0.125)
    assert np.allclose(out, ref[0].transpose(0, 1).numpy(), atol=1e-12)


def test_window_and_first_tokens_are_the_routes_that_name_them():
    L, T, window, sinks = 41, 7, 5, 3
    k, v, q = _rand(13, L, 1, 64), _rand(14, L, 1, 64), _rand(15, T, 12, 64)
    kp, table = _paged(k, 16, 16)
    vp, _ = _paged(v, 16, 16)
    routes = np.full((T, window + sinks), -1, np.int32)
    for t in range(T):
        p = L - T + t
        routes[t] = list(range(sinks)) + list(range(p - window + 1, p + 1))
    a = P.attend(q, kp, vp, table, [L], [0, T], 0.125, window=window, sinks=sinks)
    b = P.attend(q, kp, vp, table, [L], [0, T], 0.125, routes=routes)
    assert np.allclose(a[0], b[0], atol=1e-12) and np.allclose(a[1], b[1], atol=1e-12)


def test_append_then_read_back():
    kv_len, cu_q = np.array([18, 4]), np.array([0, 3, 4])
    table = np.array([[1, 3], [0, -1]], np.int32)
    k, v = _rand(17, 5, 1, 8), _rand(18, 5, 1, 8)
    pool = np.zeros((4, 16, 1, 8))
    kp, vp = P.append(k, v, pool, pool, table, kv_len, cu_q)
    assert np.array_equal(kp[1, 15], k[0]) and np.array_equal(kp[3, 0], k[1]) and np.array_equal(vp[3, 1], v[2])
    assert np.array_equal(vp[0, 3], v[3])
    assert np.count_nonzero(kp.any(-1)) == 4  # the row of no sequence went nowhere
