"""Pins of the attention oracle: closed forms, differences, and torch's own e4m3 conversion."""

import numpy as np
import pytest
import torch

import oracle.attention as ref


def _rand(rng, *shape):
    return rng.standard_normal(shape)


def test_first_token_and_equal_keys():
    rng = np.random.default_rng(0)
    q, v = _rand(rng, 1, 5, 2, 8), _rand(rng, 1, 5, 1, 8)
    k = np.broadcast_to(_rand(rng, 8), (1, 5, 1, 8))
    o, lse, _ = ref.attn_prefill(q, k, v)
    # equal keys: the mean of the values so far, and log(i + 1) above the common score
    for i in range(5):
        np.testing.assert_allclose(o[0, i], np.broadcast_to(v[0, :i + 1, 0].mean(0), (2, 8)), rtol=1e-12)
        np.testing.assert_allclose(lse[0, :, i], (q[0, i] @ k[0, 0, 0]) * 8 ** -0.5 + np.log(i + 1), rtol=1e-12)


def test_packed_is_each_alone():
    rng = np.random.default_rng(1)
    q, k, v = _rand(rng, 1, 12, 4, 8), _rand(rng, 1, 12, 2, 8), _rand(rng, 1, 12, 2, 8)
    o, lse, _ = ref.attn_prefill(q, k, v, cu=[2, 2, 7, 11])
    assert np.isnan(o[0, :2]).all() and np.isnan(o[0, 11:]).all()
    for lo, hi in ((2, 7), (7, 11)):
        a, b, _ = ref.attn_prefill(q[:, lo:hi], k[:, lo:hi], v[:, lo:hi])
        np.testing.assert_array_equal(o[:, lo:hi], a)
        np.testing.assert_array_equal(lse[:, :, lo:hi], b)


@pytest.mark.parametrize("cu", [None, [0, 3, 3, 7]])
def test_gradients_are_the_differences(cu):
    rng = np.random.default_rng(2)
    x = [_rand(rng, 1, 7, 4, 6), _rand(rng, 1, 7, 2, 6), _rand(rng, 1, 7, 2, 6)]
    up = _rand(rng, 1, 7, 4, 6)
    grads, _ = ref.attn_backward(*x, up, cu)
    for which in range(3):
        for at in [(0, 0, 0, 1), (0, 2, 1, 3), (0, 3, 0, 0), (0, 6, 1, 5)]:
            vals = []
            for step in (1e-5, -1e-5):
                y = [a.copy() for a in x]
                y[which][at] += step
                vals.append((ref.attn_prefill(*y, cu)[0] * up).sum())
            assert abs((vals[0] - vals[1]) / 2e-5 - grads[which][at]) < 1e-8


def test_e4m3_is_torchs():
    """Every bf16 value up to 448 in magnitude, and the conversion back."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = x[~(x.float().abs() > 448)]             # NaN stays in
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = ref.to_e4m3(x.double().numpy())
    nan = np.isnan(x.double().numpy())
    np.testing.assert_array_equal(got[~nan], want[~nan])
    assert ((got[nan] & 127) == 127).all()
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    np.testing.assert_array_equal(ref.e4m3_table(), codes.view(torch.float8_e4m3fn).double().numpy())


def test_scale_is_the_least_that_fits():
    for top in (0.0, 1e-30, 1.0, 447.9, 448.0, 449.0, 2.0 ** 100, 0.875, 0.8750001, 3.38e38):
        s = ref.scale_for(top)
        assert 448 * s >= top and (448 * s / 2 < top or s == 2.0 ** -64)


def test_store_keeps_and_rescales():
    rng = np.random.default_rng(3)
    cache, scale = np.zeros((3, 1, 4, 8), np.uint8), np.ones((3, 1))
    a = _rand(rng, 3, 1, 8)
    cache, scale = ref.attn_cache_store(a, cache, scale, [4, 5, -1])
    big = 100 * _rand(rng, 2, 1, 8)
    cache2, scale2 = ref.attn_cache_store(big, cache, scale, [6, 99])
    assert scale2[1, 0] > scale[1, 0] and (cache2[1, 0, 3] == 0).all() and (cache2[[0, 2]] == 0).all()
    values = ref.e4m3_table()[cache2[1, 0]] * scale2[1, 0]
    # two roundings to 4 significant bits, or half of the smallest step
    np.testing.assert_allclose(values[:2], a[:2, 0], rtol=2 * 2.0 ** -4, atol=scale2[1, 0] * 2.0 ** -10 * 1.01)


def test_tables_example():
    table = np.full((3, 3), -7)
    table[0, 0] = 9
    cu, slots, lens, table, head = ref.attn_tables([3, 0, 8], [2, 0, 1], table, [5, 6], 0, 4, 5)
    assert cu.tolist() == [0, 2, 2, 3] and lens.tolist() == [5, 0, 9] and head == 2
    assert slots.tolist() == [9 * 4 + 3, 5 * 4, 6 * 4, -1, -1]
    assert table.tolist() == [[9, 5, -7], [-7, -7, -7], [-7, -7, 6]]


def test_decode_is_the_last_rows():
    """Over a cache that holds the values exactly, the last rows of the whole attention."""
    rng = np.random.default_rng(4)
    T, P = 11, 4
    codes = [rng.integers(0, 120, (1, T, 2, 8)).astype(np.uint8) for _ in "kv"]
    k, v = (ref.e4m3_table()[c] for c in codes)
    q = _rand(rng, 1, T, 4, 8)
    caches = []
    for c in codes:
        x = np.full((5, 2, P, 8), 0x7f, np.uint8)          # NaN everywhere else
        for t in range(T):
            x[[3, 1, 4][t // P], :, t % P] = c[0, t]
        caches.append(x)
    one = np.ones((5, 2))
    o, lse, _ = ref.attn_decode(q[:, -3:], *caches, one, one, np.array([[3, 1, 4, 99]]), [T])
    want, wl, _ = ref.attn_prefill(q, k, v)
    np.testing.assert_allclose(o, want[:, -3:], rtol=1e-10)
    np.testing.assert_allclose(lse[0], wl[0, :, -3:].T, rtol=1e-10)
    o, lse, _ = ref.attn_decode(q[:, -3:], *caches, one, one, np.array([[3, 1, 4]]), [2])
    assert (o[0, 0] == 0).all() and np.isneginf(lse[0, 0]).all() and np.isfinite(lse[0, 1:]).all()
