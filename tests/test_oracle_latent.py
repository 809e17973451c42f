"""Pins of the latent-attention oracle: full attention's oracle on the same keys, differences, torch's e4m3 conversion,
and the absorbed form against the expanded one."""

import numpy as np
import pytest
import torch

import oracle.attention as attn
import oracle.latent as ref


def _inputs(seed, T, K, H, B=1):
    rng = np.random.default_rng(seed)
    return [rng.standard_normal(x) for x in ((B, T, H, 192), (B, K, H, 128), (B, K, 64), (B, K, H, 128))]


def test_is_attention_over_joined_keys():
    """192 wide keys and values padded to them: full attention's oracle, which knows nothing of a shared part."""
    q, k, s, v = _inputs(0, 9, 9, 3, B=2)
    key = np.concatenate((k, np.repeat(s[:, :, None], 3, 2)), -1)
    wide = np.concatenate((v, np.zeros((2, 9, 3, 64))), -1)
    o, lse, o_abs = ref.latent_prefill(q, k, s, v)
    a, b, c = attn.attn_prefill(q, key, wide)
    np.testing.assert_allclose(o, a[..., :128], rtol=1e-12)
    np.testing.assert_allclose(lse, b, rtol=1e-12)
    np.testing.assert_allclose(o_abs, c[..., :128], rtol=1e-12)


def test_last_queries_are_the_last_of_a_whole_prompt():
    q, k, s, v = _inputs(1, 11, 11, 2)
    o, lse, _ = ref.latent_prefill(q, k, s, v)
    a, b, _ = ref.latent_prefill(q[:, 7:], k, s, v)
    np.testing.assert_allclose(a, o[:, 7:], rtol=1e-12)
    np.testing.assert_allclose(b, lse[:, :, 7:], rtol=1e-12)
    # more queries than keys: the first see nothing
    a, b, _ = ref.latent_prefill(q, k[:, :4], s[:, :4], v[:, :4])
    assert (a[:, :7] == 0).all() and np.isneginf(b[:, :, :7]).all() and np.isfinite(b[:, :, 7:]).all()
    np.testing.assert_allclose(a[0, 7], v[0, 0], rtol=1e-12)


def test_packed_is_each_alone():
    q, k, s, v = _inputs(2, 12, 15, 2)
    cu, cu_kv = [2, 2, 7, 11], [1, 4, 9, 15]
    o, lse, _ = ref.latent_prefill(q, k, s, v, cu, cu_kv)
    assert np.isnan(o[0, :2]).all() and np.isnan(o[0, 11:]).all()
    for lo, hi, klo, khi in ((2, 7, 4, 9), (7, 11, 9, 15)):
        a, b, _ = ref.latent_prefill(q[:, lo:hi], k[:, klo:khi], s[:, klo:khi], v[:, klo:khi])
        np.testing.assert_array_equal(o[:, lo:hi], a)
        np.testing.assert_array_equal(lse[:, :, lo:hi], b)


@pytest.mark.parametrize("cu,cu_kv", [(None, None), ([0, 3, 3, 7], [0, 5, 6, 9])])
def test_gradients_are_the_differences(cu, cu_kv):
    x = _inputs(3, 7, 9, 2)
    up = np.random.default_rng(4).standard_normal((1, 7, 2, 128))
    grads, _ = ref.latent_backward(*x, up, cu, cu_kv)
    for which in range(4):
        rng = np.random.default_rng(which)
        for _ in range(5):
            at = tuple(int(rng.integers(n)) for n in x[which].shape)
            vals = []
            for step in (1e-5, -1e-5):
                y = [a.copy() for a in x]
                y[which][at] += step
                vals.append((ref.latent_prefill(*y, cu, cu_kv)[0] * up).sum())
            assert abs((vals[0] - vals[1]) / 2e-5 - grads[which][at]) < 1e-8


def test_exponent_is_the_least_that_fits():
    for top in (0.0, 1e-30, 1.0, 447.9, 448.0, 449.0, 2.0 ** 100, 0.875, 0.8750001, 448 * 2.0 ** 119):
        e = ref.exponent_for(top)
        assert 448 * 2.0 ** e >= top and (448 * 2.0 ** (e - 1) < top or e == -64)
    assert ref.exponent_for(3.38e38) == 119


def test_store_and_load():
    """What is stored comes back within half a step of its block's scale, in its place, and nothing else moves."""
    rng = np.random.default_rng(5)
    c, s = rng.standard_normal((5, 512)) * 2.0 ** rng.integers(-30, 30, (5, 4)).repeat(128, 1), rng.standard_normal((5, 64))
    codes = rng.integers(0, 120, (4, 16, 512)).astype(np.uint8)
    scales, shared = rng.integers(100, 140, (4, 16, 4)).astype(np.uint8), rng.standard_normal((4, 16, 64))
    slots = [33, 34, -1, 64, 15]
    a, b, d = ref.latent_cache_store(c, s, codes, scales, shared, slots)
    kept = np.ones((4, 16), bool)
    for t, (page, off) in ((0, (2, 1)), (1, (2, 2)), (4, (0, 15))):
        kept[page, off] = False
        step = 2.0 ** (b[page, off].astype(float) - 127)
        want, got = c[t].reshape(4, 128), ref.latents(a[page, off], b[page, off]).reshape(4, 128)
        assert (np.abs(got - want) <= np.maximum(np.abs(want) * 2.0 ** -4, step[:, None] * 2.0 ** -10)).all()
        top = np.abs(want).max(1)
        assert (top <= 448 * step).all() and (top > 224 * step).all()
        np.testing.assert_array_equal(d[page, off], s[t])
    for new, old in ((a, codes), (b, scales), (d, shared)):
        np.testing.assert_array_equal(new[kept], old[kept])
    got_c, got_s = ref.latent_cache_load(a, b, d, np.array([[2, 0], [-1, 3], [0, 1]]), [1, 4, 4, 24], 25)
    np.testing.assert_array_equal(got_c[2:4], ref.latents(a[2, 1:3], b[2, 1:3]))
    np.testing.assert_array_equal(got_s[19], d[0, 15])
    assert np.isnan(got_c[0]).all() and np.isnan(got_s[24]).all()
    got_c, _ = ref.latent_cache_load(a, b, d, np.array([[-1, 3]]), [0, 20], 20)
    assert (got_c[:16] == 0).all() and (got_c[16:] == ref.latents(a[3, :4], b[3, :4])).all()


def test_codes_are_torchs():
    rng = np.random.default_rng(6)
    c = torch.from_numpy(rng.standard_normal((40, 512))).bfloat16()
    z = np.zeros((1, 64, 512), np.uint8), np.zeros((1, 64, 4), np.uint8), np.zeros((1, 64, 64))
    a, b, _ = ref.latent_cache_store(c.double().numpy(), np.zeros((40, 64)), *z, list(range(40)))
    f = torch.exp2(127.0 - torch.from_numpy(b[0, :40]).double()).repeat_interleave(128, 1)
    want = (c.double() * f).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(a[0, :40], want)


def test_absorbed_is_expanded():
    """The two forms of one layer: projections absorbed into query and output give what expanded keys and values do."""
    rng = np.random.default_rng(7)
    H, n, Q, P = 3, 21, 4, 16
    codes = rng.integers(0, 126, (3, P, 512)).astype(np.uint8)
    scales, shared = rng.integers(118, 122, (3, P, 4)).astype(np.uint8), rng.standard_normal((3, P, 64))
    table = np.array([[2, 0]])
    c, s, _ = ref.cached(codes, scales, shared, table[0], n)
    wk, wv = rng.standard_normal((H, 128, 512)) * 0.05, rng.standard_normal((H, 128, 512)) * 0.05
    q = rng.standard_normal((1, Q, H, 192))
    k, v = (np.einsum("hdr,nr->nhd", w, c)[None] for w in (wk, wv))
    o, lse, _ = ref.latent_prefill(q, k, s[None], v)
    absorbed = np.concatenate((np.einsum("qhd,hdr->qhr", q[0, :, :, :128], wk)[None], q[..., 128:]), -1)
    a, b, _ = ref.latent_decode(absorbed, codes, scales, shared, table, [n])
    np.testing.assert_allclose(np.einsum("qhr,hdr->qhd", a[0], wv), o[0], rtol=1e-9, atol=1e-12)
    np.testing.assert_allclose(b[0].T, lse[0], rtol=1e-10)


def test_decode_without_tokens():
    rng = np.random.default_rng(8)
    codes, scales = rng.integers(0, 120, (2, 16, 512)).astype(np.uint8), np.full((2, 16, 4), 120, np.uint8)
    shared, q = rng.standard_normal((2, 16, 64)), rng.standard_normal((3, 3, 2, 576))
    table = np.array([[0], [-1], [1]])
    o, lse, _ = ref.latent_decode(q, codes, scales, shared, table, [2, 9, 99])
    assert (o[0, 0] == 0).all() and np.isneginf(lse[0, 0]).all() and np.isfinite(lse[0, 1:]).all()
    assert (o[1] == 0).all() and np.isneginf(lse[1]).all()
    np.testing.assert_allclose(o[0, 1], np.broadcast_to(ref.latents(codes[0, 0], scales[0, 0]), (2, 512)), rtol=1e-12)
    whole = ref.latent_decode(q[2:], codes, scales, shared, table[2:], [16])
    np.testing.assert_array_equal(o[2:], whole[0])           # lengths end with the table
