"""The paged cache of latents: kda_latent_cache_store and kda_latent_cache_load
exactly as the oracle, kda_latent_decode within derived bounds, and all of them
together as a server runs them.

Decode's tolerances: with ez = 2 * 576 * 2^-24 * scale * max|q| max|[c s]| + 2^-20 +
n 2^-24 (two float32 sums of 576 products, the exponential, n terms added) a weight,
rounded once to bfloat16, is off by ew = u + 2.1 ez relative; latents are widened
exactly.  So |o - ref| <= ew * sum_j P_ij |c_j| + u |o|; lse is off by ez and the
float32 sum.
"""

import numpy as np
import pytest
import torch

import oracle.attention as attn
import oracle.latent as ref
from test_gpu_attn_prompt import DEV, U, check, f64, rand

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
R, S = 512, 64


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def make_cache(seed, pages, P, pad=0, spread=2):
    """Codes of every kind but NaN, scales of several sizes; with `pad` the pages stand apart."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, (pages, P + pad, R)).astype(np.uint8)
    codes = np.where((codes & 127) == 127, codes ^ 1, codes).astype(np.uint8)
    scales = rng.integers(119, 119 + spread, (pages, P + pad, 4)).astype(np.uint8)
    shared = rand(seed, pages, P + pad, S)
    flat = [torch.from_numpy(codes).to(DEV).view(E4M3), torch.from_numpy(scales).to(DEV), shared.to(DEV)]
    return [t[:, :P] for t in flat], flat


def arrays(cache):
    return [cache[0].contiguous().view(torch.uint8).cpu().numpy(), cache[1].cpu().numpy(), f64(cache[2])]


def check_store(kda, c, s, slots, cache):
    before = arrays(cache)
    kda.latent_cache_store(c, s, *cache, ints(slots))
    want = ref.latent_cache_store(f64(c), f64(s), *before, slots)
    got = arrays(cache)
    nan = (want[0] & 127) == 127
    np.testing.assert_array_equal((got[0] & 127) == 127, nan)
    np.testing.assert_array_equal(got[0][~nan], want[0][~nan])
    np.testing.assert_array_equal(got[1], want[1])
    np.testing.assert_array_equal(got[2], want[2])


# ---------------------------------------------------------------- store

@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("T", [1, 3, 8, 9, 4500])
def test_store(gpu_lib, P, T):
    """Any slots in any order, some tokens not stored, values of all sizes, one launch shape and the other."""
    rng = np.random.default_rng(P + T)
    pages = 2 * T // P + 3
    slots = rng.permutation(pages * P)[:T]
    slots[rng.random(T) < 0.1] = -1
    if T > 8:
        slots[:4] = [-7, pages * P, 2 ** 31 - 1, -2 ** 31]
    gain = torch.exp2(torch.from_numpy(rng.integers(-20, 20, (T, 4, 1))).float())
    c = (rand(T, T, 4, 128).float() * gain).bfloat16().reshape(T, R).to(DEV)
    cache, _ = make_cache(P, pages, P)
    check_store(gpu_lib, c, rand(T + 1, T, S).to(DEV), slots, cache)


def test_store_every_value(gpu_lib):
    """All 2^16 bf16 values, beside others of their binade and mixed ones; the largest, which no scale holds exactly."""
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    mixed = every[torch.randperm(65536, generator=torch.Generator().manual_seed(1))]
    rows = torch.cat((every, mixed)).reshape(256, R).to(DEV)
    cache, _ = make_cache(70, 16, 16)
    check_store(gpu_lib, rows, torch.zeros(256, S, dtype=torch.bfloat16, device=DEV), list(range(256)), cache)
    top = torch.full((2, R), 3.3895e38, dtype=torch.bfloat16, device=DEV)
    assert torch.isfinite(top.float()).all()
    check_store(gpu_lib, top, top[:, :S], [3, 200], cache)
    c, s = gpu_lib.latent_cache_load(*cache, ints([[0]]), ints([0, 4]), 4)
    assert (c[3].float() == 448.0 * 2.0 ** 119).all() and torch.equal(s[3], top[0, :S])


def test_store_strides(gpu_lib):
    """Rows of one projection, pages that stand apart: what lies between stays."""
    cache, flat = make_cache(71, 5, 16, pad=2)
    before = [f.view(torch.uint8).clone() for f in flat]
    row = rand(72, 20, 8 + R + S + 8).to(DEV)
    check_store(gpu_lib, row[:, 8:8 + R], row[:, 8 + R:-8], list(range(30, 50)), cache)
    for a, b in zip(flat, before):
        assert torch.equal(a.view(torch.uint8)[:, 16:], b[:, 16:])


# ---------------------------------------------------------------- load

LOADS = [  # lengths, page size, tokens before and behind
    ([1], 16, 0, 0), ([5, 0, 33, 16, 0], 16, 0, 0), ([64, 1, 200], 64, 3, 9), ([0, 0, 0], 32, 2, 5), ([1000], 128, 0, 1),
    ([1] * 300, 16, 0, 0), ([0] * 99 + [700] + [0] * 99 + [3], 256, 1, 1),
]


@pytest.mark.parametrize("lens,P,lead,tail", LOADS)
@pytest.mark.parametrize("pad", [0, 2])
def test_load(gpu_lib, lens, P, lead, tail, pad):
    rng = np.random.default_rng(P)
    W = max(-(-max(lens) // P), 1)
    pages = max(len(lens) * W // 2, 3)
    cache, _ = make_cache(P + pad, pages, P, pad, spread=9)
    wide = rng.integers(-1, pages + 1, (len(lens), W + pad)).astype(np.int32)      # some without a page
    cu = np.concatenate(([lead], lead + np.cumsum(lens)))
    T = int(cu[-1]) + tail
    c = torch.full((T, R), 7.5, dtype=torch.bfloat16, device=DEV)
    s = torch.full((T, S), 7.5, dtype=torch.bfloat16, device=DEV)
    gpu_lib.latent_cache_load(*cache, ints(wide)[:, :W], ints(cu), T, c=c, k_shared=s)
    for got, want in zip((c, s), ref.latent_cache_load(*arrays(cache), wide[:, :W], cu, T)):
        np.testing.assert_array_equal(f64(got), np.where(np.isnan(want), 7.5, want))
    # lengths past the table's end: zeros
    if W > 1:
        a, b = gpu_lib.latent_cache_load(*cache, ints(wide)[:, :1], ints(cu), T)
        for got, want in zip((a, b), ref.latent_cache_load(*arrays(cache), wide[:, :1], cu, T)):
            keep = ~np.isnan(want)
            np.testing.assert_array_equal(f64(got)[keep], want[keep])


def test_load_every_code(gpu_lib):
    """Every code under every scale that a store makes, NaN too, exactly."""
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).repeat(2)
    scales = torch.arange(63, 247, dtype=torch.int32).to(torch.uint8)
    n = len(scales)
    c_cache = codes.expand(12, 16, R).contiguous().to(DEV)
    c_scale = torch.cat((scales, scales[:192 - n])).view(12, 16, 1).expand(-1, -1, 4).contiguous().to(DEV)
    k_cache = rand(1, 12, 16, S).to(DEV)
    c, s = gpu_lib.latent_cache_load(c_cache.view(E4M3), c_scale, k_cache, ints([list(range(12))]), ints([0, n]), n)
    want = attn.e4m3_table()[codes.numpy()][None] * 2.0 ** (scales.numpy().astype(float) - 127)[:, None]
    np.testing.assert_array_equal(f64(c), want)
    assert torch.equal(s, k_cache.view(-1, S)[:n])


def test_store_then_load(gpu_lib):
    """What was stored comes back within half an e4m3 step, the shared part as it was; stored again it is the same."""
    c, s = rand(80, 100, R).to(DEV), rand(81, 100, S).to(DEV)
    cache, _ = make_cache(82, 8, 32)
    slots = ints([(5, 2, 7, 0)[t // 32] * 32 + t % 32 for t in range(100)])
    gpu_lib.latent_cache_store(c, s, *cache, slots)
    a, b = gpu_lib.latent_cache_load(*cache, ints([[5, 2, 7, 0]]), ints([0, 100]), 100)
    assert torch.equal(b, s)
    top = c.float().view(100, 4, 128).abs().amax(-1, keepdim=True).expand(-1, -1, 128).reshape(100, R)
    assert ((a.float() - c.float()).abs() <= torch.maximum(c.float().abs() * 2.0 ** -4, top * 2.0 ** -17)).all()
    gpu_lib.latent_cache_store(a, b, *cache, slots)
    d, e = gpu_lib.latent_cache_load(*cache, ints([[5, 2, 7, 0]]), ints([0, 100]), 100)
    assert torch.equal(a, d) and torch.equal(b, e)


# ---------------------------------------------------------------- decode

def make_decode(seed, lens, Q, H, P, W=None, pad=0):
    rng = np.random.default_rng(seed)
    held = [-(-max(n, 0) // P) for n in lens]
    W = W or max(max(held), 1)
    pages = sum(held) + 2
    ids, at = rng.permutation(pages), 0
    table = np.full((len(lens), W), -1, np.int32)
    for row, n in zip(table, held):
        row[:min(n, W)] = ids[at:at + n][:W]
        at += n
    cache, flat = make_cache(seed, pages, P, pad)
    return rand(seed + 1, len(lens), Q, H, R + S).to(DEV), cache, table, flat


def check_decode(o, lse, q, cache, table, lens, scale=ref.SCALE):
    x, arr = f64(q), arrays(cache)
    want, wl, o_abs = ref.latent_decode(x, *arr, table, lens, scale)
    with np.errstate(invalid="ignore"):
        key = np.nanmax(np.linalg.norm(ref.latents(*arr[:2]), axis=-1)) ** 2 + np.nanmax(np.linalg.norm(arr[2], axis=-1)) ** 2
    ez = 2 * 576 * 2.0 ** -24 * scale * np.linalg.norm(x, axis=-1).max() * key ** 0.5 + 2.0 ** -20 + max(max(lens), 0) * 2.0 ** -24
    check(o, want, ((U + 2.1 * ez) * o_abs + U * np.abs(want)) * 1.01 + 1e-30, "o")
    none = np.isneginf(wl)
    assert (f64(lse)[none] == -np.inf).all() and (f64(o)[none] == 0).all()
    check(lse, np.where(none, np.nan, wl), ez + 2.0 ** -22 * (1 + np.abs(np.where(none, 0, wl))), "lse")


DECODES = [  # lengths, Q, H, page size
    ([1], 1, 1, 16), ([15, 1, 17], 1, 5, 16), ([64, 63, 65, 128, 127, 129], 1, 32, 32), ([300], 1, 33, 64),
    ([0, 200, 0, 3], 1, 16, 128), ([70, 500], 1, 64, 64), ([130, 2], 1, 65, 16), ([100, 260, 31], 1, 96, 256),
    ([90, 3], 1, 100, 32), ([200, 1, 0], 1, 128, 64), ([150, 33], 1, 129, 64), ([77], 1, 300, 16),
    ([5, 64, 1, 0, 260], 4, 8, 16), ([1, 2, 3, 70], 3, 20, 64), ([130, 131, 192], 2, 64, 32), ([40, 7], 9, 32, 16),
    ([2, 66], 130, 2, 64), ([2000, 1, 900], 1, 16, 16), ([1500, 700], 2, 40, 64), ([3000], 1, 128, 128),
    ([5, 3000, 0, 64] * 5, 1, 12, 64),
]


@pytest.mark.parametrize("lens,Q,H,P", DECODES)
def test_decode(gpu_lib, lens, Q, H, P):
    q, cache, table, _ = make_decode(len(lens) + H, lens, Q, H, P)
    o, lse = gpu_lib.latent_decode(q, *cache, ints(table), ints(lens))
    check_decode(o, lse, q, cache, table, lens)
    a, b = gpu_lib.latent_decode(q, *cache, ints(table), ints(lens))
    assert torch.equal(a, o) and torch.equal(b, lse)


def test_decode_many_sequences(gpu_lib):
    """More sequences than pieces, of every length to 80."""
    lens = [int(x) for x in np.random.default_rng(3).integers(0, 81, 700)]
    q, cache, table, _ = make_decode(5, lens, 1, 8, 16)
    o, lse = gpu_lib.latent_decode(q, *cache, ints(table), ints(lens))
    check_decode(o, lse, q, cache, table, lens)


@pytest.mark.parametrize("H", [40, 70, 130])
def test_decode_many_sequences_of_many_heads(gpu_lib, H):
    """More sequences, or row tiles of them, than pieces, with some much longer than the others."""
    lens = [int(x) for x in np.random.default_rng(H).integers(0, 40, 270)]
    lens[100] = 900
    lens[269] = 300
    q, cache, table, _ = make_decode(6, lens, 1, H, 16)
    o, lse = gpu_lib.latent_decode(q, *cache, ints(table), ints(lens))
    check_decode(o, lse, q, cache, table, lens)


@pytest.mark.parametrize("N", [300, 600])
@pytest.mark.parametrize("Q,H", [(1, 1), (1, 17), (1, 32), (4, 8), (6, 5)])
def test_decode_more_sequences_than_workgroups(gpu_lib, N, Q, H):
    """Many short histories: missing pages, NaN beside the tokens, and NaN among the newest ones, which the queries
    before them do not see."""
    rng = np.random.default_rng(40 + H)
    lens = [int(x) for x in rng.integers(0, 50, N)]
    lens[7], lens[N - 1] = 1500, 400
    q, cache, table, _ = make_decode(41, lens, Q, H, 16)
    table[7, 3] = table[20, 0] = -1
    held = np.zeros(cache[0].shape[:2], bool)
    for row, n in zip(table, lens):
        for t in range(n):
            held[row[t // 16], t % 16] |= row[t // 16] >= 0
    o, lse = gpu_lib.latent_decode(q, *cache, ints(table), ints(lens))
    check_decode(o, lse, q, cache, table, lens)
    free = torch.from_numpy(~held).to(DEV)
    cache[0].view(torch.uint8)[free] = 0x7f
    cache[1][free] = 255
    cache[2][free] = float("nan")
    a, b = gpu_lib.latent_decode(q, *cache, ints(table), ints(lens))
    assert torch.equal(a, o) and torch.equal(b, lse)
    if Q > 1:
        for row, n in zip(table, lens):
            if n > 1 and row[(n - 1) // 16] >= 0:
                cache[0].view(torch.uint8)[row[(n - 1) // 16], (n - 1) % 16, 77] = 0xff
        a, b = gpu_lib.latent_decode(q, *cache, ints(table), ints(lens))
        assert torch.equal(a[:, :Q - 1], o[:, :Q - 1]) and torch.equal(b[:, :Q - 1], lse[:, :Q - 1])
        seen = [n > 1 and row[(n - 1) // 16] >= 0 for row, n in zip(table, lens)]
        assert torch.isnan(a[:, Q - 1][torch.tensor(seen, device=DEV)]).all()


def test_decode_tables(gpu_lib):
    """Missing pages in the middle, ids out of range, lengths past the table, wide tables, slices of wider rows."""
    lens = [300, 500, -4, 10 ** 9, 64]
    q, cache, table, _ = make_decode(7, [300, 500, 0, 320, 64], 2, 24, 16, W=20, pad=2)
    table[0, 3], table[0, 18], table[1, 0], table[4, 0] = -1, 10 ** 6, -7, -1
    table[3, 10:] = -1
    wide = np.full((5, 90), 1, np.int32)
    wide[:, 5:25] = table
    o, lse = gpu_lib.latent_decode(q, *cache, ints(wide)[:, 5:25], ints(lens))
    check_decode(o, lse, q, cache, table, [300, 500, 0, 320, 64])
    # a wider table of the same pages
    more = np.full((5, 4000), -1, np.int32)
    more[:, :20] = table
    a, b = gpu_lib.latent_decode(q, *cache, ints(more), ints([300, 500, 0, 320, 64]))
    check_decode(a, b, q, cache, more, [300, 500, 0, 320, 64])


def test_decode_queries_of_wider_rows(gpu_lib):
    lens = [200, 90]
    _, cache, table, _ = make_decode(8, lens, 3, 6, 32)
    row = rand(9, 2, 3, 16 + 6 * (R + S)).to(DEV)
    q = row[..., 16:].unflatten(-1, (6, R + S))
    o, lse = gpu_lib.latent_decode(q, *cache, ints(table), ints(lens))
    a, b = gpu_lib.latent_decode(q.contiguous(), *cache, ints(table), ints(lens))
    assert torch.equal(a, o) and torch.equal(b, lse)


@pytest.mark.parametrize("scale", [0.003, 0.6])
def test_decode_scale(gpu_lib, scale):
    lens = [700, 65]
    q, cache, table, _ = make_decode(10, lens, 2, 16, 64)
    o, lse = gpu_lib.latent_decode(q, *cache, ints(table), ints(lens), scale=scale)
    check_decode(o, lse, q, cache, table, lens, scale)


@pytest.mark.parametrize("Q,H", [(1, 8), (4, 8), (3, 40), (2, 64)])
def test_decode_beside_nan(gpu_lib, Q, H):
    """NaN in everything that no sequence holds: the pages' ends, other pages, the shared parts there."""
    lens = [1, 70, 16, 130, 0]
    q, cache, table, _ = make_decode(11, lens, Q, H, 16)
    want = gpu_lib.latent_decode(q, *cache, ints(table), ints(lens))
    held = np.zeros(cache[0].shape[:2], bool)
    for row, n in zip(table, lens):
        for t in range(n):
            held[row[t // 16], t % 16] = True
    free = torch.from_numpy(~held).to(DEV)
    cache[0].view(torch.uint8)[free] = 0x7f
    cache[1][free] = 255
    cache[2][free] = float("nan")
    got = gpu_lib.latent_decode(q, *cache, ints(table), ints(lens))
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("H", [8, 30, 64])
def test_decode_later_nan(gpu_lib, H):
    """A NaN among the newest tokens, in one code or in the shared part, stays out of the queries before it."""
    lens, Q = [40, 129, 5, 64], 6
    q, cache, table, _ = make_decode(12, lens, Q, H, 16)
    o, lse = gpu_lib.latent_decode(q, *cache, ints(table), ints(lens))
    for back in range(1, 5):
        for part in range(2):
            now = [t.clone() for t in cache]
            for row, n in zip(table, lens):
                t = n - back
                if part:
                    now[2][row[t // 16], t % 16, 9] = float("inf") if back % 2 else float("nan")
                else:
                    now[0].view(torch.uint8)[row[t // 16], t % 16, 100 * back] = 0xff
            a, b = gpu_lib.latent_decode(q, *now, ints(table), ints(lens))
            assert torch.equal(a[:, :Q - back], o[:, :Q - back]) and torch.equal(b[:, :Q - back], lse[:, :Q - back])
            if not part:
                assert torch.isnan(a[:, Q - back:]).all() and torch.isnan(b[:, Q - back:]).all()


@pytest.mark.parametrize("H", [5, 8, 30, 64])
def test_decode_later_large(gpu_lib, H):
    """The newest tokens' latents under the largest scale leave the queries before them as they were, to the bit."""
    lens, Q = [40, 129, 5, 64], 6
    q, cache, table, _ = make_decode(17, lens, Q, H, 16)
    o, lse = gpu_lib.latent_decode(q, *cache, ints(table), ints(lens))
    for back in range(1, 5):
        now = [t.clone() for t in cache]
        for row, n in zip(table, lens):
            t = n - back
            now[0].view(torch.uint8)[row[t // 16], t % 16] = 0x7e           # 448
            now[1][row[t // 16], t % 16] = 246
        a, b = gpu_lib.latent_decode(q, *now, ints(table), ints(lens))
        assert torch.equal(a[:, :Q - back], o[:, :Q - back]) and torch.equal(b[:, :Q - back], lse[:, :Q - back])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("H", [8, 40, 70, 100])
def test_decode_query_that_is_not_finite(gpu_lib, H, bad):
    """It gives its own row NaN, and the others what they were."""
    lens = [300, 40]
    q, cache, table, _ = make_decode(14, lens, 2, H, 16)
    o, lse = gpu_lib.latent_decode(q, *cache, ints(table), ints(lens))
    hit = torch.zeros(2, 2, H, dtype=torch.bool)
    hit[0, 0, 3] = hit[0, 1, H - 1] = hit[1, 1, 0] = True
    other = q.clone()
    other[hit.to(DEV)] = bad
    a, b = gpu_lib.latent_decode(other, *cache, ints(table), ints(lens))
    hit = hit.to(DEV)
    assert torch.isnan(a[hit]).all()
    assert torch.equal(a[~hit], o[~hit]) and torch.equal(b[~hit], lse[~hit])


@pytest.mark.parametrize("H", [16, 48, 96])
def test_decode_beside_large_scales(gpu_lib, H):
    """Latents whose scales are far apart, between tokens and between the blocks of one."""
    lens = [90, 33]
    q, cache, table, _ = make_decode(15, lens, 1, H, 16)
    rng = np.random.default_rng(16)
    cache[1].copy_(torch.from_numpy((127 + rng.integers(-40, 1, cache[1].shape)).astype(np.uint8)))
    o, lse = gpu_lib.latent_decode(q, *cache, ints(table), ints(lens))
    check_decode(o, lse, q, cache, table, lens)


def test_decode_past_32_bits(gpu_lib):
    """Pages 2^27 codes apart, 40 of them: offsets past 2^32 in all three parts."""
    pages, P = 40, 16
    c_big = torch.empty(pages << 27, dtype=torch.uint8, device=DEV)
    k_big = torch.empty(pages << 26, dtype=torch.bfloat16, device=DEV)
    lens = [630]
    q, cache, table, _ = make_decode(13, lens, 2, 10, P)
    assert cache[0].shape[0] > pages - 1
    cache = [t[:pages] for t in cache]
    table = np.arange(pages, dtype=np.int32)[None, ::-1].copy()
    far = [c_big.as_strided((pages, P, R), (1 << 27, R, 1)).view(E4M3),
           c_big.as_strided((pages, P, 4), (1 << 27, 4, 1), 1 << 20), k_big.as_strided((pages, P, S), (1 << 26, S, 1))]
    far[0].view(torch.uint8).copy_(cache[0].view(torch.uint8))
    far[1].copy_(cache[1])
    far[2].copy_(cache[2])
    for a, b in zip(gpu_lib.latent_decode(q, *cache, ints(table), ints(lens)),
                    gpu_lib.latent_decode(q, *far, ints(table), ints(lens))):
        assert torch.equal(a, b)
    for a, b in zip(gpu_lib.latent_cache_load(*cache, ints(table), ints([0, 630]), 630),
                    gpu_lib.latent_cache_load(*far, ints(table), ints([0, 630]), 630)):
        assert torch.equal(a, b)
    check_store(gpu_lib, rand(14, 50, R).to(DEV), rand(15, 50, S).to(DEV), list(range(570, 620)), far)


def test_decodes_share_nothing_but_what_is_said(gpu_lib):
    """Two decodes at once on two streams, with a workspace each; one workspace for two calls in turn, dirty."""
    kda = gpu_lib
    sets = []
    for seed, lens, H in ((20, [900, 40, 333], 16), (21, [64, 1000], 48)):
        q, cache, table, _ = make_decode(seed, lens, 1, H, 32)
        args = (q, *cache, ints(table), ints(lens))
        sets.append((args, kda.latent_decode(*args)))
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    torch.cuda.synchronize()
    for (args, _), st in zip(sets, streams):
        with torch.cuda.stream(st):
            got.append(kda.latent_decode(*args))
    torch.cuda.synchronize()
    size = max(kda.latent_decode_workspace_size(*args[0].shape[:3]) for args, _ in sets)
    ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    for (args, want), one in zip(sets, got):
        again = kda.latent_decode(*args, workspace=ws)
        assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, one, again))


@pytest.mark.parametrize("H", [16, 72])
def test_two_graphs_of_one_workspace(gpu_lib, H):
    """Replayed in turn, with eager work between them, on inputs and lengths of their own."""
    kda = gpu_lib
    ws = torch.empty(kda.latent_decode_workspace_size(3, 1, H), dtype=torch.uint8, device=DEV)
    sets = []
    for seed, lens in ((60, [700, 5, 129]), (61, [64, 0, 1000])):
        q, cache, table, _ = make_decode(seed, lens, 1, H, 32, W=40)
        args = [q, *cache, ints(table), ints(lens)]
        kda.latent_decode(*args, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = kda.latent_decode(*args, workspace=ws)
        sets.append((graph, args, out, lens))
    for turn in range(4):
        for i, (graph, args, out, lens) in enumerate(sets):
            args[0].copy_(rand(70 + 2 * turn + i, *args[0].shape))
            args[5].copy_(ints([max(n - 31 * turn, 0) for n in lens]))
            ws.fill_(255)
            graph.replay()
            got = [t.clone() for t in out]
            want = kda.latent_decode(*args)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---------------------------------------------------------------- together

def test_serving(gpu_lib):
    """A server's run: prompts in two parts, the second over what is read back of the first, then captured steps that
    deal pages, store and decode; against float64 attention over what was stored."""
    kda, H, P, N = gpu_lib, 4, 16, 3
    rng = np.random.default_rng(30)
    wk, wv = (torch.from_numpy(rng.standard_normal((H, 128, R)) * 0.04).to(DEV) for _ in range(2))
    cache, _ = make_cache(31, 40, P)
    table, free, head = ints(np.full((N, 12), -1)), ints(rng.permutation(40)), ints([0])
    old, latents, shared = [0] * N, [np.zeros((0, R)) for _ in range(N)], [np.zeros((0, S)) for _ in range(N)]

    def expand(c):
        return torch.einsum("nr,hdr->nhd", c.double(), wk).bfloat16(), torch.einsum("nr,hdr->nhd", c.double(), wv).bfloat16()

    def absorb(q):
        return torch.cat((torch.einsum("nqhd,hdr->nqhr", q[..., :128].double(), wk), q[..., 128:].double()), -1).bfloat16()

    def kept():
        """What the cache holds now, as the oracle stores it."""
        return [ref.cached(*arrays(cache), row, n)[:2] for row, n in zip(table.cpu().numpy(), old)]

    for part, new in enumerate(([20, 33, 5], [17, 2, 40])):
        T = sum(new)
        c, s, q = rand(40 + part, T, R).to(DEV), rand(42 + part, T, S).to(DEV), rand(44 + part, 1, T, H, 192).to(DEV)
        cu, slots, lens, head = kda.attn_tables(ints(old), ints(new), table, free, head, P, T)
        kda.latent_cache_store(c, s, *cache, slots)
        old = [a + b for a, b in zip(old, new)]
        cu_kv = ints(np.concatenate(([0], np.cumsum(old))))
        all_c, all_s = kda.latent_cache_load(*cache, table, cu_kv, sum(old))
        for (x, y), lo, hi in zip(kept(), cu_kv.tolist(), cu_kv.tolist()[1:]):
            np.testing.assert_array_equal(f64(all_c[lo:hi]), x)
            np.testing.assert_array_equal(f64(all_s[lo:hi]), y)
        k, v = expand(all_c)
        o, lse = kda.latent_prefill(q, k[None], all_s[None], v[None], cu_seqlens=cu, cu_seqlens_kv=cu_kv)
        from test_gpu_latent_prompt import check_prompt
        check_prompt(o, lse, q, k[None], all_s[None], v[None], cu.tolist(), cu_kv.tolist())

    # steps: captured once, replayed with the lengths, inputs and list heads of each
    old_t, new_t, head_t = ints(old), ints([2] * N), head.clone()
    c, s, q = rand(50, 2 * N, R).to(DEV), rand(51, 2 * N, S).to(DEV), absorb(rand(52, N, 2, H, 192).to(DEV))
    ws = torch.empty(kda.latent_decode_workspace_size(N, 2, H), dtype=torch.uint8, device=DEV)
    kda.latent_decode(q, *cache, table, old_t, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cu, slots, lens, next_head = kda.attn_tables(old_t, new_t, table, free, head_t, P, 2 * N)
        kda.latent_cache_store(c, s, *cache, slots)
        o, lse = kda.latent_decode(q, *cache, table, lens, workspace=ws)
    for step in range(12):
        c.copy_(rand(60 + step, 2 * N, R))
        s.copy_(rand(80 + step, 2 * N, S))
        q.copy_(absorb(rand(100 + step, N, 2, H, 192).to(DEV)))
        before = arrays(cache)
        graph.replay()
        old = [a + 2 for a in old]
        assert lens.tolist() == old
        for got, want in zip(arrays(cache), ref.latent_cache_store(f64(c), f64(s), *before, slots.tolist())):
            np.testing.assert_array_equal(got, want)
        check_decode(o, lse, q, cache, table.cpu().numpy(), old)
        old_t.copy_(lens)
        head_t.copy_(next_head)


def test_absorbed_is_expanded(gpu_lib):
    """The two forms agree on one layer, within the roundings of the queries, keys, values and weights between them."""
    kda, H, n, Q = gpu_lib, 6, 300, 3
    rng = np.random.default_rng(32)
    wk, wv = (torch.from_numpy(rng.standard_normal((H, 128, R)) * 0.04).to(DEV) for _ in range(2))
    cache, _ = make_cache(33, 5, 64)
    table = ints([[3, 0, 4, 1, 2]])
    q = rand(34, 1, Q, H, 192).to(DEV)
    c, s = kda.latent_cache_load(*cache, table, ints([0, n]), n)
    k, v = (torch.einsum("nr,hdr->nhd", c.double(), w).bfloat16()[None] for w in (wk, wv))
    o, lse = kda.latent_prefill(q, k, s[None], v)
    absorbed = torch.cat((torch.einsum("nqhd,hdr->nqhr", q[..., :128].double(), wk), q[..., 128:].double()), -1).bfloat16()
    a, b = kda.latent_decode(absorbed, *cache, table, ints([n]))
    # a score moves by u of its products' magnitudes (key or query rounded), a weight by twice that and its own rounding
    x = (f64(absorbed), f64(c), f64(s))
    qa, key = np.abs(x[0]), np.concatenate((np.abs(x[1]), np.abs(x[2])), 1)
    moved = 2 * U * ref.SCALE * (np.einsum("qhr,nr->qhn", qa[0], key).max()
                                 + np.einsum("qhd,nhd->qhn", np.abs(f64(q[0, :, :, :128])), np.abs(f64(k[0]))).max())
    assert (np.abs(f64(lse)[0].T - f64(b)[0]) <= moved).all()
    out = torch.einsum("nqhr,hdr->nqhd", a.double(), wv)
    room = 4 * (moved + 2 * U) * float(v.float().abs().max())
    assert float((out - o.double()).abs().max()) <= room
    rel = float((out - o.double()).norm() / o.double().norm())
    assert rel < 0.1, rel


def test_refusals(gpu_lib):
    kda = gpu_lib
    q, cache, table, _ = make_decode(60, [40, 9], 1, 4, 16)
    t, lens = ints(table), ints([40, 9])
    c, s = rand(61, 3, R).to(DEV), rand(62, 3, S).to(DEV)
    slots = ints([0, 1, 2])
    for args, what in (((c[:, :500], s, *cache, slots), "c must be"), ((c, s[:2], *cache, slots), "k_shared must be"),
                       ((c, s, cache[0][:, :8], *cache[1:], slots), "c_scale must be"),
                       ((c, s, cache[0][..., :256], *cache[1:], slots), "c_cache must be"),
                       ((c, s, *cache, slots[:2]), "slots must be"), ((c, s, *cache, slots.cpu()), "slots must be a GPU"),
                       ((c, s, *cache[:2], cache[2].transpose(1, 2).contiguous().transpose(1, 2), slots), "compact")):
        with pytest.raises(ValueError, match=what):
            kda.latent_cache_store(*args)
    with pytest.raises(TypeError, match="c_scale must be"):
        kda.latent_cache_store(c, s, cache[0], cache[1].float(), cache[2], slots)
    with pytest.raises(ValueError, match="page_table must be"):
        kda.latent_cache_load(*cache, t, ints([0, 5]), 5)
    with pytest.raises(ValueError, match="num_tokens"):
        kda.latent_cache_load(*cache, t, ints([0, 5, 6]), -1)
    with pytest.raises(ValueError, match="q must be"):
        kda.latent_decode(q[..., :512], *cache, t, lens)
    with pytest.raises(ValueError, match="kv_lens must be"):
        kda.latent_decode(q, *cache, t, lens[:1])
    with pytest.raises(ValueError, match="out must be"):
        kda.latent_decode(q, *cache, t, lens, out=q)
    with pytest.raises(kda.KDAError, match="orkspace"):
        kda.latent_decode(q, *cache, t, lens, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(kda.KDAError):
        kda.latent_decode(q, *cache, t, lens, scale=0.0)
