"""The paged cache: kda_attn_tables and kda_attn_cache_store exactly as the
oracle (whole numbers and codes), kda_attn_decode within derived bounds, and
all of them together as a server runs them.

Decode's tolerances are those of the prompt kernels (test_gpu_attn_prompt.py):
codes are widened exactly, a weight times its value's scale is rounded once to
bfloat16.
"""

import numpy as np
import pytest
import torch

import oracle.attention as ref
from test_gpu_attn_prompt import D, DEV, U, check, check_prompt, eps, f64, rand

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------- tables

TABLES = [  # cached, new, page size, width, free pages, head, room
    ([0], [1], 16, 1, 4, 0, 1),
    ([0, 5, 16, 15], [33, 0, 1, 2], 16, 4, 9, 2, 36),
    ([0, 5, 16, 15], [33, 0, 1, 2], 16, 4, 9, 0, 50),            # room behind the last token
    ([0, 5, 16, 15], [33, 0, 1, 2], 16, 4, 9, 0, 20),            # less room than tokens
    ([60, 64, 0], [10, 10, 200], 64, 3, 2, 0, 220),              # pages run out, and rows are too narrow
    ([3, 3], [4, 4], 16, 2, 0, 0, 8),                            # no pages at all, none needed
    ([7, 250, 0], [250, 7, 0], 128, 5, 3, 3, 257),               # head at the end of the list
    ([-3, 4], [5, -2], 16, 2, 3, 0, 6),                          # negative lengths count as 0
    (list(range(0, 1400, 2)), [1] * 700, 32, 50, 100, 0, 700),   # more requests than threads
    ([0] * 3, [5000, 1, 4097], 16, 320, 700, 1, 9098),           # several workgroups
]


@pytest.mark.parametrize("cached,new,P,W,F,head,room", TABLES)
@pytest.mark.parametrize("pad", [0, 3])
def test_tables(gpu_lib, cached, new, P, W, F, head, room, pad):
    N = len(cached)
    rng = np.random.default_rng(N)
    free = rng.permutation(F + 50)[:F]
    wide = rng.integers(0, F + 50, (N, W + pad)).astype(np.int32)
    table = ints(wide)
    got = gpu_lib.attn_tables(ints(cached), ints(new), table[:, :W], ints(free), ints([head]), P, room)
    want = ref.attn_tables(cached, new, wide[:, :W], free, head, P, room)
    for a, b, name in zip((*got[:3], table[:, :W], got[3]), (*want[:4], [want[4]]), ("cu", "slots", "lens", "table", "head")):
        np.testing.assert_array_equal(a.cpu().numpy(), b, err_msg=name)
    np.testing.assert_array_equal(table[:, W:].cpu().numpy(), wide[:, W:])
    # the same call again writes the same
    again = gpu_lib.attn_tables(ints(cached), ints(new), table[:, :W], ints(free), ints([head]), P, room)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_tables_most_requests(gpu_lib):
    N, P, W = 8192, 16, 3
    rng = np.random.default_rng(5)
    cached, new = rng.integers(0, 30, N), rng.integers(0, 12, N)
    free, table = rng.permutation(20000), rng.integers(0, 20000, (N, W)).astype(np.int32)
    t = ints(table)
    room = int(new.sum()) + 5
    got = gpu_lib.attn_tables(ints(cached), ints(new), t, ints(free), None, P, room)
    want = ref.attn_tables(cached, new, table, free, 0, P, room)
    for a, b in zip((*got[:3], t, got[3]), (*want[:4], [want[4]])):
        np.testing.assert_array_equal(a.cpu().numpy(), b)


# ---------------------------------------------------------------- store

def make_cache(seed, pages, HKV, P, pad=0):
    """Codes of every kind but NaN, scales of several sizes; the pages `pad` bytes apart."""
    rng = np.random.default_rng(seed)
    codes = [rng.integers(0, 256, (pages, HKV * P * D + pad)).astype(np.uint8) for _ in "kv"]
    codes = [np.where((c & 127) == 127, c ^ 1, c).astype(np.uint8) for c in codes]
    scales = [2.0 ** rng.integers(-9, 2, (pages, HKV)) for _ in "kv"]
    flat = [torch.from_numpy(c).to(DEV) for c in codes]
    gpu = [f.view(E4M3)[:, :HKV * P * D].unflatten(1, (HKV, P, D)) for f in flat]
    return gpu + [torch.tensor(s, dtype=torch.float32, device=DEV) for s in scales], flat


def codes_of(c):
    return c.contiguous().view(torch.uint8).cpu().numpy()


def check_store(kda, k, v, slots, cache):
    before = [codes_of(cache[0]), codes_of(cache[1]), f64(cache[2]), f64(cache[3])]
    kda.attn_cache_store(k, v, *cache, ints(slots))
    for x, c, s, i in ((k, before[0], before[2], 0), (v, before[1], before[3], 1)):
        want, scale = ref.attn_cache_store(f64(x), c, s, slots)
        got = codes_of(cache[i])
        nan = (want & 127) == 127
        np.testing.assert_array_equal(f64(cache[2 + i]), scale)
        np.testing.assert_array_equal((got & 127) == 127, nan)
        np.testing.assert_array_equal(got[~nan], want[~nan])


def run_slots(page, P, start, n):
    return [page * P + start + i for i in range(n)]


@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("HKV", [1, 3])
def test_store_runs(gpu_lib, P, HKV):
    """Whole pages, parts of pages, single tokens, tokens that are not stored."""
    cache, _ = make_cache(P, 9, HKV, P)
    slots = run_slots(3, P, 0, P) + run_slots(7, P, 0, P // 2 + 1) + [-1, -5, 9 * P, 2 ** 31 - 1] + run_slots(0, P, 5, 3)
    slots += run_slots(5, P, P - 1, 1) + run_slots(4, P, 0, 1) + run_slots(8, P, 2, P - 2) + [-1] + run_slots(1, P, 1, 1)
    T = len(slots)
    gain = torch.exp2(torch.randint(-12, 9, (T, HKV, 1), generator=torch.Generator().manual_seed(P)).float())
    k, v = ((rand(P + i, T, HKV, D).float() * gain).bfloat16().to(DEV) for i in (1, 2))
    check_store(gpu_lib, k, v, slots, cache)
    # the next tokens of pages that are begun, small and then large: only the large ones move what is there
    for gain, seed in ((2.0 ** -20, 5), (2.0 ** 14, 6)):
        slots = run_slots(7, P, P // 2 + 1, 2) + run_slots(0, P, 8, 1) + run_slots(4, P, 1, 1)
        k, v = (rand(seed + 10 * i, 4, HKV, D, scale=gain).to(DEV) for i in (1, 2))
        check_store(gpu_lib, k, v, slots, cache)


def test_store_every_value(gpu_lib):
    """All 2^16 bf16 values, under the scales that rows of one binade each, and mixed rows, get."""
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    ordered = every.reshape(512, 1, D)
    mixed = every[torch.randperm(65536, generator=torch.Generator().manual_seed(1))].reshape(512, 1, D)
    cache, _ = make_cache(70, 64, 1, 16)
    check_store(gpu_lib, ordered.to(DEV), mixed.to(DEV), list(range(512)), cache)           # whole pages
    singles = [16 * i for i in range(64)]
    for part in range(8):                                                                   # one token a page
        check_store(gpu_lib, ordered[64 * part:64 * part + 64].to(DEV), mixed[64 * part:64 * part + 64].to(DEV), singles, cache)


def test_store_zero_and_padding(gpu_lib):
    """Zeros get the least scale; bytes between pages stay."""
    cache, flat = make_cache(71, 5, 2, 16, pad=48)
    before = [f.clone() for f in flat]
    z = torch.zeros(20, 2, D, dtype=torch.bfloat16, device=DEV)
    check_store(gpu_lib, z, z, run_slots(2, 16, 0, 16) + run_slots(4, 16, 0, 4), cache)
    assert (cache[2][2] == 2.0 ** -64).all()
    for a, b in zip(flat, before):
        assert torch.equal(a[:, 2 * 16 * D:], b[:, 2 * 16 * D:])
    # a page begun with zeros takes ordinary tokens afterwards
    k, v = rand(72, 1, 2, D).to(DEV), rand(73, 1, 2, D).to(DEV)
    check_store(gpu_lib, k, v, [4 * 16 + 4], cache)


def test_store_rows_of_a_projection(gpu_lib):
    row = rand(74, 50, 7 * D + 8).to(DEV)
    k, v = row[:, 8:8 + 3 * D].unflatten(1, (3, D)), row[:, 8 + 4 * D:].unflatten(1, (3, D))
    assert k.data_ptr() % 16 == 0
    cache, _ = make_cache(75, 4, 3, 32)
    check_store(gpu_lib, k, v, list(range(30, 80)), cache)


# ---------------------------------------------------------------- decode

def check_decode(o, lse, q, cache, table, lens, scale=None):
    codes = [codes_of(c) for c in cache[:2]]
    want, wl, o_abs = ref.attn_decode(f64(q), *codes, f64(cache[2]), f64(cache[3]), np.asarray(table), lens, scale)
    keys = np.nan_to_num(ref.e4m3_table()[codes[0]], nan=0.0) * np.nan_to_num(f64(cache[2]))[..., None, None]
    ez = eps(f64(q), keys, max(max(lens), 1), D ** -0.5 if scale is None else scale)
    check(o, want, ((U + 2.1 * ez) * o_abs + U * np.abs(want)) * 1.01 + 1e-30, "o")
    seen = np.isfinite(wl)
    assert np.array_equal(np.isneginf(f64(lse)), ~seen)
    check(lse[torch.from_numpy(seen)], wl[seen], ez + 2.0 ** -21 * (1 + np.abs(wl[seen])), "lse")


def usual_cache(seed, pages, HKV, P):
    """Codes of normal values with steps of about a hundredth, as a store makes them; NaN in a few unused places."""
    g = torch.Generator().manual_seed(seed)
    codes = [(torch.randn(pages, HKV, P, D, generator=g) * 64).clamp(-448, 448).to(E4M3).to(DEV) for _ in "kv"]
    return codes + [torch.exp2(torch.randint(-7, -5, (pages, HKV), generator=g).float()).to(DEV) for _ in "kv"]


def tables_for(lens, P, spare=2, seed=0):
    held = [-(-n // P) for n in lens]
    ids = np.random.default_rng(seed).permutation(sum(held) + spare)
    W = max(max(held), 1) + 1
    table, at = np.full((len(lens), W), -1), 0
    for row, n in zip(table, held):
        row[:n] = ids[at:at + n]
        at += n
    return table, sum(held) + spare


DECODE = [  # lengths, queries, HQ, HKV, page size
    ([1], 1, 1, 1, 16), ([15, 16, 17], 1, 4, 2, 16), ([63, 64, 65, 1], 1, 8, 2, 64), ([0, 5, 0], 1, 2, 1, 32),
    ([300], 1, 16, 1, 16),                       # one row tile, full
    ([300, 7], 1, 17, 1, 32),                    # 17 rows: two matrix tiles
    ([130, 2, 1, 64], 4, 8, 1, 64),              # 32 rows, queries before the first token
    ([200, 33], 7, 5, 1, 128),                   # 35 rows: two row tiles
    ([257, 100], 3, 48, 2, 256),                 # 72 rows
    ([1000, 1, 513, 64, 2000], 1, 8, 4, 64), ([2500], 2, 4, 2, 16), ([70] * 90, 1, 2, 2, 16),
]


@pytest.mark.parametrize("lens,Q,HQ,HKV,P", DECODE)
def test_decode(gpu_lib, lens, Q, HQ, HKV, P):
    table, pages = tables_for(lens, P)
    cache = usual_cache(len(lens), pages, HKV, P)
    q = rand(3, len(lens), Q, HQ, D).to(DEV)
    ws = torch.full((gpu_lib.attn_decode_workspace_size(len(lens), Q, HQ, HKV),), 255, dtype=torch.uint8, device=DEV)
    o, lse = gpu_lib.attn_decode(q, *cache, ints(table), ints(lens), workspace=ws)
    check_decode(o, lse, q, cache, table, lens)
    again, _ = gpu_lib.attn_decode(q, *cache, ints(table), ints(lens))
    assert torch.equal(o, again)


@pytest.mark.parametrize("Q", [1, 3])
def test_decode_reads_no_further(gpu_lib, Q):
    """NaN behind the end of the last page, in pages and scales that no sequence has, and in table entries past the end."""
    lens, P = [5, 16, 100, 47, 0, 129], 64
    table, pages = tables_for(lens, P, spare=3, seed=4)
    cache = usual_cache(8, pages, 2, P)
    q = rand(9, len(lens), Q, 4, D).to(DEV)
    o, lse = gpu_lib.attn_decode(q, *cache, ints(table), ints(lens))
    used = {int(p): min(n - i * P, P) for n, row in zip(lens, table) for i, p in enumerate(row[:-(-n // P)])}
    for c in cache[:2]:
        raw = c.view(torch.uint8)
        for p in range(pages):
            raw[p, :, used.get(p, 0):] = 0x7f
    for s in cache[2:]:
        for p in set(range(pages)) - set(used):
            s[p] = float("nan")
    junk = np.array(table)
    for n, row in zip(lens, junk):
        row[-(-n // P):] = [2 ** 31 - 1, -9, pages, 0][:len(row) - -(-n // P)] + [-1] * max(0, len(row) - -(-n // P) - 4)
    o2, lse2 = gpu_lib.attn_decode(q, *cache, ints(junk), ints(lens))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    check_decode(o2, lse2, q, cache, table, lens)


@pytest.mark.parametrize("cache_at", [0, 1])
def test_decode_nan_where_it_is_seen(gpu_lib, cache_at):
    """One NaN code (whole rows of them: all scores of some waves' pieces) reaches the rows that see it, and no others."""
    lens, P = [300, 5000, 64], 64
    table, pages = tables_for(lens, P, seed=5)
    cache = usual_cache(10, pages, 2, P)
    q = rand(11, 3, 1, 8, D).to(DEV)
    o, _ = gpu_lib.attn_decode(q, *cache, ints(table), ints(lens))
    raw = cache[cache_at].view(torch.uint8)
    raw[int(table[0, 1]), 0, 3, 9] = 0x7f
    for page in table[1, 10:40]:
        raw[int(page), 1] = 0xff
    got, lse = gpu_lib.attn_decode(q, *cache, ints(table), ints(lens))
    assert torch.equal(got[2], o[2]) and torch.equal(got[0, :, 4:], o[0, :, 4:]) and torch.equal(got[1, :, :4], o[1, :, :4])
    assert got[1, :, 4:].isnan().all()
    if cache_at == 0:
        assert got[0, :, :4].isnan().all() and lse[0, :, :4].isnan().all() and lse[1, :, 4:].isnan().all()
    else:
        assert got[0, :, :4, 9].isnan().all() and torch.equal(got[0, :, :4, :9], o[0, :, :4, :9])


@pytest.mark.parametrize("Q,HQ", [(2, 2), (5, 8), (7, 10), (70, 4)])
def test_decode_later_nan_does_not_reach_earlier_queries(gpu_lib, Q, HQ):
    """A NaN among the newest values: the queries before it are as if it were not there, the others hold it."""
    lens, P = [6, 64, 130, 300, 2 * Q], 16
    table, pages = tables_for(lens, P, seed=14)
    cache = usual_cache(40, pages, 2, P)
    q = rand(41, len(lens), Q, HQ, D).to(DEV)
    codes = [codes_of(c) for c in cache[:2]]
    want, wl, o_abs = ref.attn_decode(f64(q), *codes, f64(cache[2]), f64(cache[3]), table, lens)
    keys = ref.e4m3_table()[codes[0]] * f64(cache[2])[..., None, None]
    tol = ((U + 2.1 * eps(f64(q), keys, max(lens))) * o_abs + U * np.abs(want)) * 1.01 + 1e-30
    raw = cache[1].view(torch.uint8)
    bad = np.zeros((len(lens), Q), bool)
    for n, length in enumerate(lens):
        at = max(length - 1 - n % Q, 0)                        # a token that the last queries see, from this one on
        raw[int(table[n, at // P]), 1, at % P, 5 + n] = 0x7f
        bad[n] = np.arange(Q) >= Q - length + at
    o, lse = gpu_lib.attn_decode(q, *cache, ints(table), ints(lens))
    got = f64(o)
    clean = np.ones(got.shape, bool)
    for n in range(len(lens)):
        clean[n, bad[n], HQ // 2:, 5 + n] = False
    assert np.isnan(got[~clean]).all() and np.isfinite(got[clean]).all()
    assert (np.abs(got - want)[clean] <= tol[clean]).all()
    seen = np.isfinite(wl)
    assert np.array_equal(np.isneginf(f64(lse)), ~seen)


def test_decode_pages_missing(gpu_lib):
    """A page outside the cache holds no tokens; lengths beyond the table and below 0 are cut."""
    lens, P = [100, 64, 40, 500, -3], 16
    table, pages = tables_for([100, 64, 40, 64, 0], P, seed=6)
    table = table[:, :7]
    table[0, 2], table[0, 6], table[1, :4], table[2, 0] = pages, -2, -1, 2 ** 30
    cache = usual_cache(11, pages, 1, P)
    q = rand(12, 5, 2, 3, D).to(DEV)
    o, lse = gpu_lib.attn_decode(q, *cache, ints(table), ints(lens))
    check_decode(o, lse, q, cache, table, lens)
    assert (o[1] == 0).all() and (o[4] == 0).all()


def test_decode_peaked_and_scaled(gpu_lib):
    """Scales far apart from page to page: the running maximum moves, weights vanish."""
    lens, P = [700, 350], 32
    table, pages = tables_for(lens, P, seed=7)
    cache = usual_cache(13, pages, 2, P)
    cache[2].copy_(torch.exp2(torch.randint(-12, -1, (pages, 2), generator=torch.Generator().manual_seed(1)).float()))
    cache[3].copy_(torch.exp2(torch.randint(-30, 30, (pages, 2), generator=torch.Generator().manual_seed(2)).float()))
    q = rand(14, 2, 1, 8, D).to(DEV)
    for scale in (0.01, 0.3):
        o, lse = gpu_lib.attn_decode(q, *cache, ints(table), ints(lens), scale=scale)
        check_decode(o, lse, q, cache, table, lens, scale)


@pytest.mark.parametrize("longest", [1, 3, 40])
def test_decode_scores_are_float32(gpu_lib, longest):
    """Few tokens: lse is a score or a few, and shows what the products' sum lost.

    A score is a float32 sum of 128 exact products, then two products and, with the
    softmax, a few roundings more: at most 140, each off by at most 2^-24 of the
    sum of magnitudes A and independent of the others, so that over thousands of
    rows the errors' root mean square stays below sqrt(140) 2^-24 A.
    """
    rng = np.random.default_rng(longest)
    lens, P, HKV, HQ = [int(x) for x in rng.integers(1, longest + 1, 40)], 16, 4, 32
    table, pages = tables_for(lens, P, seed=longest)
    cache = usual_cache(30 + longest, pages, HKV, P)
    q = rand(31, len(lens), 1, HQ, D).to(DEV)
    _, lse = gpu_lib.attn_decode(q, *cache, ints(table), ints(lens))
    codes = [codes_of(c) for c in cache[:2]]
    _, want, _ = ref.attn_decode(f64(q), *codes, f64(cache[2]), f64(cache[3]), table, lens)
    keys = np.abs(ref.e4m3_table()[codes[0]]) * f64(cache[2])[..., None, None]
    size = np.zeros_like(want)                     # A: the largest of the row's scores' magnitudes
    for n, length in enumerate(lens):
        k = keys[table[n, :-(-length // P)]].transpose(1, 0, 2, 3).reshape(HKV, -1, D)[:, :length]
        for h in range(HQ):
            size[n, 0, h] = (k[h * HKV // HQ] @ np.abs(f64(q))[n, 0, h]).max() * D ** -0.5
    off = np.sqrt(np.mean((f64(lse) - want) ** 2) / np.mean(size ** 2))
    assert off <= np.sqrt(140) * 2.0 ** -24, off


def test_decode_many_waves(gpu_lib):
    """More 64-token units than waves: pieces of several units that begin and end inside sequences."""
    rng = np.random.default_rng(3)
    lens, P = [int(x) for x in rng.integers(1, 3000, 40)] + [0, 70000], 64
    table, pages = tables_for(lens, P, seed=8)
    cache = usual_cache(15, pages, 2, P)
    q = rand(16, len(lens), 1, 6, D).to(DEV)
    o, lse = gpu_lib.attn_decode(q, *cache, ints(table), ints(lens))
    check_decode(o, lse, q, cache, table, lens)


def test_decode_strides_and_far_pages(gpu_lib):
    """Queries in wider rows, a wider table, pages 2^28 bytes apart (offsets past 2^32)."""
    lens, P, far = [90, 300], 16, 1 << 28
    table, pages = tables_for(lens, P, seed=9)
    cache = usual_cache(17, pages, 1, P)
    row = rand(18, 2, 3, 5 * D).to(DEV)
    q = row[..., D:].unflatten(-1, (4, D))
    o, lse = gpu_lib.attn_decode(q.contiguous(), *cache, ints(table), ints(lens))
    check_decode(o, lse, q, cache, table, lens)
    big = torch.empty((pages - 1) * far + 2 * P * D, dtype=torch.uint8, device=DEV)
    spread = [big.as_strided((pages, 1, P, D), (far, P * D, D, 1), i * P * D).view(E4M3) for i in (0, 1)]
    for a, b in zip(spread, cache):
        a.view(torch.uint8).copy_(b.view(torch.uint8))
    wide = ints(np.concatenate([table, np.full((2, 5), 10 ** 9)], 1))
    o2, lse2 = gpu_lib.attn_decode(q, *spread, *cache[2:], wide[:, :table.shape[1]], ints(lens))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # and the store reaches them
    k, v = rand(19, 4, 1, D).to(DEV), rand(20, 4, 1, D).to(DEV)
    slots = ints(run_slots(pages - 1, P, 0, 4))
    gpu_lib.attn_cache_store(k, v, *cache, slots)
    gpu_lib.attn_cache_store(k, v, *spread, *[s.clone() for s in cache[2:]], slots)
    for a, b in zip(spread, cache):
        assert torch.equal(a.view(torch.uint8).cpu(), b.view(torch.uint8).cpu())


# ---------------------------------------------------------------- together

def server(kda, seed, N, HQ, HKV, P, W, prompts, steps, step):
    """Prompts through prefill into the cache, then `steps` decode steps, each checked."""
    total = N * W
    cache = [torch.full((total, HKV, P, D), 0x7f, dtype=torch.uint8, device=DEV).view(E4M3) for _ in "kv"]
    cache += [torch.full((total, HKV), float("nan"), device=DEV) for _ in "kv"]
    free = ints(np.random.default_rng(seed).permutation(total))
    table = ints(np.full((N, W), -1))
    held = ints([0] * N)
    cu, slots, lens, head = kda.attn_tables(held, ints(prompts), table, free, None, P, sum(prompts) + 3)
    T = sum(prompts) + 3
    q, k, v = rand(seed, 1, T, HQ, D).to(DEV), rand(seed + 1, 1, T, HKV, D).to(DEV), rand(seed + 2, 1, T, HKV, D).to(DEV)
    o, lse = kda.attn_prefill(q, k, v, cu_seqlens=cu)
    check_prompt(o, lse, q, k, v, cu.tolist())
    kda.attn_cache_store(k[0], v[0], *cache, slots)
    want = ref.attn_cache_store(f64(k[0]), np.full((total, HKV, P, D), 0x7f, np.uint8), np.ones((total, HKV)), slots.tolist())
    np.testing.assert_array_equal(codes_of(cache[0]), want[0])
    return step(cache, free, table, lens, head, steps)


def test_prompts_then_steps(gpu_lib):
    kda, N, HQ, HKV, P = gpu_lib, 5, 8, 2, 16
    prompts = [1, 40, 16, 77, 15]

    def step(cache, free, table, lens, head, steps):
        for i in range(steps):
            new = ints([1, 2, 1, 0, 2])
            cu, slots, lens, head = kda.attn_tables(lens, new, table, free, head, P, 8)
            k, v = (rand(100 + 3 * i + j, 8, HKV, D, scale=1 + i).to(DEV) for j in (0, 1))
            check_store(kda, k, v, slots.tolist(), cache)
            q = rand(102 + 3 * i, N, 2, HQ, D).to(DEV)
            o, lse = kda.attn_decode(q, *cache, table, lens)
            check_decode(o, lse, q, cache, table.cpu().numpy(), lens.tolist())
        assert lens.tolist() == [1 + steps, 40 + 2 * steps, 16 + steps, 77, 15 + 2 * steps]

    server(kda, 1, N, HQ, HKV, P, 7, prompts, 9, step)


def test_captured_steps(gpu_lib):
    """One decode step (tables, store, decode) captured once, replayed as the requests grow; two graphs share the workspace."""
    kda, N, HQ, HKV, P = gpu_lib, 5, 8, 2, 16
    prompts = [1, 40, 16, 77, 15]

    def step(cache, free, table, lens, head, steps):
        one = ints([1] * N)
        s = {n: torch.zeros(m, dtype=torch.int32, device=DEV) for n, m in
             (("cu_seqlens", N + 1), ("slots", N + 2), ("kv_lens", N), ("next_head", 1))}
        k, v = torch.zeros(N + 2, HKV, D, dtype=torch.bfloat16, device=DEV), torch.zeros(N + 2, HKV, D, dtype=torch.bfloat16, device=DEV)
        q, out, lse = torch.zeros(N, 1, HQ, D, dtype=torch.bfloat16, device=DEV), None, torch.zeros(N, 1, HQ, device=DEV)
        out = torch.zeros_like(q)
        ws = torch.full((kda.attn_decode_workspace_size(N, 1, HQ, HKV),), 255, dtype=torch.uint8, device=DEV)

        def one_step():
            kda.attn_tables(lens, one, table, free, head, P, N + 2, **s)
            kda.attn_cache_store(k, v, *cache, s["slots"])
            kda.attn_decode(q, *cache, table, s["kv_lens"], out=out, lse=lse, workspace=ws)
            lens.copy_(s["kv_lens"])
            head.copy_(s["next_head"])

        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                one_step()
            graphs.append(g)
        shadow = [c.clone() for c in cache[:2]] + [c.clone() for c in cache[2:]]
        stable, slens, shead = table.clone(), lens.clone(), head.clone()
        for i in range(steps):
            for j, t in enumerate((k, v, q)):
                t.copy_(rand(200 + 3 * i + j, *t.shape))
            graphs[i % 2].replay()
            torch.cuda.synchronize()
            cu, slots, slens, shead = kda.attn_tables(slens, one, stable, free, shead, P, N + 2)
            kda.attn_cache_store(k, v, *shadow, slots)
            o, z = kda.attn_decode(q, *shadow, stable, slens)
            torch.cuda.synchronize()
            assert torch.equal(lens, slens) and torch.equal(table, stable) and torch.equal(head, shead)
            for a, b in zip(cache[:2], shadow):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
            assert torch.equal(out, o) and torch.equal(lse, z), i
        check_decode(out, lse, q, cache, table.cpu().numpy(), lens.tolist())

    server(kda, 7, N, HQ, HKV, P, 7, prompts, 20, step)


def test_decode_continues_the_prompt(gpu_lib):
    """The last row of a prompt, once by prefill and once from the cache: as near as 8-bit keys and values are.

    With codes off by 2^-4 of their size at most (and half the smallest step),
    scores move by dz <= scale sum|q||k| 2^-4, weights by exp(2 dz) - 1, values by
    2^-4: a loose bound, but one that a wrong page or head would pass by far.
    """
    T, HQ, HKV, P = 200, 4, 2, 64
    q, k, v = rand(1, 1, T, HQ, D, scale=0.2).to(DEV), rand(2, 1, T, HKV, D, scale=0.2).to(DEV), rand(3, 1, T, HKV, D).to(DEV)
    o, _ = gpu_lib.attn_prefill(q, k, v)
    cache = [torch.zeros(8, HKV, P, D, dtype=torch.uint8, device=DEV).view(E4M3) for _ in "kv"] + [torch.ones(8, HKV, device=DEV) for _ in "kv"]
    table = ints([[-1] * 4])
    _, slots, lens, _ = gpu_lib.attn_tables(ints([0]), ints([T]), table, ints([6, 2, 7, 1]), None, P, T)
    gpu_lib.attn_cache_store(k[0], v[0], *cache, slots)
    d, _ = gpu_lib.attn_decode(q[:, -1:], *cache, table, lens)
    qq, kk = np.abs(f64(q))[0, -1], np.abs(f64(k))[0]
    dz = D ** -0.5 * np.einsum("hd,thd->ht", qq, np.repeat(kk, HQ // HKV, 1)).max() * 2.0 ** -4
    _, _, o_abs = ref.attn_prefill(f64(q), f64(k), f64(v))
    tol = (np.exp(2 * dz) * (1 + 2.0 ** -4) - 1 + 4 * U) * o_abs[0, -1]
    check(d[0, 0], f64(o)[0, -1], tol, "cache against prompt")


@pytest.mark.parametrize("lens,Q,HQ,HKV", [([700, 90, 0], 100, 2, 1), ([1300], 1024, 2, 2), ([1024, 1], 1024, 1, 1)])
def test_decode_many_queries(gpu_lib, lens, Q, HQ, HKV):
    """A stretch of a prompt against the cache: many row tiles, up to the most queries a call takes."""
    table, pages = tables_for(lens, 64, seed=21)
    cache = usual_cache(60, pages, HKV, 64)
    q = rand(61, len(lens), Q, HQ, D).to(DEV)
    o, lse = gpu_lib.attn_decode(q, *cache, ints(table), ints(lens))
    check_decode(o, lse, q, cache, table, lens)


def test_decode_two_at_once(gpu_lib):
    """Calls on two streams, each with a workspace of its own, do not meet."""
    calls = []
    for i, (lens, HQ, HKV) in enumerate((([900, 3000, 40], 8, 2), ([5000, 1], 20, 4))):
        table, pages = tables_for(lens, 32, seed=30 + i)
        cache = usual_cache(70 + i, pages, HKV, 32)
        q = rand(72 + i, len(lens), 2, HQ, D).to(DEV)
        calls.append((q, *cache, ints(table), ints(lens)))
    alone = [gpu_lib.attn_decode(*c) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[], []]
    for _ in range(8):
        for i, (c, s) in enumerate(zip(calls, streams)):
            with torch.cuda.stream(s):
                got[i].append(gpu_lib.attn_decode(*c))
    torch.cuda.synchronize()
    for want, results in zip(alone, got):
        for o, lse in results:
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


class Wide:
    """The library with page tables that could hold much more than they do: decode then cuts all sequences into equal
    pieces, where short tables give each (sequence, head) a workgroup."""

    def __init__(self, lib):
        self.lib = lib

    def __getattr__(self, name):
        return getattr(self.lib, name)

    def attn_decode(self, q, k_cache, v_cache, k_scale, v_scale, table, lens, **kw):
        pad = table.new_full((table.shape[0], 5000 // k_cache.shape[2]), -1)
        return self.lib.attn_decode(q, k_cache, v_cache, k_scale, v_scale, torch.cat([table, pad], 1), lens, **kw)


@pytest.mark.parametrize("lens,Q,HQ,HKV,P", DECODE)
def test_decode_wide_tables(gpu_lib, lens, Q, HQ, HKV, P):
    test_decode(Wide(gpu_lib), lens, Q, HQ, HKV, P)


@pytest.mark.parametrize("Q,HQ", [(1, 2), (2, 2), (5, 8), (70, 4)])
def test_decode_wide_tables_masks(gpu_lib, Q, HQ):
    """What the tests above mask, cut among waves."""
    wide = Wide(gpu_lib)
    test_decode_reads_no_further(wide, min(Q, 3))
    if Q > 1:
        test_decode_later_nan_does_not_reach_earlier_queries(wide, Q, HQ)
    test_decode_peaked_and_scaled(wide)


@pytest.mark.parametrize("N,longest", [(1, 1536), (1, 1537), (64, 1000), (65, 1000), (24, 4096), (23, 4096), (24, 4097)])
def test_decode_alone_and_cut(gpu_lib, N, longest):
    """Both sides of the rule that says which of the two it is (64-token pages, 8 heads)."""
    rng = np.random.default_rng(N + longest)
    lens = [longest] + [int(x) for x in rng.integers(0, longest + 1, N - 1)]
    table, pages = tables_for(lens, 64, spare=0, seed=22)
    table = table[:, :-(-longest // 64)]
    cache = usual_cache(62, pages, 8, 64)
    q = rand(63, N, 1, 8, D).to(DEV)
    o, lse = gpu_lib.attn_decode(q, *cache, ints(table), ints(lens))
    check_decode(o, lse, q, cache, table, lens)


def test_steps_with_wide_tables(gpu_lib):
    test_prompts_then_steps(Wide(gpu_lib))
    test_captured_steps(Wide(gpu_lib))


@pytest.mark.parametrize("HQ", [2, 20])
def test_decode_large_caches(gpu_lib, HQ):
    """A cache of more than a hundred megabytes, which is loaded another way: the same bits as from a small one."""
    lens, P, HKV = [3000, 1, 0, 9000], 64, 1
    table, pages = tables_for(lens, P, seed=23)
    table = np.concatenate([table, np.full((len(lens), 3000), -1)], 1)
    cache = usual_cache(64, pages, HKV, P)
    q = rand(65, len(lens), 1, HQ, D).to(DEV)
    o, lse = gpu_lib.attn_decode(q, *cache, ints(table), ints(lens))
    check_decode(o, lse, q, cache, table, lens)
    more = 7000 - pages
    large = [torch.cat([c.view(torch.uint8), torch.full((more, HKV, P, D), 0x7f, dtype=torch.uint8, device=DEV)]).view(E4M3)
             for c in cache[:2]] + [torch.cat([s, s.new_full((more, HKV), float("nan"))]) for s in cache[2:]]
    o2, lse2 = gpu_lib.attn_decode(q, *large, ints(table), ints(lens))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("lens,HQ,HKV,wide", [([40], 1, 1, False), ([900, 3], 16, 1, False), ([900, 3], 8, 2, True)])
def test_decode_few_rows_are_nearly_float32(gpu_lib, lens, HQ, HKV, wide):
    """Up to 16 rows carry weights as two bf16 terms, which leave 2^-16 of each: the result's own rounding is all there is."""
    table, pages = tables_for(lens, 64, seed=24)
    cache = usual_cache(66, pages, HKV, 64)
    q = rand(67, len(lens), 1, HQ, D).to(DEV)
    o, _ = (Wide(gpu_lib) if wide else gpu_lib).attn_decode(q, *cache, ints(table), ints(lens))
    codes = [codes_of(c) for c in cache[:2]]
    want, _, o_abs = ref.attn_decode(f64(q), *codes, f64(cache[2]), f64(cache[3]), table, lens)
    ez = eps(f64(q), ref.e4m3_table()[codes[0]] * f64(cache[2])[..., None, None], max(lens))
    check(o, want, ((2.0 ** -16 + 2.1 * ez) * o_abs + U * np.abs(want)) * 1.01 + 1e-30, "o")
