"""kda_attn_prefill and kda_attn_backward against the float64 oracle.

Tolerances, element by element.  u = 2^-8 is half a bfloat16 step.  With
ez = 2 * 128 * 2^-24 * scale * max|q| max|k| + 2^-20 (two float32 sums of 128
products, and the exponential), a weight is off by ew = u + 2 ez + n 2^-23
relative: rounded once to bfloat16, scores off by ez in numerator and sum, n
terms added.  So |o - ref| <= ew * sum_j P_ij |v_j|, and u |o| for its own
rounding; lse is off by ez and the float32 sum.  The gradients' bounds are sums
of the same kind that the oracle returns (`moved`).
"""

import numpy as np
import pytest
import torch

import oracle.attention as ref
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -8
D = 128


def rand(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).bfloat16()


def f64(t):
    return t.detach().double().cpu().numpy()


def eps(q, k, n, scale=D ** -0.5):
    with np.errstate(invalid="ignore"):
        size = np.nanmax(np.linalg.norm(q, axis=-1), initial=0) * np.nanmax(np.linalg.norm(k, axis=-1), initial=0)
    return 2 * 128 * 2.0 ** -24 * scale * size + 2.0 ** -20 + n * 2.0 ** -24


def check(got, want, tol, what):
    got = f64(got)
    keep = ~np.isnan(want)
    assert np.isfinite(got[keep]).all(), what
    over = np.abs(got - want)[keep] - np.broadcast_to(tol, want.shape)[keep]
    worst = float((np.abs(got - want)[keep] / np.maximum(np.broadcast_to(tol, want.shape)[keep], 1e-300)).max(initial=0))
    say(f"{what}: {worst:.2f} of its tolerance")
    assert (over <= 0).all(), f"{what}: {worst:.3f} times its tolerance"


def check_prompt(o, lse, q, k, v, cu=None, scale=None):
    q, k, v = f64(q), f64(k), f64(v)
    want, wl, o_abs = ref.attn_prefill(q, k, v, cu, scale)
    ez = eps(q, k, q.shape[1], D ** -0.5 if scale is None else scale)
    ew = U + 2.1 * ez
    check(o, want, (ew * o_abs + U * np.abs(want)) * 1.01 + 1e-30, "o")
    check(lse, wl, ez + 2.0 ** -22 * (1 + np.abs(wl)), "lse")


def check_grads(grads, q, k, v, d_out, cu=None, scale=None, rounded=True):
    q, k, v, d_out = f64(q), f64(k), f64(v), f64(d_out)
    want, moved = ref.attn_backward(q, k, v, d_out, cu, scale)
    ew = U + 4.2 * eps(q, k, q.shape[1], D ** -0.5 if scale is None else scale)
    for got, w, m, name in zip(grads, want, moved, ("dq", "dk", "dv")):
        # dS (or P) rounded, and o and its weights behind delta
        check(got, w, (2 * ew * m + (U if rounded else 0.0) * np.abs(w)) * 1.01 + 1e-30, name)


CASES = [  # B, T, HQ, HKV, offsets
    (1, 1, 1, 1, None), (1, 2, 4, 2, None), (2, 31, 5, 1, None), (1, 32, 2, 2, None), (1, 33, 6, 2, None),
    (3, 63, 4, 4, None), (1, 64, 8, 1, None), (1, 65, 3, 3, None), (2, 127, 4, 1, None), (1, 128, 2, 1, None),
    (1, 129, 10, 2, None), (1, 200, 4, 2, None), (1, 517, 6, 2, None),
    (1, 300, 4, 2, [0, 1, 2, 2, 130, 130, 258, 300]),        # one token, none, a tile and more
    (1, 257, 6, 3, [0, 0, 257, 257]),
    (1, 190, 2, 1, [5, 70, 133, 134]),                       # tokens before the first and behind the last sequence
    (1, 200, 4, 2, list(range(0, 201, 2))),                  # 100 sequences of two
    (1, 77, 1, 1, [0] * 70 + [77]),                          # 69 empty ones first
]


def case(B, T, HQ, HKV, cu, seed=1):
    q, k, v, up = (rand(seed + i, B, T, h, D).to(DEV) for i, h in enumerate((HQ, HKV, HKV, HQ)))
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
    return q, k, v, up, c


@pytest.mark.parametrize("B,T,HQ,HKV,cu", CASES)
def test_prompt_and_gradients(gpu_lib, B, T, HQ, HKV, cu):
    q, k, v, up, c = case(B, T, HQ, HKV, cu)
    o = torch.full((B, T, HQ, D), 7.5, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((B, HQ, T), 7.5, device=DEV)
    gpu_lib.attn_prefill(q, k, v, cu_seqlens=c, out=o, lse=lse)
    check_prompt(o, lse, q, k, v, cu)
    if cu is not None:                                       # tokens outside the sequences stay as they were
        out = torch.ones(T, dtype=torch.bool)
        out[cu[0]:cu[-1]] = False
        assert (o[0, out] == 7.5).all() and (lse[0][:, out] == 7.5).all()
    grads = gpu_lib.attn_backward(q, k, v, o, lse, up, cu_seqlens=c)
    check_grads(grads, q, k, v, up, cu)
    wide = gpu_lib.attn_backward(q, k, v, o, lse, up, cu_seqlens=c, grad_dtype="float32")
    check_grads(wide, q, k, v, up, cu, rounded=False)
    inside = slice(None) if cu is None else slice(cu[0], cu[-1])
    for a, b in zip(grads, wide):
        assert torch.equal(a[:, inside], b[:, inside].bfloat16())


def test_outside_rows_keep_their_gradients(gpu_lib):
    """Rows outside the sequences: neither read (they hold NaN) nor written."""
    kda, T, HQ, HKV = gpu_lib, 300, 8, 2
    q, k, v, up, c = case(1, T, HQ, HKV, [3, 100, 230], seed=9)
    for x in (q, k, v, up):
        x[:, :3] = float("nan")
        x[:, 230:] = float("nan")
    o, lse = kda.attn_prefill(q, k, v, cu_seqlens=c)
    lib = kda.load()
    for dtype, code in ((torch.bfloat16, 1), (torch.float32, 0)):
        grads = [torch.full((1, T, h, D), 3.0, dtype=dtype, device=DEV) for h in (HQ, HKV, HKV)]
        size = kda.attn_backward_workspace_size(1, T, HQ, HKV, 2)
        ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)      # NaN, read as floats
        P = [x.data_ptr() for x in (q, k, v, o, lse, up, c, *grads, ws)]
        assert lib.kda_attn_backward(*P[:3], HQ * D, HKV * D, HKV * D, *P[3:7], 2, 1, T, HQ, HKV, D, D ** -0.5,
                                     *P[7:10], code, P[10], size, torch.cuda.current_stream().cuda_stream) == 0
        for x in grads:
            assert (x[0, :3] == 3).all() and (x[0, 230:] == 3).all()
        check_grads(grads, q, k, v, up, [3, 100, 230], rounded=code == 1)


def test_shared_workgroups_sum_in_order(gpu_lib):
    """Few key tiles and a long walk: several workgroups share one (float32 parts), the same bits every time."""
    q, k, v, up, _ = case(1, 1500, 8, 1, None, seed=20)
    kda = gpu_lib
    assert kda.attn_backward_workspace_size(1, 1500, 8, 1) > 2 * 1500 * 8 * 4 + 64
    o, lse = kda.attn_prefill(q, k, v)
    check_prompt(o, lse, q, k, v)
    grads = kda.attn_backward(q, k, v, o, lse, up)
    check_grads(grads, q, k, v, up)
    for _ in range(2):
        again = kda.attn_backward(q, k, v, o, lse, up)
        assert all(torch.equal(a, b) for a, b in zip(grads, again))
        a, b = kda.attn_prefill(q, k, v)
        assert torch.equal(a, o) and torch.equal(b, lse)


@pytest.mark.parametrize("scale", [0.02, 1.0])
def test_scale_and_large_scores(gpu_lib, scale):
    """Peaked rows: the running maximum moves far, tile after tile."""
    q, k, v, up, _ = case(1, 333, 4, 2, None, seed=30)
    k = (k.float() * torch.linspace(0.1, 4, 333, device=DEV)[None, :, None, None]).bfloat16()
    o, lse = gpu_lib.attn_prefill(q, k, v, scale=scale)
    check_prompt(o, lse, q, k, v, scale=scale)
    check_grads(gpu_lib.attn_backward(q, k, v, o, lse, up, scale=scale), q, k, v, up, scale=scale)


def test_rows_of_a_projection(gpu_lib):
    """q, k and v as slices of one row per token, with padding: the same bits as dense ones."""
    HQ, HKV, B, T = 4, 2, 2, 150
    row = rand(40, B, T, (HQ + 2 * HKV) * D + 64).to(DEV)
    q, k, v = (row[..., a * D:b * D].unflatten(-1, (-1, D)) for a, b in ((0, 4), (4, 6), (6, 8)))
    up = rand(41, B, T, HQ, D).to(DEV)
    o, lse = gpu_lib.attn_prefill(q, k, v)
    grads = gpu_lib.attn_backward(q, k, v, o, lse, up)
    dense = [x.contiguous() for x in (q, k, v)]
    o2, lse2 = gpu_lib.attn_prefill(*dense)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for a, b in zip(grads, gpu_lib.attn_backward(*dense, o, lse, up)):
        assert torch.equal(a, b)
    check_prompt(o, lse, q, k, v)


def test_offsets_past_32_bits(gpu_lib):
    """Rows 2^23 elements apart: the tokens' offsets pass 2^32 bytes."""
    T, S = 300, 1 << 23
    big = torch.empty(T * S, dtype=torch.bfloat16, device=DEV)
    q, k, v, up, _ = case(1, T, 2, 1, None, seed=50)
    views = []
    for i, x in enumerate((q, k, v)):
        y = big.as_strided((1, T, x.shape[2], D), (T * S, S, D, 1), i * 1024)
        y.copy_(x)
        views.append(y)
    o, lse = gpu_lib.attn_prefill(*views)
    o2, lse2 = gpu_lib.attn_prefill(q, k, v)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for a, b in zip(gpu_lib.attn_backward(*views, o, lse, up), gpu_lib.attn_backward(q, k, v, o, lse, up)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_sequences_do_not_meet(gpu_lib, bad):
    """What is not finite in one sequence stays in it."""
    cu = [0, 70, 130, 260]
    q, k, v, up, c = case(1, 260, 4, 2, cu, seed=60)
    o, lse = gpu_lib.attn_prefill(q, k, v, cu_seqlens=c)
    grads = gpu_lib.attn_backward(q, k, v, o, lse, up, cu_seqlens=c)
    for x in (q, k, v):
        x[0, 70:130] = bad
    o2, lse2 = gpu_lib.attn_prefill(q, k, v, cu_seqlens=c)
    for a, b in ((o, o2), (lse.transpose(1, 2), lse2.transpose(1, 2)),
                 *zip(grads, gpu_lib.attn_backward(q, k, v, o2, lse2, up, cu_seqlens=c))):
        assert torch.equal(a[:, :70], b[:, :70]) and torch.equal(a[:, 130:], b[:, 130:])
    # and a key's or query's in the rows that see it
    q, k, v, up, c = case(1, 260, 4, 2, cu, seed=60)
    k[0, 40] = bad
    o3, _ = gpu_lib.attn_prefill(q, k, v, cu_seqlens=c)
    assert torch.equal(o[:, :40], o3[:, :40]) and not torch.equal(o[:, 40:70], o3[:, 40:70])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [[0], [1, 5], [31], [32, 40], [63], [64], [95, 96], [150, 299]])
def test_later_values_do_not_reach_earlier_rows(gpu_lib, at, bad):
    """Infinities and NaN in v (or k) of a token: the rows before it are as if it were not there."""
    q, k, v, up, _ = case(1, 300, 4, 2, None, seed=65)
    want, wl, o_abs = ref.attn_prefill(f64(q), f64(k), f64(v))
    ew = U + 2.1 * eps(f64(q), f64(k), 300)
    v2 = v.clone()
    for j in at:
        v2[0, j, 1, 7 * j % D] = bad
    o, lse = gpu_lib.attn_prefill(q, k, v2)
    seen = np.arange(300) >= at[0]
    clean = np.ones((300, 4, D), bool)
    for j in at:
        clean[j:, 2:, 7 * j % D] = False
    got = f64(o)[0]
    assert np.isfinite(got[clean]).all() and not np.isfinite(got[~clean]).any()
    tol = (ew * o_abs + U * np.abs(want)) * 1.01
    assert (np.abs(got - want[0])[clean] <= tol[0][clean]).all()
    check(lse, wl, eps(f64(q), f64(k), 300) + 2.0 ** -22 * (1 + np.abs(wl)), "lse")
    k2 = k.clone()
    k2[0, at[0], 1, 3] = bad
    o2, _ = gpu_lib.attn_prefill(q, k2, v)
    assert (np.abs(f64(o2) - want)[:, ~seen] <= tol[:, ~seen]).all() and torch.equal(o2[:, :, :2], gpu_lib.attn_prefill(q, k, v)[0][:, :, :2])


def test_another_stream(gpu_lib):
    q, k, v, up, _ = case(1, 400, 4, 2, None, seed=70)
    o, lse = gpu_lib.attn_prefill(q, k, v)
    grads = gpu_lib.attn_backward(q, k, v, o, lse, up)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        q2 = q * 1                                           # made on that stream just before
        o2, lse2 = gpu_lib.attn_prefill(q2, k, v)
        grads2 = gpu_lib.attn_backward(q2, k, v, o2, lse2, up)
    side.synchronize()
    assert torch.equal(o, o2) and all(torch.equal(a, b) for a, b in zip(grads, grads2))


def test_graph_replay(gpu_lib):
    """Forward and backward in one captured graph, replayed on new inputs and lengths between eager work."""
    kda, T, HQ, HKV = gpu_lib, 260, 8, 1
    q, k, v, up, c = case(1, T, HQ, HKV, [0, 100, 260], seed=80)
    bufs = dict(out=torch.empty(1, T, HQ, D, dtype=torch.bfloat16, device=DEV), lse=torch.empty(1, HQ, T, device=DEV))
    ws = torch.empty(kda.attn_backward_workspace_size(1, T, HQ, HKV, 2), dtype=torch.uint8, device=DEV)
    kda.attn_prefill(q, k, v, cu_seqlens=c, **bufs)
    kda.attn_backward(q, k, v, bufs["out"], bufs["lse"], up, cu_seqlens=c, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.attn_prefill(q, k, v, cu_seqlens=c, **bufs)
        grads = kda.attn_backward(q, k, v, bufs["out"], bufs["lse"], up, cu_seqlens=c, workspace=ws)
    for r, cu in enumerate(([0, 100, 260], [0, 1, 260], [0, 0, 260], [0, 259, 260])):
        for x, y in zip((q, k, v, up), case(1, T, HQ, HKV, cu, seed=81 + 10 * r)):
            x.copy_(y)
        c.copy_(torch.tensor(cu, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        o, lse = kda.attn_prefill(q, k, v, cu_seqlens=c)
        want = kda.attn_backward(q, k, v, o, lse, up, cu_seqlens=c)
        torch.cuda.synchronize()
        assert torch.equal(o, bufs["out"]) and torch.equal(lse, bufs["lse"])
        assert all(torch.equal(a, b) for a, b in zip(grads, want)), r


def test_gradients_are_the_differences(gpu_lib):
    """sum(o * d_out) moves along a direction as the gradients say, measured in float64 from the kernel's inputs."""
    q, k, v, up, _ = case(1, 90, 4, 2, None, seed=90)
    o, lse = gpu_lib.attn_prefill(q, k, v)
    grads = [f64(g) for g in gpu_lib.attn_backward(q, k, v, o, lse, up, grad_dtype="float32")]
    x, u = [f64(t) for t in (q, k, v)], f64(up)
    rng = np.random.default_rng(0)
    _, moved = ref.attn_backward(*x, u)
    for i in range(3):
        d = rng.standard_normal(x[i].shape)
        y = [[a + s * 1e-5 * d if j == i else a for j, a in enumerate(x)] for s in (1, -1)]
        slope = ((ref.attn_prefill(*y[0])[0] - ref.attn_prefill(*y[1])[0]) * u).sum() / 2e-5
        tol = (2 * (U + 4.2 * eps(x[0], x[1], 90)) * moved[i] * np.abs(d)).sum()
        assert abs((grads[i] * d).sum() - slope) <= tol


LONG = [  # walks long enough for two sets of waves on a row tile's keys
    (1, 512, 2, 1, None), (2, 600, 4, 2, None), (1, 1216, 4, 1, [0, 513, 1153]), (1, 1800, 2, 2, [64, 64, 1777]),
    (1, 2053, 17, 17, None),                                 # more workgroups than compute units
]


@pytest.mark.parametrize("B,T,HQ,HKV,cu", LONG)
def test_long_walks(gpu_lib, B, T, HQ, HKV, cu):
    q, k, v, up, c = case(B, T, HQ, HKV, cu, seed=200)
    o, lse = gpu_lib.attn_prefill(q, k, v, cu_seqlens=c)
    grads = gpu_lib.attn_backward(q, k, v, o, lse, up, cu_seqlens=c)
    if HQ == HKV:                                            # each head apart: the first and the last will do
        heads = [0, HQ - 1]
        q, k, v, up, o = (x[:, :, heads] for x in (q, k, v, up, o))
        lse, grads = lse[:, heads], [g[:, :, heads] for g in grads]
    check_prompt(o, lse, q, k, v, cu)
    check_grads(grads, q, k, v, up, cu)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [[3], [255], [256, 300], [448, 639], [639]])
def test_later_values_in_long_walks(gpu_lib, at, bad):
    """As above, with the keys of a row tile dealt to two sets of waves."""
    T = 640
    q, k, v, up, _ = case(1, T, 2, 2, None, seed=230)
    clean, lse = gpu_lib.attn_prefill(q, k, v)
    v2 = v.clone()
    seen = torch.zeros(T, 2, D, dtype=torch.bool, device=DEV)
    for j in at:
        v2[0, j, 1, 7 * j % D] = bad
        seen[j:, 1, 7 * j % D] = True
    o, lse2 = gpu_lib.attn_prefill(q, k, v2)
    assert torch.equal(lse, lse2) and not torch.isfinite(o[0][seen]).any()
    want, _, o_abs = ref.attn_prefill(f64(q), f64(k), f64(v))
    tol = ((U + 2.1 * eps(f64(q), f64(k), T)) * o_abs + U * np.abs(want)) * 1.01
    keep = (~seen).cpu().numpy()
    assert (np.abs(f64(o) - want)[0][keep] <= tol[0][keep]).all()
    check_prompt(clean, lse, q, k, v)


FEW = [(1, 3, 2, 2, None), (4, 2, 8, 2, None), (1, 64, 6, 2, None), (1, 30, 2, 1, [0, 3, 6, 6, 7, 30]), (1, 120, 2, 2, None)]


@pytest.mark.parametrize("B,T,HQ,HKV,cu", FEW)
def test_few_gradients_are_nearly_float32(gpu_lib, B, T, HQ, HKV, cu):
    """Small calls carry weights and score gradients as two bf16 terms, which leave 2^-16 of each."""
    q, k, v, up, c = case(B, T, HQ, HKV, cu, seed=250)
    o, lse = gpu_lib.attn_prefill(q, k, v, cu_seqlens=c)
    grads = gpu_lib.attn_backward(q, k, v, o, lse, up, cu_seqlens=c, grad_dtype="float32")
    want, moved = ref.attn_backward(f64(q), f64(k), f64(v), f64(up), cu)
    ew = 2.0 ** -16 + 4.2 * eps(f64(q), f64(k), T) + 2 * 128 * 2.0 ** -24
    for got, w, m, name in zip(grads, want, moved, ("dq", "dk", "dv")):
        check(got, w, 2 * ew * m * 1.01 + 1e-30, name)
