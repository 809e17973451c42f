"""kda_latent_prefill and kda_latent_backward against the float64 oracle.

Tolerances, element by element, are those of test_gpu_attn_prompt.py with products
of 192 terms.  u = 2^-8 is half a bfloat16 step.  With ez = 2 * 192 * 2^-24 * scale *
max|q| max|[k s]| + 2^-20 (two float32 sums of 192 products, and the exponential), a
weight is off by ew = u + 2 ez + n 2^-23 relative: rounded once to bfloat16, scores
off by ez in numerator and sum, n terms added.  So |o - ref| <= ew * sum_j P_ij |v_j|,
and u |o| for its own rounding; lse is off by ez and the float32 sum.  The gradients'
bounds are sums of the same kind that the oracle returns (`moved`).
"""

import numpy as np
import pytest
import torch

import oracle.latent as ref
from test_gpu_attn_prompt import U, check, f64, rand

pytestmark = pytest.mark.gpu
DEV = "cuda"
D, S, DQ = 128, 64, 192


def ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)


def eps(q, k, s, scale):
    with np.errstate(invalid="ignore"):
        key = np.nanmax(np.linalg.norm(k, axis=-1), initial=0) ** 2 + np.nanmax(np.linalg.norm(s, axis=-1), initial=0) ** 2
        size = np.nanmax(np.linalg.norm(q, axis=-1), initial=0) * key ** 0.5
    return 2 * DQ * 2.0 ** -24 * scale * size + 2.0 ** -20 + k.shape[1] * 2.0 ** -24


def case(B, T, K, H, seed=1):
    return [rand(seed + i, *shape).to(DEV)
            for i, shape in enumerate(((B, T, H, DQ), (B, K, H, D), (B, K, S), (B, K, H, D), (B, T, H, D)))]


def check_prompt(o, lse, q, k, s, v, cu=None, cu_kv=None, scale=ref.SCALE):
    x = [f64(t) for t in (q, k, s, v)]
    want, wl, o_abs = ref.latent_prefill(*x, cu, cu_kv, scale)
    ez = eps(*x[:3], scale)
    check(o, want, ((U + 2.1 * ez) * o_abs + U * np.abs(want)) * 1.01 + 1e-30, "o")
    none = np.isneginf(wl)
    assert (f64(lse)[none] == -np.inf).all() and (f64(o).transpose(0, 2, 1, 3)[none] == 0).all()
    check(lse, np.where(none, np.nan, wl), ez + 2.0 ** -22 * (1 + np.abs(np.where(none, 0, wl))), "lse")


def check_grads(grads, q, k, s, v, up, cu=None, cu_kv=None, scale=ref.SCALE, rounded=True):
    x = [f64(t) for t in (q, k, s, v, up)]
    want, moved = ref.latent_backward(*x, cu, cu_kv, scale)
    ew = U + 4.2 * eps(*x[:3], scale)
    for got, w, m, name in zip(grads, want, moved, ("dq", "dk", "ds", "dv")):
        # dS (or P) rounded, and o and its weights behind delta
        check(got, w, (2 * ew * m + (U if rounded else 0.0) * np.abs(w)) * 1.01 + 1e-30, name)


CASES = [  # B, T, K, H, offsets of queries, of keys
    (1, 1, 1, 1, None, None), (1, 2, 2, 3, None, None), (2, 31, 31, 5, None, None), (1, 32, 32, 2, None, None),
    (3, 63, 63, 4, None, None), (1, 65, 65, 3, None, None), (2, 127, 127, 1, None, None), (1, 129, 129, 9, None, None),
    (1, 517, 517, 3, None, None), (1, 450, 450, 70, None, None),
    (1, 1, 200, 2, None, None), (2, 3, 66, 3, None, None), (1, 33, 97, 2, None, None), (1, 100, 333, 2, None, None),
    (1, 130, 700, 1, None, None),
    (1, 5, 3, 2, None, None), (2, 200, 70, 2, None, None), (1, 300, 1, 1, None, None), (1, 9, 0, 2, None, None),
    (1, 0, 7, 2, None, None),
    (1, 300, 300, 4, [0, 1, 2, 2, 130, 130, 258, 300], None),   # one token, none, a tile and more
    (1, 190, 190, 2, [5, 70, 133, 134], None),                  # tokens before the first and behind the last sequence
    (1, 200, 200, 3, list(range(0, 201, 2)), None),             # 100 sequences of two
    (1, 260, 900, 2, [0, 1, 100, 260], [0, 500, 600, 900]),     # parts of longer prompts
    (1, 260, 300, 3, [3, 10, 150, 200], [2, 2, 60, 299]),       # without keys, more queries than keys
    (1, 70, 400, 2, [0, 0, 70, 70], [0, 150, 390, 400]),        # keys without queries
    (1, 140, 280, 1, list(range(0, 141, 2)), list(range(0, 281, 4))),
    (1, 60, 120, 1, [40, 60, 20, 40], [80, 120, 30, 75]),       # in another order (the middle one is empty)
]


@pytest.mark.parametrize("B,T,K,H,cu,cu_kv", CASES)
def test_prompt_and_gradients(gpu_lib, B, T, K, H, cu, cu_kv):
    *x, up = case(B, T, K, H)
    c = dict(cu_seqlens=ints(cu), cu_seqlens_kv=ints(cu_kv))
    o = torch.full((B, T, H, D), 7.5, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((B, H, T), 7.5, device=DEV)
    gpu_lib.latent_prefill(*x, **c, out=o, lse=lse)
    check_prompt(o, lse, *x, cu, cu_kv)
    rows, keys = torch.zeros(T, dtype=torch.bool), torch.zeros(K, dtype=torch.bool)
    for lo, hi, klo, khi in ref.pairs(cu, cu_kv, T, K):
        rows[lo:hi] = keys[klo:khi] = True
    assert (o[:, ~rows] == 7.5).all() and (lse[:, :, ~rows] == 7.5).all()   # outside the sequences all stays as it was
    for dtype, name in ((torch.bfloat16, "input"), (torch.float32, "float32")):
        made = dict(dq=(B, T, H, DQ), d_kv=(B, K, H, 2 * D), dk_shared=(B, K, S))
        made = {n: torch.full(shape, 3.0, dtype=dtype, device=DEV) for n, shape in made.items()}
        grads = gpu_lib.latent_backward(*x, o, lse, up, **c, **made, grad_dtype=name)
        check_grads(grads, *x, up, cu, cu_kv, rounded=dtype != torch.float32)
        assert (made["dq"][:, ~rows] == 3).all() and (made["d_kv"][:, ~keys] == 3).all()
        assert (made["dk_shared"][:, ~keys] == 3).all()
        if name == "input":
            first = made
    for n, wide in made.items():
        inside = rows if n == "dq" else keys
        assert torch.equal(first[n][:, inside], wide[:, inside].bfloat16())


def test_outside_rows_are_not_read(gpu_lib):
    """NaN outside the sequences, and in the workspace."""
    cu, cu_kv = [3, 100, 230], [5, 150, 350]
    q, k, s, v, up = case(1, 260, 370, 3, seed=9)
    for x in (q, up):
        x[:, :3] = x[:, 230:] = float("nan")
    for x in (k, s, v):
        x[:, :5] = x[:, 350:] = float("nan")
    c = dict(cu_seqlens=ints(cu), cu_seqlens_kv=ints(cu_kv))
    o, lse = gpu_lib.latent_prefill(q, k, s, v, **c)
    check_prompt(o, lse, q, k, s, v, cu, cu_kv)
    ws = torch.full((gpu_lib.latent_backward_workspace_size(1, 260, 370, 3, 2),), 255, dtype=torch.uint8, device=DEV)
    o[:, :3] = o[:, 230:] = float("nan")
    check_grads(gpu_lib.latent_backward(q, k, s, v, o, lse, up, **c, workspace=ws), q, k, s, v, up, cu, cu_kv)


@pytest.mark.parametrize("T,K", [(1500, 1500), (600, 2000)])
def test_shared_workgroups_sum_in_order(gpu_lib, T, K):
    """Few key tiles and a long walk: several workgroups share one (float32 parts), the same bits every time."""
    kda, H = gpu_lib, 2
    *x, up = case(1, T, K, H, seed=20)
    assert kda.latent_backward_workspace_size(1, T, K, H) > T * H * 8 + K * H * 256 + 64
    o, lse = kda.latent_prefill(*x)
    check_prompt(o, lse, *x)
    grads = kda.latent_backward(*x, o, lse, up)
    check_grads(grads, *x, up)
    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(grads, kda.latent_backward(*x, o, lse, up)))
        a, b = kda.latent_prefill(*x)
        assert torch.equal(a, o) and torch.equal(b, lse)


def test_long_prompt(gpu_lib):
    """Long enough for two sets of waves on a row tile, and for a walk of many tiles behind the others' queries."""
    *x, _ = case(1, 2100, 2100, 2, seed=25)
    o, lse = gpu_lib.latent_prefill(*x)
    check_prompt(o, lse, *x)
    a, b = gpu_lib.latent_prefill(x[0][:, 1999:], *x[1:])
    check_prompt(a, b, x[0][:, 1999:], *x[1:])


@pytest.mark.parametrize("scale", [0.02, 1.0])
def test_scale_and_large_scores(gpu_lib, scale):
    """Peaked rows: the running maximum moves far, tile after tile."""
    q, k, s, v, up = case(1, 333, 400, 3, seed=30)
    gain = torch.linspace(0.1, 4, 400, device=DEV)[None, :, None]
    k, s = (k.float() * gain[..., None]).bfloat16(), (s.float() * gain).bfloat16()
    o, lse = gpu_lib.latent_prefill(q, k, s, v, scale=scale)
    check_prompt(o, lse, q, k, s, v, scale=scale)
    check_grads(gpu_lib.latent_backward(q, k, s, v, o, lse, up, scale=scale), q, k, s, v, up, scale=scale)


def same(kda, views, dense, up):
    o, lse = kda.latent_prefill(*views)
    a, b = kda.latent_prefill(*dense)
    assert torch.equal(o, a) and torch.equal(lse, b)
    for x, y in zip(kda.latent_backward(*views, o, lse, up), kda.latent_backward(*dense, o, lse, up)):
        assert torch.equal(x, y)


def test_rows_of_projections(gpu_lib):
    """k and v as the halves of one projection's rows, the shared part behind a latent, q a slice of wider rows."""
    H, B, T = 3, 2, 150
    q = rand(40, B, T, H * DQ + 64).to(DEV)[..., 64:].unflatten(-1, (H, DQ))
    row, c = rand(41, B, T, H, 2 * D + 16).to(DEV), rand(42, B, T, 512 + S).to(DEV)
    k, v, s = row[..., :D], row[..., 16 + D:], c[..., 512:]
    up = rand(43, B, T, H, D).to(DEV)
    same(gpu_lib, (q, k, s, v), [x.contiguous() for x in (q, k, s, v)], up)


def test_heads_outermost(gpu_lib):
    H, T = 5, 140
    q, k, s, v, up = case(1, T, T, H, seed=45)
    outer = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v)]
    assert outer[0].stride(2) == T * D
    same(gpu_lib, (q, outer[0], s, outer[1]), (q, k, s, v), up)
    # one key and value for all heads: a head stride of zero, gradients head by head
    one = [x[:, :, :1].expand(-1, -1, H, -1) for x in (k, v)]
    same(gpu_lib, (q, one[0], s, one[1]), (q, one[0].contiguous(), s, one[1].contiguous()), up)


def test_offsets_past_32_bits(gpu_lib):
    """Rows 2^23 elements apart: the tokens' offsets pass 2^32 bytes."""
    T, L, H = 300, 1 << 23, 2
    big = torch.empty(T * L, dtype=torch.bfloat16, device=DEV)
    q, k, s, v, up = case(1, T, T, H, seed=50)
    views = []
    for i, x in enumerate((q, k, s, v)):
        stride = (T * L, L, x.shape[-1], 1) if x.dim() == 4 else (T * L, L, 1)
        y = big.as_strided(x.shape, stride, i * 1024)
        y.copy_(x)
        views.append(y)
    same(gpu_lib, views, (q, k, s, v), up)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_sequences_do_not_meet(gpu_lib, bad):
    """What is not finite in one sequence stays in it."""
    kda = gpu_lib
    cu, cu_kv = [0, 70, 130, 260], [0, 100, 190, 400]
    c = dict(cu_seqlens=ints(cu), cu_seqlens_kv=ints(cu_kv))
    q, k, s, v, up = case(1, 260, 400, 2, seed=60)
    o, lse = kda.latent_prefill(q, k, s, v, **c)
    grads = kda.latent_backward(q, k, s, v, o, lse, up, **c)
    q[0, 70:130] = bad
    for x in (k, s, v):
        x[0, 100:190] = bad
    o2, lse2 = kda.latent_prefill(q, k, s, v, **c)
    got = kda.latent_backward(q, k, s, v, o2, lse2, up, **c)
    pairs = [(o, o2, 70, 130), (lse.transpose(1, 2), lse2.transpose(1, 2), 70, 130), (grads[0], got[0], 70, 130)]
    for a, b, lo, hi in pairs + [(a, b, 100, 190) for a, b in zip(grads[1:], got[1:])]:
        assert torch.equal(a[:, :lo], b[:, :lo]) and torch.equal(a[:, hi:], b[:, hi:])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("T,K", [(130, 130), (100, 171), (97, 700), (2100, 2117)])
def test_later_tokens_do_not_reach_earlier_rows(gpu_lib, bad, T, K):
    """A key, shared part or value that is not finite: in the rows that see it, and in no other."""
    kda = gpu_lib
    *x, _ = case(1, T, K, 2, seed=61)
    want, wl, o_abs = ref.latent_prefill(*(f64(t) for t in x))
    ez = eps(*(f64(t) for t in x[:3]), ref.SCALE)
    tol = ((U + 2.1 * ez) * o_abs + U * np.abs(want)) * 1.01
    for token in (K - 1, K - 31, K - 64, K - T + 1, K - T // 2):
        first = token - (K - T)                              # the first row that sees it
        for which in (1, 2, 3):
            y = [t.clone() for t in x]
            y[which][0, token] = bad
            a, b = kda.latent_prefill(*y)
            # the rows before it as without it (their last bits follow what else is in their tile)
            check(a[:, :first], want[:, :first], tol[:, :first], "o")
            check(b[:, :, :first], wl[:, :, :first], ez + 2.0 ** -22 * (1 + np.abs(wl[:, :, :first])), "lse")
            if which == 3:
                assert not torch.isfinite(a[:, first:]).any()
                check(b, wl, ez + 2.0 ** -22 * (1 + np.abs(wl)), "lse")
            elif bad != bad:
                assert torch.isnan(a[:, first:]).all() and torch.isnan(b[:, :, first:]).all()


def test_scores_of_minus_infinity(gpu_lib):
    """Keys that overflow to -inf are masked: weights of zero, rows without another score give zeros and no gradient."""
    kda = gpu_lib
    q, k, s, v, up = case(1, 200, 200, 2, seed=62)
    q[..., 0], k[..., 0] = 2.0, 0.0
    k[:, :70, :, 0] = -3e38
    k[:, 150, :, 0] = -3e38
    o, lse = kda.latent_prefill(q, k, s, v, scale=1.0)
    assert (o[:, :70] == 0).all() and (lse[:, :, :70] == -float("inf")).all()
    grads = kda.latent_backward(q, k, s, v, o, lse, up, scale=1.0)
    assert all(torch.isfinite(g).all() for g in grads) and (grads[0][:, :70] == 0).all()
    assert all((g[:, :70] == 0).all() and (g[:, 150] == 0).all() for g in grads[1:])
    # the others as if those keys were not there: rows from 150 on see 149 - 70 + ... keys less
    keep = [i for i in range(200) if i >= 70 and i != 150]
    a, b = kda.latent_prefill(q[:, 151:], k[:, keep], s[:, keep], v[:, keep], scale=1.0)
    x = [f64(t) for t in (k[:, keep], s[:, keep])]
    ez = eps(f64(q), *x, 1.0)
    check(o[:, 151:], f64(a), 2 * (2 * U + 2.1 * ez) * float(v.float().abs().max()), "masked")
    check(lse[:, :, 151:], f64(b), 2 * ez + 2.0 ** -20 * (1 + f64(b).__abs__()), "masked lse")


def test_gradients_by_differences(gpu_lib):
    """A step along a direction changes sum(o * d_out) by the gradient's share of it: the gradients are of what the
    forward computes, in float64 of its definition, at inputs that bfloat16 holds."""
    T, K, H = 60, 90, 2
    *x, up = case(1, T, K, H, seed=70)
    o, lse = gpu_lib.latent_prefill(*x)
    grads = gpu_lib.latent_backward(*x, o, lse, up, grad_dtype="float32")
    y = [f64(t) for t in x]
    _, moved = ref.latent_backward(*y, f64(up))
    ew = U + 4.2 * eps(*y[:3], ref.SCALE)
    for which, (g, m) in enumerate(zip(grads, moved)):
        way = np.random.default_rng(which).choice([-1.0, 1.0], y[which].shape)
        value = []
        for step in (1e-5, -1e-5):
            z = list(y)
            z[which] = y[which] + step * way
            value.append((ref.latent_prefill(*z)[0] * f64(up)).sum())
        # each element of the gradient within its bound
        assert abs((value[0] - value[1]) / 2e-5 - (f64(g) * way).sum()) <= 2 * ew * m.sum() + 1e-6


def test_captured_on_a_side_stream(gpu_lib):
    """A forward and backward captured with their buffers, replayed on new inputs, between eager work."""
    kda = gpu_lib
    cu, cu_kv = [0, 50, 200], [0, 300, 520]
    *x, up = case(1, 200, 520, 3, seed=80)
    c = dict(cu_seqlens=ints(cu), cu_seqlens_kv=ints(cu_kv))
    ws = torch.empty(kda.latent_backward_workspace_size(1, 200, 520, 3, 2), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kda.latent_prefill(*x, **c)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = kda.latent_prefill(*x, **c)
        grads = kda.latent_backward(*x, o, lse, up, **c, workspace=ws)
    for seed in range(4):
        for t, new in zip((*x, up), case(1, 200, 520, 3, seed=90 + 10 * seed)):
            t.copy_(new)
        graph.replay()
        got = [t.clone() for t in (o, lse, *grads)]
        want = kda.latent_prefill(*x, **c)
        want = (*want, *kda.latent_backward(*x, *want, up, **c))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals(gpu_lib):
    kda = gpu_lib
    q, k, s, v, up = case(1, 20, 30, 2)
    o, lse = kda.latent_prefill(q, k, s, v)
    c, c3 = ints([0, 20]), ints([0, 10, 30])
    for args, kw, what in (
            ((q[..., :128], k, s, v), {}, "q must be"), ((q, k[..., :64], s, v), {}, "k must be"),
            ((q, k, s[:, :29], v), {}, "k_shared must be"), ((q, k, s, v[:, :, :1]), {}, "v must be"),
            ((q, k, s, v.transpose(1, 3).contiguous().transpose(1, 3)), {}, "last axis"),
            ((q.transpose(2, 3).contiguous().transpose(2, 3), k, s, v), {}, "compact"),
            ((q, k, s, v), dict(cu_seqlens_kv=c), "goes with"), ((q, k, s, v), dict(cu_seqlens=c), "is needed"),
            ((q, k, s, v), dict(cu_seqlens=c, cu_seqlens_kv=c3), "as many"),
            ((q, k, s, v), dict(cu_seqlens=c[:1], cu_seqlens_kv=c), "must be"),
            ((q, k, s, v), dict(out=o[:, :19]), "out must be")):
        with pytest.raises(ValueError, match=what):
            kda.latent_prefill(*args, **kw)
    two = [torch.cat((t, t)) for t in (q, k, s, v)]
    uneven = [t.as_strided(t.shape, (t.stride(0) - 8, *t.stride()[1:])) for t in two]
    for i, name in enumerate(("q", "k", "k_shared", "v")):
        with pytest.raises(ValueError, match=f"{name}: tokens must be evenly"):
            kda.latent_prefill(*two[:i], uneven[i], *two[i + 1:])
    with pytest.raises(ValueError, match="d_kv must be"):
        kda.latent_backward(q, k, s, v, o, lse, up, d_kv=q.new_empty(1, 30, 2, 128))
    with pytest.raises(TypeError, match="dq must be"):
        kda.latent_backward(q, k, s, v, o, lse, up, dq=q.new_empty(1, 20, 2, 192), grad_dtype="float32")
    with pytest.raises(kda.KDAError, match="orkspace"):
        kda.latent_backward(q, k, s, v, o, lse, up, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(kda.KDAError):
        kda.latent_prefill(q, k, s, v, scale=float("nan"))
