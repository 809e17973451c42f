"""kda_latent_backward against the float64 oracle by norms of errors (latent_norms.py), in every form that sizes choose:
one or two terms of weights, a key tile for one workgroup or several, packed or not, with rows outside the sequences.
The same calls' outputs and elements are held to test_gpu_latent_prompt.py's bounds."""

import numpy as np
import pytest
import torch

import latent_norms
import oracle.latent as ref
from gpu_util import say
from test_gpu_attn_prompt import f64
from test_gpu_latent_prompt import D, DEV, DQ, S, case, check_prompt, ints

pytestmark = pytest.mark.gpu


def check_norms(x, got, cu, cu_kv, rounded, two, b=0):
    y = [f64(t)[b] for t in x]
    want = [w[0] for w in ref.latent_backward(*[a[None] for a in y], cu, cu_kv)[0]]
    bound = latent_norms.bounds(*y, want, cu, cu_kv, rounded=rounded, u=2.0 ** (-16 if two else -8))
    worst = latent_norms.worst([f64(g)[b] for g in got], want, bound, cu, cu_kv)
    say(f"{worst:.2f} of the norm's bound")
    assert worst <= 1


def ends(T, N, lead, tail):
    """N sequences of unlike lengths between rows that belong to none."""
    at = np.linspace(0, 1, N + 1) ** 1.3
    return [int(x) for x in np.round(lead + at * (T - lead - tail))]


CASES = [  # B, T, K, H, offsets of queries, of keys, two terms, several workgroups for a key tile
    (1, 32, 32, 2, None, None, True, False), (1, 129, 129, 9, None, None, True, False),
    (1, 517, 517, 3, None, None, False, True), (1, 450, 450, 70, None, None, False, False),
    (1, 450, 450, 2, None, None, True, True), (1, 700, 700, 1, None, None, True, True),
    (2, 400, 640, 2, None, None, False, True), (2, 450, 500, 1, None, None, True, True),
    (1, 100, 333, 2, None, None, True, False),
    (1, 1500, 1500, 2, None, None, False, True), (2, 700, 1000, 3, None, None, False, True),
    (1, 1100, 1100, 24, None, None, False, True),
    # packed: few heads and long samples; many heads; two terms; empty samples, parts over longer caches, other orders
    (1, 1300, 1300, 2, [5, 640, 1291], None, False, True),
    (1, 1300, 1400, 2, [0, 0, 1290], [7, 100, 1400], False, True),
    (1, 2000, 2000, 32, ends(2000, 3, 3, 9), None, False, False),
    (1, 2000, 2300, 24, [2, 700, 700, 1991], [5, 900, 950, 2291], False, False),
    (1, 900, 900, 1, [0, 430, 880], None, True, True), (1, 880, 1000, 1, [20, 460, 870], [1, 520, 1000], True, True),
    (1, 500, 560, 2, [3, 3, 170, 490], [5, 60, 200, 551], True, False),
    (1, 1600, 1700, 4, [800, 1590, 0, 790], [850, 1690, 10, 840], False, True),
    (1, 1500, 1500, 5, ends(1500, 70, 4, 6), None, True, False),
]


@pytest.mark.parametrize("B,T,K,H,cu,cu_kv,two,parts", CASES)
def test_gradients_in_norm(gpu_lib, B, T, K, H, cu, cu_kv, two, parts):
    *x, up = case(B, T, K, H, seed=200)
    N = 0 if cu is None else len(cu) - 1
    # (which form it is: what is tuned anew shows here)
    assert (B * T * H * (K // N if N else K) <= 1 << 19) == two
    statistics = 2 * ((B * T * H + 3) // 4 * 4) * 4
    assert (gpu_lib.latent_backward_workspace_size(B, T, K, H, N) > statistics + B * K * H * S * 4) == parts
    c = dict(cu_seqlens=ints(cu), cu_seqlens_kv=ints(cu_kv))
    o = torch.full((B, T, H, D), 7.5, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((B, H, T), 7.5, device=DEV)
    gpu_lib.latent_prefill(*x, **c, out=o, lse=lse)
    check_prompt(o, lse, *x, cu, cu_kv)
    rows, keys = torch.zeros(T, dtype=torch.bool), torch.zeros(K, dtype=torch.bool)
    for lo, hi, klo, khi in ref.pairs(cu, cu_kv, T, K):
        rows[lo:hi] = keys[klo:khi] = True
    assert (o[:, ~rows] == 7.5).all() and (lse[:, :, ~rows] == 7.5).all()
    made = {}
    for dtype, name in ((torch.bfloat16, "input"), (torch.float32, "float32")):
        g = {n: torch.full(shape, 3.0, dtype=dtype, device=DEV)
             for n, shape in dict(dq=(B, T, H, DQ), d_kv=(B, K, H, 2 * D), dk_shared=(B, K, S)).items()}
        ws = torch.full((gpu_lib.latent_backward_workspace_size(B, T, K, H, N),), 255, dtype=torch.uint8, device=DEV)
        grads = gpu_lib.latent_backward(*x, o, lse, up, **c, **g, grad_dtype=name, workspace=ws)
        for b in range(B):
            check_norms((*x, up), grads, cu, cu_kv, name == "input", two, b)
        assert (g["dq"][:, ~rows] == 3).all() and (g["d_kv"][:, ~keys] == 3).all()
        assert (g["dk_shared"][:, ~keys] == 3).all()
        made[name] = g
    for n, wide in made["float32"].items():
        inside = rows if n == "dq" else keys
        assert torch.equal(made["input"][n][:, inside], wide[:, inside].bfloat16())


@pytest.mark.parametrize("T,K,H", [(90, 90, 4), (130, 300, 3), (300, 300, 8)])
def test_differences_along_the_gradient(gpu_lib, T, K, H):
    """sum(o * d_out) in float64 along the gradient's own direction, where its slope is the gradient's squared norm."""
    *x, up = case(1, T, K, H, seed=210)
    o, lse = gpu_lib.latent_prefill(*x)
    grads = [f64(g)[0] for g in gpu_lib.latent_backward(*x, o, lse, up, grad_dtype="float32")]
    y, u = [f64(t) for t in x], f64(up)
    want = ref.latent_backward(*y, u)[0]
    bound = latent_norms.bounds(*[a[0] for a in y], u[0], [w[0] for w in want], rounded=False)
    for i, d in enumerate(want):
        step = 1e-4 / np.abs(d).max()
        z = [[a + t * step * d if j == i else a for j, a in enumerate(y)] for t in (1, -1)]
        slope = ((ref.latent_prefill(*z[0])[0] - ref.latent_prefill(*z[1])[0]) * u).sum() / (2 * step)
        room = np.sqrt(sum(b * b for b in bound[i].values())) * np.linalg.norm(d)
        assert room < 0.02 * slope
        # the differences' own error: terms of the third order, about step^2 of the slope, and float64's rounding
        assert abs((grads[i] * d[0]).sum() - slope) <= room + 1e-5 * slope


@pytest.mark.parametrize("B,T,K,H,cu,cu_kv,two", [
    (1, 1300, 1300, 2, [5, 640, 1291], None, False), (1, 1300, 1400, 2, [0, 0, 1290], [7, 100, 1400], False),
    (1, 880, 1000, 1, [20, 460, 870], [1, 520, 1000], True), (1, 450, 450, 2, None, None, True)])
def test_parts_beside_nan(gpu_lib, B, T, K, H, cu, cu_kv, two):
    """Several workgroups for a key tile: NaN in rows outside the sequences and in the workspace, the same bits each
    time."""
    *x, up = case(B, T, K, H, seed=220)
    c = dict(cu_seqlens=ints(cu), cu_seqlens_kv=ints(cu_kv))
    o, lse = gpu_lib.latent_prefill(*x, **c)
    want = gpu_lib.latent_backward(*x, o, lse, up, **c)
    rows, keys = torch.zeros(T, dtype=torch.bool), torch.zeros(K, dtype=torch.bool)
    for lo, hi, klo, khi in ref.pairs(cu, cu_kv, T, K):
        rows[lo:hi] = keys[klo:khi] = True
    for t in (x[0], o, up):
        t[:, ~rows] = float("nan")
    for t in x[1:]:
        t[:, ~keys] = float("nan")
    lse[:, :, ~rows] = float("nan")
    N = 0 if cu is None else len(cu) - 1
    ws = torch.full((gpu_lib.latent_backward_workspace_size(B, T, K, H, N),), 255, dtype=torch.uint8, device=DEV)
    got = gpu_lib.latent_backward(*x, o, lse, up, **c, workspace=ws)
    for i, (a, b) in enumerate(zip(want, got)):
        inside = rows if i == 0 else keys
        assert torch.equal(a[:, inside], b[:, inside])


@pytest.mark.parametrize("H,cu", [(2, [0, 2]), (2, [9, 1291]), (2, [5, 640, 1291])])
def test_packed_rows_of_two_sets_of_waves(gpu_lib, H, cu):
    """Few long samples: the forward's second set of waves, in packed sequences."""
    q, k, s, v, _ = case(1, 1300, 1300, H, seed=230)
    o, lse = gpu_lib.latent_prefill(q, k, s, v, cu_seqlens=ints(cu))
    full = [t.double() for t in (q, k, s, v)]
    for lo, hi in zip(cu, cu[1:]):
        part = [f64(t[:, lo:hi]) for t in full]
        check_prompt(o[:, lo:hi], lse[:, :, lo:hi], *(torch.from_numpy(p) for p in part))
