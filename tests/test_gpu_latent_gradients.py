"""kda_latent_backward against the float64 oracle by norms of errors (latent_norms.py), in every form that sizes choose:
one or two terms of weights, a key tile for one workgroup or several.
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


CASES = [  # B, T, K, H, offsets of queries, of keys, two terms, several workgroups for a key tile
    (1, 32, 32, 2, None, None, True, False), (1, 129, 129, 9, None, None, True, False),
    (1, 517, 517, 3, None, None, False, True), (1, 450, 450, 70, None, None, False, False),
    (1, 450, 450, 2, None, None, True, True), (1, 700, 700, 1, None, None, True, True),
    (2, 400, 640, 2, None, None, False, True), (2, 450, 500, 1, None, None, True, True),
    (1, 100, 333, 2, None, None, True, False),
    (1, 1500, 1500, 2, None, None, False, True), (2, 700, 1000, 3, None, None, False, True),
    (1, 1100, 1100, 24, None, None, False, True),
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
