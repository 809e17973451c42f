"""kda_attn_backward against the float64 oracle by norms of errors (attn_norms.py),
which reject what elements' bounds let pass on long walks: a gradient of zero, a
missing delta, head or part."""

import numpy as np
import pytest
import torch

import attn_norms
import oracle.attention as ref
from gpu_util import say
from test_gpu_attn_offsets import mixed
from test_gpu_attn_prompt import D, DEV, U, case, eps, f64

pytestmark = pytest.mark.gpu


def check_norms(q, k, v, up, got, cu, rounded, b=0):
    x = [f64(t)[b] for t in (q, k, v, up)]
    want, _ = ref.attn_backward(*[a[None] for a in x], cu)
    want = [w[0] for w in want]
    u = U + 4.2 * eps(x[0], x[1], x[0].shape[0])
    bound = attn_norms.bounds(*x, want, cu, rounded=rounded, u=u)
    worst = attn_norms.worst([f64(g)[b] for g in got], want, bound, cu)
    say(f"{worst:.2f} of the norm's bound")
    assert worst <= 1


CASES = [  # B, T, HQ, HKV, offsets, whether several workgroups share a key tile
    (1, 90, 4, 2, None, False), (1, 129, 2, 2, None, False), (1, 517, 6, 2, None, True), (2, 600, 4, 2, None, True),
    (1, 700, 4, 1, [0, 130, 700], True), (1, 1500, 8, 1, None, True), (1, 1800, 2, 2, [64, 64, 1777], True),
    (1, 3000, 4, 1, mixed(70, 5, most=2990), True), (1, 3000, 2, 2, mixed(70, 6, most=2990, front=9), False),
]


@pytest.mark.parametrize("B,T,HQ,HKV,cu,parts", CASES)
def test_gradients_in_norm(gpu_lib, B, T, HQ, HKV, cu, parts):
    q, k, v, up, c = case(B, T, HQ, HKV, cu, seed=500)
    N = 0 if cu is None else len(cu) - 1
    assert (gpu_lib.attn_backward_workspace_size(B, T, HQ, HKV, N) > 2 * B * T * HQ * 4 + 32) == parts
    o, lse = gpu_lib.attn_prefill(q, k, v, cu_seqlens=c)
    for rounded in (True, False):
        grads = gpu_lib.attn_backward(q, k, v, o, lse, up, cu_seqlens=c, grad_dtype="input" if rounded else "float32")
        for b in range(B):
            check_norms(q, k, v, up, grads, cu, rounded, b)


@pytest.mark.parametrize("T,HQ,HKV", [(90, 4, 2), (300, 8, 1)])
def test_differences_along_the_gradient(gpu_lib, T, HQ, HKV):
    """sum(o * d_out) in float64 along the gradient's own direction, where its slope is the gradient's squared norm."""
    q, k, v, up, _ = case(1, T, HQ, HKV, None, seed=510)
    o, lse = gpu_lib.attn_prefill(q, k, v)
    grads = [f64(g)[0] for g in gpu_lib.attn_backward(q, k, v, o, lse, up, grad_dtype="float32")]
    x, u = [f64(t) for t in (q, k, v)], f64(up)
    want, _ = ref.attn_backward(*x, u)
    bound = attn_norms.bounds(*[a[0] for a in x], u[0], [w[0] for w in want], rounded=False, u=U + 4.2 * eps(x[0], x[1], T))
    for i, d in enumerate(want):
        step = 1e-4 / np.abs(d).max()
        y = [[a + s * step * d if j == i else a for j, a in enumerate(x)] for s in (1, -1)]
        slope = ((ref.attn_prefill(*y[0])[0] - ref.attn_prefill(*y[1])[0]) * u).sum() / (2 * step)
        room = np.sqrt(sum(b * b for b in bound[i].values())) * np.linalg.norm(d)
        assert room < 0.02 * slope
        # the differences' own error: terms of the third order, about step^2 of the slope, and float64's rounding
        assert abs((grads[i] * d[0]).sum() - slope) <= room + 1e-5 * slope
