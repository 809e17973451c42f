"""kda_attn_prefill and kda_attn_backward over packed offsets of every kind that
the header allows: outside the batch, and with sequences that would end before
they start.  Results against the float64 oracle (tolerances as in
test_gpu_attn_prompt.py); rows outside the sequences stay as they were.
"""

import random

import pytest
import torch

import oracle.attention as ref
from test_gpu_attn_prompt import D, DEV, case, check_grads, check_prompt

pytestmark = pytest.mark.gpu
MOST, LEAST = 2 ** 31 - 1, -2 ** 31


def outside(cu, T):
    rows = torch.ones(T, dtype=torch.bool)
    for lo, hi in ref.bounds_of(cu, T):
        rows[lo:hi] = False
    return rows


def backward_into(kda, q, k, v, o, lse, up, cu, fill, wide):
    """Gradients into buffers that hold `fill`, over a workspace of NaN."""
    _, T, HQ, _ = q.shape
    HKV = k.shape[2]
    grads = [torch.full((1, T, h, D), fill, dtype=torch.float32 if wide else torch.bfloat16, device=DEV) for h in (HQ, HKV, HKV)]
    N = cu.numel() - 1
    size = kda.attn_backward_workspace_size(1, T, HQ, HKV, N)
    ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    P = [x.data_ptr() for x in (q, k, v, o, lse, up, cu, *grads, ws)]
    assert kda.load().kda_attn_backward(
        *P[:3], HQ * D, HKV * D, HKV * D, *P[3:7], N, 1, T, HQ, HKV, D, D ** -0.5, *P[7:10],
        kda.GRAD_FLOAT32 if wide else kda.GRAD_INPUT_DTYPE, P[10], size, torch.cuda.current_stream().cuda_stream) == 0
    return grads


def check_all(kda, T, HQ, HKV, cu, seed):
    """Forward and backward; rows outside the sequences hold NaN in every input."""
    q, k, v, up, c = case(1, T, HQ, HKV, cu, seed)
    out = outside(cu, T)
    for x in (q, k, v, up):
        x[0, out] = float("nan")
    o = torch.full((1, T, HQ, D), 7.5, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((1, HQ, T), 7.5, device=DEV)
    kda.attn_prefill(q, k, v, cu_seqlens=c, out=o, lse=lse)
    assert (o[0, out] == 7.5).all() and (lse[0][:, out] == 7.5).all()
    check_prompt(o, lse, q, k, v, cu)
    for wide in (True, False):
        grads = backward_into(kda, q, k, v, o, lse, up, c, 3.0, wide)
        assert all((x[0, out] == 3).all() for x in grads)
        check_grads(grads, q, k, v, up, cu, rounded=not wide)


@pytest.mark.parametrize("cu", [[0, 150, LEAST], [LEAST, 40, 170], [100, MOST, LEAST, 60], [30, MOST, MOST, LEAST, 30]])
def test_offsets_outside_the_batch(gpu_lib, cu):
    """An offset counts as the nearest place in the batch, however far outside it lies."""
    HQ, HKV = 4, 2
    assert gpu_lib.attn_backward_workspace_size(1, 200, HQ, HKV, len(cu) - 1) == 2 * 200 * HQ * 4   # no parts
    check_all(gpu_lib, 200, HQ, HKV, cu, seed=300)


@pytest.mark.parametrize("HQ,HKV", [(8, 1), (8, 2), (12, 3)])
@pytest.mark.parametrize("cu", [[0, 100, 90], [50, 20, 80], [200, 331, 0, 179, 180, 150], [399, 3, 2, LEAST],
                                [350, 400] + [300] * 45 + [0, 251]])
def test_offsets_that_decrease(gpu_lib, cu, HQ, HKV):
    """A sequence that would end before it starts is empty; the others count wherever they lie, also where several
    workgroups share a key tile (float32 parts and their sum)."""
    T = 400
    assert gpu_lib.attn_backward_workspace_size(1, T, HQ, HKV, len(cu) - 1) > 2 * T * HQ * 4         # parts
    check_all(gpu_lib, T, HQ, HKV, cu, seed=310)


def mixed(N, seed, lengths=(0, 1, 127, 128, 129, 256, 300, 700), most=6000, front=0):
    """Offsets of N sequences of these lengths, each among them, those past `most` tokens empty."""
    rng = random.Random(seed)
    cu = [front]
    some = list(lengths) + [rng.choice(lengths) for _ in range(N - len(lengths))]
    rng.shuffle(some)
    for n in some:
        cu.append(cu[-1] + (n if cu[-1] + n <= most else 0))
    return cu


MANY = [  # tokens, heads, offsets, whether several workgroups share a key tile
    (6100, 4, 1, mixed(65, 1), True),
    (6100, 2, 2, mixed(65, 2, front=37), False),
    (6100, 16, 2, mixed(150, 3, front=5), True),
    (2000, 4, 2, mixed(300, 4, (0, 0, 1, 2, 5, 128, 130), 1990), False),      # more than 256
    (3000, 4, 1, [2900] * 256 + [3000, 0, 700] + [700] * 10 + [2000], True),
    (1000, 2, 1, [0, 1000] + [0] * 64, False),
    (1000, 1, 1, [0] * 70 + [1000], False),
    (900, 4, 2, [3 * n for n in range(300, -1, -1)], False),                  # nothing but ends before starts
    (1500, 4, 1, [x for n in range(9, -1, -1) for x in (150 * n, 150 * n + 129 + n)] + [0] * 60, True),
]


@pytest.mark.parametrize("T,HQ,HKV,cu,parts", MANY)
def test_more_than_64_sequences(gpu_lib, T, HQ, HKV, cu, parts):
    """Sequences of several row tiles among empty ones, beyond those that one wave ranks, in order and not."""
    N = len(cu) - 1
    assert N > 64 and (gpu_lib.attn_backward_workspace_size(1, T, HQ, HKV, N) > 2 * T * HQ * 4 + 12) == parts
    check_all(gpu_lib, T, HQ, HKV, cu, seed=320 + N)
