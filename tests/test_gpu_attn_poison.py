"""Decode over caches in which everything that no sequence holds is NaN: rows
behind the sequences' ends, unused pages and their scales; and table entries past
the ends that name such pages.  Every case of test_gpu_attn_cache.py's decode
tests, cut among waves and by segments."""

import numpy as np
import pytest
import torch

from test_gpu_attn_cache import DECODE, Wide, check_decode, ints, tables_for, usual_cache
from test_gpu_attn_prompt import D, DEV, rand

pytestmark = pytest.mark.gpu


def poisoned(cache, table, lens, P):
    """A copy with NaN wherever no sequence has a token."""
    out = [c.clone() for c in cache]
    pages = cache[0].shape[0]
    used = np.zeros((pages, P), bool)
    for row, n in zip(table, lens):
        for i in range(-(-n // P)):
            used[row[i], :min(n - i * P, P)] = True
    empty = torch.from_numpy(~used).to(DEV)
    for c in out[:2]:
        c.view(torch.uint8).masked_fill_(empty[:, None, :, None], 0x7f)
    for s in out[2:]:
        s.masked_fill_(empty.all(1)[:, None], float("nan"))
    return out


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("lens,Q,HQ,HKV,P", DECODE + [([700, 90, 0], 100, 2, 1, 64), ([1300, 20], 1024, 2, 2, 64)])
def test_decode_beside_nan(gpu_lib, lens, Q, HQ, HKV, P, wide):
    kda = Wide(gpu_lib) if wide else gpu_lib
    table, pages = tables_for(lens, P, spare=3, seed=40)
    cache = usual_cache(600 + len(lens), pages, HKV, P)
    bad = poisoned(cache, table, lens, P)
    assert any(torch.isnan(s).any() for s in bad[2:])
    unused = int(np.setdiff1d(np.arange(pages), np.concatenate([row[:-(-n // P)] for row, n in zip(table, lens)]))[0])
    for row, n in zip(table, lens):
        row[-(-n // P):] = unused                             # entries that must not be used
    q = rand(601, len(lens), Q, HQ, D).to(DEV)
    ws = torch.full((gpu_lib.attn_decode_workspace_size(len(lens), Q, HQ, HKV),), 255, dtype=torch.uint8, device=DEV)
    o, lse = kda.attn_decode(q, *bad, ints(table), ints(lens), workspace=ws)
    check_decode(o, lse, q, cache, table, lens)
    o2, lse2 = kda.attn_decode(q, *cache, ints(table), ints(lens))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
