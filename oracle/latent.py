"""Latent attention in float64: the definitions behind kda_latent_* (include/kda.h).

Plain loops over sequences, heads and tokens, nothing shared with the HIP path;
weights and e4m3 codes are attention.py's.  The functions that go with a tolerance
also return what the tolerance is made of (sums of magnitudes).
"""

import numpy as np

from .attention import bounds_of, e4m3_table, head_weights, to_e4m3

D, S, R, BLOCK = 128, 64, 512, 128
SCALE = (D + S) ** -0.5


def pairs(cu, cu_kv, T, K):
    """(start, end) of each sequence's queries and keys."""
    if cu is None:
        return [(0, T, 0, K)]
    return [(*a, *b) for a, b in zip(bounds_of(cu, T), bounds_of(cu if cu_kv is None else cu_kv, K))]


def seen(nq, nk):
    """[nq, nk]: the last query stands at the last key."""
    return np.arange(nk)[None] <= np.arange(nq)[:, None] + nk - nq


def latent_prefill(q, k, s, v, cu=None, cu_kv=None, scale=SCALE):
    """q [B,T,H,192], k, v [B,K,H,128], s [B,K,64] -> (o, lse [B,H,T], o_abs = sum_j P_ij |v_j|); rows outside the
    sequences are NaN."""
    B, T, H, _ = q.shape
    o, o_abs, lse = np.full((B, T, H, D), np.nan), np.full((B, T, H, D), np.nan), np.full((B, H, T), np.nan)
    for b in range(B):
        for lo, hi, klo, khi in pairs(cu, cu_kv, T, k.shape[1]):
            for h in range(H):
                key = np.concatenate((k[b, klo:khi, h], s[b, klo:khi]), 1)
                w, z = head_weights(q[b, lo:hi, h], key, scale, seen(hi - lo, khi - klo))
                o[b, lo:hi, h], lse[b, h, lo:hi] = w @ v[b, klo:khi, h], z
                o_abs[b, lo:hi, h] = w @ np.abs(v[b, klo:khi, h])
    return o, lse, o_abs


def latent_backward(q, k, s, v, d_out, cu=None, cu_kv=None, scale=SCALE):
    """Gradients of sum(o * d_out): (dq, dk, ds, dv), and for each the sum of the magnitudes that roundings of relative
    size 1 in P, dS and o would move it by."""
    B, T, H, _ = q.shape
    like = (q, k, s, v)
    grads, moved = ([np.full(x.shape, np.nan) for x in like] for _ in range(2))
    for b in range(B):
        for lo, hi, klo, khi in pairs(cu, cu_kv, T, k.shape[1]):
            for x in (grads, moved):
                x[0][b, lo:hi] = 0.0
                for y in x[1:]:
                    y[b, klo:khi] = 0.0
            for h in range(H):
                qh, vh, up = q[b, lo:hi, h], v[b, klo:khi, h], d_out[b, lo:hi, h]
                key = np.concatenate((k[b, klo:khi, h], s[b, klo:khi]), 1)
                w, _ = head_weights(qh, key, scale, seen(hi - lo, khi - klo))
                o, dw = w @ vh, up @ vh.T
                ds = w * (dw - (up * o).sum(1, keepdims=True))
                # dS is rounded itself; a relative error of 1 in o (and in the weights behind it) moves delta by at most
                # the second term; the third, 2^-8 of the products' magnitudes, is room for their float32 sums
                ds_abs = np.abs(ds) + w * (np.abs(up) * (np.abs(o) + w @ np.abs(vh))).sum(1, keepdims=True)
                ds_abs += w * (np.abs(up) @ np.abs(vh).T) * 2.0 ** -8
                for x, a, f, p in ((grads, ds, lambda y: y, w), (moved, ds_abs, np.abs, w)):
                    x[0][b, lo:hi, h] += scale * a @ f(key)
                    dkey = scale * a.T @ f(qh)
                    x[1][b, klo:khi, h] += dkey[:, :D]
                    x[2][b, klo:khi] += dkey[:, D:]
                    x[3][b, klo:khi, h] += p.T @ f(up)
    return grads, moved


# ---------------------------------------------------------------- the paged cache

def exponent_for(top):
    """Least e in [-64, 119] with 448 * 2^e >= top (119 if none)."""
    e = -64
    while e < 119 and 448.0 * 2.0 ** e < top:
        e += 1
    return e


def latent_cache_store(c, s, codes, scales, shared, slots):
    """c [T,512], s [T,64] into codes and scales (uint8) [pages,P,512], [pages,P,4] and shared [pages,P,64]; returns
    new ones."""
    codes, scales, shared = codes.copy(), scales.copy(), shared.copy()
    P = codes.shape[1]
    for t, slot in enumerate(slots):
        if not 0 <= slot < codes.shape[0] * P:
            continue
        page, off = int(slot) // P, int(slot) % P
        for j in range(R // BLOCK):
            x = c[t, j * BLOCK:(j + 1) * BLOCK]
            finite = np.abs(x[np.isfinite(x)])
            e = exponent_for(finite.max() if finite.size else 0.0)
            y = x * 2.0 ** -e
            y = np.where(np.isfinite(y), np.clip(y, -448.0, 448.0), y)
            codes[page, off, j * BLOCK:(j + 1) * BLOCK] = to_e4m3(y)
            scales[page, off, j] = e + 127
        shared[page, off] = s[t]
    return codes, scales, shared


def latents(codes, scales):
    """Codes [..., 512] and scales [..., 4] (uint8) as values."""
    return e4m3_table()[codes] * np.repeat(2.0 ** (scales.astype(float) - 127), BLOCK, -1)


def cached(codes, scales, shared, row, length):
    """The first `length` tokens of a page table's row: latents, shared parts, whether there is a page."""
    pages, P, _ = codes.shape
    ids = np.full(-(-length // P), -1, np.int64)
    ids[:min(len(ids), len(row))] = row[:len(ids)]
    there = np.repeat((ids >= 0) & (ids < pages), P)[:length]
    safe = np.where((ids >= 0) & (ids < pages), ids, 0)
    c = latents(codes[safe], scales[safe]).reshape(-1, R)[:length]
    return np.where(there[:, None], c, 0.0), np.where(there[:, None], shared[safe].reshape(-1, S)[:length], 0.0), there


def latent_cache_load(codes, scales, shared, table, cu, num_tokens):
    """(c [num_tokens,512], s [num_tokens,64]); rows outside the sequences are NaN."""
    c, s = np.full((num_tokens, R), np.nan), np.full((num_tokens, S), np.nan)
    for row, (lo, hi) in zip(table, bounds_of(cu, num_tokens)):
        c[lo:hi], s[lo:hi], _ = cached(codes, scales, shared, row, hi - lo)
    return c, s


def latent_decode(q, codes, scales, shared, table, lens, scale=SCALE):
    """q [N,Q,H,576] -> (o [N,Q,H,512], lse [N,Q,H], o_abs)."""
    N, Q, H, _ = q.shape
    o, o_abs, lse = np.zeros((N, Q, H, R)), np.zeros((N, Q, H, R)), np.full((N, Q, H), -np.inf)
    for n in range(N):
        length = min(max(int(lens[n]), 0), table.shape[1] * codes.shape[1])
        c, s, there = cached(codes, scales, shared, table[n], length)
        visible = (np.arange(length)[None] <= length - Q + np.arange(Q)[:, None]) & there[None]
        for h in range(H):
            w, lse[n, :, h] = head_weights(q[n, :, h], np.concatenate((c, s), 1), scale, visible)
            o[n, :, h], o_abs[n, :, h] = w @ c, w @ np.abs(c)
    return o, lse, o_abs
