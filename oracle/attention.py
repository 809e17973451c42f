"""Full attention in float64: the definitions behind kda_attn_* (include/kda.h).

Plain loops over sequences and heads, nothing shared with the HIP path.  The
functions that go with a tolerance also return what the tolerance is made of
(sums of magnitudes), so that tests can bound roundings term by term.
"""

import numpy as np

E4M3_MAX = 448.0


def bounds_of(cu, T):
    """[start, end) of each packed sequence; None: one sequence of T tokens."""
    if cu is None:
        return [(0, T)]
    at = [min(max(int(c), 0), T) for c in cu]
    return [(a, max(a, b)) for a, b in zip(at, at[1:])]


def head_weights(q, k, scale, seen):
    """q [r, D], k [n, D], seen [r, n] -> (softmax weights, log-sum-exp); a row that sees nothing: zeros, -inf."""
    z = np.where(seen, (q @ k.T) * scale, -np.inf)
    top = np.max(z, axis=1, initial=-np.inf)
    base = np.where(np.isfinite(top), top, 0.0)
    e = np.where(seen, np.exp(z - base[:, None]), 0.0)
    total = e.sum(1)
    with np.errstate(divide="ignore"):
        lse = np.where(total > 0, np.log(total) + base, -np.inf)
    return e / np.where(total > 0, total, 1.0)[:, None], lse


def causal(n):
    return np.tril(np.ones((n, n), bool))


def attn_prefill(q, k, v, cu=None, scale=None):
    """q [B,T,HQ,D], k, v [B,T,HKV,D] -> (o, lse [B,HQ,T], o_abs = sum_j P_ij |v_j|); rows outside the sequences are NaN."""
    B, T, HQ, D = q.shape
    G = HQ // k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    o, o_abs = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    lse = np.full((B, HQ, T), np.nan)
    for b in range(B):
        for lo, hi in bounds_of(cu, T):
            for h in range(HQ):
                w, z = head_weights(q[b, lo:hi, h], k[b, lo:hi, h // G], scale, causal(hi - lo))
                o[b, lo:hi, h], lse[b, h, lo:hi] = w @ v[b, lo:hi, h // G], z
                o_abs[b, lo:hi, h] = w @ np.abs(v[b, lo:hi, h // G])
    return o, lse, o_abs


def attn_backward(q, k, v, d_out, cu=None, scale=None):
    """Gradients of sum(o * d_out): dq, dk, dv, and for each the sum of the magnitudes that roundings of relative size 1 in
    P, dS and o would move it by (see the tests)."""
    B, T, HQ, D = q.shape
    G = HQ // k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    grads = [np.full(x.shape, np.nan) for x in (q, k, v)]
    moved = [np.full(x.shape, np.nan) for x in (q, k, v)]
    for b in range(B):
        for lo, hi in bounds_of(cu, T):
            for x, like in zip(grads + moved, (q, k, v) * 2):
                x[b, lo:hi] = 0.0
            for h in range(HQ):
                qh, kh, vh, up = q[b, lo:hi, h], k[b, lo:hi, h // G], v[b, lo:hi, h // G], d_out[b, lo:hi, h]
                w, _ = head_weights(qh, kh, scale, causal(hi - lo))
                o, dw = w @ vh, up @ vh.T
                delta = (up * o).sum(1, keepdims=True)
                ds = w * (dw - delta)
                grads[0][b, lo:hi, h] += scale * ds @ kh
                grads[1][b, lo:hi, h // G] += scale * ds.T @ qh
                grads[2][b, lo:hi, h // G] += w.T @ up
                # dS is rounded itself; a relative error of 1 in o (and in the weights behind it) moves delta by at most
                # the second term; the third, 2^-8 of the products' magnitudes, is room for their float32 sums
                ds_abs = np.abs(ds) + w * (np.abs(up) * (np.abs(o) + w @ np.abs(vh))).sum(1, keepdims=True)
                ds_abs += w * (np.abs(up) @ np.abs(vh).T) * 2.0 ** -8
                moved[0][b, lo:hi, h] += scale * ds_abs @ np.abs(kh)
                moved[1][b, lo:hi, h // G] += scale * ds_abs.T @ np.abs(qh)
                moved[2][b, lo:hi, h // G] += w.T @ np.abs(up)
    return grads, moved


# ---------------------------------------------------------------- the paged cache

def e4m3_table():
    """Value of each of the 256 codes (OCP e4m3: bias 7, no infinities, 0x7f and 0xff NaN)."""
    x = np.arange(256)
    sign, e, m = np.where(x & 128, -1.0, 1.0), (x >> 3) & 15, x & 7
    value = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(float) - 10))
    return np.where((x & 127) == 127, np.nan, sign * value)


def to_e4m3(x):
    """Codes nearest to x (|x| <= 448 or not finite), ties to the even code; infinities and NaN give NaN (0x7f)."""
    x = np.asarray(x, np.float64)
    table = e4m3_table()[:127]
    mag = np.where(np.isfinite(x), np.abs(x), 0.0)
    hi = np.clip(np.searchsorted(table, mag, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = table[hi] - mag, mag - table[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)) | (table[hi] == mag), hi, lo)
    code = np.where(np.isfinite(x), code, 127)
    return (code + np.where(np.signbit(x) & np.isfinite(x), 128, 0)).astype(np.uint8)


def scale_for(top):
    """Least power of two 2^e, e >= -64, with 448 * 2^e >= top."""
    if top <= 0:
        return 2.0 ** -64
    f, x = np.frexp(top)                       # top = f * 2^x, 1/2 <= f < 1; 448 = 0.875 * 2^9
    return 2.0 ** max(int(x) - 9 + int(f > 0.875), -64)


def attn_cache_store(x, cache, scale, slots):
    """x [T, HKV, D] into codes [pages, HKV, P, D] (uint8) and scale [pages, HKV]; returns new ones."""
    cache, scale = cache.copy(), scale.astype(np.float64).copy()
    pages, HKV, P, _ = cache.shape
    table = e4m3_table()
    per_page = {}
    for t, s in enumerate(slots):
        if 0 <= s < pages * P:
            per_page.setdefault(int(s) // P, []).append((int(s) % P, t))
    for page, tokens in per_page.items():
        first = tokens[0][0]
        for h in range(HKV):
            new = np.stack([x[t, h] for _, t in tokens])
            finite = np.abs(new[np.isfinite(new)])
            fits = scale_for(finite.max() if finite.size else 0.0)
            was = scale[page, h]
            now = fits if first == 0 else max(was, fits)
            if first and now != was:
                cache[page, h, :first] = to_e4m3(table[cache[page, h, :first]] * (was / now))
            scale[page, h] = now
            for (off, t), row in zip(tokens, new):
                cache[page, h, off] = to_e4m3(row / now)
    return cache, scale


def attn_tables(cached, new, table, free, head, P, num_tokens):
    """(cu_seqlens, slots, kv_lens, page table, next head)."""
    table, W = table.copy(), table.shape[1]
    cu, slots, lens, taken = [0], [], [], head
    for n, (a, b) in enumerate(zip(np.maximum(cached, 0), np.maximum(new, 0))):
        a, b = int(a), int(b)
        for c in range(min(-(-a // P), W), min(-(-(a + b) // P), W)):
            table[n, c] = free[taken] if taken < len(free) else -1
            taken += 1
        for p in range(a, a + b):
            page = table[n, p // P] if p // P < W else -1
            slots.append(page * P + p % P if page >= 0 else -1)
        cu.append(cu[-1] + b)
        lens.append(a + b)
    slots = (slots + [-1] * num_tokens)[:num_tokens]
    return np.array(cu), np.array(slots), np.array(lens), table, taken


def attn_decode(q, k_cache, v_cache, k_scale, v_scale, table, lens, scale=None):
    """q [N,Q,HQ,D], codes [pages,HKV,P,D] -> (o [N,Q,HQ,D], lse [N,Q,HQ], o_abs)."""
    N, Q, HQ, D = q.shape
    pages, HKV, P, _ = k_cache.shape
    scale = D ** -0.5 if scale is None else scale
    value = e4m3_table()
    o, o_abs, lse = np.zeros(q.shape), np.zeros(q.shape), np.full((N, Q, HQ), -np.inf)
    for n in range(N):
        length = min(max(int(lens[n]), 0), table.shape[1] * P)
        ids = table[n, :-(-length // P)]
        there = np.repeat((ids >= 0) & (ids < pages), P)[:length]
        safe = np.where((ids >= 0) & (ids < pages), ids, 0)
        at = np.arange(length)
        seen = (at[None] <= length - Q + np.arange(Q)[:, None]) & there[None]
        for h in range(HQ):
            j = h * HKV // HQ
            k, v = (np.where(there[:, None], (value[c[safe, j]] * s[safe, j][:, None, None]).reshape(-1, D)[:length], 0.0)
                    for c, s in ((k_cache, k_scale), (v_cache, v_scale)))
            w, lse[n, :, h] = head_weights(q[n, :, h], k, scale, seen)
            o[n, :, h], o_abs[n, :, h] = w @ v, w @ np.abs(v)
    return o, lse, o_abs
