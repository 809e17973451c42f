"""Bounds on the norm of an error in latent attention's gradients, as attn_norms.py's.

Independent errors, each taken at its largest, add as squares; a rounding's root mean square is below half of its
largest error, which leaves a factor of two.  With u the relative error of what is rounded as an operand (2^-8 for
one bfloat16 term, 2^-16 for two), of one sequence and head:
    a score is off by ez = 192 2^-23 scale |q| . |k s| + 2^-20 (a float32 sum of 192 products, each step off by at most
    2^-23 of the magnitudes' sum, and the exponential), its row's lse by the mean of that;
    dO V^T is off by eg = 128 2^-23 |dO| . |v|, P by ep = ez and lse's error;
    dS = P (dO V^T - delta) by u and ep of itself and P eg, and by P times what moves delta: o's own rounding and that
    of the weights behind it (2^-8 each), or, in workgroups of 128 rows whose last row sees at most 256 keys, ep and eg
    of the sum that it is made of;
    dQ by that times the keys, dK and dS's shared part times the queries, dV by u and ep of P times dO;
    and a float32 sum of n products by n 2^-24 of their magnitudes, a result by its own rounding, if it has one.
"""

import numpy as np

import oracle.attention as attn
import oracle.latent as ref

U = 2.0 ** -8
D, S = 128, 64


def norm2(x):
    return (x * x).sum(-1)


def _of_head(q, key, v, up, scale):
    nq, nk = len(q), len(key)
    w, _ = attn.head_weights(q, key, scale, ref.seen(nq, nk))
    o, dw = w @ v, up @ v.T
    return w, o, dw, w * (dw - (up * o).sum(1, keepdims=True))


def _few_keys(nq, nk):
    """Rows of workgroups whose last row sees 256 keys or fewer."""
    last = np.minimum(np.arange(nq) // 128 * 128 + 128, nq) + nk - nq
    return last <= 256


def bounds(q, k, s, v, up, grads, cu=None, cu_kv=None, scale=ref.SCALE, rounded=True, u=U):
    """For dq, dk, ds, dv (float64, of one batch row): {(sequence, head): (bound on the error's norm)}, ds by sequence
    alone."""
    T, H, _ = q.shape
    out = [{}, {}, {}, {}]
    for n, (lo, hi, klo, khi) in enumerate(ref.pairs(cu, cu_kv, T, len(k))):
        nq, nk = hi - lo, khi - klo
        ds2 = rounded * U ** 2 * norm2(grads[2][klo:khi]).sum()
        more = np.zeros((nk, S))
        for h in range(H):
            qh, vh, uh, key = q[lo:hi, h], v[klo:khi, h], up[lo:hi, h], np.concatenate((k[klo:khi, h], s[klo:khi]), 1)
            w, o, dw, ds = _of_head(qh, key, vh, uh, scale)
            ez = 192 * 2.0 ** -23 * scale * np.abs(qh) @ np.abs(key).T + 2.0 ** -20
            el = (w * ez).sum(1, keepdims=True)
            ep2 = ez ** 2 + el ** 2
            eg2 = (128 * 2.0 ** -23 * np.abs(uh) @ np.abs(vh).T) ** 2
            made = (w * w * (dw * dw * ep2 + eg2)).sum(1)
            delta2 = np.where(_few_keys(nq, nk), made, U ** 2 * (norm2(uh * o) + (w * w * dw * dw).sum(1)) + made)
            term2 = ds * ds * (u ** 2 + ep2) + w * w * eg2           # of dS, but for delta
            sums = nk * 2.0 ** -24 * np.abs(ds) @ np.abs(key)
            dq2 = scale ** 2 * ((term2 @ norm2(key)).sum() + (delta2 * norm2(w @ key)).sum() + norm2(sums).sum()
                                + (el[:, 0] ** 2 * norm2(ds @ key)).sum())
            out[0][n, h] = dq2 + rounded * U ** 2 * norm2(grads[0][lo:hi, h]).sum()
            rows = (term2 + w * w * delta2[:, None]).sum(1)
            sums = nq * 2.0 ** -24 * np.abs(ds).T @ np.abs(qh)
            more += scale * sums[:, D:]
            dk2 = scale ** 2 * ((rows * norm2(qh[:, :D])).sum() + norm2(sums[:, :D]).sum())
            out[1][n, h] = dk2 + rounded * U ** 2 * norm2(grads[1][klo:khi, h]).sum()
            ds2 += scale ** 2 * (rows * norm2(qh[:, D:])).sum()
            dv2 = ((w * w * (u ** 2 + ep2)).sum(1) * norm2(uh)).sum() + norm2(nq * 2.0 ** -24 * w.T @ np.abs(uh)).sum()
            out[3][n, h] = dv2 + rounded * U ** 2 * norm2(grads[3][klo:khi, h]).sum()
        out[2][n, None] = ds2 + norm2(more).sum() + norm2(H * 2.0 ** -24 * np.abs(grads[2][klo:khi])).sum()
    return [{at: np.sqrt(x) for at, x in b.items()} for b in out]


def worst(got, want, bound, cu=None, cu_kv=None):
    """Largest error's norm over its bound, over tensors, sequences and heads; infinite where an error is not a number
    or there is one where none is allowed."""
    most = 0.0
    ends = ref.pairs(cu, cu_kv, len(want[0]), len(want[1]))
    for i, (g, w, b) in enumerate(zip(got, want, bound)):
        for (n, h), x in b.items():
            lo, hi = ends[n][:2] if i == 0 else ends[n][2:]
            off = g[lo:hi] - w[lo:hi] if h is None else g[lo:hi, h] - w[lo:hi, h]
            off = np.sqrt(norm2(off).sum())
            most = max(most, (off / x if x else (off and np.inf)) if np.isfinite(off) else np.inf)
    return most
