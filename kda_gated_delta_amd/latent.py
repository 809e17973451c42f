"""Binding of the latent-attention entry points (include/kda.h, kda_latent_*):
what a hybrid model whose keys and values come from one latent vector per token
runs in the layers between its KDA layers.

As in attn.py these functions check arguments, allocate outputs that are not
passed, and call the library on the current stream of their tensors' device.
"""

import torch

import kda_gated_delta_amd as _kda

from .attn import _BF16, _E4M3, _F32, _I32, _call, _dense, _first, _gpu, _ptr, _table, _workspace

D = 128            # a head's own key, and its value
S = 64             # the shared key part
R = 512            # the latent
BLOCK = 128        # of the latent: values under one scale
_U8 = torch.uint8


def _scale(scale):
    return (D + S) ** -0.5 if scale is None else float(scale)


def _even(t, name, lead, inner):
    """Elements from token to token of t [*lead, ...]: evenly spaced over all leading axes; inner: the step of one
    token alone."""
    step, expect = None, None
    for size, stride in zip(reversed(lead), reversed(t.stride()[:len(lead)])):
        if size == 1:
            continue
        if step is None:
            step, expect = stride, stride * size
        elif stride == expect:
            expect = stride * size
        else:
            raise ValueError(f"{name}: tokens must be evenly spaced")
    return inner if step is None else step


def _rows(t, name, dev, shape):
    """Elements from token to token of bf16 t, of this shape, whose last axes past the tokens' (all but the last, or the
    last two of q) are compact."""
    if not (isinstance(t, torch.Tensor) and t.dtype is _BF16 and t.get_device() == dev and t.shape == shape):
        _gpu(t, name, _BF16, dev, shape)
    width = shape[-1] if len(shape) < 4 else shape[2] * shape[3]
    if t.is_contiguous():
        return width
    stride = t.stride()
    if len(shape) == 2 and stride[1] == 1:
        return stride[0] if shape[0] > 1 else width
    inner, compact = len(shape) - (2 if len(shape) == 4 else 1), 1
    for n, step in zip(reversed(shape[inner:]), reversed(stride[inner:])):
        if n > 1 and step != compact:
            raise ValueError(f"{name}: the axes behind the tokens must be compact")
        compact *= n
    return _even(t, name, shape[:inner], width)


def _heads(t, name, dev, shape):
    """Elements from token to token and from head to head of k or v [B, T, H, 128]."""
    _gpu(t, name, _BF16, dev, shape)
    if t.is_contiguous():
        return shape[2] * D, D
    stride = t.stride()
    if stride[3] != 1:
        raise ValueError(f"{name}: the last axis must be compact")
    head = stride[2] if shape[2] > 1 else D
    return _even(t, name, shape[:2], D), head


def _offsets(cu, name, dev):
    _dense(cu, name, _I32, dev)
    if cu.dim() != 1 or cu.shape[0] < 2:
        raise ValueError(f"{name} must be [N + 1]")
    return cu.shape[0] - 1


def _prompt(q, k, k_shared, v, cu_seqlens, cu_seqlens_kv):
    dev = _first(q, "q", _BF16, 4)
    B, T, H, _ = q.shape
    K = k.shape[1] if isinstance(k, torch.Tensor) and k.dim() == 4 else 0
    qs = _rows(q, "q", dev, (B, T, H, D + S))
    ks, kh = _heads(k, "k", dev, (B, K, H, D))
    vs, vh = _heads(v, "v", dev, (B, K, H, D))
    ss = _rows(k_shared, "k_shared", dev, (B, K, S))
    N = 0
    if cu_seqlens is None:
        if cu_seqlens_kv is not None:
            raise ValueError("cu_seqlens_kv goes with cu_seqlens")
    else:
        N = _offsets(cu_seqlens, "cu_seqlens", dev)
        if cu_seqlens_kv is None:
            if K != T:
                raise ValueError("cu_seqlens_kv is needed where there are more or fewer keys than queries")
            cu_seqlens_kv = cu_seqlens
        elif _offsets(cu_seqlens_kv, "cu_seqlens_kv", dev) != N:
            raise ValueError("cu_seqlens and cu_seqlens_kv must have as many sequences")
    args = (q.data_ptr(), k.data_ptr(), k_shared.data_ptr(), v.data_ptr(), qs, ks, kh, ss, vs, vh)
    return dev, B, T, K, H, N, args, (_ptr(cu_seqlens), _ptr(cu_seqlens_kv), N, B, T, K, H)


def latent_prefill(q, k, k_shared, v, cu_seqlens=None, cu_seqlens_kv=None, scale=None, out=None, lse=None):
    """Causal attention in the expanded form.  q [B,T,H,192] bf16 (tokens may be
    slices of wider rows): 128 against a head's key, 64 against the shared part; k
    and v [B,Tk,H,128] bf16 (the halves of one projection's rows, say, or with the
    heads outermost) and k_shared [B,Tk,64] bf16.  The last query stands at the last
    key: query i sees the keys up to i + Tk - T, and none gives zeros.  cu_seqlens
    int32 [N+1] (with B == 1): packed sequences, in any order; cu_seqlens_kv the
    same for the keys, by default the queries' own.  Rows outside the sequences are
    neither read nor written (and hold anything in outputs that are allocated here).
    scale defaults to 192**-0.5.  Returns (o [B,T,H,128] bf16, lse [B,H,T] float32)."""
    dev, B, T, _, H, _, args, sizes = _prompt(q, k, k_shared, v, cu_seqlens, cu_seqlens_kv)
    if out is None:
        out = q.new_empty((B, T, H, D))
    else:
        _dense(out, "out", _BF16, dev, (B, T, H, D))
    if lse is None:
        lse = q.new_empty((B, H, T), dtype=_F32)
    else:
        _dense(lse, "lse", _F32, dev, (B, H, T))
    _call(dev, "kda_latent_prefill", *args, *sizes, _scale(scale), out.data_ptr(), lse.data_ptr())
    return out, lse


def latent_backward_workspace_size(B, T, T_kv, H, num_seqs=0):
    """Bytes of workspace latent_backward needs on the current device (num_seqs = 0
    without cu_seqlens)."""
    return int(_kda.load().kda_latent_backward_workspace_size(B, T, T_kv, H, num_seqs))


def latent_backward(q, k, k_shared, v, o, lse, d_out, cu_seqlens=None, cu_seqlens_kv=None, scale=None, workspace=None,
                    grad_dtype="input", dq=None, d_kv=None, dk_shared=None):
    """Gradients of sum(o * d_out) for latent_prefill with the same inputs, of
    which o and lse are the outputs.  d_out [B,T,H,128] bf16.  Returns (dq, dk,
    dk_shared, dv), bf16 (grad_dtype "input") or float32 ("float32"); dk_shared is
    summed over the heads.  dk and dv are the halves of d_kv's rows [B,Tk,H,256], the
    gradient of the one projection that usually makes both keys and values.  Keys
    that no query sees get zeros; rows outside the sequences hold anything, or what
    dq [B,T,H,192], d_kv and dk_shared [B,Tk,64] held if they are passed."""
    if grad_dtype not in ("input", "float32"):
        raise ValueError("grad_dtype must be 'input' or 'float32'")
    dev, B, T, K, H, N, args, sizes = _prompt(q, k, k_shared, v, cu_seqlens, cu_seqlens_kv)
    _dense(o, "o", _BF16, dev, (B, T, H, D))
    _dense(d_out, "d_out", _BF16, dev, (B, T, H, D))
    _dense(lse, "lse", _F32, dev, (B, H, T))
    if workspace is None:
        workspace = _workspace(q, dev, latent_backward_workspace_size, B, T, K, H, N)
    else:
        _dense(workspace, "workspace", _U8, dev)
    dtype = _BF16 if grad_dtype == "input" else _F32

    def made(t, name, shape):
        if t is None:
            return q.new_empty(shape, dtype=dtype)
        _dense(t, name, dtype, dev, shape)
        return t
    dq, d_kv = made(dq, "dq", (B, T, H, D + S)), made(d_kv, "d_kv", (B, K, H, 2 * D))
    dk_shared = made(dk_shared, "dk_shared", (B, K, S))
    _call(dev, "kda_latent_backward", *args, o.data_ptr(), lse.data_ptr(), d_out.data_ptr(), *sizes, _scale(scale),
          dq.data_ptr(), d_kv.data_ptr(), dk_shared.data_ptr(),
          _kda.GRAD_INPUT_DTYPE if grad_dtype == "input" else _kda.GRAD_FLOAT32, workspace.data_ptr(),
          workspace.numel())
    return dq, d_kv[..., :D], dk_shared, d_kv[..., D:]


def _cache(c_cache, c_scale, k_cache, dev):
    """The arguments that a checked cache makes: pointers, page size, strides, pages."""
    _gpu(c_cache, "c_cache", _E4M3, dev)
    shape = c_cache.shape
    if len(shape) != 3 or shape[2] != R:
        raise ValueError(f"c_cache must be [pages, page_size, {R}], got {list(shape)}")
    pages, size, _ = shape
    _gpu(c_scale, "c_scale", _U8, dev, (pages, size, R // BLOCK))
    _gpu(k_cache, "k_cache", _BF16, dev, (pages, size, S))
    c, e, s = c_cache.stride(), c_scale.stride(), k_cache.stride()
    if pages > 1:
        if c[1:] != (R, 1) or e[1:] != (R // BLOCK, 1) or s[1:] != (S, 1):
            raise ValueError("c_cache, c_scale, k_cache: pages must be compact inside")
        return (c_cache.data_ptr(), c_scale.data_ptr(), k_cache.data_ptr(), size, c[0], e[0], s[0], pages)
    if pages and not (c_cache.is_contiguous() and c_scale.is_contiguous() and k_cache.is_contiguous()):
        raise ValueError("c_cache, c_scale, k_cache: pages must be compact inside")
    return (c_cache.data_ptr(), c_scale.data_ptr(), k_cache.data_ptr(), size, size * R, size * (R // BLOCK), size * S,
            pages)


def latent_cache_store(c, k_shared, c_cache, c_scale, k_cache, slots):
    """Store new tokens' latents c [T,512] and shared key parts k_shared [T,64],
    bf16 (rows may be slices of wider ones), in the paged cache: c_cache
    float8_e4m3fn [pages,page_size,512], c_scale uint8 [pages,page_size,4] (value =
    code * 2**(scale - 127), one for each 128 values) and k_cache bf16
    [pages,page_size,64], updated in place (outer strides may be padded).  slots int32
    [T]: page * page_size + offset per token; one outside the cache (-1 among them) is
    not stored."""
    dev = _first(c, "c", _BF16, 2)
    T = c.shape[0]
    cs, ss = _rows(c, "c", dev, (T, R)), _rows(k_shared, "k_shared", dev, (T, S))
    cache = _cache(c_cache, c_scale, k_cache, dev)
    _dense(slots, "slots", _I32, dev, (T,))
    _call(dev, "kda_latent_cache_store", c.data_ptr(), k_shared.data_ptr(), cs, ss, slots.data_ptr(), T, *cache)


def latent_cache_load(c_cache, c_scale, k_cache, page_table, cu_seqlens, num_tokens, c=None, k_shared=None):
    """Cached tokens back to bf16, the sequences packed: row cu_seqlens[n] + i of
    the results is token i of sequence n.  The cache as latent_cache_store leaves it,
    page_table int32 [N,W] (rows may be slices of wider ones), cu_seqlens int32 [N+1],
    not decreasing, num_tokens rows.  A token without a page gives zeros; rows behind
    the last sequence are not written.  Returns (c [num_tokens,512], k_shared
    [num_tokens,64])."""
    dev = _first(c_cache, "c_cache", _E4M3, 3)
    cache = _cache(c_cache, c_scale, k_cache, dev)
    N = _offsets(cu_seqlens, "cu_seqlens", dev)
    W, table_stride = _table(page_table, N, dev)
    if num_tokens < 0:
        raise ValueError("num_tokens must not be negative")
    if c is None:
        c = k_cache.new_empty((num_tokens, R))
    else:
        _dense(c, "c", _BF16, dev, (num_tokens, R))
    if k_shared is None:
        k_shared = k_cache.new_empty((num_tokens, S))
    else:
        _dense(k_shared, "k_shared", _BF16, dev, (num_tokens, S))
    _call(dev, "kda_latent_cache_load", *cache, page_table.data_ptr(), table_stride, W, cu_seqlens.data_ptr(), N,
          num_tokens, c.data_ptr(), k_shared.data_ptr())
    return c, k_shared


def latent_decode_workspace_size(N, Q, H):
    """Bytes of workspace latent_decode needs on the current device."""
    return int(_kda.load().kda_latent_decode_workspace_size(N, Q, H))


def latent_decode(q, c_cache, c_scale, k_cache, page_table, kv_lens, scale=None, out=None, lse=None, workspace=None):
    """Attention of Q new tokens of every sequence over the paged cache, in the
    absorbed form.  q [N,Q,H,576] bf16 (tokens may be slices of wider rows): 512
    against the latents, 64 against the shared parts; the cache as latent_cache_store
    leaves it, page_table int32 [N,W] (rows may be slices of wider ones), kv_lens int32
    [N]: tokens in the cache, the new ones included.  Query i stands at position
    kv_len - Q + i and sees the tokens up to there.  scale defaults to 192**-0.5, the
    expanded form's.  Returns (o [N,Q,H,512] bf16, the weighted latents, lse [N,Q,H]
    float32)."""
    dev = _first(q, "q", _BF16, 4)
    N, Q, H, _ = q.shape
    qs = _rows(q, "q", dev, (N, Q, H, R + S))
    cache = _cache(c_cache, c_scale, k_cache, dev)
    W, table_stride = _table(page_table, N, dev)
    _dense(kv_lens, "kv_lens", _I32, dev, (N,))
    if out is None:
        out = q.new_empty((N, Q, H, R))
    else:
        _dense(out, "out", _BF16, dev, (N, Q, H, R))
    if lse is None:
        lse = q.new_empty((N, Q, H), dtype=_F32)
    else:
        _dense(lse, "lse", _F32, dev, (N, Q, H))
    if workspace is None:
        workspace = _workspace(q, dev, latent_decode_workspace_size, N, Q, H)
    else:
        _dense(workspace, "workspace", _U8, dev)
    _call(dev, "kda_latent_decode", q.data_ptr(), qs, *cache, page_table.data_ptr(), table_stride, W,
          kv_lens.data_ptr(), N, Q, H, _scale(scale), out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
          workspace.numel())
    return out, lse
