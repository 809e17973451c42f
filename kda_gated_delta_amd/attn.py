"""Binding of the full-attention entry points (include/kda.h, kda_attn_*):
what a hybrid model runs in the layers between its KDA layers.

As in the rest of the binding, these functions check arguments, allocate
outputs that are not passed, and call the library; there is no arithmetic and
no fallback here.  They launch on the current stream of their tensors' device.
"""

import torch

import kda_gated_delta_amd as _kda

D = 128
_BF16, _F32, _I32, _E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


def _gpu(t, name, dtype, shape=None, dev=None):
    """t: a tensor of this dtype (and shape, and device) on a GPU."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t


def _dense(t, name, dtype, shape, dev):
    _gpu(t, name, dtype, shape, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _rows(t, name, heads, lead):
    """Elements from token to token of t [*lead, heads, 128]: heads compact,
    tokens evenly spaced over all leading axes (a slice of a wider row, say)."""
    if t.dim() != len(lead) + 2 or tuple(t.shape) != (*lead, heads, D):
        raise ValueError(f"{name} must be {[*lead, heads, D]}, got {list(t.shape)}")
    s = t.stride()
    if t.numel() == 0:
        return heads * D
    if s[-1] != 1 or (heads > 1 and s[-2] != D):
        raise ValueError(f"{name}: the last two axes must be compact")
    step, expect = None, None
    for size, stride in zip(reversed(lead), reversed(s[:-2])):
        if size == 1:
            continue
        if step is None:
            step, expect = stride, stride * size
        elif stride == expect:
            expect = stride * size
        else:
            raise ValueError(f"{name}: tokens must be evenly spaced")
    return heads * D if step is None else step


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _call(dev, name, *args):
    """Call an entry point with dev current, on its current stream."""
    fn = getattr(_kda.load(), name)
    if torch.cuda.current_device() == dev.index:
        code = fn(*args, torch.cuda.current_stream(dev).cuda_stream)
    else:
        with torch.cuda.device(dev):
            code = fn(*args, torch.cuda.current_stream(dev).cuda_stream)
    if code:
        _kda._check(code, name)


def _scale(scale):
    return D ** -0.5 if scale is None else float(scale)


def _prompt(q, k, v, cu_seqlens):
    _gpu(q, "q", _BF16)
    if q.dim() != 4:
        raise ValueError(f"q must be [B, T, HQ, {D}], got {list(q.shape)}")
    dev, (B, T, HQ, _) = q.device, q.shape
    _gpu(k, "k", _BF16, dev=dev)
    _gpu(v, "v", _BF16, dev=dev)
    HKV = k.shape[2] if k.dim() == 4 else 0
    strides = _rows(q, "q", HQ, (B, T)), _rows(k, "k", HKV, (B, T)), _rows(v, "v", HKV, (B, T))
    N = 0
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1:
            raise ValueError("cu_seqlens must have 1 dim")
        _dense(cu_seqlens, "cu_seqlens", _I32, tuple(cu_seqlens.shape), dev)
        N = cu_seqlens.shape[0] - 1
    return dev, (B, T, HQ, HKV), strides, N


def attn_prefill(q, k, v, cu_seqlens=None, scale=None, out=None, lse=None):
    """Causal attention over whole prompts.  q [B,T,HQ,128], k and v
    [B,T,HKV,128] bf16 (tokens may be slices of wider rows); query head h reads
    key/value head h // (HQ // HKV).  cu_seqlens int32 [N+1] (with B == 1):
    packed sequences; rows outside them are neither read nor written.  scale
    defaults to 128**-0.5.  Returns (o [B,T,HQ,128] bf16, lse [B,HQ,T] float32,
    the logarithm of each row's sum of exponentials)."""
    dev, (B, T, HQ, HKV), (qs, ks, vs), N = _prompt(q, k, v, cu_seqlens)
    out = torch.empty((B, T, HQ, D), dtype=_BF16, device=dev) if out is None else _dense(out, "out", _BF16, (B, T, HQ, D), dev)
    lse = torch.empty((B, HQ, T), dtype=_F32, device=dev) if lse is None else _dense(lse, "lse", _F32, (B, HQ, T), dev)
    _call(dev, "kda_attn_prefill", _ptr(q), _ptr(k), _ptr(v), qs, ks, vs, _ptr(cu_seqlens), N, B, T, HQ, HKV, D,
          _scale(scale), _ptr(out), _ptr(lse))
    return out, lse


def attn_backward_workspace_size(B, T, HQ, HKV, num_seqs=0):
    """Bytes of workspace attn_backward needs (num_seqs = 0 without cu_seqlens)."""
    return int(_kda.load().kda_attn_backward_workspace_size(B, T, HQ, HKV, D, num_seqs))


def attn_backward(q, k, v, o, lse, d_out, cu_seqlens=None, scale=None, workspace=None, grad_dtype="input"):
    """Gradients of sum(o * d_out) for attn_prefill with the same inputs, of
    which o and lse are the outputs.  d_out [B,T,HQ,128] bf16.  Returns (dq, dk,
    dv), bf16 (grad_dtype "input") or float32 ("float32")."""
    if grad_dtype not in ("input", "float32"):
        raise ValueError("grad_dtype must be 'input' or 'float32'")
    dev, (B, T, HQ, HKV), (qs, ks, vs), N = _prompt(q, k, v, cu_seqlens)
    _dense(o, "o", _BF16, (B, T, HQ, D), dev)
    _dense(d_out, "d_out", _BF16, (B, T, HQ, D), dev)
    _dense(lse, "lse", _F32, (B, HQ, T), dev)
    if workspace is None:
        workspace = torch.empty(max(attn_backward_workspace_size(B, T, HQ, HKV, N), 16), dtype=torch.uint8, device=dev)
    _dense(workspace, "workspace", torch.uint8, tuple(workspace.shape), dev)
    dtype = _BF16 if grad_dtype == "input" else _F32
    dq = torch.empty((B, T, HQ, D), dtype=dtype, device=dev)
    dk = torch.empty((B, T, HKV, D), dtype=dtype, device=dev)
    dv = torch.empty((B, T, HKV, D), dtype=dtype, device=dev)
    _call(dev, "kda_attn_backward", _ptr(q), _ptr(k), _ptr(v), qs, ks, vs, _ptr(o), _ptr(lse), _ptr(d_out),
          _ptr(cu_seqlens), N, B, T, HQ, HKV, D, _scale(scale), _ptr(dq), _ptr(dk), _ptr(dv),
          _kda.GRAD_INPUT_DTYPE if grad_dtype == "input" else _kda.GRAD_FLOAT32, _ptr(workspace), workspace.numel())
    return dq, dk, dv


def attn_tables(cached_lens, new_lens, page_table, free_pages, free_head, page_size, num_tokens, cu_seqlens=None,
                slots=None, kv_lens=None, next_head=None):
    """The tables of one serving step, made on the GPU.  cached_lens, new_lens
    int32 [N]: tokens of each request in the cache and in this step; page_table
    int32 [N, W] (rows may be slices of wider ones), updated in place with pages
    taken from free_pages int32 [F] from place free_head (int32 [1], or None for
    0) on, in the order of the requests; num_tokens: room for new tokens.
    Returns (cu_seqlens [N+1], slots [num_tokens], kv_lens [N], next_head [1]),
    all int32: packed offsets, page * page_size + offset per new token (-1:
    behind the last, or no page), lengths with this step's tokens, and the next
    call's free_head (past F: that many pages were missing)."""
    _gpu(cached_lens, "cached_lens", _I32)
    if cached_lens.dim() != 1:
        raise ValueError("cached_lens must have 1 dim")
    dev, N = cached_lens.device, cached_lens.shape[0]
    _dense(cached_lens, "cached_lens", _I32, (N,), dev)
    _dense(new_lens, "new_lens", _I32, (N,), dev)
    if page_table.dim() != 2:
        raise ValueError("page_table must have 2 dims")
    W = page_table.shape[1]
    _gpu(page_table, "page_table", _I32, (N, W), dev)
    if W > 1 and page_table.stride(1) != 1:
        raise ValueError("page_table rows must be compact")
    _dense(free_pages, "free_pages", _I32, (free_pages.numel(),), dev)
    if free_head is not None:
        _dense(free_head, "free_head", _I32, (1,), dev)
    def made(t, name, n):
        return torch.empty(n, dtype=_I32, device=dev) if t is None else _dense(t, name, _I32, (n,), dev)
    cu_seqlens, slots = made(cu_seqlens, "cu_seqlens", N + 1), made(slots, "slots", num_tokens)
    kv_lens, next_head = made(kv_lens, "kv_lens", N), made(next_head, "next_head", 1)
    _call(dev, "kda_attn_tables", _ptr(cached_lens), _ptr(new_lens), N, _ptr(page_table),
          page_table.stride(0) if N > 1 else W, W, _ptr(free_pages), free_pages.numel(), _ptr(free_head), page_size,
          num_tokens, _ptr(cu_seqlens), _ptr(slots), _ptr(kv_lens), _ptr(next_head))
    return cu_seqlens, slots, kv_lens, next_head


def _cache(k_cache, v_cache, k_scale, v_scale, dev, HKV):
    """(pages, page size, elements from page to page) of a checked cache."""
    _gpu(k_cache, "k_cache", _E4M3, dev=dev)
    if k_cache.dim() != 4 or k_cache.shape[1] != HKV or k_cache.shape[3] != D:
        raise ValueError(f"k_cache must be [pages, {HKV}, page_size, {D}], got {list(k_cache.shape)}")
    pages, _, size, _ = shape = tuple(k_cache.shape)
    _gpu(v_cache, "v_cache", _E4M3, shape, dev)
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if t.stride()[1:] != (size * D, D, 1) or (pages > 1 and t.stride(0) != k_cache.stride(0)):
            raise ValueError(f"{name}: pages must be compact inside and evenly spaced, keys' and values' alike")
    _dense(k_scale, "k_scale", _F32, (pages, HKV), dev)
    _dense(v_scale, "v_scale", _F32, (pages, HKV), dev)
    return pages, size, k_cache.stride(0) if pages > 1 else HKV * size * D


def attn_cache_store(k, v, k_cache, v_cache, k_scale, v_scale, slots):
    """Store new keys and values k, v [T,HKV,128] bf16 (tokens may be slices of
    wider rows) in the paged cache: k_cache, v_cache float8_e4m3fn
    [pages,HKV,page_size,128] (outer stride may be padded) and k_scale, v_scale
    float32 [pages,HKV], updated in place.  slots int32 [T]: page * page_size +
    offset per token; one outside the cache (-1 among them) is not stored."""
    _gpu(k, "k", _BF16)
    if k.dim() != 3:
        raise ValueError(f"k must be [T, HKV, {D}], got {list(k.shape)}")
    dev, (T, HKV, _) = k.device, k.shape
    _gpu(v, "v", _BF16, dev=dev)
    ks, vs = _rows(k, "k", HKV, (T,)), _rows(v, "v", HKV, (T,))
    pages, size, stride = _cache(k_cache, v_cache, k_scale, v_scale, dev, HKV)
    _dense(slots, "slots", _I32, (T,), dev)
    _call(dev, "kda_attn_cache_store", _ptr(k), _ptr(v), ks, vs, _ptr(slots), T, HKV, D, _ptr(k_cache), _ptr(v_cache),
          _ptr(k_scale), _ptr(v_scale), size, stride, pages)


def attn_decode_workspace_size(N, Q, HQ, HKV):
    """Bytes of workspace attn_decode needs."""
    return int(_kda.load().kda_attn_decode_workspace_size(N, Q, HQ, HKV, D))


def attn_decode(q, k_cache, v_cache, k_scale, v_scale, page_table, kv_lens, scale=None, out=None, lse=None,
                workspace=None):
    """Attention of Q new tokens of every sequence over the paged cache.  q
    [N,Q,HQ,128] bf16 (tokens may be slices of wider rows), the cache as
    attn_cache_store leaves it, page_table int32 [N,W] (rows may be slices of
    wider ones), kv_lens int32 [N]: tokens in the cache, the new ones included.
    Query i stands at position kv_len - Q + i and sees the tokens up to there.
    Returns (o [N,Q,HQ,128] bf16, lse [N,Q,HQ] float32)."""
    _gpu(q, "q", _BF16)
    if q.dim() != 4:
        raise ValueError(f"q must be [N, Q, HQ, {D}], got {list(q.shape)}")
    dev, (N, Q, HQ, _) = q.device, q.shape
    qs = _rows(q, "q", HQ, (N, Q))
    HKV = k_cache.shape[1] if isinstance(k_cache, torch.Tensor) and k_cache.dim() == 4 else 0
    pages, size, stride = _cache(k_cache, v_cache, k_scale, v_scale, dev, HKV)
    if page_table.dim() != 2:
        raise ValueError("page_table must have 2 dims")
    W = page_table.shape[1]
    _gpu(page_table, "page_table", _I32, (N, W), dev)
    if W > 1 and page_table.stride(1) != 1:
        raise ValueError("page_table rows must be compact")
    _dense(kv_lens, "kv_lens", _I32, (N,), dev)
    out = torch.empty((N, Q, HQ, D), dtype=_BF16, device=dev) if out is None else _dense(out, "out", _BF16, (N, Q, HQ, D), dev)
    lse = torch.empty((N, Q, HQ), dtype=_F32, device=dev) if lse is None else _dense(lse, "lse", _F32, (N, Q, HQ), dev)
    if workspace is None:
        workspace = torch.empty(max(attn_decode_workspace_size(N, Q, HQ, HKV), 16), dtype=torch.uint8, device=dev)
    _dense(workspace, "workspace", torch.uint8, tuple(workspace.shape), dev)
    _call(dev, "kda_attn_decode", _ptr(q), qs, _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), size, stride,
          pages, _ptr(page_table), page_table.stride(0) if N > 1 else W, W, _ptr(kv_lens), N, Q, HQ, HKV, D,
          _scale(scale), _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel())
    return out, lse
