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


def _wrong(t, name, dtype, shape, dev):
    """Raise what is wrong with t."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


# The checks run before every launch, also of the smallest ones: each is one
# expression, and what is wrong is looked for only when something is.
def _first(t, name, dtype, dims):
    """Device index of the tensor that the others have to agree with."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or not t.is_cuda:
        _wrong(t, name, dtype, None, None)
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dims, got {list(t.shape)}")
    return t.get_device()


def _gpu(t, name, dtype, dev, shape=None):
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev
            and (shape is None or t.shape == shape)):
        _wrong(t, name, dtype, shape, dev)


def _dense(t, name, dtype, dev, shape=None):
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev
            and (shape is None or t.shape == shape) and t.is_contiguous()):
        _wrong(t, name, dtype, shape, dev)


def _rows(t, name, heads, lead):
    """Elements from token to token of t [*lead, heads, 128]: heads compact,
    tokens evenly spaced over all leading axes (a slice of a wider row, say)."""
    if t.shape != (*lead, heads, D):
        raise ValueError(f"{name} must be {[*lead, heads, D]}, got {list(t.shape)}")
    if t.is_contiguous():
        return heads * D
    s = t.stride()
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
    """Call an entry point with device `dev` current, on its current stream."""
    fn = getattr(_kda.load(), name)
    stream = torch._C._cuda_getCurrentRawStream(dev)
    if torch._C._cuda_getDevice() == dev:                  # (a GPU tensor was made: the runtime is up)
        code = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            code = fn(*args, stream)
    if code:
        _kda._check(code, name)


def _workspace(like, dev, size, *sizes):
    """Workspace for a call on device `dev`, whose compute units its size follows."""
    if torch._C._cuda_getDevice() == dev:
        n = size(*sizes)
    else:
        with torch.cuda.device(dev):
            n = size(*sizes)
    return like.new_empty(max(n, 16), dtype=torch.uint8)


def _scale(scale):
    return D ** -0.5 if scale is None else float(scale)


def _prompt(q, k, v, cu_seqlens):
    dev = _first(q, "q", _BF16, 4)
    B, T, HQ, _ = q.shape
    _gpu(k, "k", _BF16, dev)
    _gpu(v, "v", _BF16, dev)
    HKV = k.shape[2] if k.dim() == 4 else 0
    strides = _rows(q, "q", HQ, (B, T)), _rows(k, "k", HKV, (B, T)), _rows(v, "v", HKV, (B, T))
    if cu_seqlens is None:
        return dev, B, T, HQ, HKV, strides, 0
    _dense(cu_seqlens, "cu_seqlens", _I32, dev)
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
        raise ValueError("cu_seqlens must be [N + 1]")
    return dev, B, T, HQ, HKV, strides, cu_seqlens.shape[0] - 1


def attn_prefill(q, k, v, cu_seqlens=None, scale=None, out=None, lse=None):
    """Causal attention over whole prompts.  q [B,T,HQ,128], k and v
    [B,T,HKV,128] bf16 (tokens may be slices of wider rows); query head h reads
    key/value head h // (HQ // HKV).  cu_seqlens int32 [N+1] (with B == 1):
    packed sequences, in any order; rows outside them are neither read nor
    written (and hold anything in outputs that are allocated here).  scale
    defaults to 128**-0.5.  Returns (o [B,T,HQ,128] bf16, lse [B,HQ,T] float32,
    the logarithm of each row's sum of exponentials)."""
    dev, B, T, HQ, HKV, (qs, ks, vs), N = _prompt(q, k, v, cu_seqlens)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _dense(out, "out", _BF16, dev, (B, T, HQ, D))
    if lse is None:
        lse = q.new_empty((B, HQ, T), dtype=_F32)
    else:
        _dense(lse, "lse", _F32, dev, (B, HQ, T))
    _call(dev, "kda_attn_prefill", q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs, _ptr(cu_seqlens), N, B, T,
          HQ, HKV, D, _scale(scale), out.data_ptr(), lse.data_ptr())
    return out, lse


def attn_backward_workspace_size(B, T, HQ, HKV, num_seqs=0):
    """Bytes of workspace attn_backward needs on the current device (num_seqs = 0
    without cu_seqlens)."""
    return int(_kda.load().kda_attn_backward_workspace_size(B, T, HQ, HKV, D, num_seqs))


def attn_backward(q, k, v, o, lse, d_out, cu_seqlens=None, scale=None, workspace=None, grad_dtype="input"):
    """Gradients of sum(o * d_out) for attn_prefill with the same inputs, of
    which o and lse are the outputs.  d_out [B,T,HQ,128] bf16.  Returns (dq, dk,
    dv), bf16 (grad_dtype "input") or float32 ("float32"); rows outside the
    sequences hold anything."""
    if grad_dtype not in ("input", "float32"):
        raise ValueError("grad_dtype must be 'input' or 'float32'")
    dev, B, T, HQ, HKV, (qs, ks, vs), N = _prompt(q, k, v, cu_seqlens)
    _dense(o, "o", _BF16, dev, (B, T, HQ, D))
    _dense(d_out, "d_out", _BF16, dev, (B, T, HQ, D))
    _dense(lse, "lse", _F32, dev, (B, HQ, T))
    if workspace is None:
        workspace = _workspace(q, dev, attn_backward_workspace_size, B, T, HQ, HKV, N)
    else:
        _dense(workspace, "workspace", torch.uint8, dev)
    dtype = _BF16 if grad_dtype == "input" else _F32
    dq = q.new_empty((B, T, HQ, D), dtype=dtype)
    dk = q.new_empty((B, T, HKV, D), dtype=dtype)
    dv = q.new_empty((B, T, HKV, D), dtype=dtype)
    _call(dev, "kda_attn_backward", q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs, o.data_ptr(),
          lse.data_ptr(), d_out.data_ptr(), _ptr(cu_seqlens), N, B, T, HQ, HKV, D, _scale(scale),
          dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
          _kda.GRAD_INPUT_DTYPE if grad_dtype == "input" else _kda.GRAD_FLOAT32, workspace.data_ptr(),
          workspace.numel())
    return dq, dk, dv


def _table(page_table, N, dev):
    """(entries of a row, entries from row to row) of a checked page table."""
    _gpu(page_table, "page_table", _I32, dev)
    if page_table.dim() != 2 or page_table.shape[0] != N:
        raise ValueError(f"page_table must be [{N}, W], got {list(page_table.shape)}")
    W = page_table.shape[1]
    if W > 1 and page_table.stride(1) != 1:
        raise ValueError("page_table rows must be compact")
    return W, page_table.stride(0) if N > 1 else W


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
    dev = _first(cached_lens, "cached_lens", _I32, 1)
    N = cached_lens.shape[0]
    _dense(cached_lens, "cached_lens", _I32, dev)
    _dense(new_lens, "new_lens", _I32, dev, (N,))
    W, table_stride = _table(page_table, N, dev)
    _dense(free_pages, "free_pages", _I32, dev)
    if free_head is not None:
        _dense(free_head, "free_head", _I32, dev, (1,))
    if cu_seqlens is None and slots is None and kv_lens is None and next_head is None:
        cu_seqlens, slots, kv_lens, next_head = cached_lens.new_empty(2 * N + 2 + num_tokens).split_with_sizes(
            (N + 1, num_tokens, N, 1))
    else:
        def made(t, name, n):
            if t is None:
                return cached_lens.new_empty(n)
            _dense(t, name, _I32, dev, (n,))
            return t
        cu_seqlens, slots = made(cu_seqlens, "cu_seqlens", N + 1), made(slots, "slots", num_tokens)
        kv_lens, next_head = made(kv_lens, "kv_lens", N), made(next_head, "next_head", 1)
    _call(dev, "kda_attn_tables", cached_lens.data_ptr(), new_lens.data_ptr(), N, page_table.data_ptr(),
          table_stride, W, free_pages.data_ptr(), free_pages.numel(), _ptr(free_head), page_size,
          num_tokens, cu_seqlens.data_ptr(), slots.data_ptr(), kv_lens.data_ptr(), next_head.data_ptr())
    return cu_seqlens, slots, kv_lens, next_head


def _cache(k_cache, v_cache, k_scale, v_scale, dev, HKV):
    """(pages, page size, elements from page to page) of a checked cache."""
    _gpu(k_cache, "k_cache", _E4M3, dev)
    shape = k_cache.shape
    if len(shape) != 4 or shape[1] != HKV or shape[3] != D:
        raise ValueError(f"k_cache must be [pages, {HKV}, page_size, {D}], got {list(shape)}")
    pages, _, size, _ = shape
    _gpu(v_cache, "v_cache", _E4M3, dev, shape)
    stride = k_cache.stride()
    if stride[1:] != (size * D, D, 1) or v_cache.stride() != stride:
        raise ValueError("k_cache, v_cache: pages must be compact inside and evenly spaced, keys' and values' alike")
    _dense(k_scale, "k_scale", _F32, dev, (pages, HKV))
    _dense(v_scale, "v_scale", _F32, dev, (pages, HKV))
    return pages, size, stride[0] if pages > 1 else HKV * size * D


def attn_cache_store(k, v, k_cache, v_cache, k_scale, v_scale, slots):
    """Store new keys and values k, v [T,HKV,128] bf16 (tokens may be slices of
    wider rows) in the paged cache: k_cache, v_cache float8_e4m3fn
    [pages,HKV,page_size,128] (outer stride may be padded) and k_scale, v_scale
    float32 [pages,HKV], updated in place.  slots int32 [T]: page * page_size +
    offset per token; one outside the cache (-1 among them) is not stored."""
    dev = _first(k, "k", _BF16, 3)
    T, HKV, _ = k.shape
    _gpu(v, "v", _BF16, dev)
    ks, vs = _rows(k, "k", HKV, (T,)), _rows(v, "v", HKV, (T,))
    pages, size, stride = _cache(k_cache, v_cache, k_scale, v_scale, dev, HKV)
    _dense(slots, "slots", _I32, dev, (T,))
    _call(dev, "kda_attn_cache_store", k.data_ptr(), v.data_ptr(), ks, vs, slots.data_ptr(), T, HKV, D,
          k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), size, stride, pages)


def attn_decode_workspace_size(N, Q, HQ, HKV):
    """Bytes of workspace attn_decode needs on the current device."""
    return int(_kda.load().kda_attn_decode_workspace_size(N, Q, HQ, HKV, D))


def attn_decode(q, k_cache, v_cache, k_scale, v_scale, page_table, kv_lens, scale=None, out=None, lse=None,
                workspace=None):
    """Attention of Q new tokens of every sequence over the paged cache.  q
    [N,Q,HQ,128] bf16 (tokens may be slices of wider rows), the cache as
    attn_cache_store leaves it, page_table int32 [N,W] (rows may be slices of
    wider ones), kv_lens int32 [N]: tokens in the cache, the new ones included.
    How the work is laid out follows W and the cache's size, which the host knows,
    not the lengths: a table no wider than the longest sequence needs is fastest
    for short ones.  Query i stands at position kv_len - Q + i and sees the tokens up to there.
    Returns (o [N,Q,HQ,128] bf16, lse [N,Q,HQ] float32)."""
    dev = _first(q, "q", _BF16, 4)
    N, Q, HQ, _ = q.shape
    qs = _rows(q, "q", HQ, (N, Q))
    HKV = k_cache.shape[1] if isinstance(k_cache, torch.Tensor) and k_cache.dim() == 4 else 0
    pages, size, stride = _cache(k_cache, v_cache, k_scale, v_scale, dev, HKV)
    W, table_stride = _table(page_table, N, dev)
    _dense(kv_lens, "kv_lens", _I32, dev, (N,))
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _dense(out, "out", _BF16, dev, (N, Q, HQ, D))
    if lse is None:
        lse = k_scale.new_empty((N, Q, HQ))
    else:
        _dense(lse, "lse", _F32, dev, (N, Q, HQ))
    if workspace is None:
        workspace = _workspace(q, dev, attn_decode_workspace_size, N, Q, HQ, HKV)
    else:
        _dense(workspace, "workspace", torch.uint8, dev)
    _call(dev, "kda_attn_decode", q.data_ptr(), qs, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
          v_scale.data_ptr(), size, stride, pages, page_table.data_ptr(), table_stride, W, kv_lens.data_ptr(), N, Q,
          HQ, HKV, D, _scale(scale), out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.numel())
    return out, lse
