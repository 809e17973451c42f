"""Refusals of the kda_latent_* entry points, without a GPU: every failing call
returns before any work is enqueued, and the binding names what is wrong."""

import ctypes

import pytest
import torch

import kda_gated_delta_amd as kda

NULL = ctypes.c_void_p(0)
FAKE = ctypes.c_void_p(0x1000)       # never dereferenced: every call below fails its checks first
OFF = ctypes.c_void_p(0x1008)
OFF2 = ctypes.c_void_p(0x1002)
OK, E_NULL, E_SHAPE, E_UNSUPPORTED, E_ALIGN, E_WORKSPACE = range(6)

LAYOUT = dict(q=FAKE, k=FAKE, s=FAKE, v=FAKE, qs=4 * 192, ks=4 * 256, kh=256, ss=64, vs=4 * 256, vh=256)
SIZES = dict(cu=NULL, cu_kv=NULL, n=0, B=1, T=64, K=100, H=4, scale=0.1)


def prefill(**kw):
    a = dict(**LAYOUT, **SIZES, o=FAKE, lse=NULL)
    a.update(kw)
    return kda.load().kda_latent_prefill(*a.values(), NULL)


def backward(**kw):
    a = dict(**LAYOUT, o=FAKE, lse=FAKE, up=FAKE, **SIZES, dq=FAKE, dkv=FAKE, ds=FAKE, dtype=1, ws=FAKE, wsb=1 << 60)
    a.update(kw)
    return kda.load().kda_latent_backward(*a.values(), NULL)


@pytest.mark.parametrize("call", [prefill, backward])
def test_prompt_sizes(call):
    assert call(T=0, K=0) == OK                               # nothing to do, and nothing is looked at
    assert call(T=-1) == E_SHAPE and call(K=-1) == E_SHAPE and call(B=0) == E_SHAPE
    assert call(H=0) == E_SHAPE and call(H=65536, qs=1 << 23) == E_SHAPE
    assert call(cu=FAKE) == E_SHAPE and call(cu_kv=FAKE, n=1) == E_SHAPE     # one kind of offsets without the other
    assert call(cu=FAKE, cu_kv=FAKE, n=0) == E_SHAPE and call(cu=FAKE, cu_kv=FAKE, n=2, B=2) == E_SHAPE
    assert call(qs=4 * 192 - 8) == E_SHAPE and call(qs=4 * 192 + 4) == E_ALIGN
    for name, least in (("ks", 128), ("vs", 128), ("ss", 64)):
        assert call(**{name: least - 8}) == E_SHAPE and call(**{name: least + 4}) == E_ALIGN
        assert call(**{name: (1 << 23) + 8}) == E_SHAPE and call(**{name: 0}) == E_SHAPE
    for name in ("kh", "vh"):
        assert call(**{name: -8}) == E_SHAPE and call(**{name: 12}) == E_ALIGN
        assert call(**{name: (1 << 40) + 8}) == E_SHAPE
    for scale in (0.0, -1.0, float("nan"), float("inf"), 2e30):
        assert call(scale=scale) == E_SHAPE
    # more workgroups than a launch holds
    assert call(B=1 << 20, T=1 << 16, H=4096, qs=1 << 20) == E_SHAPE


def test_more_keys_than_a_launch_holds():
    assert backward(B=1 << 20, K=1 << 16, H=4096, qs=1 << 20) == E_SHAPE


@pytest.mark.parametrize("call,names", [(prefill, "q k s v o"), (backward, "q k s v o lse up dq dkv ds ws")])
def test_prompt_pointers(call, names):
    for name in names.split():
        assert call(**{name: NULL}) == E_NULL, name
        assert call(**{name: OFF}) == E_ALIGN, name
    if call is prefill:
        assert call(lse=OFF) == E_ALIGN


def test_backward_dtype_and_workspace():
    assert backward(dtype=2) == E_UNSUPPORTED
    size = kda.latent_backward_workspace_size(1, 64, 100, 4)
    assert size == 2 * 64 * 4 * 4 + 4 * 100 * 64 * 4          # statistics, and the shared part's terms
    assert backward(wsb=size - 1) == E_WORKSPACE
    for bad in ((0, 64, 64, 4), (1, -1, 64, 4), (1, 64, -1, 4), (1, 64, 64, 0), (2, 64, 64, 4, 3), (1, 64, 64, 4, -1),
                (1, 0, 0, 4)):
        assert kda.latent_backward_workspace_size(*bad) == 0
    assert kda.latent_backward_workspace_size(1, 9, 0, 2) == 2 * 20 * 4 and kda.latent_backward_workspace_size(1, 0, 7, 2) == 2 * 7 * 64 * 4
    # shared key tiles: 1 KB per key, head and part, and the shared part's terms for each (256 compute units without a
    # device)
    more = kda.latent_backward_workspace_size(1, 8192, 8192, 2) - 8192 * 2 * 8
    part = 8192 * 2 * (1024 + 256)
    assert more > part and more % part == 0 and more // part <= 16
    assert kda.latent_backward_workspace_size(8, 8192, 8192, 16) == 8 * 8192 * 16 * (8 + 256)


CACHE = dict(cc=FAKE, cs=FAKE, kc=FAKE, P=64, cp=64 * 512, sp=64 * 4, kp=64 * 64, pages=7)


def store(**kw):
    a = dict(c=FAKE, s=FAKE, cstride=576, sstride=576, slots=FAKE, T=5, **CACHE)
    a.update(kw)
    return kda.load().kda_latent_cache_store(*a.values(), NULL)


def load(**kw):
    a = dict(**CACHE, table=FAKE, tstride=8, width=8, cu=FAKE, n=3, T=9, c=FAKE, s=FAKE)
    a.update(kw)
    return kda.load().kda_latent_cache_load(*a.values(), NULL)


def decode(**kw):
    a = dict(q=FAKE, qs=4 * 576, **CACHE, table=FAKE, tstride=8, width=8, lens=FAKE, N=3, Q=1, H=4, scale=0.1, o=FAKE,
             lse=NULL, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return kda.load().kda_latent_decode(*a.values(), NULL)


@pytest.mark.parametrize("call", [store, load, decode])
def test_cache_layout(call):
    for P in (0, 8, 100, 512):
        assert call(P=P, cp=1 << 20, sp=1 << 20, kp=1 << 20) == E_UNSUPPORTED
    assert call(cp=64 * 512 - 16) == E_SHAPE and call(cp=64 * 512 + 8) == E_ALIGN and call(cp=1 << 32) == E_SHAPE
    assert call(sp=64 * 4 - 4) == E_SHAPE and call(sp=64 * 4 + 2) == E_ALIGN and call(sp=1 << 32) == E_SHAPE
    assert call(kp=64 * 64 - 8) == E_SHAPE and call(kp=64 * 64 + 4) == E_ALIGN and call(kp=1 << 31) == E_SHAPE
    assert call(pages=-1) == E_SHAPE and call(pages=1 << 25) == E_SHAPE
    for name in ("cc", "cs", "kc"):
        assert call(**{name: NULL}) == E_NULL
    assert call(cc=OFF) == E_ALIGN and call(kc=OFF) == E_ALIGN and call(cs=OFF2) == E_ALIGN


def test_store_refusals():
    assert store(T=0) == OK and store(pages=0) == OK and store(T=-1) == E_SHAPE and store(T=1 << 30) == E_SHAPE
    assert store(cstride=504) == E_SHAPE and store(cstride=516) == E_ALIGN
    assert store(sstride=56) == E_SHAPE and store(sstride=68) == E_ALIGN
    for name in ("c", "s", "slots"):
        assert store(**{name: NULL}) == E_NULL
    assert store(c=OFF) == E_ALIGN and store(s=OFF) == E_ALIGN and store(slots=OFF2) == E_ALIGN


def test_load_refusals():
    assert load(T=0) == OK and load(T=-1) == E_SHAPE and load(T=1 << 30) == E_SHAPE
    assert load(n=0) == E_SHAPE and load(pages=0) == E_SHAPE and load(width=0) == E_SHAPE and load(tstride=7) == E_SHAPE
    for name in ("table", "cu", "c", "s"):
        assert load(**{name: NULL}) == E_NULL
    assert load(c=OFF) == E_ALIGN and load(s=OFF) == E_ALIGN and load(table=OFF2) == E_ALIGN and load(cu=OFF2) == E_ALIGN


def test_decode_refusals():
    assert decode(N=0) == OK and decode(N=-1) == E_SHAPE
    assert decode(Q=0) == E_SHAPE and decode(Q=1025) == E_SHAPE and decode(N=1 << 14, Q=1024) == E_SHAPE
    assert decode(H=0) == E_SHAPE and decode(H=65536, qs=1 << 30) == E_SHAPE
    assert decode(qs=4 * 576 - 8) == E_SHAPE and decode(qs=4 * 576 + 4) == E_ALIGN and decode(qs=(1 << 31) + 8) == E_SHAPE
    assert decode(pages=0) == E_SHAPE and decode(width=0) == E_SHAPE and decode(tstride=7) == E_SHAPE
    assert decode(width=(1 << 24) + 1, tstride=1 << 25) == E_SHAPE
    assert decode(scale=float("nan")) == E_SHAPE and decode(scale=0.0) == E_SHAPE
    for name in ("q", "table", "lens", "o", "ws"):
        assert decode(**{name: NULL}) == E_NULL
    for name in ("q", "o", "ws"):
        assert decode(**{name: OFF}) == E_ALIGN
    for name in ("table", "lens", "lse"):
        assert decode(**{name: OFF2}) == E_ALIGN
    size = kda.latent_decode_workspace_size(3, 1, 4)
    assert size > 0 and decode(wsb=size - 1) == E_WORKSPACE
    for bad in ((0, 1, 4), (3, 0, 4), (3, 1, 0), (3, 1025, 4)):
        assert kda.latent_decode_workspace_size(*bad) == 0


def test_binding_refuses_host_tensors():
    z = torch.zeros(1, 4, 2, 192, dtype=torch.bfloat16)
    k, s = z[..., :128], torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        kda.latent_prefill(z, k, s, k)
    with pytest.raises(ValueError, match="GPU"):
        kda.latent_backward(z, k, s, k, k, k, k)
    with pytest.raises(ValueError, match="grad_dtype"):
        kda.latent_backward(z, k, s, k, k, k, k, grad_dtype="half")
    with pytest.raises(TypeError, match="q must be"):
        kda.latent_prefill(z.float(), k, s, k)
    with pytest.raises(ValueError, match="GPU"):
        kda.latent_cache_store(s[0], s[0], z, z, z, i)
    with pytest.raises(TypeError, match="c_cache must be"):
        kda.latent_cache_load(z, z, z, i[None], i, 4)
    with pytest.raises(TypeError, match="Tensor"):
        kda.latent_decode(None, z, z, z, i[None], i)
