"""Refusals of the kda_attn_* entry points, without a GPU: every failing call
returns before any work is enqueued, and the binding names what is wrong."""

import ctypes

import pytest
import torch

import kda_gated_delta_amd as kda

NULL = ctypes.c_void_p(0)
FAKE = ctypes.c_void_p(0x1000)       # never dereferenced: every call below fails its checks first
OFF = ctypes.c_void_p(0x1008)
OK, E_NULL, E_SHAPE, E_UNSUPPORTED, E_ALIGN, E_WORKSPACE = range(6)


def prefill(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, qs=512, ks=256, vs=256, cu=NULL, n=0, B=1, T=64, HQ=4, HKV=2, D=128, scale=0.1,
             o=FAKE, lse=NULL)
    a.update(kw)
    return kda.load().kda_attn_prefill(*a.values(), NULL)


def backward(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, qs=512, ks=256, vs=256, o=FAKE, lse=FAKE, up=FAKE, cu=NULL, n=0, B=1, T=64, HQ=4,
             HKV=2, D=128, scale=0.1, dq=FAKE, dk=FAKE, dv=FAKE, dtype=1, ws=FAKE, wsb=1 << 60)
    a.update(kw)
    return kda.load().kda_attn_backward(*a.values(), NULL)


@pytest.mark.parametrize("call", [prefill, backward])
def test_prompt_sizes(call):
    assert call(T=0) == OK                                    # nothing to do, and nothing is looked at
    assert call(T=-1) == E_SHAPE and call(B=0) == E_SHAPE
    assert call(HQ=3) == E_SHAPE and call(HQ=0, HKV=0) == E_SHAPE and call(HKV=0) == E_SHAPE
    assert call(HQ=65536, HKV=1, qs=1 << 23) == E_SHAPE
    assert call(D=64) == E_UNSUPPORTED
    assert call(cu=FAKE, n=0) == E_SHAPE and call(cu=FAKE, n=2, B=2) == E_SHAPE
    assert call(qs=504) == E_SHAPE and call(ks=128) == E_SHAPE and call(vs=255) == E_SHAPE
    assert call(qs=516) == E_ALIGN and call(ks=260) == E_ALIGN and call(vs=260) == E_ALIGN
    assert call(ks=(1 << 23) + 8) == E_SHAPE
    for scale in (0.0, -1.0, float("nan"), float("inf"), 2e30):
        assert call(scale=scale) == E_SHAPE
    # more workgroups than a launch holds
    assert call(B=1 << 20, T=1 << 16, HQ=4096, HKV=1, qs=1 << 20) == E_SHAPE


@pytest.mark.parametrize("call,names", [(prefill, "q k v o"), (backward, "q k v o lse up dq dk dv ws")])
def test_prompt_pointers(call, names):
    for name in names.split():
        assert call(**{name: NULL}) == E_NULL, name
        assert call(**{name: OFF}) == E_ALIGN, name
    if call is prefill:
        assert call(lse=OFF) == E_ALIGN


def test_backward_dtype_and_workspace():
    assert backward(dtype=2) == E_UNSUPPORTED
    size = kda.attn_backward_workspace_size(1, 64, 4, 2)
    assert size == 2 * 64 * 4 * 4
    assert backward(wsb=size - 1) == E_WORKSPACE
    for bad in ((0, 64, 4, 2), (1, -1, 4, 2), (1, 64, 3, 2), (1, 64, 0, 0), (2, 64, 4, 2, 3), (1, 64, 4, 2, -1)):
        assert kda.attn_backward_workspace_size(*bad) == 0
    assert kda.load().kda_attn_backward_workspace_size(1, 64, 4, 2, 64, 0) == 0
    # shared key tiles: 1 KB per token, head and part beside the statistics (256 compute units without a device)
    more = kda.attn_backward_workspace_size(1, 8192, 16, 4) - 8192 * 16 * 8
    assert more > 0 and more % (8192 * 4 * 1024) == 0 and more // (8192 * 4 * 1024) <= 16
    assert kda.attn_backward_workspace_size(8, 8192, 16, 16) == 8 * 8192 * 16 * 8


def tables(**kw):
    a = dict(old=FAKE, new=ctypes.c_void_p(0x2000), N=4, table=FAKE, stride=8, width=8, free=FAKE, F=3, head=NULL, P=64,
             tokens=9, cu=FAKE, slots=FAKE, lens=ctypes.c_void_p(0x3000), next=FAKE)
    a.update(kw)
    return kda.load().kda_attn_tables(*a.values(), NULL)


def test_tables_refusals():
    for bad in (dict(N=0), dict(N=8193), dict(width=0), dict(stride=7), dict(F=-1), dict(tokens=-1)):
        assert tables(**bad) == E_SHAPE, bad
    for P in (0, 8, 48, 512, -16):
        assert tables(P=P) == E_UNSUPPORTED
    for name in ("old", "new", "table", "free", "cu", "slots", "lens", "next"):
        assert tables(**{name: NULL}) == E_NULL, name
    assert tables(lens=FAKE) == E_SHAPE and tables(lens=ctypes.c_void_p(0x2000)) == E_SHAPE
    assert tables(head=FAKE) == E_SHAPE                       # next_head must not be free_head


def store(**kw):
    a = dict(k=FAKE, v=FAKE, ks=256, vs=256, slots=FAKE, T=5, HKV=2, D=128, kc=FAKE, vc=FAKE, kscale=FAKE, vscale=FAKE,
             P=64, stride=2 * 64 * 128, pages=7)
    a.update(kw)
    return kda.load().kda_attn_cache_store(*a.values(), NULL)


def decode(**kw):
    a = dict(q=FAKE, qs=512, kc=FAKE, vc=FAKE, kscale=FAKE, vscale=FAKE, P=64, stride=2 * 64 * 128, pages=7, table=FAKE,
             tstride=8, width=8, lens=FAKE, N=3, Q=1, HQ=4, HKV=2, D=128, scale=0.1, o=FAKE, lse=NULL, ws=FAKE,
             wsb=1 << 40)
    a.update(kw)
    return kda.load().kda_attn_decode(*a.values(), NULL)


@pytest.mark.parametrize("call", [store, decode])
def test_cache_layout(call):
    for P in (0, 8, 100, 512):
        assert call(P=P, stride=1 << 20) == E_UNSUPPORTED
    assert call(stride=2 * 64 * 128 - 16) == E_SHAPE and call(stride=2 * 64 * 128 + 8) == E_ALIGN
    assert call(stride=(1 << 32) + 16) == E_SHAPE
    assert call(pages=-1) == E_SHAPE and call(pages=1 << 25) == E_SHAPE
    assert call(HKV=0) == E_SHAPE and call(D=256) == E_UNSUPPORTED
    for name in ("kc", "vc", "kscale", "vscale"):
        assert call(**{name: NULL}) == E_NULL
    assert call(kc=OFF) == E_ALIGN and call(vc=OFF) == E_ALIGN


def test_store_refusals():
    assert store(T=0) == OK and store(pages=0) == OK and store(T=-1) == E_SHAPE
    assert store(ks=248) == E_SHAPE and store(vs=260) == E_ALIGN
    for name in ("k", "v", "slots"):
        assert store(**{name: NULL}) == E_NULL
    assert store(k=OFF) == E_ALIGN and store(v=OFF) == E_ALIGN
    assert store(T=2 ** 31 - 1, HKV=65535, ks=1 << 23, vs=1 << 23, P=16, stride=1 << 30) == E_SHAPE


def test_decode_refusals():
    assert decode(N=0) == OK and decode(N=-1) == E_SHAPE
    assert decode(Q=0) == E_SHAPE and decode(Q=1025) == E_SHAPE and decode(N=1 << 20, Q=1024) == E_SHAPE
    assert decode(HQ=5) == E_SHAPE and decode(qs=504) == E_SHAPE and decode(qs=516) == E_ALIGN
    assert decode(pages=0) == E_SHAPE and decode(width=0) == E_SHAPE and decode(tstride=7) == E_SHAPE
    assert decode(width=(1 << 24) + 1, tstride=1 << 25) == E_SHAPE
    assert decode(scale=float("nan")) == E_SHAPE and decode(scale=0.0) == E_SHAPE
    for name in ("q", "table", "lens", "o", "ws"):
        assert decode(**{name: NULL}) == E_NULL
    for name in ("q", "o", "ws"):
        assert decode(**{name: OFF}) == E_ALIGN
    size = kda.attn_decode_workspace_size(3, 1, 4, 2)
    assert size > 0 and decode(wsb=size - 1) == E_WORKSPACE
    for bad in ((0, 1, 4, 2), (3, 0, 4, 2), (3, 1, 5, 2), (3, 1025, 4, 2)):
        assert kda.attn_decode_workspace_size(*bad) == 0


def test_binding_refuses_host_tensors():
    z = torch.zeros(1, 4, 2, 128, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        kda.attn_prefill(z, z, z)
    with pytest.raises(ValueError, match="GPU"):
        kda.attn_backward(z, z, z, z, z, z)
    with pytest.raises(ValueError, match="grad_dtype"):
        kda.attn_backward(z, z, z, z, z, z, grad_dtype="half")
    with pytest.raises(TypeError, match="q must be"):
        kda.attn_prefill(z.float(), z, z)
    with pytest.raises(ValueError, match="GPU"):
        kda.attn_tables(i, i, i[None], i, None, 16, 4)
    with pytest.raises(ValueError, match="GPU"):
        kda.attn_cache_store(z[0], z[0], z, z, z, z, i)
    with pytest.raises(TypeError, match="Tensor"):
        kda.attn_decode(None, z, z, z, z, i[None], i)
