"""Refusals of the block-sparse operators that need no GPU: wrong shapes, types, layouts and sizes are
reported before anything is launched, by the Python API and by the C ABI."""

import ctypes

import pytest
import torch

from free_sparse_attention_reuse_b200 import _lib, api

E4M3 = torch.float8_e4m3fn


def bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def f32(*s):
    return torch.zeros(*s)


def i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


def rotary(q=None, k=None, v=None, pos=None, axes=(32, 32), **kw):
    q = bf(1, 8, 2, 64) if q is None else q
    return api.rotary(q, k, v, i32(8, len(axes)) if pos is None else pos, axes, **kw)


@pytest.mark.parametrize("kw,says", [
    (dict(q=bf(8, 2, 64)), "4-d"),
    (dict(q=f32(1, 8, 2, 64)), "must be torch.bfloat16"),
    (dict(q=bf(1, 8, 2, 64).transpose(2, 3)), "consecutive|axes"),
    (dict(q=bf(1, 8, 2, 68)[..., :64]), "multiples of 8"),
    (dict(k=bf(1, 7, 2, 64)), "k must have shape"),
    (dict(k=bf(1, 8, 1, 64), v=bf(1, 8, 2, 64)), "v must have shape"),
    (dict(axes=(32, 34)), "even sizes"),
    (dict(axes=(31, 1)), "even sizes"),
    (dict(axes=()), "even sizes"),
    (dict(axes=(8,) * 5, pos=i32(8, 5)), "even sizes"),
    (dict(axes=(10, 10), pairs="halves"), "multiple of 16"),
    (dict(pairs="other"), "pairs"),
    (dict(norm="layer"), "norm"),
    (dict(pos=i32(8, 3)), "pos must have shape"),
    (dict(pos=i32(8, 2).long()), "pos must be"),
    (dict(q_weight=f32(64)), "need norm"),
    (dict(norm="head", q_weight=f32(2, 64)), "q_weight must have shape"),
    (dict(norm="token", q_weight=f32(64)), "q_weight must have shape"),
    (dict(norm="head", q_weight=f32(64), k=bf(1, 8, 2, 64), k_weight=bf(64)), "one dtype"),
    (dict(out=(bf(1, 2, 8, 64), bf(1, 2, 8, 64), None)), "exactly where"),
    (dict(out=(bf(1, 8, 2, 64), None, None)), "Q must have shape"),
    (dict(), "CUDA"),
])
def test_rotary_refuses(kw, says):
    with pytest.raises(ValueError, match=says):
        rotary(**kw)


@pytest.mark.parametrize("call,says", [
    (lambda: api.block_means(bf(1, 2, 64, 64), 48), "BK"),
    (lambda: api.block_means(bf(1, 2, 64, 64), 32, kv_len=i32(2)), "kv_len"),
    (lambda: api.block_means(bf(1, 2, 64, 64), 32, means=f32(1, 2, 1, 64)), "means"),
    (lambda: api.block_means(bf(1, 2, 64, 64).transpose(1, 2), 32), "contiguous"),
    (lambda: api.block_means(bf(1, 2, 64, 64), 32), "CUDA"),
    (lambda: api.block_topk(bf(1, 2, 64, 64), f32(1, 2, 4, 64), 8, 2, 32), "C must"),
    (lambda: api.block_topk(bf(1, 3, 64, 64), f32(1, 2, 4, 64), 64, 2, 32), "divide"),
    (lambda: api.block_topk(bf(1, 2, 64, 64), f32(1, 2, 4, 64), 64, 5, 32), "kb"),
    (lambda: api.block_topk(bf(1, 2, 64, 64), f32(1, 2, 4, 64), 64, 0, 32), "kb"),
    (lambda: api.block_topk(bf(1, 2, 64, 64), f32(1, 2, 4, 128), 64, 2, 32), "means"),
    (lambda: api.block_topk(bf(1, 2, 64, 64), f32(1, 2, 4, 64).bfloat16(), 64, 2, 32), "means"),
    (lambda: api.block_topk(bf(1, 2, 64, 64), f32(1, 2, 4, 64), 64, 2, 32, blocks=i32(1, 2, 1, 3)), "blocks"),
    (lambda: api.block_topk(bf(1, 2, 64, 64), f32(1, 2, 4, 64), 64, 2, 32), "CUDA"),
])
def test_selection_refuses(call, says):
    with pytest.raises(ValueError, match=says):
        call()


def attn(q=None, k=None, v=None, ids=None, C=64, BK=32, **kw):
    q = bf(1, 2, 64, 64) if q is None else q
    k = bf(1, 2, 96, 64) if k is None else k
    return api.block_attn(q, k, k if v is None else v, ids, C, BK, **kw)


@pytest.mark.parametrize("kw,says", [
    (dict(q=f32(1, 2, 64, 64)), "Q must be"),
    (dict(k=f32(1, 2, 96, 64)), "K must be"),
    (dict(v=bf(1, 2, 95, 64)), "V must have shape"),
    (dict(k=bf(1, 2, 96, 128)), "K must have shape"),
    (dict(k=bf(2, 2, 96, 64)), "K must have shape"),
    (dict(q=bf(1, 3, 64, 64)), "divide"),
    (dict(C=32), "C must"),
    (dict(BK=16), "BK must"),
    (dict(k_scale=f32(1, 2, 3)), "8-bit"),
    (dict(k=f32(1, 2, 96, 64).to(E4M3)), "k_scale"),
    (dict(k=f32(1, 2, 90, 64).to(E4M3), k_scale=f32(1, 2, 3), v_scale=f32(1, 2, 3)), "whole blocks"),
    (dict(k=f32(1, 2, 96, 64).to(E4M3), k_scale=f32(1, 2, 2), v_scale=f32(1, 2, 3)), "k_scale"),
    (dict(ids=i32(1, 2, 3)), "4-d"),
    (dict(ids=i32(1, 2, 2, 1)), "blocks must have shape"),
    (dict(ids=i32(1, 2, 1, 4)), "1 to 3"),
    (dict(ids=i32(1, 2, 1, 0)), "1 to 3"),
    (dict(ids=i32(1, 2, 1, 2).long()), "blocks must be"),
    (dict(kv_len=i32(1).long()), "kv_len"),
    (dict(R=bf(1, 2, 63, 64)), "R must"),
    (dict(out=bf(1, 2, 63, 64)), "out must"),
    (dict(lse=f32(1, 2, 63)), "lse must"),
    (dict(), "CUDA"),
])
def test_block_attn_refuses(kw, says):
    with pytest.raises((ValueError, TypeError), match=says):
        attn(**kw)


def test_outputs_apart_from_inputs():
    x = bf(2, 2, 64, 64)
    with pytest.raises(ValueError, match="share"):
        api._apart(dict(out=x), dict(Q=x))
    with pytest.raises(ValueError, match="share"):
        api._apart(dict(out=x[:1]), dict(Q=x.transpose(0, 1)))
    api._apart(dict(out=x[:1], lse=None), dict(Q=x[1:], R=None))


@pytest.mark.parametrize("kw,says", [
    (dict(start=16), "multiples"), (dict(start=-32), "multiples"), (dict(start=96), "multiples"),
    (dict(K8=f32(1, 2, 112, 64).to(E4M3)), "multiples|V8"), (dict(ks=f32(1, 2, 3)), "k_scale"),
    (dict(means=f32(1, 2, 4, 32)), "means"), (dict(lens=i32(3)), "lens"), (dict(V=bf(1, 2, 63, 64)), "V must"),
    (dict(K8=bf(1, 2, 128, 64)), "K8"), (dict(), "CUDA"),
])
def test_cache_write_refuses(kw, says):
    a = dict(K=bf(1, 2, 64, 64), V=bf(1, 2, 64, 64), K8=f32(1, 2, 128, 64).to(E4M3), V8=f32(1, 2, 128, 64).to(E4M3),
             ks=f32(1, 2, 4), vs=f32(1, 2, 4), start=0, means=None, lens=None)
    a.update(kw)
    with pytest.raises(ValueError, match=says):
        api.cache_write(a["K"], a["V"], a["K8"], a["V8"], a["ks"], a["vs"], 32, start=a["start"], means=a["means"],
                        lens=a["lens"])


def test_cache_refuses():
    for cap in (0, 100, -64):
        with pytest.raises(ValueError, match="capacity"):
            api.KVCache(1, 2, cap, 64, BK=64, device="cpu")
    for bad in ((1, 2, 128, 96), (0, 2, 128, 64), (1, 0, 128, 64)):
        with pytest.raises(ValueError, match="need d"):
            api.KVCache(*bad, BK=64, device="cpu")
    c = api.KVCache(1, 2, 128, 64, BK=64, device="cpu")
    with pytest.raises(ValueError, match="K must have shape"):
        c.append(bf(1, 1, 4, 64), bf(1, 1, 4, 64))
    with pytest.raises(ValueError, match="fit"):
        c.append(bf(1, 2, 129, 64), bf(1, 2, 129, 64))
    assert c.length == 0


# ------------------------------------------------------------------------------------------ C ABI
P = ctypes.c_void_p(4096)  # 16- and 256-byte aligned, never dereferenced: every call below is refused first


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def status(rc):
    return _lib.STATUS_NAMES[rc]


def shape(B=1, H=2, Hkv=2, Nq=64, Nk=96, d=64):
    return _lib.BlockShape(B, H, Hkv, Nq, Nk, d, 0.0)


@pytest.mark.parametrize("change,want", [
    (dict(s=shape(B=0)), "INVALID_ARG"), (dict(s=shape(Nq=0)), "INVALID_ARG"), (dict(s=shape(Nk=0)), "INVALID_ARG"),
    (dict(s=shape(d=96)), "SHAPE"), (dict(s=shape(H=3)), "SHAPE"), (dict(s=shape(Nk=1 << 25)), "SHAPE"),
    (dict(s=shape(B=300, H=300, Hkv=300)), "SHAPE"), (dict(C=32), "SHAPE"), (dict(BK=48), "SHAPE"),
    (dict(kb=0), "INVALID_ARG"), (dict(kb=4), "INVALID_ARG"), (dict(blocks=None, kb=2), "INVALID_ARG"),
    (dict(fmt=2), "INVALID_ARG"), (dict(fmt=1), "INVALID_ARG"), (dict(ks=P), "INVALID_ARG"),
    (dict(fmt=1, ks=P, vs=P, s=shape(Nk=90)), "SHAPE"), (dict(Q=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"),
    (dict(Q=ctypes.c_void_p(4104)), "DTYPE_ALIGN"), (dict(R=ctypes.c_void_p(4104)), "DTYPE_ALIGN"),
    (dict(lse=ctypes.c_void_p(4098)), "DTYPE_ALIGN"), (dict(ws=None), "WORKSPACE"), (dict(ws_bytes=0), "WORKSPACE"),
    (dict(ws=ctypes.c_void_p(4112)), "DTYPE_ALIGN"),
])
def test_block_attn_abi(lib, change, want):
    a = dict(s=shape(), Q=P, fmt=0, ks=None, vs=None, blocks=P, C=64, BK=32, kb=2, R=None, out=P, lse=None, ws=P,
             ws_bytes=1 << 30)
    a.update(change)
    i32p = ctypes.POINTER(ctypes.c_int32)
    blocks = None if a["blocks"] is None else ctypes.cast(a["blocks"], i32p)
    rc = lib.mcs_block_attn(a["s"], a["Q"], P, P, a["fmt"], a["ks"], a["vs"], blocks, a["C"], a["BK"], a["kb"], None,
                            a["R"], a["out"], a["lse"], a["ws"], a["ws_bytes"], None)
    assert want in status(rc)


def test_sizes_abi(lib):
    assert lib.mcs_block_attn_workspace_size(shape(), 64, 32, 2) > 0
    assert lib.mcs_block_attn_workspace_size(shape(d=32), 64, 32, 2) == 0
    assert lib.mcs_block_attn_workspace_size(shape(), 64, 32, 4) == 0
    assert lib.mcs_block_topk_workspace_size(shape(), 64, 32) > 0
    assert lib.mcs_block_topk_workspace_size(shape(Nk=32 * 24576), 1, 32) > 0
    assert lib.mcs_block_topk_workspace_size(shape(Nk=32 * 24576 + 1), 1, 32) == 0
