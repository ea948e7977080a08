"""Public Python API: thin wrappers over the C ABI (include/mcs.h), plus the anchor/reuse
schedule of MC-Sparse ("MC-Sparse가 확산 트랜스포머 희소 어텐션의 품질 격차를 좁힌다", section
무엇과 다른가: anchors are the last step of the dense warm-up or of a refresh interval; reuse
steps attend with the cached groups and indices and add the cached residual).

Tensors: Q, K, V bf16 [B, H, N, d] contiguous on a CUDA device; perm int32 [B, H, N];
idx int32 [B, H, N // C, k]; R bf16 [B, H, N, d].  Output tensors are allocated here with
torch when not given (the C library itself never allocates).
"""

from __future__ import annotations

from dataclasses import dataclass

import torch

from . import _lib
from ._lib import Shape, check, ptr, stream_ptr


def _shape(Q: torch.Tensor, scale=None) -> Shape:
    if Q.dim() != 4:
        raise ValueError("expected [B, H, N, d]")
    B, H, N, d = Q.shape
    return Shape(B, H, N, d, 0.0 if scale is None else float(scale))


def _spec(t, name: str, dtype, shape=None):
    """dtype, shape and layout of one tensor argument (where it lives is checked apart, so that
    a wrong shape is reported as such whatever the device)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _on_device(**tensors):
    """Every given tensor on the same CUDA device, the current one (the library launches there
    and the kernels dereference these pointers)."""
    dev = None
    for name, t in tensors.items():
        if t is None:
            continue
        if t.device.type != "cuda":
            raise ValueError(f"{name} must be a CUDA tensor")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, other arguments on {dev}")
    if dev is not None and dev.index != torch.cuda.current_device():
        raise ValueError(f"tensors are on {dev} but the current device is cuda:{torch.cuda.current_device()}")


def _req(t: torch.Tensor, dtype, name: str):
    _spec(t, name, dtype)
    _on_device(**{name: t})


def _qkv(Q, K, V=None, names=("Q", "K", "V")):
    """Q, K (and V) bf16 [B, H, N, d] of one shape; returns that shape."""
    if not isinstance(Q, torch.Tensor) or Q.dim() != 4:
        raise ValueError(f"{names[0]} must be a 4-d tensor [B, H, N, d]")
    shape = tuple(Q.shape)
    _spec(Q, names[0], torch.bfloat16, shape)
    _spec(K, names[1], torch.bfloat16, shape)
    if V is not None:
        _spec(V, names[2], torch.bfloat16, shape)
    return shape


def _groups(shape, C: int):
    """G = N // C, or None when C does not divide N (the library reports that as a shape error)."""
    N = shape[2]
    return N // C if isinstance(C, int) and C > 0 and N % C == 0 else None


def _meta(shape, C: int, perm=None, idx=None, R=None):
    """perm int32 [B, H, N], idx int32 [B, H, N // C, k], R bf16 like Q (each if given)."""
    B, H, N, _ = shape
    if perm is not None:
        _spec(perm, "perm", torch.int32, (B, H, N))
    G = _groups(shape, C)
    if idx is not None:
        if not isinstance(idx, torch.Tensor):
            raise TypeError("idx must be a torch.Tensor")
        if idx.dim() != 4 or (G is not None and tuple(idx.shape[:3]) != (B, H, G)):
            raise ValueError(f"idx must have shape {(B, H, G, 'k')}, got {tuple(idx.shape)}")
        _spec(idx, "idx", torch.int32)
    if R is not None:
        _spec(R, "R", torch.bfloat16, shape)


def workspace_size(Q: torch.Tensor, C: int, k: int, scale=None) -> int:
    return int(_lib.load().mcs_workspace_size(_shape(Q, scale), C, k))


def workspace(Q: torch.Tensor, C: int, k: int, scale=None) -> torch.Tensor:
    n = workspace_size(Q, C, k, scale)
    if n == 0:
        raise _lib.MCSError(2, "workspace_size: invalid shape")
    return torch.empty(n, dtype=torch.uint8, device=Q.device)


def dense_attn(Q, K, V, O=None, lse=None, want_out: bool = True, want_lse: bool = True, scale=None):
    """Dense attention; returns (O, lse).  want_out=False computes only the LSE; want_lse=False
    computes only O (lse is then None)."""
    B, H, N, d = shape = _qkv(Q, K, V)
    if want_out and O is None:
        O = torch.empty_like(Q)
    if want_lse and lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=Q.device)
    if not want_lse:
        lse = None
    if want_out:
        _spec(O, "O", torch.bfloat16, shape)
    if lse is not None:
        _spec(lse, "lse", torch.float32, (B, H, N))
    _on_device(Q=Q, K=K, V=V, O=O if want_out else None, lse=lse)
    check(_lib.load().mcs_dense_attn(_shape(Q, scale), ptr(Q), ptr(K), ptr(V), ptr(O if want_out else None),
                                     ptr(lse), stream_ptr()), "mcs_dense_attn")
    return O, lse


def group(Q, C: int, perm=None, ws=None, scale=None):
    """Fast PDDP grouping; returns perm int32 [B, H, N]."""
    if not isinstance(Q, torch.Tensor) or Q.dim() != 4:
        raise ValueError("Q must be a 4-d tensor [B, H, N, d]")
    _spec(Q, "Q", torch.bfloat16)
    B, H, N, d = shape = tuple(Q.shape)
    if perm is None:
        perm = torch.empty((B, H, N), dtype=torch.int32, device=Q.device)
    _meta(shape, C, perm=perm)
    _on_device(Q=Q, perm=perm)
    if ws is None:
        ws = workspace(Q, C, 1, scale)
    _spec(ws, "ws", torch.uint8)
    _on_device(Q=Q, ws=ws)
    check(_lib.load().mcs_group(_shape(Q, scale), ptr(Q), C, ptr(perm), ptr(ws), ws.numel(), stream_ptr()),
          "mcs_group")
    return perm


def select(Q, K, perm, C: int, k: int, lse=None, idx=None, ws=None, scale=None):
    """Exact two-pass top-k selection; returns idx int32 [B, H, N // C, k]."""
    B, H, N, d = shape = _qkv(Q, K)
    _meta(shape, C, perm=perm)
    if lse is not None:
        _spec(lse, "lse", torch.float32, (B, H, N))
    if idx is None:
        idx = torch.empty((B, H, N // C, k), dtype=torch.int32, device=Q.device)
    _meta(shape, C, idx=idx)
    if idx.shape[-1] != k:
        raise ValueError(f"idx must hold k = {k} indices per group, got {idx.shape[-1]}")
    _on_device(Q=Q, K=K, perm=perm, lse=lse, idx=idx)
    if ws is None:
        ws = workspace(Q, C, k, scale)
    _spec(ws, "ws", torch.uint8)
    _on_device(Q=Q, ws=ws)
    check(_lib.load().mcs_select(_shape(Q, scale), ptr(Q), ptr(K), ptr(perm), C, k, ptr(lse), ptr(idx), ptr(ws),
                                 ws.numel(), stream_ptr()), "mcs_select")
    return idx


def select_noalloc(Q, K, perm, C: int, k: int, lse, idx, scale=None):
    """mcs_select_noalloc: the same selection with no workspace and no device allocation in
    the library (its scratch is a fixed array inside libmcs.so); lse and idx must be given."""
    B, H, N, d = shape = _qkv(Q, K)
    _meta(shape, C, perm=perm, idx=idx)
    _spec(lse, "lse", torch.float32, (B, H, N))
    if idx.shape[-1] != k:
        raise ValueError(f"idx must hold k = {k} indices per group, got {idx.shape[-1]}")
    _on_device(Q=Q, K=K, perm=perm, lse=lse, idx=idx)
    check(_lib.load().mcs_select_noalloc(_shape(Q, scale), ptr(Q), ptr(K), ptr(perm), C, k, ptr(lse), ptr(idx),
                                         stream_ptr()), "mcs_select_noalloc")
    return idx


def sparse_attn(Q, K, V, perm, C: int, idx, R=None, out=None, scale=None):
    """Reuse step: SparseAttn(Q, K, V; perm, idx) + R."""
    shape = _qkv(Q, K, V)
    _meta(shape, C, perm=perm, idx=idx, R=R)
    k = idx.shape[-1]
    if out is None:
        out = torch.empty_like(Q)
    _spec(out, "out", torch.bfloat16, shape)
    _on_device(Q=Q, K=K, V=V, perm=perm, idx=idx, R=R, out=out)
    check(_lib.load().mcs_sparse_attn(_shape(Q, scale), ptr(Q), ptr(K), ptr(V), ptr(perm), C, ptr(idx), k, ptr(R),
                                      ptr(out), stream_ptr()), "mcs_sparse_attn")
    return out


def _req_host(t: torch.Tensor, name: str):
    if t.device.type != "cpu":
        raise ValueError(f"{name} must be a host (CPU) tensor")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be torch.bfloat16")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def host_staging(shape, heads_per_chunk: int = 2, device=None) -> torch.Tensor:
    """Device staging buffer for sparse_attn_host on [B, H, N, d] tensors of `shape`."""
    B, H, N, d = shape
    n = int(_lib.load().mcs_host_staging_size(Shape(B, H, N, d, 0.0), heads_per_chunk))
    if n == 0:
        raise _lib.MCSError(2, "host_staging_size: invalid shape or heads_per_chunk")
    return torch.empty(n, dtype=torch.uint8, device="cuda" if device is None else device)


def sparse_attn_host(hQ, hK, hV, perm, C: int, idx, R=None, out=None, heads_per_chunk: int = 2, staging=None,
                     scale=None):
    """Reuse step with Q, K, V and the output in host memory (pinned for overlap) and the
    cached perm, idx and R on the device; chunks of heads are copied in, computed and copied
    out on overlapping streams.  Returns `out` (a host tensor); it is complete once the
    current CUDA stream is synchronised, and the host tensors must stay alive until then."""
    shape = _qkv(hQ, hK, hV, names=("hQ", "hK", "hV"))
    _meta(shape, C, perm=perm, idx=idx, R=R)
    if out is not None:
        _spec(out, "out", torch.bfloat16, shape)
    for t, n in ((hQ, "hQ"), (hK, "hK"), (hV, "hV"), (out, "out")):
        if t is not None:
            _req_host(t, n)
    _on_device(perm=perm, idx=idx, R=R)
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, pin_memory=True)
    if staging is None:
        staging = host_staging(shape, heads_per_chunk, perm.device)
    _spec(staging, "staging", torch.uint8)
    _on_device(perm=perm, staging=staging)
    k = idx.shape[-1]
    check(_lib.load().mcs_sparse_attn_host(_shape(hQ, scale), ptr(hQ), ptr(hK), ptr(hV), ptr(perm), C, ptr(idx), k,
                                           ptr(R), ptr(out), heads_per_chunk, ptr(staging), staging.numel(),
                                           stream_ptr()), "mcs_sparse_attn_host")
    return out


def residual(Q, K, V, perm, C: int, idx, O_full, R=None, scale=None):
    """Anchor residual record: R = O_full - SparseAttn(Q, K, V; perm, idx)."""
    shape = _qkv(Q, K, V)
    _meta(shape, C, perm=perm, idx=idx)
    _spec(O_full, "O_full", torch.bfloat16, shape)
    k = idx.shape[-1]
    if R is None:
        R = torch.empty_like(Q)
    _meta(shape, C, R=R)
    _on_device(Q=Q, K=K, V=V, perm=perm, idx=idx, O_full=O_full, R=R)
    check(_lib.load().mcs_residual(_shape(Q, scale), ptr(Q), ptr(K), ptr(V), ptr(perm), C, ptr(idx), k,
                                   ptr(O_full), ptr(R), stream_ptr()), "mcs_residual")
    return R


def anchor(Q, K, V, C: int, k: int, ws=None, out=None, scale=None):
    """Whole anchor step; returns (O_full, perm, idx, R)."""
    B, H, N, d = shape = _qkv(Q, K, V)
    if out is None:
        O_full = torch.empty_like(Q)
        perm = torch.empty((B, H, N), dtype=torch.int32, device=Q.device)
        idx = torch.empty((B, H, N // C, k), dtype=torch.int32, device=Q.device)
        R = torch.empty_like(Q)
    else:
        O_full, perm, idx, R = out
    _spec(O_full, "O_full", torch.bfloat16, shape)
    _meta(shape, C, perm=perm, idx=idx, R=R)
    if idx.shape[-1] != k:
        raise ValueError(f"idx must hold k = {k} indices per group, got {idx.shape[-1]}")
    _on_device(Q=Q, K=K, V=V, O_full=O_full, perm=perm, idx=idx, R=R)
    if ws is None:
        ws = workspace(Q, C, k, scale)
    _spec(ws, "ws", torch.uint8)
    _on_device(Q=Q, ws=ws)
    check(_lib.load().mcs_anchor(_shape(Q, scale), ptr(Q), ptr(K), ptr(V), C, k, ptr(O_full), ptr(perm), ptr(idx),
                                 ptr(R), ptr(ws), ws.numel(), stream_ptr()), "mcs_anchor")
    return O_full, perm, idx, R


def select_blocks(Q, K, perm, C: int, BK: int, kb: int, method: str = "oracle", lse=None, idx=None, ws=None,
                  scale=None):
    """KV-block selection per group as token indices [B, H, N//C, kb*BK] (kb whole blocks of BK
    keys, ascending).  method "oracle": exact probability mass of each block (summed group
    scores); "bsa": mean-pooled query against mean-pooled block keys (vanilla BSA)."""
    if method not in ("oracle", "bsa"):
        raise ValueError(f"method must be 'oracle' or 'bsa', got {method!r}")
    B, H, N, d = shape = _qkv(Q, K)
    _meta(shape, C, perm=perm)
    if lse is not None:
        _spec(lse, "lse", torch.float32, (B, H, N))
    if idx is None:
        idx = torch.empty((B, H, N // C, kb * BK), dtype=torch.int32, device=Q.device)
    _meta(shape, C, idx=idx)
    if idx.shape[-1] != kb * BK:
        raise ValueError(f"idx must hold kb*BK = {kb * BK} indices per group, got {idx.shape[-1]}")
    _on_device(Q=Q, K=K, perm=perm, lse=lse, idx=idx)
    if ws is None:
        ws = workspace(Q, C, kb * BK, scale)
    _spec(ws, "ws", torch.uint8)
    _on_device(Q=Q, ws=ws)
    m = {"oracle": 0, "bsa": 1}[method]
    check(_lib.load().mcs_select_blocks(_shape(Q, scale), ptr(Q), ptr(K), ptr(perm), C, BK, kb, m, ptr(lse),
                                        ptr(idx), ptr(ws), ws.numel(), stream_ptr()), "mcs_select_blocks")
    return idx


def perquery_attn(Q, K, V, k: int, out=None, ws=None, scale=None):
    """Per-query oracle: each query attends to its own k keys of largest logit (renormalised)."""
    shape = _qkv(Q, K, V)
    if out is None:
        out = torch.empty_like(Q)
    _spec(out, "out", torch.bfloat16, shape)
    _on_device(Q=Q, K=K, V=V, out=out)
    if ws is None:
        n = int(_lib.load().mcs_perquery_workspace_size(_shape(Q, scale)))
        if n == 0:
            raise _lib.MCSError(2, "mcs_perquery_workspace_size: invalid shape")
        ws = torch.empty(n, dtype=torch.uint8, device=Q.device)
    _spec(ws, "ws", torch.uint8)
    _on_device(Q=Q, ws=ws)
    check(_lib.load().mcs_perquery_attn(_shape(Q, scale), ptr(Q), ptr(K), ptr(V), k, ptr(out), ptr(ws), ws.numel(),
                                        stream_ptr()), "mcs_perquery_attn")
    return out


def group_kmeans(Q, C: int, iters: int = 10, perm=None, ws=None, scale=None):
    """Grouping-cost baseline: equal-size groups from Lloyd's k-means (fp64); returns perm int32
    [B, H, N] laid out as group() lays it out."""
    if not isinstance(Q, torch.Tensor) or Q.dim() != 4:
        raise ValueError("Q must be a 4-d tensor [B, H, N, d]")
    _spec(Q, "Q", torch.bfloat16)
    B, H, N, d = shape = tuple(Q.shape)
    if perm is None:
        perm = torch.empty((B, H, N), dtype=torch.int32, device=Q.device)
    _meta(shape, C, perm=perm)
    _on_device(Q=Q, perm=perm)
    if ws is None:
        n = int(_lib.load().mcs_kmeans_workspace_size(_shape(Q, scale), C))
        if n == 0:
            raise _lib.MCSError(2, "mcs_kmeans_workspace_size: invalid shape")
        ws = torch.empty(n, dtype=torch.uint8, device=Q.device)
    _spec(ws, "ws", torch.uint8)
    _on_device(Q=Q, ws=ws)
    check(_lib.load().mcs_group_kmeans(_shape(Q, scale), ptr(Q), C, iters, ptr(perm), ptr(ws), ws.numel(),
                                       stream_ptr()), "mcs_group_kmeans")
    return perm


# ---------------------------------------------------------------- block-sparse attention without an anchor
E4M3 = torch.float8_e4m3fn
BLOCK_ROWS = (32, 64, 128)      # keys of a block
QUERY_ROWS = (1, 16, 64, 128)   # query rows that share a list

# Calls that passed every check, by what the checks look at (types, shapes, layout, devices and plain
# arguments; never an address): what the call needs beside its pointers.  These calls take as little as
# ten microseconds on the device, so a repeated one does not check the same shapes again.
_plans: dict = {}


def _lookup(*rest, tensors):
    """(key, plan) of a call: what the checks look at, hashable, and what passed for it before.  The key is
    None for a call that the checks have to see (an argument that is no tensor, or that cannot be a key)."""
    try:  # (`rest` holds numbers, strings and tuples of them: a tensor is equal to itself whatever it holds)
        k = rest + tuple([None if t is None else (t.dtype, t.shape, t.is_contiguous(), t.get_device()) for t in tensors])
        return k, _plans.get(k)
    except (AttributeError, TypeError):
        return None, None


def _keep(key, plan):
    if key is not None:
        if len(_plans) >= 512:
            _plans.clear()
        _plans[key] = plan
    return plan


def _here(t):
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"tensors are on {t.device} but the current device is cuda:{torch.cuda.current_device()}")


def _at(t):
    return None if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t):
    """The current stream's handle (without making a Stream object of it)."""
    return _raw_stream(t.get_device()) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream


# Stands in where a call writes no workspace (attention with one CTA to each list): 256 bytes a device, shared by
# every such call and so never handed to one that writes.
_blanks: dict = {}


def _workspace(ws, n: int, t, writes: bool = True):
    if ws is None:
        if writes:
            return t.new_empty(n, dtype=torch.uint8)
        ws = _blanks.get(t.get_device())
        if ws is None:
            ws = _blanks[t.get_device()] = torch.empty(256, dtype=torch.uint8, device=t.device)
        return ws
    _spec(ws, "ws", torch.uint8)
    if ws.device != t.device:
        raise ValueError(f"ws is on {ws.device}, other arguments on {t.device}")
    return ws


def _heads(t, name: str, dtype=torch.bfloat16):
    if not isinstance(t, torch.Tensor) or t.dim() != 4:
        raise ValueError(f"{name} must be a 4-d tensor [B, H, N, d]")
    _spec(t, name, dtype)
    return tuple(t.shape)


def _block_sizes(C=None, BK=None):
    if BK is not None and BK not in BLOCK_ROWS:
        raise ValueError(f"BK must be one of {BLOCK_ROWS}, got {BK!r}")
    if C is not None and C not in QUERY_ROWS:
        raise ValueError(f"C must be one of {QUERY_ROWS}, got {C!r}")


def _kv_heads(H: int, Hkv: int):
    if Hkv < 1 or H % Hkv:
        raise ValueError(f"the {Hkv} key/value heads must divide the {H} query heads")


def _strides(t):
    """Element strides of [B, N, H] (0 for a dimension of one entry, whose stride means nothing)."""
    return [0 if t.shape[i] == 1 else t.stride(i) for i in range(3)]


def _apart(outs: dict, ins: dict):
    """No output that the caller gives may share memory with an input or with another output: inputs are read
    after outputs have been written, and outputs are written in any order."""
    def span(t):
        n = 1 + sum((s - 1) * st for s, st in zip(t.shape, t.stride())) if t.numel() else 0
        return t.data_ptr(), t.data_ptr() + n * t.element_size()

    held = [(name, *span(t)) for name, t in ins.items() if t is not None]
    for name, t in outs.items():
        if t is None:
            continue
        lo, hi = span(t)
        for other, a, b in held:
            if lo < b and a < hi:
                raise ValueError(f"{name} must not share memory with {other}")
        held.append((name, lo, hi))


def _length(t, name: str, B: int):
    if t is not None:
        _spec(t, name, torch.int32, (B,))


def _number(x):
    """A scalar argument as a float: what a call is known by later has to be its value."""
    return None if x is None else float(x)


def _plan_rotary(q, k, v, pos, axes, theta, pairs, norm, q_weight, k_weight, eps, out):
    if pairs not in ("adjacent", "halves"):
        raise ValueError(f"pairs must be 'adjacent' or 'halves', got {pairs!r}")
    if norm not in (None, "head", "token"):
        raise ValueError(f"norm must be None, 'head' or 'token', got {norm!r}")
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a 4-d tensor [B, N, H, d]")
    B, N, H, d = q.shape
    Hkv = H
    for t, name in ((k, "k"), (v, "v")):
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or t.dim() != 4:
            raise ValueError(f"{name} must be a 4-d tensor [B, N, H, d]")
        Hkv = t.shape[2] if name == "k" or k is None else Hkv
        if tuple(t.shape) != (B, N, Hkv, d):
            raise ValueError(f"{name} must have shape {(B, N, Hkv, d)}, got {tuple(t.shape)}")
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if t is None:
            continue
        if t.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
        if t.stride(3) != 1 or any(x % 8 for x in _strides(t)):
            raise ValueError(f"{name} must have consecutive elements in a row and strides that are multiples of 8")
    if not 1 <= len(axes) <= 4 or any(a < 2 or a % 2 for a in axes) or sum(axes) > d:
        raise ValueError(f"axes must be one to four even sizes of at most {d} in all, got {axes}")
    if pairs == "halves" and sum(axes) % 16:
        raise ValueError("pairs='halves' needs the axes' sizes to sum to a multiple of 16")
    if not isinstance(pos, torch.Tensor) or pos.dtype not in (torch.int32, torch.float32):
        raise ValueError("pos must be an int32 or float32 tensor")
    if tuple(pos.shape) not in ((N, len(axes)), (B, N, len(axes))):
        raise ValueError(f"pos must have shape {(N, len(axes))} or {(B, N, len(axes))}, got {tuple(pos.shape)}")
    _spec(pos, "pos", pos.dtype)
    if norm is None and (q_weight is not None or k_weight is not None):
        raise ValueError("norm weights need norm='head' or norm='token'")
    wdt = None
    for w, name, heads in ((q_weight, "q_weight", H), (k_weight, "k_weight", Hkv)):
        if w is None:
            continue
        if not isinstance(w, torch.Tensor) or w.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError(f"{name} must be a float32 or bfloat16 tensor")
        if wdt is not None and w.dtype != wdt:
            raise ValueError("q_weight and k_weight must have one dtype")
        wdt = w.dtype
        _spec(w, name, wdt, (d,) if norm == "head" else (heads, d))
    shapes = [(B, H, N, d), None if k is None else (B, Hkv, N, d), None if v is None else (B, Hkv, N, d)]
    if out is not None:
        if len(out) != 3:
            raise ValueError(f"out must be (Q, K, V), got {len(out)} of them")
        for o, shape, name in zip(out, shapes, ("Q", "K", "V")):
            if (o is None) != (shape is None):
                raise ValueError(f"{name} must be given exactly where its input is")
            if o is not None:
                _spec(o, name, torch.bfloat16, shape)
    _on_device(q=q, k=k, v=v, pos=pos, q_weight=q_weight, k_weight=k_weight,
               **({} if out is None else dict(Q=out[0], K=out[1], V=out[2])))
    a = _lib.RotaryArgs(B=B, N=N, H=H, Hkv=Hkv, d=d, axes=len(axes), theta=theta, eps=eps,
                        pairs=int(pairs == "halves"), norm=(None, "head", "token").index(norm),
                        pos_is_float=int(pos.dtype == torch.float32), pos_per_batch=int(pos.dim() == 3),
                        weight_is_bf16=int(wdt == torch.bfloat16))
    for i, x in enumerate(axes):
        a.axis_dim[i] = x
    for i, t in enumerate((q, k, v)):
        if t is not None:
            a.stride[i][:] = _strides(t)
    return a, shapes


def rotary(q, k, v, pos, axes, theta: float = 10000.0, pairs: str = "adjacent", norm=None, q_weight=None,
           k_weight=None, eps: float = 1e-6, out=None):
    """A layer's projections to attention-ready tensors in one pass: RMS norm of q and k, rotary
    positions over several axes, and the change to head-major layout.

    q [B, N, H, d], k and v [B, N, Hkv, d]: bf16 views (for example the parts of a fused projection
    [B, N, 3, H, d]) with consecutive elements in a row; k and v may be None.  pos: int32 or fp32
    [N, A] or [B, N, A], a token's position on each of the A axes.  axes: how many of a row's d
    elements each axis turns (even; elements behind their sum stay).  theta: base of the
    frequencies.  pairs: "adjacent" (elements 2i, 2i+1) or "halves" (i, i + sum(axes)/2).  norm:
    None, "head" (over a row, weights [d]) or "token" (over all heads of a token, weights
    [heads, d]); weights fp32 or bf16, or None for ones.  Returns Q [B, H, N, d], K and V
    [B, Hkv, N, d] contiguous (None where the input is None); out = (Q, K, V) to reuse buffers."""
    given, axes, theta, eps = tuple(axes), tuple(map(int, axes)), _number(theta), _number(eps)
    if given != axes:
        raise ValueError(f"axes must be whole numbers, got {given}")
    # (q, k and v are views: their strides count)
    key, plan = _lookup("rotary", axes, theta, pairs, norm, eps, *[t.stride() for t in (q, k, v) if isinstance(t, torch.Tensor)],
                        tensors=(q, k, v, pos, q_weight, k_weight, *(out or ())))
    if plan is None:
        plan = _keep(key, _plan_rotary(q, k, v, pos, axes, theta, pairs, norm, q_weight, k_weight, eps, out))
    a, shapes = plan
    _here(q)
    if out is None:
        out = [None if s is None else q.new_empty(s) for s in shapes]
    else:
        _apart(dict(Q=out[0], K=out[1], V=out[2]), dict(q=q, k=k, v=v, pos=pos, q_weight=q_weight, k_weight=k_weight))
    Q, K, V = out
    check(_lib.load().mcs_rotary(a, _at(q), _at(k), _at(v), _at(pos), _at(q_weight), _at(k_weight), _at(Q), _at(K),
                                 _at(V), _stream(q)), "mcs_rotary")
    return Q, K, V


def _plan_means(K, BK, kv_len, means):
    B, H, N, d = _heads(K, "K")
    _block_sizes(BK=BK)
    _length(kv_len, "kv_len", B)
    shape = (B, H, -(-N // BK), d)
    if means is not None:
        _spec(means, "means", torch.float32, shape)
    _on_device(K=K, kv_len=kv_len, means=means)
    return Shape(B, H, N, d, 0.0), shape


def block_means(K, BK: int, kv_len=None, means=None):
    """Mean of the valid rows of every block of BK rows: fp32 [B, H, ceil(N / BK), d] (zero for a
    block without one).  kv_len: int32 [B], valid rows of each batch entry."""
    key, plan = _lookup("means", BK, tensors=(K, kv_len, means))
    s, shape = plan or _keep(key, _plan_means(K, BK, kv_len, means))
    _here(K)
    if means is None:
        means = K.new_empty(shape, dtype=torch.float32)
    else:
        _apart(dict(means=means), dict(K=K, kv_len=kv_len))
    check(_lib.load().mcs_block_means(s, _at(K), BK, _at(kv_len), _at(means), _stream(K)), "mcs_block_means")
    return means


def _plan_topk(Q, means, C, kb, BK, kv_len, blocks):
    B, H, Nq, d = _heads(Q, "Q")
    Hkv, nb = _heads(means, "means", torch.float32)[1:3]
    _spec(means, "means", torch.float32, (B, Hkv, nb, d))
    _kv_heads(H, Hkv)
    _block_sizes(C, BK)
    if not 1 <= kb <= nb:
        raise ValueError(f"kb must be in [1, {nb}], got {kb}")
    _length(kv_len, "kv_len", B)
    shape = (B, H, -(-Nq // C), kb)
    if blocks is not None:
        _spec(blocks, "blocks", torch.int32, shape)
    _on_device(Q=Q, means=means, kv_len=kv_len, blocks=blocks)
    s = _lib.BlockShape(B, H, Hkv, Nq, nb * BK, d, 0.0)
    n = int(_lib.load().mcs_block_topk_workspace_size(s, C, BK))
    if n == 0:
        raise _lib.MCSError(2, "mcs_block_topk_workspace_size: invalid shape")
    return s, shape, n


def block_topk(Q, means, C: int, kb: int, BK: int, kv_len=None, blocks=None, ws=None):
    """The kb key blocks of largest pooled score for every block of C query rows: int32
    [B, H, ceil(Nq / C), kb], ascending, -1 behind them where fewer blocks hold a valid key.

    means: fp32 [B, Hkv, nb, d] from block_means or cache_write.  score = (mean of the query rows) .
    (mean of the block's keys), ties to the lower block.  kv_len: int32 [B], valid keys; a block
    behind them is not a candidate."""
    key, plan = _lookup("topk", C, kb, BK, tensors=(Q, means, kv_len, blocks))
    s, shape, n = plan or _keep(key, _plan_topk(Q, means, C, kb, BK, kv_len, blocks))
    _here(Q)
    own, ws = ws is None, _workspace(ws, n, Q)
    if blocks is not None or not own:
        _apart(dict(blocks=blocks, ws=None if own else ws), dict(Q=Q, means=means, kv_len=kv_len))
    if blocks is None:
        blocks = Q.new_empty(shape, dtype=torch.int32)
    check(_lib.load().mcs_block_topk(s, _at(Q), _at(means), C, BK, kb, _at(kv_len), _at(blocks), _at(ws), ws.numel(),
                                     _stream(Q)), "mcs_block_topk")
    return blocks


def _plan_block_attn(Q, K, V, blocks, C, BK, R, kv_len, k_scale, v_scale, out, lse, scale):
    B, H, Nq, d = shape = _heads(Q, "Q")
    if not isinstance(K, torch.Tensor) or K.dtype not in (torch.bfloat16, E4M3):
        raise ValueError(f"K must be {torch.bfloat16} or {E4M3}")
    Hkv, Nk = _heads(K, "K", K.dtype)[1:3]
    _spec(K, "K", K.dtype, (B, Hkv, Nk, d))
    _spec(V, "V", K.dtype, (B, Hkv, Nk, d))
    _kv_heads(H, Hkv)
    _block_sizes(C, BK)
    nb = -(-Nk // BK)
    fp8 = K.dtype == E4M3
    if fp8:
        if Nk % BK:
            raise ValueError(f"an 8-bit cache holds whole blocks: {Nk} rows are no multiple of {BK}")
        _spec(k_scale, "k_scale", torch.float32, (B, Hkv, nb))
        _spec(v_scale, "v_scale", torch.float32, (B, Hkv, nb))
    elif k_scale is not None or v_scale is not None:
        raise ValueError("scales belong to 8-bit K and V")
    kb = nb
    if blocks is not None:
        if not isinstance(blocks, torch.Tensor) or blocks.dim() != 4:
            raise ValueError("blocks must be a 4-d tensor [B, H, ceil(Nq / C), kb]")
        kb = blocks.shape[-1]
        _spec(blocks, "blocks", torch.int32, (B, H, -(-Nq // C), kb))
        if not 1 <= kb <= nb:
            raise ValueError(f"blocks must list 1 to {nb} blocks, got {kb}")
    _length(kv_len, "kv_len", B)
    if R is not None:
        _spec(R, "R", torch.bfloat16, shape)
    if out is not None:
        _spec(out, "out", torch.bfloat16, shape)
    if lse is not None:
        _spec(lse, "lse", torch.float32, (B, H, Nq))
    _on_device(Q=Q, K=K, V=V, blocks=blocks, R=R, kv_len=kv_len, k_scale=k_scale, v_scale=v_scale, out=out, lse=lse)
    s = _lib.BlockShape(B, H, Hkv, Nq, Nk, d, 0.0 if scale is None else scale)
    n = int(_lib.load().mcs_block_attn_workspace_size(s, C, BK, kb))
    if n == 0:
        raise _lib.MCSError(2, "mcs_block_attn_workspace_size: invalid shape")
    return s, kb, n, int(fp8)


def block_attn(Q, K, V, blocks, C: int, BK: int, R=None, kv_len=None, k_scale=None, v_scale=None, out=None, lse=None,
               want_lse: bool = False, ws=None, scale=None):
    """Attention over the key blocks that each block of C query rows lists; returns (out, lse), lse
    None unless wanted.

    Q [B, H, Nq, d] bf16; K, V [B, Hkv, Nk, d] bf16, or float8_e4m3fn with k_scale and v_scale fp32
    [B, Hkv, Nk / BK].  blocks: int32 [B, H, ceil(Nq / C), kb] (a list ends at its first negative
    entry), or None for every block.  kv_len: int32 [B], valid keys of each batch entry.  R: bf16
    like Q, added to the result.  A row without a key gives R (0 without R) and lse = -inf."""
    scale = _number(scale)
    key, plan = _lookup("attn", C, BK, scale, tensors=(Q, K, V, blocks, R, kv_len, k_scale, v_scale, out, lse))
    s, kb, n, fp8 = plan or _keep(key, _plan_block_attn(Q, K, V, blocks, C, BK, R, kv_len, k_scale, v_scale,
                                                                   out, lse, scale))
    _here(Q)
    own, ws = ws is None, _workspace(ws, n, Q, writes=n > 256)  # (256: one part, joined with nothing)
    if out is not None or lse is not None or not own:
        _apart(dict(out=out, lse=lse, ws=None if own else ws), dict(Q=Q, K=K, V=V, R=R, blocks=blocks, kv_len=kv_len, k_scale=k_scale, v_scale=v_scale))
    if out is None:
        out = torch.empty_like(Q)
    if want_lse and lse is None:
        lse = Q.new_empty(Q.shape[:3], dtype=torch.float32)
    check(_lib.load().mcs_block_attn(s, _at(Q), _at(K), _at(V), fp8, _at(k_scale), _at(v_scale), _at(blocks), C, BK, kb,
                                     _at(kv_len), _at(R), _at(out), _at(lse), _at(ws), ws.numel(), _stream(Q)),
          "mcs_block_attn")
    return out, lse


def _plan_write(K, V, K8, V8, k_scale, v_scale, BK, start, means, lens):
    B, H, n, d = _heads(K, "K")
    _spec(V, "V", torch.bfloat16, (B, H, n, d))
    _block_sizes(BK=BK)
    cap = _heads(K8, "K8", E4M3)[2]
    _spec(K8, "K8", E4M3, (B, H, cap, d))
    _spec(V8, "V8", E4M3, (B, H, cap, d))
    if cap % BK or start % BK or start < 0 or start + n > cap:
        raise ValueError(f"rows [{start}, {start + n}) must lie in the store's {cap}, both multiples of BK = {BK}")
    _spec(k_scale, "k_scale", torch.float32, (B, H, cap // BK))
    _spec(v_scale, "v_scale", torch.float32, (B, H, cap // BK))
    if means is not None:
        _spec(means, "means", torch.float32, (B, H, cap // BK, d))
    _length(lens, "lens", B)
    _on_device(K=K, V=V, K8=K8, V8=V8, k_scale=k_scale, v_scale=v_scale, means=means, lens=lens)
    return Shape(B, H, n, d, 0.0), cap


def cache_write(K, V, K8, V8, k_scale, v_scale, BK: int, start: int = 0, means=None, lens=None):
    """Write K and V (bf16 [B, H, n, d]) into rows [start, start + n) of an 8-bit store K8, V8
    (float8_e4m3fn [B, H, capacity, d]) with one scale for each block of BK rows and head (fp32
    [B, H, capacity / BK]), and each block's mean key into means (fp32 [B, H, capacity / BK, d]) if
    given.  start and capacity are multiples of BK; a block's scale comes from this call's rows, so an
    unfinished block is lengthened by writing its rows again.  lens: int32 [B], valid rows of this
    call; rows behind them stay as they were.  No output may share memory with another or with an input."""
    key, plan = _lookup("write", BK, start, tensors=(K, V, K8, V8, k_scale, v_scale, means, lens))
    s, cap = plan or _keep(key, _plan_write(K, V, K8, V8, k_scale, v_scale, BK, start, means, lens))
    _here(K)
    status = _lib.load().mcs_cache_write(s, _at(K), _at(V), BK, start, cap, _at(lens), _at(K8), _at(V8), _at(k_scale),
                                         _at(v_scale), _at(means), _stream(K))
    if status == 1:  # (looked at there, where it costs nothing; here to say which)
        _apart(dict(K8=K8, V8=V8, k_scale=k_scale, v_scale=v_scale, means=means), dict(K=K, V=V, lens=lens))
    check(status, "mcs_cache_write")


class KVCache:
    """Keys and values of one layer in 8 bits, for attention from new frames or tokens to all earlier
    ones: e4m3 values, one scale per block of BK tokens and head, and each block's mean key, which
    scores the blocks without reading them.  All B sequences have one length.

    append() adds rows (an unfinished last block keeps its bf16 rows beside the store, so that it is
    quantised anew, with its own scale, whenever it grows); attend() runs attention over every
    block, or over the kb blocks that block_topk picks for each block of C query rows."""

    def __init__(self, B: int, Hkv: int, capacity: int, d: int, BK: int = 64, device=None):
        _block_sizes(BK=BK)
        if d not in (64, 128) or B < 1 or Hkv < 1:
            raise ValueError(f"need d of 64 or 128 and at least one batch entry and head, got d = {d}, B = {B}, Hkv = {Hkv}")
        if capacity < 1 or capacity % BK:
            raise ValueError(f"capacity must be a positive multiple of BK = {BK}, got {capacity}")
        dev = "cuda" if device is None else device
        self.B, self.Hkv, self.capacity, self.d, self.BK, self.length = B, Hkv, capacity, d, BK, 0
        self.K8, self.V8 = (torch.zeros((B, Hkv, capacity, d), dtype=torch.uint8, device=dev).view(E4M3) for _ in range(2))
        self.k_scale, self.v_scale = (torch.ones((B, Hkv, capacity // BK), device=dev) for _ in range(2))
        self.means = torch.zeros((B, Hkv, capacity // BK, d), device=dev)
        self.kv_len = torch.zeros(B, dtype=torch.int32, device=dev)
        # bf16 rows of the unfinished last block; held for good, since memory that one call gave back could be handed
        # out on its stream while the next call still reads it on another.  Flat, so that any number of them is
        # contiguous: as a slice of [B, Hkv, BK, d] they made an append of 1500 rows of 24 heads take 95 us, not 52
        self._open = tuple(torch.empty(B * Hkv * BK * d, dtype=torch.bfloat16, device=dev) for _ in range(2))

    def _open_rows(self, tail: int):
        """The first `tail` rows of the unfinished block's keys and values, [B, Hkv, tail, d] each."""
        return [o[:self.B * self.Hkv * tail * self.d].view(self.B, self.Hkv, tail, self.d) for o in self._open]

    def append(self, K, V):
        """Add K, V (bf16 [B, Hkv, n, d]) behind the rows held so far."""
        if torch.cuda.is_available() and torch.cuda.is_current_stream_capturing():
            raise ValueError("append() keeps its place on the host: a captured one would write the same rows again")
        n = _heads(K, "K")[2]
        shape = (self.B, self.Hkv, n, self.d)
        _spec(K, "K", torch.bfloat16, shape)
        _spec(V, "V", torch.bfloat16, shape)
        if self.length + n > self.capacity:
            raise ValueError(f"{n} more rows do not fit: {self.length} of {self.capacity} are held")
        if n == 0:
            return
        tail = self.length % self.BK
        if tail:
            K, V = (torch.cat([o, x], 2) for o, x in zip(self._open_rows(tail), (K, V)))
        cache_write(K, V, self.K8, self.V8, self.k_scale, self.v_scale, self.BK, start=self.length - tail,
                    means=self.means)
        self.length += n
        self.kv_len.fill_(self.length)
        tail = self.length % self.BK
        if tail:
            for o, x in zip(self._open_rows(tail), (K, V)):
                o.copy_(x[:, :, x.shape[2] - tail:])

    def attend(self, Q, C: int = 128, kb=None, R=None, want_lse: bool = False, scale=None):
        """(out, lse) of block_attn over the rows held; kb blocks per query block, or all of them."""
        blocks = None
        if kb is not None:
            blocks = block_topk(Q, self.means, C, kb, self.BK, kv_len=self.kv_len)
        return block_attn(Q, self.K8, self.V8, blocks, C, self.BK, R=R, kv_len=self.kv_len, k_scale=self.k_scale,
                          v_scale=self.v_scale, want_lse=want_lse, scale=scale)


def head_shard(n_heads: int, rank: int, world: int):
    """[lo, hi): the contiguous share of a layer's B*H heads that rank `rank` of `world`
    processes.  Every step of the path (grouping, selection, dense and sparse attention, the
    residual) works head by head, so a layer splits across GPUs by heads with no exchange; the
    first n_heads % world ranks take one head more."""
    if world < 1 or not 0 <= rank < world:
        raise ValueError("need 0 <= rank < world")
    base, extra = divmod(n_heads, world)
    lo = rank * base + min(rank, extra)
    return lo, lo + base + (1 if rank < extra else 0)


def sync_status():
    """Synchronise the current stream and raise if a kernel reported an error."""
    check(_lib.load().mcs_sync_status(stream_ptr()), "mcs_sync_status")


@dataclass
class Metadata:
    """The per-layer metadata cache: query groups, KV indices and the dense-sparse residual."""

    perm: torch.Tensor
    idx: torch.Tensor
    R: torch.Tensor


class Schedule:
    """Anchor/reuse schedule for one attention layer.

    Steps 0..warmup-2 run dense attention; step warmup-1 and every `period` steps after it are
    anchors (dense output, fresh metadata); all other steps reuse the cached metadata.
    """

    def __init__(self, C: int, k: int, warmup: int = 5, period: int = 10, scale=None):
        self.C, self.k, self.warmup, self.period, self.scale = C, k, warmup, period, scale
        self.meta: Metadata | None = None
        self.ws: torch.Tensor | None = None

    def kind(self, step: int) -> str:
        if step < self.warmup - 1:
            return "dense"
        if (step - (self.warmup - 1)) % self.period == 0:
            return "anchor"
        return "reuse"

    def __call__(self, step: int, Q, K, V):
        kind = self.kind(step)
        if kind == "dense":
            return dense_attn(Q, K, V, want_lse=False, scale=self.scale)[0]
        if kind == "anchor":
            if self.ws is None:
                self.ws = workspace(Q, self.C, self.k, self.scale)
            if self.meta is None:
                out = None
            else:
                out = (torch.empty_like(Q), self.meta.perm, self.meta.idx, self.meta.R)
            O_full, perm, idx, R = anchor(Q, K, V, self.C, self.k, ws=self.ws, out=out, scale=self.scale)
            self.meta = Metadata(perm, idx, R)
            return O_full
        return sparse_attn(Q, K, V, self.meta.perm, self.C, self.meta.idx, R=self.meta.R, scale=self.scale)
