"""Cases of the block-sparse path's operators: rotary, block selection, block attention and the 8-bit cache.

A case names its operator in "op":

* rotary   projections [B, N, H, d] to rotated, normalised, head-major Q, K, V;
* select   block means of the keys and the kb best key blocks of every query block;
* attn     attention over the listed key blocks (bf16 keys and values);
* write    keys and values into an 8-bit cache, one scale for each block of tokens and head;
* cached   attention over the listed blocks of such a cache.

Sizes follow the package's workloads: token grids (21, 32, 48) with 24 heads of 128 and (32, 32, 32) with 16 heads
of 64; a frame of the first grid is 1536 tokens.
"""

import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -100


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a whole clip's projections of one layer, q/k norm over the head: fused [B, N, 3, H, d] output of one GEMM
        dict(name="rotary clip", op="rotary", B=1, t=21, h=32, w=48, H=24, Hkv=24, d=128, a0=44, a1=42, a2=42,
             pairs="adjacent", norm="head", fused=True, fracpos=False),
        # a 3-D asset's grid, norm over the whole token, half-split pairs, fractional positions
        dict(name="rotary asset", op="rotary", B=1, t=32, h=32, w=32, H=16, Hkv=16, d=64, a0=20, a1=22, a2=22,
             pairs="halves", norm="token", fused=False, fracpos=True),
        # one small frame: latency
        dict(name="rotary small frame", op="rotary", B=1, t=1, h=16, w=16, H=2, Hkv=2, d=64, a0=16, a1=24, a2=24,
             pairs="adjacent", norm="head", fused=True, fracpos=False),
        # block choice for every query block of a clip, means of this step's keys included
        dict(name="select clip", op="select", B=1, H=24, Hkv=24, Nq=32256, Nk=32256, d=128, C=128, BK=128, kb=37,
             pooled=False, ragged=False),
        # one token per sequence against the kept means of a long cache, shared key heads, padded batch
        dict(name="select token", op="select", B=8, H=24, Hkv=8, Nq=1, Nk=131072, d=128, C=1, BK=128, kb=64,
             pooled=True, ragged=True),
        # the sparse step of a clip with the residual record added
        dict(name="attn clip", op="attn", B=1, H=24, Hkv=24, Nq=32256, Nk=32256, d=128, C=128, BK=128, kb=37,
             lists="full", ragged=False, resid=True),
        # a 3-D asset of odd length, small blocks, some query blocks with short or empty lists
        dict(name="attn asset odd", op="attn", B=1, H=16, Hkv=16, Nq=32701, Nk=32701, d=64, C=64, BK=64, kb=76,
             lists="holes", ragged=False, resid=False),
        # one token per sequence over every block, shared key heads, padded batch
        dict(name="attn token", op="attn", B=4, H=24, Hkv=8, Nq=1, Nk=8008, d=128, C=1, BK=64, kb=126,
             lists="all", ragged=True, resid=False),
        # a clip's keys and values into the cache
        dict(name="write clip", op="write", B=1, Hkv=24, n=32256, cap=32256, start=0, d=128, BK=128, ragged=False),
        # one odd frame behind others, padded batch
        dict(name="write frame", op="write", B=2, Hkv=16, n=1500, cap=16384, start=4096, d=64, BK=64, ragged=True),
        # the queries of one frame over a seventh of a long cache
        dict(name="cached frame", op="cached", B=1, H=24, Hkv=24, Nq=1536, Nk=129024, d=128, C=128, BK=128, kb=151,
             lists="full", ragged=False, resid=False),
        # one token per sequence, its chosen blocks of a long cache
        dict(name="cached token", op="cached", B=8, H=24, Hkv=8, Nq=1, Nk=131072, d=128, C=1, BK=64, kb=160,
             lists="full", ragged=True, resid=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotary", "select", "attn", "write", "cached"))
    d = rng.choice((64, 128))
    Hkv = rng.choice((1, 2, 5, 8, 16))
    H = Hkv * rng.choice((1, 1, 2, 3))
    B = rng.choice((1, 1, 2, 3))
    BK = rng.choice((32, 64, 128))
    if op == "rotary":
        a0, a1 = rng.choice(((16, 24), (20, 22), (22, 20), (16, 16))) if d == 64 else rng.choice(((44, 42), (16, 56), (32, 48)))
        a2 = d - a0 - a1
        return dict(op=op, B=B, t=rng.randint(1, 12), h=_log(rng, 3, 40), w=_log(rng, 3, 50), H=H, Hkv=Hkv, d=d, a0=a0,
                    a1=a1, a2=a2, pairs=rng.choice(("adjacent", "halves")), norm=rng.choice(("head", "token", "none")),
                    fused=rng.random() < 0.5 and H == Hkv, fracpos=rng.random() < 0.3)
    if op == "write":
        n = _log(rng, 1, 16000)
        start = BK * rng.randint(0, 20)
        return dict(op=op, B=B, Hkv=Hkv, n=n, cap=-(-(start + n) // BK) * BK + BK * rng.randint(0, 3), start=start, d=d,
                    BK=BK, ragged=rng.random() < 0.5)
    Nk = _log(rng, 500, 30000)
    if op == "cached":
        Nk = -(-Nk // BK) * BK
    nb = -(-Nk // BK)
    kb = max(1, int(nb * rng.uniform(0.08, 0.3)))
    small = rng.random() < 0.4
    Nq = rng.randint(1, 16) if small else _log(rng, 65, 9000)
    C = rng.choice((1, 16)) if small else rng.choice((64, 128))
    if op == "select":
        return dict(op=op, B=B, H=H, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, C=C, BK=BK, kb=kb, pooled=small, ragged=rng.random() < 0.5)
    lists = rng.choice(("full", "full", "holes", "all"))
    if lists == "all":
        kb, Nq = nb, min(Nq, 1500)
    while B * H * -(-Nq // C) * kb * BK * max(d, C) > 3e9:  # what the plain form gathers, and its logits
        Nq //= 2
    return dict(op=op, B=B, H=H, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, C=C, BK=BK, kb=kb, lists=lists, ragged=rng.random() < 0.5,
                resid=rng.random() < 0.5)


# ------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _tokens(g, B, H, n, d, off=0):
    """bf16 [B, H, n, d]: smooth functions of the position plus noise, as an attention layer's tensors are."""
    pos = torch.arange(off, off + n, device="cuda", dtype=torch.float32)
    f = 0.5 * (1.0 / 20000.0) ** (torch.arange(16, device="cuda", dtype=torch.float32) / 15)
    a = pos[:, None] * f
    phi = torch.cat([a.sin(), a.cos()], 1)
    w = torch.randn(B, H, 32, d, device="cuda", generator=g) / math.sqrt(32)
    return phi, w


def _field(g, phi, w, noise=0.5):
    x = torch.matmul(phi, w)
    x += noise * torch.randn(x.shape, device="cuda", generator=g)
    return x.bfloat16()


def _lens(case, g, most):
    if not case["ragged"]:
        return None
    return torch.randint(max(1, most // 2), most + 1, (case["B"],), device="cuda", generator=g, dtype=torch.int32)


def _lists(case, g):
    """int32 [B, H, ceil(Nq / C), kb]: ascending distinct blocks, nearer ones more often; -1 behind them."""
    if case["lists"] == "all":
        return None
    B, H, kb = case["B"], case["H"], case["kb"]
    nb, gq = -(-case["Nk"] // case["BK"]), -(-case["Nq"] // case["C"])
    at = (torch.arange(gq, device="cuda") * case["C"] + 0.5) / case["Nq"]
    to = (torch.arange(nb, device="cuda") + 0.5) / nb
    pull = -6.0 * (at[:, None] - to[None, :]).abs()
    noise = -torch.log(-torch.log(torch.rand(B, H, gq, nb, device="cuda", generator=g).clamp_(1e-7, 1 - 1e-6)))
    ids = (pull + noise).topk(kb, -1).indices.sort(-1).values.to(torch.int32)
    if case["lists"] == "holes":
        n = torch.randint(0, kb + 1, (B, H, gq, 1), device="cuda", generator=g)
        n = torch.where(torch.rand(B, H, gq, 1, device="cuda", generator=g) < 0.8, kb, n)
        ids = torch.where(torch.arange(kb, device="cuda") < n, ids, -1).to(torch.int32)
    return ids.contiguous()


def _quant(x, BK):
    """A cache's contents, laid out by plain steps: e4m3 values and fp32 scales of [B, H, n, d], n in whole blocks."""
    B, H, n, d = x.shape
    y = x.float().view(B, H, n // BK, BK * d)
    s = (y.abs().amax(-1) / E4M3_MAX).clamp_min(SCALE_MIN)
    q = (y / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(B, H, n, d), s.contiguous()


def prepare(case, seed):
    g, op, B, d = _gen(seed), case["op"], case["B"], case["d"]
    st = {"case": case}
    if op == "rotary":
        t, h, w, H, Hkv = case["t"], case["h"], case["w"], case["H"], case["Hkv"]
        n = t * h * w
        grid = torch.stack(torch.meshgrid(*(torch.arange(x, device="cuda") for x in (t, h, w)), indexing="ij"), -1).reshape(n, 3)
        # fractional positions: a grid squeezed into a smaller one's range; whole ones start at a later frame
        st["pos"] = (grid * 0.75 + 0.125).float() if case["fracpos"] else (grid + torch.tensor([int(seed) % 90, 0, 0], device="cuda")).int()
        if case["fused"]:
            x = torch.randn(B, n, 3, H, d, device="cuda", generator=g).bfloat16()
            st["q"], st["k"], st["v"] = x.unbind(2)
        else:
            st["q"], st["k"], st["v"] = (torch.randn(B, n, m, d, device="cuda", generator=g).bfloat16() for m in (H, Hkv, Hkv))
        if case["norm"] != "none":
            tok = case["norm"] == "token"
            st["qw"] = 1 + 0.1 * torch.randn(*((H, d) if tok else (d,)), device="cuda", generator=g)
            st["kw"] = 1 + 0.1 * torch.randn(*((Hkv, d) if tok else (d,)), device="cuda", generator=g)
        return st
    if op == "write":
        phi, w = _tokens(g, B, case["Hkv"], case["n"], d, case["start"])
        st["k"], st["v"] = _field(g, phi, w), _field(g, phi, w)
        nb = case["cap"] // case["BK"]
        st["k8"], st["v8"] = (torch.zeros(B, case["Hkv"], case["cap"], d, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
        st["ks"], st["vs"] = (torch.ones(B, case["Hkv"], nb, device="cuda") for _ in range(2))
        st["means"] = torch.zeros(B, case["Hkv"], nb, d, device="cuda")
        st["lens"] = _lens(case, g, case["n"])
        return st
    H, Hkv, Nq, Nk, BK = case["H"], case["Hkv"], case["Nq"], case["Nk"], case["BK"]
    phi, w = _tokens(g, B, Hkv, Nk, d)
    k = _field(g, phi, w)
    wq = w.repeat_interleave(H // Hkv, 1)
    st["q"] = _field(g, phi[torch.arange(Nk - Nq, Nk, device="cuda") % Nk], wq)
    st["len"] = _lens(case, g, Nk)
    if op == "select":
        if case["pooled"]:  # means that the program keeps beside its cache
            st["means"] = _plain_means(k, BK, st["len"])
        else:
            st["k"] = k
        return st
    v = _field(g, phi, w)
    st["ids"] = _lists(case, g)
    st["r"] = 0.1 * torch.randn(B, H, Nq, d, device="cuda", generator=g) if case["resid"] else None
    st["r"] = None if st["r"] is None else st["r"].bfloat16()
    if op == "attn":
        st["k"], st["v"] = k, v
    else:
        (st["k"], st["ks"]), (st["v"], st["vs"]) = _quant(k, BK), _quant(v, BK)
    return st


# ------------------------------------------------------------------------------------------ plain forms
def _plain_rotary(st):
    c = st["case"]
    d, axes = c["d"], (c["a0"], c["a1"], c["a2"])
    ang = torch.cat([st["pos"][:, a, None].double() * 10000.0 ** (-torch.arange(0, x, 2, device="cuda", dtype=torch.float64) / x)
                     for a, x in enumerate(axes)], -1)
    cos, sin = ang.cos().float()[None, :, None], ang.sin().float()[None, :, None]
    half = sum(axes) // 2

    def one(x, w):
        x = x.float()
        if c["norm"] != "none":
            over = (-2, -1) if c["norm"] == "token" else (-1,)
            x = x * torch.rsqrt(x.square().mean(over, keepdim=True) + 1e-6) * w
        if c["pairs"] == "adjacent":
            x1, x2 = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
            y = torch.stack([x1 * cos - x2 * sin, x1 * sin + x2 * cos], -1).flatten(-2)
        else:
            x1, x2 = x[..., :half], x[..., half:2 * half]
            y = torch.cat([x1 * cos - x2 * sin, x1 * sin + x2 * cos], -1)
        return torch.cat([y, x[..., 2 * half:]], -1).bfloat16().transpose(1, 2).contiguous()

    return one(st["q"], st.get("qw")), one(st["k"], st.get("kw")), st["v"].transpose(1, 2).contiguous()


def _plain_means(x, BK, lens=None):
    B, H, n, d = x.shape
    nb = -(-n // BK)
    y = x.double()
    count = torch.full((B,), n, device="cuda") if lens is None else lens.long()
    if lens is not None:
        y = torch.where((torch.arange(n, device="cuda") < count[:, None])[:, None, :, None], y, 0.0)
    y = torch.nn.functional.pad(y, (0, 0, 0, nb * BK - n)).view(B, H, nb, BK, d).sum(3)
    cnt = (count[:, None] - torch.arange(nb, device="cuda") * BK).clamp(0, BK)
    return (y / cnt.clamp_min(1)[:, None, :, None]).float()


def _plain_select(st):
    c = st["case"]
    means = st["means"] if c["pooled"] else _plain_means(st["k"], c["BK"], st["len"])
    nb, kb = means.shape[2], c["kb"]
    qbar = _plain_means(st["q"], c["C"]).double()
    s = torch.matmul(qbar, means.double().repeat_interleave(c["H"] // c["Hkv"], 1).transpose(-1, -2))
    n = torch.full((c["B"],), nb, device="cuda") if st["len"] is None else -(-st["len"].long() // c["BK"])
    live = torch.arange(nb, device="cuda") < n[:, None]
    s = torch.where(live[:, None, None], s, -math.inf)
    ids = torch.sort(s, dim=-1, descending=True, stable=True).indices[..., :kb]
    ids = torch.where(ids < n[:, None, None, None], ids, nb).sort(-1).values
    return means, torch.where(ids < nb, ids, -1).int()


def _plain_attn(st):
    c = st["case"]
    B, H, Hkv, Nq, Nk, d, C, BK = (c[x] for x in ("B", "H", "Hkv", "Nq", "Nk", "d", "C", "BK"))
    nb, gq = -(-Nk // BK), -(-Nq // C)
    ids = st["ids"]
    if ids is None:
        ids = torch.arange(nb, device="cuda", dtype=torch.int32).expand(B, H, 1, nb)
        gq, C = 1, Nq
    kb = ids.shape[-1]

    def blocks(x, s):  # the listed blocks of every query block: fp32 [B, H, gq, kb * BK, d]
        x = x.float() if s is None else x.float().view(B, Hkv, nb, -1).mul(s[..., None]).view(B, Hkv, Nk, d)
        x = torch.nn.functional.pad(x, (0, 0, 0, nb * BK - Nk)).view(B * Hkv, nb, BK * d)
        head = torch.arange(B * H, device="cuda") // (H // Hkv)
        return x[head[:, None], ids.clamp_min(0).view(B * H, -1).long()].view(B, H, gq, kb * BK, d)

    q = torch.nn.functional.pad(st["q"].float(), (0, 0, 0, gq * C - Nq)).view(B, H, gq, C, d)
    s = torch.matmul(q, blocks(st["k"], st.get("ks")).transpose(-1, -2)).mul_(1 / math.sqrt(d))
    key = (ids.clamp_min(0)[..., None] * BK + torch.arange(BK, device="cuda")).flatten(-2)
    most = torch.full((B,), Nk, device="cuda") if st["len"] is None else st["len"].long()
    live = (key < most[:, None, None, None]) & (ids >= 0).repeat_interleave(BK, -1)
    s.masked_fill_(~live[:, :, :, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp_min(-3e38)
    s.sub_(m).exp_()
    l = s.sum(-1, keepdim=True)
    o = torch.matmul(s, blocks(st["v"], st.get("vs"))) / torch.where(l > 0, l, 1.0)
    o = o.view(B, H, gq * C, d)[:, :, :Nq]
    o = o if st["r"] is None else o + st["r"].float()
    lse = (m + l.log()).view(B, H, gq * C)[:, :, :Nq]
    return o.bfloat16(), lse.contiguous()


def _plain_write(st):
    c = st["case"]
    B, Hkv, n, d, BK, start = (c[x] for x in ("B", "Hkv", "n", "d", "BK", "start"))
    nb, b0 = -(-n // BK), start // BK
    most = torch.full((B,), n, device="cuda") if st["lens"] is None else st["lens"].long()
    row = (torch.arange(n, device="cuda") < most[:, None])[:, None, :, None]
    blk = (torch.arange(nb, device="cuda") * BK < most[:, None])[:, None]

    def put(x, x8, s):
        y = torch.where(row, x.float(), 0.0)
        y = torch.nn.functional.pad(y, (0, 0, 0, nb * BK - n)).view(B, Hkv, nb, BK * d)
        amax = y.abs().amax(-1)
        sc = torch.where(amax > 0, (amax / E4M3_MAX).clamp_min(SCALE_MIN), 1.0)
        q = (y / sc[..., None]).clamp(-E4M3_MAX, E4M3_MAX).view(B, Hkv, nb * BK, d)[:, :, :n]
        old = x8[:, :, start:start + n]
        old.copy_(torch.where(row, q, old.float()).to(torch.float8_e4m3fn))
        s[..., b0:b0 + nb] = torch.where(blk, sc, s[..., b0:b0 + nb])

    put(st["k"], st["k8"], st["ks"])
    put(st["v"], st["v8"], st["vs"])
    m = _plain_means(st["k"], BK, most)
    st["means"][:, :, b0:b0 + nb] = torch.where(blk[..., None], m, st["means"][:, :, b0:b0 + nb])
    return st["k8"], st["v8"], st["ks"], st["vs"], st["means"]


# ------------------------------------------------------------------------------------------ one pass
def run(state):
    c, op = state["case"], state["case"]["op"]
    if own:
        from free_sparse_attention_reuse_b200 import api

        if op == "rotary":
            norm = None if c["norm"] == "none" else c["norm"]
            return api.rotary(state["q"], state["k"], state["v"], state["pos"], (c["a0"], c["a1"], c["a2"]),
                              pairs=c["pairs"], norm=norm, q_weight=state.get("qw"), k_weight=state.get("kw"))
        if op == "select":
            means = state["means"] if c["pooled"] else api.block_means(state["k"], c["BK"], kv_len=state["len"])
            return means, api.block_topk(state["q"], means, c["C"], c["kb"], BK=c["BK"], kv_len=state["len"])
        if op == "write":
            api.cache_write(state["k"], state["v"], state["k8"], state["v8"], state["ks"], state["vs"], c["BK"],
                            start=c["start"], means=state["means"], lens=state["lens"])
            return state["k8"], state["v8"], state["ks"], state["vs"], state["means"]
        return api.block_attn(state["q"], state["k"], state["v"], state["ids"], c["C"], c["BK"], R=state["r"],
                              kv_len=state["len"], k_scale=state.get("ks"), v_scale=state.get("vs"), want_lse=True)
    if op == "rotary":
        return _plain_rotary(state)
    if op == "select":
        return _plain_select(state)
    if op == "write":
        return _plain_write(state)
    return _plain_attn(state)


def work(case):
    c, op, B, d = case, case["op"], case["B"], case["d"]
    if op == "rotary":
        n = B * c["t"] * c["h"] * c["w"] * (c["H"] + 2 * c["Hkv"]) * d
        return {"bytes": 4 * n + 12 * c["t"] * c["h"] * c["w"], "flops": 8 * n}
    if op == "write":
        n = 2 * B * c["Hkv"] * c["n"] * d
        nb = -(-c["n"] // c["BK"])
        return {"bytes": 3 * n + 4 * B * c["Hkv"] * nb * (d + 2), "flops": 4 * n}
    H, Hkv, Nq, Nk, C, BK, kb = (c[x] for x in ("H", "Hkv", "Nq", "Nk", "C", "BK", "kb"))
    nb, gq = -(-Nk // BK), -(-Nq // C)
    if op == "select":
        read = 2 * B * H * Nq * d + (0 if c["pooled"] else 2 * B * Hkv * Nk * d)
        return {"bytes": read + 4 * B * Hkv * nb * d + 4 * B * H * gq * kb, "flops": 2 * B * H * gq * nb * d}
    # each block that some list names is read once: the expected number of distinct ones among the draws
    seen = nb if c["lists"] == "all" else nb * (1 - (1 - kb / nb) ** (gq * (H // Hkv)))
    kv = 2 * B * Hkv * min(seen * BK, Nk) * d * (2 if op == "attn" else 1) * (0.75 if c["ragged"] else 1)
    rows = 2 * B * H * Nq * d * (3 if c["resid"] else 2)
    ids = 0 if c["lists"] == "all" else 4 * B * H * gq * kb
    part = (0.9 if c["lists"] == "holes" else 1) * (0.75 if c["ragged"] else 1)
    return {"bytes": kv + rows + ids, "flops": 4 * B * H * Nq * min(kb * BK, Nk) * d * part}


# ------------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "rotary":
        return _exact_rotary(case, st)
    if op == "write":
        return _exact_write(case, st)
    if op == "select":
        return _exact_select(case, st)
    return _exact_attn(case, st)


def _exact_rotary(c, st):
    axes = (c["a0"], c["a1"], c["a2"])
    half = sum(axes) // 2
    freq = np.concatenate([[10000.0 ** (-2.0 * j / x) for j in range(x // 2)] for x in axes])
    axis = np.concatenate([[a] * (x // 2) for a, x in enumerate(axes)])
    pos = st["pos"].double().cpu().numpy()
    turn = torch.from_numpy(np.exp(1j * pos[:, axis] * freq)).cuda()  # [n, half]

    def one(x, w):
        heads = []
        every = x.double()
        power = every.square().mean((2, 3)) if c["norm"] == "token" else None
        for h in range(x.shape[2]):
            y = every[:, :, h].clone()
            if c["norm"] != "none":
                p = y.square().mean(-1) if power is None else power
                y *= ((p + 1e-6) ** -0.5)[..., None] * (w[h] if c["norm"] == "token" else w).double()
            i = torch.arange(half, device="cuda")
            i, j = (2 * i, 2 * i + 1) if c["pairs"] == "adjacent" else (i, i + half)
            z = torch.complex(y[..., i], y[..., j]) * turn
            y[..., i], y[..., j] = z.real, z.imag
            heads.append(y)
        return torch.stack(heads, 1)

    return one(st["q"], st.get("qw")), one(st["k"], st.get("kw")), st["v"].double().permute(0, 2, 1, 3).contiguous()


def _exact_means(x, size, count):
    """Means of blocks of `size` rows of [H, n, d] fp64, the first `count` rows alone; zero where there is none."""
    H, n, d = x.shape
    nb = -(-n // size)
    out = torch.zeros(H, nb, d, device="cuda", dtype=torch.float64)
    whole = count // size
    out[:, :whole] = x[:, :whole * size].reshape(H, whole, size, d).mean(2)
    if count % size:
        out[:, whole] = x[:, whole * size:count].mean(1)
    return out


def _exact_select(c, st):
    nb, kb = -(-c["Nk"] // c["BK"]), c["kb"]
    means, ids = [], []
    for b in range(c["B"]):
        count = c["Nk"] if st["len"] is None else int(st["len"][b])
        mk = st["means"][b].double() if c["pooled"] else _exact_means(st["k"][b].double(), c["BK"], count)
        mq = _exact_means(st["q"][b].double(), c["C"], c["Nq"])
        means.append(mk)
        n = -(-count // c["BK"])
        rows = []
        for h in range(c["H"]):
            # the scores of the means as they are held: in 32 bits
            s = (mq[h].float().double() @ mk[h // (c["H"] // c["Hkv"])].float().double().T)[:, :n].cpu().numpy()
            order = np.argsort(-s, axis=-1, kind="stable")[:, :kb]
            row = np.full((s.shape[0], kb), -1, dtype=np.int32)
            row[:, :order.shape[1]] = np.sort(order, -1)
            rows.append(torch.from_numpy(row))
        ids.append(torch.stack(rows))
    return torch.stack(means), torch.stack(ids)


def _exact_attn(c, st):
    B, H, Nq, Nk, d, C, BK = (c[x] for x in ("B", "H", "Nq", "Nk", "d", "C", "BK"))
    rep, gq = H // c["Hkv"], -(-Nq // C)
    out = torch.zeros(B, H, Nq, d, device="cuda", dtype=torch.float64)
    lse = torch.full((B, H, Nq), -math.inf, device="cuda", dtype=torch.float64)
    step = max(1, (1 << 27) // (C * c["kb"] * BK))

    def values(x, s, b, h):
        x = x[b, h].to(torch.float64)
        return x if s is None else x * s[b, h].double().repeat_interleave(BK)[:Nk, None]

    for b in range(B):
        count = Nk if st["len"] is None else int(st["len"][b])
        for h in range(H):
            k, v = values(st["k"], st.get("ks"), b, h // rep), values(st["v"], st.get("vs"), b, h // rep)
            q = st["q"][b, h].double()
            if st["ids"] is None:
                s = (q @ k[:count].T) / math.sqrt(d)
                lse[b, h] = s.logsumexp(-1)
                out[b, h] = (s - lse[b, h][:, None]).exp() @ v[:count]
                continue
            lists = st["ids"][b, h].long()
            at = torch.arange(BK, device="cuda")
            for g0 in range(0, gq, step):
                ids = lists[g0:g0 + step]
                keys = (ids[..., None] * BK + at).flatten(1)
                dead = (keys < 0) | (keys >= count)
                keys = keys.clamp(0, Nk - 1)
                rows = (torch.arange(g0, g0 + len(ids), device="cuda")[:, None] * C + torch.arange(C, device="cuda")).clamp_max(Nq - 1)
                s = torch.einsum("gcd,gkd->gck", q[rows], k[keys]) / math.sqrt(d)
                s = s.masked_fill(dead[:, None], -math.inf)
                t = s.logsumexp(-1)
                p = (s - torch.where(t > -math.inf, t, 0.0)[..., None]).exp()
                o = torch.einsum("gck,gkd->gcd", p, v[keys])
                n = min(Nq, (g0 + len(ids)) * C) - g0 * C
                out[b, h, g0 * C:g0 * C + n] = o.reshape(-1, d)[:n]
                lse[b, h, g0 * C:g0 * C + n] = t.reshape(-1)[:n]
    return out if st["r"] is None else out + st["r"].double(), lse


def _exact_write(c, st):
    B, Hkv, n, BK, start = (c[x] for x in ("B", "Hkv", "n", "BK", "start"))
    means = st["means"].double()
    outs = [st["k8"].double(), st["v8"].double()]
    scales = [st["ks"].double(), st["vs"].double()]
    for b in range(B):
        count = n if st["lens"] is None else int(st["lens"][b])
        nb, b0 = -(-count // BK), start // BK
        means[b, :, b0:b0 + nb] = _exact_means(st["k"][b].double(), BK, count)[:, :nb]
        for x, x8, sc in zip((st["k"], st["v"]), outs, scales):
            y = x[b, :, :count].double()
            top = torch.stack([y[:, j * BK:(j + 1) * BK].abs().amax((1, 2)) for j in range(nb)], 1)
            s = torch.where(top > 0, (top / E4M3_MAX).clamp_min(SCALE_MIN), 1.0)
            sc[b, :, b0:b0 + nb] = s
            x8[b, :, start:start + count] = _round_e4m3(y / s.repeat_interleave(BK, 1)[:, :count, None])
    return outs[0], outs[1], scales[0], scales[1], means


def _round_e4m3(x):
    """The nearest value of 4 exponent and 3 mantissa bits (largest 448, smallest step 2^-9), ties to even."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -20))).clamp_min(-6)
    step = 2.0 ** (e - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
