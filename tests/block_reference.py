"""Plain fp64 forms of the block-sparse operators and the error bounds of their outputs.

Roundings: a value rounded to bf16 is off by at most 2^-8 of itself (half a step), fp32 2^-24.
Everything runs on the CPU in fp64, one head at a time, from the definitions.
"""

import math

import torch

BF16, FP32 = 2.0 ** -8, 2.0 ** -24
E4M3_MAX, SCALE_MIN = 448.0, 2.0 ** -100


def rotary(q, k, v, pos, axes, theta=10000.0, pairs="adjacent", norm=None, q_weight=None, k_weight=None, eps=1e-6):
    """[B, N, H, d] views to fp64 [B, H, N, d] and, for q and k, the size that the error scales with."""
    half = sum(axes) // 2
    freq = torch.cat([theta ** (-2.0 * torch.arange(a // 2, dtype=torch.float64) / a) for a in axes])
    axis = torch.cat([torch.full((a // 2,), i) for i, a in enumerate(axes)]).long()
    p = pos.double() if pos.dim() == 3 else pos.double()[None]
    ang = p[..., axis] * freq  # [B or 1, N, half]
    c, s = ang.cos()[:, :, None], ang.sin()[:, :, None]

    def one(x, w):
        x = x.double()
        if norm is not None:
            over = (-2, -1) if norm == "token" else (-1,)
            x = x / (x.square().mean(over, keepdim=True) + eps).sqrt()
            if w is not None:
                x = x * w.double()
        if pairs == "adjacent":
            i = 2 * torch.arange(half)
            j = i + 1
        else:
            i = torch.arange(half)
            j = i + half
        y, size = x.clone(), x.abs()
        y[..., i] = x[..., i] * c - x[..., j] * s
        y[..., j] = x[..., i] * s + x[..., j] * c
        size = size.clone()
        size[..., i] = size[..., j] = torch.maximum(x[..., i].abs(), x[..., j].abs())
        return y.transpose(1, 2), size.transpose(1, 2)

    out = []
    for x, w in ((q, q_weight), (k, k_weight)):
        out.append((None, None) if x is None else one(x, w))
    return out[0], out[1], None if v is None else v.double().transpose(1, 2)


def rotary_bound(ref, size):
    """One rounding to bf16, and fp32 steps before it: the norm (at most 64 + 6 of them, an rms of up
    to 2^14 elements summed in parts), two products, and sines of an angle held to 2^-23 turns."""
    return BF16 * ref.abs() + (128 * FP32 + 2 * math.pi * 2.0 ** -23) * size


def lengths(kv_len, B, n):
    return [n] * B if kv_len is None else [int(x) for x in kv_len]


def means(x, BK, kv_len=None):
    B, H, n, d = x.shape
    nb = -(-n // BK)
    out = torch.zeros(B, H, nb, d, dtype=torch.float64)
    for b, m in enumerate(lengths(kv_len, B, n)):
        for j in range(nb):
            rows = x[b, :, j * BK:min((j + 1) * BK, m)].double()
            if rows.shape[1]:
                out[b, :, j] = rows.sum(1) / rows.shape[1]
    return out


def topk(Q, mk, C, kb, BK, kv_len=None):
    """(blocks, scores): the choice from the fp32 means as given, fp64 scores, ties to the lower block."""
    B, H, Nq, d = Q.shape
    Hkv, nb = mk.shape[1:3]
    gq = -(-Nq // C)
    mq = means(Q, C).float().double()
    s = torch.einsum("bhgd,bhjd->bhgj", mq, mk.double().repeat_interleave(H // Hkv, 1))
    out = torch.full((B, H, gq, kb), -1, dtype=torch.int32)
    for b, m in enumerate(lengths(kv_len, B, nb * BK)):
        n = -(-m // BK)
        order = torch.sort(s[b, :, :, :n], dim=-1, descending=True, stable=True).indices[..., :kb]
        out[b, :, :, :order.shape[-1]] = order.sort(-1).values.int()
    return out, s


def e4m3(x):
    """Nearest value of 4 exponent and 3 mantissa bits, ties to even, saturating (fp64 in and out)."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -20))).clamp_min(-6)
    step = 2.0 ** (e - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def block_scale(rows):
    """Scale of one block of one head ([rows, d]): fp32, as the library holds it."""
    y = rows.double()
    y = torch.where(y.isfinite(), y.abs(), 0.0)
    top = float(y.max())
    if top == 0.0:
        return 1.0
    return float(torch.tensor(top, dtype=torch.float32).div(E4M3_MAX).clamp_min(SCALE_MIN))


def attn(Q, K, V, blocks, C, BK, R=None, kv_len=None, k_scale=None, v_scale=None, scale=None):
    """(out, lse, spread, delta): fp64 results; spread = softmax-weighted |v|, delta = bound of a
    logit's error in fp32, both per row, which attn_bound turns into tolerances."""
    B, H, Nq, d = Q.shape
    Hkv, Nk = K.shape[1:3]
    nb, gq = -(-Nk // BK), -(-Nq // C)
    sc = 1 / math.sqrt(d) if scale is None else scale
    out = torch.zeros(B, H, Nq, d, dtype=torch.float64)
    spread = torch.zeros_like(out)
    lse = torch.full((B, H, Nq), -math.inf, dtype=torch.float64)
    delta = torch.zeros(B, H, Nq, 1, dtype=torch.float64)
    for b, m in enumerate(lengths(kv_len, B, Nk)):
        for h in range(H):
            hk = h // (H // Hkv)
            k, v = K[b, hk].double(), V[b, hk].double()
            if k_scale is not None:
                k = k * k_scale[b, hk].double().repeat_interleave(BK)[:, None]
                v = v * v_scale[b, hk].double().repeat_interleave(BK)[:, None]
            for g in range(gq):
                ids = range(nb) if blocks is None else blocks[b, h, g].tolist()
                keys = []
                for j in ids:
                    if j < 0:
                        break
                    if j < nb:
                        keys += range(j * BK, min((j + 1) * BK, m))
                rows = slice(g * C, min((g + 1) * C, Nq))
                if not keys:
                    continue
                q, kk, vv = Q[b, h, rows].double(), k[keys], v[keys]
                s = q @ kk.T * sc
                t = s.logsumexp(-1)
                p = (s - t[:, None]).exp()
                out[b, h, rows] = p @ vv
                spread[b, h, rows] = p @ vv.abs()
                lse[b, h, rows] = t
                # products exact or rounded once, d of them added in fp32; then scaled, in base 2,
                # and a reference of the same size subtracted
                size = (q.abs() @ kk.abs().T).amax(-1) * sc
                delta[b, h, rows, 0] = (d + 8) * FP32 * size
    if R is not None:
        out = out + R.double()
    return out, lse, spread, delta


def attn_bound(out, spread, delta):
    """Error of out: probabilities held in bf16 (2^-8 each) from logits off by delta (numerator and
    sum: twice), exponentials and partial sums in fp32 (2^-18 covers ex2's 2^-22 and the sums of a
    few thousand terms kept in parts), and the result rounded to bf16."""
    return BF16 * out.abs() + (BF16 + 2 * delta + 2.0 ** -18) * 1.01 * spread + 1e-30


def lse_bound(lse, delta):
    return delta[..., 0] + 2.0 ** -18 + 4 * FP32 * lse.abs()
