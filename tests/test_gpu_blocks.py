"""Rotary, block selection, block attention and the 8-bit cache against plain fp64 forms (needs a B200)."""

import math

import pytest
import torch

import block_reference as ref
from free_sparse_attention_reuse_b200 import _lib, api

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = torch.float8_e4m3fn


def rnd(seed, *shape, std=1.0):
    return (std * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).bfloat16()


def dev(t):
    return None if t is None else t.to(DEV)


def within(got, want, bound, what):
    d = (got.double().cpu() - want).abs()
    d = torch.where(got.double().cpu() == want, 0.0, d)  # equal infinities
    assert not d.isnan().any(), f"{what}: NaN"
    worst = (d - bound).max()
    assert worst <= 0, f"{what}: {float(worst):.3e} over the bound (error {float(d.max()):.3e})"


# ------------------------------------------------------------------------------------------ rotary
@pytest.mark.parametrize("d,H,Hkv,B,N,axes,pairs,norm,weights", [
    (128, 3, 3, 1, 100, (44, 42, 42), "adjacent", "head", torch.float32),
    (128, 4, 2, 2, 33, (16, 56, 56), "halves", "token", torch.float32),
    (64, 5, 1, 3, 17, (20, 22, 22), "halves", "head", torch.bfloat16),
    (64, 2, 2, 1, 1, (16, 24, 24), "adjacent", "token", None),
    (128, 1, 1, 1, 700, (64,), "adjacent", None, None),
    (64, 3, 3, 2, 31, (8, 8, 8, 8), "halves", None, None),
    (64, 2, 1, 1, 2500, (16, 16, 16), "adjacent", "head", torch.float32),
    (128, 17, 1, 1, 9, (2, 126), "adjacent", "token", torch.bfloat16),
])
@pytest.mark.parametrize("fpos", [False, True])
def test_rotary(d, H, Hkv, B, N, axes, pairs, norm, weights, fpos):
    q, k, v = rnd(1, B, N, H, d), rnd(2, B, N, Hkv, d), rnd(3, B, N, Hkv, d)
    g = torch.Generator().manual_seed(4)
    pos = torch.randint(-50, 100000, (B, N, len(axes)), generator=g).int()
    if fpos:
        pos = pos.float() / 8
    pos = pos if B > 1 else pos[0]
    qw = kw = None
    if weights is not None:
        shape = (lambda h: (h, d)) if norm == "token" else (lambda h: (d,))
        kw = (1 + 0.2 * torch.randn(*shape(Hkv), generator=g)).to(weights)
        qw = (1 + 0.2 * torch.randn(*shape(H), generator=g)).to(weights)
    (rq, sq), (rk, sk), rv = ref.rotary(q, k, v, pos, axes, pairs=pairs, norm=norm, q_weight=qw, k_weight=kw)
    Q, K, V = api.rotary(dev(q), dev(k), dev(v), dev(pos), axes, pairs=pairs, norm=norm, q_weight=dev(qw), k_weight=dev(kw))
    api.sync_status()
    within(Q, rq, ref.rotary_bound(rq, sq), "Q")
    within(K, rk, ref.rotary_bound(rk, sk), "K")
    assert torch.equal(V.cpu().double(), rv)


def test_rotary_fused_views_and_absent_parts():
    x = dev(rnd(5, 2, 45, 3, 4, 64))
    pos = torch.arange(45 * 2, device=DEV, dtype=torch.int32).view(45, 2)
    axes = (32, 32)
    q, k, v = x.unbind(2)
    Q, K, V = api.rotary(q, k, v, pos, axes, norm="head")
    Q2, K2, V2 = api.rotary(q.contiguous(), k.contiguous(), v.contiguous(), pos, axes, norm="head")
    assert torch.equal(Q, Q2) and torch.equal(K, K2) and torch.equal(V, V2)
    Q3, K3, V3 = api.rotary(q, None, None, pos, axes, norm="head")
    assert torch.equal(Q, Q3) and K3 is None and V3 is None
    Q4, K4, _ = api.rotary(q, k, None, pos, axes, norm="head", out=(Q3, K2, None))
    assert Q4 is Q3 and torch.equal(K4, K)
    # a slice of a longer sequence and of the batch; one token of a longer stride
    Q5, _, _ = api.rotary(q[1:, 7:30], None, None, pos[7:30], axes, norm="head")
    assert torch.equal(Q5, Q[1:, :, 7:30])
    Q6, _, _ = api.rotary(q[:, 3:4], None, None, pos[3:4], axes, norm="head")
    assert torch.equal(Q6, Q[:, :, 3:4])
    api.sync_status()


@pytest.mark.parametrize("norm,H,Hkv,d,N", [("head", 3, 2, 64, 50), ("token", 3, 2, 64, 50), ("token", 40, 40, 128, 21),
                                            ("token", 70, 1, 64, 330), ("token", 16, 16, 64, 2000)])
def test_rotary_one_weight_and_many_heads(norm, H, Hkv, d, N):
    q, k = rnd(7, 1, N, H, d), rnd(8, 1, N, Hkv, d)
    g = torch.Generator().manual_seed(9)
    pos = torch.randint(0, 500, (N, 1), generator=g).int()
    for which in (0, 1):
        shape = [(d,), (d,)] if norm == "head" else [(H, d), (Hkv, d)]
        w = [None, None]
        w[which] = 1 + 0.2 * torch.randn(*shape[which], generator=g)
        (rq, sq), (rk, sk), _ = ref.rotary(q, k, None, pos, (d // 2,), norm=norm, q_weight=w[0], k_weight=w[1])
        Q, K, _ = api.rotary(dev(q), dev(k), None, dev(pos), (d // 2,), norm=norm, q_weight=dev(w[0]), k_weight=dev(w[1]))
        within(Q, rq, ref.rotary_bound(rq, sq), "Q")
        within(K, rk, ref.rotary_bound(rk, sk), "K")


def test_rotary_zero_rows_and_large_values():
    q = rnd(6, 1, 8, 2, 64)
    q[0, 3] = 0
    q[0, 4] *= 2.0 ** 60
    q[0, 5] *= 2.0 ** -60
    pos = torch.zeros(8, 1, dtype=torch.int32)
    (rq, sq), _, _ = ref.rotary(q, None, None, pos, (64,), norm="head")
    Q, _, _ = api.rotary(dev(q), None, None, dev(pos), (64,), norm="head")
    within(Q, rq, ref.rotary_bound(rq, sq) + 2.0 ** -133, "Q")  # the last: a bf16 subnormal's half step


# ------------------------------------------------------------------------------------------ selection
@pytest.mark.parametrize("B,H,N,d,BK,lens", [
    (1, 2, 300, 64, 64, None), (2, 3, 129, 128, 128, [129, 1]), (3, 1, 1000, 64, 32, [0, 33, 1000]), (1, 1, 1, 128, 32, None),
    (2, 1, 5000, 128, 64, [4097, 64]),
])
def test_block_means(B, H, N, d, BK, lens):
    x = rnd(7, B, H, N, d)
    kv = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    want = ref.means(x, BK, kv)
    if kv is not None:  # rows behind the length are never looked at
        for b, n in enumerate(lens):
            x[b, :, n:] = math.nan
    got = api.block_means(dev(x), BK, kv_len=dev(kv))
    api.sync_status()
    # fp64 sums of at most 128 bf16 values, one division, one rounding
    within(got, want, want.abs() * (ref.FP32 + 2.0 ** -40), "means")


def _check_topk(got, want, scores, kb):
    """Equal, except where fp64 sums taken in another order may swap neighbours of the cut."""
    diff = (got.cpu() != want).any(-1)
    for b, h, g in diff.nonzero().tolist():
        a, w = set(got[b, h, g].tolist()), set(want[b, h, g].tolist())
        s = scores[b, h, g]
        assert len(a) == len(w)
        tol = 1e-13 * s.abs().max()
        cut = min(float(s[j]) for j in w)
        for j in a ^ w:
            assert abs(float(s[j]) - cut) <= tol, f"block {j} of row {(b, h, g)}"
        assert got[b, h, g].tolist() == sorted(a)


@pytest.mark.parametrize("B,H,Hkv,Nq,Nk,d,C,BK,kb,lens", [
    (1, 2, 2, 512, 512, 64, 64, 64, 3, None),
    (2, 6, 2, 333, 1000, 128, 128, 32, 7, [1000, 500]),
    (1, 4, 1, 1, 4000, 128, 1, 64, 20, None),
    (3, 2, 2, 20, 700, 64, 16, 32, 22, [700, 0, 90]),
    (1, 1, 1, 65, 65, 64, 64, 64, 2, None),
    (2, 3, 3, 7, 129, 64, 1, 128, 1, [1, 129]),
    (1, 2, 1, 1000, 20000, 64, 16, 32, 300, None),
    (1, 1, 1, 3, 70000, 128, 1, 32, 2000, None),
    (1, 2, 2, 300, 14000, 64, 64, 32, 60, [13000]),
    (2, 3, 1, 1, 40000, 64, 1, 64, 100, [40000, 12345]),
    (1, 6, 1, 200, 300, 64, 64, 128, 2, None),
])
def test_block_topk(B, H, Hkv, Nq, Nk, d, C, BK, kb, lens):
    q, k = rnd(8, B, H, Nq, d), rnd(9, B, Hkv, Nk, d)
    kv = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    mk = api.block_means(dev(k), BK, kv_len=dev(kv))
    want, scores = ref.topk(q, mk.cpu(), C, kb, BK, kv)
    if kv is not None:  # means of blocks that hold no valid key are not candidates, whatever they are
        for b, n in enumerate(lens):
            mk[b, :, -(-n // BK):] = math.inf
    got = api.block_topk(dev(q), mk, C, kb, BK, kv_len=dev(kv))
    api.sync_status()
    _check_topk(got, want, scores, kb)


def test_block_topk_ties_go_to_the_lower_block():
    B, H, nb, d, kb = 1, 2, 200, 64, 50
    q = rnd(10, B, H, 64, d)
    mk = rnd(11, B, H, 8, d).float().repeat_interleave(25, 2)  # eight scores, each 25 times
    got = api.block_topk(dev(q), dev(mk), 64, kb, 64)
    want, _ = ref.topk(q, mk, 64, kb, 64)
    assert torch.equal(got.cpu(), want)
    same = torch.zeros(B, H, nb, d)
    got = api.block_topk(dev(q), dev(same), 64, kb, 64)
    assert torch.equal(got.cpu(), torch.arange(kb, dtype=torch.int32).expand(B, H, 1, kb))


def test_block_topk_nan_and_infinite_scores():
    q = torch.ones(1, 1, 1, 64).bfloat16()
    mk = torch.zeros(1, 1, 6, 64)
    mk[0, 0, :, 0] = torch.tensor([math.nan, -math.inf, 2.0, math.inf, -1.0, math.nan])
    for kb, want in ((1, [3]), (2, [2, 3]), (3, [2, 3, 4]), (4, [1, 2, 3, 4]), (5, [0, 1, 2, 3, 4])):
        assert api.block_topk(dev(q), dev(mk), 1, kb, 32)[0, 0, 0].tolist() == want


# ------------------------------------------------------------------------------------------ attention
def lists(seed, B, H, gq, nb, kb, kind):
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand(B, H, gq, nb, generator=g).topk(kb, -1).indices.int()  # any order
    if kind == "sorted":
        ids = ids.sort(-1).values
    if kind == "holes":
        n = torch.randint(0, kb + 1, (B, H, gq, 1), generator=g)
        ids = torch.where(torch.arange(kb) < n, ids, -1).int()
    return ids


def quantised(k, BK):
    """(e4m3 values, scales) of [B, H, n, d], n a multiple of BK."""
    B, H, n, d = k.shape
    y = k.float().view(B, H, n // BK, BK * d)
    s = (y.abs().amax(-1) / 448.0).clamp_min(2.0 ** -100)
    return (y / s[..., None]).view(B, H, n, d).to(E4M3), s.contiguous()


def run_attn(q, k, v, ids, C, BK, r=None, kv=None, fp8=False, scale=None, poison=True, kvr=None):
    """One call against the plain form; keys behind the lengths are poisoned for the call."""
    ks = vs = None
    if fp8:
        (k, ks), (v, vs) = quantised(k, BK), quantised(v, BK)
    want, lse, spread, delta = ref.attn(q, k, v, ids, C, BK, r, kvr if kvr is not None else kv, ks, vs, scale)
    dk, dv = dev(k), dev(v)
    if kv is not None and poison:
        for b, n in enumerate((kvr if kvr is not None else kv).tolist()):
            for x, bad in ((dk, math.inf), (dv, math.nan)):
                if fp8:
                    x.view(torch.uint8)[b, :, n:] = 0x7F  # NaN
                else:
                    x[b, :, n:] = bad
    got, glse = api.block_attn(dev(q), dk, dv, dev(ids), C, BK, R=dev(r), kv_len=dev(kv), k_scale=dev(ks), v_scale=dev(vs),
                               want_lse=True, scale=scale)
    within(got, want, ref.attn_bound(want, spread, delta), "out")
    within(glse, lse, ref.lse_bound(lse.nan_to_num(neginf=0.0), delta), "lse")
    plain, none = api.block_attn(dev(q), dk, dv, dev(ids), C, BK, R=dev(r), kv_len=dev(kv), k_scale=dev(ks),
                                 v_scale=dev(vs), scale=scale)
    assert none is None and torch.equal(plain, got)
    return got


SHAPES = [
    # B, H, Hkv, Nq, Nk, d, C, BK, kb, kind, lens, resid
    (1, 2, 2, 256, 512, 64, 128, 128, 3, "sorted", None, False),
    (1, 2, 1, 300, 700, 128, 128, 128, 4, "any", [650], True),
    (2, 4, 2, 200, 900, 64, 64, 64, 9, "holes", [900, 130], True),
    (2, 3, 3, 129, 513, 128, 64, 32, 11, "holes", [0, 513], False),
    (1, 3, 1, 65, 333, 64, 128, 32, 11, "any", None, True),
    (1, 1, 1, 700, 70, 128, 64, 64, 1, "any", [3], False),
    (3, 2, 2, 1, 400, 64, 1, 64, 5, "holes", [400, 64, 1], True),
    (2, 6, 2, 5, 600, 128, 1, 32, 12, "any", [600, 333], False),
    (1, 4, 4, 16, 1000, 64, 16, 128, 6, "any", [930], True),
    (2, 5, 5, 33, 450, 128, 16, 64, 8, "holes", [450, 0], False),
    (2, 6, 2, 1, 800, 128, 1, 64, 13, None, [800, 301], False),
    (1, 4, 1, 7, 1500, 64, 16, 32, 47, None, None, True),
    (2, 2, 2, 150, 600, 128, 128, 64, 10, None, [600, 65], False),
    (1, 2, 1, 400, 1100, 64, 64, 128, 9, None, [1027], True),
    (1, 1, 1, 64, 64, 64, 64, 64, 1, "sorted", None, False),
    (1, 1, 1, 1, 1, 128, 1, 32, 1, None, None, False),
    (1, 1, 1, 40, 9000, 128, 64, 64, 130, "any", None, False),
    (1, 1, 1, 2, 9000, 64, 1, 32, 250, "sorted", [8999], True),
    (1, 3, 3, 1000, 8192, 64, 64, 64, 100, "holes", None, False),  # many stages, lists of unlike lengths
    (1, 3, 1, 1000, 8192, 128, 64, 32, 200, "holes", [8000], False),
    (2, 2, 2, 1100, 6000, 128, 128, 64, 60, "holes", [6000, 100], False),
    (2, 6, 2, 3, 33000, 64, 1, 32, 1032, None, [33000, 20001], False),  # whole stores: few rows, and tiles
    (2, 12, 2, 3, 33000, 128, 16, 64, 516, None, [32999, 64], True),
    (1, 6, 1, 4, 66000, 64, 64, 128, 516, None, [65999], False),
    (1, 2, 1, 70, 5000, 64, 1, 32, 157, None, None, True),
]


@pytest.mark.parametrize("B,H,Hkv,Nq,Nk,d,C,BK,kb,kind,lens,resid", SHAPES)
def test_block_attn(B, H, Hkv, Nq, Nk, d, C, BK, kb, kind, lens, resid):
    q, k, v = rnd(20, B, H, Nq, d), rnd(21, B, Hkv, Nk, d), rnd(22, B, Hkv, Nk, d)
    ids = None if kind is None else lists(23, B, H, -(-Nq // C), -(-Nk // BK), kb, kind)
    kv = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    run_attn(q, k, v, ids, C, BK, rnd(24, B, H, Nq, d) if resid else None, kv)
    api.sync_status()


@pytest.mark.parametrize("B,H,Hkv,Nq,Nk,d,C,BK,kb,kind,lens,resid", SHAPES)
def test_block_attn_8bit(B, H, Hkv, Nq, Nk, d, C, BK, kb, kind, lens, resid):
    Nk = -(-Nk // BK) * BK
    q, k = rnd(25, B, H, Nq, d), rnd(26, B, Hkv, Nk, d)
    v = rnd(27, B, Hkv, Nk, d) * torch.logspace(-3, 3, Nk)[:, None].bfloat16()  # scales of 10^-6 apart
    ids = None if kind is None else lists(28, B, H, -(-Nq // C), Nk // BK, kb, kind)
    kv = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    run_attn(q, k, v.contiguous(), ids, C, BK, rnd(29, B, H, Nq, d) if resid else None, kv, fp8=True)
    api.sync_status()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("C,Nq", [(128, 200), (64, 200), (16, 20), (1, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_block_attn_steep_logits(d, C, Nq, fp8):
    """Logits that rise by hundreds along the keys, and rows that are far below their first keys."""
    Nk, BK = 640, 64
    q, k, v = rnd(30, 1, 2, Nq, d), rnd(31, 1, 2, Nk, d), rnd(32, 1, 2, Nk, d)
    q[..., 0] = 16.0
    k[..., 0] = torch.linspace(-60, 60, Nk).bfloat16()
    q[:, 1, :, 0] = -16.0
    run_attn(q, k, v, None, C, BK, fp8=fp8)
    ids = torch.arange(10, dtype=torch.int32).expand(1, 2, -(-Nq // C), 10).contiguous()
    run_attn(q, k, v, ids, C, BK, fp8=fp8)
    run_attn(q, k, v, ids.flip(-1).contiguous(), C, BK, fp8=fp8, scale=1.0)


@pytest.mark.parametrize("C,Nq", [(128, 130), (64, 130), (16, 17), (1, 2)])
@pytest.mark.parametrize("fp8", [False, True])
def test_block_attn_repeated_and_bad_entries(C, Nq, fp8):
    Nk, BK, kb = 320, 64, 5
    gq = -(-Nq // C)
    q, k, v = rnd(33, 1, 1, Nq, 64), rnd(34, 1, 1, Nk, 64), rnd(35, 1, 1, Nk, 64)
    ids = torch.tensor([2, 2, 0, 2, 4], dtype=torch.int32).expand(1, 1, gq, kb).contiguous()
    run_attn(q, k, v, ids, C, BK, fp8=fp8)
    api.sync_status()
    ids[..., 1] = 5  # one behind the last block: reported, left out
    run_attn(q, k, v, ids, C, BK, fp8=fp8)
    with pytest.raises(_lib.MCSError):
        api.sync_status()
    api.sync_status()
    ids[..., 0] = -7
    got = run_attn(q, k, v, ids, C, BK, fp8=fp8)
    assert not got.any()
    kv = torch.tensor([Nk + 1], dtype=torch.int32)  # longer than the store: reported, clamped
    run_attn(q, k, v, None, C, BK, kv=kv, fp8=fp8, poison=False, kvr=torch.tensor([Nk]))
    with pytest.raises(_lib.MCSError):
        api.sync_status()


def test_block_attn_infinities_in_valid_keys():
    """-inf logits leave no weight; a row of nothing else is an empty one."""
    Nk, d = 256, 64
    for C, Nq in ((128, 128), (64, 64), (16, 16), (1, 1)):
        q, k, v = torch.ones(1, 1, Nq, d).bfloat16(), rnd(36, 1, 1, Nk, d), rnd(37, 1, 1, Nk, d)
        k[0, 0, 10:200, 5] = -math.inf
        keep = [i for i in range(Nk) if not 10 <= i < 200]
        want, lse, spread, delta = ref.attn(q, k[:, :, keep], v[:, :, keep], None, C, 64)
        got, gl = api.block_attn(dev(q), dev(k), dev(v), None, C, 64, want_lse=True)
        within(got, want, ref.attn_bound(want, spread, delta), f"C = {C}")
        within(gl, lse, ref.lse_bound(lse, delta), f"C = {C}")
        k[..., 5] = -math.inf
        r = rnd(38, 1, 1, Nq, d)
        got, gl = api.block_attn(dev(q), dev(k), dev(v), None, C, 64, R=dev(r), want_lse=True)
        assert torch.equal(got.cpu(), r) and bool((gl == -math.inf).all())
    api.sync_status()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("C,Nq", [(128, 130), (64, 70), (16, 16), (1, 1)])
@pytest.mark.parametrize("q_size,k_size", [(0.0, 1e-30), (1e-30, 1e-30), (1e-36, 1.0), (1e18, 1e18), (1.0, 0.0)])
def test_block_attn_tiny_and_large_operands(C, Nq, fp8, q_size, k_size):
    """Products far under and over one (logits of 0, or one key that takes all), some keys masked."""
    Nk, BK, d = 320, 64, 64
    q, k = rnd(40, 1, 2, Nq, d, std=q_size), rnd(41, 1, 2, Nk, d, std=k_size)
    q[:, :, ::3] = 0
    run_attn(q, k, rnd(42, 1, 2, Nk, d), None, C, BK, kv=torch.tensor([300], dtype=torch.int32), fp8=fp8,
             scale=1.0 if q_size < 1e10 else 1e-34)


# ------------------------------------------------------------------------------------------ 8-bit store
@pytest.mark.parametrize("B,H,n,d,BK,start,cap,lens", [
    (1, 2, 256, 64, 64, 0, 256, None), (2, 3, 300, 128, 128, 128, 1024, [300, 17]), (2, 1, 1, 64, 32, 32, 96, [1, 0]),
    (1, 5, 130, 128, 32, 0, 160, None), (3, 2, 500, 64, 128, 256, 768, [129, 128, 500]),
])
def test_cache_write(B, H, n, d, BK, start, cap, lens):
    k, v = rnd(40, B, H, n, d), rnd(41, B, H, n, d) * torch.logspace(-30, 30, n)[:, None].bfloat16()
    v = v.contiguous()
    k[0, 0, :BK] = 0
    kv = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    nb = cap // BK
    fill = torch.full((B, H, cap, d), 0x31, dtype=torch.uint8)
    K8, V8 = dev(fill).view(E4M3), dev(fill).clone().view(E4M3)
    ks, vs = torch.full((B, H, nb), 7.0, device=DEV), torch.full((B, H, nb), 9.0, device=DEV)
    mk = torch.full((B, H, nb, d), 5.0, device=DEV)
    api.cache_write(dev(k), dev(v), K8, V8, ks, vs, BK, start=start, means=mk, lens=dev(kv))
    api.sync_status()
    old = float(fill[0, 0, 0, :1].view(E4M3).float())
    for x, x8, s, untouched in ((k, K8, ks, 7.0), (v, V8, vs, 9.0)):
        want = torch.full((B, H, cap, d), old, dtype=torch.float64)
        want_s = torch.full((B, H, nb), untouched, dtype=torch.float64)
        for b, m in enumerate(ref.lengths(kv, B, n)):
            for h in range(H):
                for j in range(-(-m // BK)):
                    rows = x[b, h, j * BK:min((j + 1) * BK, m)]
                    sc = ref.block_scale(rows)
                    want_s[b, h, start // BK + j] = sc
                    # the fp32 quotient, then the nearest e4m3: bit for bit
                    quo = (rows.float() / torch.tensor(sc, dtype=torch.float32)).double()
                    want[b, h, start + j * BK:start + j * BK + len(rows)] = ref.e4m3(quo)
        assert torch.equal(s.double().cpu(), want_s)
        assert torch.equal(x8.double().cpu(), want)
    wm = torch.full((B, H, nb, d), 5.0, dtype=torch.float64)
    m = ref.means(k, BK, kv)
    for b, c in enumerate(ref.lengths(kv, B, n)):
        wm[b, :, start // BK:start // BK + -(-c // BK)] = m[b, :, :-(-c // BK)]
    within(mk, wm, wm.abs() * (ref.FP32 + 2.0 ** -40), "means")


def test_cache_write_special_values():
    x = torch.zeros(1, 1, 32, 64).bfloat16()
    x[0, 0, 0, :6] = torch.tensor([math.inf, -math.inf, math.nan, 3.5, -7.0, 1e-3])
    K8, V8 = (torch.zeros(1, 1, 32, 64, dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2))
    ks, vs = torch.empty(1, 1, 1, device=DEV), torch.empty(1, 1, 1, device=DEV)
    tiny = torch.full((1, 1, 32, 64), 2.0 ** -130).bfloat16()  # amax / 448 under the smallest scale
    api.cache_write(dev(x), dev(tiny), K8, V8, ks, vs, 32)
    got = K8.float().cpu()[0, 0, 0, :6]
    assert float(ks) == 7.0 / 448
    assert got[0] == 448 and got[1] == -448 and got[2].isnan() and got[3] == 224 and got[4] == -448
    assert float(vs) == 2.0 ** -100 and not V8.float().any()
    api.sync_status()


def test_cache_write_exact_ties():
    """Quotients that fall on the middle of two e4m3 values when the scale's reciprocal is no short number."""
    x = torch.zeros(1, 1, 32, 64).bfloat16()
    # scale = 140 / 448 = 5 / 16; x / scale = 17 * 2^k and 19 * 2^k: ties of a 4-bit mantissa
    x[0, 0, 0, 0] = 140.0
    x[0, 0, 1, :4] = torch.tensor([85.0, 95.0, -85.0, -95.0]) / 16
    K8, V8 = (torch.zeros(1, 1, 32, 64, dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2))
    ks, vs = torch.empty(1, 1, 1, device=DEV), torch.empty(1, 1, 1, device=DEV)
    api.cache_write(dev(x), dev(x), K8, V8, ks, vs, 32)
    assert float(ks) == 0.3125
    assert K8.float().cpu()[0, 0, 1, :4].tolist() == [16.0, 20.0, -16.0, -20.0]


# ------------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("d,BK,C", [(64, 64, 64), (128, 128, 128), (128, 32, 16)])
def test_frames_through_the_cache(d, BK, C):
    """Projections -> rotary -> cache -> chosen blocks -> attention, frame after frame, as they are used together."""
    B, H, Hkv, hw, frames, kb = 1, 4, 2, (6, 15), 4, 3
    n = hw[0] * hw[1]
    axes = (16, 24, 24)
    cache = api.KVCache(B, Hkv, 512, d, BK=BK)
    keys, vals = [], []
    for t in range(frames):
        q, k, v = rnd(50 + t, B, n, H, d), rnd(60 + t, B, n, Hkv, d), rnd(70 + t, B, n, Hkv, d)
        pos = torch.stack(torch.meshgrid(torch.tensor([t]), torch.arange(hw[0]), torch.arange(hw[1]), indexing="ij"), -1)
        pos = pos.reshape(n, 3).int()
        Q, K, V = api.rotary(dev(q), dev(k), dev(v), dev(pos), axes, norm="head")
        cache.append(K, V)
        keys.append(K), vals.append(V)
        K, V = torch.cat(keys, 2), torch.cat(vals, 2)
        m = K.shape[2]
        nb = -(-m // BK)
        assert cache.length == m and cache.kv_len.tolist() == [m]
        # the store holds what one write of the whole sequence would
        K8, V8 = (torch.zeros(B, Hkv, 512, d, dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2))
        ks, vs = (torch.ones(B, Hkv, 512 // BK, device=DEV) for _ in range(2))
        mk = torch.zeros(B, Hkv, 512 // BK, d, device=DEV)
        api.cache_write(K, V, K8, V8, ks, vs, BK, means=mk)
        for a, b in ((cache.K8, K8), (cache.V8, V8)):
            assert torch.equal(a.view(torch.uint8)[:, :, :m], b.view(torch.uint8)[:, :, :m])
        assert torch.equal(cache.k_scale, ks) and torch.equal(cache.v_scale, vs) and torch.equal(cache.means, mk)
        assert torch.equal(mk[:, :, :nb], api.block_means(K, BK))
        out, lse = cache.attend(Q, C=C, kb=min(kb, nb), want_lse=True)
        blocks = api.block_topk(Q, cache.means, C, min(kb, nb), BK, kv_len=cache.kv_len)
        want, wl, spread, delta = ref.attn(Q.cpu(), K8.float().cpu(), V8.float().cpu(), blocks.cpu(), C, BK,
                                           kv_len=cache.kv_len.cpu(), k_scale=ks.cpu(), v_scale=vs.cpu())
        within(out, want, ref.attn_bound(want, spread, delta), f"frame {t}")
        within(lse, wl, ref.lse_bound(wl, delta), f"frame {t} lse")
        # one token against everything
        one, _ = cache.attend(Q[:, :, -1:].contiguous(), C=1)
        want, _, spread, delta = ref.attn(Q[:, :, -1:].cpu(), K8.float().cpu(), V8.float().cpu(), None, 1, BK,
                                          kv_len=cache.kv_len.cpu(), k_scale=ks.cpu(), v_scale=vs.cpu())
        within(one, want, ref.attn_bound(want, spread, delta), f"token {t}")
    api.sync_status()


def test_cache_token_by_token_equals_one_write():
    B, H, d, BK, n = 2, 2, 64, 32, 70
    k, v = dev(rnd(80, B, H, n, d)), dev(rnd(81, B, H, n, d))
    one, many = api.KVCache(B, H, 96, d, BK=BK), api.KVCache(B, H, 96, d, BK=BK)
    one.append(k, v)
    for i in range(n):
        many.append(k[:, :, i:i + 1].contiguous(), v[:, :, i:i + 1].contiguous())
    for a, b in ((one.K8, many.K8), (one.V8, many.V8)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(one.k_scale, many.k_scale) and torch.equal(one.means, many.means)
    with pytest.raises(ValueError):
        one.append(k, v)
    api.sync_status()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("C,Nq", [(128, 300), (64, 300), (16, 16), (1, 1)])
def test_block_attn_captured_replayed_and_on_other_streams(C, Nq, fp8):
    B, H, Nk, d, BK, kb = 1, 2, 2048, 64, 64, 9
    gq = -(-Nq // C)
    q, k, v = dev(rnd(90, B, H, Nq, d)), rnd(91, B, H, Nk, d), rnd(92, B, H, Nk, d)
    ks = vs = None
    if fp8:
        (k, ks), (v, vs) = quantised(k, BK), quantised(v, BK)
    k, v, ks, vs = dev(k), dev(v), dev(ks), dev(vs)
    ids = dev(lists(93, B, H, gq, Nk // BK, kb, "holes"))
    call = lambda: api.block_attn(q, k, v, ids, C, BK, k_scale=ks, v_scale=vs, want_lse=True)  # noqa: E731
    want, wl = call()
    side = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(call())
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want) and torch.equal(l, wl)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, l = call()
        m = api.block_means(q, BK)
        t = api.block_topk(q, m, C, min(3, m.shape[2]), BK)
    for seed in (94, 95):
        q.copy_(rnd(seed, B, H, Nq, d))
        graph.replay()
        want, wl = call()
        m2 = api.block_means(q, BK)
        t2 = api.block_topk(q, m2, C, min(3, m.shape[2]), BK)
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(l, wl) and torch.equal(m, m2) and torch.equal(t, t2)
    api.sync_status()


# ------------------------------------------------------------------------------------------ the far ends
def test_block_topk_in_parts():
    """More rows than one part's score keys hold: rows of one key head, and key heads, in turn."""
    for B, Hkv, rep, Nq in ((1, 1, 1, 40000), (3, 1, 2, 9000)):
        q, k = dev(rnd(100, B, Hkv * rep, Nq, 64)), dev(rnd(101, B, Hkv, 32000, 64))
        mk = api.block_means(k, 32)
        got = api.block_topk(q, mk, 1, 5, 32)
        for lo in range(0, Nq, 3000):
            part = q[:, :, lo:lo + 3000].contiguous()
            assert torch.equal(got[:, :, lo:lo + 3000], api.block_topk(part, mk, 1, 5, 32))
    api.sync_status()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("C,Nq,BK", [(128, 128, 128), (64, 100, 32), (16, 16, 64), (1, 2, 64)])
def test_block_attn_offsets_past_32_bits(C, Nq, BK, fp8):
    """Blocks at the end of a store of 2^24 rows (4 GB of keys in bf16) give what they give in a short one."""
    Nk, d, n = 1 << 24, 128, 512
    dt = E4M3 if fp8 else torch.bfloat16
    q, k, v = dev(rnd(110, 1, 1, Nq, d)), rnd(111, 1, 1, n, d), rnd(112, 1, 1, n, d)
    kw, kw_far = {}, {}
    if fp8:
        (k, ks), (v, vs) = quantised(k, BK), quantised(v, BK)
        kw = dict(k_scale=dev(ks), v_scale=dev(vs))
        kw_far = {x: torch.ones(1, 1, Nk // BK, device=DEV) for x in kw}
        for x in kw:
            kw_far[x][..., -(n // BK):] = kw[x]
    far = [torch.empty(1, 1, Nk, d, dtype=torch.uint8 if fp8 else dt, device=DEV) for _ in range(2)]
    for t, x in zip(far, (k, v)):
        t[:, :, -n:] = dev(x.view(torch.uint8) if fp8 else x)
    far = [t.view(dt) for t in far]
    gq, nb = -(-Nq // C), n // BK
    ids = torch.randperm(nb, generator=torch.Generator().manual_seed(113))[:max(1, nb - 1)].int()
    ids = dev(ids.expand(1, 1, gq, -1).contiguous())
    want, wl = api.block_attn(q, dev(k), dev(v), ids, C, BK, want_lse=True, **kw)
    got, gl = api.block_attn(q, *far, ids + (Nk - n) // BK, C, BK, want_lse=True, **kw_far)
    api.sync_status()
    assert torch.equal(got, want) and torch.equal(gl, wl)


def test_cache_write_past_32_bits():
    cap, d, BK, n = 1 << 24, 128, 64, 200
    start = cap - 256
    k, v = dev(rnd(120, 1, 2, n, d)), dev(rnd(121, 1, 2, n, d))
    far = [torch.empty(1, 2, cap, d, dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2)]
    near = [torch.empty(1, 2, 256, d, dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2)]
    sc = [torch.empty(1, 2, m // BK, device=DEV) for m in (cap, cap, 256, 256)]
    mk = [torch.empty(1, 2, m // BK, d, device=DEV) for m in (cap, 256)]
    api.cache_write(k, v, *far, sc[0], sc[1], BK, start=start, means=mk[0])
    api.cache_write(k, v, *near, sc[2], sc[3], BK, means=mk[1])
    for a, b in zip(far, near):
        assert torch.equal(a.view(torch.uint8)[:, :, start:start + n], b.view(torch.uint8)[:, :, :n])
    assert torch.equal(sc[0][..., -4:], sc[2]) and torch.equal(sc[1][..., -4:], sc[3]) and torch.equal(mk[0][:, :, -4:], mk[1])
    api.sync_status()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("C,Nq,kb", [(128, 700, 9), (64, 700, 9), (64, 100, 200)])
def test_block_attn_wait_that_runs_out(C, Nq, kb, d, fp8):
    """A flag that nothing sets, within 20 ms: every role gives up, the call is reported, the next is right."""
    Nk, BK = 16384, 64
    q, k, v = dev(rnd(130, 1, 2, Nq, d)), rnd(131, 1, 2, Nk, d), rnd(132, 1, 2, Nk, d)
    kw = {}
    if fp8:
        (k, ks), (v, vs) = quantised(k, BK), quantised(v, BK)
        kw = dict(k_scale=dev(ks), v_scale=dev(vs))
    k, v = dev(k), dev(v)
    ids = dev(lists(133, 1, 2, -(-Nq // C), Nk // BK, kb, "holes"))
    want = api.block_attn(q, k, v, ids, C, BK, want_lse=True, **kw)
    api.sync_status()
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    lib = _lib.load()
    lib.mcs_set_attn_wait_limit(20_000_000, _lib.ptr(flag))
    try:
        api.block_attn(q, k, v, ids, C, BK, want_lse=True, **kw)
        with pytest.raises(_lib.MCSError) as e:
            api.sync_status()
        assert e.value.status == 7
    finally:
        lib.mcs_set_attn_wait_limit(0, None)
    got = api.block_attn(q, k, v, ids, C, BK, want_lse=True, **kw)
    api.sync_status()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    flag.fill_(1)
    lib.mcs_set_attn_wait_limit(20_000_000, _lib.ptr(flag))
    try:
        got = api.block_attn(q, k, v, ids, C, BK, want_lse=True, **kw)
        api.sync_status()
    finally:
        lib.mcs_set_attn_wait_limit(0, None)
    assert torch.equal(got[0], want[0])


def test_cache_refuses_a_captured_append_and_keeps_its_place():
    cache = api.KVCache(1, 1, 64, 64, BK=32)
    k = dev(rnd(140, 1, 1, 8, 64))
    cache.append(k, k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="captured"):
            cache.append(k, k)
        out, _ = cache.attend(k[:, :, :1].contiguous(), C=1)
    assert cache.length == 8
    graph.replay()
    want, _ = cache.attend(k[:, :, :1].contiguous(), C=1)
    assert torch.equal(out, want)


def test_empty_cache_gives_the_residual():
    cache = api.KVCache(2, 2, 64, 64, BK=32)
    q, r = dev(rnd(141, 2, 4, 5, 64)), dev(rnd(142, 2, 4, 5, 64))
    for kw in (dict(C=1), dict(C=1, kb=2), dict(C=64), dict(C=64, kb=1), dict(C=128)):
        out, lse = cache.attend(q, R=r, want_lse=True, **kw)
        assert torch.equal(out, r) and bool((lse == -math.inf).all())
    api.sync_status()


def test_given_outputs_and_workspace():
    q, k = dev(rnd(143, 1, 2, 3, 64)), dev(rnd(144, 1, 2, 5000, 64))
    want, wl = api.block_attn(q, k, k, None, 1, 32, want_lse=True)
    out, lse = torch.empty_like(q), torch.empty(1, 2, 3, device=DEV)
    n = _lib.load().mcs_block_attn_workspace_size(_lib.BlockShape(1, 2, 2, 3, 5000, 64, 0.0), 1, 32, -(-5000 // 32))
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    o, l = api.block_attn(q, k, k, None, 1, 32, out=out, lse=lse, ws=ws)
    assert o is out and l is lse and torch.equal(out, want) and torch.equal(lse, wl)
    with pytest.raises(_lib.MCSError):
        api.block_attn(q, k, k, None, 1, 32, ws=ws[:256])
    with pytest.raises(ValueError, match="share"):
        api.block_attn(q, k, k, None, 1, 32, out=q)
    mk = api.block_means(k, 32)
    with pytest.raises(ValueError, match="share"):
        api.block_topk(q, mk, 1, 2, 32, blocks=mk.view(torch.int32).flatten()[:12].view(1, 2, 3, 2))
    api.sync_status()
