"""Block-sparse calls side by side, with odd arguments and at their far ends (needs a B200)."""

import os
import subprocess
import sys

import pytest
import torch

import block_reference as ref
from free_sparse_attention_reuse_b200 import _lib, api

pytestmark = pytest.mark.gpu
DEV = "cuda"


def rnd(seed, *shape, std=1.0):
    return (std * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).bfloat16()


@pytest.mark.parametrize("captured", [False, True])
def test_small_choices_on_two_streams(captured):
    """Calls whose whole workspace is 256 bytes, two at a time: each gives what it gives alone."""
    H, nb, kb, n = 2, 16, 5, 300
    side = [torch.cuda.Stream() for _ in range(2)]
    q = [rnd(200 + i, 1, H, 1, 64).to(DEV) for i in range(2)]
    mk = [rnd(210 + i, 1, H, nb, 64).float().to(DEV) for i in range(2)]
    want = [ref.topk(q[i].cpu(), mk[i].cpu(), 1, kb, 32)[0] for i in range(2)]
    got = [torch.empty(n, 1, H, 1, kb, dtype=torch.int32, device=DEV) for _ in range(2)]
    graphs = []
    for i in range(2):
        if captured:
            out = torch.empty(1, H, 1, kb, dtype=torch.int32, device=DEV)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                api.block_topk(q[i], mk[i], 1, kb, 32, blocks=out)
            graphs.append((graph, out))
    torch.cuda.synchronize()
    for r in range(n):
        for i in range(2):
            with torch.cuda.stream(side[i]):
                if captured:
                    graphs[i][0].replay()
                    got[i][r].copy_(graphs[i][1])
                else:
                    api.block_topk(q[i], mk[i], 1, kb, 32, blocks=got[i][r])
    torch.cuda.synchronize()
    api.sync_status()
    for i in range(2):
        assert torch.equal(got[i].cpu(), want[i].expand(n, -1, -1, -1, -1))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("norm", ["head", "token", None])
@pytest.mark.parametrize("N,H,Hkv", [(1, 130, 65), (1, 1, 4), (1, 3, 1), (2, 5, 33), (40, 2, 2), (3, 65, 129)])
def test_rotary_heads_that_do_not_fill_a_warps_groups(N, H, Hkv, norm, d):
    """Few tokens: a token's heads are shared out over the groups of a warp, which get unlike numbers of them."""
    def within(got, want, size):
        assert ((got.cpu().double() - want).abs() <= ref.rotary_bound(want, size)).all()

    q, k = rnd(220, 1, N, H, d), rnd(221, 1, N, Hkv, d)
    pos = torch.arange(N, dtype=torch.int32)[:, None] * 37 + 5
    for pairs in ("adjacent", "halves"):
        (rq, sq), (rk, sk), _ = ref.rotary(q, k, None, pos, (d // 2,), pairs=pairs, norm=norm)
        Q, K, V = api.rotary(q.to(DEV), k.to(DEV), k.to(DEV), pos.to(DEV), (d // 2,), pairs=pairs, norm=norm)
        within(Q, rq, sq), within(K, rk, sk)
        assert torch.equal(V.cpu(), k.transpose(1, 2))


def within(got, want, bound):
    got = got.cpu().double()
    d = torch.where(got == want, 0.0, (got - want).abs())  # equal infinities
    assert not d.isnan().any() and bool((d <= bound).all()), f"{float((d - bound).max()):.3e} over the bound"


def quantised(k, BK):
    """(e4m3 values, scales) of [B, H, n, d], n a multiple of BK."""
    B, H, n, d = k.shape
    y = k.float().view(B, H, n // BK, BK * d)
    s = (y.abs().amax(-1) / 448.0).clamp_min(2.0 ** -100)
    return (y / s[..., None]).view(B, H, n, d).to(torch.float8_e4m3fn), s.contiguous()


def attn(q, k, v, ids, C, BK, kv=None, fp8=False, scale=None, r=None):
    """One call against the plain form."""
    ks = vs = None
    if fp8:
        (k, ks), (v, vs) = quantised(k, BK), quantised(v, BK)
    want, lse, spread, delta = ref.attn(q, k, v, ids, C, BK, r, kv, ks, vs, scale)
    on = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    got, gl = api.block_attn(on(q), on(k), on(v), on(ids), C, BK, R=on(r), kv_len=on(kv), k_scale=on(ks), v_scale=on(vs),
                             want_lse=True, scale=scale)
    within(got, want, ref.attn_bound(want, spread, delta))
    within(gl, lse, ref.lse_bound(lse.nan_to_num(neginf=0.0), delta))
    return got


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,BK,C", [(64, 32, 1), (128, 32, 16), (64, 128, 16), (128, 64, 1)])
def test_cut_block_between_whole_ones(d, BK, C, fp8):
    """A block that ends at the length, named again and again between whole ones: its cleared rows are filled anew."""
    nb = 6
    kv = torch.tensor([nb * BK - 5], dtype=torch.int32)
    q, k, v = rnd(230, 1, 2, C, d), rnd(231, 1, 1, nb * BK, d), rnd(232, 1, 1, nb * BK, d)
    for ids in ([5, 0, 5, 1, 5, 2], [5, 5, 5, 0, 1, 2], [0, 5, 3, 4, 5, 5]):
        attn(q, k, v, torch.tensor(ids, dtype=torch.int32).expand(1, 2, 1, nb).contiguous(), C, BK, kv, fp8)
    api.sync_status()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("C,Nq,kb", [(128, 700, 3), (64, 700, 1), (64, 100, 200), (16, 32, 40)])
def test_waits_given_up_at_once(C, Nq, kb, d, fp8):
    """No patience at all: a role may give up while copies are under way that another one issued.  They land before
    the CTA ends, the call is reported or right, and so is the next."""
    Nk, BK = 16384, 64
    q, k, v = rnd(240, 1, 2, Nq, d).to(DEV), rnd(241, 1, 2, Nk, d), rnd(242, 1, 2, Nk, d)
    kw = {}
    if fp8:
        (k, ks), (v, vs) = quantised(k, BK), quantised(v, BK)
        kw = dict(k_scale=ks.to(DEV), v_scale=vs.to(DEV))
    k, v = k.to(DEV), v.to(DEV)
    ids = torch.rand(1, 2, -(-Nq // C), Nk // BK, generator=torch.Generator().manual_seed(243)).topk(kb, -1).indices
    ids = ids.int().to(DEV)
    want = api.block_attn(q, k, v, ids, C, BK, want_lse=True, **kw)
    api.sync_status()
    for _ in range(5):
        _lib.load().mcs_set_attn_wait_limit(1, None)
        try:
            got = api.block_attn(q, k, v, ids, C, BK, want_lse=True, **kw)
            try:
                api.sync_status()
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            except _lib.MCSError as e:
                assert e.status == 7
        finally:
            _lib.load().mcs_set_attn_wait_limit(0, None)
        got = api.block_attn(q, k, v, ids, C, BK, want_lse=True, **kw)
        api.sync_status()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("C,Nq", [(1, 1), (1, 6), (16, 16), (128, 130), (64, 70)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gap,smaller", [(12, 256), (14, 256), (16, 4096), (20, 65536), (24, 2 ** 20)])
def test_first_key_takes_the_weight_but_its_value_is_small(gap, smaller, d, C, Nq):
    """8 bits: the other keys' probabilities are around e^-gap, yet their values make the result."""
    Nk, BK = 512, 32
    q, k, v = torch.zeros(1, 1, Nq, d), 0.05 * torch.randn(1, 1, Nk, d, generator=torch.Generator().manual_seed(250)), rnd(251, 1, 1, Nk, d)
    q[..., 0] = 8.0
    k[0, 0, :, 0] = 0.0
    k[0, 0, 0, 0] = gap / 8.0
    v[:, :, :BK] /= smaller
    attn(q.bfloat16(), k.bfloat16(), v.abs(), None, C, BK, fp8=True, scale=1.0)
    api.sync_status()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("C,Nq", [(128, 200), (64, 200), (16, 16), (1, 2)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [40.0, 2000.0, 1e6, 1e8])
def test_logits_far_apart(size, d, C, Nq, fp8):
    """Later keys above the first ones by up to 1e9 octaves, and rows that fall as far: one key takes all."""
    Nk, BK = 1024, 64
    q, k, v = torch.zeros(1, 2, Nq, d), rnd(260, 1, 2, Nk, d).float(), rnd(261, 1, 2, Nk, d)
    q[..., 0] = 16.0
    q[:, 1, ::2, 0] = -16.0
    k[..., 0] = torch.where(torch.arange(Nk) < 500, -size, size) + torch.arange(Nk) * size / 4096
    q, k = q.bfloat16(), k.bfloat16()
    attn(q, k, v, None, C, BK, fp8=fp8, scale=1.0)
    ids = torch.arange(Nk // BK, dtype=torch.int32).expand(1, 2, -(-Nq // C), -1).contiguous()
    attn(q, k, v, ids, C, BK, fp8=fp8, scale=1.0)
    api.sync_status()


def test_cache_grown_on_two_streams():
    """append() on one stream and then on the other, each ordered behind the one before, while both keep allocating:
    the store is that of one stream."""
    B, H, d, BK, n = 1, 2, 64, 32, 90
    k, v = rnd(270, B, H, n, d).to(DEV), rnd(271, B, H, n, d).to(DEV)
    one, two = api.KVCache(B, H, 96, d, BK=BK), api.KVCache(B, H, 96, d, BK=BK)
    one.append(k, v)
    steps = [(k[:, :, i:i + 1].contiguous(), v[:, :, i:i + 1].contiguous()) for i in range(n)]
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i, (x, y) in enumerate(steps):
        me, other = side[i % 2], side[1 - i % 2]
        me.wait_stream(other)
        with torch.cuda.stream(me):
            two.append(x, y)
        with torch.cuda.stream(other):
            torch.full((B, H, BK, d), 1e3, dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    api.sync_status()
    for a, b in ((one.K8, two.K8), (one.V8, two.V8)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(one.k_scale, two.k_scale) and torch.equal(one.means, two.means)
    assert torch.equal(one.kv_len, two.kv_len)


FIRST = {
    "rotary": "api.rotary(x, x, x, torch.zeros(64, 1, dtype=torch.int32, device='cuda'), (64,))[0]",
    "topk": "api.block_topk(x, torch.ones(1, 64, 7000, 64, device='cuda'), 1, 3, 32)",  # 56 kB of keys a row
    "attn": "api.block_attn(x, x, x, torch.zeros(1, 64, 1, 1, dtype=torch.int32, device='cuda'), 128, 32)[0]",
}


@pytest.mark.parametrize("op", FIRST)
def test_first_call_of_a_process(op):
    """Each operator makes ready what it needs itself, whichever comes first."""
    code = ("import torch; from free_sparse_attention_reuse_b200 import api; "
            "x = torch.ones(1, 64, 64, 64, dtype=torch.bfloat16, device='cuda'); "
            f"y = {FIRST[op]}; api.sync_status(); print('sum', float(y.double().sum()))")
    got = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                         cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert got.returncode == 0, got.stderr[-2000:]
    want = {"rotary": 64.0 ** 3, "topk": 64.0 * 64 * (0 + 1 + 2), "attn": 64.0 ** 3}[op]
    assert got.stdout.split() == ["sum", str(want)]


@pytest.mark.parametrize("d,BK,C", [(64, 64, 64), (128, 128, 128), (128, 32, 16), (64, 32, 1)])
def test_whole_path_captured(d, BK, C):
    """Rotary, the store, the choice and the attention in one graph, replayed on other data and on another stream,
    and beside an eager run: what the calls give one after the other."""
    B, H, Hkv, n, cap, kb = 2, 4, 2, 150, 512, 3
    axes, start = (16, 24, 24), 2 * BK
    x = [torch.empty(B, n, m, d, dtype=torch.bfloat16, device=DEV) for m in (H, Hkv, Hkv)]
    pos = torch.empty(B, n, 3, dtype=torch.int32, device=DEV)
    kv, lens = torch.empty(B, dtype=torch.int32, device=DEV), torch.empty(B, dtype=torch.int32, device=DEV)

    def store():
        e = lambda: torch.zeros(B, Hkv, cap, d, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)  # noqa: E731
        s = lambda *t: torch.ones(B, Hkv, cap // BK, *t, device=DEV)  # noqa: E731
        return e(), e(), s(), s(), s(d)

    def path(K8, V8, ks, vs, mk):
        Q, K, V = api.rotary(*x, pos, axes, norm="head")
        api.cache_write(K, V, K8, V8, ks, vs, BK, start=start, means=mk, lens=lens)
        ids = api.block_topk(Q, mk, C, kb, BK, kv_len=kv)
        out, lse = api.block_attn(Q, K8, V8, ids, C, BK, kv_len=kv, k_scale=ks, v_scale=vs, want_lse=True)
        return out, lse, ids, K8.view(torch.uint8), V8.view(torch.uint8), ks, vs, mk

    def fill(seed):
        for i, t in enumerate(x):
            t.copy_(rnd(seed + i, *t.shape))
        pos.copy_(torch.randint(0, 1000, pos.shape, generator=torch.Generator().manual_seed(seed)))
        lens.copy_(torch.tensor([n, n - seed % 97]))
        kv.copy_(start + lens)

    fill(300)
    mine, theirs = store(), store()
    path(*store())
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        got = path(*mine)
    for seed in (310, 320, 333):
        fill(seed)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        want = path(*theirs)  # beside it
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    api.sync_status()
