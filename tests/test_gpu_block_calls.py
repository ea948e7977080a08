"""Block-sparse calls side by side, with odd arguments and at their far ends (needs a B200)."""

import pytest
import torch

import block_reference as ref
from free_sparse_attention_reuse_b200 import api

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
