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
