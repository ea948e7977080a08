"""What the block-sparse calls hand to the C library, without a GPU: its launching functions are replaced by
recorders, its checks and sizes are the library's own, and the tensors live on the CPU."""

import pytest
import torch

from free_sparse_attention_reuse_b200 import _lib, api


class Recorder:
    """The library with its launches recorded: name and arguments of each, status 0."""

    LAUNCHES = ("mcs_rotary", "mcs_block_means", "mcs_block_topk", "mcs_cache_write", "mcs_block_attn")

    def __init__(self, lib):
        self.lib, self.calls = lib, []

    def __getattr__(self, name):
        if name not in self.LAUNCHES:
            return getattr(self.lib, name)

        def launch(*args):
            self.calls.append((name, args))
            return 0

        return launch


@pytest.fixture
def rec(monkeypatch):
    r = Recorder(_lib.load())
    monkeypatch.setattr(api._lib, "load", lambda: r)
    monkeypatch.setattr(api, "_on_device", lambda **kw: None)
    monkeypatch.setattr(api, "_here", lambda t: None)
    monkeypatch.setattr(api, "_stream", lambda t: None)
    monkeypatch.setattr(api, "_plans", {})
    monkeypatch.setattr(api, "_blanks", {})
    return r


def bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


@pytest.mark.parametrize("H,nb,C", [(2, 16, 1), (1, 32, 1), (8, 4, 1), (1, 1, 1), (1, 2, 16)])
def test_choice_never_writes_to_a_shared_workspace(rec, H, nb, C):
    """The choice holds its scores in the workspace, however small it is: two calls may be under way at once."""
    q, k = bf(1, H, 1, 64), bf(1, H, 32 * nb, 64)
    api.block_attn(q, k, k, torch.zeros(1, H, 1, 1, dtype=torch.int32), C, 32)  # one part: the shared tensor
    shared = {t.data_ptr() for t in api._blanks.values()}
    assert shared
    api.block_topk(q, torch.zeros(1, H, nb, 64), C, 1, 32)
    name, args = rec.calls[-1]
    assert name == "mcs_block_topk" and args[8] not in shared
    assert args[9] == rec.lib.mcs_block_topk_workspace_size(_lib.BlockShape(1, H, H, 1, 32 * nb, 64, 0.0), C, 32)
