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


def test_scalar_arguments_count_by_value(rec):
    """A tensor (or array) as a scalar argument, changed in place between two calls of the same shapes."""
    q, k, ids = bf(1, 2, 64, 64), bf(1, 2, 64, 64), torch.zeros(1, 2, 1, 1, dtype=torch.int32)
    scale = torch.tensor(0.5)
    for x in (0.5, 0.25):
        scale.fill_(x)
        api.block_attn(q, k, k, ids, 64, 32, scale=scale)
        assert rec.calls[-1][1][0].scale == x
    theta, eps = torch.tensor(100.0), torch.tensor(0.5)
    axis, pos = torch.tensor(32), torch.zeros(64, 2, dtype=torch.int32)
    for x in (0.5, 0.25):
        eps.fill_(x), theta.fill_(200 * x), axis.fill_(int(64 * x))
        api.rotary(q.transpose(1, 2), None, None, pos, (axis, 16), theta=theta, eps=eps, norm="head")
        a = rec.calls[-1][1][0]
        assert a.eps == x and a.theta == 200 * x and a.axis_dim[0] == int(64 * x)
    for key in api._plans:
        assert not any(isinstance(x, torch.Tensor) for part in key for x in (part if isinstance(part, tuple) else (part,)))


@pytest.mark.parametrize("axes", [(32.5, 16), [16, 15.5]])
def test_axes_that_are_no_whole_numbers(rec, axes):
    q = bf(1, 64, 2, 64)
    with pytest.raises(ValueError, match="whole"):
        api.rotary(q, None, None, torch.zeros(64, 2, dtype=torch.int32), axes)


def store(B=1, H=2, cap=128, d=64, BK=32):
    e4m3 = lambda: torch.zeros(B, H, cap, d).to(torch.float8_e4m3fn)  # noqa: E731
    return dict(K=bf(B, H, 64, d), V=bf(B, H, 64, d), K8=e4m3(), V8=e4m3(), ks=torch.zeros(B, H, cap // BK),
                vs=torch.zeros(B, H, cap // BK), means=torch.zeros(B, H, cap // BK, d))


def overlay(t, other):
    """A tensor like t that lies over the memory of `other` (as far as it goes)."""
    flat = other.view(torch.uint8).flatten()
    return flat[:t.numel() * t.element_size()].view(t.dtype).view(t.shape)


@pytest.mark.parametrize("a,b", [("V8", "K8"), ("K8", "means"), ("ks", "vs"), ("vs", "K8"), ("ks", "means"), ("means", "V8"),
                                 ("K8", "K"), ("V8", "V"), ("vs", "V"), ("means", "K"), ("lens", "ks"), ("lens", "K8")])
def test_store_in_overlapping_memory(rec, monkeypatch, a, b):
    big = torch.zeros(1 << 16, dtype=torch.uint8)
    t = store()
    t["lens"] = torch.zeros(1, dtype=torch.int32)
    t[b] = overlay(t[b], big)
    t[a] = overlay(t[a], big)
    monkeypatch.setattr(Recorder, "LAUNCHES", ())  # the library's own check, which comes before any launch
    with pytest.raises(ValueError, match="share"):
        api.cache_write(t["K"], t["V"], t["K8"], t["V8"], t["ks"], t["vs"], 32, means=t["means"], lens=t["lens"])


def test_store_side_by_side_in_one_buffer(rec):
    """Parts of one buffer that touch do not share memory."""
    t = store()
    buf, at = torch.zeros(1 << 16, dtype=torch.uint8), 0
    for n in ("K8", "V8", "ks", "vs", "means"):
        x = t[n]
        t[n] = overlay(x, buf[at:])
        at += x.numel() * x.element_size()
    api.cache_write(t["K"], t["V"], t["K8"], t["V8"], t["ks"], t["vs"], 32, means=t["means"])
    api._apart({n: t[n] for n in ("K8", "V8", "ks", "vs", "means")}, dict(K=t["K"], V=t["V"]))
    assert rec.calls[-1][0] == "mcs_cache_write"


def test_outputs_apart_from_each_other(rec):
    x, pos = bf(1, 8, 2, 64), torch.zeros(8, 1, dtype=torch.int32)
    o = bf(1, 2, 8, 64)
    with pytest.raises(ValueError, match="share"):
        api.rotary(x, x, None, pos, (64,), out=(o, o, None))
    with pytest.raises(ValueError, match="of them"):
        api.rotary(x, None, None, pos, (64,), out=(o, None))
    q, k = bf(1, 2, 64, 64), bf(1, 2, 64, 64)
    out, ids = bf(1, 2, 64, 64), torch.zeros(1, 2, 1, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="share"):
        api.block_attn(q, k, k, ids, 64, 32, out=out, lse=overlay(torch.zeros(1, 2, 64), out))
    with pytest.raises(ValueError, match="share"):
        api.block_attn(q, k, k, ids, 64, 32, ws=q.view(torch.uint8).flatten())
    with pytest.raises(ValueError, match="share"):
        api.block_topk(q, torch.zeros(1, 2, 2, 64), 64, 1, 32, ws=q.view(torch.uint8).flatten())
    assert not rec.calls


def test_open_rows_stay_in_their_memory(rec):
    """What append() keeps between calls, which may come on different streams, is never freed or moved; the rows
    handed to the store are the unfinished block's and the new ones."""
    c = api.KVCache(1, 2, 256, 64, BK=32, device="cpu")
    held = lambda: {t.data_ptr() for t in vars(c).values() if isinstance(t, torch.Tensor)} | {  # noqa: E731
        t.data_ptr() for t in c._open}
    memory = held()
    rows = torch.arange(1, 101).bfloat16()[None, None, :, None].expand(1, 2, 100, 64).contiguous()
    at = 0
    for n in (5, 0, 1, 40, 18, 32, 3):
        c.append(rows[:, :, at:at + n].contiguous(), -rows[:, :, at:at + n].contiguous())
        at += n
        if n:
            _, args = rec.calls[-1]
            first = (at - n) // 32 * 32
            assert args[4] == first and args[0].N == at - first
        assert c.length == at and held() == memory and int(c.kv_len[0]) == at
        tail = at % 32
        k, v = c._open_rows(tail)
        assert torch.equal(k, rows[:, :, at - tail:at])
        assert torch.equal(v, -rows[:, :, at - tail:at])
    assert len(rec.calls) == 6
