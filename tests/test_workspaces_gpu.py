"""The cached workspaces: what growing keeps and gives back."""
import weakref

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gqa():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import grouped_query_attention_fwd_b200 as m
    return m


def test_outgrown_workspaces_are_given_back(gqa):
    s = torch.cuda.Stream()
    seen, most, made = [], 0, 0
    before = torch.cuda.memory_allocated()
    for n in range(1, 40):
        ws = gqa.workspace_for("cuda", n << 20, s.cuda_stream)
        assert ws.numel() >= n << 20 and not ws[:1 << 16].any()
        made += ws.numel() > most
        most = max(most, ws.numel())
        seen.append(weakref.ref(ws))
        del ws
    held = {id(r()) for r in seen if r() is not None}
    assert len(held) == 1  # the last one
    assert most <= 2 * (39 << 20)
    assert torch.cuda.memory_allocated() - before <= most + (1 << 20)
    assert made <= 7  # few of the 39 sizes made one of their own


def test_growth_is_bounded(gqa):
    s = torch.cuda.Stream()
    gqa.workspace_for("cuda", 300 << 20, s.cuda_stream)
    ws = gqa.workspace_for("cuda", 301 << 20, s.cuda_stream)
    assert 301 << 20 <= ws.numel() <= 364 << 20
    assert gqa.workspace_for("cuda", 64 << 20, s.cuda_stream) is ws


def _qkv(B, Hq, Hkv, S, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(B, Hq, 1, D, generator=g, device="cuda").bfloat16(),
            *(torch.randn(B, Hkv, S, D, generator=g, device="cuda").bfloat16() for _ in range(2)))


def test_a_captured_workspace_stays(gqa):
    """A graph of the 16-bit forward points at its stream's workspace: growing
    that one later must not take it away."""
    q, k, v = _qkv(4, 16, 4, 4000, 128, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        want = gqa.forward(q, k, v)  # an eager call first: the workspace is in use, and zeroed
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = gqa.forward(q, k, v)
        old = weakref.ref(gqa.workspace_for("cuda", 256))
        at = old().data_ptr()
        big = gqa.workspace_for("cuda", old().numel() + 1)
        assert big.data_ptr() != at and old() is not None
        # Whoever asks for memory now does not get the graph's.
        junk = [torch.full((old().numel(),), 255, dtype=torch.uint8, device="cuda")
                for _ in range(4)]
        assert all(j.data_ptr() != at for j in junk)
        for _ in range(3):
            out.zero_()
            g.replay()
            s.synchronize()
            assert torch.equal(out, want)
    del g
