"""The recurrence's workspace: every call with rows has a header to report a wait that gave up, and clears it."""
import pytest
import torch

from gated_delta_rule_67_b200 import binding
from gated_delta_rule_67_b200.build import build
from tests.parity import cuda_or_skip

# walked by one block, by several, joined; packed
SIZES = [(1, 1, 1, 0), (2, 300, 256, 0), (3, 900, 2048, 0), (1, 9000, 40, 0), (1, 500, 72, 2)]


@pytest.mark.parametrize("B,T,D,seqs", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_every_call_with_rows_has_a_header(B, T, D, seqs, dtype):
    build()
    sizes = [binding.kda_scan_workspace_size(B, T, D, seqs, dtype, checkpoint=c) for c in (False, True)]
    assert 256 <= sizes[0] <= sizes[1]
    assert binding.kda_scan_workspace_size(B, 0, D, seqs, dtype) == 0


def test_a_call_with_rows_refuses_to_go_without():
    build()
    lib, A = binding.load(), 1 << 40
    for ws, size in ((None, 0), (None, 256), (A + (9 << 30), 255), (A + (9 << 30) + 16, 512), (A, 256)):
        st = lib.kda_scan_fwd(A, A + (1 << 30), None, None, 0, A + (2 << 30), None, None, 2, 300, 256, 1, 0, 0, ws, size, None)
        assert st == binding.KDA_ERR_INVALID_ARG, (ws, size)


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,D,seqs", SIZES)
def test_calls_clear_a_dirty_header(B, T, D, seqs):
    dev = cuda_or_skip()
    x = torch.randn(B, T, D, device=dev)
    g = -torch.rand(B, T, D, device=dev)
    cu = torch.tensor([0, 100, T], dtype=torch.int32, device=dev) if seqs else None
    ckpt = torch.empty(binding.kda_scan_checkpoint_size(B, T, D), dtype=torch.uint8, device=dev)
    want = binding.kda_scan_fwd(x, g, cu_seqlens=cu)[0]
    ws = torch.empty(binding.kda_scan_workspace_size(B, T, D, seqs, torch.float32), dtype=torch.uint8, device=dev)
    for call in (lambda: binding.kda_scan_fwd(x, g, cu_seqlens=cu, workspace=ws),
                 lambda: binding.kda_scan_fwd(x, g, cu_seqlens=cu, checkpoint=ckpt, workspace=ws),
                 lambda: binding.kda_scan_backward(None, g, want, x, cu_seqlens=cu, workspace=ws),
                 lambda: binding.kda_scan_backward_ckpt(ckpt, x, cu_seqlens=cu, workspace=ws)):
        ws.fill_(0x5a)
        assert binding.kda_chunk_fwd_check(ws) == binding.KDA_ERR_TIMEOUT
        out = call()
        assert binding.kda_chunk_fwd_check(ws) == binding.KDA_OK
        if isinstance(out, tuple):
            assert torch.equal(out[0], want)


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,D,seqs", SIZES)
def test_captured_calls_without_a_workspace(B, T, D, seqs):
    """The memory that a call takes for itself belongs to the graph while one is captured."""
    dev = cuda_or_skip()
    gen = torch.Generator(dev).manual_seed(3)
    x, dh = (torch.randn(B, T, D, device=dev, generator=gen) for _ in range(2))
    g = -torch.rand(B, T, D, device=dev, generator=gen)
    cu = torch.tensor([0, T // 3, T], dtype=torch.int32, device=dev) if seqs else None
    ckpt = torch.empty(binding.kda_scan_checkpoint_size(B, T, D), dtype=torch.uint8, device=dev)

    def step():
        h, s = binding.kda_scan_fwd(x, g, checkpoint=ckpt, cu_seqlens=cu)
        a = binding.kda_scan_backward(None, g, h, dh, cu_seqlens=cu)
        b = binding.kda_scan_backward_ckpt(ckpt, dh, cu_seqlens=cu)
        return [h, s] + [d[n] for d in (a, b) for n in ("dx", "dg", "dS0")]

    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream(dev).wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for scale in (0.5, -2.0):
        x.mul_(scale)
        graph.replay()
        got = [t.clone() for t in out]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
