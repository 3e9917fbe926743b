"""The ``stream`` argument of the scan calls: the memory that a call takes is its own, on both streams."""
import threading
import types

import pytest
import torch

from gated_delta_rule_67_b200 import (kda_scan_backward, kda_scan_backward_ckpt, kda_scan_checkpoint_size, kda_scan_fwd,
                                      kda_scan_step)
from tests.parity import cuda_or_skip

pytestmark = pytest.mark.gpu

LONG = 40_000_000  # cycles: some 20 ms, far longer than a call


def inputs(dev, seed=5, B=4, T=512, D=1024):
    gen = torch.Generator(dev).manual_seed(seed)
    x, dh = (torch.randn(B, T, D, device=dev, generator=gen) for _ in range(2))
    return x, -torch.rand(B, T, D, device=dev, generator=gen), dh, torch.randn(B, D, device=dev, generator=gen)


def outputs(r):
    return [t for t in (r.values() if isinstance(r, dict) else r if isinstance(r, tuple) else (r,)) if t is not None]


def calls(dev):
    x, g, dh, s0 = inputs(dev)
    h, _ = kda_scan_fwd(x, g, s0)
    ckpt = torch.empty(kda_scan_checkpoint_size(*x.shape), dtype=torch.uint8, device=dev)
    kda_scan_fwd(x, g, s0, checkpoint=ckpt)
    xs, gs, new = x[0].contiguous(), g[0].contiguous(), torch.empty_like(dh[0])
    return {"fwd": lambda **k: kda_scan_fwd(x, g, s0, **k), "backward": lambda **k: kda_scan_backward(None, g, h, dh, s0, **k),
            "ckpt": lambda **k: kda_scan_backward_ckpt(ckpt, dh, **k),
            "step": lambda **k: kda_scan_step(xs, gs, dh[0], out_state=new, **k)}


@pytest.mark.parametrize("name", ["fwd", "backward", "ckpt", "step"])
def test_freed_memory_with_work_pending_is_left_alone(name):
    """Tensors freed while the current stream has still to write them: a call on another stream must not get
    their memory, since nothing orders it behind that work."""
    dev = cuda_or_skip()
    call = calls(dev)[name]
    want = [t.clone() for t in outputs(call())]
    side = torch.cuda.Stream(dev)
    torch.cuda.synchronize()
    for _ in range(3):
        old = [torch.empty_like(t) for t in want]
        torch.cuda._sleep(LONG)
        for t in old:
            t.fill_(7)
        del old, t
        got = outputs(call(stream=side))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["fwd", "backward", "ckpt", "step"])
def test_results_last_while_the_current_stream_reads_them(name):
    """A result freed while the current stream has still to read it: the next call on the other stream must not
    get its memory either."""
    dev = cuda_or_skip()
    call = calls(dev)[name]
    want = [t.clone() for t in outputs(call())]
    side = torch.cuda.Stream(dev)
    torch.cuda.synchronize()
    got = outputs(call(stream=side))
    torch.cuda.current_stream(dev).wait_stream(side)
    torch.cuda._sleep(LONG)
    read = [t.clone() for t in got]
    del got
    with torch.cuda.stream(side):
        for _ in range(3):
            outputs(call(stream=side))
            for t in [torch.empty_like(t) for t in want]:
                t.fill_(7)
    torch.cuda.synchronize()
    for a, b in zip(read, want):
        assert torch.equal(a, b)


def test_stream_argument_in_a_captured_graph():
    dev = cuda_or_skip()
    x, g, _, s0 = inputs(dev)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(dev), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream(dev)
        side.wait_stream(main)
        h, s = kda_scan_fwd(x, g, s0, stream=side)
        main.wait_stream(side)
        twice = h + h
    x.mul_(0.5)
    graph.replay()
    want = kda_scan_fwd(x, g, s0)
    assert torch.equal(h, want[0]) and torch.equal(s, want[1]) and torch.equal(twice, want[0] + want[0])


def test_a_stream_of_another_device_is_refused():
    dev = cuda_or_skip()
    x, g, _, _ = inputs(dev)
    other = types.SimpleNamespace(device=torch.device("cuda", x.device.index + 1))
    with pytest.raises(ValueError, match="stream"):
        kda_scan_fwd(x, g, stream=other)


def test_two_threads_on_two_streams():
    """Calls of two threads at once, each on its own stream with memory that the calls take for themselves."""
    dev = cuda_or_skip()
    sizes = [(1, 9000, 40), (2, 700, 264)]  # joined, walked
    data = [inputs(dev, 20 + i, *s) for i, s in enumerate(sizes)]

    def step(x, g, dh, s0):
        h, s = kda_scan_fwd(x, g, s0)
        return [h, s] + outputs(kda_scan_backward(None, g, h, dh, s0))

    want = [step(*d) for d in data]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream(dev)):
            for _ in range(50):
                for a, b in zip(step(*data[i]), want[i]):
                    if not torch.equal(a, b):
                        wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
