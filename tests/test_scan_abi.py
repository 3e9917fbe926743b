"""The scan entry points on the host: sizes, and every refusal, before any CUDA call is made."""
import pytest
import torch

from gated_delta_rule_67_b200 import binding
from gated_delta_rule_67_b200.build import build

BAD, NO = binding.KDA_ERR_INVALID_ARG, binding.KDA_ERR_UNSUPPORTED
A = 1 << 40  # fake device addresses, 1 GiB apart


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.load()


def at(i):
    return A + (i << 30)


def fwd(lib, **kw):
    a = dict(x=at(0), g=at(1), s0=at(2), cu=None, n=0, h=at(3), sT=at(4), ckpt=None, B=2, T=300, D=256, dtype=1, prep=0,
             ig=0, ws=at(8), wsb=1 << 28)
    a.update(kw)
    return lib.kda_scan_fwd(*a.values(), None)


def bwd(lib, **kw):
    a = dict(x=at(0), g=at(1), h=at(2), s0=at(3), dh=at(4), dsT=at(5), cu=None, n=0, dx=at(6), dg=at(7), ds0=at(8), B=2,
             T=300, D=256, dtype=1, prep=0, ig=1, ws=at(9), wsb=1 << 28)
    a.update(kw)
    return lib.kda_scan_backward(*a.values(), None)


def ckpt(lib, **kw):
    a = dict(ckpt=at(0), dh=at(4), dsT=at(5), cu=None, n=0, dx=at(6), dg=at(7), ds0=at(8), B=2, T=300, D=256, dtype=1,
             prep=0, ig=1, ws=at(9), wsb=1 << 28)
    a.update(kw)
    return lib.kda_scan_backward_ckpt(*a.values(), None)


@pytest.mark.parametrize("call", [fwd, bwd, ckpt])
def test_sizes_and_flags(lib, call):
    for kw in (dict(B=-1), dict(T=-1), dict(D=0), dict(dtype=2), dict(prep=1), dict(prep=4), dict(prep=8), dict(ig=2),
               dict(ig=-1), dict(cu=at(10), n=3), dict(cu=at(10), n=0, B=1), dict(cu=at(10), n=-1, B=1),
               dict(cu=at(10) + 2, n=3, B=1)):
        assert call(lib, **kw) == BAD, kw
    assert call(lib, B=2 ** 30, T=2 ** 30, D=2 ** 30) == NO
    assert call(lib, B=1, T=2 ** 31 - 1, D=2 ** 31 - 1) == NO
    assert call(lib, B=1, T=1, D=2 ** 30, cu=at(10), n=2 ** 30) == NO


@pytest.mark.parametrize("call,needed,optional", [
    (fwd, ["x", "g", "h"], ["s0", "sT", "ckpt"]), (bwd, ["x", "g", "h", "dh", "dx", "dg"], ["s0", "dsT", "ds0"]),
    (ckpt, ["ckpt", "dh", "dx", "dg"], ["dsT", "ds0"])])
def test_pointers(lib, call, needed, optional):
    for name in needed:
        assert call(lib, **{name: None}) == BAD, name
    for name in needed + optional:
        assert call(lib, **{name: at(11) + 8}) == BAD, name


def test_overlaps(lib):
    big = 2 * 300 * 256 * 2 - 16  # the last 16 bytes of a [2, 300, 256] bf16 tensor
    for out in ("h", "sT", "ckpt"):
        for i in (0, 1):
            assert fwd(lib, **{out: at(i) + big}) == BAD, (out, i)
    assert fwd(lib, h=at(2)) == BAD and fwd(lib, sT=at(2) + 16) == BAD and fwd(lib, sT=at(3)) == BAD
    assert fwd(lib, ckpt=at(3)) == BAD and fwd(lib, ckpt=at(4)) == BAD
    for out in ("dx", "dg", "ds0"):
        for i in (0, 1, 2, 3, 4, 5):
            assert bwd(lib, **{out: at(i)}) == BAD, (out, i)
        for i in (0, 4, 5):
            assert ckpt(lib, **{out: at(i)}) == BAD, (out, i)
    for call in (bwd, ckpt):
        assert call(lib, dx=at(7)) == BAD and call(lib, dg=at(8)) == BAD
        assert call(lib, cu=at(10), n=3, B=1, dx=at(10) - 16) == BAD
    assert fwd(lib, cu=at(10), n=3, B=1, h=at(10) - 16) == BAD


def test_workspace(lib):
    need = lib.kda_scan_workspace_size(2, 300, 256, 0, 1)
    if need:
        for call in (fwd, bwd, ckpt):
            assert call(lib, ws=None) == BAD and call(lib, wsb=need - 1) == BAD and call(lib, ws=at(9) + 16) == BAD
            assert call(lib, ws=at(4)) == BAD
    f = lib.kda_scan_workspace_size
    assert f(-1, 1, 1, 0, 1) == f(1, -1, 1, 0, 1) == f(1, 1, 0, 0, 1) == f(1, 1, 1, -1, 1) == f(1, 1, 1, 0, 7) == 0
    assert f(2, 300, 256, 3, 1) == 0  # packed sequences need B = 1
    assert f(0, 300, 256, 0, 1) == f(2, 0, 256, 0, 1) == 0
    assert f(2 ** 30, 2 ** 30, 2 ** 30, 0, 1) == 0
    c = lib.kda_scan_checkpoint_size
    assert c(-1, 1, 1) == c(1, -1, 1) == c(1, 1, 0) == c(2 ** 30, 2 ** 30, 2 ** 30) == 0
    assert c(1, 1, 1) == 1024


@pytest.mark.parametrize("kw,size", [(dict(ckpt=at(12)), (2, 300, 256, 0, 1, 1)),
                                     (dict(B=1, cu=at(10), n=3), (1, 300, 256, 3, 1, 0)),
                                     (dict(B=1, T=100000, D=64), (1, 100000, 64, 0, 1, 0))],
                         ids=["checkpoint", "packed", "few-chains"])
def test_workspace_is_asked_for(lib, kw, size):
    need = lib.kda_scan_workspace_size_ex(*size)
    assert need > 0 and lib.kda_scan_workspace_size_ex(*size[:5], 1) >= need
    for bad in (dict(ws=None), dict(wsb=need - 1), dict(ws=at(8) + 16), dict(ws=at(3)), dict(ws=at(1))):
        assert fwd(lib, **kw, **bad) == BAD, bad
    assert lib.kda_scan_workspace_size(*size[:5]) == lib.kda_scan_workspace_size_ex(*size[:5], 0)


def test_step(lib):
    def step(x=at(0), g=at(1), s=at(2), o=at(2), h=at(3), N=4, D=256, dtype=1, prep=0, ig=0):
        return lib.kda_scan_step(x, g, s, o, h, N, D, dtype, prep, ig, None)
    for name in ("x", "g", "s", "o", "h"):
        assert step(**{name: None}) == BAD and step(**{name: at(9) + 4}) == BAD, name
    for kw in (dict(N=-1), dict(D=0), dict(dtype=3), dict(prep=1), dict(ig=5), dict(o=at(2) + 16), dict(o=at(0)),
               dict(h=at(0)), dict(h=at(1)), dict(h=at(2)), dict(o=at(3), s=at(2))):
        assert step(**kw) == BAD, kw
    assert step(N=2 ** 30, D=2 ** 30) == NO
    assert step(N=0) == binding.KDA_OK


def test_binding_refuses():
    x = torch.zeros(1, 4, 8)
    for call in (lambda: binding.kda_scan_fwd(x, x), lambda: binding.kda_scan_step(x[0], x[0], x[0]),
                 lambda: binding.kda_scan_backward(x, x, x, x), lambda: binding.kda_scan_backward_ckpt(x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        binding.kda_scan_fwd(None, x)
    with pytest.raises(TypeError):
        binding.kda_scan_workspace_size(1, 1, 1, 0, torch.float16)
