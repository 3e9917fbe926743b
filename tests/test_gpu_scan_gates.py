"""How exact the recurrence's alpha is near 1, where a memory of n rows multiplies its error by n.

u = 2^-24.  A state of 1, one row and no input give alpha itself: h_1 = alpha * 1 + 0, without a rounding.
For -1/32 < g <= 0 alpha = 1 + g q, q = (e^g - 1) / g: one rounding at the end, half a step of the values from
1/2 to 1, u / 2; q, from 0.98 to 1, is off by at most two such roundings and what its polynomial leaves out,
which is at most 0.09 u of alpha (with w for (q - 1) / g a straight line: 1 / (32^2 * 192), times g^2).  So
|error| <= (1/2 + 0.1 + 2 |g|) u.

Over n rows the state is multiplied n times, each alpha off by (0.6 + 2 |g|) u / alpha of itself, each product
by u at most; a segment's, a unit's and a tile's pair are joined by no more products than rows, and what enters
a tile passes 8 units and 4 segments more: (n (1 + (0.6 + 2 |g|) / alpha) + 16 + n / 64) u of the value.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_67_b200 import kda_scan_backward, kda_scan_backward_ckpt, kda_scan_checkpoint_size, kda_scan_fwd, \
    kda_scan_step
from gated_delta_rule_67_b200.binding import KDA_SCAN_INPUT_COMPLEMENT, KDA_SCAN_INPUT_PLAIN
from oracle import scan
from tests.parity import cuda_or_skip

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def gates(D, least):
    """D log-gates from -2^-13 down to `least`, as fp32."""
    return -torch.exp2(torch.linspace(-13.0, float(np.log2(-least)), D, dtype=torch.float64)).float()


def check(alpha, g):
    g = g.double().cpu().numpy()
    off = np.abs(alpha.double().cpu().numpy() - np.exp(g))
    bound = (0.6 + 2 * np.abs(g)) * U
    assert (off <= bound).all(), (float((off / U).max()), int((off > bound).sum()))


@pytest.mark.parametrize("input_gate", [KDA_SCAN_INPUT_PLAIN, KDA_SCAN_INPUT_COMPLEMENT], ids=["plain", "complement"])
def test_alpha_of_log_gates_is_rounded_once(input_gate):
    dev = cuda_or_skip()
    how = dict(input_gate=input_gate)
    D = 4096
    g = gates(D, -0.0312).to(dev)
    one, zero = torch.ones(1, D, device=dev), torch.zeros(1, 1, D, device=dev)
    h, s = kda_scan_fwd(zero, g.view(1, 1, D), one, **how)
    check(h[0, 0], g)
    check(s[0], g)
    check(kda_scan_step(zero[0], g.view(1, D), one.clone(), **how)[0], g)
    # dS0 = alpha_1 d_1, d_1 = 1
    check(kda_scan_backward(zero, g.view(1, 1, D), zero, one.view(1, 1, D), **how)["dS0"][0], g)
    ckpt = torch.empty(kda_scan_checkpoint_size(1, 1, D), dtype=torch.uint8, device=dev)
    kda_scan_fwd(zero, g.view(1, 1, D), one, checkpoint=ckpt, **how)
    lam = torch.from_numpy(scan.unpack(ckpt.cpu().numpy(), 1, 1, D)[0][0, 0])
    near = (lam > -1 / 32).numpy()
    got = kda_scan_backward_ckpt(ckpt, one.view(1, 1, D), **how)["dS0"][0].cpu()
    check(got[near], lam[near])


@pytest.mark.parametrize("T", [100, 1000, 4000])
def test_long_memory_keeps_its_exactness(T):
    dev = cuda_or_skip()
    D = 640
    g = gates(D, max(-0.0312, -60.0 / T))
    one, rows = torch.ones(1, D, device=dev), g.expand(1, T, D).contiguous().to(dev)
    zero = torch.zeros(1, T, D, device=dev)
    h, s = kda_scan_fwd(zero, rows, one)
    n = np.arange(1, T + 1)[:, None]
    g = g.double().numpy()[None]
    want, bound = np.exp(n * g), (n * (1 + (0.6 + 2 * np.abs(g)) * np.exp(-g)) + 16 + n / 64) * U
    off = np.abs(h[0].double().cpu().numpy() / want - 1)
    assert (off <= bound).all(), float((off / bound).max())
    # the same rows backwards: dS0 = alpha^T for dL/d final_state = 1
    back = kda_scan_backward(None, rows, zero, zero, None, one)["dS0"][0].double().cpu().numpy()
    assert (np.abs(back / want[-1] - 1) <= bound[-1]).all()


@pytest.mark.parametrize("input_gate", [KDA_SCAN_INPUT_PLAIN, KDA_SCAN_INPUT_COMPLEMENT], ids=["plain", "complement"])
def test_alpha_at_every_size_of_a_log_gate(input_gate):
    """Of either sign, as far as exp and its rounding are normal numbers: within 6 u of alpha."""
    dev = cuda_or_skip()
    half = torch.exp2(torch.linspace(-20.0, np.log2(87.0), 3000, dtype=torch.float64)).float()
    g = torch.cat([-half, torch.zeros(2), half]).to(dev)
    D = g.numel()
    one, zero = torch.ones(1, D, device=dev), torch.zeros(1, D, device=dev)
    want = np.exp(g.double().cpu().numpy())
    for got in (kda_scan_step(zero, g.view(1, D), one.clone(), input_gate=input_gate),
                kda_scan_fwd(zero[None], g.view(1, 1, D), one, input_gate=input_gate)[0][0]):
        off = np.abs(got[0].double().cpu().numpy() / want - 1)
        assert (off <= 6 * U).all(), float(off.max() / U)
