"""The recurrence's kernels on every way through them, against the fp64 oracle, with the bounds of
tests/test_gpu_scan.py.  They hold with 6 u for alpha and 1 - alpha (u = 2^-24): ex2.approx 2^-22.5 = 2.9 u and
what the exponent's rounding leaves out, with a correction of one more rounding; the sigmoid's sum u and its
reciprocal, after a Newton step, 1.5 u, times e for the smaller one.
"""
import pytest
import torch

from gated_delta_rule_67_b200 import kda_scan_backward_ckpt, kda_scan_checkpoint_size, kda_scan_fwd
from tests.parity import cuda_or_skip
from tests.test_gpu_scan import (DTYPE_IDS, DTYPES, MODE_IDS, MODES, check_backward, check_checkpoint, check_forward, how,
                                 make)

pytestmark = pytest.mark.gpu


def through_checkpoint(B, T, D, cu, dtype, raw, complement, seed):
    """Forward with checkpoint, the checkpoint's values, and the gradients for them."""
    dev = cuda_or_skip()
    x, g, s0, dh, dsT = make(B, T, D, dtype, raw, seed, cu)
    ckpt = torch.empty(kda_scan_checkpoint_size(B, T, D), dtype=torch.uint8, device=dev).fill_(0xa5)
    got = kda_scan_fwd(x.to(dev), g.to(dev), s0.to(dev), checkpoint=ckpt, **how(raw, complement, cu))
    _, z, E, lam = check_forward(x, g, s0, raw, complement, cu, got=got)
    lam8, z8 = check_checkpoint(ckpt, x, z, E, lam, raw, cu)
    got = kda_scan_backward_ckpt(ckpt, dh.to(dev), dsT.to(dev), **how(raw, complement, cu))
    check_backward(got, lam8, z8, dh, dsT, raw, complement, cu)


@pytest.mark.parametrize("raw,complement", MODES, ids=MODE_IDS)
@pytest.mark.parametrize("dtype", DTYPES, ids=DTYPE_IDS)
@pytest.mark.parametrize("B,T,D", [(60, 700, 133), (3, 330, 4001)], ids=["D133", "D4001"])
def test_checkpoint_of_ragged_rows_over_many_tiles(B, T, D, dtype, raw, complement):
    """Dense rows that are no multiple of 16 bytes, every block with several tiles one after the other: what a
    warp keeps of a tile (the scales of its rows) lasts until all its lanes are done with it."""
    through_checkpoint(B, T, D, None, dtype, raw, complement, 210)
