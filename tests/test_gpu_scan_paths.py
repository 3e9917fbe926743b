"""The recurrence's kernels on every way through them, against the fp64 oracle, with the bounds of
tests/test_gpu_scan.py.  They hold with 6 u for alpha and 1 - alpha (u = 2^-24): ex2.approx 2^-22.5 = 2.9 u and
what the exponent's rounding leaves out, with a correction of one more rounding; the sigmoid's sum u and its
reciprocal, after a Newton step, 1.5 u, times e for the smaller one.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_67_b200 import kda_scan_backward, kda_scan_backward_ckpt, kda_scan_checkpoint_size, kda_scan_fwd
from oracle import scan
from tests.parity import cuda_or_skip
from tests.test_gpu_scan import (DTYPE_IDS, DTYPES, MODE_IDS, MODES, U, check_backward, check_checkpoint, check_forward,
                                 firsts, how, make, near)

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


# bf16 and at least 128 blocks of 64 channels: two blocks walk a chain (130), one (189); packed; rows that are
# no multiple of 16 bytes; a width that ends inside a block of 64; several tiles of 104 rows each
WIDE = [(2, 330, 4104, None), (3, 330, 4000, None), (2, 120, 4097, None), (1, 330, 8200, [3, 3, 4, 104, 105, 300, 300]),
        (1, 215, 9700, [0, 104, 208, 215]), (1, 330, 8131, [0, 1, 100, 320])]


@pytest.mark.parametrize("raw,complement", MODES, ids=MODE_IDS)
@pytest.mark.parametrize("B,T,D,cu", WIDE, ids=[f"{c[0]}x{c[1]}x{c[2]}" for c in WIDE])
def test_checkpoint_of_many_chains(B, T, D, cu, raw, complement):
    through_checkpoint(B, T, D, cu, torch.bfloat16, raw, complement, 220)


# fewer than 12 chains of more than 32 tiles: joined tile by tile.  Sequences over many tiles, within one, and
# over a group of 16 tiles; rows of no sequence at both ends
JOINED = [(1, 9000, 24, None), (2, 8500, 19, None), (1, 9000, 72, [5, 100, 100, 4500, 4501, 8990]),
          (1, 9000, 19, [0, 3700, 3701, 9000])]


@pytest.mark.parametrize("complement", [False, True], ids=["plain", "complement"])
@pytest.mark.parametrize("raw", [False, True], ids=["log", "raw"])
@pytest.mark.parametrize("dtype", DTYPES, ids=DTYPE_IDS)
@pytest.mark.parametrize("B,T,D,cu", JOINED, ids=["dense", "dense-ragged", "packed", "packed-ragged"])
def test_joined_chains(B, T, D, cu, dtype, raw, complement):
    dev = cuda_or_skip()
    through_checkpoint(B, T, D, cu, dtype, raw, complement, 230)
    x, g, s0, dh, dsT = make(B, T, D, dtype, raw, 231, cu)
    h = torch.from_numpy(scan.forward(x, g, s0, raw=raw, complement=complement, cu=cu)[0]).to(dtype)
    got = kda_scan_backward(x.to(dev), g.to(dev), h.to(dev), dh.to(dev), s0.to(dev), dsT.to(dev),
                            **how(raw, complement, cu))
    check_backward(got, scan.log_gate(g, raw), scan.saved(x, h, s0, complement=complement, cu=cu), dh, dsT, raw,
                   complement, cu)


@pytest.mark.parametrize("from_checkpoint", [False, True], ids=["activations", "checkpoint"])
def test_gradients_past_32_bits(from_checkpoint):
    """2.2e9 elements, gates that forget within 600 rows: every gradient of the first rows, which have come the
    longest way, and of the last."""
    dev = cuda_or_skip()
    T, D, n, head = 540000, 4096, 700, 50
    if torch.cuda.get_device_properties(dev).total_memory < 60 << 30:
        pytest.skip("needs 45 GB")
    gen = torch.Generator(dev).manual_seed(240)
    x = torch.randn(1, T, D, dtype=torch.bfloat16, device=dev, generator=gen)
    g = torch.full((1, T, D), -1.5, dtype=torch.bfloat16, device=dev)
    g[:, :, ::3] = -0.75
    s0 = torch.randn(1, D, device=dev, generator=gen)
    cols = torch.cat([torch.arange(0, 20), torch.arange(D - 20, D)]).to(dev)
    cut = lambda t, rows: t[:, rows][..., cols].cpu()
    first, last = slice(0, n), slice(T - n, T)
    if from_checkpoint:
        ckpt = torch.empty(kda_scan_checkpoint_size(1, T, D), dtype=torch.uint8, device=dev)
        h, _ = kda_scan_fwd(x, g, s0, checkpoint=ckpt)
    else:
        h, _ = kda_scan_fwd(x, g, s0)
    # z as it is saved: the rows' h, or its codes with the scale of each row's block of 128 channels
    P, _, at = scan.layout(T, D)
    def z_of(rows):
        lo = rows.start
        if not from_checkpoint:
            before = cut(h, slice(max(lo - 1, 0), rows.stop - 1)).double()
            return (torch.cat([s0[:, cols].cpu()[None].double(), before], 1) if lo == 0 else before).numpy()
        c = ckpt[at[1]:at[1] + T * P].view(T, P)[rows][:, cols].cpu().view(torch.float8_e4m3fn).double()
        k = ckpt[at[3]:at[3] + (D // 128) * T].view(D // 128, T)[:, rows][cols.cpu() // 128].cpu().double().t() - 127
        return (c * torch.exp2(k))[None].numpy()
    z = [z_of(first), z_of(last)]
    dh = x  # any values do
    got = kda_scan_backward_ckpt(ckpt, dh) if from_checkpoint else kda_scan_backward(None, g, h, dh, s0)
    lam = np.broadcast_to(np.where(cols.cpu().numpy() % 3 == 0, -0.75, -1.5), (1, n, 40))
    for k, rows, keep in ((0, first, slice(0, head)), (1, last, slice(0, n))):
        ref = scan.backward(lam, z[k], cut(dh, rows))
        _, E = scan.scan_abs(np.exp(lam), cut(dh, rows).double().numpy(), firsts(1, n, None, True), reverse=True)
        E = 12 * U * E
        near("dx", cut(got["dx"], rows)[:, keep], ref["dx"][:, keep], E[:, keep], torch.bfloat16)
        bound = np.exp(lam) * np.abs(z[k]) * E + 20 * U * np.abs(ref["dg"])
        near("dg", cut(got["dg"], rows)[:, keep], ref["dg"][:, keep], bound[:, keep], torch.bfloat16)
        if k == 0:
            a = np.exp(lam[0, 0])
            near("dS0", got["dS0"][:, cols], ref["dS0"], a * E[:, 0] + 8 * U * a * np.abs(ref["d"][:, 0]))
