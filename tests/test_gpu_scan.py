"""Elementwise gated linear recurrence (kda_scan_*) against the fp64 oracle (oracle/scan.py).

Bounds, derived from the kernels' arithmetic with u = 2^-24 (fp32's half step):
alpha and 1 - alpha are within 6 u of their value (exp, expm1 one ulp = 2 u; the
sigmoid's 1 + e two u, its reciprocal one more, e times it 2 + 3 + 1), and each row
adds a product and a sum, one u each; where two stretches of rows are joined, a
product and a sum more.  So a term of h_t that has come through n rows is off by at
most (10 n + 8) u of its magnitude, and h_t by 12 u E_t, E_t the sum of the terms'
magnitudes, each counted once for every row it has come through (oracle.scan.scan_abs).
Gradients: the same for d_t, then at most three products more.  An output in bf16 is
off by half a step, 2^-8 of its value, on top.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_67_b200 import (kda_chunk_fwd_check, kda_scan_backward, kda_scan_backward_ckpt,
                                      kda_scan_checkpoint_size, kda_scan_fwd, kda_scan_step,
                                      kda_scan_workspace_size)
from gated_delta_rule_67_b200.binding import (KDA_OK, KDA_PREP_GATE_LOGSIGMOID, KDA_SCAN_INPUT_COMPLEMENT,
                                              KDA_SCAN_INPUT_PLAIN)
from oracle import scan
from tests.parity import cuda_or_skip

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ROUND = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}
TINY = 1e-37  # below fp32's normal numbers
MODES = [(False, False), (False, True), (True, False), (True, True)]
MODE_IDS = ["log-plain", "log-complement", "raw-plain", "raw-complement"]
DTYPES = [torch.float32, torch.bfloat16]
DTYPE_IDS = ["f32", "bf16"]


def how(raw, complement, cu=None, dev="cuda"):
    return dict(prep=KDA_PREP_GATE_LOGSIGMOID if raw else 0,
                input_gate=KDA_SCAN_INPUT_COMPLEMENT if complement else KDA_SCAN_INPUT_PLAIN,
                cu_seqlens=None if cu is None else torch.tensor(cu, dtype=torch.int32, device=dev))


def make(B, T, D, dtype, raw, seed, cu=None, strong=0.0):
    """x, g, s0, dh, dsT on the CPU: gates with a memory of a few to a thousand rows (``strong``: shifted by
    so much towards forgetting)."""
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen)
    r = n(B, T, D) + 1 + 6 * torch.rand(D, generator=gen) - strong
    g = r if raw else torch.nn.functional.logsigmoid(r)
    N = B if cu is None else len(cu) - 1
    return n(B, T, D).to(dtype), g.to(dtype), n(N, D), n(B, T, D).to(dtype), n(N, D)


def firsts(B, T, cu, last=False):
    out = np.zeros((B, T), bool)
    for _, b, lo, hi in scan.spans(B, T, cu):
        if hi > lo:
            out[b, hi - 1 if last else lo] = True
    return out


def near(name, got, ref, bound, dtype=torch.float32):
    got = got.detach().double().cpu().numpy()
    assert got.shape == ref.shape, name
    bound = bound * 1.01 + ROUND[dtype] * (np.abs(ref) + bound) + TINY
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (name, int(bad.sum()), tuple(np.argwhere(bad)[0]), got[bad][0], ref[bad][0], bound[bad][0])


def state_bound(rows, B, T, cu, pick_last, empty):
    """rows [B, T, D] at each sequence's last (first) row, by sequence; zero for empty sequences."""
    out = np.zeros((len(scan.spans(B, T, cu)), rows.shape[-1]))
    for i, b, lo, hi in scan.spans(B, T, cu):
        if hi > lo:
            out[i] = rows[b, hi - 1 if pick_last else lo]
    return out


def check_forward(x, g, s0, raw, complement, cu=None, got=None, **kw):
    dev = cuda_or_skip()
    B, T, D = x.shape
    if got is None:
        got = kda_scan_fwd(x.to(dev), g.to(dev), None if s0 is None else s0.to(dev), **how(raw, complement, cu), **kw)
    ref_h, ref_s, z = scan.forward(x, g, s0, raw=raw, complement=complement, cu=cu)
    lam = scan.log_gate(g, raw)
    u = -np.expm1(lam) * x.double().numpy() if complement else x.double().numpy()
    first = firsts(B, T, cu)
    init = np.zeros((len(scan.spans(B, T, cu)), D)) if s0 is None else s0.double().numpy()
    u = np.abs(u)
    for i, b, lo, hi in scan.spans(B, T, cu):
        if hi > lo:
            u[b, lo] += np.exp(lam[b, lo]) * np.abs(init[i])
    _, E = scan.scan_abs(np.exp(lam), u, first)
    near("h", got[0], ref_h, 12 * U * E, x.dtype)
    near("final_state", got[1], ref_s, 12 * U * state_bound(E, B, T, cu, True, None))
    return ref_h, z, E, lam


def check_backward(got, lam, z, dh, dsT, raw, complement, cu=None):
    B, T, D = dh.shape
    ref = scan.backward(lam, z, dh, dsT, raw=raw, complement=complement, cu=cu)
    alpha, beta, d = np.exp(lam), -np.expm1(lam), np.abs(ref["d"])
    src = np.abs(dh.double().numpy())
    for i, b, lo, hi in scan.spans(B, T, cu):
        if hi > lo and dsT is not None:
            src[b, hi - 1] += np.abs(dsT[i].double().numpy())
    a = np.roll(alpha, -1, axis=1)  # the factor into row t from row t + 1
    _, E = scan.scan_abs(a, src, firsts(B, T, cu, last=True), reverse=True)
    E = 12 * U * E
    bx, bg = (beta * E + 8 * U * np.abs(ref["dx"]), beta) if complement else (E, beta)
    near("dx", got["dx"], ref["dx"], bx, dh.dtype)
    eg = alpha * np.abs(z) * E * (beta if raw else 1) + 20 * U * np.abs(ref["dg"])
    if complement and not isinstance(z, np.ndarray):
        raise AssertionError
    near("dg", got["dg"], ref["dg"], eg, dh.dtype)
    first_bound = state_bound(alpha * E + 8 * U * alpha * d, B, T, cu, False, None)
    near("dS0", got["dS0"], ref["dS0"], first_bound)


SHAPES = [(1, 1, 1), (1, 1, 300), (2, 7, 130), (1, 64, 128), (3, 65, 64), (2, 63, 8), (1, 129, 257), (2, 300, 40),
          (1, 1100, 136)]


@pytest.mark.parametrize("raw,complement", MODES, ids=MODE_IDS)
@pytest.mark.parametrize("dtype", DTYPES, ids=DTYPE_IDS)
@pytest.mark.parametrize("B,T,D", SHAPES)
def test_forward(B, T, D, dtype, raw, complement):
    x, g, s0, _, _ = make(B, T, D, dtype, raw, 10 + T)
    check_forward(x, g, s0, raw, complement)


def test_forward_without_states():
    dev = cuda_or_skip()
    x, g, _, _, _ = make(2, 100, 72, torch.bfloat16, True, 20)
    check_forward(x, g, None, True, False)
    h, sT = kda_scan_fwd(x.to(dev), g.to(dev), output_final_state=False, prep=KDA_PREP_GATE_LOGSIGMOID)
    assert sT is None
    assert torch.equal(h, kda_scan_fwd(x.to(dev), g.to(dev), prep=KDA_PREP_GATE_LOGSIGMOID)[0])


# leading and trailing rows that no sequence owns, empty sequences at both ends and inside, single rows,
# boundaries on and off multiples of 64
PACKED = [(10, [0, 10]), (70, [3, 3, 4, 5, 66, 66, 66, 69, 69]), (200, [0, 64, 128, 129, 200]), (130, [5, 5, 5]),
          (700, [1, 2, 3, 320, 640, 650]), (40, list(range(0, 41)))]


@pytest.mark.parametrize("raw,complement", MODES, ids=MODE_IDS)
@pytest.mark.parametrize("dtype", DTYPES, ids=DTYPE_IDS)
@pytest.mark.parametrize("T,cu", PACKED, ids=["one", "ragged", "aligned", "all-empty", "long", "single-rows"])
@pytest.mark.parametrize("D", [136, 5])
def test_forward_packed(T, cu, D, dtype, raw, complement):
    x, g, s0, _, _ = make(1, T, D, dtype, raw, 30 + T, cu)
    check_forward(x, g, s0, raw, complement, cu)


@pytest.mark.parametrize("D", [136, 5])
def test_packed_sequences_do_not_touch(D):
    """NaN and infinities in one sequence and in rows that no sequence owns stay where they are; the rows
    outside get zeros in every output."""
    dev = cuda_or_skip()
    T, cu = 300, [2, 80, 80, 150, 290]
    for where in (1, 40, 100, 295):
        for bad in (float("nan"), float("inf")):
            x, g, s0, dh, dsT = make(1, T, D, torch.float32, False, 40, cu)
            clean = kda_scan_fwd(x.to(dev), g.to(dev), s0.to(dev), **how(False, True, cu))
            h0 = clean[0].cpu()
            grads = kda_scan_backward(x.to(dev), g.to(dev), h0.to(dev), dh.to(dev), s0.to(dev), dsT.to(dev),
                                      **how(False, True, cu))
            xb, gb, db = x.clone(), g.clone(), dh.clone()
            xb[0, where], gb[0, where], db[0, where] = bad, float("nan"), bad
            ckpt = torch.empty(kda_scan_checkpoint_size(1, T, D), dtype=torch.uint8, device=dev)
            h, sT = kda_scan_fwd(xb.to(dev), gb.to(dev), s0.to(dev), checkpoint=ckpt, **how(False, True, cu))
            bg = kda_scan_backward(xb.to(dev), gb.to(dev), h0.to(dev), db.to(dev), s0.to(dev), dsT.to(dev),
                                   **how(False, True, cu))
            cg = kda_scan_backward_ckpt(ckpt, db.to(dev), dsT.to(dev), **how(False, True, cu))
            torch.cuda.synchronize()
            seq = next((i for i in range(4) if cu[i] <= where < cu[i + 1]), None)
            for i in range(4):
                if i == seq:
                    continue
                s = slice(cu[i], cu[i + 1])
                assert torch.equal(h[0, s], clean[0][0, s]) and torch.equal(sT[i], clean[1][i])
                for n in ("dx", "dg"):
                    assert torch.equal(bg[n][0, s], grads[n][0, s]), (n, i)
                assert torch.equal(bg["dS0"][i], grads["dS0"][i])
                assert torch.isfinite(cg["dx"][0, s]).all() and torch.isfinite(cg["dg"][0, s]).all()
            if seq is not None:
                assert not torch.isfinite(h[0, where:cu[seq + 1]]).any()
            for out in (h, bg["dx"], bg["dg"], cg["dx"], cg["dg"]):
                assert not out[0, :2].any() and not out[0, 290:].any()
            lam, z, _, _ = scan.unpack(ckpt.cpu().numpy(), 1, T, D)
            assert not lam[0, :2].any() and not z[0, 290:].any()


@pytest.mark.parametrize("raw,complement", MODES, ids=MODE_IDS)
@pytest.mark.parametrize("dtype", DTYPES, ids=DTYPE_IDS)
@pytest.mark.parametrize("B,T,D", SHAPES)
def test_backward(B, T, D, dtype, raw, complement):
    dev = cuda_or_skip()
    x, g, s0, dh, dsT = make(B, T, D, dtype, raw, 50 + T)
    h = torch.from_numpy(scan.forward(x, g, s0, raw=raw, complement=complement)[0]).to(dtype)
    got = kda_scan_backward(x.to(dev) if complement else None, g.to(dev), h.to(dev), dh.to(dev), s0.to(dev),
                            dsT.to(dev), **how(raw, complement))
    z = scan.saved(x, h, s0, complement=complement)
    check_backward(got, scan.log_gate(g, raw), z, dh, dsT, raw, complement)


@pytest.mark.parametrize("raw,complement", MODES, ids=MODE_IDS)
@pytest.mark.parametrize("dtype", DTYPES, ids=DTYPE_IDS)
@pytest.mark.parametrize("T,cu", PACKED, ids=["one", "ragged", "aligned", "all-empty", "long", "single-rows"])
@pytest.mark.parametrize("D", [136, 5])
def test_backward_packed(T, cu, D, dtype, raw, complement):
    dev = cuda_or_skip()
    x, g, s0, dh, dsT = make(1, T, D, dtype, raw, 60 + T, cu)
    h = torch.from_numpy(scan.forward(x, g, s0, raw=raw, complement=complement, cu=cu)[0]).to(dtype)
    got = kda_scan_backward(x.to(dev), g.to(dev), h.to(dev), dh.to(dev), s0.to(dev), dsT.to(dev),
                            **how(raw, complement, cu))
    z = scan.saved(x, h, s0, complement=complement, cu=cu)
    check_backward(got, scan.log_gate(g, raw), z, dh, dsT, raw, complement, cu)


def test_backward_without_states():
    dev = cuda_or_skip()
    x, g, _, dh, _ = make(2, 150, 24, torch.float32, False, 70)
    h = torch.from_numpy(scan.forward(x, g)[0]).float()
    got = kda_scan_backward(None, g.to(dev), h.to(dev), dh.to(dev), **how(False, False))
    check_backward(got, scan.log_gate(g, False), scan.saved(x, h), dh, None, False, False)
    less = kda_scan_backward(None, g.to(dev), h.to(dev), dh.to(dev), want_initial_state_grad=False,
                             **how(False, False))
    assert less["dS0"] is None and torch.equal(less["dx"], got["dx"]) and torch.equal(less["dg"], got["dg"])


def check_checkpoint(buf, x, z, E, lam, raw, cu=None):
    """The bytes stand for lambda and z: the scale is the least that holds the block's largest magnitude
    (a magnitude within the bound of 448 * 2^k may fall to either side), each value is off by half a step of
    its code and by what the kernel's fp32 value may be off."""
    B, T, D = x.shape
    got = scan.unpack(buf.cpu().numpy(), B, T, D)
    own = np.zeros((B, T), bool)
    for _, b, lo, hi in scan.spans(B, T, cu):
        own[b, lo:hi] = True
    Ez = np.concatenate([E[:, :1], E[:, :-1]], axis=1)  # z_t is h_{t-1}
    Ez[firsts(B, T, cu)] = 0
    # lambda: exact, or min(g, 0) - log1p(exp(-|g|)): two ulp and a rounding; z: h's bound and a subtraction
    bounds = (5 * U * np.abs(lam) if raw else 0 * lam, 12 * U * Ez + 2 * U * np.abs(z))
    for name, v, ref, s, bound in (("lambda", got[0], lam, got[2], bounds[0]), ("z", got[1], z, got[3], bounds[1])):
        full = np.repeat(s, 128, axis=-1)[..., :D]
        for j in range(s.shape[-1]):
            c = slice(128 * j, min(D, 128 * j + 128))
            up = np.exp2(scan.scale_exponent(np.abs(ref[..., c]) + bound[..., c]).astype(float))
            down = np.exp2(scan.scale_exponent(np.maximum(np.abs(ref[..., c]) - bound[..., c], 0)).astype(float))
            assert (((s[..., j] == up) | (s[..., j] == down)) | ~own).all(), (name, j)
        half = np.maximum(np.abs(ref) * 2.0 ** -4, full * 2.0 ** -10)
        bad = ~(np.abs(v - ref) <= (half + bound) * 1.01) & own[..., None]
        assert not bad.any(), (name, int(bad.sum()), tuple(np.argwhere(bad)[0]), v[bad][0], ref[bad][0])
        assert not v[~own].any()
    return got[0], got[1]


CKPT_CASES = [(1, 1, 1, None), (2, 7, 130, None), (1, 64, 128, None), (2, 65, 40, None), (1, 300, 257, None),
              (1, 70, 136, [3, 3, 4, 5, 66, 66, 66, 69, 69]), (1, 200, 5, [0, 64, 128, 129, 200])]


@pytest.mark.parametrize("raw,complement", MODES, ids=MODE_IDS)
@pytest.mark.parametrize("dtype", DTYPES, ids=DTYPE_IDS)
@pytest.mark.parametrize("B,T,D,cu", CKPT_CASES, ids=[f"{c[1]}x{c[2]}" for c in CKPT_CASES])
def test_checkpoint_and_its_backward(B, T, D, cu, dtype, raw, complement):
    """The forward's outputs with a checkpoint are those without; the checkpoint's values; and the gradients
    are the formula's for those values."""
    dev = cuda_or_skip()
    x, g, s0, dh, dsT = make(B, T, D, dtype, raw, 80 + T, cu)
    ckpt = torch.empty(kda_scan_checkpoint_size(B, T, D), dtype=torch.uint8, device=dev).fill_(0xa5)
    plain = kda_scan_fwd(x.to(dev), g.to(dev), s0.to(dev), **how(raw, complement, cu))
    with_c = kda_scan_fwd(x.to(dev), g.to(dev), s0.to(dev), checkpoint=ckpt, **how(raw, complement, cu))
    assert torch.equal(plain[0], with_c[0]) and torch.equal(plain[1], with_c[1])
    _, z, E, lam = check_forward(x, g, s0, raw, complement, cu, got=with_c)
    lam8, z8 = check_checkpoint(ckpt, x, z, E, lam, raw, cu)
    got = kda_scan_backward_ckpt(ckpt, dh.to(dev), dsT.to(dev), **how(raw, complement, cu))
    check_backward(got, lam8, z8, dh, dsT, raw, complement, cu)


def test_checkpoint_extremes():
    """Blocks of zeros, subnormals, the largest values, and infinities and NaN, whose neighbours keep their
    values: one token, so that z is the initial state."""
    dev = cuda_or_skip()
    D = 128 * 5
    s0 = torch.randn(1, D, generator=torch.Generator().manual_seed(90))
    s0[:, :128] = 0
    s0[:, 128:256] *= 1e-40
    s0[:, 256:384] *= 1e38 / s0[:, 256:384].abs().max()
    s0[0, 384], s0[0, 400], s0[0, 511] = float("inf"), float("nan"), -float("inf")
    x, g = torch.zeros(1, 1, D), torch.full((1, 1, D), -0.5)
    ckpt = torch.empty(kda_scan_checkpoint_size(1, 1, D), dtype=torch.uint8, device=dev)
    kda_scan_fwd(x.to(dev), g.to(dev), s0.to(dev), checkpoint=ckpt)
    _, z, _, _ = scan.unpack(ckpt.cpu().numpy(), 1, 1, D)
    want = scan.quantise(s0[:, None].double().numpy())[0]
    np.testing.assert_array_equal(z, want)


@pytest.mark.parametrize("raw", [False, True])
def test_checkpoint_of_gates_that_forget_everything(raw):
    """Gates of minus infinity, of the types' lowest values and below -128 are held as -128: rows before them
    get no gradient through them, and nothing turns into NaN."""
    dev = cuda_or_skip()
    T, D = 150, 136
    x, g, s0, dh, dsT = make(1, T, D, torch.bfloat16, raw, 95)
    lowest = torch.finfo(torch.bfloat16).min
    g[0, 40], g[0, 80, ::2], g[0, 81, 1::2], g[0, 120, :5] = -float("inf"), lowest, -3e4, -200.0
    ckpt = torch.empty(kda_scan_checkpoint_size(1, T, D), dtype=torch.uint8, device=dev)
    kda_scan_fwd(x.to(dev), g.to(dev), s0.to(dev), checkpoint=ckpt, **how(raw, False))
    lam8, z8, _, _ = scan.unpack(ckpt.cpu().numpy(), 1, T, D)
    lam = np.maximum(scan.log_gate(g, raw), scan.LEAST)
    assert np.all(np.abs(lam8 - lam) <= np.maximum(np.abs(lam) * 2.0 ** -4, 2.0 ** -11) * 1.01)
    assert np.all(lam8[0, 40] == scan.LEAST)
    got = kda_scan_backward_ckpt(ckpt, dh.to(dev), dsT.to(dev), **how(raw, False))
    check_backward(got, lam8, z8, dh, dsT, raw, False)


def test_checkpoint_bytes_are_scale_times_code():
    """Values that e4m3 holds come back unchanged, on every power of two."""
    dev = cuda_or_skip()
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    s0 = torch.zeros(64, 128)
    for i in range(64):
        s0[i, :127] = codes * 2.0 ** (2 * i - 64) * (-1) ** i
    z64 = torch.zeros(64, 1, 128)
    ckpt = torch.empty(kda_scan_checkpoint_size(64, 1, 128), dtype=torch.uint8, device=dev)
    kda_scan_fwd(z64.to(dev), z64.to(dev), s0.to(dev), checkpoint=ckpt)
    _, z, _, zs = scan.unpack(ckpt.cpu().numpy(), 64, 1, 128)
    np.testing.assert_array_equal(z[:, 0], s0.double().numpy())
    np.testing.assert_array_equal(zs[:, 0, 0], 2.0 ** (2.0 * np.arange(64) - 64))


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("dtype", DTYPES, ids=DTYPE_IDS)
def test_extreme_gates(dtype, raw, complement):
    """Gates that keep everything, forget everything (-inf among them) and all between, in one sequence."""
    dev = cuda_or_skip()
    T, D = 200, 24
    x, g, s0, dh, dsT = make(1, T, D, dtype, raw, 100)
    special = [0.0, -0.0, -1e-30, -1e-4, -20.0, -80.0, -104.0, -3e4, -float("inf")]
    if raw:
        special += [30.0, 100.0, float("inf")]
    for i, v in enumerate(special):
        g[0, 10 + 13 * i, ::2] = v
        g[0, 11 + 13 * i, 1::2] = v
    ref_h, z, E, lam = check_forward(x, g, s0, raw, complement)
    lam = np.maximum(lam, -1e6)  # exp and expm1 of it are those of -inf; keeps 0 * inf out of the formula
    h = torch.from_numpy(ref_h).to(dtype)
    got = kda_scan_backward(x.to(dev), g.to(dev), h.to(dev), dh.to(dev), s0.to(dev), dsT.to(dev), **how(raw, complement))
    check_backward(got, lam, scan.saved(x, h, s0, complement=complement), dh, dsT, raw, complement)


@pytest.mark.parametrize("dtype", DTYPES, ids=DTYPE_IDS)
@pytest.mark.parametrize("B,T,D,cu", [(1, 9000, 24, None), (2, 4500, 136, None), (1, 6500, 19, [10, 3000, 3001, 6400])],
                         ids=["long", "two", "packed"])
def test_long_sequences(B, T, D, cu, dtype):
    """Many blocks of rows along one sequence, with memories of up to a thousand rows."""
    dev = cuda_or_skip()
    x, g, s0, dh, dsT = make(B, T, D, dtype, True, 110, cu)
    ref_h, z, E, lam = check_forward(x, g, s0, True, True, cu)
    h = torch.from_numpy(ref_h).to(dtype)
    got = kda_scan_backward(x.to(dev), g.to(dev), h.to(dev), dh.to(dev), s0.to(dev), dsT.to(dev), **how(True, True, cu))
    check_backward(got, lam, scan.saved(x, h, s0, complement=True, cu=cu), dh, dsT, True, True, cu)


@pytest.mark.parametrize("dtype", DTYPES, ids=DTYPE_IDS)
@pytest.mark.parametrize("B,T,D,cu", [(5, 500, 1000, None), (1, 2000, 2048, None), (3, 700, 640, None), (20, 600, 300, None),
                                      (1, 1500, 2600, [0, 1, 480, 700, 1400]), (1, 700, 2501, [5, 699])])
def test_many_chains(B, T, D, cu, dtype):
    """Enough sequences and channels that chains are walked by one block, two or four, over several blocks of
    rows each."""
    dev = cuda_or_skip()
    x, g, s0, dh, dsT = make(B, T, D, dtype, True, 115, cu)
    ckpt = torch.empty(kda_scan_checkpoint_size(B, T, D), dtype=torch.uint8, device=dev)
    got = kda_scan_fwd(x.to(dev), g.to(dev), s0.to(dev), checkpoint=ckpt, **how(True, True, cu))
    ref_h, z, E, lam = check_forward(x, g, s0, True, True, cu, got=got)
    h = torch.from_numpy(ref_h).to(dtype)
    got = kda_scan_backward(x.to(dev), g.to(dev), h.to(dev), dh.to(dev), s0.to(dev), dsT.to(dev), **how(True, True, cu))
    check_backward(got, lam, scan.saved(x, h, s0, complement=True, cu=cu), dh, dsT, True, True, cu)
    lam8, z8 = check_checkpoint(ckpt, x, z, E, lam, True, cu)
    check_backward(kda_scan_backward_ckpt(ckpt, dh.to(dev), dsT.to(dev), **how(True, True, cu)), lam8, z8, dh, dsT, True,
                   True, cu)


def test_offsets_past_32_bits():
    """2.2e9 elements: the last rows against the oracle over the rows before them (strong gates: what is
    older than 600 rows counts for less than 2^-600), forward, checkpoint and backward."""
    dev = cuda_or_skip()
    T, D, n = 540000, 4096, 700
    if torch.cuda.get_device_properties(dev).total_memory < 60 << 30:
        pytest.skip("needs 40 GB")
    x = torch.randn(1, T, D, dtype=torch.bfloat16, device=dev, generator=torch.Generator(dev).manual_seed(120))
    g = torch.full((1, T, D), -1.5, dtype=torch.bfloat16, device=dev)
    g[:, :, ::3] = -0.75
    ckpt = torch.empty(kda_scan_checkpoint_size(1, T, D), dtype=torch.uint8, device=dev)
    h, sT = kda_scan_fwd(x, g, checkpoint=ckpt)
    cols = torch.cat([torch.arange(0, 20), torch.arange(D - 20, D)])
    tail = lambda t: t[:, -n:][..., cols.to(dev)].cpu()
    ref_h, _, z = scan.forward(tail(x), tail(g))
    lam = scan.log_gate(tail(g), False)
    _, E = scan.scan_abs(np.exp(lam), tail(x).double().numpy(), firsts(1, n, None))
    near("h", tail(h)[:, 600:], ref_h[:, 600:], 12 * U * E[:, 600:], torch.bfloat16)
    near("final_state", sT[:, cols.to(dev)], ref_h[:, -1], 12 * U * E[:, -1])
    del h
    dh = x  # any values do
    for got in (kda_scan_backward_ckpt(ckpt, dh),):
        head = slice(0, 50)  # the rows whose gradients have come the longest way
        d = scan.backward(scan.log_gate(g[:, :700][..., cols.to(dev)].cpu(), False) * 0 + np.where(np.arange(D) % 3 == 0, -0.75, -1.5)[cols],
                          np.zeros((1, 700, 40)), dh[:, :700][..., cols.to(dev)].cpu())
        ref = d["dx"][:, head]
        a = np.exp(np.broadcast_to(np.where(np.arange(D) % 3 == 0, -0.75, -1.5)[cols], (1, 700, 40)))
        _, Ed = scan.scan_abs(a, dh[:, :700][..., cols.to(dev)].double().cpu().numpy(), firsts(1, 700, None, True), reverse=True)
        near("dx", got["dx"][:, head][..., cols.to(dev)], ref, 12 * U * Ed[:, head], torch.bfloat16)
        last = dh[:, -1][..., cols.to(dev)].double().cpu().numpy()
        near("dx", got["dx"][:, -1][..., cols.to(dev)], last, np.zeros_like(last), torch.bfloat16)


@pytest.mark.parametrize("raw,complement", MODES, ids=MODE_IDS)
@pytest.mark.parametrize("dtype", DTYPES, ids=DTYPE_IDS)
@pytest.mark.parametrize("N,D", [(1, 1), (3, 130), (8, 2048), (5, 1001)])
def test_step(N, D, dtype, raw, complement):
    dev = cuda_or_skip()
    x, g, s0, _, _ = make(N, 1, D, dtype, raw, 130 + N)
    kw = {k: v for k, v in how(raw, complement).items() if k != "cu_seqlens"}
    state, new = s0.to(dev), torch.empty(N, D, device=dev)
    h = kda_scan_step(x[:, 0].to(dev), g[:, 0].to(dev), state, out_state=new, **kw)
    check_forward(x, g, s0, raw, complement, got=(h[:, None], new))
    assert torch.equal(state.cpu(), s0)
    h2 = kda_scan_step(x[:, 0].to(dev), g[:, 0].to(dev), state, **kw)
    assert torch.equal(h2, h) and torch.equal(state, new)


@pytest.mark.parametrize("dtype", DTYPES, ids=DTYPE_IDS)
def test_prefill_then_decode_then_backward(dtype):
    """As they are used: a prompt in two calls (states passed on, in place), decoded further step by step,
    each row against the oracle of the whole; then the gradients of the prompt from its checkpoint, close to
    those of the activations as they were."""
    dev = cuda_or_skip()
    B, T, D, cut, steps = 2, 300, 72, 130, 20
    x, g, s0, dh, dsT = make(B, T + steps, D, dtype, True, 140)
    kw = how(True, True)
    xd, gd, state = x.to(dev), g.to(dev), s0.to(dev)
    h1, s1 = kda_scan_fwd(xd[:, :cut].contiguous(), gd[:, :cut].contiguous(), state, final_state=state, **kw)
    assert s1 is state
    h2, _ = kda_scan_fwd(xd[:, cut:T].contiguous(), gd[:, cut:T].contiguous(), state, final_state=state, **kw)
    rows = [h1, h2]
    for t in range(T, T + steps):
        rows.append(kda_scan_step(xd[:, t].contiguous(), gd[:, t].contiguous(), state, input_gate=kw["input_gate"],
                                  prep=kw["prep"])[:, None])
    check_forward(x, g, s0, True, True, got=(torch.cat(rows, 1), state))
    ckpt = torch.empty(kda_scan_checkpoint_size(B, T, D), dtype=torch.uint8, device=dev)
    xp, gp, dp = xd[:, :T].contiguous(), gd[:, :T].contiguous(), dh[:, :T].contiguous().to(dev)
    h, _ = kda_scan_fwd(xp, gp, s0.to(dev), checkpoint=ckpt, **kw)
    near_ = kda_scan_backward_ckpt(ckpt, dp, dsT.to(dev), **kw)
    full = kda_scan_backward(xp, gp, h, dp, s0.to(dev), dsT.to(dev), **kw)
    # each rate and z is off by at most 2^-4 (half a step of e4m3); a gradient of many terms by less
    for n in ("dx", "dg", "dS0"):
        a, b = near_[n].double(), full[n].double()
        assert float((a - b).norm() / b.norm()) < 2.0 ** -3, n


def _train(x, g, s0, dh, dsT, kw, ckpt, **ws):
    h, sT = kda_scan_fwd(x, g, s0, checkpoint=ckpt, **kw, **ws)
    a = kda_scan_backward(x, g, h, dh, s0, dsT, **kw, **ws)
    b = kda_scan_backward_ckpt(ckpt, dh, dsT, **kw, **ws)
    return [h, sT] + [d[n] for d in (a, b) for n in ("dx", "dg", "dS0")]


SAME = [(2, 700, 136, None), (1, 3000, 264, None), (1, 1500, 130, [3, 70, 70, 900, 1499]), (1, 9000, 96, None)]


@pytest.mark.parametrize("B,T,D,cu", SAME, ids=["two", "one", "packed", "few-chains"])
def test_same_bits_every_time(B, T, D, cu):
    dev = cuda_or_skip()
    v = [t.to(dev) for t in make(B, T, D, torch.bfloat16, True, 150, cu)]
    ckpt = torch.empty(kda_scan_checkpoint_size(B, T, D), dtype=torch.uint8, device=dev)
    ref = [t.clone() for t in _train(*v, how(True, True, cu), ckpt)]
    for _ in range(5):
        for a, b in zip(_train(*v, how(True, True, cu), ckpt), ref):
            assert torch.equal(a, b)


@pytest.mark.parametrize("B,T,D,cu", SAME, ids=["two", "one", "packed", "few-chains"])
def test_graph_replay_matches_eager(B, T, D, cu):
    """Captured once, replayed on new inputs (and new sequence boundaries), with an eager call of the same
    kind between the replays; a dirty workspace."""
    dev = cuda_or_skip()
    kw = how(True, True, cu)
    a, b = ([t.to(dev) for t in make(B, T, D, torch.bfloat16, True, s, cu)] for s in (160, 161))
    size = kda_scan_workspace_size(B, T, D, 0 if cu is None else len(cu) - 1)
    ws = torch.empty(max(size, 256), dtype=torch.uint8, device=dev).fill_(0x5a)
    buf = [t.clone() for t in a]
    c1, c2 = (torch.empty(kda_scan_checkpoint_size(B, T, D), dtype=torch.uint8, device=dev) for _ in range(2))
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        _train(*buf, kw, c1, workspace=ws)
    torch.cuda.current_stream(dev).wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _train(*buf, kw, c1, workspace=ws)
    for k, v in enumerate((a, b, a)):
        for dst, src in zip(buf, v):
            dst.copy_(src)
        if cu is not None:
            kw["cu_seqlens"].copy_(torch.tensor([c - k for c in cu], dtype=torch.int32))
        graph.replay()
        ref = _train(*v, kw, c2)
        torch.cuda.synchronize()
        for p, q in zip(out, ref):
            assert torch.equal(p, q)
    assert size == 0 or kda_chunk_fwd_check(ws) == KDA_OK


@pytest.mark.parametrize("T,D", [(5000, 512), (20000, 96), (3000, 4096)], ids=["walked", "joined", "many"])
def test_two_streams_at_once(T, D):
    """Two calls in flight on two streams, each with its own workspace; and the ``stream`` argument."""
    dev = cuda_or_skip()
    kw = how(True, False)
    v = [[t.to(dev) for t in make(1, T, D, torch.bfloat16, True, s)] for s in (170, 171)]
    ref = [kda_scan_fwd(a[0], a[1], a[2], **kw) for a in v]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    for _ in range(10):
        got = [kda_scan_fwd(a[0], a[1], a[2], stream=s, **kw) for a, s in zip(v, streams)]
        torch.cuda.synchronize()
        for p, q in zip(got, ref):
            assert torch.equal(p[0], q[0]) and torch.equal(p[1], q[1])


@pytest.mark.parametrize("B,T,D,cu", [(1, 4000, 136, None), (3, 900, 2048, None), (1, 9000, 40, None),
                                      (1, 5000, 1000, [0, 30, 30, 2000, 2001, 4999])],
                         ids=["walked", "many", "joined", "packed"])
def test_state_in_place_over_many_tiles(B, T, D, cu):
    """final_state in initial_state's buffer gives the bits of two buffers."""
    dev = cuda_or_skip()
    x, g, s0, _, _ = (t.to(dev) for t in make(B, T, D, torch.bfloat16, True, 185, cu))
    for _ in range(3):
        h, sT = kda_scan_fwd(x, g, s0, **how(True, True, cu))
        state = s0.clone()
        h2, s2 = kda_scan_fwd(x, g, state, final_state=state, **how(True, True, cu))
        assert s2 is state and torch.equal(h, h2) and torch.equal(sT, state)


@pytest.mark.parametrize("cu", [[5, 3, 9, 200, 100, 150], [-7, 10, 400], [300, 200, 100], [2 ** 31 - 1, 0, -2 ** 31, 64]])
def test_meaningless_boundaries_stay_in_bounds(cu):
    """cu_seqlens that is not non-decreasing within [0, T]: whatever comes out, nothing outside the buffers is
    touched (the sentinels around them), and the next call is right."""
    dev = cuda_or_skip()
    T, D = 150, 72
    x, g, s0, dh, dsT = (t.to(dev) for t in make(1, T, D, torch.bfloat16, False, 190, cu))
    n, N = T * D, len(cu) - 1
    big = torch.full((n + 512,), 7.0, dtype=torch.bfloat16, device=dev)
    sbig = torch.full((N * D + 128,), 5.0, device=dev)
    kw = how(False, False, cu)
    kda_scan_fwd(x, g, s0, h=big[256:256 + n].view(1, T, D), final_state=sbig[64:64 + N * D].view(N, D), **kw)
    kda_scan_backward(None, g, x, dh, s0, dsT, **kw)
    torch.cuda.synchronize()
    assert (big[:256] == 7).all() and (big[256 + n:] == 7).all()
    assert (sbig[:64] == 5).all() and (sbig[64 + N * D:] == 5).all()
    x, g, s0, _, _ = make(1, 100, 40, torch.float32, False, 191)
    check_forward(x, g, s0, False, False)


def test_buffers_beside_the_outputs_stay():
    """Outputs given by the caller inside larger buffers: nothing around them is written."""
    dev = cuda_or_skip()
    for D in (136, 130, 7):
        T = 77
        x, g, s0, dh, dsT = (t.to(dev) for t in make(1, T, D, torch.bfloat16, True, 180))
        n = T * D
        big = torch.full((n + 256,), 7.0, dtype=torch.bfloat16, device=dev)
        off = 128
        h = big[off:off + n].view(1, T, D)
        size = kda_scan_checkpoint_size(1, T, D)
        cbig = torch.full((size + 512,), 0x77, dtype=torch.uint8, device=dev)
        sbig = torch.full((D + 64,), 5.0, device=dev)
        kda_scan_fwd(x, g, s0, h=h, final_state=sbig[32:32 + D].view(1, D), checkpoint=cbig[256:256 + size],
                     prep=KDA_PREP_GATE_LOGSIGMOID)
        torch.cuda.synchronize()
        assert (big[:off] == 7).all() and (big[off + n:] == 7).all()
        assert (cbig[:256] == 0x77).all() and (cbig[256 + size:] == 0x77).all()
        assert (sbig[:32] == 5).all() and (sbig[32 + D:] == 5).all()
        check_forward(x.cpu(), g.cpu(), s0.cpu(), True, False, got=(h, sbig[32:32 + D].view(1, D)))


def test_no_rows():
    dev = cuda_or_skip()
    s0 = torch.randn(3, 16, device=dev)
    e = torch.empty(3, 0, 16, device=dev)
    h, sT = kda_scan_fwd(e, e, s0)
    assert h.shape == (3, 0, 16) and torch.equal(sT, s0)
    assert not kda_scan_fwd(e, e)[1].any()
    d = kda_scan_backward(e, e, e, e, s0, s0 + 1)
    assert torch.equal(d["dS0"], s0 + 1)
    cu = torch.zeros(4, dtype=torch.int32, device=dev)
    e1 = torch.empty(1, 0, 16, device=dev)
    assert torch.equal(kda_scan_fwd(e1, e1, s0, cu_seqlens=cu)[1], s0)
    assert torch.equal(kda_scan_backward(e1, e1, e1, e1, s0, s0, cu_seqlens=cu)["dS0"], s0)
    z = torch.empty(0, 5, 16, device=dev)
    assert kda_scan_fwd(z, z)[1].shape == (0, 16)
    n = torch.empty(0, 16, device=dev)
    assert kda_scan_step(n, n, torch.empty(0, 16, device=dev)).shape == (0, 16)
