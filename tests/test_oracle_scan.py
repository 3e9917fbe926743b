"""Pins of the recurrence's oracle (oracle/scan.py): closed forms, central
differences, torch autograd through a plain loop, and the 8-bit format
against torch's own e4m3 conversion."""
import numpy as np
import pytest
import torch

from oracle import scan


def _case(B, T, D, raw, seed, cu=None):
    r = np.random.default_rng(seed)
    g = r.normal(2.0, 1.5, (B, T, D)) if raw else -np.exp(r.normal(-2.0, 1.0, (B, T, D)))
    n = B if cu is None else len(cu) - 1
    return r.normal(size=(B, T, D)), g, r.normal(size=(n, D)), r.normal(size=(B, T, D)), r.normal(size=(n, D))


def test_forward_constant_gate_closed_form():
    """Constant gate and input: h_t = a^t s0 + x (1 - a^t) / (1 - a); weighed by 1 - a: a^t s0 + x (1 - a^t)."""
    T, a = 9, 0.75
    x, g, s0 = np.full((1, T, 1), 3.0), np.full((1, T, 1), np.log(a)), np.array([[5.0]])
    k = a ** np.arange(1, T + 1)
    h, sT, _ = scan.forward(x, g, s0)
    np.testing.assert_allclose(h[0, :, 0], k * 5 + 3 * (1 - k) / (1 - a), rtol=1e-14)
    h, sT, z = scan.forward(x, g, s0, complement=True)
    np.testing.assert_allclose(h[0, :, 0], k * 5 + 3 * (1 - k), rtol=1e-14)
    assert sT[0, 0] == h[0, -1, 0] and z[0, 0, 0] == 2.0


def test_zero_log_gate_is_a_running_sum():
    x = np.arange(24.0).reshape(2, 4, 3)
    h, _, _ = scan.forward(x, np.zeros_like(x))
    np.testing.assert_array_equal(h, np.cumsum(x, axis=1))


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("cu", [None, [1, 4, 4, 9]])
def test_backward_by_differences(raw, complement, cu):
    B, T, D = (2, 6, 3) if cu is None else (1, 11, 3)
    x, g, s0, dh, dsT = _case(B, T, D, raw, 3, cu)
    how = dict(raw=raw, complement=complement, cu=cu)

    def loss(x, g, s0):
        h, sT, _ = scan.forward(x, g, s0, **how)
        return float(np.sum(h * dh) + np.sum(sT * dsT))

    h, _, z = scan.forward(x, g, s0, **how)
    np.testing.assert_allclose(scan.saved(x, h, s0, complement=complement, cu=cu), z, rtol=1e-14)
    got = scan.backward(scan.log_gate(g, raw), z, dh, dsT, **how)
    for name, at in (("dx", 0), ("dg", 1), ("dS0", 2)):
        args = [x, g, s0]
        for i in np.ndindex(args[at].shape):
            eps, v = 1e-6, []
            for sign in (1, -1):
                moved = [a.copy() for a in args]
                moved[at][i] += sign * eps
                v.append(loss(*moved))
            # differences are off by eps^2 f'''/6 ~ 1e-12 |f'''| and 1e-16 |loss| / eps ~ 1e-9
            assert abs(got[name][i] - (v[0] - v[1]) / (2 * eps)) < 1e-7, (name, i)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("complement", [False, True])
def test_backward_by_autograd(raw, complement):
    x, g, s0, dh, dsT = (torch.from_numpy(a).requires_grad_() for a in _case(2, 17, 4, raw, 5))
    lam = torch.nn.functional.logsigmoid(g) if raw else g
    c, total = s0, 0.0
    for t in range(17):
        c = lam[:, t].exp() * c + (1 - lam[:, t].exp() if complement else 1) * x[:, t]
        total = total + (c * dh[:, t]).sum()
    (total + (c * dsT).sum()).backward()
    _, _, z = scan.forward(x, g, s0, raw=raw, complement=complement)
    got = scan.backward(scan.log_gate(g, raw), z, dh, dsT, raw=raw, complement=complement)
    for name, leaf in (("dx", x), ("dg", g), ("dS0", s0)):
        np.testing.assert_allclose(got[name], leaf.grad.numpy(), rtol=1e-11, atol=1e-12)


def test_rounding_matches_torch_e4m3():
    """Every fp32 value near every e4m3 value, its neighbours and the midpoints between them."""
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    mids = (codes[1:] + codes[:-1]) / 2
    q = np.concatenate([codes, mids, np.nextafter(np.float32(mids), np.float32(0)), np.nextafter(np.float32(mids), np.float32(999))])
    q = np.float32(np.concatenate([q, -q]))
    want = torch.from_numpy(q).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(scan.round_e4m3(q), want)


@pytest.mark.parametrize("top,k", [(448.0, 0), (448.1, 1), (224.0, -1), (1.0, -8), (1.75, -8), (1.76, -7), (0.0, -126),
                                   (1e-45, -126), (3.4e38, 120)])
def test_scale_exponent(top, k):
    assert scan.scale_exponent(np.array([0.0, -top, np.inf, np.nan])) == k


def test_quantise_error_is_half_a_step():
    v = np.random.default_rng(1).normal(size=(5, 300)) * np.exp2(np.arange(300) / 20)
    q, s = scan.quantise(v)
    full = np.repeat(s, 128, axis=-1)[:, :300]
    assert np.all(np.abs(q - v) <= np.maximum(np.abs(v) * 2.0 ** -4, full * 2.0 ** -10))
    assert np.all(np.abs(q) <= 448 * full)


def test_layout_matches_the_library():
    from gated_delta_rule_67_b200 import binding
    from gated_delta_rule_67_b200.build import build
    build()
    for B, T, D in [(1, 1, 1), (3, 7, 130), (2, 64, 128), (1, 1000, 1001), (1, 0, 5)]:
        assert binding.kda_scan_checkpoint_size(B, T, D) == scan.layout(B * T, D)[2][-1]
