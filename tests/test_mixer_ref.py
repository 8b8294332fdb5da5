"""The 64-bit references of the convolution and the scan against differences of
their own forward (CPU): a wrong formula there would hide one in a kernel."""
import os
import re

import numpy as np
import pytest
import torch

from tests import mixer_ref as R


def _differences(f, args, wrt, grad, eps=1e-6, probes=6):
    """Directional derivatives of sum(f) along random directions against <grad, direction>."""
    gen = torch.Generator().manual_seed(3)
    for _ in range(probes):
        v = torch.randn(args[wrt].shape, generator=gen, dtype=torch.float64)
        up, down = dict(args), dict(args)
        up[wrt], down[wrt] = args[wrt] + eps * v, args[wrt] - eps * v
        num = (f(up) - f(down)) / (2 * eps)
        # central differences: truncation ~eps^2 and cancellation ~1e-16 / eps of the sum's size
        assert abs(float(num - (grad * v).sum())) <= 1e-6 * (1 + float((grad * v).abs().sum())), wrt


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_gradients(silu, W):
    g = torch.Generator().manual_seed(W)
    rnd = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    lens, C = [5, 0, 1, 2, 7], 3
    a = {"x": rnd(15, C), "weight": rnd(C, W), "bias": rnd(C), "init": rnd(5, W - 1, C)}
    dout, dfin = rnd(15, C), rnd(5, W - 1, C)

    def loss(a):
        o, f = R.conv(a["x"], a["weight"], a["bias"], silu, lens, a["init"])
        return (o * dout).sum() + (f * dfin).sum()

    gr = R.conv_bwd(a["x"], a["weight"], a["bias"], silu, lens, a["init"], dout, dfin)
    for wrt, name in (("x", "dx"), ("weight", "dweight"), ("bias", "dbias"), ("init", "dinitial_state")):
        _differences(loss, a, wrt, gr[name])


@pytest.mark.parametrize("softplus,gate", [(True, True), (False, False)])
def test_scan_gradients(softplus, gate):
    g = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    lens, T, c, n, G = [4, 0, 1, 9], 14, 6, 3, 2
    a = {"u": rnd(T, c), "dt": rnd(T, c) * 0.5 + (0 if softplus else 1), "A": -rnd(c, n).abs(), "B": rnd(T, G, n),
         "C": rnd(T, G, n), "D": rnd(c), "z": rnd(T, c), "bias": rnd(c) * 0.2, "init": rnd(4, c, n)}
    dout, dfin = rnd(T, c), rnd(4, c, n)

    def loss(a):
        o, f, _, _ = R.ssm(a["u"], R.step(a["dt"], a["bias"], softplus), a["A"], a["B"], a["C"], a["D"],
                           a["z"] if gate else None, lens, a["init"])
        return (o * dout).sum() + (f * dfin).sum()

    gr = R.ssm_bwd(a["u"], a["dt"], a["A"], a["B"], a["C"], a["D"], a["z"] if gate else None, a["bias"], softplus, lens,
                   a["init"], dout, dfin)
    names = [("u", "du"), ("dt", "ddt"), ("A", "dA"), ("B", "dB"), ("C", "dC"), ("D", "dD"), ("bias", "ddt_bias"),
             ("init", "dinitial_state")] + ([("z", "dz")] if gate else [])
    for wrt, name in names:
        _differences(loss, a, wrt, gr[name])


def test_polynomials_of_the_scan():
    """The two polynomials in the scan's source, evaluated in fp32 with one rounding
    a step: 2^f on [-1/2, 1/2] and atanh(s) / s for the softplus, against 64 bits.
    The bounds are those that the source states, plus fp32's half steps (six
    and eight of 2^-24 at most, most of them far from the last one)."""
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kimi_delta_attention_26_b200",
                            "csrc", "kda_ssm.cuh")).read()
    body = src[src.index("float exp2_poly(float x)"):]
    body = body[:body.index("const float y")]
    first = re.search(r"fmaf\(f, ([-\d.e]+)f, ([-\d.e]+)f\)", body)
    c = [float(first.group(1)), float(first.group(2))] + [float(x) for x in re.findall(r"fmaf\(f, t, ([-\d.e]+)f\)", body)]
    assert len(c) == 7 and c[-1] == 1.0
    f = np.linspace(-0.5, 0.5, 100001).astype(np.float32)
    t = np.full_like(f, np.float32(c[0]))
    for k in c[1:]:  # a multiply-add rounds once: exact in 64 bits, then to fp32
        t = (t.astype(np.float64) * f + np.float64(np.float32(k))).astype(np.float32)
    err = t / np.exp2(f.astype(np.float64)) - 1
    assert np.abs(err).max() <= 1e-7 and abs(err.mean()) <= 2e-9
    exact = np.polyval(c, f.astype(np.float64)) / np.exp2(f.astype(np.float64)) - 1
    assert np.abs(exact).max() <= 3e-8  # the coefficients' own rounding to fp32 on top of 2e-9
    body = src[src.index("float step_of(float r"):]
    body = body[:body.index("return fmaf(2.f * s")]
    head = re.search(r"fmaf\(w, 1\.f / (\d+), 1\.f / (\d+)\)", body)
    c = [1 / int(head.group(1)), 1 / int(head.group(2))] + [1 / int(x) for x in re.findall(r"fmaf\(w, t, 1\.f / (\d+)\)", body)] + [1.0]
    assert c[1:] == [1 / 11, 1 / 9, 1 / 7, 1 / 5, 1 / 3, 1.0]
    e = np.linspace(1e-4, 1, 100001)
    s = e / (2 + e)
    assert np.abs(2 * s * np.polyval(c, s * s) / np.log1p(e) - 1).max() <= 2.0 ** -26
