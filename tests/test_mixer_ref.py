"""The 64-bit references of the convolution and the scan against differences of
their own forward (CPU): a wrong formula there would hide one in a kernel."""
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
