"""The short convolution and the selective scan in 64 bits on the CPU, with the
magnitudes that the tests' tolerances are derived from.

Every result is a sum of products. Evaluated in fp32 along a path of at most k
steps, each product carries at most k roundings (a few for each step: the step
size, the decay's argument, the exponential, the multiply-add), so the error is
at most k * 2^-22 times the sum of the products' absolute values. That sum is
the same formula on absolute values (``magnitude=True`` below), and the result
is then rounded once to the output's type, by at most eps / 2 of itself.
"""
import torch

STEP = 2.0 ** -22


def tolerance(ref, mag, steps, dtype, under=1.0):
    """Elementwise bound on |result - ref| for an output of type `dtype`.
    `under`: what a decay below 2^-126 (the library flushes it to zero) can be
    multiplied by on its way into the result, over all terms."""
    err = (steps + 16) * STEP * mag + under * torch.finfo(torch.float32).tiny
    return err + torch.finfo(dtype).eps / 2 * (ref.abs() + err) + torch.finfo(dtype).tiny


def check(got, ref, mag, steps, label, under=1.0):
    assert got.shape == ref.shape, f"{label}: shape {tuple(got.shape)} against {tuple(ref.shape)}"
    err = (got.detach().double().cpu() - ref).abs()
    tol = tolerance(ref, mag, steps, got.dtype, under)
    bad = ~(err <= tol)  # a NaN is bad
    assert not bool(bad.any()), (f"{label}: {int(bad.sum())} of {bad.numel()} off, worst "
                                 f"{float((err / tol).nan_to_num(1e30).max()):.3g} times the tolerance")


def spans(lens):
    out, at = [], 0
    for n in lens:
        out.append((at, at + n))
        at += n
    return out


def _act(p, silu):
    return p * torch.sigmoid(p) if silu else p


def _dact(p, silu):
    if not silu:
        return torch.ones_like(p)
    s = torch.sigmoid(p)
    return s * (1 + p * (1 - s))


# ------------------------------------------------------------- convolution
def conv(x, weight, bias, silu, lens, init, magnitude=False):
    """x [T, C], weight [C, W], init [N, W - 1, C] or None -> out, final_state.
    With `magnitude`, x, weight, bias, init are absolute values and the
    activation (whose slope is below 1.1) is left out."""
    W = weight.shape[1]
    outs, fins = [], []
    for k, (a, b) in enumerate(spans(lens)):
        past = torch.zeros(W - 1, x.shape[1], dtype=x.dtype) if init is None else init[k]
        line = torch.cat([past, x[a:b]])
        p = sum(weight[:, j] * line[j:j + b - a] for j in range(W))
        p = p if bias is None else p + bias
        outs.append(1.1 * p if magnitude else _act(p, silu))
        fins.append(line[b - a:])
    return torch.cat(outs), torch.stack(fins)


def conv_bwd(x, weight, bias, silu, lens, init, dout, dfin, magnitude=False):
    """dict of dx, dweight, dbias, dinitial_state. With `magnitude`, every input is
    an absolute value and the activation's slope its bound; its slope's
    sensitivity to the fp32 error of p (at most 0.5 |p|) is in it too."""
    W, C = weight.shape[1], x.shape[1]
    dxs, dis = [], []
    dw, db = torch.zeros(C, W, dtype=x.dtype), torch.zeros(C, dtype=x.dtype)
    for k, (a, b) in enumerate(spans(lens)):
        past = torch.zeros(W - 1, C, dtype=x.dtype) if init is None else init[k]
        line = torch.cat([past, x[a:b]])
        p = sum(weight[:, j] * line[j:j + b - a] for j in range(W))
        p = p if bias is None else p + bias
        dp = dout[a:b] * (1.1 + 0.5 * p if magnitude else _dact(p, silu))
        dl = torch.zeros_like(line)
        for j in range(W):
            dl[j:j + b - a] += weight[:, j] * dp
            dw[:, j] += (dp * line[j:j + b - a]).sum(0)
        db += dp.sum(0)
        if dfin is not None:
            dl[b - a:] += dfin[k]
        dxs.append(dl[W - 1:])
        dis.append(dl[:W - 1])
    return {"dx": torch.cat(dxs), "dweight": dw, "dbias": db, "dinitial_state": torch.stack(dis)}


# -------------------------------------------------------------------- scan
def step(dt, dt_bias, softplus):
    r = dt if dt_bias is None else dt + dt_bias
    return torch.nn.functional.softplus(r, threshold=1e9) if softplus else r


def _wide(x, c):
    return x.repeat_interleave(c // x.shape[-2], dim=-2)


def ssm(u, d, A, B, C, D, z, lens, init, magnitude=False):
    """d: the steps [T, C]. -> out, final_state, all states [T, C, S], states before each token.
    With `magnitude`: u, B, C, D, init are absolute values; the gate's slope is bounded by |z| + 1."""
    T, c = u.shape
    h_all = torch.zeros(T, c, A.shape[1], dtype=u.dtype)
    prev = torch.zeros_like(h_all)
    fins = []
    Bw, Cw = _wide(B, c), _wide(C, c)
    dm = d.abs() if magnitude else d
    for k, (a, b) in enumerate(spans(lens)):
        h = torch.zeros(c, A.shape[1], dtype=u.dtype) if init is None else init[k]
        for t in range(a, b):
            prev[t] = h
            h = torch.exp(d[t, :, None] * A) * h + dm[t, :, None] * u[t, :, None] * Bw[t]
            h_all[t] = h
        fins.append(h)
    y = (Cw * h_all).sum(2)
    if D is not None:
        y = y + D * u
    if z is not None:
        y = y * (z.abs() if magnitude else z * torch.sigmoid(z))
    return y, torch.stack(fins), h_all, prev


def ssm_bwd(u, dt, A, B, C, D, z, dt_bias, softplus, lens, init, dout, dfin, magnitude=False):
    """The gradients by the formulas. With `magnitude`, on absolute values (A in its products only)."""
    T, c = u.shape
    d = step(dt, dt_bias, softplus)
    m = (lambda x: None if x is None else x.abs()) if magnitude else (lambda x: x)
    u, B, C, D, init, dout, dfin = (m(x) for x in (u, B, C, D, init, dout, dfin))
    Am = m(A)
    dm = m(d)
    y, _, h, prev = ssm(u, d, A, B, C, D, None, lens, init, magnitude)
    dy, dz = dout, None
    if z is not None:
        s = torch.sigmoid(z)
        dz = dout * y * (1.1 + 0.5 * z.abs() if magnitude else s * (1 + z * (1 - s)))
        dy = dout * (z.abs() if magnitude else z * s)
    Bw, Cw = _wide(B, c), _wide(C, c)
    G = B.shape[1]
    g_all, q_all = torch.zeros_like(h), torch.zeros_like(h)
    dinit = torch.zeros(len(lens), c, A.shape[1], dtype=u.dtype)
    for k, (a, b) in enumerate(spans(lens)):
        g = torch.zeros(c, A.shape[1], dtype=u.dtype) if dfin is None else dfin[k]
        for t in range(b - 1, a - 1, -1):
            g = g + dy[t, :, None] * Cw[t]
            g_all[t] = g
            g = g * torch.exp(d[t, :, None] * A)
            q_all[t] = g * prev[t]
        dinit[k] = g
    gb = (g_all * Bw).sum(2)
    dd = (q_all * Am).sum(2) + gb * u
    if softplus:
        dd = dd * torch.sigmoid(dt if dt_bias is None else dt + dt_bias)
    fold = lambda x: x.reshape(T, G, c // G, -1).sum(2)  # noqa: E731
    return {"du": gb * dm + (0 if D is None else D * dy), "ddt": dd, "dA": (q_all * dm[:, :, None]).sum(0),
            "dB": fold(g_all * (dm * u)[:, :, None]), "dC": fold(h * dy[:, :, None]), "dD": (dy * u).sum(0), "dz": dz,
            "ddt_bias": dd.sum(0), "dinitial_state": dinit}
