"""What is measured of the short causal convolution and the selective state space scan.

Six calls: each operator for prompts (packed sequences), for training (its
gradients) and for serving (one token per request against resident states).

  convolution  p_t = bias + sum_j w_j x_{t-W+1+j},  y_t = p_t or silu(p_t)
  scan         d_t = softplus(dt_t + dt_bias)
               h_t[c,n] = exp(d_t[c] A[c,n]) h_{t-1}[c,n] + d_t[c] u_t[c] B_t[n]
               y_t[c] = (sum_n C_t[n] h_t[c,n] + D[c] u_t[c]) silu(z_t[c])

``run`` computes them in elementary torch operations where ``own`` is false and
through the package's entry points where it is true.
"""
import math

import numpy as np
import torch

own = False

DEVICE = torch.device("cuda", 0) if torch.cuda.is_available() else torch.device("cpu")

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # The convolution of q in front of a two-head layer's smallest prompt: latency.
        {"name": "conv_prompt_tiny", "op": "conv_fwd", "lens": "256", "channels": 256, "width": 4, "type": "bf16",
         "silu": True, "bias": False, "states": False},
        # A packed batch of mixed prompt lengths, q, k and v of 32 heads of 128 in one call, continued from states.
        {"name": "conv_prompt_mixed", "op": "conv_fwd", "lens": "2048,37,8192,130,3000,511,4096,250",
         "channels": 12288, "width": 4, "type": "bf16", "silu": True, "bias": False, "states": True},
        # Training step over eight packed sequences, q, k and v of 32 heads.
        {"name": "conv_train", "op": "conv_bwd", "lens": "1024,1024,1024,1024,1024,1024,1024,1024",
         "channels": 12288, "width": 4, "type": "bf16", "silu": True, "bias": False, "states": False},
        # Odd sizes in single precision: an odd channel count, empty and one-token sequences, three taps, a bias.
        {"name": "conv_train_odd", "op": "conv_bwd", "lens": "513,1,0,1300", "channels": 1001, "width": 3,
         "type": "f32", "silu": False, "bias": True, "states": True},
        # One token of each of 256 requests, q, k and v of 32 heads.
        {"name": "conv_token_256", "op": "conv_dec", "requests": 256, "channels": 12288, "width": 4, "type": "bf16",
         "silu": True, "bias": False},
        # One request alone: latency.
        {"name": "conv_token_1", "op": "conv_dec", "requests": 1, "channels": 4096, "width": 4, "type": "f16",
         "silu": True, "bias": True},
        # One prompt of 8192 tokens through a layer of 4096 channels with 16 states each, gated.
        {"name": "scan_prompt", "op": "scan_fwd", "lens": "8192", "channels": 4096, "state": 16, "groups": 1,
         "type": "bf16", "gate": True, "softplus": True, "states": False},
        # A long context with few channels (8 heads of 128), continued from a state.
        {"name": "scan_prompt_long", "op": "scan_fwd", "lens": "32768", "channels": 1024, "state": 16, "groups": 1,
         "type": "bf16", "gate": True, "softplus": True, "states": True},
        # Training step over eight packed sequences of 1024.
        {"name": "scan_train", "op": "scan_bwd", "lens": "1024,1024,1024,1024,1024,1024,1024,1024",
         "channels": 4096, "state": 16, "groups": 1, "type": "bf16", "gate": True, "softplus": True,
         "states": False},
        # Odd sizes in single precision: ragged lengths, a state size that is no power of two, two groups, no gate.
        {"name": "scan_train_odd", "op": "scan_bwd", "lens": "1,700,0,257", "channels": 514, "state": 24,
         "groups": 2, "type": "f32", "gate": False, "softplus": False, "states": True},
        # One token of each of 256 requests against states in a pool of 320 slots.
        {"name": "scan_token_256", "op": "scan_dec", "requests": 256, "pool": 320, "channels": 4096, "state": 16,
         "groups": 1, "type": "bf16", "gate": True, "softplus": True},
        # Three requests, wide states, single precision: latency.
        {"name": "scan_token_3", "op": "scan_dec", "requests": 3, "pool": 3, "channels": 1000, "state": 64,
         "groups": 1, "type": "f32", "gate": False, "softplus": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_lens(rng, total):
    """A ragged partition of about `total` tokens; now and then an empty or a one-token sequence."""
    parts = rng.randint(1, 6)
    weights = [rng.random() + 0.02 for _ in range(parts)]
    lens = [max(1, int(total * x / sum(weights))) for x in weights]
    if rng.random() < 0.4:
        lens.insert(rng.randint(0, len(lens)), rng.choice((0, 1)))
    return ",".join(str(x) for x in lens)


def draw(rng):
    op = rng.choice(("conv_fwd", "conv_bwd", "conv_dec", "scan_fwd", "scan_bwd", "scan_dec"))
    typ = rng.choice(("bf16", "bf16", "f16", "f32"))
    case = {"op": op, "type": typ}
    if op.startswith("conv"):
        case["channels"] = c = _log_int(rng, 16, 12288)
        if rng.random() < 0.6:
            case["channels"] = c = max(16, c // 16 * 16)
        case["width"] = rng.choice((2, 3, 4, 4))
        case["silu"] = rng.random() < 0.7
        case["bias"] = rng.random() < 0.5
        if op == "conv_dec":
            case["requests"] = _log_int(rng, 1, 256)
        else:
            most = (60_000_000 if op == "conv_bwd" else 120_000_000) // (c * BYTES[typ] // 2)
            case["lens"] = _draw_lens(rng, _log_int(rng, 1, max(2, min(20000, most))))
            case["states"] = rng.random() < 0.5
    else:
        case["state"] = n = rng.choice((16, 16, 16, 8, 32, 64, 128, 1, 5, 13, 24))
        case["groups"] = g = rng.choice((1, 1, 2, 4))
        c = _log_int(rng, 32, 4096)
        if rng.random() < 0.6:
            c = max(32, c // 32 * 32)
        case["channels"] = c = max(g, c // g * g)
        case["gate"] = rng.random() < 0.6
        case["softplus"] = rng.random() < 0.7
        if op == "scan_dec":
            case["requests"] = r = _log_int(rng, 1, max(2, min(256, 16_000_000 // (c * n))))
            case["pool"] = r + rng.choice((0, 1, r // 2))
        else:
            most = (150_000_000 if op == "scan_bwd" else 300_000_000) // (c * n)
            case["lens"] = _draw_lens(rng, _log_int(rng, 1, max(2, min(40000, most))))
            case["states"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------ inputs
class _Maker:
    def __init__(self, seed):
        self.g = torch.Generator(device=DEVICE)
        self.g.manual_seed(int(seed))

    def normal(self, *shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=self.g, device=DEVICE) * std).to(dtype)

    def uniform(self, lo, hi, *shape):
        return torch.rand(shape, generator=self.g, device=DEVICE) * (hi - lo) + lo


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _packing(s, lens):
    """What a program that packs sequences holds: the boundaries on the device."""
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    s["cu"] = torch.from_numpy(cu).to(DEVICE)
    s["tokens"] = int(cu[-1])
    s["seqs"] = len(lens)


def prepare(case, seed):
    m = _Maker(seed)
    t = TYPES[case["type"]]
    c = case["channels"]
    s = {"case": dict(case)}
    if case["op"].startswith("conv"):
        w = case["width"]
        s["weight"] = m.uniform(-1, 1, c, w) * w ** -0.5
        s["bias"] = m.uniform(-1, 1, c) * w ** -0.5 if case["bias"] else None
        if case["op"] == "conv_dec":
            r = case["requests"]
            s["x"] = m.normal(r, c, dtype=t)
            s["pool"] = m.normal(r, w - 1, c, dtype=t)
            s["index"] = torch.randperm(r, generator=m.g, device=DEVICE).to(torch.int32)
            return s
        _packing(s, _lens(case))
        s["x"] = m.normal(s["tokens"], c, dtype=t)
        s["init"] = m.normal(s["seqs"], w - 1, c, dtype=t) if case["states"] else None
        if case["op"] == "conv_bwd":
            s["dout"] = m.normal(s["tokens"], c, dtype=t)
            s["dfin"] = m.normal(s["seqs"], w - 1, c, dtype=t) if case["states"] else None
        return s
    n, g = case["state"], case["groups"]
    # decay rates -1, -2, ... -n as such layers start with, each moved a little as training moves them
    s["A"] = -torch.arange(1, n + 1, device=DEVICE, dtype=torch.float32) * torch.exp(m.normal(c, n, std=0.1))
    s["D"] = 1 + m.normal(c, std=0.1)
    # steps between 0.001 and 0.1, evenly over their logarithm
    step = torch.exp(m.uniform(math.log(1e-3), math.log(0.1), c))
    rows = case["requests"] if case["op"] == "scan_dec" else None
    if rows is None:
        _packing(s, _lens(case))
        rows = s["tokens"]
    s["u"] = torch.nn.functional.silu(m.normal(rows, c)).to(t)
    if case["softplus"]:
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))  # softplus of this is `step`
        s["dt"] = m.normal(rows, c, std=0.5, dtype=t)
    else:
        s["dt_bias"] = None
        s["dt"] = (step * torch.exp(m.normal(rows, c, std=0.5))).to(t)
    # B and C are columns of one projection's output, the gate is one half of another's
    bc = m.normal(rows, 2 * g * n, dtype=t)
    s["B"], s["C"] = (x.unflatten(1, (g, n)) for x in bc.split(g * n, dim=1))
    s["z"] = m.normal(rows, 2 * c, dtype=t)[:, c:] if case["gate"] else None
    if case["op"] == "scan_dec":
        s["pool"] = m.normal(case["pool"], c, n, std=0.3)
        s["index"] = torch.randperm(case["pool"], generator=m.g, device=DEVICE)[:rows].to(torch.int32)
        return s
    s["init"] = m.normal(s["seqs"], c, n, std=0.3) if case["states"] else None
    if case["op"] == "scan_bwd":
        s["dout"] = m.normal(rows, c, dtype=t)
        s["dfin"] = m.normal(s["seqs"], c, n) if case["states"] else None
    return s


# ------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    return (_own if own else _plain)[op](state)


def _act(case):
    return "silu" if case["silu"] else None


def _own_conv_fwd(s):
    import kimi_delta_attention_26_b200 as kda
    out, fin = kda.kda_conv_fwd(s["x"], s["weight"], s["bias"], _act(s["case"]), cu_seqlens=s["cu"],
                                initial_state=s["init"])
    return {"out": out, "final_state": fin}


def _own_conv_bwd(s):
    import kimi_delta_attention_26_b200 as kda
    return kda.kda_conv_bwd(s["x"], s["weight"], s["dout"], s["bias"], _act(s["case"]), cu_seqlens=s["cu"],
                            initial_state=s["init"], dfinal_state=s["dfin"])


def _own_conv_dec(s):
    import kimi_delta_attention_26_b200 as kda
    out = kda.kda_conv_decode(s["x"], s["weight"], s["pool"], s["bias"], _act(s["case"]), state_indices=s["index"])
    return {"out": out, "state": s["pool"]}


def _own_scan_fwd(s):
    import kimi_delta_attention_26_b200 as kda
    out, fin = kda.kda_ssm_fwd(s["u"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"],
                               s["case"]["softplus"], cu_seqlens=s["cu"], initial_state=s["init"])
    return {"out": out, "final_state": fin}


def _own_scan_bwd(s):
    import kimi_delta_attention_26_b200 as kda
    return kda.kda_ssm_bwd(s["u"], s["dt"], s["A"], s["B"], s["C"], s["dout"], s["D"], s["z"], s["dt_bias"],
                           s["case"]["softplus"], cu_seqlens=s["cu"], initial_state=s["init"],
                           dfinal_state=s["dfin"])


def _own_scan_dec(s):
    import kimi_delta_attention_26_b200 as kda
    out = kda.kda_ssm_decode(s["u"], s["dt"], s["A"], s["B"], s["C"], s["pool"], s["D"], s["z"], s["dt_bias"],
                             s["case"]["softplus"], state_indices=s["index"])
    return {"out": out, "state": s["pool"]}


_own = {"conv_fwd": _own_conv_fwd, "conv_bwd": _own_conv_bwd, "conv_dec": _own_conv_dec,
        "scan_fwd": _own_scan_fwd, "scan_bwd": _own_scan_bwd, "scan_dec": _own_scan_dec}


# -------------------------------------------------------- the plain forms
def _token_ranges(s):
    """Each token's sequence, and that sequence's first token and end."""
    cu = s["cu"].long()
    seq = torch.searchsorted(cu[1:], torch.arange(s["tokens"], device=cu.device), right=True)
    return seq, cu[seq], cu[seq + 1]


def _windows(s, w):
    """[T, W, C]: the W inputs that each output sees, from the initial state (or zero) before the sequence's start."""
    x = s["x"].float()
    seq, start, _ = _token_ranges(s)
    at = torch.arange(s["tokens"], device=x.device)[:, None] - (w - 1) + torch.arange(w, device=x.device)
    before = at < start[:, None]
    if s["init"] is None:
        old = torch.zeros((1, x.shape[1]), device=x.device)
        where = torch.zeros_like(at)
    else:
        old = s["init"].float().flatten(0, 1)
        where = seq[:, None] * (w - 1) + at - start[:, None] + (w - 1)
    return torch.cat([x, old])[torch.where(before, s["tokens"] + where, at)]


def _pre(win, s):
    p = (win * s["weight"].T).sum(1)
    return p if s["bias"] is None else p + s["bias"]


def _silu(x):
    return x / (1 + torch.exp(-x))


def _dsilu(x):
    g = 1 / (1 + torch.exp(-x))
    return g * (1 + x * (1 - g))


def _plain_conv_fwd(s):
    w = s["case"]["width"]
    p = _pre(_windows(s, w), s)
    out = _silu(p) if s["case"]["silu"] else p
    cu = s["cu"].long()
    at = cu[1:, None] - (w - 1) + torch.arange(w - 1, device=cu.device)
    back = at - cu[:-1, None]  # position within the sequence; negative: a row of the initial state
    rows = torch.cat([s["x"], s["x"].new_zeros(1, s["x"].shape[1])])[torch.where(back >= 0, at, s["tokens"])]
    if s["init"] is not None:
        seq = torch.arange(s["seqs"], device=cu.device)[:, None].expand_as(back)
        rows = torch.where((back < 0)[:, :, None], s["init"][seq, (back + w - 1).clamp(0, w - 2)], rows)
    return {"out": out.to(s["x"].dtype), "final_state": rows}


def _plain_conv_bwd(s):
    w = s["case"]["width"]
    win = _windows(s, w)
    dp = s["dout"].float()
    if s["case"]["silu"]:
        dp = dp * _dsilu(_pre(win, s))
    # positions that receive a gradient: every token, then the w - 1 rows before each sequence
    cu = s["cu"].long()
    seq, start, end = _token_ranges(s)
    taps = torch.arange(w, device=cu.device)
    pos = torch.cat([torch.arange(s["tokens"], device=cu.device), (cu[:-1, None] - (w - 1) + taps[:-1]).flatten()])
    seq = torch.cat([seq, torch.arange(s["seqs"], device=cu.device).repeat_interleave(w - 1)])
    start = torch.cat([start, cu[:-1].repeat_interleave(w - 1)])
    end = torch.cat([end, cu[1:].repeat_interleave(w - 1)])
    to = pos[:, None] + (w - 1) - taps  # the outputs that see this position, tap by tap
    seen = (to >= start[:, None]) & (to < end[:, None])
    zero = dp.new_zeros(1, dp.shape[1])
    dx = (torch.cat([dp, zero])[torch.where(seen, to, s["tokens"])] * s["weight"].T).sum(1)
    if s["dfin"] is not None:
        row = pos - (end - (w - 1))
        dfin = torch.cat([s["dfin"].float().flatten(0, 1), zero])
        dx = dx + dfin[torch.where(row >= 0, seq * (w - 1) + row, s["seqs"] * (w - 1))]
    t = s["x"].dtype
    return {"dx": dx[:s["tokens"]].to(t), "dweight": (dp[:, None] * win).sum(0).T.contiguous(),
            "dbias": dp.sum(0) if s["bias"] is not None else None,
            "dinitial_state": dx[s["tokens"]:].unflatten(0, (s["seqs"], w - 1)).to(t)}


def _plain_conv_dec(s):
    i = s["index"].long()
    win = torch.cat([s["pool"][i], s["x"][:, None]], dim=1)
    p = _pre(win.float(), s)
    s["pool"][i] = win[:, 1:]
    return {"out": (_silu(p) if s["case"]["silu"] else p).to(s["x"].dtype), "state": s["pool"]}


def _steps(s):
    """The steps d [T, C] and what they were computed from."""
    r = s["dt"].float()
    if s["dt_bias"] is not None:
        r = r + s["dt_bias"]
    return (torch.where(r > 20, r, torch.log1p(torch.exp(r.clamp(max=20)))) if s["case"]["softplus"] else r), r


def _per_channel(x, c):
    """[T, G, N] -> [T, C, N] in 32 bits: each group's row for its channels."""
    return x.float().repeat_interleave(c // x.shape[1], dim=1)


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t over the first dimension, in steps that double."""
    step = 1
    while step < a.shape[0]:
        b = torch.cat([b[:step], torch.addcmul(b[step:], a[step:], b[:-step])])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return b


def _states(s, d, decay, Bc):
    """All states [T, C, N] and, before them, each token's previous state."""
    c = d.shape[1]
    seq, start, _ = _token_ranges(s)
    first = torch.arange(s["tokens"], device=d.device) == start
    b = (d * s["u"].float())[:, :, None] * Bc
    if s["init"] is not None:
        b[first] += decay[first] * s["init"][seq[first]]
    h = _scan(torch.where(first[:, None, None], 0.0, decay), b)
    prev = torch.cat([h.new_zeros(1, c, h.shape[2]), h[:-1]])
    prev[first] = 0.0 if s["init"] is None else s["init"][seq[first]]
    return h, prev


def _last_states(s, h):
    cu = s["cu"].long()
    empty = (cu[1:] == cu[:-1])[:, None, None]
    none = torch.zeros((s["seqs"],) + s["A"].shape, device=h.device) if s["init"] is None else s["init"]
    return torch.where(empty, none, torch.cat([h, h.new_zeros(1, *s["A"].shape)])[cu[1:] - 1])


def _plain_scan_fwd(s):
    d, _ = _steps(s)
    c = d.shape[1]
    h, _ = _states(s, d, torch.exp(d[:, :, None] * s["A"]), _per_channel(s["B"], c))
    y = (h * _per_channel(s["C"], c)).sum(2) + s["D"] * s["u"].float()
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return {"out": y.to(s["u"].dtype), "final_state": _last_states(s, h)}


def _plain_scan_bwd(s):
    d, raw = _steps(s)
    c, t = d.shape[1], s["u"].dtype
    u = s["u"].float()
    decay, Bc, Cc = torch.exp(d[:, :, None] * s["A"]), _per_channel(s["B"], c), _per_channel(s["C"], c)
    h, prev = _states(s, d, decay, Bc)
    dy, dz = s["dout"].float(), None
    if s["z"] is not None:
        z = s["z"].float()
        dz = (dy * ((h * Cc).sum(2) + s["D"] * u) * _dsilu(z)).to(t)
        dy = dy * _silu(z)
    # the states' gradients, from the last token back
    seq, start, end = _token_ranges(s)
    at = torch.arange(s["tokens"], device=d.device)
    last, first = at == end - 1, at == start
    g = dy[:, :, None] * Cc
    if s["dfin"] is not None:
        g[last] += s["dfin"][seq[last]]
    after = torch.cat([decay[1:], torch.zeros_like(decay[:1])])
    after[last] = 0.0
    g = _scan(after.flip(0), g.flip(0)).flip(0)
    into = g * decay  # of the state before each token
    dexp = into * prev
    gB = (g * Bc).sum(2)
    dd = (dexp * s["A"]).sum(2) + gB * u
    if s["case"]["softplus"]:
        dd = dd / (1 + torch.exp(-raw))
    groups = s["B"].shape[1]
    dinit = torch.zeros((s["seqs"],) + s["A"].shape, device=d.device) if s["dfin"] is None else s["dfin"].clone()
    dinit[seq[first]] = into[first]
    return {"du": (gB * d + s["D"] * dy).to(t), "ddt": dd.to(t), "dA": (dexp * d[:, :, None]).sum(0),
            "dB": (g * (d * u)[:, :, None]).unflatten(1, (groups, -1)).sum(2).to(t),
            "dC": (h * dy[:, :, None]).unflatten(1, (groups, -1)).sum(2).to(t),
            "dD": (dy * u).sum(0), "dz": dz, "ddt_bias": dd.sum(0) if s["dt_bias"] is not None else None,
            "dinitial_state": dinit}


def _plain_scan_dec(s):
    d, _ = _steps(s)
    c, i = d.shape[1], s["index"].long()
    u = s["u"].float()
    h = torch.exp(d[:, :, None] * s["A"]) * s["pool"][i] + (d * u)[:, :, None] * _per_channel(s["B"], c)
    s["pool"][i] = h
    y = (h * _per_channel(s["C"], c)).sum(2) + s["D"] * u
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return {"out": y.to(s["u"].dtype), "state": s["pool"]}


_plain = {"conv_fwd": _plain_conv_fwd, "conv_bwd": _plain_conv_bwd, "conv_dec": _plain_conv_dec,
          "scan_fwd": _plain_scan_fwd, "scan_bwd": _plain_scan_bwd, "scan_dec": _plain_scan_dec}


# ------------------------------------------------------------------ work
def work(case):
    e, c, op = BYTES[case["type"]], case["channels"], case["op"]
    if op.startswith("conv"):
        w = case["width"]
        params = 4 * c * (w + (1 if case["bias"] else 0))
        per = 2 * w + (6 if case["silu"] else 0)
        if op == "conv_dec":
            r = case["requests"]
            return {"bytes": r * c * e * (2 + 2 * (w - 1)) + params, "flops": r * c * per}
        lens = _lens(case)
        rows, state = sum(lens), len(lens) * (w - 1) * c * e
        if op == "conv_fwd":
            return {"bytes": 2 * rows * c * e + params + state * (2 if case["states"] else 1), "flops": rows * c * per}
        return {"bytes": 3 * rows * c * e + 2 * params + state * (3 if case["states"] else 1),
                "flops": rows * c * (3 * per)}
    n, g = case["state"], case["groups"]
    params = 4 * (c * n + c + (c if case["softplus"] else 0))
    row = e * (2 * c + (c if case["gate"] else 0) + 2 * g * n)  # u, dt, the gate, B and C
    if op == "scan_dec":
        r = case["requests"]
        return {"bytes": r * (row + c * e + 8 * c * n) + params, "flops": 7 * r * c * n}
    lens = _lens(case)
    rows, state = sum(lens), 4 * len(lens) * c * n
    if op == "scan_fwd":
        return {"bytes": rows * (row + c * e) + params + state * (2 if case["states"] else 1),
                "flops": 7 * rows * c * n}
    return {"bytes": rows * (2 * row + c * e) + 2 * params + state * (3 if case["states"] else 1),
            "flops": 21 * rows * c * n}


# ------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if case["op"] == "conv_dec":
        return _exact_conv_dec(case, f)
    if case["op"] == "scan_dec":
        return _exact_scan_dec(case, f)
    bounds = f["cu"].tolist()
    spans = list(zip(bounds[:-1], bounds[1:]))
    if case["op"].startswith("conv"):
        return _exact_conv(case, f, spans)
    return _exact_scan(case, f, spans)


def _exact_conv_dec(case, f):
    w, slots = case["width"], f["index"].long()
    past = f["pool"].clone()
    p = f["x"] * f["weight"][:, w - 1]
    for j in range(w - 1):
        p = p + past[slots, j] * f["weight"][:, j]
    if f["bias"] is not None:
        p = p + f["bias"]
    moved = past.clone()
    for j in range(w - 2):
        moved[slots, j] = past[slots, j + 1]
    moved[slots, w - 2] = f["x"]
    return {"out": p * torch.sigmoid(p) if case["silu"] else p, "state": moved}


def _exact_conv(case, f, spans):
    w, c = case["width"], case["channels"]
    fwd = case["op"] == "conv_fwd"
    outs, lasts, dxs, dinits = [], [], [], []
    dw = torch.zeros(c, w, dtype=torch.float64, device=DEVICE)
    db = torch.zeros(c, dtype=torch.float64, device=DEVICE)
    for k, (lo, hi) in enumerate(spans):
        n = hi - lo
        old = torch.zeros(w - 1, c, dtype=torch.float64, device=DEVICE) if f["init"] is None else f["init"][k]
        line = torch.cat([old, f["x"][lo:hi]])
        p = torch.zeros(n, c, dtype=torch.float64, device=DEVICE) + (0 if f["bias"] is None else f["bias"])
        for j in range(w):
            p += f["weight"][:, j] * line[j:j + n]
        if fwd:
            outs.append(p * torch.sigmoid(p) if case["silu"] else p)
            lasts.append(line[n:])
            continue
        dp = f["dout"][lo:hi]
        if case["silu"]:
            sg = torch.sigmoid(p)
            dp = dp * (sg + p * sg * (1 - sg))
        dline = torch.zeros_like(line)
        for j in range(w):
            dline[j:j + n] += f["weight"][:, j] * dp
            dw[:, j] += (dp * line[j:j + n]).sum(0)
        db += dp.sum(0)
        if f["dfin"] is not None:
            dline[n:] += f["dfin"][k]
        dxs.append(dline[w - 1:])
        dinits.append(dline[:w - 1])
    if fwd:
        return {"out": torch.cat(outs), "final_state": torch.stack(lasts)}
    return {"dx": torch.cat(dxs), "dweight": dw, "dbias": db if f["bias"] is not None else None,
            "dinitial_state": torch.stack(dinits)}


def _exact_step(case, f):
    d = f["dt"] if f["dt_bias"] is None else f["dt"] + f["dt_bias"]
    return torch.nn.functional.softplus(d, threshold=1e9) if case["softplus"] else d


def _exact_scan_dec(case, f):
    d, slots = _exact_step(case, f), f["index"].long()
    wide = case["channels"] // case["groups"]
    B, C = (x.repeat_interleave(wide, dim=1) for x in (f["B"], f["C"]))
    h = f["pool"][slots] * torch.exp(torch.einsum("rc,cn->rcn", d, f["A"])) + torch.einsum("rc,rcn->rcn", d * f["u"], B)
    pool = f["pool"].clone()
    pool[slots] = h
    y = torch.einsum("rcn,rcn->rc", h, C) + f["D"] * f["u"]
    return {"out": y if f["z"] is None else y * f["z"] * torch.sigmoid(f["z"]), "state": pool}


def _exact_scan(case, f, spans):
    """Token by token, all sequences side by side at their own positions."""
    c, n, groups = case["channels"], case["state"], case["groups"]
    rows = spans[-1][1]
    long = max(hi - lo for lo, hi in spans)
    if rows * c * n > 600_000_000 or long > 40_000:
        return None
    wide = c // groups
    d = _exact_step(case, f)
    h = torch.zeros(len(spans), c, n, dtype=torch.float64, device=DEVICE) if f["init"] is None else f["init"].clone()
    back = case["op"] == "scan_bwd"
    y = torch.zeros(rows, c, dtype=torch.float64, device=DEVICE)
    kept = torch.zeros(rows, c, n, dtype=torch.float64, device=DEVICE) if back else None
    first = h.clone()
    alive = [[k for k, (lo, hi) in enumerate(spans) if hi - lo > i] for i in sorted({0, *(hi - lo for lo, hi in spans)})]
    edges = sorted({0, *(hi - lo for lo, hi in spans)})
    lows = torch.tensor([lo for lo, _ in spans], device=DEVICE)
    pieces = [(edges[i], edges[i + 1], torch.tensor(alive[i], device=DEVICE)) for i in range(len(edges) - 1)]

    def token(at, x):
        return x[at].repeat_interleave(wide, dim=1)

    for a, b, who in pieces:
        state, base = h[who], lows[who]
        for i in range(a, b):
            at = base + i
            state = state * torch.exp(d[at][:, :, None] * f["A"]) + (d[at] * f["u"][at])[:, :, None] * token(at, f["B"])
            y[at] = (state * token(at, f["C"])).sum(2)
            if back:
                kept[at] = state
        h[who] = state
    y = y + f["D"] * f["u"]
    if not back:
        return {"out": y if f["z"] is None else y * f["z"] * torch.sigmoid(f["z"]), "final_state": h}
    dy, dz = f["dout"], None
    if f["z"] is not None:
        sg = torch.sigmoid(f["z"])
        dz = dy * y * (sg + f["z"] * sg * (1 - sg))
        dy = dy * f["z"] * sg
    grad = torch.zeros_like(h) if f["dfin"] is None else f["dfin"].clone()
    dA = torch.zeros(len(spans), c, n, dtype=torch.float64, device=DEVICE)
    du, dd = f["D"] * dy, torch.zeros_like(dy)
    dB, dC = torch.zeros_like(f["B"]), torch.zeros_like(f["C"])
    for a, b, who in reversed(pieces):
        g, base, acc = grad[who], lows[who], dA[who]
        for i in range(b - 1, a - 1, -1):
            at = base + i
            g = g + dy[at][:, :, None] * token(at, f["C"])
            dC[at] = (kept[at] * dy[at][:, :, None]).unflatten(1, (groups, wide)).sum(2)
            dB[at] = (g * (d[at] * f["u"][at])[:, :, None]).unflatten(1, (groups, wide)).sum(2)
            through = (g * token(at, f["B"])).sum(2)
            du[at] += through * d[at]
            g = g * torch.exp(d[at][:, :, None] * f["A"])
            moved = g * (kept[at - 1] if i else first[who])
            dd[at] = (moved * f["A"]).sum(2) + through * f["u"][at]
            acc = acc + moved * d[at][:, :, None]
        grad[who], dA[who] = g, acc
    if case["softplus"]:
        dd = dd * torch.sigmoid(f["dt"] + f["dt_bias"])
    return {"du": du, "ddt": dd, "dA": dA.sum(0), "dB": dB, "dC": dC, "dD": (dy * f["u"]).sum(0), "dz": dz,
            "ddt_bias": dd.sum(0) if f["dt_bias"] is not None else None, "dinitial_state": grad}
