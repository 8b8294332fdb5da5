"""GPU tests of the convolution and the scan at the ends of their ranges: offsets
beyond 32 bits, the largest numbers of channels, groups and sequences, tensors
of another stream, calls from several threads."""
import threading

import pytest
import torch

from tests import mixer_ref as R
from tests import test_conv_gpu as TC
from tests import test_ssm_gpu as TS

pytestmark = pytest.mark.gpu

kda = TS.kda
FAR = 1 << 26  # elements between tokens: 40 of them pass 2^31


def far_rows(t):
    """The rows of t, FAR elements apart."""
    v = torch.empty(t.shape[0] * FAR, dtype=t.dtype, device="cuda").view(t.shape[0], FAR)[:, :t[0].numel()]
    v = v.view(t.shape) if t.dim() == 2 else v.unflatten(1, t.shape[1:])
    v.copy_(t)
    return v


def test_conv_tokens_far_apart(kda):
    lens, C = [39, 1], 72
    d = TC.make(lens, C, 4, torch.bfloat16, seed=1)
    cu = TC.cu_of(lens)
    x, dout, out = (far_rows(d[k]) for k in ("x", "dout", "x"))
    a, b = kda.kda_conv_fwd(d["x"], d["weight"], d["bias"], "silu", cu, d["init"])
    _, f = kda.kda_conv_fwd(x, d["weight"], d["bias"], "silu", cu, d["init"], out=out)
    assert torch.equal(out, a) and torch.equal(f, b)
    g = kda.kda_conv_bwd(d["x"], d["weight"], d["dout"], d["bias"], "silu", cu, d["init"], d["dfin"])
    h = kda.kda_conv_bwd(x, d["weight"], dout, d["bias"], "silu", cu, d["init"], d["dfin"])
    assert all(torch.equal(g[k], h[k]) for k in g)
    s1, s2 = (torch.randn(40, 3, C, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).bfloat16()
              for _ in range(2))
    ref = kda.kda_conv_decode(d["x"], d["weight"], s1, d["bias"])
    kda.kda_conv_decode(x, d["weight"], s2, d["bias"], out=x)
    assert torch.equal(x, ref) and torch.equal(s1, s2)


def test_scan_tokens_far_apart(kda):
    lens = [39, 1]
    d = TS.make(lens, 36, 16, 2, torch.bfloat16, seed=2)
    cu = TS.cu_of(lens)
    e = dict(d)
    for k in ("u", "dt", "B", "C", "z", "dout"):
        e[k] = far_rows(d[k])
    a, b = TS.fwd(kda, d, cu, initial_state=d["init"])
    out = far_rows(d["u"])
    _, f = TS.fwd(kda, e, cu, initial_state=d["init"], out=out)
    assert torch.equal(out, a) and torch.equal(f, b)
    g, h = (TS.bwd(kda, x, cu, initial_state=d["init"], dfinal_state=d["dfin"]) for x in (d, e))
    assert all(torch.equal(g[k], h[k]) for k in g)
    r = slice(30, 40)
    s1, s2 = (torch.randn(10, 36, 16, device="cuda", generator=torch.Generator("cuda").manual_seed(2)) for _ in range(2))
    o1, o2 = (kda.kda_ssm_decode(x["u"][r], x["dt"][r], x["A"], x["B"][r], x["C"][r], s, x["D"], x["z"][r], x["bias"])
              for x, s in ((d, s1), (e, s2)))
    assert torch.equal(o1, o2) and torch.equal(s1, s2)


def test_slots_far_into_a_pool(kda):
    """Slots whose states lie beyond 2^31 elements."""
    C, P = 12288, 60000
    d = TC.make([2], C, 4, torch.bfloat16, state=False, seed=3)
    pool = torch.empty(P, 3, C, dtype=torch.bfloat16, device="cuda")
    s = torch.randn(2, 3, C, device="cuda").bfloat16()
    slots = [P - 1, P - 700]
    pool[slots] = s
    idx = torch.tensor(slots, dtype=torch.int32, device="cuda")
    out = kda.kda_conv_decode(d["x"], d["weight"], pool, d["bias"], state_indices=idx)
    assert torch.equal(out, kda.kda_conv_decode(d["x"], d["weight"], s, d["bias"])) and torch.equal(pool[slots], s)
    del pool
    c, n, P = 4096, 128, 4200
    d = TS.make([2], c, n, 1, torch.bfloat16, state=False, seed=4)
    pool = torch.empty(P, c, n, device="cuda")
    s = torch.randn(2, c, n, device="cuda")
    slots = [P - 1, P - 90]
    pool[slots] = s
    idx = torch.tensor(slots, dtype=torch.int32, device="cuda")
    args = d["u"], d["dt"], d["A"], d["B"], d["C"]
    out = kda.kda_ssm_decode(*args, pool, d["D"], d["z"], d["bias"], state_indices=idx)
    assert torch.equal(out, kda.kda_ssm_decode(*args, s, d["D"], d["z"], d["bias"])) and torch.equal(pool[slots], s)


def test_kept_states_and_sums_beyond_32_bits(kda):
    """The last sequence of a batch whose kept states (2^31.0 floats) and sums of dB
    and dC (2^31.0 each) pass 32-bit offsets, bitwise as alone."""
    lens, c, n = [65400, 136], 4096, 64
    g = torch.Generator("cuda").manual_seed(5)
    T = sum(lens)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    d = {"u": rnd(T, c), "dt": rnd(T, c), "B": rnd(T, 1, n), "C": rnd(T, 1, n), "dout": rnd(T, c), "z": None, "D": None,
         "bias": None, "softplus": True, "A": -torch.exp(torch.randn(c, n, generator=g, device="cuda"))}
    try:
        kda.set_time_split(1)
        gr = TS.bwd(kda, d, TS.cu_of(lens))
        r = slice(lens[0], T)
        one = TS.bwd(kda, d, rows=r)
    finally:
        kda.set_time_split(0)
    for k in ("du", "ddt", "dB", "dC"):
        assert torch.equal(gr[k][r], one[k]), k
    assert torch.equal(gr["dinitial_state"][1:], one["dinitial_state"])


def test_most_channels_and_groups(kda):
    lens, C = [4, 1], 1 << 20
    d = TC.make(lens, C, 2, torch.float32, seed=6)
    out, fin = kda.kda_conv_fwd(d["x"], d["weight"], d["bias"], "silu", TC.cu_of(lens), d["init"])
    args = [TC.dbl(d[k]) for k in ("x", "weight", "bias")]
    ref, rfin = R.conv(*args, True, lens, TC.dbl(d["init"]))
    mag, _ = R.conv(*[a.abs() for a in args], True, lens, TC.dbl(d["init"], True), magnitude=True)
    R.check(out, ref, mag, 2, "out")
    assert torch.equal(fin.double().cpu(), rfin)
    gr = kda.kda_conv_bwd(d["x"], d["weight"], d["dout"], d["bias"], "silu", TC.cu_of(lens), d["init"], d["dfin"])
    rg = R.conv_bwd(*args, True, lens, TC.dbl(d["init"]), TC.dbl(d["dout"]), TC.dbl(d["dfin"]))
    mg = R.conv_bwd(*[a.abs() for a in args], True, lens, TC.dbl(d["init"], True), TC.dbl(d["dout"], True),
                    TC.dbl(d["dfin"], True), magnitude=True)
    for k in rg:
        R.check(gr[k], rg[k], mg[k], 5, k)
    c = 1 << 17
    for G, n in ((c, 1), (1, 2)):
        TS.check_all(kda, TS.make([3, 1], c, n, G, torch.float32, seed=G), [3, 1])


def test_most_sequences(kda):
    """65535 sequences of one token or none."""
    N, c, n = 65535, 6, 4
    g = torch.Generator().manual_seed(7)
    lens = (torch.rand(N, generator=g) < 0.8).long()
    T = int(lens.sum())
    cu = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)]).int().cuda()
    full = lens.bool()
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    u, dt, B, C, dy, D = rnd(T, c), rnd(T, c), rnd(T, 1, n), rnd(T, 1, n), rnd(T, c), rnd(c)
    A, init, dfin = -torch.exp(rnd(c, n)), rnd(N, c, n), rnd(N, c, n)
    dev = [t.cuda() for t in (u, dt, A, B, C)]
    out, fin = kda.kda_ssm_fwd(*dev, D.cuda(), cu_seqlens=cu, initial_state=init.cuda())
    gr = kda.kda_ssm_bwd(*dev, dy.cuda(), D.cuda(), cu_seqlens=cu, initial_state=init.cuda(), dfinal_state=dfin.cuda())

    def ref(m):
        """The outputs in 64 bits; m: on absolute values."""
        a = lambda t: m(t.double())  # noqa: E731
        d = R.step(dt.double(), None, True)
        e = torch.exp(d[:, :, None] * A.double())
        rf, ri = a(init).clone(), a(dfin).clone()
        rf[full] = e * a(init)[full] + (d * a(u))[:, :, None] * a(B)
        y = (a(C) * rf[full]).sum(2) + a(D) * a(u)
        gg = a(dfin)[full] + a(dy)[:, :, None] * a(C)
        ri[full] = e * gg
        return y, rf, ri, d * (gg * a(B)).sum(2) + a(D) * a(dy)

    got = out, fin, gr["dinitial_state"], gr["du"]
    for name, x, r, m in zip(("out", "final_state", "dinitial_state", "du"), got, ref(lambda t: t), ref(torch.abs)):
        R.check(x, r, m, 2 + n, name)
    W = 4
    x, w, past = rnd(T, c), rnd(c, W), rnd(N, W - 1, c)
    o, f = kda.kda_conv_fwd(x.cuda(), w.cuda(), None, None, cu, past.cuda())
    line = torch.cat([past[full], x[:, None]], 1).double()  # [T, W, c]
    R.check(o, (line * w.double().T).sum(1), (line * w.double().T).abs().sum(1), W, "conv")
    rf = past.clone()
    rf[full] = torch.cat([past[full][:, 1:], x[:, None]], 1)
    assert torch.equal(f.cpu(), rf)


def test_tensors_of_another_stream(kda):
    """With `stream`, a call's tensors may be dropped at once: their memory is not
    handed out again before the call is done."""
    lens = [100, 28]
    dc, ds = TC.make(lens, 264, 4, torch.bfloat16, seed=8), TS.make(lens, 136, 16, 1, torch.bfloat16, seed=9)
    cu = TC.cu_of(lens)

    def call(c, s, cu, **kw):
        o, f = kda.kda_conv_fwd(c["x"], c["weight"], c["bias"], "silu", cu, c["init"], **kw)
        g = kda.kda_conv_bwd(c["x"], c["weight"], c["dout"], c["bias"], "silu", cu, c["init"], c["dfin"], **kw)
        y, h = TS.fwd(kda, s, cu, initial_state=s["init"], **kw)
        e = TS.bwd(kda, s, cu, initial_state=s["init"], dfinal_state=s["dfin"], **kw)
        return [o, f, y, h] + list(g.values()) + list(e.values())

    ref = call(dc, ds, cu)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        copy = lambda d: {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in d.items()}  # noqa: E731
        a, b, c = copy(dc), copy(ds), cu.clone()
        sizes = [v.shape for d in (a, b) for v in d.values() if isinstance(v, torch.Tensor)] + [c.shape]
        types = [v.dtype for d in (a, b) for v in d.values() if isinstance(v, torch.Tensor)] + [c.dtype]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = call(a, b, c, stream=side)
        del a, b, c
        junk = [torch.full(s, 99, dtype=t, device="cuda") for s, t in zip(sizes, types)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, ref))
        del junk


def test_calls_from_several_threads(kda):
    """Four threads with a stream each, calls that take scratch, some of them split."""
    ds = [TS.make([1100], 64, 16, 1, torch.bfloat16, seed=20 + i) for i in range(4)]
    cs = [TC.make([300, 20], 264, 4, torch.bfloat16, seed=20 + i) for i in range(4)]
    cu = TC.cu_of([300, 20])

    def call(i):
        d, c = ds[i], cs[i]
        o, f = TS.fwd(kda, d, initial_state=d["init"])
        g = TS.bwd(kda, d, initial_state=d["init"], dfinal_state=d["dfin"])
        h = kda.kda_conv_bwd(c["x"], c["weight"], c["dout"], c["bias"], "silu", cu, c["init"], c["dfin"])
        return [o, f] + list(g.values()) + list(h.values())

    ref = [call(i) for i in range(4)]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got = call(i)
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(x, y) for x, y in zip(got, ref[i])):
                        wrong.append(i)
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
