"""GPU tests of the selective scan (kda_ssm_fwd, kda_ssm_decode, kda_ssm_bwd)
against the 64-bit reference; see tests/mixer_ref.py for the tolerances."""
import pytest
import torch

from tests import mixer_ref as R

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kimi_delta_attention_26_b200 as m

    m.device_status(reset=True)
    yield m
    assert m.device_status(reset=True) == 0


def make(lens, c, n, G, dtype, softplus=True, gate=True, state=True, D=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    A = -(torch.arange(n) % 16 + 1.0) * torch.exp(0.2 * rnd(c, n))
    base = torch.exp(torch.empty(c).uniform_(-6.0, -1.0, generator=g))
    d = {"u": rnd(T, c).to(dtype), "A": A, "B": rnd(T, G, n).to(dtype), "C": rnd(T, G, n).to(dtype),
         "D": rnd(c) if D else None, "z": rnd(T, c).to(dtype) if gate else None,
         "init": rnd(N, c, n) if state else None, "dout": rnd(T, c).to(dtype), "dfin": rnd(N, c, n) if state else None}
    if softplus:
        d["dt"], d["bias"] = (0.7 * rnd(T, c)).to(dtype), base + torch.log(-torch.expm1(-base))
    else:
        d["dt"], d["bias"] = (base * torch.exp(0.5 * rnd(T, c))).to(dtype), None
    d = {k: None if v is None else v.cuda() for k, v in d.items()}
    d["softplus"] = softplus
    return d


def cu_of(lens):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")


def dbl(x, mag=False):
    return None if x is None else (x.double().cpu().abs() if mag else x.double().cpu())


def fwd(kda, d, cu=None, rows=slice(None), **kw):
    at = lambda k: None if d[k] is None else d[k][rows]  # noqa: E731
    return kda.kda_ssm_fwd(at("u"), at("dt"), d["A"], at("B"), at("C"), d["D"], at("z"), d["bias"], d["softplus"], cu,
                           **kw)


def bwd(kda, d, cu=None, rows=slice(None), **kw):
    at = lambda k: None if d[k] is None else d[k][rows]  # noqa: E731
    return kda.kda_ssm_bwd(at("u"), at("dt"), d["A"], at("B"), at("C"), at("dout"), d["D"], at("z"), d["bias"],
                           d["softplus"], cu, **kw)


def check_all(kda, d, lens, large_steps=False):
    """`large_steps`: decays reach below 2^-126. Then two more terms belong to
    the bound. (1) A decay that is flushed to zero takes its products with it,
    at most 2^-126 times their other factors, over at most T tokens; a product
    has at most one of each of the step, u, the state, its gradient, A, B and C.
    (2) exp's argument carries a relative 2^-23, an error of |argument| 2^-23 of
    the decay; along a path whose product is not flushed the arguments add up
    to at most 88 and the logarithm of its other factors (below 2^60), 130 in all."""
    more_steps, under = 0, 1.0
    if large_steps:
        one = lambda v: max(1.0, float(v.abs().max()))  # noqa: E731
        st = one(R.step(dbl(d["dt"]), dbl(d["bias"]), d["softplus"]))
        u, A, B, C = (one(d[k]) for k in ("u", "A", "B", "C"))
        T = sum(lens)
        h = T * st * u * B + one(d["init"])
        g = T * one(d["dout"]) * one(d["z"]) * C + one(d["dfin"])
        more_steps, under = 130, T * st * u * A * B * C * h * g
        assert under < 2.0 ** 60
    cu, T = cu_of(lens), sum(lens)
    out, fin = fwd(kda, d, cu, initial_state=d["init"])
    x = {k: dbl(v) for k, v in d.items() if isinstance(v, torch.Tensor) or v is None}
    step = R.step(x["dt"], x["bias"], d["softplus"])
    ref, rfin, _, _ = R.ssm(x["u"], step, x["A"], x["B"], x["C"], x["D"], x["z"], lens, x["init"])
    m = {k: None if v is None else v.abs() for k, v in x.items()}
    mag, mfin, _, _ = R.ssm(m["u"], step, x["A"], m["B"], m["C"], m["D"], m["z"], lens, m["init"], magnitude=True)
    R.check(out, ref, mag, max(lens) + x["A"].shape[1] + more_steps, "out", under)
    R.check(fin, rfin, mfin, max(lens) + more_steps, "final_state", under)
    gr = bwd(kda, d, cu, initial_state=d["init"], dfinal_state=d["dfin"])
    args = [x[k] for k in ("u", "dt", "A", "B", "C", "D", "z", "bias")]
    rest = [d["softplus"], lens, x["init"], x["dout"], x["dfin"]]
    rg = R.ssm_bwd(*args, *rest)
    mg = R.ssm_bwd(*args, *rest, magnitude=True)
    for k in rg:
        if gr[k] is None:
            assert {"dz": d["z"], "dD": d["D"], "ddt_bias": d["bias"]}[k] is None
            continue
        # sums over tokens (parameters) or channels (dB, dC) come on top of the recurrences' steps
        more = {"dA": T, "dD": T, "ddt_bias": T, "dB": x["u"].shape[1], "dC": x["u"].shape[1]}.get(k, 0)
        R.check(gr[k], rg[k], mg[k], 2 * max(lens) + x["A"].shape[1] + more + more_steps, k, under)


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("n", [1, 3, 5, 8, 16, 24, 64, 100, 128])
def test_scan_state_sizes(kda, n, typ):
    check_all(kda, make([19, 0, 1, 40], 37, n, 1, TYPES[typ], softplus=n % 2 == 0, gate=n != 5, state=n != 3,
                        D=n != 8, seed=n), [19, 0, 1, 40])


@pytest.mark.parametrize("lens", [[1], [15], [16], [17], [32, 33], [2] * 20, [0, 0, 130], [200, 1, 3]],
                         ids=lambda x: f"{len(x)}seq{sum(x)}")
@pytest.mark.parametrize("c,G", [(1, 1), (8, 8), (66, 2), (96, 3), (129, 1)])
def test_scan_lengths_and_groups(kda, lens, c, G):
    check_all(kda, make(lens, c, 16, G, torch.float32, seed=c + G), lens)


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("state", [True, False])
def test_scan_options(kda, softplus, gate, state):
    check_all(kda, make([70, 5], 40, 16, 2, torch.bfloat16, softplus, gate, state, D=gate != state, seed=9), [70, 5])


@pytest.mark.parametrize("typ", list(TYPES))
def test_scan_long(kda, typ):
    """A long sequence beside short ones, with slow decays (the steps' range holds 0.0025)."""
    lens = [1, 1500, 3]
    check_all(kda, make(lens, 48, 16, 1, TYPES[typ], seed=4), lens)


@pytest.mark.parametrize("n,G,typ", [(16, 1, "bf16"), (5, 3, "f32"), (128, 1, "f16"), (30, 5, "f32")])
@pytest.mark.parametrize("lens", [[128], [700], [64, 64, 64], [1, 0, 63, 200, 64, 0, 130, 0], [300, 5]],
                         ids=lambda x: f"{len(x)}seq{sum(x)}")
def test_scan_time_split(kda, lens, n, G, typ):
    """Ranges of 64 tokens side by side: sequences that end and start at, before
    and after the ranges' borders, sequences over several ranges, empty ones."""
    d = make(lens, 45, n, G, TYPES[typ], gate=n != 5, state=n != 30, seed=n)
    try:
        kda.set_time_split(2)
        check_all(kda, d, lens)
        if d["init"] is not None:
            cu, state = cu_of(lens), d["init"].clone()
            _, ref = fwd(kda, d, cu, initial_state=d["init"])
            _, fin = fwd(kda, d, cu, initial_state=state, final_state=state)
            assert fin is state and torch.equal(state, ref)
    finally:
        kda.set_time_split(0)


def test_scan_time_split_is_taken_by_itself(kda):
    """One long sequence with few channels: the split's result agrees with the
    reference, and is not bitwise the unsplit scan's (so it was taken)."""
    d = make([2100], 64, 16, 1, torch.float32, seed=41)
    check_all(kda, d, [2100])
    a, _ = fwd(kda, d, initial_state=d["init"])
    try:
        kda.set_time_split(1)
        b, _ = fwd(kda, d, initial_state=d["init"])
    finally:
        kda.set_time_split(0)
    assert not torch.equal(a, b)


def test_scan_time_split_padded_and_bad_boundaries(kda):
    d = make([200], 40, 16, 1, torch.bfloat16, state=False, seed=43)
    for k in ("u", "dt", "B", "C", "z"):
        d[k][153:] = float("nan")
    try:
        kda.set_time_split(2)
        out = torch.full((200, 40), 5.0, dtype=torch.bfloat16, device="cuda")
        _, fin = fwd(kda, d, cu_of([100, 53]), out=out)
        ref, rfin = fwd(kda, d, cu_of([100, 53]), rows=slice(0, 153))
        assert torch.equal(out[:153], ref) and bool((out[153:] == 5).all()) and torch.equal(fin, rfin)
        assert kda.device_status(reset=True) == 0
        for bad in ([0, 150, 20, 200], [0, 130, 299, 10 ** 9], [-5, 10, 140, 200], [70, 80, 90, 200]):
            fwd(kda, d, torch.tensor(bad, dtype=torch.int32, device="cuda"))
            assert kda.device_status(reset=True) == 1, bad
    finally:
        kda.set_time_split(0)


def test_gradients_time_split_is_taken_by_itself(kda):
    """The gradients' time split: within the reference's bounds, the same at each
    call, and not bitwise the unsplit gradients (so it was taken)."""
    lens = [900, 3]
    d = make(lens, 70, 16, 1, torch.float32, seed=44)
    check_all(kda, d, lens)
    call = lambda: bwd(kda, d, cu_of(lens), initial_state=d["init"], dfinal_state=d["dfin"])  # noqa: E731
    a, b = call(), call()
    try:
        kda.set_time_split(1)
        one = call()
    finally:
        kda.set_time_split(0)
    assert all(torch.equal(a[k], b[k]) for k in a)
    assert not torch.equal(a["dinitial_state"], one["dinitial_state"])


@pytest.mark.parametrize("typ", list(TYPES))
def test_gradients_time_split_slow_decays(kda, typ):
    """Gradients that come through many ranges: decays near one all along, a gradient
    at the very end and one from the final state only."""
    lens = [1000]
    d = make(lens, 40, 8, 1, TYPES[typ], seed=45)
    d["A"] = d["A"] * 1e-3
    d["dout"][:990] = 0
    try:
        kda.set_time_split(2)
        check_all(kda, d, lens)
        d["dout"].zero_()
        check_all(kda, d, lens)
    finally:
        kda.set_time_split(0)


@pytest.mark.parametrize("typ", ["bf16", "f32"])
def test_time_split_growing_states(kda, typ):
    """Rates above 0: a range's growth (e^64 to e^140) overflows fp32, but the tokens
    with inputs are the last 30 and those with output gradients the first 30, so no
    state and no gradient does. A product's exponents add up to at most 30 * 2.2 = 66,
    each with a relative 2^-23 (33 of the tolerance's steps, of which there are 640)."""
    d = make([640], 40, 8, 1, TYPES[typ], softplus=False, state=False, seed=48)
    g = torch.Generator().manual_seed(49)
    d["A"] = (0.5 + 0.5 * torch.rand(40, 8, generator=g)).cuda()
    d["dt"] = (2 + 0.2 * torch.rand(640, 40, generator=g)).to(TYPES[typ]).cuda()
    d["u"][:610], d["dout"][30:] = 0, 0
    try:
        kda.set_time_split(2)
        check_all(kda, d, [640])
    finally:
        kda.set_time_split(0)


def test_gradients_time_split_padded_and_bad_boundaries(kda):
    T = 200
    d = make([T], 40, 16, 2, torch.bfloat16, state=False, seed=46)
    for k in ("u", "dt", "B", "C", "z", "dout"):
        d[k][153:] = float("nan")
    try:
        kda.set_time_split(2)
        cu = cu_of([100, 0, 53])
        gr, rg = bwd(kda, d, cu), bwd(kda, d, cu, rows=slice(0, 153))
        for k in ("du", "ddt", "dz", "dB", "dC"):
            assert torch.equal(gr[k][:153], rg[k]) and not bool(gr[k][153:].any()), k
        for k in ("dA", "dD", "ddt_bias", "dinitial_state"):
            assert torch.equal(gr[k], rg[k]), k
        assert kda.device_status(reset=True) == 0
        for bad in ([0, 150, 20, 200], [0, 130, 299, 10 ** 9], [-5, 10, 140, 200], [70, 80, 90, 200]):
            bwd(kda, d, torch.tensor(bad, dtype=torch.int32, device="cuda"))
            assert kda.device_status(reset=True) == 1, bad
    finally:
        kda.set_time_split(0)


def test_gradients_time_split_graphs_and_streams(kda):
    """Two captured calls that split, replayed side by side and after new inputs, beside an eager one."""
    lens = [1100]
    ds = [make(lens, 64, 16, 1, torch.bfloat16, seed=47 + i) for i in range(3)]
    call = lambda d: bwd(kda, d, initial_state=d["init"], dfinal_state=d["dfin"])  # noqa: E731
    for d in ds:
        call(d)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs, outs = [], []
    for d, s in zip(ds, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(call(d))
        graphs.append(g)
    for turn in range(2):
        for d in ds[:2]:
            d["u"].copy_(torch.randn_like(d["u"]))
            d["dout"].mul_(0.5)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = call(ds[2])
        torch.cuda.synchronize()
        for d, o in zip(ds, outs + [eager]):
            ref = call(d)
            assert all(torch.equal(o[k], ref[k]) for k in ref)


def test_scan_many_channels(kda):
    lens = [60, 90]
    check_all(kda, make(lens, 1000, 16, 1, torch.bfloat16, seed=6), lens)


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("n", [4, 8, 16, 24])
def test_scan_many_blocks(kda, n, typ):
    """More blocks than SMs (the form with two blocks on an SM): several full tiles
    of every sequence, with the paired and wide loads of even, aligned rows."""
    lens = [100 + 7 * i % 40 for i in range(15)] + [0]
    d = make(lens, 384, n, 1, TYPES[typ], seed=70 + n)
    try:
        kda.set_time_split(1)
        check_all(kda, d, lens)
    finally:
        kda.set_time_split(0)


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("n,c", [(40, 40), (64, 40), (128, 20), (128, 640)])
def test_scan_many_states_aligned(kda, n, c, typ):
    """More than 32 states with even, aligned rows: full tiles in paired and wide loads."""
    lens = [140, 33, 64]
    check_all(kda, make(lens, c, n, 1, TYPES[typ], seed=n + c), lens)


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("n", [8, 16, 24, 64])
def test_scan_alone_as_packed(kda, n, typ):
    """Unsplit, a sequence gives the same bits alone and in a batch, whose blocks
    outnumber the SMs where its own do not."""
    lens = [130, 0, 47, 200] + [1] * 12
    d = make(lens, 384, n, 1, TYPES[typ], seed=80 + n)
    try:
        kda.set_time_split(1)
        cu = cu_of(lens)
        out, fin = fwd(kda, d, cu, initial_state=d["init"])
        gr = bwd(kda, d, cu, initial_state=d["init"], dfinal_state=d["dfin"])
        for k, (a, b) in enumerate(R.spans(lens)[:5]):
            r, one = slice(a, b), slice(k, k + 1)
            o, f = fwd(kda, d, rows=r, initial_state=d["init"][one])
            g = bwd(kda, d, rows=r, initial_state=d["init"][one], dfinal_state=d["dfin"][one])
            assert torch.equal(o, out[r]) and torch.equal(f, fin[one]), k
            for name in ("du", "ddt", "dz", "dB", "dC"):
                assert torch.equal(g[name], gr[name][r]), (k, name)
            assert torch.equal(g["dinitial_state"], gr["dinitial_state"][one]), k
    finally:
        kda.set_time_split(0)


def test_scan_extreme_steps(kda):
    """Steps so large that the state is forgotten at once, and so small that it
    stays; softplus far above and below its bend."""
    d = make([50], 32, 16, 1, torch.float32, seed=13)
    d["dt"][:, ::4] = 40.0
    d["dt"][:, 1::4] = -60.0
    d["dt"][:, 2::4] = 19.0
    check_all(kda, d, [50], large_steps=True)


@pytest.mark.parametrize("typ", list(TYPES))
def test_scan_masked_steps(kda, typ):
    """A step masked by the type's lowest value or by minus infinity before the
    softplus is 0: the token leaves the state as it is (whatever u, B and C hold,
    as long as they are finite) and gets no gradient through it; plus infinity
    forgets the state, NaN stays in its channel."""
    dtype = TYPES[typ]
    d = make([40], 24, 16, 1, dtype, seed=61)
    keep = [t for t in range(40) if t not in (5, 6, 20)]
    d["dt"][5], d["dt"][6], d["dt"][20] = torch.finfo(dtype).min, float("-inf"), torch.finfo(dtype).min
    out, fin = fwd(kda, d, initial_state=d["init"])
    e = {k: (v[keep].contiguous() if k in ("u", "dt", "B", "C", "z", "dout") else v) for k, v in d.items()}
    ref, rfin = fwd(kda, e, initial_state=d["init"])
    assert torch.equal(out[keep], ref) and torch.equal(fin, rfin)
    assert bool(torch.isfinite(out).all())
    gr = bwd(kda, d, initial_state=d["init"], dfinal_state=d["dfin"])
    for k, v in gr.items():
        assert bool(torch.isfinite(v).all()), k
    assert not bool(gr["ddt"][[5, 6, 20]].any())
    state = d["init"].clone()
    r = slice(6, 7)
    kda.kda_ssm_decode(d["u"][r], d["dt"][r], d["A"], d["B"][r], d["C"][r], state, d["D"], d["z"][r], d["bias"])
    assert torch.equal(state, d["init"])
    d["dt"][10, 3] = float("nan")
    out2, _ = fwd(kda, d, initial_state=d["init"])
    same = torch.ones_like(out, dtype=torch.bool)
    same[10:, 3] = False
    assert torch.equal(out2[same], out[same]) and bool(out2[10:, 3].isnan().all())


@pytest.mark.parametrize("n,G", [(16, 1), (5, 3), (128, 1)])
def test_scan_pieces_and_tokens(kda, n, G):
    """A prompt in two pieces and then token by token agrees with the whole
    prompt within the tolerance of the reference; the final state may be the
    initial state's tensor."""
    c, T = 39, 50
    d = make([T], c, n, G, torch.float32, seed=n)
    whole, last = fwd(kda, d, initial_state=d["init"])
    state = d["init"].clone()
    o1, s = fwd(kda, d, rows=slice(0, 1), initial_state=state, final_state=state)
    assert s is state
    o2, _ = fwd(kda, d, rows=slice(1, 40), initial_state=state, final_state=state)
    outs = [o1, o2]
    for t in range(40, T):
        r = slice(t, t + 1)
        outs.append(kda.kda_ssm_decode(d["u"][r], d["dt"][r], d["A"], d["B"][r], d["C"][r], state, d["D"], d["z"][r],
                                       d["bias"], d["softplus"]))
    x = {k: dbl(v) for k, v in d.items() if isinstance(v, torch.Tensor)}
    step = R.step(x["dt"], x["bias"], True)
    ref, rfin, _, _ = R.ssm(x["u"], step, x["A"], x["B"], x["C"], x["D"], x["z"], [T], x["init"])
    m = {k: v.abs() for k, v in x.items()}
    mag, mfin, _, _ = R.ssm(m["u"], step, x["A"], m["B"], m["C"], m["D"], m["z"], [T], m["init"], magnitude=True)
    R.check(torch.cat(outs), ref, mag, T + n, "pieces")
    R.check(state, rfin, mfin, T, "state")
    R.check(whole, ref, mag, T + n, "whole")


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("n", [1, 6, 16, 40, 128])
def test_scan_decode_batch(kda, n, typ):
    rows, c, G, P = 7, 90, 2, 9
    d = make([1] * rows, c, n, G, TYPES[typ], gate=n != 6, D=n != 16, seed=n)
    g = torch.Generator().manual_seed(n)
    pool = torch.randn(P, c, n, generator=g).cuda()
    before = pool.clone()
    slots = [8, 0, 3, 7, 1, 2, 5]
    idx = torch.tensor(slots, dtype=torch.int32, device="cuda")
    out = kda.kda_ssm_decode(d["u"], d["dt"], d["A"], d["B"], d["C"], pool, d["D"], d["z"], d["bias"], True, idx)
    x = {k: dbl(v) for k, v in d.items() if isinstance(v, torch.Tensor) or v is None}
    init = before[slots].double().cpu()
    step = R.step(x["dt"], x["bias"], True)
    ref, rfin, _, _ = R.ssm(x["u"], step, x["A"], x["B"], x["C"], x["D"], x["z"], [1] * rows, init)
    m = {k: None if v is None else v.abs() for k, v in x.items()}
    mag, mfin, _, _ = R.ssm(m["u"], step, x["A"], m["B"], m["C"], m["D"], m["z"], [1] * rows, init.abs(),
                            magnitude=True)
    R.check(out, ref, mag, n, "out")
    R.check(pool[slots], rfin, mfin, 2, "state")
    assert torch.equal(pool[[4, 6]], before[[4, 6]])
    assert kda.device_status(reset=True) == 0
    out2 = torch.full_like(out, 3.0)
    pool.copy_(before)
    idx[2], idx[5] = 9, -2
    kda.kda_ssm_decode(d["u"], d["dt"], d["A"], d["B"], d["C"], pool, d["D"], d["z"], d["bias"], True, idx, out=out2)
    assert kda.device_status(reset=True) == 4
    ok = [0, 1, 3, 4, 6]
    assert torch.equal(out2[ok], out[ok]) and bool((out2[[2, 5]] == 3).all())
    assert torch.equal(pool[[2, 3, 4, 6]], before[[2, 3, 4, 6]])


def test_scan_padded_batch(kda):
    """Tokens behind the last sequence: outputs left as they were (whatever the
    inputs hold there), gradients zero."""
    lens, T, c = [20, 0, 33], 90, 40
    d = make([T], c, 16, 2, torch.bfloat16, state=False, seed=3)
    for k in ("u", "dt", "B", "C", "z", "dout"):
        d[k][53:] = float("nan")
    cu = cu_of(lens)
    out = torch.full((T, c), 5.0, dtype=torch.bfloat16, device="cuda")
    _, fin = fwd(kda, d, cu, out=out)
    ref, rfin = fwd(kda, d, cu, rows=slice(0, 53))
    assert torch.equal(out[:53], ref) and bool((out[53:] == 5).all()) and torch.equal(fin, rfin)
    gr, rg = bwd(kda, d, cu), bwd(kda, d, cu, rows=slice(0, 53))
    for k in ("du", "ddt", "dz", "dB", "dC"):
        assert torch.equal(gr[k][:53], rg[k]) and not bool(gr[k][53:].any()), k
    for k in ("dA", "dD", "ddt_bias", "dinitial_state"):
        assert torch.equal(gr[k], rg[k]), k


def test_scan_empty(kda):
    d = make([4], 24, 16, 1, torch.float32, seed=4)
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    init = torch.randn(2, 24, 16, device="cuda")
    out, fin = fwd(kda, d, cu, rows=slice(0, 0), initial_state=init)
    assert out.shape == (0, 24) and torch.equal(fin, init)
    gr = bwd(kda, d, cu, rows=slice(0, 0), initial_state=init, dfinal_state=init)
    assert torch.equal(gr["dinitial_state"], init)
    assert not any(bool(gr[k].any()) for k in ("dA", "dD", "ddt_bias"))
    e = slice(0, 0)
    assert kda.kda_ssm_decode(d["u"][e], d["dt"][e], d["A"], d["B"][e], d["C"][e], init).shape == (0, 24)


def test_scan_strided_views(kda):
    """B and C as columns of one projection, u and z as halves of another, at any
    element offset; the output into a wider buffer."""
    lens, c, n, G = [31, 9], 64, 16, 2
    d = make(lens, c, n, G, torch.bfloat16, seed=5)
    cu = cu_of(lens)
    ref, rfin = fwd(kda, d, cu, initial_state=d["init"])
    rg = bwd(kda, d, cu, initial_state=d["init"], dfinal_state=d["dfin"])
    for pad in (0, 8, 3):
        e = dict(d)
        proj = torch.zeros(40, pad + 2 * G * n + 1, dtype=torch.bfloat16, device="cuda")
        proj[:, pad:pad + G * n], proj[:, pad + G * n:pad + 2 * G * n] = d["B"].flatten(1), d["C"].flatten(1)
        e["B"] = proj[:, pad:pad + G * n].unflatten(1, (G, n))
        e["C"] = proj[:, pad + G * n:pad + 2 * G * n].unflatten(1, (G, n))
        uz = torch.cat([torch.zeros(40, pad, dtype=torch.bfloat16, device="cuda"), d["u"], d["z"]], dim=1)
        e["u"], e["z"] = uz[:, pad:pad + c], uz[:, pad + c:]
        buf = torch.zeros(40, 2 * c + pad, dtype=torch.bfloat16, device="cuda")
        out, fin = fwd(kda, e, cu, initial_state=d["init"], out=buf[:, pad:pad + c])
        assert torch.equal(out, ref) and torch.equal(fin, rfin) and not bool(buf[:, pad + c:].any())
        gr = bwd(kda, e, cu, initial_state=d["init"], dfinal_state=d["dfin"])
        for k in rg:
            assert torch.equal(gr[k], rg[k]), k


def test_scan_states_and_parameters_at_any_address(kda):
    """States, A and the other parameters at 4-byte addresses: the bits of aligned ones."""
    lens, c, n = [30, 11], 40, 16
    d = make(lens, c, n, 1, torch.bfloat16, seed=51)
    cu = cu_of(lens)

    def off(t, fill=None):
        buf = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
        v = buf[1:].view(t.shape)
        v.copy_(t)
        return v

    e = dict(d)
    for k in ("A", "D", "bias", "init", "dfin"):
        e[k] = off(d[k])
    a = fwd(kda, d, cu, initial_state=d["init"])
    b = fwd(kda, e, cu, initial_state=e["init"], final_state=off(d["init"]))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    ga = bwd(kda, d, cu, initial_state=d["init"], dfinal_state=d["dfin"])
    gb = bwd(kda, e, cu, initial_state=e["init"], dfinal_state=e["dfin"])
    assert all(torch.equal(ga[k], gb[k]) for k in ga)
    r = slice(0, 2)
    args = lambda x: (x["u"][r], x["dt"][r], x["A"], x["B"][r], x["C"][r])  # noqa: E731
    s1, s2 = d["init"].clone(), off(d["init"])
    o1 = kda.kda_ssm_decode(*args(d), s1, d["D"], d["z"][r], d["bias"])
    o2 = kda.kda_ssm_decode(*args(e), s2, e["D"], e["z"][r], e["bias"])
    assert torch.equal(o1, o2) and torch.equal(s1, s2)


def test_scan_bad_boundaries_are_recorded(kda):
    d = make([60], 40, 16, 1, torch.bfloat16, state=False, seed=6)
    for bad in ([0, 50, 20, 60], [0, 30, 99, 10 ** 9], [-5, 10, 40, 60], [4, 10, 40, 60]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        fwd(kda, d, cu)
        assert kda.device_status(reset=True) == 1, bad
        bwd(kda, d, cu)
        assert kda.device_status(reset=True) == 1, bad


def test_scan_special_values_stay_in_their_channel(kda):
    d = make([40], 72, 16, 1, torch.float32, gate=False, seed=8)
    ref, _ = fwd(kda, d, initial_state=d["init"])
    d["u"] = d["u"].clone()
    d["u"][10, 7] = float("nan")
    out, _ = fwd(kda, d, initial_state=d["init"])
    same = torch.ones_like(ref, dtype=torch.bool)
    same[10:, 7] = False
    assert torch.equal(out[same], ref[same]) and bool(out[10:, 7].isnan().all())


def test_scan_repeats_bitwise_and_alone_as_packed(kda):
    """The same call twice gives the same bits."""
    lens = [130, 0, 47, 400]
    d = make(lens, 200, 16, 2, torch.bfloat16, seed=14)
    cu = cu_of(lens)
    a = fwd(kda, d, cu, initial_state=d["init"]) + tuple(bwd(kda, d, cu, initial_state=d["init"]).values())
    b = fwd(kda, d, cu, initial_state=d["init"]) + tuple(bwd(kda, d, cu, initial_state=d["init"]).values())
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_scan_graphs_and_streams(kda):
    lens = [100, 28]
    d = [make(lens, 136, 16, 1, torch.bfloat16, seed=s) for s in (11, 12)]
    cu = cu_of(lens)

    def step(e):
        o, f = fwd(kda, e, cu, initial_state=e["init"])
        return [o, f] + list(bwd(kda, e, cu, initial_state=e["init"], dfinal_state=e["dfin"]).values())

    eager = [step(e) for e in d]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for e in d:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(e))
        graphs.append(g)
    for _ in range(3):
        for g, o in zip(graphs, outs):
            for t in o:
                t.zero_()
            g.replay()
    torch.cuda.synchronize()
    for e, o in zip(eager, outs):
        assert all(torch.equal(a, b) for a, b in zip(e, o))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gr = bwd(kda, d[0], cu, initial_state=d[0]["init"], dfinal_state=d[0]["dfin"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(gr.values(), eager[0][2:]))


def test_layer_trained_and_served(kda):
    """Convolution and scan as a layer runs them: gradients of both through the
    chain against the 64-bit formulas, then the prompt continued by single tokens."""
    lens, c, n, W = [40, 17], 48, 16, 4
    d = make(lens, c, n, 1, torch.float32, seed=31)
    cu, T = cu_of(lens), sum(lens)
    g = torch.Generator().manual_seed(32)
    x, w, b = torch.randn(T, c, generator=g).cuda(), (torch.randn(c, W, generator=g) * 0.5).cuda(), torch.randn(c, generator=g).cuda()
    u, tail = kda.kda_conv_fwd(x, w, b, "silu", cu)
    d["u"] = u
    out, state = fwd(kda, d, cu)
    gr = bwd(kda, d, cu)
    cg = kda.kda_conv_bwd(x, w, gr["du"], b, "silu", cu)
    ru, _ = R.conv(dbl(x), dbl(w), dbl(b), True, lens, None)
    r = {k: dbl(v) for k, v in d.items() if isinstance(v, torch.Tensor)}
    args = [ru] + [r[k] for k in ("dt", "A", "B", "C", "D", "z", "bias")]
    rg = R.ssm_bwd(*args, True, lens, None, r["dout"], None)
    mg = R.ssm_bwd(*args, True, lens, None, r["dout"], None, magnitude=True)
    rc = R.conv_bwd(dbl(x), dbl(w), dbl(b), True, lens, None, rg["du"], None)
    mc = R.conv_bwd(dbl(x, True), dbl(w, True), dbl(b, True), True, lens, None, mg["du"], None, magnitude=True)
    for k in rc:
        R.check(cg[k], rc[k], mc[k], 3 * T, k)
    # the next token of both sequences
    g1 = torch.randn(2, c, generator=g).cuda()
    nxt = make([1, 1], c, n, 1, torch.float32, seed=33)
    u1 = kda.kda_conv_decode(g1, w, tail, b)
    o1 = kda.kda_ssm_decode(u1, nxt["dt"], d["A"], nxt["B"], nxt["C"], state, d["D"], nxt["z"], d["bias"])
    xs = torch.cat([x[:40], g1[:1], x[40:], g1[1:]])
    lens1 = [41, 18]
    e = {k: torch.cat([d[k][:40], nxt[k][:1], d[k][40:], nxt[k][1:]]) for k in ("dt", "B", "C", "z")}
    ru, _ = R.conv(dbl(xs), dbl(w), dbl(b), True, lens1, None)
    step = R.step(dbl(e["dt"]), r["bias"], True)
    ref, rfin, _, _ = R.ssm(ru, step, r["A"], dbl(e["B"]), dbl(e["C"]), r["D"], dbl(e["z"]), lens1, None)
    mu, _ = R.conv(dbl(xs, True), dbl(w, True), dbl(b, True), True, lens1, None, magnitude=True)
    mag, mfin, _, _ = R.ssm(mu, step, r["A"], dbl(e["B"], True), dbl(e["C"], True), r["D"].abs(), dbl(e["z"], True),
                            lens1, None, magnitude=True)
    R.check(o1, ref[[40, 58]], mag[[40, 58]], 2 * 41, "token")
    R.check(state, rfin, mfin, 2 * 41, "state")
