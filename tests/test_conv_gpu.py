"""GPU tests of the short convolution (kda_conv_fwd, kda_conv_decode,
kda_conv_bwd) against the 64-bit reference; see tests/mixer_ref.py for the
tolerances."""
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


def make(lens, C, W, dtype, bias=True, state=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    d = {"x": rnd(T, C).to(dtype), "weight": rnd(C, W) * W ** -0.5, "bias": rnd(C) if bias else None,
         "init": rnd(N, W - 1, C).to(dtype) if state else None, "dout": rnd(T, C).to(dtype),
         "dfin": rnd(N, W - 1, C).to(dtype) if state else None}
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def cu_of(lens):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")


def dbl(x, mag=False):
    return None if x is None else (x.double().cpu().abs() if mag else x.double().cpu())


LENS = [[1], [37], [3, 0, 1, 2, 130, 0, 64, 1], [2] * 40, [700, 5]]


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("C", [1, 72, 333])
@pytest.mark.parametrize("lens", LENS, ids=lambda x: f"{len(x)}seq{sum(x)}")
def test_conv_forward_and_gradients(kda, lens, C, typ, W, silu):
    dtype, opt = TYPES[typ], (C + W) % 2 == 0
    d = make(lens, C, W, dtype, bias=opt or silu, state=opt or not silu, seed=C + W)
    act = "silu" if silu else None
    cu = cu_of(lens)
    out, fin = kda.kda_conv_fwd(d["x"], d["weight"], d["bias"], act, cu, d["init"])
    gr = kda.kda_conv_bwd(d["x"], d["weight"], d["dout"], d["bias"], act, cu, d["init"], d["dfin"])
    a = [dbl(d[k]) for k in ("x", "weight", "bias")]
    m = [dbl(d[k], True) for k in ("x", "weight", "bias")]
    ref, rfin = R.conv(*a, silu, lens, dbl(d["init"]))
    mag, _ = R.conv(*m, silu, lens, dbl(d["init"], True), magnitude=True)
    R.check(out, ref, mag, W, "out")
    assert torch.equal(fin.double().cpu(), rfin)
    rg = R.conv_bwd(*a, silu, lens, dbl(d["init"]), dbl(d["dout"]), dbl(d["dfin"]))
    mg = R.conv_bwd(*m, silu, lens, dbl(d["init"], True), dbl(d["dout"], True), dbl(d["dfin"], True), magnitude=True)
    assert (gr["dbias"] is None) == (d["bias"] is None)
    for k in rg:
        if gr[k] is not None:
            R.check(gr[k], rg[k], mg[k], sum(lens) if k in ("dweight", "dbias") else 2 * W, k)


@pytest.mark.parametrize("typ", list(TYPES))
def test_conv_large_packed(kda, typ):
    """Many tokens and channels: several runs of tokens per sequence and several sequences per run."""
    lens, C, W = [1500, 3, 0, 777, 1, 1, 2049], 1096, 4
    d = make(lens, C, W, TYPES[typ], seed=7)
    cu = cu_of(lens)
    out, fin = kda.kda_conv_fwd(d["x"], d["weight"], d["bias"], "silu", cu, d["init"])
    gr = kda.kda_conv_bwd(d["x"], d["weight"], d["dout"], d["bias"], "silu", cu, d["init"], d["dfin"])
    a = [dbl(d[k]) for k in ("x", "weight", "bias")]
    m = [dbl(d[k], True) for k in ("x", "weight", "bias")]
    ref, rfin = R.conv(*a, True, lens, dbl(d["init"]))
    mag, _ = R.conv(*m, True, lens, dbl(d["init"], True), magnitude=True)
    R.check(out, ref, mag, W, "out")
    assert torch.equal(fin.double().cpu(), rfin)
    rg = R.conv_bwd(*a, True, lens, dbl(d["init"]), dbl(d["dout"]), dbl(d["dfin"]))
    mg = R.conv_bwd(*m, True, lens, dbl(d["init"], True), dbl(d["dout"], True), dbl(d["dfin"], True), magnitude=True)
    for k in rg:
        R.check(gr[k], rg[k], mg[k], sum(lens) if k in ("dweight", "dbias") else 2 * W, k)


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("C", [5, 264])
def test_conv_pieces_and_tokens_equal_one_prompt(kda, typ, W, C):
    """A prompt in two pieces and then token by token gives the bits of the whole prompt."""
    d = make([50], C, W, TYPES[typ], seed=1)
    whole, last = kda.kda_conv_fwd(d["x"], d["weight"], d["bias"], "silu", initial_state=d["init"])
    o1, s1 = kda.kda_conv_fwd(d["x"][:1], d["weight"], d["bias"], "silu", initial_state=d["init"])
    o2, s2 = kda.kda_conv_fwd(d["x"][1:44], d["weight"], d["bias"], "silu", initial_state=s1)
    outs = [o1, o2]
    for t in range(44, 50):
        outs.append(kda.kda_conv_decode(d["x"][t:t + 1], d["weight"], s2, d["bias"], "silu"))
    assert torch.equal(torch.cat(outs), whole) and torch.equal(s2, last)


def test_conv_decode_slots(kda):
    """Slots of a pool in any order; other slots stay; a bad slot is skipped and recorded; out may be x."""
    d = make([1] * 4, 40, 4, torch.bfloat16, seed=2)
    g = torch.Generator().manual_seed(9)
    pool = torch.randn(6, 3, 40, generator=g).bfloat16().cuda()
    before = pool.clone()
    ref_s = pool[[5, 0, 3, 2]].contiguous()
    ref = kda.kda_conv_decode(d["x"], d["weight"], ref_s, d["bias"])
    idx = torch.tensor([5, 0, 3, 2], dtype=torch.int32, device="cuda")
    x = d["x"].clone()
    got = kda.kda_conv_decode(x, d["weight"], pool, d["bias"], state_indices=idx, out=x)
    assert got is x and torch.equal(x, ref) and torch.equal(pool[[5, 0, 3, 2]], ref_s)
    assert torch.equal(pool[[1, 4]], before[[1, 4]])
    assert kda.device_status(reset=True) == 0
    pool.copy_(before)
    out = torch.full_like(d["x"], 7.0)
    idx = torch.tensor([5, 6, -1, 2], dtype=torch.int32, device="cuda")
    kda.kda_conv_decode(d["x"], d["weight"], pool, d["bias"], state_indices=idx, out=out)
    assert kda.device_status(reset=True) == 4
    assert torch.equal(out[[0, 3]], ref[[0, 3]]) and bool((out[1:3] == 7).all())
    assert torch.equal(pool[[0, 1, 3, 4]], before[[0, 1, 3, 4]])
    assert kda.kda_conv_decode(d["x"][:0], d["weight"], pool, d["bias"]).shape == (0, 40)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("C", [12288, 12289])
def test_conv_decode_many_requests(kda, C, typ, in_place):
    """More requests than blocks: a block takes several, and loads the next one's
    state and token before it writes this one's. The bits of one call per request.
    Bad slots between good ones are skipped."""
    B, P, W = 131, 140, 4
    g = torch.Generator().manual_seed(C)
    d = make([B], C, W, TYPES[typ], state=False, seed=C)
    pool = torch.randn(P, W - 1, C, generator=g).to(TYPES[typ]).cuda()
    slots = torch.randperm(P, generator=g)[:B]
    bad = {0: -1, 30: P, 49: 2 ** 31 - 1, 98: -2 ** 31, 130: P + 5}
    for b, s in bad.items():
        slots[b] = s
    idx = slots.int().cuda()
    ref_pool, ref = pool.clone(), torch.full_like(d["x"], 7.0)
    for b in range(B):
        if b not in bad:
            s = int(slots[b])
            kda.kda_conv_decode(d["x"][b:b + 1], d["weight"], ref_pool[s:s + 1], d["bias"], out=ref[b:b + 1])
    x = d["x"].clone()
    out = x if in_place else torch.full_like(x, 7.0)
    kda.kda_conv_decode(x, d["weight"], pool, d["bias"], state_indices=idx, out=out)
    assert kda.device_status(reset=True) == 4
    good = [b for b in range(B) if b not in bad]
    assert torch.equal(out[good], ref[good]) and torch.equal(pool, ref_pool)
    assert torch.equal(out[list(bad)], d["x"][list(bad)] if in_place else ref[list(bad)])


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("C", [1000, 333])
def test_conv_alone_as_packed(kda, C, typ):
    """A sequence gives the same bits alone and in a batch."""
    lens = [130, 0, 47, 2, 400]
    d = make(lens, C, 4, TYPES[typ], seed=16)
    cu = cu_of(lens)
    out, fin = kda.kda_conv_fwd(d["x"], d["weight"], d["bias"], "silu", cu, d["init"])
    gr = kda.kda_conv_bwd(d["x"], d["weight"], d["dout"], d["bias"], "silu", cu, d["init"], d["dfin"])
    for k, (a, b) in enumerate(R.spans(lens)):
        one = slice(k, k + 1)
        o, f = kda.kda_conv_fwd(d["x"][a:b], d["weight"], d["bias"], "silu", None, d["init"][one])
        g = kda.kda_conv_bwd(d["x"][a:b], d["weight"], d["dout"][a:b], d["bias"], "silu", None, d["init"][one],
                             d["dfin"][one])
        assert torch.equal(o, out[a:b]) and torch.equal(f, fin[one]), k
        assert torch.equal(g["dx"], gr["dx"][a:b]), k
        assert torch.equal(g["dinitial_state"], gr["dinitial_state"][one]), k


def test_conv_padded_batch(kda):
    """Tokens behind the last sequence: outputs left as they were (whatever the
    inputs hold there), gradients zero."""
    lens, T, C = [20, 0, 33], 90, 136
    d = make([T], C, 4, torch.float16, seed=3)
    d["x"][53:] = float("nan")
    d["dout"][53:] = float("inf")
    cu = cu_of(lens)
    out = torch.full((T, C), 5.0, dtype=torch.float16, device="cuda")
    _, fin = kda.kda_conv_fwd(d["x"], d["weight"], d["bias"], cu_seqlens=cu, out=out)
    ref, rfin = kda.kda_conv_fwd(d["x"][:53], d["weight"], d["bias"], cu_seqlens=cu)
    assert torch.equal(out[:53], ref) and bool((out[53:] == 5).all()) and torch.equal(fin, rfin)
    gr = kda.kda_conv_bwd(d["x"], d["weight"], d["dout"], d["bias"], cu_seqlens=cu)
    rg = kda.kda_conv_bwd(d["x"][:53], d["weight"], d["dout"][:53], d["bias"], cu_seqlens=cu)
    assert torch.equal(gr["dx"][:53], rg["dx"]) and not bool(gr["dx"][53:].any())
    for k in ("dweight", "dbias"):  # the runs differ with T, and with them the order of the sums
        assert torch.allclose(gr[k], rg[k], rtol=1e-4, atol=1e-4)
    assert bool(torch.isfinite(gr["dweight"]).all())


def test_conv_empty(kda):
    d = make([3], 24, 4, torch.bfloat16, seed=4)
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    init = torch.randn(2, 3, 24, device="cuda").bfloat16()
    out, fin = kda.kda_conv_fwd(d["x"][:0], d["weight"], cu_seqlens=cu, initial_state=init)
    assert out.shape == (0, 24) and torch.equal(fin, init)
    gr = kda.kda_conv_bwd(d["x"][:0], d["weight"], d["dout"][:0], cu_seqlens=cu, initial_state=init, dfinal_state=init)
    assert torch.equal(gr["dinitial_state"], init) and not bool(gr["dweight"].any()) and gr["dbias"] is None


def test_conv_strided_and_unaligned_views(kda):
    """Columns of a wider buffer, at any element offset, and outputs into one."""
    lens, C = [31, 9], 64
    d = make(lens, C, 4, torch.bfloat16, seed=5)
    cu = cu_of(lens)
    ref, rfin = kda.kda_conv_fwd(d["x"], d["weight"], d["bias"], cu_seqlens=cu, initial_state=d["init"])
    rg = kda.kda_conv_bwd(d["x"], d["weight"], d["dout"], d["bias"], cu_seqlens=cu, initial_state=d["init"])
    for width, at, to in ((3 * C, 0, C), (2 * C + 8, 8, C + 8), (2 * C + 5, 3, C + 4)):
        buf = torch.zeros(40, width, dtype=torch.bfloat16, device="cuda")
        buf[:, at:at + C] = d["x"]
        out = buf[:, to:to + C]
        _, fin = kda.kda_conv_fwd(buf[:, at:at + C], d["weight"], d["bias"], cu_seqlens=cu, initial_state=d["init"],
                                  out=out)
        assert torch.equal(out, ref) and torch.equal(fin, rfin) and torch.equal(buf[:, at:at + C], d["x"])
        gr = kda.kda_conv_bwd(buf[:, at:at + C], d["weight"], d["dout"], d["bias"], cu_seqlens=cu,
                              initial_state=d["init"])
        assert torch.equal(gr["dx"], rg["dx"]) and torch.equal(gr["dinitial_state"], rg["dinitial_state"])


def test_conv_states_and_parameters_at_any_address(kda):
    lens, C = [31, 9], 64
    d = make(lens, C, 4, torch.float16, seed=15)
    cu = cu_of(lens)

    def off(t):
        v = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
        v.copy_(t)
        return v

    e = {k: off(v) for k, v in d.items()}
    a = kda.kda_conv_fwd(d["x"], d["weight"], d["bias"], cu_seqlens=cu, initial_state=d["init"])
    b = kda.kda_conv_fwd(e["x"], e["weight"], e["bias"], cu_seqlens=cu, initial_state=e["init"])
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    ga = kda.kda_conv_bwd(d["x"], d["weight"], d["dout"], d["bias"], "silu", cu, d["init"], d["dfin"])
    gb = kda.kda_conv_bwd(e["x"], e["weight"], e["dout"], e["bias"], "silu", cu, e["init"], e["dfin"])
    assert torch.equal(ga["dx"], gb["dx"]) and torch.equal(ga["dinitial_state"], gb["dinitial_state"])
    for k in ("dweight", "dbias"):  # other runs of tokens, another order of the sums: 40 of at most 40 roundings
        assert torch.allclose(ga[k], gb[k], rtol=1e-4, atol=1e-4)
    s1, s2 = d["init"].clone(), off(d["init"])
    o1 = kda.kda_conv_decode(d["x"][:2], d["weight"], s1, d["bias"])
    o2 = kda.kda_conv_decode(off(d["x"][:2]), e["weight"], s2, e["bias"])
    assert torch.equal(o1, o2) and torch.equal(s1, s2)


def test_conv_bad_boundaries_are_recorded(kda):
    """Boundaries that are no packing: every access is clamped, the status word tells."""
    d = make([60], 72, 4, torch.bfloat16, seed=6)
    for bad in ([0, 50, 20, 60], [0, 30, 99, 10 ** 9], [-5, 10, 40, 60], [4, 10, 40, 60]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        kda.kda_conv_fwd(d["x"], d["weight"], d["bias"], cu_seqlens=cu)
        assert kda.device_status(reset=True) == 1, bad
        kda.kda_conv_bwd(d["x"], d["weight"], d["dout"], d["bias"], cu_seqlens=cu)
        assert kda.device_status(reset=True) == 1, bad


def test_conv_special_values_stay_in_their_channel(kda):
    """An infinity or NaN in one channel's input reaches no other channel and no earlier token."""
    d = make([40], 72, 4, torch.float32, bias=False, state=False, seed=8)
    ref, _ = kda.kda_conv_fwd(d["x"], d["weight"])
    x = d["x"].clone()
    x[10, 7], x[20, 3] = float("nan"), float("inf")
    out, _ = kda.kda_conv_fwd(x, d["weight"])
    same = torch.ones_like(ref, dtype=torch.bool)
    same[10:14, 7] = False
    same[20:24, 3] = False
    assert torch.equal(out[same], ref[same]) and bool(out[10:14, 7].isnan().all())
    big = torch.full((5, 8), -1e30, device="cuda")
    out, _ = kda.kda_conv_fwd(big, torch.ones(8, 2, device="cuda"))
    assert bool((out == 0).all())  # x sigmoid(x) far below zero


def test_conv_graphs_and_streams(kda):
    """Two captured graphs replayed in turn and a call on a side stream give the eager bits."""
    lens = [100, 28]
    d = [make(lens, 264, 4, torch.bfloat16, seed=s) for s in (11, 12)]
    cu = cu_of(lens)

    def step(e):
        o, f = kda.kda_conv_fwd(e["x"], e["weight"], e["bias"], cu_seqlens=cu, initial_state=e["init"])
        g = kda.kda_conv_bwd(e["x"], e["weight"], e["dout"], e["bias"], cu_seqlens=cu, initial_state=e["init"])
        return [o, f] + [v for v in g.values()]

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
    o, f = kda.kda_conv_fwd(d[0]["x"], d[0]["weight"], d[0]["bias"], cu_seqlens=cu, initial_state=d[0]["init"],
                            stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, eager[0][0]) and torch.equal(f, eager[0][1])


def test_conv_in_front_of_the_prefill(kda):
    """q, k and v of a layer: one convolution over the three projections, then
    the fused prefill; continued token by token, as served. The tokens' outputs
    agree with the whole prompt's within the prefill's own bars."""
    from tests import helpers as H

    g = torch.Generator().manual_seed(21)
    T, P, h = 80, 64, 2
    C = 3 * h * 128
    x = torch.randn(T, C, generator=g).bfloat16().cuda()
    w = (torch.randn(C, 4, generator=g) * 0.5).cuda()
    gl = (torch.randn(T, h, 128, generator=g) * 1.5 + 3).cuda()
    bl = torch.randn(T, h, generator=g).cuda()

    def split(y):
        return [t.unflatten(1, (h, 128)) for t in y.split(h * 128, dim=1)]

    y, _ = kda.kda_conv_fwd(x, w)
    whole, state = kda.kda_fwd_fused(*split(y), gl, bl)
    y0, conv_state = kda.kda_conv_fwd(x[:P], w)
    o0, st = kda.kda_fwd_fused(*split(y0), gl[:P], bl[:P])
    outs = [o0]
    for t in range(P, T):
        q, k, v = split(kda.kda_conv_decode(x[t:t + 1], w, conv_state))
        q, k = (torch.nn.functional.normalize(a.float(), dim=-1).bfloat16() for a in (q, k))
        dec = torch.nn.functional.logsigmoid(gl[t:t + 1]).clamp(min=-5)
        outs.append(kda.kda_decode(q, k, v, dec, torch.sigmoid(bl[t:t + 1]), st))
    got = torch.cat(outs).double().cpu().numpy()
    m = H.metrics(got, whole.double().cpu().numpy())
    # the decode step rounds the normalised q and k to bf16, the fused prefill does not: a second rounding of each
    assert m["max_abs"] <= 2 * H.O_MAX_ABS and m["rel_rms"] <= 2 * H.O_REL_RMS, m
    assert H.metrics(st.double().cpu().numpy(), state.double().cpu().numpy())["rel_rms"] <= 2 * H.S_REL_RMS
