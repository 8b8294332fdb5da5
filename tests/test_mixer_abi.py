"""The convolution's and the scan's entry points refuse bad arguments on the
host before touching the GPU (CPU only; the fake addresses are never used)."""
import ctypes

import pytest

from tests.test_abi import (BF16, F32, I32, KDA_ERR_ALIGN, KDA_ERR_DTYPE, KDA_ERR_NULL, KDA_ERR_SHAPE, KDA_ERR_STRIDE,
                            KDA_ERR_VALUE, desc, lib)  # noqa: F401

F16, KDA_ERR_OVERLAP = 4, 11
T, C, W, N, S, G, R = 64, 24, 4, 2, 16, 2, 5
SIZE = 1 << 24  # between two tensors' fake addresses


def _addr(i):
    return (i + 1) * SIZE


CONV = {
    "kda_conv_fwd": ["x", "weight", "bias", "#act", "@cu", "#n", "init", "out", "fin"],
    "kda_conv_decode": ["x", "weight", "bias", "#act", "state", "@idx", "out"],
    "kda_conv_bwd": ["x", "weight", "bias", "#act", "@cu", "#n", "init", "dout", "dfin", "dx", "dweight", "dbias",
                     "dinit"],
}
SSM = {
    "kda_ssm_fwd": ["u", "dt", "A", "B", "C", "D", "z", "bias", "#sp", "@cu", "#n", "init", "out", "fin"],
    "kda_ssm_decode": ["u", "dt", "A", "B", "C", "D", "z", "bias", "#sp", "state", "@idx", "out"],
    "kda_ssm_bwd": ["u", "dt", "A", "B", "C", "D", "z", "bias", "#sp", "@cu", "#n", "init", "dout", "dfin", "du", "ddt",
                    "dA", "dB", "dC", "dD", "dz", "dbias", "dinit"],
}


def _shapes(fn):
    if "conv" in fn:
        st = [R if fn.endswith("decode") else N, W - 1, C]
        return {"x": (BF16, [T, C]), "weight": (F32, [C, W]), "bias": (F32, [C]), "init": (BF16, st),
                "out": (BF16, [T, C]), "fin": (BF16, st), "state": (BF16, [T + 3, W - 1, C]), "dout": (BF16, [T, C]),
                "dfin": (BF16, st), "dx": (BF16, [T, C]), "dweight": (F32, [C, W]), "dbias": (F32, [C]),
                "dinit": (BF16, st)}
    tok, par, st, bc = (BF16, [T, C]), (F32, [C]), (F32, [N, C, S]), (BF16, [T, G, S])
    return {"u": tok, "dt": tok, "A": (F32, [C, S]), "B": bc, "C": bc, "D": par, "z": tok, "bias": par, "init": st,
            "out": tok, "fin": st, "state": (F32, [T + 3, C, S]), "dout": tok, "dfin": st, "du": tok, "ddt": tok,
            "dA": (F32, [C, S]), "dB": bc, "dC": bc, "dD": par, "dz": tok, "dbias": par, "dinit": st}


def call(lib, fn, **over):  # noqa: F811
    args, types = [], []
    for i, name in enumerate((CONV if "conv" in fn else SSM)[fn]):
        if name[0] == "#":
            args.append(over.get(name[1:], {"act": 1, "n": N, "sp": 1}[name[1:]]))
            types.append(ctypes.c_int32)
        elif name[0] == "@":
            args.append(over.get(name[1:], 0x7000))
            types.append(ctypes.c_void_p)
        else:
            dt, shape = _shapes(fn)[name]
            d = over[name] if name in over else desc(_addr(i), dt, shape)
            args.append(None if d is None else ctypes.byref(d))
            types.append(ctypes.c_void_p)
    f = getattr(lib, fn)
    f.argtypes, f.restype = types + [ctypes.c_void_p], ctypes.c_int
    return f(*args, None)


ALL = list(CONV) + list(SSM)
OPTIONAL = {"bias", "init", "fin", "dfin", "dbias", "dinit", "D", "z", "dD", "dz"}


def tensors(fn):
    return [(i, n) for i, n in enumerate((CONV if "conv" in fn else SSM)[fn]) if n[0] not in "#@"]


@pytest.mark.parametrize("fn", ALL)
def test_a_valid_call_passes_the_checks(lib, fn):  # noqa: F811
    import torch

    if torch.cuda.is_available():
        pytest.skip("would launch on the fake addresses")
    assert call(lib, fn) in (4, 5)  # stops at the device query
    for i, n in tensors(fn):  # whatever is optional may be missing
        if n in OPTIONAL and n not in ("z", "dz"):
            assert call(lib, fn, **{n: None}) in (4, 5), n
    for dt in (F16, F32):
        over = {n: desc(_addr(i), dt, _shapes(fn)[n][1]) for i, n in tensors(fn) if _shapes(fn)[n][0] == BF16}
        assert call(lib, fn, **over) in (4, 5)


@pytest.mark.parametrize("fn", ALL)
def test_missing_wrong_typed_misshaped_tensors(lib, fn):  # noqa: F811
    for i, n in tensors(fn):
        dt, shape = _shapes(fn)[n]
        if n not in OPTIONAL:
            assert call(lib, fn, **{n: None}) == KDA_ERR_NULL, n
        assert call(lib, fn, **{n: desc(None, dt, shape)}) == KDA_ERR_NULL, n
        assert call(lib, fn, **{n: desc(_addr(i), I32, shape)}) == KDA_ERR_DTYPE, n
        for k in range(len(shape)):
            if n in ("x", "u", "A", "weight", "state") and k == len(shape) - 1 - (n in ("state",)):
                continue  # sets the size for the others
            bad = list(shape)
            bad[k] += 1
            if n == "state" and k == 0:
                bad[0] = 0
            if n == "B" and k == 1:
                bad[1] = 5  # does not divide the channels
            assert call(lib, fn, **{n: desc(_addr(i), dt, bad)}) == KDA_ERR_SHAPE, (n, k)
        assert call(lib, fn, **{n: desc(_addr(i), dt, shape + [1])}) == KDA_ERR_SHAPE, n
        assert call(lib, fn, **{n: desc(_addr(i) + 1, dt, shape)}) == KDA_ERR_ALIGN, n


@pytest.mark.parametrize("fn", ALL)
def test_strides(lib, fn):  # noqa: F811
    for i, n in tensors(fn):
        dt, shape = _shapes(fn)[n]
        wide = []
        acc = 2
        for k in reversed(shape):
            wide.insert(0, acc)
            acc *= k
        assert call(lib, fn, **{n: desc(_addr(i), dt, shape, wide)}) == KDA_ERR_STRIDE, n
        rows = dt == BF16 and shape[0] == T
        if rows and n != "state":
            for st in (0, -C):
                strides = [st] + ([S, 1] if len(shape) == 3 else [1])
                assert call(lib, fn, **{n: desc(_addr(i), dt, shape, strides)}) == KDA_ERR_STRIDE, (n, st)
            if n in ("out", "dx", "du", "ddt", "dz", "dB", "dC"):  # rows that overlap each other
                strides = [S, S, 1] if len(shape) == 3 else [C - 1, 1]
                assert call(lib, fn, **{n: desc(_addr(i), dt, shape, strides)}) == KDA_ERR_STRIDE, n


@pytest.mark.parametrize("fn", ALL)
def test_overlaps(lib, fn):  # noqa: F811
    names = dict((n, i) for i, n in tensors(fn))
    outs = [n for n in names if n in ("out", "fin", "dx", "dweight", "dbias", "dinit", "du", "ddt", "dA", "dB", "dC",
                                      "dD", "dz", "state")]
    for o in outs:
        dt, shape = _shapes(fn)[o]
        for n, i in names.items():
            if n == o or (o, n) == ("fin", "init") and "ssm" in fn or {o, n} == {"out", "x"} and fn.endswith("decode"):
                continue
            if n in outs and outs.index(n) < outs.index(o):
                continue
            # one element into the other tensor
            assert call(lib, fn, **{o: desc(_addr(i) + 4, dt, shape)}) == KDA_ERR_OVERLAP, (o, n)


def test_interleaved_columns_do_not_overlap(lib):  # noqa: F811
    import torch

    if torch.cuda.is_available():
        pytest.skip("would launch on the fake addresses")
    st = [3 * C, 1]
    x = desc(_addr(0), BF16, [T, C], st)
    assert call(lib, "kda_conv_fwd", x=x, out=desc(_addr(0) + 2 * C, BF16, [T, C], st)) in (4, 5)
    assert call(lib, "kda_conv_fwd", x=desc(_addr(0) + 4 * C, BF16, [T, C], st),
                out=desc(_addr(0), BF16, [T, C], st)) in (4, 5)
    assert call(lib, "kda_conv_fwd", x=x, out=desc(_addr(0) + 2 * C - 2, BF16, [T, C], st)) == KDA_ERR_OVERLAP
    assert call(lib, "kda_conv_fwd", x=x, out=desc(_addr(0) + 4 * C + 2, BF16, [T, C], st)) == KDA_ERR_OVERLAP
    assert call(lib, "kda_conv_fwd", x=x, out=desc(_addr(0) + 2 * C, BF16, [T, C], [3 * C + 8, 1])) == KDA_ERR_OVERLAP
    # the decode step may write its output over its input
    x = desc(_addr(0), BF16, [T, C])
    assert call(lib, "kda_conv_decode", x=x, out=x) in (4, 5)
    st = desc(_addr(9), F32, [N, C, S])
    assert call(lib, "kda_ssm_fwd", init=st, fin=st) in (4, 5)


@pytest.mark.parametrize("fn", ALL)
def test_scalars_and_boundaries(lib, fn):  # noqa: F811
    if "conv" in fn:
        for act in (-1, 2):
            assert call(lib, fn, act=act) == KDA_ERR_VALUE
    if fn.endswith("decode"):
        assert call(lib, fn, idx=0x7002) == KDA_ERR_ALIGN
        dt, shape = _shapes(fn)["state"]
        small = desc(_addr(20), dt, [T - 1] + shape[1:])
        assert call(lib, fn, idx=None, state=small) == KDA_ERR_SHAPE  # fewer slots than requests
        return
    assert call(lib, fn, cu=0x7002) == KDA_ERR_ALIGN
    assert call(lib, fn, cu=None) == KDA_ERR_SHAPE  # two sequences without boundaries
    for n in (0, -1, 65536):
        assert call(lib, fn, n=n) == KDA_ERR_SHAPE


def test_sizes(lib):  # noqa: F811
    for w in (1, 5):
        over = {"weight": desc(_addr(1), F32, [C, w])}
        for fn in CONV:
            assert call(lib, fn, **over) == KDA_ERR_SHAPE
    for s in (0, 129):
        for fn in SSM:
            assert call(lib, fn, A=desc(_addr(2), F32, [C, s])) == KDA_ERR_SHAPE
    for fn in SSM:
        assert call(lib, fn, B=desc(_addr(3), BF16, [T, 0, S])) == KDA_ERR_SHAPE
    # the gate and its gradient come together
    assert call(lib, "kda_ssm_bwd", z=None) == KDA_ERR_NULL
    assert call(lib, "kda_ssm_bwd", dz=None) == KDA_ERR_NULL
    lib.kda_status_string.restype = ctypes.c_char_p
    assert b"overlap" in lib.kda_status_string(KDA_ERR_OVERLAP)


def test_binding_refuses_cpu_tensors_and_bad_names():
    import torch

    import kimi_delta_attention_26_b200 as kda

    x, w = torch.zeros(3, 8), torch.zeros(8, 4)
    for f in (lambda: kda.kda_conv_fwd(x, w), lambda: kda.kda_conv_decode(x, w, torch.zeros(3, 3, 8)),
              lambda: kda.kda_conv_bwd(x, w, x), lambda: kda.kda_ssm_fwd(x, x, w, x, x),
              lambda: kda.kda_ssm_decode(x, x, w, x, x, x), lambda: kda.kda_ssm_bwd(x, x, w, x, x, x)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        kda.kda_conv_fwd([1], w)
    with pytest.raises(ValueError):
        kda.kda_conv_fwd(x[0], w)
