"""GPU tests of what the library leaves behind when a call fails, and of its
status words and first calls."""
import gc

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kimi_delta_attention_26_b200 as m

    m.device_status(reset=True)
    yield m
    assert m.device_status(reset=True) == 0


def too_large(kda):
    """Gradients whose scratch (over 300 GB) no device holds; the inputs' rows overlap and take no memory."""
    T, c, n = 1 << 17, 8192, 128
    rows = torch.zeros(T + c, device="cuda", dtype=torch.bfloat16).as_strided((T, c), (1, 1))
    bc = torch.zeros(T, 1, n, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(kda.KDAError) as e:
        kda.kda_ssm_bwd(rows, rows, torch.zeros(c, n, device="cuda"), bc, bc, rows)
    assert e.value.code == 5 and "out of memory" in str(e.value)


def test_a_failed_call_does_not_fail_the_next_one(kda):
    x, w = torch.randn(60, 72, device="cuda"), torch.randn(72, 4, device="cuda")
    ref, _ = kda.kda_conv_fwd(x, w)
    too_large(kda)
    out, _ = kda.kda_conv_fwd(x, w)
    assert torch.equal(out, ref)
    too_large(kda)
    assert bool(torch.isfinite(torch.exp(-x * x)).all())  # nor a launch of the caller's own


def test_a_failed_call_gives_its_memory_back(kda):
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = torch.cuda.mem_get_info()[0]
    too_large(kda)
    gc.collect()  # the error's traceback holds the binding's own outputs, 4.4 GB
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # a few pages more or less may belong to the driver
    assert torch.cuda.mem_get_info()[0] >= before - (64 << 20)


def test_the_status_word_waits_for_every_stream(kda):
    """A call that is still pending on a non-blocking stream (as torch's are) counts."""
    x, w = torch.randn(60, 72, device="cuda"), torch.randn(72, 4, device="cuda")
    good, bad = (torch.tensor(b, dtype=torch.int32, device="cuda") for b in ([0, 20, 50, 60], [0, 50, 20, 60]))
    kda.kda_conv_fwd(x, w, cu_seqlens=good)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for reset in (False, True):
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)  # about 50 ms
            kda.kda_conv_fwd(x, w, cu_seqlens=bad)
        assert kda.device_status(reset=reset) == 1
    torch.cuda.synchronize()
    assert kda.device_status() == 0  # nothing came after the reset


STATUS_TIMES = """
import time, torch
import kimi_delta_attention_26_b200 as kda
q = torch.zeros(16, 1, 128, dtype=torch.bfloat16, device="cuda")
g = torch.zeros(16, 1, 128, device="cuda")
kda.kda_fwd(q, q, q, g, g[..., 0].contiguous())
def each():
    kda.device_status()
    t = []
    for _ in range(50):
        t0 = time.perf_counter()
        kda.device_status()
        t.append(time.perf_counter() - t0)
    return sorted(t)[25]
t0 = time.perf_counter()
kda.device_status()
first, before = time.perf_counter() - t0, each()
for t in (torch.bfloat16, torch.float16, torch.float32):
    kda.kda_conv_fwd(torch.zeros(4, 8, dtype=t, device="cuda"), torch.zeros(8, 4, device="cuda"))
print(first, before, each())
"""


def test_the_status_word_reads_only_what_ran(kda):
    """Reading the status after KDA calls alone copies two words, not eight
    (2 copies and 2 resets against 8 and 2), and loads no other code onto the device."""
    import subprocess
    import sys

    from tests.conftest import ROOT

    out = subprocess.run([sys.executable, "-c", STATUS_TIMES], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr
    first, before, after = (float(v) for v in out.stdout.split()[-3:])
    assert before < 0.7 * after, (first, before, after)
    assert first < 0.010, (first, before, after)  # three units' code took 40 ms


FIRST_CALL = """
import sys, torch
import kimi_delta_attention_26_b200 as kda
g = torch.Generator(device="cuda").manual_seed(1)
rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
T, c = 1100, 64
x, w, A = rnd(T, c), rnd(c, 4), -torch.exp(rnd(c, 16))
B, C, dt = rnd(T, 1, 16), rnd(T, 1, 16), rnd(T, c)
k = torch.nn.functional.normalize(rnd(T, 1, 128), dim=-1).bfloat16()
f = (k, k, k, -torch.rand(T, 1, 128, device="cuda"), torch.rand(T, 1, device="cuda"))
calls = {
    "conv_bwd": lambda: kda.kda_conv_bwd(x, w, x).values(),
    "ssm_fwd": lambda: kda.kda_ssm_fwd(x, dt, A, B, C),
    "ssm_bwd": lambda: kda.kda_ssm_bwd(x, dt, A, B, C, x).values(),
    "fwd": lambda: kda.kda_fwd(*f),
    "bwd": lambda: kda.kda_bwd(*f, k).values(),
}
call = calls[sys.argv[1]]
kda.set_time_split(int(sys.argv[2]))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = [t for t in call() if t is not None]
for t in out:
    t.zero_()
for _ in range(2):
    graph.replay()
torch.cuda.synchronize()
assert all(torch.isfinite(t).all() for t in out)
assert all(torch.equal(a, b) for a, b in zip(out, [t for t in call() if t is not None]))
assert kda.device_status() == 0
"""


@pytest.mark.parametrize("name,split", [("conv_bwd", 0), ("ssm_fwd", 2), ("ssm_bwd", 1), ("ssm_bwd", 2), ("fwd", 1),
                                        ("fwd", 2), ("bwd", 0)])
def test_a_first_call_can_be_captured(kda, name, split):
    """The first call of a process that takes scratch, in a capture."""
    import subprocess
    import sys

    from tests.conftest import ROOT

    out = subprocess.run([sys.executable, "-c", FIRST_CALL, name, str(split)], cwd=ROOT, capture_output=True, text=True,
                         timeout=300)
    assert out.returncode == 0, out.stderr
