"""The operators between a layer's products where their values or operands lie at an edge: gates whose quotient alone is
below f32, angles far below a step of the usual ones, operands of which one is unaligned, rows around
the border between two ways of the product, first calls of several threads."""
import subprocess
import sys
import threading

import pytest
import torch

import bit_quantized_gemv_dequant_gb300 as qg
from test_gpu_serving_calls import ROOT

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {torch.float32: 0.0, torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}
TINY = {torch.float32: 2.0**-149, torch.float16: 2.0**-25, torch.bfloat16: 2.0**-134}


def gate_bound(want, out):
    """5 units of 2^-23, as for every gate, and half a step of the output's type; what is below 2^-119 may be 0."""
    lost = torch.where(want.abs() < 2.0**-119, want.abs(), torch.zeros_like(want))
    return want.abs() * (5 * 2.0**-23 + HALF[out]) + lost + TINY[out]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("K", [4096, 4099])
def test_small_gates_of_large_values(x, out, K):
    """Gates from -300 to -60, times values of every size up to f32's largest: the product is an ordinary number where the
    gate alone is not."""
    g = torch.linspace(-300, -60, K, device="cuda").to(DTYPES[x])
    exponents = [-100, -30, 0, 20, 60, 100, 120, 127]
    gate = g.repeat(2 * len(exponents), 1)
    up = torch.rand(gate.shape, generator=torch.Generator("cuda").manual_seed(K), device="cuda") * 0.99 + 1
    up *= torch.exp2(torch.tensor(exponents * 2, device="cuda").float())[:, None]
    up[len(exponents):] *= -1
    up = up.to(DTYPES[x])
    y = qg.silu_mul(gate, up, out_dtype=DTYPES[out])
    a, b = gate.double(), up.double()
    want = b * a / (1 + torch.exp(-a))
    assert (want.abs() > 2.0**-100).sum() > 10000
    bad = (y.double() - want).abs() > gate_bound(want, y.dtype)
    assert not bad.any(), (int(bad.sum()), [(float(gate[tuple(i)]), float(up[tuple(i)]), float(y[tuple(i)])) for i in bad.nonzero()[:3]])
    codes, scales = qg.silu_mul_fp8_b128(gate, up)
    same = qg.quantize_fp8_b128(qg.silu_mul(gate, up, out_dtype=torch.float32))
    assert torch.equal(codes.view(torch.uint8), same[0].view(torch.uint8)) and torch.equal(scales, same[1])


def test_small_gates_among_others():
    """A row's result is the same whether or not its neighbours have small gates."""
    g = torch.Generator("cuda").manual_seed(1)
    gate = torch.randn(64, 1024, generator=g, device="cuda") * 4
    up = torch.randn(64, 1024, generator=g, device="cuda")
    y = qg.silu_mul(gate, up)
    at = torch.rand(64, 1024, generator=g, device="cuda") < 0.05
    z = qg.silu_mul(torch.where(at, torch.full_like(gate, -90.0), gate), torch.where(at, torch.full_like(up, 1e38), up))
    assert torch.equal(z[~at], y[~at])
    want = 1e38 * -90.0 * float(torch.exp(torch.tensor(-90.0, dtype=torch.float64)))
    assert (z[at].double() / want - 1).abs().max() < 5 * 2.0**-23 + 2.0**-24  # (1e38 is rounded)
    odd = torch.tensor([[float("-inf"), -100.0, -100.0, float("nan"), -3e38, -2000.0, -90.0]], device="cuda")
    y = qg.silu_mul(odd, torch.tensor([[1.0, float("inf"), float("nan"), 1.0, 3e38, 3e38, 0.0]], device="cuda"))[0]
    assert torch.isnan(y[[0, 2, 3]]).all() and y[1] == float("-inf") and (y[4:] == 0).all()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D", [64, 40])
def test_small_angles(D, inter):
    """Pairs (a, 0) at angles down to 2^-29, of both signs: the second value is a times the sine, whose relative error is that
    of the angle in f32 (2^-24), of the sine (2 units of 2^-23) and of the product (2^-24), 6 x 2^-24, next to the angle's 2^-64
    of a turn per position and half a step of the output."""
    n = D // 2
    freq = torch.exp2(-torch.linspace(4, 29, n, device="cuda")).contiguous()
    positions = torch.tensor([1, -1, 3, -3, 1000, -1000, 0], device="cuda")
    T = positions.numel()
    q = torch.zeros(T, 2, D, device="cuda")
    first, second = (slice(0, D, 2), slice(1, D, 2)) if inter else (slice(0, n), slice(n, D))
    angle = positions.double()[:, None] * freq.double()
    a = torch.exp2(-torch.floor(torch.log2(angle.abs() + 2.0**-40)))  # a power of two: the result is about 1
    q[:, :, first] = a.float()[:, None]
    kc, vc = (torch.zeros(2, 2, 8, D, dtype=torch.float16, device="cuda") for _ in range(2))
    out = qg.kv_append_rope(q, q, q, positions, freq, kc, vc, torch.arange(T, device="cuda"), interleaved=inter)
    sine = angle.sin() * a
    bound = sine.abs() * (6 * 2.0**-24 + HALF[torch.float16]) + a * positions.abs()[:, None] * 2.0**-61
    for heads in (out, kc[0, :, :T].transpose(0, 1)):
        bad = (heads[:, :, second].double() - sine[:, None]).abs() > bound[:, None]
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist())
    assert qg.device_error() == 0


def experts(seed, rows, E, N, K):
    g = torch.Generator("cuda").manual_seed(seed)

    def codes(*shape):
        return (torch.randn(*shape, generator=g, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn)

    a, w = codes(rows, K), codes(E, N, K)
    sa = torch.rand(rows, -(-K // 128), generator=g, device="cuda") + 0.5
    sw = torch.rand(E, -(-N // 128), -(-K // 128), generator=g, device="cuda") + 0.5
    offsets = torch.linspace(0, rows, E + 1, device="cuda").to(torch.int32)
    return a, sa, w, sw, offsets


def shifted(t, by):
    flat = torch.empty(t.numel() + by, dtype=torch.uint8, device="cuda")[by:]
    flat.copy_(t.view(torch.uint8).flatten())
    return flat.view(t.dtype).view(t.shape)


@pytest.mark.parametrize("rows", [9, 700])
def test_scratch_is_for_what_is_unaligned(rows):
    """One unaligned operand takes a copy of itself alone, and the products are those of aligned ones, bit by bit."""
    E, N, K = 6, 520, 1024
    a, sa, w, sw, offsets = experts(rows, rows, E, N, K)
    want = qg.qmm_fp8_b128_grouped(a, sa, w, sw, offsets)
    for x, y, need in ((shifted(a, 1), w, rows * K), (a, shifted(w, 4), E * N * K),
                       (shifted(a, 8), shifted(w, 3), (rows + E * N) * K)):
        guarded = torch.full((need + 64,), 0x7F, dtype=torch.uint8, device="cuda")
        got = qg.qmm_fp8_b128_grouped(x, sa, y, sw, offsets, workspace=guarded[:need])
        assert torch.equal(got, want) and (guarded[need:] == 0x7F).all()
    assert qg.device_error() == 0


def test_scratch_of_a_call_without_workspace():
    E, N, K, rows = 16, 1024, 4096, 40
    a, sa, w, sw, offsets = experts(1, rows, E, N, K)
    want = qg.qmm_fp8_b128_grouped(a, sa, w, sw, offsets)
    x, out = shifted(a, 1), torch.empty_like(want)
    with torch.cuda.stream(torch.cuda.Stream()):  # one that has no scratch yet
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        qg.qmm_fp8_b128_grouped(x, sa, w, sw, offsets, out)
        torch.cuda.synchronize()
        assert torch.cuda.memory_allocated() - before <= rows * K + 1024
    assert torch.equal(out, want)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [256, 200, 131])
def test_chunks_around_the_border(N, out):
    """Chunks of up to 192 rows and of more take different sides of the product; whole numbers and scales of 1 make every
    order of the sum exact (to half a step of bf16)."""
    counts = [159, 160, 161, 191, 192, 193, 194, 223, 225, 255, 1, 257, 447, 449]
    g = torch.Generator("cuda").manual_seed(N)
    E, rows, K = len(counts), sum(counts), 384

    def codes(*shape):
        return torch.randint(-3, 4, shape, generator=g, device="cuda").float().to(torch.float8_e4m3fn)

    a, w = codes(rows, K), codes(E, N, K)
    sa, sw = torch.ones(rows, 3, device="cuda"), torch.ones(E, -(-N // 128), 3, device="cuda")
    offsets = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
    y = qg.qmm_fp8_b128_grouped(a, sa, w, sw, offsets, out_dtype=out)
    at = offsets.tolist()
    for e in range(E):
        want = a[at[e]:at[e + 1]].float() @ w[e].float().T
        assert torch.equal(y[at[e]:at[e + 1]], want.to(out)), e
    assert qg.device_error() == 0


def first_calls():
    """Each thread's first calls are the process's first ones too, of kernels whose shared memory is set at the first call.
    Later calls give the same."""
    g = torch.Generator("cuda").manual_seed(7)
    few, many = experts(8, 12, 4, 256, 512), experts(9, 700, 3, 256, 512)
    logits = torch.randn(2, 4000, generator=g, device="cuda")
    codes = torch.randint(0, 16, (256, 4096), generator=g, device="cuda", dtype=torch.uint8)
    s, b = (torch.rand(256, 64, generator=g, device="cuda").bfloat16() for _ in range(2))
    plane, meta = qg.prepare_af4_g64(codes, s, b)
    xs = [torch.randn(m, 4096, generator=g, device="cuda") for m in (3, 5, 9, 16, 24, 32)]
    a, sa, w, sw, _ = experts(10, 300, 1, 384, 512)
    plain = (a, sa, w[0], sw[0])

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            out = [qg.qmm_af4_g64(xs[i], plane, meta, 256), qg.qmm_fp8_b128_grouped(*few), qg.qmm_fp8_b128_grouped(*many),
                   qg.qmm_fp8_b128(*plain), qg.token_logprobs(logits, torch.zeros(2, dtype=torch.int64, device="cuda"), 4)[0]]
            torch.cuda.current_stream().synchronize()
        return out

    torch.cuda.synchronize()
    start, got = threading.Barrier(len(xs)), [None] * len(xs)

    def thread(i):
        start.wait(60)
        got[i] = work(i)

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(len(xs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(len(xs)):
        assert got[i] is not None and all(torch.equal(x, y) for x, y in zip(got[i], work(i), strict=True))
    assert qg.device_error() == 0


def test_first_calls_of_several_threads():
    for _ in range(3):
        code = "import sys; sys.path[:0] = ['tests', '.']; import test_gpu_layer_edges as t; t.first_calls()"
        r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]


def test_tensors_of_another_device(monkeypatch):
    """The kernels run on the current device: tensors elsewhere are refused, not read."""
    x = torch.ones(4, 256, device="cuda")
    w = torch.zeros(8 * 18, dtype=torch.uint8, device="cuda")
    assert qg.silu_mul(x, x).shape == x.shape and qg.qgemv_q4_0(w, x[:1], N=1).shape == (1, 1)
    here = torch.cuda.current_device()
    if torch.cuda.device_count() > 1:
        with torch.cuda.device(1 - min(here, 1)):
            for call in (lambda: qg.silu_mul(x, x), lambda: qg.rms_norm(x), lambda: qg.quantize_fp8_b128(x),
                         lambda: qg.qgemv_q4_0(w, x[:1], N=1)):
                with pytest.raises(ValueError, match="current device"):
                    call()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: here + 1)
    with pytest.raises(ValueError, match="current device"):
        qg.qgemv_q4_0(w, x[:1], N=1, stream=0)
    monkeypatch.undo()
    assert qg.device_error() == 0
