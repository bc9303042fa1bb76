"""silu_mul and silu_mul_fp8_b128 against their definition in 64 bits.

The exponential is off by at most 1 unit (2^-23) and enters a sum not smaller than itself, which is rounded (2^-24); the
quotient by 2 units, the product with up is rounded: 4 units, taken as 5, and half a step of the output's type. Results below
2^-119 may be 0. Codes and scales are those of the f32 output."""
import pytest
import torch

import bit_quantized_gemv_dequant_gb300 as qg

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {torch.float32: 0.0, torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}
TINY = {torch.float32: 0.0, torch.float16: 2.0**-25, torch.bfloat16: 2.0**-134}


def make(seed, M, K, x):
    both = torch.randn(M, 2 * K, generator=torch.Generator("cuda").manual_seed(seed), device="cuda") * 4
    return both.to(DTYPES[x])


def check(y, gate, up):
    g, u = gate.double(), up.double()
    want = u * g * torch.sigmoid(g)
    tol = want.abs() * (5 * 2.0**-23 + HALF[y.dtype]) + TINY[y.dtype] + 2.0**-119 * (1 + u.abs())
    bad = (y.double() - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist())


SHAPES = [(1, 1), (2, 8), (3, 127), (5, 128), (4, 136), (17, 1000), (130, 1032), (1, 12288), (64, 4096)]


@pytest.mark.parametrize("x", list(DTYPES))
@pytest.mark.parametrize("out", list(DTYPES))
@pytest.mark.parametrize("M,K", SHAPES)
def test_gate(M, K, x, out):
    both = make(M + K, M, K, x)
    gate, up = both[:, :K], both[:, K:]  # halves of one product's rows
    y = qg.silu_mul(gate, up, out_dtype=DTYPES[out])
    check(y, gate, up)
    dense = qg.silu_mul(gate.contiguous(), up.contiguous(), out_dtype=DTYPES[out])
    assert torch.equal(y, dense)
    codes, scales = qg.silu_mul_fp8_b128(gate, up)
    want = qg.quantize_fp8_b128(qg.silu_mul(gate, up, out_dtype=torch.float32))
    assert torch.equal(codes.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(scales, want[1])
    assert qg.device_error() == 0


def test_gate_of_any_size():
    g = torch.cat([torch.linspace(-200, 200, 40001), torch.tensor([0.0, -0.0, 3e38, -3e38, 1e-40, -1e-40])])
    g = g.view(1, -1).cuda()
    up = torch.randn(g.shape, generator=torch.Generator().manual_seed(1)).cuda()
    up[0, -4:-2] = 0.25
    check(qg.silu_mul(g, up), g, up)
    odd = torch.tensor([[float("nan"), float("inf"), float("-inf"), float("inf"), 1.0]], device="cuda")
    y = qg.silu_mul(odd, torch.tensor([[1.0, 2.0, 1.0, 0.0, float("inf")]], device="cuda"))[0]
    assert torch.isnan(y[0]) and y[1] == float("inf") and torch.isnan(y[2]) and torch.isnan(y[3]) and y[4] == float("inf")


def test_halves_apart_and_outputs_given():
    base = torch.randn(9, 1000, generator=torch.Generator("cuda").manual_seed(4), device="cuda").bfloat16()
    for a, b in ((0, 256), (8, 504), (3, 300)):
        gate, up = base[:, a:a + 200], base[:, b:b + 200]
        out = torch.empty(9 * 200 + 1, device="cuda")[1:].view(9, 200)
        assert qg.silu_mul(gate, up, out).data_ptr() == out.data_ptr()
        check(out, gate, up)
        codes = torch.empty(9 * 200 + 3, dtype=torch.uint8, device="cuda")[3:].view(9, 200).view(torch.float8_e4m3fn)
        qg.silu_mul_fp8_b128(gate, up, codes)
        assert torch.equal(codes.view(torch.uint8), qg.silu_mul_fp8_b128(gate.contiguous(), up.contiguous())[0].view(torch.uint8))


def test_no_rows_and_refusals():
    x = torch.ones(4, 256, device="cuda")
    assert qg.silu_mul(x[:0], x[:0]).shape == (0, 256) and qg.silu_mul_fp8_b128(x[:0], x[:0])[1].shape == (0, 2)
    for call in (lambda: qg.silu_mul(x, x[:3]), lambda: qg.silu_mul(x, x.half()), lambda: qg.silu_mul(x.cpu(), x),
                 lambda: qg.silu_mul(x[:, ::2], x[:, ::2]), lambda: qg.silu_mul(x.double(), x.double()),
                 lambda: qg.silu_mul(x, x, torch.empty(4, 255, device="cuda")), lambda: qg.silu_mul(x, x, out_dtype=torch.int8),
                 lambda: qg.silu_mul_fp8_b128(x, x, torch.empty(4, 256, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(qg.QGError):
        qg.silu_mul(x, x.clone(), x)
