"""The operators between a layer's products on tensors of more than 2^31 elements, so that offsets pass 32 bits: what
lies at their ends is held against the same call on a small copy of it (the same bits), or against 64 bits for products, whose
bound is 1e-5 * sum |terms| + 1e-6 and a bf16 rounding."""
import pytest
import torch

import bit_quantized_gemv_dequant_gb300 as qg
from test_gpu_serving_large import give_back, rng  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_and_gate(dtype):
    M, K = 2**31 // 4104 + 9, 4104
    x = torch.zeros(M, K, dtype=dtype, device="cuda")
    x[-9:] = torch.randn(9, K, generator=rng(1), device="cuda").to(dtype)
    small = x[-9:].clone()
    y, r = qg.rms_norm(x, None, x)
    want = qg.rms_norm(small, None, small)
    assert torch.equal(y[-9:], want[0]) and torch.equal(r[-9:], want[1]) and not y[:-9].any()
    del y, r
    for call in (qg.rms_norm_fp8_b128, lambda x: qg.silu_mul_fp8_b128(x, x)):
        codes, scales = call(x)
        c, s = call(small)
        assert torch.equal(codes[-9:].view(torch.uint8), c.view(torch.uint8)) and torch.equal(scales[-9:], s)
        assert not codes[:-9].view(torch.uint8).any() and (scales[:-9] == 1).all()
        del codes, scales
    y = qg.silu_mul(x, x)
    assert torch.equal(y[-9:], qg.silu_mul(small, small)) and not y[:-9].any()


def test_rope():
    hkv, page, d, T = 2, 64, 128, 2**31 // 1024 + 50
    pages = 2**31 // (hkv * page * d) + 40
    cache = [torch.zeros(pages, hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    small = [torch.zeros(40, hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    qkv = torch.zeros(T, 8, d, dtype=torch.bfloat16, device="cuda")
    qkv[-50:] = torch.randn(50, 8, d, generator=rng(2), device="cuda").bfloat16()
    freq = torch.tensor([10000.0 ** (-i / 64) for i in range(64)], device="cuda")
    positions = torch.arange(T, device="cuda")
    slots = torch.full((T,), -1, device="cuda")
    at = torch.randperm(40 * page, generator=rng(3), device="cuda")[:50]
    slots[-50:] = at + (pages - 40) * page
    q = qg.kv_append_rope(qkv, qkv[:, :2], qkv[:, 2:4], positions, freq, *cache, slots)
    last = qkv[-50:].clone()
    want = qg.kv_append_rope(last, last[:, :2], last[:, 2:4], positions[-50:], freq, *small, at)
    assert torch.equal(q[-50:], want) and not q[:-50].any()
    for c, s in zip(cache, small):
        assert torch.equal(c[-40:], s) and not c[:-40].any()
    assert qg.device_error() == 0


def codes(g, *shape):
    return torch.randint(0, 120, shape, generator=g, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)


def check(y, a, sa, w, sw, rows):
    n = w.shape[0]
    ref = (a[rows].double() * sa[rows].double().repeat_interleave(128, 1)[:, :a.shape[1]]) @ (
        w.double() * sw.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :a.shape[1]]).t()
    tol = (1e-5 + (2.0**-8 if y.dtype == torch.bfloat16 else 0.0)) * ref.abs() + 1e-6  # all terms are positive
    assert ((y[rows].double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("each", [2, 300])
@pytest.mark.parametrize("N,K", [(4100, 4096), (4100, 4088)])
def test_weights_of_many_experts(each, N, K):
    """On the tensor cores, as they are and copied into scratch."""
    g, E = rng(4), 140
    w, a = codes(g, E, N, K), codes(g, E * each, K)
    sa, sw = torch.rand(E * each, 32, generator=g, device="cuda"), torch.rand(E, 33, 32, generator=g, device="cuda")
    offsets = torch.arange(E + 1, dtype=torch.int32, device="cuda") * each
    y = qg.qmm_fp8_b128_grouped(a, sa, w, sw, offsets)
    for e in (0, 1, 127, 128, 139):
        check(y, a, sa, w[e], sw[e], slice(e * each, e * each + each))
    assert qg.device_error() == 0


@pytest.mark.parametrize("N,ws", [(4104, None), (4100, None), (4100, 16)])
def test_rows_of_few_experts(N, ws):
    """Outputs past 2^31, by TMA stores, by single ones and (K = 136, without scratch) on the CUDA cores."""
    g, M, K = rng(5), 2**31 // 4100 + 300, 128 if ws is None else 136
    a, w = codes(g, M, K), codes(g, 3, N, K)
    kb = -(-K // 128)
    sa, sw = torch.rand(M, kb, generator=g, device="cuda"), torch.rand(3, 33, kb, generator=g, device="cuda")
    cut = [0, 1000, M - 259, M]
    offsets = torch.tensor(cut, dtype=torch.int32, device="cuda")
    none = torch.empty(ws, dtype=torch.uint8, device="cuda") if ws else None
    y = qg.qmm_fp8_b128_grouped(a, sa, w, sw, offsets, out_dtype=torch.bfloat16, workspace=none)
    for e, rows in ((0, slice(990, 1000)), (1, slice(1000, 1010)), (1, slice(M - 262, M - 259)), (2, slice(M - 259, M - 250)),
                    (2, slice(M - 3, M))):
        check(y, a, sa, w[e], sw[e], rows)
    assert qg.device_error() == 0
