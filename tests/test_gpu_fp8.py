"""quantize_fp8_b128 and qmm_fp8_b128 against their definitions in 64 bits.

Codes and scales are defined to the bit and compared so. A product's bound is
the f32 paths' 1e-5 * sum |terms| + 1e-6 and, for bf16 outputs, one rounding
(2^-8 of the value) more."""
import ctypes as C

import numpy as np
import pytest
import torch

import bit_quantized_gemv_dequant_gb300 as qg

pytestmark = pytest.mark.gpu


def workspace_bytes(*shape):
    n = C.c_size_t()
    assert qg.lib().qmm_fp8_b128_workspace_size(*shape, C.byref(n)) == 0
    return n.value


E4M3 = torch.float8_e4m3fn
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def rng(seed):
    return torch.Generator("cuda").manual_seed(seed)


def e4m3_table():
    """The 256 values, decoded from the bit fields."""
    c = np.arange(256)
    sign, e, f = np.where(c & 128, -1.0, 1.0), (c >> 3) & 15, c & 7
    v = np.where(e == 0, f * 2.0**-9, (8 + f) * 2.0 ** (e - 10.0)) * sign
    v[(c & 127) == 127] = np.nan
    return v


def quantize_ref(x):
    """(codes, scales) by search among the 127 magnitudes: the nearest one, of two equally near the even code."""
    x = x.float().cpu().numpy()
    M, K = x.shape
    KB = -(-K // 128)
    pad = np.zeros((M, KB * 128), np.float32)
    pad[:, :K] = x
    pad = pad.reshape(M, KB, 128)
    scales = np.abs(pad).max(2) / np.float32(448)
    scales[scales == 0] = 1
    q = (pad / scales[:, :, None]).astype(np.float32).astype(np.float64)
    mags = e4m3_table()[:127]
    hi = np.clip(np.searchsorted(mags, np.abs(q)), 1, 126)
    down, up = np.abs(q) - mags[hi - 1], mags[hi] - np.abs(q)
    code = np.where((down < up) | ((down == up) & ((hi - 1) % 2 == 0)), hi - 1, hi)
    code = np.where(np.signbit(q), code | 128, code).astype(np.uint8)
    return code.reshape(M, KB * 128)[:, :K], scales


def decode(codes):
    return torch.from_numpy(e4m3_table()).cuda()[codes.view(torch.uint8).long()]


def product_ref(a, sa, w, sw):
    """y and sum |terms| in 64 bits."""
    M, K = a.shape
    N = w.shape[0]
    av = decode(a) * sa.double().repeat_interleave(128, 1)[:, :K]
    wv = decode(w) * sw.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return av @ wv.t(), av.abs() @ wv.abs().t()


def codes_like(g, rows, cols):
    """Random finite codes of every exponent."""
    c = torch.randint(0, 254, (rows, cols), generator=g, device="cuda")
    return (c + (c >= 127)).to(torch.uint8).view(E4M3)


def scales_like(g, *shape):
    return torch.exp2(torch.rand(*shape, generator=g, device="cuda") * 12 - 9)


def check_product(y, a, sa, w, sw):
    ref, bound = product_ref(a, sa, w, sw)
    tol = 1e-5 * bound + 1e-6
    if y.dtype == torch.bfloat16:
        tol += ref.abs() * 2.0**-8
    bad = ((y.double() - ref).abs() > tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist())


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("M,K", [(1, 1), (1, 128), (3, 127), (2, 129), (5, 4096), (33, 1000), (130, 516)])
def test_quantize_to_the_bit(dtype, M, K):
    x = torch.randn(M, K, generator=rng(M * 7 + K), device="cuda") * 3
    x[0, : min(K, 128)] = 0  # a block of zeros
    x = x.to(DTYPES[dtype])
    codes, scales = qg.quantize_fp8_b128(x)
    rc, rs = quantize_ref(x)
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(codes.view(torch.uint8).cpu().numpy(), rc)


def test_quantize_every_tie_and_range():
    """Values on and next to every midpoint of two codes, from the smallest subnormal to the largest."""
    mags = e4m3_table()[:127]
    mid = (mags[1:] + mags[:-1]) / 2
    v = np.concatenate([mags, mid, np.nextafter(mid.astype(np.float32), np.float32(0)),
                        np.nextafter(mid.astype(np.float32), np.float32(1e9))]).astype(np.float32)
    v = np.concatenate([v, -v])
    rows = np.full((-(-v.size // 127), 128), 448.0, np.float32)  # the last of each block: scale 1
    rows[:, :127].ravel()[:] = 0
    flat = np.zeros(rows.shape[0] * 127, np.float32)
    flat[: v.size] = v
    rows[:, :127] = flat.reshape(-1, 127)
    x = torch.from_numpy(rows).cuda()
    codes, scales = qg.quantize_fp8_b128(x)
    assert (scales == 1).all()
    assert np.array_equal(codes.view(torch.uint8).cpu().numpy(), quantize_ref(x)[0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_of_any_magnitude(dtype):
    """Blocks from the smallest subnormal to the largest value, and scales whose significand is all ones or nearly:
    the quotient is the correctly rounded one, so the codes are those of a division."""
    g = torch.Generator().manual_seed(3)
    e = torch.randint(-149, 128, (3000,), generator=g).double()
    amax = torch.exp2(e) * (1 + torch.rand(3000, generator=g).double() * 0.999)
    amax[::3] = 448.0 * torch.exp2(e[::3].clamp(-140, 110)) * (2 - torch.randint(1, 5, (1000,), generator=g) * 2.0**-23)
    x = (torch.rand(3000, 128, generator=g).double() * 2 - 1) * amax[:, None]
    x[:, 5] = amax
    x[:, 64:] *= torch.exp2(-torch.rand(3000, 64, generator=g).double() * 12)
    x = x.clamp(-3.0e38, 3.0e38).to(torch.float32).cuda().to(DTYPES[dtype])
    codes, scales = qg.quantize_fp8_b128(x)
    rc, rs = quantize_ref(x)
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(codes.view(torch.uint8).cpu().numpy(), rc)


def test_quantize_strided_odd_and_nonfinite():
    base = torch.randn(6, 700, generator=rng(5), device="cuda")
    x = base[:, 3:3 + 261]
    codes, scales = qg.quantize_fp8_b128(x)
    rc, rs = quantize_ref(x)
    assert np.array_equal(scales.cpu().numpy(), rs) and np.array_equal(codes.view(torch.uint8).cpu().numpy(), rc)
    y = torch.ones(3, 300, device="cuda")
    y[0, 5], y[1, 200], y[2, 299] = float("nan"), float("inf"), float("-inf")
    codes, scales = qg.quantize_fp8_b128(y)
    s = scales.cpu().numpy()
    assert np.isnan(s[0, 0]) and np.isinf(s[1, 1]) and np.isinf(s[2, 2])
    assert np.isfinite(s).sum() == 6
    tiny = torch.full((1, 128), 1e-44, device="cuda")  # max / 448 underflows to 0: the scale is 1
    codes, scales = qg.quantize_fp8_b128(tiny)
    assert scales.item() == 1 and not codes.view(torch.uint8).any()


SHAPES = [(1, 1, 1), (1, 64, 16), (1, 128, 128), (2, 300, 272), (3, 1000, 4096), (8, 256, 144), (16, 130, 1040),
          (17, 129, 2064), (33, 512, 512), (64, 77, 640), (65, 640, 384), (127, 127, 256), (128, 4096, 128),
          (129, 257, 1168), (200, 2000, 4096), (513, 384, 528), (300, 260, 100), (5, 70, 333), (70, 5, 131),
          (1, 12288, 4096), (4, 4096, 12288)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K, out):
    g = rng(M + N + K)
    a, w = codes_like(g, M, K), codes_like(g, N, K)
    sa, sw = scales_like(g, M, -(-K // 128)), scales_like(g, -(-N // 128), -(-K // 128))
    y = qg.qmm_fp8_b128(a, sa, w, sw, out_dtype=DTYPES[out])
    check_product(y, a, sa, w, sw)
    assert qg.device_error() == 0


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (3, 130, 257), (40, 200, 515), (130, 300, 1000), (5, 70, 333)])
def test_product_of_odd_rows_with_and_without_workspace(M, N, K):
    """Rows of any number of bytes, through the workspace on the tensor cores and, without one, on the CUDA cores."""
    g = rng(M * N + K)
    a, w = codes_like(g, M, K), codes_like(g, N, K)
    sa, sw = scales_like(g, M, -(-K // 128)), scales_like(g, -(-N // 128), -(-K // 128))
    need = workspace_bytes(M, N, K)
    guarded = torch.full((need + 64,), 0x7F, dtype=torch.uint8, device="cuda")  # NaN codes around and in it
    check_product(qg.qmm_fp8_b128(a, sa, w, sw, workspace=guarded[:need]), a, sa, w, sw)
    assert (guarded[need:] == 0x7F).all()
    check_product(qg.qmm_fp8_b128(a, sa, w, sw, workspace=guarded[: need - 1]), a, sa, w, sw)
    assert qg.device_error() == 0


def test_product_unaligned_operands():
    g = rng(9)
    M, N, K = 37, 200, 512
    a8 = codes_like(g, 1, M * K + 16).view(torch.uint8).flatten()
    w8 = codes_like(g, 1, N * K + 16).view(torch.uint8).flatten()
    sa, sw = scales_like(g, M, 4), scales_like(g, 2, 4)
    for oa, ow in ((1, 0), (0, 4), (8, 3), (0, 0)):
        a, w = a8[oa:oa + M * K].view(E4M3).view(M, K), w8[ow:ow + N * K].view(E4M3).view(N, K)
        check_product(qg.qmm_fp8_b128(a, sa, w, sw), a, sa, w, sw)


def test_product_repeats_to_the_bit_and_rows_do_not_mix():
    g = rng(11)
    M, N, K = 48, 640, 4096
    a, w = codes_like(g, M, K), codes_like(g, N, K)
    sa, sw = scales_like(g, M, K // 128), scales_like(g, N // 128, K // 128)
    y = qg.qmm_fp8_b128(a, sa, w, sw)
    for _ in range(5):
        assert torch.equal(qg.qmm_fp8_b128(a, sa, w, sw), y)
    sa[7, 3] = float("nan")
    z = qg.qmm_fp8_b128(a, sa, w, sw)
    assert torch.isnan(z[7]).all()
    keep = torch.arange(M, device="cuda") != 7
    assert torch.equal(z[keep], y[keep])


def test_product_of_an_exact_case():
    """Small whole numbers and power-of-two scales: every order of the sum gives the same, exact, result."""
    g = rng(12)
    for M, N, K in ((3, 130, 256), (100, 260, 1024), (130, 300, 400)):
        vals = torch.randint(-3, 4, (M, K), generator=g, device="cuda").float()
        wals = torch.randint(-3, 4, (N, K), generator=g, device="cuda").float()
        sa = torch.exp2(torch.randint(-2, 3, (M, -(-K // 128)), generator=g, device="cuda").float())
        sw = torch.exp2(torch.randint(-2, 3, (-(-N // 128), -(-K // 128)), generator=g, device="cuda").float())
        a, w = vals.to(E4M3), wals.to(E4M3)
        ref, _ = product_ref(a, sa, w, sw)
        assert torch.equal(qg.qmm_fp8_b128(a, sa, w, sw).double(), ref)


def test_product_on_another_stream():
    g = rng(13)
    a, w = codes_like(g, 40, 1024), codes_like(g, 512, 1024)
    sa, sw = scales_like(g, 40, 8), scales_like(g, 4, 8)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y = qg.qmm_fp8_b128(a, sa, w, sw)
    s.synchronize()
    check_product(y, a, sa, w, sw)


def test_refusals():
    a = torch.zeros(4, 256, dtype=torch.uint8, device="cuda").view(E4M3)
    w = torch.zeros(130, 256, dtype=torch.uint8, device="cuda").view(E4M3)
    sa, sw = torch.ones(4, 2, device="cuda"), torch.ones(2, 2, device="cuda")
    qg.qmm_fp8_b128(a, sa, w, sw)
    for bad in ((a.view(torch.uint8), sa, w, sw), (a, sa[:, :1], w, sw), (a, sa, w[:, :128], sw), (a, sa, w, sw[:1]),
                (a, sa.double(), w, sw), (a.cpu(), sa, w, sw), (a[:, ::2], sa, w, sw)):
        with pytest.raises(ValueError):
            qg.qmm_fp8_b128(*bad)
    with pytest.raises(qg.QGError):
        qg.qmm_fp8_b128(a, sa, w, sw, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        qg.quantize_fp8_b128(torch.zeros(4, 4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        qg.quantize_fp8_b128(torch.zeros(4, 8, device="cuda")[:, ::2])
    with pytest.raises(qg.QGError):
        qg.quantize_fp8_b128(torch.zeros(0, 8, device="cuda"))
