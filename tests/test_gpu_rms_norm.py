"""rms_norm and rms_norm_fp8_b128 against their definition in 64 bits.

y = h s (o + w): h is one f32 sum (2^-24 of itself). The sum of K squares passes through at most K / 1024 + 16 + 10 additions
per value, half of whose relative error reaches s; the division, the sum with eps, the root, the reciprocal, two products
and o + w are one rounding each. That is (K / 2048 + 13 + 8) 2^-24, taken as (K / 2048 + 24) 2^-24 here, and half a step of the
output's type. The new residual is the f32 sum, rounded: the same bits. Codes and scales are those of the f32 output."""
import pytest
import torch

import bit_quantized_gemv_dequant_gb300 as qg

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {torch.float32: 2.0**-24, torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}
TINY = {torch.float32: 2.0**-140, torch.float16: 2.0**-25, torch.bfloat16: 2.0**-134}  # half a subnormal step


def rng(seed):
    return torch.Generator("cuda").manual_seed(seed)


def make(seed, M, K, x, res, w):
    g = rng(seed)
    size = torch.exp(torch.randn(M, 1, generator=g, device="cuda") * 2)
    t = (torch.randn(M, K, generator=g, device="cuda") * size).to(DTYPES[x])
    r = (torch.randn(M, K, generator=g, device="cuda") * size * 3).to(DTYPES[res]) if res else None
    v = (torch.randn(K, generator=g, device="cuda")).to(DTYPES[w]) if w else None
    return t, r, v


def ref(x, w, res, eps, offset):
    h = x.double() if res is None else x.double() + res.double()
    y = h / (h.square().mean(1, keepdim=True) + eps).sqrt()
    return y if w is None else y * (w.double() + offset)


def check(y, want, K):
    tol = (K / 2048 + 24) * 2.0**-24 + HALF[y.dtype]
    bad = (y.double() - want).abs() > want.abs() * tol + TINY[y.dtype]
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist())


def sum_of(x, res):
    return (x.float() + res.float()).to(res.dtype)


SHAPES = [(1, 1), (3, 7), (2, 8), (5, 127), (4, 128), (9, 264), (7, 512), (3, 513), (6, 520), (130, 1000), (17, 1024),
          (33, 4096), (3, 5201), (2, 12288), (5, 16384), (3, 16392), (2, 20001), (1, 70000)]


@pytest.mark.parametrize("x,res,w,out", [("bf16", "bf16", "bf16", "bf16"), ("f32", "f32", "f32", "f32"), ("f16", "f32", "f16", "f16"),
                                         ("bf16", "f32", "f32", "f32"), ("f32", "", "bf16", "bf16"), ("f16", "f16", "", "f32"),
                                         ("bf16", "", "f16", "f16")])
@pytest.mark.parametrize("M,K", SHAPES)
def test_norm(M, K, x, res, w, out):
    offset = float(K % 2)
    t, r, v = make(M * 3 + K, M, K, x, res, w)
    got = qg.rms_norm(t, v, r, eps=1e-5, weight_offset=offset, out_dtype=DTYPES[out])
    y, new = got if res else (got, None)
    assert y.dtype == DTYPES[out]
    check(y, ref(t, v, r, 1e-5, offset), K)
    if res:
        assert new.dtype == r.dtype and torch.equal(new, sum_of(t, r))
    assert qg.device_error() == 0


@pytest.mark.parametrize("x,res,w", [("bf16", "bf16", "bf16"), ("f32", "f32", "f32"), ("f16", "f32", "f32"), ("bf16", "", "")])
@pytest.mark.parametrize("M,K", SHAPES)
def test_codes_are_those_of_the_f32_norm(M, K, x, res, w):
    t, r, v = make(M * 5 + K, M, K, x, res, w)
    got = qg.rms_norm_fp8_b128(t, v, r, weight_offset=0.5)
    y = qg.rms_norm(t, v, r, weight_offset=0.5, out_dtype=torch.float32)
    if res:
        assert torch.equal(got[2], sum_of(t, r))
        y = y[0]
    codes, scales = qg.quantize_fp8_b128(y)
    assert torch.equal(got[0].view(torch.uint8), codes.view(torch.uint8)) and torch.equal(got[1], scales)


@pytest.mark.parametrize("K", [256, 250, 20000])
def test_residual_in_place_and_rows_apart(K):
    base = torch.randn(11, 3 * K + 5, generator=rng(K), device="cuda").bfloat16()
    x, r = base[:, 3:3 + K], base[:, K + 3:2 * K + 3].float()
    want_y, want_r = qg.rms_norm(x.contiguous(), None, r)
    y, new = qg.rms_norm(x, None, r, residual_out=r)
    assert new.data_ptr() == r.data_ptr() and torch.equal(new, want_r) and torch.equal(y, want_y)
    # a residual stream whose rows lie apart, updated in place; what lies between is left alone
    wide = torch.randn(11, 2 * K, generator=rng(1), device="cuda").bfloat16()
    before = wide.clone()
    part = wide[:, K:]
    want_c, want_s, want_r = qg.rms_norm_fp8_b128(x.contiguous(), None, part.contiguous())
    codes, scales, _ = qg.rms_norm_fp8_b128(x, None, part, residual_out=part)
    assert torch.equal(part, want_r) and torch.equal(wide[:, :K], before[:, :K])
    assert torch.equal(codes.view(torch.uint8), want_c.view(torch.uint8)) and torch.equal(scales, want_s)


def test_special_rows():
    x = torch.zeros(7, 300, device="cuda")
    x[1, 5], x[2, 299], x[3, 0] = float("nan"), float("inf"), 1e-30
    x[4] = 3.0
    x[5, 7] = float("-inf")
    y = qg.rms_norm(x, eps=1e-6)
    assert (y[0] == 0).all() and torch.isnan(y[1]).all()
    assert torch.isnan(y[2, 299]) and (y[2, :299] == 0).all() and torch.isnan(y[5, 7])  # finite / infinity, infinity / infinity
    check(y[3:5], ref(x[3:5], None, None, 1e-6, 0.0), 300)
    codes, scales = qg.rms_norm_fp8_b128(x, eps=1e-6)
    assert (scales[0] == 1).all() and not codes[0].view(torch.uint8).any()
    assert torch.isnan(scales[1]).all() and torch.isnan(codes[1].float()).all()
    assert torch.isnan(scales[2, 2]) and (scales[2, :2] == 1).all() and (scales[6] == 1).all()
    assert torch.isnan(qg.rms_norm(x[:1], eps=0.0)).all()  # 0 / 0


def test_alignments():
    """Every start and row stride: the same bits as from dense, aligned rows."""
    for K in (64, 1032):
        for dtype in (torch.bfloat16, torch.float32):
            base = torch.randn(4 * (K + 9) + 16, generator=rng(2), device="cuda").to(dtype)
            for start, stride in ((1, K), (0, K + 1), (8, K + 8), (3, K + 5)):
                x = base.as_strided((4, K), (stride, 1), start)
                w = torch.randn(K + 1, generator=rng(3), device="cuda")[1:]
                assert torch.equal(qg.rms_norm(x, w), qg.rms_norm(x.contiguous(), w.clone()))
                out = torch.empty(4 * K + 1, dtype=dtype, device="cuda")[1:].view(4, K)
                assert torch.equal(qg.rms_norm(x, w, out=out), qg.rms_norm(x.contiguous(), w.clone()))
                codes = torch.empty(4 * K + 1, dtype=torch.uint8, device="cuda")[1:].view(4, K).view(torch.float8_e4m3fn)
                got = qg.rms_norm_fp8_b128(x, w, codes=codes)[0]
                assert got.data_ptr() == codes.data_ptr()
                assert torch.equal(codes.view(torch.uint8), qg.rms_norm_fp8_b128(x.contiguous(), w.clone())[0].view(torch.uint8))


def test_no_rows_and_refusals():
    x, w = torch.ones(4, 256, device="cuda"), torch.ones(256, device="cuda")
    assert qg.rms_norm(x[:0], w).shape == (0, 256)
    c, s, r = qg.rms_norm_fp8_b128(x[:0], w, x[:0])
    assert c.shape == (0, 256) and s.shape == (0, 2) and r.shape == (0, 256)
    for call in (lambda: qg.rms_norm(x, w[:255]), lambda: qg.rms_norm(x, w.double()), lambda: qg.rms_norm(x.cpu(), w),
                 lambda: qg.rms_norm(x[:, ::2], w[::2].contiguous()), lambda: qg.rms_norm(x, w, x[:3]),
                 lambda: qg.rms_norm(x, w, residual_out=x), lambda: qg.rms_norm(x, w, x, residual_out=x.half()),
                 lambda: qg.rms_norm(x, w, out=x[:3]), lambda: qg.rms_norm(x, w, out_dtype=torch.int32),
                 lambda: qg.rms_norm(x, w, out_dtype=3), lambda: qg.rms_norm(x.int(), w), lambda: qg.rms_norm(x[0], w),
                 lambda: qg.rms_norm_fp8_b128(x, w, codes=torch.empty(4, 256, device="cuda")),
                 lambda: qg.rms_norm_fp8_b128(x, w, scales=torch.empty(4, 3, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: qg.rms_norm(x, w, eps=-1.0), lambda: qg.rms_norm(x, w, eps=float("nan")),
                 lambda: qg.rms_norm(x, w, x.half()), lambda: qg.rms_norm(x, w, weight_offset=float("nan")),
                 lambda: qg.rms_norm(x, w, out=x), lambda: qg.rms_norm(x, w, x.clone(), residual_out=x)):
        with pytest.raises(qg.QGError):
            call()
