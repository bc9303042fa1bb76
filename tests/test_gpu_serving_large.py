"""The serving operators on tensors of more than 2^31 elements, so that offsets pass 32 bits: what lies at their ends
is held against the same call on a small copy of it, or against 64 bits where the small call may sum in another order.

Products over one block of 128 codes: 1e-5 * sum |terms| + 1e-6 and a bf16 rounding. Log probabilities: the difference
of two f32 results, each off by (V / 512 + 64 + 4 max|x|) 2^-24. Attention: the same steps of the same keys, cut over
as many CTAs, so the same bits."""
import pytest
import torch

import bit_quantized_gemv_dequant_gb300 as qg

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def i32(*a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def rng(seed):
    return torch.Generator("cuda").manual_seed(seed)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantizer(dtype):
    M, K = 2**31 // 4100 + 9, 4100
    x = torch.zeros(M, K, dtype=dtype, device="cuda")
    x[-9:] = torch.randn(9, K, generator=rng(1), device="cuda").to(dtype)
    codes, scales = qg.quantize_fp8_b128(x)
    c, s = qg.quantize_fp8_b128(x[-9:].clone())
    assert torch.equal(codes[-9:].view(torch.uint8), c.view(torch.uint8)) and torch.equal(scales[-9:], s)
    assert not codes[:-9].view(torch.uint8).any() and (scales[:-9] == 1).all()


def test_product():
    M, N, K = 2**31 // 4100 + 300, 4100, 128
    g = rng(2)
    a = torch.randint(0, 120, (M, K), generator=g, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
    w = torch.randint(0, 120, (N, K), generator=g, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
    sa = torch.rand(M, 1, generator=g, device="cuda")
    sw = torch.rand(-(-N // 128), 1, generator=g, device="cuda")
    y = qg.qmm_fp8_b128(a, sa, w, sw, out_dtype=torch.bfloat16)
    for rows in (slice(0, 3), slice(M // 2, M // 2 + 3), slice(M - 3, M)):
        ref = (a[rows].double() * sa[rows].double()) @ (w.double() * sw.double().repeat_interleave(128, 0)[:N]).t()
        assert ((y[rows].double() - ref).abs() <= (1e-5 + 2.0**-8) * ref.abs() + 1e-6).all()  # all terms are positive
    assert qg.device_error() == 0


@pytest.mark.parametrize("new,ctx", [([1, 1, 1], [1, 500, 77]), ([20, 1, 3], [300, 500, 3]), ([130, 1, 0], [400, 500, 20])])
def test_attention_and_append(new, ctx):
    hkv, page, d, hq = 2, 64, 128, 8
    pages = 2**31 // (hkv * page * d) + 40
    g = rng(3)
    big = [torch.zeros(pages, hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    small = [torch.zeros(40, hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = torch.randperm(40, generator=g, device="cuda").to(torch.int32)[:30].view(3, 10).contiguous()
    slots = torch.cat([torch.arange(n, device="cuda") % page + table[b].long().repeat_interleave(page)[:n] * page
                       for b, n in enumerate(ctx)])
    k, v = (torch.randn(sum(ctx), hkv, d, generator=g, device="cuda") for _ in range(2))
    qg.kv_append(k, v, *small, slots)
    qg.kv_append(k, v, *big, slots + (pages - 40) * page)
    for s, b in zip(small, big):
        assert torch.equal(b[-40:], s) and not b[:-40].any()
    q = torch.randn(sum(new), hq, d, generator=g, device="cuda").to(torch.bfloat16)
    off = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)
    rest = dict(max_new=max(new), return_lse=True)
    want = qg.attn_paged(q, *small, table, off, i32(*ctx), **rest)
    got = qg.attn_paged(q, *big, table + (pages - 40), off, i32(*ctx), **rest)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert qg.device_error() == 0


def test_pages():
    planes, pages, page = 3, 2**31 // (3 * 64 * 128) + 8, (64, 128)
    cache = torch.zeros(planes, pages, *page, dtype=torch.bfloat16, device="cuda")
    cache[:, -4:] = torch.randn(planes, 4, *page, generator=rng(4), device="cuda").to(torch.bfloat16)
    last = cache[:, -4:].clone()
    qg.kv_copy_pages(cache, i32(pages - 1, pages - 2), i32(0, pages - 5))
    assert torch.equal(cache[:, 0], last[:, 3]) and torch.equal(cache[:, -5], last[:, 2]) and torch.equal(cache[:, -4:], last)
    table, lens, refs = i32([0, pages - 3, pages - 4]), i32(3 * 64 - 10), torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[table.long()] = 1
    child, n, refs = qg.kv_fork(cache, table, lens, refs, i32(0), 64)
    want = torch.stack([last[:, 3], last[:, 1], last[:, 0]], 1)
    assert torch.equal(cache[:, child[0].long()][:, :2], want[:, :2])
    assert torch.equal(cache[:, child[0, 2].long(), :54], want[:, 2, :54]) and n.item() == lens.item()
    table = torch.cat([table, child])
    packed, refs, _, live = qg.kv_compact(cache, table, refs)
    assert live.item() == 4 and packed.max() == 3
    assert torch.equal(cache[:, packed[0].long()], want)
    assert qg.device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_log_probabilities(dtype):
    M, V = 2**31 // 50021 + 5, 50021
    x = torch.zeros(M, V, dtype=dtype, device="cuda")
    x[-4:] = (torch.randn(4, V, generator=rng(5), device="cuda") * 3).to(dtype)
    targets = torch.randint(0, V, (M,), generator=rng(6), device="cuda")
    got = qg.token_logprobs(x, targets, 7)
    want = qg.token_logprobs(x[-4:].clone(), targets[-4:], 7)
    tol = 2 * (V / 512 + 64 + 4 * float(x[-4:].float().abs().max())) * 2.0**-24
    for a, b in zip(got, want):
        if a.dtype.is_floating_point:
            assert ((a[-4:] - b).abs() <= (tol if a is not got[1] else 3 * tol * (1 + b))).all()
        else:
            assert torch.equal(a[-4:], b)
    assert (got[4][:-4] == torch.arange(7, device="cuda")).all() and (got[2][:-4] == 0).all()
    assert qg.device_error() == 0


@pytest.mark.parametrize("M,N", [(65535 * 128 + 1, 64), (3, 65535 * 128 + 1)])
@pytest.mark.parametrize("K,workspace", [(128, 0), (24, 0), (24, None)])
def test_product_of_more_tiles_than_a_grid_has_rows(M, N, K, workspace):
    """Few columns and millions of rows, and the reverse: on the tensor cores and, without a workspace, on the CUDA cores."""
    g = rng(7)
    a = torch.randint(0, 120, (M, K), generator=g, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
    w = torch.randint(0, 120, (N, K), generator=g, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
    sa = torch.rand(M, 1, generator=g, device="cuda")
    sw = torch.rand(-(-N // 128), 1, generator=g, device="cuda")
    none = torch.empty(16, dtype=torch.uint8, device="cuda") if workspace == 0 else None
    y = qg.qmm_fp8_b128(a, sa, w, sw, workspace=none)
    swn = sw.double().repeat_interleave(128, 0)[:N]
    m = torch.cat([torch.arange(0, M, 99991, device="cuda"), torch.arange(max(0, M - 300), M, device="cuda")])
    n = torch.cat([torch.arange(0, N, 99991, device="cuda"), torch.arange(max(0, N - 300), N, device="cuda")])
    ref = (a[m].double() * sa[m].double()) @ (w[n].double() * swn[n]).t()
    assert ((y[m][:, n].double() - ref).abs() <= 1e-5 * ref.abs() + 1e-6).all()  # all terms are positive
    assert qg.device_error() == 0
