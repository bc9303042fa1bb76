"""qmm_fp8_b128_grouped against its definition in 64 bits: qmm_fp8_b128's bound, expert by expert."""
import ctypes as C

import pytest
import torch

import bit_quantized_gemv_dequant_gb300 as qg
from test_gpu_fp8 import E4M3, check_product, codes_like, product_ref, rng, scales_like

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


class Case:
    """Experts with counts[e] rows each, `before` rows before the first one's and `behind` after the last one's."""

    def __init__(self, seed, counts, N, K, before=0, behind=0):
        g = rng(seed)
        E, kb = len(counts), -(-K // 128)
        M = before + sum(counts) + behind
        self.a, self.sa = codes_like(g, M, K), scales_like(g, M, kb)
        self.w = codes_like(g, E * N, K).view(E, N, K)
        self.sw = scales_like(g, E, -(-N // 128), kb)
        at = [before]
        for n in counts:
            at.append(at[-1] + n)
        self.at = at
        self.offsets = torch.tensor(at, dtype=torch.int32, device="cuda")

    def run(self, **more):
        return qg.qmm_fp8_b128_grouped(self.a, self.sa, self.w, self.sw, self.offsets, **more)

    def check(self, y, experts=None):
        for e in range(len(self.at) - 1) if experts is None else experts:
            r = slice(self.at[e], self.at[e + 1])
            if self.at[e] < self.at[e + 1]:
                check_product(y[r], self.a[r], self.sa[r], self.w[e], self.sw[e])

    def full(self, out):
        """A y of sevens: rows that no expert has stay what they are."""
        return torch.full((self.a.shape[0], self.w.shape[1]), 7.0, dtype=DTYPES[out], device="cuda")


COUNTS = {
    "one row": [1], "one each": [1] * 9, "some empty": [0, 3, 0, 0, 1, 17, 0], "all empty": [0, 0, 0],
    "few": [1, 2, 5, 16, 3, 8], "around tiles": [15, 16, 17, 31, 32, 33, 63, 64, 65], "one long": [0, 300, 1, 2],
    "long": [127, 128, 129, 255, 256, 257, 40], "longer": [1000, 513], "many experts": [1, 0, 2] * 100,
}


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("N,K", [(128, 128), (1, 16), (300, 272), (257, 1040), (640, 4096), (130, 384)])
@pytest.mark.parametrize("counts", list(COUNTS))
def test_grouped(counts, N, K, out):
    n = COUNTS[counts]
    before, behind = (3, 5) if len(n) % 2 else (0, 0)
    c = Case(len(n) + N + K, n, N, K, before, behind)
    y = c.full(out)
    assert c.run(y=y).data_ptr() == y.data_ptr()
    c.check(y)
    assert (y[:c.at[0]] == 7).all() and (y[c.at[-1]:] == 7).all()
    assert qg.device_error() == 0


@pytest.mark.parametrize("counts", ["few", "some empty", "long", "around tiles"])
@pytest.mark.parametrize("N,K", [(130, 257), (70, 333), (256, 100), (3, 1)])
def test_odd_rows_with_and_without_workspace(counts, N, K):
    """Rows of any number of bytes, through the workspace on the tensor cores and, without one, on the CUDA cores."""
    c = Case(N + K, COUNTS[counts], N, K, 1, 2)
    E, M = len(COUNTS[counts]), c.a.shape[0]
    n = C.c_size_t()
    assert qg.lib().qmm_fp8_b128_grouped_workspace_size(M, E, N, K, C.byref(n)) == 0
    need = n.value
    guarded = torch.full((need + 64,), 0x7F, dtype=torch.uint8, device="cuda")  # NaN codes around and in it
    for ws in (guarded[:need], guarded[:need - 1], None):
        y = c.full("f32")
        c.run(y=y, workspace=ws)
        c.check(y)
        assert (y[:1] == 7).all() and (y[-2:] == 7).all()
    assert (guarded[need:] == 0x7F).all()
    assert qg.device_error() == 0


@pytest.mark.parametrize("counts", [[5, 0, 40], [200, 3, 300]])
def test_unaligned_operands(counts):
    c = Case(3, counts, 200, 512)
    M, E = sum(counts), len(counts)
    a8 = torch.empty(M * 512 + 16, dtype=torch.uint8, device="cuda")
    w8 = torch.empty(E * 200 * 512 + 16, dtype=torch.uint8, device="cuda")
    a, w = c.a.clone(), c.w.clone()
    for oa, ow in ((1, 0), (0, 4), (8, 3)):
        c.a, c.w = a8[oa:oa + a.numel()].view(E4M3).view_as(a), w8[ow:ow + w.numel()].view(E4M3).view_as(w)
        c.a.view(torch.uint8).copy_(a.view(torch.uint8))
        c.w.view(torch.uint8).copy_(w.view(torch.uint8))
        c.check(c.run())


@pytest.mark.parametrize("counts", [[3, 1, 0, 9], [70, 300, 0, 41]])
def test_experts_and_rows_do_not_mix(counts):
    c = Case(4, counts, 260, 2048)
    y = c.run()
    for _ in range(3):
        assert torch.equal(c.run(), y)
    c.sa[1, 3] = float("nan")
    c.sw[1, 1, 2] = float("nan")
    z = c.run()
    hit = torch.zeros(y.shape, dtype=torch.bool, device="cuda")
    hit[1] = True
    hit[c.at[1]:c.at[2], 128:256] = True
    assert torch.isnan(z[hit]).all() and torch.equal(z[~hit], y[~hit])


def test_an_exact_case():
    """Small whole numbers and power-of-two scales: every order of the sum gives the same, exact, result."""
    g = rng(12)
    for counts, N, K in (([2, 0, 7, 1], 130, 1024), ([100, 31, 280], 260, 1040), ([1] * 40, 129, 4096)):
        c = Case(1, counts, N, K)
        c.a = torch.randint(-3, 4, c.a.shape, generator=g, device="cuda").float().to(E4M3)
        c.w = torch.randint(-3, 4, c.w.shape, generator=g, device="cuda").float().to(E4M3)
        c.sa = torch.exp2(torch.randint(-2, 3, c.sa.shape, generator=g, device="cuda").float())
        c.sw = torch.exp2(torch.randint(-2, 3, c.sw.shape, generator=g, device="cuda").float())
        y = c.run()
        for e in range(len(counts)):
            r = slice(c.at[e], c.at[e + 1])
            if counts[e]:
                assert torch.equal(y[r].double(), product_ref(c.a[r], c.sa[r], c.w[e], c.sw[e])[0])


@pytest.mark.parametrize("M,N,K", [(40, 300, 1024), (700, 300, 1024)])
def test_one_expert_is_the_plain_product(M, N, K):
    c = Case(6, [M], N, K)
    y = c.run()
    check_product(y, c.a, c.sa, c.w[0], c.sw[0])
    check_product(qg.qmm_fp8_b128(c.a, c.sa, c.w[0], c.sw[0]), c.a, c.sa, c.w[0], c.sw[0])


@pytest.mark.parametrize("scale", [1, 30])
def test_bad_ranges_are_empty_and_recorded(scale):
    counts = [n * scale for n in (4, 3, 5, 2)]
    c = Case(7, counts, 200, 512)
    M = sum(counts)
    for i, bad in ((1, -5), (4, M + 1), (4, 2**31 - 1), (2, -2**31)):
        c.offsets = torch.tensor(c.at, dtype=torch.int32, device="cuda")
        c.offsets[i] = bad
        o = c.offsets.tolist()
        y = c.full("f32")
        c.run(y=y)
        assert qg.device_error() == 32
        none = torch.ones(M, dtype=torch.bool, device="cuda")
        for e in range(4):
            if 0 <= o[e] <= o[e + 1] <= M:
                none[o[e]:o[e + 1]] = False
                r = slice(o[e], o[e + 1])
                check_product(y[r], c.a[r], c.sa[r], c.w[e], c.sw[e])
        assert (y[none] == 7).all()
    assert qg.device_error() == 0


def test_no_rows_and_refusals():
    c = Case(8, [2, 3], 200, 256)
    e = Case(8, [0, 0], 200, 256)
    assert e.run().shape == (0, 200)
    args = [c.a, c.sa, c.w, c.sw, c.offsets]
    for i, bad in ((0, c.a.view(torch.uint8)), (0, c.a.cpu()), (0, c.a[:, :128]), (1, c.sa[:, :1].contiguous()), (2, c.w[0]),
                   (2, c.w[:1]), (3, c.sw[:, :1].contiguous()), (3, c.sw.double()), (4, c.offsets.long()), (4, c.offsets[:2])):
        changed = list(args)
        changed[i] = bad
        with pytest.raises(ValueError):
            qg.qmm_fp8_b128_grouped(*changed)
    with pytest.raises(ValueError):
        c.run(y=torch.empty(5, 199, device="cuda"))
    with pytest.raises(qg.QGError):
        c.run(out_dtype=torch.float16)
    with pytest.raises(qg.QGError):
        qg.qmm_fp8_b128_grouped(c.a, c.sa, torch.empty(1025, 1, 256, device="cuda").to(E4M3), torch.ones(1025, 1, 2, device="cuda"),
                                torch.zeros(1026, dtype=torch.int32, device="cuda"))
