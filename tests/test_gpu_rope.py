"""kv_append_rope against its definition in 64 bits.

The fraction of a turn is exact to 2^-32 and becomes an f32 number of half turns (2^-25): pi (2^-25 + 2^-31) of an angle; sine
and cosine are off by at most 2 units (2^-23) more: 3.6 x 2^-24. A value is two products of them, each rounded, and their sum:
6 x 2^-24 (|a| + |b|), then half a step of the cache's type. Values are copied: the same bits."""
import pytest
import torch

import bit_quantized_gemv_dequant_gb300 as qg

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}
TINY = {torch.float16: 2.0**-25, torch.bfloat16: 2.0**-134}


def rng(seed):
    return torch.Generator("cuda").manual_seed(seed)


def freqs(rot, base=10000.0):
    return torch.tensor([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float32, device="cuda")


def rotate(x, positions, inv_freq, inter):
    """(value, bound of its error in f32) of x [T, heads, D]."""
    angle = positions.double()[:, None] * inv_freq.double()
    n = inv_freq.numel()
    y, size = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    for i in range(n):
        f, s = (2 * i, 2 * i + 1) if inter else (i, i + n)
        a, b = x[:, :, f].double(), x[:, :, s].double()
        c, d = angle[:, i:i + 1].cos(), angle[:, i:i + 1].sin()
        y[:, :, f], y[:, :, s] = a * c - b * d, b * c + a * d
        size[:, :, f] = size[:, :, s] = a.abs() + b.abs()
    return y, size * 6 * 2.0**-24


def check(got, want, bound):
    tol = bound + want.abs() * HALF[got.dtype] + TINY[got.dtype]
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist())


class Case:
    def __init__(self, seed, T, Hq, Hkv, D, page, x="f32", dtype="bf16", rot=None, far=4096, skip=0.2):
        g = rng(seed)
        pages = -(-T // page) + 2
        self.qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device="cuda").to(DTYPES[x])
        self.q = self.qkv[:, :Hq] if Hq else None
        self.k, self.v = self.qkv[:, Hq:Hq + Hkv], self.qkv[:, Hq + Hkv:]
        self.kc, self.vc = (torch.randn(pages, Hkv, page, D, generator=g, device="cuda").to(DTYPES[dtype]) for _ in range(2))
        self.slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].clone()
        self.slots[torch.rand(T, generator=g, device="cuda") < skip] = -1
        self.positions = torch.randint(0, far, (T,), generator=g, device="cuda")
        self.freq = freqs(rot or D)
        self.page = page

    def run(self, inter=False, **more):
        return qg.kv_append_rope(self.q, self.k, self.v, self.positions, self.freq, self.kc, self.vc, self.slots,
                                 interleaved=inter, **more)

    def check(self, inter=False, **more):
        old_k, old_v = self.kc.clone(), self.vc.clone()
        out = self.run(inter, **more)
        if self.q is None:
            assert out is None
        else:
            assert out.dtype == self.kc.dtype and out.is_contiguous()
            check(out, *rotate(self.q, self.positions, self.freq, inter))
        live = self.slots >= 0
        at = self.slots[live]
        page, place = at // self.page, at % self.page
        want, bound = rotate(self.k, self.positions, self.freq, inter)
        check(self.kc[page, :, place], want[live], bound[live])
        assert torch.equal(self.vc[page, :, place], self.v[live].to(self.vc.dtype))
        # rows that no token has are as they were
        self.kc[page, :, place], self.vc[page, :, place] = old_k[page, :, place], old_v[page, :, place]
        assert torch.equal(self.kc, old_k) and torch.equal(self.vc, old_v)
        assert qg.device_error() == 0
        return out


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("x,dtype", [("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f16"), ("f32", "f16")])
@pytest.mark.parametrize("T,Hq,Hkv,D,page,rot", [(1, 8, 2, 128, 16, 128), (3, 4, 4, 64, 8, 64), (131, 5, 1, 128, 64, 64),
                                                 (37, 0, 2, 80, 32, 80), (700, 12, 3, 96, 16, 48), (9, 2, 1, 256, 8, 256),
                                                 (5, 3, 3, 8, 8, 8), (20, 7, 7, 64, 16, 2), (11, 2, 1, 64, 16, 26),
                                                 (2, 1, 1, 1024, 8, 1000), (6, 40, 8, 128, 256, 72)])
def test_rope(T, Hq, Hkv, D, page, rot, x, dtype, inter):
    Case(T * 3 + D, T, Hq, Hkv, D, page, x, dtype, rot).check(inter)


@pytest.mark.parametrize("inter", [False, True])
def test_far_positions(inter):
    """Angles of positions up to 2^31 and of either sign, at frequencies of every size."""
    c = Case(5, 300, 4, 2, 128, 16, far=2**31 - 1)
    c.positions[::3] *= -1
    c.positions[:4] = torch.tensor([0, 1, -1, 2**31 - 1], device="cuda")
    c.freq = torch.exp2(-torch.arange(64, device="cuda").float() * 0.6).contiguous()
    c.check(inter)
    c.freq = (torch.rand(64, generator=rng(6), device="cuda") * 8 - 4).contiguous()  # above 1 and below 0
    c.check(inter)
    c.freq[:3] = torch.tensor([0.0, 1e-40, 1e-30], device="cuda")
    c.check(inter)


def test_position_zero_is_a_copy():
    c = Case(7, 50, 4, 2, 64, 16)
    c.positions.zero_()
    out = c.check()
    assert torch.equal(out, c.q.to(out.dtype))


def test_rows_apart_and_unaligned():
    for shift in (0, 1, 4, 8):
        c = Case(8 + shift, 40, 4, 2, 64, 16, "bf16")
        flat = torch.empty(40 * (8 * 64 + 24) + 8, dtype=torch.bfloat16, device="cuda")
        wide = flat[shift:shift + 40 * (8 * 64 + 24)].view(40, 8 * 64 + 24)
        wide[:, :512] = c.qkv.reshape(40, 512)
        parts = wide[:, :512].unflatten(1, (8, 64))
        c.q, c.k, c.v = parts[:, :4], parts[:, 4:6], parts[:, 6:]
        c.check()
        c.check(True, q_out=torch.empty(40, 4, 64, dtype=torch.bfloat16, device="cuda"))


def test_slots_out_of_range_are_recorded():
    c = Case(9, 10, 2, 1, 64, 16, skip=0.0)
    old = c.kc.clone()
    good = c.slots.clone()
    c.slots[3] = c.kc.shape[0] * 16
    c.slots[7] = 2**62
    out = c.run()
    check(out, *rotate(c.q, c.positions, c.freq, False))  # q is rotated all the same
    assert qg.device_error() == 32
    live = torch.tensor([i for i in range(10) if i not in (3, 7)], device="cuda")
    at = good[live]
    want, bound = rotate(c.k, c.positions, c.freq, False)
    check(c.kc[at // 16, :, at % 16], want[live], bound[live])
    c.kc[at // 16, :, at % 16] = old[at // 16, :, at % 16]
    assert torch.equal(c.kc, old)


def test_the_same_cache_as_append():
    """With angles of 0 the call is kv_append."""
    c = Case(10, 77, 3, 2, 128, 32, "bf16")
    c.positions.zero_()
    k, v = c.kc.clone(), c.vc.clone()
    qg.kv_append(c.k, c.v, k, v, c.slots)
    c.run()
    assert torch.equal(c.kc, k) and torch.equal(c.vc, v)


def test_no_tokens_and_refusals():
    c = Case(11, 4, 2, 1, 64, 16)
    e = Case(11, 4, 2, 1, 64, 16)
    e.q, e.k, e.v, e.slots, e.positions = (t[:0] for t in (e.q, e.k, e.v, e.slots, e.positions))
    assert e.run().shape == (0, 2, 64)

    def call(**change):
        a = dict(q=c.q, k=c.k, v=c.v, positions=c.positions, inv_freq=c.freq, k_cache=c.kc, v_cache=c.vc, slots=c.slots)
        a.update(change)
        return qg.kv_append_rope(**a)

    call()
    for change in (dict(q=c.q[:3]), dict(q=c.q.half()), dict(v=c.v.half()), dict(positions=c.positions.int()),
                   dict(positions=c.positions[:3]), dict(inv_freq=c.freq.double()), dict(inv_freq=c.freq.view(2, 16)),
                   dict(v_cache=c.vc.half()), dict(slots=c.slots.int()), dict(q=None, q_out=c.q.bfloat16()),
                   dict(q_out=torch.empty(4, 2, 64, device="cuda")), dict(q_out=torch.empty(4, 1, 64, device="cuda").bfloat16()),
                   dict(k=c.k.cpu()), dict(q=c.q[:, :, :32])):
        with pytest.raises(ValueError):
            call(**change)
    for change in (dict(inv_freq=c.freq[:0]), dict(inv_freq=c.freq.repeat(2)),
                   dict(k_cache=c.kc.float(), v_cache=c.vc.float())):
        with pytest.raises(qg.QGError):
            call(**change)
