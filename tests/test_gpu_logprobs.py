"""token_logprobs against log_softmax in 64 bits; ids and ranks exactly.

A sum of V exponentials in f32, in at most V / 512 + 64 steps one after the
other, is off by that many units of 2^-24; the difference to the maximum by one
unit of the logits' size: tol = (V / 512 + 64 + 4 max|x|) 2^-24. The entropy has
two such sums and a quotient: three times that, of 1 + its size."""
import math

import numpy as np
import pytest
import torch

import bit_quantized_gemv_dequant_gb300 as qg

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]


def check(x, targets, k):
    got = qg.token_logprobs(x, targets, k)
    picked, entropy, ranks, top, ids = (t.cpu() for t in got)
    M, V = x.shape
    xd, t = x.double().cpu(), targets.cpu()
    given = t >= 0
    at = t.clamp(min=0)[:, None]
    finite = xd[torch.isfinite(xd)]
    tol = (V / 512 + 64 + 4 * (float(finite.abs().max()) if finite.numel() else 0)) * 2.0**-24
    none = torch.isinf(xd).all(1)
    logp = torch.where(none[:, None], xd, torch.log_softmax(xd, 1))

    def close(a, b, tol):
        a = a.double()
        same = (a == b) | (torch.isnan(a) & torch.isnan(b))
        assert (same | ((a - b).abs() <= tol)).all(), (a - b).abs().max()

    close(picked, torch.where(given, logp.gather(1, at).squeeze(1), 0.0), tol)
    h = torch.where(none, 0.0, torch.special.entr(torch.exp(logp)).sum(1))
    close(entropy, h, 3 * tol * (1 + h))
    # NaN counts as the largest
    ordered = torch.where(torch.isnan(xd), math.inf, xd)
    over = (ordered > ordered.gather(1, at)) | (torch.isnan(xd) & ~torch.isnan(xd.gather(1, at)))
    assert torch.equal(ranks.long(), torch.where(given, over.sum(1), -1))
    n = min(k, V)
    assert top.shape == ids.shape == (M, n)
    order = np.lexsort((np.broadcast_to(np.arange(V), (M, V)), -ordered.numpy() + 0.0, ~torch.isnan(xd).numpy()))[:, :n]
    assert np.array_equal(ids.numpy(), order)
    close(top, logp.gather(1, torch.from_numpy(order.astype(np.int64))), tol)
    assert qg.device_error() == 0


def rows(seed, M, V, dtype, pad=0, spread=3.0):
    g = torch.Generator("cuda").manual_seed(seed)
    x = (torch.randn(M, V + pad, generator=g, device="cuda") * spread).to(dtype)
    return x[:, :V], torch.randint(0, V, (M,), generator=g, device="cuda")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,V,k", [(1, 1, 1), (1, 5, 32), (3, 31, 5), (2, 33, 32), (7, 257, 0), (5, 1000, 20), (1, 4095, 1),
                                   (1, 50021, 20), (4, 32003, 32), (40, 5000, 3), (200, 777, 7), (2, 151937, 8)])
def test_random_rows(M, V, k, dtype):
    check(*rows(M + V, M, V, dtype), k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad", [1, 3, 8, 64])
def test_padded_and_unaligned_rows(pad, dtype):
    x, t = rows(pad, 6, 1003, dtype, pad)
    check(x, t, 12)
    base = torch.randn(9 * 1024 + 5, device="cuda").to(dtype)
    for off in (1, 2, 3, 5):
        check(base[off:off + 9 * 1024].view(9, 1024)[:, :1000], t.new_zeros(9) + 17, 5)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [100, 20000])
def test_ties_go_to_the_lower_id(V, dtype):
    g = torch.Generator("cuda").manual_seed(V)
    x = torch.randint(-2, 3, (5, V), generator=g, device="cuda").to(dtype)
    x[0] = 0.0
    x[1, ::2] = -0.0
    x[1, 1::2] = 0.0
    check(x, torch.tensor([0, V - 1, 5, 7, -1], device="cuda"), 32)


@pytest.mark.parametrize("order", [1, -1])
def test_sorted_rows(order):
    """Ascending logits: every one is a new candidate for the top."""
    x = torch.linspace(-20, 20, 30000, device="cuda")[None].repeat(3, 1) * order
    check(x.contiguous(), torch.tensor([0, 15000, 29999], device="cuda"), 32)


@pytest.mark.parametrize("dtype", TYPES)
def test_masked_rows(dtype):
    for V in (64, 5000, 60000):
        x, t = rows(V, 8, V, dtype)
        x = x.clone()
        x[torch.rand(8, V, device="cuda") < 0.7] = -math.inf
        x[1] = -math.inf                      # nothing is left
        x[2] = -math.inf
        x[2, V - 1] = 1.5                     # one is left
        x[3, t[3]] = -math.inf                # the token itself is masked
        x[4, : V // 2] = torch.finfo(dtype).min  # masked by the type's lowest value
        x[5, V // 3:] = -math.inf
        t[6] = -1
        t[7] = -100
        check(x, t, 20)


def test_extremes():
    x = torch.zeros(4, 3000, device="cuda")
    x[0, 7] = 3e38
    x[0, 8:] = -3e38
    x[1, :10] = 1e4
    x[2] = torch.finfo(torch.float32).min
    x[3, 5] = float("nan")
    check(x, torch.tensor([7, 11, 3, 9], device="cuda"), 6)


def test_a_token_past_the_vocabulary_is_recorded():
    x, t = rows(1, 3, 100, torch.float32)
    good = qg.token_logprobs(x, t, 4)
    t2 = t.clone()
    t2[1] = 100
    got = qg.token_logprobs(x, t2, 4)
    assert qg.device_error() == 32
    assert got[0][1] == 0 and got[2][1] == -1
    assert torch.equal(got[0][[0, 2]], good[0][[0, 2]]) and torch.equal(got[4], good[4]) and torch.equal(got[1], good[1])


def test_offsets_past_32_bits():
    V, M = 1 << 20, 2100  # 2.2e9 logits: rows past 2^32 bytes and 2^31 elements
    x = torch.zeros(M, V, dtype=torch.bfloat16, device="cuda")
    x[M - 1, 12345] = 9.0
    x[M - 1, V - 1] = 8.0
    t = torch.zeros(M, dtype=torch.long, device="cuda")
    t[M - 1] = V - 1
    picked, entropy, ranks, top, ids = qg.token_logprobs(x, t, 2)
    s = V - 2 + math.exp(9) + math.exp(8)
    assert ids[M - 1].tolist() == [12345, V - 1] and ranks[M - 1] == 1
    assert abs(picked[M - 1].item() - (8 - math.log(s))) < 2e-4
    assert abs(entropy[0].item() - math.log(V)) < 2e-3 and ids[0].tolist() == [0, 1]


def test_repeats_to_the_bit_and_other_streams():
    for M, V in ((1, 50021), (300, 9001)):
        x, t = rows(M, M, V, torch.float32)
        a = qg.token_logprobs(x, t, 9)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            b = [qg.token_logprobs(x, t, 9) for _ in range(4)]
        s.synchronize()
        for r in b:
            assert all(torch.equal(p, q) for p, q in zip(a, r))


def test_nothing_to_do_and_refusals():
    x, t = rows(1, 3, 100, torch.float32)
    assert qg.token_logprobs(x[:0], t[:0], 3)[3].shape == (0, 3)
    for bad in ((x.cpu(), t, 1), (x.double(), t, 1), (x, t[:2], 1), (x, t.int(), 1), (x[:, ::2], t, 1), (x[0], t, 1)):
        with pytest.raises(ValueError):
            qg.token_logprobs(*bad)
    for k in (-1, 33):
        with pytest.raises((ValueError, RuntimeError)):
            qg.token_logprobs(x, t, k)


def adds(M, V, dtype):
    """The longest chain of f32 additions of a sum: in a chunk of 32 bytes, a thread's chunks of its share of the row
    (one of at most 8, at least 2 chunks each), 8 threads of a lane, 5 steps over the lanes, 3 over the shares."""
    n, parts = 32 // dtype.itemsize, 1
    while parts < 8 and M * parts * 2 <= 2 * torch.cuda.get_device_properties(0).multi_processor_count and V >= parts * 1024 * n:
        parts *= 2
    return n // 2 + -(-V // (256 * parts * n)) + 1 + 8 + 5 + 3


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kind", ["one at 10", "one at 18", "one at 18.7", "one at 19.5", "one at 22", "one at 40", "offset 30",
                                  "offset 1000", "offset 10000", "offset -10000", "masked 1000", "lowest -1000", "growing to 60"])
@pytest.mark.parametrize("M,V", [(128, 32000), (1, 50021), (400, 9001)])
def test_error_does_not_grow_with_the_logits(M, V, kind, dtype):
    """Rows that one logit dominates, and rows far from 0. With u = 2^-24, e = (adds + 8) u bounds the relative error of a
    sum of exponentials, each within 4 u and (d of size |d| rounded once) u |d|; H bounds the sums' mean |d|. A log
    probability is off by e and its own three roundings, an entropy by e (1 + mean |d|) for each of its two sums."""
    g = torch.Generator("cuda").manual_seed(V + len(kind))
    *what, size = kind.split()
    what, size = what[0], float(size)
    x = torch.randn(M, V, generator=g, device="cuda") * (1 if what == "one" else 3)
    if what == "one":
        x[torch.arange(M, device="cuda"), torch.randint(0, V, (M,), generator=g, device="cuda")] = size
    elif what == "growing":
        x = x / 3 + torch.arange(V, device="cuda") * (size / V)
    else:
        x = x + size
    x = x.to(dtype)
    hidden = torch.rand(M, V, generator=g, device="cuda") < 0.5
    if what == "masked":
        x[hidden] = -math.inf
    elif what == "lowest":
        x[hidden] = torch.finfo(dtype).min
    targets = torch.randint(0, V, (M,), generator=g, device="cuda")
    targets[::2] = x[::2].float().argmax(1)
    lp, h, _, top, _ = qg.token_logprobs(x, targets, 9)
    ref = torch.log_softmax(x.double(), 1)
    entropy = torch.special.entr(ref.exp()).sum(1)
    u = 2.0**-24
    e = (adds(M, V, dtype) + 8) * u
    want = ref.gather(1, targets[:, None]).squeeze(1)
    for got, exact in ((lp, want), (top, ref.sort(1, descending=True).values[:, :9])):
        room = e + u * (3 * exact.abs() + 2 * entropy.view(-1, *[1] * (exact.dim() - 1)))
        seen = ~torch.isinf(exact)
        assert torch.equal(torch.isinf(got), ~seen)
        assert ((got.double() - exact).abs() <= room)[seen].all(), float(((got.double() - exact).abs() - room)[seen].max())
        assert (got <= 0).all()
    assert ((h.double() - entropy).abs() <= 4 * e * (1 + entropy)).all(), float(((h.double() - entropy).abs() / (1 + entropy)).max() / e)
    assert (h >= 0).all() and qg.device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,V", [(1, 70), (3, 20000), (300, 3000)])
def test_logits_next_to_the_largest_numbers(M, V, dtype):
    """Logits whose multiple by log2(e) is out of range."""
    most = torch.finfo(dtype).max
    two = math.log(0.5)
    for fill, some, want in ((-most, None, -math.log(V)), (most, None, -math.log(V)), (0.0, most, two), (-most, 3.0, two),
                             (-most, most, two), (-math.inf, -most, two), (-math.inf, most, two), (-0.9 * most, 0.9 * most, two),
                             (0.8 * most, most, two), (-most, -0.8 * most, two)):
        x = torch.full((M, V), fill, dtype=dtype, device="cuda")
        if some is not None:
            x[:, [V // 3, V - 1]] = some
        targets = torch.full((M,), V - 1, device="cuda")
        targets[1::2] = 0
        lp, h, r, top, ids = qg.token_logprobs(x, targets, 2)
        tol = (adds(M, V, dtype) + 8) * 2.0**-24 + 3 * 2.0**-24 * abs(want)
        assert ((lp[::2] - want).abs() <= tol).all() and ((top - want).abs() <= tol).all()
        assert ((h + want).abs() <= 4 * tol * (1 - want)).all()
        assert (r[::2] == 0).all() and ids[0].tolist() == ([0, 1] if some is None else [V // 3, V - 1])
        if some is not None:  # -infinity where the difference passes f32's range
            away = torch.tensor(fill, dtype=dtype).double() - torch.tensor(some, dtype=dtype).double()
            assert torch.allclose(lp[1::2], away.float().cuda() + want, rtol=2.0**-20, atol=0.0)
    assert qg.device_error() == 0
