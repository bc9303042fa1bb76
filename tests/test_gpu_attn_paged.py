"""attn_paged against softmax attention in 64 bits.

With u the unit roundoff of the operands' type, S a bound of the scores'
magnitudes and A = sum_j p_j |v_j|, an output may be off by u A for the
probabilities' rounding and u |out| for its own, doubled, 1e-5 (1 + S) A for
the f32 scores and sums, and 2^-24 n max|v| for f16 probabilities below its
normal range; the log-sum by 1e-5 (1 + S)."""
import ctypes as C
import math

import pytest
import torch

import bit_quantized_gemv_dequant_gb300 as qg

pytestmark = pytest.mark.gpu


def workspace_bytes(*shape):
    n = C.c_size_t()
    assert qg.lib().attn_paged_workspace_size(*shape, C.byref(n)) == 0
    return n.value


UNIT = {torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}


def make(seed, new, ctx, hq, hkv, d, page, dtype, strided=False, spare=3):
    """A cache whose unused places are NaN, its pages in random order."""
    g = torch.Generator("cuda").manual_seed(seed)
    counts = [-(-t // page) for t in ctx]
    n = sum(counts) + spare
    order = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    k = torch.full((n, hkv, page, d), float("nan"), dtype=dtype, device="cuda")
    v = k.clone()
    table = torch.full((len(ctx), max(max(counts), 1) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, (c, t) in enumerate(zip(counts, ctx)):
        for i in range(c):
            p = int(order[at + i])
            table[b, i] = p
            fill = min(page, t - i * page)
            k[p, :, :fill] = torch.randn(hkv, fill, d, generator=g, device="cuda").to(dtype)
            v[p, :, :fill] = torch.randn(hkv, fill, d, generator=g, device="cuda").to(dtype)
        at += c
    off = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)
    q = torch.randn(sum(new), hq + (2 * hkv if strided else 0), d, generator=g, device="cuda").to(dtype)[:, :hq]
    return q, k, v, table, off, torch.tensor(ctx, dtype=torch.int32, device="cuda")


def reference(q, k, v, table, off, ctx, scale, softcap, window):
    T, hq, d = q.shape
    hkv, page = k.shape[1], k.shape[2]
    out = torch.zeros(T, hq, d, dtype=torch.float64, device="cuda")
    mass, lse = torch.zeros_like(out), torch.full((T, hq), -math.inf, dtype=torch.float64, device="cuda")
    s_max = v_max = 0.0
    offs = off.tolist()
    for b, n in enumerate(ctx.tolist()):
        c = offs[b + 1] - offs[b]
        if not c or not n:
            continue
        pages = table[b, : -(-n // page)].long()
        kk = k[pages].double().transpose(0, 1).reshape(hkv, -1, d)[:, :n].repeat_interleave(hq // hkv, 0)
        vv = v[pages].double().transpose(0, 1).reshape(hkv, -1, d)[:, :n].repeat_interleave(hq // hkv, 0)
        qq = q[offs[b]:offs[b + 1]].double().transpose(0, 1)
        s = qq @ kk.transpose(1, 2) * scale
        s_max = max(s_max, float((qq.abs() @ kk.abs().transpose(1, 2)).max()) * abs(scale))
        v_max = max(v_max, float(vv.abs().max()))
        if softcap:
            s = softcap * torch.tanh(s / softcap)
        pos = torch.arange(n - c, n, device="cuda")[:, None]
        j = torch.arange(n, device="cuda")[None, :]
        hide = (j > pos) | (j <= pos - window if window else False)
        s = s.masked_fill(hide, -math.inf)
        top = s.amax(2, keepdim=True).clamp(min=-1e300)
        e = torch.exp(s - top)
        z = e.sum(2, keepdim=True)
        p = torch.where(z > 0, e / z, 0.0)
        out[offs[b]:offs[b + 1]] = (p @ vv).transpose(0, 1)
        mass[offs[b]:offs[b + 1]] = (p @ vv.abs()).transpose(0, 1)
        lse[offs[b]:offs[b + 1]] = (top + torch.log(z)).squeeze(2).transpose(0, 1)
    return out, mass, lse, s_max, v_max


def check(args, scale=None, softcap=0.0, window=0, max_new=None):
    q, ctx = args[0], args[5]
    scale = q.shape[2] ** -0.5 if scale is None else scale
    out, lse = qg.attn_paged(*args, max_new=max_new, scale=scale, softcap=softcap, window=window, return_lse=True)
    assert qg.device_error() == 0
    ref, mass, rl, S, vm = reference(*args, scale, softcap, window)
    u, n = UNIT[q.dtype], int(ctx.max()) if ctx.numel() else 0
    tol = (2 * u + 1e-5 * (1 + S)) * mass + 2 * u * ref.abs() + 2.0**-24 * n * vm
    bad = ~((out.double() - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse), empty) and (out[empty] == 0).all()
    assert ((lse.double() - rl)[~empty].abs() <= 1e-5 * (1 + S)).all()
    return out


HEADS = [(1, 1), (4, 1), (8, 2), (6, 2), (20, 4), (32, 8), (9, 9), (32, 1)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_single_tokens(hq, hkv, d, dtype):
    ctx = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 1025]
    check(make(hq * d, [1] * len(ctx), ctx, hq, hkv, d, 16, dtype), max_new=1)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("d", [64, 128])
def test_pages_and_ragged_chunks(page, d):
    new = [1, 0, 5, 64, 17, 130, 257, 1, 300]
    ctx = [1, 40, 5, 100, 1000, 130, 500, 700, 2000]
    check(make(page + d, new, ctx, 8, 2, d, page, torch.bfloat16))


@pytest.mark.parametrize("hq,hkv", HEADS)
def test_chunk_heads(hq, hkv):
    check(make(hq, [70, 3, 129], [70, 300, 1000], hq, hkv, 128, 32, torch.float16))


def test_many_queries_per_key_head():
    check(make(3, [1, 2, 9], [100, 50, 300], 128, 1, 64, 16, torch.bfloat16))


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 100, 129, 5000])
@pytest.mark.parametrize("softcap", [0.0, 5.0, 30.0])
def test_window_and_cap(window, softcap):
    check(make(window, [1, 1, 200, 70, 513], [1, 900, 200, 400, 1500], 8, 2, 64, 16, torch.float16), softcap=softcap,
          window=window)


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 0.02])
def test_scale(scale):
    check(make(7, [1, 40, 300], [333, 40, 900], 4, 4, 64, 32, torch.bfloat16), scale=scale)


def test_rows_that_see_nothing():
    """More new tokens than keys: the first rows sit before the first key."""
    args = list(make(8, [3, 5, 1, 140], [3, 5, 1, 140], 8, 2, 128, 16, torch.bfloat16))
    args[5] = torch.tensor([1, 0, 0, 100], dtype=torch.int32, device="cuda")
    out = check(tuple(args))
    assert (out[:2] == 0).all() and (out[3:9] == 0).all() and (out[9:9 + 40] == 0).all()


def test_strided_queries_and_rows_past_the_last():
    args = make(9, [2, 130, 1], [20, 600, 90], 8, 2, 128, 16, torch.bfloat16, strided=True)
    assert not args[0].is_contiguous()
    check(args)
    q = torch.cat([args[0], args[0][:5]])
    out = torch.full((q.shape[0], 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    qg.attn_paged(q, *args[1:], out=out)
    assert (out[-5:] == 7).all() and torch.equal(out[:-5], qg.attn_paged(*args))


def test_large_scores():
    """Scores to +-1000 that grow along the keys: the running maximum moves at every step."""
    args = make(10, [1, 1, 200], [700, 2000, 900], 4, 2, 64, 16, torch.float16)
    q, k, v, table, off, ctx = args
    k = k * 20
    check((q, k, v, table, off, ctx), scale=1.0)
    page = k.shape[2]
    for b, n in enumerate(ctx.tolist()):
        for i in range(-(-n // page)):
            k[int(table[b, i])] = q[0, 0] * 0 + (torch.arange(page, device="cuda") + i * page).half()[None, :, None] / 500
    q.fill_(1.0)
    check((q, k, v, table, off, ctx), scale=1.0)


def test_long_context_and_offsets_past_32_bits():
    """A cache of over 2^32 bytes per side: the pages used are its last ones."""
    page, hkv, d = 256, 8, 128
    n = (1 << 32) // (page * hkv * d * 2) + 40
    k = torch.empty(n, hkv, page, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    g = torch.Generator("cuda").manual_seed(1)
    table = torch.arange(n - 1, n - 37, -1, device="cuda", dtype=torch.int32).view(1, 36)
    k[-36:] = torch.randn(36, hkv, page, d, generator=g, device="cuda").bfloat16()
    v[-36:] = torch.randn(36, hkv, page, d, generator=g, device="cuda").bfloat16()
    for new, ctx in ((1, 9001), (150, 9216)):
        q = torch.randn(new, 16, d, generator=g, device="cuda").bfloat16()
        check((q, k, v, table, torch.tensor([0, new], dtype=torch.int32, device="cuda"),
               torch.tensor([ctx], dtype=torch.int32, device="cuda")))


def test_repeats_to_the_bit_on_another_stream_and_in_a_graph():
    args = make(11, [1, 1, 1, 90], [4000, 100, 2500, 1200], 32, 8, 128, 64, torch.bfloat16)
    a = qg.attn_paged(*args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = qg.attn_paged(*args)
        out = torch.empty_like(a)
        need = workspace_bytes(93, 4, 93, 32, 8, 128)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            qg.attn_paged(*args, out=out, workspace=ws)
    s.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, out)


def test_bad_indexes_are_recorded_and_not_followed():
    for new, ctx in (([1, 1], [300, 300]), ([130, 64], [300, 300])):
        args = make(12, new, ctx, 8, 2, 64, 16, torch.bfloat16)
        good = qg.attn_paged(*args)
        table = args[3].clone()
        table[0, 3] = 10**6
        table[0, 5] = -5
        out = qg.attn_paged(*args[:3], table, *args[4:])
        assert qg.device_error() == 32
        assert torch.equal(out[new[0]:], good[new[0]:]) and torch.isfinite(out.float()).all()
        long = args[5].clone()
        long[1] = 10**6  # more keys than the table has room for
        out = qg.attn_paged(*args[:5], long)
        assert qg.device_error() == 32 and torch.equal(out[:new[0]], good[:new[0]])
        off = args[4].clone()
        off[2] = 10**6
        qg.attn_paged(*args[:4], off, args[5])
        assert qg.device_error() == 32
    args = make(13, [5, 2], [50, 50], 8, 2, 64, 16, torch.bfloat16)
    qg.attn_paged(*args, max_new=3)
    assert qg.device_error() == 32


@pytest.mark.parametrize("new", [[1, 1], [150, 2]])
def test_a_nan_reaches_its_rows_and_no_others(new):
    """A NaN in a visible key, value or query: NaN in the rows that see it (out and lse), the others unchanged."""
    args = make(15, new, [300, 300], 4, 2, 64, 16, torch.bfloat16)
    q, k, v, table, off, ctx = args
    good, glse = qg.attn_paged(*args, return_lse=True)
    k[int(table[0, 2]), 1, 3] = float("nan")  # key 35 of sequence 0, key head 1
    out, lse = qg.attn_paged(*args, return_lse=True)
    assert torch.isnan(out[:new[0], 2:].float()).all() and torch.isnan(lse[:new[0], 2:]).all()
    assert torch.equal(out[:new[0], :2], good[:new[0], :2]) and torch.equal(lse[:new[0], :2], glse[:new[0], :2])
    assert torch.equal(out[new[0]:], good[new[0]:])
    assert qg.device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("page", [8, 64, 256])
@pytest.mark.parametrize("window", [1, 60, 129, 300])
@pytest.mark.parametrize("new", [[1, 1, 1], [7, 1, 12], [150, 2, 129]])
def test_what_lies_before_every_window_may_be_anything(new, window, page, dtype):
    """Pages that no new token sees have left the table, and their last places before a window are NaN."""
    ctx = [700, 1500, 140]
    args = make(16, new, ctx, 8, 2, 64, page, dtype)
    good = check(args, window=window)
    q, k, v, table, off, lens = args
    for b, (n, c) in enumerate(zip(new, ctx)):
        begin = max(0, c - n + 1 - window)
        for i in range(begin // page):
            table[b, i] = -1 if i % 2 else 1 << 30
        if begin % page:
            for x in (k, v):
                x[int(table[b, begin // page]), :, :begin % page] = float("nan")
    got = qg.attn_paged(*args, window=window)
    assert torch.equal(got, good) and qg.device_error() == 0


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("softcap,window", [(0.0, 0), (20.0, 90)])
@pytest.mark.parametrize("d,dtype", [(64, torch.float16), (128, torch.bfloat16)])
@pytest.mark.parametrize("new,ctx", [([5, 1], [300, 300]), ([2, 3, 4] * 30, [200] * 90), ([40, 3], [90, 40]),
                                     ([150, 1], [150, 700]), ([600, 200, 1], [1000, 200, 3])])
def test_values_that_are_not_finite_reach_the_rows_that_see_them(new, ctx, d, dtype, softcap, window, value):
    """One value of one key among the new tokens: its column of the rows that see it, and nothing else."""
    args = make(17, new, ctx, 8, 2, d, 16, dtype)
    q, k, v, table, off, lens = args
    kw = dict(scale=d ** -0.5, softcap=softcap, window=window)
    finite = v.clone()
    spots = []
    for b, (n, c) in enumerate(zip(new, ctx)):
        if n > 1:
            j = c - n + (2 * n) // 3  # two thirds of the new tokens are before it
            finite[int(table[b, j // 16]), 1, j % 16, 5] = 0.0
            v[int(table[b, j // 16]), 1, j % 16, 5] = value
            spots.append((b, j))
    ref, mass, rl, S, vm = reference(q, k, finite, *args[3:], d ** -0.5, softcap, window)
    out, lse = qg.attn_paged(*args, return_lse=True, **kw)
    sees = torch.zeros(ref.shape, dtype=torch.bool, device="cuda")
    for b, j in spots:
        for i in range(new[b]):
            pos = ctx[b] - new[b] + i
            if pos >= j and (not window or j > pos - window):
                sees[int(off[b]) + i, 4:, 5] = True
    if value != value:
        assert torch.isnan(out[sees].float()).all()
    else:
        assert (out[sees] == value).all()
    u = UNIT[dtype]
    tol = (2 * u + 1e-5 * (1 + S)) * mass + 2 * u * ref.abs() + 2.0**-24 * max(ctx) * vm
    assert ((out.double() - ref).abs() <= tol)[~sees].all()
    assert ((lse.double() - rl).abs() <= 1e-5 * (1 + S)).all()
    assert qg.device_error() == 0


@pytest.mark.parametrize("softcap", [0.5, 30.0, 1000.0])
@pytest.mark.parametrize("scale", [0.125, -1.0])
@pytest.mark.parametrize("new", [1, 600])
def test_capped_scores_are_as_exact_as_their_size(new, scale, softcap):
    """With a window of one key the log sum is the score itself: products from 2^-24 to 2^14, exact in f32, of either
    sign. tanh is good to 5 units of 2^-24, and seven roundings (two constants, the products, the change of base) come
    on top: 12 units of the score."""
    n = 1200
    g = torch.Generator("cuda").manual_seed(18)
    sizes = torch.arange(n, device="cuda") % 38 - 24
    a = torch.ldexp(torch.randint(64, 128, (n,), generator=g, device="cuda") / 64.0, sizes // 2)
    b = torch.ldexp(torch.randint(64, 128, (n,), generator=g, device="cuda") / 64.0, sizes - sizes // 2)
    b = torch.where(torch.arange(n, device="cuda") % 3 == 0, -b, b)
    q = torch.zeros(n, 1, 64, dtype=torch.float16, device="cuda")
    k = torch.zeros(n // 16, 1, 16, 64, dtype=torch.float16, device="cuda")
    q[:, 0, 7] = a.half()
    k.view(n, 64)[:, 7] = b.half()
    assert torch.equal(q[:, 0, 7].double(), a.double()) and torch.equal(k.view(n, 64)[:, 7].double(), b.double())
    v = torch.randn(n // 16, 1, 16, 64, generator=g, device="cuda").half()
    pages = torch.arange(n // 16, dtype=torch.int32, device="cuda")
    if new == 1:  # n sequences of one token, whose windows end at keys 0, 1, 2 ...
        args = (q, k, v, pages.expand(n, -1).contiguous(), torch.arange(n + 1, dtype=torch.int32, device="cuda"),
                torch.arange(1, n + 1, dtype=torch.int32, device="cuda"))
    else:
        # two sequences of 600 tokens, 37 and a half pages each
        k2, v2 = (x.view(n, 64)[new:] for x in (k, v))
        fill = torch.zeros(8, 64, dtype=torch.float16, device="cuda")
        k = torch.cat([k.view(n, 64)[:new], fill, k2, fill]).view(-1, 1, 16, 64)
        v = torch.cat([v.view(n, 64)[:new], fill, v2, fill]).view(-1, 1, 16, 64)
        args = (q, k, v, torch.arange(76, dtype=torch.int32, device="cuda").view(2, 38),
                torch.tensor([0, new, n], dtype=torch.int32, device="cuda"),
                torch.tensor([new, n - new], dtype=torch.int32, device="cuda"))
    out, lse = qg.attn_paged(*args, max_new=new, scale=scale, softcap=softcap, window=1, return_lse=True)
    want = softcap * torch.tanh(scale * a.double() * b.double() / softcap)
    assert ((lse[:, 0].double() - want).abs() <= 12 * 2.0**-24 * want.abs()).all()
    rows = v.view(-1, 64)
    assert torch.equal(out.view(n, 64), rows if new == 1 else torch.cat([rows[:new], rows[608:608 + n - new]]))
    assert qg.device_error() == 0


def test_nothing_to_do_and_refusals():
    q, k, v, table, off, ctx = make(14, [2, 3], [20, 30], 8, 2, 64, 16, torch.bfloat16)
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert qg.attn_paged(q[:0], k, v, table, none, ctx).shape == (0, 8, 64)
    ok = (q, k, v, table, off, ctx)

    def swap(i, t):
        return ok[:i] + (t,) + ok[i + 1:]

    for bad in (swap(0, q.float()), swap(1, k.half()), swap(2, v[:, :, ::2]), swap(3, table.long()), swap(4, off[:2]),
                swap(5, ctx[:1]), swap(5, ctx.cpu()), swap(2, v[:, :1].contiguous())):
        with pytest.raises((ValueError, qg.QGError)):
            qg.attn_paged(*bad)
    for kw in (dict(softcap=-1.0), dict(window=-1), dict(scale=float("nan")), dict(max_new=-1)):
        with pytest.raises(qg.QGError):
            qg.attn_paged(*ok, **kw)
    with pytest.raises(qg.QGError):  # 8 query heads on 3 key heads
        qg.attn_paged(q, k[:, :1].repeat(1, 3, 1, 1), v[:, :1].repeat(1, 3, 1, 1), table, off, ctx)
    with pytest.raises(qg.QGError):  # a page size of 24
        qg.attn_paged(q, k.repeat(1, 1, 3, 1)[:, :, :24].contiguous(), v.repeat(1, 1, 3, 1)[:, :, :24].contiguous(),
                      table, off, ctx)
    with pytest.raises(qg.QGError):  # out over q
        qg.attn_paged(*ok, out=q)


@pytest.mark.parametrize("new,ctx", [([4, 1, 3], [1, 500, 30]), ([90, 4, 30], [20, 1, 700])])
def test_windows_longer_than_any_context(new, ctx):
    """They hide nothing, also where rows sit far before the first key."""
    args = list(make(16, [min(n, t) for n, t in zip(new, ctx)], ctx, 8, 2, 64, 16, torch.bfloat16))
    g = torch.Generator("cuda").manual_seed(17)
    args[0] = torch.randn(sum(new), 8, 64, generator=g, device="cuda").bfloat16()
    args[4] = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)
    want, wlse = qg.attn_paged(*args, return_lse=True)
    most = args[3].shape[1] * 16
    for window in (most - 1, most, most + 1, 2**31 - 2, 2**31 - 1, 2**31, 2**40, 2**63 - 1):
        out = check(tuple(args), window=window)
        assert torch.equal(out, want), window
        assert torch.equal(qg.attn_paged(*args, window=window, return_lse=True)[1], wlse), window


def test_no_new_tokens_allowed():
    """max_new = 0: sequences with new tokens are recorded, nothing is written; without any it is an empty step."""
    args = make(18, [2, 1], [20, 40], 8, 2, 64, 16, torch.bfloat16)
    out = torch.full((3, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    qg.attn_paged(*args, out=out, max_new=0)
    assert qg.device_error() == 32 and (out == 7).all()
    qg.attn_paged(*args[:4], torch.zeros_like(args[4]), args[5], out=out, max_new=0)
    assert qg.device_error() == 0 and (out == 7).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,new", [(8, 1, 1), (4, 4, 1), (12, 4, 2), (4, 2, 4), (2, 2, 8)])
def test_few_rows_are_as_exact_as_their_rounding(hq, hkv, new, d, dtype):
    """Up to 8 rows per key head: the output is a rounding of a number that is off by 2^-16 (probabilities) + 1e-5 (1 + S)
    (scores and sums) of A = sum_j p_j |v_j|, and 2^-24 n max|v| below f16's normal range: what its distance from the
    exact one exceeds half the spacing of the type's numbers there by. (A is often many times the output.)"""
    ctx = [8, 9, 13, 20, 33, 70, 150, 700]
    args = list(make(19, [new] * len(ctx), ctx, hq, hkv, d, 16, dtype))
    args[0] = args[0] * 0.1
    out = qg.attn_paged(*args, max_new=new)
    ref, mass, _, S, vm = reference(*args, d**-0.5, 0.0, 0)
    # numbers from 2^e to 2^(e + 1) are 2^e ulp apart, and the reference may round up to the next 2^e
    exponent = torch.frexp(torch.maximum(out.double().abs(), ref.abs())).exponent - 1
    spacing = torch.ldexp(torch.full_like(ref, 2 * UNIT[dtype]), exponent)
    if dtype == torch.float16:
        spacing = spacing.clamp(min=2.0**-24)
    beyond = (out.double() - ref).abs() - spacing / 2
    room = (2.0**-16 + 1e-5 * (1 + S)) * mass + (2.0**-24 * max(ctx) * vm if dtype == torch.float16 else 0.0)
    assert (beyond <= room).all(), float((beyond - room).max())
    assert qg.device_error() == 0


@pytest.mark.parametrize("hq,hkv", [(8, 2), (32, 2)])
def test_infinite_values_stay_infinite(hq, hkv):
    args = make(20, [1, 1], [40, 300], hq, hkv, 64, 16, torch.bfloat16)
    good = qg.attn_paged(*args, max_new=1)
    v, table = args[2], args[3]
    v[int(table[0, 1]), 1, 3, 5], v[int(table[1, 2]), 0, 7, 9] = math.inf, -math.inf
    out, group = qg.attn_paged(*args, max_new=1), hq // hkv
    assert (out[0, group:, 5] == math.inf).all() and (out[1, :group, 9] == -math.inf).all()
    same = torch.ones_like(out, dtype=torch.bool)
    same[0, group:, 5] = same[1, :group, 9] = False
    assert torch.equal(out[same], good[same])


@pytest.mark.parametrize("scale", [64**-0.5, 128**-0.5, 0.1, 0.3, 0.7, 0.011, 1.7, 3.1, 0.0475])
@pytest.mark.parametrize("new", [1, 600])
def test_log_sums_of_one_key_are_its_scores(new, scale):
    """With a window of one key the log sum is scale * product, products exact in f32: three roundings (the product with the
    scale, the factor back to base e, the product with that), 3 units of 2^-24 of the score. The scale is an f32."""
    n = 1200
    g = torch.Generator("cuda").manual_seed(21)
    a, b = (torch.randint(1024, 2048, (n,), generator=g, device="cuda") / 1024.0 for _ in range(2))
    q = torch.zeros(n, 1, 64, dtype=torch.float16, device="cuda")
    k = torch.zeros(n // 16, 1, 16, 64, dtype=torch.float16, device="cuda")
    q[:, 0, 7], k.view(n, 64)[:, 7] = a.half(), b.half()
    pages = torch.arange(n // 16, dtype=torch.int32, device="cuda")
    if new == 1:
        table, off = pages.expand(n, -1).contiguous(), torch.arange(n + 1, dtype=torch.int32, device="cuda")
        lens = torch.arange(1, n + 1, dtype=torch.int32, device="cuda")
    else:
        table, off = pages.expand(2, -1).contiguous(), torch.tensor([0, 600, n], dtype=torch.int32, device="cuda")
        lens = torch.tensor([600, n], dtype=torch.int32, device="cuda")
    _, lse = qg.attn_paged(q, k, k, table, off, lens, max_new=new, scale=scale, window=1, return_lse=True)
    score = a.double() * b.double() * torch.tensor(scale, dtype=torch.float32).double().item()
    assert ((lse[:, 0].double() - score).abs() <= 3.001 * 2.0**-24 * score).all(), float(((lse[:, 0].double() - score).abs() / score).max() * 2**24)
    assert qg.device_error() == 0
