"""kv_append, kv_copy_pages, kv_fork, kv_free and kv_compact against step by step
Python of the same rules. Everything here is exact."""
import numpy as np
import pytest
import torch

import bit_quantized_gemv_dequant_gb300 as qg

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def cache_of(seed, planes, pages, *shape, dtype=torch.bfloat16):
    return torch.randn(planes, pages, *shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


def book(rng, rows, width, pages, page, share=True):
    """A table of random sequences over the pages, with some of them shared, and its counts."""
    table, lens = np.full((rows, width), -1, np.int32), np.zeros(rows, np.int32)
    refs, ids = np.zeros(pages, np.int32), rng.permutation(pages)
    at = 0
    for r in range(rows):
        lens[r] = rng.integers(0, width * page + 1) if r % 5 else rng.choice([0, width * page, page])
        for i in range(-(-int(lens[r]) // page)):
            if share and r and i == 0 and table[0, 0] >= 0 and r % 3 == 0:
                table[r, 0] = table[0, 0]
            elif at < pages:
                table[r, i] = ids[at]
                at += 1
            else:
                lens[r] = i * page
                break
    np.add.at(refs, table[table >= 0], 1)
    return table, lens, refs


@pytest.mark.parametrize("x", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,hq,h,d,page", [(1, 0, 1, 64, 8), (7, 3, 2, 128, 16), (130, 8, 4, 64, 64), (65, 0, 3, 72, 256)])
def test_append(T, hq, h, d, page, dtype, x):
    pages = -(-T // page) + 2
    g = torch.Generator("cuda").manual_seed(T)
    qkv = torch.randn(T, hq + 2 * h, d, generator=g, device="cuda").to(x)
    k, v = qkv[:, hq:hq + h], qkv[:, hq + h:]
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
    slots[::5] = -1
    kc, vc = cache_of(1, 1, pages, h, page, d, dtype=dtype)[0], cache_of(2, 1, pages, h, page, d, dtype=dtype)[0]
    rk, rv = kc.clone(), vc.clone()
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            rk[s // page, :, s % page] = k[t].to(dtype)
            rv[s // page, :, s % page] = v[t].to(dtype)
    qg.kv_append(k, v, kc, vc, slots)
    assert torch.equal(kc, rk) and torch.equal(vc, rv) and qg.device_error() == 0
    slots[0], slots[-1] = pages * page, 2**40
    qg.kv_append(k, v, kc, vc, slots)
    assert qg.device_error() == 32


def test_append_odd_places_and_strides():
    """Rows that start at any element, of a stride that is no multiple of 16 bytes."""
    base = torch.randn(9, 301, device="cuda")
    k, v = base[:, 3:3 + 128].view(9, 2, 64), base[:, 150:278].view(9, 2, 64)
    kc, vc = torch.zeros(2, 2, 8, 64, device="cuda").half(), torch.zeros(2, 2, 8, 64, device="cuda").half()
    qg.kv_append(k, v, kc, vc, torch.arange(9, device="cuda"))
    assert torch.equal(kc.transpose(1, 2).reshape(16, 2, 64)[:9], k.half())
    assert torch.equal(vc.transpose(1, 2).reshape(16, 2, 64)[:9], v.half())


def test_append_past_32_bits():
    h, page, d = 8, 256, 128
    n = (1 << 32) // (h * page * d * 2) + 2
    kc, vc = torch.empty(n, h, page, d, dtype=torch.float16, device="cuda"), torch.empty(1, device="cuda")
    vc = torch.empty_like(kc)
    k = torch.randn(2, h, d, device="cuda").half()
    qg.kv_append(k, -k, kc, vc, torch.tensor([n * page - 1, 5], device="cuda"))
    assert torch.equal(kc[-1, :, -1], k[0]) and torch.equal(vc[-1, :, -1], -k[0]) and torch.equal(kc[0, :, 5], k[1])


@pytest.mark.parametrize("planes,pages,shape", [(1, 4, (8,)), (3, 50, (2, 16, 64)), (2, 40, (1, 8, 72)), (5, 300, (8, 32, 128))])
def test_copy_pages(planes, pages, shape):
    c = cache_of(3, planes, pages, *shape)
    ids = np.random.default_rng(pages).permutation(pages)
    n = pages // 2
    src, dst = ids[:n].copy(), ids[n:2 * n].copy()
    if n > 4:
        src[1] = src[0]  # one page to two places
        src[2], dst[3] = -1, -7
    ref = c.clone()
    for a, b in zip(src, dst):
        if a >= 0 and b >= 0:
            ref[:, b] = ref[:, a]
    qg.kv_copy_pages(c, i32(src), i32(dst))
    assert torch.equal(c, ref) and qg.device_error() == 0
    qg.kv_copy_pages(c, i32([0, pages]), i32([pages + 5, 1]))
    assert torch.equal(c, ref) and qg.device_error() == 32
    qg.kv_copy_pages(c, i32([]), i32([]))


def fork_ref(cache, table, lens, refs, parents, page):
    refs, free = refs.copy(), [p for p in range(len(refs)) if refs[p] == 0]
    child, out_lens = np.full((len(parents), table.shape[1]), -1, np.int32), np.zeros(len(parents), np.int32)
    for c, r in enumerate(parents):
        if not 0 <= r < len(lens):
            continue
        whole, rest = divmod(int(lens[r]), page)
        child[c, :whole] = table[r, :whole]
        out_lens[c] = lens[r]
        if rest:
            if free:
                p = free.pop(0)
                child[c, whole] = p
                cache[:, p] = cache[:, int(table[r, whole])]
            else:
                out_lens[c] = whole * page
    np.add.at(refs, child[child >= 0], 1)
    return child, out_lens, refs


@pytest.mark.parametrize("rows,width,pages,page,children", [(1, 1, 3, 8, 1), (4, 3, 40, 16, 9), (20, 7, 200, 8, 33),
                                                            (7, 40, 9000, 16, 1500), (3, 2, 5, 8, 6), (5, 4, 70, 256, 0)])
def test_fork(rows, width, pages, page, children):
    rng = np.random.default_rng(rows + children)
    table, lens, refs = book(rng, rows, width, pages, page)
    parents = rng.integers(0, rows, children).astype(np.int32)
    cache = cache_of(4, 3, pages, 2, 8)
    ref = cache.clone()
    want = fork_ref(ref, table, lens, refs, parents, page)
    short = any(lens[r] % page for r in parents) and sum(lens[r] % page > 0 for r in parents) > (refs == 0).sum()
    old = cache.clone()
    got = qg.kv_fork(cache, i32(table), i32(lens), i32(refs), i32(parents), page)
    assert qg.device_error() == (64 if short else 0)
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)
    assert torch.equal(cache, ref) and (children == 0 or not short or not torch.equal(cache, old) or (refs == 0).sum() == 0)


def test_fork_of_bad_rows():
    table, lens, refs = book(np.random.default_rng(1), 4, 3, 40, 8)
    lens[1] = 1000
    cache = cache_of(5, 1, 40, 8)
    child, out_lens, new = qg.kv_fork(cache, i32(table), i32(lens), i32(refs), i32([-1, 4, 1, 2]), 8)
    assert qg.device_error() == 32
    assert (child[:3] == -1).all() and (out_lens[:3] == 0).all() and out_lens[3] == int(lens[2])


@pytest.mark.parametrize("rows,width,pages", [(1, 1, 1), (9, 5, 60), (100, 33, 4000), (700, 3, 20000)])
def test_free(rows, width, pages):
    rng = np.random.default_rng(rows)
    table, lens, refs = book(rng, rows, width, pages, 16)
    for drop in (rng.integers(0, 2, rows), np.zeros(rows), np.ones(rows) * 255):
        drop = drop.astype(np.uint8)
        got = qg.kv_free(i32(table), i32(lens), i32(refs), torch.from_numpy(drop).cuda())
        want = refs.copy()
        gone = table[drop > 0]
        np.subtract.at(want, gone[gone >= 0], 1)
        assert np.array_equal(got[0].cpu().numpy(), np.where(drop[:, None] > 0, -1, table))
        assert np.array_equal(got[1].cpu().numpy(), np.where(drop > 0, 0, lens))
        assert np.array_equal(got[2].cpu().numpy(), want)
    assert qg.device_error() == 0


def test_free_records_what_does_not_add_up():
    t, n, r = i32([[0, 1], [1, 9]]), i32([16, 16]), i32([1, 1, 0])
    _, _, refs = qg.kv_free(t, n, r, torch.ones(2, dtype=torch.uint8, device="cuda"))
    assert qg.device_error() == (32 | 128) and refs.tolist() == [0, 0, 0]


def compact_ref(cache, table, refs):
    live = int((refs > 0).sum())
    src = [p for p in range(len(refs)) if refs[p] > 0 and p >= live]
    dst = [p for p in range(live) if refs[p] <= 0]
    page_map = np.where(refs > 0, np.arange(len(refs)), -1).astype(np.int32)
    for s, d in zip(src, dst):
        page_map[s] = d
        cache[:, d] = cache[:, s]
    new = np.zeros_like(refs)
    for p in range(len(refs)):
        if refs[p] > 0:
            new[page_map[p]] = refs[p]
    return np.where(table >= 0, page_map[np.maximum(table, 0)], -1), new, page_map, np.array([live], np.int32)


@pytest.mark.parametrize("pages", [1, 2, 7, 8, 9, 100, 1023, 5000, 30001])
@pytest.mark.parametrize("share", [0.0, 0.1, 0.5, 0.9, 1.0])
def test_compact(pages, share):
    rng = np.random.default_rng(pages)
    refs = np.where(rng.random(pages) < share, rng.integers(1, 4, pages), 0).astype(np.int32)
    table = rng.integers(-1, pages, (13, 6)).astype(np.int32)  # entries of free pages among them
    cache = cache_of(6, 2, pages, 8)
    ref = cache.clone()
    want = compact_ref(ref, table, refs)
    got = qg.kv_compact(cache, i32(table), i32(refs))
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)
    assert torch.equal(cache, ref) and qg.device_error() == 0


def test_compact_of_large_pages():
    rng = np.random.default_rng(5)
    refs = (rng.random(200) < 0.5).astype(np.int32)
    cache = cache_of(7, 3, 200, 8, 32, 128)
    ref = cache.clone()
    want = compact_ref(ref, np.zeros((1, 1), np.int32), refs)
    got = qg.kv_compact(cache, i32([[0]]), i32(refs))
    assert torch.equal(cache, ref) and np.array_equal(got[2].cpu().numpy(), want[2])


def test_a_life_of_a_cache_keeps_every_sequence():
    """Fork, free and compact in turn: what each row's pages hold never changes."""
    rng = np.random.default_rng(3)
    page, pages, width = 8, 120, 9
    table, lens, refs = (i32(a) for a in book(rng, 6, width, 60, page, share=False))
    refs = torch.cat([refs, torch.zeros(60, dtype=torch.int32, device="cuda")])
    cache = cache_of(8, 2, pages, 1, page, 8)

    def contents(t, n):
        return [torch.cat([cache[:, int(p)].flatten(1, 2) for p in row[: -(-int(m) // page)].tolist()] or
                          [cache[:, 0, :0].flatten(1, 2)], 1)[:, : int(m)].clone() for row, m in zip(t, n)]

    told = contents(table, lens)
    for turn in range(6):
        parents = rng.integers(0, table.shape[0], 3)
        child, n, refs = qg.kv_fork(cache, table, lens, refs, i32(parents), page)
        told += [told[p] for p in parents]
        table, lens = torch.cat([table, child]), torch.cat([lens, n])
        drop = np.zeros(table.shape[0], np.uint8)
        drop[rng.permutation(table.shape[0])[:3]] = 1
        table, lens, refs = qg.kv_free(table, lens, refs, torch.from_numpy(drop).cuda())
        told = [t[:, :0] if d else t for t, d in zip(told, drop)]
        table, refs, _, live = qg.kv_compact(cache, table, refs)
        used = table[table >= 0].unique()
        assert live.item() == used.numel() and (used.numel() == 0 or used.max() == used.numel() - 1)
        for a, b in zip(contents(table, lens), told):
            assert torch.equal(a, b)
    assert qg.device_error() == 0


def test_refusals():
    c = cache_of(9, 2, 10, 8)
    t, n, r, p = i32([[0, 1]]), i32([9]), i32(np.ones(10)), i32([0])
    qg.kv_fork(c, t, n, r, p, 8)
    qg.device_error()
    for bad in ((c.cpu(), t, n, r, p, 8), (c, t.long(), n, r, p, 8), (c, t, i32([9, 9]), r, p, 8), (c, t, n, r[:9], p, 8),
                (c[0, 0], t, n, r, p, 8)):
        with pytest.raises(ValueError):
            qg.kv_fork(*bad)
    for bad in ((c, t, n, r, p, 12), (c, t, n, r, p, 4), (cache_of(9, 2, 10, 7), t, n, r, p, 8)):
        with pytest.raises(qg.QGError):
            qg.kv_fork(*bad)
    with pytest.raises(ValueError):
        qg.kv_free(t, n, r, torch.ones(1, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError):
        qg.kv_compact(c, t, r[:3])
    with pytest.raises(ValueError):
        qg.kv_copy_pages(c, i32([0]), i32([1, 2]))
    k = torch.zeros(3, 2, 64, device="cuda")
    kc = torch.zeros(2, 2, 8, 64, dtype=torch.float16, device="cuda")
    s = torch.arange(3, device="cuda")
    for bad in ((k, k.half(), kc, kc.clone(), s), (k, k, kc, kc.clone(), s.int()), (k, k, kc, kc[:1].clone(), s),
                (k, k, kc, kc.clone(), s[:2])):
        with pytest.raises(ValueError):
            qg.kv_append(*bad)
    with pytest.raises(qg.QGError):  # both caches in one place
        qg.kv_append(k, k, kc, kc, s)
    with pytest.raises(qg.QGError):  # a cache of 32-bit values
        qg.kv_append(k, k, kc.float(), kc.float(), s)


@pytest.mark.parametrize("entry", [-1, -7, 6, 10**6])
def test_fork_of_a_row_without_its_last_page(entry):
    """A partly filled last page that the table does not name: recorded, and no page is read for it."""
    for where in (0, 1):
        cache = cache_of(9, 2, 6, 4, 8)
        before = cache.clone()
        table, refs = i32([[4, 2, -1], [0, 3, -1]]), i32([1, 0, 1, 1, 1, 0])
        table[0, where] = entry
        child, lens, new = qg.kv_fork(cache, table, i32([12, 13]), refs, i32([0, 1]), 8)
        assert qg.device_error() == 32
        assert lens.tolist() == [12, 13] and child[1].tolist() == [0, 5, -1]
        assert child[0].tolist() == ([-1, 1, -1] if where == 0 else [4, 1, -1])
        assert new.tolist() == [2, 1, 1, 1, 1 if where == 0 else 2, 1]
        assert torch.equal(cache[:, 5], before[:, 3]) and torch.equal(cache[:, [0, 2, 3, 4]], before[:, [0, 2, 3, 4]])
        assert torch.equal(cache[:, 1], before[:, 2] if where == 0 else before[:, 1])
