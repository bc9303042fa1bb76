"""The serving entry points refuse bad arguments before they touch a GPU: statuses through the C ABI, with
addresses that nothing ever follows."""
import ctypes as C

import pytest

import bit_quantized_gemv_dequant_gb300 as qg

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
F32, F16, BF16 = qg.QG_F32, qg.QG_F16, qg.QG_BF16
MB = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def built():
    from bit_quantized_gemv_dequant_gb300 import _build
    _build.build()


def at(i):
    """The i-th of some addresses a megabyte apart."""
    return MB * (i + 1)


def refused(name, good, **bad):
    """Calls `name` with one argument of `good` (a dict in the order of the call) replaced at a time."""
    keys = list(good)
    for key, (value, status) in bad.items():
        k = key.rstrip("_0123456789") if key not in good else key
        args = dict(good, **{k: value})
        got = getattr(qg.lib(), name)(*[args[x] for x in keys])
        assert got == status, (name, key, value, got)


def test_quantize():
    good = dict(x=at(0), dtype=F32, stride=256, codes=at(1), scales=at(2), M=4, K=256, stream=None)
    refused("quantize_fp8_b128", good, x=(None, INVALID), codes=(None, INVALID), scales=(None, INVALID),
            dtype=(3, INVALID), stride=(255, INVALID), M=(0, INVALID), K=(-1, INVALID), M_2=(1 << 31, UNSUPPORTED),
            x_2=(at(0) + 2, MISALIGNED), scales_2=(at(2) + 1, MISALIGNED), codes_2=(at(0) + 64, INVALID),
            scales_3=(at(1), INVALID))


def test_product():
    good = dict(a=at(0), sa=at(1), w=at(2), sw=at(3), y=at(4), dtype=BF16, M=4, N=300, K=256, ws=None, wsb=0,
                stream=None)
    refused("qmm_fp8_b128", good, a=(None, INVALID), sa=(None, INVALID), w=(None, INVALID), sw=(None, INVALID),
            y=(None, INVALID), dtype=(F16, INVALID), M=(0, INVALID), N=(0, INVALID), K=(0, INVALID),
            N_2=(1 << 31, UNSUPPORTED), sa_2=(at(1) + 2, MISALIGNED), y_2=(at(4) + 1, MISALIGNED), y_3=(at(0), INVALID),
            y_4=(at(2) + 256, INVALID))
    n = C.c_size_t(1)
    assert qg.lib().qmm_fp8_b128_workspace_size(0, 300, 250, C.byref(n)) == INVALID
    assert qg.lib().qmm_fp8_b128_workspace_size(4, 300, 250, C.byref(n)) == OK and n.value == 304 * 256
    big = dict(good, M=(1 << 31) - 1, N=(1 << 31) - 1)
    refused("qmm_fp8_b128", big, K=(16, UNSUPPORTED))


def test_attention():
    good = dict(q=at(0), stride=1024, k=at(10), v=at(20), table=at(30), offsets=at(31), lens=at(32), out=at(33),
                lse=at(34), dtype=BF16, tokens=5, batch=2, max_new=4, hq=8, hkv=2, d=128, pages=16, page=16, width=8,
                scale=0.1, softcap=0.0, window=0, ws=None, wsb=0, stream=None)
    refused("attn_paged", good, k=(None, INVALID), v=(None, INVALID), table=(None, INVALID), offsets=(None, INVALID),
            lens=(None, INVALID), q=(None, INVALID), out=(None, INVALID), dtype=(F32, INVALID), tokens=(-1, INVALID),
            batch=(0, INVALID), max_new=(-1, INVALID), hq=(7, INVALID), hkv=(0, INVALID), d=(96, UNSUPPORTED),
            d_2=(256, UNSUPPORTED), pages=(0, INVALID), page=(24, INVALID), page_2=(4, INVALID), page_3=(512, INVALID),
            width=(0, INVALID), scale=(float("nan"), INVALID), softcap=(-1.0, INVALID),
            softcap_2=(float("nan"), INVALID), window=(-1, INVALID), stride_2=(1023, INVALID), stride_3=(1028, INVALID),
            q_2=(at(0) + 8, MISALIGNED), k_2=(at(10) + 8, MISALIGNED), out_2=(at(33) + 2, MISALIGNED),
            lse_2=(at(34) + 2, MISALIGNED), table_2=(at(30) + 1, MISALIGNED), out_3=(at(0), INVALID),
            out_4=(at(10) + 4096, INVALID), lse_3=(at(33), INVALID))
    refused("attn_paged", dict(good, hq=1024, stride=1024 * 128), hkv=(2, UNSUPPORTED))  # 512 heads to one
    n = C.c_size_t(1)
    assert qg.lib().attn_paged_workspace_size(5, 2, 4, 8, 2, 80, C.byref(n)) == UNSUPPORTED
    assert qg.lib().attn_paged_workspace_size(5, 0, 4, 8, 2, 64, C.byref(n)) == INVALID
    assert qg.lib().attn_paged_workspace_size(5, 2, 4, 8, 2, 64, None) == INVALID


def test_append():
    good = dict(k=at(0), v=at(1), ks=256, vs=256, x=F32, kc=at(10), vc=at(20), c=F16, slots=at(30), tokens=3, heads=2,
                d=128, pages=8, page=16, stream=None)
    refused("kv_append", good, k=(None, INVALID), v=(None, INVALID), kc=(None, INVALID), vc=(None, INVALID),
            slots=(None, INVALID), x=(5, INVALID), c=(F32, INVALID), ks=(255, INVALID), vs=(0, INVALID),
            tokens=(-1, INVALID), heads=(0, INVALID), d=(0, INVALID), d_2=(100, UNSUPPORTED), pages=(0, INVALID),
            page=(20, INVALID), k_2=(at(0) + 2, MISALIGNED), kc_2=(at(10) + 8, MISALIGNED),
            slots_2=(at(30) + 4, MISALIGNED), vc_2=(at(10) + 1024, INVALID), kc_3=(at(0), INVALID))


def test_pages():
    planes = dict(cache=at(0), planes=2, pages=16, bytes=4096)
    copy = dict(planes, src=at(40), dst=at(41), n=3, stream=None)
    refused("kv_copy_pages", copy, cache=(None, INVALID), planes=(0, INVALID), pages=(0, INVALID), bytes=(0, INVALID),
            bytes_2=(24, INVALID), cache_2=(at(0) + 8, MISALIGNED), pages_2=(1 << 31, UNSUPPORTED), src=(None, INVALID),
            dst=(None, INVALID), n=(-1, INVALID), src_2=(at(40) + 2, MISALIGNED), dst_2=(at(0) + 64, INVALID))
    fork = dict(planes, page=16, table=at(40), lens=at(41), refs=at(42), rows=4, width=8, parents=at(43), children=3,
                ct=at(44), cl=at(45), nr=at(46), ws=at(47), wsb=4096, stream=None)
    refused("kv_fork", fork, page=(12, INVALID), table=(None, INVALID), lens=(None, INVALID), refs=(None, INVALID),
            rows=(0, INVALID), width=(0, INVALID), parents=(None, INVALID), children=(-1, INVALID), ct=(None, INVALID),
            cl=(None, INVALID), nr=(None, INVALID), nr_2=(at(42), INVALID), ct_2=(at(40), INVALID),
            cl_2=(at(45) + 1, MISALIGNED), ws=(None, 5), wsb=(8, 5), ws_2=(at(47) + 4, MISALIGNED))
    free = dict(table=at(40), lens=at(41), refs=at(42), drop=at(43), rows=4, width=8, pages=16, nt=at(44), nl=at(45),
                nr=at(46), stream=None)
    refused("kv_free", free, table=(None, INVALID), drop=(None, INVALID), pages=(0, INVALID), rows=(-2, INVALID),
            nt=(at(40), INVALID), nr=(at(42), INVALID), nl=(at(41) + 2, MISALIGNED))
    compact = dict(planes, table=at(40), rows=4, width=8, refs=at(42), nt=at(44), nr=at(46), map=at(47), live=at(48),
                   ws=at(49), wsb=4096, stream=None)
    refused("kv_compact", compact, table=(None, INVALID), refs=(None, INVALID), map=(None, INVALID),
            live=(None, INVALID), live_2=(at(47), INVALID), nt=(at(40), INVALID), wsb=(16, 5), bytes=(40, INVALID))
    n = C.c_size_t(1)
    assert qg.lib().kv_fork_workspace_size(-1, C.byref(n)) == INVALID
    assert qg.lib().kv_fork_workspace_size(10, C.byref(n)) == OK and n.value >= 120
    assert qg.lib().kv_compact_workspace_size(0, C.byref(n)) == INVALID
    assert qg.lib().kv_compact_workspace_size(101, C.byref(n)) == OK and n.value >= 16 + 51 * 8


def test_logprobs():
    good = dict(x=at(0), dtype=F32, stride=1000, targets=at(10), M=4, V=1000, k=5, lp=at(11), h=at(12), r=at(13),
                tv=at(14), ti=at(15), stream=None)
    refused("token_logprobs", good, x=(None, INVALID), targets=(None, INVALID), lp=(None, INVALID), h=(None, INVALID),
            r=(None, INVALID), tv=(None, INVALID), ti=(None, INVALID), dtype=(-1, INVALID), stride=(999, INVALID),
            M=(-1, INVALID), V=(0, INVALID), k=(-1, INVALID), k_2=(33, UNSUPPORTED), V_2=(4, INVALID),
            x_2=(at(0) + 2, MISALIGNED), targets_2=(at(10) + 4, MISALIGNED), h_2=(at(11), INVALID),
            ti_2=(at(0) + 4, INVALID), V_3=(1 << 30, INVALID))
    refused("token_logprobs", dict(good, stride=1 << 31), V=((1 << 30) + 1, UNSUPPORTED))


def test_sizes_next_to_31_bits():
    """Kernels step through sizes in ints: what a step could carry past 2^31 - 1 is refused, what could not is not."""
    most = (1 << 31) - (1 << 14)
    n = C.c_size_t()
    for big in (most, (1 << 31) - 1):
        status = OK if big == most else UNSUPPORTED
        for shape in ((big, 1, 16), (1, big, 16), (1, 1, big)):
            assert qg.lib().qmm_fp8_b128_workspace_size(*shape, C.byref(n)) == status, shape
        assert qg.lib().kv_fork_workspace_size(big, C.byref(n)) == status
        assert qg.lib().kv_compact_workspace_size(big, C.byref(n)) == status
    over, far = most + 1, 1 << 50
    product = dict(a=at(0), sa=far, w=2 * far, sw=3 * far, y=4 * far, dtype=F32, M=1, N=1, K=1, ws=None, wsb=0, stream=None)
    refused("qmm_fp8_b128", product, M=(over, UNSUPPORTED), N=(over, UNSUPPORTED), K=(over, UNSUPPORTED))
    quantize = dict(x=at(0), dtype=F32, stride=1 << 31, codes=far, scales=2 * far, M=1, K=1, stream=None)
    refused("quantize_fp8_b128", quantize, M=(over, UNSUPPORTED), K=(over, UNSUPPORTED))
    attn = dict(q=at(0), stride=64, k=far, v=2 * far, table=3 * far, offsets=4 * far, lens=5 * far, out=6 * far,
                lse=None, dtype=BF16, tokens=1, batch=1, max_new=1, hq=1, hkv=1, d=64, pages=1, page=256, width=1,
                scale=1.0, softcap=0.0, window=0, ws=None, wsb=0, stream=None)
    refused("attn_paged", attn, tokens=(over, UNSUPPORTED), pages=(over, UNSUPPORTED), width=(over // 256 + 1, UNSUPPORTED))
    append = dict(k=at(0), v=far, ks=1 << 33, vs=1 << 33, x=F16, kc=2 * far, vc=3 * far, c=F16, slots=4 * far, tokens=1,
                  heads=1, d=8, pages=1, page=8, stream=None)
    refused("kv_append", append, tokens=(over, UNSUPPORTED), pages=(over, UNSUPPORTED))
    refused("kv_append", dict(append, heads=65528), d=(32776, UNSUPPORTED))  # 2^31 + 2^15 - 64 values in a row
    planes = dict(cache=far, planes=1, pages=1, bytes=16)
    copy = dict(planes, src=at(40), dst=at(41), n=3, stream=None)
    refused("kv_copy_pages", copy, planes=(over, UNSUPPORTED), pages=(over, UNSUPPORTED), n=(over, UNSUPPORTED))
    free = dict(table=at(0), lens=far, refs=2 * far, drop=3 * far, rows=1, width=1, pages=1, nt=4 * far, nl=5 * far,
                nr=6 * far, stream=None)
    refused("kv_free", free, rows=(over, UNSUPPORTED), width=(over, UNSUPPORTED), pages=(over, UNSUPPORTED))
    fork = dict(planes, page=16, table=at(40), lens=2 * far, refs=3 * far, rows=1, width=1, parents=4 * far, children=1,
                ct=5 * far, cl=6 * far, nr=7 * far, ws=8 * far, wsb=4096, stream=None)
    refused("kv_fork", fork, rows=(over, UNSUPPORTED), width=(over, UNSUPPORTED), children=(over, UNSUPPORTED))
    compact = dict(planes, table=2 * far, rows=1, width=1, refs=3 * far, nt=4 * far, nr=5 * far, map=6 * far, live=7 * far,
                   ws=8 * far, wsb=4096, stream=None)
    refused("kv_compact", compact, rows=(over, UNSUPPORTED), width=(over, UNSUPPORTED), pages=(over, UNSUPPORTED))
