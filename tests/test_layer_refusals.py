"""The entry points between a layer's products refuse bad arguments before they touch a GPU, as in
test_serving_refusals.py."""
import ctypes as C

import bit_quantized_gemv_dequant_gb300 as qg
from test_serving_refusals import (BF16, F16, F32, INVALID, MISALIGNED, OK, UNSUPPORTED, at, built,  # noqa: F401
                                   refused)

NAN, INF = float("nan"), float("inf")


def test_norm():
    good = dict(x=at(0), xt=BF16, xs=256, r=at(1), rt=F32, rs=256, w=at(2), wt=F16, offset=1.0, eps=1e-6, y=at(3), yt=F32,
                ro=at(4), ros=256, M=4, K=256, stream=None)
    bad = dict(x=(None, INVALID), xt=(3, INVALID), xs=(255, INVALID), rt=(7, INVALID), rt_2=(F16, UNSUPPORTED),
               rs=(0, INVALID), wt=(-1, INVALID), offset=(NAN, INVALID), eps=(-1e-6, INVALID), eps_2=(NAN, INVALID),
               ro=(None, INVALID), ros=(255, INVALID), M=(-1, INVALID), K=(0, INVALID), M_2=(1 << 31, UNSUPPORTED),
               x_2=(at(0) + 1, MISALIGNED), r_2=(at(1) + 2, MISALIGNED), w_2=(at(2) + 1, MISALIGNED),
               ro_2=(at(4) + 2, MISALIGNED), ro_3=(at(0), INVALID), ro_4=(at(1) + 4, INVALID), ro_5=(at(2), INVALID))
    refused("rms_norm", good, y=(None, INVALID), yt=(5, INVALID), y_2=(at(3) + 2, MISALIGNED), y_3=(at(0) + 64, INVALID),
            y_4=(at(1), INVALID), y_5=(at(4) + 256, INVALID), y_6=(at(2), INVALID), **bad)
    # in place, but with another stride; the same without a residual: residual_out is not looked at
    refused("rms_norm", dict(good, ro=at(1)), ros=(512, INVALID))
    refused("rms_norm", dict(good, M=0), ros=(256, OK), x=(None, OK), K=(0, INVALID), xt=(9, INVALID))
    codes = {k: v for k, v in good.items() if k not in ("y", "yt")}
    codes = dict(list(codes.items())[:10], codes=at(5), scales=at(6), **dict(list(codes.items())[10:]))
    refused("rms_norm_fp8_b128", codes, codes=(None, INVALID), scales=(None, INVALID), scales_2=(at(6) + 2, MISALIGNED),
            codes_2=(at(6) + 1, INVALID), scales_3=(at(1), INVALID), codes_3=(at(4), INVALID), **bad)


def test_gate():
    good = dict(g=at(0), gs=512, u=at(1), us=256, xt=BF16, y=at(3), yt=F32, M=4, K=256, stream=None)
    bad = dict(g=(None, INVALID), u=(None, INVALID), gs=(255, INVALID), us=(0, INVALID), xt=(3, INVALID), M=(-1, INVALID),
               K=(0, INVALID), K_2=(1 << 31, INVALID), M_2=(1 << 31, UNSUPPORTED), g_2=(at(0) + 1, MISALIGNED),
               u_2=(at(1) + 1, MISALIGNED))
    refused("silu_mul", good, y=(None, INVALID), yt=(3, INVALID), y_2=(at(0), INVALID), y_3=(at(1) + 512, INVALID),
            y_4=(at(3) + 2, MISALIGNED), **dict(bad, K_2=(1 << 31, UNSUPPORTED)))
    refused("silu_mul", dict(good, M=0), g=(None, OK))
    codes = dict(g=at(0), gs=512, u=at(1), us=256, xt=BF16, codes=at(5), scales=at(6), M=4, K=256, stream=None)
    refused("silu_mul_fp8_b128", codes, codes=(None, INVALID), scales=(None, INVALID), codes_2=(at(1), INVALID),
            scales_2=(at(5) + 4, INVALID), scales_3=(at(6) + 1, MISALIGNED), **dict(bad, K_2=(1 << 31, UNSUPPORTED)))


def test_append_rope():
    good = dict(q=at(5), k=at(0), v=at(1), qs=512, ks=256, vs=256, x=F32, pos=at(31), freq=at(32), rot=64, inter=1,
                qo=at(6), kc=at(10), vc=at(20), c=F16, slots=at(30), tokens=3, hq=4, heads=2, d=128, pages=8, page=16,
                stream=None)
    refused("kv_append_rope", good, q=(None, INVALID), qo=(None, INVALID), k=(None, INVALID), v=(None, INVALID),
            kc=(None, INVALID), vc=(None, INVALID), slots=(None, INVALID), pos=(None, INVALID), freq=(None, INVALID),
            x=(5, INVALID), c=(F32, INVALID), qs=(511, INVALID), ks=(255, INVALID), vs=(0, INVALID), tokens=(-1, INVALID),
            hq=(-1, INVALID), heads=(0, INVALID), d=(0, INVALID), d_2=(100, UNSUPPORTED), rot=(0, INVALID),
            rot_2=(63, INVALID), rot_3=(130, INVALID), rot_4=(-2, INVALID), pages=(0, INVALID), page=(20, INVALID),
            q_2=(at(5) + 2, MISALIGNED), k_2=(at(0) + 2, MISALIGNED), kc_2=(at(10) + 8, MISALIGNED),
            qo_2=(at(6) + 8, MISALIGNED), slots_2=(at(30) + 4, MISALIGNED), pos_2=(at(31) + 4, MISALIGNED),
            freq_2=(at(32) + 2, MISALIGNED), vc_2=(at(10) + 1024, INVALID), kc_3=(at(0), INVALID), qo_3=(at(5), INVALID),
            qo_4=(at(10), INVALID), qo_5=(at(32), INVALID), pages_2=(1 << 31, UNSUPPORTED))
    refused("kv_append_rope", dict(good, qs=1 << 20, ks=1 << 20, vs=1 << 20), d=(1032, UNSUPPORTED), hq=(70000, UNSUPPORTED),
            heads=(65536, UNSUPPORTED))
    # without q neither it nor q_out is looked at
    refused("kv_append_rope", dict(good, hq=0, tokens=0), q=(None, OK), qo=(None, OK), k=(None, OK), rot=(3, INVALID))


def test_grouped_product():
    good = dict(a=at(0), sa=at(1), w=at(2), sw=at(3), o=at(5), y=at(4), dtype=BF16, M=4, E=3, N=300, K=256, ws=None, wsb=0,
                stream=None)
    refused("qmm_fp8_b128_grouped", good, a=(None, INVALID), sa=(None, INVALID), w=(None, INVALID), sw=(None, INVALID),
            o=(None, INVALID), y=(None, INVALID), dtype=(F16, INVALID), M=(-1, INVALID), E=(0, INVALID), N=(0, INVALID),
            K=(0, INVALID), E_2=(1025, UNSUPPORTED), M_2=(1 << 31, UNSUPPORTED), N_2=((1 << 31) // 3, UNSUPPORTED),
            K_2=(1 << 31, UNSUPPORTED), sa_2=(at(1) + 2, MISALIGNED), sw_2=(at(3) + 1, MISALIGNED), o_2=(at(5) + 2, MISALIGNED),
            y_2=(at(4) + 1, MISALIGNED), y_3=(at(0), INVALID), y_4=(at(2) + 200000, INVALID), y_5=(at(5), INVALID),
            ws=(at(6) + 8, MISALIGNED))
    n = C.c_size_t(1)
    size = qg.lib().qmm_fp8_b128_grouped_workspace_size
    assert size(4, 3, 300, 250, C.byref(n)) == OK and n.value == 904 * 256
    assert size(-1, 3, 300, 250, C.byref(n)) == INVALID and size(4, 0, 300, 250, C.byref(n)) == INVALID
    assert size(4, 3, 300, 250, None) == INVALID
    assert size(0, 1024, 1, 16, C.byref(n)) == OK and size(0, 1025, 1, 16, C.byref(n)) == UNSUPPORTED


def test_sizes_next_to_31_bits():
    most = (1 << 31) - (1 << 14)
    over, far = most + 1, 1 << 50
    n = C.c_size_t()
    for big, status in ((most, OK), (over, UNSUPPORTED)):
        for shape in ((big, 1, 1, 16), (1, 1, big, 16), (1, 1, 1, big)):
            assert qg.lib().qmm_fp8_b128_grouped_workspace_size(*shape, C.byref(n)) == status, shape
    gate = dict(g=far, gs=1 << 31, u=2 * far, us=1 << 31, xt=F32, y=3 * far, yt=F32, M=1, K=1, stream=None)
    refused("silu_mul", gate, M=(over, UNSUPPORTED), K=(over, UNSUPPORTED))
    norm = dict(x=far, xt=F32, xs=1 << 31, r=None, rt=F32, rs=0, w=None, wt=F32, offset=0.0, eps=1e-6, y=2 * far, yt=F32,
                ro=None, ros=0, M=1, K=1, stream=None)
    refused("rms_norm", norm, M=(over, UNSUPPORTED), K=(over, UNSUPPORTED))
    rope = dict(q=far, k=2 * far, v=3 * far, qs=1 << 33, ks=1 << 33, vs=1 << 33, x=F16, pos=4 * far, freq=5 * far, rot=8,
                inter=0, qo=6 * far, kc=7 * far, vc=8 * far, c=F16, slots=9 * far, tokens=1, hq=1, heads=1, d=8, pages=1,
                page=8, stream=None)
    refused("kv_append_rope", rope, tokens=(over, UNSUPPORTED), pages=(over, UNSUPPORTED))
    refused("kv_append_rope", dict(rope, tokens=most // 8 + 1), hq=(8, UNSUPPORTED), heads=(8, UNSUPPORTED))
