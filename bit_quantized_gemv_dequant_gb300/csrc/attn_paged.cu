// attn_paged: which kernel takes which sequences, and the workspace.
#include <algorithm>

#include "attn_work.cuh"

namespace qg {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// Parts of cut row tiles: two per CTA, RT rows of D outputs, a maximum and a sum.
size_t part_bytes(const DevCtx& dc, int rt, int d) { return (size_t)dc.num_sms * 2 * rt * (d + 2) * 4; }

}  // namespace

size_t attn_workspace_bytes(const DevCtx& dc, const AttnArgs& a) {
    return part_bytes(dc, 64, a.d);
}

int attn_launch(const DevCtx& dc, const AttnArgs& a, void* ws, size_t, cudaStream_t s) {
    attn::Work w{};
    w.a = a;
    w.group = a.hq / a.hkv;
    w.scale_log2 = a.scale * kLog2e;
    if (a.softcap > 0.f) {
        w.cap_in = 2.f * kLog2e * a.scale / a.softcap;
        w.cap_out = a.softcap * kLog2e;
    }
    w.err = dc.err;
    w.ctas = dc.num_sms;
    w.rows_min = 0;
    w.rows_max = 0x7FFFFFFF;
    const long long rows = (long long)a.max_new * w.group;
    const int rb = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    w.part = static_cast<float*>(ws);
    w.ml = reinterpret_cast<float2*>(w.part + (size_t)w.ctas * 2 * 16 * rb * a.d);
    return attn::launch_few(dc, w, rb, s);
}

}  // namespace qg
