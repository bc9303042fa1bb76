// attn_paged: which kernel takes which sequences, and the workspace.
#include <algorithm>
#include <cmath>

#include "attn_work.cuh"

namespace qg {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// Parts of cut row tiles: two per CTA, RT rows of D outputs, a maximum and a
// sum; and a note per CTA.
size_t part_bytes(const DevCtx& dc, int rt, int d) {
    return (size_t)dc.num_sms * (2 * rt * (d + 2) * 4 + sizeof(attn::Note));
}

// Rows per tile, by the most rows that a sequence can have: up to 64 the
// streaming kernel, whose tile is the least that holds them, else the
// tensor-core kernel for the whole batch, whose steps take as long for one row as
// for 128. The bound counts, not the rows: 128 single tokens over 65 to 8192 keys
// take 322 us with max_new = 1, 438 with 8 (32 rows), 727 with 16 (64 rows) and
// 401 with 17 or more. Both sides of the last border, 32/8 heads of 128: one
// sequence of 16 new tokens over 4000 keys 21 us here and 35 there, eight over 1000
// 26.5 and 27.7; 64 over 8192 keys 726 and 373, so for much work the border lies
// too high (the host does not know the lengths).
int row_tile(const AttnArgs& a) {
    const long long rows = (long long)a.max_new * (a.hq / a.hkv);
    return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 256;
}

}  // namespace

size_t attn_workspace_bytes(const DevCtx& dc, const AttnArgs& a) {
    return part_bytes(dc, row_tile(a), a.d);
}

int attn_launch(const DevCtx& dc, const AttnArgs& a, void* ws, cudaStream_t s) {
    attn::Work w{};
    w.a = a;
    w.group = a.hq / a.hkv;
    w.scale_log2 = a.scale * kLog2e;
    if (a.softcap > 0.f) {
        w.cap_in = a.scale / a.softcap;
        w.small = 0.5f / std::fabs(w.cap_in);
        w.cap_out = a.softcap * kLog2e;
    }
    w.to_ln = a.softcap > 0.f ? (float)((double)a.softcap / w.cap_out) : (float)((double)a.scale / w.scale_log2);
    if (!std::isnormal(w.to_ln)) w.to_ln = 0.69314718f;  // a scale of 0, or one out of range
    w.err = dc.err;
    w.ctas = dc.num_sms;
    const int rt = row_tile(a);
    w.part = static_cast<float*>(ws);
    w.ml = reinterpret_cast<float2*>(w.part + (size_t)w.ctas * 2 * rt * a.d);
    w.notes = reinterpret_cast<attn::Note*>(w.ml + (size_t)w.ctas * 2 * rt);
    return rt <= 64 ? attn::launch_few(dc, w, rt / 16, s) : attn::launch_chunk(dc, w, s);
}

}  // namespace qg
