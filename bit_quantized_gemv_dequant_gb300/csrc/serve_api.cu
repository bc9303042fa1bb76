// C-ABI entry points of the serving operators (block-scaled fp8 product,
// attention over a paged cache, upkeep of its pages, log probabilities):
// argument validation, then dispatch. As in qg_api.cu every check happens
// before anything is enqueued. Index arrays live on the device and are checked
// by the kernels that read them.
#include <cuda_runtime.h>

#include <algorithm>

#include "qg_internal.cuh"

namespace qg {
namespace {

constexpr int64_t kMaxInt = 0x7FFFFFFF;
// Sizes and counts that kernels step through in ints, by up to 8192 at a time.
constexpr int64_t kMaxCount = kMaxInt - 0x3FFF;
constexpr int64_t kMaxBytes = (int64_t)1 << 56;  // no buffer is larger

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
    if (!a || !b || na <= 0 || nb <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

bool is_type(int dtype) { return dtype == QG_F32 || dtype == QG_F16 || dtype == QG_BF16; }
bool is_16bit(int dtype) { return dtype == QG_F16 || dtype == QG_BF16; }
int64_t size_of(int dtype) { return dtype == QG_F32 ? 4 : 2; }

// Whether rows of `width` elements at this stride stay within kMaxBytes; the
// span in bytes goes to *bytes.
bool span(int64_t rows, int64_t width, int64_t stride, int64_t elem, int64_t* bytes) {
    if (stride < width || stride > kMaxBytes / elem / std::max<int64_t>(rows, 1)) return false;
    *bytes = rows > 0 ? ((rows - 1) * stride + width) * elem : 0;
    return true;
}

struct Region {
    const void* p;
    int64_t n;
};

// Any of the outputs over an input, or over another output?
template <int NO, int NI>
bool clash(const Region (&out)[NO], const Region (&in)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < NI; ++j)
            if (overlap(out[i].p, out[i].n, in[j].p, in[j].n)) return true;
        for (int j = i + 1; j < NO; ++j)
            if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return true;
    }
    return false;
}

int check_workspace(const void* ws, size_t have, size_t need) {
    if (need == 0) return QG_OK;
    if (!ws || have < need) return QG_ERR_WORKSPACE;
    return aligned(ws, 16) ? QG_OK : QG_ERR_MISALIGNED;
}

int check_planes(const PagePlanes& p) {
    if (!p.cache || p.planes <= 0 || p.num_pages <= 0 || p.page_bytes <= 0 || p.page_bytes % 16)
        return QG_ERR_INVALID_ARG;
    if (p.num_pages > kMaxCount || p.planes > kMaxCount ||
        p.page_bytes > kMaxBytes / p.num_pages / p.planes)
        return QG_ERR_UNSUPPORTED;
    return aligned(p.cache, 16) ? QG_OK : QG_ERR_MISALIGNED;
}

bool page_size_ok(int64_t n) { return n >= 8 && n <= 256 && (n & (n - 1)) == 0; }

int check_table(int64_t rows, int64_t width) {
    if (rows <= 0 || width <= 0) return QG_ERR_INVALID_ARG;
    return rows > kMaxCount || width > kMaxCount / rows ? QG_ERR_UNSUPPORTED : QG_OK;
}

cudaStream_t cu(qg_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// The launch configuration of an attention call, checked; pointers are not.
int attn_shape(AttnArgs* a, int64_t tokens, int64_t batch, int64_t max_new, int64_t hq, int64_t hkv,
               int64_t d) {
    if (tokens < 0 || batch <= 0 || max_new < 0 || hq <= 0 || hkv <= 0 || hq % hkv)
        return QG_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return QG_ERR_UNSUPPORTED;
    if (hq / hkv > 128 || hq > 65535 || batch > 65535 || tokens > kMaxCount / hq)
        return QG_ERR_UNSUPPORTED;
    a->tokens = (int)tokens;
    a->batch = (int)batch;
    a->max_new = (int)std::min(max_new, tokens);
    a->hq = (int)hq;
    a->hkv = (int)hkv;
    a->d = (int)d;
    return QG_OK;
}

}  // namespace
}  // namespace qg

using namespace qg;

extern "C" {

int quantize_fp8_b128(const void* x, int x_dtype, int64_t x_stride, uint8_t* codes, float* scales,
                      int64_t M, int64_t K, qg_stream_t stream) {
    if (!x || !codes || !scales || M <= 0 || K <= 0 || !is_type(x_dtype)) return QG_ERR_INVALID_ARG;
    if (M > kMaxCount || K > kMaxCount) return QG_ERR_UNSUPPORTED;
    int64_t xb = 0;
    if (!span(M, K, x_stride, size_of(x_dtype), &xb)) return QG_ERR_INVALID_ARG;
    if (!aligned(x, size_of(x_dtype)) || !aligned(scales, 4)) return QG_ERR_MISALIGNED;
    const Region out[] = {{codes, M * K}, {scales, M * ((K + 127) / 128) * 4}};
    const Region in[] = {{x, xb}};
    if (clash(out, in)) return QG_ERR_INVALID_ARG;
    const DevCtx* dc = nullptr;
    int rc = device_ctx(&dc);
    if (rc) return rc;
    return fp8_quantize_launch(*dc, x, x_dtype, x_stride, codes, scales, M, K, cu(stream));
}

int qmm_fp8_b128(const uint8_t* a, const float* a_scales, const uint8_t* w, const float* w_scales,
                 void* y, int y_dtype, int64_t M, int64_t N, int64_t K, void* workspace,
                 size_t workspace_bytes, qg_stream_t stream) {
    if (!a || !a_scales || !w || !w_scales || !y || M <= 0 || N <= 0 || K <= 0)
        return QG_ERR_INVALID_ARG;
    if (y_dtype != QG_F32 && y_dtype != QG_BF16) return QG_ERR_INVALID_ARG;
    if (M > kMaxCount || N > kMaxCount || K > kMaxCount || M > kMaxBytes / 4 / N)
        return QG_ERR_UNSUPPORTED;
    if (!aligned(a_scales, 4) || !aligned(w_scales, 4) || !aligned(y, size_of(y_dtype)))
        return QG_ERR_MISALIGNED;
    const int64_t kb = (K + 127) / 128;
    const Region out[] = {{y, M * N * size_of(y_dtype)}};
    const Region in[] = {{a, M * K}, {a_scales, M * kb * 4}, {w, N * K},
                         {w_scales, (N + 127) / 128 * kb * 4}};
    if (clash(out, in)) return QG_ERR_INVALID_ARG;
    const DevCtx* dc = nullptr;
    int rc = device_ctx(&dc);
    if (rc) return rc;
    if (workspace && !aligned(workspace, 16)) return QG_ERR_MISALIGNED;
    return fp8_mm_launch(*dc, Fp8Args{a, a_scales, w, w_scales, y, y_dtype, M, N, K}, workspace,
                         workspace ? workspace_bytes : 0, cu(stream));
}

int qmm_fp8_b128_workspace_size(int64_t M, int64_t N, int64_t K, size_t* bytes) {
    if (!bytes) return QG_ERR_INVALID_ARG;
    *bytes = 0;
    if (M <= 0 || N <= 0 || K <= 0) return QG_ERR_INVALID_ARG;
    if (M > kMaxCount || N > kMaxCount || K > kMaxCount) return QG_ERR_UNSUPPORTED;
    *bytes = (size_t)(M + N) * (size_t)((K + 15) / 16 * 16);
    return QG_OK;
}

int attn_paged(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
               const int32_t* page_table, const int32_t* q_offsets, const int32_t* context_lens,
               void* out, float* lse, int dtype, int64_t tokens, int64_t batch, int64_t max_new,
               int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t num_pages,
               int64_t page_size, int64_t table_width, float scale, float softcap, int64_t window,
               void* workspace, size_t workspace_bytes, qg_stream_t stream) {
    AttnArgs a{};
    int rc = attn_shape(&a, tokens, batch, max_new, q_heads, kv_heads, head_dim);
    if (rc) return rc;
    if (!k_cache || !v_cache || !page_table || !q_offsets || !context_lens || !is_16bit(dtype) ||
        (tokens > 0 && (!q || !out)))
        return QG_ERR_INVALID_ARG;
    if (num_pages <= 0 || !page_size_ok(page_size) || !(softcap >= 0.f) || window < 0 ||
        scale != scale)
        return QG_ERR_INVALID_ARG;
    rc = check_table(batch, table_width);
    if (rc) return rc;
    if (num_pages > kMaxCount || table_width > kMaxCount / page_size) return QG_ERR_UNSUPPORTED;
    const int64_t cb = kv_heads * page_size * head_dim * 2;
    if (num_pages > kMaxBytes / cb) return QG_ERR_UNSUPPORTED;
    int64_t qb = 0;
    if (!span(tokens, q_heads * head_dim, q_stride, 2, &qb) || q_stride % 8) return QG_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
        !aligned(lse, 4) || !aligned(page_table, 4) || !aligned(q_offsets, 4) ||
        !aligned(context_lens, 4))
        return QG_ERR_MISALIGNED;
    const Region outs[] = {{out, tokens * q_heads * head_dim * 2}, {lse, tokens * q_heads * 4}};
    const Region ins[] = {{q, qb}, {k_cache, num_pages * cb}, {v_cache, num_pages * cb},
                          {page_table, batch * table_width * 4}, {q_offsets, (batch + 1) * 4},
                          {context_lens, batch * 4}};
    if (clash(outs, ins)) return QG_ERR_INVALID_ARG;
    a.q = q; a.k = k_cache; a.v = v_cache;
    a.table = page_table; a.offsets = q_offsets; a.ctx = context_lens;
    a.out = out; a.lse = lse;
    a.q_stride = q_stride;
    a.dtype = dtype;
    a.num_pages = (int)num_pages;
    a.page_size = (int)page_size;
    a.width = (int)table_width;
    a.scale = scale;
    a.softcap = softcap;
    // A window as long as the table hides nothing: none, which keeps position - window an int.
    a.window = window < table_width * page_size ? (int)window : 0;
    const DevCtx* dc = nullptr;
    rc = device_ctx(&dc);
    if (rc) return rc;
    rc = check_workspace(workspace, workspace_bytes, attn_workspace_bytes(*dc, a));
    if (rc) return rc;
    if (a.tokens == 0) return QG_OK;  // with max_new = 0 the kernel records sequences that have some
    return attn_launch(*dc, a, workspace, cu(stream));
}

int attn_paged_workspace_size(int64_t tokens, int64_t batch, int64_t max_new, int64_t q_heads,
                              int64_t kv_heads, int64_t head_dim, size_t* bytes) {
    if (!bytes) return QG_ERR_INVALID_ARG;
    *bytes = 0;
    AttnArgs a{};
    int rc = attn_shape(&a, tokens, batch, max_new, q_heads, kv_heads, head_dim);
    if (rc) return rc;
    const DevCtx* dc = nullptr;
    rc = device_ctx(&dc);
    if (rc) return rc;
    *bytes = attn_workspace_bytes(*dc, a);
    return QG_OK;
}

int kv_append(const void* k, const void* v, int64_t k_stride, int64_t v_stride, int x_dtype,
              void* k_cache, void* v_cache, int cache_dtype, const int64_t* slots, int64_t tokens,
              int64_t kv_heads, int64_t head_dim, int64_t num_pages, int64_t page_size,
              qg_stream_t stream) {
    if (tokens < 0 || kv_heads <= 0 || head_dim <= 0 || num_pages <= 0 || !page_size_ok(page_size) ||
        !is_type(x_dtype) || !is_16bit(cache_dtype) || !k_cache || !v_cache)
        return QG_ERR_INVALID_ARG;
    if (tokens > 0 && (!k || !v || !slots)) return QG_ERR_INVALID_ARG;
    if (head_dim % 8) return QG_ERR_UNSUPPORTED;
    if (kv_heads > 65535 || head_dim > 65535 || kv_heads * head_dim > kMaxCount || tokens > kMaxCount || num_pages > kMaxCount ||
        num_pages > kMaxBytes / (kv_heads * page_size * head_dim * 2))
        return QG_ERR_UNSUPPORTED;
    int64_t kb = 0, vb = 0;
    const int64_t row = kv_heads * head_dim, es = size_of(x_dtype);
    if (!span(tokens, row, k_stride, es, &kb) || !span(tokens, row, v_stride, es, &vb))
        return QG_ERR_INVALID_ARG;
    if (!aligned(k, es) || !aligned(v, es) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(slots, 8))
        return QG_ERR_MISALIGNED;
    const int64_t cb = num_pages * page_size * row * 2;
    const Region out[] = {{k_cache, cb}, {v_cache, cb}};
    const Region in[] = {{k, kb}, {v, vb}, {slots, tokens * 8}};
    if (clash(out, in)) return QG_ERR_INVALID_ARG;
    const DevCtx* dc = nullptr;
    int rc = device_ctx(&dc);
    if (rc) return rc;
    if (tokens == 0) return QG_OK;
    const AppendArgs a{k, v, k_stride, v_stride, x_dtype, cache_dtype, k_cache, v_cache, slots,
                       tokens, num_pages, (int)kv_heads, (int)head_dim, (int)page_size};
    return kv_append_launch(*dc, a, cu(stream));
}

int kv_copy_pages(void* cache, int64_t planes, int64_t num_pages, int64_t page_bytes,
                  const int32_t* src, const int32_t* dst, int64_t n, qg_stream_t stream) {
    const PagePlanes p{static_cast<uint8_t*>(cache), planes, num_pages, page_bytes};
    int rc = check_planes(p);
    if (rc) return rc;
    if (n < 0 || (n > 0 && (!src || !dst))) return QG_ERR_INVALID_ARG;
    if (n > kMaxCount) return QG_ERR_UNSUPPORTED;
    if (!aligned(src, 4) || !aligned(dst, 4)) return QG_ERR_MISALIGNED;
    const Region out[] = {{cache, planes * num_pages * page_bytes}};
    const Region in[] = {{src, n * 4}, {dst, n * 4}};
    if (clash(out, in)) return QG_ERR_INVALID_ARG;
    const DevCtx* dc = nullptr;
    rc = device_ctx(&dc);
    if (rc) return rc;
    if (n == 0) return QG_OK;
    return kv_copy_launch(*dc, p, src, dst, n, cu(stream));
}

int kv_fork_workspace_size(int64_t children, size_t* bytes) {
    if (!bytes) return QG_ERR_INVALID_ARG;
    *bytes = 0;
    if (children < 0) return QG_ERR_INVALID_ARG;
    if (children > kMaxCount) return QG_ERR_UNSUPPORTED;
    // the children's sources and destinations, and the free pages they take
    *bytes = (size_t)children * 12 + 16;
    return QG_OK;
}

int kv_fork(void* cache, int64_t planes, int64_t num_pages, int64_t page_bytes, int64_t page_size,
            const int32_t* page_table, const int32_t* lens, const int32_t* ref_counts, int64_t rows,
            int64_t table_width, const int32_t* parents, int64_t children, int32_t* child_table,
            int32_t* child_lens, int32_t* new_refs, void* workspace, size_t workspace_bytes,
            qg_stream_t stream) {
    const PagePlanes p{static_cast<uint8_t*>(cache), planes, num_pages, page_bytes};
    int rc = check_planes(p);
    if (rc) return rc;
    rc = check_table(rows, table_width);
    if (rc) return rc;
    if (!page_size_ok(page_size) || !page_table || !lens || !ref_counts || !new_refs || children < 0)
        return QG_ERR_INVALID_ARG;
    if (children > 0 && (!parents || !child_table || !child_lens)) return QG_ERR_INVALID_ARG;
    if (children > kMaxCount / table_width) return QG_ERR_UNSUPPORTED;
    const void* ints[] = {page_table, lens, ref_counts, parents, child_table, child_lens, new_refs};
    for (const void* i : ints)
        if (!aligned(i, 4)) return QG_ERR_MISALIGNED;
    const Region out[] = {{cache, planes * num_pages * page_bytes},
                          {child_table, children * table_width * 4},
                          {child_lens, children * 4},
                          {new_refs, num_pages * 4}};
    const Region in[] = {{page_table, rows * table_width * 4}, {lens, rows * 4},
                         {ref_counts, num_pages * 4}, {parents, children * 4}};
    if (clash(out, in)) return QG_ERR_INVALID_ARG;
    size_t need = 0;
    rc = kv_fork_workspace_size(children, &need);
    if (rc) return rc;
    rc = check_workspace(workspace, workspace_bytes, need);
    if (rc) return rc;
    const DevCtx* dc = nullptr;
    rc = device_ctx(&dc);
    if (rc) return rc;
    const ForkArgs a{p, page_table, lens, ref_counts, parents, child_table, child_lens, new_refs,
                     static_cast<int32_t*>(workspace), (int)rows, (int)table_width, (int)children,
                     (int)page_size};
    return kv_fork_launch(*dc, a, cu(stream));
}

int kv_free(const int32_t* page_table, const int32_t* lens, const int32_t* ref_counts,
            const uint8_t* drop, int64_t rows, int64_t table_width, int64_t num_pages,
            int32_t* new_table, int32_t* new_lens, int32_t* new_refs, qg_stream_t stream) {
    int rc = check_table(rows, table_width);
    if (rc) return rc;
    if (!page_table || !lens || !ref_counts || !drop || !new_table || !new_lens || !new_refs ||
        num_pages <= 0)
        return QG_ERR_INVALID_ARG;
    if (num_pages > kMaxCount) return QG_ERR_UNSUPPORTED;
    const void* ints[] = {page_table, lens, ref_counts, new_table, new_lens, new_refs};
    for (const void* i : ints)
        if (!aligned(i, 4)) return QG_ERR_MISALIGNED;
    const Region out[] = {{new_table, rows * table_width * 4}, {new_lens, rows * 4},
                          {new_refs, num_pages * 4}};
    const Region in[] = {{page_table, rows * table_width * 4}, {lens, rows * 4},
                         {ref_counts, num_pages * 4}, {drop, rows}};
    if (clash(out, in)) return QG_ERR_INVALID_ARG;
    const DevCtx* dc = nullptr;
    rc = device_ctx(&dc);
    if (rc) return rc;
    const FreeArgs a{page_table, lens, ref_counts, drop, new_table, new_lens, new_refs, (int)rows,
                     (int)table_width, (int)num_pages};
    return kv_free_launch(*dc, a, cu(stream));
}

int kv_compact_workspace_size(int64_t num_pages, size_t* bytes) {
    if (!bytes) return QG_ERR_INVALID_ARG;
    *bytes = 0;
    if (num_pages <= 0) return QG_ERR_INVALID_ARG;
    if (num_pages > kMaxCount) return QG_ERR_UNSUPPORTED;
    // the number of moves, then their sources and destinations (at most half
    // of the pages move)
    *bytes = 16 + (size_t)((num_pages + 1) / 2) * 8;
    return QG_OK;
}

int kv_compact(void* cache, int64_t planes, int64_t num_pages, int64_t page_bytes,
               const int32_t* page_table, int64_t rows, int64_t table_width,
               const int32_t* ref_counts, int32_t* new_table, int32_t* new_refs, int32_t* page_map,
               int32_t* live, void* workspace, size_t workspace_bytes, qg_stream_t stream) {
    const PagePlanes p{static_cast<uint8_t*>(cache), planes, num_pages, page_bytes};
    int rc = check_planes(p);
    if (rc) return rc;
    rc = check_table(rows, table_width);
    if (rc) return rc;
    if (!page_table || !ref_counts || !new_table || !new_refs || !page_map || !live)
        return QG_ERR_INVALID_ARG;
    const void* ints[] = {page_table, ref_counts, new_table, new_refs, page_map, live};
    for (const void* i : ints)
        if (!aligned(i, 4)) return QG_ERR_MISALIGNED;
    const Region out[] = {{cache, planes * num_pages * page_bytes},
                          {new_table, rows * table_width * 4},
                          {new_refs, num_pages * 4},
                          {page_map, num_pages * 4},
                          {live, 4}};
    const Region in[] = {{page_table, rows * table_width * 4}, {ref_counts, num_pages * 4}};
    if (clash(out, in)) return QG_ERR_INVALID_ARG;
    size_t need = 0;
    rc = kv_compact_workspace_size(num_pages, &need);
    if (rc) return rc;
    rc = check_workspace(workspace, workspace_bytes, need);
    if (rc) return rc;
    const DevCtx* dc = nullptr;
    rc = device_ctx(&dc);
    if (rc) return rc;
    const CompactArgs a{p, page_table, ref_counts, new_table, new_refs, page_map, live,
                        static_cast<int32_t*>(workspace), (int)rows, (int)table_width};
    return kv_compact_launch(*dc, a, cu(stream));
}

int token_logprobs(const void* logits, int dtype, int64_t row_stride, const int64_t* targets,
                   int64_t M, int64_t V, int top_k, float* logprobs, float* entropy, int32_t* ranks,
                   float* top_values, int32_t* top_ids, qg_stream_t stream) {
    if (M < 0 || V <= 0 || top_k < 0 || top_k > V || !is_type(dtype)) return QG_ERR_INVALID_ARG;
    if (M > kMaxInt || V > kMaxInt / 2 + 1 || top_k > 32) return QG_ERR_UNSUPPORTED;
    if (M > 0 && (!logits || !targets || !logprobs || !entropy || !ranks)) return QG_ERR_INVALID_ARG;
    if (M > 0 && top_k > 0 && (!top_values || !top_ids)) return QG_ERR_INVALID_ARG;
    int64_t xb = 0;
    if (!span(M, V, row_stride, size_of(dtype), &xb)) return QG_ERR_INVALID_ARG;
    if (!aligned(logits, size_of(dtype)) || !aligned(targets, 8) || !aligned(logprobs, 4) ||
        !aligned(entropy, 4) || !aligned(ranks, 4) || !aligned(top_values, 4) || !aligned(top_ids, 4))
        return QG_ERR_MISALIGNED;
    const Region out[] = {{logprobs, M * 4}, {entropy, M * 4}, {ranks, M * 4},
                          {top_values, M * top_k * 4}, {top_ids, M * top_k * 4}};
    const Region in[] = {{logits, xb}, {targets, M * 8}};
    if (clash(out, in)) return QG_ERR_INVALID_ARG;
    const DevCtx* dc = nullptr;
    int rc = device_ctx(&dc);
    if (rc) return rc;
    if (M == 0) return QG_OK;
    const LogprobArgs a{logits, dtype, row_stride, targets, M, V, top_k, logprobs, entropy, top_values,
                        ranks, top_ids};
    return logprobs_launch(*dc, a, cu(stream));
}

}  // extern "C"
