// attention_api.hip -- the C ABI of the attention operators (declared in
// include/pq2_attention.h).  As in api.hip: every argument is checked on the
// host before the HIP runtime is touched, a status is returned instead of an
// abort, and buffers are owned by the caller.
#include "attention_internal.h"

#include <math.h>

namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 31;     // head and table strides, elements: spans stay within 64 bits
constexpr int64_t kMaxRowStride = (int64_t)1 << 23;  // row strides: 64 rows stay within a 32-bit byte offset
constexpr int64_t kMaxIndex = ((int64_t)1 << 31) - 1;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
bool dtype_ok(int d) { return d == PQ2_BF16 || d == PQ2_F16 || d == PQ2_F32; }
bool half_ok(int d) { return d == PQ2_BF16 || d == PQ2_F16; }
int esize(int d) { return d == PQ2_F32 ? 4 : 2; }
// (The kernels take exp2 of scores times scale * log2(e).)
bool scale_ok(float s) { return s > 0.0f && isfinite(s * 1.4426950408889634f); }
bool dim_ok(int64_t d) { return d == 64 || d == 128 || d == 256; }
bool page_ok(int64_t p) { return p == 16 || p == 32 || p == 64 || p == 128 || p == 256; }
bool heads_ok(int64_t heads, int64_t kv) { return kv >= 1 && heads >= kv && heads <= PQ2_MAX_ATTN_HEADS && heads % kv == 0; }
bool pages_ok(int64_t pages, int64_t page_tokens) {
    return pages >= 1 && pages <= kMaxIndex && pages * page_tokens <= ((int64_t)1 << 31);
}

// m rows of `bytes`, `stride` bytes apart.
struct Rows {
    const void* p;
    int64_t m;
    size_t stride, bytes;
    size_t span() const { return (size_t)(m - 1) * stride + bytes; }
};

// A tensor of heads: the heads of a row as one stretch where the next row
// starts behind it, else (heads outside, rows inside) the whole span.
Rows heads_rows(const void* p, int64_t rows, int64_t heads, int64_t d, int64_t stride, int64_t head, int es) {
    const size_t row = ((size_t)(heads - 1) * head + d) * es;
    if (rows == 1 || row <= (size_t)stride * es) return {p, rows, (size_t)stride * es, row};
    return {p, 1, 0, (size_t)(rows - 1) * stride * es + row};
}

Rows flat(const void* p, size_t bytes) { return {p, 1, 0, bytes}; }

// Rows of one stride may lie between each other (columns of one buffer); for
// others the whole spans count.
bool overlap(const Rows& a, const Rows& b) {
    if (!a.p || !b.p || !a.m || !b.m) return false;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    if (!(x < y + b.span() && y < x + a.span())) return false;
    if (a.m == 1 || b.m == 1 || a.stride != b.stride) return true;
    const size_t s = a.stride;
    const size_t d = y >= x ? (y - x) % s : (s - (x - y) % s) % s;  // from a row of a to the next one of b
    return d < a.bytes || d + b.bytes > s;
}

// Strides of a tensor of heads: elements of head_dim apart at least, multiples
// of 16 bytes, rows that do not meet (rows outside the heads, or heads outside
// the rows).
int check_strides(int64_t rows, int64_t heads, int64_t d, int64_t stride, int64_t head, int es) {
    if (stride < d || stride > kMaxRowStride || head < d || head > kMaxStride) return PQ2_ESHAPE;
    if (rows > 1 && heads > 1 && stride < (heads - 1) * head + d && head < (rows - 1) * stride + d) return PQ2_ESHAPE;
    if ((stride * es) % 16 || (head * es) % 16) return PQ2_EALIGN;
    return PQ2_OK;
}

bool paged_sizes_ok(int64_t seqs, int64_t max_new, int64_t heads, int64_t kv_heads, int64_t head_dim,
                    int64_t max_len) {
    return seqs >= 1 && seqs <= PQ2_MAX_ATTN_SEQS && max_new >= 1 && max_new <= PQ2_MAX_ATTN_ROWS &&
           heads_ok(heads, kv_heads) && dim_ok(head_dim) && max_len >= 1 && max_len <= kMaxIndex &&
           seqs * kv_heads * ((max_new * (heads / kv_heads) + 15) / 16) <= ((int64_t)1 << 23);
}

}  // namespace

extern "C" {

int64_t pq2_kv_page_bytes(int64_t page_tokens, int64_t kv_heads, int64_t head_dim) {
    if (!page_ok(page_tokens) || !dim_ok(head_dim) || kv_heads < 1 || kv_heads > PQ2_MAX_ATTN_HEADS) return -1;
    return kv_heads * pq2::kv_block_bytes(page_tokens, head_dim);
}

int pq2_kv_write(const pq2_kv_write_args* a, void* stream) {
    if (!a || !a->k || !a->v || (!a->q != !a->q_out)) return PQ2_EINVAL;
    if (!a->cache && !a->q_out && !a->k_out && !a->v_out) return PQ2_EINVAL;
    if (!dtype_ok(a->in_dtype) || !dtype_ok(a->out_dtype)) return PQ2_EINVAL;
    if (a->interleaved != 0 && a->interleaved != 1) return PQ2_EINVAL;
    const int64_t m = a->m, d = a->head_dim, kv = a->kv_heads, heads = a->q ? a->heads : kv;
    if (m < 1 || m > PQ2_MAX_ATTN_ROWS || !dim_ok(d) || !heads_ok(heads, kv)) return PQ2_ESHAPE;
    if (a->rot_dim < 0 || a->rot_dim > d || a->rot_dim % 8) return PQ2_ESHAPE;
    if (a->rot_dim && (!a->cos || !a->sin || !a->positions)) return PQ2_EINVAL;
    if (a->rot_dim && (a->table_rows < 1 || a->table_rows > kMaxIndex)) return PQ2_ESHAPE;
    if (a->cache && !a->slots) return PQ2_EINVAL;
    if (a->cache && (!page_ok(a->page_tokens) || !pages_ok(a->pages, a->page_tokens))) return PQ2_ESHAPE;
    const int is = esize(a->in_dtype), os = esize(a->out_dtype);
    struct T {
        const void* p;
        int64_t n, stride, head;
        int es;
    };
    const T in[3] = {{a->q, heads, a->q_stride, a->q_head, is}, {a->k, kv, a->k_stride, a->k_head, is},
                     {a->v, kv, a->v_stride, a->v_head, is}};
    const T out[3] = {{a->q_out, heads, a->qo_stride, a->qo_head, os}, {a->k_out, kv, a->ko_stride, a->ko_head, os},
                      {a->v_out, kv, a->vo_stride, a->vo_head, os}};
    for (int align = 0; align < 2; ++align)  // shapes are told before alignments
        for (const T* t : {in, out})
            for (int i = 0; i < 3; ++i) {
                if (!t[i].p) continue;
                const int rc = check_strides(m, t[i].n, d, t[i].stride, t[i].head, t[i].es);
                if (rc == PQ2_ESHAPE || (align && rc)) return rc;
                if (align && !aligned(t[i].p, 16)) return PQ2_EALIGN;
            }
    if (!aligned(a->cache, 16) || (a->cache && !aligned(a->slots, 4)) ||
        (a->rot_dim && (!aligned(a->cos, 16) || !aligned(a->sin, 16) || !aligned(a->positions, 4))))
        return PQ2_EALIGN;
    const size_t table = a->rot_dim ? (size_t)a->table_rows * (a->rot_dim / 2) * 4 : 0;
    const size_t cache = a->cache ? (size_t)a->pages * pq2_kv_page_bytes(a->page_tokens, kv, d) : 0;
    Rows rin[3], rout[4];
    for (int i = 0; i < 3; ++i) {
        rin[i] = heads_rows(in[i].p, m, in[i].n, d, in[i].stride, in[i].head, is);
        rout[i] = heads_rows(out[i].p, m, out[i].n, d, out[i].stride, out[i].head, os);
    }
    rout[3] = flat(a->cache, cache);
    const Rows fixed[4] = {flat(a->rot_dim ? a->cos : nullptr, table), flat(a->rot_dim ? a->sin : nullptr, table),
                           flat(a->rot_dim ? a->positions : nullptr, (size_t)m * 4),
                           flat(a->cache ? a->slots : nullptr, (size_t)m * 4)};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 3; ++j) {
            const bool in_place = i == j && in[i].p == out[i].p && in[i].stride == out[i].stride &&
                                  (in[i].n == 1 || in[i].head == out[i].head) && is == os &&
                                  a->in_dtype == a->out_dtype;
            if (overlap(rout[i], rin[j]) && !in_place) return PQ2_EINVAL;
        }
        for (int j = 0; j < 4; ++j) {
            if (overlap(rout[i], fixed[j])) return PQ2_EINVAL;
            if (j > i && overlap(rout[i], rout[j])) return PQ2_EINVAL;
        }
    }
    if (int rc = pq2::api_check_device()) return rc;
    return pq2::api_launch_status(pq2::launch_kv_write(*a, (hipStream_t)stream));
}

int pq2_kv_read(const pq2_kv_read_args* a, void* stream) {
    if (!a || !a->cache || !a->table || !a->starts || !a->k_out || !a->v_out) return PQ2_EINVAL;
    if (!dtype_ok(a->out_dtype)) return PQ2_EINVAL;
    const int64_t d = a->head_dim, kv = a->kv_heads;
    if (a->rows < 1 || a->rows > PQ2_MAX_ATTN_ROWS || a->seqs < 1 || a->seqs > PQ2_MAX_ATTN_SEQS || !dim_ok(d) ||
        kv < 1 || kv > PQ2_MAX_ATTN_HEADS || !page_ok(a->page_tokens) || !pages_ok(a->pages, a->page_tokens))
        return PQ2_ESHAPE;
    if (a->table_pages < 1 || a->table_stride < a->table_pages || a->table_stride > kMaxStride ||
        a->table_pages * a->page_tokens > ((int64_t)1 << 30))
        return PQ2_ESHAPE;
    const int os = esize(a->out_dtype);
    const int rk = check_strides(a->rows, kv, d, a->ko_stride, a->ko_head, os);
    const int rv = check_strides(a->rows, kv, d, a->vo_stride, a->vo_head, os);
    if (rk == PQ2_ESHAPE || rv == PQ2_ESHAPE) return PQ2_ESHAPE;
    if (rk || rv || !aligned(a->cache, 16) || !aligned(a->k_out, 16) || !aligned(a->v_out, 16) ||
        !aligned(a->table, 4) || !aligned(a->starts, 4))
        return PQ2_EALIGN;
    const Rows out[2] = {heads_rows(a->k_out, a->rows, kv, d, a->ko_stride, a->ko_head, os),
                         heads_rows(a->v_out, a->rows, kv, d, a->vo_stride, a->vo_head, os)};
    const Rows in[3] = {flat(a->cache, (size_t)a->pages * pq2_kv_page_bytes(a->page_tokens, kv, d)),
                        flat(a->table, ((size_t)(a->seqs - 1) * a->table_stride + a->table_pages) * 4),
                        flat(a->starts, (size_t)(a->seqs + 1) * 4)};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 3; ++j)
            if (overlap(out[i], in[j])) return PQ2_EINVAL;
    if (overlap(out[0], out[1])) return PQ2_EINVAL;
    if (int rc = pq2::api_check_device()) return rc;
    return pq2::api_launch_status(pq2::launch_kv_read(*a, (hipStream_t)stream));
}

int pq2_attention_paged_workspace(int64_t seqs, int64_t max_new, int64_t heads, int64_t kv_heads, int64_t head_dim,
                                  int64_t max_len, int64_t* partials, int64_t* counters) {
    if (!partials || !counters) return PQ2_EINVAL;
    if (!paged_sizes_ok(seqs, max_new, heads, kv_heads, head_dim, max_len)) return PQ2_ESHAPE;
    const pq2::PagedPlan p = pq2::paged_plan(seqs, max_new, heads, kv_heads, head_dim, max_len);
    *partials = p.partial_floats;
    *counters = p.counter_words;
    return PQ2_OK;
}

int pq2_attention_paged(const pq2_attention_paged_args* a, void* stream) {
    if (!a || !a->q || !a->out || !a->cache || !a->table || !a->lens) return PQ2_EINVAL;
    if (!half_ok(a->dtype) || !scale_ok(a->scale) || a->window < 0) return PQ2_EINVAL;
    const int64_t d = a->head_dim;
    if (!paged_sizes_ok(a->seqs, a->max_new, a->heads, a->kv_heads, d, a->max_len)) return PQ2_ESHAPE;
    if (a->rows < 1 || a->rows > PQ2_MAX_ATTN_ROWS || (!a->starts && a->rows != a->seqs)) return PQ2_ESHAPE;
    if (!page_ok(a->page_tokens) || !pages_ok(a->pages, a->page_tokens)) return PQ2_ESHAPE;
    if (a->table_pages < 1 || a->table_stride < a->table_pages || a->table_stride > kMaxStride ||
        a->table_pages * a->page_tokens > ((int64_t)1 << 30))
        return PQ2_ESHAPE;
    const int rq = check_strides(a->rows, a->heads, d, a->q_stride, a->q_head, 2);
    const int ro = check_strides(a->rows, a->heads, d, a->out_stride, a->out_head, 2);
    if (rq == PQ2_ESHAPE || ro == PQ2_ESHAPE) return PQ2_ESHAPE;
    const pq2::PagedPlan plan = pq2::paged_plan(a->seqs, a->max_new, a->heads, a->kv_heads, d, a->max_len);
    if (plan.splits > 1 && (!a->partials || !a->counters)) return PQ2_EINVAL;
    if (rq || ro || !aligned(a->q, 16) || !aligned(a->out, 16) || !aligned(a->cache, 16) || !aligned(a->table, 4) ||
        !aligned(a->lens, 4) || !aligned(a->starts, 4) || !aligned(a->partials, 16) || !aligned(a->counters, 4))
        return PQ2_EALIGN;
    const Rows out[3] = {heads_rows(a->out, a->rows, a->heads, d, a->out_stride, a->out_head, 2),
                         flat(plan.splits > 1 ? a->partials : nullptr, (size_t)plan.partial_floats * 4),
                         flat(plan.splits > 1 ? a->counters : nullptr, (size_t)plan.counter_words * 4)};
    const Rows in[5] = {heads_rows(a->q, a->rows, a->heads, d, a->q_stride, a->q_head, 2),
                        flat(a->cache, (size_t)a->pages * pq2_kv_page_bytes(a->page_tokens, a->kv_heads, d)),
                        flat(a->table, ((size_t)(a->seqs - 1) * a->table_stride + a->table_pages) * 4),
                        flat(a->lens, (size_t)a->seqs * 4), flat(a->starts, (size_t)(a->seqs + 1) * 4)};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 5; ++j)
            if (overlap(out[i], in[j])) return PQ2_EINVAL;
        for (int j = i + 1; j < 3; ++j)
            if (overlap(out[i], out[j])) return PQ2_EINVAL;
    }
    if (int rc = pq2::api_check_device()) return rc;
    return pq2::api_launch_status(pq2::launch_attention_paged(*a, plan, (hipStream_t)stream));
}

int pq2_attention_prompt(const pq2_attention_prompt_args* a, void* stream) {
    if (!a || !a->q || !a->k || !a->v || !a->out || !a->starts_q || !a->starts_k) return PQ2_EINVAL;
    if (!half_ok(a->dtype) || !scale_ok(a->scale) || (a->causal != 0 && a->causal != 1)) return PQ2_EINVAL;
    if (a->window < 0 || (a->window > 0 && !a->causal)) return PQ2_EINVAL;
    const int64_t d = a->head_dim;
    if (a->rows_q < 1 || a->rows_q > PQ2_MAX_ATTN_ROWS || a->rows_k < 1 || a->rows_k > PQ2_MAX_ATTN_ROWS ||
        a->seqs < 1 || a->seqs > PQ2_MAX_ATTN_SEQS || !heads_ok(a->heads, a->kv_heads) || !dim_ok(d) ||
        a->rows_q * (a->heads / a->kv_heads) > (int64_t)1 << 30)
        return PQ2_ESHAPE;
    const struct {
        const void* p;
        int64_t rows, n, stride, head;
    } t[4] = {{a->q, a->rows_q, a->heads, a->q_stride, a->q_head}, {a->k, a->rows_k, a->kv_heads, a->k_stride, a->k_head},
              {a->v, a->rows_k, a->kv_heads, a->v_stride, a->v_head},
              {a->out, a->rows_q, a->heads, a->out_stride, a->out_head}};
    int rc = PQ2_OK;
    for (const auto& x : t) {
        const int r = check_strides(x.rows, x.n, d, x.stride, x.head, 2);
        if (r == PQ2_ESHAPE) return r;
        if (r || !aligned(x.p, 16)) rc = PQ2_EALIGN;
    }
    if (rc || !aligned(a->starts_q, 4) || !aligned(a->starts_k, 4)) return PQ2_EALIGN;
    Rows r[4];
    for (int i = 0; i < 4; ++i) r[i] = heads_rows(t[i].p, t[i].rows, t[i].n, d, t[i].stride, t[i].head, 2);
    const size_t starts = (size_t)(a->seqs + 1) * 4;
    if (overlap(r[3], r[0]) || overlap(r[3], r[1]) || overlap(r[3], r[2]) || overlap(r[3], flat(a->starts_q, starts)) ||
        overlap(r[3], flat(a->starts_k, starts)))
        return PQ2_EINVAL;
    if ((rc = pq2::api_check_device())) return rc;
    return pq2::api_launch_status(pq2::launch_attention_prompt(*a, (hipStream_t)stream));
}

}  // extern "C"
