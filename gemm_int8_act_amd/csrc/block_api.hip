// block_api.hip -- the C ABI of the feed-forward block operators (declared in
// include/pq2_block.h).  As in api.hip: every argument is checked on the host
// before the HIP runtime is touched, a status is returned instead of an
// abort, and buffers are owned by the caller.
#include "../../include/pq2_block.h"
#include "block_internal.h"

#include <hip/hip_runtime.h>
#include <math.h>

namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 31;  // elements: spans stay within 64 bits
constexpr int64_t kMaxQuantised = (int64_t)1 << 34;  // elements of x: the quantiser's grid
constexpr double kMinEps = 1e-70;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

struct Span {
    const void* p;
    size_t bytes;
};

bool overlap(const Span& a, const Span& b) {
    if (!a.p || !b.p) return false;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return x < y + b.bytes && y < x + a.bytes;
}

bool dtype_ok(int d) { return d == PQ2_BF16 || d == PQ2_F16 || d == PQ2_F32; }
int esize(int d) { return d == PQ2_F32 ? 4 : 2; }
bool group_ok(int64_t g) { return g == 128 || g == 64 || g == 32; }
bool k_ok(int64_t k) { return k >= 128 && k % 128 == 0 && k <= PQ2_MAX_K; }

// Rows of `stride` elements, k used in each.
size_t row_span(int64_t m, int64_t stride, int64_t k, int es) { return ((size_t)(m - 1) * stride + k) * es; }

// m rows of `bytes`, `stride` bytes apart.
struct Rows {
    const void* p;
    int64_t m;
    size_t stride, bytes;
};

// Rows of one stride may lie between each other (columns of one buffer); for
// others the whole spans count.
bool overlap(const Rows& a, const Rows& b) {
    auto span = [](const Rows& r) { return Span{r.p, (size_t)(r.m - 1) * r.stride + r.bytes}; };
    if (!a.p || !b.p || !overlap(span(a), span(b))) return false;
    if (a.m == 1 || b.m == 1 || a.stride != b.stride) return true;
    const size_t s = a.stride;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    const size_t d = y >= x ? (y - x) % s : (s - (x - y) % s) % s;  // from a row of a to the next one of b
    return d < a.bytes || d + b.bytes > s;
}

// Checks of a product from q and xs (wgroup 0: ternary tiles; h_dtype < 0:
// fp32 y), and its launch description.
int check_product(const int8_t* q, const float* xs, const void* w0, const void* w1, int64_t m, int64_t n, int64_t k,
                  int64_t wgroup, bool gated, int act, void* out, int out_dtype, void* stream, pq2::BlockMatmul* p) {
    if (!q || !xs || !w0 || !out || (gated && !w1)) return PQ2_EINVAL;
    if (wgroup != 0 && !group_ok(wgroup)) return PQ2_EINVAL;
    if (gated && ((act != PQ2_ACT_SILU && act != PQ2_ACT_GELU_TANH) || !dtype_ok(out_dtype))) return PQ2_EINVAL;
    if (m < 1 || m > PQ2_MAX_BLOCK_M || n < 1 || n > PQ2_MAX_BLOCK_N || !k_ok(k)) return PQ2_ESHAPE;
    const int os = gated ? esize(out_dtype) : 4;
    if (!aligned(q, 16) || !aligned(xs, 4) || !aligned(w0, 16) || (gated && !aligned(w1, 16)) || !aligned(out, os))
        return PQ2_EALIGN;
    const size_t wbytes = (size_t)(wgroup ? pq2::w4_tiles_bytes(n, k, wgroup) : pq2::tiles_bytes(n, k));
    const Span o{out, (size_t)m * n * os};
    if (overlap(o, {q, (size_t)m * k}) || overlap(o, {xs, (size_t)m * (k / 128) * 4}) || overlap(o, {w0, wbytes}) ||
        overlap(o, {gated ? w1 : nullptr, wbytes}))
        return PQ2_EINVAL;
    *p = pq2::BlockMatmul{q, xs, static_cast<const uint8_t*>(w0), static_cast<const uint8_t*>(w1), m, n, k,
                          wgroup ? pq2::kFmtW4 : pq2::kFmtTernary, wgroup ? (int)(128 / wgroup) : 1,
                          gated ? act : -1, out, out_dtype, (hipStream_t)stream};
    return PQ2_OK;
}

int launch_product(const pq2::BlockMatmul& p) {
    if (int rc = pq2::api_check_device()) return rc;
    return pq2::api_launch_status(pq2::block_takes_small_m(p) ? pq2::launch_block_small_m(p)
                                                              : pq2::launch_block_prefill(p));
}

int product(const int8_t* q, const float* xs, const void* w0, const void* w1, int64_t m, int64_t n, int64_t k,
            int64_t wgroup, bool gated, int act, void* out, int out_dtype, void* stream) {
    pq2::BlockMatmul p;
    if (int rc = check_product(q, xs, w0, w1, m, n, k, wgroup, gated, act, out, out_dtype, stream, &p)) return rc;
    return launch_product(p);
}

// The complete call: quantiser into the scratch, then the product.
int linear(const void* x, int dtype, int64_t stride, const void* w0, const void* w1, int64_t m, int64_t n, int64_t k,
           int64_t wgroup, bool gated, int act, void* out, int out_dtype, int8_t* q, float* xs, void* stream) {
    if (!x || !dtype_ok(dtype)) return PQ2_EINVAL;
    if (m >= 1 && m <= PQ2_MAX_BLOCK_M && k_ok(k) && m * k > kMaxQuantised) return PQ2_ESHAPE;
    pq2::BlockMatmul p;
    if (int rc = check_product(q, xs, w0, w1, m, n, k, wgroup, gated, act, out, out_dtype, stream, &p)) return rc;
    if (stride < k || stride > kMaxStride) return PQ2_ESHAPE;
    if (!aligned(x, esize(dtype))) return PQ2_EALIGN;
    const size_t wbytes = (size_t)(wgroup ? pq2::w4_tiles_bytes(n, k, wgroup) : pq2::tiles_bytes(n, k));
    const Span xspan{x, row_span(m, stride, k, esize(dtype))}, qs{q, (size_t)m * k},
        ss{xs, (size_t)m * (k / 128) * 4}, o{out, (size_t)m * n * (gated ? esize(out_dtype) : 4)};
    if (overlap(qs, xspan) || overlap(ss, xspan) || overlap(qs, ss) || overlap(o, xspan) ||
        overlap(qs, {w0, wbytes}) || overlap(ss, {w0, wbytes}) || overlap(qs, {gated ? w1 : nullptr, wbytes}) ||
        overlap(ss, {gated ? w1 : nullptr, wbytes}))
        return PQ2_EINVAL;
    if (int rc = pq2::api_check_device()) return rc;
    // Few columns: one launch, which reads x with 16-byte loads and 32-bit
    // offsets (the same bits, the scratch untouched).
    const int es = esize(dtype);
    if (pq2::block_takes_x(m, k) && aligned(x, 16) && (stride * es) % 16 == 0 && xspan.bytes < ((size_t)1 << 31)) {
        p.src = pq2::src_of_dtype(dtype);
        p.x = x;
        p.x_stride = stride;
        return launch_product(p);
    }
    if (int rc = pq2::api_launch_status(pq2::launch_quantize(x, dtype, stride, m, k, q, xs, (hipStream_t)stream)))
        return rc;
    return launch_product(p);
}

}  // namespace

extern "C" {

int64_t pq2_w4_tiles_bytes(int64_t n, int64_t k, int64_t wgroup) {
    if (n < 1 || n > PQ2_MAX_BLOCK_N || !k_ok(k) || !group_ok(wgroup)) return -1;
    return pq2::w4_tiles_bytes(n, k, wgroup);
}

int pq2_prepare_w4_tiles(const uint8_t* codes, int64_t codes_row_stride_bytes, const void* scales,
                         int64_t scales_row_stride_elems, int64_t n, int64_t k, int64_t wgroup, void* tiles,
                         void* stream) {
    if (!codes || !scales || !tiles || !group_ok(wgroup)) return PQ2_EINVAL;
    if (n < 1 || n > PQ2_MAX_BLOCK_N || !k_ok(k)) return PQ2_ESHAPE;
    if (codes_row_stride_bytes < k / 2 || scales_row_stride_elems < k / wgroup) return PQ2_ESHAPE;
    if (codes_row_stride_bytes > kMaxStride || scales_row_stride_elems > kMaxStride) return PQ2_ESHAPE;
    if (!aligned(tiles, 16) || !aligned(scales, 2)) return PQ2_EALIGN;
    const Span o{tiles, (size_t)pq2::w4_tiles_bytes(n, k, wgroup)};
    if (overlap(o, {codes, row_span(n, codes_row_stride_bytes, k / 2, 1)}) ||
        overlap(o, {scales, row_span(n, scales_row_stride_elems, k / wgroup, 2)}))
        return PQ2_EINVAL;
    if (int rc = pq2::api_check_device()) return rc;
    return pq2::api_launch_status(pq2::launch_prepare_w4(codes, codes_row_stride_bytes,
                                                         static_cast<const uint16_t*>(scales), scales_row_stride_elems,
                                                         n, k, (int)wgroup, static_cast<uint8_t*>(tiles),
                                                         (hipStream_t)stream));
}

int pq2_matmul_w4(const int8_t* q, const float* xs, const void* tiles, int64_t m, int64_t n, int64_t k,
                  int64_t wgroup, float* y, void* stream) {
    if (!group_ok(wgroup)) return PQ2_EINVAL;
    return product(q, xs, tiles, nullptr, m, n, k, wgroup, false, -1, y, PQ2_F32, stream);
}

int pq2_linear_w4(const void* x, int dtype, int64_t x_row_stride_elems, const void* tiles, int64_t m, int64_t n,
                  int64_t k, int64_t wgroup, float* y, int8_t* q_work, float* xs_work, void* stream) {
    if (!group_ok(wgroup)) return PQ2_EINVAL;
    return linear(x, dtype, x_row_stride_elems, tiles, nullptr, m, n, k, wgroup, false, -1, y, PQ2_F32, q_work,
                  xs_work, stream);
}

int pq2_gated_matmul_tiles(const int8_t* q, const float* xs, const void* gate, const void* up, int64_t m, int64_t n,
                           int64_t k, int act, void* h, int h_dtype, void* stream) {
    return product(q, xs, gate, up, m, n, k, 0, true, act, h, h_dtype, stream);
}

int pq2_gated_matmul_w4(const int8_t* q, const float* xs, const void* gate, const void* up, int64_t m, int64_t n,
                        int64_t k, int64_t wgroup, int act, void* h, int h_dtype, void* stream) {
    if (!group_ok(wgroup)) return PQ2_EINVAL;
    return product(q, xs, gate, up, m, n, k, wgroup, true, act, h, h_dtype, stream);
}

int pq2_gated_linear_tiles(const void* x, int dtype, int64_t x_row_stride_elems, const void* gate, const void* up,
                           int64_t m, int64_t n, int64_t k, int act, void* h, int h_dtype, int8_t* q_work,
                           float* xs_work, void* stream) {
    return linear(x, dtype, x_row_stride_elems, gate, up, m, n, k, 0, true, act, h, h_dtype, q_work, xs_work, stream);
}

int pq2_gated_linear_w4(const void* x, int dtype, int64_t x_row_stride_elems, const void* gate, const void* up,
                        int64_t m, int64_t n, int64_t k, int64_t wgroup, int act, void* h, int h_dtype,
                        int8_t* q_work, float* xs_work, void* stream) {
    if (!group_ok(wgroup)) return PQ2_EINVAL;
    return linear(x, dtype, x_row_stride_elems, gate, up, m, n, k, wgroup, true, act, h, h_dtype, q_work, xs_work,
                  stream);
}

int pq2_block_norm(const pq2_block_norm_args* a, void* stream) {
    if (!a || !a->r || !a->w || (!a->r_out && !a->x_out && !a->q)) return PQ2_EINVAL;
    if (!a->q != !a->xs) return PQ2_EINVAL;
    if (!a->block && (a->post_w || a->gate)) return PQ2_EINVAL;
    if (!dtype_ok(a->r_dtype) || !dtype_ok(a->w_dtype) || !dtype_ok(a->x_dtype) ||
        (a->block && !dtype_ok(a->block_dtype)))
        return PQ2_EINVAL;
    if (a->q && !group_ok(a->agroup)) return PQ2_EINVAL;
    // (Below kMinEps a zero row's rstd would not be a finite float.)
    if (!(a->eps >= kMinEps) || !isfinite(a->eps) || !isfinite(a->alpha)) return PQ2_EINVAL;
    if (a->unit_offset != 0 && a->unit_offset != 1) return PQ2_EINVAL;
    const int64_t m = a->m, k = a->k;
    if (m < 1 || m > PQ2_MAX_BLOCK_M || !k_ok(k)) return PQ2_ESHAPE;
    if (a->r_stride < k || (a->block && a->block_stride < k) || (a->r_out && a->r_out_stride < k) ||
        (a->x_out && a->x_out_stride < k) || (a->gate && a->gate_stride != 0 && a->gate_stride < k))
        return PQ2_ESHAPE;
    if (a->r_stride > kMaxStride || (a->block && a->block_stride > kMaxStride) ||
        (a->r_out && a->r_out_stride > kMaxStride) || (a->x_out && a->x_out_stride > kMaxStride) ||
        (a->gate && a->gate_stride > kMaxStride))
        return PQ2_ESHAPE;
    const int rs = esize(a->r_dtype), ws = esize(a->w_dtype), xs = esize(a->x_dtype), bs = esize(a->block_dtype);
    if (!aligned(a->r, rs) || !aligned(a->r_out, rs) || !aligned(a->w, ws) || !aligned(a->post_w, ws) ||
        !aligned(a->gate, ws) || !aligned(a->x_out, xs) || (a->block && !aligned(a->block, bs)) ||
        !aligned(a->q, 8) || !aligned(a->xs, 4))
        return PQ2_EALIGN;
    auto rows = [&](const void* p, int64_t stride, int es) { return Rows{p, m, (size_t)stride * es, (size_t)k * es}; };
    auto vec = [&](const void* p) { return Rows{p, 1, 0, (size_t)k * ws}; };
    const Rows r = rows(a->r, a->r_stride, rs);
    const Rows in[4] = {rows(a->block, a->block_stride, bs), vec(a->post_w),
                        a->gate_stride ? rows(a->gate, a->gate_stride, ws) : vec(a->gate), vec(a->w)};
    const size_t xs_bytes = a->q ? (size_t)(k / a->agroup) * 4 : 0;
    const Rows out[4] = {rows(a->r_out, a->r_out_stride, rs), rows(a->x_out, a->x_out_stride, xs), rows(a->q, k, 1),
                         {a->xs, m, xs_bytes, xs_bytes}};
    const bool in_place = a->r_out == a->r && a->r_out_stride == a->r_stride;
    for (int i = 0; i < 4; ++i) {
        if (overlap(out[i], r) && !(i == 0 && in_place)) return PQ2_EINVAL;
        for (int j = 0; j < 4; ++j) {
            if (overlap(out[i], in[j])) return PQ2_EINVAL;
            if (j > i && overlap(out[i], out[j])) return PQ2_EINVAL;
        }
    }
    if (int rc = pq2::api_check_device()) return rc;
    return pq2::api_launch_status(pq2::launch_block_norm(*a, (hipStream_t)stream));
}

}  // extern "C"
