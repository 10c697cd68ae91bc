// attention_paged.hip -- attention of one to several new tokens a sequence
// over the paged INT8 cache (pq2_attention_paged).
//
// Mathematics: the query rows of one key-value head (its grouped heads times
// the new tokens, 16 rows a tile) meet 32 keys at a time.  Scores are
// transposed, keys x rows: S^T = K Q^T with v_mfma_f32_16x16x32, so that a lane
// holds four keys of one query row in each result register group, which is at
// once the operand layout of the second product o^T = V^T P^T: the weights go from one
// product to the next without leaving their lane, the row's running maximum m, sum l
// and every output of a lane belong to the one row, and a rescaling is one
// factor a lane.  The order of head dimensions and of keys inside a product is
// free as long as both operands agree; it is chosen so that every lane loads
// whole 16-byte (keys) and head_dim/16-byte (values) stretches of the cache and
// no transposition is left.
//
// Precision: codes are exact in bf16 and fp16; key scales multiply the FP32
// scores, value scales the FP32 weights, which then meet the values as the sum
// of two bf16 (16 bits of the weight, at twice the cheap second product).
//
// Bound: the cache's bytes.
#include "attention_internal.h"

#include <algorithm>

namespace pq2 {

namespace {

constexpr int kWaves = 8;
constexpr int kTile = 32;                  // keys of a wave's step
constexpr int kStep = kWaves * kTile;      // keys of a workgroup's step
constexpr int kRows = 16;                  // query rows of a tile
constexpr int kMaxSplits = 128;
constexpr int kFan = 8;                    // parts that are joined first, of more than kJoin
constexpr int kJoin = 16;                  // parts that are joined at once
constexpr int kTileCounters = 1 + kMaxSplits / kFan;
constexpr float kLog2e = 1.4426950408889634f;

struct PagedArgs {
    const uint16_t* q;
    uint16_t* out;
    int64_t q_stride, q_head, out_stride, out_head;
    const uint8_t* cache;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* starts;
    float* partials;
    uint32_t* counters;
    int64_t table_stride;
    int rows, table_pages, kv_heads, group, pages, page_shift, max_new, window, splits, row_tiles, tile_rows, min_chunk;
    float scale2;  // scale * log2(e)
};

template <typename T> struct Half;
template <> struct Half<__bf16> {
    typedef bf16x8 v8;
    static __device__ __forceinline__ v4f mfma(v8 a, v8 b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
};
template <> struct Half<_Float16> {
    typedef f16x8 v8;
    static __device__ __forceinline__ v4f mfma(v8 a, v8 b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
};

__device__ __forceinline__ float code_at(uint32_t w, int i) { return (float)(int8_t)(w >> (8 * i)); }

// Eight codes (two dwords) as an operand.
template <typename T>
__device__ __forceinline__ typename Half<T>::v8 widen(uint32_t a, uint32_t b) {
    typename Half<T>::v8 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = (T)code_at(a, i);
        v[4 + i] = (T)code_at(b, i);
    }
    return v;
}

// Maximum and sum over the four lanes (16 apart) that share a query row.
__device__ __forceinline__ float max_row(float v) {
    const uint32_t u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const uint32_t w = __float_as_uint(fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1])));
    const auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

__device__ __forceinline__ float sum_row(float v) {
    const uint32_t u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const uint32_t w = __float_as_uint(__uint_as_float(a[0]) + __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// What a wave loads of 32 keys: lane (j, kb) the 16 bytes 16 kb of each 64 of
// keys j and 16 + j, and D/16 bytes from D/16 * j of the values of keys
// 4 kb + 0..3 and 16 + 4 kb + 0..3, with these eight keys' scales.
template <int D>
struct Raw {
    uint4 k[2][D / 64];
    uint32_t v[8][D / 64];
    float4 ks[2], vs[2];
};

template <int N>
__device__ __forceinline__ void load_dwords(const uint8_t* p, uint32_t (&w)[N]) {
    if constexpr (N == 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else if constexpr (N == 2) {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        w[0] = x.x, w[1] = x.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

// Whether this workgroup is the last of `count` to come here, with all its
// stores in memory.  The counter is zero again behind the last one.
__device__ __forceinline__ bool last_of(uint32_t* counter, int count, int* shared) {
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t before = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *shared = before == (uint32_t)(count - 1);
        if (*shared) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    const bool last = *shared;
    __syncthreads();
    return last;
}

// `count` <= kJoin parts of a tile, every `every`th from `first` on, joined:
// into the output (LAST), or into the first of them.  A thread takes four
// columns of a row and reads all it needs at once, past the caches that other XCDs'
// stores do not reach.
template <int D, typename T, bool LAST>
__device__ __forceinline__ void join(const PagedArgs& a, float* first, int count, int every, int r0, int start, int nq, int kvh) {
    constexpr int kAgent = 16;  // cache policy bits of a load or store at agent scope
    const int part_bytes = every * a.tile_rows * (D + 2) * 4;
    const auto parts = make_rsrc(first, (uint32_t)(count * part_bytes));
    for (int e = threadIdx.x; e < a.tile_rows * (D / 4); e += 64 * kWaves) {
        const int row = e / (D / 4), dim = 4 * (e % (D / 4));
        const int at = (row * D + dim) * 4, at_ml = (a.tile_rows * D + 2 * row) * 4;
        u32x2_t ml[kJoin];
        uint4 v[kJoin];
#pragma unroll
        for (int s = 0; s < kJoin; ++s) {
            const int off = min(s, count - 1) * part_bytes;
            ml[s] = __builtin_amdgcn_raw_buffer_load_b64(parts, off + at_ml, 0, kAgent);
            v[s] = buf_load16<kAgent>(parts, (uint32_t)(off + at));
        }
        float top = -INFINITY;
#pragma unroll
        for (int s = 0; s < kJoin; ++s) top = fmaxf(top, __uint_as_float(ml[s][0]));
        const float ref = top == -INFINITY ? 0.0f : top;
        float l = 0.0f, sum[4] = {};
#pragma unroll
        for (int s = 0; s < kJoin; ++s) {
            const float f = s < count ? __builtin_amdgcn_exp2f(__uint_as_float(ml[s][0]) - ref) : 0.0f;
            l += __uint_as_float(ml[s][1]) * f;
#pragma unroll
            for (int c = 0; c < 4; ++c) sum[c] += __uint_as_float(word_of(v[s], c)) * f;
        }
        if constexpr (LAST) {
            const float inv = l > 0.0f ? 1.0f / l : 0.0f;
            const int i = (r0 + row) / a.group, g = r0 + row - i * a.group;
            if (i >= nq || start + i < 0 || start + i >= a.rows) continue;
            typedef T T4 __attribute__((ext_vector_type(4)));
            T* o = reinterpret_cast<T*>(a.out) + (int64_t)(start + i) * a.out_stride + (int64_t)(kvh * a.group + g) * a.out_head + dim;
            *reinterpret_cast<T4*>(o) = T4{(T)(sum[0] * inv), (T)(sum[1] * inv), (T)(sum[2] * inv), (T)(sum[3] * inv)};
        } else {
            // (A row's threads are of one wave, which has read all of the row
            // before it writes.)
            const u32x4_t w = {__float_as_uint(sum[0]), __float_as_uint(sum[1]), __float_as_uint(sum[2]), __float_as_uint(sum[3])};
            __builtin_amdgcn_raw_buffer_store_b128(w, parts, at, 0, kAgent);
            const u32x2_t w2 = {__float_as_uint(top), __float_as_uint(l)};
            if (dim == 0) __builtin_amdgcn_raw_buffer_store_b64(w2, parts, at_ml, 0, kAgent);
        }
    }
}

template <int D, typename T>
__global__ __launch_bounds__(64 * kWaves) void attention_paged_kernel(PagedArgs a) {
    typedef typename Half<T>::v8 v8;
    constexpr int F = D / 16;                 // 16-column pieces of the output
    __shared__ float red[kWaves][kRows][68];  // 64 columns of every wave's output
    __shared__ float2 wave_ml[kWaves][kRows];
    __shared__ int last;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j = lane & 15, kb = lane >> 4;
    const int split = blockIdx.x, kvh = blockIdx.y / a.row_tiles, rt = blockIdx.y % a.row_tiles, seq = blockIdx.z;

    // The sequence, this tile's rows and the keys that any of them sees.
    const int len = max(0, (int)min((int64_t)a.lens[seq], (int64_t)a.table_pages << a.page_shift));
    const int start = a.starts ? a.starts[seq] : seq;
    const int n = a.starts ? a.starts[seq + 1] - start : 1;
    const int nq = min(n, a.max_new);
    const int r0 = rt * kRows, i0 = r0 / a.group;
    if (i0 >= nq) return;
    const int i1 = min(nq - 1, (r0 + kRows - 1) / a.group);
    const int hi = min(len, len - n + i1 + 1);
    const int lo = a.window ? max(0, len - n + i0 - a.window + 1) & ~15 : 0;
    const int span = max(0, hi - lo);
    const int chunk = max(a.min_chunk, ((span + a.splits - 1) / a.splits + kStep - 1) / kStep * kStep);
    const int parts = max(1, (span + chunk - 1) / chunk);
    if (split >= parts) return;
    const int k0 = lo + split * chunk, k1 = min(hi, k0 + chunk);

    // This lane's query row.
    const int r = r0 + j, i = r / a.group, g = r - i * a.group;
    const bool valid = i < nq && start + i >= 0 && start + i < a.rows;
    const int seen_hi = valid ? min(len, len - n + i + 1) : 0;
    const int seen_lo = a.window ? max(0, len - n + i - a.window + 1) : 0;
    v8 qf[D / 32];
    if (valid) {
        const uint16_t* q = a.q + (int64_t)(start + i) * a.q_stride + (int64_t)(kvh * a.group + g) * a.q_head + 16 * kb;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            qf[2 * c] = *reinterpret_cast<const v8*>(q + 64 * c);
            qf[2 * c + 1] = *reinterpret_cast<const v8*>(q + 64 * c + 8);
        }
    } else {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) qf[c] = v8{};
    }

    const int64_t block_bytes = kv_block_bytes(1, D) << a.page_shift;
    const int32_t* table = a.table + seq * a.table_stride;
    const int page_mask = (1 << a.page_shift) - 1;

    v4f acc[F];
#pragma unroll
    for (int f = 0; f < F; ++f) acc[f] = v4f{0, 0, 0, 0};
    float m = -INFINITY, l = 0.0f;

    for (int base = k0 + wave * kTile; base < k1; base += kStep) {
        Raw<D> w;
        bool there[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int key = base + 16 * s, idx = key >> a.page_shift;
            const int page = key < k1 && idx < a.table_pages ? table[idx] : -1;
            there[s] = page >= 0 && page < a.pages;
            const int tok = key & page_mask;
            const uint8_t* block = a.cache + ((int64_t)(there[s] ? page : 0) * a.kv_heads + kvh) * block_bytes;
            const uint8_t* kc = block + (int64_t)(tok + j) * D + 16 * kb;
            const uint8_t* vc = block + ((int64_t)D << a.page_shift) + (int64_t)(tok + 4 * kb) * D + F * j;
            const float* ks = reinterpret_cast<const float*>(block + ((int64_t)(2 * D) << a.page_shift)) + tok + 4 * kb;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) w.k[s][c] = *reinterpret_cast<const uint4*>(kc + 64 * c);
#pragma unroll
            for (int x = 0; x < 4; ++x) load_dwords<D / 64>(vc + x * D, w.v[4 * s + x]);
            w.ks[s] = *reinterpret_cast<const float4*>(ks);
            w.vs[s] = *reinterpret_cast<const float4*>(ks + (1 << a.page_shift));
        }
        float p[8];
        float top = -INFINITY;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            v4f sc = {0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                sc = Half<T>::mfma(widen<T>(w.k[s][c].x, w.k[s][c].y), qf[2 * c], sc);
                sc = Half<T>::mfma(widen<T>(w.k[s][c].z, w.k[s][c].w), qf[2 * c + 1], sc);
            }
            const float ks[4] = {w.ks[s].x, w.ks[s].y, w.ks[s].z, w.ks[s].w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int key = base + 16 * s + 4 * kb + x;
                const bool seen = there[s] && key >= seen_lo && key < seen_hi;
                p[4 * s + x] = seen ? sc[x] * (ks[x] * a.scale2) : -INFINITY;
                top = fmaxf(top, p[4 * s + x]);
            }
        }
        top = fmaxf(m, max_row(top));
        const float ref = top == -INFINITY ? 0.0f : top;
        const float alpha = __builtin_amdgcn_exp2f(m - ref);
        m = top;
        l *= alpha;
#pragma unroll
        for (int f = 0; f < F; ++f) acc[f] *= alpha;
        bf16x8 ph, pl;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const float vs[4] = {w.vs[s].x, w.vs[s].y, w.vs[s].z, w.vs[s].w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float e = __builtin_amdgcn_exp2f(p[4 * s + x] - ref);
                l += e;
                // (A masked key's scale may be anything.)
                const float ev = p[4 * s + x] == -INFINITY ? 0.0f : e * vs[x];
                ph[4 * s + x] = (__bf16)ev;
                pl[4 * s + x] = (__bf16)(ev - (float)ph[4 * s + x]);
            }
        }
#pragma unroll
        for (int f = 0; f < F; ++f) {
            bf16x8 v;
#pragma unroll
            for (int x = 0; x < 8; ++x) v[x] = (__bf16)code_at(w.v[x][f / 4], f % 4);
            acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, ph, acc[f], 0, 0, 0);
            acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, pl, acc[f], 0, 0, 0);
        }
    }

    // The waves' parts joined: each scales its own to the common maximum.
    l = sum_row(l);
    if (kb == 0) wave_ml[wave][j] = make_float2(m, l);
    __syncthreads();
    float common = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) common = fmaxf(common, wave_ml[w][j].x);
    const float ref = common == -INFINITY ? 0.0f : common;
    const float mine = __builtin_amdgcn_exp2f(m - ref);

    // Thread (row, cols): two neighbouring columns of the 64 of each round.
    const int row = threadIdx.x >> 5, pair = threadIdx.x & 31;
    float row_m = -INFINITY, row_l = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) row_m = fmaxf(row_m, wave_ml[w][row].x);
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
        row_l += wave_ml[w][row].y * __builtin_amdgcn_exp2f(wave_ml[w][row].x - (row_m == -INFINITY ? 0.0f : row_m));
    const float inv = row_l > 0.0f ? 1.0f / row_l : 0.0f;
    const int out_i = (r0 + row) / a.group, out_g = r0 + row - out_i * a.group;
    const bool out_valid = out_i < nq && start + out_i >= 0 && start + out_i < a.rows;
    T* out = reinterpret_cast<T*>(a.out) + (int64_t)(start + out_i) * a.out_stride +
             (int64_t)(kvh * a.group + out_g) * a.out_head;
    const int64_t tile = ((int64_t)seq * a.kv_heads + kvh) * a.row_tiles + rt;
    const int64_t part_floats = (int64_t)a.tile_rows * (D + 2);
    float* part = a.partials + (tile * a.splits + split) * part_floats;
    const bool keep = row < a.tile_rows;
#pragma unroll
    for (int round = 0; round < F / 4; ++round) {
        if (round) __syncthreads();
#pragma unroll
        for (int x = 0; x < 4; ++x)
            *reinterpret_cast<float4*>(&red[wave][j][4 * (4 * kb + x)]) =
                make_float4(acc[4 * round][x] * mine, acc[4 * round + 1][x] * mine, acc[4 * round + 2][x] * mine,
                            acc[4 * round + 3][x] * mine);
        __syncthreads();
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float2 v = *reinterpret_cast<const float2*>(&red[w][row][2 * pair]);
            sum.x += v.x;
            sum.y += v.y;
        }
        // Column c of the round's 64: dimension F (c / 4) + 4 round + c % 4.
        const int dim = F * (pair >> 1) + 4 * round + 2 * (pair & 1);
        if (parts == 1) {
            if (out_valid) {
                out[dim] = (T)(sum.x * inv);
                out[dim + 1] = (T)(sum.y * inv);
            }
        } else if (keep) {
            __hip_atomic_store(reinterpret_cast<unsigned long long*>(part + row * D + dim),
                               __builtin_bit_cast(unsigned long long, sum), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    if (parts == 1) return;
    if (keep && pair == 0)
        __hip_atomic_store(reinterpret_cast<unsigned long long*>(part + a.tile_rows * D + 2 * row),
                           __builtin_bit_cast(unsigned long long, make_float2(row_m, row_l)), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);

    // The last workgroup of a tile joins its parts, in their order; of many
    // parts, the last workgroup of each kFan first joins these (a compute unit alone
    // reads about 20 GB/s: 64 parts of 4 KB would take it 13 us).
    const bool two = parts > kJoin;
    uint32_t* counters = a.counters + tile * kTileCounters;
    if (two) {
        const int g = split / kFan, count = min(kFan, parts - g * kFan);
        if (!last_of(counters + 1 + g, count, &last)) return;
        join<D, T, false>(a, a.partials + (tile * a.splits + g * kFan) * part_floats, count, 1, r0, start, nq, kvh);
    }
    const int count = two ? (parts + kFan - 1) / kFan : parts;
    if (!last_of(counters, count, &last)) return;
    join<D, T, true>(a, a.partials + tile * a.splits * part_floats, count, two ? kFan : 1, r0, start, nq, kvh);
}

template <int D, typename T>
void start(const PagedArgs& a, int64_t seqs, hipStream_t stream) {
    const dim3 grid((unsigned)a.splits, (unsigned)(a.kv_heads * a.row_tiles), (unsigned)seqs);
    hipLaunchKernelGGL((attention_paged_kernel<D, T>), grid, dim3(64 * kWaves), 0, stream, a);
}

}  // namespace

PagedPlan paged_plan(int64_t seqs, int64_t max_new, int64_t heads, int64_t kv_heads, int64_t head_dim,
                     int64_t max_len) {
    PagedPlan p;
    const int64_t rows = max_new * (heads / kv_heads);
    p.rows = std::min<int64_t>(rows, kRows);
    p.row_tiles = (rows + kRows - 1) / kRows;
    const int64_t base = seqs * kv_heads * p.row_tiles;
    p.splits = std::max((512 + base - 1) / base, (max_len + 2047) / 2048);
    p.splits = std::max<int64_t>(1, std::min({p.splits, (max_len + kStep - 1) / kStep, (int64_t)kMaxSplits}));
    p.min_chunk = base >= 256 ? 2 * kStep : kStep;
    p.partial_floats = p.splits > 1 ? base * p.splits * p.rows * (head_dim + 2) : 0;
    p.counter_words = p.splits > 1 ? base * kTileCounters : 0;
    return p;
}

hipError_t launch_attention_paged(const pq2_attention_paged_args& a, const PagedPlan& plan, hipStream_t stream) {
    const PagedArgs k{static_cast<const uint16_t*>(a.q), static_cast<uint16_t*>(a.out), a.q_stride, a.q_head,
                      a.out_stride, a.out_head, static_cast<const uint8_t*>(a.cache), a.table, a.lens, a.starts,
                      a.partials, a.counters, a.table_stride, (int)a.rows, (int)a.table_pages, (int)a.kv_heads,
                      (int)(a.heads / a.kv_heads), (int)a.pages, log2_of(a.page_tokens), (int)a.max_new,
                      (int)std::min<int64_t>(a.window, 0x40000000), (int)plan.splits, (int)plan.row_tiles, (int)plan.rows,
                      (int)plan.min_chunk, a.scale * kLog2e};
    clear_stale_error();
    const bool f16 = a.dtype == PQ2_F16;
    if (a.head_dim == 64) f16 ? start<64, _Float16>(k, a.seqs, stream) : start<64, __bf16>(k, a.seqs, stream);
    else if (a.head_dim == 128) f16 ? start<128, _Float16>(k, a.seqs, stream) : start<128, __bf16>(k, a.seqs, stream);
    else f16 ? start<256, _Float16>(k, a.seqs, stream) : start<256, __bf16>(k, a.seqs, stream);
    return hipGetLastError();
}

}  // namespace pq2
