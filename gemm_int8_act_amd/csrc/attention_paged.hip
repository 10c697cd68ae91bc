// attention_paged.hip -- attention of one to several new tokens a sequence
// over the paged INT8 cache (pq2_attention_paged).
//
// Mathematics: the query rows of one key-value head (its grouped heads times
// the new tokens, 16 rows a tile) meet 32 keys at a time.  Scores are
// transposed, keys x rows: S^T = K Q^T with v_mfma_f32_16x16x32, so that a lane
// holds four keys of one query row in each result register group, which is at
// once the operand layout of the second product o^T = V^T P^T: the weights go from one
// product to the next without leaving their lane, the row's reference m, sum l
// and every output of a lane belong to the one row, and a rescaling is one
// factor a lane.  The order of head dimensions and of keys inside a product is
// free as long as both operands agree; it is chosen so that every lane loads
// whole 16-byte (keys) and head_dim/16-byte (values) stretches of the cache and
// no transposition is left.
//
// Precision: key codes are exact in fp16; the queries, scaled by
// a power of two, are fp16 too.  Key scales multiply the FP32 scores, value scales the FP32 weights,
// which then meet the value codes (exact in bf16) as the sum of two bf16 (16
// bits of the weight, at twice the cheap second product).
//
// Bound: the cache's bytes where there is enough of it (64 sequences of 16384
// keys, heads of 128: 401 us, 5.5 TB/s; one of 131071 keys 54 to 61 us, 4.6 to 5.1 TB/s, of
// which some 8 us are the start and the join), else the latency of a few dependent steps: a
// wave's 32 keys take about 330 vector instructions, and a wave alone on its SIMD issues
// one in 8 cycles (1.3 us a step).  Hence workgroups of four waves, of which
// three or four share a compute unit (512 to 1024 at once), and parts of a
// length that gives each of them work: 517 keys of one sequence 9.6 us, 2000 keys 9.6.
#include "attention_internal.h"

#include <algorithm>

namespace pq2 {

namespace {

constexpr int kWaves = 4;
constexpr int kTile = 32;                  // keys of a wave's step
static_assert(64 * kWaves == kPagedThreads, "attention_plan.h");
constexpr int kStep = kWaves * kTile;      // keys of a workgroup's step
constexpr int kRows = kPagedRows;
constexpr int kJoin = 16;                  // parts that are joined at once
constexpr int kAgent = 16;                 // cache policy of a load or store at agent scope
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.0f;             // weights grow to 2^8 before a row's reference moves

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
    int seqs, split_shift;  // splits: a power of two
    int few;                // places, if fewer than eight (0: more)
    float scale2;  // scale * log2(e)
};

__device__ __forceinline__ float code_at(uint32_t w, int i) { return (float)(int8_t)(w >> (8 * i)); }

// Eight key codes (two dwords) as fp16 numbers, exact: a code's byte with its
// top bit flipped, c + 128, below the high byte of 1024 is 1152 + c (one
// instruction for two), which one more brings back to c.  (Left to the end, with
// 1152 times the sum of q taken off a score, the bias costs a score three to ten of its
// bits, most where queries have a common offset.)
__device__ __forceinline__ f16x8 widen(uint32_t a, uint32_t b) {
    constexpr uint32_t kSign = 0x80808080u, kHigh = 0x64646464u;
    a ^= kSign;
    b ^= kSign;
    const u32x4_t v = {__builtin_amdgcn_perm(a, kHigh, 0x00050004u), __builtin_amdgcn_perm(a, kHigh, 0x00070006u),
                       __builtin_amdgcn_perm(b, kHigh, 0x00050004u), __builtin_amdgcn_perm(b, kHigh, 0x00070006u)};
    return __builtin_bit_cast(f16x8, v) - (_Float16)1152.0f;
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

// A sequence as its tiles of `rows` query rows see it: all are split into parts
// of `chunk` keys, the one that sees most into `parts` (at least one; none
// without new tokens).  Keys end at `end`, the length or what the table holds.
struct Sequence {
    int len, end, start, n, chunk, parts;
};

__device__ __forceinline__ Sequence sequence(const PagedArgs& a, int seq, int rows) {
    Sequence s;
    s.len = max(0, a.lens[seq]);
    s.end = min(s.len, a.table_pages << a.page_shift);
    s.start = a.starts ? a.starts[seq] : seq;
    s.n = a.starts ? a.starts[seq + 1] - s.start : 1;
    // Of a window: the rows' own distance, and the alignment to 16 keys.
    const int most = a.window ? (int)min((int64_t)s.end, (int64_t)a.window + (rows + a.group - 1) / a.group + 16) : s.end;
    s.chunk = max(a.min_chunk, (((most + a.splits - 1) >> a.split_shift) + kStep - 1) & ~(kStep - 1));
    // (most - 1) / chunk, below 128: the reciprocal's quotient is off by one at most.
    const int about = (int)((float)(most - 1) * __builtin_amdgcn_rcpf((float)s.chunk));
    s.parts = s.n <= 0 ? 0 : parts_of(most, s.chunk, about);
    return s;
}

// Inclusive sum over the lanes of a wave (row shifts inside 16 lanes, then the
// rows' last lanes broadcast).
__device__ __forceinline__ int scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
    return v;
}

// RT: tiles of 16 query rows that share what a workgroup loads and widens.
template <int D, typename T, int RT>
__global__ __launch_bounds__(64 * kWaves, D == 256 || RT > 1 ? 2 : D == 128 ? 3 : 4) void attention_paged_kernel(PagedArgs a) {
    typedef T T8 __attribute__((ext_vector_type(8)));
    constexpr int F = D / 16;                 // 16-column pieces of the output
    constexpr int ROWS = kRows * RT;
    __shared__ float red[kWaves][kRows][68];  // 64 columns of every wave's output
    __shared__ float2 wave_ml[kWaves][ROWS];
    __shared__ int last;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j = lane & 15, kb = lane >> 4;
    // blockIdx.x counts the parts that there are, of 64 sequences at blockIdx.y:
    // only the lengths tell how many, the grid is for the most, and a workgroup that
    // starts for nothing takes the dispatcher 2.4 ns, behind the others.
    // Workgroups go to the eight XCDs in turn: the row tiles that read the same
    // keys follow each other on one of them; those of fewer than eight places go to all.
    uint32_t turn, place;
    if (a.few) {
        turn = blockIdx.x / a.few, place = blockIdx.x % a.few;
    } else {
        turn = blockIdx.x >> 3, place = turn / a.row_tiles * 8 + (blockIdx.x & 7);
    }
    const int rt = turn % a.row_tiles, kvh = place % a.kv_heads, item = place / a.kv_heads, s0 = blockIdx.y * 64;
    Sequence own_seq{0, 0, 0, 0, 1, 0};
    if (s0 + lane < a.seqs) own_seq = sequence(a, s0 + lane, ROWS);
    const int sums = scan(own_seq.parts);
    if (item >= __builtin_amdgcn_readlane(sums, 63)) return;
    const int at = __ffsll(__ballot(sums > item)) - 1, seq = __builtin_amdgcn_readfirstlane(s0 + at);
    const int split = item - __builtin_amdgcn_readlane(sums, at) + __builtin_amdgcn_readlane(own_seq.parts, at);

    // The sequence, this tile's rows and the keys that any of them sees.
    own_seq.len = __builtin_amdgcn_readlane(own_seq.len, at);
    own_seq.end = __builtin_amdgcn_readlane(own_seq.end, at);
    own_seq.start = __builtin_amdgcn_readlane(own_seq.start, at);
    own_seq.n = __builtin_amdgcn_readlane(own_seq.n, at);
    own_seq.chunk = __builtin_amdgcn_readlane(own_seq.chunk, at);
    const int end = own_seq.end, start = own_seq.start, nq = min(own_seq.n, a.max_new);
    const int r0 = rt * ROWS, i0 = r0 / a.group;
    if (i0 >= nq) return;
    const int i1 = min(nq - 1, (r0 + ROWS - 1) / a.group);
    const int first = own_seq.len - own_seq.n;  // the first new token's position
    const int hi = min(end, first + i1 + 1);
    const int lo = a.window ? max(0, first + i0 - a.window + 1) & ~15 : 0;
    const int span = max(0, hi - lo), parts = max(1, (span + own_seq.chunk - 1) / own_seq.chunk);
    if (split >= parts) return;
    const int k0 = lo + split * own_seq.chunk, k1 = min(hi, k0 + own_seq.chunk);
    // Keys that every row sees.
    const int all_hi = min(k1, first + i0 + 1), all_lo = a.window ? first + i1 - a.window + 1 : 0;

    // This lane's query rows, one a tile.
    int seen_hi[RT], seen_lo[RT];
    // Its queries as fp16, scaled by a power of two to a largest element in
    // [1, 2) (what that rounds is below 2^-24 of it).
    f16x8 qf[RT][D / 32];
    float q_scale[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int r = r0 + 16 * t + j, i = r / a.group, g = r - i * a.group;
        const bool valid = i < nq && start + i >= 0 && start + i < a.rows;
        seen_hi[t] = valid ? min(end, first + i + 1) : 0;
        seen_lo[t] = a.window ? first + i - a.window + 1 : 0;
        const uint16_t* q = a.q + (int64_t)(valid ? start + i : 0) * a.q_stride + (int64_t)(kvh * a.group + (valid ? g : 0)) * a.q_head + 16 * kb;
        T8 x[D / 32];
        float top = 0.0f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            x[c] = *reinterpret_cast<const T8*>(q + 64 * (c / 2) + 8 * (c % 2));
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf((float)x[c][e]));
        }
        const int exp = __builtin_amdgcn_frexp_expf(max_row(valid ? top : 0.0f)) - 1;  // (of 0: -1)
        q_scale[t] = __builtin_ldexpf(a.scale2, exp);
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                qf[t][c][e] = valid ? (_Float16)__builtin_ldexpf((float)x[c][e], -exp) : (_Float16)0.0f;
    }

    const int64_t block_bytes = kv_block_bytes(1, D) << a.page_shift;
    const int32_t* table = a.table + seq * a.table_stride;
    const int page_mask = (1 << a.page_shift) - 1;

    v4f acc[RT][F];
    float m[RT], ref[RT], l[RT];  // the weights' reference (-inf before the first key; 0 then), their sum
#pragma unroll
    for (int t = 0; t < RT; ++t) {
#pragma unroll
        for (int f = 0; f < F; ++f) acc[t][f] = v4f{0, 0, 0, 0};
        m[t] = -INFINITY;
        ref[t] = l[t] = 0.0f;
    }

    // Pages of the two halves of a step's keys, -1 if not to be seen; looked up
    // a step ahead.
    auto page_of = [&](int key) { return key < k1 && (key >> a.page_shift) < a.table_pages ? table[key >> a.page_shift] : -1; };
    const int base0 = k0 + wave * kTile;
    int pages[2] = {page_of(base0), page_of(base0 + 16)};

    // The next step's keys are loaded into the registers of this step's as soon
    // as its scores are formed, its values behind the output's products: either
    // arrives while the other half of a step is computed.
    Raw<D> w;
    bool there[2];
    const uint32_t lane_k = j * D + 16 * kb, lane_v = 4 * kb * D + F * j, lane_s = 16 * kb;
    const uint8_t* block[2];  // the page's block, and the offset of the step's keys in the page
    int tok[2];
    auto locate = [&](int base) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            there[s] = pages[s] >= 0 && pages[s] < a.pages;
            block[s] = a.cache + ((int64_t)(there[s] ? pages[s] : 0) * a.kv_heads + kvh) * block_bytes;
            tok[s] = (base + 16 * s) & page_mask;
        }
    };
    auto load_k = [&]() {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const uint8_t* kc = block[s] + tok[s] * D;
            const uint8_t* ks = block[s] + ((int64_t)(2 * D) << a.page_shift) + tok[s] * 4;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) w.k[s][c] = *reinterpret_cast<const uint4*>(kc + (lane_k + 64 * c));
            w.ks[s] = *reinterpret_cast<const float4*>(ks + lane_s);
        }
    };
    auto load_v = [&]() {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const uint8_t* vc = block[s] + ((int64_t)D << a.page_shift) + tok[s] * D;
            const uint8_t* vs = block[s] + ((int64_t)(2 * D + 4) << a.page_shift) + tok[s] * 4;
#pragma unroll
            for (int x = 0; x < 4; ++x) load_dwords<D / 64>(vc + (lane_v + x * D), w.v[4 * s + x]);
            w.vs[s] = *reinterpret_cast<const float4*>(vs + lane_s);
        }
    };
    if (base0 < k1) {
        locate(base0);
        load_k();
        load_v();
        pages[0] = page_of(base0 + kStep);
        pages[1] = page_of(base0 + kStep + 16);
    }
    for (int base = base0; base < k1; base += kStep) {
        // (There may be pages that are not: this step's own, before the next one's.)
        const bool seen[2] = {there[0], there[1]};
        const bool more = base + kStep < k1;
        if (more) {
            locate(base + kStep);
            pages[0] = page_of(base + 2 * kStep);
            pages[1] = page_of(base + 2 * kStep + 16);
        }
        v4f sc[RT][2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int t = 0; t < RT; ++t) sc[t][s] = v4f{0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                const uint4 k = w.k[s][c / 2];
                const f16x8 kf = c % 2 ? widen(k.z, k.w) : widen(k.x, k.y);
#pragma unroll
                for (int t = 0; t < RT; ++t) sc[t][s] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[t][c], sc[t][s], 0, 0, 0);
            }
        }
        // Scores scaled; where not every row sees every key, the hidden ones'
        // are -inf and the rows' own copies of the value scales 0 (a hidden key's may be anything).
        const float ks[8] = {w.ks[0].x, w.ks[0].y, w.ks[0].z, w.ks[0].w, w.ks[1].x, w.ks[1].y, w.ks[1].z, w.ks[1].w};
        __builtin_amdgcn_sched_barrier(0);
        if (more) load_k();
        __builtin_amdgcn_sched_barrier(0);
        float vs[RT][8];
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const float4 v = w.vs[x / 4];
                vs[t][x] = x % 4 == 0 ? v.x : x % 4 == 1 ? v.y : x % 4 == 2 ? v.z : v.w;
                sc[t][x / 4][x % 4] *= ks[x] * q_scale[t];
            }
        if (!(seen[0] && seen[1] && base + kTile <= all_hi && base >= all_lo)) {
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const int key = base + 16 * (x / 4) + 4 * kb + x % 4;
                    if (!(seen[x / 4] && key >= seen_lo[t] && key < seen_hi[t])) {
                        sc[t][x / 4][x % 4] = -INFINITY;
                        vs[t][x] = 0.0f;
                    }
                }
        }
        bf16x8 ph[RT], pl[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            float top = -INFINITY;
#pragma unroll
            for (int x = 0; x < 8; ++x) top = fmaxf(top, sc[t][x / 4][x % 4]);
            // The reference moves only when a score passes it by far.
            if (__any(top > m[t] + kSlack)) {
                top = max_row(top);
                const float old = m[t];
                if (top > old + kSlack) m[t] = top;
                ref[t] = m[t] == -INFINITY ? 0.0f : m[t];
                float alpha = __builtin_amdgcn_exp2f(old - ref[t]);
                l[t] *= alpha;
#pragma unroll
                for (int f = 0; f < F; ++f) acc[t][f] *= alpha;
            }
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const float e = __builtin_amdgcn_exp2f(sc[t][x / 4][x % 4] - ref[t]);
                l[t] += e;
                const float ev = e * vs[t][x];
                ph[t][x] = (__bf16)ev;
                pl[t][x] = (__bf16)(ev - (float)ph[t][x]);
            }
        }
#pragma unroll
        for (int f = 0; f < F; ++f) {
            bf16x8 v;
#pragma unroll
            for (int x = 0; x < 8; ++x) v[x] = (__bf16)code_at(w.v[x][f / 4], f % 4);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                acc[t][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, ph[t], acc[t][f], 0, 0, 0);
                acc[t][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, pl[t], acc[t][f], 0, 0, 0);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        if (more) load_v();
    }

    // The waves' parts joined: each scales its own to the common reference.
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        l[t] = sum_row(l[t]);
        if (kb == 0) wave_ml[wave][16 * t + j] = make_float2(m[t], l[t]);
    }
    __syncthreads();
    const int64_t tile = ((int64_t)seq * a.kv_heads + kvh) * a.row_tiles + rt;
    const int64_t part_floats = (int64_t)a.tile_rows * (D + 2);
    const auto own = make_rsrc(a.partials + (tile * a.splits + split) * part_floats, (uint32_t)(part_floats * 4));
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        float common = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) common = fmaxf(common, wave_ml[w][16 * t + j].x);
        const float mine = __builtin_amdgcn_exp2f(m[t] - (common == -INFINITY ? 0.0f : common));

        // Thread (row, quad): four neighbouring columns of the 64 of each round.
        static_assert(kWaves * 64 == kRows * 16, "threads");
        const int row = 16 * t + (threadIdx.x >> 4), quad = threadIdx.x & 15;
        float row_m = -INFINITY, row_l = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) row_m = fmaxf(row_m, wave_ml[w][row].x);
        const float row_ref = row_m == -INFINITY ? 0.0f : row_m;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) row_l += wave_ml[w][row].y * __builtin_amdgcn_exp2f(wave_ml[w][row].x - row_ref);
        const float inv = row_l > 0.0f ? 1.0f / row_l : 0.0f;
        const int out_i = (r0 + row) / a.group, out_g = r0 + row - out_i * a.group;
        const bool out_valid = out_i < nq && start + out_i >= 0 && start + out_i < a.rows;
        T* out = reinterpret_cast<T*>(a.out) + (int64_t)(start + out_i) * a.out_stride +
                 (int64_t)(kvh * a.group + out_g) * a.out_head;
        const bool keep = row < a.tile_rows;
#pragma unroll
        for (int round = 0; round < F / 4; ++round) {
            if (t || round) __syncthreads();
#pragma unroll
            for (int x = 0; x < 4; ++x)
                *reinterpret_cast<float4*>(&red[wave][j][4 * (4 * kb + x)]) =
                    make_float4(acc[t][4 * round][x] * mine, acc[t][4 * round + 1][x] * mine, acc[t][4 * round + 2][x] * mine,
                                acc[t][4 * round + 3][x] * mine);
            __syncthreads();
            float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float4 v = *reinterpret_cast<const float4*>(&red[w][threadIdx.x >> 4][4 * quad]);
                sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
            }
            // Columns 4 q .. 4 q + 3 of the round's 64: dimensions F q + 4 round .. + 3.
            const int dim = F * quad + 4 * round;
            if (parts == 1) {
                if (out_valid) {
                    typedef T T4 __attribute__((ext_vector_type(4)));
                    *reinterpret_cast<T4*>(out + dim) = T4{(T)(sum.x * inv), (T)(sum.y * inv), (T)(sum.z * inv), (T)(sum.w * inv)};
                }
            } else if (keep) {
                const u32x4_t w = {__float_as_uint(sum.x), __float_as_uint(sum.y), __float_as_uint(sum.z), __float_as_uint(sum.w)};
                __builtin_amdgcn_raw_buffer_store_b128(w, own, (row * D + dim) * 4, 0, kAgent);
            }
        }
        if (parts > 1 && keep && quad == 0) {
            const u32x2_t w = {__float_as_uint(row_m), __float_as_uint(row_l)};
            __builtin_amdgcn_raw_buffer_store_b64(w, own, (a.tile_rows * D + 2 * row) * 4, 0, kAgent);
        }
    }
    if (parts == 1) return;

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
void start(const PagedArgs& a, int64_t workgroups, hipStream_t stream) {
    const dim3 grid((unsigned)workgroups, (unsigned)((a.seqs + 63) / 64));
    if (D == 256 || a.tile_rows <= kRows) hipLaunchKernelGGL((attention_paged_kernel<D, T, 1>), grid, dim3(64 * kWaves), 0, stream, a);
    else hipLaunchKernelGGL((attention_paged_kernel<D, T, D == 256 ? 1 : 2>), grid, dim3(64 * kWaves), 0, stream, a);
}

}  // namespace

hipError_t launch_attention_paged(const pq2_attention_paged_args& a, const PagedPlan& plan, hipStream_t stream) {
    const int64_t places = paged_places(plan, a.seqs, a.kv_heads), grid = paged_workgroups(plan, a.seqs, a.kv_heads);
    const PagedArgs k{static_cast<const uint16_t*>(a.q), static_cast<uint16_t*>(a.out), a.q_stride, a.q_head,
                      a.out_stride, a.out_head, static_cast<const uint8_t*>(a.cache), a.table, a.lens, a.starts,
                      a.partials, a.counters, a.table_stride, (int)a.rows, (int)a.table_pages, (int)a.kv_heads,
                      (int)(a.heads / a.kv_heads), (int)a.pages, log2_of(a.page_tokens), (int)a.max_new,
                      (int)std::min<int64_t>(a.window, 0x40000000), (int)plan.splits, (int)plan.row_tiles, (int)plan.rows,
                      (int)plan.min_chunk, (int)a.seqs, log2_of(plan.splits), (int)(places < 8 ? places : 0), a.scale * kLog2e};
    clear_stale_error();
    const bool f16 = a.dtype == PQ2_F16;
    if (a.head_dim == 64) f16 ? start<64, _Float16>(k, grid, stream) : start<64, __bf16>(k, grid, stream);
    else if (a.head_dim == 128) f16 ? start<128, _Float16>(k, grid, stream) : start<128, __bf16>(k, grid, stream);
    else f16 ? start<256, _Float16>(k, grid, stream) : start<256, __bf16>(k, grid, stream);
    return hipGetLastError();
}

}  // namespace pq2
