// attention_prompt.hip -- attention over packed prompts (pq2_attention_prompt).
//
// Mathematics: a wave takes 32 query rows of one key-value head (a row is a
// token's query under one of the grouped heads), a workgroup 128 or 256 of them, and runs
// over the keys 64 (head_dim 256: 32) at a time with the softmax's running reference
// and sum.  Scores are transposed, keys x rows: S^T = K Q^T with
// v_mfma_f32_32x32x16, whose result registers 8t .. 8t + 7 of a lane are, as
// they stand, the weights operand of one step of o^T = V^T P^T (the order of
// the keys inside a step is free, the values are read in the same order): the weights
// never leave their lane, and a row's reference, sum and rescaling factor are
// one value a lane.  K and V tiles go straight into LDS, rows swizzled by
// 16-byte chunks; the values' operand is read transposed (ds_read_b64_tr_b16).
//
// Precision: scores, references and sums are FP32.  The weights are rounded to the
// tensors' type, what the second product's operand holds, and their sum takes the
// rounded ones: against 64 bits the result is 1.2 to 1.35 times as far off as its own
// last rounding makes it (bf16 0.0020 to 0.0022 of the norm, fp16 0.00024 to 0.00028).  Weights as two numbers, as
// over the pages, would double the second product, half of the matrix cores' work.
//
// Bound: the matrix cores (54 % of their cycles on 8192 tokens, 40 heads of
// 128: 624 to 666 us, 1.03 to 1.1 PFLOP/s, 82 to 87 % of what a large library product reaches;
// 24 heads of 256 733 to 764 us, 1.08 to 1.13 PFLOP/s) beside the softmax (41 % of the vector cycles) and LDS (40 %);
// heads of 64 by the softmax (64 % of the vector cycles, matrix cores 46 %: 371 to 395 us, 0.87 to 0.93 PFLOP/s), which is
// as long for half the products; short prompts by the
// 7 us that a workgroup's start and end take.  A step's three pieces of work are
// independent and laid out instruction by instruction, so that matrix and
// vector units of a SIMD work at once and no read of LDS is waited for; left to
// the compiler's order the same step took 710 instead of 656 us.
#include "attention_internal.h"

#include <float.h>

#include <algorithm>
#include <utility>

namespace pq2 {

namespace {

// Tiles of keys, and of values, in LDS; products that an operand is read ahead;
// 16-column pieces of the queries in LDS instead of registers (of 256 columns: or a SIMD
// holds one wave, which alone issues a vector instruction only every second time).
constexpr int bufs_of(int d, int waves) { return d == 256 || waves == 4 ? 2 : 4; }
constexpr int ahead_of(int d) { return d == 256 ? 3 : 4; }
constexpr int q_lds_of(int d) { return d == 256 ? 8 : 0; }
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.0f;      // weights grow by 2^8 before a row's reference moves
// A weight is exp2(score * scale - bias), bias the reference times the scale, one
// instruction for the exponent.  The bias is rounded, by a part of its size that moves all weights
// of the reference alike; beyond kFar the reference is taken off the scores first, or of
// 2^24 and more that part would be more than a 16-bit weight has room for.
constexpr float kFar = 1024.0f;

struct PromptArgs {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* out;
    int64_t q_stride, q_head, k_stride, k_head, v_stride, v_head, out_stride, out_head;
    const int32_t* starts_q;
    const int32_t* starts_k;
    int rows_q, rows_k, seqs, heads, group, window, causal;
    float scale2, slack;  // scale * log2(e); how far scores may pass a row's reference (in scores)
};

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// kRaise: weights are 2^kRaise for a score at the row's reference.  fp16 has
// room for 2^15, of which scores that pass the reference take 2^8; at 1, the weights
// below 2^-25 would be lost: thousands of them beside one leading key, a part of
// the result.
template <typename T> struct Half;
template <> struct Half<__bf16> {
    static constexpr float kRaise = 0.0f;
    typedef bf16x8 v8;
    typedef __bf16 v2 __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ v16f mfma(v8 a, v8 b, v16f c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }
    static __device__ __forceinline__ float add2(v2 e, float s) { return __builtin_amdgcn_fdot2_f32_bf16(e, v2{(__bf16)1.0f, (__bf16)1.0f}, s, false); }
};
template <> struct Half<_Float16> {
    static constexpr float kRaise = 7.0f;
    typedef f16x8 v8;
    typedef _Float16 v2 __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ v16f mfma(v8 a, v8 b, v16f c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }
    static __device__ __forceinline__ float add2(v2 e, float s) { return __builtin_amdgcn_fdot2(e, v2{(_Float16)1.0f, (_Float16)1.0f}, s, false); }
};

// 16-byte chunk c of row r of a tile, as it lies in LDS: keys are read 16 bytes
// a lane from neighbouring rows, values in stretches of 64 bytes from four
// neighbouring rows; both then meet different banks.
template <int D>
__device__ __forceinline__ int k_chunk(int r, int c) { return r * (D / 8) + (c ^ (r & 7)); }
template <int D>
__device__ __forceinline__ int v_chunk(int r, int c) {
    return r * (D / 8) + (c ^ ((D == 64 ? ((r >> 1) & 1) << 2 : (r & 3) << 2) | ((r >> 2) & 1) << 1));
}

__device__ __forceinline__ float max_halves(float v) {
    const uint32_t u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}

__device__ __forceinline__ float sum_halves(float v) {
    const uint32_t u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// 16 bytes a lane from a buffer straight into LDS: lane i's go to lds_addr +
// 16 i.  Its completion is waited for by wait_loads, not by the compiler.
__device__ __forceinline__ void load_lds(i32x4_t rsrc, uint32_t voff, uint32_t lds_addr) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds_addr), "v"(voff), "s"(rsrc)
                 : "memory", "m0");
}

// All but this wave's N most recent loads have arrived.
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N < 64, "vmcnt");
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);  // vmcnt(N)
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// f(0), f(1), ... f(N - 1), the index a constant in each.
template <typename F, int... I>
__device__ __forceinline__ void each_of(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F&& f) {
    each_of(f, std::make_integer_sequence<int, N>{});
}

// The first of a sequence's places among the workgroups of a key-value head:
// starts[s] * group / BM + s, enough for its tiles of BM rows, whatever the lengths.
template <int BM>
__device__ __forceinline__ int first_place(int start, int group, int s) { return (int)((uint32_t)(start * group) / BM) + s; }

// The sequence at `place`: the last one whose first place is not behind it, 64
// sequences a step of the search.
template <int BM>
__device__ __forceinline__ int sequence_at(const int32_t* starts, int group, int seqs, int place) {
    const int lane = threadIdx.x & 63;
    int lo = 0, count = seqs;
    while (true) {
        const int step = (count + 63) >> 6, at = lane * step;
        const bool below = at < count && first_place<BM>(starts[lo + at], group, lo + at) <= place;
        lo += max((int)__popcll(__ballot(below)) - 1, 0) * step;
        if (step == 1) return __builtin_amdgcn_readfirstlane(lo);
        count = min(step, seqs - lo);
    }
}

// Workgroups go to the eight XCDs in turn.  Each XCD takes one key-value head
// after the other, so that its keys and values stay in the XCD's L2, or, of fewer than eight
// heads, every 8 / kv_heads th tile of one (the longest tiles come first, so a stretch of
// them would be more work than the next); where that does not divide, tiles are dealt out in
// turn.
struct Item {
    int kvh, place;
};
__device__ __forceinline__ Item item_of(int id, int tiles, int kv_heads) {
    const int xcd = id & 7, turn = id >> 3;
    if (kv_heads <= 8 && 8 % kv_heads == 0) {
        const int share = 8 / kv_heads;
        return {xcd / share, turn * share + xcd % share};
    }
    if (kv_heads % 8 == 0) return {turn / tiles * 8 + xcd, turn % tiles};
    return {id % kv_heads, id / kv_heads};
}

template <int D, typename T, int W>
__global__ __launch_bounds__(64 * W, 2) void attention_prompt_kernel(PromptArgs a) {
    typedef typename Half<T>::v8 v8;
    typedef typename Half<T>::v2 v2;
    constexpr int BM = 32 * W;                   // query rows of a workgroup, 32 of them a wave's
    constexpr int DB = D / 32;
    constexpr int KT = D == 256 ? 32 : 64;       // keys of a step
    constexpr int KB = KT / 32, NF = KT / 16;    // in blocks of the scores, in operands of the weights
    constexpr int TILE = KT * D * 2;             // bytes of a tile in LDS
    constexpr int LOADS = TILE / 1024 / W;       // 1 KB loads of a wave for a tile
    constexpr int LROWS = 512 / D;               // rows of such a load
    constexpr int kBufs = bufs_of(D, W), kAhead = ahead_of(D), QR = D / 16 - q_lds_of(D);  // QR: pieces of q in registers
    extern __shared__ uint4 lds[];               // kBufs K tiles, kBufs V tiles, pieces of q

    const Item item = item_of(blockIdx.y * gridDim.x + blockIdx.x, gridDim.x, gridDim.y);
    const int kvh = item.kvh, place = item.place;
    const int seq = a.seqs == 1 ? 0 : sequence_at<BM>(a.starts_q, a.group, a.seqs, place);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane & 31, half = lane >> 5;
    // Queries and keys of the sequence, kept inside the tensors.
    const int qs = a.starts_q[seq], ks = a.starts_k[seq];
    const int nq = a.starts_q[seq + 1] - qs;
    // The longest tile first; places behind a sequence's last tile have no work.
    const int before = first_place<BM>(qs, a.group, seq);
    const int tile = (max(nq, 0) * a.group + BM - 1) / BM - 1 - (place - before);
    if (tile < 0 || place < before) return;
    const int nk = ks < 0 ? 0 : max(0, min(a.starts_k[seq + 1], a.rows_k) - ks);
    // Rows are queries, each with the grouped heads next to each other: a tile
    // holds few tokens, so that little of it lies behind a causal mask or a sequence's end.
    const int offset = nk - nq;  // a query's position is its index + offset
    const int q_first = tile * BM / a.group, q_last = min(nq - 1, (tile * BM + BM - 1) / a.group);
    const int hi = a.causal ? min(nk, offset + q_last + 1) : nk;
    const int lo = a.window ? max(0, offset + q_first - a.window + 1) & ~(KT - 1) : 0;

    const int r0 = tile * BM + 32 * wave, qi = (r0 + row) / a.group, head = kvh * a.group + (r0 + row) % a.group;
    const bool valid = qi < nq && qs + qi >= 0 && qs + qi < a.rows_q;
    v8 qf[QR];
    uint4* q_lds = lds + 2 * kBufs * (TILE / 16) + wave * 64 + lane;
    {
        const uint16_t* q = a.q + (int64_t)(valid ? qs + qi : 0) * a.q_stride + head * a.q_head + 8 * half;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
            const v8 x = *reinterpret_cast<const v8*>(q + 16 * s), y = valid ? x : v8{};
            if (s < QR) qf[s] = y;
            else q_lds[(s - QR) * 64 * W] = __builtin_bit_cast(uint4, y);
        }
    }
    typedef __attribute__((address_space(3))) char lds_char;
    lds_char* qat = (lds_char*)q_lds;
    auto query = [&](int s) -> v8 { return *(__attribute__((address_space(3))) v8*)(qat + (s - QR) * 1024 * W); };
    // Keys that this row, and the wave's rows all together, see.
    const int seen_hi = a.causal ? min(nk, qi + offset + 1) : nk;
    const int seen_lo = a.window ? qi + offset - a.window + 1 : 0;
    const int all_hi = a.causal ? min(nk, r0 / a.group + offset + 1) : nk;
    const int all_lo = a.window ? (r0 + 31) / a.group + offset - a.window + 1 : 0;

    // Loads: chunk `lane` of load i of this wave is row lrow + i * W * LROWS of
    // the tile (a multiple of eight apart: one swizzle).  Rows behind the last key repeat it.
    const uint16_t* kbase = a.k + (int64_t)ks * a.k_stride + kvh * a.k_head;
    const uint16_t* vbase = a.v + (int64_t)ks * a.v_stride + kvh * a.v_head;
    const int lrow = wave * LROWS + lane / (D / 8), lcol = lane % (D / 8);
    const uint32_t kcol = 16 * (k_chunk<D>(lrow, lcol) - lrow * (D / 8));
    const uint32_t vcol = 16 * (v_chunk<D>(lrow, lcol) - lrow * (D / 8));
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint4*)lds;
    auto fetch = [&](const uint16_t* base, int64_t stride, uint32_t col, int key0, uint32_t to) {
        const i32x4_t r = make_srsrc(base + (int64_t)key0 * stride, 0x7FFFFFFFu);
        const int last = nk - 1 - key0;
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            load_lds(r, (uint32_t)min(lrow + i * W * LROWS, last) * (uint32_t)(stride * 2) + col,
                     lds0 + to + 1024 * (wave + i * W));
    };

    v16f acc[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d) acc[d] = v16f{};
    float m = -INFINITY, l = 0.0f;
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    u32x4 p[NF];  // the weights, 16 keys each, as operands
#pragma unroll
    for (int f = 0; f < NF; ++f) p[f] = u32x4{};

    // Operand i of a step's products: the values' (b, t, d) for the last tile's
    // weights, then the keys' (s, b) for the next tile's scores.  A lane's place
    // depends on the swizzle in four ways; the rest is a constant offset.
    constexpr int PV = NF * DB, N = 2 * PV, RB = 2 * D;  // RB: bytes of a row
    lds_char* kat[4];
    lds_char* vat[DB < 4 ? DB : 4];
    {
        const int r3 = (lane & 15) / 4, swz = D == 64 ? r3 >> 1 : r3;
#pragma unroll
        for (int x = 0; x < 4; ++x) kat[x] = (lds_char*)lds + row * RB + 16 * ((2 * x + half) ^ (row & 7));
#pragma unroll
        for (int x = 0; x < (DB < 4 ? DB : 4); ++x)
            vat[x] = (lds_char*)lds + kBufs * TILE + (4 * half + r3) * RB +
                     16 * (4 * (x ^ swz) + 2 * (((lane >> 4) & 1) ^ half) + ((lane & 3) >> 1)) + 8 * (lane & 1);
    }
    auto operand = [&](int i, int buf) -> v8 {
        if (i < PV) {
            const int d = i % DB, bt = i / DB;
            lds_char* at = vat[d % 4] + buf * TILE + 16 * bt * RB + 256 * (d / 4);
            const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)at);
            const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at + 8 * RB));
            return __builtin_bit_cast(v8, (s16x8)__builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
        }
        const int s = (i - PV) / KB, b = i % KB;
        return *(__attribute__((address_space(3))) v8*)(kat[s % 4] + buf * TILE + 32 * b * RB + 128 * (s / 4));
    };
    auto weights = [&](int f) { return __builtin_bit_cast(v8, p[f]); };
    auto mask = [&](int key0, v16f (&s2)[KB]) {
        if (key0 + KT <= all_hi && key0 >= all_lo) return;
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int key = key0 + 32 * b + 8 * (r / 4) + 4 * half + r % 4;
                if (key >= seen_hi || key < seen_lo) s2[b][r] = -INFINITY;
            }
    };
    // One step: this tile's softmax (sc -> p), the last tile's values and the
    // next tile's scores (-> next), which do not need each other, in turns.
    // Operands are read kAhead products ahead; a piece of p is written behind
    // its last use for the last tile.  Keys kBufs tiles ahead and values kBufs - 2
    // ahead go into the buffers that the step before read last, and are waited for kBufs - 2
    // steps later (behind the last tile it is loaded again, so that the count
    // of loads on their way is always the same).
    const int last_tile = lo + (hi - 1 - lo) / KT * KT;
    auto fetch_k = [&](int key0, int buf) { fetch(kbase, a.k_stride, kcol, min(key0, last_tile), buf * TILE); };
    auto fetch_v = [&](int key0, int buf) { fetch(vbase, a.v_stride, vcol, min(key0, last_tile), (kBufs + buf) * TILE); };
    auto step = [&](int key0, auto at_buf, v16f (&sc)[KB], v16f (&next)[KB]) {
        constexpr int buf = decltype(at_buf)::value;       // of this tile
        constexpr int kbuf = (buf + 1) % kBufs, vbuf = (buf + kBufs - 1) % kBufs;
        v8 ring[kAhead], q_ring[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) ring[i] = operand(i, vbuf);
        fetch_k(key0 + kBufs * KT, buf);
        fetch_v(key0 + (kBufs - 2) * KT, (buf + kBufs - 2) % kBufs);
        float top = -INFINITY, alpha = 1.0f, bias = 0.0f;
        each<N>([&](auto at) {
            constexpr int i = decltype(at)::value;
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (i < PV) acc[i % DB] = Half<T>::mfma(ring[i % kAhead], weights(i / DB), acc[i % DB]);
            else {
                constexpr int qs = (i - PV) / KB;
                next[i % KB] = Half<T>::mfma(ring[i % kAhead], qs < QR ? qf[qs < QR ? qs : 0] : q_ring[i % kAhead],
                                             i < PV + KB ? v16f{} : next[i % KB]);
            }
            if constexpr (i + kAhead < N) {
                constexpr int ahead = i + kAhead, qs = (ahead - PV) / KB;
                ring[i % kAhead] = operand(ahead, ahead < PV ? vbuf : kbuf);
                if constexpr (ahead >= PV && qs >= QR) q_ring[i % kAhead] = query(qs);
            }
            if constexpr (i < N / 4) {
                constexpr int E = 64 * KB / N;  // scores a product
#pragma unroll
                for (int e = i * E; e < i * E + E; ++e) top = fmaxf(top, sc[e / 16][e % 16]);
            } else if constexpr (i == N / 4) {
                top = max_halves(top);
                const float old = m;
                if (top > m + a.slack) m = top;
                const float ref = m == -INFINITY ? 0.0f : m;
                alpha = __builtin_amdgcn_exp2f((old - ref) * a.scale2);
                bias = ref * a.scale2;
                if (__any(fabsf(bias) > kFar)) {
#pragma unroll
                    for (int e = 0; e < 16 * KB; ++e) sc[e / 16][e % 16] -= ref;
                    bias = 0.0f;
                }
                bias -= Half<T>::kRaise;
                l *= alpha;
            } else {
#pragma unroll
                for (int k = 0; k < 8 * KB; ++k) {
                    if (N / 4 + 1 + k * (3 * N / 4 - 1) / (8 * KB) != i) continue;
                    const int b = k / 8, r = k % 8 * 2;
                    const v2 e = {(T)__builtin_amdgcn_exp2f(__builtin_fmaf(sc[b][r], a.scale2, -bias)),
                                  (T)__builtin_amdgcn_exp2f(__builtin_fmaf(sc[b][r + 1], a.scale2, -bias))};
                    l = Half<T>::add2(e, l);
                    uint32_t w = __builtin_bit_cast(uint32_t, e);
                    asm volatile("" : "+v"(w));  // formed here, not where it is used
                    p[k / 4][k % 4] = w;
                }
            }
        });
        __builtin_amdgcn_sched_barrier(0);
        if (__any(alpha != 1.0f)) {
            float f = alpha;
            asm volatile("" : "+v"(f));  // or the products would be formed ahead of the branch
#pragma unroll
            for (int d = 0; d < DB; ++d) acc[d] *= f;
        }
        mask(key0 + KT, next);
        wait_loads<(kBufs - 2) * 2 * LOADS>();
        __syncthreads();
    };

    if (lo < hi) {
        // Values before the first tile: zeros, for the first step's product.
        for (int i = threadIdx.x; i < TILE / 16; i += 64 * W) lds[(2 * kBufs - 1) * (TILE / 16) + i] = make_uint4(0, 0, 0, 0);
        fetch_k(lo, 0);
        fetch_k(lo + KT, 1);
#pragma unroll
        for (int i = 0; i < kBufs - 2; ++i) {
            fetch_k(lo + (2 + i) * KT, 2 + i);
            fetch_v(lo + i * KT, i);
        }
        wait_loads<(kBufs - 2) * 2 * LOADS>();
        __syncthreads();
        v16f even[KB], odd[KB];
        each<PV>([&](auto at) {
            constexpr int i = PV + decltype(at)::value;
            constexpr int qs = (i - PV) / KB;
            v8 q;
            if constexpr (qs < QR) q = qf[qs];
            else q = query(qs);
            even[i % KB] = Half<T>::mfma(operand(i, 0), q, i < PV + KB ? v16f{} : even[i % KB]);
        });
        mask(lo, even);
        __syncthreads();
        int key0 = lo, last = 0;
        auto behind = [&](int buf) {
            key0 += KT;
            last = buf;
            return key0 >= hi;
        };
        while (true) {
            step(key0, std::integral_constant<int, 0>{}, even, odd);
            if (behind(0)) break;
            step(key0, std::integral_constant<int, 1>{}, odd, even);
            if (behind(1)) break;
            if constexpr (kBufs == 4) {
                step(key0, std::integral_constant<int, 2>{}, even, odd);
                if (behind(2)) break;
                step(key0, std::integral_constant<int, 3>{}, odd, even);
                if (behind(3)) break;
            }
        }
        each<PV>([&](auto at) {
            constexpr int i = decltype(at)::value;
            acc[i % DB] = Half<T>::mfma(operand(i, last), weights(i / DB), acc[i % DB]);
        });
        wait_loads<0>();  // none may reach LDS behind the workgroup's end
    }

    l = sum_halves(l);
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    if (!valid) return;
    uint16_t* out = a.out + (int64_t)(qs + qi) * a.out_stride + head * a.out_head;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const uint32_t lo2 = __builtin_bit_cast(uint32_t, v2{(T)(acc[d][4 * x] * inv), (T)(acc[d][4 * x + 1] * inv)});
            const uint32_t hi2 = __builtin_bit_cast(uint32_t, v2{(T)(acc[d][4 * x + 2] * inv), (T)(acc[d][4 * x + 3] * inv)});
            *reinterpret_cast<uint2*>(out + 32 * d + 8 * x + 4 * half) = make_uint2(lo2, hi2);
        }
}

template <int D, typename T, int W>
void start(PromptArgs a, hipStream_t stream) {
    // (A multiple of eight, for shares of any size.)
    const int tiles = ((int)(((int64_t)a.rows_q * a.group + 32 * W - 1) / (32 * W)) + a.seqs + 7) & ~7;
    const size_t lds = 2 * bufs_of(D, W) * (size_t)(D == 256 ? 32 : 64) * D * 2 + (size_t)q_lds_of(D) * 1024 * W;
    hipLaunchKernelGGL((attention_prompt_kernel<D, T, W>), dim3((unsigned)tiles, (unsigned)(a.heads / a.group)), dim3(64 * W), lds, stream, a);
}

// Workgroups of four waves, of which several share a compute unit (one starts
// while another computes), or of eight, one a unit, which read each tile of keys for twice
// the rows. us with four / eight, 40 heads of 128: 24 prompts of 500 tokens 134 / 155, one of 2048 66 / 68,
// of 3000 116 / 113, of 4096 186 / 187, of 6000 359 / 349, of 8192 639 / 620 (around 4096 it makes no difference); 24 heads of 256 (four: one workgroup a unit all the same):
// one of 1024 40 / 56, of 2048 71 / 97, four of 1500 151 / 145, 24 of 500 171 / 156; 40 heads of 64: 8192 tokens 380 / 410.
template <typename T>
void start(const PromptArgs& a, int d, hipStream_t stream) {
    const int64_t rows = (int64_t)a.rows_q * a.heads;
    if (d == 64) start<64, T, 4>(a, stream);
    else if (d == 128) rows >= 128 << 10 && a.rows_k >= (int64_t)4096 * a.seqs ? start<128, T, 8>(a, stream) : start<128, T, 4>(a, stream);
    else rows >= 64 << 10 ? start<256, T, 8>(a, stream) : start<256, T, 4>(a, stream);
}

}  // namespace

hipError_t launch_attention_prompt(const pq2_attention_prompt_args& a, hipStream_t stream) {
    const float scale2 = a.scale * kLog2e;
    // (Finite: -inf + slack, for a row's first keys, is to stay -inf.)
    const float slack = std::min(kSlack / scale2, FLT_MAX);
    const PromptArgs k{static_cast<const uint16_t*>(a.q), static_cast<const uint16_t*>(a.k),
                       static_cast<const uint16_t*>(a.v), static_cast<uint16_t*>(a.out), a.q_stride, a.q_head, a.k_stride,
                       a.k_head, a.v_stride, a.v_head, a.out_stride, a.out_head, a.starts_q, a.starts_k, (int)a.rows_q,
                       (int)a.rows_k, (int)a.seqs, (int)a.heads, (int)(a.heads / a.kv_heads),
                       (int)std::min<int64_t>(a.window, 0x40000000), a.causal, scale2, slack};
    clear_stale_error();
    a.dtype == PQ2_F16 ? start<_Float16>(k, (int)a.head_dim, stream) : start<__bf16>(k, (int)a.head_dim, stream);
    return hipGetLastError();
}

}  // namespace pq2
