// attention_prompt.hip -- attention over packed prompts (pq2_attention_prompt).
//
// Mathematics: a workgroup takes 128 query rows of one head, a wave 32 of
// them, and runs over the keys 64 at a time with the softmax's running maximum
// and sum.  Scores are transposed, keys x rows: S^T = K Q^T with
// v_mfma_f32_32x32x16, whose result registers 8t .. 8t + 7 of a lane are, as
// they stand, the weights operand of one step of o^T = V^T P^T (the order of
// the keys inside a step is free, the values are read in the same order): the weights
// never leave their lane, and a row's maximum, sum and rescaling factor are
// one value a lane.  K and V tiles go through LDS, rows swizzled by 16-byte
// chunks; the values' operand is read transposed (ds_read_b64_tr_b16).
#include "attention_internal.h"

#include <algorithm>

namespace pq2 {

namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kBM = 32 * kWaves;    // query rows of a workgroup
constexpr int kKeys = 64;           // keys of a step
constexpr float kLog2e = 1.4426950408889634f;

struct PromptArgs {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* out;
    int64_t q_stride, q_head, k_stride, k_head, v_stride, v_head, out_stride, out_head;
    const int32_t* starts_q;
    const int32_t* starts_k;
    int rows_q, rows_k, seqs, group, window, causal;
    float scale2;
};

typedef short s16x4 __attribute__((ext_vector_type(4)));

template <typename T> struct Half;
template <> struct Half<__bf16> {
    typedef bf16x8 v8;
    typedef __bf16 v2 __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ v16f mfma(v8 a, v8 b, v16f c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }
};
template <> struct Half<_Float16> {
    typedef f16x8 v8;
    typedef _Float16 v2 __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ v16f mfma(v8 a, v8 b, v16f c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }
};

// 16-byte chunk c of row r of a tile, as it lies in LDS: keys are read 16 bytes
// a lane from neighbouring rows, values in stretches of 64 bytes from four
// neighbouring rows; both then meet different banks.
template <int D>
__device__ __forceinline__ int k_chunk(int r, int c) { return r * (D / 8) + (c ^ (r & 7)); }
template <int D>
__device__ __forceinline__ int v_chunk(int r, int c) {
    return r * (D / 8) + (c ^ (D == 64 ? ((r >> 1) & 1) << 2 : (r & 3) << 2));
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

// The sequence and query tile of a workgroup: tiles are counted through the
// sequences, 64 of them a step; seq < 0 behind the last tile.
struct Place {
    int seq, tile, tiles;
};

__device__ __forceinline__ Place place_of(const int32_t* starts, int seqs, int index) {
    const int lane = threadIdx.x & 63;
    for (int s0 = 0; s0 < seqs; s0 += 64) {
        const int s = s0 + lane;
        int tiles = 0;
        if (s < seqs) tiles = (max(starts[s + 1] - starts[s], 0) + kBM - 1) / kBM;
        int sum = tiles;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(sum, d);
            if (lane >= d) sum += o;
        }
        const int total = __shfl(sum, 63);
        if (index < total) {
            const int at = __ffsll(__ballot(sum > index)) - 1;
            return {s0 + at, index - (__shfl(sum, at) - __shfl(tiles, at)), __shfl(tiles, at)};
        }
        index -= total;
    }
    return {-1, 0, 0};
}

template <int D, typename T>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void attention_prompt_kernel(PromptArgs a) {
    typedef typename Half<T>::v8 v8;
    typedef typename Half<T>::v2 v2;
    constexpr int CH = kKeys * D / 8;          // chunks of a tile
    constexpr int PER = CH / kThreads;         // of them a thread's
    constexpr int DB = D / 32;
    extern __shared__ uint4 lds[];             // [2][K tile, V tile]

    const Place place = place_of(a.starts_q, a.seqs, blockIdx.x);
    if (place.seq < 0) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int row = lane & 31, half = lane >> 5;
    const int seq = __builtin_amdgcn_readfirstlane(place.seq);
    const int tile = __builtin_amdgcn_readfirstlane(place.tiles - 1 - place.tile);  // the longest first
    const int head = blockIdx.y, kvh = head / a.group;

    // Queries and keys of the sequence, kept inside the tensors.
    const int qs = a.starts_q[seq], ks = a.starts_k[seq];
    const int nq = a.starts_q[seq + 1] - qs;
    const int nk = ks < 0 ? 0 : max(0, min(a.starts_k[seq + 1], a.rows_k) - ks);
    const int q0 = tile * kBM;
    const int offset = nk - nq;  // a query's position is its index + offset
    const int hi = a.causal ? min(nk, offset + min(q0 + kBM, nq)) : nk;
    const int lo = a.window ? max(0, offset + q0 - a.window + 1) & ~(kKeys - 1) : 0;

    const int qi = q0 + 32 * wave + row;
    const bool valid = qi < nq && qs + qi >= 0 && qs + qi < a.rows_q;
    v8 qf[D / 16];
    if (valid) {
        const uint16_t* q = a.q + (int64_t)(qs + qi) * a.q_stride + head * a.q_head + 8 * half;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) qf[s] = *reinterpret_cast<const v8*>(q + 16 * s);
    } else {
#pragma unroll
        for (int s = 0; s < D / 16; ++s) qf[s] = v8{};
    }
    // Keys that this row, and the wave's rows all together, see.
    const int seen_hi = a.causal ? min(nk, qi + offset + 1) : nk;
    const int seen_lo = a.window ? qi + offset - a.window + 1 : 0;
    const int wave_first = q0 + 32 * wave + offset;
    const int all_hi = a.causal ? min(nk, wave_first + 1) : nk;
    const int all_lo = a.window ? wave_first + 31 - a.window + 1 : 0;

    uint4 stage[2][PER];
    const uint16_t* kbase = a.k + (int64_t)ks * a.k_stride + kvh * a.k_head;
    const uint16_t* vbase = a.v + (int64_t)ks * a.v_stride + kvh * a.v_head;
    auto records = [&](int key0, int64_t stride) {
        const int64_t rows = nk - key0;
        return rows <= 0 ? 0u : (uint32_t)min((rows - 1) * stride * 2 + D * 2, (int64_t)0x7FFFFFFF);
    };
    auto fetch = [&](int key0) {
        const auto rk = make_rsrc(kbase + (int64_t)key0 * a.k_stride, records(key0, a.k_stride));
        const auto rv = make_rsrc(vbase + (int64_t)key0 * a.v_stride, records(key0, a.v_stride));
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = threadIdx.x + i * kThreads, r = c / (D / 8), col = c % (D / 8);
            stage[0][i] = buf_load16(rk, (uint32_t)r * (uint32_t)(a.k_stride * 2) + col * 16);
            stage[1][i] = buf_load16(rv, (uint32_t)r * (uint32_t)(a.v_stride * 2) + col * 16);
        }
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = threadIdx.x + i * kThreads, r = c / (D / 8), col = c % (D / 8);
            lds[buf * 2 * CH + k_chunk<D>(r, col)] = stage[0][i];
            lds[buf * 2 * CH + CH + v_chunk<D>(r, col)] = stage[1][i];
        }
    };

    v16f acc[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d) acc[d] = v16f{};
    float m = -INFINITY, l = 0.0f;

    if (lo < hi) {
        fetch(lo);
        put(0);
    }
    int buf = 0;
    for (int key0 = lo; key0 < hi; key0 += kKeys, buf ^= 1) {
        const bool more = key0 + kKeys < hi;
        if (more) fetch(key0 + kKeys);
        __syncthreads();
        const uint4* kt = lds + buf * 2 * CH;
        const uint4* vt = kt + CH;
        v16f sc[2] = {};
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
            for (int b = 0; b < 2; ++b)
                sc[b] = Half<T>::mfma(__builtin_bit_cast(v8, kt[k_chunk<D>(32 * b + row, 2 * s + half)]), qf[s], sc[b]);
        if (key0 + kKeys > all_hi || key0 < all_lo) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int key = key0 + 32 * b + 8 * (r / 4) + 4 * half + r % 4;
                    if (key >= seen_hi || key < seen_lo) sc[b][r] = -INFINITY;
                }
        }
        float top = -INFINITY;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, sc[b][r]);
        // (scale2 may be negative or zero: the maximum is of the scaled scores.)
        top = fmaxf(m, max_halves(top));
        const float ref = top == -INFINITY ? 0.0f : top;
        const float alpha = __builtin_amdgcn_exp2f((m - ref) * a.scale2);
        const float bias = ref * a.scale2;
        m = top;
        l *= alpha;
#pragma unroll
        for (int d = 0; d < DB; ++d) acc[d] *= alpha;
        v8 p[2][2];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const T e = (T)__builtin_amdgcn_exp2f(__builtin_fmaf(sc[b][r], a.scale2, -bias));
                l += (float)e;
                p[b][r / 8][r % 8] = e;
            }
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    s16x4 part[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int vr = 32 * b + 16 * t + 8 * x + 4 * half + (lane & 15) / 4;
                        const int col = 32 * d + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
                        const char* at = reinterpret_cast<const char*>(vt + v_chunk<D>(vr, col / 8)) + 2 * (col % 8);
                        part[x] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                            (__attribute__((address_space(3))) s16x4*)(at));
                    }
                    typedef short s16x8 __attribute__((ext_vector_type(8)));
                    const s16x8 v = __builtin_shufflevector(part[0], part[1], 0, 1, 2, 3, 4, 5, 6, 7);
                    acc[d] = Half<T>::mfma(__builtin_bit_cast(v8, v), p[b][t], acc[d]);
                }
        if (more) put(buf ^ 1);
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

template <int D, typename T>
void start(const PromptArgs& a, int heads, hipStream_t stream) {
    const dim3 grid((unsigned)((a.rows_q + kBM - 1) / kBM + a.seqs), (unsigned)heads);
    const size_t lds = 4 * (size_t)kKeys * D * 2;
    hipLaunchKernelGGL((attention_prompt_kernel<D, T>), grid, dim3(kThreads), lds, stream, a);
}

}  // namespace

hipError_t launch_attention_prompt(const pq2_attention_prompt_args& a, hipStream_t stream) {
    const PromptArgs k{static_cast<const uint16_t*>(a.q), static_cast<const uint16_t*>(a.k),
                       static_cast<const uint16_t*>(a.v), static_cast<uint16_t*>(a.out), a.q_stride, a.q_head, a.k_stride,
                       a.k_head, a.v_stride, a.v_head, a.out_stride, a.out_head, a.starts_q, a.starts_k, (int)a.rows_q,
                       (int)a.rows_k, (int)a.seqs, (int)(a.heads / a.kv_heads),
                       (int)std::min<int64_t>(a.window, 0x40000000), a.causal, a.scale * kLog2e};
    clear_stale_error();
    const bool f16 = a.dtype == PQ2_F16;
    if (a.head_dim == 64) f16 ? start<64, _Float16>(k, (int)a.heads, stream) : start<64, __bf16>(k, (int)a.heads, stream);
    else if (a.head_dim == 128) f16 ? start<128, _Float16>(k, (int)a.heads, stream) : start<128, __bf16>(k, (int)a.heads, stream);
    else f16 ? start<256, _Float16>(k, (int)a.heads, stream) : start<256, __bf16>(k, (int)a.heads, stream);
    return hipGetLastError();
}

}  // namespace pq2
