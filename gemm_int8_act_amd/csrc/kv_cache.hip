// kv_cache.hip -- the paged INT8 key-value cache: rotary embedding and codes of
// new tokens into its pages (pq2_kv_write), tokens out of them again
// (pq2_kv_read).
//
// Both move bytes: a row of head_dim elements is read once and written once,
// and the arithmetic between (a rotation, a maximum over the row, eight
// quotients a lane) hides behind memory for many tokens.  For one token the
// time is the launch and two dependent trips to memory (position, then its row
// of the tables; the row itself loads meanwhile).  Measured: 4096 tokens of 64 + 8 +
// 8 heads of 128 from FP32, q, k and v out in bf16, 48.5 us (265 MB, 5.4 TB/s);
// 32768 tokens of 8 heads of 128 read back to bf16 41 to 47 us (203 MB, 4.3 to 5.0 TB/s);
// one token 3 us either way.
#include "attention_internal.h"

#include <algorithm>

namespace pq2 {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxGridX = 1 << 20;
constexpr int64_t kFewElements = 4 << 20;

struct HeadRows {
    const void* p;
    int64_t stride, head;
};

struct WriteArgs {
    HeadRows in[3];   // q, k, v
    HeadRows out[3];  // p null: none
    const float* cos;
    const float* sin;
    const int32_t* positions;
    const int32_t* slots;
    uint8_t* cache;
    int m, heads, kv_heads, rot, last_row, parts, page_shift;
    int64_t slots_end;
    int in_dtype, out_dtype, interleaved;
};

// Four consecutive elements from element i of p (16-byte multiples apart).
__device__ __forceinline__ void load4(const void* p, int64_t i, int dtype, float* v) {
    if (dtype == PQ2_F32) {
        const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
        return;
    }
    const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
    if (dtype == PQ2_BF16) {
        v[0] = __uint_as_float(x.x << 16), v[1] = __uint_as_float(x.x & 0xFFFF0000u);
        v[2] = __uint_as_float(x.y << 16), v[3] = __uint_as_float(x.y & 0xFFFF0000u);
    } else {
        v[0] = half_bits(x.x & 0xFFFFu), v[1] = half_bits(x.x >> 16);
        v[2] = half_bits(x.y & 0xFFFFu), v[3] = half_bits(x.y >> 16);
    }
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    typedef T T2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, T2{(T)a, (T)b});
}

__device__ __forceinline__ void store4(const void* p, int64_t i, int dtype, const float* v) {
    if (dtype == PQ2_F32) {
        *reinterpret_cast<float4*>(static_cast<float*>(const_cast<void*>(p)) + i) = make_float4(v[0], v[1], v[2], v[3]);
        return;
    }
    const uint2 x = dtype == PQ2_BF16 ? make_uint2(pack2<__bf16>(v[0], v[1]), pack2<__bf16>(v[2], v[3]))
                                      : make_uint2(pack2<_Float16>(v[0], v[1]), pack2<_Float16>(v[2], v[3]));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(const_cast<void*>(p)) + i) = x;
}

// D / 8 lanes hold a row, each two stretches of four elements: for a rotation
// by halves the two elements of a pair are in one lane (elements 4j.. and
// rot/2 + 4j..), the rest of the row, and rows rotated in neighbouring pairs,
// as eight consecutive elements.  A workgroup takes one token, its groups of
// lanes every (groups * parts)th of the token's rows.
template <int D>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(WriteArgs a) {
#pragma clang fp contract(off)
    constexpr int LPR = D / 8, GROUPS = kThreads / LPR;
    const int j = threadIdx.x % LPR, group = threadIdx.x / LPR;
    const int rows = a.heads + 2 * a.kv_heads;
    const bool turns = 8 * j < a.rot;
    const bool halves = turns && !a.interleaved;
    const int o1 = halves ? 4 * j : 8 * j, o2 = halves ? a.rot / 2 + 4 * j : 8 * j + 4;
    for (int t = blockIdx.x; t < a.m; t += gridDim.x) {
        float c[4] = {}, s[4] = {};
        if (turns) {
            const int p = min(max(a.positions[t], 0), a.last_row);
            load4(a.cos, (int64_t)p * (a.rot / 2) + 4 * j, PQ2_F32, c);
            load4(a.sin, (int64_t)p * (a.rot / 2) + 4 * j, PQ2_F32, s);
        }
        const int64_t slot = a.cache ? a.slots[t] : -1;
        for (int r = blockIdx.y * GROUPS + group; r < rows; r += GROUPS * a.parts) {
            const int which = r < a.heads ? 0 : r < a.heads + a.kv_heads ? 1 : 2;
            const int h = which == 0 ? r : which == 1 ? r - a.heads : r - a.heads - a.kv_heads;
            const HeadRows in = a.in[which], out = a.out[which];
            float v[8];
            const int64_t at = t * in.stride + h * in.head;
            load4(in.p, at + o1, a.in_dtype, v);
            load4(in.p, at + o2, a.in_dtype, v + 4);
            if (turns && which != 2) {
                if (a.interleaved) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = v[2 * i], y = v[2 * i + 1];
                        v[2 * i] = x * c[i] - y * s[i];
                        v[2 * i + 1] = y * c[i] + x * s[i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = v[i], y = v[i + 4];
                        v[i] = x * c[i] - y * s[i];
                        v[i + 4] = y * c[i] + x * s[i];
                    }
                }
            }
            if (out.p) {
                const int64_t to = t * out.stride + h * out.head;
                store4(out.p, to + o1, a.out_dtype, v);
                store4(out.p, to + o2, a.out_dtype, v + 4);
            }
            if (which == 0 || slot < 0 || slot >= a.slots_end) continue;
            float amax = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
            amax = LPR == 8 ? max8_f(amax) : max16_f(amax);
            if constexpr (LPR == 32) amax = fmaxf(amax, __shfl_xor(amax, 16));
            float scale;
            uint32_t bits[8];
            quantise_bits(v, amax, scale, bits);
            const int64_t page = slot >> a.page_shift, tok = slot & ((1 << a.page_shift) - 1);
            uint8_t* block = a.cache + (page * a.kv_heads + h) * (kv_block_bytes(1, D) << a.page_shift);
            uint8_t* codes = block + (((int64_t)(which - 1) << a.page_shift) + tok) * D;
            *reinterpret_cast<uint32_t*>(codes + o1) = code_bytes(bits, 0);
            *reinterpret_cast<uint32_t*>(codes + o2) = code_bytes(bits, 4);
            if (j == 0)
                reinterpret_cast<float*>(block + ((int64_t)(2 * D) << a.page_shift))[((which - 1) << a.page_shift) + tok] = scale;
        }
    }
}

struct ReadArgs {
    const uint8_t* cache;
    const int32_t* table;
    const int32_t* starts;
    HeadRows out[2];  // k, v
    int64_t table_stride;
    int rows, seqs, table_pages, kv_heads, pages, page_shift, out_dtype;
};

// E elements of a row a lane, 16 bytes of output; a workgroup takes U times
// kThreads / (D / E) rows of one head, keys and values, all their loads at once.
template <int D, int E, int U>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(ReadArgs a) {
    constexpr int LPR = D / E, RB = kThreads / LPR;
    const int j = threadIdx.x % LPR, h = blockIdx.y;
    for (int64_t row0 = (int64_t)blockIdx.x * (RB * U); row0 < a.rows; row0 += (int64_t)gridDim.x * (RB * U)) {
        const int end = min(a.rows, a.starts[a.seqs]);
        int s = a.seqs == 1 ? 0 : sequence_of(a.starts, a.seqs, (int)row0);
        uint32_t code[U][2][E / 4] = {};
        float scale[U][2] = {};
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = (int)row0 + u * RB + threadIdx.x / LPR;
            if (row >= end) continue;
            while (s + 1 < a.seqs && a.starts[s + 1] <= row) ++s;
            const int t = row - a.starts[s], idx = t >> a.page_shift, tok = t & ((1 << a.page_shift) - 1);
            const int page = t >= 0 && idx < a.table_pages ? a.table[s * a.table_stride + idx] : -1;
            if (page < 0 || page >= a.pages) continue;
            const uint8_t* block = a.cache + ((int64_t)page * a.kv_heads + h) * (kv_block_bytes(1, D) << a.page_shift);
            const float* scales = reinterpret_cast<const float*>(block + ((int64_t)(2 * D) << a.page_shift));
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const uint8_t* codes = block + (((int64_t)w << a.page_shift) + tok) * D + j * E;
                scale[u][w] = scales[(w << a.page_shift) + tok];
#pragma unroll
                for (int i = 0; i < E / 4; ++i) code[u][w][i] = reinterpret_cast<const uint32_t*>(codes)[i];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = (int)row0 + u * RB + threadIdx.x / LPR;
            if (row >= end) continue;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                float v[E];
#pragma unroll
                for (int i = 0; i < E; ++i) v[i] = (float)(int8_t)(code[u][w][i / 4] >> (8 * (i % 4))) * scale[u][w];
                const int64_t to = row * a.out[w].stride + h * a.out[w].head + j * E;
                if constexpr (E == 4) {
                    store4(a.out[w].p, to, PQ2_F32, v);
                } else {
                    const uint4 x = a.out_dtype == PQ2_BF16
                                        ? make_uint4(pack2<__bf16>(v[0], v[1]), pack2<__bf16>(v[2], v[3]),
                                                     pack2<__bf16>(v[4], v[5]), pack2<__bf16>(v[6], v[7]))
                                        : make_uint4(pack2<_Float16>(v[0], v[1]), pack2<_Float16>(v[2], v[3]),
                                                     pack2<_Float16>(v[4], v[5]), pack2<_Float16>(v[6], v[7]));
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(const_cast<void*>(a.out[w].p)) + to) = x;
                }
            }
        }
    }
}

template <int D>
void start_write(const WriteArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)std::min<int64_t>(a.m, kMaxGridX), (unsigned)a.parts);
    hipLaunchKernelGGL((kv_write_kernel<D>), grid, dim3(kThreads), 0, stream, a);
}

template <int D, int E, int U>
void start_read(const ReadArgs& a, hipStream_t stream) {
    const int rb = U * kThreads * E / D;
    const dim3 grid((unsigned)std::min<int64_t>((a.rows + rb - 1) / rb, kMaxGridX), (unsigned)a.kv_heads);
    hipLaunchKernelGGL((kv_read_kernel<D, E, U>), grid, dim3(kThreads), 0, stream, a);
}

// Few rows: one a lane, over as many workgroups as there are. Many: two (32768
// tokens of 8 heads of 128 to bf16 47 us; one 54, four 49, eight 55).
template <int D>
void start_read(const ReadArgs& a, hipStream_t stream) {
    const bool few = (int64_t)a.rows * a.kv_heads * D < kFewElements;
    if (a.out_dtype == PQ2_F32) few ? start_read<D, 4, 1>(a, stream) : start_read<D, 4, 2>(a, stream);
    else few ? start_read<D, 8, 1>(a, stream) : start_read<D, 8, 2>(a, stream);
}

}  // namespace

hipError_t launch_kv_write(const pq2_kv_write_args& a, hipStream_t stream) {
    const int heads = a.q ? (int)a.heads : 0;
    const int groups = kThreads * 8 / (int)a.head_dim;
    const int rows = heads + 2 * (int)a.kv_heads;
    WriteArgs k{{{a.q, a.q_stride, a.q_head}, {a.k, a.k_stride, a.k_head}, {a.v, a.v_stride, a.v_head}},
                {{a.q_out, a.qo_stride, a.qo_head}, {a.k_out, a.ko_stride, a.ko_head}, {a.v_out, a.vo_stride, a.vo_head}},
                a.cos, a.sin, a.positions, a.slots, static_cast<uint8_t*>(a.cache), (int)a.m, heads, (int)a.kv_heads,
                (int)a.rot_dim, (int)a.table_rows - 1, 1, a.cache ? log2_of(a.page_tokens) : 0,
                a.cache ? a.pages * a.page_tokens : 0, a.in_dtype, a.out_dtype, a.interleaved};
    // Few tokens: one row a group of lanes, so that nothing waits for a second
    // trip to memory.  Many: a workgroup a token, the tables read once (two or
    // four rows of a group in flight were slower: 83 and 80 us against 68 for 4096
    // tokens and their read-back, with fewer waves a SIMD).
    if (a.m < 512) k.parts = (rows + groups - 1) / groups;
    clear_stale_error();
    if (a.head_dim == 64) start_write<64>(k, stream);
    else if (a.head_dim == 128) start_write<128>(k, stream);
    else start_write<256>(k, stream);
    return hipGetLastError();
}

hipError_t launch_kv_read(const pq2_kv_read_args& a, hipStream_t stream) {
    const ReadArgs k{static_cast<const uint8_t*>(a.cache), a.table, a.starts,
                     {{a.k_out, a.ko_stride, a.ko_head}, {a.v_out, a.vo_stride, a.vo_head}}, a.table_stride, (int)a.rows,
                     (int)a.seqs, (int)a.table_pages, (int)a.kv_heads, (int)a.pages, log2_of(a.page_tokens), a.out_dtype};
    clear_stale_error();
    if (a.head_dim == 64) start_read<64>(k, stream);
    else if (a.head_dim == 128) start_read<128>(k, stream);
    else start_read<256>(k, stream);
    return hipGetLastError();
}

}  // namespace pq2
