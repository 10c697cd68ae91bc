// norm.hip -- the norms before and after a block, fused with the block's
// gate, its residual scale, the residual add and the INT8 quantiser of the
// next product (pq2_block_norm).
//
// Mathematics: include/pq2_block.h states the exact order of the FP32
// operations.  The two sums of squares are formed in FP64 (a product of two
// fp32 values is exact there), so that rstd, one rounding to FP32 of a value
// known to about 1e-15, does not depend on the order of the sum, and the
// codes behind it do not either: a rounding border moved by one FP32 step of
// rstd would change codes.
//
// Geometry: one workgroup per row.  A thread holds CH chunks of eight
// consecutive elements (16-byte loads for 2-byte types) in registers from the
// load to the codes, so every tensor is read once and written once; chunk
// t + i * threads, so 16, 8 or 4 neighbouring lanes of a wave hold an
// activation group and its maximum is a DPP reduction inside a row of 16.
#include "../../include/pq2_block.h"
#include "block_internal.h"

namespace pq2 {

namespace {

struct NormKernelArgs {
    const void* r;
    const void* block;
    const void* post_w;
    const void* gate;
    const void* w;
    void* r_out;
    void* x_out;
    int8_t* q;
    float* xs;
    int64_t r_stride, block_stride, gate_stride, r_out_stride, x_out_stride;
    double eps;
    float alpha;
    int k, agroup, block_dtype, w_dtype, x_dtype, unit_offset;
};

__device__ __forceinline__ float from16(uint32_t b, bool f16) {
    return f16 ? half_bits(b) : __uint_as_float(b << 16);
}

// Eight consecutive elements from element i of p; dtype is uniform.
template <bool VEC>
__device__ __forceinline__ void load8(const void* p, int64_t i, int dtype, float (&v)[8]) {
    if (dtype == 2) {
        const float* f = static_cast<const float*>(p) + i;
        if constexpr (VEC) {
            const float4 a = *reinterpret_cast<const float4*>(f);
            const float4 b = *reinterpret_cast<const float4*>(f + 4);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = f[e];
        }
        return;
    }
    const uint16_t* h = static_cast<const uint16_t*>(p) + i;
    uint32_t w[4];
    if constexpr (VEC) {
        const uint4 a = *reinterpret_cast<const uint4*>(h);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = (uint32_t)h[2 * e] | ((uint32_t)h[2 * e + 1] << 16);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[2 * e] = from16(w[e] & 0xFFFFu, dtype == 1);
        v[2 * e + 1] = from16(w[e] >> 16, dtype == 1);
    }
}

// v rounded to dtype (and widened again).
__device__ __forceinline__ void round8(float (&v)[8], int dtype) {
    if (dtype == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (float)(__bf16)v[e];
    } else if (dtype == 1) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (float)(_Float16)v[e];
    }
}

// Stores eight values that dtype holds exactly.
template <bool VEC>
__device__ __forceinline__ void store8(void* p, int64_t i, int dtype, const float (&v)[8]) {
    if (dtype == 2) {
        float* f = static_cast<float*>(p) + i;
        if constexpr (VEC) {
            *reinterpret_cast<float4*>(f) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(f + 4) = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = v[e];
        }
        return;
    }
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (dtype == 0) {
            w[e] = (__float_as_uint(v[2 * e]) >> 16) | (__float_as_uint(v[2 * e + 1]) & 0xFFFF0000u);
        } else {
            w[e] = (uint32_t)__half_as_ushort(__float2half_rn(v[2 * e])) |
                   ((uint32_t)__half_as_ushort(__float2half_rn(v[2 * e + 1])) << 16);
        }
    }
    uint16_t* h = static_cast<uint16_t*>(p) + i;
    if constexpr (VEC) {
        *reinterpret_cast<uint4*>(h) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            h[2 * e] = (uint16_t)w[e];
            h[2 * e + 1] = (uint16_t)(w[e] >> 16);
        }
    }
}

// Sum over the workgroup, the same in every thread: lanes by xor steps, then
// the waves in index order.  `part` holds one double per wave and is not
// touched again before another barrier.
__device__ __forceinline__ double block_sum(double v, double* part) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) part[wave] = v;
    __syncthreads();
    const int waves = blockDim.x >> 6;
    double s = part[0];
    for (int i = 1; i < waves; ++i) s += part[i];
    return s;
}

// CH chunks per thread; RD the stream's dtype; VEC: every row base is
// 16-byte aligned.
template <int CH, int RD, bool VEC>
__global__ __launch_bounds__(1024) void block_norm_kernel(NormKernelArgs a) {
#pragma clang fp contract(off)
    __shared__ double part[2][16];
    const int64_t row = blockIdx.x;
    const int chunks = a.k >> 3;
    const int t = threadIdx.x, threads = blockDim.x;

    float v[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int ch = t + c * threads;
        if (ch < chunks) {
            load8<VEC>(a.r, row * a.r_stride + 8 * ch, RD, v[c]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[c][e] = 0.0f;
        }
    }
    if (a.block) {
        float b[CH][8];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int ch = t + c * threads;
            if (ch < chunks) {
                load8<VEC>(a.block, row * a.block_stride + 8 * ch, a.block_dtype, b[c]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) b[c][e] = 0.0f;
            }
        }
        float rstd = 1.0f;
        if (a.post_w) {
            double s = 0.0;
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e) s += (double)b[c][e] * (double)b[c][e];
            rstd = (float)(1.0 / sqrt(block_sum(s, part[0]) / (double)a.k + a.eps));
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int ch = t + c * threads;
            if (ch >= chunks) continue;
            float f[8];
            if (a.post_w) {
                load8<VEC>(a.post_w, 8 * ch, a.w_dtype, f);
#pragma unroll
                for (int e = 0; e < 8; ++e) b[c][e] = (b[c][e] * rstd) * (a.unit_offset ? 1.0f + f[e] : f[e]);
            }
            if (a.gate) {
                load8<VEC>(a.gate, row * a.gate_stride + 8 * ch, a.w_dtype, f);
#pragma unroll
                for (int e = 0; e < 8; ++e) b[c][e] *= f[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v[c][e] += b[c][e] * a.alpha;
            round8(v[c], RD);
        }
    }
    if (a.r_out) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int ch = t + c * threads;
            if (ch < chunks) store8<VEC>(a.r_out, row * a.r_out_stride + 8 * ch, RD, v[c]);
        }
    }
    if (!a.q && !a.x_out) return;

    double s = 0.0;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) s += (double)v[c][e] * (double)v[c][e];
    const float rstd = (float)(1.0 / sqrt(block_sum(s, part[1]) / (double)a.k + a.eps));
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int ch = t + c * threads;
        if (ch >= chunks) continue;  // whole groups: a group's chunks are 16, 8 or 4 aligned lanes of one wave
        float f[8];
        load8<VEC>(a.w, 8 * ch, a.w_dtype, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[c][e] = (v[c][e] * rstd) * (a.unit_offset ? 1.0f + f[e] : f[e]);
        round8(v[c], a.x_dtype);
        if (a.x_out) store8<VEC>(a.x_out, row * a.x_out_stride + 8 * ch, a.x_dtype, v[c]);
        if (!a.q) continue;
        float amax = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[c][e]));
        amax = fmaxf(amax, dpp_f<kDppXor1>(amax));
        amax = fmaxf(amax, dpp_f<kDppXor2>(amax));
        if (a.agroup >= 64) amax = fmaxf(amax, dpp_f<kDppHalfMirror>(amax));
        if (a.agroup == 128) amax = fmaxf(amax, dpp_f<kDppMirror>(amax));
        // The quantiser's steps (quantize.hip): the IEEE quotient v / d as the
        // double product v * fl64(1 / d) rounded to fp32.
        const float scale = amax / 127.0f;
        const double inv = 1.0 / (double)(scale > 0.0f ? scale : 1.0f);
        uint32_t packed[2] = {0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float r = rintf((float)((double)v[c][e] * inv));
            r = fminf(127.0f, fmaxf(-127.0f, r));
            packed[e >> 2] |= ((uint32_t)(int)r & 0xFFu) << (8 * (e & 3));
        }
        *reinterpret_cast<uint2*>(a.q + row * a.k + 8 * ch) = make_uint2(packed[0], packed[1]);
        const int lanes = a.agroup >> 3;
        if ((ch & (lanes - 1)) == 0) a.xs[row * (a.k / a.agroup) + ch / lanes] = scale;
    }
}

template <int CH, int RD>
hipError_t launch_one(const NormKernelArgs& a, int64_t m, int threads, bool vec, hipStream_t stream) {
    clear_stale_error();
    if (vec)
        hipLaunchKernelGGL((block_norm_kernel<CH, RD, true>), dim3((unsigned)m), dim3(threads), 0, stream, a);
    else
        hipLaunchKernelGGL((block_norm_kernel<CH, RD, false>), dim3((unsigned)m), dim3(threads), 0, stream, a);
    return hipGetLastError();
}

template <int CH>
hipError_t launch_ch(const NormKernelArgs& a, int rd, int64_t m, int threads, bool vec, hipStream_t stream) {
    switch (rd) {
        case 0: return launch_one<CH, 0>(a, m, threads, vec, stream);
        case 1: return launch_one<CH, 1>(a, m, threads, vec, stream);
        default: return launch_one<CH, 2>(a, m, threads, vec, stream);
    }
}

bool rows_aligned(const void* p, int64_t stride, int dtype) {
    return ((uintptr_t)p % 16) == 0 && (stride * (dtype == 2 ? 4 : 2)) % 16 == 0;
}

}  // namespace

hipError_t launch_block_norm(const pq2_block_norm_args& p, hipStream_t stream) {
    NormKernelArgs a{};
    a.r = p.r;
    a.block = p.block;
    a.post_w = p.block ? p.post_w : nullptr;
    a.gate = p.block ? p.gate : nullptr;
    a.w = p.w;
    a.r_out = p.r_out;
    a.x_out = p.x_out;
    a.q = p.q;
    a.xs = p.xs;
    a.r_stride = p.r_stride;
    a.block_stride = p.block_stride;
    a.gate_stride = p.gate_stride;
    a.r_out_stride = p.r_out_stride;
    a.x_out_stride = p.x_out_stride;
    a.eps = p.eps;
    a.alpha = p.alpha;
    a.k = (int)p.k;
    a.agroup = p.q ? (int)p.agroup : 128;
    a.block_dtype = p.block_dtype;
    a.w_dtype = p.w_dtype;
    a.x_dtype = p.x_dtype;
    a.unit_offset = p.unit_offset;
    const bool vec = rows_aligned(p.r, p.r_stride, p.r_dtype) && rows_aligned(p.w, 0, p.w_dtype) &&
                     (!a.block || rows_aligned(p.block, p.block_stride, p.block_dtype)) &&
                     (!a.post_w || rows_aligned(p.post_w, 0, p.w_dtype)) &&
                     (!a.gate || rows_aligned(p.gate, p.gate_stride, p.w_dtype)) &&
                     (!p.r_out || rows_aligned(p.r_out, p.r_out_stride, p.r_dtype)) &&
                     (!p.x_out || rows_aligned(p.x_out, p.x_out_stride, p.x_dtype));
    const int chunks = (int)(p.k / 8);
    int ch = 1;
    while ((chunks + ch - 1) / ch > 1024) ch *= 2;  // k <= 65536: at most 8
    const int threads = ((chunks + ch - 1) / ch + 63) / 64 * 64;
    switch (ch) {
        case 1: return launch_ch<1>(a, p.r_dtype, p.m, threads, vec, stream);
        case 2: return launch_ch<2>(a, p.r_dtype, p.m, threads, vec, stream);
        case 4: return launch_ch<4>(a, p.r_dtype, p.m, threads, vec, stream);
        default: return launch_ch<8>(a, p.r_dtype, p.m, threads, vec, stream);
    }
}

}  // namespace pq2
