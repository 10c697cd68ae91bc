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
// All loads, the norm weights' and the gate's among them, go out before the
// first sum, so a row waits for memory once.  Few rows are bound by that
// latency and the two reductions, many by memory.
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
    double eps, inv_k;
    float alpha;
    int k, agroup, r_dtype, block_dtype, w_dtype, x_dtype, unit_offset;
};

__device__ __forceinline__ float from16(uint32_t b, bool f16) {
    return f16 ? half_bits(b) : __uint_as_float(b << 16);
}

// Eight consecutive elements as loaded; `hi` for FP32 only.
struct Raw8 {
    uint4 lo, hi;
};

// From element i of p; dtype is uniform.
template <bool VEC>
__device__ __forceinline__ void load8(const void* p, int64_t i, int dtype, Raw8& w) {
    if (dtype == 2) {
        const uint32_t* f = static_cast<const uint32_t*>(p) + i;
        if constexpr (VEC) {
            w.lo = *reinterpret_cast<const uint4*>(f);
            w.hi = *reinterpret_cast<const uint4*>(f + 4);
        } else {
            w.lo = make_uint4(f[0], f[1], f[2], f[3]);
            w.hi = make_uint4(f[4], f[5], f[6], f[7]);
        }
        return;
    }
    const uint16_t* h = static_cast<const uint16_t*>(p) + i;
    if constexpr (VEC) {
        w.lo = *reinterpret_cast<const uint4*>(h);
    } else {
        auto two = [&](int e) { return (uint32_t)h[e] | ((uint32_t)h[e + 1] << 16); };
        w.lo = make_uint4(two(0), two(2), two(4), two(6));
    }
}

__device__ __forceinline__ void widen8(const Raw8& w, int dtype, float (&v)[8]) {
    if (dtype == 2) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = __uint_as_float(word_of(w.lo, e));
            v[4 + e] = __uint_as_float(word_of(w.hi, e));
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[2 * e] = from16(word_of(w.lo, e) & 0xFFFFu, dtype == 1);
        v[2 * e + 1] = from16(word_of(w.lo, e) >> 16, dtype == 1);
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

template <int CTRL>
__device__ __forceinline__ double dpp_d(double v) {
    const long long b = __double_as_longlong(v);
    const uint32_t lo = (uint32_t)dpp_i<CTRL>((int)(uint32_t)b), hi = (uint32_t)dpp_i<CTRL>((int)(b >> 32));
    return __longlong_as_double(((long long)hi << 32) | lo);
}

__device__ __forceinline__ void add_one(float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 1.0f + f[e];
}

// Sum over each aligned row of 16 lanes; all lanes agree.
__device__ __forceinline__ double sum16_d(double v) {
    v += dpp_d<kDppXor1>(v);
    v += dpp_d<kDppXor2>(v);
    v += dpp_d<kDppHalfMirror>(v);
    v += dpp_d<kDppMirror>(v);
    return v;
}

// Sum over the workgroup's (at most 16) waves, the same in every thread: rows
// of 16 lanes, then the 4 rows of each of the 16 waves from LDS, in a fixed
// order.  `part` holds 64 doubles, and is not touched again before another
// barrier.
__device__ __forceinline__ double block_sum(double v, double* part) {
    v = sum16_d(v);
    const int lane = threadIdx.x & 63, rows = blockDim.x >> 4;
    if ((threadIdx.x & 15) == 0) part[threadIdx.x >> 4] = v;
    __syncthreads();
    double s = lane < rows ? part[lane] : 0.0;
    s = sum16_d(s);
    // The four rows' sums, read from one lane of each.
    auto row_sum = [&](int r) {
        const long long b = __double_as_longlong(s);
        const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, 16 * r);
        const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), 16 * r);
        return __longlong_as_double(((long long)hi << 32) | lo);
    };
    return (row_sum(0) + row_sum(1)) + (row_sum(2) + row_sum(3));
}

// CH chunks per thread; VEC: every row base is 16-byte aligned; RD, BD, WD:
// element types of the stream, the block and the vectors, known at compile
// time or (-1) from the arguments (the branches per element cost a third of
// the instructions: m = 4096, K = 5120, 50.6 us, with an fp16 stream and vectors
// and all types at run time 75.6).  Eight chunks (k > 32768) spill.
template <int CH, bool VEC, int RD, int BD, int WD>
__global__ __launch_bounds__(1024) void block_norm_kernel(NormKernelArgs a) {
#pragma clang fp contract(off)
    const int r_dtype = RD >= 0 ? RD : a.r_dtype, b_dtype = BD >= 0 ? BD : a.block_dtype,
              w_dtype = WD >= 0 ? WD : a.w_dtype;
    // Longer rows load the vectors where they are used: registers.
    constexpr bool EARLY = CH <= 2;
    __shared__ double part[2][64];
    const int64_t row = blockIdx.x;
    const int chunks = a.k >> 3;
    const int t = threadIdx.x, threads = blockDim.x;
    const bool codes = a.q || a.x_out;

    Raw8 rr[CH], rb[CH], rp[EARLY ? CH : 1], rg[EARLY ? CH : 1], rw[EARLY ? CH : 1];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int ch = t + c * threads;
        rr[c] = rb[c] = Raw8{};
        if constexpr (EARLY) rp[c] = rg[c] = rw[c] = Raw8{};
        if (ch >= chunks) continue;
        if (a.block) load8<VEC>(a.block, row * a.block_stride + 8 * ch, b_dtype, rb[c]);
        load8<VEC>(a.r, row * a.r_stride + 8 * ch, r_dtype, rr[c]);
        if constexpr (EARLY) {
            if (a.post_w) load8<VEC>(a.post_w, 8 * ch, w_dtype, rp[c]);
            if (a.gate) load8<VEC>(a.gate, row * a.gate_stride + 8 * ch, w_dtype, rg[c]);
            if (codes) load8<VEC>(a.w, 8 * ch, w_dtype, rw[c]);
        }
    }
    // The vector of chunk ch, loaded now or before.
    auto vec8 = [&](const void* p, int64_t off, int ch, const Raw8& early, float (&f)[8]) {
        if constexpr (EARLY) {
            widen8(early, w_dtype, f);
        } else {
            Raw8 w{};
            if (ch < chunks) load8<VEC>(p, off + 8 * ch, w_dtype, w);
            widen8(w, w_dtype, f);
        }
    };

    float v[CH][8];
    if (a.block) {
        float b[CH][8];
#pragma unroll
        for (int c = 0; c < CH; ++c) widen8(rb[c], b_dtype, b[c]);
        if (a.post_w) {
            double s = 0.0;
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e) s = __builtin_fma((double)b[c][e], (double)b[c][e], s);
            const float rstd = (float)rsqrt(block_sum(s, part[0]) * a.inv_k + a.eps);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                float f[8];
                vec8(a.post_w, 0, t + c * threads, rp[EARLY ? c : 0], f);
                if (a.unit_offset) add_one(f);
#pragma unroll
                for (int e = 0; e < 8; ++e) b[c][e] = (b[c][e] * rstd) * f[e];
            }
        }
        if (a.gate) {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                float f[8];
                vec8(a.gate, row * a.gate_stride, t + c * threads, rg[EARLY ? c : 0], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) b[c][e] *= f[e];
            }
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            widen8(rr[c], r_dtype, v[c]);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[c][e] += b[c][e] * a.alpha;
            round8(v[c], r_dtype);
        }
    } else {
#pragma unroll
        for (int c = 0; c < CH; ++c) widen8(rr[c], r_dtype, v[c]);
    }
    if (a.r_out) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int ch = t + c * threads;
            if (ch < chunks) store8<VEC>(a.r_out, row * a.r_out_stride + 8 * ch, r_dtype, v[c]);
        }
    }
    if (!codes) return;

    double s = 0.0;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) s = __builtin_fma((double)v[c][e], (double)v[c][e], s);
    const float rstd = (float)rsqrt(block_sum(s, part[1]) * a.inv_k + a.eps);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int ch = t + c * threads;
        if (ch >= chunks) continue;  // whole groups: a group's chunks are 16, 8 or 4 aligned lanes of one wave
        float f[8];
        vec8(a.w, 0, ch, rw[EARLY ? c : 0], f);
        if (a.unit_offset) add_one(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[c][e] = (v[c][e] * rstd) * f[e];
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
        uint32_t bits[8];
        float scale;
        quantise_bits(v[c], amax, scale, bits);
        *reinterpret_cast<uint2*>(a.q + row * a.k + 8 * ch) = make_uint2(code_bytes(bits, 0), code_bytes(bits, 4));
        const int lanes = a.agroup >> 3;
        if ((ch & (lanes - 1)) == 0) a.xs[row * (a.k / a.agroup) + ch / lanes] = scale;
    }
}

template <int CH, bool VEC, int RD, int BD, int WD>
hipError_t launch_one(const NormKernelArgs& a, int64_t m, int threads, hipStream_t stream) {
    clear_stale_error();
    hipLaunchKernelGGL((block_norm_kernel<CH, VEC, RD, BD, WD>), dim3((unsigned)m), dim3(threads), 0, stream, a);
    return hipGetLastError();
}

// Streams of every type with an FP32 or bf16 block and bf16 vectors have
// kernels of their own, for rows of up to four chunks a thread.
template <int CH, int RD>
hipError_t launch_typed(const NormKernelArgs& a, int64_t m, int threads, hipStream_t stream) {
    if (a.w_dtype == 0 && a.block_dtype == 2) return launch_one<CH, true, RD, 2, 0>(a, m, threads, stream);
    if (a.w_dtype == 0 && a.block_dtype == 0) return launch_one<CH, true, RD, 0, 0>(a, m, threads, stream);
    return launch_one<CH, true, -1, -1, -1>(a, m, threads, stream);
}

template <int CH>
hipError_t launch_ch(const NormKernelArgs& a, int64_t m, int threads, bool vec, hipStream_t stream) {
    if (!vec) return launch_one<CH, false, -1, -1, -1>(a, m, threads, stream);
    if constexpr (CH <= 4) {
        switch (a.r_dtype) {
            case 0: return launch_typed<CH, 0>(a, m, threads, stream);
            case 1: return launch_typed<CH, 1>(a, m, threads, stream);
            default: return launch_typed<CH, 2>(a, m, threads, stream);
        }
    }
    return launch_one<CH, true, -1, -1, -1>(a, m, threads, stream);
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
    a.inv_k = 1.0 / (double)p.k;
    a.alpha = p.alpha;
    a.k = (int)p.k;
    a.agroup = p.q ? (int)p.agroup : 128;
    a.r_dtype = p.r_dtype;
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
    // One chunk a thread while rows are few (their latency counts), two when
    // there are enough rows to fill the chip with smaller workgroups (K = 5120,
    // norms on both sides: m = 256 7.1 against 7.4 us, m = 1024 18.2 against
    // 16.5, m = 4096 58.7 against 51.6; K = 640, m = 4096 11.3 against 11.5).
    int ch = p.m >= 768 && chunks > 128 ? 2 : 1;
    while ((chunks + ch - 1) / ch > 1024) ch *= 2;  // k <= 65536: at most 8
    const int threads = ((chunks + ch - 1) / ch + 63) / 64 * 64;
    switch (ch) {
        case 1: return launch_ch<1>(a, p.m, threads, vec, stream);
        case 2: return launch_ch<2>(a, p.m, threads, vec, stream);
        case 4: return launch_ch<4>(a, p.m, threads, vec, stream);
        default: return launch_ch<8>(a, p.m, threads, vec, stream);
    }
}

}  // namespace pq2
