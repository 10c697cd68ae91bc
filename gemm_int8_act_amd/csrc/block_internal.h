// block_internal.h -- host-side launchers of the feed-forward block operators
// (declared in include/pq2_block.h), and the pieces their kernels share.
// Arguments reaching the launchers are already validated by the C ABI layer.
#pragma once

#include "pq2_device.h"
#include "pq2_internal.h"

#include <hip/hip_fp16.h>

struct pq2_block_norm_args;

namespace pq2 {

// Weight formats of the block kernels: ternary tiles (128-weight groups) and
// w4 tiles with S = 1, 2 or 4 weight groups per 128 weights.
enum : int { kFmtTernary = 0, kFmtW4 = 1 };

struct BlockMatmul {
    const int8_t* q;
    const float* xs;
    const uint8_t* w0;   // the matrix, or the gate's
    const uint8_t* w1;   // the up matrix (gated only)
    int64_t m, n, k;
    int fmt, s;          // weight format, weight groups per 128
    int act;             // -1: plain product, fp32 out; else PQ2_ACT_*
    void* out;
    int out_dtype;
    hipStream_t stream;
    int src = kSrcNatural;      // or the type of x, quantised inside (block_takes_x)
    const void* x = nullptr;
    int64_t x_stride = 0;
};

int64_t w4_tiles_bytes(int64_t n, int64_t k, int64_t wgroup);
hipError_t launch_prepare_w4(const uint8_t* codes, int64_t codes_stride, const uint16_t* scales, int64_t scales_stride,
                             int64_t n, int64_t k, int wgroup, uint8_t* tiles, hipStream_t stream);
hipError_t launch_block_small_m(const BlockMatmul& a);
hipError_t launch_block_prefill(const BlockMatmul& a);
bool block_takes_small_m(const BlockMatmul& a);
bool block_takes_x(int64_t m, int64_t k);   // whether the decode engine quantises x itself
hipError_t launch_block_norm(const pq2_block_norm_args& a, hipStream_t stream);

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kTernaryUnit = 4352;                                    // bytes of a ternary segment unit
__host__ __device__ constexpr int w4_unit(int s) { return 8192 + 256 * s; }
__host__ __device__ constexpr int block_unit(int fmt, int s) { return fmt == kFmtTernary ? kTernaryUnit : w4_unit(s); }
__host__ __device__ constexpr int block_code_bytes(int fmt) { return fmt == kFmtTernary ? 4096 : 8192; }

// Four INT8 operand dwords (16 weights in k order) of one ternary code dword:
// code c -> c - 1 through one byte-table lookup per bit plane.
__device__ __forceinline__ v4i ternary_operand(uint32_t d) {
    constexpr uint32_t kTable = 0x020100FFu;  // bytes 0..3: the values of codes 0..3
    return v4i{(int)__builtin_amdgcn_perm(0u, kTable, d & 0x03030303u),
               (int)__builtin_amdgcn_perm(0u, kTable, (d >> 2) & 0x03030303u),
               (int)__builtin_amdgcn_perm(0u, kTable, (d >> 4) & 0x03030303u),
               (int)__builtin_amdgcn_perm(0u, kTable, (d >> 6) & 0x03030303u)};
}

// The same of two w4 code dwords.  A four-bit two's complement value in the
// high half of a byte is that value times 16 as an INT8, so no offset or sign
// extension is needed; every dot is 16 times too large and the weight scales
// take the factor back (weight_scale_at).  |16 dot| <= 16*8*127*128 < 2^24
// stays exact as a float.
__device__ __forceinline__ v4i w4_operand(uint32_t d0, uint32_t d1) {
    return v4i{(int)((d0 << 4) & 0xF0F0F0F0u), (int)(d0 & 0xF0F0F0F0u), (int)((d1 << 4) & 0xF0F0F0F0u),
               (int)(d1 & 0xF0F0F0F0u)};
}

__device__ __forceinline__ float half_bits(uint32_t h) { return __half2float(__ushort_as_half((unsigned short)h)); }

// INT8 codes of N elements v of an activation group whose largest magnitude
// is amax: q = clamp(rint(RN(v / d)), +-127), d = scale = RN(amax / 127) or 1
// for an all-zero group, the steps of pq2_quantize_act_i8.  The low byte of
// bits[e] is the code.
//
// RN(v / d) comes from FP32 operations alone (a double product per element,
// as in quantize.hip, issues at half their rate and the decode kernels
// quantise in every workgroup): with d scaled to [1, 2) by a power of two,
// y = RN(1 / d), t0 = RN(v y), e = RN(v - t0 d) and t = RN(t0 + e y), one
// Newton step.  t0 may be off by more than an ulp (1.49 occurs), so t is not
// RN(v / d) by a general theorem; what the codes need holds: t0 + e y is
// within 2 * 2^-23 ulp of the quotient, so t lies on the wrong side of a border
// h + 1/2 only for quotients that near the midpoint beside it.  With 24-bit v
// and d those are 1246, found by their residues, and on each of them t is
// RN(v / d) (test_quantiser_codes_at_the_hardest_quotients).
// Scaling v by the same power is exact for every quotient that does not round
// to 0: |v / d| >= 1/4 leaves |v| >= 1/4.
template <int N>
__device__ __forceinline__ void quantise_bits(const float (&v)[N], float amax, float& scale, uint32_t (&bits)[N]) {
#pragma clang fp contract(off)
    scale = amax / 127.0f;
    const float d = scale > 0.0f ? scale : 1.0f;
    const int exp = __builtin_amdgcn_frexp_expf(d) - 1;
    const float dn = __builtin_ldexpf(d, -exp);
    const float y = 1.0f / dn;
    constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer, ties to even
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const float x = __builtin_ldexpf(v[e], -exp);
        const float t0 = x * y;
        const float t = __builtin_fmaf(__builtin_fmaf(-t0, dn, x), y, t0);
        bits[e] = __float_as_uint(__builtin_amdgcn_fmed3f(t, -127.0f, 127.0f) + kRound);
    }
}

// Codes e .. e + 3 in one dword.
template <int N>
__device__ __forceinline__ uint32_t code_bytes(const uint32_t (&bits)[N], int e) {
    const uint32_t a = __builtin_amdgcn_perm(bits[e + 1], bits[e], 0x0C0C0400u);
    const uint32_t b = __builtin_amdgcn_perm(bits[e + 3], bits[e + 2], 0x0C0C0400u);
    return a | (b << 16);
}

// The lane's 16 elements of a 128-element activation group (eight aligned
// lanes) as codes in natural order, and the group's scale.
__device__ __forceinline__ uint4 quantize16(const float (&v)[16], float& scale) {
    float amax = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(v[e]));
    uint32_t bits[16];
    quantise_bits(v, max8_f(amax), scale, bits);
    return make_uint4(code_bytes(bits, 0), code_bytes(bits, 4), code_bytes(bits, 8), code_bytes(bits, 12));
}

// fp16 number i (0..7) of 16 bytes.
__device__ __forceinline__ float half_at(const uint4& v, int i) {
    const uint32_t w = word_of(v, i >> 1);
    return half_bits((i & 1) ? (w >> 16) : (w & 0xFFFFu));
}

// The scale of a weight group as its dot is multiplied with it: fp16 number i
// (0..7) of 16 bytes, for 4-bit weights a sixteenth of it.  Every fp16 scale
// has an exact sixteenth in FP32, so each term has the bits it has with a dot
// of the weights themselves.  (Taken off the finished sum instead, the factor
// makes sums from 2^124 on overflow on their way.)  As a fused multiply-add it
// is one mixed-precision instruction together with the conversion from fp16.
template <int FMT>
__device__ __forceinline__ float weight_scale_at(const uint4& v, int i) {
    if constexpr (FMT == kFmtW4) return __builtin_fmaf(half_at(v, i), 0.0625f, 0.0f);
    return half_at(v, i);
}

// The gate's activation on an fp32 sum (PQ2_ACT_SILU = 0, PQ2_ACT_GELU_TANH = 1).
// tanh(z) = 1 - 2 / (1 + exp(2z)) turns the GELU into g * sigmoid(2z) with
// z = sqrt(2/pi) (g + 0.044715 g^3): one exp and one division for both, and
// the limits (exp -> 0 or inf) come out as g and -0.
__device__ __forceinline__ float gate_activation(float g, int act) {
    const float z = act == 0 ? g : 1.5957691216057308f * (g + 0.044715f * g * g * g);
    return g / (1.0f + expf(-z));
}

// v rounded to nearest even into element i of `out`.
__device__ __forceinline__ void store_as(void* out, size_t i, float v, int dtype) {
    if (dtype == 0) static_cast<__bf16*>(out)[i] = (__bf16)v;
    else if (dtype == 1) static_cast<_Float16*>(out)[i] = (_Float16)v;
    else static_cast<float*>(out)[i] = v;
}

}  // namespace pq2
