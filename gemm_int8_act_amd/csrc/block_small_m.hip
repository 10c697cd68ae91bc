// block_small_m.hip -- decode engine of the block operators: products with
// 4-bit weights and the gated feed-forward product for few columns.
//
// One workgroup per tile of 16 weight rows (gated: the gate tile and the up
// tile of the same rows); its waves take consecutive slices of k, whole
// segments of 1024.  A wave loads its segment's activations, scales and codes
// (every code load one contiguous kilobyte), forms each weight group's exact
// dot with v_mfma_i32_16x16x64_i8 and adds one FP32 term per activation
// group; the slices are added in index order by the whole workgroup, which
// also applies the gate's activation, so the two products of a gated call
// never reach memory.  The order of a column's sum depends on k only.
//
//  ternary: cls[c] = fma(float(dot) * xs, ws, cls[c]) per group class c and
//           ((c0+c4)+(c1+c5))+((c2+c6)+(c3+c7)) per slice: the order of
//           small_m_tiles_kernel, hence its bits.
//  w4:      acc = fma(t, xs, acc) over the activation groups in k order, t =
//           the weight groups' float(dot) * ws added in k order.
//
// Up to four columns (WIDE false): the four A rows 4c .. 4c+3 of the matrix
// core all belong to column c, so a lane owns one output (column lane/16).
// With S = 2 or 4 weight groups per 128 the rows are told apart by masking:
// row 4c+r keeps only weight group r, and one pair of MFMAs gives the dots
// of all S groups in the four result registers.  Activations come through a
// private LDS region (one load per column).
// Up to sixteen columns (WIDE): A row = column, read straight from memory in
// operand order; a lane owns four outputs.
#include "block_internal.h"
#include "small_m_common.h"

namespace pq2 {

namespace {

struct SmallArgs {
    const int8_t* q;
    const float* xs;
    const uint8_t* w0;
    const uint8_t* w1;
    void* out;
    int n, k, groups, s8, nseg, per_wave, mtotal, act, out_dtype, region;
};

constexpr int kColPitch = 1024 + 64;  // four columns' reads fall in distinct banks

template <int FMT, int S, int NB, bool WIDE, int MAXW>
__global__ __launch_bounds__(64 * MAXW) void block_small_m_kernel(SmallArgs a) {
#pragma clang fp contract(off)
    constexpr int UNIT = block_unit(FMT, S);
    constexpr int CODES = block_code_bytes(FMT);
    constexpr int CB = CODES / 1024;   // code loads per segment
    constexpr int MC = WIDE ? 16 : 4;
    constexpr int R = WIDE ? 4 : 1;    // outputs per lane
    constexpr int C = FMT == kFmtTernary ? 8 : 1;  // accumulators per output
    extern __shared__ __align__(16) unsigned char smem[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nwaves = blockDim.x >> 6;
    const int lane = threadIdx.x & 63;
    const int j = lane & 15;
    const int kb = lane >> 4;
    const int tile = blockIdx.x;
    const int m0 = blockIdx.y * MC;
    const int mcount = min(MC, a.mtotal - m0);
    const int seg_begin = wave * a.per_wave;
    const int seg_end = min(seg_begin + a.per_wave, a.nseg);

    const size_t tile_off = (size_t)tile * a.s8 * UNIT;
    const uint32_t tile_bytes = (uint32_t)(a.s8 * UNIT);
    const __amdgpu_buffer_rsrc_t w_rs[2] = {make_rsrc(a.w0 + tile_off, tile_bytes),
                                            make_rsrc(NB == 2 ? a.w1 + tile_off : nullptr, NB == 2 ? tile_bytes : 0u)};
    const auto q_rs = make_rsrc(a.q + (size_t)m0 * a.k, (uint32_t)(mcount * a.k));
    const auto xs_rs = make_rsrc(a.xs + (size_t)m0 * a.groups, (uint32_t)(mcount * a.groups * 4));
    unsigned char* region = smem + (size_t)wave * a.region;

    // Rows of the A operand that keep weight group r = j & 3 of step h.
    uint32_t keep[2] = {~0u, ~0u};
    if constexpr (!WIDE && S > 1) {
#pragma unroll
        for (int h = 0; h < 2; ++h) keep[h] = (j & 3) == (S == 2 ? h : 2 * h + (kb >> 1)) ? ~0u : 0u;
    }
    const uint32_t low_half = kb < 2 ? ~0u : 0u;  // WIDE, S = 4: lanes of the first 32 weights of a step

    float acc[NB][C][R];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int r = 0; r < R; ++r) acc[b][c][r] = 0.0f;

    for (int s = seg_begin; s < seg_end; ++s) {
        // 1. Loads: scales of the activations, activations, then the weights.
        const int g0 = 8 * s;
        uint4 xv[2];
        uint2 xw;
        uint4 av[WIDE ? 16 : 4];
        if constexpr (WIDE) {
            xw = buf_load8(xs_rs, j < mcount && g0 + 2 * kb < a.groups ? (uint32_t)((j * a.groups + g0 + 2 * kb) * 4)
                                                                       : kBufferOOB);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int off = s * 1024 + 64 * i + 16 * kb;
                av[i] = buf_load16(q_rs, j < mcount && off < a.k ? (uint32_t)(j * a.k + off) : kBufferOOB);
            }
        } else {
            const uint32_t xoff = (uint32_t)((min(kb, mcount - 1) * a.groups + g0) * 4);
            xv[0] = buf_load16(xs_rs, xoff);
            xv[1] = buf_load16(xs_rs, xoff + 16u);
            const int off = s * 1024 + 16 * lane;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < mcount) av[i] = buf_load16(q_rs, off < a.k ? (uint32_t)(i * a.k + off) : kBufferOOB);
        }
        uint4 sc[NB][S], cw[NB][CB];
        const uint32_t unit = (uint32_t)(s * UNIT);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < S; ++i)
                sc[b][i] = buf_load16<kAuxNonTemporal>(w_rs[b], unit + CODES + 16 * S * j + 16 * i);
#pragma unroll
        for (int i = 0; i < CB; ++i)
#pragma unroll
            for (int b = 0; b < NB; ++b)
                cw[b][i] = buf_load16<kAuxNonTemporal>(w_rs[b], unit + 1024 * i + 16 * lane);

        // 2. Stage.
        if constexpr (WIDE) {
            float* xl = reinterpret_cast<float*>(region);
            xl[(2 * kb) * 16 + j] = __uint_as_float(xw.x);
            xl[(2 * kb + 1) * 16 + j] = g0 + 2 * kb + 1 < a.groups ? __uint_as_float(xw.y) : 0.0f;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < mcount) *reinterpret_cast<uint4*>(region + i * kColPitch + 16 * lane) = av[i];
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");

        // 3. Group dots and terms.
        const int col = WIDE ? 0 : ((j >> 2) < mcount ? (j >> 2) : 0);
        const unsigned char* a_base = region + col * kColPitch + 16 * kb;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
            v4i A[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint4 v;
                if constexpr (WIDE) v = av[2 * g + h];
                else v = *reinterpret_cast<const uint4*>(a_base + 128 * g + 64 * h);
                A[h] = v4i{(int)(v.x & keep[h]), (int)(v.y & keep[h]), (int)(v.z & keep[h]), (int)(v.w & keep[h])};
            }
            float xg[R];
            if constexpr (WIDE) {
                const float4 v = *reinterpret_cast<const float4*>(region + (g * 16 + 4 * kb) * 4);
                xg[0] = v.x; xg[1] = v.y; xg[2] = v.z; xg[3] = v.w;
            } else {
                // Past the last group the loads hold the next column's scales.
                xg[0] = g0 + g < a.groups ? __uint_as_float(word_of(xv[g >> 2], g & 3)) : 0.0f;
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                v4i B[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (FMT == kFmtTernary) B[h] = ternary_operand(word_of(cw[b][g >> 1], 2 * (g & 1) + h));
                    else B[h] = w4_operand(word_of(cw[b][g], 2 * h), word_of(cw[b][g], 2 * h + 1));
                }
                float dot[S][R];  // float of the weight groups' dots
                if constexpr (!WIDE || S == 1) {
                    v4i D = __builtin_amdgcn_mfma_i32_16x16x64_i8(A[0], B[0], v4i{}, 0, 0, 0);
                    D = __builtin_amdgcn_mfma_i32_16x16x64_i8(A[1], B[1], D, 0, 0, 0);
#pragma unroll
                    for (int t = 0; t < S; ++t)
#pragma unroll
                        for (int r = 0; r < R; ++r) dot[t][r] = (float)D[WIDE ? r : t];
                } else {
#pragma unroll
                    for (int t = 0; t < S; ++t) {
                        const int h = S == 2 ? t : t >> 1;
                        v4i Am = A[h];
                        if constexpr (S == 4) {
                            const int mask = (int)((t & 1) ? ~low_half : low_half);
                            Am = v4i{Am[0] & mask, Am[1] & mask, Am[2] & mask, Am[3] & mask};
                        }
                        const v4i D = __builtin_amdgcn_mfma_i32_16x16x64_i8(Am, B[h], v4i{}, 0, 0, 0);
#pragma unroll
                        for (int r = 0; r < R; ++r) dot[t][r] = (float)D[r];
                    }
                }
                if constexpr (FMT == kFmtTernary) {
                    const float ws = half_at(sc[b][0], g);
#pragma unroll
                    for (int r = 0; r < R; ++r) acc[b][g][r] = __builtin_fmaf(dot[0][r] * xg[r], ws, acc[b][g][r]);
                } else {
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        float t = dot[0][r] * half_at(sc[b][(g * S) >> 3], (g * S) & 7);
#pragma unroll
                        for (int u = 1; u < S; ++u)
                            t = __builtin_fmaf(dot[u][r], half_at(sc[b][(g * S + u) >> 3], (g * S + u) & 7), t);
                        acc[b][0][r] = __builtin_fmaf(t, xg[r], acc[b][0][r]);
                    }
                }
            }
        }
        // The next segment rewrites the region: LDS operations of one wave
        // complete in order.
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }

    // 4. Slice sums to the wave's own region, then the slices in index order.
    float* part = reinterpret_cast<float*>(region);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float v;
            if constexpr (FMT == kFmtTernary)
                v = ((acc[b][0][r] + acc[b][4][r]) + (acc[b][1][r] + acc[b][5][r])) +
                    ((acc[b][2][r] + acc[b][6][r]) + (acc[b][3][r] + acc[b][7][r]));
            else
                v = acc[b][0][r];
            const int col = WIDE ? 4 * kb + r : kb;
            if (col < mcount) part[(b * mcount + col) * 16 + j] = v;
        }
    __syncthreads();
    for (int o = threadIdx.x; o < mcount * 16; o += blockDim.x) {
        float y[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float sum = 0.0f;
            for (int w = 0; w < nwaves; ++w) {
                const float v = reinterpret_cast<const float*>(smem + (size_t)w * a.region)[b * mcount * 16 + o];
                sum = w == 0 ? v : sum + v;
            }
            y[b] = FMT == kFmtW4 ? sum * kW4Scale : sum;
        }
        const int row = tile * 16 + (o & 15);
        if (row < a.n) {
            const size_t at = (size_t)(m0 + (o >> 4)) * a.n + row;
            if constexpr (NB == 2) store_as(a.out, at, gate_activation(y[0], a.act) * y[1], a.out_dtype);
            else static_cast<float*>(a.out)[at] = y[0];
        }
    }
}

template <int FMT, int S, int NB, bool WIDE>
hipError_t launch_one(const BlockMatmul& p) {
    SmallArgs a{p.q, p.xs, p.w0, p.w1, p.out, (int)p.n, (int)p.k, (int)(p.k / 128), (int)((p.k + 1023) / 1024), 0, 0,
                (int)p.m, p.act, p.out_dtype, 0};
    a.nseg = a.s8;
    a.per_wave = (a.nseg + kTilesDefaultWaves - 1) / kTilesDefaultWaves;
    const int waves = (a.nseg + a.per_wave - 1) / a.per_wave;
    constexpr int MC = WIDE ? 16 : 4;
    const int mc = (int)(p.m < MC ? p.m : MC);
    const int partials = NB * mc * 64, staging = WIDE ? 512 : mc * kColPitch;
    a.region = partials > staging ? partials : staging;
    const dim3 grid((unsigned)((p.n + 15) / 16), (unsigned)((p.m + MC - 1) / MC));
    const size_t lds = (size_t)waves * a.region;
    clear_stale_error();
    if (waves <= 8)
        hipLaunchKernelGGL((block_small_m_kernel<FMT, S, NB, WIDE, 8>), grid, dim3(64 * waves), lds, p.stream, a);
    else
        hipLaunchKernelGGL((block_small_m_kernel<FMT, S, NB, WIDE, 16>), grid, dim3(64 * waves), lds, p.stream, a);
    return hipGetLastError();
}

template <int FMT, int S, int NB>
hipError_t launch_cols(const BlockMatmul& p) {
    return p.m <= 4 ? launch_one<FMT, S, NB, false>(p) : launch_one<FMT, S, NB, true>(p);
}

}  // namespace

bool block_takes_small_m(const BlockMatmul& p) { return p.m <= 16; }

hipError_t launch_block_small_m(const BlockMatmul& p) {
    const bool gated = p.act >= 0;
    if (p.fmt == kFmtTernary) return gated ? launch_cols<kFmtTernary, 1, 2>(p) : hipErrorInvalidValue;
    switch (p.s) {
        case 1: return gated ? launch_cols<kFmtW4, 1, 2>(p) : launch_cols<kFmtW4, 1, 1>(p);
        case 2: return gated ? launch_cols<kFmtW4, 2, 2>(p) : launch_cols<kFmtW4, 2, 1>(p);
        case 4: return gated ? launch_cols<kFmtW4, 4, 2>(p) : launch_cols<kFmtW4, 4, 1>(p);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace pq2
