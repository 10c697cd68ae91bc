// block_prefill.hip -- prefill engine of the block operators: products with
// 4-bit weights and the gated feed-forward product for many columns.
//
// A workgroup of four waves owns BM = 16 MT activation rows and 64 NT weight
// rows (gated: of each matrix); a wave owns 16 NT of them, so every weight
// is loaded and decoded once per workgroup, by the one wave that multiplies
// with it: both tile layouts hold the INT8 matrix core's B operand order, so
// codes go from memory to registers and, decoded there, to
// v_mfma_i32_16x16x64_i8 without passing through LDS.  The activations are
// shared by the waves and go through LDS, double-buffered by group of 128
// (loads run D groups ahead, in registers),
// quads XOR-swizzled so that the 16 rows of an operand read fall in distinct
// banks.  Gate and up tiles of the same rows sit in one wave's registers, so
// the gated epilogue needs no exchange.
//
// Each output adds one FP32 term per activation group, in k order, with the
// terms of block_small_m.hip.  That rescale (a conversion, a product and a
// multiply-add per output and weight group, 12 issue cycles against 8 of the
// matrix core for the group's 128 multiply-adds) bounds the kernel.
#include "../../include/pq2_block.h"
#include "block_internal.h"

#include <algorithm>
#include <type_traits>

namespace pq2 {

namespace {

struct PrefillArgs {
    const int8_t* q;
    const float* xs;
    const uint8_t* w0;
    const uint8_t* w1;
    void* out;
    int m, n, k, groups, s8, tiles, nblk, mblk, act, out_dtype;
};

// Slot (16-byte quads) of quad t of row i of an A buffer.
__device__ __forceinline__ int a_slot(int i, int t) { return i * 8 + (t ^ ((i >> 1) & 7)); }

template <int FMT, int S, int NB, int MT, int NT, int D>
__global__ __launch_bounds__(256) void block_prefill_kernel(PrefillArgs a) {
#pragma clang fp contract(off)
    constexpr int UNIT = block_unit(FMT, S);
    constexpr int CODES = block_code_bytes(FMT);
    constexpr int BM = 16 * MT;
    constexpr int AQ = BM * 8 / 256;   // quads staged per thread and group
    constexpr int XQ = BM * 8 / 256;   // activation scales staged per thread and segment
    static_assert(BM * 8 % 256 == 0, "rows per workgroup");
    __shared__ uint4 As[2][BM * 8];
    __shared__ __align__(16) float Xs[2][8][BM];

    int nb, mb;
    {
        // Consecutive workgroups go to the eight XCDs in turn: those of one
        // XCD walk the row blocks of one column block, so its weights stay in
        // that XCD's L2.
        const int bid = blockIdx.x;
        if (a.nblk >= 8) {
            const int i = bid >> 3;
            nb = (i / a.mblk) * 8 + (bid & 7);
            mb = i % a.mblk;
            if (nb >= a.nblk) return;
        } else {
            nb = bid % a.nblk;
            mb = bid / a.nblk;
        }
    }
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63;
    const int j = lane & 15;
    const int kb = lane >> 4;
    const int row0 = mb * BM;
    const int rows = min(BM, a.m - row0);
    const int tile0 = (nb * 4 + wave) * NT;  // this wave's first tile

    const auto q_rs = make_rsrc(a.q + (size_t)row0 * a.k, (uint32_t)(rows * a.k));
    const auto x_rs = make_rsrc(a.xs + (size_t)row0 * a.groups, (uint32_t)(rows * a.groups * 4));
    // Tiles past the last re-read it (their outputs are not stored).
    const int first = min(nb * 4 * NT, a.tiles - 1);
    const int here = min(4 * NT, a.tiles - first);
    const size_t w_off = (size_t)first * a.s8 * UNIT;
    const uint32_t w_bytes = (uint32_t)(here * a.s8 * UNIT);
    const __amdgpu_buffer_rsrc_t w_rs[2] = {make_rsrc(a.w0 + w_off, w_bytes),
                                            make_rsrc(NB == 2 ? a.w1 + w_off : nullptr, NB == 2 ? w_bytes : 0u)};
    uint32_t t_off[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) t_off[t] = (uint32_t)(min(tile0 + t - first, here - 1) * a.s8 * UNIT);

    // Staging roles: quad it & 7 of row it >> 3; rows past the last read it again.
    uint32_t q_off[AQ];
    int q_slot[AQ];
#pragma unroll
    for (int p = 0; p < AQ; ++p) {
        const int it = tid + 256 * p;
        q_off[p] = (uint32_t)(min(it >> 3, rows - 1) * a.k + 16 * (it & 7));
        q_slot[p] = a_slot(it >> 3, it & 7);
    }
    // D groups ahead: activations on their way to LDS, and packed codes
    // (ternary: pairs of groups), each loaded again as soon as it is used.
    // Weight scales: RS sets of 16 bytes, 8 / S groups each.
    constexpr int DC = FMT == kFmtTernary ? (D + 1) / 2 : D;
    constexpr int RS = D > 1 && S == 4 ? 4 : 2;
    constexpr int SG = 8 / S;
    uint4 areg[D][AQ];
    uint32_t xreg[XQ];
    uint4 cw[DC][NB][NT];
    uint4 sc[RS][NB][NT];

    auto load_a = [&](int g, int set) {
#pragma unroll
        for (int p = 0; p < AQ; ++p) areg[set][p] = buf_load16s(q_rs, q_off[p], 128u * g);
    };
    auto load_xs = [&](int seg) {
#pragma unroll
        for (int p = 0; p < XQ; ++p) {
            const int it = tid + 256 * p;
            const int g = 8 * seg + (it & 7);
            xreg[p] = buf_load4(x_rs, g < a.groups ? (uint32_t)((min(it >> 3, rows - 1) * a.groups + g) * 4) : kBufferOOB);
        }
    };
    auto load_codes = [&](int g, int set) {
        const uint32_t off = (uint32_t)((g >> 3) * UNIT + (FMT == kFmtTernary ? ((g & 7) >> 1) : (g & 7)) * 1024);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int t = 0; t < NT; ++t) cw[set][b][t] = buf_load16s(w_rs[b], 16 * lane, off + t_off[t]);
    };
    // The scales of groups g .. g + SG - 1 (g a multiple of SG).
    auto load_scales = [&](int g, int set) {
        const uint32_t off = (uint32_t)((g >> 3) * UNIT + CODES + 16 * ((g & 7) / SG));
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int t = 0; t < NT; ++t) sc[set][b][t] = buf_load16s(w_rs[b], 16 * S * j, off + t_off[t]);
    };
    auto store_a = [&](int buf, int set) {
#pragma unroll
        for (int p = 0; p < AQ; ++p) As[buf][q_slot[p]] = areg[set][p];
    };
    auto store_xs = [&](int buf) {
#pragma unroll
        for (int p = 0; p < XQ; ++p) {
            const int it = tid + 256 * p;
            Xs[buf][it & 7][it >> 3] = __uint_as_float(xreg[p]);
        }
    };

    v4f acc[NB][NT][MT];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[b][t][i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const int low_half = kb < 2 ? -1 : 0;

    // Loads behind the last group: a branch around them costs copies of every
    // register they write and ends the scheduler's region, so the kernels of
    // full grids (D < 4) read the last group again instead.  The latency kernel
    // (D = 4) has no VALU to spare but a short k to end: it skips them.
    const int last = a.groups - 1;
    auto wanted = [&](int g) { return D < 4 || g <= last; };
    load_a(0, 0);
    load_xs(0);
    load_codes(0, 0);
    load_scales(0, 0);
#pragma unroll
    for (int i = 1; i < D; ++i)
        if (wanted(i)) {
            load_a(min(i, last), i);
            if (FMT == kFmtW4 || i % 2 == 0) load_codes(min(i, last), FMT == kFmtW4 ? i : i / 2);
        }
#pragma unroll
    for (int i = 1; i < RS; ++i) load_scales(min(i * SG, last), i);
    store_a(0, 0);
    store_xs(0);
    __syncthreads();

    // One group; u = g modulo 8 (a constant).  Group g + D is loaded while g
    // is multiplied, and g + 1 staged into the other buffer after it.
    auto step = [&](int g, auto uc) {
        constexpr int u = decltype(uc)::value;
        constexpr int buf = u & 1;
        constexpr int cs = (FMT == kFmtTernary ? u / 2 : u) % DC;   // code set of this group
        constexpr int ss = u / SG % RS;                             // scale set
        if (wanted(g + D)) load_a(min(g + D, last), u % D);
        v4i B[NB][NT][2];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (FMT == kFmtTernary) B[b][t][h] = ternary_operand(word_of(cw[cs][b][t], 2 * (u & 1) + h));
                    else B[b][t][h] = w4_operand(word_of(cw[cs][b][t], 2 * h), word_of(cw[cs][b][t], 2 * h + 1));
                }
        if constexpr (FMT == kFmtW4) {
            if (wanted(g + D)) load_codes(min(g + D, last), cs);
        } else if constexpr (u % 2 == 1) {
            if (wanted(g - 1 + 2 * DC)) load_codes(min(g - 1 + 2 * DC, last), cs);
        }
        // The scale set before this one is free from its last group on.  (S = 1:
        // a set lasts the whole unroll, so the next one moves down.)
        if constexpr (S == 1 && u == 0) {
            if (g > 0) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int t = 0; t < NT; ++t) sc[0][b][t] = sc[1][b][t];
            }
            if (wanted(g + 8)) load_scales(min(g + 8, last), 1);
        } else if constexpr (u % SG == 0) {
            if (wanted(g + (RS - 1) * SG)) load_scales(min(g + (RS - 1) * SG, last), (ss + RS - 1) % RS);
        }
        if constexpr (u == 0) {
            if (wanted(g + 8)) load_xs((g >> 3) + 1);
        }
        const float* xrow = &Xs[(g >> 3) & 1][g & 7][0];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            v4i A[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 v = As[buf][a_slot(16 * i + j, 4 * h + kb)];
                A[h] = v4i{(int)v.x, (int)v.y, (int)v.z, (int)v.w};
            }
            const float4 xv = *reinterpret_cast<const float4*>(xrow + 16 * i + 4 * kb);
            const float x[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    if constexpr (S == 1) {
                        v4i dot = __builtin_amdgcn_mfma_i32_16x16x64_i8(A[0], B[b][t][0], v4i{}, 0, 0, 0);
                        dot = __builtin_amdgcn_mfma_i32_16x16x64_i8(A[1], B[b][t][1], dot, 0, 0, 0);
                        const float ws = weight_scale_at<FMT>(sc[ss][b][t], u);
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[b][t][i][r] = FMT == kFmtTernary
                                                  ? __builtin_fmaf((float)dot[r] * x[r], ws, acc[b][t][i][r])
                                                  : __builtin_fmaf((float)dot[r] * ws, x[r], acc[b][t][i][r]);
                    } else {
                        float sum[4];
#pragma unroll
                        for (int s = 0; s < S; ++s) {
                            const int h = S == 2 ? s : s >> 1;
                            v4i Am = A[h];
                            if constexpr (S == 4) {
                                const int mask = (s & 1) ? ~low_half : low_half;
                                Am = v4i{Am[0] & mask, Am[1] & mask, Am[2] & mask, Am[3] & mask};
                            }
                            const v4i dot = __builtin_amdgcn_mfma_i32_16x16x64_i8(Am, B[b][t][h], v4i{}, 0, 0, 0);
                            const float ws = weight_scale_at<FMT>(sc[ss][b][t], u % SG * S + s);
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                sum[r] = s == 0 ? (float)dot[r] * ws : __builtin_fmaf((float)dot[r], ws, sum[r]);
                        }
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[b][t][i][r] = __builtin_fmaf(sum[r], x[r], acc[b][t][i][r]);
                    }
                }
        }
        if (wanted(g + 1)) store_a(buf ^ 1, (u + 1) % D);
        if constexpr (u == 7) store_xs(((g >> 3) + 1) & 1);
        __syncthreads();
    };
    for (int g = 0; g < a.groups; g += 8) {
        step(g, std::integral_constant<int, 0>{});
        if (g + 1 < a.groups) step(g + 1, std::integral_constant<int, 1>{});
        if (g + 2 < a.groups) step(g + 2, std::integral_constant<int, 2>{});
        if (g + 3 < a.groups) step(g + 3, std::integral_constant<int, 3>{});
        if (g + 4 < a.groups) step(g + 4, std::integral_constant<int, 4>{});
        if (g + 5 < a.groups) step(g + 5, std::integral_constant<int, 5>{});
        if (g + 6 < a.groups) step(g + 6, std::integral_constant<int, 6>{});
        if (g + 7 < a.groups) step(g + 7, std::integral_constant<int, 7>{});
    }

#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int col = (tile0 + t) * 16 + j;
        if (col >= a.n) continue;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = row0 + 16 * i + 4 * kb + r;
                if (row >= a.m) continue;
                const size_t at = (size_t)row * a.n + col;
                if constexpr (NB == 2)
                    store_as(a.out, at, gate_activation(acc[0][t][i][r], a.act) * acc[1][t][i][r], a.out_dtype);
                else
                    static_cast<float*>(a.out)[at] = acc[0][t][i][r];
            }
    }
}

template <int FMT, int S, int NB, int MT, int NT, int D>
hipError_t launch_one(const BlockMatmul& p) {
    PrefillArgs a{p.q, p.xs, p.w0, p.w1, p.out, (int)p.m, (int)p.n, (int)p.k, (int)(p.k / 128), (int)((p.k + 1023) / 1024),
                  (int)((p.n + 15) / 16), 0, 0, p.act, p.out_dtype};
    a.nblk = (a.tiles + 4 * NT - 1) / (4 * NT);
    // A launch holds fewer than 2^32 threads: outputs of some 10^10 elements
    // take several, each of whole workgroup rows.  PQ2_MAX_BLOCK_N keeps a row
    // of the narrowest blocks (64 columns) within one.
    constexpr int64_t kMostGroups = (int64_t)UINT32_MAX / 256;
    static_assert((PQ2_MAX_BLOCK_N + 63) / 64 % 8 == 0 && (PQ2_MAX_BLOCK_N + 63) / 64 <= kMostGroups, "a row of workgroups");
    const int64_t per_row = a.nblk >= 8 ? (int64_t)8 * ((a.nblk + 7) / 8) : a.nblk;
    const int64_t most = kMostGroups / per_row * (16 * MT);
    for (int64_t m0 = 0; m0 < p.m; m0 += most) {
        a.m = (int)std::min(p.m - m0, most);
        a.mblk = (a.m + 16 * MT - 1) / (16 * MT);
        a.q = p.q + m0 * p.k;
        a.xs = p.xs + m0 * (p.k / 128);
        const int size = NB == 2 && p.out_dtype != 2 ? 2 : 4;
        a.out = static_cast<unsigned char*>(p.out) + m0 * p.n * size;
        clear_stale_error();
        hipLaunchKernelGGL((block_prefill_kernel<FMT, S, NB, MT, NT, D>), dim3((unsigned)(per_row * a.mblk)), dim3(256),
                           0, p.stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Tile choice by the number of workgroups, against the 256 CUs.
//  * While all 32-row workgroups are resident at once (four a CU; gated, which
//    needs more registers, three or two): what counts is a group's latency,
//    so loads run four groups ahead, and plain products take one 16-row
//    weight tile per wave.  (K = 5120, N = 6144: m = 64 15.8 us against 28.4 with
//    loads one group ahead and two tiles a wave; FFN down, m = 256 56 / 89;
//    FFN up gated, m = 64 41.2 / 42.5.)  Above that, fewer registers are
//    better: gated m = 96 46 us against 53, N = 6144 m = 512 32.9 against 36.4.
//  * From two 64-row workgroups a CU on, 64 rows (FFN up gated m = 1024, 335
//    against 384 us; 4-bit m = 1024 / 256 153 / 49.7 against 169 / 56.0; N =
//    6144, m = 512, one and a half a CU, 41.0 against 32.9), except with
//    smaller weight groups, whose 64-row kernels hold two waves per SIMD
//    (wgroup 64: 223 against 200).  The 4-bit kernels have the registers to
//    load two groups ahead (gated m = 1024 294 against 302 us); the ternary one
//    would drop to two waves per SIMD (382 against 330).
// Four tiles per wave or 128 rows measured no faster (327 and 341 us).
template <int FMT, int S, int NB>
hipError_t launch_variant(const BlockMatmul& p) {
    constexpr int NT = 2 / NB;
    const int64_t cols = (p.n + 64 * NT - 1) / (64 * NT);
    constexpr int kResident = 256 * (NB == 1 ? 4 : S == 4 ? 2 : 3);
    if (((p.n + 63) / 64) * ((p.m + 31) / 32) <= kResident) return launch_one<FMT, S, NB, 2, 1, 4>(p);
    if constexpr (S == 1) {
        if (cols * ((p.m + 63) / 64) >= 512) return launch_one<FMT, S, NB, 4, NT, FMT == kFmtW4 ? 2 : 1>(p);
    }
    return launch_one<FMT, S, NB, 2, NT, 1>(p);
}

}  // namespace

hipError_t launch_block_prefill(const BlockMatmul& p) {
    const bool gated = p.act >= 0;
    if (p.fmt == kFmtTernary) return gated ? launch_variant<kFmtTernary, 1, 2>(p) : hipErrorInvalidValue;
    switch (p.s) {
        case 1: return gated ? launch_variant<kFmtW4, 1, 2>(p) : launch_variant<kFmtW4, 1, 1>(p);
        case 2: return gated ? launch_variant<kFmtW4, 2, 2>(p) : launch_variant<kFmtW4, 2, 1>(p);
        case 4: return gated ? launch_variant<kFmtW4, 4, 2>(p) : launch_variant<kFmtW4, 4, 1>(p);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace pq2
