// block_small_m.hip -- decode engine of the block operators: products with
// 4-bit weights and the gated feed-forward product for few columns.
//
// A workgroup owns whole tiles of 16 weight rows (gated: the gate tile and
// the up tile of the same rows; some plain products: two tiles at a time),
// one after the other; its waves split k into consecutive slices of whole
// 1024-weight segments.  Per segment a wave forms each weight group's exact
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
// What bounds it is the weight stream, so the kernel keeps it running: a code
// register is loaded again, for the wave's next (tile, segment), as soon as
// its codes are decoded, so a wave holds a segment's loads in flight from its
// start to its end, through the reduction of one tile and into the next.
// The activations are staged once per workgroup, not once per tile.
//
// Up to four columns (MC 4): the four A rows 4c .. 4c+3 of the matrix
// core all belong to column c, so a lane owns one output (column lane/16).
// With S = 2 or 4 weight groups per 128 the rows are told apart by masking:
// row 4c+r keeps only weight group r, and one pair of MFMAs gives the dots
// of all S groups in the four result registers.  Activations sit in LDS;
// they may come unquantised (SRC): each wave then quantises its own slice of
// k while its first weights are on their way, with the exact in-kernel
// quantiser, so the codes are those of pq2_quantize_act_i8.
// Up to sixteen columns (MC 16): A row = column, held in registers in operand
// order (a wave's second segment in LDS; read again per segment where those
// are more, or do not fit); a lane owns four outputs.
#include "block_internal.h"
#include "small_m_common.h"

#include <algorithm>
#include <type_traits>

namespace pq2 {

namespace {

struct SmallArgs {
    const int8_t* q;
    const float* xs;
    const void* x;
    int64_t x_stride;
    const uint8_t* w0;
    const uint8_t* w1;
    void* out;
    int n, k, groups, s8, per_wave, tiles, mtotal, cols, act, out_dtype, part, last_tile;
};

// Waves k is split over at most: registers for three waves per SIMD remain at
// twelve.  (The ternary kernels keep the split of small_m_tiles_kernel.)
constexpr int kW4Waves = 12;

// Groups of codes a wave holds in flight, and of the activations where they
// are read per segment (loads complete in order, so both run the same distance
// ahead).  Eight, a whole segment, is slower: gated ternary at one column 14.3
// against 12.2 us, and twice the registers.
constexpr int kRing = 4;

constexpr int kColPitch = 1024 + 64;  // four columns' reads fall in distinct banks
constexpr int kRowPitch = 1024 + 16;  // sixteen columns' reads fall in distinct banks
constexpr int kLdsBytes = 160 * 1024;

// Where the activations of up to sixteen columns sit: in LDS, whole; where
// they do not fit there, in registers in operand order (a wave with one
// segment), the first segment in registers and the second in LDS (waves with
// two), or read again per segment.
enum : int { kALds = 0, kARegisters = 1, kABoth = 2, kAStream = 3 };

// LDS per wave and segment: the `cols` columns' codes and scales (MC 4), or
// the scales alone, [group][column].
__host__ __device__ constexpr int seg_lds(int mc, int cols) { return mc == 4 ? cols * (kColPitch + 32) : 512; }

template <int FMT, int S, int NB, int MC, int SRC, int AMODE, int MAXW>
__global__ __launch_bounds__(64 * MAXW) void block_small_m_kernel(SmallArgs a) {
#pragma clang fp contract(off)
    constexpr bool WIDE = MC == 16;
    constexpr bool STREAM = WIDE && AMODE == kAStream, BOTH = WIDE && AMODE == kABoth,
                   ALDS = WIDE && AMODE == kALds;
    constexpr bool FUSED = src_fused(SRC);
    constexpr int XL = src_xloads(SRC);
    static_assert(!(WIDE && FUSED), "unquantised activations: up to four columns");
    constexpr int UNIT = block_unit(FMT, S);
    constexpr int CODES = block_code_bytes(FMT);
    constexpr int CB = CODES / 1024;   // code loads per segment
    constexpr int GPL = 8 / CB;        // groups per code load
    constexpr int RG = kRing;
    constexpr int RL = RG / GPL;       // code registers
    constexpr int R = WIDE ? 4 : 1;    // outputs per lane
    constexpr int C = FMT == kFmtTernary ? 8 : 1;  // accumulators per output
    extern __shared__ __align__(16) unsigned char smem[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nwaves = blockDim.x >> 6;
    const int lane = threadIdx.x & 63;
    const int j = lane & 15;
    const int kb = lane >> 4;
    const int m0 = blockIdx.y * a.cols;
    const bool pair = FMT == kFmtW4 && NB == 2 && a.act < 0;  // two neighbouring tiles of one matrix
    const int mcount = min(a.cols, a.mtotal - m0);
    const int seg_bytes = seg_lds(MC, a.cols);
    const int seg_begin = wave * a.per_wave;
    const int seg_end = min(seg_begin + a.per_wave, a.s8);

    const auto q_rs = make_rsrc(FUSED ? nullptr : a.q + (size_t)m0 * a.k, FUSED ? 0u : (uint32_t)(mcount * a.k));
    const auto xs_rs = make_rsrc(FUSED ? nullptr : a.xs + (size_t)m0 * a.groups,
                                 FUSED ? 0u : (uint32_t)(mcount * a.groups * 4));
    const auto x_rs = make_rsrc(
        FUSED ? static_cast<const unsigned char*>(a.x) + (size_t)m0 * a.x_stride * src_esize(SRC) : nullptr,
        FUSED ? (uint32_t)(((int64_t)(mcount - 1) * a.x_stride + a.k) * src_esize(SRC)) : 0u);
    // Per wave: its segments' activations; then two sets of slice sums.
    unsigned char* region = smem + (size_t)wave * a.per_wave * seg_bytes;
    float* parts = reinterpret_cast<float*>(smem + (size_t)nwaves * a.per_wave * seg_bytes);
    // ALDS: the wave's activations; BOTH: its second segment's, if it has one.
    const int a_seg = a.cols * kRowPitch;
    unsigned char* a_lds = reinterpret_cast<unsigned char*>(parts + 2 * a.part) +
                           (size_t)(ALDS ? seg_begin : wave) * a_seg;

    // Loads of one unit (tile, segment); past the last tile they read nothing.
    uint4 cw[NB][RL], sc[NB][S], sn[NB][S == 1 ? 1 : S], av[WIDE && !ALDS ? (STREAM ? 2 * RG : 16) : 1];
    // Codes at `codes` + a scalar offset, scales at `scales`; both are past any
    // range where there is no such tile.
    struct Unit {
        __amdgpu_buffer_rsrc_t rs[2];
        uint32_t codes, scales;
    };
    auto unit_of = [&](int tile, int s) {
        Unit u;
        const bool ok = tile < a.tiles;
        const size_t off = ((size_t)(ok ? (pair ? 2 * tile : tile) : 0) * a.s8 + s) * UNIT;
        u.rs[0] = make_rsrc(a.w0 + off, UNIT);
        const size_t next = pair && 2 * tile < a.last_tile ? (size_t)a.s8 * UNIT : 0;
        u.rs[1] = make_rsrc(NB == 2 ? a.w1 + off + next : a.w0, UNIT);
        u.codes = ok ? 16u * lane : kBufferOOB;
        u.scales = ok ? (uint32_t)(16 * S * j) : kBufferOOB;
        return u;
    };
    auto load_codes = [&](const Unit& u, int i) {
#pragma unroll
        for (int b = 0; b < NB; ++b) cw[b][i % RL] = buf_load16s<kAuxNonTemporal>(u.rs[b], u.codes, 1024u * i);
    };
    auto load_scales = [&](const Unit& u, int i, uint4 (&to)[NB][S]) {
#pragma unroll
        for (int b = 0; b < NB; ++b) to[b][i] = buf_load16s<kAuxNonTemporal>(u.rs[b], u.scales, CODES + 16u * i);
    };
    // WIDE: step i (64 weights, two per group) of segment s.
    const uint32_t a_off = j < mcount ? (uint32_t)(j * a.k + 16 * kb) : kBufferOOB;
    auto load_a = [&](int s, int i) {
        const int off = s * 1024 + 64 * i;
        av[STREAM ? i % (2 * RG) : i] = buf_load16s(q_rs, off < a.k ? a_off : kBufferOOB, off < a.k ? (uint32_t)off : 0u);
    };

    // 1. Stage the wave's activations.  The loads of the first PRE segments go
    //    out first, then the first unit's weights, then the staging writes, so
    //    the weight stream starts at once.
    constexpr int PRE = !WIDE && !FUSED ? 2 : 1;
    struct Staged {
        uint4 v[WIDE && !ALDS ? 1 : MC][FUSED ? XL : 1];
        uint2 x;
    };
    auto stage_load = [&](int s, Staged& t) {
        const int g0 = 8 * s;
        const int off = s * 1024 + 16 * lane;
        if constexpr (WIDE) {
            // Lane (column j, groups 2 kb and 2 kb + 1).
            const bool ok = j < mcount && g0 + 2 * kb < a.groups;
            t.x = buf_load8(xs_rs, ok ? (uint32_t)((j * a.groups + g0 + 2 * kb) * 4) : kBufferOOB);
            if constexpr (ALDS) {
#pragma unroll
                for (int i = 0; i < MC; ++i)
                    if (i < mcount) t.v[i][0] = buf_load16(q_rs, off < a.k ? (uint32_t)(i * a.k + off) : kBufferOOB);
            }
        } else if constexpr (FUSED) {
#pragma unroll
            for (int i = 0; i < MC; ++i) {
                if (i >= mcount) continue;
                const uint32_t at = (uint32_t)((i * a.x_stride + off) * src_esize(SRC));
#pragma unroll
                for (int l = 0; l < XL; ++l) t.v[i][l] = buf_load16(x_rs, off < a.k ? at + 16u * l : kBufferOOB);
            }
        } else {
            // Lane 8 c + g: the scale of column c, group g.
            const bool ok = lane < 8 * mcount && g0 + (lane & 7) < a.groups;
            t.x.x = buf_load4(xs_rs, ok ? (uint32_t)(((lane >> 3) * a.groups + g0 + (lane & 7)) * 4) : kBufferOOB);
#pragma unroll
            for (int i = 0; i < MC; ++i)
                if (i < mcount) t.v[i][0] = buf_load16(q_rs, off < a.k ? (uint32_t)(i * a.k + off) : kBufferOOB);
        }
    };
    auto stage_store = [&](int s, const Staged& t) {
        unsigned char* to = region + (s - seg_begin) * seg_bytes;
        float* xl = reinterpret_cast<float*>(to + (WIDE ? 0 : a.cols * kColPitch));
        if constexpr (WIDE) {
            xl[(2 * kb) * 16 + j] = __uint_as_float(t.x.x);
            xl[(2 * kb + 1) * 16 + j] = 8 * s + 2 * kb + 1 < a.groups ? __uint_as_float(t.x.y) : 0.0f;
            if constexpr (ALDS) {
#pragma unroll
                for (int i = 0; i < MC; ++i)
                    if (i < mcount)
                        *reinterpret_cast<uint4*>(a_lds + (s - seg_begin) * a_seg + i * kRowPitch + 16 * lane) = t.v[i][0];
            }
        } else {
#pragma unroll
            for (int i = 0; i < MC; ++i) {
                if (i >= mcount) continue;
                uint4 v;
                if constexpr (FUSED) {
                    float f[16], scale;
                    x_to_float16<SRC>(t.v[i], f);
                    v = quantize16(f, scale);  // the eight lanes of a group agree
                    if ((lane & 7) == 0) xl[8 * i + (lane >> 3)] = scale;
                } else {
                    v = t.v[i][0];
                }
                *reinterpret_cast<uint4*>(to + i * kColPitch + 16 * lane) = v;
            }
            if constexpr (!FUSED) {
                if (lane < 8 * mcount) xl[lane] = __uint_as_float(t.x.x);
            }
        }
    };
    {
        Staged t[PRE];
#pragma unroll
        for (int i = 0; i < PRE; ++i)
            if (i == 0 || seg_begin + i < seg_end) stage_load(seg_begin + i, t[i]);
        const Unit u = unit_of(blockIdx.x, seg_begin);
        if constexpr (WIDE && !ALDS) {
            // (BOTH: the second segment's first, on their way to LDS.)
            const int s = BOTH ? min(seg_begin + 1, a.s8 - 1) : seg_begin;
#pragma unroll
            for (int i = 0; i < (STREAM ? 2 * RG : 16); ++i) load_a(s, i);
        }
#pragma unroll
        for (int i = 0; i < S; ++i) load_scales(u, i, sc);
#pragma unroll
        for (int i = 0; i < RL; ++i) load_codes(u, i);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < PRE; ++i)
            if (i == 0 || seg_begin + i < seg_end) stage_store(seg_begin + i, t[i]);
        if constexpr (BOTH) {
            if (seg_begin + 1 < seg_end) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (j < mcount) *reinterpret_cast<uint4*>(a_lds + j * kRowPitch + 64 * i + 16 * kb) = av[i];
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) load_a(seg_begin, i);
        }
        for (int s = seg_begin + PRE; s < seg_end; ++s) {
            stage_load(s, t[0]);
            stage_store(s, t[0]);
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");

    // Rows of the A operand that keep weight group r = j & 3 of step h.
    uint32_t keep[2] = {~0u, ~0u};
    if constexpr (!WIDE && S > 1) {
#pragma unroll
        for (int h = 0; h < 2; ++h) keep[h] = (j & 3) == (S == 2 ? h : 2 * h + (kb >> 1)) ? ~0u : 0u;
    }
    const uint32_t low_half = kb < 2 ? ~0u : 0u;  // WIDE, S = 4: lanes of the first 32 weights of a step
    const int a_col = (j >> 2) < mcount ? (j >> 2) : 0;
    const int x_col = kb < mcount ? kb : 0;

    float acc[NB][C][R];
    // One unit: group dots and terms; the loads of the next unit go out as this
    // one's registers become free.  (Two or four scale registers a unit are
    // used in turn and stream like the codes; a single one has a second set.)
    auto body = [&](int tile, int s, int next_tile, int next_s, auto lds_c) {
        constexpr bool LDS_A = ALDS || (BOTH && decltype(lds_c)::value);
        const unsigned char* from = region + (s - seg_begin) * seg_bytes;
        const Unit next = unit_of(next_tile, next_s);
        const Unit cur = RG < 8 ? unit_of(tile, s) : next;
        float4 xv[2];
        if constexpr (!WIDE) {
            const float4* x = reinterpret_cast<const float4*>(from + a.cols * kColPitch + 32 * x_col);
            xv[0] = x[0];
            xv[1] = x[1];
        }
        if constexpr (S == 1) load_scales(next, 0, sn);
        const unsigned char* a_base = from + a_col * kColPitch + 16 * kb;
        const unsigned char* wide_base = a_lds + (ALDS ? (s - seg_begin) * a_seg : 0) +
                                         (j < mcount ? j : 0) * kRowPitch + 16 * kb;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
            v4i A[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint4 v;
                if constexpr (LDS_A) v = *reinterpret_cast<const uint4*>(wide_base + 128 * g + 64 * h);
                else if constexpr (WIDE) v = av[STREAM ? (2 * g + h) % (2 * RG) : 2 * g + h];
                else v = *reinterpret_cast<const uint4*>(a_base + 128 * g + 64 * h);
                A[h] = v4i{(int)(v.x & keep[h]), (int)(v.y & keep[h]), (int)(v.z & keep[h]), (int)(v.w & keep[h])};
            }
            float xg[R];
            if constexpr (WIDE) {
                const float4 v = *reinterpret_cast<const float4*>(from + (g * 16 + 4 * kb) * 4);
                xg[0] = v.x; xg[1] = v.y; xg[2] = v.z; xg[3] = v.w;
            } else {
                const float4& v = xv[g >> 2];
                xg[0] = (g & 3) == 0 ? v.x : (g & 3) == 1 ? v.y : (g & 3) == 2 ? v.z : v.w;
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                v4i B[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (FMT == kFmtTernary) B[h] = ternary_operand(word_of(cw[b][(g >> 1) % RL], 2 * (g & 1) + h));
                    else B[h] = w4_operand(word_of(cw[b][g % RL], 2 * h), word_of(cw[b][g % RL], 2 * h + 1));
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
                    const float ws = weight_scale_at<FMT>(sc[b][0], g);
#pragma unroll
                    for (int r = 0; r < R; ++r) acc[b][g][r] = __builtin_fmaf(dot[0][r] * xg[r], ws, acc[b][g][r]);
                } else {
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        float t = dot[0][r] * weight_scale_at<FMT>(sc[b][(g * S) >> 3], (g * S) & 7);
#pragma unroll
                        for (int u = 1; u < S; ++u) {
                            const int i = g * S + u;
                            t = __builtin_fmaf(dot[u][r], weight_scale_at<FMT>(sc[b][i >> 3], i & 7), t);
                        }
                        acc[b][0][r] = __builtin_fmaf(t, xg[r], acc[b][0][r]);
                    }
                }
                // The fullest register kernels: one matrix after the other, or they
                // spill (K = 10240, N = 8192 gated, m = 16, wgroup 64 / 128 20.9 / 18.7
                // us, without 22.6 / 19.3).
                if constexpr (WIDE && AMODE == kARegisters && NB == 2) {
                    if (b == 0) __builtin_amdgcn_sched_barrier(0);
                }
            }
            if (g % GPL == GPL - 1) {
                const int i = g / GPL + RL;
                load_codes(i < CB ? cur : next, i % CB);
            }
            if constexpr (S != 1) {
                constexpr int kPer = 8 / S;  // groups of one scale register
                if (g % kPer == kPer - 1) load_scales(next, g / kPer, sc);
            }
            if constexpr (STREAM) {
                const int i = 2 * (g + RG);
                load_a(i < 16 ? s : next_s, i % 16);
                load_a(i < 16 ? s : next_s, i % 16 + 1);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (S == 1) {
#pragma unroll
            for (int b = 0; b < NB; ++b) sc[b][0] = sn[b][0];
        }
    };

    // 2. The tiles, with two sets of slice sums in turn: one barrier per tile.
    int turn = 0;
    for (int tile = blockIdx.x; tile < a.tiles; tile += gridDim.x, turn ^= 1) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int r = 0; r < R; ++r) acc[b][c][r] = 0.0f;
        for (int s = seg_begin; s < seg_end; ++s) {
            const bool last = s + 1 == seg_end;
            const int nt = last ? tile + (int)gridDim.x : tile, ns = last ? seg_begin : s + 1;
            if constexpr (BOTH) {
                if (s == seg_begin) body(tile, s, nt, ns, std::false_type{});
                else body(tile, s, nt, ns, std::true_type{});
            } else {
                body(tile, s, nt, ns, std::false_type{});
            }
        }
        float* part = parts + turn * a.part;
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
                if (col < mcount) part[((wave * NB + b) * mcount + col) * 16 + j] = v;
            }
        __syncthreads();
        for (int o = threadIdx.x; o < mcount * 16; o += blockDim.x) {
            float y[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float sum = 0.0f;
                for (int w = 0; w < nwaves; ++w) {
                    const float v = part[(w * NB + b) * mcount * 16 + o];
                    sum = w == 0 ? v : sum + v;
                }
                y[b] = sum;
            }
            const int row = (pair ? 2 * tile : tile) * 16 + (o & 15);
            const size_t at = (size_t)(m0 + (o >> 4)) * a.n + row;
            if (NB == 2 && !pair) {
                if (row < a.n) store_as(a.out, at, gate_activation(y[0], a.act) * y[NB - 1], a.out_dtype);
            } else {
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    if (row + 16 * b < a.n) static_cast<float*>(a.out)[at + 16 * b] = y[b];
            }
        }
    }
}

// LDS of a launch.
template <int NB, int MC, int AMODE>
size_t lds_bytes(const SmallArgs& a, int waves) {
    const int held = MC == 4 ? 0 : AMODE == kALds ? a.s8 : AMODE == kABoth ? a.s8 - waves : 0;
    return (size_t)waves * a.per_wave * seg_lds(MC, a.cols) + (size_t)2 * waves * NB * a.cols * 64 +
           (size_t)held * a.cols * kRowPitch;
}

template <int FMT, int S, int NB, int MC, int SRC, int AMODE, int MAXW>
hipError_t launch_one(const BlockMatmul& p, SmallArgs a, int waves) {
    constexpr int RG = kRing, GPL = FMT == kFmtTernary ? 2 : 1;
    a.part = waves * NB * a.cols * 16;
    const size_t lds = lds_bytes<NB, MC, AMODE>(a, waves);
    const int passes = (int)((p.m + a.cols - 1) / a.cols);
    // Persistent workgroups.  The stream is fastest with about 64 KB in flight
    // per CU, and more only slows it (FFN up, one column: 4-bit weights 10.7 /
    // 9.6 / 9.7 / 9.7 us at one / two / three / four workgroups of five waves a
    // CU; gated ternary 15.4 / 12.4 / 12.1 / 12.6).  Wide kernels have more to
    // load first: gated 4-bit m = 8 18.0 / 17.5 / 19.7 us at one / two / three,
    // m = 16 18.9 / 20.4 / 22.7.
    constexpr int kWaveKB = RG / GPL * NB;
    const int per_cu = std::max(1, (MC == 16 ? (a.cols > 8 ? 8 : 12) : 64 / kWaveKB) / waves);
    const dim3 grid((unsigned)std::min(a.tiles, 256 * per_cu), (unsigned)passes);
    clear_stale_error();
    hipLaunchKernelGGL((block_small_m_kernel<FMT, S, NB, MC, SRC, AMODE, MAXW>), grid, dim3(64 * waves), lds, p.stream,
                       a);
    return hipGetLastError();
}

template <int FMT, int S, int NB>
hipError_t launch_cols(const BlockMatmul& p) {
    const int tiles = (int)((p.n + 15) / 16);
    const bool pair = NB == 2 && p.act < 0;
    SmallArgs a{p.q, p.xs, p.x, p.x_stride, p.w0, pair ? p.w0 : p.w1, p.out, (int)p.n, (int)p.k, (int)(p.k / 128),
                (int)((p.k + 1023) / 1024), 0, pair ? (tiles + 1) / 2 : tiles, (int)p.m, 0, p.act, p.out_dtype, 0,
                tiles - 1};
    constexpr int kMany = FMT == kFmtTernary ? kTilesDefaultWaves : kW4Waves;
    a.per_wave = (a.s8 + kMany - 1) / kMany;
    const int waves = (a.s8 + a.per_wave - 1) / a.per_wave;
    if (p.m > 4) {
        a.cols = (int)std::min<int64_t>(p.m, 16);
        if (lds_bytes<NB, 16, kALds>(a, waves) <= kLdsBytes) {
            if (waves <= 8) return launch_one<FMT, S, NB, 16, kSrcNatural, kALds, 8>(p, a, waves);
            return launch_one<FMT, S, NB, 16, kSrcNatural, kALds, kMany>(p, a, waves);
        }
        if constexpr (NB == 1) {
            // K = 17408, N = 5120, m = 16: kABoth 18.9 against 23.7 us streamed; with
            // four scales a group, or two matrices, the registers spill (three of
            // them at wgroup 64 as it is).
            const bool both = S <= 2 && a.per_wave == 2 && lds_bytes<NB, 16, kABoth>(a, waves) <= kLdsBytes;
            const bool registers = S <= 2 && a.per_wave == 1;
            // Two tiles at a time: twice the weights in flight and half the
            // activations streamed.  Wins where these are streamed anyway (m = 16,
            // K = 17408, wgroup 32, N = 5120 / 8192 / 17408 26.3 / 30.6 / 63.4 us
            // against 21.5 / 25.2 / 55.9) and where one round of pairs replaces two of
            // tiles (wgroup 64, N = 5120 / 8192 20.2 / 22.8 against 18.5 / 22.1; N =
            // 10240 27.6 against 34.6); loses where half the CUs would idle (wgroup
            // 32, N = 4096 17.7 against 21.1).
            if (tiles > 256 && (both ? tiles <= 512 : !registers)) return launch_cols<FMT, S, 2>(p);
            if constexpr (S <= 2) {
                if (both) return launch_one<FMT, S, NB, 16, kSrcNatural, kABoth, kMany>(p, a, waves);
            }
        }
        // K = 10240, N = 8192 gated, m = 16: wgroup 128 in registers 18.9 us,
        // streamed 24.6; but with four scales a group (67.9 against 30.0) or the
        // ternary kernel's eight sums and sixteen waves (41.5 against 31.8) the
        // registers spill more than streaming's (45 in the ternary kernel, which
        // sixteen waves leave 128 registers; none in the 4-bit ones).
        if constexpr (FMT == kFmtW4 && S <= 2) {
            if (a.per_wave == 1) return launch_one<FMT, S, NB, 16, kSrcNatural, kARegisters, kMany>(p, a, waves);
        }
        return launch_one<FMT, S, NB, 16, kSrcNatural, kAStream, kMany>(p, a, waves);
    }
    // LDS holds all of k for the columns of a pass: two at most beyond 32768.
    a.cols = (int)(p.k > 32768 ? std::min<int64_t>(p.m, 2) : p.m);
    switch (p.src) {
        case kSrcNatural: return launch_one<FMT, S, NB, 4, kSrcNatural, kALds, kMany>(p, a, waves);
        case kSrcBf16: return launch_one<FMT, S, NB, 4, kSrcBf16, kALds, kMany>(p, a, waves);
        case kSrcF16: return launch_one<FMT, S, NB, 4, kSrcF16, kALds, kMany>(p, a, waves);
        case kSrcF32: return launch_one<FMT, S, NB, 4, kSrcF32, kALds, kMany>(p, a, waves);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

// Passes of sixteen columns read the weights again, from the Infinity Cache.
// Up to two passes, or about three workgroups a CU in all, are faster than the
// prefill engine, whose workgroups each walk k alone.  Decode / prefill: N =
// 6144, K = 5120 m = 17 9.3 / 15.5 us, FFN down m = 17 29 / 50; K = 11264, N = 109
// m = 200 / 800 (350 workgroups) 12.3 / 25.7, 21.2 / 26.0; K = 4096, N = 2700,
// wgroup 32 m = 64 (676) 10.2 / 17.8, gated ternary 13.9 / 20.5, m = 96 (1014) 14.2
// / 17.6 and 19.6 / 18.3; K = 5120, N = 300 m = 800 (950) 19.9 / 16.1.  Three
// passes hold out to 1152: N = 6144, K = 5120, m = 48 15.2 / 15.8, FFN down m =
// 40 34.2 / 44.4.  The ternary kernels stream the activations from K = 8192 on,
// slowly: one workgroup a CU there (K = 11264, N = 109 m = 400 / 800 27.8 / 41.2,
// 47.7 / 41.9).
// The rule knows neither the weight group nor k beyond that, and misses sizes on
// both sides: decode would be faster at m = 64 for N = 4096, K = 8192 wgroup 32 /
// 128 (24.4 / 33.1, 20.8 / 22.5), N = 5120, K = 17408 wgroup 32 (56.9 / 71.4) and N =
// 4096, K = 12288 gated wgroup 64 (55.0 / 60.4), but not wgroup 128 there (37.2 /
// 32.4) nor gated ternary (57.5 / 38.2 at N = 4096, K = 8192); prefill at m = 96
// for N = 2000, K = 1024 wgroup 64 (6.7 / 6.3).
bool block_takes_small_m(const BlockMatmul& p) {
    const int64_t passes = (p.m + 15) / 16, tiles = (p.n + 15) / 16;
    const int64_t most = p.fmt == kFmtTernary && p.k > 7168 ? 256 : passes == 3 ? 1152 : 768;
    return passes <= 2 || passes * tiles <= most;
}

// Quantising in the product's launch saves the quantiser's (about 2 us on the
// GPU, 3 on the host) and costs what the extra columns take to quantise in
// every workgroup.  Complete calls, one launch against two: QKV 4-bit at
// m = 1 / 2 / 3 / 4 6.7 / 7.5 / 8.5 / 9.5 against 8.8 / 8.9 / 9.2 / 9.3 us, FFN
// up gated ternary 12.1 / 12.4 / 13.4 / 15.0 against 13.8 / 14.0 / 14.2 / 14.5,
// gated 4-bit at m = 4 18.6 against 19.5.
// A wave's second segment of k is quantised behind the first: FFN down 4-bit at
// m = 2 / 4 12.5 / 16.3 against 13.5 / 16.0, from FP32 18.7 against 14.8.
bool block_takes_x(int64_t m, int64_t k) { return m * ((k + 1024 * kW4Waves - 1) / (1024 * kW4Waves)) <= 4; }

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
