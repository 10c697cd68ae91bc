// w4.hip -- the 4-bit weight layout (one-time preparation).
//
// The layout is stated in include/pq2_block.h: the 16-row tiles and segment
// units of the ternary tile layout with 1 KB per group of 128 weights, so
// that every code load of a wave reads one contiguous kilobyte in the INT8
// matrix core's operand order.  Codes are kept as the two's complement of
// c - 8: masking the halves of a byte then gives 16 times the signed weight.
#include "block_internal.h"

#include <algorithm>

namespace pq2 {

namespace {

// One 16-byte lane chunk of a code block at a time: chunk = (unit, b, lane).
__global__ __launch_bounds__(256) void prepare_w4_codes_kernel(const uint8_t* __restrict__ codes, int64_t stride,
                                                               int64_t n, int64_t k, int s8, int unit_bytes,
                                                               int64_t chunks, uint8_t* __restrict__ out) {
    const int64_t threads = (int64_t)gridDim.x * blockDim.x;
    for (int64_t c = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; c < chunks; c += threads) {
        const int lane = (int)(c & 63);
        const int b = (int)((c >> 6) & 7);
        const int64_t unit = c >> 9;  // t * S8 + sb
        const int64_t sb = unit % s8;
        const int64_t row = (unit / s8) * 16 + (lane & 15);
        const int64_t kb0 = 1024 * sb + 128 * b;
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (row < n && kb0 < k) {
            const uint8_t* src = codes + row * stride;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int64_t k0 = kb0 + 64 * (u >> 1) + 16 * (lane >> 4) + 8 * (u & 1);
                const uint8_t* p = src + k0 / 2;
                const uint32_t d = (uint32_t)p[0] | ((uint32_t)p[1] << 8) | ((uint32_t)p[2] << 16) | ((uint32_t)p[3] << 24);
                uint32_t o = 0;
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    o |= (((d >> (4 * v)) & 15u) | (((d >> (16 + 4 * v)) & 15u) << 4)) << (8 * v);
                w[u] = o ^ 0x88888888u;
            }
        }
        *reinterpret_cast<uint4*>(out + unit * unit_bytes + b * 1024 + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// One (unit, row, eight scales) at a time.
__global__ __launch_bounds__(256) void prepare_w4_scales_kernel(const uint16_t* __restrict__ scales, int64_t stride,
                                                                int64_t n, int64_t count, int s, int s8,
                                                                int unit_bytes, int64_t items,
                                                                uint8_t* __restrict__ out) {
    const int64_t threads = (int64_t)gridDim.x * blockDim.x;
    for (int64_t c = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; c < items; c += threads) {
        const int v = (int)(c % s);
        const int j = (int)((c / s) & 15);
        const int64_t unit = c / (16 * s);
        const int64_t row = (unit / s8) * 16 + j;
        const int64_t first = (unit % s8) * 8 * s + 8 * v;
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = row < n && first + e < count ? scales[row * stride + first + e] : 0u;
        *reinterpret_cast<uint4*>(out + unit * unit_bytes + 8192 + 16 * (s * j + v)) =
            make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
    }
}

}  // namespace

int64_t w4_tiles_bytes(int64_t n, int64_t k, int64_t wgroup) {
    return ((n + 15) / 16) * ((k + 1023) / 1024) * w4_unit((int)(128 / wgroup));
}

hipError_t launch_prepare_w4(const uint8_t* codes, int64_t codes_stride, const uint16_t* scales, int64_t scales_stride,
                             int64_t n, int64_t k, int wgroup, uint8_t* tiles, hipStream_t stream) {
    const int s = 128 / wgroup;
    const int s8 = (int)((k + 1023) / 1024);
    const int64_t units = ((n + 15) / 16) * s8;
    const int64_t chunks = units * 512, items = units * 16 * s;
    // (A launch holds fewer than 2^32 threads.)
    auto blocks = [](int64_t threads) { return dim3((unsigned)std::min<int64_t>((threads + 255) / 256, 1 << 22)); };
    clear_stale_error();
    hipLaunchKernelGGL(prepare_w4_codes_kernel, blocks(chunks), dim3(256), 0, stream, codes,
                       codes_stride, n, k, s8, w4_unit(s), chunks, tiles);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(prepare_w4_scales_kernel, blocks(items), dim3(256), 0, stream, scales,
                       scales_stride, n, k / wgroup, s, s8, w4_unit(s), items, tiles);
    return hipGetLastError();
}

}  // namespace pq2
