// attention_internal.h -- host-side launchers of the attention operators
// (declared in include/pq2_attention.h), and the pieces their kernels share.
// Arguments reaching the launchers are already validated by the C ABI layer.
#pragma once

#include "../../include/pq2_attention.h"
#include "attention_plan.h"
#include "block_internal.h"

namespace pq2 {

hipError_t launch_kv_write(const pq2_kv_write_args& a, hipStream_t stream);
hipError_t launch_kv_read(const pq2_kv_read_args& a, hipStream_t stream);
hipError_t launch_attention_paged(const pq2_attention_paged_args& a, const PagedPlan& plan, hipStream_t stream);
hipError_t launch_attention_prompt(const pq2_attention_prompt_args& a, hipStream_t stream);

// Bytes of one key-value head's block of a page.
__host__ __device__ constexpr int64_t kv_block_bytes(int64_t page_tokens, int64_t head_dim) {
    return page_tokens * (2 * head_dim + 8);
}

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

// Lanes of a wave whose `starts` entry is at most `row`, 64 sequences a step:
// the sequence that holds `row`, 0 <= row < starts[seqs]; the last one for a
// row behind them.  All lanes of the wave take part with the same row.
__device__ __forceinline__ int sequence_of(const int32_t* starts, int seqs, int row) {
    const int lane = threadIdx.x & 63;
    int lo = 0, count = seqs;
    while (true) {
        const int step = (count + 63) >> 6;
        const int at = lane * step;
        const bool below = at < count && starts[lo + at] <= row;
        const int n = __popcll(__ballot(below));
        lo += max(n - 1, 0) * step;
        if (step == 1) return lo;
        count = min(step, seqs - lo);
    }
}

}  // namespace pq2
