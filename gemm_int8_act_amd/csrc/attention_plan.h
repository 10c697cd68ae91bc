// attention_plan.h -- how a paged attention call is divided: plain arithmetic,
// which the host decides by and any C++ compiler takes.
#pragma once

#include <stdint.h>

#include <algorithm>

#ifdef __HIPCC__
#define PQ2_BOTH_SIDES __host__ __device__
#else
#define PQ2_BOTH_SIDES
#endif

namespace pq2 {

constexpr int kPagedThreads = 256;         // threads of a workgroup
constexpr int kPagedRows = 16;             // query rows of a tile
constexpr int kMaxSplits = 128;
constexpr int kFan = 8;                    // parts that are joined first, of more than are joined at once
constexpr int kTileCounters = 1 + kMaxSplits / kFan;

// Sizes of one paged call that its workspace follows from: `splits` parts of
// a row's cache at most, row tiles of `rows` query rows (new tokens x grouped
// heads) each, `row_tiles` of them a sequence and key-value head.
struct PagedPlan {
    int64_t splits, row_tiles, rows, min_chunk;
    int64_t partial_floats, counter_words;
};

inline int log2_of(int64_t v) {
    int s = 0;
    while (((int64_t)1 << s) < v) ++s;
    return s;
}

inline PagedPlan paged_plan(int64_t seqs, int64_t max_new, int64_t heads, int64_t kv_heads, int64_t head_dim,
                            int64_t max_len) {
    PagedPlan p;
    const int64_t rows = max_new * (heads / kv_heads);
    const int64_t most = rows > kPagedRows && head_dim != 256 ? 2 * kPagedRows : kPagedRows;
    p.rows = std::min<int64_t>(rows, most);
    p.row_tiles = (rows + most - 1) / most;
    // Parts: as many as fill the chip (512 workgroups, 1024 of heads of 64), or
    // of 2048 keys where a long sequence may stand among short ones. Measured:
    // heads of 128 with 512 / 768 workgroups, 16 sequences of 4096 keys 29 / 34 us, with 8 new tokens 62 / 74, one of
    // 8192 11.8 / 12.3, four of 4096 14.5 / 13.5;
    // 128 instead of 64 parts of 131072 keys of one sequence 70 us against 61; parts of 1024 keys
    // (64 sequences of 1 to 16384) 89 against 78.
    const int64_t base = seqs * kv_heads * p.row_tiles, fill = head_dim == 64 ? 1024 : 512;
    p.splits = std::max(fill / base, (max_len + 2047) / 2048);
    p.splits = std::max<int64_t>(1, std::min({p.splits, (max_len + 255) / 256, (int64_t)kMaxSplits}));
    p.splits = (int64_t)1 << log2_of(p.splits);
    // (2^23 workgroups, below 2^24 of them with paged_workgroups' padding: a
    // launch holds fewer than 2^32 threads along x.)
    while (p.splits > 1 && kv_heads * p.row_tiles * p.splits * std::min<int64_t>(seqs, 64) > 1 << 23) p.splits >>= 1;
    p.min_chunk = base >= fill ? 2048 : base >= fill / 4 ? 1024 : base >= fill / 16 ? 512 : 256;
    p.partial_floats = p.splits > 1 ? base * p.splits * p.rows * (head_dim + 2) : 0;
    p.counter_words = p.splits > 1 ? base * kTileCounters : 0;
    return p;
}

// Places of a launch, (part, key-value head) of up to 64 sequences; each takes
// row_tiles workgroups.
inline int64_t paged_places(const PagedPlan& p, int64_t seqs, int64_t kv_heads) {
    return kv_heads * p.splits * std::min<int64_t>(seqs, 64);
}

// Workgroups along x.  Eight places and more are rounded up to a multiple of
// eight, so that a place's row tiles follow each other on one XCD; fewer would
// leave XCDs without work, and are not (512 new tokens of 64 heads on one, 512 keys,
// heads of 128: 28 us; rounded up 166).
inline int64_t paged_workgroups(const PagedPlan& p, int64_t seqs, int64_t kv_heads) {
    const int64_t places = paged_places(p, seqs, kv_heads);
    return (places < 8 ? places : (places + 7) / 8 * 8) * p.row_tiles;
}

// Parts of `chunk` keys that `most` keys are, at least one; `about` is
// (most - 1) / chunk, off by one at most.  Unsigned: most and chunk go up to
// 2^30, the products up to 3 * 2^30.
PQ2_BOTH_SIDES inline int parts_of(int most, int chunk, int about) {
    const uint32_t all = (uint32_t)(most > 1 ? most : 1), next = (uint32_t)(about + 1) * (uint32_t)chunk;
    if (next < all) return about + 2;
    return about > 0 && next - (uint32_t)chunk >= all ? about : about + 1;
}

}  // namespace pq2
