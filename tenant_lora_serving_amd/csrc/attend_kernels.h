// attend_kernels.h -- host-side launch interface between the entry points of
// step.h's paged cache (attend_abi.cpp) and their kernels, and the division of
// an attention call among workgroups, which host and device share.  Internal to
// the library.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace st {

// A cache of keys and one of values with the same strides (in elements).
struct CacheArgs {
    void *k, *v;
    int64_t page_stride, token_stride, head_stride;
    int pages, page;               // their number, tokens of one
    const float *k_scale, *v_scale;  // of e4m3, a head each; null: bf16
};

struct AppendArgs {
    const uint16_t *q, *k, *v;  // q: null for none
    int64_t ldq, ldk, ldv;
    int n, heads, kv, dim;
    const int32_t *positions;
    const float *rotation;
    int positions_end, rot, neighbours;
    const int32_t *place;
    CacheArgs cache;
    uint16_t *q_out;
    int64_t ldo;
};
hipError_t launch_kv_append(const AppendArgs &a, hipStream_t st);

// ---------------------------------------------------------------- division of the work
// The rows of a request times the query heads that share a key head are cut
// into tiles of `tokens` rows by `each` heads.  A tile costs `fixed` and the keys
// that its last row sees.  All tiles' costs one after another, request by
// request, key head by key head, are cut into equal ranges, one for every
// workgroup.  A tile that costs more than one of `whole` keys, and more than a
// quarter of a range, is cut where the ranges meet, and its pieces' results go to
// the workspace and are joined; a smaller one belongs to the workgroup that its
// middle falls to.
// Everything follows from the lengths, so the device divides by itself and a
// captured call follows lengths that change.
struct Span {
    int rows, len;
};
__host__ __device__ inline int tiles_of(int rows, int tokens) { return (rows + tokens - 1) / tokens; }
// Keys that tile i of a request sees.
__host__ __device__ inline int tile_keys(Span s, int tokens, bool causal, int i) {
    if (!causal || i == tiles_of(s.rows, tokens) - 1) return s.len;
    const int64_t e = (int64_t)s.len - s.rows + (int64_t)(i + 1) * tokens;
    return e > 0 ? (int)e : 0;
}
// Cost of the first m tiles of a request and one key head.
__host__ __device__ inline int64_t tiles_cost(Span s, int tokens, bool causal, int fixed, int m) {
    if (!causal) return (int64_t)m * (fixed + s.len);
    const bool all = m > 0 && m == tiles_of(s.rows, tokens);
    const int64_t full = all ? m - 1 : m, a = (int64_t)s.len - s.rows;
    int64_t none = a >= 0 ? 0 : -a / tokens;  // tiles that see nothing
    if (none > full) none = full;
    const int64_t count = full - none;
    return (int64_t)m * fixed + count * a + tokens * (count * (none + 1 + full) / 2) + (all ? s.len : 0);
}
// The tile that holds cost offset `at` < tiles_cost(all).
__host__ __device__ inline int tile_at(Span s, int tokens, bool causal, int fixed, int64_t at) {
    int lo = 0, hi = tiles_of(s.rows, tokens) - 1;
    if (!causal) {
        const int64_t i = at / (fixed + s.len);
        return i < hi ? (int)i : hi;
    }
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (tiles_cost(s, tokens, causal, fixed, mid) <= at)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}
// A workgroup's range, and which part of a tile belongs to it.
struct Ranges {
    int64_t size, whole;
    int fixed;
};
__host__ __device__ inline Ranges ranges_of(int64_t total, int groups, int fixed, int least, int whole) {
    int64_t size = (total + groups - 1) / groups;
    if (size < least) size = least;
    return {size, size / 4 > fixed + whole ? size / 4 : fixed + whole, fixed};
}
struct Piece {
    bool mine, split, begins;  // (begins: with the tile's first key)
    int lo, hi;        // keys
    int first, count;  // of a split tile: the first workgroup with a piece, and how many have one
    int slot;          // of its results
};
// The part of the tile at cost `at` with `keys` keys that workgroup w computes;
// pieces begin at multiples of `step` keys.
__host__ __device__ inline Piece piece_of(const Ranges &r, int w, int64_t at, int keys, int step) {
    const int64_t cost = r.fixed + keys, u0 = w * r.size, u1 = u0 + r.size;
    Piece p{};
    if (cost <= r.whole) {
        const int64_t mid = at + cost / 2;
        p.mine = mid >= u0 && mid < u1;
        p.hi = keys;
        p.begins = true;
        return p;
    }
    p.mine = at < u1 && at + cost > u0;
    if (!p.mine) return p;
    p.begins = at >= u0;
    const int64_t lo = u0 > at ? u0 - at - r.fixed : 0, hi = u1 - at - r.fixed;
    p.lo = lo > 0 ? (int)(lo / step * step) : 0;
    p.hi = u1 >= at + cost ? keys : hi > 0 ? (int)(hi / step * step) : 0;
    p.first = (int)(at / r.size);
    p.count = (int)((at + cost - 1) / r.size) - p.first + 1;
    p.split = p.count > 1;
    p.slot = 2 * w + (at > u0 ? 1 : 0);  // (a range's first tile and its last one)
    return p;
}
// Where workgroup w of a split tile that begins at cost `at` left its results.
__host__ __device__ inline int piece_slot(const Ranges &r, int w, int64_t at) { return 2 * w + (at > w * r.size ? 1 : 0); }

// ---------------------------------------------------------------- attention
constexpr int kFewRows = 16, kManyRows = 128;  // rows of a tile: of few rows, of many
constexpr int kMaxEach = 64;                   // query heads of a key head
constexpr int kMaxDim = 256;
constexpr int kFewGroups = 768, kManyGroups = 512;  // workgroups at most
// The constants of the division, each with what other values measured.  (256
// decode: that many tokens over 64 to 4096 keys, 8 key heads of 128 where no other
// size is named; us a call.)
// What a tile costs beside its keys, in keys, some 6 us of a workgroup's time.
// Few: 256 decode 175, with 64 for it 192, with 320 181; 4 heads of 256 192, 213
// and 180.  Few of 8 bits: 99, with 128 120, with 512 105; heads of 64 94, 100 and
// 96; of 256 139, 151 and 151.  Many: prompts of 6947 rows 130, with 64 165, with
// 512 134; from 8 bits 148, 190 and 154.
constexpr int kFewFixed = 128, kFewFixed8 = 320, kManyFixed = 256;
// The least range of a workgroup.  Few: one token over 4999 keys 18.7, with 128
// 22.1, with 512 23.0.  Many: 128 and 512 within 1.5%.
constexpr int kFewLeast = 256, kManyLeast = 256;
// A tile of no more keys is not cut.  Few: 64 requests behind a shared prefix 73,
// with 64 76, with 768 73; 256 decode within 1%.  Many: 256 requests behind 8 prefixes
// 96, with 2048 116; queries to 300 to 1500 keys of another sequence 34, with 256
// 35.5, with 2048 37.
constexpr int kFewWhole = 192, kManyWhole = 768;
constexpr int kFewStep = 128, kManyStep = 64;        // keys of a round
constexpr int kJoinGroups = 512;                     // workgroups that join pieces of many rows
// A workspace begins with a ticket for every workgroup, 0 between calls, and 16
// bytes of zeros.
constexpr size_t kTicketBytes = 4096, kZerosAt = kTicketBytes - 16;
static_assert(kFewGroups * sizeof(int32_t) <= kZerosAt && kManyGroups <= kFewGroups, "a ticket a workgroup");

// key / page for keys below 2^24: (key * mul) >> shift.
struct PageDiv {
    uint32_t mul;
    int shift;
};
__host__ __device__ inline PageDiv page_div(int page) {
    int up = 0;
    while (1ll << up < page) ++up;  // (64 bits: a page may hold more than 2^30)
    return {(uint32_t)((1ull << (24 + up)) / page + 1), 24 + up};
}
__host__ __device__ inline int page_of(PageDiv d, int key) { return (int)(((uint64_t)(uint32_t)key * d.mul) >> d.shift); }

// A split tile of many rows: how many pieces, where the first one's results
// are (those of the next workgroups' in their first slots), its rows and key head.
struct Join {
    int pieces, slot, row, rows, g, unused[3];
};
struct AttendArgs {
    const uint16_t *q;
    int64_t ldq;
    int n, kv, each, dim;
    float scale;  // times log2 e
    CacheArgs cache;
    uint32_t page_units, token_units;  // strides in 16 bytes
    PageDiv div;
    const char *zeros;  // 16 bytes
    // The jobs: request j has rows starts[j] .. starts[j + 1] (row j alone
    // without starts) and lens[j] keys on the pages of row j of the table.
    // With groups, job j is the rows of the requests groups[j - 1] ..
    // groups[j] with prefix j - 1, job 0 the requests before the first group
    // and the last job those behind the last one, both without keys.
    int requests, jobs;
    const int32_t *starts, *groups, *lens, *table;
    int64_t ld_table;
    int table_cols;
    int causal;
    // What the rows bring (from their prefixes) and leave: [n][heads] pairs
    // (maximum, sum) and [n][heads][padded dim] sums of values, or null.
    const float *state_in, *sums_in;
    float *state_out, *sums_out;
    uint16_t *out;
    int64_t ldo;
    float *lse;
    // the pieces of split tiles
    int32_t *tickets;  // few rows: whoever takes the last ticket joins them
    Join *joins;       // many rows: a launch of its own does
    float *pieces;
    int groups_of_threads;
};
hipError_t launch_attend_few(const AttendArgs &a, hipStream_t st);
hipError_t launch_attend_many(const AttendArgs &a, hipStream_t st);

__host__ __device__ inline int padded_dim(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }
inline size_t piece_floats(int rows, int dim) { return (size_t)rows * (padded_dim(dim) + 2); }

}  // namespace st
