// step_kernels.h -- host-side launch interface between step.h's entry points
// (step_abi.cpp) and their kernels.  Internal to the library.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace st {

constexpr int kMaxSlices = 8;
constexpr int kMaxRank = 128;
constexpr int kMaxSlots = 8192;
constexpr int kMaxTop = 32;

struct NormArgs {
    const uint16_t *x;
    int64_t ldx;
    const uint16_t *residual;
    int64_t ldr;
    const uint16_t *weight;
    int n, h;
    float eps;
    uint16_t *residual_out;
    uint16_t *y;
    uint8_t *q;
    float *q_scale;
};
hipError_t launch_rms_norm(const NormArgs &a, hipStream_t st);

// A row of logits is cut into `parts` pieces, one workgroup each; the last
// workgroup of a row to finish joins them.
constexpr int kScoreThreads = 512;
constexpr int kScoreShortThreads = 128;  // for many short rows, one piece each
constexpr int kScoreLaneElems = 64;  // logits per thread of a piece at most
constexpr int kScoreMaxParts = 64;
// The tickets (a word a row, 0 between calls) have a place of their own, the
// same for every shape, so that no call's records are another's tickets.
constexpr int kScoreMaxRows = 1 << 16;
constexpr size_t kScoreTicketBytes = (size_t)kScoreMaxRows * sizeof(int32_t);
// What a piece leaves in the workspace, in 32-bit words: maximum, two sums, a
// count, then `top` 64-bit keys as (high, low).
__host__ __device__ inline int score_record_words(int top) { return 4 + 2 * top; }
struct ScorePlan {
    int threads;          // of a workgroup
    int parts, part_ids;  // pieces of a row, 16-byte vectors of a piece
    size_t ticket_bytes, total_bytes;
};
ScorePlan score_plan(int n, int v, int top, int fp32);
// Enough for every plan of at most n rows, v logits a row and `top`
// alternatives, of both types.
size_t score_workspace_bytes(int n, int v, int top);
struct ScoreArgs {
    const void *logits;
    int64_t ld;
    int fp32, n, v;
    const int32_t *tokens;
    int top;
    float *logprob;
    int32_t *rank;
    float *entropy;
    int32_t *top_ids;
    float *top_logprobs;
};
hipError_t launch_token_logprobs(const ScoreArgs &a, const ScorePlan &plan, void *ws, hipStream_t st);

// Longest k at which 8-bit rows are multiplied as bf16 (step_linear.h); never in large tiles.
constexpr int kExactK = 256;

struct LinearArgs {
    const uint16_t *x;
    int64_t ldx;
    int n, k;
    const uint8_t *xq;
    int64_t ldxq;
    const float *x_scale;
    const void *w;
    const float *w_scale;
    const uint16_t *a_pool;
    const uint16_t *b_pool;
    const float *scale;
    int num_slots, num_slices, R;
    int slice_off[kMaxSlices + 1];
    const int32_t *slot;
    uint16_t *y;
    int64_t ldy;
};
// Up to kUnsortedRows rows are taken as they come (unless the product is
// large), more are sorted by slot first.  The workspace holds the sorted rows' numbers and their slots
// (row_words words each), then the inner sums.
constexpr int kUnsortedRows = 256;
struct LinearPlan {
    bool sorted;
    size_t row_words, total_bytes;
};
LinearPlan linear_plan(int n, int out, int num_slices, int R);
// Rows x columns of the tiles that the product is computed in; the last two
// need sorted rows.
enum Tile { k16x16, k16x64, k32x16, k32x48, k48x64, k64x32, k64x64, k64x96, k128x128, k256x256 };
Tile linear_tile(int n, int k, int out, bool fp8, bool sorted);
struct LinearSpace {
    int32_t *perm, *key_of;
    uint16_t *xab;
};
inline LinearSpace linear_space(const LinearPlan &plan, void *ws) {
    int32_t *perm = static_cast<int32_t *>(ws), *key_of = perm + plan.row_words;
    return {perm, key_of, reinterpret_cast<uint16_t *>(key_of + plan.row_words)};
}
hipError_t launch_lora_linear(const LinearArgs &a, const LinearPlan &plan, void *ws, hipStream_t st);
void launch_sort_rows(const LinearArgs &a, const LinearSpace &s, hipStream_t st);
void launch_sorted_inner(const LinearArgs &a, const LinearSpace &s, hipStream_t st);
void launch_lora_linear_tiled(const LinearArgs &a, const int32_t *perm, const int32_t *key_of, const uint16_t *xab,
                              hipStream_t st);

}  // namespace st
