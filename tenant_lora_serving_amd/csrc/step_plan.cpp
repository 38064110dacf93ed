// step_plan.cpp -- host-side sizing of step.h's calls: how a row of logits and
// the inner sums of a projection are cut, and what their workspaces hold.
#include "step_kernels.h"

namespace st {

namespace {

size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }
long long cdiv(long long a, long long b) { return (a + b - 1) / b; }

}  // namespace

// At least as many pieces as keep a thread within kScoreLaneElems logits; for
// few rows more, until the pieces number about two per CU, but not so many
// that a thread has less than one 16-byte vector.
ScorePlan score_plan(int n, int v, int top, int fp32) {
    const int E = fp32 ? 4 : 8;
    const long long ids = v / E + 2;  // whole vectors and the two ragged ends
    ScorePlan p{};
    // enough rows to fill the chip, and each within eight vectors of 128
    // threads: 2000 rows of 1417 floats, top 1: 10 us; with 512
    // threads a row, most of them idle in every selection, 22 us
    if (n >= 256 && ids <= 8 * kScoreShortThreads) {
        p.threads = kScoreShortThreads;
        p.parts = 1;
        p.part_ids = (int)ids;
        return p;
    }
    p.threads = kScoreThreads;
    const long long least = cdiv(ids, (long long)kScoreThreads * (kScoreLaneElems / E));
    long long parts = cdiv(512, n > 0 ? n : 1);
    if (parts > cdiv(ids, kScoreThreads)) parts = cdiv(ids, kScoreThreads);
    if (parts > kScoreMaxParts) parts = kScoreMaxParts;
    if (parts < least) parts = least;
    p.part_ids = (int)cdiv(ids, parts);
    p.parts = (int)cdiv(ids, p.part_ids);
    if (p.parts > 1) {
        p.ticket_bytes = (size_t)kScoreMaxRows * sizeof(int32_t);
        p.total_bytes = p.ticket_bytes + up256((size_t)n * p.parts * score_record_words(top) * sizeof(uint32_t));
    }
    return p;
}

// Sorting costs a launch and some 5 us, and is needed for tiles larger than
// 64 x 96: worth it past two rounds of those (a step with 256 rows by 4096 x 128256 took
// 780 us without, 600 with).
LinearPlan linear_plan(int n, int out, int num_slices, int R) {
    LinearPlan p{};
    p.sorted = n > kUnsortedRows || (n > 64 && cdiv(n, 64) * cdiv(out, 96) > 512);
    const size_t inner = (size_t)n * num_slices * R * 2 * sizeof(uint16_t);
    if (p.sorted) p.row_words = up256((size_t)n * sizeof(int32_t)) / sizeof(int32_t);
    p.total_bytes = 2 * p.row_words * sizeof(int32_t) + up256(inner);
    return p;
}

}  // namespace st
