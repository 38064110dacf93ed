// step_plan.cpp -- host-side sizing of step.h's calls: how a row of logits, a
// projection and its inner sums are cut, and what their workspaces hold.
#include "step_kernels.h"

namespace st {

namespace {

size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }
long long cdiv(long long a, long long b) { return (a + b - 1) / b; }

// A row of logits as 16-byte vectors: whole ones and the two ragged ends.
long long score_ids(int v, int fp32) { return v / (fp32 ? 4 : 8) + 2; }
// The fewest pieces of a row: as many as keep a thread within kScoreLaneElems
// logits; and the most: as many as leave each thread one vector.
long long score_least(long long ids, int fp32) {
    return cdiv(ids, (long long)kScoreThreads * (kScoreLaneElems / (fp32 ? 4 : 8)));
}
long long score_most(long long ids) {
    const long long m = cdiv(ids, kScoreThreads);
    return m < kScoreMaxParts ? m : kScoreMaxParts;
}
// Pieces of all rows together that few rows are cut into, about two per CU.
constexpr int kScorePieces = 512;

}  // namespace

// The fewest pieces for many rows; for few rows more, until the pieces number
// about two per CU, but not so many that a thread has less than one vector.
ScorePlan score_plan(int n, int v, int top, int fp32) {
    const long long ids = score_ids(v, fp32);
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
    const long long least = score_least(ids, fp32), most = score_most(ids);
    long long parts = cdiv(kScorePieces, n > 0 ? n : 1);
    if (parts > most) parts = most;
    if (parts < least) parts = least;
    p.part_ids = (int)cdiv(ids, parts);
    p.parts = (int)cdiv(ids, p.part_ids);
    if (p.parts > 1) {
        p.ticket_bytes = kScoreTicketBytes;
        p.total_bytes = p.ticket_bytes + up256((size_t)n * p.parts * score_record_words(top) * sizeof(uint32_t));
    }
    return p;
}

// Fewer rows are cut into more pieces, so what n rows need does not bound what
// fewer need.  For m <= n rows a plan has at most m * least or, where that
// leaves room for more, m * min(most, cdiv(kScorePieces, m)) pieces, which is
// at most kScorePieces - 1 + m and, past kScorePieces rows, one a row, which
// leaves no record.
size_t score_workspace_bytes(int n, int v, int top) {
    long long pieces = 0;
    for (int fp32 = 0; fp32 < 2; ++fp32) {
        const long long ids = score_ids(v, fp32), least = score_least(ids, fp32), most = score_most(ids);
        const long long few = n < kScorePieces ? n : kScorePieces - 1;
        long long p = least > 1 ? n * least : 0;
        if (most > 1) {
            const long long spread = few * most < kScorePieces - 1 + few ? few * most : kScorePieces - 1 + few;
            if (spread > p) p = spread;
        }
        if (p > pieces) pieces = p;
    }
    return pieces ? kScoreTicketBytes + up256((size_t)pieces * score_record_words(top) * sizeof(uint32_t)) : 0;
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

// Microseconds of a product of `tiles` tiles, one a CU at a time: `fixed` and
// `line` those of a tile and of a line of its k.
static double rounds_us(long long tiles, double fixed, double line, double lines) {
    return 8.0 + (double)cdiv(tiles, 256) * (fixed + line * lines);
}

Tile linear_tile(int n, int k, int out, bool fp8, bool sorted) {
    const int tiles = (out + 15) / 16;
    // wide products from memory: tiles of 48 or 64 columns, of which two fit a CU
    // (12 rows by 4096 x 32008: 60 us, in tiles of 32 columns 70)
    if (n <= 16) return tiles > 768 ? k16x64 : k16x16;
    if (n <= 32) return tiles > 768 ? k32x48 : k32x16;
    // (37 rows by 4096 x 32008: 71.2 us, in 48 x 32 tiles 79.0, in 64 x 96 tiles 72.4)
    if (n <= 48) return k48x64;
    // the times below were fitted to single products (k 1008 to 4096)
    const double lines = (double)cdiv((long long)k * (fp8 ? 1 : 2), 128);  // of 128 bytes
    auto small = [&](int nt) {
        return rounds_us(cdiv(tiles, nt) * cdiv(n, 64), 4.0, 0.11 * (4 + nt), (double)cdiv((long long)lines, 4));  // four waves share the lines
    };
    const double s2 = small(2), s4 = small(4), s6 = small(6), best = s2 < s4 ? (s2 < s6 ? s2 : s6) : (s4 < s6 ? s4 : s6);
    if (sorted && !(fp8 && k <= kExactK)) {
        const double mid = rounds_us(cdiv(out, 128) * cdiv(n, 128), 4.0, 0.58, lines);
        const double large = rounds_us(cdiv(out, 256) * cdiv(n, 256), 8.0, fp8 ? 1.8 : 1.6, lines);
        if (large <= mid && large <= best) return k256x256;
        if (mid <= best) return k128x128;
    }
    if (s6 <= best) return k64x96;
    return s4 <= best ? k64x64 : k64x32;
}

}  // namespace st
