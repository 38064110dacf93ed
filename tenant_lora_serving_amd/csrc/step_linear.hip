// step_linear.hip -- step_lora_linear: the shared projection with every row's
// adapter added,
//
//     y[i] = x[i] W^T + scale[s] (x[i] A_s^T) B_s^T,   s = slot[i],
//
// in small tiles, for few rows or a small product.
//
// Two launches (and, past kUnsortedRows rows, the sort of the rows by slot
// before them).  The first computes the inner sums xa[i] = scale[s] x[i] A_s^T
// of each slot's rows.  The second computes tiles of x W^T and, before it
// rounds, adds xa B_s^T for each slot that a tile's rows name, as matrix
// products in which only that slot's rows are not zero.  (As one launch, with
// a counter between the two, q, k and v of one row took 14.9 instead of 17.9
// us, but those of 256 rows 55 instead of 45: the waiting workgroups' reads of
// the counter come one after another.)
//
// The product is bound by reading: W from memory, x from L2 by every
// workgroup.  The waves of a workgroup share one tile and take every
// kWaves-th line of k through rings of their own, so nothing that a wave
// loads is another's too and there is no barrier in the loop.  The waves'
// sums meet in shared memory once, at the end.  One row by 4096 x 6144: 10 us of
// 17, 5 TB/s; 256 rows: 27 of 35 us.
#include "step_linear.h"

namespace st {

namespace {

// ---------------------------------------------------------------- inner sums
constexpr int kInWaves = 8, kInThreads = kInWaves * kWave;

// The t-th group of up to 16 rows of one slot, numbered by the row that it
// starts with; count 0 past the last group.  Lane m < count holds row m's
// number.  Every wave finds it by itself: the lanes with a row's slot follow
// from one ballot a bit of the slot's number, so the time grows with
// log(slots).  (Slot after slot took 12 us of the kernel for 256 rows over 32
// slots and 46 over 128, ranks through LDS some 4 for their barriers.)
struct Group {
    int slot, count, row;
};
// kChunks: of 64 rows, all rows.
template <int kChunks>
__device__ __forceinline__ Group find_group(const LinearArgs &a, int t) {
    const int lane = tl::lane_id(), chunks = (a.n + kWave - 1) / kWave;
    const int bits = a.num_slots > 1 ? 32 - __builtin_clz(a.num_slots - 1) : 0;
    int s[kChunks];
    uint64_t same[kChunks][kChunks];  // [c][d]: the rows of chunk d with the slot of the lane's row in chunk c
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        s[c] = c * kWave + lane < a.n ? a.slot[c * kWave + lane] : -1;
        if (s[c] >= a.num_slots) s[c] = -1;
    }
#pragma unroll
    for (int d = 0; d < kChunks; ++d) {
        const uint64_t valid = __ballot(s[d] >= 0);
#pragma unroll
        for (int c = d; c < kChunks; ++c) same[c][d] = valid;
    }
#pragma unroll 1
    for (int b = 0; b < bits; ++b) {
#pragma unroll
        for (int d = 0; d < kChunks; ++d) {
            if (d > 0 && d >= chunks) break;
            const uint64_t set = __ballot(s[d] >> b & 1);
#pragma unroll
            for (int c = d; c < kChunks; ++c) same[c][d] &= s[c] >> b & 1 ? set : ~set;
        }
    }
    // ranks among the slot's rows; every 16th leads a group
    int rank[kChunks], before = 0, slot = -1, first = 0;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        rank[c] = __popcll(same[c][c] & tl::lanemask_lt());
#pragma unroll
        for (int d = 0; d < c; ++d) rank[c] += __popcll(same[c][d]);
        const uint64_t leads = __ballot(s[c] >= 0 && rank[c] % 16 == 0);
        const uint64_t it = __ballot((leads >> lane & 1) && before + __popcll(leads & tl::lanemask_lt()) == t);
        if (it) {
            slot = __builtin_amdgcn_readlane(s[c], __builtin_ctzll(it));
            first = __builtin_amdgcn_readlane(rank[c], __builtin_ctzll(it));
        }
        before += __popcll(leads);
    }
    if (slot < 0) return {-1, 0, 0};
    // each of the group's lanes hands its row's number + 1 to the lane of its
    // place in the group, the others a 0 to the last lane
    int row = 0, count = 0;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int i = rank[c] - first;
        const bool mine = s[c] == slot && i >= 0 && i < 16;
        row = max(row, __builtin_amdgcn_ds_permute((mine ? i : kWave - 1) * 4, mine ? c * kWave + lane + 1 : 0));
        count += __popcll(__ballot(mine));
    }
    return {slot, count, row - 1};
}

// A group of rows by 16 NT of the num_slices * R rows of A_s.  Eight waves
// split k, so that each has only a few lines to wait for.
template <int NT, int SLOTS, int CHUNKS>
__global__ __launch_bounds__(kInThreads) void inner_kernel(LinearArgs a, uint16_t *xab) {
    using Part = Partials<NT, 1>;
    using Ring = LineRing<NT, 1, SLOTS>;
    constexpr int kShared = Ring::kBytes > Part::kFloats * 4 ? Ring::kBytes : Part::kFloats * 4;
    __shared__ __align__(16) char shared[kInWaves * kShared];
    float *red = reinterpret_cast<float *>(shared);
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tl::wave_id());
    const int LR = a.num_slices * a.R, kbytes = a.k * 2, lines = (kbytes + kLine - 1) / kLine;
    const int c0 = blockIdx.y * Part::kCols;
    const Group group = find_group<CHUNKS>(a, blockIdx.x);
    const int slot = __builtin_amdgcn_readfirstlane(group.slot), count = __builtin_amdgcn_readfirstlane(group.count);
    const int row = group.row;
    if (count == 0) return;

    const uint16_t *A = a.a_pool + ((int64_t)slot * LR + c0) * a.k;
    const i32x4_t wr = words_rsrc(A, (uint32_t)(min(LR - c0, Part::kCols) * kbytes));
    const i32x4_t xr = words_rsrc(a.x, (uint32_t)(((int64_t)(a.n - 1) * a.ldx + a.k) * 2));
    const float scale = a.scale[slot];
    uint32_t wo[Ring::kW], xo[Ring::kX];
#pragma unroll
    for (int u = 0; u < Ring::kW; ++u) wo[u] = c0 + Ring::row(u) < LR ? (uint32_t)(Ring::row(u) * kbytes) : kOob;
#pragma unroll
    for (int u = 0; u < Ring::kX; ++u) {
        const int m = Ring::row(u), r = __shfl(row, m);
        xo[u] = m < count ? (uint32_t)((int64_t)r * a.ldx * 2) : kOob;
    }
    f32x4_t acc[NT][1] = {};
    ring_product<kBf16, NT, 1, SLOTS>(wr, wo, xr, xo, shared + wave * Ring::kBytes, wave, kInWaves, lines, kbytes, acc);
    __syncthreads();  // (the partial sums lie over the rings)
    Part::put(red, wave, acc);
    __syncthreads();
    constexpr int kVecs = Part::kCols / 8;
    const int m = tid / kVecs % 16, c = tid % kVecs * 8, r = __shfl(row, m);
    if (tid < 16 * kVecs && m < count && c0 + c < LR) {
        float v[8];
        Part::template sum8<kInWaves>(red, m, c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= scale;
        put_inner8(xab, r, c0 + c, a.num_slices, a.R, v);
    }
}

// ---------------------------------------------------------------- the product
constexpr int kWaves = 4, kThreads = kWaves * kWave;
struct Inner {
    const int32_t *perm, *key_of;  // sorted rows: their row numbers and slots
    const uint16_t *xab;
};

// The 8-bit form's scales: lane m holds row m's, columns from c0.  (One after
// the other, as in the large tiles: the product of two small scales may be no
// fp32 number where the result is one.)
template <int MT, int NT>
__device__ __forceinline__ void apply_scales(const LinearArgs &a, float my_scale, int c0, int cols,
                                             f32x4_t (&acc)[NT][MT]) {
    const int lane = tl::lane_id();
    float ws[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int c = 16 * j + 4 * (lane / 16) + e;
            ws[j][e] = c < cols ? a.w_scale[c0 + c] : 0.0f;
        }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const float xs = __shfl(my_scale, 16 * i + lane % 16);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][i][e] = acc[j][i][e] * xs * ws[j][e];
    }
}

// Adds xab B_s^T for the slots of the rows in `mine` to a wave's tile of rows
// from m0 (lane m holds row m's slot) and columns c0 .. c0 + cols: slice by
// slice, in steps of 32 of the 2 R terms of one slot (R rounded inner sums and
// R rests, against the same B twice), kSteps steps on the way.  With one wave a
// SIMD its own instructions bound it: everything that a step does not change
// is worked out before, and rows and columns that are not the step's read zero
// through offsets past their buffers.
// careful: a B is looked through for infinities and NaN, which are taken as
// zero; true if there were any.
constexpr int kSteps = 2;
constexpr uint32_t kFar = 0x40000000u;  // past every buffer here, also with kOob added
template <int MT, int NT>
__device__ __forceinline__ bool add_adapters(const LinearArgs &a, const uint16_t *xab, int out, int my_slot,
                                             uint64_t mine, int m0, int rows, int c0, int cols, bool careful,
                                             f32x4_t (&acc)[NT][MT]) {
    if (!mine) return false;
    bool broken = false;
    const int lane = tl::lane_id(), chunks = a.R / 8, pitch = a.num_slices * 4 * a.R;
    int first_slice = 0, end_slice = a.num_slices;
    while (a.slice_off[first_slice + 1] <= c0) ++first_slice;
    while (end_slice > first_slice + 1 && a.slice_off[end_slice - 1] >= c0 + cols) --end_slice;
    const rsrc_t xr = tl::make_rsrc(xab + (int64_t)m0 * a.num_slices * 2 * a.R, (uint32_t)(rows * pitch));
    int row_slot[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) row_slot[i] = __shfl(my_slot, 16 * i + lane % 16);
    const uint32_t x0 = (uint32_t)(lane % 16 * pitch);
#pragma unroll 1
    for (int slice = first_slice; slice < end_slice; ++slice) {
        const int lo = a.slice_off[slice] - c0, hi = min(a.slice_off[slice + 1] - c0, cols);
        uint32_t b0[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int c = 16 * j + lane % 16;
            b0[j] = c >= lo && c < hi ? (uint32_t)(c * a.R * 2) : kFar;
        }
        uint64_t todo = mine, same = 0;
        int slot = -1, q0 = 0;
        auto next_slot = [&]() {
            q0 = 0;
            slot = todo ? __builtin_amdgcn_readlane(my_slot, __builtin_ctzll(todo)) : -1;
            same = slot >= 0 ? __ballot(my_slot == slot) : 0;
            todo &= ~same;
        };
        u32x4_t bf[kSteps][NT], xf[kSteps][MT];
        uint64_t who[kSteps];
        auto load_steps = [&]() {
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                who[s] = same;
                if (slot < 0) continue;
                const int q = q0 + lane / 16;
                const bool in = q < 2 * chunks;
                const uint32_t bq = in ? (uint32_t)(q >= chunks ? q - chunks : q) * 16 : kOob;
                const uint32_t xq = in ? (uint32_t)(slice * 4 * a.R + q * 16) : kOob;
                const rsrc_t br = tl::make_rsrc(a.b_pool + ((int64_t)slot * out + c0) * a.R, (uint32_t)(cols * a.R * 2));
#pragma unroll
                for (int j = 0; j < NT; ++j) bf[s][j] = tl::buf_ld16(br, b0[j] + bq);
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    xf[s][i] = tl::buf_ld16(xr, row_slot[i] == slot ? x0 + xq + (uint32_t)(16 * i * pitch) : kOob);
                if ((q0 += 4) >= 2 * chunks) next_slot();
            }
        };
        next_slot();
        load_steps();
#pragma unroll 1
        while (who[0]) {
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                if (!who[s]) continue;
                if (careful) {
                    u16x2_t big = {};
#pragma unroll
                    for (int j = 0; j < NT; ++j) big = larger_magnitude(big, bf[s][j]);
                    if (__ballot(not_finite(big))) {
                        broken = true;
#pragma unroll
                        for (int j = 0; j < NT; ++j) drop_not_finite(bf[s][j]);
                    }
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    if (!(who[s] >> (16 * i) & 0xffff)) continue;
#pragma unroll
                    for (int j = 0; j < NT; ++j) acc[j][i] = tl::mfma_16x16x32(bf[s][j], xf[s][i], acc[j][i]);
                }
            }
            load_steps();
        }
    }
    return broken;
}
// An infinity or NaN among a wave's results.
template <int MT, int NT>
__device__ __forceinline__ bool any_not_finite(const f32x4_t (&acc)[NT][MT]) {
    float t = 0.0f;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) t = fmaf(acc[j][i][e], 0.0f, t);
    return __ballot(t != t) != 0;
}

// SLOTS lines in a wave's ring.
template <Form F, int MT, int NT, int SLOTS, bool SORTED>
__global__ __launch_bounds__(kThreads) void rows_kernel(LinearArgs a, Inner h, int out) {
    using Part = Partials<NT, MT>;
    using Ring = LineRing<NT, MT, SLOTS>;
    constexpr int kShared = Ring::kBytes > Part::kFloats * 4 ? Ring::kBytes : Part::kFloats * 4;
    __shared__ __align__(16) char shared[kWaves * kShared];
    float *red = reinterpret_cast<float *>(shared);  // over the rings, when they are done with
    const int lane = tl::lane_id(), tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tl::wave_id());
    // row tiles of the same columns run next to each other on one XCD
    const int m_tiles = (a.n + Part::kRows - 1) / Part::kRows;
    const int on_xcd = blockIdx.x / 8;
    const int c0 = (on_xcd / m_tiles * 8 + blockIdx.x % 8) * Part::kCols, m0 = on_xcd % m_tiles * Part::kRows;
    if (c0 >= out) return;
    const int rows = min(a.n - m0, Part::kRows), cols = min(out - c0, Part::kCols);
    const int my_row = lane < rows ? (SORTED ? h.perm[m0 + lane] : m0 + lane) : 0;
    int my_slot = lane < rows ? (SORTED ? h.key_of[m0 + lane] : a.slot[m0 + lane]) : -1;
    if (my_slot >= a.num_slots) my_slot = -1;

    constexpr bool FP8 = F != kBf16;
    constexpr int esz = FP8 ? 1 : 2;
    const int kbytes = a.k * esz, lines = (kbytes + kLine - 1) / kLine;
    const int64_t ldx = FP8 ? a.ldxq : a.ldx * 2;
    const i32x4_t xr = words_rsrc(FP8 ? (const void *)a.xq : (const void *)a.x,
                                  (uint32_t)((int64_t)(a.n - 1) * ldx + kbytes));
    const i32x4_t wr = words_rsrc((const char *)a.w + (int64_t)c0 * kbytes, (uint32_t)(cols * kbytes));
    uint32_t wo[Ring::kW], xo[Ring::kX];
#pragma unroll
    for (int u = 0; u < Ring::kW; ++u) wo[u] = Ring::row(u) < cols ? (uint32_t)(Ring::row(u) * kbytes) : kOob;
#pragma unroll
    for (int u = 0; u < Ring::kX; ++u) {
        const int m = Ring::row(u), r = SORTED ? __shfl(my_row, m) : m0 + m;
        xo[u] = m < rows ? (uint32_t)((int64_t)r * ldx) : kOob;
    }
    // A wave takes the adapters whose slot is its number modulo kWaves: so a
    // row's sums meet in the same order whatever other rows share its tile, and
    // the order of the sorted rows changes no result.  Infinities and NaN are
    // looked for in its sums, and only a wave that finds some computes them
    // again with care (looking through every B cost 2 of 43 us).
    const uint64_t mine = __ballot(my_slot >= 0 && my_slot % kWaves == wave);
    // (not where row tiles share x: 139 rows by 11312 x 9656 took 141 us so, 134 in step)
    const int turn = m_tiles == 1 ? c0 / Part::kCols * 7 % lines : 0;
    f32x4_t acc[NT][MT];
    bool careful = false, broken;
#pragma unroll 1
    for (;; careful = true) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[j][i] = f32x4_t{};
        ring_product<F, NT, MT, SLOTS>(wr, wo, xr, xo, shared + wave * Ring::kBytes, wave, kWaves, lines, kbytes, acc, turn);
        if constexpr (FP8) apply_scales(a, lane < rows ? a.x_scale[my_row] : 0.0f, c0, cols, acc);
        broken = add_adapters<MT, NT>(a, h.xab, out, my_slot, mine, m0, rows, c0, cols, careful, acc);
        if (careful || !mine || !any_not_finite(acc)) break;
    }

    static_assert(kWaves * Part::kFloats * 4 <= kWaves * (kShared - 4), "the waves' words follow the partial sums");
    int *broken_of = reinterpret_cast<int *>(shared + kWaves * kShared) - kWaves;
    __syncthreads();
    Part::put(red, wave, acc);
    if (lane == 0) broken_of[wave] = broken;
    __syncthreads();
    for (int t = tid; t < Part::kRows * Part::kCols / 8; t += kThreads) {
        const int m = t / (Part::kCols / 8), c = t % (Part::kCols / 8) * 8;
        if (m >= rows || c >= cols) continue;
        float v[8];
        Part::template sum8<kWaves>(red, m, c, v);
        const int64_t r = SORTED ? h.perm[m0 + m] : m0 + m;
        tl::st16(a.y + r * a.ldy + c0 + c, pack8(v));
    }
    if (broken_of[0] | broken_of[1] | broken_of[2] | broken_of[3])
        mark_broken<kThreads>(a, out, m0, rows, c0, cols, SORTED ? h.perm : nullptr, SORTED ? h.key_of : a.slot);
}

// ---------------------------------------------------------------- middling products
// 128 sorted rows x 128 columns by four waves, 64 x 64 each, for products that
// 256 x 256 tiles would not spread over the chip and 64 x 64 tiles read too
// often.  Lines go through kMidSlots buffers of LDS that the waves share; a
// wave multiplies a line from registers while it reads the next one's
// fragments, two matrix instructions to a read, and the loads of two more
// lines are out.  A line keeps the matrix cores and the LDS busy for 512 and
// 768 cycles and takes some 1300 (1000 rows by 4096 x 6144: 80 us, in 64 x 64
// tiles 100; in 256 x 256 tiles they would be a third of the chip).
constexpr int kMidTile = 128, kMidSlots = 4, kMidLoads = 8, kMidSlot = 2 * kMidTile * kLine;
template <Form F>
__global__ __launch_bounds__(kThreads) void mid_kernel(LinearArgs a, Inner h, int out) {
    __shared__ __align__(16) char lds[kMidSlots * kMidSlot];
    const int lane = tl::lane_id(), wave = __builtin_amdgcn_readfirstlane(tl::wave_id());
    // row tiles of the same columns run next to each other on one XCD
    const int m_tiles = (a.n + kMidTile - 1) / kMidTile, on_xcd = blockIdx.x / 8;
    const int c0 = (on_xcd / m_tiles * 8 + blockIdx.x % 8) * kMidTile, m0 = on_xcd % m_tiles * kMidTile;
    if (c0 >= out) return;
    const int rows = min(a.n - m0, kMidTile), cols = min(out - c0, kMidTile);
    constexpr int esz = F == kBf16 ? 2 : 1;
    const int kbytes = a.k * esz, lines = (kbytes + kLine - 1) / kLine;
    const int64_t ldx = F == kBf16 ? a.ldx * 2 : a.ldxq;

    // Waves 0 and 1 load the rows of x, 2 and 3 those of w, 8 rows an
    // instruction; LDS place c of row r holds chunk c ^ (r % 8).
    const int l8 = lane / 8, chunk = ((lane & 7) ^ l8) * 16, half = wave % 2 * 64;
    const i32x4_t rsrc = wave < 2 ? words_rsrc(F == kBf16 ? (const void *)a.x : (const void *)a.xq,
                                               (uint32_t)((int64_t)(a.n - 1) * ldx + kbytes))
                                  : words_rsrc((const char *)a.w + (int64_t)c0 * kbytes, (uint32_t)(cols * kbytes));
    uint32_t off[kMidLoads];
#pragma unroll
    for (int u = 0; u < kMidLoads; ++u) {
        const int r = half + 8 * u + l8;
        off[u] = wave < 2 ? (r < rows ? (uint32_t)((int64_t)h.perm[m0 + r] * ldx) : kOob)
                          : (r < cols ? (uint32_t)(r * kbytes) : kOob);
    }
    const uint32_t to = lds_address(lds) + wave * (kMidSlot / kWaves);
    auto start = [&](int slot, int line) __attribute__((always_inline)) {
        const int at = line * kLine + chunk;
        const uint32_t o = at < kbytes ? (uint32_t)at : kOob;
#pragma unroll
        for (int u = 0; u < kMidLoads; ++u) load_lds(rsrc, off[u] + o, 0, to + slot * kMidSlot + u * 1024);
    };
    const int wm = wave % 2 * 64, wn = wave / 2 * 64;
    const int rd = (lane % 16) * kLine + (((lane / 16) ^ (lane & 7)) * 16);
    Line x[2][4], w[2][4];
    auto read = [&](int into, int slot) __attribute__((always_inline)) {
        const char *p = lds + slot * kMidSlot;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const char *q = p + (wm + 16 * i) * kLine;
            x[into][i] = Line{tl::ld16(q + rd), tl::ld16(q + (rd ^ 64))};
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const char *q = p + (kMidTile + wn + 16 * j) * kLine;
            w[into][j] = Line{tl::ld16(q + rd), tl::ld16(q + (rd ^ 64))};
        }
    };
    f32x4_t acc[4][4] = {};
#pragma unroll
    for (int d = 0; d < kMidSlots - 1; ++d) start(d, d);
    wait_loads<(kMidSlots - 2) * kMidLoads>();
    barrier();
    read(0, 0);
#pragma unroll 1
    for (int t = 0; t < lines; t += kMidSlots) {
#pragma unroll
        for (int d = 0; d < kMidSlots; ++d) {
            // line t + d + 1 has arrived, and nobody reads line t + d - 1 any more
            wait_loads<(kMidSlots - 3) * kMidLoads>();
            barrier();
            start((d + kMidSlots - 1) % kMidSlots, t + d + kMidSlots - 1);
            read((d + 1) % 2, (d + 1) % kMidSlots);
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][i] = mma_line<F>(w[d % 2][j], x[d % 2][i], acc[j][i]);
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                // a read of LDS,
                __builtin_amdgcn_sched_group_barrier(0x008, F == kBf16 ? 2 : 1, 0);  // then matrix instructions
            }
        }
    }
    wait_loads<0>();  // (lines past the end still write zeros)
    bool broken = false;

    // ---- this wave's 64 x 64
    const int m1 = m0 + wm, c1 = c0 + wn, my_rows = rows - wm, my_cols = min(cols - wn, 64);
    const bool here = lane < my_rows;
    const int my_row = here ? h.perm[m1 + lane] : 0, key = here ? h.key_of[m1 + lane] : a.num_slots;
    const int my_slot = key < a.num_slots ? key : -1;
    if (my_rows > 0 && my_cols > 0) {
        if constexpr (F != kBf16) apply_scales(a, here ? a.x_scale[my_row] : 0.0f, c1, my_cols, acc);
        broken = add_adapters<4, 4>(a, h.xab, out, my_slot, __ballot(my_slot >= 0), m1, my_rows, c1, my_cols, true, acc);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = 16 * i + lane % 16, r = __shfl(my_row, m);
            if (m >= my_rows) continue;
            uint16_t *y = a.y + (int64_t)r * a.ldy + c1;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = 16 * j + 4 * (lane / 16);
                if (c < my_cols)
                    *reinterpret_cast<uint2 *>(y + c) = make_uint2(tl::pack_bf16x2(acc[j][i][0], acc[j][i][1]),
                                                                   tl::pack_bf16x2(acc[j][i][2], acc[j][i][3]));
            }
        }
    }
    int *broken_of = reinterpret_cast<int *>(lds);  // (every wave is past its reads of lines)
    __syncthreads();
    if (lane == 0) broken_of[wave] = broken;
    __syncthreads();
    if (broken_of[0] | broken_of[1] | broken_of[2] | broken_of[3]) mark_broken<kThreads>(a, out, m0, rows, c0, cols, h.perm, h.key_of);
}

template <Form F, int MT, int NT, int SLOTS>
void go(const LinearArgs &a, const Inner &h, int out, hipStream_t st) {
    const int m_tiles = (a.n + 16 * MT - 1) / (16 * MT), c_tiles = (out + 16 * NT - 1) / (16 * NT);
    const dim3 grid((unsigned)((c_tiles + 7) / 8 * 8) * m_tiles);
    if constexpr (MT == 4) {
        if (h.perm) {
            rows_kernel<F, MT, NT, SLOTS, true><<<grid, kThreads, 0, st>>>(a, h, out);
            return;
        }
    }
    rows_kernel<F, MT, NT, SLOTS, false><<<grid, kThreads, 0, st>>>(a, h, out);
}

template <Form F>
void go_mid(const LinearArgs &a, const Inner &h, int out, hipStream_t st) {
    const int m_tiles = (a.n + kMidTile - 1) / kMidTile, c_tiles = (out + kMidTile - 1) / kMidTile;
    mid_kernel<F><<<dim3((unsigned)((c_tiles + 7) / 8 * 8) * m_tiles), kThreads, 0, st>>>(a, h, out);
}

template <Form F>
void multiply(Tile tile, const LinearArgs &a, const Inner &h, int out, hipStream_t st) {
    switch (tile) {
        case k16x16: return go<F, 1, 1, 4>(a, h, out, st);
        case k16x64: return go<F, 1, 4, 2>(a, h, out, st);
        case k32x16: return go<F, 2, 1, 4>(a, h, out, st);
        case k32x48: return go<F, 2, 3, 2>(a, h, out, st);
        case k48x64: return go<F, 3, 4, 2>(a, h, out, st);
        case k64x32: return go<F, 4, 2, 3>(a, h, out, st);
        case k64x64: return go<F, 4, 4, 2>(a, h, out, st);
        case k64x96: return go<F, 4, 6, 2>(a, h, out, st);
        default: break;
    }
    if constexpr (F != kE4m3AsBf16) {
        if (tile == k128x128) go_mid<F>(a, h, out, st);
        else launch_lora_linear_tiled(a, h.perm, h.key_of, h.xab, st);
    }
}

}  // namespace

hipError_t launch_lora_linear(const LinearArgs &a, const LinearPlan &plan, void *ws, hipStream_t st) {
    const int out = a.slice_off[a.num_slices];
    const LinearSpace s = linear_space(plan, ws);
    if (plan.sorted) {
        launch_sort_rows(a, s, st);
        launch_sorted_inner(a, s, st);
    } else {
        // groups of up to 16 rows of one slot: every slot ends one that is not full
        const int most = a.n / 16 + a.num_slots, groups = a.n < most ? a.n : most, LR = a.num_slices * a.R;
        const dim3 narrow(groups, (LR + 15) / 16), wide(groups, (LR + 63) / 64);
        constexpr int kAll = kUnsortedRows / kWave;
        // (1168 units of 16 columns took 83 us where 236 of 64 take 50)
        if (narrow.x * narrow.y > 512) inner_kernel<4, 2, kAll><<<wide, kInThreads, 0, st>>>(a, s.xab);
        else if (a.n > kWave) inner_kernel<1, 4, kAll><<<narrow, kInThreads, 0, st>>>(a, s.xab);
        else inner_kernel<1, 4, 1><<<narrow, kInThreads, 0, st>>>(a, s.xab);
    }
    const Inner h{plan.sorted ? s.perm : nullptr, s.key_of, s.xab};
    const Tile tile = linear_tile(a.n, a.k, out, a.xq != nullptr, plan.sorted);
    if (a.xq && a.k <= kExactK) multiply<kE4m3AsBf16>(tile, a, h, out, st);
    else if (a.xq) multiply<kE4m3>(tile, a, h, out, st);
    else multiply<kBf16>(tile, a, h, out, st);
    return hipGetLastError();
}

}  // namespace st
