// step_linear_tiled.hip -- step_lora_linear for many rows, where the shared
// product is bound by the matrix cores.
//
// The rows are first sorted by slot (a permutation, nothing moves), so that a
// tile of 256 rows names few slots, and the inner sums x A_s^T are kept as
// two bf16 terms a value.  A workgroup then computes 256 rows x 256 columns as
// one long product over lines of 128 bytes: the lines of x and W, and after
// them, for each slot of the tile, the line(s) of the inner sums and of B_s,
// with zeros for the rows of other slots.  The adapters so ride in the same
// pipeline, at 2 R / 64 lines a slot (2 of 66 at rank 64 and k 4096).
//
// Pipeline.  Eight waves, 2 x 4, hold 128 x 64 results each; the operands go
// through two 64 KB buffers of LDS, filled by loads that write LDS directly.
// A line takes four phases, one per quarter (64 x 32) of a wave's results; a
// phase reads the fragments that are due, starts the loads of one quarter of
// a later line, and then multiplies.  Four of the waves run half a phase
// behind the other four (one more barrier at the start), so on every SIMD one
// wave multiplies while the other reads.  A part of a buffer is refilled two
// phases after its last read and used six phases after its refill was
// started, so the wait is for loads that are 5 phases (10 loads) old.
// 6947 rows by 4096 x 28672 with rank-64 adapters: 1.2 PFLOP/s in bf16, 2.0 to
// 2.1 in e4m3, with the matrix cores busy 60% of the cycles in bf16.
#include "step_linear.h"

namespace st {

namespace {

constexpr int BM = 256, BN = 256;          // rows of x, rows of w of a tile
constexpr int kThreads = 512;
constexpr int kPart = 128 * kLine;         // bytes of a quarter of a buffer: 128 rows
constexpr int kBuf = 4 * kPart;            // A0, A1, B0, B1

// ---------------------------------------------------------------- sort by slot
// One workgroup: a count per slot, their prefix sum, then each row takes the
// next place of its slot.  Rows without an adapter come last (key S).  Which
// row of a slot gets which place varies; no result depends on it.
constexpr int kSortThreads = 1024;
__global__ __launch_bounds__(kSortThreads) void sort_kernel(const int32_t *slot, int n, int S, int32_t *perm,
                                                            int32_t *key_of) {
    __shared__ int place[kMaxSlots + 1];
    __shared__ int scratch[kSortThreads / kWave + 1];
    const int tid = threadIdx.x;
    for (int s = tid; s <= S; s += kSortThreads) place[s] = 0;
    __syncthreads();
    auto key_at = [&](int r) {
        const int s = slot[r];
        return s >= 0 && s < S ? s : S;
    };
    // Adds 1 to the row's slot's word; its value before is the answer.  A wave
    // whose rows are all of one slot, as in a long prompt, adds once (64 lanes
    // on one word take their turns: 14 us for 6947 rows).
    auto count = [&](int key) {
        const uint64_t here = __ballot(true);
        const int first = __builtin_amdgcn_readfirstlane(key);
        if (__ballot(key == first) != here) return atomicAdd(&place[key], 1);
        const int rank = __popcll(here & tl::lanemask_lt());
        int before = 0;
        if (rank == 0) before = atomicAdd(&place[first], __popcll(here));
        return __builtin_amdgcn_readfirstlane(before) + rank;
    };
    for (int r = tid; r < n; r += kSortThreads) count(key_at(r));
    __syncthreads();
    const int per = (S + kSortThreads) / kSortThreads, s0 = min(tid * per, S + 1), s1 = min(s0 + per, S + 1);
    int mine = 0, total;
    for (int s = s0; s < s1; ++s) mine += place[s];
    int at = tl::block_excl_scan<kSortThreads>(mine, scratch, total);
    for (int s = s0; s < s1; ++s) {
        const int c = place[s];
        place[s] = at;
        at += c;
    }
    __syncthreads();
    for (int r = tid; r < n; r += kSortThreads) {
        const int key = key_at(r), p = count(key);
        perm[p] = r;
        key_of[p] = key;
    }
}

// ---------------------------------------------------------------- inner sums
// scale[s] x A_s^T for 32 sorted rows and 16 NT of the num_slices * R rows
// of A_s, for each gridDim.z-th slot that the rows name; written as [row][slice][R rounded
// values, R rests] in bf16.  The waves take
// every WAVES-th line of k.
constexpr int kInMT = 2, kInRows = 16 * kInMT;
template <int kInNT, int kInSlots, int WAVES>
__global__ __launch_bounds__(WAVES *kWave) void sorted_inner_kernel(LinearArgs a, const int32_t *perm, const int32_t *key_of,
                                                           uint16_t *xab) {
    constexpr int kInCols = 16 * kInNT, kThreads = WAVES * kWave;
    using Part = Partials<kInNT, kInMT>;
    using Ring = LineRing<kInNT, kInMT, kInSlots>;
    __shared__ __align__(16) char shared[WAVES * (Ring::kBytes > Part::kFloats * 4 ? Ring::kBytes : Part::kFloats * 4)];
    float *red = reinterpret_cast<float *>(shared);
    const int lane = tl::lane_id(), tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tl::wave_id());
    char *ring = shared + wave * Ring::kBytes;
    // Of many tiles an XCD takes a run of row tiles, all columns of each: they
    // share rows of x and, mostly, the adapter in its L2 (48 -> 43 us for 6947
    // rows).  A few are spread over all XCDs.
    const int LR = a.num_slices * a.R, c_tiles = (LR + kInCols - 1) / kInCols;
    const int on_xcd = blockIdx.x / 8, per_xcd = gridDim.x / 8 / c_tiles;
    const bool runs = per_xcd >= 8;
    const int tile = runs ? blockIdx.x % 8 * per_xcd + on_xcd / c_tiles : (int)blockIdx.x / c_tiles;
    const int p0 = tile * kInRows, c0 = (runs ? on_xcd : (int)blockIdx.x) % c_tiles * kInCols;
    if (p0 >= a.n) return;
    const int kbytes = a.k * 2, lines = (kbytes + kLine - 1) / kLine;
    const i32x4_t xr = words_rsrc(a.x, (uint32_t)(((int64_t)(a.n - 1) * a.ldx + a.k) * 2));
    const bool here = lane < kInRows && p0 + lane < a.n;
    const int my_key = here ? key_of[p0 + lane] : a.num_slots;
    const int my_row = here ? perm[p0 + lane] : 0;
    uint32_t wo[Ring::kW], xo[Ring::kX];
#pragma unroll
    for (int u = 0; u < Ring::kW; ++u)
        wo[u] = c0 + Ring::row(u) < LR ? (uint32_t)(Ring::row(u) * kbytes) : kOob;
    uint64_t left = __ballot(my_key < a.num_slots);
    for (unsigned nth = 0; left; ++nth) {
        const int slot = __builtin_amdgcn_readlane(my_key, __builtin_ctzll(left));
        const uint64_t same = __ballot(my_key == slot);
        left &= ~same;
        if (nth % gridDim.z != blockIdx.z) continue;
        const uint16_t *A = a.a_pool + ((int64_t)slot * LR + c0) * a.k;
        const i32x4_t wr = words_rsrc(A, (uint32_t)(min(LR - c0, kInCols) * kbytes));
#pragma unroll
        for (int u = 0; u < Ring::kX; ++u) {
            const int m = Ring::row(u), row = __shfl(my_row, m);
            xo[u] = same >> m & 1 ? (uint32_t)((int64_t)row * a.ldx * 2) : kOob;
        }
        f32x4_t acc[kInNT][kInMT] = {};
        ring_product<kBf16, kInNT, kInMT, kInSlots>(wr, wo, xr, xo, ring, wave, WAVES, lines, kbytes, acc);
        __syncthreads();  // (the partial sums lie over the rings)
        Part::put(red, wave, acc);
        __syncthreads();
        const float scale = a.scale[slot];
        for (int t = tid; t < kInRows * kInCols / 8; t += kThreads) {
            const int m = t / (kInCols / 8), c = t % (kInCols / 8) * 8;
            if (!(same >> m & 1) || c0 + c >= LR) continue;
            float v[8];
            Part::template sum8<WAVES>(red, m, c, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= scale;
            put_inner8(xab, p0 + m, c0 + c, a.num_slices, a.R, v);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- the tiled product
// Which line comes next: the lines of x and W (slot < 0), or a line of a
// slot's inner sums and B.  Wave-uniform.
struct Cursor {
    int line;               // lines of x and W started so far
    int slot, slice, part;  // of the adapter line
    int lo, hi;             // columns of the slice in this tile
    bool done;
};

template <Form F>
__global__ __launch_bounds__(kThreads) void tiled_kernel(LinearArgs a, const int32_t *perm, const int32_t *key_of,
                                                         const uint16_t *xab, int out) {
    __shared__ __align__(16) char lds[2 * kBuf];
    __shared__ int keys[BM];
    const int lane = tl::lane_id(), tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tl::wave_id());

    // Tile of this workgroup.  Each XCD takes a run of the full-height tiles
    // in an order that walks 4 columns of tiles down the rows (32 workgroups
    // then share 8 row and 4 column panels in its L2), then its share of the
    // short tiles of the last rows.
    const int m_full = a.n / BM, c_tiles = (out + BN - 1) / BN;
    const int xcd = blockIdx.x % 8, nth = blockIdx.x / 8;
    const int full = m_full * c_tiles, f0 = (int)((int64_t)full * xcd / 8), f1 = (int)((int64_t)full * (xcd + 1) / 8);
    int mt, ct;
    if (nth < f1 - f0) {
        const int id = f0 + nth, group = id / (4 * m_full), in = id % (4 * m_full);
        const int wide = min(4, c_tiles - 4 * group);
        mt = in / wide;
        ct = 4 * group + in % wide;
    } else {
        const int shorts = a.n % BM ? c_tiles : 0;
        const int s0 = shorts * xcd / 8, s1 = shorts * (xcd + 1) / 8;
        mt = m_full;
        ct = s0 + nth - (f1 - f0);
        if (ct >= s1) return;
    }
    const int m0 = mt * BM, c0 = ct * BN, rows = min(a.n - m0, BM), cols = min(out - c0, BN);

    if (tid < BM) keys[tid] = tid < rows ? key_of[m0 + tid] : a.num_slots;
    __syncthreads();

    static_assert(F != kE4m3AsBf16, "short k is not tiled: its widened fragments do not fit beside the sums");
    constexpr int esz = F == kBf16 ? 2 : 1;
    const int kbytes = a.k * esz, lines = (kbytes + kLine - 1) / kLine;
    const int64_t ldx = F == kBf16 ? a.ldx * 2 : a.ldxq;
    const void *xb = F == kBf16 ? (const void *)a.x : (const void *)a.xq;
    const i32x4_t xr = words_rsrc(xb, (uint32_t)((int64_t)(a.n - 1) * ldx + kbytes));
    const i32x4_t wr = words_rsrc((const char *)a.w + (int64_t)c0 * kbytes, (uint32_t)(cols * kbytes));
    const int xab_ld = a.num_slices * 2 * a.R * 2;  // bytes a row of the inner sums
    const i32x4_t ar = words_rsrc((const char *)xab + (int64_t)m0 * xab_ld, (uint32_t)(rows * xab_ld));

    // A quarter of a buffer is loaded by 16 wave loads of 8 rows, two a wave.
    // LDS slot s (16 bytes) of row r holds chunk s ^ (r % 8): the reads of 16
    // rows at one chunk then fall on different banks.
    const int l8 = lane / 8, chunk = (lane % 8) ^ l8;
    int ra[2], rb[2];  // tile rows of the lane's loads in A0 and B0; A1: + 64, B1: + 32
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = wave * 2 + u;
        ra[u] = (i / 8) * 128 + (i % 8) * 8 + l8;
        rb[u] = (i / 4) * 64 + (i % 4) * 8 + l8;
    }
    // Byte offsets of the lane's chunk in line 0 of its rows: A0, A0, A1, A1
    // and B0, B0, B1, B1.  Absent rows read the first one's: their products
    // reach no result that is stored.
    uint32_t xo[4], wo[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int r = ra[u & 1] + 64 * (u / 2), c = rb[u & 1] + 32 * (u / 2);
        xo[u] = (uint32_t)((int64_t)perm[m0 + (r < rows ? r : 0)] * ldx) + chunk * 16;
        wo[u] = (uint32_t)((c < cols ? c : 0) * kbytes) + chunk * 16;
    }

    // ---- the adapter lines of this tile
    const int parts = (2 * a.R + 63) / 64, chunks = a.R / 8;
    int first_slice = 0, end_slice = a.num_slices;
    while (a.slice_off[first_slice + 1] <= c0) ++first_slice;
    while (end_slice > first_slice + 1 && a.slice_off[end_slice - 1] >= c0 + cols) --end_slice;
    // rows with a key <= k; keys ascend, so this is the next slot's first row
    auto rows_upto = [&](int k) {
        int c = 0;
#pragma unroll
        for (int u = 0; u < BM / kWave; ++u) c += __popcll(__ballot(keys[u * kWave + lane] <= k));
        return c;
    };
    auto slot_at = [&](int p) { return p < BM ? __builtin_amdgcn_readfirstlane(keys[p]) : a.num_slots; };
    int distinct = 0;
    for (int s = slot_at(0); s < a.num_slots; s = slot_at(rows_upto(s))) ++distinct;
    const int total = lines + distinct * (end_slice - first_slice) * parts;

    Cursor cur{0, -1, first_slice, 0, 0, 0, false};
    i32x4_t br = wr;
    auto enter_slice = [&](int l) {
        cur.slice = l;
        cur.lo = a.slice_off[l] - c0;
        cur.hi = a.slice_off[l + 1] - c0;
    };
    auto enter_slot = [&](int s) {
        cur.slot = s;
        cur.done = s >= a.num_slots;
        enter_slice(first_slice);
        if (!cur.done)
            br = words_rsrc(a.b_pool + ((int64_t)s * out + c0) * a.R, (uint32_t)((int64_t)cols * a.R * 2));
    };
    auto advance = [&]() {
        if (cur.line < lines) {
            if (++cur.line == lines) enter_slot(slot_at(0));
        } else if (!cur.done) {
            if (++cur.part == parts) {
                cur.part = 0;
                if (cur.slice + 1 < end_slice) enter_slice(cur.slice + 1);
                else enter_slot(slot_at(rows_upto(cur.slot)));
            }
        }
    };
    const uint32_t lds0 =
        lds_address(lds) + wave * 2048;
    // Starts the loads of part P (0 A0, 1 A1, 2 B0, 3 B1) of a line into buffer b: a whole line of x and W, ...
    auto start_whole = [&](int b, int line, auto part_of) {
        constexpr int P = decltype(part_of)::value, H = P & 1;
#pragma unroll
        for (int u = 0; u < 2; ++u)
            load_lds(P < 2 ? xr : wr, (P < 2 ? xo : wo)[2 * H + u], line * kLine, lds0 + b * kBuf + P * kPart + u * 1024);
    };
    // ... or the cursor's line, whichever it is.
    auto start_any = [&](int b, auto part_of) {
        constexpr int P = decltype(part_of)::value, H = P & 1;
        uint32_t off[2];
        i32x4_t rsrc;
        if (cur.line < lines) {
            const int at = cur.line * kLine;
            rsrc = P < 2 ? xr : wr;
#pragma unroll
            for (int u = 0; u < 2; ++u) off[u] = at + chunk * 16 < kbytes ? (P < 2 ? xo : wo)[2 * H + u] + at : kOob;
        } else {
            const int q = cur.part * 8 + chunk;  // of R/8 chunks of rounded values, then R/8 of rests
            const bool in = (int)!cur.done & (int)(q < 2 * chunks);
            rsrc = P < 2 ? ar : br;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if constexpr (P < 2) {
                    const int r = ra[u] + 64 * H;
                    off[u] = (int)in & (int)(keys[r] == cur.slot) ? (uint32_t)(r * xab_ld + cur.slice * 4 * a.R + q * 16)
                                                                  : kOob;
                } else {
                    const int c = rb[u] + 32 * H;
                    off[u] = (int)in & (int)(c >= cur.lo) & (int)(c < cur.hi)
                                 ? (uint32_t)(c * a.R * 2 + (q >= chunks ? q - chunks : q) * 16)
                                 : kOob;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) load_lds(rsrc, off[u], 0, lds0 + b * kBuf + P * kPart + u * 1024);
    };
    using P0 = std::integral_constant<int, 0>;
    using P1 = std::integral_constant<int, 1>;
    using P2 = std::integral_constant<int, 2>;
    using P3 = std::integral_constant<int, 3>;

    // ---- fragments
    const int wm = wave / 4, wn = wave % 4;
    const int rd = (lane % 16) * kLine + (((lane / 16) ^ (lane & 7)) * 16);
    const char *ra_base = lds + wm * 64 * kLine, *rb_base = lds + 2 * kPart + wn * 32 * kLine;
    Line fa[2][4], fb[2][2];
    f32x4_t acc[4][8] = {};  // [column tile][row tile]
    auto read_a = [&](int b, int h) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const char *p = ra_base + b * kBuf + h * kPart + i * 16 * kLine;
            fa[h][i] = Line{tl::ld16(p + rd), tl::ld16(p + (rd ^ 64))};
        }
    };
    auto read_b = [&](int b, int h) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const char *p = rb_base + b * kBuf + h * kPart + j * 16 * kLine;
            fb[h][j] = Line{tl::ld16(p + rd), tl::ld16(p + (rd ^ 64))};
        }
    };
    const int live = rows - wm * 128;  // rows of this wave
    auto multiply = [&](auto form, int ha, int hb) __attribute__((always_inline)) {
        barrier();
        if (live > ha * 64) {
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[2 * hb + j][4 * ha + i] =
                        mma_line<decltype(form)::value>(fb[hb][j], fa[ha][i], acc[2 * hb + j][4 * ha + i]);
            __builtin_amdgcn_s_setprio(0);
        }
        barrier();
    };

    // ---- fill: line 0 whole, line 1 but its A1 (the first phase starts that).
    // In steady state a phase waits with the 10 newest loads still out.
    start_any(0, P0{});
    start_any(0, P2{});
    start_any(0, P3{});
    start_any(0, P1{});
    advance();
    start_any(1, P0{});
    start_any(1, P2{});
    start_any(1, P3{});
    wait_loads<12>();  // A0 of line 0 is there
    barrier();
    if (wave >= 4) barrier();  // half a phase behind
    read_a(0, 0);
    wait_loads<10>();  // and B0
    barrier();
    barrier();
    // The line t in buffer b.  whole: lines t + 1 and t + 2 are whole lines of x and W.
    bool broken = false;
    auto look_through = [&](int h) __attribute__((always_inline)) {
        u16x2_t big = {};
#pragma unroll
        for (int j = 0; j < 2; ++j) big = larger_magnitude(larger_magnitude(big, fb[h][j].a), fb[h][j].b);
        if (!__ballot(not_finite(big))) return;
        broken = true;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            drop_not_finite(fb[h][j].a);
            drop_not_finite(fb[h][j].b);
        }
    };
    auto line_step = [&](auto form, auto adapter, auto whole, int t, int b) __attribute__((always_inline)) {
        constexpr bool W = decltype(whole)::value;
        // phase 1: B0; starts A1 of the next line
        read_b(b, 0);
        if constexpr (W) start_whole(b ^ 1, t + 1, P1{});
        else start_any(b ^ 1, P1{});
        wait_loads<10>();
        if constexpr (decltype(adapter)::value) look_through(0);
        multiply(form, 0, 0);
        // phase 2: B1; starts A0 of the line after it
        if constexpr (!W) advance();
        read_b(b, 1);
        if constexpr (W) start_whole(b, t + 2, P0{});
        else start_any(b, P0{});
        wait_loads<10>();
        if constexpr (decltype(adapter)::value) look_through(1);
        multiply(form, 0, 1);
        // phase 3: A1
        read_a(b, 1);
        if constexpr (W) start_whole(b, t + 2, P2{});
        else start_any(b, P2{});
        wait_loads<10>();
        multiply(form, 1, 1);
        // phase 4: A0 of the next line
        read_a(b ^ 1, 0);
        if constexpr (W) start_whole(b, t + 2, P3{});
        else start_any(b, P3{});
        wait_loads<10>();
        multiply(form, 1, 0);
    };
    using Main = std::integral_constant<Form, F>;
    using Extra = std::integral_constant<Form, kBf16>;
    using Yes = std::true_type;
    using No = std::false_type;
    int t = 0;
    for (; t + 3 < kbytes / kLine; t += 2) {
        line_step(Main{}, No{}, Yes{}, t, 0);
        line_step(Main{}, No{}, Yes{}, t + 1, 1);
    }
    if (t > 0) cur.line = t + 1;  // (line t + 1 is started but for its A1)
#pragma unroll 1
    for (; t < lines; ++t) line_step(Main{}, No{}, No{}, t, t & 1);
    if constexpr (F != kBf16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int m = wm * 128 + 16 * i + lane % 16;
            const float xs = m < rows ? a.x_scale[perm[m0 + m]] : 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][i][e] *= xs;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = wn * 64 + 16 * j + 4 * (lane / 16) + e;
                const float ws = c < cols ? a.w_scale[c0 + c] : 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[j][i][e] *= ws;
            }
    }
#pragma unroll 1
    for (; t < total; ++t) line_step(Extra{}, Yes{}, No{}, t, t & 1);
    if (wave < 4) barrier();
    wait_loads<0>();  // nothing may still write LDS when the workgroup ends

#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int m = wm * 128 + 16 * i + lane % 16;
        if (m >= rows) continue;
        uint16_t *y = a.y + (int64_t)perm[m0 + m] * a.ldy + c0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = wn * 64 + 16 * j + 4 * (lane / 16);
            if (c < cols)
                *reinterpret_cast<uint2 *>(y + c) = make_uint2(tl::pack_bf16x2(acc[j][i][0], acc[j][i][1]),
                                                               tl::pack_bf16x2(acc[j][i][2], acc[j][i][3]));
        }
    }

    if (__syncthreads_or(broken)) mark_broken<kThreads>(a, out, m0, rows, c0, cols, perm, key_of);
}

template <Form F>
void go(const LinearArgs &a, const int32_t *perm, const int32_t *key_of, const uint16_t *xab, int out,
        hipStream_t st) {
    const int c_tiles = (out + BN - 1) / BN, full = a.n / BM * c_tiles, shorts = a.n % BM ? c_tiles : 0;
    tiled_kernel<F><<<dim3(8 * ((full + 7) / 8 + (shorts + 7) / 8)), kThreads, 0, st>>>(a, perm, key_of, xab, out);
}

}  // namespace

void launch_sort_rows(const LinearArgs &a, const LinearSpace &s, hipStream_t st) {
    sort_kernel<<<1, kSortThreads, 0, st>>>(a.slot, a.n, a.num_slots, s.perm, s.key_of);
}

void launch_sorted_inner(const LinearArgs &a, const LinearSpace &s, hipStream_t st) {
    const int tiles = (a.n + kInRows - 1) / kInRows, LR = a.num_slices * a.R, wide = (LR + 63) / 64;
    // 32 rows name 1 + S / tiles slots on average where all S are named alike;
    // one workgroup for all of them took 95 us for 300 rows of 300 slots
    const int named = 1 + a.num_slots / tiles, split = named < kInRows ? named : kInRows;
    const unsigned all = (tiles + 7) / 8 * 8;
    // columns of 64 read x less often; with few of them the CUs that idle cost more
    if (tiles * wide * split >= 256)
        sorted_inner_kernel<4, 2, 4><<<dim3(all * wide, 1, split), 256, 0, st>>>(a, s.perm, s.key_of, s.xab);
    else
        sorted_inner_kernel<1, 3, 8>
            <<<dim3(all * ((LR + 15) / 16), 1, split), 512, 0, st>>>(a, s.perm, s.key_of, s.xab);
}

void launch_lora_linear_tiled(const LinearArgs &a, const int32_t *perm, const int32_t *key_of, const uint16_t *xab,
                              hipStream_t st) {
    const int out = a.slice_off[a.num_slices];
    if (a.xq) go<kE4m3>(a, perm, key_of, xab, out, st);
    else go<kBf16>(a, perm, key_of, xab, out, st);
}

}  // namespace st
