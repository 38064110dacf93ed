// step_linear.h -- what the kernels of step_lora_linear share: the matrix
// products of one 128-byte line of k, loads from memory into LDS, the product
// of a few rows by a few weight rows that a wave streams through a ring of lines
// there, and the care that one tenant's broken adapter takes.  Internal to the
// library.
#pragma once

#include <type_traits>

#include "common.h"
#include "step_kernels.h"

namespace st {

using tl::f32x4_t;
using tl::kOob;
using tl::kWave;
using tl::rsrc_t;
using tl::u32x4_t;

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// A line is 128 bytes of k of one row: 64 bf16 or 128 e4m3 values.  Lane l of
// a wave holds, of row l % 16, the 16-byte chunks l / 16 and 4 + l / 16 of
// the line.  Which k that is does not matter as long as both operands agree.
struct Line {
    u32x4_t a, b;
};
constexpr int kLine = 128;

// How a line is multiplied.  The 8-bit instruction cuts each of 8 consecutive
// products towards zero to a multiple of 2^(E - 13), E their largest exponent
// sum, before it adds them (measured with three-term sums; the instruction of
// 32 k at half the rate cuts alike); groups of 8 are added with the bf16
// instruction's 25 bits.  That is at most 2^-10 of a group's largest product,
// and over a long k of ordinary rows 2^-15 of the result, below its rounding to
// bf16; the exact way, the values widened to bf16, would take the bf16
// instruction's time.  Over a short k, where a cut does not average out, the
// values do go through the bf16 instruction, which holds them exactly (k <=
// kExactK).
enum Form { kBf16, kE4m3, kE4m3AsBf16 };

// Eight e4m3 values as bf16 (exact).
__device__ __forceinline__ u32x4_t widen8(uint32_t lo, uint32_t hi) {
    auto two = [](uint32_t v, auto high) {
        const auto f = __builtin_amdgcn_cvt_pk_f32_fp8((int)v, decltype(high)::value);
        return tl::pack_bf16x2(f[0], f[1]);
    };
    return u32x4_t{two(lo, std::false_type{}), two(lo, std::true_type{}), two(hi, std::false_type{}),
                   two(hi, std::true_type{})};
}

// acc += W line (16 rows) * X line (16 rows)^T: lane l gets x row l % 16 and
// w rows 4 * (l / 16) + 0..3.
template <Form F>
__device__ __forceinline__ f32x4_t mma_line(const Line &w, const Line &x, f32x4_t acc) {
    if constexpr (F == kE4m3) {
        const i32x8_t a = {(int)w.a.x, (int)w.a.y, (int)w.a.z, (int)w.a.w,
                           (int)w.b.x, (int)w.b.y, (int)w.b.z, (int)w.b.w};
        const i32x8_t b = {(int)x.a.x, (int)x.a.y, (int)x.a.z, (int)x.a.w,
                           (int)x.b.x, (int)x.b.y, (int)x.b.z, (int)x.b.w};
        // formats 0 (e4m3) for both operands, no block scales
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 0, 0, 0, 0, 0, 0);
    } else if constexpr (F == kE4m3AsBf16) {
        acc = tl::mfma_16x16x32(widen8(w.a.x, w.a.y), widen8(x.a.x, x.a.y), acc);
        acc = tl::mfma_16x16x32(widen8(w.a.z, w.a.w), widen8(x.a.z, x.a.w), acc);
        acc = tl::mfma_16x16x32(widen8(w.b.x, w.b.y), widen8(x.b.x, x.b.y), acc);
        return tl::mfma_16x16x32(widen8(w.b.z, w.b.w), widen8(x.b.z, x.b.w), acc);
    } else {
        acc = tl::mfma_16x16x32(w.a, x.a, acc);
        return tl::mfma_16x16x32(w.b, x.b, acc);
    }
}

// ---------------------------------------------------------------- loads into LDS
typedef int i32x4_t __attribute__((ext_vector_type(4)));

// A buffer resource as plain words, for the asm load below.
__device__ __forceinline__ i32x4_t words_rsrc(const void *base, uint32_t bytes) {
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    return i32x4_t{__builtin_amdgcn_readfirstlane((int)(uint32_t)p),
                   __builtin_amdgcn_readfirstlane((int)(uint32_t)(p >> 32) & 0xffff),
                   __builtin_amdgcn_readfirstlane((int)bytes), tl::kBufWord3};
}
// 16 bytes a lane from the buffer into LDS at `lds` + 16 * lane; offsets past
// the buffer write zeros.  There is no register result, so what is written is
// m0 (the LDS address) and LDS, which "memory" covers; the waits are written
// out below.  (m0 is a reserved register, which the compiler writes before each
// use of its own and never keeps for us: hence the warning that is turned off.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_lds(i32x4_t rsrc, uint32_t off, uint32_t more, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(lds), "v"(off), "s"(rsrc), "s"(more)
                 : "m0", "memory");
}
#pragma clang diagnostic pop
__device__ __forceinline__ void barrier() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}
// At most N of the wave's loads are still out.
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t lds_address(const char *p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char *)p;
}

// A wave's own ring of lines in LDS: a slot holds one line of NT tiles of w
// and MT tiles of x, 16 rows each.  Chunk c (16 bytes) of row r lies at place
// c ^ (r % 8) of the row, so that 16 rows' reads of one chunk fall on
// different banks.  A load instruction fills 8 rows, whole lines of memory.
template <int NT, int MT, int SLOTS>
struct LineRing {
    static constexpr int kSlot = (NT + MT) * 16 * kLine, kBytes = SLOTS * kSlot;
    static constexpr int kW = 2 * NT, kX = 2 * MT;  // load instructions of a line
    // The row that the lane's u-th load of w (or of x) belongs to.
    static __device__ __forceinline__ int row(int u) { return 8 * u + tl::lane_id() / 8; }
};

// acc[j][i] += W tile j (16 rows) * X tile i (16 rows)^T over the lines
// first, first + stride, ... of `lines`, by one wave on its own: lines come
// through its ring SLOTS - 1 ahead of their use, and a slot is refilled as
// soon as its fragments are in registers, so there is no barrier and the
// loads never pause for the products.  (Loads straight to registers in
// matrix-core layout take 16 rows x 64 bytes an instruction and ran at a
// third of this rate: a CU's outstanding lines bound them.)
// wo / xo: byte offset of the row of each of the lane's loads (kOob for an
// absent row); chunks past `kbytes` and lines past the last read as zero on
// both sides.  The first line read is number `turn`, and line 0 follows the
// last: rows of a power of two bytes have all their lines of one number in a
// few memory channels, and workgroups that start together would read those
// alone (one row by 4096 x 6144: 18.8 us without, 17.2 with; 37 rows by 4096 x
// 32008: 72 and 69).  (An absent row's chunk past the end wraps to some offset in
// range: what it reads reaches only the absent row's products.)
template <Form F, int NT, int MT, int SLOTS>
__device__ __forceinline__ void ring_product(i32x4_t wr, const uint32_t *wo, i32x4_t xr, const uint32_t *xo, char *ring,
                                             int first, int stride, int lines, int kbytes, f32x4_t (&acc)[NT][MT],
                                             int turn = 0) {
    using Ring = LineRing<NT, MT, SLOTS>;
    static_assert((SLOTS - 1) * (Ring::kW + Ring::kX) < 64, "the wait counts to 63");
    const int lane = tl::lane_id();
    const int chunk = ((lane & 7) ^ (lane / 8)) * 16;
    const uint32_t base = lds_address(ring);
    const int rd = (lane % 16) * kLine + (((lane / 16) ^ (lane & 7)) * 16);
    auto start = [&](int slot, int line) {
        const int from = line + turn < lines ? line + turn : line + turn - lines;
        const int at = from * kLine + chunk;
        const uint32_t o = line < lines && at < kbytes ? (uint32_t)at : kOob;
#pragma unroll
        for (int u = 0; u < Ring::kW; ++u) load_lds(wr, wo[u] + o, 0, base + slot * Ring::kSlot + u * 1024);
#pragma unroll
        for (int u = 0; u < Ring::kX; ++u) load_lds(xr, xo[u] + o, 0, base + slot * Ring::kSlot + (Ring::kW + u) * 1024);
    };
#pragma unroll
    for (int d = 0; d < SLOTS; ++d) start(d, first + d * stride);
#pragma unroll 1
    for (int s = first; s < lines; s += SLOTS * stride) {
#pragma unroll
        for (int d = 0; d < SLOTS; ++d) {
            wait_loads<(SLOTS - 1) * (Ring::kW + Ring::kX)>();
            const char *p = ring + d * Ring::kSlot;
            Line w[NT], x[MT];
#pragma unroll
            for (int j = 0; j < NT; ++j)
                w[j] = Line{tl::ld16(p + j * 2048 + rd), tl::ld16(p + j * 2048 + (rd ^ 64))};
#pragma unroll
            for (int i = 0; i < MT; ++i)
                x[i] = Line{tl::ld16(p + (NT + i) * 2048 + rd), tl::ld16(p + (NT + i) * 2048 + (rd ^ 64))};
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before it is refilled
            __builtin_amdgcn_sched_barrier(0);
            start(d, s + (d + SLOTS) * stride);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < MT; ++i) acc[j][i] = mma_line<F>(w[j], x[i], acc[j][i]);
        }
    }
    wait_loads<0>();  // (lines past the end still write zeros to the ring)
}

// Partial tiles of several waves side by side in shared memory, [wave][x row]
// [w row], 4 floats between rows against bank conflicts.
template <int NT, int MT>
struct Partials {
    static constexpr int kRows = 16 * MT, kCols = 16 * NT, kLd = kCols + 4, kFloats = kRows * kLd;
    static __device__ __forceinline__ void put(float *red, int wave, const f32x4_t (&acc)[NT][MT]) {
        const int lane = tl::lane_id();
        float *mine = red + wave * kFloats + (lane % 16) * kLd + 4 * (lane / 16);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < MT; ++i) *reinterpret_cast<f32x4_t *>(mine + 16 * i * kLd + 16 * j) = acc[j][i];
    }
    // Eight columns of a row, the waves added in their order.
    template <int WAVES>
    static __device__ __forceinline__ void sum8(const float *red, int row, int col, float *v) {
        f32x4_t lo = {}, hi = {};
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const float *p = red + w * kFloats + row * kLd + col;
            lo += *reinterpret_cast<const f32x4_t *>(p);
            hi += *reinterpret_cast<const f32x4_t *>(p + 4);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = lo[i], v[4 + i] = hi[i];
    }
};

__device__ __forceinline__ u32x4_t pack8(const float *v) {
    return u32x4_t{tl::pack_bf16x2(v[0], v[1]), tl::pack_bf16x2(v[2], v[3]), tl::pack_bf16x2(v[4], v[5]),
                   tl::pack_bf16x2(v[6], v[7])};
}

// The inner sums scale[s] x A_s^T travel as two bf16 terms a value (16 bits of
// mantissa; one term alone would add an error of the size of the result's own
// rounding): [row][slice][R rounded values, then R rests].  An infinity or NaN
// has rest 0; a finite value that would round to infinity is cut instead.
__device__ __forceinline__ void put_inner8(uint16_t *xab, int64_t row, int c, int num_slices, int R, const float *v) {
    float main[8], rest[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const bool finite = fabsf(v[e]) < INFINITY;
        main[e] = tl::bf16_round(v[e]);
        if (finite && !(fabsf(main[e]) < INFINITY)) main[e] = tl::bf_hi(__float_as_uint(v[e]));
        rest[e] = finite ? v[e] - main[e] : 0.0f;
    }
    uint16_t *to = xab + ((row * num_slices + c / R) * 2) * R + c % R;
    tl::st16(to, pack8(main));
    tl::st16(to + R, pack8(rest));
}

// ---------------------------------------------------------------- adapters in shared tiles
// A product with one slot's B multiplies the rows of other slots by zero.
// That is nothing unless the B holds an infinity or NaN, which must not reach
// them: fragments are looked through for one (exponent bits all set), ...
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u16x2_t larger_magnitude(u16x2_t m, uint32_t w) {
    return __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, w & 0x7fff7fffu));
}
__device__ __forceinline__ u16x2_t larger_magnitude(u16x2_t m, const u32x4_t v) {
    return larger_magnitude(larger_magnitude(larger_magnitude(larger_magnitude(m, v.x), v.y), v.z), v.w);
}
__device__ __forceinline__ bool not_finite(u16x2_t m) { return m.x >= 0x7f80 || m.y >= 0x7f80; }
// ... what is found is taken as zero, ...
__device__ __forceinline__ void drop_not_finite(u32x4_t &v) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint32_t w = v[e];
        if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
        if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
        v[e] = w;
    }
}
// ... and the results that it belongs to become NaN after the tile is stored.
// By every thread of the workgroup; slots: of the tile's rows m0 .. m0 + rows.
template <int THREADS>
__device__ __forceinline__ void mark_broken(const LinearArgs &a, int out, int m0, int rows, int c0, int cols,
                                            const int32_t *perm, const int32_t *slots) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the results themselves are stored
    __syncthreads();
#pragma unroll 1
    for (int t = threadIdx.x; t < rows * cols; t += THREADS) {
        const int m = m0 + t / cols, c = c0 + t % cols, slot = slots[m];
        if (slot < 0 || slot >= a.num_slots) continue;
        const uint16_t *B = a.b_pool + ((int64_t)slot * out + c) * a.R;
        u16x2_t big = {};
#pragma unroll 1
        for (int r = 0; r < a.R; r += 8) big = larger_magnitude(big, tl::ld16(B + r));
        if (not_finite(big)) a.y[(int64_t)(perm ? perm[m] : m) * a.ldy + c] = 0x7fc0;
    }
}

}  // namespace st
