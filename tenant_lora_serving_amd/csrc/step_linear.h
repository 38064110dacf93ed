// step_linear.h -- what the kernels of step_lora_linear share: the matrix
// products of one 128-byte line of k, and the streamed product of a few rows
// by a few weight rows, straight from memory to matrix-core registers.
// Internal to the library.
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

// How a line is multiplied.  The 8-bit instruction aligns the 16 to 32
// products that it adds at a time to the largest of them and drops what is
// more than about 2^14 smaller (measured with three-term sums).  Over a long k
// that averages out far below the result's rounding; over a short one it would
// show, so there the 8-bit values, which bf16 holds exactly, go through the
// bf16 instruction (k <= kExactK).
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

// acc[j][i] += W tile j (16 rows) * X tile i (16 rows)^T over the lines
// first, first + stride, ... of `lines`, both operands loaded in matrix-core
// layout from memory, one line ahead of its use.  wo / xo: byte offset of the
// lane's row (kOob for an absent row); a chunk past `kbytes` reads as zero on
// both sides.  (An absent row's chunk past the end wraps to some offset in
// range: what it reads reaches only the absent row's products.)
template <Form F, int NT, int MT>
__device__ __forceinline__ void stream_product(rsrc_t wr, const uint32_t *wo, rsrc_t xr, const uint32_t *xo, int first,
                                               int stride, int lines, int kbytes, f32x4_t (&acc)[NT][MT]) {
    const int g = (tl::lane_id() / 16) * 16;
    Line w[2][NT], x[2][MT];
    auto fetch = [&](int b, int s) {
        const int at = s * kLine + g;
        const uint32_t o0 = at < kbytes ? (uint32_t)at : kOob, o1 = at + 64 < kbytes ? (uint32_t)at + 64 : kOob;
#pragma unroll
        for (int j = 0; j < NT; ++j) w[b][j] = Line{tl::buf_ld16(wr, wo[j] + o0), tl::buf_ld16(wr, wo[j] + o1)};
#pragma unroll
        for (int i = 0; i < MT; ++i) x[b][i] = Line{tl::buf_ld16(xr, xo[i] + o0), tl::buf_ld16(xr, xo[i] + o1)};
    };
    auto use = [&](int b) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[j][i] = mma_line<F>(w[b][j], x[b][i], acc[j][i]);
    };
    if (first >= lines) return;
    fetch(0, first);
    for (int s = first; s < lines; s += 2 * stride) {
        if (s + stride < lines) fetch(1, s + stride);
        use(0);
        if (s + 2 * stride < lines) fetch(0, s + 2 * stride);
        if (s + stride < lines) use(1);
    }
}

}  // namespace st
