// step_linear.hip -- step_lora_linear: the shared projection with every row's
// adapter added,
//
//     y[i] = x[i] W^T + scale[s] (x[i] A_s^T) B_s^T,   s = slot[i].
//
// Two launches.  The first computes the inner sums xa[i] = scale[s] x[i] A_s^T
// of each slot's rows.  The second computes tiles of x W^T and, before it
// rounds, adds xa B_s^T for each slot that a tile's rows name, as matrix
// products in which only that slot's rows are not zero.
//
// With up to some hundred rows the product is bound by reading: W from memory,
// x from L2 by every workgroup.  The waves of a workgroup share one tile and
// take every kWaves-th line of k through rings of their own, so nothing that a
// wave loads is another's too and there is no barrier in the loop.  The waves'
// sums meet in shared memory once, at the end.
#include "step_linear.h"

namespace st {

namespace {

// ---------------------------------------------------------------- inner sums
// 16 rows of slot blockIdx.x (the blockIdx.y-th 16 of them) times 64 of the
// num_slices * R rows of A_s, 16 of these a workgroup: one CU alone draws no
// more than some 30 GB/s from memory, so A_s is spread over many.  Eight waves
// split k, so that each has only a few lines to wait for.
constexpr int kInWaves = 8, kInThreads = kInWaves * kWave, kInNT = 1, kInSlots = 4;
__global__ __launch_bounds__(kInThreads) void inner_kernel(LinearArgs a, uint16_t *xab) {
    using Part = Partials<kInNT, 1>;
    __shared__ int rows[16];
    __shared__ int before[kInWaves + 1];
    using Ring = LineRing<kInNT, 1, kInSlots>;
    __shared__ __align__(16) char rings[kInWaves * Ring::kBytes];
    __shared__ float red[kInWaves * Part::kFloats];
    const int slot = blockIdx.x, r_first = blockIdx.y * 16, c0 = blockIdx.z * Part::kCols;
    const int lane = tl::lane_id(), tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tl::wave_id());
    const int LR = a.num_slices * a.R, kbytes = a.k * 2, lines = (kbytes + kLine - 1) / kLine;

    // the slot's rows r_first .. r_first + 16, in order
    int found = 0;
    for (int r0 = 0; r0 < a.n && found < r_first + 16; r0 += kInThreads) {
        const bool hit = r0 + tid < a.n && a.slot[r0 + tid] == slot;
        const uint64_t mask = __ballot(hit);
        if (lane == 0) before[wave] = __popcll(mask);
        __syncthreads();
        int at = found + __popcll(mask & tl::lanemask_lt()), all = 0;
#pragma unroll
        for (int w = 0; w < kInWaves; ++w) {
            at += w < wave ? before[w] : 0;
            all += before[w];
        }
        if (hit && at >= r_first && at < r_first + 16) rows[at - r_first] = r0 + tid;
        found += all;
        __syncthreads();
    }
    const int count = min(found - r_first, 16);
    if (count <= 0) return;

    const uint16_t *A = a.a_pool + ((int64_t)slot * LR + c0) * a.k;
    const i32x4_t wr = words_rsrc(A, (uint32_t)(min(LR - c0, Part::kCols) * kbytes));
    const i32x4_t xr = words_rsrc(a.x, (uint32_t)(((int64_t)(a.n - 1) * a.ldx + a.k) * 2));
    const float scale = a.scale[slot];
    uint32_t wo[Ring::kW], xo[Ring::kX];
#pragma unroll
    for (int u = 0; u < Ring::kW; ++u) wo[u] = c0 + Ring::row(u) < LR ? (uint32_t)(Ring::row(u) * kbytes) : kOob;
#pragma unroll
    for (int u = 0; u < Ring::kX; ++u)
        xo[u] = Ring::row(u) < count ? (uint32_t)((int64_t)rows[Ring::row(u)] * a.ldx * 2) : kOob;
    f32x4_t acc[kInNT][1] = {};
    ring_product<kBf16, kInNT, 1, kInSlots>(wr, wo, xr, xo, rings + wave * Ring::kBytes, wave, kInWaves, lines, kbytes,
                                            acc);
    Part::put(red, wave, acc);
    __syncthreads();
    for (int t = tid; t < 16 * Part::kCols / 8; t += kInThreads) {
        const int m = t / (Part::kCols / 8), c = t % (Part::kCols / 8) * 8;
        if (m >= count || c0 + c >= LR) continue;
        float v[8];
        Part::sum8<kInWaves>(red, m, c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= scale;
        put_inner8(xab, rows[m], c0 + c, a.num_slices, a.R, v);
    }
}

// ---------------------------------------------------------------- the product
constexpr int kWaves = 4, kThreads = kWaves * kWave;

// SLOTS lines in a wave's ring; IT adapter steps in flight.
template <Form F, int MT, int NT, int SLOTS, int IT>
__global__ __launch_bounds__(kThreads) void linear_kernel(LinearArgs a, const uint16_t *xab, int out) {
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

    constexpr bool FP8 = F != kBf16;
    constexpr int esz = FP8 ? 1 : 2;
    const int kbytes = a.k * esz, lines = (kbytes + kLine - 1) / kLine;
    const int64_t ldx = FP8 ? a.ldxq : a.ldx * 2;
    const char *x = (FP8 ? (const char *)a.xq : (const char *)a.x) + m0 * ldx;
    const i32x4_t xr = words_rsrc(x, (uint32_t)((rows - 1) * ldx + kbytes));
    const i32x4_t wr = words_rsrc((const char *)a.w + (int64_t)c0 * kbytes, (uint32_t)(cols * kbytes));
    uint32_t wo[Ring::kW], xo[Ring::kX];
#pragma unroll
    for (int u = 0; u < Ring::kW; ++u) wo[u] = Ring::row(u) < cols ? (uint32_t)(Ring::row(u) * kbytes) : kOob;
#pragma unroll
    for (int u = 0; u < Ring::kX; ++u) xo[u] = Ring::row(u) < rows ? (uint32_t)(Ring::row(u) * ldx) : kOob;
    int my_slot = lane < rows ? a.slot[m0 + lane] : -1;
    if (my_slot >= a.num_slots) my_slot = -1;
    f32x4_t acc[NT][MT] = {};
    ring_product<F, NT, MT, SLOTS>(wr, wo, xr, xo, shared + wave * Ring::kBytes, wave, kWaves, lines, kbytes, acc);

    if constexpr (FP8) {
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
            const int m = 16 * i + lane % 16;
            const float xs = m < rows ? a.x_scale[m0 + m] : 0.0f;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][i][e] *= xs * ws[j][e];
        }
    }

    // ---- the adapters, in steps of 32 of the 2 R terms of one slice of one
    // slot (R rounded inner sums and R rests, against the same B twice); the
    // waves take every kWaves-th slot, IT steps at a time.
    const int chunks = a.R / 8;
    int first_slice = 0, end_slice = a.num_slices;
    while (a.slice_off[first_slice + 1] <= c0) ++first_slice;
    while (end_slice > first_slice + 1 && a.slice_off[end_slice - 1] >= c0 + cols) --end_slice;
    uint64_t left = __ballot(my_slot >= 0), same = 0;
    int slot = -1, slice = 0, q0 = 0;
    auto next_slot = [&](int skip) {  // skips `skip` slots, then takes one
        slice = first_slice;
        q0 = 0;
        do {
            if (!left) {
                slot = -1;
                same = 0;
                return;
            }
            slot = __builtin_amdgcn_readlane(my_slot, __builtin_ctzll(left));
            same = __ballot(my_slot == slot);
            left &= ~same;
        } while (skip--);
    };
    next_slot(wave);
    while (slot >= 0) {
        u32x4_t bf[IT][NT], xf[IT][MT];
        uint64_t who[IT];
#pragma unroll
        for (int s = 0; s < IT; ++s) {
            who[s] = same;
            const int q = q0 + lane / 16, r = (q >= chunks ? q - chunks : q) * 8;
            const bool in = q < 2 * chunks && slot >= 0;
            const uint16_t *B = a.b_pool + ((int64_t)slot * out + c0) * a.R + r;
            const uint16_t *X = xab + ((int64_t)m0 * a.num_slices + slice) * 2 * a.R + q * 8;
            const int lo = a.slice_off[slice] - c0, hi = min(a.slice_off[slice + 1] - c0, cols);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int c = 16 * j + lane % 16;
                bf[s][j] = in && c >= lo && c < hi ? tl::ld16(B + (int64_t)c * a.R) : tl::zero4();
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int m = 16 * i + lane % 16;
                xf[s][i] = in && (same >> m & 1) ? tl::ld16(X + (int64_t)m * a.num_slices * 2 * a.R) : tl::zero4();
            }
            if (slot >= 0 && (q0 += 4) >= 2 * chunks) {
                q0 = 0;
                if (++slice == end_slice) next_slot(kWaves - 1);
            }
        }
#pragma unroll
        for (int s = 0; s < IT; ++s)
#pragma unroll
            for (int i = 0; i < MT; ++i)
                if (who[s] >> (16 * i) & 0xffff)
#pragma unroll
                    for (int j = 0; j < NT; ++j) acc[j][i] = tl::mfma_16x16x32(bf[s][j], xf[s][i], acc[j][i]);
    }

    __syncthreads();
    Part::put(red, wave, acc);
    __syncthreads();
    for (int t = tid; t < Part::kRows * Part::kCols / 8; t += kThreads) {
        const int m = t / (Part::kCols / 8), c = t % (Part::kCols / 8) * 8;
        if (m >= rows || c >= cols) continue;
        float v[8];
        Part::template sum8<kWaves>(red, m, c, v);
        tl::st16(a.y + (int64_t)(m0 + m) * a.ldy + c0 + c, pack8(v));
    }
}

template <Form F, int MT, int NT, int SLOTS>
hipError_t go(const LinearArgs &a, const uint16_t *xab, int out, hipStream_t st) {
    const int m_tiles = (a.n + 16 * MT - 1) / (16 * MT), c_tiles = (out + 16 * NT - 1) / (16 * NT);
    linear_kernel<F, MT, NT, SLOTS, 2>
        <<<dim3((unsigned)((c_tiles + 7) / 8 * 8) * m_tiles), kThreads, 0, st>>>(a, xab, out);
    return hipGetLastError();
}

template <Form F>
hipError_t pick(const LinearArgs &a, const uint16_t *xab, int out, hipStream_t st) {
    const int tiles = (out + 15) / 16;
    if (a.n <= 16) return tiles > 768 ? go<F, 1, 2, 3>(a, xab, out, st) : go<F, 1, 1, 4>(a, xab, out, st);
    if (a.n <= 32) return tiles > 768 ? go<F, 2, 4, 2>(a, xab, out, st) : go<F, 2, 1, 4>(a, xab, out, st);
    const int m_tiles = (a.n + 63) / 64;
    auto rounds = [&](int nt) { return ((tiles + nt - 1) / nt * m_tiles + 255) / 256 * (4 + nt + 3); };
    if (rounds(6) <= rounds(4) && rounds(6) <= rounds(2)) return go<F, 4, 6, 2>(a, xab, out, st);
    return rounds(4) <= rounds(2) ? go<F, 4, 4, 2>(a, xab, out, st) : go<F, 4, 2, 3>(a, xab, out, st);
}

}  // namespace

hipError_t launch_lora_linear(const LinearArgs &a, const LinearPlan &plan, void *ws, hipStream_t st) {
    (void)plan;
    uint16_t *xab = static_cast<uint16_t *>(ws);
    const int out = a.slice_off[a.num_slices], cols = 16 * kInNT;
    inner_kernel<<<dim3(a.num_slots, (a.n + 15) / 16, (a.num_slices * a.R + cols - 1) / cols), kInThreads, 0, st>>>(
        a, xab);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.xq && a.k <= kExactK) return go<kE4m3AsBf16, 4, 4, 2>(a, xab, out, st);
    return a.xq ? pick<kE4m3>(a, xab, out, st) : pick<kBf16>(a, xab, out, st);
}

}  // namespace st
