// step_linear.hip -- step_lora_linear: the shared projection with every row's
// adapter added,
//
//     y[i] = x[i] W^T + scale[s] (x[i] A_s^T) B_s^T,   s = slot[i].
//
// Two launches.  The first computes the inner sums xa[i] = scale[s] x[i] A_s^T
// (fp32, a slot's rows gathered into matrix-core tiles).  The second computes
// a tile of x W^T and, before it rounds, adds xa B_s^T for each slot that the
// tile's rows name, as matrix products in which only that slot's rows are not
// zero.  A group of four waves shares a tile, each taking every fourth line
// of k and every fourth slot; their sums meet in shared memory.
#include "step_linear.h"

namespace st {

namespace {

constexpr int kWaves = 4, kThreads = kWaves * kWave;
constexpr int MT = 4, NT = 4;              // 16-row tiles of x and of w in a workgroup's tile
constexpr int kRows = 16 * MT, kCols = 16 * NT;
constexpr int kRedLd = kCols + 4;          // floats a row in shared memory

// The waves' partial tiles side by side in shared memory, summed in the order
// of the waves: red[wave][row][column].
__device__ __forceinline__ void put_partial(float *red, int wave, const f32x4_t (&acc)[NT][MT]) {
    const int lane = tl::lane_id();
    float *mine = red + wave * kRows * kRedLd;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i)
            *reinterpret_cast<f32x4_t *>(mine + (16 * i + lane % 16) * kRedLd + 16 * j + 4 * (lane / 16)) = acc[j][i];
}
__device__ __forceinline__ void sum8(const float *red, int row, int col, float *v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const float *p = red + (w * kRows + row) * kRedLd + col;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += p[i];
    }
}

// xa[piece][row][c] for the rows of slot blockIdx.x, columns 64 blockIdx.z ..
// of the num_slices * R rows of A_s, over piece blockIdx.y of k.
__global__ __launch_bounds__(kThreads) void inner_kernel(LinearArgs a, float *xa, int pieces) {
    __shared__ int rows[kThreads];
    __shared__ int n_rows;
    __shared__ float red[kWaves * kRows * kRedLd];
    const int slot = blockIdx.x, piece = blockIdx.y, c0 = blockIdx.z * kCols;
    const int lane = tl::lane_id(), wave = tl::wave_id(), tid = threadIdx.x;
    const int LR = a.num_slices * a.R, kbytes = a.k * 2, lines = (kbytes + kLine - 1) / kLine;
    const uint16_t *A = a.a_pool + (int64_t)slot * LR * a.k;
    const rsrc_t wr = tl::make_rsrc(A + (int64_t)c0 * a.k, (uint32_t)(min(LR - c0, kCols) * kbytes));
    const rsrc_t xr = tl::make_rsrc(a.x, (uint32_t)(((int64_t)(a.n - 1) * a.ldx + a.k) * 2));
    const float scale = a.scale[slot];
    uint32_t wo[NT], xo[MT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int c = 16 * j + lane % 16;
        wo[j] = c0 + c < LR ? (uint32_t)(c * kbytes) : kOob;
    }
    for (int r0 = 0; r0 < a.n; r0 += kThreads) {
        if (tid == 0) n_rows = 0;
        __syncthreads();
        if (r0 + tid < a.n && a.slot[r0 + tid] == slot) rows[atomicAdd(&n_rows, 1)] = r0 + tid;
        __syncthreads();
        const int found = n_rows;
        for (int b = 0; b < found; b += kRows) {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int m = b + 16 * i + lane % 16;
                xo[i] = m < found ? (uint32_t)((int64_t)rows[m] * a.ldx * 2) : kOob;
            }
            f32x4_t acc[NT][MT] = {};
            stream_product<kBf16, NT, MT>(wr, wo, xr, xo, piece * kWaves + wave, pieces * kWaves, lines, kbytes, acc);
            put_partial(red, wave, acc);
            __syncthreads();
            for (int t = tid; t < kRows * kCols / 8; t += kThreads) {
                const int m = t / (kCols / 8), c = t % (kCols / 8) * 8;
                if (b + m >= found || c0 + c >= LR) continue;
                float v[8];
                sum8(red, m, c, v);
                float *to = xa + ((int64_t)piece * a.n + rows[b + m]) * LR + c0 + c;
#pragma unroll
                for (int i = 0; i < 8; ++i) to[i] = v[i] * scale;
            }
            __syncthreads();
        }
        __syncthreads();
    }
}

// Eight inner sums of a row as bf16: the rounded values, or what the rounding left.
__device__ __forceinline__ u32x4_t xa_chunk(const float *xa, int64_t piece_stride, int pieces, bool rest) {
    float v[8] = {};
    for (int p = 0; p < pieces; ++p)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += xa[p * piece_stride + i];
    if (rest)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] -= tl::bf16_round(v[i]);
    return u32x4_t{tl::pack_bf16x2(v[0], v[1]), tl::pack_bf16x2(v[2], v[3]), tl::pack_bf16x2(v[4], v[5]),
                   tl::pack_bf16x2(v[6], v[7])};
}

template <Form F>
__global__ __launch_bounds__(kThreads) void linear_kernel(LinearArgs a, const float *xa, int pieces, int out) {
    __shared__ float red[kWaves * kRows * kRedLd];
    const int lane = tl::lane_id(), wave = tl::wave_id(), tid = threadIdx.x;
    // row tiles of the same columns run next to each other on one XCD
    const int m_tiles = (a.n + kRows - 1) / kRows;
    const int on_xcd = blockIdx.x / 8;
    const int c0 = (on_xcd / m_tiles * 8 + blockIdx.x % 8) * kCols, m0 = on_xcd % m_tiles * kRows;
    if (c0 >= out) return;
    const int rows = min(a.n - m0, kRows), cols = min(out - c0, kCols);

    constexpr bool FP8 = F != kBf16;
    constexpr int esz = FP8 ? 1 : 2;
    const int kbytes = a.k * esz, lines = (kbytes + kLine - 1) / kLine;
    const int64_t ldx = FP8 ? a.ldxq : a.ldx * 2;
    const char *x = (FP8 ? (const char *)a.xq : (const char *)a.x) + m0 * ldx;
    const rsrc_t xr = tl::make_rsrc(x, (uint32_t)((rows - 1) * ldx + kbytes));
    const rsrc_t wr = tl::make_rsrc((const char *)a.w + (int64_t)c0 * kbytes, (uint32_t)(cols * kbytes));
    uint32_t wo[NT], xo[MT];
#pragma unroll
    for (int j = 0; j < NT; ++j) wo[j] = 16 * j + lane % 16 < cols ? (uint32_t)((16 * j + lane % 16) * kbytes) : kOob;
#pragma unroll
    for (int i = 0; i < MT; ++i) xo[i] = 16 * i + lane % 16 < rows ? (uint32_t)((16 * i + lane % 16) * ldx) : kOob;
    f32x4_t acc[NT][MT] = {};
    stream_product<F, NT, MT>(wr, wo, xr, xo, wave, kWaves, lines, kbytes, acc);

    if constexpr (FP8) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int m = 16 * i + lane % 16;
            const float xs = m < rows ? a.x_scale[m0 + m] : 0.0f;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int c = 16 * j + 4 * (lane / 16) + e;
                    acc[j][i][e] *= xs * (c < cols ? a.w_scale[c0 + c] : 0.0f);
                }
        }
    }

    // ---- the adapters: each distinct slot of the tile's rows once
    const int LR = a.num_slices * a.R, chunks = a.R / 8;
    const int64_t piece_stride = (int64_t)a.n * LR;
    int my_slot = lane < rows ? a.slot[m0 + lane] : -1;
    if (my_slot >= a.num_slots) my_slot = -1;
    uint64_t left = __ballot(my_slot >= 0);
    for (int nth = 0; left; ++nth) {
        const int slot = __builtin_amdgcn_readlane(my_slot, __builtin_ctzll(left));
        const uint64_t same = __ballot(my_slot == slot);
        left &= ~same;
        if (nth % kWaves != wave) continue;
        const uint16_t *B = a.b_pool + ((int64_t)slot * out + c0) * a.R;
        for (int l = 0; l < a.num_slices; ++l) {
            const int lo = max(a.slice_off[l] - c0, 0), hi = min(a.slice_off[l + 1] - c0, cols);
            if (lo >= hi) continue;
            // the rounded inner sums, then what rounding left of them, against the same B
            for (int q0 = 0; q0 < 2 * chunks; q0 += 4) {
                const int q = q0 + lane / 16, r = (q >= chunks ? q - chunks : q) * 8;
                u32x4_t xf[MT];
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const int m = 16 * i + lane % 16;
                    xf[i] = q < 2 * chunks && (same >> m & 1)
                                ? xa_chunk(xa + (int64_t)(m0 + m) * LR + l * a.R + r, piece_stride, pieces, q >= chunks)
                                : tl::zero4();
                }
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const int c = 16 * j + lane % 16;
                    const u32x4_t bf =
                        q < 2 * chunks && c >= lo && c < hi ? tl::ld16(B + (int64_t)c * a.R + r) : tl::zero4();
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        if (same >> (16 * i) & 0xffff) acc[j][i] = tl::mfma_16x16x32(bf, xf[i], acc[j][i]);
                }
            }
        }
    }

    put_partial(red, wave, acc);
    __syncthreads();
    for (int t = tid; t < kRows * kCols / 8; t += kThreads) {
        const int m = t / (kCols / 8), c = t % (kCols / 8) * 8;
        if (m >= rows || c >= cols) continue;
        float v[8];
        sum8(red, m, c, v);
        tl::st16(a.y + (int64_t)(m0 + m) * a.ldy + c0 + c,
                 u32x4_t{tl::pack_bf16x2(v[0], v[1]), tl::pack_bf16x2(v[2], v[3]), tl::pack_bf16x2(v[4], v[5]),
                         tl::pack_bf16x2(v[6], v[7])});
    }
}

}  // namespace

hipError_t launch_lora_linear(const LinearArgs &a, const LinearPlan &plan, void *ws, hipStream_t st) {
    float *xa = static_cast<float *>(ws);
    const int out = a.slice_off[a.num_slices];
    inner_kernel<<<dim3(a.num_slots, plan.k_pieces, (a.num_slices * a.R + kCols - 1) / kCols), kThreads, 0, st>>>(
        a, xa, plan.k_pieces);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int m_tiles = (a.n + kRows - 1) / kRows, c_tiles = (out + kCols - 1) / kCols;
    const dim3 grid((unsigned)((c_tiles + 7) / 8 * 8) * m_tiles);
    if (a.xq && a.k <= kExactK) linear_kernel<kE4m3AsBf16><<<grid, kThreads, 0, st>>>(a, xa, plan.k_pieces, out);
    else if (a.xq) linear_kernel<kE4m3><<<grid, kThreads, 0, st>>>(a, xa, plan.k_pieces, out);
    else linear_kernel<kBf16><<<grid, kThreads, 0, st>>>(a, xa, plan.k_pieces, out);
    return hipGetLastError();
}

}  // namespace st
