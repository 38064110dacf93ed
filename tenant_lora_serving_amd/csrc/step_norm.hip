// step_norm.hip -- step_rms_norm: the root-mean-square norm with the
// residual's addition and an e4m3 copy of the result.
//
//     s = x + residual;  y = s * w / sqrt(mean(s^2) + eps);  q = y / (max|y| / 448)
//
// A row is held in fp32 registers by the threads that read it, so it is read
// once: the sum of squares and the largest |s w| are reduced together and
// everything else is elementwise (max|y| = max|s w| * rstd).  Rows whose squares
// or products leave fp32's range, or that hold a NaN or an infinity, take
// another reduction.  Bound by memory
// traffic when there are many rows (6947 x 4096 with residual, both outputs:
// 41 us, 6.2 TB/s of the least bytes) and by the latency of one load, one
// reduction and one store when there are few (1 x 4096: 2.8 us).
#include "common.h"
#include "step_kernels.h"

namespace st {

using tl::bf_hi;
using tl::bf_lo;
using tl::kWave;
using tl::ld16;
using tl::ld16_stream;
using tl::pack_bf16x2;
using tl::st16;
using tl::u32x4_t;

namespace {

constexpr float kE4m3Max = 448.0f;

__device__ __forceinline__ float wave_sum(float v) {
    for (int d = kWave / 2; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}
// The larger of two magnitudes, NaN if one is (v_maximum3_f32; fmaxf would drop it).
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }
__device__ __forceinline__ float wave_max(float v) {
    for (int d = kWave / 2; d; d >>= 1) v = larger(v, __shfl_xor(v, d));
    return v;
}

// Sum of `a` and maximum of `b` over the NT threads of a row.
template <int NT>
__device__ __forceinline__ void row_reduce(float &a, float &b, float2 *scratch) {
    a = wave_sum(a);
    b = wave_max(b);
    if constexpr (NT > kWave) {
        const int w = threadIdx.x / kWave;
        __syncthreads();
        if (tl::lane_id() == 0) scratch[w] = make_float2(a, b);
        __syncthreads();
        a = 0.0f;
        b = 0.0f;
        for (int i = 0; i < NT / kWave; ++i) {
            a += scratch[i].x;
            b = larger(b, scratch[i].y);
        }
    }
}

__device__ __forceinline__ void unpack8(const u32x4_t v, float *f) {
    f[0] = bf_lo(v.x), f[1] = bf_hi(v.x), f[2] = bf_lo(v.y), f[3] = bf_hi(v.y);
    f[4] = bf_lo(v.z), f[5] = bf_hi(v.z), f[6] = bf_lo(v.w), f[7] = bf_hi(v.w);
}
__device__ __forceinline__ u32x4_t pack8(const float *f) {
    return u32x4_t{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                   pack_bf16x2(f[6], f[7])};
}
// Eight floats -> e4m3, round to nearest even (v_cvt_pk_fp8_f32, OCP on gfx950).
__device__ __forceinline__ uint2 pack8_e4m3(const float *f) {
    int a = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], a, true);
    int b = __builtin_amdgcn_cvt_pk_fp8_f32(f[4], f[5], 0, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(f[6], f[7], b, true);
    return make_uint2((uint32_t)a, (uint32_t)b);
}

// NT threads a row, VPT 16-byte vectors (8 values) a thread, ROWS rows a
// workgroup (ROWS > 1 only where a wave holds a row).
template <int NT, int VPT, int ROWS>
__global__ __launch_bounds__(NT *ROWS) void rms_norm_kernel(NormArgs a) {
    __shared__ float2 scratch[NT / kWave];
    const int t = threadIdx.x % NT;
    const int row = (blockIdx.y * gridDim.x + blockIdx.x) * ROWS + threadIdx.x / NT;
    if (row >= a.n) return;  // (a whole wave; with ROWS > 1 there is no barrier)
    const int vecs = a.h / 8;
    const uint16_t *xr = a.x + (int64_t)row * a.ldx;
    const uint16_t *rr = a.residual ? a.residual + (int64_t)row * a.ldr : nullptr;

    u32x4_t xv[VPT], rv[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = t + j * NT;
        xv[j] = v < vecs ? ld16_stream(xr + v * 8) : tl::zero4();
        rv[j] = rr && v < vecs ? ld16_stream(rr + v * 8) : tl::zero4();
    }
    float s[VPT][8], w[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = t + j * NT;
        unpack8(v < vecs ? ld16(a.weight + v * 8) : tl::zero4(), w[j]);
    }
    float ss = 0.0f, am = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        float r[8];
        unpack8(xv[j], s[j]);
        unpack8(rv[j], r);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (rr) s[j][i] += r[i];
            ss = fmaf(s[j][i], s[j][i], ss);
            am = larger(am, fabsf(s[j][i] * w[j][i]));
        }
    }
    if (a.residual_out) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = t + j * NT;
            if (v < vecs) st16(a.residual_out + (int64_t)row * a.h + v * 8, pack8(s[j]));
        }
    }
    row_reduce<NT>(ss, am, scratch);
    float mean = ss / (float)a.h + a.eps;
    float rstd = 1.0f / sqrtf(mean);
    if (mean < 0x1p-100f) {
        // squares below fp32's smallest numbers, and an eps that does not hide
        // them: the row is lifted by 2^80, which keeps every s (2^-133 at
        // least, or 0) and its square in range.  A row of zeros stays one.
        ss = 0.0f;
        am = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s[j][i] *= 0x1p80f;
                ss = fmaf(s[j][i], s[j][i], ss);
                am = larger(am, fabsf(s[j][i] * w[j][i]));
            }
        row_reduce<NT>(ss, am, scratch);
        mean = ss / (float)a.h + a.eps * 0x1p80f * 0x1p80f;
        rstd = mean > 0.0f ? 1.0f / sqrtf(mean) : 0.0f;
    }
    const bool in_range = am > 1e-30f && am < INFINITY && ss < INFINITY;
    am *= rstd;
    if (!in_range) {
        // an infinity or NaN in the row or the weight, squares or products past
        // fp32, or no product above its smallest numbers: the maximum is taken
        // of the results themselves
        float none = 0.0f;
        am = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) am = larger(am, fabsf(s[j][i] * rstd * w[j][i]));
        row_reduce<NT>(none, am, scratch);
        if (!(am < INFINITY)) am = NAN;
    }
    // 1 / scale would overflow for a row whose largest |y| is below 448 / 3.4e38:
    // such a row is lifted by 2^64 first
    const float lift = am < 1e-30f ? 0x1p64f : 1.0f;
    const float inv = am > 0.0f ? kE4m3Max / (am * lift) : 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = t + j * NT;
        if (v >= vecs) continue;
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = s[j][i] * rstd * w[j][i];
        if (a.y) st16(a.y + (int64_t)row * a.h + v * 8, pack8(y));
        if (a.q) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = am > 0.0f ? y[i] * lift * inv : 0.0f;
            *reinterpret_cast<uint2 *>(a.q + (int64_t)row * a.h + v * 8) = pack8_e4m3(y);
        }
    }
    if (a.q && t == 0) a.q_scale[row] = am / kE4m3Max;
}

template <int NT, int VPT, int ROWS>
hipError_t go(const NormArgs &a, hipStream_t st) {
    // (a grid's first side times the threads has to stay below 2^32)
    const unsigned blocks = (a.n + ROWS - 1) / ROWS, side = blocks < (1u << 20) ? blocks : 1u << 20;
    rms_norm_kernel<NT, VPT, ROWS><<<dim3(side, (blocks + side - 1) / side), dim3(NT * ROWS), 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs &a, hipStream_t st) {
    const int vecs = a.h / 8;
    if (vecs <= 64) return go<64, 1, 4>(a, st);
    if (vecs <= 128) return go<64, 2, 4>(a, st);
    if (vecs <= 256) return go<256, 1, 1>(a, st);
    if (vecs <= 512) return go<256, 2, 1>(a, st);
    if (vecs <= 1024) return go<512, 2, 1>(a, st);
    if (vecs <= 2048) return go<1024, 2, 1>(a, st);
    return go<1024, 4, 1>(a, st);
}

}  // namespace st
