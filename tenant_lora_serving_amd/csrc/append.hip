// append.hip -- step_kv_append: new tokens' keys and values into the paged
// cache, keys and queries turned by their positions' angles on the way.
//
//     pair (a, b) at angle t -> (a cos t - b sin t, b cos t + a sin t)
//
// in fp32, rounded once to bf16 or, over the head's scale, to e4m3.  A thread
// takes one unit: 16 bytes of a head, or the two 16 bytes whose halves pair up,
// so q may be turned in place.  Bound by memory traffic for many tokens (6947 with
// 32 query and 8 key heads of 128: 41 us, 4.2 TB/s) and by latency for few (one
// token: 3 us, and 10 more of host time).
#include "attend_kernels.h"
#include "common.h"

namespace st {

using tl::u32x4_t;

namespace {

constexpr int kThreads = 256;
constexpr float kE4m3Max = 448.0f;

__device__ __forceinline__ void unpack8(const u32x4_t v, float *f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = tl::bf_lo(v[i]), f[2 * i + 1] = tl::bf_hi(v[i]);
}
__device__ __forceinline__ u32x4_t pack8(const float *f) {
    return u32x4_t{tl::pack_bf16x2(f[0], f[1]), tl::pack_bf16x2(f[2], f[3]), tl::pack_bf16x2(f[4], f[5]),
                   tl::pack_bf16x2(f[6], f[7])};
}
// Into e4m3's range; a NaN stays one.
__device__ __forceinline__ float saturate(float v) {
    return v > kE4m3Max ? kE4m3Max : v < -kE4m3Max ? -kE4m3Max : v;
}
// Eight values over a scale as e4m3, round to nearest even.  (Divided, not
// multiplied by 1 / scale: that rounds twice and moves values across the border
// between two neighbours.  A 0 over a scale of 0, that of a head which held only
// zeros, stays a 0.)
__device__ __forceinline__ uint2 pack8_e4m3(const float *f, float scale) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = f[i] == 0.0f && scale == 0.0f ? f[i] : saturate(f[i] / scale);
    int a = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], a, true);
    int b = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], b, true);
    return make_uint2((uint32_t)a, (uint32_t)b);
}
__device__ __forceinline__ void load8(const float *p, float *f) {
    const u32x4_t a = tl::ld16(p), b = tl::ld16(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(a[i]), f[4 + i] = __uint_as_float(b[i]);
}

// Units of a turned head and of one copied.
__host__ __device__ inline int turned_units(const AppendArgs &a) {
    return a.neighbours ? a.dim / 8 : a.rot / 16 + (a.dim - a.rot) / 8;
}
__host__ __device__ inline int token_units(const AppendArgs &a) {
    return ((a.q ? a.heads : 0) + a.kv) * turned_units(a) + a.kv * (a.dim / 8);
}

// `tokens` tokens a workgroup, or one token's units over gridDim.y workgroups.
__global__ __launch_bounds__(kThreads) void append_kernel(AppendArgs a, int tokens) {
    const int per_head = turned_units(a), per_token = token_units(a), copied = a.dim / 8;
    const int q_units = a.q ? a.heads * per_head : 0, k_units = a.kv * per_head;
    const int t0 = blockIdx.x * tokens, count = min(tokens, a.n - t0) * per_token;
    for (int e = blockIdx.y * kThreads + threadIdx.x; e < count; e += gridDim.y * kThreads) {
        const int t = t0 + e / per_token;
        int u = e % per_token;
        // where the unit comes from
        const uint16_t *from;
        int head, at, which;  // at: the unit's first column; which: 0 q, 1 k, 2 v
        bool turn = false, pair = false;
        if (u < q_units + k_units) {
            which = u < q_units ? 0 : 1;
            if (which) u -= q_units;
            head = u / per_head;
            u %= per_head;
            turn = a.neighbours ? 8 * u < a.rot : u < a.rot / 16;
            pair = turn && !a.neighbours;
            at = a.neighbours || turn ? 8 * u : a.rot + 8 * (u - a.rot / 16);
            from = which ? a.k + t * a.ldk : a.q + t * a.ldq;
        } else {
            u -= q_units + k_units;
            which = 2;
            head = u / copied;
            at = u % copied * 8;
            from = a.v + t * a.ldv;
        }
        from += head * a.dim + at;
        // (a position outside the table: q is NaN, and nothing goes into the cache)
        int position = 0;
        bool known = true;
        if (a.rot) {
            position = a.positions[t];
            known = (uint32_t)position < (uint32_t)a.positions_end;
        }
        int place = -1;
        if (which) {
            place = a.place[t];
            if (!known || place < 0 || place / a.cache.page >= a.cache.pages) continue;
        }
        float x[8], y[8];
        const int half = a.rot / 2;
        unpack8(tl::ld16(from), x);
        if (pair) unpack8(tl::ld16(from + half), y);
        if (turn && known) {
            const float *row = a.rotation + (int64_t)position * a.rot;
            if (pair) {
                float c[8], s[8];
                load8(row + at, c);
                load8(row + half + at, s);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p = x[i], q = y[i];
                    x[i] = p * c[i] - q * s[i];
                    y[i] = q * c[i] + p * s[i];
                }
            } else {
                const u32x4_t c = tl::ld16(row + at / 2), s = tl::ld16(row + half + at / 2);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p = x[2 * i], q = x[2 * i + 1];
                    const float cos = __uint_as_float(c[i]), sin = __uint_as_float(s[i]);
                    x[2 * i] = p * cos - q * sin;
                    x[2 * i + 1] = q * cos + p * sin;
                }
            }
        }
        if (which == 0) {
            if (!known)
                for (int i = 0; i < 8; ++i) x[i] = y[i] = NAN;
            uint16_t *to = a.q_out + t * a.ldo + head * a.dim + at;
            tl::st16(to, pack8(x));
            if (pair) tl::st16(to + half, pack8(y));
            continue;
        }
        const int64_t to = place / a.cache.page * a.cache.page_stride + place % a.cache.page * a.cache.token_stride +
                           head * a.cache.head_stride + at;
        void *const cache = which == 1 ? a.cache.k : a.cache.v;
        if (a.cache.k_scale) {
            const float scale = (which == 1 ? a.cache.k_scale : a.cache.v_scale)[head];
            uint8_t *p = static_cast<uint8_t *>(cache) + to;
            *reinterpret_cast<uint2 *>(p) = pack8_e4m3(x, scale);
            if (pair) *reinterpret_cast<uint2 *>(p + half) = pack8_e4m3(y, scale);
        } else {
            uint16_t *p = static_cast<uint16_t *>(cache) + to;
            tl::st16(p, pack8(x));
            if (pair) tl::st16(p + half, pack8(y));
        }
    }
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs &a, hipStream_t st) {
    const int units = token_units(a), blocks = (units + kThreads - 1) / kThreads;
    // a workgroup a token or, of a few small ones, up to 1024 units, once there are enough to fill the chip
    int tokens = 1;
    while (tokens * units < 1024 && a.n / tokens > 4096) tokens *= 2;
    const bool many = a.n > 2048;
    append_kernel<<<dim3((a.n + tokens - 1) / tokens, many ? 1 : blocks), dim3(kThreads), 0, st>>>(a, tokens);
    return hipGetLastError();
}

}  // namespace st
