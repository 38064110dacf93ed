// attend_many.hip -- step_paged_attention for many rows that share keys
// (prompts, pieces of prompts, the requests of a shared prefix, queries to an
// encoder's states): tiles of up to 128 rows, a row being one query head of one
// token, by 64 keys.
//
//     o = sum_j p_j v_j / sum_j p_j,   p_j = 2^(c q k_j - m),   c = scale log2 e
//
// in one pass over the keys with the running maximum m and sum.  Bound by the
// matrix cores and the exponentials.  Each of the four waves holds 32 rows; all
// read the keys and values from LDS, two buffers in turn, the next 64 keys on
// their way through registers meanwhile, one barrier a round.
//
// S^T = K Q^T gives a lane one row of q and half of the keys, and p as it lies
// there is the operand that O^T = V^T P^T wants, with the keys of the product
// in the order 4 h .. 4 h + 3, 8 + 4 h .. 8 + 4 h + 3 of 16 for the lanes of half h;
// V^T comes from transposed reads of LDS in the same order.  A row's maximum
// and sum are so one number a lane, and p never leaves its registers.  p is
// rounded to bf16 for the product (off by at most 2^-8 of itself, as much as the
// result's own rounding, and over several keys less); the sums are fp32 and
// take the p before it.
#include "attend.h"

namespace st {

namespace {

typedef float f32x16_t __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16_t mfma_32x32x16(const u32x4_t a, const u32x4_t b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(tl::bf16x8_t, a),
                                                   __builtin_bit_cast(tl::bf16x8_t, b), c, 0, 0, 0);
}

constexpr int kKeys = kManyStep;
template <int D>
struct ManyShared {
    // (16 bytes between rows of K, 32 between rows of V against bank conflicts)
    static constexpr int kK = 2 * D + 16, kV = 2 * D + 32;
    char k[2][kKeys * kK], v[2][kKeys * kV];
    uint64_t there[2][kWaves];  // keys that are in the cache
    int broken[2];              // 1 + the first key of a tile with values that are not finite
    Found found;
    int last;
};

// What a lane holds of its row: maximum, sum (of its half of the keys on the
// way), and columns 32 j + 8 (i / 4) + 4 h + i % 4 of the weighted sum.
template <int D>
struct RowState {
    float m, l;
    f32x16_t o[D / 32];
};

template <int D>
__device__ __forceinline__ void many_results(const AttendArgs &a, const Walk &w, const RowState<D> &x, int64_t row,
                                             int qh, int h) {
    const int64_t rh = row * (a.kv * a.each) + qh;
    if (a.state_out) {
        if (h == 0) *reinterpret_cast<float2 *>(a.state_out + 2 * rh) = make_float2(x.m, x.l);
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<f32x4_t *>(a.sums_out + rh * D + 32 * j + 8 * i + 4 * h) =
                    f32x4_t{x.o[j][4 * i], x.o[j][4 * i + 1], x.o[j][4 * i + 2], x.o[j][4 * i + 3]};
        return;
    }
    const float vs = a.cache.v_scale ? a.cache.v_scale[w.g] : 1.0f, f = x.l == 0.0f ? 0.0f : vs / x.l;
    uint16_t *const to = a.out + row * a.ldo + qh * a.dim;
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = 32 * j + 8 * i + 4 * h;
            if (c < a.dim)
                *reinterpret_cast<uint2 *>(to + c) =
                    make_uint2(tl::pack_bf16x2(x.o[j][4 * i] * f, x.o[j][4 * i + 1] * f),
                               tl::pack_bf16x2(x.o[j][4 * i + 2] * f, x.o[j][4 * i + 3] * f));
        }
    if (h == 0 && a.lse) a.lse[rh] = x.l == 0.0f ? -INFINITY : (base_of(x.m) + log2f(x.l)) * kLn2;
}

// Pieces' results lie as the lanes hold them.
template <int D>
__device__ __forceinline__ float *piece_sums(const AttendArgs &a, int slot, int wave, int pair) {
    return a.pieces + (int64_t)slot * (kManyRows * (D + 2)) + ((wave * (D / 4) + pair) * kWave + tl::lane_id()) * 2;
}
template <int D>
__device__ __forceinline__ float *piece_stats(const AttendArgs &a, int slot, int wave) {
    return a.pieces + (int64_t)slot * (kManyRows * (D + 2)) + kManyRows * D + (wave * 32 + tl::lane_id() % 32) * 2;
}

template <int D, bool F8>
__global__ __launch_bounds__(kThreads, D > 128 ? 1 : 2) void attend_many_kernel(AttendArgs a) {
    using Sh = ManyShared<D>;
    constexpr int kSize = F8 ? 1 : 2;
    constexpr int kLanes = D * kSize / 16, kRows = kThreads / kLanes, kLoads = kKeys / kRows;  // of a key; keys of a load
    __shared__ Sh sh;
    Walk w;
    if (threadIdx.x < 2) sh.broken[threadIdx.x] = 0;
    if (!w.find(a, kManyRows, kManyLeast, kManyWhole, sh.found)) return;
    const int tid = threadIdx.x, lane = tl::lane_id(), wave = scalar(tl::wave_id()), h = lane / 32;
    const int lc = tid % kLanes, lr = tid / kLanes;  // this thread's chunk and key of a load
    const bool in_dim = lc < a.dim * kSize / 16;
    const int64_t chunk = in_dim ? lc * 16 : 0;
    const char *const kc = static_cast<const char *>(a.cache.k), *const vc = static_cast<const char *>(a.cache.v);
    do {
        const int keys = w.keys(a);
        const Piece p = piece_of(w.r, w.w, w.at, keys, kManyStep);
        if (!p.mine) continue;
        const TileRows t(a, w);
        const int32_t *const table = table_of(a, w.j);
        const int64_t head = w.g * a.cache.head_stride * kSize + chunk;
        const char *const kh = kc + head, *const vh = vc + head;
        // this lane's row of q
        const int r = wave * 32 + lane % 32, r_first = wave * 32, r_last = min(r_first + 31, t.count - 1);
        const bool live = r < t.count, any = r_first < t.count;
        const int token = t.first + (live ? r / a.each : 0);
        const int64_t row = t.row0 + token;
        const int qh = w.g * a.each + (live ? r % a.each : 0);
        const int seen = live ? TileRows::seen(a, w.job.s, token) : 0;
        const int all_see = TileRows::seen(a, w.job.s, t.first);  // the tile's rows
        const int wave_sees = any ? TileRows::seen(a, w.job.s, t.first + r_last / a.each) : 0;
        const int wave_all_see = TileRows::seen(a, w.job.s, t.first + r_first / a.each);
        u32x4_t q[D / 16];
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const int c = 16 * kk + 8 * h;
            q[kk] = live && c < a.dim ? tl::ld16(a.q + row * a.ldq + qh * a.dim + c) : tl::zero4();
        }
        // (a scale of 0, of a head that is all zeros, must not meet the masks' infinity)
        const float cf = fmaxf(a.scale * (F8 ? a.cache.k_scale[w.g] : 1.0f), 1e-30f);
        RowState<D> x;
        x.m = -INFINITY;
        x.l = 0.0f;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) x.o[j] = f32x16_t{};
        if (a.state_in && p.begins && live) {
            const int64_t rh = row * (a.kv * a.each) + qh;
            const float2 ml = *reinterpret_cast<const float2 *>(a.state_in + 2 * rh);
            x.m = ml.x;
            x.l = h == 0 ? ml.y : 0.0f;  // (the sum is one over the two lanes of a row)
            if (x.m != -INFINITY)
#pragma unroll
                for (int j = 0; j < D / 32; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const f32x4_t o = *reinterpret_cast<const f32x4_t *>(a.sums_in + rh * D + 32 * j + 8 * i + 4 * h);
                        for (int e = 0; e < 4; ++e) x.o[j][4 * i + e] = o[e];
                    }
        }

        u32x4_t kr[kLoads], vr[kLoads];
        int page[kLoads];
        bool there[kLoads];
        auto pages = [&](int k0) {
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const int key = k0 + u * kRows + lr;
                page[u] = key < p.hi ? table[page_of(a.div, key)] : -1;
            }
        };
        auto start = [&](int k0) {
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const int key = k0 + u * kRows + lr;
                const int64_t off = token_offset<kSize>(a, page[u], key - page_of(a.div, key) * a.cache.page);
                there[u] = off >= 0;
                const int64_t o = off >= 0 ? off : 0;
                kr[u] = tl::ld16(kh + o);
                vr[u] = tl::ld16(vh + o);
            }
        };
        auto store = [&](int k0, int buf) {
            bool broken = false;
            uint64_t ok = 0;
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const int key = u * kRows + lr;
                if (!in_dim) kr[u] = tl::zero4();
                // (values of absent keys meet p = 0, which an infinity or NaN there would turn into NaN)
                if (!there[u]) vr[u] = tl::zero4();
                // one bit a key, from the first of its lanes
                uint64_t bits = __ballot(there[u]);
                constexpr int kOfWave = kWave / kLanes;  // keys of a wave's load
                uint64_t mine = 0;
#pragma unroll
                for (int e = 0; e < kOfWave; ++e) mine |= ((bits >> (e * kLanes)) & 1) << e;
                ok |= mine << (u * kRows + wave * kOfWave);
                char *const ks = sh.k[buf] + key * Sh::kK, *const vs = sh.v[buf] + key * Sh::kV;
                if constexpr (F8) {
                    const u32x4_t v0 = widen8(vr[u].x, vr[u].y), v1 = widen8(vr[u].z, vr[u].w);
                    tl::st16(ks + lc * 32, widen8(kr[u].x, kr[u].y));
                    tl::st16(ks + lc * 32 + 16, widen8(kr[u].z, kr[u].w));
                    tl::st16(vs + lc * 32, v0);
                    tl::st16(vs + lc * 32 + 16, v1);
                    if (k0 + kKeys > all_see) broken |= not_finite(v0) || not_finite(v1);
                } else {
                    tl::st16(ks + lc * 16, kr[u]);
                    tl::st16(vs + lc * 16, vr[u]);
                    if (k0 + kKeys > all_see) broken |= not_finite(vr[u]);
                }
            }
            if (lane == 0) sh.there[buf][wave] = ok;
            if (broken) sh.broken[buf] = k0 + 1;
        };
        if (p.lo < p.hi) {
            pages(p.lo);
            start(p.lo);
            pages(p.lo + kKeys);
            store(p.lo, 0);
            __syncthreads();
        }
        int buf = 0;
#pragma unroll 1
        for (int k0 = p.lo; k0 < p.hi; k0 += kKeys, buf ^= 1) {
            if (k0 + kKeys < p.hi) {
                start(k0 + kKeys);
                pages(k0 + 2 * kKeys);
            }
            if (any && k0 < wave_sees) {
                const char *const lk = sh.k[buf] + (lane % 32) * Sh::kK + 16 * h;
                f32x16_t s[2];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    s[b] = f32x16_t{};
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        s[b] = mfma_32x32x16(tl::ld16(lk + 32 * b * Sh::kK + 32 * kk), q[kk], s[b]);
                }
                uint64_t ok = 0;
                for (int k = 0; k < kWaves; ++k) ok |= sh.there[buf][k];
                if (k0 + kKeys > wave_all_see || ok != ~0ull) {
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int key = 32 * b + 8 * (i / 4) + 4 * h + i % 4;
                            if (k0 + key >= seen || !((ok >> key) & 1)) s[b][i] = -INFINITY;
                        }
                }
                float big = -INFINITY;
#pragma unroll
                for (int i = 0; i < 16; ++i) big = fmaxf(big, fmaxf(s[0][i], s[1][i]));
                big = fmaxf(big, __shfl_xor(big, 32));
                const float m2 = fmaxf(x.m, big * cf), base = base_of(m2), f = exp2_fast(x.m - base);
                x.m = m2;
                x.l *= f;
                u32x4_t pk[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {  // 16 keys each
                    float pr[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        pr[i] = exp2_fast(fmaf(s[c / 2][8 * (c % 2) + i], cf, -base));
                        x.l += pr[i];
                    }
                    pk[c] = u32x4_t{tl::pack_bf16x2(pr[0], pr[1]), tl::pack_bf16x2(pr[2], pr[3]),
                                    tl::pack_bf16x2(pr[4], pr[5]), tl::pack_bf16x2(pr[6], pr[7])};
                }
                const char *const lv =
                    sh.v[buf] + (4 * h + lane % 16 / 4) * Sh::kV + (lane / 16 % 2) * 32 + lane % 4 * 8;
                auto add = [&](auto care) {
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) {
                        x.o[j] *= f;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint2 lo = read_transposed(lv + 16 * c * Sh::kV + 64 * j),
                                        hi = read_transposed(lv + (16 * c + 8) * Sh::kV + 64 * j);
                            u32x4_t v = {lo.x, lo.y, hi.x, hi.y};
                            if constexpr (decltype(care)::value)
                                for (int e = 0; e < 4; ++e) v[e] = drop_not_finite(v[e]);
                            x.o[j] = mfma_32x32x16(v, pk[c], x.o[j]);
                        }
                    }
                };
                if (scalar(sh.broken[buf]) != k0 + 1) {
                    add(std::false_type{});
                } else {
                    add(std::true_type{});
#pragma unroll 1
                    for (int key = 0; key < kKeys; ++key)
#pragma unroll
                        for (int j = 0; j < D / 32; ++j)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                add_not_finite(reinterpret_cast<float *>(&x.o[j]) + 4 * i,
                                               *reinterpret_cast<const uint2 *>(sh.v[buf] + key * Sh::kV + 64 * j +
                                                                                16 * i + 8 * h),
                                               k0 + key < seen);
                }
            }
            if (k0 + kKeys < p.hi) store(k0 + kKeys, buf ^ 1);
            __syncthreads();
        }
        x.l += __shfl_xor(x.l, 32);
        if (!p.split) {
            if (live) many_results<D>(a, w, x, row, qh, h);
        } else {
            if (any) {
#pragma unroll
                for (int j = 0; j < D / 32; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        put_pair(piece_sums<D>(a, p.slot, wave, 8 * j + i), x.o[j][2 * i], x.o[j][2 * i + 1]);
                if (h == 0) put_pair(piece_stats<D>(a, p.slot, wave), x.m, x.l);
            }
            if (last_of(a, p, &sh.last) && any) {
                x.m = -INFINITY;
                x.l = 0.0f;
#pragma unroll
                for (int j = 0; j < D / 32; ++j) x.o[j] = f32x16_t{};
#pragma unroll 1
                for (int k = 0; k < p.count; ++k) {  // in their order
                    const int slot = piece_slot(w.r, p.first + k, w.at);
                    const float2 ml = get_pair(piece_stats<D>(a, slot, wave));
                    const float m2 = fmaxf(x.m, ml.x), base = base_of(m2);
                    const float f = exp2_fast(x.m - base), f2 = exp2_fast(ml.x - base);
                    x.m = m2;
                    x.l = x.l * f + ml.y * f2;
#pragma unroll
                    for (int j = 0; j < D / 32; ++j)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 o = get_pair(piece_sums<D>(a, slot, wave, 8 * j + i));
                            x.o[j][2 * i] = x.o[j][2 * i] * f + o.x * f2;
                            x.o[j][2 * i + 1] = x.o[j][2 * i + 1] * f + o.y * f2;
                        }
                }
                if (live) many_results<D>(a, w, x, row, qh, h);
            }
        }
        if (tid < 2) sh.broken[tid] = 0;
        __syncthreads();
    } while (w.next(a));
}

template <int D>
hipError_t go(const AttendArgs &a, hipStream_t st) {
    const dim3 grid(a.groups_of_threads), block(kThreads);
    if (a.cache.k_scale)
        attend_many_kernel<D, true><<<grid, block, 0, st>>>(a);
    else
        attend_many_kernel<D, false><<<grid, block, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attend_many(const AttendArgs &a, hipStream_t st) {
    switch (padded_dim(a.dim)) {
        case 64: return go<64>(a, st);
        case 128: return go<128>(a, st);
        default: return go<256>(a, st);
    }
}

}  // namespace st
