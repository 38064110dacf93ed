// attend_few.hip -- step_paged_attention for few rows that share keys (single
// tokens being decoded): tiles of up to 16 rows, a row being one query head of
// one token.
//
//     o = sum_j p_j v_j / sum_j p_j,   p_j = 2^(c q k_j - m),   c = scale log2 e
//
// in one pass over the keys with the running maximum m and sum.  Bound by the
// read of keys and values: a wave takes 32 keys at a time, whole rows of the
// cache into registers while the 32 before are computed, and through its own
// part of LDS into the layout of the matrix cores, without a barrier.  The four
// waves of a workgroup take the tiles of 32 keys in turn and their results are
// joined in LDS.  256 tokens over 64 to 4096 keys, 8 key heads of 128: 178 us, 5.7
// TB/s; from 8 bits 103 us, 4.9 TB/s, where the time that a tile costs beside its
// keys counts more (keys for two rounds ahead in registers, and the next tile's
// first keys sent before the end of a tile, changed neither).  One token over 4999
// keys: 17 us, the latency of lengths, pages, keys and the join of 20 pieces.
//
// S^T = K Q^T gives a lane one row of q and 8 of the 32 keys, and p as it lies
// there is the operand that O^T = V^T P^T wants, with the keys of the product
// in the order 4 h .. 4 h + 3, 16 + 4 h .. 16 + 4 h + 3 for the lanes of group
// h = lane / 16; V^T comes from transposed reads of LDS in the same order.
// p is rounded to bf16 for the product (off by at most 2^-8 of itself, as much as the
// result's own rounding, and over several keys less); the sums are fp32 and take
// the p before it.
#include "attend.h"

namespace st {

namespace {

template <int D>
struct FewShared {
    static constexpr int kKeys = 32;
    // (16 bytes between rows of K, 32 between rows of V against bank conflicts)
    static constexpr int kK = 2 * D + 16, kV = 2 * D + 32, kWaveBytes = kKeys * (kK + kV);
    static constexpr int kO = D + 4;  // floats of a row of results
    static_assert(kFewRows * kO * 4 <= kWaveBytes, "a wave's results take the place of its keys");
    char wave[kWaves][kWaveBytes];
    float2 stats[kWaves][kFewRows];  // maximum, sum
    Found found;
    int last;
};

// A row's weighted sum over the waves' results, then out, or on to the next reader.
template <int D>
__device__ __forceinline__ void few_results(const AttendArgs &a, const Walk &w, const TileRows &t, const Piece &p,
                                            const FewShared<D> &sh, bool whole) {
    using Sh = FewShared<D>;
    const Finish finish(a, w.g);
    for (int e = threadIdx.x; e < t.count * (D / 4); e += kThreads) {
        const int r = e / (D / 4), c = e % (D / 4) * 4;
        float m = -INFINITY, l = 0.0f;
        for (int k = 0; k < kWaves; ++k) m = fmaxf(m, sh.stats[k][r].x);
        const float base = base_of(m);
        f32x4_t o = {};
        for (int k = 0; k < kWaves; ++k) {
            const float f = exp2_fast(sh.stats[k][r].x - base);
            l += f * sh.stats[k][r].y;
            o += f * *reinterpret_cast<const f32x4_t *>(sh.wave[k] + (r * Sh::kO + c) * 4);
        }
        if (!whole) {
            float *slot = a.pieces + (int64_t)p.slot * (kFewRows * (D + 2));
            put_pair(slot + r * D + c, o[0], o[1]);
            put_pair(slot + r * D + c + 2, o[2], o[3]);
            if (c == 0) put_pair(slot + kFewRows * D + 2 * r, m, l);
            continue;
        }
        const int row = t.row0 + t.first + r / a.each, head = w.g * a.each + r % a.each, heads = a.kv * a.each;
        const int64_t rh = (int64_t)row * heads + head;
        if (a.state_out) {
            if (c == 0) *reinterpret_cast<float2 *>(a.state_out + 2 * rh) = make_float2(m, l);
            *reinterpret_cast<f32x4_t *>(a.sums_out + rh * D + c) = o;
            continue;
        }
        const float f = finish.factor(l);
        if (c < a.dim)
            *reinterpret_cast<uint2 *>(a.out + row * a.ldo + head * a.dim + c) =
                make_uint2(tl::pack_bf16x2(o[0] * f, o[1] * f), tl::pack_bf16x2(o[2] * f, o[3] * f));
        if (c == 0 && a.lse) a.lse[rh] = finish.log_sum(m, l);
    }
}

// The last workgroup's waves take the pieces in turn, in their order.
template <int D>
__device__ __forceinline__ void few_join(const AttendArgs &a, const Walk &w, const TileRows &t, const Piece &p,
                                         FewShared<D> &sh) {
    using Sh = FewShared<D>;
    const int lane = tl::lane_id(), wave = tl::wave_id();
    for (int e = lane; e < t.count * (D / 4); e += kWave) {
        const int r = e / (D / 4), c = e % (D / 4) * 4;
        float m = -INFINITY, l = 0.0f;
        f32x4_t o = {};
        constexpr int kAt = 8;
        for (int k0 = wave; k0 < p.count; k0 += kWaves * kAt) {
            float2 ml[kAt], lo[kAt], hi[kAt];
#pragma unroll
            for (int u = 0; u < kAt; ++u) {
                const int k = k0 + u * kWaves < p.count ? k0 + u * kWaves : k0;
                const float *slot =
                    a.pieces + (int64_t)piece_slot(w.r, p.first + k, w.at) * (kFewRows * (D + 2));
                ml[u] = get_pair(slot + kFewRows * D + 2 * r);
                lo[u] = get_pair(slot + r * D + c);
                hi[u] = get_pair(slot + r * D + c + 2);
            }
#pragma unroll
            for (int u = 0; u < kAt; ++u) {
                if (k0 + u * kWaves >= p.count) break;
                const float m2 = fmaxf(m, ml[u].x), base = base_of(m2);
                const float f = exp2_fast(m - base), f2 = exp2_fast(ml[u].x - base);
                l = l * f + ml[u].y * f2;
                o = o * f + f32x4_t{lo[u].x, lo[u].y, hi[u].x, hi[u].y} * f2;
                m = m2;
            }
        }
        *reinterpret_cast<f32x4_t *>(sh.wave[wave] + (r * Sh::kO + c) * 4) = o;
        if (c == 0) sh.stats[wave][r] = make_float2(m, l);
    }
}

template <int D, bool F8>
__global__ __launch_bounds__(kThreads, D > 128 ? 1 : D > 64 ? 2 : 3) void attend_few_kernel(AttendArgs a) {
    using Sh = FewShared<D>;
    constexpr int kSize = F8 ? 1 : 2, kKeys = Sh::kKeys;
    constexpr int kLanes = D * kSize / 16, kRows = kWave / kLanes, kLoads = kKeys / kRows;  // lanes of a key; keys of a load
    __shared__ Sh sh;
    Walk w;
    if (!w.find(a, kFewRows, F8 ? kFewFixed8 : kFewFixed, kFewLeast, kFewWhole, sh.found)) return;
    const int lane = tl::lane_id(), wave = scalar(tl::wave_id()), h = lane / 16, r = lane % 16;
    char *const lk = sh.wave[wave], *const lv = lk + kKeys * Sh::kK;
    const int lc = lane % kLanes, lr = lane / kLanes;      // this lane's chunk and row of a load
    const bool in_dim = lc < a.dim * kSize / 16;
    const int64_t chunk = in_dim ? lc * 16 : 0;
    const char *const kc = static_cast<const char *>(a.cache.k), *const vc = static_cast<const char *>(a.cache.v);
    do {
        const int keys = w.keys(a);
        const Piece p = w.piece(keys, kFewStep);
        if (!p.mine) continue;
        const TileRows t(a, w);
        const int32_t *const table = table_of(a, w.j);
        const int64_t head = w.g * a.cache.head_stride * kSize + chunk;
        const char *const kh = kc + head, *const vh = vc + head;
        // this lane's row of q
        const bool live = r < t.count;
        const int token = t.first + (live ? r / a.each : 0);
        const int64_t row = t.row0 + token;
        const int qh = w.g * a.each + (live ? r % a.each : 0);
        const int seen = live ? TileRows::seen(a, w.job.s, token) : 0;
        const int all_see = TileRows::seen(a, w.job.s, t.first);
        u32x4_t q[D / 32];
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk) {
            const int c = 32 * kk + 8 * h;
            q[kk] = live && c < a.dim ? tl::ld16(a.q + row * a.ldq + qh * a.dim + c) : tl::zero4();
        }
        const float cf = exponent_factor(a, w.g);
        float m = -INFINITY, l = 0.0f;
        f32x4_t acc[D / 16] = {};
        if (a.state_in && wave == 0 && p.begins && live) {
            const int64_t rh = row * (a.kv * a.each) + qh;
            const float2 ml = *reinterpret_cast<const float2 *>(a.state_in + 2 * rh);
            m = ml.x;
            l = h == 0 ? ml.y : 0.0f;  // (the sum is one over the four lanes of a row)
            if (m != -INFINITY)
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
                    acc[j] = *reinterpret_cast<const f32x4_t *>(a.sums_in + rh * D + 16 * j + 4 * h);
        }

        // offset of key k0 + lane % 32, its page being known
        auto page_at = [&](int k0) {
            const int key = k0 + lane % 32;
            return key < p.hi ? table[page_of(a.div, key)] : -1;
        };
        auto offset_at = [&](int k0, int page) {
            const int key = k0 + lane % 32;
            return (uint32_t)page < (uint32_t)a.cache.pages
                       ? (int64_t)token_offset(a, page, key - page_of(a.div, key) * a.cache.page)
                       : -1;
        };
        u32x4_t kr[kLoads], vr[kLoads];
        uint32_t there = 0;  // keys of the 32 in registers that are in the cache
        auto start = [&](int64_t off) {
            there = (uint32_t)__ballot(off >= 0);
            const int64_t at = off >= 0 ? off : 0;
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const int64_t o = __shfl((long long)at, u * kRows + lr);
                kr[u] = tl::ld16_stream(kh + o);
                vr[u] = tl::ld16_stream(vh + o);
            }
        };
        const int k_first = p.lo + wave * kKeys;
        constexpr int kNext = kWaves * kKeys;
        if (k_first < p.hi) start(offset_at(k_first, page_at(k_first)));
        int page_next = page_at(k_first + kNext);
#pragma unroll 1
        for (int k0 = k_first; k0 < p.hi; k0 += kNext) {
            const uint32_t ok = (uint32_t)scalar((int)there);
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const int key = u * kRows + lr;
                if (!in_dim) kr[u] = tl::zero4();
                // (values of absent keys meet p = 0, which an infinity or NaN there would turn into NaN)
                if (ok != ~0u && !((ok >> key) & 1)) vr[u] = tl::zero4();
                char *const ks = lk + key * Sh::kK, *const vs = lv + key * Sh::kV;
                if constexpr (F8) {
                    // (some lanes' second half first, so that 8 lanes' 16 bytes fall on different banks)
                    const bool swap_v = lane & 4, swap_k = swap_v && D > 64;
                    auto put = [&](char *to, const u32x4_t x, bool swap) {
                        const int first = lc * 32 + (swap ? 16 : 0), second = lc * 32 + (swap ? 0 : 16);
                        tl::st16(to + first, widen8(swap ? x.z : x.x, swap ? x.w : x.y));
                        tl::st16(to + second, widen8(swap ? x.x : x.z, swap ? x.y : x.w));
                    };
                    put(ks, kr[u], swap_k);
                    put(vs, vr[u], swap_v);
                } else {
                    tl::st16(ks + lc * 16, kr[u]);
                    tl::st16(vs + lc * 16, vr[u]);
                }
            }
            // (rows that see different keys)
            bool broken = false;
            if (k0 + kKeys > all_see && all_see < keys) {
#pragma unroll
                for (int u = 0; u < kLoads; ++u) {
                    if constexpr (F8)
                        broken |= not_finite(widen8(vr[u].x, vr[u].y)) || not_finite(widen8(vr[u].z, vr[u].w));
                    else
                        broken |= not_finite(vr[u]);
                }
                broken = __any(broken);
            }
            if (k0 + kNext < p.hi) start(offset_at(k0 + kNext, page_next));
            page_next = page_at(k0 + 2 * kNext);
            wave_sync();

            f32x4_t s[2];
#pragma unroll
            for (int kt = 0; kt < 2; ++kt) {
                s[kt] = f32x4_t{};
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk)
                    s[kt] = tl::mfma_16x16x32(tl::ld16(lk + (16 * kt + r) * Sh::kK + 64 * kk + 16 * h), q[kk], s[kt]);
            }
            if (ok != ~0u || k0 + kKeys > all_see) {
#pragma unroll
                for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = 16 * kt + 4 * h + i;
                        if (k0 + key >= seen || !((ok >> key) & 1)) s[kt][i] = -INFINITY;
                    }
            }
            float big = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                              fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
            big = fmaxf(big, __shfl_xor(big, 16));
            big = fmaxf(big, __shfl_xor(big, 32));
            const float m2 = fmaxf(m, big * cf), base = base_of(m2), f = exp2_fast(m - base);
            m = m2;
            l *= f;
            float pr[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                pr[i] = exp2_fast(fmaf(s[i / 4][i % 4], cf, -base));
                l += pr[i];
            }
            const u32x4_t pk = {tl::pack_bf16x2(pr[0], pr[1]), tl::pack_bf16x2(pr[2], pr[3]),
                                tl::pack_bf16x2(pr[4], pr[5]), tl::pack_bf16x2(pr[6], pr[7])};
            const char *const vt = lv + (4 * h + r / 4) * Sh::kV + r % 4 * 8;
            auto add = [&](auto care) {
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    acc[j] *= f;
                    const uint2 lo = read_transposed(vt + 32 * j), hi = read_transposed(vt + 16 * Sh::kV + 32 * j);
                    u32x4_t v = {lo.x, lo.y, hi.x, hi.y};
                    if constexpr (decltype(care)::value)
                        for (int e = 0; e < 4; ++e) v[e] = drop_not_finite(v[e]);
                    acc[j] = tl::mfma_16x16x32(v, pk, acc[j]);
                }
            };
            if (!broken) {
                add(std::false_type{});
            } else {
                add(std::true_type{});
#pragma unroll 1
                for (int key = 0; key < kKeys; ++key)
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        float x[4] = {};
                        add_not_finite(x, *reinterpret_cast<const uint2 *>(lv + key * Sh::kV + 32 * j + 8 * h),
                                       k0 + key < seen);
                        acc[j] += f32x4_t{x[0], x[1], x[2], x[3]};
                    }
            }
            wave_sync();
        }
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
        wave_sync();
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
            *reinterpret_cast<f32x4_t *>(sh.wave[wave] + (r * Sh::kO + 16 * j + 4 * h) * 4) = acc[j];
        if (h == 0) sh.stats[wave][r] = make_float2(m, l);
        __syncthreads();
        few_results<D>(a, w, t, p, sh, !p.split);
        if (p.split && last_of(a, p, &sh.last)) {
            few_join<D>(a, w, t, p, sh);
            __syncthreads();
            few_results<D>(a, w, t, p, sh, true);
        }
        __syncthreads();
    } while (w.next(a));
}

template <int D>
hipError_t go(const AttendArgs &a, hipStream_t st) {
    const dim3 grid(a.groups_of_threads), block(kThreads);
    if (a.cache.k_scale)
        attend_few_kernel<D, true><<<grid, block, 0, st>>>(a);
    else
        attend_few_kernel<D, false><<<grid, block, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attend_few(const AttendArgs &a, hipStream_t st) {
    switch (padded_dim(a.dim)) {
        case 64: return go<64>(a, st);
        case 128: return go<128>(a, st);
        default: return go<256>(a, st);
    }
}

}  // namespace st
