// attend_many.hip -- step_paged_attention for many rows that share keys
// (prompts, pieces of prompts, the requests of a shared prefix, queries to an
// encoder's states): tiles of up to 128 rows, a row being one query head of one
// token, by 64 keys.
//
//     o = sum_j p_j v_j / sum_j p_j,   p_j = 2^(c q k_j - m),   c = scale log2 e
//
// in one pass over the keys with the running maximum m and sum.  Bound by the
// matrix cores, the exponentials and LDS reads.  Each of the four waves holds 32
// rows; all read the keys and values from LDS, two buffers in turn, the next 64
// keys on their way meanwhile, one barrier a round.  2048 rows of 4 requests over
// 4000 to 24000 keys, 32 heads of 128: 712 us in all, 0.8 PFLOP/s, matrix
// instructions busy 50% of the cycles and vector ones 53%, waves waiting 26% of
// their time; whole prompts of 6947 rows: 144 us, of
// which 14 join pieces.
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

constexpr int kKeys = kManyStep, kHalf = kKeys / 2;
constexpr int kWaitLoads = 0x0f70;  // s_waitcnt vmcnt(0)
// The larger of two, NaN if one is (v_maximum3_f32; fmaxf takes a step more for each).
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }
// The larger of a lane's value and that of the lane 32 away.
__device__ __forceinline__ float larger_of_halves(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return larger(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
// Rows of keys lie side by side, 16-byte chunk c of key j at place c ^ k_turn(j)
// or c ^ v_turn(j): 16 keys' reads of one chunk of K, and 4 keys' reads of 64
// bytes of V, then fall on different banks.
template <int D>
struct ManyShared {
    static constexpr int kRow = 2 * D;
    char k[2][kKeys * kRow], v[2][kKeys * kRow];
    uint64_t absent[2][kWaves];  // keys whose page the cache does not have (when careful)
    Found found;
    int again;
    static __device__ __forceinline__ int k_turn(int key) { return key & (D == 64 ? 7 : 15); }
    static __device__ __forceinline__ int v_turn(int key) {
        return D == 64 ? (key & 2) << 1 : (key & 3) << 2 | (key & 4) >> 1;
    }
};

// 16 bytes a lane from memory into LDS at `lds` + 16 * lane.  There is no
// register result, so what is written is m0 (the LDS address) and LDS, which
// "memory" covers; the wait is written out where the data is needed.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_lds(const char *p, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"(lds), "v"(p) : "m0", "memory");
}
// The same from `base` (of the wave) + `off` (of the lane).
__device__ __forceinline__ void load_lds(const char *base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(off), "s"(base)
                 : "m0", "memory");
}
#pragma clang diagnostic pop
__device__ __forceinline__ uint32_t lds_address(const char *p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char *)p;
}

// What a lane holds of its row: maximum, sum (of its half of the keys on the
// way), and columns 32 j + 8 (i / 4) + 4 h + i % 4 of the weighted sum.
template <int D>
struct RowState {
    float m, l;
    f32x16_t o[D / 32];
};

// Four columns of a row's result, or of what it leaves for its next keys.
__device__ __forceinline__ void put_columns(const AttendArgs &a, int64_t row, int qh, int dim, int c, float f,
                                            const f32x4_t o) {
    if (a.sums_out)
        *reinterpret_cast<f32x4_t *>(a.sums_out + (row * (a.kv * a.each) + qh) * dim + c) = o;
    else if (c < a.dim)
        *reinterpret_cast<uint2 *>(a.out + row * a.ldo + qh * a.dim + c) =
            make_uint2(tl::pack_bf16x2(o[0] * f, o[1] * f), tl::pack_bf16x2(o[2] * f, o[3] * f));
}
__device__ __forceinline__ void put_stats(const AttendArgs &a, int64_t row, int qh, const Finish &finish, float m, float l) {
    const int64_t rh = row * (a.kv * a.each) + qh;
    if (a.state_out)
        *reinterpret_cast<float2 *>(a.state_out + 2 * rh) = make_float2(m, l);
    else if (a.lse)
        a.lse[rh] = finish.log_sum(m, l);
}

// Pieces' results lie as the lanes hold them: pair i of a lane's columns, then the rows' maxima and sums.
template <int D>
__device__ __forceinline__ float2 *piece_sums(const AttendArgs &a, int slot, int wave, int pair) {
    return reinterpret_cast<float2 *>(a.pieces + (int64_t)slot * (kManyRows * (D + 2))) +
           (wave * (D / 4) + pair) * kWave + tl::lane_id();
}
template <int D>
__device__ __forceinline__ float2 *piece_stats(const AttendArgs &a, int slot, int wave) {
    return reinterpret_cast<float2 *>(a.pieces + (int64_t)slot * (kManyRows * (D + 2)) + kManyRows * D) + wave * 32 +
           tl::lane_id() % 32;
}

// Even: pages hold whole groups of the keys that a load instruction takes, so
// that a place is worked out for each group, not by every lane for its key.
template <int D, bool F8>
constexpr int kKeysOfLoad = kWave * 16 / (D * (F8 ? 1 : 2));
template <int D, bool F8, bool Even>
__global__ __launch_bounds__(kThreads, D > 128 ? 1 : 2) void attend_many_kernel(AttendArgs a) {
    using Sh = ManyShared<D>;
    constexpr int kSize = F8 ? 1 : 2;
    constexpr int kLanes = D * kSize / 16, kOfWave = kKeysOfLoad<D, F8>;  // lanes of a key; keys of a wave's load
    constexpr int kLoads = kKeys / (kWaves * kOfWave);
    __shared__ Sh sh;
    Walk w;
    if (threadIdx.x == 0) a.joins[workgroup_of(a)].pieces = 0;
    if (!w.find(a, kManyRows, kManyFixed, kManyLeast, kManyWhole, sh.found)) return;
    const int lane = tl::lane_id(), wave = scalar(tl::wave_id()), h = lane / 32;
    // this lane's key of load u is (u * kWaves + wave) * kOfWave + lr
    const int lc = lane % kLanes, lr = lane / kLanes;
    auto key_of = [&](int u) { return (u * kWaves + wave) * kOfWave + lr; };
    const uint32_t from = lr * a.token_units * 16;  // (used where the keys of a load are on one page)
    const char *const kc = static_cast<const char *>(a.cache.k), *const vc = static_cast<const char *>(a.cache.v);
    do {
        const int keys = w.keys(a);
        const Piece p = w.piece(keys, kManyStep);
        if (!p.mine) continue;
        const TileRows t(a, w);
        const int32_t *const table = table_of(a, w.j);
        const int64_t head = w.g * a.cache.head_stride * kSize;
        const char *const kh = kc + head, *const vh = vc + head;
        // this lane's row of q
        const int r = wave * 32 + lane % 32, r_first = wave * 32, r_last = min(r_first + 31, t.count - 1);
        const bool live = r < t.count, any = r_first < t.count;
        const int token = t.first + (live ? r / a.each : 0);
        const int64_t row = t.row0 + token;
        const int qh = w.g * a.each + (live ? r % a.each : 0);
        const int seen = live ? TileRows::seen(a, w.job.s, token) : 0;
        // the keys that some of the wave's rows see, and that all rows of the tile do
        const int wave_sees = scalar(any ? TileRows::seen(a, w.job.s, t.first + r_last / a.each) : 0);
        const int tile_all_see = scalar(TileRows::seen(a, w.job.s, t.first));
        u32x4_t q[D / 16];
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const int c = 16 * kk + 8 * h;
            q[kk] = live && c < a.dim ? tl::ld16(a.q + row * a.ldq + qh * a.dim + c) : tl::zero4();
        }
        const float cf = exponent_factor(a, w.g);
        RowState<D> x;
        // The piece's keys.  The quick way leaves out two things that hardly ever
        // happen, keys on pages that the cache does not have and, among the values of
        // keys that some rows must not see, infinities and NaN, which p = 0 turns into
        // NaN; it returns whether it met one, and then all is done again carefully.
        auto attend = [&](auto careful) {
            constexpr bool kCareful = decltype(careful)::value, kQuick = Even && !kCareful;
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
                            const f32x4_t o =
                                *reinterpret_cast<const f32x4_t *>(a.sums_in + rh * D + 32 * j + 8 * i + 4 * h);
                            for (int e = 0; e < 4; ++e) x.o[j][4 * i + e] = o[e];
                        }
            }
            bool met = false;
            u32x4_t kr[F8 ? kLoads : 1], vr[F8 ? kLoads : 1];
            // Round k0 sends for V's keys k0 + 64 .. and K's k0 + 96 ..; their pages are looked up
            // a round before.  In even pages lane i works out the place of the i-th load
            // instruction's keys, first those of V, then of K: a few vector instructions
            // for all of them, where scalar ones for each took longer than the loads.
            constexpr int kAhead[2] = {kKeys, kKeys + kHalf};
            int page[kQuick ? 1 : 2 * kLoads];
            const char *place = nullptr;
            auto first_key = [&](int k0, int i) {  // of load i's keys; of the lane's, where each has its own
                const int u = (i % kLoads * kWaves + wave) * kOfWave + (kQuick ? 0 : lr);
                return k0 + (i < kLoads ? kAhead[0] : kAhead[1]) + u;
            };
            auto has = [&](int key) { return key >= p.lo && key < p.hi; };
            auto look_up = [&](int k0) {
#pragma unroll
                for (int i = 0; i < (kQuick ? 1 : 2 * kLoads); ++i) {
                    const int key = first_key(k0, kQuick ? lane % (2 * kLoads) : i);
                    page[i] = has(key) ? table[page_of(a.div, key)] : kQuick ? 0 : -1;
                }
            };
            auto find_places = [&](int k0) {
                if constexpr (kQuick) {
                    const int key = first_key(k0, lane % (2 * kLoads)), in_page = key - page_of(a.div, key) * a.cache.page;
                    const bool known = (uint32_t)page[0] < (uint32_t)a.cache.pages;
                    met |= !known;
                    place = (lane % (2 * kLoads) < kLoads ? vh : kh) +
                            token_offset(a, known ? page[0] : 0, has(key) ? in_page : 0);
                }
            };
            auto place_of = [&](int i) {  // of load i's first key
                const int64_t at = reinterpret_cast<int64_t>(place);
                const uint32_t lo = __builtin_amdgcn_readlane((int)at, i), hi = __builtin_amdgcn_readlane((int)(at >> 32), i);
                return reinterpret_cast<const char *>((uint64_t)hi << 32 | lo);
            };
            // Chunks of absent keys and past the head's columns are read from zeros:
            // their scores are masked, but an infinity or NaN among their values
            // would make NaN of p = 0.
            auto send = [&](int k0, auto of_k, char *buf, auto turn, u32x4_t *regs) {
                constexpr int kFirst = decltype(of_k)::value ? kLoads : 0;
                const int from_key = k0 + kAhead[decltype(of_k)::value ? 1 : 0];
                const uint32_t lds = lds_address(buf) + wave * kWave * 16;
                if (kQuick && a.dim == D && from_key >= p.lo && from_key + kKeys <= p.hi) {
#pragma unroll
                    for (int u = 0; u < kLoads; ++u) {
                        const char *const base = place_of(kFirst + u);
                        if constexpr (F8)
                            regs[u] = tl::ld16(base + (from + lc * 16));
                        else
                            load_lds(base, from + (lc ^ turn(key_of(u))) * 16, lds + u * kThreads * 16);
                    }
                    return;
                }
                // (places worked out here, not kept in registers through the rounds that do without)
                int l = lane;
                asm volatile("" : "+v"(l));
#pragma unroll
                for (int u = 0; u < kLoads; ++u) {
                    const int key = (u * kWaves + wave) * kOfWave + l / kLanes;
                    const int chunk = F8 ? l % kLanes : l % kLanes ^ turn(key);
                    bool there = has(from_key + key) && chunk < a.dim * kSize / 16;
                    const char *at;
                    if constexpr (kQuick) {
                        at = place_of(kFirst + u) + l / kLanes * a.token_units * 16;
                    } else {
                        const int of = page[kFirst + u], in_page =
                            from_key + key - page_of(a.div, from_key + key) * a.cache.page;
                        const bool known = (uint32_t)of < (uint32_t)a.cache.pages;
                        met |= !known && has(from_key + key);
                        there = there && known;
                        at = (decltype(of_k)::value ? kh : vh) + token_offset(a, of, in_page);
                    }
                    at = there ? at + chunk * 16 : a.zeros;
                    if constexpr (F8)
                        regs[u] = tl::ld16(at);
                    else
                        load_lds(at, lds + u * kThreads * 16);
                }
            };
            auto store = [&](char *buf, auto turn, const u32x4_t *regs) {
#pragma unroll
                for (int u = 0; u < kLoads; ++u) {
                    const int key = key_of(u), by = turn(key);
                    char *const to = buf + key * Sh::kRow;
                    tl::st16(to + ((2 * lc) ^ by) * 16, widen8(regs[u].x, regs[u].y));
                    tl::st16(to + ((2 * lc + 1) ^ by) * 16, widen8(regs[u].z, regs[u].w));
                }
            };
            auto k_turn = [](int key) { return Sh::k_turn(key); };
            auto v_turn = [](int key) { return Sh::v_turn(key); };
            // In round k0, whose buffer is buf: for V into the other buffer, for K into this one.
            auto send_v = [&](int k0, int buf) {
                if (k0 + kAhead[0] < p.hi) send(k0, std::false_type{}, sh.v[buf ^ 1], v_turn, vr);
            };
            auto send_k = [&](int k0, int buf) {
                if (k0 + kAhead[1] >= p.hi) return;
                send(k0, std::true_type{}, sh.k[buf], k_turn, kr);
                if constexpr (kCareful) {  // one bit a key, from the first of its lanes
                    uint64_t absent = 0;
#pragma unroll
                    for (int u = 0; u < kLoads; ++u) {
                        const uint64_t bits = __ballot((uint32_t)page[kLoads + u] >= (uint32_t)a.cache.pages);
                        for (int e = 0; e < kOfWave; ++e)
                            absent |= ((bits >> (e * kLanes)) & 1) << ((u * kWaves + wave) * kOfWave + e);
                    }
                    if (lane == 0) sh.absent[buf][wave] = absent;
                }
            };
            auto store_v = [&](int k0, int buf) {
                if (F8 && k0 + kAhead[0] < p.hi) store(sh.v[buf ^ 1], v_turn, vr);
            };
            auto store_k = [&](int k0, int buf) {
                if (F8 && k0 + kAhead[1] < p.hi) store(sh.k[buf], k_turn, kr);
            };
            // Scores of the lane's row with 32 keys: 8 (i / 4) + 4 h + i % 4 in register i.
            // b: which half of the buffer.
            const char *const lk = sh.k[0] + lane % 32 * Sh::kRow;
            const int tk = Sh::k_turn(lane % 32);  // (key 32 more has the same)
            auto scores = [&](int buf, int b) {
                f32x16_t s = {};
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    s = mfma_32x32x16(tl::ld16(lk + (buf * kKeys + kHalf * b) * Sh::kRow + ((2 * kk + h) ^ tk) * 16), q[kk], s);
                return s;
            };
            auto largest = [&](const f32x16_t &s) {
                float big = s[0];
#pragma unroll
                for (int i = 1; i < 16; ++i) big = larger(big, s[i]);
                return big;  // (of the lane's half of the keys)
            };
            // The sums stay relative to an older maximum until a score passes it by
            // 2^8: p may be that large as well, and scaling the sums costs as much
            // as a quarter of a product.
            auto rescale = [&](float big) {
                big = larger_of_halves(big);
                const float m2 = fmaxf(x.m, big * cf);
                if (__any(m2 > x.m + 8.0f)) {
                    const float f = exp2_fast(x.m - base_of(m2));
                    x.m = m2;
                    x.l *= f;
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) x.o[j] *= f;
                }
            };
            // o += p V for 32 keys, the first or second half of the buffer.  V: keys 16 c +
            // 4 h + lane % 16 / 4 and 8 more, columns 32 j + 16 (lane / 16 % 2) + 4 (lane % 4) ..
            const int vkey = 4 * h + lane % 16 / 4;
            const char *const lv = sh.v[0] + vkey * Sh::kRow + lane % 2 * 8;
            const int tv = Sh::v_turn(vkey), vchunk = lane / 16 % 2 * 2 + lane % 4 / 2;
            auto add = [&](const f32x16_t &s, int buf, int b) {
                const float base = base_of(x.m);
                float l[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {  // 16 keys each
                    float pr[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) pr[i] = exp2_fast(fmaf(s[8 * c + i], cf, -base));
                    l[c] = ((pr[0] + pr[1]) + (pr[2] + pr[3])) + ((pr[4] + pr[5]) + (pr[6] + pr[7]));
                    const u32x4_t pk = {tl::pack_bf16x2(pr[0], pr[1]), tl::pack_bf16x2(pr[2], pr[3]),
                                        tl::pack_bf16x2(pr[4], pr[5]), tl::pack_bf16x2(pr[6], pr[7])};
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) {  // (key 8 more has the same turn)
                        const char *const at =
                            lv + (buf * kKeys + kHalf * b + 16 * c) * Sh::kRow + ((4 * j + vchunk) ^ tv) * 16;
                        const uint2 lo = read_transposed(at), hi = read_transposed(at + 8 * Sh::kRow);
                        u32x4_t v = {lo.x, lo.y, hi.x, hi.y};
                        if constexpr (kCareful)
                            for (int e = 0; e < 4; ++e) v[e] = drop_not_finite(v[e]);
                        x.o[j] = mfma_32x32x16(v, pk, x.o[j]);
                    }
                }
                x.l += l[0] + l[1];
            };
            // add(s, buf, b) and, beside it, the next scores and the largest of them: each
            // product has exponentials or maxima to run beside, and fragments that were
            // read some products before.  (Left to the compiler, each fragment is read
            // right before its product and waited for, and products, exponentials and
            // products follow one another: pieces of prompts 840 us, so 779.)
            auto mixed = [&](const f32x16_t &s, int buf, int b, f32x16_t &next, int next_buf, int next_b) {
                constexpr int kN = D / 16, kT = D / 32, kAhead = 4, kExps = 16 / kN;
                const float base = base_of(x.m);
                const char *const bk = lk + (next_buf * kKeys + kHalf * next_b) * Sh::kRow;
                const char *const bv = lv + (buf * kKeys + kHalf * b) * Sh::kRow;
                u32x4_t kf[kAhead], vf[2][kT], pk[2];
                float pr[16], l[2], big = 0.0f;
                auto read_k = [&](int i) { kf[i % kAhead] = tl::ld16(bk + ((2 * i + h) ^ tk) * 16); };
                auto read_v = [&](int c, int j) {
                    const char *const at = bv + 16 * c * Sh::kRow + ((4 * j + vchunk) ^ tv) * 16;
                    const uint2 lo = read_transposed(at), hi = read_transposed(at + 8 * Sh::kRow);
                    vf[c][j] = u32x4_t{lo.x, lo.y, hi.x, hi.y};
                };
                auto pack = [&](int c) {
                    const float *const e = pr + 8 * c;
                    l[c] = ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
                    pk[c] = u32x4_t{tl::pack_bf16x2(e[0], e[1]), tl::pack_bf16x2(e[2], e[3]), tl::pack_bf16x2(e[4], e[5]),
                                    tl::pack_bf16x2(e[6], e[7])};
                };
                next = f32x16_t{};
#pragma unroll
                for (int i = 0; i < kAhead; ++i) read_k(i);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    next = mfma_32x32x16(kf[i % kAhead], q[i], next);
                    if (i + kAhead < kN) read_k(i + kAhead);
                    if (i >= kN - kT) read_v(0, i - (kN - kT));
#pragma unroll
                    for (int e = i * kExps; e < (i + 1) * kExps; ++e) pr[e] = exp2_fast(fmaf(s[e], cf, -base));
                    if ((i + 1) * kExps == 8) pack(0);
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int j = 0; j < kT; ++j) {
                        x.o[j] = mfma_32x32x16(vf[c][j], pk[c], x.o[j]);
                        if (c == 0) {
                            read_v(1, j);
                            if (j == 0) pack(1);
                        } else {
#pragma unroll
                            for (int e = j * (16 / kT); e < (j + 1) * (16 / kT); ++e)
                                big = e == 0 ? next[0] : larger(big, next[e]);
                            if (j == 0) x.l += l[0] + l[1];
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                return big;
            };
            // The builtin, since the compiler counts what it waits for: it would
            // otherwise wait for the rows of q in the loop, and so for the next keys.
            auto arrive = [&]() {
                __builtin_amdgcn_s_waitcnt(kWaitLoads);
                __syncthreads();
            };

            // Rounds of 64 keys.  Before round k0 the buffers of K hold or are being sent
            // the keys from k0 - 32 and from k0 + 32, that of V those from k0.
            if (p.lo < p.hi) {
                look_up(p.lo - 2 * kKeys);
                find_places(p.lo - 2 * kKeys);
                send_k(p.lo - 2 * kKeys, 0);
                store_k(p.lo - 2 * kKeys, 0);
                look_up(p.lo - kKeys);
                find_places(p.lo - kKeys);
                send_v(p.lo - kKeys, 1);
                store_v(p.lo - kKeys, 1);
                send_k(p.lo - kKeys, 1);
                store_k(p.lo - kKeys, 1);
                look_up(p.lo);
            }
            int k0 = p.lo;
            if constexpr (!kCareful) {
                // Keys that all rows see: scores 32 keys ahead, so that products and
                // exponentials, which different units compute, have something of the other
                // to run beside.
                const int full = p.lo + max(0, min(p.hi, tile_all_see) - p.lo) / kKeys * kKeys;
                if (k0 < full) {
                    f32x16_t s0, s1;
                    float big = 0.0f;
                    arrive();
                    if (any) {
                        s0 = scores(0, 1);
                        big = largest(s0);
                    }
                    auto step = [&](auto buffer) {
                        constexpr int buf = decltype(buffer)::value;
                        const bool more = k0 + kKeys < full;
                        arrive();
                        find_places(k0);
                        send_v(k0, buf);
                        send_k(k0, buf);
                        look_up(k0 + kKeys);
                        if (any) {
                            rescale(big);
                            big = mixed(s0, buf, 0, s1, buf ^ 1, 0);
                            rescale(big);
                            big = mixed(s1, buf, 1, s0, buf ^ 1, 1);  // (the latter's not used after the last round)
                        }
                        store_v(k0, buf);
                        store_k(k0, buf);
                        k0 += kKeys;
                        return more;
                    };
#pragma unroll 1
                    while (step(std::integral_constant<int, 0>{}) && step(std::integral_constant<int, 1>{})) {
                    }
                }
            }
            // The rest, whose scores are masked.
#pragma unroll 1
            for (; k0 < p.hi; k0 += kKeys) {
                const int buf = (k0 - p.lo) / kKeys & 1;
                arrive();
                find_places(k0);
                send_v(k0, buf);
                f32x16_t s[2];
                const bool busy = k0 < wave_sees;
                if (busy) {
                    uint64_t absent[2] = {};
                    if constexpr (kCareful)
                        for (int k = 0; k < kWaves; ++k) {
                            absent[0] |= sh.absent[buf][k] >> 32;
                            absent[1] |= sh.absent[buf ^ 1][k];
                        }
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const int left = seen - k0 - kHalf * b - 4 * h;
                        if (k0 + kHalf * b >= p.hi) {  // (not even sent)
                            for (int i = 0; i < 16; ++i) s[b][i] = -INFINITY;
                            continue;
                        }
                        s[b] = scores(buf ^ b, b ^ 1);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int key = 8 * (i / 4) + i % 4;
                            if (key >= left || (kCareful && ((absent[b] >> (key + 4 * h)) & 1))) s[b][i] = -INFINITY;
                        }
                    }
                }
                __syncthreads();  // (the first keys are read by all)
                send_k(k0, buf);
                look_up(k0 + kKeys);
                if (busy) {
                    rescale(larger(largest(s[0]), largest(s[1])));
                    add(s[0], buf, 0);
                    add(s[1], buf, 1);
                    if constexpr (kCareful) {
#pragma unroll 1
                        for (int key = 0; key < kKeys; ++key) {
                            const char *const at = sh.v[buf] + key * Sh::kRow + 8 * h;
#pragma unroll
                            for (int j = 0; j < D / 32; ++j)
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const uint2 v =
                                        *reinterpret_cast<const uint2 *>(at + ((4 * j + i) ^ Sh::v_turn(key)) * 16);
                                    float f[4] = {};
                                    add_not_finite(f, v, k0 + key < seen);
                                    for (int e = 0; e < 4; ++e) x.o[j][4 * i + e] += f[e];
                                }
                        }
                    }
                }
                store_v(k0, buf);
                store_k(k0, buf);
            }
            x.l += __shfl_xor(x.l, 32);
            if constexpr (kCareful) return false;
            if (live) {
                float size = 0.0f;
#pragma unroll
                for (int j = 0; j < D / 32; ++j)
#pragma unroll
                    for (int i = 0; i < 16; ++i) size = larger(size, fabsf(x.o[j][i]));
                met |= !(size < INFINITY);
            }
            return met;
        };
        if (threadIdx.x == 0) sh.again = 0;
        __syncthreads();
        if (__any(attend(std::false_type{})) && lane == 0) sh.again = 1;
        __syncthreads();
        if (scalar(sh.again)) {
            attend(std::true_type{});
            __syncthreads();
        }
        if (!p.split) {
            if (live) {
                const Finish finish(a, w.g);
                const float f = finish.factor(x.l);
#pragma unroll
                for (int j = 0; j < D / 32; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        put_columns(a, row, qh, D, 32 * j + 8 * i + 4 * h, f,
                                    f32x4_t{x.o[j][4 * i], x.o[j][4 * i + 1], x.o[j][4 * i + 2], x.o[j][4 * i + 3]});
                if (h == 0) put_stats(a, row, qh, finish, x.m, x.l);
            }
        } else {
            if (any) {
#pragma unroll
                for (int j = 0; j < D / 32; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *piece_sums<D>(a, p.slot, wave, 8 * j + i) = make_float2(x.o[j][2 * i], x.o[j][2 * i + 1]);
                if (h == 0) *piece_stats<D>(a, p.slot, wave) = make_float2(x.m, x.l);
            }
            if (p.begins && threadIdx.x == 0)
                a.joins[w.w] = {p.count, p.slot, t.row0 + t.first, t.count, w.g, {}};
        }
        __syncthreads();
    } while (w.next(a));
}

// The pieces of split tiles, in their order.  A wave takes 32 rows of a tile and
// 16 columns of each; the tiles are those that the workgroups before noted.
template <int D>
__global__ __launch_bounds__(kThreads) void attend_join_kernel(AttendArgs a) {
    constexpr int kPairs = 4, kItems = kWaves * (D / 4 / kPairs);  // of a lane; of a tile
    __shared__ int tiles[kManyGroups], scratch[kWaves + 1];
    const int lane = tl::lane_id(), h = lane / 32;
    constexpr int kEach = kManyGroups / kThreads;
    bool split[kEach];
    int mine = 0, total;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int e = threadIdx.x * kEach + k;
        split[k] = e < a.groups_of_threads && a.joins[e].pieces > 0;
        mine += split[k];
    }
    int at = tl::block_excl_scan<kThreads>(mine, scratch, total);
#pragma unroll
    for (int k = 0; k < kEach; ++k)
        if (split[k]) tiles[at++] = threadIdx.x * kEach + k;
    __syncthreads();
    for (int item = blockIdx.x * kWaves + tl::wave_id(); item < total * kItems; item += gridDim.x * kWaves) {
        const int first = scalar(tiles[item / kItems]), quarter = item % kItems % kWaves, pair = item % kItems / kWaves * kPairs;
        const Join t = a.joins[first];
        const int r = quarter * 32 + lane % 32;
        if (quarter * 32 >= t.rows) continue;
        float m = -INFINITY, l = 0.0f;
        float2 o[kPairs] = {};
        constexpr int kAt = 8;
        const int pieces = scalar(t.pieces), first_slot = scalar(t.slot);
        for (int k0 = 0; k0 < pieces; k0 += kAt) {
            float2 ml[kAt], v[kAt][kPairs];
#pragma unroll
            for (int u = 0; u < kAt; ++u) {
                if (k0 + u >= pieces) break;
                const int slot = k0 + u == 0 ? first_slot : 2 * (first + k0 + u);
                ml[u] = *piece_stats<D>(a, slot, quarter);
#pragma unroll
                for (int i = 0; i < kPairs; ++i) v[u][i] = *piece_sums<D>(a, slot, quarter, pair + i);
            }
#pragma unroll
            for (int u = 0; u < kAt; ++u) {
                if (k0 + u >= pieces) break;
                const float m2 = fmaxf(m, ml[u].x), base = base_of(m2);
                const float f = exp2_fast(m - base), f2 = exp2_fast(ml[u].x - base);
                m = m2;
                l = l * f + ml[u].y * f2;
#pragma unroll
                for (int i = 0; i < kPairs; ++i)
                    o[i] = make_float2(o[i].x * f + v[u][i].x * f2, o[i].y * f + v[u][i].y * f2);
            }
        }
        if (r >= t.rows) continue;
        const int64_t row = t.row + r / a.each;
        const int qh = t.g * a.each + r % a.each;
        const Finish finish(a, t.g);
        const float f = finish.factor(l);
#pragma unroll
        for (int i = 0; i < kPairs; i += 2)  // (four columns)
            put_columns(a, row, qh, D, 32 * ((pair + i) / 8) + 8 * ((pair + i) % 8 / 2) + 4 * h, f,
                        f32x4_t{o[i].x, o[i].y, o[i + 1].x, o[i + 1].y});
        if (pair == 0 && h == 0) put_stats(a, row, qh, finish, m, l);
    }
}

template <int D, bool F8>
void launch_rows(const AttendArgs &a, hipStream_t st) {
    const dim3 grid(a.groups_of_threads), block(kThreads);
    constexpr int kOfLoad = kKeysOfLoad<D, F8>;
    // (with the lane's offset in 32 bits)
    if (a.cache.page % kOfLoad == 0 && a.token_units < (1u << 31) / (16 * kOfLoad))
        attend_many_kernel<D, F8, true><<<grid, block, 0, st>>>(a);
    else
        attend_many_kernel<D, F8, false><<<grid, block, 0, st>>>(a);
}

template <int D>
hipError_t go(const AttendArgs &a, hipStream_t st) {
    if (a.cache.k_scale)
        launch_rows<D, true>(a, st);
    else
        launch_rows<D, false>(a, st);
    if (hipError_t e = hipGetLastError()) return e;
    // (no tile that the table allows is worth cutting)
    if ((int64_t)a.table_cols * a.cache.page <= kManyWhole) return hipSuccess;
    attend_join_kernel<D><<<dim3(kJoinGroups), dim3(kThreads), 0, st>>>(a);
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
