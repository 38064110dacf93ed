// attend.h -- what the two kernels of step_paged_attention share: how a
// workgroup finds its part of the work, keys' places in the paged cache, and
// how pieces' results pass from one workgroup to another.  Internal to the
// library.
#pragma once

#include <type_traits>

#include "attend_kernels.h"
#include "common.h"

namespace st {

using tl::f32x4_t;
using tl::kWave;
using tl::u32x4_t;

namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr float kLn2 = 0.69314718055994530942f;

// v_exp_f32: results below the smallest normal number are 0.
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
// A maximum that exponents can be taken from: that of a row without keys is -infinity.
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.0f : m; }
__device__ __forceinline__ int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t scalar64(int64_t v) {
    return (int64_t)((uint64_t)(uint32_t)scalar((int)(v >> 32)) << 32 | (uint32_t)scalar((int)v));
}
// LDS written by some lanes of a wave is read by others of the same wave.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Eight e4m3 values as bf16 (exact).
__device__ __forceinline__ u32x4_t widen8(uint32_t lo, uint32_t hi) {
    auto two = [](uint32_t v, auto high) {
        const auto f = __builtin_amdgcn_cvt_pk_f32_fp8((int)v, decltype(high)::value);
        return tl::pack_bf16x2(f[0], f[1]);
    };
    return u32x4_t{two(lo, std::false_type{}), two(lo, std::true_type{}), two(hi, std::false_type{}),
                   two(hi, std::true_type{})};
}

typedef short i16x4_t __attribute__((ext_vector_type(4)));
// Transposed read: lane i of 16 gives the address of 4 values (row i / 4,
// columns 4 * (i % 4) ..) and gets column i of the four rows.
__device__ __forceinline__ uint2 read_transposed(const char *p) {
    return __builtin_bit_cast(
        uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t *)p));
}

// ---------------------------------------------------------------- values that are not finite
// A key that one row of a tile must not see is masked by p = 0, and 0 times an
// infinity or NaN among its values would be NaN.  Such values are left out of
// the product and added to the sums of the rows that do see the key, which they
// make infinite or NaN whatever p is.
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ bool not_finite(const u32x4_t v) {
    u16x2_t m = {};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, (uint32_t)(v[e] & 0x7fff7fffu)));
    return m.x >= 0x7f80 || m.y >= 0x7f80;
}
__device__ __forceinline__ uint32_t drop_not_finite(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    return w;
}
__device__ __forceinline__ float only_not_finite(float v) { return fabsf(v) < INFINITY ? 0.0f : v; }
// acc += four values of a key where they are not finite.
__device__ __forceinline__ void add_not_finite(float *acc, uint2 v, bool seen) {
    const float f[4] = {tl::bf_lo(v.x), tl::bf_hi(v.x), tl::bf_lo(v.y), tl::bf_hi(v.y)};
    for (int e = 0; e < 4; ++e) acc[e] += seen ? only_not_finite(f[e]) : 0.0f;
}

// ---------------------------------------------------------------- requests
struct Job {
    Span s;
    int row0;
};
// Whatever the arrays hold, rows stay in [0, n) and keys on the table.
__device__ __forceinline__ Job job_of(const AttendArgs &a, int j) {
    int b0 = j, b1 = j + 1, len = 0;
    if (a.groups) {
        b0 = j > 0 ? min(max(a.groups[j - 1], 0), a.requests) : 0;
        b1 = j < a.jobs - 1 ? min(max(a.groups[j], 0), a.requests) : a.requests;
        if (j > 0 && j < a.jobs - 1) len = a.lens[j - 1];
    } else {
        len = a.lens[j];
    }
    const int r0 = a.starts ? min(max(a.starts[b0], 0), a.n) : b0;
    const int r1 = a.starts ? min(max(a.starts[b1], 0), a.n) : b1;
    const int64_t most = (int64_t)a.table_cols * a.cache.page;
    return {{max(r1 - r0, 0), max(0, (int)min((int64_t)len, most))}, r0};
}
__device__ __forceinline__ const int32_t *table_of(const AttendArgs &a, int j) {
    // (the first and the last job of groups have no keys)
    const int row = a.groups ? min(max(j - 1, 0), a.jobs - 3) : j;
    return a.table + row * a.ld_table;
}
__device__ __forceinline__ int64_t job_cost(const AttendArgs &a, Span s, int tokens, int fixed) {
    return tiles_cost(s, tokens, a.causal, fixed, tiles_of(s.rows, tokens));
}

// Neighbouring ranges, which share keys, go to one XCD.
__device__ __forceinline__ int workgroup_of(const AttendArgs &a) {
    const int groups = a.groups_of_threads, blk = blockIdx.x;
    return groups % 8 == 0 ? (blk % 8) * (groups / 8) + blk / 8 : blk;
}

struct Found {
    int64_t wave_sum[kWaves], base;
    int job;
};

// A workgroup's walk through the tiles of its range.  (All of it is the same in
// every lane; divisions are computed by the vector unit, and what follows from
// them stays there, in registers that the kernels are short of, unless it is
// taken back to scalar ones.)
struct Walk {
    Ranges r;
    int64_t total, at, end;  // cost at which the tile begins; at which the range ends
    int w, tokens;
    int j, g, i, tiles;
    Job job;

    // By every thread of the workgroup; false if nothing is left for it.
    __device__ __forceinline__ bool find(const AttendArgs &a, int rows, int fixed, int least, int whole,
                                         Found &found) {
        const int tid = threadIdx.x, lane = tl::lane_id();
        tokens = scalar(rows / a.each);
        w = workgroup_of(a);
        const int per = (a.jobs + kThreads - 1) / kThreads, j0 = min(tid * per, a.jobs), j1 = min(j0 + per, a.jobs);
        int64_t mine = 0;
        for (int k = j0; k < j1; ++k) mine += a.kv * job_cost(a, job_of(a, k).s, tokens, fixed);
        int64_t incl = mine;
        for (int d = 1; d < kWave; d *= 2) {
            const int64_t up = __shfl_up((long long)incl, d);
            if (lane >= d) incl += up;
        }
        if (lane == kWave - 1) found.wave_sum[tid / kWave] = incl;
        __syncthreads();
        total = 0;
        for (int k = 0; k < kWaves; ++k) {
            if (k == tid / kWave) incl += total;
            total += found.wave_sum[k];
        }
        total = scalar64(total);
        r = ranges_of(total, a.groups_of_threads, fixed, least, whole);
        r = {scalar64(r.size), scalar64(r.whole), fixed};
        const int64_t begin = w * r.size;
        end = begin + r.size < total ? begin + r.size : total;
        if (begin >= total) return false;
        if (begin >= incl - mine && begin < incl) {
            int64_t base = incl - mine;
            int k = j0;
            for (;; ++k) {
                const int64_t c = a.kv * job_cost(a, job_of(a, k).s, tokens, fixed);
                if (begin < base + c) break;
                base += c;
            }
            found.job = k;
            found.base = base;
        }
        __syncthreads();
        j = scalar(found.job);
        load(a);
        const int64_t base = scalar64(found.base), head = scalar64(job_cost(a, job.s, tokens, fixed));
        g = scalar((int)((begin - base) / head));
        i = scalar(tile_at(job.s, tokens, a.causal, fixed, begin - base - g * head));
        at = scalar64(base + g * head + tiles_cost(job.s, tokens, a.causal, fixed, i));
        return true;
    }
    __device__ __forceinline__ void load(const AttendArgs &a) {
        const Job b = job_of(a, j);
        job = {{scalar(b.s.rows), scalar(b.s.len)}, scalar(b.row0)};
        tiles = scalar(tiles_of(job.s.rows, tokens));
    }
    __device__ __forceinline__ int keys(const AttendArgs &a) const {
        return scalar(tile_keys(job.s, tokens, a.causal, i));
    }
    __device__ __forceinline__ Piece piece(int keys, int step) const {
        const Piece p = piece_of(r, w, at, keys, step);
        return {scalar(p.mine) != 0, scalar(p.split) != 0, scalar(p.begins) != 0, scalar(p.lo), scalar(p.hi),
                scalar(p.first), scalar(p.count), scalar(p.slot)};
    }
    // The next tile; false behind the range's last one.
    __device__ __forceinline__ bool next(const AttendArgs &a) {
        at += r.fixed + keys(a);
        if (at >= end) return false;
        if (++i < tiles) return true;
        i = 0;
        if (++g < a.kv) return true;
        g = 0;
        do {
            ++j;
            load(a);
        } while (job.s.rows == 0);
        return true;
    }
};

// Rows of a tile: row r is token r / each of the tile and head r % each of the key head.
struct TileRows {
    int row0, first, count;  // the request's first row; the tile's first token; its rows
    __device__ __forceinline__ TileRows(const AttendArgs &a, const Walk &w)
        : row0(w.job.row0), first(w.i * w.tokens), count(min(w.tokens, w.job.s.rows - w.i * w.tokens) * a.each) {}
    // Keys that token t of the tile sees.
    static __device__ __forceinline__ int seen(const AttendArgs &a, Span s, int token) {
        return a.causal ? max(0, min(s.len, s.len - s.rows + token + 1)) : s.len;
    }
};

// ---------------------------------------------------------------- keys in the cache
// Byte offset of a token in the cache.  (Strides are whole 16-byte units, of
// which less than 2^32 make one.)
__device__ __forceinline__ uint64_t token_offset(const AttendArgs &a, int page, int in_page) {
    return ((uint64_t)(uint32_t)page * a.page_units + (uint64_t)(uint32_t)in_page * a.token_units) * 16;
}

// ---------------------------------------------------------------- scales of a head
// What turns scores into exponents.  A scale of 0, of a head that is all zeros,
// must not meet the masks' infinity; one that is not finite is left out, and the
// rows that see such keys become NaN when they are finished.
__device__ __forceinline__ float scale_of_scores(const AttendArgs &a, int g) {
    return a.scale * (a.cache.k_scale ? a.cache.k_scale[g] : 1.0f);
}
__device__ __forceinline__ float exponent_factor(const AttendArgs &a, int g) {
    const float c = scale_of_scores(a, g);
    return c < INFINITY ? fmaxf(c, 1e-30f) : 1.0f;
}
// What a row's weighted sum of values is multiplied by, and the logarithm of its sum.
struct Finish {
    bool finite;
    float values;
    __device__ __forceinline__ Finish(const AttendArgs &a, int g)
        : finite(scale_of_scores(a, g) < INFINITY), values(a.cache.v_scale ? a.cache.v_scale[g] : 1.0f) {}
    __device__ __forceinline__ float factor(float l) const { return l == 0.0f ? 0.0f : finite ? values / l : NAN; }
    __device__ __forceinline__ float log_sum(float m, float l) const {
        return l == 0.0f ? -INFINITY : finite ? (base_of(m) + log2f(l)) * kLn2 : NAN;
    }
};

// ---------------------------------------------------------------- results of pieces
// Words that another workgroup, perhaps on another XCD, reads: written through
// to memory and read from there.
__device__ __forceinline__ void put_pair(float *p, float x, float y) {
    tl::store_word64(reinterpret_cast<uint64_t *>(p), ((uint64_t)__float_as_uint(y) << 32) | __float_as_uint(x));
}
__device__ __forceinline__ float2 get_pair(const float *p) {
    const uint64_t v = tl::load_word64(reinterpret_cast<const uint64_t *>(p));
    return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}
// By every thread, after its piece's results are written: whether this
// workgroup is the last of the tile's.  The words went through to memory
// before the ticket is taken, so the ticket needs no fences.
__device__ __forceinline__ bool last_of(const AttendArgs &a, const Piece &p, int *flag) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) {
        const bool last = tl::atomic_add_relaxed(a.tickets + p.first, 1) == p.count - 1;
        if (last) tl::store_relaxed(a.tickets + p.first, 0);  // ready for the next call
        *flag = last;
    }
    __syncthreads();
    asm volatile("" ::: "memory");
    return *flag;
}

}  // namespace

}  // namespace st
