// step_score.hip -- step_token_logprobs: log probabilities of given tokens,
// their ranks, the rows' entropies and their most likely tokens.
//
// One pass over a row of logits with a running maximum m per thread,
//     T = sum e^(z-m),  U = sum e^(z-m) (z-m),  C = #{z > z_token},
// joined at the end by rescaling to the largest m:
//     logp = z - m - ln T,  entropy = ln T - U / T,  rank = 1 + C.
// (Every term of the entropy is >= 0, so nothing cancels.)
//
// The top k come from the same pass: a thread keeps only its maximum and the
// vector that holds it.  The k-th largest of the thread maxima bounds the
// k-th largest logit from below and only the k threads that reach it can hold
// one that is larger, so the workgroup reads those threads' vectors again (a
// few dozen, from the cache) and ranks the few values at or above the bound.
// Logits are ordered by 64-bit keys (value, lowest index first), which are
// all different, so ties need no case of their own and no count depends on
// the order in which threads add to a list.
//
// A row is cut into parts, a workgroup each; the last one of a row to finish
// joins the parts' sums and sorted lists.  Bound by the read of the logits
// (6947 x 32003 floats: 155 us, 5.7 TB/s), in bf16 (135 us) and for fewer rows by the pass's
// instructions (256 x 128256 bf16: 22 us, 31 with 20 alternatives), and for a
// single row by the latency of the chain read, select, join (12 us).
#include "common.h"
#include "step_kernels.h"

namespace st {

using tl::kWave;
using tl::u32x4_t;

namespace {

constexpr int kCandidates = kMaxTop * kScoreLaneElems;
constexpr int kUnroll = 4;
static_assert(kScoreMaxParts <= kWave && kMaxTop * kMaxTop <= kCandidates, "one wave joins a row's parts");
constexpr float kLog2e = 1.44269504088896340736f;
// (z - m) log2 e below this adds nothing to fp32 sums; it keeps 0 * -inf out of U.
constexpr float kFloor = -300.0f;

// v_exp_f32: results below the smallest normal number are 0.
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Larger key = larger logit, or the same logit at a lower index.  0 stands
// for "no logit" (masked ones and absent ones).  (z + 0 turns -0 into +0.)
__device__ __forceinline__ uint64_t make_key(float z, int idx) {
    if (!(z > -INFINITY)) return 0;
    const uint32_t u = __float_as_uint(z + 0.0f);
    const uint32_t ord = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    return ((uint64_t)ord << 32) | (uint32_t)~idx;
}
__device__ __forceinline__ float key_value(uint64_t key) {
    const uint32_t ord = (uint32_t)(key >> 32);
    return __uint_as_float((ord & 0x80000000u) ? ord ^ 0x80000000u : ~ord);
}
__device__ __forceinline__ int key_index(uint64_t key) { return (int)~(uint32_t)key; }

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int d) {
    const uint32_t lo = __shfl_xor((int)(uint32_t)v, d), hi = __shfl_xor((int)(uint32_t)(v >> 32), d);
    return ((uint64_t)hi << 32) | lo;
}

struct Stat {
    float m, t, u;
    int c;
};
// Joins two sets' sums at the larger maximum.
__device__ __forceinline__ Stat join(const Stat a, const Stat b) {
    const float m = fmaxf(a.m, b.m);
    const float da = a.m > -INFINITY ? a.m - m : 0.0f, db = b.m > -INFINITY ? b.m - m : 0.0f;
    const float fa = exp2_fast(da * kLog2e), fb = exp2_fast(db * kLog2e);
    return {m, a.t * fa + b.t * fb, fa * fmaf(a.t, fmaxf(da, kFloor), a.u) + fb * fmaf(b.t, fmaxf(db, kFloor), b.u),
            a.c + b.c};
}
__device__ __forceinline__ Stat wave_join(Stat s) {
    for (int d = 1; d < kWave; d <<= 1)
        s = join(s, Stat{__shfl_xor(s.m, d), __shfl_xor(s.t, d), __shfl_xor(s.u, d), __shfl_xor(s.c, d)});
    return s;
}

// A row as vectors: id 0 the logits before the first 16-byte boundary, ids
// 1..nvec the whole vectors, id nvec + 1 the rest (the first and last may be
// empty); E logits a vector.
template <bool F32>
struct Row {
    static constexpr int E = F32 ? 4 : 8;
    const char *base;
    int v, head, nvec;

    __device__ Row(const void *logits, int64_t ld, int row, int v_) : v(v_) {
        constexpr int esz = F32 ? 4 : 2;
        base = static_cast<const char *>(logits) + (int64_t)row * ld * esz;
        const int to16 = (int)((16 - (reinterpret_cast<uintptr_t>(base) & 15)) & 15) / esz;
        head = to16 < v ? to16 : v;
        nvec = (v - head) / E;
    }
    __device__ __forceinline__ float at(int i) const {
        if constexpr (F32) return reinterpret_cast<const float *>(base)[i];
        return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(base)[i] << 16);
    }
    __device__ __forceinline__ int start(int id) const { return id == 0 ? 0 : head + (id - 1) * E; }
    __device__ __forceinline__ bool whole(int id) const { return id >= 1 && id <= nvec; }
    __device__ __forceinline__ const void *vec(int id) const {
        return base + (int64_t)(head + (id - 1) * E) * (F32 ? 4 : 2);
    }
    static __device__ __forceinline__ void unpack(const u32x4_t w, float *z) {
        if constexpr (F32) {
            z[0] = __uint_as_float(w.x), z[1] = __uint_as_float(w.y), z[2] = __uint_as_float(w.z),
            z[3] = __uint_as_float(w.w);
        } else {
            z[0] = tl::bf_lo(w.x), z[1] = tl::bf_hi(w.x), z[2] = tl::bf_lo(w.y), z[3] = tl::bf_hi(w.y);
            z[4] = tl::bf_lo(w.z), z[5] = tl::bf_hi(w.z), z[6] = tl::bf_lo(w.w), z[7] = tl::bf_hi(w.w);
        }
    }
    // Any id; absent logits read as -infinity, which adds nothing anywhere.
    __device__ __forceinline__ void load(int id, float *z) const {
        if (whole(id)) {
            unpack(tl::ld16(vec(id)), z);
            return;
        }
        const int first = start(id), last = id == 0 ? head : v;
#pragma unroll
        for (int i = 0; i < E; ++i) z[i] = first + i < last ? at(first + i) : -INFINITY;
    }
};

template <int E>
__device__ __forceinline__ float max_of(const float *z) {
    float m = z[0];
#pragma unroll
    for (int i = 1; i < E; ++i) m = fmaxf(m, z[i]);
    return m;
}

// Running sums of a thread: `best` is the vector id of the first maximum.
struct Lane {
    float m, t, u;
    int c, best;

    template <int E>
    __device__ __forceinline__ void add(const float *z, float z_tok) {
        const float ref = m > -INFINITY ? m : 0.0f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float d = (z[i] - ref) * kLog2e;
            const float e = exp2_fast(d);
            t += e;
            u = fmaf(e, fmaxf(d, kFloor), u);  // in units of log2; scaled when the pass ends
            c += z[i] > z_tok ? 1 : 0;
        }
    }
};

// The key of rank k - 1 (0 = largest) among 64 keys in LDS, or 0 when fewer
// than k are present.  Every wave computes it.
__device__ __forceinline__ uint64_t kth_of_64(const uint64_t *keys, int k) {
    const uint64_t mine = keys[tl::lane_id()];
    int rank = 0;
#pragma unroll 16
    for (int j = 0; j < kWave; ++j) rank += keys[j] > mine ? 1 : 0;
    const uint64_t hit = __ballot(mine != 0 && rank == k - 1);
    if (!hit) return 0;
    return keys[__builtin_ctzll(hit)];
}

// T threads a workgroup: T / 64 threads per group of the first selection, so
// 64 groups.
template <int T>
struct Shared {
    static constexpr int kGroup = T / kWave;
    uint64_t groups[kWave];
    uint64_t lanes[kMaxTop * kGroup];  // thread maxima at or above the first bound
    int owner[kMaxTop * kGroup];
    int sel[kMaxTop];
    uint64_t cand[kCandidates];
    Stat stats[T / kWave];
    uint64_t bound;
    int n_lanes, n_cand, last;
};

// Ranks the collected candidates and hands each of the first k to `put`.
template <int T, class Put>
__device__ __forceinline__ void rank_candidates(const Shared<T> &sh, int k, Put put) {
    const int n = sh.n_cand;
    for (int i = threadIdx.x; i < n; i += T) {
        const uint64_t mine = sh.cand[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += sh.cand[j] > mine ? 1 : 0;
        if (rank < k) put(rank, mine);
    }
}

template <bool F32, int T>
__device__ __forceinline__ void part_top(const Row<F32> &r, const Lane &a, int id0, int id1, int k, Shared<T> &sh) {
    constexpr int kGroup = Shared<T>::kGroup;
    constexpr int E = Row<F32>::E;
    const int tid = threadIdx.x;
    const uint64_t mine = make_key(a.m, a.best < 0 ? 0 : r.start(a.best));
    uint64_t g = mine;
    for (int d = 1; d < kGroup; d <<= 1) {
        const uint64_t o = shfl_xor64(g, d);
        g = o > g ? o : g;
    }
    if (tid % kGroup == 0) sh.groups[tid / kGroup] = g;
    if (tid == 0) sh.n_lanes = sh.n_cand = 0;
    __syncthreads();
    // at most k groups reach the first bound, so at most k * kGroup threads do
    const uint64_t first = kth_of_64(sh.groups, k);
    if (mine != 0 && mine >= first && g >= first) {
        const int at = atomicAdd(&sh.n_lanes, 1);
        sh.lanes[at] = mine;
        sh.owner[at] = tid;
    }
    if (tid == 0) sh.bound = 0;
    __syncthreads();
    const int nl = sh.n_lanes;
    if (tid < nl) {
        const uint64_t key = sh.lanes[tid];
        int rank = 0;
        for (int j = 0; j < nl; ++j) rank += sh.lanes[j] > key ? 1 : 0;
        if (rank < k) sh.sel[rank] = sh.owner[tid];
        // (a thread's key names its vector's first place: the logit itself may
        // sit up to E - 1 places later)
        if (rank == k - 1) sh.bound = key - (E - 1);
    }
    __syncthreads();
    const uint64_t bound = sh.bound;
    const int nsel = nl < k ? nl : k, per = (id1 - id0 + T - 1) / T;
    for (int i = tid; i < nsel * per; i += T) {
        const int id = id0 + sh.sel[i / per] + (i % per) * T;
        if (id >= id1) continue;
        float z[E];
        r.load(id, z);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const uint64_t key = make_key(z[e], r.start(id) + e);
            if (key != 0 && key >= bound) sh.cand[atomicAdd(&sh.n_cand, 1)] = key;
        }
    }
    __syncthreads();
}

__device__ __forceinline__ void put_top(const ScoreArgs &a, int row, int rank, uint64_t key, float m, float log_t) {
    const int64_t at = (int64_t)row * a.top + rank;
    a.top_ids[at] = key ? key_index(key) : -1;
    a.top_logprobs[at] = key ? key_value(key) - m - log_t : -INFINITY;
}

// The row's answers from its joined sums (by one thread).
template <bool F32>
__device__ __forceinline__ void put_row(const ScoreArgs &a, const Row<F32> &r, int row, int token, const Stat s) {
    const float log_t = logf(s.t);
    const float ref = s.m > -INFINITY ? s.m : 0.0f;
    float lp = 0.0f;
    int rank = 0;
    if (token >= a.v) {
        lp = NAN;
    } else if (token >= 0) {
        const float z = r.at(token);
        lp = z > -INFINITY || z != z ? z - ref - log_t : -INFINITY;
        if (s.t != s.t) lp = NAN;
        rank = 1 + s.c;
    }
    a.logprob[row] = lp;
    a.rank[row] = rank;
    a.entropy[row] = s.m > -INFINITY ? log_t - s.u / s.t : (s.t != s.t ? NAN : 0.0f);
}

__device__ __forceinline__ uint32_t ld_agent(const uint32_t *p) {
    return __hip_atomic_load(const_cast<uint32_t *>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void st_agent(uint32_t *p, uint32_t v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <bool F32, int T>
__global__ __launch_bounds__(T) void score_kernel(ScoreArgs a, int parts, int part_ids, int32_t *tickets,
                                                         uint32_t *records) {
    constexpr int E = Row<F32>::E;
    __shared__ Shared<T> sh;
    const int tid = threadIdx.x, k = a.top;
    const int row = blockIdx.x / parts, part = blockIdx.x % parts;
    const Row<F32> r(a.logits, a.ld, row, a.v);
    const int token = a.tokens[row];
    const float z_tok = token >= 0 && token < a.v ? r.at(token) : INFINITY;
    const int ids = r.nvec + 2;
    const int id0 = min(part * part_ids, ids), id1 = min(id0 + part_ids, ids);

    // ---- the pass over this part's logits
    Lane s{-INFINITY, 0.0f, 0.0f, 0, -1};
    for (int id = id0 + tid; id < id1; id += kUnroll * T) {
        float z[kUnroll][E];
        if (id >= 1 && id + (kUnroll - 1) * T < id1 && id + (kUnroll - 1) * T <= r.nvec) {
            u32x4_t w[kUnroll];
#pragma unroll
            for (int j = 0; j < kUnroll; ++j) w[j] = tl::ld16(r.vec(id + j * T));
#pragma unroll
            for (int j = 0; j < kUnroll; ++j) Row<F32>::unpack(w[j], z[j]);
        } else {
#pragma unroll
            for (int j = 0; j < kUnroll; ++j) {
                if (id + j * T < id1) {
                    r.load(id + j * T, z[j]);
                } else {
#pragma unroll
                    for (int i = 0; i < E; ++i) z[j][i] = -INFINITY;
                }
            }
        }
        float big[kUnroll], all = -INFINITY;
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) all = fmaxf(all, big[j] = max_of<E>(z[j]));
        if (all > s.m) {
            int at = 0;
#pragma unroll
            for (int j = kUnroll - 1; j >= 0; --j) at = big[j] == all ? id + j * T : at;
            // U is kept in units of log2 during the pass
            const float d = s.m > -INFINITY ? (s.m - all) * kLog2e : 0.0f, f = exp2_fast(d);
            s.u = f * fmaf(s.t, fmaxf(d, kFloor), s.u);
            s.t *= f;
            s.m = all;
            s.best = at;
        }
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) s.add<E>(z[j], z_tok);
    }
    s.u *= 1.0f / kLog2e;

    // ---- sums of the part
    const Stat ws = wave_join(Stat{s.m, s.t, s.u, s.c});
    if (tl::lane_id() == 0) sh.stats[tid / kWave] = ws;
    if (k > 0) part_top(r, s, id0, id1, k, sh);
    else __syncthreads();
    Stat all = sh.stats[0];
    for (int w = 1; w < T / kWave; ++w) all = join(all, sh.stats[w]);

    if (parts == 1) {
        const float ref = all.m > -INFINITY ? all.m : 0.0f, log_t = logf(all.t);
        if (tid == 0) put_row(a, r, row, token, all);
        if (k > 0) {
            rank_candidates(sh, k, [&](int rank, uint64_t key) { put_top(a, row, rank, key, ref, log_t); });
            if (tid < k && tid >= sh.n_cand) put_top(a, row, tid, 0, ref, log_t);
        }
        return;
    }

    // ---- leave the part's record, and join the row if it is the last one
    // Records are written and read as agent-scope words, which go past the
    // caches that other XCDs cannot see; a wave's stores are complete (vmcnt
    // 0) before its barrier, so before the ticket is taken.  The ticket itself
    // needs no fences then: an acquire and release a workgroup writes back and
    // empties its XCD's L2 each time (256 rows of
    // 128256: 48 us with them, 31 without).
    const int words = score_record_words(k);
    uint32_t *rec = records + ((int64_t)row * parts + part) * words;
    if (tid == 0) {
        st_agent(rec, __float_as_uint(all.m));
        st_agent(rec + 1, __float_as_uint(all.t));
        st_agent(rec + 2, __float_as_uint(all.u));
        st_agent(rec + 3, (uint32_t)all.c);
    }
    if (k > 0) {
        rank_candidates(sh, k, [&](int rank, uint64_t key) {
            st_agent(rec + 4 + 2 * rank, (uint32_t)(key >> 32));
            st_agent(rec + 5 + 2 * rank, (uint32_t)key);
        });
        if (tid < k && tid >= sh.n_cand) {
            st_agent(rec + 4 + 2 * tid, 0);
            st_agent(rec + 5 + 2 * tid, 0);
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid == 0) sh.last = tl::atomic_add_relaxed(tickets + row, 1) == parts - 1;
    __syncthreads();
    asm volatile("" ::: "memory");
    if (!sh.last) return;

    const uint32_t *recs = records + (int64_t)row * parts * words;
    if (tid < kWave) {
        Stat p{-INFINITY, 0.0f, 0.0f, 0};
        uint64_t head = 0;
        if (tid < parts) {
            const uint32_t *q = recs + (int64_t)tid * words;
            p = Stat{__uint_as_float(ld_agent(q)), __uint_as_float(ld_agent(q + 1)), __uint_as_float(ld_agent(q + 2)),
                     (int)ld_agent(q + 3)};
            if (k > 0) head = ((uint64_t)ld_agent(q + 4) << 32) | ld_agent(q + 5);
        }
        p = wave_join(p);
        if (tid == 0) {
            sh.stats[0] = p;
            sh.n_cand = 0;
            tl::store_relaxed(tickets + row, 0);  // ready for the next call
        }
        sh.groups[tid] = head;
    }
    __syncthreads();
    all = sh.stats[0];
    if (tid == 0) put_row(a, r, row, token, all);
    if (k == 0) return;
    // only the k lists whose first key reaches the k-th first key can matter
    const uint64_t bound = kth_of_64(sh.groups, k);
    for (int i = tid; i < parts * k; i += T) {
        const int p = i / k, j = i % k;
        if (sh.groups[p] == 0 || sh.groups[p] < bound) continue;
        const uint32_t *q = recs + (int64_t)p * words + 4 + 2 * j;
        const uint64_t key = ((uint64_t)ld_agent(q) << 32) | ld_agent(q + 1);
        if (key != 0 && key >= bound) sh.cand[atomicAdd(&sh.n_cand, 1)] = key;
    }
    __syncthreads();
    const float ref = all.m > -INFINITY ? all.m : 0.0f, log_t = logf(all.t);
    rank_candidates(sh, k, [&](int rank, uint64_t key) { put_top(a, row, rank, key, ref, log_t); });
    if (tid < k && tid >= sh.n_cand) put_top(a, row, tid, 0, ref, log_t);
}

}  // namespace

hipError_t launch_token_logprobs(const ScoreArgs &a, const ScorePlan &plan, void *ws, hipStream_t st) {
    int32_t *tickets = static_cast<int32_t *>(ws);
    uint32_t *records = reinterpret_cast<uint32_t *>(static_cast<char *>(ws) + plan.ticket_bytes);
    const dim3 grid((unsigned)a.n * plan.parts), block(plan.threads);
    auto launch = [&](auto kernel) { kernel<<<grid, block, 0, st>>>(a, plan.parts, plan.part_ids, tickets, records); };
    if (plan.threads == kScoreShortThreads)
        launch(a.fp32 ? score_kernel<true, kScoreShortThreads> : score_kernel<false, kScoreShortThreads>);
    else
        launch(a.fp32 ? score_kernel<true, kScoreThreads> : score_kernel<false, kScoreThreads>);
    return hipGetLastError();
}

}  // namespace st
