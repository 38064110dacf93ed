// attend_abi.cpp -- step.h's entry points of the paged cache: host-side
// validation, workspaces and launches.  Nothing here allocates, frees or
// synchronizes; every check runs before any launch.
#include <hip/hip_runtime.h>

#include "../../include/step.h"
#include "attend_kernels.h"

namespace {

bool aligned(const void *p, unsigned to) { return p && (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool aligned_or_null(const void *p, unsigned to) { return !p || aligned(p, to); }
int launched(hipError_t e) { return e == hipSuccess ? STEP_OK : STEP_ELAUNCH; }

constexpr int64_t kMostStride = 1LL << 40, kMostCacheStride = 1LL << 35;  // (the latter in 16 bytes: 32 bits)
constexpr int kMostKeys = 1 << 24;

int check_heads(int n, int heads, int kv, int dim) {
    if (n < 0 || kv < 1 || heads < kv || heads % kv != 0 || dim < 16 || dim % 16 != 0) return STEP_EINVAL;
    if (n > STEP_MAX_TOKENS || heads > 4096 || heads / kv > st::kMaxEach || dim > st::kMaxDim) return STEP_EUNSUPPORTED;
    return STEP_OK;
}

// The cache and its strides; those of an axis of length one mean nothing and become 0.
int check_cache(st::CacheArgs &c, int kv, int dim) {
    const int unit = c.k_scale ? 16 : 8;
    if (c.pages < 1 || c.page < 1) return STEP_EINVAL;
    if ((int64_t)c.pages * c.page > INT32_MAX) return STEP_EUNSUPPORTED;
    if (!aligned(c.k, 16) || !aligned(c.v, 16)) return STEP_EINVAL;
    if ((c.k_scale == nullptr) != (c.v_scale == nullptr)) return STEP_EINVAL;
    if (!aligned_or_null(c.k_scale, 4) || !aligned_or_null(c.v_scale, 4)) return STEP_EINVAL;
    struct {
        int64_t &stride;
        int size;
    } axes[] = {{c.page_stride, c.pages}, {c.token_stride, c.page}, {c.head_stride, kv}};
    for (auto &x : axes) {
        if (x.size == 1) x.stride = 0;
        else if (x.stride < dim || x.stride % unit != 0) return STEP_EINVAL;
        else if (x.stride >= kMostCacheStride) return STEP_EUNSUPPORTED;
    }
    return STEP_OK;
}

size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

// What an attention's workspace holds: tickets, notes of split tiles, what the
// rows bring from their prefixes, results of pieces.
struct AttendPlan {
    size_t joins, state, sums, pieces, total;
};
int few_groups(int dim) { return dim <= 64 ? st::kFewGroups : dim <= 128 ? 512 : 256; }
int many_groups(int dim) { return dim <= 128 ? st::kManyGroups : 256; }
AttendPlan attend_plan(int n, int heads, int dim, bool prefixes) {
    AttendPlan p{};
    const size_t rows = (size_t)n * heads, few = few_groups(dim) * st::piece_floats(st::kFewRows, dim),
                 many = many_groups(dim) * st::piece_floats(st::kManyRows, dim);
    p.joins = st::kTicketBytes;
    p.state = p.joins + up256(st::kManyGroups * sizeof(st::Join));
    p.sums = p.state + (prefixes ? up256(rows * 2 * sizeof(float)) : 0);
    p.pieces = p.sums + (prefixes ? up256(rows * st::padded_dim(dim) * sizeof(float)) : 0);
    p.total = p.pieces + up256(2 * (few > many ? few : many) * sizeof(float));
    return p;
}

// Workgroups for a call: no more than the chip holds at once, nor than there
// are least ranges in the most that the tables allow.
int groups_for(int64_t tiles, int64_t cost, int least, int most) {
    const int64_t g = (tiles * cost + least - 1) / least;
    return g < 1 ? 1 : g > most ? most : (int)g;
}

hipError_t launch(st::AttendArgs &a, int64_t rows_of_job, hipStream_t stream) {
    // Few rows: 16 a tile, the waves share the keys among them.  Many: 128, the
    // waves share the rows.
    const bool few = a.each <= st::kFewRows && rows_of_job * a.each <= st::kFewRows;
    const int tokens = (few ? st::kFewRows : st::kManyRows) / a.each;
    const int64_t tiles = ((int64_t)a.n / tokens + a.jobs) * a.kv, keys = (int64_t)a.table_cols * a.cache.page;
    a.groups_of_threads = few ? groups_for(tiles, (a.cache.k_scale ? st::kFewFixed8 : st::kFewFixed) + keys, st::kFewLeast, few_groups(a.dim))
                              : groups_for(tiles, st::kManyFixed + keys, st::kManyLeast, many_groups(a.dim));
    return few ? st::launch_attend_few(a, stream) : st::launch_attend_many(a, stream);
}

}  // namespace

extern "C" {

int step_kv_append(const uint16_t *q, int64_t ldq, const uint16_t *k, int64_t ldk, const uint16_t *v, int64_t ldv,
                   int32_t n, int32_t heads, int32_t kv_heads, int32_t dim, const int32_t *positions,
                   const float *rotation, int32_t rotation_rows, int32_t rot, int32_t neighbours, const int32_t *place,
                   void *k_cache, void *v_cache, int64_t page_stride, int64_t token_stride, int64_t head_stride,
                   int32_t pages, int32_t page, const float *k_scale, const float *v_scale, uint16_t *q_out,
                   int64_t ldo, void *stream) {
    if (int rc = check_heads(n, q ? heads : kv_heads, kv_heads, dim)) return rc;
    if (rot < 0 || rot > dim || rot % 16 != 0) return STEP_EINVAL;
    st::CacheArgs c{k_cache, v_cache, page_stride, token_stride, head_stride, pages, page, k_scale, v_scale};
    if (int rc = check_cache(c, kv_heads, dim)) return rc;
    if (n == 0) return STEP_OK;
    const int64_t wide = (int64_t)heads * dim, kv_wide = (int64_t)kv_heads * dim;
    if (!aligned(k, 16) || !aligned(v, 16) || ldk < kv_wide || ldk % 8 != 0 || ldv < kv_wide || ldv % 8 != 0)
        return STEP_EINVAL;
    if ((q == nullptr) != (q_out == nullptr)) return STEP_EINVAL;
    if (q && (!aligned(q, 16) || !aligned(q_out, 16) || ldq < wide || ldq % 8 != 0 || ldo < wide || ldo % 8 != 0))
        return STEP_EINVAL;
    if (q && q == q_out && ldq != ldo) return STEP_EINVAL;
    if (ldk >= kMostStride || ldv >= kMostStride || (q && (ldq >= kMostStride || ldo >= kMostStride)))
        return STEP_EUNSUPPORTED;
    if (rot && (!aligned(positions, 4) || !aligned(rotation, 16) || rotation_rows < 1)) return STEP_EINVAL;
    if (!aligned(place, 4)) return STEP_EINVAL;
    const st::AppendArgs a{q,        k,         v,        ldq,           ldk, ldv,        n,     heads, kv_heads,
                           dim,      positions, rotation, rotation_rows, rot, neighbours, place, c,     q_out,
                           ldo};
    return launched(st::launch_kv_append(a, static_cast<hipStream_t>(stream)));
}

size_t step_paged_attention_workspace_bytes(int32_t n, int32_t heads, int32_t kv_heads, int32_t dim,
                                            int32_t prefixes) {
    if (check_heads(n, heads, kv_heads, dim) != STEP_OK || prefixes < 0) return 0;
    return attend_plan(n, heads, dim, prefixes > 0).total;
}

int step_paged_attention(const uint16_t *q, int64_t ldq, int32_t n, int32_t requests, int32_t heads, int32_t kv_heads,
                         int32_t dim, const void *k_cache, const void *v_cache, int64_t page_stride,
                         int64_t token_stride, int64_t head_stride, int32_t pages, int32_t page, const float *k_scale,
                         const float *v_scale, const int32_t *table, int64_t ld_table, int32_t table_cols,
                         const int32_t *lens, const int32_t *starts, int32_t max_rows, int32_t causal, float scale,
                         int32_t prefixes, const int32_t *prefix_table, int64_t ld_prefix_table, int32_t prefix_cols,
                         const int32_t *prefix_lens, const int32_t *prefix_starts, uint16_t *out, int64_t ldo,
                         float *lse, void *ws, size_t ws_bytes, void *stream) {
    if (int rc = check_heads(n, heads, kv_heads, dim)) return rc;
    if (requests < 0 || (!starts && requests != n) || (starts && max_rows < 1)) return STEP_EINVAL;
    if (requests > STEP_MAX_REQUESTS || prefixes > STEP_MAX_REQUESTS) return STEP_EUNSUPPORTED;
    st::CacheArgs c{const_cast<void *>(k_cache), const_cast<void *>(v_cache), page_stride, token_stride, head_stride,
                    pages, page, k_scale, v_scale};
    if (int rc = check_cache(c, kv_heads, dim)) return rc;
    if (!(scale >= 1e-30f && scale <= 1e30f)) return STEP_EINVAL;
    if (table_cols < 0 || ld_table < table_cols || prefixes < 0) return STEP_EINVAL;
    if ((int64_t)table_cols * page > kMostKeys || ld_table >= kMostStride) return STEP_EUNSUPPORTED;
    if (prefixes > 0) {
        if (prefix_cols < 0 || ld_prefix_table < prefix_cols) return STEP_EINVAL;
        if ((int64_t)prefix_cols * page > kMostKeys || ld_prefix_table >= kMostStride) return STEP_EUNSUPPORTED;
    }
    if (n == 0 || requests == 0) return STEP_OK;
    const int64_t wide = (int64_t)heads * dim;
    if (!aligned(q, 16) || ldq < wide || ldq % 8 != 0 || !aligned(out, 16) || ldo < wide || ldo % 8 != 0)
        return STEP_EINVAL;
    if (ldq >= kMostStride || ldo >= kMostStride) return STEP_EUNSUPPORTED;
    if (!aligned(lens, 4) || !aligned_or_null(starts, 4) || !aligned_or_null(lse, 4)) return STEP_EINVAL;
    if (table_cols > 0 && !aligned(table, 4)) return STEP_EINVAL;
    if (prefixes > 0 && (!aligned(prefix_lens, 4) || !aligned(prefix_starts, 4) ||
                         (prefix_cols > 0 && !aligned(prefix_table, 4))))
        return STEP_EINVAL;
    const AttendPlan plan = attend_plan(n, heads, dim, prefixes > 0);
    if (!aligned(ws, 16) || ws_bytes < plan.total) return STEP_EWORKSPACE;

    st::AttendArgs a{};
    a.q = q;
    a.ldq = ldq;
    a.n = n;
    a.kv = kv_heads;
    a.each = heads / kv_heads;
    a.dim = dim;
    a.scale = scale * 1.44269504088896340736f;
    a.cache = c;
    const int unit = k_scale ? 16 : 8;
    a.page_units = (uint32_t)(c.page_stride / unit);
    a.token_units = (uint32_t)(c.token_stride / unit);
    a.div = st::page_div(page);
    a.requests = requests;
    a.starts = starts;
    a.out = out;
    a.ldo = ldo;
    a.lse = lse;
    char *const base = static_cast<char *>(ws);
    a.tickets = reinterpret_cast<int32_t *>(base);
    a.zeros = base + st::kZerosAt;
    a.joins = reinterpret_cast<st::Join *>(base + plan.joins);
    a.pieces = reinterpret_cast<float *>(base + plan.pieces);
    const hipStream_t on = static_cast<hipStream_t>(stream);
    st::AttendArgs own = a;
    own.jobs = requests;
    own.lens = lens;
    own.table = table;
    own.ld_table = ld_table;
    own.table_cols = table_cols;
    own.causal = causal;
    if (prefixes > 0) {
        // the prefixes first, each for all its requests' rows; every row's
        // softmax then goes on over the request's own keys
        float *const state = reinterpret_cast<float *>(base + plan.state), *const sums =
            reinterpret_cast<float *>(base + plan.sums);
        st::AttendArgs pre = a;
        pre.jobs = prefixes + 2;
        pre.groups = prefix_starts;
        pre.lens = prefix_lens;
        pre.table = prefix_table;
        pre.ld_table = ld_prefix_table;
        pre.table_cols = prefix_cols;
        pre.state_out = state;
        pre.sums_out = sums;
        if (int rc = launched(launch(pre, n / prefixes > 0 ? n / prefixes : 1, on))) return rc;
        own.state_in = state;
        own.sums_in = sums;
    }
    return launched(launch(own, starts ? max_rows : 1, on));
}

}  // extern "C"
