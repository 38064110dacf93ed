// step_abi.cpp -- step.h's entry points: host-side validation and launches.
// Nothing here allocates, frees or synchronizes; every check runs before any
// launch.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/step.h"
#include "step_kernels.h"

namespace {

bool aligned(const void *p, unsigned to) { return p && (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool aligned_or_null(const void *p, unsigned to) { return !p || aligned(p, to); }
int launched(hipError_t e) { return e == hipSuccess ? STEP_OK : STEP_ELAUNCH; }

// n * ld >= limit, for any ld (the product of a long stride would wrap around).
bool spans(int n, int64_t ld, int64_t limit) { return n > 0 && (ld >= limit || n * ld >= limit); }

int check_score(int n, int v, int top) {
    if (n < 0 || v < 1 || top < 0) return STEP_EINVAL;
    if (n > st::kScoreMaxRows || v > (1 << 20) || top > STEP_MAX_TOP) return STEP_EUNSUPPORTED;
    return STEP_OK;
}

int check_linear(int n, int k, long long out, int num_slices, int R) {
    if (n < 0 || k < 16 || k % 16 != 0 || out < 8 || out % 8 != 0) return STEP_EINVAL;
    if (num_slices < 1 || num_slices > st::kMaxSlices) return STEP_EINVAL;
    if (n > (1 << 18) || k > (1 << 18) || out > (1 << 24)) return STEP_EUNSUPPORTED;
    if (R < 8 || R > st::kMaxRank || R % 8 != 0) return STEP_EUNSUPPORTED;
    return STEP_OK;
}

}  // namespace

extern "C" {

int step_rms_norm(const uint16_t *x, int64_t ldx, const uint16_t *residual, int64_t ldr, const uint16_t *weight,
                  int32_t n, int32_t h, float eps, uint16_t *residual_out, uint16_t *y, uint8_t *q, float *q_scale,
                  void *stream) {
    if (n < 0 || h < 8 || h % 8 != 0 || !(eps >= 0.0f) || std::isinf(eps)) return STEP_EINVAL;
    if (n > (1 << 24) || h > 32768) return STEP_EUNSUPPORTED;
    if (n == 0) return STEP_OK;
    if (!aligned(x, 16) || ldx < h || ldx % 8 != 0 || !aligned(weight, 16)) return STEP_EINVAL;
    if ((residual == nullptr) != (residual_out == nullptr)) return STEP_EINVAL;
    if (residual && (!aligned(residual, 16) || ldr < h || ldr % 8 != 0 || !aligned(residual_out, 16)))
        return STEP_EINVAL;
    if (residual_out == residual && residual && ldr != h) return STEP_EINVAL;
    if (!y && !q) return STEP_EINVAL;
    if (!aligned_or_null(y, 16) || !aligned_or_null(q, 8) || !aligned_or_null(q_scale, 4)) return STEP_EINVAL;
    if ((q == nullptr) != (q_scale == nullptr)) return STEP_EINVAL;
    const st::NormArgs a{x, ldx, residual, ldr, weight, n, h, eps, residual_out, y, q, q_scale};
    return launched(st::launch_rms_norm(a, static_cast<hipStream_t>(stream)));
}

size_t step_lora_linear_workspace_bytes(int32_t n, int32_t k, int32_t out, int32_t num_slices, int32_t max_rank) {
    if (check_linear(n, k, out, num_slices, max_rank) != STEP_OK) return 0;
    return st::linear_plan(n, out, num_slices, max_rank).total_bytes;
}

int step_lora_linear(const uint16_t *x, int64_t ldx, int32_t n, int32_t k, const uint8_t *xq, int64_t ldxq,
                     const float *x_scale, const void *w, const float *w_scale, const uint16_t *a_pool,
                     const uint16_t *b_pool, const float *scale, int32_t num_slots, int32_t num_slices,
                     const int32_t *slice_sizes, int32_t max_rank, const int32_t *slot, uint16_t *y, int64_t ldy,
                     void *ws, size_t ws_bytes, void *stream) {
    st::LinearArgs a{};
    if (!slice_sizes || num_slices < 1 || num_slices > st::kMaxSlices) return STEP_EINVAL;
    long long out = 0;
    for (int l = 0; l < num_slices; ++l) {
        if (slice_sizes[l] <= 0 || slice_sizes[l] % 8 != 0) return STEP_EINVAL;
        out += slice_sizes[l];
        if (out > (1 << 24)) return STEP_EUNSUPPORTED;
        a.slice_off[l + 1] = (int)out;
    }
    for (int l = num_slices + 1; l <= st::kMaxSlices; ++l) a.slice_off[l] = (int)out;
    if (int rc = check_linear(n, k, out, num_slices, max_rank)) return rc;
    if (num_slots < 1) return STEP_EINVAL;
    if (num_slots > st::kMaxSlots) return STEP_EUNSUPPORTED;
    if (ldx < k || ldx % 8 != 0 || ldy < out || ldy % 8 != 0) return STEP_EINVAL;
    if (xq && (ldxq < k || ldxq % 16 != 0)) return STEP_EINVAL;
    if (xq && k <= st::kExactK && n * out >= 100000000000LL) return STEP_EUNSUPPORTED;  // (64-row tiles: the grid)
    if (spans(n, ldx, 1LL << 30) || (xq && spans(n, ldxq, 1LL << 31))) return STEP_EUNSUPPORTED;
    if (n == 0) return STEP_OK;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(a_pool, 16) || !aligned(b_pool, 16) || !aligned(scale, 4) ||
        !aligned(slot, 4) || !aligned(y, 16))
        return STEP_EINVAL;
    if (!aligned_or_null(xq, 16) || !aligned_or_null(x_scale, 4) || !aligned_or_null(w_scale, 4)) return STEP_EINVAL;
    if ((xq == nullptr) != (x_scale == nullptr) || (xq == nullptr) != (w_scale == nullptr)) return STEP_EINVAL;
    const st::LinearPlan plan = st::linear_plan(n, (int)out, num_slices, max_rank);
    if (!ws || ws_bytes < plan.total_bytes || !aligned(ws, 16)) return STEP_EWORKSPACE;
    a.x = x;
    a.ldx = ldx;
    a.n = n;
    a.k = k;
    a.xq = xq;
    a.ldxq = ldxq;
    a.x_scale = x_scale;
    a.w = w;
    a.w_scale = w_scale;
    a.a_pool = a_pool;
    a.b_pool = b_pool;
    a.scale = scale;
    a.num_slots = num_slots;
    a.num_slices = num_slices;
    a.R = max_rank;
    a.slot = slot;
    a.y = y;
    a.ldy = ldy;
    return launched(st::launch_lora_linear(a, plan, ws, static_cast<hipStream_t>(stream)));
}

size_t step_token_logprobs_workspace_bytes(int32_t n, int32_t v, int32_t top) {
    if (check_score(n, v, top) != STEP_OK) return 0;
    return n > 0 ? st::score_workspace_bytes(n, v, top) : 0;
}

int step_token_logprobs(const void *logits, int64_t ld, int32_t fp32, int32_t n, int32_t v, const int32_t *tokens,
                        int32_t top, float *logprob, int32_t *rank, float *entropy, int32_t *top_ids,
                        float *top_logprobs, void *ws, size_t ws_bytes, void *stream) {
    if (int rc = check_score(n, v, top)) return rc;
    if (ld < v) return STEP_EINVAL;
    if (n == 0) return STEP_OK;
    if (!aligned(logits, fp32 ? 4 : 2) || !aligned(tokens, 4) || !aligned(logprob, 4) || !aligned(rank, 4) ||
        !aligned(entropy, 4))
        return STEP_EINVAL;
    if (top > 0 ? (!aligned(top_ids, 4) || !aligned(top_logprobs, 4)) : (top_ids || top_logprobs))
        return STEP_EINVAL;
    const st::ScorePlan plan = st::score_plan(n, v, top, fp32);
    if (plan.total_bytes && (!aligned(ws, 16) || ws_bytes < plan.total_bytes)) return STEP_EWORKSPACE;
    const st::ScoreArgs a{logits, ld, fp32, n, v, tokens, top, logprob, rank, entropy, top_ids, top_logprobs};
    return launched(st::launch_token_logprobs(a, plan, ws, static_cast<hipStream_t>(stream)));
}

const char *step_status_string(int status) {
    switch (status) {
        case STEP_OK: return "ok";
        case STEP_EINVAL: return "bad pointer, size, alignment or leading dimension";
        case STEP_EUNSUPPORTED: return "unsupported shape";
        case STEP_EWORKSPACE: return "workspace missing or too small";
        case STEP_ELAUNCH: return "the HIP runtime refused a launch";
        default: return "unknown status";
    }
}

}  // extern "C"
