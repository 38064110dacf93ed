// step_host_stubs.cpp -- host stand-ins for the launchers of the serving-step
// operators, linked with step_abi.cpp and step_plan.cpp into a host-only build
// of step.h's C ABI.  Each stub counts its calls; nothing is launched and no
// device address is read, so accepted calls can be made with made-up pointers.
#include "../tenant_lora_serving_amd/csrc/step_kernels.h"

namespace {
enum Kind { kNorm, kLinear, kScore, kKinds };
long long g_calls[kKinds];
}  // namespace

extern "C" {
void stub_reset(void) {
    for (long long &c : g_calls) c = 0;
}
// The tiles of a call's product, as rows * 1000 + columns.
int stub_linear_tile(int n, int k, int out, int num_slices, int R, int fp8) {
    static const int kTiles[] = {16016, 16064, 32016, 32048, 48064, 64032, 64064, 64096, 128128, 256256};
    return kTiles[st::linear_tile(n, k, out, fp8 != 0, st::linear_plan(n, out, num_slices, R).sorted)];
}
long long stub_calls(int kind) { return kind >= 0 && kind < kKinds ? g_calls[kind] : -1; }
}

namespace st {
hipError_t launch_rms_norm(const NormArgs &, hipStream_t) { return ++g_calls[kNorm], hipSuccess; }
hipError_t launch_lora_linear(const LinearArgs &, const LinearPlan &, void *, hipStream_t) {
    return ++g_calls[kLinear], hipSuccess;
}
hipError_t launch_token_logprobs(const ScoreArgs &, const ScorePlan &, void *, hipStream_t) {
    return ++g_calls[kScore], hipSuccess;
}
}  // namespace st
