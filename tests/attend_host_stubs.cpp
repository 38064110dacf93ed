// attend_host_stubs.cpp -- host stand-ins for the launchers of the paged cache's
// operators, linked with attend_abi.cpp into a host-only build of its entry
// points, and the division of an attention call among workgroups as the device
// makes it.  Nothing is launched and no device address is read.
#include "../tenant_lora_serving_amd/csrc/attend_kernels.h"

namespace {
struct Launch {
    int kind, groups, jobs, brings, leaves;  // kind 0: few rows, 1: many rows, 2: append
} g_launches[8];
int g_count;
void note(int kind, const st::AttendArgs &a) {
    if (g_count < 8)
        g_launches[g_count++] = {kind, a.groups_of_threads, a.jobs, a.state_in != nullptr, a.state_out != nullptr};
}
}  // namespace

namespace st {
hipError_t launch_kv_append(const AppendArgs &, hipStream_t) {
    if (g_count < 8) g_launches[g_count++] = {2, 0, 0, 0, 0};
    return hipSuccess;
}
hipError_t launch_attend_few(const AttendArgs &a, hipStream_t) { return note(0, a), hipSuccess; }
hipError_t launch_attend_many(const AttendArgs &a, hipStream_t) { return note(1, a), hipSuccess; }
}  // namespace st

extern "C" {
void stub_reset(void) { g_count = 0; }
int stub_count(void) { return g_count; }
void stub_launch(int i, int *to) {
    const Launch &l = g_launches[i];
    to[0] = l.kind, to[1] = l.groups, to[2] = l.jobs, to[3] = l.brings, to[4] = l.leaves;
}
int stub_page_of(int page, int key) { return st::page_of(st::page_div(page), key); }

// The pieces of a call: 12 numbers each (workgroup, job, head, tile, keys of the
// tile, lo, hi, begins, split, first, count, slot); returns how many there are,
// or -1 if `most` is too small.
int stub_divide(int jobs, const int *rows, const int *lens, int kv, int tokens, int causal, int groups, int fixed, int least,
                int whole, int step, int *to, int most) {
    auto cost_of = [&](int j) {
        const st::Span s{rows[j], lens[j]};
        return st::tiles_cost(s, tokens, causal, fixed, st::tiles_of(s.rows, tokens));
    };
    int64_t total = 0;
    for (int j = 0; j < jobs; ++j) total += kv * cost_of(j);
    const st::Ranges r = st::ranges_of(total, groups, fixed, least, whole);
    int n = 0;
    for (int w = 0; w < groups; ++w) {
        const int64_t begin = w * r.size, end = begin + r.size < total ? begin + r.size : total;
        if (begin >= total) continue;
        int j = 0;
        int64_t base = 0;
        while (begin >= base + kv * cost_of(j)) base += kv * cost_of(j++);
        const int64_t head = cost_of(j);
        int g = (int)((begin - base) / head);
        int i = st::tile_at({rows[j], lens[j]}, tokens, causal, fixed, begin - base - g * head);
        int64_t at = base + g * head + st::tiles_cost({rows[j], lens[j]}, tokens, causal, fixed, i);
        for (;;) {
            const st::Span s{rows[j], lens[j]};
            const int keys = st::tile_keys(s, tokens, causal, i);
            const st::Piece p = st::piece_of(r, w, at, keys, step);
            if (p.mine) {
                if (n == most) return -1;
                const int slot = p.split ? st::piece_slot(r, w, at) : 0;
                const int v[12] = {w,    j,        g,        i,        keys,    p.lo,
                                   p.hi, p.begins, p.split, p.first, p.count, p.split && slot != p.slot ? -1 : p.slot};
                for (int k = 0; k < 12; ++k) to[12 * n + k] = v[k];
                ++n;
            }
            at += fixed + keys;
            if (at >= end) break;
            if (++i < st::tiles_of(s.rows, tokens)) continue;
            i = 0;
            if (++g < kv) continue;
            g = 0;
            do ++j;
            while (rows[j] == 0);
        }
    }
    return n;
}
}
