// Sanitizer driver for the host logic of the feed-forward entry points (test
// infrastructure): csrc/ffn_api.cpp is compiled with the address and undefined
// behaviour sanitizers together with this file, which stands in for the
// kernels' launchers and the current device. Every entry point is called on
// edge and random arguments; the launchers check what reaches them: workspace
// ranges inside the caller's and apart from each other, launches below 2^32
// threads, k's covered. Pointers are stand-ins that nothing reads.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <utility>
#include <vector>

#include "context.h"
#include "ffn.h"
#include "tlg.h"

static uint64_t rng_state = 0x243f6a8885a308d3ull;
static uint64_t rnd() {
    rng_state ^= rng_state >> 12;
    rng_state ^= rng_state << 25;
    rng_state ^= rng_state >> 27;
    return rng_state * 2685821657736338717ull;
}
static int failures = 0;
static char where[256];
static void check(bool ok, const char *what) {
    if (!ok && failures++ < 20) fprintf(stderr, "ffn_plan_driver: %s: %s\n", what, where);
}

// The caller's workspace and what the call used of it.
static __int128 ws_begin, ws_end;
static std::vector<std::pair<__int128, __int128>> used;
static long launches;
static void use(const void *p, __int128 bytes) {
    const __int128 b = (__int128)(uintptr_t)p;
    check(bytes >= 0 && b >= ws_begin && b + bytes <= ws_end, "workspace range outside the workspace");
    for (const auto &u : used) check(b + bytes <= u.first || b >= u.second, "workspace ranges overlap");
    used.push_back({b, b + bytes});
}
static void threads(__int128 n) { check(n > 0 && n < ((__int128)1 << 32), "threads of a launch"); }
static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

static const int kBM[] = {256, 256, 128, 128, 64}, kBN[] = {256, 128, 128, 128, 128};
static __int128 groups(int config, const tlg::FfnPanelCall &c) {
    check(config >= 0 && config < tlg::FFN_PANEL_CONFIGS, "tile shape");
    const int bn = c.p.mode == tlg::FFN_GATED ? kBN[config] / 2 : kBN[config];
    const int64_t tiles = ceil_div(c.p.M, kBM[config]) * ceil_div(c.p.N, bn) * (c.p.mode == tlg::FFN_PAIR ? 2 : 1);
    check(c.splits >= 1, "parts");
    check(c.kmain >= 0 && c.kmain <= c.p.K, "kmain");
    const int64_t chunk = c.p.type == tlg::FFN_I8 ? 16 : 8;
    check(c.p.K - c.kmain <= chunk, "k's left to stage");
    if (c.splits < 2) return tiles;
    check(c.whole >= 0 && c.whole < tiles, "whole tiles");
    use(c.part, (__int128)(tiles - c.whole) * c.splits * (c.p.M < kBM[config] ? c.p.M : kBM[config]) * kBN[config] * 4);
    return c.whole + (tiles - c.whole) * c.splits;
}
static hipError_t panel(int config, const tlg::FfnPanelCall &c) {
    ++launches;
    threads(groups(config, c) * 256);
    // the parts of one product are joined before the next product runs
    if (c.splits > 1) used.pop_back();
    return hipSuccess;
}
static hipError_t grads(int config, const tlg::FfnPanelCall &x, const tlg::FfnPanelCall &w) {
    ++launches;
    check(x.p.mode == tlg::FFN_SUM2 && w.p.mode == tlg::FFN_PAIR, "products of a backward pass");
    threads((groups(config, x) + groups(config, w)) * 256);
    return hipSuccess;
}
static void packs(const tlg::FfnPack &p) {
    check(p.count >= 0 && p.count <= 3 && p.pitch >= 0 && p.pitch % 16 == 0, "copies");
    for (int i = 0; i < p.count; ++i) {
        check(p.row_bytes[i] <= p.pitch && p.ld_bytes[i] >= p.row_bytes[i], "rows of a copy");
        use(p.dst[i], (__int128)p.rows[i] * p.pitch);
    }
}

hipError_t hipGetDevice(int *d) {
    *d = 0;
    return hipSuccess;
}
namespace tlg {
hipError_t launch_ffn_general(const FfnProduct &p, hipStream_t) {
    ++launches;
    threads((__int128)ceil_div(p.M, 64) * ceil_div(p.N, 64) * 256);
    return hipSuccess;
}
hipError_t launch_ffn_panel_f16(int config, const FfnPanelCall &c, hipStream_t) { return panel(config, c); }
hipError_t launch_ffn_panel_bf16(int config, const FfnPanelCall &c, hipStream_t) { return panel(config, c); }
hipError_t launch_ffn_panel_i8(int config, const FfnPanelCall &c, hipStream_t) { return panel(config, c); }
hipError_t launch_ffn_panel_grads_f16(int config, const FfnPanelCall &x, const FfnPanelCall &w, bool, hipStream_t) {
    return grads(config, x, w);
}
hipError_t launch_ffn_panel_grads_bf16(int config, const FfnPanelCall &x, const FfnPanelCall &w, bool, hipStream_t) {
    return grads(config, x, w);
}
hipError_t launch_ffn_skinny(const FfnProduct &p, int kmain, hipStream_t) {
    ++launches;
    check(p.M >= 1 && p.M <= 64 && kmain >= 0 && kmain <= p.K, "strips");
    threads((__int128)ceil_div(p.N, 16) * 512);
    return hipSuccess;
}
hipError_t launch_quantize_i8(int, int64_t, int64_t, const void *, int64_t, int8_t *, int64_t, float *, hipStream_t) {
    ++launches;
    return hipSuccess;
}
hipError_t launch_ffn_pack(const FfnPack &p, hipStream_t) {
    packs(p);
    return hipSuccess;
}
hipError_t launch_ffn_gate_grad(int, int, int M, int N, const void *, int64_t, const void *, int64_t, const void *,
                                int64_t, void *dG, void *dU, int64_t pitch, FfnGateScale *scale, const FfnPack &copies,
                                hipStream_t) {
    check(pitch >= N && pitch % 64 == 0, "pitch of the gradients' planes");
    use(scale, sizeof *scale);
    use(dG, (__int128)M * pitch * 2);
    use(dU, (__int128)M * pitch * 2);
    packs(copies);
    return hipSuccess;
}
hipError_t launch_ffn_zero(void *, int64_t, int64_t, int64_t, hipStream_t) { return hipSuccess; }
}  // namespace tlg

static const int64_t kSizes[] = {0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 255, 256, 257, 300, 1000,
                                 1537, 2049, 3001, 4096, 8192, 14336, 65536, 131071, 1 << 20, 1 << 27, 1 << 30,
                                 (1ll << 31) - 1025, (1ll << 31) - 1024, 1ll << 31, 1ll << 40, -1};
static int64_t size() {
    const uint64_t r = rnd();
    if (r % 3 == 0) return (int64_t)(rnd() % 9000);
    return kSizes[r / 3 % (sizeof kSizes / sizeof kSizes[0])];
}
// A leading dimension: the row's width, a wider one, or the largest there is.
static int64_t ld(int64_t cols) {
    const int64_t c = cols > 1 ? cols : 1;
    switch (rnd() % 8) {
        case 0: return c + (int64_t)(rnd() % 100);
        case 1: return rnd() % 4 ? c : INT64_MAX - (int64_t)(rnd() % 3);
        case 2: return rnd() % 4 ? c : (int64_t)1 << (40 + rnd() % 23);
        default: return c;
    }
}
static void *at(int bytes) { return (void *)(uintptr_t)((1ull << 40) + (rnd() % 2 ? 0 : bytes * (rnd() % 64))); }
static void *workspace(int64_t bytes) {
    used.clear();
    ws_begin = bytes ? (__int128)1 << 44 : 0;
    ws_end = ws_begin + bytes;
    return (void *)(uintptr_t)ws_begin;
}

int main() {
    tlg_context ctx = {};
    ctx.cus = 256;
    long served = 0, calls = 0;
    for (int t = 0; t < 300000; ++t) {
        const int64_t M = size(), N = size(), K = size();
        const int config = rnd() % 2 ? -1 : (int)(rnd() % 24) - 1;
        const int dtype = rnd() % 2 ? TLG_F16 : TLG_BF16, act = 1 + (int)(rnd() % 4);
        snprintf(where, sizeof where, "M=%lld N=%lld K=%lld config=%d call %d", (long long)M, (long long)N,
                 (long long)K, config, t);
        const long before = launches;
        tlg_status st = TLG_SUCCESS;
        int64_t want = 0;
        const auto room = [&](int64_t w) {
            check(w >= 0, "workspace size");
            want = w;
            switch (rnd() % 8) {
                case 0: return (int64_t)0;
                case 1: return (int64_t)(rnd() % (64 << 20));
                case 2: return config >= 0 ? (int64_t)1 << 34 : w;
                case 3: return (int64_t)(rnd() % 4 ? 1ll << 40 : INT64_MAX >> (1 + rnd() % 3));
                default: return w > INT64_MAX / 2 ? INT64_MAX / 2 : w;
            }
        };
        switch (rnd() % 5) {
            case 0: {
                const int64_t bytes = room(tlg_gated_ffn_workspace(M, N, K));
                const bool save = rnd() % 2;
                const tlg_gated_ffn_desc d = {M, N, K, at(2), ld(K), at(2), ld(K), at(2), ld(K), at(2), ld(N),
                                              save ? at(2) : nullptr, ld(N), save ? at(2) : nullptr, ld(N)};
                st = tlg_gated_ffn_variant(&ctx, config, dtype, act, &d, workspace(bytes), bytes, nullptr);
                break;
            }
            case 1: {
                const int64_t bytes = room(tlg_gated_ffn_backward_workspace(M, N, K));
                const bool x = rnd() % 8, w = rnd() % 8;
                const tlg_gated_ffn_grad_desc d = {M, N, K, at(2), ld(N), at(2), ld(K), at(2), ld(K), at(2), ld(K),
                                                   at(2), ld(N), at(2), ld(N), x ? at(2) : nullptr, ld(K),
                                                   w ? at(2) : nullptr, ld(K), w ? at(2) : nullptr, ld(K)};
                st = tlg_gated_ffn_backward_variant(&ctx, config, dtype, act, &d, workspace(bytes), bytes, nullptr);
                break;
            }
            case 2: {
                const int64_t bytes = room(tlg_gemm_i8_workspace(M, N, K));
                st = tlg_gemm_i8_variant(&ctx, config, 1 + (int)(rnd() % 3), (int)(rnd() % 2), M, N, K,
                                         (const int8_t *)at(1), ld(K), (const float *)at(4), (const int8_t *)at(1),
                                         ld(K), (const float *)at(4), at(4), ld(N), workspace(bytes), bytes, nullptr);
                break;
            }
            case 3: {
                const int64_t bytes = room(tlg_gated_ffn_i8_workspace(M, N, K));
                const tlg_gated_ffn_desc d = {M, N, K, at(1), ld(K), at(1), ld(K), at(1), ld(K), at(2), ld(N),
                                              nullptr, ld(N), nullptr, ld(N)};
                st = tlg_gated_ffn_i8_variant(&ctx, config, dtype, act, &d, (const float *)at(4), (const float *)at(4),
                                              (const float *)at(4), workspace(bytes), bytes, nullptr);
                break;
            }
            default: {
                const int64_t ws = rnd() % 2 ? 0 : (int64_t)1 << (rnd() % 62);
                int32_t splits = 0;
                const int product = (int)(rnd() % 8) - 1, cfg = tlg_ffn_plan(product, M, N, K, (int)(rnd() % 4), ws, &splits);
                check(cfg >= -1 && (cfg < 0 || (splits >= 1 && tlg_ffn_config_name(cfg)[0])), "plan");
                continue;
            }
        }
        ++calls;
        check(st == TLG_SUCCESS || launches == before, "a refused call launched");
        check(st != TLG_ERROR_HIP, "status");
        check(want < ((int64_t)1 << 62) || st != TLG_SUCCESS || launches == before, "workspace of no real call");
        served += st == TLG_SUCCESS && launches > before;
    }
    check(served > calls / 20, "calls that launch");
    if (failures) return 1;
    printf("ffn_plan_driver: ok (%ld of %ld calls launched)\n", served, calls);
    return 0;
}
