// C ABI of the gated feed-forward block and its 8-bit products: argument
// checks, kernel choice, launches. include/tlg.h holds the contracts.
#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "context.h"
#include "ffn.h"
#include "ffn_panel.h"
#include "tlg.h"

namespace {

using tlg::FfnProduct;

constexpr int64_t kMaxDim = (1ll << 31) - 1024;
// |code| <= 128, so K products of two codes stay within 2^14 K < 2^31
constexpr int64_t kMaxK8 = 131071;

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// A matrix of `rows` rows of `cols` elements of `bytes` bytes: its leading
// dimension, and its pointer unless nothing is read or written through it.
bool matrix_ok(const void *p, int64_t rows, int64_t cols, int64_t ld, int bytes) {
    if (ld < (cols > 1 ? cols : 1)) return false;
    return rows == 0 || cols == 0 || (p && aligned(p, bytes));
}

bool is16(int32_t dtype) { return dtype == TLG_F16 || dtype == TLG_BF16; }
bool is_act(int32_t act) { return act >= TLG_ACT_SILU && act <= TLG_ACT_RELU; }
int type_of(int32_t dtype) { return dtype == TLG_BF16 ? tlg::FFN_BF16 : tlg::FFN_F16; }
int bytes_of(int32_t dtype) { return dtype == TLG_F32 ? 4 : 2; }

// The handle's device must be current.
tlg_status check_device(tlg_handle h) {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess) return TLG_ERROR_HIP;
    return dev == h->device ? TLG_SUCCESS : TLG_ERROR_INVALID_VALUE;
}

tlg_status status_of(hipError_t e) { return e == hipSuccess ? TLG_SUCCESS : TLG_ERROR_HIP; }

// Kernel configurations (tlg_ffn_config_name): the general kernel, the
// pipelined kernel's tile shapes, 16-token strips, the tile shapes with the
// sum in as many parts as fit, those on aligned copies of the operands, and
// those that take both products of a backward pass in one launch.
enum {
    CFG_GENERAL = 0,
    CFG_PANEL = 1,  // + a tile shape
    CFG_SKINNY = CFG_PANEL + tlg::FFN_PANEL_CONFIGS,
    CFG_SPLIT = CFG_SKINNY + 1,  // + a tile shape
    CFG_PACKED = CFG_SPLIT + tlg::FFN_PANEL_CONFIGS,  // + a tile shape
    CFG_BOTH = CFG_PACKED + tlg::FFN_PANEL_CONFIGS,  // + a tile shape, but the 64-token one
    CFG_COUNT = CFG_BOTH + tlg::FFN_PANEL_CONFIGS - 1
};

// Tile shapes with their measured times in microseconds: a 128-byte-deep
// stage with a CU's work-groups resident (`pair`: a lone one of two), and what
// a round of work-groups costs besides (first loads, results). From products
// of one to fourteen rounds and one to 112 stages, bf16 and int8 alike, for
// example: 256 x 256, 224 tiles of 64 stages 97; 256 x 128, 224 tiles 72; 128 x
// 128, 448 tiles 82 in pairs; deep, 224 tiles 55; 64 x 128, 32 tiles of 112
// stages 44; 192 tiles of 256 x 256 of one stage 13. On 210 random problems
// of the operators' ranges, every kernel forced, the choice took 1.006 times the
// best one's time.
struct Shape {
    const char *name, *split_name, *packed_name, *both_name;
    int bm, bn;
    int per_cu;  // work-groups a CU holds
    double stage, pair, round;
    double loose[2];  // a stage's time where rows straddle 128-byte lines, and 4-byte words
};
constexpr Shape kShapes[tlg::FFN_PANEL_CONFIGS] = {
    {"panel_256x256", "panel_256x256_split", "panel_256x256_packed", "panel_256x256_both", 256, 256, 1, 1.35, 1.35, 11, {1.2, 1.35}},
    {"panel_256x128", "panel_256x128_split", "panel_256x128_packed", "panel_256x128_both", 256, 128, 1, 0.98, 0.98, 7, {1.25, 1.4}},
    {"panel_128x128", "panel_128x128_split", "panel_128x128_packed", "panel_128x128_both", 128, 128, 2, 1.08, 0.72, 4, {1.2, 1.45}},
    {"panel_128x128_deep", "panel_128x128_deep_split", "panel_128x128_deep_packed", "panel_128x128_deep_both", 128, 128, 1, 0.62, 0.62, 4, {1.3, 1.45}},
    {"panel_64x128", "panel_64x128_split", "panel_64x128_packed", "", 64, 128, 1, 0.42, 0.42, 3, {1.5, 1.7}},
};

constexpr int64_t kMaxOffset = 0x7ffffff0ll - 4096;  // in-tile byte offsets of the pipelined kernel
constexpr int64_t kSplitBytes = 64ll << 20;          // partial sums of a split product, at most

constexpr int64_t kPackBytes = 1ll << 34;            // aligned copies and partial sums, at most

constexpr int64_t kNever = 1ll << 60;                // more than any device has

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The sizes that a plan goes by. loose: 0, all rows of the caller's operands
// start on 128-byte boundaries; 1, on 4-byte ones; 2, some do not.
struct Sizes {
    int mode;
    bool i8;
    int64_t M, N, K;
    int loose = 0;
};
int loose_level(uint64_t bits) { return bits % 128 == 0 ? 0 : bits % 4 == 0 ? 1 : 2; }
int64_t tiles_of(const Sizes &z, int shape) {
    const int64_t bn = z.mode == tlg::FFN_GATED ? kShapes[shape].bn / 2 : kShapes[shape].bn;
    return ceil_div(z.M, kShapes[shape].bm) * ceil_div(z.N, bn) * (z.mode == tlg::FFN_PAIR ? 2 : 1);
}
int64_t stages_of(const Sizes &z) {
    return ceil_div(z.K, z.i8 ? 128 : 64) * (z.mode == tlg::FFN_SUM2 ? 2 : 1);
}
// Whether a launch holds the product's tiles (and the parts of split ones, which
// fill the card once), or its strips of 16 outputs.
bool tiles_fit(int64_t tiles) { return tiles <= tlg::kMaxThreads / 256 - 512; }
bool strips_fit(const Sizes &z) { return ceil_div(z.N, 16) <= tlg::kMaxThreads / 512; }
// Work-groups that run side by side, and the tiles that fill them in whole
// rounds: the tiles past those may be split.
int64_t slots_of(int shape) { return 256 * kShapes[shape].per_cu; }
int64_t whole_tiles(const Sizes &z, int shape) {
    const int64_t tiles = tiles_of(z, shape);
    return tiles - tiles % slots_of(shape);
}
// fp32 (int32) sums of every part of the split tiles
int64_t split_bytes(const Sizes &z, int shape, int64_t splits) {
    const Shape &c = kShapes[shape];
    return (tiles_of(z, shape) - whole_tiles(z, shape)) * splits * (z.M < c.bm ? z.M : c.bm) * c.bn * 4;
}
// Aligned copies of the operands that come from the caller, rows in whole
// 128-byte stages of K (forward) or of columns (the operands of a gradient,
// whose other side is the workspace's own).
int64_t pack_pitch(const Sizes &z) {
    const bool fwd = z.mode == tlg::FFN_GATED || z.mode == tlg::FFN_LINEAR;
    return round_up((fwd ? z.K : z.N) * (z.i8 ? 1 : 2), 128);
}
int64_t pack_bytes(const Sizes &z) {
    const int64_t rows = z.mode == tlg::FFN_GATED    ? z.M + 2 * z.N
                         : z.mode == tlg::FFN_LINEAR ? z.M + z.N
                         : z.mode == tlg::FFN_SUM2   ? 2 * z.K
                                                     : z.K;
    const int64_t pitch = pack_pitch(z);
    return pitch && rows > kNever / pitch ? kNever : rows * pitch;
}
bool forward_mode(int mode) { return mode == tlg::FFN_GATED || mode == tlg::FFN_LINEAR; }

// As many parts as give every CU its work-groups, no part without a stage,
// within the workspace; below 2: not worth a split.
int64_t most_splits(const Sizes &z, int shape) {
    const int64_t rest = tiles_of(z, shape) - whole_tiles(z, shape);
    if (!rest) return 1;
    int64_t s = slots_of(shape) / rest;
    const int64_t stages = stages_of(z);
    if (s > stages) s = stages;
    while (s > 1 && split_bytes(z, shape, s) > kSplitBytes) --s;
    return s;
}

struct Plan {
    int cfg;
    int64_t splits;
    bool packed;
};

// How much longer a stage takes than on rows of whole 128-byte lines.
// 1024 tokens bf16 from 4096, 4104 and 4097: 256 x 128 65, 87, 95; the
// gradients' other operand is the workspace's own: dX 74.7, 86.0 from 1537.
double stage_slowdown(const Sizes &z, const Shape &c, bool packed) {
    const double slow = z.loose && !packed ? c.loose[z.loose - 1] + (z.i8 && z.loose == 2 ? 0.15 : 0.0) : 1;
    return forward_mode(z.mode) ? slow : 1 + 0.35 * (slow - 1);
}
// A work-group's microseconds besides its stages: elements past the last
// whole chunk (or row) are staged apart.
double round_time(const Sizes &z, const Shape &c, bool packed) {
    const bool odd = !packed && (forward_mode(z.mode) ? z.K * (z.i8 ? 1 : 2) % 16 : z.N % 8) != 0;
    return c.round + (odd ? 2 : 0);
}
// Operands from HBM at 5.1 TB/s at most (the weights of few tokens: 4096 ->
// 14336, 48 tokens, 235 MB in 48 us).
double read_time(const Sizes &z) {
    const double summands = z.mode == tlg::FFN_SUM2 ? 2 : 1;
    const double bytes = (z.i8 ? 1.0 : 2.0) * z.K * ((z.mode == tlg::FFN_PAIR ? 2 : summands) * z.M +
                                                     (z.mode == tlg::FFN_GATED ? 2 : summands) * z.N);
    return bytes / 5.1e6;
}
// Work and reading overlap, not quite wholly.
double overlapped(double work, double read) { return work > read ? work + 0.15 * read : read + 0.15 * work; }

// Estimated microseconds. A split costs the second kernel, its reads of one
// part after another and the sums' way through memory (512 x 1024 from 8192:
// 128 x 128 deep, 82 whole, 30.5 in eight parts). A forward product's copies
// are a launch of their own (1088 x 485 from 871: 16.7 against 14.3 without
// them), a gradient's are made by the launch that makes dG and dU.
constexpr double kLaunch = 2;
double split_time(int64_t splits, double bytes) { return splits > 1 ? 5 + 0.08 * (double)splits + 1.5 * bytes / 4e6 : 0; }
double copies_time(const Sizes &z, bool packed) {
    return packed ? (forward_mode(z.mode) ? 4.5 : 1) + 2 * (double)pack_bytes(z) / 4e6 : 0;
}

// A product in one tile shape, as the estimates below want it.
struct Tiling {
    int64_t tiles, whole, slots, stages;
    int64_t part;  // bytes of one part's sums of every split tile
    double stage, pair, round, read;
};
Tiling tiling(const Sizes &z, int shape, bool packed) {
    const Shape &c = kShapes[shape];
    const double slow = stage_slowdown(z, c, packed);
    Tiling t;
    t.tiles = tiles_of(z, shape);
    t.slots = slots_of(shape);
    t.whole = t.tiles - t.tiles % t.slots;
    t.stages = stages_of(z);
    t.part = (t.tiles - t.whole) * (z.M < c.bm ? z.M : c.bm) * c.bn * 4;
    t.stage = slow * c.stage;
    t.pair = slow * c.pair;
    t.round = round_time(z, c, packed);
    t.read = read_time(z);
    return t;
}
// (copies not counted)
double panel_time(const Tiling &t, int64_t splits) {
    const int64_t full = t.whole / t.slots, groups = (t.tiles - t.whole) * splits;  // groups: of the last round
    double work = full * (t.stages * t.stage + t.round);
    if (groups) work += ceil_div(t.stages, splits) * (full || groups > 256 ? t.stage : t.pair) + t.round;
    return overlapped(work, t.read) + kLaunch + split_time(splits, (double)(t.part * splits));
}

// When the last of n1 work-groups of t1 microseconds and then n2 of t2 ends,
// each taken by the first free one of `slots` places.
double makespan(int64_t n1, double t1, int64_t n2, double t2, int64_t slots) {
    if (n1 + n2 <= slots) return t1 > t2 ? t1 : t2;
    if (n1 + n2 > 16 * slots) return (n1 * t1 + n2 * t2) / slots + (t1 > t2 ? t1 : t2) / 2;
    struct Free {
        double at;
        int64_t count;
    } q[40] = {{0, slots}};
    int n = 1;
    for (int turn = 0; turn < 2; ++turn) {
        int64_t left = turn ? n2 : n1;
        const double t = turn ? t2 : t1;
        while (left > 0) {
            int first = 0;
            for (int i = 1; i < n; ++i)
                if (q[i].at < q[first].at) first = i;
            const int64_t take = left < q[first].count ? left : q[first].count;
            left -= take;
            if (take == q[first].count) {
                q[first].at += t;
            } else {
                q[first].count -= take;
                q[n++] = {q[first].at + t, take};  // only the last of a turn leaves some: 3 entries at most
            }
        }
    }
    double end = 0;
    for (int i = 0; i < n; ++i)
        if (q[i].at > end) end = q[i].at;
    return end;
}
// Strips of 16 outputs read the weights a little faster and need no second
// kernel, but every strip reads all of X, from L2: 20 TB/s for one tile of
// tokens, 7 for more (4096 -> 14336: 1 token 43, 16 tokens 49, 48
// tokens 91).
double strip_time(const Sizes &z) {
    const double eb = z.i8 ? 1 : 2, nb = z.mode == tlg::FFN_GATED ? 2 : 1, weights = eb * z.K * z.N * nb;
    const double x = eb * z.K * z.M * (double)ceil_div(z.N, 16);
    // fewer strips than CUs: each streams at 40 GB/s
    // (1 token bf16 -> 4096 from 4096 and 4098: 15.3, 18.1)
    const double slow = z.loose ? 0.8 : 1.0;
    const double rate = 5.4e6 * (z.N < 16 * 128 ? z.N / (16 * 128.0) : 1.0) * slow;
    const double t = 4 + weights / rate + x / ((z.M <= 16 ? 20e6 : 7e6) * slow);
    if (z.loose < 2) return t;
    // Rows off 4-byte boundaries: a 64-byte piece of 16 rows takes a CU 95 ns
    // (bf16 -> 4096 from 4097: 1 token 29.1, 16 tokens 39.9, 48 tokens 68.4;
    // 16 tokens -> 389 from 2561 25.8; int8 -> 2319 from 6021, 17 tokens, 18.0)
    const double rounds = z.N > 16 * 256 ? z.N / (16 * 256.0) : 1.0;
    const double pieces = 4 + rounds * (eb * z.K / 64) * (nb + z.M / 16.0) * 0.095;
    return pieces > t ? pieces : t;
}

int shape_of(int cfg) {
    return cfg >= CFG_BOTH ? cfg - CFG_BOTH : cfg >= CFG_PACKED ? cfg - CFG_PACKED : cfg >= CFG_SPLIT ? cfg - CFG_SPLIT : cfg - CFG_PANEL;
}
int64_t plan_bytes(const Sizes &z, const Plan &p) {
    return (p.packed ? round_up(pack_bytes(z), 256) : 0) +
           (p.splits > 1 ? split_bytes(z, shape_of(p.cfg), p.splits) : 0);
}

// The plan of the least estimated time that the workspace allows.
Plan plan_auto(const Sizes &z, int64_t ws_bytes) {
    Plan best = {CFG_GENERAL, 1, false};
    double least = 1e300;
    if (forward_mode(z.mode) && z.M <= 64 && strips_fit(z)) {
        least = strip_time(z);
        best.cfg = CFG_SKINNY;
    }
    const double copies = z.loose ? copies_time(z, true) : 0;
    for (int shape = 0; shape < tlg::FFN_PANEL_CONFIGS; ++shape) {
        if (shape == tlg::FFN_PANEL_64x128 && !forward_mode(z.mode)) continue;
        if (!tiles_fit(tiles_of(z, shape))) continue;
        // mostly rows of nothing; but wider, where the others have too many tiles
        if (z.M <= 64 && kShapes[shape].bm > 128 && tiles_fit(tiles_of(z, tlg::FFN_PANEL_128x128))) continue;
        const int64_t most = most_splits(z, shape);
        for (int packed = 0; packed < (z.loose ? 2 : 1); ++packed) {
            const Tiling t = tiling(z, shape, packed != 0);
            for (int64_t s = 1;; s = s * 2 < most ? s * 2 : most) {
                const Plan p = {(s > 1 ? CFG_SPLIT : CFG_PANEL) + shape, s, packed != 0};
                const double us = panel_time(t, s) + (packed ? copies : 0);
                if (us < least && ((s == 1 && !packed) || plan_bytes(z, p) <= ws_bytes)) {
                    least = us;
                    best = p;
                }
                if (s >= most) break;
            }
        }
    }
    return best;
}

// The plans of a backward pass's two products where one launch of both is
// estimated faster than theirs alone (`x` and `w` as plan_auto has them), by
// 3 % at least: with the same copies, in one tile shape, and a split only of a
// product with fewer tiles than places. 3001 x 1537 from 2049: 114 against 124
// us, 353 x 4409 from 1117: 45 against 60; where both fill whole rounds it
// gains nothing (8192 x 4096 from 14336: 3059 against 3008).
void plan_both(const Sizes &zx, const Sizes &zw, Plan &x, Plan &w, int64_t ws_bytes) {
    if (x.cfg == CFG_GENERAL || w.cfg == CFG_GENERAL) return;  // too many tiles of any shape
    const bool px = x.packed, pw = w.packed;
    double least = 0.97 * (panel_time(tiling(zx, shape_of(x.cfg), px), x.splits) +
                           panel_time(tiling(zw, shape_of(w.cfg), pw), w.splits));
    for (int shape = 0; shape < tlg::FFN_PANEL_64x128; ++shape) {
        const Tiling tx = tiling(zx, shape, px), tw = tiling(zw, shape, pw);
        if (!tiles_fit(tx.tiles + tw.tiles)) continue;
        const int64_t mx = tx.whole ? 1 : most_splits(zx, shape), mw = tw.whole ? 1 : most_splits(zw, shape);
        for (int64_t sx = 1;; sx = sx * 2 < mx ? sx * 2 : mx) {
            const int64_t nx = tx.tiles * sx, kx = ceil_div(tx.stages, sx);
            for (int64_t sw = 1;; sw = sw * 2 < mw ? sw * 2 : mw) {
                const int64_t nw = tw.tiles * sw, kw = ceil_div(tw.stages, sw);
                const bool paired = nx + nw > 256;
                const double ux = kx * (paired ? tx.stage : tx.pair) + tx.round;  // of one work-group
                const double uw = kw * (paired ? tw.stage : tw.pair) + tw.round;
                if ((nx * ux + nw * uw) / tx.slots < least) {
                    const double work = ux >= uw ? makespan(nx, ux, nw, uw, tx.slots) : makespan(nw, uw, nx, ux, tx.slots);
                    const double parts = (sx > 1 ? (double)(tx.part * sx) : 0) + (sw > 1 ? (double)(tw.part * sw) : 0);
                    const double us = overlapped(work, tx.read + tw.read) + kLaunch + split_time(sx > sw ? sx : sw, parts);
                    const Plan bx = {CFG_BOTH + shape, sx, px}, bw = {CFG_BOTH + shape, sw, pw};
                    if (us < least && plan_bytes(zx, bx) + plan_bytes(zw, bw) <= ws_bytes) {
                        least = us;
                        x = bx;
                        w = bw;
                    }
                }
                if (sw >= mw) break;
            }
            if (sx >= mx) break;
        }
    }
}

// Bytes that the planned kernels want (0: none), for operands without padding.
int64_t plan_workspace(Sizes z) {
    if (z.M <= 0 || z.N <= 0 || z.K <= 0 || z.M > kMaxDim || z.N > kMaxDim || z.K > kMaxDim) return 0;
    z.loose = loose_level((forward_mode(z.mode) ? z.K : z.N) * (z.i8 ? 1 : 2));
    return plan_bytes(z, plan_auto(z, kPackBytes));
}

// What the pipelined kernel's loads cover of K, or -1 where it cannot serve
// the problem. Row-layout operands are loaded in whole 16-byte chunks of K,
// column-layout ones in whole rows of k (pcol_kmain). (dG and dU have zeros up
// to their pitch.)
int64_t panel_kmain(const FfnProduct &p) {
    const bool i8 = p.type == tlg::FFN_I8, acol = p.A[0].ks != 1 || p.mode == tlg::FFN_PAIR;
    const int64_t eb = i8 ? 1 : 2;
    const bool bcol = p.mode == tlg::FFN_SUM2 || p.mode == tlg::FFN_PAIR;
    // (leading dimensions are the caller's, up to the largest int64: divided, not multiplied)
    for (int s = 0; s < (p.mode == tlg::FFN_SUM2 || p.mode == tlg::FFN_PAIR ? 2 : 1); ++s)
        if ((acol ? p.A[s].ks : p.A[s].rs) > kMaxOffset / ((acol ? 64 : 256) * eb)) return -1;
    for (int s = 0; s < (p.mode == tlg::FFN_SUM2 || p.mode == tlg::FFN_GATED ? 2 : 1); ++s)
        if ((bcol ? p.B[s].ks : p.B[s].rs) > kMaxOffset / ((bcol ? 64 : 256) * eb)) return -1;
    for (int o = 0; o < 3; ++o)
        if (p.C[o] && p.ldc[o] > kMaxOffset / (128 * 4)) return -1;
    if (bcol) {
        if (p.N < 8) return -1;
        return tlg::pcol_kmain(p.K, p.N, p.mode == tlg::FFN_SUM2);
    }
    return p.K / (16 / eb) * (16 / eb);
}

// How the rows of the caller's operands start (Sizes::loose).
int loose_rows(const FfnProduct &p) {
    const uint64_t eb = p.type == tlg::FFN_I8 ? 1 : 2;
    const auto bits = [&](const tlg::FfnOperand &o) {
        return (uint64_t)(uintptr_t)o.p | (uint64_t)(o.rs == 1 ? o.ks : o.rs) * eb;
    };
    uint64_t all = bits(p.B[0]);
    if (p.mode == tlg::FFN_GATED || p.mode == tlg::FFN_SUM2) all |= bits(p.B[1]);
    if (forward_mode(p.mode)) all |= bits(p.A[0]);
    return loose_level(all);
}

// A product with its kernel chosen.
struct Chosen {
    FfnProduct p;
    Sizes z;
    Plan plan;
    int shape;
    int64_t kmain;
    int ext_b;  // readable columns of a column-layout B
};

tlg_status choose(int32_t config, const FfnProduct &p, int64_t ws_bytes, Chosen *o) {
    if (config >= CFG_COUNT || config < -1) return TLG_ERROR_INVALID_VALUE;
    *o = {p, {p.mode, p.type == tlg::FFN_I8, p.M, p.N, p.K, loose_rows(p)}, {config, 1, false}, 0, panel_kmain(p), p.N};
    const Sizes &z = o->z;
    Plan &plan = o->plan;
    if (config < 0) plan = o->kmain < 0 ? Plan{CFG_GENERAL, 1, false} : plan_auto(z, ws_bytes);
    if (plan.cfg == CFG_GENERAL)
        return ceil_div(p.M, 64) * ceil_div(p.N, 64) > tlg::kMaxThreads / 256 ? TLG_ERROR_NOT_SUPPORTED : TLG_SUCCESS;
    if (o->kmain < 0) return TLG_ERROR_NOT_SUPPORTED;
    if (plan.cfg == CFG_SKINNY)
        return forward_mode(p.mode) && p.M <= 64 && strips_fit(z) ? TLG_SUCCESS : TLG_ERROR_NOT_SUPPORTED;
    o->shape = shape_of(plan.cfg);
    if (o->shape == tlg::FFN_PANEL_64x128 && !forward_mode(p.mode)) return TLG_ERROR_NOT_SUPPORTED;
    if (!tiles_fit(tiles_of(z, o->shape))) return TLG_ERROR_NOT_SUPPORTED;
    if (config >= CFG_BOTH) {
        if (forward_mode(p.mode)) return TLG_ERROR_NOT_SUPPORTED;
        plan.splits = most_splits(z, o->shape);  // (1 for many tiles)
    } else if (config >= CFG_PACKED) {
        plan.packed = true;
    } else if (config >= CFG_SPLIT) {
        plan.splits = most_splits(z, o->shape);
        if (plan.splits < 2) return TLG_ERROR_NOT_SUPPORTED;
    }
    return plan_bytes(z, plan) > ws_bytes && (plan.packed || plan.splits > 1) ? TLG_ERROR_NOT_SUPPORTED : TLG_SUCCESS;
}

// Adds the caller's operands to the copies, at `ws`, and puts the copies in
// their place.
void add_copies(Chosen &c, char *ws, tlg::FfnPack &k) {
    const int64_t eb = c.z.i8 ? 1 : 2, pitch = pack_pitch(c.z);
    const bool fwd = forward_mode(c.z.mode), b1 = c.z.mode == tlg::FFN_GATED || c.z.mode == tlg::FFN_SUM2;
    k.pitch = pitch;  // the same for a backward pass's two products
    const auto add = [&](tlg::FfnOperand &o, int64_t rows) {
        k.src[k.count] = o.p;
        k.dst[k.count] = ws;
        k.rows[k.count] = rows;
        k.row_bytes[k.count] = (fwd ? c.z.K : c.z.N) * eb;
        k.ld_bytes[k.count++] = (fwd ? o.rs : o.ks) * eb;
        o = {ws, fwd ? pitch / eb : 1, fwd ? 1 : pitch / eb};
        ws += rows * pitch;
    };
    if (fwd) add(c.p.A[0], c.z.M);
    add(c.p.B[0], fwd ? c.z.N : c.z.K);
    if (b1) add(c.p.B[1], fwd ? c.z.N : c.z.K);
    if (fwd)
        c.p.K = (int)(pitch / eb);  // zeros add nothing
    else
        c.ext_b = (int)(pitch / eb);
    c.kmain = c.p.K;
}

// A chosen product for the pipelined kernel; `part`: room for the sums of its parts.
tlg::FfnPanelCall panel_call(const Chosen &c, void *part) {
    // the columns of a column-layout A that may be read
    const int ext_a = c.p.mode == tlg::FFN_PAIR ? (int)c.p.A[0].ks : c.p.M;
    return {c.p, (int)c.kmain, ext_a, c.ext_b, (int)whole_tiles(c.z, c.shape), (int)c.plan.splits, part};
}
tlg_status launch(const Chosen &c, void *part, hipStream_t stream) {
    const FfnProduct &p = c.p;
    if (c.plan.cfg == CFG_GENERAL) return status_of(tlg::launch_ffn_general(p, stream));
    if (c.plan.cfg == CFG_SKINNY) return status_of(tlg::launch_ffn_skinny(p, (int)c.kmain, stream));
    const auto fn = p.type == tlg::FFN_F16    ? tlg::launch_ffn_panel_f16
                    : p.type == tlg::FFN_BF16 ? tlg::launch_ffn_panel_bf16
                                              : tlg::launch_ffn_panel_i8;
    return status_of(fn(c.shape, panel_call(c, part), stream));
}

int64_t copies_bytes(const Chosen &c) { return c.plan.packed ? round_up(pack_bytes(c.z), 256) : 0; }
int64_t parts_bytes(const Chosen &c) { return c.plan.splits > 1 ? split_bytes(c.z, c.shape, c.plan.splits) : 0; }

tlg_status run_product(int32_t config, const FfnProduct &p, void *ws, int64_t ws_bytes, hipStream_t stream) {
    Chosen c;
    tlg_status st = choose(config, p, ws_bytes, &c);
    if (st != TLG_SUCCESS) return st;
    char *part = (char *)ws + copies_bytes(c);
    if (c.plan.packed) {
        tlg::FfnPack k = {};
        add_copies(c, (char *)ws, k);
        st = status_of(tlg::launch_ffn_pack(k, stream));
        if (st != TLG_SUCCESS) return st;
    }
    return launch(c, part, stream);
}

// An optional workspace: none, or 16-byte aligned.
bool workspace_ok(const void *ws, int64_t bytes) { return bytes >= 0 && (ws ? aligned(ws, 16) : bytes == 0); }

tlg_status gated(tlg_handle h, int32_t config, int type, int32_t out_dtype, int32_t act, const tlg_gated_ffn_desc *d,
                 const float *SX, const float *SG, const float *SU, void *ws, int64_t ws_bytes, hipStream_t stream) {
    if (!h || !d || !is16(out_dtype) || !is_act(act) || !workspace_ok(ws, ws_bytes)) return TLG_ERROR_INVALID_VALUE;
    const bool i8 = type == tlg::FFN_I8;
    const int eb = i8 ? 1 : 2;
    if (d->M < 0 || d->N < 0 || d->K < 0) return TLG_ERROR_INVALID_VALUE;
    if (!d->G != !d->U || (i8 && d->G)) return TLG_ERROR_INVALID_VALUE;
    const bool none = d->M == 0 || d->N == 0;  // nothing is read or written
    const int64_t M = none ? 0 : d->M, N = none ? 0 : d->N;
    if (!matrix_ok(d->X, M, d->K, d->ldx, eb) || !matrix_ok(d->Wg, N, d->K, d->ldwg, eb) ||
        !matrix_ok(d->Wu, N, d->K, d->ldwu, eb) || !matrix_ok(d->H, M, none ? 0 : d->N, d->ldh, 2))
        return TLG_ERROR_INVALID_VALUE;
    if (d->ldh < d->N) return TLG_ERROR_INVALID_VALUE;
    if (d->G && (d->ldg < d->N || d->ldu < d->N || !aligned(d->G, 2) || !aligned(d->U, 2)))
        return TLG_ERROR_INVALID_VALUE;
    if (none) return TLG_SUCCESS;
    if (i8 && (!SX || !SG || !SU || !aligned(SX, 4) || !aligned(SG, 4) || !aligned(SU, 4)))
        return TLG_ERROR_INVALID_VALUE;
    if (d->M > kMaxDim || d->N > kMaxDim || d->K > (i8 ? kMaxK8 : kMaxDim)) return TLG_ERROR_NOT_SUPPORTED;
    const tlg_status st = check_device(h);
    if (st != TLG_SUCCESS) return st;
    FfnProduct p = {};
    p.type = type;
    p.mode = tlg::FFN_GATED;
    p.act = act;
    p.out_type = out_dtype;
    p.M = (int)d->M;
    p.N = (int)d->N;
    p.K = (int)d->K;
    p.A[0] = {d->X, d->ldx, 1};
    p.B[0] = {d->Wg, d->ldwg, 1};
    p.B[1] = {d->Wu, d->ldwu, 1};
    p.sa = SX;
    p.sb[0] = SG;
    p.sb[1] = SU;
    p.C[0] = d->H;
    p.ldc[0] = d->ldh;
    p.C[1] = d->G;
    p.ldc[1] = d->ldg;
    p.C[2] = d->U;
    p.ldc[2] = d->ldu;
    return run_product(config, p, ws, ws_bytes, stream);
}

// The workspace of a backward pass: the dG and dU planes, rows on 128-byte
// boundaries, and their scale, then aligned copies and the parts of split sums.
int64_t grad_pitch(int64_t N) { return round_up(N, 64); }
constexpr int64_t kScaleBytes = (sizeof(tlg::FfnGateScale) + 255) / 256 * 256;
int64_t planes_bytes(int64_t M, int64_t N) { return kScaleBytes + round_up(4 * M * grad_pitch(N), 256); }

tlg_status backward(tlg_handle h, int32_t config, int32_t dtype, int32_t act, const tlg_gated_ffn_grad_desc *d,
                    void *workspace, int64_t workspace_bytes, hipStream_t stream) {
    if (!h || !d || !is16(dtype) || !is_act(act)) return TLG_ERROR_INVALID_VALUE;
    const int64_t M = d->M, N = d->N, K = d->K;
    if (M < 0 || N < 0 || K < 0) return TLG_ERROR_INVALID_VALUE;
    if (!d->dWg != !d->dWu) return TLG_ERROR_INVALID_VALUE;
    const bool want_x = d->dX && M > 0 && K > 0, want_w = d->dWg && N > 0 && K > 0;
    const bool sums = M > 0 && N > 0 && (want_x || want_w);  // any product to take
    if (!matrix_ok(d->dH, sums ? M : 0, N, d->lddh, 2) || !matrix_ok(d->G, sums ? M : 0, N, d->ldg, 2) ||
        !matrix_ok(d->U, sums ? M : 0, N, d->ldu, 2))
        return TLG_ERROR_INVALID_VALUE;
    if (d->dWg && (!matrix_ok(d->X, sums && want_w ? M : 0, K, d->ldx, 2) || !matrix_ok(d->dWg, N, K, d->lddwg, 2) ||
                   !matrix_ok(d->dWu, N, K, d->lddwu, 2)))
        return TLG_ERROR_INVALID_VALUE;
    if (d->dX && (!matrix_ok(d->Wg, sums && want_x ? N : 0, K, d->ldwg, 2) ||
                  !matrix_ok(d->Wu, sums && want_x ? N : 0, K, d->ldwu, 2) || !matrix_ok(d->dX, M, K, d->lddx, 2)))
        return TLG_ERROR_INVALID_VALUE;
    if (!want_x && !want_w) return TLG_SUCCESS;
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return TLG_ERROR_NOT_SUPPORTED;
    tlg_status st = check_device(h);
    if (st != TLG_SUCCESS) return st;
    if (!sums) {  // M == 0: no token; N == 0: no channel
        hipError_t e = hipSuccess;
        if (want_x) e = tlg::launch_ffn_zero(d->dX, M, K, d->lddx, stream);
        if (want_w && e == hipSuccess) e = tlg::launch_ffn_zero(d->dWg, N, K, d->lddwg, stream);
        if (want_w && e == hipSuccess) e = tlg::launch_ffn_zero(d->dWu, N, K, d->lddwu, stream);
        return status_of(e);
    }
    const int64_t needed = tlg_gated_ffn_backward_workspace(M, N, K);
    if (!workspace || !aligned(workspace, 16) || needed == INT64_MAX || workspace_bytes < needed)
        return TLG_ERROR_INVALID_VALUE;
    const int64_t pitch = grad_pitch(N);
    tlg::FfnGateScale *scale = (tlg::FfnGateScale *)workspace;
    uint16_t *dG = (uint16_t *)((char *)workspace + kScaleBytes), *dU = dG + M * pitch;
    char *ws = (char *)workspace + planes_bytes(M, N);
    const int64_t left = workspace_bytes - planes_bytes(M, N);
    const int type = type_of(dtype);
    FfnProduct px = {}, pw = {};
    px.type = pw.type = type;
    px.out_type = pw.out_type = dtype;
    px.undo = pw.undo = &scale->undo;
    px.mode = tlg::FFN_SUM2;
    px.M = (int)M;
    px.N = (int)K;
    px.K = (int)N;
    px.A[0] = {dG, pitch, 1};
    px.A[1] = {dU, pitch, 1};
    px.B[0] = {d->Wg, 1, d->ldwg};
    px.B[1] = {d->Wu, 1, d->ldwu};
    px.C[0] = d->dX;
    px.ldc[0] = d->lddx;
    pw.mode = tlg::FFN_PAIR;
    pw.M = (int)N;
    pw.N = (int)K;
    pw.K = (int)M;
    pw.A[0] = {dG, 1, pitch};
    pw.A[1] = {dU, 1, pitch};
    pw.B[0] = {d->X, 1, d->ldx};
    pw.C[0] = d->dWg;
    pw.ldc[0] = d->lddwg;
    pw.C[1] = d->dWu;
    pw.ldc[1] = d->lddwu;
    // both products' kernels first: their copies are made with dG and dU
    Chosen x = {}, w = {};
    bool both = config >= CFG_BOTH;
    if (both && !(want_x && want_w)) return TLG_ERROR_NOT_SUPPORTED;
    const auto too_many = [&] { return !tiles_fit(tiles_of(x.z, x.shape) + tiles_of(w.z, w.shape)); };
    for (int64_t room = left;; room = 0) {
        if (want_x) st = choose(config, px, room, &x);
        if (want_w && st == TLG_SUCCESS) st = choose(config, pw, room, &w);
        if (st != TLG_SUCCESS) return st;
        if (both && too_many()) return TLG_ERROR_NOT_SUPPORTED;
        if (config < 0 && want_x && want_w && x.kmain >= 0 && w.kmain >= 0) {
            plan_both(x.z, w.z, x.plan, w.plan, room);
            both = x.plan.cfg >= CFG_BOTH;
            x.shape = shape_of(x.plan.cfg);
            w.shape = shape_of(w.plan.cfg);
        }
        const int64_t px_parts = want_x ? parts_bytes(x) : 0, pw_parts = want_w ? parts_bytes(w) : 0;
        const int64_t need = (want_x ? copies_bytes(x) : 0) + (want_w ? copies_bytes(w) : 0) +
                             (both                  ? px_parts + pw_parts
                              : px_parts > pw_parts ? px_parts
                                                    : pw_parts);
        if (need <= left) break;
        if (config >= 0) return TLG_ERROR_NOT_SUPPORTED;
    }
    tlg::FfnPack k = {};
    k.pitch = 16;
    if (want_x && x.plan.packed) {
        const int64_t bytes = copies_bytes(x);
        add_copies(x, ws, k);
        ws += bytes;
    }
    if (want_w && w.plan.packed) {
        const int64_t bytes = copies_bytes(w);
        add_copies(w, ws, k);
        ws += bytes;
    }
    st = status_of(tlg::launch_ffn_gate_grad(type, act, (int)M, (int)N, d->dH, d->lddh, d->G, d->ldg, d->U, d->ldu, dG,
                                             dU, pitch, scale, k, stream));
    if (both && st == TLG_SUCCESS) {
        const auto fn = type == tlg::FFN_F16 ? tlg::launch_ffn_panel_grads_f16 : tlg::launch_ffn_panel_grads_bf16;
        // the longer sums first
        const bool lead = stages_of(x.z) * w.plan.splits >= stages_of(w.z) * x.plan.splits;
        return status_of(fn(x.shape, panel_call(x, ws), panel_call(w, ws + parts_bytes(x)), lead, stream));
    }
    if (want_x && st == TLG_SUCCESS) st = launch(x, ws, stream);
    if (want_w && st == TLG_SUCCESS) st = launch(w, ws, stream);
    return st;
}

tlg_status linear_i8(tlg_handle h, int32_t config, int32_t out_dtype, int32_t relu, int64_t M, int64_t N, int64_t K,
                     const int8_t *A, int64_t lda, const float *SA, const int8_t *B, int64_t ldb, const float *SB,
                     void *C, int64_t ldc, void *ws, int64_t ws_bytes, hipStream_t stream) {
    if (!h || (!is16(out_dtype) && out_dtype != TLG_F32) || !workspace_ok(ws, ws_bytes))
        return TLG_ERROR_INVALID_VALUE;
    if (M < 0 || N < 0 || K < 0) return TLG_ERROR_INVALID_VALUE;
    const bool none = M == 0 || N == 0;
    if (!matrix_ok(A, none ? 0 : M, K, lda, 1) || !matrix_ok(B, none ? 0 : N, K, ldb, 1) ||
        !matrix_ok(C, none ? 0 : M, N, ldc, bytes_of(out_dtype)))
        return TLG_ERROR_INVALID_VALUE;
    if (none) return TLG_SUCCESS;
    if (!SA || !SB || !aligned(SA, 4) || !aligned(SB, 4)) return TLG_ERROR_INVALID_VALUE;
    if (M > kMaxDim || N > kMaxDim || K > kMaxK8) return TLG_ERROR_NOT_SUPPORTED;
    const tlg_status st = check_device(h);
    if (st != TLG_SUCCESS) return st;
    FfnProduct p = {};
    p.type = tlg::FFN_I8;
    p.mode = tlg::FFN_LINEAR;
    p.relu = relu != 0;
    p.out_type = out_dtype;
    p.M = (int)M;
    p.N = (int)N;
    p.K = (int)K;
    p.A[0] = {A, lda, 1};
    p.B[0] = {B, ldb, 1};
    p.sa = SA;
    p.sb[0] = SB;
    p.C[0] = C;
    p.ldc[0] = ldc;
    return run_product(config, p, ws, ws_bytes, stream);
}

}  // namespace

extern "C" {

int64_t tlg_gated_ffn_workspace(int64_t M, int64_t N, int64_t K) {
    return plan_workspace({tlg::FFN_GATED, false, M, N, K});
}
tlg_status tlg_gated_ffn(tlg_handle h, int32_t dtype, int32_t act, const tlg_gated_ffn_desc *d, void *workspace,
                         int64_t workspace_bytes, hipStream_t stream) {
    return gated(h, -1, type_of(dtype), dtype, act, d, nullptr, nullptr, nullptr, workspace, workspace_bytes, stream);
}
tlg_status tlg_gated_ffn_variant(tlg_handle h, int32_t config, int32_t dtype, int32_t act,
                                 const tlg_gated_ffn_desc *d, void *workspace, int64_t workspace_bytes,
                                 hipStream_t stream) {
    return gated(h, config, type_of(dtype), dtype, act, d, nullptr, nullptr, nullptr, workspace, workspace_bytes,
                 stream);
}

int64_t tlg_gated_ffn_backward_workspace(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || K <= 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return 0;
    if (M > kNever / 4 / grad_pitch(N)) return INT64_MAX;
    const int loose = loose_level(2 * (uint64_t)K);
    const Sizes x = {tlg::FFN_SUM2, false, M, K, N, loose}, w = {tlg::FFN_PAIR, false, N, K, M, loose};
    Plan px = plan_auto(x, kPackBytes), pw = plan_auto(w, kPackBytes);
    const int64_t apart = plan_bytes(x, px) + plan_bytes(w, pw);
    plan_both(x, w, px, pw, kPackBytes);
    const int64_t both = px.cfg >= CFG_BOTH ? plan_bytes(x, px) + plan_bytes(w, pw) : 0;
    return planes_bytes(M, N) + (apart > both ? apart : both);
}
tlg_status tlg_gated_ffn_backward(tlg_handle h, int32_t dtype, int32_t act, const tlg_gated_ffn_grad_desc *d,
                                  void *workspace, int64_t workspace_bytes, hipStream_t stream) {
    return backward(h, -1, dtype, act, d, workspace, workspace_bytes, stream);
}
tlg_status tlg_gated_ffn_backward_variant(tlg_handle h, int32_t config, int32_t dtype, int32_t act,
                                          const tlg_gated_ffn_grad_desc *d, void *workspace, int64_t workspace_bytes,
                                          hipStream_t stream) {
    return backward(h, config, dtype, act, d, workspace, workspace_bytes, stream);
}

tlg_status tlg_quantize_i8(tlg_handle h, int32_t dtype, int64_t M, int64_t K, const void *X, int64_t ldx, int8_t *Q,
                           int64_t ldq, float *S, hipStream_t stream) {
    if (!h || (!is16(dtype) && dtype != TLG_F32) || M < 0 || K < 0) return TLG_ERROR_INVALID_VALUE;
    if (!matrix_ok(X, M, K, ldx, bytes_of(dtype)) || !matrix_ok(Q, M, K, ldq, 1)) return TLG_ERROR_INVALID_VALUE;
    if (M == 0) return TLG_SUCCESS;
    if (!S || !aligned(S, 4)) return TLG_ERROR_INVALID_VALUE;
    if (M > kMaxDim || K > kMaxDim) return TLG_ERROR_NOT_SUPPORTED;
    const tlg_status st = check_device(h);
    if (st != TLG_SUCCESS) return st;
    return status_of(tlg::launch_quantize_i8(dtype, M, K, X, ldx, Q, ldq, S, stream));
}

int64_t tlg_gemm_i8_workspace(int64_t M, int64_t N, int64_t K) {
    return plan_workspace({tlg::FFN_LINEAR, true, M, N, K});
}
tlg_status tlg_gemm_i8(tlg_handle h, int32_t out_dtype, int32_t relu, int64_t M, int64_t N, int64_t K,
                       const int8_t *A, int64_t lda, const float *SA, const int8_t *B, int64_t ldb, const float *SB,
                       void *C, int64_t ldc, void *workspace, int64_t workspace_bytes, hipStream_t stream) {
    return linear_i8(h, -1, out_dtype, relu, M, N, K, A, lda, SA, B, ldb, SB, C, ldc, workspace, workspace_bytes,
                     stream);
}
tlg_status tlg_gemm_i8_variant(tlg_handle h, int32_t config, int32_t out_dtype, int32_t relu, int64_t M, int64_t N,
                               int64_t K, const int8_t *A, int64_t lda, const float *SA, const int8_t *B, int64_t ldb,
                               const float *SB, void *C, int64_t ldc, void *workspace, int64_t workspace_bytes,
                               hipStream_t stream) {
    return linear_i8(h, config, out_dtype, relu, M, N, K, A, lda, SA, B, ldb, SB, C, ldc, workspace, workspace_bytes,
                     stream);
}

int64_t tlg_gated_ffn_i8_workspace(int64_t M, int64_t N, int64_t K) {
    return plan_workspace({tlg::FFN_GATED, true, M, N, K});
}
tlg_status tlg_gated_ffn_i8(tlg_handle h, int32_t out_dtype, int32_t act, const tlg_gated_ffn_desc *d,
                            const float *SX, const float *SG, const float *SU, void *workspace,
                            int64_t workspace_bytes, hipStream_t stream) {
    return gated(h, -1, tlg::FFN_I8, out_dtype, act, d, SX, SG, SU, workspace, workspace_bytes, stream);
}
tlg_status tlg_gated_ffn_i8_variant(tlg_handle h, int32_t config, int32_t out_dtype, int32_t act,
                                    const tlg_gated_ffn_desc *d, const float *SX, const float *SG, const float *SU,
                                    void *workspace, int64_t workspace_bytes, hipStream_t stream) {
    return gated(h, config, tlg::FFN_I8, out_dtype, act, d, SX, SG, SU, workspace, workspace_bytes, stream);
}

int32_t tlg_ffn_plan(int32_t product, int64_t M, int64_t N, int64_t K, int32_t loose, int64_t workspace_bytes,
                     int32_t *splits) {
    if (M < 1 || N < 1 || K < 1 || M > kMaxDim || N > kMaxDim || K > kMaxDim || workspace_bytes < 0 || loose < 0 ||
        loose > 2)
        return -1;
    Sizes z;
    switch (product) {
        case TLG_FFN_GATED: z = {tlg::FFN_GATED, false, M, N, K, loose}; break;
        case TLG_FFN_DX: z = {tlg::FFN_SUM2, false, M, K, N, loose}; break;
        case TLG_FFN_DW: z = {tlg::FFN_PAIR, false, N, K, M, loose}; break;
        case TLG_FFN_I8: z = {tlg::FFN_LINEAR, true, M, N, K, loose}; break;
        case TLG_FFN_GATED_I8: z = {tlg::FFN_GATED, true, M, N, K, loose}; break;
        case TLG_FFN_GRADS: z = {tlg::FFN_SUM2, false, M, K, N, loose}; break;
        default: return -1;
    }
    Plan p = plan_auto(z, workspace_bytes);
    if (product == TLG_FFN_GRADS) {
        const Sizes zw = {tlg::FFN_PAIR, false, N, K, M, loose};
        Plan w = plan_auto(zw, workspace_bytes);
        plan_both(z, zw, p, w, workspace_bytes);
    }
    if (splits) *splits = (int32_t)p.splits;
    if (!p.packed || p.cfg >= CFG_BOTH) return p.cfg;
    return CFG_PACKED + p.cfg - (p.splits > 1 ? CFG_SPLIT : CFG_PANEL);
}

const char *tlg_ffn_config_name(int32_t config) {
    if (config < 0 || config >= CFG_COUNT) return "";
    if (config == CFG_GENERAL) return "general_64x64";
    if (config == CFG_SKINNY) return "strip_16";
    if (config < CFG_SKINNY) return kShapes[config - CFG_PANEL].name;
    if (config >= CFG_BOTH) return kShapes[config - CFG_BOTH].both_name;
    return config < CFG_PACKED ? kShapes[config - CFG_SPLIT].split_name : kShapes[config - CFG_PACKED].packed_name;
}

}  // extern "C"
