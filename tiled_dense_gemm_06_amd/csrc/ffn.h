// Internal interface between the feed-forward entry points (ffn_api.cpp) and
// their gfx950 kernels.
#ifndef TLG_FFN_H
#define TLG_FFN_H

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "tlg.h"

namespace tlg {

// What a product computes from its operands. Every operand is a set of rows
// of length K (element k of row r at p + r*rs + k*ks, one of rs, ks being 1),
// and every product sums over k.
enum FfnMode {
    FFN_GATED = 0,   // H = act(A B0^T) * (A B1^T); the two products are stored too where C[1] is not null
    FFN_SUM2 = 1,    // C = A0 B0^T + A1 B1^T
    FFN_PAIR = 2,    // C0 = A0 B0^T, C1 = A1 B0^T
    FFN_LINEAR = 3   // C = A0 B0^T (8-bit codes with scales)
};

// Element type of the operands.
enum FfnType { FFN_F16 = 0, FFN_BF16 = 1, FFN_I8 = 2 };

struct FfnOperand {
    const void *p;
    int64_t rs, ks;  // strides in elements
};

struct FfnProduct {
    int type, mode;
    int act;       // tlg_act (FFN_GATED)
    int relu;      // FFN_LINEAR: ReLU on the scaled sum
    int out_type;  // tlg_dtype of C
    int M, N, K;   // rows and columns of one output; K of one summand
    FfnOperand A[2], B[2];
    const float *sa;     // FFN_I8: scales of A's rows
    const float *sb[2];  // ... and of B's
    const float *undo;   // FFN_F16 gradients: a factor of the sums (launch_ffn_gate_grad)
    void *C[3];
    int64_t ldc[3];
};

// A launch has fewer than 2^32 threads along a dimension of its grid.
constexpr int64_t kMaxThreads = (1ll << 32) - 1;

// Kernel families, and what tlg_ffn_plan reports as `config`.
hipError_t launch_ffn_general(const FfnProduct &p, hipStream_t stream);

// A product for the pipelined kernel. K's first kmain elements are loaded in
// 16-byte chunks, the rest (fewer than two chunks) one by one: kmain is a
// multiple of the chunk where a row-layout operand has elements past it that
// are not zero. ext_a and ext_b are the readable elements of a row of a
// column-layout operand (ks != 1). splits > 1: the tiles past the first `whole` are cut into that many
// parts each, whose sums go through `part`, min(M, BM) x BN x 4 bytes a tile
// and part.
struct FfnPanelCall {
    FfnProduct p;
    int kmain, ext_a, ext_b, whole, splits;
    void *part;
};
enum {
    FFN_PANEL_256x256 = 0,
    FFN_PANEL_256x128 = 1,
    FFN_PANEL_128x128 = 2,
    FFN_PANEL_128x128_DEEP = 3,
    FFN_PANEL_64x128 = 4,  // the forward pass only
    FFN_PANEL_CONFIGS = 5
};
hipError_t launch_ffn_panel_f16(int config, const FfnPanelCall &c, hipStream_t stream);
hipError_t launch_ffn_panel_bf16(int config, const FfnPanelCall &c, hipStream_t stream);
hipError_t launch_ffn_panel_i8(int config, const FfnPanelCall &c, hipStream_t stream);
// Both products of a backward pass (FFN_SUM2 and FFN_PAIR) in one launch of
// one tile shape; `lead`: the first one's work-groups come first.
hipError_t launch_ffn_panel_grads_f16(int config, const FfnPanelCall &x, const FfnPanelCall &w, bool lead,
                                      hipStream_t stream);
hipError_t launch_ffn_panel_grads_bf16(int config, const FfnPanelCall &x, const FfnPanelCall &w, bool lead,
                                       hipStream_t stream);

// Few tokens (M <= 64): FFN_GATED, and FFN_LINEAR on codes; kmain as above.
hipError_t launch_ffn_skinny(const FfnProduct &p, int kmain, hipStream_t stream);

// One scale and `K` int8 codes a row (dtype: tlg_dtype of X).
hipError_t launch_quantize_i8(int dtype, int64_t M, int64_t K, const void *X, int64_t ldx, int8_t *Q, int64_t ldq,
                              float *S, hipStream_t stream);

// Copies of up to three matrices with rows `pitch` bytes apart (a multiple of
// 16), zeros past each row's end.
struct FfnPack {
    int count;
    int64_t pitch;
    const void *src[3];
    void *dst[3];
    int64_t rows[3], row_bytes[3], ld_bytes[3];
};
hipError_t launch_ffn_pack(const FfnPack &p, hipStream_t stream);

// dG = dH * U * act'(G) and dU = dH * act(G) for an M x N window, written as
// two planes of M rows of `pitch` elements (a multiple of 8); columns N ..
// pitch-1 become zero. In fp16 both come times a power of two that the values
// decide, and scale->undo is its reciprocal; bf16 leaves `scale` as it is.
struct FfnGateScale {
    static constexpr int kTops = 256;
    uint32_t top[kTops];  // bounds of the magnitudes, by work-group
    float undo;
};
hipError_t launch_ffn_gate_grad(int type, int act, int M, int N, const void *dH, int64_t lddh, const void *G,
                                int64_t ldg, const void *U, int64_t ldu, void *dG, void *dU, int64_t pitch,
                                FfnGateScale *scale, const FfnPack &copies, hipStream_t stream);

// rows x cols elements of 16 bits to zero.
hipError_t launch_ffn_zero(void *p, int64_t rows, int64_t cols, int64_t ld, hipStream_t stream);

}  // namespace tlg

#endif
