// Pipelined feed-forward products for gfx950: the gated block, its gradients
// and the 8-bit products on one kernel.
//
// Mathematics. Every product sums rows against rows, sum_k A[m][k] B[n][k]:
//   gated   two of them, against Wg and Wu, then act(g) * u
//   sum2    dX = dG Wg + dU Wu, one sum over both (the second's K follows the first's)
//   pair    dWg = dG^T X and dWu = dU^T X, tiles of one launch
//   linear  int8 codes, then the scales
// so the gated block reads X once for both projections, dX is written once,
// and neither g nor u leaves the registers unless it is kept.
//
// Bound and layout. A large product is bound by the matrix cores at the clock
// that its power allows. A work-group of four waves, one per SIMD, holds 256 x 256
// products (128 x 128 a wave: 256 accumulators in AGPRs); a stage is 128 bytes
// of each row, brought by direct-to-LDS loads three (A) and two (B) buffers
// deep in the whole 160 KiB. A step is 2 * TM * TN matrix instructions with
// the LDS reads of the next fragments and the loads of a later stage slotted
// between them, so that a lone wave never waits for an operand. For the gated
// product the tile's 256 rows of B are 128 of Wg and 128 of Wu, alternating so
// that each wave has both sums of the same outputs in its registers.
// K's end is masked in the loads (a lane past it gets zeros), so the last
// stage needs no other code; only what is left past the last whole 16-byte
// chunk (K no multiple of 8 elements of 16 bits, 16 of 8 bits), or past the rows
// that a column-layout operand's chunks may cross (pcol_kmain), is staged one
// by one after the loop.
#ifndef TLG_FFN_PANEL_KERNEL_H
#define TLG_FFN_PANEL_KERNEL_H

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ffn.h"
#include "ffn_ops.h"
#include "ffn_panel.h"

namespace tlg {

namespace {

// A product with its tiles.
struct PanelArgs : FfnPanelCall {
    int tiles_m, tiles_n;  // of one output
    int group_m;
};

// The work of a launch: `whole` tiles, then the parts of the others.
template <int MODE>
__host__ __device__ __forceinline__ int panel_tile_rows(const PanelArgs &a) {
    return MODE == FFN_PAIR ? 2 * a.tiles_m : a.tiles_m;  // the pair's second output follows the first's rows
}
// Rows of a tile that its parts keep: all of them, or those of a product with fewer.
template <class S>
__host__ __device__ __forceinline__ int panel_part_rows(const PanelArgs &a) {
    return a.p.M < S::BM ? a.p.M : S::BM;
}

// 64 bytes of k of an operand's tiles in registers.
template <int T>
struct PanelFrag {
    int2_t lo[T], hi[T];
};

__device__ __forceinline__ int4_t join4(int2_t a, int2_t b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3); }

// Accumulators stay in their own AGPRs (the compiler's assignment for the
// builtin moves them to and from VGPRs around every instruction at this
// register load). What the compiler cannot see is excluded by the schedule: a
// fragment is rewritten, and an accumulator used again, only half a step of
// matrix instructions after its last use; `panel_settle` waits before anything
// else reads a result.
template <int TYPE, class Acc>
__device__ __forceinline__ void panel_mfma(Acc &acc, int4_t b, int4_t a) {
    if constexpr (TYPE == FFN_F16)
        asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
    else if constexpr (TYPE == FFN_BF16)
        asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
    else
        asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
}
// A column of them (tiles TM0 .. of fragment b) as blocks of eight or four that
// end with the wait states of a result, for code outside the schedule:
// whatever the compiler places behind such a block finds results.
template <int TYPE, int N, class Acc, int TM, int TF>
__device__ __forceinline__ void panel_mfma_fenced(Acc (&c)[TM], const PanelFrag<TF> &f, int4_t b, int m) {
    static_assert(N == 8 || N == 4, "blocks of eight or four");
#define TLG_PANEL_A(i) join4(f.lo[m + i], f.hi[m + i])
#define TLG_PANEL_FOUR(OP)                                                                             \
    asm volatile(OP " %0, %4, %5, %0\n\t" OP " %1, %4, %6, %1\n\t" OP " %2, %4, %7, %2\n\t" OP          \
                    " %3, %4, %8, %3\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7"                                  \
                 : "+a"(c[m]), "+a"(c[m + 1]), "+a"(c[m + 2]), "+a"(c[m + 3])                          \
                 : "v"(b), "v"(TLG_PANEL_A(0)), "v"(TLG_PANEL_A(1)), "v"(TLG_PANEL_A(2)), "v"(TLG_PANEL_A(3)))
#define TLG_PANEL_EIGHT(OP)                                                                            \
    asm volatile(OP " %0, %8, %9, %0\n\t" OP " %1, %8, %10, %1\n\t" OP " %2, %8, %11, %2\n\t" OP        \
                    " %3, %8, %12, %3\n\t" OP " %4, %8, %13, %4\n\t" OP " %5, %8, %14, %5\n\t" OP         \
                    " %6, %8, %15, %6\n\t" OP " %7, %8, %16, %7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7"        \
                 : "+a"(c[m]), "+a"(c[m + 1]), "+a"(c[m + 2]), "+a"(c[m + 3]), "+a"(c[m + 4]),         \
                   "+a"(c[m + 5]), "+a"(c[m + 6]), "+a"(c[m + 7])                                      \
                 : "v"(b), "v"(TLG_PANEL_A(0)), "v"(TLG_PANEL_A(1)), "v"(TLG_PANEL_A(2)),              \
                   "v"(TLG_PANEL_A(3)), "v"(TLG_PANEL_A(4)), "v"(TLG_PANEL_A(5)), "v"(TLG_PANEL_A(6)), \
                   "v"(TLG_PANEL_A(7)))
    if constexpr (N == 8) {
        if constexpr (TYPE == FFN_F16)
            TLG_PANEL_EIGHT("v_mfma_f32_16x16x32_f16");
        else if constexpr (TYPE == FFN_BF16)
            TLG_PANEL_EIGHT("v_mfma_f32_16x16x32_bf16");
        else
            TLG_PANEL_EIGHT("v_mfma_i32_16x16x64_i8");
    } else {
        if constexpr (TYPE == FFN_F16)
            TLG_PANEL_FOUR("v_mfma_f32_16x16x32_f16");
        else if constexpr (TYPE == FFN_BF16)
            TLG_PANEL_FOUR("v_mfma_f32_16x16x32_bf16");
        else
            TLG_PANEL_FOUR("v_mfma_i32_16x16x64_i8");
    }
#undef TLG_PANEL_FOUR
#undef TLG_PANEL_EIGHT
#undef TLG_PANEL_A
}
// At the end of a step: the wait states of the step's last results, taken only
// by the last one, inside the loop, so that they precede any copy of an
// accumulator that the compiler places on the way out. Only the kernels in
// which it places some have it (the assembly is scanned for such copies by a
// test): it costs a small backward pass 3 %, the large gated products nothing.
__device__ __forceinline__ void panel_leave(int next, int end) {
    asm volatile(
        "s_cmp_lt_i32 %0, %1\n\t"
        "s_cbranch_scc1 1f\n\t"
        "s_nop 7\n\ts_nop 7\n\ts_nop 7\n"
        "1:" ::"s"(next),
        "s"(end)
        : "scc", "memory");
}
// Every matrix instruction issued so far has written its result, and no read
// of an accumulator moves above this point.
template <class S, class Acc>
__device__ __forceinline__ void panel_settle(Acc (&acc)[S::TN][S::TM]) {
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
#pragma unroll
    for (int tn = 0; tn < S::TN; ++tn)
#pragma unroll
        for (int tm = 0; tm < S::TM; ++tm) asm volatile("" : "+a"(acc[tn][tm]));
}

// Defines four tiles' accumulators anew, in their AGPRs: no copy of one to a
// VGPR moves above this point. Without it the compiler makes all 256 copies
// before the choice of the activation, and spills.
template <class Acc, int TM>
__device__ __forceinline__ void panel_pin(Acc (&acc)[TM], int tm) {
#pragma unroll
    for (int i = 0; i < 4; ++i) asm volatile("" : "+a"(acc[tm + i]));
}

#define TLG_PANEL_FENCE() __builtin_amdgcn_sched_barrier(0)

template <bool COL, int T>
constexpr int kPanelReads = (COL ? 2 : 1) * T;

// Per-lane offsets of an operand's fragments: row layout, one for each 64-byte
// step; column layout, one for each tile.
template <bool COL, int T>
struct PanelLanes {
    uint32_t o[COL ? T : 2];
};
template <bool COL, int T, int BX>
__device__ __forceinline__ void panel_lanes(PanelLanes<COL, T> &l, int x0, int lane) {
    if constexpr (COL) {
#pragma unroll
        for (int t = 0; t < T; ++t) l.o[t] = (uint32_t)pcol_frag<BX>(x0, t, lane);
    } else {
        l.o[0] = (uint32_t)prow_frag(x0, 0, lane);
        l.o[1] = (uint32_t)prow_frag(x0, 1, lane);
    }
}
// Read r (0 .. kPanelReads-1) of step s.
template <bool COL, int T, int BX>
__device__ __forceinline__ void panel_read(PanelFrag<T> &f, LDS_PTR(const char) base, const PanelLanes<COL, T> &l,
                                           int s, int r) {
    if constexpr (COL) {
        const int t = r / 2, h = r % 2;
        LDS_PTR(short4_t) p = (LDS_PTR(short4_t))(base + l.o[t] + (32 * s + 4 * h) * BX * 2);
        const int2_t v = __builtin_bit_cast(int2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p));
        (h ? f.hi : f.lo)[t] = v;
    } else {
        const int4_t v = *(LDS_PTR(const int4_t))(base + l.o[s] + r * 2048);
        f.lo[r] = __builtin_shufflevector(v, v, 0, 1);
        f.hi[r] = __builtin_shufflevector(v, v, 2, 3);
    }
}

// ---- operands ----
// A tile's rows of one operand: where each load of this wave reads.
template <bool COL, int EB, int BX, int DMA>
struct PanelLoads {
    uint32_t off[DMA];  // bytes from the stage's start
    int klane[2];       // row layout: first k of the lane's chunk, by slab parity; column layout: [0] its row of k
};

template <bool COL, int EB, int BX, int DMA>
__device__ __forceinline__ void panel_loads_init(PanelLoads<COL, EB, BX, DMA> &l, int lane) {
    if constexpr (COL) {
        l.klane[0] = lane / (BX / 8);
    } else {
        l.klane[0] = prow_k(0, lane, EB);
        l.klane[1] = prow_k(1, lane, EB);
    }
}

template <bool COL, int EB, int BX, int DMA>
__device__ __forceinline__ uint32_t panel_off(const PanelLoads<COL, EB, BX, DMA> &l, int slab, int i, int klim) {
    if constexpr (COL)
        return l.klane[0] < klim - slab * (512 / BX) ? l.off[i] : kOOB;
    else
        return l.klane[slab & 1] < klim ? l.off[i] : kOOB;
}

// ---- results ----
// ROWS x COLS 16-bit results from a wave's piece of LDS to rows m .. and
// columns n .. of C, 16 bytes a lane, whole row segments an instruction.
template <int ROWS, int COLS>
__device__ __forceinline__ void panel_rows16(void *C, int64_t ldc, int M, int N, int m, int n, int lane,
                                             LDS_PTR(char) q) {
    constexpr int P = COLS / 8, RPI = 64 / P;  // rows an instruction
    const __amdgpu_buffer_rsrc_t rc =
        __builtin_amdgcn_make_buffer_rsrc((uint16_t *)C + (int64_t)m * ldc + n, (short)0, (int)kRange, 0x00020000);
    const int first = lane / P, piece = lane % P;
    if (m + ROWS <= M && n + COLS <= N) {  // the whole block
#pragma unroll
        for (int k = 0; k < ROWS / RPI; ++k) {
            const int row = k * RPI + first;
            const int4_t w = *(LDS_PTR(const int4_t))(q + presult_offset<COLS>(row, piece));
            __builtin_amdgcn_raw_buffer_store_b128(w, rc, (uint32_t)((row * ldc + 8 * piece) * 2), 0, 0);
        }
        return;
    }
#pragma unroll 4
    for (int k = 0; k < ROWS / RPI; ++k) {
        const int row = k * RPI + first;
        const int4_t w = *(LDS_PTR(const int4_t))(q + presult_offset<COLS>(row, piece));
        if (m + row >= M) continue;
        if (n + 8 * piece + 8 <= N) {
            __builtin_amdgcn_raw_buffer_store_b128(w, rc, (uint32_t)((row * ldc + 8 * piece) * 2), 0, 0);
        } else {
            uint16_t *at = (uint16_t *)C + (int64_t)(m + row) * ldc + n + 8 * piece;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (n + 8 * piece + e < N) at[e] = (uint16_t)((uint32_t)w[e / 2] >> (16 * (e % 2)));
        }
    }
}

// One wave's block of TM x T tiles of 16-bit results through its piece of LDS
// to whole row segments. val(tn, tm, v) gives the four results a lane has of
// each of the tiles (tn, tm .. tm+3).
template <class S, int T, int OUT, class F>
__device__ __forceinline__ void panel_store16(void *C, int64_t ldc, int M, int N, int m, int n, int lane,
                                              LDS_PTR(char) q, F val) {
    constexpr int COLS = T * 16;
    static_assert(S::TM % 4 == 0, "four tiles at a time");
#pragma unroll
    for (int tn = 0; tn < T; ++tn)
#pragma unroll
        for (int tm = 0; tm < S::TM; tm += 4) {
            TLG_PANEL_FENCE();  // accumulators leave the AGPRs four tiles at a time
            float v[16];
            val(tn, tm, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int2_t w = {ffn_pack32<OUT>(v[4 * i], v[4 * i + 1]), ffn_pack32<OUT>(v[4 * i + 2], v[4 * i + 3])};
                const int row = 16 * (tm + i) + lane % 16, col = 16 * tn + 4 * (lane / 16);
                *(LDS_PTR(int2_t))(q + presult_offset<COLS>(row, col / 8) + 2 * (col % 8)) = w;
            }
        }
    panel_rows16<S::WTM, COLS>(C, ldc, M, N, m, n, lane, q);
}

// A gated tile's results with the products that are kept, in one pass over the
// accumulators: 64 rows at a time, the three blocks side by side in LDS.
template <class S, int T, int TYPE, int ACT, class Acc>
__device__ __forceinline__ void panel_store_saved(const FfnProduct &p, int m, int n, int wave, int lane,
                                                  Acc (&acc)[S::TN][S::TM], LDS_PTR(char) lds) {
    constexpr int COLS = T * 16, BLOCK = 64 * COLS * 2;
    static_assert(S::WAVES * 3 * BLOCK <= S::LDS_BYTES, "three blocks a wave fit the stages' LDS");
    LDS_PTR(char) q = lds + wave * 3 * BLOCK;
#pragma unroll
    for (int tm = 0; tm < S::TM; tm += 4) {
#pragma unroll
        for (int tn = 0; tn < T; ++tn) {
            TLG_PANEL_FENCE();
            panel_pin(acc[tn], tm);
            panel_pin(acc[T + tn], tm);
            float g[16], u[16], h[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                g[i] = acc[tn][tm + i / 4][i % 4];
                u[i] = acc[T + tn][tm + i / 4][i % 4];
            }
            ffn_gate<ACT>(g, u, h);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int col = 16 * tn + 4 * (lane / 16);
                const int at = presult_offset<COLS>(16 * i + lane % 16, col / 8) + 2 * (col % 8);
                *(LDS_PTR(int2_t))(q + at) = int2_t{ffn_pack32<TYPE>(h[4 * i], h[4 * i + 1]),
                                                    ffn_pack32<TYPE>(h[4 * i + 2], h[4 * i + 3])};
                *(LDS_PTR(int2_t))(q + BLOCK + at) = int2_t{ffn_pack32<TYPE>(g[4 * i], g[4 * i + 1]),
                                                            ffn_pack32<TYPE>(g[4 * i + 2], g[4 * i + 3])};
                *(LDS_PTR(int2_t))(q + 2 * BLOCK + at) = int2_t{ffn_pack32<TYPE>(u[4 * i], u[4 * i + 1]),
                                                                ffn_pack32<TYPE>(u[4 * i + 2], u[4 * i + 3])};
            }
        }
#pragma unroll
        for (int b = 0; b < 3; ++b)
            panel_rows16<64, COLS>(p.C[b], p.ldc[b], p.M, p.N, m + 16 * tm, n, lane, q + b * BLOCK);
    }
}

// The results of a tile: m0, n0 its first row and column of the output (of
// H for a gated tile). No wave uses the stages any more.
template <class S, int TYPE, int MODE, bool SAVE, class Acc>
__device__ __forceinline__ void panel_results(const FfnProduct &p, int out, int m0, int n0, int wave, int lane,
                                              Acc (&acc)[S::TN][S::TM], LDS_PTR(char) lds) {
    constexpr int T = MODE == FFN_GATED ? S::TN / 2 : S::TN;
    const int m = m0 + (wave / S::WN) * S::WTM, n = n0 + (wave % S::WN) * (T * 16);
    LDS_PTR(char) q = lds + wave * (S::WTM * T * 32);
    if constexpr (TYPE == FFN_I8) {
        // The tile's scales, behind the results' LDS: BM of the rows, then
        // those of the columns (gated: of Wg's, then of Wu's).
        constexpr int NB = MODE == FFN_GATED ? 2 : 1, COLS = S::WN * T * 16;
        static_assert(S::BM * COLS * 2 + (S::BM + NB * COLS) * 4 <= S::LDS_BYTES, "scales fit the stages' LDS");
        LDS_PTR(float) scales = (LDS_PTR(float))(lds + S::BM * COLS * 2);
        for (int i = threadIdx.x; i < S::BM + NB * COLS; i += S::NT) {
            const int b = (i - S::BM) / COLS, row = m0 + i, col = n0 + (i - S::BM) % COLS;
            scales[i] = i < S::BM ? p.sa[row < p.M ? row : p.M - 1]
                                  : (NB == 2 && b ? p.sb[1] : p.sb[0])[col < p.N ? col : p.N - 1];
        }
        barrier_lds();
        LDS_PTR(const float) sa = scales + (wave / S::WN) * S::WTM + lane % 16;                      // + 16 * tm
        LDS_PTR(const float) sb = scales + S::BM + (wave % S::WN) * (T * 16) + 4 * (lane / 16);      // + 16 * tn
        if constexpr (MODE == FFN_GATED) {
            ffn_with_out16(p.out_type, [&](auto o) {
                ffn_with_act(p.act, [&](auto act) {
                    panel_store16<S, T, decltype(o)::value>(
                        p.C[0], p.ldc[0], p.M, p.N, m, n, lane, q, [&](int tn, int tm, float (&v)[16]) {
                            float g[16], u[16];
                            panel_pin(acc[tn], tm);
                            panel_pin(acc[T + tn], tm);
                            const float4_t bg = *(LDS_PTR(const float4_t))(sb + 16 * tn);
                            const float4_t bu = *(LDS_PTR(const float4_t))(sb + COLS + 16 * tn);
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float a = sa[16 * (tm + i / 4)];
                                g[i] = (float)acc[tn][tm + i / 4][i % 4] * (a * bg[i % 4]);
                                u[i] = (float)acc[T + tn][tm + i / 4][i % 4] * (a * bu[i % 4]);
                            }
                            ffn_gate<decltype(act)::value>(g, u, v);
                        });
                });
            });
        } else {
            auto val = [&](int tn, int tm, float (&v)[16]) {
                const float4_t b = *(LDS_PTR(const float4_t))(sb + 16 * tn);
                panel_pin(acc[tn], tm);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    v[i] = (float)acc[tn][tm + i / 4][i % 4] * (sa[16 * (tm + i / 4)] * b[i % 4]);
                    if (p.relu) v[i] = v[i] > 0.0f ? v[i] : 0.0f;
                }
            };
            if (p.out_type == TLG_F32) {
#pragma unroll
                for (int tn = 0; tn < T; ++tn)
#pragma unroll
                    for (int tm = 0; tm < S::TM; tm += 4) {
                        TLG_PANEL_FENCE();
                        float v[16];
                        val(tn, tm, v);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float w[4] = {v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
                            ffn_store4(p.C[0], p.ldc[0], TLG_F32, p.M, p.N, m + 16 * (tm + i) + lane % 16,
                                       n + 16 * tn + 4 * (lane / 16), w);
                        }
                    }
            } else {
                ffn_with_out16(p.out_type, [&](auto o) {
                    panel_store16<S, T, decltype(o)::value>(p.C[0], p.ldc[0], p.M, p.N, m, n, lane, q, val);
                });
            }
        }
    } else if constexpr (MODE == FFN_GATED) {
        ffn_with_act(p.act, [&](auto act) {
            if constexpr (SAVE) {
                panel_store_saved<S, T, TYPE, decltype(act)::value>(p, m, n, wave, lane, acc, lds);
                return;
            }
            panel_store16<S, T, TYPE>(p.C[0], p.ldc[0], p.M, p.N, m, n, lane, q,
                                      [&](int tn, int tm, float (&v)[16]) {
                                          float g[16], u[16];
                                          panel_pin(acc[tn], tm);
                                          panel_pin(acc[T + tn], tm);
#pragma unroll
                                          for (int i = 0; i < 16; ++i) {
                                              g[i] = acc[tn][tm + i / 4][i % 4];
                                              u[i] = acc[T + tn][tm + i / 4][i % 4];
                                          }
                                          ffn_gate<decltype(act)::value>(g, u, v);
                                      });
        });
    } else {
        const float undo = TYPE == FFN_F16 ? *p.undo : 1.0f;
        panel_store16<S, T, TYPE>(p.C[out], p.ldc[out], p.M, p.N, m, n, lane, q, [&](int tn, int tm, float (&v)[16]) {
            panel_pin(acc[tn], tm);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                v[i] = TYPE == FFN_F16 ? acc[tn][tm + i / 4][i % 4] * undo : acc[tn][tm + i / 4][i % 4];
        });
    }
}

// ---- the tile ----
// SAVE: a gated tile's two products are stored as well.
// Work-group `block` of a product.
template <class S, int TYPE, int MODE, bool ACOL, bool BCOL, bool SAVE>
__device__ __forceinline__ void panel_product(const PanelArgs &a, const int block, LDS_PTR(char) lds) {
    using Acc = typename FfnT<TYPE>::Acc;
    constexpr int EB = FfnT<TYPE>::EB, BK = 128 / EB;
    static_assert(EB == 2 || (!ACOL && !BCOL), "the transposing reads take 16-bit elements");
    constexpr int T = S::TM * S::TN, H = T / 2, SLOTS = 2 * T;
    constexpr int RA = kPanelReads<ACOL, S::TM>, RB = kPanelReads<BCOL, S::TN>, READS = RA + RB;
    constexpr int PER = (READS + H - 1) / H;  // LDS reads a slot
    constexpr int LOADS = S::DMA_A + S::DMA_B, SPACING = SLOTS / LOADS;
    constexpr int AHEAD_A = S::AST - 1, AHEAD_B = S::BST - 1;
    static_assert(AHEAD_A == AHEAD_B + 1, "A is one buffer deeper");
    constexpr int WAIT = (AHEAD_A - 1) * S::DMA_A + (AHEAD_B - 1) * S::DMA_B;
    constexpr int B_REGION = S::AST * S::A_BYTES;
    static_assert(1 + (LOADS - 1) * SPACING < SLOTS, "loads fit a step");
    static_assert(S::BM * S::BN * 2 <= S::LDS_BYTES, "a tile's results fit the stages");
    const FfnProduct &p = a.p;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm0 = (wave / S::WN) * S::WTM, wn0 = (wave % S::WN) * S::WTN;
    const int rows_of_tiles = panel_tile_rows<MODE>(a);
    const bool split = block >= a.whole;
    const int over = block - a.whole;
    const int tile = split ? a.whole + over / a.splits : xcd_remap(block, a.whole);
    const int part = split ? over % a.splits : 0, parts = split ? a.splits : 1;
    int tm_idx, tn_idx;
    grouped_tile(tile, rows_of_tiles, a.tiles_n, a.group_m, &tm_idx, &tn_idx);
    const int out = MODE == FFN_PAIR && tm_idx >= a.tiles_m ? 1 : 0;
    if (out) tm_idx -= a.tiles_m;
    constexpr int BNOUT = MODE == FFN_GATED ? S::BN / 2 : S::BN;
    const int m0 = tm_idx * S::BM, n0 = tn_idx * BNOUT;

    // Stages of this part; a sum2's second summand follows the first's.
    const int nks = (a.kmain + BK - 1) / BK;
    const int total = MODE == FFN_SUM2 ? 2 * nks : nks;
    const int kbeg = (int)((int64_t)part * total / parts);
    const int nk = (int)((int64_t)(part + 1) * total / parts);

    // Loads. Offsets in the tile fit 31 bits (checked by the host); a lane
    // past K, or a stage past the part's end, gets kOOB and writes zeros.
    PanelLoads<ACOL, EB, S::BM, S::DMA_A> la;
    PanelLoads<BCOL, EB, S::BN, S::DMA_B> lb;
    // A sum2's or pair's two A operands (the planes of dG and dU) have one pitch.
    const int64_t lda = ACOL ? p.A[0].ks : p.A[0].rs;
    // A gated tile's rows of B that this wave loads are all of one weight, or
    // which weight load i takes is the same for every wave.
    constexpr bool ONE_WEIGHT = MODE != FFN_GATED || (S::WTN / 16) % S::DMA_B == 0;
    static_assert(ONE_WEIGHT || S::DMA_B % (S::WTN / 8) == 0, "whole runs of both weights a wave");
    const int gate = MODE == FFN_GATED && ONE_WEIGHT ? panel_gate_half<S>(8 * wave * S::DMA_B) : 0;
    const FfnOperand &wb = gate ? p.B[1] : p.B[0];
    panel_loads_init(la, lane);
    panel_loads_init(lb, lane);
#pragma unroll
    for (int i = 0; i < S::DMA_A; ++i) {
        const int slab = wave * S::DMA_A + i;
        if constexpr (ACOL)
            la.off[i] = (uint32_t)pcol_load<S::BM>(slab, lane, lda, a.ext_a - m0);
        else
            la.off[i] = (uint32_t)prow_load(slab, lane, lda, EB, p.M - 1 - m0);
    }
    // a sum2's two weights may have leading dimensions of their own
    constexpr int SETS_B = MODE == FFN_SUM2 ? 2 : 1;
    uint32_t offb[SETS_B][S::DMA_B];
#pragma unroll
    for (int set = 0; set < SETS_B; ++set)
#pragma unroll
        for (int i = 0; i < S::DMA_B; ++i) {
            const int slab = wave * S::DMA_B + i;
            if constexpr (BCOL)
                offb[set][i] = (uint32_t)pcol_load<S::BN>(slab, lane, p.B[set].ks, a.ext_b - n0);
            else if constexpr (MODE == FFN_GATED)
                offb[set][i] = (uint32_t)pgate_load<S>(
                    slab, lane, !ONE_WEIGHT && panel_gate_half<S>(8 * i) ? p.B[1].rs : wb.rs, EB, p.N - 1 - n0);
            else
                offb[set][i] = (uint32_t)prow_load(slab, lane, wb.rs, EB, p.N - 1 - n0);
        }
    const FfnOperand &a0 = MODE == FFN_PAIR && out ? p.A[1] : p.A[0];
    const char *const abase0 = (const char *)a0.p + (int64_t)m0 * a0.rs * EB;
    const char *const bbase0 = (const char *)wb.p + (int64_t)n0 * wb.rs * EB;
    const char *const abase1 = (const char *)p.A[1].p + (int64_t)m0 * p.A[1].rs * EB;  // sum2
    const char *const bbase1 = (const char *)p.B[1].p + (int64_t)n0 * p.B[1].rs * EB;  // ... or the other weight

    // With one row of tiles every row of B is read by one work-group, and they
    // all walk along K together: rows a power of two apart then meet in the same
    // memory channels (14336 rows of 8 KiB twice, 48 tokens: 43 to 55 us by
    // where the weights lie). So each starts at a stage of its own and wraps.
    const int turn = rows_of_tiles == 1 && nk > kbeg ? tile % (nk - kbeg) : 0;

    // Load j of stage kt into buffer buf of its operand.
    auto dma = [&](int j, int kt, int buf) {
        int at = kt + turn;
        if (at >= nk) at -= nk - kbeg;
        const int seg = MODE == FFN_SUM2 && at >= nks ? 1 : 0;
        const int k0 = (at - seg * nks) * BK;
        const int klim = kt < nk ? a.kmain - k0 : 0;
        if (j < S::DMA_A) {
            const int slab = wave * S::DMA_A + j;
            const char *base = (seg ? abase1 : abase0) + (ACOL ? (int64_t)k0 * lda : (int64_t)k0) * EB;
            dma16(make_srd(base), (uint32_t)(uintptr_t)(lds + buf * S::A_BYTES + slab * 1024),
                  panel_off(la, slab, j, klim));
        } else {
            const int i = j - S::DMA_A, slab = wave * S::DMA_B + i;
            const int64_t step = BCOL ? (seg ? p.B[1].ks : p.B[0].ks) : 1;
            const bool other = MODE == FFN_GATED && !ONE_WEIGHT ? panel_gate_half<S>(8 * i) : seg;
            const char *base = (other ? bbase1 : bbase0) + (int64_t)k0 * step * EB;
            lb.off[i] = SETS_B == 2 && seg ? offb[SETS_B - 1][i] : offb[0][i];
            dma16(make_srd(base), (uint32_t)(uintptr_t)(lds + B_REGION + buf * S::B_BYTES + slab * 1024),
                  panel_off(lb, slab, i, klim));
        }
    };

    PanelLanes<ACOL, S::TM> fla;
    PanelLanes<BCOL, S::TN> flb;
    panel_lanes<ACOL, S::TM, S::BM>(fla, wm0, lane);
    panel_lanes<BCOL, S::TN, S::BN>(flb, wn0, lane);

    Acc acc[S::TN][S::TM];
#pragma unroll
    for (int i = 0; i < S::TN; ++i)
#pragma unroll
        for (int j = 0; j < S::TM; ++j) acc[i][j] = Acc{0, 0, 0, 0};
    // the first step's first half multiplies zeros
    PanelFrag<S::TM> fa[2];
    PanelFrag<S::TN> fb[2];
#pragma unroll
    for (int t = 0; t < S::TM; ++t) fa[1].lo[t] = fa[1].hi[t] = int2_t{0, 0};
#pragma unroll
    for (int t = 0; t < S::TN; ++t) fb[1].lo[t] = fb[1].hi[t] = int2_t{0, 0};

    auto read = [&](int f, LDS_PTR(const char) sA, LDS_PTR(const char) sB, int s, int r) {
        // in the order of use: b[0], every a, the other b
        constexpr int B0 = BCOL ? 2 : 1;
        if (r < B0)
            panel_read<BCOL, S::TN, S::BN>(fb[f], sB, flb, s, r);
        else if (r < B0 + RA)
            panel_read<ACOL, S::TM, S::BM>(fa[f], sA, fla, s, r - B0);
        else
            panel_read<BCOL, S::TN, S::BN>(fb[f], sB, flb, s, r - RA);
    };
    auto mfma = [&](int f, int i) {
        const int tn = i / S::TM, tm = i % S::TM;
        panel_mfma<TYPE>(acc[tn][tm], join4(fb[f].lo[tn], fb[f].hi[tn]), join4(fa[f].lo[tm], fa[f].hi[tm]));
    };

    // B is loaded AHEAD_B stages ahead, A one more; each step issues B's loads first
#pragma unroll
    for (int s = 0; s < AHEAD_A; ++s) {
        if (s < AHEAD_B)
#pragma unroll
            for (int j = S::DMA_A; j < LOADS; ++j) dma(j, kbeg + s, s);
#pragma unroll
        for (int j = 0; j < S::DMA_A; ++j) dma(j, kbeg + s, s);
    }
    wait_vmcnt<WAIT>();
    barrier_lds();

    int abuf = 0, bbuf = 0;
    for (int kt = kbeg; kt < nk; ++kt) {
        const int nabuf = abuf == 0 ? S::AST - 1 : abuf - 1, nbbuf = bbuf == 0 ? S::BST - 1 : bbuf - 1;
        LDS_PTR(const char) sA = lds + abuf * S::A_BYTES;
        LDS_PTR(const char) sB = lds + B_REGION + bbuf * S::B_BYTES;
        TLG_PANEL_FENCE();
        // slots 0 .. H-1: the last half of the previous stage's second step,
        // with the reads of this stage's first; H .. H+T-1: the first step,
        // with the reads of the second; the rest: the second step's first half
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) {
            if (q < H) {
                mfma(1, H + q);
#pragma unroll
                for (int r = q * PER; r < (q + 1) * PER; ++r)
                    if (r < READS) read(0, sA, sB, 0, r);
            } else if (q < H + T) {
                mfma(0, q - H);
#pragma unroll
                for (int r = (q - H) * PER; r < (q - H + 1) * PER; ++r)
                    if (r < READS) read(1, sA, sB, 1, r);
            } else {
                mfma(1, q - H - T);
            }
            if (q >= 1 && (q - 1) % SPACING == 0 && (q - 1) / SPACING < LOADS) {
                const int i = (q - 1) / SPACING, j = i < S::DMA_B ? S::DMA_A + i : i - S::DMA_B;
                if (j < S::DMA_A)
                    dma(j, kt + AHEAD_A, nabuf);
                else
                    dma(j, kt + AHEAD_B, nbbuf);
            }
            TLG_PANEL_FENCE();
        }
        wait_vmcnt<WAIT>();  // this wave's loads of the next stage are in LDS
        barrier_lds();       // ... and every wave's; no wave reads this stage any more
        abuf = abuf == S::AST - 1 ? 0 : abuf + 1;
        bbuf = bbuf == S::BST - 1 ? 0 : bbuf + 1;
        if constexpr (MODE == FFN_GATED && (SAVE || TYPE == FFN_I8)) panel_leave(kt + 1, nk);
    }
    constexpr int BLOCK = S::TM % 8 == 0 ? 8 : 4;
#pragma unroll
    for (int i = H; i < T; i += BLOCK)
        panel_mfma_fenced<TYPE, BLOCK>(acc[i / S::TM], fa[1], join4(fb[1].lo[i / S::TM], fb[1].hi[i / S::TM]),
                                       i % S::TM);
    wait_vmcnt<0>();  // no load may still be writing LDS
    panel_settle<S>(acc);

    // The k's past kmain (fewer than two chunks): 64 bytes of each row staged
    // by element, zeros outside. Of a sum2 the first summand's come as the
    // first 32 bytes and the second's as the others.
    if (a.kmain < p.K && part == parts - 1) {
        using E = typename FfnT<TYPE>::Elem;
        constexpr int SEGS = MODE == FFN_SUM2 ? 2 : 1, PER = 16 / EB;  // elements of a chunk
        barrier_lds();
        // The first of the two chunks of a half holds the k's, the second zeros.
        // All of a thread's loads are issued before the first is used.
        auto stage = [&](auto col, auto bx, LDS_PTR(char) dst, auto at) {
            constexpr int BX = decltype(bx)::value;
            if constexpr (decltype(col)::value) {
                // rows k = 0..7 of each half, eight columns a thread
                constexpr int CHUNKS = 32 * BX / 8, PASSES = CHUNKS / S::NT;
                E v[PASSES][8];
#pragma unroll
                for (int i = 0; i < PASSES; ++i) {
                    const int q = i * S::NT + threadIdx.x, k = q / (BX / 8), x = q % (BX / 8) * 8;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[i][e] = k % 16 < 8 && k / 16 < SEGS ? at(x + e, k / 16, a.kmain + k % 16) : (E)0;
                }
#pragma unroll
                for (int i = 0; i < PASSES; ++i) {
                    const int q = i * S::NT + threadIdx.x;
                    int4_t w;
                    __builtin_memcpy(&w, v[i], 16);
                    *(LDS_PTR(int4_t))(dst + pcol_offset<BX>(q / (BX / 8), q % (BX / 8))) = w;
                }
            } else {
                constexpr int PASSES = (BX + S::NT - 1) / S::NT;
#pragma unroll
                for (int i = 0; i < PASSES; ++i) {
                    const int x = i * S::NT + threadIdx.x;
                    if (x >= BX) break;
                    E v[SEGS][PER];
#pragma unroll
                    for (int g = 0; g < SEGS; ++g)
#pragma unroll
                        for (int e = 0; e < PER; ++e) v[g][e] = at(x, g, a.kmain + e);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        int4_t w = {0, 0, 0, 0};
                        if (c % 2 == 0 && c / 2 < SEGS) __builtin_memcpy(&w, v[c / 2 < SEGS ? c / 2 : 0], 16);
                        *(LDS_PTR(int4_t))(dst + prow_offset(x, c)) = w;
                    }
                }
            }
        };
        stage(FfnConst<ACOL>(), FfnConst<S::BM>(), lds, [&](int x, int seg, int k) {
            const FfnOperand &o = p.A[MODE == FFN_PAIR ? out : seg];
            return m0 + x < p.M && k < p.K ? ((const E *)o.p)[(int64_t)(m0 + x) * o.rs + (int64_t)k * o.ks] : (E)0;
        });
        stage(FfnConst<BCOL>(), FfnConst<S::BN>(), lds + B_REGION, [&](int x, int seg, int k) {
            const int which = MODE == FFN_GATED ? panel_gate_half<S>(x) : seg;
            const int n = n0 + (MODE == FFN_GATED ? panel_gate_n<S>(x) : x);
            const FfnOperand &o = p.B[which];
            return n < p.N && k < p.K ? ((const E *)o.p)[(int64_t)n * o.rs + (int64_t)k * o.ks] : (E)0;
        });
        barrier_lds();
#pragma unroll
        for (int r = 0; r < READS; ++r) read(0, lds, lds + B_REGION, 0, r);
#pragma unroll
        for (int tn = 0; tn < S::TN; ++tn)
#pragma unroll
            for (int tm = 0; tm < S::TM; tm += BLOCK)
                panel_mfma_fenced<TYPE, BLOCK>(acc[tn], fa[0], join4(fb[0].lo[tn], fb[0].hi[tn]), tm);
    }
    barrier_lds();  // every wave is done with the stages
    if (split) {
        // raw sums of the tile, [tile][part][product][row][column]
        constexpr int PRODUCTS = MODE == FFN_GATED ? 2 : 1, TO = S::TN / PRODUCTS;
        const int rows = panel_part_rows<S>(a), row = wm0 + lane % 16;
        const int col = (wave % S::WN) * (TO * 16) + 4 * (lane / 16);
#pragma unroll
        for (int tn = 0; tn < S::TN; ++tn) {
            Acc *to = (Acc *)a.part + (((int64_t)over * PRODUCTS + tn / TO) * rows * BNOUT + col + 16 * (tn % TO)) / 4;
#pragma unroll
            for (int tm = 0; tm < S::TM; tm += 4) panel_pin(acc[tn], tm);
#pragma unroll
            for (int tm = 0; tm < S::TM; ++tm)
                if (row + 16 * tm < rows) to[(row + 16 * tm) * (BNOUT / 4)] = acc[tn][tm];
        }
        return;
    }
    panel_results<S, TYPE, MODE, SAVE>(p, out, m0, n0, wave, lane, acc, lds);
}

template <class S>
constexpr int kPanelGroupsPerCu = S::LDS_BYTES <= 80 * 1024 ? 2 : 1;

template <class S, int TYPE, int MODE, bool ACOL, bool BCOL, bool SAVE>
__global__ __launch_bounds__(S::NT, kPanelGroupsPerCu<S>) void k_ffn_panel(const PanelArgs a) {
    __shared__ __attribute__((aligned(1024))) char smem[S::LDS_BYTES];
    panel_product<S, TYPE, MODE, ACOL, BCOL, SAVE>(a, blockIdx.x, (LDS_PTR(char))smem);
}

// Both products of a backward pass: the first `lead` work-groups are of the
// one with the longer sums, so that the other's fill what it leaves free, and
// neither a launch nor a round's end lies between them. Two launches against
// this one: 3001 x 1537 from 2049 123.5 against 112.7 us, 353 x 4409 from 1117
// 59.7 against 44.6 (31 random backward passes: 0.81 of the time).
template <class S, int TYPE>
__global__ __launch_bounds__(S::NT, kPanelGroupsPerCu<S>) void k_ffn_panel_grads(const PanelArgs x, const PanelArgs w,
                                                                                 int lead, int x_leads) {
    __shared__ __attribute__((aligned(1024))) char smem[S::LDS_BYTES];
    const int b = blockIdx.x;
    const bool leads = b < lead;
    const int block = leads ? b : b - lead;
    if (leads == (x_leads != 0))
        panel_product<S, TYPE, FFN_SUM2, false, true, false>(x, block, (LDS_PTR(char))smem);
    else
        panel_product<S, TYPE, FFN_PAIR, true, true, false>(w, block, (LDS_PTR(char))smem);
}

// The parts of split tile `over` added in order, then its results: four of a
// row a thread.
template <class S, int TYPE, int MODE>
__device__ __forceinline__ void panel_join(const PanelArgs &a, int over) {
    using Acc = typename FfnT<TYPE>::Acc;
    constexpr int NB = MODE == FFN_GATED ? 2 : 1, BNOUT = S::BN / NB, QUADS = BNOUT / 4;
    const FfnProduct &p = a.p;
    int tm_idx, tn_idx;
    grouped_tile(a.whole + over, panel_tile_rows<MODE>(a), a.tiles_n, a.group_m, &tm_idx, &tn_idx);
    const int out = MODE == FFN_PAIR && tm_idx >= a.tiles_m ? 1 : 0;
    if (out) tm_idx -= a.tiles_m;
    const int rows = panel_part_rows<S>(a), i = blockIdx.x * 256 + threadIdx.x;
    const int m = tm_idx * S::BM + i / QUADS, n = tn_idx * BNOUT + i % QUADS * 4;
    if (i >= rows * QUADS || m >= p.M || n >= p.N) return;
    Acc sum[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) sum[b] = Acc{0, 0, 0, 0};
    const Acc *from = (const Acc *)a.part + (int64_t)over * a.splits * NB * rows * QUADS + i;
    // eight parts' loads in flight, added in order
    int s = 0;
    for (; s + 8 <= a.splits; s += 8) {
        Acc v[8][NB];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int b = 0; b < NB; ++b) v[j][b] = from[(int64_t)((s + j) * NB + b) * rows * QUADS];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int b = 0; b < NB; ++b) sum[b] += v[j][b];
    }
#pragma unroll 4
    for (; s < a.splits; ++s)
#pragma unroll
        for (int b = 0; b < NB; ++b) sum[b] += from[(int64_t)(s * NB + b) * rows * QUADS];
    float v[NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[b][e] = (float)sum[b][e];
            if constexpr (TYPE == FFN_I8) v[b][e] *= p.sa[m] * p.sb[b][n + e < p.N ? n + e : p.N - 1];
        }
    if constexpr (MODE == FFN_GATED) {
        float h[4];
        ffn_with_act(p.act, [&](auto act) {
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = ffn_act<decltype(act)::value>(v[0][e]) * v[1][e];
        });
        ffn_store4(p.C[0], p.ldc[0], p.out_type, p.M, p.N, m, n, h);
        if (p.C[1]) {
            ffn_store4(p.C[1], p.ldc[1], p.out_type, p.M, p.N, m, n, v[0]);
            ffn_store4(p.C[2], p.ldc[2], p.out_type, p.M, p.N, m, n, v[1]);
        }
    } else {
        if (MODE == FFN_LINEAR && p.relu)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[0][e] = v[0][e] > 0.0f ? v[0][e] : 0.0f;
        if constexpr (TYPE == FFN_F16) {
            const float undo = *p.undo;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[0][e] *= undo;
        }
        ffn_store4(p.C[out], p.ldc[out], p.out_type, p.M, p.N, m, n, v[0]);
    }
}

template <class S, int TYPE, int MODE>
__global__ __launch_bounds__(256) void k_ffn_panel_join(const PanelArgs a) {
    panel_join<S, TYPE, MODE>(a, blockIdx.y);
}
template <class S, int TYPE>
__global__ __launch_bounds__(256) void k_ffn_panel_grads_join(const PanelArgs x, const PanelArgs w, int x_tiles) {
    if ((int)blockIdx.y < x_tiles)
        panel_join<S, TYPE, FFN_SUM2>(x, blockIdx.y);
    else
        panel_join<S, TYPE, FFN_PAIR>(w, blockIdx.y - x_tiles);
}

// Waves of 128 x 128, one work-group a CU.
using Panel256 = PanelShape<256, 256, 2, 2, 3, 2>;
// Waves of 128 x 64, one work-group a CU.
using Panel256x128 = PanelShape<256, 128, 2, 2, 3, 2>;
// Waves of 64 x 64: two work-groups a CU, or one with four stages in flight.
using Panel128 = PanelShape<128, 128, 2, 2, 3, 2>;
using Panel128Deep = PanelShape<128, 128, 2, 2, 5, 4>;
// Waves of 64 x 32, six stages in flight: weights at the rate of HBM.
using Panel64 = PanelShape<64, 128, 1, 4, 7, 6>;

// A call's tiles and work-groups, and the blocks of its join.
template <class S, int MODE>
struct PanelGrid {
    PanelArgs a;
    int tiles;
    explicit PanelGrid(const FfnPanelCall &c) : a{c, 0, 0, 4} {
        const int n = MODE == FFN_GATED ? S::BN / 2 : S::BN;
        a.tiles_m = (a.p.M + S::BM - 1) / S::BM;
        a.tiles_n = (a.p.N + n - 1) / n;
        tiles = panel_tile_rows<MODE>(a) * a.tiles_n;
        if (a.splits < 2) a.whole = tiles;
    }
    unsigned groups() const { return (unsigned)(a.whole + (tiles - a.whole) * a.splits); }
    unsigned split_tiles() const { return (unsigned)(tiles - a.whole); }
    unsigned join_blocks() const {
        const int quads = panel_part_rows<S>(a) * ((MODE == FFN_GATED ? S::BN / 2 : S::BN) / 4);
        return split_tiles() ? (unsigned)((quads + 255) / 256) : 0;
    }
};

template <class S, int TYPE, int MODE, bool ACOL, bool BCOL>
hipError_t launch_t(const FfnPanelCall &c, hipStream_t stream) {
    const PanelGrid<S, MODE> g(c);
    constexpr bool CAN_SAVE = MODE == FFN_GATED && TYPE != FFN_I8;
    if (CAN_SAVE && c.p.C[1])
        hipLaunchKernelGGL((k_ffn_panel<S, TYPE, MODE, ACOL, BCOL, CAN_SAVE>), dim3(g.groups()), dim3(S::NT), 0,
                           stream, g.a);
    else
        hipLaunchKernelGGL((k_ffn_panel<S, TYPE, MODE, ACOL, BCOL, false>), dim3(g.groups()), dim3(S::NT), 0, stream,
                           g.a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !g.split_tiles()) return e;
    hipLaunchKernelGGL((k_ffn_panel_join<S, TYPE, MODE>), dim3(g.join_blocks(), g.split_tiles()), dim3(256), 0, stream,
                       g.a);
    return hipGetLastError();
}

template <class S, int TYPE>
hipError_t launch_grads(const FfnPanelCall &x, const FfnPanelCall &w, bool lead, hipStream_t stream) {
    const PanelGrid<S, FFN_SUM2> gx(x);
    const PanelGrid<S, FFN_PAIR> gw(w);
    hipLaunchKernelGGL((k_ffn_panel_grads<S, TYPE>), dim3(gx.groups() + gw.groups()), dim3(S::NT), 0, stream, gx.a,
                       gw.a, (int)(lead ? gx.groups() : gw.groups()), (int)lead);
    hipError_t e = hipGetLastError();
    const unsigned joins = gx.split_tiles() + gw.split_tiles();
    if (e != hipSuccess || !joins) return e;
    const unsigned bx = gx.join_blocks(), bw = gw.join_blocks();
    hipLaunchKernelGGL((k_ffn_panel_grads_join<S, TYPE>), dim3(bx > bw ? bx : bw, joins), dim3(256), 0, stream, gx.a,
                       gw.a, (int)gx.split_tiles());
    return hipGetLastError();
}

template <class S, int TYPE, bool BACKWARD>
hipError_t launch_shape(const FfnPanelCall &a, hipStream_t stream) {
    if constexpr (TYPE == FFN_I8) {
        if (a.p.mode == FFN_GATED) return launch_t<S, TYPE, FFN_GATED, false, false>(a, stream);
        if (a.p.mode == FFN_LINEAR) return launch_t<S, TYPE, FFN_LINEAR, false, false>(a, stream);
    } else {
        if (a.p.mode == FFN_GATED) return launch_t<S, TYPE, FFN_GATED, false, false>(a, stream);
        if constexpr (BACKWARD) {
            if (a.p.mode == FFN_SUM2) return launch_t<S, TYPE, FFN_SUM2, false, true>(a, stream);
            if (a.p.mode == FFN_PAIR) return launch_t<S, TYPE, FFN_PAIR, true, true>(a, stream);
        }
    }
    return hipErrorInvalidValue;
}

}  // namespace

// The kernels of one operand type (a source file each).
template <int TYPE>
hipError_t launch_ffn_panel_type(int config, const FfnPanelCall &a, hipStream_t stream) {
    switch (config) {
        case FFN_PANEL_256x256: return launch_shape<Panel256, TYPE, true>(a, stream);
        case FFN_PANEL_256x128: return launch_shape<Panel256x128, TYPE, true>(a, stream);
        case FFN_PANEL_128x128: return launch_shape<Panel128, TYPE, true>(a, stream);
        case FFN_PANEL_128x128_DEEP: return launch_shape<Panel128Deep, TYPE, true>(a, stream);
        case FFN_PANEL_64x128: return launch_shape<Panel64, TYPE, false>(a, stream);
        default: return hipErrorInvalidValue;
    }
}
template <int TYPE>
hipError_t launch_ffn_panel_grads_type(int config, const FfnPanelCall &x, const FfnPanelCall &w, bool lead,
                                       hipStream_t stream) {
    switch (config) {
        case FFN_PANEL_256x256: return launch_grads<Panel256, TYPE>(x, w, lead, stream);
        case FFN_PANEL_256x128: return launch_grads<Panel256x128, TYPE>(x, w, lead, stream);
        case FFN_PANEL_128x128: return launch_grads<Panel128, TYPE>(x, w, lead, stream);
        case FFN_PANEL_128x128_DEEP: return launch_grads<Panel128Deep, TYPE>(x, w, lead, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace tlg

#endif
