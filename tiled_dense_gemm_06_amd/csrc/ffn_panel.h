// Index arithmetic of the feed-forward block's pipelined kernel: tile shapes,
// LDS layouts, what each lane of a direct-to-LDS load fetches and where each
// operand fragment is read. Plain integer arithmetic, shared with the CPU
// emulation of the kernel's data movement.
//
// An LDS stage holds 64 bytes x 2 of every row of the tile's operands: 64
// elements of 16 bits or 128 of 8. An operand comes in one of two layouts:
//   row     rows of 128 bytes, k contiguous: fragments are 16-byte reads
//   column  64 rows of k, the tile's 16-bit elements contiguous: fragments
//           are pairs of transposing 8-byte reads
// Both are BX * 128 bytes a stage, in 1 KiB slabs of one load instruction.
#ifndef TLG_FFN_PANEL_H
#define TLG_FFN_PANEL_H

#include <stdint.h>

#if defined(__HIPCC__)
#define TLG_PHD __host__ __device__ __forceinline__
#else
#define TLG_PHD inline
#endif

namespace tlg {

// BM x BN products per work-group of WM x WN waves; AST and BST LDS buffers.
template <int BM_, int BN_, int WM_, int WN_, int AST_, int BST_>
struct PanelShape {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, AST = AST_, BST = BST_;
    static constexpr int WAVES = WM * WN, NT = WAVES * 64;
    static constexpr int WTM = BM / WM, WTN = BN / WN;   // a wave's block
    static constexpr int TM = WTM / 16, TN = WTN / 16;   // 16 x 16 tiles of it
    static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
    static constexpr int DMA_A = BM / 8 / WAVES, DMA_B = BN / 8 / WAVES;  // loads a wave and stage
    static constexpr int LDS_BYTES = AST * A_BYTES + BST * B_BYTES;
    static_assert(BM % (8 * WAVES) == 0 && BN % (8 * WAVES) == 0, "whole slabs a wave");
    static_assert(WTM % 16 == 0 && WTN % 32 == 0, "whole 16 x 16 tiles, gate and up alike");
    static_assert(LDS_BYTES <= 160 * 1024, "LDS of a work-group");
};

// ---- row layout ----
// Chunk c (16 bytes) of row r lies at position c ^ ((r / 2) % 8): the 16 rows
// that a fragment read takes at one chunk fall into 16 different 16-byte slots.
TLG_PHD constexpr int prow_swizzle(int r) { return (r / 2) % 8; }
TLG_PHD constexpr int prow_offset(int r, int c) { return r * 128 + 16 * (c ^ prow_swizzle(r)); }
// Load `slab` fills rows 8*slab .. +7; lane t writes position t % 8 of row 8*slab + t/8.
TLG_PHD int prow_row(int slab, int lane) { return 8 * slab + lane / 8; }
TLG_PHD int prow_chunk(int slab, int lane) { return (lane % 8) ^ prow_swizzle(prow_row(slab, lane)); }
// The lane's byte offset from the tile's first row at the stage's first k (rows
// past `last` read that one again, their results are not stored), and its
// chunk's first k in the stage.
TLG_PHD int64_t prow_load(int slab, int lane, int64_t ld, int eb, int64_t last) {
    const int r = prow_row(slab, lane);
    return (r < last ? r : last) * ld * eb + 16 * prow_chunk(slab, lane);
}
TLG_PHD int prow_k(int slab, int lane, int eb) { return prow_chunk(slab, lane) * (16 / eb); }
// Fragment of the tile at rows r0 + 16*t (r0 a multiple of 16), 64-byte step s
// (0 or 1): 16 bytes at this offset + 2048*t.
TLG_PHD int prow_frag(int r0, int s, int lane) { return prow_offset(r0 + lane % 16, 4 * s + lane / 16); }

// ---- column layout (16-bit elements) ----
// Row k is BX elements in BX / 8 chunks; chunk c at position c ^ swizzle(k).
// The 32 lanes of half a transposing read take rows 8g + 4h + q (g = 0, 1; q =
// 0..3) of two adjacent chunks, and 4q ^ 2g spreads them over 16 slots.
TLG_PHD constexpr int pcol_swizzle(int k) { return (4 * (k & 3)) ^ (2 * ((k >> 3) & 1)); }
template <int BX>
TLG_PHD constexpr int pcol_offset(int k, int c) { return k * BX * 2 + 16 * (c ^ pcol_swizzle(k)); }
// Load `slab` fills 512 / BX rows of k; lane t writes position t % (BX / 8).
template <int BX>
TLG_PHD int pcol_k(int slab, int lane) { return slab * (512 / BX) + lane / (BX / 8); }
template <int BX>
TLG_PHD int pcol_chunk(int slab, int lane) { return (lane % (BX / 8)) ^ pcol_swizzle(pcol_k<BX>(slab, lane)); }
// The lane's byte offset from the tile's first column at the stage's first k;
// chunks that start at or past `avail` columns read the first one again.
template <int BX>
TLG_PHD int64_t pcol_load(int slab, int lane, int64_t ld, int64_t avail) {
    const int c = pcol_chunk<BX>(slab, lane);
    return pcol_k<BX>(slab, lane) * ld * 2 + (8 * c < avail ? 16 * c : 0);
}
// Transposing read of the tile at columns x0 + 16*t: this offset, + (32*s +
// 4*h) rows for 32-deep step s and half h. Lane l then holds k = 32*s +
// 8*(l/16) + 4*h + 0..3 of column x0 + 16*t + l%16.
template <int BX>
TLG_PHD int pcol_frag(int x0, int t, int lane) {
    const int i = lane % 16, k = 8 * (lane / 16) + i / 4, x = x0 + 16 * t + 4 * (i % 4);
    return pcol_offset<BX>(k, x / 8) + 2 * (x % 8);
}

// How many of the K k's of a product with a column-layout operand the loads
// cover; the others, eight at most, are staged one by one. A column-layout
// chunk that crosses the end of its row (`cols` elements, no multiple of 8)
// reads into the next row, so the last row is staged. Against a column-layout
// operand that is all: both are masked by single rows of k. A row-layout one is
// masked by whole chunks of eight, so it stops at a whole chunk: an element
// past kmain that came with its chunk would meet zeros, and an infinity times
// zero is NaN.
TLG_PHD int64_t pcol_kmain(int64_t K, int64_t cols, bool against_rows) {
    if (cols % 8 == 0) return K;
    return against_rows ? (K - 1) / 8 * 8 : K - 1;
}

// ---- gate and up side by side ----
// A gated tile's BN rows of B alternate between Wg and Wu in runs of half a
// wave's block, so that a wave holds both products of the same outputs: row r
// is row `panel_gate_n(r)` of (r / (WTN/2)) % 2 ? Wu : Wg, from the tile's first output.
template <class S>
TLG_PHD int panel_gate_half(int r) { return (r / (S::WTN / 2)) % 2; }
template <class S>
TLG_PHD int panel_gate_n(int r) { return (r / S::WTN) * (S::WTN / 2) + r % (S::WTN / 2); }

template <class S>
TLG_PHD int64_t pgate_load(int slab, int lane, int64_t ld, int eb, int64_t last) {
    const int n = panel_gate_n<S>(prow_row(slab, lane));
    return (n < last ? n : last) * ld * eb + 16 * prow_chunk(slab, lane);
}

// ---- results ----
// A wave's block of ROWS x COLS 16-bit results in LDS: piece c (8 columns) of
// row r at position c ^ (r / (16 / P)) % P, P pieces a row, so that both the
// 8-byte writes of 16 rows and the 16-byte reads of whole rows are spread over
// the banks.
template <int COLS>
TLG_PHD int presult_offset(int row, int piece) {
    constexpr int P = COLS / 8, D = P >= 16 ? 1 : 16 / P;
    return row * COLS * 2 + 16 * (piece ^ ((row / D) % P));
}

}  // namespace tlg

#endif
