// Host emulation of the sum of the pipelined kernel's products with a
// column-layout operand: which k's of each operand the masked loads bring
// (index functions of ffn_panel.h), the products of what they bring, zeros in
// the place of what they leave out, and the staged k's after them. Values are
// floats with an infinity among them, so an element that meets the zeros of
// the other operand shows as NaN.
//
// usage: ffn_mixed_emu; prints "ok" or what is wrong
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "ffn_panel.h"

using namespace tlg;

static int failures = 0;
static void fail(const char *what, int64_t K, int64_t cols, int at) {
    if (failures++ < 10) printf("%s: K %lld, rows of %lld, infinity at %d\n", what, (long long)K, (long long)cols, at);
}

// Elements of the stage at k0 that a row-layout, and a column-layout, operand's loads bring.
static void row_in(bool (&in)[64], int64_t left) {
    for (bool &b : in) b = false;
    for (int lane = 0; lane < 64; ++lane)
        if (prow_row(0, lane) == 0 && prow_k(0, lane, 2) < left)
            for (int e = 0; e < 8; ++e) in[prow_k(0, lane, 2) + e] = true;
}
template <int BX>
static void col_in(bool (&in)[64], int64_t left) {
    for (int k = 0; k < 64; ++k) in[k] = false;
    for (int slab = 0; slab < BX / 8; ++slab)
        for (int lane = 0; lane < 64; ++lane)
            if (pcol_k<BX>(slab, lane) < left) in[pcol_k<BX>(slab, lane)] = true;
}

// One output of a product over K, an infinity in A's element `at`.
template <int BX>
static void check(int64_t K, int64_t cols, bool rows, int at) {
    const auto a = [&](int64_t k) { return k >= K ? 0.0f : k == at ? INFINITY : (float)(k % 5 + 1); };  // zeros past a plane's rows
    const auto b = [&](int64_t k) { return k >= K ? 99.0f : (float)(k % 3 + 1); };
    const int64_t kmain = pcol_kmain(K, cols, rows);
    if (kmain < 0 || kmain > K || K - kmain > 8) fail("k's left to stage", K, cols, at);
    if (cols % 8 && kmain > K - 1) fail("the last row's chunks cross its end", K, cols, at);
    float sum = 0, want = 0;
    int64_t seen = 0;
    for (int64_t k0 = 0; k0 < kmain; k0 += 64) {
        bool ain[64], bin[64];
        if (rows)
            row_in(ain, kmain - k0);
        else
            col_in<BX>(ain, kmain - k0);
        col_in<BX>(bin, kmain - k0);
        for (int k = 0; k < 64; ++k) {
            sum += (ain[k] ? a(k0 + k) : 0.0f) * (bin[k] ? b(k0 + k) : 0.0f);
            seen += ain[k] && bin[k] && k0 + k < K;
        }
    }
    for (int64_t k = kmain; k < K; ++k, ++seen) sum += a(k) * b(k);
    for (int64_t k = 0; k < K; ++k) want += a(k) * b(k);
    if (seen != K) fail("not every k once", K, cols, at);
    if (!(sum == want)) fail("sum", K, cols, at);  // NaN included
}

int main() {
    for (int64_t K = 1; K <= 200; ++K)
        for (int64_t cols = 8; cols < 24; ++cols)
            for (int rows = 0; rows < 2; ++rows)
                for (int64_t at = K - 10; at < K; ++at) {
                    check<256>(K, cols, rows, (int)at);
                    check<128>(K, cols, rows, (int)at);
                }
    if (failures) {
        printf("%d failures\n", failures);
        return 1;
    }
    printf("ok\n");
    return 0;
}
