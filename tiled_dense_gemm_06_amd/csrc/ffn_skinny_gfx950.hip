// Feed-forward products of few tokens (M <= 64) for gfx950: the gated block
// and the int8 products while decoding.
//
// Bound. Every weight is read once and used for M tokens only, so the call is
// a read of the weights at the rate that HBM gives, and what matters is bytes
// in flight: a work-group takes a strip of 16 outputs (with both weights' rows
// of them), its waves interleave over K in blocks of 256 bytes a row, and
// each wave holds a block's loads while it multiplies the one before. Weights
// go from memory to the matrix cores' operand registers without LDS: a lane
// reads 16 bytes of row lane % 16, four loads cover 256 contiguous bytes of
// each row. X is small enough to stay in L2 and is read the same way. The
// waves' sums meet in LDS and are added in wave order, so results do not
// depend on timing.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ffn.h"
#include "ffn_ops.h"

namespace tlg {

namespace {

__device__ __forceinline__ __amdgpu_buffer_rsrc_t skinny_rsrc(const void *base) {
    return __builtin_amdgcn_make_buffer_rsrc((void *)base, (short)0, (int)kRange, 0x00020000);
}
__device__ __forceinline__ int4_t skinny_load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(int4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// TM tiles of 16 tokens, 16 outputs, K split over WAVES waves.
template <int TYPE, int MODE, int TM, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void k_ffn_skinny(const FfnProduct p, int kmain) {
    using T = FfnT<TYPE>;
    using Acc = typename T::Acc;
    using E = typename T::Elem;
    constexpr int EB = T::EB, NB = MODE == FFN_GATED ? 2 : 1, J = 4;  // J loads: 256 bytes of a row
    constexpr int BK = J * 64 / EB, PER = 16 / EB;
    __shared__ Acc part[WAVES][NB * TM][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane % 16, g = lane / 16;
    const int64_t n0 = (int64_t)blockIdx.x * 16;

    // rows past the last one read the last one again; their sums are not stored
    uint32_t offa[TM], offb[NB];
#pragma unroll
    for (int t = 0; t < TM; ++t) {
        const int m = 16 * t + r;
        offa[t] = (uint32_t)((m < p.M ? m : p.M - 1) * p.A[0].rs * EB + 16 * g);
    }
    const int64_t last = p.N - 1 - n0;
#pragma unroll
    for (int b = 0; b < NB; ++b) offb[b] = (uint32_t)((r < last ? r : last) * p.B[b].rs * EB + 16 * g);
    const __amdgpu_buffer_rsrc_t ra = skinny_rsrc(p.A[0].p);
    __amdgpu_buffer_rsrc_t rb[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) rb[b] = skinny_rsrc((const char *)p.B[b].p + n0 * p.B[b].rs * EB);

    struct Block {
        int4_t a[TM][J], b[NB][J];
    };
    // Block `i` of K; a lane whose 16 bytes start at or past kmain gets zeros.
    auto load = [&](Block &x, int i) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int k = i * BK + j * (64 / EB);
            const bool in = k + g * PER < kmain;
            const uint32_t at = (uint32_t)(k * EB);
#pragma unroll
            for (int b = 0; b < NB; ++b) x.b[b][j] = skinny_load(rb[b], in ? offb[b] + at : kOOB);
#pragma unroll
            for (int t = 0; t < TM; ++t) x.a[t][j] = skinny_load(ra, in ? offa[t] + at : kOOB);
        }
    };
    Acc acc[NB][TM];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int m = 0; m < TM; ++m) acc[b][m] = Acc{0, 0, 0, 0};
    auto multiply = [&](const Block &x) {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int m = 0; m < TM; ++m) acc[b][m] = T::mfma(x.b[b][j], x.a[m][j], acc[b][m]);
    };
    // (a start of its own for every strip, as the 64-token tiles have, costs
    // here: 1 token 4096 -> 14336 43.8 against 42.8 us; the waves' blocks
    // already cover 2 KiB of each row at a time)
    const int blocks = (kmain + BK - 1) / BK;
    Block x[2];
    if (wave < blocks) load(x[0], wave);
    for (int i = wave; i < blocks; i += 2 * WAVES) {
        if (i + WAVES < blocks) load(x[1], i + WAVES);
        multiply(x[0]);
        if (i + WAVES < blocks) {
            if (i + 2 * WAVES < blocks) load(x[0], i + 2 * WAVES);
            multiply(x[1]);
        }
    }
    if (kmain < p.K && wave == WAVES - 1) {
        // the k's past the last whole 16 bytes, by element, in the lanes of g == 0
        Block y;
        auto tail = [&](const void *base, int64_t row, int64_t rs) {
            E v[PER];
#pragma unroll
            for (int e = 0; e < PER; ++e)
                v[e] = g == 0 && kmain + e < p.K ? ((const E *)base)[row * rs + kmain + e] : (E)0;
            int4_t w;
            __builtin_memcpy(&w, v, 16);
            return w;
        };
#pragma unroll
        for (int t = 0; t < TM; ++t) {
            const int m = 16 * t + r;
            y.a[t][0] = tail(p.A[0].p, m < p.M ? m : p.M - 1, p.A[0].rs);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            y.b[b][0] = tail(p.B[b].p, n0 + (r < last ? r : last), p.B[b].rs);
#pragma unroll
            for (int m = 0; m < TM; ++m) acc[b][m] = T::mfma(y.b[b][0], y.a[m][0], acc[b][m]);
        }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int m = 0; m < TM; ++m) part[wave][b * TM + m][lane] = acc[b][m];
    __syncthreads();
    // lane l: token 16 * m + l % 16, outputs 4 * (l / 16) .. +3
    for (int m = wave; m < TM; m += WAVES) {
        const int row = 16 * m + r, col = (int)n0 + 4 * g;
        float v[NB][4];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            Acc s = part[0][b * TM + m][lane];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) s += part[w][b * TM + m][lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[b][e] = (float)s[e];
                if constexpr (TYPE == FFN_I8)
                    v[b][e] *= p.sa[row < p.M ? row : p.M - 1] * p.sb[b][col + e < p.N ? col + e : p.N - 1];
            }
        }
        if constexpr (MODE == FFN_GATED) {
            float h[4];
            ffn_with_act(p.act, [&](auto act) {
#pragma unroll
                for (int e = 0; e < 4; ++e) h[e] = ffn_act<decltype(act)::value>(v[0][e]) * v[1][e];
            });
            ffn_store4(p.C[0], p.ldc[0], p.out_type, p.M, p.N, row, col, h);
            if (p.C[1]) {
                ffn_store4(p.C[1], p.ldc[1], p.out_type, p.M, p.N, row, col, v[0]);
                ffn_store4(p.C[2], p.ldc[2], p.out_type, p.M, p.N, row, col, v[1]);
            }
        } else {
            if (p.relu)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[0][e] = v[0][e] > 0.0f ? v[0][e] : 0.0f;
            ffn_store4(p.C[0], p.ldc[0], p.out_type, p.M, p.N, row, col, v[0]);
        }
    }
}

template <int TYPE, int MODE, int TM, int WAVES>
hipError_t launch_t(const FfnProduct &p, int kmain, hipStream_t stream) {
    const unsigned strips = (unsigned)(((int64_t)p.N + 15) / 16);
    hipLaunchKernelGGL((k_ffn_skinny<TYPE, MODE, TM, WAVES>), dim3(strips), dim3(WAVES * 64), 0, stream, p,
                       kmain);
    return hipGetLastError();
}

template <int TYPE, int MODE>
hipError_t launch_rows(const FfnProduct &p, int kmain, hipStream_t stream) {
    const int tm = (p.M + 15) / 16;
    switch (tm) {
        case 1: return launch_t<TYPE, MODE, 1, 8>(p, kmain, stream);
        case 2: return launch_t<TYPE, MODE, 2, 8>(p, kmain, stream);
        case 3:
        case 4: return launch_t<TYPE, MODE, 4, 8>(p, kmain, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_ffn_skinny(const FfnProduct &p, int kmain, hipStream_t stream) {
    if (p.M < 1 || p.M > 64 || p.N < 1) return hipErrorInvalidValue;
    switch (p.type * 4 + p.mode) {
        case FFN_F16 * 4 + FFN_GATED: return launch_rows<FFN_F16, FFN_GATED>(p, kmain, stream);
        case FFN_BF16 * 4 + FFN_GATED: return launch_rows<FFN_BF16, FFN_GATED>(p, kmain, stream);
        case FFN_I8 * 4 + FFN_GATED: return launch_rows<FFN_I8, FFN_GATED>(p, kmain, stream);
        case FFN_I8 * 4 + FFN_LINEAR: return launch_rows<FFN_I8, FFN_LINEAR>(p, kmain, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace tlg
