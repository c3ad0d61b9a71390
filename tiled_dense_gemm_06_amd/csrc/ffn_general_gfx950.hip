// Feed-forward kernels for gfx950: the general product (any strides, any
// alignment), the gradient of the gate, the token quantiser and a zero fill.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ffn.h"
#include "ffn_ops.h"

namespace tlg {

namespace {

// ---- the general product ----
// 64 x 64 outputs per work-group of four waves, each 32 x 32 in 2 x 2 tiles
// of 16 x 16. A stage is 64 bytes of each row (32 elements of 16 bits or 64
// of 8), fetched element by element with bounds checks and zeros outside, so
// every stride and alignment works; rows are 80 bytes apart in LDS. It serves
// what the pipelined kernels refuse: leading dimensions whose tile offsets do
// not fit 31 bits, and gradients of fewer than 8 columns.
constexpr int GT = 64, GROW = 80;

template <int TYPE>
__device__ __forceinline__ void gen_stage(const FfnOperand &o, int rows, int K, int r0, int k0, char *dst, int tid) {
    using E = typename FfnT<TYPE>::Elem;
    constexpr int PER = 16 / FfnT<TYPE>::EB;
    const int r = tid / 4, c = tid % 4;
    const E *p = (const E *)o.p + (int64_t)(r0 + r) * o.rs;
    E v[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        const int k = k0 + c * PER + e;
        v[e] = (r0 + r < rows && k < K) ? p[(int64_t)k * o.ks] : (E)0;
    }
    int4_t w;
    __builtin_memcpy(&w, v, 16);
    *(int4_t *)(dst + r * GROW + c * 16) = w;
}

template <int TYPE, int MODE>
__global__ __launch_bounds__(256) void k_ffn_general(const FfnProduct p, int tiles_n) {
    using T = FfnT<TYPE>;
    constexpr int NB = MODE == FFN_GATED ? 2 : 1;
    constexpr int BK = 64 / T::EB;
    __shared__ __attribute__((aligned(16))) char lds[(1 + NB) * GT * GROW];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int m0 = (int)(blockIdx.x / tiles_n) * GT, n0 = (int)(blockIdx.x % tiles_n) * GT;
    const int wm = (wave / 2) * 32, wn = (wave % 2) * 32;
    const int pair = blockIdx.y;
    typename T::Acc acc[NB][2][2] = {};
    for (int seg = 0; seg < (MODE == FFN_SUM2 ? 2 : 1); ++seg) {
        const FfnOperand &a = p.A[MODE == FFN_PAIR ? pair : seg];
        for (int k0 = 0; k0 < p.K; k0 += BK) {
            __syncthreads();
            gen_stage<TYPE>(a, p.M, p.K, m0, k0, lds, tid);
#pragma unroll
            for (int b = 0; b < NB; ++b)
                gen_stage<TYPE>(p.B[MODE == FFN_GATED ? b : seg], p.N, p.K, n0, k0, lds + (1 + b) * GT * GROW, tid);
            __syncthreads();
            int4_t fa[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                fa[i] = *(const int4_t *)(lds + (wm + 16 * i + lane % 16) * GROW + 16 * (lane / 16));
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int4_t fb = *(const int4_t *)(lds + (1 + b) * GT * GROW +
                                                        (wn + 16 * j + lane % 16) * GROW + 16 * (lane / 16));
#pragma unroll
                    for (int i = 0; i < 2; ++i) acc[b][j][i] = T::mfma(fb, fa[i], acc[b][j][i]);
                }
        }
    }
    // lane l holds row m = l % 16 and columns 4 * (l / 16) .. +3 of a tile
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int m = m0 + wm + 16 * i + lane % 16, n = n0 + wn + 16 * j + 4 * (lane / 16);
            float v[NB][4];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[b][e] = (float)acc[b][j][i][e];
                    if constexpr (TYPE == FFN_I8)
                        v[b][e] *= m < p.M && n + e < p.N ? p.sa[m] * p.sb[b][n + e] : 0.0f;
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
                const int q = MODE == FFN_PAIR ? pair : 0;
                ffn_store4(p.C[q], p.ldc[q], p.out_type, p.M, p.N, m, n, v[0]);
            }
        }
}

// ---- aligned copies ----
// Matrix w of p, 16 bytes a thread, from rows that start anywhere.
__device__ __forceinline__ void pack_rows(const FfnPack &p, int w) {
    const int64_t chunks = p.pitch / 16, total = p.rows[w] * chunks, bytes = p.row_bytes[w];
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / chunks, c = (i % chunks) * 16;
        const char *from = (const char *)p.src[w] + r * p.ld_bytes[w] + c;
        int4_t v = {0, 0, 0, 0};
        if (c + 16 <= bytes) {
            __builtin_memcpy(&v, from, 16);
        } else {
            uint32_t t[4] = {0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (c + e < bytes) t[e / 4] |= (uint32_t)(uint8_t)from[e] << (8 * (e % 4));
            v = int4_t{(int)t[0], (int)t[1], (int)t[2], (int)t[3]};
        }
        *(int4_t *)((char *)p.dst[w] + r * p.pitch + c) = v;
    }
}
__global__ __launch_bounds__(256) void k_ffn_pack(const FfnPack p) { pack_rows(p, blockIdx.y); }

// ---- gradient of the gate ----
// dH, G and U read, dG and dU written, eight columns a thread. Each is rounded
// once to the operands' type: they are matrix-core operands next, and their
// rounding errors average out over the sums (against 64 bits the gradients are
// 1.4 times as far off as a single final rounding, one such error from dG or
// dU and one from the result).
//
// fp16 also has too few exponents: dH U act'(G) of finite values passes 65504,
// and what is below 2^-25 is gone before the sum over tokens or channels that
// would make it a number again. So a pass before takes the largest finite
// |dH U| and |dH a(G)|, a(g) = g for g > 0 and min(|g|, 0.28) for the others,
// which bound both gradients (|act(g)| <= a(g) and |act'| < 1.13 for every
// activation), and they are stored times the power of two that puts the bound
// into [2^14, 2^15); the products undo it on their fp32 sums, exactly. Lost is
// what is below 2^-38 of the largest |dH U| or |dH a(G)|. bf16 has fp32's
// exponents and needs none of it. Without the activation the pass is a read of three
// matrices: 3001 x 2049 8.8 us, the backward call 112 to 124 us (130 with the
// exact gradients in their place); 8192 x 14336 from 4096 3.14 to 3.27 ms.
template <int TYPE>
__device__ __forceinline__ void load8(const uint16_t *row, int n, int N, float (&v)[8]) {
    uint32_t w[4];
    if (n + 8 <= N) {
        __builtin_memcpy(w, row + n, 16);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t lo = n + 2 * e < N ? row[n + 2 * e] : 0, hi = n + 2 * e + 1 < N ? row[n + 2 * e + 1] : 0;
            w[e] = lo | hi << 16;
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = ffn_unpack16<TYPE>((w[e / 2] >> (16 * (e % 2))) & 0xffffu);
}

// The largest of a work-group's values, in every thread.
template <int NT>
__device__ __forceinline__ uint32_t block_top(uint32_t top) {
    __shared__ uint32_t part[NT / 64];
#pragma unroll
    for (int d = 32; d; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) top = max(top, part[i]);
    return top;
}
// A magnitude's bits, ordered as integers; infinities and NaN count as 0.
__device__ __forceinline__ uint32_t finite_bits(float x) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
    return b < 0x7f800000u ? b : 0;
}

// One work-group of 16 waves a CU, so that few results are left for the next
// kernel to read; a wave takes 512 columns of a row at a time.
constexpr int kGateTopThreads = 1024, kGateTopCols = 512;
__global__ __launch_bounds__(kGateTopThreads) void k_ffn_gate_top(int M, int N, const uint16_t *dH, int64_t lddh,
                                                                  const uint16_t *G, int64_t ldg, const uint16_t *U,
                                                                  int64_t ldu, FfnGateScale *scale) {
    const int pieces = (N - 1) / kGateTopCols + 1;  // of a row
    const int waves = (int)gridDim.x * (kGateTopThreads / 64);
    const int wave = (int)blockIdx.x * (kGateTopThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int rows = waves / pieces, rest = waves % pieces;
    uint32_t by_u = 0, by_g = 0;
    int piece = wave % pieces;
    for (int64_t m = wave / pieces; m < M;) {
        const int64_t n = (int64_t)piece * kGateTopCols + 8 * (threadIdx.x % 64);
        if (n < N) {
            float d[8], g[8], u[8];  // zeros past N
            load8<FFN_F16>(dH + m * lddh, (int)n, N, d);
            load8<FFN_F16>(G + m * ldg, (int)n, N, g);
            load8<FFN_F16>(U + m * ldu, (int)n, N, u);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                by_u = max(by_u, finite_bits(d[e] * u[e]));
                by_g = max(by_g, finite_bits(d[e] * fmaxf(g[e], fminf(-g[e], 0.28f))));
            }
        }
        m += rows;
        piece += rest;
        if (piece >= pieces) {
            piece -= pieces;
            ++m;
        }
    }
    // a finite product of two fp16 numbers is far from fp32's end
    const float bound = fmaxf(1.25f * __builtin_bit_cast(float, by_u), __builtin_bit_cast(float, by_g));
    const uint32_t top = block_top<kGateTopThreads>(__builtin_bit_cast(uint32_t, bound));
    if (threadIdx.x == 0) scale->top[blockIdx.x] = top;
}

template <int TYPE, int ACT>
__global__ __launch_bounds__(256) void k_ffn_gate_grad(int M, int N, const uint16_t *dH, int64_t lddh,
                                                       const uint16_t *G, int64_t ldg, const uint16_t *U, int64_t ldu,
                                                       uint16_t *dG, uint16_t *dU, int64_t pitch, int chunks,
                                                       FfnGateScale *scale, int tops, const FfnPack copies) {
    if (blockIdx.y) {
        pack_rows(copies, blockIdx.y - 1);
        return;
    }
    float times = 1.0f;
    if constexpr (TYPE == FFN_F16) {
        static_assert(FfnGateScale::kTops <= 256, "a bound a thread");
        const uint32_t top = block_top<256>((int)threadIdx.x < tops ? scale->top[threadIdx.x] : 0);
        // 2^14 over the bound's power of two (a product of two fp16 numbers is 2^-48 at least)
        const int exponent = top ? (int)(top >> 23) - 127 : 14;
        times = __builtin_bit_cast(float, (uint32_t)(127 + 14 - exponent) << 23);
        if (blockIdx.x == 0 && threadIdx.x == 0)
            scale->undo = __builtin_bit_cast(float, (uint32_t)(127 - 14 + exponent) << 23);
    }
    const int64_t total = (int64_t)M * chunks;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int m = (int)(i / chunks), n = (int)(i % chunks) * 8;
        float d[8], g[8], u[8];
        load8<TYPE>(dH + (int64_t)m * lddh, n, N, d);
        load8<TYPE>(G + (int64_t)m * ldg, n, N, g);
        load8<TYPE>(U + (int64_t)m * ldu, n, N, u);
        uint32_t wg[4], wu[4];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float slope;
            const float value = ffn_act_grad<ACT>(g[e], &slope);
            // columns past N stay zero whatever the activation makes of 0
            const bool in = n + e < N;
            const uint32_t bg = in ? ffn_pack16<TYPE>(d[e] * u[e] * slope * times) : 0;
            const uint32_t bu = in ? ffn_pack16<TYPE>(d[e] * value * times) : 0;
            wg[e / 2] = e % 2 ? wg[e / 2] | bg << 16 : bg;
            wu[e / 2] = e % 2 ? wu[e / 2] | bu << 16 : bu;
        }
        *(int4_t *)(dG + (int64_t)m * pitch + n) = int4_t{(int)wg[0], (int)wg[1], (int)wg[2], (int)wg[3]};
        *(int4_t *)(dU + (int64_t)m * pitch + n) = int4_t{(int)wu[0], (int)wu[1], (int)wu[2], (int)wu[3]};
    }
}

// ---- token quantiser ----
// round-half-even(x / s) for |x| <= 127.5 s. The fp32 quotient is itself
// rounded, which can carry a value just beside a border onto it; the sign of
// the remainder x - q s (one rounding in the fused form, so its order
// against s/2 is that of the exact remainder) says so and moves the code back.
__device__ __forceinline__ int quant_code(float x, float s) {
    float q = rintf(x / s);
    const float r = __builtin_fmaf(-q, s, x), half = 0.5f * s;
    if (r > half) q += 1.0f;
    if (r < -half) q -= 1.0f;
    return (int)fminf(fmaxf(q, -127.0f), 127.0f);
}

// Sixteen elements of a row from k0 on, zeros past K. VEC: every row starts on
// a 16-byte boundary and K is a multiple of 16, so they are all there.
template <int DTYPE, bool VEC>
__device__ __forceinline__ void quant_load16(const char *row, int64_t k0, int64_t K, uint32_t (&w)[DTYPE == TLG_F32 ? 16 : 8]) {
    constexpr int EB = DTYPE == TLG_F32 ? 4 : 2;
    if (VEC || k0 + 16 <= K) {
        __builtin_memcpy(w, row + k0 * EB, 16 * EB);
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const bool in = k0 + e < K;
            if constexpr (EB == 4) {
                w[e] = in ? ((const uint32_t *)row)[k0 + e] : 0;
            } else {
                const uint32_t v = in ? ((const uint16_t *)row)[k0 + e] : 0;
                w[e / 2] = e % 2 ? w[e / 2] | v << 16 : v;
            }
        }
    }
}
template <int DTYPE>
__device__ __forceinline__ float quant_value(const uint32_t *w, int e) {
    if constexpr (DTYPE == TLG_F32)
        return __builtin_bit_cast(float, w[e]);
    else
        return ffn_unpack16<DTYPE == TLG_BF16 ? FFN_BF16 : FFN_F16>((w[e / 2] >> (16 * (e % 2))) & 0xffffu);
}
// The magnitude's bits: ordered as integers, infinities and NaN on top.
template <int DTYPE>
__device__ __forceinline__ uint32_t quant_top(const uint32_t *w, uint32_t top) {
    if constexpr (DTYPE == TLG_F32) {
#pragma unroll
        for (int e = 0; e < 16; ++e) top = max(top, w[e] & 0x7fffffffu);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
    }
    return top;
}

// One work-group of NT threads a token. HELD sixteens of the row stay in each
// thread's registers between the search for the largest magnitude and the
// codes, so a row of up to 16 * NT * HELD elements is read once; what is
// longer is read again (from L2). A code comes from a product with 1 / s,
// whose error stays below 2^-14 for codes up to 127: only a product that
// close to a border between two codes needs the quotient itself.
template <int DTYPE, int NT, int HELD, bool VEC>
__global__ __launch_bounds__(NT) void k_quantize_i8(int64_t K, const char *X, int64_t ldx, int8_t *Q, int64_t ldq,
                                                    float *S) {
    constexpr int EB = DTYPE == TLG_F32 ? 4 : 2, W = 4 * EB;
    const int64_t m = blockIdx.x;
    const char *row = X + m * ldx * EB;
    int8_t *codes = Q + m * ldq;
    __shared__ uint32_t part[NT / 64];
    uint32_t w[HELD][W], top = 0;
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
        const int64_t k0 = ((int64_t)h * NT + threadIdx.x) * 16;
        if (k0 < K) quant_load16<DTYPE, VEC>(row, k0, K, w[h]);
    }
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
        const int64_t k0 = ((int64_t)h * NT + threadIdx.x) * 16;
        if (k0 < K) top = quant_top<DTYPE>(w[h], top);
    }
    for (int64_t k0 = ((int64_t)HELD * NT + threadIdx.x) * 16; k0 < K; k0 += NT * 16) {
        uint32_t v[W];
        quant_load16<DTYPE, VEC>(row, k0, K, v);
        top = quant_top<DTYPE>(v, top);
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    if (NT > 64) {
        if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NT / 64; ++i) top = max(top, part[i]);
    }
    const float largest = DTYPE == TLG_F32 ? __builtin_bit_cast(float, top)
                                           : ffn_unpack16<DTYPE == TLG_BF16 ? FFN_BF16 : FFN_F16>(top);
    const bool finite = largest < __builtin_inff();
    const float s = finite ? largest / 127.0f : __builtin_nanf("");
    if (threadIdx.x == 0) S[m] = s;
    const bool zero = !finite || s == 0.0f;
    const float inverse = zero ? 0.0f : 1.0f / s;
    auto emit = [&](const uint32_t *v, int64_t k0) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float x = quant_value<DTYPE>(v, e);
            // x / s up to two roundings and that of 1 / s: a subnormal s makes 1 / s
            // infinite, which the comparison catches too
            float q = x * inverse;
            const float r = rintf(q);
            const int c = !zero && !(fabsf(fabsf(q - r) - 0.5f) > 6.103515625e-05f && fabsf(q) < 256.0f)
                              ? quant_code(x, s)
                              : (int)fminf(fmaxf(zero ? 0.0f : r, -127.0f), 127.0f);
            o[e / 4] = e % 4 ? o[e / 4] | (uint32_t)(c & 255) << (8 * (e % 4)) : (uint32_t)(c & 255);
        }
        if (VEC || k0 + 16 <= K) {
            __builtin_memcpy(codes + k0, o, 16);
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (k0 + e < K) codes[k0 + e] = (int8_t)(o[e / 4] >> (8 * (e % 4)));
        }
    };
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
        const int64_t k0 = ((int64_t)h * NT + threadIdx.x) * 16;
        if (k0 < K) emit(w[h], k0);
    }
    for (int64_t k0 = ((int64_t)HELD * NT + threadIdx.x) * 16; k0 < K; k0 += NT * 16) {
        uint32_t v[W];
        quant_load16<DTYPE, VEC>(row, k0, K, v);
        emit(v, k0);
    }
}

__global__ __launch_bounds__(256) void k_ffn_zero(uint16_t *p, int64_t rows, int64_t cols, int64_t ld) {
    const int64_t total = rows * cols;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256)
        p[i / cols * ld + i % cols] = 0;
}

unsigned grid_for(int64_t items) {
    const int64_t g = (items + 255) / 256;
    return (unsigned)(g > 65536 ? 65536 : g);
}

template <int TYPE, int MODE>
hipError_t launch_general_t(const FfnProduct &p, hipStream_t stream) {
    const int64_t tm = ((int64_t)p.M + GT - 1) / GT, tn = ((int64_t)p.N + GT - 1) / GT;
    if (tm * tn > kMaxThreads / 256) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_ffn_general<TYPE, MODE>), dim3((unsigned)(tm * tn), MODE == FFN_PAIR ? 2 : 1), dim3(256), 0,
                       stream, p, (int)tn);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ffn_general(const FfnProduct &p, hipStream_t stream) {
    if (p.M <= 0 || p.N <= 0) return hipErrorInvalidValue;
    switch (p.type * 4 + p.mode) {
        case FFN_F16 * 4 + FFN_GATED: return launch_general_t<FFN_F16, FFN_GATED>(p, stream);
        case FFN_F16 * 4 + FFN_SUM2: return launch_general_t<FFN_F16, FFN_SUM2>(p, stream);
        case FFN_F16 * 4 + FFN_PAIR: return launch_general_t<FFN_F16, FFN_PAIR>(p, stream);
        case FFN_BF16 * 4 + FFN_GATED: return launch_general_t<FFN_BF16, FFN_GATED>(p, stream);
        case FFN_BF16 * 4 + FFN_SUM2: return launch_general_t<FFN_BF16, FFN_SUM2>(p, stream);
        case FFN_BF16 * 4 + FFN_PAIR: return launch_general_t<FFN_BF16, FFN_PAIR>(p, stream);
        case FFN_I8 * 4 + FFN_GATED: return launch_general_t<FFN_I8, FFN_GATED>(p, stream);
        case FFN_I8 * 4 + FFN_LINEAR: return launch_general_t<FFN_I8, FFN_LINEAR>(p, stream);
        default: return hipErrorInvalidValue;
    }
}

template <int TYPE, int ACT>
static hipError_t launch_gate_grad_t(int M, int N, const void *dH, int64_t lddh, const void *G, int64_t ldg,
                                     const void *U, int64_t ldu, void *dG, void *dU, int64_t pitch,
                                     FfnGateScale *scale, const FfnPack &copies, hipStream_t stream) {
    const int chunks = (int)(pitch / 8);
    int64_t most = (int64_t)M * chunks;
    int tops = 0;
    if constexpr (TYPE == FFN_F16) {
        const int64_t pieces = (int64_t)M * ((N - 1) / kGateTopCols + 1);
        const int64_t groups = (pieces - 1) / (kGateTopThreads / 64) + 1;
        tops = groups < FfnGateScale::kTops ? (int)groups : FfnGateScale::kTops;
        hipLaunchKernelGGL(k_ffn_gate_top, dim3((unsigned)tops), dim3(kGateTopThreads), 0, stream, M, N,
                           (const uint16_t *)dH, lddh, (const uint16_t *)G, ldg, (const uint16_t *)U, ldu, scale);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    for (int i = 0; i < copies.count; ++i)
        most = copies.rows[i] * (copies.pitch / 16) > most ? copies.rows[i] * (copies.pitch / 16) : most;
    hipLaunchKernelGGL((k_ffn_gate_grad<TYPE, ACT>), dim3(grid_for(most), 1 + (unsigned)copies.count), dim3(256), 0,
                       stream, M, N, (const uint16_t *)dH, lddh, (const uint16_t *)G, ldg, (const uint16_t *)U, ldu,
                       (uint16_t *)dG, (uint16_t *)dU, pitch, chunks, scale, tops, copies);
    return hipGetLastError();
}

hipError_t launch_ffn_gate_grad(int type, int act, int M, int N, const void *dH, int64_t lddh, const void *G,
                                int64_t ldg, const void *U, int64_t ldu, void *dG, void *dU, int64_t pitch,
                                FfnGateScale *scale, const FfnPack &copies, hipStream_t stream) {
#define TLG_GATE_GRAD(TYPE, ACT) \
    case TYPE * 8 + ACT:           \
        return launch_gate_grad_t<TYPE, ACT>(M, N, dH, lddh, G, ldg, U, ldu, dG, dU, pitch, scale, copies, stream)
    switch (type * 8 + act) {
        TLG_GATE_GRAD(FFN_F16, TLG_ACT_SILU);
        TLG_GATE_GRAD(FFN_F16, TLG_ACT_GELU);
        TLG_GATE_GRAD(FFN_F16, TLG_ACT_GELU_TANH);
        TLG_GATE_GRAD(FFN_F16, TLG_ACT_RELU);
        TLG_GATE_GRAD(FFN_BF16, TLG_ACT_SILU);
        TLG_GATE_GRAD(FFN_BF16, TLG_ACT_GELU);
        TLG_GATE_GRAD(FFN_BF16, TLG_ACT_GELU_TANH);
        TLG_GATE_GRAD(FFN_BF16, TLG_ACT_RELU);
        default: return hipErrorInvalidValue;
    }
#undef TLG_GATE_GRAD
}

template <int DTYPE, int NT, int HELD>
static hipError_t launch_quantize_t(int64_t M, int64_t K, const void *X, int64_t ldx, int8_t *Q, int64_t ldq, float *S,
                                    hipStream_t stream) {
    constexpr int EB = DTYPE == TLG_F32 ? 4 : 2;
    const bool vec = K % 16 == 0 && (uintptr_t)X % 16 == 0 && ldx * EB % 16 == 0 && (uintptr_t)Q % 16 == 0 &&
                     ldq % 16 == 0;
    // a launch's threads must stay below 2^32: the tokens of a longer call in several
    constexpr int64_t most = kMaxThreads / NT;
    hipError_t e = hipSuccess;
    for (int64_t m = 0; m < M && e == hipSuccess; m += most) {
        const char *x = (const char *)X + m * ldx * EB;
        const dim3 grid((unsigned)(M - m < most ? M - m : most));
        if (vec)
            hipLaunchKernelGGL((k_quantize_i8<DTYPE, NT, HELD, true>), grid, dim3(NT), 0, stream, K, x, ldx,
                               Q + m * ldq, ldq, S + m);
        else
            hipLaunchKernelGGL((k_quantize_i8<DTYPE, NT, HELD, false>), grid, dim3(NT), 0, stream, K, x, ldx,
                               Q + m * ldq, ldq, S + m);
        e = hipGetLastError();
    }
    return e;
}

template <int DTYPE>
static hipError_t launch_quantize_d(int64_t M, int64_t K, const void *X, int64_t ldx, int8_t *Q, int64_t ldq, float *S,
                                    hipStream_t stream) {
    // threads for one sixteen of the row each while rows are short, then four
    if (K <= 1024) return launch_quantize_t<DTYPE, 64, 1>(M, K, X, ldx, Q, ldq, S, stream);
    if (K <= 4096) return launch_quantize_t<DTYPE, 256, 1>(M, K, X, ldx, Q, ldq, S, stream);
    return launch_quantize_t<DTYPE, 256, 4>(M, K, X, ldx, Q, ldq, S, stream);
}

hipError_t launch_quantize_i8(int dtype, int64_t M, int64_t K, const void *X, int64_t ldx, int8_t *Q, int64_t ldq,
                              float *S, hipStream_t stream) {
    if (M <= 0 || M > 0x7fffffff) return hipErrorInvalidValue;
    switch (dtype) {
        case TLG_F16: return launch_quantize_d<TLG_F16>(M, K, X, ldx, Q, ldq, S, stream);
        case TLG_BF16: return launch_quantize_d<TLG_BF16>(M, K, X, ldx, Q, ldq, S, stream);
        case TLG_F32: return launch_quantize_d<TLG_F32>(M, K, X, ldx, Q, ldq, S, stream);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_ffn_pack(const FfnPack &p, hipStream_t stream) {
    int64_t most = 0;
    for (int i = 0; i < p.count; ++i) most = p.rows[i] > most ? p.rows[i] : most;
    if (!most || !p.pitch) return hipSuccess;  // rows of no element
    hipLaunchKernelGGL(k_ffn_pack, dim3(grid_for(most * (p.pitch / 16)), (unsigned)p.count), dim3(256), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_ffn_zero(void *p, int64_t rows, int64_t cols, int64_t ld, hipStream_t stream) {
    if (rows <= 0 || cols <= 0) return hipSuccess;
    hipLaunchKernelGGL(k_ffn_zero, dim3(grid_for(rows * cols)), dim3(256), 0, stream, (uint16_t *)p, rows, cols, ld);
    return hipGetLastError();
}

}  // namespace tlg
