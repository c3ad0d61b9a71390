// Device-side building blocks of the feed-forward kernels: operand types, the
// gating activations and their derivatives, stores of results.
#ifndef TLG_FFN_OPS_H
#define TLG_FFN_OPS_H

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ffn.h"
#include "gfx950_ops.h"

namespace tlg {

typedef __bf16 bf8_t __attribute__((ext_vector_type(8)));

// Operand types: the bytes of an element, and the 16 x 16 matrix product of
// one 64-byte row piece. A lane's fragment is 16 bytes of one row (8 elements
// of 16 bits, 16 of 8), lane l holding bytes 16*(l/16) .. +15 of row l % 16.
template <int TYPE>
struct FfnT;
template <>
struct FfnT<FFN_F16> {
    static constexpr int EB = 2;
    typedef float4_t Acc;
    typedef _Float16 Elem;
    static __device__ __forceinline__ Acc mfma(int4_t x, int4_t y, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, x), __builtin_bit_cast(half8_t, y),
                                                      c, 0, 0, 0);
    }
};
template <>
struct FfnT<FFN_BF16> {
    static constexpr int EB = 2;
    typedef float4_t Acc;
    typedef __bf16 Elem;
    static __device__ __forceinline__ Acc mfma(int4_t x, int4_t y, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8_t, x), __builtin_bit_cast(bf8_t, y), c,
                                                       0, 0, 0);
    }
};
template <>
struct FfnT<FFN_I8> {
    static constexpr int EB = 1;
    typedef int4_t Acc;
    typedef int8_t Elem;
    static __device__ __forceinline__ Acc mfma(int4_t x, int4_t y, Acc c) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(x, y, c, 0, 0, 0);
    }
};

// fp32 to a 16-bit result, rounded to nearest even; the bits of it.
template <int TYPE>
__device__ __forceinline__ uint32_t ffn_pack16(float x) {
    if constexpr (TYPE == FFN_BF16)
        return __builtin_bit_cast(uint16_t, (__bf16)x);
    else
        return __builtin_bit_cast(uint16_t, (_Float16)x);
}
// Two of them, x in the low half.
typedef float float2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));
template <int TYPE>
__device__ __forceinline__ int ffn_pack32(float x, float y) {
    if constexpr (TYPE == FFN_BF16)
        return __builtin_bit_cast(int, __builtin_convertvector(float2_t{x, y}, bf2_t));
    else
        return __builtin_bit_cast(int, half2_t{(_Float16)x, (_Float16)y});
}
template <int TYPE>
__device__ __forceinline__ float ffn_unpack16(uint32_t bits) {
    if constexpr (TYPE == FFN_BF16)
        return __builtin_bit_cast(float, bits << 16);
    else
        return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}

// 1 / (1 + e^-x) from the hardware's 2^x and reciprocal (one unit in the last
// place each): far below the 16-bit rounding of every result it goes into.
__device__ __forceinline__ float ffn_sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * x));
}
constexpr float kGeluC = 1.5957691216057308f;   // 2 sqrt(2 / pi): tanh(z) = 2 sigmoid(2z) - 1
constexpr float kGeluA = 0.044715f;

// Phi(g), the normal distribution function, and *gauss = e^(-g^2/2). With z =
// |g| / sqrt 2 and t = 1 / (1 + z/2), erfc(z) = t e^(-z^2) R(t), where R is
// smooth on [0, 1]; the polynomial is a least-squares fit of R at Chebyshev
// points, weighted to even out its relative error (with these coefficients in
// fp32 1.3e-7 at most up to z = 31, past which e^(-z^2) is zero). So Phi keeps
// its relative precision for negative g, from one exponential and one reciprocal.
__device__ __forceinline__ float ffn_phi(float g, float *gauss) {
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.35355339059327376f * fabsf(g));
    float r = -0.012611449f;
    r = __builtin_fmaf(r, t, 0.0033185645f);
    r = __builtin_fmaf(r, t, 0.1530851f);
    r = __builtin_fmaf(r, t, -0.33314738f);
    r = __builtin_fmaf(r, t, 0.16829163f);
    r = __builtin_fmaf(r, t, 0.022282181f);
    r = __builtin_fmaf(r, t, 0.1892118f);
    r = __builtin_fmaf(r, t, 0.24528679f);
    r = __builtin_fmaf(r, t, 0.2821902f);
    r = __builtin_fmaf(r, t, 0.28209248f);
    *gauss = __builtin_amdgcn_exp2f(-0.72134752044448170f * g * g);
    const float tail = 0.5f * t * *gauss * r;
    return g < 0.0f ? tail : 1.0f - tail;
}

// act(g); relu maps everything not above 0, NaN included, to +0, as the dense
// kernels' does.
template <int ACT>
__device__ __forceinline__ float ffn_act(float g) {
    if constexpr (ACT == TLG_ACT_SILU) {
        return g * ffn_sigmoid(g);
    } else if constexpr (ACT == TLG_ACT_GELU) {
        float gauss;
        return g * ffn_phi(g, &gauss);
    } else if constexpr (ACT == TLG_ACT_GELU_TANH) {
        return g * ffn_sigmoid(kGeluC * (g + kGeluA * g * g * g));
    } else {
        return g > 0.0f ? g : 0.0f;
    }
}
// act(g) * u of N values side by side: a lone wave on its SIMD waits out every
// dependent instruction, so each step is taken for all of them before the next
// (one value after the other took 9 us for a 256 x 256 tile, this 4).
template <int ACT, int N>
__device__ __forceinline__ void ffn_gate(const float (&g)[N], const float (&u)[N], float (&h)[N]) {
    if constexpr (ACT == TLG_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) h[i] = ffn_act<ACT>(g[i]) * u[i];
        return;
    }
    float t[N];
    if constexpr (ACT == TLG_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) t[i] = ffn_act<ACT>(g[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            t[i] = ACT == TLG_ACT_SILU
                       ? -1.4426950408889634f * g[i]
                       : g[i] * __builtin_fmaf(-1.4426950408889634f * kGeluC * kGeluA, g[i] * g[i],
                                               -1.4426950408889634f * kGeluC);
#pragma unroll
        for (int i = 0; i < N; ++i) t[i] = __builtin_amdgcn_exp2f(t[i]);
#pragma unroll
        for (int i = 0; i < N; ++i) t[i] = 1.0f + t[i];
#pragma unroll
        for (int i = 0; i < N; ++i) t[i] = __builtin_amdgcn_rcpf(t[i]);
#pragma unroll
        for (int i = 0; i < N; ++i) t[i] = g[i] * t[i];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) h[i] = t[i] * u[i];
}
// act(g) and act'(g).
template <int ACT>
__device__ __forceinline__ float ffn_act_grad(float g, float *slope) {
    if constexpr (ACT == TLG_ACT_SILU) {
        const float p = ffn_sigmoid(g), v = g * p;
        *slope = p + v * (1.0f - p);
        return v;
    } else if constexpr (ACT == TLG_ACT_GELU) {
        float gauss;
        const float cdf = ffn_phi(g, &gauss);
        *slope = cdf + g * 0.3989422804014327f * gauss;  // phi(g) = e^(-g^2/2) / sqrt(2 pi)
        return g * cdf;
    } else if constexpr (ACT == TLG_ACT_GELU_TANH) {
        const float p = ffn_sigmoid(kGeluC * (g + kGeluA * g * g * g)), v = g * p;
        // (past the range of g^2, v (1 - p) is zero: no infinity may meet it)
        *slope = p + v * (1.0f - p) * kGeluC * (1.0f + 3.0f * kGeluA * fminf(g * g, 1e30f));
        return v;
    } else {
        *slope = g > 0.0f ? 1.0f : 0.0f;
        return g > 0.0f ? g : 0.0f;
    }
}

// f(std::integral_constant-like value) for the call's activation, so that the
// choice is made once and not for every element.
template <int V>
struct FfnConst {
    static constexpr int value = V;
};
template <class F>
__device__ __forceinline__ void ffn_with_out16(int out_type, F f) {
    if (out_type == TLG_BF16)
        f(FfnConst<FFN_BF16>());
    else
        f(FfnConst<FFN_F16>());
}
template <class F>
__device__ __forceinline__ void ffn_with_act(int act, F f) {
    switch (act) {
        case TLG_ACT_SILU: f(FfnConst<TLG_ACT_SILU>()); break;
        case TLG_ACT_GELU: f(FfnConst<TLG_ACT_GELU>()); break;
        case TLG_ACT_GELU_TANH: f(FfnConst<TLG_ACT_GELU_TANH>()); break;
        default: f(FfnConst<TLG_ACT_RELU>()); break;
    }
}

// Up to four results of row m, columns n .. n+3 of an M x N window: as one
// store where the place allows it, by element elsewhere.
__device__ __forceinline__ void ffn_store4(void *C, int64_t ldc, int out_type, int M, int N, int m, int n,
                                           const float (&v)[4]) {
    if (m >= M) return;
    const int64_t at = (int64_t)m * ldc + n;
    if (out_type == TLG_F32) {
        float *c = (float *)C + at;
        if (n + 4 <= N && (uintptr_t)c % 16 == 0) {
            *(float4_t *)c = float4_t{v[0], v[1], v[2], v[3]};
            return;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n + e < N) c[e] = v[e];
        return;
    }
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = out_type == TLG_BF16 ? ffn_pack16<FFN_BF16>(v[e]) : ffn_pack16<FFN_F16>(v[e]);
    uint16_t *c = (uint16_t *)C + at;
    if (n + 4 <= N && (uintptr_t)c % 8 == 0) {
        *(int2_t *)c = int2_t{(int)(w[0] | w[1] << 16), (int)(w[2] | w[3] << 16)};
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (n + e < N) c[e] = (uint16_t)w[e];
}

}  // namespace tlg

#endif
