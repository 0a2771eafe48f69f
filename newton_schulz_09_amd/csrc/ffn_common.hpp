// Device helpers of the feed-forward kernels: activations, packing, the matrix
// instruction.
#pragma once

#include "attn_common.hpp"
#include "layer_common.hpp"

namespace muon {
namespace ffn {

using attn::u32x2;
using attn::u32x4;

// D[4 (l / 16) + i][l % 16] += sum_k A B for lane l, whose 8 values of A are row
// l % 16 (of B: column), k = 8 (l / 16) .. + 7.  Sustained on random values the
// 16 x 16 x 32 form reaches 1980 TFLOP/s on this card, the 32 x 32 x 16 form, whose
// sums are read and written twice as often, 1745.
__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

constexpr float kLog2E = 1.4426950408889634f;
__device__ __forceinline__ float sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2E * x));
}
// The normal distribution's function Phi(g), from e = exp(-g^2 / 2): Phi(-|g|) = e q(|g|), where q = erfcx(|g| / sqrt 2) / 2
// is smooth and falls as 1 / |g|; here a polynomial in t = 1 / (1 + 0.3 |g|) without
// constant term, fitted for the least relative error over |g| <= 13.5 (1.3e-7; in
// float32 5e-7), past which e vanishes in float32.  (1 + erf) / 2 cancels in the
// negative tail: of a gate of -5 it leaves 4%, of one below -5.6 nothing.
__device__ __forceinline__ float normal_cdf(float g, float e) {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.3f, fabsf(g), 1.0f));
    float q = 0.03593172878026962f;
    q = fmaf(q, t, -0.15827596187591553f);
    q = fmaf(q, t, 0.20820654928684235f);
    q = fmaf(q, t, -0.05539378523826599f);
    q = fmaf(q, t, 0.12946917116641998f);
    q = fmaf(q, t, 0.09963750094175339f);
    q = fmaf(q, t, 0.12079835683107376f);
    q = fmaf(q, t, 0.11962638795375824f);
    const float tail = q * t * e;
    return g < 0.0f ? tail : 1.0f - tail;
}
// act(g), and its derivative.  The hardware's exponential and reciprocal are
// good to an ulp, and no branch cancels where its value is small, so the steps
// of float32 stay far below the bfloat16 that the results are rounded to.
template <int ACT>
__device__ __forceinline__ void activate(float g, float& a, float& da) {
    if constexpr (ACT == ACT_SILU) {
        const float s = sigmoid(g);
        a = g * s;
        da = fmaf(a, 1.0f - s, s);
    } else if constexpr (ACT == ACT_GELU) {
        const float e = __builtin_amdgcn_exp2f(-0.5f * kLog2E * g * g), c = normal_cdf(g, e);
        a = g * c;
        da = fmaf(g * 0.3989422804014327f, e, c);
    } else if constexpr (ACT == ACT_GELU_TANH) {
        // (1 + tanh v) / 2 = sigmoid(2 v)
        const float s = sigmoid(1.5957691216057308f * g * fmaf(0.044715f * g, g, 1.0f));
        a = g * s;
        // (the slope of v is infinite from |g| = 5e19 on, where 1 - s or a is zero)
        da = fmaf(a * (1.0f - s), 1.5957691216057308f * fminf(fmaf(0.134145f * g, g, 1.0f), 1e38f), s);
    } else {
        a = g < 0.0f ? 0.0f : g;
        da = g > 0.0f ? 1.0f : 0.0f;
    }
}
// f(integral_constant<int, act>): one branch around a lane's 8 values.
template <typename F>
__device__ __forceinline__ void by_act(int act, F&& f) {
    if (act == ACT_SILU) f(std::integral_constant<int, ACT_SILU>{});
    else if (act == ACT_GELU) f(std::integral_constant<int, ACT_GELU>{});
    else if (act == ACT_GELU_TANH) f(std::integral_constant<int, ACT_GELU_TANH>{});
    else f(std::integral_constant<int, ACT_RELU>{});
}

__device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
    return u32x4{f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]), f32x2_to_bf16x2(v[4], v[5]),
                 f32x2_to_bf16x2(v[6], v[7])};
}
__device__ __forceinline__ void spread8(u32x4 u, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
}  // namespace ffn
}  // namespace muon
