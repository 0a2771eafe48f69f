// RMS norm of every query and key head and the rotation by position, one pass:
//     r = 1 / sqrt(mean x^2 + eps), y = x r w, (a, b) = halves of y,
//     z = (a cos - b sin, b cos + a sin)
// and its gradient
//     t = (a cos + b sin, b cos - a sin) of dz, dw = sum t x r, g = t w,
//     dx = r (g - x r mean(g x r)).
//
// Bound by memory: every head is read once and written once.  A head is held
// by 2^k lanes, each with one 16-byte piece of either half, so the rotation
// needs no exchange between lanes and the norm k of them; a wave takes one
// token at a time, whose angles its lanes load once for all heads.
#include "../../include/muon.h"
#include "lm_common.hpp"

namespace muon {

namespace {

template <typename T, int V>
__device__ __forceinline__ void load_v(const T* p, float (&x)[V]) {
    if constexpr (V == 1) {
        if constexpr (sizeof(T) == 2) x[0] = bf16_to_f32(p[0]);
        else x[0] = p[0];
    } else if constexpr (sizeof(T) == 2) {
        typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
        static_assert(V == 8, "16 bytes");
        const u32x4 u = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    } else {
        static_assert(V == 4, "16 bytes");
        const f32x4 u = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = u[i];
    }
}

template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, const float (&x)[V]) {
    if constexpr (V == 1) {
        if constexpr (sizeof(T) == 2) p[0] = f32_to_bf16(x[0]);
        else p[0] = x[0];
    } else if constexpr (sizeof(T) == 2) {
        typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
        const u32x4 u = {f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]), f32x2_to_bf16x2(x[4], x[5]),
                         f32x2_to_bf16x2(x[6], x[7])};
        *reinterpret_cast<u32x4*>(p) = u;
    } else {
        *reinterpret_cast<f32x4*>(p) = f32x4{x[0], x[1], x[2], x[3]};
    }
}

// Sum over the aligned group of `lanes` lanes.
__device__ __forceinline__ float group_sum(float x, int lanes) {
    for (int m = 1; m < lanes; m <<= 1) x += __shfl_xor(x, m);
    return x;
}

// NP pieces of V values a lane holds of either half.
template <typename T, int V, int NP, bool BWD>
__global__ __launch_bounds__(256) void k_qk_norm(const QkArgs a, int lanes) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int sub = lane / lanes, l = lane % lanes, per = 64 / lanes;
    const int half = a.d / 2, pieces = half / V;
    const float inv_d = 1.0f / static_cast<float>(a.d);
    const int64_t tokens = static_cast<int64_t>(a.b) * a.s;
    float wv[2][NP][2][V], dw[2][NP][2][V];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int c = (l + p * lanes) * V;
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    wv[k][p][s][i] = a.w[k] && l + p * lanes < pieces ? a.w[k][s * half + c + i] : 1.0f;
                    if constexpr (BWD) dw[k][p][s][i] = 0.0f;
                }
        }
    for (int64_t tok = static_cast<int64_t>(blockIdx.x) * 4 + wave; tok < tokens; tok += static_cast<int64_t>(gridDim.x) * 4) {
        const int bb = static_cast<int>(tok / a.s), ss = static_cast<int>(tok % a.s);
        const int pos = a.positions ? a.positions[tok] : ss;
        const bool known = pos >= 0 && pos < a.limit;  // a position outside the table gives NaN
        float cs[NP][V], sn[NP][V];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int c = (l + p * lanes) * V;
            const float* t = a.table + (static_cast<int64_t>(known ? pos : 0) * half + c) * 2;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                cs[p][i] = sn[p][i] = __builtin_nanf("");
                if (known && l + p * lanes < pieces) {
                    cs[p][i] = t[2 * i];
                    sn[p][i] = t[2 * i + 1];
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const T* xb = static_cast<const T*>(a.x[k]) + bb * a.x_b[k] + ss * a.x_s[k];
            const T* zb = BWD ? static_cast<const T*>(a.dz[k]) + bb * a.z_b[k] + ss * a.z_s[k] : nullptr;
            T* yb = static_cast<T*>(a.y[k]) + tok * a.heads[k] * a.d;
            for (int h = sub; h < a.heads[k]; h += per) {
                float x[NP][2][V], z[NP][2][V], sq = 0.0f;
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    const int c = (l + p * lanes) * V;
                    const bool in = l + p * lanes < pieces;
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
#pragma unroll
                        for (int i = 0; i < V; ++i) x[p][s][i] = z[p][s][i] = 0.0f;
                        if (in) {
                            load_v<T, V>(xb + h * a.x_h[k] + s * half + c, x[p][s]);
                            if constexpr (BWD) load_v<T, V>(zb + h * a.z_h[k] + s * half + c, z[p][s]);
                        }
#pragma unroll
                        for (int i = 0; i < V; ++i) sq = fmaf(x[p][s][i], x[p][s][i], sq);
                    }
                }
                const float r = 1.0f / sqrtf(group_sum(sq, lanes) * inv_d + a.eps);
                if constexpr (!BWD) {
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        const int c = (l + p * lanes) * V;
                        float o[2][V];
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const float u = x[p][0][i] * r * wv[k][p][0][i], v = x[p][1][i] * r * wv[k][p][1][i];
                            o[0][i] = fmaf(u, cs[p][i], -v * sn[p][i]);
                            o[1][i] = fmaf(v, cs[p][i], u * sn[p][i]);
                        }
                        if (l + p * lanes < pieces) {
                            store_v<T, V>(yb + h * a.d + c, o[0]);
                            store_v<T, V>(yb + h * a.d + half + c, o[1]);
                        }
                    }
                } else {
                    float dot = 0.0f;
#pragma unroll
                    for (int p = 0; p < NP; ++p)
#pragma unroll
                        for (int i = 0; i < V; ++i)
                            if (l + p * lanes < pieces) {
                                const float u = fmaf(z[p][0][i], cs[p][i], z[p][1][i] * sn[p][i]);
                                const float v = fmaf(z[p][1][i], cs[p][i], -z[p][0][i] * sn[p][i]);
                                x[p][0][i] *= r;
                                x[p][1][i] *= r;
                                dw[k][p][0][i] = fmaf(u, x[p][0][i], dw[k][p][0][i]);
                                dw[k][p][1][i] = fmaf(v, x[p][1][i], dw[k][p][1][i]);
                                z[p][0][i] = u * wv[k][p][0][i];
                                z[p][1][i] = v * wv[k][p][1][i];
                                dot = fmaf(z[p][0][i], x[p][0][i], dot);
                                dot = fmaf(z[p][1][i], x[p][1][i], dot);
                            }
                    dot = group_sum(dot, lanes) * inv_d;
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        const int c = (l + p * lanes) * V;
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            float o[V];
#pragma unroll
                            for (int i = 0; i < V; ++i) o[i] = r * fmaf(-x[p][s][i], dot, z[p][s][i]);
                            if (l + p * lanes < pieces) store_v<T, V>(yb + h * a.d + s * half + c, o);
                        }
                    }
                }
            }
        }
    }
    if constexpr (BWD) {
        // weight gradients of the workgroup: lanes of one piece, then waves
        if (!a.part) return;
        __shared__ float s_dw[4][2][512];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        float x = dw[k][p][s][i];
                        for (int m = lanes; m < 64; m <<= 1) x += __shfl_xor(x, m);
                        if (sub == 0 && l + p * lanes < pieces) s_dw[wave][k][s * half + (l + p * lanes) * V + i] = x;
                    }
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * a.d; c += 256) {
            const int k = c / a.d, i = c % a.d;
            a.part[static_cast<int64_t>(blockIdx.x) * 2 * a.d + c] =
                (s_dw[0][k][i] + s_dw[1][k][i]) + (s_dw[2][k][i] + s_dw[3][k][i]);
        }
    }
}

// Weight gradients: the workgroups' sums of 64 columns, in their order.
__global__ __launch_bounds__(1024) void k_qk_dw(const QkArgs a) {
    __shared__ float s[16][64];
    const int c = blockIdx.x * 64 + (threadIdx.x & 63), y = threadIdx.x >> 6;
    float x = 0.0f;
    if (c < 2 * a.d)
        for (int i = y; i < a.blocks; i += 16) x += a.part[static_cast<int64_t>(i) * 2 * a.d + c];
    s[y][threadIdx.x & 63] = x;
    __syncthreads();
    if (y == 0 && c < 2 * a.d) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) t += s[i][threadIdx.x & 63];
        float* dw = a.dw[c / a.d];
        if (dw) dw[c % a.d] = t;
    }
}

template <bool BWD>
void run(const QkArgs& a, hipStream_t stream) {
    int lanes = 1;
    if (a.vector) {
        const int v = a.type == MUON_BF16 ? 8 : 4;
        while (lanes * v < a.d / 2) lanes <<= 1;
        if (a.type == MUON_BF16) k_qk_norm<bf16_t, 8, 1, BWD><<<a.blocks, 256, 0, stream>>>(a, lanes);
        else k_qk_norm<float, 4, 1, BWD><<<a.blocks, 256, 0, stream>>>(a, lanes);
    } else {
        // odd sizes or alignment: value by value, up to 4 of either half a lane
        while (lanes < 64 && lanes < a.d / 2) lanes <<= 1;
        if (a.type == MUON_BF16) k_qk_norm<bf16_t, 1, 4, BWD><<<a.blocks, 256, 0, stream>>>(a, lanes);
        else k_qk_norm<float, 1, 4, BWD><<<a.blocks, 256, 0, stream>>>(a, lanes);
    }
}

}  // namespace

hipError_t launch_qk_norm(const QkArgs& a, hipStream_t stream) {
    run<false>(a, stream);
    return hipGetLastError();
}

hipError_t launch_qk_norm_bwd(const QkArgs& a, hipStream_t stream) {
    run<true>(a, stream);
    if (a.part) k_qk_dw<<<(2 * a.d + 63) / 64, 1024, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace muon
