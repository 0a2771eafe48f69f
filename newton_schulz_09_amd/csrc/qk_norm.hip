// RMS norm of every query and key head and the rotation by position, one pass:
//     r = 1 / sqrt(mean x^2 + eps), y = x r w, (a, b) = halves of y,
//     z = (a cos - b sin, b cos + a sin)
// and its gradient
//     t = (a cos + b sin, b cos - a sin) of dz, dw = sum t x r, g = t w,
//     dx = r (g - x r mean(g x r)).
//
// Bound by memory: every head is read once and written once.  A head is held
// by 2^k lanes, each with one 16-byte piece of either half, so the rotation
// needs no exchange between lanes and the norm k of them.  Such a group takes
// the heads of one token in turn (65536 tokens of 12 + 12 bf16 heads of 64: 93 us
// and 139 with gradients, 90 % of the rate of a large copy; a wave per token,
// its groups side by side on the heads: 163 and 265).
#include <type_traits>

#include "../../include/muon.h"
#include "lm_common.hpp"

namespace muon {

namespace {

// V values as they lie in memory: 16 bytes, or one value.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <typename T, int V>
using Piece = std::conditional_t<V == 1, T, u32x4>;

template <typename T, int V>
__device__ __forceinline__ Piece<T, V> load_v(const T* p) {
    static_assert(V == 1 || V * sizeof(T) == 16, "16 bytes");
    return *reinterpret_cast<const Piece<T, V>*>(p);
}
template <typename T, int V>
__device__ __forceinline__ void spread(const Piece<T, V>& u, float (&x)[V]) {
    if constexpr (V == 1) {
        if constexpr (sizeof(T) == 2) x[0] = bf16_to_f32(u);
        else x[0] = u;
    } else if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(u[i]);
    }
}

template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, const float (&x)[V]) {
    if constexpr (V == 1) {
        if constexpr (sizeof(T) == 2) p[0] = f32_to_bf16(x[0]);
        else p[0] = x[0];
    } else if constexpr (sizeof(T) == 2) {
        const u32x4 u = {f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]), f32x2_to_bf16x2(x[4], x[5]),
                         f32x2_to_bf16x2(x[6], x[7])};
        *reinterpret_cast<u32x4*>(p) = u;
    } else {
        *reinterpret_cast<f32x4*>(p) = f32x4{x[0], x[1], x[2], x[3]};
    }
}

// Values at an address that is aligned to 4 bytes only.
template <int N>
__device__ __forceinline__ void load_f(const float* p, float (&x)[N]) {
    typedef f32x4 __attribute__((aligned(4))) f32x4u;
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const f32x4 u = reinterpret_cast<const f32x4u*>(p)[i];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[4 * i + k] = u[k];
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = p[i];
    }
}

// Sum over the aligned group of `lanes` lanes.
__device__ __forceinline__ float group_sum(float x, int lanes) {
    for (int m = 1; m < lanes; m <<= 1) x += __shfl_xor(x, m);
    return x;
}

// NP pieces of V values a lane holds of either half.  A group of `lanes` lanes
// takes one token and a.chunk of its heads, HU of them at a time so that their
// loads are on their way together; blockIdx.y is the run of heads.
template <typename T, int V, int NP, bool BWD>
__global__ __launch_bounds__(256) void k_qk_norm(const QkArgs a, int lanes) {
    constexpr int HU = NP > 1 ? 1 : (BWD ? 2 : 4);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int l = lane % lanes, groups = 256 / lanes;
    const int half = a.d / 2, pieces = half / V;
    const float inv_d = 1.0f / static_cast<float>(a.d);
    const int64_t tokens = static_cast<int64_t>(a.b) * a.s;
    const int k = static_cast<int>(blockIdx.y) < a.runs_q ? 0 : 1;
    const int h0 = (static_cast<int>(blockIdx.y) - (k ? a.runs_q : 0)) * a.chunk;
    const int h1 = h0 + a.chunk < a.heads[k] ? h0 + a.chunk : a.heads[k];
    float wv[NP][2][V], dw[NP][2][V];
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                wv[p][s][i] = 1.0f;
                dw[p][s][i] = 0.0f;
            }
            if (a.w[k] && l + p * lanes < pieces) load_f<V>(a.w[k] + s * half + (l + p * lanes) * V, wv[p][s]);
        }
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * groups; t0 < tokens; t0 += static_cast<int64_t>(gridDim.x) * groups) {
        const int64_t tok = t0 + threadIdx.x / lanes;
        const bool real = tok < tokens;  // (a group past the end takes part in its wave's exchanges)
        int64_t bb = 0;
        int ss = 0;
        if (real) {
            if (tokens <= 0x7fffffff) {
                bb = static_cast<uint32_t>(tok) / static_cast<uint32_t>(a.s);
                ss = static_cast<int>(static_cast<uint32_t>(tok) % static_cast<uint32_t>(a.s));
            } else {
                bb = tok / a.s;
                ss = static_cast<int>(tok % a.s);
            }
        }
        const T* xb = static_cast<const T*>(a.x[k]) + bb * a.x_b[k] + ss * a.x_s[k];
        const T* zb = BWD ? static_cast<const T*>(a.dz[k]) + bb * a.z_b[k] + ss * a.z_s[k] : nullptr;
        T* yb = static_cast<T*>(a.y[k]) + (real ? tok : 0) * a.heads[k] * a.d;
        const int pos = a.positions && real ? a.positions[tok] : ss;
        const bool known = pos >= 0 && pos < a.limit;  // a position outside the table gives NaN
        float cs[NP][V], sn[NP][V];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            float t[2 * V];
#pragma unroll
            for (int i = 0; i < 2 * V; ++i) t[i] = __builtin_nanf("");
            if (known && real && l + p * lanes < pieces)
                load_f<2 * V>(a.table + (static_cast<int64_t>(pos) * half + (l + p * lanes) * V) * 2, t);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                cs[p][i] = t[2 * i];
                sn[p][i] = t[2 * i + 1];
            }
        }
        for (int h = h0; h < h1; h += HU) {
            Piece<T, V> rx[HU][NP][2], rz[HU][NP][2];
#pragma unroll
            for (int u = 0; u < HU; ++u)
#pragma unroll
                for (int p = 0; p < NP; ++p)
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const int c = s * half + (l + p * lanes) * V;
                        rx[u][p][s] = rz[u][p][s] = {};
                        if (real && l + p * lanes < pieces && h + u < h1) {
                            rx[u][p][s] = load_v<T, V>(xb + (h + u) * a.x_h[k] + c);
                            if constexpr (BWD) rz[u][p][s] = load_v<T, V>(zb + (h + u) * a.z_h[k] + c);
                        }
                    }
#pragma unroll
            for (int u = 0; u < HU; ++u) {
                if (h + u >= h1) break;
                float x[NP][2][V], z[NP][2][V], sq = 0.0f;
#pragma unroll
                for (int p = 0; p < NP; ++p)
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        spread<T, V>(rx[u][p][s], x[p][s]);
                        if constexpr (BWD) spread<T, V>(rz[u][p][s], z[p][s]);
#pragma unroll
                        for (int i = 0; i < V; ++i) sq = fmaf(x[p][s][i], x[p][s][i], sq);
                    }
                const float r = 1.0f / sqrtf(group_sum(sq, lanes) * inv_d + a.eps);
                T* y = yb + static_cast<int64_t>(h + u) * a.d;
                if constexpr (!BWD) {
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        const int c = (l + p * lanes) * V;
                        float o[2][V];
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const float e = x[p][0][i] * r * wv[p][0][i], f = x[p][1][i] * r * wv[p][1][i];
                            o[0][i] = fmaf(e, cs[p][i], -f * sn[p][i]);
                            o[1][i] = fmaf(f, cs[p][i], e * sn[p][i]);
                        }
                        if (real && l + p * lanes < pieces) {
                            store_v<T, V>(y + c, o[0]);
                            store_v<T, V>(y + half + c, o[1]);
                        }
                    }
                } else {
                    float dot = 0.0f;
#pragma unroll
                    for (int p = 0; p < NP; ++p)
#pragma unroll
                        for (int i = 0; i < V; ++i)
                            if (real && l + p * lanes < pieces) {
                                const float e = fmaf(z[p][0][i], cs[p][i], z[p][1][i] * sn[p][i]);
                                const float f = fmaf(z[p][1][i], cs[p][i], -z[p][0][i] * sn[p][i]);
                                x[p][0][i] *= r;
                                x[p][1][i] *= r;
                                dw[p][0][i] = fmaf(e, x[p][0][i], dw[p][0][i]);
                                dw[p][1][i] = fmaf(f, x[p][1][i], dw[p][1][i]);
                                z[p][0][i] = e * wv[p][0][i];
                                z[p][1][i] = f * wv[p][1][i];
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
                            if (real && l + p * lanes < pieces) store_v<T, V>(y + s * half + c, o);
                        }
                    }
                }
            }
        }
    }
    if constexpr (BWD) {
        // weight gradients of the workgroup: groups of a wave, then waves
        if (!a.part) return;
        __shared__ float s_dw[4][512];
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float x = dw[p][s][i];
                    for (int m = lanes; m < 64; m <<= 1) x += __shfl_xor(x, m);
                    if (lane < lanes && l + p * lanes < pieces) s_dw[wave][s * half + (l + p * lanes) * V + i] = x;
                }
        __syncthreads();
        float* part = a.part + (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * a.d;
        for (int c = threadIdx.x; c < a.d; c += 256) part[c] = (s_dw[0][c] + s_dw[1][c]) + (s_dw[2][c] + s_dw[3][c]);
    }
}

// Weight gradients: 64 threads per column sum the workgroups' rows, and are
// joined in one order.  Workgroups of 16 columns.
__global__ __launch_bounds__(1024) void k_qk_dw(const QkArgs a, int gx, int runs) {
    __shared__ float s[64][17];
    const int k = blockIdx.y, c = blockIdx.x * 16 + (threadIdx.x & 15), y = threadIdx.x >> 4;
    if (!a.dw[k]) return;
    const int rows = gx * (k ? runs - a.runs_q : a.runs_q);
    const float* part = a.part + (k ? static_cast<int64_t>(a.runs_q) * gx * a.d : 0);
    float x = 0.0f;
    if (c < a.d) {
#pragma unroll 8
        for (int i = y; i < rows; i += 64) x += part[static_cast<int64_t>(i) * a.d + c];
    }
    s[y][threadIdx.x & 15] = x;
    __syncthreads();
    for (int m = 32; m; m >>= 1) {
        if (y < m) s[y][threadIdx.x & 15] += s[y + m][threadIdx.x & 15];
        __syncthreads();
    }
    if (y == 0 && c < a.d) a.dw[k][c] = s[0][threadIdx.x & 15];
}

template <typename T, int V, int NP, bool BWD>
void start(const QkArgs& a, int lanes, hipStream_t stream) {
    const int runs = a.runs_q + (a.heads[1] + a.chunk - 1) / a.chunk;
    if (runs > 0) k_qk_norm<T, V, NP, BWD><<<dim3(a.blocks, runs), 256, 0, stream>>>(a, lanes);
    if (BWD && a.part) k_qk_dw<<<dim3((a.d + 15) / 16, 2), 1024, 0, stream>>>(a, a.blocks, runs);
}

template <bool BWD>
void run(const QkArgs& a, hipStream_t stream) {
    const int lanes = a.lanes;
    if (a.vector) {
        if (a.type == MUON_BF16) start<bf16_t, 8, 1, BWD>(a, lanes, stream);
        else start<float, 4, 1, BWD>(a, lanes, stream);
    } else {
        // odd sizes or alignment: value by value, up to 4 of either half a lane
        if (a.type == MUON_BF16) start<bf16_t, 1, 4, BWD>(a, lanes, stream);
        else start<float, 1, 4, BWD>(a, lanes, stream);
    }
}

}  // namespace

hipError_t launch_qk_norm(const QkArgs& a, hipStream_t stream) {
    run<false>(a, stream);
    return hipGetLastError();
}

hipError_t launch_qk_norm_bwd(const QkArgs& a, hipStream_t stream) {
    run<true>(a, stream);
    return hipGetLastError();
}

}  // namespace muon
