// The norms around a block of a decoder layer, its gate and residual scale, in
// one pass over a token's row:
//     r = 1 / sqrt(mean y^2 + eps), n = y r postw (or y), n dropped out,
//     v = scale x + gate n,  r' = 1 / sqrt(mean v^2 + eps),  z = v r' prew
// and its gradients, from dz and what arrives at v (dv):
//     t = dz prew, e = r' (t - v r' mean(t v r')) + dv,
//     dx = scale e, dscale = sum e x, dgate = sum e n, dn = gate e (dropped out),
//     u = dn postw, dy = r (u - y r mean(u y r)), dpostw = sum dn y r,
//     dprew = sum dz v r'.
//
// Bound by memory: every row is read once and written once and stays in
// registers between.  W waves hold a row, 8 values a piece and 2 pieces a lane,
// so a row of 1024 values needs no exchange but that inside its wave.
// Workgroups walk rows, so weights are loaded and gradients of weights summed
// in registers; a second, small kernel joins the workgroups' sums in one order.
#include <type_traits>

#include "../../include/muon.h"
#include "layer_common.hpp"

namespace muon {

namespace {

// V values as they lie in memory.
template <typename T, int V>
struct Raw {
    static constexpr int N = V * sizeof(T) / 16;
    u32x4_t u[N];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < N; ++i) u[i] = reinterpret_cast<const u32x4_t*>(p)[i];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < N; ++i) u[i] = u32x4_t{0, 0, 0, 0};
    }
    __device__ __forceinline__ float at(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(u[i >> 2][i & 3]);
        else return __uint_as_float(i & 1 ? u[0][i >> 1] & 0xffff0000u : u[0][i >> 1] << 16);
    }
};
template <typename T>
struct Raw<T, 1> {
    T u;
    __device__ __forceinline__ void load(const T* p) { u = *p; }
    __device__ __forceinline__ void zero() { u = 0; }
    __device__ __forceinline__ float at(int) const {
        if constexpr (sizeof(T) == 4) return u;
        else return bf16_to_f32(u);
    }
};
template <typename T, int V>
__device__ __forceinline__ void store_piece(T* p, const float (&x)[V]) {
    if constexpr (V == 1) {
        if constexpr (sizeof(T) == 2) *p = f32_to_bf16(x[0]);
        else *p = x[0];
    } else if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<u32x4_t*>(p) = u32x4_t{f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]),
                                                 f32x2_to_bf16x2(x[4], x[5]), f32x2_to_bf16x2(x[6], x[7])};
    } else {
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
            reinterpret_cast<f32x4*>(p)[i] = f32x4{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
    }
}
// V float32 values aligned to 4 bytes, or ones.
template <int V>
__device__ __forceinline__ void load_weights(const float* p, int64_t at, float (&x)[V], float other) {
    typedef f32x4 __attribute__((aligned(4))) f32x4u;
    if (!p) {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = other;
    } else if constexpr (V == 1) {
        x[0] = p[at];
    } else {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const f32x4 u = reinterpret_cast<const f32x4u*>(p + at)[i];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[4 * i + k] = u[k];
        }
    }
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
// Sum over the wave, in every lane.
__device__ __forceinline__ float wave_sum(float x) {
    x = dpp_add<0xB1>(x);   // lanes 1 0 3 2
    x = dpp_add<0x4E>(x);   // lanes 2 3 0 1
    x = dpp_add<0x141>(x);  // 8 lanes mirrored
    x = dpp_add<0x140>(x);  // 16 lanes mirrored
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

template <int W>
constexpr int threads_of() { return 64 * (W > 4 ? W : 4); }

// Sums of K values over the W waves of each row, in every lane of the row.
template <int W, int K>
struct RowSum {
    static constexpr int ROWS = threads_of<W>() / 64 / W;
    float (*s)[ROWS][W][4];
    int flip = 0;
    __device__ __forceinline__ void operator()(float (&x)[K]) {
#pragma unroll
        for (int k = 0; k < K; ++k) x[k] = wave_sum(x[k]);
        if constexpr (W > 1) {
            // two buffers in turn: a barrier lies between a buffer's reads and its next writes
            const int wave = threadIdx.x >> 6, row = wave / W;
            if ((threadIdx.x & 63) == 0)
#pragma unroll
                for (int k = 0; k < K; ++k) s[flip][row][wave % W][k] = x[k];
            __syncthreads();
#pragma unroll
            for (int k = 0; k < K; ++k) {
                x[k] = 0.0f;
#pragma unroll
                for (int w = 0; w < W; ++w) x[k] += s[flip][row][w][k];
            }
            flip ^= 1;
        }
    }
};

// The factors of dropout of V elements from element `at` on.
template <int V>
__device__ __forceinline__ void drop_factors(const DropState& d, uint64_t seed, uint64_t first, int64_t at, float (&f)[V],
                                             bool (&keep)[V]) {
    const u32x4_t w = philox(seed, first + static_cast<uint64_t>(at >> 3));
#pragma unroll
    for (int i = 0; i < V; ++i) {
        keep[i] = V == 8 ? drop_keeps(w, i, d.threshold) : drop_keeps(w, static_cast<int>(at & 7), d.threshold);
        f[i] = d.factor;
    }
}

template <typename TX, typename TY, int V, int NP, int W>
__global__ __launch_bounds__(threads_of<W>()) void k_resid_norm(const ResidArgs a) {
    constexpr int ROWS = threads_of<W>() / 64 / W;
    __shared__ float s_sum[2][ROWS][W][4];
    RowSum<W, 1> row_sum{s_sum};
    const int l = threadIdx.x % (64 * W), sub = threadIdx.x / (64 * W);
    const float inv = 1.0f / static_cast<float>(a.width);
    uint64_t seed = 0, first = 0;
    if (a.drop.threshold) drop_start(a.drop, seed, first);
    float postw[NP][V], prew[NP][V], scale[NP][V], gate[NP][V];
    bool has[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int c = (p * 64 * W + l) * V;
        has[p] = c < a.width;
        load_weights<V>(has[p] ? a.postw : nullptr, c, postw[p], 1.0f);
        load_weights<V>(has[p] ? a.prew : nullptr, c, prew[p], 1.0f);
        load_weights<V>(has[p] ? a.scale : nullptr, c, scale[p], 1.0f);
        load_weights<V>(has[p] && a.gate_kind == GATE_CHANNEL ? static_cast<const float*>(a.gate) : nullptr, c, gate[p], 1.0f);
    }
    for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * ROWS; row0 < a.rows; row0 += static_cast<int64_t>(gridDim.x) * ROWS) {
        const int64_t row = row0 + sub;
        const bool real = row < a.rows;  // (the others take part in the exchanges)
        Raw<TX, V> rx[NP];
        Raw<TY, V> ry[NP], rg[NP];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int c = (p * 64 * W + l) * V;
            rx[p].zero();
            ry[p].zero();
            rg[p].zero();
            if (real && has[p]) {
                rx[p].load(static_cast<const TX*>(a.x) + row * a.x_s + c);
                if (a.y) ry[p].load(static_cast<const TY*>(a.y) + row * a.y_s + c);
                if (a.gate_kind == GATE_FULL) rg[p].load(static_cast<const TY*>(a.gate) + row * a.g_s + c);
                else if (a.gate_kind == GATE_SEQUENCE)
                    load_weights<V>(static_cast<const float*>(a.gate), row / a.s * a.width + c, gate[p], 1.0f);
            }
        }
        float v[NP][V], sum[1] = {0.0f};
        if (a.y) {
            float r = 1.0f;
            if (a.post) {
#pragma unroll
                for (int p = 0; p < NP; ++p)
#pragma unroll
                    for (int i = 0; i < V; ++i) sum[0] = fmaf(ry[p].at(i), ry[p].at(i), sum[0]);
                row_sum(sum);
                r = 1.0f / sqrtf(fmaf(sum[0], inv, a.eps));
            }
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const int c = (p * 64 * W + l) * V;
                float n[V];
#pragma unroll
                for (int i = 0; i < V; ++i) n[i] = a.post ? ry[p].at(i) * r * postw[p][i] : ry[p].at(i);
                if (a.drop.threshold && has[p]) {
                    float f[V];
                    bool keep[V];
                    drop_factors<V>(a.drop, seed, first, row * a.width + c, f, keep);
#pragma unroll
                    for (int i = 0; i < V; ++i) n[i] = keep[i] ? n[i] * f[i] : 0.0f;
                }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float g = a.gate_kind == GATE_FULL ? rg[p].at(i) : gate[p][i];
                    v[p][i] = fmaf(rx[p].at(i), scale[p][i], g * n[i]);
                }
            }
        } else {
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
                for (int i = 0; i < V; ++i) v[p][i] = rx[p].at(i) * scale[p][i];
        }
        sum[0] = 0.0f;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int c = (p * 64 * W + l) * V;
            if (real && has[p] && a.x_out) store_piece<TX, V>(static_cast<TX*>(a.x_out) + row * a.width + c, v[p]);
#pragma unroll
            for (int i = 0; i < V; ++i) sum[0] = has[p] ? fmaf(v[p][i], v[p][i], sum[0]) : sum[0];
        }
        row_sum(sum);
        const float r = 1.0f / sqrtf(fmaf(sum[0], inv, a.eps));
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int c = (p * 64 * W + l) * V;
            float z[V];
#pragma unroll
            for (int i = 0; i < V; ++i) z[i] = v[p][i] * r * prew[p][i];
            if (real && has[p]) store_piece<TY, V>(static_cast<TY*>(a.z) + row * a.width + c, z);
        }
    }
}

// Sum of every row of the workgroup, column by column: the waves that hold the
// same columns are added in one order.  s: ROWS x width.
template <int V, int NP, int W>
__device__ __forceinline__ void sum_rows(const float (&x)[NP][V], float* s, float* dst, int width) {
    constexpr int ROWS = threads_of<W>() / 64 / W;
    const int l = threadIdx.x % (64 * W), sub = threadIdx.x / (64 * W);
    if constexpr (ROWS == 1) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int c = (p * 64 * W + l) * V;
            if (c < width) {
#pragma unroll
                for (int i = 0; i < V; ++i) dst[c + i] = x[p][i];
            }
        }
    } else {
        __syncthreads();
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int c = (p * 64 * W + l) * V;
            if (c < width) {
#pragma unroll
                for (int i = 0; i < V; ++i) s[sub * width + c + i] = x[p][i];
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < width; c += threads_of<W>()) {
            float t = s[c];
#pragma unroll
            for (int r = 1; r < ROWS; ++r) t += s[r * width + c];
            dst[c] = t;
        }
    }
}

template <typename TX, typename TY, int V, int NP, int W>
__global__ __launch_bounds__(threads_of<W>()) void k_resid_norm_bwd(const ResidArgs a) {
    constexpr int ROWS = threads_of<W>() / 64 / W;
    __shared__ float s_sum[2][ROWS][W][4];
    __shared__ float s_col[ROWS > 1 ? ROWS * 64 * W * NP * V : 1];
    RowSum<W, 3> row_sums{s_sum};
    const int l = threadIdx.x % (64 * W), sub = threadIdx.x / (64 * W);
    const float inv = 1.0f / static_cast<float>(a.width);
    uint64_t seed = 0, first = 0;
    if (a.drop.threshold) drop_start(a.drop, seed, first);
    float postw[NP][V], prew[NP][V], scale[NP][V], gate[NP][V];
    float dpre[NP][V], dpost[NP][V], dscale[NP][V], dgate[NP][V];
    bool has[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int c = (p * 64 * W + l) * V;
        has[p] = c < a.width;
        load_weights<V>(has[p] ? a.postw : nullptr, c, postw[p], 1.0f);
        load_weights<V>(has[p] ? a.prew : nullptr, c, prew[p], 1.0f);
        load_weights<V>(has[p] ? a.scale : nullptr, c, scale[p], 1.0f);
        load_weights<V>(has[p] && a.gate_kind == GATE_CHANNEL ? static_cast<const float*>(a.gate) : nullptr, c, gate[p], 1.0f);
#pragma unroll
        for (int i = 0; i < V; ++i) dpre[p][i] = dpost[p][i] = dscale[p][i] = dgate[p][i] = 0.0f;
    }
    const bool by_sequence = a.gate_kind == GATE_SEQUENCE;
    const int64_t group_rows = by_sequence ? a.s : a.rows;
    const int64_t g0 = static_cast<int64_t>(blockIdx.x) / a.chunks * a.per;
    const int64_t g1 = g0 + a.per < a.groups ? g0 + a.per : a.groups;
    const int chunk = static_cast<int>(blockIdx.x) % a.chunks;
    for (int64_t g = g0; g < g1; ++g) {
        if (by_sequence) {
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                load_weights<V>(has[p] ? static_cast<const float*>(a.gate) : nullptr,
                                g * a.width + (p * 64 * W + l) * V, gate[p], 1.0f);
#pragma unroll
                for (int i = 0; i < V; ++i) dgate[p][i] = 0.0f;
            }
        }
        for (int64_t i0 = static_cast<int64_t>(chunk) * ROWS; i0 < group_rows; i0 += static_cast<int64_t>(a.chunks) * ROWS) {
            const bool real = i0 + sub < group_rows;
            const int64_t row = g * group_rows + i0 + sub;
            Raw<TX, V> rv[NP], rdv[NP], rx[NP];
            Raw<TY, V> rdz[NP], ry[NP], rg[NP];
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const int c = (p * 64 * W + l) * V;
                rv[p].zero();
                rdv[p].zero();
                rx[p].zero();
                rdz[p].zero();
                ry[p].zero();
                rg[p].zero();
                if (real && has[p]) {
                    rv[p].load(static_cast<const TX*>(a.xo) + row * a.xo_s + c);
                    rdz[p].load(static_cast<const TY*>(a.dz) + row * a.dz_s + c);
                    if (a.dxo) rdv[p].load(static_cast<const TX*>(a.dxo) + row * a.dxo_s + c);
                    if (a.dscale) rx[p].load(static_cast<const TX*>(a.x) + row * a.x_s + c);
                    if (a.y) ry[p].load(static_cast<const TY*>(a.y) + row * a.y_s + c);
                    if (a.gate_kind == GATE_FULL) rg[p].load(static_cast<const TY*>(a.gate) + row * a.g_s + c);
                }
            }
            float sum[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    sum[0] = fmaf(rv[p].at(i), rv[p].at(i), sum[0]);
                    sum[1] = fmaf(rdz[p].at(i) * prew[p][i], rv[p].at(i), sum[1]);
                    sum[2] = fmaf(ry[p].at(i), ry[p].at(i), sum[2]);
                }
            row_sums(sum);
            const float r2 = 1.0f / sqrtf(fmaf(sum[0], inv, a.eps)), mean2 = sum[1] * r2 * inv;
            const float r = a.post ? 1.0f / sqrtf(fmaf(sum[2], inv, a.eps)) : 1.0f;
            float u[NP][V];
            float dot[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const int c = (p * 64 * W + l) * V;
                float e[V], o[V], f[V];
                bool keep[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float unit = rv[p].at(i) * r2, dz = rdz[p].at(i);
                    dpre[p][i] = real ? fmaf(dz, unit, dpre[p][i]) : dpre[p][i];
                    e[i] = fmaf(r2, fmaf(-unit, mean2, dz * prew[p][i]), rdv[p].at(i));
                    if (!real) e[i] = 0.0f;
                    o[i] = e[i] * scale[p][i];
                    dscale[p][i] = fmaf(e[i], rx[p].at(i), dscale[p][i]);
                    f[i] = 1.0f;
                    keep[i] = true;
                }
                if (real && has[p] && a.dx) store_piece<TX, V>(static_cast<TX*>(a.dx) + row * a.width + c, o);
                if (!a.y) continue;
                if (a.drop.threshold && real && has[p]) drop_factors<V>(a.drop, seed, first, row * a.width + c, f, keep);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float yu = a.post ? ry[p].at(i) * r : ry[p].at(i), n = a.post ? yu * postw[p][i] : yu;
                    o[i] = keep[i] ? e[i] * n * f[i] : 0.0f;  // gradient of the gate
                    if (a.gate_kind == GATE_CHANNEL || by_sequence) dgate[p][i] += real && has[p] ? o[i] : 0.0f;
                    const float gt = a.gate_kind == GATE_FULL ? rg[p].at(i) : gate[p][i];
                    const float dn = keep[i] ? e[i] * gt * f[i] : 0.0f;
                    if (a.post) {
                        dpost[p][i] = real && has[p] ? fmaf(dn, yu, dpost[p][i]) : dpost[p][i];
                        u[p][i] = dn * postw[p][i];
                        dot[0] = has[p] ? fmaf(u[p][i], yu, dot[0]) : dot[0];
                    } else {
                        u[p][i] = dn;
                    }
                }
                if (a.gate_kind == GATE_FULL && real && has[p])
                    store_piece<TY, V>(static_cast<TY*>(a.dgate) + row * a.width + c, o);
            }
            if (!a.y) continue;
            if (a.post) {
                row_sums(dot);
                dot[0] *= inv;
            }
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const int c = (p * 64 * W + l) * V;
                if (a.post) {
#pragma unroll
                    for (int i = 0; i < V; ++i) u[p][i] = r * fmaf(-ry[p].at(i) * r, dot[0], u[p][i]);
                }
                if (real && has[p]) store_piece<TY, V>(static_cast<TY*>(a.dy) + row * a.width + c, u[p]);
            }
        }
        if (by_sequence)
            sum_rows<V, NP, W>(dgate, s_col,
                               a.gate_part ? a.gate_part + (g * a.chunks + chunk) * a.width : static_cast<float*>(a.dgate) + g * a.width,
                               a.width);
    }
    float* part = a.part + static_cast<int64_t>(blockIdx.x) * 4 * a.width;
    if (a.dprew) sum_rows<V, NP, W>(dpre, s_col, part, a.width);
    if (a.dpostw) sum_rows<V, NP, W>(dpost, s_col, part + a.width, a.width);
    if (a.dscale) sum_rows<V, NP, W>(dscale, s_col, part + 2 * a.width, a.width);
    if (a.dgate && a.gate_kind == GATE_CHANNEL) sum_rows<V, NP, W>(dgate, s_col, part + 3 * a.width, a.width);
}

// Sums of the workgroups' rows: blockIdx.y < 4 of the vectors, and from 4 on of
// the sequences' gates.  64 threads a column, joined in one order; workgroups of
// 16 columns.
__global__ __launch_bounds__(1024) void k_resid_join(const ResidArgs a) {
    __shared__ float s[64][17];
    const int job = blockIdx.y, c = blockIdx.x * 16 + (threadIdx.x & 15), y = threadIdx.x >> 4;
    const float* src;
    float* dst;
    int64_t rows, step;
    if (job < 4) {
        float* const out[4] = {a.dprew, a.dpostw, a.dscale, a.gate_kind == GATE_CHANNEL ? static_cast<float*>(a.dgate) : nullptr};
        dst = out[job];
        src = a.part + job * a.width;
        rows = a.blocks;
        step = 4 * static_cast<int64_t>(a.width);
    } else {
        dst = static_cast<float*>(a.dgate) + static_cast<int64_t>(job - 4) * a.width;
        src = a.gate_part + static_cast<int64_t>(job - 4) * a.chunks * a.width;
        rows = a.chunks;
        step = a.width;
    }
    if (!dst) return;
    float x = 0.0f;
    if (c < a.width) {
#pragma unroll 8
        for (int64_t i = y; i < rows; i += 64) x += src[i * step + c];
    }
    s[y][threadIdx.x & 15] = x;
    __syncthreads();
    for (int m = 32; m; m >>= 1) {
        if (y < m) s[y][threadIdx.x & 15] += s[y + m][threadIdx.x & 15];
        __syncthreads();
    }
    if (y == 0 && c < a.width) dst[c] = s[0][threadIdx.x & 15];
}

template <typename TX, typename TY, int V, int NP, int W>
void start(const ResidArgs& a, bool backward, hipStream_t stream) {
    if (backward) k_resid_norm_bwd<TX, TY, V, NP, W><<<static_cast<uint32_t>(a.blocks), threads_of<W>(), 0, stream>>>(a);
    else k_resid_norm<TX, TY, V, NP, W><<<static_cast<uint32_t>(a.blocks), threads_of<W>(), 0, stream>>>(a);
}

template <typename TX, typename TY>
void by_width(const ResidArgs& a, bool backward, hipStream_t stream) {
    if (a.vector) {
        if (a.waves == 1 && a.pieces == 1) start<TX, TY, 8, 1, 1>(a, backward, stream);
        else if (a.waves == 1) start<TX, TY, 8, 2, 1>(a, backward, stream);
        else if (a.waves == 2) start<TX, TY, 8, 2, 2>(a, backward, stream);
        else if (a.waves == 4) start<TX, TY, 8, 2, 4>(a, backward, stream);
        else start<TX, TY, 8, 2, 8>(a, backward, stream);
    } else {
        // odd widths or alignment: value by value
        if (a.waves == 1) start<TX, TY, 1, 4, 1>(a, backward, stream);
        else if (a.waves == 4) start<TX, TY, 1, 8, 4>(a, backward, stream);
        else start<TX, TY, 1, 16, 8>(a, backward, stream);
    }
}

void run(const ResidArgs& a, bool backward, hipStream_t stream) {
    if (a.x_type == MUON_BF16) by_width<bf16_t, bf16_t>(a, backward, stream);
    else if (a.y_type == MUON_BF16) by_width<float, bf16_t>(a, backward, stream);
    else by_width<float, float>(a, backward, stream);
}

}  // namespace

hipError_t launch_resid_norm(const ResidArgs& a, hipStream_t stream) {
    run(a, false, stream);
    return hipGetLastError();
}

hipError_t launch_resid_norm_bwd(const ResidArgs& a, hipStream_t stream) {
    if (a.blocks > 0) run(a, true, stream);
    const bool vectors = a.dprew || a.dpostw || a.dscale || (a.dgate && a.gate_kind == GATE_CHANNEL);
    const int64_t gates = a.gate_part ? a.groups : 0;
    if (vectors || gates > 0)
        k_resid_join<<<dim3((a.width + 15) / 16, static_cast<uint32_t>(4 + gates)), 1024, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace muon
