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
// registers between.  T threads hold a row, 8 values a piece and 1 or 2 pieces each,
// so a row of 1024 values needs no exchange but that inside its wave.
// Workgroups walk rows, so weights are loaded and gradients of weights summed
// in registers; a second, small kernel joins the workgroups' sums in one order.
// Measured, forward: 65536 rows of 768 bf16 76 us (403 MB, 5.3 TB/s).  Gradients: the
// same with dropout and four vectors' gradients 155 us and 5 for the join (4.5 TB/s),
// 8192 rows of 2048 with a gate each element 49 us (5.4), 2331 of 1600 with a float32
// stream 26 us (2.5: 294 workgroups with eight rows each, two at a time, whose loads
// wait for the sums of the rows before).
#include <type_traits>

#include "../../include/muon.h"
#include "layer_common.hpp"

namespace muon {

namespace {

constexpr int V = 8;  // values of a piece
typedef u32x4_t __attribute__((aligned(4))) u32x4_by4;
typedef u32x4_t __attribute__((aligned(2))) u32x4_by2;

// A piece as it lies in memory.  ALIGNED: to 16 bytes, and rows are whole
// pieces; else loads and stores of any alignment, value by value where the row
// ends inside the piece (`n` values are left; the others come as zeros).
template <typename T, bool ALIGNED>
struct Raw {
    static constexpr int N = V * sizeof(T) / 16;
    using Part = std::conditional_t<ALIGNED, u32x4_t, std::conditional_t<sizeof(T) == 4, u32x4_by4, u32x4_by2>>;
    u32x4_t u[N];
    __device__ __forceinline__ void load(const T* p, int n) {
        if (ALIGNED || n >= V) {
#pragma unroll
            for (int i = 0; i < N; ++i) u[i] = reinterpret_cast<const Part*>(p)[i];
        } else {
#pragma unroll
            for (int i = 0; i < V - 1; ++i)
                if (i < n) {
                    if constexpr (sizeof(T) == 4) u[i >> 2][i & 3] = __float_as_uint(p[i]);
                    else u[0][i >> 1] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
                }
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < N; ++i) u[i] = u32x4_t{0, 0, 0, 0};
    }
    // What was unpacked before is unpacked again, and not kept.
    __device__ __forceinline__ void again() {
#pragma unroll
        for (int i = 0; i < N; ++i) asm volatile("" : "+v"(u[i]));
    }
    __device__ __forceinline__ float at(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(u[i >> 2][i & 3]);
        else return __uint_as_float(i & 1 ? u[0][i >> 1] & 0xffff0000u : u[0][i >> 1] << 16);
    }
};
template <typename T, bool ALIGNED>
__device__ __forceinline__ void store_piece(T* p, const float (&x)[V], int n) {
    typedef typename Raw<T, ALIGNED>::Part Part;
    if (!ALIGNED && n < V) {
#pragma unroll
        for (int i = 0; i < V - 1; ++i)
            if (i < n) {
                if constexpr (sizeof(T) == 2) p[i] = f32_to_bf16(x[i]);
                else p[i] = x[i];
            }
    } else if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<Part*>(p) = u32x4_t{f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]),
                                              f32x2_to_bf16x2(x[4], x[5]), f32x2_to_bf16x2(x[6], x[7])};
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            reinterpret_cast<Part*>(p)[i] = u32x4_t{__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]),
                                                    __float_as_uint(x[4 * i + 2]), __float_as_uint(x[4 * i + 3])};
    }
}
// float32 values p[at ..], of which n are there; ones without p and past the end.
template <bool ALIGNED>
__device__ __forceinline__ void load_weights(const float* p, int64_t at, int n, float (&x)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = 1.0f;
    if (!p || n <= 0) return;
    if (ALIGNED || n >= V) {
        typedef f32x4 __attribute__((aligned(4))) f32x4u;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const f32x4 u = reinterpret_cast<const f32x4u*>(p + at)[i];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[4 * i + k] = u[k];
        }
    } else {
#pragma unroll
        for (int i = 0; i < V - 1; ++i)
            if (i < n) x[i] = p[at + i];
    }
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
// Sum over groups of T lanes (at most 64), in every lane.
template <int T>
__device__ __forceinline__ float lanes_sum(float x) {
    x = dpp_add<0xB1>(x);   // lanes 1 0 3 2
    x = dpp_add<0x4E>(x);   // lanes 2 3 0 1
    x = dpp_add<0x141>(x);  // 8 lanes mirrored
    if constexpr (T == 8) return x;
    x = dpp_add<0x140>(x);  // 16 lanes mirrored
    if constexpr (T == 16) return x;
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    if constexpr (T == 32) return x;
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Threads of a workgroup whose rows have T threads each.
template <int T>
constexpr int threads_of() { return T > 256 ? T : 256; }

// Sums of K values over the T threads of each row, in every lane of the row.
template <int T>
struct RowSum {
    static constexpr int ROWS = threads_of<T>() / T, W = T > 64 ? T / 64 : 1;
    float (*s)[ROWS][W][4];
    int flip = 0;
    template <int K>
    __device__ __forceinline__ void operator()(float (&x)[K]) {
#pragma unroll
        for (int k = 0; k < K; ++k) x[k] = lanes_sum<(T < 64 ? T : 64)>(x[k]);
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

// Drops the V elements from element `at` on, and scales the others.
template <bool ALIGNED>
struct Dropper {
    u32x4_t lo, hi;
    int shift;
    __device__ __forceinline__ void init(const DropState& d, uint64_t seed, uint64_t first, int64_t at) {
        lo = philox(seed, first + static_cast<uint64_t>(at >> 3));
        shift = ALIGNED ? 0 : static_cast<int>(at & 7);
        if (!ALIGNED && shift) {  // the elements lie in two blocks: the first one's end, then the second one's beginning
            hi = philox(seed, first + static_cast<uint64_t>(at >> 3) + 1);
            uint32_t w[9] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3], 0};
            const int words = shift >> 1, odd = shift & 1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t a = w[i], b = w[i + 1];
#pragma unroll
                for (int k = 1; k < 4; ++k)
                    if (words == k) {
                        a = w[i + k];
                        b = w[i + k + 1];
                    }
                lo[i] = odd ? (a >> 16) | (b << 16) : a;
            }
        }
    }
    __device__ __forceinline__ float operator()(const DropState& d, int i, float x) const {
        return drop_keeps(lo, i, d.threshold) ? x * d.factor : 0.0f;
    }
};

template <typename TX, typename TY, int NP, int T, bool ALIGNED>
__global__ __launch_bounds__(threads_of<T>()) void k_resid_norm(const ResidArgs a) {
    constexpr int ROWS = threads_of<T>() / T;
    __shared__ float s_sum[2][ROWS][RowSum<T>::W][4];
    RowSum<T> row_sum{s_sum};
    const int l = threadIdx.x % T, sub = threadIdx.x / T;
    const float inv = 1.0f / static_cast<float>(a.width);
    uint64_t seed = 0, first = 0;
    if (a.drop.threshold) drop_start(a.drop, seed, first);
    float postw[NP][V], prew[NP][V], scale[NP][V], gate[NP][V];
    int left[NP];  // values of the row from the piece on
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int c = (p * T + l) * V;
        left[p] = a.width - c;
        load_weights<ALIGNED>(a.postw, c, left[p], postw[p]);
        load_weights<ALIGNED>(a.prew, c, left[p], prew[p]);
        load_weights<ALIGNED>(a.scale, c, left[p], scale[p]);
        load_weights<ALIGNED>(a.gate_kind == GATE_CHANNEL ? static_cast<const float*>(a.gate) : nullptr, c, left[p], gate[p]);
    }
    for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * ROWS; row0 < a.rows; row0 += static_cast<int64_t>(gridDim.x) * ROWS) {
        const int64_t row = row0 + sub;
        const bool real = row < a.rows;  // (the others take part in the exchanges)
        Raw<TX, ALIGNED> rx[NP];
        Raw<TY, ALIGNED> ry[NP], rg[NP];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int c = (p * T + l) * V;
            rx[p].zero();
            ry[p].zero();
            rg[p].zero();
            if (real && left[p] > 0) {
                rx[p].load(static_cast<const TX*>(a.x) + row * a.x_s + c, left[p]);
                if (a.y) ry[p].load(static_cast<const TY*>(a.y) + row * a.y_s + c, left[p]);
                if (a.gate_kind == GATE_FULL) rg[p].load(static_cast<const TY*>(a.gate) + row * a.g_s + c, left[p]);
                else if (a.gate_kind == GATE_SEQUENCE)
                    load_weights<ALIGNED>(static_cast<const float*>(a.gate), row / a.s * a.width + c, left[p], gate[p]);
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
                const int c = (p * T + l) * V;
                const float mine = left[p] > 0 ? r : 0.0f;  // (r is infinite for a row of zeros without eps)
                float n[V];
#pragma unroll
                for (int i = 0; i < V; ++i) n[i] = ry[p].at(i) * mine * postw[p][i];
                if (a.drop.threshold) {
                    Dropper<ALIGNED> drop;
                    drop.init(a.drop, seed, first, row * a.width + c);
#pragma unroll
                    for (int i = 0; i < V; ++i) n[i] = drop(a.drop, i, n[i]);
                }
                if (a.gate_kind == GATE_FULL) {
#pragma unroll
                    for (int i = 0; i < V; ++i) n[i] *= rg[p].at(i);
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) n[i] *= gate[p][i];
                }
#pragma unroll
                for (int i = 0; i < V; ++i) v[p][i] = fmaf(rx[p].at(i), scale[p][i], n[i]);
                // past the row's end there are zeros in ry: nothing that a sum would notice but 0 * inf
                if (!ALIGNED && left[p] < V) {
#pragma unroll
                    for (int i = 1; i < V; ++i)
                        if (i >= left[p]) v[p][i] = 0.0f;
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
            const int c = (p * T + l) * V;
            if (real && left[p] > 0 && a.x_out) store_piece<TX, ALIGNED>(static_cast<TX*>(a.x_out) + row * a.width + c, v[p], left[p]);
#pragma unroll
            for (int i = 0; i < V; ++i) sum[0] = fmaf(v[p][i], v[p][i], sum[0]);
        }
        row_sum(sum);
        const float r = 1.0f / sqrtf(fmaf(sum[0], inv, a.eps));
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int c = (p * T + l) * V;
            float z[V];
#pragma unroll
            for (int i = 0; i < V; ++i) z[i] = v[p][i] * r * prew[p][i];
            if (real && left[p] > 0) store_piece<TY, ALIGNED>(static_cast<TY*>(a.z) + row * a.width + c, z, left[p]);
        }
    }
}

// Sum of every row of the workgroup, column by column: the waves that hold the
// same columns are added in one order.  s: ROWS x width.
template <int NP, int T>
__device__ __forceinline__ void sum_rows(const float (&x)[NP][V], float* s, float* dst, int width) {
    constexpr int ROWS = threads_of<T>() / T;
    const int l = threadIdx.x % T, sub = threadIdx.x / T;
    if constexpr (ROWS == 1) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int c = (p * T + l) * V;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (c + i < width) dst[c + i] = x[p][i];
        }
    } else {
        __syncthreads();
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int c = (p * T + l) * V;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (c + i < width) s[sub * width + c + i] = x[p][i];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < width; c += threads_of<T>()) {
            float t = s[c];
#pragma unroll
            for (int r = 1; r < ROWS; ++r) t += s[r * width + c];
            dst[c] = t;
        }
    }
}

// Backward the vectors lie in LDS, 4 values of a lane side by side with the
// next lane's: with them in registers beside the sums of their gradients fewer
// waves fit.
template <typename TX, typename TY, int NP, int T, bool ALIGNED>
__global__ __launch_bounds__(threads_of<T>(), 2) void k_resid_norm_bwd(const ResidArgs a) {
    constexpr int ROWS = threads_of<T>() / T;
    __shared__ float s_sum[2][ROWS][RowSum<T>::W][4];
    __shared__ float s_col[ROWS > 1 ? ROWS * T * NP * V : 1];
    __shared__ f32x4 s_w[4][NP * 2 * T];  // prew, scale, gate, postw
    RowSum<T> row_sum{s_sum};
    const int l = threadIdx.x % T, sub = threadIdx.x / T;
    const float inv = 1.0f / static_cast<float>(a.width);
    uint64_t seed = 0, first = 0;
    if (a.drop.threshold) drop_start(a.drop, seed, first);
    float dpre[NP][V], dpost[NP][V], dscale[NP][V], dgate[NP][V];
    int left[NP];
    auto put = [&](int k, const float* p, int64_t at) {
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            float x[V];
            load_weights<ALIGNED>(p, at + (q * T + l) * V, left[q], x);
            s_w[k][2 * q * T + l] = f32x4{x[0], x[1], x[2], x[3]};
            s_w[k][(2 * q + 1) * T + l] = f32x4{x[4], x[5], x[6], x[7]};
        }
    };
    auto get = [&](int k, int q, float (&x)[V]) {
        int at = l;
        asm volatile("" : "+v"(at));  // (read where it is used, and not kept over the rows)
        const f32x4 lo = s_w[k][2 * q * T + at], hi = s_w[k][(2 * q + 1) * T + at];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = lo[i];
            x[4 + i] = hi[i];
        }
    };
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        left[p] = a.width - (p * T + l) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) dpre[p][i] = dpost[p][i] = dscale[p][i] = dgate[p][i] = 0.0f;
    }
    const bool by_sequence = a.gate_kind == GATE_SEQUENCE;
    if (sub == 0) {
        put(0, a.prew, 0);
        put(1, a.scale, 0);
        put(2, a.gate_kind == GATE_CHANNEL ? static_cast<const float*>(a.gate) : nullptr, 0);
        put(3, a.postw, 0);
    }
    __syncthreads();
    const int64_t group_rows = by_sequence ? a.s : a.rows;
    const int64_t g0 = static_cast<int64_t>(blockIdx.x) / a.chunks * a.per;
    const int64_t g1 = g0 + a.per < a.groups ? g0 + a.per : a.groups;
    const int chunk = static_cast<int>(blockIdx.x) % a.chunks;
    for (int64_t g = g0; g < g1; ++g) {
        if (by_sequence) {
            __syncthreads();
            if (sub == 0) put(2, static_cast<const float*>(a.gate), g * a.width);
            __syncthreads();
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
                for (int i = 0; i < V; ++i) dgate[p][i] = 0.0f;
        }
        for (int64_t i0 = static_cast<int64_t>(chunk) * ROWS; i0 < group_rows; i0 += static_cast<int64_t>(a.chunks) * ROWS) {
            const bool real = i0 + sub < group_rows;
            const int64_t row = g * group_rows + i0 + sub;
            Raw<TX, ALIGNED> rv[NP], rdv[NP], rx[NP];
            Raw<TY, ALIGNED> rdz[NP], ry[NP], rg[NP];
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const int c = (p * T + l) * V;
                rv[p].zero();
                rdv[p].zero();
                rx[p].zero();
                rdz[p].zero();
                ry[p].zero();
                rg[p].zero();
                if (real && left[p] > 0) {
                    rv[p].load(static_cast<const TX*>(a.xo) + row * a.xo_s + c, left[p]);
                    rdz[p].load(static_cast<const TY*>(a.dz) + row * a.dz_s + c, left[p]);
                    if (a.dxo) rdv[p].load(static_cast<const TX*>(a.dxo) + row * a.dxo_s + c, left[p]);
                    if (a.dscale) rx[p].load(static_cast<const TX*>(a.x) + row * a.x_s + c, left[p]);
                    if (a.y) ry[p].load(static_cast<const TY*>(a.y) + row * a.y_s + c, left[p]);
                    if (a.gate_kind == GATE_FULL) rg[p].load(static_cast<const TY*>(a.gate) + row * a.g_s + c, left[p]);
                }
            }
            float sum[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                float w[V];
                get(0, p, w);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    sum[0] = fmaf(rv[p].at(i), rv[p].at(i), sum[0]);
                    sum[1] = fmaf(rdz[p].at(i) * w[i], rv[p].at(i), sum[1]);
                }
            }
            if (a.post) {
#pragma unroll
                for (int p = 0; p < NP; ++p)
#pragma unroll
                    for (int i = 0; i < V; ++i) sum[2] = fmaf(ry[p].at(i), ry[p].at(i), sum[2]);
            }
            row_sum(sum);
            // past the row's end and the last row everything is zero (r would be
            // infinite there without eps)
            const float r2 = 1.0f / sqrtf(fmaf(sum[0], inv, a.eps)), mean2 = sum[1] * r2 * inv;
            const float r = a.post ? 1.0f / sqrtf(fmaf(sum[2], inv, a.eps)) : 1.0f;
            float u[NP][V];
            float dot[1] = {0.0f};
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const int c = (p * T + l) * V;
                const bool here = real && left[p] > 0;
                __builtin_amdgcn_sched_barrier(0);
                rv[p].again();
                rdz[p].again();
                ry[p].again();
                const float r2p = here ? r2 : 0.0f, mean2p = here ? mean2 : 0.0f, rp = here ? r : 0.0f;
                float e[V], w[V], o[V];
                get(0, p, w);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float unit = rv[p].at(i) * r2p, dz = rdz[p].at(i);
                    dpre[p][i] = fmaf(dz, unit, dpre[p][i]);
                    e[i] = fmaf(r2p, fmaf(-unit, mean2p, dz * w[i]), rdv[p].at(i));
                }
                get(1, p, w);
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] = e[i] * w[i];
                if (a.dscale) {
#pragma unroll
                    for (int i = 0; i < V; ++i) dscale[p][i] = fmaf(e[i], rx[p].at(i), dscale[p][i]);
                }
                if (here) store_piece<TX, ALIGNED>(static_cast<TX*>(a.dx) + row * a.width + c, o, left[p]);
                if (!a.y) continue;
                float yu[V], n[V];
                get(3, p, w);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    yu[i] = ry[p].at(i) * rp;
                    n[i] = yu[i] * w[i];
                    u[p][i] = e[i];
                }
                if (a.drop.threshold) {
                    Dropper<ALIGNED> drop;
                    drop.init(a.drop, seed, first, row * a.width + c);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        n[i] = drop(a.drop, i, n[i]);
                        u[p][i] = drop(a.drop, i, u[p][i]);
                    }
                }
                if (a.gate_kind == GATE_FULL) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        o[i] = e[i] * n[i];
                        u[p][i] *= rg[p].at(i);
                    }
                    if (here) store_piece<TY, ALIGNED>(static_cast<TY*>(a.dgate) + row * a.width + c, o, left[p]);
                } else if (a.gate_kind != GATE_NONE) {
                    float gt[V];
                    get(2, p, gt);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        dgate[p][i] = fmaf(e[i], n[i], dgate[p][i]);
                        u[p][i] *= gt[i];
                    }
                }
                if (a.post) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        dpost[p][i] = fmaf(u[p][i], yu[i], dpost[p][i]);
                        u[p][i] *= w[i];
                        dot[0] = fmaf(u[p][i], yu[i], dot[0]);
                    }
                }
            }
            if (!a.y) continue;
            if (a.post) {
                row_sum(dot);
                dot[0] *= inv;
#pragma unroll
                for (int p = 0; p < NP; ++p) ry[p].again();
#pragma unroll
                for (int p = 0; p < NP; ++p)
#pragma unroll
                    for (int i = 0; i < V; ++i) u[p][i] = r * fmaf(-ry[p].at(i) * r, dot[0], u[p][i]);
            }
#pragma unroll
            for (int p = 0; p < NP; ++p)
                if (real && left[p] > 0)
                    store_piece<TY, ALIGNED>(static_cast<TY*>(a.dy) + row * a.width + (p * T + l) * V, u[p], left[p]);
        }
        if (by_sequence)
            sum_rows<NP, T>(dgate, s_col,
                            a.gate_part ? a.gate_part + (g * a.chunks + chunk) * a.width : static_cast<float*>(a.dgate) + g * a.width,
                            a.width);
    }
    float* part = a.part + static_cast<int64_t>(blockIdx.x) * 4 * a.width;
    if (a.dprew) sum_rows<NP, T>(dpre, s_col, part, a.width);
    if (a.dpostw) sum_rows<NP, T>(dpost, s_col, part + a.width, a.width);
    if (a.dscale) sum_rows<NP, T>(dscale, s_col, part + 2 * a.width, a.width);
    if (a.dgate && a.gate_kind == GATE_CHANNEL) sum_rows<NP, T>(dgate, s_col, part + 3 * a.width, a.width);
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

template <typename TX, typename TY, int NP, int T, bool ALIGNED>
void start(const ResidArgs& a, bool backward, hipStream_t stream) {
    const uint32_t blocks = static_cast<uint32_t>(a.blocks);
    if (backward) k_resid_norm_bwd<TX, TY, NP, T, ALIGNED><<<blocks, threads_of<T>(), 0, stream>>>(a);
    else k_resid_norm<TX, TY, NP, T, ALIGNED><<<blocks, threads_of<T>(), 0, stream>>>(a);
}

template <typename TX, typename TY, bool ALIGNED>
void by_width(const ResidArgs& a, bool backward, hipStream_t stream) {
    switch (a.threads) {
        case 8: return start<TX, TY, 1, 8, ALIGNED>(a, backward, stream);
        case 16: return start<TX, TY, 1, 16, ALIGNED>(a, backward, stream);
        case 32: return start<TX, TY, 1, 32, ALIGNED>(a, backward, stream);
        case 64: return a.pieces == 1 ? start<TX, TY, 1, 64, ALIGNED>(a, backward, stream) : start<TX, TY, 2, 64, ALIGNED>(a, backward, stream);
        case 128: return start<TX, TY, 2, 128, ALIGNED>(a, backward, stream);
        case 256: return start<TX, TY, 2, 256, ALIGNED>(a, backward, stream);
        default: return start<TX, TY, 2, 512, ALIGNED>(a, backward, stream);
    }
}

template <typename TX, typename TY>
void by_alignment(const ResidArgs& a, bool backward, hipStream_t stream) {
    if (a.vector) by_width<TX, TY, true>(a, backward, stream);
    else by_width<TX, TY, false>(a, backward, stream);
}

void run(const ResidArgs& a, bool backward, hipStream_t stream) {
    if (a.x_type == MUON_BF16) by_alignment<bf16_t, bf16_t>(a, backward, stream);
    else if (a.y_type == MUON_BF16) by_alignment<float, bf16_t>(a, backward, stream);
    else by_alignment<float, float>(a, backward, stream);
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
