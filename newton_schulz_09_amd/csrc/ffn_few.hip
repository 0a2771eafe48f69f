// The feed-forward block of a few tokens (a step of generation):
//     h = act(x Wg^T) (x Wu^T),  out = h Wd^T.
//
// Bound by the bytes of the matrices.  Each wave streams 16 rows of a matrix
// straight into the matrix cores' operand registers (lane l: row l % 16, 8
// values of K), with the tokens as the other operand, so a matrix is read once
// and never passes through LDS.  K is split over the waves of a workgroup,
// whose sums are joined through LDS in one order: 16 rows a workgroup, hidden / 16
// workgroups for h and width / 16 for the result.  The latter are fewer than the
// 256 CUs below a width of 4096 (48 at 768, 100 at 1600), which then read less
// than memory gives.  Measured: one token of 768 to 2048 4.5 and 4.5 us (9.4 MB; the
// time of a launch and one trip to memory), of 1600 to 4264 23 us a call (41 MB, 1.8
// TB/s), of 4096 to 10240 63 (252 MB, 4.0 TB/s).
#include "../../include/muon.h"
#include "ffn_common.hpp"

namespace muon {

namespace {

using namespace ffn;

// The products of steps [s, s + U) of 32 K values: NM matrix fragments by MT
// token fragments.  Loads of one batch are on their way while the one before is
// multiplied.
template <int NM, int MT, int U, bool PACKED>
struct Batch {
    u32x4 w[U][NM], x[U][MT];
    __device__ __forceinline__ void load(const bf16_t* const (&wp)[NM], const bf16_t* const (&xp)[MT], int s, int s1, int k_lane, int k) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = (s + u) * 32 + k_lane;
            const bool in = s + u < s1 && at < k;
#pragma unroll
            for (int i = 0; i < NM; ++i) {
                w[u][i] = u32x4{0, 0, 0, 0};
                if (in) w[u][i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(wp[i] + at));
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                x[u][m] = u32x4{0, 0, 0, 0};
                if (in) x[u][m] = *reinterpret_cast<const u32x4*>(xp[m] + (PACKED ? (s + u) * (MT * 512) : at));
            }
        }
    }
    __device__ __forceinline__ void multiply(f32x4 (&acc)[NM][MT]) const {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < NM; ++i)
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    acc[i][m] = mfma16(__builtin_bit_cast(bf16x8, w[u][i]), __builtin_bit_cast(bf16x8, x[u][m]), acc[i][m]);
    }
};

// This wave's part of NM x MT fragments over K values.
template <int NM, int MT, int WAVES, bool PACKED>
__device__ __forceinline__ void stream(const bf16_t* const (&wp)[NM], const bf16_t* const (&xp)[MT], int k, f32x4 (&acc)[NM][MT]) {
    constexpr int U = NM * MT >= 4 ? 2 : 4;
    const int wave = attn::wave_id(), k_lane = 8 * (attn::lane_id() >> 4);
    const int steps = (k + 31) / 32, per = (steps + WAVES - 1) / WAVES;
    const int s0 = wave * per, s1 = s0 + per < steps ? s0 + per : steps;
#pragma unroll
    for (int i = 0; i < NM; ++i)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[i][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    Batch<NM, MT, U, PACKED> a, b;
    if (s0 < s1) a.load(wp, xp, s0, s1, k_lane, k);
    for (int s = s0; s < s1; s += 2 * U) {
        if (s + U < s1) b.load(wp, xp, s + U, s1, k_lane, k);
        a.multiply(acc);
        if (s + U < s1) {
            if (s + 2 * U < s1) a.load(wp, xp, s + 2 * U, s1, k_lane, k);
            b.multiply(acc);
        }
    }
}

// The rows of tokens that a lane reads: those past the last one read it again,
// and their results are not stored.
template <int MT>
__device__ __forceinline__ void token_rows(const bf16_t* p, int64_t stride, int tokens, const bf16_t* (&xp)[MT]) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        int t = 16 * m + (attn::lane_id() & 15);
        if (t >= tokens) t = tokens - 1;
        xp[m] = p + t * stride;
    }
}

// 16 hidden values a workgroup.
template <int MT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_few_gated(const FfnFew a) {
    __shared__ f32x4 s[WAVES][2 * MT][64];
    const int lane = attn::lane_id(), wave = attn::wave_id();
    const bf16_t *wp[2], *xp[MT];
    int row = blockIdx.x * 16 + (lane & 15);
    if (row >= a.hidden) row = a.hidden - 1;
    wp[0] = a.w_gate + row * a.w_stride;
    wp[1] = a.w_up + row * a.w_stride;
    token_rows<MT>(a.x, a.x_stride, a.tokens, xp);
    f32x4 acc[2][MT];
    stream<2, MT, WAVES, false>(wp, xp, a.width, acc);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int m = 0; m < MT; ++m) s[wave][i * MT + m][lane] = acc[i][m];
    __syncthreads();
    for (int item = threadIdx.x; item < MT * 64; item += 64 * WAVES) {
        const int m = item / 64, l = item % 64;
        f32x4 gate = s[0][m][l], up = s[0][MT + m][l];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) {
            gate += s[w][m][l];
            up += s[w][MT + m][l];
        }
        // lane l holds token l % 16, hidden values 4 (l / 16) .. + 3
        const int token = 16 * m + (l & 15), col = blockIdx.x * 16 + 4 * (l >> 4);
        if (token >= a.tokens || col >= a.hidden) continue;
        float h[4];
        by_act(a.act, [&](auto act) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v, unused;
                activate<act>(gate[i], v, unused);
                h[i] = v * up[i];
            }
        });
        // in the order in which the next kernel reads it: a fragment of 16 tokens
        // by 32 values is one piece of 1 KB
        *reinterpret_cast<u32x2*>(a.h + ((static_cast<int64_t>(col / 32) * MT + m) * 64 + (l & 15) + col % 32 / 8 * 16) * 8 + col % 8) =
            u32x2{f32x2_to_bf16x2(h[0], h[1]), f32x2_to_bf16x2(h[2], h[3])};
    }
}

// 16 values of width a workgroup.
template <int MT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_few_down(const FfnFew a) {
    __shared__ f32x4 s[WAVES][MT][64];
    const int lane = attn::lane_id(), wave = attn::wave_id();
    const bf16_t *wp[1], *xp[MT];
    int row = blockIdx.x * 16 + (lane & 15);
    if (row >= a.width) row = a.width - 1;
    wp[0] = a.w_down + row * a.w_down_stride;
#pragma unroll
    for (int m = 0; m < MT; ++m) xp[m] = a.h + (m * 64 + lane) * 8;
    f32x4 acc[1][MT];
    stream<1, MT, WAVES, true>(wp, xp, a.hidden, acc);
#pragma unroll
    for (int m = 0; m < MT; ++m) s[wave][m][lane] = acc[0][m];
    __syncthreads();
    for (int item = threadIdx.x; item < MT * 64; item += 64 * WAVES) {
        const int m = item / 64, l = item % 64;
        f32x4 v = s[0][m][l];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) v += s[w][m][l];
        const int token = 16 * m + (l & 15), col = blockIdx.x * 16 + 4 * (l >> 4);
        if (token < a.tokens && col < a.width)
            *reinterpret_cast<u32x2*>(a.out + static_cast<int64_t>(token) * a.width + col) =
                u32x2{f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3])};
    }
}

template <int MT>
void start(const FfnFew& a, hipStream_t stream) {
    k_few_gated<MT, 8><<<(a.hidden + 15) / 16, 512, 0, stream>>>(a);
    k_few_down<MT, 16><<<(a.width + 15) / 16, 1024, 0, stream>>>(a);
}

}  // namespace

hipError_t launch_ffn_few(const FfnFew& a, hipStream_t stream) {
    if (a.tokens <= 16) start<1>(a, stream);
    else start<2>(a, stream);
    return hipGetLastError();
}

}  // namespace muon
