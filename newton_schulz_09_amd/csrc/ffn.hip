// The products of a gated feed-forward block and its gradients, in bfloat16 on
// the matrix cores with float32 sums:
//     gate = x Wg^T, up = x Wu^T, h = act(gate) up       (one kernel)
//     out = h Wd^T
//     dh = dout Wd, dgate = dh up act'(gate), dup = dh act(gate)  (one kernel)
//     dx = dgate Wg + dup Wu                              (one sum)
//     dWg = dgate^T x, dWu = dup^T x, dWd = dout^T h      (one launch)
//
// Bound by the matrix cores for many tokens.  One engine: a workgroup computes
// a BM x BN tile with WGM x WGN waves of 32 x 32 fragments; K advances 64 at a
// time through two LDS stages that direct loads fill while the other is
// multiplied, one barrier a step.  Operands contiguous along K lie in LDS as
// rows of K and are read 16 bytes a lane; operands contiguous along the output
// lie as rows of output and are read with transposing reads, so nothing is
// ever transposed in memory.  Rows and columns past the matrices' ends come as
// zeros from the loads' bounds checks, so every size runs the same loop.
//
// The matrix instruction takes Q first, so a lane holds 4 consecutive columns
// of one output row; two lanes swap halves and each stores 16 bytes.
#include "../../include/muon.h"
#include "attn_common.hpp"
#include "layer_common.hpp"

namespace muon {

namespace {

using attn::descriptor;
using attn::each;
using attn::in_order;
using attn::landed;
using attn::lane_id;
using attn::lds_addr;
using attn::load_lds16;
using attn::mfma;
using attn::s16x4;
using attn::u32x2;
using attn::u32x4;

constexpr int kBk = 64;      // K values of a step
constexpr int kXcds = 8;
constexpr uint32_t kOut = 0x80000000u;  // an offset past every buffer's end

// Workgroup b of n -> place, so that each XCD (workgroups b = x, x + 8, ...)
// takes one contiguous range.
__device__ __forceinline__ int xcd_place(int b, int n) {
    const int q = n / kXcds, r = n % kXcds, x = b % kXcds;
    return x * q + (x < r ? x : r) + b / kXcds;
}

// Slot of 16-byte chunk c of row r is c ^ f(r).  Rows of K (8 chunks): 16 rows
// of one chunk fall on distinct banks.
__device__ __forceinline__ int rows_swizzle(int r) { return ((r >> 1) ^ (r << 2)) & 7; }
// Rows of output (CPR chunks): the 8 rows that a transposing read touches (two
// runs of 4, 8 apart) fall on distinct banks.
template <int CPR>
__device__ __forceinline__ int columns_swizzle(int r) {
    return ((((r & 3) << 1) | ((r >> 3) & 1)) * (CPR >= 16 ? 2 : 1)) & (CPR - 1);
}

// One operand's tile: B output rows (or columns) by kBk of K, COL: contiguous
// along the output.  NW waves load it, N loads of 1 KB a wave.
template <int B, bool COL, int NW>
struct Operand {
    static constexpr int CPR = COL ? B / 8 : kBk / 8;
    static constexpr int RPI = 64 / CPR;  // rows per load
    static constexpr int LROWS = COL ? kBk : B;
    static constexpr int N = LROWS / RPI / NW;
    static constexpr int BYTES = B * kBk * 2;
    static_assert(N * RPI * NW == LROWS, "whole loads per wave");
    uint32_t voff[N];
    uint64_t base;     // of the tile, at K = 0
    uint32_t ld2;      // bytes between rows
    int left;          // output rows (columns) from here to the end
    bool masked;

    __device__ __forceinline__ static int row_of(int wave, int i) { return (wave * N + i) * RPI + lane_id() / CPR; }
    __device__ __forceinline__ static int chunk_of(int row) {
        return (lane_id() % CPR) ^ (COL ? columns_swizzle<CPR>(row) : rows_swizzle(row));
    }
    // first: the tile's first output row; n: their number; place(row): the row's place from `first` on
    template <typename F>
    __device__ __forceinline__ void init(const bf16_t* p, int64_t ld, int64_t first, int n, int wave, F&& place) {
        base = reinterpret_cast<uint64_t>(p + (COL ? first : first * ld));
        ld2 = static_cast<uint32_t>(2 * ld);
        left = static_cast<int>(n - first);
        masked = false;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int row = row_of(wave, i), c = chunk_of(row);
            voff[i] = static_cast<uint32_t>(COL ? row : place(row)) * ld2 + 16 * c;
            if (COL && 8 * c >= left) voff[i] = kOut;
        }
    }
    // Lets through the first `lim` K values of a step (rows of K).
    __device__ __forceinline__ void limit(int64_t lim, int wave) {
        if constexpr (!COL) {
            if (lim >= kBk && !masked) return;
            masked = lim < kBk;
#pragma unroll
            for (int i = 0; i < N; ++i)
                voff[i] = 8 * chunk_of(row_of(wave, i)) >= lim ? voff[i] | kOut : voff[i] & ~kOut;
        }
    }
    // Descriptor of the step from K = k0 on, lim = K - k0 > 0; rows: output rows of the tile
    __device__ __forceinline__ u32x4 step(uint64_t at, int64_t k0, int64_t lim, int rows) const {
        if constexpr (COL) {
            const uint32_t n = static_cast<uint32_t>(lim < kBk ? lim : kBk);
            return descriptor(reinterpret_cast<const void*>(at + k0 * ld2),
                              (n - 1) * ld2 + 2 * static_cast<uint32_t>(left < B ? left : B));
        } else {
            const uint32_t n = static_cast<uint32_t>(left < rows ? left : rows);
            return descriptor(reinterpret_cast<const void*>(at + 2 * k0),
                              (n - 1) * ld2 + 2 * static_cast<uint32_t>(lim < kBk ? lim : kBk));
        }
    }
    __device__ __forceinline__ void load(int i, uint32_t lds, int wave, u32x4 desc) const {
        load_lds16(lds + (wave * N + i) * 1024, voff[i], desc);
    }
};

// Fragments of 32 output rows from `row0` on, for the 16 K values of slice kk:
// lane l holds row l % 32, K 8 (l / 32) .. + 7.
template <int B, bool COL, int NF>
struct Frags {
    uint32_t off[COL ? NF : kBk / 16];
    __device__ __forceinline__ void init(int row0) {
        const int l = lane_id();
        if constexpr (COL) {
            const int g = l >> 4, r = l & 15, row = 8 * (g >> 1) + (r >> 2);
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                const int col = row0 + 32 * f + 16 * (g & 1) + 4 * (r & 3);
                off[f] = 2 * (row * B + (((col >> 3) ^ columns_swizzle<B / 8>(row)) << 3) + (col & 7));
            }
        } else {
            const int r = l & 31, h = l >> 5;
#pragma unroll
            for (int kk = 0; kk < kBk / 16; ++kk) off[kk] = 2 * ((row0 + r) * kBk + (((2 * kk + h) ^ rows_swizzle(r)) << 3));
        }
    }
    __device__ __forceinline__ bf16x8 read(uint32_t tile, int kk, int f) const {
        if constexpr (COL) {
            const uint32_t at = tile + off[f] + 32 * kk * B;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at));
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at + 8 * B));
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            return __builtin_bit_cast(bf16x8, *(__attribute__((address_space(3))) const u32x4*)(tile + off[kk] + 64 * f * kBk));
        }
    }
};

constexpr float kLog2E = 1.4426950408889634f;
__device__ __forceinline__ float sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2E * x));
}
// act(g), and its derivative.  The hardware's exponential and reciprocal are
// good to an ulp, far below the bfloat16 that the results are rounded to.
__device__ __forceinline__ float activate(int act, float g) {
    if (act == ACT_SILU) return g * sigmoid(g);
    if (act == ACT_GELU) return 0.5f * g * (1.0f + erff(g * 0.70710678118654752f));
    // (1 + tanh v) / 2 = sigmoid(2 v)
    if (act == ACT_GELU_TANH) return g * sigmoid(1.5957691216057308f * g * fmaf(0.044715f * g, g, 1.0f));
    return g < 0.0f ? 0.0f : g;
}
__device__ __forceinline__ void activate_both(int act, float g, float& a, float& da) {
    if (act == ACT_SILU) {
        const float s = sigmoid(g);
        a = g * s;
        da = fmaf(a, 1.0f - s, s);
    } else if (act == ACT_GELU) {
        const float c = 0.5f * (1.0f + erff(g * 0.70710678118654752f));
        a = g * c;
        da = fmaf(g * 0.3989422804014327f, __builtin_amdgcn_exp2f(-0.5f * kLog2E * g * g), c);
    } else if (act == ACT_GELU_TANH) {
        const float s = sigmoid(1.5957691216057308f * g * fmaf(0.044715f * g, g, 1.0f));
        a = g * s;
        da = fmaf(a * (1.0f - s), 1.5957691216057308f * fmaf(0.134145f * g, g, 1.0f), s);
    } else {
        a = g < 0.0f ? 0.0f : g;
        da = g > 0.0f ? 1.0f : 0.0f;
    }
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
// Results 8 t .. 8 t + 7 of a fragment as the 8 consecutive columns 16 t + 8
// half .. + 7: the halves of the wave swap runs of 4.
__device__ __forceinline__ void columns8(const f32x16& c, int t, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(c[8 * t + i]), __float_as_uint(c[8 * t + 4 + i]), false, false);
        v[i] = __uint_as_float(r[0]);
        v[4 + i] = __uint_as_float(r[1]);
    }
}

template <int KIND, int BM, int BN, int WGM, int WGN>
__global__ __launch_bounds__(64 * WGM * WGN) void k_ffn(const FfnGemm g) {
    constexpr bool PT = KIND == FFN_WEIGHTS, QT = KIND == FFN_HIDDEN || KIND == FFN_INPUT || KIND == FFN_WEIGHTS;
    constexpr bool GATED = KIND == FFN_GATED;
    constexpr int NW = WGM * WGN, WTM = BM / WGM, WTN = BN / WGN, FM = WTM / 32, FN = WTN / 32;
    static_assert(!GATED || FN % 2 == 0, "a wave holds the gate and up columns of the same h");
    using P = Operand<BM, PT, NW>;
    using Q = Operand<BN, QT, NW>;
    static_assert(!GATED || 32 % (Q::N * Q::RPI) == 0, "a wave loads rows of one matrix");
    constexpr int STAGE = P::BYTES + Q::BYTES;
    __shared__ __attribute__((aligned(1024))) char lds_mem[2 * STAGE];
    const uint32_t lds = lds_addr(lds_mem);

    // ---- which split, segment and tile
    const int place = xcd_place(static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
    const int split = place / g.tiles, tile = place - split * g.tiles;
    int si = 0;
#pragma unroll
    for (int i = 1; i < 3; ++i)
        if (i < g.nseg && tile >= g.seg[i].first) si = i;
    const FfnSeg& seg = g.seg[si];
    const int t = tile - seg.first, per_band = g.band * seg.tiles_n, band = t / per_band, first_row = band * g.band;
    const int band_rows = seg.tiles_m - first_row < g.band ? seg.tiles_m - first_row : g.band;
    const int in_band = t - band * per_band;
    const int ti = first_row + in_band % band_rows, tj = in_band / band_rows;
    constexpr int BNO = GATED ? BN / 2 : BN;  // output columns of a tile
    const int64_t i0 = static_cast<int64_t>(ti) * BM, j0 = static_cast<int64_t>(tj) * BNO;
    const int lane = lane_id(), wave = attn::wave_id(), wm = wave / WGN, wn = wave % WGN;

    // ---- operands.  FFN_GATED: rows of a wave's columns alternate between 32
    // of the gate matrix and the same 32 of the up matrix.
    P p;
    Q q;
    p.init(seg.p[0], seg.ldp, i0, seg.m, wave, [](int r) { return r; });
    const bool up_rows = GATED && (wave * Q::N * Q::RPI / 32) & 1;
    q.init(up_rows ? seg.q[1] : seg.q[0], seg.ldq, j0, seg.n, wave,
           [](int r) { return GATED ? r / 64 * 32 + r % 32 : r; });
    const uint64_t p_next = KIND == FFN_INPUT ? p.base + (reinterpret_cast<uint64_t>(seg.p[1]) - reinterpret_cast<uint64_t>(seg.p[0])) : p.base;
    const uint64_t q_next = KIND == FFN_INPUT ? q.base + (reinterpret_cast<uint64_t>(seg.q[1]) - reinterpret_cast<uint64_t>(seg.q[0])) : q.base;

    const int phase_steps = static_cast<int>((g.k + kBk - 1) / kBk), steps = phase_steps * g.phases;
    const int s0 = split * g.split_steps, s1 = s0 + g.split_steps < steps ? s0 + g.split_steps : steps;
    u32x4 dp, dq;
    auto aim = [&](int s) {  // the loads of step s
        const bool second = KIND == FFN_INPUT && s >= phase_steps;
        const int64_t k0 = static_cast<int64_t>(second ? s - phase_steps : s) * kBk, lim = g.k - k0;
        p.limit(lim, wave);
        q.limit(lim, wave);
        dp = p.step(second ? p_next : p.base, k0, lim, BM);
        dq = q.step(second ? q_next : q.base, k0, lim, BNO);
    };
    auto load = [&](int L, uint32_t stage) {
        if (L < P::N) p.load(L, stage, wave, dp);
        else q.load(L - P::N, stage + P::BYTES, wave, dq);
    };
    Frags<BM, PT, FM> fp;
    Frags<BN, QT, FN> fq;
    fp.init(wm * WTM);
    fq.init(wn * WTN);

    f32x16 acc[FM][FN];
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
        for (int n = 0; n < FN; ++n) acc[m][n] = attn::splat(0.0f);

    constexpr int NL = P::N + Q::N, NKK = kBk / 16, NMF = FM * FN, NR = FM + FN, TOT = NKK * NMF;
    constexpr int RWIN = NMF * 3 / 4 > 0 ? NMF * 3 / 4 : 1, LWIN = TOT / 2;
    if (s0 < s1) {
        aim(s0);
#pragma unroll
        for (int L = 0; L < NL; ++L) load(L, lds);
    }
    for (int s = s0; s < s1; ++s) {
        landed();
        const uint32_t here = lds + ((s - s0) & 1) * STAGE, there = lds + ((s - s0 + 1) & 1) * STAGE;
        const bool more = s + 1 < s1;
        if (more) aim(s + 1);
        bf16x8 a[2][FM], b[2][FN];
#pragma unroll
        for (int m = 0; m < FM; ++m) a[0][m] = fp.read(here, 0, m);
#pragma unroll
        for (int n = 0; n < FN; ++n) b[0][n] = fq.read(here + P::BYTES, 0, n);
        // products of slice kk, with the reads of slice kk + 1 and the next
        // step's loads between them in this order
#pragma unroll
        for (int kk = 0; kk < NKK; ++kk) {
            const int c = kk & 1, o = c ^ 1;
#pragma unroll
            for (int i = 0; i < NMF; ++i) {
                in_order();
                acc[i / FN][i % FN] = mfma(b[c][i % FN], a[c][i / FN], acc[i / FN][i % FN]);
                in_order();
                if (kk + 1 < NKK) {
#pragma unroll
                    for (int r = 0; r < NR; ++r)
                        if (r * RWIN / NR == i) {
                            if (r < FM) a[o][r] = fp.read(here, kk + 1, r);
                            else b[o][r - FM] = fq.read(here + P::BYTES, kk + 1, r - FM);
                        }
                }
                if (more) {
#pragma unroll
                    for (int L = 0; L < NL; ++L)
                        if (L * LWIN / NL == kk * NMF + i) load(L, there);
                }
            }
        }
        in_order();
    }

    // ---- results: lane l holds row l % 32 of a fragment
    const int half = lane >> 5;
    const int64_t row0 = i0 + wm * WTM + (lane & 31);
    if constexpr (GATED) {
#pragma unroll
        for (int m = 0; m < FM; ++m) {
            const int64_t row = row0 + 32 * m;
#pragma unroll
            for (int n = 0; n < FN / 2; ++n)
#pragma unroll
                for (int t8 = 0; t8 < 2; ++t8) {
                    const int64_t col = j0 + wn * (WTN / 2) + 32 * n + 16 * t8 + 8 * half;
                    float gt[8], up[8], h[8];
                    columns8(acc[m][2 * n], t8, gt);
                    columns8(acc[m][2 * n + 1], t8, up);
#pragma unroll
                    for (int i = 0; i < 8; ++i) h[i] = activate(g.act, gt[i]) * up[i];
                    if (row < seg.m && col < seg.n) {
                        const int64_t at = row * seg.n + col;
                        *reinterpret_cast<u32x4*>(static_cast<bf16_t*>(seg.out) + at) = pack8(h);
                        if (g.gate) {
                            *reinterpret_cast<u32x4*>(g.gate + at) = pack8(gt);
                            *reinterpret_cast<u32x4*>(g.up + at) = pack8(up);
                        }
                    }
                }
        }
    } else if constexpr (KIND == FFN_HIDDEN) {
#pragma unroll
        for (int m = 0; m < FM; ++m) {
            const int64_t row = row0 + 32 * m;
#pragma unroll
            for (int n = 0; n < FN; ++n)
#pragma unroll
                for (int t8 = 0; t8 < 2; ++t8) {
                    const int64_t col = j0 + wn * WTN + 32 * n + 16 * t8 + 8 * half;
                    float dh[8], gt[8], up[8];
                    columns8(acc[m][n], t8, dh);
                    if (row < seg.m && col < seg.n) {
                        const int64_t at = row * seg.n + col;
                        spread8(*reinterpret_cast<const u32x4*>(g.gate + at), gt);
                        spread8(*reinterpret_cast<const u32x4*>(g.up + at), up);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float v, dv;
                            activate_both(g.act, gt[i], v, dv);
                            gt[i] = dh[i] * up[i] * dv;
                            up[i] = dh[i] * v;
                        }
                        *reinterpret_cast<u32x4*>(g.dgate + at) = pack8(gt);
                        *reinterpret_cast<u32x4*>(g.dup + at) = pack8(up);
                    }
                }
        }
    } else {
        float* part = seg.part ? seg.part + static_cast<int64_t>(split) * seg.m * seg.n : nullptr;
#pragma unroll
        for (int m = 0; m < FM; ++m) {
            const int64_t row = row0 + 32 * m;
#pragma unroll
            for (int n = 0; n < FN; ++n)
#pragma unroll
                for (int t8 = 0; t8 < 2; ++t8) {
                    const int64_t col = j0 + wn * WTN + 32 * n + 16 * t8 + 8 * half;
                    float v[8];
                    columns8(acc[m][n], t8, v);
                    if (row < seg.m && col < seg.n) {
                        const int64_t at = row * seg.n + col;
                        if (part || g.out_f32) {
                            float* o = (part ? part : static_cast<float*>(seg.out)) + at;
                            reinterpret_cast<f32x4*>(o)[0] = f32x4{v[0], v[1], v[2], v[3]};
                            reinterpret_cast<f32x4*>(o)[1] = f32x4{v[4], v[5], v[6], v[7]};
                        } else {
                            *reinterpret_cast<u32x4*>(static_cast<bf16_t*>(seg.out) + at) = pack8(v);
                        }
                    }
                }
        }
    }
}

// Sums of the splits, in their order: 8 values a thread.
__global__ __launch_bounds__(256) void k_ffn_join(const FfnGemm g) {
    const FfnSeg& seg = g.seg[blockIdx.y];
    const int64_t n = static_cast<int64_t>(seg.m) * seg.n, at = 8 * (static_cast<int64_t>(block_place()) * 256 + threadIdx.x);
    if (at >= n) return;
    float v[8] = {};
    for (int s = 0; s < g.splits; ++s) {
        const f32x4* src = reinterpret_cast<const f32x4*>(seg.part + s * n + at);
        const f32x4 lo = src[0], hi = src[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] += lo[i];
            v[4 + i] += hi[i];
        }
    }
    if (g.out_f32) {
        f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(seg.out) + at);
        o[0] = f32x4{v[0], v[1], v[2], v[3]};
        o[1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
        *reinterpret_cast<u32x4*>(static_cast<bf16_t*>(seg.out) + at) = pack8(v);
    }
}

template <int KIND>
void start(int tile, const FfnGemm& g, hipStream_t stream) {
    const uint32_t blocks = static_cast<uint32_t>(g.tiles) * g.splits;
    if (tile == 256) k_ffn<KIND, 256, 256, 2, 4><<<blocks, 512, 0, stream>>>(g);
    else k_ffn<KIND, 128, 128, 2, 2><<<blocks, 256, 0, stream>>>(g);
}

}  // namespace

hipError_t launch_ffn(FfnKind kind, int tile, const FfnGemm& g, hipStream_t stream) {
    switch (kind) {
        case FFN_GATED: start<FFN_GATED>(tile, g, stream); break;
        case FFN_PLAIN: start<FFN_PLAIN>(tile, g, stream); break;
        case FFN_HIDDEN: start<FFN_HIDDEN>(tile, g, stream); break;
        case FFN_INPUT: start<FFN_INPUT>(tile, g, stream); break;
        case FFN_WEIGHTS: start<FFN_WEIGHTS>(tile, g, stream); break;
    }
    if (g.splits > 1) {
        int64_t most = 0;
        for (int i = 0; i < g.nseg; ++i) {
            const int64_t n = static_cast<int64_t>(g.seg[i].m) * g.seg[i].n;
            if (n > most) most = n;
        }
        k_ffn_join<<<long_grid((most / 8 + 255) / 256, 256, g.nseg), 256, 0, stream>>>(g);
    }
    return hipGetLastError();
}

}  // namespace muon
