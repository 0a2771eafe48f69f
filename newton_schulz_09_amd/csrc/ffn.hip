// The products of a gated feed-forward block and its gradients, in bfloat16 on
// the matrix cores with float32 sums:
//     gate = x Wg^T, up = x Wu^T, h = act(gate) up       (one kernel)
//     out = h Wd^T
//     dh = dout Wd, dgate = dh up act'(gate), dup = dh act(gate)  (one kernel)
//     dx = dgate Wg + dup Wu                              (one sum)
//     dWg = dgate^T x, dWu = dup^T x, dWd = dout^T h      (one launch)
//
// Bound by the matrix cores, and on this card by the power they draw, for many
// tokens.  One engine: a workgroup computes a 256 x 256 tile with 8 waves or a 128 x
// 128 tile with 4, from 16 x 16 x 32 products, the form that draws least.  K
// advances 64 at a time through LDS stages (three of P, two of Q) that direct
// loads fill.  Operands contiguous along K lie in LDS as rows of K and are read
// 16 bytes a lane; operands contiguous along the output lie as rows of output and
// are read with transposing reads, so nothing is ever transposed in memory.  Rows
// and columns past the matrices' ends come as zeros from the loads' bounds checks,
// so every size runs the same loop.  The matrix instruction takes Q first, so a
// lane holds 4 consecutive columns of one output row.
//
// Measured (averages of 12 calls; after a pause the third to tenth take up to 40% longer
// than those from the thirtieth on): prefill of
// 4001 tokens, 4096 to 10240: gate and up 623 us, down 293 (1.08 and 1.15 PFLOP/s; a
// library's product of 8192^3 1.1 to 1.4).  GPT-2 124M batch, 65536 tokens, 768 to 2048:
// gate and up 515 us (0.80 PFLOP/s: 12 steps a tile, then 805 MB of results), down 205
// (1.0), gradients of the hidden values 410 (206 GFLOP, 1.1 GB), of x 398 (1.04), of
// the matrices 588 and 24 for the sums over 7 splits (1.01).
#include "../../include/muon.h"
#include "ffn_common.hpp"

namespace muon {

namespace {

using attn::descriptor;
using attn::each;
using attn::in_order;
using attn::landed;
using attn::lane_id;
using attn::lds_addr;
using attn::load_lds16;
using attn::s16x4;
using namespace ffn;

constexpr int kXcds = 8;
constexpr int BK = kFfnStep;
constexpr uint32_t kOut = 0x80000000u;  // an offset past every buffer's end

// Workgroup b of n -> place, so that each XCD (workgroups b = x, x + 8, ...)
// takes one contiguous range.
__device__ __forceinline__ int xcd_place(int b, int n) {
    const int q = n / kXcds, r = n % kXcds, x = b % kXcds;
    return x * q + (x < r ? x : r) + b / kXcds;
}

// Slot of 16-byte chunk c of row r is c ^ f(r).  Rows of K (8 chunks): 16 rows of
// one chunk fall on distinct banks.
__device__ __forceinline__ int rows_swizzle(int r) { return ((r >> 1) ^ (r << 2)) & 7; }
// Rows of output (16 or 32 chunks): the 8 rows that half a transposing read
// touches (two runs of 4, 8 apart) fall on distinct banks.
__device__ __forceinline__ int columns_swizzle(int r) { return (((r & 3) << 1) | ((r >> 3) & 1)) * 2; }

// One operand's tile: B output rows (or columns) by BK of K, COL: contiguous
// along the output.  NW waves load it, N loads of 1 KB a wave.
template <int B, bool COL, int NW>
struct Operand {
    static constexpr int CPR = COL ? B / 8 : BK / 8;
    static constexpr int RPI = 64 / CPR;  // rows per load
    static constexpr int LROWS = COL ? BK : B;
    static constexpr int N = LROWS / RPI / NW;
    static constexpr int BYTES = B * BK * 2;
    static_assert(N * RPI * NW == LROWS, "whole loads per wave");
    uint32_t voff[N];
    uint64_t base;     // of the tile, at K = 0
    uint32_t ld2;      // bytes between rows
    int left;          // output rows (columns) from here to the end
    bool masked;

    __device__ __forceinline__ static int row_of(int wave, int i) { return (wave * N + i) * RPI + lane_id() / CPR; }
    __device__ __forceinline__ static int chunk_of(int row) {
        return (lane_id() % CPR) ^ (COL ? columns_swizzle(row) : rows_swizzle(row));
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
            if (lim >= BK && !masked) return;
            masked = lim < BK;
#pragma unroll
            for (int i = 0; i < N; ++i)
                voff[i] = 8 * chunk_of(row_of(wave, i)) >= lim ? voff[i] | kOut : voff[i] & ~kOut;
        }
    }
    // Descriptor of the step from K = k0 on, lim = K - k0 > 0; rows: output rows of the tile
    __device__ __forceinline__ u32x4 step(uint64_t at, int64_t k0, int64_t lim, int rows) const {
        if constexpr (COL) {
            const uint32_t n = static_cast<uint32_t>(lim < BK ? lim : BK);
            return descriptor(reinterpret_cast<const void*>(at + k0 * ld2),
                              (n - 1) * ld2 + 2 * static_cast<uint32_t>(left < B ? left : B));
        } else {
            const uint32_t n = static_cast<uint32_t>(left < rows ? left : rows);
            return descriptor(reinterpret_cast<const void*>(at + 2 * k0),
                              (n - 1) * ld2 + 2 * static_cast<uint32_t>(lim < BK ? lim : BK));
        }
    }
    // The next step's, where that is a whole one of the same product.
    __device__ __forceinline__ void advance(u32x4& d) const {
        const uint64_t at = (static_cast<uint64_t>(d.y) << 32 | d.x) + (COL ? static_cast<uint64_t>(BK) * ld2 : 2 * BK);
        d.x = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(at)));
        d.y = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(at >> 32)));
    }
    __device__ __forceinline__ void load(int i, uint32_t lds, int wave, u32x4 desc) const {
        load_lds16(lds + (wave * N + i) * 1024, voff[i], desc);
    }
};

// Fragments of 16 output rows, f of them from `row0` on, for the 32 K values of
// slice kk: lane l holds row l % 16, K 8 (l / 16) .. + 7.
template <int B, bool COL>
struct Frags {
    uint32_t off;
    __device__ __forceinline__ void init(int row0) {
        const int l = lane_id(), g = l >> 4, r = l & 15;
        if constexpr (COL) {
            // transposing reads: lane r of 16 points at K r / 4 and 4 columns
            const int row = 8 * g + (r >> 2), col = row0 + 4 * (r & 3);
            off = 2 * (row * B + (((col >> 3) ^ columns_swizzle(row)) << 3) + (col & 7));
        } else {
            off = 2 * ((row0 + r) * BK + ((g ^ rows_swizzle(r)) << 3));
        }
    }
    // (the fragment's number, and of rows of K the slice's, are bits of the
    // chunk apart from those of row0: they go in by exclusive or, as the swizzle does)
    template <int KK, int F>
    __device__ __forceinline__ bf16x8 read(uint32_t tile) const {
        if constexpr (COL) {
            const uint32_t at = ((tile + off) ^ (32 * F)) + 64 * KK * B;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at));
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at + 8 * B));
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            return __builtin_bit_cast(bf16x8, *(__attribute__((address_space(3))) const u32x4*)(((tile + off) ^ (64 * KK)) + 32 * F * BK));
        }
    }
};

// This wave's loads have landed but for the last N, and its LDS reads are done,
// and so for every wave of the workgroup.
template <int N>
__device__ __forceinline__ void landed_but() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Segment, tile row and tile column of a launch's tile.
__device__ __forceinline__ void locate(const FfnGemm& g, int tile, int& si, int& ti, int& tj) {
    si = 0;
#pragma unroll
    for (int i = 1; i < 3; ++i)
        if (i < g.nseg && tile >= g.seg[i].first) si = i;
    const FfnSeg& seg = g.seg[si];
    const int t = tile - seg.first, per_band = seg.band * seg.tiles_n, band = t / per_band, first_row = band * seg.band;
    const int band_rows = seg.tiles_m - first_row < seg.band ? seg.tiles_m - first_row : seg.band;
    const int in_band = t - band * per_band;
    ti = first_row + in_band % band_rows;
    tj = in_band / band_rows;
}

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    reinterpret_cast<f32x4*>(p)[0] = f32x4{v[0], v[1], v[2], v[3]};
    reinterpret_cast<f32x4*>(p)[1] = f32x4{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void add8(const float* p, float (&v)[8]) {
    const f32x4 lo = reinterpret_cast<const f32x4*>(p)[0], hi = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] += lo[i];
        v[4 + i] += hi[i];
    }
}

// What becomes of 8 sums at element `at` of the output (`in`: inside it).
__device__ __forceinline__ void finish_plain(const FfnGemm& g, const FfnSeg& seg, int64_t at, const float (&v)[8]) {
    if (g.out_f32) store8(static_cast<float*>(seg.out) + at, v);
    else *reinterpret_cast<u32x4*>(static_cast<bf16_t*>(seg.out) + at) = pack8(v);
}
__device__ __forceinline__ void finish_gated(const FfnGemm& g, const FfnSeg& seg, int64_t at, bool in, const float (&gt)[8],
                                             const float (&up)[8]) {
    float h[8];
    by_act(g.act, [&](auto act) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v, unused;
            activate<act>(gt[i], v, unused);
            h[i] = v * up[i];
        }
    });
    if (!in) return;
    *reinterpret_cast<u32x4*>(static_cast<bf16_t*>(seg.out) + at) = pack8(h);
    if (g.gate) {
        *reinterpret_cast<u32x4*>(g.gate + at) = pack8(gt);
        *reinterpret_cast<u32x4*>(g.up + at) = pack8(up);
    }
}
__device__ __forceinline__ void finish_hidden(const FfnGemm& g, int64_t at, bool in, const float (&dh)[8], u32x4 gate, u32x4 up) {
    float gt[8], u[8];
    spread8(gate, gt);
    spread8(up, u);
    by_act(g.act, [&](auto act) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v, dv;
            activate<act>(gt[i], v, dv);
            gt[i] = dh[i] * u[i] * dv;
            u[i] = dh[i] * v;
        }
    });
    if (!in) return;
    *reinterpret_cast<u32x4*>(g.dgate + at) = pack8(gt);
    *reinterpret_cast<u32x4*>(g.dup + at) = pack8(u);
}

// ONE: K is one step (gradients of the matrices from up to 64 tokens), so the operands
// have a stage each and four workgroups fit a CU: 36 tokens of 3056 to 11600, 213 MB of
// gradients, 66 us with two workgroups and 50 with four.
template <int KIND, int BM, int BN, int WGM, int WGN, bool ONE = false>
__global__ __launch_bounds__(64 * WGM * WGN, ONE ? 4 : BM * BN / (WGM * WGN) > 8192 ? 1 : 2) void k_ffn(const FfnGemm g) {
    constexpr bool PT = KIND == FFN_WEIGHTS, QT = KIND == FFN_HIDDEN || KIND == FFN_INPUT || KIND == FFN_WEIGHTS;
    constexpr bool GATED = KIND == FFN_GATED;
    constexpr int NW = WGM * WGN, WTM = BM / WGM, WTN = BN / WGN, FM = WTM / 16, FN = WTN / 16;
    static_assert(!GATED || FN % 4 == 0, "a wave holds the gate and up columns of the same h");
    using P = Operand<BM, PT, NW>;
    using Q = Operand<BN, QT, NW>;
    static_assert(!GATED || 32 % Q::RPI == 0, "a load takes rows of one matrix");
    constexpr int STRIP = 32 * WTN * 4, QAT = (ONE ? 1 : 3) * P::BYTES, LDS = QAT + (ONE ? 1 : 2) * Q::BYTES;
    static_assert(NW * STRIP <= LDS, "the results pass through the stages' memory");
    __shared__ __attribute__((aligned(1024))) char lds_mem[LDS];
    const uint32_t lds = lds_addr(lds_mem);

    // ---- which split, segment and tile: workgroups of whole tiles, then those of
    // the tiles whose K is split
    const int b = static_cast<int>(blockIdx.x), tail = g.tiles - g.full;
    const bool whole = b < g.full;
    const int place = whole ? xcd_place(b, g.full) : xcd_place(b - g.full, tail * g.splits);
    const int split = whole ? 0 : place / tail, tile = whole ? place : g.full + place - split * tail;
    int si, ti, tj;
    locate(g, tile, si, ti, tj);
    const FfnSeg& seg = g.seg[si];
    constexpr int BNO = GATED ? BN / 2 : BN;  // output columns of a tile
    const int64_t i0 = static_cast<int64_t>(ti) * BM, j0 = static_cast<int64_t>(tj) * BNO;
    const int lane = lane_id(), wave = attn::wave_id(), wm = wave / WGN, wn = wave % WGN;

    // ---- operands.  FFN_GATED: rows of a wave's columns alternate between 32
    // of the gate matrix and the same 32 of the up matrix.
    P p;
    Q q;
    p.init(seg.p[0], seg.ldp, i0, seg.m, wave, [](int r) { return r; });
    q.init(seg.q[0], seg.ldq, j0, seg.n, wave,
           [](int r) { return GATED ? r / 64 * 32 + r % 32 : r; });
    const uint64_t p_next = KIND == FFN_INPUT ? p.base + (reinterpret_cast<uint64_t>(seg.p[1]) - reinterpret_cast<uint64_t>(seg.p[0])) : p.base;
    const uint64_t q_next = KIND == FFN_INPUT || GATED ? q.base + (reinterpret_cast<uint64_t>(seg.q[1]) - reinterpret_cast<uint64_t>(seg.q[0])) : q.base;

    const int phase_steps = static_cast<int>((g.k + BK - 1) / BK), steps = phase_steps * g.phases;
    const int s0 = split * g.split_steps, s1 = !whole && s0 + g.split_steps < steps ? s0 + g.split_steps : steps;
    u32x4 dp, dq, dq_up;
    // Aims the loads at step s, the one after the step they were aimed at.  Most
    // steps move the descriptors on; the first and last ones of a product make
    // them anew (made anew at every step they cost a tenth of the loop's time).
    auto plain = [&](int s) {
        return s > s0 && s != phase_steps - 1 && (KIND != FFN_INPUT || (s != phase_steps && s != 2 * phase_steps - 1));
    };
    auto place_of = [&](int s, bool& second, int64_t& k0) {
        second = KIND == FFN_INPUT && s >= phase_steps;
        k0 = static_cast<int64_t>(second ? s - phase_steps : s) * BK;
    };
    auto aim_p = [&](int s) {
        if (plain(s)) return p.advance(dp);
        bool second;
        int64_t k0;
        place_of(s, second, k0);
        p.limit(g.k - k0, wave);
        dp = p.step(second ? p_next : p.base, k0, g.k - k0, BM);
    };
    auto aim_q = [&](int s) {
        if (plain(s)) {
            if constexpr (GATED) q.advance(dq_up);
            return q.advance(dq);
        }
        bool second;
        int64_t k0;
        place_of(s, second, k0);
        q.limit(g.k - k0, wave);
        dq = q.step(second ? q_next : q.base, k0, g.k - k0, BNO);
        if constexpr (GATED) dq_up = q.step(q_next, k0, g.k - k0, BNO);
    };
    auto load_p = [&](int i, uint32_t to) { p.load(i, to, wave, dp); };
    auto load_q = [&](int i, uint32_t to) { q.load(i, to, wave, GATED && ((wave * Q::N + i) * Q::RPI / 32) & 1 ? dq_up : dq); };
    Frags<BM, PT> fp;
    Frags<BN, QT> fq;
    fp.init(wm * WTM);
    fq.init(wn * WTN);

    // A step is two slices of 32 K.  The operand of which a wave holds more
    // fragments is the outer one: each of its fragments meets all of the inner
    // operand's, and is then replaced by its successor of the next slice, so the
    // outer operand is held once and the inner twice.
    constexpr bool P_OUTER = FM >= FN;
    constexpr int NO = P_OUTER ? FM : FN, NI = P_OUTER ? FN : FM;
    f32x4 acc[NO][NI];
    each<0, NO>([&](auto o) { each<0, NI>([&](auto i) { acc[o][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f}; }); });
    bf16x8 outer[NO], inner[2][NI];
    auto read_outer = [&](auto kk, auto f, uint32_t p_tile, uint32_t q_tile) {
        if constexpr (P_OUTER) outer[f] = fp.template read<kk, f>(p_tile);
        else outer[f] = fq.template read<kk, f>(q_tile);
    };
    auto read_inner = [&](auto kk, auto f, uint32_t p_tile, uint32_t q_tile) {
        if constexpr (P_OUTER) inner[kk][f] = fq.template read<kk, f>(q_tile);
        else inner[kk][f] = fp.template read<kk, f>(p_tile);
    };

    // The barrier lies behind a quarter of the second slice, when the next step
    // has landed and every wave has read all of this one: the products before it
    // cover the last reads of this step, those behind it the first reads of the
    // next.  Loads are spread over the products (in a burst they fill the memory
    // pipe's queue, and the products behind them wait): those of P, which has
    // three stages, two steps early in the first slice, those of Q one step early
    // behind the barrier.
    constexpr int WAIT = NO / 4;  // groups of the second slice in front of the barrier
    static_assert(BK == 64 && NO >= 4, "two slices, four groups");
    constexpr std::integral_constant<int, 0> first{};
    constexpr std::integral_constant<int, 1> second{};
    if (s0 < s1) {
        aim_p(s0);
        each<0, P::N>([&](auto i) { load_p(i, lds); });
        aim_q(s0);
        each<0, Q::N>([&](auto i) { load_q(i, lds + QAT); });
        if (!ONE && s0 + 1 < s1) {
            aim_p(s0 + 1);
            each<0, P::N>([&](auto i) { load_p(i, lds + P::BYTES); });
            aim_q(s0 + 1);
            each<0, Q::N>([&](auto i) { load_q(i, lds + QAT + Q::BYTES); });
            landed_but<P::N + Q::N>();
        } else {
            landed();
        }
        each<0, NI>([&](auto i) { read_inner(first, i, lds, lds + QAT); });
        each<0, NO>([&](auto o) { read_outer(first, o, lds, lds + QAT); });
    }
    uint32_t p_here = lds, p_there = lds + P::BYTES, p_third = lds + 2 * P::BYTES;
    uint32_t q_here = lds + QAT, q_there = lds + QAT + Q::BYTES;
    for (int s = s0; s < s1; ++s) {
        const bool more = !ONE && s + 1 < s1, more2 = !ONE && s + 2 < s1;
        in_order();
        if (more2) aim_p(s + 2);
        each<0, 2>([&](auto kk) {
            each<0, NO>([&](auto o) {
                if constexpr (kk == 1 && o == WAIT) {
                    in_order();
                    if (more2) {
                        landed_but<P::N>();  // (P of two steps on is under way)
                        aim_q(s + 2);
                    } else {
                        landed();
                    }
                    if (more) each<0, WAIT>([&](auto f) { read_outer(first, f, p_there, q_there); });
                }
                each<0, NI>([&](auto i) {
                    in_order();
                    if constexpr (P_OUTER) acc[o][i] = mfma16(inner[kk][i], outer[o], acc[o][i]);
                    else acc[o][i] = mfma16(outer[o], inner[kk][i], acc[o][i]);
                });
                in_order();
                // the next slice's fragments
                if constexpr (kk == 0) {
                    read_outer(second, o, p_here, q_here);
                    each<0, NI>([&](auto i) {
                        if constexpr (i * NO / NI == o) read_inner(second, i, p_here, q_here);
                    });
                    if (more2)
                        each<0, P::N>([&](auto L) {
                            if constexpr (L * NO / P::N == o) load_p(L, p_third);
                        });
                } else if constexpr (o >= WAIT) {
                    if (more) {
                        read_outer(first, o, p_there, q_there);
                        each<0, NI>([&](auto i) {
                            if constexpr (WAIT + i * (NO - WAIT) / NI == o) read_inner(first, i, p_there, q_there);
                        });
                    }
                    if (more2)
                        each<0, Q::N>([&](auto L) {
                            if constexpr (WAIT + L * (NO - WAIT) / Q::N == o) load_q(L, q_here);
                        });
                }
            });
        });
        in_order();
        const uint32_t free = p_here;
        p_here = p_there;
        p_there = p_third;
        p_third = free;
        const uint32_t other = q_here;
        q_here = q_there;
        q_there = other;
    }

    // ---- results.  Lane l holds row l % 16 of a fragment, the 4 columns 4 (l / 16)
    // .. + 3.  Strips of 32 rows pass through LDS in float32, 16-byte chunk c
    // of row r at slot c ^ r, so that memory is read and written in whole rows of
    // a wave's columns, 8 columns a lane.
    constexpr int CH = WTN / 4, COLS = GATED ? WTN / 2 : WTN, LPR = COLS / 8, RPS = 64 / LPR;  // lanes a row, rows a turn
    const uint32_t strip = lds + wave * STRIP;
    const int64_t row0 = i0 + wm * WTM, col = j0 + wn * COLS + 8 * (lane % LPR);
    typedef __attribute__((address_space(3))) f32x4* Chunk;
    // of a split tile: its sums, as the tile lies (FFN_GATED: 32 columns of the gate
    // and of the up projection in turn)
    float* part = whole ? nullptr : g.part + (static_cast<int64_t>(split) * tail + (tile - g.full)) * (BM * BN) + wm * WTM * BN + wn * WTN;
    constexpr int TURNS = 32 / RPS;
    u32x4 gates[2][KIND == FFN_HIDDEN ? TURNS : 1][2];  // gate and up of this strip and the next, under way
    auto fetch = [&](auto m) {
        if constexpr (KIND == FFN_HIDDEN && m < WTM / 32) {
            if (part) return;
            each<0, TURNS>([&](auto k) {
                int64_t row = row0 + 32 * m + k * RPS + lane / LPR;
                if (row >= seg.m) row = seg.m - 1;
                const int64_t at = row * seg.n + (col < seg.n ? col : 0);
                gates[m & 1][k][0] = *reinterpret_cast<const u32x4*>(g.gate + at);
                gates[m & 1][k][1] = *reinterpret_cast<const u32x4*>(g.up + at);
            });
        }
    };
    fetch(first);
    // every wave has read its last fragments (no load to LDS is under way)
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    each<0, WTM / 32>([&](auto m) {
        fetch(std::integral_constant<int, m + 1>{});
        each<0, 2>([&](auto h) {
            each<0, FN>([&](auto n) {
                constexpr int o = P_OUTER ? 2 * m + h : n, i = P_OUTER ? n : 2 * m + h;
                const int r = 16 * h + (lane & 15), c = 4 * n + (lane >> 4);
                *(Chunk)(strip + r * WTN * 4 + ((c ^ r) & (CH - 1)) * 16) = acc[o][i];
            });
        });
        each<0, TURNS>([&](auto k) {
            const int r = k * RPS + lane / LPR;
            const int64_t row = row0 + 32 * m + r;
            auto take = [&](int c, float (&v)[8]) {  // chunks c and c + 1 of the row
                const f32x4 lo = *(Chunk)(strip + r * WTN * 4 + ((c ^ r) & (CH - 1)) * 16);
                const f32x4 hi = *(Chunk)(strip + r * WTN * 4 + (((c + 1) ^ r) & (CH - 1)) * 16);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = lo[i];
                    v[4 + i] = hi[i];
                }
            };
            const bool in = row < seg.m && col < seg.n;
            float* to = part + (32 * m + r) * BN;
            if constexpr (GATED) {
                // 32 columns of the gate, then the same 32 of the up projection
                const int q8 = lane % LPR, c = q8 / 4 * 16 + q8 % 4 * 2;
                float gt[8], up[8];
                take(c, gt);
                take(c + 8, up);
                if (part) {
                    if (in) {
                        store8(to + 4 * c, gt);
                        store8(to + 4 * c + 32, up);
                    }
                } else {
                    finish_gated(g, seg, row * seg.n + col, in, gt, up);
                }
            } else {
                float v[8];
                take(2 * (lane % LPR), v);
                if (part) {
                    if (in) store8(to + 8 * (lane % LPR), v);
                } else if constexpr (KIND == FFN_HIDDEN) {
                    finish_hidden(g, row * seg.n + col, in, v, gates[m & 1][k][0], gates[m & 1][k][1]);
                } else if (in) {
                    finish_plain(g, seg, row * seg.n + col, v);
                }
            }
        });
    });
}

// The results of the split tiles, from their sums added in the splits' order: 8
// columns a thread, a workgroup the BM BN / 2048 th part of a tile's columns.
template <int KIND, int B>
__global__ __launch_bounds__(256) void k_ffn_join(const FfnGemm g) {
    constexpr bool GATED = KIND == FFN_GATED;
    constexpr int BNO = GATED ? B / 2 : B, PER = B * BNO / 8 / 256;  // workgroups a tile
    const int tail = g.tiles - g.full, tt = blockIdx.x / PER;
    int si, ti, tj;
    locate(g, g.full + tt, si, ti, tj);
    const FfnSeg& seg = g.seg[si];
    const int at = (blockIdx.x % PER) * 256 + threadIdx.x, r = at / (BNO / 8), o = at % (BNO / 8) * 8;
    const int64_t row = static_cast<int64_t>(ti) * B + r, col = static_cast<int64_t>(tj) * BNO + o;
    if (row >= seg.m || col >= seg.n) return;
    const float* part = g.part + static_cast<int64_t>(tt) * (B * B) + r * B + (GATED ? o / 32 * 64 + o % 32 : o);
    float v[8] = {}, up[8] = {};
    for (int s = 0; s < g.splits; ++s, part += static_cast<int64_t>(tail) * (B * B)) {
        add8(part, v);
        if constexpr (GATED) add8(part + 32, up);
    }
    if constexpr (GATED) {
        finish_gated(g, seg, row * seg.n + col, true, v, up);
    } else if constexpr (KIND == FFN_HIDDEN) {
        const int64_t to = row * seg.n + col;
        finish_hidden(g, to, true, v, *reinterpret_cast<const u32x4*>(g.gate + to), *reinterpret_cast<const u32x4*>(g.up + to));
    } else {
        finish_plain(g, seg, row * seg.n + col, v);
    }
}

template <int KIND, int B>
void join(const FfnGemm& g, hipStream_t stream) {
    constexpr int PER = B * (KIND == FFN_GATED ? B / 2 : B) / 8 / 256;
    k_ffn_join<KIND, B><<<static_cast<uint32_t>(g.tiles - g.full) * PER, 256, 0, stream>>>(g);
}

template <int KIND>
void start(FfnTile tile, const FfnGemm& g, hipStream_t stream) {
    const uint32_t blocks = static_cast<uint32_t>(g.full + (g.tiles - g.full) * g.splits);
    // The gated product's waves hold 64 rows by 128 columns, so that each writes
    // rows of 64 hidden values; the others' 128 by 64.  (GPT-2 124M batch: gated
    // 500 us against 540, gradients of the matrices 565 us and 552.)
    constexpr int WGM = KIND == FFN_GATED ? 4 : 2;
    if (KIND == FFN_WEIGHTS && tile == FFN_128 && g.k <= BK) {
        k_ffn<FFN_WEIGHTS, 128, 128, 2, 2, true><<<blocks, 256, 0, stream>>>(g);
        return;
    }
    if (tile == FFN_256) k_ffn<KIND, 256, 256, WGM, 8 / WGM><<<blocks, 512, 0, stream>>>(g);
    else k_ffn<KIND, 128, 128, 2, 2><<<blocks, 256, 0, stream>>>(g);
    if (g.full == g.tiles) return;
    if (tile == FFN_256) join<KIND, 256>(g, stream);
    else join<KIND, 128>(g, stream);
}

}  // namespace

hipError_t launch_ffn(FfnKind kind, FfnTile tile, const FfnGemm& g, hipStream_t stream) {
    switch (kind) {
        case FFN_GATED: start<FFN_GATED>(tile, g, stream); break;
        case FFN_PLAIN: start<FFN_PLAIN>(tile, g, stream); break;
        case FFN_HIDDEN: start<FFN_HIDDEN>(tile, g, stream); break;
        case FFN_INPUT: start<FFN_INPUT>(tile, g, stream); break;
        case FFN_WEIGHTS: start<FFN_WEIGHTS>(tile, g, stream); break;
    }
    return hipGetLastError();
}

}  // namespace muon
