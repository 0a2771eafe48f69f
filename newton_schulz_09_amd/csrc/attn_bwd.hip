// Attention, backward, as two kernels without atomics (the sums have one
// order, so the gradients are the same bits every time): dQ with the keys
// walked per block of queries, then dK and dV with the queries walked per
// block of keys.  P is made again from the scores and lse; recomputing the
// two products S and dO V^T costs 7 products instead of 5.
//
// 16 x 1024 tokens of 12 heads of 64, causal: dQ 61 us, dK and dV 72.  By counters
// no pipe bounds them: of the cycles in which a CU holds waves (over 90 % of the
// kernel) the vector pipe is busy for 44 and 40 %, the matrix pipe for 34 and 38 %,
// LDS for 17 and 28 %; the rest are waits of two waves a SIMD for each other's
// steps.  One packed sequence of 16384 tokens, 6 heads of 128, capped scores,
// window 4096, documents: 190 and 224 us, vector 55 and 42 %, matrix 39 and 30 %,
// and CUs hold waves for 55 and 76 % of the kernel (blocks of unequal work).
// delta = sum dO O is taken from the bf16 O that the caller holds.
#include "attn_common.hpp"

namespace muon {

namespace {

using namespace attn;

// Result i of a block: s holds q . k, dp holds dO . v - delta; they become P
// and dS, with a cap a quarter of dS (dQ and dK are scaled by 4 at the end).
// term: what is subtracted from the scores in units of log 2, lse or with a
// cap up to kMaxPlainCap lse minus the cap; LSE: the products started from -lse,
// nothing is left to do.  With the cap's r = 1 / (exp(2 y) + 1): score = cap - 2
// cap r, derivative 4 (r - r^2), which is exact near zero too.
template <int MOD, bool LSE>
__device__ __forceinline__ void grad1(const Score& sc, f32x16& s, f32x16& dp, int i, float term, float dist) {
    float z, r = 0.0f;
    if constexpr (MOD & kWide) {
        z = capped<MOD>(sc, s[i], r) - term;
    } else if constexpr (MOD & kCap) {
        r = __builtin_amdgcn_rcpf(exp2_fast(s[i] * sc.c) + 1.0f);
        z = fmaf(-2.0f * sc.a, r, -term);
    } else {
        z = LSE && MOD == 0 ? s[i] * sc.c : fmaf(s[i], sc.c, -term);
    }
    if constexpr (MOD & kBias) z = fmaf(-sc.slope, dist, z);
    const float p = exp2_fast(z);
    float ds = p * dp[i];
    if constexpr (MOD & kCap) ds *= fmaf(-r, r, r);
    s[i] = p;
    dp[i] = ds;
}

// grad1's term of a row; +inf for one that saw nothing (its P is then zero).
template <int MOD>
__device__ __forceinline__ float row_term(float lse, const Score& sc) {
    if (lse == neg_inf()) return __builtin_inff();
    return (MOD & kCap) && !(MOD & kWide) ? fmaf(lse, kLog2e, -sc.a) : lse * kLog2e;
}
// The second kernel's: without extras -lse in units of the product q . k, where
// its products start.
template <int MOD>
__device__ __forceinline__ float start_term(float lse, const Score& sc, float scale) {
    if constexpr (MOD != 0) return row_term<MOD>(lse, sc);
    else return lse == neg_inf() ? neg_inf() : -lse / scale;
}
template <int MOD>
__device__ __forceinline__ float grad_scale(float scale) {
    return (MOD & kCap) ? 4.0f * scale : scale;
}

// dQ.  32 keys are one block; the gradients of the scores of a block are made
// in the shadow of products of the other block of the tile:
//     products   S, dP (0)   S, dP (1)   dQ (0)    dQ (1)
//     vector                 block 0     block 1
template <int DP, int NW, int MOD>
__global__ __launch_bounds__(64 * NW, 2) void k_attn_dq(const AttnArgs) {
    constexpr int BM = 32 * NW, NT = 64 * NW, TB = 2 * Tile<DP>::ELEMS;
    constexpr int ST = 2;  // one tile lands while the other is used (with three: 1 to 8 % slower)
    __shared__ __align__(16) bf16_t lds[ST][2][Tile<DP>::ELEMS];
    __shared__ __align__(16) int sdocs[ST][kTile];
    const Args a = arguments();
    const int H = a->b * a->hq, U = a->b * a->hkv;
    const int blocks = (a->sq + BM - 1) / BM;
    if (block_place() >= static_cast<uint32_t>(blocks) * H) return;
    const int blk = block_place(), e = blk % H;
    const int u = e % U, b = u / a->hkv, kvh = u % a->hkv, h = kvh * a->grp + e / U;
    const int i0 = (blocks - 1 - blk / H) * BM;
    const int i1 = i0 + BM < a->sq ? i0 + BM : a->sq;
    const Seq seq = sequence(a, b);
    const int w0 = i0 + wave_id() * 32, w1 = w0 + 32 < a->sq ? w0 + 32 : a->sq;
    Span g = query_span(seq, a, i0, i1), w = query_span(seq, a, w0, w1);

    Direct<DP, NT> lk, lv;
    lk.init(a->k + b * a->k_b + kvh * a->k_h, a->k_s, seq.n, a->d);
    lv.init(a->v + b * a->v_b + kvh * a->v_h, a->v_s, seq.n, a->d);
    const uint32_t at = lds_addr(lds);
    const int sk = a->sk;
    KeyTiles it;
    it.init(seq, a, g, w);
    in_vectors(g);
    in_vectors(w);
    int tile[ST], mode[ST];
    auto fetch = [&](int x) {
        tile[x] = it.next(seq, a, g, w, mode[x]);
        if (tile[x] < 0) return;
        lk.load(tile[x] * kTile, at + 2 * x * TB);
        lv.load(tile[x] * kTile, at + (2 * x + 1) * TB);
        if (seq.doc) load_values(seq.doc, tile[x] * kTile, sk, lds_addr(sdocs[x]));
    };
    fetch(0);

    const int i = w0 + (lane_id() & 31);
    const Row row = row_of(seq, a, seq.start + i);
    const bool real = i < a->sq && real_row(seq, a, seq.start + i);
    const Score sc = score_of<MOD>(a, h);
    bf16x8 qf[DP / 16], dof[DP / 16];
    load_rows<DP>(qf, a->q + b * a->q_b + h * a->q_h, a->q_s, i, real, a->d);
    load_rows<DP>(dof, a->dout + b * a->do_b + h * a->do_h, a->do_s, i, real, a->d);
    float delta = 0.0f;
    {
        bf16x8 of[DP / 16];
        load_rows<DP>(of, a->out + b * a->o_b + h * a->o_h, a->o_s, i, real, a->d);
#pragma unroll
        for (int t = 0; t < DP / 16; ++t)
#pragma unroll
            for (int c = 0; c < 8; ++c) delta = fmaf(static_cast<float>(dof[t][c]), static_cast<float>(of[t][c]), delta);
        delta = half_sum(delta);
    }
    const int64_t stat = (static_cast<int64_t>(b) * a->hq + h) * a->sq + i;
    const float given = real ? a->lse[stat] : neg_inf();
    const float term = row_term<MOD>(given, sc);
    if (i < a->sq && lane_id() < 32) {
        // for the second kernel: what it starts its products from
        a->stats[stat] = start_term<MOD>(given, sc, a->scale);
        a->stats[stat + a->delta_at] = -delta;
    }
    RowFrag<DP> rf;
    ColFrag<DP> cf;
    rf.init();
    cf.init();
    f32x16 dq[DP / 32];
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt) dq[dt] = splat(0.0f);
    settle(qf);
    settle(dof);

    constexpr int KT = DP / 16, DT = DP / 32, kAhead = 3;
    auto step = [&](uint32_t tk, uint32_t tv, bool masked, const int* sdoc, int k0) {
        const int h4 = 4 * (lane_id() >> 5);
        f32x16 s[2], dp[2];
        bf16x8 p[2][2], ring[kAhead];
        float dp0 = -delta;
        if constexpr (DP > 64) asm volatile("" : "+v"(dp0));  // (no room to keep its 16 copies between tiles)
        auto operand = [&](int y) {  // K and V along the row in turn, both blocks; then K across
            return y < 4 * KT ? rf.read(y % 2 ? tv : tk, y / (2 * KT), y % (2 * KT) / 2)
                              : cf.read(tk, (y - 4 * KT) / DT, (y - 4 * KT) % DT);
        };
        auto grads = [&](int kb, int i) {
            grad1<MOD, false>(sc, s[kb], dp[kb], i, term,
                       fabsf(static_cast<float>(row.pos - k0 - h4) - static_cast<float>(32 * kb + place(i))));
        };
        auto finish = [&](int kb) {
            if (masked) {
                const Bits m = keys_seen(row, seq, a, k0 + h4);
                each<0, 16>([&](auto i) { dp[kb][i.value] = where(m, kb, i.value, dp[kb][i.value], 0.0f); });
                if (sdoc)
                    each<0, 16>([&](auto i_) {
                        constexpr int i = decltype(i_)::value;
                        dp[kb][i] = sdoc[32 * kb + place(i) + h4] == row.doc ? dp[kb][i] : 0.0f;
                    });
            }
            p[kb][0] = pack(dp[kb], 0);
            p[kb][1] = pack(dp[kb], 1);
        };
        each<0, kAhead>([&](auto y) { ring[y] = operand(y); });
        in_order();
        each<0, 6 * KT>([&](auto y_) {
            constexpr int y = decltype(y_)::value;
            if constexpr (y < 4 * KT) {
                constexpr int kb = y / (2 * KT), t = y % (2 * KT) / 2;
                if constexpr (y % 2 == 0) s[kb] = mfma(ring[y % kAhead], qf[t], t == 0 ? splat(0.0f) : s[kb]);
                else dp[kb] = mfma(ring[y % kAhead], dof[t], t == 0 ? splat(dp0) : dp[kb]);
            } else {
                constexpr int x = y - 4 * KT, dt = x % DT, kb = x / (2 * DT), t = x / DT % 2;
                dq[dt] = mfma(ring[y % kAhead], p[kb][t], dq[dt]);
            }
            if constexpr (y + kAhead < 6 * KT) ring[y % kAhead] = operand(y + kAhead);
            if constexpr (y >= 2 * KT + 2 && y < 4 * KT) {
                constexpr int x = y - 2 * KT - 2, n = 2 * KT - 2;
                each<16 * x / n, 16 * (x + 1) / n>([&](auto i) { grads(0, i); });
            }
            if constexpr (y == 4 * KT - 1) finish(0);
            if constexpr (y >= 4 * KT && y < 5 * KT) {
                constexpr int x = y - 4 * KT;
                each<16 * x / KT, 16 * (x + 1) / KT>([&](auto i) { grads(1, i); });
            }
            if constexpr (y == 5 * KT - 1) finish(1);
            in_order();
        });
    };
    // (the two buffers' code side by side: as one loop, 3 to 25 % slower)
    for (;;) {
#pragma unroll
        for (int x = 0; x < ST; ++x) {
            if (tile[x] < 0) goto done;
            landed();
            fetch(1 - x);
            if (mode[x] != 0)
                step(at + 2 * x * TB, at + (2 * x + 1) * TB, mode[x] == 1, seq.doc ? sdocs[x] : nullptr, tile[x] * kTile);
        }
    }
done:
    const Args z = again(a);
    // dq is contiguous (b, sq, hq, d)
    store_rows<DP>(dq, grad_scale<MOD>(z->scale), z->dq + ((static_cast<int64_t>(b) * z->sq + i) * z->hq + h) * z->d, i < z->sq, z->d);
}

// dK and dV of 32 NW keys, walked over the queries of every head that shares
// them.  32 queries are one block of a tile; as above
//     products   S, dP (0)   S, dP (1)   dV, dK (0)   dV, dK (1)
//     vector                 block 0     block 1
// PAIR: two waves share 32 keys.  Each makes P and dS of one block of a tile
// and hands them to the other (they are operands as they lie, so the other's
// lanes read them back unchanged), and each sums half of the columns of dV and
// dK over both blocks: the same products, with half of the accumulators, so
// two waves fit on a SIMD (heads of 128: 440 registers, 240 as pairs).
template <int DP, int NW, bool PAIR, int MOD>
__global__ __launch_bounds__(64 * NW, DP == 64 || PAIR ? 2 : 1) void k_attn_dkv(const AttnArgs) {
    constexpr int BN = PAIR ? 16 * NW : 32 * NW, NT = 64 * NW, TB = 2 * Tile<DP>::ELEMS;
    static_assert(!PAIR || DP == 128, "halves of the columns differ in one address bit");
    constexpr int ST = 2;  // one tile lands while the other is used (with three: 1 to 8 % slower)
    __shared__ __align__(16) bf16_t lds[ST][2][Tile<DP>::ELEMS];
    __shared__ __align__(16) float sstat[ST][2][kTile];
    __shared__ __align__(16) int sdocs[ST][kTile];
    __shared__ __align__(16) bf16x8 handed[PAIR ? NW : 1][PAIR ? 4 : 1][64];
    const Args a = arguments();
    const int U = a->b * a->hkv;
    if (block_place() >= static_cast<uint32_t>((a->sk + BN - 1) / BN) * U) return;
    const int blk = block_place(), u = blk % U, b = u / a->hkv, kvh = u % a->hkv;
    const int j0 = blk / U * BN;
    Seq seq = sequence(a, b);
    const int lead = only_queries_that_see(seq, a);
    const int part = PAIR ? wave_id() & 1 : 0;
    const int w0 = j0 + (PAIR ? wave_id() >> 1 : wave_id()) * 32;
    auto key_span = [&](int lo, int hi) {
        Span r;
        r.p0 = lo;
        r.p1 = hi < seq.n ? hi - 1 : seq.n - 1;
        doc_range(seq, a, r.p0, r.p1, r.d0, r.d1);
        return r;
    };
    Span g = key_span(j0, j0 + BN), w = key_span(w0, w0 + 32);
    // whole blocks of real keys only: the rest is masked one by one
    const bool whole = w0 + 32 <= seq.n;
    const int j = w0 + (lane_id() & 31);
    const Col col = col_of(seq, a, j);
    bf16x8 kf[DP / 16], vf[DP / 16];
    load_rows<DP>(kf, a->k + b * a->k_b + kvh * a->k_h, a->k_s, j, j < seq.n, a->d);
    load_rows<DP>(vf, a->v + b * a->v_b + kvh * a->v_h, a->v_s, j, j < seq.n, a->d);

    // the tiles of all the heads that share the keys, one after the other
    QueryTiles it;
    it.init(seq, a, g, w);
    in_vectors(g);
    in_vectors(w);
    Direct<DP, NT> lq, ld;
    lq.init(a->q + b * a->q_b + static_cast<int64_t>(kvh) * a->grp * a->q_h + lead * a->q_s, a->q_s, it.rows, a->d);
    ld.init(a->dout + b * a->do_b + static_cast<int64_t>(kvh) * a->grp * a->do_h + lead * a->do_s, a->do_s, it.rows, a->d);
    const float* stat = a->stats + (static_cast<int64_t>(b) * a->hq + kvh * a->grp) * a->sq + lead;
    const uint32_t at = lds_addr(lds);
    int tile[ST], mode[ST], left = a->grp - 1;  // heads after the tiles' own
    Score sc[ST], head = score_of<MOD>(a, kvh * a->grp);
    auto fetch = [&](int x) {
        tile[x] = it.next(seq, a, g, w, mode[x]);
        if (tile[x] < 0 && left > 0) {
            const Args z = again(a);
            --left;
            it.init(seq, z, g, w);
            lq.base += z->q_h;
            ld.base += z->do_h;
            stat += z->sq;
            head = score_of<MOD>(z, kvh * z->grp + z->grp - 1 - left);
            tile[x] = it.next(seq, z, g, w, mode[x]);
        }
        sc[x] = head;
        if (tile[x] < 0) return;
        const int row0 = tile[x] * kTile;
        lq.load(row0, at + 2 * x * TB);
        ld.load(row0, at + (2 * x + 1) * TB);
        load_values(stat, row0, it.rows, lds_addr(sstat[x][0]));
        load_values(stat + again(a)->delta_at, row0, it.rows, lds_addr(sstat[x][1]));
        if (seq.doc) load_docs(seq.doc, seq.start + row0, again(a)->sk, lds_addr(sdocs[x]));
    };
    fetch(0);
    RowFrag<DP> rf;
    ColFrag<DP> cf;
    rf.init();
    cf.init();
    constexpr int OT = DP / 32 / (PAIR ? 2 : 1);  // this wave's 32 columns of dK and dV
    if constexpr (PAIR)
#pragma unroll
        for (int dt = 0; dt < OT; ++dt)
#pragma unroll
            for (int e = 0; e < 2; ++e) cf.off[dt][e] ^= DP * part;
    f32x16 dk[OT], dv[OT];
#pragma unroll
    for (int dt = 0; dt < OT; ++dt) dk[dt] = dv[dt] = splat(0.0f);
    settle(kf);
    settle(vf);

    constexpr int KT = DP / 16, DT = DP / 32, kAhead = DP == 64 ? 3 : 8;
    // (with a parameter of a template, so that it exists only where it is called)
    auto step = [&](auto, uint32_t tq, uint32_t td, const float* sl, const float* sdel, const int* sdoc, bool masked, const Score& score, int q0) {
        const int h4 = 4 * (lane_id() >> 5);
        f32x16 s[2], dp[2];
        bf16x8 pp[2][2], pd[2][2], ring[kAhead];
        auto operand = [&](int y) {  // Q and dO along the row in turn, both blocks; then dO and Q across
            return y < 4 * KT ? rf.read(y % 2 ? td : tq, y / (2 * KT), y % (2 * KT) / 2)
                              : cf.read(y % 2 ? tq : td, (y - 4 * KT) / 2 / DT, (y - 4 * KT) / 2 % DT);
        };
        auto starts = [&](int qb) {
            each<0, 16>([&](auto i_) {
                constexpr int i = decltype(i_)::value;
                const int r = 32 * qb + 8 * (i / 4) + h4 + i % 4;
                s[qb][i] = MOD ? 0.0f : sl[r];
                dp[qb][i] = sdel[r];
            });
        };
        auto grads = [&](int qb, int i) {
            const int r = 32 * qb + 8 * (i / 4) + i % 4;
            grad1<MOD, true>(score, s[qb], dp[qb], i, MOD ? sl[r + h4] : 0.0f,
                       fabsf(static_cast<float>(seq.start + q0 + h4 - col.pos) + static_cast<float>(r)));
        };
        auto finish = [&](int qb) {
            if (masked) {
                const int p0 = seq.start + q0 + h4;
                const Bits m = bits_of(col.lo - p0, col.hi - p0, 0);
                each<0, 16>([&](auto i) {
                    s[qb][i.value] = where(m, qb, i.value, s[qb][i.value], 0.0f);
                    dp[qb][i.value] = where(m, qb, i.value, dp[qb][i.value], 0.0f);
                });
                if (sdoc)
                    each<0, 16>([&](auto i_) {
                        constexpr int i = decltype(i_)::value;
                        const bool mine = sdoc[32 * qb + place(i) + h4] == col.doc;
                        s[qb][i] = mine ? s[qb][i] : 0.0f;
                        dp[qb][i] = mine ? dp[qb][i] : 0.0f;
                    });
            }
            pp[qb][0] = pack(s[qb], 0);
            pp[qb][1] = pack(s[qb], 1);
            pd[qb][0] = pack(dp[qb], 0);
            pd[qb][1] = pack(dp[qb], 1);
        };
        starts(0);
        each<0, kAhead>([&](auto y) { ring[y] = operand(y); });
        in_order();
        each<0, 8 * KT>([&](auto y_) {
            constexpr int y = decltype(y_)::value;
            if constexpr (y < 4 * KT) {
                constexpr int qb = y / (2 * KT), t = y % (2 * KT) / 2;
                if constexpr (y % 2 == 0) s[qb] = mfma(ring[y % kAhead], kf[t], s[qb]);
                else dp[qb] = mfma(ring[y % kAhead], vf[t], dp[qb]);
            } else {
                constexpr int x = (y - 4 * KT) / 2, dt = x % DT, qb = x / (2 * DT), t = x / DT % 2;
                if constexpr (y % 2 == 0) dv[dt] = mfma(ring[y % kAhead], pp[qb][t], dv[dt]);
                else dk[dt] = mfma(ring[y % kAhead], pd[qb][t], dk[dt]);
            }
            if constexpr (y + kAhead < 8 * KT) ring[y % kAhead] = operand(y + kAhead);
            if constexpr (y == KT) starts(1);
            if constexpr (y >= 2 * KT + 2 && y < 4 * KT) {
                constexpr int x = y - 2 * KT - 2, n = 2 * KT - 2;
                each<16 * x / n, 16 * (x + 1) / n>([&](auto i) { grads(0, i); });
            }
            if constexpr (y == 4 * KT - 1) finish(0);
            if constexpr (y >= 4 * KT + 1 && y < 6 * KT) {
                constexpr int x = y - 4 * KT - 1, n = 2 * KT - 1;
                each<16 * x / n, 16 * (x + 1) / n>([&](auto i) { grads(1, i); });
            }
            if constexpr (y == 6 * KT - 1) finish(1);
            in_order();
        });
    };
    auto share = [&](auto, uint32_t tq, uint32_t td, const float* sl, const float* sdel, const int* sdoc, int seen, const Score& score, int q0) {
        // this wave's block is `part`
        const int h4 = 4 * (lane_id() >> 5), r0 = 32 * part + h4;
        constexpr int kRing = 4;
        bf16x8 ring[kRing], p[4];
        auto across = [&](int y, int block) {  // dO and Q in turn, 2 steps of OT column tiles
            return cf.read((y % 2 ? tq : td) + 64 * block * Tile<DP>::LD, y / 2 / OT, y / 2 % OT);
        };
        auto products = [&](int block) {
            each<0, kRing>([&](auto y) { ring[y.value] = across(y.value, block); });
            in_order();
            each<0, 4 * OT>([&](auto y_) {
                constexpr int y = decltype(y_)::value, dt = y / 2 % OT, t = y / 2 / OT;
                if constexpr (y % 2 == 0) dv[dt] = mfma(ring[y % kRing], p[t], dv[dt]);
                else dk[dt] = mfma(ring[y % kRing], p[2 + t], dk[dt]);
                if constexpr (y + kRing < 4 * OT) ring[y % kRing] = across(y + kRing, block);
                in_order();
            });
        };
        if (seen) {
            f32x16 s, dp;
            each<0, 16>([&](auto i_) {
                constexpr int i = decltype(i_)::value;
                s[i] = MOD ? 0.0f : sl[r0 + place(i)];
                dp[i] = sdel[r0 + place(i)];
            });
            auto along = [&](int y) { return rf.read((y % 2 ? td : tq) + 64 * part * Tile<DP>::LD, 0, y / 2); };
            each<0, kRing>([&](auto y) { ring[y.value] = along(y.value); });
            in_order();
            each<0, 2 * KT>([&](auto y_) {
                constexpr int y = decltype(y_)::value;
                if constexpr (y % 2 == 0) s = mfma(ring[y % kRing], kf[y / 2], s);
                else dp = mfma(ring[y % kRing], vf[y / 2], dp);
                if constexpr (y + kRing < 2 * KT) ring[y % kRing] = along(y + kRing);
                in_order();
            });
            each<0, 16>([&](auto i_) {
                constexpr int i = decltype(i_)::value;
                grad1<MOD, true>(score, s, dp, i, MOD ? sl[r0 + place(i)] : 0.0f,
                                 fabsf(static_cast<float>(seq.start + q0 + r0 - col.pos) + static_cast<float>(place(i))));
            });
            if (seen == 1 || !whole) {
                const int p0 = seq.start + q0 + r0;
                const Bits m = bits_of(col.lo - p0, col.hi - p0, 0);
                each<0, 16>([&](auto i) {
                    s[i.value] = where(m, 0, i.value, s[i.value], 0.0f);
                    dp[i.value] = where(m, 0, i.value, dp[i.value], 0.0f);
                });
                if (sdoc)
                    each<0, 16>([&](auto i_) {
                        constexpr int i = decltype(i_)::value;
                        const bool mine = sdoc[r0 + place(i)] == col.doc;
                        s[i] = mine ? s[i] : 0.0f;
                        dp[i] = mine ? dp[i] : 0.0f;
                    });
            }
            p[0] = pack(s, 0);
            p[1] = pack(s, 1);
            p[2] = pack(dp, 0);
            p[3] = pack(dp, 1);
#pragma unroll
            for (int e = 0; e < 4; ++e) handed[wave_id()][e][lane_id()] = p[e];
            products(part);
        }
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (seen) {
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = handed[wave_id() ^ 1][e][lane_id()];
            products(1 - part);
        }
    };
    // (the two buffers' code side by side: as one loop, 3 to 25 % slower)
    for (;;) {
#pragma unroll
        for (int x = 0; x < ST; ++x) {
            if (tile[x] < 0) goto done;
            landed();
            fetch(1 - x);
            if constexpr (PAIR)
                share(0, at + 2 * x * TB, at + (2 * x + 1) * TB, sstat[x][0], sstat[x][1], seq.doc ? sdocs[x] : nullptr, mode[x], sc[x],
                      tile[x] * kTile);
            else if (mode[x] != 0)
                step(0, at + 2 * x * TB, at + (2 * x + 1) * TB, sstat[x][0], sstat[x][1], seq.doc ? sdocs[x] : nullptr, mode[x] == 1 || !whole, sc[x],
                     tile[x] * kTile);
        }
    }
done:
    const Args z = again(a);
    // dk and dv are contiguous (b, sk, hkv, d)
    const int64_t to = ((static_cast<int64_t>(b) * z->sk + j) * z->hkv + kvh) * z->d;
    store_rows<32 * OT>(dk, grad_scale<MOD>(z->scale), z->dk + to + 32 * OT * part, j < z->sk, z->d - 32 * OT * part);
    store_rows<32 * OT>(dv, 1.0f, z->dv + to + 32 * OT * part, j < z->sk, z->d - 32 * OT * part);
}

template <int DP, int MOD>
void dq(const AttnArgs& a, hipStream_t stream) {
    constexpr int NW = 4, BM = 32 * NW;
    const int64_t blocks = static_cast<int64_t>((a.sq + BM - 1) / BM) * a.b * a.hq;
    k_attn_dq<DP, NW, MOD><<<long_grid(blocks, 64 * NW), 64 * NW, 0, stream>>>(a);
}
template <int DP, int MOD>
void dkv(const AttnArgs& a, hipStream_t stream) {
    constexpr int BN = 128;
    const int64_t blocks = static_cast<int64_t>((a.sk + BN - 1) / BN) * a.b * a.hkv;
    // pairs where the cap makes the vector work long enough to hide the
    // handing over: capped documents of 16384 tokens 258 -> 232 us, capped 2 x
    // 2048 tokens of 12 heads (both kernels) 160 -> 155; without a cap 16 x 1024
    // tokens of 6 heads 151 -> 159, 4 x 4096 of 16 heads over 4 945 -> 975
    if constexpr (DP == 128 && (MOD & kCap) != 0) k_attn_dkv<DP, 8, true, MOD><<<long_grid(blocks, 512), 512, 0, stream>>>(a);
    else k_attn_dkv<DP, 4, false, MOD><<<long_grid(blocks, 256), 256, 0, stream>>>(a);
}

}  // namespace

hipError_t launch_attn_bwd_dq(const AttnArgs& a, hipStream_t stream) {
    MUON_ATTN_DISPATCH(dq, a, stream);
    return hipGetLastError();
}

hipError_t launch_attn_bwd_dkv(const AttnArgs& a, hipStream_t stream) {
    MUON_ATTN_DISPATCH(dkv, a, stream);
    return hipGetLastError();
}

}  // namespace muon
