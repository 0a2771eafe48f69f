// Attention, backward, as two kernels without atomics (the sums have one
// order, so the gradients are the same bits every time): dQ with the keys
// walked per block of queries, then dK and dV with the queries walked per
// block of keys.  P is made again from the scores and lse; recomputing the
// two products S and dO V^T costs 7 products instead of 5.
#include <type_traits>

#include "attn_common.hpp"

namespace muon {

namespace {

using namespace attn;

// p and dS of 16 results: s holds q . k, dp holds dO . v - delta.  lse2 in
// units of log 2.
template <int MOD>
__device__ __forceinline__ void grad1(const Score& sc, f32x16& s, f32x16& dp, int i, float lse2, float dist) {
    float r = 0.0f;
    const float p = exp2_fast(MOD ? score<MOD>(sc, s[i], dist, r) - lse2 : fmaf(s[i], sc.c, -lse2));
    float ds = p * dp[i];
    if constexpr (MOD & kCap) ds *= 4.0f * fmaf(-r, r, r);
    s[i] = p;
    dp[i] = ds;
}

// The row statistic the kernels subtract: a row that saw nothing has lse
// -inf, and +inf makes its P zero.
__device__ __forceinline__ float lse2_of(float lse) { return lse == neg_inf() ? __builtin_inff() : lse * kLog2e; }

template <int DP, int QB, int NW, int MOD>
__global__ __launch_bounds__(64 * NW, QB == 1 ? 2 : 1) void k_attn_dq(const AttnArgs a) {
    constexpr int BM = 32 * QB * NW, NT = 64 * NW;
    __shared__ __align__(16) bf16_t lds[2][2][Tile<DP>::ELEMS];
    __shared__ __align__(16) int sdocs[2][kTile];
    const int H = a.b * a.hq, U = a.b * a.hkv;
    const int blk = blockIdx.x, e = blk % H;
    const int u = e % U, b = u / a.hkv, kvh = u % a.hkv, h = kvh * a.grp + e / U;
    const int i0 = ((gridDim.x / H) - 1 - blk / H) * BM;
    const int i1 = i0 + BM < a.sq ? i0 + BM : a.sq;
    const Seq seq = sequence(a, b);
    const int w0 = i0 + wave_id() * 32 * QB, w1 = w0 + 32 * QB < a.sq ? w0 + 32 * QB : a.sq;
    const Span g = query_span(seq, a, i0, i1), w = query_span(seq, a, w0, w1);
    const int2* docs = a.doc_tiles + static_cast<int64_t>(b) * a.n_tiles;

    bf16x8 qf[QB][DP / 16], dof[QB][DP / 16];
    Row row[QB];
    float lse2[QB], delta[QB];
    const Score sc = score_of<MOD>(a, h);
#pragma unroll
    for (int x = 0; x < QB; ++x) {
        const int i = w0 + 32 * x + (lane_id() & 31);
        row[x] = row_of(seq, a, seq.start + i);
        const bool ok = i < a.sq && real_row(seq, a, seq.start + i);
        load_rows<DP>(qf[x], a.q + b * a.q_b + h * a.q_h, a.q_s, i, ok, a.d);
        load_rows<DP>(dof[x], a.dout + b * a.do_b + h * a.do_h, a.do_s, i, ok, a.d);
        bf16x8 of[DP / 16];
        load_rows<DP>(of, a.out + b * a.o_b + h * a.o_h, a.o_s, i, ok, a.d);
        float sum = 0.0f;
#pragma unroll
        for (int t = 0; t < DP / 16; ++t)
#pragma unroll
            for (int c = 0; c < 8; ++c)
                sum = fmaf(static_cast<float>(dof[x][t][c]), static_cast<float>(of[t][c]), sum);
        delta[x] = half_sum(sum);
        const int64_t at = (static_cast<int64_t>(b) * a.hq + h) * a.sq + i;
        lse2[x] = ok ? lse2_of(a.lse[at]) : __builtin_inff();
        if (i < a.sq && lane_id() < 32) a.delta[at] = delta[x];
    }
    Loader<DP, NT> lk, lv;
    lk.init(a.k + b * a.k_b + kvh * a.k_h, a.k_s, seq.n, a.d);
    lv.init(a.v + b * a.v_b + kvh * a.v_h, a.v_s, seq.n, a.d);
    RowFrag<DP> rf;
    ColFrag<DP> cf;
    rf.init();
    cf.init();
    f32x16 dq[QB][DP / 32];
#pragma unroll
    for (int x = 0; x < QB; ++x)
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt) dq[x][dt] = splat(0.0f);

    auto step = [&](auto masked, const bf16_t* sk, const bf16_t* sv, const int* sdoc, int k0) {
        const int h4 = 4 * (lane_id() >> 5);
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            f32x16 s[QB], dp[QB];
#pragma unroll
            for (int x = 0; x < QB; ++x) {
                s[x] = splat(0.0f);
                dp[x] = splat(-delta[x]);
            }
#pragma unroll
            for (int t = 0; t < DP / 16; ++t) {
                const bf16x8 kf = rf.read(sk, kb, t), vf = rf.read(sv, kb, t);
#pragma unroll
                for (int x = 0; x < QB; ++x) {
                    s[x] = mfma(kf, qf[x][t], s[x]);
                    dp[x] = mfma(vf, dof[x][t], dp[x]);
                }
            }
            bf16x8 p[QB][2];
#pragma unroll
            for (int x = 0; x < QB; ++x) {
                const float base = static_cast<float>(row[x].pos - k0 - h4);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    grad1<MOD>(sc, s[x], dp[x], i, lse2[x],
                               fabsf(base - static_cast<float>(32 * kb + 8 * (i / 4) + i % 4)));
                if constexpr (decltype(masked)::value) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int j = 32 * kb + 8 * (i / 4) + h4 + i % 4, jj = k0 + j;
                        bool vis = (jj >= row[x].lo && jj <= row[x].hi) || jj < row[x].pre;
                        if (sdoc) vis = vis && sdoc[j] == row[x].doc;
                        if (!vis) dp[x][i] = 0.0f;
                    }
                }
                p[x][0] = pack(dp[x], 0);
                p[x][1] = pack(dp[x], 1);
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int dt = 0; dt < DP / 32; ++dt) {
                    const bf16x8 kf = cf.read(sk, 2 * kb + t, dt);
#pragma unroll
                    for (int x = 0; x < QB; ++x) dq[x][dt] = mfma(kf, p[x][t], dq[x][dt]);
                }
        }
    };

    KeyTiles it;
    it.init(seq, a, g, w, docs);
    int mode = 0, dcur = 0;
    int t = it.next(seq, a, g, w, docs, mode);
    auto load = [&](int tile) {
        lk.load(tile * kTile);
        lv.load(tile * kTile);
        if (seq.doc && threadIdx.x < kTile) dcur = doc_of(seq, a, tile * kTile + threadIdx.x);
    };
    auto store = [&](int buf) {
        lk.store(lds[buf][0]);
        lv.store(lds[buf][1]);
        if (seq.doc && threadIdx.x < kTile) sdocs[buf][threadIdx.x] = dcur;
    };
    if (t >= 0) {
        load(t);
        store(0);
    }
    int buf = 0;
    while (t >= 0) {
        __syncthreads();
        int nmode = 0;
        const int nt = it.next(seq, a, g, w, docs, nmode);
        if (nt >= 0) load(nt);
        if (mode == 2) step(std::false_type{}, lds[buf][0], lds[buf][1], nullptr, t * kTile);
        else if (mode == 1) step(std::true_type{}, lds[buf][0], lds[buf][1], seq.doc ? sdocs[buf] : nullptr, t * kTile);
        if (nt >= 0) store(buf ^ 1);
        buf ^= 1;
        t = nt;
        mode = nmode;
    }
#pragma unroll
    for (int x = 0; x < QB; ++x) {
        const int i = w0 + 32 * x + (lane_id() & 31);
        // dq is contiguous (b, sq, hq, d)
        bf16_t* o = a.dq + ((static_cast<int64_t>(b) * a.sq + i) * a.hq + h) * a.d;
        store_rows<DP>(dq[x], a.scale, o, i < a.sq, a.d);
    }
}

template <int DP, int KB, int NW, int MOD>
__global__ __launch_bounds__(64 * NW, 1) void k_attn_dkv(const AttnArgs a) {
    constexpr int BN = 32 * KB * NW, NT = 64 * NW;
    __shared__ __align__(16) bf16_t lds[2][2][Tile<DP>::ELEMS];
    __shared__ __align__(16) int sdocs[2][kTile];
    __shared__ __align__(16) float sstat[2][2][kTile];
    const int U = a.b * a.hkv;
    const int blk = blockIdx.x, u = blk % U, b = u / a.hkv, kvh = u % a.hkv;
    const int j0 = blk / U * BN;
    const Seq seq = sequence(a, b);
    const int w0 = j0 + wave_id() * 32 * KB;
    auto key_span = [&](int lo, int hi) {
        Span r;
        r.p0 = lo;
        r.p1 = hi < seq.n ? hi - 1 : seq.n - 1;
        doc_range(seq, a, r.p0, r.p1, r.d0, r.d1);
        return r;
    };
    const Span g = key_span(j0, j0 + BN), w = key_span(w0, w0 + 32 * KB);
    // whole blocks of real keys only: the rest is masked one by one
    const bool whole = w0 + 32 * KB <= seq.n;
    const int2* docs = a.doc_tiles + static_cast<int64_t>(b) * a.n_tiles;

    bf16x8 kf[KB][DP / 16], vf[KB][DP / 16];
    Row col[KB];
#pragma unroll
    for (int x = 0; x < KB; ++x) {
        const int j = w0 + 32 * x + (lane_id() & 31);
        col[x] = col_of(seq, a, j);
        load_rows<DP>(kf[x], a.k + b * a.k_b + kvh * a.k_h, a.k_s, j, j < seq.n, a.d);
        load_rows<DP>(vf[x], a.v + b * a.v_b + kvh * a.v_h, a.v_s, j, j < seq.n, a.d);
    }
    RowFrag<DP> rf;
    ColFrag<DP> cf;
    rf.init();
    cf.init();
    f32x16 dk[KB][DP / 32], dv[KB][DP / 32];
#pragma unroll
    for (int x = 0; x < KB; ++x)
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt) dk[x][dt] = dv[x][dt] = splat(0.0f);

    for (int r = 0; r < a.grp; ++r) {
        const int h = kvh * a.grp + r;
        const Score sc = score_of<MOD>(a, h);
        const float inv_scale = 1.0f / a.scale;
        QueryTiles it;
        it.init(seq, a, g, w, docs);
        Loader<DP, NT> lq, ld;
        lq.init(a.q + b * a.q_b + h * a.q_h, a.q_s, it.rows, a.d);
        ld.init(a.dout + b * a.do_b + h * a.do_h, a.do_s, it.rows, a.d);
        const int64_t stat = (static_cast<int64_t>(b) * a.hq + h) * a.sq;
        float st0 = 0.0f, st1 = 0.0f;
        int dcur = 0;

        // s starts at -lse in units of the product (no extras), dp at -delta
        auto step = [&](auto masked, const bf16_t* sq, const bf16_t* sd, const float* sl, const float* sdel,
                        const int* sdoc, int q0) {
            const int h4 = 4 * (lane_id() >> 5);
#pragma unroll
            for (int qb = 0; qb < 2; ++qb) {
                f32x16 s[KB], dp[KB], lse;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int at = 32 * qb + 8 * (i / 4) + h4 + i % 4;
                    lse[i] = sl[at];
                    dp[0][i] = sdel[at];
                }
#pragma unroll
                for (int x = KB - 1; x >= 0; --x) {
                    dp[x] = dp[0];
                    s[x] = MOD ? splat(0.0f) : lse;
                }
#pragma unroll
                for (int t = 0; t < DP / 16; ++t) {
                    const bf16x8 qa = rf.read(sq, qb, t), da = rf.read(sd, qb, t);
#pragma unroll
                    for (int x = 0; x < KB; ++x) {
                        s[x] = mfma(qa, kf[x][t], s[x]);
                        dp[x] = mfma(da, vf[x][t], dp[x]);
                    }
                }
                bf16x8 pp[KB][2], pd[KB][2];
#pragma unroll
                for (int x = 0; x < KB; ++x) {
                    const float base = static_cast<float>(seq.start + q0 + h4 - col[x].pos);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        grad1<MOD>(sc, s[x], dp[x], i, MOD ? lse[i] : 0.0f,
                                   fabsf(base + static_cast<float>(32 * qb + 8 * (i / 4) + i % 4)));
                    if constexpr (decltype(masked)::value) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int at = 32 * qb + 8 * (i / 4) + h4 + i % 4, p = seq.start + q0 + at;
                            bool vis = p >= col[x].lo && p <= col[x].hi;
                            if (sdoc) vis = vis && sdoc[at] == col[x].doc;
                            if (!vis) s[x][i] = dp[x][i] = 0.0f;
                        }
                    }
                    pp[x][0] = pack(s[x], 0);
                    pp[x][1] = pack(s[x], 1);
                    pd[x][0] = pack(dp[x], 0);
                    pd[x][1] = pack(dp[x], 1);
                }
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int dt = 0; dt < DP / 32; ++dt) {
                        const bf16x8 da = cf.read(sd, 2 * qb + t, dt), qa = cf.read(sq, 2 * qb + t, dt);
#pragma unroll
                        for (int x = 0; x < KB; ++x) {
                            dv[x][dt] = mfma(da, pp[x][t], dv[x][dt]);
                            dk[x][dt] = mfma(qa, pd[x][t], dk[x][dt]);
                        }
                    }
            }
        };

        auto load = [&](int tile) {
            lq.load(tile * kTile);
            ld.load(tile * kTile);
            if (threadIdx.x < kTile) {
                const int i = tile * kTile + threadIdx.x;
                float l = __builtin_inff(), d = 0.0f;
                if (i < it.rows) {
                    l = lse2_of(a.lse[stat + i]);
                    d = a.delta[stat + i];
                }
                st0 = MOD ? l : -l * kLn2 * inv_scale;
                st1 = -d;
                if (seq.doc) dcur = doc_of(seq, a, seq.start + i);
            }
        };
        auto store = [&](int buf) {
            lq.store(lds[buf][0]);
            ld.store(lds[buf][1]);
            if (threadIdx.x < kTile) {
                sstat[buf][0][threadIdx.x] = st0;
                sstat[buf][1][threadIdx.x] = st1;
                if (seq.doc) sdocs[buf][threadIdx.x] = dcur;
            }
        };
        int mode = 0;
        int t = it.next(seq, a, g, w, docs, mode);
        if (r > 0) __syncthreads();  // the last head's tiles are read
        if (t >= 0) {
            load(t);
            store(0);
        }
        int buf = 0;
        while (t >= 0) {
            __syncthreads();
            int nmode = 0;
            const int nt = it.next(seq, a, g, w, docs, nmode);
            if (nt >= 0) load(nt);
            const int* sdoc = seq.doc ? sdocs[buf] : nullptr;
            if (mode == 2 && whole)
                step(std::false_type{}, lds[buf][0], lds[buf][1], sstat[buf][0], sstat[buf][1], nullptr, t * kTile);
            else if (mode != 0)
                step(std::true_type{}, lds[buf][0], lds[buf][1], sstat[buf][0], sstat[buf][1], sdoc, t * kTile);
            if (nt >= 0) store(buf ^ 1);
            buf ^= 1;
            t = nt;
            mode = nmode;
        }
    }
#pragma unroll
    for (int x = 0; x < KB; ++x) {
        const int j = w0 + 32 * x + (lane_id() & 31);
        // dk and dv are contiguous (b, sk, hkv, d)
        const int64_t at = ((static_cast<int64_t>(b) * a.sk + j) * a.hkv + kvh) * a.d;
        store_rows<DP>(dk[x], a.scale, a.dk + at, j < a.sk, a.d);
        store_rows<DP>(dv[x], 1.0f, a.dv + at, j < a.sk, a.d);
    }
}

template <int DP, int MOD>
void dq(const AttnArgs& a, hipStream_t stream) {
    constexpr int QB = 1, NW = 4, BM = 32 * QB * NW;
    const int blocks = (a.sq + BM - 1) / BM * a.b * a.hq;
    k_attn_dq<DP, QB, NW, MOD><<<blocks, 64 * NW, 0, stream>>>(a);
}
template <int DP, int MOD>
void dkv(const AttnArgs& a, hipStream_t stream) {
    constexpr int KB = 1, NW = 4, BN = 32 * KB * NW;
    const int blocks = (a.sk + BN - 1) / BN * a.b * a.hkv;
    k_attn_dkv<DP, KB, NW, MOD><<<blocks, 64 * NW, 0, stream>>>(a);
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
