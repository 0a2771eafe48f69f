// Attention, forward: out = softmax(scores) V with the running maximum and
// sum of the softmax, one pass over the keys each query sees.
#include "attn_common.hpp"

namespace muon {

namespace {

using namespace attn;

// The maximum is raised (and the sums so far rescaled) only once a score
// exceeds it by this many powers of two: sums stay below 2^8 times the number
// of keys, and most tiles skip the rescaling of the accumulators.
constexpr float kSlack = 8.0f;

// Running softmax and output of QB blocks of 32 queries (lane l % 32 of
// either half holds query l % 32; sums are per half until the end).
template <int DP, int QB>
struct Running {
    f32x16 o[QB][DP / 32];
    float m[QB], l[QB];
    __device__ __forceinline__ void init() {
#pragma unroll
        for (int q = 0; q < QB; ++q) {
            m[q] = neg_inf();
            l[q] = 0.0f;
#pragma unroll
            for (int dt = 0; dt < DP / 32; ++dt) o[q][dt] = splat(0.0f);
        }
    }
};

// One tile of keys at positions k0 ..: scores, softmax, output.
template <int DP, int QB, int MOD, bool MASK>
__device__ __forceinline__ void tile_step(Running<DP, QB>& run, const bf16x8 (&qf)[QB][DP / 16],
                                          const RowFrag<DP>& rf, const ColFrag<DP>& cf, const bf16_t* sk,
                                          const bf16_t* sv, const int* sdoc, const Row (&row)[QB], const Score (&sc)[QB],
                                          int k0) {
    const int h4 = 4 * (lane_id() >> 5);
    bf16x8 p[QB][4];
    f32x16 s[QB][2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
        for (int q = 0; q < QB; ++q) s[q][kb] = splat(0.0f);
#pragma unroll
        for (int t = 0; t < DP / 16; ++t) {
            const bf16x8 kf = rf.read(sk, kb, t);
#pragma unroll
            for (int q = 0; q < QB; ++q) s[q][kb] = mfma(kf, qf[q][t], s[q][kb]);
        }
    }
#pragma unroll
    for (int q = 0; q < QB; ++q) {
        if constexpr (MOD != 0) {
            const float base = static_cast<float>(row[q].pos - k0 - h4);
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float r;
                    const float dist = fabsf(base - static_cast<float>(32 * kb + 8 * (i / 4) + i % 4));
                    s[q][kb][i] = score<MOD>(sc[q], s[q][kb][i], dist, r);
                }
        }
        if constexpr (MASK) {
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    int e[4] = {0, 0, 0, 0};
                    if (sdoc) {
                        const int4 x = *reinterpret_cast<const int4*>(sdoc + 32 * kb + 8 * g + h4);
                        e[0] = x.x;
                        e[1] = x.y;
                        e[2] = x.z;
                        e[3] = x.w;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = k0 + 32 * kb + 8 * g + h4 + i;
                        bool vis = (j >= row[q].lo && j <= row[q].hi) || j < row[q].pre;
                        if (sdoc) vis = vis && e[i] == row[q].doc;
                        if (!vis) s[q][kb][4 * g + i] = neg_inf();
                    }
                }
        }
        const float c = MOD ? 1.0f : sc[q].c;
        float mx = s[q][0][0];
#pragma unroll
        for (int i = 1; i < 16; ++i) mx = fmaxf(mx, s[q][0][i]);
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[q][1][i]);
        mx = half_max(mx) * c;
        if (__any(mx > run.m[q] + kSlack)) {
            const float m = fmaxf(run.m[q], mx);
            const float alpha = m == neg_inf() ? 1.0f : exp2_fast(run.m[q] - m);
            run.m[q] = m;
            run.l[q] *= alpha;
#pragma unroll
            for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
                for (int i = 0; i < 16; ++i) run.o[q][dt][i] *= alpha;
        }
        const float m = run.m[q] == neg_inf() ? 0.0f : run.m[q];
        float l = 0.0f;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[q][kb][i] = exp2_fast(MOD ? s[q][kb][i] - m : fmaf(s[q][kb][i], c, -m));
                l += s[q][kb][i];
            }
            p[q][2 * kb] = pack(s[q][kb], 0);
            p[q][2 * kb + 1] = pack(s[q][kb], 1);
        }
        run.l[q] += l;
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt) {
            const bf16x8 vf = cf.read(sv, t, dt);
#pragma unroll
            for (int q = 0; q < QB; ++q) run.o[q][dt] = mfma(vf, p[q][t], run.o[q][dt]);
        }
}

// Workgroups of NW waves, 32 QB queries of one head each.
template <int DP, int QB, int NW, int MOD>
__global__ __launch_bounds__(64 * NW, QB == 1 ? 2 : 1) void k_attn_fwd(const AttnArgs a) {
    constexpr int BM = 32 * QB * NW, NT = 64 * NW;
    __shared__ __align__(16) bf16_t lds[2][2][Tile<DP>::ELEMS];
    __shared__ __align__(16) int sdocs[2][kTile];
    // heads that share keys run side by side; the longest tiles go first
    const int H = a.b * a.hq, U = a.b * a.hkv;
    const int blk = blockIdx.x, e = blk % H;
    const int u = e % U, b = u / a.hkv, kvh = u % a.hkv, h = kvh * a.grp + e / U;
    const int i0 = ((gridDim.x / H) - 1 - blk / H) * BM;
    const int i1 = i0 + BM < a.sq ? i0 + BM : a.sq;
    const Seq seq = sequence(a, b);
    const int w0 = i0 + wave_id() * 32 * QB, w1 = w0 + 32 * QB < a.sq ? w0 + 32 * QB : a.sq;
    const Span g = query_span(seq, a, i0, i1), w = query_span(seq, a, w0, w1);
    const int2* docs = a.doc_tiles + static_cast<int64_t>(b) * a.n_tiles;

    bf16x8 qf[QB][DP / 16];
    Row row[QB];
    Score sc[QB];
    const bf16_t* q = a.q + b * a.q_b + h * a.q_h;
#pragma unroll
    for (int x = 0; x < QB; ++x) {
        const int i = w0 + 32 * x + (lane_id() & 31);
        row[x] = row_of(seq, a, seq.start + i);
        sc[x] = score_of<MOD>(a, h);
        load_rows<DP>(qf[x], q, a.q_s, i, i < a.sq, a.d);
    }
    Loader<DP, NT> lk, lv;
    lk.init(a.k + b * a.k_b + kvh * a.k_h, a.k_s, seq.n, a.d);
    lv.init(a.v + b * a.v_b + kvh * a.v_h, a.v_s, seq.n, a.d);
    RowFrag<DP> rf;
    ColFrag<DP> cf;
    rf.init();
    cf.init();
    Running<DP, QB> run;
    run.init();

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
        if (mode == 2)
            tile_step<DP, QB, MOD, false>(run, qf, rf, cf, lds[buf][0], lds[buf][1], nullptr, row, sc, t * kTile);
        else if (mode == 1)
            tile_step<DP, QB, MOD, true>(run, qf, rf, cf, lds[buf][0], lds[buf][1], seq.doc ? sdocs[buf] : nullptr, row,
                                         sc, t * kTile);
        if (nt >= 0) store(buf ^ 1);
        buf ^= 1;
        t = nt;
        mode = nmode;
    }

#pragma unroll
    for (int x = 0; x < QB; ++x) {
        const int i = w0 + 32 * x + (lane_id() & 31);
        const bool ok = i < a.sq;
        const float l = half_sum(run.l[x]);
        // (a NaN sum is not empty: it goes to the output)
        const bool empty = l == 0.0f || !real_row(seq, a, seq.start + i);
        const float inv = empty ? 0.0f : 1.0f / l;
        if (empty)
#pragma unroll
            for (int dt = 0; dt < DP / 32; ++dt) run.o[x][dt] = splat(0.0f);
        bf16_t* o = a.out + b * a.o_b + h * a.o_h + static_cast<int64_t>(i) * a.o_s;
        store_rows<DP>(run.o[x], inv, o, ok, a.d);
        if (ok && lane_id() < 32)
            a.lse[(static_cast<int64_t>(b) * a.hq + h) * a.sq + i] =
                empty ? neg_inf() : (run.m[x] + __builtin_amdgcn_logf(l)) * kLn2;
    }
}

// LDS written by one wave and read by its other lanes: the wave's LDS
// operations run in order, so only the compiler has to keep them so.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Few queries over many keys: a workgroup takes 32 rows (query, head) of the
// heads that share one key head and `chunk` key tiles; its NW waves take the
// tiles in turn, each with LDS of its own and no barrier, and merge at the
// end.  With one chunk the result is final; otherwise the maximum, sum and
// float32 output go to `part` for k_attn_merge.
template <int DP, int NW, int MOD>
__global__ __launch_bounds__(64 * NW, 1) void k_attn_split(const AttnArgs a) {
    __shared__ __align__(16) bf16_t lds[NW][2][Tile<DP>::ELEMS];
    __shared__ __align__(16) int sdocs[NW][kTile];
    __shared__ float sml[NW][2][32];
    const int U = a.b * a.hkv, rows = a.grp * a.sq;
    const int blk = blockIdx.x, u = blk % U, b = u / a.hkv, kvh = u % a.hkv;
    const int split = blk / U % a.splits, rt = blk / U / a.splits;
    const Seq seq = sequence(a, b);
    const int wave = wave_id(), lane = lane_id();
    // row -> head r / sq of the group, query r % sq
    const int r = rt * 32 + (lane & 31);
    const bool ok = r < rows;
    const int i = ok ? r % a.sq : 0, h = kvh * a.grp + (ok ? r / a.sq : 0);
    const int r1 = rt * 32 + 32 < rows ? rt * 32 + 32 : rows;
    // the positions of the tile's rows (whole heads wrap around)
    const bool wraps = rt * 32 / a.sq != (r1 - 1) / a.sq;
    const Span g = query_span(seq, a, wraps ? 0 : rt * 32 % a.sq, wraps ? a.sq : (r1 - 1) % a.sq + 1);
    const int2* docs = a.doc_tiles + static_cast<int64_t>(b) * a.n_tiles;

    bf16x8 qf[1][DP / 16];
    Row row[1] = {row_of(seq, a, seq.start + i)};
    Score sc[1] = {score_of<MOD>(a, h)};
    load_rows<DP>(qf[0], a.q + b * a.q_b + h * a.q_h, a.q_s, i, ok, a.d);
    Loader<DP, 64> lk, lv;
    lk.init(a.k + b * a.k_b + kvh * a.k_h, a.k_s, seq.n, a.d);
    lv.init(a.v + b * a.v_b + kvh * a.v_h, a.v_s, seq.n, a.d);
    RowFrag<DP> rf;
    ColFrag<DP> cf;
    rf.init();
    cf.init();
    Running<DP, 1> run;
    run.init();

    KeyTiles it;
    it.init(seq, a, g, g, docs);
    const int first = split * a.chunk, last = first + a.chunk;
    // this wave's next tile of the chunk, in turn over the tiles that are seen
    int turn = 0;
    auto next = [&](int& mode) {
        for (;;) {
            const int t = it.next(seq, a, g, g, docs, mode);
            if (t < 0 || t >= last) return -1;
            if (t >= first && turn++ % NW == wave) return t;
        }
    };
    int mode = 0, dcur = 0;
    int t = next(mode);
    auto load = [&](int tile) {
        lk.load(tile * kTile);
        lv.load(tile * kTile);
        if (seq.doc) dcur = doc_of(seq, a, tile * kTile + lane);
    };
    auto store = [&]() {
        lk.store(lds[wave][0]);
        lv.store(lds[wave][1]);
        if (seq.doc) sdocs[wave][lane] = dcur;
    };
    if (t >= 0) load(t);
    while (t >= 0) {
        wave_fence();
        store();
        wave_fence();
        int nmode = 0;
        const int nt = next(nmode);
        if (nt >= 0) load(nt);
        if (mode == 2)
            tile_step<DP, 1, MOD, false>(run, qf, rf, cf, lds[wave][0], lds[wave][1], nullptr, row, sc, t * kTile);
        else if (mode == 1)
            tile_step<DP, 1, MOD, true>(run, qf, rf, cf, lds[wave][0], lds[wave][1], seq.doc ? sdocs[wave] : nullptr,
                                        row, sc, t * kTile);
        t = nt;
        mode = nmode;
    }

    // merge: every wave's (m, l), then the sum of the scaled outputs wave by wave
    const float l = half_sum(run.l[0]);
    if (lane < 32) {
        sml[wave][0][lane] = run.m[0];
        sml[wave][1][lane] = l;
    }
    __syncthreads();
    float m = neg_inf(), sum = 0.0f;
#pragma unroll
    for (int x = 0; x < NW; ++x) m = fmaxf(m, sml[x][0][lane & 31]);
    const float ms = m == neg_inf() ? 0.0f : m;
#pragma unroll
    for (int x = 0; x < NW; ++x) sum += sml[x][1][lane & 31] * exp2_fast(sml[x][0][lane & 31] - ms);
    const float mine = exp2_fast(run.m[0] - ms);
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) run.o[0][dt][i] *= mine;
    // the tiles are free: waves 1 .. leave their outputs there, lane by lane
    float* so = reinterpret_cast<float*>(&lds[0][0][0]);
    static_assert(sizeof(lds) >= static_cast<size_t>(NW - 1) * DP * 32 * 4, "room for the merge");
    if (wave > 0) {
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i) so[((wave - 1) * (DP / 2) + dt * 16 + i) * 64 + lane] = run.o[0][dt][i];
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int x = 1; x < NW; ++x)
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i) run.o[0][dt][i] += so[((x - 1) * (DP / 2) + dt * 16 + i) * 64 + lane];

    const bool empty = sum == 0.0f || !real_row(seq, a, seq.start + i);
    const int64_t at = (static_cast<int64_t>(b) * a.hq + h) * a.sq + i;
    if (a.splits == 1) {
        if (empty)
#pragma unroll
            for (int dt = 0; dt < DP / 32; ++dt) run.o[0][dt] = splat(0.0f);
        bf16_t* o = a.out + b * a.o_b + h * a.o_h + static_cast<int64_t>(i) * a.o_s;
        store_rows<DP>(run.o[0], empty ? 0.0f : 1.0f / sum, o, ok, a.d);
        if (ok && lane < 32) a.lse[at] = empty ? neg_inf() : (m + __builtin_amdgcn_logf(sum)) * kLn2;
        return;
    }
    // part: (m, l) of every row and split, then the outputs
    const int64_t n = static_cast<int64_t>(a.b) * a.hq * a.sq * a.splits, p = at * a.splits + split;
    if (!ok) return;
    if (lane < 32) {
        a.part[2 * p] = m;
        a.part[2 * p + 1] = empty ? 0.0f : sum;
    }
    float* o = a.part + 2 * n + p * a.d;
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
        for (int g4 = 0; g4 < 4; ++g4) {
            const int col = 32 * dt + 8 * g4 + 4 * (lane >> 5);
            if (col < a.d && !empty)
                *reinterpret_cast<f32x4*>(o + col) = f32x4{run.o[0][dt][4 * g4], run.o[0][dt][4 * g4 + 1],
                                                           run.o[0][dt][4 * g4 + 2], run.o[0][dt][4 * g4 + 3]};
        }
}

// One wave per (query, head): the chunks' outputs joined in their order.
__global__ __launch_bounds__(256) void k_attn_merge(const AttnArgs a) {
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 4 + wave_id(), rows = static_cast<int64_t>(a.b) * a.hq * a.sq;
    if (at >= rows) return;
    const float* ml = a.part + 2 * at * a.splits;
    const float* o = a.part + 2 * rows * a.splits + at * a.splits * a.d;
    float m = neg_inf(), l = 0.0f;
    for (int s = 0; s < a.splits; ++s) m = fmaxf(m, ml[2 * s + 1] != 0.0f ? ml[2 * s] : neg_inf());
    const float ms = m == neg_inf() ? 0.0f : m;
    const int c = 2 * lane_id();
    float x = 0.0f, y = 0.0f;
    for (int s = 0; s < a.splits; ++s) {
        const float ls = ml[2 * s + 1];
        if (ls == 0.0f) continue;  // nothing was seen, nothing written
        const float f = exp2_fast(ml[2 * s] - ms);
        l = fmaf(ls, f, l);
        if (c < a.d) {
            x = fmaf(o[s * a.d + c], f, x);
            y = fmaf(o[s * a.d + c + 1], f, y);
        }
    }
    const bool empty = l == 0.0f;
    const float inv = empty ? 0.0f : 1.0f / l;
    const int i = static_cast<int>(at % a.sq), h = static_cast<int>(at / a.sq % a.hq), b = static_cast<int>(at / a.sq / a.hq);
    if (c < a.d)
        *reinterpret_cast<uint32_t*>(a.out + b * a.o_b + h * a.o_h + static_cast<int64_t>(i) * a.o_s + c) =
            f32x2_to_bf16x2(x * inv, y * inv);
    if (lane_id() == 0) a.lse[at] = empty ? neg_inf() : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// (lowest, highest) document of each kTile tokens, one wave per tile.
__global__ __launch_bounds__(256) void k_doc_tiles(const AttnArgs a) {
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + wave_id();
    const int b = static_cast<int>(w / a.n_tiles), t = static_cast<int>(w % a.n_tiles);
    if (b >= a.b) return;
    const int j = t * kTile + lane_id();
    int lo = 0x7fffffff, hi = static_cast<int>(0x80000000u);
    if (j < a.sk) lo = hi = a.documents[b * a.doc_b + j];
#pragma unroll
    for (int m = 32; m; m >>= 1) {
        const int x = __shfl_xor(lo, m), y = __shfl_xor(hi, m);
        lo = x < lo ? x : lo;
        hi = y > hi ? y : hi;
    }
    if (lane_id() == 0) a.doc_tiles[w] = {lo, hi};
}

template <int DP, int MOD>
void fwd(const AttnArgs& a, hipStream_t stream) {
    constexpr int QB = 1, NW = 4, BM = 32 * QB * NW;
    const int blocks = (a.sq + BM - 1) / BM * a.b * a.hq;
    k_attn_fwd<DP, QB, NW, MOD><<<blocks, 64 * NW, 0, stream>>>(a);
}

template <int DP, int MOD>
void split(const AttnArgs& a, hipStream_t stream) {
    constexpr int NW = 4;
    const int blocks = (a.grp * a.sq + 31) / 32 * a.splits * a.b * a.hkv;
    k_attn_split<DP, NW, MOD><<<blocks, 64 * NW, 0, stream>>>(a);
    if (a.splits > 1) {
        const int64_t rows = static_cast<int64_t>(a.b) * a.hq * a.sq;
        k_attn_merge<<<static_cast<int>((rows + 3) / 4), 256, 0, stream>>>(a);
    }
}

}  // namespace

hipError_t launch_attn_doc_tiles(const AttnArgs& a, hipStream_t stream) {
    const int64_t waves = static_cast<int64_t>(a.b) * a.n_tiles;
    k_doc_tiles<<<static_cast<int>((waves + 3) / 4), 256, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_attn_fwd(const AttnArgs& a, hipStream_t stream) {
    MUON_ATTN_DISPATCH(fwd, a, stream);
    return hipGetLastError();
}

hipError_t launch_attn_split(const AttnArgs& a, hipStream_t stream) {
    MUON_ATTN_DISPATCH(split, a, stream);
    return hipGetLastError();
}

}  // namespace muon
