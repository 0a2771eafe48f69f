// Attention, forward: out = softmax(scores) V with the running maximum and
// sum of the softmax, one pass over the keys each query sees.
//
// Scores are made transposed (keys x queries), so a lane holds scores of one
// query only: maximum and sum take one exchange between the halves of the
// wave, and the probabilities are the next product's operand as they lie.
// By counters, of the cycles in which a CU holds waves: heads of 64 (16 x 1024
// tokens of 12 heads, causal: 43 us, 600 TFLOP/s of visible pairs) have the vector
// pipe busy for 67 % (4.4 instructions a score) and the matrix pipe for 33 %, one
// after the other rather than side by side: the scores' products have no vector
// work under them, nor the maximum and the first half of the exponentials any
// products.  Heads of 128 (4 x 4001 tokens, 32 heads over 8, prefix: 549 to 600 us,
// 910 to 1000 TFLOP/s, where a library product of 8192^3 reaches 1200): 51 % and
// 55 %.  LDS reads take 17 to 33 % and 28 to 55 % (a wave reads a whole tile for 32
// queries; the counter's busy cycles, and 128 bytes a clock).  Packed documents of
// 16384 tokens, cap, 6 heads of 128 (162 us): 59 % and 30 %, but CUs hold waves for
// half of the kernel only: 768 workgroups whose work depends on the place in the
// document, dealt by position.
#include "attn_common.hpp"

namespace muon {

namespace {

using namespace attn;

// The maximum is raised (and the sums so far rescaled) only once a score
// exceeds it by this many powers of two: sums stay below 2^8 times the number
// of keys, and most tiles skip the rescaling of the accumulators.
constexpr float kSlack = 8.0f;

// Running softmax and output of 32 queries (lane l % 32 of either half holds
// query l % 32; sums are per half until the end).
template <int DP>
struct Running {
    f32x16 o[DP / 32];
    float m, l;
    __device__ __forceinline__ void init() {
        m = neg_inf();
        l = 0.0f;
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt) o[dt] = splat(0.0f);
    }
};

// One tile of keys at positions k0 ..: scores, softmax, output.  A wave issues
// vector work while the matrix cores are busy with its last product, so extras
// of the scores of the first 32 keys are computed while the products of the
// second run, and the second's probabilities under the first's products with
// V; operands are read from LDS kAhead products early.  `masked` is a branch
// inside rather than a variant of the whole step: two variants made the
// compiler copy the accumulators between them on every tile.
constexpr int kAhead = 3;
template <int DP, int MOD>
__device__ __forceinline__ void tile_step(Running<DP>& run, const bf16x8 (&qf)[DP / 16], const RowFrag<DP>& rf,
                                          const ColFrag<DP>& cf, uint32_t sk, uint32_t sv, bool masked, const int* sdoc,
                                          const Row& row, const Score& sc, const Seq& seq, Args a, int k0) {
    constexpr int KT = DP / 16, DT = DP / 32;
    const int h4 = 4 * (lane_id() >> 5);
    bf16x8 p[4], ring[kAhead];
    f32x16 s[2];
    auto extras = [&](int kb, int i) {
        const float dist = fabsf(static_cast<float>(row.pos - k0 - h4) - static_cast<float>(32 * kb + place(i)));
        s[kb][i] = score<MOD>(sc, s[kb][i], dist);
    };
    auto operand = [&](int x) {  // of product x: keys along the row, then V across
        return x < 2 * KT ? rf.read(sk, x / KT, x % KT) : cf.read(sv, (x - 2 * KT) / DT, (x - 2 * KT) % DT);
    };
    each<0, kAhead>([&](auto x) { ring[x] = operand(x); });
    in_order();
    each<0, 2 * KT>([&](auto x_) {
        constexpr int x = decltype(x_)::value, kb = x / KT, t = x % KT;
        s[kb] = mfma(ring[x % kAhead], qf[t], t == 0 ? splat(0.0f) : s[kb]);
        ring[x % kAhead] = operand(x + kAhead);
        if constexpr (MOD != 0 && kb == 1 && t >= 2)
            each<16 * (t - 2) / (KT - 2), 16 * (t - 1) / (KT - 2)>([&](auto i) { extras(0, i); });
        in_order();
    });
    if constexpr (MOD != 0) each<0, 16>([&](auto i) { extras(1, i); });
    if (masked) {
        const Bits m = keys_seen(row, seq, a, k0 + h4);
        each<0, 32>([&](auto e) {
            constexpr int kb = decltype(e)::value / 16, i = decltype(e)::value % 16;
            s[kb][i] = where(m, kb, i, s[kb][i], neg_inf());
        });
        if (sdoc)
            each<0, 32>([&](auto e) {
                constexpr int kb = decltype(e)::value / 16, i = decltype(e)::value % 16;
                s[kb][i] = sdoc[32 * kb + place(i) + h4] == row.doc ? s[kb][i] : neg_inf();
            });
    }
    float top = s[0][0];
    each<1, 32>([&](auto e) { top = fmaxf(top, s[e / 16][e % 16]); });
    top = half_max(top) * (MOD ? 1.0f : sc.c);
    if (__any(top > run.m + kSlack)) {
        const float m = fmaxf(run.m, top);
        const float alpha = m == neg_inf() ? 1.0f : exp2_fast(run.m - m);
        run.m = m;
        run.l *= alpha;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i) run.o[dt][i] *= alpha;
    }
    const float m = run.m == neg_inf() ? 0.0f : run.m;
    auto prob = [&](int kb, int i) {
        s[kb][i] = exp2_fast(MOD ? s[kb][i] - m : fmaf(s[kb][i], sc.c, -m));
        run.l += s[kb][i];
        if (i == 7) p[2 * kb] = pack(s[kb], 0);
        if (i == 15) p[2 * kb + 1] = pack(s[kb], 1);
    };
    each<0, 16>([&](auto i) { prob(0, i); });
    in_order();
    each<0, 4 * DT>([&](auto x_) {
        constexpr int x = decltype(x_)::value, t = x / DT, dt = x % DT, at = 2 * KT + x;
        run.o[dt] = mfma(ring[at % kAhead], p[t], run.o[dt]);
        if constexpr (x + kAhead < 4 * DT) ring[at % kAhead] = operand(at + kAhead);
        if constexpr (x < 2 * DT) each<16 * x / (2 * DT), 16 * (x + 1) / (2 * DT)>([&](auto i) { prob(1, i); });
        in_order();
    });
}

// Workgroups of NW waves, 32 queries of one head each: 128 queries share every
// tile.  Registers (144 for heads of 64, 208 for 128) let 3 and 2 waves on a
// SIMD; forcing a fourth spilled and took 10 % longer.
template <int DP, int NW, int MOD>
__global__ __launch_bounds__(64 * NW, DP == 64 ? 3 : 2) void k_attn_fwd(const AttnArgs) {
    constexpr int BM = 32 * NW, NT = 64 * NW, TB = 2 * Tile<DP>::ELEMS;
    constexpr int ST = 2;  // one tile lands while the other is used (with three: 1 to 8 % slower)
    __shared__ __align__(16) bf16_t lds[ST][2][Tile<DP>::ELEMS];
    __shared__ __align__(16) int sdocs[ST][kTile];
    const Args a = arguments();
    // heads that share keys run side by side; the longest tiles go first
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
    const Score sc = score_of<MOD>(a, h);
    bf16x8 qf[DP / 16];
    load_rows<DP>(qf, a->q + b * a->q_b + h * a->q_h, a->q_s, i, i < a->sq, a->d);
    RowFrag<DP> rf;
    ColFrag<DP> cf;
    rf.init();
    cf.init();
    Running<DP> run;
    run.init();
    settle(qf);
    // (the two buffers' code side by side: as one loop, 3 to 25 % slower)
    auto use = [&](auto x_) {
        constexpr int x = decltype(x_)::value;
        landed();
        fetch(1 - x);
        if (mode[x] != 0)
            tile_step<DP, MOD>(run, qf, rf, cf, at + 2 * x * TB, at + (2 * x + 1) * TB, mode[x] == 1,
                               seq.doc ? sdocs[x] : nullptr, row, sc, seq, a, tile[x] * kTile);
    };
    for (;;) {
        if (tile[0] < 0) break;
        use(std::integral_constant<int, 0>{});
        if (tile[1] < 0) break;
        use(std::integral_constant<int, 1>{});
    }
    const Args z = again(a);
    const bool ok = i < z->sq;
    const float l = half_sum(run.l);
    // (a NaN sum is not empty: it goes to the output)
    const bool empty = l == 0.0f || !real_row(seq, z, seq.start + i);
    if (empty)
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt) run.o[dt] = splat(0.0f);
    store_rows<DP>(run.o, empty ? 0.0f : 1.0f / l,
                   z->out + b * z->o_b + h * z->o_h + static_cast<int64_t>(i) * z->o_s, ok, z->d);
    if (ok && lane_id() < 32)
        z->lse[(static_cast<int64_t>(b) * z->hq + h) * z->sq + i] =
            empty ? neg_inf() : (run.m + __builtin_amdgcn_logf(l)) * kLn2;
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
// float32 output go to `part` for k_attn_merge.  Bound by the cache: 32 caches
// of up to 16384 keys, 8 heads of 128, capped scores: 288 us, 5.6 TB/s of reads
// (a kernel that only reads them in this order: 6.0).
template <int DP, int NW, int MOD>
__global__ __launch_bounds__(64 * NW, 1) void k_attn_split(const AttnArgs) {
    const Args a = arguments();
    __shared__ __align__(16) bf16_t lds[NW][2][Tile<DP>::ELEMS];
    __shared__ __align__(16) int sdocs[NW][kTile];
    __shared__ float sml[NW][2][32];
    const int U = a->b * a->hkv, rows = a->grp * a->sq;
    if (block_place() >= static_cast<uint32_t>((rows + 31) / 32) * a->splits * U) return;
    const int blk = block_place(), u = blk % U, b = u / a->hkv, kvh = u % a->hkv;
    const int split = blk / U % a->splits, rt = blk / U / a->splits;
    const Seq seq = sequence(a, b);
    const int wave = wave_id(), lane = lane_id();
    // row -> head r / sq of the group, query r % sq
    const int r = rt * 32 + (lane & 31);
    const bool ok = r < rows;
    const int i = ok ? r % a->sq : 0, h = kvh * a->grp + (ok ? r / a->sq : 0);
    const int r1 = rt * 32 + 32 < rows ? rt * 32 + 32 : rows;
    // the positions of the tile's rows (whole heads wrap around)
    const bool wraps = rt * 32 / a->sq != (r1 - 1) / a->sq;
    Span g = query_span(seq, a, wraps ? 0 : rt * 32 % a->sq, wraps ? a->sq : (r1 - 1) % a->sq + 1);

    bf16x8 qf[DP / 16];
    const Row row = row_of(seq, a, seq.start + i);
    const Score sc = score_of<MOD>(a, h);
    load_rows<DP>(qf, a->q + b * a->q_b + h * a->q_h, a->q_s, i, ok, a->d);
    Loader<DP, 64> lk, lv;
    lk.init(a->k + b * a->k_b + kvh * a->k_h, a->k_s, seq.n, a->d);
    lv.init(a->v + b * a->v_b + kvh * a->v_h, a->v_s, seq.n, a->d);
    RowFrag<DP> rf;
    ColFrag<DP> cf;
    rf.init();
    cf.init();
    Running<DP> run;
    run.init();

    // the chunk's tiles in turn
    KeyTiles it;
    it.turns = NW;
    it.turn = wave;
    it.init(seq, a, g, g, split * a->chunk, split * a->chunk + a->chunk);
    in_vectors(g);
    static_assert((NW & (NW - 1)) == 0, "turns");
    auto next = [&](int& mode) { return it.next(seq, a, g, g, mode); };
    int mode = 0, dcur = 0;
    int t = next(mode);
    auto load = [&](int tile) {
        lk.load(tile * kTile);
        lv.load(tile * kTile);
        if (seq.doc) dcur = doc_of(seq, a, tile * kTile + lane);
    };
    const uint32_t tk = lds_addr(lds[wave][0]), tv = lds_addr(lds[wave][1]);
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
        if (mode != 0)
            tile_step<DP, MOD>(run, qf, rf, cf, tk, tv, mode == 1, seq.doc ? sdocs[wave] : nullptr, row, sc, seq, a,
                               t * kTile);
        t = nt;
        mode = nmode;
    }

    // merge: every wave's (m, l), then the sum of the scaled outputs wave by wave
    const float l = half_sum(run.l);
    if (lane < 32) {
        sml[wave][0][lane] = run.m;
        sml[wave][1][lane] = l;
    }
    __syncthreads();
    float m = neg_inf(), sum = 0.0f;
#pragma unroll
    for (int x = 0; x < NW; ++x) m = fmaxf(m, sml[x][0][lane & 31]);
    const float ms = m == neg_inf() ? 0.0f : m;
#pragma unroll
    for (int x = 0; x < NW; ++x) sum += sml[x][1][lane & 31] * exp2_fast(sml[x][0][lane & 31] - ms);
    const float mine = exp2_fast(run.m - ms);
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) run.o[dt][i] *= mine;
    // the tiles are free: waves 1 .. leave their outputs there, lane by lane
    float* so = reinterpret_cast<float*>(&lds[0][0][0]);
    static_assert(sizeof(lds) >= static_cast<size_t>(NW - 1) * DP * 32 * 4, "room for the merge");
    if (wave > 0) {
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i) so[((wave - 1) * (DP / 2) + dt * 16 + i) * 64 + lane] = run.o[dt][i];
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int x = 1; x < NW; ++x)
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i) run.o[dt][i] += so[((x - 1) * (DP / 2) + dt * 16 + i) * 64 + lane];

    const bool empty = sum == 0.0f || !real_row(seq, a, seq.start + i);
    const int64_t at = (static_cast<int64_t>(b) * a->hq + h) * a->sq + i;
    if (a->splits == 1) {
        if (empty)
#pragma unroll
            for (int dt = 0; dt < DP / 32; ++dt) run.o[dt] = splat(0.0f);
        bf16_t* o = a->out + b * a->o_b + h * a->o_h + static_cast<int64_t>(i) * a->o_s;
        store_rows<DP>(run.o, empty ? 0.0f : 1.0f / sum, o, ok, a->d);
        if (ok && lane < 32) a->lse[at] = empty ? neg_inf() : (m + __builtin_amdgcn_logf(sum)) * kLn2;
        return;
    }
    // part: (m, l) of every row and split, then the outputs
    const int64_t n = static_cast<int64_t>(a->b) * a->hq * a->sq * a->splits, p = at * a->splits + split;
    if (!ok) return;
    if (lane < 32) {
        a->part[2 * p] = m;
        a->part[2 * p + 1] = empty ? 0.0f : sum;
    }
    float* o = a->part + part_outputs(n) + p * a->d;
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
        for (int g4 = 0; g4 < 4; ++g4) {
            const int col = 32 * dt + 8 * g4 + 4 * (lane >> 5);
            if (col < a->d && !empty)
                *reinterpret_cast<f32x4*>(o + col) = f32x4{run.o[dt][4 * g4], run.o[dt][4 * g4 + 1],
                                                           run.o[dt][4 * g4 + 2], run.o[dt][4 * g4 + 3]};
        }
}

// One wave per (query, head): the chunks' outputs joined in their order.  Lane
// s holds the factor of chunk s (64 at a time); loads go 8 chunks at once.
__global__ __launch_bounds__(256) void k_attn_merge(const AttnArgs) {
    const Args a = arguments();
    const int lane = lane_id(), splits = a->splits, d = a->d;
    const int64_t at = static_cast<int64_t>(block_place()) * 4 + wave_id(), rows = static_cast<int64_t>(a->b) * a->hq * a->sq;
    if (at >= rows) return;
    const float* ml = a->part + 2 * at * splits;
    const float* o = a->part + part_outputs(rows * splits) + at * splits * d;
    float m = neg_inf(), l = 0.0f;
    for (int s = lane; s < splits; s += 64) m = fmaxf(m, ml[2 * s + 1] != 0.0f ? ml[2 * s] : neg_inf());
#pragma unroll
    for (int x = 32; x; x >>= 1) m = fmaxf(m, __shfl_xor(m, x));
    const float ms = m == neg_inf() ? 0.0f : m;
    const int c = 2 * lane, cc = c < d ? c : 0;
    float x = 0.0f, y = 0.0f;
    for (int s0 = 0; s0 < splits; s0 += 64) {
        const int s = s0 + lane, n = splits - s0 < 64 ? splits - s0 : 64;
        // a chunk with a sum of zero saw nothing and wrote nothing
        float ls = s < splits ? ml[2 * s + 1] : 0.0f;
        const float f = ls != 0.0f ? exp2_fast(ml[2 * s] - ms) : 0.0f;
        const uint64_t live = __ballot(ls != 0.0f);
        ls *= f;
#pragma unroll
        for (int w = 32; w; w >>= 1) ls += __shfl_xor(ls, w);
        l += ls;
        for (int e = 0; e < n; e += 8) {
            f32x2_t v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int r = e + u < n ? e + u : e;
                v[u] = *reinterpret_cast<const f32x2_t*>(o + static_cast<int64_t>(s0 + r) * d + cc);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float g = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), (e + u) & 63));
                if (e + u < n && ((live >> (e + u)) & 1)) {
                    x = fmaf(v[u].x, g, x);
                    y = fmaf(v[u].y, g, y);
                }
            }
        }
    }
    const bool empty = l == 0.0f;
    const float inv = empty ? 0.0f : 1.0f / l;
    const int i = static_cast<int>(at % a->sq), h = static_cast<int>(at / a->sq % a->hq), b = static_cast<int>(at / a->sq / a->hq);
    if (c < d)
        *reinterpret_cast<uint32_t*>(a->out + b * a->o_b + h * a->o_h + static_cast<int64_t>(i) * a->o_s + c) =
            f32x2_to_bf16x2(x * inv, y * inv);
    if (lane == 0) a->lse[at] = empty ? neg_inf() : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// (lowest, highest) document of each kTile tokens, one wave per tile.
__global__ __launch_bounds__(256) void k_doc_tiles(const AttnArgs) {
    const Args a = arguments();
    const int64_t w = static_cast<int64_t>(block_place()) * 4 + wave_id();
    if (w >= static_cast<int64_t>(a->b) * a->n_tiles) return;
    const int b = static_cast<int>(w / a->n_tiles), t = static_cast<int>(w % a->n_tiles);
    const int j = t * kTile + lane_id();
    int lo = 0x7fffffff, hi = static_cast<int>(0x80000000u);
    if (j < a->sk) lo = hi = a->documents[b * a->doc_b + j];
#pragma unroll
    for (int m = 32; m; m >>= 1) {
        const int x = __shfl_xor(lo, m), y = __shfl_xor(hi, m);
        lo = x < lo ? x : lo;
        hi = y > hi ? y : hi;
    }
    if (lane_id() == 0) a->doc_tiles[w] = {lo, hi};
}

template <int DP, int MOD>
void fwd(const AttnArgs& a, hipStream_t stream) {
    constexpr int NW = 4, BM = 32 * NW;
    const int64_t blocks = static_cast<int64_t>((a.sq + BM - 1) / BM) * a.b * a.hq;
    k_attn_fwd<DP, NW, MOD><<<long_grid(blocks, 64 * NW), 64 * NW, 0, stream>>>(a);
}

template <int DP, int MOD>
void split(const AttnArgs& a, hipStream_t stream) {
    const int64_t blocks = static_cast<int64_t>((a.grp * a.sq + 31) / 32) * a.splits * a.b * a.hkv;
    // 8 waves fill a CU's LDS with tiles of 64; with more workgroups than CUs
    // two of 4 waves share it, one computing while the other starts or ends
    if (DP == 64 && blocks <= 256) k_attn_split<DP, DP == 64 ? 8 : 4, MOD><<<static_cast<int>(blocks), 64 * (DP == 64 ? 8 : 4), 0, stream>>>(a);
    else k_attn_split<DP, 4, MOD><<<long_grid(blocks, 256), 256, 0, stream>>>(a);
    if (a.splits > 1) {
        const int64_t rows = static_cast<int64_t>(a.b) * a.hq * a.sq;
        k_attn_merge<<<long_grid((rows + 3) / 4, 256), 256, 0, stream>>>(a);
    }
}

}  // namespace

hipError_t launch_attn_doc_tiles(const AttnArgs& a, hipStream_t stream) {
    const int64_t waves = static_cast<int64_t>(a.b) * a.n_tiles;
    k_doc_tiles<<<long_grid((waves + 3) / 4, 256), 256, 0, stream>>>(a);
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
