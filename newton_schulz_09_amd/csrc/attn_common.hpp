// Device helpers of the attention kernels: visibility of keys, LDS tiles and
// matrix-core fragments.
//
// Every product runs on v_mfma_f32_32x32x16_bf16.  Lane l of a wave is (l %
// 32, half l / 32); its 8 values of an A or B operand are k = 8 half .. 8
// half + 7 of row (column) l % 32, and its 16 results are column l % 32, rows
// 8 (i / 4) + 4 half + i % 4.  A product whose result is the next product's B
// operand (P of the scores, dS) stays in registers: the results i = 8 t .. 8 t
// + 7 are taken as the operand of step t, which makes the contracted index of
// slot e the row 16 t + 8 (e / 4) + 4 half + e % 4, and the A operand is read
// from LDS in that order.
#pragma once

#include <type_traits>
#include <utility>

#include "lm_common.hpp"

// LDS addresses are 32-bit integers on the device; the host pass of the
// compiler, which runs none of this, sees them cast to 64-bit pointers.
#pragma clang diagnostic ignored "-Wint-to-pointer-cast"

namespace muon {
namespace attn {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// The launch arguments where the launch left them.  A kernel that held them
// all would run out of scalar registers inside its loop; again() makes a rare
// path read them once more instead.
typedef __attribute__((address_space(4))) const AttnArgs* Args;
__device__ __forceinline__ Args arguments() { return (Args)__builtin_amdgcn_kernarg_segment_ptr(); }
__device__ __forceinline__ Args again(Args a) {
    asm volatile("" : "+s"(a));
    return a;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxPos = 1 << 29;

// Extras of the scores, as template bits.  kWide: a cap above kMaxPlainCap (with
// kCap and kBias; the slope is 0 where none is given).
constexpr int kCap = 1;
constexpr int kBias = 2;
constexpr int kWide = 4;

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ int lane_id() { return threadIdx.x & 63; }
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Maximum and sum over the two lanes (l, l ^ 32) that hold a column.
__device__ __forceinline__ float half_max(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Buffer descriptor over `bytes` bytes at p: loads past the end give zero.
__device__ __forceinline__ auto rsrc(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00027000);
}

// LDS tile of kTile rows of DP (head size padded to 64, 96 or 128) bf16.
// Chunk c (16 bytes) of row r lies at slot c ^ f(r).  f makes 16 consecutive
// rows of one chunk fall on distinct banks (operands read along the row, 16
// bytes a lane) and 4 rows of one 64-byte piece too (transposing reads).
template <int DP>
struct Tile {
    static constexpr int CPR = DP / 8;
    static constexpr int LD = DP;
    static constexpr int ELEMS = kTile * LD;
    __device__ static __forceinline__ int f(int r) {
        if constexpr (DP == 128) return ((r & 3) << 2) | ((r >> 2) & 3);
        else if constexpr (DP == 64) return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
        else return (r >> 2) & 3;  // 192-byte rows already step by 4 chunks
    }
    __device__ static __forceinline__ int at(int r, int c) { return r * LD + ((c ^ f(r)) << 3); }
};

// Byte address of LDS memory, as the direct loads take it.
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void*)(p)));
}

// Direct loads from memory to LDS: lane l's 16 (4) bytes land at lds + 16 l
// (4 l).  In asm, because the compiler cannot tell which LDS reads such a
// load in flight concerns and would wait for it before every one; the loads
// have no result registers, and landed() orders them.  The wait states are
// those between a lane instruction's write of a scalar register (the
// descriptor) and a memory instruction that reads it, 5, which the compiler
// counts only for its own instructions; m0 needs 1.
__device__ __forceinline__ void load_lds16(uint32_t lds, uint32_t voff, u32x4 desc) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(voff), "s"(desc)
                 : "memory", "m0");
}
__device__ __forceinline__ void load_lds4(uint32_t lds, uint32_t voff, u32x4 desc) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds), "v"(voff), "s"(desc)
                 : "memory", "m0");
}
// This wave's loads have landed and its LDS reads are done, and so for every
// wave of the workgroup.
__device__ __forceinline__ void landed() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
__device__ __forceinline__ u32x4 descriptor(const void* p, uint32_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    return u32x4{static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(a))),
                 static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(a >> 32))) & 0xffffu,
                 static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(bytes))), 0x00027000u};
}

// Loads tiles of kTile rows straight into LDS, NT threads together.  Rows past
// `rows` and values past the head size come as zeros, whatever memory holds
// there.
template <int DP, int NT>
struct Direct {
    static constexpr int N = kTile * Tile<DP>::CPR / NT;  // loads per thread
    static_assert(N * NT == kTile * Tile<DP>::CPR, "whole chunks per thread");
    // loads of whole multiples of 16 rows differ by a fixed step (the layout
    // repeats): one offset is kept, and the others made from it
    static constexpr bool kSteps = NT % Tile<DP>::CPR == 0 && NT / Tile<DP>::CPR % 16 == 0;
    uint32_t voff[kSteps ? 1 : N];
    const bf16_t* base;  // row 0 of the sequence
    int64_t stride;      // elements per row
    int rows;
    uint32_t row_bytes;

    __device__ __forceinline__ void init(const bf16_t* p, int64_t s, int nrows, int d) {
        base = p;
        stride = s;
        rows = nrows;
        row_bytes = 2 * d;
#pragma unroll
        for (int i = 0; i < (kSteps ? 1 : N); ++i) {
            const int id = static_cast<int>(threadIdx.x) % NT + i * NT;
            const int r = id / Tile<DP>::CPR, c = (id % Tile<DP>::CPR) ^ Tile<DP>::f(r);
            voff[i] = 8 * c < d ? static_cast<uint32_t>(r) * static_cast<uint32_t>(2 * s) + 16 * c : 0x80000000u;
        }
    }
    // row0 < rows; tile: byte address
    __device__ __forceinline__ void load(int row0, uint32_t tile) const {
        const int left = rows - row0 < kTile ? rows - row0 : kTile;
        const u32x4 d = descriptor(base + static_cast<int64_t>(row0) * stride,
                                   static_cast<uint32_t>(left - 1) * static_cast<uint32_t>(2 * stride) + row_bytes);
        const uint32_t lds = tile + wave_id() * 64 % NT * 16;
        uint32_t v = voff[0];
        asm volatile("" : "+v"(v));  // (the sums below are not kept in registers)
#pragma unroll
        for (int i = 0; i < N; ++i)
            load_lds16(lds + i * NT * 16, kSteps ? v + i * (NT / Tile<DP>::CPR) * static_cast<uint32_t>(2 * stride) : voff[kSteps ? 0 : i], d);
    }
};
// One 4-byte value of each of kTile rows (row0 < rows), every wave loading all
// of them.
__device__ __forceinline__ void load_values(const void* p, int row0, int rows, uint32_t lds) {
    const int left = rows - row0 < kTile ? rows - row0 : kTile;
    load_lds4(lds, 4 * lane_id(), descriptor(static_cast<const char*>(p) + 4 * static_cast<int64_t>(row0), 4 * left));
}

// The documents of kTile positions from pos0 on, positions clamped to 0 .. sk - 1.
__device__ __forceinline__ void load_docs(const int32_t* docs, int pos0, int sk, uint32_t lds) {
    int p = pos0 + lane_id();
    p = p < 0 ? 0 : (p < sk ? p : sk - 1);
    load_lds4(lds, 4 * static_cast<uint32_t>(p), descriptor(docs, 4 * static_cast<uint32_t>(sk)));
}

// Moves one tile of kTile rows from memory through registers to LDS.  Rows
// past `rows` and values past the head size come as zeros, whatever memory
// holds there.
template <int DP, int NT>
struct Loader {
    static constexpr int N = kTile * Tile<DP>::CPR / NT;
    static_assert(N * NT == kTile * Tile<DP>::CPR, "whole chunks per thread");
    uint32_t voff[N];
    int lds[N];
    u32x4 reg[N];
    const bf16_t* base;  // row 0 of the sequence
    int64_t stride;      // elements per row
    int rows;
    uint32_t row_bytes;

    __device__ __forceinline__ void init(const bf16_t* p, int64_t s, int nrows, int d) {
        base = p;
        stride = s;
        rows = nrows;
        row_bytes = 2 * d;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int id = static_cast<int>(threadIdx.x) % NT + i * NT;
            const int r = id / Tile<DP>::CPR, c = id % Tile<DP>::CPR;
            voff[i] = 8 * c < d ? static_cast<uint32_t>(r) * static_cast<uint32_t>(2 * s) + 16 * c : 0x80000000u;
            lds[i] = Tile<DP>::at(r, c);
        }
    }
    __device__ __forceinline__ void load(int row0) {
        const int left = rows - row0 < kTile ? rows - row0 : kTile;
        const uint32_t bytes = left > 0 ? static_cast<uint32_t>(left - 1) * static_cast<uint32_t>(2 * stride) + row_bytes : 0;
        const auto r = rsrc(base + static_cast<int64_t>(row0) * stride, bytes);
        // non-temporal: the cache is read once (32 caches of 16384 keys: 312 -> 293 us)
#pragma unroll
        for (int i = 0; i < N; ++i)
            reg[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, voff[i], 0, 2));
    }
    __device__ __forceinline__ void store(bf16_t* tile) {
#pragma unroll
        for (int i = 0; i < N; ++i) *reinterpret_cast<u32x4*>(tile + lds[i]) = reg[i];
    }
};

// A operand read along the rows of the tile at byte address `tile`: rows 32 rb
// + lane % 32, columns 16 t + 8 half .. + 7.
template <int DP>
struct RowFrag {
    uint32_t off[DP / 16];
    __device__ __forceinline__ void init() {
        const int r = lane_id() & 31, h = lane_id() >> 5;
#pragma unroll
        for (int t = 0; t < DP / 16; ++t) off[t] = 2 * Tile<DP>::at(r, 2 * t + h);
    }
    __device__ __forceinline__ bf16x8 read(uint32_t tile, int rb, int t) const {
        return __builtin_bit_cast(bf16x8, *(__attribute__((address_space(3))) const u32x4*)(off[t] + (tile + 64 * rb * Tile<DP>::LD)));
    }
};

// A operand read across the rows (the tile's transpose): columns 32 dt + lane
// % 32, contracted rows 16 t + 8 (e / 4) + 4 half + e % 4 for e = 0 .. 7.
// ds_read_b64_tr_b16: in every 16 lanes, lane r supplies the address of 4
// values (k + r / 4, c + 4 (r % 4)) and lane i receives (k .. k + 3, c + i).
template <int DP>
struct ColFrag {
    uint32_t off[DP / 32][2];
    __device__ __forceinline__ void init() {
        const int g = lane_id() >> 4, r = lane_id() & 15, h = g >> 1;
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = 8 * e + 4 * h + (r >> 2);
                const int col = 32 * dt + 16 * (g & 1) + 4 * (r & 3);
                off[dt][e] = 2 * (Tile<DP>::at(row, col >> 3) + (col & 7));
            }
    }
    __device__ __forceinline__ bf16x8 read(uint32_t tile, int t, int dt) const {
        const uint32_t at = tile + 32 * t * Tile<DP>::LD;
        const s16x4 lo = tr(off[dt][0] + at), hi = tr(off[dt][1] + at);
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    __device__ static __forceinline__ s16x4 tr(uint32_t at) {
        return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at));
    }
};

__device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ f32x16 splat(float x) {
    f32x16 v;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = x;
    return v;
}

// Results 8 t .. 8 t + 7 of a product, rounded to bf16 (nearest even), as the
// B operand of step t of the next product.
__device__ __forceinline__ bf16x8 pack(const f32x16& s, int t) {
    const u32x4 u = {f32x2_to_bf16x2(s[8 * t], s[8 * t + 1]), f32x2_to_bf16x2(s[8 * t + 2], s[8 * t + 3]),
                     f32x2_to_bf16x2(s[8 * t + 4], s[8 * t + 5]), f32x2_to_bf16x2(s[8 * t + 6], s[8 * t + 7])};
    return __builtin_bit_cast(bf16x8, u);
}

// B operand read straight from memory: row `row` of a row-major matrix (zero
// where !ok), columns 16 t + 8 half .. + 7.
template <int DP>
__device__ __forceinline__ void load_rows(bf16x8 (&f)[DP / 16], const bf16_t* base, int64_t stride, int row, bool ok,
                                          int d) {
    const int h = lane_id() >> 5;
    const bf16_t* p = base + static_cast<int64_t>(row) * stride + 8 * h;
#pragma unroll
    for (int t = 0; t < DP / 16; ++t) {
        u32x4 v = {0u, 0u, 0u, 0u};
        if (ok && 16 * t + 8 * h < d) v = *reinterpret_cast<const u32x4*>(p + 16 * t);
        f[t] = __builtin_bit_cast(bf16x8, v);
    }
}

// The values are in registers from here on (else the compiler waits for them
// inside the loop that uses them, and with them for every direct load).
template <int N>
__device__ __forceinline__ void settle(bf16x8 (&f)[N]) {
#pragma unroll
    for (int t = 0; t < N; ++t) {
        u32x4 v = __builtin_bit_cast(u32x4, f[t]);
        asm volatile("" : "+v"(v));
        f[t] = __builtin_bit_cast(bf16x8, v);
    }
}

// f(integral_constant<int, I>) for I = A .. B - 1.
template <int A, int... I, typename F>
__device__ __forceinline__ void each_of(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, A + I>{}), ...);
}
template <int A, int B, typename F>
__device__ __forceinline__ void each(F&& f) {
    each_of<A>(f, std::make_integer_sequence<int, (B > A ? B - A : 0)>{});
}

// Nothing is scheduled across: keeps matrix instructions, the LDS reads of
// later ones and the vector work between them in the order written.
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

// Stores a transposed result (column l % 32 = a row of the output, rows = its
// columns 32 dt ..): the halves swap pieces so that every lane stores 16
// contiguous bytes.
template <int DP>
__device__ __forceinline__ void store_rows(const f32x16 (&o)[DP / 32], float mul, bf16_t* row, bool ok, int d) {
    const int h = lane_id() >> 5;
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int i = 8 * g;
            // pieces of columns 16 g + 4 half (lo) and 16 g + 8 + 4 half (hi)
            const u32x2 lo = {f32x2_to_bf16x2(o[dt][i] * mul, o[dt][i + 1] * mul),
                              f32x2_to_bf16x2(o[dt][i + 2] * mul, o[dt][i + 3] * mul)};
            const u32x2 hi = {f32x2_to_bf16x2(o[dt][i + 4] * mul, o[dt][i + 5] * mul),
                              f32x2_to_bf16x2(o[dt][i + 6] * mul, o[dt][i + 7] * mul)};
            // swap exchanges the first operand's upper half with the second's
            // lower half: half 0 then holds lo of both halves (columns 16 g ..
            // 16 g + 7), half 1 hi of both
            const auto x = __builtin_amdgcn_permlane32_swap(lo.x, hi.x, false, false);
            const auto y = __builtin_amdgcn_permlane32_swap(lo.y, hi.y, false, false);
            const u32x4 v = {x[0], y[0], x[1], y[1]};
            const int col = 32 * dt + 16 * g + 8 * h;
            if (ok && col < d) *reinterpret_cast<u32x4*>(row + col) = v;
        }
}

// What one sequence of the batch sees.
struct Seq {
    int n;      // keys (and positions) below this one are real, and within reach of a query
    int start;  // position of query 0
    int sq;     // queries from there on
    int pre;    // keys below this one are seen by every query
    int b;
    const int32_t* doc;
};
__device__ __forceinline__ Seq sequence(Args a, int b) {
    Seq s;
    s.b = b;
    s.n = a->sk;
    if (a->lengths) {
        const int len = a->lengths[b];
        s.n = len < 0 ? 0 : (len < a->sk ? len : a->sk);
    }
    int st = a->sk - a->sq;
    if (a->starts) st = a->starts[b];
    s.start = st < -kMaxPos ? -kMaxPos : (st > kMaxPos ? kMaxPos : st);
    s.sq = a->sq;
    s.pre = 0;
    if (a->prefix) {
        const int p = a->prefix[b];
        s.pre = p < 0 ? 0 : (p < s.n ? p : s.n);
    }
    s.doc = a->documents ? a->documents + static_cast<int64_t>(b) * a->doc_b : nullptr;
    // keys past the last query's reach are not read (0 times what lies there
    // need not be 0: a cache may hold anything past its last position)
    if (a->causal || a->window) {
        int end = s.start + s.sq;
        if (!a->causal) end += a->window - 1;
        if (end < s.pre) end = s.pre;
        if (end < s.n) s.n = end;
    }
    return s;
}
// Leaves out the queries before the first and past the last that see any key
// (dK and dV, which read every query's rows, must not read theirs); returns how
// many were left out in front.  With a prefix every query sees keys, but for
// those past the last key's window if the prefix holds other documents only.
__device__ __forceinline__ int only_queries_that_see(Seq& s, Args a) {
    if (s.pre > 0 || (!a->causal && !a->window)) return 0;
    int lead = (a->causal ? 0 : 1 - a->window) - s.start;
    if (a->window && s.n + a->window - 1 - s.start < s.sq) s.sq = s.n + a->window - 1 - s.start;
    if (lead > s.sq) lead = s.sq;
    if (lead < 0) lead = 0;
    s.start += lead;
    s.sq -= lead;
    return lead;
}
__device__ __forceinline__ int doc_of(const Seq& s, Args a, int pos) {
    const int p = pos < 0 ? 0 : (pos < a->sk ? pos : a->sk - 1);
    return s.doc[p];
}
// A query's position is real: with lengths, positions past the length are
// padding and see nothing.
__device__ __forceinline__ bool real_row(const Seq& s, Args a, int pos) {
    return a->lengths == nullptr || pos < s.n;
}

// One query: its position and document.  The keys it sees outside the
// document rule are lo <= j <= hi, or j < pre.
struct Row {
    int pos, doc;
};
__device__ __forceinline__ Row row_of(const Seq& s, Args a, int pos) {
    return {pos, s.doc ? doc_of(s, a, pos) : 0};
}
// Which of the 32 results a lane holds of a tile are seen, as bits: result (kb,
// i) is bit place(i) of word kb, its row 32 kb + place(i) rows past the lane
// half's first.
struct Bits {
    uint32_t w[2];
};
__device__ constexpr int place(int i) { return 8 * (i / 4) + i % 4; }
// Rows lo .. hi, and those below pre.
__device__ __forceinline__ Bits bits_of(int lo, int hi, int pre) {
    auto below = [](int n) { return n <= 0 ? uint64_t{0} : (n >= 64 ? ~uint64_t{0} : (uint64_t{1} << n) - 1); };
    const uint64_t m = (below(hi + 1) & ~below(lo)) | below(pre);
    return {{static_cast<uint32_t>(m), static_cast<uint32_t>(m >> 32)}};
}
// x where result (kb, i) is seen, `other` elsewhere: two instructions, and a
// NaN that is not seen leaves nothing behind.
__device__ __forceinline__ float where(const Bits& m, int kb, int i, float x, float other) {
    const uint32_t on = static_cast<uint32_t>(__builtin_amdgcn_sbfe(static_cast<int>(m.w[kb]), place(i), 1));
    return __uint_as_float((__float_as_uint(x) & on) | (__float_as_uint(other) & ~on));
}
// The keys that query r sees of the tile whose first key of the lane's half is
// j0, but for the document rule.
__device__ __forceinline__ Bits keys_seen(const Row& r, const Seq& s, Args a, int j0) {
    a = again(a);
    int lo = 0, hi = s.n - 1;
    if (a->causal && r.pos < hi) hi = r.pos;
    if (a->window) {
        if (r.pos - a->window + 1 > lo) lo = r.pos - a->window + 1;
        if (r.pos + a->window - 1 < hi) hi = r.pos + a->window - 1;
    }
    return bits_of(lo - j0, hi - j0, s.pre - j0);
}

// Whether a block of queries at positions [p0, p1] (documents in [d0, d1])
// sees any key of [j0, j1] (documents in [e0, e1]), and whether every one of
// those queries sees every one of those keys.  j1 is below n.  `some` may
// be too generous (elements are then masked one by one), never too strict.
struct Sight {
    bool some, all;
};
__device__ __forceinline__ Sight sight(const Seq& s, Args a, int p0, int p1, int d0, int d1, int j0, int j1,
                                       int e0, int e1) {
    const bool span_some = (!a->causal || j0 <= p1) && (!a->window || (j1 > p0 - a->window && j0 < p1 + a->window));
    const bool span_all = (!a->causal || j1 <= p0) && (!a->window || (p1 - j0 < a->window && j1 - p0 < a->window));
    Sight r;
    r.some = j0 <= j1 && (span_some || j0 < s.pre);
    r.all = span_all || j1 < s.pre;
    if (s.doc) {
        r.some = r.some && e0 <= d1 && d0 <= e1;
        r.all = r.all && e0 == e1 && d0 == d1 && e0 == d0;
    }
    return r;
}

// Lowest and highest document of the positions [p0, p1] of a sequence, over
// the wave.
__device__ __forceinline__ void doc_range(const Seq& s, Args a, int p0, int p1, int& lo, int& hi) {
    lo = 0x7fffffff;
    hi = static_cast<int>(0x80000000u);
    if (!s.doc) return;
    for (int p = p0 + lane_id(); p <= p1; p += 64) {
        const int e = doc_of(s, a, p);
        lo = e < lo ? e : lo;
        hi = e > hi ? e : hi;
    }
#pragma unroll
    for (int m = 32; m; m >>= 1) {
        const int x = __shfl_xor(lo, m), y = __shfl_xor(hi, m);
        lo = x < lo ? x : lo;
        hi = y > hi ? y : hi;
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    hi = __builtin_amdgcn_readfirstlane(hi);
}

// A run of query positions with its documents.
struct Span {
    int p0, p1, d0, d1;
};
__device__ __forceinline__ Span query_span(const Seq& s, Args a, int i0, int i1) {
    Span r;
    r.p0 = s.start + i0;
    r.p1 = s.start + i1 - 1;
    if (a->lengths && r.p1 >= s.n) r.p1 = s.n - 1;
    doc_range(s, a, r.p0, r.p1, r.d0, r.d1);
    return r;
}

// Keeps what only the tests of tiles use in vector registers: the scalar ones
// would run out inside the loops.
__device__ __forceinline__ void in_vectors(Span& r) {
    asm volatile("" : "+v"(r.p0), "+v"(r.p1), "+v"(r.d0), "+v"(r.d1));
}

// The key tiles a workgroup's queries see, in order.  64 tiles are tested at
// a time, one per lane; the answers stay in scalar registers.
struct KeyTiles {
    uint64_t wg, some, all;
    int base, end;
    int turns = 1, turn = 0;  // tiles t with t % turns = turn (a power of two)
    __device__ __forceinline__ void fill(const Seq& s, Args a, const Span& g, const Span& w) {
        a = again(a);
        const int t = base + lane_id(), j0 = t * kTile;
        int j1 = j0 + kTile - 1;
        if (j1 >= s.n) j1 = s.n - 1;
        int2 e = {0, 0};
        if (s.doc && t < a->n_tiles) e = a->doc_tiles[static_cast<int64_t>(s.b) * a->n_tiles + t];
        const bool in = t < end && (t & (turns - 1)) == turn;
        const Sight x = sight(s, a, g.p0, g.p1, g.d0, g.d1, j0, j1, e.x, e.y);
        const Sight y = sight(s, a, w.p0, w.p1, w.d0, w.d1, j0, j1, e.x, e.y);
        wg = __ballot(in && x.some);
        some = __ballot(in && w.p0 <= w.p1 && y.some);
        all = __ballot(in && y.all && j0 + kTile <= s.n);
    }
    // of the tiles first .. last - 1
    __device__ __forceinline__ void init(const Seq& s, Args a, const Span& g, const Span& w, int first = 0,
                                         int last = 0x7fffffff) {
        int lo = 0, hi = s.n - 1;
        if (a->causal && g.p1 < hi) hi = g.p1;
        if (a->window) {
            if (g.p0 - a->window + 1 > lo) lo = g.p0 - a->window + 1;
            if (g.p1 + a->window - 1 < hi) hi = g.p1 + a->window - 1;
        }
        if (s.pre > 0) {
            lo = 0;
            if (s.pre - 1 > hi) hi = s.pre - 1;
        }
        if (g.p0 > g.p1) hi = -1;
        base = __builtin_amdgcn_readfirstlane(lo / kTile);
        end = __builtin_amdgcn_readfirstlane(hi < 0 ? 0 : hi / kTile + 1);
        base = base > first ? base : first;
        end = end < last ? end : last;
        wg = some = all = 0;
        if (base < end) fill(s, a, g, w);
    }
    // Next tile, or -1.  mode: 0 this wave sees nothing of it, 1 some, 2 all.
    __device__ __forceinline__ int next(const Seq& s, Args a, const Span& g, const Span& w, int& mode) {
        while (wg == 0) {
            base += 64;
            if (base >= end) return -1;
            fill(s, a, g, w);
        }
        const int i = __builtin_ctzll(wg);
        wg &= wg - 1;
        mode = !((some >> i) & 1) ? 0 : (((all >> i) & 1) ? 2 : 1);
        return base + i;
    }
};

// Queries that see one key: those at positions lo .. hi of its document.
struct Col {
    int pos, lo, hi, doc;
};
__device__ __forceinline__ Col col_of(const Seq& s, Args a, int j) {
    Col r;
    r.pos = j;
    r.lo = s.start;
    r.hi = s.start + s.sq - 1;
    if (a->lengths && r.hi >= s.n) r.hi = s.n - 1;
    if (j >= s.pre) {
        if (a->causal && j > r.lo) r.lo = j;
        if (a->window) {
            if (j - a->window + 1 > r.lo) r.lo = j - a->window + 1;
            if (j + a->window - 1 < r.hi) r.hi = j + a->window - 1;
        }
    }
    if (j >= s.n) r.hi = r.lo - 1;
    r.doc = s.doc ? doc_of(s, a, j) : 0;
    return r;
}

// The tiles of kTile queries that see a workgroup's keys, as KeyTiles.
struct QueryTiles {
    uint64_t wg, some, all;
    int base, end, rows;
    __device__ __forceinline__ void fill(const Seq& s, Args a, const Span& g, const Span& w) {
        a = again(a);
        const int i0 = (base + lane_id()) * kTile;
        const int i1 = i0 + kTile < rows ? i0 + kTile : rows;
        const int p0 = s.start + i0, p1 = s.start + i1 - 1;
        int2 e = {0, 0};
        if (s.doc && i0 < rows) {
            const int x = p0 < 0 ? 0 : (p0 < a->sk ? p0 : a->sk - 1), y = p1 < 0 ? 0 : (p1 < a->sk ? p1 : a->sk - 1);
            const int2* docs = a->doc_tiles + static_cast<int64_t>(s.b) * a->n_tiles;
            const int2 ex = docs[x / kTile], ey = docs[y / kTile];
            e = {ex.x < ey.x ? ex.x : ey.x, ex.y > ey.y ? ex.y : ey.y};
        }
        const bool in = i0 < rows;
        const Sight x = sight(s, a, p0, p1, e.x, e.y, g.p0, g.p1, g.d0, g.d1);
        const Sight y = sight(s, a, p0, p1, e.x, e.y, w.p0, w.p1, w.d0, w.d1);
        wg = __ballot(in && x.some);
        some = __ballot(in && y.some);
        all = __ballot(in && y.all && i0 + kTile <= rows);
    }
    // rows: queries that are real
    __device__ __forceinline__ void init(const Seq& s, Args a, const Span& g, const Span& w) {
        rows = s.sq;
        if (a->lengths && s.n - s.start < rows) rows = s.n - s.start;
        int lo = 0, hi = rows - 1;
        if (g.p0 >= s.pre) {
            if (a->causal && g.p0 - s.start > lo) lo = g.p0 - s.start;
            if (a->window) {
                if (g.p0 - a->window + 1 - s.start > lo) lo = g.p0 - a->window + 1 - s.start;
                if (g.p1 + a->window - 1 - s.start < hi) hi = g.p1 + a->window - 1 - s.start;
            }
        }
        if (g.p0 > g.p1) hi = -1;
        base = __builtin_amdgcn_readfirstlane(lo / kTile);
        end = __builtin_amdgcn_readfirstlane(hi < 0 ? 0 : hi / kTile + 1);
        wg = some = all = 0;
        if (base < end) fill(s, a, g, w);
    }
    __device__ __forceinline__ int next(const Seq& s, Args a, const Span& g, const Span& w, int& mode) {
        while (wg == 0) {
            base += 64;
            if (base >= end) return -1;
            fill(s, a, g, w);
        }
        const int i = __builtin_ctzll(wg);
        wg &= wg - 1;
        mode = !((some >> i) & 1) ? 0 : (((all >> i) & 1) ? 2 : 1);
        return base + i;
    }
};

// Scores in units of log 2 from the product x = q . k, as p = exp2(z - lse2).
// cap: z = cap log2e tanh(scale x / cap), with tanh(y) = 1 - 2 r, r = 1 / (exp(2
// y) + 1).  That is exact to float32 rounding of the cap, not of the score: near
// zero r is 1/2 and the score what is left of the difference, off by about 2^-23
// of the cap (6e-6 at 30, 1.3e-5 at 64, but 0.01 at 1e5).  Above kMaxPlainCap
// scores below a quarter of the cap are taken from the series y - y^3 / 3 + 2
// y^5 / 15 - ..., whose first term left out is 9e-9 of the sum there; packed
// documents of 16384 tokens take 219 us forward and 512 backward so, and 162 and
// 387 up to it; a step over 32 caches of up to 16384 keys 296 and 288.
constexpr float kMaxPlainCap = 64.0f;
struct Score {
    float c;      // scale * log2e (no cap) or 2 scale log2e / cap
    float a;      // cap * log2e
    float slope;  // slope * log2e
    float line, over;  // kWide: scale * log2e, scale / cap
};
template <int MOD>
__device__ __forceinline__ Score score_of(Args a, int head) {
    // (a product past float32's range is that range's end: 0 times it is 0)
    constexpr float most = 3.4028234663852886e38f;
    Score s;
    s.a = fminf(a->softcap * kLog2e, most);
    s.line = fminf(a->scale * kLog2e, most);
    s.c = (MOD & kCap) ? fminf(2.0f * (s.line / a->softcap), most) : s.line;
    s.over = a->scale / a->softcap;
    s.slope = (MOD & kBias) && a->slopes ? a->slopes[head] * kLog2e : 0.0f;
    return s;
}
// The capped score of x without a bias, and r.
template <int MOD>
__device__ __forceinline__ float capped(const Score& s, float x, float& r) {
    r = __builtin_amdgcn_rcpf(exp2_fast(x * s.c) + 1.0f);
    if constexpr (!(MOD & kWide)) return fmaf(-2.0f * s.a, r, s.a);
    const float y = x * s.over, w = y * y;
    const float near = fmaf(w * fmaf(w, fmaf(w, fmaf(w, 62.0f / 2835.0f, -17.0f / 315.0f), 2.0f / 15.0f), -1.0f / 3.0f),
                            x * s.line, x * s.line);
    return w < 0.0625f ? near : s.a * fmaf(-2.0f, r, 1.0f);
}
// dist: |query position - key|.
template <int MOD>
__device__ __forceinline__ float score(const Score& s, float x, float dist) {
    float z, r;
    if constexpr (MOD & kCap) z = capped<MOD>(s, x, r);
    else z = x * s.c;
    if constexpr (MOD & kBias) z = fmaf(-s.slope, dist, z);
    return z;
}

// The extras of a call.  Without any, dK and dV start their products from -lse /
// scale, which passes float32's range at scales near 2^-124: small ones go the
// way of a bias of zero, which subtracts lse afterwards.
constexpr float kMinPlainScale = 0x1p-100f;
inline int score_extras(const AttnArgs& a) {
    if (a.softcap > kMaxPlainCap) return kCap | kBias | kWide;
    return (a.softcap > 0.0f ? kCap : 0) | (a.slopes || a.scale < kMinPlainScale ? kBias : 0);
}

}  // namespace attn
}  // namespace muon

// fn<DP, MOD>(a, stream) for the head size and the extras of the scores
#define MUON_ATTN_DISPATCH(fn, a, stream)                                                     \
    do {                                                                                      \
        const int mod = score_extras(a);                                                      \
        const int size = (a).d <= 64 ? 64 : ((a).d <= 96 ? 96 : 128);                         \
        switch (size + mod) {                                                                 \
            case 64: fn<64, 0>(a, stream); break;                                             \
            case 65: fn<64, 1>(a, stream); break;                                             \
            case 66: fn<64, 2>(a, stream); break;                                             \
            case 67: fn<64, 3>(a, stream); break;                                             \
            case 71: fn<64, 7>(a, stream); break;                                             \
            case 96: fn<96, 0>(a, stream); break;                                             \
            case 97: fn<96, 1>(a, stream); break;                                             \
            case 98: fn<96, 2>(a, stream); break;                                             \
            case 99: fn<96, 3>(a, stream); break;                                             \
            case 103: fn<96, 7>(a, stream); break;                                            \
            case 128: fn<128, 0>(a, stream); break;                                           \
            case 129: fn<128, 1>(a, stream); break;                                           \
            case 130: fn<128, 2>(a, stream); break;                                           \
            case 131: fn<128, 3>(a, stream); break;                                           \
            case 135: fn<128, 7>(a, stream); break;                                           \
        }                                                                                     \
    } while (0)
