// Embedding: out[i] = scale * table[token[i]], and the table's gradient
// dtable[v] = scale * sum of dout[i] over the i with token[i] = v, summed in
// float32 in one fixed order (that of i within a window, windows by fours),
// without atomics on floating values.
//
// Both are bound by memory.  The gradient sorts the tokens first (k_embed_sort,
// stable), then sums windows of sorted entries and writes the rows of tokens
// that do not occur (k_embed_sum), so that a token's work is spread over many
// workgroups however often it occurs, and last joins the runs that cross
// windows (k_embed_join).  Few tokens take one launch (k_embed_direct).
//
// 65536 tokens, 50304 x 768 float32 rows: forward 29 us (5 TB/s); gradient 66 to
// 78: sort 19, sums and zeros 39 (255 MB), joins 9.
#include "../../include/muon.h"
#include "lm_common.hpp"

namespace muon {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <typename T, int V>
__device__ __forceinline__ void load_e(const T* p, float (&x)[V]) {
    if constexpr (V == 1) {
        if constexpr (sizeof(T) == 2) x[0] = bf16_to_f32(p[0]);
        else x[0] = p[0];
    } else if constexpr (sizeof(T) == 2 && V == 4) {
        const u32x2 u = *reinterpret_cast<const u32x2*>(p);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    } else if constexpr (sizeof(T) == 2) {
        const u32x4 u = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    } else if constexpr (V == 4) {
        const f32x4 u = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = u[i];
    } else {
        const f32x4 u = reinterpret_cast<const f32x4*>(p)[0], v = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = u[i];
            x[4 + i] = v[i];
        }
    }
}
template <typename T, int V>
__device__ __forceinline__ void store_e(T* p, const float (&x)[V]) {
    if constexpr (V == 1) {
        if constexpr (sizeof(T) == 2) p[0] = f32_to_bf16(x[0]);
        else p[0] = x[0];
    } else if constexpr (sizeof(T) == 2 && V == 4) {
        const u32x2 u = {f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3])};
        __builtin_nontemporal_store(u, reinterpret_cast<u32x2*>(p));
    } else if constexpr (sizeof(T) == 2) {
        const u32x4 u = {f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]), f32x2_to_bf16x2(x[4], x[5]),
                         f32x2_to_bf16x2(x[6], x[7])};
        __builtin_nontemporal_store(u, reinterpret_cast<u32x4*>(p));
    } else {
        __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]}, reinterpret_cast<f32x4*>(p));
        if constexpr (V == 8) __builtin_nontemporal_store(f32x4{x[4], x[5], x[6], x[7]}, reinterpret_cast<f32x4*>(p) + 1);
    }
}

__device__ __forceinline__ int64_t token_at(const EmbedArgs& a, int64_t i) {
    return a.tokens64 ? static_cast<const int64_t*>(a.tokens)[i] : static_cast<const int32_t*>(a.tokens)[i];
}

// One row per 2^k lanes; a token outside the table gives a row of NaN.
template <typename TS, typename TD, int V>
__global__ __launch_bounds__(256) void k_embed(const EmbedArgs a, int lanes) {
    const int l = threadIdx.x % lanes, per = 256 / lanes;
    const int pieces = a.width / V;
    const int64_t i = static_cast<int64_t>(block_place()) * per + threadIdx.x / lanes;
    if (i >= a.n) return;
    const int64_t t = token_at(a, i);
    const bool known = t >= 0 && t < a.vocab;
    const TS* src = static_cast<const TS*>(a.src) + (known ? t : 0) * a.width;
    TD* dst = static_cast<TD*>(a.dst) + i * a.width;
    for (int c = l; c < pieces; c += lanes) {
        float x[V];
        if (known) {
            load_e<TS, V>(src + c * V, x);
#pragma unroll
            for (int k = 0; k < V; ++k) x[k] *= a.scale;
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) x[k] = __builtin_nanf("");
        }
        store_e<TD, V>(dst + c * V, x);
    }
}

// Stable sort of the tokens: workgroup g owns the `span` table rows from g
// span.  Its 16 waves take 16 consecutive parts of the tokens and look through
// them once: they count (per wave and row, and the tokens of lower rows, which
// is where the workgroup's entries begin) and list their own in LDS; then they
// place the listed ones.  A wave whose list is full (a table of few rows, or
// one token everywhere) looks through its part again instead.  No workgroup
// waits for another one.  Every workgroup reads all the tokens from the
// caches: 65536 of them are 512 KiB.
constexpr int kSortWaves = 16;
constexpr int kSortSpan = 512;   // table rows per workgroup at most
constexpr int kSortList = 1024;  // entries a wave can list
template <bool T64>
__global__ __launch_bounds__(64 * kSortWaves) void k_embed_sort(const EmbedArgs a, int span) {
    __shared__ int32_t cnt[kSortWaves][kSortSpan];
    __shared__ uint32_t list[kSortWaves][kSortList];  // place in the part * kSortSpan + row
    __shared__ int32_t below[kSortWaves];
    __shared__ int32_t wsum[kSortWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t lo = static_cast<int64_t>(block_place()) * span;
    if (lo >= a.vocab) return;
    const uint32_t base32 = static_cast<uint32_t>(lo);  // vocab is below 2^31
    const uint32_t rows = static_cast<uint32_t>(lo + span <= a.vocab ? span : a.vocab - lo);
    for (int i = threadIdx.x; i < kSortWaves * kSortSpan; i += blockDim.x) (&cnt[0][0])[i] = 0;
    __syncthreads();
    const int64_t part = ((a.n + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
    const int64_t i0 = wave * part, i1 = i0 + part < a.n ? i0 + part : a.n;
    constexpr int U = 16;
    // tokens as 32 bits (all ones: outside the table), all of a batch in flight
    auto load = [&](int64_t at) {
        if constexpr (T64) return static_cast<const u32x2*>(a.tokens)[at];
        else return static_cast<const uint32_t*>(a.tokens)[at];
    };
    auto narrow = [](auto w) -> uint32_t {
        if constexpr (T64) return w.y == 0 ? w.x : 0xffffffffu;
        else return w;
    };
    // f(place, token) for the part's tokens, 64 at a time
    auto walk = [&](auto&& f) {
        int64_t i = i0;
        for (; i + 64 * U <= i1; i += 64 * U) {
            decltype(load(0)) t[U];
#pragma unroll
            for (int k = 0; k < U; ++k) t[k] = load(i + 64 * k + lane);
#pragma unroll
            for (int k = 0; k < U; ++k) f(i + 64 * k + lane, narrow(t[k]));
        }
        for (; i < i1; i += 64) f(i + lane, i + lane < i1 ? narrow(load(i + lane)) : 0xffffffffu);
    };
    int32_t low = 0, listed = 0;
    walk([&](int64_t i, uint32_t t) {
        low += __popcll(__ballot(t < base32));
        const bool mine = t - base32 < rows;
        const uint64_t all = __ballot(mine);
        if (all == 0) return;
        if (mine) {
            atomicAdd(&cnt[wave][t - base32], 1);
            const int at = listed + __popcll(all & ((1ull << lane) - 1));
            if (at < kSortList) list[wave][at] = static_cast<uint32_t>(i - i0) * kSortSpan + (t - base32);
        }
        listed += __popcll(all);
    });
    if (lane == 0) below[wave] = low;
    __syncthreads();
    // thread x < kSortSpan: row x's entries per wave -> where they begin
    int32_t base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) base += below[w];
    const int x = threadIdx.x;
    if (x < kSortSpan)
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            const int32_t c = cnt[w][x];
            cnt[w][x] = total;
            total += c;
        }
    int32_t incl = total;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const int32_t y = __shfl_up(incl, m);
        if (lane >= m) incl += y;
    }
    if (lane == 63) wsum[wave] = incl;
    __syncthreads();
    for (int w = 0; w < wave; ++w) base += wsum[w];
    const int32_t first = base + incl - total;
    if (x < kSortSpan) {
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) cnt[w][x] += first;
        if (x < static_cast<int>(rows)) a.offset[lo + x] = first;
        if (x == static_cast<int>(rows) - 1 && lo + rows == a.vocab) a.offset[a.vocab] = first + total;
    }
    __syncthreads();
    // the lanes that hold the first one's row take places in order, and so on
    auto place = [&](int64_t i, int32_t y, bool mine) {
        uint64_t left = __ballot(mine);
        while (left) {
            const int lead = __builtin_ctzll(left);
            const int32_t who = __builtin_amdgcn_readlane(y, lead);
            const bool same = mine && y == who;
            const uint64_t all = __ballot(same);
            const int32_t at = cnt[wave][who];
            if (same) {
                const int32_t p = at + __popcll(all & ((1ull << lane) - 1));
                a.perm[p] = static_cast<int32_t>(i);
                a.ids[p] = static_cast<int32_t>(lo) + y;
            }
            if (lane == lead) cnt[wave][who] = at + __popcll(all);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            left &= ~all;
        }
    };
    if (listed <= kSortList && part <= (int64_t{1} << 32) / kSortSpan) {
        for (int e = 0; e < listed; e += 64) {
            const bool mine = e + lane < listed;
            const uint32_t u = mine ? list[wave][e + lane] : 0;
            place(i0 + u / kSortSpan, static_cast<int32_t>(u % kSortSpan), mine);
        }
    } else {
        walk([&](int64_t i, uint32_t t) { place(i, static_cast<int32_t>(t - base32), t - base32 < rows); });
    }
}

// The first workgroups: sums of the runs of equal tokens of one window.  A run
// inside the window is written as the table's row; where the first and the
// last run cross the window's border, their sums go to part rows 2 w and
// 2 w + 1.  The workgroups after them write the rows of tokens that do not
// occur, kZeroRows of the table each (in one launch, because the sums wait
// for memory and the zeros do not).
constexpr int kZeroRows = 32;
constexpr int kMaxWindow = 32;
template <typename TS, typename TD, int V>
__global__ __launch_bounds__(256) void k_embed_sum(const EmbedArgs a, int windows) {
    __shared__ int32_t s_perm[kMaxWindow], s_ids[kMaxWindow + 2], s_off[kZeroRows + 1];
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    float acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.0f;
    const int64_t block = block_place();
    if (block >= windows) {
        const int64_t r0 = (block - windows) * kZeroRows;
        if (r0 >= a.vocab) return;
        const int rows = a.vocab - r0 < kZeroRows ? static_cast<int>(a.vocab - r0) : kZeroRows;
        if (static_cast<int>(threadIdx.x) <= rows) s_off[threadIdx.x] = a.offset[r0 + threadIdx.x];
        __syncthreads();
        if (c >= a.width) return;
        for (int r = 0; r < rows; ++r)
            if (s_off[r] == s_off[r + 1]) store_e<TD, V>(static_cast<TD*>(a.dst) + (r0 + r) * a.width + c, acc);
        return;
    }
    const int64_t total = a.offset[a.vocab], w0 = block * a.window;
    if (w0 >= total) return;
    const int n = total - w0 < a.window ? static_cast<int>(total - w0) : a.window;
    if (static_cast<int>(threadIdx.x) < n + 2) {
        // with the neighbours on either side (-1: none)
        const int64_t i = w0 + threadIdx.x - 1;
        const bool in = i >= 0 && i < total;
        s_ids[threadIdx.x] = in ? a.ids[i] : -1;
        if (threadIdx.x >= 1 && static_cast<int>(threadIdx.x) <= n) s_perm[threadIdx.x - 1] = a.perm[i];
    }
    __syncthreads();
    if (c >= a.width) return;
    const TS* src = static_cast<const TS*>(a.src) + c;
    bool crosses = s_ids[0] == s_ids[1];  // the current run began before the window
    constexpr int U = 8;
    for (int e0 = 0; e0 < n; e0 += U) {
        float x[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e = e0 + u < n ? e0 + u : n - 1;
            load_e<TS, V>(src + static_cast<int64_t>(__builtin_amdgcn_readfirstlane(s_perm[e])) * a.width, x[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e = e0 + u;
            if (e < n) {
#pragma unroll
                for (int k = 0; k < V; ++k) acc[k] += x[u][k];
                const int id = __builtin_amdgcn_readfirstlane(s_ids[e + 1]);
                const int after = __builtin_amdgcn_readfirstlane(s_ids[e + 2]);
                const bool ends = after != id;
                if (ends || e == n - 1) {
                    if (crosses || !ends) {
                        // began before, or goes on after: a part (the first
                        // run's if it began before)
                        float* p = a.part + (block * 2 + (crosses ? 0 : 1)) * a.width + c;
#pragma unroll
                        for (int k = 0; k < V; ++k) p[k] = acc[k];
                    } else {
#pragma unroll
                        for (int k = 0; k < V; ++k) acc[k] *= a.scale;
                        store_e<TD, V>(static_cast<TD*>(a.dst) + static_cast<int64_t>(id) * a.width + c, acc);
                    }
#pragma unroll
                    for (int k = 0; k < V; ++k) acc[k] = 0.0f;
                    crosses = false;
                }
            }
        }
    }
}

// The run that begins in window block_place() and goes on after it: the sum of its
// parts, every fourth by each wave, the waves' sums joined in their order.
template <typename TD, int V>
__global__ __launch_bounds__(256) void k_embed_join(const EmbedArgs a) {
    __shared__ float s[3][64][V];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t total = a.offset[a.vocab], w = block_place(), next = (w + 1) * a.window;
    if (next >= total) return;
    const int t = a.ids[next - 1];
    if (a.ids[next] != t) return;
    const int64_t first = a.offset[t], w1 = (static_cast<int64_t>(a.offset[t + 1]) - 1) / a.window;
    if (first < w * a.window) return;
    const int c = (blockIdx.y * 64 + lane) * V;
    const bool in = c < a.width;
    // part rows of the run: 2 w + 1, then 2 (w + 1), 2 (w + 2), ...
    float acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.0f;
    if (in) {
        constexpr int U = 8;
        for (int64_t x0 = w + wave; x0 <= w1; x0 += 4 * U) {
            float x[U][V];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t x1 = x0 + 4 * u <= w1 ? x0 + 4 * u : w1;
                load_e<float, V>(a.part + (2 * x1 + (x1 == w ? 1 : 0)) * a.width + c, x[u]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (x0 + 4 * u <= w1)
#pragma unroll
                    for (int k = 0; k < V; ++k) acc[k] += x[u][k];
        }
    }
    if (wave > 0)
#pragma unroll
        for (int k = 0; k < V; ++k) s[wave - 1][lane][k] = acc[k];
    __syncthreads();
    if (wave > 0 || !in) return;
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = (((acc[k] + s[0][lane][k]) + s[1][lane][k]) + s[2][lane][k]) * a.scale;
    store_e<TD, V>(static_cast<TD*>(a.dst) + static_cast<int64_t>(t) * a.width + c, acc);
}

// Few tokens, in one launch: a workgroup owns `rows` rows of the table.  Its 4
// waves look through a quarter of the tokens each and list the workgroup's own
// in order; one wave sorts them by row, stably; then groups of `lanes` threads
// take a row each.  Bound by the table's zeros (999 tokens, 50257 x 1600
// bfloat16: 161 MB).
constexpr int kDirectTokens = 1024;
constexpr int kDirectRows = 32;
template <typename TS, typename TD, int V>
__global__ __launch_bounds__(256) void k_embed_direct(const EmbedArgs a, int rows, int lanes) {
    __shared__ uint32_t list[4][kDirectTokens / 4];  // token's place * kDirectRows + row
    __shared__ uint16_t sorted[kDirectTokens];
    __shared__ int32_t count[4], first[kDirectRows + 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t r0 = static_cast<int64_t>(block_place()) * rows;
    if (r0 >= a.vocab) return;
    const int mine = a.vocab - r0 < rows ? static_cast<int>(a.vocab - r0) : rows;
    const int n = static_cast<int>(a.n), part = (n + 3) / 4;
    const int i1 = (wave + 1) * part < n ? (wave + 1) * part : n;
    int listed = 0;
    for (int i = wave * part; i < i1; i += 64) {
        const int64_t y = i + lane < i1 ? token_at(a, i + lane) - r0 : -1;
        const bool in = y >= 0 && y < mine;
        const uint64_t all = __ballot(in);
        if (in) list[wave][listed + __popcll(all & ((1ull << lane) - 1))] = (i + lane) * kDirectRows + static_cast<int>(y);
        listed += __popcll(all);
    }
    if (lane == 0) count[wave] = listed;
    __syncthreads();
    if (wave == 0) {
        // lane r < kDirectRows: row r
        int c = 0;
        for (int w = 0; w < 4; ++w)
            for (int e = 0; e < count[w]; ++e) c += static_cast<int>(list[w][e] % kDirectRows) == lane;
        int incl = c;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const int y = __shfl_up(incl, m);
            if (lane >= m) incl += y;
        }
        int at = incl - c;
        if (lane <= kDirectRows) first[lane] = at;
        for (int w = 0; w < 4; ++w)
            for (int e = 0; e < count[w]; ++e) {
                const uint32_t u = list[w][e];
                if (static_cast<int>(u % kDirectRows) == lane) sorted[at++] = static_cast<uint16_t>(u / kDirectRows);
            }
    }
    __syncthreads();
    const int c = (static_cast<int>(blockIdx.y) * lanes + static_cast<int>(threadIdx.x) % lanes) * V;
    if (c >= a.width) return;
    const TS* src = static_cast<const TS*>(a.src) + c;
    for (int r = threadIdx.x / lanes; r < mine; r += 256 / lanes) {
        const int e0 = first[r], e1 = first[r + 1];
        float acc[V];
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = 0.0f;
        constexpr int U = 8;
        for (int e = e0; e < e1; e += U) {
            float x[U][V];
#pragma unroll
            for (int u = 0; u < U; ++u)
                load_e<TS, V>(src + static_cast<int64_t>(sorted[e + u < e1 ? e + u : e]) * a.width, x[u]);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (e + u < e1)
#pragma unroll
                    for (int k = 0; k < V; ++k) acc[k] += x[u][k];
        }
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] *= a.scale;
        store_e<TD, V>(static_cast<TD*>(a.dst) + (r0 + r) * a.width + c, acc);
    }
}

int row_lanes(int pieces) {
    int lanes = 1;
    while (lanes < 64 && lanes < pieces) lanes <<= 1;
    return lanes;
}

template <typename TS, typename TD, int V>
void fwd(const EmbedArgs& a, hipStream_t stream) {
    const int lanes = row_lanes(a.width / V), per = 256 / lanes;
    k_embed<TS, TD, V><<<long_grid((a.n + per - 1) / per, 256), 256, 0, stream>>>(a, lanes);
}

template <typename TS, typename TD, int V>
void bwd(const EmbedArgs& a, hipStream_t stream) {
    // pieces whose stores are contiguous over a wave
    constexpr int W = V == 1 ? 1 : (sizeof(TS) == 2 && sizeof(TD) == 2 ? 8 : 4), J = V == 1 ? 1 : 4;
    const int pieces = a.width / W;
    if (a.n <= kDirectTokens) {
        // a workgroup per CU at least, where the table has the rows
        int64_t rows = a.vocab / 256;
        rows = rows < 1 ? 1 : (rows < kDirectRows ? rows : kDirectRows);
        int lanes = 1;
        while (lanes < 256 && lanes < pieces) lanes <<= 1;
        k_embed_direct<TS, TD, W><<<long_grid((a.vocab + rows - 1) / rows, 256, (pieces + lanes - 1) / lanes), 256, 0, stream>>>(
            a, static_cast<int>(rows), lanes);
        return;
    }
    // 256 workgroups, one per CU, unless the table needs more
    int64_t span = (a.vocab + 255) / 256;
    if (span > kSortSpan) span = kSortSpan;
    const dim3 sorts = long_grid((a.vocab + span - 1) / span, 64 * kSortWaves);
    if (a.tokens64) k_embed_sort<true><<<sorts, 64 * kSortWaves, 0, stream>>>(a, static_cast<int>(span));
    else k_embed_sort<false><<<sorts, 64 * kSortWaves, 0, stream>>>(a, static_cast<int>(span));
    int threads = (pieces + 63) / 64 * 64;
    if (threads > 256) threads = 256;
    const int64_t windows = (a.n + a.window - 1) / a.window, zeros = (a.vocab + kZeroRows - 1) / kZeroRows;
    k_embed_sum<TS, TD, W><<<long_grid(windows + zeros, threads, (pieces + threads - 1) / threads), threads, 0, stream>>>(
        a, static_cast<int>(windows));
    if (windows > 1)
        k_embed_join<TD, J><<<long_grid(windows - 1, 256, (a.width / J + 63) / 64), 256, 0, stream>>>(a);
}

// fn<source, target, values a piece>
#define MUON_EMBED_DISPATCH(fn, a, stream)                                                              \
    do {                                                                                                \
        switch (((a).src_type == MUON_BF16 ? 1 : 0) | ((a).dst_type == MUON_BF16 ? 2 : 0) | ((a).vector ? 4 : 0)) { \
            case 0: fn<float, float, 1>(a, stream); break;                                              \
            case 1: fn<bf16_t, float, 1>(a, stream); break;                                             \
            case 2: fn<float, bf16_t, 1>(a, stream); break;                                             \
            case 3: fn<bf16_t, bf16_t, 1>(a, stream); break;                                            \
            case 4: fn<float, float, 8>(a, stream); break;                                              \
            case 5: fn<bf16_t, float, 8>(a, stream); break;                                             \
            case 6: fn<float, bf16_t, 8>(a, stream); break;                                             \
            case 7: fn<bf16_t, bf16_t, 8>(a, stream); break;                                            \
        }                                                                                               \
    } while (0)

}  // namespace

hipError_t launch_embed(const EmbedArgs& a, hipStream_t stream) {
    MUON_EMBED_DISPATCH(fwd, a, stream);
    return hipGetLastError();
}

hipError_t launch_embed_bwd(const EmbedArgs& a, hipStream_t stream) {
    MUON_EMBED_DISPATCH(bwd, a, stream);
    return hipGetLastError();
}

}  // namespace muon
