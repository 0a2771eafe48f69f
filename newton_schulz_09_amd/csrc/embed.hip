// Embedding: out[i] = scale * table[token[i]], and the table's gradient
// dtable[v] = scale * sum of dout[i] over the i with token[i] = v, summed in
// the order of i in float32, without atomics on floating values.
//
// Both are bound by memory.  The gradient sorts the tokens first (k_embed_sort,
// stable), then sums windows of kEmbedWindow sorted entries (k_embed_sum), so
// that a token's work is spread over many workgroups however often it occurs,
// and last joins the runs that cross windows and writes the rows of tokens
// that do not occur (k_embed_rest).
#include "../../include/muon.h"
#include "lm_common.hpp"

namespace muon {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <typename T, int V>
__device__ __forceinline__ void load_e(const T* p, float (&x)[V]) {
    if constexpr (V == 1) {
        if constexpr (sizeof(T) == 2) x[0] = bf16_to_f32(p[0]);
        else x[0] = p[0];
    } else if constexpr (sizeof(T) == 2) {
        const u32x4 u = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
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
    } else if constexpr (sizeof(T) == 2) {
        const u32x4 u = {f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]), f32x2_to_bf16x2(x[4], x[5]),
                         f32x2_to_bf16x2(x[6], x[7])};
        __builtin_nontemporal_store(u, reinterpret_cast<u32x4*>(p));
    } else {
        __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]}, reinterpret_cast<f32x4*>(p));
        __builtin_nontemporal_store(f32x4{x[4], x[5], x[6], x[7]}, reinterpret_cast<f32x4*>(p) + 1);
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
    const int64_t i = static_cast<int64_t>(blockIdx.x) * per + threadIdx.x / lanes;
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
// span.  Its 16 waves take 16 consecutive parts of the tokens; a first pass
// counts (per wave and row, and the tokens of lower rows, which is where the
// workgroup's entries begin), a second one places.  No workgroup waits for
// another one.  Every workgroup reads all the tokens from the caches: 65536
// of them are 512 KiB.
constexpr int kSortWaves = 16;
constexpr int kSortSpan = 512;  // table rows per workgroup at most
__global__ __launch_bounds__(64 * kSortWaves) void k_embed_sort(const EmbedArgs a, int span) {
    __shared__ int32_t cnt[kSortWaves][kSortSpan];
    __shared__ int32_t below[kSortWaves];
    __shared__ int32_t wsum[kSortWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t lo = static_cast<int64_t>(blockIdx.x) * span;
    const int rows = static_cast<int>(lo + span <= a.vocab ? span : a.vocab - lo);
    for (int i = threadIdx.x; i < kSortWaves * kSortSpan; i += blockDim.x) (&cnt[0][0])[i] = 0;
    __syncthreads();
    const int64_t part = ((a.n + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
    const int64_t i0 = wave * part, i1 = i0 + part < a.n ? i0 + part : a.n;
    constexpr int U = 8;
    int32_t low = 0;
    for (int64_t i = i0; i < i1; i += 64 * U) {
        int64_t t[U];
#pragma unroll
        for (int k = 0; k < U; ++k) t[k] = i + 64 * k + lane < i1 ? token_at(a, i + 64 * k + lane) : -1;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            low += t[k] >= 0 && t[k] < lo;
            const int64_t x = t[k] - lo;
            if (t[k] >= 0 && x >= 0 && x < rows) atomicAdd(&cnt[wave][x], 1);
        }
    }
#pragma unroll
    for (int m = 32; m; m >>= 1) low += __shfl_xor(low, m);
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
        if (x < rows) a.offset[lo + x] = first;
        if (x == rows - 1 && lo + rows == a.vocab) a.offset[a.vocab] = first + total;
    }
    __syncthreads();
    for (int64_t i = i0; i < i1; i += 64 * U) {
        int64_t t[U];
#pragma unroll
        for (int k = 0; k < U; ++k) t[k] = i + 64 * k + lane < i1 ? token_at(a, i + 64 * k + lane) : -1;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int64_t y = t[k] - lo;
            const bool mine = t[k] >= 0 && y >= 0 && y < rows;
            uint64_t left = __ballot(mine);
            while (left) {
                // the lanes that hold the first one's token take places in order
                const int lead = __builtin_ctzll(left);
                const int32_t who = __shfl(static_cast<int32_t>(y), lead);
                const bool same = mine && static_cast<int32_t>(y) == who;
                const uint64_t all = __ballot(same);
                const int32_t at = cnt[wave][who];
                if (same) {
                    const int32_t p = at + __popcll(all & ((1ull << lane) - 1));
                    a.perm[p] = static_cast<int32_t>(i + 64 * k + lane);
                    a.ids[p] = static_cast<int32_t>(t[k]);
                }
                if (lane == lead) cnt[wave][who] = at + __popcll(all);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
                left &= ~all;
            }
        }
    }
}

// Sums of the runs of equal tokens of one window.  A run inside the window is
// written as the table's row; the first run goes to part row 2 w and the last
// to 2 w + 1 where they cross the window's border.
template <typename TS, typename TD, int V>
__global__ __launch_bounds__(256) void k_embed_sum(const EmbedArgs a) {
    __shared__ int32_t s_perm[kEmbedWindow], s_ids[kEmbedWindow + 2];
    const int64_t total = a.offset[a.vocab], w0 = static_cast<int64_t>(blockIdx.x) * kEmbedWindow;
    if (w0 >= total) return;
    const int n = total - w0 < kEmbedWindow ? static_cast<int>(total - w0) : kEmbedWindow;
    if (threadIdx.x < kEmbedWindow + 2) {
        // with the neighbours on either side (-1: none)
        const int64_t i = w0 + threadIdx.x - 1;
        const bool in = i >= 0 && i < total;
        s_ids[threadIdx.x] = in ? a.ids[i] : -1;
        if (threadIdx.x >= 1 && static_cast<int>(threadIdx.x) <= n) s_perm[threadIdx.x - 1] = a.perm[i];
    }
    if (blockDim.x < kEmbedWindow + 2 && threadIdx.x < 2) {  // a workgroup of one wave: the last two
        const int64_t i = w0 + kEmbedWindow + threadIdx.x - 1;
        s_ids[kEmbedWindow + threadIdx.x] = i < total ? a.ids[i] : -1;
        if (kEmbedWindow - 1 + static_cast<int>(threadIdx.x) < n && threadIdx.x == 0) s_perm[kEmbedWindow - 1] = a.perm[i];
    }
    __syncthreads();
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    if (c >= a.width) return;
    const TS* src = static_cast<const TS*>(a.src) + c;
    float acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.0f;
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
                        float* p = a.part + (static_cast<int64_t>(blockIdx.x) * 2 + (crosses ? 0 : 1)) * a.width + c;
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

// Rows of tokens that do not occur (zeros) and of those whose run crosses
// windows (the sum of its parts in their order).
template <typename TD, int V>
__global__ __launch_bounds__(256) void k_embed_rest(const EmbedArgs a, int lanes) {
    const int l = threadIdx.x % lanes, per = 256 / lanes;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * per + threadIdx.x / lanes;
    if (t >= a.vocab) return;
    const int64_t first = a.offset[t], end = a.offset[t + 1];
    const int64_t w0 = first / kEmbedWindow, w1 = (end - 1) / kEmbedWindow;
    if (end > first && w0 == w1) return;
    TD* dst = static_cast<TD*>(a.dst) + t * a.width;
    const int pieces = a.width / V;
    for (int c = l; c < pieces; c += lanes) {
        float acc[V];
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = 0.0f;
        if (end > first) {
            for (int64_t w = w0; w <= w1; ++w) {
                const float* p = a.part + (2 * w + (w == w0 ? 1 : 0)) * a.width + c * V;
#pragma unroll
                for (int k = 0; k < V; ++k) acc[k] += p[k];
            }
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] *= a.scale;
        }
        store_e<TD, V>(dst + c * V, acc);
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
    k_embed<TS, TD, V><<<static_cast<uint32_t>((a.n + per - 1) / per), 256, 0, stream>>>(a, lanes);
}

template <typename TS, typename TD, int V>
void bwd(const EmbedArgs& a, hipStream_t stream) {
    // 256 workgroups, one per CU, unless the table needs more
    int64_t span = (a.vocab + 255) / 256;
    if (span > kSortSpan) span = kSortSpan;
    k_embed_sort<<<static_cast<uint32_t>((a.vocab + span - 1) / span), 64 * kSortWaves, 0, stream>>>(a, static_cast<int>(span));
    if (a.n > 0) {
        const int pieces = a.width / V;
        int threads = (pieces + 63) / 64 * 64;
        if (threads > 256) threads = 256;
        k_embed_sum<TS, TD, V><<<dim3(static_cast<uint32_t>((a.n + kEmbedWindow - 1) / kEmbedWindow),
                                      static_cast<uint32_t>((pieces + threads - 1) / threads)),
                                 threads, 0, stream>>>(a);
    }
    const int lanes = row_lanes(a.width / V), per = 256 / lanes;
    k_embed_rest<TD, V><<<static_cast<uint32_t>((a.vocab + per - 1) / per), 256, 0, stream>>>(a, lanes);
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
