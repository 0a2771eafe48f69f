// Shared definitions of the operators of a decoder layer (muon_lm.h): the
// feed-forward block, the norms around a block, dropout.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"

namespace muon {

// Dropout's random bits: block b of the stream of `seed` is Philox4x32-10
// (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3",
// 2011) of the counter (b, 0) under the key `seed`: 8 elements of 16 bits.  An
// element is dropped where its bits are below `threshold` = round(65536 p).
struct DropState {
    uint64_t seed, offset;
    const int64_t* state;  // null, or (seed, block) on the device: the seed, and what is added to offset
    uint32_t threshold;    // 0 .. 65536
    float factor;          // of the elements kept: 65536 / (65536 - threshold), or 0
};

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ u32x4_t philox(uint64_t seed, uint64_t block) {
    uint32_t c0 = static_cast<uint32_t>(block), c1 = static_cast<uint32_t>(block >> 32), c2 = 0, c3 = 0;
    uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u, b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
        c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
        c1 = static_cast<uint32_t>(b);
        c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
        c3 = static_cast<uint32_t>(a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return u32x4_t{c0, c1, c2, c3};
}

// The seed and the first block.
__device__ __forceinline__ void drop_start(const DropState& d, uint64_t& seed, uint64_t& first) {
    seed = d.state ? static_cast<uint64_t>(d.state[0]) : d.seed;
    first = d.state ? static_cast<uint64_t>(d.state[1]) + d.offset : d.offset;
}

// Whether element j of a block is kept.
__device__ __forceinline__ bool drop_keeps(const u32x4_t& w, int j, uint32_t threshold) {
    return ((w[j >> 1] >> (16 * (j & 1))) & 0xffffu) >= threshold;
}

struct DropArgs {
    const void* x;
    void* out;
    int64_t n;
    int type;    // muon_dtype
    int vector;  // 16-byte aligned
    DropState drop;
};
hipError_t launch_dropout(const DropArgs& a, hipStream_t stream);

enum { GATE_NONE = 0, GATE_CHANNEL = 1, GATE_SEQUENCE = 2, GATE_FULL = 3 };

// The norms around a block (resid_norm.hip).  Rows are tokens; strides in
// elements; outputs are contiguous.
struct ResidArgs {
    const void *x, *y, *xo, *gate, *dz, *dxo;
    void *x_out, *z, *dx, *dy, *dgate;
    const float *scale, *postw, *prew;
    float *dscale, *dpostw, *dprew;
    int64_t x_s, y_s, xo_s, g_s, dz_s, dxo_s;
    int64_t rows, s;        // s: rows of a sequence
    int width;
    int x_type, y_type;     // muon_dtype of the stream and of the block
    int gate_kind, post;
    int vector;             // rows of aligned pieces of 8
    int threads, pieces;    // threads that hold a row, pieces a thread
    int64_t blocks;
    // backward: groups of rows share a gate (GATE_SEQUENCE: a sequence each); a
    // group is split into `chunks` workgroups, or a workgroup takes `per` groups
    int64_t groups;
    int chunks, per;
    float* part;            // [blocks][4][width]: sums for prew, postw, scale, gate (GATE_CHANNEL)
    float* gate_part;       // [groups][chunks][width], or null where chunks = 1
    float eps;
    DropState drop;         // threshold 0: none
};
hipError_t launch_resid_norm(const ResidArgs& a, hipStream_t stream);
hipError_t launch_resid_norm_bwd(const ResidArgs& a, hipStream_t stream);

// The feed-forward block's products (ffn.hip).  C[m][n] = sum_k P(m, k) Q(n, k)
// of bfloat16 operands, each "rows" (contiguous along k: P[m][k]) or "columns"
// (contiguous along its output index: P[k][m]).
enum FfnKind {
    FFN_GATED = 0,  // rows, rows: gate and up projections, h = act(gate) up
    FFN_PLAIN = 1,  // rows, rows: the down projection
    FFN_HIDDEN = 2, // rows, columns: gradient of h, and from it those of gate and up
    FFN_INPUT = 3,  // rows, columns: gradient of x, a sum of two products
    FFN_WEIGHTS = 4 // columns, columns: gradients of the matrices
};
enum FfnAct { ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2, ACT_RELU = 3 };

struct FfnSeg {
    const bf16_t *p[2], *q[2];  // FFN_GATED: q are the gate and up matrices; FFN_INPUT: two products
    int64_t ldp, ldq;
    int m, n;
    int tiles_m, tiles_n, first;  // first: its first tile of the launch
    int band;                     // tile rows that go column by column together
    void* out;                    // m x n, contiguous
};
struct FfnGemm {
    FfnSeg seg[3];
    int nseg, tiles;         // tiles of all segments
    int64_t k;               // contracted length of one product
    int phases;              // products summed
    int full;                // the first `full` tiles are computed whole, K of the others is split
    int splits, split_steps; // into so many parts of so many steps
    float* part;             // [splits][tiles - full][tile][tile], or null where full = tiles
    int out_f32;
    int act;
    bf16_t *gate, *up, *dgate, *dup;  // FFN_GATED writes gate and up where given; FFN_HIDDEN reads them
};
enum FfnTile { FFN_256 = 256, FFN_128 = 128 };  // output rows and columns of a workgroup
constexpr int kFfnStep = 64;                    // K values of a step
hipError_t launch_ffn(FfnKind kind, FfnTile tile, const FfnGemm& g, hipStream_t stream);

// A few tokens, without what a backward pass needs (ffn_few.hip).
constexpr int kFewTokens = 32;
struct FfnFew {
    const bf16_t *x, *w_gate, *w_up, *w_down;
    bf16_t *h, *out;  // h: as fragments of 16 tokens by 32 values; out: contiguous
    int64_t x_stride, w_stride, w_down_stride;
    int tokens, width, hidden, act;
};
hipError_t launch_ffn_few(const FfnFew& a, hipStream_t stream);

}  // namespace muon
