// Shared definitions of the language-model operators (muon_lm.h): grids and
// launch arguments.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.hpp"

namespace muon {

// A launch of `blocks` workgroups (below 2^31): HIP takes fewer than 2^32 threads
// along x, so longer grids go on along z.  A kernel finds its place with
// block_place(), which may be past the last one.
inline dim3 long_grid(int64_t blocks, int threads, int64_t y = 1) {
    const int64_t most = ((int64_t{1} << 32) - 1) / threads, z = (blocks + most - 1) / most;
    return dim3(static_cast<uint32_t>((blocks + z - 1) / z), static_cast<uint32_t>(y), static_cast<uint32_t>(z));
}
__device__ __forceinline__ uint32_t block_place() { return blockIdx.z * gridDim.x + blockIdx.x; }

// Keys per LDS tile of every attention kernel, and tokens per entry of the
// document-range table.
constexpr int kTile = 64;

// Arguments of every attention kernel, passed by value.  Strides are in
// elements; the last dimension is contiguous.  lse, dq, dk and dv are contiguous.
struct AttnArgs {
    const bf16_t *q, *k, *v, *dout;
    bf16_t *out, *dq, *dk, *dv;
    float *lse;
    float* stats;       // backward: lse terms, then -delta, delta_at floats on
    int64_t delta_at;
    int64_t q_b, q_s, q_h, k_b, k_s, k_h, v_b, v_s, v_h, do_b, do_s, do_h, o_b, o_s, o_h;
    int64_t doc_b;
    const float* slopes;
    const int32_t *documents, *prefix, *lengths, *starts;
    int2* doc_tiles;  // (lowest, highest) document of each kTile tokens: [b][n_tiles]
    float* part;      // partial results of a split over keys
    int b, sq, sk, hq, hkv, grp, d;
    int causal, window;  // window 0: none
    int n_tiles;         // ceil(sk / kTile)
    int splits, chunk;   // key split: chunks of `chunk` tiles
    float scale, softcap;
};

// The partial results of n (row, chunk) pairs: 2 n floats of maxima and sums,
// then d floats of output each from here on, aligned to their 16-byte stores.
__host__ __device__ inline int64_t part_outputs(int64_t n) { return (2 * n + 3) / 4 * 4; }

hipError_t launch_attn_doc_tiles(const AttnArgs& a, hipStream_t stream);
hipError_t launch_attn_fwd(const AttnArgs& a, hipStream_t stream);
hipError_t launch_attn_split(const AttnArgs& a, hipStream_t stream);
hipError_t launch_attn_bwd_dq(const AttnArgs& a, hipStream_t stream);
hipError_t launch_attn_bwd_dkv(const AttnArgs& a, hipStream_t stream);

// Norm and rotation of query and key heads (qk_norm.hip).  x[0] are the
// queries, x[1] the keys; y and dx are contiguous.  type: muon_dtype.
struct QkArgs {
    const void* x[2];
    const void* dz[2];
    void* y[2];              // forward: outputs; backward: gradients of x
    const float* w[2];       // null: ones
    float* dw[2];            // null: not wanted
    int64_t x_b[2], x_s[2], x_h[2];
    int64_t z_b[2], z_s[2], z_h[2];
    int heads[2];
    const float* table;      // (limit, d / 2, 2): cos, sin
    const int32_t* positions;  // (b, s), or null: 0 .. s - 1
    float* part;             // weight gradients of every workgroup
    int b, s, d, limit, type;
    int lanes;         // lanes that hold one head: a power of two
    int chunk, runs_q;  // heads per workgroup; runs of so many query heads (the keys' follow)
    int blocks, vector;
    float eps;
};
hipError_t launch_qk_norm(const QkArgs& a, hipStream_t stream);
hipError_t launch_qk_norm_bwd(const QkArgs& a, hipStream_t stream);

// Scaled rows of a table and the table's gradient (embed.hip).
struct EmbedArgs {
    const void* tokens;  // int64 or int32
    int tokens64;
    int64_t n, vocab;
    int width;
    const void* src;     // table (forward) or gradient of the rows (backward)
    void* dst;           // rows (forward) or gradient of the table (backward)
    int src_type, dst_type;  // muon_dtype
    int vector;          // rows of whole aligned 16-byte pieces
    float scale;
    int32_t *perm, *ids, *offset;  // backward: sorted order, its tokens, first place of each token
    // backward: sorted entries per window, and the sums of its first and last
    // run where they cross its border (rows 2 w, 2 w + 1)
    int window;
    float* part;
};
hipError_t launch_embed(const EmbedArgs& a, hipStream_t stream);
hipError_t launch_embed_bwd(const EmbedArgs& a, hipStream_t stream);

}  // namespace muon
