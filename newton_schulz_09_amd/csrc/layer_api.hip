// C ABI of the operators of a decoder layer: validation, plans and workspace
// layout (declared and documented in include/muon_lm.h).
#include <math.h>

#include "../../include/muon_lm.h"
#include "layer_common.hpp"
#include "lm_host.hpp"

namespace muon {

namespace {

int64_t type_bytes(int64_t dtype) { return dtype == MUON_BF16 ? 2 : 4; }
bool known_type(int64_t dtype) { return dtype == MUON_F32 || dtype == MUON_BF16; }

// --------------------------------------------------------------- dropout

int make_drop(double p, uint64_t seed, uint64_t offset, const int64_t* state, DropState& d) {
    if (!(p >= 0.0 && p <= 1.0)) return refuse(MUON_ERR_INVALID_ARG, "p must be within 0 .. 1");
    if (!aligned(state, 8)) return refuse(MUON_ERR_INVALID_ARG, "state is not aligned to 8 bytes");
    d.seed = seed;
    d.offset = offset;
    d.state = state;
    d.threshold = static_cast<uint32_t>(floor(p * 65536.0 + 0.5));
    d.factor = d.threshold < 65536 ? static_cast<float>(65536.0 / (65536 - static_cast<int>(d.threshold))) : 0.0f;
    return MUON_OK;
}

// ---------------------------------------------------- norms around a block

int check_resid(const muon_residual_norm_args* x) {
    if (!x) return refuse(MUON_ERR_INVALID_ARG, "null arguments");
    if (x->batch < 0 || x->s < 0) return refuse(MUON_ERR_INVALID_ARG, "negative size");
    if (x->width <= 0 || x->width > MUON_RESIDUAL_NORM_MAX_WIDTH)
        return refuse(MUON_ERR_UNSUPPORTED, "width %lld is not within 1 .. %d", (long long)x->width,
                      MUON_RESIDUAL_NORM_MAX_WIDTH);
    if (x->batch >= kMaxSeq || x->s >= kMaxSeq) return refuse(MUON_ERR_UNSUPPORTED, "a size of 2^29 or more");
    const int64_t n = times(times(x->batch, x->s), x->width);
    if (n < 0) return refuse(MUON_ERR_UNSUPPORTED, "too many rows");
    if (!known_type(x->stream_type) || !known_type(x->block_type)) return refuse(MUON_ERR_INVALID_ARG, "unknown dtype");
    if (x->stream_type == MUON_BF16 && x->block_type == MUON_F32)
        return refuse(MUON_ERR_UNSUPPORTED, "a float32 block on a bfloat16 stream");
    if (x->gate_kind < GATE_NONE || x->gate_kind > GATE_FULL) return refuse(MUON_ERR_INVALID_ARG, "unknown gate_kind");
    if (x->gate_kind == GATE_SEQUENCE && x->batch > (int64_t{1} << 20))
        return refuse(MUON_ERR_UNSUPPORTED, "more than 2^20 sequences with a gate each");
    if (!(x->eps >= 0.0) || !isfinite(static_cast<float>(x->eps)))
        return refuse(MUON_ERR_INVALID_ARG, "eps must be >= 0 and finite");
    return MUON_OK;
}

struct ResidPlan {
    int threads, pieces, chunks, per;
    int64_t blocks, groups;
    size_t off_gate, bytes;
};

// Threads that hold a row: a part of a wave that fits it up to 256 values, a wave
// up to 1024, then as many as keep it at two pieces of 8 a thread.  (49728 rows of
// 256 bf16, a wave and half a wave: 25 and 19 us, gradients 50 and 35; 65536 rows of
// 100, a wave and 16 lanes: 57 and 20, gradients 152 and 49.)
//
// Backward, a workgroup leaves a row of up to 4 sums, which are written and read
// again (as much as two rows of data): at most as many workgroups as the chip
// holds, and 4 turns of rows each.
ResidPlan plan_resid(const muon_residual_norm_args* x, bool backward) {
    ResidPlan p{};
    const int64_t pieces = div_up(x->width, 8);
    const int64_t least = pieces <= 64 ? pieces : div_up(pieces, 2);
    p.threads = 8;
    while (p.threads < least) p.threads *= 2;
    p.pieces = pieces <= 64 ? 1 : 2;
    const int64_t rows = x->batch * x->s, per_block = p.threads >= 256 ? 1 : 256 / p.threads;
    p.chunks = p.per = 1;
    p.groups = 1;
    if (!backward) {
        const int64_t n = div_up(rows, per_block), most = p.threads == 512 ? 1024 : 2048;
        p.blocks = n < most ? n : most;
        p.bytes = 256;
        return p;
    }
    const int64_t most = p.threads == 512 ? 256 : 512;
    const bool by_sequence = x->gate_kind == GATE_SEQUENCE;
    p.groups = by_sequence ? x->batch : 1;
    const int64_t n = div_up(by_sequence ? x->s : rows, 4 * per_block);
    if (p.groups >= most) {
        p.per = static_cast<int>(div_up(p.groups, most));
        p.blocks = div_up(p.groups, p.per);
    } else if (p.groups > 0) {
        const int64_t c = most / p.groups;
        p.chunks = static_cast<int>(n < 1 ? 1 : n < c ? n : c);
        p.blocks = p.groups * p.chunks;
    }
    p.off_gate = align256(static_cast<size_t>(p.blocks) * 4 * x->width * sizeof(float));
    p.bytes = p.off_gate;
    if (by_sequence && p.chunks > 1) p.bytes += align256(static_cast<size_t>(p.blocks) * x->width * sizeof(float));
    if (p.bytes < 256) p.bytes = 256;
    return p;
}

int run_resid(const muon_residual_norm_args* x, bool backward, void* ws, size_t ws_bytes, hipStream_t stream) {
    if (int st = check_resid(x)) return st;
    ResidArgs a{};
    if (int st = make_drop(x->p, x->seed, x->offset, x->state, a.drop)) return st;
    const int64_t rows = x->batch * x->s, xb = type_bytes(x->stream_type), yb = type_bytes(x->block_type);
    const bool block = x->has_block != 0;
    if (!block && (x->gate_kind != GATE_NONE || x->post || a.drop.threshold))
        return refuse(MUON_ERR_INVALID_ARG, "a gate, post norm or dropout without a block's output");
    if (!x->post && (x->post_weight || x->dpost_weight))
        return refuse(MUON_ERR_INVALID_ARG, "a weight of the post norm without that norm");
    bool vec = x->width % 8 == 0;
    const char* bad = nullptr;
    // a tensor of rows that the call reads or writes
    auto row = [&](const char* name, const void* p, int64_t bytes, int64_t stride) {
        if (rows == 0 || bad) return;
        if (!p || !aligned(p, bytes) || (rows > 1 && stride < 0)) bad = name;
        vec = vec && aligned(p, 16) && (rows <= 1 || stride % 8 == 0);
    };
    const bool full = x->gate_kind == GATE_FULL;
    if (!backward) {
        row("x", x->x, xb, x->x_stride);
        if (block) row("y", x->y, yb, x->y_stride);
        if (x->x_out) row("x_out", x->x_out, xb, 0);
        row("z", x->z, yb, 0);
    } else {
        row("x_out", x->x_out, xb, x->x_out_stride);
        row("dz", x->dz, yb, x->dz_stride);
        if (x->dx_out) row("dx_out", x->dx_out, xb, x->dx_out_stride);
        if (x->dresidual_scale) row("x", x->x, xb, x->x_stride);
        if (block) row("y", x->y, yb, x->y_stride);
        row("dx", x->dx, xb, 0);
        if (block) row("dy", x->dy, yb, 0);
        if (full) row("dgate", x->dgate, yb, 0);
    }
    if (full) row("gate", x->gate, yb, x->gate_stride);
    if (bad) return refuse(MUON_ERR_INVALID_ARG, "%s is null or not aligned to its type, or its stride is negative", bad);
    const bool vector_gate = x->gate_kind == GATE_CHANNEL || (x->gate_kind == GATE_SEQUENCE && x->batch > 0);
    if (vector_gate && !x->gate) return refuse(MUON_ERR_INVALID_ARG, "gate is null");
    if (backward && vector_gate && !x->dgate) return refuse(MUON_ERR_INVALID_ARG, "dgate is null");
    if (backward && x->dresidual_scale && !x->residual_scale)
        return refuse(MUON_ERR_INVALID_ARG, "dresidual_scale without residual_scale");
    for (const void* p : {static_cast<const void*>(x->residual_scale), static_cast<const void*>(x->post_weight),
                          static_cast<const void*>(x->pre_weight), static_cast<const void*>(full ? nullptr : x->gate),
                          static_cast<const void*>(backward ? x->dresidual_scale : nullptr),
                          static_cast<const void*>(backward ? x->dpost_weight : nullptr),
                          static_cast<const void*>(backward ? x->dpre_weight : nullptr),
                          static_cast<const void*>(backward && !full ? x->dgate : nullptr)})
        if (!aligned(p, 4)) return refuse(MUON_ERR_INVALID_ARG, "a vector is not aligned to 4 bytes");
    if (backward)
        if (int st = check_workspace(ws, ws_bytes, muon_residual_norm_backward_workspace_size(x))) return st;
    if (!backward && rows == 0) return done();
    const ResidPlan p = plan_resid(x, backward);
    auto step = [&](int64_t stride) { return rows > 1 ? stride : 0; };
    a.x = x->x;
    a.y = block ? x->y : nullptr;
    a.gate = x->gate;
    a.x_s = step(x->x_stride);
    a.y_s = step(x->y_stride);
    a.g_s = step(x->gate_stride);
    if (backward) {
        a.xo = x->x_out;
        a.dz = x->dz;
        a.dxo = x->dx_out;
        a.xo_s = step(x->x_out_stride);
        a.dz_s = step(x->dz_stride);
        a.dxo_s = step(x->dx_out_stride);
        a.dx = x->dx;
        a.dy = x->dy;
        a.dgate = x->gate_kind == GATE_NONE ? nullptr : x->dgate;
        a.dscale = x->dresidual_scale;
        a.dpostw = x->dpost_weight;
        a.dprew = x->dpre_weight;
        a.part = static_cast<float*>(ws);
        if (x->gate_kind == GATE_SEQUENCE && p.chunks > 1)
            a.gate_part = reinterpret_cast<float*>(static_cast<char*>(ws) + p.off_gate);
    } else {
        a.x_out = x->x_out;
        a.z = x->z;
    }
    a.scale = x->residual_scale;
    a.postw = x->post_weight;
    a.prew = x->pre_weight;
    a.rows = rows;
    a.s = x->s;
    a.width = static_cast<int>(x->width);
    a.x_type = static_cast<int>(x->stream_type);
    a.y_type = static_cast<int>(x->block_type);
    a.gate_kind = static_cast<int>(x->gate_kind);
    a.post = x->post != 0;
    a.vector = vec;
    a.threads = p.threads;
    a.pieces = p.pieces;
    a.blocks = p.blocks;
    a.groups = p.groups;
    a.chunks = p.chunks;
    a.per = p.per;
    a.eps = static_cast<float>(x->eps);
    const int st = launched(backward ? launch_resid_norm_bwd(a, stream) : launch_resid_norm(a, stream), "norms of a block");
    return st ? st : done();
}

// ----------------------------------------------------------- feed-forward

constexpr int64_t kMaxFfnStride = int64_t{1} << 21;  // elements: a tile's offsets stay below 2^31 bytes
constexpr int64_t kMaxFfnTiles = (int64_t{1} << 23) - 1;  // workgroups of 512 threads below 2^32 threads

int check_ffn(const muon_feed_forward_args* x) {
    if (!x) return refuse(MUON_ERR_INVALID_ARG, "null arguments");
    if (x->tokens < 0) return refuse(MUON_ERR_INVALID_ARG, "negative size");
    if (x->width <= 0 || x->hidden <= 0 || x->width % 8 != 0 || x->hidden % 8 != 0)
        return refuse(MUON_ERR_UNSUPPORTED, "width (%lld) and hidden (%lld) must be positive multiples of 8",
                      (long long)x->width, (long long)x->hidden);
    if (x->width >= kMaxFfnStride || x->hidden >= kMaxFfnStride)
        return refuse(MUON_ERR_UNSUPPORTED, "a width of 2^21 or more");
    if (x->tokens >= kMaxSeq) return refuse(MUON_ERR_UNSUPPORTED, "2^29 tokens or more");
    if (x->activation < ACT_SILU || x->activation > ACT_RELU) return refuse(MUON_ERR_INVALID_ARG, "unknown activation");
    const int64_t most = x->width > x->hidden ? x->width : x->hidden;
    if (div_up(x->tokens, 128) * div_up(most, 64) > kMaxFfnTiles || div_up(most, 128) * div_up(most, 128) * 3 > kMaxFfnTiles)
        return refuse(MUON_ERR_UNSUPPORTED, "too many tokens or columns");
    return MUON_OK;
}

// Rows of a matrix that the matrix cores' loads read 16 bytes at a time.
int check_matrix(const char* name, const void* p, int64_t rows, int64_t cols, int64_t stride) {
    if (rows == 0) return MUON_OK;
    if (!p) return refuse(MUON_ERR_INVALID_ARG, "%s is null", name);
    if (!aligned(p, 16)) return refuse(MUON_ERR_INVALID_ARG, "%s is not aligned to 16 bytes", name);
    // (rows that share memory would put values where the loads expect the end)
    if (rows > 1 && (stride < cols || stride % 8 != 0))
        return refuse(MUON_ERR_INVALID_ARG, "%s: stride %lld is not a multiple of 8 elements from %lld on", name,
                      (long long)stride, (long long)cols);
    if (rows > 1 && stride >= kMaxFfnStride) return refuse(MUON_ERR_UNSUPPORTED, "%s: row stride of 2^21 elements or more", name);
    return MUON_OK;
}

struct FfnPlan {
    FfnTile tile;
    int64_t full;  // tiles computed whole; K of the others is split
    int splits;
    size_t part;   // bytes of the splits' sums
};

// The tile, the number of tiles that are computed whole and the number of splits
// of the others' K that take the least time: rounds of workgroups over the CUs
// times the steps of one.  Either whole rounds of tiles are computed whole and
// the rest is split, so that the last round is no shorter than the others are
// wide, or all tiles are split, or none.  k: length of one product; phases:
// products summed; columns: of a tile, of the sums' and the output's.
//
// The figures are fitted to the times of 572 plans of the five products at 11
// sizes (64 to 8192 tokens, 768 to 4096 wide; off by 10% on average, and the plan
// they choose is 1% slower than the fastest of those measured), in microseconds:
// a step of a 256 tile, one of which a CU holds, 1.37; of 128 tiles 1.08 where a
// CU holds two and 0.86 where it holds one; around the steps of a tile, where
// results are written, `over`; the sums of splits 7, and 2.7 TB/s.
FfnPlan plan_ffn(FfnKind kind, int64_t m, int64_t n, int64_t k, int phases, int count) {
    FfnPlan best{};
    double least = 1e300;
    const int64_t steps = div_up(k, kFfnStep) * phases;
    if (kind == FFN_WEIGHTS && steps <= 1) {  // the kernel of one step; nothing to split
        best.tile = FFN_128;
        best.full = div_up(m, FFN_128) * div_up(n, FFN_128) * count;
        best.splits = 1;
        return best;
    }
    // gated, plain, hidden, input, weights
    static const double over256[5] = {12.5, 2.5, 30.0, 5.5, 8.0}, over128[5] = {5.0, 0.0, 9.0, 0.5, 3.5};
    for (const FfnTile tile : {FFN_256, FFN_128}) {
        const bool big = tile == FFN_256;
        const int64_t tiles = div_up(m, tile) * div_up(n, kind == FFN_GATED ? tile / 2 : tile) * count, slots = big ? 256 : 512;
        const double over = big ? over256[kind] : over128[kind];
        // n workgroups of `steps` steps each, and `around` them
        auto rounds = [&](int64_t n, int64_t steps, double around) {
            const int64_t left = n % slots;
            double t = static_cast<double>(n / slots) * (static_cast<double>(steps) * (big ? 1.37 : 1.08) + around);
            if (left) t += static_cast<double>(steps) * (big ? 1.37 : left > 256 ? 1.08 : 0.86) + around;
            return t;
        };
        for (const int64_t full : {tiles, tiles / slots * slots, int64_t{0}}) {
            const int64_t tail = tiles - full;
            for (int s = tail ? 2 : 1; s <= 32; ++s) {
                if (s > 1 && (tail == 0 || s > steps / 2 || full + tail * s > kMaxFfnTiles)) break;
                double t = rounds(full, steps, over);
                if (tail) t += rounds(tail * s, div_up(steps, s), big ? 3.5 : 1.0) + 7.0 + static_cast<double>(tail) * tile * tile * s * 4.0 / 2.7e6;
                if (t < least) {
                    least = t;
                    best.tile = tile;
                    best.full = full;
                    best.splits = s;
                    best.part = align256(static_cast<size_t>(tail) * s * tile * tile * sizeof(float));
                }
            }
        }
    }
    return best;
}

FfnPlan plan_gated(const muon_feed_forward_args* x) { return plan_ffn(FFN_GATED, x->tokens, x->hidden, x->width, 1, 1); }
FfnPlan plan_down(const muon_feed_forward_args* x) { return plan_ffn(FFN_PLAIN, x->tokens, x->width, x->hidden, 1, 1); }
FfnPlan plan_hidden(const muon_feed_forward_args* x) { return plan_ffn(FFN_HIDDEN, x->tokens, x->hidden, x->width, 1, 1); }
FfnPlan plan_input(const muon_feed_forward_args* x) { return plan_ffn(FFN_INPUT, x->tokens, x->width, x->hidden, 2, 1); }
FfnPlan plan_weights(const muon_feed_forward_args* x) { return plan_ffn(FFN_WEIGHTS, x->hidden, x->width, x->tokens, 1, 3); }

size_t larger(size_t a, size_t b) { return a > b ? a : b; }
size_t hidden_bytes(const muon_feed_forward_args* x) { return align256(static_cast<size_t>(x->tokens) * x->hidden * 2); }

// Whether the matrices are streamed past the tokens (ffn_few.hip) or tiles are
// computed: 768 x 2048, 32 tokens 13 us and 23; 1600 x 4264, one token 23 and 28,
// 16 tokens 26 and 29, 32 tokens 32 and 31; 4096 x 10240, one token 63 and 64, 8
// tokens 66 and 64, 32 tokens 91 and 69.
bool few_tokens(const muon_feed_forward_args* x) {
    return !x->kept && x->tokens > 0 && x->tokens <= kFewTokens &&
           static_cast<double>(x->tokens) * static_cast<double>(x->width) * static_cast<double>(x->hidden) < 2e8;
}

size_t forward_bytes(const muon_feed_forward_args* x) {
    // few tokens: h as whole fragments of 16 tokens by 32 values
    if (few_tokens(x)) return larger(static_cast<size_t>(div_up(x->hidden, 32)) * div_up(x->tokens, 16) * 1024, 256);
    return larger((x->kept ? 0 : hidden_bytes(x)) + larger(plan_gated(x).part, plan_down(x).part), 256);
}
size_t backward_bytes(const muon_feed_forward_args* x) {
    const size_t part = larger(plan_hidden(x).part, larger(plan_input(x).part, plan_weights(x).part));
    return larger(2 * hidden_bytes(x) + part, 256);
}

// One product of a launch; first: tiles of those before it.
void add_seg(FfnGemm& g, FfnTile tile, bool gated, const bf16_t* p0, const bf16_t* p1, int64_t ldp, const bf16_t* q0,
             const bf16_t* q1, int64_t ldq, int64_t m, int64_t n, void* out) {
    FfnSeg& s = g.seg[g.nseg++];
    s.p[0] = p0;
    s.p[1] = p1;
    s.q[0] = q0;
    s.q[1] = q1;
    s.ldp = ldp;
    s.ldq = ldq;
    s.m = static_cast<int>(m);
    s.n = static_cast<int>(n);
    s.tiles_m = static_cast<int>(div_up(m, tile));
    s.tiles_n = static_cast<int>(div_up(n, gated ? tile / 2 : tile));
    s.first = g.tiles;
    // tile rows that go column by column together: with few columns the tiles that
    // run at once on an XCD share all of them, else 8 rows (GPT-2 124M batch: down
    // projection, 3 columns, 206 us with 1 and 215 with 8; gradient of the hidden
    // values, 16 columns, 414 with 8, 427 with 4, 460 with 16)
    s.band = s.tiles_n <= 4 ? 1 : 8;
    s.out = out;
    g.tiles += s.tiles_m * s.tiles_n;
}
void set_steps(FfnGemm& g, const FfnPlan& p, int64_t k, int phases, float* part) {
    g.k = k;
    g.phases = phases;
    g.full = p.full < g.tiles ? static_cast<int>(p.full) : g.tiles;
    const int64_t steps = div_up(k, kFfnStep) * phases;
    g.splits = p.splits;
    g.split_steps = static_cast<int>(div_up(steps, p.splits));
    g.part = g.full < g.tiles ? part : nullptr;
}

}  // namespace

}  // namespace muon

extern "C" {

int muon_dropout(const void* x, void* out, int64_t n, int dtype, double p, uint64_t seed, uint64_t offset,
                 const int64_t* state, void* stream) {
    using namespace muon;
    if (n < 0) return refuse(MUON_ERR_INVALID_ARG, "negative size");
    if (!known_type(dtype)) return refuse(MUON_ERR_INVALID_ARG, "unknown dtype");
    if (n > (int64_t{1} << 41)) return refuse(MUON_ERR_UNSUPPORTED, "more than 2^41 elements");
    DropArgs a{};
    if (int st = make_drop(p, seed, offset, state, a.drop)) return st;
    if (n == 0) return done();
    if (!x || !out) return refuse(MUON_ERR_INVALID_ARG, "null pointer argument");
    if (!aligned(x, type_bytes(dtype)) || !aligned(out, type_bytes(dtype)))
        return refuse(MUON_ERR_INVALID_ARG, "a tensor is not aligned to its type");
    a.x = x;
    a.out = out;
    a.n = n;
    a.type = dtype;
    a.vector = aligned(x, 16) && aligned(out, 16);
    const int st = launched(launch_dropout(a, static_cast<hipStream_t>(stream)), "dropout");
    return st ? st : done();
}

size_t muon_residual_norm_backward_workspace_size(const muon_residual_norm_args* x) {
    using namespace muon;
    if (check_resid(x)) return 0;
    return plan_resid(x, true).bytes;
}

int muon_residual_norm(const muon_residual_norm_args* x, void* stream) {
    return muon::run_resid(x, false, nullptr, 0, static_cast<hipStream_t>(stream));
}

int muon_residual_norm_backward(const muon_residual_norm_args* x, void* ws, size_t ws_bytes, void* stream) {
    return muon::run_resid(x, true, ws, ws_bytes, static_cast<hipStream_t>(stream));
}

size_t muon_feed_forward_workspace_size(const muon_feed_forward_args* x) {
    using namespace muon;
    return check_ffn(x) ? 0 : forward_bytes(x);
}

size_t muon_feed_forward_backward_workspace_size(const muon_feed_forward_args* x) {
    using namespace muon;
    return check_ffn(x) ? 0 : backward_bytes(x);
}

int muon_feed_forward(const muon_feed_forward_args* x, void* ws, size_t ws_bytes, void* stream) {
    using namespace muon;
    if (int st = check_ffn(x)) return st;
    if (int st = check_matrix("x", x->x, x->tokens, x->width, x->x_stride)) return st;
    if (int st = check_matrix("w_gate", x->w_gate, x->hidden, x->width, x->w_stride)) return st;
    if (int st = check_matrix("w_up", x->w_up, x->hidden, x->width, x->w_stride)) return st;
    if (int st = check_matrix("w_down", x->w_down, x->width, x->hidden, x->w_down_stride)) return st;
    if (int st = check_matrix("out", x->out, x->tokens, x->width, x->width)) return st;
    if (!aligned(x->kept, 16)) return refuse(MUON_ERR_INVALID_ARG, "kept is not aligned to 16 bytes");
    if (int st = check_workspace(ws, ws_bytes, forward_bytes(x))) return st;
    if (x->tokens == 0) return done();
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t t = x->tokens, h = x->hidden, w = x->width;
    const int64_t x_step = t > 1 ? x->x_stride : w;  // (of one row it may be anything)
    bf16_t* hid = x->kept ? x->kept + 2 * t * h : static_cast<bf16_t*>(ws);
    if (few_tokens(x)) {
        FfnFew a{};
        a.x = x->x;
        a.w_gate = x->w_gate;
        a.w_up = x->w_up;
        a.w_down = x->w_down;
        a.h = hid;
        a.out = x->out;
        a.x_stride = x_step;
        a.w_stride = x->w_stride;
        a.w_down_stride = x->w_down_stride;
        a.tokens = static_cast<int>(t);
        a.width = static_cast<int>(w);
        a.hidden = static_cast<int>(h);
        a.act = static_cast<int>(x->activation);
        const int st = launched(launch_ffn_few(a, s), "feed-forward block of a few tokens");
        return st ? st : done();
    }
    float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + (x->kept ? 0 : hidden_bytes(x)));
    {
        const FfnPlan p = plan_gated(x);
        FfnGemm g{};
        add_seg(g, p.tile, true, x->x, nullptr, x_step, x->w_gate, x->w_up, x->w_stride, t, h, hid);
        set_steps(g, p, w, 1, part);
        g.act = static_cast<int>(x->activation);
        if (x->kept) {
            g.gate = x->kept;
            g.up = x->kept + t * h;
        }
        if (int st = launched(launch_ffn(FFN_GATED, p.tile, g, s), "gate and up projections")) return st;
    }
    {
        const FfnPlan p = plan_down(x);
        FfnGemm g{};
        add_seg(g, p.tile, false, hid, nullptr, h, x->w_down, nullptr, x->w_down_stride, t, w, x->out);
        set_steps(g, p, h, 1, part);
        if (int st = launched(launch_ffn(FFN_PLAIN, p.tile, g, s), "down projection")) return st;
    }
    return done();
}

int muon_feed_forward_backward(const muon_feed_forward_args* x, void* ws, size_t ws_bytes, void* stream) {
    using namespace muon;
    if (int st = check_ffn(x)) return st;
    if (int st = check_matrix("x", x->x, x->tokens, x->width, x->x_stride)) return st;
    if (int st = check_matrix("dout", x->dout, x->tokens, x->width, x->dout_stride)) return st;
    if (int st = check_matrix("w_gate", x->w_gate, x->hidden, x->width, x->w_stride)) return st;
    if (int st = check_matrix("w_up", x->w_up, x->hidden, x->width, x->w_stride)) return st;
    if (int st = check_matrix("w_down", x->w_down, x->width, x->hidden, x->w_down_stride)) return st;
    if (int st = check_matrix("dx", x->dx, x->tokens, x->width, x->width)) return st;
    if (int st = check_matrix("kept", x->kept, x->tokens, x->hidden, x->hidden)) return st;
    if (int st = check_matrix("dw_gate", x->dw_gate, x->hidden, x->width, x->width)) return st;
    if (int st = check_matrix("dw_up", x->dw_up, x->hidden, x->width, x->width)) return st;
    if (int st = check_matrix("dw_down", x->dw_down, x->width, x->hidden, x->hidden)) return st;
    if (!known_type(x->dw_type)) return refuse(MUON_ERR_INVALID_ARG, "unknown dtype");
    if (int st = check_workspace(ws, ws_bytes, backward_bytes(x))) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t t = x->tokens, h = x->hidden, w = x->width;
    const int64_t x_step = t > 1 ? x->x_stride : w;  // (of one row it may be anything)
    const int64_t do_step = t > 1 ? x->dout_stride : w;
    char* at = static_cast<char*>(ws);
    bf16_t* dgate = reinterpret_cast<bf16_t*>(at);
    bf16_t* dup = reinterpret_cast<bf16_t*>(at + hidden_bytes(x));
    float* part = reinterpret_cast<float*>(at + 2 * hidden_bytes(x));
    if (t > 0) {
        const FfnPlan p = plan_hidden(x);
        FfnGemm g{};
        add_seg(g, p.tile, false, x->dout, nullptr, do_step, x->w_down, nullptr, x->w_down_stride, t, h, nullptr);
        set_steps(g, p, w, 1, part);
        g.act = static_cast<int>(x->activation);
        g.gate = x->kept;
        g.up = x->kept + t * h;
        g.dgate = dgate;
        g.dup = dup;
        if (int st = launched(launch_ffn(FFN_HIDDEN, p.tile, g, s), "gradient of the hidden values")) return st;
    }
    if (t > 0) {
        const FfnPlan p = plan_input(x);
        FfnGemm g{};
        add_seg(g, p.tile, false, dgate, dup, h, x->w_gate, x->w_up, x->w_stride, t, w, x->dx);
        set_steps(g, p, h, 2, part);
        if (int st = launched(launch_ffn(FFN_INPUT, p.tile, g, s), "gradient of x")) return st;
    }
    {
        const FfnPlan p = plan_weights(x);
        FfnGemm g{};
        add_seg(g, p.tile, false, dgate, nullptr, h, x->x, nullptr, x_step, h, w, x->dw_gate);
        add_seg(g, p.tile, false, dup, nullptr, h, x->x, nullptr, x_step, h, w, x->dw_up);
        add_seg(g, p.tile, false, x->dout, nullptr, do_step, x->kept + 2 * t * h, nullptr, h, w, h, x->dw_down);
        set_steps(g, p, t, 1, part);
        g.out_f32 = x->dw_type == MUON_F32;
        if (int st = launched(launch_ffn(FFN_WEIGHTS, p.tile, g, s), "gradients of the matrices")) return st;
    }
    return done();
}

}  // extern "C"
