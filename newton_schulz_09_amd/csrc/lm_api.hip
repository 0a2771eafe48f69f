// C ABI of the language-model operators: validation, plans and workspace
// layout (declared and documented in include/muon_lm.h).
#include <math.h>

#include "../../include/muon_lm.h"
#include "internal.hpp"
#include "lm_common.hpp"
#include "lm_host.hpp"

namespace muon {

namespace {

// ------------------------------------------------------------- attention

int check_sizes(const muon_attention_args* x) {
    if (!x) return refuse(MUON_ERR_INVALID_ARG, "null arguments");
    if (x->batch < 0 || x->sq < 0 || x->sk < 0) return refuse(MUON_ERR_INVALID_ARG, "negative size");
    if (x->heads <= 0 || x->kv_heads <= 0 || x->heads % x->kv_heads != 0)
        return refuse(MUON_ERR_INVALID_ARG, "heads (%lld) must be a multiple of kv_heads (%lld)", (long long)x->heads,
                      (long long)x->kv_heads);
    if (x->d <= 0 || x->d % 8 != 0 || x->d > MUON_ATTENTION_MAX_D)
        return refuse(MUON_ERR_UNSUPPORTED, "head size %lld is not a multiple of 8 up to %d", (long long)x->d,
                      MUON_ATTENTION_MAX_D);
    if (x->sq >= kMaxSeq || x->sk >= kMaxSeq) return refuse(MUON_ERR_UNSUPPORTED, "a length of 2^29 or more");
    if (!(x->scale > 0.0) || !isfinite(x->scale) || !(static_cast<float>(x->scale) > 0.0f) ||
        !isfinite(static_cast<float>(x->scale)))
        return refuse(MUON_ERR_INVALID_ARG, "scale must be positive and finite");
    if (!(x->softcap >= 0.0) || !isfinite(static_cast<float>(x->softcap)) ||
        (x->softcap > 0.0 && !(static_cast<float>(x->softcap) > 0.0f)))
        return refuse(MUON_ERR_INVALID_ARG, "softcap must be zero or positive and finite");
    if (x->window < 0) return refuse(MUON_ERR_INVALID_ARG, "window must be >= 0 (got %lld)", (long long)x->window);
    // every grid is at most one workgroup per 32 rows and 4 key tiles of a head
    const int64_t heads = times(x->batch, x->heads);
    const int64_t rows = times(heads, x->sq > x->sk ? x->sq : x->sk);
    if (heads < 0 || rows < 0 || heads > kMaxBlocks || rows / 32 + heads > kMaxBlocks)
        return refuse(MUON_ERR_UNSUPPORTED, "too many rows");
    return MUON_OK;
}

int check_rows(const char* name, const void* p, const int64_t* strides, int64_t batch, int64_t s, int64_t heads) {
    if (batch == 0 || s == 0) return MUON_OK;
    if (!p) return refuse(MUON_ERR_INVALID_ARG, "%s is null", name);
    if (!aligned(p, 16)) return refuse(MUON_ERR_INVALID_ARG, "%s is not aligned to 16 bytes", name);
    const int64_t sizes[3] = {batch, s, heads};
    for (int i = 0; i < 3; ++i)
        if (sizes[i] > 1 && (strides[i] < 0 || strides[i] % 8 != 0))
            return refuse(MUON_ERR_INVALID_ARG, "%s: stride %lld is not a multiple of 8 elements", name,
                          (long long)strides[i]);
    if (s > 1 && strides[1] >= kMaxRowStride)
        return refuse(MUON_ERR_UNSUPPORTED, "%s: position stride of 2^24 elements or more", name);
    return MUON_OK;
}

int check_masks(const muon_attention_args* x) {
    for (const void* p : {static_cast<const void*>(x->slopes), static_cast<const void*>(x->documents),
                          static_cast<const void*>(x->prefix), static_cast<const void*>(x->lengths),
                          static_cast<const void*>(x->starts)})
        if (!aligned(p, 4)) return refuse(MUON_ERR_INVALID_ARG, "slopes or a mask is not aligned to 4 bytes");
    if (x->documents && x->batch > 1 && x->documents_stride < 0)
        return refuse(MUON_ERR_INVALID_ARG, "documents: stride %lld is negative", (long long)x->documents_stride);
    return MUON_OK;
}

struct AttnPlan {
    bool split;
    int splits, chunk;
    size_t off_docs, off_part, off_stats, bytes;
};

// Few rows per key head (a step of generation), or many keys and at most 48
// blocks of 128 queries for 256 CUs: the keys are split.  (64 queries of 32
// heads of 128 over 16384 keys, 32 blocks: 301 -> 86 us; 256 of 24 heads over
// 2048, 48 blocks: 42 -> 39; 2048 of 6 heads, 96 blocks: 43 -> 57, not split.)
AttnPlan plan_forward(const muon_attention_args* x) {
    AttnPlan p{};
    const int64_t grp = x->heads / x->kv_heads, rows = grp * x->sq, tiles = div_up(x->sk, kTile);
    const int64_t blocks = div_up(x->sq, 128) * x->batch * x->heads;
    p.split = rows <= 32 || (blocks <= 48 && tiles >= 32);
    p.splits = 1;
    p.chunk = static_cast<int>(tiles > 0 ? tiles : 1);
    if (p.split) {
        const int64_t base = div_up(rows, 32) * x->batch * x->kv_heads;
        int64_t n = base > 0 ? div_up(2048, base) : 1;
        if (n > tiles / 16) n = tiles / 16;
        if (n < 1) n = 1;
        p.chunk = static_cast<int>(tiles > 0 ? div_up(tiles, n) : 1);
        p.splits = static_cast<int>(tiles > 0 ? div_up(tiles, p.chunk) : 1);
    }
    size_t at = 0;
    p.off_docs = at;
    if (x->documents) at = align256(at + static_cast<size_t>(x->batch) * tiles * sizeof(int2));
    p.off_part = at;
    if (p.splits > 1) {
        const int64_t n = x->batch * x->heads * x->sq * p.splits;
        at = align256(at + static_cast<size_t>(part_outputs(n) + n * x->d) * sizeof(float));
    }
    p.bytes = at > 256 ? at : 256;
    return p;
}

AttnPlan plan_backward(const muon_attention_args* x) {
    AttnPlan p{};
    const int64_t tiles = div_up(x->sk, kTile);
    size_t at = 0;
    p.off_docs = at;
    if (x->documents) at = align256(at + static_cast<size_t>(x->batch) * tiles * sizeof(int2));
    p.off_stats = at;
    at = align256(at + static_cast<size_t>(x->batch) * x->heads * x->sq * 2 * sizeof(float));
    p.bytes = at > 256 ? at : 256;
    return p;
}

AttnArgs attn_args(const muon_attention_args* x, const AttnPlan& p, void* ws) {
    AttnArgs a{};
    a.q = x->q;
    a.k = x->k;
    a.v = x->v;
    a.out = x->out;
    a.lse = x->lse;
    a.dout = x->dout;
    a.dq = x->dq;
    a.dk = x->dk;
    a.dv = x->dv;
    // the stride of a dimension of one entry is never used: any value may be
    // there, and the kernels' products of it must not pass their types
    auto st = [](const int64_t* s, int64_t b, int64_t n, int64_t h, int64_t& sb, int64_t& ss, int64_t& sh) {
        sb = b > 1 ? s[0] : 0;
        ss = n > 1 ? s[1] : 0;
        sh = h > 1 ? s[2] : 0;
    };
    st(x->q_strides, x->batch, x->sq, x->heads, a.q_b, a.q_s, a.q_h);
    st(x->k_strides, x->batch, x->sk, x->kv_heads, a.k_b, a.k_s, a.k_h);
    st(x->v_strides, x->batch, x->sk, x->kv_heads, a.v_b, a.v_s, a.v_h);
    st(x->out_strides, x->batch, x->sq, x->heads, a.o_b, a.o_s, a.o_h);
    st(x->dout_strides, x->batch, x->sq, x->heads, a.do_b, a.do_s, a.do_h);
    a.doc_b = x->batch > 1 ? x->documents_stride : 0;
    a.slopes = x->slopes;
    a.documents = x->sk > 0 ? x->documents : nullptr;
    a.prefix = x->prefix;
    a.lengths = x->lengths;
    a.starts = x->starts;
    char* w = static_cast<char*>(ws);
    a.doc_tiles = reinterpret_cast<int2*>(w + p.off_docs);
    a.part = reinterpret_cast<float*>(w + p.off_part);
    a.stats = reinterpret_cast<float*>(w + p.off_stats);
    a.delta_at = x->batch * x->heads * x->sq;
    a.b = static_cast<int>(x->batch);
    a.sq = static_cast<int>(x->sq);
    a.sk = static_cast<int>(x->sk);
    a.hq = static_cast<int>(x->heads);
    a.hkv = static_cast<int>(x->kv_heads);
    a.grp = a.hq / a.hkv;
    a.d = static_cast<int>(x->d);
    a.causal = x->causal != 0;
    a.window = static_cast<int>(x->window < kMaxSeq ? x->window : 0);
    a.n_tiles = static_cast<int>(div_up(x->sk, kTile));
    a.splits = p.splits;
    a.chunk = p.chunk;
    a.scale = static_cast<float>(x->scale);
    a.softcap = static_cast<float>(x->softcap);
    return a;
}

// -------------------------------------------------------------- QK norm

int check_qk(const muon_qk_norm_rope_args* x) {
    if (!x) return refuse(MUON_ERR_INVALID_ARG, "null arguments");
    if (x->batch < 0 || x->s < 0 || x->heads[0] < 0 || x->heads[1] < 0 || x->limit < 0)
        return refuse(MUON_ERR_INVALID_ARG, "negative size");
    if (x->dtype != MUON_F32 && x->dtype != MUON_BF16) return refuse(MUON_ERR_INVALID_ARG, "unknown dtype");
    if (x->d <= 0 || x->d % 2 != 0 || x->d > MUON_QK_NORM_MAX_D)
        return refuse(MUON_ERR_UNSUPPORTED, "head size %lld is not even and up to %d", (long long)x->d, MUON_QK_NORM_MAX_D);
    if (!(x->eps >= 0.0) || !isfinite(static_cast<float>(x->eps)))
        return refuse(MUON_ERR_INVALID_ARG, "eps must be >= 0 and finite");
    if (x->batch >= kMaxSeq || x->s >= kMaxSeq || x->heads[0] >= (1 << 15) || x->heads[1] >= (1 << 15) ||
        x->limit > kMaxBlocks)
        return refuse(MUON_ERR_UNSUPPORTED, "too many rows");
    return MUON_OK;
}

struct QkPlan {
    bool vector;
    int lanes, chunk, runs_q, runs, blocks;
};

// A group of lanes takes one token and a run of its heads, so the token's
// angles are loaded once for all of them; the runs are halved until the chip
// has 8 waves per CU to work on (32 tokens of 40 float32 heads of 128: one
// head per group).  The backward pass, whose workgroups leave a row of weight
// gradients each, takes about 4 workgroups per CU and walks the tokens.
QkPlan plan_qk(const muon_qk_norm_rope_args* x, bool vector, bool backward) {
    QkPlan p{};
    p.vector = vector;
    const int v = vector ? (x->dtype == MUON_BF16 ? 8 : 4) : 1;
    p.lanes = 1;
    while (p.lanes < 64 && p.lanes * v < x->d / 2) p.lanes <<= 1;
    const int64_t tokens = x->batch * x->s, groups = 256 / p.lanes, blocks = div_up(tokens, groups);
    const int64_t most = x->heads[0] > x->heads[1] ? x->heads[0] : x->heads[1];
    int64_t chunk = most > 0 ? most : 1;
    auto runs = [&](int64_t heads) { return div_up(heads, chunk); };
    while (chunk > 1 && blocks * (runs(x->heads[0]) + runs(x->heads[1])) < 512) chunk = div_up(chunk, 2);
    p.chunk = static_cast<int>(chunk);
    p.runs_q = static_cast<int>(runs(x->heads[0]));
    p.runs = p.runs_q + static_cast<int>(runs(x->heads[1]));
    int64_t limit = 1 << 20;
    if (backward) limit = p.runs > 0 && p.runs < 1024 ? 1024 / p.runs : 1;
    p.blocks = static_cast<int>(blocks < 1 ? 1 : (blocks < limit ? blocks : limit));
    return p;
}

int run_qk(const muon_qk_norm_rope_args* x, bool backward, void* ws, size_t ws_bytes, hipStream_t stream) {
    if (int st = check_qk(x)) return st;
    const bool rows = x->batch > 0 && x->s > 0;
    const int64_t align = x->dtype == MUON_BF16 ? 8 : 4;
    bool vec = x->d % (2 * align) == 0 && x->d / 2 <= 64 * align;
    for (int i = 0; i < 2; ++i) {
        if (rows && x->heads[i] > 0) {
            if (!x->x[i] || !x->out[i] || (backward && !x->dz[i])) return refuse(MUON_ERR_INVALID_ARG, "null pointer argument");
            const int64_t elem = x->dtype == MUON_BF16 ? 2 : 4;
            if (!aligned(x->x[i], elem) || !aligned(x->out[i], elem) || (backward && !aligned(x->dz[i], elem)))
                return refuse(MUON_ERR_INVALID_ARG, "a tensor is not aligned to its type");
            vec = vec && aligned(x->x[i], 16) && aligned(x->out[i], 16) && (!backward || aligned(x->dz[i], 16));
            const int64_t sizes[3] = {x->batch, x->s, x->heads[i]};
            for (int j = 0; j < 3; ++j)
                if (sizes[j] > 1) {
                    if (x->x_strides[i][j] < 0 || (backward && x->dz_strides[i][j] < 0))
                        return refuse(MUON_ERR_INVALID_ARG, "negative stride");
                    vec = vec && x->x_strides[i][j] % align == 0 && (!backward || x->dz_strides[i][j] % align == 0);
                }
        }
    }
    for (const void* p : {static_cast<const void*>(x->weight[0]), static_cast<const void*>(x->weight[1]),
                          static_cast<const void*>(backward ? x->dweight[0] : nullptr),
                          static_cast<const void*>(backward ? x->dweight[1] : nullptr),
                          static_cast<const void*>(x->table), static_cast<const void*>(x->positions)})
        if (!aligned(p, 4)) return refuse(MUON_ERR_INVALID_ARG, "a weight, the table or positions are not aligned to 4 bytes");
    const bool any = rows && (x->heads[0] > 0 || x->heads[1] > 0);
    if (any && !x->table) return refuse(MUON_ERR_INVALID_ARG, "table is null");
    const bool want_dw = backward && (x->dweight[0] || x->dweight[1]);
    if (backward)
        if (int st = check_workspace(ws, ws_bytes, muon_qk_norm_rope_backward_workspace_size(x))) return st;
    if (!any && !want_dw) return done();
    QkArgs a{};
    for (int i = 0; i < 2; ++i) {
        a.x[i] = x->x[i];
        a.dz[i] = x->dz[i];
        a.y[i] = x->out[i];
        a.w[i] = x->weight[i];
        a.dw[i] = x->dweight[i];
        a.x_b[i] = x->batch > 1 ? x->x_strides[i][0] : 0;
        a.x_s[i] = x->s > 1 ? x->x_strides[i][1] : 0;
        a.x_h[i] = x->heads[i] > 1 ? x->x_strides[i][2] : 0;
        a.z_b[i] = x->batch > 1 ? x->dz_strides[i][0] : 0;
        a.z_s[i] = x->s > 1 ? x->dz_strides[i][1] : 0;
        a.z_h[i] = x->heads[i] > 1 ? x->dz_strides[i][2] : 0;
        a.heads[i] = static_cast<int>(x->heads[i]);
    }
    a.table = x->table;
    a.positions = x->positions;
    a.b = static_cast<int>(x->batch);
    a.s = static_cast<int>(x->s);
    a.d = static_cast<int>(x->d);
    a.limit = static_cast<int>(x->limit);
    a.type = static_cast<int>(x->dtype);
    const QkPlan p = plan_qk(x, vec, backward);
    a.lanes = p.lanes;
    a.chunk = p.chunk;
    a.runs_q = p.runs_q;
    a.blocks = p.blocks;
    a.vector = vec;
    a.eps = static_cast<float>(x->eps);
    if (!any) a.b = 0;
    a.part = want_dw ? static_cast<float*>(ws) : nullptr;
    const int st = launched(backward ? launch_qk_norm_bwd(a, stream) : launch_qk_norm(a, stream), "norm and rotation");
    return st ? st : done();
}

// ------------------------------------------------------------ embedding

struct EmbedPlan {
    size_t off_perm, off_ids, off_offset, off_part, bytes;
};
bool embed_sizes_ok(int64_t n, int64_t vocab, int64_t width) {
    return n >= 0 && vocab > 0 && width > 0 && n < kMaxBlocks && vocab < kMaxBlocks && width <= (1 << 20) &&
           times(n, width) >= 0 && times(vocab, width) >= 0;
}
// 8 entries for a few thousand tokens (one batch of loads), 32 for many: longer
// windows leave fewer sums to join, shorter ones keep more of the chip busy.
int embed_window(int64_t n) {
    int w = 8;
    while (w < 32 && n / (2 * w) >= 512) w *= 2;
    return w;
}
EmbedPlan embed_plan(int64_t n, int64_t vocab, int64_t width) {
    EmbedPlan p{};
    size_t at = 0;
    p.off_perm = at;
    at = align256(at + static_cast<size_t>(n) * 4);
    p.off_ids = at;
    at = align256(at + static_cast<size_t>(n) * 4);
    p.off_offset = at;
    at = align256(at + (static_cast<size_t>(vocab) + 1) * 4);
    p.off_part = at;
    at = align256(at + static_cast<size_t>(div_up(n, embed_window(n))) * 2 * width * sizeof(float));
    p.bytes = at;
    return p;
}

int check_embed(const void* tokens, int token_bytes, const void* src, int src_type, const void* dst, int dst_type,
                int64_t n, int64_t vocab, int64_t width, float scale) {
    if (n < 0 || vocab <= 0 || width <= 0) return refuse(MUON_ERR_INVALID_ARG, "n must be >= 0, vocab and width > 0");
    if (!embed_sizes_ok(n, vocab, width)) return refuse(MUON_ERR_UNSUPPORTED, "too many tokens, rows or columns");
    if (token_bytes != 4 && token_bytes != 8) return refuse(MUON_ERR_INVALID_ARG, "tokens are int32 or int64");
    for (int t : {src_type, dst_type})
        if (t != MUON_F32 && t != MUON_BF16) return refuse(MUON_ERR_INVALID_ARG, "unknown dtype");
    if (!isfinite(scale)) return refuse(MUON_ERR_INVALID_ARG, "scale must be finite");
    if (n > 0 && (!tokens || !src)) return refuse(MUON_ERR_INVALID_ARG, "null pointer argument");
    if (!aligned(tokens, token_bytes) || !aligned(src, src_type == MUON_BF16 ? 2 : 4) ||
        !aligned(dst, dst_type == MUON_BF16 ? 2 : 4))
        return refuse(MUON_ERR_INVALID_ARG, "a tensor is not aligned to its type");
    return MUON_OK;
}

EmbedArgs embed_args(const void* tokens, int token_bytes, const void* src, int src_type, void* dst, int dst_type,
                     int64_t n, int64_t vocab, int64_t width, float scale) {
    EmbedArgs a{};
    a.tokens = tokens;
    a.tokens64 = token_bytes == 8;
    a.n = n;
    a.vocab = vocab;
    a.width = static_cast<int>(width);
    a.src = src;
    a.dst = dst;
    a.src_type = src_type;
    a.dst_type = dst_type;
    a.vector = width % 8 == 0 && aligned(src, 16) && aligned(dst, 16);
    a.scale = scale;
    return a;
}

}  // namespace

}  // namespace muon

extern "C" {

size_t muon_attention_workspace_size(const muon_attention_args* args) {
    using namespace muon;
    return check_sizes(args) ? 0 : plan_forward(args).bytes;
}

size_t muon_attention_backward_workspace_size(const muon_attention_args* args) {
    using namespace muon;
    return check_sizes(args) ? 0 : plan_backward(args).bytes;
}

int muon_attention(const muon_attention_args* x, void* ws, size_t ws_bytes, void* stream) {
    using namespace muon;
    if (int st = check_sizes(x)) return st;
    if (int st = check_masks(x)) return st;
    if (int st = check_rows("q", x->q, x->q_strides, x->batch, x->sq, x->heads)) return st;
    if (int st = check_rows("k", x->k, x->k_strides, x->batch, x->sk, x->kv_heads)) return st;
    if (int st = check_rows("v", x->v, x->v_strides, x->batch, x->sk, x->kv_heads)) return st;
    if (int st = check_rows("out", x->out, x->out_strides, x->batch, x->sq, x->heads)) return st;
    if (x->batch > 0 && x->sq > 0 && (!x->lse || !aligned(x->lse, 4)))
        return refuse(MUON_ERR_INVALID_ARG, "lse is null or not aligned");
    const AttnPlan p = plan_forward(x);
    if (int st = check_workspace(ws, ws_bytes, p.bytes)) return st;
    if (x->batch == 0 || x->sq == 0) return done();
    const AttnArgs a = attn_args(x, p, ws);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (a.documents)
        if (int st = launched(launch_attn_doc_tiles(a, s), "document ranges")) return st;
    if (int st = launched(p.split ? launch_attn_split(a, s) : launch_attn_fwd(a, s), "attention")) return st;
    return done();
}

int muon_attention_backward(const muon_attention_args* x, void* ws, size_t ws_bytes, void* stream) {
    using namespace muon;
    if (int st = check_sizes(x)) return st;
    if (int st = check_masks(x)) return st;
    if (int st = check_rows("q", x->q, x->q_strides, x->batch, x->sq, x->heads)) return st;
    if (int st = check_rows("k", x->k, x->k_strides, x->batch, x->sk, x->kv_heads)) return st;
    if (int st = check_rows("v", x->v, x->v_strides, x->batch, x->sk, x->kv_heads)) return st;
    if (int st = check_rows("out", x->out, x->out_strides, x->batch, x->sq, x->heads)) return st;
    if (int st = check_rows("dout", x->dout, x->dout_strides, x->batch, x->sq, x->heads)) return st;
    if (x->batch > 0 && x->sq > 0 && (!x->lse || !x->dq || !aligned(x->lse, 4) || !aligned(x->dq, 16)))
        return refuse(MUON_ERR_INVALID_ARG, "lse or dq is null or not aligned");
    if (x->batch > 0 && x->sk > 0 && (!x->dk || !x->dv || !aligned(x->dk, 16) || !aligned(x->dv, 16)))
        return refuse(MUON_ERR_INVALID_ARG, "dk or dv is null or not aligned");
    const AttnPlan p = plan_backward(x);
    if (int st = check_workspace(ws, ws_bytes, p.bytes)) return st;
    if (x->batch == 0) return done();
    const AttnArgs a = attn_args(x, p, ws);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (a.documents)
        if (int st = launched(launch_attn_doc_tiles(a, s), "document ranges")) return st;
    if (x->sq > 0)
        if (int st = launched(launch_attn_bwd_dq(a, s), "gradient of the queries")) return st;
    if (x->sk > 0)
        if (int st = launched(launch_attn_bwd_dkv(a, s), "gradients of keys and values")) return st;
    return done();
}

size_t muon_qk_norm_rope_backward_workspace_size(const muon_qk_norm_rope_args* x) {
    using namespace muon;
    if (check_qk(x)) return 0;
    // a row of sums per workgroup; the pointers' alignment, which decides
    // between the two plans, is not looked at here
    size_t n = 256;
    for (const bool vector : {false, true}) {
        const QkPlan p = plan_qk(x, vector, true);
        const size_t bytes = align256(static_cast<size_t>(p.blocks) * p.runs * x->d * sizeof(float));
        if (bytes > n) n = bytes;
    }
    return n;
}

int muon_qk_norm_rope(const muon_qk_norm_rope_args* x, void* stream) {
    return muon::run_qk(x, false, nullptr, 0, static_cast<hipStream_t>(stream));
}

int muon_qk_norm_rope_backward(const muon_qk_norm_rope_args* x, void* ws, size_t ws_bytes, void* stream) {
    return muon::run_qk(x, true, ws, ws_bytes, static_cast<hipStream_t>(stream));
}

int muon_embedding(const void* tokens, int token_bytes, const void* table, int table_type, void* out, int out_type,
                   int64_t n, int64_t vocab, int64_t width, float scale, void* stream) {
    using namespace muon;
    if (int st = check_embed(tokens, token_bytes, table, table_type, out, out_type, n, vocab, width, scale)) return st;
    if (n > 0 && !out) return refuse(MUON_ERR_INVALID_ARG, "null pointer argument");
    if (n == 0) return done();
    const EmbedArgs a = embed_args(tokens, token_bytes, table, table_type, out, out_type, n, vocab, width, scale);
    const int st = launched(launch_embed(a, static_cast<hipStream_t>(stream)), "embedding");
    return st ? st : done();
}

size_t muon_embedding_backward_workspace_size(int64_t n, int64_t vocab, int64_t width) {
    using namespace muon;
    return embed_sizes_ok(n, vocab, width) ? embed_plan(n, vocab, width).bytes : 0;
}

int muon_embedding_backward(const void* tokens, int token_bytes, const void* dout, int dout_type, void* dtable,
                            int table_type, int64_t n, int64_t vocab, int64_t width, float scale, void* ws,
                            size_t ws_bytes, void* stream) {
    using namespace muon;
    if (int st = check_embed(tokens, token_bytes, dout, dout_type, dtable, table_type, n, vocab, width, scale)) return st;
    if (!dtable) return refuse(MUON_ERR_INVALID_ARG, "null pointer argument");
    const EmbedPlan p = embed_plan(n, vocab, width);
    if (int st = check_workspace(ws, ws_bytes, p.bytes)) return st;
    EmbedArgs a = embed_args(tokens, token_bytes, dout, dout_type, dtable, table_type, n, vocab, width, scale);
    char* w = static_cast<char*>(ws);
    a.perm = reinterpret_cast<int32_t*>(w + p.off_perm);
    a.ids = reinterpret_cast<int32_t*>(w + p.off_ids);
    a.offset = reinterpret_cast<int32_t*>(w + p.off_offset);
    a.part = reinterpret_cast<float*>(w + p.off_part);
    a.window = embed_window(n);
    const int st = launched(launch_embed_bwd(a, static_cast<hipStream_t>(stream)), "gradient of the embedding");
    return st ? st : done();
}

}  // extern "C"
