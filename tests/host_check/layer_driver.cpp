// CPU driver of the host code of the decoder layer's operators (layer_api.hip):
// their entry points are called over a sweep of sizes with made-up addresses,
// and stand-ins for the kernel launchers check, in 64-bit arithmetic or wider,
// that every workspace range a kernel addresses lies inside the workspace that
// the library asked for, that tiles, steps and rows are covered, and that grids
// fit.  Nothing is launched or dereferenced.  Built with AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_layer_host.py; prints "host check ok:
// N launches".
#include <stdio.h>
#include <stdlib.h>

#include "../../include/muon_lm.h"
#include "../../newton_schulz_09_amd/csrc/internal.hpp"
#include "../../newton_schulz_09_amd/csrc/layer_common.hpp"

namespace {

constexpr uintptr_t kWs = uintptr_t{1} << 44;
size_t g_shrink = 0, g_bytes = 0;
long g_launches = 0;
typedef __int128 wide;

[[noreturn]] void die(const char* what, long long a, long long b) {
    fprintf(stderr, "host check failed: %s (%lld, %lld)\n", what, a, b);
    abort();
}
bool is_ws(const void* p) { return reinterpret_cast<uintptr_t>(p) >= kWs; }
void in_ws(const void* p, wide bytes, const char* what) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (lo < kWs || lo % 16 != 0 || lo - kWs + bytes > g_bytes) die(what, static_cast<long long>(lo - kWs), static_cast<long long>(bytes));
}
// (HIP takes fewer than 2^32 threads along x)
void grid(wide blocks, int threads, const char* what) {
    if (blocks <= 0 || blocks * threads >= (wide{1} << 32)) die(what, static_cast<long long>(blocks), threads);
    ++g_launches;
}
// ranges of the workspace that one launch reads and writes
struct Range {
    uintptr_t lo;
    wide bytes;
} g_used[8];
int g_n = 0;
void apart(const void* p, wide bytes, const char* what) {
    in_ws(p, bytes, what);
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    for (int i = 0; i < g_n; ++i)
        if (static_cast<wide>(lo) < g_used[i].lo + g_used[i].bytes && static_cast<wide>(g_used[i].lo) < lo + bytes) die(what, i, g_n);
    g_used[g_n++] = {lo, bytes};
}

}  // namespace

namespace muon {

int fail_status(int status, const char* msg) {
    if (status == MUON_ERR_HIP) die(msg, status, 0);
    return status;
}

hipError_t launch_dropout(const DropArgs& a, hipStream_t) {
    const wide blocks = ((wide{a.n} + 7) / 8 + 255) / 256;
    if (blocks <= 0 || blocks >= (wide{1} << 31)) die("dropout", static_cast<long long>(blocks), 0);
    if (a.drop.threshold > 65536) die("threshold", a.drop.threshold, 0);
    ++g_launches;
    return hipSuccess;
}

static void rows_of(const ResidArgs& a) {
    if (static_cast<int64_t>(a.threads) * a.pieces * 8 < a.width) die("a row does not fit its threads", a.threads, a.width);
    if (a.threads < 8 || a.threads > 512 || (a.threads & (a.threads - 1)) || a.pieces < 1 || a.pieces > 2 ||
        (a.pieces == 1 ? a.threads > 64 : a.threads < 64))
        die("no kernel", a.threads, a.pieces);
}
hipError_t launch_resid_norm(const ResidArgs& a, hipStream_t) {
    rows_of(a);
    grid(a.blocks, a.threads == 512 ? 512 : 256, "norms");
    return hipSuccess;
}
hipError_t launch_resid_norm_bwd(const ResidArgs& a, hipStream_t) {
    rows_of(a);
    g_n = 0;
    if (a.blocks > 0) grid(a.blocks, a.threads == 512 ? 512 : 256, "norms backward");
    apart(a.part, wide{a.blocks} * 4 * a.width * 4, "sums of vectors");
    if (a.gate_part) apart(a.gate_part, wide{a.groups} * a.chunks * a.width * 4, "sums of gates");
    if (a.chunks < 1 || a.per < 1 || (a.chunks > 1 && a.per > 1)) die("chunks", a.chunks, a.per);
    if (a.chunks > 1 ? a.blocks != a.groups * a.chunks : wide{a.blocks} * a.per < a.groups) die("groups", a.blocks, a.groups);
    if (a.gate_kind == GATE_SEQUENCE && a.chunks > 1 && !a.gate_part) die("no place for the gates' sums", a.chunks, 0);
    if ((a.gate_part ? a.groups : 0) + 4 > 65535) die("grid rows", a.groups, 0);
    if (wide{a.groups} * (a.gate_kind == GATE_SEQUENCE ? a.s : a.rows) != a.rows) die("rows", a.groups, a.rows);
    return hipSuccess;
}

hipError_t launch_ffn(FfnKind kind, FfnTile tile, const FfnGemm& g, hipStream_t) {
    if (g.nseg < 1 || g.nseg > 3 || (tile != FFN_256 && tile != FFN_128)) die("segments", g.nseg, tile);
    g_n = 0;
    const int cols = kind == FFN_GATED ? tile / 2 : tile;
    int64_t tiles = 0;
    for (int i = 0; i < g.nseg; ++i) {
        const FfnSeg& s = g.seg[i];
        if (s.first != tiles) die("first tile", s.first, tiles);
        if (wide{s.tiles_m} * tile < s.m || wide{s.tiles_n} * cols < s.n || s.tiles_m < 1 || s.tiles_n < 1) die("tiles", s.m, s.n);
        if (s.band < 1) die("band", s.band, 0);
        tiles += static_cast<int64_t>(s.tiles_m) * s.tiles_n;
        // offsets inside a tile stay below the one that means "past the end"
        if (s.ldp < 0 || s.ldq < 0 || wide{s.ldp} * 2 * 256 >= (wide{1} << 31) || wide{s.ldq} * 2 * 256 >= (wide{1} << 31)) die("strides", s.ldp, s.ldq);
        for (const bf16_t* p : {s.p[0], s.p[1], s.q[0]})
            if (p && is_ws(p)) in_ws(p, (kind == FFN_WEIGHTS ? wide{g.k} : wide{s.m}) * s.ldp * 2, "operand");
        if (s.out && is_ws(s.out)) in_ws(s.out, wide{s.m} * s.n * 2, "hidden values");
        if ((kind == FFN_HIDDEN) != (s.out == nullptr)) die("out", kind, 0);
    }
    if (tiles != g.tiles || g.full < 0 || g.full > g.tiles) die("tiles of all", tiles, g.tiles);
    const wide tail = g.tiles - g.full;
    if (tail) apart(g.part, tail * g.splits * tile * tile * 4, "sums of splits");
    else if (g.part) die("parts without splits", 0, 0);
    grid(g.full + tail * g.splits, tile == FFN_256 ? 512 : 256, "feed-forward");
    if (tail) grid(tail * tile * cols / 2048, 256, "join");
    const wide steps = (wide{g.k} + kFfnStep - 1) / kFfnStep * g.phases;
    if (g.splits < 1 || wide{g.splits} * g.split_steps < steps || steps > 0x7fffffff) die("steps", g.splits, g.split_steps);
    if (kind == FFN_HIDDEN)
        for (const bf16_t* p : {g.dgate, g.dup}) apart(p, wide{g.seg[0].m} * g.seg[0].n * 2, "gradients of gate and up");
    return hipSuccess;
}

hipError_t launch_ffn_few(const FfnFew& a, hipStream_t) {
    if (a.tokens < 1 || a.tokens > kFewTokens) die("few tokens", a.tokens, 0);
    g_n = 0;
    const int m = a.tokens <= 16 ? 1 : 2;
    apart(a.h, (wide{a.hidden} + 31) / 32 * m * 1024, "hidden values in fragments");
    grid((a.hidden + 15) / 16, 512, "few, gated");
    grid((a.width + 15) / 16, 1024, "few, down");
    return hipSuccess;
}

}  // namespace muon

namespace {

void* ws(size_t bytes) {
    if (bytes == 0) die("no workspace size", 0, 0);
    g_bytes = bytes - g_shrink;
    return reinterpret_cast<void*>(kWs);
}
template <typename T>
T* fake() { return reinterpret_cast<T*>(uintptr_t{1} << 40); }
void ok(int st, const char* what) {
    if (st != MUON_OK) die(what, st, 0);
}
uint64_t g_state = 12345;
uint64_t next() {
    g_state = g_state * 6364136223846793005ull + 1442695040888963407ull;
    return g_state >> 33;
}
int64_t pick(int64_t lo, int64_t hi) {  // log-uniform
    int64_t x = hi;
    for (int i = 0; i < static_cast<int>(next() % 40) && x > lo; ++i) x = x / 2;
    x += static_cast<int64_t>(next() % 7);
    return x < lo ? lo : (x > hi ? hi : x);
}

}  // namespace

int main(int argc, char** argv) {
    if (argc > 1) g_shrink = 256;
    long refused = 0;
    for (int it = 0; it < 40000; ++it) {
        muon_feed_forward_args x{};
        x.x = x.w_gate = x.w_up = x.w_down = x.dout = fake<uint16_t>();
        x.out = x.dx = fake<uint16_t>();
        x.kept = it & 1 ? fake<uint16_t>() : nullptr;
        x.dw_gate = x.dw_up = x.dw_down = fake<char>();
        x.tokens = it % 3 == 0 ? pick(0, 64) : pick(0, (int64_t{1} << 29) - 1);
        x.width = 8 * pick(1, (1 << 18) - 1);
        x.hidden = 8 * pick(1, (1 << 18) - 1);
        const int64_t more = it % 5 == 0 ? 8 * pick(0, 100) : 0;
        auto stride = [&](int64_t n) { return n + more < (1 << 21) ? n + more : n; };
        x.x_stride = x.tokens > 1 ? stride(x.width) : -5;  // (of one row it may be anything)
        x.dout_stride = x.tokens > 1 ? stride(x.width) : int64_t{1} << 60;
        x.w_stride = stride(x.width);
        x.w_down_stride = stride(x.hidden);
        x.activation = it % 4;
        x.dw_type = it & 1 ? MUON_F32 : MUON_BF16;
        const size_t f = muon_feed_forward_workspace_size(&x), b = muon_feed_forward_backward_workspace_size(&x);
        if ((f == 0) != (b == 0)) die("one direction is refused", it, 0);
        if (f == 0) {
            ++refused;
            continue;
        }
        ok(muon_feed_forward(&x, ws(f), f, nullptr), "feed-forward");
        if (!x.kept) x.kept = fake<uint16_t>();
        ok(muon_feed_forward_backward(&x, ws(b), b, nullptr), "feed-forward backward");
    }
    if (refused > 30000) die("sizes refused", refused, 0);  // (products of more than 2^23 tiles)
    for (int it = 0; it < 40000; ++it) {
        muon_residual_norm_args x{};
        x.has_block = it % 7 != 0;
        x.x = x.y = x.dz = x.dx_out = fake<char>() + (it % 11 == 0 ? 4 : 0);
        x.x_out = x.z = x.dx = x.dy = fake<char>();
        x.gate_kind = x.has_block ? it % 4 : 0;
        x.gate = fake<char>();
        x.dgate = x.gate_kind ? fake<char>() : nullptr;
        x.post = x.has_block && (it & 8);
        if (it & 16) x.residual_scale = x.dresidual_scale = fake<float>();
        if (it & 32) x.dpre_weight = fake<float>();
        if (x.post && (it & 64)) x.post_weight = x.dpost_weight = fake<float>();
        x.width = pick(1, MUON_RESIDUAL_NORM_MAX_WIDTH);
        x.batch = pick(0, x.gate_kind == MUON_GATE_SEQUENCE ? 1 << 20 : (1 << 29) - 1);
        x.s = pick(0, (1 << 29) - 1);
        x.x_stride = x.y_stride = x.gate_stride = x.x_out_stride = x.dz_stride = x.dx_out_stride = x.width + (it % 13 == 0 ? 3 : 0);
        x.stream_type = it & 2 ? MUON_F32 : MUON_BF16;
        x.block_type = it & 2 && it & 4 ? MUON_F32 : MUON_BF16;
        x.eps = 1e-6;
        x.p = x.has_block ? 0.25 * (it % 5) : 0.0;
        const size_t b = muon_residual_norm_backward_workspace_size(&x);
        if (b == 0) {  // (2^62 elements and more)
            if (wide{x.batch} * x.s * x.width <= (wide{1} << 62)) die("norms refused", x.batch, x.s);
            continue;
        }
        ok(muon_residual_norm(&x, nullptr), "norms");
        ok(muon_residual_norm_backward(&x, ws(b), b, nullptr), "norms backward");
    }
    for (int it = 0; it < 2000; ++it)
        ok(muon_dropout(fake<char>(), fake<char>(), pick(0, int64_t{1} << 41), it & 1 ? MUON_F32 : MUON_BF16, 0.001 * (it % 1001), 1, 2,
                        it & 2 ? fake<int64_t>() : nullptr, nullptr),
           "dropout");
    printf("host check ok: %ld launches\n", g_launches);
    return 0;
}
