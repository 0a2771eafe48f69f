// CPU driver of the host code of the language-model operators (lm_api.hip):
// their entry points are called over a sweep of sizes with made-up addresses,
// and stand-ins for the kernel launchers check, in 64-bit arithmetic, that
// every workspace range a kernel addresses lies inside the workspace that the
// library asked for and that grids fit.  Nothing is launched or dereferenced.
// Built with AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_lm_host.py; prints "host check ok: N launches".
#include <stdio.h>
#include <stdlib.h>

#include "../../include/muon_lm.h"
#include "../../newton_schulz_09_amd/csrc/internal.hpp"
#include "../../newton_schulz_09_amd/csrc/lm_common.hpp"

namespace {

constexpr uintptr_t kWs = uintptr_t{1} << 44;
size_t g_shrink = 0, g_bytes = 0;
long g_launches = 0;

[[noreturn]] void die(const char* what, long long a, long long b) {
    fprintf(stderr, "host check failed: %s (%lld, %lld)\n", what, a, b);
    abort();
}
void in_ws(const void* p, __int128 bytes, const char* what) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (lo < kWs || lo % 256 != 0 || lo - kWs + bytes > g_bytes) die(what, static_cast<long long>(lo - kWs), static_cast<long long>(bytes));
}
void grid(__int128 blocks, const char* what) {
    if (blocks <= 0 || blocks > 0x7fffffff) die(what, static_cast<long long>(blocks), 0);
    ++g_launches;
}

}  // namespace

namespace muon {

int fail_status(int status, const char* msg) {
    if (status == MUON_ERR_HIP) die(msg, status, 0);
    return status;
}

hipError_t launch_attn_doc_tiles(const AttnArgs& a, hipStream_t) {
    in_ws(a.doc_tiles, static_cast<__int128>(a.b) * a.n_tiles * 8, "document ranges");
    grid((static_cast<__int128>(a.b) * a.n_tiles + 3) / 4, "document ranges");
    return hipSuccess;
}
hipError_t launch_attn_fwd(const AttnArgs& a, hipStream_t) {
    grid(static_cast<__int128>((static_cast<int64_t>(a.sq) + 127) / 128) * a.b * a.hq, "forward");
    return hipSuccess;
}
hipError_t launch_attn_split(const AttnArgs& a, hipStream_t) {
    const __int128 rows = static_cast<__int128>(a.b) * a.hq * a.sq, group = static_cast<__int128>(a.grp) * a.sq;
    if (group > 0x7fffff00) die("rows of a key head", static_cast<long long>(group), 0);
    grid((group + 31) / 32 * a.splits * a.b * a.hkv, "split");
    if (a.splits < 1 || a.chunk < 1 || static_cast<int64_t>(a.splits) * a.chunk < a.n_tiles) die("chunks", a.splits, a.chunk);
    if (static_cast<int64_t>(a.splits) * a.chunk > 0x7fffffff) die("last tile", a.splits, a.chunk);
    if (a.splits > 1) {
        in_ws(a.part, rows * a.splits * (a.d + 2) * 4, "parts");
        grid((rows + 3) / 4, "merge");
    }
    return hipSuccess;
}
hipError_t launch_attn_bwd_dq(const AttnArgs& a, hipStream_t) {
    const __int128 rows = static_cast<__int128>(a.b) * a.hq * a.sq;
    if (a.delta_at < rows) die("terms overlap", a.delta_at, static_cast<long long>(rows));
    in_ws(a.stats, (a.delta_at + rows) * 4, "row terms");
    grid(static_cast<__int128>((static_cast<int64_t>(a.sq) + 127) / 128) * a.b * a.hq, "dQ");
    return hipSuccess;
}
hipError_t launch_attn_bwd_dkv(const AttnArgs& a, hipStream_t) {
    grid(static_cast<__int128>((static_cast<int64_t>(a.sk) + 127) / 128) * a.b * a.hkv, "dK and dV");
    return hipSuccess;
}
static void check_qk_args(const QkArgs& a, bool backward) {
    const int64_t runs = a.runs_q + (a.heads[1] + a.chunk - 1) / a.chunk;
    if (a.lanes < 1 || a.lanes > 64 || (a.lanes & (a.lanes - 1))) die("lanes", a.lanes, 0);
    const int v = a.vector ? (a.type == MUON_BF16 ? 8 : 4) : 1, per = a.vector ? 1 : 4;
    if (static_cast<int64_t>(a.lanes) * v * per < a.d / 2) die("lanes hold less than a half", a.lanes, a.d);
    if (a.chunk < 1 || static_cast<int64_t>(a.runs_q) * a.chunk < a.heads[0]) die("runs", a.runs_q, a.chunk);
    if (runs > 65535) die("grid rows", runs, 0);
    if (runs > 0) grid(a.blocks, "norm and rotation");
    if (backward && a.part) in_ws(a.part, static_cast<__int128>(a.blocks) * runs * a.d * 4, "weight gradients");
}
hipError_t launch_qk_norm(const QkArgs& a, hipStream_t) {
    check_qk_args(a, false);
    return hipSuccess;
}
hipError_t launch_qk_norm_bwd(const QkArgs& a, hipStream_t) {
    check_qk_args(a, true);
    return hipSuccess;
}
hipError_t launch_embed(const EmbedArgs&, hipStream_t) {
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_embed_bwd(const EmbedArgs& a, hipStream_t) {
    in_ws(a.perm, static_cast<__int128>(a.n) * 4, "order");
    in_ws(a.ids, static_cast<__int128>(a.n) * 4, "sorted tokens");
    in_ws(a.offset, (static_cast<__int128>(a.vocab) + 1) * 4, "first places");
    if (a.window < 1 || a.window > 32) die("window", a.window, 0);
    in_ws(a.part, (static_cast<__int128>(a.n) + a.window - 1) / a.window * 2 * a.width * 4, "parts of runs");
    grid((a.n + a.window - 1) / a.window + (a.vocab + 31) / 32, "sums");
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
int64_t pick(int64_t lo, int64_t hi) {  // log-uniform
    g_state = g_state * 6364136223846793005ull + 1442695040888963407ull;
    int64_t x = hi;
    for (int i = 0; i < static_cast<int>((g_state >> 33) % 40) && x > lo; ++i) x = x / 2;
    g_state = g_state * 6364136223846793005ull + 1442695040888963407ull;
    x += static_cast<int64_t>((g_state >> 33) % 7);
    return x < lo ? lo : (x > hi ? hi : x);
}

}  // namespace

int main(int argc, char** argv) {
    if (argc > 1) g_shrink = 256;
    for (int it = 0; it < 20000; ++it) {
        muon_attention_args x{};
        x.q = x.k = x.v = x.dout = fake<uint16_t>();
        x.out = x.dq = x.dk = x.dv = fake<uint16_t>();
        x.lse = fake<float>();
        for (int64_t(*s)[3] : {&x.q_strides, &x.k_strides, &x.v_strides, &x.out_strides, &x.dout_strides})
            for (int i = 0; i < 3; ++i) (*s)[i] = 64;
        if (it & 1) x.documents = fake<int32_t>();
        if (it & 2) x.slopes = fake<float>();
        x.batch = pick(1, 1 << 16);
        x.kv_heads = pick(1, 64);
        x.heads = x.kv_heads * pick(1, 64);
        x.sq = pick(1, (int64_t{1} << 29) - 1);
        x.sk = it % 5 == 0 ? x.sq : pick(it % 7 == 0 ? 0 : 1, (int64_t{1} << 29) - 1);
        x.d = 8 * pick(1, 16);
        x.causal = it & 1;
        x.scale = 1.0;
        const size_t f = muon_attention_workspace_size(&x), b = muon_attention_backward_workspace_size(&x);
        if ((f == 0) != (b == 0)) die("one direction is refused", it, 0);
        if (f == 0) continue;
        ok(muon_attention(&x, ws(f), f, nullptr), "attention");
        ok(muon_attention_backward(&x, ws(b), b, nullptr), "attention backward");
    }
    for (int it = 0; it < 20000; ++it) {
        muon_qk_norm_rope_args x{};
        for (int i = 0; i < 2; ++i) {
            x.x[i] = x.dz[i] = fake<char>() + (it % 11 == 0 ? 4 : 0);
            x.out[i] = fake<char>();
            if (it & 1) x.weight[i] = fake<float>();
            if (it & 1) x.dweight[i] = fake<float>();
            x.heads[i] = pick(it % 13 == 0 ? 0 : 1, 32767);
            for (int j = 0; j < 3; ++j) x.x_strides[i][j] = x.dz_strides[i][j] = it % 17 == 0 ? 12 : 64;
        }
        x.table = fake<float>();
        x.limit = 100;
        x.batch = pick(0, (1 << 29) - 1);
        x.s = pick(0, (1 << 29) - 1);
        x.d = 2 * pick(1, 256);
        x.dtype = it & 2 ? MUON_F32 : MUON_BF16;
        x.eps = 1e-6;
        ok(muon_qk_norm_rope(&x, nullptr), "norm and rotation");
        const size_t b = muon_qk_norm_rope_backward_workspace_size(&x);
        ok(muon_qk_norm_rope_backward(&x, ws(b), b, nullptr), "norm and rotation backward");
    }
    for (int it = 0; it < 20000; ++it) {
        const int64_t n = pick(0, 0x7ffffffe), vocab = pick(1, 0x7ffffffe), width = pick(1, 1 << 20);
        const size_t b = muon_embedding_backward_workspace_size(n, vocab, width);
        if (b == 0) die("embedding refused", n, vocab);
        ok(muon_embedding_backward(fake<char>(), it & 1 ? 8 : 4, fake<char>(), MUON_F32, fake<char>(), MUON_BF16, n, vocab, width, 1.0f,
                                   ws(b), b, nullptr),
           "embedding backward");
    }
    printf("host check ok: %ld launches\n", g_launches);
    return 0;
}
