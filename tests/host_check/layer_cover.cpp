// CPU driver of the host code of the feed-forward block (layer_api.hip): prints
// which kernels the entry points launch for sizes given as arguments, a line each:
// tokens width hidden, product, tile, and how K is split.  Nothing is launched or
// dereferenced.  Built and read by tests/test_layer_cover.py.
#include <stdio.h>
#include <stdlib.h>

#include "../../include/muon_lm.h"
#include "../../newton_schulz_09_amd/csrc/internal.hpp"
#include "../../newton_schulz_09_amd/csrc/layer_common.hpp"

static muon_feed_forward_args g_args;

namespace muon {

int fail_status(int status, const char* msg) {
    if (status != MUON_OK) {
        fprintf(stderr, "%s\n", msg);
        exit(1);
    }
    return status;
}
hipError_t launch_dropout(const DropArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_resid_norm(const ResidArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_resid_norm_bwd(const ResidArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_ffn_few(const FfnFew&, hipStream_t) { return hipSuccess; }
hipError_t launch_ffn(FfnKind kind, FfnTile tile, const FfnGemm& g, hipStream_t) {
    static const char* const kinds[] = {"gated", "plain", "hidden", "input", "weights"};
    printf("%lld %lld %lld %s %d %s\n", (long long)g_args.tokens, (long long)g_args.width, (long long)g_args.hidden, kinds[kind],
           static_cast<int>(tile), g.full == g.tiles ? "whole" : g.full == 0 ? "split" : "mixed");
    return hipSuccess;
}

}  // namespace muon

int main(int argc, char** argv) {
    uint16_t* const fake = reinterpret_cast<uint16_t*>(uintptr_t{1} << 40);
    for (int i = 1; i + 2 < argc; i += 3) {
        muon_feed_forward_args& x = g_args;
        x = muon_feed_forward_args{};
        x.x = x.w_gate = x.w_up = x.w_down = x.dout = fake;
        x.out = x.dx = x.kept = fake;
        x.dw_gate = x.dw_up = x.dw_down = fake;
        x.tokens = atoll(argv[i]);
        x.width = x.x_stride = x.dout_stride = x.w_stride = atoll(argv[i + 1]);
        x.hidden = x.w_down_stride = atoll(argv[i + 2]);
        void* const ws = reinterpret_cast<void*>(uintptr_t{1} << 44);
        if (muon_feed_forward(&x, ws, muon_feed_forward_workspace_size(&x), nullptr) != MUON_OK ||
            muon_feed_forward_backward(&x, ws, muon_feed_forward_backward_workspace_size(&x), nullptr) != MUON_OK)
            return 1;
    }
    return 0;
}
