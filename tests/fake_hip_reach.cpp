// fake_hip_reach.cpp -- which kernels of the feed-forward block and the adapters no call
// reaches: every call over a wide range of sizes, by the HIP runtime of fake_hip.cpp.
// Prints the names of the kernels that were never launched.
#define main fake_hip_main
#include "fake_hip.cpp"
#undef main

#include <set>

#include "gemm_ffn.h"
#include "gemm_lora.h"

namespace {

template <class T = void>
T *far(int i) {
    return reinterpret_cast<T *>(uintptr_t(i) << 42);   // apart whatever the sizes, and followed by nothing
}
std::set<std::string> launched;
int refused = 0;

void take(int rc) {
    refused += rc != GEMM_OK;
    for (const Event &e : events)
        if (e.what.rfind("launch ", 0) == 0) launched.insert(e.what.substr(7));
    events.clear();
}

void ffn(int64_t T, int64_t H, int64_t F, uint32_t layout) {
    gemm_ffn_args_t a;
    std::memset(&a, 0, sizeof a);
    a.T = T, a.H = H, a.F = F, a.layout = layout, a.num_cus = 256;
    a.x = far(1), a.w_gate = far(2), a.w_up = far(3), a.w_down = far(4);
    a.gate = far(5), a.up = far(6), a.y = far(7), a.dy = far(8);
    a.workspace = far(9), a.workspace_bytes = size_t(1) << 42;
    take(gemm_ffn_forward(&a));
    a.dx = far(10);
    for (uint32_t type : {GEMM_FFN_DW_SAME, GEMM_FFN_DW_FP32, GEMM_FFN_DW_FP32_ADD})
        for (int64_t more : {0, 8}) {
            a.ldw_gate = more ? ((layout & 0xF) == GEMM_B_NK ? H : F) + more : 0;
            a.dw_type = type, a.dw_gate = far(11), a.dw_up = far(12), a.dw_down = far(13);
            take(gemm_ffn_backward(&a));
        }
}

void lora(int64_t T, int64_t H, int64_t N, int32_t L, int32_t R, uint32_t layout) {
    gemm_lora_args_t a;
    std::memset(&a, 0, sizeof a);
    a.T = T, a.H = H, a.N = N, a.adapters = L, a.R = R, a.layout = layout, a.num_cus = 256;
    a.x = far(1), a.w = far(2), a.a = far(3), a.b = far(4), a.adapter = far<int64_t>(5), a.y = far(7), a.dy = far(8);
    a.workspace = far(9), a.workspace_bytes = size_t(1) << 42;
    take(gemm_lora_forward(&a));
    for (int what = 1; what < 4; ++what) {   // dx, da and db, both
        a.dx = what & 1 ? far(10) : nullptr;
        a.da = what & 2 ? far(11) : nullptr;
        a.db = what & 2 ? far(12) : nullptr;
        take(gemm_lora_backward(&a));
    }
}

}  // namespace

int main() {
    const int64_t rows[] = {1, 2, 4, 20, 50, 100, 200, 300, 1000, 5000}, sizes[] = {64, 1032, 4104, 30000};
    for (uint32_t layout : {GEMM_B_NK | GEMM_BF16, GEMM_B_NK | GEMM_FP16, GEMM_B_KN | GEMM_BF16, GEMM_B_KN | GEMM_FP16})
        for (int64_t T : rows)
            for (int64_t H : sizes)
                for (int64_t F : sizes) {
                    ffn(T, H, F, layout);
                    for (int32_t R : {16, 40, 72, 320})
                        for (int32_t L : {1, 6, 64}) lora(T, H, F, L, R, layout);
                }
    if (refused) {
        std::printf("%d calls refused: %s\n", refused, gemm_last_error());
        return 1;
    }
    for (const auto &k : kernels())
        for (const char *of : {"ffn_", "lora_", "loss_outers"})
            if (k.second.find(of) != std::string::npos && !launched.count(k.second)) std::puts(k.second.c_str());
    return 0;
}
