// fake_hip_layers.cpp -- the C calls of the feed-forward block and the adapters on the
// host alone, by the HIP runtime of fake_hip.cpp.  One scenario per run.
#define main fake_hip_main
#include "fake_hip.cpp"
#undef main

#include "gemm_ffn.h"
#include "gemm_lora.h"

namespace {

gemm_ffn_args_t ffn_args(int64_t T) {
    gemm_ffn_args_t a;
    std::memset(&a, 0, sizeof a);
    a.T = T, a.H = 64, a.F = 4096;
    a.layout = GEMM_B_NK | GEMM_BF16;
    a.x = at(1), a.w_gate = at(2), a.w_up = at(3), a.w_down = at(4);
    a.gate = at(10), a.up = at(20), a.y = at(30);
    a.dy = at(31), a.dx = at(32), a.dw_gate = at(33), a.dw_up = at(34), a.dw_down = at(35);
    return a;
}
gemm_lora_args_t lora_args(int64_t T) {
    gemm_lora_args_t a;
    std::memset(&a, 0, sizeof a);
    a.T = T, a.H = 4096, a.N = 128, a.R = 8, a.adapters = 3;
    a.layout = GEMM_B_NK | GEMM_BF16;
    a.x = at(1), a.w = at(12), a.a = at(14), a.b = at(15);
    a.adapter = at<int64_t>(16), a.scale = at<float>(17), a.y = at(18);
    a.dy = at(20), a.dx = at(30), a.da = at(40), a.db = at(41);
    return a;
}
// f(call, name) for every call at few, some and many rows
template <class F>
void every_call(F &&f) {
    for (int64_t T : {1, 16, 100, 1000}) {
        gemm_ffn_args_t a = ffn_args(T);
        gemm_lora_args_t b = lora_args(T);
        f([&](void *s) { a.stream = s; return gemm_ffn_forward(&a); });
        f([&](void *s) { a.stream = s; return gemm_ffn_backward(&a); });
        f([&](void *s) { b.stream = s; return gemm_lora_forward(&b); });
        f([&](void *s) { b.stream = s; return gemm_lora_backward(&b); });
    }
}

int layers_stream() {
    void *const own = at(100), *const given = at(101);
    for (void *thread : {static_cast<void *>(nullptr), own}) {
        REQUIRE(gemm_set_stream(thread) == GEMM_OK);
        every_call([&](auto &&call) {
            REQUIRE(runs_on(thread, [&] { REQUIRE(call(nullptr) == GEMM_OK); }));
            REQUIRE(runs_on(given, [&] { REQUIRE(call(given) == GEMM_OK); }));
            REQUIRE(runs_on(nullptr, [&] { REQUIRE(call(GEMM_NULL_STREAM) == GEMM_OK); }));
        });
        gemm_ffn_args_t a = ffn_args(0);   // the gradients are cleared
        gemm_lora_args_t b = lora_args(0);
        REQUIRE(runs_on(thread, [&] { REQUIRE(gemm_ffn_backward(&a) == GEMM_OK); }));
        REQUIRE(runs_on(thread, [&] { REQUIRE(gemm_lora_backward(&b) == GEMM_OK); }));
    }
    return 0;
}

int layers_workspace() {
    // calls of two threads on the library workspace are enqueued one after the other, and
    // gemm_release() waits for them
    gemm_ffn_args_t a = ffn_args(16);
    gemm_lora_args_t b = lora_args(1000);
    REQUIRE(gemm_ffn_backward(&a) == GEMM_OK && gemm_lora_backward(&b) == GEMM_OK);
    auto ffn = [&] { REQUIRE(gemm_ffn_backward(&a) == GEMM_OK); };
    auto lora = [&] { REQUIRE(gemm_lora_backward(&b) == GEMM_OK); };
    REQUIRE(!interleaves(ffn, lora));
    REQUIRE(!interleaves(lora, ffn));
    REQUIRE(!interleaves(ffn, [] { gemm_release(); }));
    return 0;
}

int layers_no_exceptions() {
    gemm_ffn_args_t a = ffn_args(16);
    gemm_lora_args_t b = lora_args(16);
    gemm_ffn_plan_t pa;
    gemm_lora_plan_t pb;
    a.H = 36, b.H = 36;
    int rc[6] = {1, 1, 1, 1, 1, 1};
    try {
        no_memory = true;
        rc[0] = gemm_ffn_forward(&a);
        rc[1] = gemm_ffn_backward(&a);
        rc[2] = gemm_ffn_plan(&a, 1, 256, &pa);
        rc[3] = gemm_lora_forward(&b);
        rc[4] = gemm_lora_backward(&b);
        rc[5] = gemm_lora_plan(&b, 1, 256, &pb);
        no_memory = false;
    } catch (...) {
        no_memory = false;
        std::puts("an exception left a C call");
        return 1;
    }
    for (int r : rc) REQUIRE(r < 0);
    REQUIRE(std::strlen(gemm_last_error()) > 0);
    every_call([&](auto &&call) { REQUIRE(call(nullptr) == GEMM_OK); });
    return 0;
}

}  // namespace

int main(int argc, char **argv) {
    const std::map<std::string, int (*)()> scenarios = {{"stream", layers_stream}, {"workspace", layers_workspace}, {"no_exceptions", layers_no_exceptions}};
    const auto s = scenarios.find(argc > 1 ? argv[1] : "");
    if (s == scenarios.end()) return 2;
    const int rc = s->second();
    if (rc == 0) std::puts("ok");
    return rc;
}
