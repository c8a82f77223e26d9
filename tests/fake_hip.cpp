// fake_hip.cpp -- the library's C calls on the host alone: this program defines the
// HIP runtime functions that libdgw_gemm.so calls, so its own definitions are the
// ones the library binds to.  Launches, allocations and frees are recorded with
// their thread and stream and nothing runs.  One scenario per run, named by argv[1];
// exit status 0 and "ok" where it holds.
#include <atomic>
#include <chrono>
#include <condition_variable>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <mutex>
#include <new>
#include <string>
#include <thread>
#include <vector>

#include "gemm_loss.h"

struct Dim {
    uint32_t x, y, z;
};

thread_local bool no_memory = false;   // operator new of this thread fails

void *operator new(size_t n) {
    void *p = no_memory ? nullptr : std::malloc(n);
    if (!p) throw std::bad_alloc();
    return p;
}
void operator delete(void *p) noexcept { std::free(p); }
void operator delete(void *p, size_t) noexcept { std::free(p); }

namespace {

struct Event {
    std::string what;   // "launch <kernel>", "malloc", "free"
    std::thread::id thread;
    void *stream;
};
std::mutex mu;
std::condition_variable changed;
std::vector<Event> events;
// filled by the library's constructors, which run before this program's
std::map<const void *, std::string> &kernels() {
    static std::map<const void *, std::string> names;
    return names;
}
std::atomic<uintptr_t> next_address{uintptr_t(1) << 32};
void (*on_launch)() = nullptr;   // called in the launching thread, after the record

void record(const std::string &what, void *stream = nullptr) {
    std::lock_guard<std::mutex> lock(mu);
    events.push_back({what, std::this_thread::get_id(), stream});
    changed.notify_all();
}
struct Config {
    Dim grid, block;
    size_t shared;
    void *stream;
};
thread_local Config config;

}  // namespace

extern "C" {
void **__hipRegisterFatBinary(const void *) {
    static void *handle;
    return &handle;
}
void __hipUnregisterFatBinary(void **) {}
void __hipRegisterFunction(void **, const void *host, char *, const char *name, unsigned, void *, void *, void *, void *, int *) {
    kernels()[host] = name;
}
void __hipRegisterVar(void **, void *, char *, char *, int, size_t, int, int) {}
int __hipPushCallConfiguration(Dim grid, Dim block, size_t shared, void *stream) {
    config = {grid, block, shared, stream};
    return 0;
}
int __hipPopCallConfiguration(Dim *grid, Dim *block, size_t *shared, void **stream) {
    *grid = config.grid, *block = config.block, *shared = config.shared, *stream = config.stream;
    return 0;
}
int hipLaunchKernel(const void *host, Dim, Dim, void **, size_t, void *stream) {
    record("launch " + kernels()[host], stream);
    if (on_launch) on_launch();
    return 0;
}
int hipGetLastError() { return 0; }
const char *hipGetErrorString(int) { return "error"; }
int hipGetDevice(int *d) { return *d = 0, 0; }
int hipSetDevice(int) { return 0; }
int hipDeviceGetAttribute(int *v, int, int) { return *v = 256, 0; }
int hipDeviceSynchronize() { return 0; }
int hipStreamSynchronize(void *) { return 0; }
int hipStreamIsCapturing(void *, int *s) { return *s = 0, 0; }
int hipMalloc(void **p, size_t n) {
    *p = reinterpret_cast<void *>(next_address.fetch_add((n + 4095) / 4096 * 4096));
    record("malloc");
    return 0;
}
int hipFree(void *) {
    record("free");
    return 0;
}
int hipMemset(void *, int, size_t) { return 0; }
int hipMemcpy(void *dst, const void *, size_t n, int) {
    std::memset(dst, 0, n < 4 ? n : 4);
    return 0;
}
int hipGetSymbolAddress(void **p, const void *) { return *p = reinterpret_cast<void *>(uintptr_t(1) << 31), 0; }
int hipOccupancyMaxActiveBlocksPerMultiprocessor(int *n, const void *, int, size_t) { return *n = 2, 0; }
}

namespace {

constexpr uintptr_t MB = 1 << 20;
template <class T = void>
T *at(int megabyte) {
    return reinterpret_cast<T *>(megabyte * MB);   // addresses that nothing follows
}

// A backward call of several launches: distillation in fp16, dx in slices.
gemm_loss_args_t backward_args() {
    gemm_loss_args_t a;
    std::memset(&a, 0, sizeof a);
    a.T = 16, a.V = 4096, a.H = 64;
    a.layout = GEMM_B_NK | GEMM_FP16;
    a.kind = GEMM_LOSS_DISTILL;
    a.entries = 4, a.temperature = 1.0f;
    a.x = at(1), a.w = at(2);
    a.teacher_index = at<int64_t>(10), a.teacher_logits = at(11);
    a.loss = at<float>(12), a.lse = at<float>(13), a.grad = at<float>(14);
    a.dx = at(15), a.dw = at(16);
    return a;
}

#define REQUIRE(c)                                                                     \
    do {                                                                               \
        if (!(c)) {                                                                    \
            std::printf("line %d: " #c " does not hold (%s)\n", __LINE__, gemm_last_error()); \
            std::exit(1);                                                              \
        }                                                                              \
    } while (0)

// Runs `first` on this thread and, once its first kernel is launched, `second` on
// another one; every launch of `first` leaves `second` 50 ms to get ahead.  Returns
// whether any event of the second thread lies between the first's first and last
// launches.
template <class F, class G>
bool interleaves(F &&first, G &&second) {
    static std::thread::id one;
    static std::atomic<bool> started, ended;
    one = std::this_thread::get_id();
    started = ended = false;
    events.clear();
    on_launch = [] {
        if (std::this_thread::get_id() != one || ended) return;
        std::unique_lock<std::mutex> lock(mu);
        const size_t n = events.size();
        started = true;
        changed.notify_all();
        changed.wait_for(lock, std::chrono::milliseconds(50), [&] { return events.size() > n; });
    };
    std::thread other([&] {
        std::unique_lock<std::mutex> lock(mu);
        changed.wait(lock, [] { return started.load(); });
        lock.unlock();
        second();
    });
    first();
    ended = true;
    other.join();
    on_launch = nullptr;
    size_t from = events.size(), to = 0, own = 0;
    for (size_t i = 0; i < events.size(); ++i)
        if (events[i].thread == one && events[i].what.rfind("launch", 0) == 0) {
            if (from > i) from = i;
            to = i;
            ++own;
        }
    REQUIRE(own >= 3 && events.size() > own);
    return to - from + 1 != own;
}

int release() {
    // gemm_release() frees the library workspace before or after a call, not within it
    gemm_loss_args_t a = backward_args();
    REQUIRE(gemm_loss_backward(&a) == GEMM_OK);   // sizes the workspace
    REQUIRE(!interleaves([&] { REQUIRE(gemm_loss_backward(&a) == GEMM_OK); }, [] { gemm_release(); }));
    REQUIRE(events.back().what == "free");
    return 0;
}

int two_threads() {
    // calls of two threads on one stream and the library workspace are enqueued one after the other
    gemm_loss_args_t a = backward_args(), b = backward_args();
    b.kind = GEMM_LOSS_XENT;
    b.target = at<int64_t>(17);
    REQUIRE(gemm_loss_backward(&a) == GEMM_OK);
    REQUIRE(!interleaves([&] { REQUIRE(gemm_loss_backward(&a) == GEMM_OK); }, [&] { REQUIRE(gemm_loss_forward(&b) == GEMM_OK); }));
    REQUIRE(!interleaves([&] { REQUIRE(gemm_loss_backward(&a) == GEMM_OK); }, [&] { REQUIRE(gemm_loss_backward(&b) == GEMM_OK); }));
    auto product = [] {
        REQUIRE(gemm(at(1), at(2), at<float>(40), 128, 128, 4096, GEMM_B_NK, GEMM_SPLITK | GEMM_TWO_PASS, 8) == GEMM_OK);
    };
    product();
    REQUIRE(!interleaves([&] { REQUIRE(gemm_loss_backward(&a) == GEMM_OK); }, product));
    // a refused call leaves the library usable
    gemm_loss_args_t bad = backward_args();
    bad.temperature = -1.0f;
    REQUIRE(gemm_loss_backward(&bad) == GEMM_ERR_INVALID && gemm_loss_backward(&a) == GEMM_OK);
    return 0;
}

// Whether `call` launched something, all of it on `stream`.
template <class F>
bool runs_on(void *stream, F &&call) {
    events.clear();
    call();
    bool any = false;
    for (const Event &e : events)
        if (e.what.rfind("launch", 0) == 0) {
            any = true;
            if (e.stream != stream) return false;
        }
    return any;
}

int streams() {
    // NULL: the thread's stream; GEMM_NULL_STREAM: HIP's, whatever the thread's is
    void *const own = at(100), *const given = at(101);
    gemm_loss_args_t a = backward_args(), none = backward_args();
    none.T = 0;   // dw is cleared
    gemm_args_t g;
    std::memset(&g, 0, sizeof g);
    g.A = at(1), g.B = at(2), g.C = at<float>(40);
    g.M = g.N = g.K = 256;
    gemm_args_t common;
    std::memset(&common, 0, sizeof common);
    common.K = 256;
    const gemm_group_t group = {at(1), at(2), at<float>(40), 256, 256};
    for (void *thread : {static_cast<void *>(nullptr), own}) {
        REQUIRE(gemm_set_stream(thread) == GEMM_OK);
        struct {
            void *argument, *want;
        } const cases[] = {{nullptr, thread}, {given, given}, {GEMM_NULL_STREAM, nullptr}};
        for (const auto &c : cases) {
            a.stream = none.stream = g.stream = common.stream = c.argument;
            REQUIRE(runs_on(c.want, [&] { REQUIRE(gemm_loss_forward(&a) == GEMM_OK); }));
            REQUIRE(runs_on(c.want, [&] { REQUIRE(gemm_loss_backward(&a) == GEMM_OK); }));
            REQUIRE(runs_on(c.want, [&] { REQUIRE(gemm_loss_backward(&none) == GEMM_OK); }));
            REQUIRE(runs_on(c.want, [&] { REQUIRE(gemm_ex(&g) == GEMM_OK); }));
            REQUIRE(runs_on(c.want, [&] { REQUIRE(gemm_grouped(&common, &group, 1) == GEMM_OK); }));
        }
        REQUIRE(runs_on(thread, [] { REQUIRE(gemm(at(1), at(2), at<float>(40), 256, 256, 256, 0, 0, 0) == GEMM_OK); }));
    }
    REQUIRE(gemm_set_stream(GEMM_NULL_STREAM) == GEMM_OK);
    a.stream = nullptr;
    REQUIRE(runs_on(nullptr, [&] { REQUIRE(gemm_loss_forward(&a) == GEMM_OK); }));
    return 0;
}

int no_exceptions() {
    // without host memory for its message a refused call still returns, to C callers too
    gemm_loss_args_t a = backward_args();
    gemm_loss_plan_t plan;
    a.temperature = -1.0f;
    a.H = 36;
    int rc[3] = {1, 1, 1};
    try {
        no_memory = true;
        rc[0] = gemm_loss_forward(&a);
        rc[1] = gemm_loss_backward(&a);
        rc[2] = gemm_loss_plan(&a, 1, 256, &plan);
        no_memory = false;
    } catch (...) {
        no_memory = false;
        std::puts("an exception left a C call");
        return 1;
    }
    for (int r : rc) REQUIRE(r < 0);
    REQUIRE(std::strlen(gemm_last_error()) > 0);
    a = backward_args();
    REQUIRE(gemm_loss_forward(&a) == GEMM_OK && gemm_loss_backward(&a) == GEMM_OK);
    return 0;
}

}  // namespace

int main(int argc, char **argv) {
    const std::map<std::string, int (*)()> scenarios = {{"release", release}, {"two_threads", two_threads}, {"streams", streams}, {"no_exceptions", no_exceptions}};
    const auto s = scenarios.find(argc > 1 ? argv[1] : "");
    if (s == scenarios.end()) return 2;
    const int rc = s->second();
    if (rc == 0) std::puts("ok");
    return rc;
}
