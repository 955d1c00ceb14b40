// The entry points' host code against a CUDA runtime that fails on demand: a call that fails returns GQ_ERR_CUDA, gives
// back what it had allocated, and leaves no error behind for the thread's next launch to report as its own.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <set>
#include <vector>

#include <cuda_runtime.h>

#include "gq.h"
#include "gq_adamw.h"
#include "gq_internal.h"

// ---- the runtime: `fail_at` counts down calls that can fail; the last error stays until it is taken ----
static int calls = 0, fail_at = -1;
static cudaError_t last = cudaSuccess;
static std::set<void *> blocks;

static cudaError_t done(cudaError_t bad)
{
    if (calls++ != fail_at) return cudaSuccess;
    return last = bad;
}

extern "C" {
cudaError_t cudaGetLastError()
{
    const cudaError_t e = last;
    last = cudaSuccess;
    return e;
}
cudaError_t cudaGetDevice(int *d)
{
    *d = 0;
    return done(cudaErrorInvalidDevice);
}
cudaError_t cudaMalloc(void **p, size_t n)
{
    const cudaError_t e = done(cudaErrorMemoryAllocation);
    if (e == cudaSuccess) blocks.insert(*p = std::malloc(n ? n : 1));
    return e;
}
cudaError_t cudaFree(void *p)
{
    if (p && !blocks.erase(p)) return last = cudaErrorInvalidValue;
    std::free(p);
    return done(cudaErrorUnknown);
}
cudaError_t cudaMemset(void *p, int v, size_t n)
{
    std::memset(p, v, n);
    return done(cudaErrorInvalidValue);
}
cudaError_t cudaMemsetAsync(void *p, int v, size_t n, cudaStream_t)
{
    std::memset(p, v, n);
    return done(cudaErrorInvalidValue);
}
cudaError_t cudaMemcpy(void *to, const void *from, size_t n, cudaMemcpyKind)
{
    std::memcpy(to, from, n);
    return done(cudaErrorInvalidValue);
}
cudaError_t cudaMemcpyAsync(void *to, const void *from, size_t n, cudaMemcpyKind, cudaStream_t)
{
    std::memcpy(to, from, n);
    return done(cudaErrorInvalidValue);
}
cudaError_t cudaStreamSynchronize(cudaStream_t) { return done(cudaErrorUnknown); }
}

// ---- the kernels' launches, which fail on demand too ----
namespace gq {
cudaError_t launch_adamw(const AdamArgs &, const AdamStep &, cudaStream_t) { return done(cudaErrorInvalidConfiguration); }
cudaError_t launch_adamw_moments(const AdamArgs &, int, void *, void *, cudaStream_t) { return done(cudaErrorInvalidConfiguration); }
cudaError_t launch_adamw_norm(const AdamArgs &, double, double *, float *, cudaStream_t) { return done(cudaErrorInvalidConfiguration); }
int64_t err_scratch_doubles(int64_t nb) { return 3 * nb; }
cudaError_t launch_wait_selftest(unsigned int *, unsigned long long, cudaStream_t) { return done(cudaErrorInvalidConfiguration); }
cudaError_t launch_warp_err(const KParams &, double *, cudaStream_t) { return done(cudaErrorInvalidConfiguration); }
cudaError_t launch_cta_err(const KParams &, double *, cudaStream_t) { return done(cudaErrorInvalidConfiguration); }
cudaError_t launch_err_reduce(const double *, int64_t, double *, double *, cudaStream_t, const unsigned int *)
{
    return done(cudaErrorInvalidConfiguration);
}
}  // namespace gq

static int wrong = 0;
static void expect(bool ok, const char *what, int at)
{
    if (ok) return;
    ++wrong;
    std::printf("%s, failing call %d\n", what, at);
}

// Runs `body` (which returns a status) with each of the calls that it makes failing in turn, and once with none failing.
template <typename F>
static void each_failure(const char *what, F body)
{
    fail_at = -1;
    calls = 0;
    expect(body() == GQ_OK && last == cudaSuccess, what, -1);
    const int n = calls;
    expect(n > 0, what, -2);
    for (int i = 0; i < n; ++i) {
        const size_t held = blocks.size();
        calls = 0;
        fail_at = i;
        const gq_status_t st = body();
        expect(st == GQ_ERR_CUDA, what, i);
        expect(last == cudaSuccess, "left an error", i);
        expect(blocks.size() == held, "left memory", i);
        last = cudaSuccess;
        fail_at = -1;
    }
}

int main()
{
    std::vector<float> mem(5 * 1200);
    const gq_adamw_config_t cfg = {GQ_FLOAT32, GQ_FLOAT32, 32, 1};
    const gq_adamw_tensor_t t = {&mem[0], &mem[1200], nullptr, &mem[2400], &mem[3600], 1000, 0.0f, 1.0f};
    float *const out = &mem[4800];
    alignas(16) static float spare[1000];
    // an optimizer made and destroyed: a failing cudaFree has freed its block here
    each_failure("gq_adamw_create", [&] {
        gq_adamw_t opt = nullptr;
        const gq_status_t st = gq_adamw_create(&cfg, &t, 1, &opt);
        if (st != GQ_OK) return opt ? GQ_OK : st;
        return gq_adamw_destroy(opt);
    });
    gq_adamw_t opt = nullptr;
    expect(gq_adamw_create(&cfg, &t, 1, &opt) == GQ_OK, "create", -1);
    each_failure("gq_adamw_norm", [&] { return gq_adamw_norm(opt, 1.0, out, nullptr); });
    each_failure("gq_adamw_step", [&] { return gq_adamw_step(opt, 1e-3, 0.9, 0.999, 1e-8, 1, nullptr, nullptr, nullptr); });
    each_failure("gq_adamw_moments", [&] { return gq_adamw_moments(opt, GQ_FLOAT32, nullptr, spare, nullptr); });
    expect(gq_adamw_destroy(opt) == GQ_OK, "destroy", -1);

    gq_config_t plan_cfg = {};
    plan_cfg.scheme = GQ_ORQ;
    plan_cfg.levels = 5;
    plan_cfg.bucket = 512;
    plan_cfg.workers = 1;
    plan_cfg.n = 2048;
    each_failure("gq_plan_create", [&] {
        gq_plan_t plan = nullptr;
        const gq_status_t st = gq_plan_create(&plan_cfg, &plan);
        if (st != GQ_OK) return plan ? GQ_OK : st;
        return gq_plan_destroy(plan);
    });
    gq_plan_t plan = nullptr;
    expect(gq_plan_create(&plan_cfg, &plan) == GQ_OK, "create", -1);
    double errs[3];
    each_failure("gq_plan_status", [&] { return gq_plan_status(plan, nullptr); });
    each_failure("gq_selftest_bounded_wait", [&] { return gq_selftest_bounded_wait(plan, 1000000, nullptr); });
    each_failure("gq_quant_error", [&] { return gq_quant_error(plan, 0, 0, &mem[0], nullptr, errs, nullptr); });
    expect(gq_plan_destroy(plan) == GQ_OK, "destroy", -1);

    plan_cfg.scheme = GQ_TERNGRAD_LAYER;
    plan_cfg.levels = 3;
    expect(gq_plan_create(&plan_cfg, &plan) == GQ_OK, "create", -1);
    const int64_t offsets[3] = {0, 1000, 2048};
    // it gives its old arrays back first, so that only the calls that can return an error count
    expect(gq_plan_set_segments(plan, offsets, 2) == GQ_OK, "segments", -1);
    expect(gq_plan_destroy(plan) == GQ_OK, "destroy", -1);
    for (int i = 0; i < 4; ++i) {
        expect(gq_plan_create(&plan_cfg, &plan) == GQ_OK, "create", -1);
        calls = 0;
        fail_at = i;
        expect(gq_plan_set_segments(plan, offsets, 2) == GQ_ERR_CUDA, "gq_plan_set_segments", i);
        expect(last == cudaSuccess, "left an error", i);
        fail_at = -1;
        last = cudaSuccess;
        expect(gq_plan_destroy(plan) == GQ_OK, "destroy", -1);
    }
    expect(blocks.empty(), "left memory", -1);
    std::printf(wrong ? "%d wrong\n" : "ok\n", wrong);
    return wrong != 0;
}
