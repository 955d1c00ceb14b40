// gq_adamw_api.cu -- host side of the AdamW entry points (include/gq.h): argument checks, and the optimizer's
// table of tensors on the device.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <memory>
#include <vector>

#include "gq_adamw.h"
#include "gq_check.h"

namespace gq {
struct Span {
    uintptr_t from, to;
    bool written;
};
}  // namespace gq

struct gq_adamw {
    gq::AdamArgs a;
    std::vector<gq::Span> all, written;  // the tensors' memory, and what a step writes of it: apart, by address
    void *memory;   // device: the table of chunks, the norm's partial sums
    double *parts;
    int64_t total;  // elements
    int device;
};

namespace {

using namespace gq;

constexpr int64_t kMaxElements = int64_t(1) << 40;

gq_status_t check_device(const gq_adamw &o)
{
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return cuda_failed();
    return dev == o.device ? GQ_OK : GQ_ERR_INVALID;
}

// Whether anything that a step writes overlaps something else that it reads or writes.
bool any_shared(std::vector<Span> &s)
{
    std::sort(s.begin(), s.end(), [](const Span &a, const Span &b) { return a.from < b.from; });
    uintptr_t read = 0, written = 0;  // ends of what came before
    for (const Span &x : s) {
        if (x.from < written || (x.written && x.from < read)) return true;
        uintptr_t &end = x.written ? written : read;
        if (x.to > end) end = x.to;
    }
    return false;
}

// The union of spans sorted by address (of the written ones among them), as spans that do not touch.
std::vector<Span> merged(const std::vector<Span> &s, bool written)
{
    std::vector<Span> out;
    for (const Span &x : s) {
        if (written && !x.written) continue;
        if (!out.empty() && x.from <= out.back().to) out.back().to = std::max(out.back().to, x.to);
        else out.push_back(x);
    }
    return out;
}

// Whether `bytes` from p share a byte with one of them.
bool meets(const std::vector<Span> &s, const void *p, size_t bytes)
{
    if (!p || !bytes) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    // the first that ends behind p
    auto x = std::upper_bound(s.begin(), s.end(), a, [](uintptr_t at, const Span &b) { return at < b.to; });
    return x != s.end() && x->from < a + bytes;
}

bool factor_ok(float x) { return x >= 0.0f && x <= 3.0e38f; }

gq_status_t check_tensors(const gq_adamw_config_t &c, const gq_adamw_tensor_t *t, int count, std::vector<Span> &spans)
{
    const uintptr_t ps = (uintptr_t)elem_size(c.param_dtype), gs = (uintptr_t)elem_size(c.grad_dtype);
    const bool eight = c.state_bits == 8;
    spans.reserve((size_t)count * 5);
    int64_t total = 0;
    int masters = 0, filled = 0;
    for (int i = 0; i < count; ++i) {
        const gq_adamw_tensor_t &x = t[i];
        if (x.n < 0 || x.n >= kMaxElements || !factor_ok(x.weight_decay) || !factor_ok(x.lr_scale)) return GQ_ERR_INVALID;
        if (x.n == 0) continue;
        total += x.n;
        if (total >= kMaxElements) return GQ_ERR_INVALID;
        const uintptr_t state = eight ? 16 : 4;
        if (!x.param || !x.grad || !x.m || !x.v || !aligned(x.param, ps) || !aligned(x.grad, gs) || !aligned(x.master, 4) ||
            !aligned(x.m, state) || !aligned(x.v, state))
            return GQ_ERR_INVALID;
        ++filled;
        masters += x.master != nullptr;
        const uintptr_t n = (uintptr_t)x.n, sb = eight ? (uintptr_t)adam_bytes(x.n) : 4 * n;
        auto add = [&](const void *p, uintptr_t bytes, bool written) {
            const uintptr_t a = reinterpret_cast<uintptr_t>(p);
            spans.push_back(Span{a, a + bytes, written});
        };
        add(x.param, n * ps, true);
        add(x.grad, n * gs, false);
        if (x.master) add(x.master, n * 4, true);
        add(x.m, sb, true);
        add(x.v, sb, true);
    }
    if (masters && (masters != filled || c.param_dtype == GQ_FLOAT32)) return GQ_ERR_INVALID;
    return any_shared(spans) ? GQ_ERR_INVALID : GQ_OK;
}

// Elements before the tensor's first to where all its arrays lie on 16 bytes, below 8; -1: there is no such place.
int head_of(const gq_adamw_tensor_t &x, uintptr_t ps, uintptr_t gs, bool eight)
{
    for (uintptr_t h = 0; h < (eight ? 1 : 8); ++h) {
        auto on16 = [h](const void *p, uintptr_t size) { return !p || ((reinterpret_cast<uintptr_t>(p) - h * size) & 15) == 0; };
        if (on16(x.param, ps) && on16(x.grad, gs) && on16(x.master, 4) && on16(x.m, 4) && on16(x.v, 4)) return (int)h;
    }
    return -1;
}

gq_status_t create(const gq_adamw_config_t &c, const gq_adamw_tensor_t *list, int count, gq_adamw_t *out)
{
    std::vector<Span> spans;
    const gq_status_t st = check_tensors(c, list, count, spans);
    if (st != GQ_OK) return st;
    std::vector<AdamChunk> table;
    int64_t total = 0, chunks = 0, aligned_chunks = 0;
    for (int i = 0; i < count; ++i) chunks += (list[i].n + 7 + kAdamChunk - 1) / kAdamChunk;
    if (chunks > (int64_t(1) << 31) - 1) return GQ_ERR_UNSUPPORTED;
    table.reserve((size_t)chunks);
    bool master = false;
    const int64_t ps = elem_size(c.param_dtype), gs = elem_size(c.grad_dtype), ss = c.state_bits == 8 ? 1 : 4;
    for (int pass = 0; pass < 2; ++pass) {  // tensors whose arrays can be read by 16 bytes, then the others
        total = 0;
        for (int i = 0; i < count; ++i) {
            const gq_adamw_tensor_t &x = list[i];
            const int h = head_of(x, (uintptr_t)ps, (uintptr_t)gs, ss == 1), head = h < 0 ? 0 : h;
            const int64_t end = x.n ? x.n + head : 0;
            for (int64_t at = 0; at < end && (h >= 0) == (pass == 0); at += kAdamChunk) {
                auto plus = [at, head](const void *p, int64_t size) {  // `head` elements back may be no place of the array
                    return reinterpret_cast<void *>(reinterpret_cast<uintptr_t>(p) + (uintptr_t)((at - head) * size));
                };
                AdamChunk t = {};
                t.param = plus(x.param, ps);
                t.grad = plus(x.grad, gs);
                t.master = x.master ? static_cast<float *>(plus(x.master, 4)) : nullptr;
                t.m = plus(x.m, ss);
                t.v = plus(x.v, ss);
                if (ss == 1) {
                    t.em = static_cast<uint8_t *>(x.m) + adam_exps_off(x.n) + at / 128;
                    t.ev = static_cast<uint8_t *>(x.v) + adam_exps_off(x.n) + at / 128;
                }
                t.group = at / 8;
                t.start = total + at - head;
                t.n = (int32_t)(end - at < kAdamChunk ? end - at : kAdamChunk);
                t.head = at ? 0 : head;
                t.number = (uint32_t)i;
                t.decay = x.weight_decay;
                t.lr_scale = x.lr_scale;
                master = master || x.master;
                table.push_back(t);
            }
            total += x.n;
        }
        if (pass == 0) aligned_chunks = (int64_t)table.size();
    }
    chunks = (int64_t)table.size();
    std::unique_ptr<gq_adamw> o(new gq_adamw);
    o->all = merged(spans, false);
    o->written = merged(spans, true);
    o->total = total;
    o->memory = nullptr;
    const size_t bytes = table.size() * sizeof(AdamChunk);
    if (cudaGetDevice(&o->device) != cudaSuccess || cudaMalloc(&o->memory, bytes + kNormParts * sizeof(double)) != cudaSuccess)
        return cuda_failed();
    unsigned char *mem = static_cast<unsigned char *>(o->memory);
    // a copy from pageable memory may return before its last bytes have arrived, and steps run on any stream
    if (bytes && (cudaMemcpy(mem, table.data(), bytes, cudaMemcpyHostToDevice) != cudaSuccess ||
                  cudaStreamSynchronize(nullptr) != cudaSuccess)) {
        cudaFree(o->memory);
        return cuda_failed();
    }
    o->a = AdamArgs{c.param_dtype, c.grad_dtype, c.state_bits, master, aligned_chunks, chunks, reinterpret_cast<AdamChunk *>(mem), c.seed};
    o->parts = reinterpret_cast<double *>(mem + bytes);
    *out = o.release();
    return GQ_OK;
}

}  // namespace

extern "C" {

gq_status_t gq_adamw_layout(int64_t n, size_t *bytes, size_t *exps_off)
{
    if (n < 0 || n >= kMaxElements) return GQ_ERR_INVALID;
    if (bytes) *bytes = adam_bytes(n);
    if (exps_off) *exps_off = adam_exps_off(n);
    return GQ_OK;
}

gq_status_t gq_adamw_create(const gq_adamw_config_t *cfg, const gq_adamw_tensor_t *tensors, int count, gq_adamw_t *out)
{
    if (!out) return GQ_ERR_INVALID;
    *out = nullptr;
    if (!cfg || !elem_size(cfg->param_dtype) || !elem_size(cfg->grad_dtype) || (cfg->state_bits != 8 && cfg->state_bits != 32))
        return GQ_ERR_INVALID;
    if (count < 0 || count > GQ_ADAMW_MAX_TENSORS || (count && !tensors)) return GQ_ERR_INVALID;
    try {
        return create(*cfg, tensors, count, out);
    } catch (...) {  // std::bad_alloc, or a length that no vector takes
        return GQ_ERR_NOMEM;
    }
}

gq_status_t gq_adamw_destroy(gq_adamw_t opt)
{
    if (!opt) return GQ_ERR_INVALID;
    const cudaError_t e = cudaFree(opt->memory);
    delete opt;
    return from_cuda(e);
}

gq_status_t gq_adamw_norm(gq_adamw_t opt, double max_norm, float *out, void *stream)
{
    Range range("gq_adamw_norm");
    if (!opt || !out || !aligned(out, 4) || !(max_norm > 0.0)) return GQ_ERR_INVALID;
    const gq_status_t st = check_device(*opt);
    if (st != GQ_OK) return st;
    if (meets(opt->all, out, 8)) return GQ_ERR_INVALID;
    return from_cuda(launch_adamw_norm(opt->a, max_norm, opt->parts, out, static_cast<cudaStream_t>(stream)));
}

gq_status_t gq_adamw_scalars(double lr, double beta1, double beta2, int64_t step, gq_adamw_scalars_t *out)
{
    if (!out || !(lr >= 0.0 && lr <= 3.0e38) || !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || step < 1 ||
        step >= int64_t(1) << 32)
        return GQ_ERR_INVALID;
    out->lr = (float)lr;
    out->inv1 = (float)(1.0 / (1.0 - std::pow(beta1, (double)step)));
    out->inv2 = (float)(1.0 / std::sqrt(1.0 - std::pow(beta2, (double)step)));
    out->step = (uint32_t)step;
    return GQ_OK;
}

gq_status_t gq_adamw_step(gq_adamw_t opt, double lr, double beta1, double beta2, double eps, int64_t step, const float *scale,
                          const void *scalars, void *stream)
{
    Range range("gq_adamw_step");
    AdamStep s = {};
    const gq_status_t bad = gq_adamw_scalars(lr, beta1, beta2, step, &s.now);
    if (!opt || bad != GQ_OK || !(eps >= 0.0 && eps <= 3.0e38) || !aligned(scale, 4) || !aligned(scalars, 16)) return GQ_ERR_INVALID;
    if (opt->a.chunks == 0) return GQ_OK;
    const gq_status_t st = check_device(*opt);
    if (st != GQ_OK) return st;
    if (meets(opt->written, scale, 4) || meets(opt->written, scalars, 16)) return GQ_ERR_INVALID;
    s.beta1 = (float)beta1;
    s.rest1 = (float)(1.0 - beta1);
    s.beta2 = (float)beta2;
    s.rest2 = (float)(1.0 - beta2);
    s.eps = (float)eps;
    // 2^-63 times inv2 at its largest, t = 1, is below 2^-24 eps; and with 2^64 times inv2 the divisor is below 2^126, whose
    // reciprocal would be subnormal
    s.fast = eps >= 0x1p-39 / std::sqrt(1.0 - beta2) && eps <= 0x1p64 && (s.beta1 == 0.0f || s.beta1 >= 0x1p-9f);
    // e4m3's widest step for its size: half of it is 1/18 of 1.125, which a tie at 17/18 still leaves for the even code below
    s.spread = (double)s.beta1 * 18.0 > 17.0;
    s.scale = scale;
    s.scalars = static_cast<const gq_adamw_scalars_t *>(scalars);
    return from_cuda(launch_adamw(opt->a, s, static_cast<cudaStream_t>(stream)));
}

gq_status_t gq_adamw_moments(gq_adamw_t opt, int dtype, void *m, void *v, void *stream)
{
    Range range("gq_adamw_moments");
    const int size = elem_size(dtype);
    if (!opt || !size || (!m && !v) || !aligned(m, 16) || !aligned(v, 16)) return GQ_ERR_INVALID;
    if (opt->a.chunks == 0) return GQ_OK;
    if (overlap(region(m, (size_t)opt->total * size), region(v, (size_t)opt->total * size))) return GQ_ERR_INVALID;
    const gq_status_t st = check_device(*opt);
    if (st != GQ_OK) return st;
    if (meets(opt->all, m, (size_t)opt->total * size) || meets(opt->all, v, (size_t)opt->total * size))
        return GQ_ERR_INVALID;
    return from_cuda(launch_adamw_moments(opt->a, dtype, m, v, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
