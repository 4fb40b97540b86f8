// params.hip -- the entry points of the step over many separate tensors
// (fp_params_*) and of the MXFP8 conversions: argument checks, the plans and
// their device tables.  Every check runs before anything is enqueued.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <new>
#include <vector>

#include "fp_params.h"

using namespace fpk;

namespace {

fp_status bad(fp_status st, const char* fmt, ...) {
    char text[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof text, fmt, ap);
    va_end(ap);
    return report_error(st, text);
}

fp_status device_error(hipError_t e, const char* what) {
    return bad(FP_ERR_DEVICE, "%s: %s", what, hipGetErrorString(e));
}

bool on(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A dispatch holds at most this many workgroups of kThreads lanes.
constexpr int64_t kMaxGroups = 0xFFFFFFFFLL / kThreads;

int64_t dtype_bytes(int32_t dtype) { return dtype == FP_DTYPE_F32 ? 4 : 2; }

// Bytes [lo, hi) of a buffer.
struct Span {
    uintptr_t lo, hi;
    bool operator<(const Span& o) const { return lo < o.lo; }
};

Span span_of(const void* p, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, a + (uintptr_t)bytes};
}

bool meet(const Span& a, const Span& b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

// Sorted, disjoint spans that cover the same bytes (touching ones joined).
std::vector<Span> joined(std::vector<Span> v) {
    std::sort(v.begin(), v.end());
    std::vector<Span> r;
    for (const Span& s : v) {
        if (s.lo >= s.hi) continue;
        if (!r.empty() && s.lo <= r.back().hi) r.back().hi = std::max(r.back().hi, s.hi);
        else r.push_back(s);
    }
    return r;
}

bool meets_any(const Span& a, const std::vector<Span>& sorted) {
    if (a.lo >= a.hi) return false;
    auto it = std::upper_bound(sorted.begin(), sorted.end(), a);
    if (it != sorted.end() && meet(a, *it)) return true;
    return it != sorted.begin() && meet(a, *(it - 1));
}

}  // namespace

struct fp_params {
    int32_t n = 0;
    int device = -1;
    int32_t grad_dtype = FP_DTYPE_F32, copy_dtype = FP_DTYPE_BF16;
    bool has_master = false;
    int32_t max_group = 0;
    int64_t partition = 0, tiles = 0;
    std::vector<int64_t> numel, offset;
    std::vector<Span> written;         // weights and copies
    void* dev = nullptr;               // records, gradient table, tile table
    void* staging = nullptr;           // pinned, of the gradient table's uploads
    hipEvent_t uploaded = nullptr;
    std::mutex mu;                     // guards the fields below
    std::vector<Span> read;            // gradients
    const void* checked[4] = {};       // moments that last passed the overlap checks
    bool have_checked = false;

    const ParamRec* recs() const { return static_cast<const ParamRec*>(dev); }
    const void** grads() const { return reinterpret_cast<const void**>(static_cast<char*>(dev) + sizeof(ParamRec) * (size_t)n); }
    const ParamTile* tile_table() const { return reinterpret_cast<const ParamTile*>(grads() + n); }
};

namespace {

void free_params(fp_params* p) {
    int cur = -1;
    (void)hipGetDevice(&cur);
    if (p->device >= 0) (void)hipSetDevice(p->device);
    if (p->uploaded) (void)hipEventSynchronize(p->uploaded), (void)hipEventDestroy(p->uploaded);
    if (p->staging) (void)hipHostFree(p->staging);
    if (p->dev) (void)hipFree(p->dev);
    if (cur >= 0) (void)hipSetDevice(cur);
    delete p;
}

fp_status check_device(const fp_params* p) {
    int device = -1;
    hipError_t e = hipGetDevice(&device);
    if (e != hipSuccess) return device_error(e, "hipGetDevice");
    if (device != p->device)
        return bad(FP_ERR_INVALID, "params plan was created on device %d, current is %d", p->device, device);
    return FP_OK;
}

// Checks a gradient table against the plan; *spans receives the gradients'
// bytes, joined.
fp_status check_grads(const std::vector<int64_t>& numel, int32_t dtype, const std::vector<Span>& written,
                      const void* const* grads, std::vector<Span>* spans) {
    const int64_t es = dtype_bytes(dtype);
    std::vector<Span> v;
    v.reserve(numel.size());
    for (size_t i = 0; i < numel.size(); ++i) {
        if (numel[i] == 0) continue;
        if (grads[i] == nullptr) return bad(FP_ERR_INVALID, "grads[%zu] is NULL", i);
        if (!on(grads[i], (uintptr_t)es)) return bad(FP_ERR_ALIGN, "grads[%zu] misaligned", i);
        v.push_back(span_of(grads[i], numel[i] * es));
        if (meets_any(v.back(), written)) return bad(FP_ERR_INVALID, "grads[%zu] overlaps a weight or a copy", i);
    }
    *spans = joined(std::move(v));
    return FP_OK;
}

fp_status create(int32_t n, const int64_t* numel, const int32_t* group, int32_t grad_dtype, const void* const* grads,
                 float* const* master, int32_t copy_dtype, void* const* copies, fp_params** out) {
    if (out == nullptr) return bad(FP_ERR_INVALID, "out is NULL");
    *out = nullptr;
    if (n < 1) return bad(FP_ERR_RANGE, "n must be >= 1");
    if (numel == nullptr || grads == nullptr) return bad(FP_ERR_INVALID, "numel or grads is NULL");
    if (grad_dtype < FP_DTYPE_F32 || grad_dtype > FP_DTYPE_F16) return bad(FP_ERR_INVALID, "unknown grad_dtype %d", grad_dtype);
    if (copies != nullptr && copy_dtype != FP_DTYPE_BF16 && copy_dtype != FP_DTYPE_F16)
        return bad(FP_ERR_INVALID, "copy_dtype must be bf16 or fp16 (got %d)", copy_dtype);
    if (copies != nullptr && master == nullptr) return bad(FP_ERR_INVALID, "copies need master weights");
    int64_t partition = 0, tiles = 0;
    int32_t max_group = 0;
    std::vector<Span> written;
    for (int32_t i = 0; i < n; ++i) {
        if (numel[i] < 0 || numel[i] > ((int64_t)1 << 40))
            return bad(FP_ERR_RANGE, "tensor %d: numel %lld out of range", i, (long long)numel[i]);
        if (group != nullptr) {
            if (group[i] < 0 || group[i] >= FP_MAX_GROUPS)
                return bad(FP_ERR_RANGE, "tensor %d: group %d outside [0, %d)", i, group[i], FP_MAX_GROUPS);
            max_group = std::max(max_group, group[i]);
        }
        if (numel[i] == 0) continue;
        if (master != nullptr) {
            if (master[i] == nullptr) return bad(FP_ERR_INVALID, "master[%d] is NULL", i);
            if (!on(master[i], 4)) return bad(FP_ERR_ALIGN, "master[%d] misaligned", i);
            written.push_back(span_of(master[i], numel[i] * 4));
        }
        if (copies != nullptr) {
            if (copies[i] == nullptr) return bad(FP_ERR_INVALID, "copies[%d] is NULL", i);
            if (!on(copies[i], 2)) return bad(FP_ERR_ALIGN, "copies[%d] misaligned", i);
            written.push_back(span_of(copies[i], numel[i] * 2));
        }
        partition += ceil_div64(numel[i], kMxBlock) * kMxBlock;
        tiles += param_tiles(numel[i]);
        if (ceil_div64(tiles * kParamQuads, kWaves) > kMaxGroups)  // one wave per quad of a lane at most
            return bad(FP_ERR_RANGE, "the tensors need more workgroups than one launch holds (%lld)", (long long)kMaxGroups);
    }
    std::sort(written.begin(), written.end());
    for (size_t i = 1; i < written.size(); ++i)
        if (meet(written[i - 1], written[i])) return bad(FP_ERR_INVALID, "two of the weights and copies overlap");
    written = joined(std::move(written));
    const std::vector<int64_t> sizes(numel, numel + n);
    std::vector<Span> read;
    fp_status st = check_grads(sizes, grad_dtype, written, grads, &read);
    if (st != FP_OK) return st;

    // host image of the device tables
    const size_t rec_b = sizeof(ParamRec) * (size_t)n, ptr_b = sizeof(void*) * (size_t)n;
    std::vector<unsigned char> image(rec_b + ptr_b + sizeof(ParamTile) * (size_t)tiles, 0);
    fp_params* p = new fp_params();
    p->n = n;
    p->grad_dtype = grad_dtype;
    p->copy_dtype = copy_dtype;
    p->has_master = master != nullptr;
    p->max_group = max_group;
    p->partition = partition;
    p->tiles = tiles;
    p->numel = sizes;
    p->written = std::move(written);
    p->read = std::move(read);
    ParamRec* rec = reinterpret_cast<ParamRec*>(image.data());
    const void** ptr = reinterpret_cast<const void**>(image.data() + rec_b);
    ParamTile* tile = reinterpret_cast<ParamTile*>(image.data() + rec_b + ptr_b);
    int64_t offset = 0;
    for (int32_t i = 0; i < n; ++i) {
        rec[i].master = master != nullptr ? master[i] : nullptr;
        rec[i].copy = copies != nullptr ? copies[i] : nullptr;
        rec[i].numel = numel[i];
        rec[i].offset = offset;
        rec[i].group = group != nullptr ? group[i] : 0;
        ptr[i] = grads[i];
        const int64_t nt = param_tiles(numel[i]);
        for (int64_t t = 0; t < nt; ++t) *tile++ = {i, (int32_t)t};
        p->offset.push_back(offset);
        offset += ceil_div64(numel[i], kMxBlock) * kMxBlock;
    }
    hipError_t e = hipGetDevice(&p->device);
    if (e == hipSuccess) e = hipMalloc(&p->dev, image.size());
    if (e == hipSuccess) e = hipMemcpy(p->dev, image.data(), image.size(), hipMemcpyHostToDevice);
    if (e != hipSuccess) {
        free_params(p);
        return device_error(e, "building the params tables");
    }
    *out = p;
    return FP_OK;
}

fp_status set_grads(fp_params* p, const void* const* grads, void* stream) {
    if (p == nullptr || grads == nullptr) return bad(FP_ERR_INVALID, "params or grads is NULL");
    fp_status st = check_device(p);
    if (st != FP_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
    hipError_t e = hipStreamIsCapturing(s, &capture);
    if (e != hipSuccess) return device_error(e, "hipStreamIsCapturing");
    if (capture != hipStreamCaptureStatusNone)
        return bad(FP_ERR_INVALID, "the gradients cannot be changed while the stream is captured");
    std::vector<Span> read;
    if ((st = check_grads(p->numel, p->grad_dtype, p->written, grads, &read)) != FP_OK) return st;
    std::lock_guard<std::mutex> lock(p->mu);
    const size_t bytes = sizeof(void*) * (size_t)p->n;
    if (p->staging == nullptr) {
        if ((e = hipHostMalloc(&p->staging, bytes, hipHostMallocDefault)) != hipSuccess) {
            p->staging = nullptr;
            return device_error(e, "allocating the gradient table's staging");
        }
    }
    if (p->uploaded == nullptr) {
        if ((e = hipEventCreateWithFlags(&p->uploaded, hipEventDisableTiming)) != hipSuccess) {
            p->uploaded = nullptr;
            return device_error(e, "creating the upload event");
        }
    } else if ((e = hipEventSynchronize(p->uploaded)) != hipSuccess) {  // the staging may still feed the last upload
        return device_error(e, "hipEventSynchronize");
    }
    std::memcpy(p->staging, grads, bytes);
    if ((e = hipMemcpyAsync(p->grads(), p->staging, bytes, hipMemcpyHostToDevice, s)) != hipSuccess)
        return device_error(e, "uploading the gradient table");
    if ((e = hipEventRecord(p->uploaded, s)) != hipSuccess) return device_error(e, "hipEventRecord");
    p->read = std::move(read);
    p->have_checked = false;
    return FP_OK;
}

// The moments of a step: alignment, and no overlap with each other or with
// the plan's tensors.  A set that passed last time is not checked again.
fp_status check_moments(fp_params* p, const void* const* ptr, const int64_t* bytes, const uintptr_t* align,
                        const char* const* name, int count) {
    for (int i = 0; i < count; ++i) {
        if (ptr[i] == nullptr && p->partition > 0) return bad(FP_ERR_INVALID, "%s is NULL", name[i]);
        if (!on(ptr[i], align[i])) return bad(FP_ERR_ALIGN, "%s is not %d-byte aligned", name[i], (int)align[i]);
    }
    const void* key[4] = {ptr[0], ptr[1], count > 2 ? ptr[2] : nullptr, count > 2 ? ptr[3] : nullptr};
    std::lock_guard<std::mutex> lock(p->mu);
    if (p->have_checked && std::equal(key, key + 4, p->checked)) return FP_OK;
    for (int i = 0; i < count; ++i) {
        const Span s = span_of(ptr[i], bytes[i]);
        for (int j = 0; j < i; ++j)
            if (meet(s, span_of(ptr[j], bytes[j]))) return bad(FP_ERR_INVALID, "%s overlaps %s", name[i], name[j]);
        if (meets_any(s, p->written)) return bad(FP_ERR_INVALID, "%s overlaps a weight or a copy", name[i]);
        if (meets_any(s, p->read)) return bad(FP_ERR_INVALID, "%s overlaps a gradient", name[i]);
    }
    std::copy(key, key + 4, p->checked);
    p->have_checked = true;
    return FP_OK;
}

// The arguments that both forms of the step share.
fp_status step_args(const fp_params* p, int32_t n_groups, const fp_adamw_hparams* hp, const int32_t* found_inf,
                    const double* grad_coef, ParamsArgs* a) {
    if (!p->has_master) return bad(FP_ERR_INVALID, "params plan has no master weights");
    if (n_groups <= p->max_group || n_groups > FP_MAX_GROUPS)
        return bad(FP_ERR_RANGE, "n_groups %d: the tensors use groups up to %d, at most %d", n_groups, p->max_group,
                   FP_MAX_GROUPS);
    if (hp == nullptr) return bad(FP_ERR_INVALID, "hparams is NULL");
    std::memset(a, 0, sizeof *a);
    for (int32_t g = 0; g < n_groups; ++g) {
        fp_status st = adam_coef(&hp[g], &a->c[g]);
        if (st != FP_OK) return st;
    }
    if (!on(found_inf, 4)) return bad(FP_ERR_ALIGN, "found_inf misaligned");
    if (!on(grad_coef, 8)) return bad(FP_ERR_ALIGN, "grad_coef misaligned");
    a->recs = p->recs();
    a->grads = p->grads();
    a->tiles = p->tile_table();
    a->n_tiles = p->tiles;
    a->found_inf = found_inf;
    a->g_coef = grad_coef;
    a->copy_f16 = p->copy_dtype == FP_DTYPE_F16 ? 1 : 0;
    return FP_OK;
}

// The stochastic rounding's key: the seed through two rounds of
// multiplication, so that seeds that count steps give unrelated keys.  The
// first multiplier is 2^64 over the golden ratio; the second, with the shifts by
// 32 around it, is the published 64-bit integer mixer known as degski's.
uint32_t key_of(uint64_t seed) {
    uint64_t z = seed * 0x9E3779B97F4A7C15ull;
    z ^= z >> 32;
    z *= 0xD6E8FEB86659FD93ull;
    return (uint32_t)(z ^ (z >> 32));
}

fp_status run_step(const fp_params* p, const ParamsArgs& a, bool mx8, void* stream) {
    fp_status st = check_device(p);
    if (st != FP_OK || p->tiles == 0) return st;
    hipError_t e = launch_params_step(a, p->partition, p->grad_dtype, mx8, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? FP_OK : device_error(e, "params step launch");
}

fp_status mx8_call(int64_t n, bool quantize, int32_t root, const float* x, const uint8_t* codes, const uint8_t* scales,
                   void* stream) {
    if (n < 0) return bad(FP_ERR_RANGE, "n must be >= 0");
    if (n == 0) return FP_OK;
    if (ceil_div64(n, kMxTile) > kMaxGroups)
        return bad(FP_ERR_RANGE, "n %lld needs more workgroups than one launch holds", (long long)n);
    if (x == nullptr || codes == nullptr || scales == nullptr)
        return bad(FP_ERR_INVALID, "the fp32 buffer, codes or scales is NULL");
    if (!on(x, 16) || !on(codes, 16)) return bad(FP_ERR_ALIGN, "the fp32 buffer and codes must be 16-byte aligned");
    const Span sx = span_of(x, 4 * n), sc = span_of(codes, n), ss = span_of(scales, ceil_div64(n, kMxBlock));
    if (meet(sx, sc) || meet(sx, ss) || meet(sc, ss)) return bad(FP_ERR_INVALID, "two of the buffers overlap");
    const MxArgs a = {const_cast<float*>(x), const_cast<uint8_t*>(codes), const_cast<uint8_t*>(scales), n};
    hipError_t e = launch_mx8(a, quantize, root != 0, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? FP_OK : device_error(e, "mx8 launch");
}

// Runs `f`; no C++ exception leaves an entry point.
template <class F>
fp_status guarded(F f) {
    try {
        return f();
    } catch (const std::bad_alloc&) {
        return bad(FP_ERR_DEVICE, "out of host memory");
    } catch (...) {
        return bad(FP_ERR_DEVICE, "unexpected host error");
    }
}

}  // namespace

extern "C" fp_status fp_params_create(int32_t n, const int64_t* numel, const int32_t* group, int32_t grad_dtype,
                                      const void* const* grads, float* const* master, int32_t copy_dtype,
                                      void* const* copies, fp_params** out) {
    return guarded([&] { return create(n, numel, group, grad_dtype, grads, master, copy_dtype, copies, out); });
}

extern "C" void fp_params_destroy(fp_params* params) {
    if (params != nullptr) free_params(params);
}

extern "C" fp_status fp_params_info(const fp_params* params, int64_t* partition, int64_t* workspace_bytes) {
    if (params == nullptr) return bad(FP_ERR_INVALID, "params is NULL");
    if (partition) *partition = params->partition;
    if (workspace_bytes) *workspace_bytes = kNormHeader + 8 * params_norm_groups(params->tiles);
    return FP_OK;
}

extern "C" fp_status fp_params_offsets(const fp_params* params, int64_t* offsets) {
    if (params == nullptr || offsets == nullptr) return bad(FP_ERR_INVALID, "params or offsets is NULL");
    std::copy(params->offset.begin(), params->offset.end(), offsets);
    return FP_OK;
}

extern "C" fp_status fp_params_set_grads(fp_params* params, const void* const* grads, void* stream) {
    return guarded([&] { return set_grads(params, grads, stream); });
}

extern "C" fp_status fp_params_grad_norm(const fp_params* params, int32_t* found_inf, double* sq_norm, void* workspace,
                                         void* stream) {
    if (params == nullptr || sq_norm == nullptr) return bad(FP_ERR_INVALID, "params or sq_norm is NULL");
    if (workspace == nullptr) return bad(FP_ERR_INVALID, "workspace is NULL");
    if (!on(found_inf, 4)) return bad(FP_ERR_ALIGN, "found_inf misaligned");
    if (!on(sq_norm, 8)) return bad(FP_ERR_ALIGN, "sq_norm misaligned");
    if (!on(workspace, 16)) return bad(FP_ERR_ALIGN, "workspace is not 16-byte aligned");
    fp_status st = check_device(params);
    if (st != FP_OK) return st;
    const ParamsNormArgs a = {params->recs(), params->grads(), params->tile_table(), params->tiles, found_inf,
                              reinterpret_cast<double*>(static_cast<char*>(workspace) + kNormHeader),
                              static_cast<uint32_t*>(workspace), sq_norm};
    hipError_t e = launch_params_norm(a, params->grad_dtype, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? FP_OK : device_error(e, "gradient norm launch");
}

extern "C" fp_status fp_params_adamw(fp_params* params, int32_t n_groups, const fp_adamw_hparams* hp, float* exp_avg,
                                     float* exp_avg_sq, const int32_t* found_inf, const double* grad_coef,
                                     void* stream) {
    return guarded([&]() -> fp_status {
        if (params == nullptr) return bad(FP_ERR_INVALID, "params is NULL");
        ParamsArgs a;
        fp_status st = step_args(params, n_groups, hp, found_inf, grad_coef, &a);
        if (st != FP_OK) return st;
        const void* ptr[] = {exp_avg, exp_avg_sq};
        const int64_t bytes[] = {4 * params->partition, 4 * params->partition};
        const uintptr_t align[] = {16, 16};
        const char* const name[] = {"exp_avg", "exp_avg_sq"};
        if ((st = check_moments(params, ptr, bytes, align, name, 2)) != FP_OK) return st;
        a.exp_avg = exp_avg;
        a.exp_avg_sq = exp_avg_sq;
        return run_step(params, a, false, stream);
    });
}

extern "C" fp_status fp_params_adamw8(fp_params* params, int32_t n_groups, const fp_adamw_hparams* hp, uint8_t* exp_avg,
                                      uint8_t* exp_avg_scale, uint8_t* root, uint8_t* root_scale, uint64_t seed,
                                      const int32_t* found_inf, const double* grad_coef, void* stream) {
    return guarded([&]() -> fp_status {
        if (params == nullptr) return bad(FP_ERR_INVALID, "params is NULL");
        ParamsArgs a;
        fp_status st = step_args(params, n_groups, hp, found_inf, grad_coef, &a);
        if (st != FP_OK) return st;
        const int64_t P = params->partition;
        const void* ptr[] = {exp_avg, exp_avg_scale, root, root_scale};
        const int64_t bytes[] = {P, P / kMxBlock, P, P / kMxBlock};
        const uintptr_t align[] = {16, 1, 16, 1};
        const char* const name[] = {"exp_avg", "exp_avg_scale", "root", "root_scale"};
        if ((st = check_moments(params, ptr, bytes, align, name, 4)) != FP_OK) return st;
        a.exp_avg = exp_avg;
        a.exp_avg_sq = root;
        a.exp_avg_scale = exp_avg_scale;
        a.root_scale = root_scale;
        a.key = key_of(seed);
        for (int32_t g = 0; g < n_groups; ++g) a.c[g].eps = std::max(a.c[g].eps, 0x1p-126);  // no denominator is 0
        return run_step(params, a, true, stream);
    });
}

extern "C" fp_status fp_mx8_quantize(int64_t n, int32_t root, const float* x, uint8_t* codes, uint8_t* scales,
                                     void* stream) {
    return mx8_call(n, true, root, x, codes, scales, stream);
}

extern "C" fp_status fp_mx8_dequantize(int64_t n, int32_t root, const uint8_t* codes, const uint8_t* scales, float* x,
                                       void* stream) {
    return mx8_call(n, false, root, x, codes, scales, stream);
}
