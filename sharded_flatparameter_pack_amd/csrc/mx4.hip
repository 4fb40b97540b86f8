// mx4.hip -- the entry points of MXFP4 (fp_mx4_*): argument checks.  Every
// check runs before anything is enqueued.

#include <hip/hip_runtime.h>

#include <cstring>

#include "fp_matrix.h"
#include "plan_util.h"

using namespace fpk;

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 31;   // rows and columns
constexpr int64_t kMaxK = (int64_t)1 << 22;     // of a product: a tile's byte offsets are 32-bit
constexpr int64_t kMaxLanes = 0xFFFFFFFFLL;     // of a launch

int64_t dtype_bytes(int32_t dtype) { return dtype == FP_DTYPE_F32 ? 4 : 2; }
bool known(int32_t dtype) { return dtype >= FP_DTYPE_F32 && dtype <= FP_DTYPE_F16; }

// A matrix with rows `pitch` elements apart.
Span matrix_span(const void* p, int64_t rows, int64_t cols, int64_t pitch, int32_t dtype) {
    return span_of(p, rows > 0 ? ((rows - 1) * pitch + cols) * dtype_bytes(dtype) : 0);
}

// One MXFP4 form of `rows` rows of `width` elements: both pointers or none.
fp_status check_form(const uint8_t* codes, const uint8_t* scales, const char* name) {
    if (codes == nullptr || scales == nullptr) return bad(FP_ERR_INVALID, "%s: codes or scales is NULL", name);
    if (!on(codes, 16) || !on(scales, 8)) return bad(FP_ERR_ALIGN, "%s: codes must be 16-byte aligned, scales 8-byte", name);
    return FP_OK;
}
Span codes_span(const uint8_t* p, int64_t rows, int64_t width) { return span_of(p, rows * mx4_pad(width) / 2); }
Span scales_span(const uint8_t* p, int64_t rows, int64_t width) { return span_of(p, rows * mx4_pad(width) / kMx4Block); }

fp_status check_shape(int64_t rows, int64_t cols, int64_t pitch) {
    if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim)
        return bad(FP_ERR_RANGE, "%lld x %lld out of range", (long long)rows, (long long)cols);
    if (pitch < cols || pitch > ((int64_t)1 << 40)) return bad(FP_ERR_RANGE, "row pitch %lld of %lld columns", (long long)pitch, (long long)cols);
    return FP_OK;
}

}  // namespace

extern "C" int64_t fp_mx4_padded(int64_t n) { return n < 0 || n > kMaxDim ? -1 : mx4_pad(n); }

extern "C" fp_status fp_mx4_quantize(int64_t rows, int64_t cols, int64_t pitch, int32_t dtype, const void* x, uint8_t* codes,
                                     uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t, int32_t stochastic,
                                     uint64_t seed, void* stream) {
    return guarded([&]() -> fp_status {
        fp_status st = check_shape(rows, cols, pitch);
        if (st != FP_OK) return st;
        if (!known(dtype)) return bad(FP_ERR_INVALID, "unknown dtype %d", dtype);
        const bool by_row = codes != nullptr || scales != nullptr, by_col = codes_t != nullptr || scales_t != nullptr;
        if (rows == 0 || cols == 0) return FP_OK;
        if (!by_row && !by_col) return bad(FP_ERR_INVALID, "neither the rows' nor the columns' form is wanted");
        if (x == nullptr) return bad(FP_ERR_INVALID, "x is NULL");
        if (!on(x, (uintptr_t)dtype_bytes(dtype))) return bad(FP_ERR_ALIGN, "x misaligned");
        std::vector<Span> spans;
        spans.push_back(matrix_span(x, rows, cols, pitch, dtype));
        if (by_row) {
            if ((st = check_form(codes, scales, "rows' form")) != FP_OK) return st;
            spans.push_back(codes_span(codes, rows, cols));
            spans.push_back(scales_span(scales, rows, cols));
        }
        if (by_col) {
            if ((st = check_form(codes_t, scales_t, "columns' form")) != FP_OK) return st;
            spans.push_back(codes_span(codes_t, cols, rows));
            spans.push_back(scales_span(scales_t, cols, rows));
        }
        for (size_t i = 0; i < spans.size(); ++i)
            for (size_t j = 0; j < i; ++j)
                if (meet(spans[i], spans[j])) return bad(FP_ERR_INVALID, "two of the buffers overlap");
        Mx4QuantArgs a = {x, rows, cols, pitch, codes, scales, codes_t, scales_t, mx4_pad(cols), mx4_pad(rows),
                          stochastic ? key_of(seed) : 0u, dtype, stochastic != 0};
        if (mx4_quantize_lanes(a) > kMaxLanes)
            return bad(FP_ERR_RANGE, "%lld x %lld needs more workgroups than one launch holds", (long long)rows, (long long)cols);
        hipError_t e = launch_mx4_quantize(a, static_cast<hipStream_t>(stream));
        return e == hipSuccess ? FP_OK : device_error(e, "mx4 quantize launch");
    });
}

extern "C" fp_status fp_mx4_dequantize(int64_t rows, int64_t cols, const uint8_t* codes, const uint8_t* scales, int32_t dtype,
                                       void* out, int64_t pitch, void* stream) {
    return guarded([&]() -> fp_status {
        fp_status st = check_shape(rows, cols, pitch);
        if (st != FP_OK) return st;
        if (!known(dtype)) return bad(FP_ERR_INVALID, "unknown dtype %d", dtype);
        if (rows == 0 || cols == 0) return FP_OK;
        if ((st = check_form(codes, scales, "rows' form")) != FP_OK) return st;
        if (out == nullptr) return bad(FP_ERR_INVALID, "out is NULL");
        if (!on(out, (uintptr_t)dtype_bytes(dtype))) return bad(FP_ERR_ALIGN, "out misaligned");
        const Span so = matrix_span(out, rows, cols, pitch, dtype);
        if (meet(so, codes_span(codes, rows, cols)) || meet(so, scales_span(scales, rows, cols)))
            return bad(FP_ERR_INVALID, "out overlaps codes or scales");
        if (rows * ceil_div64(cols, 8) > kMaxLanes)
            return bad(FP_ERR_RANGE, "%lld x %lld needs more workgroups than one launch holds", (long long)rows, (long long)cols);
        const Mx4DequantArgs a = {codes, scales, out, rows, cols, pitch, mx4_pad(cols), dtype};
        hipError_t e = launch_mx4_dequantize(a, static_cast<hipStream_t>(stream));
        return e == hipSuccess ? FP_OK : device_error(e, "mx4 dequantize launch");
    });
}

extern "C" fp_status fp_mx4_matmul(int64_t m, int64_t n, int64_t k, const uint8_t* a_codes, const uint8_t* a_scales,
                                   const uint8_t* b_codes, const uint8_t* b_scales, int32_t dtype, void* out, int64_t pitch,
                                   int32_t accumulate, void* stream) {
    return guarded([&]() -> fp_status {
        fp_status st = check_shape(m, n, pitch);
        if (st != FP_OK) return st;
        const bool empty = m == 0 || n == 0;
        if (k < (empty ? 0 : 1) || k > kMaxK) return bad(FP_ERR_RANGE, "k %lld outside [1, %lld]", (long long)k, (long long)kMaxK);
        if (!known(dtype)) return bad(FP_ERR_INVALID, "unknown dtype %d", dtype);
        if (empty) return FP_OK;
        if ((st = check_form(a_codes, a_scales, "a")) != FP_OK) return st;
        if ((st = check_form(b_codes, b_scales, "b")) != FP_OK) return st;
        if (out == nullptr) return bad(FP_ERR_INVALID, "out is NULL");
        if (!on(out, (uintptr_t)dtype_bytes(dtype))) return bad(FP_ERR_ALIGN, "out misaligned");
        const Span so = matrix_span(out, m, n, pitch, dtype);
        if (meet(so, codes_span(a_codes, m, k)) || meet(so, scales_span(a_scales, m, k)) ||
            meet(so, codes_span(b_codes, n, k)) || meet(so, scales_span(b_scales, n, k)))
            return bad(FP_ERR_INVALID, "out overlaps an operand");
        Mx4MatmulArgs a;
        std::memset(&a, 0, sizeof a);
        a.a = a_codes; a.as = a_scales; a.b = b_codes; a.bs = b_scales;
        a.out = out; a.m = m; a.n = n; a.kp = mx4_pad(k); a.pitch = pitch;
        a.dtype = dtype; a.accumulate = accumulate != 0;
        if (mx4_matmul_lanes(a) > kMaxLanes)
            return bad(FP_ERR_RANGE, "%lld x %lld needs more workgroups than one launch holds", (long long)m, (long long)n);
        hipError_t e = launch_mx4_matmul(a, static_cast<hipStream_t>(stream));
        return e == hipSuccess ? FP_OK : device_error(e, "mx4 product launch");
    });
}
