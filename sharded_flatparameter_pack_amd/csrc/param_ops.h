// param_ops.h -- device helpers of the kernels that work on separate tensors:
// gradient quads of any type at any element, and the stochastic rounding's
// dither.
#pragma once

#include "fp_device.h"

namespace fpk {
namespace {

// Addresses in global memory (see FP_GLOBAL).
template <class T>
__device__ __forceinline__ FP_GLOBAL T* gptr(void* p) {
    return static_cast<FP_GLOBAL T*>((FP_GLOBAL void*)p);
}
template <class T>
__device__ __forceinline__ const FP_GLOBAL T* gptr(const void* p) {
    return static_cast<const FP_GLOBAL T*>((const FP_GLOBAL void*)p);
}

// ---------------------------------------------------------------- gradients

template <int kGrad>
struct GradQuad {
    uint2 w;
};
template <>
struct GradQuad<FP_DTYPE_F32> {
    uint4 w;
};

__device__ __forceinline__ float f16_lo(uint32_t w) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)(w & 0xFFFFu));
}
__device__ __forceinline__ float f16_hi(uint32_t w) { return f16_lo(w >> 16); }

// Gradient quad starting at element e, all four elements present.
template <int kGrad>
__device__ __forceinline__ GradQuad<kGrad> ld_grad(const void* g, int64_t e) {
    GradQuad<kGrad> q;
    if constexpr (kGrad == FP_DTYPE_F32) q.w = ld16u(static_cast<const float*>(g) + e);
    else q.w = ld8u(static_cast<const uint16_t*>(g) + e);
    return q;
}

// The first n < 4 elements of a tensor that has no more, as a quad.
template <int kGrad>
__device__ __forceinline__ GradQuad<kGrad> ld_grad_few(const void* g, int n) {
    uint32_t w[3] = {0u, 0u, 0u};
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (k < n) {
            if constexpr (kGrad == FP_DTYPE_F32) w[k] = gptr<uint32_t>(g)[k];
            else w[k] = gptr<uint16_t>(g)[k];
        }
    GradQuad<kGrad> q;
    if constexpr (kGrad == FP_DTYPE_F32) q.w = make_uint4(w[0], w[1], w[2], 0u);
    else q.w = make_uint2(w[0] | (w[1] << 16), w[2]);
    return q;
}

// A quad without its first s elements (s >= 4: without any), zeros behind.
__device__ __forceinline__ uint4 drop(const uint4 w, int s) {
    const uint32_t a = s & 1 ? w.y : w.x, b = s & 1 ? w.z : w.y, c = s & 1 ? w.w : w.z, d = s & 1 ? 0u : w.w;
    const uint4 r = s & 2 ? make_uint4(c, d, 0u, 0u) : make_uint4(a, b, c, d);
    return s >= 4 ? make_uint4(0u, 0u, 0u, 0u) : r;
}
__device__ __forceinline__ uint2 drop(const uint2 w, int s) {
    const uint64_t x = (((uint64_t)w.y << 32) | w.x) >> (16 * (s & 3));
    return s >= 4 ? make_uint2(0u, 0u) : make_uint2((uint32_t)x, (uint32_t)(x >> 32));
}

template <int kGrad>
__device__ __forceinline__ void grad_f32(const GradQuad<kGrad>& q, float f[4]) {
    if constexpr (kGrad == FP_DTYPE_F32) {
        f[0] = __uint_as_float(q.w.x); f[1] = __uint_as_float(q.w.y);
        f[2] = __uint_as_float(q.w.z); f[3] = __uint_as_float(q.w.w);
    } else if constexpr (kGrad == FP_DTYPE_BF16) {
        bf16x4_to_f32(q.w, f);
    } else {
        f[0] = f16_lo(q.w.x); f[1] = f16_hi(q.w.x);
        f[2] = f16_lo(q.w.y); f[3] = f16_hi(q.w.y);
    }
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)lo) |
           ((uint32_t)__builtin_bit_cast(uint16_t, (_Float16)hi) << 16);
}

// The same in one instruction.
__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
    typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{lo, hi}), f16x2_t));
}

__device__ __forceinline__ void f32x4_of(const uint4 w, float f[4]) {
    f[0] = __uint_as_float(w.x); f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z); f[3] = __uint_as_float(w.w);
}

__device__ __forceinline__ uint4 bits_of(const float f[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

typedef unsigned int u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// 16 bytes to a 4-byte boundary (fp32 weights that are views of a buffer).
__device__ __forceinline__ void st16u(void* p, const uint4 v) {
    const u32x4_a4 w = {v.x, v.y, v.z, v.w};
    __builtin_nontemporal_store(w, (FP_GLOBAL u32x4_a4*)(p));
}

// 16 and 8 bytes without the non-temporal hint: data that is used again, and
// stores whose lines several instructions write (non-temporal ones do not meet in
// the L2: a step's weights and copies went to memory twice).
__device__ __forceinline__ uint4 get16(const void* p) {
    const u32x4_t v = *gptr<u32x4_t>(p);
    return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ uint2 get8(const void* p) {
    const u32x2_t v = *gptr<u32x2_t>(p);
    return make_uint2(v.x, v.y);
}
__device__ __forceinline__ void st16h(void* p, const uint4 v) {  // non-temporal, from a 2-byte boundary
    __builtin_nontemporal_store((u32x4_a2{v.x, v.y, v.z, v.w}), (FP_GLOBAL u32x4_a2*)(p));
}
__device__ __forceinline__ void put16u(void* p, const uint4 v) {  // from a 4-byte boundary
    *gptr<u32x4_a4>(p) = u32x4_a4{v.x, v.y, v.z, v.w};
}
__device__ __forceinline__ uint4 get16u(const void* p) {
    const u32x4_a4 v = *gptr<u32x4_a4>(p);
    return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ uint2 get8h(const void* p) {
    const u32x2_a2 v = *gptr<u32x2_a2>(p);
    return make_uint2(v.x, v.y);
}
__device__ __forceinline__ void put8h(void* p, const uint2 v) { *gptr<u32x2_a2>(p) = u32x2_a2{v.x, v.y}; }
__device__ __forceinline__ void put16(void* p, const uint4 v) { *gptr<u32x4_t>(p) = u32x4_t{v.x, v.y, v.z, v.w}; }

// 32 bits of dither for partition element e: the element's index and the
// call's key through two multiplications.  The multipliers are the golden
// ratio's and the fractions of sqrt(2) and sqrt(3).
constexpr uint32_t kDitherStep = 0x9E3779B1u;
__device__ __forceinline__ uint32_t dither_at(uint32_t product, uint32_t key) {  // of e kDitherStep
    uint32_t x = product ^ key;
    x ^= x >> 16;
    x *= 0x6A09E667u;
    x ^= x >> 15;
    x *= 0xBB67AE85u;
    return x;
}
__device__ __forceinline__ uint32_t dither(uint32_t e, uint32_t key) { return dither_at(e * kDitherStep, key); }

}  // namespace
}  // namespace fpk
