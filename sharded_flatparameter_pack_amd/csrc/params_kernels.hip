// params_kernels.hip -- gfx950 kernels of the optimizer step over many
// separate tensors: AdamW with fp32 or MXFP8 moments, the gradients' sum of
// squares with the overflow check, and the MXFP8 conversions.
//
// A wave works on a tile of one tensor (the step also on half of one), found
// through the tile table (tensor, tile), so that tensors of any size share
// one launch and a small one costs one wave.  Inside a tile the quad layout
// of the step kernels holds: lane t has elements [4 t, 4 t + 4), every access
// of a wave covers one contiguous span.  The tensors may start anywhere on
// their element size, so their accesses are the unaligned ones (one
// instruction, as the aligned).
//
// MXFP8: 32 consecutive elements, 8 lanes, share the scale 2^(b - 127), one
// byte b (e8m0; 255 is NaN); an element is an e4m3 code times the scale.
// With f the exponent field of the block's largest magnitude, rounded to
// e4m3's four significant bits, b = max(0, f - 7): the largest value lands
// in [124, 248], so rounding up never leaves e4m3's range (448).  A block
// with f >= 255 gets b = 255 and reads as NaN: its largest value is not finite
// or is at least 1.9375 * 2^127, which rounds to 2^128, past fp32's range.
// The hardware's scaled conversions give and take codes under such a scale.
//
// Compiled with -ffp-contract=off: every operation is one IEEE
// round-to-nearest-even operation, in the order written.

#include "fp_params.h"
#include "step_ops.h"

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

// ---------------------------------------------------------------- MXFP8

typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef short s16x2_t __attribute__((ext_vector_type(2)));

// The conversions take the scale as an fp32 of which they use the exponent
// field, the e8m0 byte itself: 0 is 2^-127, 255 gives NaN.
__device__ __forceinline__ float mx_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// The values of four codes; code times scale is exact (4 significant bits).
__device__ __forceinline__ void mx_decode(uint32_t codes, uint32_t byte, float f[4]) {
    const f32x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes, mx_scale(byte), false);
    const f32x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes, mx_scale(byte), true);
    f[0] = lo.x; f[1] = lo.y; f[2] = hi.x; f[3] = hi.y;
}

// Largest of x over the 8 lanes of a block.
__device__ __forceinline__ uint32_t block_max(uint32_t x) {
    uint32_t y = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1 /* quad_perm 1,0,3,2 */, 0xF, 0xF, true);
    x = x > y ? x : y;
    y = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E /* quad_perm 2,3,0,1 */, 0xF, 0xF, true);
    x = x > y ? x : y;
    y = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x141 /* row_half_mirror */, 0xF, 0xF, true);
    return x > y ? x : y;
}

// Scale byte of the block that the lane's four values belong to.  All lanes
// of the block take part; elements that do not exist are 0.  kRoot: the
// values have no sign (a NaN may have one, which leaves it above all others).
template <bool kRoot>
__device__ __forceinline__ uint32_t mx_byte(const float f[4]) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t a = kRoot ? __float_as_uint(f[e]) : __float_as_uint(f[e]) & 0x7FFFFFFFu;
        top = top > a ? top : a;
    }
    top = block_max(top);
    const uint32_t field = ((kRoot && top > 0x7FFFFFFFu ? 0x7FFFFFFFu : top) + 0x00080000u) >> 23;
    return field >= 255u ? 255u : field < 7u ? 0u : field - 7u;
}

// A root that is not zero does not round to zero, so that a second moment
// never becomes a division by eps alone: one below the smallest code's value
// is raised to it.  A wave without a value below it skips that; zeros are below
// it too, so one with rows that no token has reached does not.
__device__ __forceinline__ void mx_raise(float r[4], uint32_t byte) {
    const float least = __builtin_amdgcn_ldexpf(1.0f, (int)byte - 136);
    const float low = fminf(fminf(r[0], r[1]), fminf(r[2], r[3]));
    if (low < least) {
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = r[e] > 0.0f ? fmaxf(r[e], least) : r[e];
    }
}

// Codes of the lane's four values, rounded stochastically: |x| / scale has
// 20 bits of random[e] (its high bits) added below e4m3's last bit and is cut
// there, as the hardware's conversion does in the normal and the subnormal
// range alike.
__device__ __forceinline__ uint32_t mx_encode(const float f[4], uint32_t byte, const uint32_t random[4]) {
    const float s = mx_scale(byte);
    int w = 0;
    w = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(w, f[0], random[0], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(w, f[1], random[1], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(w, f[2], random[2], s, 2);
    w = __builtin_amdgcn_cvt_scalef32_sr_fp8_f32(w, f[3], random[3], s, 3);
    return byte == 255u ? 0u : (uint32_t)w;
}

// The same rounded to nearest even.
__device__ __forceinline__ uint32_t mx_encode(const float f[4], uint32_t byte) {
    const float s = mx_scale(byte);
    s16x2_t w = {0, 0};
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, f[0], f[1], s, false);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, f[2], f[3], s, true);
    return byte == 255u ? 0u : __builtin_bit_cast(uint32_t, w);
}

// 32 bits of dither for partition element e: the element's index and the
// call's key through two multiplications.  The multipliers are the golden
// ratio's and the fractions of sqrt(2) and sqrt(3).
__device__ __forceinline__ uint32_t dither(uint32_t e, uint32_t key) {
    uint32_t x = (e * 0x9E3779B1u) ^ key;
    x ^= x >> 16;
    x *= 0x6A09E667u;
    x ^= x >> 15;
    x *= 0xBB67AE85u;
    return x;
}

// ---------------------------------------------------------------- AdamW

// sqrt(v) from the hardware's estimate of 1 / sqrt (accurate to 2^-23) with one
// Newton step, to 1.5 * 2^-46.  kTiny added to v keeps a zero out of the
// estimate's pole; beside any other v here it is lost.
constexpr double kTiny = 1e-290;
__device__ __forceinline__ double root_f64(double v) {
    const double y = __builtin_amdgcn_rsq(v);
    const double s = v * y;
    return __builtin_fma(0.5 * y, __builtin_fma(-s, s, v), s);
}

// adamw_elem with the second moment given and kept as its root: all in fp64,
// the weight and the two moments, which the 8-bit codes are rounded from, each
// rounded once to fp32.  The quotient is the hardware's reciprocal (accurate to
// 2^-23) with one Newton step, to 2^-46; with the root's error the weight's
// change is within 2^-44 of its terms before the weight is rounded.  The
// denominator is at least 2^-126 (eps) and below 2^160, far inside fp64.  The
// change in fp32 is faster (1.57M elements 6.8 against 7.3 us, 226.5M 617 and
// 622), but off by up to 2^-20 of itself, which shows in weights near zero, and
// its reciprocal is lost above 2^126, which a root of 2^121 reaches at the first
// step.
__device__ __forceinline__ void adamw_root_elem(const AdamCoef& c, float g, float& th, float& m, float& r) {
    const double gd = (double)g, rd = (double)r;
    const double md = __builtin_fma(c.one_m_beta1, gd, c.beta1 * (double)m);
    const double root = root_f64(__builtin_fma(c.one_m_beta2 * gd, gd, __builtin_fma(c.beta2, rd * rd, kTiny)));
    const double denom = __builtin_fma(root, c.inv_sqrt_bias2, c.eps);
    double y = __builtin_amdgcn_rcp(denom);
    y = __builtin_fma(__builtin_fma(-denom, y, 1.0), y, y);
    th = (float)__builtin_fma(-c.step_size * md, y, c.decay * (double)th);
    m = (float)md;
    r = (float)root;
}

}  // namespace

// What a wave works on.
struct TileAt {
    ParamRec rec;
    const void* grad;
    int64_t e0;   // its first element
};

// The first `have` elements of a quad (kFull: all four).
template <bool kFull>
__device__ __forceinline__ void st_f32_part(float* p, const float f[4], int have) {
    if (kFull || have == 4) {
        st16u(p, bits_of(f));
        return;
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (k < have) gptr<float>((void*)p)[k] = f[k];
}
template <bool kFull>
__device__ __forceinline__ void st_codes(uint8_t* p, uint32_t codes, int have) {
    if (kFull || have == 4) {
        *gptr<uint32_t>((void*)p) = codes;
        return;
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (k < have) gptr<uint8_t>((void*)p)[k] = (uint8_t)(codes >> (8 * k));
}

// What a lane reads: kU quads, 64 quads apart.
template <int kGrad, bool kMx8, int kU>
struct TileRaw {
    GradQuad<kGrad> g[kU];
    uint4 th[kU];
    uint4 m[kU], v[kU];
};
template <int kGrad, int kU>
struct TileRaw<kGrad, true, kU> {
    GradQuad<kGrad> g[kU];
    uint4 th[kU];
    uint32_t m[kU], v[kU];    // four codes
    uint32_t bm[kU], bv[kU];  // the scale byte of their block
};

// Elements of the lane's quad u that the tensor has.
__device__ __forceinline__ int quad_have(const TileAt& t, int u) {
    const int64_t left = t.rec.numel - (t.e0 + 256 * u + 4 * (threadIdx.x & 63));
    return left >= 4 ? 4 : left > 0 ? (int)left : 0;
}

// kFull: the tensor has all of the tile's elements.  Else a quad that would
// pass its end is read so that it ends there (quad_drop says by how many
// elements early), and moments with the tensor's last quad (the partition has
// room up to the next multiple of 32): lanes all load, and none waits here.
// Element by element, tensors of 4001 elements took a quarter longer.
template <int kGrad, bool kMx8, int kU, bool kFull>
__device__ __forceinline__ void load_tile(const ParamsArgs& a, const TileAt& t, TileRaw<kGrad, kMx8, kU>& r) {
    const int64_t last = t.rec.numel - 4, last_quad = (t.rec.numel - 1) & ~(int64_t)3;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const int64_t e = t.e0 + 256 * u + 4 * (threadIdx.x & 63);
        const int64_t p = t.rec.offset + (kFull || e < last_quad ? e : last_quad);
        if (kFull || last >= 0) {
            const int64_t from = kFull || e < last ? e : last;
            r.g[u] = ld_grad<kGrad>(t.grad, from);
            r.th[u] = ld16u(t.rec.master + from);
        } else {
            const int n = (int)t.rec.numel;
            const FP_GLOBAL uint32_t* w = gptr<uint32_t>((const void*)t.rec.master);
            r.g[u] = ld_grad_few<kGrad>(t.grad, n);
            r.th[u] = make_uint4(w[0], n > 1 ? w[1] : 0u, n > 2 ? w[2] : 0u, 0u);
        }
        if constexpr (kMx8) {
            r.m[u] = gptr<uint32_t>(a.exp_avg)[p >> 2];
            r.v[u] = gptr<uint32_t>(a.exp_avg_sq)[p >> 2];
            r.bm[u] = gptr<uint8_t>(a.exp_avg_scale)[p / kMxBlock];
            r.bv[u] = gptr<uint8_t>(a.root_scale)[p / kMxBlock];
        } else {
            r.m[u] = ld16(static_cast<const float*>(a.exp_avg) + p);
            r.v[u] = ld16(static_cast<const float*>(a.exp_avg_sq) + p);
        }
    }
}

// Elements that quad u was read early by (see load_tile).
__device__ __forceinline__ int quad_drop(const TileAt& t, int u) {
    const int64_t last = t.rec.numel - 4, e = t.e0 + 256 * u + 4 * (threadIdx.x & 63);
    if (last < 0) return e == 0 ? 0 : 4;
    return e <= last ? 0 : e - last < 4 ? (int)(e - last) : 4;
}

// The tile's update, then its stores, one stream after the other; on a skip
// only the copy of the unchanged weights is stored.  Partition elements past
// the tensor are left as they are.
template <int kGrad, bool kMx8, int kU, bool kFull>
__device__ __forceinline__ void step_tile(const ParamsArgs& a, const TileAt& t, const TileRaw<kGrad, kMx8, kU>& r,
                                          bool skip) {
    const AdamCoef c = coef_for(a.c[t.rec.group], a.g_coef);
    const int64_t e0 = t.e0 + 4 * (threadIdx.x & 63), p0 = t.rec.offset + e0;
    int have[kU];
    float th[kU][4], m[kU][4], v[kU][4];
    uint32_t cm[kU], cv[kU], bm[kU], bv[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        have[u] = kFull ? 4 : quad_have(t, u);
        GradQuad<kGrad> gq = r.g[u];
        uint4 tq = r.th[u];
        if (!kFull) {
            gq.w = drop(gq.w, quad_drop(t, u));
            tq = drop(tq, quad_drop(t, u));
        }
        f32x4_of(tq, th[u]);
        if (skip) continue;
        float g[4];
        grad_f32<kGrad>(gq, g);
        if constexpr (kMx8) {
            mx_decode(r.m[u], r.bm[u], m[u]);
            mx_decode(r.v[u], r.bv[u], v[u]);
#pragma unroll
            for (int k = 0; k < 4; ++k) adamw_root_elem(c, g[k], th[u][k], m[u][k], v[u][k]);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (!kFull && k >= have[u]) m[u][k] = v[u][k] = 0.0f;
            bm[u] = mx_byte<false>(m[u]);
            bv[u] = mx_byte<true>(v[u]);
            uint32_t dm[4], dv[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t d = dither((uint32_t)(p0 + 256 * u) + (uint32_t)k, a.key);
                dm[k] = d & 0xFFFF0000u;
                dv[k] = d << 16;
            }
            mx_raise(v[u], bv[u]);
            cm[u] = mx_encode(m[u], bm[u], dm);
            cv[u] = mx_encode(v[u], bv[u], dv);
        } else {
            f32x4_of(r.m[u], m[u]);
            f32x4_of(r.v[u], v[u]);
#pragma unroll
            for (int k = 0; k < 4; ++k) adamw_elem(c, g[k], th[u][k], m[u][k], v[u][k]);
        }
    }
    if (!skip) {
#pragma unroll
        for (int u = 0; u < kU; ++u) st_f32_part<kFull>(t.rec.master + e0 + 256 * u, th[u], have[u]);
        if constexpr (kMx8) {
#pragma unroll
            for (int u = 0; u < kU; ++u) st_codes<kFull>(static_cast<uint8_t*>(a.exp_avg) + p0 + 256 * u, cm[u], have[u]);
#pragma unroll
            for (int u = 0; u < kU; ++u) st_codes<kFull>(static_cast<uint8_t*>(a.exp_avg_sq) + p0 + 256 * u, cv[u], have[u]);
#pragma unroll
            for (int u = 0; u < kU; ++u)
                if ((kFull || have[u] > 0) && (threadIdx.x & 7) == 0) {
                    gptr<uint8_t>(a.exp_avg_scale)[(p0 + 256 * u) / kMxBlock] = (uint8_t)bm[u];
                    gptr<uint8_t>(a.root_scale)[(p0 + 256 * u) / kMxBlock] = (uint8_t)bv[u];
                }
        } else {
#pragma unroll
            for (int u = 0; u < kU; ++u) st_f32_part<kFull>(static_cast<float*>(a.exp_avg) + p0 + 256 * u, m[u], have[u]);
#pragma unroll
            for (int u = 0; u < kU; ++u) st_f32_part<kFull>(static_cast<float*>(a.exp_avg_sq) + p0 + 256 * u, v[u], have[u]);
        }
    }
    if (t.rec.copy == nullptr) return;
    uint16_t* copy = static_cast<uint16_t*>(t.rec.copy) + e0;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const uint2 w = a.copy_f16 ? make_uint2(f16x2(th[u][0], th[u][1]), f16x2(th[u][2], th[u][3])) : f32x4_to_bf16(th[u]);
        if (kFull || have[u] == 4) {
            st8u(copy + 256 * u, w);
        } else {
            const uint32_t h[3] = {w.x, w.x >> 16, w.y};
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (k < have[u]) gptr<uint16_t>((void*)copy)[256 * u + k] = (uint16_t)h[k];
        }
    }
}

// The step: a wave has a tile, or with kU = 1 half of one; fp_params.h says
// which form runs when and what they measured.  One pass: 16.1 bytes per
// element with 8-bit moments, bf16 gradients and copies (226.5M elements 622
// us, 5.9 TB/s; the loads and stores without the arithmetic 646, so the memory
// sets it, while 42.6M in 10 000 short tensors take 131 with and 122 without),
// 28 with fp32 moments (226.5M 1004 us, 6.3 TB/s).  The loads do not wait for
// the overflow flag, as in the flat step.  A wave ends after its stores: with
// several tiles per wave and the next one's loads in flight it had to wait for
// them (one counter for both), and took 711 us where it otherwise took 640.
template <int kGrad, bool kMx8, int kU>
__global__ __launch_bounds__(kThreads) void params_step_kernel(const ParamsArgs a) {
    constexpr int kPer = kParamQuads / kU;   // waves per tile
    const int64_t i = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (i >= a.n_tiles * kPer) return;
    const ParamTile tile = a.tiles[i / kPer];
    const TileAt t = {a.recs[tile.tensor], a.grads[tile.tensor],
                      (int64_t)tile.index * kParamTile + (i % kPer) * (256 * kU)};
    const int64_t left = t.rec.numel - t.e0;
    if (left <= 0) return;
    TileRaw<kGrad, kMx8, kU> r;
    if (left >= 256 * kU) load_tile<kGrad, kMx8, kU, true>(a, t, r);
    else load_tile<kGrad, kMx8, kU, false>(a, t, r);
    const bool skip = a.found_inf != nullptr && *a.found_inf != 0;
    if (left >= 256 * kU) step_tile<kGrad, kMx8, kU, true>(a, t, r, skip);
    else step_tile<kGrad, kMx8, kU, false>(a, t, r, skip);
}

// Squares of the 8 elements of a 16-byte word (4 of fp32) added to sq[0..3].
template <int kGrad>
__device__ __forceinline__ void add_squares(const uint4 w, double sq[4]) {
    float f[8];
    constexpr int kN = kGrad == FP_DTYPE_F32 ? 4 : 8;
    if constexpr (kGrad == FP_DTYPE_F32) {
        f32x4_of(w, f);
    } else {
        GradQuad<kGrad> lo, hi;
        lo.w = make_uint2(w.x, w.y);
        hi.w = make_uint2(w.z, w.w);
        grad_f32<kGrad>(lo, f);
        grad_f32<kGrad>(hi, f + 4);
    }
#pragma unroll
    for (int k = 0; k < kN; ++k) sq[k & 3] = __builtin_fma((double)f[k], (double)f[k], sq[k & 3]);
}

// A tile of the norm: the elements of its tensor from it on, and where.
struct NormTile {
    int64_t left;
    const char* from;
};
template <int kGrad>
__device__ __forceinline__ NormTile find_norm_tile(const ParamsNormArgs& a, int64_t i) {
    const ParamTile tile = a.tiles[i];
    const int64_t e0 = (int64_t)tile.index * kParamTile;
    return {a.recs[tile.tensor].numel - e0,
            static_cast<const char*>(a.grads[tile.tensor]) + e0 * (kGrad == FP_DTYPE_F32 ? 4 : 2)};
}

// What a lane reads of it: whole words, 64 words apart, and in the tensor's
// last tile one of the elements behind the last whole word.
template <int kGrad>
struct NormRaw {
    static constexpr int kPer = kGrad == FP_DTYPE_F32 ? 4 : 8;      // elements of a word
    static constexpr int kWords = (int)(kParamTile / (64 * kPer));
    uint4 w[kWords];
    uint32_t rest;
};
template <int kGrad>
__device__ __forceinline__ void load_norm_tile(const NormTile& t, NormRaw<kGrad>& r) {
    constexpr int kPer = NormRaw<kGrad>::kPer;
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int u = 0; u < NormRaw<kGrad>::kWords; ++u) {
        r.w[u] = make_uint4(0u, 0u, 0u, 0u);
        if ((64 * u + lane + 1) * kPer <= t.left) r.w[u] = ld16u(t.from + 16 * (64 * u + lane));
    }
    r.rest = 0u;
    if (t.left < kParamTile && lane < t.left % kPer) {
        const int64_t e = t.left - t.left % kPer + lane;
        if constexpr (kGrad == FP_DTYPE_F32) r.rest = gptr<uint32_t>((const void*)t.from)[e];
        else r.rest = gptr<uint16_t>((const void*)t.from)[e];
    }
}
template <int kGrad>
__device__ __forceinline__ void add_norm_tile(const NormTile& t, const NormRaw<kGrad>& r, double sq[4]) {
#pragma unroll
    for (int u = 0; u < NormRaw<kGrad>::kWords; ++u) add_squares<kGrad>(r.w[u], sq);
    if (t.left < kParamTile) {
        const float g = kGrad == FP_DTYPE_F32 ? __uint_as_float(r.rest) : kGrad == FP_DTYPE_BF16 ? bf16_lo(r.rest) : f16_lo(r.rest);
        sq[0] = __builtin_fma((double)g, (double)g, sq[0]);
    }
}

// Sum over the norm's workgroup in a fixed order, valid in thread 0.
__device__ __forceinline__ double norm_group_sum(double x) {
    __shared__ double waves[kNormWaves];
    x = wave_sum(x);
    __syncthreads();   // a call before may still read
    if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = x;
    __syncthreads();
    double r = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < kNormWaves; ++w) r += waves[w];
    return r;
}

// Counts workgroup b of n in; true for the last one, which also leaves the
// counters at 0 for the next call.  Two levels on lines of their own, as in
// the step's grid barrier: one counter for all took 35 ns per workgroup.
__device__ __forceinline__ bool norm_arrive(uint32_t* done, unsigned b, unsigned n) {
    const unsigned group = b % kSyncGroups;
    const unsigned members = n / kSyncGroups + (group < n % kSyncGroups ? 1u : 0u);
    if (sync_add(&done[group * kLineWords], 1u) + 1u != members) return false;
    sync_store(&done[group * kLineWords], 0u);
    uint32_t* top = &done[kSyncGroups * kLineWords];
    if (sync_add(top, 1u) + 1u != sync_groups(n)) return false;
    sync_store(top, 0u);
    return true;
}

// The sum of squares in fp64 and the overflow check, in one launch.  Squares
// are not negative and their fp64 sum cannot overflow, so a sum that is not
// finite is the overflow check: three instructions per element, unpack,
// widen, fused multiply-add, leave the kernel to its loads.  Waves take tiles
// in turn, so that those in flight cover one window of memory; two, four and
// eight tiles of a wave in flight at once measured slower (226.5M bf16
// elements 74, 83 and 90 us against 72, 6.3 TB/s), as did the next tile's
// loads before a tile's sums (74) and three quarters or half of the waves
// that are resident together (81 and 107 us).  The last workgroup to finish
// adds the partial sums in their order, so the result does not depend on who
// was last.
template <int kGrad>
__global__ __launch_bounds__(kNormThreads) void params_norm_kernel(const ParamsNormArgs a) {
    double sq[4] = {0.0, 0.0, 0.0, 0.0};
    for (int64_t i = (int64_t)blockIdx.x * kNormWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); i < a.n_tiles;
         i += (int64_t)gridDim.x * kNormWaves) {
        const NormTile t = find_norm_tile<kGrad>(a, i);
        NormRaw<kGrad> r;
        load_norm_tile<kGrad>(t, r);
        add_norm_tile<kGrad>(t, r, sq);
    }
    const double mine = (sq[0] + sq[1]) + (sq[2] + sq[3]);
    flag_if_any(!__builtin_isfinite(mine), a.found_inf);
    const double t = norm_group_sum(mine);
    if (gridDim.x == 1) {
        if (threadIdx.x == 0) *a.sq_norm = t;
        return;
    }
    __shared__ int last;
    if (threadIdx.x == 0) {
        // The partial sum travels in an exchange at agent scope, whose result
        // has to be there before the count goes up; the counts go up by
        // read-modify-write, and the last workgroup's loads are at agent scope
        // too.  So every partial is in memory before it is read, without a
        // write-back of the caches.
        const double old = __hip_atomic_exchange(&a.partials[blockIdx.x], t, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("" ::"v"(old) : "memory");
        last = norm_arrive(a.done, blockIdx.x, gridDim.x);
    }
    __syncthreads();
    if (!last) return;
    double s = 0.0;
    for (unsigned k = threadIdx.x; k < gridDim.x; k += kNormThreads)
        s += __hip_atomic_load(&a.partials[k], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    s = norm_group_sum(s);
    if (threadIdx.x == 0) *a.sq_norm = s;
}

// The conversions, streams of 5 bytes per element, kMxQuads quads per lane,
// 256 quads apart.  Two measured best for 134M elements (one, two, four): out
// of 8 bits 148, 100 and 116 us (6.7 TB/s at two), second moments into 8 bits
// 128, 120 and 120, first moments 110, 113 and 116.
template <bool kRoot>
__global__ __launch_bounds__(kThreads) void mx8_quantize_kernel(const MxArgs a) {
    const int64_t e0 = ((int64_t)blockIdx.x * (kThreads * kMxQuads) + threadIdx.x) * 4;
    float f[kMxQuads][4];
#pragma unroll
    for (int u = 0; u < kMxQuads; ++u) {
        const int64_t e = e0 + 4 * kThreads * u;
        f32x4_of(make_uint4(0u, 0u, 0u, 0u), f[u]);
        if (e + 4 <= a.n) {
            f32x4_of(ld16(a.x + e), f[u]);
        } else {
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (e + k < a.n) f[u][k] = a.x[e + k];
        }
    }
#pragma unroll
    for (int u = 0; u < kMxQuads; ++u) {
        const int64_t e = e0 + 4 * kThreads * u;
        if (kRoot) {
#pragma unroll
            for (int k = 0; k < 4; ++k) f[u][k] = (float)root_f64((double)f[u][k] + kTiny);
        }
        const uint32_t byte = mx_byte<kRoot>(f[u]);
        if (kRoot) mx_raise(f[u], byte);
        const uint32_t w = mx_encode(f[u], byte);
        if (e + 4 <= a.n) {
            *reinterpret_cast<uint32_t*>(a.codes + e) = w;
        } else {
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (e + k < a.n) a.codes[e + k] = (uint8_t)(w >> (8 * k));
        }
        if (e < a.n && (threadIdx.x & 7) == 0) a.scales[e / kMxBlock] = (uint8_t)byte;
    }
}

template <bool kRoot>
__global__ __launch_bounds__(kThreads) void mx8_dequantize_kernel(const MxArgs a) {
    const int64_t e0 = ((int64_t)blockIdx.x * (kThreads * kMxQuads) + threadIdx.x) * 4;
    uint32_t w[kMxQuads], byte[kMxQuads];
#pragma unroll
    for (int u = 0; u < kMxQuads; ++u) {
        const int64_t e = e0 + 4 * kThreads * u;
        w[u] = byte[u] = 0u;
        if (e < a.n) byte[u] = a.scales[e / kMxBlock];
        if (e + 4 <= a.n) {
            w[u] = *reinterpret_cast<const uint32_t*>(a.codes + e);
        } else {
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (e + k < a.n) w[u] |= (uint32_t)a.codes[e + k] << (8 * k);
        }
    }
#pragma unroll
    for (int u = 0; u < kMxQuads; ++u) {
        const int64_t e = e0 + 4 * kThreads * u;
        float f[4];
        mx_decode(w[u], byte[u], f);
        if (kRoot) {
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = f[k] * f[k];
        }
        if (e + 4 <= a.n) {
            st16(a.x + e, bits_of(f));
        } else {
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (e + k < a.n) a.x[e + k] = f[k];
        }
    }
}

// ---------------------------------------------------------------- launchers

template <int kGrad>
void launch_step_of(const ParamsArgs& a, int64_t partition, bool mx8, hipStream_t s) {
    const unsigned whole = (unsigned)ceil_div64(a.n_tiles, kWaves), half = (unsigned)ceil_div64(2 * a.n_tiles, kWaves);
    static_assert(kParamQuads == 2, "half a tile is one quad per lane");
    if (!mx8) params_step_kernel<kGrad, false, 1><<<half, kThreads, partition < kParamCapElems ? 0 : kParamCapLds, s>>>(a);
    else if (partition < kMx8WholeElems) params_step_kernel<kGrad, true, 1><<<half, kThreads, 0, s>>>(a);
    else params_step_kernel<kGrad, true, 2><<<whole, kThreads, 0, s>>>(a);
}

hipError_t launch_params_step(const ParamsArgs& a, int64_t partition, int grad_dtype, bool mx8, hipStream_t s) {
    switch (grad_dtype) {
        case FP_DTYPE_F32: launch_step_of<FP_DTYPE_F32>(a, partition, mx8, s); break;
        case FP_DTYPE_BF16: launch_step_of<FP_DTYPE_BF16>(a, partition, mx8, s); break;
        default: launch_step_of<FP_DTYPE_F16>(a, partition, mx8, s);
    }
    return hipGetLastError();
}

hipError_t launch_params_norm(const ParamsNormArgs& a, int grad_dtype, hipStream_t s) {
    const unsigned grid = (unsigned)params_norm_groups(a.n_tiles);
    switch (grad_dtype) {
        case FP_DTYPE_F32: params_norm_kernel<FP_DTYPE_F32><<<grid, kNormThreads, 0, s>>>(a); break;
        case FP_DTYPE_BF16: params_norm_kernel<FP_DTYPE_BF16><<<grid, kNormThreads, 0, s>>>(a); break;
        default: params_norm_kernel<FP_DTYPE_F16><<<grid, kNormThreads, 0, s>>>(a);
    }
    return hipGetLastError();
}

hipError_t launch_mx8(const MxArgs& a, bool quantize, bool root, hipStream_t s) {
    const unsigned grid = (unsigned)ceil_div64(a.n, kMxTile);
    if (quantize) {
        if (root) mx8_quantize_kernel<true><<<grid, kThreads, 0, s>>>(a);
        else mx8_quantize_kernel<false><<<grid, kThreads, 0, s>>>(a);
    } else {
        if (root) mx8_dequantize_kernel<true><<<grid, kThreads, 0, s>>>(a);
        else mx8_dequantize_kernel<false><<<grid, kThreads, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace fpk
