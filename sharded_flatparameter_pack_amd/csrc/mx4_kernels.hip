// mx4_kernels.hip -- gfx950 kernels of MXFP4: quantisation of a matrix along
// its rows and its columns, the values read back, and the product of two
// MXFP4 operands along their rows.
//
// MXFP4: 32 consecutive elements of a row share the scale 2^(b - 127), one byte
// b (e8m0; 255 is NaN); an element is an e2m1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6
// and their negatives; two per byte, the first in the low half) times it.  With
// f the exponent field of the block's largest magnitude after rounding,
// b = max(0, f - 2): the largest value lands on 4 or 6 without being cut.
// Rounding to nearest even carries f up from 1.75 * 2^e on (a value below 7
// rounds to 6 at most); the stochastic rounding, which may go up to the next
// value from anywhere, from above 1.5 * 2^e on (so none passes 6).  f >= 255
// gives b = 255: the block reads as NaN.
//
// Compiled with -ffp-contract=off.

#include <type_traits>

#include "fp_matrix.h"
#include "mma_tile.h"
#include "param_ops.h"

namespace fpk {

namespace {

typedef float f32x2_v __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float scale_f32(uint32_t byte) { return __uint_as_float(byte << 23); }

template <int kDtype>
__device__ __forceinline__ float to_f32(uint32_t bits) {
    if constexpr (kDtype == FP_DTYPE_F32) return __uint_as_float(bits);
    else if constexpr (kDtype == FP_DTYPE_BF16) return bf16_lo(bits);
    else return f16_lo(bits);
}

// Scale byte from the bits of the block's largest magnitude.
template <bool kRandom>
__device__ __forceinline__ uint32_t mx4_byte(uint32_t top) {
    const uint32_t f = (top + (kRandom ? 0x003FFFFFu : 0x00200000u)) >> 23;
    return f >= 255u ? 255u : f < 2u ? 0u : f - 2u;
}

// Codes of eight values, rounded to nearest even.
__device__ __forceinline__ uint32_t mx4_encode(const float f[8], uint32_t byte) {
    const float s = scale_f32(byte);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[0], f[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[2], f[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[4], f[5], s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[6], f[7], s, 3);
    return byte == 255u ? 0u : w;
}

// Eight values rounded stochastically: with y = |x| / scale in [0, 6] and q the
// distance of the codes' values around y (0.5, 1 or 2), the code is that of
// q floor(y / q + d / 2^16).  y 2^-126 in fp32 has e2m1's exponent steps, and
// below y = 1, where fp32's subnormals begin, e2m1's even ones: its bits, with d
// added below e2m1's last one (bit 22), are the code after a cut.  The product
// that gives y 2^-126 has to be cut too, not rounded (what is cut lies below d's
// last bit): the kernel's rounding is towards zero (round_to_zero).
__device__ __forceinline__ uint32_t mx4_encode(const float f[8], uint32_t byte, const uint32_t d[8]) {
    uint32_t w = 0, c[8];  // c: sign, 6 zeros, code, 22 bits to cut
#pragma unroll
    for (int k = 0; k < 8; ++k) c[k] = __float_as_uint(__builtin_amdgcn_ldexpf(f[k], 1 - (int)byte)) + (d[k] << 6);  // times 2^(127 - byte) 2^-126
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // two at a time, in the word's halves
        const uint32_t p = __builtin_amdgcn_perm(c[k + 4], c[k], 0x07060302u);
        w |= ((p >> 6 & 0x00070007u) | (p >> 12 & 0x00080008u)) << (4 * k);
    }
    return byte == 255u ? 0u : w;
}

// fp32 operations of the wave round towards zero from here on.
__device__ __forceinline__ void round_to_zero() {
    __builtin_amdgcn_s_setreg(1 /* MODE */ | 0 << 6 | (2 - 1) << 11, 3);
}

// Elements [at, at + 8) of x as they are in memory, those past `have` 0.
template <int kDtype>
struct Eight {
    uint32_t w[kDtype == FP_DTYPE_F32 ? 8 : 4];
};
template <int kDtype>
__device__ __forceinline__ Eight<kDtype> ld_eight(const void* x, int64_t at, int have) {
    Eight<kDtype> r;
    if constexpr (kDtype == FP_DTYPE_F32) {
        const float* p = static_cast<const float*>(x) + at;
        if (have >= 8) {
            const uint4 a = ld16u(p), b = ld16u(p + 4);
            r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
            r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
            return r;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) r.w[k] = k < have ? gptr<uint32_t>((const void*)p)[k] : 0u;
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(x) + at;
        if (have >= 8) {
            const uint4 a = ld16u(p);
            r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
            return r;
        }
        uint32_t e[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] = k < have ? (uint32_t)gptr<uint16_t>((const void*)p)[k] : 0u;
#pragma unroll
        for (int k = 0; k < 4; ++k) r.w[k] = e[2 * k] | e[2 * k + 1] << 16;
    }
    return r;
}
// Element k's bits.
template <int kDtype>
__device__ __forceinline__ uint32_t bits_at(const Eight<kDtype>& r, int k) {
    if constexpr (kDtype == FP_DTYPE_F32) return r.w[k];
    else return k & 1 ? r.w[k >> 1] >> 16 : r.w[k >> 1] & 0xFFFFu;
}

// The dither of elements e .. e + 7.
__device__ __forceinline__ void dither8(uint32_t e, uint32_t key, uint32_t h[8]) {
    const uint32_t p = e * kDitherStep;
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] = dither_at(p + (uint32_t)k * kDitherStep, key);
}

// A block's eight elements of four lanes, along a row: its codes and scale.
template <int kDtype, bool kRandom>
__device__ __forceinline__ void row_block(const Mx4QuantArgs& a, const Eight<kDtype>& r, const uint32_t (&h)[8], int64_t row, int64_t col) {
    float f[8];
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        f[k] = to_f32<kDtype>(bits_at<kDtype>(r, k));
        const uint32_t m = __float_as_uint(f[k]) & 0x7FFFFFFFu;
        top = top > m ? top : m;
    }
    uint32_t y = (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0xB1 /* quad_perm 1,0,3,2 */, 0xF, 0xF, true);
    top = top > y ? top : y;
    y = (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0x4E /* quad_perm 2,3,0,1 */, 0xF, 0xF, true);
    top = top > y ? top : y;
    const uint32_t byte = mx4_byte<kRandom>(top);
    uint32_t codes;
    if constexpr (kRandom) {
        uint32_t d[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k] = h[k] >> 16;
        codes = mx4_encode(f, byte, d);
    } else {
        codes = mx4_encode(f, byte);
    }
    if (row >= a.rows || col >= a.cp) return;
    gptr<uint32_t>((void*)a.codes)[(row * a.cp + col) >> 3] = codes;
    if ((threadIdx.x & 3) == 0) gptr<uint8_t>((void*)a.scales)[(row * a.cp + col) >> 5] = (uint8_t)byte;
}

// The rows' form alone: eight elements per lane, rows behind each other, so that a
// single row's blocks spread over many CUs (1 x 4096: 2 us, a launch's latency; in
// 128 x 128 tiles 4.9).
template <int kDtype, bool kRandom>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const Mx4QuantArgs a) {
    if (kRandom) round_to_zero();
    const uint32_t lane = blockIdx.x * 256u + threadIdx.x, across = (uint32_t)(a.cp >> 3);
    const int64_t row = lane / across, col = (int64_t)(lane - (uint32_t)row * across) * 8, left = a.cols - col;
    const int have = row >= a.rows || left <= 0 ? 0 : left < 8 ? (int)left : 8;
    const Eight<kDtype> r = ld_eight<kDtype>(a.x, row * a.pitch + col, have);
    uint32_t h[8] = {};
    if constexpr (kRandom) dither8((uint32_t)(row * a.cols + col), a.key, h);
    row_block<kDtype, kRandom>(a, r, h, row, col);
}

// A 128 x 128 tile.  Rows' form: four lanes hold a block, eight elements each,
// and all of a lane's rows are loaded before the first is worked on.  Columns'
// form: a lane holds a block, read down a column of the tile in LDS, where an
// element of 16 bits has its half of the dither beside it (a hash of its own for each
// form: 118 us for 8192 x 8192 bf16, so 77 to 87).  A tile's part of a row's or a
// column's codes is half a line: its neighbours follow on the same die, so that one
// L2 gets both halves (else 45 % more is written: 5003 x 2730 stochastically 31 us, so
// 28).  To nearest, memory bounds it (8192 x 8192 fp32: 77 us, 4.4 TB/s);
// stochastically its instructions do, 31 per element, the hash's two products as
// long as four others each.
constexpr int kQTile = 128;
template <int kDtype, bool kRows, bool kRandom>
__global__ __launch_bounds__(256) void quantize_kernel(const Mx4QuantArgs a) {
    constexpr bool kWide = kDtype == FP_DTYPE_F32, kBeside = kRandom && !kWide;
    typedef typename std::conditional<kWide || kBeside, uint32_t, uint16_t>::type held_t;
    __shared__ held_t tile[kQTile][kQTile + 2];
    if (kRandom) round_to_zero();
    const unsigned across = kRows ? (unsigned)(a.cp / kQTile) : (unsigned)((a.cols + kQTile - 1) / kQTile), fours = (across + 1) / 2;
    // blockIdx % 8 is the die, on which 2 x 2 tiles follow each other
    const unsigned in = blockIdx.x >> 3, four = (in >> 2) * 8 + (blockIdx.x & 7);
    const int64_t row0 = ((int64_t)(four / fours) * 2 + (in >> 1 & 1)) * kQTile, col0 = ((int64_t)(four % fours) * 2 + (in & 1)) * kQTile;
    if (row0 >= a.rp || col0 >= (int64_t)across * kQTile) return;
    const int c8 = (threadIdx.x & 15) * 8, r0 = threadIdx.x >> 4;
    const int64_t left = a.cols - (col0 + c8);
    Eight<kDtype> r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = row0 + r0 + 16 * i;
        r[i] = ld_eight<kDtype>(a.x, row * a.pitch + col0 + c8, row >= a.rows || left <= 0 ? 0 : left < 8 ? (int)left : 8);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int lr = r0 + 16 * i;
        uint32_t h[8] = {};
        if constexpr (kRandom && (kRows || kBeside)) dither8((uint32_t)((row0 + lr) * a.cols + col0 + c8), a.key, h);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t w = bits_at<kDtype>(r[i], k);
            tile[lr][c8 + k] = (held_t)(kBeside ? w | h[k] << 16 : w);
        }
        if constexpr (kRows) row_block<kDtype, kRandom>(a, r[i], h, row0 + lr, col0 + c8);
    }
    __syncthreads();
    const int lc = threadIdx.x & 127;
    const int64_t col = col0 + lc;
    if (col >= a.cols) return;
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        const int lr = ((threadIdx.x >> 7) * 2 + i) * 32;
        held_t e[32];
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
            e[k] = tile[lr + k][lc];
            const uint32_t m = __float_as_uint(to_f32<kDtype>(kBeside ? e[k] & 0xFFFFu : (uint32_t)e[k])) & 0x7FFFFFFFu;
            top = top > m ? top : m;
        }
        const uint32_t byte = mx4_byte<kRandom>(top);
        const uint32_t step = (uint32_t)a.cols * kDitherStep;
        uint32_t product = (uint32_t)((row0 + lr) * a.cols + col) * kDitherStep;
        uint32_t codes[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float f[8];
            uint32_t d[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t w = (uint32_t)e[8 * q + k];
                f[k] = to_f32<kDtype>(kBeside ? w & 0xFFFFu : w);
                if constexpr (kBeside) d[k] = w >> 16;
                else if constexpr (kRandom) d[k] = dither_at(product, a.key) & 0xFFFFu, product += step;
            }
            if constexpr (kRandom) codes[q] = mx4_encode(f, byte, d);
            else codes[q] = mx4_encode(f, byte);
        }
        const int64_t at = col * a.rp + row0 + lr;
        put16(a.codes_t + (at >> 1), make_uint4(codes[0], codes[1], codes[2], codes[3]));
        gptr<uint8_t>((void*)a.scales_t)[at >> 5] = (uint8_t)byte;
    }
}

// ---------------------------------------------------------------- dequantize

// Values of eight codes.
__device__ __forceinline__ void mx4_decode(uint32_t codes, uint32_t byte, float f[8]) {
    const float s = scale_f32(byte);
    const f32x2_v a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 0);
    const f32x2_v b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 1);
    const f32x2_v c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 2);
    const f32x2_v d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 3);
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
    f[4] = c.x; f[5] = c.y; f[6] = d.x; f[7] = d.y;
}

// Eight values per lane, a row's columns side by side.  Its writes bound it (8192 x
// 8192 to bf16: 25 us, 6.8 TB/s with the codes in the last-level cache).
template <int kDtype>
__global__ __launch_bounds__(256) void dequantize_kernel(const Mx4DequantArgs a, uint32_t across) {
    const uint32_t lane = blockIdx.x * 256u + threadIdx.x;
    const int64_t row = lane / across, col = (int64_t)(lane - (uint32_t)row * across) * 8;
    if (row >= a.rows || col >= a.cols) return;
    const int64_t e = row * a.cp + col;
    float f[8];
    mx4_decode(gptr<uint32_t>((const void*)a.codes)[e >> 3], gptr<uint8_t>((const void*)a.scales)[e >> 5], f);
    const int64_t left = a.cols - col, to = row * a.pitch + col;
    if constexpr (kDtype == FP_DTYPE_F32) {
        float* p = static_cast<float*>(a.out) + to;
        if (left >= 8) {
            put16u(p, bits_of(f));
            put16u(p + 4, bits_of(f + 4));
        } else {
            for (int k = 0; k < (int)left; ++k) gptr<float>((void*)p)[k] = f[k];
        }
    } else {
        uint16_t* p = static_cast<uint16_t*>(a.out) + to;
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            w[k] = kDtype == FP_DTYPE_F16 ? f16_pair(f[2 * k], f[2 * k + 1]) : bf16x2(f[2 * k], f[2 * k + 1]);
        if (left >= 8) {
            st16h(p, make_uint4(w[0], w[1], w[2], w[3]));
        } else {
            for (int k = 0; k < (int)left; ++k) gptr<uint16_t>((void*)p)[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
        }
    }
}

// ---------------------------------------------------------------- product

// kVec neighbouring elements of the output, 4 of fp32 or 8 of 16 bits, as they are
// in memory: 16 bytes.
struct Old {
    uint4 w;
};

// The output's old values, where they are added to; those past its end are 0.
template <int kVec>
__device__ __forceinline__ Old ld_old(const Mx4MatmulArgs& a, int64_t row, int64_t col) {
    Old o = {make_uint4(0u, 0u, 0u, 0u)};
    if (!a.accumulate || row >= a.m || col >= a.n) return o;
    const int64_t left = a.n - col, at = row * a.pitch + col;
    if constexpr (kVec == 4) {
        const float* p = static_cast<const float*>(a.out) + at;
        if (left >= 4) {
            o.w = ld16u(p);
        } else {
            const FP_GLOBAL uint32_t* q = gptr<uint32_t>((const void*)p);
            o.w = make_uint4(q[0], left > 1 ? q[1] : 0u, left > 2 ? q[2] : 0u, 0u);
        }
    } else {
        const Eight<FP_DTYPE_BF16> e = ld_eight<FP_DTYPE_BF16>(a.out, at, left < 8 ? (int)left : 8);
        o.w = make_uint4(e.w[0], e.w[1], e.w[2], e.w[3]);
    }
    return o;
}

// Stores kVec neighbouring elements (row, col ..), those that the output has.
template <int kVec>
__device__ __forceinline__ void st_out(const Mx4MatmulArgs& a, int64_t row, int64_t col, const float* v, const Old& o) {
    if (row >= a.m || col >= a.n) return;
    const int64_t left = a.n - col, at = row * a.pitch + col;
    const uint32_t old[4] = {o.w.x, o.w.y, o.w.z, o.w.w};
    if constexpr (kVec == 4) {
        float* p = static_cast<float*>(a.out) + at;
        float f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = a.accumulate ? v[k] + __uint_as_float(old[k]) : v[k];
        if (left >= 4) {
            st16u(p, bits_of(f));
            return;
        }
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if (k < left) gptr<float>((void*)p)[k] = f[k];
    } else {
        const bool half = a.dtype == FP_DTYPE_F16;
        uint16_t* p = static_cast<uint16_t*>(a.out) + at;
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float lo = v[2 * k], hi = v[2 * k + 1];
            if (a.accumulate) {
                lo += half ? f16_lo(old[k]) : bf16_lo(old[k]);
                hi += half ? f16_hi(old[k]) : bf16_hi(old[k]);
            }
            w[k] = half ? f16_pair(lo, hi) : bf16x2(lo, hi);
        }
        if (left >= 8) {
            st16h(p, make_uint4(w[0], w[1], w[2], w[3]));
            return;
        }
#pragma unroll
        for (int k = 0; k < 7; ++k)
            if (k < left) gptr<uint16_t>((void*)p)[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
    }
}

// A tile per workgroup.  8192 x 8192 x 4096 (16 steps a tile) to bf16: 167 us (3.3
// PFLOP/s), of which a tile's start and its outputs take a third; 8192 x 4096 x 8192 to
// bf16 140, with fp32 outputs 150.
template <class S, int kVec>
__global__ __launch_bounds__(S::kThreadsWg, S::kWavesSimd) void matmul_kernel(const Mx4MatmulArgs a) {
    extern __shared__ __align__(16) char lds[];
    const int t = die_tile(blockIdx.x, a.tiles_m * a.tiles_n);
    // bands of kBand rows of tiles, column by column: tiles that run together read few operands
    constexpr int kBand = 4;
    const int band = t / (kBand * a.tiles_n), in = t - band * kBand * a.tiles_n;
    const int rows = a.tiles_m - band * kBand < kBand ? a.tiles_m - band * kBand : kBand;
    const int64_t i0 = (int64_t)(band * kBand + in % rows) * S::kBM, j0 = (int64_t)(in / rows) * S::kBN;
    const int64_t pitch = a.kp >> 1, spitch = a.kp >> 5;
    const int64_t lm = a.m - i0, ln = a.n - j0;
    TileProduct<S> tile;
    run_tile<kRowsFp4, kRowsFp4>(tile, {a.a + i0 * pitch, pitch, lm < S::kBM ? (int)lm : S::kBM, a.as + i0 * spitch},
                                 {a.b + j0 * pitch, pitch, ln < S::kBN ? (int)ln : S::kBN, a.bs + j0 * spitch},
                                 (int)(a.kp >> 8), lds);
    tile.template each<2, kVec>(
        lds, [&](int r, int c) { return ld_old<kVec>(a, i0 + r, j0 + c); },
        [&](int r, int c, const float* v, const Old& o) { st_out<kVec>(a, i0 + r, j0 + c, v, o); });
}

// Products of few rows (a: up to 16 kF; tokens of a generation) with a matrix that
// is no larger than its workgroups fill the card (shape_of): b is read once, and
// that bounds them, so a workgroup has 16 of its rows and its waves share K.  Fragments come straight from memory, a wave's
// steps kAhead at a time; the waves' sums meet in LDS, in their order.  1 x 8192 x
// 4096: 5.6 us with b in the last-level cache, 7.2 from memory (2.5 TB/s; b's bytes alone
// 2.9), a launch's latency and two trips to memory; on 64-wide tiles 7.4 and 14.8.
constexpr int kThinWaves = 8;
template <int kF>
__global__ __launch_bounds__(64 * kThinWaves, 2) void thin_kernel(const Mx4MatmulArgs a) {
    __shared__ f32x4_t sums[kThinWaves][kF][64];
    constexpr int kAhead = kF == 1 ? 4 : 2;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int g = lane >> 4, j = lane & 15;
    const int64_t pitch = a.kp >> 1, j0 = (int64_t)blockIdx.x * 16;
    const int64_t rb = j0 + j < a.n ? j0 + j : a.n - 1;
    const uint8_t* pb = a.b + rb * pitch + 32 * g;
    const uint8_t* sb = a.bs + rb * (pitch >> 4) + 2 * g;
    const uint8_t *pa[kF], *sa[kF];
#pragma unroll
    for (int m = 0; m < kF; ++m) {
        const int64_t ra = 16 * m + j < a.m ? 16 * m + j : a.m - 1;
        pa[m] = a.a + ra * pitch + 32 * g;
        sa[m] = a.as + ra * (pitch >> 4) + 2 * g;
    }
    f32x4_t acc[kF];
#pragma unroll
    for (int m = 0; m < kF; ++m) acc[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    struct Step {  // a lane's 64 codes of a row, with their two scales
        uint4 lo, hi;
        uint32_t s;
    };
    auto ld = [&](const uint8_t* p, const uint8_t* s, int k) {
        return Step{get16(p + (int64_t)k * kStepBytes), get16(p + (int64_t)k * kStepBytes + 16), *gptr<uint16_t>(s + (int64_t)k * 8)};
    };
    auto wide = [](const uint4 v) { return i32x8_t{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0}; };
    const int steps = (int)(a.kp >> 8), each = (steps + kThinWaves - 1) / kThinWaves;
    const int from = wave * each, to = from + each < steps ? from + each : steps;
    for (int k = from; k < to; k += kAhead) {
        Step b[kAhead], x[kAhead][kF];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int at = k + i < to ? k + i : to - 1;
            b[i] = ld(pb, sb, at);
#pragma unroll
            for (int m = 0; m < kF; ++m) x[i][m] = ld(pa[m], sa[m], at);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (k + i >= to) break;
#pragma unroll
            for (int m = 0; m < kF; ++m) {
                acc[m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(b[i].lo), wide(x[i][m].lo), acc[m], 4, 4, 0, (int)b[i].s, 0, (int)x[i][m].s);
                acc[m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(b[i].hi), wide(x[i][m].hi), acc[m], 4, 4, 1, (int)b[i].s, 1, (int)x[i][m].s);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < kF; ++m) sums[wave][m][lane] = acc[m];
    __syncthreads();
    if (wave >= kF) return;
    f32x4_t v = sums[0][wave][lane];
#pragma unroll
    for (int w = 1; w < kThinWaves; ++w) v += sums[w][wave][lane];
    // row 16 wave + j, columns j0 + 4 g .. + 3
    const int64_t row = 16 * wave + j, col = j0 + 4 * g;
    if (row >= a.m) return;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        if (col + q < a.n) {
            const int64_t at = row * a.pitch + col + q;
            float f = v[q];
            if (a.dtype == FP_DTYPE_F32) {
                FP_GLOBAL float* o = gptr<float>(a.out) + at;
                *o = a.accumulate ? f + *o : f;
            } else {
                FP_GLOBAL uint16_t* o = gptr<uint16_t>(a.out) + at;
                const bool half = a.dtype == FP_DTYPE_F16;
                if (a.accumulate) f += half ? f16_lo(*o) : bf16_lo(*o);
                *o = (uint16_t)(half ? f16_pair(f, f) : bf16x2(f, f));
            }
        }
}

using Shape256 = TileShape<256, 256, 128, 64>;
using Shape128 = TileShape<128, 128, 64, 64>;
using Shape64 = TileShape<64, 64, 32, 32>;

template <class S, int kVec>
hipError_t run_matmul(Mx4MatmulArgs a, hipStream_t s) {
    a.tiles_m = (int32_t)ceil_div64(a.m, S::kBM);
    a.tiles_n = (int32_t)ceil_div64(a.n, S::kBN);
    return launch<matmul_kernel<S, kVec>>((unsigned)(a.tiles_m * a.tiles_n), S::kThreadsWg, S::kLdsFp4, s, a);
}
template <class S>
hipError_t run_matmul(const Mx4MatmulArgs& a, hipStream_t s) {
    return a.dtype == FP_DTYPE_F32 ? run_matmul<S, 4>(a, s) : run_matmul<S, 8>(a, s);
}

// Workgroups: whole 2 x 2 tiles (columns in padding that no form wants have none),
// as many on each die.
int64_t quant_tiles(const Mx4QuantArgs& a) {
    const int64_t across = ceil_div64(a.codes != nullptr ? a.cp : a.cols, kQTile), down = a.rp / kQTile;
    return ceil_div64(ceil_div64(across, 2) * (down / 2), 8) * 8 * 4;
}
int64_t quant_groups(const Mx4QuantArgs& a) { return a.codes_t != nullptr ? quant_tiles(a) : ceil_div64(a.rows * a.cp, 8 * 256); }

template <int kDtype, bool kRandom>
hipError_t run_quantize(const Mx4QuantArgs& a, hipStream_t s) {
    const unsigned grid = (unsigned)quant_groups(a);
    if (a.codes_t == nullptr) quantize_rows_kernel<kDtype, kRandom><<<grid, 256, 0, s>>>(a);
    else if (a.codes != nullptr) quantize_kernel<kDtype, true, kRandom><<<grid, 256, 0, s>>>(a);
    else quantize_kernel<kDtype, false, kRandom><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

int64_t mx4_quantize_lanes(const Mx4QuantArgs& a) { return quant_groups(a) * 256; }

// What a product is run on.  Tiles are the smaller the fewer there are: a shape
// serves while two workgroups per CU hold all of its tiles at once, for then a
// product takes as long as one tile does (4096 wide in K and across, to bf16: 512
// rows on 64-wide tiles 11.7 us, on 128-wide ones 15.9; 1024 rows 24.2 and 17.6; 2048
// rows on 128-wide tiles 27.6, on 256-wide ones 33.7; 2304 rows 40.7 and 33.8), and
// where larger tiles would be mostly empty.  The thin kernel, whose workgroups
// read all of a, for as many workgroups per 16 rows of a (with b in the last-level
// cache, 1 x 8192 x 4096: 5.6 us, on 64-wide tiles 7.4; 16 x 8192 x 16384: 24 and 34; 32 x
// 2048 x 4096: 6.4 and 7.7; 32 x 8192 x 4096: 10.6 and 7.7; 64 x 2048 x 4096 with kF 4: 9.2
// and 8.2; with b from memory 7.2 and 14.8, 30 and 51, 7.3 and 15, 12 and 15 for the first
// four).
enum { kThin1, kThin2, kTiles64, kTiles128, kTiles256 };
static int64_t tiles_of(const Mx4MatmulArgs& a, int64_t side) { return ceil_div64(a.m, side) * ceil_div64(a.n, side); }
static int shape_of(const Mx4MatmulArgs& a) {
    constexpr int64_t kAtOnce = 512, kMaxLanes = 0xFFFFFFFFLL;
    const int64_t least = a.m < a.n ? a.m : a.n, thin = ceil_div64(a.n, 16);
    if (a.m <= 16 && thin <= kAtOnce) return kThin1;
    if (a.m <= 32 && 2 * thin <= kAtOnce) return kThin2;
    auto serves = [&](int64_t side, int64_t threads) {
        const int64_t tiles = tiles_of(a, side);
        return tiles <= kAtOnce || (least <= side && tiles * threads <= kMaxLanes);
    };
    return serves(64, Shape64::kThreadsWg) ? kTiles64 : serves(128, Shape128::kThreadsWg) ? kTiles128 : kTiles256;
}
// More than a launch holds only where the largest tiles do not suffice.
int64_t mx4_matmul_lanes(const Mx4MatmulArgs& a) {
    return shape_of(a) == kTiles256 ? tiles_of(a, 256) * Shape256::kThreadsWg : 0;
}

hipError_t launch_mx4_quantize(const Mx4QuantArgs& a, hipStream_t s) {
#define FP_QUANT(D) (a.stochastic ? run_quantize<D, true>(a, s) : run_quantize<D, false>(a, s))
    return a.dtype == FP_DTYPE_F32 ? FP_QUANT(FP_DTYPE_F32) : a.dtype == FP_DTYPE_BF16 ? FP_QUANT(FP_DTYPE_BF16) : FP_QUANT(FP_DTYPE_F16);
#undef FP_QUANT
}

hipError_t launch_mx4_dequantize(const Mx4DequantArgs& a, hipStream_t s) {
    const uint32_t lanes = (uint32_t)ceil_div64(a.cols, 8);
    const unsigned grid = (unsigned)ceil_div64(a.rows * (int64_t)lanes, 256);
    if (a.dtype == FP_DTYPE_F32) dequantize_kernel<FP_DTYPE_F32><<<grid, 256, 0, s>>>(a, lanes);
    else if (a.dtype == FP_DTYPE_BF16) dequantize_kernel<FP_DTYPE_BF16><<<grid, 256, 0, s>>>(a, lanes);
    else dequantize_kernel<FP_DTYPE_F16><<<grid, 256, 0, s>>>(a, lanes);
    return hipGetLastError();
}

hipError_t launch_mx4_matmul(const Mx4MatmulArgs& a, hipStream_t s) {
    const unsigned thin = (unsigned)ceil_div64(a.n, 16);
    switch (shape_of(a)) {
        case kThin1: return launch<thin_kernel<1>>(thin, 64 * kThinWaves, 0, s, a);
        case kThin2: return launch<thin_kernel<2>>(thin, 64 * kThinWaves, 0, s, a);
        case kTiles64: return run_matmul<Shape64>(a, s);
        case kTiles128: return run_matmul<Shape128>(a, s);
        default: return run_matmul<Shape256>(a, s);
    }
}

}  // namespace fpk
