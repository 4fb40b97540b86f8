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

// Code of one value, rounded stochastically: with y = |x| / scale in [0, 6] and
// q the distance of the codes' values around y (0.5, 1 or 2), that of
// q floor(y / q + d / 2^16), d in [0, 2^16), in whole numbers.
__device__ __forceinline__ uint32_t mx4_encode_one(float x, float unscale, uint32_t d) {
    const float y = fabsf(x) * unscale;
    const bool two = y >= 2.0f, four = y >= 4.0f;
    const float t = y * (four ? 32768.0f : two ? 65536.0f : 131072.0f);
    const uint32_t u = ((uint32_t)t + d) >> 16;  // exact: y has 24 bits, its last one at 2^-24 of t or cut by the floor
    return (u + (four ? 4u : two ? 2u : 0u)) | (__float_as_uint(x) >> 31 << 3);
}

// 1 / scale, in two factors' range: 2^(127 - byte) for byte <= 254.
__device__ __forceinline__ float unscale_f32(uint32_t byte) {
    return byte == 255u ? 0.0f : __builtin_amdgcn_ldexpf(1.0f, 127 - (int)byte);
}

template <int kDtype>
struct Held {  // what LDS keeps of an element
    typedef uint16_t type;
};
template <>
struct Held<FP_DTYPE_F32> {
    typedef uint32_t type;
};

constexpr int kQTile = 128;

// Elements [col, col + 8) of a row as bits, those past `cols` 0.
template <int kDtype>
__device__ __forceinline__ void ld_bits(const void* x, int64_t at, int have, uint32_t w[8]) {
    if constexpr (kDtype == FP_DTYPE_F32) {
        const float* p = static_cast<const float*>(x) + at;
        if (have >= 8) {
            const uint4 a = ld16u(p), b = ld16u(p + 4);
            w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
            w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
            return;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = k < have ? gptr<uint32_t>((const void*)p)[k] : 0u;
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(x) + at;
        if (have >= 8) {
            const uint4 a = ld16u(p);
            w[0] = a.x & 0xFFFFu; w[1] = a.x >> 16; w[2] = a.y & 0xFFFFu; w[3] = a.y >> 16;
            w[4] = a.z & 0xFFFFu; w[5] = a.z >> 16; w[6] = a.w & 0xFFFFu; w[7] = a.w >> 16;
            return;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = k < have ? (uint32_t)gptr<uint16_t>((const void*)p)[k] : 0u;
    }
}

// A 128 x 128 tile.  Rows' form: four lanes hold a block, eight elements each.
// Columns' form: a lane holds a block, read down a column of the tile in LDS.
template <int kDtype, bool kRows, bool kColumns, bool kRandom>
__global__ __launch_bounds__(256) void quantize_kernel(const Mx4QuantArgs a) {
    typedef typename Held<kDtype>::type held_t;
    __shared__ held_t tile[kColumns ? kQTile : 1][kQTile + 2];
    const unsigned across = kRows ? (unsigned)(a.cp / kQTile) : (unsigned)((a.cols + kQTile - 1) / kQTile);
    const int64_t row0 = (int64_t)(blockIdx.x / across) * kQTile, col0 = (int64_t)(blockIdx.x % across) * kQTile;
    const int c8 = (threadIdx.x & 15) * 8;
    const int64_t left = a.cols - (col0 + c8);
    for (int i = 0; i < 8; ++i) {
        const int lr = (threadIdx.x >> 4) + 16 * i;
        const int64_t row = row0 + lr;
        const int have = row >= a.rows || left <= 0 ? 0 : left < 8 ? (int)left : 8;
        uint32_t w[8];
        ld_bits<kDtype>(a.x, row * a.pitch + col0 + c8, have, w);
        if constexpr (kColumns) {
#pragma unroll
            for (int k = 0; k < 8; ++k) tile[lr][c8 + k] = (held_t)w[k];
        }
        if constexpr (kRows) {
            float f[8];
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                f[k] = to_f32<kDtype>(w[k]);
                const uint32_t m = __float_as_uint(f[k]) & 0x7FFFFFFFu;
                top = top > m ? top : m;
            }
            uint32_t y = (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0xB1 /* quad_perm 1,0,3,2 */, 0xF, 0xF, true);
            top = top > y ? top : y;
            y = (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0x4E /* quad_perm 2,3,0,1 */, 0xF, 0xF, true);
            top = top > y ? top : y;
            const uint32_t byte = mx4_byte<kRandom>(top);
            uint32_t codes = 0;
            if constexpr (kRandom) {
                const float u = unscale_f32(byte);
                const uint32_t e = (uint32_t)(row * a.cols + col0 + c8);
#pragma unroll
                for (int k = 0; k < 8; ++k) codes |= mx4_encode_one(f[k], u, dither(e + k, a.key) >> 16) << (4 * k);
                codes = byte == 255u ? 0u : codes;
            } else {
                codes = mx4_encode(f, byte);
            }
            if (row < a.rows && col0 + c8 < a.cp) {
                gptr<uint32_t>((void*)a.codes)[(row * a.cp + col0 + c8) >> 3] = codes;
                if ((threadIdx.x & 3) == 0) gptr<uint8_t>((void*)a.scales)[(row * a.cp + col0 + c8) >> 5] = (uint8_t)byte;
            }
        }
    }
    if constexpr (kColumns) {
        __syncthreads();
        const int lc = threadIdx.x & 127;
        const int64_t col = col0 + lc;
        if (col >= a.cols) return;
        for (int i = 0; i < 2; ++i) {
            const int lr = ((threadIdx.x >> 7) * 2 + i) * 32;
            float f[32];
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
                f[k] = to_f32<kDtype>(tile[lr + k][lc]);
                const uint32_t m = __float_as_uint(f[k]) & 0x7FFFFFFFu;
                top = top > m ? top : m;
            }
            const uint32_t byte = mx4_byte<kRandom>(top);
            uint32_t codes[4] = {0u, 0u, 0u, 0u};
            if constexpr (kRandom) {
                const float u = unscale_f32(byte);
                uint32_t e = (uint32_t)((row0 + lr) * a.cols + col);
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    codes[k >> 3] |= mx4_encode_one(f[k], u, dither(e, a.key) & 0xFFFFu) << (4 * (k & 7));
                    e += (uint32_t)a.cols;
                }
                if (byte == 255u) codes[0] = codes[1] = codes[2] = codes[3] = 0u;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) codes[k] = mx4_encode(f + 8 * k, byte);
            }
            const int64_t at = col * a.rp + row0 + lr;
            put16(a.codes_t + (at >> 1), make_uint4(codes[0], codes[1], codes[2], codes[3]));
            gptr<uint8_t>((void*)a.scales_t)[at >> 5] = (uint8_t)byte;
        }
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

// Eight values per lane, a row's columns side by side.
template <int kDtype>
__global__ __launch_bounds__(256) void dequantize_kernel(const Mx4DequantArgs a, int lanes) {
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = at / lanes;
    const int64_t col = (at - row * lanes) * 8;
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

// Up to eight neighbouring elements of the output, as bits.
struct Old {
    uint32_t w[8];
};

// The output's old values, where they are added to.
__device__ __forceinline__ Old ld_old(const Mx4MatmulArgs& a, int64_t row, int64_t col) {
    Old o;
#pragma unroll
    for (int k = 0; k < 8; ++k) o.w[k] = 0u;
    if (a.accumulate && row < a.m && col < a.n) {
        const int64_t left = a.n - col, at = row * a.pitch + col;
        const int have = left < 8 ? (int)left : 8;
        if (a.dtype == FP_DTYPE_F32) ld_bits<FP_DTYPE_F32>(a.out, at, have, o.w);
        else ld_bits<FP_DTYPE_BF16>(a.out, at, have, o.w);
    }
    return o;
}

// Stores eight neighbouring elements (row, col ..), those that the output has.
__device__ __forceinline__ void st_out(const Mx4MatmulArgs& a, int64_t row, int64_t col, const float v[8], const Old& o) {
    if (row >= a.m || col >= a.n) return;
    const int64_t left = a.n - col, at = row * a.pitch + col;
    const int have = left < 8 ? (int)left : 8;
    const bool half = a.dtype == FP_DTYPE_F16;
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        f[k] = v[k];
        if (a.accumulate) f[k] += a.dtype == FP_DTYPE_F32 ? __uint_as_float(o.w[k]) : half ? f16_lo(o.w[k]) : bf16_lo(o.w[k]);
    }
    if (a.dtype == FP_DTYPE_F32) {
        float* p = static_cast<float*>(a.out) + at;
        if (have == 8) {
            put16u(p, bits_of(f));
            put16u(p + 4, bits_of(f + 4));
            return;
        }
#pragma unroll
        for (int k = 0; k < 7; ++k)
            if (k < have) gptr<float>((void*)p)[k] = f[k];
        return;
    }
    uint16_t* p = static_cast<uint16_t*>(a.out) + at;
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = half ? f16_pair(f[2 * k], f[2 * k + 1]) : bf16x2(f[2 * k], f[2 * k + 1]);
    if (have == 8) {
        st16h(p, make_uint4(w[0], w[1], w[2], w[3]));
        return;
    }
#pragma unroll
    for (int k = 0; k < 7; ++k)
        if (k < have) gptr<uint16_t>((void*)p)[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
}

template <class S>
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
    tile.template each<S::kFM < 2 ? 1 : 2>(
        lds, [&](int r, int c) { return ld_old(a, i0 + r, j0 + c); },
        [&](int r, int c, const float* v, const Old& o) { st_out(a, i0 + r, j0 + c, v, o); });
}

using Shape256 = TileShape<256, 256, 128, 64>;
using Shape128 = TileShape<128, 128, 64, 64>;
using Shape64 = TileShape<64, 64, 32, 32>;

template <class S>
hipError_t run_matmul(Mx4MatmulArgs a, hipStream_t s) {
    a.tiles_m = (int32_t)ceil_div64(a.m, S::kBM);
    a.tiles_n = (int32_t)ceil_div64(a.n, S::kBN);
    if (S::kLdsFp4 > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(matmul_kernel<S>), hipFuncAttributeMaxDynamicSharedMemorySize, S::kLdsFp4);
        if (e != hipSuccess) return e;
    }
    matmul_kernel<S><<<(unsigned)(a.tiles_m * a.tiles_n), S::kThreadsWg, S::kLdsFp4, s>>>(a);
    return hipGetLastError();
}

// Tiles across and down: the padding of a form that is wanted is written too.
int64_t quant_tiles_x(const Mx4QuantArgs& a) { return ceil_div64(a.codes != nullptr ? a.cp : a.cols, kQTile); }
int64_t quant_tiles_y(const Mx4QuantArgs& a) { return ceil_div64(a.codes_t != nullptr ? a.rp : a.rows, kQTile); }

template <int kDtype, bool kRandom>
hipError_t run_quantize(const Mx4QuantArgs& a, hipStream_t s) {
    const bool rows = a.codes != nullptr, columns = a.codes_t != nullptr;
    const unsigned grid = (unsigned)(quant_tiles_x(a) * quant_tiles_y(a));
    if (rows && columns) quantize_kernel<kDtype, true, true, kRandom><<<grid, 256, 0, s>>>(a);
    else if (rows) quantize_kernel<kDtype, true, false, kRandom><<<grid, 256, 0, s>>>(a);
    else quantize_kernel<kDtype, false, true, kRandom><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

int64_t mx4_quantize_lanes(const Mx4QuantArgs& a) { return quant_tiles_x(a) * quant_tiles_y(a) * 256; }
// Of the 256-wide tiles, which a product with so many lanes is run on.
int64_t mx4_matmul_lanes(const Mx4MatmulArgs& a) { return ceil_div64(a.m, 256) * ceil_div64(a.n, 256) * Shape256::kThreadsWg; }

hipError_t launch_mx4_quantize(const Mx4QuantArgs& a, hipStream_t s) {
#define FP_QUANT(D) (a.stochastic ? run_quantize<D, true>(a, s) : run_quantize<D, false>(a, s))
    return a.dtype == FP_DTYPE_F32 ? FP_QUANT(FP_DTYPE_F32) : a.dtype == FP_DTYPE_BF16 ? FP_QUANT(FP_DTYPE_BF16) : FP_QUANT(FP_DTYPE_F16);
#undef FP_QUANT
}

hipError_t launch_mx4_dequantize(const Mx4DequantArgs& a, hipStream_t s) {
    const int lanes = (int)ceil_div64(a.cols, 8);
    const unsigned grid = (unsigned)ceil_div64(a.rows * lanes, 256);
    if (a.dtype == FP_DTYPE_F32) dequantize_kernel<FP_DTYPE_F32><<<grid, 256, 0, s>>>(a, lanes);
    else if (a.dtype == FP_DTYPE_BF16) dequantize_kernel<FP_DTYPE_BF16><<<grid, 256, 0, s>>>(a, lanes);
    else dequantize_kernel<FP_DTYPE_F16><<<grid, 256, 0, s>>>(a, lanes);
    return hipGetLastError();
}

hipError_t launch_mx4_matmul(const Mx4MatmulArgs& a, hipStream_t s) {
    auto tiles = [&](int64_t side) { return ceil_div64(a.m, side) * ceil_div64(a.n, side); };
    if (tiles(256) >= 160) return run_matmul<Shape256>(a, s);
    if (tiles(128) >= 160) return run_matmul<Shape128>(a, s);
    return run_matmul<Shape64>(a, s);
}

}  // namespace fpk
