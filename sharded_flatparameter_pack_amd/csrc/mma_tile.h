// mma_tile.h -- one workgroup's tile of a matrix product on the matrix cores,
//   out[i][j] = sum over k of left(i, k) right(j, k),
// with operands in fp16 that lie row by row (k along a row) or column by
// column (k from row to row), and in MXFP4 row by row.
//
// A 16x16 instruction takes 16 bytes per lane of each operand: 8 fp16 of
// K = 32, or 32 e2m1 codes of K = 128, which is one MXFP4 block with one scale.
// So one loop serves all: it walks K in steps of 128 bytes per row (64 fp16,
// 256 codes), each in two halves, of one instruction's K.  Which k an operand's
// lane holds is free as long as both agree: lane group g = lane / 16 has word
// 2 g + h (16 bytes) of the step's 128 in half h.
//
// What bounds it: LDS.  A 256 x 256 tile on 8 waves of 128 x 64 reads 192 KiB
// of fragments per step and takes 64 KiB in, at 128 bytes per clock as long as
// its 512 fp16 instructions; smaller wave tiles read more for the same work.
// Measured on MI355X, fp16 at 4096^3: 128 x 64 waves 109 us (1.26 PFLOP/s),
// 128 x 128 on 4 waves 169 (one wave per SIMD hides nothing), a 128-wide
// tile on 4 waves of 64 x 64 145, a 64-wide one 275.  MXFP4 at 4096^2 x 16384
// (scales from LDS): 125 us (4.4 PFLOP/s).
//
// The loop: two stages in LDS, filled by loads that go to LDS directly, and two
// sets of fragments in registers.  While the first half's products run, the
// second half's fragments are read; then, behind the step's one barrier, the
// stage just read is refilled for the step after next and the next step's first
// fragments are read under the second half's products.  Read as they are needed
// instead, the same tiles take 121 and 250 us.
#pragma once

#include <type_traits>

#include "fp_device.h"

namespace fpk {
namespace {

#define FP_LDS __attribute__((address_space(3)))

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

constexpr int kStepBytes = 128;  // of a row, per step along K
constexpr int kStepF16 = 64;

// kBM x kBN of the output per workgroup, kWM x kWN of it per wave.
template <int kBM_, int kBN_, int kWM_, int kWN_>
struct TileShape {
    static constexpr int kBM = kBM_, kBN = kBN_, kWM = kWM_, kWN = kWN_;
    static constexpr int kRows = kBM / kWM, kCols = kBN / kWN;  // of waves
    static constexpr int kWavesWg = kRows * kCols, kThreadsWg = 64 * kWavesWg;
    static constexpr int kFM = kWM / 16, kFN = kWN / 16;        // 16x16 fragments of a wave
    static constexpr int kStage = (kBM + kBN) * kStepBytes;
    static constexpr int kScaleStage = (kBM + kBN) * 8;
    static constexpr int kLds = 2 * kStage;
    static constexpr int kLdsFp4 = kLds + 2 * kScaleStage;
};

// How an operand lies in memory.
enum { kRowsF16 = 0, kColumnsF16 = 1, kRowsFp4 = 2 };

// kRows*: `base` is the tile's first row.  kColumns*: its first column in the
// first row.  `count` rows (columns) of the tile exist, at least 1; those behind
// them are read as the last ones, and what they give is not stored.  Columns
// come in multiples of 8.
struct Operand {
    const void* base;
    int64_t pitch;           // bytes
    int count;
    const uint8_t* scales;   // MXFP4: of the first row, pitch / 16 bytes a row
};

// One operand's part of a stage: its loads, and the fragments of the wave.
//
// A load writes its 64 lanes' 16-byte words one behind the other.  Where a word
// goes is therefore chosen by the address that a lane loads from, and words are
// placed so that those one fragment read covers at a time sit in different
// banks.  Rows: 128 bytes, word w of row r in place w ^ (r % 8).  Columns: 64
// rows (k) of kB elements, the 32-byte chunk c of row k in place
// c ^ (k % 4 + 4 (k / 16)); four lanes take a chunk's 8 bytes each, and the
// transposing read gives lane i the chunk's column i.
template <class S, int kKind, int kB, int kW, int kF>
struct Side {
    static constexpr int kLoads = kB / (8 * S::kWavesWg);  // per wave and step
    static_assert(kB % (8 * S::kWavesWg) == 0, "whole loads per wave");
    static constexpr bool kColumns = kKind == kColumnsF16;

    const char* base;
    int64_t pitch;
    int voffset[kLoads];
    int at[kColumns ? kF : 2];  // of the fragments: rows per half, columns per fragment

    // wave0: first row (column) of the wave in the tile.
    __device__ __forceinline__ Side(const Operand& o, int wave, int lane, int wave0) {
        base = static_cast<const char*>(o.base);
        pitch = o.pitch;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int word = (i * S::kWavesWg + wave) * 64 + lane;
            if constexpr (kColumns) {
                const int k = word / (kB / 8), place = word % (kB / 8);
                const int from = place ^ (swizzle(k & 3, k >> 4) << 1);
                voffset[i] = k * (int)pitch + 16 * (from * 8 < o.count ? from : o.count / 8 - 1);
            } else {
                const int r = word >> 3;
                voffset[i] = (r < o.count ? r : o.count - 1) * (int)pitch + (((lane & 7) ^ (r & 7)) << 4);
            }
        }
        const int g = lane >> 4, j = lane & 15;
        if constexpr (kColumns) {
#pragma unroll
            for (int f = 0; f < kF; ++f)
                at[f] = (16 * g + (j >> 2)) * (2 * kB) + (((wave0 / 16 + f) ^ swizzle(j >> 2, g)) << 5) + (j & 3) * 8;
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) at[h] = (wave0 + j) * kStepBytes + (((2 * g + h) ^ (j & 7)) << 4);
        }
    }
    static __device__ __forceinline__ int swizzle(int k4, int k16) { return (k4 | k16 << 2) & (kB / 16 - 1); }

    __device__ __forceinline__ void load(char* stage, int wave, int step) const {
        const char* from = kColumns ? base + (int64_t)step * kStepF16 * pitch : base;
        const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(from), 0, -1, 0x00020000);
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (FP_LDS void*)(stage + (i * S::kWavesWg + wave) * 1024), 16,
                                                     voffset[i], kColumns ? 0 : step * kStepBytes, 0, 0);
    }
    template <int kH>
    __device__ __forceinline__ void read(const char* stage, i32x4_t (&f)[kF]) const {
#pragma unroll
        for (int n = 0; n < kF; ++n) {
            if constexpr (kColumns) {
                typedef int i32x2_t __attribute__((ext_vector_type(2)));
                const char* p = stage + at[n] + kH * 8 * (2 * kB);
                const i32x2_t lo = __builtin_bit_cast(i32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((FP_LDS s16x4_t*)p));
                const i32x2_t hi =
                    __builtin_bit_cast(i32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((FP_LDS s16x4_t*)(p + 4 * (2 * kB))));
                f[n] = i32x4_t{lo.x, lo.y, hi.x, hi.y};
            } else {
                f[n] = *(const i32x4_t*)(stage + at[kH] + n * 16 * kStepBytes);
            }
        }
    }
};

// The tile's sums, spread over the workgroup.  A lane's acc[fm][fn] holds row
// row0() + 16 fm of the tile and its columns col0() + 16 fn + {0, 1, 2, 3}.
template <class S>
struct TileProduct {
    f32x4_t acc[S::kFM][S::kFN];
    int wave, lane;

    __device__ __forceinline__ TileProduct() {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    }
    __device__ __forceinline__ int row0() const { return wave / S::kCols * S::kWM + (lane & 15); }
    __device__ __forceinline__ int col0() const { return wave % S::kCols * S::kWN + (lane >> 4) * 4; }

    struct Frags {
        i32x4_t a[S::kFM], b[S::kFN];
    };
    // MXFP4 scales of a step: per fragment the lane's two bytes (one per half), two fragments in a register.
    struct Scales {
        uint32_t a[(S::kFM + 1) / 2], b[(S::kFN + 1) / 2];
    };

    template <bool kFp4, int kH>
    __device__ __forceinline__ void multiply(const Frags& f, const Scales& s) {
#pragma unroll
        for (int m = 0; m < S::kFM; ++m)
#pragma unroll
            for (int n = 0; n < S::kFN; ++n) {
                if constexpr (kFp4) {
                    const i32x8_t x = {f.b[n].x, f.b[n].y, f.b[n].z, f.b[n].w, 0, 0, 0, 0};
                    const i32x8_t y = {f.a[m].x, f.a[m].y, f.a[m].z, f.a[m].w, 0, 0, 0, 0};
                    const int sx = (int)s.b[n / 2], sy = (int)s.a[m / 2];
#define FP_MFMA(OX, OY) \
    acc[m][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc[m][n], 4, 4, OX + kH, sx, OY + kH, sy)
                    if (n & 1) {
                        if (m & 1) FP_MFMA(2, 2);
                        else FP_MFMA(2, 0);
                    } else {
                        if (m & 1) FP_MFMA(0, 2);
                        else FP_MFMA(0, 0);
                    }
#undef FP_MFMA
                } else {
                    acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, f.b[n]),
                                                                       __builtin_bit_cast(f16x8_t, f.a[m]), acc[m][n], 0, 0, 0);
                }
            }
    }

    // Asks the scheduler for fragment reads spread among the products.
    template <int kLeft, int kRight>
    static __device__ __forceinline__ void interleave() {
        constexpr int kReads = S::kFM * (kLeft == kColumnsF16 ? 2 : 1) + S::kFN * (kRight == kColumnsF16 ? 2 : 1);
        constexpr int kPer = S::kFM * S::kFN / kReads > 0 ? S::kFM * S::kFN / kReads : 1;
#pragma unroll
        for (int i = 0; i < kReads; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x100 /* LDS reads */, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008 /* products */, kPer, 0);
        }
    }

    // lds: S::kLds bytes (MXFP4: kLdsFp4), free again afterwards.  steps >= 1.
    template <int kLeft, int kRight>
    __device__ __forceinline__ void run(const Operand& left, const Operand& right, int steps, char* lds) {
        constexpr bool kFp4 = kLeft == kRowsFp4;
        static_assert(kFp4 == (kRight == kRowsFp4), "both operands in MXFP4, or none");
        const int row0 = wave / S::kCols * S::kWM, col0 = wave % S::kCols * S::kWN;
        const Side<S, kLeft, S::kBM, S::kWM, S::kFM> l(left, wave, lane, row0);
        const Side<S, kRight, S::kBN, S::kWN, S::kFN> r(right, wave, lane, col0);
#pragma unroll
        for (int m = 0; m < S::kFM; ++m)
#pragma unroll
            for (int n = 0; n < S::kFN; ++n) acc[m][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};

        // MXFP4 scales: 8 bytes of each row per step, loaded as dwords.
        constexpr int kSLoads = kFp4 ? (S::kBM + S::kBN) * 2 / S::kThreadsWg : 1;
        int soffset[kSLoads];
        if constexpr (kFp4) {
#pragma unroll
            for (int i = 0; i < kSLoads; ++i) {
                const int at = (i * S::kThreadsWg + (int)threadIdx.x) >> 1;
                const bool other = at >= S::kBM;
                const int row = other ? at - S::kBM : at, count = other ? right.count : left.count;
                soffset[i] = (row < count ? row : count - 1) * (int)(left.pitch >> 4) + (lane & 1) * 4;
            }
        }
        char* const scales = lds + S::kLds;
        const int sa = (row0 + (lane & 15)) * 8 + (lane >> 4) * 2, sb = (S::kBM + col0 + (lane & 15)) * 8 + (lane >> 4) * 2;

        auto load = [&](int k) {  // past the end the last step again: nothing reads it
            const int step = k < steps ? k : steps - 1;
            char* to = lds + (k & 1) * S::kStage;
            l.load(to, wave, step);
            r.load(to + S::kBM * kStepBytes, wave, step);
            if constexpr (kFp4) {
#pragma unroll
                for (int i = 0; i < kSLoads; ++i) {
                    const int dword = i * S::kThreadsWg + wave * 64;
                    const uint8_t* from = dword / 2 >= S::kBM ? right.scales : left.scales;
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(
                        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(from), 0, -1, 0x00020000),
                        (FP_LDS void*)(scales + (k & 1) * S::kScaleStage + dword * 4), 4, soffset[i], step * 8, 0, 0);
                }
            }
        };
        auto read = [&](int k, auto half, Frags& f) {
            const char* from = lds + (k & 1) * S::kStage;
            r.template read<decltype(half)::value>(from + S::kBM * kStepBytes, f.b);
            l.template read<decltype(half)::value>(from, f.a);
        };
        auto read_scales = [&](int k, Scales& s) {
            if constexpr (kFp4) {
                const char* from = scales + (k & 1) * S::kScaleStage;
                auto two = [&](int at) { return *(const uint16_t*)(from + at) | (uint32_t) * (const uint16_t*)(from + at + 128) << 16; };
#pragma unroll
                for (int n = 0; n < S::kFN; n += 2) s.b[n / 2] = two(sb + n * 128);
#pragma unroll
                for (int m = 0; m < S::kFM; m += 2) s.a[m / 2] = two(sa + m * 128);
            }
        };
        const std::integral_constant<int, 0> first{};
        const std::integral_constant<int, 1> second{};

        Frags f0, f1;
        Scales s0, s1;
        load(0);
        __syncthreads();
        load(1);
        read(0, first, f0);
        read_scales(0, s0);
        for (int k = 0; k < steps; ++k) {
            read(k, second, f1);
            multiply<kFp4, 0>(f0, s0);
            interleave<kLeft, kRight>();
            __syncthreads();  // the next step's stage is there, and this one is read to its end
            load(k + 2);
            read(k + 1, first, f0);
            read_scales(k + 1, s1);
            multiply<kFp4, 1>(f1, s0);
            interleave<kLeft, kRight>();
            if constexpr (kFp4) s0 = s1;
        }
        __syncthreads();
    }

    // Walks the tile along its rows: body(row, col, v) with 8 neighbouring
    // columns from `col` on, a row's neighbours in neighbouring lanes, through
    // LDS (the lanes' own fragments are 16 rows of 8 or 16 bytes).  kTurned
    // also calls turned(row, col, v) with 8 neighbouring rows from `row` on.
    // The values are read from registers a few fragments at a time, 64 rows of
    // the tile for a 256-wide one.
    template <bool kTurned, class F, class G>
    __device__ __forceinline__ void each(char* lds, F body, G turned) {
        constexpr int kPer = S::kFM < 2 ? S::kFM : 2;   // fragments along the rows, per pass
        constexpr int kPitch = S::kBN + 4;              // floats
        constexpr int kPassRows = S::kRows * kPer * 16;
        static_assert(kPassRows * kPitch * 4 <= S::kLds, "a pass fits into the stages");
        float* to = reinterpret_cast<float*>(lds);
#pragma unroll
        for (int p = 0; p < S::kFM; p += kPer) {
            if (p > 0) __syncthreads();
#pragma unroll
            for (int m = 0; m < kPer; ++m)
#pragma unroll
                for (int n = 0; n < S::kFN; ++n)
                    *(f32x4_t*)(to + (wave / S::kCols * kPer * 16 + m * 16 + (lane & 15)) * kPitch + col0() + 16 * n) = acc[p + m][n];
            __syncthreads();
            auto tile_row = [&](int r) { return r / (kPer * 16) * S::kWM + p * 16 + r % (kPer * 16); };
#pragma unroll 1
            for (int i = threadIdx.x; i < kPassRows * S::kBN / 8; i += S::kThreadsWg) {
                const int r = i / (S::kBN / 8), c = i % (S::kBN / 8) * 8;
                const f32x4_t a = *(const f32x4_t*)(to + r * kPitch + c), b = *(const f32x4_t*)(to + r * kPitch + c + 4);
                const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                body(tile_row(r), c, v);
            }
            if constexpr (kTurned) {
#pragma unroll 1
                for (int i = threadIdx.x; i < kPassRows * S::kBN / 8; i += S::kThreadsWg) {
                    const int r = i % (kPassRows / 8) * 8, c = i / (kPassRows / 8);
                    float v[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = to[(r + k) * kPitch + c];
                    turned(tile_row(r), c, v);
                }
            }
        }
    }
    template <class F>
    __device__ __forceinline__ void each(char* lds, F body) {
        each<false>(lds, body, 0);
    }
};

template <int kLeft, int kRight, class S>
__device__ __forceinline__ void run_tile(TileProduct<S>& tile, const Operand& left, const Operand& right, int steps, char* lds) {
    tile.template run<kLeft, kRight>(left, right, steps, lds);
}

// Tile number of a workgroup: the hardware deals workgroups out to the 8 dies
// in turn, each with an L2 of its own, so that a die's share of the numbers is
// made one run of neighbours, which read the same rows.
__device__ __forceinline__ int die_tile(int workgroup, int n) {
    const int per = n >> 3, more = n & 7, die = workgroup & 7;
    return die * per + (die < more ? die : more) + (workgroup >> 3);
}

}  // namespace
}  // namespace fpk
