// mma_tile.h -- one workgroup's tile of a product of two row-major operands
// along their rows: out[i][j] = sum over k of left[i][k] right[j][k], on the
// matrix cores, for operands in fp16 and in MXFP4.
//
// Both kinds feed a 16x16 instruction with 16 bytes per lane and operand: 8
// fp16 of K = 32, or 32 e2m1 codes of K = 128, which is one MXFP4 block with
// one scale.  So one loop serves both: it walks K in steps of 128 bytes per
// row (64 fp16, 256 codes).
//
// LDS: two stages of (kBM + kBN) rows of 128 bytes, filled by direct
// global-to-LDS loads of 16 bytes per lane while the other stage is worked
// on, with one barrier per step.  Such a load writes its 64 lanes' words one
// behind the other, 8 rows of 8 words; word w of row r holds the row's word
// w ^ (r % 8), chosen by the address that the lane loads from, so that the 8
// rows a fragment read covers at a time sit in different banks.
#pragma once

#include "fp_device.h"

namespace fpk {
namespace {

#define FP_LDS __attribute__((address_space(3)))

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

constexpr int kStepBytes = 128;  // of a row, per step along K

// kBM x kBN of the output per workgroup, kWM x kWN of it per wave.
template <int kBM_, int kBN_, int kWM_, int kWN_>
struct TileShape {
    static constexpr int kBM = kBM_, kBN = kBN_, kWM = kWM_, kWN = kWN_;
    static constexpr int kRows = kBM / kWM, kCols = kBN / kWN;  // of waves
    static constexpr int kWavesWg = kRows * kCols, kThreadsWg = 64 * kWavesWg;
    static constexpr int kFM = kWM / 16, kFN = kWN / 16;        // 16x16 fragments of a wave
    static constexpr int kStage = (kBM + kBN) * kStepBytes;
    static constexpr int kLds = 2 * kStage;
};

// Rows of one operand: `base` is the tile's first row, `rows` how many of
// them exist (at least 1; those behind are read as the last one, and what
// they give is not stored).
struct Operand {
    const void* base;
    int64_t pitch;           // bytes; a multiple of kStepBytes
    int rows;
    const uint8_t* scales;   // MXFP4: of the first row, pitch / 16 bytes a row
};

// The loads of one operand's rows into a stage.
template <class S, int kB>
struct Loader {
    static constexpr int kLoads = kB / (8 * S::kWavesWg);  // per wave: 8 rows each
    static_assert(kB % (8 * S::kWavesWg) == 0, "whole loads per wave");
    __amdgpu_buffer_rsrc_t rsrc;
    int voffset[kLoads];

    __device__ __forceinline__ Loader(const Operand& o, int wave, int lane) {
        rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(o.base), 0, -1, 0x00020000);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            int row = (i * S::kWavesWg + wave) * 8 + (lane >> 3);
            row = row < o.rows ? row : o.rows - 1;
            voffset[i] = row * (int)o.pitch + (((lane & 7) ^ (lane >> 3)) << 4);
        }
    }
    __device__ __forceinline__ void load(char* stage, int wave, int step) const {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (FP_LDS void*)(stage + (i * S::kWavesWg + wave) * 1024), 16,
                                                     voffset[i], step * kStepBytes, 0, 0);
    }
};

// The tile's sums, spread over the workgroup.  A lane's acc[fm][fn] holds row
// row0() + 16 fm of the tile and its columns col0() + 16 fn + {0, 1, 2, 3}.
template <class S, bool kFp4>
struct TileProduct {
    f32x4_t acc[S::kFM][S::kFN];
    int wave, lane;

    __device__ __forceinline__ int row0() const { return wave / S::kCols * S::kWM + (lane & 15); }
    __device__ __forceinline__ int col0() const { return wave % S::kCols * S::kWN + (lane >> 4) * 4; }

    // lds: S::kLds bytes.  steps >= 1.
    __device__ __forceinline__ void run(const Operand& left, const Operand& right, int steps, char* lds) {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        const Loader<S, S::kBM> ll(left, wave, lane);
        const Loader<S, S::kBN> lr(right, wave, lane);
#pragma unroll
        for (int m = 0; m < S::kFM; ++m)
#pragma unroll
            for (int n = 0; n < S::kFN; ++n) acc[m][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};

        // Fragment reads: in the first half of a step the lane's group g takes
        // word 2 g of its row, in the second word 2 g + 1 (any order serves,
        // as long as both operands have it), so that its two MXFP4 scales
        // are neighbours.
        const int g2 = (lane >> 4) * 2, r8 = lane & 7;
        const int at = (lane & 15) * kStepBytes;
        const int w0 = at + ((g2 ^ r8) << 4), w1 = at + (((g2 + 1) ^ r8) << 4);
        const int lbase = wave / S::kCols * S::kWM * kStepBytes;
        const int rbase = S::kBM * kStepBytes + wave % S::kCols * S::kWN * kStepBytes;

        int ls[S::kFM], rs[S::kFN];  // MXFP4: where the lane's scales are
        uint32_t lb[S::kFM], rb[S::kFN];
        const int spitch = (int)(left.pitch >> 4);
        __amdgpu_buffer_rsrc_t lsr, rsr;
        if constexpr (kFp4) {
            lsr = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(left.scales), 0, -1, 0x00020000);
            rsr = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(right.scales), 0, -1, 0x00020000);
#pragma unroll
            for (int m = 0; m < S::kFM; ++m) {
                const int row = row0() + 16 * m;
                ls[m] = (row < left.rows ? row : left.rows - 1) * spitch + g2;
            }
#pragma unroll
            for (int n = 0; n < S::kFN; ++n) {
                const int row = wave % S::kCols * S::kWN + (lane & 15) + 16 * n;
                rs[n] = (row < right.rows ? row : right.rows - 1) * spitch + g2;
            }
        }

        ll.load(lds, wave, 0);
        lr.load(lds + S::kBM * kStepBytes, wave, 0);
        for (int k = 0; k < steps; ++k) {
            char* here = lds + (k & 1) * S::kStage;
            if constexpr (kFp4) {
#pragma unroll
                for (int m = 0; m < S::kFM; ++m) lb[m] = __builtin_amdgcn_raw_buffer_load_b16(lsr, ls[m], 8 * k, 0);
#pragma unroll
                for (int n = 0; n < S::kFN; ++n) rb[n] = __builtin_amdgcn_raw_buffer_load_b16(rsr, rs[n], 8 * k, 0);
            }
            __syncthreads();  // this step's rows are there, and the other stage is read to its end
            if (k + 1 < steps) {
                char* there = lds + ((k + 1) & 1) * S::kStage;
                ll.load(there, wave, k + 1);
                lr.load(there + S::kBM * kStepBytes, wave, k + 1);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int w = h ? w1 : w0;
                i32x4_t a[S::kFM], b[S::kFN];
#pragma unroll
                for (int m = 0; m < S::kFM; ++m) a[m] = *(const i32x4_t*)(here + lbase + w + m * 16 * kStepBytes);
#pragma unroll
                for (int n = 0; n < S::kFN; ++n) b[n] = *(const i32x4_t*)(here + rbase + w + n * 16 * kStepBytes);
#pragma unroll
                for (int m = 0; m < S::kFM; ++m)
#pragma unroll
                    for (int n = 0; n < S::kFN; ++n) {
                        if constexpr (kFp4) {
                            const i32x8_t x = {b[n].x, b[n].y, b[n].z, b[n].w, 0, 0, 0, 0};
                            const i32x8_t y = {a[m].x, a[m].y, a[m].z, a[m].w, 0, 0, 0, 0};
                            if (h == 0)
                                acc[m][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc[m][n], 4, 4, 0,
                                                                                             (int)rb[n], 0, (int)lb[m]);
                            else
                                acc[m][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc[m][n], 4, 4, 1,
                                                                                             (int)rb[n], 1, (int)lb[m]);
                        } else {
                            acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, b[n]),
                                                                               __builtin_bit_cast(f16x8_t, a[m]),
                                                                               acc[m][n], 0, 0, 0);
                        }
                    }
            }
        }
    }
};

// Tile number of a workgroup: the hardware deals workgroups out to the 8 dies
// in turn, each with an L2 of its own, so that a die's share of the numbers is
// made one run of neighbours, which read the same rows.
__device__ __forceinline__ int die_tile(int workgroup, int n) {
    const int per = n >> 3, more = n & 7, die = workgroup & 7;
    return die * per + (die < more ? die : more) + (workgroup >> 3);
}

}  // namespace
}  // namespace fpk
