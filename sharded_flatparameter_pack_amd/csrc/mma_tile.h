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
// What bounds it: the matrix cores' clock under load, with LDS close behind.  A
// 256 x 256 tile on 8 waves of 128 x 64 reads 192 KiB of fragments per step and
// takes 64 KiB in, at 128 bytes per clock as long as its 512 fp16 instructions;
// smaller wave tiles read more for the same work.  Measured on MI355X, fp16 at
// 4096^3 without an epilogue: 101 us (1.36 PFLOP/s; the same tiles with waves of
// 128 x 128 took 169, one wave per SIMD hiding nothing, 128-wide tiles of 64 x 64
// waves 145, 64-wide ones 275).  MXFP4 at 4096^2 x 16384: 107 to 120 us (4.6 to
// 5.1 PFLOP/s).  Swizzles that spread a fragment's rows over all banks or half of
// them, and 32 x 32 instructions, make no difference.
//
// The loop: stages in LDS, filled by loads that go to LDS directly, and two sets
// of fragments in registers.  While the first half's products run, the second
// half's fragments are read; then, behind the step's one barrier, the stage just
// read is refilled for a later step and the next step's first fragments are read
// under the second half's products.  Read as they are needed
// instead, the same tiles take 121 us.
#pragma once

#include <atomic>
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

// Loads kBytes (16 or 4) per lane into LDS, the wave's one behind the other from
// `to` on; base, `to` and soffset are the same in all lanes.  kWritten: as written
// out here, for loops with transposing reads of LDS, before each of which the
// compiler waits for all the loads that it knows of (a 1400 x 64 matrix's A: 16
// us, without 10).  It counts neither such loads nor waits for them; the loop
// does, for both (wait_loads).  M0 is LDS's base and needs a wait state behind its
// write.
template <bool kWritten, int kBytes>
__device__ __forceinline__ void load_lds(const void* base, const char* to, int voffset, int soffset) {
    if constexpr (kWritten) {
        const uint64_t p = (uint64_t)base;
        const i32x4_t buffer = {__builtin_amdgcn_readfirstlane((int)(uint32_t)p),
                                __builtin_amdgcn_readfirstlane((int)(uint32_t)(p >> 32) & 0xFFFF), -1, 0x00020000};
        const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(FP_LDS const char*)to);
        static_assert(kBytes == 16, "rows and columns of fp16");
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                     :: "s"(at), "v"(voffset), "s"(buffer), "s"(__builtin_amdgcn_readfirstlane(soffset)) : "memory", "m0");
    } else {
        const __amdgpu_buffer_rsrc_t buffer = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, -1, 0x00020000);
        if constexpr (kBytes == 16) __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer, (FP_LDS void*)to, 16, voffset, soffset, 0, 0);
        else __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer, (FP_LDS void*)to, 4, voffset, soffset, 0, 0);
    }
}

// kBM x kBN of the output per workgroup, kWM x kWN of it per wave; a power of
// two of stages.
template <int kBM_, int kBN_, int kWM_, int kWN_, int kStages_ = 2>
struct TileShape {
    static constexpr int kBM = kBM_, kBN = kBN_, kWM = kWM_, kWN = kWN_;
    static constexpr int kRows = kBM / kWM, kCols = kBN / kWN;  // of waves
    static constexpr int kWavesWg = kRows * kCols, kThreadsWg = 64 * kWavesWg;
    // Waves per SIMD that registers are kept free for: so many as are resident
    // with the tile's LDS.  Said to the compiler, it holds everything in plain
    // registers; unsaid, it moved 88 in and out of the accumulation ones per step
    // of a 128-wide tile.
    static constexpr int kWavesSimd = kBM < 128 ? 4 : kWavesWg > 8 ? kWavesWg / 4 : 2;
    static constexpr int kFM = kWM / 16, kFN = kWN / 16;        // 16x16 fragments of a wave
    static constexpr int kStage = (kBM + kBN) * kStepBytes;
    static constexpr int kScaleStage = (kBM + kBN) * 8;
    static constexpr int kStages = kStages_;
    static constexpr int kLds = kStages * kStage;
    static constexpr int kLdsFp4 = kLds + kStages * kScaleStage;
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
    static __device__ __forceinline__ int swizzle(int k4, int k16) {
        if constexpr ((kB & (kB - 1)) == 0) return (k4 | k16 << 2) & (kB / 16 - 1);
        else return (k4 >> 1) ^ k16;  // rows of an odd number of 128 bytes: k4's lowest bit is in the address already
    }

    template <bool kWritten>
    __device__ __forceinline__ void load(char* stage, int wave, int step) const {
        const char* from = kColumns ? base + (int64_t)step * kStepF16 * pitch : base;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            load_lds<kWritten, 16>(from, stage + (i * S::kWavesWg + wave) * 1024, voffset[i], kColumns ? 0 : step * kStepBytes);
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
        constexpr bool kWritten = kLeft == kColumnsF16 || kRight == kColumnsF16;
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
            char* to = lds + k % S::kStages * S::kStage;
            l.template load<kWritten>(to, wave, step);
            r.template load<kWritten>(to + S::kBM * kStepBytes, wave, step);
            if constexpr (kFp4) {
#pragma unroll
                for (int i = 0; i < kSLoads; ++i) {
                    const int dword = i * S::kThreadsWg + wave * 64;
                    const uint8_t* from = dword / 2 >= S::kBM ? right.scales : left.scales;
                    load_lds<false, 4>(from, scales + k % S::kStages * S::kScaleStage + dword * 4, soffset[i], step * 8);
                }
            }
        };
        auto read = [&](int k, auto half, Frags& f) {
            const char* from = lds + k % S::kStages * S::kStage;
            r.template read<decltype(half)::value>(from + S::kBM * kStepBytes, f.b);
            l.template read<decltype(half)::value>(from, f.a);
        };
        auto read_scales = [&](int k, Scales& s) {
            if constexpr (kFp4) {
                const char* from = scales + k % S::kStages * S::kScaleStage;
                auto two = [&](int at) { return *(const uint16_t*)(from + at) | (uint32_t) * (const uint16_t*)(from + at + 128) << 16; };
#pragma unroll
                for (int n = 0; n < S::kFN; n += 2) s.b[n / 2] = two(sb + n * 128);
#pragma unroll
                for (int m = 0; m < S::kFM; m += 2) s.a[m / 2] = two(sa + m * 128);
            }
        };
        const std::integral_constant<int, 0> first{};
        const std::integral_constant<int, 1> second{};

        // Loads of a wave per stage: a stage is there once no more than those of
        // the stages behind it are on their way (they end in order).
        constexpr int kPerStage = S::kStage / 1024 / S::kWavesWg + (kFp4 ? kSLoads : 0);
        Frags f0, f1;
        Scales s0, s1;
#pragma unroll
        for (int k = 0; k < S::kStages; ++k) load(k);
        wait_loads<(S::kStages - 1) * kPerStage>();
        barrier_lds();
        read(0, first, f0);
        read_scales(0, s0);
        for (int k = 0; k < steps; ++k) {
            read(k, second, f1);
            multiply<kFp4, 0>(f0, s0);
            interleave<kLeft, kRight>();
            wait_loads<(S::kStages - 2) * kPerStage>();
            barrier_lds();  // the next step's stage is there, and this one is read to its end
            load(k + S::kStages);
            read(k + 1, first, f0);
            read_scales(k + 1, s1);
            multiply<kFp4, 1>(f1, s0);
            interleave<kLeft, kRight>();
            if constexpr (kFp4) s0 = s1;
        }
        wait_loads<0>();
        barrier_lds();
    }

    // The column that a lane has in each(): the first of its kVec.
    template <int kVec>
    static __device__ __forceinline__ int each_col() { return (int)threadIdx.x % (S::kBN / kVec) * kVec; }

    // Walks the tile along its rows, through LDS (the lanes' own fragments are
    // 16 rows of 16 bytes): body(row, col, v, f) with kVec (8 or 4) neighbouring
    // columns from each_col() on, a row's neighbours in neighbouring lanes: 8 for
    // values that are 16 bits in memory, 4 for 32, so that a wave's access is one
    // run.  f is what fetch(row, col) gave: it is called one pass of kPer fragments
    // ahead, so that what the lane reads from memory is there when it is needed
    // (without, the tile of a 1024-wide product waited 25 us for its 16 reads, one
    // by one).  kTurned: also turned(row, col, v, f) with 8 neighbouring rows from
    // `row` on and f = fetch_turned(row, col).
    // fetch_early: the same for the whole tile, for what is fetched before the
    // product; body gets it as one more argument.
    template <int kPer, int kVec, class L>
    static __device__ __forceinline__ auto fetch_early(L fetch) {
        constexpr int kPassRows = S::kRows * kPer * 16, kAcross = S::kBN / kVec;
        constexpr int kTimes = kPassRows * kAcross / S::kThreadsWg;
        struct All {
            decltype(fetch(0, 0)) f[S::kFM / kPer][kTimes];
        } all;
#pragma unroll
        for (int p = 0; p < S::kFM; p += kPer)
#pragma unroll
            for (int t = 0; t < kTimes; ++t) {
                const int i = (int)threadIdx.x / kAcross + t * (S::kThreadsWg / kAcross);
                all.f[p / kPer][t] = fetch(i / (kPer * 16) * S::kWM + p * 16 + i % (kPer * 16), each_col<kVec>());
            }
        return all;
    }
    struct Nothing {};
    static __device__ __forceinline__ Nothing nothing(int, int) { return {}; }

    template <int kPer, int kVec, bool kTurned, class L, class F, class M, class G, class E = Nothing>
    __device__ __forceinline__ void each(char* lds, L fetch, F body, M fetch_turned, G turned, E&& early = E{}) {
        constexpr bool kEarly = !std::is_same<std::decay_t<E>, Nothing>::value;
        constexpr int kPitch = S::kBN + 4;              // floats
        constexpr int kPassRows = S::kRows * kPer * 16;
        constexpr int kAcross = S::kBN / kVec, kDown = kPassRows / 8;
        constexpr int kTimes = kPassRows * kAcross / S::kThreadsWg;
        constexpr int kTimesTurned = kTurned ? kPassRows * S::kBN / 8 / S::kThreadsWg : 1;
        static_assert(S::kFM % kPer == 0 && kTimes >= 1 && kTimes * S::kThreadsWg == kPassRows * kAcross, "whole passes");
        static_assert(S::kThreadsWg % kAcross == 0 && S::kThreadsWg % kDown == 0, "whole rows");
        static_assert(kPassRows * kPitch * 4 <= S::kLds, "a pass fits into the stages");
        float* to = reinterpret_cast<float*>(lds);
        const int c = each_col<kVec>(), r = (int)threadIdx.x / kAcross;
        const int tr = (int)threadIdx.x % kDown * 8, tc = (int)threadIdx.x / kDown;
        auto tile_row = [&](int p, int i) { return i / (kPer * 16) * S::kWM + p * 16 + i % (kPer * 16); };
        decltype(fetch(0, 0)) f[kTimes], ahead[kTimes];
        decltype(fetch_turned(0, 0)) ft[kTimesTurned], ahead_t[kTimesTurned];
        auto fetch_pass = [&](int p) {
#pragma unroll
            for (int t = 0; t < kTimes; ++t) ahead[t] = fetch(tile_row(p, r + t * (S::kThreadsWg / kAcross)), c);
            if constexpr (kTurned) {
#pragma unroll
                for (int t = 0; t < kTimesTurned; ++t)
                    ahead_t[t] = fetch_turned(tile_row(p, tr), tc + t * (S::kThreadsWg / kDown));
            }
        };
        fetch_pass(0);
#pragma unroll
        for (int p = 0; p < S::kFM; p += kPer) {
            if (p > 0) barrier_lds();
#pragma unroll
            for (int m = 0; m < kPer; ++m)
#pragma unroll
                for (int n = 0; n < S::kFN; ++n)
                    *(f32x4_t*)(to + (wave / S::kCols * kPer * 16 + m * 16 + (lane & 15)) * kPitch + col0() + 16 * n) = acc[p + m][n];
#pragma unroll
            for (int t = 0; t < kTimes; ++t) f[t] = ahead[t];
            if constexpr (kTurned) {
#pragma unroll
                for (int t = 0; t < kTimesTurned; ++t) ft[t] = ahead_t[t];
            }
            if (p + kPer < S::kFM) fetch_pass(p + kPer);
            barrier_lds();
#pragma unroll
            for (int t = 0; t < kTimes; ++t) {
                const int i = r + t * (S::kThreadsWg / kAcross);
                float v[kVec];
#pragma unroll
                for (int q = 0; q < kVec; q += 4) {
                    const f32x4_t x = *(const f32x4_t*)(to + i * kPitch + c + q);
                    v[q] = x.x; v[q + 1] = x.y; v[q + 2] = x.z; v[q + 3] = x.w;
                }
                if constexpr (kEarly) body(tile_row(p, i), c, v, f[t], early.f[p / kPer][t]);
                else body(tile_row(p, i), c, v, f[t]);
            }
            if constexpr (kTurned) {
#pragma unroll
                for (int t = 0; t < kTimesTurned; ++t) {
                    const int i = tc + t * (S::kThreadsWg / kDown);
                    float v[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = to[(tr + k) * kPitch + i];
                    turned(tile_row(p, tr), i, v, ft[t]);
                }
            }
        }
    }
    template <int kPer, int kVec, class L, class F, class E = Nothing>
    __device__ __forceinline__ void each(char* lds, L fetch, F body, E&& early = E{}) {
        each<kPer, kVec, false>(lds, fetch, body, nothing, 0, early);
    }

    // Waits until at most kN of the wave's memory accesses are on their way.
    template <int kN>
    static __device__ __forceinline__ void wait_loads() {
        static_assert(kN >= 0 && kN < 64, "six bits");
        __builtin_amdgcn_s_waitcnt((kN & 15) | (kN >> 4) << 14 | 7 << 4 | 15 << 8);  // the other counters: no wait
    }

    // A barrier for what was written to LDS: loads from memory stay in flight.
    static __device__ __forceinline__ void barrier_lds() {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    }
};

template <int kLeft, int kRight, class S>
__device__ __forceinline__ void run_tile(TileProduct<S>& tile, const Operand& left, const Operand& right, int steps, char* lds) {
    tile.template run<kLeft, kRight>(left, right, steps, lds);
}

constexpr unsigned kMaxLds = (160u << 10) - 512;  // a workgroup's, without what a kernel declares itself

// Launches a kernel.  Beyond 64 KiB, LDS is asked for once per kernel and device.
template <auto kKernel, class... Args>
hipError_t launch(unsigned groups, int threads, unsigned lds, hipStream_t s, const Args&... args) {
    if (lds > 65536u) {
        static std::atomic<uint64_t> asked{0};
        int device = 0;
        hipError_t e = hipGetDevice(&device);
        if (e != hipSuccess) return e;
        const uint64_t bit = 1ull << (device & 63);
        if (!(asked.load() & bit)) {
            e = hipFuncSetAttribute(reinterpret_cast<const void*>(kKernel), hipFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxLds);
            if (e != hipSuccess) return e;
            asked.fetch_or(bit);
        }
    }
    kKernel<<<groups, threads, lds, s>>>(args...);
    return hipGetLastError();
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
