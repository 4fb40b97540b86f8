// fp_params.h -- argument blocks and launcher declarations of the step over
// many separate tensors (params_kernels.hip) and of the MXFP8 conversions.
#pragma once

#include "fp_internal.h"

namespace fpk {

// MXFP8: blocks of kMxBlock consecutive elements share one power-of-two scale.
constexpr int kMxBlock = 32;

// One tensor of a plan.  The moments sit in the rank's partition at element
// `offset`, a multiple of kMxBlock, so blocks never cross tensors; the
// gradient pointers have a table of their own, which fp_params_set_grads
// rewrites.
struct ParamRec {
    float* master;    // null in a plan that only takes the norm
    void* copy;       // bf16 / fp16 weights, or null
    int64_t numel;
    int64_t offset;
    int32_t group;    // parameter group
    int32_t pad[7];
};
static_assert(sizeof(ParamRec) == 64, "one 64-byte record per tensor");

// Tile `index` of tensor `tensor`.
struct ParamTile {
    int32_t tensor;
    int32_t index;
};

// A tile: 64 lanes x kParamQuads quads.
constexpr int kParamQuads = 2;
constexpr int64_t kParamTile = 256 * kParamQuads;
inline int64_t param_tiles(int64_t numel) { return ceil_div64(numel, kParamTile); }
// How many of the step's streams are open at a time decides how fast HBM
// serves them: too many, and it slows.  Measured on MI355X with bf16
// gradients and copies, medians in us:
// fp32 moments: a wave takes half a tile (one quad per lane; two measured
//   652 against 616 at 134M elements), and from kParamCapElems on a launch asks
//   for LDS that it never touches, so that three workgroups are resident in a
//   CU.  With that and without: 2M 11.6 and 11.1, 4M 20.6 and 20.8, 17M 77 and
//   79, 50M 224 and 231, 134M 593 and 622, 226M 1004 (6.3 TB/s) and 1058.
constexpr unsigned kParamCapLds = 53504u;
constexpr int64_t kParamCapElems = 4000000;
// 8-bit moments: the vector units are busy most of the kernel's time beside the
//   memory.  A wave takes a tile, whose two quads per lane hide each other's
//   latencies, and below kMx8WholeElems, where waves are few, half of one.  Half
//   and whole, in 12 tensors: 1.6M elements 7.9 and 8.1, 3M 12.8 and 12.2, 4M
//   15.3 and 15.0, 17M 51.6 and 49.2, 42M 118 and 111, 134M 385 and 366, 200M
//   595 and 611, 226M 660 and 660, 450M 1289 and 1342; the 226M of eight
//   matrices and their biases 665 and 622.  In 10 000 tensors, whose last tiles
//   are mostly empty: 1.6M 15.5 and 19.5, 3M 19.4 and 22.7, 10M 37.7 and 38.8,
//   17M 56.5 and 56.0, 42M 125 and 119, 200M 591 and 567.
constexpr int64_t kMx8WholeElems = 3000000;

// Workgroups of the norm, a partial sum each, at most as many as are resident
// together.  Of 512 lanes, 4 per CU: counting them in at the end takes time of
// its own, which 256 lanes and 8 per CU (4M bf16 elements 8.1 against 7.0 us,
// 42M 20.0 and 17.8, the 10k tensors 21.1 and 19.6) have more of, while 1024
// and 2 start a small norm later (100k elements 5.8 against 4.9 us).
constexpr int kNormThreads = 512, kNormWaves = kNormThreads / 64;
constexpr int64_t kNormGroups = 1024;
inline int64_t params_norm_groups(int64_t tiles) {
    const int64_t g = ceil_div64(tiles, kNormWaves);
    return g < 1 ? 1 : g < kNormGroups ? g : kNormGroups;
}
// Workspace of the norm: the counts of finished workgroups, each in a line of
// its own, then the partial sums.
constexpr int64_t kNormHeader = 4 * kLineWords * (kSyncGroups + 1);

struct ParamsArgs {
    const ParamRec* recs;
    const void* const* grads;
    const ParamTile* tiles;
    int64_t n_tiles;
    void* exp_avg;            // fp32 or e4m3 [partition]
    void* exp_avg_sq;         // fp32 second moment, or e4m3 of its root
    uint8_t* exp_avg_scale;   // e8m0 [partition / kMxBlock]
    uint8_t* root_scale;
    const int32_t* found_inf; // may be null: never skip
    const double* g_coef;     // factor applied to the gradient, may be null (1)
    uint32_t key;             // of the stochastic rounding
    int32_t copy_f16;         // the copies are fp16, else bf16
    AdamCoef c[FP_MAX_GROUPS];
};

struct ParamsNormArgs {
    const ParamRec* recs;
    const void* const* grads;
    const ParamTile* tiles;
    int64_t n_tiles;
    int32_t* found_inf;       // may be null
    double* partials;         // one per workgroup
    uint32_t* done;           // counts of workgroups that have stored theirs; 0 between calls
    double* sq_norm;
};

// Elements of a workgroup of the MXFP8 conversions.
constexpr int kMxQuads = 2;
constexpr int64_t kMxTile = 4 * (int64_t)kThreads * kMxQuads;

struct MxArgs {
    float* x;                 // read by the quantization, written by the other
    uint8_t* codes;
    uint8_t* scales;
    int64_t n;
};

// abi.hip: checks hyperparameters and fills the coefficients of one AdamW step.
fp_status adam_coef(const fp_adamw_hparams* hp, AdamCoef* c);

// Launchers (return the HIP error of the launch); grad_dtype is FP_DTYPE_*.
hipError_t launch_params_step(const ParamsArgs& a, int64_t partition, int grad_dtype, bool mx8, hipStream_t s);
hipError_t launch_params_norm(const ParamsNormArgs& a, int grad_dtype, hipStream_t s);
hipError_t launch_mx8(const MxArgs& a, bool quantize, bool root, hipStream_t s);

}  // namespace fpk
