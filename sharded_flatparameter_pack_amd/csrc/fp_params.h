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

// Tile `index` of tensor `tensor`: what one wave works on.
struct ParamTile {
    int32_t tensor;
    int32_t index;
};

// A tile: 64 lanes x kParamQuads quads.
constexpr int kParamQuads = 2;
constexpr int64_t kParamTile = 256 * kParamQuads;
inline int64_t param_tiles(int64_t numel) { return ceil_div64(numel, kParamTile); }
// LDS that a launch of the step asks for and never touches, so that fewer of
// its workgroups are resident in a CU: with more, HBM serves their streams
// slower.  Measured on MI355X with bf16 gradients and copies:
//   fp32 moments, three per CU against no limit: 2.5M elements 14.1 and 13.2
//     us, 4M 21.0 and 20.5, 8M 38.8 and 38.8, 17M 78.8 and 79.9, 34M 155.3 and
//     158.6, 50M 225.6 and 233.0, 134M 618.5 and 657.9 (two per CU: 666);
//   8-bit moments, five per CU against no limit: 34M 88.0 and 86.0 us, 42M
//     108.7 and 105.8, 46M 120.0 and 119.8, 50M 133.8 and 138.8, 134M 360.8
//     and 376.3 -- their arithmetic wants more waves as long as the memory
//     side keeps up, so their limit starts later.
constexpr unsigned kParamCapLds = 53504u, kMx8CapLds = 32000u;
constexpr int64_t kParamCapTiles = 16000000 / kParamTile, kMx8CapTiles = 46000000 / kParamTile;
inline unsigned params_step_lds(int64_t tiles, bool mx8) {
    if (!mx8) return tiles >= kParamCapTiles ? kParamCapLds : 0u;
    return tiles >= kMx8CapTiles ? kMx8CapLds : 0u;
}
// Workgroups of the norm, a partial sum each: at most as many as are resident
// together (8 per CU).
constexpr int64_t kNormGroups = 2048;
inline int64_t params_norm_groups(int64_t tiles) {
    const int64_t g = ceil_div64(tiles, kWaves);
    return g < 1 ? 1 : g < kNormGroups ? g : kNormGroups;
}
// Workspace of the norm: the counts of finished workgroups, each in a line of
// its own, then the partial sums.
constexpr int64_t kNormHeader = 4 * kLineWords * (kSyncGroups + 1);

// The coefficients of a weight's change in fp32, from AdamCoef's.
struct WeightCoef {
    float step_size;
    float inv_sqrt_bias2;
    float eps;     // at least the smallest normal number, so that no denominator is 0
    float decay;   // lr * weight_decay
};

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
    WeightCoef w[FP_MAX_GROUPS];  // of the step with 8-bit moments
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
hipError_t launch_params_step(const ParamsArgs& a, int grad_dtype, bool mx8, hipStream_t s);
hipError_t launch_params_norm(const ParamsNormArgs& a, int grad_dtype, hipStream_t s);
hipError_t launch_mx8(const MxArgs& a, bool quantize, bool root, hipStream_t s);

}  // namespace fpk
