// fp_matrix.h -- argument blocks and launcher declarations of the operators on
// matrix parameters: Newton-Schulz orthogonalisation and the step that takes
// it (muon_kernels.hip), MXFP4 quantisation and product (mx4_kernels.hip).
#pragma once

#include "fp_internal.h"

namespace fpk {

// ---------------------------------------------------------------- muon

// One matrix of a plan.  Inside the workspace it is padded with zeros to
// multiples of kPad rows and columns, and held in two parts, X times a power of
// two being h (fp16) + l (bf16).  m: the smaller padded side.  Offsets are bytes
// from the workspace's start.
struct MuonRec {
    float* master;            // null in a plan that only orthogonalises
    void* copy;               // bf16 / fp16 weights, or null
    void* update;             // receives the orthogonalised matrix, or null
    int64_t offset;           // of the momentum, in the partition
    int32_t rows, cols;
    int32_t rp, cp;           // padded
    int32_t group;
    int32_t chunks;           // of the norm's partial sums
    int64_t chunk;            // elements of one
    int64_t h[2], l;          // h has two places: a step of the iteration reads one and writes the other
    int64_t a, b;             // fp16 [m][m], their diagonals zero
    int64_t da, db;           // fp32 [m]: the diagonals
    int64_t part;             // fp64 [chunks + 1]: the norm's partial sums, and 1 / (norm + eps)
    int64_t split;            // fp32 [slices][tiles][kTile64Deep's]: A's sums over slices of n
    int32_t slices, slice_steps;  // 1: none
};

constexpr int kPad = 64;
inline int64_t pad64(int64_t n) { return (n + kPad - 1) / kPad * kPad; }

// Tile (ti, tj) of matrix `mat`; what a tile is depends on the kernel.  mat < 0:
// none, in the tables of the products, which deal each die its own.  slice: of A's
// sums.
struct MatTile {
    int32_t mat, ti, tj, slice;
};

struct MuonGroup {
    double lr, beta, decay;   // decay = 1 - lr * weight_decay
    int32_t nesterov, adjust;
};

// The scales of one step of the iteration: powers of two by which the fp16
// forms are multiplied so that no element passes fp16's range.
struct MuonScale {
    float x, b, x_next;       // X's, B's and the next X's
    float gram;               // what the products of X's fp16 forms become A's by: a / x^2
    float un_x, un_xx, un_a, un_bx;  // 1 / x, 1 / x^2, 1 / a, 1 / (b x)
    int32_t whole;            // B's diagonal multiplies X as it is, not its fp16 form
};

// A whole iteration, for the kernel that runs all of it.
struct MuonSteps {
    int32_t n;
    MuonScale s[FP_MUON_MAX_STEPS];
    float c[FP_MUON_MAX_STEPS][3];
};

// What every kernel takes.  Arguments lie in host memory: the fewer lines, the
// sooner a small product starts.
struct MuonArgs {
    const MatTile* tiles;
    const MuonRec* recs;
    char* ws;
    const int32_t* found_inf;
    MuonScale s;
    float ca, cb, cc;         // the iteration's coefficients
    int32_t step;             // of the iteration: which h is read
    int32_t n_tiles;
    int32_t update_dtype, copy_dtype;
};

// What those that read the gradients or write the weights take besides.
struct MuonMore {
    const void* const* grads;
    float* momentum;          // null: the gradients themselves are orthogonalised
    const double* g_coef;
    double eps;
    int32_t grad_dtype;
    MuonGroup g[FP_MAX_GROUPS];
};

// A chunk of the norm's sum: kChunk elements, or so many that a matrix has
// kMaxChunks.
constexpr int64_t kChunk = 8192, kMaxChunks = 1024;
constexpr int kOwnChunks = 64;  // up to so many, the kernel that writes X adds them up itself

// Of the kernel that writes X: the padded matrix in pieces of so many rows and columns.
constexpr int kCastRows = 16, kCastCols = 128;

// Tiles of the products.  kTile64Deep: with eight stages in LDS, for a
// workgroup that has its CU to itself.  kTile192: of the symmetric products, where
// a triangle's 256-wide tiles leave CUs idle (4096 x 4096: 136 tiles, A 107 us and B
// 119; 253 of these 92 and 98).
enum { kTile256 = 0, kTile128 = 1, kTile64 = 2, kTile64Deep = 3, kFullShapes = 4, kTile192 = 4, kHalfShapes = 5 };
constexpr int kTileSide[kHalfShapes] = {256, 128, 64, 64, 192};

// Of the kernel that adds A's slices up.
constexpr int kJoins = 4, kMaxSlices = 32;

// Small matrices: what one workgroup needs for one of rows x cols, in bytes of
// LDS and in 16 x 16 tiles per wave: up to 4 as they come, else four by four.
constexpr int kSmallThreads = 512;
constexpr int kSmallTiles = 16;
inline int64_t small_lds(int64_t rows, int64_t cols) {
    const int64_t m = ceil_div64(rows < cols ? rows : cols, 32) * 32, n = ceil_div64(rows < cols ? cols : rows, 32) * 32;
    return m * (2 * n + 16) + 2 * m * (2 * m + 16) + 8 * m;
}
inline int64_t small_tiles(int64_t rows, int64_t cols) {
    const int64_t blocks = ceil_div64(rows, 32) * ceil_div64(cols, 32), waves = kSmallThreads / 64;
    return 4 * blocks <= 4 * waves ? ceil_div64(4 * blocks, waves) : 4 * ceil_div64(blocks, waves);
}
inline bool is_small(int64_t rows, int64_t cols) {
    return small_tiles(rows, cols) <= kSmallTiles && small_lds(rows, cols) <= (160 << 10) - 512;
}

hipError_t launch_muon_small(const MuonArgs& a, const MuonMore& more, const MuonSteps& steps, int tiles, unsigned lds, hipStream_t s);
hipError_t launch_muon_moment(const MuonArgs& a, const MuonMore& more, hipStream_t s);
hipError_t launch_muon_norm(const MuonArgs& a, double eps, hipStream_t s);
hipError_t launch_muon_cast(const MuonArgs& a, const MuonMore& more, hipStream_t s);
hipError_t launch_muon_gram(const MuonArgs& a, int shape, hipStream_t s);
hipError_t launch_muon_join(const MuonArgs& a, hipStream_t s);  // kJoins workgroups a tile
hipError_t launch_muon_poly(const MuonArgs& a, int shape, hipStream_t s);
// The matrix goes on, or (the iteration's last) leaves as update or, where there
// are weights to change, into them.
hipError_t launch_muon_next(const MuonArgs& a, int shape, hipStream_t s);
hipError_t launch_muon_last(const MuonArgs& a, const MuonMore* weights, int shape, hipStream_t s);

// ---------------------------------------------------------------- MXFP4

constexpr int kMx4Block = 32;
constexpr int kMx4Pad = 256;  // rows are padded to multiples of so many elements
inline int64_t mx4_pad(int64_t n) { return (n + kMx4Pad - 1) / kMx4Pad * kMx4Pad; }

struct Mx4QuantArgs {
    const void* x;
    int64_t rows, cols, pitch;      // elements
    uint8_t *codes, *scales;        // rows' form, or null
    uint8_t *codes_t, *scales_t;    // columns' form, or null
    int64_t cp, rp;                 // padded columns and rows
    uint32_t key;
    int32_t dtype, stochastic;
};

struct Mx4DequantArgs {
    const uint8_t *codes, *scales;
    void* out;
    int64_t rows, cols, pitch, cp;
    int32_t dtype;
};

struct Mx4MatmulArgs {
    const uint8_t *a, *as, *b, *bs;
    void* out;
    int64_t m, n, kp, pitch;
    int32_t dtype, accumulate;
    int32_t tiles_m, tiles_n;
};

// Lanes of a launch.
int64_t mx4_quantize_lanes(const Mx4QuantArgs& a);
int64_t mx4_matmul_lanes(const Mx4MatmulArgs& a);
hipError_t launch_mx4_quantize(const Mx4QuantArgs& a, hipStream_t s);
hipError_t launch_mx4_dequantize(const Mx4DequantArgs& a, hipStream_t s);
hipError_t launch_mx4_matmul(const Mx4MatmulArgs& a, hipStream_t s);

}  // namespace fpk
