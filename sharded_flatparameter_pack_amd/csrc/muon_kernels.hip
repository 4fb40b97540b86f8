// muon_kernels.hip -- gfx950 kernels of the orthogonalisation of matrices by a
// Newton-Schulz iteration, and of the optimizer step that takes it.
//
// With U the momentum's matrix (or the gradient), turned in thought so that it
// has m rows, its smaller side, and n columns:
//   X = U / (|U|_F + eps);  steps times  A = X X^T,  B = b A + c A^2,
//   X <- a X + B X.
// Launches: the momentum and |U|_F^2's partial sums (moment); X (cast); for
// every step of the iteration A (gram), B (poly) and the next X (next), the last
// of which writes the weights.  All matrices of a batch share each launch.  A
// matrix stays as it lies: where a product contracts its rows, its fragments
// come out of LDS through the transposing read.
//
// Precision.  The products run on fp16 operands with fp32 sums.  What fp16
// loses is kept small by holding apart what carries most: X, of which only the
// first of two parts goes into products (h in fp16 + l in bf16: 20 bits, and
// fp32's range for a matrix far below eps), and in fp32 the diagonals of A and
// B, which stand far above the other elements.  With D the diagonal of B and R the
// rest, a step is X <- a X + D X_h + R X_h, and in the last ones X <- (a + D) X + R X_h.
// In a matrix of full rank the second is the better: only R's product sees the rounded X.  But B = D + R is 0 in directions that X does
// not hold and R alone is not: X - X_h has parts there, R leaves |D| 2^-12 of them,
// and every later step multiplies those by a = 3.44 (a gradient of rank 1: off by 4e-2
// for 2 x 512, and at any size if few of its rows are not zero).  With D
// and R on the same X_h nothing leaves X's rank but products of two roundings; the
// roundings of A and R act on X from its left and cannot.  So the second form is for the
// steps after which such a part grows by 4 at most (the last two of five).  Relative
// 2-norm errors of five steps against 64 bits (512 x 512, this arithmetic in torch: normal /
// singular values i^-1 / 8 of them 8 times the rest's norm / rank 1 / rank 1 in three rows):
// 8e-4 / 3e-4 / 3e-4 / 3e-4 / 1.5e-3, the second form throughout 7e-4 / 3e-4 / 3e-4 / 9e-4 /
// 3.4e-2, the first 1.2e-3 / 4e-4 / 5e-4 / 3e-4 / 1.6e-3; fp16 for everything 1.7e-3 / 3e-3 /
// 6e-3 for the first three, bf16 1e-2 / 2e-2 / 5e-2 (2^-8 is 4e-3).
// Powers of two (MuonScale) keep every fp16 form in its normal range.
//
// Compiled with -ffp-contract=off.

#include <type_traits>

#include "fp_matrix.h"
#include "mma_tile.h"
#include "param_ops.h"

namespace fpk {

namespace {

using Shape256 = TileShape<256, 256, 128, 64>;
using Shape128 = TileShape<128, 128, 64, 64>;
using Shape64 = TileShape<64, 64, 32, 32>;
using Shape64Deep = TileShape<64, 64, 32, 32, 8>;
using Shape192 = TileShape<192, 192, 64, 48>;

__device__ __forceinline__ bool skipped(const MuonArgs& a) { return a.found_inf != nullptr && *a.found_inf != 0; }

__device__ __forceinline__ double sum256(double x, double* lds) {
    x = wave_sum(x);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

// Elements [e, e + have) of a gradient, have in [1, 4]; kKept: to be found in the
// caches afterwards.
template <int kGrad, bool kKept>
__device__ __forceinline__ void grad4(const void* g, int64_t e, int have, float f[4]) {
    constexpr int kSize = kGrad == FP_DTYPE_F32 ? 4 : 2;
    const char* p = static_cast<const char*>(g) + e * kSize;
    GradQuad<kGrad> q;
    if (have < 4) q = ld_grad_few<kGrad>(p, have);
    else if constexpr (!kKept) q = ld_grad<kGrad>(g, e);
    else if constexpr (kGrad == FP_DTYPE_F32) q.w = get16u(p);
    else q.w = get8h(p);
    grad_f32(q, f);
}

// Four fp32 from a 4-byte boundary, the first `have` of them.
__device__ __forceinline__ void ld_f32(const float* p, int have, float f[4]) {
    if (have == 4) {
        f32x4_of(ld16u(p), f);
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = k < have ? gptr<float>((const void*)p)[k] : 0.0f;
}

__device__ __forceinline__ void st_f32(float* p, int have, const float f[4]) {
    if (have == 4) {
        put16u(p, bits_of(f));
        return;
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (k < have) gptr<float>((void*)p)[k] = f[k];
}

__device__ __forceinline__ void st_16bit(void* p, int have, uint2 w) {
    if (have == 4) {
        put8h(p, w);
        return;
    }
    const uint64_t x = ((uint64_t)w.y << 32) | w.x;
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (k < have) gptr<uint16_t>(p)[k] = (uint16_t)(x >> (16 * k));
}

__device__ __forceinline__ uint2 f16x4(const float f[4]) { return make_uint2(f16_pair(f[0], f[1]), f16_pair(f[2], f[3])); }

// ---------------------------------------------------------------- moment

// One chunk of one matrix: the momentum m' = beta m + (1 - beta) k g, in fp64
// rounded once, and the sum of u^2 in fp64, in an order of its own.  Memory bounds
// it (201M elements, bf16 gradients: 420 us, 4.8 TB/s), so that four loads are under
// way per lane.
template <int kGrad, bool kStep>
__global__ __launch_bounds__(256) void moment_kernel(const MuonArgs a, const MuonMore b) {
    __shared__ double lds[4];
    if (kStep && skipped(a)) return;
    const MatTile t = a.tiles[blockIdx.x];
    const MuonRec& r = a.recs[t.mat];
    const void* grad = b.grads[t.mat];
    const int64_t n = (int64_t)r.rows * r.cols;
    const int64_t from = r.chunk * t.ti, to = from + r.chunk < n ? from + r.chunk : n;
    const MuonGroup& hp = b.g[kStep ? r.group : 0];
    const double k = kStep && b.g_coef != nullptr ? *b.g_coef : 1.0;
    const double mine = kStep ? (1.0 - hp.beta) * k : 1.0;
    double sum = 0.0;
    constexpr int kAtOnce = 4;  // loads under way per lane
    for (int64_t e0 = from + 4 * threadIdx.x; e0 < to; e0 += 1024 * kAtOnce) {
        float g[kAtOnce][4], m[kAtOnce][4];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int64_t e = e0 + 1024 * i;
            if (e >= to) continue;
            grad4<kGrad, false>(grad, e, to - e < 4 ? (int)(to - e) : 4, g[i]);
            if constexpr (kStep) f32x4_of(get16(b.momentum + r.offset + e), m[i]);  // room up to the next multiple of 32
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int64_t e = e0 + 1024 * i;
            if (e >= to) continue;
            const int have = to - e < 4 ? (int)(to - e) : 4;
            double u[4];
            if constexpr (kStep) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    m[i][q] = (float)(hp.beta * (double)m[i][q] + mine * (double)g[i][q]);
                    u[q] = hp.nesterov ? hp.beta * (double)m[i][q] + mine * (double)g[i][q] : (double)m[i][q];
                }
                st_f32(b.momentum + r.offset + e, have, m[i]);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) u[q] = (double)g[i][q];
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (q < have) sum += u[q] * u[q];
        }
    }
    sum = sum256(sum, lds);
    if (threadIdx.x == 0) gptr<double>((void*)(a.ws + r.part))[t.ti] = sum;
}

// ---------------------------------------------------------------- the forms of X

// Eight values, scaled, into both parts, `at` elements from a tile's start (less
// than 2^28: an offset in one register, beside a base that all lanes share).
__device__ __forceinline__ void st_x(char* h, char* l, uint32_t at, const float x[8]) {
    uint32_t hw[4], lw[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        hw[k] = f16_pair(x[2 * k], x[2 * k + 1]);
        lw[k] = bf16x2(x[2 * k] - f16_lo(hw[k]), x[2 * k + 1] - f16_hi(hw[k]));
    }
    put16(h + 2 * at, make_uint4(hw[0], hw[1], hw[2], hw[3]));
    put16(l + 2 * at, make_uint4(lw[0], lw[1], lw[2], lw[3]));
}
template <int kVec>
__device__ __forceinline__ void x_of(const uint32_t* hw, const uint32_t* lw, float* x) {
#pragma unroll
    for (int k = 0; k < kVec / 2; ++k) {
        x[2 * k] = f16_lo(hw[k]) + bf16_lo(lw[k]);
        x[2 * k + 1] = f16_hi(hw[k]) + bf16_hi(lw[k]);
    }
}
__device__ __forceinline__ void f16x8_to_f32(const uint4 a, float x[8]) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) x[2 * k] = f16_lo(w[k]), x[2 * k + 1] = f16_hi(w[k]);
}
__device__ __forceinline__ void st_f16(void* p, const float x[8]) {
    put16(p, make_uint4(f16_pair(x[0], x[1]), f16_pair(x[2], x[3]), f16_pair(x[4], x[5]), f16_pair(x[6], x[7])));
}

// ---------------------------------------------------------------- norm

// Each matrix's 1 / (|U| + eps), behind its partial sums, where those are more
// than the cast kernel's waves add up themselves.
__global__ __launch_bounds__(256) void norm_kernel(const MuonArgs a, const double eps) {
    __shared__ double lds[4];
    if (skipped(a)) return;
    const MuonRec& r = a.recs[a.tiles[blockIdx.x].mat];
    FP_GLOBAL double* part = gptr<double>((void*)(a.ws + r.part));
    double sum = 0.0;
    for (int i = threadIdx.x; i < r.chunks; i += 256) sum += part[i];
    sum = sum256(sum, lds);
    if (threadIdx.x == 0) part[r.chunks] = 1.0 / (sqrt(sum) + eps);
}

// ---------------------------------------------------------------- cast

// kCastRows x kCastCols of the padded matrix: X = U / (|U| + eps), U again from the
// momentum and the gradient, which is less to move than U between two launches.
// Memory bounds it (201M elements: 375 us, 5.4 TB/s).
template <int kGrad, bool kStep>
__global__ __launch_bounds__(256) void cast_kernel(const MuonArgs a, const MuonMore b) {
    if (kStep && skipped(a)) return;
    const MatTile t = a.tiles[blockIdx.x];
    const MuonRec& r = a.recs[t.mat];
    const FP_GLOBAL double* part = gptr<double>((const void*)(a.ws + r.part));
    double scale;
    if (r.chunks > kOwnChunks) {
        scale = part[r.chunks];
    } else {
        const int lane = threadIdx.x & 63;
        scale = 1.0 / (sqrt(wave_sum(lane < r.chunks ? part[lane] : 0.0)) + b.eps);
    }
    const void* grad = b.grads[t.mat];
    const MuonGroup& hp = b.g[kStep ? r.group : 0];
    const double k = kStep && b.g_coef != nullptr ? *b.g_coef : 1.0;
    const double mine = kStep ? (1.0 - hp.beta) * k : 1.0;
    const int row0 = t.ti * kCastRows, col0 = t.tj * kCastCols;
    const int row = row0 + (threadIdx.x >> 4), col = col0 + (threadIdx.x & 15) * 8;
    if (row >= r.rp || col >= r.cp) return;
    const int left = row < r.rows ? r.cols - col : 0;
    const int64_t e = (int64_t)row * r.cols + col;
    const bool both = !kStep || hp.nesterov;  // else the gradient is in the momentum
    float g[8] = {}, m[8] = {};
    if (left >= 8) {  // both halves of a lane's run at once, through the cache: apart they were read twice over
        if (both) grad4<kGrad, true>(grad, e, 4, g), grad4<kGrad, true>(grad, e + 4, 4, g + 4);
        if constexpr (kStep) f32x4_of(get16u(b.momentum + r.offset + e), m), f32x4_of(get16u(b.momentum + r.offset + e + 4), m + 4);
    } else {
#pragma unroll
        for (int q = 0; q < 8; q += 4) {
            const int have = left - q < 4 ? left - q : 4;
            if (have <= 0) break;
            if (both) grad4<kGrad, true>(grad, e + q, have, g + q);
            if constexpr (kStep) ld_f32(b.momentum + r.offset + e + q, have, m + q);
        }
    }
    float x[8];
#pragma unroll
    for (int k8 = 0; k8 < 8; ++k8) {
        double u = kStep ? (double)m[k8] : (double)g[k8];
        if (kStep && hp.nesterov) u = hp.beta * u + mine * (double)g[k8];
        x[k8] = k8 < left ? (float)(u * scale) * a.s.x : 0.0f;
    }
    const int64_t base = 2 * ((int64_t)row0 * r.cp + col0);
    st_x(a.ws + r.h[0] + base, a.ws + r.l + base, (uint32_t)((row - row0) * r.cp + col - col0), x);
}

// ---------------------------------------------------------------- products

struct Sides {
    int m, n;     // padded
    bool turned;  // tall: m counts the columns
};
__device__ __forceinline__ Sides sides(const MuonRec& r) {
    const bool turned = r.rows > r.cols;
    return turned ? Sides{r.cp, r.rp, true} : Sides{r.rp, r.cp, false};
}

// The tile's rows (columns) from `first` on, of fp16 rows of `width`.
__device__ __forceinline__ Operand rows_of(const char* base, int64_t first, int64_t rows, int64_t width) {
    return {base + 2 * first * width, 2 * width, (int)(rows - first), nullptr};
}
__device__ __forceinline__ Operand columns_of(const char* base, int64_t first, int64_t width) {
    return {base + 2 * first, 2 * width, (int)(width - first), nullptr};
}

// A slice's sums of tile (ti, tj) of A.
__device__ __forceinline__ float* slice_sums(const MuonArgs& a, const MuonRec& r, const Sides& z, int slice, int ti, int tj) {
    constexpr int kSide = Shape64Deep::kBM;
    const int t = (z.m + kSide - 1) / kSide, tile = ti * (ti + 1) / 2 + tj;
    return reinterpret_cast<float*>(a.ws + r.split) + (int64_t)(slice * (t * (t + 1) / 2) + tile) * (kSide * kSide);
}

// A = X X^T (X^T X of a tall matrix): the tiles on and below the diagonal, and
// their mirror images, half the work of all tiles.  4096 x 4096: 92 us, 253 tiles at
// once on 256 CUs (0.75 PFLOP/s of the half; it ends with its last tile, and the
// tile's 64 steps take 75); the four matrices of a d = 4096 layer 795 us.
template <class S>
__global__ __launch_bounds__(S::kThreadsWg, S::kWavesSimd) void gram_kernel(const MuonArgs a) {
    extern __shared__ __align__(16) char lds[];
    if (skipped(a)) return;
    const MatTile t = a.tiles[blockIdx.x];
    if (t.mat < 0) return;
    const MuonRec& r = a.recs[t.mat];
    const Sides z = sides(r);
    constexpr bool kSlices = std::is_same<S, Shape64Deep>::value;
    const bool sliced = kSlices && r.slices > 1;
    const int i0 = t.ti * S::kBM, j0 = t.tj * S::kBN, from = sliced ? t.slice * r.slice_steps : 0;
    const int left = z.n / kStepF16 - from, steps = sliced && r.slice_steps < left ? r.slice_steps : left;
    const char* h = a.ws + r.h[a.step & 1] + (int64_t)from * kStepBytes * (z.turned ? z.m : 1);
    TileProduct<S> tile;
    if (z.turned) run_tile<kColumnsF16, kColumnsF16>(tile, columns_of(h, i0, z.m), columns_of(h, j0, z.m), steps, lds);
    else run_tile<kRowsF16, kRowsF16>(tile, rows_of(h, i0, z.m, z.n), rows_of(h, j0, z.m, z.n), steps, lds);
    if constexpr (kSlices) {
        if (sliced) {
            float* const sums = slice_sums(a, r, z, t.slice, t.ti, t.tj);
            tile.template each<2, 4>(lds, tile.nothing, [&](int tr, int tc, const float* v, typename TileProduct<S>::Nothing) {
                put16(sums + tr * S::kBN + tc, bits_of(v));
            });
            return;
        }
    }
    const float unscale = a.s.un_xx, out = a.s.gram;
    char* const to = a.ws + r.a + 2 * ((int64_t)i0 * z.m + j0);
    char* const mirror = a.ws + r.a + 2 * ((int64_t)j0 * z.m + i0);
    typedef typename TileProduct<S>::Nothing Nothing;
    auto body = [&](int tr, int tc, const float* v, Nothing) {
        const int row = i0 + tr, col = j0 + tc;
        if (row >= z.m || col >= z.m) return;
        float f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            f[k] = v[k] * out;
            if (row == col + k) {
                gptr<float>((void*)(a.ws + r.da))[row] = v[k] * unscale;
                f[k] = 0.0f;
            }
        }
        st_f16(to + 2 * (uint32_t)(tr * z.m + tc), f);
    };
    if (t.ti == t.tj) {
        tile.template each<2, 8>(lds, tile.nothing, body);
        return;
    }
    tile.template each<2, 8, true>(lds, tile.nothing, body, tile.nothing, [&](int tr, int tc, const float* v, Nothing) {
        const int row = i0 + tr, col = j0 + tc;
        if (row >= z.m || col >= z.m) return;
        float f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = v[k] * out;
        st_f16(mirror + 2 * (uint32_t)(tc * z.m + tr), f);
    });
}

// A from its slices' sums, in their order: a quarter of a tile per workgroup, four
// neighbours of a row per lane.
__global__ __launch_bounds__(256) void join_kernel(const MuonArgs a) {
    if (skipped(a)) return;
    const MatTile t = a.tiles[blockIdx.x / kJoins];
    const MuonRec& r = a.recs[t.mat];
    const Sides z = sides(r);
    constexpr int kSide = Shape64Deep::kBM;
    const int tr = (int)(blockIdx.x % kJoins) * 16 + (int)(threadIdx.x >> 4), tc = (int)(threadIdx.x & 15) * 4;
    const float* const sums = slice_sums(a, r, z, 0, t.ti, t.tj) + tr * kSide + tc;
    const int64_t apart = slice_sums(a, r, z, 1, 0, 0) - slice_sums(a, r, z, 0, 0, 0);
    float v[4] = {};
#pragma unroll 8
    for (int k = 0; k < r.slices; ++k) {
        float f[4];
        f32x4_of(get16(sums + k * apart), f);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] += f[q];
    }
    const int row = t.ti * kSide + tr, col = t.tj * kSide + tc;
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float f = v[q] * a.s.gram;
        if (row == col + q) {
            gptr<float>((void*)(a.ws + r.da))[row] = v[q] * a.s.un_xx;
            f = 0.0f;
        }
        w[q] = f16_pair(f, f);
    }
    FP_GLOBAL uint16_t* const out = gptr<uint16_t>((void*)(a.ws + r.a));
    *reinterpret_cast<FP_GLOBAL u32x2_t*>(out + (int64_t)row * z.m + col) =
        u32x2_t{(w[0] & 0xFFFFu) | w[1] << 16, (w[2] & 0xFFFFu) | w[3] << 16};
    if (t.ti == t.tj) return;
#pragma unroll
    for (int q = 0; q < 4; ++q) out[(int64_t)(col + q) * z.m + row] = (uint16_t)w[q];
}

// B = b A + c A^2 in the same way; db holds a + B's diagonal.  With d the
// diagonal of A and N the rest, A^2 = N^2 + (d_i + d_j) N off the diagonal.  4096 x
// 4096: 97 us; a d = 4096 layer 375.
template <class S>
__global__ __launch_bounds__(S::kThreadsWg, S::kWavesSimd) void poly_kernel(const MuonArgs a) {
    extern __shared__ __align__(16) char lds[];
    if (skipped(a)) return;
    const MatTile t = a.tiles[blockIdx.x];
    if (t.mat < 0) return;
    const MuonRec& r = a.recs[t.mat];
    const Sides z = sides(r);
    const char* n = a.ws + r.a;
    const int i0 = t.ti * S::kBM, j0 = t.tj * S::kBN;
    TileProduct<S> tile;
    run_tile<kRowsF16, kRowsF16>(tile, rows_of(n, i0, z.m, z.m), rows_of(n, j0, z.m, z.m), z.m / kStepF16, lds);
    const float un_a = a.s.un_a, un_s = un_a * un_a;
    const FP_GLOBAL float* d = gptr<float>((const void*)(a.ws + r.da));
    // eight elements (row, col ..) of N, with their part of the diagonals; the
    // mirror images of a tile are those of the other row, N being symmetric
    struct Fetched {
        uint4 n;
        float row;
    };
    const int64_t straight_at = 2 * ((int64_t)i0 * z.m + j0), mirror_at = 2 * ((int64_t)j0 * z.m + i0);
    auto fetch = [&](int row, int col, int64_t base, uint32_t at) {
        Fetched f = {make_uint4(0u, 0u, 0u, 0u), 0.0f};
        if (row < z.m && col < z.m) f = {get16(n + base + 2 * at), d[row]};
        return f;
    };
    auto poly = [&](int row, int col, int64_t base, uint32_t at, const float* v, const Fetched& e, const float dc[8]) {
        if (row >= z.m || col >= z.m) return;
        float x[8], f[8];
        f16x8_to_f32(e.n, x);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float square = v[k] * un_s;
            x[k] *= un_a;
            f[k] = __builtin_fmaf(a.cb, x[k], a.cc * __builtin_fmaf(e.row + dc[k], x[k], square)) * a.s.b;
            if (row == col + k) {
                gptr<float>((void*)(a.ws + r.db))[row] = a.ca + (a.cb * e.row + a.cc * (square + e.row * e.row));
                f[k] = 0.0f;
            }
        }
        st_f16(a.ws + r.b + base + 2 * at, f);
    };
    float dc[8], dr[8];  // of the lane's columns; of the eight rows of a mirror image, per pass
#pragma unroll
    for (int k = 0; k < 8; ++k) dc[k] = j0 + tile.template each_col<8>() < z.m ? d[j0 + tile.template each_col<8>() + k] : 0.0f;
    auto body = [&](int tr, int tc, const float* v, const Fetched& e) {
        poly(i0 + tr, j0 + tc, straight_at, (uint32_t)(tr * z.m + tc), v, e, dc);
    };
    auto straight = [&](int tr, int tc) { return fetch(i0 + tr, j0 + tc, straight_at, (uint32_t)(tr * z.m + tc)); };
    constexpr int kPer = S::kFM > 4 ? 1 : 2;  // as many registers as there are
    if (t.ti == t.tj) {
        tile.template each<kPer, 8>(lds, straight, body);
        return;
    }
    int had = -1;
    tile.template each<kPer, 8, true>(
        lds, straight, body,
        [&](int tr, int tc) { return fetch(j0 + tc, i0 + tr, mirror_at, (uint32_t)(tc * z.m + tr)); },
        [&](int tr, int tc, const float* v, const Fetched& e) {
            if (tr != had) {
                had = tr;
#pragma unroll
                for (int k = 0; k < 8; ++k) dr[k] = i0 + tr < z.m ? d[i0 + tr + k] : 0.0f;
            }
            poly(j0 + tc, i0 + tr, mirror_at, (uint32_t)(tc * z.m + tr), v, e, dr);
        });
}

// What the update is multiplied by beside the learning rate.
__device__ __forceinline__ double adjust_of(int adjust, double rows, double cols) {
    return adjust == FP_MUON_ADJUST_RMS     ? 0.2 * sqrt(rows > cols ? rows : cols)
           : adjust == FP_MUON_ADJUST_SHAPE ? sqrt(rows > cols ? rows / cols : 1.0)
                                            : 1.0;
}

// How the matrix leaves: into the next step, orthogonalised as an update or into the
// weights; kGoesOnHalf: into the next step, with B's diagonal on X_h (MuonScale::whole).
enum { kGoesOn = 0, kToUpdate = 1, kToWeights = 2, kGoesOnHalf = 3 };

// X <- a X + D X_h + R X_h or (a + D) X + R X_h, in the matrix's own orientation: B X of a
// wide matrix, X B of a tall one.  What stands between it and the product alone is the
// epilogue, which reads and writes 8 bytes per element (14 with weights and copies)
// while the matrix cores wait, a 256-wide tile having its CU to itself.  4096 x 4096:
// 150 us, the product alone 101; a d = 4096 layer 1550, with weights 2110 (memory
// alone 260 and 455).
template <class S, int kAs, class More>
__device__ __forceinline__ void next_tile(const MuonArgs& a, const More& more) {
    extern __shared__ __align__(16) char lds[];
    constexpr bool kWhole = kAs != kGoesOnHalf;
    constexpr int kOut = kWhole ? kAs : kGoesOn;
    const MatTile t = a.tiles[blockIdx.x];
    if (t.mat < 0) return;
    const MuonRec& r = a.recs[t.mat];
    const Sides z = sides(r);
    const int i0 = t.ti * S::kBM, j0 = t.tj * S::kBN;
    const bool skip = skipped(a);
    if (skip && (kOut != kToWeights || r.copy == nullptr)) return;
    const char* h = a.ws + r.h[a.step & 1];
    const char* b = a.ws + r.b;
    // x = ((a + D) x_old + sums) as the next step wants it, or as it is
    const float next = kOut == kGoesOn ? a.s.x_next : 1.0f;
    const float un_x = a.s.un_x * next, unscale = a.s.un_bx * next, a_x = a.ca * un_x;
    const FP_GLOBAL float* d = gptr<float>((const void*)(a.ws + r.db));
    double rate = 0.0, decay = 1.0;
    if constexpr (kOut == kToWeights) {
        const MuonGroup& hp = more.g[r.group];
        rate = hp.lr * adjust_of(hp.adjust, r.rows, r.cols);
        decay = hp.decay;
    }
    const int rows = (kOut == kGoesOn ? r.rp : r.rows) - i0, cols = (kOut == kGoesOn ? r.cp : r.cols) - j0;
    const int64_t base = 2 * ((int64_t)i0 * r.cp + j0);         // of the tile, in X's parts
    const int64_t out = (int64_t)i0 * r.cols + j0;              // in the matrix
    const char* const h_old = h + base;
    char* const h_new = a.ws + r.h[(a.step + 1) & 1] + base;
    char* const l = a.ws + r.l + base;
    // eight columns a lane, or four with the weights, and passes of one fragment
    constexpr int kVec = kOut == kToWeights ? 4 : 8, kPer = kOut == kToWeights ? 1 : 2;
    // What comes from memory: X's old value and the weights.  Tiles of 128 and less
    // have registers for the weights beside the product's, and fetch them before it
    // (32 matrices of 1408 x 512: 113 us, else 148; X, which is in the caches, gains
    // nothing by it).
    constexpr bool kEarly = kOut == kToWeights && S::kBM <= 128;
    struct OldX {
        uint32_t h[kVec / 2], l[kVec / 2];
    };
    struct OldW {
        float w[kOut == kToWeights ? kVec : 1];
    };
    struct Row {
        float d;
    };
    auto inside = [&](int tr, int tc) { return tr < rows && tc < cols; };
    auto have_of = [&](int tc, int q) { const int left = cols - tc - q; return left < 4 ? left : 4; };
    auto fetch_x = [&](int tr, int tc) {
        OldX f = {};
        if (skip || !inside(tr, tc)) return f;
        const uint32_t at = 2 * (uint32_t)(tr * r.cp + tc);
        if constexpr (kVec == 8) {
            const uint4 hi = get16(h_old + at), lo = get16(l + at);
            f.h[0] = hi.x; f.h[1] = hi.y; f.h[2] = hi.z; f.h[3] = hi.w;
            f.l[0] = lo.x; f.l[1] = lo.y; f.l[2] = lo.z; f.l[3] = lo.w;
        } else {
            const uint2 hi = get8(h_old + at), lo = get8(l + at);
            f.h[0] = hi.x; f.h[1] = hi.y;
            f.l[0] = lo.x; f.l[1] = lo.y;
        }
        return f;
    };
    auto fetch_w = [&](int tr, int tc) {
        OldW f = {};
        if constexpr (kOut == kToWeights)
            if (inside(tr, tc)) ld_f32(r.master + out + (uint32_t)(tr * r.cols + tc), have_of(tc, 0), f.w);
        return f;
    };
    auto fetch_d = [&](int tr, int) { return Row{!skip && !z.turned && tr < rows ? d[i0 + tr] * un_x : 0.0f}; };
    typedef TileProduct<S> Tile;
    Tile tile;
    float dc[kVec];  // of a tall matrix: of the lane's columns
    auto leave = [&](int tr, int tc, const float* v, const Row& row, const OldX& old, float* w) {
        if (!inside(tr, tc)) return;
        float x[kVec];
        if constexpr (kWhole) {
            x_of<kVec>(old.h, old.l, x);
#pragma unroll
            for (int k = 0; k < kVec; ++k) x[k] = __builtin_fmaf(z.turned ? dc[k] : row.d, x[k], v[k] * unscale);
        } else {
#pragma unroll
            for (int k = 0; k < kVec; ++k)
                x[k] = __builtin_fmaf(z.turned ? dc[k] : row.d, k & 1 ? f16_hi(old.h[k / 2]) : f16_lo(old.h[k / 2]), v[k] * unscale);
#pragma unroll
            for (int k = 0; k < kVec; ++k) x[k] = __builtin_fmaf(a_x, k & 1 ? bf16_hi(old.l[k / 2]) : bf16_lo(old.l[k / 2]), x[k]);
        }
        const uint32_t e = (uint32_t)(tr * r.cols + tc);
        if constexpr (kOut == kGoesOn) {
            st_x(h_new, l, (uint32_t)(tr * r.cp + tc), x);
        } else if constexpr (kOut == kToUpdate) {
#pragma unroll
            for (int q = 0; q < kVec; q += 4) {
                const int have = have_of(tc, q);
                if (have <= 0) break;
                if (a.update_dtype == FP_DTYPE_F32) st_f32(static_cast<float*>(r.update) + out + e + q, have, x + q);
                else st_16bit(static_cast<uint16_t*>(r.update) + out + e + q, have,
                              a.update_dtype == FP_DTYPE_F16 ? f16x4(x + q) : f32x4_to_bf16(x + q));
            }
        } else {
            const int have = have_of(tc, 0);
            if (!skip) {
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = (float)(decay * (double)w[k] - rate * (double)x[k]);
                st_f32(r.master + out + e, have, w);
            }
            if (r.copy != nullptr)
                st_16bit(static_cast<uint16_t*>(r.copy) + out + e, have, a.copy_dtype == FP_DTYPE_F16 ? f16x4(w) : f32x4_to_bf16(w));
        }
    };
    auto multiply = [&] {
        if (!skip) {
            const int steps = z.m / kStepF16;
            if (z.turned) run_tile<kRowsF16, kRowsF16>(tile, rows_of(h, i0, z.n, z.m), rows_of(b, j0, z.m, z.m), steps, lds);
            else run_tile<kRowsF16, kColumnsF16>(tile, rows_of(b, i0, z.m, z.m), columns_of(h, j0, z.n), steps, lds);
        }
        const int tc = Tile::template each_col<kVec>();
#pragma unroll
        for (int k = 0; k < kVec; ++k) dc[k] = !skip && z.turned && tc < cols && j0 + tc + k < z.m ? d[j0 + tc + k] * un_x : 0.0f;
    };
    if constexpr (kEarly) {
        struct XD {
            OldX x;
            Row d;
        };
        auto early = Tile::template fetch_early<kPer, kVec>(fetch_w);
        multiply();
        tile.template each<kPer, kVec>(
            lds, [&](int tr, int tc) { return XD{fetch_x(tr, tc), fetch_d(tr, tc)}; },
            [&](int tr, int tc, const float* v, const XD& f, OldW& w) { leave(tr, tc, v, f.d, f.x, w.w); }, early);
    } else {
        struct All {
            OldX x;
            OldW w;
            Row d;
        };
        multiply();
        tile.template each<kPer, kVec>(
            lds, [&](int tr, int tc) { return All{fetch_x(tr, tc), fetch_w(tr, tc), fetch_d(tr, tc)}; },
            [&](int tr, int tc, const float* v, All& f) { leave(tr, tc, v, f.d, f.x, f.w.w); });
    }
}

template <class S, int kOut>
__global__ __launch_bounds__(S::kThreadsWg, S::kWavesSimd) void next_kernel(const MuonArgs a) {
    next_tile<S, kOut>(a, 0);
}
template <class S>
__global__ __launch_bounds__(S::kThreadsWg, S::kWavesSimd) void weights_kernel(const MuonArgs a, const MuonMore b) {
    next_tile<S, kToWeights>(a, b);
}

// ---------------------------------------------------------------- small matrices

__device__ __forceinline__ void put8_lds(char* p, float a, float b, float c, float d) {
    *(u32x2_t*)p = u32x2_t{f16_pair(a, b), f16_pair(c, d)};
}

// A matrix that fits into one workgroup's LDS goes through all of it there: its
// momentum, |U|, every step of the iteration and the weights, in one launch for
// all such matrices (32 x 48 in five steps: 16 launches took 72 us).  It is worked
// on as m x n with m <= n, a tall one turned while it is loaded.  The lane that
// has an element of X in the product's output keeps it in fp32 from step to step;
// LDS has h, A and B, with rows 16 bytes longer than their elements, so that the
// 16 rows of a fragment sit in different banks.  A wave works on blocks of kSub x
// kSub tiles of 16 x 16: 2 x 2, four products for four fragments, where LDS reads
// bound a step (128 x 128 with 1 x 1: 11 us a step, with 2 x 2 6.2), 1 x 1 for the
// smallest, whose steps are all latency and want every wave (32 x 48: 1.2 us a step,
// with 2 x 2 2.3); A and B of at most 64 rows in blocks of 2 x 1, of which there is
// one for each wave (64 x 256: 3.5 us a step, so 3.2; 32 x 1024: 5.8, so 4.4).  Where
// B's diagonal multiplies X_h, a step takes 0.1 to 0.8 more (32 x 48 1.3, 64 x 256 3.5, 32 x
// 1024 5.2, 128 x 128 6.6).  The rest of a step with weights, 16 us for 64 x 256, is one
// CU's loads, fp64 and stores.
//
// kTiles: tiles of X per wave.
constexpr int kSmallWaves = kSmallThreads / 64;

template <int kTiles, int kSub, int kGrad>
__global__ __launch_bounds__(kSmallThreads, 2) void small_kernel(const MuonArgs a, const MuonMore b, const MuonSteps it) {
    extern __shared__ __align__(16) char lds[];
    __shared__ double sums[kSmallWaves];
    const int mat = a.tiles[blockIdx.x].mat;
    const MuonRec& r = a.recs[mat];
    const bool step = b.momentum != nullptr, turned = r.rows > r.cols;
    const bool skip = step && skipped(a);
    const int m0 = turned ? r.cols : r.rows, n0 = turned ? r.rows : r.cols;
    const int m = (m0 + 31) & ~31, n = (n0 + 31) & ~31;
    const int hp = 2 * n + 16, ap = 2 * m + 16;
    char* const h = lds;
    char* const la = h + m * hp;
    char* const lb = la + m * ap;
    float* const da = reinterpret_cast<float*>(lb + m * ap);
    float* const db = da + m;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int g = lane >> 4, j = lane & 15;
    constexpr int kBlock = 16 * kSub;
    const int across = n / kBlock, blocks = m / kBlock * across;
    const MuonGroup& hy = b.g[r.group];
    const void* grad = b.grads[mat];

    // The lane's four elements of its tile i: row `row` of X, columns col ..
    // col + 3; `have` of them exist.  In memory they are neighbours, or a row
    // apart.
    struct At {
        int row, col, have;
        uint32_t e, apart;
    };
    auto at = [&](int i) {
        At p;
        const int t = wave + i / (kSub * kSub) * kSmallWaves;
        p.row = t / across * kBlock + i / kSub % kSub * 16 + j;
        p.col = t % across * kBlock + i % kSub * 16 + 4 * g;
        const int left = n0 - p.col;
        p.have = t >= blocks || p.row >= m0 || left <= 0 ? 0 : left < 4 ? left : 4;
        p.e = (uint32_t)(turned ? p.col * m0 + p.row : p.row * n0 + p.col);
        p.apart = turned ? (uint32_t)m0 : 1u;
        return p;
    };
    // The loads of kGroup tiles are under way before the first is waited for;
    // lanes without an element load the first one.
    constexpr int kGroup = kTiles < 8 ? kTiles : 8;
    auto ld = [&](const auto* from, auto convert, int first, float (&f)[kGroup][4]) {
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
            const At p = at(first + i);
            if (!turned && p.have == 4) {
                typedef std::remove_cv_t<std::remove_reference_t<decltype(from[0])>> T;
                typedef T four_t __attribute__((ext_vector_type(4), aligned(sizeof(T))));
                const four_t v = *(const FP_GLOBAL four_t*)(from + p.e);
#pragma unroll
                for (int k = 0; k < 4; ++k) f[i][k] = convert(v[k]);
                continue;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) f[i][k] = convert(from[k < p.have ? p.e + (uint32_t)k * p.apart : 0u]);
        }
    };
    auto st = [&](auto* to, const At& p, const auto (&f)[4]) {
        if (!turned && p.have == 4) {
            typedef std::remove_reference_t<decltype(to[0])> T;
            typedef T four_t __attribute__((ext_vector_type(4), aligned(sizeof(T))));
            *(FP_GLOBAL four_t*)(to + p.e) = four_t{f[0], f[1], f[2], f[3]};
            return;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < p.have) to[p.e + (uint32_t)k * p.apart] = f[k];
    };
    auto same = [](float f) { return f; };

    float x[kTiles][4];
    double sum = 0.0;
    if (!skip) {
        const double k = step && b.g_coef != nullptr ? *b.g_coef : 1.0;
        const double beta = step ? hy.beta : 0.0, mine = step ? (1.0 - beta) * k : 1.0;
#pragma unroll
        for (int i0 = 0; i0 < kTiles; i0 += kGroup) {
            float u[kGroup][4], w[kGroup][4];
            if constexpr (kGrad == FP_DTYPE_F32) ld(gptr<float>(grad), same, i0, u);
            else ld(gptr<uint16_t>(grad), [](uint16_t v) { return kGrad == FP_DTYPE_BF16 ? bf16_lo(v) : f16_lo(v); }, i0, u);
            if (step) ld(gptr<float>((const void*)(b.momentum + r.offset)), same, i0, w);
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {
                const At p = at(i0 + i);
                if (step) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) w[i][q] = (float)(beta * (double)w[i][q] + mine * (double)u[i][q]);
                    st(gptr<float>((void*)(b.momentum + r.offset)), p, w[i]);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    double v = (double)u[i][q];
                    if (step) v = hy.nesterov ? beta * (double)w[i][q] + mine * v : (double)w[i][q];
                    v = q < p.have ? v : 0.0;
                    x[i0 + i][q] = (float)v;
                    sum += v * v;
                }
            }
            __builtin_amdgcn_sched_barrier(0);  // more at a time would not fit into the registers
        }
        sum = wave_sum(sum);
        if (lane == 0) sums[wave] = sum;
        __syncthreads();
        sum = 0.0;
#pragma unroll
        for (int w = 0; w < kSmallWaves; ++w) sum += sums[w];
        // x / norm in fp32, whose operations take a quarter of fp64's: times a power
        // of two, then by a number in (1, 2]
        const double norm = sqrt(sum) + b.eps;
        const int e = __builtin_amdgcn_frexp_exp(norm);
        const float scale = (float)(1.0 / __builtin_amdgcn_ldexp(norm, -e));
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) x[i][q] = __builtin_amdgcn_ldexpf(x[i][q], -e) * scale;

        auto st_h = [&](float s) {
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                const int t = wave + i / (kSub * kSub) * kSmallWaves;
                if (t >= blocks) continue;
                const At p = at(i);
                put8_lds(h + p.row * hp + 2 * p.col, x[i][0] * s, x[i][1] * s, x[i][2] * s, x[i][3] * s);
            }
        };
        // kN fragments of 16 rows from `row` on, the lane's 8 elements from k + 8 g on
        auto rows_at = [&](const char* base, int pitch, int row, int k, auto& f) {
            const char* p = base + (row + j) * pitch + 2 * (k + 8 * g);
#pragma unroll
            for (int y = 0; y < (int)(sizeof f / sizeof f[0]); ++y) f[y] = *(const f16x8_t*)(p + 16 * y * pitch);
        };
        auto product = [&](const auto& right, const auto& left, auto& acc) {
#pragma unroll
            for (int y = 0; y < kSub; ++y)
#pragma unroll
                for (int z = 0; z < (int)(sizeof right / sizeof right[0]); ++z)
                    acc[y][z] = __builtin_amdgcn_mfma_f32_16x16x32_f16(right[z], left[y], acc[y][z], 0, 0, 0);
        };
        // base base^T, m x m, block by block: out(row, col, four values from col
        // on, whether the diagonal may be among them).  Blocks are kBlock down, and
        // across kBlock or, where that leaves waves without one, half of it.
        const int side = m / kBlock, by_side = (256 + side - 1) / side;  // t / side = t by_side / 256 for t < 64
        auto square_by = [&](auto wide, const char* base, int pitch, int width, auto out) {
            constexpr int kWide = decltype(wide)::value, kParts = kSub / kWide;
            for (int t = wave; t < side * side * kParts; t += kSmallWaves) {
                const int block = t / kParts, bi = block * by_side >> 8, ti = bi * kBlock;
                const int tj = (block - bi * side) * kBlock + t % kParts * 16;
                f32x4_t acc[kSub][kWide] = {};
#pragma unroll 4
                for (int k = 0; k < width; k += 32) {
                    f16x8_t left[kSub], right[kWide];
                    rows_at(base, pitch, tj, k, right);
                    rows_at(base, pitch, ti, k, left);
                    product(right, left, acc);
                }
#pragma unroll
                for (int y = 0; y < kSub; ++y)
#pragma unroll
                    for (int z = 0; z < kWide; ++z)
                        out(ti + 16 * y + j, tj + 16 * z + 4 * g, acc[y][z], ti + 16 * y == tj + 16 * z);
            }
        };
        auto square = [&](const char* base, int pitch, int width, auto out) {
            if (kSub == 1 || side * side >= kSmallWaves) square_by(std::integral_constant<int, kSub>{}, base, pitch, width, out);
            else square_by(std::integral_constant<int, 1>{}, base, pitch, width, out);
        };
        st_h(it.s[0].x);
        for (int s = 0; s < it.n; ++s) {
            const MuonScale sc = it.s[s];
            const float ca = it.c[s][0], cb = it.c[s][1], cc = it.c[s][2];
            __syncthreads();
            square(h, hp, n, [&](int row, int col, const f32x4_t v, bool diagonal) {  // A
                float f[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) f[q] = v[q] * sc.gram;
                if (diagonal) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (row == col + q) {
                            da[row] = v[q] * sc.un_xx;
                            f[q] = 0.0f;
                        }
                }
                put8_lds(la + row * ap + 2 * col, f[0], f[1], f[2], f[3]);
            });
            __syncthreads();
            square(la, ap, m, [&](int row, int col, const f32x4_t v, bool diagonal) {  // B
                const u32x2_t w = *(const u32x2_t*)(la + row * ap + 2 * col);
                const f32x4_t dc = *(const f32x4_t*)(da + col);
                const float e[4] = {f16_lo(w.x), f16_hi(w.x), f16_lo(w.y), f16_hi(w.y)};
                const float di = da[row];
                float f[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float a2 = v[q] * (sc.un_a * sc.un_a), a1 = e[q] * sc.un_a;
                    f[q] = __builtin_fmaf(cb, a1, cc * __builtin_fmaf(di + dc[q], a1, a2)) * sc.b;
                    if (diagonal && row == col + q) {
                        db[row] = ca + (cb * di + cc * (a2 + di * di));
                        f[q] = 0.0f;
                    }
                }
                put8_lds(lb + row * ap + 2 * col, f[0], f[1], f[2], f[3]);
            });
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kTiles; i += kSub * kSub) {  // X
                const int t = wave + i / (kSub * kSub) * kSmallWaves;
                if (t >= blocks) continue;
                const int ti = t / across * kBlock, tj = t % across * kBlock;
                f32x4_t acc[kSub][kSub] = {};
#pragma unroll 2
                for (int k = 0; k < m; k += 32) {
                    // rows k + 8 g .. + 7 of h, columns tj + j, tj + 16 + j
                    const char* p = h + (k + 8 * g + (j >> 2)) * hp + 2 * (tj + (j & 3) * 4);
                    f16x8_t left[kSub], right[kSub];
#pragma unroll
                    for (int z = 0; z < kSub; ++z) {
                        typedef short s16x8_t __attribute__((ext_vector_type(8)));
                        const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((FP_LDS s16x4_t*)(p + 32 * z));
                        const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((FP_LDS s16x4_t*)(p + 32 * z + 4 * hp));
                        right[z] = __builtin_bit_cast(f16x8_t, (s16x8_t)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                    }
                    rows_at(lb, ap, ti, k, left);
                    product(right, left, acc);
                }
#pragma unroll
                for (int y = 0; y < kSub; ++y) {
                    const float d = db[ti + 16 * y + j];
                    if (sc.whole) {
#pragma unroll
                        for (int z = 0; z < kSub; ++z)
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                float& e = x[i + kSub * y + z][q];
                                e = __builtin_fmaf(d, e, acc[y][z][q] * sc.un_bx);
                            }
                    } else {
                        const float dh = (d - ca) * sc.un_x;  // of X_h as it is in LDS
#pragma unroll
                        for (int z = 0; z < kSub; ++z)
#pragma unroll
                            for (int q = 0; q < 4; q += 2) {
                                float* const e = x[i + kSub * y + z] + q;
                                const uint32_t h2 = f16_pair(e[0] * sc.x, e[1] * sc.x);
                                e[0] = __builtin_fmaf(dh, f16_lo(h2), __builtin_fmaf(ca, e[0], acc[y][z][q] * sc.un_bx));
                                e[1] = __builtin_fmaf(dh, f16_hi(h2), __builtin_fmaf(ca, e[1], acc[y][z][q + 1] * sc.un_bx));
                            }
                    }
                }
            }
            if (s + 1 < it.n) {
                __syncthreads();
                st_h(sc.x_next);
            }
        }
    } else if (r.copy == nullptr) {
        return;
    }

    const double rate = step ? hy.lr * adjust_of(hy.adjust, r.rows, r.cols) : 0.0;
    void* const to = step ? r.copy : r.update;
    const int dtype = step ? a.copy_dtype : a.update_dtype;
#pragma unroll
    for (int i0 = 0; i0 < kTiles; i0 += kGroup) {
        float w[kGroup][4];
        if (step) ld(gptr<float>((const void*)r.master), same, i0, w);
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
            const At p = at(i0 + i);
            if (step && !skip) {
#pragma unroll
                for (int q = 0; q < 4; ++q) w[i][q] = (float)(hy.decay * (double)w[i][q] - rate * (double)x[i0 + i][q]);
                st(gptr<float>((void*)r.master), p, w[i]);
            }
            if (to == nullptr) continue;
            float f[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                f[q] = x[i0 + i][q];
                if (step) f[q] = w[i][q];
            }
            if (dtype == FP_DTYPE_F32) {
                st(gptr<float>(to), p, f);
                continue;
            }
            const uint32_t lo = dtype == FP_DTYPE_F16 ? f16_pair(f[0], f[1]) : bf16x2(f[0], f[1]);
            const uint32_t hi = dtype == FP_DTYPE_F16 ? f16_pair(f[2], f[3]) : bf16x2(f[2], f[3]);
            const uint16_t v[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
            st(gptr<uint16_t>(to), p, v);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

}  // namespace

hipError_t launch_muon_moment(const MuonArgs& a, const MuonMore& b, hipStream_t s) {
#define FP_CALL(G)                                                                                  \
    (b.momentum != nullptr ? launch<moment_kernel<G, true>>((unsigned)a.n_tiles, 256, 0, s, a, b) \
                           : launch<moment_kernel<G, false>>((unsigned)a.n_tiles, 256, 0, s, a, b))
    return b.grad_dtype == FP_DTYPE_F32 ? FP_CALL(FP_DTYPE_F32) : b.grad_dtype == FP_DTYPE_BF16 ? FP_CALL(FP_DTYPE_BF16) : FP_CALL(FP_DTYPE_F16);
#undef FP_CALL
}

hipError_t launch_muon_norm(const MuonArgs& a, double eps, hipStream_t s) {
    return launch<norm_kernel>((unsigned)a.n_tiles, 256, 0, s, a, eps);
}

hipError_t launch_muon_cast(const MuonArgs& a, const MuonMore& b, hipStream_t s) {
#define FP_CALL(G)                                                                                \
    (b.momentum != nullptr ? launch<cast_kernel<G, true>>((unsigned)a.n_tiles, 256, 0, s, a, b) \
                           : launch<cast_kernel<G, false>>((unsigned)a.n_tiles, 256, 0, s, a, b))
    return b.grad_dtype == FP_DTYPE_F32 ? FP_CALL(FP_DTYPE_F32) : b.grad_dtype == FP_DTYPE_BF16 ? FP_CALL(FP_DTYPE_BF16) : FP_CALL(FP_DTYPE_F16);
#undef FP_CALL
}

#define FP_BY_SHAPE(CALL)                                                                                            \
    (shape == kTile256 ? CALL(Shape256) : shape == kTile128 ? CALL(Shape128) : shape == kTile64 ? CALL(Shape64) \
                                                                                                : CALL(Shape64Deep))

hipError_t launch_muon_gram(const MuonArgs& a, int shape, hipStream_t s) {
#define FP_CALL(S) launch<gram_kernel<S>>((unsigned)a.n_tiles, S::kThreadsWg, S::kLds, s, a)
    return shape == kTile192 ? FP_CALL(Shape192) : FP_BY_SHAPE(FP_CALL);
#undef FP_CALL
}

hipError_t launch_muon_join(const MuonArgs& a, hipStream_t s) {
    return launch<join_kernel>((unsigned)(a.n_tiles * kJoins), 256, 0, s, a);
}

hipError_t launch_muon_poly(const MuonArgs& a, int shape, hipStream_t s) {
#define FP_CALL(S) launch<poly_kernel<S>>((unsigned)a.n_tiles, S::kThreadsWg, S::kLds, s, a)
    return shape == kTile192 ? FP_CALL(Shape192) : FP_BY_SHAPE(FP_CALL);
#undef FP_CALL
}

hipError_t launch_muon_next(const MuonArgs& a, int shape, hipStream_t s) {
#define FP_CALL(S)                                                                                    \
    (a.s.whole ? launch<next_kernel<S, kGoesOn>>((unsigned)a.n_tiles, S::kThreadsWg, S::kLds, s, a) \
               : launch<next_kernel<S, kGoesOnHalf>>((unsigned)a.n_tiles, S::kThreadsWg, S::kLds, s, a))
    return FP_BY_SHAPE(FP_CALL);
#undef FP_CALL
}

hipError_t launch_muon_last(const MuonArgs& a, const MuonMore* weights, int shape, hipStream_t s) {
#define FP_WEIGHTS(S) launch<weights_kernel<S>>((unsigned)a.n_tiles, S::kThreadsWg, S::kLds, s, a, *weights)
#define FP_UPDATE(S) launch<next_kernel<S, kToUpdate>>((unsigned)a.n_tiles, S::kThreadsWg, S::kLds, s, a)
    return weights != nullptr ? FP_BY_SHAPE(FP_WEIGHTS) : FP_BY_SHAPE(FP_UPDATE);
#undef FP_WEIGHTS
#undef FP_UPDATE
}
#undef FP_BY_SHAPE

template <int kTiles, int kSub>
static hipError_t launch_small(const MuonArgs& a, const MuonMore& b, const MuonSteps& steps, unsigned lds, hipStream_t s) {
#define FP_CALL(G) launch<small_kernel<kTiles, kSub, G>>((unsigned)a.n_tiles, kSmallThreads, lds, s, a, b, steps)
    return b.grad_dtype == FP_DTYPE_F32 ? FP_CALL(FP_DTYPE_F32) : b.grad_dtype == FP_DTYPE_BF16 ? FP_CALL(FP_DTYPE_BF16) : FP_CALL(FP_DTYPE_F16);
#undef FP_CALL
}

hipError_t launch_muon_small(const MuonArgs& a, const MuonMore& b, const MuonSteps& steps, int tiles, unsigned lds,
                             hipStream_t s) {
    return tiles <= 2   ? launch_small<2, 1>(a, b, steps, lds, s)
           : tiles <= 4 ? launch_small<4, 1>(a, b, steps, lds, s)
           : tiles <= 8 ? launch_small<8, 2>(a, b, steps, lds, s)
                        : launch_small<kSmallTiles, 2>(a, b, steps, lds, s);
}

}  // namespace fpk
