// muon_kernels.hip -- gfx950 kernels of the orthogonalisation of matrices by a
// Newton-Schulz iteration, and of the optimizer step that takes it.
//
// With U the momentum's matrix (or the gradient), turned in thought so that it
// has m rows, its smaller side, and n columns:
//   X = U / (|U|_F + eps);  steps times  A = X X^T,  B = b A + c A^2,
//   X <- a X + B X.
// Launches: the momentum and |U|_F^2's partial sums (moment); X in fp32 and
// fp16, both ways round (cast); for every step of the iteration A (gram), B
// (poly) and the next X (next), the last of which writes the weights.  All
// matrices of a batch share each launch.
//
// Precision.  The products run on fp16 operands with fp32 sums.  What fp16
// loses is kept small by holding apart, in fp32, what carries most: X itself,
// and the diagonals of A and B, which stand far above the other elements.  With
// D the diagonal of B and R the rest, X <- (a + D) X + R X_h, X_h in fp16:
// only R's product sees the rounded X.  Relative 2-norm errors of five steps
// against 64 bits (512 x 512: normal / singular values i^-1 / 8 of them 8 times
// the rest's norm): 7e-4 / 3e-4 / 1e-4; fp16 for everything 1.7e-3 / 3e-3 /
// 6e-3, bf16 for everything 1e-2 / 2e-2 / 5e-2 (2^-8 is 4e-3).
// Powers of two (MuonScale) keep every fp16 form in its normal range.
//
// Compiled with -ffp-contract=off.

#include "fp_matrix.h"
#include "mma_tile.h"
#include "param_ops.h"

namespace fpk {

namespace {

using Shape256 = TileShape<256, 256, 128, 64>;
using Shape128 = TileShape<128, 128, 64, 64>;
using Shape64 = TileShape<64, 64, 32, 32>;

__device__ __forceinline__ bool skipped(const MuonArgs& a) { return a.found_inf != nullptr && *a.found_inf != 0; }

__device__ __forceinline__ double sum256(double x, double* lds) {
    x = wave_sum(x);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

// Elements [e, e + have) of a gradient, have in [1, 4].
template <int kGrad>
__device__ __forceinline__ void grad4(const void* g, int64_t e, int have, float f[4]) {
    constexpr int kSize = kGrad == FP_DTYPE_F32 ? 4 : 2;
    const GradQuad<kGrad> q = have == 4 ? ld_grad<kGrad>(g, e)
                                        : ld_grad_few<kGrad>(static_cast<const char*>(g) + e * kSize, have);
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
        st16u(p, bits_of(f));
        return;
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (k < have) gptr<float>((void*)p)[k] = f[k];
}

__device__ __forceinline__ void st_16bit(void* p, int have, uint2 w) {
    if (have == 4) {
        st8u(p, w);
        return;
    }
    const uint64_t x = ((uint64_t)w.y << 32) | w.x;
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (k < have) gptr<uint16_t>(p)[k] = (uint16_t)(x >> (16 * k));
}

__device__ __forceinline__ uint2 f16x4(const float f[4]) { return make_uint2(f16x2(f[0], f[1]), f16x2(f[2], f[3])); }

// ---------------------------------------------------------------- moment

// One chunk of one matrix: the momentum m' = beta m + (1 - beta) k g, in fp64
// rounded once, and the sum of u^2 in fp64, in an order of its own.
template <int kGrad, bool kStep>
__global__ __launch_bounds__(256) void moment_kernel(const MuonArgs a) {
    __shared__ double lds[4];
    if (kStep && skipped(a)) return;
    const MatTile t = a.tiles[blockIdx.x];
    const MuonRec& r = a.recs[t.mat];
    const void* grad = a.grads[t.mat];
    const int64_t n = (int64_t)r.rows * r.cols;
    const int64_t from = r.chunk * t.ti, to = from + r.chunk < n ? from + r.chunk : n;
    const MuonGroup& hp = a.g[kStep ? r.group : 0];
    const double k = kStep && a.g_coef != nullptr ? *a.g_coef : 1.0;
    const double mine = kStep ? (1.0 - hp.beta) * k : 1.0;
    double sum = 0.0;
    for (int64_t e = from + 4 * threadIdx.x; e < to; e += 1024) {
        const int have = to - e < 4 ? (int)(to - e) : 4;
        float g[4];
        grad4<kGrad>(grad, e, have, g);
        double u[4];
        if constexpr (kStep) {
            float m[4];
            float* at = a.momentum + r.offset + e;  // room up to the next multiple of 32
            f32x4_of(ld16(at), m);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                m[i] = (float)(hp.beta * (double)m[i] + mine * (double)g[i]);
                u[i] = hp.nesterov ? hp.beta * (double)m[i] + mine * (double)g[i] : (double)m[i];
            }
            st_f32(at, have, m);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = (double)g[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < have) sum += u[i] * u[i];
    }
    sum = sum256(sum, lds);
    if (threadIdx.x == 0) gptr<double>((void*)(a.ws + r.part))[t.ti] = sum;
}

// ---------------------------------------------------------------- cast

// A 64 x 64 tile of the padded matrix: X in fp32 and in fp16 both ways round.
template <int kGrad, bool kStep>
__global__ __launch_bounds__(256) void cast_kernel(const MuonArgs a) {
    __shared__ double lds[4];
    __shared__ uint16_t turn[64][64 + 4];
    if (kStep && skipped(a)) return;
    const MatTile t = a.tiles[blockIdx.x];
    const MuonRec& r = a.recs[t.mat];
    double sum = 0.0;
    for (int i = threadIdx.x; i < r.chunks; i += 256) sum += gptr<double>((const void*)(a.ws + r.part))[i];
    const double scale = 1.0 / (sqrt(sum256(sum, lds)) + a.eps);
    const void* grad = a.grads[t.mat];
    const MuonGroup& hp = a.g[kStep ? r.group : 0];
    const double k = kStep && a.g_coef != nullptr ? *a.g_coef : 1.0;
    const double mine = kStep ? (1.0 - hp.beta) * k : 1.0;
    const bool turned = r.rows > r.cols;
    char* own = a.ws + (turned ? r.q[0] : r.p);
    char* other = a.ws + (turned ? r.p : r.q[0]);
    const int c4 = (threadIdx.x & 15) * 4, col = t.tj * 64 + c4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int lr = (threadIdx.x >> 4) + 16 * i, row = t.ti * 64 + lr;
        const int left = r.cols - col, have = row >= r.rows || left <= 0 ? 0 : left < 4 ? left : 4;
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        if (have > 0) {
            const int64_t e = (int64_t)row * r.cols + col;
            float g[4], m[4];
            if (!kStep || hp.nesterov) grad4<kGrad>(grad, e, have, g);
            if constexpr (kStep) ld_f32(a.momentum + r.offset + e, have, m);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < have) {
                    const double u = !kStep ? (double)g[j]
                                     : hp.nesterov ? hp.beta * (double)m[j] + mine * (double)g[j] : (double)m[j];
                    x[j] = (float)(u * scale);
                }
        }
        const int64_t to = (int64_t)row * r.cp + col;
        put16(a.ws + r.x + 4 * to, bits_of(x));
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] *= a.s.x;
        const uint2 h = f16x4(x);
        put8(own + 2 * to, h);
        turn[c4][lr] = (uint16_t)h.x;
        turn[c4 + 1][lr] = (uint16_t)(h.x >> 16);
        turn[c4 + 2][lr] = (uint16_t)h.y;
        turn[c4 + 3][lr] = (uint16_t)(h.y >> 16);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int lc = (threadIdx.x >> 4) + 16 * i;
        const uint16_t* from = &turn[lc][c4];
        const uint2 h = make_uint2(from[0] | (uint32_t)from[1] << 16, from[2] | (uint32_t)from[3] << 16);
        put8(other + 2 * ((int64_t)(t.tj * 64 + lc) * r.rp + t.ti * 64 + c4), h);
    }
}

// ---------------------------------------------------------------- products

struct Sides {
    int m, n;     // padded
    bool turned;
};
__device__ __forceinline__ Sides sides(const MuonRec& r) {
    const bool turned = r.rows > r.cols;
    return turned ? Sides{r.cp, r.rp, true} : Sides{r.rp, r.cp, false};
}

__device__ __forceinline__ Operand f16_rows(const char* base, int64_t row, int64_t rows, int64_t width) {
    return {base + 2 * row * width, 2 * width, (int)(rows - row), nullptr};
}

// Four elements (row, col .. col + 3) of a symmetric matrix's lower half, and
// their mirror images.
__device__ __forceinline__ void st_symmetric(char* to, int64_t side, int row, int col, uint2 h, bool mirror) {
    put8(to + 2 * (row * side + col), h);
    if (mirror) {
        FP_GLOBAL uint16_t* p = gptr<uint16_t>((void*)(to + 2 * (col * side + row)));
        p[0] = (uint16_t)h.x;
        p[side] = (uint16_t)(h.x >> 16);
        p[2 * side] = (uint16_t)h.y;
        p[3 * side] = (uint16_t)(h.y >> 16);
    }
}

// A = X X^T: the tiles on and below the diagonal, and their mirror images.
template <class S>
__global__ __launch_bounds__(S::kThreadsWg) void gram_kernel(const MuonArgs a) {
    extern __shared__ __align__(16) char lds[];
    if (skipped(a)) return;
    const MatTile t = a.tiles[die_tile(blockIdx.x, a.n_tiles)];
    const MuonRec& r = a.recs[t.mat];
    const Sides z = sides(r);
    const char* p = a.ws + r.p;
    const int i0 = t.ti * S::kBM, j0 = t.tj * S::kBN;
    TileProduct<S, false> tile;
    tile.run(f16_rows(p, i0, z.m, z.n), f16_rows(p, j0, z.m, z.n), z.n / 64, lds);
    const float unscale = 1.0f / (a.s.x * a.s.x);
    const float out = a.s.a * unscale;
#pragma unroll
    for (int fm = 0; fm < S::kFM; ++fm) {
        const int row = i0 + tile.row0() + 16 * fm;
        if (row >= z.m) continue;
#pragma unroll
        for (int fn = 0; fn < S::kFN; ++fn) {
            const int col = j0 + tile.col0() + 16 * fn;
            if (col >= z.m) continue;
            float f[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                f[q] = tile.acc[fm][fn][q] * out;
                if (row == col + q) {
                    gptr<float>((void*)(a.ws + r.da))[row] = tile.acc[fm][fn][q] * unscale;
                    f[q] = 0.0f;
                }
            }
            st_symmetric(a.ws + r.a, z.m, row, col, f16x4(f), t.ti != t.tj);
        }
    }
}

// B = b A + c A^2 in the same way; db holds a + B's diagonal.  With d the
// diagonal of A and N the rest, A^2 = N^2 + (d_i + d_j) N off the diagonal.
template <class S>
__global__ __launch_bounds__(S::kThreadsWg) void poly_kernel(const MuonArgs a) {
    extern __shared__ __align__(16) char lds[];
    if (skipped(a)) return;
    const MatTile t = a.tiles[die_tile(blockIdx.x, a.n_tiles)];
    const MuonRec& r = a.recs[t.mat];
    const Sides z = sides(r);
    const char* p = a.ws + r.a;
    const int i0 = t.ti * S::kBM, j0 = t.tj * S::kBN;
    TileProduct<S, false> tile;
    tile.run(f16_rows(p, i0, z.m, z.m), f16_rows(p, j0, z.m, z.m), z.m / 64, lds);
    const float un_a = 1.0f / a.s.a, un_s = un_a * un_a;
    const FP_GLOBAL float* d = gptr<float>((const void*)(a.ws + r.da));
#pragma unroll
    for (int fm = 0; fm < S::kFM; ++fm) {
        const int row = i0 + tile.row0() + 16 * fm;
        if (row >= z.m) continue;
        const float di = d[row];
#pragma unroll
        for (int fn = 0; fn < S::kFN; ++fn) {
            const int col = j0 + tile.col0() + 16 * fn;
            if (col >= z.m) continue;
            const uint2 w = get8(p + 2 * ((int64_t)row * z.m + col));
            const float n[4] = {f16_lo(w.x), f16_hi(w.x), f16_lo(w.y), f16_hi(w.y)};
            float f[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float square = tile.acc[fm][fn][q] * un_s, x = n[q] * un_a;
                f[q] = (a.cb * x + a.cc * (square + (di + d[col + q]) * x)) * a.s.b;
                if (row == col + q) {
                    gptr<float>((void*)(a.ws + r.db))[row] = a.ca + (a.cb * di + a.cc * (square + di * di));
                    f[q] = 0.0f;
                }
            }
            st_symmetric(a.ws + r.b, z.m, row, col, f16x4(f), t.ti != t.tj);
        }
    }
}

// How the orthogonalised matrix leaves.
enum { kGoesOn = 0, kToUpdate = 1, kToWeights = 2 };

// X <- (a + D) X + R X_h, in the matrix's own orientation: B X of a wide
// matrix, X B of a tall one.
template <class S, int kOut>
__global__ __launch_bounds__(S::kThreadsWg) void next_kernel(const MuonArgs a) {
    extern __shared__ __align__(16) char lds[];
    const MatTile t = a.tiles[die_tile(blockIdx.x, a.n_tiles)];
    const MuonRec& r = a.recs[t.mat];
    const Sides z = sides(r);
    const int i0 = t.ti * S::kBM, j0 = t.tj * S::kBN;
    const bool skip = skipped(a);
    if (kOut == kToWeights ? skip && r.copy == nullptr : skip) return;
    const char* q = a.ws + r.q[a.step & 1];
    const char* b = a.ws + r.b;
    TileProduct<S, false> tile;
    if (!(kOut == kToWeights && skip)) {
        if (z.turned) tile.run(f16_rows(q, i0, r.rp, z.m), f16_rows(b, j0, z.m, z.m), z.m / 64, lds);
        else tile.run(f16_rows(b, i0, z.m, z.m), f16_rows(q, j0, r.cp, z.m), z.m / 64, lds);
    } else {
        tile.lane = threadIdx.x & 63;
        tile.wave = threadIdx.x >> 6;
    }
    const float unscale = 1.0f / (a.s.b * a.s.x);
    const FP_GLOBAL float* d = gptr<float>((const void*)(a.ws + r.db));
    char* own = a.ws + (z.turned ? r.q[(a.step + 1) & 1] : r.p);
    char* other = a.ws + (z.turned ? r.p : r.q[(a.step + 1) & 1]);
    double rate = 0.0, decay = 1.0;
    if constexpr (kOut == kToWeights) {
        const MuonGroup& hp = a.g[r.group];
        const double rows = r.rows, cols = r.cols, most = rows > cols ? rows : cols;
        rate = hp.lr * (hp.adjust == FP_MUON_ADJUST_RMS     ? 0.2 * sqrt(most)
                        : hp.adjust == FP_MUON_ADJUST_SHAPE ? sqrt(rows > cols ? rows / cols : 1.0)
                                                            : 1.0);
        decay = hp.decay;
    }
#pragma unroll
    for (int fm = 0; fm < S::kFM; ++fm) {
        const int row = i0 + tile.row0() + 16 * fm;
        if (row >= (kOut == kGoesOn ? r.rp : r.rows)) continue;
#pragma unroll
        for (int fn = 0; fn < S::kFN; ++fn) {
            const int col = j0 + tile.col0() + 16 * fn;
            if (col >= (kOut == kGoesOn ? r.cp : r.cols)) continue;
            const int64_t at = (int64_t)row * r.cp + col;
            float x[4] = {0.f, 0.f, 0.f, 0.f};
            if (!(kOut == kToWeights && skip)) {
                f32x4_of(get16(a.ws + r.x + 4 * at), x);
#pragma unroll
                for (int k = 0; k < 4; ++k) x[k] = d[z.turned ? col + k : row] * x[k] + tile.acc[fm][fn][k] * unscale;
            }
            if constexpr (kOut == kGoesOn) {
                put16(a.ws + r.x + 4 * at, bits_of(x));
#pragma unroll
                for (int k = 0; k < 4; ++k) x[k] *= a.s.x_next;
                const uint2 h = f16x4(x);
                put8(own + 2 * at, h);
                FP_GLOBAL uint16_t* o = gptr<uint16_t>((void*)(other + 2 * ((int64_t)col * r.rp + row)));
                o[0] = (uint16_t)h.x;
                o[r.rp] = (uint16_t)(h.x >> 16);
                o[2 * (int64_t)r.rp] = (uint16_t)h.y;
                o[3 * (int64_t)r.rp] = (uint16_t)(h.y >> 16);
            } else {
                const int have = r.cols - col < 4 ? r.cols - col : 4;
                const int64_t e = (int64_t)row * r.cols + col;
                if constexpr (kOut == kToUpdate) {
                    if (a.update_dtype == FP_DTYPE_F32) st_f32(static_cast<float*>(r.update) + e, have, x);
                    else st_16bit(static_cast<uint16_t*>(r.update) + e, have,
                                  a.update_dtype == FP_DTYPE_F16 ? f16x4(x) : f32x4_to_bf16(x));
                } else {
                    float w[4];
                    ld_f32(r.master + e, have, w);
                    if (!skip) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) w[k] = (float)(decay * (double)w[k] - rate * (double)x[k]);
                        st_f32(r.master + e, have, w);
                    }
                    if (r.copy != nullptr)
                        st_16bit(static_cast<uint16_t*>(r.copy) + e, have,
                                 a.copy_dtype == FP_DTYPE_F16 ? f16x4(w) : f32x4_to_bf16(w));
                }
            }
        }
    }
}

// Launches kernel(a) over the argument block's tiles.
template <class K>
hipError_t launch(K kernel, const MuonArgs& a, int threads, unsigned lds, hipStream_t s) {
    if (lds > 65536u) {  // beyond 64 KiB dynamic LDS is asked for once per kernel and device
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    kernel<<<(unsigned)a.n_tiles, threads, lds, s>>>(a);
    return hipGetLastError();
}


}  // namespace

hipError_t launch_muon_moment(const MuonArgs& a, hipStream_t s) {
#define FP_MOMENT(G) (a.momentum != nullptr ? launch(moment_kernel<G, true>, a, 256, 0, s) : launch(moment_kernel<G, false>, a, 256, 0, s))
    return a.grad_dtype == FP_DTYPE_F32 ? FP_MOMENT(FP_DTYPE_F32) : a.grad_dtype == FP_DTYPE_BF16 ? FP_MOMENT(FP_DTYPE_BF16) : FP_MOMENT(FP_DTYPE_F16);
#undef FP_MOMENT
}

hipError_t launch_muon_cast(const MuonArgs& a, hipStream_t s) {
#define FP_CAST(G) (a.momentum != nullptr ? launch(cast_kernel<G, true>, a, 256, 0, s) : launch(cast_kernel<G, false>, a, 256, 0, s))
    return a.grad_dtype == FP_DTYPE_F32 ? FP_CAST(FP_DTYPE_F32) : a.grad_dtype == FP_DTYPE_BF16 ? FP_CAST(FP_DTYPE_BF16) : FP_CAST(FP_DTYPE_F16);
#undef FP_CAST
}

hipError_t launch_muon_gram(const MuonArgs& a, int shape, hipStream_t s) {
    return shape == kTile256   ? launch(gram_kernel<Shape256>, a, Shape256::kThreadsWg, Shape256::kLds, s)
           : shape == kTile128 ? launch(gram_kernel<Shape128>, a, Shape128::kThreadsWg, Shape128::kLds, s)
                               : launch(gram_kernel<Shape64>, a, Shape64::kThreadsWg, Shape64::kLds, s);
}

hipError_t launch_muon_poly(const MuonArgs& a, int shape, hipStream_t s) {
    return shape == kTile256   ? launch(poly_kernel<Shape256>, a, Shape256::kThreadsWg, Shape256::kLds, s)
           : shape == kTile128 ? launch(poly_kernel<Shape128>, a, Shape128::kThreadsWg, Shape128::kLds, s)
                               : launch(poly_kernel<Shape64>, a, Shape64::kThreadsWg, Shape64::kLds, s);
}

template <int kOut>
static hipError_t launch_next(const MuonArgs& a, int shape, hipStream_t s) {
    return shape == kTile256   ? launch(next_kernel<Shape256, kOut>, a, Shape256::kThreadsWg, Shape256::kLds, s)
           : shape == kTile128 ? launch(next_kernel<Shape128, kOut>, a, Shape128::kThreadsWg, Shape128::kLds, s)
                               : launch(next_kernel<Shape64, kOut>, a, Shape64::kThreadsWg, Shape64::kLds, s);
}

hipError_t launch_muon_next(const MuonArgs& a, int shape, bool last, bool to_weights, hipStream_t s) {
    return !last ? launch_next<kGoesOn>(a, shape, s) : to_weights ? launch_next<kToWeights>(a, shape, s) : launch_next<kToUpdate>(a, shape, s);
}

}  // namespace fpk
