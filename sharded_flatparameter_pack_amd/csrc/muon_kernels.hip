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
// B, which stand far above the other elements.  With D the
// diagonal of B and R the rest, X <- (a + D) X + R X_h: only R's product sees the
// rounded X.  Relative 2-norm errors of five steps
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

// ---------------------------------------------------------------- the forms of X

// Eight values, scaled, into both parts.
__device__ __forceinline__ void st_x(char* ws, int64_t h, int64_t l, int64_t at, const float x[8]) {
    uint32_t hw[4], lw[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        hw[k] = f16_pair(x[2 * k], x[2 * k + 1]);
        lw[k] = bf16x2(x[2 * k] - f16_lo(hw[k]), x[2 * k + 1] - f16_hi(hw[k]));
    }
    put16(ws + h + 2 * at, make_uint4(hw[0], hw[1], hw[2], hw[3]));
    put16(ws + l + 2 * at, make_uint4(lw[0], lw[1], lw[2], lw[3]));
}
__device__ __forceinline__ void x_of(const uint4 a, const uint4 b, float x[8]) {
    const uint32_t hw[4] = {a.x, a.y, a.z, a.w}, lw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
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

// ---------------------------------------------------------------- cast

// kCastRows x kCastCols of the padded matrix: X = U / (|U| + eps).
template <int kGrad, bool kStep>
__global__ __launch_bounds__(256) void cast_kernel(const MuonArgs a) {
    __shared__ double lds[4];
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
    const int row = t.ti * kCastRows + (threadIdx.x >> 4), col = t.tj * kCastCols + (threadIdx.x & 15) * 8;
    if (row >= r.rp || col >= r.cp) return;
    float x[8];
#pragma unroll
    for (int q = 0; q < 8; q += 4) {
        const int left = r.cols - col - q, have = row >= r.rows || left <= 0 ? 0 : left < 4 ? left : 4;
        x[q] = x[q + 1] = x[q + 2] = x[q + 3] = 0.0f;
        if (have > 0) {
            const int64_t e = (int64_t)row * r.cols + col + q;
            float g[4], m[4];
            if (!kStep || hp.nesterov) grad4<kGrad>(grad, e, have, g);
            if constexpr (kStep) ld_f32(a.momentum + r.offset + e, have, m);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < have) {
                    const double u = !kStep ? (double)g[j]
                                     : hp.nesterov ? hp.beta * (double)m[j] + mine * (double)g[j] : (double)m[j];
                    x[q + j] = (float)(u * scale) * a.s.x;
                }
        }
    }
    st_x(a.ws, r.h[0], r.l, (int64_t)row * r.cp + col, x);
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

// A = X X^T (X^T X of a tall matrix): the tiles on and below the diagonal, and
// their mirror images.
template <class S>
__global__ __launch_bounds__(S::kThreadsWg, S::kWavesSimd) void gram_kernel(const MuonArgs a) {
    extern __shared__ __align__(16) char lds[];
    if (skipped(a)) return;
    const MatTile t = a.tiles[blockIdx.x];
    if (t.mat < 0) return;
    const MuonRec& r = a.recs[t.mat];
    const Sides z = sides(r);
    const char* h = a.ws + r.h[a.step & 1];
    const int i0 = t.ti * S::kBM, j0 = t.tj * S::kBN, steps = z.n / kStepF16;
    TileProduct<S> tile;
    if (z.turned) run_tile<kColumnsF16, kColumnsF16>(tile, columns_of(h, i0, z.m), columns_of(h, j0, z.m), steps, lds);
    else run_tile<kRowsF16, kRowsF16>(tile, rows_of(h, i0, z.m, z.n), rows_of(h, j0, z.m, z.n), steps, lds);
    const float unscale = 1.0f / (a.s.x * a.s.x);
    const float out = a.s.a * unscale;
    char* to = a.ws + r.a;
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
        st_f16(to + 2 * ((int64_t)row * z.m + col), f);
    };
    if (t.ti == t.tj) {
        tile.template each<2>(lds, tile.nothing, body);
        return;
    }
    tile.template each<2, true>(lds, tile.nothing, body, tile.nothing, [&](int tr, int tc, const float* v, Nothing) {
        const int row = i0 + tr, col = j0 + tc;
        if (row >= z.m || col >= z.m) return;
        float f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = v[k] * out;
        st_f16(to + 2 * ((int64_t)col * z.m + row), f);
    });
}

// B = b A + c A^2 in the same way; db holds a + B's diagonal.  With d the
// diagonal of A and N the rest, A^2 = N^2 + (d_i + d_j) N off the diagonal.
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
    const float un_a = 1.0f / a.s.a, un_s = un_a * un_a;
    const FP_GLOBAL float* d = gptr<float>((const void*)(a.ws + r.da));
    char* to = a.ws + r.b;
    // eight elements (row, col ..) of N, with their part of the diagonals; the
    // mirror images of a tile are those of the other row, N being symmetric
    struct Fetched {
        uint4 n;
        float row;
    };
    auto fetch = [&](int row, int col) {
        Fetched f = {make_uint4(0u, 0u, 0u, 0u), 0.0f};
        if (row < z.m && col < z.m) f = {get16(n + 2 * ((int64_t)row * z.m + col)), d[row]};
        return f;
    };
    auto poly = [&](int row, int col, const float* v, const Fetched& e, const float dc[8]) {
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
        st_f16(to + 2 * ((int64_t)row * z.m + col), f);
    };
    float dc[8], dr[8];  // of the lane's columns; of the eight rows of a mirror image, per pass
#pragma unroll
    for (int k = 0; k < 8; ++k) dc[k] = j0 + tile.each_col() < z.m ? d[j0 + tile.each_col() + k] : 0.0f;
    auto body = [&](int tr, int tc, const float* v, const Fetched& e) { poly(i0 + tr, j0 + tc, v, e, dc); };
    auto straight = [&](int tr, int tc) { return fetch(i0 + tr, j0 + tc); };
    constexpr int kPer = S::kFM > 4 ? 1 : 2;  // as many registers as there are
    if (t.ti == t.tj) {
        tile.template each<kPer>(lds, straight, body);
        return;
    }
    int had = -1;
    tile.template each<kPer, true>(
        lds, straight, body, [&](int tr, int tc) { return fetch(j0 + tc, i0 + tr); },
        [&](int tr, int tc, const float* v, const Fetched& e) {
            if (tr != had) {
                had = tr;
#pragma unroll
                for (int k = 0; k < 8; ++k) dr[k] = i0 + tr < z.m ? d[i0 + tr + k] : 0.0f;
            }
            poly(j0 + tc, i0 + tr, v, e, dr);
        });
}

// How the orthogonalised matrix leaves.
enum { kGoesOn = 0, kToUpdate = 1, kToWeights = 2 };

// X <- (a + D) X + R X_h, in the matrix's own orientation: B X of a wide
// matrix, X B of a tall one.
template <class S, int kOut>
__global__ __launch_bounds__(S::kThreadsWg, S::kWavesSimd) void next_kernel(const MuonArgs a) {
    extern __shared__ __align__(16) char lds[];
    const MatTile t = a.tiles[blockIdx.x];
    if (t.mat < 0) return;
    const MuonRec& r = a.recs[t.mat];
    const Sides z = sides(r);
    const int i0 = t.ti * S::kBM, j0 = t.tj * S::kBN;
    const bool skip = skipped(a);
    if (skip && (kOut != kToWeights || r.copy == nullptr)) return;
    const char* h = a.ws + r.h[a.step & 1];
    const char* b = a.ws + r.b;
    TileProduct<S> tile;
    if (!skip) {
        const int steps = z.m / kStepF16;
        if (z.turned) run_tile<kRowsF16, kRowsF16>(tile, rows_of(h, i0, z.n, z.m), rows_of(b, j0, z.m, z.m), steps, lds);
        else run_tile<kRowsF16, kColumnsF16>(tile, rows_of(b, i0, z.m, z.m), columns_of(h, j0, z.n), steps, lds);
    }
    const float unscale = 1.0f / (a.s.b * a.s.x), un_x = 1.0f / a.s.x;
    const FP_GLOBAL float* d = gptr<float>((const void*)(a.ws + r.db));
    double rate = 0.0, decay = 1.0;
    if constexpr (kOut == kToWeights) {
        const MuonGroup& hp = a.g[r.group];
        const double rows = r.rows, cols = r.cols, most = rows > cols ? rows : cols;
        rate = hp.lr * (hp.adjust == FP_MUON_ADJUST_RMS     ? 0.2 * sqrt(most)
                        : hp.adjust == FP_MUON_ADJUST_SHAPE ? sqrt(rows > cols ? rows / cols : 1.0)
                                                            : 1.0);
        decay = hp.decay;
    }
    const int rows = kOut == kGoesOn ? r.rp : r.rows, cols = kOut == kGoesOn ? r.cp : r.cols;
    float dc[8];  // of a tall matrix: of the lane's columns
    const int c0 = j0 + tile.each_col();
#pragma unroll
    for (int k = 0; k < 8; ++k) dc[k] = !skip && z.turned && c0 < z.m ? d[c0 + k] : 0.0f;
    struct Fetched {
        uint4 h, l;
        float d;
        float w[kOut == kToWeights ? 8 : 1];
    };
    auto have_of = [&](int col, int q) { const int left = cols - col - q; return left < 4 ? left : 4; };
    // a pass ahead: two fragments' rows, or one's with the weights, which take as many registers again
    tile.template each<kOut == kToWeights ? 1 : 2>(
        lds,
        [&](int tr, int tc) {
            const int row = i0 + tr, col = j0 + tc;
            const uint4 none = make_uint4(0u, 0u, 0u, 0u);
            Fetched f;
            f.h = f.l = none;
            f.d = 0.0f;
            if (row >= rows || col >= cols) return f;
            const int64_t at = 2 * ((int64_t)row * r.cp + col);
            if (!skip) {
                f.h = get16(h + at);
                f.l = get16(a.ws + r.l + at);
                f.d = z.turned ? 0.0f : d[row];
            }
            if constexpr (kOut == kToWeights) {
#pragma unroll
                for (int q = 0; q < 8; q += 4)
                    if (have_of(col, q) > 0) ld_f32(r.master + (int64_t)row * r.cols + col + q, have_of(col, q), f.w + q);
            }
            return f;
        },
        [&](int tr, int tc, const float* v, Fetched& f) {
            const int row = i0 + tr, col = j0 + tc;
            if (row >= rows || col >= cols) return;
            float x[8];
            x_of(f.h, f.l, x);
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = __builtin_fmaf((z.turned ? dc[k] : f.d) * un_x, x[k], v[k] * unscale);
            if constexpr (kOut == kGoesOn) {
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] *= a.s.x_next;
                st_x(a.ws, r.h[(a.step + 1) & 1], r.l, (int64_t)row * r.cp + col, x);
            } else {
#pragma unroll
                for (int q = 0; q < 8; q += 4) {
                    const int have = have_of(col, q);
                    if (have <= 0) break;
                    const int64_t e = (int64_t)row * r.cols + col + q;
                    if constexpr (kOut == kToUpdate) {
                        if (a.update_dtype == FP_DTYPE_F32) st_f32(static_cast<float*>(r.update) + e, have, x + q);
                        else st_16bit(static_cast<uint16_t*>(r.update) + e, have,
                                      a.update_dtype == FP_DTYPE_F16 ? f16x4(x + q) : f32x4_to_bf16(x + q));
                    } else {
                        float* w = f.w + q;
                        if (!skip) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) w[k] = (float)(decay * (double)w[k] - rate * (double)x[q + k]);
                            st_f32(r.master + e, have, w);
                        }
                        if (r.copy != nullptr)
                            st_16bit(static_cast<uint16_t*>(r.copy) + e, have,
                                     a.copy_dtype == FP_DTYPE_F16 ? f16x4(w) : f32x4_to_bf16(w));
                    }
                }
            }
        });
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
