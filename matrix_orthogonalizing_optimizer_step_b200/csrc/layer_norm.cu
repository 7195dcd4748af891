// LayerNorm over the last dimension, forward and backward.
//
//   mu = mean(x),  r = 1 / sqrt(mean((x - mu)^2) + eps),  xh = (x - mu) r
//   y  = xh w + b
//   dx = r (q - mean(q) - xh mean(q xh)),  q = dy w
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Bound by memory: forward reads and writes rows x dim once, backward reads
// x and dy and writes dx.  A row stays in the registers of the warps that own
// it (up to 16384 elements), so each element is loaded once and the variance
// is the sum of squares about the mean, not a difference of moments.  Wider
// rows are read again from L2 for each pass.
//
// The parameter gradients are sums over all rows.  Backward CTAs are
// persistent: each adds the rows it handles into fp32 registers, writes one
// partial row pair at the end, and a second launch adds the partial rows in
// order.  The rows of a CTA and the order of the partial rows depend on the
// sizes alone, so results repeat bit for bit.
//
// Statistics and sums are fp32; outputs are rounded once.
#include "lane.h"
#include "rows.cuh"

namespace muon {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A row is held by W warps, NV groups of 8 elements per thread.  CTA: enough
// row groups for 4 warps.
template <int W>
struct RowCta {
    static constexpr int rows = W >= 4 ? 1 : 4 / W;
    static constexpr int threads = rows * W * 32;
};

// Sum of v over the W warps of this row (every thread of the CTA calls it).
template <int W>
__device__ __forceinline__ float row_sum(float v, float* red, int rg, int wr, int lane) {
    v = warp_sum(v);
    if (W == 1) return v;
    __syncthreads();  // the previous sum's readers are done
    if (lane == 0) red[rg * W + wr] = v;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) t += red[rg * W + i];
    return t;
}

// Column of element j of group i: 8 consecutive ones per thread, or (element
// access) consecutive columns across the row's threads.
template <int W, bool VEC>
__device__ __forceinline__ int row_col(int i, int j, int tr) {
    return VEC ? (i * W * 32 + tr) * 8 + j : (i * 8 + j) * W * 32 + tr;
}

template <typename T, int W, int NV, bool VEC>
__device__ __forceinline__ void load_row(const T* p, int dim, int tr, float (&v)[NV][8]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if constexpr (VEC) {
            if (row_col<W, VEC>(i, 0, tr) < dim) {
                to_float8(ld8(p + row_col<W, VEC>(i, 0, tr)), v[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = row_col<W, VEC>(i, j, tr);
                v[i][j] = c < dim ? to_float(p[c]) : 0.f;
            }
        }
    }
}

// w or b: fp32 or bf16 by p_dt (uniform), `none` where there is no such parameter
template <int W, bool VEC>
__device__ __forceinline__ void load_param(const void* p, int p_dt, int dim, int tr, int i, float none, float (&v)[8]) {
    if (!p) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = none;
        return;
    }
    if constexpr (VEC) {
        const int c = row_col<W, VEC>(i, 0, tr);
        if (c >= dim) return;
        if (p_dt == DT_F32)
            to_float8(ld8(static_cast<const float*>(p) + c), v);
        else
            to_float8(ld8(static_cast<const __nv_bfloat16*>(p) + c), v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = row_col<W, VEC>(i, j, tr);
            if (c >= dim) continue;
            v[j] = p_dt == DT_F32 ? static_cast<const float*>(p)[c]
                                  : to_float(static_cast<const __nv_bfloat16*>(p)[c]);
        }
    }
}

template <typename T, int W, bool VEC>
__device__ __forceinline__ void store_group(T* p, int dim, int tr, int i, const float (&v)[8]) {
    if constexpr (VEC) {
        const int c = row_col<W, VEC>(i, 0, tr);
        if (c < dim) st8(p + c, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = row_col<W, VEC>(i, j, tr);
            if (c < dim) st1(p + c, v[j]);
        }
    }
}

template <typename T, int W, int NV, bool VEC>
__global__ void __launch_bounds__(RowCta<W>::threads) norm_kernel(const NormFwd L) {
    __shared__ float red[W == 1 ? 1 : RowCta<W>::rows * W];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rg = warp / W, wr = warp % W, tr = wr * 32 + lane;
    const long long row = static_cast<long long>(blockIdx.x) * RowCta<W>::rows + rg;
    const bool on = row < L.rows;
    const int dim = static_cast<int>(L.dim);
    float v[NV][8];
    load_row<T, W, NV, VEC>(static_cast<const T*>(L.x) + (on ? row : 0) * L.ldx, dim, tr, v);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s += v[i][j];
    const float inv = 1.f / static_cast<float>(dim);
    const float mu = row_sum<W>(s, red, rg, wr, lane) * inv;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[i][j] -= mu;
            if (row_col<W, VEC>(i, j, tr) < dim) s = fmaf(v[i][j], v[i][j], s);
        }
    const float r = 1.f / sqrtf(row_sum<W>(s, red, rg, wr, lane) * inv + L.eps);
    if (!on) return;
    if (tr == 0) {
        L.mean[row] = mu;
        L.rstd[row] = r;
    }
    T* y = static_cast<T*>(L.y) + row * L.dim;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float w[8], b[8], o[8];
        load_param<W, VEC>(L.w, L.p_dt, dim, tr, i, 1.f, w);
        load_param<W, VEC>(L.b, L.p_dt, dim, tr, i, 0.f, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = fmaf(v[i][j] * r, w[j], b[j]);
        store_group<T, W, VEC>(y, dim, tr, i, o);
    }
}

// Backward: partial rows of this CTA at part[cta][0] (dw) and part[cta][1] (db).
template <typename T, int W, int NV, bool VEC>
__global__ void __launch_bounds__(RowCta<W>::threads) norm_grad_kernel(const NormBwd L, float* part) {
    constexpr int kRows = RowCta<W>::rows;
    __shared__ float red[W == 1 ? 1 : kRows * W];
    __shared__ float comb[kRows == 1 ? 1 : 1024];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rg = warp / W, wr = warp % W, tr = wr * 32 + lane;
    const int dim = static_cast<int>(L.dim);
    const float inv = 1.f / static_cast<float>(dim);
    float aw[NV][8], ab[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) aw[i][j] = ab[i][j] = 0.f;
    const long long step = static_cast<long long>(gridDim.x) * kRows;
    for (long long r0 = static_cast<long long>(blockIdx.x) * kRows; r0 < L.rows; r0 += step) {
        const long long row = r0 + rg;
        const bool on = row < L.rows;  // warp-uniform; every warp takes part in the sums
        const long long at = on ? row : 0;
        float x[NV][8], g[NV][8];
        load_row<T, W, NV, VEC>(static_cast<const T*>(L.x) + at * L.ldx, dim, tr, x);
        load_row<T, W, NV, VEC>(static_cast<const T*>(L.dy) + at * L.ldy, dim, tr, g);
        const float mu = L.mean[at], r = L.rstd[at];
        float sq = 0.f, sqx = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float w[8];
            load_param<W, VEC>(L.w, L.p_dt, dim, tr, i, 1.f, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (row_col<W, VEC>(i, j, tr) >= dim) continue;
                const float xh = (x[i][j] - mu) * r;
                x[i][j] = xh;
                if (on) {
                    aw[i][j] = fmaf(g[i][j], xh, aw[i][j]);
                    ab[i][j] += g[i][j];
                }
                g[i][j] *= w[j];
                sq += g[i][j];
                sqx = fmaf(g[i][j], xh, sqx);
            }
        }
        const float mq = row_sum<W>(sq, red, rg, wr, lane) * inv;
        const float mqx = row_sum<W>(sqx, red, rg, wr, lane) * inv;
        if (on) {
            T* dx = static_cast<T*>(L.dx) + row * L.dim;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = r * (g[i][j] - mq - x[i][j] * mqx);
                store_group<T, W, VEC>(dx, dim, tr, i, o);
            }
        }
    }
    // the CTA's row groups are added in order through shared memory (1024
    // columns hold any row of up to two warps), then written as one partial row
    float* pw = part + static_cast<long long>(blockIdx.x) * 2 * L.dim;
    for (int which = 0; which < 2; ++which) {
        float* dst = pw + which * L.dim;
        if constexpr (kRows > 1) {
            static_assert(W * 32 * NV * 8 <= 2048, "row groups share rows of at most 2048 columns");
            for (int half = 0; half < (W * 32 * NV * 8 + 1023) / 1024; ++half) {
                for (int k = 0; k < kRows; ++k) {
                    __syncthreads();
                    if (rg == k) {
#pragma unroll
                        for (int i = 0; i < NV; ++i)
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const int c = row_col<W, VEC>(i, j, tr) - half * 1024;
                                if (c < 0 || c >= 1024) continue;
                                const float v = which ? ab[i][j] : aw[i][j];
                                comb[c] = k == 0 ? v : comb[c] + v;
                            }
                    }
                }
                __syncthreads();
                for (int c = threadIdx.x; c < 1024 && half * 1024 + c < dim; c += RowCta<W>::threads)
                    dst[half * 1024 + c] = comb[c];
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int c = row_col<W, VEC>(i, j, tr);
                    if (c < dim) dst[c] = which ? ab[i][j] : aw[i][j];
                }
        }
    }
}

// ---- rows wider than the registers of 16 warps hold ------------------------------

constexpr int kWideThreads = 1024;

__device__ __forceinline__ float cta_sum(float v, float* red) {
    v = warp_sum(v);
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    float t = 0.f;
    for (int i = 0; i < kWideThreads / 32; ++i) t += red[i];
    return t;
}

__device__ __forceinline__ float param_at(const void* p, int p_dt, long long c, float none) {
    if (!p) return none;
    return p_dt == DT_F32 ? static_cast<const float*>(p)[c] : to_float(static_cast<const __nv_bfloat16*>(p)[c]);
}

template <typename T>
__global__ void __launch_bounds__(kWideThreads) norm_wide_kernel(const NormFwd L) {
    __shared__ float red[kWideThreads / 32];
    const long long row = blockIdx.x;
    const T* x = static_cast<const T*>(L.x) + row * L.ldx;
    const float inv = 1.f / static_cast<float>(L.dim);
    float s = 0.f;
    for (long long c = threadIdx.x; c < L.dim; c += kWideThreads) s += to_float(x[c]);
    const float mu = cta_sum(s, red) * inv;
    s = 0.f;
    for (long long c = threadIdx.x; c < L.dim; c += kWideThreads) {
        const float d = to_float(x[c]) - mu;
        s = fmaf(d, d, s);
    }
    const float r = 1.f / sqrtf(cta_sum(s, red) * inv + L.eps);
    if (threadIdx.x == 0) {
        L.mean[row] = mu;
        L.rstd[row] = r;
    }
    T* y = static_cast<T*>(L.y) + row * L.dim;
    for (long long c = threadIdx.x; c < L.dim; c += kWideThreads)
        st1(y + c, fmaf((to_float(x[c]) - mu) * r, param_at(L.w, L.p_dt, c, 1.f), param_at(L.b, L.p_dt, c, 0.f)));
}

template <typename T>
__global__ void __launch_bounds__(kWideThreads) norm_grad_wide_kernel(const NormBwd L) {
    __shared__ float red[kWideThreads / 32];
    const long long row = blockIdx.x;
    const T* x = static_cast<const T*>(L.x) + row * L.ldx;
    const T* dy = static_cast<const T*>(L.dy) + row * L.ldy;
    const float inv = 1.f / static_cast<float>(L.dim);
    const float mu = L.mean[row], r = L.rstd[row];
    float sq = 0.f, sqx = 0.f;
    for (long long c = threadIdx.x; c < L.dim; c += kWideThreads) {
        const float q = to_float(dy[c]) * param_at(L.w, L.p_dt, c, 1.f);
        sq += q;
        sqx = fmaf(q, (to_float(x[c]) - mu) * r, sqx);
    }
    const float mq = cta_sum(sq, red) * inv, mqx = cta_sum(sqx, red) * inv;
    T* dx = static_cast<T*>(L.dx) + row * L.dim;
    for (long long c = threadIdx.x; c < L.dim; c += kWideThreads) {
        const float q = to_float(dy[c]) * param_at(L.w, L.p_dt, c, 1.f);
        st1(dx + c, r * (q - mq - (to_float(x[c]) - mu) * r * mqx));
    }
}

// Parameter gradients of wide rows: CTA (x, y) adds rows y, y + gridDim.y, ... of 256 columns.
template <typename T>
__global__ void __launch_bounds__(256) norm_param_wide_kernel(const NormBwd L, float* part) {
    const long long c = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    if (c >= L.dim) return;
    float aw = 0.f, ab = 0.f;
    for (long long row = blockIdx.y; row < L.rows; row += gridDim.y) {
        const float g = to_float(static_cast<const T*>(L.dy)[row * L.ldy + c]);
        const float xh = (to_float(static_cast<const T*>(L.x)[row * L.ldx + c]) - L.mean[row]) * L.rstd[row];
        aw = fmaf(g, xh, aw);
        ab += g;
    }
    float* dst = part + static_cast<long long>(blockIdx.y) * 2 * L.dim;
    dst[c] = aw;
    dst[L.dim + c] = ab;
}

// dw (blockIdx.y = 0) and db (1): add the nparts partial rows, 32 columns per
// CTA, warp w taking rows w, w + 8, ...; the warps' sums are added in order.
constexpr int kSumWarps = 8;
__global__ void __launch_bounds__(kSumWarps * 32)
    norm_param_sum_kernel(const float* part, int nparts, long long dim, void* dw, void* db, int p_dt) {
    __shared__ float red[kSumWarps][32];
    void* out = blockIdx.y ? db : dw;
    if (!out) return;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const long long c = static_cast<long long>(blockIdx.x) * 32 + lane;
    float s = 0.f;
    if (c < dim) {
        const float* p = part + blockIdx.y * dim + c;
#pragma unroll 8
        for (int i = warp; i < nparts; i += kSumWarps) s += p[static_cast<long long>(i) * 2 * dim];
    }
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < dim) {
        s = 0.f;
        for (int w = 0; w < kSumWarps; ++w) s += red[w][lane];
        if (p_dt == DT_F32)
            static_cast<float*>(out)[c] = s;
        else
            static_cast<__nv_bfloat16*>(out)[c] = __float2bfloat16_rn(s);
    }
}

// Calls f with the row shape that holds dim: (warps per row, groups per thread).
template <int W_, int NV_>
struct Shape {
    static constexpr int W = W_, NV = NV_;
};
constexpr long long kMaxHeldDim = 16384;
template <typename F>
void with_shape(long long dim, F&& f) {
    if (dim <= 256)
        f(Shape<1, 1>{});
    else if (dim <= 512)
        f(Shape<1, 2>{});
    else if (dim <= 1024)
        f(Shape<1, 4>{});
    else if (dim <= 2048)
        f(Shape<2, 4>{});
    else if (dim <= 4096)
        f(Shape<4, 4>{});
    else if (dim <= 8192)
        f(Shape<8, 4>{});
    else
        f(Shape<16, 4>{});
}

template <typename F>
void with_type(int dt, F&& f) {
    if (dt == DT_F32)
        f(0.f);
    else
        f(__nv_bfloat16{});
}

bool param_vec_ok(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// partial row pairs of a backward pass
int backward_parts(long long rows, long long dim, int num_sms) {
    if (dim > kMaxHeldDim) return static_cast<int>(rows < 64 ? rows : 64);
    int per_cta = 1, per_sm = 4;
    with_shape(dim, [&](auto s) {
        per_cta = RowCta<decltype(s)::W>::rows;
        per_sm = decltype(s)::W <= 4 ? 3 : 1;
    });
    const long long need = (rows + per_cta - 1) / per_cta, most = static_cast<long long>(num_sms) * per_sm;
    return static_cast<int>(need < most ? need : most);
}

}  // namespace

cudaError_t launch_layer_norm(const NormFwd& L, cudaStream_t stream) {
    if (L.dim > kMaxHeldDim) {
        with_type(L.x_dt, [&](auto t) {
            norm_wide_kernel<decltype(t)><<<static_cast<unsigned>(L.rows), kWideThreads, 0, stream>>>(L);
        });
        return cudaGetLastError();
    }
    const bool vec = L.dim % 8 == 0 && rows_vec_ok(L.x, L.ldx, L.x_dt) && rows_vec_ok(L.y, L.dim, L.x_dt) &&
                     param_vec_ok(L.w) && param_vec_ok(L.b);
    with_type(L.x_dt, [&](auto t) {
        with_shape(L.dim, [&](auto s) {
            using S = decltype(s);
            using C = RowCta<S::W>;
            const unsigned grid = static_cast<unsigned>((L.rows + C::rows - 1) / C::rows);
            if (vec)
                norm_kernel<decltype(t), S::W, S::NV, true><<<grid, C::threads, 0, stream>>>(L);
            else
                norm_kernel<decltype(t), S::W, S::NV, false><<<grid, C::threads, 0, stream>>>(L);
        });
    });
    return cudaGetLastError();
}

size_t layer_norm_backward_workspace(long long rows, long long dim, int num_sms) {
    return sizeof(float) * 2 * static_cast<size_t>(backward_parts(rows, dim, num_sms)) * dim;
}

cudaError_t launch_layer_norm_backward(const NormBwd& L, int num_sms, cudaStream_t stream, int* launches) {
    const int parts = backward_parts(L.rows, L.dim, num_sms);
    float* part = static_cast<float*>(L.workspace);
    cudaError_t e = cudaSuccess;
    if (L.rows > 0) {
        if (L.dim > kMaxHeldDim) {
            with_type(L.x_dt, [&](auto t) {
                norm_grad_wide_kernel<decltype(t)><<<static_cast<unsigned>(L.rows), kWideThreads, 0, stream>>>(L);
                norm_param_wide_kernel<decltype(t)>
                    <<<dim3(static_cast<unsigned>((L.dim + 255) / 256), parts), 256, 0, stream>>>(L, part);
            });
            *launches += 2;
        } else {
            const bool vec = L.dim % 8 == 0 && rows_vec_ok(L.x, L.ldx, L.x_dt) && rows_vec_ok(L.dy, L.ldy, L.x_dt) &&
                             rows_vec_ok(L.dx, L.dim, L.x_dt) && param_vec_ok(L.w);
            with_type(L.x_dt, [&](auto t) {
                with_shape(L.dim, [&](auto s) {
                    using S = decltype(s);
                    using C = RowCta<S::W>;
                    if (vec)
                        norm_grad_kernel<decltype(t), S::W, S::NV, true><<<parts, C::threads, 0, stream>>>(L, part);
                    else
                        norm_grad_kernel<decltype(t), S::W, S::NV, false><<<parts, C::threads, 0, stream>>>(L, part);
                });
            });
            ++*launches;
        }
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (L.dw || L.db) {
        norm_param_sum_kernel<<<dim3(static_cast<unsigned>((L.dim + 31) / 32), 2), kSumWarps * 32, 0, stream>>>(
            part, parts, L.dim, L.dw, L.db, L.p_dt);
        ++*launches;
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace muon
