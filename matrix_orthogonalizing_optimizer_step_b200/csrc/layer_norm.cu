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
// is the sum of squares about the mean, not a difference of moments.  CTAs are
// persistent and copy the rows to come into shared memory while they work on
// one: a row's two sums are a chain of latencies, and without the copies in
// flight the loads wait for it.  Wider rows are read again from L2 for each pass.
//
// The parameter gradients are sums over all rows: a backward CTA adds the rows
// it handles into fp32 registers, writes one partial row pair at the end, and
// a second launch adds the partial rows in order.  The rows of a CTA and the
// order of the partial rows depend on the sizes alone, so results repeat bit
// for bit.
//
// Statistics and sums are fp32; outputs are rounded once.
//
// Measured (bf16; calls behind one another on changing inputs, in brackets
// replayed from a graph on one input, which L2 then holds): forward 16384 x 4096
// 52 us (46: 268 MB, 5.2-5.8 TB/s), 16 x 4096 6.5 us (2.5); backward 16384 x 768 with
// fp32 parameters 20.5 us (15.5; 75 MB, 11.7 us at the copy rate: rows' chains of
// latencies and the second launch), 4099 x 1025 fp32 19.3 us (16.4; 50 MB, 7.8 us:
// 4-byte copies, and a third of the rows' 1536 places empty).
#include <atomic>

#include "lane.h"
#include "pdl.h"
#include "rows.cuh"

namespace muon {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A row is held by W warps, NU units of 16 bytes per thread.  CTA: enough row
// groups for 4 warps.
template <int W>
struct RowCta {
    static constexpr int rows = W >= 4 ? 1 : 4 / W;
    static constexpr int threads = rows * W * 32;
};

// How a thread reads its units.  VEC: 16-byte copies into shared memory, ahead
// of their use.  ELEM4: the same with 4-byte copies (fp32 rows that do not
// start on 16-byte boundaries, or whose width is not a multiple of the unit).
// DIRECT: element loads when the row is due (bf16 rows of that kind, and rows
// whose copies would not fit).
enum Access { VEC = 0, ELEM4 = 1, DIRECT = 2 };

#pragma nv_diag_suppress 177  // members that an instance does not use
template <typename T, int W_, int NU_, int ACCESS_, int ARRAYS>
struct RowShape {
    static constexpr int W = W_, NU = NU_, ACCESS = ACCESS_;
    static constexpr int VL = 16 / sizeof(T);            // elements of a unit
    static constexpr int NE = NU * VL;                    // elements per thread
    // the parameters stay in registers; threads with more elements read them
    // again for every row (a row of fp32 parameters costs L1 as much as two
    // rows of bf16), and so do CTAs of 512 threads backward, which have 128
    // registers a thread
    static constexpr bool keep = NE <= 24 && !(ARRAYS == 2 && W == 16);
    static constexpr int threads = RowCta<W>::threads;
    static constexpr int stage_bytes = ARRAYS * NU * threads * 16;
    // rows in flight per row group, in about 48 KB per CTA: up to 3 forward
    // (16384 x 4096 bf16: 47.5 us; 2: 49.9, 4: 49.0), 2 backward, where the
    // registers hold more (16384 x 768, two inputs in a loop: 19.0 us; 3 and 4: 20.5)
    static constexpr int fit = 49152 / stage_bytes, most = ARRAYS == 1 ? 3 : 2;
    static constexpr int stages = ACCESS == DIRECT ? 0 : (fit > most ? most : (fit < 2 ? 2 : fit));
    // the ring, or the sums of a backward CTA's row groups
    static constexpr int comb_bytes = ARRAYS == 2 && RowCta<W>::rows > 1 ? RowCta<W>::rows * 2 * W * 32 * NE * 4 : 0;
    static constexpr int ring_bytes = stages * stage_bytes;
    static constexpr int smem = ring_bytes > comb_bytes ? ring_bytes : comb_bytes;
};

// Column of element j of unit u: a unit's elements are consecutive for one
// thread (VEC) or lie one row group apart (coalesced element access).
template <class S>
__device__ __forceinline__ int row_col(int u, int j, int tr) {
    return S::ACCESS == VEC ? (u * S::W * 32 + tr) * S::VL + j : (u * S::VL + j) * S::W * 32 + tr;
}

__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// This thread's units of a row, copied to its own slots of stage memory (a
// thread reads only what it copied itself, so no barrier is involved).
template <typename T, class S>
__device__ __forceinline__ void copy_row(uint32_t slot, const T* p, int dim, int tr) {
#pragma unroll
    for (int u = 0; u < S::NU; ++u) {
        const uint32_t dst = slot + u * S::threads * 16;
        if (S::ACCESS == VEC) {
            const int c = row_col<S>(u, 0, tr);
            if (c < dim) copy_async16(dst, p + c);
        } else {
#pragma unroll
            for (int j = 0; j < S::VL; ++j) {
                const int c = row_col<S>(u, j, tr);
                if (c < dim) copy_async4(dst + 4 * j, p + c);
            }
        }
    }
}

// Units of this thread as floats, `none` behind the last column.
template <typename T, class S>
__device__ __forceinline__ void read_row(const uint4* slot, const T* p, int dim, int tr, float (&v)[S::NU][S::VL],
                                         float none = 0.f) {
#pragma unroll
    for (int u = 0; u < S::NU; ++u) {
        if (S::ACCESS == DIRECT) {
#pragma unroll
            for (int j = 0; j < S::VL; ++j) {
                const int c = row_col<S>(u, j, tr);
                v[u][j] = c < dim ? to_float(p[c]) : none;
            }
        } else {
            const uint4 raw = slot[u * S::threads];
            const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
            for (int j = 0; j < S::VL; ++j) {
                const bool in = row_col<S>(u, S::ACCESS == VEC ? 0 : j, tr) < dim;
                float f;
                if (S::VL == 4)
                    f = __uint_as_float(w[j & 3]);
                else
                    f = __uint_as_float((j & 1) ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
                v[u][j] = in ? f : none;
            }
        }
    }
}

// A unit of w or b: fp32 or bf16 by p_dt (uniform), `none` where there is no such parameter.
template <class S>
__device__ __forceinline__ void load_param(const void* p, int p_dt, int dim, int tr, int u, float none,
                                           float (&v)[S::VL]) {
#pragma unroll
    for (int j = 0; j < S::VL; ++j) v[j] = none;
    if (!p) return;
    if constexpr (S::ACCESS == VEC) {
        const int c = row_col<S>(u, 0, tr);
        if (c >= dim) return;
        if (p_dt == DT_F32) {
            const float* f = static_cast<const float*>(p) + c;
#pragma unroll
            for (int q = 0; q < S::VL / 4; ++q) {
                const float4 a = *reinterpret_cast<const float4*>(f + 4 * q);
                v[4 * q] = a.x, v[4 * q + 1] = a.y, v[4 * q + 2] = a.z, v[4 * q + 3] = a.w;
            }
        } else {
            const __nv_bfloat16* h = static_cast<const __nv_bfloat16*>(p) + c;
#pragma unroll
            for (int q = 0; q < S::VL / 4; ++q) {
                const uint2 a = *reinterpret_cast<const uint2*>(h + 4 * q);
                v[4 * q] = __uint_as_float(a.x << 16), v[4 * q + 1] = __uint_as_float(a.x & 0xffff0000u);
                v[4 * q + 2] = __uint_as_float(a.y << 16), v[4 * q + 3] = __uint_as_float(a.y & 0xffff0000u);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < S::VL; ++j) {
            const int c = row_col<S>(u, j, tr);
            if (c >= dim) continue;
            v[j] = p_dt == DT_F32 ? static_cast<const float*>(p)[c]
                                  : to_float(static_cast<const __nv_bfloat16*>(p)[c]);
        }
    }
}

template <typename T, class S>
__device__ __forceinline__ void store_unit(T* p, int dim, int tr, int u, const float (&v)[S::VL]) {
    if constexpr (S::ACCESS == VEC) {
        const int c = row_col<S>(u, 0, tr);
        if (c >= dim) return;
        if constexpr (S::VL == 8)
            st8(p + c, v);
        else
            *reinterpret_cast<float4*>(p + c) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int j = 0; j < S::VL; ++j) {
            const int c = row_col<S>(u, j, tr);
            if (c < dim) st1(p + c, v[j]);
        }
    }
}

// Sum over the W warps of this row.  With W > 1 every thread of the CTA calls
// it; two buffers take turns, so that one barrier per sum is enough (a buffer
// is written again two sums later, behind the barrier between).
template <int W, int N>
struct RowSum {
    static constexpr int slots = RowCta<W>::rows * W;
    float (*red)[slots][N];  // [2][slots][N] in shared memory
    int turn = 0;
    __device__ __forceinline__ void operator()(float (&v)[N], int rg, int wr, int lane) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
        if (W == 1) return;
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < N; ++k) red[turn][rg * W + wr][k] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) {
            v[k] = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) v[k] += red[turn][rg * W + i][k];
        }
        turn ^= 1;
    }
};

// Persistent CTAs: row groups take rows g, g + G, ... (G row groups in the
// grid) and keep S::stages - 1 later rows on their way while they work on one.
template <typename T, class S>
__global__ void __launch_bounds__(S::threads) norm_kernel(const NormFwd L) {
    constexpr int W = S::W, kRows = RowCta<W>::rows;
    extern __shared__ uint4 ring[];
    __shared__ float red[2][kRows * W][1];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rg = warp / W, wr = warp % W, tr = wr * 32 + lane;
    const int dim = static_cast<int>(L.dim);
    const float inv = 1.f / static_cast<float>(dim);
    const T* x = static_cast<const T*>(L.x);
    const long long step = static_cast<long long>(gridDim.x) * kRows;
    const long long first = static_cast<long long>(blockIdx.x) * kRows;  // row of the CTA's first row group
    auto slot = [&](int st) { return ring + st * (S::stage_bytes / 16) + threadIdx.x; };
    auto fetch = [&](long long r0, int st) {
        if (S::stages > 0) {
            if (r0 + rg < L.rows)
                copy_row<T, S>(static_cast<uint32_t>(__cvta_generic_to_shared(slot(st))), x + (r0 + rg) * L.ldx, dim, tr);
            copy_commit();
        }
    };
    constexpr int kAhead = S::stages > 0 ? S::stages - 1 : 0;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(first + i * step, i);
    RowSum<W, 1> sum{red};
    constexpr int kKept = S::keep ? S::NU : 1;
    float wk[kKept][S::VL], bk[kKept][S::VL];
    if (S::keep) {
#pragma unroll
        for (int u = 0; u < kKept; ++u) {
            load_param<S>(L.w, L.p_dt, dim, tr, u, 1.f, wk[u]);
            load_param<S>(L.b, L.p_dt, dim, tr, u, 0.f, bk[u]);
        }
    }
    int st = 0;
    for (long long r0 = first; r0 < L.rows; r0 += step) {
        const long long row = r0 + rg;
        const bool on = row < L.rows;  // warp-uniform; every warp takes part in the sums
        if (S::stages > 0) {
            fetch(r0 + kAhead * step, st == 0 ? S::stages - 1 : st - 1);
            copy_wait<kAhead>();
        }
        float v[S::NU][S::VL];
        read_row<T, S>(slot(st), x + (on ? row : 0) * L.ldx, dim, tr, v);
        if (S::stages > 0 && ++st == S::stages) st = 0;
        // each unit's sum is a chain of its own
        float s[1], su[S::NU];
#pragma unroll
        for (int u = 0; u < S::NU; ++u) {
            su[u] = v[u][0];
#pragma unroll
            for (int j = 1; j < S::VL; ++j) su[u] += v[u][j];
        }
        s[0] = su[0];
#pragma unroll
        for (int u = 1; u < S::NU; ++u) s[0] += su[u];
        sum(s, rg, wr, lane);
        const float mu = s[0] * inv;
#pragma unroll
        for (int u = 0; u < S::NU; ++u) {
            su[u] = 0.f;
#pragma unroll
            for (int j = 0; j < S::VL; ++j) {
                v[u][j] -= mu;
                if (row_col<S>(u, S::ACCESS == VEC ? 0 : j, tr) < dim) su[u] = fmaf(v[u][j], v[u][j], su[u]);
            }
        }
        s[0] = su[0];
#pragma unroll
        for (int u = 1; u < S::NU; ++u) s[0] += su[u];
        sum(s, rg, wr, lane);
        const float r = 1.f / sqrtf(s[0] * inv + L.eps);
        if (!on) continue;
        if (tr == 0) {
            L.mean[row] = mu;
            L.rstd[row] = r;
        }
        T* y = static_cast<T*>(L.y) + row * L.dim;
#pragma unroll
        for (int u = 0; u < S::NU; ++u) {
            float o[S::VL];
            float(&w)[S::VL] = wk[S::keep ? u : 0];
            float(&b)[S::VL] = bk[S::keep ? u : 0];
            if (!S::keep) {
                load_param<S>(L.w, L.p_dt, dim, tr, u, 1.f, w);
                load_param<S>(L.b, L.p_dt, dim, tr, u, 0.f, b);
            }
#pragma unroll
            for (int j = 0; j < S::VL; ++j) o[j] = fmaf(v[u][j] * r, w[j], b[j]);
            store_unit<T, S>(y, dim, tr, u, o);
        }
    }
    if (S::stages > 0) copy_wait<0>();
}

// Backward, persistent in the same way: partial rows of this CTA at
// part[cta][0] (dw) and part[cta][1] (db).
template <typename T, class S>
__global__ void __launch_bounds__(S::threads) norm_grad_kernel(const NormBwd L, float* part) {
    constexpr int W = S::W, kRows = RowCta<W>::rows;
    extern __shared__ uint4 ring[];
    __shared__ float red[2][kRows * W][2];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rg = warp / W, wr = warp % W, tr = wr * 32 + lane;
    allow_successor();
    const int dim = static_cast<int>(L.dim);
    const float inv = 1.f / static_cast<float>(dim);
    const T* x = static_cast<const T*>(L.x);
    const T* dy = static_cast<const T*>(L.dy);
    float aw[S::NU][S::VL], ab[S::NU][S::VL];
#pragma unroll
    for (int u = 0; u < S::NU; ++u)
#pragma unroll
        for (int j = 0; j < S::VL; ++j) aw[u][j] = ab[u][j] = 0.f;
    const long long step = static_cast<long long>(gridDim.x) * kRows;
    const long long first = static_cast<long long>(blockIdx.x) * kRows;
    auto slot = [&](int st, int a) { return ring + st * (S::stage_bytes / 16) + a * S::NU * S::threads + threadIdx.x; };
    auto fetch = [&](long long r0, int st) {
        if (S::stages > 0) {
            const long long row = r0 + rg;
            if (row < L.rows) {
                copy_row<T, S>(static_cast<uint32_t>(__cvta_generic_to_shared(slot(st, 0))), x + row * L.ldx, dim, tr);
                copy_row<T, S>(static_cast<uint32_t>(__cvta_generic_to_shared(slot(st, 1))), dy + row * L.ldy, dim, tr);
            }
            copy_commit();
        }
    };
    constexpr int kAhead = S::stages > 0 ? S::stages - 1 : 0;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(first + i * step, i);
    RowSum<W, 2> sum{red};
    constexpr int kKept = S::keep ? S::NU : 1;
    float wk[kKept][S::VL];
    if (S::keep) {
#pragma unroll
        for (int u = 0; u < kKept; ++u) load_param<S>(L.w, L.p_dt, dim, tr, u, 1.f, wk[u]);
    }
    int st = 0;
    float mu = 0.f, r = 0.f;
    if (first + rg < L.rows) mu = L.mean[first + rg], r = L.rstd[first + rg];
    for (long long r0 = first; r0 < L.rows; r0 += step) {
        const long long row = r0 + rg;
        const bool on = row < L.rows;  // warp-uniform; every warp takes part in the sums
        const long long at = on ? row : 0;
        float mu_next = 0.f, r_next = 0.f;
        if (row + step < L.rows) mu_next = L.mean[row + step], r_next = L.rstd[row + step];
        if (S::stages > 0) {
            fetch(r0 + kAhead * step, st == 0 ? S::stages - 1 : st - 1);
            copy_wait<kAhead>();
        }
        float xv[S::NU][S::VL], g[S::NU][S::VL];
        read_row<T, S>(slot(st, 0), x + at * L.ldx, dim, tr, xv, mu);
        read_row<T, S>(slot(st, 1), dy + at * L.ldy, dim, tr, g);
        if (S::stages > 0 && ++st == S::stages) st = 0;
        float s[2] = {0.f, 0.f};
        if (on) {
            float s0[S::NU], s1[S::NU];  // each unit's sums are chains of their own
#pragma unroll
            for (int u = 0; u < S::NU; ++u) {
                s0[u] = s1[u] = 0.f;
                float(&w)[S::VL] = wk[S::keep ? u : 0];
                if (!S::keep) load_param<S>(L.w, L.p_dt, dim, tr, u, 1.f, w);
#pragma unroll
                for (int j = 0; j < S::VL; ++j) {
                    // columns behind the last hold x = mu and g = 0: they add
                    // nothing, however large mu and r are
                    const float xh = (xv[u][j] - mu) * r;
                    xv[u][j] = xh;
                    aw[u][j] = fmaf(g[u][j], xh, aw[u][j]);
                    ab[u][j] += g[u][j];
                    g[u][j] *= w[j];
                    s0[u] += g[u][j];
                    s1[u] = fmaf(g[u][j], xh, s1[u]);
                }
                s[0] += s0[u];
                s[1] += s1[u];
            }
        }
        sum(s, rg, wr, lane);
        if (on) {
            const float mq = s[0] * inv, mqx = s[1] * inv;
            T* dx = static_cast<T*>(L.dx) + row * L.dim;
#pragma unroll
            for (int u = 0; u < S::NU; ++u) {
                float o[S::VL];
#pragma unroll
                for (int j = 0; j < S::VL; ++j) o[j] = r * (g[u][j] - mq - xv[u][j] * mqx);
                store_unit<T, S>(dx, dim, tr, u, o);
            }
        }
        mu = mu_next;
        r = r_next;
    }
    if (S::stages > 0) copy_wait<0>();
    // the CTA's row groups are added in order through shared memory (the ring
    // is free: every thread has used its last row), then written as one partial row
    float* pw = part + static_cast<long long>(blockIdx.x) * 2 * L.dim;
    if constexpr (kRows > 1) {
        constexpr int kCols = W * 32 * S::NE;
        float* comb = reinterpret_cast<float*>(ring);  // [row group][dw, db][kCols]
        __syncthreads();
#pragma unroll
        for (int u = 0; u < S::NU; ++u)
#pragma unroll
            for (int j = 0; j < S::VL; ++j) {
                const int c = row_col<S>(u, j, tr);
                comb[rg * 2 * kCols + c] = aw[u][j];
                comb[rg * 2 * kCols + kCols + c] = ab[u][j];
            }
        __syncthreads();
        for (int c = threadIdx.x; c < dim; c += S::threads) {
            float a = comb[c], b = comb[kCols + c];
#pragma unroll
            for (int k = 1; k < kRows; ++k) {
                a += comb[k * 2 * kCols + c];
                b += comb[k * 2 * kCols + kCols + c];
            }
            pw[c] = a;
            pw[L.dim + c] = b;
        }
    } else {
#pragma unroll
        for (int u = 0; u < S::NU; ++u)
#pragma unroll
            for (int j = 0; j < S::VL; ++j) {
                const int c = row_col<S>(u, j, tr);
                if (c >= dim) continue;
                pw[c] = aw[u][j];
                pw[L.dim + c] = ab[u][j];
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
// CTA, warp w taking rows w, w + 32, ...; the warps' sums are added in order.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(kSumWarps * 32)
    norm_param_sum_kernel(const float* part, int nparts, long long dim, void* dw, void* db, int p_dt) {
    __shared__ float red[kSumWarps][32];
    void* out = blockIdx.y ? db : dw;
    wait_predecessor();
    if (!out) return;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const long long c = static_cast<long long>(blockIdx.x) * 32 + lane;
    float s = 0.f;
    if (c < dim) {
        const float* p = part + (2ll * warp + blockIdx.y) * dim + c;
        const long long step = 2ll * kSumWarps * dim;
        // two CTAs' rows per SM in one trip to L2; the addresses are stepped, since a
        // kernel this short waits for its own code (a product per load: 18.8 and
        // 17.1 instead of 16.2 us for the whole backward pass of 4099 x 1025 and
        // 16384 x 768 replayed from a graph; eight loads at a time with a remainder
        // loop 17.1 and 17.3)
        constexpr int kAhead = 10;
#pragma unroll 1
        for (int left = nparts - warp; left > 0; left -= kAhead * kSumWarps) {
            float v[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                v[k] = left > k * kSumWarps ? *p : 0.f;
                p += step;
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) s += v[k];
        }
    }
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < dim) {
        s = 0.f;
#pragma unroll
        for (int w = 0; w < kSumWarps; ++w) s += red[w][lane];
        if (p_dt == DT_F32)
            static_cast<float*>(out)[c] = s;
        else
            static_cast<__nv_bfloat16*>(out)[c] = __float2bfloat16_rn(s);
    }
}

// Calls f with the row shape that holds dim: W warps per row and G groups of 8
// elements per thread, W the smallest power of two for which 2 or 3 groups do
// (one warp takes a single group too, and 16 warps four).
template <int W_, int G_>
struct Hold {
    static constexpr int W = W_, G = G_;
};
constexpr long long kMaxHeldDim = 16384;
template <typename F>
void with_hold(long long dim, F&& f) {
    const long long g = (dim + 255) / 256;  // groups of one warp
    if (g <= 1)
        f(Hold<1, 1>{});
    else if (g <= 2)
        f(Hold<1, 2>{});
    else if (g <= 3)
        f(Hold<1, 3>{});
    else if (g <= 4)
        f(Hold<2, 2>{});
    else if (g <= 6)
        f(Hold<2, 3>{});
    else if (g <= 8)
        f(Hold<4, 2>{});
    else if (g <= 12)
        f(Hold<4, 3>{});
    else if (g <= 16)
        f(Hold<8, 2>{});
    else if (g <= 24)
        f(Hold<8, 3>{});
    else if (g <= 32)
        f(Hold<16, 2>{});
    else if (g <= 48)
        f(Hold<16, 3>{});
    else
        f(Hold<16, 4>{});
}

template <typename F>
void with_type(int dt, F&& f) {
    if (dt == DT_F32)
        f(0.f);
    else
        f(__nv_bfloat16{});
}

bool param_vec_ok(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Partial row pairs that a backward pass may leave: one per CTA of a grid of
// at most kPartsPerSm CTAs per SM.
constexpr int kPartsPerSm = 4;
int backward_parts_bound(long long rows, int num_sms) {
    const long long most = static_cast<long long>(num_sms) * kPartsPerSm;
    return static_cast<int>(rows < most ? rows : most);
}

// CTAs of a persistent launch: what the row groups need, and no more than are
// resident at once (asked once per instance: a property of the build).
template <typename K>
cudaError_t persistent_grid(K kernel, int threads, int smem, int num_sms, std::atomic<int>& resident, long long need, int most_per_sm,
                            unsigned& grid) {
    // above the 48 KB that every kernel may use (static shared memory counts
    // too) the limit is raised, for the current device, on every call
    if (smem > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    int per_sm = resident.load(std::memory_order_relaxed);
    if (per_sm == 0) {
        int n = 0;
        const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem);
        if (e != cudaSuccess) return e;
        per_sm = n < 1 ? 1 : n;
        resident.store(per_sm, std::memory_order_relaxed);
    }
    const long long most = static_cast<long long>(num_sms) * (per_sm < most_per_sm ? per_sm : most_per_sm);
    grid = static_cast<unsigned>(need < most ? need : most);
    return cudaSuccess;
}

template <typename T, class S>
cudaError_t launch_norm(const NormFwd& L, int num_sms, cudaStream_t stream) {
    static std::atomic<int> per_sm{0};
    unsigned grid = 0;
    const long long need = (L.rows + RowCta<S::W>::rows - 1) / RowCta<S::W>::rows;
    const cudaError_t e = persistent_grid(norm_kernel<T, S>, S::threads, S::smem, num_sms, per_sm, need, 32, grid);
    if (e != cudaSuccess) return e;
    norm_kernel<T, S><<<grid, S::threads, S::smem, stream>>>(L);
    return cudaGetLastError();
}

template <typename T, class S>
cudaError_t launch_norm_grad(const NormBwd& L, int num_sms, cudaStream_t stream, float* part, int& parts) {
    static std::atomic<int> per_sm{0};
    unsigned grid = 0;
    const long long need = (L.rows + RowCta<S::W>::rows - 1) / RowCta<S::W>::rows;
    const cudaError_t e =
        persistent_grid(norm_grad_kernel<T, S>, S::threads, S::smem, num_sms, per_sm, need, kPartsPerSm, grid);
    if (e != cudaSuccess) return e;
    norm_grad_kernel<T, S><<<grid, S::threads, S::smem, stream>>>(L, part);
    parts = static_cast<int>(grid);
    return cudaGetLastError();
}

// Calls f with T and the row shape for dim and `vec`: rows too wide for two
// stages of shared memory are read directly.
template <int ARRAYS, typename F>
void with_shape(int x_dt, long long dim, bool vec, F&& f) {
    with_type(x_dt, [&](auto t) {
        using T = decltype(t);
        with_hold(dim, [&](auto h) {
            using H = decltype(h);
            constexpr int NU = H::G * static_cast<int>(sizeof(T)) / 2;  // 8 elements: one unit of bf16, two of fp32
            using V = RowShape<T, H::W, NU, VEC, ARRAYS>;
            // fp32 rows copy single elements; bf16 elements are too small for a copy
            constexpr int kElem = sizeof(T) == 4 && V::ring_bytes <= 128 * 1024 ? ELEM4 : DIRECT;
            using E = RowShape<T, H::W, NU, kElem, ARRAYS>;
            if constexpr (V::ring_bytes <= 128 * 1024) {
                if (vec) return f(t, V{});
            }
            return f(t, E{});
        });
    });
}

}  // namespace

cudaError_t launch_layer_norm(const NormFwd& L, int num_sms, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    if (L.dim > kMaxHeldDim) {
        with_type(L.x_dt, [&](auto t) {
            norm_wide_kernel<decltype(t)><<<static_cast<unsigned>(L.rows), kWideThreads, 0, stream>>>(L);
        });
        return cudaGetLastError();
    }
    const bool vec = L.dim % 8 == 0 && rows_vec_ok(L.x, L.ldx, L.x_dt) && rows_vec_ok(L.y, L.dim, L.x_dt) &&
                     param_vec_ok(L.w) && param_vec_ok(L.b);
    with_shape<1>(L.x_dt, L.dim, vec,
                  [&](auto t, auto s) { e = launch_norm<decltype(t), decltype(s)>(L, num_sms, stream); });
    return e;
}

size_t layer_norm_backward_workspace(long long rows, long long dim, int num_sms) {
    return sizeof(float) * 2 * static_cast<size_t>(backward_parts_bound(rows, num_sms)) * dim;
}

cudaError_t launch_layer_norm_backward(const NormBwd& L, int num_sms, cudaStream_t stream, int* launches) {
    int parts = 0;
    float* part = static_cast<float*>(L.workspace);
    cudaError_t e = cudaSuccess;
    if (L.rows > 0) {
        if (L.dim > kMaxHeldDim) {
            parts = static_cast<int>(L.rows < 64 ? L.rows : 64);
            with_type(L.x_dt, [&](auto t) {
                norm_grad_wide_kernel<decltype(t)><<<static_cast<unsigned>(L.rows), kWideThreads, 0, stream>>>(L);
                norm_param_wide_kernel<decltype(t)>
                    <<<dim3(static_cast<unsigned>((L.dim + 255) / 256), parts), 256, 0, stream>>>(L, part);
            });
            *launches += 2;
            e = cudaGetLastError();
        } else {
            const bool vec = L.dim % 8 == 0 && rows_vec_ok(L.x, L.ldx, L.x_dt) && rows_vec_ok(L.dy, L.ldy, L.x_dt) &&
                             rows_vec_ok(L.dx, L.dim, L.x_dt) && param_vec_ok(L.w);
            with_shape<2>(L.x_dt, L.dim, vec, [&](auto t, auto s) {
                e = launch_norm_grad<decltype(t), decltype(s)>(L, num_sms, stream, part, parts);
            });
            ++*launches;
        }
        if (e != cudaSuccess) return e;
    }
    if (L.dw || L.db) {
        ++*launches;
        e = launch_dependent(norm_param_sum_kernel, dim3(static_cast<unsigned>((L.dim + 31) / 32), 2), kSumWarps * 32, 0,
                             stream, part, parts, L.dim, L.dw, L.db, L.p_dt);
    }
    return e;
}

}  // namespace muon
