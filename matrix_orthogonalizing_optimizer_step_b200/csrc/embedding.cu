// Token embedding: lookup with scaling, and the gradient of the table.
//
//   out[t] = scale * E[id_t]
//   dE[v]  = scale * sum over { t : id_t = v, v != padding } of g[t]
//
// Both are bound by memory: the lookup reads and writes count x dim elements,
// the gradient reads count x dim and writes the whole vocab x dim table (the
// AdamW step that follows reads all of it).
//
// The gradient sorts the tokens, so that each table row is summed by whoever
// owns its run of the sorted order and no atomic add is needed: the order of
// every sum is fixed by the tokens alone, and results repeat bit for bit.
//   1. one launch whose first cluster of 8 CTAs sorts (token, position) pairs
//      (stable radix sort over the bits a token needs) while all other CTAs
//      write zeros over the table: the zero fill needs no order and is the
//      longer of the two at every size where either matters;
//   2. the sorted order is cut into chunks of kChunk positions; a warp sums
//      the rows of one chunk for 256 columns.  A token whose run lies inside
//      a chunk is written at once.  A run that crosses chunk borders leaves
//      one fp32 partial row per chunk;
//   3. the partial rows of each crossing run are added in order.
// The cut at fixed positions keeps a frequent token (or a padding token that
// fills half a batch) from becoming one warp's serial loop.
//
// Sums are fp32 and rounded once to the gradient's type.
#include "lane.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace muon {
namespace {

// ---- lookup -------------------------------------------------------------------

constexpr int kFwdWarps = 4;
constexpr int kSeg = 1024;  // columns per warp: four independent 8-element loads per lane

__device__ __forceinline__ long long token_at(const void* tokens, int i64, long long t) {
    return i64 ? static_cast<const long long*>(tokens)[t] : static_cast<const int*>(tokens)[t];
}

__device__ __forceinline__ void report_bad_token(DeviceStatus* st, long long t) {
    atomicMin(&st->first_bad_token, static_cast<int>(t));
    atomicOr(&st->bits, ST_INDEX);
}

template <typename TT, typename TO, bool VEC>
__global__ void __launch_bounds__(kFwdWarps * 32) embedding_kernel(const EmbedFwd L, int nseg) {
    const int lane = threadIdx.x % 32;
    const long long item = static_cast<long long>(blockIdx.x) * kFwdWarps + threadIdx.x / 32;
    const long long t = item / nseg;
    if (t >= L.count) return;
    const int seg = static_cast<int>(item - t * nseg);
    const long long c0 = static_cast<long long>(seg) * kSeg;
    const long long id = token_at(L.tokens, L.tokens_i64, t);
    const bool bad = id < 0 || id >= L.vocab;
    if (bad && seg == 0 && lane == 0) report_bad_token(L.status, t);
    const TT* src = static_cast<const TT*>(L.table) + (bad ? 0 : id) * L.dim;
    TO* dst = static_cast<TO*>(L.out) + t * L.dim;
    const float nan = __int_as_float(0x7fc00000);
    if (VEC) {
        Raw8<TT> r[kSeg / 256];
#pragma unroll
        for (int i = 0; i < kSeg / 256; ++i) {
            const long long c = c0 + i * 256 + lane * 8;
            if (c < L.dim) r[i] = ld8(src + c);
        }
#pragma unroll
        for (int i = 0; i < kSeg / 256; ++i) {
            const long long c = c0 + i * 256 + lane * 8;
            if (c >= L.dim) continue;
            float v[8];
            to_float8(r[i], v);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = bad ? nan : v[j] * L.scale;
            st8(dst + c, v);
        }
    } else {
#pragma unroll 8
        for (int i = 0; i < kSeg / 32; ++i) {
            const long long c = c0 + i * 32 + lane;
            if (c < L.dim) st1(dst + c, bad ? nan : to_float(src[c]) * L.scale);
        }
    }
}

// ---- gradient: sort and zero fill -----------------------------------------------

constexpr int kCluster = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxBins = 256;
constexpr int kItems = 4;                             // pairs per thread and tile
constexpr int kSortTile = kSortThreads * kItems;      // pairs per CTA and tile
constexpr int kChunk = 16;                            // sorted positions per reduction chunk

struct SortArgs {
    const void* tokens;
    int tokens_i64;
    unsigned count;
    unsigned vocab;          // sentinel key: padding and bad tokens sort behind every real one
    long long padding;
    unsigned* keys[2];       // ping-pong buffers; the result is in keys[passes & 1], pos[passes & 1]
    unsigned* pos[2];
    unsigned* counts;        // kCluster x kMaxBins
    int passes, digit_bits;
    DeviceStatus* status;
};

struct FillArgs {
    void* out;
    long long bytes;
};

struct SortShared {
    unsigned warp_hist[kSortWarps][kMaxBins];
    unsigned base[kMaxBins];   // next output position of each digit for this CTA
    unsigned scan[kMaxBins];
};

// key of token t in pass 0
__device__ __forceinline__ unsigned first_key(const SortArgs& S, unsigned t) {
    const long long id = token_at(S.tokens, S.tokens_i64, t);
    if (id < 0 || id >= S.vocab) {
        report_bad_token(S.status, t);
        return S.vocab;
    }
    return id == S.padding ? S.vocab : static_cast<unsigned>(id);
}

__device__ void sort_cluster(const SortArgs& S, SortShared& sh, int rank) {
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int bins = 1 << S.digit_bits;
    // CTA `rank` owns a contiguous stretch of the pairs
    const unsigned len = ((S.count + kCluster - 1) / kCluster + 31) / 32 * 32;
    const unsigned lo = min(static_cast<unsigned>(rank) * len, S.count), hi = min(lo + len, S.count);
    for (int p = 0; p < S.passes; ++p) {
        const unsigned* kin = S.keys[p & 1];
        const unsigned* pin = S.pos[p & 1];
        unsigned* kout = S.keys[(p & 1) ^ 1];
        unsigned* pout = S.pos[(p & 1) ^ 1];
        const int shift = p * S.digit_bits;
        // earlier passes' pairs come from other CTAs: read at L2
        auto key_of = [&](unsigned i) { return p == 0 ? first_key(S, i) : __ldcg(kin + i); };
        // digit counts of the whole stretch
        for (int b = tid; b < kMaxBins; b += kSortThreads) sh.base[b] = 0;
        __syncthreads();
        for (unsigned i = lo + tid; i < hi; i += kSortThreads)
            atomicAdd(&sh.base[(key_of(i) >> shift) & (bins - 1)], 1u);
        __syncthreads();
        for (int b = tid; b < bins; b += kSortThreads) S.counts[rank * kMaxBins + b] = sh.base[b];
        cluster_sync_all();
        // base[d] = pairs of smaller digits anywhere + pairs of digit d in earlier CTAs
        unsigned total = 0, before = 0;
        if (tid < bins) {
            for (int c = 0; c < kCluster; ++c) {
                const unsigned n = __ldcg(S.counts + c * kMaxBins + tid);
                if (c < rank) before += n;
                total += n;
            }
            sh.scan[tid] = total;
        }
        __syncthreads();
        for (int o = 1; o < bins; o <<= 1) {
            unsigned add = 0;
            if (tid < bins && tid >= o) add = sh.scan[tid - o];
            __syncthreads();
            if (tid < bins) sh.scan[tid] += add;
            __syncthreads();
        }
        if (tid < bins) sh.base[tid] = sh.scan[tid] - total + before;
        __syncthreads();
        // stable scatter, one tile at a time: warp w takes 32 * kItems consecutive pairs
        for (unsigned t0 = lo; t0 < hi; t0 += kSortTile) {
            for (int b = tid; b < kSortWarps * kMaxBins; b += kSortThreads) (&sh.warp_hist[0][0])[b] = 0;
            __syncthreads();
            unsigned key[kItems], val[kItems], rnk[kItems];
            bool on[kItems];
#pragma unroll
            for (int r = 0; r < kItems; ++r) {
                const unsigned i = t0 + (warp * kItems + r) * 32 + lane;
                on[r] = i < hi;
                key[r] = on[r] ? key_of(i) : 0;
                val[r] = on[r] ? (p == 0 ? i : __ldcg(pin + i)) : 0;
            }
#pragma unroll
            for (int r = 0; r < kItems; ++r) {
                const unsigned d = (key[r] >> shift) & (bins - 1);
                const unsigned peers = __match_any_sync(0xffffffffu, on[r] ? d : kMaxBins + lane);
                rnk[r] = __popc(peers & ((1u << lane) - 1));
                if (on[r]) rnk[r] += sh.warp_hist[warp][d];
                __syncwarp();
                if (on[r] && (peers >> lane) == 1u) sh.warp_hist[warp][d] += __popc(peers);  // the last peer
                __syncwarp();
            }
            __syncthreads();
            if (tid < bins) {
                unsigned run = sh.base[tid];
                for (int w = 0; w < kSortWarps; ++w) {
                    const unsigned n = sh.warp_hist[w][tid];
                    sh.warp_hist[w][tid] = run;
                    run += n;
                }
                sh.base[tid] = run;
            }
            __syncthreads();
#pragma unroll
            for (int r = 0; r < kItems; ++r) {
                if (!on[r]) continue;
                const unsigned at = sh.warp_hist[warp][(key[r] >> shift) & (bins - 1)] + rnk[r];
                kout[at] = key[r];
                pout[at] = val[r];
            }
            __syncthreads();
        }
        cluster_sync_all();  // the next pass reads every CTA's output
    }
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSortThreads)
    sort_and_fill_kernel(const SortArgs S, const FillArgs F) {
    __shared__ SortShared sh;
    if (blockIdx.x < kCluster) {
        sort_cluster(S, sh, static_cast<int>(blockIdx.x));
        return;
    }
    // zeros over the table (the runs' rows are written by the next launch);
    // every part writes whole 16-byte units from the first aligned address on
    const long long nthr = static_cast<long long>(gridDim.x - kCluster) * kSortThreads;
    const long long i0 = static_cast<long long>(blockIdx.x - kCluster) * kSortThreads + threadIdx.x;
    char* base = static_cast<char*>(F.out);
    const long long head = min(static_cast<long long>((16 - (reinterpret_cast<uintptr_t>(base) & 15)) & 15), F.bytes);
    const long long n16 = (F.bytes - head) / 16;
    uint4* q = reinterpret_cast<uint4*>(base + head);
    for (long long i = i0; i < n16; i += nthr) q[i] = make_uint4(0, 0, 0, 0);
    const long long tail = head + n16 * 16;
    if (i0 < head) base[i0] = 0;
    if (i0 < F.bytes - tail) base[tail + i0] = 0;
}

// ---- gradient: sums over runs of equal tokens ------------------------------------

struct RunArgs {
    const unsigned* keys;  // sorted tokens (sentinel `vocab` last)
    const unsigned* pos;   // their positions
    unsigned count, vocab;
    const void* grad;
    long long ld, dim;
    float scale;
    void* out;
    float* partial;        // per chunk: [0] the run that came in, [1] the run that goes on; dim fp32 each
    int nslab;             // 256-column slabs
};

constexpr int kRunWarps = 4;

template <typename TG, typename TO, bool VEC>
__global__ void __launch_bounds__(kRunWarps * 32) run_sum_kernel(const RunArgs R) {
    const int lane = threadIdx.x % 32;
    const long long item = static_cast<long long>(blockIdx.x) * kRunWarps + threadIdx.x / 32;
    const long long chunk = item / R.nslab;
    const unsigned p0 = static_cast<unsigned>(chunk) * kChunk;
    if (chunk * kChunk >= R.count) return;
    const int n = min(static_cast<unsigned>(kChunk), R.count - p0);
    const long long c0 = (item - chunk * R.nslab) * 256;
    // lane i < n: pair i; lane 30: the key before the chunk; lane 31: the key after it
    unsigned k = R.vocab, q = 0;
    if (lane < n) {
        k = R.keys[p0 + lane];
        q = R.pos[p0 + lane];
    } else if (lane == 30) {
        k = p0 > 0 ? R.keys[p0 - 1] : R.vocab;
    } else if (lane == 31) {
        k = p0 + n < R.count ? R.keys[p0 + n] : R.vocab;
    }
    const unsigned prev = __shfl_sync(0xffffffffu, k, 30), next = __shfl_sync(0xffffffffu, k, 31);
    const TG* grad = static_cast<const TG*>(R.grad);
    float acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    bool first_run = true;
    // column of element j of this lane
    auto col = [&](int j) { return VEC ? c0 + lane * 8 + j : c0 + j * 32 + lane; };
    auto flush = [&](unsigned key, bool came_in, bool goes_on) {
        if (came_in || goes_on) {
            float* dst = R.partial + (chunk * 2 + (came_in ? 0 : 1)) * R.dim;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (col(j) < R.dim) dst[col(j)] = acc[j];
        } else {
            TO* dst = static_cast<TO*>(R.out) + static_cast<long long>(key) * R.dim;
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] *= R.scale;
            if (VEC) {
                if (col(0) < R.dim) st8(dst + col(0), acc);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col(j) < R.dim) st1(dst + col(j), acc[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    };
    constexpr int kBatch = 8;
#pragma unroll
    for (int b = 0; b < kChunk; b += kBatch) {
        if (b >= n) break;
        Raw8<TG> raw[VEC ? kBatch : 1];
        float el[VEC ? 1 : kBatch][8];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const unsigned key = __shfl_sync(0xffffffffu, k, b + i);
            const long long row = __shfl_sync(0xffffffffu, q, b + i);
            if (b + i >= n || key >= R.vocab) continue;
            const TG* src = grad + row * R.ld;
            if constexpr (VEC) {
                if (col(0) < R.dim) raw[i] = ld8(src + col(0));
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) el[i][j] = col(j) < R.dim ? to_float(src[col(j)]) : 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const unsigned key = __shfl_sync(0xffffffffu, k, b + i);
            const unsigned after = b + i + 1 < n ? __shfl_sync(0xffffffffu, k, (b + i + 1) & 31) : next;
            if (b + i >= n || key >= R.vocab) continue;  // the sentinels are last
            float v[8];
            if constexpr (VEC) {
                to_float8(raw[i], v);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = el[i][j];
            }
            // lanes past the last column hold nothing and store nothing
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += v[j];
            if (after != key) {
                flush(key, first_run && prev == key, false);
                first_run = false;
            } else if (b + i + 1 == n) {
                flush(key, first_run && prev == key, true);
            }
        }
    }
}

// First index in [lo, count) whose key differs from `key` (keys are sorted).
__device__ __forceinline__ unsigned run_end(const unsigned* keys, unsigned lo, unsigned count, unsigned key) {
    unsigned hi = count;
    while (lo < hi) {
        const unsigned mid = lo + (hi - lo) / 2;
        if (keys[mid] == key)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;

// One CTA per chunk: if a run starts in the chunk and goes on, add its partial
// rows in chunk order.  Up to kJoinWarps rows are added by one thread per
// column; a longer run is cut into kJoinWarps stretches, one per warp, whose
// sums are added in order (the cut depends on the run alone).
template <typename TO>
__global__ void __launch_bounds__(kJoinThreads) run_join_kernel(const RunArgs R) {
    __shared__ float part[kJoinWarps][32];
    const long long chunk = blockIdx.x;
    const unsigned p0 = static_cast<unsigned>(chunk) * kChunk;
    const unsigned p1 = p0 + kChunk;
    if (p1 >= R.count) return;  // the last chunk's runs end in it
    const unsigned key = R.keys[p1 - 1];
    if (key >= R.vocab || R.keys[p1] != key) return;
    if (R.keys[p0] == key && p0 > 0 && R.keys[p0 - 1] == key) return;  // it started earlier
    const unsigned end = run_end(R.keys, p1, R.count, key);
    const long long last = (end - 1) / kChunk;  // chunk of its last pair
    const long long m = last - chunk;           // incoming partial rows
    const float* mine = R.partial + (chunk * 2 + 1) * R.dim;
    const float* in = R.partial + (chunk + 1) * 2 * R.dim;  // row i at in + 2 * i * dim
    TO* dst = static_cast<TO*>(R.out) + static_cast<long long>(key) * R.dim;
    if (m <= kJoinWarps) {
        for (long long c = threadIdx.x; c < R.dim; c += kJoinThreads) {
            float s = mine[c];
            for (long long i = 0; i < m; ++i) s += in[2 * i * R.dim + c];
            st1(dst + c, s * R.scale);
        }
        return;
    }
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const long long per = (m + kJoinWarps - 1) / kJoinWarps;
    const long long i0 = min(per * warp, m), i1 = min(i0 + per, m);
    for (long long c = lane; c - lane < R.dim; c += 32) {
        float s = 0.f;
        if (c < R.dim) {
#pragma unroll 8
            for (long long i = i0; i < i1; ++i) s += in[2 * i * R.dim + c];
        }
        part[warp][lane] = s;
        __syncthreads();
        if (warp == 0 && c < R.dim) {
            float t = mine[c];
            for (int w = 0; w < kJoinWarps; ++w) t += part[w][lane];
            st1(dst + c, t * R.scale);
        }
        __syncthreads();
    }
}

struct BwdLayout {
    size_t keys[2], pos[2], counts, partial, total;
};

BwdLayout bwd_layout(long long count, long long dim) {
    BwdLayout l{};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at = align_up(at + bytes, 256);
        return o;
    };
    for (int i = 0; i < 2; ++i) {
        l.keys[i] = take(sizeof(unsigned) * count);
        l.pos[i] = take(sizeof(unsigned) * count);
    }
    l.counts = take(sizeof(unsigned) * kCluster * kMaxBins);
    l.partial = take(sizeof(float) * 2 * ((count + kChunk - 1) / kChunk) * dim);
    l.total = at;
    return l;
}

template <typename TG, typename TO>
void launch_run_sum(const RunArgs& R, bool vec, unsigned blocks, cudaStream_t stream) {
    if (vec)
        run_sum_kernel<TG, TO, true><<<blocks, kRunWarps * 32, 0, stream>>>(R);
    else
        run_sum_kernel<TG, TO, false><<<blocks, kRunWarps * 32, 0, stream>>>(R);
}

}  // namespace

cudaError_t launch_embedding(const EmbedFwd& L, cudaStream_t stream) {
    const int nseg = static_cast<int>((L.dim + kSeg - 1) / kSeg);
    const unsigned blocks = static_cast<unsigned>((L.count * nseg + kFwdWarps - 1) / kFwdWarps);
    const bool vec = rows_vec_ok(L.table, L.dim, L.table_dt) && rows_vec_ok(L.out, L.dim, L.out_dt) && L.dim % 8 == 0;
    auto go = [&](auto tt, auto to) {
        using TT = decltype(tt);
        using TO = decltype(to);
        if (vec)
            embedding_kernel<TT, TO, true><<<blocks, kFwdWarps * 32, 0, stream>>>(L, nseg);
        else
            embedding_kernel<TT, TO, false><<<blocks, kFwdWarps * 32, 0, stream>>>(L, nseg);
    };
    const __nv_bfloat16 h{};
    if (L.table_dt == DT_F32)
        L.out_dt == DT_F32 ? go(0.f, 0.f) : go(0.f, h);
    else
        L.out_dt == DT_F32 ? go(h, 0.f) : go(h, h);
    return cudaGetLastError();
}

size_t embedding_backward_workspace(long long count, long long dim) { return bwd_layout(count, dim).total; }

cudaError_t launch_embedding_backward(const EmbedBwd& L, int num_sms, cudaStream_t stream, int* launches) {
    const BwdLayout lay = bwd_layout(L.count, L.dim);
    char* ws = static_cast<char*>(L.workspace);
    SortArgs S{};
    S.tokens = L.tokens;
    S.tokens_i64 = L.tokens_i64;
    S.count = static_cast<unsigned>(L.count);
    S.vocab = static_cast<unsigned>(L.vocab);
    S.padding = L.padding;
    for (int i = 0; i < 2; ++i) {
        S.keys[i] = reinterpret_cast<unsigned*>(ws + lay.keys[i]);
        S.pos[i] = reinterpret_cast<unsigned*>(ws + lay.pos[i]);
    }
    S.counts = reinterpret_cast<unsigned*>(ws + lay.counts);
    int bits = 1;
    while ((static_cast<unsigned long long>(L.vocab) >> bits) != 0) ++bits;  // keys are 0 .. vocab
    S.passes = L.count > 0 ? (bits + 7) / 8 : 0;
    S.digit_bits = S.passes ? (bits + S.passes - 1) / S.passes : 0;
    S.status = L.status;
    FillArgs F{L.out, L.vocab * L.dim * dtype_size(L.out_dt)};
    // two CTAs of 1024 threads per SM; no more than the fill has 16-byte units for
    long long fill_ctas = (F.bytes / 16 + kSortThreads - 1) / kSortThreads;
    const long long most = static_cast<long long>(num_sms) * 2 / kCluster * kCluster - kCluster;
    fill_ctas = fill_ctas < 1 ? 1 : (fill_ctas > most ? most : fill_ctas);
    const unsigned grid = static_cast<unsigned>((fill_ctas + kCluster - 1) / kCluster * kCluster + kCluster);
    sort_and_fill_kernel<<<grid, kSortThreads, 0, stream>>>(S, F);
    ++*launches;
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || L.count == 0) return e;

    RunArgs R{};
    R.keys = S.keys[S.passes & 1];
    R.pos = S.pos[S.passes & 1];
    R.count = S.count;
    R.vocab = S.vocab;
    R.grad = L.grad;
    R.ld = L.ld;
    R.dim = L.dim;
    R.scale = L.scale;
    R.out = L.out;
    R.partial = reinterpret_cast<float*>(ws + lay.partial);
    R.nslab = static_cast<int>((L.dim + 255) / 256);
    const long long nchunks = (L.count + kChunk - 1) / kChunk;
    const unsigned blocks = static_cast<unsigned>((nchunks * R.nslab + kRunWarps - 1) / kRunWarps);
    const bool vec = rows_vec_ok(L.grad, L.ld, L.grad_dt) && rows_vec_ok(L.out, L.dim, L.out_dt) && L.dim % 8 == 0;
    if (L.grad_dt == DT_F32)
        L.out_dt == DT_F32 ? launch_run_sum<float, float>(R, vec, blocks, stream)
                           : launch_run_sum<float, __nv_bfloat16>(R, vec, blocks, stream);
    else
        L.out_dt == DT_F32 ? launch_run_sum<__nv_bfloat16, float>(R, vec, blocks, stream)
                           : launch_run_sum<__nv_bfloat16, __nv_bfloat16>(R, vec, blocks, stream);
    ++*launches;
    e = cudaGetLastError();
    if (e != cudaSuccess || nchunks < 2) return e;
    if (L.out_dt == DT_F32)
        run_join_kernel<float><<<static_cast<unsigned>(nchunks), kJoinThreads, 0, stream>>>(R);
    else
        run_join_kernel<__nv_bfloat16><<<static_cast<unsigned>(nchunks), kJoinThreads, 0, stream>>>(R);
    ++*launches;
    return cudaGetLastError();
}

}  // namespace muon
