// Token embedding: lookup with scaling, and the gradient of the table.
//
//   out[t] = scale * E[id_t]
//   dE[v]  = scale * sum over { t : id_t = v, v != padding } of g[t]
//
// Both are bound by memory: the lookup reads and writes count x dim elements,
// the gradient reads count x dim and writes the whole vocab x dim table (the
// AdamW step that follows reads all of it).
//
// The gradient puts the tokens in order, so that each table row is summed by
// whoever owns its stretch of the order and no atomic add is needed: every sum
// is in the order of the tokens' positions and results repeat bit for bit.
//   1. one launch orders (token, position) pairs.  Up to 16384 tokens: one CTA
//      per SM owns a class of the vocabulary, finds its tokens among all and
//      groups them.  More tokens: a cluster of 8 CTAs sorts them.
//   2. zeros are written over the table, beside the first launch, by one of
//      their own; where a large part of the rows is asked for, or the table is
//      small, by the classes' CTAs after their grouping, over the other rows.
//   3. the order is cut into chunks of 16 positions (8 in short batches); a warp
//      sums the rows of one chunk for 256 columns.  A token whose run lies inside a chunk is
//      written at once.  A run that crosses chunk borders leaves one fp32
//      partial row per chunk, and the warp that finishes the last of the run's
//      chunks adds them in order.
// The cut at fixed positions keeps a frequent token (or a padding token that
// fills half a batch) from becoming one warp's serial loop.  The zeros are
// written before the sums: loads beside a memory system that takes writes at
// its full rate are several times slower (zeroing CTAs among the summing ones:
// 35-39 instead of 31 us for 8192 tokens of 50257 x 768, 236-400 instead of 216 us
// for 16384 of 128256 x 4096).
//
// Sums are fp32 and rounded once to the gradient's type.
//
// Measured (bf16, calls behind one another on changing inputs): lookup of 16384
// tokens from 128256 x 4096 35 us, 134 MB written and up to as much read (the
// repeats come from L2); 16 tokens 1.6 us replayed from a graph.  Gradient of
// 8192 tokens of 50257 x 768 28 us (13.9 us at the copy rate; 23.4 from a
// graph), of 16384 of 128256 x 4096 187 us (183), of 1237 of 5003 x 333 fp32
// 14.3-15.3 us (12.6 from a graph).
#include <algorithm>

#include "lane.h"
#include "pdl.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace muon {
namespace {

// ---- lookup -------------------------------------------------------------------

// A warp copies 1024 columns of one row, four independent 8-element loads per
// lane: enough in flight at full occupancy (28 registers) for 6 TB/s of reads
// and writes from cold caches at 65536 x 768, and few rows still spread over several warps.
constexpr int kFwdWarps = 4;
constexpr int kSeg = 1024;

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
    // a CTA has one segment of 4 tokens (32-bit division: a 64-bit one is a call)
    const unsigned group = blockIdx.x / static_cast<unsigned>(nseg);
    const long long t = static_cast<long long>(group) * kFwdWarps + threadIdx.x / 32;
    if (t >= L.count) return;
    const int seg = static_cast<int>(blockIdx.x - group * nseg);
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

// ---- gradient: order of up to kClassTokens tokens by classes of the vocabulary -----

// Ordered positions of a reduction chunk.  A short batch is a chain of latencies
// and a chunk of 8 is one trip to memory less (300 tokens of 20000 x 768 fp32 16.5
// instead of 18.8 us with 16); in a longer one more runs cross chunks of 8, and
// their partial rows are added one after another (512 tokens, half of them equal,
// 768 wide 19.5 instead of 16.3, 2000 29.6 instead of 22.8; 32768 of 50257 x 768 62
// instead of 52).
constexpr int kLongChunk = 16, kShortChunk = 8;
constexpr long long kShortCount = 384;
__host__ __device__ constexpr int chunk_of(long long count) { return count <= kShortCount ? kShortChunk : kLongChunk; }
constexpr int kClassTokens = 16384;
constexpr int kClassRows = 2048;          // table rows of a class at most
constexpr long long kClassVocab = 1 << 20;
constexpr int kMostClasses = 148;         // one CTA per SM
constexpr int kClassThreads = 512;
constexpr int kClassWarps = kClassThreads / 32;
constexpr int kPosBits = 14;
static_assert(kClassTokens <= 1 << kPosBits, "positions of a class's tokens");

struct ClassArgs {
    const void* tokens;
    int tokens_i64;
    int count, vocab, classes;
    unsigned magic;     // ceil(2^32 / classes): token / classes = umulhi(token, magic), exact for tokens below 2^20
    long long padding;
    unsigned* keys;     // tokens in order, `vocab` for those that take no part (last)
    unsigned* pos;      // their positions
    unsigned* done;     // counters to zero for the adding launch
    int ndone;
    int zero;           // write zeros over the rows that no token asks for
    void* out;
    long long dim;
    DeviceStatus* status;
};

// 32-bit words of the list of a class's tokens.
__host__ __device__ constexpr int class_list_words(int count) {
    return (count + kClassThreads - 1) / kClassThreads * kClassThreads;
}

// Zeros over one table row by one warp, 16 bytes a lane from the first aligned address on.
template <typename TO>
__device__ __forceinline__ void zero_row(TO* row, long long dim, int lane) {
    char* p = reinterpret_cast<char*>(row);
    const long long bytes = dim * sizeof(TO);
    const long long head = min(static_cast<long long>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15), bytes);
    const long long n16 = (bytes - head) / 16;
    uint4* q = reinterpret_cast<uint4*>(p + head);
    for (long long i = lane; i < n16; i += 32) q[i] = make_uint4(0, 0, 0, 0);
    if (lane < head) p[lane] = 0;
    if (lane < bytes - head - n16 * 16) p[head + n16 * 16 + lane] = 0;
}

// CTA c owns the table rows c, c + classes, c + 2 classes, ...: it finds the
// tokens of its class among all (each CTA reads all of them, from L2) and
// groups them by row in the order of their positions.  Then, where the zeros
// have no launch of their own, it writes them over the rows that no token asks
// for.  The order is ready after 4 us (8192 tokens; 10 beside the zeros' launch),
// where the sort's two passes take 20: no step of it leaves the CTA.
template <typename TO>
__global__ void __launch_bounds__(kClassThreads) class_group_kernel(const ClassArgs A) {
    extern __shared__ unsigned class_smem[];
    __shared__ int count[kClassRows];
    __shared__ unsigned short start[kClassRows];  // the row's next place in the order
    __shared__ int warp_n[kClassWarps], warp_before[kClassWarps], warp_sum[kClassWarps];
    unsigned* list = class_smem;  // row << 14 | position: each warp's finds from its first token's place on
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int classes = A.classes, cls = blockIdx.x;
    const int rows = (A.vocab - cls + classes - 1) / classes;
    allow_successor();
    for (int r = tid; r < kClassRows; r += kClassThreads) count[r] = 0;
    for (int i = cls * kClassThreads + tid; i < A.ndone; i += classes * kClassThreads) A.done[i] = 0;
    __syncthreads();
    // this warp's stretch of the tokens, 32 at a time
    const int items = (A.count + kClassThreads - 1) / kClassThreads;
    const int w0 = warp * items * 32;
    int found = 0, before = 0;
    constexpr int kLoads = 8;
#pragma unroll 1
    for (int i0 = 0; i0 < items; i0 += kLoads) {
        long long id[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int t = w0 + (i0 + i) * 32 + lane;
            id[i] = i0 + i < items && t < A.count ? token_at(A.tokens, A.tokens_i64, t) : A.padding;
            if (id[i] == A.padding) id[i] = -2;  // takes no part
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int t = w0 + (i0 + i) * 32 + lane;
            const bool in = i0 + i < items && t < A.count;
            const bool ok = in && id[i] >= 0 && id[i] < A.vocab;
            const unsigned q = __umulhi(static_cast<unsigned>(id[i]), A.magic);
            const int c = static_cast<int>(static_cast<unsigned>(id[i]) - q * classes);
            const unsigned votes = __ballot_sync(0xffffffffu, ok && c == cls);
            before += __popc(__ballot_sync(0xffffffffu, ok && c < cls));
            if (ok && c == cls) {
                list[w0 + found + __popc(votes & ((1u << lane) - 1))] = q << kPosBits | static_cast<unsigned>(t);
                atomicAdd(&count[q], 1);
            }
            found += __popc(votes);
            if (cls == 0 && in && !ok) {
                const long long tok = token_at(A.tokens, A.tokens_i64, t);
                if (tok < 0 || tok >= A.vocab) report_bad_token(A.status, t);
            }
        }
    }
    if (lane == 0) {
        warp_n[warp] = found;
        warp_before[warp] = before;
    }
    __syncthreads();
    // first place of every row's group: kClassRows / kClassThreads rows per thread
    {
        constexpr int kPer = kClassRows / kClassThreads;
        int n[kPer], mine = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            n[i] = count[tid * kPer + i];
            mine += n[i];
        }
        int scan = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, scan, o);
            if (lane >= o) scan += up;
        }
        if (lane == 31) warp_sum[warp] = scan;
        __syncthreads();
        int at = scan - mine;
        for (int w = 0; w < warp; ++w) at += warp_sum[w];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            start[tid * kPer + i] = static_cast<unsigned short>(at);
            at += n[i];
        }
    }
    // the warps' finds as one list, where they are few enough to move
    int lists = kClassWarps, total = 0, at = 0, most = 0;
    before = 0;
    for (int w = 0; w < kClassWarps; ++w) {
        if (w == warp) at = total;
        total += warp_n[w];
        most = max(most, warp_n[w]);
        before += warp_before[w];
    }
    if (most <= 4 * 32) {
        unsigned e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i * 32 + lane < found) e[i] = list[w0 + i * 32 + lane];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i * 32 + lane < found) list[at + i * 32 + lane] = e[i];
        lists = 1;
    }
    __syncthreads();
    // A warp groups the rows r = warp, warp + 16, ... in one pass over the list: a
    // token's place is its row's next one, the row's first lanes first.  (16384
    // tokens in 2000 rows, all of one class: 122 us for the call, with a pass per
    // row 5.9 ms; spread over the classes 33.)
    for (int w = 0; w < lists; ++w) {
        const int k = lists == 1 ? total : warp_n[w];
        const unsigned* l = list + w * items * 32;
        constexpr int kAhead = 4;
        for (int i0 = 0; i0 < k; i0 += kAhead * 32) {
            unsigned e[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) e[i] = i0 + i * 32 + lane < k ? l[i0 + i * 32 + lane] : 0;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const unsigned r = e[i] >> kPosBits;
                const bool on = i0 + i * 32 + lane < k && r % kClassWarps == warp;
                if (!__any_sync(0xffffffffu, on)) continue;
                const unsigned peers = __match_any_sync(0xffffffffu, on ? r : ~0u);
                unsigned at = 0;
                if (on) {
                    at = start[r] + __popc(peers & ((1u << lane) - 1));
                    A.keys[before + at] = cls + r * classes;
                    A.pos[before + at] = e[i] & ((1u << kPosBits) - 1);
                }
                __syncwarp();
                if (on && (peers >> lane) == 1u) start[r] = static_cast<unsigned short>(at + 1);  // the last of them
                __syncwarp();
            }
        }
    }
    if (cls == classes - 1)  // tokens that take no part
        for (int k = before + total + tid; k < A.count; k += kClassThreads) A.keys[k] = A.vocab;
    if (!A.zero) return;
    for (int r = warp; r < rows; r += kClassWarps)
        if (count[r] == 0) zero_row(static_cast<TO*>(A.out) + static_cast<long long>(cls + r * classes) * A.dim, A.dim, lane);
}

// ---- gradient: order by sorting, zeros -----------------------------------------------

constexpr int kCluster = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxBits = 9;                           // digit: two passes hold any vocabulary below 2^18
constexpr int kMaxBins = 1 << kMaxBits;
constexpr int kItems = 4;                             // pairs per thread and tile
constexpr int kSortTile = kSortThreads * kItems;      // pairs per CTA and tile

struct SortArgs {
    const void* tokens;
    int tokens_i64;
    unsigned count;
    unsigned vocab;          // keys from here on (padding, bad tokens) sort behind every real one
    long long padding;
    unsigned* keys[2];       // ping-pong buffers; the result is in keys[passes & 1], pos[passes & 1]
    unsigned* pos[2];
    int passes, digit_bits;
    unsigned* done;          // counters to zero for the adding launch
    long long ndone;
    DeviceStatus* status;
};

struct SortShared {
    unsigned short warp_hist[kSortWarps][kMaxBins];  // counts, then places within the tile
    unsigned totals[kCluster][kMaxBins];             // every CTA's digit counts (written by that CTA)
    unsigned base[kMaxBins];                         // next output position of each digit for this CTA
    unsigned warp_sum[kSortWarps];
};

// Key of token t in pass 0: the sentinel `vocab` for padding, vocab + 1 for a
// token outside the vocabulary (reported once the loads are under way).
__device__ __forceinline__ unsigned first_key(const SortArgs& S, unsigned t) {
    const long long id = token_at(S.tokens, S.tokens_i64, t);
    const unsigned k = id == S.padding ? S.vocab : static_cast<unsigned>(id);
    return id < 0 || id >= S.vocab ? S.vocab + 1 : k;
}

// base[d] = `before` + the total of all smaller digits; thread d brings the total of digit d.
__device__ __forceinline__ void digit_bases(unsigned* base, unsigned* warp_sum, int bins, unsigned total,
                                            unsigned before) {
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    unsigned scan = total;  // inclusive, within the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned up = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += up;
    }
    if (lane == 31) warp_sum[warp] = scan;
    __syncthreads();
    if (tid < bins) {
        unsigned below = 0;
        for (int w = 0; w < warp; ++w) below += warp_sum[w];
        base[tid] = below + scan - total + before;
    }
    __syncthreads();
}

// Every CTA of the cluster learns this CTA's count of digit `tid`, then
// base[d] = pairs of smaller digits anywhere + pairs of digit d in earlier CTAs.
__device__ void sort_bases(SortShared& sh, int bins, int rank, unsigned mine) {
    const int tid = threadIdx.x;
    if (tid < bins) {
        const uint32_t at = smem_u32(&sh.totals[rank][tid]);
#pragma unroll
        for (int c = 0; c < kCluster; ++c)
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_to_cta(at, c)), "r"(mine) : "memory");
    }
    cluster_sync_all();
    unsigned total = 0, before = 0;
    if (tid < bins) {
#pragma unroll
        for (int c = 0; c < kCluster; ++c) {
            const unsigned n = sh.totals[c][tid];
            if (c < rank) before += n;
            total += n;
        }
    }
    digit_bases(sh.base, sh.warp_sum, bins, total, before);
}

// Lanes of the warp that are on and hold the same digit as this one (this
// lane's own bit included if it is on): one vote per bit of the digit.
__device__ __forceinline__ unsigned digit_peers(unsigned d, int bits, bool on) {
    unsigned peers = __ballot_sync(0xffffffffu, on);
    for (int b = 0; b < bits; ++b) {
        const bool bit = (d >> b) & 1u;
        const unsigned votes = __ballot_sync(0xffffffffu, bit);
        peers &= bit ? votes : ~votes;
    }
    return peers;
}

// For more tokens than the classes' CTAs would each want to read, and for larger
// vocabularies.  (The whole gradient either way: 8192 tokens of 50257 x 768 36.8
// us by sorting, 31.4 by classes; 16384 of 128256 x 4096 248 and 223; 16384 of
// 50257 x 768 39.4 and 41.4, which is where the classes end.)
//
// Stable radix sort of the pairs (token, position) by the cluster's CTAs, each
// owning a contiguous stretch.  Within a tile, warp w takes 32 * kItems
// consecutive pairs; a pair's place is the count of its digit in earlier CTAs,
// tiles, warps, rows and lanes.  A stretch of one tile (any count up to
// kCluster * kSortTile) is read once per pass.
//
// The caller has arrived at the cluster's barrier: the wait for the other CTAs'
// arrival, which says that they run and their shared memory may be written,
// stands before the first digit counts are sent.
__device__ void sort_cluster(const SortArgs& S, SortShared& sh, int rank) {
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int bins = 1 << S.digit_bits;
    const unsigned len = ((S.count + kCluster - 1) / kCluster + 31) / 32 * 32;
    const unsigned lo = min(static_cast<unsigned>(rank) * len, S.count), hi = min(lo + len, S.count);
    const bool one_tile = len <= kSortTile;
    bool peers_run = false;
    auto await_peers = [&] {
        if (!peers_run) cluster_wait();
        peers_run = true;
    };
    for (int p = 0; p < S.passes; ++p) {
        const unsigned* kin = S.keys[p & 1];
        const unsigned* pin = S.pos[p & 1];
        unsigned* kout = S.keys[(p & 1) ^ 1];
        unsigned* pout = S.pos[(p & 1) ^ 1];
        const int shift = p * S.digit_bits;
        // earlier passes' pairs come from other CTAs: read at L2
        auto key_of = [&](unsigned i) { return p == 0 ? first_key(S, i) : __ldcg(kin + i); };
        if (!one_tile) {  // digit counts of the whole stretch first
            for (int b = tid; b < bins; b += kSortThreads) sh.base[b] = 0;
            __syncthreads();
            for (unsigned i = lo + tid; i < hi; i += kSortThreads)
                atomicAdd(&sh.base[(key_of(i) >> shift) & (bins - 1)], 1u);
            __syncthreads();
            const unsigned mine = tid < bins ? sh.base[tid] : 0;
            await_peers();
            sort_bases(sh, bins, rank, mine);
        }
        // (a stretch without pairs still takes part in the exchange)
        for (unsigned t0 = lo; t0 < hi || (one_tile && t0 == lo); t0 += kSortTile) {
            uint4* z = reinterpret_cast<uint4*>(&sh.warp_hist[0][0]);
            for (int b = tid; b < kSortWarps * kMaxBins / 8; b += kSortThreads) z[b] = make_uint4(0, 0, 0, 0);
            unsigned key[kItems], val[kItems], rnk[kItems];
            bool on[kItems];
#pragma unroll
            for (int r = 0; r < kItems; ++r) {
                const unsigned i = t0 + (warp * kItems + r) * 32 + lane;
                on[r] = i < hi;
                key[r] = on[r] ? key_of(i) : 0;
                val[r] = on[r] ? (p == 0 ? i : __ldcg(pin + i)) : 0;
            }
            if (p == 0) {
#pragma unroll
                for (int r = 0; r < kItems; ++r)
                    if (key[r] == S.vocab + 1) report_bad_token(S.status, val[r]);
            }
            __syncthreads();
#pragma unroll
            for (int r = 0; r < kItems; ++r) {
                const unsigned d = (key[r] >> shift) & (bins - 1);
                const unsigned peers = digit_peers(d, S.digit_bits, on[r]);
                rnk[r] = __popc(peers & ((1u << lane) - 1));
                if (on[r]) rnk[r] += sh.warp_hist[warp][d];
                __syncwarp();
                if (on[r] && (peers >> lane) == 1u) sh.warp_hist[warp][d] = rnk[r] + 1;  // the last peer
                __syncwarp();
            }
            __syncthreads();
            unsigned tile = 0;
            if (tid < bins) {
                unsigned n[kSortWarps];
#pragma unroll
                for (int w = 0; w < kSortWarps; ++w) n[w] = sh.warp_hist[w][tid];
#pragma unroll
                for (int w = 0; w < kSortWarps; ++w) {
                    sh.warp_hist[w][tid] = static_cast<unsigned short>(tile);
                    tile += n[w];
                }
            }
            if (one_tile) {
                await_peers();
                sort_bases(sh, bins, rank, tile);
            } else {
                __syncthreads();
            }
#pragma unroll
            for (int r = 0; r < kItems; ++r) {
                if (!on[r]) continue;
                const unsigned d = (key[r] >> shift) & (bins - 1);
                const unsigned at = sh.base[d] + sh.warp_hist[warp][d] + rnk[r];
                kout[at] = key[r];
                pout[at] = val[r];
            }
            __syncthreads();
            if (tid < bins) sh.base[tid] += tile;
        }
        cluster_sync_all();  // the next pass reads every CTA's output
    }
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSortThreads) sort_kernel(const SortArgs S) {
    extern __shared__ uint4 sort_smem[];
    cluster_arrive();
    allow_successor();
    const long long i0 = static_cast<long long>(blockIdx.x) * kSortThreads + threadIdx.x;
    for (long long i = i0; i < S.ndone; i += kCluster * kSortThreads) S.done[i] = 0;
    sort_cluster(S, *reinterpret_cast<SortShared*>(sort_smem), static_cast<int>(blockIdx.x));
}

// Zeros over the whole table, beside the launch that orders the tokens, which
// is its predecessor: whole 16-byte units from the first aligned address on.
// Short CTAs in the order of the addresses write 7.5 TB/s, a little more than a
// memset; persistent ones, which drift apart, 6.3 in any pattern (2.1 GB: 280 and
// 330-340 us; 16-byte, 32-byte and bulk stores and cache hints alike).
constexpr int kZeroThreads = 256;
constexpr int kZeroUnits = 4;
constexpr long long kZeroBytes = 16ll * kZeroThreads * kZeroUnits;  // of a CTA
__global__ void __launch_bounds__(kZeroThreads) zero_kernel(char* base, long long bytes) {
    allow_successor();
    const long long head = min(static_cast<long long>((16 - (reinterpret_cast<uintptr_t>(base) & 15)) & 15), bytes);
    const long long n16 = (bytes - head) / 16;
    uint4* q = reinterpret_cast<uint4*>(base + head);
    const long long i0 = static_cast<long long>(blockIdx.x) * (kZeroThreads * kZeroUnits) + threadIdx.x;
#pragma unroll
    for (int u = 0; u < kZeroUnits; ++u)
        if (i0 + u * kZeroThreads < n16) q[i0 + u * kZeroThreads] = make_uint4(0, 0, 0, 0);
    if (blockIdx.x > 0) return;
    const long long tail = head + n16 * 16;
    if (threadIdx.x < head) base[threadIdx.x] = 0;
    if (threadIdx.x < bytes - tail) base[tail + threadIdx.x] = 0;
    wait_predecessor();  // one CTA is enough for this launch to end after it
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
    unsigned* done;        // per (chunk, slab): finished pieces of the run that starts in the chunk and goes on
};

constexpr int kRunWarps = 4;

// Chunks behind `chunk` (up) or before it (down) that the run of `key` reaches
// into: up, the later chunks that start with it, down, the earlier ones that
// end with it (whole warp).  Equal keys lie together, so a chunk that the run
// does not reach ends it: two looks at the 32 nearest and the next 32 chunks, one
// at doubling distances, then at 32 places between the last hit and the first
// miss until they meet.  A run of m chunks costs each of them log m looks (2^21
// equal tokens, 8 wide: 6.7 ms, almost all of it the joining warp's; with looks
// at 32 chunks at a time to the run's end 56 ms).
template <int kChunk>
__device__ __forceinline__ unsigned chunks_of_run(const RunArgs& R, unsigned chunk, unsigned key, bool up, int lane) {
    auto misses = [&](unsigned long long k) {  // lanes whose chunk, k away, the run does not reach
        const unsigned long long at = up ? (chunk + k) * kChunk : (chunk + 1ull - k) * kChunk - 1;
        const bool in = up ? at < R.count : k <= chunk;
        return __ballot_sync(0xffffffffu, !(in && R.keys[in ? at : 0] == key));
    };
    unsigned miss = misses(lane + 1);
    if (miss) return __ffs(miss) - 1;
    miss = misses(lane + 33);
    if (miss) return __ffs(miss) + 31;
    miss = misses(128ull << lane);  // (behind the last chunk from the 26th lane on at the latest)
    const int first = __ffs(miss) - 1;
    unsigned long long hit = 64ull << first, end = 128ull << first;  // the run reaches `hit` chunks, not `end`
    while (end - hit > 1) {
        const unsigned long long step = (end - hit + 31) / 32;
        const unsigned long long k = min(hit + step * (lane + 1), end);
        const int f = __ffs(misses(k)) - 1;  // the last lane's is `end`
        end = min(hit + step * (f + 1), end);
        hit += step * f;
    }
    return static_cast<unsigned>(hit);
}

// A warp adds the rows of one chunk for 256 columns: items of equal size with
// 8 rows' loads in flight each (10-13 us for 8192 x 768, 50 us for 16384 x 4096
// with the zeros' last lines still on their way to memory; units of one token's
// rows, of unequal size, took 18 and 75-110 us).  A run inside the chunk is
// written at once.  A run that crosses the chunk's borders leaves a partial
// row; the warp that finishes the last of the run's chunks for these columns
// adds the partial rows in order.
template <typename TG, typename TO, bool VEC, int kChunk>
__global__ void __launch_bounds__(kRunWarps * 32) run_sum_kernel(const RunArgs R) {
    const int lane = threadIdx.x % 32;
    // a CTA has one slab of 4 chunks
    const unsigned group = blockIdx.x / static_cast<unsigned>(R.nslab);
    const int slab = static_cast<int>(blockIdx.x - group * R.nslab);
    const long long chunk = static_cast<long long>(group) * kRunWarps + threadIdx.x / 32;
    const unsigned p0 = static_cast<unsigned>(chunk) * kChunk;
    wait_predecessor();
    if (chunk * kChunk >= R.count) return;
    const int n = min(static_cast<unsigned>(kChunk), R.count - p0);
    const long long c0 = slab * 256ll;
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
    unsigned in_key = R.vocab, out_key = R.vocab;  // runs that came in, that start here and go on
    // column of element j of this lane
    auto col = [&](int j) { return VEC ? c0 + lane * 8 + j : c0 + j * 32 + lane; };
    auto flush = [&](unsigned key, bool came_in, bool goes_on) {
        if (came_in || goes_on) {
            (came_in ? in_key : out_key) = key;
            float* dst = R.partial + (chunk * 2 + (came_in ? 0 : 1)) * R.dim;
            if (VEC) {
                if (col(0) < R.dim) st8(dst + col(0), acc);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col(j) < R.dim) dst[col(j)] = acc[j];
            }
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
    constexpr int kBatch = 8;  // rows whose loads are in flight at once
#pragma unroll 1
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
            if (b + i >= n || key >= R.vocab) continue;  // those that take no part are last
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
            if (after != key || b + i + 1 == n) {
                flush(key, first_run && prev == key, after == key);
                first_run = false;
            }
        }
    }
    if (in_key >= R.vocab && out_key >= R.vocab) return;
    __threadfence();  // the partial rows before the counts
    __syncwarp();
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
        const unsigned key = e == 0 ? in_key : out_key;
        if (key >= R.vocab) continue;
        const unsigned me = static_cast<unsigned>(chunk);
        const unsigned a = e == 0 ? me - chunks_of_run<kChunk>(R, me, key, false, lane) : me;
        // a run that came in and ends here reaches no further
        const unsigned z = e == 0 && next != key ? me : me + chunks_of_run<kChunk>(R, me, key, true, lane);
        unsigned old = 0;
        if (lane == 0) old = atomicAdd(&R.done[static_cast<long long>(a) * R.nslab + slab], 1u);
        old = __shfl_sync(0xffffffffu, old, 0);
        if (old != z - a) continue;  // not the last of z - a + 1 chunks
        __threadfence();
        const float* src = R.partial + (2ll * a + 1) * R.dim;  // the row that goes on, then every chunk's that came in
        float s[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = 0.f;
        TO* dst = static_cast<TO*>(R.out) + static_cast<long long>(key) * R.dim;
        if constexpr (VEC) {
            if (col(0) >= R.dim) continue;
            auto add = [&](const float* p) {
                const float4 x = __ldcg(reinterpret_cast<const float4*>(p)), y = __ldcg(reinterpret_cast<const float4*>(p + 4));
                s[0] += x.x, s[1] += x.y, s[2] += x.z, s[3] += x.w;
                s[4] += y.x, s[5] += y.y, s[6] += y.z, s[7] += y.w;
            };
            add(src + col(0));
            const float* in = src + R.dim + col(0);
#pragma unroll 8
            for (unsigned i = a; i < z; ++i, in += 2 * R.dim) add(in);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] *= R.scale;
            st8(dst + col(0), s);
        } else {
            for (int j = 0; j < 8; ++j)
                if (col(j) < R.dim) s[j] = __ldcg(src + col(j));
#pragma unroll 2
            for (unsigned i = a; i < z; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col(j) < R.dim) s[j] += __ldcg(src + (2ll * (i - a) + 1) * R.dim + col(j));
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (col(j) < R.dim) st1(dst + col(j), s[j] * R.scale);
        }
    }
}

struct BwdLayout {
    size_t keys[2], pos[2], done, partial, total;
    size_t chunks, ndone;
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
    const int chunk = chunk_of(count);
    l.chunks = (count + chunk - 1) / chunk;
    l.ndone = l.chunks * ((dim + 255) / 256);
    // a workspace for many tokens is one for fewer, whose chunks are shorter
    const size_t room = std::max<size_t>(l.chunks, (std::min(count, kShortCount) + kShortChunk - 1) / kShortChunk);
    l.done = take(sizeof(unsigned) * room * ((dim + 255) / 256));
    l.partial = take(sizeof(float) * 2 * room * dim);
    l.total = at;
    return l;
}

// Orders up to kClassTokens tokens into keys[0], pos[0]; `zero`: and fills the table with zeros.
cudaError_t launch_class_group(const EmbedBwd& L, int classes, bool zero, const BwdLayout& lay, cudaStream_t stream) {
    char* ws = static_cast<char*>(L.workspace);
    ClassArgs A{};
    A.tokens = L.tokens;
    A.tokens_i64 = L.tokens_i64;
    A.count = static_cast<int>(L.count);
    A.vocab = static_cast<int>(L.vocab);
    A.classes = classes;
    A.magic = static_cast<unsigned>(((1ull << 32) + classes - 1) / classes);
    A.padding = L.padding;
    A.keys = reinterpret_cast<unsigned*>(ws + lay.keys[0]);
    A.pos = reinterpret_cast<unsigned*>(ws + lay.pos[0]);
    A.done = reinterpret_cast<unsigned*>(ws + lay.done);
    A.ndone = static_cast<int>(lay.ndone);
    A.zero = zero;
    A.out = L.out;
    A.dim = L.dim;
    A.status = L.status;
    const size_t smem = 4 * static_cast<size_t>(class_list_words(A.count));
    auto kernel = L.out_dt == DT_F32 ? class_group_kernel<float> : class_group_kernel<__nv_bfloat16>;
    // above the 48 KB that every kernel may use, 13 of them static
    if (smem > 32 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    kernel<<<classes, kClassThreads, smem, stream>>>(A);
    return cudaGetLastError();
}

// Orders any number of tokens by sorting; *side says which pair of buffers has the result.
cudaError_t launch_sort(const EmbedBwd& L, const BwdLayout& lay, cudaStream_t stream, int* side) {
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
    int bits = 1;
    while ((static_cast<unsigned long long>(L.vocab + 1) >> bits) != 0) ++bits;  // keys are 0 .. vocab + 1
    S.passes = (bits + kMaxBits - 1) / kMaxBits;
    S.digit_bits = (bits + S.passes - 1) / S.passes;
    S.done = reinterpret_cast<unsigned*>(ws + lay.done);
    S.ndone = static_cast<long long>(lay.ndone);
    S.status = L.status;
    *side = S.passes & 1;
    const cudaError_t e =
        cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(SortShared)));
    if (e != cudaSuccess) return e;
    sort_kernel<<<kCluster, kSortThreads, sizeof(SortShared), stream>>>(S);
    return cudaGetLastError();
}

// Zeros over the table; after a launch of this call that orders the tokens, or on its own.
cudaError_t launch_zero(const EmbedBwd& L, bool dependent, cudaStream_t stream) {
    const long long bytes = L.vocab * L.dim * dtype_size(L.out_dt);
    const unsigned blocks = static_cast<unsigned>((bytes + kZeroBytes - 1) / kZeroBytes);
    char* out = static_cast<char*>(L.out);
    if (dependent) return launch_dependent(zero_kernel, dim3(blocks), kZeroThreads, 0, stream, out, bytes);
    zero_kernel<<<blocks, kZeroThreads, 0, stream>>>(out, bytes);
    return cudaGetLastError();
}

template <typename TG, typename TO>
cudaError_t launch_run_sum(const RunArgs& R, bool vec, unsigned blocks, cudaStream_t stream) {
    auto kernel = R.count <= kShortCount ? (vec ? run_sum_kernel<TG, TO, true, kShortChunk> : run_sum_kernel<TG, TO, false, kShortChunk>)
                                         : (vec ? run_sum_kernel<TG, TO, true, kLongChunk> : run_sum_kernel<TG, TO, false, kLongChunk>);
    return launch_dependent(kernel, dim3(blocks), kRunWarps * 32, 0, stream, R);
}

}  // namespace

cudaError_t launch_embedding(const EmbedFwd& L, cudaStream_t stream) {
    const int nseg = static_cast<int>((L.dim + kSeg - 1) / kSeg);
    const unsigned blocks = static_cast<unsigned>((L.count + kFwdWarps - 1) / kFwdWarps * nseg);
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
    // the order within the call: by class and token, or by token; either keeps
    // the tokens of a row together and their positions ascending
    const int classes = static_cast<int>(std::min<long long>(std::min(num_sms, kMostClasses), L.vocab));
    const bool by_class = L.count > 0 && L.count <= kClassTokens && L.vocab <= kClassVocab &&
                          (L.vocab + classes - 1) / classes <= kClassRows;
    // The zeros' own launch writes 7.5 TB/s from the first microseconds on and the
    // rows that tokens ask for twice, the classes' CTAs 6.3 TB/s of the others
    // after the ordering: even where a sixth of the rows is asked for.  (One input
    // set in a loop, distinct to language-like tokens: 8192 of 50257 x 768 bf16
    // 22.8-26.6 instead of 24.1-28.6 us, 16384 of 128256 x 4096 190 instead of 203-212,
    // 300 of 128256 x 2001 fp32 147-149 instead of 194-197.)  A launch more costs as
    // much as it gains below 8 MiB (300 of 2500 x 768 fp32: 10.4 and 10.3).
    constexpr long long kZeroApart = 8ll << 20;
    const bool zero_apart = !by_class || (L.vocab * L.dim * dtype_size(L.out_dt) >= kZeroApart && L.count * 6 <= L.vocab);
    int side = 0;
    cudaError_t e = cudaSuccess;
    if (L.count > 0) {
        e = by_class ? launch_class_group(L, classes, !zero_apart, lay, stream) : launch_sort(L, lay, stream, &side);
        ++*launches;
    }
    if (e == cudaSuccess && zero_apart) {
        e = launch_zero(L, L.count > 0, stream);
        ++*launches;
    }
    if (e != cudaSuccess || L.count == 0) return e;

    RunArgs R{};
    R.keys = reinterpret_cast<const unsigned*>(ws + lay.keys[side]);
    R.pos = reinterpret_cast<const unsigned*>(ws + lay.pos[side]);
    R.count = static_cast<unsigned>(L.count);
    R.vocab = static_cast<unsigned>(L.vocab);
    R.grad = L.grad;
    R.ld = L.ld;
    R.dim = L.dim;
    R.scale = L.scale;
    R.out = L.out;
    R.partial = reinterpret_cast<float*>(ws + lay.partial);
    R.done = reinterpret_cast<unsigned*>(ws + lay.done);
    R.nslab = static_cast<int>((L.dim + 255) / 256);
    const unsigned blocks = static_cast<unsigned>((lay.chunks + kRunWarps - 1) / kRunWarps * R.nslab);
    const bool vec = rows_vec_ok(L.grad, L.ld, L.grad_dt) && rows_vec_ok(L.out, L.dim, L.out_dt) && L.dim % 8 == 0;
    ++*launches;
    if (L.grad_dt == DT_F32)
        return L.out_dt == DT_F32 ? launch_run_sum<float, float>(R, vec, blocks, stream)
                                  : launch_run_sum<float, __nv_bfloat16>(R, vec, blocks, stream);
    return L.out_dt == DT_F32 ? launch_run_sum<__nv_bfloat16, float>(R, vec, blocks, stream)
                              : launch_run_sum<__nv_bfloat16, __nv_bfloat16>(R, vec, blocks, stream);
}

}  // namespace muon
