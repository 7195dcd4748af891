// Softmax cross entropy of the output head, with the gradients of the hidden
// states and of the head's weight, in pieces of the vocabulary: the tokens x
// vocab matrix of logits is never kept.
//
//   l = h W^T,  lse_t = log sum_v exp(l_tv),  loss_t = lse_t - l_t,y(t)
//   P_tv = dloss_t (exp(l_tv - lse_t) - [v = y(t)]),  dh = P W,  dW = P^T h
//
// Forward is one product whose epilogue reduces each 128-column stretch of a
// row to (max, sum of exp) and picks the target's logit; a second kernel joins
// a row's stretches.  Backward walks the vocabulary in pieces.  For each piece
// one product makes the logits again and its epilogue writes P as bf16 into a
// tokens x piece buffer; one launch then runs both products that read it, the
// piece's rows of dW and its share of dh (fp32, added up over the pieces).
// That is 2 T V D operations forward and 6 T V D backward: the products are
// the bound, on the tensor cores, except for short batches, where reading the
// weight is.
//
// Tokens whose target is ignored take no part: if there are any, the rows that
// count are first copied together, so they cost nothing in the products, and
// whatever an ignored row holds (infinities, NaN) reaches no result.
//
// P is rounded to bf16 for the two products that read it.  Its common factor,
// the largest |dloss|, is left out and multiplied into the fp32 sums instead:
// with equal dloss (the mean's gradient) a target's entry is then p - 1, not
// dloss (p - 1), whose rounding would be off the same way in every row.  What
// the rounding takes off the target's entry, the largest of its row, is added
// back to dh in fp32.
//
// The products use CTA pairs (tcgen05 cta_group::2, M = 256, N = 256, K = 16,
// bf16 operands, fp32 accumulation in tensor memory) fed by TMA:
//   warp 10     claims a pair's tiles but the first from a counter (leader CTA)
//               and publishes them to both CTAs through a ring in shared memory
//   warp 0      TMA producer: 64-wide K slices into a 5-stage ring
//   warp 1      tensor memory owner, MMA issuer (leader CTA)
//   warps 2..9  epilogue; two accumulators, so it overlaps the next tile
// Row blocks run fastest in the forward order, so the pairs share a few weight
// tiles at a time and the weight is read from memory about once (20000 x 2048,
// 2048 tokens: 90 MB of 82; tensor pipe 84 % active).  Backward, dh tiles come
// first: their K is the piece, the longest.
//
// The tensor cores add into their fp32 accumulator without rounding to
// nearest, so long sums drift towards zero, the large ones most: the targets'
// logits, which a trained model makes large.  An epilogue warp therefore makes
// the target's logit of its rows itself, in fp32 with every addition rounded to
// nearest, while the tile's MMAs run, and puts it in the place of the
// product's, forward and backward alike.  Losses of targets that lead by 7 are
// then off by 1e-7 of their value at dim 768 and 1.1e-6 at 4096, where what is
// left is the drift of the sum of the others (1.3e-6 and 4e-6 with the
// product's; a plain fp32 product: 5e-7 and 8e-7), for no measurable time.
// Ending the sums every 768 elements and adding the parts in registers gave
// 7e-7 at 4096 and cost 9-14 % of the forward product.
//
// Measured (calls behind one another on changing inputs): loss and gradients of
// 8192 tokens, 50257 x 768, 2.18-2.20 ms (2.53 TFLOP: 1.15 PFLOP/s); 3/4 of 4096
// tokens, 128256 x 4096, 9.73-9.81 ms (12.9 TFLOP: 1.32 PFLOP/s under the power
// cap, where a plain bf16 product sustains 1.43); 61 tokens, 5003 x 256, forward
// 14.3 us (11.0 replayed from a graph).
//
// Every wait is bounded; on expiry the kernel records a timeout in the device
// status word, drains its copies and MMAs, frees tensor memory and exits.
#include <algorithm>
#include <atomic>
#include <cstring>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "epilogue.cuh"
#include "lane.h"
#include "pdl.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int BM = 128;        // rows per CTA
constexpr int BMP = 2 * BM;    // rows per CTA pair
constexpr int BN = 256;        // columns per tile
constexpr int BNH = BN / 2;    // B rows loaded per CTA
constexpr int BK = 64;
constexpr int STAGES = 5;
constexpr int A_BYTES = BM * BK * 2;
constexpr int B_BYTES = BNH * BK * 2;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int MN_BLOCK_BYTES = 64 * BK * 2;  // one 64 (MN) x 64 (K) box
constexpr int EPI_WARPS = 8;
constexpr int SCHED_WARP = 2 + EPI_WARPS;
constexpr int NUM_THREADS = 96 + 32 * EPI_WARPS;
constexpr uint32_t TMEM_COLS = 512;  // two accumulators of 256 fp32 columns
constexpr int STORE_BOX_BYTES = 64 * 32;  // 32 rows of 64 bytes
constexpr int STORE_BYTES = EPI_WARPS * 2 * STORE_BOX_BYTES;
constexpr int RING = 4;
constexpr size_t SMEM_BYTES = STAGES * STAGE_BYTES + STORE_BYTES + 1024 /*align slack*/ + 1024 /*barriers*/;
static_assert(SMEM_BYTES <= 232448, "over the 227 KB of shared memory a CTA may use");

constexpr int PART_COLS = 128;  // columns of one (max, sum) pair

// exp(x) as 2^(x log2 e) on the special function unit.  The unit's relative
// error is about 2^-22; the roundings of x log2 e and of the constant add up to
// |x| 2^-24 and |x| 2^-26: 2^-20 to 2^-19 in all at |x| = 12.  The logits' own error is
// larger, and P is rounded by up to 2^-8 of its value.  Callers pass differences
// to a row's maximum or log sum, formed before the scaling.
__device__ __forceinline__ float exp_diff(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}

// Row index of a token in the copied rows, or why it has none.
constexpr int kIgnored = -1, kBadTarget = -2;

enum Mode { STATS = 0, PROB = 1, GRAD = 2 };

struct HeadGemm {
    CUtensorMap a;      // STATS, PROB: copied hidden rows, K-major.   GRAD: P, K-major (dh)
    CUtensorMap b;      // STATS, PROB: weight, K-major.               GRAD: weight, MN-major (dh)
    CUtensorMap a2;     // GRAD: P, MN-major (dW)
    CUtensorMap b2;     // GRAD: copied hidden rows, MN-major (dW)
    CUtensorMap all;    // the caller's hidden rows as a or b2: read instead where every row counts
    CUtensorMap o;      // PROB: P store.                              GRAD: fp32 dh slots
    CUtensorMap o2;     // GRAD: dW store
    const __nv_bfloat16* hidden;  // STATS, PROB: the caller's hidden rows, `ldh` apart,
    const __nv_bfloat16* rows;    // the copied ones, `dim` apart,
    const __nv_bfloat16* weight;  // and the weight's rows, for the targets' logits
    long long ldh;
    const int* nvalid;  // rows that count
    unsigned* ticket;   // tiles claimed after the pairs' first ones
    const int* target;  // per copied row
    const float* lse;
    const float* dloss; // per copied row, over *scale
    const float* scale; // GRAD: the common factor of dloss
    float* rest;        // PROB: per copied row, what rounding took off the target's entry
    int tokens;         // all rows
    float2* part;       // STATS: (max, sum) [2 * vocab tiles][row_pitch]
    float* tlogit;      // STATS: the target's logit per copied row
    long long row_pitch;
    int vocab, dim;
    int v0;             // first vocabulary row of the piece
    int vtiles;         // 256-wide vocabulary tiles (of the piece)
    int splits;         // GRAD: stretches of the piece that dh tiles are cut into along K (0: no dh)
    int dw_tiles;       // GRAD: 256-row tiles of dW, vtiles or 0 (no dW)
    int split_slices;   // GRAD: K slices per stretch
    int add;            // GRAD: add to the dh slots (a piece after the first)
    DeviceStatus* status;
    unsigned long long wait_ns;
};

struct Shared {
    uint64_t full[STAGES];   // leader: both CTAs' operand bytes landed
    uint64_t empty[STAGES];  // each CTA: its slot may be refilled
    uint64_t tfull[2];       // each CTA: accumulator ready
    uint64_t tempty[2];      // leader: both CTAs' epilogue warps drained the accumulator
    uint64_t sfull[RING];    // each CTA: ring slot holds a tile
    uint64_t sempty_l[RING]; // leader: the leader's readers have read the slot
    uint64_t sempty_p[RING]; // leader: the peer's readers have read the slot
    uint64_t drain;
    uint32_t ring[RING];
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(Shared) <= 1024, "barrier area");
constexpr uint32_t kEnd = 0xFFFFFFFFu;

// One tile: A rows [m0, m0 + 256) and B rows [n0, n0 + 256) over K slices
// [k0, k0 + nk).
struct Tile {
    int m0, n0, k0, nk;
    int dw;     // GRAD: 1 = a tile of dW, 0 = of dh
    int split;  // GRAD: dh slot
};

// Rows of the products: the rows that count, rounded up to whole tiles (at
// least one, so that a batch without any still writes its zero gradients).
__device__ __forceinline__ int row_blocks(int nvalid) { return max(1, (nvalid + BMP - 1) / BMP); }

template <int MODE>
__device__ __forceinline__ uint32_t tile_count(const HeadGemm& L, int nvalid) {
    const int R = row_blocks(nvalid);
    if (MODE != GRAD) return static_cast<uint32_t>(R) * L.vtiles;
    const int nd = (L.dim + BN - 1) / BN;
    return static_cast<uint32_t>(R) * nd * L.splits + static_cast<uint32_t>(L.dw_tiles) * nd;
}

template <int MODE>
__device__ __forceinline__ Tile tile_at(const HeadGemm& L, int nvalid, uint32_t t) {
    const uint32_t R = row_blocks(nvalid);
    Tile x{};
    if (MODE != GRAD) {
        // row blocks run fastest: the pairs share a few weight tiles at a time
        x.m0 = static_cast<int>(t % R) * BMP;
        x.n0 = static_cast<int>(t / R) * BN;
        x.nk = (L.dim + BK - 1) / BK;
        return x;
    }
    const uint32_t nd = (L.dim + BN - 1) / BN;
    const uint32_t nh = R * nd * L.splits;
    if (t < nh) {  // dh first: its K is the longest
        const uint32_t s = t / (R * nd), u = t - s * (R * nd);
        x.split = static_cast<int>(s);
        x.m0 = static_cast<int>(u / nd) * BMP;
        x.n0 = static_cast<int>(u % nd) * BN;
        x.k0 = static_cast<int>(s) * L.split_slices;
        x.nk = min(L.split_slices, L.vtiles * (BN / BK) - x.k0);
    } else {
        t -= nh;
        x.dw = 1;
        x.m0 = static_cast<int>(t / nd) * BMP;
        x.n0 = static_cast<int>(t % nd) * BN;
        x.nk = max(1, (nvalid + BK - 1) / BK);
    }
    return x;
}

// The first tile of a pair is its own number: all its warps know it without the
// scheduler.
template <int MODE>
__device__ __forceinline__ uint32_t first_tile(const HeadGemm& L, int nvalid) {
    const uint32_t t = blockIdx.x / 2;
    return t < tile_count<MODE>(L, nvalid) ? t : kEnd;
}

__device__ __forceinline__ void record_timeout(Shared* sh, DeviceStatus* st) {
    atomicOr(&st->bits, ST_TIMEOUT);
    *reinterpret_cast<volatile int*>(&sh->abort) = 1;
}

__device__ __forceinline__ void st_shared_cluster_u32(uint32_t cluster_addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}

// Writer of the tile ring (one thread of the leader CTA): a tile goes into the
// same slot of both CTAs' rings once every reader has read the slot's last one.
struct RingWriter {
    int slot = 0;
    uint32_t phase = 0;
    __device__ bool push(Shared* sh, uint32_t tile, unsigned long long limit) {
        volatile int* abort_flag = &sh->abort;
        if (!mbar_wait(&sh->sempty_l[slot], phase ^ 1u, abort_flag, limit)) return false;
        if (!mbar_wait_cluster(&sh->sempty_p[slot], phase ^ 1u, abort_flag, limit)) return false;
        *reinterpret_cast<volatile uint32_t*>(&sh->ring[slot]) = tile;
        mbar_arrive(&sh->sfull[slot]);
        st_shared_cluster_u32(map_to_cta(smem_u32(&sh->ring[slot]), 1), tile);
        mbar_arrive_cluster(map_to_cta(smem_u32(&sh->sfull[slot]), 1));
        if (++slot == RING) {
            slot = 0;
            phase ^= 1u;
        }
        return true;
    }
};

struct RingReader {
    int slot = 0;
    uint32_t phase = 0;
    __device__ bool pop(Shared* sh, uint32_t& tile, bool leader, unsigned long long limit) {
        volatile int* abort_flag = &sh->abort;
        const bool got = leader ? mbar_wait(&sh->sfull[slot], phase, abort_flag, limit)
                                : mbar_wait_cluster(&sh->sfull[slot], phase, abort_flag, limit);
        if (!got) return false;
        tile = *reinterpret_cast<volatile uint32_t*>(&sh->ring[slot]);
        if (leader)
            mbar_arrive(&sh->sempty_l[slot]);
        else
            mbar_arrive_cluster(map_to_cta(smem_u32(&sh->sempty_p[slot]), 0));
        if (++slot == RING) {
            slot = 0;
            phase ^= 1u;
        }
        return true;
    }
};

template <int MODE>
__device__ void producer(const HeadGemm& L, int nvalid, uint8_t* tiles_smem, Shared* sh, uint32_t rank) {
    volatile int* abort_flag = &sh->abort;
    const unsigned long long lim = L.wait_ns;
    const bool leader = rank == 0;
    const CUtensorMap* hidden = nvalid == L.tokens ? &L.all : (MODE == GRAD ? &L.b2 : &L.a);
    int stage = 0;
    uint32_t phase = 0, issued = 0, t = first_tile<MODE>(L, nvalid);
    bool ok = true;
    RingReader rd;
    while (ok && t != kEnd) {
        const Tile x = tile_at<MODE>(L, nvalid, t);
        const int arow = x.m0 + static_cast<int>(rank) * BM, brow = x.n0 + static_cast<int>(rank) * BNH;
        for (int i = 0; i < x.nk; ++i) {
            if (!mbar_wait(&sh->empty[stage], phase ^ 1u, abort_flag, lim)) {
                ok = false;
                break;
            }
            uint8_t* sa = tiles_smem + stage * STAGE_BYTES;
            uint8_t* sb = sa + A_BYTES;
            const uint32_t full = map_to_cta(smem_u32(&sh->full[stage]), 0);
            if (leader) mbar_arrive_expect_tx(&sh->full[stage], 2 * STAGE_BYTES);
            const int k = (x.k0 + i) * BK;
            if (MODE != GRAD) {
                tma_load_3d_pair(sa, hidden, full, k, arow, 0);
                tma_load_3d_pair(sb, &L.b, full, k, L.v0 + brow, 0);
            } else if (!x.dw) {
                tma_load_3d_pair(sa, &L.a, full, k, arow, 0);
#pragma unroll
                for (int j = 0; j < BNH / 64; ++j)
                    tma_load_3d_pair(sb + j * MN_BLOCK_BYTES, &L.b, full, brow + 64 * j, L.v0 + k, 0);
            } else {
#pragma unroll
                for (int j = 0; j < BM / 64; ++j)
                    tma_load_3d_pair(sa + j * MN_BLOCK_BYTES, &L.a2, full, arow + 64 * j, k, 0);
#pragma unroll
                for (int j = 0; j < BNH / 64; ++j)
                    tma_load_3d_pair(sb + j * MN_BLOCK_BYTES, hidden, full, brow + 64 * j, k, 0);
            }
            ++issued;
            if (++stage == STAGES) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (ok) ok = rd.pop(sh, t, leader, lim);
    }
    if (!ok) record_timeout(sh, L.status);
    // the last fills of every stage must have landed before the pair exits
    if (leader) {
        int never = 0;
        for (uint32_t i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i) {
            if (!mbar_wait(&sh->full[i % STAGES], (i / STAGES) & 1u, &never, lim)) {
                atomicOr(&L.status->bits, ST_TIMEOUT);
                break;
            }
        }
    }
}

template <int MODE>
__device__ void scheduler(const HeadGemm& L, int nvalid, Shared* sh) {
    const uint32_t n = tile_count<MODE>(L, nvalid), pairs = gridDim.x / 2;
    RingWriter wr;
    if (first_tile<MODE>(L, nvalid) == kEnd) return;
    while (true) {
        const uint32_t t = pairs + atomicAdd(L.ticket, 1u);
        if (!wr.push(sh, t < n ? t : kEnd, L.wait_ns)) {
            record_timeout(sh, L.status);
            return;
        }
        if (t >= n) return;
    }
}

template <int MODE>
__device__ void mma_issuer(const HeadGemm& L, int nvalid, uint8_t* tiles_smem, Shared* sh, uint32_t tmem_base) {
    volatile int* abort_flag = &sh->abort;
    const unsigned long long lim = L.wait_ns;
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0, t = first_tile<MODE>(L, nvalid);
    bool ok = true, issued_any = false;
    const uint32_t tiles_base = smem_u32(tiles_smem);
    RingReader rd;
    while (ok && t != kEnd) {
        const Tile x = tile_at<MODE>(L, nvalid, t);
        const int a_mn = MODE == GRAD && x.dw, b_mn = MODE == GRAD;
        const uint32_t idesc = make_instr_desc(1, a_mn, b_mn, BMP, BN);
        if (!mbar_wait(&sh->tempty[acc], acc_phase ^ 1u, abort_flag, lim)) {
            ok = false;
            break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
        for (int i = 0; i < x.nk; ++i) {
            if (!mbar_wait(&sh->full[stage], phase, abort_flag, lim)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t a = tiles_base + stage * STAGE_BYTES, b = a + A_BYTES;
#pragma unroll
            for (int k = 0; k < BK / 16; ++k) {
                // K-major: 16 elements further inside the swizzled row; MN-major: 16 K rows further
                const uint64_t ad = a_mn ? make_smem_desc(a + k * 2048, MN_BLOCK_BYTES, 1024)
                                         : make_smem_desc(a + k * 32, 16, 1024);
                const uint64_t bd = b_mn ? make_smem_desc(b + k * 2048, MN_BLOCK_BYTES, 1024)
                                         : make_smem_desc(b + k * 32, 16, 1024);
                umma_f16_pair(d_tmem, ad, bd, idesc, (i > 0 || k > 0) ? 1u : 0u);
            }
            issued_any = true;
            umma_commit_pair(&sh->empty[stage], 0x3);
            if (++stage == STAGES) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (!ok) break;
        umma_commit_pair(&sh->tfull[acc], 0x3);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
        ok = rd.pop(sh, t, true, lim);
    }
    if (!ok) {
        record_timeout(sh, L.status);
        if (issued_any) {  // this thread's MMAs end before tensor memory is released
            int never = 0;
            umma_commit_pair(&sh->drain, 0x1);
            if (!mbar_wait(&sh->drain, 0, &never, lim)) atomicOr(&L.status->bits, ST_TIMEOUT);
        }
    }
}

// Scalar products of N pairs of rows of 8 * units bf16 values, by a warp:
// products are exact in fp32, the fused additions and the tree's are rounded to
// nearest.
template <int N>
__device__ __forceinline__ void warp_dot(const __nv_bfloat16* const (&a)[N], const __nv_bfloat16* const (&b)[N],
                                         int units, int lane, float (&sum)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) sum[i] = 0.f;
#pragma unroll(N == 1 ? 4 : 1)
    for (int u = lane; u < units; u += 32) {
        uint4 p[N], q[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            p[i] = reinterpret_cast<const uint4*>(a[i])[u];
            q[i] = reinterpret_cast<const uint4*>(b[i])[u];
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float x[8], y[8];
            unpack8(p[i], DT_BF16, x);
            unpack8(q[i], DT_BF16, y);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[i] = fmaf(x[j], y[j], sum[i]);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
        for (int i = 0; i < N; ++i) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
    }
}

// Takes the N lowest lanes off `here` (at least one; where fewer are left, the
// last of them again) and makes their rows' target logits.
template <int N>
__device__ __forceinline__ void target_logits(const HeadGemm& L, int nvalid, int row0, int y, int lane,
                                              unsigned& here, float& ly) {
    int of[N];
    const __nv_bfloat16 *h[N], *w[N];
    float l[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        of[i] = __ffs(here) - 1;
        if (here & (here - 1) || i == N - 1) here &= here - 1;
        const long long r = row0 + of[i], v = L.v0 + __shfl_sync(0xffffffffu, y, of[i]);
        h[i] = nvalid == L.tokens ? L.hidden + r * L.ldh : L.rows + r * L.dim;
        w[i] = L.weight + v * L.dim;
    }
    warp_dot<N>(h, w, L.dim / 8, lane, l);
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (lane == of[i]) ly = l[i];
}

template <int MODE>
__device__ void epilogue_warps(const HeadGemm& L, int nvalid, Shared* sh, uint32_t stg, uint32_t tmem_base, int warp,
                               int lane, uint32_t rank) {
    volatile int* abort_flag = &sh->abort;
    const unsigned long long lim = L.wait_ns;
    const int q = warp & 3;             // tensor memory lane quarter of this warp
    const int part = (warp - 2) >> 2;   // column half of the tile
    const uint32_t tempty_leader[2] = {map_to_cta(smem_u32(&sh->tempty[0]), 0),
                                       map_to_cta(smem_u32(&sh->tempty[1]), 0)};
    int acc = 0;
    uint32_t acc_phase = 0, nstored = 0;
    const uint32_t row_off = static_cast<uint32_t>(lane) * 64;
    const uint32_t sw = (static_cast<uint32_t>(lane) >> 1) & 3u;
    RingReader rd;
    // one 64-byte-wide box of this warp's 32 rows: 16 fp32 or 32 bf16 columns
    auto store_box = [&](const CUtensorMap* map, const uint4 (&unit)[4], int col, int row, int z, bool add) {
        const uint32_t buf = stg + (nstored & 1u) * STORE_BOX_BYTES;
        if (lane == 0 && nstored >= 2) bulk_wait_read<1>();
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 4; ++u) st_shared_v4(buf + row_off + ((static_cast<uint32_t>(u) ^ sw) << 4), unit[u]);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
            if (add)
                tma_reduce_add_3d(map, buf, col, row, z);
            else
                tma_store_3d(map, buf, col, row, z);
            bulk_commit();
        }
        ++nstored;
    };
    uint32_t t = first_tile<MODE>(L, nvalid);
    while (t != kEnd) {
        const Tile x = tile_at<MODE>(L, nvalid, t);
        const int row0 = x.m0 + static_cast<int>(rank) * BM + q * 32, row = row0 + lane;
        const int cbase = x.n0 + part * PART_COLS;
        int y = -1;
        float lse = 0.f, dl = 0.f, ly = 0.f;
        if (MODE != GRAD) {
            if (row < nvalid) {
                y = L.target[row] - L.v0;  // column of the target in this piece
                if (MODE == PROB) {
                    lse = L.lse[row];
                    dl = L.dloss[row];
                }
            }
            // the targets' logits of the rows that have theirs in these columns
            unsigned here = __ballot_sync(0xffffffffu, y >= cbase && y < cbase + PART_COLS);
            while (here) {
                if (here & (here - 1))
                    target_logits<4>(L, nvalid, row0, y, lane, here, ly);
                else
                    target_logits<1>(L, nvalid, row0, y, lane, here, ly);
            }
        }
        const bool got = mbar_wait(&sh->tfull[acc], acc_phase, abort_flag, lim);
        if (!__all_sync(0xffffffffu, got)) {
            if (lane == 0) record_timeout(sh, L.status);
            break;
        }
        tc_fence_after();
        const float scale = MODE == GRAD ? *L.scale : 1.f;
        float m = -INFINITY, s = 0.f;  // STATS: maximum and sum of exp(l - m)
#pragma unroll 1
        for (int c = 0; c < PART_COLS; c += 32) {
            const int col0 = cbase + c;
            const int ncols = (MODE == GRAD ? L.dim : L.vocab - L.v0) - col0;  // columns left
            if (MODE != PROB && ncols <= 0) break;
            uint32_t r[32];
            __syncwarp();
            tmem_ld_32x32b_x32(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * BN + part * PART_COLS + c, r);
            tmem_wait_ld();
            float v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
            if (MODE == STATS) {
                const int at = y - col0;
                if (__any_sync(0xffffffffu, at >= 0 && at < 32)) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j == at) v[j] = ly;
                    if (at >= 0 && at < 32) L.tlogit[row] = ly;
                }
                if (ncols < 32) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j >= ncols) v[j] = -INFINITY;
                }
                // four chains of each kind
                float t4[4] = {m, v[1], v[2], v[3]};
#pragma unroll
                for (int j = 0; j < 32; ++j) t4[j % 4] = fmaxf(t4[j % 4], v[j]);
                const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
                // all terms so far are zero: any finite reference will do
                const float ref = top == -INFINITY ? 0.f : top;
                float s4[4] = {s * exp_diff(m - ref), 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < 32; ++j) s4[j % 4] += exp_diff(v[j] - ref);
                s = (s4[0] + s4[1]) + (s4[2] + s4[3]);
                m = top;
            } else if (MODE == PROB) {
                const int at = y - col0;
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = dl * exp_diff(v[j] - lse);
                if (__any_sync(0xffffffffu, at >= 0 && at < 32)) {
                    // (lse is one fp32 number: off by up to 2^-24 |lse| dl, which is all
                    // there is of g where the loss is that small)
                    const float g = dl * exp_diff(ly - lse) - dl;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j == at) v[j] = g;
                    if (at >= 0 && at < 32) L.rest[row] = g - __bfloat162float(__float2bfloat16_rn(g));
                }
                // rows behind the last that counts and columns behind the
                // vocabulary hold zeros, whatever the accumulator holds
                if (row0 + 32 > nvalid || ncols < 32) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (row >= nvalid || j >= ncols) v[j] = 0.f;
                }
                uint4 u[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) u[i] = pack8(v + 8 * i, DT_BF16);
                store_box(&L.o, u, col0, row0, 0, false);
            } else if (x.dw) {
                if (L.v0 + row0 >= L.vocab) continue;  // warp-uniform
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] *= scale;
                uint4 u[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) u[i] = pack8(v + 8 * i, DT_BF16);
                store_box(&L.o2, u, col0, L.v0 + row0, 0, false);
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (16 * h >= ncols) continue;  // no box starts past the last column
                    uint4 u[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t* f = r + 16 * h + 4 * i;
                        u[i] = make_uint4(f[0], f[1], f[2], f[3]);
                    }
                    store_box(&L.o, u, col0 + 16 * h, row0, x.split, L.add != 0);
                }
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty_leader[acc]);
        if (MODE == STATS) L.part[static_cast<long long>(cbase / PART_COLS) * L.row_pitch + row] = make_float2(m, s);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
        int got_tile = 1;
        if (lane == 0) got_tile = rd.pop(sh, t, rank == 0, lim) ? 1 : 0;
        if (!__shfl_sync(0xffffffffu, got_tile, 0)) {
            if (lane == 0) record_timeout(sh, L.status);
            break;
        }
        t = __shfl_sync(0xffffffffu, t, 0);
    }
    if (lane == 0) bulk_wait_all();  // the staging boxes stay valid until every store has read them
    __syncwarp();
}

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NUM_THREADS, 1)
    head_gemm_kernel(const __grid_constant__ HeadGemm L) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* tiles_smem =
        reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* store_smem = tiles_smem + STAGES * STAGE_BYTES;
    Shared* sh = reinterpret_cast<Shared*>(store_smem + STORE_BYTES);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_cta_rank();
    allow_successor();
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&sh->full[s], 1);
            mbar_init(&sh->empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&sh->tfull[a], 1);
            mbar_init(&sh->tempty[a], 2 * EPI_WARPS);
        }
        for (int r = 0; r < RING; ++r) {
            mbar_init(&sh->sfull[r], 1);
            mbar_init(&sh->sempty_l[r], 2 + EPI_WARPS);
            mbar_init(&sh->sempty_p[r], 1 + EPI_WARPS);
        }
        mbar_init(&sh->drain, 1);
        sh->abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(&sh->tmem_base, TMEM_COLS);
        tmem_relinquish_pair();
    }
    if (warp == 0 && lane == 0) {  // the maps' first use waits for their fetch otherwise
        tma_prefetch_map(&L.a);
        tma_prefetch_map(&L.b);
        tma_prefetch_map(&L.all);
        if (MODE == GRAD) {
            tma_prefetch_map(&L.a2);
            tma_prefetch_map(&L.b2);
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = sh->tmem_base;
    wait_predecessor();
    const int nvalid = *reinterpret_cast<const volatile int*>(L.nvalid);
    if (warp == 0) {
        if (lane == 0) producer<MODE>(L, nvalid, tiles_smem, sh, rank);
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) mma_issuer<MODE>(L, nvalid, tiles_smem, sh, tmem_base);
    } else if (warp == SCHED_WARP) {
        if (lane == 0 && rank == 0) scheduler<MODE>(L, nvalid, sh);
    } else {
        epilogue_warps<MODE>(L, nvalid, sh, smem_u32(store_smem + (warp - 2) * 2 * STORE_BOX_BYTES), tmem_base, warp,
                             lane, rank);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // no CTA leaves while its peer may still touch its memory or tensor memory
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
}

// ---- rows that count -------------------------------------------------------------

struct RowsArgs {
    const void* targets;
    int targets_i64;
    int tokens, vocab, dim;
    long long ignore;
    const __nv_bfloat16* hidden;
    long long ldh;
    const float* lse_in;    // backward, or null
    const float* dloss_in;  // backward, or null
    __nv_bfloat16* rows;    // copied rows, dim each
    int* index;             // per token: its copied row, kIgnored or kBadTarget
    int* target;            // per copied row
    float* lse;             // per copied row (backward)
    float* dloss;           // over *scale
    float* scale;           // or null
    int* nvalid;
    unsigned* tickets;
    int ntickets;
    DeviceStatus* status;
};

constexpr int kRowsThreads = 1024;
constexpr int kRowsWarps = kRowsThreads / 32;
constexpr int kRowsMostCtas = 256;  // each reads all targets: two CTAs per SM, 8 bytes x tokens x 256 from L2

__device__ __forceinline__ long long target_at(const RowsArgs& A, int t) {
    return A.targets_i64 ? static_cast<const long long*>(A.targets)[t] : static_cast<const int*>(A.targets)[t];
}
__device__ __forceinline__ bool counts(const RowsArgs& A, long long y) {
    return y != A.ignore && y >= 0 && y < A.vocab;
}

// End of CTA `cta`'s stretch of `per` tokens; cta * per + per may pass 2^31 where
// the tokens do not.
__host__ __device__ constexpr int rows_end(unsigned cta, int per, int tokens) {
    const unsigned end = cta * static_cast<unsigned>(per) + static_cast<unsigned>(per);
    return end < static_cast<unsigned>(tokens) ? static_cast<int>(end) : tokens;
}
static_assert(rows_end(0, 32, 20) == 20 && rows_end(1, 32, 100) == 64, "stretches");
static_assert(rows_end(255, 1 << 23, 0x7fffffff - 1024) == 0x7fffffff - 1024, "the most tokens a call may have");

// Finds the place of every row that counts among those that do and, if some do
// not, copies the ones that do together, in order; the copied rows up to the
// next multiple of 256 are zeroed.  A CTA has `per` tokens and counts all
// targets before them itself: 1024 threads, so that this is a trip or two to L2
// (8192 tokens: 8 us forward, 9 backward; 256 threads in 1024 CTAs 12 and 17).
__global__ void __launch_bounds__(kRowsThreads) head_rows_kernel(const RowsArgs A, int per) {
    __shared__ int red[2][kRowsWarps];
    __shared__ float red_dl[kRowsWarps];
    __shared__ int warp_n[kRowsWarps];
    __shared__ int dst_of[kRowsThreads];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    allow_successor();
    const int t0 = blockIdx.x * per, t1 = rows_end(blockIdx.x, per, A.tokens);
    int before = 0, all = 0;
    float top = 0.f;
#pragma unroll 8
    for (int t = tid; t < A.tokens; t += kRowsThreads) {
        const bool c = counts(A, target_at(A, t));
        all += c ? 1 : 0;
        if (t < t0) before += c ? 1 : 0;
        if (A.dloss_in && c) top = fmaxf(top, fabsf(A.dloss_in[t]));
    }
    before = __reduce_add_sync(0xffffffffu, before);
    all = __reduce_add_sync(0xffffffffu, all);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) {
        red[0][warp] = before;
        red[1][warp] = all;
        red_dl[warp] = top;
    }
    __syncthreads();
    before = __reduce_add_sync(0xffffffffu, red[0][lane]);
    all = __reduce_add_sync(0xffffffffu, red[1][lane]);
    top = red_dl[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // the common factor of dloss; 1 where it would not be one
    const float scale = top > 0.f && top <= 3.4e38f ? top : 1.f;
    if (blockIdx.x == 0) {
        if (tid == 0) {
            *A.nvalid = all;
            if (A.scale) *A.scale = scale;
        }
        for (int i = tid; i < A.ntickets; i += kRowsThreads) A.tickets[i] = 0;
    }
    const int units = A.dim / 8;  // 16-byte units of a row
    for (int s0 = t0; s0 < t1; s0 += kRowsThreads) {
        const int t = s0 + tid;
        const bool in = t < t1;
        const long long y = in ? target_at(A, t) : A.ignore;
        const bool on = in && counts(A, y);
        const unsigned mask = __ballot_sync(0xffffffffu, on);
        if (lane == 0) warp_n[warp] = __popc(mask);
        __syncthreads();
        const int n = warp_n[lane];
        const int r = before + __reduce_add_sync(0xffffffffu, lane < warp ? n : 0) + __popc(mask & ((1u << lane) - 1));
        before += __reduce_add_sync(0xffffffffu, n);
        dst_of[tid] = on ? r : -1;
        if (on) {
            A.target[r] = static_cast<int>(y);
            if (A.dloss_in) {
                A.lse[r] = A.lse_in[t];
                A.dloss[r] = A.dloss_in[t] / scale;
            }
        }
        if (in) {
            const bool bad = !on && y != A.ignore;
            A.index[t] = on ? r : (bad ? kBadTarget : kIgnored);
            if (bad) {
                atomicMin(&A.status->first_bad_token, t);
                atomicOr(&A.status->bits, ST_INDEX);
            }
        }
        __syncthreads();
        if (all == A.tokens) continue;  // the products read the caller's rows
        for (int i = warp; i < min(kRowsThreads, t1 - s0); i += kRowsWarps) {
            if (dst_of[i] < 0) continue;
            const uint4* src = reinterpret_cast<const uint4*>(A.hidden + (s0 + i) * A.ldh);
            uint4* dst = reinterpret_cast<uint4*>(A.rows + static_cast<long long>(dst_of[i]) * A.dim);
#pragma unroll 8
            for (int u = lane; u < units; u += 32) dst[u] = src[u];
        }
        __syncthreads();
    }
    if (all == A.tokens) return;
    // rows behind the last
    const unsigned end = max(BMP, (all + BMP - 1) / BMP * BMP);
    for (unsigned r = all + blockIdx.x * kRowsWarps + warp; r < end; r += gridDim.x * kRowsWarps) {
        uint4* dst = reinterpret_cast<uint4*>(A.rows + static_cast<long long>(r) * A.dim);
        for (int u = lane; u < units; u += 32) dst[u] = make_uint4(0, 0, 0, 0);
    }
}

// ---- joins -----------------------------------------------------------------------

constexpr int kJoinWarps = 32;

// (max, sum) pairs as one: the sum of s exp(m - max).
__device__ __forceinline__ float2 join_pairs(float2 a, float2 b) {
    const float m = fmaxf(a.x, b.x), ref = m == -INFINITY ? 0.f : m;
    return make_float2(m, a.y * exp_diff(a.x - ref) + b.y * exp_diff(b.x - ref));
}

// A CTA joins the (max, sum) pairs of TOKENS tokens (8 or 32): group g of G takes
// the pairs g, g + G, ... of a token, eight loads in flight; then the groups'
// pairs are joined in a fixed order.  8 tokens are 128 groups, one trip to
// memory for a vocabulary of 131072, and more CTAs; 32 tokens read whole lines.
template <int TOKENS>
__global__ void __launch_bounds__(32 * kJoinWarps)
    head_join_kernel(const float2* part, int nparts, long long row_pitch, const float* tlogit, const int* index,
                     int tokens, float* loss, float* lse) {
    constexpr int kPerWarp = 32 / TOKENS, kGroups = kPerWarp * kJoinWarps;
    __shared__ float2 red[kJoinWarps][TOKENS];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int at = lane % TOKENS, g = warp * kPerWarp + lane / TOKENS;
    const int t = blockIdx.x * TOKENS + at;
    wait_predecessor();
    const int r = t < tokens ? index[t] : kIgnored;
    float m = -INFINITY, s = 0.f;  // several pairs at a time: one maximum, then independent terms
    if (r >= 0) {
        constexpr int kAhead = 8;
        for (int i0 = g; i0 < nparts; i0 += kAhead * kGroups) {
            float2 p[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int k = i0 + i * kGroups;
                p[i] = k < nparts ? part[k * row_pitch + r] : make_float2(-INFINITY, 0.f);
            }
            float top = m;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) top = fmaxf(top, p[i].x);
            const float ref = top == -INFINITY ? 0.f : top;
            s *= exp_diff(m - ref);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) s += p[i].y * exp_diff(p[i].x - ref);
            m = top;
        }
    }
    float2 v = make_float2(m, s);
#pragma unroll
    for (int o = TOKENS; o < 32; o <<= 1) {
        const float2 w = make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o));
        v = join_pairs(v, w);
    }
    if (lane < TOKENS) red[warp][at] = v;
    __syncthreads();
    if (warp != 0) return;
    // of each token's warps' pairs every kPerWarp-th to a lane, then the lanes'
    v = red[lane / TOKENS][at];
#pragma unroll
    for (int i = kPerWarp; i < kJoinWarps; i += kPerWarp) v = join_pairs(v, red[i + lane / TOKENS][at]);
#pragma unroll
    for (int o = TOKENS; o < 32; o <<= 1) {
        const float2 w = make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o));
        v = join_pairs(v, w);
    }
    if (lane >= TOKENS || t >= tokens) return;
    m = v.x;
    s = v.y;
    // the maximum is at least the target's logit and the sum at least its share,
    // so a loss made of their differences keeps its digits where it is small and
    // is never negative
    const float log_sum = logf(s);
    const float none = r == kBadTarget ? __int_as_float(0x7fc00000) : 0.f;
    lse[t] = r >= 0 ? m + log_sum : none;
    loss[t] = r >= 0 ? (m - tlogit[r]) + log_sum : none;
}

// dh: the sum of a row's slots and what rounding took off the target's entry,
// times the common factor, rounded to bf16; zero for tokens that take no part.
// AHEAD: slots whose loads are in flight at once.
template <int AHEAD>
__global__ void __launch_bounds__(128)
    head_dhidden_kernel(const float* slots, int nslots, long long slot_pitch, const int* index, const int* target,
                        const float* rest, const float* scale, const __nv_bfloat16* weight, int dim,
                        __nv_bfloat16* dhidden) {
    const int t = blockIdx.x;
    wait_predecessor();
    const int r = index[t];
    __nv_bfloat16* dst = dhidden + static_cast<long long>(t) * dim;
    const float f = *scale, d = r >= 0 ? rest[r] : 0.f;
    const __nv_bfloat16* w = weight + static_cast<long long>(r >= 0 ? target[r] : 0) * dim;
    for (int c = threadIdx.x * 8; c < dim; c += 128 * 8) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.f;
        if (r >= 0) {
            const uint4 wc = *reinterpret_cast<const uint4*>(w + c);
            const float* src = slots + static_cast<long long>(r) * dim + c;
            for (int s0 = 0; s0 < nslots; s0 += AHEAD) {
                float4 a[AHEAD], b[AHEAD];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    if (s0 + i >= nslots) break;
                    a[i] = *reinterpret_cast<const float4*>(src + (s0 + i) * slot_pitch);
                    b[i] = *reinterpret_cast<const float4*>(src + (s0 + i) * slot_pitch + 4);
                }
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    if (s0 + i >= nslots) break;
                    v[0] += a[i].x, v[1] += a[i].y, v[2] += a[i].z, v[3] += a[i].w;
                    v[4] += b[i].x, v[5] += b[i].y, v[6] += b[i].z, v[7] += b[i].w;
                }
            }
            float x[8];
            unpack8(wc, DT_BF16, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = f * fmaf(d, x[j], v[j]);
        }
        *reinterpret_cast<uint4*>(dst + c) = pack8(v, DT_BF16);
    }
}

// ---- host ------------------------------------------------------------------------

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encoder() {
    static std::atomic<EncodeTiledFn> fn{nullptr};
    if (EncodeTiledFn known = fn.load()) return known;
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
        cudaGetLastError();
        return nullptr;
    }
    fn = reinterpret_cast<EncodeTiledFn>(p);
    return reinterpret_cast<EncodeTiledFn>(p);
}

enum Box { BOX_K = 0 /* 64 x 128 rows */, BOX_MN = 1 /* 64 x 64 rows */, BOX_STORE = 2 /* 64 bytes x 32 rows */ };

bool encode(CUtensorMap* m, Box box, const void* base, bool f32, long long cols, long long rows, long long pitch,
            long long batch = 1, long long batch_pitch = 0) {
    const int es = f32 ? 4 : 2;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(batch)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(pitch) * es,
                             static_cast<cuuint64_t>(batch > 1 ? batch_pitch * es : pitch * es)};
    cuuint32_t boxd[3] = {box == BOX_STORE ? 64u / es : 64u, box == BOX_K ? 128u : (box == BOX_MN ? 64u : 32u), 1};
    cuuint32_t step[3] = {1, 1, 1};
    std::memset(m, 0, sizeof(*m));
    return encoder()(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                     const_cast<void*>(base), dims, strides, boxd, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     box == BOX_STORE ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                     box == BOX_STORE ? CU_TENSOR_MAP_L2_PROMOTION_NONE : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The CTA pairs that can be resident at once: the grid of a persistent launch.
template <int MODE>
int max_pairs() {
    static std::atomic<int> cached{-1};
    if (const int known = cached.load(); known > 0) return known;
    if (cudaFuncSetAttribute(head_gemm_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(SMEM_BYTES)) != cudaSuccess)
        return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2, 1, 1);
    cfg.blockDim = dim3(NUM_THREADS, 1, 1);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, head_gemm_kernel<MODE>, &cfg) != cudaSuccess) return 0;
    cached = n;
    return n;
}

template <int MODE>
cudaError_t launch_gemm(const HeadGemm& G, long long tiles, cudaStream_t stream) {
    // the attribute belongs to the device: set once on each
    static std::atomic<bool> raised[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !raised[dev]) {
        e = cudaFuncSetAttribute(head_gemm_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(SMEM_BYTES));
        if (e != cudaSuccess) return e;
        if (dev < 64) raised[dev] = true;
    }
    const int pairs = max_pairs<MODE>();
    if (pairs < 1) return cudaErrorInvalidConfiguration;
    const unsigned grid = 2 * static_cast<unsigned>(std::min<long long>(pairs, tiles));
    return launch_dependent(head_gemm_kernel<MODE>, dim3(grid), NUM_THREADS, SMEM_BYTES, stream, G);
}

constexpr int kPairsNominal = 74;             // CTA pairs of a B200, for the split of short batches
constexpr size_t kPieceBytes = 512ull << 20;  // of P (8192 x 50257 x 768: 2055 us; 256 MB 2257, 1 GB 2028)
constexpr int kMaxPieces = 512;

struct Layout {
    long long tpad;       // tokens rounded up to whole tiles
    long long vtiles;     // 256-wide tiles of the vocabulary
    long long piece_tiles, pieces;
    int splits, split_slices;  // of the first piece
    size_t rows, index, target, nvalid, tickets, part, tlogit, lse, dloss, rest, scale, p, slots, total;
    int ntickets;
};

Layout layout(long long tokens, long long vocab, long long dim, bool backward) {
    Layout l{};
    l.tpad = (tokens + BMP - 1) / BMP * BMP;
    l.vtiles = (vocab + BN - 1) / BN;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at = align_up(at + bytes, 1024);
        return o;
    };
    l.rows = take(2ull * l.tpad * dim);
    l.index = take(4ull * tokens);
    l.target = take(4ull * l.tpad);
    l.nvalid = take(4);
    if (!backward) {
        l.ntickets = 1;
        l.part = take(8ull * 2 * l.vtiles * l.tpad);
        l.tlogit = take(4ull * l.tpad);
    } else {
        long long most = static_cast<long long>(kPieceBytes / (2ull * BN * l.tpad));
        most = std::max(most, (l.vtiles + kMaxPieces - 1) / kMaxPieces);
        most = std::max(1ll, std::min(most, l.vtiles));
        l.pieces = (l.vtiles + most - 1) / most;
        l.piece_tiles = (l.vtiles + l.pieces - 1) / l.pieces;
        l.pieces = (l.vtiles + l.piece_tiles - 1) / l.piece_tiles;
        // K of a dh tile is the piece.  The dh tiles come first and the shorter
        // dW tiles fill up, so a tile is cut only until the pairs with the most
        // dh tiles stay below 3/5 of an equal share of the launch: fewer cuts are
        // fewer fp32 slots to write and add.  (Against 16 to a quarter of a
        // share: 512 tokens, 50257 x 768 160 instead of 174 us, 2048, 20000 x
        // 2048 435 instead of 470; 9/10 was 7 % slower at 8192, 50257 x 768,
        // 9/20, which short batches cannot reach, 15-40 % slower.)
        const long long nd = (dim + BN - 1) / BN, R = l.tpad / BMP, kv = l.piece_tiles * (BN / BK);
        const long long share = (R * nd * kv + l.piece_tiles * nd * (l.tpad / BK)) / kPairsNominal;
        long long cuts = 1, slices = kv;
        while (slices > 16 && (R * nd * cuts + kPairsNominal - 1) / kPairsNominal * slices > share * 3 / 5) {
            ++cuts;
            slices = (kv + cuts - 1) / cuts;
        }
        l.split_slices = static_cast<int>(slices);
        l.splits = static_cast<int>((kv + slices - 1) / slices);
        l.ntickets = static_cast<int>(2 * l.pieces);
        l.lse = take(4ull * l.tpad);
        l.dloss = take(4ull * l.tpad);
        l.rest = take(4ull * l.tpad);
        l.scale = take(4);
        l.p = take(2ull * l.tpad * l.piece_tiles * BN);
        l.slots = take(4ull * l.splits * l.tpad * dim);
    }
    l.tickets = take(4ull * l.ntickets);
    l.total = at;
    return l;
}

cudaError_t launch_rows(const HeadLoss& L, const Layout& l, bool backward, cudaStream_t stream) {
    char* ws = static_cast<char*>(L.workspace);
    RowsArgs A{};
    A.targets = L.targets;
    A.targets_i64 = L.targets_i64;
    A.tokens = static_cast<int>(L.tokens);
    A.vocab = static_cast<int>(L.vocab);
    A.dim = static_cast<int>(L.dim);
    A.ignore = L.ignore;
    A.hidden = static_cast<const __nv_bfloat16*>(L.hidden);
    A.ldh = L.ldh;
    A.rows = reinterpret_cast<__nv_bfloat16*>(ws + l.rows);
    A.index = reinterpret_cast<int*>(ws + l.index);
    A.target = reinterpret_cast<int*>(ws + l.target);
    if (backward) {
        A.lse_in = L.lse;
        A.dloss_in = L.dloss;
        A.lse = reinterpret_cast<float*>(ws + l.lse);
        A.dloss = reinterpret_cast<float*>(ws + l.dloss);
        A.scale = reinterpret_cast<float*>(ws + l.scale);
    }
    A.nvalid = reinterpret_cast<int*>(ws + l.nvalid);
    A.tickets = reinterpret_cast<unsigned*>(ws + l.tickets);
    A.ntickets = l.ntickets;
    A.status = L.status;
    const long long per = align_up((L.tokens + kRowsMostCtas - 1) / kRowsMostCtas, 32);
    head_rows_kernel<<<static_cast<unsigned>((L.tokens + per - 1) / per), kRowsThreads, 0, stream>>>(A, static_cast<int>(per));
    return cudaGetLastError();
}

HeadGemm gemm_args(const HeadLoss& L, const Layout& l) {
    char* ws = static_cast<char*>(L.workspace);
    HeadGemm G{};
    G.nvalid = reinterpret_cast<const int*>(ws + l.nvalid);
    G.target = reinterpret_cast<const int*>(ws + l.target);
    G.hidden = static_cast<const __nv_bfloat16*>(L.hidden);
    G.rows = reinterpret_cast<const __nv_bfloat16*>(ws + l.rows);
    G.weight = static_cast<const __nv_bfloat16*>(L.weight);
    G.ldh = L.ldh;
    G.vocab = static_cast<int>(L.vocab);
    G.dim = static_cast<int>(L.dim);
    G.tokens = static_cast<int>(L.tokens);
    G.vtiles = static_cast<int>(l.vtiles);
    G.row_pitch = l.tpad;
    G.status = L.status;
    G.wait_ns = L.wait_ns;
    return G;
}

}  // namespace

size_t head_loss_workspace(long long tokens, long long vocab, long long dim, int backward) {
    return layout(tokens, vocab, dim, backward != 0).total;
}

cudaError_t launch_head_loss(const HeadLoss& L, cudaStream_t stream, int* launches, const char** why) {
    if (!encoder()) {
        *why = "cuTensorMapEncodeTiled unavailable";
        return cudaErrorNotSupported;
    }
    const Layout l = layout(L.tokens, L.vocab, L.dim, false);
    char* ws = static_cast<char*>(L.workspace);
    HeadGemm G = gemm_args(L, l);
    if (!encode(&G.a, BOX_K, ws + l.rows, false, L.dim, l.tpad, L.dim) ||
        !encode(&G.all, BOX_K, L.hidden, false, L.dim, L.tokens, L.ldh) ||
        !encode(&G.b, BOX_K, L.weight, false, L.dim, L.vocab, L.dim)) {
        *why = "tensor map encoding failed";
        return cudaErrorInvalidValue;
    }
    cudaError_t e = launch_rows(L, l, false, stream);
    if (e != cudaSuccess) return e;
    G.ticket = reinterpret_cast<unsigned*>(ws + l.tickets);
    G.part = reinterpret_cast<float2*>(ws + l.part);
    G.tlogit = reinterpret_cast<float*>(ws + l.tlogit);
    e = launch_gemm<STATS>(G, l.tpad / BMP * l.vtiles, stream);
    if (e != cudaSuccess) return e;
    const int nparts = static_cast<int>((L.vocab + PART_COLS - 1) / PART_COLS);
    *launches += 3;
    // 8 tokens per CTA against 32: 256 tokens of 128256 4.6 instead of 8.6 us, 512 of
    // 50257 3.1 instead of 4.2, 2048 of 20000 6.7 instead of 3.9
    const int per = L.tokens <= 1024 ? 8 : 32;
    return launch_dependent(per == 8 ? head_join_kernel<8> : head_join_kernel<32>,
                            dim3(static_cast<unsigned>((L.tokens + per - 1) / per)), 32 * kJoinWarps, 0, stream, G.part,
                            nparts, l.tpad, G.tlogit, reinterpret_cast<const int*>(ws + l.index),
                            static_cast<int>(L.tokens), L.loss, L.lse);
}

cudaError_t launch_head_loss_backward(const HeadLoss& L, cudaStream_t stream, int* launches, const char** why) {
    if (!encoder()) {
        *why = "cuTensorMapEncodeTiled unavailable";
        return cudaErrorNotSupported;
    }
    const Layout l = layout(L.tokens, L.vocab, L.dim, true);
    char* ws = static_cast<char*>(L.workspace);
    const long long pitch = l.piece_tiles * BN;
    HeadGemm P = gemm_args(L, l), D = P;
    P.lse = reinterpret_cast<const float*>(ws + l.lse);
    P.dloss = reinterpret_cast<const float*>(ws + l.dloss);
    P.rest = reinterpret_cast<float*>(ws + l.rest);
    D.scale = reinterpret_cast<const float*>(ws + l.scale);
    const bool ok = encode(&P.a, BOX_K, ws + l.rows, false, L.dim, l.tpad, L.dim) &&
                    encode(&P.all, BOX_K, L.hidden, false, L.dim, L.tokens, L.ldh) &&
                    encode(&D.all, BOX_MN, L.hidden, false, L.dim, L.tokens, L.ldh) &&
                    encode(&P.b, BOX_K, L.weight, false, L.dim, L.vocab, L.dim) &&
                    encode(&P.o, BOX_STORE, ws + l.p, false, pitch, l.tpad, pitch) &&
                    encode(&D.a, BOX_K, ws + l.p, false, pitch, l.tpad, pitch) &&
                    encode(&D.b, BOX_MN, L.weight, false, L.dim, L.vocab, L.dim) &&
                    encode(&D.a2, BOX_MN, ws + l.p, false, pitch, l.tpad, pitch) &&
                    encode(&D.b2, BOX_MN, ws + l.rows, false, L.dim, l.tpad, L.dim) &&
                    encode(&D.o, BOX_STORE, ws + l.slots, true, L.dim, l.tpad, L.dim, l.splits, l.tpad * L.dim) &&
                    (!L.dweight || encode(&D.o2, BOX_STORE, L.dweight, false, L.dim, L.vocab, L.dim));
    if (!ok) {
        *why = "tensor map encoding failed";
        return cudaErrorInvalidValue;
    }
    cudaError_t e = launch_rows(L, l, true, stream);
    if (e != cudaSuccess) return e;
    ++*launches;
    unsigned* tickets = reinterpret_cast<unsigned*>(ws + l.tickets);
    const long long R = l.tpad / BMP, nd = (L.dim + BN - 1) / BN;
    for (long long k = 0; k < l.pieces; ++k) {
        const long long first = k * l.piece_tiles, tiles = std::min(l.piece_tiles, l.vtiles - first);
        P.v0 = D.v0 = static_cast<int>(first * BN);
        P.vtiles = D.vtiles = static_cast<int>(tiles);
        P.ticket = tickets + 2 * k;
        e = launch_gemm<PROB>(P, R * tiles, stream);
        if (e != cudaSuccess) return e;
        const long long kv = tiles * (BN / BK);
        D.ticket = tickets + 2 * k + 1;
        D.split_slices = l.split_slices;
        D.splits = L.dhidden ? static_cast<int>((kv + l.split_slices - 1) / l.split_slices) : 0;
        D.dw_tiles = L.dweight ? static_cast<int>(tiles) : 0;
        D.add = k > 0;
        e = launch_gemm<GRAD>(D, (R * D.splits + D.dw_tiles) * nd, stream);
        if (e != cudaSuccess) return e;
        *launches += 2;
    }
    if (!L.dhidden) return cudaSuccess;
    ++*launches;
    // one slot per token wants many CTAs on an SM (40 registers), many slots want
    // loads in flight (200 tokens, 30000 x 1000: 6 instead of 13 us; 8192 tokens of
    // one slot of 768: 18 instead of 30 us)
    return launch_dependent(l.splits < 4 ? head_dhidden_kernel<1> : head_dhidden_kernel<8>, dim3(static_cast<unsigned>(L.tokens)), 128, 0, stream,
                            reinterpret_cast<const float*>(ws + l.slots), l.splits, l.tpad * L.dim,
                            reinterpret_cast<const int*>(ws + l.index), reinterpret_cast<const int*>(ws + l.target),
                            P.rest, D.scale, static_cast<const __nv_bfloat16*>(L.weight), static_cast<int>(L.dim),
                            static_cast<__nv_bfloat16*>(L.dhidden));
}

}  // namespace muon
