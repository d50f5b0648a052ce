// attn_tree.cuh - attention of a draft tree's rows over the resident pool
// slots and the tree's own keys and values, on the 5th-generation tensor cores.
//
// OasisKV: Scaling In-Decode KV Cache Beyond HBM with Lookahead Sparse
// Prefetching, Figure 7 (right): the verification query and the drafts are
// attended in one pass over the resident working set.  Here the drafts form a
// tree: a row also sees the nodes that its visibility word names.
//
// Shapes.  A (sequence, KV head) unit has T*G query rows, up to 64 G.  Rows are
// the MMA's M dimension, 128 at a time (as many whole nodes as fit), and a KV
// tile is 8 pool slots (128 tokens) or, as a unit's first tile, the tree itself:
//   S [128 rows x 128 tokens]  = Q [128 x 128] . K_tile^T       8 MMAs, both in shared memory
//   O [128 rows x 128 dims]   += P [128 x 128] . V_tile         one MMA per occupied slot,
//                                                              P bf16 in TMEM over S
// A softmax thread owns a row: no shuffles, no votes across threads but the
// (rare) one that rescales O.  Rows do not meet in any sum, so the padding rows
// of the last 128 hold whatever they hold.
//
// Two softmax warpgroups keep the tensor core and the exponentials busy at
// once: step s of a segment belongs to warpgroup s & 1.  Its 128 tokens go in two
// halves: while the second half's weights are made, the first half's product and
// S of the first half of step s + 2 run.  (S of 64 tokens takes 51 cycles an MMA
// where 128 take 67, as the query rows are read from shared memory twice as
// often; but whole steps left each warpgroup waiting for its own two MMAs, and the
// 16 x 64-node case at 104 us instead of 87.  Handing the exponentials from one
// warpgroup to the other by turns changed nothing.)  With two row tiles (an item's
// 256 rows) steps 2i and 2i + 1 are the two row tiles on KV tile i, so a KV tile
// is read once for both; with one row tile (128 rows or fewer) they are KV tiles
// 2i and 2i + 1, each warpgroup with its own O, joined at the end.
//
// Rounding.  Softmax weights are rounded to bf16 (2^-8 each, independent of one
// another) because the value rows are bf16 and the MMA takes one type for both;
// the sum of the weights is of the unrounded ones in fp32.  The output is
// rounded to bf16 anyway, by as much again: 0.0023 from fp64 (relative, 16 x 8
// nodes) where fp32 weights give 0.0017.  A remainder beside each weight in TMEM and
// a second product with it give 0.0017 too, and take 36.7 us instead of 33.6 there,
// 97 instead of 84 with 16 x 64 nodes.
//
// Work split.  The KV tiles of all items stand in one row (a unit's row tiles far
// apart, so that they are worked on at the same time and DRAM gives the unit's
// tiles once), and each CTA takes an equal stretch of it (`per` tiles).  Where whole
// items make a stretch at most four tiles longer it is rounded up to them, which can
// leave CTAs without work (128 of 132 have some in both cases of 16 sequences below;
// 16 SMs are left to the gather).  An item that lies in one stretch is written directly;
// the parts of others go to the workspace, normalised, with their log2-sum-exp, and
// a second kernel joins them, a warp a row.  (Joined by the item's last CTA
// instead, 28 rows of 9 parts took 20 us: one SM for each item, all its loads
// waiting for one another, and code that no SM had fetched yet.)
//
// Measured on B200 (back to back, other inputs each time): 16 sequences x 8 nodes,
// 64 / 8 heads, 128 slots a KV head, a tenth of them free: 33.5 us (the 142 MB that
// are read at 5.8 TB/s while the tiles stream, 46,000 of 58,000 cycles; the rest is
// the list, the first tile and the last epilogue); 16 x 64 nodes: 84 us, 0.84
// PFLOP/s (the tensor pipe active in 34 % of all SMs' cycles of a cold launch of 96 us,
// the softmax chain the limit: ~1,500 cycles a half tile for both warpgroups; 154 MB
// read from DRAM, what there is to read); one sequence x 7 nodes, 32 / 8 heads: 16.7 us
// (8.5 us of attention by 68 CTAs, then the join).  KV tiles are read evict-first:
// 33.6 us where the default takes 35.3 (16 x 8) and 84.5 where it takes 85.0 (16 x 64);
// one sequence's 8 MB, which L2 can hold from call to call, 16.6 where it takes 16.0.
//
// Roles (12 warps, mbarriers for every hand-off, every wait bounded):
//   warps 0-3, 4-7  softmax of the even / odd steps and the epilogue
//   warp 8          loader: lane 0 K tiles, lane 1 V tiles, lane 2 query rows
//   warps 9, 10     issue the MMAs of the even / odd steps (9 holds the TMEM allocation)
//   warp 11         lists the tiles of a segment that hold a valid token, and cleans value rows
//                   that no row may meet (tokens past the context in a partly filled slot,
//                   padding nodes): they read as zeros before they are used, since zero times a
//                   stale NaN is NaN; a node's infinite or NaN values too, and the epilogue adds
//                   them to the rows that see the node
#pragma once

#include "attn.cuh"
#include "common.cuh"
#include "tree.cuh"

namespace oasis {

constexpr int kTaThreads = 32 * 12;
constexpr int kTaLoader = 8, kTaMma = 9, kTaLister = 11;            // (9 and 10 issue)
constexpr int kTaRows = 128;                                       // the MMA's M
constexpr int kTaMaxTiles = 1024 / kAttnTileSlots + 1;             // of a unit: budget_blocks <= 1024, and the tree's
constexpr int kTaInfoInts = 16 + 4 * kTaMaxTiles;                  // header, then 4 ints a tile
constexpr int kTaOffK = 0;                                         // K ring, 2 stages of 32 KiB
constexpr int kTaOffV = kTaOffK + 2 * kAttnStageBytes;             // V ring
constexpr int kTaOffQ = kTaOffV + 2 * kAttnStageBytes;             // 2 row tiles of [2 halves][128 rows][128 B]
constexpr int kTaQTile = 2 * kAttnHalf;
constexpr int kTaOffInfo = kTaOffQ + 2 * kTaQTile;
constexpr int kTaOffBar = kTaOffInfo + 2 * kTaInfoInts * 4;
constexpr int kTaNumBars = 32;
constexpr int kTaOffMl = kTaOffBar + kTaNumBars * 8;               // [2][128] max, [2][128] sum
constexpr int kTaOffMisc = kTaOffMl + 4 * 128 * 4;                 // 16 ints
constexpr int kTaStagePitch = 80;                                  // 64 B of a row, and 16 B against bank conflicts
constexpr int kTaOffStage = kTaOffMisc + 64;                       // [8 warps][32 rows]
constexpr int kTaSmem = kTaOffStage + 8 * 32 * kTaStagePitch + 1024;   // + alignment slack
static_assert(kTaSmem <= 227 * 1024, "tree attention shared memory");
static_assert(kTaOffBar % 8 == 0 && kTaOffMl % 16 == 0 && kTaOffStage % 16 == 0, "alignment");

// mbarriers
constexpr int kTbKFull = 0, kTbKEmpty = 2, kTbVFull = 4, kTbVEmpty = 6, kTbVClean = 8;   // [2] by ring stage
constexpr int kTbSFull = 10, kTbPFull = 14, kTbPvDone = 18, kTbPvA = 20;                  // by warpgroup (and half: [2][2])
constexpr int kTbLFull = 22, kTbLFree = 24;                                              // [2] by list buffer
constexpr int kTbQFull = 26, kTbQFree = 27, kTbOFree = 28, kTbFinal = 29;                // (kTbFinal: [2] by issuer)
constexpr int kTaLFreeCount = 8 + 3 + 2 + 1;                       // softmax warps, loader lanes, issuers, cleaner
constexpr uint32_t kTnVote = 1, kTnSync = 2;                       // named barriers of the softmax warps

// Every kTaPolyEvery-th pair of weights is made on the multiply-add pipes.
constexpr int kTaPolyEvery = 4;

// TMEM columns: S (and P over it) of the two warpgroups, then their O
constexpr uint32_t kTcS = 0, kTcO = 256;

// Header of a segment's list.
enum { kTiN = 0, kTiItem, kTiDirect, kTiSlot, kTiSeenLo, kTiSeenHi, kTiWildLo, kTiWildHi };
// Flags of a tile (4th int).
constexpr int kTfMask = 1, kTfClean = 2;

struct TreeAttnArgs {
    const int32_t* slot_table;
    const int32_t* ctx_len;
    const uint64_t* mask;        // [B][T]
    const uint16_t* v_tree;      // [B][Hkv][T][128]
    __nv_bfloat16* out;          // [B][T][Hq][128]
    float* lse;                  // [B][T][Hq]
    float* ws_o;                 // [2 CTAs][256][128]
    float* ws_lse;               // [2 CTAs][256]
    float scale_log2;
    int T;
    int nt;                      // nodes a row tile
    int units;                   // an item: one of a unit's pairs of row tiles, unit fastest
    int tpu;                     // KV tiles a unit, the tree's among them
    int per;                     // KV tiles a CTA
    int total;                   // KV tiles in all
};

// Whether a pair of bf16 holds an infinity or NaN in its low / high half.
__device__ __forceinline__ bool bf16_lo_wild(uint32_t w) { return (w & 0x00007F80u) == 0x00007F80u; }
__device__ __forceinline__ bool bf16_hi_wild(uint32_t w) { return (w & 0x7F800000u) == 0x7F800000u; }

// D[tmem] += A[tmem] . B[smem descriptor]
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Largest of three, NaN if one of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// 2^x of two values on the multiply-add pipes, for x <= 32 (the multi-function
// unit makes 4 a cycle for each of an SM's quarters, half of what the softmax
// could use).  x = n + f with n the nearest whole number, |f| <= 1/2, found by
// adding and taking off 1.5 * 2^23; 2^f by a polynomial of degree 4 with p(0) = 1
// fitted for the smallest largest relative error (2.9e-6, mean 3e-7); n goes to
// the exponent field.  x below -127 gives 0: -127 itself does, exactly.
__device__ __forceinline__ uint64_t exp2_poly_f32x2(uint64_t x) {
    const uint64_t magic = f32x2(12582912.f, 12582912.f);
    x = f32x2(fmaxf(f32x2_lo(x), -127.f), fmaxf(f32x2_hi(x), -127.f));
    const uint64_t t = add_f32x2(x, magic);
    const uint64_t n = add_f32x2(t, f32x2(-12582912.f, -12582912.f));
    const uint64_t f = fma_f32x2(n, f32x2(-1.f, -1.f), x);
    uint64_t p = fma_f32x2(f, f32x2(0.009582853f, 0.009582853f), f32x2(0.055906426f, 0.055906426f));
    p = fma_f32x2(p, f, f32x2(0.24024099f, 0.24024099f));
    p = fma_f32x2(p, f, f32x2(0.6931242f, 0.6931242f));
    p = fma_f32x2(p, f, f32x2(1.f, 1.f));
    const uint32_t lo = static_cast<uint32_t>(p) + (static_cast<uint32_t>(t) << 23);
    const uint32_t hi = static_cast<uint32_t>(p >> 32) + (static_cast<uint32_t>(t >> 32) << 23);
    return f32x2(__uint_as_float(lo), __uint_as_float(hi));
}

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}\n" : "=r"(r));
    return r != 0;
}

// As cta_wait, with the barrier looked at before the abort flag.
__device__ __forceinline__ bool ta_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    return mbar_try_wait(bar, parity) || cta_wait(bar, parity, abort_flag);
}

// The step sequence of a segment: with two row tiles a KV tile serves two steps.
struct TaSteps {
    int two;                     // 1: two row tiles
    int n;                       // KV tiles
    __device__ __forceinline__ int count() const { return n << two; }
    __device__ __forceinline__ int tile(int s) const { return s >> two; }
    __device__ __forceinline__ int count_of(int wg) const { return (count() - wg + 1) >> 1; }
};

__global__ void __launch_bounds__(kTaThreads, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_tk,
                     const __grid_constant__ CUtensorMap tm_tv, const Dims d, const TreeAttnArgs a) {
    const float kNegInf = -__int_as_float(0x7f800000);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sK = smem + kTaOffK;
    uint8_t* sV = smem + kTaOffV;
    uint8_t* sQ = smem + kTaOffQ;
    int* s_info = reinterpret_cast<int*>(smem + kTaOffInfo);
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + kTaOffBar);
    float* s_m = reinterpret_cast<float*>(smem + kTaOffMl);
    float* s_l = s_m + 2 * 128;
    int* misc = reinterpret_cast<int*>(smem + kTaOffMisc);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(misc);
    volatile int* s_abort = misc + 1;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = d.G(), K = d.K;
    const int t16 = (a.T + kBlockTokens - 1) / kBlockTokens * kBlockTokens;

    // Lists the next segment of this CTA's stretch into list buffer p & 1 (the
    // lister's lanes, a tile each).
    long long at = static_cast<long long>(blockIdx.x) * a.per;
    const long long end = min(at + a.per, static_cast<long long>(a.total));
    auto list_segment = [&](int p) {
        int* info = s_info + (p & 1) * kTaInfoInts;
        if (__any_sync(0xFFFFFFFFu, at >= end || *s_abort)) {
            if (lane == 0) info[kTiN] = -1;
            __syncwarp();
            return;
        }
        const int item = static_cast<int>(at) / a.tpu;
        const int lo = static_cast<int>(at) - item * a.tpu;
        const int hi = static_cast<int>(min(static_cast<long long>(a.tpu), lo + (end - at)));
        at += hi - lo;
        const int pr = item / a.units, u = item - pr * a.units;
        const int b = u / d.Hkv;
        const int first = max(lo, 1) - 1, pool_hi = hi - 1;       // pool tiles: the unit's first tile is the tree's
        int blk[kAttnTileSlots];
        auto load = [&](int tile) {
            const int s0 = kAttnTileSlots * tile;
#pragma unroll
            for (int jj = 0; jj < kAttnTileSlots; ++jj)
                blk[jj] = tile < pool_hi && s0 + jj < K ? a.slot_table[static_cast<long long>(u) * K + s0 + jj] : -1;
        };
        load(first + lane);
        const int ctx = a.ctx_len[b];
        // nodes that some row of the item sees
        const uint64_t real = a.T >= 64 ? ~0ull : (1ull << a.T) - 1;
        uint64_t seen = 0;
        for (int j = pr * 2 * a.nt + lane; j < min(a.T, (pr + 1) * 2 * a.nt); j += 32)
            seen |= a.mask[static_cast<long long>(b) * a.T + j];
        seen &= real;
        seen = __reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(seen)) |
               (static_cast<uint64_t>(__reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(seen >> 32))) << 32);
        int n = 0;
        if (lo == 0 && seen != 0) {
            if (lane == 0) {
                uint32_t nv = 0;
#pragma unroll
                for (int jj = 0; jj < 4; ++jj)
                    nv |= static_cast<uint32_t>(min(kBlockTokens, max(0, a.T - kBlockTokens * jj))) << (8 * jj);
                info[16] = -1;
                info[17] = static_cast<int>(nv);
                info[18] = 0;
                info[19] = kTfMask | kTfClean;
            }
            n = 1;
        }
        for (int t0 = first; t0 < pool_hi && seen != 0; t0 += 32) {
            if (t0 > first) load(t0 + lane);
            uint32_t nvlo = 0u, nvhi = 0u;
            bool any = false, full = true, clean = false;
#pragma unroll
            for (int jj = 0; jj < kAttnTileSlots; ++jj) {
                int bk = blk[jj];
                if (bk < -1 || bk >= d.N) {
                    raise_dev_error(OASIS_DEVERR_ID_RANGE);
                    bk = -1;
                }
                const int nv = bk >= 0 ? min(kBlockTokens, max(0, ctx - bk * kBlockTokens)) : 0;
                if (jj < 4)
                    nvlo |= static_cast<uint32_t>(nv) << (8 * jj);
                else
                    nvhi |= static_cast<uint32_t>(nv) << (8 * (jj - 4));
                any |= nv > 0;
                full &= nv == kBlockTokens;
                clean |= nv > 0 && nv < kBlockTokens;
            }
            const unsigned m = __ballot_sync(0xFFFFFFFFu, any);
            if (any) {
                int* e = info + 16 + 4 * (n + __popc(m & ((1u << lane) - 1u)));
                e[0] = kAttnTileSlots * (t0 + lane);
                e[1] = static_cast<int>(nvlo);
                e[2] = static_cast<int>(nvhi);
                e[3] = (full ? 0 : kTfMask) | (clean ? kTfClean : 0);
            }
            n += __popc(m);
        }
        if (lane == 0) {
            const int base = item * a.tpu;
            const int c0 = base / a.per, c1 = (base + a.tpu - 1) / a.per;
            info[kTiN] = n;
            info[kTiItem] = item;
            info[kTiDirect] = c0 == c1;
            // a CTA's first segment goes to its first place in the workspace, its last to its second
            info[kTiSlot] = 2 * static_cast<int>(blockIdx.x) + (p == 0 ? 0 : 1);
            info[kTiSeenLo] = static_cast<int>(static_cast<uint32_t>(seen));
            info[kTiSeenHi] = static_cast<int>(static_cast<uint32_t>(seen >> 32));
            info[kTiWildLo] = info[kTiWildHi] = 0;
        }
        __syncwarp();
    };

    // ---------------------------------------------------------- set-up
    // (the first segment is listed meanwhile: its loads are the longest wait of the start)
    if (tid == 0) {
        for (int i = 0; i < kTaNumBars; ++i) {
            int cnt = 1;
            if (i >= kTbPFull && i < kTbPFull + 4) cnt = 4;
            if (i == kTbOFree) cnt = 8;
            // a tile, and the query rows, are done with when both issuers say so
            if (i == kTbKEmpty || i == kTbKEmpty + 1 || i == kTbVEmpty || i == kTbVEmpty + 1 || i == kTbQFree) cnt = 2;
            if (i == kTbLFree || i == kTbLFree + 1) cnt = kTaLFreeCount;
            mbar_init(&bar[i], cnt);
        }
        fence_mbar_init();
    }
    if (warp == kTaLister) {
        if (lane == 0) *s_abort = 0;
        __syncwarp();
        list_segment(0);
    }
    if (warp == kTaLoader && lane == 0) {
        prefetch_tensormap(&tm_q);
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
        prefetch_tensormap(&tm_tk);
        prefetch_tensormap(&tm_tv);
    }
    if (warp == kTaMma) {
        tmem_alloc(s_tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *s_tmem;

    if (warp == kTaLister) {
        // ================================================ lister, cleaner
        // segment p + 1 is listed before segment p is cleaned
        int pos = 0;
        for (int p = 0;; ++p) {
            for (int q = p == 0 ? 0 : p + 1; q <= p + 1; ++q) {
                if (q >= 2) cta_wait(&bar[kTbLFree + (q & 1)], ((q >> 1) - 1) & 1, s_abort);
                __syncwarp();
                if (q > 0) list_segment(q);
                if (lane == 0) mbar_arrive(&bar[kTbLFull + (q & 1)]);
                if (q == 0 && s_info[kTiN] < 0) break;
            }
            const int pb = p & 1;
            int* info = s_info + pb * kTaInfoInts;
            const int n = info[kTiN];
            if (n < 0) break;
            const uint64_t seen = static_cast<uint32_t>(info[kTiSeenLo]) |
                                  (static_cast<uint64_t>(static_cast<uint32_t>(info[kTiSeenHi])) << 32);
            for (int i = 0; i < n; ++i, ++pos) {
                const int st = pos & 1;
                const int* e = info + 16 + 4 * i;
                ta_wait(&bar[kTbVFull + st], (pos >> 1) & 1, s_abort);
                __syncwarp();
                if (e[3] & kTfClean) {
                    // 16 lanes a row (16 B each, both 64-channel halves), a slot's 16 rows at a time
                    const bool tree = e[0] < 0;
                    const uint64_t nvs = static_cast<uint32_t>(e[1]) | (static_cast<uint64_t>(static_cast<uint32_t>(e[2])) << 32);
                    const int part = lane & 15;
                    for (int slot = 0; slot < kAttnTileSlots; ++slot) {
                        const int nv = static_cast<int>(nvs >> (8 * slot)) & 0xFF;
                        if (nv == 0 || (nv == kBlockTokens && !tree)) continue;   // never multiplied in, or sound
                        uint8_t* base = sV + st * kAttnStageBytes + (part >> 3) * kAttnHalf + (part & 7) * 16 +
                                        (16 * slot + (lane >> 4)) * 128;
                        uint4 v[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[k] = *reinterpret_cast<const uint4*>(base + 256 * k);
                        uint32_t rows = 0;                        // this lane's rows of the slot with a wild value
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int t = 2 * k + (lane >> 4);
                            const bool zero = t >= nv || (tree && !(seen >> (16 * (slot & 3) + t) & 1));
                            uint32_t vv[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
                            bool wild = false;
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                const bool wl = bf16_lo_wild(vv[c]), wh = bf16_hi_wild(vv[c]);
                                wild |= wl | wh;
                                vv[c] &= (wl ? 0u : 0xFFFFu) | (wh ? 0u : 0xFFFF0000u);
                            }
                            if (zero) {
                                *reinterpret_cast<uint4*>(base + 256 * k) = make_uint4(0u, 0u, 0u, 0u);
                            } else if (tree && wild) {
                                *reinterpret_cast<uint4*>(base + 256 * k) = make_uint4(vv[0], vv[1], vv[2], vv[3]);
                                rows |= 1u << t;
                            }
                        }
                        if (rows) atomicOr(reinterpret_cast<unsigned int*>(info + kTiWildLo) + (slot >> 1 & 1), rows << (16 * (slot & 1)));
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[kTbVClean + st]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[kTbLFree + pb]);
            if (s_info[(pb ^ 1) * kTaInfoInts + kTiN] < 0) break;
            __syncwarp();
        }
        // The last tile is under way: the joining kernel may take its place on the SMs and wait there for this one's
        // end.  (Not earlier: its CTAs would fill the SMs left to a gather, which then ran behind the attention.)
        asm volatile("griddepcontrol.launch_dependents;");
    } else if (warp == kTaLoader) {
        // ======================================================= loader
        if (lane < 2) {
            const bool is_k = lane == 0;
            const CUtensorMap* tm = is_k ? &tm_k : &tm_v;
            const CUtensorMap* tt = is_k ? &tm_tk : &tm_tv;
            uint8_t* ring = is_k ? sK : sV;
            const int bar_full = is_k ? kTbKFull : kTbVFull, bar_empty = is_k ? kTbKEmpty : kTbVEmpty;
            const uint64_t pol = l2_policy_evict_first();
            int pos = 0;
            int last[2] = {-1, -1};
            for (int p = 0;; ++p) {
                const int pb = p & 1;
                if (!cta_wait(&bar[kTbLFull + pb], (p >> 1) & 1, s_abort)) break;
                const int* info = s_info + pb * kTaInfoInts;
                const int n = info[kTiN];
                if (n < 0) break;
                const int u = info[kTiItem] % a.units;
                for (int i = 0; i < n; ++i, ++pos) {
                    const int st = pos & 1;
                    const int first = info[16 + 4 * i];
                    if (pos >= 2) cta_wait(&bar[bar_empty + st], ((pos >> 1) - 1) & 1, s_abort);
                    mbar_arrive_expect_tx(&bar[bar_full + st], first >= 0 ? kAttnStageBytes : t16 * kRowBytes);
                    if (!*s_abort) {
                        last[st] = pos;
                        uint8_t* dst = ring + st * kAttnStageBytes;
                        const int z = first >= 0 ? u * K + first : u;
                        const CUtensorMap* m = first >= 0 ? tm : tt;
                        tma_load_3d(dst, m, &bar[bar_full + st], 0, 0, z, pol);
                        tma_load_3d(dst + kAttnHalf, m, &bar[bar_full + st], 64, 0, z, pol);
                    }
                }
                mbar_arrive(&bar[kTbLFree + pb]);
            }
            // no copy may still be writing this CTA's shared memory when it exits
            for (int st = 0; st < 2; ++st)
                if (last[st] >= 0) mbar_wait(&bar[bar_full + st], static_cast<uint32_t>((last[st] >> 1) & 1));
        } else if (lane == 2) {
            const uint64_t pol = l2_policy_evict_first();
            int nz = 0, loaded = -1;
            for (int p = 0;; ++p) {
                const int pb = p & 1;
                if (!cta_wait(&bar[kTbLFull + pb], (p >> 1) & 1, s_abort)) break;
                const int* info = s_info + pb * kTaInfoInts;
                const int n = info[kTiN];
                if (n < 0) break;
                if (n > 0) {
                    const int item = info[kTiItem];
                    const int pr = item / a.units, u = item - pr * a.units;
                    const int b = u / d.Hkv, h = u - b * d.Hkv;
                    const int tiles = (2 * pr + 1) * a.nt < a.T ? 2 : 1;
                    if (nz > 0) cta_wait(&bar[kTbQFree], (nz - 1) & 1, s_abort);
                    mbar_arrive_expect_tx(&bar[kTbQFull], static_cast<uint32_t>(tiles * a.nt * G) * kRowBytes);
                    if (!*s_abort) {
                        loaded = nz;
                        for (int t = 0; t < tiles; ++t) {
                            const int node = b * a.T + (2 * pr + t) * a.nt;
                            tma_load_3d(sQ + t * kTaQTile, &tm_q, &bar[kTbQFull], 0, h * G, node, pol);
                            tma_load_3d(sQ + t * kTaQTile + kAttnHalf, &tm_q, &bar[kTbQFull], 64, h * G, node, pol);
                        }
                    }
                    ++nz;
                }
                mbar_arrive(&bar[kTbLFree + pb]);
            }
            if (loaded >= 0) mbar_wait(&bar[kTbQFull], static_cast<uint32_t>(loaded & 1));
        }
        __syncwarp();
    } else if (warp == kTaMma || warp == kTaMma + 1) {
        // ================================================= MMA issuers
        // One a softmax warpgroup: whatever can be waited for beforehand is, so that when the warpgroup's P is
        // there its product and the next S go out at once.  The warps stay converged and one elected lane
        // issues: descriptors and addresses then live in uniform registers (a single-lane branch took 150
        // cycles an MMA to issue, over twice the MMA's own time; one warp for both warpgroups 2,250 cycles a
        // step).
        constexpr uint32_t idesc_s = umma_idesc_bf16_f32(kTaRows, kAttnTileTokens / 2);
        constexpr uint32_t idesc_o = umma_idesc_bf16_f32_bmn(kTaRows, kHeadDim);
        const int wg = warp - kTaMma;
        const uint64_t k_desc = umma_desc_sw128_lbo_sbo(smem_addr(sK), 16, 1024);
        const uint64_t v_desc = umma_desc_sw128_lbo_sbo(smem_addr(sV), kAttnHalf, 1024);
        const uint32_t t_s = tmem + kTcS + wg * 128, t_o = tmem + kTcO + wg * 128;
        int pos = 0, nz = 0, done = 0;                            // KV tiles, segments (with tiles) and own steps behind
        for (int p = 0;; ++p) {
            const int pb = p & 1;
            const bool got = ta_wait(&bar[kTbLFull + pb], (p >> 1) & 1, s_abort);
            const int* info = s_info + pb * kTaInfoInts;
            const int n = __shfl_sync(0xFFFFFFFFu, got ? info[kTiN] : -1, 0);
            if (n < 0) break;
            if (n > 0) {
                const int pr = __shfl_sync(0xFFFFFFFFu, info[kTiItem], 0) / a.units;
                const TaSteps sq{(2 * pr + 1) * a.nt < a.T ? 1 : 0, n};
                const int mine = sq.count_of(wg);
                const uint64_t q_desc =
                    umma_desc_sw128_lbo_sbo(smem_addr(sQ) + (sq.two ? wg : 0) * kTaQTile, 16, 1024);
                auto wait_k = [&](int s) {
                    const int kt = pos + sq.tile(s);
                    return ta_wait(&bar[kTbKFull + (kt & 1)], (kt >> 1) & 1, s_abort);
                };
                // S of 64 tokens of step s (by the elected lane)
                auto issue_s = [&](int s, int half) {
                    const uint64_t ka = k_desc + (((pos + sq.tile(s)) & 1) * kAttnStageBytes + half * (kAttnHalf / 2) >> 4);
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        const int off = ((ks >> 2) * kAttnHalf + (ks & 3) * 32) >> 4;
                        umma_bf16(t_s + 64 * half, q_desc + off, ka + off, idesc_s, ks > 0 ? 1u : 0u);
                    }
                };
                // with one row tile a KV tile has one user, who says both words
                auto release = [&](uint64_t* b) {
                    umma_commit(b);
                    if (!sq.two) umma_commit(b);
                };
                ta_wait(&bar[kTbQFull], nz & 1, s_abort);
                if (mine > 0) {
                    const bool ok = __shfl_sync(0xFFFFFFFFu, wait_k(wg), 0);
                    tc_fence_after_sync();
                    if (elect_one()) {
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            if (ok) issue_s(wg, half);
                            umma_commit(&bar[kTbSFull + 2 * wg + half]);
                        }
                        release(&bar[kTbKEmpty + ((pos + sq.tile(wg)) & 1)]);
                    }
                    __syncwarp();
                }
                if (mine < 2 && elect_one()) umma_commit(&bar[kTbQFree]);
                // The last segment's O is read.  (Only where this issuer writes O: a segment of one tile and one row
                // tile ends without the second issuer, which could then come here a whole phase late, and a parity
                // that has come round again reads as not done.)
                if (nz > 0 && mine > 0) ta_wait(&bar[kTbOFree], (nz - 1) & 1, s_abort);
                uint32_t acc = 0u;                                // the first product overwrites O
                for (int k = 0; k < mine; ++k, ++done) {
                    const int s = 2 * k + wg, i = sq.tile(s), vt = pos + i, st = vt & 1;
                    const bool more = k + 1 < mine;
                    bool ok = ta_wait(&bar[kTbVClean + st], (vt >> 1) & 1, s_abort);
                    if (more) ok = wait_k(s + 2) && ok;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t nv = __shfl_sync(0xFFFFFFFFu, static_cast<uint32_t>(info[16 + 4 * i + 1 + half]), 0);
                        ok = ta_wait(&bar[kTbPFull + 2 * wg + half], done & 1, s_abort) && ok;
                        ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
                        tc_fence_after_sync();
                        if (elect_one()) {
                            const uint64_t va = v_desc + (st * kAttnStageBytes + half * 4 * kBlockTokens * 128 >> 4);
                            const uint32_t pa = t_s + 64 * half;
                            constexpr int kSlot = kBlockTokens * 128 >> 4;
                            if (ok && !((nv - 0x01010101u) & ~nv & 0x80808080u)) {   // no byte is 0: every slot counts
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    umma_bf16_ts(t_o, pa + 8 * kk, va + kk * kSlot, idesc_o, kk > 0 ? 1u : acc);
                            } else if (ok) {
                                uint32_t on = acc;
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk) {
                                    if ((nv >> (8 * kk) & 0xFFu) == 0) continue;     // free: no product
                                    umma_bf16_ts(t_o, pa + 8 * kk, va + kk * kSlot, idesc_o, on);
                                    on = 1u;
                                }
                            }
                            if (half == 0) umma_commit(&bar[kTbPvA + wg]);
                            if (more) {
                                if (ok) issue_s(s + 2, half);     // behind the product that reads P over this S
                                umma_commit(&bar[kTbSFull + 2 * wg + half]);
                            }
                            if (half == 1) {
                                if (!more) umma_commit(&bar[kTbPvDone + wg]);
                                release(&bar[kTbVEmpty + st]);
                                if (more) release(&bar[kTbKEmpty + ((pos + sq.tile(s + 2)) & 1)]);
                                if (k + 2 == mine) umma_commit(&bar[kTbQFree]);
                            }
                        }
                        acc |= nv != 0 ? 1u : 0u;
                        __syncwarp();
                    }
                }
                pos += n;
                ++nz;
            }
            if (elect_one()) mbar_arrive(&bar[kTbLFree + pb]);
            __syncwarp();
        }
        if (elect_one()) {
            umma_commit(&bar[kTbFinal + wg]);
            mbar_wait(&bar[kTbFinal + wg], 0);
        }
        __syncwarp();
    } else {
        // ============================================ softmax and epilogue (row / thread)
        const int wg = warp >> 2, q = warp & 3;
        const int r = 32 * q + lane;                              // row of the row tile
        const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16;
        const uint32_t t_s = tmem + lane_base + kTcS + wg * 128;
        const uint32_t t_o = tmem + lane_base + kTcO;
        int done = 0;                                             // own steps so far
        int segs[2] = {0, 0};                                     // segments in which each warpgroup had a step
        for (int p = 0;; ++p) {
            const int pb = p & 1;
            const bool got = cta_wait(&bar[kTbLFull + pb], (p >> 1) & 1, s_abort);
            const int* info = s_info + pb * kTaInfoInts;
            const int n = got ? info[kTiN] : -1;
            if (named_bar_or(kTnVote, 256, n < 0 || *s_abort)) break;
            const int item = info[kTiItem];
            const int pr = item / a.units, u = item - pr * a.units;
            const int b = u / d.Hkv, h = u - b * d.Hkv;
            const TaSteps sq{(2 * pr + 1) * a.nt < a.T ? 1 : 0, n};
            const int my_tile = 2 * pr + (sq.two ? wg : 0);
            const int j = my_tile * a.nt + r / G;                 // node of this row
            const bool live0 = r < a.nt * G && j < a.T;
            const uint64_t real = a.T >= 64 ? ~0ull : (1ull << a.T) - 1;
            const uint64_t word = live0 ? a.mask[static_cast<long long>(b) * a.T + j] & real : 0ull;
            const bool live = word != 0;
            const bool warp_live = __any_sync(0xFFFFFFFFu, live);
            float m = kNegInf, l = 0.f;                           // running max (log2 units) and sum
            bool begun = false;
            const int mine = sq.count_of(wg);
            for (int k = 0; k < mine; ++k, ++done) {
                const int* e = info + 16 + 4 * sq.tile(2 * k + wg);
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    const uint32_t nv = static_cast<uint32_t>(e[1 + half]);
                    const uint32_t t_x = t_s + 64 * half;
                    ta_wait(&bar[kTbSFull + 2 * wg + half], done & 1, s_abort);
                    __syncwarp();
                    tc_fence_after_sync();
                    if (warp_live && nv != 0) {
                        uint32_t x[2][32];
#pragma unroll
                        for (int c = 0; c < 2; ++c) tmem_ld_32x32b_x32(t_x + 32 * c, x[c]);
                        tmem_ld_wait();
                        if (e[3] & kTfMask) {
                            if (e[0] < 0) {
#pragma unroll
                                for (int c = 0; c < 2; ++c) {
                                    const uint32_t w = static_cast<uint32_t>(word >> (32 * c));
#pragma unroll
                                    for (int i = 0; i < 32; ++i)
                                        if (!(w >> i & 1)) x[c][i] = 0xFF800000u;
                                }
                            } else {
#pragma unroll
                                for (int c = 0; c < 2; ++c) {
                                    const int n0 = nv >> (16 * c) & 0xFF, n1 = nv >> (16 * c + 8) & 0xFF;
#pragma unroll
                                    for (int i = 0; i < 32; ++i)
                                        if ((i & 15) >= (i < 16 ? n0 : n1)) x[c][i] = 0xFF800000u;
                                }
                            }
                        }
                        float mx[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint32_t* y = x[c >> 1] + 16 * (c & 1);
                            mx[c] = __uint_as_float(y[0]);
#pragma unroll
                            for (int i = 2; i < 16; i += 2)
                                mx[c] = max3_nan(mx[c], __uint_as_float(y[i - 1]), __uint_as_float(y[i]));
                        }
                        float top = max3_nan(max3_nan(mx[0], mx[1], __uint_as_float(x[0][15])),
                                             max3_nan(mx[2], mx[3], __uint_as_float(x[0][31])),
                                             max3_nan(__uint_as_float(x[1][15]), __uint_as_float(x[1][31]), kNegInf)) *
                                    a.scale_log2;
                        if (!(top < __int_as_float(0x7f800000))) top = __int_as_float(0x7fc00000);   // an infinite score: NaN
                        if (!begun) {
                            m = top;
                            begun = true;
                        } else {
                            // the running max moves only when a half tile exceeds it by more than 2^32
                            const bool up = live && !(top <= m + kAttnLazy);
                            if (__any_sync(0xFFFFFFFFu, up)) {
                                const float alpha = up ? attn_exp2(m - top) : 1.f;
                                if (up) m = top;
                                l *= alpha;
                                // the product before this one has landed in O
                                if (half == 0)
                                    cta_wait(&bar[kTbSFull + 2 * wg + 1], done & 1, s_abort);
                                else
                                    cta_wait(&bar[kTbPvA + wg], done & 1, s_abort);
                                __syncwarp();
                                tc_fence_after_sync();
#pragma unroll 1
                                for (int c = 0; c < 8; ++c) {
                                    uint32_t o[16];
                                    tmem_ld_x16(t_o + wg * 128 + 16 * c, o);
                                    tmem_ld_wait();
#pragma unroll
                                    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                                    tmem_st_x16(t_o + wg * 128 + 16 * c, o);
                                }
                                tmem_st_wait();
                            }
                        }
                        // (all scores so far -inf: their weights are 0, and the first finite one moves m)
                        const float off = m == kNegInf ? 0.f : -m;
                        const uint64_t sc2 = f32x2(a.scale_log2, a.scale_log2), m2 = f32x2(off, off);
                        uint64_t sum2 = 0ull;
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t w[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const uint64_t y =
                                    fma_f32x2(f32x2(__uint_as_float(x[c][2 * i]), __uint_as_float(x[c][2 * i + 1])), sc2, m2);
                                const uint64_t p2 = i % kTaPolyEvery == kTaPolyEvery - 1
                                                        ? exp2_poly_f32x2(y)
                                                        : f32x2(attn_exp2(f32x2_lo(y)), attn_exp2(f32x2_hi(y)));
                                sum2 = add_f32x2(sum2, p2);
                                w[i] = pack_bf16x2(f32x2_lo(p2), f32x2_hi(p2));
                            }
                            tmem_st_x16(t_x + 16 * c, w);
                        }
                        l += f32x2_lo(sum2) + f32x2_hi(sum2);
                        tmem_st_wait();
                    }
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar[kTbPFull + 2 * wg + half]);
                }
            }
            segs[0] += sq.count_of(0) > 0;
            segs[1] += sq.count_of(1) > 0;
            // ------------------------------------------------- epilogue
            if (!sq.two) {
                s_m[wg * 128 + r] = m;
                s_l[wg * 128 + r] = l;
                named_bar_sync(kTnSync, 256);
            }
            const int used = sq.two ? 1 : min(2, n);              // accumulators of a row
            float w0 = 0.f, w1 = 0.f, lse2 = kNegInf;
            if (live && n > 0) {
                if (sq.two) {
                    w0 = l == 0.f ? 0.f : 1.f / l;
                    lse2 = m + log2f(l);
                } else {
                    const float m0 = s_m[r], l0 = s_l[r];
                    const float m1 = used > 1 ? s_m[128 + r] : kNegInf, l1 = used > 1 ? s_l[128 + r] : 0.f;
                    const float M = fmaxf(m0, m1);
                    const float e0 = m0 == kNegInf ? 0.f : attn_exp2(m0 - M), e1 = m1 == kNegInf ? 0.f : attn_exp2(m1 - M);
                    const float L = l0 * e0 + l1 * e1;
                    w0 = L == 0.f ? 0.f : e0 / L;
                    w1 = L == 0.f ? 0.f : e1 / L;
                    lse2 = M + log2f(L);
                }
            }
            if (n > 0) {
                if (sq.two) {
                    cta_wait(&bar[kTbPvDone + wg], (segs[wg] - 1) & 1, s_abort);
                } else {
                    cta_wait(&bar[kTbPvDone], (segs[0] - 1) & 1, s_abort);
                    if (used > 1) cta_wait(&bar[kTbPvDone + 1], (segs[1] - 1) & 1, s_abort);
                }
                __syncwarp();
                tc_fence_after_sync();
            }
            const bool direct = info[kTiDirect] != 0;
            const uint64_t wild = static_cast<uint32_t>(info[kTiWildLo]) |
                                  (static_cast<uint64_t>(static_cast<uint32_t>(info[kTiWildHi])) << 32);
            // (at most 65535 units x 64 nodes x 64 heads: rows fit an int)
            const int prow = (sq.two ? wg : 0) * 128 + r;         // row of the item
            const int orow = !live0 ? -1
                             : direct ? (b * a.T + j) * d.Hq + h * G + r % G : info[kTiSlot] * 256 + prow;
            uint4* const stage = reinterpret_cast<uint4*>(smem + kTaOffStage + warp * 32 * kTaStagePitch);
            // 32 channels at a time; with one row tile the warpgroups take 64 channels each, with two a row tile each
            const int c_lo = sq.two ? 0 : 2 * wg, c_hi = sq.two ? 4 : 2 * wg + 2;
#pragma unroll 1
            for (int c = c_lo; c < c_hi; ++c) {
                float o[32];
                if (n > 0) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(t_o + (sq.two ? wg * 128 : 0) + 32 * c, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = live ? __uint_as_float(v[i]) * w0 : 0.f;
                    if (used > 1) {
                        tmem_ld_32x32b_x32(t_o + 128 + 32 * c, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] += live ? __uint_as_float(v[i]) * w1 : 0.f;
                    }
                    for (uint64_t ww = wild & word; ww != 0; ww &= ww - 1) {
                        const int node = __ffsll(static_cast<long long>(ww)) - 1;
                        const uint16_t* vr = a.v_tree + (static_cast<long long>(u) * a.T + node) * kHeadDim + 32 * c;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const uint32_t bits = static_cast<uint32_t>(vr[i]) << 16;
                            if (bf16_hi_wild(bits)) o[i] += __uint_as_float(bits);
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0.f;
                }
                if (!direct) {
                    float4* to = reinterpret_cast<float4*>(a.ws_o + static_cast<long long>(orow) * kHeadDim + 32 * c);
                    if (live0) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) to[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                    continue;
                }
                // through the warp's staging rows, so that four lanes write a row's 64 B
                uint4* const own = stage + lane * (kTaStagePitch / 16);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    own[i] = make_uint4(pack_bf16x2(o[8 * i], o[8 * i + 1]), pack_bf16x2(o[8 * i + 2], o[8 * i + 3]),
                                        pack_bf16x2(o[8 * i + 4], o[8 * i + 5]), pack_bf16x2(o[8 * i + 6], o[8 * i + 7]));
                __syncwarp();
                uint4 v[4];
                int row[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int from = 8 * i + (lane >> 2);
                    row[i] = __shfl_sync(0xFFFFFFFFu, orow, from);
                    v[i] = stage[from * (kTaStagePitch / 16) + (lane & 3)];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (row[i] >= 0)
                        *reinterpret_cast<uint4*>(a.out + static_cast<long long>(row[i]) * kHeadDim + 32 * c + 8 * (lane & 3)) = v[i];
                __syncwarp();
            }
            if (live0 && (sq.two || wg == 0)) {
                if (direct)
                    a.lse[orow] = lse2 * kLn2;
                else
                    a.ws_lse[orow] = lse2;
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0 && n > 0) mbar_arrive(&bar[kTbOFree]);
            if (lane == 0) mbar_arrive(&bar[kTbLFree + pb]);
        }
    }

    // ---------------------------------------------------------- teardown
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == kTaMma) tmem_dealloc(tmem, 512);
}

// Joins the parts of the rows of split items: out = sum_k 2^(lse_k - M) o_k /
// sum_k 2^(lse_k - M).  A warp a row, a part a lane for the weights, then a
// float4 a lane for the channels.  Launched once every CTA of the attention is at
// its last tile (its CTAs fit beside one of the attention's), so its launch is not
// waited for.
constexpr int kTjWarps = 4;
__global__ void __launch_bounds__(32 * kTjWarps) tree_join_kernel(const Dims d, const TreeAttnArgs a) {
    const float kNegInf = -__int_as_float(0x7f800000);
    asm volatile("griddepcontrol.wait;" ::: "memory");            // the attention has ended, its parts are written
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x * kTjWarps + (threadIdx.x >> 5);   // (b, node, head)
    if (row >= d.B * a.T * d.Hq) return;
    const int G = d.G();
    const int hq = row % d.Hq, bj = row / d.Hq;
    const int j = bj % a.T, b = bj / a.T;
    const int h = hq / G, tile = j / a.nt;
    const int item = (tile >> 1) * a.units + b * d.Hkv + h;
    const int base = item * a.tpu;
    const int c0 = base / a.per, parts = (base + a.tpu - 1) / a.per - c0 + 1;
    if (parts == 1) return;                                       // written directly
    const long long prow = (tile & 1) * 128 + (j - tile * a.nt) * G + hq - h * G;
    // the item is the last segment of its first CTA, and the first one of the others
    const long long place0 = 2 * c0 + (c0 * a.per / a.tpu == item ? 0 : 1);
    auto at = [&](int k) { return (k == 0 ? place0 : 2ll * (c0 + k)) * 256 + prow; };
    float M = kNegInf, L = 0.f;
    for (int k0 = 0; k0 < parts; k0 += 32) {
        const float lk = k0 + lane < parts ? a.ws_lse[at(k0 + lane)] : kNegInf;
        const float m = fmaxf(M, warp_max_f32(lk));
        L = m != kNegInf ? L * exp2f(M - m) : L;
        L += lk == kNegInf ? 0.f : exp2f(lk - m);                 // an empty part: 0
        M = m;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, o);
    const float inv = L != 0.f ? 1.f / L : 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < parts; k0 += 32) {
        const float lk = k0 + lane < parts ? a.ws_lse[at(k0 + lane)] : kNegInf;
        const float w = lk == kNegInf ? 0.f : exp2f(lk - M) * inv;
        const int nk = min(32, parts - k0);
#pragma unroll 8
        for (int k = 0; k < nk; ++k) {
            const float wk = __shfl_sync(0xFFFFFFFFu, w, k);
            const float4 v = reinterpret_cast<const float4*>(a.ws_o + at(k0 + k) * kHeadDim)[lane];
            acc.x += wk * v.x;
            acc.y += wk * v.y;
            acc.z += wk * v.z;
            acc.w += wk * v.w;
        }
    }
    reinterpret_cast<uint2*>(a.out + static_cast<long long>(row) * kHeadDim)[lane] =
        make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
    if (lane == 0) a.lse[row] = L != 0.f ? (M + log2f(L)) * kLn2 : kNegInf;
}

}  // namespace oasis
