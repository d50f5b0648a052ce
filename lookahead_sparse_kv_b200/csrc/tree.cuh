// tree.cuh - the draft tree's bookkeeping: visibility words and positions
// from the nodes' parents, and the accepted path's rows into the cache.
//
// OasisKV: Scaling In-Decode KV Cache Beyond HBM with Lookahead Sparse
// Prefetching, Figure 8: the drafts of a step are verified together; what
// stands becomes part of the cache before the next step.
#pragma once

#include "common.cuh"
#include "summaries.cuh"

namespace oasis {

constexpr int kMaxTree = 64;                       // nodes a tree: one bit each of a 64-bit word
constexpr int kLayoutTrees = 4;                    // trees a CTA

// One thread per node.  word[j] = bit j | word[parent[j]]: after round i a
// node knows its 2^i nearest ancestors and who stands beyond them, so six
// rounds do for 64 nodes whatever their depth.  What bounds it is the launch
// and two dependent loads: 264 KB in all at 256 trees of 64 nodes, 1.8 us.
__global__ void __launch_bounds__(kLayoutTrees * kMaxTree) tree_layout_kernel(
    int B, int T, const int32_t* __restrict__ parent, const int32_t* __restrict__ n_nodes,
    const int32_t* __restrict__ ctx_len, uint64_t* __restrict__ mask, int32_t* __restrict__ pos) {
    __shared__ uint64_t s_word[kLayoutTrees][kMaxTree];
    __shared__ int s_up[kLayoutTrees][kMaxTree];
    const int g = threadIdx.x / kMaxTree, j = threadIdx.x % kMaxTree;
    const int b = blockIdx.x * kLayoutTrees + g;
    const bool in = b < B && j < T;
    const long long at = static_cast<long long>(b) * T + j;
    int n = T, up = -1, ctx = 0;
    if (in) {
        up = parent[at];
        if (n_nodes != nullptr) n = n_nodes[b];
        ctx = ctx_len[b];
        if (n < 0 || n > T) raise_dev_error(OASIS_DEVERR_ID_RANGE);
    }
    const bool real = in && j < n;
    if (real && (up < -1 || up >= j)) {
        raise_dev_error(OASIS_DEVERR_ID_RANGE);
        up = -1;                                   // taken as a root
    }
    uint64_t word = real ? 1ull << j : 0ull;
    if (!real) up = -1;
    s_word[g][j] = word;
    s_up[g][j] = up;
    __syncthreads();
    for (int have = 1; have < T; have <<= 1) {
        const uint64_t w = up >= 0 ? s_word[g][up] : 0ull;
        const int u2 = up >= 0 ? s_up[g][up] : -1;
        __syncthreads();
        s_word[g][j] = word |= w;
        s_up[g][j] = up = u2;
        __syncthreads();
    }
    if (in) {
        mask[at] = word;
        pos[at] = ctx + max(0, __popcll(word) - 1);
    }
}

// The cache buffers of up to kCommitLayers layers, passed by value.
constexpr int kCommitLayers = 64;
constexpr int kCommitThreads = 128;
constexpr int kCommitBlocks = kMaxTree / kBlockTokens + 1;   // blocks that 64 consecutive tokens can touch
struct CommitLayers {
    uint4* host[kCommitLayers];
    uint4* pool[kCommitLayers];
    uint4* kmin[kCommitLayers];
    uint4* kmax[kCommitLayers];
    const int32_t* slot_table[kCommitLayers];
};

// One CTA per (unit, layer), every layer of a stack in one launch.  16 lanes
// move a 256-B row; a unit's rows are few (the path's length), so the CTA's
// eight groups take them together and then fold the keys into the touched
// blocks' summaries, one group a block, in path order (min and max do not
// depend on it).  The host copy is written over PCIe straight from here; that
// link bounds the call (512 B a row, layer and KV head), not HBM: 2.36 MB of a 64-layer
// stack take 47-50 us, 42 us at the link's 56.7 GB/s; without a host copy 8 us.
__global__ void __launch_bounds__(kCommitThreads) commit_path_kernel(
    const __grid_constant__ CommitLayers L, Dims d, int T, const uint4* __restrict__ k_tree, const uint4* __restrict__ v_tree,
    const int32_t* __restrict__ path, const int32_t* __restrict__ n_accept, const int32_t* __restrict__ ctx_len,
    int32_t* __restrict__ ctx_len_out) {
    __shared__ int s_node[kMaxTree];
    __shared__ int s_slot[kCommitBlocks];
    const int bh = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x;
    const int b = bh / d.Hkv;
    const int ctx = ctx_len[b];
    int n = n_accept[b];
    if (n < 0 || n > T) {
        if (tid == 0) raise_dev_error(OASIS_DEVERR_ID_RANGE);
        n = n < 0 ? 0 : T;
    }
    const int room = ctx < 0 ? 0 : max(0, d.N * kBlockTokens - ctx);
    if (n > room) {
        if (tid == 0) raise_dev_error(OASIS_DEVERR_APPEND_FULL);
        n = room;
    }
    if (ctx_len_out != nullptr && layer == 0 && bh % d.Hkv == 0 && tid == 0) ctx_len_out[b] = ctx + n;
    if (n == 0) return;
    if (tid < n) {
        int node = path[static_cast<long long>(b) * T + tid];
        if (node < 0 || node >= T) {
            raise_dev_error(OASIS_DEVERR_ID_RANGE);
            node = -1;                             // its position is taken, and left as it was
        }
        s_node[tid] = node;
    }
    if (tid < kCommitBlocks) s_slot[tid] = 0x7FFFFFFF;
    __syncthreads();
    const int first = ctx / kBlockTokens, last = (ctx + n - 1) / kBlockTokens;
    uint4* pool = L.pool[layer];
    if (pool != nullptr) {
        const int32_t* st = L.slot_table[layer] + static_cast<long long>(bh) * d.K;
        for (int s = tid; s < d.K; s += kCommitThreads) {
            const int blk = st[s];
            if (blk >= first && blk <= last) atomicMin(&s_slot[blk - first], s);
        }
        __syncthreads();
    }
    const int lane = tid & 15, group = tid >> 4;
    const long long tree0 = (static_cast<long long>(layer) * d.B * d.Hkv + bh) * T;
    uint4* host = L.host[layer];
    for (int it = group; it < 2 * n; it += kCommitThreads / 16) {
        const int i = it >> 1, kv = it & 1;
        const int node = s_node[i];
        if (node < 0) continue;
        const uint4 row = (kv ? v_tree : k_tree)[(tree0 + node) * 16 + lane];
        const int blk = (ctx + i) / kBlockTokens, t = (ctx + i) % kBlockTokens;
        const int in_block = (kv * kBlockTokens + t) * 16 + lane;
        if (host != nullptr) host[(static_cast<long long>(bh) * d.N + blk) * (kBlockBytes / 16) + in_block] = row;
        const int slot = s_slot[blk - first];
        if (slot < d.K) pool[(static_cast<long long>(bh) * d.K + slot) * (kBlockBytes / 16) + in_block] = row;
    }
    if (group <= last - first) {
        const int blk = first + group;
        const int i0 = max(0, blk * kBlockTokens - ctx), i1 = min(n, (blk + 1) * kBlockTokens - ctx);
        const long long o = (static_cast<long long>(bh) * d.N + blk) * 16 + lane;
        float lo[8], hi[8];
        bool have = (ctx + i0) % kBlockTokens != 0;
        if (have) {
            bf16x8_to_f32(L.kmin[layer][o], lo);
            bf16x8_to_f32(L.kmax[layer][o], hi);
        }
        for (int i = i0; i < i1; ++i) {
            const int node = s_node[i];
            if (node < 0) continue;
            float a[8];
            bf16x8_to_f32(k_tree[(tree0 + node) * 16 + lane], a);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                lo[c] = have ? fminf(lo[c], a[c]) : a[c];
                hi[c] = have ? fmaxf(hi[c], a[c]) : a[c];
            }
            have = true;
        }
        if (have) {
            L.kmin[layer][o] = f32x8_to_bf16(lo);
            L.kmax[layer][o] = f32x8_to_bf16(hi);
        }
    }
}

}  // namespace oasis
