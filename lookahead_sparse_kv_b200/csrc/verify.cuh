// verify.cuh - which drafted tokens stand: rejection sampling down the draft
// tree from given random numbers.
//
// At node `cur` the target's row p and (where the drafts were sampled) the
// draft's row d of that node, children tested in index order:
//   r_0 = p, S_0 = 1;  child x stands if r_k(x) > 0 and u S_k d(x) < r_k(x);
//   else r_{k+1} = max(r_k - S_k d, 0), S_{k+1} = sum r_{k+1}
// (without draft rows d is 1 at the child's token: S_{k+1} = S_k - r_k(x) and
// r_{k+1}(x) = 0).  When no child stands the next token is drawn from r: the
// first index whose running sum passes u times the sum.  Everything is fp64:
// sums in another order then differ by about 1e-15, so which token comes out
// does not hang on how the row is split.  Entries that are not positive finite
// numbers count as 0.
//
// r_k is never stored: it is recomputed from p, d and S_0..S_{k-1}.  One
// cluster of 8 CTAs per sequence.  CTA 0 walks the tree on single entries
// gathered up front (all nodes' parents, tokens, p and d at the token) and
// sends the others a command when a sum over the vocabulary is needed: after a
// rejection with children left, and for the draw.  Each CTA sums its eighth of
// the row and pushes the sum to the peers.  HBM bounds it at many sequences
// (the rows p and d of the last node, once), latency at one: the walk's
// gathers, a pass over an eighth of the row and three cluster barriers.
#pragma once

#include <cooperative_groups.h>

#include "common.cuh"
#include "tree.cuh"

namespace oasis {

constexpr int kVerCluster = 8;
constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kVerUnroll = 8;

struct VerifyArgs {
    const float* probs;          // [B][T] rows of `vocab` floats, row_stride apart
    const float* draft;          // same, or NULL
    const int32_t* tokens;       // [B][T]
    const int32_t* parent;       // [B][T]
    const int32_t* n_nodes;      // [B] or NULL
    const float* u_accept;       // [B][T]
    const float* u_sample;       // [B]
    int32_t* path;               // [B][T]
    int32_t* n_accept;           // [B]
    int32_t* next_token;         // [B]
    long long row_stride;
    int B, T, vocab;
};

struct VerifyCmd {
    int cur, rounds, last;                         // node, rejections before this sum, whether the draw follows
};

// Probabilities that are no positive finite numbers count as 0.
__device__ __forceinline__ double ver_clean(float x) {
    return x > 0.f && x < __int_as_float(0x7f800000) ? static_cast<double>(x) : 0.0;
}

// The row that is summed or drawn from: r after `rounds` rejections at a node.
struct VerifyRow {
    const float* p;
    const float* d;              // NULL without draft rows, or where none is needed
    const double* S;             // S_0 .. S_{rounds-1}
    const int* gone;             // without draft rows: the tokens turned down
    int rounds;
    __device__ __forceinline__ double left(float pv, float dv, int i) const {
        double x = ver_clean(pv);
        if (d != nullptr) {
            const double dq = ver_clean(dv);
            for (int k = 0; k < rounds; ++k) x = fmax(x - S[k] * dq, 0.0);
        } else {
            for (int k = 0; k < rounds; ++k)
                if (gone[k] == i) x = 0.0;
        }
        return x;
    }
};

// A warp's entries i0 + 32k + lane of the row, loads in flight together.
__device__ __forceinline__ void ver_load(const VerifyRow& r, int i0, int hi, int lane, double (&x)[kVerUnroll]) {
    float pv[kVerUnroll], dv[kVerUnroll];
#pragma unroll
    for (int k = 0; k < kVerUnroll; ++k) {
        const int i = i0 + 32 * k + lane;
        pv[k] = i < hi ? r.p[i] : 0.f;
        dv[k] = r.d != nullptr && i < hi ? r.d[i] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kVerUnroll; ++k) x[k] = r.left(pv[k], dv[k], i0 + 32 * k + lane);
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

__global__ void __cluster_dims__(kVerCluster, 1, 1) __launch_bounds__(kVerThreads)
    verify_tree_kernel(const VerifyArgs a) {
    namespace cg = cooperative_groups;
    cg::cluster_group cl = cg::this_cluster();
    __shared__ int s_parent[kMaxTree], s_token[kMaxTree], s_path[kMaxTree];
    __shared__ float s_u[kMaxTree], s_p[kMaxTree], s_d[kMaxTree];
    __shared__ double s_S[kMaxTree + 1];           // S_0 .. of the node being tested
    __shared__ int s_gone[kMaxTree];               // without draft rows: tokens turned down at this node
    __shared__ VerifyCmd s_cmd;
    __shared__ double s_part[2][kVerCluster];      // the CTAs' sums of a pass, two passes deep
    __shared__ double s_warp[kVerWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = static_cast<int>(cl.block_rank());
    const int b = static_cast<int>(blockIdx.x) / kVerCluster;
    const int T = a.T;
    const bool has_draft = a.draft != nullptr;
    const long long row0 = static_cast<long long>(b) * T;
    int n = a.n_nodes != nullptr ? a.n_nodes[b] : T;
    if (n < 0 || n > T) {
        if (rank == 0 && tid == 0) raise_dev_error(OASIS_DEVERR_ID_RANGE);
        n = n < 0 ? 0 : T;
    }
    if (rank == 0) {
        if (tid < T) {
            const int j = tid;
            int par = -1, x = -1;
            float pj = 0.f, dj = 0.f;
            if (j > 0 && j < n) {
                par = a.parent[row0 + j];
                x = a.tokens[row0 + j];
                if (par < -1 || par >= j || x < 0 || x >= a.vocab) {
                    raise_dev_error(OASIS_DEVERR_ID_RANGE);
                    par = -1;                      // never tested
                }
                if (par >= 0) {
                    const long long at = (row0 + par) * a.row_stride + x;
                    pj = a.probs[at];
                    if (has_draft) dj = a.draft[at];
                }
            }
            s_parent[j] = par;
            s_token[j] = x;
            s_p[j] = pj;
            s_d[j] = dj;
            s_u[j] = a.u_accept[row0 + j];
            s_path[j] = j == 0 && n > 0 ? 0 : -1;
        }
        if (tid == 0) s_S[0] = 1.0;
        __syncthreads();
    }
    // the entries that a warp sums, in order over ranks and warps
    const int per_cta = ((a.vocab + kVerCluster - 1) / kVerCluster + 31) / 32 * 32;
    const int c_lo = min(a.vocab, rank * per_cta), c_hi = min(a.vocab, c_lo + per_cta);
    const int per_warp = ((c_hi - c_lo + kVerWarps - 1) / kVerWarps + 31) / 32 * 32;
    const int w_lo = min(c_hi, c_lo + warp * per_warp), w_hi = min(c_hi, w_lo + per_warp);

    int cur = 0, tested = 0, count = 1, rounds = 0;   // the walk (CTA 0's thread 0)
    double total = 0.0, before = 0.0;
    int slot = 0;
    VerifyRow row;
    while (true) {
        if (rank == 0) {
            if (tid == 0) {
                VerifyCmd c;
                c.last = 1;
                while (true) {
                    int j = max(cur, tested) + 1;
                    while (j < n && s_parent[j] != cur) ++j;
                    if (j >= n) break;
                    tested = j;
                    const double S = s_S[rounds];
                    double p = ver_clean(s_p[j]), dq = 1.0;
                    if (has_draft) {
                        dq = ver_clean(s_d[j]);
                        for (int i = 0; i < rounds; ++i) p = fmax(p - s_S[i] * dq, 0.0);
                    } else {
                        for (int i = 0; i < rounds; ++i)
                            if (s_gone[i] == s_token[j]) p = 0.0;
                    }
                    if (p > 0.0 && static_cast<double>(s_u[j]) * S * dq < p) {
                        s_path[count++] = j;
                        cur = j;
                        rounds = 0;                // (s_S[0] stays 1)
                        continue;
                    }
                    ++rounds;
                    if (!has_draft) {
                        s_gone[rounds - 1] = s_token[j];
                        s_S[rounds] = S - p;
                        continue;
                    }
                    // the sum after this rejection: for the next child, or for the draw
                    int k = j + 1;
                    while (k < n && s_parent[k] != cur) ++k;
                    c.last = k >= n;
                    break;
                }
                c.cur = cur;
                c.rounds = rounds;
                s_cmd = c;
            }
            __syncthreads();
            if (tid > 0 && tid < kVerCluster) {
                *cl.map_shared_rank(&s_cmd, tid) = s_cmd;
                double* S = cl.map_shared_rank(&s_S[0], tid);
                int* gone = cl.map_shared_rank(&s_gone[0], tid);
                for (int i = 0; i < s_cmd.rounds; ++i) {
                    S[i] = s_S[i];
                    if (!has_draft) gone[i] = s_gone[i];
                }
            }
        }
        cl.sync();
        const VerifyCmd c = s_cmd;
        row.p = a.probs + (row0 + c.cur) * a.row_stride;
        row.d = has_draft && c.rounds > 0 ? a.draft + (row0 + c.cur) * a.row_stride : nullptr;
        row.S = s_S;
        row.gone = s_gone;
        row.rounds = c.rounds;
        while (true) {
            double mine = 0.0;
            for (int i0 = w_lo; i0 < w_hi; i0 += 32 * kVerUnroll) {
                double x[kVerUnroll];
                ver_load(row, i0, w_hi, lane, x);
#pragma unroll
                for (int k = 0; k < kVerUnroll; ++k) mine += x[k];
            }
            mine = warp_sum(mine);
            if (lane == 0) s_warp[warp] = mine;
            __syncthreads();
            if (tid < kVerCluster) {
                double sum = 0.0;
                for (int k = 0; k < kVerWarps; ++k) sum += s_warp[k];
                cl.map_shared_rank(&s_part[0][0], tid)[slot * kVerCluster + rank] = sum;
            }
            cl.sync();
            total = 0.0;
            for (int r = 0; r < kVerCluster; ++r) {
                if (r == rank) before = total;
                total += s_part[slot][r];
            }
            if (!c.last || total > 0.0 || row.rounds == 0) break;
            row.rounds = 0;                        // nothing is left of the row: drawn from the row itself
            row.d = nullptr;
            slot ^= 1;
        }
        if (c.last) break;
        if (rank == 0 && tid == 0) s_S[rounds] = total;
        slot ^= 1;
    }
    // No CTA touches another's shared memory from here on, so each may leave.

    if (rank == 0) {
        if (tid < T) a.path[row0 + tid] = s_path[tid];
        if (tid == 0) {
            a.n_accept[b] = n > 0 ? count : 0;
            if (n == 0 || !(total > 0.0)) a.next_token[b] = -1;
        }
    }
    if (n == 0 || !(total > 0.0)) return;
    // The draw.  Every CTA holds the same eight sums, so they agree on the one
    // that holds the crossing; sums are carried on in the same order level by
    // level, and a crossing that rounding hides from the last level is at the
    // last entry with mass.
    const double t = fmax(static_cast<double>(a.u_sample[b]), 0.0) * total;
    int owner = -1;
    {
        double run = 0.0;
        int some = 0;
        for (int r = 0; r < kVerCluster; ++r) {
            const double s = s_part[slot][r];
            if (s > 0.0) some = r;
            if (owner < 0 && run + s > t) owner = r;
            run += s;
        }
        if (owner < 0) owner = some;
    }
    if (rank != owner) return;
    int wo = -1;
    double base = before;
    {
        double run = 0.0;
        int some = 0;
        double some_base = before;
        for (int w = 0; w < kVerWarps; ++w) {
            const double s = s_warp[w];
            if (s > 0.0) some = w, some_base = before + run;
            if (wo < 0 && before + (run + s) > t) wo = w, base = before + run;
            run += s;
        }
        if (wo < 0) wo = some, base = some_base;
    }
    if (warp != wo) return;
    int found = -1, fallback = 0;
    double carry = base;
    for (int i0 = w_lo; i0 < w_hi && found < 0; i0 += 32 * kVerUnroll) {
        double x[kVerUnroll];
        ver_load(row, i0, w_hi, lane, x);
#pragma unroll
        for (int k = 0; k < kVerUnroll; ++k) {
            double inc = x[k];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
                if (lane >= o) inc += y;
            }
            const unsigned some = __ballot_sync(0xFFFFFFFFu, x[k] > 0.0);
            const unsigned over = __ballot_sync(0xFFFFFFFFu, x[k] > 0.0 && carry + inc > t);
            if (found < 0 && over != 0) found = i0 + 32 * k + __ffs(over) - 1;
            if (some != 0) fallback = i0 + 32 * k + 31 - __clz(some);
            carry += __shfl_sync(0xFFFFFFFFu, inc, 31);
        }
    }
    if (lane == 0) a.next_token[b] = found >= 0 ? found : fallback;
}

}  // namespace oasis
