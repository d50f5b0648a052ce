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
// r_k is never stored.  Subtracting and cutting at 0 again and again is doing it
// once with the sum, r_k = max(p - c_k d, 0), c_k = S_0 + .. + S_{k-1}, so a row is
// always p, d and one number.  One cluster of 8 or 16 CTAs per sequence.  CTA 0
// walks the tree on single entries gathered up front (all nodes' parents, tokens,
// p and d at the token) and sends the others a command when a sum over the
// vocabulary is needed: after a rejection with children left, and for the draw.
// Each CTA keeps its share of the node's rows in shared memory, copied there with
// all of its loads in flight at once, sums it, and pushes the sum to the peers;
// further sums at the same node, and the draw, read no memory.  HBM bounds it at
// many sequences (the rows p and d of the last node, once), latency at one: the
// walk's gathers, a share of the row and three cluster barriers.
#pragma once

#include <cooperative_groups.h>

#include "common.cuh"
#include "tree.cuh"

namespace oasis {

constexpr int kVerMaxCluster = 16;
constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kVerMaxVocab = 1 << 18;              // 16 CTAs hold two rows of as many in 131 KiB each

// 16-byte groups of a row that a CTA holds at most (rows begin anywhere in a group).
__host__ __device__ constexpr int ver_cap(int vocab, int cluster) { return ((vocab + 6) / 4 + cluster - 1) / cluster; }

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
    double c;                                      // what of the draft's row is taken off
    int cur, rounds, last;                         // node, rejections before this sum, whether the draw follows
};

// What is no positive finite number counts as 0.
__device__ __forceinline__ double ver_clean(float x) {
    return x > 0.f && x < __int_as_float(0x7f800000) ? static_cast<double>(x) : 0.0;
}

// x 2^-896 as a double, for finite x >= 0: an fp32 number's bits moved 29 places
// up are that double's, subnormals and 0 included, as the exponents differ by
// 127 - 1023.  (The conversion instruction runs at 16 a cycle and SM; sums need no
// scale until they are done.)
__device__ __forceinline__ double ver_wide(float x) {
    unsigned long long w;
    asm("mul.wide.u32 %0, %1, 0x20000000;" : "=l"(w) : "r"(__float_as_uint(x)));
    return __longlong_as_double(static_cast<long long>(w));
}
constexpr double kVerScale = 0x1p896;

// A CTA's share of the row that is summed or drawn from, r after some
// rejections at a node, in shared memory.  Rows are taken in 16-byte groups of 4
// entries; a row begins anywhere (an odd vocabulary), so group g holds entries
// 4g - off .. 4g - off + 3.
struct VerifyRow {
    const float4 *p, *d;         // groups c_lo.. of the target's and the draft's row
    double c;                    // r = max(p - c d, 0); 0: p
    const int* gone;             // without draft rows: the tokens turned down
    int n_gone, off, c_lo;

    // Copies groups [lo, hi) of a row to `to` (the calling warp's lanes; the ends entry by entry).
    __device__ __forceinline__ void fetch(const float* r, int vocab, int lo, int hi, int lane, float4* to) const {
        for (int g = lo + lane; g < hi; g += 32) {
            const int i = 4 * g - off;
            if (i >= 0 && i + 3 < vocab) {
                cp_async_16(to + (g - c_lo), r + i);
            } else {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = i + e >= 0 && i + e < vocab ? __ldg(r + i + e) : 0.f;
                to[g - c_lo] = make_float4(v[0], v[1], v[2], v[3]);
            }
        }
    }
    // r of an entry, times 2^-896, before it is cut at 0
    __device__ __forceinline__ double raw(float pv, float dv) const { return fma(-c, ver_wide(dv), ver_wide(pv)); }
    __device__ __forceinline__ double left(float pv, float dv) const {
        const double y = raw(pv, dv);
        return y > 0.0 ? y : 0.0;
    }
    // Group g (zeros from hi on), 0 for what is no positive finite number and for tokens turned down; the warp's
    // lanes hold consecutive groups.
    __device__ __forceinline__ void get(int g, int hi, int lane, float4& pv, float4& dv) const {
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
        pv = g < hi ? p[g - c_lo] : zero;
        dv = c != 0.0 && g < hi ? d[g - c_lo] : zero;
        if (__any_sync(0xFFFFFFFFu, max(top(pv), top(dv)) > 0x7F7FFFFFu)) {   // a sign, an infinity or NaN
            pv = sound(pv);
            dv = sound(dv);
        }
        for (int j = 0; j < n_gone; j += 32) {
            const int e = j + lane < n_gone ? gone[j + lane] + off - 4 * (g - lane) : -1;
            unsigned hit = __ballot_sync(0xFFFFFFFFu, e >= 0 && e < 128);
            for (; hit != 0; hit &= hit - 1) {
                const int at = __shfl_sync(0xFFFFFFFFu, e, __ffs(hit) - 1);
                if (at >> 2 == lane) {
                    if ((at & 3) == 0) pv.x = 0.f;
                    if ((at & 3) == 1) pv.y = 0.f;
                    if ((at & 3) == 2) pv.z = 0.f;
                    if ((at & 3) == 3) pv.w = 0.f;
                }
            }
        }
    }
    __device__ __forceinline__ static uint32_t top(const float4& v) {
        return max(max(__float_as_uint(v.x), __float_as_uint(v.y)), max(__float_as_uint(v.z), __float_as_uint(v.w)));
    }
    __device__ __forceinline__ static float sound(float x) { return x > 0.f && x < __int_as_float(0x7f800000) ? x : 0.f; }
    __device__ __forceinline__ static float4 sound(const float4& v) {
        return make_float4(sound(v.x), sound(v.y), sound(v.z), sound(v.w));
    }
};

// sum += y where y >= 0
__device__ __forceinline__ void ver_add(double& sum, double y) {
    asm("{\n\t.reg .pred q;\n\tsetp.ge.s32 q, %1, 0;\n\t@q add.rn.f64 %0, %0, %2;\n\t}\n"
        : "+d"(sum)
        : "r"(__double2hiint(y)), "d"(y));
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

__global__ void __launch_bounds__(kVerThreads, 2) verify_tree_kernel(const VerifyArgs a) {
    namespace cg = cooperative_groups;
    cg::cluster_group cl = cg::this_cluster();
    __shared__ int s_token[kMaxTree], s_path[kMaxTree];
    __shared__ float s_u[kMaxTree], s_p[kMaxTree], s_d[kMaxTree];
    __shared__ unsigned int s_kids[kMaxTree][2];   // each node's children, a bit each
    __shared__ int s_gone[kMaxTree];               // without draft rows: tokens turned down at this node
    __shared__ VerifyCmd s_cmd;
    __shared__ double s_part[2][kVerMaxCluster];   // the CTAs' sums of a pass, two passes deep
    extern __shared__ float4 s_rows[];             // the shares of p and d
    __shared__ double s_warp[kVerWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = static_cast<int>(cl.block_rank());
    const int cta = static_cast<int>(cl.num_blocks());
    const int b = static_cast<int>(blockIdx.x) / cta;
    const int T = a.T;
    const bool has_draft = a.draft != nullptr;
    const long long row0 = static_cast<long long>(b) * T;
    int par = -1, x = -1;
    if (rank == 0 && tid < T) {                    // (in flight together with the count)
        par = a.parent[row0 + tid];
        x = a.tokens[row0 + tid];
        s_kids[tid][0] = s_kids[tid][1] = 0u;
    }
    int n = a.n_nodes != nullptr ? a.n_nodes[b] : T;
    if (n < 0 || n > T) {
        if (rank == 0 && tid == 0) raise_dev_error(OASIS_DEVERR_ID_RANGE);
        n = n < 0 ? 0 : T;
    }
    if (rank == 0) {
        __syncthreads();
        if (tid < T) {
            const int j = tid;
            const bool real = j > 0 && j < n;
            const bool sound = par >= -1 && par < j && x >= 0 && x < a.vocab;
            if (real && !sound) raise_dev_error(OASIS_DEVERR_ID_RANGE);   // never tested
            float pj = 0.f, dj = 0.f;
            if (real && sound && par >= 0) {
                const long long at = (row0 + par) * a.row_stride + x;
                pj = a.probs[at];
                if (has_draft) dj = a.draft[at];
                atomicOr(&s_kids[par][j >> 5], 1u << (j & 31));
            }
            s_token[j] = x;
            s_p[j] = pj;
            s_d[j] = dj;
            s_u[j] = a.u_accept[row0 + j];
            s_path[j] = j == 0 && n > 0 ? 0 : -1;
        }
        __syncthreads();
    }
    // the walk (CTA 0's thread 0): current node, its children not tested yet, S and the sum of the S before
    int cur = 0, count = 1, rounds = 0;
    uint64_t kids = 0;
    double S = 1.0, c_off = 0.0;
    if (rank == 0) kids = s_kids[0][0] | (static_cast<uint64_t>(s_kids[0][1]) << 32);
    double total = 0.0, before = 0.0;              // (times 2^-896)
    int slot = 0;
    VerifyRow row;
    row.gone = s_gone;
    row.p = s_rows;
    row.d = s_rows + ver_cap(a.vocab, cta);
    int w_lo = 0, w_hi = 0;                        // the groups that this warp sums
    int have = -1;                                 // node whose rows are here
    while (true) {
        if (rank == 0) {
            if (tid == 0) {
                VerifyCmd c;
                c.last = 1;
                while (kids != 0) {
                    const int j = __ffsll(static_cast<long long>(kids)) - 1;
                    kids &= kids - 1;
                    double p = ver_clean(s_p[j]), dq = 1.0;
                    if (has_draft) {
                        dq = ver_clean(s_d[j]);
                        p = fma(-c_off, dq, p);
                    } else {
                        for (int i = 0; i < rounds; ++i)
                            if (s_gone[i] == s_token[j]) p = 0.0;
                    }
                    if (p > 0.0 && static_cast<double>(s_u[j]) * S * dq < p) {
                        s_path[count++] = j;
                        cur = j;
                        kids = s_kids[j][0] | (static_cast<uint64_t>(s_kids[j][1]) << 32);
                        rounds = 0;
                        S = 1.0;
                        c_off = 0.0;
                        continue;
                    }
                    if (!has_draft) {
                        s_gone[rounds++] = s_token[j];
                        S -= p;
                        continue;
                    }
                    // the sum after this rejection: for the next child, or for the draw
                    ++rounds;
                    c_off += S;
                    c.last = kids == 0;
                    break;
                }
                c.cur = cur;
                c.rounds = rounds;
                c.c = c_off;
                s_cmd = c;
            }
            __syncthreads();
            if (tid > 0 && tid < cta) {
                *cl.map_shared_rank(&s_cmd, tid) = s_cmd;
                if (!has_draft) {
                    int* gone = cl.map_shared_rank(&s_gone[0], tid);
                    for (int i = 0; i < s_cmd.rounds; ++i) gone[i] = s_gone[i];
                }
            }
        }
        cl.sync();
        const VerifyCmd c = s_cmd;
        row.c = c.c;
        row.n_gone = has_draft ? 0 : c.rounds;
        if (have != c.cur) {
            // in order over CTAs and warps; a warp reads what it copied itself
            const long long at = (row0 + c.cur) * a.row_stride;
            row.off = static_cast<int>(at & 3);
            const int groups = (a.vocab + row.off + 3) / 4;
            const int per_cta = (groups + cta - 1) / cta;
            const int c_hi = min(groups, (rank + 1) * per_cta);
            row.c_lo = min(groups, rank * per_cta);
            const int per_warp = (c_hi - row.c_lo + kVerWarps - 1) / kVerWarps;
            w_lo = min(c_hi, row.c_lo + warp * per_warp);
            w_hi = min(c_hi, w_lo + per_warp);
            row.fetch(a.probs + at, a.vocab, w_lo, w_hi, lane, const_cast<float4*>(row.p));
            if (c.c != 0.0) row.fetch(a.draft + at, a.vocab, w_lo, w_hi, lane, const_cast<float4*>(row.d));
            have = c.cur;
            cp_async_wait_all();
            __syncwarp();
        }
        for (int again = 0;; ++again) {
            double sum[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 2
            for (int g0 = w_lo; g0 < w_hi; g0 += 32) {
                float4 pv, dv;
                row.get(g0 + lane, w_hi, lane, pv, dv);
                ver_add(sum[0], row.raw(pv.x, dv.x));
                ver_add(sum[1], row.raw(pv.y, dv.y));
                ver_add(sum[2], row.raw(pv.z, dv.z));
                ver_add(sum[3], row.raw(pv.w, dv.w));
            }
            const double mine = warp_sum((sum[0] + sum[1]) + (sum[2] + sum[3]));
            if (lane == 0) s_warp[warp] = mine;
            __syncthreads();
            if (tid < cta) {
                double sum = 0.0;
#pragma unroll
                for (int k = 0; k < kVerWarps; ++k) sum += s_warp[k];
                cl.map_shared_rank(&s_part[0][0], tid)[slot * kVerMaxCluster + rank] = sum;
            }
            cl.sync();
            total = 0.0;
            for (int r = 0; r < cta; ++r) {
                if (r == rank) before = total;
                total += s_part[slot][r];
            }
            if (!c.last || total > 0.0 || c.rounds == 0 || again) break;
            row.c = 0.0;                           // nothing is left of the row: drawn from the row itself
            row.n_gone = 0;
            slot ^= 1;
        }
        if (c.last) break;
        S = total * kVerScale;
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
    // The draw.  Every CTA holds the same sums, so they agree on the one
    // that holds the crossing; sums are carried on in the same order level by
    // level, and a crossing that rounding hides from the last level is at the
    // last entry with mass.
    const double t = fmax(static_cast<double>(a.u_sample[b]), 0.0) * total;
    int owner = -1;
    {
        double run = 0.0;
        int some = 0;
        for (int r = 0; r < cta; ++r) {
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
    int found = -1, fallback = -1;
    double carry = base;
    for (int g0 = w_lo; g0 < w_hi && found < 0; g0 += 32) {
        float4 pv, dv;
        row.get(g0 + lane, w_hi, lane, pv, dv);
        const double x[4] = {row.left(pv.x, dv.x), row.left(pv.y, dv.y), row.left(pv.z, dv.z), row.left(pv.w, dv.w)};
        const int i = 4 * (g0 + lane) - row.off;
        const double sum = (x[0] + x[1]) + (x[2] + x[3]);
        double inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += y;
        }
        double run = __shfl_up_sync(0xFFFFFFFFu, inc, 1);
        run = carry + (lane > 0 ? run : 0.0);
        int over = -1, last = -1;                  // this lane's first entry past t, and its last one with mass
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            run += x[e];
            if (x[e] > 0.0) {
                last = i + e;
                if (over < 0 && run > t) over = i + e;
            }
        }
        const unsigned has = __ballot_sync(0xFFFFFFFFu, over >= 0);
        const unsigned some = __ballot_sync(0xFFFFFFFFu, last >= 0);
        if (has != 0) found = __shfl_sync(0xFFFFFFFFu, over, __ffs(has) - 1);
        if (some != 0) fallback = __shfl_sync(0xFFFFFFFFu, last, 31 - __clz(some));
        carry += __shfl_sync(0xFFFFFFFFu, inc, 31);
    }
    if (lane == 0) a.next_token[b] = found >= 0 ? found : fallback;
}

}  // namespace oasis
