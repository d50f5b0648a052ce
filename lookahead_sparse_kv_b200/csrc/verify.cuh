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
// gathers single entries up front (all nodes' parents, tokens, p and d at the
// token) and hands them to the others, so that every CTA walks the tree on the same
// numbers (nothing else decides how often the cluster meets) and they agree when a
// sum over the vocabulary is needed: after a rejection with children left, and for
// the draw.
// Each CTA sums its share of the row and pushes the sum to the peers.  Every lane
// streams its entries through a ring of its own in shared memory (six stages of 32
// bytes in flight, 96 KiB a CTA), so no load waits for another and no thread for
// another's; rows are read again for each sum, from L2.  HBM bounds it at many
// sequences (the rows p and d of the last node, once), latency at one: the walk's
// gathers, a share of the row and two cluster barriers.  32 trees of 26 nodes over
// 151,669 entries: 33.6 us (up to four sums one after another, ~6 us each, of which the
// first waits for HBM; 40 MB read); one chain of 5 over 32,000: 8.2 us; trees of 8 over
// 151,669, one sequence 12.5 us, without draft rows 11.1 (a sum for the draw alone).
#pragma once

#include <cooperative_groups.h>

#include <utility>

#include "common.cuh"
#include "tree.cuh"

namespace oasis {

constexpr int kVerMaxCluster = 16;
constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kVerRing = 6;                        // stages of a lane's ring: 16 bytes of each row
constexpr int kVerSmem = kVerThreads * kVerRing * 2 * 16;

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
    int cur, rounds, last, count;                  // node, rejections before this sum, whether the draw follows, path so far
};

// What the walk looks at, the same in every CTA of a cluster.
struct VerifyIn {
    int token[kMaxTree];
    float p[kMaxTree], d[kMaxTree], u[kMaxTree];   // the parent's rows at the token, and the node's number
    unsigned int kids[kMaxTree][2];                // each node's children, a bit each
    int n;
    float u_sample;
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

// The row that is summed or drawn from, r after some rejections at a node.  It is
// read in 16-byte groups of 4 entries; a row begins anywhere (an odd vocabulary),
// so group g holds entries 4g - off .. 4g - off + 3.
struct VerifyRow {
    const float *p, *d;          // d: NULL without draft rows, or where none is needed
    double c;                    // r = max(p - c d, 0)
    const int* gone;             // without draft rows: the tokens turned down
    int n_gone, off, vocab;

    // Starts copying this lane's group g of both rows to `to` (the ends of a row entry by entry).
    __device__ __forceinline__ void fetch(int g, float4* to) const {
        const int i = 4 * g - off;
        if (i >= 0 && i + 3 < vocab) {
            cp_async_16(to, p + i);
            if (d != nullptr) cp_async_16(to + 32, d + i);
            return;
        }
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool in = i + e >= 0 && i + e < vocab;
            v[e] = in ? __ldg(p + i + e) : 0.f;
            v[4 + e] = in && d != nullptr ? __ldg(d + i + e) : 0.f;
        }
        to[0] = make_float4(v[0], v[1], v[2], v[3]);
        to[32] = make_float4(v[4], v[5], v[6], v[7]);
    }
    // The warp's groups [lo, hi), 32 at a time in order, through this lane's ring: f(group, p, d) until it says stop.
    // Without kClean they come as they are.
    template <bool kClean, class F>
    __device__ __forceinline__ void stream(int lo, int hi, int lane, float4* ring, F&& f) const {
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int s = 0; s < kVerRing; ++s) {
            const int g = lo + 32 * s + lane;
            if (g < hi) fetch(g, ring + 64 * s);
            cp_async_commit();
        }
        int at = 0;
        for (int g0 = lo; g0 < hi; g0 += 32) {
            cp_async_wait_group<kVerRing - 1>();
            const int g = g0 + lane;
            float4 pv = g < hi ? ring[64 * at] : zero;
            float4 dv = g < hi && d != nullptr ? ring[64 * at + 32] : zero;
            if (g + 32 * kVerRing < hi) fetch(g + 32 * kVerRing, ring + 64 * at);
            cp_async_commit();
            at = at + 1 == kVerRing ? 0 : at + 1;
            if (kClean) settle(g0, lane, pv, dv);
            if (f(g, pv, dv)) break;
        }
        cp_async_wait_all();
    }
    // r of an entry, times 2^-896, before it is cut at 0
    __device__ __forceinline__ double raw(float pv, float dv) const { return fma(-c, ver_wide(dv), ver_wide(pv)); }
    __device__ __forceinline__ double left(float pv, float dv) const {
        const double y = raw(pv, dv);
        return y > 0.0 ? y : 0.0;
    }
    // 0 for what is no positive finite number, and for tokens turned down
    __device__ __forceinline__ void settle(int g0, int lane, float4& pv, float4& dv) const {
        if (__any_sync(0xFFFFFFFFu, max(top(pv), top(dv)) > 0x7F7FFFFFu)) {   // a sign, an infinity or NaN
            pv = sound(pv);
            dv = sound(dv);
        }
        for (int j = 0; j < n_gone; j += 32) {
            const int e = j + lane < n_gone ? gone[j + lane] + off - 4 * g0 : -1;
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
    __shared__ VerifyIn s_in;
    __shared__ int s_path[kMaxTree];
    __shared__ int s_gone[kMaxTree];               // without draft rows: tokens turned down at this node
    __shared__ VerifyCmd s_cmd;
    __shared__ double s_part[2][kVerMaxCluster];   // the CTAs' sums of a pass, two passes deep
    extern __shared__ float4 s_rings[];
    __shared__ double s_warp[kVerWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = static_cast<int>(cl.block_rank());
    const int cta = static_cast<int>(cl.num_blocks());
    const int b = static_cast<int>(blockIdx.x) / cta;
    const int T = a.T;
    const bool has_draft = a.draft != nullptr;
    const long long row0 = static_cast<long long>(b) * T;
    // (a peer's shared memory may be written once that peer runs: its arrival here says so)
    auto started = cl.barrier_arrive();
    int n = 0;
    if (rank == 0) {
        int par = -1, x = -1;
        if (tid < T) {                             // (in flight together with the count)
            par = a.parent[row0 + tid];
            x = a.tokens[row0 + tid];
            s_in.kids[tid][0] = s_in.kids[tid][1] = 0u;
        }
        n = a.n_nodes != nullptr ? a.n_nodes[b] : T;
        if (n < 0 || n > T) {
            if (tid == 0) raise_dev_error(OASIS_DEVERR_ID_RANGE);
            n = n < 0 ? 0 : T;
        }
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
                atomicOr(&s_in.kids[par][j >> 5], 1u << (j & 31));
            }
            s_in.token[j] = x;
            s_in.p[j] = pj;
            s_in.d[j] = dj;
            s_in.u[j] = a.u_accept[row0 + j];
        }
        if (tid == 0) {
            s_in.n = n;
            s_in.u_sample = a.u_sample[b];
        }
        __syncthreads();
    }
    cl.barrier_wait(std::move(started));
    if (rank == 0) {
        constexpr int kWords = sizeof(VerifyIn) / 4;
        for (int i = tid; i < kWords * (cta - 1); i += kVerThreads) {
            const int w = i % kWords;
            reinterpret_cast<uint32_t*>(cl.map_shared_rank(&s_in, 1 + i / kWords))[w] = reinterpret_cast<const uint32_t*>(&s_in)[w];
        }
    }
    cl.sync();
    n = s_in.n;

    // the walk (thread 0): current node, its children not tested yet, S and the sum of the S before
    int cur = 0, count = 1, rounds = 0;
    uint64_t kids = 0;
    double S = 1.0, c_off = 0.0;
    if (tid == 0) {
        kids = s_in.kids[0][0] | (static_cast<uint64_t>(s_in.kids[0][1]) << 32);
        s_path[0] = 0;
    }
    double total = 0.0, before = 0.0;              // (times 2^-896)
    int slot = 0;
    VerifyRow row;
    row.gone = s_gone;
    row.vocab = a.vocab;
    float4* const ring = s_rings + warp * 64 * kVerRing + lane;   // [stage][row][lane]
    int w_lo = 0, w_hi = 0;                        // the groups that this warp sums
    while (true) {
        if (tid == 0) {
            VerifyCmd c;
            c.last = 1;
            while (kids != 0) {
                const int j = __ffsll(static_cast<long long>(kids)) - 1;
                kids &= kids - 1;
                double p = ver_clean(s_in.p[j]), dq = 1.0;
                if (has_draft) {
                    dq = ver_clean(s_in.d[j]);
                    p = fma(-c_off, dq, p);
                } else {
                    for (int i = 0; i < rounds; ++i)
                        if (s_gone[i] == s_in.token[j]) p = 0.0;
                }
                if (p > 0.0 && static_cast<double>(s_in.u[j]) * S * dq < p) {
                    s_path[count++] = j;
                    cur = j;
                    kids = s_in.kids[j][0] | (static_cast<uint64_t>(s_in.kids[j][1]) << 32);
                    rounds = 0;
                    S = 1.0;
                    c_off = 0.0;
                    continue;
                }
                if (!has_draft) {
                    s_gone[rounds++] = s_in.token[j];
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
            c.count = count;
            c.c = c_off;
            s_cmd = c;
        }
        __syncthreads();
        const VerifyCmd c = s_cmd;
        row.c = c.c;
        row.n_gone = has_draft ? 0 : c.rounds;
        const long long at = (row0 + c.cur) * a.row_stride;
        row.p = a.probs + at;
        row.d = c.c != 0.0 ? a.draft + at : nullptr;
        row.off = static_cast<int>(at & 3);
        // in order over CTAs and warps
        const int groups = (a.vocab + row.off + 3) / 4;
        const int per_cta = (groups + cta - 1) / cta;
        const int c_lo = min(groups, rank * per_cta), c_hi = min(groups, c_lo + per_cta);
        const int per_warp = (c_hi - c_lo + kVerWarps - 1) / kVerWarps;
        w_lo = min(c_hi, c_lo + warp * per_warp);
        w_hi = min(c_hi, w_lo + per_warp);
        for (int again = 0;; ++again) {
            double sum[4];
            uint32_t most = 0;
            auto add = [&](int, const float4& pv, const float4& dv) {
                most = max(most, max(VerifyRow::top(pv), VerifyRow::top(dv)));
                ver_add(sum[0], row.raw(pv.x, dv.x));
                ver_add(sum[1], row.raw(pv.y, dv.y));
                ver_add(sum[2], row.raw(pv.z, dv.z));
                ver_add(sum[3], row.raw(pv.w, dv.w));
                return false;
            };
            sum[0] = sum[1] = sum[2] = sum[3] = 0.0;
            if (row.n_gone == 0) row.stream<false>(w_lo, w_hi, lane, ring, add);
            // entries that are no positive finite numbers were taken for large ones: once more, looking at each
            if (row.n_gone != 0 || __any_sync(0xFFFFFFFFu, most > 0x7F7FFFFFu)) {
                sum[0] = sum[1] = sum[2] = sum[3] = 0.0;
                row.stream<true>(w_lo, w_hi, lane, ring, add);
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
            row.d = nullptr;
            row.n_gone = 0;
            slot ^= 1;
        }
        if (c.last) break;
        S = total * kVerScale;
        slot ^= 1;
    }
    // No CTA touches another's shared memory from here on, so each may leave.

    if (rank == 0) {
        const int steps = n > 0 ? s_cmd.count : 0;
        if (tid < T) a.path[row0 + tid] = tid < steps ? s_path[tid] : -1;
        if (tid == 0) {
            a.n_accept[b] = steps;
            if (n == 0 || !(total > 0.0)) a.next_token[b] = -1;
        }
    }
    if (n == 0 || !(total > 0.0)) return;
    // The draw.  Every CTA holds the same sums, so they agree on the one
    // that holds the crossing; sums are carried on in the same order level by
    // level, and a crossing that rounding hides from the last level is at the
    // last entry with mass.
    const double t = fmax(static_cast<double>(s_in.u_sample), 0.0) * total;
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
    row.stream<true>(w_lo, w_hi, lane, ring, [&](int g, const float4& pv, const float4& dv) {
        const double x[4] = {row.left(pv.x, dv.x), row.left(pv.y, dv.y), row.left(pv.z, dv.z), row.left(pv.w, dv.w)};
        const int i = 4 * g - row.off;
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
        return found >= 0;
    });
    if (lane == 0) a.next_token[b] = found >= 0 ? found : fallback;
}

}  // namespace oasis
