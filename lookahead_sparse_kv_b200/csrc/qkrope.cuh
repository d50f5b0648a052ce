// qkrope.cuh - projection rows to query rows and draft keys / values: per-head
// RMS norm of queries and keys and the rotation by the token's position.
//
//   y = x / sqrt(mean(x^2) + eps) * w          (no weight: y = x)
//   (y_i, y_{i+64}) -> (y_i cos a_i - y_{i+64} sin a_i, y_{i+64} cos a_i + y_i sin a_i)
//   a_i = pos * inv_freq_i, i < 64
//
// The angle of a far position has more turns than fp32 can hold beside its
// fraction (524,287 rad needs 19 bits before the point), so pos * inv_freq is
// formed and reduced to [-1, 1] half-turns in fp64 (24 + 20 bits: the product
// is exact) and only the rest goes to fp32 sine and cosine.  Norm and
// rotation are fp32; the one rounding to bf16 is the store.
//
// HBM bounds it at many tokens: every byte is read once and written once.  8
// lanes own a head's row: lane l the channels 8l..8l+7 and 64+8l..64+8l+7, so
// the rotation stays in a thread, the norm is three shuffles, and both loads
// and stores of a warp are four 128-B segments.  A warp keeps one token (its 64
// angles are made once, two a lane, and read from shared memory at each step: kept in
// registers they cost a CTA an SM) and walks the heads, 4 at a step.  16,111 tokens
// of 48 heads: 396 MB in 70 us, 5.65 TB/s; a plain copy of as many bytes takes 67 us
// (stores that stay in L2 as long as others: 73 us; CTAs of 8 warps: 71 us).
#pragma once

#include "common.cuh"
#include "summaries.cuh"

namespace oasis {

constexpr int kRopeWarps = 4;
constexpr int kRopeThreads = 32 * kRopeWarps;
constexpr int kRopeStep = 4;                       // heads a warp takes at a time

__device__ __forceinline__ uint4 f32x8_round_bf16(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

__global__ void __launch_bounds__(kRopeThreads, 10) qk_norm_rope_kernel(
    Dims d, int T, int split, const uint16_t* __restrict__ qkv, long long row_stride, const uint16_t* __restrict__ wq,
    const uint16_t* __restrict__ wk, float eps, const float* __restrict__ inv_freq, const int32_t* __restrict__ pos,
    uint16_t* __restrict__ q, uint16_t* __restrict__ k, uint16_t* __restrict__ v) {
    __shared__ float4 s_cos[kRopeWarps][16], s_sin[kRopeWarps][16];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long tokens = static_cast<long long>(d.B) * T;
    const long long w = static_cast<long long>(blockIdx.x) * kRopeWarps + warp;
    const long long tok = w / split;
    if (tok >= tokens) return;                     // whole warps leave; no CTA-wide barrier below
    const int part = static_cast<int>(w - tok * split);
    const int b = static_cast<int>(tok / T), t = static_cast<int>(tok - static_cast<long long>(b) * T);
    const int heads = d.Hq + 2 * d.Hkv;
    const int steps = (heads + kRopeStep - 1) / kRopeStep;
    const int per = (steps + split - 1) / split;
    const int sub = lane & 7, hl = lane >> 3;
    {
        const double p = static_cast<double>(pos[tok]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = lane + 32 * i;
            double turns = p * static_cast<double>(inv_freq[c]) * 0.31830988618379067154;   // half-turns
            turns -= 2.0 * rint(0.5 * turns);
            float sn, cs;
            sincospif(static_cast<float>(turns), &sn, &cs);
            reinterpret_cast<float*>(s_cos[warp])[c] = cs;
            reinterpret_cast<float*>(s_sin[warp])[c] = sn;
        }
    }
    __syncwarp();
    const bool norm = wq != nullptr || wk != nullptr;
    const uint16_t* row = qkv + tok * row_stride;
    for (int s = part * per; s < min(steps, (part + 1) * per); ++s) {
        const int hd = kRopeStep * s + hl;
        const bool on = hd < heads;
        uint4 a4 = make_uint4(0, 0, 0, 0), c4 = a4;
        if (on) {
            a4 = *reinterpret_cast<const uint4*>(row + hd * kHeadDim + 8 * sub);
            c4 = *reinterpret_cast<const uint4*>(row + hd * kHeadDim + 64 + 8 * sub);
        }
        const bool is_q = hd < d.Hq, is_v = hd >= d.Hq + d.Hkv;
        float lo[8], hi[8];
        bf16x8_to_f32(a4, lo);
        bf16x8_to_f32(c4, hi);
        const uint16_t* wt = is_q ? wq : wk;
        float ss = 0.f;
        if (norm) {
#pragma unroll
            for (int i = 0; i < 8; ++i) ss += lo[i] * lo[i] + hi[i] * hi[i];
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        }
        if (on && !is_v) {
            if (wt != nullptr) {
                const float r = rsqrtf(ss * (1.f / kHeadDim) + eps);
                float wl[8], wh[8];
                bf16x8_to_f32(*reinterpret_cast<const uint4*>(wt + 8 * sub), wl);
                bf16x8_to_f32(*reinterpret_cast<const uint4*>(wt + 64 + 8 * sub), wh);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    lo[i] *= r * wl[i];
                    hi[i] *= r * wh[i];
                }
            }
#pragma unroll
            for (int k4 = 0; k4 < 2; ++k4) {
                const float4 c = s_cos[warp][2 * sub + k4], n = s_sin[warp][2 * sub + k4];
                const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = lo[4 * k4 + i], y = hi[4 * k4 + i];
                    lo[4 * k4 + i] = x * cs[i] - y * sn[i];
                    hi[4 * k4 + i] = y * cs[i] + x * sn[i];
                }
            }
            a4 = f32x8_round_bf16(lo);
            c4 = f32x8_round_bf16(hi);
        }
        if (on) {
            uint16_t* dst;
            if (is_q)
                dst = q + (tok * d.Hq + hd) * kHeadDim;
            else {
                const int h = hd - d.Hq - (is_v ? d.Hkv : 0);
                dst = (is_v ? v : k) + ((static_cast<long long>(b) * d.Hkv + h) * T + t) * kHeadDim;
            }
            __stcs(reinterpret_cast<uint4*>(dst + 8 * sub), a4);
            __stcs(reinterpret_cast<uint4*>(dst + 64 + 8 * sub), c4);
        }
    }
}

}  // namespace oasis
