// eva_rope.cuh -- rotary positions of a step's queries and keys, with the
// per-head RMS norm in the same pass.
//
//   y = x / sqrt(mean(x^2) + eps) * (w + offset)              (with the norm)
//   (a, b) -> (a cos - b sin, b cos + a sin),  angle = position * f_i
//
// for the pairs (i, i + R/2) (half layout) or (2i, 2i + 1) (interleaved) of the
// first R dimensions of a head; the others pass through.
//
// Angles.  f_i is kept as a fraction of a turn in 64-bit fixed point (2^64 =
// one turn), so position * f_i wraps exactly for every 32-bit position; its
// top 32 bits go through sincospi.  The error is the table's half step times
// the position (2^-34 turns at position 2^30) plus the fp32 rounding of the
// reduced angle (2^-24 of half a turn): far positions lose nothing.
//
// What bounds it: bytes.  Every element is read and written once; the sines
// of a token are computed once per CTA (one per thread and pair) and shared
// through shared memory by all its heads.
//
//  eva_rope_kernel        16-byte accesses: a lane owns 16 dimensions of a head
//                         (the two 8-element chunks of its pairs), D/16 lanes a head
//  eva_rope_any_kernel    any head size, rotary size, stride and alignment: one warp
//                         a head, one element an access
#pragma once
#include <cuda_fp16.h>
#include <stdint.h>

#include "eva_vq_kernels.cuh"

namespace eva {

constexpr int kRopeThreads = 256;

struct RopeParams {
    const void *q, *k;
    void *qo, *ko;
    long long ldq, ldk, ldqo, ldko;       // elements from one token to the next
    const int32_t *pos;
    const unsigned long long *turns;      // [R/2] turns a position, 2^64 = one turn
    const __half *qw, *kw;                // norm weights [D]; null: every dimension times 1
    int T, Hq, H, D, R;                   // H = query heads + key heads
    int interleaved, norm;
    int tb, hs;                           // tokens and heads a CTA
    float eps, offset, magnitude;
};

// cos and sin of the tokens t0 .. t0 + nt - 1, [token][pair], by the whole CTA.
__device__ __forceinline__ void rope_angles(const RopeParams &p, int t0, int nt, float2 *cs) {
    const int half = p.R >> 1;
    for (int i = threadIdx.x; i < nt * half; i += blockDim.x) {
        const int t = i / half, j = i - t * half;
        const unsigned long long a = (unsigned long long)(long long)p.pos[t0 + t] * p.turns[j];
        float s, c;
        sincospif((float)(int32_t)(a >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns in [-1, 1)
        cs[i] = make_float2(c * p.magnitude, s * p.magnitude);
    }
}

template <typename T>
__device__ __forceinline__ void rope_load8(const T *p, float (&v)[8]);
template <>
__device__ __forceinline__ void rope_load8<__half>(const __half *p, float (&v)[8]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
template <>
__device__ __forceinline__ void rope_load8<float>(const float *p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void rope_store8(__half *p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void rope_store8(float *p, const float (&v)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// W lanes a head (a power of two >= D/16).  Needs D and R multiples of 16, and
// every pointer and stride a multiple of 16 bytes.
template <typename TI, typename TO, int W>
__global__ void __launch_bounds__(kRopeThreads) eva_rope_kernel(RopeParams p) {
    float2 *cs = reinterpret_cast<float2 *>(eva_smem);
    const int unit = threadIdx.x % W, group = threadIdx.x / W, groups = kRopeThreads / W;
    const int t0 = blockIdx.x * p.tb, nt = min(p.tb, p.T - t0), half = p.R >> 1;
    const bool live = unit * 16 < p.D, turned = unit * 16 < p.R;
    // the two chunks of this lane
    const bool split = turned && !p.interleaved;
    const int oa = split ? unit * 8 : unit * 16, ob = split ? half + unit * 8 : oa + 8;
    pdl_wait();
    pdl_launch();
    float wq[2][8], wk[2][8];            // weight + offset, or 1
    if (p.norm && live) {
#pragma unroll
        for (int i = 0; i < 8; ++i) wq[0][i] = wq[1][i] = wk[0][i] = wk[1][i] = 1.f;
        if (p.qw) { rope_load8(p.qw + oa, wq[0]); rope_load8(p.qw + ob, wq[1]); }
        if (p.kw) { rope_load8(p.kw + oa, wk[0]); rope_load8(p.kw + ob, wk[1]); }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (p.qw) { wq[0][i] += p.offset; wq[1][i] += p.offset; }
            if (p.kw) { wk[0][i] += p.offset; wk[1][i] += p.offset; }
        }
    }
    // (token, head) pairs of this CTA: heads [h0, h1) of each token
    const int h0 = blockIdx.y * p.hs, nh = min(p.hs, p.H - h0);
    float a[8], b[8];
    auto load = [&](int i) {
        const int t = t0 + i / nh, h = h0 + i % nh;
        const TI *src = h < p.Hq ? static_cast<const TI *>(p.q) + t * p.ldq + (long long)h * p.D
                                 : static_cast<const TI *>(p.k) + t * p.ldk + (long long)(h - p.Hq) * p.D;
        if (live) {
            rope_load8(src + oa, a);
            rope_load8(src + ob, b);
        }
    };
    const int n = nt * nh;
    if (group < n) load(group);          // in flight while the angles are computed
    rope_angles(p, t0, nt, cs);
    __syncthreads();
    // every group takes the same number of turns, so the shuffles see whole warps
    for (int i = group, first = 1; i - group < n; i += groups, first = 0) {
        const bool on = i < n && live;
        if (!first && i < n) load(i);
        const int t = i / nh, h = h0 + i % nh;
        if (p.norm) {
            float ss = 0.f;
            if (on) {
#pragma unroll
                for (int j = 0; j < 8; ++j) ss += a[j] * a[j] + b[j] * b[j];
            }
#pragma unroll
            for (int o = W / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, W);
            const float r = rsqrtf(ss / (float)p.D + p.eps);
            const bool isq = h < p.Hq;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                a[j] *= r * (isq ? wq[0][j] : wk[0][j]);
                b[j] *= r * (isq ? wq[1][j] : wk[1][j]);
            }
        }
        if (!on) continue;
        if (turned) {
            const float4 *row = reinterpret_cast<const float4 *>(cs + t * half + unit * 8);
            if (!p.interleaved) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 c = row[j];
                    const float a0 = a[2 * j], a1 = a[2 * j + 1];
                    a[2 * j] = a0 * c.x - b[2 * j] * c.y;
                    b[2 * j] = b[2 * j] * c.x + a0 * c.y;
                    a[2 * j + 1] = a1 * c.z - b[2 * j + 1] * c.w;
                    b[2 * j + 1] = b[2 * j + 1] * c.z + a1 * c.w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {     // pairs of a, then pairs of b
                    const float4 c = row[j >> 1], d = row[2 + (j >> 1)];
                    const float ca = j & 1 ? c.z : c.x, sa = j & 1 ? c.w : c.y;
                    const float cb = j & 1 ? d.z : d.x, sb = j & 1 ? d.w : d.y;
                    const float a0 = a[2 * j], b0 = b[2 * j];
                    a[2 * j] = a0 * ca - a[2 * j + 1] * sa;
                    a[2 * j + 1] = a[2 * j + 1] * ca + a0 * sa;
                    b[2 * j] = b0 * cb - b[2 * j + 1] * sb;
                    b[2 * j + 1] = b[2 * j + 1] * cb + b0 * sb;
                }
            }
        }
        TO *dst = h < p.Hq ? static_cast<TO *>(p.qo) + (t0 + t) * p.ldqo + (long long)h * p.D
                           : static_cast<TO *>(p.ko) + (t0 + t) * p.ldko + (long long)(h - p.Hq) * p.D;
        rope_store8(dst + oa, a);
        rope_store8(dst + ob, b);
    }
}

template <typename TI, typename TO>
__global__ void __launch_bounds__(kRopeThreads) eva_rope_any_kernel(RopeParams p) {
    float2 *cs = reinterpret_cast<float2 *>(eva_smem);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t0 = blockIdx.x * p.tb, nt = min(p.tb, p.T - t0), half = p.R >> 1;
    pdl_wait();
    pdl_launch();
    rope_angles(p, t0, nt, cs);
    __syncthreads();
    const int h0 = blockIdx.y * p.hs, nh = min(p.hs, p.H - h0);
    for (int i = warp; i < nt * nh; i += kRopeThreads / 32) {
        const int t = i / nh, h = h0 + i % nh;
        const bool isq = h < p.Hq;
        const int hh = isq ? h : h - p.Hq;
        const TI *src = static_cast<const TI *>(isq ? p.q : p.k) + (t0 + t) * (isq ? p.ldq : p.ldk) + (long long)hh * p.D;
        TO *dst = static_cast<TO *>(isq ? p.qo : p.ko) + (t0 + t) * (isq ? p.ldqo : p.ldko) + (long long)hh * p.D;
        const __half *w = isq ? p.qw : p.kw;
        float r = 1.f;
        if (p.norm) {
            float ss = 0.f;
            for (int j = lane; j < p.D; j += 32) {
                const float x = (float)src[j];
                ss += x * x;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            r = rsqrtf(ss / (float)p.D + p.eps);
        }
        auto scaled = [&](int j) {
            float x = (float)src[j];
            if (p.norm) x *= r * (w ? __half2float(w[j]) + p.offset : 1.f);
            return x;
        };
        for (int j = lane; j < half; j += 32) {
            const int ja = p.interleaved ? 2 * j : j, jb = p.interleaved ? 2 * j + 1 : j + half;
            const float2 c = cs[t * half + j];
            const float xa = scaled(ja), xb = scaled(jb);
            dst[ja] = (TO)(xa * c.x - xb * c.y);
            dst[jb] = (TO)(xb * c.x + xa * c.y);
        }
        for (int j = p.R + lane; j < p.D; j += 32) dst[j] = (TO)scaled(j);
    }
}

}  // namespace eva
