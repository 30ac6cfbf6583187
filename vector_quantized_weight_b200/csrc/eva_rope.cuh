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

// Pairs of a token's row in the tables: a multiple of 8 (the ones behind the last are not used).
__host__ __device__ __forceinline__ int rope_row(int R) { return (R / 2 + 7) & ~7; }

// cos and sin of the tokens t0 .. t0 + nt - 1, [token][rope_row] each, by the whole CTA.
__device__ __forceinline__ void rope_angles(const RopeParams &p, int t0, int nt, float *cos, float *sin) {
    const int half = p.R >> 1, row = rope_row(p.R);
    for (int i = threadIdx.x; i < nt * row; i += blockDim.x) {
        const int t = i / row, j = i - t * row;
        float s = 0.f, c = 1.f;
        if (j < half) {
            const unsigned long long a = (unsigned long long)(long long)p.pos[t0 + t] * p.turns[j];
            sincospif((float)(int32_t)(a >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns in [-1, 1)
            c *= p.magnitude;
            s *= p.magnitude;
        }
        cos[i] = c;
        sin[i] = s;
    }
}

// Two fp32 operations an instruction.
struct F2 {
    float x, y;
};
__device__ __forceinline__ unsigned long long f2_bits(F2 a) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
    return r;
}
__device__ __forceinline__ F2 f2_of(unsigned long long r) {
    F2 a;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r));
    return a;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
    return f2_of(r);
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)), "l"(f2_bits(c)));
    return f2_of(r);
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

// 16 elements of a lane as they were loaded: two chunks of 8.
template <typename T>
struct RopeRaw {
    uint4 v[sizeof(T)];                  // 2 x 16 bytes of fp16, 4 of fp32
    __device__ __forceinline__ void load(const T *a, const T *b) {
        constexpr int h = sizeof(T) / 2;
#pragma unroll
        for (int i = 0; i < h; ++i) {
            v[i] = reinterpret_cast<const uint4 *>(a)[i];
            v[h + i] = reinterpret_cast<const uint4 *>(b)[i];
        }
    }
    __device__ __forceinline__ void get(F2 (&x)[4], F2 (&y)[4]) const {
        if constexpr (sizeof(T) == 2) {
            const __half2 *e = reinterpret_cast<const __half2 *>(v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 a = __half22float2(e[i]), b = __half22float2(e[4 + i]);
                x[i] = {a.x, a.y};
                y[i] = {b.x, b.y};
            }
        } else {
            const F2 *e = reinterpret_cast<const F2 *>(v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = e[i];
                y[i] = e[4 + i];
            }
        }
    }
};

// W lanes a head (a power of two >= D/16).  Needs D a multiple of 16, R too in the
// half layout, and every pointer and stride a multiple of 16 bytes.  A lane keeps the loads of its
// next turns in flight (with one turn's, a prompt of 8192 tokens and 72 heads of
// 128 took 86 us: 24 KB an SM are too few for the memory's latency; now 62 us, 4.9
// TB/s).  What it waits for now is shared memory: a turn reads its sines and weights
// again, which keeps that path 74 % busy, with a third of the warps resident (80
// registers); issue slots and DRAM are half busy.
template <typename TI, typename TO, int W>
__global__ void __launch_bounds__(kRopeThreads, 3) eva_rope_kernel(RopeParams p) {
    constexpr int kAhead = sizeof(TI) == 2 ? 2 : 1;
    float *ws = reinterpret_cast<float *>(eva_smem);       // weight + offset (or 1) of queries and of keys
    float *cos = ws + (p.norm ? 2 * p.D : 0), *sin = cos + p.tb * rope_row(p.R);
    const int unit = threadIdx.x % W, group = threadIdx.x / W, groups = kRopeThreads / W;
    const int t0 = blockIdx.x * p.tb, nt = min(p.tb, p.T - t0), half = p.R >> 1;
    const bool live = unit * 16 < p.D, turned = unit * 16 < p.R;
    // the two chunks of this lane
    const bool split = turned && !p.interleaved;
    const int oa = split ? unit * 8 : unit * 16, ob = split ? half : 8;    // ob: from the first
    if (p.norm)
        for (int i = threadIdx.x; i < 2 * p.D; i += kRopeThreads) {
            const __half *w = i < p.D ? p.qw : p.kw;
            ws[i] = w ? __half2float(w[i < p.D ? i : i - p.D]) + p.offset : 1.f;
        }
    pdl_wait();
    pdl_launch();
    // (token, head) pairs of this CTA: heads [h0, h1) of each token
    const int h0 = blockIdx.y * p.hs, nh = min(p.hs, p.H - h0), n = nt * nh;
    const float inv_d = 1.f / (float)p.D;
    RopeRaw<TI> raw[kAhead];
    // the pair `groups` further on, without a division a turn
    struct At {
        int t, h;
    };
    const int dt = groups / nh, dh = groups - dt * nh;
    auto step = [&](At &a) {
        a.t += dt;
        a.h += dh;
        if (a.h >= nh) {
            a.h -= nh;
            ++a.t;
        }
    };
    At in = {group / nh, group % nh}, out = in;
    // this CTA's first token, head h0 (the keys' pointers count the query heads in), this lane's first chunk; within
    // the CTA offsets are 32-bit
    const int nq = p.Hq - h0, ldq = (int)p.ldq, ldk = (int)p.ldk, ldqo = (int)p.ldqo, ldko = (int)p.ldko;
    const TI *q0 = static_cast<const TI *>(p.q) + t0 * p.ldq + (h0 * p.D + oa);
    const TI *k0 = static_cast<const TI *>(p.k) + t0 * p.ldk + (oa - nq * p.D);
    TO *qo0 = static_cast<TO *>(p.qo) + t0 * p.ldqo + (h0 * p.D + oa);
    TO *ko0 = static_cast<TO *>(p.ko) + t0 * p.ldko + (oa - nq * p.D);
    auto load = [&](RopeRaw<TI> &r) {
        const bool on = in.t < nt && live, isq = in.h < nq;
        const TI *src = (isq ? q0 : k0) + (in.t * (isq ? ldq : ldk) + in.h * p.D);
        step(in);
        if (on) r.load(src, src + ob);
    };
#pragma unroll
    for (int j = 0; j < kAhead; ++j) load(raw[j]);      // in flight while the angles are computed
    rope_angles(p, t0, nt, cos, sin);
    __syncthreads();
    auto turn = [&](const RopeRaw<TI> &r) {
        const int t = out.t;
        const bool on = t < nt && live, isq = out.h < nq;
        TO *dst = (isq ? qo0 : ko0) + (t * (isq ? ldqo : ldko) + out.h * p.D);
        step(out);
        F2 a[4], b[4];
        r.get(a, b);
        if (p.norm) {
            float ss = 0.f;
            if (on) {
                F2 q = {0.f, 0.f};
#pragma unroll
                for (int j = 0; j < 4; ++j) q = f2_fma(b[j], b[j], f2_fma(a[j], a[j], q));
                ss = q.x + q.y;
            }
#pragma unroll
            for (int o = W / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, W);
            const float s = rsqrtf(ss * inv_d + p.eps);
            if (on) {
                const float *w = ws + (isq ? oa : p.D + oa);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float4 wa = reinterpret_cast<const float4 *>(w)[j], wb = reinterpret_cast<const float4 *>(w + ob)[j];
                    a[2 * j] = f2_mul(f2_mul(a[2 * j], {s, s}), {wa.x, wa.y});
                    a[2 * j + 1] = f2_mul(f2_mul(a[2 * j + 1], {s, s}), {wa.z, wa.w});
                    b[2 * j] = f2_mul(f2_mul(b[2 * j], {s, s}), {wb.x, wb.y});
                    b[2 * j + 1] = f2_mul(f2_mul(b[2 * j + 1], {s, s}), {wb.z, wb.w});
                }
            }
        }
        if (!on) return;
        if (turned) {
            const int at = t * rope_row(p.R) + unit * 8;
            const float4 *cr = reinterpret_cast<const float4 *>(cos + at), *sr = reinterpret_cast<const float4 *>(sin + at);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float4 c = cr[j], n = sr[j];
                if (!p.interleaved) {
                    const F2 c0 = {c.x, c.y}, c1 = {c.z, c.w}, s0 = {n.x, n.y}, s1 = {n.z, n.w};
                    const F2 x0 = a[2 * j], x1 = a[2 * j + 1], y0 = b[2 * j], y1 = b[2 * j + 1];
                    a[2 * j] = f2_fma(y0, {-s0.x, -s0.y}, f2_mul(x0, c0));
                    a[2 * j + 1] = f2_fma(y1, {-s1.x, -s1.y}, f2_mul(x1, c1));
                    b[2 * j] = f2_fma(x0, s0, f2_mul(y0, c0));
                    b[2 * j + 1] = f2_fma(x1, s1, f2_mul(y1, c1));
                } else {                  // four pairs of a, then four of b
                    F2 *v = j ? b : a;
                    const float cc[4] = {c.x, c.y, c.z, c.w}, nn[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        // (pairs behind the last turned one are copies: a product with 0 would carry an infinity over)
                        const F2 x = v[i];
                        if (unit * 8 + 4 * j + i < half) v[i] = f2_fma({x.y, x.x}, {-nn[i], nn[i]}, f2_mul(x, {cc[i], cc[i]}));
                    }
                }
            }
        }
        rope_store8(dst, reinterpret_cast<const float(&)[8]>(a));
        rope_store8(dst + ob, reinterpret_cast<const float(&)[8]>(b));
    };
    // every group takes the same number of turns, so the shuffles see whole warps
    for (int i = 0; i < n; i += kAhead * groups) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (i + j * groups >= n) break;
            const RopeRaw<TI> r = raw[j];
            load(raw[j]);
            turn(r);
        }
    }
}

template <typename TI, typename TO>
__global__ void __launch_bounds__(kRopeThreads) eva_rope_any_kernel(RopeParams p) {
    float *cos = reinterpret_cast<float *>(eva_smem), *sin = cos + p.tb * rope_row(p.R);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t0 = blockIdx.x * p.tb, nt = min(p.tb, p.T - t0), half = p.R >> 1;
    pdl_wait();
    pdl_launch();
    rope_angles(p, t0, nt, cos, sin);
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
            const float2 c = make_float2(cos[t * rope_row(p.R) + j], sin[t * rope_row(p.R) + j]);
            const float xa = scaled(ja), xb = scaled(jb);
            dst[ja] = (TO)(xa * c.x - xb * c.y);
            dst[jb] = (TO)(xb * c.x + xa * c.y);
        }
        for (int j = p.R + lane; j < p.D; j += 32) dst[j] = (TO)scaled(j);
    }
}

}  // namespace eva
