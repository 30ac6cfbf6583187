// eva_kv.cuh -- the paged 8-bit cache of keys and values: writing new tokens
// and reading tokens back.
//
// A page holds `page` tokens of every key head; a (page, head) tile is
// [page][D] codes and one fp32 scale, for keys and for values:
//   int8   scale = amax / 127,  code = rint(x / scale)
//   e4m3   scale = amax / 448,  code = e4m3(x / scale)   (nearest, ties to even)
// both quotients IEEE fp32.  Writing into a page whose earlier slots are kept
// takes scale' = max(scale, amax of the new tokens / 127 or 448); where that
// grows, the kept codes become round(code * (scale / scale')).  Writing slot 0
// starts the page anew.  Inputs are clamped to +-65504 and a NaN counts as 0,
// so no code is ever NaN.
//
// What bounds them: a decode step is a chain of dependent lookups (lengths, page,
// scale: 11 us for both at 64 sequences).  A prompt (3 x 2100 tokens of 8 heads of
// 128: 30 us for both; 36 with a division an element) writes at the quantizer's
// instructions, 30 an element (issue slots 71 % busy while CTAs are there), and reads
// back at the latency of one load of codes a lane at a time (DRAM 11 %, issue 32 %).
//
//  eva_kv_append_kernel  one CTA per (sequence's page, head, keys or values)
//  eva_kv_read_kernel    one warp per token (or 8 of them), keys or values
#pragma once
#include <cuda_fp16.h>
#include <stdint.h>

#include "eva_rope.cuh"

namespace eva {

constexpr int kKvThreads = 128;
constexpr int kKvStatusIndex = 8;      // status bit: an index on the device was out of range

// Where the tokens of a call lie: rows starts[b] .. starts[b+1] - 1 of the
// packed inputs belong to sequence b; lens[b] is its length with them.
struct KvTokens {
    const int32_t *starts, *lens, *table;
    int B, T, page, log_page, max_pages, num_pages;
};

// Rows of sequence b and its length; a sequence whose numbers cannot be right
// has no rows (and sets `bad`).
struct KvSeq {
    int row, n, len;
};
__device__ __forceinline__ KvSeq kv_seq(const KvTokens &k, int b, bool &bad) {
    KvSeq s;
    s.row = k.starts[b];
    const int end = k.starts[b + 1];
    s.len = k.lens[b];
    s.n = end - s.row;
    if (s.row < 0 || s.n < 0 || end > k.T || s.len < 0 || s.len > k.max_pages * (long long)k.page) {
        bad = true;
        s.n = 0;
    }
    return s;
}

template <bool E4M3>
struct KvCode;
template <>
struct KvCode<false> {
    static constexpr float kLargest = 127.f;
    static __device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
        const int w = (__float2int_rn(fminf(fmaxf(a, -127.f), 127.f)) & 255) |
                      (__float2int_rn(fminf(fmaxf(b, -127.f), 127.f)) & 255) << 8 |
                      (__float2int_rn(fminf(fmaxf(c, -127.f), 127.f)) & 255) << 16 |
                      __float2int_rn(fminf(fmaxf(d, -127.f), 127.f)) << 24;
        return (uint32_t)w;
    }
    static __device__ __forceinline__ void unpack4(uint32_t w, float (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i)      // 2^23 + 128 + code, exactly
            v[i] = __uint_as_float(__byte_perm(w ^ 0x80808080u, 0x4b000000u, 0x7440 + i)) - 8388736.f;
    }
};
template <>
struct KvCode<true> {
    static constexpr float kLargest = 448.f;
    static __device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
        uint16_t lo, hi;       // the first source lands in the upper byte
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
        return (uint32_t)lo | (uint32_t)hi << 16;
    }
    static __device__ __forceinline__ void unpack4(uint32_t w, float (&v)[4]) {
        uint32_t lo, hi;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)w));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(w >> 16)));
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
        const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
        v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
    }
};

struct KvAppendParams {
    KvTokens tok;
    const void *x[2];                    // keys, values: [T][H][D], ld elements a token
    long long ld[2];
    uint8_t *pages[2];
    float *scale[2];
    int H, D, log_d;
    int *status;
};

// Eight elements as they were loaded.  clean() makes them finite (+-65504 at
// most, 0 for a NaN), in a few integer instructions where they are already,
// and returns the largest magnitude.
template <typename T>
struct KvRaw;
template <>
struct KvRaw<__half> {
    uint4 v;
    __device__ __forceinline__ void load(const __half *p) { v = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ float clean() {
        uint32_t *w = &v.x, odd = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) odd |= ((w[i] & 0x7fff7fffu) + 0x04000400u) & 0x80008000u;    // exponent 31
        if (odd) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int s = 0; s < 32; s += 16) {
                    const uint32_t e = (w[i] >> s) & 0x7fffu;
                    if (e > 0x7c00u) w[i] &= ~(0xffffu << s);
                    if (e == 0x7c00u) w[i] -= 1u << s;
                }
        }
        __half2 m = __float2half2_rn(0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) m = __hmax2(m, __habs2(*reinterpret_cast<const __half2 *>(&w[i])));
        return fmaxf(__low2float(m), __high2float(m));
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const __half2 *h = reinterpret_cast<const __half2 *>(&v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(h[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
};
template <>
struct KvRaw<float> {
    float4 v[2];
    __device__ __forceinline__ void load(const float *p) {
        v[0] = reinterpret_cast<const float4 *>(p)[0];
        v[1] = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ float clean() {
        float *x = &v[0].x, m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = x[i] == x[i] ? fminf(fmaxf(x[i], -65504.f), 65504.f) : 0.f;
            m = fmaxf(m, fabsf(x[i]));
        }
        return m;
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const float *e = &v[0].x;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = e[i];
    }
};

// Four codes of x / scale, rounded from the IEEE quotient.  A product with the
// reciprocal is within 2^-22 of it, so it rounds to the same code unless it
// lies that near to a border between two codes; then, and only then, `sure`
// becomes false (one element in some thousands) and the caller divides.
template <bool E4M3>
__device__ __forceinline__ uint32_t kv_codes(const float *x, float inv, bool &sure) {
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = x[i] * inv;
    if constexpr (E4M3) {
        // borders: half way between neighbours, three fraction bits apart (below 2^-6 every code has the same step:
        // left to the division)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t tail = (__float_as_uint(q[i]) & 0xfffffu) - 0x7fff8u;
            if (tail <= 16u || (fabsf(q[i]) < 0.015626f && q[i] != 0.f)) sure = false;
        }
        return KvCode<true>::pack4(q[0], q[1], q[2], q[3]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float t = q[i] + 12582912.f;                 // 1.5 * 2^23: the integer lies in the low bits
            if (fabsf(q[i] - (t - 12582912.f)) > 0.4999f) sure = false;
            w[i] = __float_as_uint(t);
        }
        return __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
    }
}

// The unit-th page that the call writes, counting through the sequences; every
// lane gets the answer.  Tokens before position 0 (a length below the row
// count) are dropped.
struct KvUnit {
    int b, row, lo, hi, page_index;      // rows from `row` on go to slots [lo, hi)
};
__device__ __forceinline__ bool kv_find_unit(const KvTokens &k, int unit, KvUnit &u, bool &bad) {
    const int lane = threadIdx.x & 31;
    int before = 0;
    for (int b0 = 0; b0 < k.B; b0 += 32) {
        const int b = b0 + lane;
        int count = 0, first = 0, begin = 0, end = 0, row = 0;
        if (b < k.B) {
            const KvSeq s = kv_seq(k, b, bad);
            end = s.len;
            begin = max(0, s.len - s.n);
            row = s.row + s.n - (end - begin);
            if (s.n > 0 && end > begin) {
                first = begin >> k.log_page;
                count = ((end - 1) >> k.log_page) - first + 1;
            }
        }
        int sum = count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        const bool mine = unit < before + sum && unit >= before + sum - count;
        const unsigned who = __ballot_sync(0xffffffffu, mine);
        if (who) {
            const int src = __ffs(who) - 1;
            const int idx = unit - (before + sum - count) + first;
            u.page_index = __shfl_sync(0xffffffffu, idx, src);
            begin = __shfl_sync(0xffffffffu, begin, src);
            end = __shfl_sync(0xffffffffu, end, src);
            row = __shfl_sync(0xffffffffu, row, src);
            u.b = b0 + src;
            const int p0 = u.page_index * k.page;
            u.lo = max(begin, p0) - p0;
            u.hi = min(end, p0 + k.page) - p0;
            u.row = row + p0 + u.lo - begin;
            return true;
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
    }
    return false;
}

template <typename TI, bool E4M3>
__global__ void __launch_bounds__(kKvThreads) eva_kv_append_kernel(KvAppendParams p) {
    __shared__ float red[kKvThreads / 32];
    pdl_wait();
    pdl_launch();
    bool bad = false;
    KvUnit u;
    const bool found = kv_find_unit(p.tok, blockIdx.x, u, bad);
    if (bad) atomicOr(p.status, kKvStatusIndex);
    if (!found) return;
    const int h = blockIdx.y, kv = blockIdx.z, D = p.D, tid = threadIdx.x;
    const int log_per = p.log_d - 3, chunks = (u.hi - u.lo) << log_per;          // 8 elements a chunk
    const long long ld = kv ? p.ld[1] : p.ld[0];
    const TI *src = static_cast<const TI *>(kv ? p.x[1] : p.x[0]) + u.row * ld + (long long)h * D;
    // The first chunks of a thread stay in registers between the two passes; they are on their way while the page and
    // its scale are looked up.
    constexpr int kKeep = sizeof(TI) == 2 ? 8 : 4;
    KvRaw<TI> keep[kKeep];
    float amax = 0.f;
    auto load = [&](int c, KvRaw<TI> &r) {
        const int t = c >> log_per;
        r.load(src + t * ld + (c - (t << log_per)) * 8);
    };
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
        if (tid + i * kKvThreads < chunks) load(tid + i * kKvThreads, keep[i]);
    const int page = p.tok.table[(long long)u.b * p.tok.max_pages + u.page_index];
    if (page < 0 || page >= p.tok.num_pages) {
        if (threadIdx.x == 0) atomicOr(p.status, kKvStatusIndex);
        return;
    }
    const long long tile = (long long)page * p.H + h;
    uint8_t *dst = (kv ? p.pages[1] : p.pages[0]) + tile * p.tok.page * D;
    float *scale = (kv ? p.scale[1] : p.scale[0]) + tile;
    const float was = u.lo > 0 ? *scale : 0.f;
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
        if (tid + i * kKvThreads < chunks) amax = fmaxf(amax, keep[i].clean());
    for (int c = tid + kKeep * kKvThreads; c < chunks; c += kKvThreads) {
        KvRaw<TI> r;
        load(c, r);
        amax = fmaxf(amax, r.clean());
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((tid & 31) == 0) red[tid >> 5] = amax;
    __syncthreads();                     // also: every thread has read the old scale
#pragma unroll
    for (int w = 0; w < kKvThreads / 32; ++w) amax = fmaxf(amax, red[w]);
    const float now = fmaxf(was, __fdiv_rn(amax, KvCode<E4M3>::kLargest));
    if (tid == 0) *scale = now;
    if (u.lo > 0 && was < now) {         // the kept codes in units of the new scale
        const float ratio = __fdiv_rn(was, now);
        for (int i = tid; i < u.lo * D / 16; i += kKvThreads) {
            uint4 w = reinterpret_cast<uint4 *>(dst)[i];
            uint32_t *ws = &w.x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float v[4];
                KvCode<E4M3>::unpack4(ws[j], v);
                ws[j] = KvCode<E4M3>::pack4(v[0] * ratio, v[1] * ratio, v[2] * ratio, v[3] * ratio);
            }
            reinterpret_cast<uint4 *>(dst)[i] = w;
        }
    }
    const float inv = now > 0.f ? __fdiv_rn(1.f, now) : 0.f;
    const bool usual = now > 1e-30f;     // the reciprocal is a normal number
    auto store = [&](int c, const KvRaw<TI> &r) {
        float x[8];
        r.get(x);
        bool sure = usual;
        uint2 w;
        w.x = kv_codes<E4M3>(x, inv, sure);
        w.y = kv_codes<E4M3>(x + 4, inv, sure);
        if (!sure) {
            float q[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] = now > 0.f ? __fdiv_rn(x[j], now) : 0.f;
            w.x = KvCode<E4M3>::pack4(q[0], q[1], q[2], q[3]);
            w.y = KvCode<E4M3>::pack4(q[4], q[5], q[6], q[7]);
        }
        *reinterpret_cast<uint2 *>(dst + (long long)u.lo * D + c * 8) = w;
    };
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
        const int c = tid + i * kKvThreads;
        if (c < chunks) store(c, keep[i]);
    }
    for (int c = tid + kKeep * kKvThreads; c < chunks; c += kKvThreads) {
        KvRaw<TI> r;
        load(c, r);
        r.clean();
        store(c, r);
    }
}

struct KvReadParams {
    KvTokens tok;                        // starts: rows of the outputs; lens: first position of each sequence
    const uint8_t *pages[2];
    const float *scale[2];
    void *out[2];                        // [T][H][D], contiguous; either may be null
    int H, D, log_d, rows;               // rows: of a warp, at most 8
    int *status;
};

template <typename TO, bool E4M3>
__global__ void __launch_bounds__(kKvThreads) eva_kv_read_kernel(KvReadParams p) {
    const int lane = threadIdx.x & 31, kv = blockIdx.y;
    const int row0 = (blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5)) * p.rows;
    pdl_wait();
    pdl_launch();
    void *dst = kv ? p.out[1] : p.out[0];
    if (row0 >= p.tok.T || !dst) return;
    // Lane r looks up row r of the warp: the sequence whose range has it, if any.  A range that goes backwards or leaves
    // the T rows has none.
    const int row = row0 + lane;
    const bool mine = lane < p.rows && row < p.tok.T;
    int b = -1, first = 0;
    bool bad = false;
    for (int b0 = 0; b0 < p.tok.B; b0 += 32) {
        int lo = 0, hi = 0;
        if (b0 + lane < p.tok.B) {
            lo = p.tok.starts[b0 + lane];
            hi = p.tok.starts[b0 + lane + 1];
            if (lo < 0 || hi < lo || hi > p.tok.T) {
                bad = true;
                hi = lo;
            }
        }
        for (int r = 0; r < p.rows; ++r) {
            const unsigned who = __ballot_sync(0xffffffffu, lo <= row0 + r && row0 + r < hi);
            const int src = who ? __ffs(who) - 1 : 0, at = __shfl_sync(0xffffffffu, lo, src);
            if (lane == r && who && b < 0) {
                b = b0 + src;
                first = at;
            }
        }
    }
    if (bad) atomicOr(p.status, kKvStatusIndex);
    long long tile = -1;                 // (page, head 0), -1: nothing to read
    int slot = 0;
    if (mine && b >= 0) {                // rows of no sequence stay as they were
        const int begin = p.tok.lens[b];
        const long long pos = (long long)begin + row - first;
        int page = -1;
        if (begin >= 0 && pos < (long long)p.tok.max_pages * p.tok.page) {
            page = p.tok.table[(long long)b * p.tok.max_pages + (pos >> p.tok.log_page)];
            slot = (int)(pos & (p.tok.page - 1));
        }
        if (page < 0 || page >= p.tok.num_pages)
            atomicOr(p.status, kKvStatusIndex);
        else
            tile = (long long)page * p.H;
    }
    const uint8_t *pages = kv ? p.pages[1] : p.pages[0];
    const float *scale = kv ? p.scale[1] : p.scale[0];
    for (int r = 0; r < p.rows; ++r) {
        const long long tr = __shfl_sync(0xffffffffu, tile, r);
        const int sr = __shfl_sync(0xffffffffu, slot, r);
        if (tr < 0) continue;
        TO *out = static_cast<TO *>(dst) + (long long)(row0 + r) * p.H * p.D;
        for (int e = lane * 16; e < p.H * p.D; e += 512) {
            const int h = e >> p.log_d;
            const float s = scale[tr + h];
            const uint4 w = *reinterpret_cast<const uint4 *>(pages + (((tr + h) * p.tok.page + sr) << p.log_d) + (e & (p.D - 1)));
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float v[8], a[4], c[4];
                KvCode<E4M3>::unpack4(ws[2 * i], a);
                KvCode<E4M3>::unpack4(ws[2 * i + 1], c);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[j] = a[j] * s;
                    v[4 + j] = c[j] * s;
                }
                rope_store8(out + e + 8 * i, v);
            }
        }
    }
}

}  // namespace eva
