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
//  eva_kv_append_kernel  one CTA per (sequence's page, head, keys or values)
//  eva_kv_read_kernel    one warp per token, keys and values
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
    int B, T, page, max_pages, num_pages;
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
        for (int i = 0; i < 4; ++i) v[i] = (float)(int8_t)(w >> (8 * i));
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
    int H, D;
    int *status;
};

__device__ __forceinline__ float kv_clean(float x) {
    return x == x ? fminf(fmaxf(x, -65504.f), 65504.f) : 0.f;
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
                first = begin / k.page;
                count = (end - 1) / k.page - first + 1;
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
    const int page = p.tok.table[(long long)u.b * p.tok.max_pages + u.page_index];
    if (page < 0 || page >= p.tok.num_pages) {
        if (threadIdx.x == 0) atomicOr(p.status, kKvStatusIndex);
        return;
    }
    const int h = blockIdx.y, kv = blockIdx.z, D = p.D, tid = threadIdx.x;
    const int per = D >> 3, chunks = (u.hi - u.lo) * per;          // 8 elements a chunk
    const long long ld = kv ? p.ld[1] : p.ld[0];
    const TI *src = static_cast<const TI *>(kv ? p.x[1] : p.x[0]) + u.row * ld + (long long)h * D;
    const long long tile = (long long)page * p.H + h;
    uint8_t *dst = (kv ? p.pages[1] : p.pages[0]) + tile * p.tok.page * D;
    float *scale = (kv ? p.scale[1] : p.scale[0]) + tile;
    const float was = u.lo > 0 ? *scale : 0.f;
    // The first chunks of a thread stay in registers between the two passes.
    constexpr int kKeep = 4;
    float keep[kKeep][8];
    float amax = 0.f;
    auto load = [&](int c, float (&v)[8]) {
        const int t = c / per;
        rope_load8(src + t * ld + (c - t * per) * 8, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = kv_clean(v[j]);
    };
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
        const int c = tid + i * kKvThreads;
        if (c >= chunks) continue;
        load(c, keep[i]);
    }
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
        if (tid + i * kKvThreads >= chunks) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(keep[i][j]));
    }
    for (int c = tid + kKeep * kKvThreads; c < chunks; c += kKvThreads) {
        float v[8];
        load(c, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
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
    auto store = [&](int c, const float (&v)[8]) {
        float q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = now > 0.f ? __fdiv_rn(v[j], now) : 0.f;
        *reinterpret_cast<uint2 *>(dst + (long long)u.lo * D + c * 8) =
            make_uint2(KvCode<E4M3>::pack4(q[0], q[1], q[2], q[3]), KvCode<E4M3>::pack4(q[4], q[5], q[6], q[7]));
    };
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
        const int c = tid + i * kKvThreads;
        if (c < chunks) store(c, keep[i]);
    }
    for (int c = tid + kKeep * kKvThreads; c < chunks; c += kKvThreads) {
        float v[8];
        load(c, v);
        store(c, v);
    }
}

struct KvReadParams {
    KvTokens tok;                        // starts: rows of the outputs; lens: first position of each sequence
    const uint8_t *pages[2];
    const float *scale[2];
    void *out[2];                        // [T][H][D], contiguous; either may be null
    int H, D;
    int *status;
};

template <typename TO, bool E4M3>
__global__ void __launch_bounds__(kKvThreads) eva_kv_read_kernel(KvReadParams p) {
    const int lane = threadIdx.x & 31, kv = blockIdx.y;
    const int row = blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5);
    pdl_wait();
    pdl_launch();
    void *dst = kv ? p.out[1] : p.out[0];
    if (row >= p.tok.T || !dst) return;
    // the sequence: how many of starts[1 .. B] are at or before this row
    int b = 0;
    for (int b0 = 1; b0 <= p.tok.B; b0 += 32) {
        const bool le = b0 + lane <= p.tok.B && p.tok.starts[b0 + lane] <= row;
        b += __popc(__ballot_sync(0xffffffffu, le));
    }
    if (b >= p.tok.B) return;            // behind the last sequence: left as it was
    const int first = p.tok.starts[b], begin = p.tok.lens[b];
    const long long pos = (long long)begin + row - first;
    int page = -1;
    if (first >= 0 && row >= first && begin >= 0 && pos < (long long)p.tok.max_pages * p.tok.page)
        page = p.tok.table[(long long)b * p.tok.max_pages + pos / p.tok.page];
    if (page < 0 || page >= p.tok.num_pages) {
        if (lane == 0) atomicOr(p.status, kKvStatusIndex);
        return;
    }
    const int slot = (int)(pos % p.tok.page);
    TO *out = static_cast<TO *>(dst) + (long long)row * p.H * p.D;
    const uint8_t *pages = kv ? p.pages[1] : p.pages[0];
    const float *scale = kv ? p.scale[1] : p.scale[0];
    for (int e = lane * 8; e < p.H * p.D; e += 256) {
        const int h = e / p.D;
        const long long tile = (long long)page * p.H + h;
        const float s = scale[tile];
        const uint2 w = *reinterpret_cast<const uint2 *>(pages + (tile * p.tok.page + slot) * p.D + e - h * p.D);
        float v[8], a[4], c[4];
        KvCode<E4M3>::unpack4(w.x, a);
        KvCode<E4M3>::unpack4(w.y, c);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = a[j] * s;
            v[4 + j] = c[j] * s;
        }
        rope_store8(out + e, v);
    }
}

}  // namespace eva
