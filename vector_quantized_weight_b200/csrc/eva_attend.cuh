// eva_attend.cuh -- attention of new tokens over the paged 8-bit cache.
//
// For every row (token, query head) at position p of its sequence
//   z_j = scale * q.k_j,  optionally cap * tanh(z_j / cap),  j <= p, j > p - window
//   o = sum_j e^(z_j - m) v_j / sum_j e^(z_j - m)
// in one pass over the cache with the running maximum m and sum.  k_j = sk c_j
// and v_j = sv d_j with 8-bit codes and one scale a page and head.
//
// What bounds it: a decode step reads each cached byte once for a handful of
// multiplications, so bytes; everything else has to fit beside the stream.
//  - Codes become f16 exactly (int8: a byte under exponent 2^10, minus 1152;
//    e4m3: the conversion instruction -- shifting sign and magnitude into place
//    kept the integer pipe 72 % busy and took half as long again on heads of
//    256) and go to the tensor cores as the A operand: 16 tokens x 16
//    dimensions of keys, 16 dimensions x 16 tokens of values.  Rows are the MMA's
//    N, 8 at a time, so a decode step of one to eight queries a key head wastes
//    nothing, and more rows reuse the converted codes.  Warp-level MMAs: at
//    eight rows the tensor pipe is 11 % busy at full stream speed and the
//    conversion into registers is the work.  With many rows (64 tokens of a
//    prompt with eight queries a key head: 512) the products bound it, and
//    these MMAs reach 169 TFLOP/s there, a tenth of the tensor peak.
//  - Scales never touch the codes: sk multiplies the finished score, sv enters
//    the exponent.  With w_j = e^(z_j - M) sv and M a reference 2^11 to 2^15 below
//    the maximum of z_j + ln sv, the weights stay in (0, 2^15] whatever the pages'
//    scales are; the sum of the softmax gets w_j / sv.  w_j is rounded to f16 for
//    the value product: at most 2^-11 of it (the products run at the f16 rate and
//    the error averages over the keys), and below 2^-14 a step of 2^-24, which is
//    at most 2^-36 of the largest weight for each key.  (M at the maximum itself
//    left the upper half of f16's range unused: beside one key 18 nats above
//    131,071 others the step was larger than their weights.)  All sums and
//    statistics are fp32.
//  - One warp of a CTA walks the work, looks pages and scales up, 32 steps at a
//    time, one a lane, and copies each step's codes (TMA, swizzled: both
//    ldmatrix patterns are free of bank conflicts) into a ring in shared
//    memory; the others take turns at the steps.  (Copies issued by the warp
//    that needs them, into buffers of its own, took 72 us for 268 MB of 64
//    sequences against 64: the issue then sits between a step's products.)  A
//    page id outside the cache is never used as an address: its tokens count as
//    masked and the status word is set.
//  - Work is cut on the device, because only the device knows the lengths
//    (AtWalk).  An item (sequence, row tile, key head) that several CTAs share
//    is joined by the last of them to finish, in the order of the parts, so
//    results do not depend on timing.
//
// Measured (device time): 268 MB of cache as 64 sequences 59 us (4.5 TB/s), as
// one 54 us (5.0 TB/s, of which 39 us stream at the memory's rate and the rest
// is the start's three dependent lookups, the joins and the slowest CTAs); 517
// tokens of 32 heads 10.3 us, all of it latency.
#pragma once
#include <cuda.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "eva_kv.cuh"

namespace eva {

constexpr int kAtStatusWait = 1;       // status bit: a bounded wait gave up

struct AttendParams {
    KvTokens tok;
    const __half *q;                   // [T][Hq][D], ldq elements a token
    long long ldq;
    const float *k_scale, *v_scale;    // [pages][H]
    void *out;                         // [T][Hq][D]
    float *lse;                        // [T][Hq] or null
    float *part;                       // [2 grid][rows][D] unnormalised outputs of shared items
    float2 *part_ml;                   // [2 grid][rows] reference (base 2) and sum
    int *counters;                     // [3][grid], zero between calls
    int *status;
    int Hq, H, G;                      // query heads, key heads, queries a key head
    int window, out_f32, min_steps, wait_rounds;
    int inject;                        // test hook, 1: stream nothing, so that every wait runs out; 2: work on nothing
    float scale, cap;                  // cap 0: none
    uint32_t nothing;                  // 0, but not to the compiler
};

struct alignas(64) AttendMaps {
    CUtensorMap k, v;                  // codes as rows of D bytes, [pages * H * page][D] (D = 256: [2][rows][128])
};

// ---------------------------------------------------------------- small PTX

// One copy of a map's box: rows of at most 128 bytes, or both 128-byte halves of each row, one behind the other.
template <int D>
__device__ __forceinline__ void at_tma(uint32_t dst, const CUtensorMap *m, int y, uint32_t bar) {
    if constexpr (D <= 128)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
            ::"r"(dst), "l"(m), "r"(0), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
            ::"r"(dst), "l"(m), "r"(0), "r"(y), "r"(0), "r"(bar)
            : "memory");
}
__device__ __forceinline__ void at_ldsm(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void at_ldsm_t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
// mbar_wait_bounded with its loop inside the statement: no reconvergence code around it.
__device__ __forceinline__ bool at_wait(uint32_t bar, uint32_t parity, int rounds) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 n;\n\t"
        "mov.b32 n, %3;\n\t"
        "LOOP:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE;\n\t"
        "sub.s32 n, n, 1;\n\t"
        "setp.gt.s32 q, n, 0;\n\t"
        "@q bra LOOP;\n\t"
        "DONE:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(rounds)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ uint32_t at_transpose(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void at_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float at_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// cap * tanh(x).  1 - 2 / (1 + e^2x) is off by some 2^-22 of 1, which is no longer small beside a small tanh (scores far
// below a large cap would be lost): below 1/4 the series, whose next term is 2^-26 of x there.
__device__ __forceinline__ float at_capped(float x, float cap) {
    const float x2 = x * x;
    const float series = 1.f + x2 * (-1.f / 3.f + x2 * (2.f / 15.f + x2 * (-17.f / 315.f + x2 * (62.f / 2835.f))));
    return x2 < 0.0625f ? cap * x * series : cap - __fdividef(2.f * cap, 1.f + __expf(2.f * x));
}

// 2^(x / 2).  Sums are brought to another reference by two such factors: over pages of zeros they are up to 2^100 times
// larger than their weights, and 2^x alone would be 0 for what still counts.
__device__ __forceinline__ float at_half_exp2(float x) { return at_exp2(0.5f * x); }

// Four codes -> two pairs of f16: neighbours (b0 b1, b2 b3: dimensions of a
// key) or every other (b0 b2, b1 b3: a dimension of two tokens' values).
// (Leaving int8 values 1152 too large and taking 1152 times the sum of the
// weights off at the end would save two subtractions in five operations, but
// the tensor cores' sums truncate, and over a long context that bias is no
// longer small beside an average of values of both signs.)
template <bool E4M3>
struct AtCode;
template <>
struct AtCode<false> {
    static __device__ __forceinline__ uint32_t exact(uint32_t w) {
        const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&w), __half2half2(__ushort_as_half(0x6480)));
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ void key(uint32_t x, uint32_t &a, uint32_t &b) {
        x ^= 0x80808080u;
        a = exact(__byte_perm(x, 0x64646464u, 0x4140));
        b = exact(__byte_perm(x, 0x64646464u, 0x4342));
    }
    static __device__ __forceinline__ void value(uint32_t x, uint32_t &a, uint32_t &b) {
        x ^= 0x80808080u;
        a = exact(__byte_perm(x, 0x64646464u, 0x4240));
        b = exact(__byte_perm(x, 0x64646464u, 0x4341));
    }
};
template <>
struct AtCode<true> {
    static __device__ __forceinline__ void key(uint32_t x, uint32_t &a, uint32_t &b) {
        asm("{\n\t.reg .b16 lo, hi;\n\t"
            "mov.b32 {lo, hi}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
            : "=r"(a), "=r"(b)
            : "r"(x));
    }
    static __device__ __forceinline__ void value(uint32_t x, uint32_t &a, uint32_t &b) { key(__byte_perm(x, 0u, 0x3120), a, b); }
};

// ------------------------------------------------------- the line of steps

// Steps of row tile rt of a sequence: [s0, s0 + n); a tile that sees no key has
// one step, all of it masked.
struct AtTile {
    int s0, n;
};
template <int TS>
__device__ __forceinline__ AtTile at_tile(const KvSeq &s, int rt, int rows, int G, int window) {
    const int r0 = rt * rows, r1 = min(r0 + rows, s.n * G) - 1;
    const int hi = s.len - s.n + r1 / G;
    const int lo = window > 0 ? max(0, s.len - s.n + r0 / G - window + 1) : 0;
    AtTile t;
    t.s0 = hi < lo ? 0 : lo / TS;
    t.n = hi < lo ? 1 : hi / TS - t.s0 + 1;
    return t;
}
__device__ __forceinline__ int at_tiles(const KvSeq &s, int rows, int G) { return (s.n * G + rows - 1) / rows; }

// A CTA's share of the work, walked piece by piece; uniform over a warp.
//
// Few items (at most half as many as CTAs): each is cut into equal parts of at
// most S steps, S the smallest for which the parts are no more than the CTAs
// (and at least min_steps: joining costs more than that many steps).  A CTA
// has one piece.
// Many items: they form one line, in which an item takes kAtItemCost steps
// besides its own (starting and finishing it costs a CTA about that), and
// every CTA takes an equal stretch, whatever the items' borders.
constexpr int kAtItemCost = 4;
template <int TS>
struct AtWalk {
    long long total, at;               // the line's length, the current item's place in it
    int left;                          // of this CTA's stretch from the current place on (few items: 1 or 0)
    int parts;                         // CTAs that take a stretch (0: few items)
    int b, rt, nrt, h;                 // the item
    KvSeq seq;
    AtTile tile;
    int off;                           // of the item that lies before this CTA's stretch; few items: which part of
    int k;                             // how many

    // (an item half as long again as the least part stays whole: 17 steps in one part or two, 10.1 or 10.6 us)
    static __device__ __forceinline__ int cuts(int n, int S, int least) { return 2 * n <= 3 * least ? 1 : (n + S - 1) / S; }

    __device__ __forceinline__ void init(const AttendParams &p, int rows, bool &bad) {
        const int lane = threadIdx.x & 31;
        KvSeq first = {0, 0, 0};       // of the first 32 sequences, not loaded again
        auto seq_of = [&](int b0) {
            KvSeq s = first;
            if (b0 > 0) {
                s.n = 0;
                if (b0 + lane < p.tok.B) s = kv_seq(p.tok, b0 + lane, bad);
            }
            return s;
        };
        if (lane < p.tok.B) first = kv_seq(p.tok, lane, bad);
        long long steps = 0, items = 0;
        for (int b0 = 0; b0 < p.tok.B; b0 += 32) {
            const KvSeq s = seq_of(b0);
            const int n = at_tiles(s, rows, p.G);
            for (int t = 0; t < n; ++t) steps += at_tile<TS>(s, t, rows, p.G, p.window).n;
            items += n;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            steps += __shfl_xor_sync(0xffffffffu, steps, o);
            items += __shfl_xor_sync(0xffffffffu, items, o);
        }
        steps *= p.H;
        items *= p.H;
        const int c = blockIdx.x, grid = gridDim.x;
        const bool few = items * 2 <= grid;
        int S = 0;
        left = parts = 0;
        at = total = 0;
        if (items == 0) return;
        long long place;               // this CTA's first part, or first step of the line
        if (few) {
            S = (int)max((long long)p.min_steps, (steps + grid - items - 1) / (grid - items));
            place = c;
        } else {
            total = steps + items * kAtItemCost;
            parts = (int)min((long long)grid, (total + p.min_steps - 1) / p.min_steps);
            if (c >= parts) return;
            if (total / parts >= (1 << 30)) {  // a CTA counts its steps in 32 bits
                bad = true;
                return;
            }
            place = total * c / parts;
            left = (int)(total * (c + 1) / parts - place);
        }
        // the sequence, the row tile and the head that hold `place`
        long long before = 0;
        unsigned who = 0;
        for (int b0 = 0; b0 < p.tok.B && !who; b0 += 32) {
            const KvSeq s = seq_of(b0);
            long long w = 0;
            for (int t = 0, n = at_tiles(s, rows, p.G); t < n; ++t) {
                const int m = at_tile<TS>(s, t, rows, p.G, p.window).n;
                w += few ? cuts(m, S, p.min_steps) : m + kAtItemCost;
            }
            w *= p.H;
            long long sum = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += v;
            }
            who = __ballot_sync(0xffffffffu, place >= before + sum - w && place < before + sum);
            const int src = who ? __ffs(who) - 1 : 31;
            b = b0 + src;
            before += __shfl_sync(0xffffffffu, who ? sum - w : sum, src);
            seq.row = __shfl_sync(0xffffffffu, s.row, src);
            seq.n = __shfl_sync(0xffffffffu, s.n, src);
            seq.len = __shfl_sync(0xffffffffu, s.len, src);
        }
        if (!who) {                    // few items, and fewer parts than CTAs
            left = 0;
            return;
        }
        nrt = at_tiles(seq, rows, p.G);
        long long in = place - before;
        int w = 1;
        for (rt = 0;; ++rt) {
            tile = at_tile<TS>(seq, rt, rows, p.G, p.window);
            w = few ? cuts(tile.n, S, p.min_steps) : tile.n + kAtItemCost;
            if (in < (long long)w * p.H || rt + 1 >= nrt) break;
            in -= (long long)w * p.H;
        }
        h = (int)(in / w);
        off = (int)(in - (long long)h * w);
        k = w;
        at = place - off;
        if (few) left = 1;
    }

    // This CTA's steps [lo, hi) of the current item (none: the stretch holds only some of its extra), and the CTAs
    // c0 .. c1 that share the item.
    __device__ __forceinline__ void piece(int &lo, int &hi, int &c0, int &c1) const {
        if (parts == 0) {
            lo = (int)((long long)tile.n * off / k);
            hi = (int)((long long)tile.n * (off + 1) / k);
            c0 = blockIdx.x - off;
            c1 = c0 + k - 1;
        } else {
            lo = max(0, off - kAtItemCost);
            hi = min(tile.n, off + left - kAtItemCost);
            c0 = part_of(at + kAtItemCost);
            c1 = part_of(at + kAtItemCost + tile.n - 1);
        }
    }
    __device__ __forceinline__ void next(const AttendParams &p, int rows, bool &bad) {
        if (parts == 0) {
            left = 0;
            return;
        }
        left -= tile.n + kAtItemCost - off;
        if (left <= 0) return;
        at += tile.n + kAtItemCost;
        off = 0;
        if (++h < p.H) return;
        h = 0;
        if (++rt >= nrt) {
            rt = 0;
            do seq = kv_seq(p.tok, ++b, bad);
            while (seq.n == 0 && b + 1 < p.tok.B);
            nrt = at_tiles(seq, rows, p.G);
        }
        tile = at_tile<TS>(seq, rt, rows, p.G, p.window);
    }
    // the part that holds step s of the line
    __device__ __forceinline__ int part_of(long long s) const { return (int)(((s + 1) * parts - 1) / total); }
};

// --------------------------------------------------------------- the kernel

// What the walking warp leaves beside a step's codes, for each 16 tokens: the
// score's factor (negative: no token there), log2 of the value scale, and
// kAtSumScale over it.
struct alignas(16) AtScales {
    float sk[2], lsv[2], rsv[2];
    int tag, pad;                      // the step's number in its CTA
};
// A piece of work: the steps t0 .. t0 + n - 1 of the CTA (n 0: no more).
struct AtPiece {
    int t0, n, s_first;                // and the first one's number in its sequence
    int row, rows, len;                // first packed row and row count of the sequence, its length
    int rt, h;
    int c0, c1;                        // CTAs that share the item
    int pad[2];
};
constexpr int kAtPieces = 2;           // handed over ahead, with their queries (the code below knows it is two)
constexpr int kAtTurn = 2;             // steps copied at a time (divides 8)
constexpr int kAtSmemPerSm = 228 * 1024;
constexpr int kAtSegment = 8;          // parts that are joined at a time
// A page of zeros counts as one of a very small value scale, so that it leaves the reference to the others: weights over
// that scale are as large as 2^115, and 2^13 of them would leave fp32.  The sums are kept 2^20 times smaller.
constexpr float kAtLeastScale = 1e-30f, kAtSumScale = 9.5367431640625e-07f, kAtLog2SumScale = -20.f;

template <int D, int NT, int WARPS, int CTAS>
struct AtShape {
    static constexpr int kRows = 8 * NT;                   // rows of an item
    static constexpr int kStep = D > 128 ? 16 : 32;        // tokens a step: 8 KB of keys and values, 4 at D = 64
    static constexpr int kStepBytes = 2 * kStep * D;
    static constexpr int kThreads = 32 * (WARPS + 1);
    static constexpr int kQStride = D + 16;                // halves; 8 g + 2 c words: no conflicts
    static constexpr int kOStride = D + 4;                 // floats; 8 c + 2 g words: no conflicts
    static constexpr size_t kQBytes = (size_t)kRows * kQStride * 2;
    static constexpr size_t kOBytes = (size_t)WARPS * kRows * kOStride * 4;
    static constexpr size_t kMlBytes = (size_t)WARPS * kRows * 8;
    static constexpr size_t kFixedBytes = 1024 + kAtPieces * kQBytes + kOBytes + kMlBytes + kAtPieces * (sizeof(AtPiece) + 16) + 128;
    static constexpr size_t kStageBytes = kStepBytes + sizeof(AtScales) + 16;
    // the ring takes what a CTA's share of the 228 KB leaves (1 KB a CTA is the system's)
    static constexpr int kRoom = (int)((kAtSmemPerSm / CTAS - 1024 - kFixedBytes) / kStageBytes);
    static constexpr int kStages = kRoom < 16 ? kRoom : 16;
    static constexpr bool kTagged = kStages % WARPS != 0;
    static constexpr size_t kSmem = kFixedBytes + kStages * kStageBytes;
    static_assert(kStages >= WARPS, "each warp needs a stage of its own");
    // lanes that share a row when parts are joined: a power of two, at least one row a thread
    static constexpr int kJoinLanes = 32 * WARPS / kRows >= 16 ? 16 : 32 * WARPS / kRows >= 8 ? 8 : 4;
    static_assert(kRows * kJoinLanes <= 32 * WARPS, "a few lanes join the maxima of a row");
};

// Resident CTAs an SM: warps are dealt to four schedulers of 16384 registers
// each, so 16 warps get 128 registers each, 12 get 168, 8 get 255.
template <int D, int NT, int WARPS, int CTAS, bool E4M3>
__global__ void __launch_bounds__(32 * (WARPS + 1), CTAS)
    eva_attend_kernel(const __grid_constant__ AttendMaps maps, AttendParams p) {
    using S = AtShape<D, NT, WARPS, CTAS>;
    constexpr int kRows = S::kRows, kChunks = D / 16, kStep = S::kStep, MT = kStep / 16, kStages = S::kStages;
    // shared memory: ring | scales | pieces | queries | outputs | statistics | barriers (stages full and free, pieces
    // full and free, the warps') | flags
    const uint32_t base0 = (uint32_t)__cvta_generic_to_shared(eva_smem);
    const uint32_t skip = ((base0 + 1023) & ~1023u) - base0, ring_a = base0 + skip;
    AtScales *scales = reinterpret_cast<AtScales *>(eva_smem + skip + kStages * S::kStepBytes);
    AtPiece *pieces = reinterpret_cast<AtPiece *>(scales + kStages);
    __half *qs = reinterpret_cast<__half *>(pieces + kAtPieces);
    float *os = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(qs) + kAtPieces * S::kQBytes);
    float2 *mls = reinterpret_cast<float2 *>(reinterpret_cast<uint8_t *>(os) + S::kOBytes);
    const uint32_t full_a = (uint32_t)__cvta_generic_to_shared(reinterpret_cast<uint8_t *>(mls) + S::kMlBytes);
    const uint32_t free_a = full_a + 8 * kStages, pfull_a = free_a + 8 * kStages, pfree_a = pfull_a + 8 * kAtPieces;
    const uint32_t meet_a = pfree_a + 8 * kAtPieces, q_a = (uint32_t)__cvta_generic_to_shared(qs);
    volatile int *flag = reinterpret_cast<volatile int *>(eva_smem + (meet_a + 8 - base0));

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            scales[i].tag = -1;
            mbar_init(full_a + 8 * i, 2);      // the copies' bytes, and the scales
            mbar_init(free_a + 8 * i, 1);
        }
        for (int i = 0; i < kAtPieces; ++i) {
            mbar_init(pfull_a + 8 * i, 1);
            mbar_init(pfree_a + 8 * i, WARPS);
        }
        mbar_init(meet_a, WARPS);
    }
    __syncthreads();
    pdl_wait();
    pdl_launch();

    if (warp == WARPS) {
        // -------------------------------------------------- the walking warp
        bool bad = false, ok = true;
        AtWalk<kStep> walk;
        walk.init(p, kRows, bad);
        const int page = p.tok.page;
        const bool split = page < kStep;                   // a step's halves lie on two pages
        const int box = split ? 16 : kStep;
        int t = 0, st = 0, ahead = 0;  // steps so far, the next one's stage, steps copied before their scales were known
        int landed = 0;                // of the last steps, where the warp gave up
        auto land = [&](int step) { mbar_wait_bounded(full_a + 8 * (step % kStages), (step / kStages) & 1, kWaitRounds); };
        uint32_t parity = 1;           // of the free barriers: the first round passes at once
        int ps = 0, handed = 0;        // the next piece's place, pieces so far
        int used0 = kRows, used1 = kRows;      // rows of each place's queries that may not be zeros
        uint32_t pparity = 1;
        while (ok && walk.left > 0) {
            int lo, hi, c0, c1;
            walk.piece(lo, hi, c0, c1);
            const int s_first = walk.tile.s0 + lo, n = hi - lo;
            if (n > 0) {
                const int32_t *table = p.tok.table + (long long)walk.b * p.tok.max_pages;
                // (a step of two pages may begin with one that is wholly before the window: gone, maybe, and not looked at)
                const int seen = split && p.window > 0 ? walk.seq.len - walk.seq.n + walk.rt * kRows / p.G - p.window + 1 : 0;
                auto there = [&](int tok) { return tok < walk.seq.len && tok + 16 > seen; };
                int pid[2] = {-1, -1}, pid_next[2];        // pages of this lane's step, -1: no token there
                auto look = [&](int s, int (&id)[2]) {
                    id[0] = id[1] = -1;
                    if (s >= n) return;
                    const int tok0 = (s_first + s) * kStep;
                    if (there(tok0)) id[0] = table[tok0 >> p.tok.log_page];
                    if (MT > 1 && there(tok0 + 16)) id[1] = split ? table[(tok0 >> p.tok.log_page) + 1] : id[0];
                };
                auto check = [&](int s, int (&id)[2]) {    // a page outside the cache: no token there, and say so
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        if (id[i] >= 0 && id[i] < p.tok.num_pages) continue;
                        if (s < n && there((s_first + s) * kStep + 16 * i)) bad = true;
                        id[i] = -1;
                    }
                };
                auto scale = [&](const int (&id)[2], float (&k)[2], float (&v)[2]) {
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        const bool in = id[i] >= 0;
                        k[i] = in ? p.k_scale[(long long)id[i] * p.H + walk.h] : -1.f;
                        v[i] = in ? p.v_scale[(long long)id[i] * p.H + walk.h] : 1.f;
                    }
                };
                auto copy = [&](int s, int stage) {        // this lane's step s into a stage
                    const bool two = MT > 1 && split && pid[1] >= 0;
                    const uint32_t bytes = (uint32_t)(((pid[0] >= 0) + two) * 2 * box * D);
                    const uint32_t bar = full_a + 8 * stage, dst = ring_a + stage * S::kStepBytes;
                    if (bytes)
                        mbar_arrive_expect_tx(bar, bytes);
                    else
                        mbar_arrive(bar);
                    const int y0 = (pid[0] * p.H + walk.h) * page + ((s_first + s) * kStep & (page - 1));
                    const int y1 = (pid[1] * p.H + walk.h) * page;
                    if (pid[0] >= 0) {
                        at_tma<D>(dst, &maps.k, y0, bar);
                        at_tma<D>(dst + kStep * D, &maps.v, y0, bar);
                    }
                    if (two) {
                        at_tma<D>(dst + 16 * D, &maps.k, y1, bar);
                        at_tma<D>(dst + kStep * D + 16 * D, &maps.v, y1, bar);
                    }
                };
                look(lane, pid);
                check(lane, pid);
                if (t == 0 && p.inject != 1) {
                    ahead = min(min(n, 32), kStages);
                    if (lane < ahead) copy(lane, lane);
                }
                float sk[2], sv[2], sk_next[2] = {}, sv_next[2] = {};
                scale(pid, sk, sv);
                ok = at_wait(pfree_a + 8 * ps, pparity, p.wait_rounds);
                if (!ok) break;
                if (lane == 0) {
                    AtPiece &q = pieces[ps];
                    q.t0 = t;
                    q.n = n;
                    q.s_first = s_first;
                    q.row = walk.seq.row;
                    q.rows = walk.seq.n;
                    q.len = walk.seq.len;
                    q.rt = walk.rt;
                    q.h = walk.h;
                    q.c0 = c0;
                    q.c1 = c1;
                }
                {
                    // The queries, a row a copy; zeros behind the last one, where an earlier piece's rows (at first,
                    // anything) would pull the references of this one's.
                    const int r0 = walk.rt * kRows, rows = min(kRows, walk.seq.n * p.G - r0);
                    const uint32_t bar = pfull_a + 8 * ps;
                    const int used = ps ? used1 : used0;
                    for (int i = rows * (D / 8) + lane; i < used * (D / 8); i += 32)
                        *reinterpret_cast<uint4 *>(qs + ps * (S::kQBytes / 2) + i / (D / 8) * S::kQStride + i % (D / 8) * 8) =
                            make_uint4(0, 0, 0, 0);
                    if (rows < used) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before later copies
                    if (ps) used1 = rows; else used0 = rows;
                    __syncwarp();
                    if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(rows * D * 2));
                    __syncwarp();
                    if (lane < rows) {
                        const int ti = (r0 + lane) / p.G, hq = walk.h * p.G + (r0 + lane) - ti * p.G;
                        bulk_copy_g2s(q_a + (uint32_t)(ps * S::kQBytes) + (uint32_t)(lane * S::kQStride * 2),
                                      p.q + (walk.seq.row + ti) * p.ldq + (long long)hq * D, D * 2, bar);
                    }
                }
                ++handed;
                if (++ps == kAtPieces) {
                    ps = 0;
                    pparity ^= 1;
                }
                ok = p.inject != 1;
                for (int s0 = 0; s0 < n && ok; s0 += 32) {
                    look(s0 + 32 + lane, pid_next);        // in flight while these steps go out
                    AtScales sc = {};
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        const float v = fmaxf(sv[i], kAtLeastScale);
                        sc.sk[i] = sk[i];
                        sc.lsv[i] = log2f(v);
                        sc.rsv[i] = kAtSumScale / v;
                    }
                    const int count = min(32, n - s0);
                    // kAtTurn lanes at a time wait for their stages and fill them: one step at a time took the warp
                    // 500 to 750 cycles each, more than all the others need for the work.
                    for (int i = 0; i < count; i += kAtTurn) {
                        const int mine = lane - i, turn = min(kAtTurn, count - i);
                        bool there = true;
                        if (mine >= 0 && mine < turn) {
                            const bool wrap = st + mine >= kStages;
                            const int to = wrap ? st + mine - kStages : st + mine;
                            there = at_wait(free_a + 8 * to, wrap ? parity ^ 1 : parity, p.wait_rounds);
                            if (there) {
                                sc.tag = t + mine;
                                scales[to] = sc;
                                mbar_arrive(full_a + 8 * to);
                                if (t + mine >= ahead) copy(s0 + lane, to);
                            }
                        }
                        ok = __all_sync(0xffffffffu, there);
                        if (!ok) {             // the turn's stages hold these steps, or still those of a round before
                            if (mine >= 0 && mine < turn) land(t + mine - (there ? 0 : kStages));
                            t += turn;
                            landed = turn;
                            break;
                        }
                        t += turn;
                        st += turn;
                        if (st >= kStages) {
                            st -= kStages;
                            parity ^= 1;
                        }
                        if (i == 8) {
                            check(s0 + 32 + lane, pid_next);
                            scale(pid_next, sk_next, sv_next);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        pid[i] = pid_next[i];
                        sk[i] = sk_next[i];
                        sv[i] = sv_next[i];
                    }
                }
            }
            walk.next(p, kRows, bad);
        }
        if (ok) ok = at_wait(pfree_a + 8 * ps, pparity, p.wait_rounds);
        if (ok && lane == 0) {
            pieces[ps].n = 0;
            mbar_arrive(pfull_a + 8 * ps);
        }
        if (bad) atomicOr(p.status, kKvStatusIndex);
        if (!ok) {                     // another warp gave up: say so
            if (lane == 0) atomicOr(p.status, kAtStatusWait);
            for (; t < ahead; ++t)
                if (lane == 0) mbar_arrive(full_a + 8 * t);
        }
        // No copy outlives its CTA, whether or not the working warps are there to wait for it.  (Of the last two pieces the
        // first is done with where the CTA's end was handed over in its place.)
        const int piece = handed - 1 - lane, step = t - landed - 1 - lane;
        if (piece >= 0 && lane < (ok ? kAtPieces - 1 : kAtPieces))
            mbar_wait_bounded(pfull_a + 8 * (piece % kAtPieces), (piece / kAtPieces) & 1, kWaitRounds);
        if (step >= 0 && lane < kStages - landed) land(step);
        return;
    }

    // ---------------------------------------------------- the working warps
    const int g = lane >> 2, c = lane & 3, tid = threadIdx.x;      // tid < 32 * WARPS
    // the reference trails the largest score by kLift when it moves and by kLift + kLag, 2^15, at most (8 and 7, 4 and
    // 11, 2 and 13 take 102.4, 102.5 and 103.0 us on 64 tokens over 8191)
    constexpr float kLog2e = 1.4426950408889634f, kLag = 4.f, kLift = 11.f;
    const float zscale = p.cap > 0.f ? p.scale / p.cap : p.scale * kLog2e;
    const float zcap = p.cap * kLog2e;

    // All warps of the CTA have come here (and their shared-memory writes are seen); a bounded wait like the others,
    // so that a warp that gave up leaves nobody waiting.
    uint32_t meet_parity = 0;
    auto come = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(meet_a);
    };
    auto all_here = [&]() {
        const bool r = at_wait(meet_a, meet_parity, p.wait_rounds);
        meet_parity ^= 1;
        return r;
    };
    auto meet = [&]() {
        come();
        return all_here();
    };

    auto addr = [&](uint32_t tile, int tok, int ch) {
        if constexpr (D >= 128)
            return tile + (uint32_t)((ch >> 3) * (kStep * 128) + tok * 128 + (((ch & 7) ^ (tok & 7)) << 4));
        else
            return tile + (uint32_t)(tok * 64 + ((ch ^ ((tok >> 1) & 3)) << 4));
    };

    float o[NT][kChunks][4], m[NT][2], l[NT][2];
    int pmin = 0, pmax = 0;            // the last key that the item's first and its last row see
    int ps = 0, ct = warp;             // the piece's place; this warp's next step of the CTA
    int own = warp;                    // and its stage, and that stage's parity
    uint32_t pparity = 0, own_parity = 0;
    bool ok = true, first = true;
    for (;;) {
        ok = p.inject != 2 && at_wait(pfull_a + 8 * ps, pparity, p.wait_rounds);
        if (!ok) break;
        const AtPiece &bt = pieces[ps];
        const int t_end = bt.t0 + bt.n, step0 = bt.s_first - bt.t0;
        if (bt.n == 0) break;
        {
            const int r0 = bt.rt * kRows, nrows = min(kRows, bt.rows * p.G - r0);
            const int pos0 = bt.len - bt.rows;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    m[nt][e] = -INFINITY;
                    l[nt][e] = 0.f;
                }
#pragma unroll
                for (int ch = 0; ch < kChunks; ++ch)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[nt][ch][e] = 0.f;
            }
            pmin = pos0 + r0 / p.G;
            pmax = pos0 + (r0 + nrows - 1) / p.G;
        }
        const __half *qp = qs + ps * (S::kQBytes / 2);
        for (; ct < t_end; ct += WARPS) {
            const int st = own;
            if constexpr (S::kTagged) {
                // Where a stage passes from warp to warp, a warp may be two rounds behind, and a barrier's parity
                // would tell it that its step is there.  Once the stage carries this step's number, every earlier
                // round is over and the parity is unambiguous.
                int tries = 0;
                while (*reinterpret_cast<volatile int *>(&scales[st].tag) != ct && ++tries < p.wait_rounds) __nanosleep(20);
                ok = tries < p.wait_rounds;
                if (!ok) break;
            }
            ok = at_wait(full_a + 8 * st, own_parity, p.wait_rounds);
            if (!ok) break;
            own += WARPS;
            if (own >= kStages) {
                own -= kStages;
                own_parity ^= 1;
            }
            const uint32_t kt = ring_a + st * S::kStepBytes, vt = kt + kStep * D;
            const AtScales sc = scales[st];
            // S^T = K Q^T: kStep tokens x 8 NT rows
            float z[NT][MT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[nt][mt][e] = 0.f;
#pragma unroll
            for (int ch = 0; ch < kChunks; ch += 2) {
                uint32_t a[MT][2][4];  // [16 tokens][chunk][fragment]
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    uint32_t r[4];
                    at_ldsm(addr(kt, mt * 16 + (lane & 15), ch + (lane >> 4)), r);
                    AtCode<E4M3>::key(r[0], a[mt][0][0], a[mt][0][2]);
                    AtCode<E4M3>::key(r[1], a[mt][0][1], a[mt][0][3]);
                    AtCode<E4M3>::key(r[2], a[mt][1][0], a[mt][1][2]);
                    AtCode<E4M3>::key(r[3], a[mt][1][1], a[mt][1][3]);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint2 v = *reinterpret_cast<const uint2 *>(qp + (nt * 8 + g) * S::kQStride + (ch + x) * 16 + 4 * c);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) at_mma(z[nt][mt], a[mt][x], v.x, v.y);
                    }
                }
            }
            // scores, in base 2 and with the value scale's logarithm added
            const int tok0 = (step0 + ct) * kStep;
            const bool edge = tok0 + kStep - 1 > pmin || (p.window > 0 && tok0 <= pmax - p.window) || sc.sk[0] < 0.f ||
                              (MT > 1 && sc.sk[MT - 1] < 0.f);
            uint32_t pb[NT][MT][2];
            float mx[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (p.cap > 0.f) {
                            z[nt][mt][e] = at_capped(z[nt][mt][e] * (sc.sk[mt] * zscale), zcap) + sc.lsv[mt];
                        } else {
                            z[nt][mt][e] = z[nt][mt][e] * (sc.sk[mt] * zscale) + sc.lsv[mt];
                        }
                    }
                if (edge) {                    // (few steps: worked out here rather than kept in registers)
                    const int r0 = bt.rt * kRows, rl = min(kRows, bt.rows * p.G - r0) - 1, pos0 = bt.len - bt.rows;
                    const int last[2] = {pos0 + (r0 + min(rl, nt * 8 + 2 * c)) / p.G, pos0 + (r0 + min(rl, nt * 8 + 2 * c + 1)) / p.G};
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = tok0 + mt * 16 + g + (e >> 1) * 8, pos = last[e & 1];
                            if (j > pos || (p.window > 0 && j <= pos - p.window) || sc.sk[mt] < 0.f)
                                z[nt][mt][e] = -INFINITY;
                        }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mx[nt][e] = fmaxf(z[nt][0][e], z[nt][0][e + 2]);
                    if (MT > 1) mx[nt][e] = fmaxf(mx[nt][e], fmaxf(z[nt][MT - 1][e], z[nt][MT - 1][e + 2]));
                }
            }
            bool grows = false;
#pragma unroll
            for (int d = 4; d < 32; d <<= 1)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) mx[nt][e] = fmaxf(mx[nt][e], __shfl_xor_sync(0xffffffffu, mx[nt][e], d));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) grows |= mx[nt][e] - m[nt][e] > kLift + kLag;
            // The reference moves only when a score passes the one that set it by 2^4: rescaling the sums is as much
            // work as a step's softmax.  (The difference is the weights' exponent, so none of them passes 2^15.)
            if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float mn = fmaxf(m[nt][e], mx[nt][e] - kLift);
                        const float hf = mn == -INFINITY ? 1.f : at_half_exp2(m[nt][e] - mn), f = hf * hf;
                        l[nt][e] = l[nt][e] * hf * hf;     // 0 for the first keys
#pragma unroll
                        for (int ch = 0; ch < kChunks; ++ch) {
                            o[nt][ch][e] *= f;
                            o[nt][ch][e + 2] *= f;
                        }
                        m[nt][e] = mn;
                    }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float ref = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const float w0 = at_exp2(z[nt][mt][e] - ref), w1 = at_exp2(z[nt][mt][e + 2] - ref);
                        z[nt][mt][e] = w0;
                        z[nt][mt][e + 2] = w1;
                        l[nt][e] += (w0 + w1) * sc.rsv[mt];
                    }
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const __half2 w = __floats2half2_rn(z[nt][mt][2 * e], z[nt][mt][2 * e + 1]);
                        pb[nt][mt][e] = at_transpose(*reinterpret_cast<const uint32_t *>(&w));
                    }
            }
            if (E4M3 && edge) {
                // what lies where no token is may be a NaN, and 0 * NaN is one: zeros instead
                const int tok = lane % kStep;
                if (tok0 + tok >= bt.len || (MT > 1 && tok >= 16 ? sc.sk[MT - 1] : sc.sk[0]) < 0.f)
                    for (int x = 0; x < D; x += 16)
                        *reinterpret_cast<uint4 *>(eva_smem + (vt - base0) + (D >= 128 ? (x >> 7) * (kStep * 128) + tok * 128 + (x & 127)
                                                                                       : tok * 64 + x)) = make_uint4(0, 0, 0, 0);
                __syncwarp();
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");       // before the stage's next copy
            }
            // O^T += V^T P^T; at 16 tokens a step one load brings two chunks of dimensions.  `read` takes a register of each
            // load: the stage is handed back when their data are there.  The order of the instructions alone does not do it:
            // the next copy into a stage overtook the last load of a part's first step, and 32 dimensions got the values of
            // another step (seen in repeated calls on a cache in the L2).
            uint32_t read = 0;
            if constexpr (MT > 1) {
#pragma unroll
                for (int ch = 0; ch < kChunks; ++ch) {
                    uint32_t r[4], a[2][4];
                    at_ldsm_t(addr(vt, lane, ch), r);
                    read |= r[0];
                    AtCode<E4M3>::value(r[0], a[0][0], a[0][1]);
                    AtCode<E4M3>::value(r[1], a[0][2], a[0][3]);
                    AtCode<E4M3>::value(r[2], a[1][0], a[1][1]);
                    AtCode<E4M3>::value(r[3], a[1][2], a[1][3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        at_mma(o[nt][ch], a[0], pb[nt][0][0], pb[nt][0][1]);
                        at_mma(o[nt][ch], a[1], pb[nt][MT - 1][0], pb[nt][MT - 1][1]);
                    }
                }
            } else {
#pragma unroll
                for (int ch = 0; ch < kChunks; ch += 2) {
                    uint32_t r[4], a[2][4];
                    at_ldsm_t(addr(vt, lane & 15, ch + (lane >> 4)), r);
                    read |= r[0];
                    AtCode<E4M3>::value(r[0], a[0][0], a[0][1]);
                    AtCode<E4M3>::value(r[1], a[0][2], a[0][3]);
                    AtCode<E4M3>::value(r[2], a[1][0], a[1][1]);
                    AtCode<E4M3>::value(r[3], a[1][2], a[1][3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        at_mma(o[nt][ch], a[0], pb[nt][0][0], pb[nt][0][1]);
                        at_mma(o[nt][ch + 1], a[1], pb[nt][0][0], pb[nt][0][1]);
                    }
                }
            }
            __syncwarp();
            if ((lane | (read & p.nothing)) == 0) mbar_arrive(free_a + 8 * st);
        }
        if (!ok) break;
        {
            // The piece's sums: the warps of different steps meet in shared memory, once all are done with what the last
            // piece left there.
            if (!first) ok = all_here();
            if (!ok) break;
            first = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], d);
                    const int r = nt * 8 + 2 * c + e;
                    if (g == 0) mls[warp * kRows + r] = make_float2(m[nt][e], l[nt][e]);
                    float *dst = os + (size_t)(warp * kRows + r) * S::kOStride + 2 * g;
#pragma unroll
                    for (int ch = 0; ch < kChunks; ++ch)
                        *reinterpret_cast<float2 *>(dst + ch * 16) = make_float2(o[nt][ch][e], o[nt][ch][e + 2]);
                }
            ok = meet();
            if (!ok) break;
            const int e0 = bt.rt * kRows, erows = min(kRows, bt.rows * p.G - e0), eh = bt.h, erow = bt.row;
            const int c0 = bt.c0, c1 = bt.c1, grid = gridDim.x, me = blockIdx.x;
            auto slot_of = [&](int cc) { return (size_t)(2 * cc + (cc == c0)); };    // a CTA begins at most one shared item
            auto emit = [&](int r, int x, const float4 &v, float mm, float ll) {
                const int i = (e0 + r) / p.G, hq = eh * p.G + (e0 + r) - i * p.G;
                const float f = ll > 0.f ? kAtSumScale / ll : 0.f;
                const long long at = ((long long)(erow + i) * p.Hq + hq) * D + x;
                if (p.out_f32) {
                    *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) =
                        make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
                } else {
                    const __half2 a = __floats2half2_rn(v.x * f, v.y * f), b = __floats2half2_rn(v.z * f, v.w * f);
                    *reinterpret_cast<uint2 *>(static_cast<__half *>(p.out) + at) =
                        make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
                }
                if (p.lse && x == 0)
                    p.lse[(long long)(erow + i) * p.Hq + hq] = ll == 0.f ? -INFINITY : (mm + (log2f(ll) - kAtLog2SumScale)) * 0.6931471805599453f;
            };
#pragma unroll 1
            for (int i = tid; i < erows * (D / 4); i += 32 * WARPS) {
                const int r = i / (D / 4), x = (i - r * (D / 4)) * 4;
                float mm = -INFINITY;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) mm = fmaxf(mm, mls[w * kRows + r].x);
                const float ref = mm == -INFINITY ? 0.f : mm;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                float ll = 0.f;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) {
                    const float2 ml = mls[w * kRows + r];
                    const float hf = at_half_exp2(ml.x - ref), f = hf * hf;
                    const float4 y = *reinterpret_cast<const float4 *>(os + (size_t)(w * kRows + r) * S::kOStride + x);
                    v.x += y.x * f; v.y += y.y * f; v.z += y.z * f; v.w += y.w * f;
                    ll += ml.y * hf * hf;
                }
                if (c0 == c1) {
                    emit(r, x, v, mm, ll);
                } else {
                    reinterpret_cast<float4 *>(p.part)[(slot_of(me) * kRows + r) * (D / 4) + x / 4] = v;
                    if (x == 0) p.part_ml[slot_of(me) * kRows + r] = make_float2(mm, ll);
                }
            }
            // Shared items.  Parts are joined kAtSegment (or a multiple, for very many) at a time by the last of them
            // to finish, and the segments by the last segment: from L2, many loads in flight.
            if (c0 != c1) {
                int seg = kAtSegment;
                while (seg * seg < c1 - c0 + 1) seg += kAtSegment;
                const int sc0 = c0 + (me - c0) / seg * seg, sc1 = min(c1, sc0 + seg - 1), segs = (c1 - c0) / seg + 1;
                float *top = reinterpret_cast<float *>(mls);
                // counts one more of `all` in; true for the last, which then sees what the others wrote
                auto last_of = [&](int *counter, int all) {
                    bool r = meet();
                    if (tid == 0) {
                        __threadfence();       // of what all warps wrote before they met
                        const bool last = atomicAdd(counter, 1) == all - 1;
                        if (last) {
                            *counter = 0;
                            __threadfence();
                        }
                        flag[0] = last;
                    }
                    r = meet() && r;
                    ok = r;
                    return r && flag[0];
                };
                auto join = [&](int from, int to, int by, bool final) {
                    constexpr int kLanes = S::kJoinLanes, kBatch = 8;
                    {
                        const int r = tid / kLanes;
                        float mm = -INFINITY;
                        if (r < erows)
                            for (int cc = from + tid % kLanes * by; cc <= to; cc += kLanes * by)
                                mm = fmaxf(mm, __ldcg(p.part_ml + slot_of(cc) * kRows + r).x);
#pragma unroll
                        for (int d = kLanes / 2; d > 0; d >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, d));
                        if (r < erows && tid % kLanes == 0) top[r] = mm;
                    }
                    if (!(ok = meet())) return;
#pragma unroll 1
                    for (int i = tid; i < erows * (D / 4); i += 32 * WARPS) {
                        const int r = i / (D / 4), x = i - r * (D / 4);
                        const float mm = top[r], ref = mm == -INFINITY ? 0.f : mm;
                        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                        float ll = 0.f;
                        for (int cb = from; cb <= to; cb += kBatch * by) {
                            float2 ml[kBatch];
                            float4 y[kBatch];
#pragma unroll
                            for (int j = 0; j < kBatch; ++j) {
                                const size_t at = slot_of(min(cb + j * by, to)) * kRows + r;
                                ml[j] = __ldcg(p.part_ml + at);
                                y[j] = __ldcg(reinterpret_cast<const float4 *>(p.part) + at * (D / 4) + x);
                            }
#pragma unroll
                            for (int j = 0; j < kBatch; ++j) {
                                const float hf = cb + j * by <= to ? at_half_exp2(ml[j].x - ref) : 0.f, f = hf * hf;
                                v.x += y[j].x * f; v.y += y[j].y * f; v.z += y[j].z * f; v.w += y[j].w * f;
                                ll += ml[j].y * hf * hf;
                            }
                        }
                        if (final) {
                            emit(r, 4 * x, v, mm, ll);
                        } else {               // over the segment's first part; the maxima and sums once all have read
                            reinterpret_cast<float4 *>(p.part)[(slot_of(from) * kRows + r) * (D / 4) + x] = v;
                            if (x == 0) top[kRows + r] = ll;
                        }
                    }
                    if (!final) {
                        if (!(ok = meet())) return;
                        if (tid < erows) p.part_ml[slot_of(from) * kRows + tid] = make_float2(top[tid], top[kRows + tid]);
                    }
                };
                if (last_of(p.counters + (sc0 == c0 ? 0 : grid) + sc0, sc1 - sc0 + 1)) {
                    join(sc0, sc1, 1, segs == 1);
                    if (ok && segs > 1 && last_of(p.counters + 2 * grid + c0, segs)) join(c0, c0 + (segs - 1) * seg, seg, true);
                }
                if (!ok) break;
            }
            come();
        }
        if (lane == 0) mbar_arrive(pfree_a + 8 * ps);
        if (++ps == kAtPieces) {
            ps = 0;
            pparity ^= 1;
        }
    }
    if (!ok && lane == 0) atomicOr(p.status, kAtStatusWait);
}

}  // namespace eva
