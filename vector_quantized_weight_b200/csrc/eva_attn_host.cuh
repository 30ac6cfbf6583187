// eva_attn_host.cuh -- host side of the rotary-position, cache and attention
// entry points (see include/eva_vq.h): argument validation, handle-owned
// device memory, the choice of kernel instance and the launches.  Part of
// eva_vq.cu's translation unit.
#pragma once
#include "eva_attend.cuh"
#include "eva_kv.cuh"
#include "eva_rope.cuh"

struct eva_rope {
    eva_rope_desc desc;
    int device = 0, sm_count = 0;
    void *memory = nullptr;                // what follows
    unsigned long long *turns = nullptr;   // [rotary_dim / 2]
    __half *w[2] = {nullptr, nullptr};     // norm weights of queries and keys
    float magnitude = 1.f;
};

struct eva_kv {
    eva_kv_desc desc;
    int device = 0, sm_count = 0;
    uint8_t *pages[2] = {nullptr, nullptr};   // the caller's
    float *scale[2] = {nullptr, nullptr};
    AttendMaps maps;
    uint8_t *memory = nullptr;             // what follows; the counters and the status word first
    int *counters = nullptr, *status = nullptr;
    float *part = nullptr;
    float2 *part_ml = nullptr;
    int max_grid = 0;
    int64_t workspace_bytes = 0;
    // attention instances: items of 8, 16 and 24 or 32 rows
    struct Plan { const void *fn = nullptr; int rows = 0, stages = 0, grid = 0, threads = 0; size_t smem = 0; } plan[3];
    int last_plan = 0;
    int inject_wait_rounds = 0;        // failure-detection test hook, as for the linear
};

namespace {

// The handle's device is made current for the call and the caller's put back.
struct DeviceGuard {
    int before = -1;
    bool ok = true;
    explicit DeviceGuard(int dev) {
        int cur = 0;
        if (cudaGetDevice(&cur) != cudaSuccess) { ok = false; return; }
        if (cur == dev) return;
        before = cur;
        ok = cudaSetDevice(dev) == cudaSuccess;
    }
    ~DeviceGuard() {
        if (before >= 0) cudaSetDevice(before);
    }
};

// The current device, its SMs and the shared memory a block may have; attributes, as the whole property structure takes
// most of a millisecond.
eva_status_t sm100_device(int *dev, int *sms, int *optin) {
    int major = 0;
    if (cudaGetDevice(dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev) != cudaSuccess ||
        cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess ||
        cudaDeviceGetAttribute(optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, *dev) != cudaSuccess) return EVA_ERR_NO_DEVICE;
    return major == 10 ? EVA_OK : EVA_ERR_NO_DEVICE;
}

bool valid_dtype(eva_dtype_t t) { return t == EVA_F16 || t == EVA_F32; }
int dtype_bytes(eva_dtype_t t) { return t == EVA_F32 ? 4 : 2; }
bool finite_pos(double v) { return std::isfinite(v) && v > 0; }

eva_status_t validate_rope(const eva_rope_desc *d) {
    if (!d) return EVA_ERR_INVALID_ARG;
    if (d->q_heads < 0 || d->kv_heads < 0 || d->q_heads > 65536 || d->kv_heads > 65536 ||
        d->q_heads + d->kv_heads < 1) return EVA_ERR_INVALID_ARG;
    if (d->head_dim < 1 || d->rotary_dim < 0 || d->rotary_dim > d->head_dim || d->rotary_dim % 2) return EVA_ERR_INVALID_ARG;
    if (d->head_dim > 1024) return EVA_ERR_UNSUPPORTED;
    if (d->layout != EVA_ROPE_HALF && d->layout != EVA_ROPE_INTERLEAVED) return EVA_ERR_INVALID_ARG;
    if (!valid_dtype(d->in_dtype) || !valid_dtype(d->out_dtype)) return EVA_ERR_INVALID_ARG;
    if (d->norm != 0 && d->norm != 1) return EVA_ERR_INVALID_ARG;
    if (d->norm && !(std::isfinite(d->eps) && d->eps >= 0 && std::isfinite(d->weight_offset))) return EVA_ERR_INVALID_ARG;
    if (!(std::isfinite(d->magnitude) && d->magnitude >= 0)) return EVA_ERR_INVALID_ARG;
    if (d->rotary_dim == 0) return EVA_OK;
    if (!finite_pos(d->theta)) return EVA_ERR_INVALID_ARG;
    switch (d->scaling) {
        case EVA_ROPE_UNSCALED: return EVA_OK;
        case EVA_ROPE_LINEAR: return finite_pos(d->factor) ? EVA_OK : EVA_ERR_INVALID_ARG;
        case EVA_ROPE_NTK: return finite_pos(d->factor) && d->rotary_dim > 2 ? EVA_OK : EVA_ERR_INVALID_ARG;
        case EVA_ROPE_YARN:
            return finite_pos(d->factor) && finite_pos(d->original) && finite_pos(d->low) && finite_pos(d->high) &&
                           d->low <= d->high && d->theta > 1 ? EVA_OK : EVA_ERR_INVALID_ARG;
        case EVA_ROPE_BANDS:
            return finite_pos(d->factor) && finite_pos(d->original) && finite_pos(d->low) && finite_pos(d->high) &&
                           d->low < d->high ? EVA_OK : EVA_ERR_INVALID_ARG;
    }
    return EVA_ERR_INVALID_ARG;
}

// Radians a position of pair i (see the header).
long double rope_frequency(const eva_rope_desc &d, int i) {
    const long double R = d.rotary_dim, two_pi = 6.283185307179586476925286766559L;
    long double theta = d.theta;
    if (d.scaling == EVA_ROPE_NTK) theta *= powl(d.factor, R / (R - 2));
    const long double f = powl(theta, -2.0L * i / R);
    if (d.scaling == EVA_ROPE_LINEAR) return f / d.factor;
    if (d.scaling == EVA_ROPE_YARN) {
        auto edge = [&](double beta) { return R * logl(d.original / (two_pi * beta)) / (2 * logl(theta)); };
        const long double lo = std::max(floorl(edge(d.high)), 0.0L), hi = std::min(ceill(edge(d.low)), R - 1);
        const long double ramp = std::min(std::max((i - lo) / std::max(hi - lo, 0.001L), 0.0L), 1.0L);
        return f * (1 - ramp) + f / d.factor * ramp;
    }
    if (d.scaling == EVA_ROPE_BANDS) {
        const long double turns = d.original * f / two_pi;     // over the original context
        const long double keep = std::min(std::max((turns - d.low) / ((long double)d.high - d.low), 0.0L), 1.0L);
        return f / d.factor * (1 - keep) + f * keep;
    }
    return f;
}

// A turn is 2^64: the fraction of a turn a position, whole turns dropped.
unsigned long long rope_turns(long double radians) {
    const long double turns = radians / 6.283185307179586476925286766559L;
    const long double frac = turns - floorl(turns);
    const long double scaled = roundl(ldexpl(frac, 64));
    return scaled >= ldexpl(1.0L, 64) ? 0ull : (unsigned long long)scaled;
}

using RopeFn = void (*)(RopeParams);
template <typename TI, typename TO>
RopeFn rope_fn(int lanes) {
    switch (lanes) {
        case 4: return eva_rope_kernel<TI, TO, 4>;
        case 8: return eva_rope_kernel<TI, TO, 8>;
        case 16: return eva_rope_kernel<TI, TO, 16>;
        case 32: return eva_rope_kernel<TI, TO, 32>;
    }
    return eva_rope_any_kernel<TI, TO>;
}
RopeFn rope_fn(eva_dtype_t in, eva_dtype_t out, int lanes) {
    if (in == EVA_F16) return out == EVA_F16 ? rope_fn<__half, __half>(lanes) : rope_fn<__half, float>(lanes);
    return out == EVA_F16 ? rope_fn<float, __half>(lanes) : rope_fn<float, float>(lanes);
}

eva_status_t validate_kv(const eva_kv_desc *d) {
    if (!d) return EVA_ERR_INVALID_ARG;
    if (d->q_heads < 1 || d->kv_heads < 1 || d->q_heads > 65535 || d->kv_heads > 65535 || d->q_heads % d->kv_heads)
        return EVA_ERR_INVALID_ARG;
    if (d->head_dim < 1 || d->page_size < 1 || d->num_pages < 1 || d->max_seqs < 1 || d->max_pages < 1)
        return EVA_ERR_INVALID_ARG;
    if (d->cache_dtype != EVA_CACHE_INT8 && d->cache_dtype != EVA_CACHE_E4M3) return EVA_ERR_INVALID_ARG;
    if (!valid_dtype(d->out_dtype) || d->window < 0 || d->window > (1 << 30)) return EVA_ERR_INVALID_ARG;
    if (!(std::isfinite(d->softcap) && d->softcap >= 0) || !(std::isfinite(d->scale) && d->scale >= 0)) return EVA_ERR_INVALID_ARG;
    if (d->softcap > 1e30f) return EVA_ERR_UNSUPPORTED;        // scores over it would be subnormal
    if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) return EVA_ERR_UNSUPPORTED;
    if (d->page_size != 16 && d->page_size != 32 && d->page_size != 64 && d->page_size != 128 && d->page_size != 256)
        return EVA_ERR_UNSUPPORTED;
    // token positions and rows of the cache are 32-bit
    if ((int64_t)d->max_pages * d->page_size > (1 << 30)) return EVA_ERR_UNSUPPORTED;
    if ((int64_t)d->num_pages * d->kv_heads * d->page_size > INT32_MAX) return EVA_ERR_UNSUPPORTED;
    return EVA_OK;
}

using AttendFn = void (*)(const AttendMaps, AttendParams);

// One attention instance: its shared memory and the CTAs the GPU holds at once.
template <int D, int NT, int WARPS, int CTAS, bool E4M3>
cudaError_t plan_attend(eva_kv *h, int i, int optin) {
    using S = AtShape<D, NT, WARPS, CTAS>;
    auto fn = eva_attend_kernel<D, NT, WARPS, CTAS, E4M3>;
    eva_kv::Plan &p = h->plan[i];
    p.fn = reinterpret_cast<const void *>(fn);
    p.rows = S::kRows;
    p.threads = S::kThreads;
    p.stages = S::kStages;
    p.smem = S::kSmem;
    if (p.smem > (size_t)optin) return cudaErrorInvalidConfiguration;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)p.smem);
    if (e != cudaSuccess) return e;
    int per_sm = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, fn, S::kThreads, p.smem);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    p.grid = per_sm * h->sm_count;
    return cudaSuccess;
}
// Warps and CTAs an SM, all measured (us, 517 tokens of 32 heads / 268 MB of 64 sequences / of one): for up to eight
// rows two CTAs of 5 working warps 10.7 / 57.8 / 54.3, three of 4 11.7 / 55.5 / 54.0, two of 4 11.0 / 58.4 / 54.5,
// four of 3 12.6 / 56.7 / 57.5, two of 7 11.5 / 61.9 / 55.9; heads of 256 two of 4 50.0 against two of 5 52.4.  The
// first is taken for all of them: a ninth less on the short call for 4 % more on many sequences.
// Many rows take registers: one CTA of 7, with items of 32 rows; of 24 for int8 at heads of 128, where 32 spill a
// little (128, 256, 512, 1024 rows over 8191 tokens: 24 an item 38.4, 59.4, 102, 185; 32 39.2, 60.4, 97, 177).
template <int D, bool E4M3>
cudaError_t plan_attends(eva_kv *h, int optin) {
    if constexpr (D <= 128) {
        cudaError_t e = plan_attend<D, 1, 5, 2, E4M3>(h, 0, optin);
        if (e == cudaSuccess) e = plan_attend<D, 2, 5, 2, E4M3>(h, 1, optin);
        if (e == cudaSuccess) e = plan_attend<D, D < 128 || E4M3 ? 4 : 3, 7, 1, E4M3>(h, 2, optin);
        return e;
    } else {     // items of 8 rows for all: of 16 (one CTA of 7 warps) 34.2 against 29.4 us for three drafted tokens of
                 // eight queries a key head, 39.3 / 36.9 for five, but 74 / 91 for 128 rows over 8191 tokens
        return plan_attend<D, 1, 4, 2, E4M3>(h, 0, optin);
    }
}
cudaError_t plan_attends(eva_kv *h, int optin) {
    const bool e4 = h->desc.cache_dtype == EVA_CACHE_E4M3;
    switch (h->desc.head_dim) {
        case 64: return e4 ? plan_attends<64, true>(h, optin) : plan_attends<64, false>(h, optin);
        case 128: return e4 ? plan_attends<128, true>(h, optin) : plan_attends<128, false>(h, optin);
    }
    return e4 ? plan_attends<256, true>(h, optin) : plan_attends<256, false>(h, optin);
}

// The cache as rows of head_dim bytes; a box is 16 or 32 tokens.  Rows of 256 bytes are two halves of 128, the
// swizzle's width: a third dimension, so that one copy brings both.
eva_status_t cache_map(CUtensorMap *m, const eva_kv_desc &d, void *pages) {
    using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &found) != cudaSuccess || !fn ||
        found != cudaDriverEntryPointSuccess) return EVA_ERR_CUDA;
    const bool wide = d.head_dim > 128;
    const cuuint64_t dims[3] = {(cuuint64_t)std::min(d.head_dim, 128), (cuuint64_t)d.num_pages * d.kv_heads * d.page_size, 2};
    const cuuint64_t strides[2] = {(cuuint64_t)d.head_dim, 128};
    const cuuint32_t box[3] = {(cuuint32_t)dims[0], (cuuint32_t)std::min(d.page_size, wide ? 16 : 32), 2};
    const cuuint32_t ones[3] = {1, 1, 1};
    const CUresult r = reinterpret_cast<Encode>(fn)(
        m, CU_TENSOR_MAP_DATA_TYPE_UINT8, wide ? 3 : 2, pages, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
        d.head_dim >= 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? EVA_OK : EVA_ERR_CUDA;
}

void free_rope(eva_rope *h) {
    if (!h) return;
    DeviceGuard guard(h->device);
    if (h->memory) cudaFree(h->memory);
    delete h;
}

void free_kv(eva_kv *h) {
    if (!h) return;
    DeviceGuard guard(h->device);
    if (h->memory) cudaFree(h->memory);
    delete h;
}

// Packed inputs and outputs: non-negative counts, 16-byte rows.
bool row_ok(const void *p, int64_t ld, int64_t least, int bytes) {
    return p && aligned16(p) && ld >= least && ld * bytes % 16 == 0;
}

int log2_of(int pow2) {
    int l = 0;
    while (pow2 >> (l + 1)) ++l;
    return l;
}

KvTokens kv_tokens(const eva_kv *h, const int32_t *starts, const int32_t *lens, const int32_t *table, int B, int T) {
    KvTokens t;
    t.starts = starts;
    t.lens = lens;
    t.table = table;
    t.B = B;
    t.T = T;
    t.page = h->desc.page_size;
    t.log_page = log2_of(t.page);
    t.max_pages = h->desc.max_pages;
    t.num_pages = h->desc.num_pages;
    return t;
}

bool kv_call_ok(const eva_kv *h, const int32_t *starts, const int32_t *lens, const int32_t *table, int B, int64_t T) {
    return h && starts && lens && table && B >= 1 && B <= h->desc.max_seqs && T >= 0 && T <= (1 << 30);
}

}  // namespace

extern "C" {

eva_status_t eva_rope_create(eva_rope_t *out, const eva_rope_desc *desc, const void *q_weight, const void *k_weight,
                             eva_stream_t stream) {
    if (!out) return EVA_ERR_INVALID_ARG;
    *out = nullptr;
    eva_status_t st = validate_rope(desc);
    if (st != EVA_OK) return st;
    if (!desc->norm && (q_weight || k_weight)) return EVA_ERR_INVALID_ARG;
    if (!aligned16(q_weight) || !aligned16(k_weight)) return EVA_ERR_INVALID_ARG;
    int dev = 0, sms = 0, optin = 0;
    st = sm100_device(&dev, &sms, &optin);
    if (st != EVA_OK) return st;
    eva_rope *h = new (std::nothrow) eva_rope();
    if (!h) return EVA_ERR_OOM;
    h->desc = *desc;
    h->device = dev;
    h->sm_count = sms;
    if (desc->magnitude > 0) h->magnitude = (float)desc->magnitude;
    else if (desc->scaling == EVA_ROPE_YARN && desc->factor > 1) h->magnitude = (float)(0.1 * std::log(desc->factor) + 1.0);
    unsigned long long turns[512];
    const int pairs = desc->rotary_dim / 2;
    for (int i = 0; i < pairs; ++i) turns[i] = rope_turns(rope_frequency(*desc, i));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const size_t table = (pairs * sizeof(turns[0]) + 15) / 16 * 16, weight = ((size_t)desc->head_dim * sizeof(__half) + 15) / 16 * 16;
    uint8_t *m = nullptr;
    cudaError_t e = dalloc(&m, table + 2 * weight, nullptr);
    h->memory = m;
    if (e == cudaSuccess && pairs) {
        h->turns = reinterpret_cast<unsigned long long *>(m);
        e = cudaMemcpyAsync(h->turns, turns, pairs * sizeof(turns[0]), cudaMemcpyHostToDevice, s);
    }
    const void *w[2] = {q_weight, k_weight};
    for (int i = 0; i < 2; ++i) {
        if (e != cudaSuccess || !w[i]) continue;
        h->w[i] = reinterpret_cast<__half *>(m + table + i * weight);
        e = cudaMemcpyAsync(h->w[i], w[i], desc->head_dim * sizeof(__half), cudaMemcpyDeviceToDevice, s);
    }
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);   // the table is this call's stack; the weights may go
    if (e != cudaSuccess) {
        free_rope(h);
        return cuda_status(e);
    }
    *out = h;
    return EVA_OK;
}

eva_status_t eva_rope_run(eva_rope_t h, const void *q, int64_t ldq, const void *k, int64_t ldk, const int32_t *positions,
                          int32_t T, void *q_out, int64_t ldqo, void *k_out, int64_t ldko, eva_stream_t stream) {
    if (!h || T < 0 || T > (1 << 30)) return EVA_ERR_INVALID_ARG;
    if (T == 0) return EVA_OK;
    const eva_rope_desc &d = h->desc;
    if (d.rotary_dim && !positions) return EVA_ERR_INVALID_ARG;
    const int64_t wq = (int64_t)d.q_heads * d.head_dim, wk = (int64_t)d.kv_heads * d.head_dim;
    if (d.q_heads && (!q || !q_out || ldq < wq || ldqo < wq)) return EVA_ERR_INVALID_ARG;
    if (d.kv_heads && (!k || !k_out || ldk < wk || ldko < wk)) return EVA_ERR_INVALID_ARG;
    DeviceGuard guard(h->device);
    if (!guard.ok) return EVA_ERR_CUDA;
    RopeParams p = {};
    p.q = q; p.k = k; p.qo = q_out; p.ko = k_out;
    p.ldq = ldq; p.ldk = ldk; p.ldqo = ldqo; p.ldko = ldko;
    p.pos = positions;
    p.turns = h->turns;
    p.qw = h->w[0]; p.kw = h->w[1];
    p.T = T; p.Hq = d.q_heads; p.H = d.q_heads + d.kv_heads; p.D = d.head_dim; p.R = d.rotary_dim;
    p.interleaved = d.layout == EVA_ROPE_INTERLEAVED;
    p.norm = d.norm;
    p.eps = d.eps; p.offset = d.weight_offset; p.magnitude = h->magnitude;
    // 16-byte accesses where every row allows them (and 8 rows' offsets fit 32 bits)
    const int bi = dtype_bytes(d.in_dtype), bo = dtype_bytes(d.out_dtype);
    auto wide = [](const void *a, int64_t ld, int bytes) { return aligned16(a) && ld * bytes % 16 == 0 && ld <= 1 << 27; };
    int lanes = 0;
    if (d.head_dim % 16 == 0 && (d.rotary_dim % 16 == 0 || p.interleaved) && d.head_dim <= 512 &&
        (!d.q_heads || (wide(q, ldq, bi) && wide(q_out, ldqo, bo))) &&
        (!d.kv_heads || (wide(k, ldk, bi) && wide(k_out, ldko, bo))))
        for (lanes = 4; lanes * 16 < d.head_dim;) lanes *= 2;
    // Few tokens: one a CTA, and as many heads as its lanes hold at once, until that fills the GPU.  Then whole tokens, 1
    // to 8 a CTA: a CTA's cost is its turns and about two more for the sines, its waves (three CTAs an SM) end half
    // a wave late.  (8192 tokens of 72 heads: 4 a CTA 63 us, 8 67; 1777 of 40 heads: 4 10.9, 1 12.0.)
    const int groups = lanes ? kRopeThreads / lanes : kRopeThreads / 32;
    p.tb = 1;
    p.hs = std::min(p.H, groups);
    if ((int64_t)T * ((p.H + p.hs - 1) / p.hs) > (int64_t)h->sm_count * 4) {
        p.hs = p.H;
        double least = 0;
        for (int tb = 1; tb <= 8; tb *= 2) {
            const double cost = ((double)((T + tb - 1) / tb) / (3 * h->sm_count) + 0.5) * ((tb * (int64_t)p.H + groups - 1) / groups + 2);
            if (tb == 1 || cost < least * 0.99) {
                least = cost;
                p.tb = tb;
            }
        }
    }
    const dim3 grid((unsigned)((T + p.tb - 1) / p.tb), (unsigned)((p.H + p.hs - 1) / p.hs));
    const size_t smem = (size_t)p.tb * rope_row(d.rotary_dim) * 2 * sizeof(float) + (lanes && d.norm ? 2 * d.head_dim * sizeof(float) : 0);
    return cuda_status(launch_pdl(rope_fn(d.in_dtype, d.out_dtype, lanes), grid, dim3(kRopeThreads), smem,
                                  reinterpret_cast<cudaStream_t>(stream), 0, p));
}

eva_status_t eva_rope_destroy(eva_rope_t h) {
    free_rope(h);
    return EVA_OK;
}

eva_status_t eva_kv_create(eva_kv_t *out, const eva_kv_desc *desc, void *k_pages, void *v_pages, float *k_scale,
                           float *v_scale, eva_stream_t stream) {
    if (!out) return EVA_ERR_INVALID_ARG;
    *out = nullptr;
    eva_status_t st = validate_kv(desc);
    if (st != EVA_OK) return st;
    if (!k_pages || !v_pages || !k_scale || !v_scale || !aligned16(k_pages) || !aligned16(v_pages) ||
        !aligned16(k_scale) || !aligned16(v_scale)) return EVA_ERR_INVALID_ARG;
    int dev = 0, sms = 0, optin = 0;
    st = sm100_device(&dev, &sms, &optin);
    if (st != EVA_OK) return st;
    eva_kv *h = new (std::nothrow) eva_kv();
    if (!h) return EVA_ERR_OOM;
    h->desc = *desc;
    h->device = dev;
    h->sm_count = sms;
    h->pages[0] = static_cast<uint8_t *>(k_pages);
    h->pages[1] = static_cast<uint8_t *>(v_pages);
    h->scale[0] = k_scale;
    h->scale[1] = v_scale;
    st = cache_map(&h->maps.k, *desc, k_pages);
    if (st == EVA_OK) st = cache_map(&h->maps.v, *desc, v_pages);
    if (st != EVA_OK) {
        free_kv(h);
        return st;
    }
    cudaError_t e = plan_attends(h, optin);
    size_t slots = 0;
    for (const auto &p : h->plan) {
        slots = std::max(slots, (size_t)2 * p.grid * p.rows);
        h->max_grid = std::max(h->max_grid, p.grid);
    }
    auto chk = [&](cudaError_t r) { if (e == cudaSuccess) e = r; };
    const size_t words = ((size_t)(3 * h->max_grid + 1) * sizeof(int) + 255) / 256 * 256;
    const size_t outs = slots * desc->head_dim * sizeof(float);
    if (e == cudaSuccess) chk(dalloc(&h->memory, words + outs + slots * sizeof(float2), &h->workspace_bytes));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (e == cudaSuccess) {
        h->counters = reinterpret_cast<int *>(h->memory);
        h->status = h->counters + 3 * h->max_grid;
        h->part = reinterpret_cast<float *>(h->memory + words);
        h->part_ml = reinterpret_cast<float2 *>(h->memory + words + outs);
        chk(cudaMemsetAsync(h->memory, 0, words, s));
    }
    if (e == cudaSuccess) chk(cudaStreamSynchronize(s));   // any stream may use the handle from here on
    if (e != cudaSuccess) {
        free_kv(h);
        return cuda_status(e);
    }
    *out = h;
    return EVA_OK;
}

eva_status_t eva_kv_append(eva_kv_t h, const void *k, int64_t ldk, const void *v, int64_t ldv, eva_dtype_t in_dtype,
                           const int32_t *starts, const int32_t *lens, const int32_t *page_table, int32_t B, int32_t T,
                           eva_stream_t stream) {
    if (!kv_call_ok(h, starts, lens, page_table, B, T) || !valid_dtype(in_dtype)) return EVA_ERR_INVALID_ARG;
    if (T == 0) return EVA_OK;
    const eva_kv_desc &d = h->desc;
    const int64_t width = (int64_t)d.kv_heads * d.head_dim;
    if (!row_ok(k, ldk, width, dtype_bytes(in_dtype)) || !row_ok(v, ldv, width, dtype_bytes(in_dtype)))
        return EVA_ERR_INVALID_ARG;
    DeviceGuard guard(h->device);
    if (!guard.ok) return EVA_ERR_CUDA;
    KvAppendParams p = {};
    p.tok = kv_tokens(h, starts, lens, page_table, B, T);
    p.x[0] = k; p.x[1] = v;
    p.ld[0] = ldk; p.ld[1] = ldv;
    for (int i = 0; i < 2; ++i) {
        p.pages[i] = h->pages[i];
        p.scale[i] = h->scale[i];
    }
    p.H = d.kv_heads;
    p.D = d.head_dim;
    p.log_d = log2_of(p.D);
    p.status = h->status;
    // n tokens lie on at most n / page + 2 pages, and on at most n
    const int64_t units = std::min<int64_t>(T, T / d.page_size + 2 * (int64_t)B);
    const dim3 grid((unsigned)units, (unsigned)d.kv_heads, 2);
    const bool e4 = d.cache_dtype == EVA_CACHE_E4M3;
    auto fn = in_dtype == EVA_F16 ? (e4 ? eva_kv_append_kernel<__half, true> : eva_kv_append_kernel<__half, false>)
                                  : (e4 ? eva_kv_append_kernel<float, true> : eva_kv_append_kernel<float, false>);
    return cuda_status(launch_pdl(fn, grid, dim3(kKvThreads), 0, reinterpret_cast<cudaStream_t>(stream), 0, p));
}

eva_status_t eva_kv_read(eva_kv_t h, const int32_t *starts, const int32_t *begins, const int32_t *page_table, int32_t B,
                         int32_t T, eva_dtype_t out_dtype, void *k_out, void *v_out, eva_stream_t stream) {
    if (!kv_call_ok(h, starts, begins, page_table, B, T) || !valid_dtype(out_dtype)) return EVA_ERR_INVALID_ARG;
    if (T == 0) return EVA_OK;
    if ((!k_out && !v_out) || !aligned16(k_out) || !aligned16(v_out)) return EVA_ERR_INVALID_ARG;
    DeviceGuard guard(h->device);
    if (!guard.ok) return EVA_ERR_CUDA;
    KvReadParams p = {};
    p.tok = kv_tokens(h, starts, begins, page_table, B, T);
    // a warp's lookups serve up to 8 rows, once that leaves enough warps
    p.rows = 1;
    while (p.rows < 8 && T >= (int64_t)h->sm_count * 32 * p.rows) p.rows *= 2;
    for (int i = 0; i < 2; ++i) {
        p.pages[i] = h->pages[i];
        p.scale[i] = h->scale[i];
    }
    p.out[0] = k_out; p.out[1] = v_out;
    p.H = h->desc.kv_heads;
    p.D = h->desc.head_dim;
    p.log_d = log2_of(p.D);
    p.status = h->status;
    const dim3 grid(blocks_for(T, kKvThreads / 32 * p.rows), 2);
    const bool e4 = h->desc.cache_dtype == EVA_CACHE_E4M3;
    auto fn = out_dtype == EVA_F16 ? (e4 ? eva_kv_read_kernel<__half, true> : eva_kv_read_kernel<__half, false>)
                                   : (e4 ? eva_kv_read_kernel<float, true> : eva_kv_read_kernel<float, false>);
    return cuda_status(launch_pdl(fn, grid, dim3(kKvThreads), 0, reinterpret_cast<cudaStream_t>(stream), 0, p));
}

eva_status_t eva_kv_attend(eva_kv_t h, const void *q, int64_t ldq, const int32_t *starts, const int32_t *lens,
                           const int32_t *page_table, int32_t B, int32_t T, void *out, float *lse, eva_stream_t stream) {
    if (!kv_call_ok(h, starts, lens, page_table, B, T)) return EVA_ERR_INVALID_ARG;
    if (T == 0) return EVA_OK;
    const eva_kv_desc &d = h->desc;
    if (!row_ok(q, ldq, (int64_t)d.q_heads * d.head_dim, 2) || !out || !aligned16(out)) return EVA_ERR_INVALID_ARG;
    if ((int64_t)T * (d.q_heads / d.kv_heads) > (1 << 30)) return EVA_ERR_UNSUPPORTED;      // rows of a key head are 32-bit
    DeviceGuard guard(h->device);
    if (!guard.ok) return EVA_ERR_CUDA;
    AttendParams p = {};
    p.tok = kv_tokens(h, starts, lens, page_table, B, T);
    p.q = static_cast<const __half *>(q);
    p.ldq = ldq;
    p.k_scale = h->scale[0];
    p.v_scale = h->scale[1];
    p.out = out;
    p.lse = lse;
    p.part = h->part;
    p.part_ml = h->part_ml;
    p.counters = h->counters;
    p.status = h->status;
    p.Hq = d.q_heads;
    p.H = d.kv_heads;
    p.G = d.q_heads / d.kv_heads;
    p.window = d.window;
    p.out_f32 = d.out_dtype == EVA_F32;
    p.min_steps = 16;
    p.inject = h->inject_wait_rounds > 0 ? 1 : h->inject_wait_rounds < 0 ? 2 : 0;
    p.wait_rounds = p.inject ? std::abs(h->inject_wait_rounds) : kWaitRounds;
    h->inject_wait_rounds = 0;
    p.scale = d.scale > 0 ? d.scale : 1.0f / std::sqrt((float)d.head_dim);
    p.cap = d.softcap;
    // Rows of a sequence and key head, on average (the real counts are on the device).  Up to 64, items of 16 rows with
    // more warps an SM (us, items of 16 / of 24 or 32: 32 rows 26 / 33, 40 rows 18 / 23, 64 rows 22.2 / 22.9, 128 rows
    // 40 / 37, 512 rows 108 / 100).
    const int64_t rows = (T + B - 1) / B * (int64_t)p.G;
    int i = rows <= 8 ? 0 : rows <= 64 ? 1 : 2;
    while (!h->plan[i].fn) --i;
    h->last_plan = i;
    const eva_kv::Plan &pl = h->plan[i];
    return cuda_status(launch_pdl(reinterpret_cast<AttendFn>(const_cast<void *>(pl.fn)), dim3(pl.grid), dim3(pl.threads),
                                  pl.smem, reinterpret_cast<cudaStream_t>(stream), 0, h->maps, p));
}

eva_status_t eva_kv_sync_status(eva_kv_t h) {
    if (!h) return EVA_ERR_INVALID_ARG;
    DeviceGuard guard(h->device);
    if (!guard.ok) return EVA_ERR_CUDA;
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_status(e);
    int word = 0;
    e = cudaMemcpy(&word, h->status, sizeof(int), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_status(e);
    if (!word) return EVA_OK;
    // the next call starts clean: a CTA that gave up may have left an item's count behind
    e = cudaMemset(h->status, 0, sizeof(int));
    if (e == cudaSuccess) e = cudaMemset(h->counters, 0, 3 * h->max_grid * sizeof(int));
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_status(e);
    return word & kAtStatusWait ? EVA_ERR_DEVICE_TIMEOUT : EVA_ERR_BAD_INDEX;
}

eva_status_t eva_kv_cache_info(eva_kv_t h, eva_kv_info *info) {
    if (!h || !info) return EVA_ERR_INVALID_ARG;
    info->workspace_bytes = h->workspace_bytes;
    info->sm_count = h->sm_count;
    info->rows = h->plan[h->last_plan].rows;
    info->grid = h->plan[h->last_plan].grid;
    info->stages = h->plan[h->last_plan].stages;
    return EVA_OK;
}

eva_status_t eva_kv_debug_inject_wait_timeout(eva_kv_t h, int32_t rounds) {
    if (!h || rounds == 0 || rounds > kWaitRounds || rounds < -kWaitRounds) return EVA_ERR_INVALID_ARG;
    h->inject_wait_rounds = rounds;
    return EVA_OK;
}

eva_status_t eva_kv_destroy(eva_kv_t h) {
    free_kv(h);
    return EVA_OK;
}

}  // extern "C"
