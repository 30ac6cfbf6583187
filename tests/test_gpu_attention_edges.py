"""Rotary positions, the 8-bit cache and attention over it where numbers, rows or pages are unusual: infinities and
NaN, dominating keys, large caps, released pages, very many parts, waits that run out, other streams."""
import numpy as np
import pytest
import torch

from tests import attn_reference as ref
from tests.conftest import cuda_available
from tests.test_gpu_attention import close, codes, cuda, i32, make_cache, rng
from vector_quantized_weight_b200 import eva_vq

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]


# ------------------------------------------------------------------ rotary positions

@pytest.mark.parametrize("T,D,R,layout,tin,tout", [
    (3, 64, 24, "interleaved", "float16", "float16"), (700, 64, 24, "interleaved", "float32", "float32"),
    (5, 256, 2, "interleaved", "float16", "float32"), (3, 128, 100, "interleaved", "float32", "float16"),
    (3, 128, 64, "interleaved", "float16", "float16"), (3, 128, 64, "half", "float16", "float16"),
    (3, 64, 24, "half", "float32", "float32"), (3, 72, 24, "interleaved", "float16", "float16"),
])
def test_rope_keeps_infinities_and_nans_where_they_are(T, D, R, layout, tin, tout):
    """Dimensions behind the rotary ones are copies whatever their neighbours hold, and a NaN or an infinity reaches
    the two dimensions of its own pair only."""
    r = rng(101)
    di, do = getattr(torch, tin), getattr(torch, tout)
    x = cuda(r.standard_normal((T, 3, D)), di)
    pos = r.integers(1, 100000, T)
    rope = eva_vq.HeadRope(3, 3, D, rotary_dim=R, layout=layout, in_dtype=tin, out_dtype=tout)
    clean, _ = rope(x, x, i32(pos))
    odd = x.clone()
    for d in range(R, D, 3):                        # behind the rotary dimensions
        odd[:, 0, d] = (float("inf"), float("-inf"), float("nan"))[d % 3]
    odd[:, 1, 0] = float("inf")                     # one rotary dimension
    odd[:, 2, R + 1 if R + 1 < D else 0] = float("nan")
    got, again = rope(odd, odd, i32(pos))
    torch.cuda.synchronize()
    assert torch.equal(got.nan_to_num(7.0, 8.0, 9.0), again.nan_to_num(7.0, 8.0, 9.0))
    assert torch.equal(got[..., R:].nan_to_num(7.0, 8.0, 9.0), odd[..., R:].to(do).nan_to_num(7.0, 8.0, 9.0))
    assert torch.equal(got[:, 0, :R], clean[:, 0, :R]) and torch.equal(got[:, 2, :R], clean[:, 2, :R])
    pair = [0, R // 2 if layout == "half" else 1]
    rest = [d for d in range(R) if d not in pair]
    assert not torch.isfinite(got[:, 1, pair]).any() and torch.equal(got[:, 1, rest], clean[:, 1, rest])
    rope.close()


# ------------------------------------------------------------------ attention

def packed(tokens, P):
    """[tokens][H][D] -> pages [pages][H][P][D], zeros behind the last token."""
    n, H, D = tokens.shape
    pages = -(-n // P)
    x = np.zeros((pages * P, H, D), tokens.dtype)
    x[:n] = tokens
    return x.reshape(pages, P, H, D).transpose(0, 2, 1, 3)


def one_sequence(cache, P, Hq, k, v, sk, sv, **kw):
    """A cache that holds one sequence: code numbers k, v [tokens][H][D], scales [pages][H]; pages in order."""
    kind = torch.int8 if cache == "int8" else torch.float8_e4m3fn
    ts = [cuda(packed(np.asarray(x, np.float32), P)).to(kind) for x in (k, v)]
    assert all(np.array_equal(codes(t), packed(np.asarray(x, np.float64), P)) for t, x in zip(ts, (k, v)))
    pages, H, _, D = ts[0].shape
    c = eva_vq.KVCache(Hq, H, D, num_pages=pages, max_seqs=1, max_pages=pages, page_size=P, dtype=cache, k=ts[0], v=ts[1],
                       k_scale=cuda(sk, torch.float32), v_scale=cuda(sv, torch.float32), **kw)
    return c, torch.arange(pages, dtype=torch.int32, device="cuda").view(1, pages)


def softmax_of(q, k, v, sk, sv, P, scale, softcap=0.0):
    """Rows q [n][Hq][D] at the last n positions of one sequence: outputs, lse and the error bound of an output before it is
    rounded, in 64 bits.

    The bound.  A weight w_j = p_j sv_j is rounded to fp16, 11 bits or a step of 2^-25 with the largest of them at 2^11
    or more: 2^-11 w_j + 2^-36 max w.  A score is off by dz: its fp32 sums and products (as in attn_reference, relative
    to the sum of their sizes) and, capped, by 2^-18 of itself; it enters a weight and the sum, so twice.  The fp32
    sums of a warp's and a part's products: 2e-6."""
    n, Hq, D = q.shape
    total, H, _ = k.shape
    G, page = Hq // H, np.arange(total) // P
    out, lse, bound = np.zeros((n, Hq, D)), np.zeros((n, Hq)), np.zeros((n, Hq, D))
    for hq in range(Hq):
        h = hq // G
        fk, fv = k[:, h] * sk[page, h][:, None], np.abs(v[:, h])
        for i in range(n):
            end = total - n + i + 1
            z = fk[:end] @ q[i, hq] * scale
            dz = 32 * 2.0 ** -24 * (np.abs(fk[:end]) @ np.abs(q[i, hq])) * scale + 4e-7 * np.abs(z).max()
            if softcap:
                z = softcap * np.tanh(z / softcap)
                dz = dz + 2.0 ** -18 * np.abs(z)
            m = z.max()
            p = np.exp(z - m)
            l, w = p.sum(), p * sv[page[:end], h]
            out[i, hq], lse[i, hq] = w @ v[:end, h] / l, m + np.log(l)
            bound[i, hq] = (2.0 ** -11 + 2 * dz.max() + 2e-6) * (w @ fv[:end]) / l + 2.0 ** -36 * w.max() * fv[:end].sum(0) / l
    return out, lse, bound


@pytest.mark.parametrize("cache,P,Hq,D,total,n,gap,scale_of_first", [
    ("int8", 64, 1, 128, 131072, 1, 14.0, 60.0), ("e4m3", 64, 8, 64, 131071, 1, 18.0, 1.0),
    ("int8", 16, 2, 64, 4097, 1, 14.0, 100.0), ("int8", 64, 8, 128, 5000, 2, 7.0, 1000.0),
    ("e4m3", 32, 4, 256, 20001, 1, 10.0, 1000.0), ("int8", 128, 8, 128, 9000, 12, 14.0, 60.0),
    ("e4m3", 64, 8, 64, 9001, 9, 16.0, 10.0), ("int8", 64, 1, 256, 4097, 5, 9.0, 500.0),
])
def test_attend_keeps_the_tail_beside_a_dominating_key(cache, P, Hq, D, total, n, gap, scale_of_first):
    """The first token takes nearly all the softmax (or its page has by far the largest value scale) and its own values are
    zero, as a first token's often are: the output is the tail's, and right relative to itself."""
    r = rng(int(total + gap))
    pages = -(-total // P)
    k, v = np.zeros((total, 1, D)), r.integers(16, 31, (total, 1, D)).astype(float)
    if cache == "e4m3":
        v = np.floor(v / 2) * 2                  # 16 .. 30 in steps of 2: e4m3 numbers
    k[1:, 0, 0] = r.integers(-2, 3, total - 1)
    k[0, 0, 1] = 96.0
    v[0] = 0.0
    sk, sv = np.full((pages, 1), 0.125), np.full((pages, 1), 0.03125)
    sv[0] *= scale_of_first
    scale = D ** -0.5
    q = 0.01 * r.standard_normal((n, Hq, D))
    q[..., 0], q[..., 1] = 1.0, gap / (96 * 0.125 * scale)
    q = cuda(q, torch.float16)
    c, table = one_sequence(cache, P, Hq, k, v, sk, sv, out_dtype="float32")
    lse = torch.empty((n, Hq), device="cuda")
    out = c.attend(q, i32([0, n]), i32([total]), table, lse=lse)
    assert c.status() == eva_vq.EVA_OK
    want, wlse, bound = softmax_of(q.double().cpu().numpy(), k, v, sk, sv, P, scale)
    assert bound.max() < 0.01 * want.min()       # the bound is relative to the output itself
    close(out, want, bound, torch.float32)
    np.testing.assert_allclose(lse.double().cpu().numpy(), wlse, atol=2e-5, rtol=2e-6)
    c.close()


@pytest.mark.parametrize("softcap", [5.0, 50.0, 1e3, 1e5, 1e9, 1e30])
@pytest.mark.parametrize("cache,P,Hq,D,total,n", [("int8", 64, 4, 128, 700, 1), ("e4m3", 16, 2, 256, 300, 3), ("int8", 32, 8, 64, 500, 5)])
def test_attend_with_small_and_large_caps(cache, P, Hq, D, total, n, softcap):
    """A cap far above the scores leaves them as they are: the error is relative to the score, not to the cap."""
    r = rng(total)
    pages = -(-total // P)
    k = ref.encode(ref.f32(r.standard_normal((total, 1, D)) * 30), cache)
    v = ref.encode(ref.f32(r.standard_normal((total, 1, D)) * 30), cache)
    sk, sv = (ref.f32((0.5 + r.random((pages, 1))) / 30) for _ in range(2))
    q = cuda(2 * r.standard_normal((n, Hq, D)), torch.float16)
    c, table = one_sequence(cache, P, Hq, k, v, sk, sv, softcap=softcap, out_dtype="float32")
    lse = torch.empty((n, Hq), device="cuda")
    out = c.attend(q, i32([0, n]), i32([total]), table, lse=lse)
    assert c.status() == eva_vq.EVA_OK
    want, wlse, bound = softmax_of(q.double().cpu().numpy(), k, v, sk, sv, P, D ** -0.5, softcap)
    close(out, want, bound, torch.float32)
    np.testing.assert_allclose(lse.double().cpu().numpy(), wlse, atol=2e-5, rtol=8e-6)
    c.close()


@pytest.mark.parametrize("cache", ["int8", "e4m3"])
@pytest.mark.parametrize("P,D,window,lens,n", [
    (16, 64, 20, [70, 100, 37, 129], [1, 1, 1, 1]), (16, 128, 33, [97, 80, 64, 33], [1, 1, 1, 1]),
    (16, 128, 17, [200, 48, 90], [3, 20, 9]), (16, 64, 1, [47, 48, 49, 33], [1, 1, 1, 1]),
    (16, 256, 20, [70, 100, 37], [1, 4, 1]), (32, 128, 20, [70, 100, 37], [1, 4, 1]), (128, 64, 40, [300, 129], [1, 2]),
])
def test_attend_leaves_released_pages_alone(cache, P, D, window, lens, n):
    """Pages wholly before the window of every row may be gone from the table, or hold another sequence's tokens by now
    (here: a page of NaN codes, or of bytes with every bit set, and scales that are NaN)."""
    Hq, H = 4, 2
    r = rng(P + D + window)
    used = [-(-x // P) for x in lens]
    num_pages, width = sum(used) + 1, max(used)
    free = num_pages - 1                         # the page that stands for what the released ones hold by now
    first = [max(0, x - m + 1 - window) // P for x, m in zip(lens, n)]
    gone, other = np.full((len(lens), width), -1), np.full((len(lens), width), -1)
    at = 0
    for b, u in enumerate(used):
        gone[b, :u] = other[b, :u] = np.arange(at, at + u)
        gone[b, :first[b]], other[b, :first[b]] = -1, free
        at += u
    raw = [r.integers(-100, 101, (num_pages, H, P, D)).astype(np.int8) for _ in range(2)]
    for x in raw:
        if cache == "e4m3":
            x[(x & 127) == 127] = 3
        x[free] = -1 if cache == "int8" else 127
    kind = torch.int8 if cache == "int8" else torch.float8_e4m3fn
    scales = [(0.5 + r.random((num_pages, H))) / (50 if cache == "int8" else 200) for _ in range(2)]
    ts, ss = [cuda(x).view(kind) for x in raw], [cuda(x, torch.float32) for x in scales]
    for s in ss:
        s[free] = float("nan")
    c = eva_vq.KVCache(Hq, H, D, num_pages=num_pages, max_seqs=len(lens), max_pages=width, page_size=P, dtype=cache, window=window,
                       k=ts[0], v=ts[1], k_scale=ss[0], v_scale=ss[1])
    starts = np.concatenate([[0], np.cumsum(n)])
    q = cuda(r.standard_normal((int(starts[-1]), Hq, D)), torch.float16)
    want, _, bound = ref.attend(q.double().cpu().numpy(), np.nan_to_num(codes(c.k)), scales_of(c.k_scale), np.nan_to_num(codes(c.v)),
                                scales_of(c.v_scale), starts, lens, np.where(gone < 0, free, gone), window=window)
    for table in (gone, other):
        out = c.attend(q, i32(starts), i32(lens), i32(table))
        assert c.status() == eva_vq.EVA_OK
        close(out, want, bound, torch.float16)
    c.close()


def scales_of(t):
    return t.nan_to_num(1.0).double().cpu().numpy()


@pytest.mark.parametrize("P,Hq,D,total,n", [
    (64, 1, 128, 70001, 1),           # 137 parts of one item: segments of 16, the last of 9
    (128, 8, 64, 131071, 1),          # 256 parts: 16 full segments
    (64, 2, 128, 66000, 1),           # 129 parts: the last segment is one part
    (32, 1, 256, 36000, 1),           # heads of 256: steps of 16 tokens, 141 parts
    (64, 5, 128, 70001, 3),           # 15 rows: items of 16
    (64, 16, 64, 50001, 9),           # many rows: several items, many parts each
])
@pytest.mark.parametrize("cache", ["int8", "e4m3"])
def test_attend_joins_very_many_parts(cache, P, Hq, D, total, n):
    r = rng(total + D)
    pages = -(-total // P)
    k = ref.encode(ref.f32(r.standard_normal((total, 1, D)) * 30), cache)
    v = ref.encode(ref.f32(r.standard_normal((total, 1, D)) * 30 + 20), cache)
    sk, sv = (ref.f32((0.5 + r.random((pages, 1))) / 30) for _ in range(2))
    q = cuda(r.standard_normal((n, Hq, D)), torch.float16)
    c, table = one_sequence(cache, P, Hq, k, v, sk, sv, out_dtype="float32")
    lse = torch.empty((n, Hq), device="cuda")
    args = (q, i32([0, n]), i32([total]), table)
    out = c.attend(*args, lse=lse)
    want, wlse, bound = softmax_of(q.double().cpu().numpy(), k, v, sk, sv, P, D ** -0.5)
    close(out, want, bound, torch.float32)
    np.testing.assert_allclose(lse.double().cpu().numpy(), wlse, atol=2e-5, rtol=2e-6)
    for _ in range(20):
        assert torch.equal(c.attend(*args), out)
    assert c.status() == eva_vq.EVA_OK
    c.close()


@pytest.mark.parametrize("cache,P,H,D,G,lens,n,softcap", [
    ("e4m3", 32, 3, 256, 16, [1, 0, 0, 1491, 1, 900, 1, 1359, 1], [0, 0, 0, 1, 6, 4, 1, 1, 0], 30.0),
    ("int8", 32, 3, 256, 8, [1491, 900, 1359], [1, 4, 1], 0.0), ("e4m3", 16, 2, 256, 2, [4000, 3100], [1, 1], 0.0),
    ("int8", 64, 3, 128, 8, [3000, 1, 2500, 2700], [1, 6, 2, 1], 0.0), ("e4m3", 64, 3, 128, 8, [3000, 1, 2500], [1, 6, 2], 30.0),
    ("int8", 32, 4, 64, 4, [5000, 4000], [1, 2], 0.0), ("e4m3", 32, 2, 64, 16, [4000, 3100], [5, 1], 0.0),
    ("int8", 64, 2, 128, 8, [2500], [30], 0.0), ("e4m3", 64, 2, 128, 4, [2500], [40], 0.0),
])
def test_attend_repeats_itself_bit_for_bit(cache, P, H, D, G, lens, n, softcap):
    """Many calls on one cache, all of it in the L2, so that copies come back fast: no stage is filled again before all of it
    has been read."""
    c, table = make_cache(cache, lens, P, H, D, 22294, Hq=H * G, softcap=softcap, out_dtype="float32")
    starts = np.concatenate([[0], np.cumsum(n)])
    rows = int(starts[-1])
    q = cuda(rng(22294).standard_normal((rows, H * G, D)), torch.float16)
    args = (i32(starts), i32(lens), i32(table))
    outs = [c.attend(q, *args) for _ in range(200)]
    assert c.status() == eva_vq.EVA_OK
    with np.errstate(invalid="ignore"):
        want, _, bound = ref.attend(q.double().cpu().numpy(), codes(c.k), c.k_scale.double().cpu().numpy(), codes(c.v),
                                    c.v_scale.double().cpu().numpy(), starts, lens, table, softcap=softcap)
    close(outs[0], want, bound, torch.float32)
    for i, out in enumerate(outs):
        assert torch.equal(out, outs[0]), i
    c.close()


def test_attend_sums_of_pages_of_zero_values():
    """2,200,000 keys whose values are all zero: zeros, and the logarithm of a sum that keeps within fp32."""
    P, D, total = 256, 64, 2200000
    pages = -(-total // P)
    c = eva_vq.KVCache(1, 1, D, num_pages=pages, max_seqs=1, max_pages=pages, page_size=P, out_dtype="float32")
    c.k.random_(-60, 61, generator=torch.Generator(device="cuda").manual_seed(3))
    c.k[0, 0, 32:] = 0
    c.k_scale.fill_(0.01)
    q = cuda(0.5 * rng(3).standard_normal((1, 1, D)), torch.float16)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, pages)
    lse = torch.empty((1, 1), device="cuda")
    out = c.attend(q, i32([0, 1]), i32([total]), table, lse=lse)
    assert c.status() == eva_vq.EVA_OK and torch.all(out == 0)
    z = (c.k.view(-1, D)[:total].float() @ q[0, 0].float()).double() * float(np.float32(0.01)) * D ** -0.5
    # of the 2^-24 of exponents near 100 that a logarithm, a score and the reference lose each, and some 100 fp32 sums
    assert abs(float(torch.logsumexp(z, 0)) - float(lse)) <= 3e-5
    c.close()


def test_attend_counts_keys_of_zero_pages_beside_others():
    """One page of values, hundreds of zeros: the zeros' keys are all of the sum's tail."""
    P, D, n = 256, 64, 200000
    pages = -(-n // P)
    c = eva_vq.KVCache(1, 1, D, num_pages=pages, max_seqs=1, max_pages=pages, page_size=P, out_dtype="float32")
    c.k[0, 0, 0, 0] = 127
    c.v[0, 0] = 1
    c.v_scale[0, 0] = 1.0
    c.k_scale.fill_(0.03125)
    q = torch.zeros((1, 1, D), dtype=torch.float16, device="cuda")
    q[..., 0] = 40.0
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, pages)
    lse = torch.empty((1, 1), device="cuda")
    out = c.attend(q, i32([0, 1]), i32([n]), table, lse=lse)
    top = 127 * 0.03125 * 40.0 * D ** -0.5
    want = (np.exp(0.0) + 255 * np.exp(-top)) / (np.exp(0.0) + (n - 1) * np.exp(-top))
    assert c.status() == eva_vq.EVA_OK
    assert abs(float(out[0, 0, 0]) - want) <= 1e-5 and abs(float(lse) - (top + np.log1p((n - 1) * np.exp(-top)))) <= 1e-5
    c.close()


@pytest.mark.parametrize("low,high", [(1e-30, 1e-30), (1e30, 1e30), (1e-30, 1e-12), (1e12, 1e30)])
def test_attend_with_value_scales_at_the_ends_of_their_range(low, high):
    P, D, total = 16, 64, 900
    r, pages = rng(151), -(-900 // 16)
    k, v = (r.integers(-100, 101, (total, 1, D)).astype(float) for _ in range(2))
    sk = np.full((pages, 1), 0.0078125)
    sv = ref.f32(np.exp(np.log(low) + r.random((pages, 1)) * np.log(high / low)))
    q = cuda(r.standard_normal((3, 2, D)), torch.float16)
    c, table = one_sequence("int8", P, 2, k, v, sk, sv, out_dtype="float32")
    lse = torch.empty((3, 2), device="cuda")
    out = c.attend(q, i32([0, 3]), i32([total]), table, lse=lse)
    assert c.status() == eva_vq.EVA_OK
    want, wlse, bound = softmax_of(q.double().cpu().numpy(), k, v, sk, sv, P, D ** -0.5)
    close(out, want, 1.02 * bound, torch.float32)      # an exponent near 110 is rounded by 2^-18, twice: each 1 % of 2^-11
    np.testing.assert_allclose(lse.double().cpu().numpy(), wlse, atol=4e-5, rtol=2e-6)
    c.close()


@pytest.mark.parametrize("D,Hq,n,total", [(128, 8, 1, 300), (64, 4, 4, 90), (256, 4, 1, 200), (128, 8, 12, 900)])
def test_attend_keeps_a_nan_in_its_row(D, Hq, n, total):
    c, table = make_cache("int8", [total], 64, 2, D, 111, Hq=Hq)
    q = cuda(rng(112).standard_normal((n, Hq, D)), torch.float16)
    args = (i32([0, n]), i32([total]), i32(table))
    lse, lse2 = (torch.empty((n, Hq), device="cuda") for _ in range(2))
    c.attend(q, *args, lse=lse)
    want, _, bound = ref.attend(q.double().cpu().numpy(), codes(c.k), c.k_scale.double().cpu().numpy(), codes(c.v),
                                c.v_scale.double().cpu().numpy(), [0, n], [total], table)
    odd = q.clone()
    odd[0, 1, 3], odd[n - 1, Hq - 1, 0] = float("nan"), float("inf")
    out = c.attend(odd, *args, lse=lse2)
    assert c.status() == eva_vq.EVA_OK
    hit = torch.zeros((n, Hq), dtype=torch.bool, device="cuda")
    hit[0, 1] = hit[n - 1, Hq - 1] = True
    rest = ~hit.cpu().numpy()
    close(out[~hit], want[rest], bound[rest], torch.float16)
    assert float((lse2[~hit] - lse[~hit]).abs().max()) <= 1e-5
    assert torch.isnan(out[hit]).all() and torch.isnan(lse2[hit]).all()
    c.close()


# ------------------------------------------------------------------ the cache

def test_read_leaves_rows_of_no_sequence_and_drops_ranges_that_cannot_be_right():
    H, D, P = 2, 64, 16
    c, table = make_cache("int8", [40, 33], P, H, D, 121)
    values = codes(c.k)[:, :, :, :] * c.k_scale.double().cpu().numpy()[..., None, None]

    def token(b, pos):
        return ref.f32(values[table[b][pos // P], :, pos % P])

    def read(starts, begins, rows):
        k, v = (torch.full((rows, H, D), 7.0, device="cuda") for _ in range(2))
        c.read(i32(starts), i32(begins), i32(table), rows, k_out=k, v_out=v, dtype="float32")
        return k.cpu().numpy(), c.status()

    # rows before the first sequence and behind the last are nobody's
    k, st = read([2, 5, 7], [10, 20], 9)
    assert st == eva_vq.EVA_OK
    for row, (b, pos) in {2: (0, 10), 3: (0, 11), 4: (0, 12), 5: (1, 20), 6: (1, 21)}.items():
        np.testing.assert_array_equal(k[row], token(b, pos))
    assert np.all(k[[0, 1, 7, 8]] == 7.0)
    # a range that goes backwards, past the rows, or begins before them drops its sequence, no other
    for starts, begins, kept in (([0, 2, 0], [10, 20], {0: (0, 10), 1: (0, 11)}), ([0, 2, 99], [10, 20], {0: (0, 10), 1: (0, 11)}),
                                 ([-1, 2, 4], [10, 20], {2: (1, 20), 3: (1, 21)}), ([0, 2, 4], [-3, 20], {2: (1, 20), 3: (1, 21)})):
        k, st = read(starts, begins, 4)
        assert st == eva_vq.EVA_ERR_BAD_INDEX
        for row in range(4):
            np.testing.assert_array_equal(k[row], token(*kept[row]) if row in kept else np.full((H, D), 7.0))
    c.close()


def test_attend_gives_up_with_copies_in_flight():
    """The working warps give up at once while the streaming warp fills the ring: the call ends with the status, and what
    follows eva_kv_sync_status is right."""
    for cache, P, Hq, H, D, lens, n in (("int8", 64, 16, 2, 128, [3000, 20], [1, 1]), ("e4m3", 16, 8, 4, 64, [2000], [5]),
                                        ("int8", 32, 4, 2, 256, [1500, 900], [1, 1]), ("int8", 64, 8, 1, 128, [4000], [40])):
        c, table = make_cache(cache, lens, P, H, D, 131, Hq=Hq)
        starts = np.concatenate([[0], np.cumsum(n)])
        q = cuda(rng(132).standard_normal((int(starts[-1]), Hq, D)), torch.float16)
        args = (q, i32(starts), i32(lens), i32(table))
        good = c.attend(*args)
        assert c.status() == eva_vq.EVA_OK
        for _ in range(3):
            eva_vq.eva_kv_debug_inject_wait_timeout(c.handle, -64)
            c.attend(*args)
            assert c.status() == eva_vq.EVA_ERR_DEVICE_TIMEOUT
            assert torch.equal(c.attend(*args), good) and c.status() == eva_vq.EVA_OK
        c.close()


def test_buffers_made_for_a_stream_are_ready_on_it():
    """A cache made with stream=s fills its buffers on s: what s writes next is not overwritten by zeros that another,
    busy stream still owes."""
    H, D, P = 2, 64, 16
    s = torch.cuda.Stream()
    x = cuda(rng(141).standard_normal((5, H, D)), torch.float16)
    starts, lens, table = i32([0, 5]), i32([5]), i32([[0]])
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)               # about 0.1 s on the current stream
    c = eva_vq.KVCache(H, H, D, num_pages=2, max_seqs=1, max_pages=1, page_size=P, stream=s)
    c.append(x, x, starts, lens, table, stream=s)
    torch.cuda.synchronize()
    assert c.status() == eva_vq.EVA_OK
    k, _ = c.read(starts, i32([0]), table, 5, dtype="float32")
    assert float((k - x.float()).abs().max()) <= 0.51 * float(c.k_scale[0].max())
    assert torch.all(c.k[1] == 0) and torch.all(c.k_scale[1] == 0)
    c.close()


def test_device_without_a_number_is_the_current_one():
    dev = torch.device("cuda", torch.cuda.current_device())
    c = eva_vq.KVCache(1, 1, 64, num_pages=1, max_seqs=1, max_pages=1, device="cuda")
    rope = eva_vq.HeadRope(1, 1, 64, device="cuda")
    assert c.device == dev and rope.device == dev and c.k.device == dev
    c.close()
    rope.close()


def test_attend_refuses_more_steps_than_a_cta_counts():
    """More than 300,000 rows at the end of a sequence of 2^30 tokens: nothing is read or written, and the status says so."""
    P, D, n = 256, 64, 40000
    c = eva_vq.KVCache(8, 1, D, num_pages=1, max_seqs=1, max_pages=1 << 22, page_size=P)
    q = torch.zeros((n, 8, D), dtype=torch.float16, device="cuda")
    out = torch.full_like(q, 7.0)
    table = torch.full((1, 1 << 22), -1, dtype=torch.int32, device="cuda")
    c.attend(q, i32([0, n]), i32([1 << 30]), table, out=out)
    assert c.status() == eva_vq.EVA_ERR_BAD_INDEX
    assert torch.all(out == 7.0)
    c.close()


def test_calls_of_more_than_a_billion_rows_are_refused():
    rope = eva_vq.HeadRope(1, 1, 2)
    lib, x = eva_vq.load(), torch.zeros((4, 2), dtype=torch.float16, device="cuda")
    P = x.data_ptr()
    for T in ((1 << 30) + 1, (1 << 31) - 1, -1):
        assert lib.eva_rope_run(rope.handle, P, 2, P, 2, P, T, P, 2, P, 2, None) == eva_vq.EVA_ERR_INVALID_ARG
    rope.close()
