"""Rotary positions, the 8-bit cache and attention over it on the GPU, against 64-bit references; and the attention
half of a decoder block as it is used: q, k, v layers -> positions -> cache -> attention -> o layer."""
import numpy as np
import pytest
import torch

import oracle
from tests import attn_reference as ref
from tests.conftest import cuda_available
from tests.gpu_helpers import TOL, norm_rel_err
from vector_quantized_weight_b200 import eva_vq, synth

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]


def rng(seed):
    return np.random.default_rng(seed)


def cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def close(got, want, bound, dtype):
    got = got.double().cpu().numpy()
    tol = ref.rounded(want, bound, dtype)
    off = np.abs(got - want)
    assert np.all(off <= tol), (float((off / tol).max()), float(off.max()))


# ------------------------------------------------------------------ rotary positions

ROPE = [
    # T, Hq, Hk, D, R, layout, scaling, norm, in, out
    (1, 32, 32, 128, 128, "half", None, False, "float16", "float16"),
    (1, 8, 1, 64, 64, "interleaved", None, True, "float16", "float16"),
    (67, 5, 3, 256, 64, "half", {"type": "linear", "factor": 4.0}, True, "float16", "float16"),
    (33, 4, 2, 128, 48, "interleaved", {"type": "ntk", "factor": 8.0}, False, "float32", "float16"),
    (130, 3, 1, 80, 80, "half", {"type": "yarn", "factor": 16.0, "original": 4096}, True, "float32", "float32"),
    (700, 7, 2, 96, 32, "half", {"type": "bands", "factor": 8.0, "original": 8192}, True, "float16", "float32"),
    (9, 2, 2, 72, 24, "half", None, True, "float16", "float16"),            # not multiples of 16: one element an access
    (4, 2, 1, 35, 34, "interleaved", None, True, "float32", "float32"),
    (5, 1, 1, 512, 512, "half", None, False, "float16", "float16"),
    (3, 1, 1, 1000, 998, "half", None, True, "float16", "float16"),
    (700, 3, 2, 64, 24, "interleaved", None, True, "float16", "float16"),    # the last 16 turned dimensions half
    (40, 2, 1, 256, 2, "interleaved", {"type": "yarn", "factor": 4.0, "original": 100}, False, "float32", "float16"),
    (6, 4, 4, 128, 0, "half", None, True, "float16", "float16"),             # the norm alone
    (6, 0, 4, 128, 128, "half", None, False, "float16", "float16"),          # keys alone
    (2500, 2, 1, 64, 64, "half", None, False, "float16", "float16"),         # four tokens a CTA
]


@pytest.mark.parametrize("T,Hq,Hk,D,R,layout,scaling,norm,tin,tout", ROPE)
def test_rope_matches_the_formula(T, Hq, Hk, D, R, layout, scaling, norm, tin, tout):
    r = rng(T * 1000 + D)
    di, do = getattr(torch, tin), getattr(torch, tout)
    q, k = cuda(r.standard_normal((T, Hq, D)), di), cuda(r.standard_normal((T, Hk, D)), di)
    w = cuda(1 + 0.2 * r.standard_normal(D), torch.float16) if norm else None
    pos = r.integers(0, 100000, T)
    pos[: min(T, 4)] = [2 ** 31 - 1, 0, -7, 1048577][: min(T, 4)]
    rope = eva_vq.HeadRope(Hq, Hk, D, rotary_dim=R, layout=layout, scaling=scaling, norm=norm, q_weight=w, eps=1e-5,
                           weight_offset=0.5, in_dtype=tin, out_dtype=tout)
    got = rope(q, k, i32(pos) if R else None)
    torch.cuda.synchronize()
    freq, mag = ref.frequencies(R, 10000.0, scaling)
    for x, y, weight in ((q, got[0], w), (k, got[1], None)):
        if x.numel():
            want, bound = ref.rope(x.double().cpu().numpy(), pos, R, layout, freq, mag, norm,
                                   None if weight is None else weight.double().cpu().numpy(), 1e-5, 0.5)
            close(y, want, bound, do)
    rope.close()


@pytest.mark.parametrize("D,R,offset", [(128, 128, 0), (128, 64, 3), (64, 40, 0)])
def test_rope_strided_and_in_place(D, R, offset):
    """q and k as column ranges of a fused projection (offset: a misaligned one), written in place, v untouched."""
    r = rng(5)
    T, Hq, Hk = 21, 6, 2
    buf = torch.zeros((T, offset + (Hq + 2 * Hk) * D + 5), dtype=torch.float16, device="cuda")
    buf[:] = cuda(r.standard_normal(tuple(buf.shape)), torch.float16)
    q = buf[:, offset:offset + Hq * D].unflatten(1, (Hq, D))
    k = buf[:, offset + Hq * D:offset + (Hq + Hk) * D].unflatten(1, (Hk, D))
    before, pos = buf.clone(), r.integers(0, 5000, T)
    rope = eva_vq.HeadRope(Hq, Hk, D, rotary_dim=R)
    fresh = rope(q, k, i32(pos))
    rope(q, k, i32(pos), q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert torch.equal(q, fresh[0]) and torch.equal(k, fresh[1])
    end = offset + (Hq + Hk) * D
    assert torch.equal(buf[:, end:], before[:, end:]) and torch.equal(buf[:, :offset], before[:, :offset])
    freq, mag = ref.frequencies(R)
    want, bound = ref.rope(before[:, offset:offset + Hq * D].double().cpu().numpy().reshape(T, Hq, D), pos, R, "half", freq, mag)
    close(q, want, bound, torch.float16)
    assert rope(q[:0], k[:0], i32(pos[:0]))[0].shape == (0, Hq, D)
    rope.close()


# ------------------------------------------------------------------ the cache

# A value is off by half a step of its scale, and by two fp32 roundings of at most 127 steps (the quotient x / scale and
# the product code * scale): 2 * 127 * 2^-24 < 2^-16 of a step, 2^-15 of the half step.
HALF = 0.5 * (1 + 2.0 ** -15)


def tables(lens, P, max_pages, num_pages, seed):
    order = rng(seed).permutation(num_pages)
    table, at = np.full((len(lens), max_pages), -1), 0
    for b, n in enumerate(lens):
        used = -(-int(n) // P)
        table[b, :used] = order[at:at + used]
        at += used
    return table


def make_cache(cache, lens, P, H, D, seed, *, spare=2, max_pages=None, extreme=False, Hq=None, **kw):
    """A cache with random codes everywhere (behind a sequence's end too, where e4m3 bytes may be NaN)."""
    r = rng(seed)
    max_pages = max_pages or max(1, -(-int(max(lens)) // P))
    num_pages = int(sum(-(-int(n) // P) for n in lens)) + spare
    raw = [r.integers(0, 256, (num_pages, H, P, D), dtype=np.uint8) for _ in range(2)]
    scales = [(0.2 + r.random((num_pages, H))) / ref.LARGEST[cache] * 2 for _ in range(2)]
    if extreme:      # page scales twenty orders of magnitude apart, and pages of zeros
        scales[1] = scales[1] * 10.0 ** r.integers(-18, 2, (num_pages, H))
        scales[0][1::3] = 0.0
        scales[1][2::5] = 0.0
    table = tables(lens, P, max_pages, num_pages, seed + 1)
    kind = torch.int8 if cache == "int8" else torch.float8_e4m3fn
    for x in raw:
        if cache == "int8":
            x[x == 128] = 129
        else:
            for b, n in enumerate(lens):      # no NaN among the tokens that are there
                for j in range(-(-int(n) // P)):
                    part = x[table[b][j], :, :max(0, min(P, int(n) - j * P))]
                    part[(part & 127) == 127] = 5
    ts = [torch.from_numpy(x).cuda().view(kind) for x in raw]
    ss = [cuda(s, torch.float32) for s in scales]
    c = eva_vq.KVCache(Hq or H, H, D, num_pages=num_pages, max_seqs=len(lens), max_pages=max_pages, page_size=P, dtype=cache,
                       k=ts[0], v=ts[1], k_scale=ss[0], v_scale=ss[1], **kw)
    return c, table


def codes(t):
    return t.float().double().cpu().numpy()


WRITE = [
    # cache, P, H, D, old lengths, new tokens of each, dtype
    ("int8", 64, 8, 128, [63, 64, 65, 0], [1, 1, 1, 1], "float16"),
    ("e4m3", 16, 2, 64, [5, 31, 0], [40, 1, 17], "float16"),
    ("int8", 32, 3, 256, [100, 7], [0, 70], "float32"),
    ("e4m3", 128, 1, 128, [1, 250], [300, 3], "float32"),
    ("int8", 256, 2, 64, [255, 10], [2, 600], "float16"),
    ("e4m3", 64, 2, 256, [33] * 40, [1] * 40, "float16"),
]


@pytest.mark.parametrize("cache,P,H,D,old,new,dtype", WRITE)
def test_append_matches_the_definition_exactly(cache, P, H, D, old, new, dtype):
    lens = [a + n for a, n in zip(old, new)]
    c, table = make_cache(cache, lens, P, H, D, 11)
    r = rng(12)
    starts = np.concatenate([[0], np.cumsum(new)])
    T = int(starts[-1]) + 3                       # three rows behind the last sequence
    dt = getattr(torch, dtype)
    rows = cuda(r.standard_normal((T, 2 * H * D)) * np.exp(2 * r.standard_normal((T, 1))), dt)
    k, v = rows[:, :H * D].unflatten(1, (H, D)), rows[:, H * D:].unflatten(1, (H, D))
    k[0, 0, 0], v[0, 0, 1] = float("nan"), float("inf")
    if len(rows) > 5:
        k[1, 0], v[1, 0] = 0.0, 0.0
    want = [codes(c.k), c.k_scale.double().cpu().numpy(), codes(c.v), c.v_scale.double().cpu().numpy()]
    with np.errstate(invalid="ignore"):
        ref.append(want[0], want[1], k.double().cpu().numpy(), starts, lens, table, cache)
        ref.append(want[2], want[3], v.double().cpu().numpy(), starts, lens, table, cache)
    c.append(k, v, i32(starts), i32(lens), i32(table))
    assert c.status() == eva_vq.EVA_OK
    for got, w in zip((c.k, c.k_scale, c.v, c.v_scale), want):
        got = codes(got) if got.dim() == 4 else got.double().cpu().numpy()
        assert np.array_equal(got, w, equal_nan=True)
    # the same tokens again change nothing; then read every sequence back whole
    again = [t.clone().view(torch.uint8) for t in (c.k, c.v)]
    c.append(k, v, i32(starts), i32(lens), i32(table))
    assert torch.equal(again[0], c.k.view(torch.uint8)) and torch.equal(again[1], c.v.view(torch.uint8))
    back = np.concatenate([[0], np.cumsum(lens)])
    for dt in ("float16", "float32"):
        out = c.read(i32(back), i32([0] * len(lens)), i32(table), int(back[-1]), dtype=dt)
        for got, w, s in ((out[0], want[0], want[1]), (out[1], want[2], want[3])):
            vals = np.concatenate([w[table[b][np.arange(n) // P], :, np.arange(n) % P] *
                                   s[table[b][np.arange(n) // P]][..., None] for b, n in enumerate(lens)])
            np.testing.assert_array_equal(got.cpu().numpy(), ref.f32(vals).astype(dt))
    assert c.status() == eva_vq.EVA_OK
    c.close()


def test_append_token_by_token_keeps_within_the_steps():
    """A page filled one token at a time: every stored value within the roundings it has been through, each half a
    step of a scale that only grows."""
    P, H, D = 32, 2, 64
    c = eva_vq.KVCache(H, H, D, num_pages=2, max_seqs=1, max_pages=2, page_size=P)
    x = rng(3).standard_normal((P, H, D)) * np.linspace(0.2, 4, P)[:, None, None]
    t = cuda(x, torch.float16)
    table = i32([[1, 0]])
    for i in range(P):
        c.append(t[i:i + 1], t[i:i + 1], i32([0, 1]), i32([i + 1]), table)
    k, _ = c.read(i32([0, P]), i32([0]), table, P, dtype="float32")
    grown = c.k_scale[1].double().cpu().numpy()
    off = np.abs(k.double().cpu().numpy() - t.double().cpu().numpy())
    assert np.all(off <= P * HALF * grown[None, :, None])
    assert np.all(off[-1] <= HALF * grown[:, None])
    assert torch.equal(c.k_scale[0], torch.zeros_like(c.k_scale[0]))      # the other page is as it was
    c.close()


def test_append_drops_rows_before_position_zero_and_padded_sequences():
    P, H, D = 16, 1, 64
    c, table = make_cache("int8", [3, 0, 20], P, H, D, 4)
    before = c.k.clone()
    x = cuda(rng(5).standard_normal((7, H, D)), torch.float16)
    starts, lens = [0, 5, 6, 6], [3, 0, 20]       # five rows for three positions; a padded row; no row
    want = [codes(c.k), c.k_scale.double().cpu().numpy()]
    ref.append(want[0], want[1], x.double().cpu().numpy(), starts, lens, table, "int8")
    c.append(x, x, i32(starts), i32(lens), i32(table))
    assert c.status() == eva_vq.EVA_OK
    assert np.array_equal(codes(c.k), want[0]) and not torch.equal(c.k, before)
    c.close()


# ------------------------------------------------------------------ attention

ATTEND = [
    # cache, P, Hq, H, D, lens, rows of each, window, softcap, out
    ("int8", 64, 32, 32, 128, [517], [1], 0, 0.0, "float16"),
    ("int8", 64, 16, 2, 128, [1, 2, 31, 32, 33, 64, 65, 1000], [1] * 8, 0, 0.0, "float16"),
    ("e4m3", 16, 6, 3, 256, [700, 15, 16, 17], [1, 1, 1, 1], 100, 50.0, "float16"),
    ("e4m3", 32, 32, 4, 64, [301, 5, 77], [5, 5, 5], 0, 0.0, "float16"),
    ("int8", 128, 8, 1, 64, [0, 1, 400], [1, 1, 1], 0, 0.0, "float32"),
    ("int8", 256, 14, 2, 128, [900, 40], [2, 1], 0, 30.0, "float32"),           # 7 queries a key head: 16 rows an item
    ("int8", 16, 16, 2, 128, [130], [64], 0, 0.0, "float16"),                   # a chunk of a prompt: rows share steps
    ("e4m3", 64, 9, 3, 64, [50, 0, 37, 200], [50, 0, 37, 9], 0, 0.0, "float16"),
    ("int8", 32, 4, 2, 256, [90, 33], [70, 20], 33, 0.0, "float16"),
    ("e4m3", 64, 5, 1, 128, [260, 3], [4, 3], 0, 20.0, "float16"),              # 20 rows: 32 an item
    ("int8", 32, 24, 1, 64, [333], [1], 0, 0.0, "float16"),
    ("e4m3", 16, 12, 1, 256, [100, 280], [3, 1], 0, 0.0, "float32"),
    ("int8", 64, 8, 8, 128, [12, 9], [15, 12], 0, 0.0, "float16"),              # more rows than positions: zeros
    ("int8", 64, 1, 1, 128, [6000], [1], 0, 0.0, "float16"),                    # one item over many CTAs
    ("e4m3", 32, 8, 1, 128, [4001, 60], [1, 1], 1, 0.0, "float16"),             # a window of the row itself
    # many steps and many items a CTA: the ring and the pieces come round many times
    ("int8", 64, 8, 8, 128, [1400 - 21 * i for i in range(66)], [1] * 66, 0, 0.0, "float16"),
    ("e4m3", 16, 32, 8, 64, [1 + 37 * i for i in range(50)], [1] * 50, 0, 0.0, "float16"),
    ("int8", 32, 8, 4, 256, [2 + 90 * (i % 17) for i in range(35)], [1] * 35, 0, 0.0, "float16"),
    ("int8", 64, 16, 4, 128, [3000, 2999, 1], [8, 5, 1], 0, 0.0, "float16"),
    ("e4m3", 128, 32, 4, 64, [2500, 90, 2600], [40, 3, 33], 0, 0.0, "float16"),
    ("int8", 16, 16, 8, 128, [60 + i for i in range(40)], [4] * 40, 0, 0.0, "float16"),
]


@pytest.mark.parametrize("extreme", [False, True])
@pytest.mark.parametrize("cache,P,Hq,H,D,lens,n,window,softcap,tout", ATTEND)
def test_attend_matches_the_formula(cache, P, Hq, H, D, lens, n, window, softcap, tout, extreme):
    c, table = make_cache(cache, lens, P, H, D, 21, extreme=extreme, Hq=Hq, window=window, softcap=softcap, out_dtype=tout)
    r = rng(22)
    starts = np.concatenate([[0], np.cumsum(n)])
    T = int(starts[-1]) + 2
    q = cuda(r.standard_normal((T, Hq * D + 8)), torch.float16)[:, :Hq * D].unflatten(1, (Hq, D))
    dt = getattr(torch, tout)
    out = torch.full((T, Hq, D), 7.0, dtype=dt, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    c.attend(q, i32(starts), i32(lens), i32(table), out=out, lse=lse)
    assert c.status() == eva_vq.EVA_OK
    with np.errstate(invalid="ignore"):
        want, wlse, bound = ref.attend(q.double().cpu().numpy(), codes(c.k), c.k_scale.double().cpu().numpy(), codes(c.v),
                                       c.v_scale.double().cpu().numpy(), starts, lens, table, window=window, softcap=softcap)
    rows = int(starts[-1])
    assert torch.all(out[rows:] == 7.0) and torch.all(lse[rows:] == 7.0)
    close(out[:rows], want[:rows], bound[:rows], dt)
    got = lse[:rows].double().cpu().numpy()
    seen = np.isfinite(wlse[:rows])
    assert np.array_equal(got[~seen], wlse[:rows][~seen])
    np.testing.assert_allclose(got[seen], wlse[:rows][seen], atol=2e-5 + 1e-6 * softcap, rtol=2e-6)
    # again: the same bits, and the join's counters are back at zero
    out2 = c.attend(q, i32(starts), i32(lens), i32(table))
    assert torch.equal(out2[:rows], out[:rows])
    c.close()


def test_attend_on_pages_outside_the_cache_masks_them_and_says_so():
    lens, P = [100, 200], 32
    c, table = make_cache("e4m3", lens, P, 2, 128, 31, Hq=4)
    bad = table.copy()
    bad[0, 1], bad[1, 0], bad[1, 6] = c.k.shape[0], -5, 2 ** 30
    q = cuda(rng(32).standard_normal((2, 4, 128)), torch.float16)
    out = c.attend(q, i32([0, 1, 2]), i32(lens), i32(bad))
    assert c.status() == eva_vq.EVA_ERR_BAD_INDEX and c.status() == eva_vq.EVA_OK
    with np.errstate(invalid="ignore"):
        want, _, bound = ref.attend(q.double().cpu().numpy(), codes(c.k), c.k_scale.double().cpu().numpy(), codes(c.v),
                                    c.v_scale.double().cpu().numpy(), [0, 1, 2], lens, bad)
    close(out, want, bound, torch.float16)
    k, before = q[:, :2].contiguous(), c.k.view(torch.uint8).clone()
    c.append(k, k, i32([0, 1, 2]), i32(lens), i32(np.full_like(table, 10 ** 6)))
    assert c.status() == eva_vq.EVA_ERR_BAD_INDEX and torch.equal(before, c.k.view(torch.uint8))
    c.read(i32([0, 2, 4]), i32([0, 0]), i32(np.full_like(table, -1)), 4)
    assert c.status() == eva_vq.EVA_ERR_BAD_INDEX
    # lengths and row ranges that cannot be right drop their sequence
    for starts, ls in (([0, 1, 2], [100, 10 ** 9]), ([0, 1, 0], [100, 200]), ([0, 1, 99], [100, 200]), ([0, 1, 2], [100, -1])):
        o = torch.zeros_like(out)
        c.attend(q, i32(starts), i32(ls), i32(table), out=o)
        assert c.status() == eva_vq.EVA_ERR_BAD_INDEX
        assert torch.all(o[1] == 0) and torch.any(o[0] != 0)
    c.close()


def test_attend_gives_up_bounded_waits():
    lens = [300]
    c, table = make_cache("int8", lens, 32, 2, 64, 41)
    q = cuda(rng(42).standard_normal((1, 2, 64)), torch.float16)
    args = (q, i32([0, 1]), i32(lens), i32(table))
    good = c.attend(*args)
    assert c.status() == eva_vq.EVA_OK
    eva_vq.eva_kv_debug_inject_wait_timeout(c.handle, 64)
    c.attend(*args)
    assert c.status() == eva_vq.EVA_ERR_DEVICE_TIMEOUT
    assert torch.equal(c.attend(*args), good) and c.status() == eva_vq.EVA_OK
    c.close()


def test_cache_beyond_four_gigabytes():
    """Pages whose byte offsets pass 2^32."""
    P, H, D, pages = 64, 8, 256, 36000            # 131072 bytes a page: 4.7e9
    k, v = (torch.empty((pages, H, P, D), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pages, H), 0.01, device="cuda") for _ in range(2))
    table = [pages - 1, 5, pages - 3]
    c = eva_vq.KVCache(H, H, D, num_pages=pages, max_seqs=1, max_pages=3, page_size=P, k=k, v=v, k_scale=ks, v_scale=vs)
    r, n = rng(51), 150
    x, y = cuda(r.standard_normal((n, H, D)), torch.float16), cuda(r.standard_normal((n, H, D)), torch.float16)
    c.append(x, y, i32([0, n]), i32([n]), i32([table]))
    q = cuda(r.standard_normal((1, H, D)), torch.float16)
    out = c.attend(q, i32([0, 1]), i32([n]), i32([table]))
    assert c.status() == eva_vq.EVA_OK
    small = [codes(t[table]) for t in (k, v)]
    sc = [t[table].double().cpu().numpy() for t in (ks, vs)]
    want, _, bound = ref.attend(q.double().cpu().numpy(), small[0], sc[0], small[1], sc[1], [0, 1], [n], [[0, 1, 2]])
    close(out, want, bound, torch.float16)
    step = sc[0][np.arange(n) // P]
    back, _ = c.read(i32([0, n]), i32([0]), i32([table]), n, dtype="float32")
    assert np.all(np.abs(back.double().cpu().numpy() - x.double().cpu().numpy()) <= HALF * step[..., None])
    c.close()
    del k, v
    torch.cuda.empty_cache()


def test_captured_step_follows_the_device_arrays_and_other_streams():
    """append + attend captured once on a side stream and replayed for later tokens; a clone on another stream."""
    P, H, D, B = 16, 2, 128, 3
    lens0 = [40, 15, 16]
    c, table = make_cache("int8", [n + 5 for n in lens0], P, H, D, 61, Hq=4)
    r = rng(62)
    k, v = (torch.zeros((B, H, D), dtype=torch.float16, device="cuda") for _ in range(2))
    q = torch.zeros((B, 4, D), dtype=torch.float16, device="cuda")
    starts, lens, tab = i32(range(B + 1)), i32(lens0), i32(table)
    out = torch.zeros((B, 4, D), dtype=torch.float16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.append(k, v, starts, lens, tab)
        c.attend(q, starts, lens, tab, out=out)
    other = c.clone()
    for step in range(5):
        for t in (k, v, q):
            t.copy_(cuda(r.standard_normal(tuple(t.shape)), torch.float16))
        lens += 1
        graph.replay()
        with np.errstate(invalid="ignore"):
            want, _, bound = ref.attend(q.double().cpu().numpy(), codes(c.k), c.k_scale.double().cpu().numpy(), codes(c.v),
                                        c.v_scale.double().cpu().numpy(), range(B + 1), lens.tolist(), table)
        close(out, want, bound, torch.float16)
        s.wait_stream(torch.cuda.current_stream())
        again = other.attend(q, starts, lens, tab, stream=s)
        s.synchronize()
        assert torch.equal(again, out)
    assert c.status() == eva_vq.EVA_OK and other.status() == eva_vq.EVA_OK
    other.close()
    c.close()


def test_refusals():
    """What the entry points refuse with a handle in hand, before any launch."""
    D, H = 64, 2
    c, table = make_cache("int8", [40], 32, H, D, 81, Hq=4)
    q = torch.zeros((1, 4, D), dtype=torch.float16, device="cuda")
    k = torch.zeros((1, H, D), dtype=torch.float16, device="cuda")
    s, n, t = i32([0, 1]), i32([40]), i32(table)
    bad = [lambda: c.attend(q.float(), s, n, t), lambda: c.attend(q[:, :2], s, n, t), lambda: c.attend(q.cpu(), s, n, t),
           lambda: c.attend(q, s.long(), n, t), lambda: c.attend(q, s, n, t[:, :1]), lambda: c.attend(q, s[:1], n, t),
           lambda: c.attend(q, i32([0, 1, 1]), i32([40, 1]), i32(np.tile(table, (2, 1)))),      # more sequences than planned
           lambda: c.attend(q, s, n, t, out=torch.zeros((1, 4, D), device="cuda")),
           lambda: c.attend(q, s, n, t, lse=torch.zeros((1, 3), device="cuda")),
           lambda: c.append(k, k.float(), s, n, t), lambda: c.append(k.bfloat16(), k.bfloat16(), s, n, t),
           lambda: c.append(k, k[:0], s, n, t), lambda: c.append(k.transpose(1, 2), k, s, n, t),
           lambda: c.read(s, n, t, 1, k_out=k.float()),
           lambda: eva_vq.KVCache(4, H, D, num_pages=1, max_seqs=1, max_pages=1, k=c.k),
           lambda: eva_vq.HeadRope(1, 1, D, norm=True, q_weight=torch.ones(D, device="cuda"))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    rope = eva_vq.HeadRope(4, H, D)
    for call in (lambda: rope(q, k[:0], i32([0])), lambda: rope(q, k, i32([0, 1])), lambda: rope(q, k, None)):
        with pytest.raises(ValueError):
            call()
    wide = torch.zeros((3, 4 * D + 4), dtype=torch.float16, device="cuda")
    rows = wide[:, :4 * D].unflatten(1, (4, D))                        # rows 8 bytes off a 16-byte border
    for call in (lambda: c.attend(rows, i32([0, 3]), n, t), lambda: c.append(rows[:, :H], rows[:, :H], i32([0, 3]), n, t)):
        with pytest.raises(eva_vq.EvaError):
            call()
    lib = eva_vq.load()
    P = q.data_ptr()
    assert lib.eva_kv_attend(c.handle, P, 4 * D - 8, P, P, P, 1, 1, P, None, None) == eva_vq.EVA_ERR_INVALID_ARG
    assert lib.eva_kv_attend(c.handle, P, 4 * D, P, P, P, 1, 1 << 30, P, None, None) == eva_vq.EVA_ERR_UNSUPPORTED
    assert lib.eva_kv_attend(c.handle, P, 4 * D, P, P, P, 0, 1, P, None, None) == eva_vq.EVA_ERR_INVALID_ARG
    assert lib.eva_kv_append(c.handle, P, H * D, P, H * D, 5, P, P, P, 1, 1, None) == eva_vq.EVA_ERR_INVALID_ARG
    assert lib.eva_kv_read(c.handle, P, P, P, 1, 1, 0, None, None, None) == eva_vq.EVA_ERR_INVALID_ARG
    assert lib.eva_rope_run(rope.handle, P, 4 * D - 1, P, H * D, P, 1, P, 4 * D, P, H * D, None) == eva_vq.EVA_ERR_INVALID_ARG
    assert lib.eva_rope_run(rope.handle, P, 4 * D, P, H * D, None, 1, P, 4 * D, P, H * D, None) == eva_vq.EVA_ERR_INVALID_ARG
    assert c.status() == eva_vq.EVA_OK
    # nothing to do is not an error
    assert c.attend(q[:0], i32([0, 0]), n, t).shape == (0, 4, D)
    c.append(k[:0], k[:0], i32([0, 0]), n, t)
    assert c.read(i32([0, 0]), i32([0]), t, 0)[0].shape == (0, H, D)
    rope.close()
    c.close()
    with pytest.raises(eva_vq.EvaError):
        c.attend(q, s, n, t)


def test_two_handles_at_once_and_a_shared_prefix():
    """Two sequences whose tables name the same pages, read by two handles on two streams at the same time, many
    times over."""
    H, D, P = 4, 128, 32
    lens = [700, 700]
    c, table = make_cache("int8", lens, P, H, D, 91, Hq=16)
    table[1, :20] = table[0, :20]
    q = cuda(rng(92).standard_normal((2, 16, D)), torch.float16)
    args = (q, i32([0, 1, 2]), i32(lens), i32(table))
    want, _, bound = ref.attend(q.double().cpu().numpy(), codes(c.k), c.k_scale.double().cpu().numpy(), codes(c.v),
                                c.v_scale.double().cpu().numpy(), [0, 1, 2], lens, table)
    other, streams = c.clone(), [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [[h.attend(*args, stream=s) for h, s in zip((c, other), streams)] for _ in range(40)]
    torch.cuda.synchronize()
    for pair in outs:
        for o in pair:
            assert torch.equal(o, outs[0][0])
    close(outs[0][0], want, bound, torch.float16)
    assert c.status() == eva_vq.EVA_OK and other.status() == eva_vq.EVA_OK
    other.close()
    c.close()


@pytest.mark.parametrize("B", [1, 5])
def test_attention_half_of_a_block(B):
    """q, k and v layers in one launch, positions and cache, attention, the o layer: three steps on a prompt's cache,
    each stage against its reference fed the GPU's own inputs of that stage."""
    cfg = synth.CONFIGS["llama7b_block"]
    H, D, P = 32, 128, 32
    datas = [synth.make_layer(sh, synth.layer_seed(cfg.index, li)) for li, sh in enumerate(cfg.layers[:4])]
    lins = [eva_vq.from_layer(d, max_batch=B) for d in datas]
    lens0 = [70 + 13 * b for b in range(B)]
    steps = 3
    c, table = make_cache("int8", [n + steps for n in lens0], P, H, D, 71)
    rope = eva_vq.HeadRope(H, H, D)
    starts, tab, lens, positions = i32(range(B + 1)), i32(table), i32(lens0), i32(lens0)
    x = cuda(synth.make_x(4096, B, 72))
    freq, mag = ref.frequencies(D)
    for step in range(steps):
        lens += 1
        ys = eva_vq.run_group(lins[:3], [x] * 3)
        q, k = rope(ys[0], ys[1], positions)
        kept = [codes(c.k), c.k_scale.double().cpu().numpy()]
        c.append(k, ys[2], starts, lens, tab)
        a = c.attend(q, starts, lens, tab)
        y = lins[3](a.view(B, H * D))
        assert c.status() == eva_vq.EVA_OK
        want, bound = ref.rope(ys[0].double().cpu().numpy().reshape(B, H, D), positions.tolist(), D, "half", freq, mag)
        close(q, want, bound, torch.float16)
        ref.append(kept[0], kept[1], k.double().cpu().numpy(), range(B + 1), lens.tolist(), table, "int8")
        assert np.array_equal(codes(c.k), kept[0])
        want, _, bound = ref.attend(q.double().cpu().numpy(), codes(c.k), c.k_scale.double().cpu().numpy(), codes(c.v),
                                    c.v_scale.double().cpu().numpy(), range(B + 1), lens.tolist(), table)
        close(a, want, bound, torch.float16)
        want = oracle.layer_linear(datas[3], a.view(B, H * D).cpu().numpy(), nthreads=8)
        assert np.all(norm_rel_err(y.float().cpu().numpy(), want) <= TOL)
        positions += 1
        x = y.view(B, 4096).half()
    for t in (*lins, rope, c):
        t.close()
