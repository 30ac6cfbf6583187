"""The operators between a decoder block's q/k/v linears and its o linear, as they are measured:

  rope    rotary positions on queries and keys, optionally with the per-head RMS norm in the same pass
  write   new keys and values into a paged 8-bit cache (one scale for each page and head), and read back
  attend  attention of new tokens over that cache

`own` chooses between the plain form (elementary torch operations, 32 or 64 bits, rounded once at the end) and
the calls a user makes of the framework.
"""
import math

import torch

own = False

DEV = "cuda"
LARGEST = {"int8": 127.0, "e4m3": 448.0}      # the largest code
SPREAD = {"int8": 32.0, "e4m3": 100.0}        # the standard deviation of the codes that are made up


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of one sequence: a decode step of the 32-head, 4096-wide block, where latency counts
        dict(name="rope_one_token", op="rope", T=1, q_heads=32, kv_heads=32, head_dim=128, rotary=128, layout="half",
             scaling="none", norm=False, dtype="float16", fused=False, far=4096),
        # a long document's stretch at positions near a million: interleaved pairs, half of each head, fp32 from the linears
        dict(name="rope_far_interleaved", op="rope", T=1777, q_heads=32, kv_heads=8, head_dim=128, rotary=64,
             layout="interleaved", scaling="yarn", norm=False, dtype="float32", fused=False, far=1000000),
        # a decode step of 64 sequences (the linears' largest batch) in the 8192-wide block with normed heads
        dict(name="norm_rope_batch", op="rope", T=64, q_heads=64, kv_heads=8, head_dim=128, rotary=128, layout="half",
             scaling="none", norm=True, dtype="float16", fused=False, far=8192),
        # a prompt's tokens, q and k as column ranges of one fused projection buffer
        dict(name="norm_rope_prompt", op="rope", T=8192, q_heads=64, kv_heads=8, head_dim=128, rotary=128,
             layout="half", scaling="bands", norm=True, dtype="float16", fused=True, far=131072),
        # the cache's share of a 64-sequence decode step: one token each into partly filled pages
        dict(name="write_step", op="write", seqs=64, new=1, context=4096, kv_heads=8, head_dim=128, page=64,
             cache="int8", dtype="float16"),
        # the prompts of three requests at once, the first page of each partly filled by what came before
        dict(name="write_prompt", op="write", seqs=3, new=2100, context=500, kv_heads=8, head_dim=128, page=32,
             cache="e4m3", dtype="float16"),
        # one chat turn at batch 1, 32 heads of their own keys: the smallest call
        dict(name="attend_one_short", op="attend", seqs=1, new=1, context=517, ragged=False, q_heads=32, kv_heads=32,
             head_dim=128, page=64, cache="int8", window=0, softcap=0.0),
        # a decode step of 64 sequences of very different lengths, eight queries to a key head
        dict(name="attend_batch", op="attend", seqs=64, new=1, context=4096, ragged=True, q_heads=64, kv_heads=8,
             head_dim=128, page=64, cache="int8", window=0, softcap=0.0),
        # one sequence with a long context, an odd length
        dict(name="attend_long", op="attend", seqs=1, new=1, context=131071, ragged=False, q_heads=64, kv_heads=8,
             head_dim=128, page=128, cache="int8", window=0, softcap=0.0),
        # heads of 256 with a sliding window and capped scores, small pages, e4m3
        dict(name="attend_window", op="attend", seqs=16, new=1, context=9001, ragged=True, q_heads=16, kv_heads=8,
             head_dim=256, page=16, cache="e4m3", window=4096, softcap=50.0),
        # a prompt's chunk of 64 tokens (the linears' largest batch) over what is cached already
        dict(name="attend_chunk", op="attend", seqs=1, new=64, context=8191, ragged=False, q_heads=64, kv_heads=8,
             head_dim=128, page=64, cache="int8", window=0, softcap=0.0),
        # drafted tokens checked in one call: five for each of eight sequences, heads of 64
        dict(name="attend_draft", op="attend", seqs=8, new=5, context=3001, ragged=True, q_heads=32, kv_heads=4,
             head_dim=64, page=32, cache="e4m3", window=0, softcap=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "write", "attend", "attend"])
    D = rng.choice([64, 128, 256])
    kv, group = rng.choice([(1, 8), (2, 7), (4, 4), (8, 1), (8, 2), (8, 8), (5, 3), (32, 1)])
    cache = rng.choice(["int8", "e4m3"])
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        T = max(1, min(_log(rng, 1, 16384), (8192 * 72 * 128) // ((kv + kv * group) * D)))
        rotary = rng.choice([D, D, D // 2, D // 4, 3 * D // 8])
        return dict(op="rope", T=T, q_heads=kv * group, kv_heads=kv, head_dim=D, rotary=rotary,
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]), norm=rng.random() < 0.5,
                    dtype=rng.choice(["float16", "float16", "float32"]), fused=rng.random() < 0.5,
                    far=_log(rng, 1000, 1000000))
    seqs = _log(rng, 1, 64)
    if op == "write":
        new = min(rng.choice([1, 1, _log(rng, 2, 6000)]), max(1, 6300 * 1024 // (seqs * kv * D)))
        context = min(_log(rng, 1, 4096), max(1, 64 * 4096 * 1024 // (seqs * kv * D)))
        return dict(op="write", seqs=seqs, new=new, context=context, kv_heads=kv, head_dim=D, page=page, cache=cache,
                    dtype=rng.choice(["float16", "float16", "float32"]))
    new = rng.choice([1, 1, 1, _log(rng, 2, 64)])
    context = _log(rng, 1, 131072)
    context = max(1, min(context, 131072 * 1024 // (seqs * kv * D)))                       # bytes of the cache
    context = max(1, min(context, 64 * 64 * 8191 * 128 // (seqs * new * kv * group * D)))  # products
    return dict(op="attend", seqs=seqs, new=new, context=context, ragged=rng.random() < 0.7, q_heads=kv * group,
                kv_heads=kv, head_dim=D, page=page, cache=cache, window=rng.choice([0, 0, 0, 1000]),
                softcap=rng.choice([0.0, 0.0, 30.0]))


# ------------------------------------------------------------------ inputs

THETA = 10000.0
SCALING = {"none": None,
           "linear": {"type": "linear", "factor": 4.0},
           "ntk": {"type": "ntk", "factor": 8.0},
           "yarn": {"type": "yarn", "factor": 16.0, "original": 4096},
           "bands": {"type": "bands", "factor": 8.0, "low": 1.0, "high": 4.0, "original": 8192}}
EPS = 1e-6


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _ints(g, lo, hi, n):
    return torch.randint(lo, hi, (n,), generator=g, device=DEV, dtype=torch.int64)


def _rope_inputs(case, seed):
    g = _gen(seed)
    T, Hq, Hk, D = case["T"], case["q_heads"], case["kv_heads"], case["head_dim"]
    dtype = getattr(torch, case["dtype"])
    if case["fused"]:      # columns of one projection's output, which holds v as well
        rows = _randn(g, T, (Hq + 2 * Hk) * D, dtype=dtype)
        q = rows[:, :Hq * D].view(T, Hq, D)
        k = rows[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    else:
        q, k = _randn(g, T, Hq, D, dtype=dtype), _randn(g, T, Hk, D, dtype=dtype)
    s = dict(case=case, q=q, k=k, positions=_ints(g, 0, case["far"], T).sort().values.to(torch.int32))
    if case["norm"]:
        s["q_weight"] = (1 + 0.1 * _randn(g, D)).half()
        s["k_weight"] = (1 + 0.1 * _randn(g, D)).half()
    return s


def _lengths(case, g):
    """Cached tokens of each sequence before the call: the longest is `context`.  The lengths go by the case, and
    the seed says which sequence has which, so that what comes back always has the same shape."""
    B, context = case["seqs"], case["context"]
    if case.get("ragged", True) and B > 1:
        n = _ints(_gen(context), 1, context + 1, B)
        n[0] = context
        return n[torch.randperm(B, generator=g, device=DEV)]
    return torch.full((B,), context, device=DEV, dtype=torch.int64)


def _codes(g, cache, *shape):
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float16) * SPREAD[cache]
    if cache == "int8":
        return x.round_().clamp_(-127, 127).to(torch.int8)
    return x.clamp_(-448, 448).to(torch.float8_e4m3fn)


def _paged(case, g, total):
    """A page table of random pages for sequences of `total` tokens, and the cache's buffers."""
    B, P, H, D = case["seqs"], case["page"], case["kv_heads"], case["head_dim"]
    longest = case["context"] + case["new"]
    width = -(-longest // P)
    used = -(-total // P)
    pages = int(used.sum())
    order = torch.randperm(pages, generator=g, device=DEV)
    col = torch.arange(width, device=DEV)
    valid = col[None] < used[:, None]
    first = used.cumsum(0) - used
    table = torch.where(valid, order[(first[:, None] + col[None]).clamp_(max=pages - 1)], -1).to(torch.int32)
    s = dict(page_table=table)
    for x in ("k", "v"):
        s[x + "_pages"] = _codes(g, case["cache"], pages, H, P, D)
        s[x + "_scale"] = (0.5 + torch.rand((pages, H), generator=g, device=DEV)) / SPREAD[case["cache"]]
        # what lies behind a sequence's last token in its last page is whatever was there: every bit set but the sign
        last = table.gather(1, (used - 1)[:, None])[:, 0].long()
        behind = torch.arange(P, device=DEV)[None] >= (total - (used - 1) * P)[:, None]
        raw = s[x + "_pages"].view(torch.uint8)
        raw[last] = torch.where(behind[:, None, :, None], torch.full_like(raw[:1], 127), raw[last])
    return s


def _write_inputs(case, seed):
    g = _gen(seed)
    B, n, H, D = case["seqs"], case["new"], case["kv_heads"], case["head_dim"]
    old = _lengths(case, g)
    s = dict(case=case, old=old, **_paged(case, g, old + n))
    dtype = getattr(torch, case["dtype"])
    channel = torch.exp(0.5 * _randn(g, 1, H, D))       # some channels of keys are larger than others
    s["k"] = (_randn(g, B * n, H, D) * channel).to(dtype)
    s["v"] = _randn(g, B * n, H, D).to(dtype)
    s["starts"] = (torch.arange(B + 1, device=DEV) * n).to(torch.int32)
    s["lens"] = (old + n).to(torch.int32)
    # read back: from the start of the first page that is written
    P = case["page"]
    begin = old // P * P
    s["begin"] = begin.to(torch.int32)
    s["back"] = torch.cat([torch.zeros(1, device=DEV, dtype=torch.int64), (old + n - begin).cumsum(0)]).to(torch.int32)
    s["rows"] = int(s["back"][-1])
    s["touched"] = int(((old + n - 1) // P - old // P).max()) + 1
    return s


def _attend_inputs(case, seed):
    g = _gen(seed)
    B, n, Hq, D = case["seqs"], case["new"], case["q_heads"], case["head_dim"]
    old = _lengths(case, g)
    s = dict(case=case, **_paged(case, g, old + n))
    s["q"] = _randn(g, B * n, Hq, D, dtype=torch.float16)
    s["starts"] = (torch.arange(B + 1, device=DEV) * n).to(torch.int32)
    s["lens"] = (old + n).to(torch.int32)
    return s


INPUTS = {"rope": _rope_inputs, "write": _write_inputs, "attend": _attend_inputs}


def _frequencies(case):
    """Rotations a position of each pair of dimensions, in 64 bits, and the magnitude of cos and sin."""
    R, how = case["rotary"], SCALING[case["scaling"]]
    i = torch.arange(R // 2, device=DEV, dtype=torch.float64)
    theta = THETA
    if case["scaling"] == "ntk":
        theta = THETA * how["factor"] ** (R / (R - 2))
    f = theta ** (-2 * i / R)
    if case["scaling"] == "linear":
        return f / how["factor"], 1.0
    if case["scaling"] == "yarn":
        at = [R * math.log(how["original"] / (2 * math.pi * b)) / (2 * math.log(theta)) for b in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), R - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f * (1 - ramp) + f / how["factor"] * ramp, 0.1 * math.log(how["factor"]) + 1
    if case["scaling"] == "bands":
        turns = how["original"] * f / (2 * math.pi)
        blend = ((turns - how["low"]) / (how["high"] - how["low"])).clamp(0, 1)
        return f / how["factor"] * (1 - blend) + f * blend, 1.0
    return f, 1.0


def prepare(case, seed):
    s = INPUTS[case["op"]](case, seed)
    if case["op"] == "rope":
        s["freq"], s["magnitude"] = _frequencies(case)
    if case["op"] == "attend":
        s["scale"] = case["head_dim"] ** -0.5
    if own:
        from vector_quantized_weight_b200 import eva_vq
        if case["op"] == "rope":
            s["rope"] = eva_vq.HeadRope(case["q_heads"], case["kv_heads"], case["head_dim"], rotary_dim=case["rotary"],
                                        layout=case["layout"], theta=THETA, scaling=SCALING[case["scaling"]],
                                        norm=case["norm"], q_weight=s.get("q_weight"), k_weight=s.get("k_weight"),
                                        eps=EPS, in_dtype=case["dtype"])
        else:
            pages = s["k_pages"].shape[0]
            s["cache"] = eva_vq.KVCache(case.get("q_heads", case["kv_heads"]), case["kv_heads"], case["head_dim"],
                                        num_pages=pages, page_size=case["page"], max_seqs=case["seqs"],
                                        max_pages=s["page_table"].shape[1], dtype=case["cache"],
                                        window=case.get("window", 0), softcap=case.get("softcap", 0.0),
                                        k=s["k_pages"], v=s["v_pages"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return s


# ------------------------------------------------------------------ the plain forms

def _rotate(x, weight, s):
    case = s["case"]
    R, out = case["rotary"], torch.float16
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    angle = (s["positions"].double()[:, None] * s["freq"][None])[:, None]
    cos, sin = (angle.cos() * s["magnitude"]).float(), (angle.sin() * s["magnitude"]).float()
    if case["layout"] == "half":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., R:]], -1).to(out)
    a, b = x[..., 0:R:2], x[..., 1:R:2]
    turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., R:]], -1).to(out)


def _to_codes(x, cache):
    if cache == "int8":
        return x.round().clamp(-127, 127).to(torch.int8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.int8)


def _from_codes(raw, cache):
    return raw.float() if cache == "int8" else raw.view(torch.float8_e4m3fn).float()


def _write(x, pages, scale, s):
    """x [T][H][D] into `pages`, each page's scale the largest it has needed since its first slot was written."""
    case = s["case"]
    P, n, B = case["page"], case["new"], case["seqs"]
    raw = pages.view(torch.int8)
    x = x.float()
    pos = (s["old"][:, None] + torch.arange(n, device=DEV)[None]).reshape(-1)
    seq = torch.arange(B, device=DEV).repeat_interleave(n)
    page, slot = s["page_table"][seq, pos // P].long(), pos % P
    # the pages that are written: each sequence's, the last one repeated where it has fewer than the others
    at = torch.minimum((s["old"] // P)[:, None] + torch.arange(s["touched"], device=DEV)[None],
                       ((s["old"] + n - 1) // P)[:, None])
    mine = s["page_table"].gather(1, at).long().reshape(-1)
    first = torch.where(at == (s["old"] // P)[:, None], (s["old"] % P)[:, None], 0).reshape(-1)
    new = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(-1), "amax")[mine]
    new = new / torch.full_like(new, LARGEST[case["cache"]])
    was = torch.where(first[:, None] > 0, scale[mine], 0.0)
    now = torch.maximum(was, new)
    ratio = torch.where(now > 0, was / now, 0.0)
    kept = raw[mine]
    again = _to_codes(_from_codes(kept, case["cache"]) * ratio[:, :, None, None], case["cache"])
    before = torch.arange(P, device=DEV)[None] < first[:, None]
    raw[mine] = torch.where((before[:, None, :] & (was < now)[:, :, None])[..., None], again, kept)
    scale[mine] = now
    by = scale[page][..., None]
    raw[page, :, slot] = _to_codes(torch.where(by > 0, x / by, 0.0), case["cache"])


def _read(pages, scale, s):
    case = s["case"]
    P = case["page"]
    row = torch.arange(s["rows"], device=DEV)
    seq = torch.searchsorted(s["back"].long(), row, right=True) - 1
    pos = s["begin"].long()[seq] + row - s["back"].long()[seq]
    page = s["page_table"][seq, pos // P].long()
    x = _from_codes(pages.view(torch.int8)[page, :, pos % P], case["cache"])
    return (x * scale[page][..., None]).half()


def _attend(s):
    case = s["case"]
    B, n, Hq, H, D, P = (case[x] for x in ("seqs", "new", "q_heads", "kv_heads", "head_dim", "page"))
    table, lens = s["page_table"].long().clamp(min=0), s["lens"].long()
    L = table.shape[1] * P
    position = lens[:, None] - n + torch.arange(n, device=DEV)[None]                    # [B][n]
    j = torch.arange(L, device=DEV)
    seen = j[None, None] <= position[:, :, None]
    if case["window"]:
        seen = seen & (j[None, None] > position[:, :, None] - case["window"])           # [B][n][L]

    def gathered(x):
        v = _from_codes(s[x + "_pages"].view(torch.int8)[table], case["cache"]) * s[x + "_scale"][table][..., None, None]
        v = v.permute(0, 2, 1, 3, 4).reshape(B, H, L, D)
        return torch.where((j[None] < lens[:, None])[:, None, :, None], v, 0.0)

    q = s["q"].float().view(B, n, H, Hq // H, D).permute(0, 2, 1, 3, 4).reshape(B, H, n * (Hq // H), D)
    z = (q * s["scale"]) @ gathered("k").transpose(-1, -2)
    if case["softcap"]:
        z = case["softcap"] * torch.tanh(z / case["softcap"])
    z = torch.where(seen.repeat_interleave(Hq // H, 1)[:, None], z, -math.inf)
    z = z - z.amax(-1, keepdim=True)
    p = z.exp()
    o = (p @ gathered("v")) / p.sum(-1, keepdim=True)
    return o.view(B, H, n, Hq // H, D).permute(0, 2, 1, 3, 4).reshape(B * n, Hq, D).half()


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        if op == "rope":
            return s["rope"](s["q"], s["k"], s["positions"])
        if op == "write":
            s["cache"].append(s["k"], s["v"], s["starts"], s["lens"], s["page_table"])
            return s["cache"].read(s["back"], s["begin"], s["page_table"], s["rows"])
        return s["cache"].attend(s["q"], s["starts"], s["lens"], s["page_table"])
    if op == "rope":
        return _rotate(s["q"], s.get("q_weight"), s), _rotate(s["k"], s.get("k_weight"), s)
    if op == "write":
        _write(s["k"], s["k_pages"], s["k_scale"], s)
        _write(s["v"], s["v_pages"], s["v_scale"], s)
        return _read(s["k_pages"], s["k_scale"], s), _read(s["v_pages"], s["v_scale"], s)
    return _attend(s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    size = {"float16": 2, "float32": 4}.get(case.get("dtype"), 2)
    D = case["head_dim"]
    if case["op"] == "rope":
        n = case["T"] * (case["q_heads"] + case["kv_heads"]) * D
        return {"bytes": n * (size + 2) + 4 * case["T"], "flops": n * (7 if case["norm"] else 3)}
    B, H, new, context = case["seqs"], case["kv_heads"], case["new"], case["context"]
    ragged = case.get("ragged", True) and B > 1
    if case["op"] == "write":
        n = B * new * H * D * 2                       # in, codes out; read back: codes in, values out
        back = n + B * H * D * (case["page"] - 1)     # on average half a page of older tokens, k and v
        return {"bytes": n * (size + 1) + back * 3, "flops": 4 * n}
    mean = context + new if not ragged else (context + 1) / 2 + new
    if case["window"]:
        w = case["window"] + new - 1
        spread = context + new if ragged else 0
        mean = min(mean, w) if not spread else (w - w * w / (2 * spread) if spread > w else mean)
    rows = B * new * case["q_heads"]
    return {"bytes": B * mean * H * (D * 2 + 8 / case["page"]) + rows * D * 4,
            "flops": 4 * rows * D * max(1.0, mean - (new - 1) / 2)}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_rope(s):
    case = s["case"]
    D, R = case["head_dim"], case["rotary"]
    how, outs = SCALING[case["scaling"]], []
    freqs = []
    for i in range(R // 2):
        f = THETA ** (-2.0 * i / R)
        if case["scaling"] == "linear":
            f /= how["factor"]
        elif case["scaling"] == "ntk":
            f = (THETA * how["factor"] ** (R / (R - 2.0))) ** (-2.0 * i / R)
        elif case["scaling"] == "yarn":
            def edge(beta):
                return R * math.log(how["original"] / (beta * 2 * math.pi)) / (2 * math.log(THETA))
            lo, hi = max(math.floor(edge(32.0)), 0), min(math.ceil(edge(1.0)), R - 1)
            far = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = f / how["factor"] * far + f * (1 - far)
        elif case["scaling"] == "bands":
            wave = 2 * math.pi / f
            if wave > how["original"] / how["low"]:
                f /= how["factor"]
            elif wave >= how["original"] / how["high"]:
                t = (how["original"] / wave - how["low"]) / (how["high"] - how["low"])
                f = (1 - t) * f / how["factor"] + t * f
        freqs.append(f)
    m = 0.1 * math.log(how["factor"]) + 1 if case["scaling"] == "yarn" else 1.0
    z = torch.polar(torch.full((case["T"], R // 2), m, device=DEV, dtype=torch.float64),
                    s["positions"].double()[:, None] * torch.tensor(freqs, device=DEV, dtype=torch.float64))
    low = torch.arange(R // 2, device=DEV)
    first, second = (low, low + R // 2) if case["layout"] == "half" else (2 * low, 2 * low + 1)
    for name in ("q", "k"):
        x = s[name].double().clone()
        if case["norm"]:
            x = x / ((x ** 2).sum(-1, keepdim=True) / D + EPS).sqrt() * s[name + "_weight"].double()
        y = torch.complex(x[..., first], x[..., second]) * z[:, None]
        x[..., first], x[..., second] = y.real, y.imag
        outs.append(x)
    return tuple(outs)


def _nearest_e4m3(x):
    """The nearest value with 4 exponent and 3 fraction bits (ties to even), at most 448."""
    _, e = torch.frexp(x.abs().clamp(min=2.0 ** -6))
    step = torch.ldexp(torch.ones_like(x), e - 4)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_write(s):
    """Page by page.  A scale is a 32-bit number and a code is the rounded 32-bit quotient: both by definition."""
    case = s["case"]
    P, cache, n = case["page"], case["cache"], case["new"]
    single = lambda x: x.float().double()                                              # noqa: E731
    nearest = (lambda x: x.round().clamp(-127, 127)) if cache == "int8" else _nearest_e4m3
    old, table, outs = s["old"].tolist(), s["page_table"].tolist(), []
    for name in ("k", "v"):
        back = []
        for b in range(case["seqs"]):
            for index in range(old[b] // P, (old[b] + n - 1) // P + 1):
                page = table[b][index]
                lo, hi = max(index * P, old[b]), min((index + 1) * P, old[b] + n)
                x = s[name][b * n + lo - old[b]:b * n + hi - old[b]].double()          # [t][H][D]
                codes = s[name + "_pages"][page].double()[:, :lo - index * P].transpose(0, 1)
                was = s[name + "_scale"][page].double() if lo > index * P else torch.zeros_like(x[0, :, 0])
                now = torch.maximum(was, single(x.abs().amax((0, 2)) / LARGEST[cache]))
                ratio = single(torch.where(now > 0, was / now, 0.0))[None, :, None]
                codes = torch.where((now > was)[None, :, None], nearest(single(codes * ratio)), codes)
                fresh = nearest(single(torch.where(now[None, :, None] > 0, x / now[None, :, None], 0.0)))
                back.append(torch.cat([codes, fresh]) * now[None, :, None])
        outs.append(torch.cat(back))
    return tuple(outs)


def _exact_attend(s):
    case = s["case"]
    n, Hq, H, D, P = (case[x] for x in ("new", "q_heads", "kv_heads", "head_dim", "page"))
    G, outs = Hq // H, []
    for b, total in enumerate(s["lens"].tolist()):
        pages = s["page_table"][b, :-(-total // P)].long()
        k, v = ((s[x + "_pages"].view(torch.uint8)[pages].view(s[x + "_pages"].dtype).double()
                 * s[x + "_scale"][pages].double()[..., None, None]).transpose(0, 1).reshape(H, -1, D)[:, :total]
                for x in ("k", "v"))
        for i in range(n):
            end = total - n + i + 1
            begin = max(0, end - case["window"]) if case["window"] else 0
            q = s["q"][b * n + i].double().view(H, G, D)
            z = torch.einsum("hgd,htd->hgt", q, k[:, begin:end]) / math.sqrt(D)
            if case["softcap"]:
                z = case["softcap"] * torch.tanh(z / case["softcap"])
            outs.append(torch.einsum("hgt,htd->hgd", torch.softmax(z, -1), v[:, begin:end]).reshape(Hq, D))
    return torch.stack(outs)


def exact(case, seed):
    return {"rope": _exact_rope, "write": _exact_write, "attend": _exact_attend}[case["op"]](INPUTS[case["op"]](case, seed))
