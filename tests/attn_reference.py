"""64-bit references of the rotary positions, the 8-bit cache and the attention over it, from their formulas, one
loop at a time (test infrastructure; shares no code with the library), and the error bounds the tests use."""
from __future__ import annotations

import math

import numpy as np
import torch

LARGEST = {"int8": 127.0, "e4m3": 448.0}


# ------------------------------------------------------------------ rotary positions

def frequencies(R, theta=10000.0, scaling=None):
    how = dict(scaling or {})
    kind, out = how.get("type", "none"), []
    for i in range(R // 2):
        base = theta * how["factor"] ** (R / (R - 2)) if kind == "ntk" else theta
        f = base ** (-2 * i / R)
        if kind == "linear":
            f = f / how["factor"]
        if kind == "yarn":
            def dim(turns):
                return R * math.log(how["original"] / (2 * math.pi * turns)) / (2 * math.log(theta))
            a, b = max(math.floor(dim(how.get("high", 32.0))), 0), min(math.ceil(dim(how.get("low", 1.0))), R - 1)
            r = min(max((i - a) / max(b - a, 0.001), 0.0), 1.0)
            f = f * (1 - r) + f / how["factor"] * r
        if kind == "bands":
            n = how["original"] * f / (2 * math.pi)
            s = min(max((n - how.get("low", 1.0)) / (how.get("high", 4.0) - how.get("low", 1.0)), 0.0), 1.0)
            f = f / how["factor"] * (1 - s) + f * s
        out.append(f)
    m = how.get("magnitude") or (0.1 * math.log(how["factor"]) + 1 if kind == "yarn" and how["factor"] > 1 else 1.0)
    return np.array(out, dtype=np.longdouble), m


def rope(x, positions, R, layout, freq, magnitude, norm=False, weight=None, eps=1e-6, offset=0.0):
    """x [T][H][D] (any float array) -> (float64 result, bound on the fp32 error of each element before it is rounded).

    The bound: the reduced angle is off by at most 2^-24 of half a turn (2e-7), cos and sin by 2 ulp (2.4e-7), four
    products and sums by 2^-24 each, the norm by 2^-22 (rsqrt) and half a ulp for each of the at most 32 sums of a
    lane and shuffles: 3e-6 of the pair's length in all."""
    x = np.asarray(x, np.float64)
    T, H, D = x.shape
    if norm:
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        x = x * r * (1.0 if weight is None else np.asarray(weight, np.float64) + offset)
    y, size = x.copy(), np.abs(x)
    for i in range(R // 2):
        a, b = (i, i + R // 2) if layout == "half" else (2 * i, 2 * i + 1)
        turns = np.asarray(positions, np.longdouble) * freq[i] / (2 * np.longdouble(math.pi) + np.longdouble(2.4492935982947064e-16))
        ang = (turns - np.floor(turns)).astype(np.float64) * 2 * math.pi
        c, s = np.cos(ang)[:, None] * magnitude, np.sin(ang)[:, None] * magnitude
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        size[..., a] = size[..., b] = np.hypot(x[..., a], x[..., b]) * max(1.0, magnitude)
    return y, 3e-6 * size


def rounded(y, bound, dtype):
    """The bound with the final rounding to `dtype` (half a step; half of the smallest subnormal near zero)."""
    eps = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -149
    return bound * (1 + eps) + eps * np.abs(y) + tiny


# ------------------------------------------------------------------ the cache

def encode(x, cache):
    """float64 values that are fp32 numbers -> codes as float64 (int8: round half to even; e4m3: nearest even)."""
    if cache == "int8":
        return np.clip(np.rint(x), -127, 127)
    ax = np.minimum(np.abs(x), 448.0)
    step = 2.0 ** (np.floor(np.log2(np.maximum(ax, 2.0 ** -6))) - 3)
    return np.sign(x) * np.minimum(np.rint(ax / step) * step, 448.0)


def f32(x):
    return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def append(codes, scale, x, starts, lens, table, cache):
    """codes [pages][H][P][D] and scale [pages][H] (float64, changed in place) after x [T][H][D] is written."""
    P = codes.shape[2]
    x = np.clip(np.nan_to_num(np.asarray(x, np.float64), nan=0.0, posinf=65504.0, neginf=-65504.0), -65504, 65504)
    for b in range(len(lens)):
        n = int(starts[b + 1] - starts[b])
        by_page = {}
        for i in range(n):
            pos = int(lens[b]) - n + i
            if pos >= 0:
                by_page.setdefault(pos // P, []).append((pos % P, int(starts[b]) + i))
        for j, rows in by_page.items():
            page = int(table[b][j])
            if not 0 <= page < codes.shape[0]:
                continue
            slots, at = [r[0] for r in rows], [r[1] for r in rows]
            for h in range(codes.shape[1]):
                v = x[at, h]
                was = scale[page, h] if slots[0] > 0 else 0.0
                now = max(was, f32(np.abs(v).max() / LARGEST[cache]))
                if slots[0] > 0 and now > was:
                    kept = codes[page, h, :slots[0]]
                    codes[page, h, :slots[0]] = encode(f32(kept * f32(was / now)), cache)
                codes[page, h, slots] = encode(f32(v / now), cache) if now > 0 else 0.0
                scale[page, h] = now


# ------------------------------------------------------------------ attention

def attend(q, codes_k, scale_k, codes_v, scale_v, starts, lens, table, *, window=0, softcap=0.0, scale=None, T=None):
    """float64 outputs and lse, and the error bound of each output element before it is rounded; rows that no
    sequence has stay NaN.  Codes are float64 values (the code numbers).

    The bound: a weight is rounded to fp16 (2^-11 of it; below 2^-14 of the largest, 2^-25 of the largest), a score
    is off by the fp32 sums of its products (2^-24 of the sum of their sizes for each of the at most 16 additions
    the tensor cores chain, twice for scale and exponential) and by 1e-6 of the cap."""
    q = np.asarray(q, np.float64)
    rows, Hq, D = q.shape
    H, P = codes_k.shape[1], codes_k.shape[2]
    G = Hq // H
    scale = D ** -0.5 if scale is None else scale
    out = np.full((rows, Hq, D), np.nan)
    lse = np.full((rows, Hq), np.nan)
    bound = np.zeros((rows, Hq, D))
    for b in range(len(lens)):
        n, total = int(starts[b + 1] - starts[b]), int(lens[b])
        for i in range(n):
            pos = total - n + i
            keys = [j for j in range(max(0, pos - window + 1) if window else 0, pos + 1)
                    if 0 <= int(table[b][j // P]) < codes_k.shape[0]]
            page = np.array([int(table[b][j // P]) for j in keys], int)
            slot = np.array([j % P for j in keys], int)
            for hq in range(Hq):
                h, r = hq // G, int(starts[b]) + i
                if not keys:
                    out[r, hq], lse[r, hq] = 0.0, -np.inf
                    continue
                k = codes_k[page, h, slot] * scale_k[page, h][:, None]
                v = codes_v[page, h, slot] * scale_v[page, h][:, None]
                z = k @ q[r, hq] * scale
                dz = 2 * 16 * 2.0 ** -24 * (np.abs(k) @ np.abs(q[r, hq])) * scale + 4e-7 * np.abs(z).max()
                if softcap:
                    z = softcap * np.tanh(z / softcap)
                    dz = dz + 1e-6 * softcap
                m = z.max()
                p = np.exp(z - m)
                l = p.sum()
                out[r, hq], lse[r, hq] = p @ v / l, m + np.log(l)
                av = p @ np.abs(v) / l
                big = np.abs(codes_v[page, h, slot]).max() * scale_v[page, h].max()
                bound[r, hq] = (2.0 ** -11 + 2 * dz.max() + 2e-6) * av + len(keys) * 2.0 ** -25 * big
    return out, lse, bound
