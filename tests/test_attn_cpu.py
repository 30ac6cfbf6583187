"""Rotary positions, cache and attention without a GPU: what the entry points refuse before any device work, and the
references against identities of their own."""
import ctypes

import numpy as np
import pytest

from tests import attn_reference as ref
from vector_quantized_weight_b200 import eva_vq

BAD, UNSUPPORTED = eva_vq.EVA_ERR_INVALID_ARG, eva_vq.EVA_ERR_UNSUPPORTED
P = 0x1000


def _rope(**kw):
    base = dict(q_heads=8, kv_heads=2, head_dim=128, rotary_dim=128, layout=0, norm=0, in_dtype=0, out_dtype=0, scaling=0,
                eps=1e-6, weight_offset=0.0, theta=1e4, factor=4.0, original=4096.0, low=1.0, high=32.0, magnitude=0.0)
    base.update(kw)
    return eva_vq.eva_rope_desc(*[base[f] for f, _ in eva_vq.eva_rope_desc._fields_])


def _rope_create(desc, qw=None, kw=None):
    h = ctypes.c_void_p()
    return eva_vq.load().eva_rope_create(ctypes.byref(h), ctypes.byref(desc), qw, kw, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(q_heads=0, kv_heads=0), BAD), (dict(q_heads=-1), BAD), (dict(head_dim=0), BAD), (dict(head_dim=1026, rotary_dim=64), UNSUPPORTED),
    (dict(rotary_dim=130), BAD), (dict(rotary_dim=63), BAD), (dict(layout=2), BAD), (dict(norm=2), BAD),
    (dict(in_dtype=2), BAD), (dict(out_dtype=7), BAD), (dict(theta=0.0), BAD), (dict(theta=float("nan")), BAD),
    (dict(scaling=5), BAD), (dict(scaling=1, factor=0.0), BAD), (dict(scaling=2, rotary_dim=2), BAD),
    (dict(scaling=3, original=0.0), BAD), (dict(scaling=3, low=40.0), BAD), (dict(scaling=3, theta=1.0), BAD),
    (dict(scaling=4, low=32.0), BAD), (dict(norm=1, eps=-1.0), BAD), (dict(norm=1, weight_offset=float("inf")), BAD),
    (dict(magnitude=-1.0), BAD),
])
def test_rope_refuses_bad_descriptors(kw, expect):
    assert _rope_create(_rope(**kw)) == expect


def test_rope_refuses_bad_pointers():
    lib = eva_vq.load()
    assert _rope_create(_rope(), qw=P) == BAD                      # weights without a norm
    assert _rope_create(_rope(norm=1), qw=P + 2) == BAD            # misaligned
    assert lib.eva_rope_create(None, ctypes.byref(_rope()), None, None, None) == BAD
    assert lib.eva_rope_run(None, P, 1024, P, 256, P, 1, P, 1024, P, 256, None) == BAD
    assert lib.eva_rope_destroy(None) == eva_vq.EVA_OK


def _kv(**kw):
    base = dict(q_heads=8, kv_heads=2, head_dim=128, page_size=64, num_pages=100, max_seqs=4, max_pages=10, cache_dtype=0,
                out_dtype=0, window=0, softcap=0.0, scale=0.0)
    base.update(kw)
    return eva_vq.eva_kv_desc(*[base[f] for f, _ in eva_vq.eva_kv_desc._fields_])


def _kv_create(desc, k=P, v=P, ks=P, vs=P):
    h = ctypes.c_void_p()
    return eva_vq.load().eva_kv_create(ctypes.byref(h), ctypes.byref(desc), k, v, ks, vs, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(q_heads=0), BAD), (dict(q_heads=7), BAD), (dict(kv_heads=0), BAD), (dict(head_dim=0), BAD),
    (dict(head_dim=96), UNSUPPORTED), (dict(page_size=0), BAD), (dict(page_size=48), UNSUPPORTED), (dict(num_pages=0), BAD),
    (dict(max_seqs=0), BAD), (dict(max_pages=0), BAD), (dict(cache_dtype=2), BAD), (dict(out_dtype=3), BAD),
    (dict(window=-1), BAD), (dict(softcap=-1.0), BAD), (dict(softcap=float("nan")), BAD), (dict(scale=-0.5), BAD),
    (dict(scale=float("inf")), BAD), (dict(max_pages=1 << 25), UNSUPPORTED), (dict(num_pages=1 << 30), UNSUPPORTED),
])
def test_cache_refuses_bad_descriptors(kw, expect):
    assert _kv_create(_kv(**kw)) == expect


def test_cache_refuses_bad_pointers_and_null_handles():
    lib = eva_vq.load()
    for kw in (dict(k=None), dict(v=None), dict(ks=None), dict(vs=None), dict(k=P + 8), dict(vs=P + 4)):
        assert _kv_create(_kv(), **kw) == BAD
    assert lib.eva_kv_create(None, ctypes.byref(_kv()), P, P, P, P, None) == BAD
    assert lib.eva_kv_append(None, P, 256, P, 256, 0, P, P, P, 1, 1, None) == BAD
    assert lib.eva_kv_read(None, P, P, P, 1, 1, 0, P, P, None) == BAD
    assert lib.eva_kv_attend(None, P, 1024, P, P, P, 1, 1, P, None, None) == BAD
    assert lib.eva_kv_sync_status(None) == BAD
    assert lib.eva_kv_debug_inject_wait_timeout(None, 5) == BAD
    assert lib.eva_kv_cache_info(None, None) == BAD
    assert lib.eva_kv_destroy(None) == eva_vq.EVA_OK


def test_create_without_device_reports_no_device():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    assert _rope_create(_rope()) == eva_vq.EVA_ERR_NO_DEVICE
    assert _kv_create(_kv()) == eva_vq.EVA_ERR_NO_DEVICE


def test_python_refusals():
    for kw in (dict(layout="both"), dict(in_dtype="bfloat16"), dict(scaling={"type": "cubic"}), dict(scaling={"factor": 2.0}),
               dict(scaling={"type": "linear", "factor": 2.0, "base": 3})):
        with pytest.raises(ValueError):
            eva_vq.HeadRope(2, 2, 64, **kw)
    for kw in (dict(dtype="int4"), dict(scale=0.0), dict(scale=-1.0), dict(out_dtype="bfloat16")):
        with pytest.raises(ValueError):
            eva_vq.KVCache(2, 2, 64, num_pages=1, max_seqs=1, max_pages=1, **kw)


def test_reference_rotation_keeps_lengths_and_relative_positions():
    r = np.random.default_rng(0)
    for layout in ("half", "interleaved"):
        freq, mag = ref.frequencies(32, 1e4, {"type": "ntk", "factor": 3.0})
        x, y = r.standard_normal((2, 1, 1, 48))
        at = lambda v, p: ref.rope(v, [p], 32, layout, freq, mag)[0]        # noqa: E731
        assert np.allclose(np.linalg.norm(at(x, 12345)), np.linalg.norm(x))
        assert np.allclose((at(x, 1007) * at(y, 1000)).sum(), (at(x, 7) * at(y, 0)).sum())
        assert np.array_equal(at(x, 99)[..., 32:], x[..., 32:])


def test_reference_e4m3_is_torchs():
    import torch
    x = np.concatenate([np.random.default_rng(1).standard_normal(4000) * 100, [0.0, 448, -449, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9]])
    x = ref.f32(x)
    want = torch.from_numpy(np.clip(x, -448, 448)).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.encode(x, "e4m3"), want)


def test_reference_attention_of_one_page_is_a_softmax():
    r = np.random.default_rng(2)
    k, v = r.integers(-127, 128, (2, 1, 1, 16, 8)).astype(float)
    q = r.standard_normal((2, 1, 8))
    out, lse, _ = ref.attend(q, k, np.full((1, 1), 0.01), v, np.full((1, 1), 0.02), [0, 2], [16], [[0]])
    for i in range(2):
        z = (k[0, 0, :15 + i] * 0.01) @ q[i, 0] / np.sqrt(8)
        p = np.exp(z) / np.exp(z).sum()
        assert np.allclose(out[i, 0], p @ (v[0, 0, :15 + i] * 0.02)) and np.isclose(lse[i, 0], np.log(np.exp(z).sum()))
