"""Rotary positions, the 8-bit cache and attention over it where numbers, rows or pages are unusual: infinities and
NaN, dominating keys, large caps, released pages, very many parts, waits that run out, other streams."""
import numpy as np
import pytest
import torch

from tests.conftest import cuda_available
from tests.test_gpu_attention import cuda, i32, rng
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
