"""Scores whose size leaves a float no room for what tells them apart: the
largest one still has weight 1 and what lies far below it none."""
import numpy as np
import pytest

from gpu_support import say, torch_cuda
from kv_support import dev_rows
from oracle import kv_oracle as K
from test_gpu_kv_attention_forms import _case, _put

pytestmark = pytest.mark.gpu

BATCHES = {"few": ([1, 2, 1], [40, 150, 4000]), "many": ([70, 30], [70, 700])}


@pytest.mark.parametrize("exponent", [20, 27, 29, 33, 40, 90])
@pytest.mark.parametrize("form", ["whole", "parts"])
@pytest.mark.parametrize("name", sorted(BATCHES))
def test_the_largest_of_huge_scores(name, form, exponent):
    """Keys are one of -1, -1/2, 1/2 and 1 in all channels (times 2^b) and a
    query has one number in all of them (8 significant bits, times 2^a), so every
    product and sum is exact in fp32, scores are those of 2^exponent, their
    products with scale * log2(e) have more bits than a float, and tokens that
    share the largest share the weight.  Tolerance: the probabilities' rounding to bf16
    and the output's, 2^-8 each of sum p |v|, and 2^-12 for sums in fp32 (at
    most 4000 terms of 2^-24)."""
    new, total = BATCHES[name]
    if form == "whole":
        total = [min(n, 700) for n in total]
    c = _case(form, 100 + exponent, new, total, 2, 64, 16)
    a = exponent // 2
    # scores: 64 * 2^(a + b) / 8 = 2^exponent times the keys' factor
    b = exponent - 3 - a
    size = np.array([0x28, 0x30, 0xb0, 0xa8], np.uint8)  # 1/4, 1/2, -1/2, -1/4: times 2^(b + 1)
    page, heads = c.cache["k"].shape[:2]
    factor = size[c.rng.choice(4, p=[0.45, 0.05, 0.05, 0.45], size=(page, heads, c.block, 1))]
    c.cache["k"][:] = factor
    c.cache["k_scale"][:] = 2.0 ** (b + 1)
    sign = np.where(c.rng.random((c.n_rows, 8, 1)) < 0.5, -1.0, 1.0)
    q = sign * (1 + c.rng.integers(0, 128, size=(c.n_rows, 8, 1)) / 128) * np.full(64, 2.0 ** a)
    _put(c)
    say(f"kv attention huge scores {name} {form} 2^{exponent}")
    got = c.M.kv_attention(c.dev, 0, dev_rows(q), c.dev_batch()).double().cpu().numpy()
    ref, _ = K.attention(c.cache, q, c.batch)
    c.cache["v"] = np.where((c.cache["v"] & 0x7f) == 0x7f, c.cache["v"], c.cache["v"] & 0x7f).astype(np.uint8)
    size, _ = K.attention(c.cache, q, c.batch)  # sum p |v|
    assert np.isfinite(ref).all() and np.isfinite(got).all()
    err = np.abs(got - ref) - size * (2.0 ** -7 + 2.0 ** -12)
    at = np.unravel_index(np.argmax(err), err.shape)
    assert err[at] <= 0, f"{got[at]} != {ref[at]} at {at}"
