"""Pages that the caller filled, with scales outside the range that kv_append
gives: the older tokens' values stay what they were, as far as a scale of the
range can hold them.  Equal bit for bit."""
import numpy as np
import pytest

from gpu_support import say, torch_cuda
from kv_support import Case, dev_rows
from oracle import kv_oracle as K

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,total,block", [([1, 1], [20, 31], 16), ([3, 20], [20, 60], 32), ([5, 40], [70, 90], 64)])
@pytest.mark.parametrize("old", [-90, -66, -65, 120, 122, 127])
@pytest.mark.parametrize("zeros", [False, True])
def test_a_given_scale_outside_the_range(zeros, old, new, total, block):
    torch = torch_cuda()
    c = Case(20, new, total, 2, 64, block)
    lut = K.code_values()
    first = [n - m for m, n in zip(new, total)]
    pages = [int(c.table[i, a // block]) for i, a in enumerate(first)]
    for p in pages:
        c.cache["k_scale"][p] = c.cache["v_scale"][p] = 2.0 ** old
    before = {n: a.copy() for n, a in c.cache.items()}
    for n in c.cache:
        getattr(c.dev, n)[0].copy_(torch.from_numpy(c.cache[n]))
    x = c.row(c.n_rows) * (not zeros)  # of ordinary size, or asking for the least scale
    say(f"kv append, scale 2^{old} new={new} block={block}")
    c.M.kv_append(c.dev, 0, dev_rows(x), dev_rows(x), c.dev_batch())
    got = {n: getattr(c.dev, n)[0].cpu().numpy() for n in c.cache}
    for i, (p, a) in enumerate(zip(pages, first)):
        t0 = a % block
        assert t0 > 0
        in_page = x[c.row_off[i]:c.row_off[i] + min(new[i], block - t0)]
        for h in range(2):
            need = K.scale_exp(np.abs(in_page[:, h]).max())
            e = min(max(need, old), K.EXP_MAX)
            for n in ("k", "v"):
                assert got[n + "_scale"][p, h] == np.float32(2.0 ** e), (n, i)
                for t in range(t0):
                    at = (p, h, t) if n == "k" else (p, h, t // 16, slice(None), t % 16)
                    want = K.to_code(lut[before[n][at]] * 2.0 ** (old - e))
                    np.testing.assert_array_equal(got[n][at], want, f"{n} of sequence {i}, token {t}")
