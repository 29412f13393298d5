"""kv_attention's forms against the numpy oracle where a mask splits a step:
an item whole in one workgroup (narrow tables), and the work dealt in parts
whose pieces are joined (wide ones).  Tolerances are the oracle's bounds."""
import numpy as np
import pytest

from gpu_support import say, torch_cuda
from kv_support import Case, bf16, dev_rows
from oracle import kv_oracle as K

pytestmark = pytest.mark.gpu

WIDE = 8192  # tokens that a table has room for in the form of parts


def _put(c):
    """The oracle's cache to the device."""
    torch = torch_cuda()
    for n in ("k", "v", "k_scale", "v_scale"):
        getattr(c.dev, n)[c.layer].copy_(torch.from_numpy(c.cache[n]))


def _case(form, seed, new, total, heads, dim, block, **kw):
    """A case whose new rows' tokens have content."""
    c = Case(seed, new, total, heads, dim, block, width=WIDE // block if form == "parts" else None, **kw)
    K.append(c.cache, c.row(c.n_rows), c.row(c.n_rows), c.batch)
    return c


def _check(got, ref, bound, what):
    got = got.double().cpu().numpy()
    nan = np.isnan(ref)
    assert (np.isnan(got) == nan).all(), f"{what}: NaN in other places"
    err = np.where(nan, 0, np.abs(np.where(nan, 0, got) - np.where(nan, 0, ref)) - np.where(nan, 0, bound))
    at = np.unravel_index(np.argmax(err), err.shape)
    assert err[at] <= 0, f"{what}: {got[at]} != {ref[at]} +- {bound[at]} at {at}"


def _run(c, q, what, ref=None, **kw):
    """One call, checked; ref: (out, bound) where the oracle's own are not meant."""
    _put(c)
    say(f"kv attention {what}")
    got = c.M.kv_attention(c.dev, c.layer, dev_rows(q), c.dev_batch(), **kw)
    kw.pop("work", None)
    _check(got, *(ref or K.attention(c.cache, q, c.batch, **kw)), what)
    return got


def _queries(c, group):
    return bf16(c.rng.normal(size=(c.n_rows, c.heads * group, c.dim)))


def _nan_value(c, i, t, head, channel):
    c.cache["v"][int(c.table[i, t // c.block]), head, t % c.block // 16, channel, t % 16] = 0x7f


@pytest.mark.parametrize("form", ["whole", "parts"])
@pytest.mark.parametrize("dim,block", [(64, 16), (80, 16), (112, 32), (128, 64), (192, 128), (256, 16)])
def test_nan_values_in_each_block_of_the_first_step(form, dim, block):
    """Each of a step's four 16-token blocks is brought in by a wave of its
    own, before the workgroup has met a barrier: the mark that a wave leaves for
    a NaN there has to be seen by the rows of all of them."""
    new, total = [70, 3, 40], [70, 66, 200]
    c = _case(form, 90 + dim, new, total, 2, dim, block)
    for i, first in ((0, 0), (1, 0), (2, 128)):  # first token of the step
        for b in range(4):
            t = first + 16 * b + 3 * b + 1
            if t < total[i]:
                _nan_value(c, i, t, b & 1, (16 * b + 5) % dim)
                _nan_value(c, i, t, b & 1, dim - 1 - b)
    q = _queries(c, 4)
    _run(c, q, f"first step's NaN values, {form} dim={dim}")
    _run(c, q, f"first step's NaN values, window, {form} dim={dim}", window=25)
