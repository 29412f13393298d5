"""Tokens that kv_append drops (no page, a negative position, a length at the
end of its type) leave every byte of the pool as it was, except where a token
that has a page belongs."""
import numpy as np
import pytest

from gpu_support import say, torch_cuda
from kv_support import Case, dev_rows
from oracle import kv_oracle as K

pytestmark = pytest.mark.gpu
NAMES = ("k", "v", "k_scale", "v_scale")


def _bytes(c):
    return {n: getattr(c.dev, n).view(torch_cuda().uint8).cpu().numpy().copy() for n in NAMES}


def _append(c, max_new=None):
    x, y = c.row(c.n_rows), c.row(c.n_rows)
    c.M.kv_append(c.dev, c.layer, dev_rows(x), dev_rows(y), c.dev_batch(max_new))


def _written(c):
    """Pages that hold a new token, with the end of what they hold."""
    pages = {}
    for i, _, pos in K.rows_of(c.batch):
        page = K.page_of(c.cache, c.batch, i, pos)
        if page >= 0:
            pages[page] = max(pages.get(page, 0), pos % c.block + 1)
    return pages


@pytest.mark.parametrize("dim,block", [(64, 16), (80, 32), (256, 64)])
def test_dropped_tokens_touch_no_page(dim, block):
    new, total = [2 * block + 8, 5, 1, block + 4, 3], [2 * block + 8, 3, 1, 3 * block + 2, 5]
    c = Case(30, new, total, 2, dim, block, layers=2, extra=4)
    c.table[0, 1], c.table[2, 0], c.table[3, 2:], c.table[4, 0] = 10 ** 6, -7, -1, c.cache["k"].shape[0]
    before = _bytes(c)
    say(f"kv append, dropped tokens dim={dim} block={block}")
    _append(c)
    after = _bytes(c)
    pages = _written(c)
    assert 0 < len(pages) < c.cache["k"].shape[0]
    for n in NAMES:
        a, b = after[n].reshape(2, c.cache["k"].shape[0], -1), before[n].reshape(2, c.cache["k"].shape[0], -1)
        assert np.array_equal(a[0], b[0]), f"{n} of the other layer"
        for p in range(a.shape[1]):
            if p not in pages:
                assert np.array_equal(a[1, p], b[1, p]), f"{n} of page {p}"
    # keys: no token past the last one of a page (values' pieces hold 16 tokens, and those to come may be cleared)
    for p, hi in pages.items():
        a = after["k"].reshape(2, -1, 2, block, dim)[1, p, :, hi:]
        assert np.array_equal(a, before["k"].reshape(2, -1, 2, block, dim)[1, p, :, hi:]), f"keys of page {p}"


@pytest.mark.parametrize("rows", [1, 2])
def test_lengths_that_no_sequence_has_touch_no_page(rows):
    c = Case(31, [rows] * 4, [rows] * 4, 1, 64, 16)
    for lens in ([-2 ** 31, 2 ** 31 - 1, -1, 0], [2 ** 30, 2 ** 30 + 1, -2 ** 30, 16 * c.table.shape[1] + rows]):
        c.kv_len = np.array(lens, np.int64).astype(np.int32)
        before = _bytes(c)
        say(f"kv append, lengths {lens}")
        _append(c)
        after = _bytes(c)
        for n in NAMES:
            assert np.array_equal(after[n], before[n]), n
