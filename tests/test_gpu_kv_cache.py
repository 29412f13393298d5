"""kv_append and kv_read against the numpy oracle: codes, scales and values
are equal bit for bit (each rounding is defined), so no tolerance."""
import numpy as np
import pytest

from gpu_support import say, torch_cuda
from kv_support import Case, dev_rows
from oracle import kv_oracle as K

pytestmark = pytest.mark.gpu

# (new, total): one token each with an idle slot and a first token; prompts over
# page ends; chunks that start inside a page; nothing but idle slots
BATCHES = {
    "decode": ([1, 1, 0, 1, 1, 1], [1, 17, 0, 16, 300, 33]),
    "prompt": ([5, 130, 1, 16, 64], [5, 130, 1, 16, 64]),
    "chunk": ([3, 40, 18, 0, 129], [20, 47, 32, 9, 200]),
    "idle": ([0, 0], [0, 5]),
}


def _append(c, k, v, **kw):
    K.append(c.cache, k, v, c.batch)
    c.M.kv_append(c.dev, c.layer, dev_rows(k, **kw), dev_rows(v, **kw), c.dev_batch())


def _read_equal(c, batch=None):
    torch = torch_cuda()
    got = c.M.kv_read(c.dev, c.layer, c.dev_batch())
    for x, ref in zip(got, K.read(c.cache, c.batch)):
        np.testing.assert_array_equal(x.double().cpu().numpy(), ref)


@pytest.mark.parametrize("name", sorted(BATCHES))
@pytest.mark.parametrize("heads,dim,block", [(2, 64, 16), (1, 16, 32), (3, 80, 16), (2, 128, 64), (1, 256, 128), (1, 48, 256)])
def test_append_then_read(name, heads, dim, block):
    new, total = BATCHES[name]
    say(f"kv append {name} heads={heads} dim={dim} block={block}")
    c = Case(dim + len(name), new, total, heads, dim, block, layers=2)
    _append(c, c.row(c.n_rows), c.row(c.n_rows))
    assert c.pages_equal() == ""
    _read_equal(c)


@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (16, 8)])
def test_strided_and_unaligned_rows(pad, offset):
    new, total = BATCHES["chunk"]
    c = Case(7, new, total, 2, 80, 16)
    say(f"kv append pad={pad} offset={offset}")
    _append(c, c.row(c.n_rows), c.row(c.n_rows), pad=pad, offset=offset)
    assert c.pages_equal() == ""


def test_keys_and_values_of_other_strides():
    torch = torch_cuda()
    c = Case(8, [4, 1], [9, 1], 2, 64, 16)
    k, v = c.row(5), c.row(5)
    K.append(c.cache, k, v, c.batch)
    c.M.kv_append(c.dev, 0, dev_rows(k, pad=8), dev_rows(v), c.dev_batch())
    assert c.pages_equal() == ""


def test_growing_scales_round_the_older_tokens():
    """Tokens one at a time, each far larger or smaller than the last: every
    scale change of a page is met, up to both ends of the exponent's range."""
    rng = np.random.default_rng(3)
    c = Case(4, [1, 1], [1, 1], 2, 32, 16, width=2, extra=8)
    c.table[:] = [[0, 1], [2, 3]]
    from kv_support import bf16
    for step, e in enumerate([-3, 4, 4.5, -20, 30, 90, 127.9, -120, 20, 0, 1, 2, 3, 4, 5, 6, -70, -66, -60]):
        c.kv_len[:] = step + 1
        x = np.clip(rng.normal(size=(2, 2, 32)) * 2.0 ** e, -3.38e38, 3.38e38)
        say(f"kv append step {step}")
        _append(c, bf16(x), bf16(-x))
        assert c.pages_equal() == "", f"step {step}"
        _read_equal(c)


def test_zero_nan_and_infinite_tokens():
    c = Case(5, [6, 1], [6, 17], 1, 64, 16)
    k, v = c.row(7), c.row(7)
    k[1] = 0.0
    k[2, 0, 5], v[3, 0, 9], v[4, 0, 2], k[6, 0, 0] = np.nan, np.inf, -np.inf, np.nan
    v[6] = 0.0
    _append(c, k, v)
    assert c.pages_equal() == ""
    _read_equal(c)
    c2 = Case(6, [3], [3], 1, 64, 16)  # a page of zeros has the least scale
    _append(c2, np.zeros((3, 1, 64)), np.zeros((3, 1, 64)))
    assert c2.pages_equal() == "" and np.nanmin(c2.cache["k_scale"]) == 2.0 ** -64


def test_pages_that_do_not_exist_and_negative_positions():
    """Their tokens are dropped and read as NaN; the rest is as ever."""
    c = Case(9, [40, 5, 1, 20], [40, 3, 1, 50], 2, 64, 16)
    c.table[0, 1] = 10 ** 6
    c.table[2, 0] = -7
    c.table[3, 2:] = -1
    before = [x.clone() for x in (c.dev.k, c.dev.v)]
    k, v = c.row(c.n_rows), c.row(c.n_rows)
    say("kv append, bad pages")
    _append(c, k, v)
    assert c.pages_equal() == ""
    _read_equal(c)
    assert np.isnan(K.read(c.cache, c.batch)[0]).any()
    # a table narrower than the sequence
    d = Case(10, [40], [40], 1, 64, 16)
    d.table = d.table[:, :2].copy()
    say("kv append, narrow table")
    _append(d, d.row(40), d.row(40))
    assert d.pages_equal() == ""
    _read_equal(d)


def test_lengths_at_the_ends_of_their_type():
    """Nothing is written for them, and their rows are NaN."""
    torch = torch_cuda()
    c = Case(14, [2, 1, 1], [2, 1, 1], 1, 64, 16)
    before = [c.dev.k.clone(), c.dev.v.clone()]
    c.kv_len[0], c.kv_len[1], c.kv_len[2] = -2 ** 31, 2 ** 31 - 1, -1
    x = dev_rows(c.row(4))
    say("kv append and read, extreme lengths")
    c.M.kv_append(c.dev, 0, x, x, c.dev_batch())
    assert torch.equal(c.dev.k, before[0]) and torch.equal(c.dev.v, before[1])
    for y in c.M.kv_read(c.dev, 0, c.dev_batch()):
        assert torch.isnan(y).all()
    one = c.M.KVBatch(c.dev_batch().table[1:2].contiguous(), torch.tensor([-2 ** 31], dtype=torch.int32, device="cuda"),
                      torch.tensor([0, 1], dtype=torch.int32, device="cuda"), 1)
    c.M.kv_append(c.dev, 0, x[:1], x[:1], one)
    for y in c.M.kv_read(c.dev, 0, one):
        assert torch.isnan(y).all()


@pytest.mark.parametrize("block,dim", [(32, 96), (64, 128), (128, 192), (256, 256)])
def test_pages_of_many_blocks(block, dim):
    """A page written by several waves, in chunks that end anywhere in it, with
    scales that grow and values that are not finite in any of its blocks."""
    c = Case(15, [1, 1], [1, 1], 2, dim, block, width=3, extra=8)
    c.table[:] = [[0, 1, 2], [3, 4, 5]]
    rng = np.random.default_rng(6)
    c.kv_len[:] = 0
    for step, (m0, m1) in enumerate([(17, 1), (1, 40), (30, 100), (0, 15), (100, 1), (1, 16)]):
        c.kv_len += np.array([m0, m1], np.int32)
        c.row_off = np.array([0, m0, m0 + m1], np.int32)
        c.n_rows, c.max_new = m0 + m1, max(m0, m1)
        k, v = c.row(c.n_rows) * 2.0 ** (step % 3 * 3), c.row(c.n_rows) * 2.0 ** (step % 2 * 4)
        k[rng.integers(c.n_rows), 1, 3], v[rng.integers(c.n_rows), 0, 5] = np.inf, np.nan
        say(f"kv append, blocks of a page, {block} {dim} step {step}")
        _append(c, k, v)
        assert c.pages_equal() == "", f"step {step}"
        _read_equal(c)


def test_untouched_pages_keep_their_bytes():
    torch = torch_cuda()
    c = Case(11, [1, 1], [18, 40], 2, 64, 16)
    before = [getattr(c.dev, n).clone() for n in ("k", "v", "k_scale", "v_scale")]
    _append(c, c.row(2), c.row(2))
    touched = {int(c.table[0, 1]), int(c.table[1, 2])}
    for n, b in zip(("k", "v", "k_scale", "v_scale"), before):
        a = getattr(c.dev, n)
        for p in set(range(a.shape[1])) - touched:
            assert torch.equal(a[:, p].view(torch.uint8), b[:, p].view(torch.uint8)), (n, p)


def test_many_sequences_and_a_loose_bound():
    """More sequences than a workgroup looks at in one pass, and max_new left
    at its default."""
    rng = np.random.default_rng(1)
    new = [int(x) for x in rng.integers(0, 4, size=700)]
    total = [m + int(x) for m, x in zip(new, rng.integers(0, 30, size=700))]
    c = Case(12, new, total, 1, 32, 16)
    k, v = c.row(c.n_rows), c.row(c.n_rows)
    K.append(c.cache, k, v, c.batch)
    say("kv append, 700 sequences")
    c.M.kv_append(c.dev, 0, dev_rows(k), dev_rows(v), c.dev_batch(max_new=c.n_rows))
    assert c.pages_equal() == ""
    _read_equal(c)


def test_refusals():
    torch = torch_cuda()
    c = Case(13, [1, 1], [4, 4], 2, 64, 16)
    b = c.dev_batch()
    x = dev_rows(c.row(2))
    bad = lambda *a: pytest.raises((TypeError, ValueError, c.M.MloraError))
    with bad():
        c.M.kv_append(c.dev, 1, x, x, b)                      # no such layer
    with bad():
        c.M.kv_append(c.dev, 0, x.float(), x, b)              # type
    with bad():
        c.M.kv_append(c.dev, 0, x[:, :1], x[:, :1], b)        # heads
    with bad():
        c.M.kv_append(c.dev, 0, x[:1], x[:1], b)              # rows
    with bad():
        c.M.kv_append(c.dev, 0, x.transpose(1, 2), x.transpose(1, 2), b)
    with bad():
        c.M.KVBatch(b.table.long(), b.kv_len, b.row_off, 2)
    with bad():
        c.M.KVBatch(b.table[:1], b.kv_len, b.row_off, 2)
    with bad():
        c.M.KVCache(1, 4, 2, 64, 24)
    with bad():
        c.M.KVCache(1, 4, 2, 64, 16, storage=(c.dev.k, c.dev.v, c.dev.k_scale, c.dev.v_scale))
    with bad():
        c.M.kv_append(c.dev, 0, x, x, c.M.KVBatch(b.table, b.kv_len, b.row_off, 2, max_new=3))
