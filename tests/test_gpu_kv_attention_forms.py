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
    got = c.M.kv_attention(c.dev, c.layer, dev_rows(q), c.dev_batch(kw.pop("max_new", None)), **kw)
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


# long histories beside short ones; with a window of 1500 the form of parts
# keeps to its last steps
LONG = {
    "decode": ([1, 1, 0, 1, 1, 1], [4000, 17, 0, 1600, 2301, 300]),
    "drafts": ([4, 1, 3], [3000, 1, 1700]),
    "chunks": ([40, 1, 97], [2500, 1900, 97]),
}
SHAPES = [(2, 4, 64, 16), (1, 5, 80, 32), (1, 4, 128, 16), (1, 4, 256, 64)]


@pytest.mark.parametrize("name", sorted(LONG))
@pytest.mark.parametrize("heads,group,dim,block", SHAPES)
@pytest.mark.parametrize("kw", [dict(causal=False), dict(window=1500), dict(window=1281), dict(window=3500),
                                dict(scale=0.7)], ids=str)
def test_masks_in_parts(name, heads, group, dim, block, kw):
    c = _case("parts", 200 + dim, *LONG[name], heads, dim, block)
    _run(c, _queries(c, group), f"parts {name} {heads}x{group} dim={dim} {kw}", **kw)


@pytest.mark.parametrize("name", sorted(LONG))
@pytest.mark.parametrize("heads,group,dim,block", SHAPES + [(1, 4, 112, 16), (1, 4, 192, 32)])
def test_hidden_nan_in_parts(name, heads, group, dim, block):
    """NaN keys and values among the newest tokens, on both sides of the
    window's edge and far behind it: seen by the rows that see the token (a
    value's in its channel alone), by no other."""
    new, total = LONG[name]
    c = _case("parts", 210 + dim, new, total, heads, dim, block)
    for i, n in enumerate(total):
        for j, back in enumerate((1, 2, 1499, 1502, 1530, 2290)):
            t = n - back
            if t < 0 or new[i] == 0:
                continue
            page, s = int(c.table[i, t // block]), t % block
            if j % 2:
                _nan_value(c, i, t, 0, (17 * j) % dim)
                _nan_value(c, i, t, 0, dim - 1)
            elif j == 0 and i == 0 or j == 4:
                c.cache["k"][page, heads - 1, s, 3] = 0xff
    for kw in (dict(window=1500), dict(window=1281), dict(), dict(causal=False)):
        _run(c, _queries(c, group), f"parts, hidden NaN {name} dim={dim} {kw}", **kw)


@pytest.mark.parametrize("heads,group,dim,block", SHAPES)
def test_pages_that_do_not_exist_in_parts(heads, group, dim, block):
    for new in ([1, 2, 1, 1], [3, 60, 1, 40]):
        c = _case("parts", 220 + dim, new, [3500, 2000, 70, 2600], heads, dim, block)
        c.table[0, 100 // block], c.table[1, 0], c.table[3, 2000 // block] = -1, 10 ** 8, -5
        q = _queries(c, group)
        ref, _ = K.attention(c.cache, q, c.batch)
        assert np.isnan(ref[0]).all() and not np.isnan(ref[new[0] + new[1]]).any()
        _run(c, q, f"parts, bad pages {new} dim={dim}")
        _run(c, q, f"parts, bad pages, window {new} dim={dim}", window=1400)
        c.kv_len[2] = block * c.table.shape[1] + 1  # longer than its table
        _run(c, q, f"parts, past the table {new} dim={dim}")


@pytest.mark.parametrize("heads,group,dim,block", SHAPES)
def test_rows_that_see_nothing_in_parts(heads, group, dim, block):
    c = _case("parts", 230 + dim, [4, 2, 40, 1, 70, 3], [2, 2, 20, 2000, 70, 1800], heads, dim, block)
    c.kv_len[1] = 0
    q = _queries(c, group)
    got = _run(c, q, f"parts, negative positions dim={dim}").double().cpu().numpy()
    assert (got[:2] == 0).all() and (got[4:26] == 0).all() and (got[2:4] != 0).any()
    _run(c, q, f"parts, negative positions, window dim={dim}", window=1400)
    _run(c, q, f"parts, no tokens, no mask dim={dim}", causal=False)


@pytest.mark.parametrize("heads,group,dim,block", SHAPES)
@pytest.mark.parametrize("new,total", [([1, 1], [3000, 40]), ([40, 3], [2000, 900])])
def test_queries_that_are_not_finite_in_parts(heads, group, dim, block, new, total):
    c = _case("parts", 240 + dim, new, total, heads, dim, block)
    c.cache["k"] = np.where((c.cache["k"] & 0x7f) == 0x7f, c.cache["k"], c.cache["k"] & 0x7f).astype(np.uint8)
    c.cache["k"][c.cache["k"] == 0] = 1  # no zero among the keys (0 times infinity)
    q = _queries(c, group)
    ref, bound = K.attention(c.cache, q, c.batch)
    q[0, 1, 3] = np.nan
    q[-1, 0, 5], q[0, 0] = np.inf, -np.inf  # a score of +infinity, every score -infinity
    ref[0, 1] = ref[-1, 0] = ref[0, 0] = np.nan
    _run(c, q, f"parts, queries not finite {new} dim={dim}", ref=(ref, bound))


def _weighted(c, q):
    """The oracle's result, with the bound 2^-7 + 2^-12 of sum p |v|: both
    roundings to bf16 and sums of up to 4000 terms in fp32."""
    ref, _ = K.attention(c.cache, q, c.batch)
    signed = c.cache["v"]
    c.cache["v"] = np.where((signed & 0x7f) == 0x7f, signed, signed & 0x7f).astype(np.uint8)
    size, _ = K.attention(c.cache, q, c.batch)
    c.cache["v"] = signed
    return ref, size * (2.0 ** -7 + 2.0 ** -12)


@pytest.mark.filterwarnings("ignore::RuntimeWarning")
@pytest.mark.parametrize("form", ["whole", "parts"])
@pytest.mark.parametrize("heads,group,dim,block", SHAPES)
@pytest.mark.parametrize("new", [[1, 2, 1], [40, 30, 1]])
def test_pieces_whose_scores_are_all_minus_infinity(form, new, heads, group, dim, block):
    """Scores of the first, the second or the middle part of the tokens pass
    fp32's range downwards (-2^140), the others are 2^-2 at most: no weight on
    the former, the same weight on the latter, however the work is cut."""
    total = [3000, 2000, 1500] if form == "parts" else [900, 700, 300]
    c = _case(form, 250 + dim, new, total, heads, dim, block)
    c.cache["k"][:] = 0x38  # 1
    c.cache["k_scale"][:] = 2.0 ** -102
    for i, (lo, hi) in enumerate(((0, 0.5), (0.6, 0.9), (0.3, 0.7))):
        for p in c.table[i, int(lo * total[i]) // block:int(hi * total[i]) // block]:
            c.cache["k_scale"][p] = 2.0 ** 40
    q = np.zeros((c.n_rows, heads * group, dim))
    q[:, :, 3] = -2.0 ** 100
    _run(c, q, f"{form}, pieces of minus infinity {new} dim={dim}", ref=_weighted(c, q), scale=None)


@pytest.mark.parametrize("heads,group,dim,block", SHAPES)
@pytest.mark.parametrize("new,total", [([1, 1], [4000, 64]), ([70, 2], [1500, 2000])])
def test_values_of_scales_far_apart_in_parts(heads, group, dim, block, new, total):
    """Every token has the same weight (the queries are zero), and the pages'
    scales lie up to 2^30 apart."""
    c = _case("parts", 260 + dim, new, total, heads, dim, block)
    for p in range(c.cache["v_scale"].shape[0]):
        c.cache["v_scale"][p] *= 2.0 ** ((p * 7) % 31 - 15)
    q = np.zeros((c.n_rows, heads * group, dim))
    _run(c, q, f"parts, scales far apart {new} dim={dim}", ref=_weighted(c, q))


@pytest.mark.parametrize("dim,block", [(64, 16), (128, 64)])
def test_more_sequences_than_are_dealt_with_side_by_side(dim, block):
    """300 and 600 sequences of both kinds, two key/value heads, some with long
    histories, others idle, in the form of parts."""
    rng = np.random.default_rng(9)
    for n in (300, 600):
        seqs = [(1, int(x)) if x % 7 else (0, 0) for x in rng.integers(1, 120, size=n)]
        for at, s in ((0, (40, 40)), (n // 2, (33, 700)), (n - 1, (70, 1400)), (n // 3, (1, 2500)), (n // 4, (5, 900))):
            seqs[at] = s
        c = _case("parts", 270, [m for m, _ in seqs], [t for _, t in seqs], 2, dim, block)
        q = _queries(c, 4)
        _run(c, q, f"parts, {n} sequences dim={dim}")
        _run(c, q, f"parts, {n} sequences, a loose bound dim={dim}", max_new=c.n_rows)
        if n == 300:
            _run(c, q, f"parts, {n} sequences, window dim={dim}", window=1300)
            _run(c, q, f"parts, {n} sequences, no mask dim={dim}", causal=False)


def _graph(f):
    torch = torch_cuda()
    f()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f()
    return g


@pytest.mark.parametrize("window", [0, 1500])
@pytest.mark.parametrize("name", sorted(LONG))
def test_replays_of_parts_over_lengths_that_move_the_cuts(name, window):
    """One captured call and one work buffer, its contents those of the replay
    before or overwritten between; the eager call with a buffer of its own gives
    the same bits."""
    torch = torch_cuda()
    new, total = LONG[name]
    c = _case("parts", 280, new, total, 2, 128, 16)
    _put(c)
    b = c.dev_batch()
    q = dev_rows(_queries(c, 4))
    out = torch.empty((c.n_rows, 8, 128), dtype=torch.bfloat16, device="cuda")
    work = c.M.new_kv_work(c.dev, b, 8)
    say(f"kv graph of parts, capture {name} window={window}")
    g = _graph(lambda: c.M.kv_attention(c.dev, 0, q, b, window=window, work=work, out=out))
    rng = np.random.default_rng(4)
    full = np.array(total)
    for r in range(6):
        short = rng.integers(np.array(new), np.maximum(full, np.array(new)) + 1)
        c.kv_len = (full if r == 3 else np.minimum(short, 40 + full // 9) if r == 4 else short).astype(np.int32)
        qn = _queries(c, 4)
        q.copy_(torch.from_numpy(qn.astype(np.float32)))
        b.kv_len.copy_(torch.from_numpy(c.kv_len))
        if r % 2:
            work.fill_(0xff)
        out.zero_()
        torch.cuda.synchronize()
        say(f"kv graph of parts, replay {r} {name} window={window}")
        g.replay()
        torch.cuda.synchronize()
        _check(out, *K.attention(c.cache, qn, c.batch, window=window), f"replay {r}")
        again = c.M.kv_attention(c.dev, 0, q, b, window=window)
        assert torch.equal(again.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("name", sorted(LONG))
def test_replays_of_parts_as_tokens_are_added(name):
    """Write and attention of a layer with a window, captured: a token more of
    each sequence in every replay, over page ends."""
    torch = torch_cuda()
    new, total = LONG[name]
    total = [n - n % 16 + 13 if n else 0 for n in total]
    c = Case(290, new, total, 2, 128, 16, width=WIDE // 16, extra=60)
    free = [p for p in range(c.cache["k"].shape[0]) if p not in set(c.table.ravel().tolist())]
    for i, n in enumerate(total):
        if n:
            c.table[i, -(-n // 16):-(-n // 16) + 2] = free.pop(), free.pop()
    _put(c)
    b = c.dev_batch()
    k, v, q = dev_rows(c.row(c.n_rows)), dev_rows(c.row(c.n_rows)), dev_rows(_queries(c, 4))
    out = torch.empty((c.n_rows, 8, 128), dtype=torch.bfloat16, device="cuda")
    work = c.M.new_kv_work(c.dev, b, 8)
    # what the eager call before the capture writes is put back after it
    say(f"kv graph of a windowed layer, capture {name}")
    g = _graph(lambda: (c.M.kv_append(c.dev, 0, k, v, b),
                        c.M.kv_attention(c.dev, 0, q, b, window=1500, work=work, out=out)))
    _put(c)
    for r in range(5):
        kn, vn, qn = c.row(c.n_rows), c.row(c.n_rows), _queries(c, 4)
        for dst, src in ((k, kn), (v, vn), (q, qn)):
            dst.copy_(torch.from_numpy(src.astype(np.float32)))
        torch.cuda.synchronize()
        say(f"kv graph of a windowed layer, replay {r} {name}")
        g.replay()
        torch.cuda.synchronize()
        K.append(c.cache, kn, vn, c.batch)
        assert c.pages_equal() == "", f"replay {r}"
        _check(out, *K.attention(c.cache, qn, c.batch, window=1500), f"replay {r}")
        c.kv_len += (np.diff(c.row_off) > 0).astype(np.int32)
        b.kv_len.copy_(torch.from_numpy(c.kv_len))
