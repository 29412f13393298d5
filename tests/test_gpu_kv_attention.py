"""kv_attention against the numpy oracle.  The tolerance of each output is the
oracle's bound: what rounding the probabilities and the result to bf16 (2^-8
relative each) and computing scores, exponentials and sums in fp32 allow."""
import numpy as np
import pytest

from gpu_support import say, torch_cuda
from kv_support import Case, bf16, dev_rows
from oracle import kv_oracle as K

pytestmark = pytest.mark.gpu


def _check(got, ref, bound, what):
    got = got.double().cpu().numpy()
    nan = np.isnan(ref)
    assert (np.isnan(got) == nan).all(), f"{what}: NaN in other places"
    err = np.where(nan, 0, np.abs(got - ref) - bound)
    at = np.unravel_index(np.argmax(err), err.shape)
    assert err[at] <= 0, f"{what}: {got[at]} != {ref[at]} +- {bound[at]} at {at}"


def _queries(c, group, n=None):
    return bf16(c.rng.normal(size=(c.n_rows if n is None else n, c.heads * group, c.dim)))


def _run(c, q, what, **kw):
    say(f"kv attention {what}")
    dev = {k: kw.pop(k) for k in ("max_new", "pad", "offset") if k in kw}
    b = c.dev_batch(dev.pop("max_new", None))
    got = c.M.kv_attention(c.dev, c.layer, dev_rows(q, **dev), b, **kw)
    kw.pop("work", None)
    ref, bound = K.attention(c.cache, q, c.batch, **kw)
    _check(got, ref, bound, what)
    return got


BATCHES = {
    "one": ([1], [1]),
    "decode": ([1, 1, 0, 1, 1, 1, 1], [1, 17, 0, 16, 300, 64, 129]),
    "drafts": ([3, 1, 5, 0, 2], [3, 70, 260, 11, 16]),
    "prompts": ([5, 130, 1, 63], [5, 130, 1, 63]),
    "chunks": ([33, 100, 1], [200, 165, 400]),
}
SHAPES = [(2, 4, 128, 16), (1, 1, 64, 32), (2, 7, 64, 16), (1, 16, 128, 64), (2, 5, 80, 16), (1, 2, 96, 32),
          (1, 8, 192, 128), (1, 4, 256, 16), (1, 3, 32, 16), (1, 2, 112, 256), (1, 4, 160, 16)]


@pytest.mark.parametrize("name", sorted(BATCHES))
@pytest.mark.parametrize("heads,group,dim,block", SHAPES)
def test_causal(name, heads, group, dim, block):
    new, total = BATCHES[name]
    c = Case(dim + len(name), new, total, heads, dim, block, layers=2)
    _run(c, _queries(c, group), f"{name} heads={heads}x{group} dim={dim} block={block}")


@pytest.mark.parametrize("name", sorted(BATCHES))
@pytest.mark.parametrize("heads,group,dim,block", SHAPES)
def test_wide_tables(name, heads, group, dim, block):
    """Tables with room for long sequences: the work is dealt in parts, and
    cut sequences are joined."""
    new, total = BATCHES[name]
    total = [n + 700 * (i % 3 == 1 and m > 0) for i, (m, n) in enumerate(zip(new, total))]
    c = Case(dim + len(name), new, total, heads, dim, block, width=8192 // block)
    _run(c, _queries(c, group), f"wide {name} heads={heads}x{group} dim={dim} block={block}")


def test_many_ragged_sequences():
    rng = np.random.default_rng(2)
    for lo, hi in ((0, 2), (0, 40)):
        new = [int(x) for x in rng.integers(lo, hi, size=600 if hi == 2 else 40)]
        total = [m + int(x) * (m > 0) for m, x in zip(new, rng.integers(0, 300, size=len(new)))]
        c = Case(79, new, total, 1, 64, 16, width=512)
        _fill_new_plain(c)
        _run(c, _queries(c, 3), f"ragged {hi}")
        _run(c, _queries(c, 3), f"ragged {hi}, window", window=33, max_new=c.n_rows)


@pytest.mark.parametrize("name", sorted(BATCHES))
@pytest.mark.parametrize("kw", [dict(causal=False), dict(window=1), dict(window=7), dict(window=64), dict(window=100),
                                dict(window=5000), dict(scale=0.7)], ids=str)
def test_masks(name, kw):
    new, total = BATCHES[name]
    c = Case(40 + len(name), new, total, 2, 64, 16)
    _run(c, _queries(c, 4), f"{name} {kw}", **kw)


def test_the_largest_window():
    new, total = BATCHES["chunks"]
    c = Case(41, new, total, 2, 64, 16, width=512)
    q = _queries(c, 4)
    _fill_new_plain(c)
    a = _run(c, q, "no window")
    b = _run(c, q, "window 2^31 - 1", window=2 ** 31 - 1)
    torch = torch_cuda()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1)])
def test_strided_and_unaligned_queries(pad, offset):
    new, total = BATCHES["chunks"]
    c = Case(50, new, total, 2, 128, 16)
    _run(c, _queries(c, 2), f"pad={pad} offset={offset}", pad=pad, offset=offset)


@pytest.mark.parametrize("name", ["decode", "drafts", "chunks"])
def test_what_is_hidden_does_not_reach_a_row(name):
    """NaN keys and values behind the window, and in tokens newer than a row;
    a row that sees one is NaN, in that channel for a value, else it is as if
    the token were not there."""
    new, total = BATCHES[name]
    for window in (0, 20):
        c = Case(60, new, total, 2, 64, 16)
        for i, n in enumerate(total):
            for back in (1, 2, 40, 77):  # tokens from the end
                t = n - back
                if t < 0:
                    continue
                page, s = int(c.table[i, t // 16]), t % 16
                if back in (2, 77):
                    c.cache["v"][page, 0, 0, 5, s] = 0x7f
                else:
                    c.cache["k"][page, 1, s, 3] = 0xff
        torch = torch_cuda()
        c.dev.k[0].copy_(torch.from_numpy(c.cache["k"]))
        c.dev.v[0].copy_(torch.from_numpy(c.cache["v"]))
        # the new rows' content comes from the cache as it is: fill what has no content yet
        _fill_new(c)
        q = _queries(c, 2)
        b = c.dev_batch()
        say(f"kv attention hidden NaN {name} window={window}")
        got = c.M.kv_attention(c.dev, 0, dev_rows(q), b, window=window)
        ref, bound = K.attention(c.cache, q, c.batch, window=window)
        _check(got, ref, np.where(np.isnan(bound), 0, bound), f"{name} window={window}")


def _fill_new(c):
    """Gives the new rows' tokens content (some tests do not append)."""
    torch = torch_cuda()
    keep = {n: c.cache[n].copy() for n in ("k", "v")}
    x, y = c.row(c.n_rows), c.row(c.n_rows)
    K.append(c.cache, x, y, c.batch)
    for name in ("k", "v"):  # NaN marks stay
        marked = (keep[name] & 0x7f) == 0x7f
        held = np.zeros_like(marked)
        for i, n in enumerate(c.kv_len):
            for back in (1, 2, 40, 77):
                t = int(n) - back
                if t >= 0:
                    page, s = int(c.table[i, t // c.block]), t % c.block
                    if name == "k" and back in (1, 40):
                        held[page, 1, s, 3] = True
                    if name == "v" and back in (2, 77):
                        held[page, 0, s // 16, 5, s % 16] = True
        c.cache[name][marked & held] = 0x7f
    for n in ("k", "v", "k_scale", "v_scale"):
        getattr(c.dev, n)[c.layer].copy_(torch.from_numpy(c.cache[n]))


def test_rows_that_see_nothing_are_zero():
    """Rows at negative positions (more new rows than tokens) and sequences
    without tokens."""
    c = Case(70, [4, 2, 3], [2, 2, 3], 2, 64, 16)
    _fill_new_plain(c)
    q = _queries(c, 4)
    c.kv_len[1] = 0
    got = _run(c, q, "negative positions")
    got = got.double().cpu().numpy()
    assert (got[:2] == 0).all() and (got[4:6] == 0).all() and (got[2:4] != 0).any()
    _run(c, q, "no tokens, no mask", causal=False)


def _fill_new_plain(c):
    torch = torch_cuda()
    K.append(c.cache, c.row(c.n_rows), c.row(c.n_rows), c.batch)
    for n in ("k", "v", "k_scale", "v_scale"):
        getattr(c.dev, n)[c.layer].copy_(torch.from_numpy(c.cache[n]))


def test_pages_that_do_not_exist():
    """NaN in the rows that see them; with a window past them (their pages may
    have been given back), nothing."""
    for new in ([1, 1, 1], [3, 40, 1]):
        c = Case(71, new, [150, 150, 30], 1, 64, 16)
        _fill_new_plain(c)
        q = _queries(c, 4)
        c.table[0, 2], c.table[1, 0], c.table[1, 1] = -1, 10 ** 8, -5
        ref, bound = K.attention(c.cache, q, c.batch)
        say(f"kv attention bad pages {new}")
        got = c.M.kv_attention(c.dev, 0, dev_rows(q), c.dev_batch())
        _check(got, ref, np.where(np.isnan(bound), 0, bound), "bad pages")
        assert np.isnan(ref[0]).all() and not np.isnan(ref[-1]).any()
        ref, bound = K.attention(c.cache, q, c.batch, window=50)
        say(f"kv attention bad pages, window {new}")
        got = c.M.kv_attention(c.dev, 0, dev_rows(q), c.dev_batch(), window=50)
        _check(got, ref, bound, "bad pages behind the window")
        assert not np.isnan(ref).any()
        # a sequence longer than its table
        c.kv_len[2] = 16 * c.table.shape[1] + 1
        say(f"kv attention past the table {new}")
        got = c.M.kv_attention(c.dev, 0, dev_rows(q), c.dev_batch()).float().cpu().numpy()
        assert np.isnan(got[-1]).all()


def test_queries_that_are_not_finite():
    c = Case(72, [1, 5], [100, 90], 1, 64, 16)
    _fill_new_plain(c)
    q = _queries(c, 4)
    q[0, 1, 3], q[4, 2, 7] = np.nan, np.inf
    ref, bound = K.attention(c.cache, np.where(np.isfinite(q), q, 0), c.batch)
    say("kv attention NaN queries")
    got = c.M.kv_attention(c.dev, 0, dev_rows(q), c.dev_batch())
    ref[0, 1], ref[4, 2] = np.nan, np.nan
    _check(got, ref, bound, "NaN queries")


@pytest.mark.parametrize("new,total", [([1, 1], [1, 700]), ([40], [40])])
def test_rows_whose_every_score_is_minus_infinity(new, total):
    """They see tokens, so they are NaN (0 / 0), not the zero of a row that
    sees none; rows of other queries are as ever."""
    c = Case(80, new, total, 1, 64, 16)
    x = np.abs(c.row(c.n_rows))
    K.append(c.cache, x, x, c.batch)
    lut = K.code_values()
    c.cache["k"] = np.where(np.isnan(lut[c.cache["k"]]), c.cache["k"], c.cache["k"] & 0x7f).astype(np.uint8)
    torch = torch_cuda()
    c.cache["k"][c.cache["k"] == 0] = 1  # no zero among the keys (0 times infinity)
    for n in ("k", "v", "k_scale", "v_scale"):
        getattr(c.dev, n)[c.layer].copy_(torch.from_numpy(c.cache[n]))
    q = _queries(c, 4)
    ref, bound = K.attention(c.cache, q, c.batch)
    q[0, 1], q[-1, 3] = -np.inf, -np.inf
    ref[0, 1], ref[-1, 3] = np.nan, np.nan
    say(f"kv attention scores of minus infinity {new}")
    got = c.M.kv_attention(c.dev, 0, dev_rows(q), c.dev_batch())
    _check(got, ref, bound, "minus infinity")


@pytest.mark.parametrize("order", ["prompts first", "prompts last", "between"])
def test_few_and_many_rows_in_one_batch(order):
    """Sequences of both kinds, among them idle ones, in more sequences than a
    workgroup deals with side by side as well."""
    rng = np.random.default_rng(5)
    for n_single in (20, 300):
        prompts = [(33, 200), (70, 70), (5, 900)]
        singles = [(1, int(x)) if x % 7 else (0, 0) for x in rng.integers(1, 120, size=n_single)]
        half = n_single // 2
        seqs = {"prompts first": prompts + singles, "prompts last": singles + prompts,
                "between": prompts[:1] + singles[:half] + prompts[1:2] + singles[half:] + prompts[2:]}[order]
        c = Case(81, [m for m, _ in seqs], [n for _, n in seqs], 1, 64, 16)
        _fill_new_plain(c)
        _run(c, _queries(c, 4), f"{order}, {n_single} singles")


def test_large_scores():
    """Scores in the thousands, rising and falling along the sequence, and
    pages whose scales lie 2^30 apart."""
    for new, total in (([1, 1], [700, 64]), ([70], [300])):
        c = Case(73, new, total, 1, 64, 16)
        _fill_new_plain(c)
        for p in range(c.cache["v_scale"].shape[0]):
            c.cache["v_scale"][p] *= 2.0 ** ((p * 7) % 31 - 15)
        torch = torch_cuda()
        c.dev.v_scale[0].copy_(torch.from_numpy(c.cache["v_scale"]))
        q = bf16(_queries(c, 4) * 200)
        _run(c, q, "large scores")


def test_long_sequence_splits():
    """One long and many short sequences: pieces of a sequence are joined."""
    c = Case(74, [1, 1, 1, 2], [6000, 10, 1, 2500], 1, 128, 64)
    _fill_new_plain(c)
    q = _queries(c, 4)
    a = _run(c, q, "long")
    b = _run(c, q, "long, work given", work=c.M.new_kv_work(c.dev, c.dev_batch(), 4))
    torch = torch_cuda()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_offsets_past_32_bits():
    """Pages more than 4 GiB from the start of the pool."""
    torch = torch_cuda()
    import lora_serving_mlora_amd as M
    c = Case(75, [1, 20], [100, 50], 2, 128, 16)
    _fill_new_plain(c)
    nb = (5 << 30) // (2 * 16 * 128)
    dev = M.KVCache(1, nb, 2, 128, 16, storage=(
        torch.empty((1, nb, 2, 16, 128), dtype=torch.uint8, device="cuda"),
        torch.empty((1, nb, 2, 1, 128, 16), dtype=torch.uint8, device="cuda"),
        torch.empty((1, nb, 2), dtype=torch.float32, device="cuda"),
        torch.empty((1, nb, 2), dtype=torch.float32, device="cuda")))
    used = c.cache["k"].shape[0]
    far = nb - used
    for n in ("k", "v", "k_scale", "v_scale"):
        getattr(dev, n)[0, far:] = torch.from_numpy(c.cache[n]).cuda()
    q = _queries(c, 2)
    ref, bound = K.attention(c.cache, q, c.batch)
    x, y = K.read(c.cache, c.batch)
    c.table = np.where(c.table >= 0, c.table + far, -1).astype(np.int32)
    say("kv attention past 4 GiB")
    _check(M.kv_attention(dev, 0, dev_rows(q), c.dev_batch()), ref, bound, "past 4 GiB")
    gk, gv = M.kv_read(dev, 0, c.dev_batch())
    assert np.array_equal(gk.double().cpu().numpy(), x) and np.array_equal(gv.double().cpu().numpy(), y)
    M.kv_append(dev, 0, dev_rows(x), dev_rows(y), c.dev_batch())
    gk2, _ = M.kv_read(dev, 0, c.dev_batch())
    assert np.array_equal(gk2.double().cpu().numpy(), x)  # values a page's scale holds already


@pytest.mark.parametrize("name", ["decode", "chunks"])
def test_graph_replays_and_streams(name):
    """Captured once, replayed over lengths and rows that change in place; the
    eager call on a stream of its own gives the same bits."""
    torch = torch_cuda()
    new, total = BATCHES[name]
    c = Case(76, new, total, 2, 128, 16, width=40, extra=60)
    free = [p for p in range(c.cache["k"].shape[0]) if p not in set(c.table.ravel().tolist())]
    for i in range(len(new)):  # room for the tokens to come
        if new[i]:
            for p in range(40):
                if c.table[i, p] < 0 and p < total[i] // 16 + 3:
                    c.table[i, p] = free.pop()
    b = c.dev_batch()
    k, v, q = (dev_rows(c.row(c.n_rows)), dev_rows(c.row(c.n_rows)), dev_rows(_queries(c, 4)))
    out = torch.empty((c.n_rows, 8, 128), dtype=torch.bfloat16, device="cuda")
    work = c.M.new_kv_work(c.dev, b, 8)
    step = lambda: (c.M.kv_append(c.dev, 0, k, v, b), c.M.kv_attention(c.dev, 0, q, b, work=work, out=out))
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    say(f"kv graph capture {name}")
    with torch.cuda.graph(g):
        step()
    side = torch.cuda.Stream()
    for r in range(3):
        kn, vn, qn = c.row(c.n_rows), c.row(c.n_rows), _queries(c, 4)
        for dst, src in ((k, kn), (v, vn), (q, qn)):
            dst.copy_(torch.from_numpy(src.astype(np.float32)))
        torch.cuda.synchronize()
        say(f"kv graph replay {r} {name}")
        g.replay()
        torch.cuda.synchronize()
        first = out.clone()
        K.append(c.cache, kn, vn, c.batch)
        ref, bound = K.attention(c.cache, qn, c.batch)
        _check(first, ref, bound, f"replay {r}")
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            again = c.M.kv_attention(c.dev, 0, q, b)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert torch.equal(again.view(torch.int16), first.view(torch.int16))
        c.kv_len += (np.diff(c.row_off) > 0).astype(np.int32)
        b.kv_len.copy_(torch.from_numpy(c.kv_len))


def test_refusals():
    torch = torch_cuda()
    c = Case(77, [1, 1], [4, 4], 2, 64, 16)
    b, q = c.dev_batch(), dev_rows(_queries(c, 2))
    A = c.M.kv_attention
    for make in (lambda: A(c.dev, 1, q, b), lambda: A(c.dev, 0, q.float(), b), lambda: A(c.dev, 0, q[:, :3], b),
                 lambda: A(c.dev, 0, q[:1], b), lambda: A(c.dev, 0, q[:, :, :32], b),
                 lambda: A(c.dev, 0, q, b, window=-1), lambda: A(c.dev, 0, q, b, causal=False, window=4),
                 lambda: A(c.dev, 0, q, b, scale=0.0), lambda: A(c.dev, 0, q, b, scale=float("nan")),
                 lambda: A(c.dev, 0, q, b, out=torch.empty((2, 4, 32), dtype=torch.bfloat16, device="cuda")),
                 lambda: A(c.dev, 0, q, b, work=torch.empty(256, dtype=torch.uint8, device="cuda")[1:])):
        with pytest.raises((TypeError, ValueError, c.M.MloraError)):
            make()
    odd = Case(78, [1], [4], 1, 48, 16)  # a size that the cache takes and attention does not
    with pytest.raises(c.M.MloraError):
        A(odd.dev, 0, dev_rows(_queries(odd, 1)), odd.dev_batch())
    empty = c.M.KVBatch(b.table, b.kv_len, torch.zeros(3, dtype=torch.int32, device="cuda"), 0)
    assert A(c.dev, 0, q[:0], empty).shape == (0, 4, 64)
