"""The sampler on the GPU: the same tokens as the 64-bit oracle.  The kernel
holds weights to 2^-42 of the largest, so a token can differ only where u lies
that close to a border; the random numbers here are multiples of 2^-24 from a
fixed seed."""
import numpy as np
import pytest

from gpu_support import say, torch_cuda
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def M():
    torch_cuda()
    import lora_serving_mlora_amd as M
    return M


def run(M, logits, u, f32, pad=0, **kw):
    """Tokens of the kernel and of the oracle for float64 logits [n][V]."""
    torch = torch_cuda()
    n, V = logits.shape
    dt = torch.float32 if f32 else torch.bfloat16
    buf = torch.full((n, V + pad), INF, dtype=dt, device="cuda")
    x = buf[:, pad:]
    x.copy_(torch.from_numpy(logits.astype(np.float32)).to(dt))
    held = x.double().cpu().numpy()
    dev = {k: None if v is None else torch.tensor(np.asarray(v), dtype=torch.int32 if k == "top_k" else torch.float32,
                                                  device="cuda") for k, v in kw.items()}
    ud = torch.tensor(np.asarray(u), dtype=torch.float32, device="cuda")
    got = M.sample(x, ud, **dev).cpu().numpy()
    ref = S.sample(held, ud.cpu().numpy(), **{k: None if v is None else v.cpu().numpy() for k, v in dev.items()})
    return got, ref


def random_logits(rng, n, V, spread=2.2):
    x = spread * rng.normal(size=(n, V))
    for i in range(n):
        x[i, rng.integers(0, V, 20)] += rng.exponential(4, 20)
    return x


VOCABS = [1, 2, 3, 63, 64, 1000, 1025, 4097, 50001]


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("V", VOCABS)
def test_filters(M, V, f32):
    """Every mix of filters, each row with its own."""
    say(f"sample {V} f32={f32}")
    rng = np.random.default_rng(V)
    n = 24
    x = random_logits(rng, n, V)
    u = rng.random(n, dtype=np.float32)
    kw = dict(temperature=rng.choice([0.0, 0.3, 0.7, 1.0, 1.7, 5.0], n), top_k=rng.choice([0, 1, 2, 5, 40, 300, 10 ** 6], n),
              top_p=rng.choice([0.0, 0.1, 0.5, 0.9, 0.99, 1.0, 1.5], n), min_p=rng.choice([0.0, 0.01, 0.1, 0.5, 1.0, 2.0], n))
    for names in (("temperature",), ("top_k",), ("top_p",), ("min_p",), ("temperature", "top_k", "top_p"),
                  ("temperature", "top_k", "top_p", "min_p"), ()):
        got, ref = run(M, x, u, f32, pad=V % 3, **{k: kw[k] for k in names})
        assert np.array_equal(got, ref), f"{names}: rows {np.flatnonzero(got != ref)}"


@pytest.mark.parametrize("f32,V", [(False, 131072), (True, 131072), (False, 1 << 20), (True, 200001)])
def test_large_vocabularies(M, f32, V):
    say(f"sample {V} f32={f32}")
    rng = np.random.default_rng(V + f32)
    n = 4
    x = random_logits(rng, n, V)
    u = rng.random(n, dtype=np.float32)
    for kw in (dict(), dict(top_p=[0.9, 0.5, 0.999, 1.0]), dict(top_k=[50, 5000, 0, V - 1], top_p=[1.0, 0.9, 0.8, 0.99999])):
        got, ref = run(M, x, u, f32, **kw)
        assert np.array_equal(got, ref), str(kw)


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("V", [300, 5000, 70001])
def test_ties(M, V, f32):
    """All logits alike, a few values only, and a tie at every border."""
    say(f"ties {V} f32={f32}")
    rng = np.random.default_rng(V)
    alike = np.full((6, V), 1.5)
    few = rng.choice([2.0, 1.0, 0.0], (6, V), p=[0.001, 0.3, 0.699])
    signs = np.where(rng.random((6, V)) < 0.5, 0.0, -0.0)
    u = np.array([0.0, 0.25, 0.5, 0.75, 0.9999, 0.3], np.float32)
    for x in (alike, few, signs, 100 + few):
        for kw in (dict(), dict(top_k=[1, 2, 100, V // 2, V, 0]), dict(top_p=[0.5, 0.25, 0.125, 0.75, 0.5, 0.0625]),
                   dict(top_k=[5, 50, 64, 128, 256, 200], top_p=[0.5] * 6),
                   dict(min_p=[0.2, 0.4, 1.0, 0.1, 0.5, 0.0], temperature=[1, 2, 0.5, 1, 1, 0])):
            got, ref = run(M, x, u, f32, **kw)
            assert np.array_equal(got, ref), f"{kw} {got} {ref}"


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
def test_many_tokens_close_together(M, f32):
    """More tokens than a range's list holds, and apart from them a few."""
    say(f"close together f32={f32}")
    rng = np.random.default_rng(4)
    V, n = 60000, 6
    x = rng.normal(size=(n, V)) * 1e-3
    x[:, 7] = -25
    x[3:, 11] = 3
    u = rng.random(n, dtype=np.float32)
    for kw in (dict(), dict(top_p=[0.3, 0.6, 0.9] * 2), dict(top_k=[10, 30000, 59999] * 2, top_p=[0.9] * 6),
               dict(temperature=[INF, 1e30, 100.0, 1e-3, 1e-6, 1e-40])):
        got, ref = run(M, x, u, f32, **kw)
        assert np.array_equal(got, ref), str(kw)


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("V", [5, 3000])
def test_infinities_and_nan(M, V, f32):
    say(f"infinities {V} f32={f32}")
    rng = np.random.default_rng(V)
    x = rng.normal(size=(10, V))
    x[0] = -INF
    x[1] = NAN
    x[2, 1:] = -INF
    x[3, :2] = INF
    x[4, 3] = NAN
    x[5] = INF
    x[6, ::2] = -INF
    x[7, 1] = 3e38
    x[8, 1], x[8, 2] = -3e38, NAN
    x[9] = NAN
    x[9, 4] = -5
    lowest = -3.3895313892515355e38  # a mask of the type's lowest value
    x[6, 1] = lowest
    u = rng.random(10, dtype=np.float32)
    for kw in (dict(), dict(temperature=[0.0] * 10), dict(temperature=[INF] * 10), dict(temperature=[NAN, -1.0] * 5),
               dict(temperature=[1e-40] * 10), dict(top_k=[2] * 10, top_p=[0.9] * 10, min_p=[0.1] * 10),
               dict(top_p=[NAN] * 10, min_p=[NAN] * 10), dict(top_p=[-1.0] * 10), dict(top_k=[-3] * 10)):
        got, ref = run(M, x, u, f32, **kw)
        assert np.array_equal(got, ref), f"{kw} {got} {ref}"


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("V", [129, 700, 1024, 1025, 2352, 5000])
def test_long_lists(M, V, f32):
    """Hundreds of tokens in the list: spread out, close together beside a few
    far above, many of a value; top-k whose list overruns."""
    say(f"long lists {V} f32={f32}")
    rng = np.random.default_rng(V + 3)
    n = 16
    x = rng.normal(size=(n, V)) * np.repeat([0.5, 2.0, 1e-3, 8.0], 4)[:, None]
    x[::4, 3] += 12.0
    x[1::4, V // 2:V // 2 + 5] += 30.0
    x[2::4] = np.round(x[2::4] * 4) / 4
    u = rng.random(n, dtype=np.float32)
    t = rng.choice([0.4, 0.7, 1.0, 1.4], n)
    for kw in (dict(temperature=t), dict(temperature=t, top_k=rng.integers(200, 513, n)),
               dict(temperature=t, top_k=rng.integers(300, 900, n), top_p=[0.95] * n),
               dict(temperature=t, top_p=rng.random(n), min_p=[0.0, 0.01] * 8),
               dict(temperature=t, top_k=[V - 1, V, V + 1, 512] * 4, min_p=[1e-6] * n), dict(temperature=[1e-3] * n)):
        got, ref = run(M, x, u, f32, **kw)
        assert np.array_equal(got, ref), f"{kw}: rows {np.flatnonzero(got != ref)}"


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("V", [16384, 16391, 70000])
def test_masks_in_large_vocabularies(M, V, f32):
    """Infinities, NaN, both zeros and masks of the lowest value in rows whose
    values are counted; unaligned rows; every mix of filters."""
    say(f"masks {V} f32={f32}")
    rng = np.random.default_rng(V + 7)
    n = 12
    x = rng.normal(size=(n, V)) * 2
    lowest = -3.3895313892515355e38
    x[0] = -INF
    x[1] = NAN
    x[2, 5:] = -INF
    x[3, :9] = INF
    x[4, rng.random(V) < 0.999] = lowest
    x[5] = lowest
    x[6, rng.random(V) < 0.9] = -INF
    x[7] = np.where(rng.random(V) < 0.5, 0.0, -0.0)
    x[8, rng.random(V) < 0.5] = NAN
    x[9] = np.where(rng.random(V) < 0.01, -0.0, -2.0)
    x[10] = -np.abs(x[10]) * 1e-40
    x[11, 7] = INF
    u = rng.random(n, dtype=np.float32)
    for kw in (dict(), dict(temperature=[0.0] * n), dict(temperature=[INF] * n), dict(temperature=[1e-40, 1e30, 1e38] * 4),
               dict(top_k=[600, 5000, 2, V] * 3), dict(top_p=[0.9, 0.3, 0.9999] * 4),
               dict(top_k=[700] * n, top_p=[0.9] * n, min_p=[0.01] * n), dict(min_p=[0.5, 1.0, 1e-9] * 4),
               dict(top_p=[NAN, -1.0, 0.0] * 4, min_p=[NAN, 0.2, 0.0] * 4)):
        got, ref = run(M, x, u, f32, pad=V % 4 + 1, **kw)
        assert np.array_equal(got, ref), f"{kw}: rows {np.flatnonzero(got != ref)}"


@pytest.mark.parametrize("V", [65535, 65536, 65537, 131072, 200003])
def test_more_equal_logits_than_16_bits_count(M, V):
    say(f"equal logits {V}")
    x = np.full((5, V), 0.25)
    x[1, 1000] = 3.0
    x[2, ::2] = -1.0
    x[3, :3], x[3, -3:] = 8.0, 8.0
    x[4, V // 2:] = 0.2490234375  # the next value below
    u = np.array([0.9999, 0.5, 0.75, 0.9, 0.6], np.float32)
    for kw in (dict(), dict(top_k=[V - 1, V // 2, 66000, 7, 40000]), dict(top_p=[0.99, 0.5, 0.75, 0.3, 0.6]),
               dict(top_k=[1000] * 5, top_p=[0.999] * 5), dict(min_p=[0.9, 0.01, 0.5, 0.001, 1.0])):
        got, ref = run(M, x, u, False, **kw)
        assert np.array_equal(got, ref), f"{kw}: {got} {ref}"


def test_random_numbers_at_and_past_the_ends(M):
    say("u outside [0, 1)")
    x = np.log(np.array([[1.0, 4.0, 2.0, 4.0, 0.5]])).repeat(6, 0)
    got, _ = run(M, x, [0.0, 1.0 - 2.0 ** -24, 1.0, 5.0, -1.0, NAN], True)
    assert got.tolist() == [1, 4, 4, 4, 1, 1]


def test_same_every_time_and_on_one_row_alone(M):
    """Twice the same, and a row's token does not depend on the other rows."""
    torch = torch_cuda()
    say("sample twice")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = 2 * torch.randn(40, 30011, device="cuda", generator=g)
    u = torch.rand(40, device="cuda", generator=g)
    p = torch.full((40,), 0.95, device="cuda")
    a, b = M.sample(x, u, top_p=p), M.sample(x, u, top_p=p)
    assert torch.equal(a, b)
    for i in (0, 17, 39):
        assert M.sample(x[i:i + 1], u[i:i + 1], top_p=p[i:i + 1]).item() == a[i].item()


def test_rows_of_one_logit_vector(M):
    """One row of logits for many draws (a row stride of 0): the frequencies of
    a counted sweep of u are those of the weights."""
    torch = torch_cuda()
    say("one row, many draws")
    w = np.array([0.5, 0.25, 0.125, 0.125])
    x = torch.tensor(np.log(w), dtype=torch.float32, device="cuda")[None].expand(4000, 4)
    u = (torch.arange(4000, device="cuda") + 0.5) / 4000
    got = torch.bincount(M.sample(x, u).long(), minlength=4).cpu().numpy()
    assert np.abs(got - 4000 * w).max() <= 1


def test_no_rows(M):
    torch = torch_cuda()
    assert M.sample(torch.empty(0, 10, device="cuda"), torch.empty(0, device="cuda")).shape == (0,)


def test_graph_and_streams(M):
    """A captured draw replayed over new logits, eager draws of another size
    between the replays."""
    torch = torch_cuda()
    say("sample in a graph")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x = torch.randn(3, 20000, device="cuda").to(torch.bfloat16)
        u = torch.rand(3, device="cuda")
        k = torch.full((3,), 30, dtype=torch.int32, device="cuda")
        work = M.new_sample_work(3, 20000)
        M.sample(x, u, top_k=k, work=work)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = M.sample(x, u, top_k=k, work=work)
        for i in range(5):
            x.copy_(torch.randn(3, 20000, device="cuda"))
            u.copy_(torch.rand(3, device="cuda"))
            g.replay()
            eager = M.sample(x, u, top_k=k)
            M.sample(x[:1, :777], u[:1], top_k=k[:1])
            side.synchronize()
            assert torch.equal(out, eager), f"replay {i}"
