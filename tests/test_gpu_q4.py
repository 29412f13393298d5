"""4-bit weights on the GPU: the quantiser and the way back bit for bit, the
products and the layer against 64 bits.

Tolerance of a product: each bf16 x bf16 product is exact in fp32; a sum of K
of them in any order, each addition off by a step at most (2^-23), is within
K 2^-23 of the sum of magnitudes; the low-rank term adds its own two sums, and
one bf16 rounding of its inner values where the batch has more than 1024 rows;
the result is rounded to bf16 once (2^-8)."""
import numpy as np
import pytest

import oracle as O
import synth
from gpu_support import dev_to_f64, ids_dev, make_pool, oracle_adapters, say, to_dev_bf16, torch_cuda
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    torch_cuda()
    import lora_serving_mlora_amd as M
    return M


def bf16(x):
    torch = torch_cuda()
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).double().numpy()


def dev(x):
    torch = torch_cuda()
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).cuda()


def weight(M, rng, dout, din, lo=118, hi=126):
    torch = torch_cuda()
    codes = rng.integers(0, 256, (dout, din // 2)).astype(np.uint8)
    scales = rng.integers(lo, hi, (dout, din // 32)).astype(np.uint8)
    return codes, scales, M.Q4Weight(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())


@pytest.mark.parametrize("dout,din", [(1, 32), (3, 64), (7, 96), (65, 160), (16, 4096)])
def test_quantizer(M, dout, din):
    say(f"quantise {dout}x{din}")
    rng = np.random.default_rng(dout * din)
    w = bf16(rng.normal(size=(dout, din)) * np.exp2(rng.integers(-20, 20, (dout, din // 32))).repeat(32, 1))
    flat = w.reshape(-1)
    flat[:32] = bf16(np.array([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, 5.5] * 2))
    if flat.size > 128:
        flat[32:64] = 0
        flat[64:96] = bf16(np.linspace(-3.3e38, 3.3e38, 32))
        flat[96:128] = bf16(np.linspace(-1e-37, 1e-37, 32))
    codes, scales = S.q4_quantize(w)
    q = M.q4_quantize(dev(w))
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    same = lambda c: np.stack((c & 15, c >> 4))
    neg0 = lambda c: np.where(c == 8, 0, c)  # -0 and 0 are the same weight
    assert np.array_equal(neg0(same(q.codes.cpu().numpy())), neg0(same(codes)))
    assert np.array_equal(dev_to_f64(M.q4_dequantize(q)), S.q4_values(codes, scales))


def test_quantizer_of_every_value(M):
    """Every finite bf16 value as the largest of its group and beside it, in
    groups whose scale another value sets, the smallest numbers included."""
    torch = torch_cuda()
    say("quantise every value")
    bits = np.arange(1 << 16)
    bits = bits[(bits & 0x7f80) != 0x7f80].astype(np.uint16)
    value = lambda b: (b.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    rng = np.random.default_rng(12)
    x = value(bits)
    beside = value(rng.choice(bits, (len(x), 15)))
    near = bf16(x[:, None] * rng.uniform(-1, 1, (len(x), 8)))
    halves = bf16(np.clip(np.exp2(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -133)))[:, None] - 2)
                          * np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]), 0, 3.3e38))
    for other in (np.zeros((len(x), 31)), np.concatenate([x[:, None] * 0, near, near / 4, near / 64, x[:, None] * 0 + 0.0,
                                                          near[:, :5]], 1),
                  np.concatenate([halves, -halves, beside * 0], 1), np.concatenate([beside, beside, x[:, None]], 1)):
        w = bf16(np.concatenate([x[:, None], other], 1))
        w = w[np.isfinite(w).all(1)]
        # the oracle's definition, all groups at once
        m, ex = np.frexp(np.abs(w).max(1))  # 6 * 2^e is 0.75 * 2^(e + 3)
        e = np.where(m == 0, -125, np.clip(np.where(m <= 0.75, ex - 3, ex - 2), -125, 125))
        a = np.minimum(np.abs(w) / np.exp2(e)[:, None], 6.0)
        d = np.abs(a[..., None] - S.LEVELS)
        k = d.argmin(-1)
        tie = np.take_along_axis(d, np.minimum(k + 1, 7)[..., None], -1)[..., 0] == d.min(-1)
        k += (tie & (k % 2 == 1) & (k < 7)).astype(k.dtype)
        q = M.q4_quantize(dev(w))
        assert np.array_equal(q.scales.cpu().numpy()[:, 0], e + 127)
        got = dev_to_f64(M.q4_dequantize(q))
        want = np.where(np.signbit(w), -S.LEVELS[k], S.LEVELS[k]) * np.exp2(e)[:, None]
        bad = np.argwhere(got != want)
        assert len(bad) == 0, f"{len(bad)}, first {w[tuple(bad[0])]}: {got[tuple(bad[0])]}, not {want[tuple(bad[0])]}"
        rows = rng.choice(len(w), 40, replace=False)
        codes, scales = S.q4_quantize(w[rows])
        assert np.array_equal(S.q4_values(codes, scales), want[rows])


def test_quantizer_of_infinities_and_nan(M):
    torch = torch_cuda()
    w = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    w[0, 3], w[1, 40], w[2, 63] = float("inf"), float("nan"), float("-inf")
    say("quantise infinities")
    q = M.q4_quantize(w)
    assert q.scales.cpu().tolist() == [[255, 125], [125, 255], [125, 255], [125, 125]]
    nan = torch.isnan(M.q4_dequantize(q)).view(4, 2, 32)
    assert nan.all(-1).cpu().tolist() == [[True, False], [False, True], [False, True], [False, False]]


def test_every_code_and_scale(M):
    """All 16 codes under all 256 scale bytes."""
    torch = torch_cuda()
    codes = np.tile((np.arange(16) | (np.arange(16) ^ 15) << 4).astype(np.uint8), (256, 1))
    scales = np.arange(256, dtype=np.uint8)[:, None]
    say("every code and scale")
    got = dev_to_f64(M.q4_dequantize(M.Q4Weight(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())))
    assert np.array_equal(got, S.q4_values(codes, scales), equal_nan=True)


def within(y, ref, mag, din, extra=0.0):
    err = mag * (din + 8) * 2.0 ** -23 + extra
    bad = np.abs(y - ref) - (err + (np.abs(ref) + err) * 2.0 ** -8)
    assert bad.max() <= 0, f"{bad.max()} over the bound at {np.unravel_index(bad.argmax(), bad.shape)}"


SHAPES = [(1, 32, 1), (1, 4096, 256), (2, 96, 17), (5, 160, 64), (16, 4064, 200), (16, 128, 8), (17, 2048, 72),
          (33, 1056, 257), (48, 512, 16), (63, 544, 130), (64, 4096, 128), (64, 11008, 64), (16, 11008, 40),
          (3, 20000, 24), (65, 512, 128), (100, 96, 33), (257, 1024, 264), (1025, 256, 136), (128, 4064, 200),
          (300, 2080, 41), (511, 256, 520), (513, 256, 520), (700, 160, 1032), (1000, 96, 24), (1024, 1056, 17),
          (1200, 1056, 264), (2100, 96, 2052), (1030, 32, 40), (800, 256, 4104), (1600, 256, 2056),
          (2100, 256, 2056), (1100, 160, 2880), (4000, 128, 72)]


@pytest.mark.parametrize("n,din,dout", SHAPES)
def test_product(M, n, din, dout):
    say(f"4-bit product {n}x{din}x{dout}")
    rng = np.random.default_rng(n + din + dout)
    codes, scales, w4 = weight(M, rng, dout, din)
    w = S.q4_values(codes, scales)
    x = bf16(rng.normal(size=(n, din)))
    y = dev_to_f64(M.q4_gemm(dev(x), w4))
    within(y, x @ w.T, np.abs(x) @ np.abs(w).T, din)


@pytest.mark.parametrize("n", [1, 20, 64])
def test_nan_stays_in_its_row_and_column(M, n):
    """A NaN row of X, a NaN group of the weight and a ragged last step reach
    nothing else."""
    say(f"NaN row, {n} rows")
    rng = np.random.default_rng(n)
    din, dout = 1056, 40
    codes, scales, _ = weight(M, rng, dout, din)
    scales[7, 32] = 255  # the last group of row 7
    torch = torch_cuda()
    w4 = M.Q4Weight(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    x = bf16(rng.normal(size=(n, din)))
    x[n // 2, 5] = np.nan
    y = dev_to_f64(M.q4_gemm(dev(x), w4))
    expect = np.zeros((n, dout), bool)
    expect[n // 2] = expect[:, 7] = True
    assert np.array_equal(np.isnan(y), expect)


LAYERS = [(1, 256, 64, {0: 8}), (13, 1056, 72, {0: 1, 1: 16, 2: 64}), (32, 4096, 256, {0: 16, 1: 16, 2: 16}),
          (48, 512, 33, {0: 4, 2: 33}), (64, 2080, 136, {0: 128, 1: 3}), (65, 512, 128, {0: 16, 1: 5}),
          (200, 1024, 72, {0: 8, 1: 64}), (1100, 128, 72, {0: 8, 1: 40}), (130, 2080, 72, {0: 128, 1: 16}),
          (255, 512, 264, {0: 1, 1: 16, 2: 33}), (257, 512, 264, {0: 8, 1: 16}), (300, 1056, 33, {0: 16, 1: 3}),
          (1000, 160, 72, {0: 8, 1: 40}), (70, 96, 40, {0: 4}), (1100, 160, 72, {0: 8, 1: 40}),
          (2100, 160, 2050, {0: 8, 1: 40}), (5, 256, 5, {0: 8}), (20, 256, 9, {0: 16}), (70, 1056, 517, {0: 64, 2: 17}),
          (800, 256, 4104, {0: 8, 1: 40}), (1600, 256, 2056, {0: 8, 1: 40}), (2100, 256, 2048, {0: 16, 1: 40}),
          (1100, 160, 2880, {0: 8, 1: 40}), (3000, 256, 64, {0: 8, 1: 16})]


@pytest.mark.parametrize("n,din,dout,ranks", LAYERS)
def test_layer(M, n, din, dout, ranks):
    say(f"4-bit layer {n}x{din}x{dout} {ranks}")
    w = synth.custom("q4", n + din, din, dout, synth.random_ids(n + din, n, sorted(ranks), 0.25), ranks)
    pool = make_pool(M, w)
    rng = np.random.default_rng(n)
    codes, scales, w4 = weight(M, rng, dout, din, 114, 122)
    ids = w.row_adapter.copy()
    if n > 4:
        ids[3] = w.max_adapters + 5  # an id that is not there: a row of NaN
    X = w.x_bits()
    seg = M.build_segments(pool, ids_dev(ids))
    work = torch_cuda().full((max(M.q4_work_bytes(w4, n, pool), 256),), 0xff, dtype=torch_cuda().uint8, device="cuda")
    Y = M.q4_apply(pool, 0, to_dev_bf16(X), w4, seg, work=work)
    y = dev_to_f64(Y)
    x, wv = O.widen_bf16(X), S.q4_values(codes, scales)
    ref, mag, extra = x @ wv.T, np.abs(x) @ np.abs(wv).T, np.zeros((n, dout))
    for a, (s, down, up) in oracle_adapters(w).items():
        rows = ids == a
        t, ta = s * (x[rows] @ down.T), abs(s) * (np.abs(x[rows]) @ np.abs(down).T)
        ref[rows] += t @ up.T
        mag[rows] += (ta @ np.abs(up).T) * (1 + ranks[a] / din)
        if n > 1024:
            # the grouped plan of a small shape stores the base product as bf16
            # and adds the low-rank term to that: a second rounding, of the
            # base product; other shapes round the inner values t instead
            extra[rows] = (np.abs(t) @ np.abs(up).T + np.abs(x[rows] @ wv.T)) * 2.0 ** -8
    if n > 4:
        assert np.isnan(y[3]).all()
        y[3] = ref[3] = mag[3] = 0
    within(y, ref, mag, 2 * din + max(ranks.values()), extra)
    again = M.q4_apply(pool, 0, to_dev_bf16(X), w4, seg)
    assert torch_cuda().equal(Y.view(torch_cuda().int16), again.view(torch_cuda().int16)), "not the same twice"
    pool.close()


def test_a_merged_weight_in_4_bits(M):
    """merge, then quantise: the layer without adapters on the merged weight."""
    w = synth.custom("q4merge", 5, 256, 64, np.zeros(9, np.int32), {0: 8})
    pool = make_pool(M, w)
    say("merge, quantise, product")
    W0 = to_dev_bf16(w.w0_bits())
    M.merge(pool, 0, 0, W0)
    w4 = M.q4_quantize(W0)
    wv = S.q4_values(*S.q4_quantize(dev_to_f64(W0)))
    x = O.widen_bf16(w.x_bits())
    y = dev_to_f64(M.q4_gemm(to_dev_bf16(w.x_bits()), w4))
    within(y, x @ wv.T, np.abs(x) @ np.abs(wv).T, 256)
    pool.close()


def test_no_rows(M):
    torch = torch_cuda()
    _, _, w4 = weight(M, np.random.default_rng(0), 8, 64)
    assert tuple(M.q4_gemm(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), w4).shape) == (0, 8)


def test_graph_and_streams(M):
    """A captured step, replayed with new inputs and eager work of another
    batch size between the replays, on a stream of its own."""
    torch = torch_cuda()
    say("4-bit layer in a graph")
    w = synth.custom("q4graph", 9, 512, 256, synth.random_ids(9, 24, [0, 1], 0.25), {0: 16, 1: 8})
    pool = make_pool(M, w)
    rng = np.random.default_rng(1)
    _, _, w4 = weight(M, rng, 256, 512)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ids = ids_dev(w.row_adapter)
        X = to_dev_bf16(w.x_bits())
        seg = M.build_segments(pool, ids)
        work = M.new_q4_work(w4, 24, pool)
        M.q4_apply(pool, 0, X, w4, seg, work=work)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            Y = M.q4_apply(pool, 0, X, w4, seg, work=work)
        for i in range(4):
            X.copy_(dev(rng.normal(size=(24, 512))))
            g.replay()
            eager = M.q4_apply(pool, 0, X, w4, seg)
            other = M.q4_gemm(X[:3].clone(), w4)
            big = M.q4_gemm(X.repeat(4, 1), w4)
            side.synchronize()
            assert torch.equal(Y.view(torch.int16), eager.view(torch.int16)), f"replay {i}"
            assert torch.isfinite(other).all() and torch.isfinite(big).all()
    pool.close()


def test_two_graphs_and_an_eager_call_side_by_side(M):
    """Two captured layers with work buffers of their own, replayed on two
    streams at once while a third call runs, each as when alone."""
    torch = torch_cuda()
    say("4-bit layers side by side")
    w = synth.custom("q4two", 4, 1056, 136, synth.random_ids(4, 40, [0, 1], 0.25), {0: 33, 1: 8})
    pool = make_pool(M, w)
    _, _, w4 = weight(M, np.random.default_rng(2), 136, 1056)
    X, ids = to_dev_bf16(w.x_bits()), ids_dev(w.row_adapter)
    seg = M.build_segments(pool, ids)
    want = M.q4_apply(pool, 0, X, w4, seg)
    want2 = M.q4_gemm(X, w4)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            work = M.new_q4_work(w4, 40, pool)
            M.q4_apply(pool, 0, X, w4, seg, work=work)
            side.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                Y = M.q4_apply(pool, 0, X, w4, seg, work=work)
        graphs.append((side, g, Y, work))
    for i in range(4):
        for side, g, Y, _ in graphs:
            with torch.cuda.stream(side):
                Y.zero_()
                g.replay()
        Y2 = M.q4_gemm(X, w4)
        torch.cuda.synchronize()
        assert all(torch.equal(Y, want) for _, _, Y, _ in graphs) and torch.equal(Y2, want2), f"replay {i}"
    pool.close()


def test_outputs_end_where_they_end(M):
    """Nothing is written before or behind Y, whatever its alignment."""
    torch = torch_cuda()
    rng = np.random.default_rng(8)
    w = synth.custom("q4ends", 6, 256, 45, synth.random_ids(6, 70, [0], 0.25), {0: 16})
    pool = make_pool(M, w)
    _, _, w4 = weight(M, rng, 45, 256)
    X, seg = to_dev_bf16(w.x_bits()), M.build_segments(pool, ids_dev(w.row_adapter))
    for n in (1, 33, 70):
        say(f"guarded outputs, {n} rows")
        buf = torch.full((3 + n * 45 + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
        Y = buf[3:3 + n * 45].view(n, 45)
        M.q4_gemm(X[:n], w4, Y=Y)
        assert torch.equal(Y, M.q4_gemm(X[:n], w4)) and (buf[:3] == 7).all() and (buf[3 + n * 45:] == 7).all()
    buf = torch.full((3 + 70 * 45 + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    Y = M.q4_apply(pool, 0, X, w4, seg, Y=buf[3:3 + 70 * 45].view(70, 45))
    again = M.q4_apply(pool, 0, X, w4, seg)
    assert torch.equal(Y, again) and (buf[:3] == 7).all() and (buf[3 + 70 * 45:] == 7).all()
    pool.close()
