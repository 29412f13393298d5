"""4-bit products and the layer on inputs whose sums are exact in fp32 in any
order (small whole numbers, scales of 1/2, 1 and 2): the result is then the
exact one rounded to bf16 once, bit for bit, so that a value held in fewer bits
on the way, or a group or rank left out, shows."""
import numpy as np
import pytest

from gpu_support import ids_dev, say, torch_cuda
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    torch_cuda()
    import lora_serving_mlora_amd as M
    return M


def dev(x):
    torch = torch_cuda()
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).cuda()


def weight(M, rng, dout, din):
    torch = torch_cuda()
    codes = rng.integers(0, 256, (dout, din // 2)).astype(np.uint8)
    scales = rng.integers(126, 129, (dout, din // 32)).astype(np.uint8)
    return S.q4_values(codes, scales), M.Q4Weight(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())


def same(got, want):
    """got, bf16, is `want`, exact in fp32, rounded once."""
    torch = torch_cuda()
    assert (np.abs(want).max() * 16 < 2.0 ** 24), "the inputs are not exact"
    ref = torch.from_numpy(want.astype(np.float32)).to(torch.bfloat16)
    got = got.cpu()
    bad = (got != ref).nonzero()
    assert len(bad) == 0, f"{len(bad)} of {got.numel()}, first {bad[0].tolist()}: {got[tuple(bad[0])]}, not {ref[tuple(bad[0])]}"


@pytest.mark.parametrize("n,din,dout", [(1, 32, 3), (1, 4096, 256), (3, 20000, 24), (16, 4064, 200), (16, 11008, 40),
                                        (33, 1056, 257), (61, 11008, 64), (128, 4064, 200), (256, 2048, 512),
                                        (300, 2080, 41), (513, 256, 520), (800, 256, 4104), (1024, 4096, 3080),
                                        (1200, 1056, 264), (2100, 96, 2052), (1100, 4096, 4104)])
def test_product(M, n, din, dout):
    say(f"exact product {n}x{din}x{dout}")
    rng = np.random.default_rng(n + din + dout)
    w, w4 = weight(M, rng, dout, din)
    x = rng.integers(-4, 5, (n, din)).astype(np.float64)
    same(M.q4_gemm(dev(x), w4), x @ w.T)


LAYERS = [  # rows, channels, columns, ranks of the adapters
    (1, 256, 64, [8]), (13, 1056, 72, [1, 16, 64]), (61, 2048, 136, [8, 16, 64]), (200, 1024, 72, [8, 64]),
    (300, 1056, 33, [16, 3]), (1000, 160, 72, [8, 40]), (1024, 1024, 3080, [16, 64]), (70, 96, 40, [4]),
    # more than 1024 rows: the codes as they are, then the bf16 weight with the
    # adapters side by side, and with more of them than fit
    (1100, 128, 72, [8, 40]), (1100, 160, 3900, [8, 40]), (2100, 160, 2050, [8, 40]), (2100, 256, 2048, [16, 33, 64]),
    (1500, 256, 2800, [128, 128]), (2048, 512, 2056, [64] * 6), (1600, 320, 2700, [1] * 40), (1300, 256, 3300, [128, 7, 100]),
    # and small products of that many rows
    (1100, 160, 2880, [8, 40]), (4000, 1024, 1000, [8, 40]), (1100, 96, 40, [4, 17]), (1025, 32, 5, [3]),
    (2100, 64, 1500, [64] * 9), (3000, 96, 1, [2, 128]), (1200, 1056, 3071, [16]),
]


@pytest.mark.parametrize("n,din,dout,ranks", LAYERS, ids=lambda v: "x".join(map(str, v)) if isinstance(v, list) else str(v))
def test_layer(M, n, din, dout, ranks):
    torch = torch_cuda()
    say(f"exact layer {n}x{din}x{dout} {ranks}")
    rng = np.random.default_rng(n + din + dout)
    w, w4 = weight(M, rng, dout, din)
    x = rng.integers(1, 5, (n, din)).astype(np.float64)
    ids = rng.integers(-1, len(ranks), n).astype(np.int32)
    want = x @ w.T
    pool = M.Pool(din, dout, 1, len(ranks), max(ranks), sum(ranks))
    for a, r in enumerate(ranks):
        # inner values of some thousands, more than bf16 holds, of either sign
        down = rng.integers(1, 4, (r, din)) * rng.choice([-1, 1], (r, 1)).astype(np.float64)
        up = rng.choice([-0.25, 0.0, 0.25], (dout, r))
        s = 2.0 ** (a % 3 - 1)
        pool.load(a, r, s, dev(down)[None], dev(up)[None])
        rows = ids == a
        want[rows] += s * (x[rows] @ down.T) @ up.T
    seg = M.build_segments(pool, ids_dev(ids))
    work = torch.full((max(M.q4_work_bytes(w4, n, pool), 256),), 0xff, dtype=torch.uint8, device="cuda")
    same(M.q4_apply(pool, 0, dev(x), w4, seg, work=work), want)
    pool.close()
