"""An adapter whose Up holds an infinity or NaN reaches the rows that it serves
and no others, in every form of the 4-bit layer."""
import numpy as np
import pytest

from gpu_support import ids_dev, say, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,din,dout,more", [(20, 256, 64, 0), (300, 1056, 33, 0), (1000, 96, 24, 0), (1100, 160, 2880, 0),
                                             (1500, 256, 2816, 0), (1500, 256, 2816, 8), (1030, 96, 33, 0)])
def test_other_rows_stay(n, din, dout, more):
    torch = torch_cuda()
    import lora_serving_mlora_amd as M
    say(f"broken adapters, {n}x{din}x{dout}, {more} more")
    rng = np.random.default_rng(n + more)
    part = lambda *s: torch.from_numpy(rng.normal(size=s).astype(np.float32)).to(torch.bfloat16)
    ranks = [16, 5, 8] + [64] * more
    pool = M.Pool(din, dout, 1, len(ranks), max(ranks), sum(ranks))
    parts = [(part(1, r, din), part(1, dout, r)) for r in ranks]
    for a, (down, up) in enumerate(parts):
        up = up.clone()
        if a < 2:
            up[0, 7 + a, a] = (float("nan"), float("inf"))[a]
        pool.load(a, ranks[a], 1.0, down, up)
    ids = rng.integers(-1, len(ranks), n).astype(np.int32)
    ids[:4] = 0, 1, 2, -1
    seg = M.build_segments(pool, ids_dev(ids))
    w4 = M.q4_quantize(part(dout, din).cuda())
    x = part(n, din).cuda()
    bad = ~torch.isfinite(M.q4_apply(pool, 0, x, w4, seg)).cpu().numpy()
    expect = np.zeros((n, dout), bool)
    expect[ids == 0, 7] = expect[ids == 1, 8] = True
    assert np.array_equal(bad, expect), np.argwhere(bad != expect)[:4]
    # loaded anew without them: as if they had never been
    for a in (0, 1):
        pool.unload(a)
        pool.load(a, ranks[a], 1.0, *parts[a])
    other = M.Pool(din, dout, 1, len(ranks), max(ranks), sum(ranks))
    for a in range(len(ranks)):
        other.load(a, ranks[a], 1.0, *parts[a])
    y, z = (M.q4_apply(p, 0, x, w4, M.build_segments(p, ids_dev(ids))) for p in (pool, other))
    assert torch.isfinite(y).all() and torch.equal(y, z)
    pool.close()
    other.close()
