"""Norms of queries and keys with the rotation, on the GPU, against 64 bits;
the bound is derived in oracle/step_oracle.py beside its terms."""
import numpy as np
import pytest

from gpu_support import dev_to_f64, say, torch_cuda
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


def batch_of(M, new, total, n_rows=None, width=1):
    torch = torch_cuda()
    ints = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")
    off = np.concatenate([[0], np.cumsum(new)])
    n = int(off[-1]) if n_rows is None else n_rows
    table = torch.zeros(len(new), width, dtype=torch.int32, device="cuda")
    return M.KVBatch(table, ints(total), ints(off), n, max_new=max(max(new), 1)), (np.array(total), off), n


def check(y, ref, bound):
    y = dev_to_f64(y)
    had = ~np.isnan(ref)
    bad = (np.abs(y - ref) - bound)[had]
    assert bad.max() <= 0, f"{bad.max()} over the bound"


CASES = [  # new, total, heads, kv_heads, dim, rot, norm, interleaved
    ([1], [1], 1, 1, 16, 8, True, False),
    ([1, 1, 1, 1], [5, 300, 17, 1], 32, 8, 128, 128, True, False),
    ([1] * 70, list(range(1, 71)), 4, 1, 64, 64, True, True),
    ([0, 3, 0, 0, 7, 1, 0], [0, 3, 50, 0, 1000, 131000, 9], 7, 7, 80, 32, True, False),
    ([40, 25], [40, 90], 5, 1, 96, 96, False, True),
    ([300, 1, 200], [5000, 70, 200], 8, 2, 256, 64, True, False),
    ([9], [(1 << 30) - 1], 3, 1, 192, 192, True, False),
    ([2, 2], [100000, 999999], 2, 2, 112, 16, False, False),
    ([1] * 300, [3] * 300, 2, 1, 32, 32, True, False),
    ([1500], [1500], 40, 8, 64, 64, True, False),
    ([700, 800], [700, 900], 40, 8, 256, 256, True, False),
    ([3000], [3007], 9, 9, 80, 32, True, True),
    ([5], [2], 2, 1, 48, 40, True, True),  # three rows at negative positions
]


@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{sum(c[0])}rows-{c[2]}x{c[4]}-rot{c[5]}")
def test_against_64_bits(M, case, pad):
    """Slices of a joint projection's rows; with pad also rows that no wide
    load can take."""
    torch = torch_cuda()
    new, total, H, Hk, D, rot, norm, inter = case
    say(f"rotation {case[2:]} {sum(new)} rows pad {pad}")
    rng = np.random.default_rng(sum(new) + D)
    b, ob, n = batch_of(M, new, total)
    x = bf16(rng.normal(size=(n, H + 2 * Hk, D)) * np.exp(rng.normal(size=(n, H + 2 * Hk, 1))))
    buf = torch.zeros(n, (H + 2 * Hk) * (D + pad) + pad, dtype=torch.bfloat16, device="cuda")
    heads = buf[:, pad:].unflatten(1, (H + 2 * Hk, D + pad))[:, :, :D]
    heads.copy_(dev(x))
    qw, kw = (bf16(1 + 0.3 * rng.normal(size=D)) for _ in range(2)) if norm else (None, None)
    r = M.Rotary(rot, base=10000.0, interleaved=inter, factor=1.25)
    freqs = 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    wd = lambda w: None if w is None else dev(w)
    q, k = M.qk_norm_rotary(heads[:, :H], heads[:, H:H + Hk], b, r, q_weight=wd(qw), k_weight=wd(kw), eps=1e-5)
    rq = S.qk_norm_rotary(x[:, :H], qw, 1e-5, ob, freqs, inter, 1.25)
    rk = S.qk_norm_rotary(x[:, H:H + Hk], kw, 1e-5, ob, freqs, inter, 1.25)
    check(q, *rq)
    check(k, *rk)
    before = buf.clone()
    q2, k2 = M.qk_norm_rotary(heads[:, :H], heads[:, H:H + Hk], b, r, q_weight=wd(qw), k_weight=wd(kw), eps=1e-5,
                              q_out=heads[:, :H], k_out=heads[:, H:H + Hk])
    assert torch.equal(q2, q) and torch.equal(k2, k), "in place differs"
    was = before[:, pad:].unflatten(1, (H + 2 * Hk, D + pad))
    now = buf[:, pad:].unflatten(1, (H + 2 * Hk, D + pad))
    assert torch.equal(was[:, H + Hk:], now[:, H + Hk:]) and torch.equal(was[..., D:], now[..., D:])


def test_one_side_and_other_weights(M):
    torch = torch_cuda()
    say("queries alone; a norm on one side")
    rng = np.random.default_rng(3)
    b, ob, n = batch_of(M, [4, 2], [9, 2])
    x, y = bf16(rng.normal(size=(n, 3, 64))), bf16(rng.normal(size=(n, 1, 64)))
    w = bf16(1 + 0.1 * rng.normal(size=64))
    freqs = rng.uniform(0, 3, 32)
    r = M.Rotary(64, freqs=freqs)
    q, none = M.qk_norm_rotary(dev(x), None, b, r, q_weight=dev(w))
    assert none is None
    check(q, *S.qk_norm_rotary(x, w, 1e-6, ob, freqs))
    q, k = M.qk_norm_rotary(dev(x), dev(y), b, r, k_weight=dev(w))
    check(q, *S.qk_norm_rotary(x, None, 0, ob, freqs))
    check(k, *S.qk_norm_rotary(y, w, 1e-6, ob, freqs))


def test_rows_past_the_last_sequence(M):
    torch = torch_cuda()
    say("rows past the last sequence")
    b, _, n = batch_of(M, [2, 0, 1], [5, 0, 1], n_rows=9)
    x = torch.randn(n, 4, 64, device="cuda").to(torch.bfloat16)
    out, kout = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    M.qk_norm_rotary(x, x.clone(), b, M.Rotary(64), q_out=out, k_out=kout)
    assert (out[3:] == 7).all() and (kout[3:] == 7).all() and not (out[:3] == 7).all()


def test_offsets_that_make_no_sense(M):
    """Offsets out of order or past the batch: nothing outside the rows is
    read or written (a guard around the output)."""
    torch = torch_cuda()
    say("offsets out of order")
    for off in ([0, 9, 2, 6], [3, 4, 5, 6], [-5, 2, 100, 1 << 30], [6, 6, 6, 6], [0, 0, 0, 0]):
        t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
        b = M.KVBatch(torch.zeros(3, 1, dtype=torch.int32, device="cuda"), t([7, -(1 << 31), (1 << 31) - 1]), t(off), 6)
        x = torch.randn(6, 2, 32, device="cuda").to(torch.bfloat16)
        guard = torch.full((18, 2, 32), 3.0, dtype=torch.bfloat16, device="cuda")
        M.qk_norm_rotary(x, None, b, M.Rotary(32), q_out=guard[6:12])
        assert (guard[:6] == 3).all() and (guard[12:] == 3).all()


def test_infinities_and_nan_stay_in_their_head(M):
    torch = torch_cuda()
    say("NaN heads")
    b, _, n = batch_of(M, [3], [3])
    x = torch.randn(n, 4, 64, device="cuda").to(torch.bfloat16)
    x[1, 2, 5], x[0, 1, 60] = float("nan"), float("inf")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    q, _ = M.qk_norm_rotary(x, None, b, M.Rotary(64), q_weight=w)
    bad = (~torch.isfinite(q)).any(-1).cpu().tolist()
    assert bad == [[False, True, False, False], [False, False, True, False], [False] * 4]


def test_zero_heads_with_eps(M):
    torch = torch_cuda()
    b, _, n = batch_of(M, [2], [2])
    x = torch.zeros(n, 2, 64, device="cuda", dtype=torch.bfloat16)
    q, _ = M.qk_norm_rotary(x, None, b, M.Rotary(64), q_weight=torch.ones(64, dtype=torch.bfloat16, device="cuda"))
    assert (q == 0).all()


def test_graph_with_advancing_lengths(M):
    torch = torch_cuda()
    say("rotation in a graph")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b, _, n = batch_of(M, [1] * 5, [10, 20, 30, 40, 50])
        x = torch.randn(n, 6, 128, device="cuda").to(torch.bfloat16)
        r = M.Rotary(128)
        M.qk_norm_rotary(x[:, :4], x[:, 4:], b, r)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            b.kv_len.add_(1)
            q, k = M.qk_norm_rotary(x[:, :4], x[:, 4:], b, r)
        for i in range(4):
            x.copy_(torch.randn(n, 6, 128, device="cuda"))
            g.replay()
            eq, ek = M.qk_norm_rotary(x[:, :4], x[:, 4:], b, r)
            side.synchronize()
            assert torch.equal(q, eq) and torch.equal(k, ek), f"replay {i}"
