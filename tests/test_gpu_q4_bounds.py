"""Where the 4-bit products read and write: outputs and work buffers between
guards in every form, operands wherever their element size lets them begin."""
import numpy as np
import pytest

from gpu_support import ids_dev, say, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    torch_cuda()
    import lora_serving_mlora_amd as M
    return M


def weight(M, rng, dout, din, odd=0):
    """odd: the scales begin so many bytes past an aligned address."""
    torch = torch_cuda()
    codes = torch.from_numpy(rng.integers(0, 256, (dout, din // 2)).astype(np.uint8)).cuda()
    held = torch.from_numpy(rng.integers(118, 126, odd + dout * din // 32).astype(np.uint8)).cuda()
    return M.Q4Weight(codes, held[odd:].view(dout, din // 32))


def layer(M, rng, n, din, dout, ranks):
    torch = torch_cuda()
    x = torch.from_numpy(rng.normal(size=(n, din)).astype(np.float32)).to(torch.bfloat16).cuda()
    pool = M.Pool(din, dout, 1, len(ranks), max(ranks), sum(ranks))
    for a, r in enumerate(ranks):
        part = lambda *s: torch.from_numpy(rng.normal(size=s).astype(np.float32)).to(torch.bfloat16)
        pool.load(a, r, 0.5, part(1, r, din), part(1, dout, r))
    return x, pool, M.build_segments(pool, ids_dev(rng.integers(-1, len(ranks), n).astype(np.int32)))


FORMS = [(1, 256, 45), (70, 1056, 40), (300, 2080, 41), (700, 160, 1032), (1024, 96, 24), (1030, 96, 33), (1100, 160, 2880),
         (2100, 160, 2050), (4096, 512, 64)]


@pytest.mark.parametrize("n,din,dout", FORMS)
def test_work_ends_where_it_ends(M, n, din, dout):
    """A work buffer of the stated size: what lies behind it stays, and the
    result does not depend on what it held."""
    torch = torch_cuda()
    say(f"guarded work {n}x{din}x{dout}")
    rng = np.random.default_rng(n + dout)
    w4 = weight(M, rng, dout, din)
    x, pool, seg = layer(M, rng, n, din, dout, [3, 40])
    for size, call in ((M.q4_work_bytes(w4, n), lambda work: M.q4_gemm(x, w4, work=work)),
                       (M.q4_work_bytes(w4, n, pool), lambda work: M.q4_apply(pool, 0, x, w4, seg, work=work))):
        out = []
        for fill in (0, 0xff):
            buf = torch.full((size + 4096,), fill, dtype=torch.uint8, device="cuda")
            out.append(call(buf[:size]) if size else call(buf[:256]))
            assert (buf[max(size, 256):] == fill).all()
        assert torch.equal(out[0].view(torch.int16), out[1].view(torch.int16))
    pool.close()


def test_work_of_the_inner_products(M):
    """One slice of inner values where one is all that the width asks for."""
    w4 = weight(M, np.random.default_rng(0), 64, 512)
    n, rank = 8192, 128
    pool = M.Pool(512, 64, 1, 1, rank, rank)
    assert M.q4_work_bytes(w4, n, pool) <= n * rank * 4 + n * 64 * 4 + 512
    pool.close()


@pytest.mark.parametrize("n,din,dout", FORMS)
def test_outputs_end_where_they_end(M, n, din, dout):
    """Nothing is written before or behind Y, aligned or not."""
    torch = torch_cuda()
    say(f"guarded outputs {n}x{din}x{dout}")
    rng = np.random.default_rng(n + din)
    w4 = weight(M, rng, dout, din)
    x, pool, seg = layer(M, rng, n, din, dout, [17, 8])
    for call in (lambda Y=None: M.q4_gemm(x, w4, Y=Y), lambda Y=None: M.q4_apply(pool, 0, x, w4, seg, Y=Y)):
        want = call()
        assert torch.isfinite(want).all()
        for at in (3, 8):
            buf = torch.full((at + n * dout + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
            call(buf[at:at + n * dout].view(n, dout))
            # (where another form takes outputs without alignment, its sums have an order of their own: a
            # step of bf16 apart, 2^-7, doubled, and what cancels; here it is the place that is looked at)
            near = torch.isclose(buf[at:at + n * dout].view(n, dout).float(), want.float(), rtol=2.0 ** -6, atol=0.05)
            assert near.all() and (buf[:at] == 7).all() and (buf[at + n * dout:] == 7).all()
    pool.close()


@pytest.mark.parametrize("n,din,dout", [(1, 256, 45), (17, 1056, 40), (70, 1056, 40), (300, 2080, 41), (1100, 160, 2880)])
@pytest.mark.parametrize("odd", [1, 2, 3])
def test_scales_at_any_address(M, n, din, dout, odd):
    """Scale bytes that begin at no word's address give the same bits."""
    torch = torch_cuda()
    say(f"scales {odd} bytes on, {n}x{din}x{dout}")
    rng = np.random.default_rng(n)
    w4 = weight(M, rng, dout, din, odd)
    again = M.Q4Weight(w4.codes, w4.scales.clone())
    assert w4.scales.data_ptr() % 4 == odd and again.scales.data_ptr() % 4 == 0
    x, pool, seg = layer(M, rng, n, din, dout, [17, 8])
    bits = lambda t: t.view(torch.int16)
    assert torch.equal(bits(M.q4_dequantize(w4)), bits(M.q4_dequantize(again)))
    assert torch.equal(bits(M.q4_gemm(x, w4)), bits(M.q4_gemm(x, again)))
    assert torch.equal(bits(M.q4_apply(pool, 0, x, w4, seg)), bits(M.q4_apply(pool, 0, x, again, seg)))
    pool.close()
