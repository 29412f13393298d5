"""Captured calls of the forms for many rows and large vocabularies, replayed
over new inputs with eager work of other sizes between the replays, and beside
each other on two streams."""
import numpy as np
import pytest

from gpu_support import ids_dev, say, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    torch_cuda()
    import lora_serving_mlora_amd as M
    return M


def same(a, b):
    torch = torch_cuda()
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("n,din,dout,ranks", [(700, 512, 1024, [16, 5]), (1100, 160, 2880, [8, 40]),
                                              (1500, 256, 2816, [64] * 9), (1025, 96, 40, [4])])
def test_layer_of_many_rows(M, n, din, dout, ranks):
    torch = torch_cuda()
    say(f"captured layer {n}x{din}x{dout}")
    g = torch.Generator(device="cuda").manual_seed(n)
    part = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)
    pool = M.Pool(din, dout, 1, len(ranks), max(ranks), sum(ranks))
    for a, r in enumerate(ranks):
        pool.load(a, r, 0.5, part(1, r, din).cpu(), part(1, dout, r).cpu())
    w4 = M.q4_quantize(part(dout, din))
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            x = part(n, din)
            ids = ids_dev(np.random.default_rng(i).integers(-1, len(ranks), n).astype(np.int32))
            work = M.new_q4_work(w4, n, pool)
            seg = M.build_segments(pool, ids)
            M.q4_apply(pool, 0, x, w4, seg, work=work)
            side.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                seg = M.build_segments(pool, ids)
                y = M.q4_apply(pool, 0, x, w4, seg, work=work)
        graphs.append((side, graph, x, ids, seg, work, y))
    torch.cuda.synchronize()
    for replay in range(4):
        for _, _, x, ids, *_ in graphs:
            x.copy_(part(n, din))
            ids.copy_(torch.randint(-1, len(ranks), (n,), dtype=torch.int32, device="cuda", generator=g))
        torch.cuda.synchronize()
        for side, graph, *_ in graphs:
            with torch.cuda.stream(side):
                graph.replay()
        other = M.q4_gemm(part(33, din), w4)
        torch.cuda.synchronize()
        assert torch.isfinite(other).all()
        for _, _, x, ids, _, _, y in graphs:
            assert same(y, M.q4_apply(pool, 0, x, w4, M.build_segments(pool, ids))), f"replay {replay}"
    pool.close()


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("V", [900, 40000])
def test_sampling(M, V, f32):
    """Without a small top-k: counted values in bf16, the histogram in fp32."""
    torch = torch_cuda()
    say(f"captured draws of {V} f32={f32}")
    n, dt = 5, torch.float32 if f32 else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(V)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x = torch.randn(n, V, device="cuda", generator=g).to(dt)
        u = torch.rand(n, device="cuda", generator=g)
        t, p = torch.ones(n, device="cuda"), torch.full((n,), 0.9, device="cuda")
        M.sample(x, u, t, top_p=p)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = M.sample(x, u, t, top_p=p)
        for replay in range(5):
            x.copy_(3 * torch.randn(n, V, device="cuda", generator=g))
            u.copy_(torch.rand(n, device="cuda", generator=g))
            t.copy_(torch.tensor([0.0, 1e-8, 0.5, 1.0, 3.0], device="cuda").roll(replay))
            graph.replay()
            eager = M.sample(x, u, t, top_p=p)
            M.sample(x[:2, :333], u[:2])
            side.synchronize()
            assert torch.equal(out, eager), f"replay {replay}"
