"""The sampler at temperatures far below the logits' last places, and at logits
far above any temperature: the tokens of the 64-bit oracle, with every output
written.  31 temperatures below the largest logit lie, in fp32, at that logit
itself here; what has a weight is then the largest logits alone, and those a
place or two below them where the temperature is no less than 1/30 of it."""
import numpy as np
import pytest

from gpu_support import say, torch_cuda
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu

TOPS = [2.0, 12.0, 30.5, -20.0, 1000.0, 1e9, -1e9, 1e20]


def logits_of(rng, V, f32):
    """A row for each of TOPS: a bulk well below it, the largest four times and
    the three values below it, a few times each."""
    torch = torch_cuda()
    dt, bits = (torch.float32, torch.int32) if f32 else (torch.bfloat16, torch.int16)
    x = torch.from_numpy(2.2 * rng.normal(size=(len(TOPS), V))).to(torch.float32)
    top = torch.tensor(TOPS, dtype=torch.float32).to(dt)
    x = (top.float()[:, None] - 1 - x.abs() * top.float().abs()[:, None]).to(dt)
    down = top.clone()
    for k, times in enumerate((4, 3, 2, 5)):
        for i in range(len(TOPS)):
            x[i, rng.integers(0, V, times)] = down[i]
        # the value below: nearer to zero by its bits where positive, farther where negative
        down = (down.view(bits) + torch.where(down > 0, -1, 1).to(bits)).view(dt)
    return x.cuda()


COLD = [1e-3, 1e-6, 1e-7, 1e-8, 1e-9, 1e-12, 1e-19, 1.1e-20]


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("V", [40, 1024, 1025, 5000, 16384, 70000])
def test_cold_rows(V, f32):
    torch = torch_cuda()
    import lora_serving_mlora_amd as M
    rng = np.random.default_rng(V + f32)
    n = len(TOPS)
    x = logits_of(rng, V, f32)
    held = x.double().cpu().numpy()
    top = np.abs(held.max(1))
    step = np.abs(held.max(1) - np.array([r[r < r.max()].max() for r in held]))  # to the value below
    mixes = [dict(), dict(top_p=[0.3, 0.9] * (n // 2)), dict(min_p=[0.5, 1e-9] * (n // 2)), dict(top_k=[2] * n),
             dict(top_k=[min(V, 600)] * n, top_p=[0.95] * n, min_p=[1e-6] * n), dict(top_k=[513, 5] * (n // 2))]
    # the fixed ones, 1 over logits of every size, and some around a last place: T = step / 40 .. step * 2
    colds = [np.full(n, t) for t in COLD] + [np.ones(n), step / 40, step / 20, step / 3, step * 2, top * 1e-7, top * 3e-9]
    for j, cold in enumerate(colds):
        kw = dict(mixes[j % len(mixes)], temperature=cold) if j < len(COLD) - 2 else dict(mixes[(j + 1) % 3], temperature=cold)
        say(f"cold rows, {V} f32={f32} T={cold[1]:.3g} {sorted(kw)}")
        dev = {k: torch.tensor(np.asarray(v), dtype=torch.int32 if k == "top_k" else torch.float32, device="cuda")
               for k, v in kw.items()}
        u = torch.tensor(rng.random(n, dtype=np.float32), device="cuda")
        out = torch.full((n,), -77, dtype=torch.int32, device="cuda")
        M.sample(x, u, out=out, **dev)
        ref = S.sample(held, u.cpu().numpy(), **{k: v.cpu().numpy() for k, v in dev.items()})
        got = out.cpu().numpy()
        assert np.array_equal(got, ref), f"{kw}: {got}, not {ref}"


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("V", [2000, 20000])
def test_every_filter_on_cold_rows(V, f32):
    """Each mix of filters at a temperature of 1e-8, the usual stand-in for 0."""
    torch = torch_cuda()
    import lora_serving_mlora_amd as M
    rng = np.random.default_rng(V)
    n = len(TOPS)
    x = logits_of(rng, V, f32)
    held = x.double().cpu().numpy()
    full = dict(top_k=[0, 1, 3, 100, 512, 513, 1500, V], top_p=[1.0, 0.9, 0.5, 0.1, 0.0, 0.7, 0.99, 0.3],
                min_p=[0.0, 1.0, 0.5, 0.1, 1e-12, 2.0, 0.3, 0.01])
    for names in ((), ("top_k",), ("top_p",), ("min_p",), ("top_k", "top_p"), ("top_p", "min_p"),
                  ("top_k", "min_p"), ("top_k", "top_p", "min_p")):
        say(f"filters on cold rows, {V} f32={f32} {names}")
        kw = {k: full[k] for k in names}
        dev = {k: torch.tensor(v, dtype=torch.int32 if k == "top_k" else torch.float32, device="cuda")
               for k, v in kw.items()}
        dev["temperature"] = torch.full((n,), 1e-8, device="cuda")
        u = torch.tensor(rng.random(n, dtype=np.float32), device="cuda")
        out = torch.full((n,), -77, dtype=torch.int32, device="cuda")
        M.sample(x, u, out=out, **dev)
        ref = S.sample(held, u.cpu().numpy(), **{k: v.cpu().numpy() for k, v in dev.items()})
        assert np.array_equal(out.cpu().numpy(), ref), f"{names}: {out.cpu().numpy()}, not {ref}"
