"""The example's attention layer, step by step, eager and from its graph: each
stage against the oracles on what the stage before it gave (projections within
the layer's tolerance, the cache bit for bit, attention within its bound)."""
import os
import sys

import numpy as np
import pytest

import oracle as O
from gpu_support import assert_close, dev_to_f64, say, torch_cuda
from oracle import kv_oracle as K

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _adapters(w):
    return {a: (w.scales[a], O.widen_bf16(w.down_bits(a, 0)), O.widen_bf16(w.up_bits(a, 0))) for a in w.adapter_ids()}


@pytest.mark.parametrize("requests,prompt,heads,kv_heads,dim,block", [(3, 40, 4, 2, 64, 16), (7, 90, 8, 1, 128, 32)])
def test_layer(requests, prompt, heads, kv_heads, dim, block):
    torch = torch_cuda()
    import attention_layer as E
    held = {}
    seen = []

    def check(layer, X, ids, cache, batch, results):
        torch.cuda.synchronize()
        out, att, qkv = (dev_to_f64(r) for r in results)
        ids, n = ids.cpu().numpy(), batch.n_rows
        say(f"attention layer, {n} rows, step {len(seen)}")
        w = layer.workloads
        x = dev_to_f64(X)
        ref = O.linear(x, O.widen_bf16(w[0].w0_bits(0)), ids, _adapters(w[0]), w[0].max_adapters)
        assert_close(qkv, ref, f"q/k/v, step {len(seen)}")
        got = {name: getattr(cache, name)[0].cpu().numpy() for name in ("k", "v", "k_scale", "v_scale")}
        if not held:
            held.update({name: np.zeros_like(a) for name, a in got.items()})
        rows = qkv.reshape(n, -1, dim)
        b = tuple(t.cpu().numpy() for t in (batch.table, batch.kv_len, batch.row_off))
        K.append(held, rows[:, heads:heads + kv_heads], rows[:, heads + kv_heads:], b)
        everything = (b[0], b[1], np.concatenate([[0], np.cumsum(b[1])]))
        for mine, theirs in zip(K.read(got, everything), K.read(held, everything)):
            np.testing.assert_array_equal(mine, theirs)
        ref, bound = K.attention(held, rows[:, :heads], b)
        err = np.abs(att.reshape(ref.shape) - ref) - bound
        assert err.max() <= 0, f"attention, step {len(seen)}: {err.max()} over the bound"
        ref = O.linear(att.reshape(n, -1), O.widen_bf16(w[1].w0_bits(0)), ids, _adapters(w[1]), w[1].max_adapters)
        assert_close(out, ref, f"output, step {len(seen)}")
        seen.append(n)

    E.run(requests=requests, prompt=prompt, steps=4, hidden=256, heads=heads, kv_heads=kv_heads, dim=dim, block=block,
          ranks={0: 4, 1: 16}, seed=3, chunk=64, on_step=check)
    assert len(seen) >= 5 and set(seen[-4:]) == {requests}
