"""The example's layer in 4 bits with normed and rotated heads and sampled
tokens, step by step, eager and from its graph: each stage against 64 bits on
what the stage before it gave.

Tolerances: a projection's as tests/test_gpu_q4.py derives it (at most 64 rows
here, one rounding), the heads' as oracle/step_oracle.py, attention's as its
oracle; the cache and the tokens exactly."""
import os
import sys

import numpy as np
import pytest

import oracle as O
from gpu_support import dev_to_f64, say, torch_cuda
from oracle import kv_oracle as K
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _projection(y, x, w4, what, w=None, ids=None):
    wv = S.q4_values(w4.codes.cpu().numpy(), w4.scales.cpu().numpy())
    ref, mag, rank = x @ wv.T, np.abs(x) @ np.abs(wv).T, 0
    for a in w.adapter_ids() if w else ():
        s, down, up = w.scales[a], O.widen_bf16(w.down_bits(a, 0)), O.widen_bf16(w.up_bits(a, 0))
        rows, rank = ids == a, max(rank, w.ranks[a])
        ref[rows] += s * (x[rows] @ down.T) @ up.T
        mag[rows] += abs(s) * (np.abs(x[rows]) @ np.abs(down).T) @ np.abs(up).T * (1 + w.ranks[a] / x.shape[1])
    err = mag * (2 * x.shape[1] + rank + 8) * 2.0 ** -23
    bad = np.abs(y - ref) - (err + (np.abs(ref) + err) * 2.0 ** -8)
    assert bad.max() <= 0, f"{what}: {bad.max()} over the bound"


@pytest.mark.parametrize("requests,prompt,heads,kv_heads,dim,block,vocab",
                         [(3, 40, 4, 2, 64, 16, 1000), (7, 90, 8, 1, 128, 32, 20011)])
def test_layer(requests, prompt, heads, kv_heads, dim, block, vocab):
    torch = torch_cuda()
    import attention_layer as E
    held, seen, drawn = {}, [], []

    def check(layer, X, ids, cache, batch, results):
        torch.cuda.synchronize()
        out, att, qkv, q, k, logits = (dev_to_f64(r) for r in results[:6])
        u, tokens = (t.cpu().numpy() for t in results[6:])
        ids, n, step = ids.cpu().numpy(), batch.n_rows, len(seen)
        say(f"layer in 4 bits, {n} rows, step {step}")
        w = layer.workloads
        _projection(qkv, dev_to_f64(X), layer.W0[0], f"q/k/v, step {step}", w[0], ids)
        rows = qkv.reshape(n, -1, dim)
        b = tuple(t.cpu().numpy() for t in (batch.table, batch.kv_len, batch.row_off))
        freqs = 500000.0 ** (-2.0 * np.arange(dim // 2) / dim)
        for mine, at, weight in ((q, slice(0, heads), layer.norms[0]), (k, slice(heads, heads + kv_heads), layer.norms[1])):
            ref, bound = S.qk_norm_rotary(rows[:, at], dev_to_f64(weight), 1e-6, b[1:], freqs)
            assert (np.abs(mine - ref) - bound).max() <= 0, f"heads, step {step}"
        got = {name: getattr(cache, name)[0].cpu().numpy() for name in ("k", "v", "k_scale", "v_scale")}
        if not held:
            held.update({name: np.zeros_like(a) for name, a in got.items()})
        K.append(held, k, rows[:, heads + kv_heads:], b)
        everything = (b[0], b[1], np.concatenate([[0], np.cumsum(b[1])]))
        for mine, theirs in zip(K.read(got, everything), K.read(held, everything)):
            np.testing.assert_array_equal(mine, theirs)
        ref, bound = K.attention(held, q, b)
        err = np.abs(att.reshape(ref.shape) - ref) - bound
        assert err.max() <= 0, f"attention, step {step}: {err.max()} over the bound"
        _projection(out, att.reshape(n, -1), layer.W0[1], f"output, step {step}", w[1], ids)
        _projection(logits, out[np.maximum(b[2][1:] - 1, 0)], layer.head, f"logits, step {step}")
        ref = S.sample(logits, u, temperature=layer.temperature.cpu().numpy(), top_p=layer.top_p.cpu().numpy())
        assert np.array_equal(tokens, ref), f"tokens, step {step}"
        seen.append(n)
        drawn.append(u)

    E.run(requests=requests, prompt=prompt, steps=4, hidden=256, heads=heads, kv_heads=kv_heads, dim=dim, block=block,
          ranks={0: 4, 1: 16}, seed=3, chunk=64, on_step=check, vocab=vocab)
    assert len(seen) >= 5 and set(seen[-4:]) == {requests}
    assert not np.array_equal(drawn[-1], drawn[-2]), "replays draw anew"


def test_the_example_runs():
    import attention_layer as E
    say("the example in 4 bits")
    assert E.run(requests=5, prompt=30, steps=3, vocab=32000) > 0
