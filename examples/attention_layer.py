"""One attention layer of a multi-LoRA server: the joint q/k/v projection with
each row's own adapter, the new keys and values into the paged 8-bit cache,
attention over it, and the output projection.

    python examples/attention_layer.py [--requests 32] [--prompt 300] [--steps 64] [--four-bit]

With --four-bit the projections' weights are in 4 bits, the heads of q and k
are normed and rotated before the cache takes them, and each request's next
token is sampled from an output head of 32000 words, in 4 bits as well.

Prompts of different lengths are taken in first, in ragged batches; then every
request decodes one token a step from a HIP graph that is captured once: the
lengths advance on the device, so a replay needs nothing from the host.
"""
import argparse
import os
import sys
import time

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import lora_serving_mlora_amd as M  # noqa: E402
import synth  # noqa: E402


def _dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


class AttentionLayer:
    """Weights and adapters of the two projections (seeded, synthetic)."""

    def __init__(self, seed, hidden, heads, kv_heads, dim, ranks):
        self.hidden, self.heads, self.kv_heads, self.dim = hidden, heads, kv_heads, dim
        n_ad = max(ranks) + 1
        self.workloads, self.pools, self.W0 = [], [], []
        for i, (din, dout) in enumerate(((hidden, (heads + 2 * kv_heads) * dim), (heads * dim, hidden))):
            w = synth.custom(f"attention{i}", seed + i, din, dout, np.zeros(1, np.int32), ranks, max_adapters=n_ad)
            pool = M.Pool(din, dout, 1, n_ad, max(ranks.values()), sum(ranks.values()))
            for a in w.adapter_ids():
                pool.load(a, w.ranks[a], w.scales[a], w.down_all_bits(a), w.up_all_bits(a))
            self.workloads.append(w)
            self.pools.append(pool)
            self.W0.append(_dev(w.w0_bits(0)))

    def scratch(self, cache, batch):
        """Work buffers of a batch of this size: the projections', the attention's."""
        return ([M.new_work(p, batch.n_rows) for p in self.pools], M.new_kv_work(cache, batch, self.heads))

    def __call__(self, X, row_adapter, cache, layer, batch, scratch, window=0):
        """Returns (output, attention's output, q/k/v), bf16 [n_rows][...]."""
        n, (proj_work, kv_work) = batch.n_rows, scratch
        qkv, seg = M.forward(self.pools[0], 0, X, self.W0[0], row_adapter, work=proj_work[0])
        q, k, v = qkv.view(n, -1, self.dim).split((self.heads, self.kv_heads, self.kv_heads), dim=1)
        M.kv_append(cache, layer, k, v, batch)
        att = M.kv_attention(cache, layer, q, batch, window=window, work=kv_work)
        # the rows' adapters are the same: the segments serve again
        out = M.apply(self.pools[1], 0, att.view(n, -1), self.W0[1], seg, work=proj_work[1])
        return out, att, qkv

    def close(self):
        for p in self.pools:
            p.close()


class StepLayer(AttentionLayer):
    """The layer with its weights in 4 bits, norms and a rotation of the heads,
    and behind it an output head whose logits the next tokens are drawn from."""

    def __init__(self, seed, hidden, heads, kv_heads, dim, ranks, vocab, requests):
        super().__init__(seed, hidden, heads, kv_heads, dim, ranks)
        self.W0 = [M.q4_quantize(W) for W in self.W0]
        rng = np.random.default_rng(seed)
        part = lambda *shape: torch.from_numpy(rng.normal(size=shape).astype(np.float32)).to(torch.bfloat16).cuda()
        self.head = M.q4_quantize(part(vocab, hidden) * (2.0 / hidden ** 0.5))
        self.norms = [1 + part(dim) / 8 for _ in range(2)]
        self.rotary = M.Rotary(dim, base=500000.0)
        # each request's own temperature and top-p; the first takes the likeliest token
        self.temperature = torch.linspace(0.0, 1.2, requests, device="cuda")
        self.top_p = torch.full((requests,), 0.9, device="cuda")

    def scratch(self, cache, batch):
        requests = len(self.top_p)
        return ([M.new_q4_work(W, batch.n_rows, p) for W, p in zip(self.W0, self.pools)],
                M.new_kv_work(cache, batch, self.heads), M.new_q4_work(self.head, requests),
                M.new_sample_work(requests, self.head.dout))

    def __call__(self, X, row_adapter, cache, layer, batch, scratch, window=0):
        """As above, with the normed and rotated q and k, and of each request's
        last row the logits, the random numbers and the tokens."""
        n, (proj_work, kv_work, head_work, sample_work) = batch.n_rows, scratch
        seg = M.build_segments(self.pools[0], row_adapter)
        qkv = M.q4_apply(self.pools[0], 0, X, self.W0[0], seg, work=proj_work[0])
        q, k, v = qkv.view(n, -1, self.dim).split((self.heads, self.kv_heads, self.kv_heads), dim=1)
        q, k = M.qk_norm_rotary(q, k, batch, self.rotary, *self.norms)
        M.kv_append(cache, layer, k, v, batch)
        att = M.kv_attention(cache, layer, q, batch, window=window, work=kv_work)
        out = M.q4_apply(self.pools[1], 0, att.view(n, -1), self.W0[1], seg, work=proj_work[1])
        # (a request without a row in this batch takes another's; its token is not used)
        last = out.index_select(0, (batch.row_off[1:] - 1).clamp_(min=0))
        logits = M.q4_gemm(last, self.head, work=head_work)
        u = torch.rand_like(self.top_p)
        tokens = M.sample(logits, u, temperature=self.temperature, top_p=self.top_p, work=sample_work)
        return out, att, qkv, q, k, logits, u, tokens


def make_table(lengths, block, n_blocks, rng):
    """Pages for `lengths` tokens of each sequence, in any order; -1 past them."""
    pages = [-(-n // block) for n in lengths]
    ids = rng.permutation(n_blocks)[:sum(pages)].astype(np.int32)
    table = np.full((len(lengths), max(pages)), -1, np.int32)
    at = 0
    for i, p in enumerate(pages):
        table[i, :p] = ids[at:at + p]
        at += p
    return table


def prompt_batches(lens, limit):
    """Rows of each sequence in batches of at most `limit` rows together."""
    left = np.array(lens)
    while left.any():
        before = np.concatenate([[0], np.cumsum(left)[:-1]])
        new = np.clip(limit - before, 0, left)
        yield new
        left = left - new


def run(requests=32, prompt=300, steps=64, hidden=4096, heads=32, kv_heads=8, dim=128, block=16, ranks=None, seed=1,
        chunk=8192, on_step=None, vocab=0):
    """Prompts, then `steps` decoded tokens a request; microseconds of a decode
    step.  With `vocab` the layer in 4 bits, with tokens sampled from so many
    words.  on_step(layer, X, ids, cache, batch, results) sees every step."""
    ranks = ranks or {0: 16, 1: 8, 2: 64}
    rng = np.random.default_rng(seed)
    if vocab:
        layer = StepLayer(seed, hidden, heads, kv_heads, dim, ranks, vocab, requests)
    else:
        layer = AttentionLayer(seed, hidden, heads, kv_heads, dim, ranks)
    lens = rng.integers(max(1, prompt // 4), prompt + 1, size=requests)
    adapter = rng.integers(-1, max(ranks) + 1, size=requests).astype(np.int32)
    need = sum(-(-(int(n) + steps) // block) for n in lens)
    cache = M.KVCache(1, need + 8, kv_heads, dim, block)
    table = torch.from_numpy(make_table([int(n) + steps for n in lens], block, need + 8, rng)).cuda()
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()

    # the prompts, ragged rows of some sequences at a time; the others idle
    kv_len = torch.zeros(requests, dtype=torch.int32, device="cuda")
    for new in prompt_batches(lens, chunk):
        kv_len.add_(dev(new))
        off = np.concatenate([[0], np.cumsum(new)])
        batch = M.KVBatch(table, kv_len, dev(off), int(off[-1]), max_new=int(new.max()))
        X = torch.randn(batch.n_rows, hidden, device="cuda").to(torch.bfloat16)
        ids = dev(np.repeat(adapter, new))
        results = layer(X, ids, cache, 0, batch, layer.scratch(cache, batch))
        if on_step:
            on_step(layer, X, ids, cache, batch, results)

    # one token a request and step
    batch = M.KVBatch(table, kv_len, dev(np.arange(requests + 1)), requests, max_new=1)
    X, ids = torch.randn(requests, hidden, device="cuda").to(torch.bfloat16), dev(adapter)
    scratch = layer.scratch(cache, batch)

    def step():
        kv_len.add_(1)
        return layer(X, ids, cache, 0, batch, scratch)

    results = step()  # outside the graph first
    if on_step:
        on_step(layer, X, ids, cache, batch, results)
    if steps == 1:
        layer.close()
        return None
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        results = step()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(steps - 1):
        graph.replay()
        if on_step:
            on_step(layer, X, ids, cache, batch, results)
    torch.cuda.synchronize()
    us = (time.perf_counter() - t0) / (steps - 1) * 1e6
    layer.close()
    return us


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--requests", type=int, default=32)
    p.add_argument("--prompt", type=int, default=300, help="longest prompt; the shortest is a quarter of it")
    p.add_argument("--steps", type=int, default=64, help="tokens decoded by each request")
    p.add_argument("--four-bit", action="store_true",
                   help="weights in 4 bits, normed and rotated heads, the next token sampled")
    a = p.parse_args()
    us = run(a.requests, a.prompt, a.steps, vocab=32000 if a.four_bit else 0)
    if us is not None:
        print(f"{a.requests} requests, prompts up to {a.prompt} tokens: {us:.1f} us a decode step of one layer, "
              f"{a.requests / us * 1e6:.0f} tokens/s")


if __name__ == "__main__":
    main()
