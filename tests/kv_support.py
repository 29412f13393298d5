"""Caches and batches of the key/value tests: the same content for the oracle
(numpy) and the device, from a numpy generator."""
import numpy as np

from gpu_support import torch_cuda
from oracle import kv_oracle as K


def bf16(x):
    """float64 -> the nearest bf16 values (float64)."""
    torch = torch_cuda()
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).double().numpy()


def dev_rows(x, pad=0, offset=0):
    """bf16 CUDA rows of a float64 [n][heads][dim] array; pad channels between
    heads and an offset (in elements) make them strided and unaligned."""
    torch = torch_cuda()
    n, h, d = x.shape
    buf = torch.full((n * h * (d + pad) + offset,), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = buf[offset:].view(n, h, d + pad)[:, :, :d]
    view.copy_(torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16))
    return view


class Case:
    """new[i] new rows of sequence i, total[i] tokens with them; pages in
    random order, a few more than needed.  Unwritten codes and scales hold
    NaN, so nothing outside the sequences may be used."""

    def __init__(self, seed, new, total, heads=2, dim=64, block=16, layers=1, extra=3, width=None, spread=1.0):
        torch = torch_cuda()
        import lora_serving_mlora_amd as M
        rng = self.rng = np.random.default_rng(seed)
        self.heads, self.dim, self.block = heads, dim, block
        pages = [-(-n // block) if n > 0 else 0 for n in total]
        nb = sum(pages) + extra
        ids = rng.permutation(nb).astype(np.int32)
        width = width or max(max(pages), 1)
        table = np.full((len(new), width), -1, np.int32)
        at = 0
        for i, p in enumerate(pages):
            table[i, :p] = ids[at:at + p]
            at += p
        self.table = table
        self.kv_len = np.array(total, np.int32)
        self.row_off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.n_rows = int(self.row_off[-1])
        self.cache = dict(k=np.full((nb, heads, block, dim), 0x7f, np.uint8),
                          v=np.full((nb, heads, block // 16, dim, 16), 0xff, np.uint8),
                          k_scale=np.full((nb, heads), np.nan, np.float32),
                          v_scale=np.full((nb, heads), np.nan, np.float32))
        size = np.exp(0.4 * rng.normal(size=(1, heads, dim))) * spread
        row = lambda n: bf16(rng.normal(size=(n, heads, dim)) * size * np.exp2(0.7 * rng.normal(size=(n, heads, 1))))
        # what is cached before the new rows
        old = [max(n - m, 0) for m, n in zip(new, total)]
        ob = (table, np.array(old, np.int32), np.concatenate([[0], np.cumsum(old)]).astype(np.int32))
        K.append(self.cache, row(sum(old)), row(sum(old)), ob)
        self.row = row
        self.M = M
        dev = {n: torch.from_numpy(a.copy()).cuda() for n, a in self.cache.items()}
        other = lambda t: torch.full_like(t, 0x7f if t.dtype == torch.uint8 else float("nan"))
        stack = lambda t: torch.stack([other(t)] * (layers - 1) + [t])
        self.layer = layers - 1
        self.dev = M.KVCache(layers, nb, heads, dim, block,
                             storage=tuple(stack(dev[n]) for n in ("k", "v", "k_scale", "v_scale")))
        self.max_new = max(max(new), 1) if self.n_rows else 0

    @property
    def batch(self):
        return self.table, self.kv_len, self.row_off

    def dev_batch(self, max_new=None):
        torch = torch_cuda()
        t = [torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda() for a in self.batch]
        return self.M.KVBatch(*t, self.n_rows, max_new=self.max_new if max_new is None else max_new)

    def pages_equal(self):
        """The device's codes and scales against the oracle's, at the tokens
        that sequences hold."""
        one_nan = lambda a: np.where((a & 0x7f) == 0x7f, 0x7f, a) if a.dtype == np.uint8 else a  # either sign is NaN
        got = {n: one_nan(getattr(self.dev, n)[self.layer].cpu().numpy()) for n in self.cache}
        ref = {n: one_nan(a) for n, a in self.cache.items()}
        for i, n in enumerate(self.kv_len):
            for t in range(int(n)):
                page, s = K.page_of(self.cache, self.batch, i, t), t % self.block
                if page < 0:
                    continue
                for name in ("k_scale", "v_scale"):
                    if not np.array_equal(got[name][page], ref[name][page]):
                        return f"{name} of page {page}: {got[name][page]} != {ref[name][page]}"
                if not np.array_equal(got["k"][page, :, s], ref["k"][page, :, s]):
                    return f"keys of sequence {i}, token {t}"
                if not np.array_equal(got["v"][page, :, s // 16, :, s % 16], ref["v"][page, :, s // 16, :, s % 16]):
                    return f"values of sequence {i}, token {t}"
        return ""
