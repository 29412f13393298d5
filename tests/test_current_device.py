"""Calls whose tensors are on another device than the current one are refused
before they reach the library (no GPU: the tensors only look like device
tensors, and the library records its calls)."""
import pytest

import lora_serving_mlora_amd as M

torch = pytest.importorskip("torch")

U8, I32, F32 = torch.uint8, torch.int32, torch.float32


class Fake(torch.Tensor):
    """A tensor that says it is on a GPU and has no storage."""

    @staticmethod
    def __new__(cls, shape, dtype=torch.bfloat16, device="cuda:1"):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device=device)

    @classmethod
    def __torch_dispatch__(cls, func, types_, args=(), kwargs=None):
        if func is torch.ops.aten.empty_like.default or func is torch.ops.aten.new_empty.default:
            shape = args[1] if len(args) > 1 else args[0].shape
            return Fake(shape, (kwargs or {}).get("dtype") or args[0].dtype, args[0].device)
        raise AssertionError(f"{func} of a tensor without storage")

    def data_ptr(self):
        return 4096


def run_all(device):
    """Every call that goes by its tensors' device: (name, call)."""
    t = lambda *shape, dtype=torch.bfloat16: Fake(shape, dtype, device)
    work = t(4096, dtype=U8)
    cache = M.KVCache(1, 8, 2, 64, 16, storage=(t(1, 8, 2, 16, 64, dtype=U8), t(1, 8, 2, 1, 64, 16, dtype=U8),
                                                t(1, 8, 2, dtype=F32), t(1, 8, 2, dtype=F32)))
    batch = M.KVBatch(t(2, 4, dtype=I32), t(2, dtype=I32), t(3, dtype=I32), 2)
    w4 = M.Q4Weight(t(5, 32, dtype=U8), t(5, 2, dtype=U8))

    class Pool:
        din, dout, handle, meta = 64, 5, 1, t(256, dtype=U8)

    class Rotary:
        dim, _ref, device_index = 64, 4096, w4.device_index
    q, k = t(2, 4, 64), t(2, 2, 64)
    return {
        "mlora_kv_append": lambda: M.kv_append(cache, 0, k, k, batch),
        "mlora_kv_attention": lambda: M.kv_attention(cache, 0, q, batch, work=work, out=t(2, 4, 64)),
        "mlora_q4_quantize": lambda: M.q4_quantize(t(5, 64)),
        "mlora_q4_dequantize": lambda: M.q4_dequantize(w4, t(5, 64)),
        "mlora_q4_gemm": lambda: M.q4_gemm(t(3, 64), w4, Y=t(3, 5), work=work),
        "mlora_q4_apply": lambda: M.q4_apply(Pool, 0, t(3, 64), w4, t(64, dtype=I32), Y=t(3, 5), work=work),
        "mlora_qk_norm_rotary": lambda: M.qk_norm_rotary(q, k, batch, Rotary, q_out=q, k_out=k),
        "mlora_sample": lambda: M.sample(t(2, 9), t(2, dtype=F32), out=t(2, dtype=I32), work=work),
    }


@pytest.fixture
def calls(monkeypatch):
    """(name, stream) of the launching entries that were called, with device 0
    the current one and 100 + d the stream of device d."""
    seen = []

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                seen.append((name, args[-1]))
                return M.OK
            return call

        def mlora_segments_bytes(self, n):
            return 256

        def mlora_kv_work_bytes(self, *args):
            return 4096
    monkeypatch.setattr(M, "lib", lambda: Lib())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 100 + device)
    return seen


@pytest.mark.parametrize("name", sorted(run_all("cuda:1")))
def test_another_device(calls, name):
    with pytest.raises(ValueError, match="current device"):
        run_all("cuda:1")[name]()
    assert calls == []
    run_all("cuda:0")[name]()
    assert calls == [(name, 100)]
