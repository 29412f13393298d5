"""What the key/value cache's Python calls refuse before they reach the library
(no GPU: the tensors only look like device tensors, and the library records
its calls)."""
import types

import pytest

import lora_serving_mlora_amd as M

torch = pytest.importorskip("torch")


class Fake(torch.Tensor):
    """A tensor that says it is on a GPU and has no storage."""

    @staticmethod
    def __new__(cls, shape, dtype=torch.bfloat16, device="cuda:0", strides=None):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device=device, strides=strides)

    @classmethod
    def __torch_dispatch__(cls, func, types_, args=(), kwargs=None):
        raise AssertionError(f"{func} of a tensor without storage")

    def data_ptr(self):
        return 4096


@pytest.fixture
def calls(monkeypatch):
    """The names of the launching entries that were called."""
    seen = []

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                seen.append(name)
                return M.OK
            return call

        def mlora_kv_work_bytes(self, *args):
            return 4096
    monkeypatch.setattr(M, "lib", lambda: Lib())
    monkeypatch.setattr(M, "_kv_stream", lambda cache: 0)
    return seen


def _cache(device="cuda:0", other=None):
    shapes = ((1, 8, 2, 16, 64), (1, 8, 2, 1, 64, 16), (1, 8, 2), (1, 8, 2))
    kinds = (torch.uint8, torch.uint8, torch.float32, torch.float32)
    st = [Fake(s, t, device) for s, t in zip(shapes, kinds)]
    if other:
        st[2] = Fake(shapes[2], kinds[2], other)
    return M.KVCache(1, 8, 2, 64, 16, storage=tuple(st))


def _batch(device="cuda:0", kv_len=None):
    ints = lambda shape, d=device: Fake(shape, torch.int32, d)
    return M.KVBatch(ints((2, 4)), ints((2,), kv_len or device), ints((3,)), 2)


def _rows(heads=2, device="cuda:0", **kw):
    return Fake((2, heads, 64), device=device, **kw)


def test_the_calls_as_they_are_meant(calls):
    c, b = _cache(), _batch()
    M.kv_append(c, 0, _rows(), _rows(), b)
    M.kv_attention(c, 0, _rows(4), b, work=Fake((4096,), torch.uint8), out=_rows(4))
    assert calls == ["mlora_kv_append", "mlora_kv_attention"]


WORK = {
    "on the host": lambda: torch.empty(4096, dtype=torch.uint8),
    "on another device": lambda: Fake((4096,), torch.uint8, "cuda:1"),
    "every other byte": lambda: Fake((4096,), torch.uint8, strides=(2,)),
    "not a tensor": lambda: types.SimpleNamespace(data_ptr=lambda: 4096, nbytes=4096),
}


@pytest.mark.parametrize("what", sorted(WORK))
def test_a_work_buffer_that_the_kernels_could_not_use(calls, what):
    with pytest.raises((TypeError, ValueError)):
        M.kv_attention(_cache(), 0, _rows(4), _batch(), work=WORK[what](), out=_rows(4))
    assert calls == []


def test_tensors_that_are_not_where_the_cache_is(calls):
    c, b, far = _cache(), _batch(), "cuda:1"
    work = Fake((4096,), torch.uint8)
    for call in (lambda: M.kv_append(c, 0, _rows(device=far), _rows(device=far), b),
                 lambda: M.kv_append(c, 0, _rows(), _rows(device=far), b),
                 lambda: M.kv_append(c, 0, _rows(), _rows(), _batch(far)),
                 lambda: M.kv_read(c, 0, _batch(far)),
                 lambda: M.kv_attention(c, 0, _rows(4, far), b, work=work, out=_rows(4)),
                 lambda: M.kv_attention(c, 0, _rows(4), b, work=work, out=_rows(4, far)),
                 lambda: M.kv_attention(c, 0, _rows(4), _batch(far), work=work, out=_rows(4)),
                 lambda: _cache(other=far), lambda: _batch(kv_len=far)):
        with pytest.raises((TypeError, ValueError)):
            call()
    assert calls == []
