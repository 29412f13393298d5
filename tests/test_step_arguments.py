"""Refusals of the entries for 4-bit weights, norms and rotation, and sampling
(no GPU): the C entries return, and the Python calls raise, before anything
touches the device."""
import ctypes
import os

import pytest

import lora_serving_mlora_amd as M

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(M.LIB_PATH):
        pytest.skip("libmlora.so not built")
    return M.lib()


def _w(codes=4096, scales=4097, din=64, dout=5):
    return ctypes.byref(M._Q4Desc(codes, scales, din, dout))


BAD_W = [dict(codes=None), dict(codes=4104), dict(scales=None), dict(din=0), dict(din=48), dict(din=(1 << 20) + 32),
         dict(dout=0), dict(dout=(1 << 24) + 1), dict(din=-32)]


@pytest.mark.parametrize("kw", BAD_W, ids=str)
def test_bad_weights(L, kw):
    assert L.mlora_q4_gemm(_w(**kw), 4096, 4096, 1, 4096, 1 << 40, None) == M.EINVAL
    assert L.mlora_last_error() != b""
    assert L.mlora_q4_dequantize(_w(**kw), 4096, None) == M.EINVAL
    assert L.mlora_q4_work_bytes(_w(**kw), None, 100) == 0


def test_q4_arguments(L):
    gemm = lambda w=None, x=4096, y=4096, n=1, work=4096, size=1 << 40: L.mlora_q4_gemm(w or _w(), x, y, n, work, size, None)
    assert L.mlora_q4_gemm(None, 4096, 4096, 1, 4096, 1 << 40, None) == M.EINVAL
    for kw in (dict(x=None), dict(x=4104), dict(y=None), dict(n=-1), dict(n=16385), dict(n=100, work=None),
               dict(n=100, size=64), dict(n=100, work=4100)):
        assert gemm(**kw) == M.EINVAL, kw
    assert gemm(n=0, x=None, y=None, work=None) == M.OK
    need = L.mlora_q4_work_bytes(_w(), None, 100)
    assert need >= 5 * 64 * 2  # the weight as bf16
    assert L.mlora_q4_work_bytes(_w(), None, 0) == 0 and L.mlora_q4_work_bytes(_w(), None, -1) == 0
    assert L.mlora_q4_apply(None, 0, 4096, _w(), 4096, 4096, 1, 4096, 1 << 40, None) == M.EINVAL
    for w, dout, din, codes, scales in ((None, 5, 64, 4096, 4096), (4104, 5, 64, 4096, 4096), (4096, 0, 64, 4096, 4096),
                                        (4096, 5, 40, 4096, 4096), (4096, 5, 64, None, 4096), (4096, 5, 64, 4104, 4096),
                                        (4096, 5, 64, 4096, None)):
        assert L.mlora_q4_quantize(w, dout, din, codes, scales, None) == M.EINVAL
    assert L.mlora_q4_dequantize(_w(), None, None) == M.EINVAL
    assert L.mlora_q4_dequantize(_w(), 4104, None) == M.EINVAL


P = 1 << 20  # an address


def _rotate(L, q=None, k=None, dim=64, rot=64, freq=P, factor=1.0, eps=1e-6, n_rows=3, n_seq=2, kv_len=P, row_off=P,
            none=()):
    sides = []
    for s in (q, k):
        d = dict(x=P, y=P, row_stride=512, head_stride=64, out_row_stride=512, out_head_stride=64, weight=None, heads=4)
        d.update(s or {})
        sides.append(M._head_rows(*(v or 0 for v in d.values())))
    if k is None:
        sides[1] = None
    b = M._KVBatchDesc(None, kv_len, row_off, n_seq, 0, 0, n_rows, 0)
    r = M._RotaryDesc(freq, rot, 0, factor)
    args = [ctypes.byref(b), dim, ctypes.byref(r), sides[0], sides[1], eps, None]
    for i in none:
        args[i] = None
    return L.mlora_qk_norm_rotary(*args)


BAD_R = [dict(none=(0,)), dict(none=(2,)), dict(none=(3,)), dict(dim=0), dict(dim=24), dict(dim=272), dict(rot=0),
         dict(rot=4), dict(rot=12), dict(rot=72), dict(freq=None), dict(freq=P + 4), dict(factor=float("nan")),
         dict(factor=float("inf")), dict(eps=-1.0), dict(eps=float("nan")), dict(n_rows=-1), dict(n_rows=(1 << 24) + 1),
         dict(n_seq=0), dict(n_seq=-1), dict(n_seq=(1 << 20) + 1), dict(kv_len=None), dict(row_off=None),
         dict(q=dict(heads=0)), dict(q=dict(heads=1025)), dict(q=dict(x=None)), dict(q=dict(y=None)),
         dict(q=dict(row_stride=-1)), dict(q=dict(head_stride=1 << 31)),
         dict(q=dict(y=2 * P, out_head_stride=32)), dict(q=dict(y=2 * P, out_row_stride=255)),
         dict(q=dict(y=P + 128)), dict(q=dict(out_row_stride=256)), dict(q=dict(y=P + 2)),
         # the keys' output over the queries' input, over the queries' output, the same rows for both
         dict(q=dict(y=2 * P), k=dict(x=3 * P, y=P)), dict(q=dict(y=2 * P), k=dict(x=3 * P, y=2 * P)), dict(k=dict()),
         dict(k=dict(x=P + 256, y=P + 256)), dict(k=dict(x=P + 514, y=P + 514, row_stride=512))]


@pytest.mark.parametrize("kw", BAD_R, ids=str)
def test_bad_rotations(L, kw):
    assert _rotate(L, **kw) == M.EINVAL
    assert L.mlora_last_error() != b""


def test_rotation_of_nothing(L):
    assert _rotate(L, n_rows=0, n_seq=0, kv_len=None, row_off=None, q=dict(x=None, y=None)) == M.OK


def _sample(L, logits=4096, f32=1, stride=100, n=2, vocab=100, u=4096, out=4096, work=4096, size=1 << 40):
    return L.mlora_sample(logits, f32, stride, n, vocab, u, None, None, None, None, out, work, size, None)


def test_sample_arguments(L):
    for kw in (dict(logits=None), dict(logits=4098), dict(logits=4097, f32=0), dict(stride=-1), dict(stride=1 << 31),
               dict(n=-1), dict(n=16385), dict(vocab=0), dict(vocab=(1 << 20) + 1), dict(u=None), dict(out=None),
               dict(work=4100)):
        assert _sample(L, **kw) == M.EINVAL, kw
        assert L.mlora_last_error() != b""
    assert _sample(L, n=0, logits=None, u=None, out=None, work=None) == M.OK
    need = L.mlora_sample_work_bytes(2, 100)
    if need:
        assert _sample(L, size=need - 1) == M.EINVAL and _sample(L, work=None) == M.EINVAL
    assert L.mlora_sample_work_bytes(-1, 100) == 0 and L.mlora_sample_work_bytes(1, 0) == 0


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

        def mlora_segments_bytes(self, n):
            return 256
    monkeypatch.setattr(M, "lib", lambda: Lib())
    monkeypatch.setattr(M, "_raw_stream", lambda device: 0)
    return seen


class FakePool:
    din, dout, handle = 64, 5, 1

    def __init__(self, device="cuda:0"):
        self.meta = Fake((256,), torch.uint8, device)


def _q4(device="cuda:0"):
    return M.Q4Weight(Fake((5, 32), torch.uint8, device), Fake((5, 2), torch.uint8, device))


class FakeRotary:
    dim, _ref, device_index = 64, 4096, 0


def _batch(device="cuda:0"):
    ints = lambda shape: Fake(shape, torch.int32, device)
    return M.KVBatch(ints((2, 4)), ints((2,)), ints((3,)), 2)


U8, I32, F32, FAR = torch.uint8, torch.int32, torch.float32, "cuda:1"


def test_the_calls_as_they_are_meant(calls):
    work = Fake((4096,), U8)
    M.q4_gemm(Fake((3, 64)), _q4(), Y=Fake((3, 5)), work=work)
    M.q4_apply(FakePool(), 0, Fake((3, 64)), _q4(), Fake((64,), I32), Y=Fake((3, 5)), work=work)
    M.qk_norm_rotary(Fake((2, 4, 64)), Fake((2, 1, 64)), _batch(), FakeRotary(), q_weight=Fake((64,)),
                     q_out=Fake((2, 4, 64)), k_out=Fake((2, 1, 64)))
    M.sample(Fake((2, 9), F32), Fake((2,), F32), top_k=Fake((2,), I32), out=Fake((2,), I32), work=work)
    assert calls == ["mlora_q4_gemm", "mlora_q4_apply", "mlora_qk_norm_rotary", "mlora_sample"]


def _bad_calls():
    work, far = Fake((4096,), U8), Fake((4096,), U8, FAR)
    x, y, seg = Fake((3, 64)), Fake((3, 5)), Fake((64,), I32)
    q, k, rot = Fake((2, 4, 64)), Fake((2, 1, 64)), FakeRotary()
    lg, u, out = Fake((2, 9), F32), Fake((2,), F32), Fake((2,), I32)
    rotate = lambda q=q, k=k, b=None, **kw: M.qk_norm_rotary(q, k, b or _batch(), rot, q_out=kw.pop("q_out", q),
                                                             k_out=kw.pop("k_out", k), **kw)
    pick = lambda lg=lg, u=u, **kw: M.sample(lg, u, out=kw.pop("out", out), work=kw.pop("work", work), **kw)
    return {
        "codes of floats": lambda: M.Q4Weight(Fake((5, 32)), Fake((5, 2), U8)),
        "scales of another shape": lambda: M.Q4Weight(Fake((5, 32), U8), Fake((5, 3), U8)),
        "din not whole groups": lambda: M.Q4Weight(Fake((5, 24), U8), Fake((5, 1), U8)),
        "scales elsewhere": lambda: M.Q4Weight(Fake((5, 32), U8), Fake((5, 2), U8, FAR)),
        "weight of a vector": lambda: M.q4_quantize(Fake((64,))),
        "weight not whole groups": lambda: M.q4_quantize(Fake((5, 48))),
        "weight in fp32": lambda: M.q4_quantize(Fake((5, 64), F32)),
        "bf16 weight of another shape": lambda: M.q4_dequantize(_q4(), Fake((5, 32))),
        "X of another din": lambda: M.q4_gemm(Fake((3, 96)), _q4(), Y=y, work=work),
        "X in fp32": lambda: M.q4_gemm(Fake((3, 64), F32), _q4(), Y=y, work=work),
        "X elsewhere": lambda: M.q4_gemm(Fake((3, 64), device=FAR), _q4(), Y=y, work=work),
        "X strided": lambda: M.q4_gemm(Fake((3, 64), strides=(128, 1)), _q4(), Y=y, work=work),
        "Y of another shape": lambda: M.q4_gemm(x, _q4(), Y=Fake((3, 6)), work=work),
        "Y elsewhere": lambda: M.q4_gemm(x, _q4(), Y=Fake((3, 5), device=FAR), work=work),
        "work elsewhere": lambda: M.q4_gemm(x, _q4(), Y=y, work=far),
        "work strided": lambda: M.q4_gemm(x, _q4(), Y=y, work=Fake((64,), U8, strides=(2,))),
        "pool elsewhere": lambda: M.q4_apply(FakePool(FAR), 0, x, _q4(), seg, Y=y, work=work),
        "segments too small": lambda: M.q4_apply(FakePool(), 0, x, _q4(), Fake((8,), I32), Y=y, work=work),
        "segments elsewhere": lambda: M.q4_apply(FakePool(), 0, x, _q4(), Fake((64,), I32, FAR), Y=y, work=work),
        "q in fp32": lambda: rotate(q=Fake((2, 4, 64), F32)),
        "q elsewhere": lambda: rotate(q=Fake((2, 4, 64), device=FAR)),
        "q of other rows": lambda: rotate(q=Fake((3, 4, 64))),
        "k of another dim": lambda: rotate(k=Fake((2, 1, 32))),
        "q not dense": lambda: rotate(q=Fake((2, 4, 64), strides=(512, 128, 2))),
        "q_out of another shape": lambda: rotate(q_out=Fake((2, 5, 64))),
        "q_out elsewhere": lambda: rotate(q_out=Fake((2, 4, 64), device=FAR)),
        "weight of another dim": lambda: rotate(q_weight=Fake((32,))),
        "weight elsewhere": lambda: rotate(k_weight=Fake((64,), device=FAR)),
        "batch elsewhere": lambda: rotate(b=_batch(FAR)),
        "a weight without keys": lambda: M.qk_norm_rotary(q, None, _batch(), rot, k_weight=Fake((64,)), q_out=q),
        "logits of ints": lambda: pick(lg=Fake((2, 9), I32)),
        "logits of a vector": lambda: pick(lg=Fake((9,), F32)),
        "logits not dense": lambda: pick(lg=Fake((2, 9), F32, strides=(18, 2))),
        "u in 64 bits": lambda: pick(u=Fake((2,), torch.float64)),
        "u of other rows": lambda: pick(u=Fake((3,), F32)),
        "u elsewhere": lambda: pick(u=Fake((2,), F32, FAR)),
        "top_k in floats": lambda: pick(top_k=Fake((2,), F32)),
        "temperature elsewhere": lambda: pick(temperature=Fake((2,), F32, FAR)),
        "a number for top_p": lambda: pick(top_p=0.9),
        "tokens in 64 bits": lambda: pick(out=Fake((2,), torch.int64)),
        "sampling's work elsewhere": lambda: pick(work=far),
    }


@pytest.mark.parametrize("what", sorted(_bad_calls()))
def test_tensors_that_the_kernels_could_not_use(calls, what):
    with pytest.raises((TypeError, ValueError)):
        _bad_calls()[what]()
    assert calls == []


def test_frequencies():
    for kw in (dict(dim=0), dict(dim=12), dict(dim=16, freqs=[1.0] * 7), dict(dim=16, freqs=[float("inf")] * 8)):
        with pytest.raises(ValueError):
            M.Rotary(**kw)
