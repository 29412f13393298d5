"""Refusals of the key/value cache's C entries (no GPU): every one returns
before it touches the device."""
import ctypes
import os

import pytest

import lora_serving_mlora_amd as M


def _descs(**kw):
    if not os.path.exists(M.LIB_PATH):
        pytest.skip("libmlora.so not built")
    c = M._KVCacheDesc(1, 2, 64, 16, 8, 4096, 4096, 4096, 4096)
    b = M._KVBatchDesc(4096, 4096, 4096, 2, 4, 4, 2, 1)
    for k, v in kw.items():
        setattr(c if hasattr(c, k) else b, k, v)
    return ctypes.byref(c), ctypes.byref(b)


BAD = [dict(n_layers=0), dict(kv_heads=0), dict(kv_heads=1025), dict(dim=8), dict(dim=40), dict(dim=272), dict(block=8),
       dict(block=48), dict(block=512), dict(n_blocks=0), dict(n_blocks=1 << 31), dict(k=None), dict(v=4097),
       dict(k_scale=None), dict(n_seq=-1), dict(n_seq=0), dict(n_rows=-1), dict(width=0), dict(table_stride=3),
       dict(max_new=0), dict(max_new=3), dict(n_rows=3, max_new=1), dict(table=None), dict(kv_len=None),
       dict(row_off=None), dict(width=1 << 27, table_stride=1 << 27)]


@pytest.mark.parametrize("kw", BAD, ids=str)
def test_bad_descriptors(kw):
    c, b = _descs(**kw)
    L = M.lib()
    assert L.mlora_kv_append(c, 0, 4096, 4096, 128, 64, b, None) == M.EINVAL
    assert L.mlora_last_error() != b""
    assert L.mlora_kv_read(c, 0, b, 4096, 4096, None) == M.EINVAL
    assert L.mlora_kv_attention(c, 0, 4096, 128, 64, 2, b, 1, 0, 0.125, 4096, 4096, 1 << 40, None) == M.EINVAL
    assert L.mlora_kv_work_bytes(c, b, 2) == 0


def test_bad_arguments():
    c, b = _descs()
    L = M.lib()
    assert L.mlora_kv_append(None, 0, 4096, 4096, 128, 64, b, None) == M.EINVAL
    assert L.mlora_kv_append(c, 0, 4096, 4096, 128, 64, None, None) == M.EINVAL
    assert L.mlora_kv_append(c, 1, 4096, 4096, 128, 64, b, None) == M.EINVAL
    assert L.mlora_kv_append(c, -1, 4096, 4096, 128, 64, b, None) == M.EINVAL
    assert L.mlora_kv_append(c, 0, None, 4096, 128, 64, b, None) == M.EINVAL
    assert L.mlora_kv_append(c, 0, 4096, 4096, -1, 64, b, None) == M.EINVAL
    assert L.mlora_kv_read(c, 0, b, 4096, None, None) == M.EINVAL
    assert L.mlora_kv_read(c, 0, b, 4096, 4098, None) == M.EINVAL

    def attend(layer=0, q=4096, rs=128, hs=64, heads=2, causal=1, window=0, scale=0.125, out=4096, work=4096,
               size=1 << 40):
        return L.mlora_kv_attention(c, layer, q, rs, hs, heads, b, causal, window, scale, out, work, size, None)
    for kw in (dict(layer=1), dict(q=None), dict(rs=-1), dict(hs=1 << 31), dict(heads=0), dict(heads=1), dict(heads=3),
               dict(heads=2048), dict(window=-1), dict(causal=0, window=5), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("inf")), dict(scale=float("nan")), dict(out=None), dict(out=4104), dict(work=4097)):
        assert attend(**kw) == M.EINVAL, kw
    assert L.mlora_kv_work_bytes(c, b, 3) == 0


def test_nothing_to_do():
    c, b = _descs(n_rows=0, max_new=0)
    L = M.lib()
    assert L.mlora_kv_append(c, 0, None, None, 128, 64, b, None) == M.OK
    assert L.mlora_kv_read(c, 0, b, None, None, None) == M.OK
    assert L.mlora_kv_attention(c, 0, None, 128, 64, 2, b, 1, 0, 0.125, None, None, 0, None) == M.OK


def test_rows_past_what_the_kernels_count():
    """2^24 rows of 32 query heads to a key/value head: refused, not wrapped."""
    L = M.lib()
    for rows, heads in ((1 << 24, 64), ((1 << 23) + 1, 64)):
        c, b = _descs(n_rows=rows, max_new=rows)
        assert L.mlora_kv_attention(c, 0, 4096, 128, 64, heads, b, 1, 0, 0.125, 4096, 4096, 1 << 60, None) == M.EINVAL
        assert b"2^28" in L.mlora_last_error()
