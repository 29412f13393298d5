"""The cache oracle against facts worked out by hand (no GPU)."""
import numpy as np
import pytest

from oracle import kv_oracle as K


def _cache(pages=3, heads=1, block=16, dim=16):
    return dict(k=np.zeros((pages, heads, block, dim), np.uint8), v=np.zeros((pages, heads, block // 16, dim, 16), np.uint8),
                k_scale=np.zeros((pages, heads), np.float32), v_scale=np.zeros((pages, heads), np.float32))


def test_codes():
    v = K.code_values()
    assert v[0x7e] == 448 and v[0x01] == 2.0 ** -9 and v[0x38] == 1 and v[0xb8] == -1 and np.isnan(v[0x7f])
    assert (K.to_code(v[:127]) == np.arange(127)).all()
    # halfway between 1 and 1.125 goes to the even code; past 448 saturates
    assert K.to_code(np.array([1.0625, 1.1875, 1e6, -1e6, np.inf])).tolist() == [0x38, 0x3a, 0x7e, 0xfe, 0x7f]
    torch = pytest.importorskip("torch")
    x = np.concatenate([np.random.default_rng(0).normal(size=4000) * 2.0 ** np.random.default_rng(1).integers(-12, 7, 4000)])
    t = torch.tensor(np.clip(x, -448, 448), dtype=torch.float32)
    assert (t.to(torch.float8_e4m3fn).view(torch.uint8).numpy() == K.to_code(t.double().numpy())).all()


def test_scale_is_the_least_that_covers():
    assert K.scale_exp(448.0) == 0 and K.scale_exp(448.5) == 1 and K.scale_exp(224.0) == -1 and K.scale_exp(0.0) == -64
    assert K.scale_exp(1e-30) == -64 and K.scale_exp(3.3e38) == 119


def test_append_keeps_grows_and_starts_afresh():
    c = _cache()
    table = np.array([[2, 0]], np.int32)
    one = lambda x: np.full((1, 1, 16), x)
    K.append(c, one(448.0), one(1.0), (table, np.array([1], np.int32), np.array([0, 1], np.int32)))
    assert c["k_scale"][2, 0] == 1 and (c["k"][2, 0, 0] == 0x7e).all() and (c["v"][2, 0, 0, :, 0] == 0x78).all()
    K.append(c, one(1000.0), one(0.5), (table, np.array([2], np.int32), np.array([0, 1], np.int32)))
    assert c["k_scale"][2, 0] == 4  # 448 -> 112 * 4, 1000 -> 256 * 4 (250 lies nearer to 256 than to 240)
    k, v = K.read(c, (table, np.array([2], np.int32), np.array([0, 2], np.int32)))
    assert (k[:, 0, 0] == [448, 1024]).all() and (v[:, 0, 0] == [1.0, 0.5]).all()
    K.append(c, one(1.0), one(1.0), (table, np.array([1], np.int32), np.array([0, 1], np.int32)))
    assert c["k_scale"][2, 0] == 2.0 ** -8


def test_attention_of_equal_keys_is_the_mean():
    c = _cache()
    table = np.array([[0, 1]], np.int32)
    rng = np.random.default_rng(0)
    x = np.ones((20, 1, 16))
    vals = rng.integers(-8, 9, size=(20, 1, 16)).astype(float)
    b = (table, np.array([20], np.int32), np.array([0, 20], np.int32))
    K.append(c, x, vals, b)
    out, _ = K.attention(c, np.ones((20, 1, 16)), b)
    for j in range(20):
        assert np.allclose(out[j, 0], vals[:j + 1, 0].mean(0))
    out, _ = K.attention(c, np.ones((20, 1, 16)), b, window=3)
    assert np.allclose(out[10, 0], vals[8:11, 0].mean(0)) and np.allclose(out[0, 0], vals[0, 0])
    out, _ = K.attention(c, np.ones((20, 1, 16)), b, causal=False)
    assert np.allclose(out[0, 0], vals[:, 0].mean(0))
