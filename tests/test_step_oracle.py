"""The oracle of the 4-bit weights, the rotation and the sampler against
values worked out by hand."""
import numpy as np

from oracle import step_oracle as S


def test_codes_and_scales():
    codes = np.array([[0x10, 0x32, 0x54, 0x76, 0x98, 0xba, 0xdc, 0xfe] * 2])  # all 16 codes, twice
    v = S.q4_values(codes.astype(np.uint8), np.array([[128]], np.uint8))
    half = [0, 1, 2, 3, 4, 6, 8, 12]
    assert v[0, :16].tolist() == half + [-x for x in half]
    bad = S.q4_values(np.zeros((1, 32), np.uint8), np.array([[1, 253]], np.uint8))
    assert np.isnan(bad).all()


def test_quantizer():
    w = np.zeros((1, 64))
    w[0, :10] = [6, 0.25, 0.26, 0.75, -1.25, 1.75, 2.5, -3.5, 5, -0.2]
    w[0, 32:35] = [6.1, 0.5, 1.5]  # a scale of 2: 3.05, 0.25, 0.75
    codes, scales = S.q4_quantize(w)
    assert scales.tolist() == [[127, 128]]
    v = S.q4_values(codes, scales)
    assert v[0, :10].tolist() == [6, 0, 0.5, 1, -1, 2, 2, -4, 4, 0]
    assert v[0, 32:35].tolist() == [6, 0, 2]
    zero = S.q4_quantize(np.zeros((1, 32)))
    assert zero[1].tolist() == [[2]] and not zero[0].any()
    assert S.q4_quantize(np.full((1, 32), np.inf))[1].tolist() == [[255]]
    huge = S.q4_quantize(np.full((1, 32), 3e38))
    assert huge[1].tolist() == [[252]] and (S.q4_values(*huge) == 6 * 2.0 ** 125).all()


def test_rotation():
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    batch = (np.array([3]), np.array([0, 1]))  # one row at position 2
    quarter = np.full(2, np.pi / 4)  # half a turn of a right angle a position
    y, _ = S.qk_norm_rotary(x, None, 0.0, batch, quarter)
    np.testing.assert_allclose(y[0, 0], [-3, -4, 1, 2, 5, 6, 7, 8], atol=1e-12)
    y, _ = S.qk_norm_rotary(x, None, 0.0, batch, quarter, interleaved=True)
    np.testing.assert_allclose(y[0, 0], [-2, 1, -4, 3, 5, 6, 7, 8], atol=1e-12)
    y, _ = S.qk_norm_rotary(np.full((1, 1, 8), 3.0), np.full(8, 2.0), 7.0, batch, np.zeros(4))
    np.testing.assert_allclose(y[0, 0], 1.5)  # 2 * 3 / sqrt(9 + 7)


def test_sampler():
    x = np.log(np.array([1.0, 4.0, 2.0, 4.0, 0.5]))  # order: 1, 3, 2, 0, 4; weights 1, 1, 1/2, 1/4, 1/8
    draw = lambda u, **kw: S.sample_row(x, u, **kw)
    total = 2.875
    assert [draw((c - 1e-6) / total) for c in (1, 2, 2.5, 2.75, 2.875)] == [1, 3, 2, 0, 4]
    assert draw(0.99, top_k=2) == 3 and draw(0.99, top_k=1) == 1
    assert draw(0.999, top_p=0.8) == 2  # 2.3 of 2.875: three tokens
    assert draw(0.999, top_p=0.0) == 1
    assert draw(0.999, min_p=0.25) == 0 and draw(0.999, min_p=0.26) == 2
    assert draw(0.999, top_k=3, top_p=0.7) == 3  # 1.75 of 2.5
    assert draw(0.9, temperature=0.0) == 1
    assert draw(0.999, temperature=0.5, min_p=0.2) == 2  # weights 1, 1, 1/4, 1/16
    assert S.sample_row(np.array([np.nan, -np.inf]), 0.5) == -1
    assert S.sample_row(np.array([np.nan, 1.0, np.inf, np.inf]), 0.6) == 3
