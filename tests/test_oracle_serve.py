"""The 64-bit statement of the serving operators, against facts that do not come from it."""
import numpy as np
import pytest

from oracle import serve


def test_e4m3_values_by_hand():
    # 0x01 = 2^-9, 0x08 = 2^-6 (first normal), 0x38 = 1, 0x7e = 448, 0xb8 = -1
    assert serve.e4m3_value([0x00, 0x01, 0x08, 0x38, 0x7e, 0xb8]).tolist() == [
        0.0, 2.0 ** -9, 2.0 ** -6, 1.0, 448.0, -1.0]
    assert np.isnan(serve.e4m3_value([0x7f, 0xff])).all()


def test_e4m3_rounding_matches_torch_and_saturates():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(0)
    v = (rng.standard_normal(20000) * 2.0 ** rng.integers(-12, 9, 20000)).astype(np.float32)
    v = np.clip(v, -448, 448)
    # all values and all midpoints (ties) too
    v = np.concatenate([v, serve._TABLE, serve._MID, -serve._MID]).astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(serve.e4m3_byte(v), want)
    assert serve.e4m3_byte([449.0, -1e9]).tolist() == [0x7e, 0xfe]
    assert serve.e4m3_byte([np.nan, np.inf]).tolist() == [127, 127]


@pytest.mark.parametrize("bits", [4, 8])
def test_cache_codes_are_the_nearest_grid_points(bits):
    rng = np.random.default_rng(1)
    X = rng.standard_normal((5, 2, 64)).astype(np.float32)
    q = serve.cache_quantize(X, bits, 32)
    s = np.repeat(q["scales"].astype(np.float64), 32, -1).reshape(X.shape)
    z = np.repeat(q["zeros"].astype(np.float64), 32, -1).reshape(X.shape)
    grid = np.arange(2 ** bits)
    best = np.abs((grid - z[..., None]) * s[..., None] - X[..., None].astype(np.float64)).min(-1)
    assert np.abs(np.abs(q["values"] - X) - best).max() <= 1e-6 * s.max()


def test_cache_zero_group_and_symmetric_range():
    q = serve.cache_quantize(np.zeros((1, 8)), 4, 8)
    assert q["values"].max() == 0 and q["scales"][0, 0] == np.float32(2 / 15)
    # -1 .. 1: the zero-point's quotient is 7.5, a tie that goes to 8
    x = np.array([[-1.0, 1.0, 0, 0, 0, 0, 0, 0]])
    assert serve.cache_quantize(x, 4, 8)["zeros"][0, 0] == 8


def test_pack4_by_hand():
    assert serve.pack4(np.array([[1, 2, 15, 0]])).tolist() == [[0x21, 0x0f]]


def test_matmul_is_the_dequantized_product():
    rng = np.random.default_rng(2)
    A, B = rng.standard_normal((3, 300)), rng.standard_normal((130, 300))
    a, sa = serve.fp8_quantize(A, 1)
    b, sb = serve.fp8_quantize(B, 128)
    da = serve.e4m3_value(a) * np.repeat(sa, 128, 1)[:, :300]
    db = serve.e4m3_value(b) * np.repeat(np.repeat(sb, 128, 0)[:130], 128, 1)[:, :300]
    Y, M = serve.fp8_matmul(a, sa, b, sb)
    assert np.allclose(Y, da @ db.T, rtol=1e-12, atol=1e-12) and (M >= np.abs(Y) - 1e-12).all()
