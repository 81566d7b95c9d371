"""Writes at the ends of bf16's range."""
import numpy as np
import pytest
import torch

import kv8_ref as ref
from kv8_forms import bf16, host, i32

pytestmark = pytest.mark.gpu

BIG = 1.9921875 * 2.0 ** 127                     # bf16's largest


@pytest.fixture(scope="module")
def lsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import clustered_key_indexing_b200 as m
    m.check_device_error()
    return m


def exponent(amax, fmt):
    """The smallest e with amax <= 2^e QMAX, from -100 to the largest scale of the format."""
    return next(e for e in range(-100, 130) if amax <= 2.0 ** e * ref.QMAX[fmt] or e == {"e4m3": 120, "int8": 121}[fmt])


def codes(x, s, fmt):
    """Nearest codes whose value is finite in fp32: at 2^120 e4m3 ends at 240."""
    y = np.clip(np.nan_to_num(x, nan=0.0, posinf=2.0 ** 128, neginf=-2.0 ** 128) / s, -448, 448)
    if fmt == "e4m3" and s == 2.0 ** 120:
        y = np.clip(y, -240, 240)
    return ref.encode(np.where(np.isnan(x), np.nan, y), fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_largest_magnitudes(lsa, fmt, page):
    """A page for each largest magnitude (and one of infinities and NaN beside
    it): the values of all codes are finite in fp32."""
    rng = np.random.default_rng(page)
    tops = [BIG, 1.984375 * 2.0 ** 127, 1.9765625 * 2.0 ** 127, 1.9375 * 2.0 ** 127, 1.75 * 2.0 ** 127, 2.0 ** 127,
            1.9921875 * 2.0 ** 126, 1.984375 * 2.0 ** 126, 1.75 * 2.0 ** 120]
    n = page * len(tops)
    xs = []
    for i in range(2):
        x = rng.uniform(-1, 1, (n, 1, 128)).reshape(len(tops), page, 1, 128) * np.array(tops)[:, None, None, None]
        x[:, 3, 0, 5 + i] = tops
        x[:, 7, 0, 9] = -np.array(tops)
        x[::2, 1, 0, 0], x[::2, 2, 0, 1], x[::2, 9, 0, 2] = np.inf, -np.inf, np.nan
        xs.append(bf16(x.reshape(n, 1, 128)))
    kv = lsa.KV8(len(tops), 1, page=page, fmt=fmt)
    lsa.kv8_write(kv, xs[0][0], xs[1][0], i32(np.arange(len(tops))[None]), i32([0]), cu=i32([0, n]))
    got = host(kv)
    for i, (_, x) in enumerate(xs):
        for p in range(len(tops)):
            y = x[p * page:(p + 1) * page, 0]
            s = 2.0 ** exponent(np.abs(y[np.isfinite(y)]).max(), fmt)
            assert got[2][p, 0, i] == s
            c, w = got[i][p, 0], codes(y, s, fmt)
            nan = np.isnan(ref.values(w, fmt))
            assert np.array_equal(np.isnan(ref.values(c, fmt)), nan)
            np.testing.assert_array_equal(c[~nan], w[~nan])
            value = ref.values(c, fmt)[~nan] * s
            assert (np.abs(value) < 2.0 ** 128).all()
    lsa.check_device_error()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_an_open_page_grows_to_the_largest_magnitudes(lsa, fmt):
    rng = np.random.default_rng(4)
    page, first = 32, 9
    x = rng.uniform(-1, 1, (page, 1, 128))
    x[:first] *= 2.0 ** 118
    x[first:] *= 2.0 ** 127
    x[first, 0, 0], x[first + 1, 0, 1], x[first + 2, 0, 2] = BIG, -BIG, np.inf
    d, h = bf16(x)
    kv = lsa.KV8(1, 1, page=page, fmt=fmt)
    table = i32([[0]])
    lsa.kv8_write(kv, d[:first], d[:first], table, i32([0]), cu=i32([0, first]))
    old = 2.0 ** exponent(np.abs(h[:first]).max(), fmt)
    lsa.kv8_write(kv, d[first:], d[first:], table, i32([first]), cu=i32([0, page - first]))
    s = 2.0 ** exponent(BIG, fmt)
    K, V, scale = host(kv)
    assert (scale == s).all()
    want = np.concatenate([ref.encode(ref.values(codes(h[:first, 0], old, fmt), fmt) * (old / s), fmt), codes(h[first:, 0], s, fmt)])
    np.testing.assert_array_equal(K[0, 0], want)
    np.testing.assert_array_equal(V[0, 0], want)
    lsa.check_device_error()
