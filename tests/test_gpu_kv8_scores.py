"""Attention over the 8-bit cache where the scores are large: what a float's
spacing does to a score next to the running maximum."""
import numpy as np
import pytest
import torch

from kv8_forms import FORMS, attend, bf16, check, one_sequence, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import clustered_key_indexing_b200 as m
    m.check_device_error()
    return m


def large_queries(rng, nq, G, sign, spread):
    """Queries whose first element makes scores of 2^25 to 2^28 (base 2) against
    keys that hold 100 there."""
    q = rng.integers(-3, 4, (nq, G, 128)) * spread
    q[..., 0] = sign * np.exp2(np.linspace(21.4, 24.4, nq * G)).reshape(nq, G)
    return q


def lse_bound(q, k):
    """A score is off by at most 2^-23 (128 + 8) of the sum of its products'
    magnitudes and 2^-25 of Q's largest element against each key element."""
    S = (np.abs(q) @ np.abs(k).T).max(-1) + np.abs(q).max(-1) * np.abs(k).sum(-1).max() * 0.25
    return 2.0 ** -23 * 136 * S * np.log2(np.e) / np.sqrt(128) + 1e-5


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("fmt,sign", [("e4m3", 1), ("int8", -1)])
def test_equal_scores_of_large_magnitude(lsa, fmt, sign, form):
    """Equal keys: the output is the mean of the values, whatever the score.
    Probabilities are powers of two, exact in any format: what is left is the
    sums in fp32 (n / 16 + 32 terms and partial sums a lane) and one bf16 rounding."""
    rng = np.random.default_rng(60)
    n, nq, G = 600, 16, 4
    k = np.zeros((n, 1, 128))
    k[..., 0] = 100.0
    kv, table = one_sequence(lsa, k, rng.standard_normal((n, 1, 128)) + 1.0, 32, fmt)
    q, hq = bf16(large_queries(rng, nq, G, sign, 0))
    o, lse, keys = attend(lsa, form, q, kv, table, n)
    hk, hv, _ = values(kv, table, fmt, 0)
    for i, j in enumerate(keys):
        want, A = hv[j].mean(0), np.abs(hv[j]).mean(0)
        check(o[i], np.tile(want, (G, 1)), np.tile(2.0 ** -8 * np.abs(want) + (n / 16 + 32) * 2.0 ** -23 * A, (G, 1)))
        x = hq[i, :, 0] * hk[0, 0] * np.log2(np.e) / np.sqrt(128)
        check(lse[i], x + np.log2(len(j)), lse_bound(hq[i], hk[j]))
    lsa.check_device_error()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("fmt,sign", [("e4m3", -1), ("int8", 1)])
def test_scores_a_float_apart(lsa, fmt, sign, form):
    """Scores of large magnitude that differ by a few of their floats' spacings.
    Equal values: the output is that value, whatever the probabilities, up to
    their rounding to fp16 (2^-11 of each) and the fp32 sums."""
    rng = np.random.default_rng(61)
    n, nq, G = 600, 16, 4
    k = rng.integers(-1, 2, (n, 1, 128)).astype(float)
    k[..., 0] = 100.0
    row = rng.standard_normal(128) + np.where(rng.random(128) < 0.5, -2.0, 2.0)
    kv, table = one_sequence(lsa, k, np.tile(row, (n, 1, 1)), 32, fmt)
    q, hq = bf16(large_queries(rng, nq, G, sign, 8))
    o, lse, keys = attend(lsa, form, q, kv, table, n)
    hk, hv, _ = values(kv, table, fmt, 0)
    for i, j in enumerate(keys):
        check(o[i], np.tile(hv[0], (G, 1)), np.tile((2.0 ** -8 + 2.0 ** -11 + (n / 16 + 32) * 2.0 ** -23) * np.abs(hv[0]), (G, 1)))
        x = hq[i] @ hk[j].T * np.log2(np.e) / np.sqrt(128)
        m = x.max(1)
        check(lse[i], m + np.log2(np.exp2(x - m[:, None]).sum(1)), lse_bound(hq[i], hk[j]))
    lsa.check_device_error()


@pytest.mark.parametrize("form", FORMS)
def test_queries_of_the_largest_magnitudes(lsa, form):
    """Elements up to bf16's largest, against equal keys: the mean of the
    values, to ordinary precision."""
    rng = np.random.default_rng(62)
    n, nq, G = 300, 8, 2
    k = np.zeros((n, 1, 128))
    k[..., 3] = 2.0 ** -20
    kv, table = one_sequence(lsa, k, rng.standard_normal((n, 1, 128)) + 1.0, 64, "e4m3")
    q = rng.standard_normal((nq, G, 128)) * 2.0 ** 100
    q[..., 3] = np.array([1.0, 1.25, -1.5, 1.9921875])[rng.integers(0, 4, (nq, G))] * 2.0 ** rng.integers(125, 128, (nq, G))
    q, hq = bf16(q)
    o, lse, keys = attend(lsa, form, q, kv, table, n)
    hk, hv, _ = values(kv, table, "e4m3", 0)
    for i, j in enumerate(keys):
        want, A = hv[j].mean(0), np.abs(hv[j]).mean(0)
        check(o[i], np.tile(want, (G, 1)), np.tile(2.0 ** -8 * np.abs(want) + (n / 16 + 32) * 2.0 ** -23 * A, (G, 1)))
        x = hq[i, :, 3] * hk[0, 3] * np.log2(np.e) / np.sqrt(128)
        check(lse[i], x + np.log2(len(j)), lse_bound(hq[i], hk[j]))
    lsa.check_device_error()
