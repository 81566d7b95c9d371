"""Attention over the 8-bit cache where the values' magnitudes are large, tiny
or far apart."""
import numpy as np
import pytest
import torch

import kv8_ref as ref
from kv8_forms import FORMS, attend, bf16, check, i32, one_sequence, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import clustered_key_indexing_b200 as m
    m.check_device_error()
    return m


def attended(q, k, v, vs, fmt):
    """kv8_ref.attend with the values' share of the bound taken from what is
    attended: a probability's absolute rounding is 2^-25 where the largest
    product of a probability and a V scale is held as 2^12 or more, so a key
    adds 2^-37 of that product times the largest code, over l."""
    o, lse, tol, tl = ref.attend(q, k, v, 0.0)
    x = q @ k.T / np.sqrt(128)
    p = np.exp(x - x.max(1, keepdims=True))
    return o, lse, tol + (k.shape[0] * 2.0 ** -37 * ref.QMAX[fmt] * (p * vs).max(1) / p.sum(1))[:, None], tl


def compare(lsa, form, kv, table, n, q, hq, fmt):
    o, lse, keys = attend(lsa, form, q, kv, table, n)
    G = q.shape[1]
    k, v, vs = values(kv, table, fmt, 0)
    for i, j in enumerate(keys):
        want, wl, tol, tl = attended(hq[i], k[j], v[j], vs[j], fmt)
        for h in range(G):
            check(o[i, h], want[h], tol[h])
        check(lse[i], wl, tl)
    lsa.check_device_error()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("fmt,e", [("e4m3", 126), ("int8", 118), ("e4m3", -90), ("int8", 100)])
def test_values_of_any_magnitude(lsa, fmt, e, form):
    rng = np.random.default_rng(170 + e)
    n, nq, G = 1500, 16, 4
    v = np.clip(rng.standard_normal((n, 1, 128)) + 0.5, -1.9, 1.9) * 2.0 ** e
    kv, table = one_sequence(lsa, rng.standard_normal((n, 1, 128)), v, 32, fmt)
    q, hq = bf16(rng.standard_normal((nq, G, 128)))
    compare(lsa, form, kv, table, n, q, hq, fmt)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("fmt,apart,first", [("e4m3", 30, True), ("int8", 45, False), ("e4m3", 90, False), ("int8", 70, True)])
def test_unattended_pages_of_large_values(lsa, fmt, apart, first, form):
    """Pages whose values are 2^apart larger and that some heads do not attend
    (their scores are 150 or more below): those heads' outputs keep the precision
    that the other pages give them."""
    rng = np.random.default_rng(apart)
    n, nq, G, page = 512, 16, 4, 32
    k = rng.standard_normal((n, 1, 128)) * 0.5
    v = rng.standard_normal((n, 1, 128)) + 0.5
    large = np.zeros(n, bool)
    for p in ((0, 1, 7) if first else (5, 14)):
        large[p * page:(p + 1) * page] = True
    k[large, :, 0] = 30.0
    k[~large, :, 0] = 0.0
    v[large] *= 2.0 ** apart
    kv, table = one_sequence(lsa, k, v, page, fmt)
    q = rng.standard_normal((nq, G, 128))
    q[..., 0] = -60.0                            # 60 * 30 / sqrt(128): 159 below
    q[:, 2, 0] = 1.0                             # one head attends them
    q, hq = bf16(q)
    compare(lsa, form, kv, table, n, q, hq, fmt)


@pytest.mark.parametrize("form", FORMS)
def test_scores_that_climb_past_large_values(lsa, form):
    """The running maximum leaves large pages behind step by step: what was
    attended first is 2^40 larger and ends with no weight."""
    rng = np.random.default_rng(77)
    n, nq, G, page = 640, 16, 4, 16
    k = rng.standard_normal((n, 1, 128)) * 0.1
    k[..., 0] = (np.arange(n) // page)[:, None] * 1.0 + 1.0
    v = (rng.standard_normal((n, 1, 128)) + 0.5) * 2.0 ** (40.0 - np.arange(n) // page)[:, None, None]
    kv, table = one_sequence(lsa, k, v, page, "e4m3")
    q = rng.standard_normal((nq, G, 128)) * 0.5
    q[..., 0] = np.array([30.0, 64.0, 3.0, 100.0])  # a page's scores are up to 8.8 above the one before
    q, hq = bf16(q)
    compare(lsa, form, kv, table, n, q, hq, "e4m3")


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_where_one_key_outweighs_the_others(lsa, fmt, form):
    """The probability of a key that holds nearly all the weight is not rounded:
    the output is the correctly rounded one, but for the few elements that lie
    within the others' roundings of the middle between two bf16 numbers.  Those
    are at most 2^-11 of what the others add, here below 0.08 of the whole, and
    bf16 numbers are 2^-8 or more apart: fewer than 1 in 100 (a rounding of the
    large one, 2^-13 on average, would move 3 in 100)."""
    rng = np.random.default_rng(90)
    n, nq, G = 600, 16, 4
    k = rng.standard_normal((n, 1, 128)) * 0.25
    at = 317
    v = rng.standard_normal((n, 1, 128))
    v = np.sign(v) * np.maximum(np.abs(v), 0.5)
    q = rng.standard_normal((nq, G, 128))
    k[:, :, 0], k[at, :, 0] = 0.0, 16.0
    q[..., 0] = np.linspace(6.7, 7.2, nq * G).reshape(nq, G)     # the others' weight: 600 / e^9.5 or less
    kv, table = one_sequence(lsa, k, v, 32, fmt)
    q, hq = bf16(q)
    o, _, keys = attend(lsa, form, q, kv, table, n)
    hk, hv, _ = values(kv, table, fmt, 0)
    wrong = 0
    for i, j in enumerate(keys):
        x = hq[i] @ hk[j].T / np.sqrt(128)
        p = np.exp(x - x.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        assert (p[:, at] > 0.92).all()
        want = torch.from_numpy(p @ hv[j]).to(torch.bfloat16)
        wrong += int((o[i].cpu() != want).sum())
    assert wrong < nq * G * 128 / 100
    lsa.check_device_error()


@pytest.mark.parametrize("tokens", [200, 2048, 64000])   # what the table has room for: CTAs, clusters, pieces
@pytest.mark.parametrize("fmt,e,new,G", [("e4m3", 30, 24, 4), ("int8", 100, 3, 2), ("e4m3", 118, 9, 8), ("int8", 17, 40, 1)])
def test_large_values_that_some_queries_do_not_see_yet(lsa, fmt, e, new, G, tokens):
    """New tokens whose windows begin at different keys: the first keys of a
    walk are hidden from some of its columns, in pages of large values."""
    rng = np.random.default_rng(e)
    n, page = 200, 16
    v = np.clip(rng.standard_normal((n, 1, 128)) + 0.5, -1.9, 1.9) * 2.0 ** e
    kv, table = one_sequence(lsa, rng.standard_normal((n, 1, 128)), v, page, fmt)
    q, hq = bf16(rng.standard_normal((new, G, 128)))
    wide = np.full((1, -(-tokens // page)), -1, np.int32)
    wide[:, :table.shape[1]] = table
    for window in (21, 70):
        o, lse = lsa.kv8_attn(q, kv, i32(wide), i32([n]), cu=i32([0, new]), window=window)
        k, w, vs = values(kv, table, fmt, 0)
        for i in range(new):
            t = n - new + i
            j = np.arange(max(0, t - window + 1), t + 1)
            want, wl, tol, tl = attended(hq[i], k[j], w[j], vs[j], fmt)
            check(o[i], want, tol)
            check(lse[i], wl, tl)
    lsa.check_device_error()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("first", [True, False])
def test_values_of_zero_beside_large_ones(lsa, first, form):
    """Pages of zeros hold all the weight, pages of the largest values none."""
    rng = np.random.default_rng(95)
    n, nq, G, page = 512, 16, 4, 32
    k, v = rng.standard_normal((n, 1, 128)) * 0.5, np.zeros((n, 1, 128))
    large = (np.arange(n) // page % 4 == 2) if first else (np.arange(n) // page % 4 == 0)
    v[large] = rng.standard_normal((int(large.sum()), 1, 128)) * 2.0 ** 110
    k[..., 0] = np.where(large, 30.0, 0.0)[:, None]
    kv, table = one_sequence(lsa, k, v, page, "e4m3")
    q = rng.standard_normal((nq, G, 128))
    q[..., 0] = -100.0                           # 100 * 30 / sqrt(128): 265, or 382 in base 2, below
    o, lse, _ = attend(lsa, form, bf16(q)[0], kv, table, n)
    assert not o.any() and torch.isfinite(lse).all()
    lsa.check_device_error()
