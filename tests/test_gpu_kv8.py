"""The paged 8-bit K/V cache on the GPU, through the binding, against the
same operators written out in 64 bits (kv8_ref)."""
import numpy as np
import pytest
import torch

import kv8_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import clustered_key_indexing_b200 as m
    m.check_device_error()
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bf16(x):
    """fp32 values rounded to bf16: (device tensor, the same values in 64 bits)."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def host(kv):
    return [kv.K.view(torch.uint8).cpu().numpy().copy(), kv.V.view(torch.uint8).cpu().numpy().copy(),
            kv.scale.cpu().numpy().astype(np.float64)]


def random_cache(lsa, rng, n_pages, hkv, page, fmt):
    """A pool of arbitrary bytes (NaN codes among them) with filled values on
    top in every page: unwritten rows are garbage, as in a recycled page."""
    kv = lsa.KV8(n_pages, hkv, page=page, fmt=fmt)
    for P in (kv.K, kv.V):
        P.view(torch.uint8).copy_(torch.from_numpy(rng.integers(0, 256, tuple(P.shape), dtype=np.uint8)))
    kv.scale.copy_(torch.from_numpy(np.exp2(rng.integers(-8, 1, tuple(kv.scale.shape))).astype(np.float32)))
    return kv


def scattered(rng, lens, page, spare=2):
    need = [-(-n // page) for n in lens]
    order = rng.permutation(sum(need) + spare)
    width = max(1, max(need))
    table, at = np.full((len(lens), width), -1, np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, len(order)


def filled(lsa, rng, lens, hkv, page, fmt):
    """A cache holding `lens` tokens per sequence, written by the library."""
    table, n_pages = scattered(rng, lens, page)
    kv = random_cache(lsa, rng, n_pages, hkv, page, fmt)
    cu = np.concatenate([[0], np.cumsum(lens)])
    k, v = (bf16(rng.standard_normal((cu[-1], hkv, 128)) * np.exp2(rng.integers(-2, 3, (cu[-1], 1, 1))))[0] for _ in range(2))
    lsa.kv8_write(kv, k, v, i32(table), i32([0] * len(lens)), cu=i32(cu))
    return kv, table


def close(got, want, tol):
    got = got.float().cpu().numpy().astype(np.float64)
    assert got.shape == want.shape
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf])
    e = np.abs(got[~inf] - want[~inf])
    assert np.isfinite(got[~inf]).all()
    assert (e <= tol[~inf]).all(), f"{(e - tol[~inf]).max()} above the bound; error {e.max()}"


# ------------------------------------------------------------------- write

@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("page,hkv,new,old", [(16, 1, [1], [0]), (64, 2, [1, 1, 1], [5, 64, 127]), (32, 3, [70, 0, 1, 33], [31, 7, 0, 64]),
                                              (128, 2, [300, 2], [100, 126]), (256, 1, [513], [255])])
def test_write_equals_the_formula(lsa, fmt, page, hkv, new, old):
    rng = np.random.default_rng(page + hkv)
    total = [a + b for a, b in zip(new, old)]
    table, n_pages = scattered(rng, [max(1, t) for t in total], page)
    kv = random_cache(lsa, rng, n_pages, hkv, page, fmt)
    K, V, scale = host(kv)
    cu = np.concatenate([[0], np.cumsum(new)])
    xs = []
    for _ in range(2):
        x = rng.standard_normal((cu[-1], hkv, 128)) * np.exp2(rng.integers(-9, 9, (cu[-1], hkv, 1)))
        x[rng.random(x.shape) < 0.01] = 0.0
        x.reshape(-1)[::97] = np.inf
        x.reshape(-1)[1::113] = -np.inf
        x.reshape(-1)[5::131] = np.nan
        xs.append(bf16(x))
    one = all(n == 1 for n in new)
    lsa.kv8_write(kv, xs[0][0], xs[1][0], i32(table), i32(old), cu=None if one else i32(cu))
    ref.write(K, V, scale, xs[0][1], xs[1][1], table, old, cu, fmt)
    gK, gV, gs = host(kv)
    np.testing.assert_array_equal(gs, scale)
    for g, w in ((gK, K), (gV, V)):
        if fmt == "e4m3":   # either NaN code is a NaN; the rows behind the new ones keep their bytes
            nan = np.isnan(ref.E4M3)
            assert np.array_equal(nan[g], nan[w])
            g, w = np.where(nan[g], 0x7F, g), np.where(nan[w], 0x7F, w)
        np.testing.assert_array_equal(g, w)
    lsa.check_device_error()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_write_token_by_token_grows_the_open_page(lsa, fmt):
    rng = np.random.default_rng(5)
    page, hkv, n = 16, 2, 37
    table, n_pages = scattered(rng, [n, n], page)
    kv = random_cache(lsa, rng, n_pages, hkv, page, fmt)
    K, V, scale = host(kv)
    k, v = (rng.standard_normal((n, 2, hkv, 128)) * np.exp2(np.arange(n) % 11 - 5)[:, None, None, None] for _ in range(2))
    k[3] = 0.0
    for t in range(n):
        (dk, hk), (dv, hv) = bf16(k[t]), bf16(v[t])
        lsa.kv8_write(kv, dk, dv, i32(table), i32([t, t]))
        ref.write(K, V, scale, hk, hv, table, [t, t], [0, 1, 2], fmt)
    for g, w in zip(host(kv), (K, V, scale)):
        np.testing.assert_array_equal(g, w)


def test_write_reads_strided_rows(lsa):
    """K and V as slices of one fused projection."""
    rng = np.random.default_rng(6)
    qkv, _ = bf16(rng.standard_normal((40, 3 * 2 * 128)))
    k, v = (qkv[:, a:a + 256].view(40, 2, 128) for a in (256, 512))
    a, b = (lsa.KV8(4, 2, page=16, fmt="e4m3") for _ in range(2))
    table = i32([[3, 0, 1]])
    lsa.kv8_write(a, k, v, table, i32([2]), cu=i32([0, 40]))
    lsa.kv8_write(b, k.contiguous(), v.contiguous(), table, i32([2]), cu=i32([0, 40]))
    for x, y in zip(host(a), host(b)):
        np.testing.assert_array_equal(x, y)
    q = qkv[:, :256].view(40, 2, 128)
    o1, l1 = lsa.kv8_attn(q, a, table, i32([42]), cu=i32([0, 40]))
    o2, l2 = lsa.kv8_attn(q.contiguous(), a, table, i32([42]), cu=i32([0, 40]))
    assert torch.equal(o1, o2) and torch.equal(l1, l2)


# --------------------------------------------------------------- attention

@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("page,hkv,G,lens,new,sinks,window", [
    (16, 1, 1, [1], [1], 0, 0),
    (16, 1, 4, [777], [1], 0, 0),
    (64, 2, 8, [15, 0, 300, 64], [1, 1, 1, 1], 0, 0),
    (32, 3, 2, [100, 33, 5, 4097], [3, 0, 5, 2], 0, 0),
    (64, 1, 4, [200, 90], [5, 7], 4, 33),
    (128, 2, 8, [1000, 17], [4, 2], 0, 1),
    (16, 2, 4, [130, 129, 3], [1, 1, 1], 20, 50),
    (256, 1, 1, [600], [40], 3, 100),
    (64, 1, 4, [3, 2], [6, 2], 0, 0),          # more queries than tokens: the first see nothing
    (16, 8, 4, [20000], [1], 0, 0),
    (32, 1, 8, [70000, 1], [1, 1], 0, 0),
])
def test_attention_against_64_bits(lsa, fmt, page, hkv, G, lens, new, sinks, window):
    rng = np.random.default_rng(sum(lens) + page)
    kv, table = filled(lsa, rng, [max(n, 1) for n in lens], hkv, page, fmt)
    cu = np.concatenate([[0], np.cumsum(new)])
    q, hq = bf16(rng.standard_normal((cu[-1], hkv * G, 128)) * 1.5)
    one = all(n == 1 for n in new)
    o, lse = lsa.kv8_attn(q, kv, i32(table), i32(lens), cu=None if one else i32(cu), sinks=sinks, window=window)
    lsa.check_device_error()
    K, V, scale = host(kv)
    wo, wl, to, tl = ref.attn(hq, K, V, scale, table, lens, cu, fmt, sinks, window)
    close(o, wo, to)
    close(lse, wl, tl)


@pytest.mark.parametrize("n_seq,hkv,G,top,spread", [(300, 1, 4, 90, 1), (700, 2, 1, 40, 1), (33, 8, 8, 500, 7), (520, 1, 2, 3000, 1)])
def test_ragged_batches(lsa, n_seq, hkv, G, top, spread):
    """Many sequences of very different lengths (none, one long), some without
    a new token, in tables wider than they need."""
    rng = np.random.default_rng(n_seq)
    lens = (np.exp(rng.uniform(0, np.log(top), n_seq)).astype(int) * (rng.random(n_seq) < 0.9)).tolist()
    lens[n_seq // 2] = 4 * top
    new = rng.integers(0, spread + 1, n_seq)
    new[-1] = spread
    kv, table = filled(lsa, rng, [max(n, 1) for n in lens], hkv, 16, "e4m3")
    K, V, scale = host(kv)
    wide = np.full((n_seq, 1000), -1, np.int32)
    wide[:, :table.shape[1]] = table
    cu = np.concatenate([[0], np.cumsum(new)])
    q, hq = bf16(rng.standard_normal((cu[-1], hkv * G, 128)))
    wo, wl, to, tl = ref.attn(hq, K, V, scale, table, lens, cu, "e4m3", 2, 64)
    for tb in (table, wide):
        o, lse = lsa.kv8_attn(q, kv, i32(tb), i32(lens), cu=i32(cu), sinks=2, window=64)
        close(o, wo, to)
        close(lse, wl, tl)
    each, heach = bf16(rng.standard_normal((n_seq, hkv * G, 128)))
    wo, wl, to, tl = ref.attn(heach, K, V, scale, table, lens, np.arange(n_seq + 1), "e4m3")
    for tb in (table, wide):
        o, lse = lsa.kv8_attn(each, kv, i32(tb), i32(lens))
        close(o, wo, to)
        close(lse, wl, tl)
    lsa.check_device_error()


def random_lists(rng, nq, hkv, n_idx, lens, seq, pads=0.2):
    idx = np.full((nq, hkv, n_idx), -1, np.int32)
    for i in range(nq):
        for h in range(hkv):
            if lens[seq[i]] > 0:
                x = rng.integers(0, lens[seq[i]], n_idx)
                idx[i, h] = np.where(rng.random(n_idx) < pads, -1, x)
    return idx


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("page,hkv,G,lens,nq,n_idx", [
    (16, 1, 1, [1], 1, 1),
    (64, 2, 4, [500, 70, 16], 3, 100),
    (32, 1, 8, [3000], 9, 333),
    (128, 2, 2, [40, 900], 50, 16),
    (16, 8, 4, [5000], 1, 2500),
    (256, 3, 4, [300, 1], 5, 0),
    (64, 4, 2, [700, 600], 1300, 40),          # enough rows for one warp each
])
def test_lists_against_64_bits(lsa, fmt, page, hkv, G, lens, nq, n_idx):
    rng = np.random.default_rng(nq + n_idx)
    kv, table = filled(lsa, rng, lens, hkv, page, fmt)
    seq = np.arange(nq) if nq == len(lens) else rng.integers(0, len(lens), nq)
    idx = random_lists(rng, nq, hkv, n_idx, lens, seq)
    if nq > 3:
        idx[2] = -1                              # a row without keys
    q, hq = bf16(rng.standard_normal((nq, hkv * G, 128)) * 1.5)
    o, lse = lsa.kv8_sparse_attn(q, kv, i32(table), i32(lens), torch.from_numpy(idx).cuda(), seq=None if nq == len(lens) else i32(seq))
    lsa.check_device_error()
    K, V, scale = host(kv)
    wo, wl, to, tl = ref.lists(hq, K, V, scale, table, lens, seq, idx, fmt)
    close(o, wo, to)
    close(lse, wl, tl)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_scales_far_apart(lsa, fmt):
    """Pages whose V (and K) scales differ by 2^20, the large one almost
    unattended, and a Q of 2^40 against K of 2^-40."""
    rng = np.random.default_rng(9)
    page, hkv, G, n = 16, 1, 4, 96
    table, n_pages = scattered(rng, [n], page)
    kv = lsa.KV8(n_pages, hkv, page=page, fmt=fmt)
    k = rng.standard_normal((n, hkv, 128)) * 2.0 ** -40
    v = rng.standard_normal((n, hkv, 128))
    k[:16] *= 0.25
    v[32:48] *= 2.0 ** 20
    qx = rng.standard_normal((1, G, 128))
    k[32:48] = -np.abs(rng.standard_normal((16, hkv, 1))) * np.sign(qx[0].sum(0))[None, None] * 2.0 ** -40
    (dk, _), (dv, _), (q, hq) = bf16(k), bf16(v), bf16(qx * 2.0 ** 40)
    lsa.kv8_write(kv, dk, dv, i32(table), i32([0]), cu=i32([0, n]))
    K, V, scale = host(kv)
    o, lse = lsa.kv8_attn(q, kv, i32(table), i32([n]))
    wo, wl, to, tl = ref.attn(hq, K, V, scale, table, [n], [0, 1], fmt)
    close(o, wo, to)
    close(lse, wl, tl)
    idx = np.tile(rng.permutation(n).astype(np.int32), (1, 1, 1))
    o, lse = lsa.kv8_sparse_attn(q, kv, i32(table), i32([n]), torch.from_numpy(idx).cuda())
    close(o, wo, to)
    close(lse, wl, tl)


def test_nan_under_the_mask_stays_there(lsa):
    """A NaN value row reaches the queries that attend it and no other: rows
    behind the sequence, keys outside the window, tokens newer than the query."""
    rng = np.random.default_rng(10)
    page, n, new = 16, 90, 4
    kv, table = filled(lsa, rng, [n], 1, page, "e4m3")
    bad = [20, 88]                               # outside every window below; the last but one query's own token
    for t in bad:
        kv.V.view(torch.uint8)[int(table[0, t // page]), 0, t % page] = 0x7F
    q, hq = bf16(rng.standard_normal((new, 4, 128)))
    o, lse = lsa.kv8_attn(q, kv, i32(table), i32([n]), cu=i32([0, new]), sinks=4, window=30)
    K, V, scale = host(kv)
    wo, wl, to, tl = ref.attn(hq, K, V, scale, table, [n], [0, new], "e4m3", 4, 30)
    assert np.isnan(wo[2:]).all() and np.isfinite(wo[:2]).all()
    close(o[:2], wo[:2], to[:2])
    assert torch.isnan(o[2:]).all()
    close(lse, wl, tl)
    idx = i32([[[0, 1, 19, 21, -1, 87, 89]]])
    o, lse = lsa.kv8_sparse_attn(q[:1], kv, i32(table), i32([n]), idx)
    assert torch.isfinite(o.float()).all()


# -------------------------------------------------------------------- pages

@pytest.mark.parametrize("fmt,page,hkv,n", [("e4m3", 16, 1, 1), ("int8", 64, 8, 3), ("e4m3", 256, 3, 61), ("int8", 16, 2, 2001)])
def test_copy_pages(lsa, fmt, page, hkv, n):
    rng = np.random.default_rng(n)
    kv = random_cache(lsa, rng, 2 * n + 5, hkv, page, fmt)
    K, V, scale = host(kv)
    order = rng.permutation(2 * n + 5)
    src, dst = order[:n], order[n:2 * n]
    lsa.kv8_copy_pages(kv, src, dst.tolist())
    for P in (K, V, scale):
        P[dst] = P[src]
    for g, w in zip(host(kv), (K, V, scale)):
        np.testing.assert_array_equal(g, w)
