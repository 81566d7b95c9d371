"""The paged 8-bit K/V cache on the GPU, through the binding, against the
same operators written out in 64 bits (kv8_ref)."""
import os
import subprocess
import sys

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


def test_write_many_sequences(lsa):
    rng = np.random.default_rng(77)
    n_seq, hkv, page = 700, 1, 16
    old, new = rng.integers(0, 20, n_seq), rng.integers(0, 3, n_seq) * rng.integers(0, 12, n_seq)
    table, n_pages = scattered(rng, (old + new).tolist(), page)
    kv = random_cache(lsa, rng, n_pages, hkv, page, "int8")
    K, V, scale = host(kv)
    cu = np.concatenate([[0], np.cumsum(new)])
    (k, hk), (v, hv) = (bf16(rng.standard_normal((cu[-1], hkv, 128)) * np.exp2(rng.integers(-3, 4, (cu[-1], 1, 1)))) for _ in range(2))
    lsa.kv8_write(kv, k, v, i32(table), i32(old), cu=i32(cu))
    ref.write(K, V, scale, hk, hv, table, old.tolist(), cu, "int8")
    for g, w in zip(host(kv), (K, V, scale)):
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
    (64, 1, 8, [30000, 50], [5, 3], 0, 0),     # pieces of rows, 16 columns
    (16, 2, 4, [40000, 3], [1, 1], 0, 0),
    (64, 2, 4, [5000, 0, 700, 9], [6, 0, 4, 12], 4, 2000),   # clusters, 16 columns
    (64, 8, 1, [3000, 600, 33], [1, 1, 1], 0, 0),            # clusters of four
    (64, 8, 1, [60000, 17000, 300, 0, 7], [1, 1, 1, 1, 1], 0, 0),   # pieces long enough that short rows count more
    (32, 8, 4, [24000, 17000, 300, 9], [4, 8, 3, 1], 0, 0),
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
    (64, 4, 2, [700, 600], 300, 1100),         # a warp a row, long lists
    (64, 4, 2, [700, 600], 160, 40),           # a warp a row, short lists
    (32, 8, 1, [700, 600], 100, 200),          # a CTA a row, more rows than SMs
    (16, 2, 8, [900, 600], 60, 4200),          # a CTA a row, as many rows as SMs
    (16, 2, 8, [900, 600], 60, 5300),          # pieces of rows
    (16, 1, 4, [900, 600], 2, 27000),          # pieces of few rows
    (64, 2, 1, [900, 600], 35, 1000),          # clusters of two
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


@pytest.mark.parametrize("e", [-120, 126])
def test_queries_at_the_ends_of_the_range(lsa, e):
    """Elements near bf16's largest and smallest magnitudes: no overflow on the
    way to fp16 (against keys that bring the scores back to ordinary size)."""
    rng = np.random.default_rng(12)
    n = 40
    kv = lsa.KV8(2, 1, page=32)
    k, v = (bf16(rng.standard_normal((n, 1, 128)) * s)[0] for s in (2.0 ** max(-80, -e), 1.0))
    lsa.kv8_write(kv, k, v, i32([[0, 1]]), i32([0]), cu=i32([0, n]))
    q, hq = bf16(np.clip(rng.standard_normal((1, 2, 128)) * 0.9, -1.9, 1.9) * 2.0 ** e)
    if e > 100:                                  # scores of 2^40 would be one key's: only one element of each query is large
        q[..., 1:] = 0.0
        hq[..., 1:] = 0.0
        q[..., 0] = hq[..., 0] = 1.5 * 2.0 ** 126
        kv.K.view(torch.uint8)[:, :, :, 0] = 0x38      # 1.0
    o, lse = lsa.kv8_attn(q, kv, i32([[0, 1]]), i32([n]))
    K, V, scale = host(kv)
    wo, wl, to, tl = ref.attn(hq, K, V, scale, np.array([[0, 1]]), [n], [0, 1], "e4m3")
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


def test_offsets_past_32_bits(lsa):
    """Pages at the end of pools of more than 2^32 bytes."""
    rng = np.random.default_rng(21)
    hkv, page, n, n_pages = 8, 256, 700, 17000
    k, v = (bf16(rng.standard_normal((n, hkv, 128)))[0] for _ in range(2))
    q = bf16(rng.standard_normal((1, hkv * 2, 128)))[0]
    idx = torch.from_numpy(rng.permutation(n)[None, None].repeat(hkv, 1).astype(np.int32)).cuda()
    got = []
    for size, table in ((3, [0, 1, 2]), (n_pages, [n_pages - 1, n_pages - 3, n_pages - 2])):
        kv = lsa.KV8(size, hkv, page=page)
        lsa.kv8_write(kv, k, v, i32([table]), i32([0]), cu=i32([0, n]))
        if size > 3:
            lsa.kv8_copy_pages(kv, [n_pages - 1], [n_pages - 5])
            table = [n_pages - 5] + table[1:]
        got.append(lsa.kv8_attn(q, kv, i32([table]), i32([n])) + lsa.kv8_sparse_attn(q, kv, i32([table]), i32([n]), idx))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    lsa.check_device_error()


# ------------------------------------------------- streams, graphs, errors

def small_case(lsa, rng, fmt="e4m3", wide=2):
    """wide: the rows that the call's shapes allow get a CTA each (0), a cluster
    each (1), or are cut into pieces (2)."""
    lens, hkv, page = [300, 77, 5], 2, 32
    kv, table = filled(lsa, rng, lens, hkv, page, fmt)
    if wide:
        t = np.full((3, (0, 200, 900)[wide]), -1, np.int32)
        t[:, :table.shape[1]] = table
        table = t
    return kv, i32(table), i32(lens), torch.from_numpy(random_lists(rng, 3, hkv, (90, 1700, 27000)[wide], lens, [0, 1, 2])).cuda()


@pytest.mark.parametrize("wide", [0, 1, 2])
def test_graphs_share_nothing(lsa, wide):
    """Two captured graphs of the same calls, replayed in turn on two streams
    and with an eager call between, each with inputs of its own."""
    rng = np.random.default_rng(30)
    kv, table, lens, idx = small_case(lsa, rng, wide=wide)
    qs = [bf16(rng.standard_normal((3, 8, 128)))[0] for _ in range(3)]

    def calls(q):
        return lsa.kv8_attn(q, kv, table, lens) + lsa.kv8_sparse_attn(q, kv, table, lens, idx)

    want = [calls(q) for q in qs]
    graphs = []
    for q in qs[:2]:
        g = torch.cuda.CUDAGraph()
        buf = q.clone()
        with torch.cuda.graph(g):
            out = calls(buf)
        graphs.append((g, buf, out))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for s, (g, _, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        eager = calls(qs[2])
        torch.cuda.synchronize()
        for (_, _, out), w in zip(graphs + [(0, 0, eager)], want):
            for x, y in zip(out, w):
                assert torch.equal(x, y)
    graphs[0][1].copy_(qs[1])                    # a replay takes what the buffer holds then
    graphs[0][0].replay()
    torch.cuda.synchronize()
    for x, y in zip(graphs[0][2], want[1]):
        assert torch.equal(x, y)


def test_a_captured_decode_step(lsa):
    """Write and attend in one graph: lens and start are read on replay."""
    rng = np.random.default_rng(31)
    kv, table = filled(lsa, rng, [70, 33], 2, 16, "int8")
    table = i32(np.concatenate([table, np.full((2, 2), -1, np.int32)], 1))
    own = lsa.KV8(40, 2, page=16, fmt="int8")    # a second pool for the eager calls
    table2 = i32(np.arange(2 * table.shape[1]).reshape(2, -1))
    for b in range(2):
        for j in range(5):
            if table[b, j] >= 0:
                for x, y in ((own.K, kv.K), (own.V, kv.V), (own.scale, kv.scale)):
                    x[table2[b, j]] = y[table[b, j]]
    k, v, q = (bf16(rng.standard_normal((2, h, 128)))[0] for h in (2, 2, 8))
    start, lens = i32([70, 33]), i32([71, 34])
    before = [t.clone() for t in (kv.K.view(torch.uint8), kv.V.view(torch.uint8), kv.scale)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lsa.kv8_write(kv, k, v, table, start)
        o, lse = lsa.kv8_attn(q, kv, table, lens)
    for t, b in zip((kv.K.view(torch.uint8), kv.V.view(torch.uint8), kv.scale), before):
        assert torch.equal(t, b)                 # a capture runs nothing
    for step in range(4):
        for t in (k, v, q):
            t.copy_(bf16(rng.standard_normal(tuple(t.shape)) * 2.0 ** step)[0])
        g.replay()
        lsa.kv8_write(own, k, v, table2, start)
        wo, wl = lsa.kv8_attn(q, own, table2, lens)
        torch.cuda.synchronize()
        assert torch.equal(o, wo) and torch.equal(lse, wl)
        start += 1
        lens += 1
    lsa.check_device_error()


def test_first_calls_inside_a_capture():
    """A process whose first calls are captured: what the library asks the
    device for once is allowed there."""
    code = """
import torch, clustered_key_indexing_b200 as lsa
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
kv = lsa.KV8(400, 2, page=64)
table = torch.arange(400, dtype=torch.int32, device="cuda")[None]
wide = torch.cat([table] * 8, 1)
k, q = torch.randn(1, 2, 128, device="cuda").bfloat16(), torch.randn(1, 8, 128, device="cuda").bfloat16()
idx, lens, start, pages = torch.randint(0, 19000, (1, 2, 3000), dtype=torch.int32, device="cuda"), i32([20000]), i32([19999]), ([1, 2], [350, 351])
def calls():
    lsa.kv8_write(kv, k, k, table, start)
    lsa.kv8_copy_pages(kv, *pages)
    return lsa.kv8_attn(q, kv, table, lens) + lsa.kv8_attn(q, kv, wide, lens) + lsa.kv8_sparse_attn(q, kv, table, lens, idx)
g = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g):
    out = calls()
g.replay()
want = calls()
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(out, want)) and out[0].abs().max() >= 0
lsa.check_device_error()
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr


def test_another_stream(lsa):
    rng = np.random.default_rng(32)
    kv, table, lens, idx = small_case(lsa, rng)
    q = bf16(rng.standard_normal((3, 8, 128)))[0]
    want = lsa.kv8_attn(q, kv, table, lens) + lsa.kv8_sparse_attn(q, kv, table, lens, idx)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = lsa.kv8_attn(q, kv, table, lens, stream=s) + lsa.kv8_sparse_attn(q, kv, table, lens, idx, stream=s)
    junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(8)]   # what the calls freed is not reused yet
    torch.cuda.current_stream().wait_stream(s)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    del junk
    O, lse = torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 8, device="cuda")
    ws = torch.empty(lsa.kv8_attn_workspace_bytes(kv, 3, 8, 3, table.shape[1]), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    r = lsa.kv8_attn(q, kv, table, lens, O=O, lse=lse, ws=ws)
    assert r[0] is O and r[1] is lse and torch.equal(O, want[0]) and torch.equal(lse, want[1])


def test_outputs_made_for_a_stream_are_its_own_memory(lsa):
    """A block that the current stream gave back may still be read there, so a
    call on another stream does not take it."""
    rng = np.random.default_rng(34)
    kv, table, lens, idx = small_case(lsa, rng)
    q = bf16(rng.standard_normal((3, 8, 128)))[0]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call in (lambda: lsa.kv8_attn(q, kv, table, lens, stream=s), lambda: lsa.kv8_sparse_attn(q, kv, table, lens, idx, stream=s)):
        used = [torch.empty_like(q) for _ in range(3)] + [torch.empty(3, 8, device="cuda") for _ in range(3)]
        places = {x.data_ptr() for x in used}
        del used
        assert not places & {x.data_ptr() for x in call()}
    torch.cuda.synchronize()


def test_a_window_longer_than_everything(lsa):
    """The same as none, for queries before the first token too."""
    rng = np.random.default_rng(35)
    kv, table = filled(lsa, rng, [2, 90], 2, 16, "e4m3")
    q = bf16(rng.standard_normal((12, 4, 128)))[0]
    cu, lens = i32([0, 9, 12]), i32([2, 90])
    want = lsa.kv8_attn(q, kv, i32(table), lens, cu=cu)
    for window in (table.shape[1] * 16, 2 ** 31 - 1):
        got = lsa.kv8_attn(q, kv, i32(table), lens, cu=cu, sinks=3, window=window)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    lsa.check_device_error()


def test_bad_pages_and_ranges_are_reported(lsa):
    from clustered_key_indexing_b200._lib import LSA_EDEVICE, LSAError

    def reported(what):
        torch.cuda.synchronize()
        with pytest.raises(LSAError, match=what) as e:
            lsa.check_device_error()
        assert e.value.status == LSA_EDEVICE
        lsa.check_device_error()

    rng = np.random.default_rng(33)
    kv, table, lens, idx = small_case(lsa, rng, wide=0)
    K, V, scale = host(kv)
    q, hq = bf16(rng.standard_normal((3, 8, 128)))
    for bad in (-1, kv.n_pages, 2 ** 31 - 1):
        t = table.clone()
        t[0, 1] = bad                            # keys 32 .. 63 of the first sequence are skipped
        o, lse = lsa.kv8_attn(q, kv, t, lens)
        reported("page number outside")
        k = [j for j in range(300) if not 32 <= j < 64]
        want = ref.lists(hq, K, V, scale, table.cpu().numpy(), [300, 77, 5], [0, 1, 2],
                         np.array([[k] * 2, [list(range(77)) + [-1] * (len(k) - 77)] * 2, [list(range(5)) + [-1] * (len(k) - 5)] * 2]), "e4m3")
        close(o, want[0], want[2])
        o, lse = lsa.kv8_sparse_attn(q, kv, t, lens, idx)
        reported("page number outside")
        ix = idx.cpu().numpy().copy()
        ix[0][(ix[0] >= 32) & (ix[0] < 64)] = -1
        want = ref.lists(hq, K, V, scale, table.cpu().numpy(), [300, 77, 5], [0, 1, 2], ix, "e4m3")
        close(o, want[0], want[2])
    over = idx.clone()
    over[1, 0, 3] = 77                           # a position past its sequence
    o, _ = lsa.kv8_sparse_attn(q, kv, table, lens, over)
    reported("index entry")
    over[1, 0, 3] = -1
    assert torch.equal(o, lsa.kv8_sparse_attn(q, kv, table, lens, over)[0])
    lsa.kv8_sparse_attn(q, kv, table, lens, idx, seq=i32([0, 3, -1]))
    reported("range outside")
    lsa.kv8_attn(q, kv, table, i32([300, table.shape[1] * 32 + 1, -4]))
    reported("range outside")
    for cu in ([0, 2, 1, 3], [0, 1, 2, 4], [-1, 1, 2, 3]):
        lsa.kv8_attn(q, kv, table, lens, cu=i32(cu))
        reported("range outside")
    k = bf16(rng.standard_normal((3, 2, 128)))[0]
    before = host(kv)
    t = table.clone()
    t[:, :] = kv.n_pages
    lsa.kv8_write(kv, k, k, t, i32([300, 77, 5]))
    reported("page number outside")
    for start, cu in (([-1, -5, 320 + 32 * table.shape[1]], None), ([table.shape[1] * 32] * 3, None), ([0, 0, 0], [0, 4, 5, 6])):
        lsa.kv8_write(kv, k, k, table, i32(start), cu=None if cu is None else i32(cu))
        reported("range outside")
        if cu is None:
            for x, y in zip(host(kv), before):
                np.testing.assert_array_equal(x, y)


def test_empty_calls(lsa):
    rng = np.random.default_rng(34)
    kv, table, lens, idx = small_case(lsa, rng)
    none = torch.empty(0, 8, 128, dtype=torch.bfloat16, device="cuda")
    o, lse = lsa.kv8_attn(none, kv, table, lens, cu=i32([0, 0, 0, 0]))
    assert o.shape == (0, 8, 128) and lse.shape == (0, 8)
    o, lse = lsa.kv8_sparse_attn(none, kv, table, lens, idx[:0], seq=i32([]))
    assert o.shape == (0, 8, 128) and lse.shape == (0, 8)
    before = host(kv)
    kz = none[:, :2]
    lsa.kv8_write(kv, kz, kz, table, lens, cu=i32([0, 0, 0, 0]))
    lsa.kv8_copy_pages(kv, [], [])
    for x, y in zip(host(kv), before):
        np.testing.assert_array_equal(x, y)
    q = bf16(rng.standard_normal((3, 8, 128)))[0]
    o, lse = lsa.kv8_attn(q, kv, table, i32([0, 0, 0]))
    assert not o.any() and torch.isneginf(lse).all()
    o, lse = lsa.kv8_sparse_attn(q, kv, table, lens, torch.full_like(idx, -1))
    assert not o.any() and torch.isneginf(lse).all()
    o, lse = lsa.kv8_attn(q, kv, table[:, :0].contiguous(), i32([0, 0, 0]))
    assert not o.any() and torch.isneginf(lse).all()
    lsa.check_device_error()


def test_results_do_not_depend_on_the_run(lsa):
    rng = np.random.default_rng(35)
    kv, table, lens, idx = small_case(lsa, rng)
    q = bf16(rng.standard_normal((3, 8, 128)))[0]
    first = lsa.kv8_attn(q, kv, table, lens) + lsa.kv8_sparse_attn(q, kv, table, lens, idx)
    for _ in range(5):
        for x, y in zip(lsa.kv8_attn(q, kv, table, lens) + lsa.kv8_sparse_attn(q, kv, table, lens, idx), first):
            assert torch.equal(x, y)


# ---------------------------------------------------------- as they are used

@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_a_layer_over_the_cache(lsa, fmt):
    """A prompt written into pages, selected and attended in chunks, then
    decoded: appends, a fork, drafts that are partly rejected, a compaction."""
    rng = np.random.default_rng(40)
    T, hkv, hq, page = 2048, 2, 8, 64
    cfg = lsa.Config(k=256, sinks=4, window=128)
    W = torch.linalg.qr(torch.from_numpy(rng.standard_normal((128, 64))))[0].float().contiguous().cuda()
    (K, hK), (V, hV), (Q, hQ) = (bf16(rng.standard_normal((T + 40, h, 128))) for h in (hkv, hkv, hq))
    pages = lsa.KV8Pages(lsa.KV8(90, hkv, page=page, fmt=fmt))
    hole, a = pages.add(), pages.add()
    pages.append([hole], K[:100], V[:100], [100])
    pages.append([a], K[:T], V[:T], [T])
    # the prompt: index rows from the bf16 keys, attention over the codes
    cache = lsa.Cache(hkv, T, cfg)
    lsa.build_buckets(K[:T], W, cfg, cache)
    table, lens = pages.table([a])
    for t0, nq in ((0, 300), (T - 64, 64)):
        idx = lsa.select(Q[t0:t0 + nq], t0, W, cache, cfg)
        o, lse = lsa.kv8_sparse_attn(Q[t0:t0 + nq], pages.kv, table, lens, idx, seq=i32([0] * nq))
        some = rng.permutation(nq)[:12]
        wo, wl, to, tl = ref.lists(hQ[t0:t0 + nq][some], *host(pages.kv), table.cpu().numpy(), [T], [0] * 12, idx.cpu().numpy()[some], fmt)
        close(o[torch.from_numpy(some).cuda()], wo, to)
        close(lse[torch.from_numpy(some).cuda()], wl, tl)
        # near the bf16 attention: the codes' relative error, averaged over the keys
        full = lsa.sparse_attn(Q[t0:t0 + nq], K[:T], V[:T], idx).float()
        assert (o.float() - full).norm() < 0.1 * full.norm()
    # decode: one token, a fork, five drafts each of which two are kept
    pages.append([a], K[T:T + 1], V[T:T + 1])
    b = pages.fork(a)
    used = pages.used_pages
    pages.append([a, b], torch.cat([K[T + 1:T + 6], K[T + 11:T + 16]]), torch.cat([V[T + 1:T + 6], V[T + 11:T + 16]]), [5, 5])
    assert pages.used_pages == used + 1          # the open page, copied once
    qd, hqd = Q[T:T + 10], hQ[T:T + 10]

    def attend(n):
        table, lens = pages.table([a, b])
        got = lsa.kv8_attn(qd[:2 * n], pages.kv, table, lens, cu=i32([0, n, 2 * n]), sinks=4, window=128)
        want = ref.attn(hqd[:2 * n], *host(pages.kv), table.cpu().numpy(), lens.tolist(), [0, n, 2 * n], fmt, 4, 128)
        close(got[0], want[0], want[2])
        close(got[1], want[1], want[3])
        return got

    attend(5)
    for s in (a, b):
        pages.truncate(s, T + 3)
    pages.append([b, a], K[T + 20:T + 22], V[T + 20:T + 22])
    before = attend(2)
    pages.free(hole)
    assert pages.compact() > 0
    after = attend(2)
    assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
    assert pages.used_pages == len(set(pages.pages(a)) | set(pages.pages(b))) == max(pages.pages(a) + pages.pages(b)) + 1
    lsa.check_device_error()


@pytest.mark.parametrize("fmt,mode", [("e4m3", 0), ("int8", 1)])
def test_decode_over_the_cache(lsa, fmt, mode):
    """Decode steps with paged 8-bit keys and values select the same rows as
    with bf16 pools, and attend over the codes."""
    rng = np.random.default_rng(50)
    batch, hkv, hq, cap, steps = 3, 2, 8, 2048, 6
    cfg = lsa.Config(k=128, sinks=4, window=600, mode=mode)
    W = torch.linalg.qr(torch.from_numpy(rng.standard_normal((128, 64))))[0].float().contiguous().cuda()
    lens = [1021, 1534, 700]                     # two of them complete a block on the way
    data = [[bf16(rng.standard_normal((n + steps, h, 128)))[0] for h in (hkv, hkv, hq)] for n in lens]
    plain = lsa.Decode(batch, hkv, hq, cap, cfg)
    dec = lsa.Decode(batch, hkv, hq, cap, cfg, kv8=fmt)
    for r, (K, V, _) in enumerate(data):
        for d in (plain, dec):
            d.load(r, K[:lens[r]], V[:lens[r]], W)
    assert dec.len == lens
    for i in range(steps):
        k, v, q = (torch.stack([data[r][j][lens[r] + i] for r in range(batch)]) for j in range(3))
        rows = [torch.empty(batch, hkv, cfg.row, dtype=torch.int32, device="cuda") for _ in range(2)]
        plain.step(q, k, v, W, W, idx_out=rows[0])
        o = dec.step(q, k, v, W, W, idx_out=rows[1])
        assert torch.equal(rows[0], rows[1])
        now = [n + i + 1 for n in lens]
        want = ref.lists(q.double().cpu().numpy(), *host(dec.kv8), dec.kv8_table.cpu().numpy(), now, [0, 1, 2],
                         rows[1].cpu().numpy(), fmt)
        close(o, want[0], want[2])
    assert dec.len == now
    lsa.check_device_error()


def test_decode_requests_share_the_pages_of_a_prefix(lsa):
    rng = np.random.default_rng(51)
    hkv, hq, cap, n, steps = 2, 4, 1024, 700, 3
    cfg = lsa.Config(k=64, sinks=4, window=512)
    W = torch.linalg.qr(torch.from_numpy(rng.standard_normal((128, 64))))[0].float().contiguous().cuda()
    K, V = (bf16(rng.standard_normal((n, hkv, 128)))[0] for _ in range(2))
    pages = lsa.KV8Pages(lsa.KV8(30, hkv, page=64))
    a = pages.add()
    pages.append([a], K, V, [n])
    ids = [a, pages.fork(a)]
    table = torch.full((2, cap // 64), -1, dtype=torch.int32, device="cuda")
    dec = lsa.Decode(2, hkv, hq, cap, cfg, kv8=pages.kv, kv8_table=table)
    own = lsa.Decode(2, hkv, hq, cap, cfg, kv8="e4m3")
    for r in range(2):
        dec.load(r, K, V, W, written=True)
        own.load(r, K, V, W)
    for _ in range(steps):
        q, k, v = (bf16(rng.standard_normal((2, h, 128)))[0] for h in (hq, hkv, hkv))
        pages.reserve(ids)
        table.copy_(pages.table(ids, width=table.shape[1])[0])
        o = dec.step(q, k, v, W, W)
        pages.advance(ids)
        assert torch.equal(o, own.step(q, k, v, W, W))
    assert pages.used_pages == 11 + 1            # eleven pages of the prompt, the open one twice
    lsa.check_device_error()
