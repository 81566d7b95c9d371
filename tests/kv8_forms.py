"""The forms that attention over the 8-bit cache takes, for tests that must
hold in each: one sequence's pages, read by queries that all see its tokens."""
import numpy as np
import torch

import kv8_ref as ref


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def bf16(x):
    """fp32 values rounded to bf16: (device tensor, the same values in 64 bits)."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def host(kv):
    return [kv.K.view(torch.uint8).cpu().numpy().copy(), kv.V.view(torch.uint8).cpu().numpy().copy(),
            kv.scale.cpu().numpy().astype(np.float64)]


def one_sequence(lsa, k, v, page, fmt):
    """A cache that holds k, v [n, hkv, 128] as one sequence, in order."""
    n, hkv, _ = k.shape
    kv = lsa.KV8(-(-n // page), hkv, page=page, fmt=fmt)
    table = np.arange(kv.n_pages, dtype=np.int32)[None]
    lsa.kv8_write(kv, bf16(k)[0], bf16(v)[0], i32(table), i32([0]), cu=i32([0, n]))
    return kv, table


FORMS = ("CTA of 16 warps", "CTA of 8 warps", "cluster", "stream", "columns by CTAs", "columns by clusters", "columns in the stream",
         "list by warps", "list by CTAs", "list by clusters", "list in the stream")


def attend(lsa, form, q, kv, table, n):
    """q [nq, hq, 128] over the first n tokens in one of the forms, which go by
    the numbers of rows and the widths of tables and lists: (o, lse, the keys of
    each query).  A form that wants many rows gets the queries several times."""
    nq, hq, _ = q.shape
    rows, page, hkv = nq * kv.hkv, kv.page, kv.hkv

    def wide(n_seq, tokens):
        t = np.full((n_seq, max(table.shape[1], -(-tokens // page))), -1, np.int32)
        t[:, :table.shape[1]] = table
        return i32(t)

    def once(o, lse, reps):
        o, lse = o.view(reps, -1, hq, 128), lse.view(reps, -1, hq)
        assert o.isnan().any() or (torch.equal(o, o[:1].expand_as(o)) and torch.equal(lse, lse[:1].expand_as(lse)))
        return o[0], lse[0]

    kind, tokens, many = {"CTA of 16 warps": ("one", n, 100), "CTA of 8 warps": ("one", n, 200), "cluster": ("one", 2048, 0),
                          "stream": ("one", 64000, 0), "columns by CTAs": ("columns", n, 100), "columns by clusters": ("columns", n, 0),
                          "columns in the stream": ("columns", 64000, 0), "list by warps": ("list", n, 1200), "list by CTAs": ("list", n, 100),
                          "list by clusters": ("list", n, 0), "list in the stream": ("list", 48000, 0)}[form]
    if kind == "columns":                       # the queries are the last tokens of one sequence
        reps = max(1, -(-many * 16 // (nq * hq)))
        out = once(*lsa.kv8_attn(q.repeat(reps, 1, 1), kv, wide(reps, tokens), i32([n] * reps), cu=i32(np.arange(reps + 1) * nq)), reps)
        return out + ([np.arange(n - nq + i + 1) for i in range(nq)],)
    reps = max(1, -(-many // rows))
    step = nq if many else 4
    out = []
    for a in range(0, nq, step):
        x = q[a:a + step].repeat(reps, 1, 1)
        if kind == "one":
            r = lsa.kv8_attn(x, kv, wide(len(x), tokens), i32([n] * len(x)))
        else:
            idx = np.full((len(x), hkv, tokens), -1, np.int32)
            idx[:, :, :n] = np.arange(n)
            r = lsa.kv8_sparse_attn(x, kv, wide(1, n), i32([n]), torch.from_numpy(idx).cuda(), seq=i32([0] * len(x)))
        out.append(once(*r, reps))
    return torch.cat([o for o, _ in out]), torch.cat([e for _, e in out]), [np.arange(n)] * nq


def values(kv, table, fmt, h):
    """(k, v, V's scale) of the tokens of one kv-head, in 64 bits."""
    K, V, scale = host(kv)
    k, v = ref.gather(K, V, scale, table[0], fmt, h)
    return k, v, np.repeat(scale[table[0], h, 1], kv.page)


def check(got, want, tol):
    """Every element within its bound; the bounds are such that zeros would not pass."""
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert np.linalg.norm(tol) < 0.1 * np.linalg.norm(want)
    e = np.abs(got - want)
    assert (e <= tol).all(), f"{(e - tol).max()} above the bound; error {e.max()}"
