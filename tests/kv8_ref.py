"""The paged 8-bit cache and its attentions written out in 64 bits (numpy),
for the tests of the library's kernels."""
import numpy as np

D = 128
QMAX = {"e4m3": 448.0, "int8": 127.0}
E4M3 = np.array([(-1.0) ** (c >> 7) * ((c & 7) * 2.0 ** -9 if (c >> 3) & 15 == 0
                                       else (8 + (c & 7)) * 2.0 ** (((c >> 3) & 15) - 10)) for c in range(256)])
E4M3[0x7F] = E4M3[0xFF] = np.nan


def values(codes: np.ndarray, fmt: str) -> np.ndarray:
    """Values of codes (uint8 bytes), without their scale."""
    return E4M3[codes] if fmt == "e4m3" else codes.view(np.int8).astype(np.float64)


def encode(y: np.ndarray, fmt: str) -> np.ndarray:
    """Codes of values already divided by their scale: nearest, ties to even,
    saturating; NaN is 0x7F (either sign) in e4m3 and 0 in int8."""
    y = np.asarray(y, np.float64)
    if fmt == "int8":
        return np.clip(np.rint(np.nan_to_num(y, nan=0.0, posinf=127.0, neginf=-127.0)), -127, 127).astype(np.int8).view(np.uint8)
    a = np.minimum(np.abs(np.nan_to_num(y, nan=0.0, posinf=448.0, neginf=-448.0)), 448.0)
    grid = E4M3[:0x7F]                                   # ascending, 0 .. 448
    hi = np.clip(np.searchsorted(grid, a, side="left"), 1, 0x7E)
    lo = hi - 1
    up = (a - grid[lo] > grid[hi] - a) | ((a - grid[lo] == grid[hi] - a) & (hi % 2 == 0))
    c = np.where(up, hi, lo).astype(np.uint8)
    return np.where(np.isnan(y), 0x7F, c | (np.signbit(y).astype(np.uint8) << 7)).astype(np.uint8)


def scale_of(amax: np.ndarray, fmt: str) -> np.ndarray:
    """Smallest 2^e, e >= -100, with amax <= 2^e QMAX."""
    out = np.full(amax.shape, 2.0 ** -100)
    for e in range(-99, 121):
        out = np.where(amax > 2.0 ** (e - 1) * QMAX[fmt], 2.0 ** e, out)
    return out


def write(K, V, scale, k, v, table, start, cu, fmt):
    """In place: pools of bytes [n_pages, hkv, page, 128], scale [n_pages,
    hkv, 2], new rows k, v [n, hkv, 128] (values), as lsa_kv8_write."""
    page = K.shape[2]
    for b in range(len(start)):
        rows = range(cu[b], cu[b + 1])
        if len(rows) == 0:
            continue
        s, e = start[b], start[b] + len(rows)
        for pg in range(s // page, (e - 1) // page + 1):
            pid = table[b][pg]
            r0, r1 = max(0, s - pg * page), min(page, e - pg * page)
            t0 = cu[b] + pg * page + r0 - s
            for i, (P, x) in enumerate(((K, k), (V, v))):
                new = x[t0:t0 + r1 - r0].transpose(1, 0, 2)          # [hkv, rows, 128]
                need = scale_of(np.where(np.isfinite(new), np.abs(new), 0.0).max((1, 2)), fmt)
                for h in range(K.shape[1]):
                    sc = need[h]
                    if r0 > 0:
                        old = scale[pid, h, i]
                        sc = max(old, sc)
                        if sc > old:
                            P[pid, h, :r0] = encode(values(P[pid, h, :r0], fmt) * (old / sc), fmt)
                    P[pid, h, r0:r1] = encode(new[h] / sc, fmt)
                    scale[pid, h, i] = sc


def gather(K, V, scale, pages, fmt, h):
    """Values of a sequence's K and V rows of one head, in order."""
    return tuple((values(P[pages, h], fmt) * scale[pages, h, i][:, None, None]).reshape(-1, D) for i, P in enumerate((K, V)))


def attend(q, k, v, vtop):
    """q [G, 128] over keys k, v [n, 128]: (o, lse base 2, bound on o's error,
    bound on lse's error).  vtop: the largest value V's scales can stand for.

    The bounds: a score is a sum of 128 exact products in fp32 and a few
    roundings of it, so it is off by at most d = 2^-23 (128 + 8) S with S the
    largest sum of |q k| / sqrt(128) (tensor cores may truncate: a step, not
    half), plus 2^-25 of Q's largest element against each k; probabilities
    are off by 2 d relatively and are rounded to fp16 (2^-11); sums of n terms
    in fp32 are off by (n + 16) 2^-23 of the sum of magnitudes (A for o); o is
    rounded to bf16 (2^-8).  Below fp16's normal range a probability's rounding
    is 2^-25 absolutely, where the largest possible one is held as 2^12 and V
    as its code times its scale: at most 2^-37 vtop / l a key."""
    G, n = q.shape[0], k.shape[0]
    if n == 0:
        return np.zeros((G, D)), np.full(G, -np.inf), np.zeros((G, D)), np.zeros(G)
    x = q @ k.T / np.sqrt(D)
    S = (np.abs(q) @ np.abs(k).T).max(1) / np.sqrt(D) + np.abs(q).max(1) * np.abs(k).sum(1).max() * 0.25 / np.sqrt(D)
    m = x.max(1, keepdims=True)
    p = np.exp(x - m)
    l = p.sum(1, keepdims=True)
    o, A = p @ v / l, p @ np.abs(v) / l
    d = 2.0 ** -23 * 136 * S + (n / 16 + 16) * 2.0 ** -23
    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2 * np.expm1(np.minimum(2 * d, 50.0)))[:, None] * A + n * 2.0 ** -37 * vtop / l
    lse = (m[:, 0] + np.log(l[:, 0])) / np.log(2.0)
    return o, lse, tol, d / np.log(2.0) + np.abs(lse) * 2.0 ** -22 + 1e-6


def attn(Q, K, V, scale, table, lens, cu, fmt, sinks=0, window=0):
    """lsa_kv8_attn in 64 bits: (o, lse, bounds on both)."""
    hkv, page = K.shape[1], K.shape[2]
    nq, hq = Q.shape[:2]
    G = hq // hkv
    out = [np.zeros((nq, hq, D)), np.zeros((nq, hq)), np.zeros((nq, hq, D)), np.zeros((nq, hq))]
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        pages = table[b][:-(-lens[b] // page)]
        for h in range(hkv):
            k, v = gather(K, V, scale, pages, fmt, h)
            vtop = QMAX[fmt] * scale[pages, h, 1].max(initial=0.0)
            for i in range(n):
                t = lens[b] - n + i
                j = np.arange(max(0, t + 1))
                keep = j[(j > t - window) | (j < sinks)] if window > 0 else j
                for o, r in zip(out, attend(Q[cu[b] + i, h * G:(h + 1) * G], k[keep], v[keep], vtop)):
                    o[cu[b] + i, h * G:(h + 1) * G] = r
    return out


def lists(Q, K, V, scale, table, lens, seq, idx, fmt):
    """lsa_kv8_sparse_attn in 64 bits: (o, lse, bounds on both)."""
    hkv, page = K.shape[1], K.shape[2]
    nq, hq = Q.shape[:2]
    G = hq // hkv
    out = [np.zeros((nq, hq, D)), np.zeros((nq, hq)), np.zeros((nq, hq, D)), np.zeros((nq, hq))]
    for i in range(nq):
        b = seq[i]
        for h in range(hkv):
            j = idx[i, h][idx[i, h] >= 0]
            j = j[j < lens[b]]
            pid = np.asarray(table[b], np.int64)[j // page]
            k, v = (values(P[pid, h, j % page], fmt) * scale[pid, h, c][:, None] for c, P in enumerate((K, V)))
            for o, r in zip(out, attend(Q[i, h * G:(h + 1) * G], k, v, QMAX[fmt] * scale[pid, h, 1].max(initial=0.0))):
                o[i, h * G:(h + 1) * G] = r
    return out
