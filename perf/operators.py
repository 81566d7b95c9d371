"""Cases of the paged 8-bit key/value cache: writing tokens into its pages, attention of new tokens over a whole
sequence, attention over index lists, and copies of pages.

The cache of one layer: `page` consecutive tokens of a sequence share a page.  K and V are pools of codes
[n_pages, hkv, page, 128] (e4m3 or int8), scale is [n_pages, hkv, 2] (K's and V's), powers of two; the value of a
code is code * scale.  A sequence's page numbers stand in its row of `table`, in order.
"""
import math

import torch

own = False

D = 128
QMAX = {"e4m3": 448.0, "int8": 127.0}
MIN_EXP = -100  # smallest exponent of a page's scale
DEV = "cuda"


def listed():
    return [
        # one decoded token of one request goes into its open page: the smallest call, all latency
        dict(name="write-append-1", op="write", fmt="e4m3", n_seq=1, new=1, old=4001, ragged=0.0, hkv=8, page=64),
        # one decoded token of each of 32 requests whose open pages are filled to different heights
        dict(name="write-append-32", op="write", fmt="int8", n_seq=32, new=1, old=8190, ragged=0.7, hkv=8, page=64),
        # a whole 128K-token prompt of one layer
        dict(name="write-prompt-128k", op="write", fmt="e4m3", n_seq=1, new=131072, old=0, ragged=0.0, hkv=8, page=64),
        # decode over a short sequence of an odd length, one kv-head with 4 query heads
        dict(name="attn-1x777", op="attn", fmt="e4m3", n_seq=1, new=1, len=777, ragged=0.0, hkv=1, G=4, page=16, sinks=0, window=0),
        # a batch of 32 requests of different lengths up to 32K
        dict(name="attn-32x32k", op="attn", fmt="e4m3", n_seq=32, new=1, len=32768, ragged=0.9, hkv=8, G=4, page=64, sinks=0, window=0),
        # one request with a million tokens: the cache's one pass over HBM
        dict(name="attn-1x1m", op="attn", fmt="int8", n_seq=1, new=1, len=1 << 20, ragged=0.0, hkv=8, G=4, page=64, sinks=0, window=0),
        # five drafted tokens a request are checked at once, in a layer with sinks and a sliding window
        dict(name="attn-drafts-16x9k", op="attn", fmt="int8", n_seq=16, new=5, len=9001, ragged=0.8, hkv=2, G=8, page=32, sinks=4, window=1024),
        # decode over selected keys, the small decode batch: 4 sinks, 256 long-range keys, a window of 600
        dict(name="lists-decode-3x4k", op="lists", fmt="e4m3", n_seq=3, new=1, len=4096, ragged=0.3, hkv=2, G=4, page=64, k=256, sinks=4, window=600),
        # decode over selected keys, 32 requests, 2048 long-range keys each
        dict(name="lists-decode-32x32k", op="lists", fmt="e4m3", n_seq=32, new=1, len=32768, ragged=0.5, hkv=8, G=4, page=64, k=2048, sinks=4, window=1024),
        # a chunk of 1000 prompt positions over selected keys of a 128K-token context
        dict(name="lists-prefill-1000", op="lists", fmt="e4m3", n_seq=1, new=1000, len=131072, ragged=0.0, hkv=8, G=4, page=64, k=2048, sinks=4, window=1024),
        # four requests fork: their open pages are copied
        dict(name="copy-fork-4", op="copy", fmt="e4m3", pairs=4, n_pages=512, hkv=8, page=64),
        # compaction moves 4096 pages
        dict(name="copy-compact-4096", op="copy", fmt="int8", pairs=4096, n_pages=12288, hkv=8, page=64),
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["write", "attn", "attn", "lists", "lists", "copy"])
    c = dict(op=op, fmt=rng.choice(["e4m3", "int8"]), hkv=rng.choice([1, 2, 4, 8]), page=rng.choice([16, 32, 64, 128, 256]))
    if op == "copy":
        c["pairs"] = log(1, 4096 * 512 // (c["hkv"] * c["page"]) // 2 if c["hkv"] * c["page"] > 512 else 4096)
        c["n_pages"] = 2 * c["pairs"] + rng.randrange(1, 100)
        return c
    c["n_seq"] = log(1, 64)
    c["ragged"] = rng.choice([0.0, rng.uniform(0.1, 1.0)])
    if op == "write":
        c["new"] = rng.choice([1, log(1, max(1, 131072 * 8 // (c["hkv"] * c["n_seq"]) // 2))])
        c["old"] = log(1, max(2, 262144 // (c["hkv"] * c["n_seq"]))) - 1
        return c
    c["G"] = rng.choice([1, 2, 4, 8])
    if op == "attn":
        c["len"] = log(1, 4194304 // (c["hkv"] * c["n_seq"]))
        c["new"] = rng.choice([1, 1, rng.randrange(1, 9)])
        c["sinks"], c["window"] = rng.choice([(0, 0), (0, 0), (rng.randrange(0, 9), log(1, 4096))])
        return c
    c["len"] = log(1, 1048576 // (c["hkv"] * c["n_seq"]))
    c["new"] = rng.choice([1, 1, log(1, max(1, 1000 // c["n_seq"]))])
    c["k"], c["sinks"], c["window"] = 4 * log(4, 512), rng.randrange(0, 9), log(1, 1024)
    return c


# ------------------------------------------------------------------ inputs


def _sizes(top, case, least):
    """A size of each sequence: `top` for the first, the others smaller by up to the share case["ragged"]."""
    return [max(least, int(round(top * (1.0 - case["ragged"] * ((b * 0.6180339887) % 1.0))))) for b in range(case["n_seq"])]


def _lens(case):
    """(tokens held before the call's new ones or None, new tokens, tokens in all) of each sequence."""
    new = _sizes(case["new"], case, 1)
    if case["op"] == "write":
        old = _sizes(case["old"], case, 0)
        return old, new, [a + b for a, b in zip(old, new)]
    total = _sizes(case["len"], case, 1)
    new = [min(a, b) for a, b in zip(new, total)]
    return None, new, total


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _codes_of(y, fmt):
    """Codes of values that are already divided by their scale (round to nearest, ties to even, saturating)."""
    top = QMAX[fmt]
    if fmt == "e4m3":
        return y.clamp(-top, top).to(torch.float8_e4m3fn)
    return torch.nan_to_num(y, nan=0.0).round().clamp(-top, top).to(torch.int8)


def _scale_of(amax, fmt):
    """Smallest power of two s >= 2^MIN_EXP with amax <= s * QMAX."""
    m, e = torch.frexp(amax)
    e = e - 9 + (m > 0.875).to(e.dtype) if fmt == "e4m3" else e - 7 + (m > 127.0 / 128.0).to(e.dtype)
    e = torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)
    return torch.ldexp(torch.ones_like(amax), e)


def _pool(g, n_pages, hkv, page, fmt):
    """A filled pool: normal values whose size differs from page to page."""
    dt = torch.float8_e4m3fn if fmt == "e4m3" else torch.int8
    K = torch.empty(n_pages, hkv, page, D, dtype=dt, device=DEV)
    V = torch.empty_like(K)
    scale = torch.empty(n_pages, hkv, 2, dtype=torch.float32, device=DEV)
    step = max(1, (1 << 28) // (hkv * page * D))
    for i, P in enumerate((K, V)):
        for a in range(0, n_pages, step):
            x = torch.randn(min(step, n_pages - a), hkv, page, D, generator=g, device=DEV)
            x *= torch.exp2(torch.rand(x.shape[0], hkv, 1, 1, generator=g, device=DEV) * 2 - 1)
            s = _scale_of(x.abs().amax((2, 3)), fmt)
            scale[a:a + step, :, i] = s
            P[a:a + step] = _codes_of(x / s[:, :, None, None], fmt)
    return K, V, scale


def _table(g, total, page, spare=3):
    """Pages of every sequence, scattered over the pool; places behind a sequence's last page hold -1."""
    need = [-(-n // page) for n in total]
    n_pages, width = sum(need) + spare, max(1, max(need))
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(total), width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, n_pages


def _lists(g, case, new, total):
    """Index lists as the selection gives them: sinks, runs of four long-range keys ascending, the window; -1 pads."""
    S, k, W, hkv = case["sinks"], case["k"], case["window"], case["hkv"]
    t = torch.cat([torch.arange(n - m, n) for m, n in zip(new, total)]).to(DEV)[:, None, None]  # the queries' positions
    nq, runs = t.shape[0], k // 4
    s = torch.arange(S, device=DEV)
    sinks = torch.where(s <= t, s, -1).expand(nq, hkv, S)
    units = ((t - W + 1 - S).clamp(min=0) // 4)  # whole runs between the sinks and the window
    j = torch.arange(runs, device=DEV)
    lo, hi = j * units // runs, (j + 1) * units // runs
    u = lo + (torch.rand(nq, hkv, runs, generator=g, device=DEV) * (hi - lo)).long().clamp(max=(hi - lo - 1).clamp(min=0))
    u = torch.where(units > runs, u, torch.where(j < units, j, -1))
    keys = torch.where(u[..., None] >= 0, S + 4 * u[..., None] + torch.arange(4, device=DEV), -1).reshape(nq, hkv, k)
    w0 = (t - W + 1).clamp(min=S)
    w = w0 + torch.arange(W, device=DEV)
    window = torch.where(w <= t, w, -1).expand(nq, hkv, W)
    return torch.cat([sinks, keys, window], 2).to(torch.int32).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    hkv, page, fmt = case["hkv"], case["page"], case["fmt"]
    if case["op"] == "copy":
        K, V, scale = _pool(g, case["n_pages"], hkv, page, fmt)
        order = torch.randperm(case["n_pages"], generator=g, device=DEV)[:2 * case["pairs"]].to(torch.int32).cpu().numpy()
        return dict(case=case, K=K, V=V, scale=scale, src=order[:case["pairs"]].copy(), dst=order[case["pairs"]:].copy())
    old, new, total = _lens(case)
    table, n_pages = _table(g, total, page)
    K, V, scale = _pool(g, n_pages, hkv, page, fmt)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s = dict(case=case, K=K, V=V, scale=scale, table=table, cu=_i32(cu) if cu[-1] != len(new) else None)
    if case["op"] == "write":
        s["start"] = _i32(old)
        for name in ("k", "v"):
            x = torch.randn(cu[-1], hkv, D, generator=g, device=DEV)
            x *= torch.exp2(torch.rand(cu[-1], 1, 1, generator=g, device=DEV) * 4 - 2)
            s[name] = x.to(torch.bfloat16)
        return s
    s["lens"], s["max_new"] = _i32(total), max(new)
    s["q"] = (torch.randn(cu[-1], hkv * case["G"], D, generator=g, device=DEV) * 1.5).to(torch.bfloat16)
    if case["op"] == "lists":
        s["idx"] = _lists(g, case, new, total)
        s["seq"] = None if s["cu"] is None else torch.repeat_interleave(torch.arange(len(new), device=DEV), torch.tensor(new, device=DEV)).to(torch.int32)
    return s


# ------------------------------------------------------------- plain forms


def _bytes(codes):
    return codes.view(torch.uint8)


def _take(codes, *at):
    """Rows of a pool of codes, as fp32 values without their scale."""
    return _bytes(codes)[at].view(codes.dtype).float()


def _write_plain(s):
    K, V, scale, table, start, fmt = s["K"], s["V"], s["scale"], s["table"].long(), s["start"].long(), s["case"]["fmt"]
    n, n_seq, page = s["k"].shape[0], table.shape[0], K.shape[2]
    if s["cu"] is None:
        seq, within, count = torch.arange(n, device=DEV), torch.zeros(n, dtype=torch.long, device=DEV), torch.ones(n_seq, dtype=torch.long, device=DEV)
    else:
        cu = s["cu"].long()
        seq = torch.searchsorted(cu, torch.arange(n, device=DEV), right=True) - 1
        within, count = torch.arange(n, device=DEV) - cu[seq], cu[1:] - cu[:-1]
    pos = start[seq] + within
    pid, row = table[seq, pos // page], pos % page
    # the page that is open at the call's start keeps its rows below r0; its scale only grows
    open_, r0 = (start % page > 0) & (count > 0), start % page
    first = table.gather(1, (start // page).clamp(max=table.shape[1] - 1)[:, None])[:, 0].clamp(min=0)
    was = torch.zeros(K.shape[0], dtype=torch.bool, device=DEV).index_fill_(0, first[open_], True)
    for i, (P, x) in enumerate(((K, s["k"]), (V, s["v"]))):
        x = x.float()
        a = torch.where(x.isfinite(), x.abs(), 0.0).amax(2)  # [n, hkv]
        top = torch.zeros(K.shape[0], K.shape[1], device=DEV).scatter_reduce_(0, pid[:, None].expand_as(a), a, "amax")
        need = _scale_of(top, fmt)
        now = scale[:, :, i].clone()
        grown = torch.where(was[:, None], torch.maximum(now, need), need)
        f, before = first[open_], _take(P, first[open_])
        again = _codes_of(before * (now[f] / grown[f])[:, :, None, None], fmt)
        kept = (torch.arange(page, device=DEV) < r0[open_][:, None])[:, None, :, None]
        _bytes(P)[f] = torch.where(kept, _bytes(again), _bytes(P)[f])
        hit = torch.zeros(K.shape[0], dtype=torch.bool, device=DEV).index_fill_(0, pid, True)
        scale[:, :, i] = torch.where(hit[:, None], grown, now)
        _bytes(P)[pid, :, row] = _bytes(_codes_of(x / scale[pid, :, i][:, :, None], fmt))
    return {"K": K, "V": V, "scale": scale}


def _softmax_v(x, mask, v):
    """(softmax over the last axis where mask holds) v and the base-2 log of the sum of exponentials."""
    x = x.masked_fill(~mask, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m.isinf(), 0.0, m)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    o = torch.where(l > 0, torch.matmul(p, v) / l, 0.0)
    return o, ((m + torch.log(l)) / math.log(2.0))[..., 0]


def _attn_plain(s):
    case, q = s["case"], s["q"].float()
    table, lens = s["table"].long(), s["lens"].long()
    n_seq, hkv, G, L, mq = table.shape[0], case["hkv"], case["G"], table.shape[1] * case["page"], s["max_new"]
    if s["cu"] is None:
        seq, within, count = torch.arange(n_seq, device=DEV), torch.zeros(n_seq, dtype=torch.long, device=DEV), torch.ones_like(lens)
    else:
        cu = s["cu"].long()
        seq = torch.searchsorted(cu, torch.arange(q.shape[0], device=DEV), right=True) - 1
        within, count = torch.arange(q.shape[0], device=DEV) - cu[seq], cu[1:] - cu[:-1]
    qp = q.new_zeros(n_seq, mq, hkv, G, D)
    qp[seq, within] = q.view(-1, hkv, G, D)
    pages = table.clamp(min=0)
    k, v = ((_take(P, pages) * s["scale"][pages][..., i, None, None]).permute(0, 2, 1, 3, 4).reshape(n_seq, hkv, L, D) for i, P in enumerate((s["K"], s["V"])))
    x = torch.matmul(qp.permute(0, 2, 1, 3, 4).reshape(n_seq, hkv, mq * G, D), k.transpose(2, 3)) / math.sqrt(D)
    t = (lens - count)[:, None] + torch.arange(mq, device=DEV)  # [n_seq, mq]
    j = torch.arange(L, device=DEV)
    mask = j <= t[..., None]
    if case["window"] > 0:
        mask = mask & ((j > t[..., None] - case["window"]) | (j < case["sinks"]))
    o, lse = _softmax_v(x, mask.repeat_interleave(G, 1)[:, None], v)
    o = o.view(n_seq, hkv, mq, G, D).permute(0, 2, 1, 3, 4)[seq, within].reshape(-1, hkv * G, D)
    lse = lse.view(n_seq, hkv, mq, G).permute(0, 2, 1, 3)[seq, within].reshape(-1, hkv * G)
    return {"o": o.to(torch.bfloat16), "lse": lse}


def _lists_plain(s):
    case, idx, table = s["case"], s["idx"].long(), s["table"].long()
    nq, hkv, page, G = idx.shape[0], case["hkv"], case["page"], case["G"]
    seq = torch.arange(nq, device=DEV) if s["seq"] is None else s["seq"].long()
    mask = (idx >= 0) & (idx < s["lens"].long()[seq][:, None, None])
    at = torch.where(mask, idx, 0)
    pid = table[seq[:, None, None], at // page].clamp(min=0)
    head = torch.arange(hkv, device=DEV)[None, :, None]
    k, v = (_take(P, pid, head, at % page) * s["scale"][pid, head][..., i, None] for i, P in enumerate((s["K"], s["V"])))
    x = torch.matmul(s["q"].float().view(nq, hkv, G, D), k.transpose(2, 3)) / math.sqrt(D)
    o, lse = _softmax_v(x, mask[:, :, None], v)
    return {"o": o.reshape(nq, hkv * G, D).to(torch.bfloat16), "lse": lse.reshape(nq, hkv * G)}


def _copy_plain(s):
    src, dst = (torch.from_numpy(s[n]).to(DEV).long() for n in ("src", "dst"))
    for P in (_bytes(s["K"]), _bytes(s["V"]), s["scale"]):
        P[dst] = P[src]
    return {"K": s["K"], "V": s["V"], "scale": s["scale"]}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"write": _write_plain, "attn": _attn_plain, "lists": _lists_plain, "copy": _copy_plain}[op](s)
    import clustered_key_indexing_b200 as lsa
    kv = lsa.KV8.of(s["K"], s["V"], s["scale"])
    if op == "write":
        lsa.kv8_write(kv, s["k"], s["v"], s["table"], s["start"], cu=s["cu"])
    elif op == "copy":
        lsa.kv8_copy_pages(kv, s["src"], s["dst"])
    elif op == "attn":
        o, lse = lsa.kv8_attn(s["q"], kv, s["table"], s["lens"], cu=s["cu"], sinks=s["case"]["sinks"], window=s["case"]["window"])
        return {"o": o, "lse": lse}
    else:
        o, lse = lsa.kv8_sparse_attn(s["q"], kv, s["table"], s["lens"], s["idx"], seq=s["seq"])
        return {"o": o, "lse": lse}
    return {"K": s["K"], "V": s["V"], "scale": s["scale"]}


# -------------------------------------------------------------- work, exact


def work(case):
    hkv, page = case["hkv"], case["page"]
    row = 2 * hkv * D  # a token's K and V codes
    if case["op"] == "copy":
        return {"bytes": 2.0 * case["pairs"] * (page * row + 8 * hkv), "flops": 0.0}
    old, new, total = _lens(case)
    n = sum(new)
    if case["op"] == "write":
        touched = sum((a + m - 1) // page - a // page + 1 for a, m in zip(old, new))
        return {"bytes": float(n * row * 3 + touched * (8 * hkv + 4)), "flops": 4.0 * n * row}
    qo = n * hkv * case["G"] * (2 * D * 2 + 4)
    if case["op"] == "attn":
        S, W = case["sinks"], case["window"]
        keys = pairs = 0
        for m, t in zip(new, total):
            keys += t if W <= 0 else min(t, min(S, t) + min(t, W + m - 1))
            pairs += sum(u + 1 if W <= 0 else min(u + 1, min(S, u + 1) + W) for u in range(t - m, t))
        return {"bytes": float(keys * row + keys // page * 8 * hkv + qo), "flops": 4.0 * D * hkv * case["G"] * pairs}
    S, k, W = case["sinks"], case["k"], case["window"]
    entries = sum(min(u + 1, S + k + W) for m, t in zip(new, total) for u in range(t - m, t))
    distinct = sum(min(t, sum(min(u + 1, S + k + W) for u in range(t - m, t))) for m, t in zip(new, total))
    return {"bytes": float(distinct * row + n * hkv * (S + k + W) * 4 + qo), "flops": 4.0 * D * hkv * case["G"] * entries}


def _round64(y, fmt):
    """The nearest value of the format to each y, in 64 bits."""
    if fmt == "int8":
        return torch.round(y).clamp(-127.0, 127.0)
    y = y.clamp(-448.0, 448.0)
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0)
    e = e + (y.abs() >= torch.exp2(e + 1)).double() - (y.abs() < torch.exp2(e)).double() * (e > -6).double()
    step = torch.exp2(e - 3)
    return torch.round(y / step) * step


def _exact_write(case, s):
    """Page by page: the new rows' largest magnitude, the scale, the kept rows at the new scale, the new rows."""
    old, new, total = _lens(case)
    page, fmt, top = case["page"], case["fmt"], QMAX[case["fmt"]]
    K, V, scale, table = s["K"].double(), s["V"].double(), s["scale"].double(), s["table"].tolist()
    at = 0
    for b in range(case["n_seq"]):
        a, z = old[b], total[b]
        lo = a // page
        hi = (z - 1) // page + 1
        pids = torch.tensor(table[b][lo:hi], device=DEV)
        for i, (P, x) in enumerate(((K, s["k"]), (V, s["v"]))):
            rows = torch.zeros((hi - lo) * page, case["hkv"], D, dtype=torch.float64, device=DEV)
            rows[a - lo * page:z - lo * page] = x[at:at + new[b]].double()
            rows = rows.view(hi - lo, page, case["hkv"], D).transpose(1, 2)
            amax = rows.abs().amax((2, 3))
            e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -130) / top))
            e = e - (torch.exp2(e - 1) * top >= amax).double()  # a logarithm that was rounded up over a whole number
            sc = torch.exp2((e + (torch.exp2(e) * top < amax).double()).clamp(min=float(MIN_EXP)))
            if a % page:
                sc[0] = torch.maximum(sc[0], scale[pids[0], :, i])
                keep = _round64(P[pids[0]] * (scale[pids[0], :, i] / sc[0])[:, None, None], fmt)
            codes = _round64(rows / sc[:, :, None, None], fmt)
            have = P[pids]
            p = torch.arange(lo * page, hi * page, device=DEV).view(hi - lo, 1, page, 1)
            have = torch.where((p >= a) & (p < z), codes, have)
            if a % page:
                have[0] = torch.where(p[0] < a, keep, have[0])
            P[pids] = have
            scale[pids, :, i] = sc
        at += new[b]
    return {"K": K, "V": V, "scale": scale} if fmt == "e4m3" else {"K": None, "V": None, "scale": scale}


def _attend64(q, k, v, keep):
    """One kv-head: q [n, G, 128], k and v [keys, 128] or [n, keys, 128], keep [n, keys]; in 64 bits."""
    if k.dim() == 2:
        k, v = k[None], v[None]
    x = (q @ k.transpose(1, 2)) * D ** -0.5
    x[~keep[:, None, :].expand_as(x)] = -math.inf
    lse = torch.logsumexp(x, -1)
    w = torch.exp(x - torch.where(lse.isinf(), 0.0, lse)[..., None])
    return w @ v, lse / math.log(2.0)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "write":
        return _exact_write(case, s)
    if case["op"] == "copy":
        if case["fmt"] == "int8":
            K = V = None
        else:
            K, V = s["K"].double(), s["V"].double()
        scale = s["scale"].double()
        for P in (K, V, scale):
            if P is not None:
                P[torch.from_numpy(s["dst"]).long().to(DEV)] = P[torch.from_numpy(s["src"]).long().to(DEV)]
        return {"K": K, "V": V, "scale": scale}
    _, new, total = _lens(case)
    hkv, G, page = case["hkv"], case["G"], case["page"]
    if sum(new) * hkv > 40000:
        return None
    o = torch.empty(sum(new), hkv, G, D, dtype=torch.float64, device=DEV)
    lse = torch.empty(sum(new), hkv, G, dtype=torch.float64, device=DEV)
    at = 0
    for b in range(case["n_seq"]):
        m, t = new[b], total[b]
        pids = s["table"][b, :-(-t // page)].long()
        pos = torch.arange(t - m, t, device=DEV)[:, None]
        for h in range(hkv):
            k, v = ((P.view(torch.uint8)[pids, h].view(P.dtype).double() * s["scale"][pids, h, i].double()[:, None, None]).reshape(-1, D)[:t] for i, P in enumerate((s["K"], s["V"])))
            q = s["q"][at:at + m, h * G:(h + 1) * G].double()
            if case["op"] == "attn":
                j = torch.arange(t, device=DEV)[None]
                keep = j <= pos
                if case["window"] > 0:
                    keep &= (j + case["window"] > pos) | (j < case["sinks"])
                o[at:at + m, h], lse[at:at + m, h] = _attend64(q, k, v, keep)
                continue
            for a in range(0, m, 256):
                ix = s["idx"][at + a:at + min(m, a + 256), h].long()
                row = ix.clamp(min=0)
                o[at + a:at + a + ix.shape[0], h], lse[at + a:at + a + ix.shape[0], h] = _attend64(q[a:a + 256], k[row], v[row], ix >= 0)
        at += m
    return {"o": o.reshape(-1, hkv * G, D), "lse": lse.reshape(-1, hkv * G)}
