"""The sequences of a paged 8-bit cache (host logic, no GPU): random appends,
forks, truncations, frees and compactions against sequences that are kept
whole, with the device calls done in 64 bits."""
import types

import numpy as np
import pytest
import torch

import kv8_ref as ref
from clustered_key_indexing_b200._lib import LSA_ENOSPACE, LSAError
from clustered_key_indexing_b200.pages import KV8Pages

HKV, PAGE = 1, 16


class HostOps:
    """lsa_kv8_write and lsa_kv8_copy_pages on host arrays."""

    def __init__(self):
        self.fail = False
        self.copied = []

    def write(self, kv, K, V, table, start, cu, stream):
        if self.fail:
            raise RuntimeError("dropped call")
        n = table.shape[0]
        cu = list(range(n + 1)) if cu is None else cu.tolist()
        ref.write(kv.arrays[0], kv.arrays[1], kv.arrays[2], K.double().numpy(), V.double().numpy(), table.numpy(),
                  start.tolist(), cu, "int8")

    def copy(self, kv, src, dst, stream):
        assert len(set(dst)) == len(dst) and not set(src) & set(dst)
        self.copied.append(len(src))
        for a in kv.arrays:
            a[list(dst)] = a[list(src)]


def pool(n_pages):
    arrays = [np.zeros((n_pages, HKV, PAGE, 128), np.uint8), np.zeros((n_pages, HKV, PAGE, 128), np.uint8),
              np.full((n_pages, HKV, 2), 2.0 ** -100)]
    kv = types.SimpleNamespace(n_pages=n_pages, hkv=HKV, page=PAGE, device=torch.device("cpu"), arrays=arrays)
    return KV8Pages(kv, HostOps())


def rows(rng, n):
    # integers of one size: a code is the value itself, whatever page it went through
    x = rng.integers(-60, 61, (n, HKV, 128)).astype(np.float32)
    x[..., 0] = 100.0
    return torch.from_numpy(x).to(torch.bfloat16)


def content(p, sid):
    kv = p.kv
    k, v = ref.gather(kv.arrays[0], kv.arrays[1], kv.arrays[2], np.array(p.pages(sid), int), "int8", 0)
    return k[:p.len(sid)], v[:p.len(sid)]


def check(p, whole):
    refs = [0] * p.kv.n_pages
    for sid, (k, v) in whole.items():
        assert p.len(sid) == len(k)
        assert len(p.pages(sid)) == -(-len(k) // PAGE)
        for q in p.pages(sid):
            refs[q] += 1
        gk, gv = content(p, sid)
        np.testing.assert_array_equal(gk, k)
        np.testing.assert_array_equal(gv, v)
    assert refs == p.refs
    assert sorted(p._free) == [i for i, r in enumerate(refs) if r == 0]
    assert p.used_pages + p.free_pages == p.kv.n_pages


@pytest.mark.parametrize("seed", [0, 1, 2])
def test_random_life_of_sequences(seed):
    rng = np.random.default_rng(seed)
    p, whole = pool(40), {}
    for _ in range(250):
        op = rng.integers(0, 7)
        ids = list(whole)
        if op == 0 or not ids:
            whole[p.add()] = (np.zeros((0, 128)), np.zeros((0, 128)))
        elif op <= 2:
            some = [int(s) for s in rng.permutation(ids)[:rng.integers(1, 5)]]
            counts = [int(c) for c in rng.integers(0, 30, len(some))] if op == 1 else None
            n = sum(counts) if counts else len(some)
            k, v = rows(rng, n), rows(rng, n)
            need_before = (p.free_pages, [list(p.pages(s)) for s in some])
            try:
                p.append(some, k, v, counts)
            except LSAError as e:
                assert e.status == LSA_ENOSPACE
                assert need_before == (p.free_pages, [list(p.pages(s)) for s in some])
                check(p, whole)
                p.free(ids[0])
                del whole[ids[0]]
                continue
            at = 0
            for i, s in enumerate(some):
                c = counts[i] if counts else 1
                whole[s] = tuple(np.concatenate([w, x[at:at + c, 0].double().numpy()]) for w, x in zip(whole[s], (k, v)))
                at += c
        elif op == 3:
            s = int(rng.choice(ids))
            whole[p.fork(s)] = whole[s]
        elif op == 4:
            s = int(rng.choice(ids))
            p.free(s)
            del whole[s]
        elif op == 5:
            s = int(rng.choice(ids))
            n = int(rng.integers(0, p.len(s) + 1))
            p.truncate(s, n)
            whole[s] = tuple(w[:n] for w in whole[s])
        else:
            used = p.used_pages
            moved = p.compact()
            assert moved <= used and p.used_pages == used
            assert all(r > 0 for r in p.refs[:used]) and not any(p.refs[used:])
            assert p.compact() == 0
        check(p, whole)


def test_fork_copies_only_the_open_page_and_only_once_needed():
    rng = np.random.default_rng(3)
    p = pool(20)
    a = p.add()
    p.append([a], rows(rng, 40), rows(rng, 40), [40])          # two full pages and an open one
    b, c = p.fork(a), p.fork(a)
    assert p.used_pages == 3 and p.ops.copied == []
    p.append([a, b, c], rows(rng, 3), rows(rng, 3))
    assert p.ops.copied == [2]                                 # the last owner writes in place
    assert p.used_pages == 5
    assert p.pages(a)[:2] == p.pages(b)[:2] == p.pages(c)[:2]
    assert len({p.pages(s)[2] for s in (a, b, c)}) == 3
    d = p.fork(a)
    p.truncate(d, 32)                                          # ends on a page's border: nothing to copy
    p.append([d], rows(rng, 1), rows(rng, 1))
    assert p.ops.copied == [2]


def test_refusals_change_nothing():
    rng = np.random.default_rng(4)
    p = pool(4)
    a = p.add()
    p.append([a], rows(rng, 20), rows(rng, 20), [20])
    b = p.fork(a)
    state = (p.free_pages, p.pages(a), p.pages(b), list(p.refs))
    for call, err in ((lambda: p.append([a, a], rows(rng, 2), rows(rng, 2)), ValueError),
                      (lambda: p.append([99], rows(rng, 1), rows(rng, 1)), ValueError),
                      (lambda: p.append([a], rows(rng, 2), rows(rng, 2)), ValueError),
                      (lambda: p.append([a], rows(rng, 1), rows(rng, 1).float()), TypeError),
                      (lambda: p.append([a], rows(rng, 1), rows(rng, 1), [-1]), ValueError),
                      (lambda: p.append([a, b], rows(rng, 2), rows(rng, 2), [1]), ValueError),
                      (lambda: p.append([a], rows(rng, 60), rows(rng, 60), [60]), LSAError),
                      (lambda: p.truncate(a, 21), ValueError), (lambda: p.truncate(a, -1), ValueError),
                      (lambda: p.fork(7), ValueError), (lambda: p.free(7), ValueError), (lambda: p.len(7), ValueError),
                      (lambda: p.table([a], width=1), ValueError)):
        with pytest.raises(err):
            call()
        assert state == (p.free_pages, p.pages(a), p.pages(b), list(p.refs))
    p.ops.fail = True
    with pytest.raises(RuntimeError, match="dropped"):
        p.append([a, b], rows(rng, 2), rows(rng, 2))
    assert state == (p.free_pages, p.pages(a), p.pages(b), list(p.refs))
    table, lens = p.table([a, b], width=3)
    assert table.tolist() == [p.pages(a) + [-1], p.pages(b) + [-1]] and lens.tolist() == [20, 20]
    assert p.table([])[0].shape == (0, 1)
    p.append([], rows(rng, 0), rows(rng, 0))
    p.append([a], rows(rng, 0), rows(rng, 0), [0])
    assert state == (p.free_pages, p.pages(a), p.pages(b), list(p.refs))


def test_reserve_and_advance():
    rng = np.random.default_rng(6)
    p = pool(8)
    a = p.add()
    p.append([a], rows(rng, 20), rows(rng, 20), [20])
    b = p.fork(a)
    before = content(p, a)
    p.reserve([a, b], [13, 1])                                 # a third page for a, the open page copied for it
    assert p.ops.copied == [1] and len(p.pages(a)) == 3 and len(p.pages(b)) == 2
    assert p.pages(a)[0] == p.pages(b)[0] and p.pages(a)[1] != p.pages(b)[1]
    assert p.len(a) == p.len(b) == 20
    for s in (a, b):
        for x, y in zip(content(p, s), before):
            np.testing.assert_array_equal(x, y)
    p.reserve([a, b], [13, 1])                                 # it has them
    assert p.ops.copied == [1] and p.used_pages == 4
    with pytest.raises(ValueError, match="pages for 32"):
        p.advance([a, b], [5, 13])
    assert p.len(a) == 20
    p.advance([a], [13])
    p.append([a], rows(rng, 15), rows(rng, 15), [15])          # fills the reserved page
    assert p.len(a) == 48 and p.used_pages == 4
    c = p.fork(a)
    p.reserve([a], [20])
    p.truncate(a, 40)                                          # gives the reserved pages back
    assert len(p.pages(a)) == 3 and p.refs[p.pages(a)[2]] == 2
    p.free(c)
    with pytest.raises(LSAError):
        p.reserve([a], [200])
    assert len(p.pages(a)) == 3 and p.used_pages == 4


def test_sequences_may_come_from_a_generator():
    p = pool(4)
    a, b = p.add(), p.add()
    p.reserve((s for s in (a, b)), [3, 20])
    with pytest.raises(ValueError, match="advance"):
        p.advance((s for s in (a, b)), [3, 40])
    p.advance((s for s in (a, b)), [3, 20])
    assert (p.len(a), p.len(b)) == (3, 20) and p.used_pages == 3


@pytest.mark.parametrize("held", [16, 20])
def test_a_fork_does_not_share_reserved_pages(held):
    rng = np.random.default_rng(7)
    p = pool(8)
    a = p.add()
    p.append([a], rows(rng, held), rows(rng, held), [held])
    p.reserve([a], [20])
    b = p.fork(a)
    for s in (a, b):
        p.append([s], rows(rng, 20), rows(rng, 20), [20])
    assert not set(p.pages(a)[1:]) & set(p.pages(b)[1:])
    p.free(a)
    p.free(b)
    assert p.free_pages == 8
