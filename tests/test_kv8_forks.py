"""Forks of sequences that hold reserved pages (host logic, no GPU): tokens
that something else writes into them, a decode step for one, stay out of the
fork's pages."""
import numpy as np
import pytest
import torch

import kv8_ref as ref
from clustered_key_indexing_b200._lib import LSA_ENOSPACE, LSAError
from test_kv8_pages import PAGE, check, content, pool, rows


def write(p, sid, k, v, table):
    """What a decode step does: rows into the pages that a table named earlier."""
    a = p.kv.arrays
    ref.write(a[0], a[1], a[2], k.double().numpy(), v.double().numpy(), [table], [p.len(sid)], [0, len(k)], "int8")


@pytest.mark.parametrize("held", [10, 16, 20])
def test_a_fork_between_reserve_and_advance_keeps_its_tokens(held):
    rng = np.random.default_rng(held)
    p = pool(8)
    a = p.add()
    whole = tuple(rows(rng, held) for _ in range(2))
    p.append([a], *whole, [held])
    p.reserve([a], [20])
    table = p.pages(a)                           # what the decode step was given
    b = p.fork(a)
    assert p.pages(a) == table                   # stays true
    open_ = held % PAGE > 0
    assert sum(p.ops.copied) == open_
    kept = tuple(x[:, 0].double().numpy() for x in whole)
    new = tuple(rows(rng, 20) * 1000 for _ in range(2))
    write(p, a, *new, table)
    p.advance([a], [20])
    for x, y in zip(content(p, b), kept):
        np.testing.assert_array_equal(x, y)
    assert p.len(a) == held + 20 and p.len(b) == held
    assert p.pages(a)[:held // PAGE] == p.pages(b)[:held // PAGE]
    assert not set(p.pages(a)[held // PAGE:]) & set(p.pages(b)[held // PAGE:])
    p.append([b], rows(rng, 3), rows(rng, 3), [3])
    assert sum(p.ops.copied) == open_            # the fork's open page is its own already
    p.free(a)
    p.free(b)
    assert p.free_pages == 8


def test_a_fork_after_the_reserved_tokens_shares_again():
    rng = np.random.default_rng(1)
    p = pool(8)
    a = p.add()
    p.append([a], rows(rng, 10), rows(rng, 10), [10])
    p.reserve([a], [2])
    write(p, a, rows(rng, 2), rows(rng, 2), p.pages(a))
    p.advance([a], [1])
    b = p.fork(a)                                # one token is still to come
    assert p.pages(a) != p.pages(b) and p.ops.copied == [1]
    p.advance([a], [1])
    c = p.fork(a)
    assert p.pages(a) == p.pages(c) and p.ops.copied == [1]
    p.reserve([a], [2])                          # what is reserved for tokens that are appended is used up too
    p.append([a], rows(rng, 2), rows(rng, 2), [2])
    copied = sum(p.ops.copied)
    d = p.fork(a)
    assert p.pages(a) == p.pages(d) and sum(p.ops.copied) == copied
    p.reserve([a], [2])                          # the open page again becomes its own
    p.truncate(a, p.len(a))                      # which gives it back
    e = p.fork(a)
    assert p.pages(a) == p.pages(e)
    for s in (a, b, c, d, e):
        p.free(s)
    assert p.free_pages == 8


def test_advance_refuses_pages_that_others_share():
    rng = np.random.default_rng(2)
    p = pool(8)
    a = p.add()
    p.append([a], rows(rng, 20), rows(rng, 20), [20])
    b = p.fork(a)
    for sids in ([a], [b], [a, b]):
        with pytest.raises(ValueError, match="advance"):
            p.advance(sids)
    assert p.len(a) == p.len(b) == 20
    p.advance([a, b], [0, 0])
    p.reserve([b])
    p.advance([b])
    p.advance([a])                               # its page is nobody else's now
    assert p.len(a) == p.len(b) == 21 and p.pages(a)[1] != p.pages(b)[1]
    c = p.add()
    p.reserve([c], [40])
    p.advance([c], [40])
    p.free(b)
    assert p.len(c) == 40


def test_a_fork_without_room_for_its_page_changes_nothing():
    rng = np.random.default_rng(3)
    p = pool(2)
    a = p.add()
    k, v = rows(rng, 20), rows(rng, 20)
    p.append([a], k, v, [20])
    p.reserve([a], [5])
    with pytest.raises(LSAError) as e:
        p.fork(a)
    assert e.value.status == LSA_ENOSPACE
    check(p, {a: tuple(x[:, 0].double().numpy() for x in (k, v))})
    p.truncate(a, 20)
    assert p.pages(p.fork(a)) == p.pages(a)


def test_a_dropped_copy_leaves_no_fork():
    rng = np.random.default_rng(4)
    p = pool(4)
    a = p.add()
    p.append([a], rows(rng, 20), rows(rng, 20), [20])
    p.reserve([a])
    state = (p.free_pages, p.pages(a), list(p.refs))

    def dropped(*args):
        raise RuntimeError("dropped call")

    p.ops.copy = dropped
    with pytest.raises(RuntimeError, match="dropped"):
        p.fork(a)
    assert state == (p.free_pages, p.pages(a), list(p.refs))


def test_streams_of_copies():
    """A fork's copy is made on the stream that it is given."""
    rng = np.random.default_rng(5)
    p = pool(4)
    a = p.add()
    p.append([a], rows(rng, 3), rows(rng, 3), [3])
    p.reserve([a])
    seen = []
    p.ops.copy = lambda kv, src, dst, stream: seen.append((list(src), list(dst), stream))
    b = p.fork(a, stream="side")
    assert seen == [(p.pages(a), p.pages(b), "side")]
    assert torch.is_tensor(p.table([a, b])[0])
