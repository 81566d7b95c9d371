"""A fork of a sequence whose reserved tokens are still being written, on the
GPU: the fork's tokens, and the attention over them, stay what they were."""
import numpy as np
import pytest
import torch

from kv8_forms import bf16, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import clustered_key_indexing_b200 as m
    m.check_device_error()
    return m


@pytest.mark.parametrize("fmt,held", [("int8", 90), ("e4m3", 90), ("int8", 64)])
def test_a_fork_between_a_step_and_its_tokens(lsa, fmt, held):
    rng = np.random.default_rng(held)
    hkv, page = 2, 32
    pages = lsa.KV8Pages(lsa.KV8(12, hkv, page=page, fmt=fmt))
    a = pages.add()
    pages.append([a], bf16(rng.standard_normal((held, hkv, 128)))[0], bf16(rng.standard_normal((held, hkv, 128)))[0], [held])
    q = bf16(rng.standard_normal((1, hkv * 4, 128)))[0]
    first = lsa.kv8_attn(q, pages.kv, *pages.table([a]))
    pages.reserve([a], [3])
    table, lens = pages.table([a])
    b = pages.fork(a)
    k, v = (bf16(rng.standard_normal((3, hkv, 128)) * 2.0 ** 12)[0] for _ in range(2))
    cu = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    lsa.kv8_write(pages.kv, k, v, table, lens, cu=cu)      # the step, into the pages that it was given
    pages.advance([a], [3])
    for x, y in zip(lsa.kv8_attn(q, pages.kv, *pages.table([b])), first):
        assert torch.equal(x, y)
    codes = [x[pages.pages(b)].copy() for x in host(pages.kv)]
    pages.append([b], k[:1], v[:1])
    pages.append([a], k[1:2], v[1:2])
    assert not set(pages.pages(a)[held // page:]) & set(pages.pages(b)[held // page:])
    for x, y in zip(host(pages.kv), codes):                # the fork's full pages
        np.testing.assert_array_equal(x[pages.pages(b)[:held // page]], y[:held // page])
    assert pages.len(a) == held + 4 and pages.len(b) == held + 1
    lsa.check_device_error()
