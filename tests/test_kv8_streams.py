"""Streams that the paged 8-bit cache's calls are given: another device's is
refused before any launch, one of the cache's own is used."""
import types

import numpy as np
import pytest
import torch

import clustered_key_indexing_b200 as lsa
from test_kv8_binding import fake_cache


def other(dev):
    return types.SimpleNamespace(device_index=dev + 1, cuda_stream=0)


def test_page_copies_refuse_another_devices_stream():
    kv = fake_cache()
    kv.index = 0                                 # as if its arrays were on the first GPU
    with pytest.raises(ValueError, match="stream: expected one of device 0, got one of device 1"):
        lsa.kv8_copy_pages(kv, [0], [1], stream=other(0))


def bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16).cuda()


@pytest.mark.gpu
def test_calls_refuse_another_devices_stream():
    rng = np.random.default_rng(1)
    kv = lsa.KV8(4, 2, page=16)
    k, q = bf16(rng, 1, 2, 128), bf16(rng, 1, 4, 128)
    table, one = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([[0, 1]], [1]))
    idx = torch.zeros((1, 2, 3), dtype=torch.int32, device="cuda")
    before = kv.K.view(torch.uint8).clone()
    s = other(kv.index)
    for call in (lambda: lsa.kv8_write(kv, k, k, table, one, stream=s), lambda: lsa.kv8_copy_pages(kv, [0], [1], stream=s),
                 lambda: lsa.kv8_attn(q, kv, table, one, stream=s), lambda: lsa.kv8_sparse_attn(q, kv, table, one, idx, stream=s)):
        with pytest.raises(ValueError, match="stream: expected one of device"):
            call()
    assert torch.equal(kv.K.view(torch.uint8), before)
    lsa.check_device_error()


@pytest.mark.gpu
def test_writes_and_copies_on_a_stream_of_their_own():
    rng = np.random.default_rng(2)
    a, b = (lsa.KV8(6, 2, page=16, fmt="int8") for _ in range(2))
    k, v = bf16(rng, 40, 2, 128), bf16(rng, 40, 2, 128)
    table, start, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([[3, 0, 1]], [2], [0, 40]))
    lsa.kv8_write(a, k, v, table, start, cu=cu)
    lsa.kv8_copy_pages(a, [3, 0], [4, 5])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lsa.kv8_write(b, k, v, table, start, cu=cu, stream=s)
    lsa.kv8_copy_pages(b, [3, 0], [4, 5], stream=s)
    torch.cuda.synchronize()
    for x, y in ((a.K, b.K), (a.V, b.V)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert torch.equal(a.scale, b.scale)
    lsa.check_device_error()
