"""Batches over the 8-bit cache that are padded: queries that no sequence
claims."""
import numpy as np
import pytest
import torch

from kv8_forms import bf16, i32, one_sequence

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import clustered_key_indexing_b200 as m
    m.check_device_error()
    return m


@pytest.mark.parametrize("tokens", [300, 3000, 64000])   # what the table has room for: a CTA or cluster a row, pieces
@pytest.mark.parametrize("new", [[1, 0, 2], [5, 7, 0], [1, 1, 1]])
@pytest.mark.parametrize("G", [1, 8])
def test_rows_that_no_sequence_claims_are_left_as_they_were(lsa, G, new, tokens):
    rng = np.random.default_rng(sum(new) + tokens)
    n, page, first, behind = 300, 32, 2, 3
    kv, table = one_sequence(lsa, rng.standard_normal((n, 1, 128)), rng.standard_normal((n, 1, 128)), page, "e4m3")
    wide = np.full((3, -(-tokens // page)), -1, np.int32)
    wide[:, :table.shape[1]] = table
    cu = first + np.concatenate([[0], np.cumsum(new)])
    nq = int(cu[-1]) + behind
    q, _ = bf16(rng.standard_normal((nq, G, 128)))
    O = torch.full((nq, G, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((nq, G), -3.0, device="cuda")
    lsa.kv8_attn(q, kv, i32(wide), i32([n, 40, 9]), cu=i32(cu), O=O, lse=lse)
    mine = slice(first, int(cu[-1]))
    o, e = lsa.kv8_attn(q[mine], kv, i32(wide), i32([n, 40, 9]), cu=i32(cu - first))
    assert torch.isfinite(o.float()).all() and torch.isfinite(e).all()
    assert torch.allclose(O[mine].float(), o.float(), rtol=2.0 ** -7, atol=2.0 ** -9) and torch.allclose(lse[mine], e, atol=1e-4)
    for rows in (slice(0, first), slice(int(cu[-1]), nq)):
        assert (O[rows] == 7.0).all() and (lse[rows] == -3.0).all()
    lsa.check_device_error()
