"""The paged 8-bit cache's calls refuse bad arguments before any launch: in the
binding (dtype, shape, layout, device; no GPU needed) and in the C ABI."""
import ctypes

import numpy as np
import pytest
import torch

import clustered_key_indexing_b200 as lsa
from clustered_key_indexing_b200 import _lib
from clustered_key_indexing_b200._lib import LSA_EINVAL, LSA_ENOSPACE, LSA_EUNSUPPORTED, LSA_OK, lsa_kv8

bf16, f32, i32, e4m3, i8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn, torch.int8


def z(*shape, dtype=bf16):
    return torch.zeros(shape, dtype=dtype)


def fake_cache(hkv=2, page=16, n_pages=4):
    """A KV8 over CPU arrays: its checks run, no call gets past them."""
    kv = lsa.KV8.__new__(lsa.KV8)
    K, V, scale = z(n_pages, hkv, page, 128, dtype=i8), z(n_pages, hkv, page, 128, dtype=i8), z(n_pages, hkv, 2, dtype=f32)
    kv._wrap(K, V, scale, K.data_ptr(), V.data_ptr(), scale.data_ptr(), K.get_device())
    return kv


def test_cache_arrays():
    K, s = z(4, 2, 16, 128, dtype=i8), z(4, 2, 2, dtype=f32)
    with pytest.raises(TypeError, match="K: expected one of"):
        lsa.KV8.of(z(4, 2, 16, 128, dtype=torch.uint8), K, s)
    with pytest.raises(TypeError, match="V: expected torch.int8"):
        lsa.KV8.of(K, K.view(e4m3), s)
    with pytest.raises(ValueError, match="V: expected shape"):
        lsa.KV8.of(K, z(4, 2, 32, 128, dtype=i8), s)
    with pytest.raises(ValueError, match="K: expected shape"):
        lsa.KV8.of(z(4, 2, 16, 64, dtype=i8), K, s)
    with pytest.raises(ValueError, match="scale: expected shape"):
        lsa.KV8.of(K, K, z(4, 2, dtype=f32))
    with pytest.raises(ValueError, match="page: expected one of"):
        lsa.KV8.of(z(4, 2, 24, 128, dtype=i8), z(4, 2, 24, 128, dtype=i8), s)
    with pytest.raises(ValueError, match="CUDA tensors"):
        lsa.KV8.of(K, K, s)
    for kw in (dict(fmt="fp8"), dict(page=48), dict(n_pages=0), dict(hkv=0), dict(device="cpu")):
        with pytest.raises(ValueError):
            lsa.KV8(**{**dict(n_pages=2, hkv=1), **kw})


def test_call_arguments():
    kv = fake_cache()
    table, one, lens = z(3, 5, dtype=i32), z(3, 2, 128), z(3, dtype=i32)
    with pytest.raises(TypeError, match="K: expected torch.bfloat16"):
        lsa.kv8_write(kv, one.float(), one, table, lens)
    with pytest.raises(ValueError, match="V: expected shape"):
        lsa.kv8_write(kv, one, z(3, 1, 128), table, lens)
    with pytest.raises(ValueError, match="CUDA tensors"):
        lsa.kv8_write(kv, one, one, table, lens)
    with pytest.raises(TypeError, match="Q: expected torch.bfloat16"):
        lsa.kv8_attn(z(3, 8, 128, dtype=f32), kv, table, lens)
    with pytest.raises(ValueError, match="Q: expected shape"):
        lsa.kv8_attn(z(3, 8, 64), kv, table, lens)
    with pytest.raises(ValueError, match="CUDA tensors"):
        lsa.kv8_sparse_attn(z(3, 8, 128), kv, table, lens, z(3, 2, 7, dtype=i32))
    with pytest.raises(ValueError, match="page numbers must be in"):
        lsa.kv8_copy_pages(kv, [0, 4], [1, 2])
    with pytest.raises(ValueError, match="one length"):
        lsa.kv8_copy_pages(kv, [0, 1], [2])
    with pytest.raises(ValueError, match="list of page numbers"):
        lsa.kv8_copy_pages(kv, [0.5], [1])


@pytest.fixture(scope="module")
def L():
    from clustered_key_indexing_b200.build import build
    build()
    return _lib.lib()


@pytest.mark.skipif(torch.cuda.is_available(), reason="passes fake device addresses: runs only where no GPU is present")
def test_abi_refusals(L):
    f = ctypes.c_void_p(0x10000)
    odd = ctypes.c_void_p(0x10008)

    def cache(**kw):
        return ctypes.byref(lsa_kv8(**{**dict(fmt=0, hkv=2, page=64, n_pages=8, K=0x10000, V=0x20000, scale=0x30000), **kw}))

    def write(kv=None, K=f, ks=256, V=f, vs=256, n=3, cu=None, start=f, table=f, n_seq=3, mp=4):
        return L.lsa_kv8_write(kv or cache(), K, ks, V, vs, n, cu, start, table, n_seq, mp, None)

    for kw, want in ((dict(fmt=2), LSA_EINVAL), (dict(hkv=0), LSA_EINVAL), (dict(n_pages=0), LSA_EINVAL),
                     (dict(page=48), LSA_EUNSUPPORTED), (dict(page=512), LSA_EUNSUPPORTED), (dict(K=None), LSA_EINVAL),
                     (dict(scale=None), LSA_EINVAL), (dict(V=0x10010), LSA_EINVAL), (dict(scale=0x10004), LSA_EINVAL),
                     (dict(n_pages=1 << 30), LSA_EUNSUPPORTED), (dict(hkv=70000), LSA_EUNSUPPORTED)):
        assert write(cache(**kw)) == want, kw
    assert L.lsa_kv8_write(None, f, 256, f, 256, 3, None, f, f, 3, 4, None) == LSA_EINVAL
    for kw in (dict(n=-1), dict(n_seq=-1), dict(mp=-1), dict(n=4), dict(K=None), dict(V=None), dict(start=None),
               dict(table=None), dict(ks=128), dict(vs=260), dict(K=odd), dict(V=odd)):
        assert write(**kw) == LSA_EINVAL, kw
    assert write(n=1 << 40, cu=f) == LSA_EUNSUPPORTED
    assert write(n=0, cu=f) == LSA_OK and write(n=0, n_seq=0) == LSA_OK

    def attn(kv=None, Q=f, qs=8 * 128, nq=3, hq=8, cu=None, table=f, lens=f, n_seq=3, mp=4, S=0, W=0, O=f, lse=f, ws=f,
             nws=1 << 30):
        return L.lsa_kv8_attn(kv or cache(), Q, qs, nq, hq, cu, table, lens, n_seq, mp, S, W, O, lse, ws, nws, None)

    for kw in (dict(Q=None), dict(table=None), dict(lens=None), dict(O=None), dict(nq=-1), dict(n_seq=-1), dict(mp=-1),
               dict(S=-1), dict(W=-1), dict(nq=4), dict(hq=9), dict(qs=512), dict(qs=1028), dict(Q=odd), dict(O=odd),
               dict(ws=odd), dict(n_seq=0, cu=f)):
        assert attn(**kw) == LSA_EINVAL, kw
    assert attn(hq=6) == LSA_EUNSUPPORTED and attn(hq=32) == LSA_EUNSUPPORTED
    assert attn(mp=1 << 26) == LSA_EUNSUPPORTED
    assert attn(nq=0, n_seq=0) == LSA_OK and attn(nq=0, cu=f) == LSA_OK
    need = L.lsa_kv8_attn_workspace_bytes(cache(), 3, 8, 1, 3, 4000, 0, 0)
    assert need > 0 and L.lsa_kv8_attn_workspace_bytes(cache(), 3, 8, 1, 3, 4, 0, 0) == 0
    assert L.lsa_kv8_attn_workspace_bytes(cache(), 3, 8, 1, 3, 4000, 4, 600) == 0
    assert attn(mp=4000, nws=need - 1) == LSA_ENOSPACE and attn(mp=4000, ws=None) == LSA_ENOSPACE

    def lists(Q=f, nq=3, hq=8, seq=None, n_seq=3, idx=f, n_idx=40000, ws=f, nws=1 << 30):
        return L.lsa_kv8_sparse_attn(cache(), Q, 8 * 128, nq, hq, seq, f, f, n_seq, 4, idx, n_idx, f, f, ws, nws, None)

    for kw in (dict(Q=None), dict(idx=None), dict(n_idx=-1), dict(nq=4), dict(nq=-1), dict(n_seq=0, seq=f)):
        assert lists(**kw) == LSA_EINVAL, kw
    assert lists(hq=6) == LSA_EUNSUPPORTED and lists(n_idx=2 ** 31 - 1) == LSA_EUNSUPPORTED
    assert lists(nq=0, n_seq=0) == LSA_OK
    assert lists(nws=0) == LSA_ENOSPACE and lists(ws=None) == LSA_ENOSPACE
    assert L.lsa_kv8_sparse_attn_workspace_bytes(cache(), 3, 8, 100) == 0
    assert L.lsa_kv8_sparse_attn_workspace_bytes(cache(), 100000, 8, 5000) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="passes fake device addresses: runs only where no GPU is present")
def test_abi_copy_refusals(L):
    kv = ctypes.byref(lsa_kv8(0, 2, 64, 100, 0x10000, 0x20000, 0x30000))

    def copy(src, dst, n=None):
        s, d = (np.array(x, np.int32) for x in (src, dst))
        return L.lsa_kv8_copy_pages(kv, s.ctypes.data, d.ctypes.data, len(src) if n is None else n, None)

    assert copy([], []) == LSA_OK
    for src, dst in (([0], [100]), ([100], [0]), ([-1], [0]), ([0], [-1]), ([1, 2], [3, 3]), ([1, 2], [2, 4]),
                     ([5], [5]), ([7, 8], [9, 7])):
        assert copy(src, dst) == LSA_EINVAL, (src, dst)
        assert b"lsa_kv8_copy_pages" in L.lsa_last_error()
    assert copy([0], [1], n=-1) == LSA_EINVAL and copy([0], [1], n=101) == LSA_EINVAL
    assert L.lsa_kv8_copy_pages(kv, None, None, 1, None) == LSA_EINVAL


@pytest.mark.skipif(torch.cuda.is_available(), reason="passes fake device addresses: runs only where no GPU is present")
def test_decode_refusals(L):
    cfg = _lib.lsa_cfg()
    L.lsa_cfg_default(ctypes.byref(cfg))
    f = ctypes.c_void_p(0x10000)

    def state(kv=(), **kw):
        d = _lib.lsa_decode()
        d.batch, d.hkv, d.hq, d.cap, d.U_blk = 2, 2, 8, 1024, 0x10000
        c = d.cache
        c.hkv, c.cap_units, c.cap_buckets = 4, 256, 128
        for a in ("bucket_of_unit", "members", "offsets", "cnt_lr", "minlr", "maxpos", "sum", "cent", "units"):
            setattr(c, a, 0x10000)
        d.kv8 = ctypes.pointer(lsa_kv8(**{**dict(fmt=0, hkv=2, page=64, n_pages=64, K=0x10000, V=0x20000, scale=0x30000), **dict(kv)}))
        d.kv8_table, d.kv8_max_pages = 0x10000, 16
        for k, v in kw.items():
            setattr(d, k, v)
        return ctypes.byref(d)

    def step(d, q=f, ws=f, nws=1 << 40):
        return L.lsa_decode_step(d, q, f, f, f, f, ctypes.byref(cfg), f, None, ws, nws, None)

    assert L.lsa_decode_workspace_bytes(ctypes.byref(cfg), state()) > 0
    for d, want in ((state(kv8_max_pages=15), LSA_EINVAL), (state(kv8_table=None), LSA_EINVAL), (state(dict(hkv=4)), LSA_EINVAL),
                    (state(dict(fmt=3)), LSA_EINVAL), (state(dict(page=40)), LSA_EUNSUPPORTED), (state(U_blk=None), LSA_EINVAL),
                    (state(shared_len=512, K_shared=0x10000, V_shared=0x10000), LSA_EINVAL)):
        assert step(d) == want
        assert L.lsa_decode_workspace_bytes(ctypes.byref(cfg), d) == 0
    assert step(state(), q=ctypes.c_void_p(0x10008)) == LSA_EINVAL
    assert step(state(), ws=ctypes.c_void_p(0x10008)) == LSA_EINVAL
    assert step(state(), nws=100) == LSA_ENOSPACE
    load = lambda d, n=600: L.lsa_decode_load(d, 0, n, f, ctypes.byref(cfg), f, 1 << 40, None)  # noqa: E731
    assert load(state()) == LSA_EINVAL and b"prompt" in L.lsa_last_error()
    assert load(state(K=0x10008, V=0x10000)) == LSA_EINVAL
