"""Refusals of the operators between a layer's products, on the host: a bad argument launches nothing."""
import ctypes

import pytest

N = ctypes.c_void_p(0)
X = ctypes.c_void_p(0x1000)     # never dereferenced: validation fails first
O8, O2, O1 = ctypes.c_void_p(0x1008), ctypes.c_void_p(0x1002), ctypes.c_void_p(0x1001)


@pytest.fixture(scope="module")
def L():
    from gemm_q1_q8_gb300 import build
    build.build()
    import gemm_q1_q8_gb300 as gq
    return gq.lib()


def norm(L, **k):
    a = dict(x=X, xs=64, r=X, rs=64, w=X, eps=1e-5, type=0, m=2, k=64, h=X, y=X, act=X, d=X, q=X, op=X) | k
    return L.gq_rmsnorm(*a.values(), N)


@pytest.mark.parametrize("change,expect", [
    (dict(m=0), 1), (dict(k=0), 1), (dict(k=65568, xs=65568, rs=65568), 1), (dict(k=33), 1), (dict(xs=63), 1), (dict(rs=63), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(type=3), 3), (dict(x=N), 2), (dict(w=N), 2), (dict(q=N), 2), (dict(d=N), 2),
    (dict(d=N, q=N), 2), (dict(h=N, y=N, act=N, d=N, q=N, op=N), 2), (dict(act=O1), 2), (dict(q=O8), 2), (dict(op=O8), 2),
    (dict(x=O2), 2), (dict(r=O1, type=1), 2), (dict(h=X, x=X, xs=128), 2), (dict(h=X, x=ctypes.c_void_p(0x9000), rs=96), 2)])
def test_rmsnorm_refusals(L, change, expect):
    assert norm(L, **change) == expect


@pytest.mark.parametrize("args,expect", [
    ((X, 0, 0, X), 1), ((X, 1 << 41, 0, X), 1), ((X, 1, 7, X), 3), ((N, 1, 0, X), 2), ((O1, 1, 0, X), 2), ((X, 1, 1, O8), 2)])
def test_dequantize_refusals(L, args, expect):
    assert L.gq_dequantize_q8_0(*args, N) == expect


@pytest.mark.parametrize("args,expect", [
    ((X, 0, 64, 1e4, 0, 1.0, 0.0), 1), ((X, 4, 0, 1e4, 0, 1.0, 0.0), 1), ((X, 4, 12, 1e4, 0, 1.0, 0.0), 1), ((X, 4, 264, 1e4, 0, 1.0, 0.0), 1),
    ((X, 4, 64, 1.0, 0, 1.0, 0.0), 1), ((X, 4, 64, 1e4, 1, 0.5, 0.0), 1), ((X, 4, 64, 1e4, 3, 2.0, 0.0), 1), ((X, 4, 64, 1e4, 4, 1.0, 0.0), 3),
    ((N, 4, 64, 1e4, 0, 1.0, 0.0), 2), ((ctypes.c_void_p(0x1004), 4, 64, 1e4, 0, 1.0, 0.0), 2)])
def test_rope_table_refusals(L, args, expect):
    assert L.gq_rope_table(*args, N) == expect


def append(L, **k):
    a = dict(q=X, qs=512, qo=X, qos=512, k=X, ks=256, v=X, vs=256, type=0, rope=X, rows=10, rot=128, layout=0, pos=X, slots=X, n=3,
             hq=4, hkv=2, hd=128, cache=X, pages=4, page=64) | k
    return L.gq_rope_kv_append(*a.values(), N)


@pytest.mark.parametrize("change,expect", [
    (dict(n=0), 1), (dict(hq=-1), 1), (dict(hkv=0), 1), (dict(hd=96), 1), (dict(page=24), 1), (dict(page=0), 1), (dict(pages=0), 1),
    (dict(rot=12), 1), (dict(rot=136), 1), (dict(rot=-8), 1), (dict(rows=0), 1), (dict(qs=511), 1), (dict(qos=500), 1), (dict(ks=255), 1),
    (dict(vs=0), 1), (dict(type=5), 3), (dict(layout=2), 3), (dict(q=N), 2), (dict(qo=N), 2), (dict(k=N), 2), (dict(v=N), 2),
    (dict(slots=N), 2), (dict(pos=N), 2), (dict(cache=N), 2), (dict(cache=O8), 2), (dict(k=O8), 2), (dict(v=O8), 2), (dict(q=O8), 2),
    (dict(rope=O8), 2), (dict(ks=257), 2), (dict(qs=514), 2), (dict(qs=516), 2), (dict(slots=ctypes.c_void_p(0x1004)), 2),
    (dict(type=1, v=ctypes.c_void_p(0x1004)), 2)])
def test_append_refusals(L, change, expect):
    assert append(L, **change) == expect


@pytest.mark.parametrize("args,expect", [
    ((X, 4, 64, 2, 128, X, 0, 0, X, X), 1), ((X, 4, 60, 2, 128, X, 1, 0, X, X), 1), ((X, 4, 64, 2, 80, X, 1, 0, X, X), 1),
    ((X, 4, 64, 2, 128, X, 1, 3, X, X), 3), ((N, 4, 64, 2, 128, X, 1, 0, X, X), 2), ((X, 4, 64, 2, 128, N, 1, 0, X, X), 2),
    ((X, 4, 64, 2, 128, X, 1, 0, N, N), 2), ((X, 4, 64, 2, 128, X, 1, 0, O8, X), 2), ((O8, 4, 64, 2, 128, X, 1, 0, X, X), 2)])
def test_read_refusals(L, args, expect):
    assert L.gq_kv_read(*args, N) == expect


def attn(L, **k):
    a = dict(q=X, qs=512, o=X, os=512, type=0, cache=X, pages=9, page=64, table=X, ts=4, kv=X, start=X, tree=N, seqs=2, max_q=1, max_kv=256,
             hq=4, hkv=2, hd=128, scale=0.1, cap=0.0, work=X) | k
    return L.gq_attn_q8_0(*a.values(), N)


@pytest.mark.parametrize("change,expect", [
    (dict(seqs=0), 1), (dict(seqs=65536), 1), (dict(max_q=0), 1), (dict(max_kv=0), 1), (dict(hq=3), 1), (dict(hq=0), 1), (dict(hkv=0), 1),
    (dict(hd=32), 1), (dict(hq=130, qs=99999, os=99999), 1), (dict(page=20), 1), (dict(pages=0), 1), (dict(qs=511), 1), (dict(os=100), 1),
    (dict(ts=3), 1), (dict(tree=X, max_q=65), 1), (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1), (dict(cap=-1.0), 1),
    (dict(cap=float("inf")), 1), (dict(type=-1), 3), (dict(q=N), 2), (dict(o=N), 2), (dict(cache=N), 2), (dict(table=N), 2), (dict(kv=N), 2),
    (dict(start=N), 2), (dict(work=N), 2), (dict(q=O8), 2), (dict(o=O8), 2), (dict(work=O8), 2), (dict(cache=O8), 2), (dict(qs=514), 2),
    (dict(tree=ctypes.c_void_p(0x1004)), 2), (dict(table=O2), 2)])
def test_attn_refusals(L, change, expect):
    assert attn(L, **change) == expect


def test_sizes(L):
    assert L.gq_kv_cache_bytes(3, 64, 5, 128) == 3 * 4 * 5 * 34 * 128
    for bad in ((0, 64, 5, 128), (3, 8, 5, 128), (3, 64, 0, 128), (3, 64, 5, 100), (2 ** 31 - 1, 65536, 1, 64), (1, 16, 1025, 64)):
        assert L.gq_kv_cache_bytes(*bad) == 0
    assert L.gq_attn_workspace_bytes(4, 1, 8, 2, 128, 0) > 0
    for bad in ((0, 1, 8, 2, 128, 0), (4, 0, 8, 2, 128, 0), (4, 1, 7, 2, 128, 0), (4, 1, 8, 2, 96, 0), (4, 1, 8, 2, 128, 3)):
        assert L.gq_attn_workspace_bytes(*bad) == 0


def test_binding_refuses_host_tensors():
    import torch

    import gemm_q1_q8_gb300 as gq
    x = torch.zeros(2, 64)
    with pytest.raises(gq.GQError):
        gq.rmsnorm(x, torch.ones(64))
    with pytest.raises(gq.GQError):
        gq.rmsnorm_q8_0(torch.zeros(2, 33), torch.ones(33))
    with pytest.raises(gq.GQError):
        gq.KVCacheQ8_0(1, 16, 1, 64, data=torch.zeros(34 * 64, dtype=torch.uint8))
    with pytest.raises(gq.GQError):
        gq.KVCacheQ8_0(1, 17, 1, 64)
    with pytest.raises(gq.GQError):
        gq.rope_table(4, 64, scaling="other", device="cpu")


def test_scale_by_product_is_the_division():
    """A block's scale is amax / 127 rounded: the kernels' product, corrected by its exact remainder, for every mantissa."""
    import numpy as np
    a = (np.arange(1 << 23, dtype=np.uint32) | np.uint32(127 << 23)).view(np.float32)
    r = np.float32(1) / np.float32(127)
    q = a * r
    rem = (a.astype(np.float64) - 127.0 * q.astype(np.float64)).astype(np.float32)          # exact
    fixed = (rem.astype(np.longdouble) * np.longdouble(r) + q.astype(np.longdouble)).astype(np.float32)
    assert np.array_equal(fixed, a / np.float32(127))
