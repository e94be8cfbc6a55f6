"""Attention's entry points on the host."""
import ctypes

import pytest

N = ctypes.c_void_p(0)
X = ctypes.c_void_p(0x1000)     # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def L():
    from gemm_q1_q8_gb300 import build
    build.build()
    import gemm_q1_q8_gb300 as gq
    return gq.lib()


def bounded(L, **k):
    a = dict(q=X, qs=512, o=X, os=512, type=0, cache=X, pages=9, page=64, table=X, ts=4, kv=X, start=X, tree=N, rows=7, seqs=2, max_q=1,
             max_kv=256, hq=4, hkv=2, hd=128, scale=0.1, cap=0.0, work=X) | k
    return L.gq_attn_q8_0_bounded(*a.values(), N)


@pytest.mark.parametrize("change,expect", [(dict(rows=-1), 1), (dict(seqs=0), 1), (dict(ts=3), 1), (dict(type=4), 3), (dict(work=N), 2)])
def test_bounded_attention_refusals(L, change, expect):
    assert bounded(L, **change) == expect
