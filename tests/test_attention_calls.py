"""Attention's entry points on the host."""
import ctypes
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))

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


@pytest.fixture(scope="module")
def fake_runtime(L, tmp_path_factory):
    """tests/fake_cudart.c, compiled."""
    from gemm_q1_q8_gb300 import build
    so = str(tmp_path_factory.mktemp("fake") / "libfake.so")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build._nvcc()))), "include")
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-I", include, "-o", so, os.path.join(HERE, "fake_cudart.c")], check=True)
    return so


ON_DEVICES = """
import ctypes, sys
fake, lib, call = ctypes.CDLL(sys.argv[1]), ctypes.CDLL(sys.argv[2]), sys.argv[3]
X, F, LL = ctypes.c_void_p(0x1000), ctypes.c_float, ctypes.c_longlong
def attn(type, max_q, hd, cap):
    w = LL(4 * hd)
    return lib.gq_attn_q8_0(X, w, X, w, type, X, 9, 64, X, 4, X, X, None, 2, max_q, 256, 4, 2, hd, F(0.1), F(cap), X, None)
calls = {
    "attn": lambda: [attn(t, q, hd, cap) for t in (0, 1, 2) for q in (1, 3, 40, 300) for hd in (64, 128, 256) for cap in (0.0, 5.0)],
    "prefill": lambda: [lib.q1s32_q8_gemm(X, X, X, X, X, X, M, 300, 256, 3, None) for M in (64, 333)],
}[call]
for device in (0, 1, 0, 3, 1):
    fake.fake_set_device(device)
    assert not any(calls()), (device, calls())
raised = fake.fake_raised()
for device in (0, 1, 3):
    fake.fake_set_device(device)
    assert not any(calls())
assert fake.fake_raised() == raised, "raised again where it had been"
"""


@pytest.mark.parametrize("call", ["attn", "prefill"])
def test_on_every_device_of_a_process(fake_runtime, call):
    """The shared-memory limit belongs to the device: each device's first call raises it, and no later one again."""
    from gemm_q1_q8_gb300 import build
    r = subprocess.run([sys.executable, "-c", ON_DEVICES, fake_runtime, build.LIB, call], env=dict(os.environ, LD_PRELOAD=fake_runtime),
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_rope_table_on_the_host_is_refused():
    """A kernel is never given a host address."""
    import gemm_q1_q8_gb300 as gq
    with pytest.raises(gq.GQError, match="expected a CUDA tensor"):
        gq.rope_table(4, 64, device="cpu")
