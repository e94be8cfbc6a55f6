"""Refusals of the products with an epilogue, the norms around a block and the log probabilities, on the host: a bad argument
launches nothing."""
import ctypes

import pytest

N = ctypes.c_void_p(0)
X = ctypes.c_void_p(0x1000)     # never dereferenced: validation fails first
Z = ctypes.c_void_p(0x9000)
O8, O2, O1 = ctypes.c_void_p(0x1008), ctypes.c_void_p(0x1002), ctypes.c_void_p(0x1001)


@pytest.fixture(scope="module")
def L():
    from gemm_q1_q8_gb300 import build
    build.build()
    import gemm_q1_q8_gb300 as gq
    return gq.lib()


def linear(L, **k):
    a = dict(w=X, act=X, rows=64, n=256, cols=3, bias=X, fn=0, r=X, rs=64, type=0, y=Z, ys=64, blocks=N, work=X) | k
    return L.q1_q8_linear(*a.values(), N)


def glu(L, **k):
    a = dict(g=X, u=X, act=X, rows=64, n=256, cols=3, bg=X, bu=X, fn=3, type=0, y=X, ys=64, blocks=X, work=X) | k
    return L.q1_q8_glu(*a.values(), N)


SIZES = [(dict(rows=0), 1), (dict(rows=(1 << 30) + 1, ys=1 << 31, blocks=N), 1), (dict(n=0), 1), (dict(n=200), 1), (dict(n=(1 << 20) + 128), 1), (dict(cols=0), 1), (dict(cols=(1 << 20) + 1), 1),
         (dict(ys=63), 1), (dict(rows=33, blocks=X), 1), (dict(type=3), 3), (dict(fn=-1), 3), (dict(fn=6), 3), (dict(act=N), 2), (dict(act=O1), 2),
         (dict(y=N, blocks=N), 2), (dict(y=O2), 2), (dict(y=O1, type=2), 2), (dict(blocks=O1), 2), (dict(work=N), 2), (dict(work=O8), 2)]


@pytest.mark.parametrize("change,expect", SIZES + [
    (dict(rs=63), 1), (dict(w=N), 2), (dict(w=O8), 2), (dict(bias=O2), 2), (dict(r=O2), 2), (dict(r=O1, type=1), 2),
    (dict(y=X, r=X, ys=96), 2)])
def test_linear_refusals(L, change, expect):
    assert linear(L, **change) == expect


@pytest.mark.parametrize("change,expect", SIZES + [(dict(g=N), 2), (dict(u=N), 2), (dict(g=O8), 2), (dict(u=O8), 2), (dict(bg=O2), 2), (dict(bu=O1), 2)])
def test_glu_refusals(L, change, expect):
    assert glu(L, **change) == expect


def norm(L, **k):
    a = dict(b=X, bs=64, x=X, xs=64, post=X, g=X, gs=64, beta=1.0, alpha=1.0, w=X, eps=1e-5, type=0, m=2, k=64, h=Z, y=X, act=X, d=X, q=X, op=X) | k
    return L.gq_rmsnorm_block(*a.values(), N)


@pytest.mark.parametrize("change,expect", [
    (dict(m=0), 1), (dict(k=0), 1), (dict(k=65568, bs=65568, xs=65568, gs=0), 1), (dict(k=33), 1), (dict(xs=63), 1), (dict(bs=63), 1),
    (dict(gs=63), 1), (dict(gs=-1), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(beta=float("inf")), 1), (dict(alpha=float("nan")), 1),
    (dict(type=3), 3), (dict(b=N), 2), (dict(x=N), 2), (dict(w=N), 2), (dict(q=N), 2), (dict(d=N), 2), (dict(d=N, q=N), 2),
    (dict(h=N, y=N, act=N, d=N, q=N, op=N), 2), (dict(act=O1), 2), (dict(q=O8), 2), (dict(op=O8), 2), (dict(b=O2), 2), (dict(post=O2), 2),
    (dict(g=O1, type=1), 2), (dict(h=X), 2), (dict(h=X, g=N, xs=128), 2), (dict(h=X, g=N, bs=128), 2)])
def test_rmsnorm_block_refusals(L, change, expect):
    assert norm(L, **change) == expect


def logprobs(L, **k):
    a = dict(x=X, s=100, type=0, m=2, v=100, scale=1.0, tok=X, lp=X, h=X, top=5, ids=X, best=X, work=X) | k
    return L.gq_logprobs(*a.values(), N)


@pytest.mark.parametrize("change,expect", [
    (dict(m=0), 1), (dict(m=(1 << 24) + 1), 1), (dict(v=0), 1), (dict(v=(1 << 20) + 1, s=1 << 21), 1), (dict(s=99), 1), (dict(top=-1), 1), (dict(top=33), 1),
    (dict(v=4), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(scale=1.1e30), 1), (dict(type=4), 3),
    (dict(x=N), 2), (dict(x=O2), 2), (dict(x=O1, type=1), 2), (dict(tok=N), 2), (dict(lp=N), 2), (dict(tok=N, lp=N, h=N, top=0), 2),
    (dict(ids=N), 2), (dict(best=N), 2), (dict(tok=ctypes.c_void_p(0x1004)), 2), (dict(ids=ctypes.c_void_p(0x1004)), 2), (dict(best=O2), 2),
    (dict(lp=O2), 2), (dict(h=O2), 2), (dict(work=N), 2), (dict(work=O8), 2)])
def test_logprobs_refusals(L, change, expect):
    assert logprobs(L, **change) == expect


def test_sizes(L):
    assert L.gq_q1_q8_linear_workspace_bytes(64, 256, 3, 0) > 0
    for bad in ((0, 256, 3, 0), (64, 200, 3, 0), (64, 0, 3, 0), (64, 256, 0, 0), (64, 256, 3, 3), (64, (1 << 20) + 128, 3, 0)):
        assert L.gq_q1_q8_linear_workspace_bytes(*bad) == 0
    assert L.gq_logprobs_workspace_bytes(1, 49152, 20) > 0 and L.gq_logprobs_workspace_bytes(4096, 1000, 0) > 0
    for bad in ((0, 100, 0), (1, 0, 0), (1, 100, 33), (1, 100, -1), (1, 3, 4), (1, (1 << 20) + 1, 0)):
        assert L.gq_logprobs_workspace_bytes(*bad) == 0


def test_binding_refuses_host_tensors():
    import torch

    import gemm_q1_q8_gb300 as gq
    x = torch.zeros(2, 64)
    for call in (lambda: gq.rmsnorm_block(x, x, torch.ones(64)), lambda: gq.rmsnorm_block_q8_0(x, x, torch.ones(64)),
                 lambda: gq.rmsnorm_block_q8_0(torch.zeros(2, 33), torch.zeros(2, 33), torch.ones(33)), lambda: gq.logprobs(x, top=1),
                 lambda: gq.logprobs(None), lambda: gq.q1_q8_linear_workspace(64, 200, 1), lambda: gq.logprobs_workspace(1, 3, 4),
                 lambda: gq.q1_q8_linear(torch.zeros(2304, dtype=torch.uint8), torch.zeros(136, dtype=torch.uint8), 8, 128, 1),
                 lambda: gq.q1_q8_glu(None, None, None, 8, 128, 1, activation="swish"),
                 lambda: gq.q1_q8_linear(None, None, 33, 128, 1, q8_0=True)):
        with pytest.raises(gq.GQError):
            call()


ON_DEVICES = """
import ctypes, sys
fake, lib = ctypes.CDLL(sys.argv[1]), ctypes.CDLL(sys.argv[2])
X, LL = ctypes.c_void_p(0x1000), ctypes.c_longlong
def calls():
    for rows, n in ((64, 256), (2560, 6912), (14336, 4096), (6400, 16384)):
        for m in (1, 9, 30, 64, 97, 400, 4096):
            for t in (0, 2):
                yield lib.q1_q8_linear(X, X, rows, n, m, None, 0, None, LL(0), t, X, LL(rows), None, X, None)
                yield lib.q1_q8_glu(X, X, X, rows, n, m, None, None, 3, t, None, LL(0), X, X, None)
for device in (0, 1, 0, 3, 1):
    fake.fake_set_device(device)
    assert not any(calls()), (device, list(calls()))
raised = fake.fake_raised()
for device in (0, 1, 3):
    fake.fake_set_device(device)
    assert not any(calls())
assert fake.fake_raised() == raised, "raised again where it had been"
"""


def test_products_on_every_device_of_a_process(L, tmp_path):
    """The shared-memory limit belongs to the device: each device's first call raises it, and no later one again."""
    import os
    import subprocess
    import sys

    from gemm_q1_q8_gb300 import build
    so, here = str(tmp_path / "libfake.so"), os.path.dirname(os.path.abspath(__file__))
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build._nvcc()))), "include")
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-I", include, "-o", so, os.path.join(here, "fake_cudart.c")], check=True)
    r = subprocess.run([sys.executable, "-c", ON_DEVICES, so, build.LIB], env=dict(os.environ, LD_PRELOAD=so), capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_workspaces_hold_what_calls_take(L):
    """The size for a call's sizes and type serves both products, whatever their outputs: at least the activations' parts where tokens are many."""
    for rows, n in ((64, 256), (2560, 2560), (14336, 4096)):
        sizes = [L.gq_q1_q8_linear_workspace_bytes(rows, n, m, t) for t in (0, 1, 2) for m in (1, 40, 500)]
        assert all(s > 0 and s % 16 == 0 for s in sizes)
        assert L.gq_q1_q8_linear_workspace_bytes(rows, n, 500, 0) >= 2 * 500 * n * 2 + 500 * 4
        assert L.gq_q1_q8_linear_workspace_bytes(rows, n, 500, 2) >= L.gq_q1_q8_linear_workspace_bytes(rows, n, 500, 0)
