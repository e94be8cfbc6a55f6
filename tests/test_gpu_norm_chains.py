"""A norm and the product that reads it, one after another into the same buffers without a pause (a CUDA graph): the product is launched while
the norm runs and must read what it wrote.  The results equal those of calls with the device idle between them, bit for bit."""
import numpy as np
import pytest
import torch

import workloads as wl
from tests.gpu_util import need_gpu, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    need_gpu()
    import gemm_q1_q8_gb300 as m
    return m


def ints(a):
    return to_dev(a.view(np.int32) if a.dtype == np.uint32 else a)


def products(gq, name, m, k):
    """(kind of activation, call(activation, out), outputs' shape) of a product over rows of k."""
    rows, rng = 640, wl.Rng(3)
    if name in ("q1_gemv", "q1_gemm", "q1_lut4", "q1_raw", "q1_f32"):
        w = wl.q1_0_weights(rng, rows, k)
        packed = gq.q1_0_pack(to_dev(w), rows, k)
        if name == "q1_gemv":
            return "q8", lambda a, y: gq.q1_q8_gemv(packed, a, rows, k, out=y[0])
        if name == "q1_raw":
            raw = to_dev(w)
            return "q8", lambda a, y: gq.q1_q8_gemv_raw(raw, a, rows, k, out=y[0])
        if name == "q1_f32":
            return "f32", lambda a, y: gq.q1_q8_gemv_f32(packed, a[0], rows, k, out=y[0])
        path = gq.PATH_LUT4 if name == "q1_lut4" else gq.PATH_AUTO
        return "q8", lambda a, y: gq.q1_q8_gemm(packed, a, rows, k, m, path=path, out=y)
    if name in ("q1s32", "q1s32_mma", "q1s32_f32", "q1s32_f32_mma"):
        signs, ws, _ = wl.prefill_inputs(rng, m, k, rows)
        signs, ws = ints(signs), ints(ws)
        if name == "q1s32_f32":
            return "f32", lambda a, y: gq.q1s32_f32_gemm(signs, ws, a, out=y)
        if name == "q1s32_f32_mma":
            return "f32", lambda a, y: gq.q1s32_f32_gemm_mma(signs, ws, a, out=y)
        if name == "q1s32_mma":
            return "split", lambda a, y: gq.q1s32_q8_gemm(signs, ws, *a, path=gq.PATH_MMA, out=y)
        return "split", lambda a, y: gq.q1s32_q8_gemm(signs, ws, a[0], a[1], path=gq.PATH_LUT4, out=y)
    if name == "block_q8":
        _, q, sc = wl.block_q8_inputs(rng, m, k, rows)
        q, sc = ints(q), ints(sc)
        return "f32", lambda a, y: gq.block_q8_matmul_nt(a, q, sc, out=y)
    bits = 8 if "8" in name else 4
    w, sc, _ = wl.wq_inputs(rng, 1, k, rows, bits)
    w, sc = ints(w), ints(sc)
    call = {"matvec_q8": gq.matvec_q8, "matvec_q4": gq.matvec_q4g128, "matmul_q8": gq.matmul_q8, "matmul_q4": gq.matmul_q4g128,
            "matmul_q8_mma": gq.matmul_q8_mma, "matmul_q4_mma": gq.matmul_q4g128_mma}[name]
    return "f32", lambda a, y: call(w, sc, a, out=y)


@pytest.mark.parametrize("name,m,k", [
    ("q1_gemv", 1, 256), ("q1_gemv", 1, 2560), ("q1_gemv", 1, 6912), ("q1_raw", 1, 2560), ("q1_f32", 1, 2560), ("q1_gemm", 3, 256),
    ("q1_gemm", 3, 6912), ("q1_gemm", 17, 2560), ("q1_lut4", 17, 2560), ("q1s32", 17, 1024), ("q1s32_mma", 130, 1024), ("q1s32_f32", 1, 4096),
    ("q1s32_f32", 17, 1024), ("q1s32_f32_mma", 130, 1024), ("block_q8", 1, 960), ("block_q8", 4, 960), ("block_q8", 16, 960),
    ("matvec_q8", 1, 4096), ("matvec_q4", 1, 4096), ("matmul_q8", 5, 1024), ("matmul_q4", 5, 1024), ("matmul_q8_mma", 130, 1024),
    ("matmul_q4_mma", 130, 1024)])
def test_norm_then_product(gq, name, m, k):
    kind, call = products(gq, name, m, k)
    n = 8
    xs = [to_dev(wl.f32_normal(wl.Rng(20 + i), m * k).reshape(m, k)) for i in range(n)]
    w = 1 + 0.1 * to_dev(wl.f32_normal(wl.Rng(9), k))
    out = [torch.zeros(m, 640, device="cuda") for _ in range(n)]
    act = {"q8": torch.zeros(m * (k // 32) * 34, dtype=torch.uint8, device="cuda"), "f32": torch.zeros(m, k, device="cuda"),
           "split": (torch.zeros(m, k // 32, dtype=torch.int16, device="cuda"), torch.zeros(m, k, dtype=torch.int8, device="cuda"),
                     torch.zeros(3, m, k, dtype=torch.int16, device="cuda"))}[kind]

    def step(i):
        if kind == "q8":
            gq.rmsnorm_q8_0(xs[i], w, out=act)
        elif kind == "f32":
            gq.rmsnorm(xs[i], w, out=act)
        else:
            gq.rmsnorm_q8_0(xs[i], w, split=True, mma_operand=True, out=act)
        call(act, out[i])

    for i in range(n):
        step(i)
        torch.cuda.synchronize()
    want = [y.clone() for y in out]
    assert all(torch.isfinite(y).all() and (y != 0).any() for y in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(n):
            step(i)
    for _ in range(5):
        for y in out:
            y.zero_()
        graph.replay()
        for y, z in zip(out, want):
            assert torch.equal(y, z)
