"""Q1_0 products with an epilogue (q1_q8_linear, q1_q8_glu) against the formula in 64 bits.

Bounds (u = 2^-24, A = sum |d0 d1 q| of a result): products are exact and a part of an activation is lost only below 2^-39 of its vector's
largest.  A tensor-core step is taken to be off by two units (its truncated sum); a chain has at most 16 steps before it is added
in f32 (n / 16 where the result is bf16), and there are at most n / 32 + 8 such additions.  A bf16 result takes activations rounded to 2^-12."""
import math

import numpy as np
import pytest
import torch

from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ROUND = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}      # half the distance of f16's subnormals


@pytest.fixture(scope="module")
def gq():
    need_gpu()
    import gemm_q1_q8_gb300 as m
    return m


def weights(gq, seed, rows, n):
    """(packed, f64 values [rows, n]) of random Q1_0 blocks."""
    rng = np.random.default_rng(seed)
    raw = rng.integers(0, 256, (rows, n // 128, 18), dtype=np.uint8)
    d = (n ** -0.5 * rng.uniform(0.2, 2.0, (rows, n // 128, 1))).astype(np.float16)
    d[rng.random(d.shape) < 0.02] = 0
    d *= np.where(rng.random(d.shape) < 0.1, -1, 1).astype(np.float16)
    raw[..., :2] = d.view(np.uint8)
    bits = np.unpackbits(raw[..., 2:], axis=-1, bitorder="little").astype(np.float64)
    w = ((2 * bits - 1) * d.astype(np.float64)).reshape(rows, n)
    return gq.q1_0_pack(torch.from_numpy(raw.reshape(-1)).cuda(), rows, n), torch.from_numpy(w).cuda()


def activations(seed, m, n, wide=False):
    """(blocks as uint8, f64 values [m, n]); wide: scales over f16's whole range, within a vector too."""
    rng = np.random.default_rng(seed)
    raw = rng.integers(0, 256, (m, n // 32, 34), dtype=np.uint8)
    d = 2.0 ** rng.uniform(-24, 15.9, (m, n // 32, 1)) if wide else rng.uniform(0.001, 0.02, (m, n // 32, 1)) * rng.uniform(0.1, 3, (m, 1, 1))
    d = d.astype(np.float16)
    d[rng.random(d.shape) < 0.02] = 0
    raw[..., :2] = d.view(np.uint8)
    x = raw[..., 2:].view(np.int8).astype(np.float64) * d.astype(np.float64)
    return torch.from_numpy(raw.reshape(-1)).cuda(), torch.from_numpy(x.reshape(m, n)).cuda()


def product(x, w, bias, one_part):
    """(z, the bound of its error)."""
    z, a = x @ w.T, x.abs() @ w.abs().T
    n = x.shape[1]
    chain = n // 16 if one_part else 16
    tol = (2 * chain + n // 32 + 8) * U * a + 2.0 ** -39 * x.abs().amax(-1, keepdim=True) * w.abs().sum(-1)
    if one_part:
        tol = tol + 2.0 ** -12 * a
    if bias is not None:
        z = z + bias.double()
    return z, tol + 2 * U * z.abs()


def bent(name, z, tol):
    """(function, the bound of its error): the slope times the argument's, and some units of the function itself (the exponential's
    argument is off by 2^-22 of itself, so the exponential by |z| times that; it and the division by 4 units each)."""
    if name == "none":
        return z, tol
    if name == "relu":
        return z.clamp_min(0), tol
    if name == "relu2":
        y = z.clamp_min(0) ** 2
        return y, (2 * z.clamp_min(0) + tol) * tol + U * y
    if name == "silu":
        y = z * torch.sigmoid(z)
        return y, 1.1 * tol + (12 + 4 * z.abs()) * U * y.abs()
    if name == "gelu":
        y = z * torch.special.ndtr(z)
        return y, 1.13 * tol + (16 + 4 * z * z) * U * y.abs()
    v = z + 0.044715 * z ** 3
    y = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * v)
    return y, 1.13 * tol + (12 + 16 * v.abs()) * U * y.abs()


def check(got, want, tol, kind):
    # below 2^-120 the exponentials may give nothing
    tol = tol + (ROUND[kind] + U) * (want.abs() + tol) + TINY[kind] + 2.0 ** -120
    err = (got.double() - want).abs()
    assert torch.all(err <= tol), (float((err / tol).max()), int((err > tol).sum()))


SHAPES = [(1, 1, 128), (1, 33, 256), (2, 127, 1152), (3, 64, 4224), (4, 300, 2560), (5, 129, 640), (8, 32, 128), (9, 160, 384), (16, 257, 1024),
          (17, 96, 6912), (31, 513, 256), (33, 130, 896), (64, 64, 2176), (65, 256, 512), (97, 200, 1280), (130, 384, 2560), (257, 129, 128),
          (300, 640, 1152), (513, 40, 256)]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,rows,n", SHAPES)
def test_linear_values(gq, m, rows, n, kind):
    """Every function in turn, with and without bias and residual."""
    fn = list(gq.FUNCTIONS)[(m + rows + n // 128) % 6]
    w, wv = weights(gq, m, rows, n)
    act, x = activations(m + 1, m, n)
    gen = torch.Generator(device="cuda").manual_seed(m)
    bias = torch.randn(rows, device="cuda", generator=gen) if m % 3 else None
    r = torch.randn(m, rows, device="cuda", generator=gen).to(TYPES[kind]) if m % 2 else None
    y = gq.q1_q8_linear(w, act, rows, n, m, bias=bias, activation=fn, residual=r, dtype=TYPES[kind])
    want, tol = bent(fn, *product(x, wv, bias, kind == "bf16"))
    if r is not None:
        want = want + r.double()
    check(y, want, tol, kind)
    assert torch.equal(y, gq.q1_q8_linear(w, act, rows, n, m, bias=bias, activation=fn, residual=r, dtype=TYPES[kind]))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,rows,n", SHAPES)
def test_glu_values(gq, m, rows, n, kind):
    fn = list(gq.FUNCTIONS)[(m + 2 * rows + n // 128) % 6]
    (g, gv), (u, uv) = weights(gq, m, rows, n), weights(gq, m + 100, rows, n)
    act, x = activations(m + 1, m, n)
    gen = torch.Generator(device="cuda").manual_seed(m)
    bg, bu = (torch.randn(rows, device="cuda", generator=gen) for _ in range(2)) if m % 3 else (None, None)
    y = gq.q1_q8_glu(g, u, act, rows, n, m, activation=fn, bias_gate=bg, bias_up=bu, dtype=TYPES[kind])
    a, ta = bent(fn, *product(x, gv, bg, kind == "bf16"))
    b, tb = product(x, uv, bu, kind == "bf16")
    check(y, a * b, ta * b.abs() + a.abs() * tb + ta * tb, kind)


def hard_blocks(count, seed=0):
    """`count` values, a multiple of 32, in blocks of ties, of zeros and of sizes over f32's range, in an order that mixes them."""
    rng = np.random.default_rng(seed)
    ties = np.concatenate([[127.0], np.arange(31) - 14.5])                # with a scale of one
    kinds = [ties * 2.0 ** e for e in (0, -100, -119, -121, -126, -133, 118)] + [np.zeros(32), np.where(np.arange(32) % 3, 0.0, -0.0), 2.0 ** -149 * np.arange(32.0)]
    kinds += [rng.standard_normal(32) * 10.0 ** e for e in (-30, -5, 0, 5, 30)] + [np.where(np.arange(32) == 7, 3e38, 1.0)]
    return torch.from_numpy(np.concatenate([kinds[i] for i in rng.integers(0, len(kinds), count // 32)]).astype(np.float32)).cuda()


@pytest.mark.parametrize("m", [1, 20, 40, 70, 90, 105, 130, 517])
def test_blocks_of_hard_values(gq, m):
    """Activations of zeros leave the bias: ties, zeros and scales out of f16's and f32's normal range, as quantize_q8_0 has them."""
    rows, n = 6912, 256
    w, _ = weights(gq, 1, rows, n)
    act = torch.zeros(m * n // 32 * 34, dtype=torch.uint8, device="cuda")
    bias = hard_blocks(rows, m)
    d, q, _ = gq.quantize_q8_0(bias[None].contiguous())
    blocks = gq.q1_q8_linear(w, act, rows, n, m, bias=bias, q8_0=True).view(m, rows // 32, 34)
    assert torch.equal(blocks[..., :2].contiguous().view(torch.int16)[..., 0], d.view(1, -1).expand(m, -1))
    assert torch.equal(blocks[..., 2:].contiguous().view(torch.int8).reshape(m, -1), q.view(1, -1).expand(m, -1))


@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("m,rows,n", [(1, 32, 128), (3, 160, 2560), (20, 96, 256), (70, 416, 640), (300, 128, 1152)])
def test_blocks_are_the_quantizer_on_the_values(gq, m, rows, n, pair):
    """Q8_0 outputs of every type are those of quantize_q8_0 on the f32 call's values, bit for bit."""
    (g, _), (u, _) = weights(gq, 1, rows, n), weights(gq, 2, rows, n)
    act, _ = activations(3, m, n)
    bias = torch.randn(rows, device="cuda")
    if pair:
        f = lambda **k: gq.q1_q8_glu(g, u, act, rows, n, m, activation="relu2", bias_gate=bias, **k)  # noqa: E731
    else:
        f = lambda **k: gq.q1_q8_linear(g, act, rows, n, m, activation="relu2", bias=bias, **k)  # noqa: E731
    y = f()
    d, q, _ = gq.quantize_q8_0(y)
    for t in TYPES.values():
        blocks = f(dtype=t, q8_0=True).view(-1, 34)
        assert torch.equal(blocks[:, :2].contiguous().view(torch.int16).flatten(), d.flatten())
        assert torch.equal(blocks[:, 2:].contiguous().view(torch.int8).flatten(), q.flatten())


@pytest.mark.parametrize("m", [2, 40, 200])
def test_scales_of_any_size(gq, m):
    """Scales from f16's least to its largest, beside each other: values down to 2^-20 of the largest are whole."""
    rows, n = 130, 640
    w, wv = weights(gq, 5, rows, n)
    act, x = activations(6, m, n, wide=True)
    check(gq.q1_q8_linear(w, act, rows, n, m), *product(x, wv, None, False), "f32")


@pytest.mark.parametrize("m", [3, 150])
def test_weights_of_small_scales(gq, m):
    """Scales that are f16 subnormals count in full."""
    rows, n = 130, 640
    rng = np.random.default_rng(1)
    raw = rng.integers(0, 256, (rows, n // 128, 18), dtype=np.uint8)
    d = rng.integers(1, 40, (rows, n // 128, 1)).astype(np.uint16)          # multiples of 2^-24
    raw[..., :2] = d.view(np.uint8)
    bits = np.unpackbits(raw[..., 2:], axis=-1, bitorder="little").astype(np.float64)
    wv = torch.from_numpy(((2 * bits - 1) * d * 2.0 ** -24).reshape(rows, n)).cuda()
    w = gq.q1_0_pack(torch.from_numpy(raw.reshape(-1)).cuda(), rows, n)
    act, x = activations(2, m, n)
    check(gq.q1_q8_linear(w, act, rows, n, m), *product(x, wv, None, False), "f32")


@pytest.mark.parametrize("m", [3, 150])
def test_a_vector_that_is_not_finite(gq, m):
    rows, n = 64, 512
    w, _ = weights(gq, 7, rows, n)
    act, _ = activations(8, m, n)
    want = gq.q1_q8_linear(w, act, rows, n, m)
    for bits in (0x7c00, 0xfe00):
        bad = act.clone().view(m, -1)
        bad[1, 34:36] = torch.tensor([bits & 255, bits >> 8], dtype=torch.uint8, device="cuda")
        bad[1, 36:68] = 5
        y = gq.q1_q8_linear(w, bad.view(-1), rows, n, m)
        assert not torch.isfinite(y[1]).any()
        keep = [i for i in range(m) if i != 1]
        assert torch.equal(y[keep], want[keep])


@pytest.mark.parametrize("m,kind", [(1, "f32"), (7, "f16"), (90, "bf16"), (200, "f32")])
def test_strides_and_in_place(gq, m, kind):
    """Outputs and residuals with a stride, the residual updated in place, and nothing written beside the rows."""
    rows, n = 100, 384
    w, _ = weights(gq, 9, rows, n)
    act, _ = activations(10, m, n)
    t = TYPES[kind]
    r = torch.randn(m, rows, device="cuda").to(t)
    want = gq.q1_q8_linear(w, act, rows, n, m, residual=r, dtype=t)
    base = torch.full((m + 1, 3 * rows + 1), 7.0, dtype=t, device="cuda")
    view = base[:m, rows + 1:2 * rows + 1]
    view.copy_(r)
    out = gq.q1_q8_linear(w, act, rows, n, m, residual=view, dtype=t, out=view)
    assert torch.equal(out, want)
    assert torch.all(base[:, :rows + 1] == 7) and torch.all(base[:, 2 * rows + 1:] == 7) and torch.all(base[m] == 7)
    room = torch.full((m * 128 * 34 // 32 + 64,), 9, dtype=torch.uint8, device="cuda")
    wb, _ = weights(gq, 11, 128, n)
    got = gq.q1_q8_linear(wb, act, 128, n, m, q8_0=True, out=room[:-64])
    assert torch.equal(got, gq.q1_q8_linear(wb, act, 128, n, m, q8_0=True)) and torch.all(room[-64:] == 9)


@pytest.mark.parametrize("m,rows,n", [(1, 64, 512), (7, 300, 1280), (20, 96, 256), (50, 640, 2560)])
def test_activations_of_any_alignment(gq, m, rows, n):
    w, _ = weights(gq, 3, rows, n)
    act, _ = activations(4, m, n)
    want = gq.q1_q8_linear(w, act, rows, n, m)
    for shift in (2, 4, 6):
        room = torch.empty(act.numel() + 8, dtype=torch.uint8, device="cuda")
        moved = room[shift:shift + act.numel()]
        moved.copy_(act)
        assert torch.equal(gq.q1_q8_linear(w, moved, rows, n, m), want)


def test_both_outputs_through_the_c_abi(gq):
    m, rows, n = 5, 64, 256
    w, _ = weights(gq, 12, rows, n)
    act, _ = activations(13, m, n)
    y, blocks = torch.empty(m, rows, device="cuda"), torch.empty(m * 2 * 34, dtype=torch.uint8, device="cuda")
    work = gq.q1_q8_linear_workspace(rows, n, m)
    p = lambda t: t.data_ptr()  # noqa: E731
    assert gq.lib().q1_q8_linear(p(w), p(act), rows, n, m, None, 3, None, 0, 0, p(y), rows, p(blocks), p(work),
                                 torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(y, gq.q1_q8_linear(w, act, rows, n, m, activation="silu"))
    assert torch.equal(blocks, gq.q1_q8_linear(w, act, rows, n, m, activation="silu", q8_0=True))


@pytest.mark.parametrize("m", [1, 6, 60, 260])
def test_two_streams_and_a_graph(gq, m):
    """Two calls at once with workspaces of their own, and captured calls replayed on new inputs."""
    rows, n = 384, 1280
    (g, _), (u, _) = weights(gq, 14, rows, n), weights(gq, 15, rows, n)
    acts = [activations(s, m, n)[0] for s in (16, 17)]
    want = [gq.q1_q8_glu(g, u, a, rows, n, m) for a in acts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in acts]
    outs = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(gq.q1_q8_glu(g, u, acts[i], rows, n, m))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in (0, 1) for o in outs[i])
    x, work, y = acts[0].clone(), gq.q1_q8_linear_workspace(rows, n, m), torch.empty(m, rows, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gq.q1_q8_glu(g, u, x, rows, n, m, out=y, workspace=work)
    for a, b in zip(acts[::-1], want[::-1]):
        x.copy_(a)
        graph.replay()
        assert torch.equal(y, b)


def test_chain_of_dependents(gq):
    """Each product's blocks are the next one's activations, launched without a wait between them."""
    rows, n, m = 256, 256, 2
    ws = [weights(gq, 20 + i, rows, n)[0] for i in range(6)]
    act, _ = activations(30, m, n)
    a, b = act, act
    for w in ws:
        a = gq.q1_q8_linear(w, a, rows, n, m, activation="gelu", q8_0=True)
    for w in ws:
        b = gq.q1_q8_linear(w, b, rows, n, m, activation="gelu", q8_0=True)
        torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_refusals(gq):
    w, _ = weights(gq, 1, 64, 256)
    act, _ = activations(2, 3, 256)
    for bad in (dict(out=torch.empty(3, 64, device="cuda", dtype=torch.float16)), dict(out=torch.empty(2, 64, device="cuda")),
                dict(residual=torch.empty(3, 65, device="cuda")), dict(residual=torch.empty(64, 3, device="cuda").t()),
                dict(bias=torch.empty(63, device="cuda")), dict(workspace=torch.empty(0, dtype=torch.uint8, device="cuda")), dict(dtype=torch.float64),
                dict(activation="tanh")):
        with pytest.raises(gq.GQError):
            gq.q1_q8_linear(w, act, 64, 256, 3, **bad)
    with pytest.raises(gq.GQError):
        gq.q1_q8_linear(w, act, 64, 256, 4)
    with pytest.raises(gq.GQError):
        gq.q1_q8_linear(w, act, 32, 256, 3)[:0] if gq.q1_0_packed_bytes(32, 256) != w.numel() else gq.q1_q8_linear(w, act, 200, 256, 3)
    assert gq.device_error() == 0
