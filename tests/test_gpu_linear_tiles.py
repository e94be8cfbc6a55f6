"""Every tile of the products with an epilogue, more than one of them an SM, their shares of n, and the blocks of four shares of the kernel for few vectors.
The sizes are chosen by gq_q1_q8_linear_plan; test_sizes_reach_every_kernel holds them to it.  Bounds as in the tests of the same calls beside this."""
import pytest
import torch

from tests.gpu_util import need_gpu
from tests.test_gpu_linear import TYPES, U, activations, bent, check, product, weights

SMS = 152
# (pair, vectors, rows, n): several tiles an SM, odd counts of vectors and rows among them; then shares of n; then few vectors of many rows, over several segments
TILES = [(False, 401, 13997, 128), (False, 321, 13999, 128), (False, 577, 12000, 256), (False, 401, 14016, 1024), (False, 577, 12000, 384), (False, 1001, 8997, 2560), (False, 2501, 4998, 1280),
         (True, 129, 13997, 128), (True, 257, 14016, 640), (True, 129, 14016, 2560), (True, 321, 14001, 256), (True, 385, 14016, 384), (True, 481, 13998, 384)]
SHARES = [(False, 33, 100, 640), (False, 65, 6912, 2560), (False, 81, 12000, 2560), (True, 33, 100, 640), (True, 65, 5000, 2560), (True, 65, 3251, 2560), (True, 97, 5000, 2560)]
FEW = [(pair, m, 9000 + m, n) for pair in (False, True) for m, n in ((1, 4224), (8, 4224), (9, 2176))]
BLOCKS = [(False, 401, 14016, 128), (False, 577, 12000, 256), (False, 401, 14016, 1024), (False, 577, 12000, 384), (False, 1000, 9024, 2560), (False, 81, 12000, 2560),
          (True, 129, 14016, 128), (True, 257, 14016, 640), (True, 321, 14016, 256), (True, 385, 14016, 384), (True, 481, 14016, 384), (True, 65, 3264, 2560),
          (False, 8, 9024, 4224), (True, 9, 9024, 2176)]


@pytest.fixture(scope="module")
def gq():
    need_gpu()
    import gemm_q1_q8_gb300 as m
    return m


def plan(pair, m, rows, n, code, q8_0=False):
    """(vectors a tile, shares, tiles an SM at most); (0, 0, 0): the kernel for few vectors."""
    import gemm_q1_q8_gb300 as lib
    p = lib.lib().gq_q1_q8_linear_plan(rows, n, m, code, int(q8_0), int(pair))
    assert p >= 0
    if p == 0:
        return 0, 0, 0
    shares, tile = divmod(p, 256)
    tiles = -(-rows // 128)
    return tile, shares, -(-(tiles if pair else -(-tiles // 2)) * -(-m // tile) * shares // SMS)


def test_sizes_reach_every_kernel():
    from gemm_q1_q8_gb300 import build
    build.build()
    import gemm_q1_q8_gb300 as lib
    for pair in (False, True):
        for cases, q8_0 in ((TILES, False), (BLOCKS, True)):
            reached = {plan(*c, 0, q8_0)[0] for c in cases if c[0] == pair and plan(*c, 0, q8_0)[2] > 1}
            assert reached == {64, 80, 96, 112, 128}, (pair, q8_0, reached)
        one_part = {plan(*c, 2)[0] for c in TILES if c[0] == pair and plan(*c, 2)[2] > 1}
        assert one_part == {64, 80, 96, 112, 128}, (pair, one_part)
        assert {plan(*c, 0)[0] for c in SHARES if c[0] == pair and plan(*c, 0)[1] > 1} == {64, 80, 96}, pair
    assert plan(True, 97, 5000, 2560, 2)[:2] == (112, 2)
    assert all(plan(*c, 0)[0] == 0 for c in FEW)
    # a call takes the same for any outputs, and what it takes fits its workspace
    for pair, m, rows, n in TILES + SHARES + FEW + BLOCKS:
        for code in (0, 1, 2):
            tile, shares, _ = plan(pair, m, rows, n, code)
            need = 0 if tile == 0 else 4 * m * n + 4 * m + (shares * (2 if pair else 1) * m * -(-rows // 128) * 128 * 4 if shares > 1 else 0)
            assert lib.lib().gq_q1_q8_linear_workspace_bytes(rows, n, m, code) >= need
    assert lib.lib().gq_q1_q8_linear_plan(64, 200, 1, 0, 0, 0) == -1 and lib.lib().gq_q1_q8_linear_plan(64, 256, 1, 7, 0, 0) == -1


@pytest.mark.gpu
@pytest.mark.parametrize("pair,m,rows,n", TILES + SHARES + FEW)
def test_values(gq, pair, m, rows, n):
    fn = list(gq.FUNCTIONS)[(m + rows + n // 128) % 6]
    (g, gv), (u, uv) = weights(gq, m, rows, n), weights(gq, m + 1, rows, n) if pair else (None, None)
    act, x = activations(m + 2, m, n)
    gen = torch.Generator(device="cuda").manual_seed(m)
    bias, up = (torch.randn(rows, device="cuda", generator=gen) for _ in range(2))
    for kind, t in TYPES.items():
        need = gq.q1_q8_linear_workspace_bytes(rows, n, m, t)
        room = torch.full((need + 4096,), 0xa5, dtype=torch.uint8, device="cuda")
        if pair:
            f = lambda w: gq.q1_q8_glu(g, u, act, rows, n, m, activation=fn, bias_gate=bias, bias_up=up, dtype=t, workspace=w)  # noqa: E731
            a, ta = bent(fn, *product(x, gv, bias, kind == "bf16"))
            b, tb = product(x, uv, up, kind == "bf16")
            want, tol = a * b, ta * b.abs() + a.abs() * tb + ta * tb
        else:
            r = torch.randn(m, rows, device="cuda", generator=gen).to(t)
            f = lambda w: gq.q1_q8_linear(g, act, rows, n, m, bias=bias, activation=fn, residual=r, dtype=t, workspace=w)  # noqa: E731
            want, tol = bent(fn, *product(x, gv, bias, kind == "bf16"))
            want = want + r.double()
        y = f(room[:need])
        check(y, want, tol, kind)
        assert torch.all(room[need:] == 0xa5)
        # the bits do not depend on what the workspace held, or on its being one for more vectors
        larger = gq.q1_q8_linear_workspace(rows, n, 2 * m + 33, t)
        assert torch.equal(y, f(larger))
    assert gq.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("pair,m,rows,n", BLOCKS)
def test_blocks(gq, pair, m, rows, n):
    """Q8_0 outputs are those of quantize_q8_0 on the f32 call's values, bit for bit."""
    (g, _), (u, _) = weights(gq, 1, rows, n), weights(gq, 2, rows, n) if pair else (None, None)
    act, _ = activations(3, m, n)
    bias = torch.randn(rows, device="cuda", generator=torch.Generator(device="cuda").manual_seed(m))
    if pair:
        f = lambda **k: gq.q1_q8_glu(g, u, act, rows, n, m, activation="relu2", bias_up=bias, **k)  # noqa: E731
    else:
        f = lambda **k: gq.q1_q8_linear(g, act, rows, n, m, activation="relu2", bias=bias, **k)  # noqa: E731
    d, q, _ = gq.quantize_q8_0(f())
    for t in TYPES.values():
        blocks = f(dtype=t, q8_0=True).view(-1, 34)
        assert torch.equal(blocks[:, :2].contiguous().view(torch.int16).flatten(), d.flatten())
        assert torch.equal(blocks[:, 2:].contiguous().view(torch.int8).flatten(), q.flatten())


@pytest.mark.gpu
@pytest.mark.parametrize("pair,m,rows", [(False, 897, 2600), (True, 897, 1300)])
def test_sums_of_several_rounds_in_one_part(gq, pair, m, rows):
    """bf16 results over more than 65536 of n in one share: a round is left out in neither matrix.  Every term is positive, so that one would be missed: the
    result is the sum of its absolute terms."""
    n = 73728
    tile, shares, _ = plan(pair, m, rows, n, 2)
    assert tile and shares == 1
    gen = torch.Generator(device="cuda").manual_seed(1)
    raw = torch.randint(1, 128, (m, n // 32, 34), dtype=torch.uint8, device="cuda", generator=gen)
    d1 = (0.5 + torch.rand(m, n // 32, 1, device="cuda", generator=gen)).half()
    raw[..., :2] = d1.view(torch.uint8)
    x = (raw[..., 2:].double().sum(-1) * d1[..., 0].double()).view(m, n // 128, 4).sum(-1)       # of 128 weights

    def positive():
        w = torch.full((rows, n // 128, 18), 255, dtype=torch.uint8, device="cuda")
        d0 = ((0.5 + torch.rand(rows, n // 128, 1, device="cuda", generator=gen)) * 2.0 ** -21).half()
        w[..., :2] = d0.view(torch.uint8)
        return gq.q1_0_pack(w.view(-1), rows, n), x @ d0[..., 0].double().T

    (g, z), (u, zu) = positive(), positive()
    off = (2 * (n // 16) + n // 32 + 8) * U + 2.0 ** -12
    if pair:
        y = gq.q1_q8_glu(g, u, raw.view(-1), rows, n, m, activation="none", dtype=torch.bfloat16)
        check(y, z * zu, (2 * off + off * off) * z * zu, "bf16")
    else:
        check(gq.q1_q8_linear(g, raw.view(-1), rows, n, m, dtype=torch.bfloat16), z, off * z, "bf16")


@pytest.mark.gpu
def test_refuses_weights_of_other_sizes(gq):
    w, _ = weights(gq, 1, 64, 256)
    act, _ = activations(2, 3, 256)
    for rows, n in ((200, 256), (64, 128)):
        with pytest.raises(gq.GQError):
            gq.q1_q8_linear(w, act, rows, n, 3 if n == 256 else 6)
        with pytest.raises(gq.GQError):
            gq.q1_q8_glu(w, w, act, rows, n, 3 if n == 256 else 6)
    assert gq.device_error() == 0
