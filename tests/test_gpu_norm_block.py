"""The norms around a block (rmsnorm_block) against the formula in 64 bits, and a feed-forward half of a layer with its answer: norm, gated
pair, down product with the residual stream's norms, output product, log probabilities.

Bounds: u = 2^-24; a norm's sum has at most k / (4 threads) + 20 roundings of positive terms, half of which count in the root."""
import math

import numpy as np
import pytest
import torch

import workloads as wl
from tests.gpu_util import need_gpu
from tests.test_gpu_linear import activations, hard_blocks, product, weights

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ROUND = {"f32": U, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}


@pytest.fixture(scope="module")
def gq():
    need_gpu()
    import gemm_q1_q8_gb300 as m
    return m


def normal(seed, *shape):
    return torch.from_numpy(wl.f32_normal(wl.Rng(seed), int(np.prod(shape))).reshape(shape)).cuda()


def exact(y, x, w, post, gate, beta, alpha, eps):
    """(h, z, the sizes that their roundings go with)."""
    n = y.double()
    if post is not None:
        n = n / torch.sqrt(n.square().mean(-1, keepdim=True) + eps) * post.double()
    if gate is not None:
        n = gate.double() * n
    h = alpha * x.double() + beta * n
    size = abs(alpha) * x.double().abs() + abs(beta) * n.abs()
    r = 1 / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)
    return h, h * r * w.double(), size, size * r * w.double().abs()


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("m,k,kind,gated", [
    (1, 1, "f32", "row"), (1, 2560, "f32", "none"), (3, 33, "f32", "token"), (5, 31, "bf16", "row"), (2, 4098, "f16", "token"),
    (200, 4096, "f32", "none"), (160, 6912, "bf16", "token"), (153, 960, "f16", "row"), (2, 65536, "f32", "token"),
    (1, 40001, "f16", "token"), (333, 96, "f32", "row"), (1000, 16384, "bf16", "none"), (160, 5120, "f32", "row"), (154, 8192, "bf16", "token")])
def test_values(gq, m, k, kind, gated, post):
    t = TYPES[kind]
    y, x = normal(1, m, k).to(t), (3 * normal(2, m, k)).to(t)
    gate = {"none": None, "row": normal(3, k).to(t), "token": normal(4, m, k).to(t)}[gated]
    w, pw = 1 + 0.3 * normal(5, k), 0.5 + 0.3 * normal(6, k) if post else None
    h_out = torch.empty_like(x)
    z = gq.rmsnorm_block(y, x, w, post_weight=pw, eps=1e-5, gate=gate, block_scale=0.75, residual_scale=-1.5, sum_out=h_out)
    h, want, hs, zs = exact(y, x, w, pw, gate, 0.75, -1.5, 1e-5)
    steps = (min(k, 4 * 16) + 22) / 2 + 8
    th = (steps + 6) * U * hs
    assert torch.all((h_out.double() - h).abs() <= th + ROUND[kind] * (h.abs() + th) + TINY[kind])
    # h's error, as it stands in the result and in the root, and the second norm's own
    tz = (2 * (steps + 6) + steps) * U * zs
    # in the root h's error counts as the mean of |h| its error / h^2, at most the ratio of the sizes' squares
    tz = tz + (steps + 6) * U * want.abs() * (hs.square().mean(-1, keepdim=True) / (h.square().mean(-1, keepdim=True) + 1e-5)).sqrt()
    assert torch.all((z.double() - want).abs() <= tz + ROUND[kind] * (want.abs() + tz) + TINY[kind])


@pytest.mark.parametrize("m,k,kind", [(1, 2560, "f32"), (7, 32, "f32"), (300, 4096, "bf16"), (2, 40960, "f16"), (170, 6912, "f32"), (156, 5120, "f16"), (155, 8192, "bf16")])
def test_q8_0_is_the_quantizer_on_the_norm(gq, m, k, kind):
    t = TYPES[kind]
    y, x, g = normal(1, m, k).to(t), normal(2, m, k).to(t), normal(3, m, k).to(t)
    w, pw = 1 + 0.3 * normal(5, k), 0.5 + 0.3 * normal(6, k)
    y[0, :32] = 0
    x[0, :32] = 0                                        # a block of zeros: d = 0
    z = gq.rmsnorm_block(y.float(), x.float(), w, post_weight=pw, gate=g.float(), block_scale=0.5)
    d, q, op = gq.quantize_q8_0(z, mma_operand=True)
    act = gq.rmsnorm_block_q8_0(y, x, w, post_weight=pw, gate=g, block_scale=0.5)
    d2, q2, op2 = gq.rmsnorm_block_q8_0(y, x, w, post_weight=pw, gate=g, block_scale=0.5, split=True, mma_operand=True)
    assert torch.equal(d, d2) and torch.equal(q, q2) and torch.equal(op, op2)
    blocks = act.view(-1, 34)
    assert torch.equal(blocks[:, :2].contiguous().view(torch.int16).flatten(), d.flatten())
    assert torch.equal(blocks[:, 2:].contiguous().view(torch.int8).flatten(), q.flatten())


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("m,k", [(2, 4096), (200, 4096), (153, 960), (160, 5120), (154, 8192), (153, 6912), (153, 16384), (2, 65536)])
def test_blocks_of_hard_values(gq, m, k, kind):
    """A stream of ones leaves the weight: ties, zeros and scales out of f16's and f32's normal range, as quantize_q8_0 has them."""
    w = hard_blocks(k, m)
    one, zero = torch.ones(m, k, device="cuda", dtype=TYPES[kind]), torch.zeros(m, k, device="cuda", dtype=TYPES[kind])
    d, q, op = gq.quantize_q8_0(w[None].contiguous(), mma_operand=True)
    d, q = d.view(1, -1).expand(m, -1), q.view(1, -1).expand(m, -1)
    blocks = gq.rmsnorm_block_q8_0(zero, one, w, eps=0.0).view(m, k // 32, 34)
    assert torch.equal(blocks[..., :2].contiguous().view(torch.int16)[..., 0], d)
    assert torch.equal(blocks[..., 2:].contiguous().view(torch.int8).reshape(m, k), q)
    for operand in (False, True):
        d2, q2, op2 = gq.rmsnorm_block_q8_0(zero, one, w, eps=0.0, split=True, mma_operand=operand)
        assert torch.equal(d2, d) and torch.equal(q2, q)
        assert not operand or torch.equal(op2.view(3, m, k), op.view(3, 1, k).expand(3, m, k))


@pytest.mark.parametrize("m,k", [(3, 1024), (400, 1024), (2, 65536)])
def test_in_place_strided_and_plain(gq, m, k):
    base = normal(7, m, 3 * k)
    y, x, g = base[:, :k], base[:, k:2 * k], base[:, 2 * k:]
    w, pw = 1 + 0.1 * normal(9, k), 1 + 0.1 * normal(10, k)
    h = torch.empty(m, k, device="cuda")
    want = gq.rmsnorm_block(y.contiguous(), x.contiguous(), w, post_weight=pw, gate=g.contiguous(), sum_out=h)
    assert torch.equal(gq.rmsnorm_block(y, x, w, post_weight=pw, gate=g), want)
    for own in (0, 1):                                    # h over the stream, or over the block's output
        a, b = y.contiguous().clone(), x.contiguous().clone()
        z = gq.rmsnorm_block(a, b, w, post_weight=pw, gate=g, sum_out=(a, b)[own])
        assert torch.equal(z, want) and torch.equal((a, b)[own], h)
    odd = torch.empty(m * k + 1, device="cuda")[1:].view(m, k)    # rows that are not 16-byte aligned
    odd.copy_(y)
    assert torch.allclose(gq.rmsnorm_block(odd, x, w, post_weight=pw, gate=g), want, rtol=1e-5, atol=1e-6)
    # without gate, first norm and scales it is the norm with a residual
    assert torch.equal(gq.rmsnorm_block(y, x, w), gq.rmsnorm(x, w, residual=y))


def test_refusals(gq):
    x = normal(1, 4, 64)
    w = torch.ones(64, device="cuda")
    for bad in (dict(gate=normal(2, 3, 64)), dict(gate=normal(2, 4, 64).half()), dict(gate=normal(2, 2, 4, 64)), dict(post_weight=torch.ones(63, device="cuda")),
                dict(block_scale=math.inf), dict(eps=-1.0), dict(out=torch.empty(4, 63, device="cuda")), dict(sum_out=torch.empty(4, 64, device="cuda").half())):
        with pytest.raises(gq.GQError):
            gq.rmsnorm_block(x, x, w, **bad)
    with pytest.raises(gq.GQError):
        gq.rmsnorm_block(x.half(), x, w)


def q8_values(gq, act, m, k):
    return gq.dequantize_q8_0(act, m, k).double()


@pytest.mark.parametrize("m", [1, 5, 140])
def test_a_feed_forward_half_and_its_answer(gq, m):
    """The operators as a decoder runs them, in a graph: each result against the formula on what the operator before it gave."""
    hidden, ffn, vocab = 640, 1792, 3000
    (g, gv), (u, uv), (dn, dv), (head, hv) = (weights(gq, s, r, n) for s, r, n in ((1, ffn, hidden), (2, ffn, hidden), (3, hidden, ffn), (4, vocab, hidden)))
    w1, w2, w3 = (1 + 0.2 * normal(s, hidden) for s in (5, 6, 7))
    x = torch.empty(m, hidden, device="cuda")
    tokens = torch.arange(m, device="cuda") * 7 % vocab
    kept = {}

    def half():
        act = gq.rmsnorm_q8_0(x, w1)
        mid = gq.q1_q8_glu(g, u, act, ffn, hidden, m, activation="relu2", q8_0=True)
        y = gq.q1_q8_linear(dn, mid, hidden, ffn, m)
        h = torch.empty_like(x)
        act2 = gq.rmsnorm_block_q8_0(y, x, w3, post_weight=w2, residual_scale=1.25, sum_out=h)
        logits = gq.q1_q8_linear(head, act2, vocab, hidden, m)
        kept.update(act=act, mid=mid, y=y, h=h, act2=act2, logits=logits, answer=gq.logprobs(logits, tokens=tokens, top=4))

    x.copy_(normal(8, m, hidden))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        half()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        half()
    x.copy_(normal(9, m, hidden))
    graph.replay()
    torch.cuda.synchronize()
    a = q8_values(gq, kept["act"], m, hidden)
    want = (a @ gv.T).clamp_min(0) ** 2 * (a @ uv.T)
    got = q8_values(gq, kept["mid"], m, ffn)
    # a code is off by at most half a step and the scale by 2^-11 of itself, each step 1 / 127 of the block's largest; a thousandth for the products
    top = want.view(m, -1, 32).abs().amax(-1, keepdim=True)
    assert torch.all((got - want).view(m, -1, 32).abs() <= top * (0.5 / 127 + 2.0 ** -11 + 1e-3))
    z, tol = product(got, dv, None, False)
    assert torch.all((kept["y"].double() - z).abs() <= tol)
    h, want, hs, _ = exact(kept["y"], x, w3, w2, None, 1.0, 1.25, 1e-5)
    assert torch.all((kept["h"].double() - h).abs() <= 64 * U * hs)
    got = q8_values(gq, kept["act2"], m, hidden)
    top = want.view(m, -1, 32).abs().amax(-1, keepdim=True)
    assert torch.all((got - want).view(m, -1, 32).abs() <= top * (0.5 / 127 + 2.0 ** -11 + 1e-4))
    z, tol = product(got, hv, None, False)
    assert torch.all((kept["logits"].double() - z).abs() <= tol)
    lp = torch.log_softmax(kept["logits"].double(), -1)
    r = kept["answer"]
    assert torch.all((r.logprob - lp.gather(1, tokens[:, None]).squeeze(1)).abs() <= 1e-4)
    assert torch.equal(r.top_ids, torch.sort(kept["logits"].cpu(), dim=-1, descending=True, stable=True).indices[:, :4].cuda())
    assert gq.device_error() == 0
