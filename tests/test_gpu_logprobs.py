"""Log probabilities, entropy and the best alternatives (logprobs) against the formula in 64 bits.

Bounds (u = 2^-24): a term 2^t of the sum is off by 4 units (the exponential) and by the rounding of its argument, 3 units of |t| ln 2; of the
terms that count |t| averages at most ln(vocab) + 10.  A sum is a chain of at most 130 terms, 9 + 4 joins and 64 parts' joins."""
import math

import pytest
import torch

from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def gq():
    need_gpu()
    import gemm_q1_q8_gb300 as m
    return m


def exact(x, tokens, top, scale):
    lp = torch.log_softmax(scale * x.double(), -1)
    h = -torch.where(lp == -math.inf, 0.0, lp.exp() * lp).sum(-1)
    order = torch.sort(x.float(), dim=-1, descending=True, stable=True).indices[:, :top]
    return lp.gather(1, tokens[:, None]).squeeze(1), h, order, lp.gather(1, order)


def check(gq, x, top, scale=1.0, seed=0):
    m, vocab = x.shape
    gen = torch.Generator(device="cuda").manual_seed(seed)
    tokens = torch.randint(0, vocab, (m,), device="cuda", generator=gen)
    r = gq.logprobs(x, tokens=tokens, top=top, scale=scale)
    lp, h, order, best = exact(x, tokens, top, scale)
    s = (4 + 3 * (math.log(vocab) + 10) + 210) * U                   # of the sum, so of its logarithm
    tol = s + 4 * U * (lp.abs() + math.log(vocab) + 1)
    same = (r.logprob == lp) | ((r.logprob.double() - lp).abs() <= tol)
    assert same.all(), (r.logprob, lp)
    # the mean of t is off by the sum's error twice and by its terms'
    assert torch.all((r.entropy.double() - h).abs() <= 3 * s * (h + math.log(vocab) + 2))
    if top:
        assert torch.equal(r.top_ids, order)
        assert ((r.top_logprobs == best) | ((r.top_logprobs.double() - best).abs() <= s + 4 * U * (best.abs() + math.log(vocab) + 1))).all()
    else:
        assert r.top_ids is None and r.top_logprobs is None
    again = gq.logprobs(x, tokens=tokens, top=top, scale=scale)
    assert all(a is b or torch.equal(a, b) for a, b in zip(r, again))


def normal(seed, m, vocab, size=3.0):
    return size * torch.randn(m, vocab, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,vocab,top", [
    (1, 1, 1), (1, 2, 2), (3, 7, 5), (2, 33, 32), (5, 511, 0), (4, 513, 1), (2, 4095, 32), (1, 49152, 20), (3, 49153, 5), (40, 5000, 10),
    (305, 1000, 7), (310, 8191, 32), (7, 128256, 20), (2, 200001, 32), (1, 1 << 20, 32), (306, 70000, 3), (1216, 4099, 5), (1300, 999, 32), (2000, 12000, 1)])
def test_values(gq, m, vocab, top, kind):
    check(gq, normal(m + vocab, m, vocab).to(TYPES[kind]), top)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("stride,first", [(1003, 1), (1001, 3), (1024, 8), (1007, 5)])
def test_rows_of_any_alignment(gq, stride, first, kind):
    base = normal(1, 9, stride + 16).to(TYPES[kind])
    base[:, :first] = 1e4                                  # neighbours that would be seen
    base[:, first + 990:] = 1e4
    check(gq, base[:, first:first + 990], 8)


@pytest.mark.parametrize("scale", [0.01, 0.7, 5.0, 1e4])
def test_temperatures(gq, scale):
    check(gq, normal(2, 5, 3001), 4, scale=scale)
    check(gq, normal(2, 400, 3001, 0.5), 4, scale=scale)


@pytest.mark.parametrize("m,vocab", [(2, 9001), (460, 9001), (1, 300001)])
@pytest.mark.parametrize("first,size", [(7e5, 3.0), (-7e5, 3.0), (7.3e5, 30.0), (-7.26842e5, 5.0), (1e9, 1e3), (-1e9, 1e3), (0.0, 1e30), (0.0, 1e37), (3.3e38, 1e32),
                                        (-3.39e38, 1e31)])
def test_logits_far_from_zero(gq, m, vocab, first, size):
    """Whatever their size, up to the type's; 7.268e5 is where the form of the sums changes, in parts of a row before others."""
    x = (first + normal(4, m, vocab, size).double()).clamp(-3.4e38, 3.4e38).float()
    x[:, :vocab // 2] -= 6 * size if abs(first) > 1e5 and size < 1e3 else 0
    check(gq, x, 6)


@pytest.mark.parametrize("m,vocab,threads", [(400, 65536, 512), (1300, 20000, 128), (2, 500000, 512)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_more_candidates_than_fit(gq, m, vocab, threads, kind):
    """Thousands of a row's logits with fewer threads than alternatives are asked for, above the others' maxima."""
    x = normal(11, m, vocab, 0.25).abs().to(TYPES[kind])
    width = 4 if kind == "f32" else 8
    x[:, torch.arange(vocab, device="cuda") // width % threads >= 24] = 0
    check(gq, x, 32)


@pytest.mark.parametrize("m", [2, 400, 1300])
@pytest.mark.parametrize("top", [1, 5, 32])
def test_ties_go_by_index(gq, m, top):
    """Equal logits everywhere, two values, a few values, both zeros, and sorted rows (the best ones all with one thread's neighbours)."""
    vocab = 20000
    gen = torch.Generator(device="cuda").manual_seed(3)
    check(gq, torch.full((m, vocab), 1.5, device="cuda"), top)
    check(gq, torch.randint(0, 2, (m, vocab), device="cuda", generator=gen).float(), top)
    check(gq, torch.randint(0, 40, (m, vocab), device="cuda", generator=gen).to(torch.bfloat16), top)
    zeros = torch.zeros(m, vocab, device="cuda")
    zeros[:, ::3] = -0.0
    check(gq, zeros, top)
    rising = torch.arange(vocab, device="cuda").float().repeat(m, 1) * 1e-3
    check(gq, rising, top)
    check(gq, -rising, top)
    clustered = torch.zeros(m, vocab, device="cuda")       # one thread's logits are the best ones
    clustered[:, 64:vocab:2048] = 1 + torch.arange(len(range(64, vocab, 2048)), device="cuda") * 1e-4
    check(gq, clustered, top)
    near = 5 + torch.randint(0, 30000, (m, vocab), device="cuda", generator=gen).float() * 2.0 ** -21     # one bucket of the first search
    check(gq, near, top)


@pytest.mark.parametrize("m,vocab", [(1, 49152), (3, 999), (330, 5001), (1300, 3001), (2, 300001)])
@pytest.mark.parametrize("left", [0, 1, 3, 40])
def test_masked_rows(gq, m, vocab, left):
    """-inf, or the type's lowest value, but for `left` logits of a row."""
    for kind, t in TYPES.items():
        x = normal(4, m, vocab).to(t)
        keep = torch.rand(m, vocab, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).argsort(-1)[:, :left]
        for hidden in (-math.inf, torch.finfo(t).min):
            y = torch.full_like(x, hidden).scatter(1, keep, x.gather(1, keep))
            if left or hidden > -math.inf:
                check(gq, y, 5)
                continue
            tokens = torch.zeros(m, dtype=torch.int64, device="cuda")
            r = gq.logprobs(y, tokens=tokens, top=5)
            assert torch.all(r.logprob == -math.inf) and torch.all(r.entropy == 0) and torch.all(r.top_logprobs == -math.inf)
            assert torch.equal(r.top_ids, torch.arange(5, device="cuda").repeat(m, 1))


@pytest.mark.parametrize("m", [3, 400, 1300])
def test_rows_with_nan_or_infinity(gq, m):
    """They give NaN, their alternatives in order (NaN first), and the other rows what they would."""
    x = normal(6, m, 6000)
    tokens = torch.arange(m, device="cuda") % 6000
    want = gq.logprobs(x, tokens=tokens, top=3)
    for bad in (math.nan, math.inf):
        y = x.clone()
        y[1, 4321] = bad
        y[1, 77] = bad
        r = gq.logprobs(y, tokens=tokens, top=3)
        assert torch.isnan(r.logprob[1]) and torch.isnan(r.entropy[1]) and torch.isnan(r.top_logprobs[1]).all()
        assert r.top_ids[1].tolist() == [77, 4321, int(want.top_ids[1, 0])]
        keep = [i for i in range(m) if i != 1]
        assert all(torch.equal(a[keep], b[keep]) for a, b in zip(r, want))


def test_given_tokens(gq):
    """Negative ones count for nothing; one past the vocabulary gives NaN and an error."""
    assert gq.device_error() == 0
    for m in (4, 500, 1300):
        x = normal(7, m, 2000)
        tokens = torch.full((m,), 5, dtype=torch.int64, device="cuda")
        tokens[1], tokens[2] = -100, 1999
        r = gq.logprobs(x, tokens=tokens, entropy=False)
        lp = torch.log_softmax(x.double(), -1)
        assert r.logprob[1] == 0 and r.entropy is None and abs(float(r.logprob[2] - lp[2, 1999])) < 1e-5 and abs(float(r.logprob[0] - lp[0, 5])) < 1e-5
        assert gq.device_error() == 0
        tokens[3] = 2000
        r = gq.logprobs(x, tokens=tokens)
        assert torch.isnan(r.logprob[3]) and torch.isfinite(r.logprob[:3]).all() and gq.device_error() == 8


def test_graph_and_streams(gq):
    xs = [normal(s, 3, 30000) for s in (8, 9)]
    tokens = torch.tensor([1, 2, 3], device="cuda")
    want = [gq.logprobs(x, tokens=tokens, top=6) for x in xs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in xs], []
    for _ in range(3):
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                got.append(gq.logprobs(x, tokens=tokens, top=6))
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(r, want[i % 2]))
    x, work = xs[0].clone(), gq.logprobs_workspace(3, 30000, 6)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = gq.logprobs(x, tokens=tokens, top=6, workspace=work)
    for a, b in zip(xs[::-1], want[::-1]):
        x.copy_(a)
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip(r, b))


def test_refusals(gq):
    x = normal(1, 2, 100)
    for bad in (dict(top=33), dict(top=-1), dict(entropy=False), dict(scale=0.0), dict(tokens=torch.zeros(2, dtype=torch.int32, device="cuda")),
                dict(tokens=torch.zeros(3, dtype=torch.int64, device="cuda")), dict(workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(gq.GQError):
            gq.logprobs(x, **bad)
    with pytest.raises(gq.GQError):
        gq.logprobs(x.double(), top=1)
    with pytest.raises(gq.GQError):
        gq.logprobs(x.t(), top=1)
