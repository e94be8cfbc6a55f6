"""Log probabilities and entropies of rows with one likely token, against the formula in 64 bits: what is left beside it counts, and no sign is wrong.

Bounds (u = 2^-24; R the others' weight relative to the best one's, whose own term is 1).  R is off by s of itself: a term by the exponential (4 u) and its
argument (3 u |t| ln 2, |t| averaging at most ln(vocab) + 10), chains of at most 130 terms and 77 joins, as for other rows.  An addition to a sum that holds the best
term loses at most u of it, and at most what is added: with a gap of more than kRise = 8 (in powers of two) the thread's reference is the best logit, and
there are at most vocab / 1024 + 10 such additions in a thread and 16 joins; a smaller gap leaves terms of up to 2^8, and 8 u a step in the mean of t.
With the reference m at the best logit its own t is not 0 but fma(c, m, -r), r = c m rounded: at most u c |m|.  It is in the sum of 2^t t, so that an addition there
loses at most u of it, u^2 c |m|, however small the others' terms are (1.6e-13 was seen where m = 57: 2^-48 * 1.443 * 57 = 2.9e-13)."""
import math

import pytest
import torch

from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# one part by blocks of 128 and of 512 threads, clusters of two, four and eight, parts through the workspace
ROWS = [(1300, 16384), (400, 16384), (140, 5003), (60, 16384), (3, 49152), (2, 300001), (5, 700)]


@pytest.fixture(scope="module")
def gq():
    need_gpu()
    import gemm_q1_q8_gb300 as m
    return m


def confident(m, vocab, gap, kind, at):
    """Normal rows (deviation 2.5) with one logit `gap` above the largest other one."""
    gen = torch.Generator(device="cuda").manual_seed(m + vocab)
    x = (2.5 * torch.randn(m, vocab, device="cuda", generator=gen)).to(TYPES[kind])
    where = {"first": torch.zeros(m, dtype=torch.int64, device="cuda"), "last": torch.full((m,), vocab - 1, device="cuda"),
             "any": torch.randint(0, vocab, (m,), device="cuda", generator=gen)}[at]
    best = (x.float().amax(-1) + gap).to(TYPES[kind])
    return x.scatter(1, where[:, None], best[:, None]), where


@pytest.mark.parametrize("m,vocab", ROWS)
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("gap", [0.5, 3.0, 6.5, 10.0, 15.0, 20.0, 30.0, 45.0])
def test_one_likely_token(gq, m, vocab, kind, gap):
    for at in ("first", "last", "any"):
        x, where = confident(m, vocab, gap, kind, at)
        other = (where + 1) % vocab
        r, o = gq.logprobs(x, tokens=where, top=3), gq.logprobs(x, tokens=other)
        lp = torch.log_softmax(x.double(), -1)
        h = -(lp.exp() * lp).sum(-1)
        rest = (x.double() - x.double().amax(-1, keepdim=True)).exp().scatter(1, where[:, None], 0.0).sum(-1)
        s = (4 + 3 * (math.log(vocab) + 10) + 210) * U
        adds = (vocab / 1024 + 26) * U
        clear = gap > 6                                                    # 8 ln 2 = 5.6, and a bf16 gap is rounded
        tol = s * rest / (1 + rest) + (torch.minimum(torch.full_like(rest, adds), 2 * rest) if clear else adds)
        tol_h = tol + 2 * s * h + adds * (U * 1.443 * x.double().amax(-1).abs() if clear else 8)
        best = lp.gather(1, where[:, None]).squeeze(1)
        err = (r.logprob.double() - best).abs()
        assert torch.all(err <= tol + 4 * U * best.abs()), (at, float(err.max()))
        err = (r.entropy.double() - h).abs()
        assert torch.all(err <= tol_h + 4 * U * h), (at, float(err.max()))
        assert torch.all(r.logprob <= 0) and torch.all(r.top_logprobs <= 0) and torch.all(r.entropy >= 0)
        assert torch.equal(r.top_logprobs[:, 0], r.logprob) and torch.equal(r.top_ids[:, 0], where)
        want = lp.gather(1, other[:, None]).squeeze(1)
        assert torch.all((o.logprob.double() - want).abs() <= tol + 4 * U * want.abs())


@pytest.mark.parametrize("m,vocab", ROWS)
@pytest.mark.parametrize("kind", TYPES)
def test_one_allowed_token(gq, m, vocab, kind):
    """Its log probability and the entropy are 0, whatever hides the others."""
    for at in ("first", "last", "any"):
        x, where = confident(m, vocab, 0.0, kind, at)
        for hidden in (-math.inf, torch.finfo(TYPES[kind]).min):
            for value in (1.5, -37.3, 1000.0):
                y = torch.full_like(x, hidden).scatter(1, where[:, None], value)
                r = gq.logprobs(y, tokens=where, top=2)
                assert torch.all(r.logprob == 0) and torch.all(r.entropy == 0) and torch.all(r.top_logprobs[:, 0] == 0), (at, hidden, value)
                assert torch.equal(r.top_ids[:, 0], where) and torch.all(r.top_logprobs[:, 1] < -1e4)
