"""Attention over the Q8_0 cache where it can go wrong, against the formula in 64 bits: row numbers outside the call, precision, and values of very
different sizes."""
import ctypes

import numpy as np
import pytest
import torch

from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def gq():
    need_gpu()
    import gemm_q1_q8_gb300 as m
    return m


def normal(seed, *shape):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape, dtype=np.float32)).cuda()


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def cached(gq, keys, values, page=16):
    """A cache of one sequence per (keys, values) [L, heads, hd], its block table, and the values it holds."""
    hkv, hd = keys[0].shape[1:]
    need = [-(-len(k) // page) for k in keys]
    cache = gq.KVCacheQ8_0(sum(need), page, hkv, hd)
    table = torch.full((len(keys), max(need)), -1, dtype=torch.int32, device="cuda")
    held, first = [], 0
    for b, (k, v) in enumerate(zip(keys, values)):
        table[b, :need[b]] = torch.arange(first, first + need[b], device="cuda")
        slots = first * page + torch.arange(len(k), device="cuda")
        gq.rope_kv_append(None, k, v, cache, slots)
        held.append(gq.kv_read(cache, slots))
        first += need[b]
    return cache, table, held


INDEX_ERROR = 8                                                    # GQ_DEVERR_INDEX


@pytest.mark.parametrize("hd,heads,t,kind", [(128, 2, 6, "f32"), (64, 2, 12, "bf16"), (64, 4, 40, "bf16"), (256, 2, 20, "f32"), (128, 8, 90, "f32"),
                                             (64, 8, 90, "bf16")])
def test_row_numbers_outside_the_call(gq, hd, heads, t, kind):
    """Sequences that begin before the rows or past them, end before they begin, or end past the rows.  q and out lie inside larger
    tensors; what is around them stays as it was."""
    L = [200, 130, 140, 0, 150]
    cache, table, _ = cached(gq, [normal(i, max(n, 1), 1, hd) for i, n in enumerate(L)], [normal(9 + i, max(n, 1), 1, hd) for i, n in enumerate(L)])
    kv_len = i32(*L)
    pad, n = 2 * t, 2 * t + 5                                     # the call's rows: pad .. pad + n of the tensors
    big = normal(20, n + 2 * pad, heads, hd).to(TYPES[kind])
    q = big[pad:pad + n]
    # what each leaves whole: (sequence, first row, last row)
    for start, whole in (((-t, t, 2 * t, 0, t, t), [(1, t, 2 * t), (3, 0, t)]), ((0, t, n + t, n + 2 * t, n, n), [(0, 0, t), (1, t, n)])):
        out = torch.full_like(big, 7.0)
        gq.attn_q8_0(q, cache, table, kv_len, i32(*start), 3 * t, 200, out=out[pad:pad + n])
        assert gq.device_error() == INDEX_ERROR
        assert torch.all(out[:pad] == 7) and torch.all(out[pad + n:] == 7)
        got, written = out[pad:pad + n], torch.zeros(n, dtype=torch.bool, device="cuda")
        for b, lo, hi in whole:
            written[lo:hi] = True
            T = start[b + 1] - start[b]
            alone = torch.zeros(T, heads, hd, dtype=q.dtype, device="cuda")
            alone[:hi - lo] = q[lo:hi]
            want = gq.attn_q8_0(alone, cache, table[b:b + 1].contiguous(), kv_len[b:b + 1].contiguous(), i32(0, T), 3 * t, 200)
            tol = dict(rtol=1e-4, atol=1e-5) if kind == "f32" else dict(rtol=2e-2, atol=2e-2)
            assert torch.allclose(got[lo:hi].float(), want[:hi - lo].float(), **tol), (b, lo, hi)
        assert torch.all(got[~written] == 7) and gq.device_error() == 0


def test_rows_of_the_plain_entry_are_those_of_q_start(gq):
    """gq_attn_q8_0 takes q_start's last element as the number of rows: an earlier one past it, or a negative one, is left out."""
    hd, heads, L = 64, 2, 40
    cache, table, _ = cached(gq, [normal(1, L, 1, hd)] * 3, [normal(2, L, 1, hd)] * 3)
    q = normal(3, 12, heads, hd)
    out = torch.full_like(q, 7.0)
    kv_len = i32(L, L, L)
    work = gq.attn_workspace(cache, heads, 3, 4)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731

    def call(start, rows=None):
        args = [p(q[4:]), heads * hd, p(out[4:]), heads * hd, 0, p(cache.data), cache.pages, cache.page_size, p(table), table.shape[1], p(kv_len),
                p(start), None, 3, 4, L, heads, 1, hd, hd ** -0.5, 0.0, p(work), stream]
        if rows is None:
            return gq.lib().gq_attn_q8_0(*args)
        return gq.lib().gq_attn_q8_0_bounded(*args[:13], rows, *args[13:])

    start = i32(-4, 0, 4, 3)                                      # three rows: -4 .. -1 are not theirs, of the third's none is left
    assert call(start) == 0 and gq.device_error() == INDEX_ERROR
    assert torch.all(out[:4] == 7) and torch.all(out[7:] == 7)
    want = gq.attn_q8_0(q[4:8].contiguous(), cache, table[1:2].contiguous(), i32(L), i32(0, 4), 4, L)
    assert torch.allclose(out[4:7], want[:3], rtol=1e-5, atol=1e-6)
    assert call(start, -1) == 1
    out.fill_(7.0)
    assert call(i32(0, 4, 8, 8), 2) == 0 and gq.device_error() == INDEX_ERROR
    assert torch.allclose(out[4:6], want[:2], rtol=1e-5, atol=1e-6) and torch.all(out[6:] == 7) and torch.all(out[:4] == 7)


def exact(q, k, v, scale, seen=None, cap=0.0):
    """o and sum w |v| of one sequence in 64 bits: q [T, heads, hd], k, v [L, kv heads, hd], seen [T, L] (None: causal)."""
    T, L, group = len(q), len(k), q.shape[1] // k.shape[1]
    k, v = k.double().repeat_interleave(group, 1), v.double().repeat_interleave(group, 1)
    s = torch.einsum("thd,lhd->htl", q.double(), k) * scale
    if cap:
        s = cap * torch.tanh(s / cap)
    if seen is None:
        seen = torch.arange(L, device="cuda")[None] <= L - T + torch.arange(T, device="cuda")[:, None]
    w = torch.softmax(s.masked_fill(~seen[None], -torch.inf), -1)
    return torch.einsum("htl,lhd->thd", w, v), torch.einsum("htl,lhd->thd", w, v.abs())


def attend(gq, q, cache, table, L, **kw):
    T = len(q)
    o = gq.attn_q8_0(q, cache, table, i32(L), i32(0, T), T, L, **kw)
    assert gq.device_error() == 0
    return o


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("heads", [4, 8, 64])
@pytest.mark.parametrize("L", [2, 5, 40])
def test_f32_weights_of_small_scores(gq, hd, heads, L):
    """Scores near 0, so that what is left of the error is the exponentials' and the sums': few units of f32's last place."""
    k, v, q = normal(1, L, 1, hd), normal(2, L, 1, hd), 0.005 * normal(3, 1, heads, hd)
    cache, table, [(k, v)] = cached(gq, [k], [v])
    o = attend(gq, q, cache, table, L)
    want, big = exact(q, k, v, hd ** -0.5)
    size = torch.einsum("thd,lhd->thl", q.abs(), k.abs().expand(-1, heads, -1)).amax(-1, keepdim=True) * hd ** -0.5
    # a score's products of 22 bits and sums (as large scores have it); two exponentials of 2^-22; a sum's matrix products, truncated, two for every 16
    # keys; a weight times its scale, and its three parts; the sum's division and product
    rel = 2 * size.double() * 2.0 ** -19 + 2 * 2.0 ** -22 + (L / 16 + 1) * 2 * 2.0 ** -23 + 2.0 ** -23 + 3 * 2.0 ** -24
    assert torch.all((o.double() - want).abs() <= rel * big), float(((o.double() - want).abs() / big).max())


@pytest.mark.parametrize("hd,heads,hkv,seqs,T,L", [(128, 16, 4, 64, 1, 16384), (64, 32, 4, 64, 1, 16384), (128, 16, 1, 16, 8, 8192), (256, 8, 1, 1, 1024, 8192)])
def test_f32_sums_over_long_runs(gq, hd, heads, hkv, seqs, T, L):
    """Many rows over the same pages, so that a warp adds hundreds of chunks.  Equal weights and positive values: what each addition loses has one
    sign if it is truncated, and none if it is rounded."""
    k, v = normal(1, L, hkv, hd), 1 + normal(2, L, hkv, hd).abs()
    cache, table, [(k, v)] = cached(gq, [k], [v], page=64)
    q = torch.zeros(seqs * T, heads, hd, device="cuda")
    o = gq.attn_q8_0(q, cache, table.expand(seqs, -1).contiguous(), i32(*[L] * seqs), i32(*[T * b for b in range(seqs + 1)]), T, L)
    assert gq.device_error() == 0
    mean = v.double().cumsum(0)[L - T:] / (L - T + 1 + torch.arange(T, device="cuda"))[:, None, None]
    want = mean.repeat_interleave(heads // hkv, 1).repeat(seqs, 1, 1)
    rel = (o.double() - want) / want
    # a chunk's two matrix products, truncated (2^-23 each of a sum that is rounded besides), and the division; rounded additions of a run's at most
    # L / 16 chunks, 2^-24 at most of a sum that grows: a third of them all, by their square root
    bias = 2 * 2.0 ** -23 + 2 * 2.0 ** -24
    assert abs(float(rel.mean())) <= bias, float(rel.mean())
    assert float(rel.square().mean().sqrt()) <= bias + 2.0 ** -24 * (L / 16 / 3) ** 0.5, float(rel.square().mean().sqrt())


ROUND = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}               # half the distance of f16's subnormals


def bound(kind, size, L, big, want):
    """Of an output's error, `size` the largest sum |q k| of a score that its row sees.  A score: products of 22-bit (f32) or 11-bit parts, sums in f32; a
    weight: the score's error twice, the exponential's and its own rounding; the sums over L keys; the output's rounding."""
    if kind == "f32":
        rel = 2 * size * 2.0 ** -19 + 2.0 ** -18 + (L / 16 + 64) * 2.0 ** -23
    else:
        rel = 2 * size * 2.0 ** -10 + 3 * 2.0 ** -11 + 2.0 ** -18 + (L / 16 + 64) * 2.0 ** -23
    return rel * big + ROUND[kind] * want.abs() + 2 * TINY[kind]


def one_large_value(gq, kind, spread, where, hd, T, heads, at=10, cap=0.0):
    """One token's values (and keys) are 2^spread times the others'; every row either gives it a weight of some 2^-100 or does not see it."""
    L = 333
    base = 2.0 ** (-6 if kind == "f16" else -12 if spread <= 32 else -17)      # (block scales of 2^-22, the smallest but two)
    k, v, q = normal(1, L, 1, hd), base * normal(2, L, 1, hd), 0.5 * normal(3, T, heads, hd)
    tree = None
    seen = torch.arange(L, device="cuda")[None] <= L - T + torch.arange(T, device="cuda")[:, None]
    if where == "hidden":
        at = L - T                                                # the first of the newest tokens
        k[at] *= 2.0 ** (spread // 2)
        seen[:, at] = False
        tree = torch.tensor([((2 << i) - 1) & ~1 for i in range(T)], dtype=torch.int64, device="cuda")
    else:
        q[..., 0] = q[..., 0].abs() + 8
        k[..., 0] = 0
        k[at] = 0
        k[at, :, 0] = -200.0
    v[at] *= 2.0 ** spread
    cache, table, [(k, v)] = cached(gq, [k], [v])
    q = q.to(TYPES[kind])
    o = attend(gq, q, cache, table, L, tree_mask=tree, softcap=cap)
    want, big = exact(q, k, v, hd ** -0.5, seen=seen, cap=cap)
    size = torch.einsum("thd,lhd->thl", q.double().abs(), k.double().abs().expand(-1, heads, -1)) * hd ** -0.5
    if where != "hidden":
        seen = seen.clone()
        seen[:, at] = False                                       # its weight is nothing, whatever its score's error is
    size = size.masked_fill(~seen[:, None], 0).amax(-1, keepdim=True)
    err = (o.double() - want).abs() / bound(kind, size, L, big, want)
    assert torch.all(err <= 1), float(err.max())


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("T,heads", [(1, 4), (1, 8), (5, 8)])
@pytest.mark.parametrize("where", ["hidden", "faint"])
@pytest.mark.parametrize("kind,spread", [("f32", 32), ("f32", 38), ("f16", 21), ("bf16", 24), ("bf16", 32), ("bf16", 38)])
def test_one_large_value_few_rows(gq, kind, spread, where, hd, T, heads):
    one_large_value(gq, kind, spread, where, hd, T, heads)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("where", ["hidden", "faint", "faint and late"])
@pytest.mark.parametrize("kind,spread", [("f32", 3), ("f32", 16), ("f32", 24), ("f32", 32), ("f16", 21), ("bf16", 24), ("bf16", 32), ("bf16", 38)])
def test_one_large_value_many_rows(gq, kind, spread, where, hd, cap):
    """As above with rows enough for the tensor-core tiles: keys and values of a tile share an exponent only where their own are near."""
    one_large_value(gq, kind, spread, where, hd, 40, 8, at=292 if where == "faint and late" else 10, cap=cap)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("kind,spread", [("f32", 4), ("f32", 14), ("f16", 14), ("bf16", 20)])
def test_many_rows_blocks_of_different_sizes(gq, kind, spread, hd):
    """Every token's first 32 values are 2^spread times the others', its keys by turns; the tokens themselves differ too."""
    L, T, heads = 300, 40, 8
    size = torch.exp2(torch.arange(L, device="cuda") * 5 % 7 - 3.0)[:, None, None]
    k, v, q = 0.1 * normal(1, L, 1, hd), 2.0 ** -8 * size * normal(2, L, 1, hd), normal(3, T, heads, hd)
    v[..., :32] *= 2.0 ** spread
    k[::2, :, 32:] *= 2.0 ** -spread
    cache, table, [(k, v)] = cached(gq, [k], [v])
    q = q.to(TYPES[kind])
    o = attend(gq, q, cache, table, L)
    want, big = exact(q, k, v, hd ** -0.5)
    size = torch.einsum("thd,lhd->thl", q.double().abs(), k.double().abs().expand(-1, heads, -1)) * hd ** -0.5
    err = (o.double() - want).abs() / bound(kind, size.amax(-1, keepdim=True), L, big, want)
    assert torch.all(err <= 1), float(err.max())


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_many_rows_tiles_of_different_sizes(gq, kind, hd):
    """Runs of 64 tokens whose values are by turns 2^-12 to 2^10 of the others': the large ones' weights are nothing, so that what is left is the small
    ones', after sums that have gone up and down with them (f32: some of them have left tensor memory)."""
    L, T, heads = 64 * 44 + 7, 40, 8
    run = torch.arange(L, device="cuda") // 64
    power = torch.tensor([0, -4, 10, 0, 3, -12, 0, 8], device="cuda")[run % 8]
    k, v, q = normal(1, L, 1, hd), torch.exp2(power - 3.0)[:, None, None] * normal(2, L, 1, hd), 0.5 * normal(3, T, heads, hd)
    q[..., 0] = q[..., 0].abs() + 8
    k[..., 0] = torch.where(power <= 0, 0.0, -100.0)[:, None]
    cache, table, [(k, v)] = cached(gq, [k], [v])
    q = q.to(TYPES[kind])
    o = attend(gq, q, cache, table, L)
    want, big = exact(q, k, v, hd ** -0.5)
    faint = (power > 0)[None, None]
    size = (torch.einsum("thd,lhd->thl", q.double().abs(), k.double().abs().expand(-1, heads, -1)) * hd ** -0.5).masked_fill(faint, 0)
    err = (o.double() - want).abs() / bound(kind, size.amax(-1, keepdim=True), L, big, want)
    assert torch.all(err <= 1), float(err.max())


@pytest.mark.parametrize("spread", [9, 11, 12, 13, 14, 18])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_many_rows_around_the_limit_of_a_tile(gq, kind, spread):
    """Tokens' keys and values that differ by about as much as a tile's may share an exponent, all of them with weight; the last tile is not full."""
    L, T, heads, hd = 1000, 40, 8, 128
    j = torch.arange(L, device="cuda")
    large = (j % 7 == 3)[:, None, None]
    k, v, q = 0.1 * normal(1, L, 1, hd), normal(2, L, 1, hd), normal(3, T, heads, hd)
    k, v = torch.where(large, k, k * 2.0 ** -spread), torch.where(large, v * 2.0 ** -spread, v)
    cache, table, [(k, v)] = cached(gq, [k], [v])
    q = q.to(TYPES[kind])
    for cap in (0.0, 20.0):
        o = attend(gq, q, cache, table, L, softcap=cap)
        want, big = exact(q, k, v, hd ** -0.5, cap=cap)
        size = torch.einsum("thd,lhd->thl", q.double().abs(), k.double().abs().expand(-1, heads, -1)) * hd ** -0.5
        err = (o.double() - want).abs() / bound(kind, size.amax(-1, keepdim=True), L, big, want)
        assert torch.all(err <= 1), float(err.max())


def test_two_tokens_with_one_slot(gq):
    """Of a slot that two tokens of a call name nothing is promised; all others hold their token."""
    n, hkv, hd = 500, 4, 128
    k, v = normal(1, n, hkv, hd), normal(2, n, hkv, hd)
    a, b = gq.KVCacheQ8_0(32, 16, hkv, hd), gq.KVCacheQ8_0(32, 16, hkv, hd)
    slots = torch.arange(n, device="cuda")
    gq.rope_kv_append(None, k, v, a, slots)
    twice = slots.clone()
    twice[300] = 17
    gq.rope_kv_append(None, k, v, b, twice)
    others = slots[(slots != 17) & (slots != 300)]
    for x, y in zip(gq.kv_read(a, others), gq.kv_read(b, others)):
        assert torch.equal(x, y)
    assert gq.device_error() == 0


@pytest.mark.parametrize("hd,T,heads", [(128, 1, 8), (64, 4, 8), (256, 5, 8), (128, 40, 8), (64, 40, 8)])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cap", [3e-38, 400.0, 600.0, 3e4, 1e6, 1e9, 3e38])
def test_caps_of_any_size(gq, kind, cap, hd, T, heads):
    """A cap that is large beside the scores leaves them as they are, however large it is; a tiny one makes all weights equal."""
    L = 200
    cache, table, [(k, v)] = cached(gq, [normal(1, L, 1, hd)], [normal(2, L, 1, hd)])
    q = normal(3, T, heads, hd).to(TYPES[kind])
    o = attend(gq, q, cache, table, L, softcap=cap)
    want, big = exact(q, k, v, hd ** -0.5, cap=cap)
    size = torch.einsum("thd,lhd->thl", q.double().abs(), k.double().abs().expand(-1, heads, -1)) * hd ** -0.5
    err = (o.double() - want).abs() / bound(kind, size.amax(-1, keepdim=True), L, big, want)
    assert torch.all(err <= 1), float(err.max())


@pytest.mark.parametrize("hd,T,heads", [(128, 1, 4), (128, 1, 8), (64, 4, 8), (256, 5, 8), (128, 40, 8), (64, 40, 8)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("size,scale,cap", [(-1e33, 1.0, 0.0), (-1e36, 0.1, 0.0), (1e36, 0.1, 0.0), (1e37, 0.01, 0.0), (1e-37, 1e-4, 0.0), (1e-30, 1e-20, 0.0),
                                            (1e37, 0.01, 50.0), (1e-37, 1e-4, 50.0)])
def test_queries_near_the_ends_of_the_range(gq, size, scale, cap, kind, hd, T, heads):
    """Equal keys have equal weights, however large, small or negative the scores are (the largest ones' scores are finite); small keys besides."""
    L = 200
    for key in (1.0, 2.0 ** -14):
        if abs(size) < 1:
            key *= 2.0 ** -9                                      # the smallest block scales
        cache, table, [(k, v)] = cached(gq, [torch.full((L, 1, hd), key, device="cuda")], [normal(2, L, 1, hd)])
        q = torch.full((T, heads, hd), size, device="cuda").to(TYPES[kind])
        o = attend(gq, q, cache, table, L, scale=scale, softcap=cap)
        want = (v.double().cumsum(0)[L - T:] / (L - T + 1 + torch.arange(T, device="cuda"))[:, None, None]).expand(T, heads, hd)
        big = (v.double().abs().cumsum(0)[L - T:] / (L - T + 1 + torch.arange(T, device="cuda"))[:, None, None]).expand(T, heads, hd)
        err = (o.double() - want).abs() / bound(kind, 0.0, L, big, want)
        assert torch.all(err <= 1), float(err.max())


def test_f32_error_over_long_runs(gq):
    """As above with weights that differ: no loss to one side beyond what plain f32 has of either."""
    T, L, heads, hd = 1024, 8192, 8, 256
    k, v = 0.1 * normal(1, L, 1, hd), 1 + normal(2, L, 1, hd).abs()
    cache, table, [(k, v)] = cached(gq, [k], [v], page=64)
    q = normal(3, T, heads, hd)
    o = attend(gq, q, cache, table, L)
    want, _ = exact(q, k, v, hd ** -0.5)
    # 64 chunks of two products, each truncated by 2^-24 on the average of a sum that grows, half of it on the average; the scores' 32 products likewise, of
    # scores below 1/8
    rel = (o.double() - want) / want
    assert abs(float(rel.mean())) <= 64 * 2.0 ** -24 / 2 / 2 + 2.0 ** -24 and float(rel.square().mean().sqrt()) <= 64 * 2.0 ** -24 / 2


@pytest.mark.parametrize("hd,T,heads", [(128, 4, 1), (64, 5, 8), (256, 40, 8), (128, 40, 8), (64, 64, 8)])
@pytest.mark.parametrize("kind,spread", [("f32", 0), ("bf16", 0), ("f32", 20)])
def test_tree_of_more_tokens_than_are_cached(gq, kind, spread, hd, T, heads):
    """The queries before the first cached token see nothing, whatever their masks say."""
    L = T - 3
    k, v = normal(1, L, 1, hd), normal(2, L, 1, hd)
    v[L // 2] *= 2.0 ** -spread
    cache, table, [(k, v)] = cached(gq, [k], [v])
    q = normal(3, T, heads, hd).to(TYPES[kind])
    o = attend(gq, q, cache, table, L, tree_mask=torch.full((T,), -1, dtype=torch.int64, device="cuda"))
    assert torch.all(o[:3] == 0)
    want, big = exact(q[3:], k, v, hd ** -0.5, seen=torch.ones(T - 3, L, dtype=torch.bool, device="cuda"))
    size = torch.einsum("thd,lhd->thl", q[3:].double().abs(), k.double().abs().expand(-1, heads, -1)) * hd ** -0.5
    assert torch.all((o[3:].double() - want).abs() <= bound(kind, size.amax(-1, keepdim=True), L, big, want))


@pytest.mark.parametrize("power", [17, 19, 20, 21, 22, 23, 24, 25, 27, 40])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_scores_beyond_what_f32_resolves(gq, kind, power):
    """Two keys by turns, whose scores are some 2^power apart or equal: of equal ones each has its share, the lower ones have none.  Causal rows see from none
    to all of the high ones of the last tile."""
    L, T, heads, hd = 300, 40, 8, 128
    high = torch.arange(L, device="cuda") % 3 == 1
    k = torch.where(high[:, None, None], 0.75, -0.5) * torch.ones(L, 1, hd, device="cuda")
    v = normal(2, L, 1, hd)
    cache, table, [(k, v)] = cached(gq, [k], [v])
    q = torch.full((T, heads, hd), 1.37 * 2.0 ** power / hd, device="cuda").to(TYPES[kind])
    for scale in (1.0, -1.0):
        o = attend(gq, q, cache, table, L, scale=scale)
        some = high if scale > 0 else ~high
        seen = (torch.arange(L, device="cuda")[None] <= L - T + torch.arange(T, device="cuda")[:, None]) & some[None]
        w = seen.double() / seen.sum(-1, keepdim=True)
        want, big = (torch.einsum("tl,lhd->thd", w, x.double()).expand(T, heads, hd) for x in (v, v.abs()))
        assert torch.all((o.double() - want).abs() <= bound(kind, 0.0, L, big, want))
