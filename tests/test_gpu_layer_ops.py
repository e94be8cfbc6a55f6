"""The operators between a layer's products against plain 64-bit forms: RMS norm with a Q8_0 output, rotary
positions with the append to the paged Q8_0 cache, reading it back, and attention over it.

Where the arithmetic is fixed (quantization, rotation of f32 values, reading back) the results are compared bit
for bit; elsewhere against bounds that follow from the number formats (u = 2^-24; u_t = 2^-24, 2^-11, 2^-8 for an
f32, f16, bf16 result)."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl
from tests.gpu_util import assert_same_bits, need_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ROUND = {"f32": U, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}      # half the distance of f16's subnormals


@pytest.fixture(scope="module")
def gq():
    need_gpu()
    import gemm_q1_q8_gb300 as m
    return m


def normal(seed, *shape):
    return torch.from_numpy(wl.f32_normal(wl.Rng(seed), int(np.prod(shape))).reshape(shape)).cuda()


# ----------------------------------------------------------------------------- norm

def norm_exact(x, r, w, eps):
    h = x.double() + (0 if r is None else r.double())
    return h, h * w.double() / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)


@pytest.mark.parametrize("m,k,kind,residual", [
    (1, 1, "f32", False), (1, 2560, "f32", True), (3, 33, "f32", True), (5, 31, "bf16", True), (2, 4098, "f16", False),
    (200, 4096, "f32", True), (160, 6912, "bf16", True), (153, 960, "f16", True), (2, 65536, "f32", True),
    (1, 40001, "f16", True), (333, 96, "f32", False), (1000, 16384, "bf16", True)])
def test_norm_values(gq, m, k, kind, residual):
    x = normal(1, m, k).to(TYPES[kind])
    r = (3 * normal(2, m, k)).to(TYPES[kind]) if residual else None
    w = 1 + 0.3 * normal(3, k)
    h_out = torch.empty_like(x)
    y = gq.rmsnorm(x, w, 1e-5, residual=r, sum_out=h_out)
    h, want = norm_exact(x, r, w, 1e-5)
    # h: one f32 addition, one rounding to the type
    assert torch.all((h_out.double() - h).abs() <= (ROUND[kind] + U) * h.abs() + TINY[kind])
    # the sum of squares: at most k/(4 threads) + 20 roundings of a running sum of positive terms, and h's own (2 u in h^2);
    # half of that in the root, then a division, an addition, a root, a division, two products
    steps = min(k, 4 * 16) + 20 + 2
    assert torch.all((y.double() - want).abs() <= ((steps / 2 + 8) * U + ROUND[kind]) * want.abs() + TINY[kind])


@pytest.mark.parametrize("m,k,kind", [(1, 2560, "f32"), (7, 32, "f32"), (300, 4096, "bf16"), (2, 40960, "f16"), (170, 6912, "f32")])
def test_norm_q8_0_is_the_quantizer_on_the_norm(gq, m, k, kind):
    """The blocks, the split form and the operand are those of quantize_q8_0 on the f32 norm, bit for bit."""
    x, r = normal(4, m, k).to(TYPES[kind]), normal(5, m, k).to(TYPES[kind])
    w = 1 + 0.3 * normal(6, k)
    x[0, :32] = 0
    r[0, :32] = 0                                        # a block of zeros: d = 0
    y = gq.rmsnorm(x.float(), w, 1e-5, residual=r.float())
    d, q, op = gq.quantize_q8_0(y, mma_operand=True)
    act = gq.rmsnorm_q8_0(x, w, 1e-5, residual=r)
    d2, q2, op2 = gq.rmsnorm_q8_0(x, w, 1e-5, residual=r, split=True, mma_operand=True)
    assert torch.equal(d, d2) and torch.equal(q, q2) and torch.equal(op, op2)
    blocks = act.view(-1, 34)
    assert torch.equal(blocks[:, :2].contiguous().view(torch.int16).flatten(), d.flatten())
    assert torch.equal(blocks[:, 2:].contiguous().view(torch.int8).flatten(), q.flatten())
    for t in TYPES.values():
        back = gq.dequantize_q8_0(act, m, k, dtype=t)
        want = (q.view(m, k // 32, 32).float() * d.view(torch.float16).float()[..., None]).view(m, k).to(t)
        assert torch.equal(back, want)


def test_norm_in_place_and_strided(gq):
    m, k = 40, 1024
    base = normal(7, m, 3 * k)
    x, r = base[:, k:2 * k], normal(8, m, k)
    w = 1 + 0.1 * normal(9, k)
    want = gq.rmsnorm(x.contiguous(), w, 1e-6, residual=r)
    h = x + r
    y = gq.rmsnorm(x, w, 1e-6, residual=r, sum_out=r)     # the residual is updated in place
    assert torch.equal(y, want) and torch.equal(r, h)
    odd = torch.empty(m * k + 1, device="cuda")[1:].view(m, k)    # rows that are not 16-byte aligned
    odd.copy_(h)
    assert torch.equal(gq.rmsnorm(odd, w, 1e-6), gq.rmsnorm(h, w, 1e-6))


# ----------------------------------------------------------------------------- rope and the cache

def rope_reference(positions, rot, base, scaling, factor, original):
    i = np.arange(0, rot, 2, dtype=np.float64)
    size = 1.0
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        c = lambda n: rot * np.log(original / (n * 2 * np.pi)) / (2 * np.log(base))  # noqa: E731
        low, high = (min(max(v, 0), rot - 1) for v in (np.floor(c(32)), np.ceil(c(1))))
        if low == high:
            high += 0.001
        keep = 1 - np.clip((np.arange(rot // 2) - low) / (high - low), 0, 1)
        f = f * keep + f / factor * (1 - keep)
        size = 0.1 * np.log(factor) + 1
    a = np.arange(positions)[:, None] * f
    return np.stack([np.cos(a) * size, np.sin(a) * size], -1)


@pytest.mark.parametrize("scaling,factor,original", [("plain", 1.0, 0), ("linear", 4.0, 0), ("ntk", 2.0, 0), ("yarn", 8.0, 4096),
                                                     ("yarn", 1.0, 64)])
@pytest.mark.parametrize("positions,rot,base", [(1, 8, 10000.0), (5000, 128, 10000.0), (777, 64, 500000.0)])
def test_rope_table(gq, positions, rot, base, scaling, factor, original):
    got = gq.rope_table(positions, rot, base, scaling, factor, original).cpu().numpy()
    want = rope_reference(positions, rot, base, scaling, factor, original)
    # f32 rounding, and an angle's error of a few 2^-53 of itself
    assert np.all(np.abs(got - want) <= U * np.abs(want) + 2e-15 * positions + 1e-12)


def bits16(t, kind):
    return torch.from_numpy(np.ascontiguousarray(t)).to(TYPES[kind])


def rotate_f32(x, cs, rot, inter):
    """The rotation in f32 with every product and sum rounded (x [n, heads, hd], cs [n, rot/2, 2])."""
    y = x.copy()
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    p, q = a * c - b * s, b * c + a * s
    if inter:
        y[..., 0:rot:2], y[..., 1:rot:2] = p, q
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = p, q
    return y


def chunk_bytes(cache, hkv, hd, page, slot, h, pages):
    """One slot's codes and scales by the layout that include/gq.h states."""
    raw = cache.view(pages, hkv, page // 16, 34 * hd)
    c = raw[slot // page, h, (slot % page) // 16].cpu().numpy()
    tok = slot % 16
    t, p = (tok & 7) >> 1, (tok & 1) + 2 * (tok >> 3)
    k, v = np.empty(hd, np.int32), np.empty(hd, np.int32)
    for d in range(hd):
        u = 4 * (d >> 6) + ((d >> 2) & 3)
        if hd > 64 and tok & 1:
            u ^= 4
        k[d] = c[tok * hd + 16 * u + 4 * ((d >> 4) & 3) + (d & 3)]
        g = (d >> 2) & 7
        if hd == 64:
            at = (4 * p + t) * 64 + 8 * (g ^ (4 * (t >> 1))) + 4 * (d >> 5) + (d & 3)
        else:
            at = (4 * p + t) * hd + 128 * (d >> 7) + 16 * (g ^ (2 * t)) + 4 * ((d >> 5) & 3) + (d & 3)
        v[d] = c[16 * hd + at]
    nb = hd // 32
    ks = c[32 * hd:33 * hd].view(np.uint16)[(4 * t + p) * nb:(4 * t + p + 1) * nb]
    vs = c[33 * hd:34 * hd].view(np.uint16)[(4 * t + p) * nb:(4 * t + p + 1) * nb]
    sign = lambda x: np.where(x & 128, -(x & 127), x & 127)  # noqa: E731
    return sign(k), ks, sign(v), vs


@pytest.mark.parametrize("n,hq,hkv,hd,rot,inter,page,kind", [
    (1, 20, 5, 128, 128, False, 64, "f32"), (33, 3, 1, 64, 32, True, 16, "f32"), (17, 4, 2, 256, 256, False, 32, "f32"),
    (50, 8, 8, 128, 64, True, 48, "f32"), (19, 6, 3, 64, 64, False, 128, "bf16"), (40, 2, 1, 256, 8, True, 16, "f16"),
    (21, 0, 2, 128, 0, False, 16, "f32"), (9, 5, 5, 64, 40, False, 64, "f16"), (70, 7, 1, 256, 136, False, 16, "f32")])
def test_append_and_read_back(gq, n, hq, hkv, hd, rot, inter, page, kind):
    pages = -(-n // page) + 3
    qkv = normal(11, n, hq + 2 * hkv, hd).to(TYPES[kind])
    qkv[0, hq, :32] = 0                                      # a block of zeros
    rng = np.random.default_rng(5)
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    if n > 3:
        slots[2] = -1
    cache = gq.KVCacheQ8_0(pages, page, hkv, hd)
    cache.data.fill_(255)
    rope = positions = None
    x = qkv.float().cpu().numpy()
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if rot:
        rope = gq.rope_table(100, rot)
        positions = torch.from_numpy(rng.integers(0, 100, n).astype(np.int32)).cuda()
        cs = rope.cpu().numpy()[positions.cpu().numpy()]
        q, k = rotate_f32(q, cs, rot, inter), rotate_f32(k, cs, rot, inter)
    dslots = torch.from_numpy(slots).cuda()
    got = gq.rope_kv_append(qkv[:, :hq] if hq else None, qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], cache, dslots, rope=rope,
                            positions=positions, interleaved=inter)
    if hq:
        assert torch.equal(got.cpu(), bits16(q, kind))
    want = {}
    for name, t in (("k", k), ("v", v)):
        d, c = oracle.quantize_q8_0(np.ascontiguousarray(t.reshape(n * hkv, hd)), n * hkv, hd)
        want[name] = (np.asarray(d).reshape(n, hkv, hd // 32), np.asarray(c).reshape(n, hkv, hd))
    kept = slots >= 0
    for tk in (torch.float32, torch.bfloat16):
        rk, rv = gq.kv_read(cache, dslots, dtype=tk)
        for t, name in ((rk, "k"), (rv, "v")):
            d, c = want[name]
            val = (c.reshape(n, hkv, hd // 32, 32).astype(np.float32) * d.view(np.float16).astype(np.float32)[..., None]).reshape(n, hkv, hd)
            val[~kept] = 0
            assert torch.equal(t.cpu(), torch.from_numpy(val).to(tk)), name
    for i in [j for j in (0, n // 2, n - 1) if kept[j]]:
        for h in (0, hkv - 1):
            ck, ks, cv, vs = chunk_bytes(cache.data, hkv, hd, page, int(slots[i]), h, pages)
            assert np.array_equal(ck, want["k"][1][i, h]) and np.array_equal(ks, want["k"][0][i, h])
            assert np.array_equal(cv, want["v"][1][i, h]) and np.array_equal(vs, want["v"][0][i, h])
    # nothing but the slots given was written
    untouched = torch.ones(pages * page, dtype=torch.bool)
    untouched[torch.from_numpy(slots[kept])] = False
    other = torch.nonzero(untouched).flatten().cuda()
    rk, rv = gq.kv_read(cache, other)
    assert torch.isnan(rk).all() and torch.isnan(rv).all()   # f16 scales of 0xffff
    assert gq.device_error() == 0


def test_rotation_in_place_and_index_errors(gq):
    n, hq, hkv, hd, page, pages = 12, 4, 2, 256, 16, 2
    qkv = normal(13, n, hq + 2 * hkv, hd)
    rope = gq.rope_table(20, hd)
    positions = torch.arange(n, dtype=torch.int32, device="cuda")
    slots = torch.arange(n, dtype=torch.int64, device="cuda")
    a, b = gq.KVCacheQ8_0(pages, page, hkv, hd), gq.KVCacheQ8_0(pages, page, hkv, hd)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    want = gq.rope_kv_append(q, k, v, a, slots, rope=rope, positions=positions)
    before = qkv.clone()
    got = gq.rope_kv_append(q, k, v, b, slots, rope=rope, positions=positions, q_out=q)
    assert torch.equal(got, want) and torch.equal(qkv[:, hq:], before[:, hq:])
    assert gq.device_error() == 0
    # a position and a slot out of range: that token is left out, the others are as before, the error word says so
    b.data.fill_(0)
    bad_pos, bad_slot = positions.clone(), slots.clone()
    bad_pos[3], bad_slot[5] = 20, pages * page
    out = torch.full_like(want, 7.0)
    gq.rope_kv_append(before[:, :hq], before[:, hq:hq + hkv], before[:, hq + hkv:], b, bad_slot, rope=rope, positions=bad_pos, q_out=out)
    assert gq.device_error() == 8 and gq.device_error() == 0
    keep = torch.ones(n, dtype=torch.bool)
    keep[3] = False
    assert torch.equal(out[keep.cuda()], want[keep.cuda()]) and torch.all(out[3] == 7)
    keep[5] = False
    ka, kb = gq.kv_read(a, slots), gq.kv_read(b, slots)
    for x, y in zip(ka, kb):
        assert torch.equal(x[keep.cuda()], y[keep.cuda()]) and torch.all(y[3] == 0) and torch.all(y[5] == 0)
    rk, _ = gq.kv_read(a, torch.tensor([0, pages * page], device="cuda"))
    assert torch.equal(rk[0], ka[0][0]) and torch.all(rk[1] == 0) and gq.device_error() == 8


# ----------------------------------------------------------------------------- attention

class Filled:
    """A cache of sequences with these lengths, their pages in random order among unwritten ones (whose
    scales are NaN), and the values that it holds."""

    def __init__(self, gq, lens, hkv, hd, page, seed=21, extra=3, size=1.0, first_page=0, data=None, pages=None):
        need = [-(-n // page) for n in lens]
        self.pages = pages or sum(need) + extra
        self.cache = gq.KVCacheQ8_0(self.pages, page, hkv, hd, data=data)
        if data is None:
            self.cache.data.fill_(255)
        order = first_page + np.random.default_rng(seed).permutation(sum(need) + extra).astype(np.int32)
        table = np.full((len(lens), max(max(need), 1)), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.table = torch.from_numpy(table).cuda()
        self.k, self.v = [], []
        for b, n in enumerate(lens):
            if n == 0:
                self.k.append(torch.empty(0, hkv, hd, device="cuda"))
                self.v.append(self.k[-1])
                continue
            j = np.arange(n)
            slots = torch.from_numpy(table[b, j // page].astype(np.int64) * page + j % page).cuda()
            k, v = size * normal(seed + 10 * b + 1, n, hkv, hd), size * normal(seed + 10 * b + 2, n, hkv, hd)
            v *= torch.exp(normal(seed + 10 * b + 3, n, hkv, 1))          # tokens differ in size
            gq.rope_kv_append(None, k, v, self.cache, slots)
            k, v = gq.kv_read(self.cache, slots)
            self.k.append(k)
            self.v.append(v)
        self.lens, self.kv_len = lens, torch.tensor(lens, dtype=torch.int32, device="cuda")


def attention_check(gq, f, counts, hq, kind, cap=0.0, tree=None, q=None, scale=None, out=None):
    """attn_q8_0 on the filled cache against the formula in 64 bits."""
    hkv, hd, n = f.cache.kv_heads, f.cache.head_dim, sum(counts)
    if q is None:
        q = normal(99, n, hq, hd).to(TYPES[kind])
    start = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    o = gq.attn_q8_0(q, f.cache, f.table, f.kv_len, start, max(max(counts), 1), max(max(f.lens), 1), scale=scale, softcap=cap,
                     tree_mask=tree, out=out)
    assert gq.device_error() == 0
    sc = hd ** -0.5 if scale is None else scale
    at = 0
    for b, (t, L) in enumerate(zip(counts, f.lens)):
        if t == 0:
            continue
        kk = f.k[b].double().repeat_interleave(hq // hkv, 1).permute(1, 2, 0)       # [hq, hd, L]
        vv = f.v[b].double().repeat_interleave(hq // hkv, 1).permute(1, 0, 2)       # [hq, L, hd]
        qq = q[at:at + t].double().permute(1, 0, 2)                                 # [hq, t, hd]
        s = sc * qq @ kk
        size = abs(sc) * qq.abs() @ kk.abs()                                        # sum |q k|: what a score's roundings scale with
        if cap:
            s = cap * torch.tanh(s / cap)
        rel = torch.arange(L, device="cuda") - (L - t)
        if tree is None:
            seen = rel[None] <= torch.arange(t, device="cuda")[:, None]
        else:
            seen = (rel[None] < 0) | ((tree[at:at + t][:, None] >> rel.clamp(0, 63)[None]) & 1 == 1)
        s = s.masked_fill(~seen[None], -np.inf)
        top = s.amax(-1, keepdim=True) if L else s.new_full((hq, t, 1), -np.inf)
        p = torch.exp(s - top.clamp_min(-1e300))
        l = p.sum(-1, keepdim=True)
        w = p / torch.where(l == 0, torch.ones_like(l), l)
        want, big = w @ vv, w @ vv.abs()
        ds = (size * seen[None]).amax(-1, keepdim=True) if L else 0.0
        # a score: products of 22-bit (f32) or 11-bit (16-bit types) parts with exact or 11-bit keys, sums in f32;
        # a weight: the score's error twice (itself, and through the sum), the exponential's and its own rounding;
        # the sums over L keys in f32, a rounding for every 16 of them at worst towards one side
        if kind == "f32":
            rel_err = 2 * ds * 2.0 ** -19 + 2.0 ** -18 + (L / 16 + 64) * 2.0 ** -23
        else:
            rel_err = 2 * ds * 2.0 ** -10 + 3 * 2.0 ** -11 + 2.0 ** -18 + (L / 16 + 64) * 2.0 ** -23
        got = o[at:at + t].double().permute(1, 0, 2)
        bound = rel_err * big + ROUND[kind] * want.abs() + 2 * TINY[kind] + 1e-30
        bad = ~((got - want).abs() <= bound)
        assert not bad.any(), (b, t, L, int(bad.sum()), float(((got - want).abs() / bound).max()))
        assert not seen.any(-1).logical_not().any() or torch.all(got[:, ~seen.any(-1)] == 0)
        at += t
    return q, o, start


def trees(counts, seed=3, empty=()):
    """Random drafted trees; the rows in `empty` see no drafted token."""
    rng, bits = np.random.default_rng(seed), []
    for t in counts:
        mine = []
        for i in range(t):
            parent = int(rng.integers(0, i)) if i and rng.random() < 0.9 else None
            mine.append((1 << i) | (mine[parent] if parent is not None else 0))
        bits += mine
    for i in empty:
        bits[i] = 0
    return torch.tensor([b - (1 << 64) if b >> 63 else b for b in bits], dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("lens,hq,hkv,hd,page,kind", [
    ([1], 1, 1, 64, 16, "f32"), ([17, 1, 300], 20, 5, 128, 64, "f32"), ([1000, 16, 15], 3, 1, 256, 32, "f32"),
    ([513], 64, 1, 128, 16, "f32"), ([4097, 5], 8, 8, 64, 128, "f32"), ([33, 64], 32, 8, 128, 64, "f16"),
    ([129] * 40, 4, 2, 64, 48, "bf16"), ([0, 7, 0], 6, 2, 128, 16, "f32"), ([2000, 31], 16, 2, 256, 16, "bf16"),
    ([12345, 3, 700], 5, 1, 128, 256, "f32"), ([5000] * 3, 30, 10, 64, 16, "f16"), ([100000], 4, 1, 128, 64, "f32")])
def test_decode(gq, lens, hq, hkv, hd, page, kind):
    """One token a sequence, from one key to many, lengths of zero, pages that end inside a tile."""
    attention_check(gq, Filled(gq, lens, hkv, hd, page), [1] * len(lens), hq, kind)


@pytest.mark.parametrize("lens,counts,hq,hkv,hd,page,kind,cap", [
    ([40, 100], [8, 3], 4, 2, 64, 16, "f32", 0.0), ([64], [64], 8, 1, 128, 64, "f32", 0.0), ([700, 9, 65], [33, 9, 64], 15, 5, 64, 16, "bf16", 30.0),
    ([3000], [16], 32, 8, 128, 64, "f32", 20.0), ([500, 30], [64, 2], 6, 2, 256, 32, "f16", 0.0), ([2, 1], [2, 1], 3, 3, 128, 16, "f32", 5.0),
    ([9000, 1111], [19, 33], 15, 5, 64, 16, "bf16", 30.0), ([777, 1200], [40, 17], 16, 2, 128, 16, "bf16", 0.0)])
def test_tree(gq, lens, counts, hq, hkv, hd, page, kind, cap):
    """Drafted trees over a cache, with rows that see none of the drafted tokens."""
    empty = [0, counts[0] - 1]
    attention_check(gq, Filled(gq, lens, hkv, hd, page), counts, hq, kind, cap=cap, tree=trees(counts, empty=empty))


@pytest.mark.parametrize("lens,counts,hq,hkv,hd,page,kind,cap", [
    ([5], [5], 1, 1, 64, 16, "f32", 0.0), ([200], [200], 4, 1, 128, 64, "f32", 0.0), ([1000, 130, 65], [300, 130, 0], 8, 2, 64, 16, "f32", 0.0),
    ([700], [257], 2, 2, 256, 32, "f32", 15.0), ([900, 77], [500, 77], 15, 5, 64, 64, "bf16", 0.0), ([640], [513], 6, 1, 128, 16, "f16", 40.0),
    ([4, 0, 300], [9, 3, 310], 4, 4, 128, 16, "f32", 0.0), ([3000], [100], 16, 2, 128, 128, "f16", 0.0), ([300], [300], 3, 1, 256, 16, "bf16", 0.0),
    ([2500, 129], [1100, 127], 12, 4, 128, 64, "f32", 0.0), ([128], [128], 1, 1, 128, 64, "f16", 0.0), ([4000], [90], 5, 1, 64, 16, "f32", 25.0)])
def test_prefill(gq, lens, counts, hq, hkv, hd, page, kind, cap):
    """Causal chunks over what came before them; more queries than cached tokens leave the first ones without keys."""
    attention_check(gq, Filled(gq, lens, hkv, hd, page), counts, hq, kind, cap=cap)


@pytest.mark.parametrize("counts", [[1, 1], [70, 33]])
@pytest.mark.parametrize("size,scale", [(1e-3, 1.0), (40.0, 0.5), (300.0, 0.002)])
def test_sizes_of_values(gq, counts, size, scale):
    """Small and large keys and values (peaked and flat weights), and another scale."""
    f = Filled(gq, [600, 90], 2, 128, 16, size=size)
    attention_check(gq, f, counts, 6, "f32", scale=scale)
    attention_check(gq, f, counts, 6, "f16", scale=scale)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("t", [1, 20, 64])
def test_infinity_and_nan_in_masked_places(gq, hd, t):
    """A drafted token that a row does not see may hold anything: its values do not reach the row."""
    hq, hkv, L = 4, 2, 200
    f = Filled(gq, [L], hkv, hd, 16)
    bits = (1 << t) - 1
    hide = t // 2 if t > 1 else 0
    rows = [bits & ~(1 << hide) & ((1 << (i + 1)) - 1) for i in range(t)]
    tree = torch.tensor([r - (1 << 64) if r >> 63 else r for r in rows], dtype=torch.int64, device="cuda")
    q, want, start = attention_check(gq, f, [t], hq, "f32", tree=tree)
    slot = torch.tensor([int(f.table[0, (L - t + hide) // 16]) * 16 + (L - t + hide) % 16], device="cuda")
    for bad in (float("inf"), 1e30):
        gq.rope_kv_append(None, torch.full((1, hkv, hd), bad, device="cuda"), torch.full((1, hkv, hd), bad, device="cuda"), f.cache, slot)
        got = gq.attn_q8_0(q, f.cache, f.table, f.kv_len, start, t, L, tree_mask=tree)
        assert torch.isfinite(got).all() and torch.allclose(got, want, rtol=1e-4, atol=1e-5)


def test_strided_and_other_stream(gq):
    """q inside a fused row, an output inside a wider one, an append and the attention on a stream of their own."""
    hq, hkv, hd, page, L = 6, 2, 64, 16, 90
    f = Filled(gq, [L, 50], hkv, hd, page)
    counts = [4, 1]
    qkv = normal(31, 5, hq + 2 * hkv, hd)
    q = qkv[:, :hq]
    start = torch.tensor([0, 4, 5], dtype=torch.int32, device="cuda")
    want = gq.attn_q8_0(q.contiguous(), f.cache, f.table, f.kv_len, start, 4, L)
    wide = torch.full((5, 2 * hq, hd), 3.0, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gq.attn_q8_0(q, f.cache, f.table, f.kv_len, start, 4, L, out=wide[:, hq:])
        k2, v2 = normal(32, 1, hkv, hd), normal(33, 1, hkv, hd)
        slot = torch.tensor([int(f.table[0, (L - 1) // page]) * page + (L - 1) % page], device="cuda")
        gq.rope_kv_append(None, k2, v2, f.cache, slot)              # the newest token again: read right after on the stream
        second = gq.attn_q8_0(q, f.cache, f.table, f.kv_len, start, 4, L)
    side.synchronize()
    assert torch.equal(wide[:, hq:], want) and torch.all(wide[:, :hq] == 3)
    f.k[0][L - 1:], f.v[0][L - 1:] = (x for x in gq.kv_read(f.cache, slot))
    _, again, _ = attention_check(gq, f, counts, hq, "f32", q=q.contiguous())
    assert torch.equal(second, again)


@pytest.mark.parametrize("t", [1, 30, 200])
def test_same_bits_every_time(gq, t):
    f = Filled(gq, [3000, 700, 210], 2, 128, 64)
    start = torch.tensor([0, t, 2 * t, 3 * t], dtype=torch.int32, device="cuda")
    q = normal(41, 3 * t, 8, 128)
    work = gq.attn_workspace(f.cache, 8, 3, t)
    runs = []
    for fill in (0, 255, 7):
        work.fill_(fill)
        runs.append(gq.attn_q8_0(q, f.cache, f.table, f.kv_len, start, t, 3000, workspace=work))
    assert torch.equal(runs[0], runs[1]) and torch.equal(runs[0], runs[2])


@pytest.mark.parametrize("t", [1, 100])
def test_offsets_past_32_bits(gq, t):
    """A cache of over 4 GB with the sequence's pages at its end."""
    hkv, hd, page, L = 4, 128, 64, 300
    pages = (5 << 30) // (page * hkv * 34 * hd // 16)
    data = torch.empty(gq.kv_cache_bytes(pages, page, hkv, hd), dtype=torch.uint8, device="cuda")
    assert data.numel() > 1 << 32
    f = Filled(gq, [L], hkv, hd, page, first_page=pages - 8, extra=3, data=data, pages=pages)
    attention_check(gq, f, [t], 8, "f32")


@pytest.mark.parametrize("t", [1, 90])
def test_indices_out_of_range(gq, t):
    """Page indices outside the cache are not seen, lengths past the bounds are cut, and the error word says so."""
    hq, hkv, hd, page, L = 4, 2, 64, 16, 200
    f = Filled(gq, [L, 100], hkv, hd, page)
    start = torch.tensor([0, t, 2 * t], dtype=torch.int32, device="cuda")
    q = normal(51, 2 * t, hq, hd)
    good = gq.attn_q8_0(q, f.cache, f.table, f.kv_len, start, t, L)
    assert gq.device_error() == 0
    bad = f.table.clone()
    bad[0, 1], bad[0, 4] = f.pages, -5
    got = gq.attn_q8_0(q, f.cache, bad, f.kv_len, start, t, L)
    assert gq.device_error() == 8
    assert torch.equal(got[t:], good[t:]) and torch.isfinite(got).all()
    k = torch.cat([f.k[0][:16], f.k[0][32:64], f.k[0][80:]])
    v = torch.cat([f.v[0][:16], f.v[0][32:64], f.v[0][80:]])
    s = torch.einsum("qhd,lhd->qhl", q[:t].double(), k.double().repeat_interleave(2, 1)) * hd ** -0.5
    hidden = torch.arange(k.shape[0], device="cuda")[None] > k.shape[0] - t + torch.arange(t, device="cuda")[:, None]
    w = torch.softmax(s.masked_fill(hidden[:, None], -np.inf), -1)
    want = torch.einsum("qhl,lhd->qhd", w, v.double().repeat_interleave(2, 1))
    assert torch.allclose(got[:t].double(), want, rtol=1e-4, atol=1e-4)
    gq.attn_q8_0(q, f.cache, f.table, f.kv_len, start, t, L - 1)
    assert gq.device_error() == 8


@pytest.mark.parametrize("hd,kind", [(64, "f32"), (128, "f32"), (128, "bf16")])
def test_many_rows_infinity_and_nan_in_masked_places(gq, hd, kind):
    """As above with rows enough for the tensor-core tiles; a row that does see the token is not finite."""
    hq, hkv, L, t = 16, 2, 300, 64
    f = Filled(gq, [L], hkv, hd, 16)
    hide = 20
    rows = [((1 << t) - 1) & ~(1 << hide) & ((1 << (i + 1)) - 1) | (1 << hide if i == 40 else 0) for i in range(t)]
    tree = torch.tensor([r - (1 << 64) if r >> 63 else r for r in rows], dtype=torch.int64, device="cuda")
    q, want, start = attention_check(gq, f, [t], hq, kind, tree=tree)
    slot = torch.tensor([int(f.table[0, (L - t + hide) // 16]) * 16 + (L - t + hide) % 16], device="cuda")
    inf = torch.full((1, hkv, hd), float("inf"), device="cuda")
    for k in (inf, torch.ones_like(inf)):
        gq.rope_kv_append(None, k, inf, f.cache, slot)
        got = gq.attn_q8_0(q, f.cache, f.table, f.kv_len, start, t, L, tree_mask=tree)
        seen = torch.arange(t, device="cuda") == 40
        assert not torch.isfinite(got[seen]).any()
        tol = dict(rtol=1e-4, atol=1e-5) if kind == "f32" else dict(rtol=2e-2, atol=2e-2)
        assert torch.allclose(got[~seen].float(), want[~seen].float(), **tol)
    assert gq.device_error() == 0


def test_many_rows_indices_and_offsets(gq):
    """Page indices outside the cache are not seen, in a cache of over 4 GB, with rows enough for the tensor-core tiles."""
    hkv, hd, page, L, t, hq = 4, 128, 64, 700, 100, 16
    pages = (5 << 30) // (page * hkv * 34 * hd // 16)
    data = torch.empty(gq.kv_cache_bytes(pages, page, hkv, hd), dtype=torch.uint8, device="cuda")
    f = Filled(gq, [L], hkv, hd, page, first_page=pages - 14, extra=3, data=data, pages=pages)
    q, _, start = attention_check(gq, f, [t], hq, "f32")
    bad = f.table.clone()
    bad[0, 1], bad[0, 4] = f.pages, -5
    got = gq.attn_q8_0(q, f.cache, bad, f.kv_len, start, t, L)
    assert gq.device_error() == 8
    keep = torch.ones(L, dtype=torch.bool, device="cuda")
    keep[64:128], keep[256:320] = False, False
    s = torch.einsum("qhd,lhd->qhl", q.double(), f.k[0].double().repeat_interleave(hq // hkv, 1)) * hd ** -0.5
    hidden = (torch.arange(L, device="cuda")[None] > L - t + torch.arange(t, device="cuda")[:, None]) | ~keep[None]
    w = torch.softmax(s.masked_fill(hidden[:, None], -np.inf), -1)
    want = torch.einsum("qhl,lhd->qhd", w, f.v[0].double().repeat_interleave(hq // hkv, 1))
    assert torch.allclose(got.double(), want, rtol=1e-4, atol=1e-4)


@pytest.mark.parametrize("kind", ["f32", "f16"])
def test_many_rows_scales_that_differ(gq, kind):
    """Sequences whose later keys and values are far larger or smaller than the first, over several tiles."""
    hkv, hd, page, L, t, hq = 1, 64, 16, 500, 70, 4
    f = Filled(gq, [L], hkv, hd, page)
    j = torch.arange(L, device="cuda")
    slots = f.table[0, j // page].long() * page + j % page
    size = torch.exp2(((j // 50) * 7 % 11 - 5).float())[:, None, None]
    gq.rope_kv_append(None, normal(61, L, hkv, hd) * size.clamp(max=2.0), normal(62, L, hkv, hd) * size, f.cache, slots)
    f.k[0], f.v[0] = gq.kv_read(f.cache, slots)
    attention_check(gq, f, [t], hq, kind)


@pytest.mark.parametrize("hd,kind,scale,cap", [(64, "f32", None, 0.0), (64, "f32", 1.0, 0.0), (128, "f32", None, 20.0), (64, "bf16", None, 0.0)])
def test_many_rows_over_long_contexts(gq, hd, kind, scale, cap):
    """Runs of so many tiles that f32 sums leave tensor memory several times, also where the maxima move late (large scores)."""
    t, L, heads = 511, 17001, 8
    f = Filled(gq, [L], heads, hd, 64)
    q, o, _ = attention_check(gq, f, [t], heads, kind, scale=scale, cap=cap)
    if kind == "f32" and scale is None and cap == 0.0:
        s = torch.einsum("qhd,lhd->hql", q.double(), f.k[0].double()) * hd ** -0.5
        w = torch.softmax(s.masked_fill(torch.arange(L, device="cuda")[None] > L - t + torch.arange(t, device="cuda")[:, None], -np.inf), -1)
        want = torch.einsum("hql,lhd->qhd", w, f.v[0].double())
        # sums of 96 products of 16, each truncated by up to 2^-23 of a sum that grows (a quarter of it on the average), the scores' 24 likewise
        assert (o.double() - want).norm() <= (96 / 4 + 24 / 4 + 8) * 2.0 ** -23 * want.norm()
