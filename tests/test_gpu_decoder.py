"""The small decoder of examples/decoder.py: each value on the way against its formula in 64 bits from the values before it, and what has to
agree bit for bit whichever way the tokens came."""
import numpy as np
import pytest
import torch

from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def ex():
    need_gpu()
    from examples import decoder
    return decoder


def small(ex, **k):
    return ex.Shape(**(dict(hidden=256, q_heads=6, kv_heads=2, head_dim=64, ffn=640, layers=2, context=400) | k))


def tokens(n, hidden, seed):
    return torch.randn(n, hidden, generator=torch.Generator().manual_seed(seed)).cuda()


def quantized_close(got, want, blur):
    """Values read back from Q8_0 against the exact ones (known to a relative `blur`): half a step, the f16 rounding of the step (times at
    most 127 codes), the roundings of step and quotient, and the blur."""
    step = want.unflatten(-1, (-1, 32)).abs().amax(-1, keepdim=True) / 127
    bound = (0.5 + 127 * 5 * U + 127 * 2.0 ** -11 + 127 * 2 * blur) * step + 127 * 2.0 ** -25
    return bool(torch.all((got - want).unflatten(-1, (-1, 32)).abs() <= bound))


@pytest.mark.parametrize("head_dim,counts", [(64, [5, 0, 33, 1]), (128, [40, 17]), (64, [100, 3])])
def test_every_value_on_the_way(ex, head_dim, counts):
    gq = ex.gq
    s = small(ex, head_dim=head_dim)
    net = ex.Decoder(s, len(counts), page=16)
    net.prefill(tokens(sum(counts) * 2, s.hidden, 1), [2 * c for c in counts])         # what came before
    hq, hkv, hd, n = s.q_heads, s.kv_heads, head_dim, sum(counts)
    before = net.kv_len.tolist()
    at = np.concatenate([np.arange(b, b + c) for b, c in zip(before, counts)])
    found = []

    def seen(name, i, value):
        layer = net.layers[i]
        found.append(name)
        if name == "act":
            x, w, act = value
            want = x.double() * w.double() / torch.sqrt(x.double().square().mean(-1, keepdim=True) + 1e-5)
            assert quantized_close(gq.dequantize_q8_0(act, n, s.hidden).double(), want, 100 * U)
        elif name == "qkv":
            act, y = value
            a = gq.dequantize_q8_0(act, n, s.hidden).double().cpu()
            raw = layer.raw["qkv"].numpy()
            sign = np.unpackbits(raw[:, 2:], axis=1, bitorder="little").astype(np.float64) * 2 - 1
            w = torch.from_numpy((sign * raw[:, :2].copy().view(np.float16).astype(np.float64)).reshape(layer.sizes["qkv"]))
            # exact integer sums of 32, then two products and a sum in f32 for every block
            assert torch.all((y.double().cpu() - a @ w.T).abs() <= (3 * s.hidden / 32 + 4) * U * (a.abs() @ w.abs().T))
        elif name == "cache":
            qkv, q = value
            z = torch.view_as_complex(net.rope.double())[torch.from_numpy(at).cuda()][:, None]
            x = qkv.double()
            turned = torch.view_as_complex(torch.stack([x[..., :hd // 2], x[..., hd // 2:]], -1)) * z
            turned = torch.cat([turned.real, turned.imag], -1)
            size = x.abs() + x.roll(hd // 2, -1).abs()                                 # two products and their sum
            assert torch.all((q.double() - turned[:, :hq]).abs() <= 2 * U * size[:, :hq])
            b = torch.from_numpy(np.repeat(np.arange(len(counts)), counts)).cuda()
            k, v = gq.kv_read(net.caches[i], net.slots(b, torch.from_numpy(at).cuda()))
            want = turned[:, hq:hq + hkv]
            blur = float((2 * U * size).max() / want.unflatten(-1, (-1, 32)).abs().amax(-1).min())
            assert quantized_close(k.double(), want, blur)
            assert quantized_close(v.double(), x[:, hq + hkv:], U)
        elif name == "attention":
            q, o = value
            done = 0
            for b, c in enumerate(counts):
                if c == 0:
                    continue
                L = before[b] + c
                j = torch.arange(L, device="cuda")
                k, v = (t.double().repeat_interleave(hq // hkv, 1) for t in gq.kv_read(net.caches[i], net.slots(torch.full_like(j, b), j)))
                qq = q[done:done + c].double()
                sc = torch.einsum("thd,lhd->htl", qq, k) * hd ** -0.5
                size = torch.einsum("thd,lhd->htl", qq.abs(), k.abs()) * hd ** -0.5
                hidden = j[None] > before[b] + torch.arange(c, device="cuda")[:, None]
                p = torch.softmax(sc.masked_fill(hidden, -np.inf), -1)
                ds = size.masked_fill(hidden, 0).amax(-1, keepdim=True)
                # a score's products of 22 bits and sums in f32, twice; the exponential and the weight's parts; the sums over the keys
                rel = (2 * ds * 2.0 ** -19 + 2.0 ** -18 + (L / 16 + 64) * 2.0 ** -23).transpose(0, 1)
                want = torch.einsum("htl,lhd->thd", p, v)
                big = torch.einsum("htl,lhd->thd", p, v.abs())
                assert torch.all((o[done:done + c].double() - want).abs() <= rel * big + U * want.abs() + 1e-30)
                done += c

    net.prefill(tokens(n, s.hidden, 2), counts, seen)
    assert found == ["act", "qkv", "cache", "attention"] * s.layers and gq.device_error() == 0


def test_chunks_and_tokens_fill_the_same_cache(ex):
    """The first layer's keys and values depend on their own token alone: bit for bit the same in any split of a prompt."""
    s = small(ex)
    x = tokens(48, s.hidden, 3)
    a, b = ex.Decoder(s, 1, page=16), ex.Decoder(s, 1, page=16)
    a.prefill(x.clone(), [48])
    b.prefill(x[:31].clone(), [31])
    b.prefill(x[31:47].clone(), [16])
    b.prefill(x[47:].clone(), [1])
    j = torch.arange(48, device="cuda")
    for u, v in zip(ex.gq.kv_read(a.caches[0], a.slots(0 * j, j)), ex.gq.kv_read(b.caches[0], b.slots(0 * j, j))):
        assert torch.equal(u, v)
    assert a.kv_len.item() == b.kv_len.item() == 48 and ex.gq.device_error() == 0


def test_decoding_in_a_graph(ex):
    """A captured step gives what a call gives, from the lengths that the steps before left."""
    s = small(ex)
    counts = [7, 64, 1]
    a, b = ex.Decoder(s, 3, page=16), ex.Decoder(s, 3, page=16)
    for net in (a, b):
        net.prefill(tokens(sum(counts), s.hidden, 4), counts)
    x = tokens(3, s.hidden, 5)
    graph, out = a.decoding(x)
    for seed in range(6, 26):
        x.copy_(tokens(3, s.hidden, seed))
        graph.replay()
        assert torch.equal(out, b.prefill(x.clone(), [1, 1, 1]))
    assert a.kv_len.tolist() == b.kv_len.tolist() == [c + 20 for c in counts] and ex.gq.device_error() == 0


def test_drafted_tree(ex):
    """A tree that is a chain gives what the causal mask gives; an accepted branch's keys and values move without change."""
    s = small(ex)
    counts = [20, 3]
    nets = [ex.Decoder(s, 2, page=16) for _ in range(2)]
    for net in nets:
        net.prefill(tokens(23, s.hidden, 7), counts)
    a, b = nets
    x = tokens(10, s.hidden, 8)
    chain = a.verify(x.clone(), [-1, 0, 1, 2, 3])
    assert torch.equal(chain, b.prefill(x.clone(), [5, 5]))
    a.kv_len += 5
    parents, path = [-1, 0, 0, 2, 1, 3, -1], [0, 2, 3, 5]
    a.verify(tokens(14, s.hidden, 9), parents)
    seq = torch.arange(2, device="cuda").repeat_interleave(len(path))
    tree = torch.tensor(path, device="cuda").repeat(2)
    want = [ex.gq.kv_read(c, a.slots(seq, a.kv_len[seq] + tree)) for c in a.caches]
    a.accept(path)
    got = [ex.gq.kv_read(c, a.slots(seq, a.kv_len[seq] - len(path) + torch.arange(len(path), device="cuda").repeat(2))) for c in a.caches]
    for u, v in zip(want, got):
        assert torch.equal(u[0], v[0]) and torch.equal(u[1], v[1])
    assert a.kv_len.tolist() == [29, 12] and ex.gq.device_error() == 0
