"""A small 1-bit decoder on the library's calls: prefill of ragged prompts, decoding in a CUDA graph, and drafted trees.

A layer is norm -> Q8_0 -> qkv product -> rotation and append to the paged Q8_0 cache -> attention over it -> norm -> output product, and
norm -> up product -> squared relu -> norm -> down product.  Every product takes its activations in Q8_0 straight from a norm, the residual
stream is added inside the norms, and the cache is only ever read in its quantized form.  Weights and inputs are random.

    python examples/decoder.py
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gemm_q1_q8_gb300 as gq  # noqa: E402


class Shape:
    def __init__(self, hidden=2560, q_heads=20, kv_heads=5, head_dim=128, ffn=6912, layers=2, context=4096):
        self.hidden, self.q_heads, self.kv_heads, self.head_dim = hidden, q_heads, kv_heads, head_dim
        self.ffn, self.layers, self.context = ffn, layers, context


def q1_0(rng, rows, n):
    """Random Q1_0 blocks of a rows x n matrix (f16 scale, 128 sign bits), packed for the library."""
    raw = np.empty((rows * (n // 128), 18), np.uint8)
    raw[:, :2] = (n ** -0.5 * rng.uniform(0.5, 1.5, len(raw))).astype(np.float16).view(np.uint8).reshape(-1, 2)
    raw[:, 2:] = rng.integers(0, 256, (len(raw), 16), dtype=np.uint8)
    return gq.q1_0_pack(torch.from_numpy(raw.reshape(-1)).cuda(), rows, n), torch.from_numpy(raw)


class Layer:
    def __init__(self, s, rng):
        norm = lambda k: torch.from_numpy(rng.uniform(0.8, 1.2, k).astype(np.float32)).cuda()  # noqa: E731
        self.norm, self.norm_o, self.norm_ffn, self.norm_down = norm(s.hidden), norm(s.q_heads * s.head_dim), norm(s.hidden), norm(s.ffn)
        heads = s.q_heads + 2 * s.kv_heads
        self.sizes = {"qkv": (heads * s.head_dim, s.hidden), "o": (s.hidden, s.q_heads * s.head_dim), "up": (s.ffn, s.hidden),
                      "down": (s.hidden, s.ffn)}
        self.packed, self.raw = {}, {}
        for name, (rows, n) in self.sizes.items():
            self.packed[name], self.raw[name] = q1_0(rng, rows, n)


class Batch:
    """What a call's tokens are: their slots and positions, and each sequence's share of them."""

    def __init__(self, slots, positions, kv_len, q_start, max_q, tree_mask=None):
        self.slots, self.positions, self.kv_len, self.q_start, self.max_q, self.tree_mask = slots, positions, kv_len, q_start, max_q, tree_mask


class Decoder:
    def __init__(self, shape, seqs, page=64, seed=0):
        s = self.shape = shape
        rng = np.random.default_rng(seed)
        self.layers = [Layer(s, rng) for _ in range(s.layers)]
        self.final = torch.ones(s.hidden, device="cuda")
        self.rope = gq.rope_table(s.context, s.head_dim, base=500000.0)
        per = -(-s.context // page)
        self.page, self.seqs = page, seqs
        self.caches = [gq.KVCacheQ8_0(seqs * per, page, s.kv_heads, s.head_dim) for _ in self.layers]
        self.table = torch.from_numpy(rng.permutation(seqs * per).astype(np.int32).reshape(seqs, per)).cuda()
        self.kv_len = torch.zeros(seqs, dtype=torch.int32, device="cuda")     # cached tokens of each sequence
        self.every = torch.arange(seqs, device="cuda")
        self.one_each = torch.arange(seqs + 1, dtype=torch.int32, device="cuda")
        self.spaces = {}                                                      # of attention, kept: a captured step holds their addresses

    def workspace(self, max_q):
        need = gq.attn_workspace_bytes(self.caches[0], self.shape.q_heads, self.seqs, max_q)
        if need not in self.spaces:
            self.spaces[need] = torch.empty(need, dtype=torch.uint8, device="cuda")
        return self.spaces[need]

    def slots(self, seq, at):
        """The slots of places `at` of sequences `seq` (equal shapes)."""
        return self.table[seq, at // self.page].long() * self.page + at % self.page

    def product(self, layer, name, act, m):
        rows, n = layer.sizes[name]
        if m == 1:
            return gq.q1_q8_gemv(layer.packed[name], act, rows, n).view(1, rows)
        return gq.q1_q8_gemm(layer.packed[name], act, rows, n, m)

    def forward(self, x, b, seen=None):
        """The residual stream x [n, hidden] (overwritten) of a batch's tokens through the layers; their normed outputs.  The
        tokens' keys and values go to the caches.  seen(name, layer, value): called with each value on the way."""
        s, n = self.shape, x.shape[0]
        tell = seen or (lambda *a: None)
        hq, hkv, hd = s.q_heads, s.kv_heads, s.head_dim
        added = None                                             # what the layer before adds to x, added by the next norm
        for i, (layer, cache) in enumerate(zip(self.layers, self.caches)):
            act = gq.rmsnorm_q8_0(x, layer.norm, residual=added, sum_out=x if added is not None else None)
            tell("act", i, (x, layer.norm, act))
            qkv = self.product(layer, "qkv", act, n)
            tell("qkv", i, (act, qkv))
            qkv = qkv.view(n, hq + 2 * hkv, hd)
            q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
            q = gq.rope_kv_append(q, k, v, cache, b.slots, rope=self.rope, positions=b.positions)
            tell("cache", i, (qkv, q))
            o = gq.attn_q8_0(q, cache, self.table, b.kv_len, b.q_start, b.max_q, s.context, tree_mask=b.tree_mask,
                             workspace=self.workspace(b.max_q))
            tell("attention", i, (q, o))
            act = gq.rmsnorm_q8_0(o.view(n, hq * hd), layer.norm_o)
            y = self.product(layer, "o", act, n)
            act = gq.rmsnorm_q8_0(y, layer.norm_ffn, residual=x, sum_out=x)
            u = self.product(layer, "up", act, n)
            act = gq.rmsnorm_q8_0(torch.relu(u).square(), layer.norm_down)
            added = self.product(layer, "down", act, n)
        return gq.rmsnorm(x, self.final, residual=added)

    def prefill(self, x, counts, seen=None):
        """counts[b] more tokens of each sequence (zero: none)."""
        c = torch.tensor(counts, device="cuda")
        seq = torch.repeat_interleave(self.every, c)
        start = torch.zeros(self.seqs + 1, dtype=torch.int32, device="cuda")
        start[1:] = c.cumsum(0)
        at = torch.arange(len(seq), device="cuda") - start[seq] + self.kv_len[seq]
        self.kv_len += c.int()
        return self.forward(x, Batch(self.slots(seq, at), at.int(), self.kv_len, start, max(counts)), seen)

    def decoding(self, x):
        """A CUDA graph of one token for every sequence, from x [seqs, hidden]: (graph, outputs).  A replay takes x's new
        contents, and advances kv_len."""
        def step():
            at = self.kv_len.clone()
            self.kv_len += 1
            return self.forward(x.clone(), Batch(self.slots(self.every, at), at, self.kv_len, self.one_each, 1))

        kept = self.kv_len.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()                                               # the first call of each kernel outside the graph
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        self.kv_len.copy_(kept)                                  # what the first call wrote lies past the end
        return graph, out

    def verify(self, x, parents):
        """A drafted tree of tokens for every sequence, x [seqs * len(parents), hidden], in order; parents[j] is the index of token
        j's parent (smaller than j), -1 for the newest cached token.  The caches hold the tree past kv_len, which stays."""
        t = len(parents)
        depth, mask = [], []
        for j, p in enumerate(parents):
            depth.append(depth[p] + 1 if p >= 0 else 0)
            mask.append((mask[p] if p >= 0 else 0) | 1 << j)
        mask = [m - (1 << 64) if m >> 63 else m for m in mask]
        seq = self.every.repeat_interleave(t)
        base = self.kv_len[seq]
        at = base + torch.arange(t, device="cuda").repeat(self.seqs)
        positions = base + torch.tensor(depth, device="cuda").repeat(self.seqs)
        start = t * self.one_each
        tree = torch.tensor(mask, dtype=torch.int64, device="cuda").repeat(self.seqs)
        return self.forward(x, Batch(self.slots(seq, at), positions.int(), self.kv_len + t, start, t, tree))

    def accept(self, path):
        """Of the tree just verified the tokens `path` (indices, from the root down) become the sequences' newest.  Values that
        are read back from Q8_0 go to the same codes again, so moving them is exact."""
        seq = self.every.repeat_interleave(len(path))
        base = self.kv_len[seq]
        old = self.slots(seq, base + torch.tensor(path, device="cuda").repeat(self.seqs))
        new = self.slots(seq, base + torch.arange(len(path), device="cuda").repeat(self.seqs))
        for cache in self.caches:
            k, v = gq.kv_read(cache, old)
            gq.rope_kv_append(None, k, v, cache, new)
        self.kv_len += len(path)


def main():
    s = Shape()
    prompts = [517, 33, 1200, 1]
    net = Decoder(s, len(prompts))
    gen = torch.Generator(device="cuda").manual_seed(1)
    tokens = lambda n: torch.randn(n, s.hidden, device="cuda", generator=gen)  # noqa: E731
    net.prefill(tokens(sum(prompts)), prompts)
    x = tokens(len(prompts))
    graph, out = net.decoding(x)
    times = []
    for _ in range(32):
        x.copy_(tokens(len(prompts)))
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b) * 1000)
    print(f"{s.layers} layers, {len(prompts)} sequences of {net.kv_len.tolist()} tokens: {np.median(times):.1f} us a decoding step")
    parents = [-1, 0, 0, 1, 1, 2, 3]                             # seven drafted tokens a sequence
    drafted = tokens(len(prompts) * len(parents))
    y = net.verify(drafted.clone(), parents).view(len(prompts), len(parents), -1)
    path = [0, 1, 3, 6]
    net.accept(path)
    # the accepted tokens again, one after another: the same up to the quantizers' ties
    net.kv_len -= len(path)
    worst = 0.0
    for j in path:
        x.copy_(drafted.view(len(prompts), len(parents), -1)[:, j])
        graph.replay()
        worst = max(worst, float((out - y[:, j]).norm() / y[:, j].norm()))
    print(f"drafted tree against the same tokens in turn: relative difference {worst:.1e}")
    if gq.device_error():
        raise SystemExit("the library reported a device-side error")


if __name__ == "__main__":
    main()
