"""The operators between a layer's quantised products, as measured cases: RMS norm with a Q8_0 output,
rotary positions with the append to a Q8_0 key/value cache, reading the cache back, and attention over it.

Each case is run in two forms on the same inputs: a plain one in elementary torch operations in 32 bits, and the
library's entry points.  Outputs held in 8 bits are returned as the values they stand for, in 16-bit
floating point (what a reader of the cache would ask for)."""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ----------------------------------------------------------------------------- the cases

def listed():
    return [
        # one decoded token's norm before the projections: the residual is added, the GEMVs take Q8_0 blocks
        {"name": "norm_1x2560", "op": "norm", "m": 1, "k": 2560, "type": "f32", "residual": True},
        # a prefill chunk of 16-bit activations at the feed-forward width, an odd number of rows, no residual
        {"name": "norm_777x6912_bf16", "op": "norm", "m": 777, "k": 6912, "type": "bf16", "residual": False},
        # a large prefill batch with its residual stream
        {"name": "norm_8192x4096", "op": "norm", "m": 8192, "k": 4096, "type": "f32", "residual": True},
        # one decoded token: 20 query and 5 kv heads, appended to a cache
        {"name": "append_1", "op": "append", "seqs": 1, "t_lo": 1, "t_hi": 1, "ctx": 1000, "hq": 20, "hkv": 5, "hd": 128,
         "rot": 128, "inter": False, "page": 64, "type": "f32"},
        # ragged prompts of one batch, interleaved pairs on half of a 64-wide head, 16 bits
        {"name": "append_ragged_bf16", "op": "append", "seqs": 7, "t_lo": 33, "t_hi": 601, "ctx": 0, "hq": 15, "hkv": 5, "hd": 64,
         "rot": 32, "inter": True, "page": 16, "type": "bf16"},
        # a long prompt
        {"name": "append_8192", "op": "append", "seqs": 1, "t_lo": 8192, "t_hi": 8192, "ctx": 0, "hq": 32, "hkv": 8, "hd": 128,
         "rot": 128, "inter": False, "page": 64, "type": "f32"},
        # a short prefix read back (to move a sequence, or to check a cache)
        {"name": "read_97", "op": "read", "n": 97, "hkv": 5, "hd": 128, "page": 64, "type": "f16"},
        # a whole long sequence read back
        {"name": "read_65536", "op": "read", "n": 65536, "hkv": 8, "hd": 128, "page": 64, "type": "f16"},
        # one sequence decoding: latency counts
        {"name": "attn_1x4096", "op": "attn", "seqs": 1, "t_lo": 1, "t_hi": 1, "l_lo": 4096, "l_hi": 4096, "hq": 20, "hkv": 5, "hd": 128,
         "page": 64, "type": "f32", "tree": False, "cap": 0.0},
        # a serving batch of ragged lengths, one token each
        {"name": "attn_32_ragged", "op": "attn", "seqs": 32, "t_lo": 1, "t_hi": 1, "l_lo": 501, "l_hi": 32768, "hq": 32, "hkv": 8, "hd": 128,
         "page": 64, "type": "f32", "tree": False, "cap": 0.0},
        # drafted trees verified over medium contexts, capped scores
        {"name": "attn_tree_bf16", "op": "attn", "seqs": 8, "t_lo": 9, "t_hi": 33, "l_lo": 1111, "l_hi": 9000, "hq": 15, "hkv": 5, "hd": 64,
         "page": 16, "type": "bf16", "tree": True, "cap": 30.0},
        # a prefill chunk over what came before it
        {"name": "attn_prefill_2048", "op": "attn", "seqs": 1, "t_lo": 2048, "t_hi": 2048, "l_lo": 6144, "l_hi": 6144, "hq": 32, "hkv": 8,
         "hd": 128, "page": 64, "type": "f32", "tree": False, "cap": 0.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        case = _drawn(rng)
        w = work(case)
        if w["flops"] < 1.5e11 and w["bytes"] < 5e8:   # no more than the largest listed cases
            return case


def _drawn(rng):
    op = rng.choice(["norm", "append", "read", "attn", "attn", "attn"])
    kind = rng.choice(["f32", "f32", "f16", "bf16"])
    hkv, group, hd = rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([64, 64, 128, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "norm":
        return {"op": op, "m": _log(rng, 1, 4096), "k": 32 * _log(rng, 8, 256), "type": kind, "residual": rng.random() < 0.7}
    if op == "append":
        seqs = _log(rng, 1, 32)
        hi = _log(rng, 1, 4096 // seqs)
        rot = rng.choice([hd, hd, hd // 2])
        return {"op": op, "seqs": seqs, "t_lo": max(1, hi // rng.choice([1, 2, 5])), "t_hi": hi, "ctx": rng.choice([0, _log(rng, 1, 1000)]),
                "hq": hkv * group, "hkv": hkv, "hd": hd, "rot": rot, "inter": rng.random() < 0.5, "page": page, "type": kind}
    if op == "read":
        return {"op": op, "n": _log(rng, 1, 32768), "hkv": hkv, "hd": hd, "page": page, "type": kind}
    cap = rng.choice([0.0, 0.0, 20.0, 50.0])
    mode = rng.choice(["decode", "decode", "tree", "prefill"])
    if mode == "prefill":
        seqs, t = _log(rng, 1, 4), _log(rng, 65, 1500)
        low = max(1, t // rng.choice([1, 2, 4]))
        ctx = rng.choice([0, _log(rng, 1, 3000)])
        return {"op": op, "seqs": seqs, "t_lo": low, "t_hi": t, "l_lo": t + ctx // 2, "l_hi": t + ctx, "hq": hkv * group, "hkv": hkv, "hd": hd,
                "page": page, "type": kind, "tree": False, "cap": cap}
    seqs = _log(rng, 1, 64)
    longest = _log(rng, 64, 32768 if seqs <= 8 else 8192)
    t = 1 if mode == "decode" else _log(rng, 2, 64)
    return {"op": op, "seqs": seqs, "t_lo": max(1, t // 2), "t_hi": t, "l_lo": max(t, longest // rng.choice([1, 3, 30])), "l_hi": max(t, longest),
            "hq": hkv * group, "hkv": hkv, "hd": hd, "page": page, "type": kind, "tree": mode == "tree", "cap": cap}


def _spread(n, lo, hi):
    """n whole numbers from lo to hi, evenly over their logarithm, in an order that is not sorted."""
    if n == 1:
        return [hi]
    v = [int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)]
    return [v[(i * 7 + 3) % n] for i in range(n)] if n % 7 else v[::-1]


def _lens(case):
    t = _spread(case["seqs"], case["t_lo"], case["t_hi"])
    kv = [max(a, b) for a, b in zip(t, _spread(case["seqs"], case["l_lo"], case["l_hi"])[::-1])]
    return t, kv


# ----------------------------------------------------------------------------- inputs

def _values(gen, *shape):
    """Normal values whose rows differ in size, as activations do."""
    x = torch.randn(*shape, generator=gen, device="cuda")
    return x * (0.3 + 1.4 * torch.rand(*shape[:-1], 1, generator=gen, device="cuda"))


def _quantised(x):
    """Q8_0 over the last axis: int8 codes of x's shape and f16 scales, one per 32 values."""
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    amax = b.abs().amax(-1, keepdim=True)
    d = amax / 127.0
    v = b / torch.where(d == 0, torch.ones_like(d), d)
    low = torch.floor(v)
    q = torch.clamp(low + (v - low >= 0.5).float(), -127, 127)
    return q.reshape(x.shape).to(torch.int8), d.squeeze(-1).half()


def _worth(q, d):
    """The values that Q8_0 codes and scales stand for, in 32 bits."""
    b = q.reshape(*d.shape, 32).float() * d.float().unsqueeze(-1)
    return b.reshape(q.shape)


def _orders(hd, device):
    """Where the cache's chunk of 16 tokens holds its bytes (include/gq.h): for K and V codes and for the scales,
    the (token, element) that stands at each place, flattened."""
    tok, d = torch.meshgrid(torch.arange(16), torch.arange(hd), indexing="ij")
    g, t = tok & 7, (d >> 2) & 3
    unit = 4 * (d >> 6) + t
    if hd > 64:
        unit = unit ^ (4 * (g & 1))
    at_k = tok * hd + unit * 16 + ((d >> 4) & 3) * 4 + (d & 3)
    t, p, g, c = (tok & 7) >> 1, (tok & 1) + 2 * (tok >> 3), (d >> 2) & 7, d >> 5
    row = 4 * p + t
    if hd == 64:
        at_v = row * 64 + (g ^ (4 * (t >> 1))) * 8 + c * 4 + (d & 3)
    else:
        at_v = row * hd + (c >> 2) * 128 + (g ^ (2 * t)) * 16 + (c & 3) * 4 + (d & 3)
    nb = hd // 32
    tok, b = torch.meshgrid(torch.arange(16), torch.arange(nb), indexing="ij")
    at_s = (((tok & 7) >> 1) * 4 + (tok & 1) + 2 * (tok >> 3)) * nb + b
    return [torch.argsort(a.reshape(-1)).to(device) for a in (at_k, at_v, at_s)]


def _laid_out(kq, kd, vq, vd, page):
    """The library's cache of pages that hold these codes [slots, hkv, hd] and scales [slots, hkv, hd / 32]."""
    slots, hkv, hd = kq.shape
    order_k, order_v, order_s = _orders(hd, kq.device)

    def codes(q, order):
        u = q.to(torch.int16)
        u = torch.where(u < 0, 128 - u, u).to(torch.uint8)
        return u.reshape(-1, page // 16, 16, hkv, hd).permute(0, 3, 1, 2, 4).reshape(-1, hkv, page // 16, 16 * hd)[..., order]

    def scales(d):
        s = d.reshape(-1, page // 16, 16, hkv, hd // 32).permute(0, 3, 1, 2, 4).reshape(-1, hkv, page // 16, hd // 2)
        return s[..., order_s].contiguous().view(torch.uint8)

    return torch.cat([codes(kq, order_k), codes(vq, order_v), scales(kd), scales(vd)], dim=-1).contiguous().reshape(-1)


def _paged(gen, lens, page):
    """A block table of sequences of these lengths over pages in random order, and the number of pages."""
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need) + 1, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), max(need), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(need) + 1


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kind = TYPES[case["type"]]
    s = dict(case)
    if case["op"] == "norm":
        m, k = case["m"], case["k"]
        s["x"] = _values(gen, m, k).to(kind)
        s["r"] = (2 * _values(gen, m, k)).to(kind) if case["residual"] else None
        s["w"] = 1 + 0.2 * torch.randn(k, generator=gen, device="cuda")
        s["h"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["act"] = torch.empty(m * (k // 32) * 34, dtype=torch.uint8, device="cuda")
        s["y"] = torch.empty(m, k, dtype=torch.float16, device="cuda")
        return s
    hkv, hd, page = case["hkv"], case["hd"], case["page"]
    if case["op"] == "append":
        lens = _spread(case["seqs"], case["t_lo"], case["t_hi"])
        n, hq, rot = sum(lens), case["hq"], case["rot"]
        table, pages = _paged(gen, [case["ctx"] + v for v in lens], page)
        seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), _i32(lens).long())
        start = torch.cumsum(_i32([0] + lens[:-1]), 0)
        pos = torch.arange(n, device="cuda") - start[seq] + case["ctx"]
        s["slots"] = table[seq, pos // page].long() * page + pos % page
        s["positions"] = pos.to(torch.int32)
        top = case["ctx"] + max(lens)
        angle = torch.arange(top, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        s["rope"] = torch.stack([torch.cos(angle), torch.sin(angle)], -1).float().contiguous()
        # one row of q, k and v a token, as a fused projection writes it
        s["qkv"] = _values(gen, n, hq + 2 * hkv, hd).to(kind)
        s["q_out"] = torch.empty(n, hq, hd, dtype=kind, device="cuda")
        s["pages"] = pages
        s["cache"] = torch.zeros(pages * hkv * (page // 16) * (32 * hd + 2 * hd), dtype=torch.uint8, device="cuda")
        s["k"] = torch.empty(n, hkv, hd, dtype=torch.float16, device="cuda")
        s["v"] = torch.empty(n, hkv, hd, dtype=torch.float16, device="cuda")
        return s
    if case["op"] == "read":
        lens, kv = [], [case["n"]]
    else:
        lens, kv = _lens(case)
    table, pages = _paged(gen, kv, page)
    slots = pages * page
    kq, kd = _quantised(_values(gen, slots, hkv, hd))
    vq, vd = _quantised(_values(gen, slots, hkv, hd))
    s.update(pages=pages, kq=kq, kd=kd, vq=vq, vd=vd, cache=_laid_out(kq, kd, vq, vd, page))
    if case["op"] == "read":
        pos = torch.arange(case["n"], device="cuda")
        s["slots"] = table[0, pos // page].long() * page + pos % page
        s["k"] = torch.empty(case["n"], hkv, hd, dtype=kind, device="cuda")
        s["v"] = torch.empty_like(s["k"])
        return s
    n, hq = sum(lens), case["hq"]
    s.update(table=table, max_q=max(lens), max_kv=max(kv), kv_len=_i32(kv), q_start=torch.cumsum(_i32([0] + lens), 0).to(torch.int32))
    s["q"] = _values(gen, n, hq, hd).to(kind)
    s["out"] = torch.empty_like(s["q"])
    s["tree_mask"] = None
    if case["tree"]:
        # each drafted token follows a random earlier one of its sequence, or the context
        bits = []
        for t in lens:
            parent = (torch.rand(t, generator=gen, device="cuda") * torch.arange(t, device="cuda")).long().tolist()
            mine = []
            for i in range(t):
                mine.append((1 << i) | (mine[parent[i]] if i and parent[i] < i else 0))
            bits += mine
        s["tree_mask"] = torch.tensor([b - (1 << 64) if b >> 63 else b for b in bits], dtype=torch.int64, device="cuda")
    return s


# ----------------------------------------------------------------------------- the plain forms

def _norm(s):
    h = s["x"].float()
    if s["r"] is not None:
        h = h + s["r"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-5) * s["w"]
    out = {"y": _worth(*_quantised(y)).half()}
    if s["r"] is not None:
        out["h"] = h.to(s["x"].dtype)
    return out


def _turned(x, cs, rot, inter):
    cos, sin = cs[..., 0].unsqueeze(1), cs[..., 1].unsqueeze(1)
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _append(s):
    hq, hkv = s["hq"], s["hkv"]
    x = s["qkv"].float()
    cs = s["rope"][s["positions"].long()]
    q = _turned(x[:, :hq], cs, s["rot"], s["inter"])
    k = _turned(x[:, hq:hq + hkv], cs, s["rot"], s["inter"])
    return {"q": q.to(s["qkv"].dtype), "k": _worth(*_quantised(k)).half(), "v": _worth(*_quantised(x[:, hq + hkv:])).half()}


def _read(s):
    kind = s["k"].dtype
    return {"k": _worth(s["kq"][s["slots"]], s["kd"][s["slots"]]).to(kind), "v": _worth(s["vq"][s["slots"]], s["vd"][s["slots"]]).to(kind)}


def _attention(s):
    hq, hkv, hd, page, longest, t = s["hq"], s["hkv"], s["hd"], s["page"], s["max_kv"], s["max_q"]
    seqs, group = s["seqs"], s["hq"] // s["hkv"]
    j = torch.arange(longest, device="cuda")
    slot = s["table"][:, j // page].long() * page + j % page                       # [seqs, longest]
    k = _worth(s["kq"][slot], s["kd"][slot]).permute(0, 2, 3, 1)                   # [seqs, hkv, hd, longest]
    v = _worth(s["vq"][slot], s["vd"][slot]).permute(0, 2, 1, 3)                   # [seqs, hkv, longest, hd]
    begin, count = s["q_start"][:-1].long(), (s["q_start"][1:] - s["q_start"][:-1]).long()
    i = torch.arange(t, device="cuda")
    at = begin[:, None] + torch.minimum(i, count[:, None] - 1)                     # [seqs, t]: short ones repeat their last
    q = s["q"][at].float().reshape(seqs, t, hkv, group, hd).permute(0, 2, 3, 1, 4).reshape(seqs, hkv, group * t, hd)
    score = torch.matmul(q, k) * hd ** -0.5
    if s["cap"]:
        score = s["cap"] * torch.tanh(score / s["cap"])
    new = j - (s["kv_len"].long() - count)[:, None]                                # [seqs, longest]: place among the new tokens
    if s["tree_mask"] is not None:
        bit = (s["tree_mask"][at][:, :, None] >> new.clamp(0, 63)[:, None, :]) & 1
        seen = (new[:, None, :] < 0) | ((bit == 1) & (new < count[:, None])[:, None, :])
    else:
        seen = new[:, None, :] <= torch.minimum(i, count[:, None] - 1)[:, :, None]
    seen = seen & (j < s["kv_len"][:, None])[:, None, :]                           # [seqs, t, longest]
    score = score.reshape(seqs, hkv, group, t, longest).masked_fill(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(seqs, hkv, group * t, longest), v).reshape(seqs, hkv, group, t, hd) / torch.where(total == 0, torch.ones_like(total), total)
    o = o.permute(0, 3, 1, 2, 4).reshape(seqs, t, hq, hd)
    return {"o": o[i < count[:, None]].to(s["q"].dtype)}


PLAIN = {"norm": _norm, "append": _append, "read": _read, "attn": _attention}


# ----------------------------------------------------------------------------- the library's calls

def _own(s):
    import gemm_q1_q8_gb300 as gq
    op = s["op"]
    if op == "norm":
        gq.rmsnorm_q8_0(s["x"], s["w"], 1e-5, residual=s["r"], out=s["act"], sum_out=s["h"])
        gq.dequantize_q8_0(s["act"], s["m"], s["k"], out=s["y"])
        return {"y": s["y"], "h": s["h"]} if s["r"] is not None else {"y": s["y"]}
    kv = s.get("handle")
    if kv is None:
        kv = s["handle"] = gq.KVCacheQ8_0(s["pages"], s["page"], s["hkv"], s["hd"], data=s["cache"])
    if op == "append":
        hq, hkv, x = s["hq"], s["hkv"], s["qkv"]
        gq.rope_kv_append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], kv, s["slots"], rope=s["rope"], positions=s["positions"],
                          interleaved=s["inter"], q_out=s["q_out"])
        gq.kv_read(kv, s["slots"], k_out=s["k"], v_out=s["v"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    if op == "read":
        gq.kv_read(kv, s["slots"], k_out=s["k"], v_out=s["v"])
        return {"k": s["k"], "v": s["v"]}
    work = s.get("work")
    if work is None:
        work = s["work"] = gq.attn_workspace(kv, s["hq"], s["seqs"], s["max_q"], s["q"].dtype)
    gq.attn_q8_0(s["q"], kv, s["table"], s["kv_len"], s["q_start"], s["max_q"], s["max_kv"], softcap=s["cap"],
                 tree_mask=s["tree_mask"], out=s["out"], workspace=work)
    return {"o": s["out"]}


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ----------------------------------------------------------------------------- what a pass needs

def _pairs(case):
    """Query-key pairs that are visible, a query head."""
    t, kv = _lens(case)
    if case["tree"]:
        return sum(a * (b - a) + a for a, b in zip(t, kv))
    return sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(t, kv))


def work(case):
    size = SIZE[case["type"]]
    if case["op"] == "norm":
        n = case["m"] * case["k"]
        streams = size * (3 if case["residual"] else 1)
        # x, the residual, the sum; the blocks written and read back, the f16 values, the weight
        return {"bytes": n * (streams + 2 * 34 / 32 + 2) + 4 * case["k"], "flops": 7 * n}
    hkv, hd = case["hkv"], case["hd"]
    if case["op"] == "append":
        n = sum(_spread(case["seqs"], case["t_lo"], case["t_hi"]))
        new = n * hkv * hd
        q = n * case["hq"] * hd
        # q in and out, k and v in, the cache written and read back, the f16 values, a table row and indices a token
        return {"bytes": 2 * q * size + 2 * new * (size + 2 * 17 / 16 + 2) + n * (4 * case["rot"] + 12), "flops": 3 * (q + new) + 8 * new}
    if case["op"] == "read":
        n = case["n"] * hkv * hd
        return {"bytes": 2 * n * (17 / 16 + size) + 8 * case["n"], "flops": 2 * n}
    t, kv = _lens(case)
    return {"bytes": 2 * sum(kv) * hkv * hd * 17 / 16 + 2 * sum(t) * case["hq"] * hd * size, "flops": 4 * _pairs(case) * case["hq"] * hd}


# ----------------------------------------------------------------------------- the definition in 64 bits

def _blocks64(x):
    """Values of Q8_0 blocks of a float64 array's last axis, from the definition: d = max|x| / 127 kept in f16, codes rounded half up."""
    z = x.unflatten(-1, (-1, 32))
    step = z.abs().max(-1, keepdim=True).values / 127
    code = torch.floor(torch.where(step > 0, z / step.clamp_min(1e-300), 0 * z) + 0.5).clamp(-127, 127)
    return (code * step.to(torch.float32).to(torch.float16).double()).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "norm":
        h = s["x"].double() + (0 if s["r"] is None else s["r"].double())
        y = s["w"].double() * h / torch.sqrt(h.square().sum(-1, keepdim=True) / s["k"] + 1e-5)
        return {"y": _blocks64(y), "h": h} if s["r"] is not None else {"y": _blocks64(y)}
    if s["op"] == "append":
        x, hq, hkv, rot = s["qkv"].double(), s["hq"], s["hkv"], s["rot"]
        z = torch.view_as_complex(s["rope"].double())[s["positions"].long()][:, None]
        pairs = x[..., :rot].unflatten(-1, (-1, 2)) if s["inter"] else x[..., :rot].unflatten(-1, (2, -1)).transpose(-1, -2)
        turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
        y = x.clone()
        y[..., :rot] = turned.flatten(-2) if s["inter"] else turned.transpose(-1, -2).flatten(-2)
        return {"q": y[:, :hq], "k": _blocks64(y[:, hq:hq + hkv]), "v": _blocks64(x[:, hq + hkv:])}

    def values(q, d, at):
        return q[at].double().unflatten(-1, (-1, 32)).mul(d[at].double()[..., None]).flatten(-2)

    if s["op"] == "read":
        return {"k": values(s["kq"], s["kd"], s["slots"]), "v": values(s["vq"], s["vd"], s["slots"])}
    t, kv = _lens(case)
    if 4 * _pairs(case) * case["hq"] * case["hd"] > 2e12:
        return None
    group, cap, page = s["hq"] // s["hkv"], s["cap"], s["page"]
    out, done = [], 0
    for b, (new, n) in enumerate(zip(t, kv)):
        j = torch.arange(n, device="cuda")
        at = s["table"][b].long()[j // page] * page + j % page
        k, v = values(s["kq"], s["kd"], at), values(s["vq"], s["vd"], at)
        place = j - (n - new)
        if s["tree_mask"] is None:
            hidden = place[None] > torch.arange(new, device="cuda")[:, None]
        else:
            mask = s["tree_mask"][done:done + new]
            hidden = (place[None] >= 0) & (torch.bitwise_right_shift(mask[:, None], place.clamp_min(0)[None]) & 1 == 0)
        o = torch.empty(new, s["hq"], s["hd"], dtype=torch.float64, device="cuda")
        for h in range(s["hq"]):
            x = s["q"][done:done + new, h].double() @ k[:, h // group].T / math.sqrt(s["hd"])
            if cap:
                x = cap * torch.tanh(x / cap)
            o[:, h] = torch.softmax(x.masked_fill(hidden, -math.inf), -1) @ v[:, h // group]
        out.append(o)
        done += new
    return {"o": torch.cat(out)}
