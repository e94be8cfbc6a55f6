"""What stands around a layer's 1-bit products and after the last one, as measured cases: a product with bias, activation and
residual in its epilogue, the gated pair of a feed-forward block, the norms after a block and before the next one with the gate
and the residual's addition between them, and the log probabilities of given tokens with entropy and the best alternatives.

Each case is run in two forms on the same inputs: a plain one in elementary torch operations in 32 bits, and the
library's entry points.  Outputs held in 8 bits are returned as the values they stand for, in 16-bit floating point."""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ----------------------------------------------------------------------------- the cases

def listed():
    return [
        # one decoded token: the down projection of a feed-forward block, added to the residual stream
        {"name": "linear_1_down", "op": "linear", "m": 1, "rows": 2560, "n": 6912, "type": "f32", "bias": False, "act": "none",
         "residual": True, "q8": False},
        # a drafted or batched step of an odd number of tokens, with bias and activation, in 16 bits
        {"name": "linear_97_f16", "op": "linear", "m": 97, "rows": 2560, "n": 2560, "type": "f16", "bias": True, "act": "gelu",
         "residual": False, "q8": False},
        # a prefill chunk through the down projection
        {"name": "linear_4096_down", "op": "linear", "m": 4096, "rows": 2560, "n": 6912, "type": "f32", "bias": False, "act": "none",
         "residual": True, "q8": False},
        # one decoded token through gate and up, in Q8_0 for the down product
        {"name": "glu_1", "op": "glu", "m": 1, "rows": 6912, "n": 2560, "type": "f32", "bias": False, "act": "relu2", "q8": True},
        # a serving batch of an odd number of tokens on the wider layer, biases
        {"name": "glu_33_bf16", "op": "glu", "m": 33, "rows": 14336, "n": 4096, "type": "bf16", "bias": True, "act": "silu", "q8": False},
        # a prompt, in Q8_0 for the down product
        {"name": "glu_517", "op": "glu", "m": 517, "rows": 6912, "n": 2560, "type": "f32", "bias": False, "act": "relu2", "q8": True},
        # a large prefill batch on the wider layer
        {"name": "glu_4096_bf16", "op": "glu", "m": 4096, "rows": 14336, "n": 4096, "type": "bf16", "bias": False, "act": "silu", "q8": False},
        # one decoded token between two blocks, Q8_0 for the next products
        {"name": "norm_1x2560", "op": "norm", "m": 1, "k": 2560, "type": "f32", "post": True, "gate": "none", "q8": True},
        # a prefill chunk in 16 bits with a gate for each token
        {"name": "norm_8192x4096_bf16", "op": "norm", "m": 8192, "k": 4096, "type": "bf16", "post": True, "gate": "token", "q8": True},
        # one decoded token's answer with its 20 best alternatives
        {"name": "logprobs_1", "op": "logprobs", "m": 1, "vocab": 49152, "type": "f32", "top": 20, "masked": False},
        # a serving batch under a grammar that allows a tenth of the vocabulary
        {"name": "logprobs_129_masked", "op": "logprobs", "m": 129, "vocab": 49152, "type": "f32", "top": 5, "masked": True},
        # the tokens of a prompt scored
        {"name": "logprobs_4096_bf16", "op": "logprobs", "m": 4096, "vocab": 49152, "type": "bf16", "top": 1, "masked": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        case = _drawn(rng)
        w = work(case)
        if w["flops"] < 9e11 and w["bytes"] < 4e8:   # no more than the largest listed cases
            return case


def _drawn(rng):
    op = rng.choice(["linear", "glu", "norm", "logprobs"])
    kind = rng.choice(["f32", "f32", "f16", "bf16"])
    if op == "norm":
        return {"op": op, "m": _log(rng, 1, 8192), "k": 32 * _log(rng, 8, 256), "type": kind, "post": rng.random() < 0.8,
                "gate": rng.choice(["none", "row", "token"]), "q8": rng.random() < 0.6}
    if op == "logprobs":
        return {"op": op, "m": _log(rng, 1, 2048), "vocab": _log(rng, 500, 200000), "type": kind, "top": rng.choice([0, 1, 2, 5, 20, 32]),
                "masked": rng.random() < 0.3}
    q8 = rng.random() < 0.4
    rows = 32 * _log(rng, 4, 448) if q8 else _log(rng, 100, 14336)
    case = {"op": op, "m": _log(rng, 1, 4096), "rows": rows, "n": 128 * _log(rng, 2, 64), "type": kind, "bias": rng.random() < 0.4,
            "act": rng.choice(["relu2", "silu", "gelu", "gelu_tanh", "relu"]), "q8": q8}
    if op == "linear":
        case["act"] = rng.choice(["none", "none", case["act"]])
        case["residual"] = rng.random() < 0.6
    return case


# ----------------------------------------------------------------------------- inputs

def _values(gen, *shape):
    """Normal values whose rows differ in size, as activations do."""
    x = torch.randn(*shape, generator=gen, device="cuda")
    return x * (0.3 + 1.4 * torch.rand(*shape[:-1], 1, generator=gen, device="cuda"))


def _weights(gen, rows, n):
    """Q1_0 blocks [rows, n / 128, 18] of random signs; scales about n^-1/2, so that products stay of the activations' size."""
    raw = torch.randint(0, 256, (rows, n // 128, 18), generator=gen, device="cuda", dtype=torch.uint8)
    d = n ** -0.5 * (0.5 + torch.rand(rows, n // 128, 1, generator=gen, device="cuda"))
    raw[..., :2] = d.half().view(torch.uint8)
    return raw


def _quantised(x):
    """Q8_0 over the last axis: codes (whole numbers, in f32) [..., blocks, 32] and f16 scales [..., blocks, 1]."""
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    d = b.abs().amax(-1, keepdim=True) / 127.0
    v = b / torch.where(d == 0, torch.ones_like(d), d)
    low = torch.floor(v)
    return torch.clamp(low + (v - low >= 0.5).float(), -127, 127), d.half()


def _blocks(x):
    """The 34-byte Q8_0 blocks of x's rows, [m, k / 32, 34]."""
    q, d = _quantised(x)
    return torch.cat([d.view(torch.uint8), q.to(torch.int8).view(torch.uint8)], -1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kind = TYPES[case["type"]]
    s = dict(case)
    if case["op"] == "norm":
        m, k = case["m"], case["k"]
        s["y"] = _values(gen, m, k).to(kind)                               # what the block gives
        s["x"] = (2 * _values(gen, m, k)).to(kind)                         # the residual stream
        s["post_w"] = 0.5 + 0.2 * torch.randn(k, generator=gen, device="cuda") if case["post"] else None
        s["w"] = 1 + 0.2 * torch.randn(k, generator=gen, device="cuda")
        s["gate_v"] = None
        if case["gate"] != "none":
            s["gate_v"] = (0.7 * torch.randn(1 if case["gate"] == "row" else m, k, generator=gen, device="cuda")).to(kind)
        s["block_scale"], s["residual_scale"] = 0.75, 1.125
        s["h"] = torch.empty(m, k, dtype=kind, device="cuda")
        s["out"] = torch.empty(m * (k // 32) * 34, dtype=torch.uint8, device="cuda") if case["q8"] else torch.empty_like(s["h"])
        s["worth"] = torch.empty(m, k, dtype=torch.float16, device="cuda") if case["q8"] else None
        return s
    if case["op"] == "logprobs":
        m, vocab = case["m"], case["vocab"]
        x = 2.5 * torch.randn(m, vocab, generator=gen, device="cuda")
        x += 8 * torch.rand(m, 1, generator=gen, device="cuda") - 4
        if case["masked"]:
            allowed = torch.rand(m, vocab, generator=gen, device="cuda") < 0.1
            x.masked_fill_(~allowed, float("-inf"))
            x[:, 7 % vocab] = 1.5                                          # one token is always allowed
        s["logits"] = x.to(kind)
        # most given tokens are likely ones
        pick = torch.randint(0, vocab, (m, 8), generator=gen, device="cuda")
        s["tokens"] = pick.gather(1, s["logits"].float().gather(1, pick).argmax(1, keepdim=True)).squeeze(1)
        return s
    m, rows, n = case["m"], case["rows"], case["n"]
    s["act_in"] = _blocks(_values(gen, m, n)).contiguous()
    names = ["w", "up"] if case["op"] == "glu" else ["w"]
    for name in names:
        s[name] = _weights(gen, rows, n)
        s[name + "_bias"] = 0.3 * torch.randn(rows, generator=gen, device="cuda") if case["bias"] else None
    s["r"] = (2 * _values(gen, m, rows)).to(kind) if case.get("residual") else None
    s["out"] = torch.empty(m * (rows // 32) * 34, dtype=torch.uint8, device="cuda") if case["q8"] else torch.empty(m, rows, dtype=kind, device="cuda")
    s["worth"] = torch.empty(m, rows, dtype=torch.float16, device="cuda") if case["q8"] else None
    return s


# ----------------------------------------------------------------------------- the plain forms

def _back(x):
    """The f16 values of x's Q8_0 blocks."""
    q, d = _quantised(x)
    return (q * d.float()).reshape(x.shape).half()


def _signs(raw):
    """The weights of Q1_0 blocks in 32 bits, [rows, n]."""
    bits = (raw[..., 2:, None] >> torch.arange(8, device="cuda", dtype=torch.uint8)) & 1
    one = 2 * bits.reshape(*raw.shape[:2], 128).float() - 1
    return (one * raw[..., :2].contiguous().view(torch.float16).float()).reshape(raw.shape[0], -1)


def _activations(blocks):
    """The values of Q8_0 blocks in 32 bits, [m, k]."""
    d = blocks[..., :2].contiguous().view(torch.float16).float()
    return (blocks[..., 2:].contiguous().view(torch.int8).float() * d).reshape(blocks.shape[0], -1)


def _bent(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "relu2":
        return z.clamp_min(0) * z.clamp_min(0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _sum(x, raw, bias):
    z = torch.matmul(x, _signs(raw).t())
    return z if bias is None else z + bias


def _linear(s):
    z = _bent(_sum(_activations(s["act_in"]), s["w"], s["w_bias"]), s["act"])
    if s["r"] is not None:
        z = z + s["r"].float()
    return {"y": _back(z) if s["q8"] else z.to(s["out"].dtype)}


def _glu(s):
    x = _activations(s["act_in"])
    z = _bent(_sum(x, s["w"], s["w_bias"]), s["act"]) * _sum(x, s["up"], s["up_bias"])
    return {"y": _back(z) if s["q8"] else z.to(s["out"].dtype)}


def _norm(s):
    n = s["y"].float()
    if s["post_w"] is not None:
        n = n * torch.rsqrt((n * n).mean(-1, keepdim=True) + 1e-5) * s["post_w"]
    if s["gate_v"] is not None:
        n = n * s["gate_v"].float()
    h = s["residual_scale"] * s["x"].float() + s["block_scale"] * n
    z = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-5) * s["w"]
    return {"y": _back(z) if s["q8"] else z.to(s["x"].dtype), "h": h.to(s["x"].dtype)}


def _logprobs(s):
    x = s["logits"].float()
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    lse = top + torch.log(total)
    # the entropy: the log of the sum less the mean of what was exponentiated, over the tokens that have any weight
    out = {"logprob": (x.gather(1, s["tokens"][:, None]) - lse).squeeze(1),
           "entropy": (torch.log(total) - torch.where(e > 0, e * (x - top), torch.zeros_like(e)).sum(-1, keepdim=True) / total).squeeze(1)}
    if s["top"]:
        # one whole number for value and place, so that equal values go by their place: a float's bits in the order of its
        # values (both zeros are one value) above the place, backwards
        bits = (x + 0.0).view(torch.int32).long()
        bits = torch.where(bits < 0, -(bits & 0x7fffffff), bits)
        key = bits * (1 << 18) + ((1 << 18) - 1 - torch.arange(x.shape[1], device="cuda"))
        best = torch.topk(key, s["top"], dim=-1).values
        out["top_ids"] = (1 << 18) - 1 - (best & ((1 << 18) - 1))
        out["top_logprobs"] = x.gather(1, out["top_ids"]) - lse
    return out


PLAIN = {"linear": _linear, "glu": _glu, "norm": _norm, "logprobs": _logprobs}


# ----------------------------------------------------------------------------- the library's calls

def _own(s):
    import gemm_q1_q8_gb300 as gq
    op = s["op"]
    if op == "norm":
        f = gq.rmsnorm_block_q8_0 if s["q8"] else gq.rmsnorm_block
        f(s["y"], s["x"], s["w"], post_weight=s["post_w"], eps=1e-5, gate=s["gate_v"], block_scale=s["block_scale"],
          residual_scale=s["residual_scale"], out=s["out"], sum_out=s["h"])
        if s["q8"]:
            gq.dequantize_q8_0(s["out"], s["m"], s["k"], out=s["worth"])
        return {"y": s["worth"] if s["q8"] else s["out"], "h": s["h"]}
    if op == "logprobs":
        work = s.get("work")
        if work is None:
            work = s["work"] = gq.logprobs_workspace(s["m"], s["vocab"], s["top"], device="cuda")
        r = gq.logprobs(s["logits"], tokens=s["tokens"], top=s["top"], workspace=work)
        out = {"logprob": r.logprob, "entropy": r.entropy}
        return {**out, "top_ids": r.top_ids, "top_logprobs": r.top_logprobs} if s["top"] else out
    m, rows, n, kind = s["m"], s["rows"], s["n"], TYPES[s["type"]]
    if "packed" not in s:                                                  # once, when a program loads its weights
        s["packed"] = {name: gq.q1_0_pack(s[name].reshape(-1), rows, n) for name in ("w", "up") if name in s}
        s["work"] = gq.q1_q8_linear_workspace(rows, n, m, dtype=kind, device="cuda")
    act = s["act_in"].view(-1)
    if op == "glu":
        gq.q1_q8_glu(s["packed"]["w"], s["packed"]["up"], act, rows, n, m, activation=s["act"], bias_gate=s["w_bias"], bias_up=s["up_bias"],
                     dtype=kind, q8_0=s["q8"], out=s["out"], workspace=s["work"])
    else:
        gq.q1_q8_linear(s["packed"]["w"], act, rows, n, m, bias=s["w_bias"], activation=s["act"], residual=s["r"], dtype=kind,
                        q8_0=s["q8"], out=s["out"], workspace=s["work"])
    if s["q8"]:
        gq.dequantize_q8_0(s["out"], m, rows, out=s["worth"])
        return {"y": s["worth"]}
    return {"y": s["out"]}


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ----------------------------------------------------------------------------- what a pass needs

def work(case):
    size = SIZE[case["type"]]
    if case["op"] == "norm":
        n = case["m"] * case["k"]
        gate = {"none": 0, "row": case["k"], "token": n}[case["gate"]]
        # the block's output, the stream in and out, the gate; the result, or its blocks written and read back and their f16 values
        result = 2 * 34 / 32 + 2 if case["q8"] else size
        return {"bytes": n * (3 * size + result) + gate * size + 4 * case["k"] * (2 if case["post"] else 1), "flops": 12 * n}
    if case["op"] == "logprobs":
        n = case["m"] * case["vocab"]
        return {"bytes": n * size + case["m"] * (16 + 12 * case["top"]), "flops": 5 * n}
    m, rows, n = case["m"], case["rows"], case["n"]
    pair = 2 if case["op"] == "glu" else 1
    result = 2 * 34 / 32 + 2 if case["q8"] else size
    return {"bytes": pair * rows * (n * 18 / 128 + (4 if case["bias"] else 0)) + m * n * 34 / 32 + m * rows * (result + (size if case.get("residual") else 0)),
            "flops": 2 * pair * m * rows * n}


# ----------------------------------------------------------------------------- the definition in 64 bits

def _blocks64(x):
    """Values of the Q8_0 blocks of a float64 array's last axis, from the definition: d = max|x| / 127 kept in f16, codes rounded half up."""
    z = x.unflatten(-1, (-1, 32))
    step = z.abs().max(-1, keepdim=True).values / 127
    code = torch.floor(torch.where(step > 0, z / step.clamp_min(1e-300), 0 * z) + 0.5).clamp(-127, 127)
    return (code * step.to(torch.float32).to(torch.float16).double()).flatten(-2)


def _function64(name, z):
    if name == "silu":
        return z * torch.special.expit(z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return z * torch.special.expit(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return {"none": z, "relu": torch.relu(z), "relu2": torch.relu(z) ** 2}[name]


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "logprobs":
        lp = s["logits"].double()
        lp = lp - torch.logsumexp(lp, -1, keepdim=True)
        weight = torch.where(lp > -700, lp, 0 * s["tokens"][:, None].double()).mul(lp.exp())
        out = {"logprob": lp[torch.arange(s["m"], device="cuda"), s["tokens"]], "entropy": -weight.sum(-1)}
        if s["top"]:
            order = torch.sort(s["logits"].float(), dim=-1, descending=True, stable=True).indices[:, :s["top"]]
            out.update(top_ids=order, top_logprobs=torch.take_along_dim(lp, order, 1))
        return out
    if s["op"] == "norm":
        def unit(z, w):
            return w.double() * z / torch.sqrt(z.square().sum(-1, keepdim=True) / s["k"] + 1e-5)
        block = s["y"].double() if s["post_w"] is None else unit(s["y"].double(), s["post_w"])
        h = s["x"].double().mul(s["residual_scale"]) + block.mul(s["block_scale"]).mul(1 if s["gate_v"] is None else s["gate_v"].double())
        z = unit(h, s["w"])
        return {"y": _blocks64(z) if s["q8"] else z, "h": h}
    if work(case)["flops"] > 4e12:
        return None
    m, rows, n = s["m"], s["rows"], s["n"]
    byte = s["act_in"]
    x = byte[..., 2:].to(torch.int16)
    x = torch.where(x > 127, x - 256, x).double() * byte[..., :2].contiguous().view(torch.float16).double()
    x = x.reshape(m, n)

    def product(name):
        # the sum over set bits twice, less the sum over all, block of 128 by block
        raw = s[name]
        z = torch.zeros(m, rows, dtype=torch.float64, device="cuda")
        place = torch.arange(128, device="cuda")
        for b in range(n // 128):
            part = x[:, 128 * b:128 * b + 128]
            bit = torch.bitwise_and(raw[:, b, 2:].int()[:, place // 8], torch.bitwise_left_shift(torch.ones_like(place), place % 8).int()) != 0
            z += (2 * part @ bit.double().T - part.sum(-1, keepdim=True)) * raw[:, b, :2].contiguous().view(torch.float16).double().T
        return z if s[name + "_bias"] is None else z + s[name + "_bias"].double()

    z = _function64(s["act"], product("w"))
    if s["op"] == "glu":
        z = z * product("up")
    elif s["r"] is not None:
        z = z + s["r"].double()
    return {"y": _blocks64(z) if s["q8"] else z}
