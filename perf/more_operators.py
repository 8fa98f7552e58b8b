"""Cases of the operators around products in 8 bits and of what a model answers with: the root-mean-square norm and the
gated quantization that write activations as MXFP8 (``rmsnorm_mx8``, ``quantize_mx8``), the Q4 product that reads them
(``linear_mx8``), and log probabilities of tokens from logits (``logprobs``) or straight from the vocabulary's product
(``linear_logprobs``).  ``run`` computes them in plain torch operations, or with the library where ``own`` is true;
``exact`` computes them in binary64."""
import math

import torch

own = False

EPS = 1e-6


def _norm(name, t, k, residual):
    return {"name": name, "op": "norm", "t": t, "k": k, "residual": residual}


def _quant(name, t, k, gated):
    return {"name": name, "op": "quant", "t": t, "k": k, "gated": gated}


def _linear(name, n, k, t, residual):
    return {"name": name, "op": "linear", "n": n, "k": k, "t": t, "residual": residual}


def _logprobs(name, n, t, top, wide, masked):
    return {"name": name, "op": "logprobs", "n": n, "t": t, "top": top, "wide": wide, "masked": masked}


def _scores(name, n, k, t, top):
    return {"name": name, "op": "scores", "n": n, "k": k, "t": t, "top": top}


def listed():
    return [
        # one token's norm between two layers: latency
        _norm("norm_t1", 1, 5120, True),
        # a long prompt's norm: the stream of activations
        _norm("norm_t4096", 4096, 5120, True),
        # the input of a down projection, an odd batch of requests: gate and up halves of wide rows
        _quant("quant_t9_gated", 9, 17408, True),
        # attention's outputs of a prompt on their way to the output projection
        _quant("quant_t2048", 2048, 6144, False),
        # one token's projection: latency and the weight stream
        _linear("linear_t1", 6144, 5120, 1, False),
        # a down projection (long rows) of an odd batch, added to the residual stream
        _linear("linear_t23_long", 5120, 17408, 23, True),
        # a ragged row count and K, a large batch
        _linear("linear_t101_odd", 7703, 1984, 101, False),
        # a prompt's projection: the matrix cores
        _linear("linear_t1024", 6144, 5120, 1024, False),
        # one request's logits with its alternatives: latency
        _logprobs("logprobs_t1", 131072, 1, 20, False, 0.0),
        # scoring a prompt under a grammar that rules some of the vocabulary out, an odd vocabulary
        _logprobs("logprobs_t500", 50001, 500, 5, True, 0.3),
        # the last product of three requests, with alternatives: the weight stream
        _scores("scores_t3", 131072, 5120, 3, 20),
        # scoring a prompt without keeping its logits
        _scores("scores_t500", 65000, 2048, 500, 2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quant", "linear", "linear", "linear", "logprobs", "scores"])
    while True:
        if op == "norm":
            c = {"op": op, "t": _log(rng, 1, 8192), "k": 64 * _log(rng, 4, 272), "residual": rng.random() < 0.7}
            if c["t"] * c["k"] <= 4096 * 5120:
                return c
        elif op == "quant":
            c = {"op": op, "t": _log(rng, 1, 8192), "k": 64 * _log(rng, 4, 272), "gated": rng.random() < 0.6}
            if c["t"] * c["k"] <= 2048 * 6144:
                return c
        elif op == "linear":
            c = {"op": op, "n": _log(rng, 256, 34816), "k": 64 * _log(rng, 8, 272), "t": _log(rng, 1, 2048),
                 "residual": rng.random() < 0.3}
            if c["n"] * c["k"] <= 34816 * 5120 and c["n"] * c["k"] * c["t"] <= 6144 * 5120 * 1024:
                return c
        elif op == "logprobs":
            c = {"op": op, "n": _log(rng, 1000, 131072), "t": _log(rng, 1, 1024), "top": rng.randint(0, 20),
                 "wide": rng.random() < 0.5, "masked": rng.choice([0.0, 0.0, 0.3, 0.9])}
            if c["n"] * c["t"] <= 50001 * 500:
                return c
        else:
            c = {"op": op, "n": _log(rng, 8000, 131072), "k": 64 * _log(rng, 8, 80), "t": _log(rng, 1, 256)}
            c["top"] = rng.randint(0, 20) if c["t"] <= 8 else rng.randint(0, 3)
            if c["n"] * c["k"] * c["t"] <= 65000 * 2048 * 500:
                return c


# -- inputs -----------------------------------------------------------------
def _gen(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 29)
    return g


def _randn(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _weight(g, n, k):
    """Q4 codes and scales whose rows give outputs of about one for activations of about one."""
    codes = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.rand(n, k // 64, generator=g, device="cuda") + 0.5) * (k ** -0.5 / 4.6)
    return codes, scales.to(torch.float16)


def _activations(g, t, k):
    """MXFP8 activations: a normed row's values, a few channels far larger than the others."""
    v = torch.randn(t, k, generator=g, device="cuda")
    v *= torch.where(torch.rand(k, generator=g, device="cuda") < 0.004, 12.0, 1.0)
    return _to_mx8(v)


def prepare(case, seed):
    g = _gen(case, seed)
    op, t = case["op"], case["t"]
    s = {"case": case}
    if op == "norm":
        k = case["k"]
        s["x"] = _randn(g, t, k, std=0.5)
        s["weight"] = (torch.rand(k, generator=g, device="cuda") + 0.5).to(torch.bfloat16)
        s["residual"] = None
        if case["residual"]:  # the residual stream: larger, with channels that stand out
            wide = torch.where(torch.rand(k, generator=g, device="cuda") < 0.004, 30.0, 2.0)
            s["residual"] = (torch.randn(t, k, generator=g, device="cuda") * wide).to(torch.bfloat16)
        return s
    if op == "quant":
        k = case["k"]
        if case["gated"]:  # both halves of one product's rows
            both = _randn(g, t, 2 * k)
            s["gate"], s["x"] = both[:, :k], both[:, k:]
        else:
            s["gate"], s["x"] = None, _randn(g, t, k)
        return s
    n = case["n"]
    if op == "logprobs":
        logits = torch.randn(t, n, generator=g, device="cuda") * 2.5
        if case["masked"]:
            logits.masked_fill_(torch.rand(t, n, generator=g, device="cuda") < case["masked"], -math.inf)
        s["logits"] = logits if case["wide"] else logits.to(torch.bfloat16)
        s["tokens"] = torch.randint(0, n, (t,), generator=g, device="cuda", dtype=torch.int32)
        return s
    k = case["k"]
    s["values"], s["vscales"] = _activations(g, t, k)
    s["codes"], s["scales"] = _weight(g, n, k)
    if op == "scores":
        s["scales"] *= 2.5  # logits that spread as a model's do
        s["tokens"] = torch.randint(0, n, (t,), generator=g, device="cuda", dtype=torch.int32)
    else:
        s["residual"] = _randn(g, t, n) if case["residual"] else None
    return s


# -- the plain form ---------------------------------------------------------
def _to_mx8(v):
    """Blocks of 32 of ``v`` as E4M3 values and E8M0 scales: the least power of two with which none passes 448."""
    blocks = v.unflatten(-1, (-1, 32))
    man, exp = torch.frexp(blocks.abs().amax(-1))           # the largest magnitude is man 2^exp, 448 = 0.875 2^9
    e = torch.where(man > 0, exp - 9 + (man > 0.875).int(), -127).clamp(min=-127)
    inverse = ((127 - e) << 23).view(torch.float32)         # 2^-e
    values = (blocks * inverse[..., None]).flatten(-2).to(torch.float8_e4m3fn)
    return values, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _from_mx8(values, scales):
    return (values.float().unflatten(-1, (-1, 32)) * scales.float()[..., None]).flatten(-2)


def _dequant(codes, scales):
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8
    return (q.unflatten(-1, (-1, 64)) * scales.float()[..., None]).flatten(-2)


def _plain_norm(s):
    v = s["x"].float()
    if s["residual"] is not None:
        v = v + s["residual"].float()
    y = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    values, scales = _to_mx8(y)
    out = {"values": values, "scales": scales}
    if s["residual"] is not None:
        out["h"] = v.to(torch.bfloat16)
    return out


def _plain_quant(s):
    v = s["x"].float()
    if s["gate"] is not None:
        gate = s["gate"].float()
        v = gate / (1 + torch.exp(-gate)) * v
    values, scales = _to_mx8(v)
    return {"values": values, "scales": scales}


def _plain_linear(s):
    y = _from_mx8(s["values"], s["vscales"]) @ _dequant(s["codes"], s["scales"]).t()
    if s["residual"] is not None:
        y += s["residual"].float()
    return y.to(torch.bfloat16)


def _plain_logprobs(logits, tokens, top):
    m = logits.amax(-1, keepdim=True)
    shifted = logits - m
    e = torch.exp(shifted)
    z = e.sum(-1, keepdim=True)
    lse = torch.log(z)
    entropy = lse[:, 0] - torch.where(e > 0, e * shifted, 0.0).sum(-1) / z[:, 0]
    out = {"logprob": (shifted.gather(1, tokens.long()[:, None]) - lse)[:, 0].float(), "entropy": entropy.float()}
    if top:  # equal ones: the lowest number first
        best, ids = torch.sort(shifted, dim=-1, descending=True, stable=True)
        out["top"] = (best[:, :top] - lse).float()
        out["ids"] = ids[:, :top].to(torch.int32)
    return out


def _plain_scores(s):
    # the products in 64 bits: which of two near logits is the larger depends on them
    logits = _from_mx8(s["values"], s["vscales"]).double() @ _dequant(s["codes"], s["scales"]).double().t()
    return _plain_logprobs(logits, s["tokens"], s["case"]["top"])


def _named(out, top):
    logprob, entropy, best, ids = out
    named = {"logprob": logprob, "entropy": entropy}
    return dict(named, top=best, ids=ids) if top else named


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        import weight_only_bit_q4_amd as q4
        if op == "norm":
            out = q4.rmsnorm_mx8(s["x"], s["weight"], EPS, residual=s["residual"])
            return dict(zip(("values", "scales", "h"), out))
        if op == "quant":
            return dict(zip(("values", "scales"), q4.quantize_mx8(s["x"], gate=s["gate"])))
        if op == "linear":
            return q4.linear_mx8(s["values"], s["vscales"], s["codes"], s["scales"], residual=s["residual"])
        if op == "logprobs":
            return _named(q4.logprobs(s["logits"], s["tokens"], c["top"]), c["top"])
        return _named(q4.linear_logprobs(s["values"], s["vscales"], s["codes"], s["scales"], s["tokens"], c["top"]),
                      c["top"])
    if op == "norm":
        return _plain_norm(s)
    if op == "quant":
        return _plain_quant(s)
    if op == "linear":
        return _plain_linear(s)
    if op == "logprobs":
        return _plain_logprobs(s["logits"].float(), s["tokens"], c["top"])
    return _plain_scores(s)


# -- what a pass cannot do without -------------------------------------------
def work(case):
    op, t = case["op"], case["t"]
    if op == "norm":
        k = case["k"]
        moved = 2 + 33 / 32 + (4 if case["residual"] else 0)
        return {"bytes": moved * t * k + 2 * k, "flops": 4 * t * k}
    if op == "quant":
        k = case["k"]
        return {"bytes": ((4 if case["gated"] else 2) + 33 / 32) * t * k, "flops": (6 if case["gated"] else 2) * t * k}
    n = case["n"]
    if op == "logprobs":
        return {"bytes": (4 if case["wide"] else 2) * t * n + 12 * t + 8 * t * case["top"], "flops": 5 * t * n}
    k = case["k"]
    product = {"bytes": n * k * 34 / 64 + t * k * 33 / 32, "flops": 2 * n * k * t}
    if op == "linear":
        product["bytes"] += (4 if case["residual"] else 2) * t * n
    else:  # the logits need not be stored
        product["bytes"] += 12 * t + 8 * t * case["top"]
        product["flops"] += 5 * t * n
    return product


# -- the definition in 64 bits -----------------------------------------------
def _blocks64(v):
    """The blocks' scaled values before their rounding to E4M3 (whose error both sides then show).  None for the scales:
    one whose block's largest value lies on a border goes either way."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    largest = b.abs().max(-1).values
    e = torch.ceil(torch.log2(torch.clamp(largest, min=448 * 2.0 ** -127) / 448))
    e = torch.where(largest > 448 * torch.exp2(e), e + 1, e)          # log2 is off by its rounding at a power of two
    e = torch.where(largest <= 448 * torch.exp2(e - 1), e - 1, e).clamp(min=-127)
    return (b / torch.exp2(e)[..., None]).reshape(v.shape), None


def _e4m3_64(values):
    b = values.view(torch.uint8).to(torch.int64)
    exp, man = (b // 8) % 16, (b % 8).double()
    v = torch.where(exp > 0, (1 + man / 8) * torch.exp2(exp.double() - 7), man / 8 * 2.0 ** -6)
    return torch.where(b >= 128, -v, v)


def _rows64(s, rows):
    """``x W^T`` for some rows of the weight."""
    x = _e4m3_64(s["values"]) * torch.exp2(s["vscales"].view(torch.uint8).double() - 127).repeat_interleave(32, -1)
    c = s["codes"][rows].to(torch.int64)
    w = torch.empty(c.shape[0], 2 * c.shape[1], dtype=torch.float64, device=c.device)
    w[:, 0::2], w[:, 1::2] = (c % 16 - 8).double(), (c // 16 - 8).double()
    w *= s["scales"][rows].double().repeat_interleave(64, -1)
    return x @ w.t()


def _product64(s, n, k):
    step = max(1, (1 << 27) // k)
    return torch.cat([_rows64(s, slice(i, i + step)) for i in range(0, n, step)], 1)


def _logprobs64(logits, tokens, top):
    lse = torch.logsumexp(logits, -1)
    p = torch.softmax(logits, -1)
    entropy = -torch.special.xlogy(p, p).sum(-1)
    out = {"logprob": logits[torch.arange(len(tokens), device=logits.device), tokens.long()] - lse, "entropy": entropy}
    if top:
        out["top"] = logits.topk(top, -1).values - lse[:, None]
        out["ids"] = None
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        v = s["x"].double()
        if s["residual"] is not None:
            v = v + s["residual"].double()
        y = v / torch.sqrt((v * v).sum(-1, keepdim=True) / case["k"] + EPS) * s["weight"].double()
        values, scales = _blocks64(y)
        out = {"values": values, "scales": scales}
        return dict(out, h=v) if case["residual"] else out
    if op == "quant":
        v = s["x"].double()
        if case["gated"]:
            v = v * s["gate"].double() * torch.sigmoid(s["gate"].double())
        return dict(zip(("values", "scales"), _blocks64(v)))
    if op == "logprobs":
        return _logprobs64(s["logits"].double(), s["tokens"], case["top"])
    y = _product64(s, case["n"], case["k"])
    if op == "linear":
        return y + s["residual"].double() if case["residual"] else y
    return _logprobs64(y, s["tokens"], case["top"])
