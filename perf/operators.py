"""Cases of the operators in which each token picks its own weights: low-rank adapters beside a quantized
projection (``linear_lora``), a mixture-of-experts layer with Q4 experts (``moe``) and its experts alone on given
routing (``moe_experts``).  ``run`` computes them in plain torch operations, or with the library where ``own`` is
true; ``exact`` computes them in binary64."""
import math

import torch

own = False

# the library's weight formats, by number
Q4, Q5, Q6, W8, NVFP4, BF16 = range(6)


def _lora(name, fmt, n, k, t, adapters, rank, order, none):
    return {"name": name, "op": "lora", "fmt": fmt, "n": n, "k": k, "t": t, "adapters": adapters, "rank": rank,
            "order": order, "none": none}


def _moe(name, op, t, experts, top_k, k, inner, renorm, off):
    return {"name": name, "op": op, "t": t, "experts": experts, "top_k": top_k, "k": k, "inner": inner,
            "renorm": renorm, "off": off}


def listed():
    return [
        # one request decoding with its adapter: latency
        _lora("lora_t1", Q4, 6144, 5120, 1, 8, 16, "mixed", 0.0),
        # a few requests, ragged row count and K, a six-bit weight
        _lora("lora_t5_ragged", Q6, 1000, 1984, 5, 6, 24, "mixed", 0.2),
        # a decode batch in which nearly every request has another adapter, some none
        _lora("lora_t32_batch", Q4, 6144, 5120, 32, 32, 64, "mixed", 0.1),
        # an 8-bit down projection (long rows), an odd batch
        _lora("lora_t13_w8", W8, 5120, 17408, 13, 4, 32, "mixed", 0.0),
        # prompts of several requests behind one another
        _lora("lora_t1024_prompts", Q4, 6144, 5120, 1024, 8, 32, "runs", 0.1),
        # one token through many narrow experts: latency
        _moe("moe_t1_narrow", "moe", 1, 128, 8, 2048, 768, True, 0.0),
        # one token through few wide experts: the weight stream
        _moe("moe_t1_wide", "moe", 1, 8, 2, 5120, 14336, True, 0.0),
        # an odd number of tokens, experts and channels; plain softmax weights
        _moe("moe_t7_odd", "moe", 7, 60, 4, 1984, 704, False, 0.0),
        # a decode batch: most experts hit by one or two tokens
        _moe("moe_t16", "moe", 16, 64, 6, 2048, 1408, False, 0.0),
        # a larger batch: every expert hit by a few tokens
        _moe("moe_t64", "moe", 64, 128, 8, 2048, 768, True, 0.0),
        # one rank's share of the experts: three quarters of the choices lie elsewhere
        _moe("experts_t32_share", "experts", 32, 16, 8, 5120, 1536, True, 0.75),
        # few wide experts, each with many tokens
        _moe("moe_t96_wide", "moe", 96, 8, 2, 5120, 14336, True, 0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.45:
        while True:
            fmt = rng.choice([Q4, Q4, Q4, Q5, Q6, W8, NVFP4, BF16])
            n, k, t = _log(rng, 256, 16384), 64 * _log(rng, 8, 160), _log(rng, 1, 1024)
            if n * k <= 6144 * 5120 * 2 and n * k * t <= 6144 * 5120 * 1024:
                break
        return {"op": "lora", "fmt": fmt, "n": n, "k": k, "t": t, "adapters": rng.randint(1, 32),
                "rank": 8 * rng.choice([1, 2, 2, 3, 4, 5, 8, 8, 16]), "order": rng.choice(["mixed", "runs"]),
                "none": rng.choice([0.0, 0.1, 0.5])}
    while True:
        op = rng.choice(["moe", "moe", "experts"])
        t, experts = _log(rng, 1, 128), _log(rng, 4, 200)
        top_k = rng.randint(1, min(8, experts))
        k, inner = 64 * _log(rng, 8, 96), 64 * _log(rng, 4, 96)
        if experts * k * inner <= 400e6 and t * top_k * k * inner <= 96 * 2 * 5120 * 14336:
            break
    return {"op": op, "t": t, "experts": experts, "top_k": top_k, "k": k, "inner": inner,
            "renorm": rng.random() < 0.5, "off": rng.choice([0.0, 0.25, 0.75]) if op == "experts" else 0.0}


# -- inputs -----------------------------------------------------------------
def _gen(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    return g


def _randn(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _bytes(g, *shape):
    return torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)


def _scales(g, *shape, size):
    """fp16 scales between half and one and a half times ``size``."""
    return ((torch.rand(*shape, generator=g, device="cuda") + 0.5) * size).to(torch.float16)


def _weight(g, fmt, n, k):
    """(codes, codes_hi, scales) whose rows give outputs of about one for activations of about one."""
    one = k ** -0.5
    if fmt == Q4:
        return _bytes(g, n, k // 2), None, _scales(g, n, k // 64, size=one / 4.6)
    if fmt == Q5:
        return _bytes(g, n, k // 2), _bytes(g, n, k // 8), _scales(g, n, k // 64, size=one / 9.2)
    if fmt == Q6:
        return _bytes(g, n, k // 2), _bytes(g, n, k // 4), _scales(g, n, k // 64, size=one / 18.5)
    if fmt == W8:
        return _bytes(g, n, k), None, _scales(g, n, k // 32, size=one / 74)
    if fmt == NVFP4:
        # E4M3 with exponent fields 2..4: 2^-5 to 2^-2
        return _bytes(g, n, k // 2), None, torch.randint(0x10, 0x28, (n, k // 16), generator=g, device="cuda",
                                                         dtype=torch.uint8)
    return _randn(g, n, k, std=one), None, None


def prepare(case, seed):
    g = _gen(case, seed)
    t, k = case["t"], case["k"]
    s = {"case": case, "x": _randn(g, t, k)}
    if case["op"] == "lora":
        n, r, l = case["n"], case["rank"], case["adapters"]
        s["w"], s["w_hi"], s["scales"] = _weight(g, case["fmt"], n, k)
        s["a"] = _randn(g, l, r, k, std=k ** -0.5)
        s["b"] = _randn(g, l, n, r, std=r ** -0.5)
        s["lora_scale"] = torch.rand(l, generator=g, device="cuda") + 0.25
        ids = torch.randint(0, l, (t,), generator=g, device="cuda", dtype=torch.int32)
        ids[torch.rand(t, generator=g, device="cuda") < case["none"]] = -1
        if case["order"] == "runs":  # tokens of a request lie behind one another
            ids = ids.sort().values
        s["ids"] = ids
        return s
    e, i = case["experts"], case["inner"]
    for name, n, kk in (("gate", i, k), ("up", i, k), ("down", k, i)):
        s[name] = _bytes(g, e, n, kk // 2), _scales(g, e, n, kk // 64, size=kk ** -0.5 / 4.6)
    if case["op"] == "moe":
        s["router"] = _randn(g, e, k, std=1.5 * k ** -0.5)
        return s
    # routing over all ranks' experts, those of other ranks outside 0..E-1
    every = max(case["top_k"], int(round(e / (1.0 - case["off"]))))
    p = torch.rand(t, every, generator=g, device="cuda")
    w, ids = p.topk(case["top_k"], dim=1)
    s["ids"] = torch.where(ids < e, ids, -1).to(torch.int32)
    s["weights"] = w / w.sum(1, keepdim=True)
    return s


# -- the plain form ---------------------------------------------------------
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _nibbles(codes):
    return torch.stack((codes & 15, codes >> 4), -1).flatten(-2)


def _bits(plane, width):
    shift = torch.arange(0, 8, width, device=plane.device, dtype=torch.uint8)
    return ((plane[..., None] >> shift) & ((1 << width) - 1)).flatten(-2)


def _scaled(values, scales, group):
    return (values.unflatten(-1, (-1, group)) * scales.float()[..., None]).flatten(-2)


def _dequant(fmt, codes, hi, scales):
    """The weight's values in 32 bits."""
    if fmt == Q4:
        return _scaled(_nibbles(codes).float() - 8, scales, 64)
    if fmt == Q5:
        return _scaled((_nibbles(codes) + 16 * _bits(hi, 1)).float() - 16, scales, 64)
    if fmt == Q6:
        return _scaled((_nibbles(codes) + 16 * _bits(hi, 2)).float() - 32, scales, 64)
    if fmt == W8:
        return _scaled(codes.view(torch.int8).float(), scales, 32)
    if fmt == NVFP4:
        table = torch.tensor(_E2M1, device=codes.device)
        return _scaled(table[_nibbles(codes).long()], scales.view(torch.float8_e4m3fn), 16)
    return codes.float()


def _plain_lora(s):
    c = s["case"]
    l, r, t, n = c["adapters"], c["rank"], c["t"], c["n"]
    x = s["x"].float()
    y = x @ _dequant(c["fmt"], s["w"], s["w_hi"], s["scales"]).t()
    u = (x @ s["a"].float().flatten(0, 1).t()).view(t, l, r)
    mine = s["ids"][:, None] == torch.arange(l, device=x.device)  # [T, L]
    u = torch.where(mine[..., None], u * s["lora_scale"][:, None], 0.0)
    y += u.view(t, l * r) @ s["b"].float().transpose(1, 2).reshape(l * r, n)
    return y.to(torch.bfloat16)


def _plain_route(s):
    c = s["case"]
    logits = s["x"].double() @ s["router"].double().t()
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :c["top_k"]]
    w = torch.softmax(logits, 1).gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return ids.to(torch.int32), w.float()


def _plain_experts(s, ids, weights):
    c = s["case"]
    t, e, top_k = c["t"], c["experts"], c["top_k"]
    x = s["x"].float()
    valid = (ids >= 0) & (ids < e)
    w = torch.where(valid, weights, 0.0)
    at = torch.where(valid, ids, 0).long()
    if t * top_k < e:  # the chosen experts' weights, one copy for each choice
        pick = at.flatten()
        deq = lambda m: _dequant(Q4, s[m][0][pick], None, s[m][1][pick])  # noqa: E731
        xp = x.repeat_interleave(top_k, 0)[..., None]
        h = torch.nn.functional.silu(deq("gate") @ xp) * (deq("up") @ xp)
        y = ((deq("down") @ h).view(t, top_k, -1) * w[..., None]).sum(1)
        return y.to(torch.bfloat16)
    # every expert on every token, weighted
    mix = torch.zeros(t, e, device=x.device).scatter_add_(1, at, w)
    deq = lambda m: _dequant(Q4, s[m][0], None, s[m][1])  # noqa: E731
    xt = x.t().contiguous()
    h = torch.nn.functional.silu(deq("gate") @ xt) * (deq("up") @ xt) * mix.t()[:, None, :]
    return (deq("down") @ h).sum(0).t().to(torch.bfloat16).contiguous()


def run(state):
    s, c = state, state["case"]
    if own:
        import weight_only_bit_q4_amd as q4
        if c["op"] == "lora":
            return q4.linear_lora(s["x"], s["w"], s["scales"], s["a"], s["b"], s["ids"], s["lora_scale"],
                                  fmt=c["fmt"], codes_hi=s["w_hi"])
        if c["op"] == "moe":
            y, ids, weights = q4.moe(s["x"], s["router"], *s["gate"], *s["up"], *s["down"], c["top_k"],
                                     renormalize=c["renorm"])
            return {"y": y, "ids": ids, "weights": weights}
        return {"y": q4.moe_experts(s["x"], s["ids"], s["weights"], *s["gate"], *s["up"], *s["down"])}
    if c["op"] == "lora":
        return _plain_lora(s)
    if c["op"] == "moe":
        ids, weights = _plain_route(s)
        return {"y": _plain_experts(s, ids, weights), "ids": ids, "weights": weights}
    return {"y": _plain_experts(s, s["ids"], s["weights"])}


# -- what a pass cannot do without -------------------------------------------
_PER_WEIGHT = {Q4: 34 / 64, Q5: 42 / 64, Q6: 50 / 64, W8: 34 / 32, NVFP4: 9 / 16, BF16: 2.0}


def work(case):
    t, k = case["t"], case["k"]
    if case["op"] == "lora":
        n, r, l = case["n"], case["rank"], case["adapters"]
        used = t * (1 - case["none"])                                    # tokens with an adapter
        hit = l * (1 - (1 - 1 / l) ** used)                              # adapters that some token has
        return {"bytes": n * k * _PER_WEIGHT[case["fmt"]] + hit * r * (n + k) * 2 + 2 * t * (n + k) + 4 * t,
                "flops": 2 * n * k * t + 2 * r * (n + k) * used}
    e, i, top_k = case["experts"], case["inner"], case["top_k"]
    pairs = t * top_k * (1 - case["off"])
    hit = e * (1 - (1 - min(1.0, top_k * (1 - case["off"]) / e)) ** t)  # experts that some token chose
    route = case["op"] == "moe"
    return {"bytes": hit * 3 * i * k * _PER_WEIGHT[Q4] + (2 * e * k if route else 0) + 4 * t * k + 8 * t * top_k,
            "flops": 2 * pairs * 3 * i * k + (2 * t * e * k if route else 0)}


# -- the definition in 64 bits -----------------------------------------------
def _values64(fmt, w, hi, scales):
    """The weight's values, written from the formats' definitions."""
    if fmt == BF16:
        return w.double()
    if fmt == W8:
        v, group = w.to(torch.int64), 32
        v = torch.where(v > 127, v - 256, v).double()
    else:
        b = w.to(torch.int64)
        v = torch.empty(*b.shape[:-1], 2 * b.shape[-1], dtype=torch.int64, device=b.device)
        v[..., 0::2], v[..., 1::2] = b % 16, b // 16
        group = 64
        if fmt in (Q5, Q6):
            width = 1 if fmt == Q5 else 2
            per = 8 // width
            h = hi.to(torch.int64)
            for j in range(per):
                v[..., j::per] += 16 * ((h // (1 << (width * j))) % (1 << width))
        if fmt == NVFP4:
            # E2M1: sign, two exponent bits (bias 1), one mantissa bit
            sign, exp, man = v // 8, (v // 2) % 4, (v % 2).double()
            v = torch.where(exp > 0, (1 + man / 2) * 2.0 ** (exp - 1).double(), man / 2)
            v, group = torch.where(sign > 0, -v, v), 16
        else:
            v = v.double() - {Q4: 8, Q5: 16, Q6: 32}[fmt]
    if fmt == NVFP4:
        # E4M3: four exponent bits (bias 7), three mantissa bits
        b = scales.to(torch.int64)
        exp, man = (b // 8) % 16, (b % 8).double()
        sc = torch.where(exp > 0, (1 + man / 8) * 2.0 ** (exp - 7).double(), man / 8 * 2.0 ** -6)
        sc = torch.where(b >= 128, -sc, sc)
    else:
        sc = scales.double()
    return v * sc.repeat_interleave(group, dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    t, k = case["t"], case["k"]
    x = s["x"].double()
    if case["op"] == "lora":
        y = torch.empty(t, case["n"], dtype=torch.float64, device=x.device)
        rows = max(1, (1 << 27) // k)
        for n0 in range(0, case["n"], rows):
            part = [p[n0:n0 + rows] if p is not None else None for p in (s["w"], s["w_hi"], s["scales"])]
            y[:, n0:n0 + rows] = x @ _values64(case["fmt"], *part).t()
        for a in range(case["adapters"]):
            at = (s["ids"] == a).nonzero().flatten()
            if at.numel():
                u = x[at] @ s["a"][a].double().t()
                y[at] += float(s["lora_scale"][a]) * (u @ s["b"][a].double().t())
        return y
    e, top_k = case["experts"], case["top_k"]
    if case["op"] == "moe":
        logits = x @ s["router"].double().t()
        left = logits.clone()
        ids = torch.empty(t, top_k, dtype=torch.int64, device=x.device)
        for j in range(top_k):  # the largest left, the lowest index among equals
            best = left.max(1, keepdim=True).values
            ids[:, j] = torch.where(left == best, torch.arange(e, device=x.device), e).min(1).values
            left.scatter_(1, ids[:, j:j + 1], -math.inf)
        p = (logits - logits.max(1, keepdim=True).values).exp()
        w = p.gather(1, ids) / (p.gather(1, ids) if case["renorm"] else p).sum(1, keepdim=True)
    else:
        ids, w = s["ids"].long(), s["weights"].double()
    y = torch.zeros(t, k, dtype=torch.float64, device=x.device)
    for a in sorted(set(ids.flatten().tolist())):
        if not 0 <= a < e:
            continue
        tok, slot = (ids == a).nonzero(as_tuple=True)
        wg, wu, wd = (_values64(Q4, s[m][0][a], None, s[m][1][a]) for m in ("gate", "up", "down"))
        gate, up = x[tok] @ wg.t(), x[tok] @ wu.t()
        h = gate / (1 + torch.exp(-gate)) * up
        y.index_add_(0, tok, w[tok, slot][:, None] * (h @ wd.t()))
    if case["op"] == "moe":
        return {"y": y, "ids": None, "weights": w}
    return {"y": y}
