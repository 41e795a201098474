"""Timing cases of the operators around a model with 4-bit weights and experts: the
matrix-vector product with 4-bit weights and group scales (dense, and of the experts that
each token goes to), the routing to experts and its gradient, and the adjustment of logits
(penalties for repeated tokens, biases, grammar masks) before a token is chosen.

`own` picks what `run` calls: the framework's entry points, or the operators' plain form in
elementary torch operations (32 bits whatever the inputs' type, 64 where a choice lies next
to a border; rounded once at the end).  `exact` gives the definitions' results in 64 bits.

Definitions shared by the plain form, `exact` and the entry points:
  4-bit product  signed nibbles, eight to an int32 word, element j in bits 4j .. 4j + 3;
                 y[t][r] = scale_x[t] * sum_g scale_w[r][g] * (sum over group g of W x) + bias[r]
  experts        the same with the matrix ids[t][j] for the pair (t, j)
  routing        score = softmax or sigmoid of the logits; choice by score + bias: of equal
                 groups the best `top_groups` (by the sum of their `group_best` best), of
                 their experts the top_k, falling, ties to the lower index; weights are the
                 chosen scores, divided by their sum where renormalised, times a factor
  gradient       of those weights to the logits, the choice held fixed
  logits         a seen token's logit is divided (above zero) or multiplied by `repetition`;
                 minus frequency * count, minus presence where count > 0 (count: occurrences
                 behind the prompt); plus its bias; -infinity where the mask's bit is 0
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
LARGEST_WEIGHT = 8192 * 16384           # elements of a dense matrix
LARGEST_EXPERTS = 64 * 2048 * 4096      # elements of all experts' matrices
LARGEST_LOGITS = 256 * 131072


# ---- cases -----------------------------------------------------------------------------
def listed():
    return [
        # one new token against a large weight
        {"name": "matvec_1", "op": "matvec", "tokens": 1, "n": 8192, "k": 16384, "group": 128, "scale": "f16", "y": "f32", "bias": False},
        # sixteen sequences decoding together
        {"name": "matvec_16", "op": "matvec", "tokens": 16, "n": 8192, "k": 16384, "group": 64, "scale": "f16", "y": "bf16", "bias": True},
        # rows that are not whole 16-byte pieces, a last group that is not full, exact scales
        {"name": "matvec_5_ragged", "op": "matvec", "tokens": 5, "n": 5001, "k": 4104, "group": 32, "scale": "f32", "y": "f32", "bias": True},
        # a small projection of one token: latency
        {"name": "matvec_1_small", "op": "matvec", "tokens": 1, "n": 1024, "k": 1024, "group": 128, "scale": "bf16", "y": "bf16", "bias": False},
        # one token through the experts that it goes to
        {"name": "experts_1", "op": "experts", "tokens": 1, "experts": 64, "routes": 8, "n": 2048, "k": 4096, "group": 128, "scale": "f16", "y": "f32"},
        # a decoding batch that reaches nearly all experts
        {"name": "experts_32", "op": "experts", "tokens": 32, "experts": 64, "routes": 8, "n": 2048, "k": 4096, "group": 128, "scale": "f16", "y": "f32"},
        # one token's routing: latency
        {"name": "route_1", "op": "route", "tokens": 1, "experts": 64, "top_k": 8, "score": "softmax", "bias": False, "groups": 1,
         "top_groups": 1, "group_best": 1, "renormalise": True, "x": "f32"},
        # a long batch with a bias for balance and a choice of groups
        {"name": "route_16384", "op": "route", "tokens": 16384, "experts": 256, "top_k": 8, "score": "sigmoid", "bias": True, "groups": 8,
         "top_groups": 4, "group_best": 2, "renormalise": True, "x": "f32"},
        # a training batch's gradient through a softmax over all experts, odd number of experts
        {"name": "route_grad_4097", "op": "route_grad", "tokens": 4097, "experts": 60, "top_k": 4, "score": "softmax", "renormalise": False, "x": "bf16"},
        # a larger one through renormalised sigmoids
        {"name": "route_grad_16384", "op": "route_grad", "tokens": 16384, "experts": 256, "top_k": 8, "score": "sigmoid", "renormalise": True, "x": "f32"},
        # one sequence's logits, everything on
        {"name": "adjust_1", "op": "adjust", "rows": 1, "vocab": 32768, "x": "f32", "history": 2000, "biases": 16, "masks": 1},
        # a serving batch with long histories, a grammar for some rows
        {"name": "adjust_256", "op": "adjust", "rows": 256, "vocab": 131072, "x": "f32", "history": 4096, "biases": 64, "masks": 8},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("matvec", "matvec", "experts", "route", "route_grad", "adjust"))
    if op in ("matvec", "experts"):
        c = {"op": op, "tokens": _log(rng, 1, 48), "n": _log(rng, 256, 16384 if op == "matvec" else 4096),
             "k": 8 * _log(rng, 32, 2048) if rng.random() < 0.4 else 64 * _log(rng, 4, 256),
             "group": rng.choice((32, 64, 128, 128, 256)), "scale": rng.choice(("f32", "f16", "bf16")), "y": rng.choice(("f32", "bf16", "f16"))}
        if op == "matvec":
            c["bias"] = rng.random() < 0.5
            while c["n"] * c["k"] > LARGEST_WEIGHT:
                c["n"] = (c["n"] + 1) // 2
            return c
        c["experts"] = _log(rng, 4, 128)
        c["routes"] = rng.randint(1, min(8, c["experts"]))
        while c["experts"] * c["n"] * c["k"] > LARGEST_EXPERTS:
            c["n"] = (c["n"] + 1) // 2
        return c
    if op in ("route", "route_grad"):
        groups = rng.choice((1, 1, 4, 8)) if op == "route" else 1
        e = groups * _log(rng, 4, 512 // groups)
        top = rng.randint(1, groups)
        c = {"op": op, "tokens": _log(rng, 1, 16384), "experts": e, "top_k": rng.randint(1, min(12, e // groups * top)),
             "score": rng.choice(("softmax", "sigmoid")), "renormalise": rng.random() < 0.6, "x": rng.choice(("f32", "bf16", "f16"))}
        while c["tokens"] * e > 16384 * 256:
            c["tokens"] = (c["tokens"] + 1) // 2
        if op == "route":
            c.update(bias=rng.random() < 0.5, groups=groups, top_groups=top, group_best=rng.choice((1, 2)))
        return c
    c = {"op": op, "rows": _log(rng, 1, 256), "vocab": _log(rng, 1000, 200000), "x": rng.choice(("f32", "bf16", "f16")),
         "history": _log(rng, 1, 8192), "biases": rng.choice((0, 1, 16, 300)), "masks": rng.choice((0, 1, 5))}
    while c["rows"] * c["vocab"] > LARGEST_LOGITS:
        c["rows"] = (c["rows"] + 1) // 2
    return c


def _groups(c):
    return -(-c["k"] // c["group"])


def work(c):
    if c["op"] == "matvec":
        t, n, k = c["tokens"], c["n"], c["k"]
        return {"bytes": n * k // 2 + n * _groups(c) * SIZE[c["scale"]] + t * (k + 4) + (4 * n if c["bias"] else 0) + t * n * SIZE[c["y"]],
                "flops": 2.0 * t * n * k}
    if c["op"] == "experts":
        t, n, k, e, j = c["tokens"], c["n"], c["k"], c["experts"], c["routes"]
        used = e * (1 - (1 - j / e) ** t)       # experts that some token goes to, on average
        return {"bytes": int(used * n * (k / 2 + _groups(c) * SIZE[c["scale"]])) + t * (k + 4) + t * j * (4 + n * SIZE[c["y"]]),
                "flops": 2.0 * t * j * n * k}
    if c["op"] == "route":
        return {"bytes": c["tokens"] * (c["experts"] * SIZE[c["x"]] + 8 * c["top_k"]) + (4 * c["experts"] if c["bias"] else 0),
                "flops": 8.0 * c["tokens"] * c["experts"]}
    if c["op"] == "route_grad":     # renormalised, or by sigmoids, the chosen logits alone are needed
        t, e, s, j = c["tokens"], c["experts"], SIZE[c["x"]], c["top_k"]
        few = c["renormalise"] or c["score"] == "sigmoid"
        return {"bytes": t * (e * s + 8 * j + (j if few else e) * s), "flops": 6.0 * t * (j if few else e)}
    r, v = c["rows"], c["vocab"]
    return {"bytes": 2 * r * v * SIZE[c["x"]] + 2 * r * c["history"] + 8 * r * c["biases"] + min(r, c["masks"]) * v // 8 + 28 * r,
            "flops": 2.0 * r * v}


# ---- inputs ----------------------------------------------------------------------------
def _nibbles(normal, n, k):
    """A matrix of 4-bit weights, packed."""
    v = (normal(n, k // 8, 8) * 2.6).round_().clamp_(-8, 7).to(torch.int32) & 15
    word = v[..., 7].clone()
    for j in range(6, -1, -1):
        word = (word << 4) | v[..., j]
    return word


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1_000_003 * int(seed) + 29)
    normal = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    uniform = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    integers = lambda hi, *s: torch.randint(0, hi, s, generator=g, device="cuda", dtype=torch.int32)  # noqa: E731
    c, s = case, {"case": case, "op": case["op"]}
    if c["op"] in ("matvec", "experts"):
        t, n, k = c["tokens"], c["n"], c["k"]
        lead = (n,) if c["op"] == "matvec" else (c["experts"], n)
        if c["op"] == "matvec":
            s["w"] = _nibbles(normal, n, k)
            s["bias"] = normal(n) if c["bias"] else None
        else:
            s["w"] = torch.stack([_nibbles(normal, n, k) for _ in range(c["experts"])])
            s["ids"] = torch.topk(uniform(t, c["experts"]), c["routes"], dim=1)[1].to(torch.int32)
        s["scale_w"] = (2e-3 + 8e-3 * uniform(*lead, _groups(c))).to(DTYPES[c["scale"]])
        s["x"] = (normal(t, k) * 30).round_().clamp_(-127, 127).to(torch.int8)
        s["scale_x"] = 1e-3 + 9e-3 * uniform(t)
        s["y"] = DTYPES[c["y"]]
        return s
    if c["op"] in ("route", "route_grad"):
        t, e = c["tokens"], c["experts"]
        s["logits"] = (normal(t, e) * 1.5 + 0.3 * normal(1, e)).to(DTYPES[c["x"]])
        if c["op"] == "route":
            s["bias"] = 0.05 * normal(e) if c["bias"] else None
        else:
            s["ids"] = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True)[1][:, :c["top_k"]].to(torch.int32).contiguous()
            s["dweights"] = normal(t, c["top_k"])
        s["factor"] = 2.5 if c["score"] == "sigmoid" else 1.0
        return s
    r, v, h, b = c["rows"], c["vocab"], c["history"], c["biases"]
    s["logits"] = (normal(r, v) * 2.5).to(DTYPES[c["x"]])
    # text repeats itself: few tokens often, many once
    s["history"] = (v * uniform(r, h) ** 4).to(torch.int32).clamp_(0, v - 1)
    s["lengths"] = integers(h + 1, r)
    s["prompts"] = (s["lengths"] * uniform(r)).to(torch.int32)
    s["history"].masked_fill_(torch.arange(h, device="cuda")[None, :] >= s["lengths"][:, None], -1)
    pick = lambda values: torch.tensor(values, device="cuda")[integers(len(values), r).long()]  # noqa: E731
    s["repetition"], s["frequency"], s["presence"] = pick([1.0, 1.0, 1.1, 1.3]), pick([0.0, 0.0, 0.2, 0.7]), pick([0.0, 0.5, 1.5])
    s["bias_ids"] = s["bias_values"] = s["mask"] = s["mask_rows"] = None
    if b:       # lists shorter than the longest end in -1; no token twice in a list
        ids = torch.argsort(uniform(r, min(v, 4 * b + 8)), dim=1)[:, :b] * (v // min(v, 4 * b + 8))
        s["bias_ids"] = torch.where(torch.arange(b, device="cuda")[None, :] < integers(b + 1, r)[:, None], ids, -1).to(torch.int32)
        s["bias_values"] = 4 * normal(r, b)
    if c["masks"]:      # a grammar allows few tokens, or most; rows without one have -1
        words = -(-v // 32)
        share = torch.where(uniform(c["masks"], 1, 1) < 0.5, 0.02, 0.9)
        bits = (uniform(c["masks"], words, 32) < share).to(torch.int64) << torch.arange(32, device="cuda")
        s["mask"] = bits.sum(2).to(torch.int32)      # (the low 32 bits)
        s["mask_rows"] = torch.where(uniform(r) < 0.5, integers(c["masks"], r), -1).to(torch.int32)
    return s


# ---- the operators -----------------------------------------------------------------------
def _dequantised(w, scale, group, k):
    """The f32 matrix of packed words [n][k / 8] and scales [n][groups]."""
    n = w.shape[0]
    shift = 4 * torch.arange(8, device=w.device, dtype=torch.int32)
    v = ((((w[..., None] >> shift) & 15) ^ 8) - 8).reshape(n, k).float()
    return v * scale.float().repeat_interleave(group, 1)[:, :k]


def _plain_product(w, scale_w, s, rows=slice(None)):
    m = _dequantised(w, scale_w, s["case"]["group"], s["case"]["k"])
    return torch.matmul(s["x"][rows].float(), m.t()) * s["scale_x"][rows, None]


def _scores(l, case):
    if case["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _choice(choose, case):
    """The chosen experts of `choose` (scores + bias, 64 bits), falling, ties to the lower index."""
    t, e = choose.shape
    if case["groups"] > 1:
        grouped = choose.view(t, case["groups"], e // case["groups"])
        best = torch.sort(grouped, dim=2, descending=True)[0][:, :, :case["group_best"]].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True)[1][:, :case["top_groups"]]
        out = torch.ones_like(best, dtype=torch.bool).scatter_(1, kept, False)
        choose = grouped.masked_fill(out[:, :, None], -math.inf).view(t, e)
    return torch.sort(choose, dim=1, descending=True, stable=True)[1][:, :case["top_k"]]


def _plain_route(s):
    case = s["case"]
    choose = _scores(s["logits"].double(), case)
    if s["bias"] is not None:
        choose = choose + s["bias"].double()
    ids = _choice(choose, case)
    w = _scores(s["logits"].float(), case).gather(1, ids)
    if case["renormalise"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": w * s["factor"]}


def _plain_route_grad(s):
    case, ids = s["case"], s["ids"].long()
    score = _scores(s["logits"].float(), case)
    g = s["dweights"] * s["factor"]
    if case["renormalise"]:
        w = score.gather(1, ids)
        total = w.sum(1, keepdim=True)
        g = (g - (g * w).sum(1, keepdim=True) / total) / total
    full = torch.zeros_like(score).scatter_add_(1, ids, g)
    if case["score"] == "sigmoid":
        d = full * score * (1 - score)
    else:
        d = score * (full - (full * score).sum(1, keepdim=True))
    return d.to(s["logits"].dtype)


def _marks(s):
    """(seen, count, bias, allowed) of every token of every row."""
    r, v = s["logits"].shape
    at = torch.arange(s["history"].shape[1], device="cuda")[None, :]
    token = torch.where((at < s["lengths"][:, None]) & (s["history"] >= 0), s["history"].long(), v)
    seen = torch.zeros(r, v + 1, dtype=torch.bool, device="cuda").scatter_(1, token, True)[:, :v]
    count = torch.zeros(r, v + 1, device="cuda").scatter_add_(1, token, (at >= s["prompts"][:, None]).float())[:, :v]
    bias = allowed = None
    if s["bias_ids"] is not None:
        ids = torch.where(s["bias_ids"] >= 0, s["bias_ids"].long(), v)
        bias = torch.zeros(r, v + 1, device="cuda").scatter_(1, ids, s["bias_values"])[:, :v]
    if s["mask"] is not None:
        bits = (s["mask"][:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        bits = bits.bool().view(s["mask"].shape[0], -1)[:, :v]
        allowed = bits[s["mask_rows"].clamp(min=0).long()] | (s["mask_rows"] < 0)[:, None]
    return seen, count, bias, allowed


def _plain_adjust(s):
    seen, count, bias, allowed = _marks(s)
    l = s["logits"].float()
    rep = s["repetition"][:, None]
    l = torch.where(seen, torch.where(l > 0, l / rep, l * rep), l)
    l = l - s["frequency"][:, None] * count
    l = torch.where(count > 0, l - s["presence"][:, None], l)
    if bias is not None:
        l = l + bias
    if allowed is not None:
        l = l.masked_fill(~allowed, -math.inf)
    return l.to(s["logits"].dtype)


def _plain(s):
    if s["op"] == "matvec":
        y = _plain_product(s["w"], s["scale_w"], s)
        return (y if s["bias"] is None else y + s["bias"]).to(s["y"])
    if s["op"] == "experts":
        t, n, routes = s["x"].shape[0], s["w"].shape[1], s["ids"].shape[1]
        if t * routes <= s["w"].shape[0]:      # few pairs: the matrices that they want
            flat = s["ids"].view(-1)
            pick = lambda t, i: t.index_select(0, flat[i:i + 1])[0]  # noqa: E731
            of = [_plain_product(pick(s["w"], i), pick(s["scale_w"], i), s, slice(i // routes, i // routes + 1)) for i in range(t * routes)]
            return torch.cat(of).to(s["y"])
        y = torch.zeros(t, routes, n, device="cuda")
        for e in range(s["w"].shape[0]):
            of_e = _plain_product(s["w"][e], s["scale_w"][e], s)
            y = torch.where((s["ids"] == e)[:, :, None], of_e[:, None, :], y)
        return y.view(-1, n).to(s["y"])
    if s["op"] == "route":
        return _plain_route(s)
    if s["op"] == "route_grad":
        return _plain_route_grad(s)
    return _plain_adjust(s)


def _own(s):
    import int8_dequant_dot_gb300 as loom
    c = s["case"]
    if s["op"] == "matvec":
        return loom.loom_i4_matvec(s["w"], s["scale_w"], c["n"], c["k"], c["group"], s["x"], s["scale_x"], c["tokens"], bias=s["bias"],
                                   y_dtype=s["y"])
    if s["op"] == "experts":
        return loom.loom_i4_matvec_routed(s["w"], s["scale_w"], c["experts"], c["n"], c["k"], c["group"], s["x"], s["scale_x"], s["ids"],
                                          y_dtype=s["y"])
    if s["op"] == "route":
        ids, weights = loom.loom_route_tokens(s["logits"], c["top_k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                                              top_groups=c["top_groups"], group_best=c["group_best"], renormalise=c["renormalise"],
                                              factor=s["factor"])
        return {"ids": ids, "weights": weights}
    if s["op"] == "route_grad":
        return loom.loom_route_tokens_backward(s["dweights"], s["logits"], s["ids"], score=c["score"], renormalise=c["renormalise"],
                                               factor=s["factor"])
    return loom.loom_adjust_logits(s["logits"], history=s["history"], lengths=s["lengths"], prompts=s["prompts"], repetition=s["repetition"],
                                   frequency=s["frequency"], presence=s["presence"], bias_ids=s["bias_ids"], bias_values=s["bias_values"],
                                   mask=s["mask"], mask_rows=s["mask_rows"])


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definitions in 64 bits ------------------------------------------------------------
def _exact_product(w, scale, group, x):
    n, k = w.shape[0], x.shape[1]
    v = torch.empty(n, k, dtype=torch.float64, device=w.device)
    for j in range(8):      # the sign by an arithmetic shift
        v[:, j::8] = ((w << (28 - 4 * j)) >> 28).double()
    y = torch.zeros(x.shape[0], n, dtype=torch.float64, device=w.device)
    for g in range(scale.shape[1]):
        part = slice(g * group, (g + 1) * group)
        y += (x[:, part].double() @ v[:, part].t()) * scale[:, g].double()
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "matvec":
        y = _exact_product(s["w"], s["scale_w"], case["group"], s["x"]) * s["scale_x"].double()[:, None]
        return y if s["bias"] is None else y + s["bias"].double()
    if s["op"] == "experts":
        ids, n = s["ids"].view(-1).long(), s["w"].shape[1]
        y = torch.empty(ids.numel(), n, dtype=torch.float64, device="cuda")
        for e in torch.unique(ids).tolist():
            pairs = (ids == e).nonzero()[:, 0]
            rows = pairs // case["routes"]
            y[pairs] = _exact_product(s["w"][e], s["scale_w"][e], case["group"], s["x"][rows]) * s["scale_x"][rows].double()[:, None]
        return y
    if s["op"] == "route":
        l = s["logits"].double()
        score = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
        ids = _choice(score if s["bias"] is None else score + s["bias"].double(), case)
        w = score.gather(1, ids)
        return {"ids": None, "weights": s["factor"] * (w / w.sum(1, keepdim=True) if case["renormalise"] else w)}
    if s["op"] == "route_grad":     # the chain rule, one chosen weight at a time
        l, ids = s["logits"].double(), s["ids"].long()
        score = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
        chosen, g = score.gather(1, ids), s["dweights"].double() * s["factor"]
        total = chosen.sum(1, keepdim=True)
        out = torch.zeros_like(l)
        for j in range(ids.shape[1]):
            ds = g[:, j:j + 1]          # gradient of the j-th chosen score
            if case["renormalise"]:
                ds = ds / total - (g * chosen).sum(1, keepdim=True) / total ** 2
            own_part = chosen[:, j:j + 1] * (1 - chosen[:, j:j + 1]) * ds if case["score"] == "sigmoid" else chosen[:, j:j + 1] * ds
            out.scatter_add_(1, ids[:, j:j + 1], own_part)
            if case["score"] == "softmax" and not case["renormalise"]:
                out -= chosen[:, j:j + 1] * ds * score
        return out      # (renormalised, the softmax's common part drops out: its terms add up to zero)
    seen, count, bias, allowed = _marks(s)
    l, rep = s["logits"].double(), s["repetition"].double()[:, None]
    l = torch.where(seen, l * torch.where(l > 0, 1 / rep, rep), l)
    l = l - s["frequency"].double()[:, None] * count.double() - s["presence"].double()[:, None] * (count > 0)
    if bias is not None:
        l = l + bias.double()
    return l if allowed is None else torch.where(allowed, l, torch.full_like(l, -math.inf))
