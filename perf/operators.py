"""The token operators' timing cases: the 8-bit matrix product with scales for each
token and channel (alone, and behind the quantisation of its tokens), layer norm's
forward and backward pass, layer norm handing 8-bit tokens to the product, and
sampling from logits.

`own` picks what `run` calls: the framework's entry points, or the operators' plain
form in elementary torch operations (32 bits whatever the inputs' type, rounded once
at the end).  `exact` gives the results of the definitions in 64 bits.

Definitions shared by the plain form, `exact` and the entry points:
  quantisation  scale = amax / 127, q = rint(x * (127 / amax)), each step one f32
                rounding (a token of zeros: scale 0, q 0)
  product       y[t][n] = acc * (scale_w[n] * scale_x[t]) + bias[n], acc = sum_k x w
  layer norm    y = (x - mean) * rstd * gain + bias, rstd = 1 / sqrt(var + eps)
  sampling      w_i = floor(exp((l_i - max l) / T) * 2^31); of the tokens in order of
                falling logit (ties: lower index first) the first top_k; of those the
                ones whose predecessors' weights sum to less than top_p times their
                total; of those the ones with w >= min_p * 2^31; the token is the first
                index whose running weight (index order) exceeds floor(u * total), its
                log probability log(w / total).  T = 0: the largest logit.
"""
import math

import torch

own = False

EPS = 1e-5
FULL = 1 << 31          # the weight of the largest logit
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
SMALL = 10 ** 30        # "no limit" for top_k


# ---- cases -----------------------------------------------------------------------------
def listed():
    return [
        # one new token against a large weight: the latency of a decoding step
        {"name": "matmul_1", "op": "matmul", "tokens": 1, "n": 8192, "k": 16384, "x": "i8", "y": "f32", "bias": False},
        # sixteen sequences decoding together
        {"name": "matmul_16", "op": "matmul", "tokens": 16, "n": 8192, "k": 16384, "x": "i8", "y": "bf16", "bias": True},
        # a ragged batch of short prompts, from float activations; rows that are not whole 16-byte pieces
        {"name": "linear_203", "op": "matmul", "tokens": 203, "n": 5001, "k": 4108, "x": "f32", "y": "f32", "bias": True},
        # a long prompt through a large projection
        {"name": "linear_4096", "op": "matmul", "tokens": 4096, "n": 16384, "k": 8192, "x": "bf16", "y": "bf16", "bias": False},
        # the output head for one token: norm, 8-bit token, product
        {"name": "head_1", "op": "head", "tokens": 1, "n": 32768, "k": 2048, "x": "f32", "y": "f16", "bias": False},
        # the output head for a batch of decoding sequences
        {"name": "head_96", "op": "head", "tokens": 96, "n": 65536, "k": 4096, "x": "bf16", "y": "bf16", "bias": False},
        # a few tokens through one norm: launch latency
        {"name": "norm_8x2048", "op": "norm", "rows": 8, "width": 2048, "x": "f32"},
        # a training batch's activations
        {"name": "norm_16384x8192", "op": "norm", "rows": 16384, "width": 8192, "x": "bf16"},
        # an odd width, where rows start at any 4-byte boundary
        {"name": "norm_grad_1001x5001", "op": "norm_grad", "rows": 1001, "width": 5001, "x": "f32"},
        # a training batch's gradients
        {"name": "norm_grad_16384x4096", "op": "norm_grad", "rows": 16384, "width": 4096, "x": "bf16"},
        # one sequence's next token, every filter on
        {"name": "sample_1", "op": "sample", "rows": 1, "vocab": 32768, "x": "f32", "filters": "all"},
        # a serving batch, each row with settings of its own
        {"name": "sample_256", "op": "sample", "rows": 256, "vocab": 131072, "x": "f32", "filters": "mixed"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("matmul", "matmul", "head", "norm", "norm_grad", "sample"))
    if op in ("matmul", "head"):
        t, n = _log(rng, 1, 4096), _log(rng, 256, 16384)
        k = 4 * _log(rng, 64, 4096) if rng.random() < 0.4 else 16 * _log(rng, 16, 1024)
        while t * n * k > 4096 * 16384 * 8192:
            t = max(1, t // 2)
        x = rng.choice(("i8", "f32", "bf16", "f16")) if op == "matmul" else rng.choice(("f32", "bf16", "f16"))
        y = rng.choice(("f32", "bf16", "f16")) if op == "matmul" else rng.choice(("bf16", "f16"))
        return {"op": op, "tokens": t, "n": n, "k": k, "x": x, "y": y, "bias": rng.random() < 0.5}
    if op in ("norm", "norm_grad"):
        r, w = _log(rng, 1, 16384), _log(rng, 64, 16384)
        while r * w > 16384 * (8192 if op == "norm" else 4096) // 2:
            r = max(1, r // 2)
        return {"op": op, "rows": r, "width": w, "x": rng.choice(("f32", "bf16", "f16"))}
    return {"op": op, "rows": _log(rng, 1, 256), "vocab": _log(rng, 1000, 131072), "x": rng.choice(("f32", "bf16", "f16")),
            "filters": rng.choice(("none", "all", "mixed"))}


def work(c):
    if c["op"] in ("matmul", "head"):
        t, n, k = c["tokens"], c["n"], c["k"]
        xb = t * k * SIZE[c["x"]] if c["x"] != "i8" else t * k + 4 * t
        return {"bytes": xb + n * k + 4 * n * (2 if c["bias"] else 1) + t * n * SIZE[c["y"]] + (8 * k if c["op"] == "head" else 0),
                "flops": 2.0 * t * n * k}
    if c["op"] == "norm":
        return {"bytes": 2 * c["rows"] * c["width"] * SIZE[c["x"]] + 8 * c["width"] + 8 * c["rows"], "flops": 7.0 * c["rows"] * c["width"]}
    if c["op"] == "norm_grad":
        return {"bytes": 3 * c["rows"] * c["width"] * SIZE[c["x"]] + 12 * c["width"] + 8 * c["rows"], "flops": 13.0 * c["rows"] * c["width"]}
    return {"bytes": c["rows"] * c["vocab"] * SIZE[c["x"]] + 32 * c["rows"], "flops": 6.0 * c["rows"] * c["vocab"]}


# ---- inputs ----------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1_000_003 * int(seed) + 17)
    normal = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    uniform = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    s = {"case": case, "op": case["op"]}
    if case["op"] in ("matmul", "head"):
        t, n, k = case["tokens"], case["n"], case["k"]
        s["w"] = (normal(n, k) * 36).round_().clamp_(-127, 127).to(torch.int8)
        s["scale_w"] = 1e-3 + 9e-3 * uniform(n)
        s["bias"] = normal(n) if case["bias"] else None
        s["y"] = DTYPES[case["y"]]
        if case["x"] == "i8":
            s["x"] = (normal(t, k) * 30).round_().clamp_(-127, 127).to(torch.int8)
            s["scale_x"] = 1e-3 + 9e-3 * uniform(t)
        else:   # tokens of different sizes
            s["x"] = (normal(t, k) * (0.2 + 2 * uniform(t, 1))).to(DTYPES[case["x"]])
        if case["op"] == "head":
            s["gain"], s["shift"] = 1 + 0.2 * normal(k), 0.1 * normal(k)
        return s
    if case["op"] in ("norm", "norm_grad"):
        r, w = case["rows"], case["width"]
        s["x"] = (normal(r, w) * (0.5 + uniform(r, 1)) + 0.3 * normal(r, 1)).to(DTYPES[case["x"]])
        s["gain"], s["shift"] = 1 + 0.2 * normal(w), 0.1 * normal(w)
        if case["op"] == "norm_grad":
            s["dy"] = (normal(r, w) * 0.1).to(DTYPES[case["x"]])
            x = s["x"].double()   # what the forward pass left behind
            mean = x.mean(1)
            s["mean"], s["rstd"] = mean.float(), (1 / torch.sqrt((x - mean[:, None]).square().mean(1) + EPS)).float()
        return s
    r, v = case["rows"], case["vocab"]
    s["logits"] = (normal(r, v) * 2.5).to(DTYPES[case["x"]])
    s["logits"].masked_fill_(uniform(1, v) < 0.01, float("-inf"))   # tokens that may not be chosen
    s["uniform"] = uniform(r)
    if case["filters"] == "none":
        s["temperature"], s["top_k"], s["top_p"], s["min_p"] = 1.0, 0, 1.0, 0.0
    elif case["filters"] == "all":
        s["temperature"], s["top_k"], s["top_p"], s["min_p"] = 0.8, 50, 0.95, 0.02
    else:       # settings of each row's own, off in some
        pick = lambda values, dtype: torch.tensor(values, dtype=dtype, device="cuda")[  # noqa: E731
            torch.randint(0, len(values), (r,), generator=g, device="cuda")]
        s["temperature"] = pick([0.0, 0.6, 0.8, 1.0, 1.0, 1.3], torch.float32)
        s["top_k"] = pick([0, 0, 1, 20, 50, 1000], torch.int32)
        s["top_p"] = pick([1.0, 1.0, 0.95, 0.9, 0.5], torch.float32)
        s["min_p"] = pick([0.0, 0.0, 0.0, 0.05, 0.2], torch.float32)
    return s


# ---- the operators -----------------------------------------------------------------------
def _plain_quantize(x):
    amax = x.abs().amax(1)
    full = torch.full_like(amax, 127.0)
    inv = torch.where(amax > 0, torch.div(full, amax), torch.zeros_like(amax))
    return torch.round(x * inv[:, None]), torch.div(amax, full)


def _plain_norm(x, gain, shift):
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = 1.0 / torch.sqrt(xc.square().mean(1) + EPS)
    return xc * rstd[:, None] * gain + shift, mean, rstd


def _plain_product(x, scale_x, s):
    y = torch.matmul(x, s["w"].float().t()) * (s["scale_w"][None, :] * scale_x[:, None])
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["y"])


def _rows(v, like, dtype):
    return v if isinstance(v, torch.Tensor) else torch.full((like.shape[0],), v, dtype=dtype, device=like.device)


def _choose(weight, order, s):
    """The token of each row and its log probability, from the weights in index order (int64)."""
    u = s["uniform"].double()
    top_k, top_p = _rows(s["top_k"], u, torch.int64).long(), _rows(s["top_p"], u, torch.float32).double()
    min_p = _rows(s["min_p"], u, torch.float32).double()
    v = weight.shape[1]
    ranked = weight.gather(1, order)
    rank = torch.arange(v, device=weight.device)[None, :]
    keep = rank < torch.where(top_k > 0, top_k, torch.full_like(top_k, v))[:, None]
    ranked = torch.where(keep, ranked, torch.zeros_like(ranked))
    before = torch.cumsum(ranked, 1) - ranked
    mass = ranked.sum(1)
    keep &= (before.double() < torch.where(top_p < 1, top_p * mass.double(), torch.full_like(u, math.inf))[:, None]) | (rank == 0)
    keep &= ranked.double() >= (min_p * FULL)[:, None]
    kept = torch.zeros_like(weight).scatter_(1, order, torch.where(keep, ranked, torch.zeros_like(ranked)))
    total = kept.sum(1)
    at = torch.minimum(torch.floor(u * total.double()).long(), total - 1)
    running = torch.cumsum(kept, 1)
    token = (running <= at[:, None]).sum(1)
    chosen = kept.gather(1, token[:, None])[:, 0]
    return token.to(torch.int32), torch.log(chosen.double() / total.double())


def _plain_sample(s):
    l = s["logits"].float()
    t = _rows(s["temperature"], l, torch.float32)
    m = l.amax(1)
    greedy = t == 0
    one = torch.ones_like(t)
    inv = torch.div(one, torch.where(greedy, one, t))
    weight = (torch.exp((l - m[:, None]) * inv[:, None]) * float(FULL)).to(torch.int64)
    order = torch.sort(l, dim=1, descending=True, stable=True)[1]
    first = torch.zeros_like(weight).scatter_(1, order[:, :1], FULL)
    weight = torch.where(greedy[:, None], first, weight)
    token, logprob = _choose(weight, order, s)
    return {"token": token, "logprob": logprob.float()}


def _plain(s):
    if s["op"] == "matmul":
        if s["case"]["x"] == "i8":
            return _plain_product(s["x"].float(), s["scale_x"], s)
        return _plain_product(*_plain_quantize(s["x"].float()), s)
    if s["op"] == "head":
        return _plain_product(*_plain_quantize(_plain_norm(s["x"].float(), s["gain"], s["shift"])[0]), s)
    if s["op"] == "norm":
        y, mean, rstd = _plain_norm(s["x"].float(), s["gain"], s["shift"])
        return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}
    if s["op"] == "norm_grad":
        x, dy = s["x"].float(), s["dy"].float()
        xhat = (x - s["mean"][:, None]) * s["rstd"][:, None]
        g = dy * s["gain"]
        dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
        return {"dx": dx.to(s["x"].dtype), "dgain": (dy * xhat).sum(0), "dbias": dy.sum(0)}
    return _plain_sample(s)


def _own(s):
    import int8_dequant_dot_gb300 as loom
    if s["op"] in ("matmul", "head"):
        t, k = s["x"].shape
        n = s["w"].shape[0]
        if s["op"] == "head":
            q, scale = loom.loom_layer_norm_i8(s["x"], s["gain"], s["shift"], EPS)
        elif s["case"]["x"] == "i8":
            q, scale = s["x"], s["scale_x"]
        else:
            q, scale = loom.loom_quantize_tokens(s["x"])
        return loom.loom_i8_matmul(s["w"], s["scale_w"], n, k, q, scale, t, bias=s["bias"], y_dtype=s["y"])[0]
    if s["op"] == "norm":
        y, mean, rstd = loom.loom_layer_norm(s["x"], s["gain"], s["shift"], EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if s["op"] == "norm_grad":
        dx, dgain, dbias = loom.loom_layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["gain"])
        return {"dx": dx, "dgain": dgain, "dbias": dbias}
    token, logprob = loom.loom_sample_tokens(s["logits"], s["uniform"], temperature=s["temperature"], top_k=s["top_k"],
                                             top_p=s["top_p"], min_p=s["min_p"])
    return {"token": token, "logprob": logprob}


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definitions in 64 bits ------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] in ("matmul", "head"):
        x = s["x"].double()
        if s["op"] == "head":
            mean = x.mean(1, keepdim=True)
            var = (x - mean).square().mean(1, keepdim=True)
            x = (x - mean) / torch.sqrt(var + EPS) * s["gain"].double() + s["shift"].double()
        if case["x"] == "i8":
            scale = s["scale_x"].double()
        else:
            amax = x.abs().amax(1)
            scale = amax / 127
            # (x * 127 / amax) lies next to a tie only where the definition's own f32 steps say which side:
            # the matrix case takes those steps, the norm's output is not an f32 value to begin with
            inv = torch.where(amax > 0, 127 / amax, torch.zeros_like(amax))
            if s["op"] == "matmul":
                x = (x * inv.float().double()[:, None]).float().double()
            else:
                x = x * inv[:, None]
            x = torch.round(x)
        y = torch.matmul(x, s["w"].double().t()) * scale[:, None] * s["scale_w"].double()
        return y if s["bias"] is None else y + s["bias"].double()
    if s["op"] == "norm":
        x = s["x"].double()
        mean = x.mean(1)
        rstd = (x.var(1, unbiased=False) + EPS).rsqrt()
        return {"y": (x - mean[:, None]) * rstd[:, None] * s["gain"].double() + s["shift"].double(), "mean": mean, "rstd": rstd}
    if s["op"] == "norm_grad":
        x, dy, rstd = s["x"].double(), s["dy"].double(), s["rstd"].double()[:, None]
        xhat = (x - s["mean"].double()[:, None]) * rstd
        g = dy * s["gain"].double()
        w = x.shape[1]
        dx = rstd / w * (w * g - g.sum(1, keepdim=True) - xhat * (g * xhat).sum(1, keepdim=True))
        return {"dx": dx, "dgain": torch.einsum("rw,rw->w", dy, xhat), "dbias": dy.sum(0)}
    l = s["logits"].double()
    t = _rows(s["temperature"], l, torch.float32).double()
    cold = (t == 0)[:, None]
    e = torch.exp((l - l.amax(1, keepdim=True)) / torch.where(cold, torch.ones_like(t)[:, None], t[:, None]))
    order = torch.sort(-l, dim=1, stable=True)[1]
    e = torch.where(cold, torch.zeros_like(e).scatter_(1, order[:, :1], 1.0), e)
    return {"token": None, "logprob": _choose(torch.floor(e * FULL).long(), order, s)[1]}
