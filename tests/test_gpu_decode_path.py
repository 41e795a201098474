"""The token operators together, as a decoding step of a model with 4-bit experts takes them: norm to
bytes, routing, the experts' products, their combination, a 4-bit head, the adjustment of its logits and the choice
of a token; on its own stream, in a graph, on two streams at once."""
import pytest

from gpu_util import loom_module, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    return require_gpu(), loom_module()


class Model:
    def __init__(self, torch, loom, width=512, experts=16, routes=4, vocab=4000, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.torch, self.loom, self.width, self.experts, self.routes, self.vocab = torch, loom, width, experts, routes, vocab
        words = lambda *s: torch.randint(-2 ** 31, 2 ** 31 - 1, s, generator=g, device="cuda", dtype=torch.int32)   # noqa: E731
        rand = lambda *s: torch.rand(s, generator=g, device="cuda")   # noqa: E731
        self.expert, self.expert_scale = words(experts, width, width // 8), (0.001 + 0.002 * rand(experts, width, width // 64)).to(torch.float16)
        self.head, self.head_scale = words(vocab, width // 8), (0.001 + 0.002 * rand(vocab, width // 128)).to(torch.bfloat16)
        self.router = torch.randint(-128, 128, (experts, width), generator=g, device="cuda", dtype=torch.int8)
        self.router_scale, self.balance = torch.full((experts,), 2e-4, device="cuda"), 0.05 * rand(experts)
        self.gain, self.shift = 1 + 0.1 * rand(width), 0.1 * rand(width)

    def step(self, x, history, lengths, uniform, stream=None):
        loom, t = self.loom, x.shape[0]
        q, sx = loom.loom_layer_norm_i8(x, self.gain, self.shift, stream=stream)
        logits, _ = loom.loom_i8_matmul(self.router, self.router_scale, self.experts, self.width, q, sx, t, stream=stream)
        ids, weights = loom.loom_route_tokens(logits, self.routes, score="sigmoid", bias=self.balance, groups=4, top_groups=2, group_best=2, stream=stream)
        rows = loom.loom_i4_matvec_routed(self.expert, self.expert_scale, self.experts, self.width, self.width, 64, q, sx, ids, stream=stream)
        pairs = self.torch.arange(t * self.routes, dtype=self.torch.int32, device="cuda").view(t, self.routes)
        mixed = loom.loom_routed_combine(pairs, weights, rows, stream=stream)
        q, sx = loom.loom_layer_norm_i8(mixed, stream=stream)
        logits = loom.loom_i4_matvec(self.head, self.head_scale, self.vocab, self.width, 128, q, sx, t, stream=stream)
        adjusted = loom.loom_adjust_logits(logits, history=history, lengths=lengths, repetition=1.3, presence=0.2, stream=stream)
        token, logprob = loom.loom_sample_tokens(adjusted, uniform, temperature=0.8, top_k=40, stream=stream)
        return {"ids": ids, "weights": weights, "rows": rows, "mixed": mixed, "logits": logits, "adjusted": adjusted, "token": token, "logprob": logprob}


def inputs(torch, t, vocab, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(t, 512, generator=g, device="cuda").to(torch.bfloat16), torch.randint(0, vocab, (t, 60), generator=g, device="cuda", dtype=torch.int32),
            torch.randint(0, 61, (t,), generator=g, device="cuda", dtype=torch.int32), torch.rand(t, generator=g, device="cuda"))


@pytest.mark.parametrize("t", [1, 5, 40])
def test_a_step(env, t):
    torch, loom = env
    m = Model(torch, loom)
    x, history, lengths, u = inputs(torch, t, m.vocab, t)
    out = m.step(x, history, lengths, u)
    # the experts' rows and their combination from the step's own inputs, in 64 bits
    q, sx = loom.loom_layer_norm_i8(x, m.gain, m.shift)
    q = q.view(torch.int8).view(t, -1).double()
    shift = 4 * torch.arange(8, device="cuda", dtype=torch.int32)
    w = ((((m.expert[..., None] >> shift) & 15) ^ 8) - 8).view(m.experts, m.width, m.width).double() * m.expert_scale.double().repeat_interleave(64, 2)
    rows = torch.stack([w[e] @ q[p // m.routes] * sx[p // m.routes].double() for p, e in enumerate(out["ids"].view(-1).tolist())])
    size = torch.stack([w[e].abs() @ q[p // m.routes].abs() * sx[p // m.routes].double() for p, e in enumerate(out["ids"].view(-1).tolist())])
    assert bool(((out["rows"].double() - rows).abs() <= 32 * 2.0 ** -24 * size).all())
    mixed = (out["weights"].double()[:, :, None] * out["rows"].double().view(t, m.routes, -1)).sum(1)
    spread = (out["weights"].double()[:, :, None] * out["rows"].double().abs().view(t, m.routes, -1)).sum(1)
    assert bool(((out["mixed"].double() - mixed).abs() <= 8 * 2.0 ** -24 * spread).all())
    # penalties: the seen tokens alone have changed
    seen = torch.zeros(t, m.vocab, dtype=torch.bool, device="cuda")
    for r in range(t):
        seen[r, history[r, :int(lengths[r])].long()] = True
    assert torch.equal(out["adjusted"] != out["logits"], seen)
    assert bool((out["token"] >= 0).all()) and bool((out["token"] < m.vocab).all()) and bool(torch.isfinite(out["logprob"]).all())


def test_in_a_graph_and_on_two_streams(env):
    torch, loom = env
    m = Model(torch, loom, seed=3)
    a, b = inputs(torch, 7, m.vocab, 1), inputs(torch, 33, m.vocab, 2)
    want_a, want_b = m.step(*a), m.step(*b)
    torch.cuda.synchronize()
    graphs, got = [], []
    for given in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(m.step(*given))
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):          # two graphs and two eager calls at once
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        with torch.cuda.stream(torch.cuda.Stream()):
            eager_b = m.step(*b)
        eager_a = m.step(*a)
        torch.cuda.synchronize()
        for one, want in ((got[0], want_a), (got[1], want_b), (eager_a, want_a), (eager_b, want_b)):
            assert all(torch.equal(one[key], want[key]) for key in want)


def test_a_stream_that_is_not_the_current_one(env):
    torch, loom = env
    m = Model(torch, loom, seed=4)
    given = inputs(torch, 9, m.vocab, 5)
    want = m.step(*given)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = m.step(*given, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(got[key], want[key]) for key in want)
