"""loom_adjust_logits on the GPU against its definition, step by step in 64 bits with the f32 rounding that
the definition names after each (a sum, difference, product or quotient of f32 values is rounded to f32 the same
way from 64 bits): results are compared bit for bit."""
import pytest

from gpu_util import loom_module, require_gpu

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def env():
    return require_gpu(), loom_module()


def f32(v):
    return v.float().double()


def definition(torch, logits, history=None, lengths=None, prompts=None, repetition=1.0, frequency=0.0, presence=0.0, bias_ids=None, bias_values=None,
               mask=None, mask_rows=None):
    rows, vocab = logits.shape
    out = logits.clone()
    for r in range(rows):
        at = lambda v: float(v[r]) if isinstance(v, torch.Tensor) else float(torch.tensor(v, dtype=torch.float32))   # noqa: E731
        l, touched = logits[r].double(), torch.zeros(vocab, dtype=torch.bool, device="cuda")
        if history is not None and history.shape[1]:
            n = history.shape[1]
            length = min(max(int(lengths[r]), 0), n) if lengths is not None else n
            prompt = min(max(int(prompts[r]), 0), length) if prompts is not None else 0
            rep = at(repetition)
            rep = rep if rep > 0 else 1.0
            known = lambda h: h[(h >= 0) & (h < vocab)].long()   # noqa: E731
            seen = torch.zeros(vocab, dtype=torch.bool, device="cuda")
            seen[known(history[r, :length])] = True
            count = torch.bincount(known(history[r, prompt:length]), minlength=vocab).double()
            l = torch.where(seen, f32(torch.where(l > 0, l / rep, l * rep)), l)
            l = torch.where(count > 0, f32(f32(l - f32(at(frequency) * count)) - at(presence)), l)
            touched |= seen
        if bias_ids is not None:
            done = set()
            for i, v in zip(bias_ids[r].tolist(), bias_values[r].double().tolist()):
                if 0 <= i < vocab and i not in done:
                    done.add(i)
                    l[i] = f32(l[i] + v)
                    touched[i] = True
        row = torch.where(touched, l.float().to(logits.dtype), logits[r])
        if mask is not None:
            m = int(mask_rows[r]) if mask_rows is not None else (0 if mask.shape[0] == 1 else r)
            if 0 <= m < mask.shape[0]:
                i = torch.arange(vocab, device="cuda")
                row = torch.where((mask[m][i // 32] >> (i % 32)) & 1 == 1, row, torch.full_like(row, -INF))
        out[r] = row
    return out


def same(torch, a, b):
    """Equal bits, any NaN for a NaN."""
    nan = torch.isnan(a) & torch.isnan(b)
    size = torch.int32 if a.dtype == torch.float32 else torch.int16
    return bool(((a.contiguous().view(size) == b.contiguous().view(size)) | nan).all())


def everything(torch, rows, vocab, n, biases, masks, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ints = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device="cuda", dtype=torch.int32)   # noqa: E731
    rand = lambda *s: torch.rand(s, generator=g, device="cuda")   # noqa: E731
    kw = {"history": (vocab * rand(rows, n) ** 3).to(torch.int32) if n else None, "lengths": ints(0, n + 1, rows), "prompts": ints(0, n // 2 + 1, rows),
          "repetition": 1 + 0.5 * rand(rows), "frequency": rand(rows) - 0.3, "presence": 2 * rand(rows) - 0.5}
    if biases:
        kw["bias_ids"], kw["bias_values"] = ints(-1, vocab, rows, biases), 5 * torch.randn(rows, biases, generator=g, device="cuda")
    if masks:
        kw["mask"], kw["mask_rows"] = ints(-2 ** 31, 2 ** 31 - 1, masks, -(-vocab // 32)), ints(-1, masks, rows)
    return kw


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("rows,vocab,n,biases,masks", [(1, 1, 3, 2, 1), (3, 31, 10, 4, 2), (4, 33, 0, 5, 0), (5, 1000, 200, 0, 3), (2, 4097, 5000, 30, 1), (3, 8192, 64, 1024, 5),
                                                       (300, 777, 20, 3, 4), (2, 32768, 300, 16, 1), (1, 131072, 4096, 64, 1), (2, 131071, 1000, 7, 2), (1, 393216, 100, 10, 1),
                                                       (40, 50000, 500, 20, 3), (170, 16385, 100, 5, 2)])
def test_everything_on(env, rows, vocab, n, biases, masks, dtype):
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(vocab + rows)
    logits = (torch.randn(rows, vocab, generator=g, device="cuda") * 3).to(getattr(torch, dtype))
    kw = everything(torch, rows, vocab, n, biases, masks, rows + vocab)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = loom.loom_adjust_logits(logits, error=err, **kw)
    assert same(torch, y, definition(torch, logits, **kw)) and int(err) == 0
    # in place
    copy = logits.clone()
    assert loom.loom_adjust_logits(copy, y=copy, **kw) is copy and same(torch, copy, y)
    # rows with room around them, and rows that start anywhere
    wide = torch.full((rows, vocab + 7), 7.5, dtype=logits.dtype, device="cuda")
    wide[:, 3:3 + vocab] = logits
    out = torch.full((rows, vocab + 4), 9.5, dtype=logits.dtype, device="cuda")
    loom.loom_adjust_logits(wide[:, 3:3 + vocab], y=out[:, 1:1 + vocab], **kw)
    assert same(torch, out[:, 1:1 + vocab], y) and bool((out[:, 0] == 9.5).all()) and bool((out[:, 1 + vocab:] == 9.5).all())
    loom.loom_adjust_logits(wide[:, 3:3 + vocab], y=wide[:, 3:3 + vocab], **kw)
    assert same(torch, wide[:, 3:3 + vocab], y) and bool((wide[:, :3] == 7.5).all()) and bool((wide[:, 3 + vocab:] == 7.5).all())


@pytest.mark.parametrize("part", ["history", "bias", "mask", "none"])
@pytest.mark.parametrize("rows,vocab", [(2, 5000), (200, 2000), (3, 60003)])
def test_parts_alone(env, part, rows, vocab):
    torch, loom = env
    logits = torch.randn(rows, vocab, device="cuda")
    logits[0, 5], logits[0, 6], logits[1, 7] = INF, -INF, float("nan")
    kw = everything(torch, rows, vocab, 50, 9, 2, vocab)
    keys = {"history": ("history", "lengths", "prompts", "repetition", "frequency", "presence"), "bias": ("bias_ids", "bias_values"), "mask": ("mask", "mask_rows"), "none": ()}[part]
    kw = {k: v for k, v in kw.items() if k in keys}
    y = loom.loom_adjust_logits(logits, **kw)
    assert same(torch, y, definition(torch, logits, **kw))
    copy = logits.clone()
    loom.loom_adjust_logits(copy, y=copy, **kw)
    assert same(torch, copy, y)


def test_host_settings_and_whole_histories(env):
    torch, loom = env
    logits = torch.randn(3, 500, device="cuda") * 2
    history = torch.randint(0, 500, (3, 40), device="cuda", dtype=torch.int32)
    for kw in ({"repetition": 1.3}, {"frequency": 0.25}, {"presence": -0.5}, {"repetition": 0.7, "frequency": -0.1, "presence": 1.0}, {}):
        assert same(torch, loom.loom_adjust_logits(logits, history=history, **kw), definition(torch, logits, history=history, **kw))
    # a device repetition that is not above zero counts as one
    rep = torch.tensor([0.0, -2.0, float("nan")], device="cuda")
    assert torch.equal(loom.loom_adjust_logits(logits, history=history, repetition=rep), logits)
    assert loom.loom_adjust_logits(logits[:0], history=history[:0]).shape == (0, 500)
    assert torch.equal(loom.loom_adjust_logits(logits, history=history[:, :0], repetition=2.0), logits)


def test_one_token_many_times_and_every_token_once(env):
    torch, loom = env
    vocab, n = 3000, 100000
    logits = torch.randn(2, vocab, device="cuda")
    history = torch.full((2, n), 2999, dtype=torch.int32, device="cuda")
    history[1] = torch.arange(n, device="cuda", dtype=torch.int32) % vocab
    kw = {"history": history, "repetition": 1.1, "frequency": 0.01, "presence": 0.3, "prompts": torch.tensor([99999, 97000], dtype=torch.int32, device="cuda")}
    assert same(torch, loom.loom_adjust_logits(logits, **kw), definition(torch, logits, **kw))
    kw["prompts"] = None
    assert same(torch, loom.loom_adjust_logits(logits, **kw), definition(torch, logits, **kw))
    longest = torch.zeros(1, (1 << 20) - 1, dtype=torch.int32, device="cuda")        # the longest history, all one token
    y = loom.loom_adjust_logits(logits[:1], history=longest, frequency=0.5)
    assert same(torch, y, definition(torch, logits[:1], history=longest, frequency=0.5))


def test_the_same_bias_twice_and_tokens_out_of_range(env):
    torch, loom = env
    logits = torch.randn(2, 70, device="cuda")
    ids = torch.tensor([[5, 5, -1, 69, 70, 2 ** 31 - 1, 5, 0], [-2 ** 31, 3, 4, 3, 4, 4, 69, 69]], dtype=torch.int32, device="cuda")
    values = torch.randn(2, 8, device="cuda")
    values[0, 3], values[1, 1] = -INF, INF
    history = torch.tensor([[-1, 70, 2 ** 31 - 1, 69], [-2 ** 31, 0, 0, 5]], dtype=torch.int32, device="cuda")
    kw = {"bias_ids": ids, "bias_values": values, "history": history, "repetition": 2.0, "presence": 0.5}
    assert same(torch, loom.loom_adjust_logits(logits, **kw), definition(torch, logits, **kw))
    most = torch.randint(0, 70, (2, 1024), device="cuda", dtype=torch.int32)
    kw = {"bias_ids": most, "bias_values": torch.randn(2, 1024, device="cuda")}
    assert same(torch, loom.loom_adjust_logits(logits, **kw), definition(torch, logits, **kw))


def test_what_is_cut_is_flagged(env):
    torch, loom = env
    logits = torch.randn(3, 100, device="cuda")
    history = torch.randint(0, 100, (3, 10), device="cuda", dtype=torch.int32)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    mask = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    for kw, flagged in (({"lengths": i32(11, 3, 0)}, True), ({"lengths": i32(2, -1, 10)}, True), ({"lengths": i32(10, 0, 5), "prompts": i32(-5, 9, 100)}, False),
                        ({"mask": mask, "mask_rows": i32(2, -1, 0)}, True), ({"mask": mask, "mask_rows": i32(1, -7, 0)}, False)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        kw = {"history": history, "repetition": 1.5, "presence": 0.25, **kw}
        assert same(torch, loom.loom_adjust_logits(logits, error=err, **kw), definition(torch, logits, **kw))
        assert int(err) == (loom.LOOM_DEVERR_COUNT_RANGE if flagged else 0)


def test_masks(env):
    torch, loom = env
    vocab = 4100
    logits = torch.randn(3, vocab, device="cuda")
    logits[:, 17] = float("nan")
    words = -(-vocab // 32)
    one = torch.zeros(1, words, dtype=torch.int32, device="cuda")
    assert bool((loom.loom_adjust_logits(logits, mask=one) == -INF).all())                       # nothing allowed
    assert same(torch, loom.loom_adjust_logits(logits, mask=~one), logits)                        # all allowed
    own = torch.randint(-2 ** 31, 2 ** 31 - 1, (4, words), device="cuda", dtype=torch.int32)       # one a row, one over
    assert same(torch, loom.loom_adjust_logits(logits, mask=own), definition(torch, logits, mask=own))
    token, _ = loom.loom_sample_tokens(loom.loom_adjust_logits(logits, mask=one), torch.rand(3, device="cuda"))
    assert token.tolist() == [-1, -1, -1]


def test_rows_past_31_bits(env):
    torch, loom = env
    vocab, stride = 5000, (1 << 30) + 8
    buf = torch.empty(2 * stride + vocab, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((3, vocab), (stride, 1))
    x.copy_(torch.randn(3, vocab, device="cuda"))
    kw = everything(torch, 3, vocab, 30, 4, 2, 1)
    want = loom.loom_adjust_logits(x.contiguous(), **kw)
    assert same(torch, loom.loom_adjust_logits(x, **kw), want)
    loom.loom_adjust_logits(x, y=x, **kw)
    assert same(torch, x, want)


def test_history_rows_apart(env):
    torch, loom = env
    logits = torch.randn(4, 300, device="cuda")
    buffer = torch.randint(0, 300, (4, 64), device="cuda", dtype=torch.int32)
    view = buffer[:, 5:25]
    assert torch.equal(loom.loom_adjust_logits(logits, history=view, repetition=1.5), loom.loom_adjust_logits(logits, history=view.contiguous(), repetition=1.5))


# many rows: slices of the largest size, with histories on both sides of 4096 tokens (lists of marked tokens, or all marks looked through)
@pytest.mark.parametrize("rows,vocab,n,biases,masks", [(320, 2000, 300, 9, 0), (330, 9000, 9000, 1024, 3), (400, 3001, 12000, 5, 2), (310, 70001, 11000, 20, 2), (305, 40, 10240, 0, 1),
                                                       (306, 64, 0, 1024, 0), (700, 1, 5, 3, 1)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_many_rows(env, rows, vocab, n, biases, masks, dtype):
    torch, loom = env
    g = torch.Generator(device="cuda").manual_seed(vocab + rows)
    logits = (torch.randn(rows, vocab, generator=g, device="cuda") * 3).to(getattr(torch, dtype))
    kw = everything(torch, rows, vocab, n, biases, masks, rows + vocab)
    some = torch.randperm(rows, generator=g, device="cuda")[:12].sort()[0]
    at = lambda r: {k: v[r] if isinstance(v, torch.Tensor) and k != "mask" else v for k, v in kw.items()}   # noqa: E731
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = loom.loom_adjust_logits(logits, error=err, **kw)
    assert same(torch, y[some], definition(torch, logits[some], **at(some))) and int(err) == 0
    # each row by itself is the same row
    for lo in range(0, rows, 64):
        part = torch.arange(lo, min(lo + 64, rows), device="cuda")
        assert same(torch, loom.loom_adjust_logits(logits[part], **at(part)), y[part])
    copy = logits.clone()
    assert loom.loom_adjust_logits(copy, y=copy, **kw) is copy and same(torch, copy, y)
    wide = torch.full((rows, vocab + 7), 7.5, dtype=logits.dtype, device="cuda")
    wide[:, 3:3 + vocab] = logits
    out = torch.full((rows, vocab + 4), 9.5, dtype=logits.dtype, device="cuda")
    loom.loom_adjust_logits(wide[:, 3:3 + vocab], y=out[:, 1:1 + vocab], **kw)
    assert same(torch, out[:, 1:1 + vocab], y) and bool((out[:, 0] == 9.5).all()) and bool((out[:, 1 + vocab:] == 9.5).all())
    loom.loom_adjust_logits(wide[:, 3:3 + vocab], y=wide[:, 3:3 + vocab], **kw)
    assert same(torch, wide[:, 3:3 + vocab], y) and bool((wide[:, :3] == 7.5).all()) and bool((wide[:, 3 + vocab:] == 7.5).all())
    kw["lengths"][rows - 1] = n + 1
    if n:
        loom.loom_adjust_logits(logits, error=err, **kw)
        assert int(err) == loom.LOOM_DEVERR_COUNT_RANGE


def test_kernels_in_a_row(env):
    # inputs written by the kernel before, at once: a kernel is scheduled before the one in front of it has ended
    torch, loom = env
    rows, vocab, n = 400, 20000, 600
    logits = torch.randn(rows, vocab, device="cuda")
    history = torch.zeros(rows, n, dtype=torch.int32, device="cuda")
    lengths = torch.zeros(rows, dtype=torch.int32, device="cuda")
    for turn in range(20):
        g = torch.Generator(device="cuda").manual_seed(turn)
        new = torch.randint(0, vocab, (rows, n), generator=g, device="cuda", dtype=torch.int32)
        torch.cuda.synchronize()
        history.copy_(new)
        lengths.fill_(n - turn)
        logits.copy_(logits.flip(0))
        y = loom.loom_adjust_logits(logits, history=history, lengths=lengths, repetition=1.5, presence=0.25)
        z = loom.loom_adjust_logits(y, history=history, frequency=0.5)
        token, _ = loom.loom_sample_tokens(z, torch.zeros(rows, device="cuda"), temperature=0.0)
        seen = torch.zeros(rows, vocab + 1, dtype=torch.bool, device="cuda").scatter_(1, history[:, :n - turn].long(), True)[:, :vocab]
        count = torch.zeros(rows, vocab, device="cuda").scatter_add_(1, history.long(), torch.ones(rows, n, device="cuda"))
        # (a quotient by way of 64 bits: torch divides f32 by a number as a product with its reciprocal)
        want = torch.where(seen, torch.where(logits > 0, (logits.double() / 1.5).float(), logits * 1.5), logits)
        first = torch.zeros(rows, vocab, device="cuda").scatter_add_(1, history[:, :n - turn].long(), torch.ones(rows, n - turn, device="cuda"))
        want = torch.where(first > 0, want - 0.25, want)
        want = torch.where(count > 0, want - 0.5 * count, want)
        assert torch.equal(z, want) and torch.equal(token.long(), want.argmax(1))
