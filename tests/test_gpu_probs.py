"""dsa_logits_probs against its definition in 64 bits, and the whole verify step."""
import math

import pytest
import torch

from verify_step import DQK, DV, Batch, attention, attention_bounds, probabilities, rope, frequencies

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dsa():
    import sparse_long_context_score_b200 as m
    from sparse_long_context_score_b200 import build
    build.build()
    m.lib()
    return m


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _inputs(B, S, V, seed=0, dtype=torch.float32, hist=0, bias=0, mask=False, greedy=(), spread=False):
    g = _gen(seed)
    u = lambda lo, hi: lo + (hi - lo) * torch.rand(B, generator=g, device="cuda")  # noqa: E731
    a = dict(logits=(torch.randn((B, S, V), generator=g, device="cuda") * 3).to(dtype), temperature=u(0.4, 1.5))
    for b in greedy:
        a["temperature"][b] = 0.0
    ids = V if spread else 300  # (a history's tokens: many times the same, or anywhere)
    if hist:
        a["history"] = torch.randint(-2, min(V + 2, ids), (B, hist), generator=g, device="cuda", dtype=torch.int32)
        a["history_len"] = torch.randint(0, hist + 5, (B,), generator=g, device="cuda", dtype=torch.int32)
        a["prompt_len"] = torch.randint(0, hist, (B,), generator=g, device="cuda", dtype=torch.int32)
        a["draft"] = torch.randint(-1, min(V + 1, ids), (B, S), generator=g, device="cuda", dtype=torch.int32)
        a["repetition"], a["frequency"], a["presence"] = u(0.8, 1.4), u(-0.3, 0.6), u(-0.3, 0.6)
    if bias:
        a["bias_ids"] = torch.randint(-1, V + 1 if spread else min(V + 1, 2 * bias), (B, bias), generator=g, device="cuda", dtype=torch.int32)
        a["bias_values"] = torch.randn((B, bias), generator=g, device="cuda") * 3
    if mask:
        a["mask"] = torch.randint(-(1 << 31), 1 << 31, (B, S, (V + 31) // 32), generator=g, device="cuda").to(torch.int32)
    return a


def _check(dsa, a):
    got = dsa.dsa_logits_probs(**a).cpu().double()
    p, size = probabilities(**a)
    B, S, V = p.shape
    T = torch.ones(B) if a.get("temperature") is None else a["temperature"].cpu()
    T = torch.where(T > 0, T, 1.0).double()[:, None, None].expand(B, S, 1)
    nb = 0 if a.get("bias_ids") is None else a["bias_ids"].shape[1]
    # a logit takes at most 8 roundings and its biases' on the way to the exponent, each half a
    # step of the largest value passed; the exponential is good to 2^-22, the sum of V terms to
    # 1024 half steps (its additions are at most that deep)
    dz = (8 + nb) * 2.0 ** -24 * size[..., None] / T
    exponent = -torch.where(p > 0, p, 1.0).log()
    bound = p * (2 * dz + 4 * 2.0 ** -24 * exponent.abs() + 2.0 ** -21 + 1024 * 2.0 ** -24) + 1e-37
    err = (got - p).abs()
    assert bool((err <= bound).all()), f"{float((err - bound).max())} over the bound"
    greedy = (a["temperature"].cpu() <= 0) if a.get("temperature") is not None else torch.zeros(B, dtype=torch.bool)
    assert torch.equal(got[greedy], p[greedy])
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,S,V,kw", [
    (1, 1, 1, {}), (1, 1, 2, dict(mask=True)), (2, 3, 31, dict(hist=9, bias=3, mask=True)), (3, 1, 33, dict(greedy=(1,))),
    (2, 2, 1000, dict(hist=200, bias=20, mask=True, greedy=(0,))), (1, 4, 4097, dict(hist=50)),
    (5, 1, 20480, dict(bias=5)), (2, 1, 32003, dict(mask=True)), (1, 7, 50257, dict(hist=3000, bias=100, mask=True)),
    (2, 2, 151552, dict(hist=1000, bias=8, mask=True, greedy=(1,))), (1, 2, 163841, dict(hist=100)),
    (1, 1, 262144, dict(mask=True, hist=10)), (1, 1, 327681, {}), (1, 1, 700001, dict(hist=64, bias=4, mask=True)),
    # many rows: two passes over chunks
    (300, 1, 1, {}), (70, 5, 31, dict(hist=20, bias=5, mask=True, greedy=(3, 69))), (320, 1, 64, dict(hist=1)),
    (100, 3, 1000, dict(hist=700, spread=True)), (40, 4, 5003, dict(hist=300, bias=40, mask=True, greedy=(0, 7))),
    (16, 7, 20480, dict(hist=6000, bias=32, mask=True, spread=True, greedy=(5,))), (50, 4, 4096, dict(bias=300, spread=True)),
    (30, 5, 8193, dict(hist=40, bias=1, spread=True)), (2, 90, 12289, dict(hist=500, mask=True, spread=True))])
def test_matches_its_definition(dsa, dtype, B, S, V, kw):
    _check(dsa, _inputs(B, S, V, seed=V, dtype=dtype, **kw))


@pytest.mark.parametrize("B", [3, 50])
def test_each_step_alone(dsa, B):
    full = _inputs(B, 4, 5003, seed=1, hist=400, bias=30, mask=True, greedy=(2,))
    for keep in [(), ("history",), ("draft",), ("history", "repetition"), ("history", "history_len", "frequency"),
                 ("history", "prompt_len", "presence"), ("draft", "repetition", "presence"), ("draft", "frequency"),
                 ("bias_ids", "bias_values"), ("mask",), ("temperature",), ("repetition", "frequency", "presence")]:
        _check(dsa, {"logits": full["logits"], **{k: full[k] for k in keep}})


def test_vocabularies_beyond_the_second_level_cache(dsa):
    """145 MB of logits, taken in groups of sequences; the last one is smaller."""
    _check(dsa, _inputs(37, 3, 325001, seed=3, hist=100, bias=3, spread=True, greedy=(36,)))


def test_the_most_positions(dsa):
    """4096 positions, each with the drafts before it."""
    a = _inputs(1, 4096, 130, seed=12, hist=5)
    a["draft"] = torch.randint(0, 130, (1, 4096), generator=_gen(13), device="cuda", dtype=torch.int32)
    a["frequency"], a["presence"] = torch.full((1,), 0.01, device="cuda"), torch.full((1,), 0.5, device="cuda")
    _check(dsa, a)


def test_very_many_short_rows(dsa):
    """A CTA takes all 80 rows of a sequence."""
    z = torch.randn((600, 80, 64), generator=_gen(6), device="cuda") * 4
    T = 0.5 + torch.rand(600, generator=_gen(7), device="cuda")
    want = torch.softmax(z.double() / T.double()[:, None, None], -1)
    assert bool(((dsa.dsa_logits_probs(z, T).double() - want).abs() <= 2.0 ** -14 * want + 1e-37).all())
    history = torch.full((600, 3), 9, dtype=torch.int32, device="cuda")
    got = dsa.dsa_logits_probs(z, T, history=history, frequency=torch.full((600,), 0.5, device="cuda"))
    z[..., 9] -= 1.5
    want = torch.softmax(z.double() / T.double()[:, None, None], -1)
    assert bool(((got.double() - want).abs() <= 2.0 ** -14 * want + 1e-37).all())


@pytest.mark.parametrize("V", [3000, 400000])
def test_counts_are_exact(dsa, V):
    """One token said thousands of times, one in the prompt alone, one only drafted; the same
    bias twice: values exact in 32 bits."""
    L = 5000
    z = torch.zeros((1, 3, V), device="cuda")
    z[..., 17], z[..., 18], z[..., 19], z[..., 20] = 2000.0, 8.0, -4.0, 5.0
    history = torch.full((1, L), 17, dtype=torch.int32, device="cuda")
    history[0, :100] = 18
    one = lambda x: torch.tensor([x], device="cuda")  # noqa: E731
    a = dict(logits=z, history=history, prompt_len=one(100).int(), draft=torch.tensor([[19, 19, 20]], device="cuda").int(),
             repetition=one(2.0), frequency=one(0.25), presence=one(1.0),
             bias_ids=torch.tensor([[20, 20, 17]], device="cuda").int(),
             bias_values=torch.tensor([[1.0, 2.0, 0.5]], device="cuda"))
    got = dsa.dsa_logits_probs(**a).cpu().double()
    for j, (drafted, z19) in enumerate([(0, -4.0), (1, -8.0 - 0.25 - 1), (2, -8.0 - 0.5 - 1)]):
        want = torch.zeros(V, dtype=torch.float64)
        want[17] = 1000 - 4900 * 0.25 - 1 + 0.5
        want[18], want[19], want[20] = 4.0, z19, 8.0
        want = torch.softmax(want, -1)
        assert float(((got[0, j] - want).abs() / want.clamp(min=1e-300)).nan_to_num(0)[want > 1e-30].max()) <= 2.0 ** -13


@pytest.mark.parametrize("V", [40, 50000, 400000])
def test_empty_rows_infinities_and_nan(dsa, V):
    z = torch.randn((1, 8, V), generator=_gen(2), device="cuda")
    mask = torch.full((1, 8, (V + 31) // 32), -1, dtype=torch.int32, device="cuda")
    mask[0, 0] = 0                                            # nothing is allowed
    z[0, 1] = -math.inf                                       # nothing is possible
    z[0, 2, 3:9], z[0, 2, 30] = math.inf, math.nan            # six share the probability
    z[0, 3, 5:] = math.nan
    z[0, 4, 7] = math.inf
    mask[0, 4, 0] = ~(1 << 7)                                 # the infinite one is not allowed
    z[0, 5], z[0, 5, 11] = math.nan, -5.0                     # one entry is left
    mask[0, 6] = 0
    mask[0, 6, 1] = 1 << 2                                    # one entry is allowed
    z[0, 7] = torch.finfo(torch.float32).min
    z[0, 7, 9] = torch.finfo(torch.float32).max
    got = _check(dsa, dict(logits=z, mask=mask))
    assert bool((got[0, 0] == 0).all()) and bool((got[0, 1] == 0).all())
    assert got[0, 2, 3:9].tolist() == [pytest.approx(1 / 6, rel=1e-6)] * 6 and got[0, 5, 11] == 1 and got[0, 6, 34] == 1
    assert got[0, 7, 9] == 1
    for T in (0.0, -1.0, math.nan):
        hot = dsa.dsa_logits_probs(z, torch.tensor([T], device="cuda"), mask=mask).cpu()
        assert bool((hot[0, :2] == 0).all())
        assert hot[0, 2:].sum(-1).tolist() == [1.0] * 6
        assert [int(r.argmax()) for r in hot[0, 2:]] == [3, int(z[0, 3, :5].argmax()), int(got[0, 4].argmax()), 11, 34, 9]


@pytest.mark.parametrize("T", [1e-40, 1e-6, 1e6, math.inf])
def test_extreme_temperatures(dsa, T):
    z = torch.randn((1, 2, 777), generator=_gen(3), device="cuda")
    z[0, 1, 5:9] = 50.0                                       # a tie
    z[0, 0, 3] = -math.inf
    got = dsa.dsa_logits_probs(z, torch.tensor([T], device="cuda")).cpu().double()
    want = torch.softmax((z.cpu().double() - z.cpu().double().amax(-1, keepdim=True)) / float(torch.tensor(T)), -1)
    if T == math.inf:
        want = (z.cpu() > -math.inf).double()
        want /= want.sum(-1, keepdim=True)
    assert bool(((got - want).abs() <= 2.0 ** -14 * want + 1e-37).all())


def test_greedy_ties_go_to_the_lowest_index(dsa):
    for V in (64, 30000, 151552, 400001):
        z = torch.zeros((1, 3, V), device="cuda")
        z[0, 1, [V - 1, V // 2, V // 3]] = 4.0
        z[0, 2, V - 1] = 1.0
        hot = dsa.dsa_logits_probs(z, torch.zeros(1, device="cuda")).cpu()
        assert [int(r.nonzero()[0, 0]) for r in hot[0]] == [0, V // 3, V - 1] and hot.sum() == 3


def test_unaligned_rows_outputs_and_repeats(dsa):
    """Rows that start at any element; the bytes around the output stay; two runs agree bit for bit."""
    V = 20011
    buffer = torch.randn(3 * V + 8, generator=_gen(4), device="cuda")
    for lead in range(4):
        for dtype in (torch.float32, torch.bfloat16):
            z = buffer.to(dtype)[lead:lead + 3 * V].view(1, 3, V)
            target = torch.full((3 * V + 8,), 9.0, device="cuda")
            out = target[1 + lead:1 + lead + 3 * V].view(1, 3, V)
            dsa.dsa_logits_probs(z, out=out)
            want = torch.softmax(z.double(), -1)
            assert bool(((out.double() - want).abs() <= 2.0 ** -13 * want).all())
            assert bool((target[:1 + lead] == 9).all()) and bool((target[1 + lead + 3 * V:] == 9).all())
            assert torch.equal(dsa.dsa_logits_probs(z), out)


@pytest.mark.parametrize("B,V", [(2, 60000), (20, 60000), (1, 400000)])
def test_a_captured_call_reads_the_present_history(dsa, B, V):
    a = _inputs(B, 3, V, seed=5, hist=500, bias=10, mask=True)
    out = torch.zeros((B, 3, V), device="cuda")
    dsa.dsa_logits_probs(**a, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.dsa_logits_probs(**a, out=out)
    for seed in (6, 7):
        b = _inputs(B, 3, V, seed=seed, hist=500, bias=10, mask=True)
        for k in a:
            a[k].copy_(b[k])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, dsa.dsa_logits_probs(**b))


@pytest.mark.parametrize("B,V", [(2, 30000), (24, 60000), (1, 700000)])
def test_repeats_bit_for_bit(dsa, B, V):
    a = _inputs(B, 4, V, seed=11, hist=3000, bias=40, mask=True, spread=True)
    first = dsa.dsa_logits_probs(**a)
    for _ in range(30):
        assert torch.equal(dsa.dsa_logits_probs(**a), first)


@pytest.mark.parametrize("B,V", [(3, 30000), (20, 60001)])
def test_two_calls_at_once_and_lists_that_name_nothing(dsa, B, V):
    """Two streams with a workspace each; one call's history, drafts and biases are all padding."""
    jobs = []
    for seed in (1, 2):
        a = _inputs(B, 4, V, seed=seed, hist=300, bias=6, mask=seed == 1)
        if seed == 2:
            for name in ("history", "draft", "bias_ids"):
                a[name].fill_(-1)
        jobs.append((a, torch.full((B, 4, V), 7.0, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for a, out, stream in jobs:
            dsa.dsa_logits_probs(**a, out=out, stream=stream)
    torch.cuda.synchronize()
    for a, out, _ in jobs:
        assert torch.equal(out, dsa.dsa_logits_probs(**a))
    _check(dsa, jobs[0][0])
    _check(dsa, jobs[1][0])


def test_results_of_another_stream_keep_to_themselves(dsa):
    """What a call on another stream makes for itself is not a block that the current stream has
    freed and still writes."""
    stream = torch.cuda.Stream()
    z = torch.randn((4, 5, 50000), generator=_gen(8), device="cuda")
    want = dsa.dsa_logits_probs(z)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # (some 10 ms)
    block = torch.empty_like(want).fill_(3.0)
    del block
    got = dsa.dsa_logits_probs(z, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    again = dsa.dsa_logits_probs(z, stream=stream.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(again, want)


def test_binding_refusals(dsa):
    z = torch.zeros((2, 1, 64), device="cuda")
    ints = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    for kw, err in [(dict(temperature=torch.zeros(3, device="cuda")), ValueError), (dict(history=ints(3, 4)), ValueError),
                    (dict(history_len=ints(2)), ValueError), (dict(bias_ids=ints(2, 1)), ValueError),
                    (dict(mask=ints(2, 1, 3)), ValueError), (dict(draft=ints(2, 1).long()), TypeError),
                    (dict(out=torch.zeros((2, 1, 64), dtype=torch.bfloat16, device="cuda")), TypeError)]:
        with pytest.raises(err):
            dsa.dsa_logits_probs(z, **kw)
    with pytest.raises(TypeError):
        dsa.dsa_logits_probs(z.half())
    with pytest.raises(dsa.DsaError) as err:
        dsa.dsa_logits_probs(z, out=z)
    assert err.value.status == -1
    with pytest.raises(dsa.DsaError) as err:
        dsa.dsa_logits_probs(z, bias_ids=ints(2, 5000), bias_values=torch.zeros((2, 5000), device="cuda"))
    assert err.value.status == -2
    assert dsa.dsa_logits_probs(z[:0]).shape == (0, 1, 64)


def test_a_verify_step_over_a_paged_cache(dsa):
    """The run of a step: rotate the queries, append the new rows, attend over the pages, turn
    logits into probabilities, and verify the drafts with them."""
    H, page, V, S, theta = 16, 64, 5000, 3, 1e6
    new, ctx = [S + 1, S + 1], [500, 130]
    batch = Batch(new, ctx, page, seed=8).fill()
    f, m = frequencies(64, theta)
    plan = dsa.dsa_rope_init(64, "interleaved", theta)
    g = _gen(9)
    x = torch.randn((batch.n, DQK), generator=g, device="cuda").to(torch.bfloat16)
    gamma = torch.ones(DV, device="cuda", dtype=torch.bfloat16)
    q = torch.randn((batch.n, H, DQK), generator=g, device="cuda").to(torch.bfloat16)
    positions = torch.cat([torch.arange(c - k, c) for k, c in zip(new, ctx)]).cuda()
    raw = q.clone()
    dsa.dsa_rope(q[..., DV:], positions, plan, out=q[..., DV:])
    want, size = rope(raw[..., DV:], positions, f, m, "interleaved")
    assert bool(((q[..., DV:].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * size).all())
    assert torch.equal(q[..., :DV], raw[..., :DV])
    dsa.dsa_cache_append(x, gamma, 1e-6, plan, batch.cache, batch.table, batch.cu_q, batch.ctx_len)
    out, lse = dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, 1 / 24)
    r_out, r_lse, r_size, reach = attention(batch, q, 1 / 24)
    b_out, b_lse = attention_bounds(r_out, r_lse, r_size, reach, max(ctx))
    assert bool(((out.double() - r_out).abs() <= b_out).all()) and bool(((lse.double() - r_lse).abs() <= b_lse).all())
    # an output projection stands for the model between: logits of the two models
    head = torch.randn((H * DV, V), generator=g, device="cuda") * 0.05
    target = (out.float().view(2, S + 1, -1) @ head)[:, :S].contiguous()
    drafter = (target + torch.randn(target.shape, generator=g, device="cuda")).contiguous()
    history = torch.randint(0, V, (2, 500), generator=g, device="cuda", dtype=torch.int32)
    kw = dict(history=history, history_len=torch.tensor(ctx, device="cuda").int() - S, repetition=torch.full((2,), 1.1, device="cuda"))
    q_probs = dsa.dsa_logits_probs(drafter, **kw)
    draft = torch.multinomial(q_probs.view(-1, V), 1, generator=g).view(2, S).int()
    p = dsa.dsa_logits_probs(target, draft=draft, **kw)
    ref, _ = probabilities(target, draft=draft, **kw)
    assert bool(((p.cpu().double() - ref).abs() <= 2.0 ** -12 * ref + 1e-37).all())
    u, u2 = torch.rand((2, S), generator=g, device="cuda"), torch.rand((2, S), generator=g, device="cuda")
    alpha, accept, token, length = dsa.dsa_verify(p, q_probs, draft, u, u2)
    torch.cuda.synchronize()
    at = draft.long()[..., None]
    assert torch.equal(accept.bool(), (u * q_probs.gather(2, at)[..., 0]) < p.gather(2, at)[..., 0])
    assert torch.equal(token[accept.bool()], draft[accept.bool()])
    for b in range(2):
        flags = accept[b].tolist() + [0]
        assert int(length[b]) == flags.index(0)
    assert dsa.dsa_check_device_status() == 0


def test_a_captured_verify_step_equals_the_calls_one_by_one(dsa):
    """The five calls in one graph, replayed while lengths, pages, drafts and histories change; the
    batch is padded."""
    H, page, V, S, pool = 16, 64, 60001, 3, 40
    plan = dsa.dsa_rope_init(64, "half", 1e4, 4.0, 4096)
    gamma = torch.ones(DV, device="cuda", dtype=torch.bfloat16)
    n = 2 * (S + 1) + 3
    bf = lambda *s: torch.zeros(s, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    ints = lambda *s: torch.zeros(s, device="cuda", dtype=torch.int32)  # noqa: E731
    a = dict(q=bf(n, H, DQK), x=bf(n, DQK), positions=torch.zeros(n, dtype=torch.int64, device="cuda"),
             cache=bf(pool, page, DQK), table=ints(2, 16), cu_q=ints(3), ctx=ints(2), logits=torch.zeros((2, S, V), device="cuda"),
             drafter=torch.zeros((2, S, V), device="cuda"), history=ints(2, 600), length=ints(2), draft=ints(2, S),
             u=torch.zeros((2, S), device="cuda"), u2=torch.zeros((2, S), device="cuda"),
             r=torch.full((2,), 1.2, device="cuda"))

    def step(a):
        dsa.dsa_rope(a["q"][..., DV:], a["positions"], plan, out=a["q"][..., DV:])
        dsa.dsa_cache_append(a["x"], gamma, 1e-6, plan, a["cache"], a["table"], a["cu_q"], a["ctx"])
        out, lse = dsa.dsa_paged_attn(a["q"], a["cache"], a["table"], a["cu_q"], a["ctx"], 1 / 24)
        kw = dict(history=a["history"], history_len=a["length"], draft=a["draft"], repetition=a["r"])
        p, qp = dsa.dsa_logits_probs(a["logits"], **kw), dsa.dsa_logits_probs(a["drafter"], **kw)
        return out, lse, p, qp, *dsa.dsa_verify(p, qp, a["draft"], a["u"], a["u2"])

    def fill(seed, new, ctx):
        g = _gen(seed)
        batch = Batch(new, ctx, page, seed=seed)
        for name in ("q", "x", "logits", "drafter", "cache"):
            a[name].normal_(generator=g)
        for name in ("u", "u2"):
            a[name].uniform_(generator=g)
        a["history"].random_(0, V, generator=g)
        a["draft"].random_(0, V, generator=g)
        a["length"].copy_(torch.tensor([17 * seed, 600 - seed]))
        a["table"].fill_(-1)
        a["table"][:, :batch.table.shape[1]] = batch.table
        a["cu_q"].copy_(batch.cu_q)
        a["ctx"].copy_(batch.ctx_len)
        a["positions"].fill_(0)
        a["positions"][:batch.n] = torch.cat([torch.arange(c - k, c) for k, c in zip(new, ctx)]).cuda()
        return batch.n

    fill(1, [4, 4], [700, 100])
    step(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(a)
    for seed, new, ctx in [(2, [4, 4], [704, 104]), (3, [1, 4], [900, 4]), (4, [4, 0], [63, 0])]:
        m = fill(seed, new, ctx)
        same = {k: v.clone() for k, v in a.items()}
        graph.replay()
        torch.cuda.synchronize()
        want = step(same)
        torch.cuda.synchronize()
        assert torch.equal(a["cache"], same["cache"]) and torch.equal(a["q"], same["q"])
        assert torch.equal(got[0][:m], want[0][:m]) and torch.equal(got[1][:m], want[1][:m])
        for x, y in zip(got[2:], want[2:]):
            assert torch.equal(x, y)
    assert dsa.dsa_check_device_status() == 0


@pytest.mark.parametrize("B,S,V", [(16, 7, 20480), (40, 4, 5003), (37, 3, 325001)])
def test_calls_in_a_row_share_a_workspace(dsa, B, S, V):
    """Calls one right behind the other on one workspace, their lists, maxima and greedy rows all
    different: none reads what the one before it left there."""
    jobs = [_inputs(B, S, V, seed=30 + i, hist=(900, 40, 300)[i], bias=(0, 20, 7)[i], mask=i == 1, spread=True,
                    greedy=((1,), (), (0, B - 1))[i]) for i in range(3)]
    jobs[2]["logits"] += 50.0
    alone = []
    for a in jobs:
        alone.append(dsa.dsa_logits_probs(**a))
        torch.cuda.synchronize()
    ws = torch.empty(max(dsa.lib().dsa_probs_workspace_size(B, S, V, 900, 20), 1), dtype=torch.uint8, device="cuda")
    outs = [[torch.empty_like(p) for _ in range(2)] for p in alone]
    for round_ in range(10):
        ws.fill_(255 if round_ % 2 else 0)
        for k in range(2):
            for a, out in zip(jobs, outs):
                dsa.dsa_logits_probs(**a, out=out[k], ws=ws)
        for p, out in zip(alone, outs):
            assert torch.equal(out[0], p) and torch.equal(out[1], p)


@pytest.mark.parametrize("B,V", [(1, 3000), (1, 50000), (1, 400000), (200, 3000)])
def test_large_counts_move_the_probability(dsa, B, V):
    """A token said thousands of times whose adjusted logit, 6.5, is near the largest, 8: one count
    more or less moves its probability by 28%.  All values are exact in 32 bits."""
    L = 5000
    z = torch.zeros((B, 3, V), device="cuda")
    z[..., 17], z[..., 18] = 2464.0, 16.0
    history = torch.full((B, L), 17, dtype=torch.int32, device="cuda")
    history[:, :100] = 18
    full = lambda x, dtype=torch.float32: torch.full((B,), x, dtype=dtype, device="cuda")  # noqa: E731
    got = dsa.dsa_logits_probs(
        z, history=history, prompt_len=full(100, torch.int32), draft=torch.tensor([[17, 9, 9]], device="cuda").int().repeat(B, 1),
        repetition=full(2.0), frequency=full(0.25), presence=full(1.0),
        bias_ids=torch.tensor([[17]], device="cuda").int().repeat(B, 1), bias_values=full(0.5)[:, None]).double()
    for j, count in enumerate([4900, 4901, 4901]):  # (the first draft counts in the rows behind it)
        want = torch.zeros(V, dtype=torch.float64, device="cuda")
        want[17], want[18] = 1232 - 0.25 * count - 1 + 0.5, 8.0
        if j == 2:
            want[9] = -0.25 - 1
        want = torch.softmax(want, -1)
        # exact logits; a product with log2 e, an exponential, a sum of at most 400000 terms (fewer
        # than 1024 additions deep) and a quotient: under 2^-13
        assert float(want[17]) > 1e-4 and bool(((got[:, j] - want).abs() <= 2.0 ** -13 * want).all())


def test_workspace_refusals_on_a_device(dsa):
    """Many rows need their workspace, whole and aligned; few rows need none."""
    z = torch.zeros((400, 3, 5000), device="cuda")
    size = dsa.lib().dsa_probs_workspace_size(400, 3, 5000, 0, 0)
    assert size > 0
    room = torch.empty(size + 256, dtype=torch.uint8, device="cuda")
    for ws in (room[:size - 1], room[16:16 + size], room[:0]):
        with pytest.raises(dsa.DsaError) as err:
            dsa.dsa_logits_probs(z, ws=ws)
        assert err.value.status == -3
    p = dsa.dsa_logits_probs(z, ws=room[:size])
    assert bool(((p.double() - 1 / 5000).abs() <= 2.0 ** -20 / 5000).all())
    assert dsa.lib().dsa_probs_workspace_size(2, 3, 100, 0, 0) == 0
    few, p = torch.zeros((2, 3, 100), device="cuda"), torch.empty((2, 3, 100), device="cuda")
    none = [None] * 5
    rc = dsa.lib().dsa_logits_probs(few.data_ptr(), 1, 2, 3, 100, *none, 0, None, None, None, None, None, 0, None, p.data_ptr(),
                                    None, 0, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    assert bool(((p.double() - 0.01).abs() <= 2.0 ** -20 * 0.01).all())


@pytest.mark.parametrize("B,S,V", [(2, 1, 50257), (3, 2, 151552), (60, 4, 5003)])
@pytest.mark.parametrize("cap,told", [(200_000, 200_000), (1 << 20, 1000)])
def test_long_histories(dsa, B, S, V, cap, told):
    """Histories of a long context: all of it counts, or a thousand tokens of much room."""
    g = _gen(cap + V)
    history = torch.full((B, cap), -7, dtype=torch.int32, device="cuda")
    history[:, :told] = torch.randint(0, V, (B, told), generator=g, device="cuda", dtype=torch.int32)
    history[0, told // 2:told] = 11                              # one token very often
    history[:, told:told + 50] = 3                               # behind the length: not told
    lens = torch.full((B,), told, dtype=torch.int32, device="cuda")
    lens[B - 1] = told - 7
    prompt = torch.full((B,), told // 3, dtype=torch.int32, device="cuda")
    draft = torch.randint(0, V, (B, S), generator=g, device="cuda", dtype=torch.int32)
    z = torch.randn((B, S, V), generator=g, device="cuda") * 3
    full = lambda x: torch.full((B,), x, device="cuda")  # noqa: E731
    rep, freq, pres, T = full(1.25), full(0.125), full(0.5), full(0.75)
    got = dsa.dsa_logits_probs(z, T, history=history, history_len=lens, prompt_len=prompt, draft=draft, repetition=rep,
                               frequency=freq, presence=pres)
    for b in range(B):
        for j in range(S):
            heard = history[b, :int(lens[b])].long()
            said = torch.cat((heard[int(prompt[b]):], draft[b, :j].long()))
            count = torch.bincount(said, minlength=V).double()
            seen = (torch.bincount(heard, minlength=V) + count) > 0
            y = z[b, j].double()
            y = torch.where(seen, torch.where(y > 0, y / 1.25, y * 1.25), y) - 0.125 * count - 0.5 * (count > 0)
            want = torch.softmax(y / 0.75, -1)
            # an adjusted logit passes three roundings of values up to 2^7 for what is not negligible
            # (p > 1e-30: y within 60 of the largest), and the temperature's and the exponent's
            keep = want > 1e-30
            assert bool(((got[b, j].double() - want).abs() <= 2.0 ** -12 * want)[keep].all())
            assert float(got[b, j].double()[~keep].sum()) < 1e-20
