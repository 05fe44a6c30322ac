"""dsa_rope and dsa_cache_append against their definitions in 64 bits."""
import math

import pytest
import torch

from verify_step import DQK, DV, Batch, frequencies, rope

pytestmark = pytest.mark.gpu
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


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


def _check_rope(x, got, positions, off, rot, layout, theta=1e4, factor=1.0, orig=0):
    f, m = frequencies(rot, theta, factor, orig)
    want, size = rope(x[..., off:off + rot], positions, f, m, layout)
    # one rounding to the type; in 32 bits: the angle (2^-24 of half a revolution, pi 2^-24),
    # sine and cosine (2 units each), their scale, two products and a sum: under 2^-20 of |a| + |b|
    bound = HALF_STEP[x.dtype] * want.abs() + 2.0 ** -20 * size
    err = (got[..., off:off + rot].double() - want).abs()
    assert bool((err <= bound).all()), f"{float((err - bound).max())} over the bound"
    assert torch.equal(got[..., :off], x[..., :off]) and torch.equal(got[..., off + rot:], x[..., off + rot:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,heads,dim,off,rot", [(1, 1, 64, 0, 64), (5, 64, 64, 0, 64), (3, 7, 576, 512, 64),
                                                 (257, 32, 128, 0, 64), (33, 3, 128, 64, 32), (9, 2, 256, 0, 256),
                                                 (4, 5, 71, 3, 6), (6, 1, 2, 0, 2), (2, 3, 96, 8, 48), (1500, 16, 64, 0, 64),
                                                 (4, 129, 128, 8, 112)])
def test_rope_matches_its_definition(dsa, layout, dtype, n, heads, dim, off, rot):
    g = _gen(n * 1000 + dim)
    x = torch.randn((n, heads, dim), generator=g, device="cuda").to(dtype)
    positions = torch.randint(0, 1 << 20, (n,), generator=g, device="cuda")
    got = dsa.dsa_rope(x, positions, dsa.dsa_rope_init(rot, layout), rot_offset=off)
    _check_rope(x, got, positions, off, rot, layout)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_far_and_negative_positions_and_a_scaled_window(dsa, layout):
    positions = torch.tensor([0, 1, -1, (1 << 20) - 1, 1 << 20, 1 << 31, -(1 << 31), 123456789], device="cuda")
    x = torch.randn((8, 4, 64), generator=_gen(1), device="cuda")
    for theta, factor, orig in [(1e4, 1.0, 0), (1e6, 1.0, 0), (1e4, 8.0, 16384), (5e5, 40.0, 4096)]:
        got = dsa.dsa_rope(x, positions, dsa.dsa_rope_init(64, layout, theta, factor, orig))
        _check_rope(x, got, positions, 0, 64, layout, theta, factor, orig)
    # a position and its negative undo each other
    plan = dsa.dsa_rope_init(64, layout)
    back = dsa.dsa_rope(dsa.dsa_rope(x, positions, plan), -positions, plan)
    assert float((back - x).abs().max()) <= 2.0 ** -19 * 2 * float(x.abs().max())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("lead,tail,dim", [(128, 512, 64), (1, 3, 64), (8, 8, 72), (0, 4, 64), (3, 0, 65)])
def test_rope_strided_in_place_and_heads_outermost(dsa, layout, lead, tail, dim):
    n, heads = 37, 6
    plan = dsa.dsa_rope_init(64, layout)
    whole = torch.randn((n, heads, lead + dim + 1), generator=_gen(2), device="cuda").to(torch.bfloat16)
    x = whole[..., lead:lead + dim]
    positions = torch.arange(5000, 5000 + n, device="cuda")
    target = torch.full((n, heads, tail + dim + 2), 7.0, device="cuda", dtype=torch.bfloat16)
    got = dsa.dsa_rope(x, positions, plan, out=target[..., tail:tail + dim])
    _check_rope(x, got, positions, 0, 64, layout)
    assert bool((target[..., :tail] == 7).all()) and bool((target[..., tail + dim:] == 7).all())
    again = whole.clone()
    dsa.dsa_rope(again[..., lead:lead + dim], positions, plan, out=again[..., lead:lead + dim])
    assert torch.equal(again[..., lead:lead + dim], got)
    assert torch.equal(again[..., :lead], whole[..., :lead]) and torch.equal(again[..., lead + dim:], whole[..., lead + dim:])
    turned = torch.empty((heads, n, dim), device="cuda", dtype=torch.bfloat16).transpose(0, 1)
    assert torch.equal(dsa.dsa_rope(x, positions, plan, out=turned), got)
    # one head read for all of them
    shared = x[:, :1].expand(n, heads, dim)
    assert torch.equal(dsa.dsa_rope(shared, positions, plan), dsa.dsa_rope(shared.contiguous(), positions, plan))


def test_rope_binding_refusals(dsa):
    plan = dsa.dsa_rope_init(64)
    x = torch.zeros((2, 3, 64), device="cuda", dtype=torch.bfloat16)
    positions = torch.zeros(2, device="cuda", dtype=torch.int64)
    with pytest.raises(TypeError):
        dsa.dsa_rope(x.half(), positions, plan)
    with pytest.raises(TypeError):
        dsa.dsa_rope(x, positions.int(), plan)
    with pytest.raises(TypeError):
        dsa.dsa_rope(x, positions, plan, out=torch.zeros_like(x, dtype=torch.float32))
    with pytest.raises(ValueError):
        dsa.dsa_rope(x, positions[:1], plan)
    with pytest.raises(ValueError):
        dsa.dsa_rope(x.transpose(1, 2), positions, plan)
    with pytest.raises(dsa.DsaError):
        dsa.dsa_rope(x, positions, plan, out=x[:, :1].expand(2, 3, 64))
    with pytest.raises(dsa.DsaError):
        dsa.dsa_rope(x, positions, plan, rot_offset=2)
    empty = dsa.dsa_rope(x[:0], positions[:0], plan)
    assert empty.shape == (0, 3, 64)


def _append_reference(batch, x, gamma, eps, f, m, layout):
    """Rows that the append writes, and how far they may be: {pool row: (value, bound)} as tensors."""
    rows, want, bound = [], [], []
    for b, n_b in enumerate(batch.new):
        where = batch.rows(b)
        for t in range(n_b):
            s = batch.ctx[b] - n_b + t
            if s < 0 or s >= len(where) or where[s] < 0:
                continue
            v = x[batch.ends[b] + t].double()
            y = v[:DV] / (v[:DV].pow(2).mean() + eps).sqrt() * gamma.double()
            z, size = rope(v[None, None, DV:], torch.tensor([s], device=x.device), f, m, layout)
            rows.append(int(where[s]))
            want.append(torch.cat((y, z[0, 0])))
            # sum of 512 squares in 32 bits (at most 64 additions deep), root, two products: under 2^-17
            bound.append(torch.cat(((2.0 ** -8 + 2.0 ** -17) * y.abs(), 2.0 ** -8 * z[0, 0].abs() + 2.0 ** -20 * size[0, 0])))
    return rows, torch.stack(want) if want else None, torch.stack(bound) if bound else None


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("new,ctx,page,stride", [
    ([1], [1], 16, 576), ([1] * 70, list(range(1, 71)), 16, 576), ([3, 0, 5, 0, 1], [3, 9, 700, 0, 64], 48, 584),
    ([130, 1, 257], [130, 4097, 1000], 64, 576), ([5, 2], [2, 2], 80, 640), ([0, 0, 4], [0, 5, 100004], 128, 576)])
def test_append_writes_the_rows(dsa, layout, new, ctx, page, stride):
    batch = Batch(new, ctx, page, seed=len(new))
    g = _gen(3)
    batch.cache.normal_(generator=g)
    whole = (torch.randn((max(batch.n, 1), stride), generator=g, device="cuda") * 4).to(torch.bfloat16)
    x = whole[:batch.n, :DQK]
    gamma = (torch.rand(DV, generator=g, device="cuda") + 0.5).to(torch.bfloat16)
    before = batch.cache.clone()
    plan = dsa.dsa_rope_init(64, layout, 1e4, 4.0, 8192)
    got = dsa.dsa_cache_append(x, gamma, 1e-6, plan, batch.cache, batch.table, batch.cu_q, batch.ctx_len)
    assert got is batch.cache
    rows, want, bound = _append_reference(batch, x, gamma, 1e-6, *frequencies(64, 1e4, 4.0, 8192), layout)
    flat = got.view(-1, DQK)
    assert bool(((flat[rows].double() - want).abs() <= bound).all())
    rest = torch.ones(len(flat), dtype=torch.bool, device="cuda")
    rest[rows] = False
    assert torch.equal(flat[rest], before.view(-1, DQK)[rest])


def test_append_zero_rows_eps_and_infinities(dsa):
    batch = Batch([4], [4], 16)
    x = torch.zeros((4, DQK), device="cuda", dtype=torch.bfloat16)
    x[1, :DV], x[2, :] = 1e18, 1e-20  # the mean square is 1e36 and 1e-40 (below the smallest normal)
    x[3, 0] = math.nan
    gamma = torch.ones(DV, device="cuda", dtype=torch.bfloat16)
    plan = dsa.dsa_rope_init(64)
    flat = dsa.dsa_cache_append(x, gamma, 1e-6, plan, batch.cache, batch.table, batch.cu_q, batch.ctx_len).view(-1, DQK)
    rows = batch.rows(0)
    assert bool((flat[rows[0]] == 0).all())
    assert bool((flat[rows[1], :DV] - 1).abs().max() <= 2.0 ** -8)
    assert bool(flat[rows[2]].isfinite().all())
    assert bool(flat[rows[3], :DV].isnan().all()) and bool((flat[rows[3], DV:] == 0).all())


def test_append_skips_what_is_not_there(dsa):
    """Tokens behind the last sequence, positions behind the table and bad table entries are
    left alone; each new token's other rows are written."""
    new, ctx, page = [20, 40, 3], [20, 90, 3], 16
    batch = Batch(new, ctx, page, seed=9)
    batch.cache.normal_(generator=_gen(4))
    batch.table[0, 1] = -1
    batch.table[1, 4] = batch.P + 7
    batch.table[2, 0] = -(1 << 31)
    batch.table = batch.table[:, :5].contiguous()          # sequence 1 loses its last page
    x = torch.randn((batch.n + 6, DQK), generator=_gen(5), device="cuda").to(torch.bfloat16)
    gamma = torch.ones(DV, device="cuda", dtype=torch.bfloat16)
    before = batch.cache.clone()
    plan = dsa.dsa_rope_init(64)
    flat = dsa.dsa_cache_append(x, gamma, 1e-6, plan, batch.cache, batch.table, batch.cu_q, batch.ctx_len).view(-1, DQK)
    rows, want, bound = _append_reference(batch, x, gamma, 1e-6, *frequencies(64, 1e4), "interleaved")
    assert len(rows) == 16 + 14 and bool(((flat[rows].double() - want).abs() <= bound).all())
    rest = torch.ones(len(flat), dtype=torch.bool, device="cuda")
    rest[rows] = False
    assert torch.equal(flat[rest], before.view(-1, DQK)[rest])


def test_append_over_many_sequences(dsa):
    """More sequences than a warp has lanes, many of them empty."""
    new = [(7 * i) % 4 for i in range(2500)]
    ctx = [k + (13 * i) % 50 for i, k in enumerate(new)]
    batch = Batch(new, ctx, 16, seed=5)
    batch.cache.zero_()
    x = torch.randn((batch.n, DQK), generator=_gen(6), device="cuda").to(torch.bfloat16)
    gamma = torch.ones(DV, device="cuda", dtype=torch.bfloat16)
    flat = dsa.dsa_cache_append(x, gamma, 1e-6, dsa.dsa_rope_init(64), batch.cache, batch.table, batch.cu_q,
                                batch.ctx_len).view(-1, DQK)
    where = torch.cat([batch.rows(b)[c - k:] for b, (k, c) in enumerate(zip(new, ctx))])
    y = x[:, :DV].double()
    want = y / (y.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()
    assert bool(((flat[where.cuda(), :DV].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -17) * want.abs()).all())
    assert int((flat != 0).any(-1).sum()) == batch.n


def test_captured_calls_follow_positions_lengths_and_tables(dsa):
    """A graph on a side stream: queries rotated in place, rows appended; replayed with other
    positions, sequences and pages, on a padded batch."""
    n, H, plan = 9, 8, dsa.dsa_rope_init(64)
    q = torch.zeros((n, H, DQK), dtype=torch.bfloat16, device="cuda")
    x = torch.zeros((n, DQK), dtype=torch.bfloat16, device="cuda")
    positions = torch.zeros(n, dtype=torch.int64, device="cuda")
    gamma = torch.ones(DV, device="cuda", dtype=torch.bfloat16)
    cache = torch.zeros((64, 16, DQK), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((3, 40), dtype=torch.int32, device="cuda")
    cu_q, ctx_len = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")

    def step():
        dsa.dsa_rope(q[..., DV:], positions, plan, out=q[..., DV:])
        dsa.dsa_cache_append(x, gamma, 1e-6, plan, cache, table, cu_q, ctx_len)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i, (new, ctx) in enumerate([([1, 1, 1], [5, 300, 16]), ([3, 0, 2], [8, 0, 18]), ([0, 9, 0], [0, 9, 0])]):
        batch = Batch(new, ctx, 16, seed=i)
        g = _gen(i)
        raw = torch.randn((n, H, DQK), generator=g, device="cuda").to(torch.bfloat16)
        q.copy_(raw)
        x.normal_(generator=g)
        positions.copy_(torch.randint(0, 1 << 20, (n,), generator=g, device="cuda"))
        cache.normal_(generator=g)
        table.fill_(-1)
        table[:, :batch.table.shape[1]] = batch.table
        cu_q.copy_(batch.cu_q)
        ctx_len.copy_(batch.ctx_len)
        before = cache.clone()
        graph.replay()
        torch.cuda.synchronize()
        _check_rope(raw, q, positions, DV, 64, "interleaved")
        rows, want, bound = _append_reference(batch, x, gamma, 1e-6, *frequencies(64, 1e4), "interleaved")
        flat = cache.view(-1, DQK)
        assert len(rows) == sum(new) and bool(((flat[rows].double() - want).abs() <= bound).all())
        rest = torch.ones(len(flat), dtype=torch.bool, device="cuda")
        rest[rows] = False
        assert torch.equal(flat[rest], before.view(-1, DQK)[rest])


def test_a_rotation_on_another_stream_keeps_its_result(dsa):
    """Its output is not a block that the current stream has freed and still writes."""
    x = torch.randn((500, 16, 64), generator=_gen(7), device="cuda")
    positions = torch.arange(500, device="cuda")
    plan, side = dsa.dsa_rope_init(64), torch.cuda.Stream()
    want = dsa.dsa_rope(x, positions, plan)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # (some 10 ms)
    block = torch.empty_like(want).fill_(3.0)
    del block
    got = dsa.dsa_rope(x, positions, plan, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-38, 1e-30, 1e-12])
def test_append_rows_of_any_magnitude(dsa, eps):
    """From the smallest subnormal entries to the largest ones, alone in their row, all alike or of
    many sizes; without an eps that would hide them."""
    g, rows = _gen(8), []
    for size in (2.0 ** -133, 2.0 ** -130, 2.0 ** -128, 2.0 ** -126, 1e-30, 1e-20, 2.0 ** -50, 1.0, 1e18, 1e30, 3.38e38):
        rows.append(torch.full((DV,), size, device="cuda"))
        one = torch.zeros(DV, device="cuda")
        one[17], one[400] = size, -size / 2
        rows.append(one)
        rows.append((torch.rand(DV, generator=g, device="cuda") - 0.5) * size)
        spread = torch.full((DV,), size, device="cuda") * 2.0 ** -torch.arange(DV, device="cuda").remainder(40)
        rows.append(spread)
    n = len(rows)
    x = torch.zeros((n, DQK), device="cuda", dtype=torch.bfloat16)
    x[:, :DV] = torch.stack(rows).to(torch.bfloat16)
    batch = Batch([n], [n], 16)
    gamma = (torch.rand(DV, generator=g, device="cuda") + 0.5).to(torch.bfloat16)
    flat = dsa.dsa_cache_append(x, gamma, eps, dsa.dsa_rope_init(64), batch.cache, batch.table, batch.cu_q,
                                batch.ctx_len).view(-1, DQK)
    y = x[:, :DV].double()
    # (eps as the 32-bit number that the call takes)
    want = y / (y.pow(2).mean(-1, keepdim=True) + torch.tensor(eps, dtype=torch.float32).double().item()).sqrt() * gamma.double()
    got = flat[batch.rows(0).cuda(), :DV].double()
    # a value below bf16's normal range is off by half of its smallest subnormal, 2^-134, and on the
    # way in 32 bits by a few of 2^-149, of which gamma < 2 makes at most twice as many
    bound = (2.0 ** -8 + 2.0 ** -17) * want.abs() + 2.0 ** -134 + 2.0 ** -145
    bad = ~((got - want).abs() <= bound)
    there = (y != 0).any(-1)  # (a row without an entry left has no direction where eps is 0)
    assert not bool(bad[there].any()), [(int(i), float(got[i, j]), float(want[i, j])) for i, j in bad.nonzero()[:5]]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_between_views_of_one_buffer(dsa, layout):
    """Same strides, any shift: refused where the two views share an element, right where they
    lie between one another."""
    import random
    rng, plan, refused = random.Random(3), dsa.dsa_rope_init(8, layout), 0
    for i in range(300):
        n, heads, dim = rng.randint(1, 5), rng.randint(1, 4), rng.choice([8, 9, 16])
        head = dim + rng.randint(0, 40)
        token = (heads - 1) * head + dim + rng.randint(0, 90)
        if i % 2:  # heads outermost
            token = dim + rng.randint(0, 40)
            head = (n - 1) * token + dim + rng.randint(0, 90)
        shift = rng.randint(1, 400)
        reach = (n - 1) * token + (heads - 1) * head + dim
        buffer = torch.randn(reach + shift, generator=_gen(i), device="cuda")
        at = [t * token + h * head + d for t in range(n) for h in range(heads) for d in range(dim)]
        meet = bool(set(at) & {s + shift for s in at})
        first, second = (buffer[k:].as_strided((n, heads, dim), (token, head, 1)) for k in (0, shift))
        x, out = (first, second) if i % 3 else (second, first)
        positions = torch.arange(n, device="cuda") * 1001
        before, was = x.clone(), buffer.clone()
        if meet:
            refused += 1
            with pytest.raises(dsa.DsaError):
                dsa.dsa_rope(x, positions, plan, out=out)
            assert torch.equal(buffer, was)
        else:
            dsa.dsa_rope(x, positions, plan, out=out)
            _check_rope(before, out, positions, 0, 8, layout)
            assert torch.equal(x, before)
    assert 50 < refused < 250
