"""dsa_paged_attn against its definition in 64 bits."""
import math

import pytest
import torch

from verify_step import DQK, DV, Batch, attention, attention_bounds, marked_bounds

pytestmark = pytest.mark.gpu
SCALE = 1 / 24


@pytest.fixture(scope="module")
def dsa():
    import sparse_long_context_score_b200 as m
    from sparse_long_context_score_b200 import build
    build.build()
    m.lib()
    return m


def _queries(n, H, seed=7, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn((n, H, DQK), generator=g, device="cuda") * std).to(torch.bfloat16)


def _check(got, batch, q, scale=SCALE, table=None):
    out, lse, size, reach = attention(batch, q, scale, table)
    most = max(batch.ctx + [1])
    b_out, b_lse = attention_bounds(out, lse, size, reach, most)
    none = lse == -math.inf
    o, l = got[0][:batch.n].double(), got[1][:batch.n].double()
    assert bool((l[none] == -math.inf).all()) and bool((o[none] == 0).all())
    assert bool(o.isfinite().all())
    err = (o - out).abs()
    assert bool((err <= b_out).all()), f"out: {float((err - b_out).max())} over the bound"
    err = (l[~none] - lse[~none]).abs()
    assert bool((err <= b_lse[~none]).all()), f"lse: {float((err - b_lse[~none]).max())} over the bound"


CASES = [
    # new tokens, cached tokens, heads, page
    ([1], [1], 16, 16),
    ([1] * 6, [1, 63, 64, 65, 127, 128], 64, 64),
    ([1] * 5, [129, 255, 256, 257, 1000], 32, 16),
    ([3, 0, 5, 1], [3, 9, 700, 64], 48, 48),
    ([2, 1], [130, 77], 1, 16),
    ([7, 4], [300, 4], 3, 80),
    ([9], [400], 5, 32),
    ([3, 2], [140, 513], 128, 256),
    ([200], [200], 16, 64),
    ([130, 1, 66], [130, 900, 1000], 64, 128),
    ([1, 1, 1], [5000, 12345, 20000], 64, 64),
    ([8, 8], [6001, 300], 64, 16),
    ([0, 0, 1, 0], [0, 4, 200, 0], 16, 16),
    ([1] * 300, [1 + (37 * i) % 500 for i in range(300)], 16, 16),
    ([1], [70000], 16, 128),
]


@pytest.mark.parametrize("new,ctx,heads,page", CASES)
def test_matches_its_definition(dsa, new, ctx, heads, page):
    batch = Batch(new, ctx, page, seed=heads + page).fill()
    q = _queries(batch.n, heads)
    _check(dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, SCALE), batch, q)
    assert dsa.dsa_check_device_status() == 0


@pytest.mark.parametrize("std,order", [(1.0, 1), (4.0, 1), (4.0, -1), (0.0, 1)])
def test_sharp_flat_and_growing_logits(dsa, std, order):
    """Logits of hundreds, whose running maximum grows (or falls) along the row; all equal."""
    batch = Batch([1, 6], [1500, 900], 64, seed=3).fill(std=std)
    flat = batch.cache.view(-1, DQK)
    for b in range(2):
        r = batch.rows(b).cuda()
        ramp = torch.linspace(0.05, 1.0, len(r), device="cuda")
        flat[r] = (flat[r].float() * (ramp if order > 0 else ramp.flip(0))[:, None]).to(torch.bfloat16)
    q = _queries(batch.n, 64, std=4.0)
    _check(dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, SCALE), batch, q)
    _check(dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, -0.5 * SCALE), batch, q, -0.5 * SCALE)
    _check(dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, 0.0), batch, q, 0.0)


def _long_batch(growing, seed):
    """48 sequences of 4 new tokens over some 20 key tiles each: a CTA's share is a few whole
    query tiles, so most key tiles lie in the middle of one."""
    batch = Batch([4] * 48, [2300 + 17 * i for i in range(48)], 64, seed=seed).fill(seed=seed)
    flat = batch.cache.view(-1, DQK)
    for b in range(48):
        r = batch.rows(b).cuda()
        steps = torch.linspace(0.02, 1.0, len(r), device="cuda") if growing else torch.linspace(1.0, 0.02, len(r), device="cuda")
        flat[r] = (flat[r].float() * steps[:, None]).to(torch.bfloat16)
    return batch


@pytest.mark.parametrize("growing", [True, False])
def test_the_maximum_moves_in_the_middle_of_a_long_row(dsa, growing):
    batch = _long_batch(growing, 11)
    q = _queries(batch.n, 64, std=8.0)
    for scale in (SCALE, -SCALE):
        got = dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, scale)
        _check(got, batch, q, scale)
        for _ in range(5):
            again = dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, scale)
            assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


def test_single_keys_far_above_the_rest(dsa):
    """One row's logit jumps by 2^30 and more at one key, or at key after key of one tile, while the
    63 rows beside it go on as they were."""
    batch = _long_batch(False, 12)
    q = _queries(batch.n, 64)
    flat = batch.cache.view(-1, DQK)
    for b in range(48):
        r = batch.rows(b)
        for i, s in enumerate((700, 701, 1003, 1500 + b, 2000)):
            t, h = batch.ends[b] + i % 4, (7 * b + 13 * i) % 64
            flat[r[s]] = (q[t, h].float() * (1 + i)).to(torch.bfloat16)
    _check(dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, SCALE), batch, q)


def test_rows_that_see_their_first_key_late(dsa):
    """The pages at the start of every context are missing, whole key tiles of them."""
    batch = _long_batch(False, 13)
    for b in range(48):
        batch.table[b, :3 + b % 24] = -1
    q = _queries(batch.n, 64)
    _check(dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, SCALE), batch, q)


@pytest.mark.parametrize("heads,new,ctx", [(64, 4, 300), (16, 7, 385), (1, 66, 66), (128, 3, 127)])
@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_what_a_token_does_not_see_may_hold_anything(dsa, heads, new, ctx, what):
    """The last new token's cached row is NaN or infinite: that token's business alone."""
    batch = Batch([new, new], [ctx, 40 + new], 16, seed=heads).fill()
    flat = batch.cache.view(-1, DQK)
    for b in range(2):
        flat[batch.rows(b)[-1]] = what
    q = _queries(batch.n, heads)
    out, lse = dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, SCALE)
    last = torch.tensor([new - 1, 2 * new - 1], device="cuda")
    assert bool(lse[last].isnan().all()) and bool(out[last].isnan().all())
    keep = torch.ones(batch.n, dtype=torch.bool, device="cuda")
    keep[last] = False
    ref = attention(batch, q, SCALE)
    b_out, b_lse = attention_bounds(*ref, ctx)
    assert bool(((out.double() - ref[0]).abs() <= b_out)[keep].all())
    assert bool(((lse.double() - ref[1]).abs() <= b_lse)[keep].all())


def test_a_bad_query_row_is_its_own_business(dsa):
    batch = Batch([3, 2], [2000, 90], 64).fill()
    q = _queries(batch.n, 64)
    q[1, 5, 17], q[4, 63, 570] = math.nan, math.inf
    out, lse = dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, SCALE)
    bad = torch.zeros((batch.n, 64), dtype=torch.bool, device="cuda")
    bad[1, 5] = bad[4, 63] = True
    assert bool(out[bad].isnan().all()) and bool(lse[bad].isnan().all())
    ref = attention(batch, q, SCALE)
    b_out, b_lse = attention_bounds(*ref, 2000)
    assert bool(((out.double() - ref[0]).abs() <= b_out)[~bad].all())
    assert bool(((lse.double() - ref[1]).abs() <= b_lse)[~bad].all())


def test_logits_of_minus_infinity_weigh_nothing(dsa):
    """Infinite rotary entries, as a mask would make them: those keys' logits are -inf, first ones,
    whole tiles and last ones among them."""
    batch = _long_batch(False, 14)
    q = _queries(batch.n, 64)
    q[..., DV] = 1.0
    flat = batch.cache.view(-1, DQK)
    for b in range(48):
        r = batch.rows(b)
        at = torch.cat((torch.arange(100 + 5 * b), torch.arange(900, 1400), torch.arange(len(r) - 3, len(r))))
        flat[r[at], DV] = -math.inf
    got = dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, SCALE)
    _check(got, batch, q)


def test_more_sequences_than_threads_of_a_block(dsa):
    new = [(0, 1, 2, 1)[i % 4] for i in range(1000)]
    ctx = [(37 * i) % 400 + 2 for i in range(1000)]
    batch = Batch(new, ctx, 16, seed=2).fill()
    q = _queries(batch.n, 24)
    _check(dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, SCALE), batch, q)


def test_two_calls_at_once(dsa):
    """Two streams, two workspaces: neither call sees the other's parts."""
    jobs = []
    for i, (new, ctx) in enumerate([([2, 1], [9000, 3000]), ([1, 3, 1], [700, 12000, 5000])]):
        batch = Batch(new, ctx, 64, seed=i).fill(seed=i)
        q = _queries(batch.n, 64, seed=i)
        out, lse = torch.empty((batch.n, 64, DV), dtype=torch.bfloat16, device="cuda"), torch.empty((batch.n, 64), device="cuda")
        jobs.append((batch, q, out, lse, dsa.paged_workspace(batch.n, len(new), 64), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for batch, q, out, lse, ws, stream in jobs:
            dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, SCALE, out=out, lse=lse, ws=ws, stream=stream)
    torch.cuda.synchronize()
    for batch, q, out, lse, _, _ in jobs:
        _check((out, lse), batch, q)

@pytest.mark.parametrize("heads", [16, 64])
def test_tokens_that_see_nothing_and_rows_that_are_not_there(dsa, heads):
    # sequence 0 has more new tokens than cached ones: its first three see nothing
    new, ctx, page = [5, 2, 4, 1, 1], [2, 300, 500, 40, 90], 16
    batch = Batch(new, ctx, page, seed=4).fill()
    batch.table[1, 3], batch.table[1, 18] = -1, batch.P          # bad entries inside and at the end
    batch.table[2, :20] = -(1 << 31)
    batch.table[3, :] = 1 << 30                                  # a sequence with no page at all
    batch.table = batch.table[:, :30].contiguous()               # sequence 2 loses its last pages
    q = _queries(batch.n, heads)
    _check(dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, SCALE), batch, q)


def test_a_padded_batch_leaves_the_rows_behind_alone(dsa):
    batch = Batch([3, 1], [90, 200], 32).fill()
    q = _queries(batch.n + 5, 32)
    q[batch.n:] = math.nan
    out = torch.full((batch.n + 5, 32, DV), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((batch.n + 5, 32), 5.0, device="cuda")
    got = dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, SCALE, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    _check(got, batch, q[:batch.n])
    assert bool((out[batch.n:] == 3).all()) and bool((lse[batch.n:] == 5).all())


def test_pages_shared_by_sequences_and_extra_table_columns(dsa):
    batch = Batch([2, 2], [256, 256], 64, extra_columns=9).fill()
    batch.table[1, :3] = batch.table[0, :3]
    q = _queries(batch.n, 16)
    _check(dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, SCALE), batch, q)


def test_repeats_bit_for_bit_and_ignores_the_workspace(dsa):
    batch = Batch([4, 1, 9], [3000, 9000, 700], 64).fill()
    q = _queries(batch.n, 64)
    first = dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, SCALE)
    ws = dsa.paged_workspace(batch.n, 3, 64)
    for fill in (0, 255, 127):
        ws.fill_(fill)
        again = dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, SCALE, ws=ws)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


def test_a_captured_call_follows_the_lengths_and_the_table(dsa):
    """One graph, replayed while the chats grow, sequences leave and pages move."""
    steps = [([1, 1, 1], [100, 2000, 17]), ([1, 1, 1], [101, 2001, 18]), ([1, 0, 1], [5000, 0, 64]), ([0, 1, 0], [0, 1, 0])]
    n, columns, page, pool = 3, 80, 64, 128
    q = _queries(n, 32)
    cache = torch.zeros((pool, page, DQK), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((3, columns), dtype=torch.int32, device="cuda")
    cu_q, ctx_len = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    out, lse = torch.zeros((n, 32, DV), dtype=torch.bfloat16, device="cuda"), torch.zeros((n, 32), device="cuda")
    ws = dsa.paged_workspace(n, 3, 32)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        dsa.dsa_paged_attn(q, cache, table, cu_q, ctx_len, SCALE, out=out, lse=lse, ws=ws)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.dsa_paged_attn(q, cache, table, cu_q, ctx_len, SCALE, out=out, lse=lse, ws=ws)
    for i, (new, ctx) in enumerate(steps):
        batch = Batch(new, ctx, page, seed=i).fill(seed=i)
        cache[:batch.P] = batch.cache
        table.fill_(-1)
        table[:, :batch.table.shape[1]] = batch.table
        cu_q.copy_(batch.cu_q)
        ctx_len.copy_(batch.ctx_len)
        graph.replay()
        torch.cuda.synchronize()
        _check((out, lse), batch, q[:batch.n])


def test_another_stream(dsa):
    batch = Batch([2], [4000], 64).fill()
    q = _queries(2, 64)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out, lse = torch.empty((2, 64, DV), dtype=torch.bfloat16, device="cuda"), torch.empty((2, 64), device="cuda")
    ws = dsa.paged_workspace(2, 1, 64)
    dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, SCALE, out=out, lse=lse, ws=ws, stream=side)
    side.synchronize()
    _check((out, lse), batch, q)
    # a block that the current stream has freed and still writes is none of that stream's
    torch.cuda._sleep(20_000_000)
    blocks = [torch.empty_like(t).fill_(3) for t in (out, lse, ws)]
    del blocks
    got = dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, SCALE, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], out) and torch.equal(got[1], lse)


def test_without_lse_and_on_the_default_stream(dsa):
    batch = Batch([2, 1], [3000, 90], 64).fill()
    q = _queries(3, 64)
    out = torch.empty((3, 64, DV), dtype=torch.bfloat16, device="cuda")
    ws = dsa.paged_workspace(3, 2, 64)
    rc = dsa.lib().dsa_paged_attn(q.data_ptr(), batch.cache.data_ptr(), batch.table.data_ptr(), batch.cu_q.data_ptr(),
                                  batch.ctx_len.data_ptr(), 3, 2, 64, batch.P, 64, batch.table.shape[1], SCALE, out.data_ptr(),
                                  None, ws.data_ptr(), ws.numel(), None)
    assert rc == 0
    torch.cuda.synchronize()
    got = dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, SCALE, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got[0], out)


def test_a_length_of_2_to_31(dsa):
    """One page again and again behind a context of 2^31 - 1: the new token's position is past what
    a table row holds, so it sees the table's 2^20 rows."""
    batch = Batch([1], [16], 16).fill()
    table = batch.table[:, :1].expand(1, 1 << 16).contiguous()
    ctx = torch.tensor([(1 << 31) - 1], dtype=torch.int32, device="cuda")
    q = _queries(1, 16)
    out, lse = dsa.dsa_paged_attn(q, batch.cache, table, batch.cu_q, ctx, SCALE)
    want, want_lse, size, reach = attention(batch, q, SCALE)
    b_out, b_lse = attention_bounds(want, want_lse, size, reach, 1 << 20)
    assert bool(((out.double() - want).abs() <= b_out).all())
    assert bool(((lse.double() - want_lse - math.log(1 << 16)).abs() <= b_lse).all())


def test_offsets_past_32_bits(dsa):
    """A pool of 5 GB: the last pages start behind 2^32 bytes."""
    batch = Batch([1], [400], 64)
    pages = (5 << 30) // (64 * DQK * 2)
    cache = torch.zeros((pages, 64, DQK), dtype=torch.bfloat16, device="cuda")
    batch.table = torch.tensor([[pages - 1, 3, pages - 5, pages - 2, 0, pages - 3, pages - 4]], dtype=torch.int32, device="cuda")
    batch.cache, batch.P = cache, pages
    batch.fill()
    q = _queries(1, 64)
    _check(dsa.dsa_paged_attn(q, cache, batch.table, batch.cu_q, batch.ctx_len, SCALE), batch, q)


def test_binding_refusals(dsa):
    batch = Batch([1], [20], 16).fill()
    q = _queries(1, 16)
    args = (batch.cache, batch.table, batch.cu_q, batch.ctx_len, SCALE)
    with pytest.raises(ValueError):
        dsa.dsa_paged_attn(q[..., :570], *args)
    with pytest.raises(TypeError):
        dsa.dsa_paged_attn(q.float(), *args)
    with pytest.raises(TypeError):
        dsa.dsa_paged_attn(q, batch.cache, batch.table.long(), batch.cu_q, batch.ctx_len, SCALE)
    with pytest.raises(ValueError):
        dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q[:1], batch.ctx_len, SCALE)
    with pytest.raises(ValueError):
        dsa.dsa_paged_attn(q.cpu(), *args, ws=torch.empty(1, dtype=torch.uint8))
    with pytest.raises(dsa.DsaError) as err:
        dsa.dsa_paged_attn(q, *args, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert err.value.status == -3
    with pytest.raises(dsa.DsaError) as err:
        dsa.dsa_paged_attn(q, batch.cache.view(-1, 8, DQK), *args[1:])
    assert err.value.status == -2
    none = dsa.dsa_paged_attn(q[:0], *args)
    assert none[0].shape == (0, 16, DV)


class _Without:
    """A batch as `attention` takes it, some of its cached positions left out: {sequence: positions}."""

    def __init__(self, batch, gone):
        self.batch, self.gone = batch, gone

    def __getattr__(self, name):
        return getattr(self.batch, name)

    def rows(self, b, table=None):
        r = self.batch.rows(b, table)
        r[self.gone[b]] = -1
        return r


@pytest.mark.parametrize("what", [math.inf, -math.inf])
@pytest.mark.parametrize("std", [1.0, 8.0])
@pytest.mark.parametrize("shape", ["chunks", "one long", "short"])
def test_infinite_latents_under_a_logit_of_minus_infinity(dsa, shape, std, what):
    """Rows with an infinite latent entry, which is a value too: where a query's sign makes the
    logit -inf the row weighs nothing, wherever it lies in its key tile, its context or a CTA's share;
    where it makes it +inf the result is NaN."""
    H = 64
    if shape == "chunks":
        batch = _long_batch(False, 21)
    elif shape == "one long":
        batch = Batch([1], [50000], 128, seed=21).fill(seed=21)
    else:
        batch = Batch([3, 1, 2], [40, 128, 300], 16, seed=21).fill(seed=21)
    q = _queries(batch.n, H, std=std)
    up = (torch.arange(H, device="cuda") * 5 % 7 < 3)
    columns = (7, 200, 511)
    for d in columns:
        q[:, :, d] = torch.where(up, 1.0, -1.0).to(torch.bfloat16)
    flat, gone = batch.cache.view(-1, DQK), {}
    for b, (new, ctx) in enumerate(zip(batch.new, batch.ctx)):
        r = batch.rows(b)
        at = {0, 1, 63, 127, 128, 700 + 3 * b, 1300, 1301, ctx // 2, ctx - new - 1, ctx - new, ctx - 1} | set(range(900, ctx, 4097))
        gone[b] = torch.tensor(sorted(s for s in at if 0 <= s < ctx))
        for i, s in enumerate(gone[b].tolist()):
            flat[r[s], columns[(i + b) % 3]] = what
    out, lse = dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, SCALE)
    assert dsa.dsa_check_device_status() == 0
    nan = up if what > 0 else ~up
    for b, (new, ctx) in enumerate(zip(batch.new, batch.ctx)):
        if int(gone[b][0]) <= ctx - new:  # (every token sees one)
            o, l = out[batch.ends[b]:batch.ends[b + 1], nan], lse[batch.ends[b]:batch.ends[b + 1], nan]
            assert bool(l.isnan().all()) and bool(o.isnan().all())
    keep = ~nan
    want = attention(_Without(batch, gone), q[:, keep].contiguous(), SCALE)
    b_out, b_lse = attention_bounds(*want, max(batch.ctx))
    o, l, none = out[:, keep].double(), lse[:, keep].double(), want[1] == -math.inf
    assert bool(o.isfinite().all())
    assert bool((l[none] == -math.inf).all()) and bool((o[none] == 0).all())
    assert bool(((o - want[0]).abs() <= b_out).all())
    assert bool(((l - want[1]).abs() <= b_lse)[~none].all())


@pytest.mark.parametrize("ctx", [100, 30000])
def test_infinite_latents_that_some_queries_multiply_by_zero(dsa, ctx):
    """0 x infinity makes those heads' logits NaN; the heads whose logit is -inf do without the row."""
    batch = Batch([2], [ctx], 64, seed=5).fill(seed=5)
    q = _queries(2, 64)
    kind = torch.arange(64, device="cuda") % 3  # 0: NaN, 1: -inf, 2: +inf
    q[:, :, 40] = torch.where(kind == 0, 0.0, torch.where(kind == 1, -1.0, 1.0)).to(torch.bfloat16)
    at = torch.tensor([0, 64, ctx // 2, ctx - 3])
    batch.cache.view(-1, DQK)[batch.rows(0)[at], 40] = math.inf
    out, lse = dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, SCALE)
    assert bool(out[:, kind != 1].isnan().all()) and bool(lse[:, kind != 1].isnan().all())
    want = attention(_Without(batch, {0: at}), q[:, kind == 1].contiguous(), SCALE)
    b_out, b_lse = attention_bounds(*want, ctx)
    assert bool(((out[:, kind == 1].double() - want[0]).abs() <= b_out).all())
    assert bool(((lse[:, kind == 1].double() - want[1]).abs() <= b_lse).all())


LONG = [
    ([1], [65536], 16, 64),
    ([1], [65499], 64, 128),
    ([1, 1, 1], [40000, 23000, 129], 64, 16),
    ([8, 3, 1], [30011, 52345, 900], 48, 64),
    ([1], [262143], 16, 256),
    ([200, 1], [33000, 128], 16, 48),
    ([2] * 40, [1000 + 313 * i for i in range(40)], 64, 64),
    ([5], [50001], 1, 32),
    ([1] * 7, [9000] * 7, 128, 128),
]


def _marked(new, ctx, page, column, seed=0):
    """A batch whose cached row at position s is zero but for a one in entry column(s)."""
    batch = Batch(new, ctx, page, seed=seed)
    flat = batch.cache.view(-1, DQK)
    for b in range(len(new)):
        r = batch.rows(b).cuda()
        flat[r] = 0
        flat[r, column(torch.arange(len(r), device="cuda"))] = 1
    return batch


def _tokens(batch):
    """(token, sequence, cached rows that it sees) of each new token."""
    for b, (new, ctx) in enumerate(zip(batch.new, batch.ctx)):
        for t in range(new):
            yield batch.ends[b] + t, b, ctx - new + t + 1


@pytest.mark.parametrize("mark", ["tile", "place"])
@pytest.mark.parametrize("new,ctx,heads,page", LONG)
def test_every_cached_row_counts_once(dsa, new, ctx, heads, page, mark):
    """Equal logits, the rows of a key tile (or those at the same place of all tiles) marked in an
    entry of their own: each entry of the output is their part of the rows seen."""
    column = (lambda s: s // 128 % DV) if mark == "tile" else (lambda s: s % 128 * 4 + s // 128 % 4)
    batch = _marked(new, ctx, page, column)
    q = torch.zeros((batch.n, heads, DQK), dtype=torch.bfloat16, device="cuda")
    out, lse = dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, SCALE)
    at = column(torch.arange(max(ctx), device="cuda"))
    want = torch.empty((batch.n, DV), dtype=torch.float64, device="cuda")
    seen = torch.empty(batch.n, dtype=torch.float64, device="cuda")
    for i, _, rows in _tokens(batch):
        want[i], seen[i] = torch.bincount(at[:rows], minlength=DV) / rows, rows
    b_out, b_lse = marked_bounds(want, seen.log())
    assert bool(((out.double() - want[:, None]).abs() <= b_out[:, None]).all())
    assert bool(((lse.double() - seen.log()[:, None]).abs() <= b_lse[:, None]).all())


@pytest.mark.parametrize("shape", ["up", "down", "zigzag", "peaks"])
@pytest.mark.parametrize("new,ctx,heads,page", LONG)
def test_every_key_tile_has_its_weight(dsa, new, ctx, heads, page, shape):
    """Key tiles marked as above, each at a logit of its own, so that maxima grow, fall, jump and are
    guessed wrong; heads with other factors, two signs.  S is one exact product."""
    batch = _marked(new, ctx, page, lambda s: s // 128 % DV)
    tiles = (max(ctx) + 127) // 128
    g = torch.Generator().manual_seed(tiles)
    level = {"up": torch.linspace(0, 240, tiles).round(), "down": torch.linspace(240, 0, tiles).round(),
             "zigzag": torch.randint(-80, 81, (tiles,), generator=g).float(),
             "peaks": torch.where(torch.rand(tiles, generator=g) < 0.1, 160.0, 0.0)}[shape]
    flat, entry, scale = batch.cache.view(-1, DQK), DV + 3, 0.125
    for b in range(len(new)):
        r = batch.rows(b)
        flat[r.cuda(), entry] = level[torch.arange(len(r)) // 128].to(torch.bfloat16).cuda()
    factor = torch.tensor([1.0, -1.0, 0.5, 2.0], dtype=torch.float64, device="cuda").repeat(32)[:heads]
    q = torch.zeros((batch.n, heads, DQK), dtype=torch.bfloat16, device="cuda")
    q[:, :, entry] = factor.to(torch.bfloat16)
    out, lse = dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, scale)
    z = factor[:, None] * level.cuda().double() * scale                                # [heads, tiles], below 60
    for i, _, rows in _tokens(batch):
        count = (rows - 128 * torch.arange(tiles, device="cuda")).clamp(0, 128).double()
        weight = z + count.log()
        total = torch.logsumexp(weight, -1)
        want = torch.zeros((heads, DV), dtype=torch.float64, device="cuda")
        want.index_add_(1, torch.arange(tiles, device="cuda") % DV, (weight - total[:, None]).exp())
        # The weights' and the output's roundings; in 32 bits, an exponent passes three roundings of
        # up to 87 (in base 2) and an exponential (2^-22), once for its weight, for each of at most
        # 87 / 8 moves of the maximum and for the join: 13 (3 x 87 x 2^-24 + 2^-22) < 2^-12
        bound = (2.0 ** -7 + 2.0 ** -11) * want + 1e-36
        assert bool(((out[i].double() - want).abs() <= bound).all()), i
        assert bool(((lse[i].double() - total).abs() <= 2.0 ** -11).all()), i
    assert dsa.dsa_check_device_status() == 0



@pytest.mark.parametrize("ctx", [5, 128, 3000, 40000])
@pytest.mark.parametrize("logit,counts", [(-1.9e38, True), (1.9e38, True), (-2.2e38, False), (-3.3e38, False)])
def test_logits_at_the_ends_of_their_range(dsa, ctx, logit, counts):
    """All rows as if masked by a number that large: equal weights up to 2e38; below -2e38 a row of
    nothing."""
    batch = Batch([1], [ctx], 64).fill()
    entry = torch.tensor(logit).to(torch.bfloat16)
    flat, r = batch.cache.view(-1, DQK), batch.rows(0).cuda()
    flat[r, DV:] = 0
    flat[r, DV] = entry.cuda()
    q = torch.zeros((1, 16, DQK), dtype=torch.bfloat16, device="cuda")
    q[..., DV] = 1
    out, lse = dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, 1.0)
    if not counts:
        assert bool((out == 0).all()) and bool((lse == -math.inf).all())
        return
    rows = flat[r, :DV].double()
    assert bool(((out.double() - rows.mean(0)).abs() <= 2.0 ** -8 * rows.mean(0).abs() + ctx * 2.0 ** -24 * rows.abs().mean(0)).all())
    # base 2 and back: four roundings
    assert bool(((lse.double() - float(entry)).abs() <= 2.0 ** -22 * abs(float(entry))).all())


@pytest.mark.parametrize("new,ctx,heads", [([1], [100], 16), ([1, 3], [3000, 129], 64), ([1], [40000], 16), ([4] * 48, [2300] * 48, 64)])
@pytest.mark.parametrize("logit", [1e5, 3e7, 1e9, 1e10, 1e20, 1.9e38, -1e5, -3e7, -1e9, -1e10, -1e20, -1.9e38])
def test_huge_logits_share_what_the_largest_have(dsa, new, ctx, heads, logit):
    """Logits of one size, some rows' a step of bf16 above the others': those share the weight."""
    batch = Batch(new, ctx, 64, seed=3).fill(seed=3)
    low = torch.tensor(logit).to(torch.bfloat16)
    bits = low.view(torch.int16)
    high = (bits - 1 if logit < 0 else bits + 1).view(torch.bfloat16)  # the next one above
    flat, scale = batch.cache.view(-1, DQK), 1.0
    q = torch.zeros((batch.n, heads, DQK), dtype=torch.bfloat16, device="cuda")
    q[..., DV] = 1
    g, best = torch.Generator().manual_seed(4), []
    for b in range(len(new)):
        r = batch.rows(b)
        top = torch.rand(len(r), generator=g) < 0.05
        top[:1 + len(r) // 2] &= b % 2 == 0            # (not before the middle of every other context)
        flat[r.cuda(), DV:] = 0
        flat[r.cuda(), DV] = torch.where(top, high, low).cuda()
        best.append(top)
    out, lse = dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, scale)
    for i, b, seen in _tokens(batch):
        top = best[b][:seen]
        top = top if top.any() else ~top
        rows = flat[batch.rows(b)[:seen][top].cuda(), :DV].double()
        value = float(high if best[b][:seen].any() else low)
        # weights of one among themselves; the next ones' are e^(-2^-8 10^5) at most
        bound = 2.0 ** -8 * rows.mean(0).abs() + (2.0 ** -8 + len(rows) * 2.0 ** -23) * rows.abs().mean(0) + 1e-30
        assert bool(((out[i].double() - rows.mean(0)).abs() <= bound).all()), i
        # base 2 and back: four roundings of that size
        assert bool(((lse[i].double() - value - math.log(len(rows))).abs() <= 2.0 ** -21 * abs(value)).all()), i


@pytest.mark.parametrize("scale", [SCALE, -SCALE])
@pytest.mark.parametrize("size", [1e7, 1e12, 1e30])
@pytest.mark.parametrize("shape", ["chunks", "one long"])
def test_huge_logits_among_ordinary_ones(dsa, shape, size, scale):
    """Whole key tiles and single rows far below and, for some heads, far above the rest, from the
    middle of the contexts on: heads without one above weigh the ordinary rows as ever, the others'
    largest ones share all of the weight."""
    batch = _long_batch(False, 31) if shape == "chunks" else Batch([2], [40000], 64, seed=31).fill(seed=31)
    q = _queries(batch.n, 64)
    kind = torch.arange(64, device="cuda") % 3  # 0: no huge logit, 1: above, 2: below
    q[:, :, DV + 1] = torch.where(kind == 0, 0.0, torch.where(kind == 1, 1.0, -1.0)).to(torch.bfloat16) * (1 if scale > 0 else -1)
    flat, gone = batch.cache.view(-1, DQK), {}
    for b, ctx in enumerate(batch.ctx):
        r = batch.rows(b)
        start = ctx // 2 + 7 * (b % 20)
        gone[b] = torch.tensor(sorted(set(range(start, start + 300)) | {start + 511, ctx - 200, ctx - 99}))
        flat[r.cuda(), DV + 1] = 0
        flat[r[gone[b]].cuda(), DV + 1] = size
        flat[r[gone[b]].cuda(), DV + 2:] = 0    # (the huge product alone)
        flat[r[gone[b]].cuda(), DV] = 0
    out, lse = dsa.dsa_paged_attn(q, batch.cache, batch.table, batch.cu_q, batch.ctx_len, scale)
    assert dsa.dsa_check_device_status() == 0
    for k, left_out in ((0, {b: torch.tensor([], dtype=torch.int64) for b in gone}), (2, gone)):
        part = q[:, kind == k].contiguous()
        want = attention(_Without(batch, left_out), part, scale)
        b_out, b_lse = attention_bounds(*want, max(batch.ctx))
        assert bool(((out[:, kind == k].double() - want[0]).abs() <= b_out).all()), k
        assert bool(((lse[:, kind == k].double() - want[1]).abs() <= b_lse).all()), k
    # above: which of the huge rows is largest depends on what 32 bits leave of the latent part beside
    # the huge product, so only that no other row counts is told here
    top = float(torch.tensor(size).to(torch.bfloat16)) * abs(scale)
    assert bool(((lse[:, kind == 1].double() - top).abs() <= 2.0 ** -20 * top + 100).all())
    most = max(float(flat[batch.rows(b)[gone[b]].cuda(), :DV].double().abs().max()) for b in gone)
    assert bool((out[:, kind == 1].double().abs() <= most * (1 + 2.0 ** -7)).all()) and bool(out.isfinite().all())
    assert bool((out[:, kind == 1].double().abs().amax(-1) > 0).all())
