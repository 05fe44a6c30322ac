"""The operators of a speculative verify step over a paged compressed cache, case by case.

One step of a serving loop: the queries' rotary part is rotated (rope), the new tokens'
compressed rows are normalised, rotated and written to the pages of their sequences
(append), the chunk of new tokens attends over the pages (attn), and the logits of the
draft positions become the probabilities that the rejection sampling takes (probs).

``run`` computes an operator in elementary torch operations where ``own`` is false, and
through the library's entry points where it is true.  ``exact`` is the definition in 64
bits.
"""
import math

import torch

own = False

DQK, DV, ROT = 576, 512, 64      # a compressed row: 512 latent entries and 64 rotary ones
SCALE = 1.0 / math.sqrt(DQK)
VOCAB = 151552
EPS = 1e-6


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # queries of a decode step: 8 sequences, 64 heads, far positions, a rotary part that
        # a projection left inside wider heads, written beside the absorbed latent part
        dict(name="rope_decode", op="rope", n=8, heads=64, dim=64, off=0, rot=64, lead=128, tail=512, layout="interleaved",
             theta=1.0e6, factor=1.0, orig=0, reach=131072, dtype="bf16"),
        # index queries of a prefill chunk: half of a 128-wide head rotates, the rest passes
        # through; positions of a window that was extended eightfold
        dict(name="rope_index_prefill", op="rope", n=4096, heads=32, dim=128, off=0, rot=64, lead=0, tail=0, layout="half",
             theta=1.0e4, factor=8.0, orig=16384, reach=131072, dtype="bf16"),
        # queries of the same chunk: 4096 x 64 heads
        dict(name="rope_prefill", op="rope", n=4096, heads=64, dim=64, off=0, rot=64, lead=128, tail=512, layout="interleaved",
             theta=1.0e6, factor=1.0, orig=0, reach=131072, dtype="bf16"),
        # a verify step: 16 sequences, the newest token and 7 drafts each
        dict(name="append_verify", op="append", seqs=16, new=8, ragged=False, ctx=32771, page=64, layout="interleaved",
             theta=1.0e6, factor=1.0, orig=0),
        # a packed prefill: 4 prompts of unequal lengths, 8000 odd tokens in all
        dict(name="append_prefill", op="append", seqs=4, new=4001, ragged=True, ctx=4001, page=64, layout="half",
             theta=1.0e4, factor=4.0, orig=8192),
        # short chats, one token each, few heads: the smallest attention call
        dict(name="attn_decode_short", op="attn", seqs=4, new=1, ragged=True, ctx=1021, heads=16, page=16),
        # decode at 128K, 64 heads
        dict(name="attn_decode_128k", op="attn", seqs=8, new=1, ragged=False, ctx=131072, heads=64, page=64),
        # the verify step's chunk: 8 new tokens per sequence over unequal contexts
        dict(name="attn_verify", op="attn", seqs=16, new=8, ragged=True, ctx=32771, heads=64, page=64),
        # a prefill chunk of two prompts
        dict(name="attn_prefill", op="attn", seqs=2, new=512, ragged=False, ctx=16384, heads=64, page=128),
        # sampling of one sequence over a small vocabulary of odd size
        dict(name="probs_one", op="probs", seqs=1, rows=1, vocab=50257, dtype="f32", hist=0, bias=0, mask=False, greedy=False),
        # a decode step's logits in bf16, chats of 1000 odd tokens
        dict(name="probs_decode", op="probs", seqs=8, rows=1, vocab=VOCAB, dtype="bf16", hist=1000, bias=0, mask=False, greedy=False),
        # the verify step: 7 draft positions of 16 sequences, penalties over 4096 tokens,
        # biases and a grammar's mask
        dict(name="probs_verify", op="probs", seqs=16, rows=7, vocab=VOCAB, dtype="f32", hist=4096, bias=32, mask=True, greedy=True),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn", "probs"])
    layout = rng.choice(["half", "interleaved"])
    theta, factor = rng.choice([1.0e4, 1.0e6]), rng.choice([1.0, 1.0, 4.0, 8.0])
    orig = 0 if factor == 1.0 else rng.choice([8192, 16384])
    if op == "rope":
        rot = rng.choice([32, 64, 64, 128])
        dim = rot + rng.choice([0, 0, 64])
        return dict(op=op, n=_spread(rng, 1, 2048), heads=rng.choice([1, 16, 32, 48, 64]), dim=dim,
                    off=rng.choice([0, dim - rot]), rot=rot, lead=rng.choice([0, 128]), tail=rng.choice([0, 512]),
                    layout=layout, theta=theta, factor=factor, orig=orig, reach=_spread(rng, 64, 1 << 20),
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "append":
        new = _spread(rng, 1, 4001)
        return dict(op=op, seqs=_spread(rng, 1, max(1, 8192 // new)) if new > 64 else _spread(rng, 1, 64), new=new,
                    ragged=rng.random() < 0.5, ctx=new + _spread(rng, 1, 32768), page=rng.choice([16, 64, 128]),
                    layout=layout, theta=theta, factor=factor, orig=orig)
    if op == "attn":
        new = rng.choice([1, 1, 2, 4, 8, _spread(rng, 9, 300)])
        ctx = new + _spread(rng, 1, 40000 if new <= 8 else 8192)
        return dict(op=op, seqs=_spread(rng, 1, 24) if new <= 8 else rng.randint(1, 3), new=new, ragged=rng.random() < 0.6,
                    ctx=ctx, heads=rng.choice([16, 32, 48, 64]), page=rng.choice([16, 32, 64, 128]))
    return dict(op=op, seqs=_spread(rng, 1, 16), rows=rng.choice([1, 1, 2, 4, 7]), vocab=_spread(rng, 20011, VOCAB),
                dtype=rng.choice(["f32", "bf16"]), hist=rng.choice([0, _spread(rng, 1, 8192)]),
                bias=rng.choice([0, _spread(rng, 1, 256)]), mask=rng.random() < 0.5, greedy=rng.random() < 0.3)


# ------------------------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _frequencies(rot, theta, factor, orig):
    """Angular steps of the rotary pairs (64 bits, host).  With factor > 1 the pairs that
    turn fewer than once over the original length are slowed down by the factor, those that
    turn more than 32 times are kept, and the ones between are blended linearly; cosines
    and sines are multiplied by 0.1 ln(factor) + 1."""
    freq = [theta ** (-2.0 * i / rot) for i in range(rot // 2)]
    if factor == 1.0:
        return freq, 1.0
    pair = lambda turns: rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
    lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
    ramp = [min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(rot // 2)]
    return [f * (1 - r) + f / factor * r for f, r in zip(freq, ramp)], 0.1 * math.log(factor) + 1.0


def _rope_plan(case, rot):
    if not own:
        return None
    import sparse_long_context_score_b200 as dsa
    return dsa.dsa_rope_init(rot, layout=case["layout"], theta=case["theta"], factor=case["factor"], orig_len=case["orig"])


def _lengths(case):
    """New tokens and cached tokens (the new ones among them) of each sequence: a ragged
    batch's lengths are spread evenly below the longest, which is the first sequence's."""
    B, new, ctx = case["seqs"], case["new"], case["ctx"]
    if not case["ragged"]:
        return [new] * B, [ctx] * B
    spread = lambda b, step: (b * step) % 1.0  # noqa: E731
    n = [max(1, round(new * (1.0 - 0.75 * spread(b, 0.618034)))) for b in range(B)]
    c = [max(n[b], round(ctx * (1.0 - 0.9 * spread(b, 0.414214)))) for b in range(B)]
    return n, c


def _pages(case, g, ctx):
    """A table of pages in shuffled order, and the number of pages of the pool."""
    page, B = case["page"], len(ctx)
    need = [-(-c // page) for c in ctx]
    order = torch.randperm(sum(need) + 3, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    return table, sum(need) + 3


def prepare(case, seed):
    g = _generator(seed)
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    s = {"case": case}
    if case["op"] == "rope":
        n, heads, dim, dt = case["n"], case["heads"], case["dim"], torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        s["x"] = torch.randn((n, heads, case["lead"] + dim), generator=g, device="cuda").to(dt)[..., case["lead"]:]
        s["out"] = torch.zeros((n, heads, case["tail"] + dim), device="cuda", dtype=dt)[..., case["tail"]:]
        first = int(torch.randint(0, max(1, case["reach"] - n), (1,), generator=g, device="cuda"))
        s["positions"] = torch.arange(first, first + n, device="cuda") if n > 64 else torch.randint(
            0, case["reach"], (n,), generator=g, device="cuda")
        freq, s["mscale"] = _frequencies(case["rot"], case["theta"], case["factor"], case["orig"])
        s["freq"] = torch.tensor(freq, dtype=torch.float64, device="cuda")
        s["rope"] = _rope_plan(case, case["rot"])
        return s
    if case["op"] in ("append", "attn"):
        new, ctx = _lengths(case)
        s["table"], P = _pages(case, g, ctx)
        ends = [0]
        for k in new:
            ends.append(ends[-1] + k)
        s["cu_q"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        s["ctx_len"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        s["n"], s["most_new"], s["most_ctx"] = ends[-1], max(new), max(ctx)
        s["cache"] = normal(P, case["page"], DQK)
        if case["op"] == "attn":
            s["q"] = normal(s["n"], case["heads"], DQK)
            if own:
                import sparse_long_context_score_b200 as dsa
                s["ws"] = dsa.paged_workspace(s["n"], len(new), case["heads"])
            return s
        s["x"] = normal(s["n"], DQK) * 3
        s["gamma"] = (torch.rand(DV, generator=g, device="cuda") + 0.5).to(torch.bfloat16)
        freq, s["mscale"] = _frequencies(ROT, case["theta"], case["factor"], case["orig"])
        s["freq"] = torch.tensor(freq, dtype=torch.float64, device="cuda")
        s["rope"] = _rope_plan(case, ROT)
        return s
    B, S, V = case["seqs"], case["rows"], case["vocab"]
    s["logits"] = torch.randn((B, S, V), generator=g, device="cuda") * 3.0
    if case["dtype"] == "bf16":
        s["logits"] = s["logits"].to(torch.bfloat16)
    uniform = lambda lo, hi: lo + (hi - lo) * torch.rand(B, generator=g, device="cuda")  # noqa: E731
    s["temperature"] = uniform(0.5, 1.3)
    if case["greedy"]:
        s["temperature"][B // 2] = 0.0
    s["repetition"] = s["frequency"] = s["presence"] = s["history"] = s["history_len"] = s["prompt_len"] = s["draft"] = None
    s["bias_ids"] = s["bias_values"] = s["mask"] = None
    if case["hist"]:
        s["repetition"], s["frequency"], s["presence"] = uniform(1.0, 1.3), uniform(0.0, 0.5), uniform(0.0, 0.5)
        # few tokens are frequent, most are rare
        s["history"] = (V * torch.rand((B, case["hist"]), generator=g, device="cuda") ** 4).to(torch.int32).clamp_(max=V - 1)
        s["history_len"] = (case["hist"] * uniform(0.3, 1.0)).to(torch.int32).clamp_(min=1)
        s["history_len"][0] = case["hist"]
        s["prompt_len"] = (s["history_len"] * uniform(0.2, 0.9)).to(torch.int32)
        s["draft"] = torch.randint(0, V, (B, S), generator=g, device="cuda", dtype=torch.int32)
    if case["bias"]:
        s["bias_ids"] = torch.randint(0, V, (B, case["bias"]), generator=g, device="cuda", dtype=torch.int32)
        s["bias_values"] = torch.randn((B, case["bias"]), generator=g, device="cuda") * 4.0
    if case["mask"]:
        s["mask"] = torch.randint(-(1 << 31), 1 << 31, (B, S, (V + 31) // 32), generator=g, device="cuda").to(torch.int32)
    s["out"] = torch.empty((B, S, V), dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------------------- plain forms
def _rotate(x, positions, s, layout):
    """x [n, heads, rot] in 32 bits, rotated; angles in 64 bits."""
    angle = positions.to(torch.float64)[:, None] * s["freq"]
    cos, sin = (angle.cos() * s["mscale"]).float()[:, None], (angle.sin() * s["mscale"]).float()[:, None]
    half = x.shape[-1] // 2
    a, b = (x[..., :half], x[..., half:]) if layout == "half" else (x[..., 0::2], x[..., 1::2])
    a, b = a * cos - b * sin, a * sin + b * cos
    return torch.cat((a, b), -1) if layout == "half" else torch.stack((a, b), -1).flatten(-2)


def _token_places(s):
    """Sequence, place in the chunk and cached position of every new token."""
    t = torch.arange(s["n"], device="cuda")
    b = torch.searchsorted(s["cu_q"], t.to(torch.int32), right=True) - 1
    place = t - s["cu_q"][b]
    return b, place, s["ctx_len"][b] - (s["cu_q"][b + 1] - s["cu_q"][b]) + place


def _plain_rope(s, c):
    lo, hi = c["off"], c["off"] + c["rot"]
    x = s["x"].float()
    y = torch.cat((x[..., :lo], _rotate(x[..., lo:hi], s["positions"], s, c["layout"]), x[..., hi:]), -1)
    return s["out"].copy_(y)


def _plain_append(s, c):
    b, _, position = _token_places(s)
    x = s["x"].float()
    latent = x[:, :DV] * torch.rsqrt(x[:, :DV].square().mean(-1, keepdim=True) + EPS) * s["gamma"].float()
    turned = _rotate(x[:, None, DV:], position, s, c["layout"])[:, 0]
    rows = torch.cat((latent, turned), -1).to(torch.bfloat16)
    page = s["table"][b, torch.div(position, c["page"], rounding_mode="floor").long()]
    s["cache"].view(-1, DQK)[page.long() * c["page"] + position % c["page"]] = rows
    return s["cache"]


def _plain_attn(s, c):
    B, H, T = s["table"].shape[0], c["heads"], s["most_new"]
    keys = s["cache"][s["table"].clamp(min=0).long()].view(B, -1, DQK).float()
    t = torch.arange(T, device="cuda")
    new = s["cu_q"][1:] - s["cu_q"][:-1]
    there = t[None] < new[:, None]
    at = torch.where(there, s["cu_q"][:-1, None] + t[None], s["n"])         # row n: nobody's
    z = torch.bmm(s["q"][at.clamp(max=s["n"] - 1)].float().view(B, T * H, DQK), keys.transpose(1, 2)).mul_(SCALE)
    last = s["ctx_len"][:, None] - new[:, None] + t[None]
    hidden = torch.arange(keys.shape[1], device="cuda")[None, None] > last[:, :, None]
    z.view(B, T, H, -1).masked_fill_(hidden[:, :, None], -math.inf)
    most = z.amax(-1, keepdim=True)
    most = torch.where(most == -math.inf, 0.0, most)
    z = z.sub_(most).exp_()
    total = z.sum(-1, keepdim=True)
    o = torch.bmm(z, keys[..., :DV]).div_(total)
    out = torch.empty((s["n"] + 1, H, DV), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((s["n"] + 1, H), dtype=torch.float32, device="cuda")
    out[at] = o.view(B, T, H, DV).to(torch.bfloat16)
    lse[at] = (most + total.log()).view(B, T, H)
    return out[:-1], lse[:-1]


def _plain_probs(s, c):
    B, S, V = c["seqs"], c["rows"], c["vocab"]
    z = s["logits"].float()
    if s["history"] is not None:
        L = c["hist"]
        place = torch.arange(L, device="cuda")[None]
        ids = s["history"].long()
        valid = place < s["history_len"][:, None]
        spoken = (valid & (place >= s["prompt_len"][:, None])).float()
        seen = torch.zeros((B, V), device="cuda").scatter_add_(1, ids, valid.float())
        count = torch.zeros((B, V), device="cuda").scatter_add_(1, ids, spoken)
        earlier = torch.tril(torch.ones((S, S), device="cuda"), -1)                       # drafts before row j
        drafts = s["draft"].long()[:, None].expand(B, S, S)
        count = count[:, None].repeat(1, S, 1).scatter_add_(2, drafts, earlier.expand(B, S, S).contiguous())
        rep = s["repetition"][:, None, None]
        z = torch.where((seen[:, None] > 0) | (count > 0), torch.where(z > 0, z / rep, z * rep), z)
        z = z - s["frequency"][:, None, None] * count - s["presence"][:, None, None] * (count > 0)
    if s["bias_ids"] is not None:
        z = z + torch.zeros((B, V), device="cuda").scatter_add_(1, s["bias_ids"].long(), s["bias_values"])[:, None]
    v = torch.arange(V, device="cuda")
    if s["mask"] is not None:
        allowed = (s["mask"][..., v // 32] >> (v % 32).to(torch.int32)) & 1
        z = z.masked_fill(allowed == 0, -math.inf)
    most = z.amax(-1, keepdim=True)
    first = torch.where(z == most, v, V).amin(-1, keepdim=True)
    t = s["temperature"][:, None, None]
    e = ((z - most) / torch.where(t > 0, t, 1.0)).exp()
    return s["out"].copy_(torch.where(t > 0, e / e.sum(-1, keepdim=True), (v == first).float()))


def run(s):
    c = s["case"]
    if own:
        import sparse_long_context_score_b200 as dsa
        if c["op"] == "rope":
            return dsa.dsa_rope(s["x"], s["positions"], s["rope"], rot_offset=c["off"], out=s["out"])
        if c["op"] == "append":
            return dsa.dsa_cache_append(s["x"], s["gamma"], EPS, s["rope"], s["cache"], s["table"], s["cu_q"], s["ctx_len"])
        if c["op"] == "attn":
            return dsa.dsa_paged_attn(s["q"], s["cache"], s["table"], s["cu_q"], s["ctx_len"], SCALE, ws=s["ws"])
        return dsa.dsa_logits_probs(s["logits"], s["temperature"], history=s["history"], history_len=s["history_len"],
                                    prompt_len=s["prompt_len"], draft=s["draft"], repetition=s["repetition"],
                                    frequency=s["frequency"], presence=s["presence"], bias_ids=s["bias_ids"],
                                    bias_values=s["bias_values"], mask=s["mask"], out=s["out"])
    return {"rope": _plain_rope, "append": _plain_append, "attn": _plain_attn, "probs": _plain_probs}[c["op"]](s, c)


# ------------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "rope":
        size = 4 if c["dtype"] == "f32" else 2
        cells = c["n"] * c["heads"]
        return {"bytes": 2 * size * cells * c["dim"] + 8 * c["n"], "flops": 3 * cells * c["rot"]}
    if c["op"] == "probs":
        cells = c["seqs"] * c["rows"] * c["vocab"]
        size = 4 if c["dtype"] == "f32" else 2
        lists = 4 * c["seqs"] * (c["hist"] + 2 * c["bias"])
        return {"bytes": cells * (size + 4) + (cells // 8 if c["mask"] else 0) + lists, "flops": 5 * cells}
    new, ctx = _lengths(c)
    n = sum(new)
    if c["op"] == "append":
        return {"bytes": n * 2 * DQK * 2 + 2 * DV, "flops": n * (4 * DV + 3 * ROT)}
    pairs = c["heads"] * sum(k * x - k * (k - 1) // 2 for k, x in zip(new, ctx))   # (query, visible row) pairs
    return {"bytes": 2 * DQK * sum(ctx) + n * c["heads"] * (2 * DQK + 2 * DV + 4), "flops": 2 * (DQK + DV) * pairs}


# ------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The definitions, token by token or sequence by sequence, in 64 bits."""
    s, d = prepare(case, seed), torch.float64
    if case["op"] in ("rope", "append"):
        freq, mscale = _frequencies(case["rot"] if case["op"] == "rope" else ROT, case["theta"], case["factor"], case["orig"])
        freq = torch.tensor(freq, dtype=d, device="cuda")

        def turn(x, positions):  # pairs as complex numbers, times exp(i position frequency)
            w = torch.polar(torch.full((len(positions), len(freq)), mscale, dtype=d, device="cuda"), positions.to(d)[:, None] * freq)
            if case["layout"] == "half":
                pairs = x.unflatten(-1, (2, -1)).transpose(-1, -2)
            else:
                pairs = x.unflatten(-1, (-1, 2))
            y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w[:, None])
            return (y.transpose(-1, -2) if case["layout"] == "half" else y).flatten(-2)

        if case["op"] == "rope":
            y = s["x"].to(d)
            part = slice(case["off"], case["off"] + case["rot"])
            y[..., part] = turn(y[..., part].clone(), s["positions"])
            return y
        pool = s["cache"].to(d)
        for b in range(case["seqs"]):
            lo, hi, end = int(s["cu_q"][b]), int(s["cu_q"][b + 1]), int(s["ctx_len"][b])
            x = s["x"][lo:hi].to(d)
            p = torch.arange(end - (hi - lo), end, device="cuda")
            rms = (x[:, :DV].pow(2).sum(-1, keepdim=True) / DV + EPS).sqrt()
            row = torch.cat((x[:, :DV] / rms * s["gamma"].to(d), turn(x[:, None, DV:], p)[:, 0]), -1)
            pool[s["table"][b].long()[p // case["page"]], p % case["page"]] = row
        return pool
    if case["op"] == "attn":
        out = torch.empty((s["n"], case["heads"], DV), dtype=d, device="cuda")
        lse = torch.empty((s["n"], case["heads"]), dtype=d, device="cuda")
        for b in range(case["seqs"]):
            lo, hi, end = int(s["cu_q"][b]), int(s["cu_q"][b + 1]), int(s["ctx_len"][b])
            used = -(-end // case["page"])
            rows = torch.cat([s["cache"][int(p)] for p in s["table"][b, :used].cpu()])[:end].to(d)
            for t in range(lo, hi, 64):
                q = s["q"][t:min(hi, t + 64)].to(d)
                z = torch.einsum("thd,sd->ths", q, rows) * SCALE
                seen = end - hi + torch.arange(t, t + len(q), device="cuda") + 1
                z[(torch.arange(end, device="cuda")[None] >= seen[:, None])[:, None].expand_as(z)] = -math.inf
                lse[t:t + len(q)] = torch.logsumexp(z, -1)
                out[t:t + len(q)] = torch.einsum("ths,sd->thd", (z - lse[t:t + len(q), :, None]).exp(), rows[:, :DV])
        return out, lse
    B, S, V = case["seqs"], case["rows"], case["vocab"]
    p = torch.empty((B, S, V), dtype=d, device="cuda")
    for b in range(B):
        for j in range(S):
            z = s["logits"][b, j].to(d)
            if s["history"] is not None:
                told = s["history"][b, :int(s["history_len"][b])].long()
                said = torch.cat((told[int(s["prompt_len"][b]):], s["draft"][b, :j].long()))
                often = torch.bincount(said, minlength=V)
                known = torch.bincount(told, minlength=V) + often > 0
                r = s["repetition"][b].to(d)
                z[known] = torch.where(z[known] > 0, z[known] / r, z[known] * r)
                z -= s["frequency"][b].to(d) * often + s["presence"][b].to(d) * (often > 0)
            if s["bias_ids"] is not None:
                z.index_put_((s["bias_ids"][b].long(),), s["bias_values"][b].to(d), accumulate=True)
            if s["mask"] is not None:
                bits = s["mask"][b, j].to(torch.int64).remainder(1 << 32)
                word = torch.stack([(bits >> k) & 1 for k in range(32)], -1).flatten()[:V]
                z[word == 0] = -math.inf
            if s["temperature"][b] > 0:
                p[b, j] = torch.softmax(z / s["temperature"][b].to(d), -1)
            else:
                p[b, j] = 0
                p[b, j, (z == z.max()).nonzero()[0, 0]] = 1
    return p
