"""Definitions in 64 bits of the operators around the verify step, and batches to test them on."""
from __future__ import annotations

import math

import torch

DQK, DV = 576, 512


def frequencies(rot, theta, factor=1.0, orig=0):
    """(f_i, m) of a rotary embedding, on the host."""
    f = [theta ** (-2.0 * i / rot) for i in range(rot // 2)]
    if factor == 1.0:
        return f, 1.0
    at = lambda turns: rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
    lo, hi = max(math.floor(at(32)), 0), min(math.ceil(at(1)), rot - 1)
    r = [min(max((i - lo) / max(hi - lo, 0.001), 0), 1) for i in range(rot // 2)]
    return [x * (1 - y) + x / factor * y for x, y in zip(f, r)], 0.1 * math.log(factor) + 1


def rope(x, positions, f, m, layout):
    """x [n, heads, rot] rotated, and |a| + |b| of each entry's pair (x's own device, 64 bits)."""
    x = x.double()
    half = x.shape[-1] // 2
    angle = positions.double()[:, None, None] * torch.tensor(f, dtype=torch.float64, device=x.device)
    if layout == "half":
        a, b = x[..., :half], x[..., half:]
    else:
        a, b = x[..., 0::2], x[..., 1::2]
    y0, y1, w = m * (a * angle.cos() - b * angle.sin()), m * (a * angle.sin() + b * angle.cos()), m * (a.abs() + b.abs())
    if layout == "half":
        return torch.cat((y0, y1), -1), torch.cat((w, w), -1)
    return torch.stack((y0, y1), -1).flatten(-2), torch.stack((w, w), -1).flatten(-2)


class Batch:
    """Sequences with `new` new tokens of `ctx` cached ones over shuffled pages; the pool's
    unused rows hold NaN."""

    def __init__(self, new, ctx, page, seed=0, spare=3, device="cuda", extra_columns=0):
        g = torch.Generator().manual_seed(seed)
        need = [-(-max(c, 0) // page) for c in ctx]
        self.page, self.new, self.ctx, self.P = page, list(new), list(ctx), sum(need) + spare
        order = torch.randperm(self.P, generator=g).to(torch.int32)
        table = torch.full((len(new), max(max(need), 1) + extra_columns), -1, dtype=torch.int32)
        at = 0
        for b, k in enumerate(need):
            table[b, :k] = order[at:at + k]
            at += k
        self.table = table.to(device)
        ends = [0]
        for k in new:
            ends.append(ends[-1] + k)
        self.ends, self.n = ends, ends[-1]
        self.cu_q = torch.tensor(ends, dtype=torch.int32, device=device)
        self.ctx_len = torch.tensor(ctx, dtype=torch.int32, device=device)
        self.cache = torch.full((self.P, page, DQK), math.nan, dtype=torch.bfloat16, device=device)

    def rows(self, b, table=None):
        """Pool rows of sequence b's cached positions, -1 where the table holds none."""
        table = (self.table if table is None else table)[b].cpu().tolist()
        out = []
        for s in range(self.ctx[b]):
            i = s // self.page
            page = table[i] if i < len(table) else -1
            out.append(page * self.page + s % self.page if 0 <= page < self.P else -1)
        return torch.tensor(out, dtype=torch.int64)

    def fill(self, seed=1, std=1.0):
        g = torch.Generator(device=self.cache.device).manual_seed(seed)
        flat = self.cache.view(-1, DQK)
        for b in range(len(self.new)):
            r = self.rows(b).to(flat.device)
            r = r[r >= 0]
            flat[r] = (torch.randn((len(r), DQK), generator=g, device=flat.device) * std).to(torch.bfloat16)
        return self


def attention(batch, q, scale, table=None):
    """(out, lse, sum of p |v|, sum of |q c| scale) in 64 bits; a token that sees nothing: 0, -inf."""
    H = q.shape[1]
    shape = (batch.n, H, DV)
    out = torch.zeros(shape, dtype=torch.float64, device=q.device)
    size, lse = torch.zeros_like(out), torch.full(shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    reach = torch.zeros_like(lse)
    flat = batch.cache.view(-1, DQK)
    for b, n_b in enumerate(batch.new):
        rows = batch.rows(b, table).to(q.device)
        for t in range(n_b):
            seen = rows[:max(batch.ctx[b] - n_b + t + 1, 0)]
            seen = seen[seen >= 0]
            if len(seen) == 0:
                continue
            c, x, i = flat[seen].double(), q[batch.ends[b] + t].double(), batch.ends[b] + t
            z = x @ c.T * scale
            lse[i] = torch.logsumexp(z, -1)
            p = (z - lse[i][:, None]).exp()
            out[i], size[i] = p @ c[:, :DV], p @ c[:, :DV].abs()
            reach[i] = (x.abs() @ c.abs().T * abs(scale)).amax(-1)
    return out, lse, size, reach


def attention_bounds(out, lse, size, reach, most):
    """How far (out, lse) may be.  Each logit is a sum of 576 products in 32 bits: off by at
    most 576 half steps of its summands' absolute sum; a weight carries its logit's and the
    normaliser's error, one bf16 rounding (2^-8), the exponential's and the sums' 2^-24 each
    (at most `most` additions); the output is rounded to bf16 once more."""
    dz = 576 * 2.0 ** -24 * reach + 4 * 2.0 ** -24 * (reach + 1)
    weight = 2 * dz + 2.0 ** -8 + (most + 8) * 2.0 ** -24
    return 2.0 ** -8 * out.abs() + 1.01 * weight[..., None] * size + 1e-30, dz + (most + 8) * 2.0 ** -24 + 2.0 ** -22 * lse.abs()


def marked_bounds(out, lse):
    """How far (out, lse) may be where all logits are zero and values zero or one.  Weights of one
    and their sums are exact in 32 bits; left are the quotient (2^-24), the product (2^-24) and the
    output's rounding (2^-8), and of lse a logarithm (one unit), its product with ln 2 and that
    constant (2^-21 in all)."""
    return (2.0 ** -8 + 2.0 ** -22) * out, 2.0 ** -21 * lse + 2.0 ** -40


def probabilities(logits, temperature=None, history=None, history_len=None, prompt_len=None, draft=None, repetition=None,
                  frequency=None, presence=None, bias_ids=None, bias_values=None, mask=None):
    """(p, size) in 64 bits, on the CPU: size[b, j] the largest magnitude that a finite logit
    takes on its way."""
    cpu = lambda t: None if t is None else t.cpu()  # noqa: E731
    logits = logits.cpu()
    history, history_len, prompt_len, draft = cpu(history), cpu(history_len), cpu(prompt_len), cpu(draft)
    bias_ids, bias_values, mask = cpu(bias_ids), cpu(bias_values), cpu(mask)
    B, S, V = logits.shape
    p, size = torch.zeros((B, S, V), dtype=torch.float64), torch.zeros((B, S), dtype=torch.float64)
    of = lambda t, b, default: default if t is None else float(t[b])  # noqa: E731
    for b in range(B):
        for j in range(S):
            z = logits[b, j].double()
            told, said = [], []
            if history is not None:
                end = history.shape[1] if history_len is None else min(int(history_len[b]), history.shape[1])
                start = 0 if prompt_len is None else int(prompt_len[b])
                for i, v in enumerate(history[b, :max(end, 0)].tolist()):
                    if 0 <= v < V:
                        told.append(v)
                        if i >= start:
                            said.append(v)
            if draft is not None:
                said += [v for v in draft[b, :j].tolist() if 0 <= v < V]
            big = z.abs()
            seen = torch.zeros(V, dtype=torch.bool)
            if told + said:
                seen[torch.tensor(told + said)] = True
            count = torch.bincount(torch.tensor(said, dtype=torch.int64), minlength=V).double()
            r, f, o = of(repetition, b, 1.0), of(frequency, b, 0.0), of(presence, b, 0.0)
            z = torch.where(seen, torch.where(z > 0, z / r, z * r), z)
            big = torch.maximum(big, z.abs()) + abs(f) * count + abs(o)
            z = z - f * count - o * (count > 0)
            if bias_ids is not None:
                for v, x in zip(bias_ids[b].tolist(), bias_values[b].double().tolist()):
                    if 0 <= v < V:
                        z[v] += x
                        big[v] += abs(x)
            z = torch.where(z.isnan(), -math.inf, z)
            if mask is not None:
                bits = mask[b, j].to(torch.int64) & 0xFFFFFFFF
                word = (bits[:, None] >> torch.arange(32)) & 1
                z[word.flatten()[:V] == 0] = -math.inf
            size[b, j] = big[z.isfinite()].max() if z.isfinite().any() else 0.0
            most = z.max()
            if most == -math.inf:
                continue
            T = of(temperature, b, 1.0)
            if not T > 0:
                p[b, j, (z == most).nonzero()[0, 0]] = 1.0
            elif most == math.inf:
                p[b, j] = (z == math.inf).double() / (z == math.inf).sum()
            else:
                p[b, j] = torch.softmax((z - most) / T, -1)
    return p, size
