"""Refusals of the entry points around the verify step and the rotary plan's frequencies.
CPU only: no call here reaches a kernel launch."""
import ctypes
import math

import pytest

import sparse_long_context_score_b200 as dsa
from verify_step import DV, frequencies, marked_bounds

FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced: every call below fails validation
AT = 1 << 20
ODD = ctypes.c_void_p((1 << 20) + 1)
TWO = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def L():
    from sparse_long_context_score_b200 import build
    build.build()
    return dsa.lib()


@pytest.mark.parametrize("layout", dsa.ROPE_LAYOUTS)
@pytest.mark.parametrize("rot,theta,factor,orig", [(2, 10.0, 1.0, 0), (64, 1e4, 1.0, 0), (64, 1e6, 8.0, 16384),
                                                   (128, 1e4, 40.0, 4096), (256, 1e4, 1.5, 1), (6, 5e5, 4.0, 100)])
def test_plan_frequencies(L, layout, rot, theta, factor, orig):
    plan = dsa.dsa_rope_init(rot, layout, theta, factor, orig)
    f, m = frequencies(rot, theta, factor, orig)
    assert plan.rot_dim == rot and plan.layout == dsa.ROPE_LAYOUTS.index(layout)
    assert plan.mscale == ctypes.c_float(m).value
    for i in range(128):
        want = f[i] / (2 * math.pi) if i < rot // 2 else 0.0
        assert abs(plan.turns[i] - want) <= 8 * 2.0 ** -53 * want


def test_plan_refusals(L):
    plan = dsa.RopePlan()
    at = ctypes.addressof(plan)
    assert L.dsa_rope_init(None, 64, 0, 1e4, 1.0, 0) == -1
    for rot, layout, theta, factor, orig in [(0, 0, 1e4, 1.0, 0), (-2, 0, 1e4, 1.0, 0), (63, 0, 1e4, 1.0, 0),
                                             (64, 2, 1e4, 1.0, 0), (64, 0, 1.0, 1.0, 0), (64, 0, math.nan, 1.0, 0),
                                             (64, 0, math.inf, 1.0, 0), (64, 0, 1e4, 0.5, 0), (64, 0, 1e4, math.nan, 0),
                                             (64, 0, 1e4, math.inf, 4096), (64, 0, 1e4, 4.0, 0)]:
        assert L.dsa_rope_init(at, rot, layout, theta, factor, orig) == -1, (rot, layout, theta, factor, orig)
    assert L.dsa_rope_init(at, 258, 0, 1e4, 1.0, 0) == -2
    with pytest.raises(ValueError):
        dsa.dsa_rope_init(64, "quarter")


def test_rope_refusals(L):
    plan = dsa.dsa_rope_init(64)
    p = ctypes.addressof(plan)
    ok = dict(x=FAKE, pos=FAKE, n=4, heads=2, dim=64, off=0, plan=p, dtype=0, xt=128, xh=64,
              out=ctypes.c_void_p(1 << 24), ot=128, oh=64)

    def call(**kw):
        a = {**ok, **kw}
        return L.dsa_rope(a["x"], a["pos"], a["n"], a["heads"], a["dim"], a["off"], a["plan"], a["dtype"], a["xt"], a["xh"],
                          a["out"], a["ot"], a["oh"], None)

    assert call(n=0) == 0                                      # nothing to do
    for kw in [dict(x=None), dict(pos=None), dict(out=None), dict(plan=None), dict(n=-1), dict(heads=0), dict(dim=0),
               dict(off=-1), dict(off=1), dict(dim=63), dict(x=ODD), dict(out=ODD), dict(pos=TWO), dict(xt=-128),
               dict(oh=-64), dict(x=TWO, dtype=1),
               dict(oh=63), dict(ot=127), dict(ot=0), dict(oh=0),  # heads of the output overlap
               dict(out=FAKE, ot=256)]:                        # in place with other strides
        assert call(**kw) == -1, kw
    assert call(dtype=2) == -2
    assert call(n=1 << 50) == -2
    assert call(n=0, ot=64, oh=256) == 0                       # heads outermost
    bad = dsa.RopePlan()
    for rot, layout in [(0, 0), (63, 0), (258, 0), (64, 2), (64, -1)]:
        bad.rot_dim, bad.layout = rot, layout
        assert call(plan=ctypes.addressof(bad), dim=512, xt=1024, xh=512, ot=1024, oh=512) == -1


def test_append_refusals(L):
    plan = dsa.dsa_rope_init(64)
    p = ctypes.addressof(plan)
    wide = dsa.dsa_rope_init(128)
    ok = dict(x=FAKE, stride=576, gamma=FAKE, eps=1e-6, plan=p, cache=FAKE, table=FAKE, cu=FAKE, ctx=FAKE, n=4, B=2, P=8,
              page=64, most=4)

    def call(**kw):
        a = {**ok, **kw}
        return L.dsa_cache_append(a["x"], a["stride"], a["gamma"], a["eps"], a["plan"], a["cache"], a["table"], a["cu"],
                                  a["ctx"], a["n"], a["B"], a["P"], a["page"], a["most"], None)

    assert call(n=0) == 0
    for kw in [dict(x=None), dict(gamma=None), dict(plan=None), dict(cache=None), dict(table=None), dict(cu=None),
               dict(ctx=None), dict(n=-1), dict(B=0), dict(P=0), dict(page=0), dict(most=0), dict(stride=575),
               dict(stride=577), dict(stride=580), dict(x=TWO), dict(gamma=TWO), dict(cache=TWO), dict(table=TWO),
               dict(eps=-1.0), dict(eps=math.nan)]:
        assert call(**kw) == -1, kw
    assert call() == -1 and call(x=AT + 8 * 64 * 1152 - 16) == -1 and call(x=AT - 4 * 1152 + 16) == -1  # x in the cache
    assert call(page=24) == -2
    assert call(P=1 << 26, page=64) == -2
    assert call(plan=ctypes.addressof(wide)) == -2


def test_paged_attn_refusals(L):
    ok = dict(q=FAKE, cache=FAKE, table=FAKE, cu=FAKE, ctx=FAKE, n=4, B=2, H=16, P=8, page=64, most=4, scale=0.1, out=FAKE,
              lse=FAKE, ws=FAKE, size=1 << 40)

    def call(**kw):
        a = {**ok, **kw}
        return L.dsa_paged_attn(a["q"], a["cache"], a["table"], a["cu"], a["ctx"], a["n"], a["B"], a["H"], a["P"], a["page"],
                                a["most"], a["scale"], a["out"], a["lse"], a["ws"], a["size"], None)

    assert call(n=0) == 0
    for kw in [dict(q=None), dict(cache=None), dict(table=None), dict(cu=None), dict(ctx=None), dict(out=None), dict(n=-1),
               dict(B=0), dict(H=0), dict(P=0), dict(page=0), dict(most=0), dict(q=TWO), dict(cache=TWO), dict(out=TWO),
               dict(lse=TWO), dict(ctx=TWO), dict(scale=math.nan), dict(scale=math.inf), dict(scale=-3e38)]:
        assert call(**kw) == -1, kw
    apart = dict(q=FAKE, out=AT + (1 << 20), lse=AT + (1 << 21), cache=AT + (1 << 22))
    for kw in [dict(out=FAKE), dict(out=AT + 4 * 16 * 1152 - 16), dict(out=AT + (1 << 22) + 1152), dict(lse=AT + 16),
               dict(lse=AT + (1 << 20) + 64), dict(lse=AT + (1 << 22))]:  # outputs over inputs or one another
        assert call(**{**apart, **kw}) == -1, kw
    for kw in [dict(H=129), dict(page=40), dict(P=1 << 26), dict(n=1 << 30)]:
        assert call(**kw) == -2, kw
    for n, B, H in [(-1, 1, 1), (1, 0, 1), (1, 1, 0), (1, 1, 129), (1 << 30, 1, 16)]:
        assert L.dsa_paged_workspace_size(n, B, H) == 0


def test_logits_probs_refusals(L):
    names = ["logits", "dtype", "B", "S", "V", "temperature", "repetition", "frequency", "presence", "history", "cap",
             "history_len", "prompt_len", "draft", "bias_ids", "bias_values", "nbias", "mask", "p", "ws", "size"]
    ok = dict(logits=FAKE, dtype=1, B=2, S=3, V=100, p=FAKE, cap=0, nbias=0, ws=FAKE, size=1 << 30)

    def call(**kw):
        a = {**ok, **kw}
        return L.dsa_logits_probs(*[a.get(k) for k in names], None)

    assert call(B=0) == 0 and call(S=0) == 0
    for kw in [dict(logits=None), dict(p=None), dict(B=-1), dict(S=-1), dict(V=0), dict(V=1 << 24), dict(cap=-1),
               dict(nbias=-1), dict(nbias=1), dict(nbias=1, bias_ids=FAKE), dict(logits=TWO), dict(logits=ODD, dtype=0),
               dict(p=TWO), dict(mask=TWO), dict(draft=TWO), dict(temperature=TWO), dict(B=1 << 20, S=1 << 20)]:
        assert call(**kw) == -1, kw
    assert call(dtype=2) == -2
    assert call(cap=1 << 30, history=FAKE) == -2
    need = L.dsa_probs_workspace_size(2, 3, 100, 0, 0)
    assert need > 0
    for kw in [dict(ws=None), dict(size=need - 1), dict(ws=TWO)]:
        assert call(**kw) == -3, kw
    more = L.dsa_probs_workspace_size(2, 3, 100, 5000, 4)
    assert more > need
    assert call(cap=5000, history=FAKE, nbias=4, bias_ids=FAKE, bias_values=FAKE, size=more - 1) == -3
    assert call() == -1 and call(p=AT + 600 * 4 - 4) == -1 and call(p=AT + 600 * 2 - 4, dtype=0) == -1  # p over the logits
    assert call(S=4097) == -2 and call(nbias=4097, bias_ids=FAKE, bias_values=FAKE) == -2
    for sizes in [(0, 1, 10, 0, 0), (1, 0, 10, 0, 0), (1, 1, 0, 0, 0), (1, 1, 1 << 24, 0, 0), (1 << 20, 1 << 20, 10, 0, 0),
                  (1, 1, 10, -1, 0), (1, 1, 10, 0, -1), (1, 4097, 10, 0, 0), (1, 1, 10, 1 << 28, 0), (1, 1, 10, 0, 4097)]:
        assert L.dsa_probs_workspace_size(*sizes) == 0


def test_binding_refuses_cpu_tensors():
    import torch
    plan = dsa.dsa_rope_init(64)
    bf = torch.bfloat16
    i32 = torch.int32
    with pytest.raises(ValueError):
        dsa.dsa_rope(torch.zeros(2, 1, 64, dtype=bf), torch.zeros(2, dtype=torch.int64), plan)
    with pytest.raises(ValueError):
        dsa.dsa_cache_append(torch.zeros(1, 576, dtype=bf), torch.zeros(512, dtype=bf), 1e-6, plan,
                             torch.zeros(1, 16, 576, dtype=bf), torch.zeros(1, 1, dtype=i32), torch.zeros(2, dtype=i32),
                             torch.zeros(1, dtype=i32))
    with pytest.raises(ValueError):
        dsa.dsa_paged_attn(torch.zeros(1, 16, 576, dtype=bf), torch.zeros(1, 16, 576, dtype=bf),
                           torch.zeros(1, 1, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(1, dtype=i32), 0.1,
                           ws=torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError):
        dsa.dsa_logits_probs(torch.zeros(1, 1, 32))


def test_rope_refuses_views_that_meet(L):
    """x and out as shifted views of one buffer, with the same strides (none of these calls may run)."""
    plan = dsa.dsa_rope_init(64)
    p = ctypes.addressof(plan)

    def call(shift, n=4, heads=2, dim=64, token=128, head=64):
        return L.dsa_rope(AT, FAKE, n, heads, dim, 0, p, 0, token, head, AT + 2 * shift, token, head, None)

    for shift in (1, 63, 64, 65, 128, 3 * 128 + 127, -1, -64, -(3 * 128 + 127)):
        assert call(shift) == -1, shift
    for shift in (63, 192, 192 + 63, 192 * 9 - 63, -(192 * 9 + 63), 192 * 3 + 65 - 2):  # heads of wider rows
        assert call(shift, n=10, heads=1, token=192, head=5) == -1, shift
    for shift in (64 * 5, 1000 - 63, 1000 + 64 * 9 + 63, -(1000 - 64)):                  # heads outermost
        assert call(shift, n=10, heads=2, token=64, head=1000) == -1, shift
    assert call(64, n=1, heads=3, token=7) == -1 and call(2 * 64, n=1, heads=3, token=7) == -1


def test_outputs_over_any_input_are_refused(L):
    far = lambda i: AT + (i << 24)  # noqa: E731
    names = ["q", "cache", "table", "cu", "ctx"]
    size = dict(q=4 * 16 * 1152, cache=8 * 64 * 1152, table=2 * 4 * 4, cu=3 * 4, ctx=2 * 4)
    out_size, lse_size = 4 * 16 * 1024, 4 * 16 * 4
    a = {k: far(i) for i, k in enumerate(names)}

    def attn(out, lse):
        return L.dsa_paged_attn(a["q"], a["cache"], a["table"], a["cu"], a["ctx"], 4, 2, 16, 8, 64, 4, 0.1, out, lse, FAKE,
                                1 << 40, None)

    for k in names:
        last = size[k] - size[k] % 16 - (16 if size[k] % 16 == 0 else 0)
        for out in (a[k], a[k] + last, a[k] - out_size + 16):
            assert attn(out, None) == -1, (k, out - a[k])
        for lse in (a[k], a[k] + size[k] - 4, a[k] - lse_size + 4):
            assert attn(far(9), lse) == -1, (k, lse - a[k])
    assert attn(far(9), far(9) + out_size - 4) == -1 and attn(far(9), far(9) - lse_size + 4) == -1

    # (sizes that take two passes, and so a workspace, on any device)
    B, S, V, cap, nb = 400, 3, 5000, 10, 4
    names = ["temperature", "repetition", "frequency", "presence", "history", "history_len", "prompt_len", "draft", "bias_ids",
             "bias_values", "mask"]
    size = dict.fromkeys(names, B * 4)
    size.update(history=B * cap * 4, draft=B * S * 4, bias_ids=B * nb * 4, bias_values=B * nb * 4, mask=B * S * 157 * 4)
    a = {k: far(2 * i + 2) for i, k in enumerate(names)}

    def probs(p, **kw):
        x = {**a, **kw}
        return L.dsa_logits_probs(far(40), 1, B, S, V, x["temperature"], x["repetition"], x["frequency"], x["presence"],
                                  x["history"], cap, x["history_len"], x["prompt_len"], x["draft"], x["bias_ids"],
                                  x["bias_values"], nb, x["mask"], p, FAKE, 1 << 40, None)

    for k in names:
        for p in (a[k], a[k] + size[k] - 4, a[k] - B * S * V * 4 + 4):
            assert probs(p) == -1, (k, p - a[k])


@pytest.mark.parametrize("ctx,lost", [(900, 1), (65499, 1), (65536, 1), (65536, -1), (65536, 128), (65536, -128), (262143, 128),
                                      (262143, -128)])
def test_marked_rows_show_what_is_lost_or_taken_twice(ctx, lost):
    """Planted mistakes: one row, or one key tile of 128, is left out or counts twice.  The bounds that
    equal logits over marked rows are held to see it, in the output and in the log-sum-exp."""
    import torch
    count = torch.bincount(torch.arange(ctx) // 128 % DV, minlength=DV).double()
    b_out, b_lse = marked_bounds(count / ctx, torch.tensor(ctx, dtype=torch.float64).log())
    wrong = count.clone()
    wrong[ctx // 2 // 128 % DV] -= lost
    assert bool(((wrong / wrong.sum() - count / ctx).abs() > b_out).any())
    assert abs(math.log(ctx - lost) - math.log(ctx)) > float(b_lse)


def test_logits_probs_workspace_refusals_on_any_machine(L):
    """Sizes that take two passes whatever the number of SMs, outputs apart from the logits."""
    B, S, V, cap, nb = 400, 3, 5000, 700, 4
    need, more = L.dsa_probs_workspace_size(B, S, V, 0, 0), L.dsa_probs_workspace_size(B, S, V, cap, nb)
    assert 0 < need < more

    def call(ws, size, lists):
        history, bias = (AT + (1 << 28), AT + (1 << 29)) if lists else (None, None)
        return L.dsa_logits_probs(AT, 1, B, S, V, None, None, None, None, history, cap if lists else 0, None, None, None, bias,
                                  bias, nb if lists else 0, None, AT + (1 << 26), ws, size, None)

    for lists, size in ((False, need), (True, more)):
        for ws, n in ((None, size), (AT, size - 1), (AT, 0), (AT + 16, size)):
            assert call(ws, n, lists) == -3
