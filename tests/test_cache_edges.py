"""The paged key/value cache at its edges: scores far below zero, keys hidden by
the bias, contexts cut between CTAs, and what the calls refuse or report."""

import numpy as np
import pytest
import torch

from tests.test_cache import Case, compare, i32, jg, sizes  # noqa: F401  (jg: the fixture)

gpu = pytest.mark.gpu

U = 2.0 ** -8  # half a bf16 step, relative


def status_of(jg, case, **kw):  # noqa: F811
    """(out, lse, status) of a call with a workspace of its own."""
    ws = torch.empty(max(256, jg.jgdpa_cache_fwd_workspace_bytes(case.heads, case.kv_heads, case.d, kw["max_q"])),
                     dtype=torch.uint8, device="cuda")
    out, lse = jg.jgdpa_cache_fwd(**kw, workspace=ws)
    return out, lse, jg.jgdpa_read_device_status(ws)


def seen(case, b):
    """Which of its tokens the new tokens of request b see, [new, length]."""
    lo, n, length = int(case.off[b]), int(case.new[b]), int(case.kv[b])
    ctx = length - n
    depth = np.arange(n) if case.depth is None else np.asarray(case.depth[lo:lo + n])
    sees = np.ones((n, length), bool)
    for t in range(n):
        for u in range(n):
            sees[t, ctx + u] = u <= t if case.mask is None else bool((int(case.mask[lo + t][u // 32]) >> (u % 32)) & 1)
    if case.window:
        pos = np.concatenate([np.arange(ctx), ctx + depth])
        sees &= np.abs((ctx + depth)[:, None] - pos) < case.window
    return sees


# ------------------------------------------------------------ small weights (GPU)
@gpu
@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("group,new,window", [(1, 1, 0), (4, 6, 0), (2, 20, 0), (2, 40, 90), (8, 40, 0)])
def test_scores_far_below_zero(jg, act, d, group, new, window):  # noqa: F811
    """A bias that pushes every score to -4 and below: the weights are small, and
    each is right relative to itself.  Roundings of an output, relative to
    sum |P||V| (u = 2^-8):
      P: u for its rounding to bf16, at most 2^-8 for the device's act, and the
        score's error times |act'/act|: at most |x| + 1/|x| + 1 <= 16 for the
        scores from -14 on (weights below that are 1e-30 of the others)
      O: 2^-12 for the fp32 sums, u for the final rounding"""
    rng = np.random.default_rng(new + d)
    c = Case(d + new, [700, 0, 130, 61], [new, new, 1, new], 4, group, d, 16, act, bias=33, window=window, mask=new > 1)
    c.bias = torch.from_numpy(rng.uniform(-9.0, -8.0, c.bias.shape).astype(np.float32))
    out, _ = jg.jgdpa_cache_fwd(**c.kwargs())
    want, _, size, dot, _ = c.oracle()
    # scores: fp32 sums of d products, the bias, the fused rounding
    score = d * 2.0 ** -23 * dot + 2.0 ** -19
    tol = size * (2 * U + 2.0 ** -12 + 16 * score.T[..., None])
    tol = tol + U * (np.abs(want) + tol)
    got = out.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= tol), f"worst {np.nanmax(np.abs(got - want) / (tol + 1e-300)):.1f} tolerances"


@gpu
@pytest.mark.parametrize("act,lo", [("gelu", -12.5), ("silu", -80.0)])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("kv_heads,group", [(256, 16), (32, 128)])
def test_one_weight(jg, act, lo, d, kv_heads, group):  # noqa: F811
    """One token that sees itself, q = 0, v = 1 and a bias of one entry per head:
    out = act(bias), rounded to bf16 as a weight and as an output (u each), the
    device's act within 2^-10 of itself, from where bf16 holds it on."""
    c = Case(0, [0], [1], kv_heads, group, d, 16, act, bias=1, nan=False)
    x = torch.linspace(lo, 16.0, c.heads - 2, dtype=torch.float32)
    c.bias = torch.cat([x, torch.zeros(2)])[:, None].contiguous()
    c.q.zero_()
    c.v.fill_(1.0)
    out, _ = jg.jgdpa_cache_fwd(**c.kwargs())
    y = c.bias.double()
    want = 0.5 * y * torch.erfc(-y * 0.5 ** 0.5) if act == "gelu" else y * torch.sigmoid(y)
    got = out[0].double().cpu()
    assert torch.all((got - want).abs() <= want.abs() * (2 * U + U * U + 2.0 ** -10))
    assert not out[0, -2:].any()


# ------------------------------------------------------------ reports (GPU)
@gpu
@pytest.mark.parametrize("act", ["gelu", "softmax"])
@pytest.mark.parametrize("d,kv_heads", [(32, 4), (64, 2), (128, 1)])
@pytest.mark.parametrize("most", [0, 1, 40])
def test_calls_without_rows_report_bad_offsets(jg, act, d, kv_heads, most):  # noqa: F811
    """max_q = 0, or a q without rows, where the offsets hold new tokens."""
    c = Case(1, [5, 40], [3, 2], kv_heads, 2, d, 16, act)
    kw = c.kwargs()
    out = torch.full_like(kw["q"], 7.0)
    if most == 0:  # rows, but no token allowed
        got, _, status = status_of(jg, c, **{**kw, "max_q": 0, "out": out})
        assert status == 6 and torch.all(got == 7.0)
    assert status_of(jg, c, **{**kw, "max_q": most, "q": kw["q"][:0]})[2] == 6
    none = {**kw, "max_q": most, "q_offsets": torch.zeros_like(kw["q_offsets"])}
    got, _, status = status_of(jg, c, **{**none, "out": out})
    assert status == 0 and torch.all(got == 7.0)  # padding rows alone
    assert status_of(jg, c, **{**none, "q": kw["q"][:0]})[2] == 0
    assert status_of(jg, c, **{**none, "q": kw["q"][:0], "kv_lens": i32([5, -1], "cuda")})[2] == 6


@gpu
@pytest.mark.parametrize("act", ["gelu", "softmax"])
@pytest.mark.parametrize("new,window", [(3, 0), (3, 50), (40, 0), (40, 50)])
@pytest.mark.parametrize("depth", [-1, -2 ** 31, 2 ** 31 - 70, 2 ** 31 - 1])
def test_depths_out_of_range_are_reported(jg, act, new, window, depth):  # noqa: F811
    """A negative depth, or one that leads beyond position 2^31 - 1: status
    BAD_OFFSETS, and the other request is as without it."""
    c = Case(13, [100, 30], [new, new], 2, 2, 64, 16, act, bias=33, window=window, mask=True, nan=False)
    kw = c.kwargs()
    good, good_lse, status = status_of(jg, c, **kw)
    assert status == 0
    depths = kw["depths"].clone()
    depths[1] = depth
    out, lse, status = status_of(jg, c, **{**kw, "depths": depths})
    assert status == 6
    n = int(c.off[1])
    assert torch.equal(out[n:], good[n:])
    if lse is not None:
        assert torch.equal(lse[:, n:], good_lse[:, n:])


@gpu
@pytest.mark.parametrize("act", ["gelu", "softmax"])
@pytest.mark.parametrize("new,window", [(3, 0), (3, 50), (40, 50)])
def test_the_largest_depths(jg, act, new, window):  # noqa: F811
    """Positions up to 2^31 - 1."""
    c = Case(14, [100, 30], [new, new], 2, 2, 64, 16, act, bias=33, window=window, mask=True)
    for b in range(2):
        lo, hi = int(c.off[b]), int(c.off[b + 1])
        top = 2 ** 31 - 1 - int(c.kv[b] - c.new[b])
        c.depth[lo + 1:hi] = top - np.arange(hi - lo - 1)[::-1]
    out, lse, status = status_of(jg, c, **c.kwargs())
    assert status == 0
    compare(c, out, lse)


# ------------------------------------------------------------ keys hidden by the bias (GPU)
@gpu
@pytest.mark.parametrize("d,kv_heads,new,group", [(32, 4, 3, 1), (32, 3, 20, 1), (64, 2, 1, 4), (64, 2, 12, 2), (128, 2, 1, 2),
                                                  (32, 4, 40, 1), (64, 2, 30, 4), (128, 2, 70, 2)])
@pytest.mark.parametrize("room", [0, 1 << 16])
@pytest.mark.parametrize("where", ["far", "near", "one head"])
def test_keys_hidden_by_the_bias_hold_anything(jg, d, kv_heads, new, group, room, where):  # noqa: F811
    """Softmax with bias entries of -inf: NaN and infinities in keys and values
    that they hide change nothing."""
    c = Case(19, [900, 0, 300, 64], [new] * 4, kv_heads, group, d, 32, "softmax", bias=257, mask=new > 1)
    kw = c.kwargs(room=room)
    bias = kw["bias_table"]
    # distances to hide (the index is distance + 128, the last entry all from 128 on)
    hide = {"far": slice(128 + 100, None), "near": slice(128 + 70, 128 + 90), "one head": slice(128 + 100, None)}[where]
    heads = slice(0, group) if where == "one head" else slice(None)  # the query heads of key/value head 0
    bias[heads, hide] = -float("inf")
    clean, clean_lse = jg.jgdpa_cache_fwd(**kw)
    # key j of request 0 is 900 + depth - j away from its tokens: hidden from all of them
    top = 0 if c.depth is None else int(np.max(c.depth[:new]))
    keys = range(900 - 90 + top + 1, 900 - 70) if where == "near" else range(0, 900 - 100 + 1)
    kv = slice(0, 1) if where == "one head" else slice(None)
    assert len(keys) > 0 and top < 19
    for value in (float("nan"), float("inf"), -float("inf")):
        k, v = kw["k_cache"].clone(), kw["v_cache"].clone()
        for j in list(keys)[::5]:
            page, at = int(c.table[0, j // 32]), j % 32
            v[page, at, kv] = value
            if j % 2:
                k[page, at, kv, 3] = value
        out, lse = jg.jgdpa_cache_fwd(**{**kw, "k_cache": k, "v_cache": v})
        assert torch.equal(out, clean) and torch.equal(lse, clean_lse)


@gpu
@pytest.mark.parametrize("d,kv_heads,new,group", [(32, 4, 3, 1), (64, 2, 12, 2), (128, 2, 1, 2), (64, 2, 40, 2), (128, 2, 70, 2)])
@pytest.mark.parametrize("value", [torch.finfo(torch.float32).min, torch.finfo(torch.float32).max])
def test_biases_of_the_largest_finite_size(jg, d, kv_heads, new, group, value):  # noqa: F811
    """Softmax whose every score is the lowest (or highest) fp32: the scores
    are lost beside it, so that all seen keys weigh the same, and the LSE is
    that value."""
    c = Case(27, [900, 0, 300, 64], [new] * 4, kv_heads, group, d, 32, "softmax", bias=257, mask=new > 1)
    c.bias[:] = value
    out, lse = jg.jgdpa_cache_fwd(**c.kwargs())
    want, want_lse, size, _, _ = c.oracle()
    # weights 1 / n: 2^-12 for fp32 sums, u for O (a weight of 1 is exact in bf16)
    got = out.double().cpu().numpy()
    tol = size * 2.0 ** -12
    tol = tol + U * (np.abs(want) + tol)
    assert np.all(np.abs(got - want) <= tol)
    assert np.all(np.abs(lse.double().cpu().numpy() / want_lse - 1) <= 2.0 ** -22)


# ------------------------------------------------------------ refusals (CPU)
@pytest.mark.parametrize("field,value", [("max_q", 2 ** 32 + 4), ("window", 2 ** 32 + 5), ("max_q", 2 ** 31), ("window", -2 ** 32)])
def test_attention_refuses_numbers_beyond_32_bits(jg, field, value):  # noqa: F811
    """They would reach the library as other numbers."""
    kw = Case(0, [40, 20], [3, 4], 2, 2, 64, 16).kwargs("cpu")
    kw[field] = value
    with pytest.raises(ValueError, match=f"{field} must fit in 32 bits"):
        jg.jgdpa_cache_fwd(**kw)


@pytest.mark.parametrize("field,value", [("page_size", 2 ** 32 + 16), ("total_new", 2 ** 32 + 1), ("total_new", 2 ** 31)])
def test_plan_refuses_numbers_beyond_32_bits(jg, field, value):  # noqa: F811
    kw = dict(ctx_lens=i32([1]), new_lens=i32([1]), held_pages=i32([0]), block_table=i32([[0]]), free_pages=i32([0]),
              free_count=i32([1]), page_size=16, total_new=1)
    kw[field] = value
    with pytest.raises(ValueError, match=f"{field} must fit in 32 bits"):
        jg.jgdpa_cache_plan(**kw)


# ------------------------------------------------------------ calls that follow one another (GPU)
@gpu
@pytest.mark.parametrize("d,new,group", [(32, 2, 2), (64, 3, 4), (128, 1, 8), (128, 40, 2)])
def test_outputs_as_the_next_queries(jg, d, new, group):  # noqa: F811
    """Attention calls back to back, each on the rows that the one before wrote,
    into two buffers in turn."""
    rng = np.random.default_rng(d)
    batch = 24
    c = Case(51, sizes(rng, batch, 900), np.full(batch, new), 2, group, d, 16, "softmax", nan=False)
    kw = c.kwargs()
    kw["k_cache"] = kw["k_cache"] * 4  # so that the rows stay apart from one another
    steps = 30

    def chain(wait):
        buffers = [kw["q"].clone(), torch.full_like(kw["q"], float("nan"))]
        torch.cuda.synchronize()
        for i in range(steps):
            jg.jgdpa_cache_fwd(**{**kw, "q": buffers[i % 2], "out": buffers[(i + 1) % 2]})
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return [b.clone() for b in buffers]

    want = chain(True)
    for _ in range(10):
        for a, b in zip(chain(False), want):
            assert torch.equal(a, b)


# ------------------------------------------------------------ nothing is lost (GPU)
@gpu
@pytest.mark.parametrize("act", ["gelu", "softmax"])
@pytest.mark.parametrize("d,kv_heads,new,group,length", [(32, 1, 16, 1, 6000), (32, 4, 4, 4, 6000), (64, 1, 3, 5, 20000),
                                                         (64, 1, 8, 4, 9000), (64, 2, 4, 4, 9000), (128, 1, 4, 4, 20000),
                                                         (32, 1, 40, 2, 6000), (64, 1, 64, 2, 9000), (128, 1, 25, 5, 6000),
                                                         (64, 1, 50, 5, 9000), (128, 1, 64, 8, 6000)])
def test_every_block_of_a_long_context_counts(jg, act, d, kv_heads, new, group, length):  # noqa: F811
    """Each query row looks for one key, which takes (nearly) all the weight; over
    the calls, one key in each 16 of a long context that is cut between CTAs.
    Keys are +-1, so a row's own key scores c d (c = 64 / d a unit of scale), any
    other a sum of d random signs.  The reference is in 64 bits; the bound, the
    usual roundings (see `compare` in test_cache.py), is a few hundredths of the
    weight that a lost key would take away."""
    rng = np.random.default_rng(length + d)
    page, heads = 64, kv_heads * group
    c = Case(2, [length - new, 40], [new, 1], kv_heads, group, d, page, act, nan=False)
    kw = c.kwargs()
    sign = torch.from_numpy(rng.choice([-1.0, 1.0], size=tuple(kw["k_cache"].shape))).to(torch.bfloat16).cuda()
    kw["k_cache"] = sign
    kw["scale"] = 64.0 / d
    if act == "gelu":
        kw["bias_table"] = torch.full((heads, 3), -60.0, device="cuda")  # the own key scores 4, another at most 0 (d = 32)
    ids = torch.from_numpy(c.table[0, :-(-length // page)]).cuda().long()
    k, v = (kw[x][ids].flatten(0, 1)[:length].double() for x in ("k_cache", "v_cache"))
    blocks = -(-(length - new) // 16)
    rows = new * group
    for first in range(0, blocks, rows):
        block = torch.arange(first, first + rows) % blocks
        target = torch.minimum(block * 16 + torch.from_numpy(rng.integers(0, 16, rows)), torch.tensor(length - new - 1))
        target = target.view(new, group).cuda()
        q = kw["q"].clone()
        for h in range(kv_heads):
            q[:new, h * group:(h + 1) * group] = k[target.view(-1), h].view(new, group, d).to(torch.bfloat16)
        out, lse = jg.jgdpa_cache_fwd(**{**kw, "q": q})
        ahead = torch.arange(length, device="cuda")[None] > length - new + torch.arange(new, device="cuda")[:, None]
        for h in range(heads):
            x = q[:new, h].double() @ k[:, h // group].t() * kw["scale"]
            if act == "gelu":
                x = x - 60.0
                p = (0.5 * x * torch.erfc(-x * 0.5 ** 0.5)).masked_fill(ahead, 0.0)
            else:
                p = torch.softmax(x.masked_fill(ahead, -torch.inf), 1)
            own = p.gather(1, target[:, h % group, None])
            assert torch.all(own > (0.9 if act == "softmax" else 3.5))
            want, size = p @ v[:, h // group], p.abs() @ v[:, h // group].abs()
            # scores are exact (sums of d signs times a power of two, less 60); the device's act: 2^-8
            tol = size * (2 * U + 2.0 ** -12)
            tol = tol + U * (want.abs() + tol)
            got = out[:new, h].double()
            assert torch.all((got - want).abs() <= tol), (first, h)
            # the row without its key would be out of the bound in most columns
            without = want - own * v[target[:, h % group], h // group]
            assert torch.all(((without - want).abs() > tol).double().mean(1) > 0.8)


@gpu
@pytest.mark.parametrize("act", ["gelu", "softmax"])
@pytest.mark.parametrize("d,kv_heads,new,group", [(32, 4, 4, 2), (64, 2, 8, 4), (128, 1, 4, 4), (32, 1, 40, 1), (64, 1, 30, 3),
                                                  (128, 1, 24, 3), (64, 1, 50, 5), (128, 2, 60, 4)])
@pytest.mark.parametrize("window", [0, 3000])
def test_infinities_in_requests_cut_between_ctas(jg, act, d, kv_heads, new, group, window):  # noqa: F811
    """NaN and infinities in V of drafted tokens and of context tokens at the
    window's edge, of a request whose keys many CTAs share: the rows that see
    them are not finite in that column, and the others keep their bits."""
    c = Case(43, [5000, 40], [new, new], kv_heads, group, d, 16, act, window=window, mask=True, nan=False)
    kw = c.kwargs()
    clean, clean_lse = jg.jgdpa_cache_fwd(**kw)
    assert torch.isfinite(clean).all()
    sees = seen(c, 0)
    keys = [5000, 5000 + new // 2, 5000 + new - 1] + ([5000 - window + 1, 5000 - window + 2] if window else [])
    for i, j in enumerate(keys):
        head, col = i % kv_heads, (7 * i + 3) % d
        v = kw["v_cache"].clone()
        v[int(c.table[0, j // 16]), j % 16, head, col] = (float("inf"), float("nan"), -float("inf"))[i % 3]
        out, lse = jg.jgdpa_cache_fwd(**{**kw, "v_cache": v})
        rows = torch.from_numpy(np.nonzero(sees[:, j])[0]).cuda()
        same = torch.ones_like(out, dtype=torch.bool)
        for h in range(head * group, (head + 1) * group):
            same[rows, h, col] = False
            assert not torch.isfinite(out[rows, h, col]).any()
        assert torch.equal(out[same], clean[same])
        assert lse is None or torch.equal(lse, clean_lse)


@gpu
@pytest.mark.parametrize("act", ["silu", "softmax"])
@pytest.mark.parametrize("d,new,group", [(32, 40, 1), (64, 12, 4), (128, 10, 4), (128, 40, 5)])
def test_infinities_in_many_requests_per_cta(jg, act, d, new, group):  # noqa: F811
    """Requests by the thousand, so that each CTA walks far more than 16 parts,
    some of which hold infinities in V of a drafted token."""
    rng = np.random.default_rng(d + new)
    kinds = 6
    c = Case(47, rng.integers(1, 300, kinds), np.full(kinds, new), 2, group, d, 16, act, mask=True, nan=False)
    kw = c.kwargs()
    order = np.concatenate([np.arange(kinds)] * 2 + [rng.integers(0, kinds, 3000)])
    rows = torch.from_numpy(np.concatenate([np.arange(c.off[b], c.off[b + 1]) for b in order])).cuda()
    many = {**kw, "q_offsets": i32(np.arange(len(order) + 1) * new, "cuda"), "kv_lens": i32(c.kv[order], "cuda"),
            "block_table": kw["block_table"][torch.from_numpy(order).cuda()].contiguous()}
    for k in ("q", "tree_mask", "depths"):
        many[k] = kw[k][rows].contiguous()
    v = kw["v_cache"].clone()
    odd = torch.zeros(c.q.shape[0], c.heads, d, dtype=torch.bool, device="cuda")
    for b, u in ((1, 0), (4, new // 2)):
        j = int(c.kv[b]) - new + u
        v[int(c.table[b, j // 16]), j % 16, 1, 5] = float("inf")
        hit = torch.from_numpy(np.nonzero(seen(c, b)[:, j])[0]).cuda() + int(c.off[b])
        for h in range(group, 2 * group):
            odd[hit, h, 5] = True
    clean = jg.jgdpa_cache_fwd(**many)[0]
    out = jg.jgdpa_cache_fwd(**{**many, "v_cache": v})[0]
    assert torch.isfinite(clean).all()
    odd = odd[rows]
    assert not torch.isfinite(out[odd]).any()
    assert torch.equal(out[~odd], clean[~odd])


# ------------------------------------------------------------ waits, and plans of nothing (GPU)
@gpu
@pytest.mark.parametrize("d,new,group,act", [(128, 1, 4, "softmax"), (64, 1, 1, "softmax"), (32, 1, 2, "gelu"),
                                             (128, 30, 2, "gelu"), (64, 60, 8, "softmax"), (32, 40, 1, "silu")])
def test_waits_that_run_out_are_reported(jg, d, new, group, act):  # noqa: F811
    """Under a limit of 1 ns the waits of a batch that keeps every SM waiting for
    its loads run out, in the kernel for few rows and in the 128-row one, and
    the next call is as before.  (A wait looks at its clock only after a
    suspended test returns, so that a single call may end without noticing.)"""
    rng = np.random.default_rng(d)
    batch, pages, kv_heads = 64, 96, 4
    c = Case(3, [1], [1], kv_heads, group, d, 64, act, nan=False)
    g = torch.Generator("cuda").manual_seed(d)
    k, v = (torch.randn(batch * pages, 64, kv_heads, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    kw = dict(q=torch.randn(batch * new, c.heads, d, generator=g, device="cuda").to(torch.bfloat16), k_cache=k, v_cache=v,
              block_table=i32(rng.permutation(batch * pages).reshape(batch, pages), "cuda"),
              q_offsets=i32(np.arange(batch + 1) * new, "cuda"), kv_lens=i32(np.full(batch, pages * 64), "cuda"), act=act,
              scale=c.scale, max_q=new)
    good, _, status = status_of(jg, c, **kw)
    assert status == 0
    jg.jgdpa_set_wait_limit_ns(1)
    try:
        reports = {status_of(jg, c, **kw)[2] for _ in range(20)}
    finally:
        jg.jgdpa_set_wait_limit_ns(0)
    assert 7 in reports and reports <= {0, 7}
    out, _, status = status_of(jg, c, **kw)
    assert status == 0 and torch.equal(out, good)


@gpu
def test_plan_of_no_requests(jg):  # noqa: F811
    """Every row of slots is one behind the last token; the pool stays as it is."""
    free, none = i32([3, 1, -1], "cuda"), i32([], "cuda")
    slots, off, kv, held, count = jg.jgdpa_cache_plan(none, none, none, i32(np.zeros((0, 4)), "cuda"), free, i32([2], "cuda"), 16, 5)
    assert slots.tolist() == [-1] * 5 and off.tolist() == [0] and count.tolist() == [2] and free.tolist() == [3, 1, -1]
    assert kv.numel() == 0 and held.numel() == 0
