"""The paged key/value cache: page plans, writes, attention over the pages."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import cache as oracle

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def jg():
    from jagged_gdpa_gb300 import build as b
    b.build()
    import jagged_gdpa_gb300 as m
    return m


def i32(x, device="cpu"):
    return torch.tensor(np.asarray(x, dtype=np.int64).astype(np.int32), device=device)


# ------------------------------------------------------------ inputs
def tree(rng, new, words):
    """Ancestor masks and depths of random trees of drafted tokens."""
    masks, depths = [], []
    for n in new:
        seen, depth = [], []
        for t in range(n):
            up = int(rng.integers(-1, t)) if t else -1
            seen.append((seen[up] if up >= 0 else 0) | 1 << t)
            depth.append(depth[up] + 1 if up >= 0 else 0)
        masks += [[(s >> 32 * w) & 0xFFFFFFFF for w in range(words)] for s in seen]
        depths += depth
    return np.array(masks, dtype=np.int64).reshape(-1, words), np.array(depths, dtype=np.int64)


class Case:
    """A batch on the CPU: bf16 values held as fp64 arrays for the oracle."""

    def __init__(self, seed, ctx, new, kv_heads, group, d, page, act="softmax", bias=0, window=0, mask=False,
                 extra=0, nan=True, spare=2):
        rng = np.random.default_rng(seed)
        self.act, self.window, self.d, self.page = act, window, d, page
        self.heads, self.kv_heads, self.scale = kv_heads * group, kv_heads, d ** -0.5
        ctx, new = np.asarray(ctx), np.asarray(new)
        self.new, self.kv = new, ctx + new
        self.off = np.concatenate([[0], np.cumsum(new)])
        need = -(-self.kv // page)
        self.pages = int(need.sum()) + spare
        self.table = np.full((len(ctx), max(1, int(need.max()))), 2 ** 31 - 7)  # entries of no token: no page
        ids = rng.permutation(self.pages)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        total = int(self.off[-1]) + extra

        def normal(*shape):
            return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32)).to(torch.bfloat16)

        self.q = normal(total, self.heads, d)
        self.k, self.v = normal(self.pages, page, kv_heads, d), normal(self.pages, page, kv_heads, d)
        if nan:  # places that hold no token hold anything
            live = torch.zeros(self.pages, page, dtype=torch.bool)
            for b, n in enumerate(self.kv):
                for j in range(n):
                    live[self.table[b, j // page], j % page] = True
            self.k[~live] = float("nan")
            self.v[~live] = float("nan")
        self.bias = torch.from_numpy((0.5 * rng.standard_normal((self.heads, bias))).astype(np.float32)) if bias else None
        words = -(-int(max(1, new.max())) // 32)
        self.mask, self.depth = tree(rng, new, words) if mask else (None, None)
        if mask and extra:
            self.mask = np.concatenate([self.mask, np.zeros((extra, words), np.int64)])
            self.depth = np.concatenate([self.depth, np.zeros(extra, np.int64)])

    def oracle(self):
        f = lambda t: t.double().numpy()  # noqa: E731
        return oracle.attend(f(self.q), f(self.k), f(self.v), self.table, self.off, self.kv, self.act, self.scale,
                             None if self.bias is None else f(self.bias), self.window, self.mask, self.depth)

    def kwargs(self, device="cuda", room=0):
        """room: columns of the table beyond the longest request's pages."""
        mask = None if self.mask is None else torch.from_numpy(self.mask.astype(np.uint32).view(np.int32)).to(device)
        return dict(q=self.q.to(device), k_cache=self.k.to(device), v_cache=self.v.to(device),
                    block_table=i32(np.pad(self.table, ((0, 0), (0, room)), constant_values=-3), device), q_offsets=i32(self.off, device),
                    kv_lens=i32(self.kv, device), act=self.act, scale=self.scale,
                    max_q=int(max(1, self.new.max())), bias_table=None if self.bias is None else self.bias.to(device),
                    window=self.window, tree_mask=mask, depths=None if self.depth is None else i32(self.depth, device))


def compare(case, out, lse, want=None):
    """Every element within the roundings on its way (u = 2^-8, half a bf16 step):
      scores: fp32 sums of d products in the tensor core, at most d 2^-23 of
        sum |q||k| scale, plus a few fp32 roundings of the score and the bias
      P: that score error (times |act'| <= 1.13, or times P for softmax), u for
        its rounding to bf16, and for GELU / SiLU the device's evaluation of
        act, within 1.2e-3 of the exact one (tests/test_act.py)
      O: fp32 sums (absorbed in 2^-12 of sum |P||V|), u for the final rounding"""
    o, ls, size, dot, vsum = want if want is not None else case.oracle()
    u = 2.0 ** -8
    n = case.off[-1]
    got = out.double().cpu().numpy()[:n]
    o, size, vsum, dot = o[:n], size[:n], vsum[:n], dot[:, :n]
    es = case.d * 2.0 ** -23 * dot + 2.0 ** -20
    if case.act == "softmax":
        tol = size * (u + 2.0 ** -12 + 2 * es.T[..., None])
        le = lse.double().cpu().numpy()[:, :n]
        assert np.array_equal(np.isneginf(le), np.isneginf(ls[:, :n]))
        fin = np.isfinite(ls[:, :n])
        assert np.all(np.abs(le - ls[:, :n])[fin] <= (es + 2.0 ** -20 * np.abs(ls[:, :n]))[fin])
    else:
        tol = size * (u + 2.0 ** -12) + vsum * (1.13 * es.T[..., None] + 1.2e-3)
        assert lse is None
    tol = tol + u * (np.abs(o) + tol)
    bad = ~(np.abs(got - o) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} elements, worst {np.nanmax(np.abs(got - o) / (tol + 1e-30)):.2f} tolerances"


def sizes(rng, batch, hi):
    return np.minimum(hi, np.round(np.exp(rng.uniform(0, np.log(hi + 1), batch)))).astype(np.int64)


# ------------------------------------------------------------ refusals (CPU)
def _fwd_args(**kw):
    a = dict(q=1 << 20, qs=512, k=1 << 20, v=1 << 20, kps=16 * 4 * 64, vps=16 * 4 * 64, pages=8, page=16, table=1 << 20,
             width=4, off=1 << 20, kv=1 << 20, batch=1, total=4, max_q=4, heads=8, kv_heads=4, d=64, act=2, scale=0.125,
             bias=None, blen=0, window=0, mask=None, words=0, depth=None, out=1 << 20, lse=1 << 20, ws=1 << 20,
             wsb=1 << 30, stream=None)
    a.update(kw)
    a["scale"] = ctypes.c_float(a["scale"])
    return list(a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(d=48, kps=16 * 4 * 48), 2), (dict(page=24), 2), (dict(page=8), 2), (dict(page=2048, kps=1 << 30, vps=1 << 30), 2),
    (dict(pages=0), 1), (dict(pages=1 << 28), 2), (dict(kps=16 * 4 * 64 - 8), 1), (dict(vps=16 * 4 * 64 + 4), 3),
    (dict(k=(1 << 20) + 8), 3), (dict(k=None), 1), (dict(kv_heads=3, kps=1 << 20, vps=1 << 20), 1), (dict(kv_heads=0), 1),
    (dict(act=3), 1), (dict(scale=float("inf")), 1), (dict(blen=4, bias=1 << 20), 1), (dict(blen=5), 1),
    (dict(blen=8191, bias=1 << 20), 2), (dict(window=-1), 1), (dict(words=1), 1), (dict(mask=1 << 20), 1),
    (dict(act=0), 1), (dict(batch=16385), 2), (dict(off=None), 1), (dict(q=None), 1), (dict(qs=504), 1),
    (dict(qs=516), 3), (dict(q=(1 << 20) + 2), 3), (dict(out=(1 << 20) + 8), 3), (dict(batch=-1), 1), (dict(max_q=-1), 1),
    (dict(width=1 << 28), 2),
])
def test_fwd_rejects_bad_arguments_without_a_launch(jg, kw, code):
    assert jg.load().jgdpa_cache_fwd(*_fwd_args(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(k=None), 1), (dict(slots=None), 1), (dict(ks=248), 1), (dict(ks=260), 3),
    (dict(k=(1 << 20) + 8), 3), (dict(d=16), 2), (dict(page=12), 2), (dict(pages=0), 1), (dict(kps=16), 1),
])
def test_append_rejects_bad_arguments_without_a_launch(jg, kw, code):
    a = dict(k=1 << 20, v=1 << 20, ks=256, vs=256, slots=1 << 20, rows=3, kc=1 << 20, vc=1 << 20, kps=16 * 256,
             vps=16 * 256, pages=4, page=16, heads=4, d=64, stream=None)
    a.update(kw)
    assert jg.load().jgdpa_cache_append(*a.values()) == code


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), 1), (dict(batch=16385), 2), (dict(page=10), 2), (dict(total=-1), 1), (dict(count=None), 1),
    (dict(ctx=None), 1), (dict(slots=None), 1), (dict(pages=1 << 28), 2), (dict(width=1 << 28), 2),
    (dict(held_out=3 << 20), 1), (dict(count_out=6 << 20), 1), (dict(wsb=16), 4), (dict(ctx=(1 << 20) + 2), 3),
])
def test_plan_rejects_bad_arguments_without_a_launch(jg, kw, code):
    a = dict(ctx=1 << 20, new=2 << 20, held=3 << 20, batch=2, page=16, table=4 << 20, width=8, free=5 << 20, pages=64,
             count=6 << 20, total=10, held_out=7 << 20, count_out=8 << 20, off=9 << 20, kv=10 << 20, slots=11 << 20,
             ws=12 << 20, wsb=256, stream=None)
    a.update(kw)
    assert jg.load().jgdpa_cache_plan(*a.values()) == code


def test_workspace_query(jg):
    assert jg.jgdpa_cache_fwd_workspace_bytes(8, 3, 64, 1) == 0
    assert jg.jgdpa_cache_fwd_workspace_bytes(8, 4, 48, 1) == 0


@pytest.mark.parametrize("field,change,match", [
    ("q", lambda t: t.float(), "q must have dtype"),
    ("q", lambda t: t[:, :, :32], "q must have shape"),
    ("q", lambda t: t.transpose(0, 1).contiguous().transpose(0, 1), "contiguous inside"),
    ("k_cache", lambda t: t[0], "k_cache must be"),
    ("v_cache", lambda t: t[:-1], "v_cache must have shape"),
    ("k_cache", lambda t: t.transpose(1, 2).contiguous().transpose(1, 2), "contiguous inside"),
    ("v_cache", lambda t: t[:1].expand(t.shape), "must not overlap"),
    ("block_table", lambda t: t.long(), "block_table must have dtype"),
    ("block_table", lambda t: t[:1], "block_table must have shape"),
    ("block_table", lambda t: t.t().contiguous().t(), "block_table must be contiguous"),
    ("q_offsets", lambda t: t[:-1], "q_offsets must have shape"),
    ("tree_mask", lambda t: t[:-1], "tree_mask must have shape"),
    ("depths", lambda t: t.long(), "depths must have dtype"),
    ("bias_table", lambda t: t[:-1], "bias_table must have shape"),
    ("q", lambda t: t, "CUDA device"),
])
def test_wrapper_rejects_bad_tensors(jg, field, change, match):
    kw = Case(0, [40, 20], [3, 4], 2, 2, 64, 16, bias=5, mask=True, spare=3).kwargs("cpu")
    kw[field] = change(kw[field])
    with pytest.raises(ValueError, match=match):
        jg.jgdpa_cache_fwd(**kw)


@pytest.mark.parametrize("field", ["tree_mask", "bias_table"])
def test_wrapper_rejects_tables_without_columns(jg, field):
    """They would reach the library as no mask, or no bias."""
    kw = Case(0, [40, 20], [3, 4], 2, 2, 64, 16, bias=5, mask=True).kwargs("cpu")
    kw[field] = kw[field][:, :0]
    with pytest.raises(ValueError, match=f"{field} must have columns"):
        jg.jgdpa_cache_fwd(**kw)


def test_wrappers_reject_other_bad_calls(jg):
    c = Case(0, [40], [3], 2, 2, 64, 16)
    kw = c.kwargs("cpu")
    with pytest.raises(ValueError, match="softmax mode only"):
        jg.jgdpa_cache_fwd(**{**kw, "act": "gelu"}, lse=torch.zeros(4, 3))
    with pytest.raises(ValueError, match="workspace must have dtype"):
        jg.jgdpa_cache_fwd(**kw, workspace=torch.zeros(4096))
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="slots must have shape"):
        jg.jgdpa_cache_append(k, k, i32([0, 1]), c.k, c.v)
    with pytest.raises(ValueError, match="v_new must have shape"):
        jg.jgdpa_cache_append(k, k[:2], i32([0, 1, 2]), c.k, c.v)
    with pytest.raises(ValueError, match="held_pages must have shape"):
        jg.jgdpa_cache_plan(i32([1]), i32([1]), i32([1, 2]), i32([[0]]), i32([0]), i32([0]), 16, 1)


def test_oracle_plan_by_hand():
    got = oracle.plan([20, 0], [13, 40], [2, 0], [[5, 6, -1], [-1, -1, -1]], [9, 8, 7, 4] + [-1] * 6, 4, 16, 55)
    slots, off, kv, held, count, table, free = got
    assert table == [[5, 6, 4], [7, 8, 9]] and held == [3, 3] and count == 0 and kv == [33, 40]
    assert slots[:13] == [6 * 16 + 4 + i for i in range(12)] + [4 * 16] and slots[-2:] == [-1, -1]
    # pages given back go out again first, the last one given back before the others
    got = oracle.plan([0, 16], [0, 20], [2, 1], [[5, 6, -1], [7, -1, -1]], [9] + [-1] * 9, 1, 16, 20)
    assert got[5] == [[5, 6, -1], [7, 6, 5]] and got[4] == 1 and got[6] == [9] + [-1] * 9


# ------------------------------------------------------------ plan (GPU)
def random_plan(seed, batch, page, width, most, ended=0.3):
    rng = np.random.default_rng(seed)
    new = rng.integers(0, most + 1, batch)
    ctx = np.array([int(rng.integers(0, width * page - n + 1)) for n in new])
    held = np.minimum(width, -(-ctx // page) + rng.integers(0, 3, batch))
    held = np.where(rng.random(batch) < 0.2, 0, held)
    gone = rng.random(batch) < ended
    ctx, new = np.where(gone, 0, ctx), np.where(gone, 0, new)
    want = -(-(ctx + new) // page)
    pool = int(held.sum() + np.maximum(0, want - held).sum()) + 3
    ids = rng.permutation(pool)
    table = np.full((batch, width), -1)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = ids[at:at + h]
        at += h
    free = np.full(pool, -2)
    free[:pool - at] = ids[at:]
    return ctx, new, held, table, free, pool - at


def check_plan(jg, ctx, new, held, table, free, count, page, total, stream=None):
    d = [i32(x, "cuda") for x in (ctx, new, held, table, free, [count])]
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    want = oracle.plan(*(np.asarray(x).tolist() for x in (ctx, new, held, table, free)), count, page, total)
    for _ in range(2):  # the same inputs again: the same values
        got = jg.jgdpa_cache_plan(*d, page, total, workspace=ws)
        status = jg.jgdpa_read_device_status(ws)
        if isinstance(want, int):
            assert status == want
            exp = ([-1] * total, [0] * (len(ctx) + 1), ctx, held, count, table, free)
        else:
            assert status == 0
            exp = want
        for name, g, e in zip(("slots", "q_offsets", "kv_lens", "held", "count", "table", "free"),
                              (*got, d[3], d[4]), exp):
            assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(e).reshape(-1)), name


@gpu
@pytest.mark.parametrize("seed,batch,page,width,most,extra", [
    (0, 1, 16, 1, 1, 0), (1, 1, 16, 300, 2000, 0), (2, 7, 32, 9, 64, 5), (3, 300, 16, 40, 70, 0), (4, 64, 128, 70, 8000, 77),
    (5, 257, 1024, 3, 5, 1), (6, 2049, 16, 5, 3, 0), (7, 33, 64, 12, 0, 3),
])
def test_plan(jg, seed, batch, page, width, most, extra):
    ctx, new, held, table, free, count = random_plan(seed, batch, page, width, most)
    check_plan(jg, ctx, new, held, table, free, count, page, int(new.sum()) + extra)


@gpu
def test_plan_of_the_most_requests(jg):
    batch = 16384
    ctx, new, held, table, free, count = random_plan(11, batch, 16, 4, 9)
    check_plan(jg, ctx, new, held, table, free, count, 16, int(new.sum()))


@gpu
def test_plan_edges(jg):
    one = [[0, 1, -1, -1]]
    check_plan(jg, [32], [0], [2], one, [3, 2], 2, 16, 0)          # nothing to do
    check_plan(jg, [0], [0], [2], one, [3, 2, -1, -1], 2, 16, 0)   # ended: all pages back
    check_plan(jg, [33], [31], [2], one, [3, 2], 2, 16, 31)        # the last free page
    check_plan(jg, [33], [32], [2], [[0, 1, -1, -1, -1]], [3, 2], 2, 16, 32)  # one more than there is
    check_plan(jg, [60], [5], [2], one, [3, 2], 2, 16, 5)          # more than the table row holds
    check_plan(jg, [-1], [5], [2], one, [3, 2], 2, 16, 5)
    check_plan(jg, [20], [-5], [2], one, [3, 2], 2, 16, 5)
    check_plan(jg, [20], [5], [9], one, [3, 2], 2, 16, 5)
    check_plan(jg, [20], [5], [2], one, [3, 2], 2, 16, 4)          # too few rows for the slots
    check_plan(jg, [0], [0], [2], one, [3, 2], 2, 16, 0)           # more pages than the pool's stack holds
    check_plan(jg, [20], [5], [2], one, [3, 2], 3, 16, 5)          # a count beyond the stack
    check_plan(jg, [20], [30], [2], [[0, 77, -1, -1]], [3, 99], 2, 16, 30)  # ids outside the pool: no slots
    check_plan(jg, [2 ** 31 - 1], [2 ** 31 - 1], [2], one, [3, 2], 2, 16, 5)


# ------------------------------------------------------------ append (GPU)
@gpu
@pytest.mark.parametrize("rows,heads,d,page", [(1, 1, 32, 16), (3, 1, 64, 32), (17, 5, 64, 16), (100, 8, 128, 64),
                                               (33, 40, 128, 16), (5, 3, 32, 1024)])
def test_append(jg, rows, heads, d, page):
    g = torch.Generator().manual_seed(rows)
    pages = -(-rows // page) + 3
    wide = torch.randn(rows, 3, heads, d, generator=g).to(torch.bfloat16).cuda()
    pool = torch.randn(pages, 2, page, heads, d, generator=g).to(torch.bfloat16).cuda()
    slots = torch.randperm(pages * page, generator=g)[:rows].int()
    slots[::3] = torch.where(torch.arange(len(slots[::3])) % 2 == 0, -1, pages * page).int()
    slots = slots.cuda()
    kc, vc = pool[:, 0], pool[:, 1]  # pages of one pool, keys beside values
    want = pool.clone()
    for r, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            want[s // page, 0, s % page] = wide[r, 1]
            want[s // page, 1, s % page] = wide[r, 2]
    jg.jgdpa_cache_append(wide[:, 1], wide[:, 2], slots, kc, vc)
    assert torch.equal(pool.view(torch.int16), want.view(torch.int16))


@gpu
def test_append_of_nothing(jg):
    c = torch.zeros(2, 16, 1, 32, dtype=torch.bfloat16, device="cuda")
    e = torch.zeros(0, 1, 32, dtype=torch.bfloat16, device="cuda")
    jg.jgdpa_cache_append(e, e, i32([], "cuda"), c, c.clone())
    assert not c.any()


# ------------------------------------------------------------ attention (GPU)
@gpu
@pytest.mark.parametrize("act", ["gelu", "silu", "softmax"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("group,new", [(1, 1), (4, 1), (3, 4), (8, 2), (5, 7), (1, 33), (7, 19), (16, 1)])
def test_attention(jg, act, d, group, new):
    rng = np.random.default_rng(group * 100 + new)
    batch = 6
    c = Case(d + new, sizes(rng, batch, 700) - 1, rng.integers(1, new + 1, batch), 2, group, d, 16 << (new % 3), act)
    compare(c, *jg.jgdpa_cache_fwd(**c.kwargs()))


@gpu
@pytest.mark.parametrize("act", ["gelu", "silu", "softmax"])
@pytest.mark.parametrize("d,kv_heads", [(32, 4), (32, 8), (32, 3), (64, 4), (64, 3)])
@pytest.mark.parametrize("group,new", [(1, 1), (3, 2), (4, 7)])
@pytest.mark.parametrize("room", [0, 1 << 16])
def test_small_heads_side_by_side(jg, act, d, kv_heads, group, new, room):
    """One by one in a table of few tokens, side by side in one with room for many."""
    c = Case(d + new, [0, 700, 64, 3000], [new, 1, new, new], kv_heads, group, d, 16, act, bias=65, window=0 if new < 7 else 200,
             mask=True)
    kw = c.kwargs(room=room)
    out = torch.full_like(kw["q"], float("nan"))
    compare(c, *jg.jgdpa_cache_fwd(**kw, out=out))


@gpu
@pytest.mark.parametrize("act", ["silu", "softmax"])
@pytest.mark.parametrize("group", [100, 128, 130])
def test_very_many_heads_per_group(jg, act, group):
    c = Case(group, [70, 5], [3, 1], 1, group, 32, 16, act, bias=9)
    compare(c, *jg.jgdpa_cache_fwd(**c.kwargs()))


@gpu
@pytest.mark.parametrize("act", ["silu", "softmax"])
@pytest.mark.parametrize("new,group,bias,window,page", [
    (1, 1, 257, 0, 16), (9, 2, 33, 0, 64), (33, 1, 5, 100, 32), (64, 4, 0, 1, 128), (20, 3, 1, 64, 256), (40, 1, 129, 7, 1024),
    (5, 1, 4095, 0, 16), (65, 2, 9, 300, 16), (70, 3, 0, 50, 32), (50, 7, 65, 0, 16),
])
def test_trees_bias_and_window(jg, act, new, group, bias, window, page):
    rng = np.random.default_rng(new + bias)
    batch = 4
    c = Case(new, sizes(rng, batch, 900), rng.integers(0, new + 1, batch), 3, group, 64, page, act, bias, window, mask=True,
             extra=3)
    kw = c.kwargs()
    out = torch.full_like(kw["q"], 7.0)
    _, lse = jg.jgdpa_cache_fwd(**kw, out=out)
    compare(c, out, lse)
    assert torch.all(out[c.off[-1]:] == 7.0)  # rows behind the last request


@gpu
@pytest.mark.parametrize("act", ["silu", "softmax"])
@pytest.mark.parametrize("d,kv_heads,new,group", [(32, 4, 3, 2), (32, 3, 20, 1), (32, 4, 40, 1), (64, 2, 5, 3), (64, 2, 10, 3),
                                                  (64, 3, 70, 1), (128, 2, 2, 2), (128, 1, 90, 2)])
@pytest.mark.parametrize("window", [1, 30, 190, 2 ** 31 - 1])
@pytest.mark.parametrize("room", [0, 1 << 16])
def test_windows_of_tokens_in_order(jg, act, d, kv_heads, new, group, window, room):
    """Without a mask and depths."""
    c = Case(d + window % 97, [0, 450, 131, 1], [new, new, 1, new], kv_heads, group, d, 32, act, bias=17, window=window)
    compare(c, *jg.jgdpa_cache_fwd(**c.kwargs(room=room)))


@gpu
@pytest.mark.parametrize("d,new,group", [(32, 5, 2), (64, 20, 1), (128, 33, 2)])
@pytest.mark.parametrize("drop", ["mask", "depth"])
@pytest.mark.parametrize("room", [0, 1 << 16])
def test_a_mask_or_depths_alone(jg, d, new, group, drop, room):
    c = Case(29, [70, 0, 300], [new, new, 2], 4, group, d, 16, "softmax", bias=33, window=60, mask=True)
    setattr(c, drop, None)
    compare(c, *jg.jgdpa_cache_fwd(**c.kwargs(room=room)))


@gpu
@pytest.mark.parametrize("d,group", [(64, 130), (128, 129), (128, 200)])
def test_more_heads_per_group_than_a_tile_has_rows(jg, d, group):
    c = Case(group, [70, 5, 600], [3, 1, 1], 1, group, d, 16, "gelu", bias=9)
    compare(c, *jg.jgdpa_cache_fwd(**c.kwargs()))


@gpu
@pytest.mark.parametrize("act", ["gelu", "softmax"])
@pytest.mark.parametrize("d,kv_heads,new,group", [(32, 4, 6, 1), (32, 4, 25, 1), (32, 3, 5, 2), (64, 2, 9, 3), (128, 2, 6, 2),
                                                  (128, 2, 30, 2)])
@pytest.mark.parametrize("room", [0, 1 << 16])
def test_infinities_in_any_place(jg, act, d, kv_heads, new, group, room):
    """An infinity in one column of one head's value of a drafted token, and NaN
    in values out of every window: only that column of the rows that see it changes."""
    c = Case(41, [150, 40], [new, new], kv_heads, group, d, 16, act, window=60, mask=True)
    kw = c.kwargs(room=room)
    clean, _ = jg.jgdpa_cache_fwd(**kw)
    rng = np.random.default_rng(d + new)
    n = int(c.off[1])
    for u in {0, new // 2, new - 1}:
        sees = torch.tensor([(int(c.mask[t, u // 32]) >> (u % 32)) & 1 for t in range(n)], dtype=torch.bool)
        head, col = int(rng.integers(kv_heads)), int(rng.integers(d))
        v = kw["v_cache"].clone()
        j = 150 + u
        v[int(c.table[0, j // 16]), j % 16, head, col] = float("inf")
        v[int(c.table[0, 17 // 16]), 17 % 16] = float("nan")
        got = jg.jgdpa_cache_fwd(**{**kw, "v_cache": v})[0].cpu()
        same = torch.ones_like(got, dtype=torch.bool)
        rows = torch.nonzero(sees).flatten()
        for h in range(head * group, (head + 1) * group):
            same[rows, h, col] = False
            assert not torch.isfinite(got[rows, h, col]).any()
        assert torch.equal(got[same], clean.cpu()[same])


@gpu
@pytest.mark.parametrize("act", ["gelu", "softmax"])
@pytest.mark.parametrize("length", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257])
def test_lengths_at_tile_and_page_borders(jg, act, length):
    for new in (1, min(length, 8)):
        c = Case(length, [length - new, 0, length - new], [new, 1, new], 1, 2, 64, 16, act, bias=65)
        compare(c, *jg.jgdpa_cache_fwd(**c.kwargs()))


@gpu
@pytest.mark.parametrize("act", ["silu", "softmax"])
def test_prompts_longer_than_a_row_tile(jg, act):
    """New tokens without a mask: causal over any number of them."""
    c = Case(5, [0, 70, 300], [200, 131, 1], 2, 2, 64, 32, act, bias=33)
    compare(c, *jg.jgdpa_cache_fwd(**c.kwargs()))


@gpu
@pytest.mark.parametrize("act", ["gelu", "softmax"])
@pytest.mark.parametrize("new,group,length", [(1, 4, 20000), (3, 4, 20000), (6, 5, 9000), (20, 3, 6000), (40, 4, 5000), (50, 5, 4000)])
def test_long_contexts_are_cut_between_ctas(jg, act, new, group, length):
    """One long and some short requests: the long one's keys are split."""
    c = Case(9, [length, 3, 700], [new, 1, 2], 1, group, 64, 64, act, bias=129, nan=False)
    kw = c.kwargs()
    out = torch.full_like(kw["q"], float("nan"))  # every row is written
    compare(c, *jg.jgdpa_cache_fwd(**kw, out=out))


@gpu
@pytest.mark.parametrize("act", ["gelu", "softmax"])
@pytest.mark.parametrize("d", [32, 128])
@pytest.mark.parametrize("new,group,window", [(1, 3, 0), (9, 2, 0), (40, 2, 0), (40, 5, 70)])
def test_many_requests_per_cta(jg, act, d, new, group, window):
    """Six requests, each there 200 times: every CTA walks several items."""
    rng = np.random.default_rng(new)
    c = Case(d + new, sizes(rng, 6, 500), rng.integers(1, new + 1, 6), 2, group, d, 16, act, bias=33, window=window, mask=True)
    want = c.oracle()
    kw = c.kwargs()
    n, times = int(c.off[-1]), 200
    order = rng.permutation(np.repeat(np.arange(6), times))
    rows = np.concatenate([np.arange(c.off[b], c.off[b + 1]) for b in order])
    off = np.concatenate([[0], np.cumsum(c.new[order])])
    for k in ("q", "tree_mask", "depths"):
        kw[k] = kw[k][torch.from_numpy(rows).cuda()].contiguous()
    kw["block_table"] = kw["block_table"][torch.from_numpy(order).cuda()].contiguous()
    out, lse = jg.jgdpa_cache_fwd(**{**kw, "q_offsets": i32(off, "cuda"), "kv_lens": i32(c.kv[order], "cuda")})
    c.off = off
    assert len(rows) == n * times
    compare(c, out, lse, (want[0][rows], want[1][:, rows], want[2][rows], want[3][:, rows], want[4][rows]))


@gpu
@pytest.mark.parametrize("act", ["gelu", "softmax"])
@pytest.mark.parametrize("new", [4, 40])
def test_rows_that_see_nothing(jg, act, new):
    c = Case(3, [0, 50], [new, new], 1, 2, 64, 16, act, window=3, mask=True)
    c.mask[::3] = 0                # no drafted token, and the window hides the context from deep ones
    c.depth = c.depth * 5 + 5
    out, lse = jg.jgdpa_cache_fwd(**c.kwargs())
    want = c.oracle()
    compare(c, out, lse, want)
    empty = torch.from_numpy(np.all(want[2] == 0, axis=-1))
    assert empty.any() and not out.cpu()[empty].any()


@gpu
@pytest.mark.parametrize("up", [True, False])
@pytest.mark.parametrize("d,new", [(32, 3), (128, 1), (64, 8), (32, 30), (64, 24), (128, 50)])
@pytest.mark.parametrize("room", [0, 1 << 16])
def test_scores_that_rise_and_fall(jg, d, new, up, room):
    """Softmax whose scores grow (or shrink) along the keys, a little per tile
    and by jumps: the running maximum has to follow."""
    c = Case(23, [900, 77], [new, new], 4, 2, d, 64, "softmax", nan=False)
    for b, n in enumerate(c.kv):
        for j in range(n):
            at = j / n if up else 1 - j / n
            c.k[c.table[b, j // 64], j % 64] *= 8.0 * at ** 2 + (12.0 if at > 0.8 else 0.0)
    out, lse = jg.jgdpa_cache_fwd(**c.kwargs(room=room))
    compare(c, out, lse)


@gpu
@pytest.mark.parametrize("new", [1, 20, 70])
@pytest.mark.parametrize("value", [-float("inf"), torch.finfo(torch.float32).min])
def test_bias_entries_that_hide_keys(jg, new, value):
    """Softmax with bias entries of -inf or the lowest fp32: keys 12 and more
    behind get no weight, whole tiles of them among the others."""
    c = Case(17, [700, 0, 129, 64], [new] * 4, 2, 2, 64, 32, "softmax", bias=33)
    c.bias[:, 28:] = value
    out, lse = jg.jgdpa_cache_fwd(**c.kwargs())
    compare(c, out, lse)
    c.bias[1] = -float("inf")  # a head that sees nothing
    out, lse = jg.jgdpa_cache_fwd(**c.kwargs())
    assert not out[:, 1].any() and torch.isneginf(lse[1]).all() and torch.isfinite(lse[0]).all()


@gpu
@pytest.mark.parametrize("act", ["gelu", "silu", "softmax"])
@pytest.mark.parametrize("new,group", [(6, 2), (30, 4), (40, 8)])
def test_infinities_reach_only_the_rows_that_see_them(jg, act, new, group):
    """NaN and infinities in one drafted token's key and value, and in a context
    token out of the window: rows that do not see it are as without it."""
    c = Case(4, [90, 40], [new, new], 2, group, 64, 16, act, window=60, mask=True)
    kw = c.kwargs()
    clean, clean_lse = jg.jgdpa_cache_fwd(**kw)
    lo, u = 0, 2
    sees = torch.tensor([(int(c.mask[t, u // 32]) >> (u % 32)) & 1 for t in range(c.off[1])], dtype=torch.bool)
    assert sees.any() and not sees.all()
    for value in (float("nan"), float("inf"), -float("inf")):
        bad = {**kw, "k_cache": kw["k_cache"].clone(), "v_cache": kw["v_cache"].clone()}
        j = 90 + u
        bad["v_cache"][int(c.table[0, j // 16]), j % 16, :, 3] = value
        bad["k_cache"][int(c.table[0, j // 16]), j % 16, 0, 5] = value
        bad["v_cache"][int(c.table[0, 20 // 16]), 20 % 16] = value  # behind every row's window
        out, lse = jg.jgdpa_cache_fwd(**bad)
        n = c.off[1]
        assert torch.equal(out[lo:n].cpu()[~sees], clean[lo:n].cpu()[~sees])
        assert torch.equal(out[n:], clean[n:])
        # kv head 1's keys are clean: the infinity reaches column 3 of the rows that see it, and only that
        h = slice(group, 2 * group)
        got = out[lo:n, h].float().cpu()[sees]
        assert not torch.isfinite(got[..., 3]).any()
        assert torch.equal(got[..., :3], clean[lo:n, h].float().cpu()[sees][..., :3])
        if lse is not None:
            assert torch.equal(lse[:, lo:n].cpu()[:, ~sees], clean_lse[:, lo:n].cpu()[:, ~sees])


@gpu
def test_strided_queries_and_interleaved_pool(jg):
    c = Case(6, [100, 30], [2, 3], 2, 2, 64, 16, "softmax", bias=9)
    kw = c.kwargs()
    clean, clean_lse = jg.jgdpa_cache_fwd(**kw)
    wide = torch.randn(c.q.shape[0], 3 * c.heads, 64, device="cuda").to(torch.bfloat16)
    wide[:, c.heads:2 * c.heads] = kw["q"]
    pool = torch.stack([kw["k_cache"], kw["v_cache"]], 1)
    out, lse = jg.jgdpa_cache_fwd(**{**kw, "q": wide[:, c.heads:2 * c.heads], "k_cache": pool[:, 0], "v_cache": pool[:, 1]})
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)
    compare(c, out, lse)


@gpu
@pytest.mark.parametrize("new", [1, 40])
def test_device_detected_errors_leave_the_outputs(jg, new):
    c = Case(7, [100, 30], [new, new], 2, 2, 64, 16, "softmax", nan=False)
    kw = c.kwargs()
    n = jg.jgdpa_cache_fwd_workspace_bytes(c.heads, c.kv_heads, 64, kw["max_q"])
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    good, _ = jg.jgdpa_cache_fwd(**kw, workspace=ws)
    assert jg.jgdpa_read_device_status(ws) == 0
    off, kv = c.off, c.kv
    for change in (dict(q_offsets=[1, off[1], off[2]]), dict(q_offsets=[0, off[2], off[1]]), dict(q_offsets=[0, off[1], off[2] + 1]),
                   dict(kv_lens=[new - 1, kv[1]]), dict(kv_lens=[kv[0], 16 * c.table.shape[1] + 1]), dict(kv_lens=[-5, kv[1]]),
                   dict(kv_lens=[2 ** 31 - 1, kv[1]])):
        bad = {k: i32(v, "cuda") for k, v in change.items()}
        out = torch.full_like(good, 7.0)
        jg.jgdpa_cache_fwd(**{**kw, **bad}, out=out, workspace=ws)
        assert jg.jgdpa_read_device_status(ws) == 6, change
        assert torch.all(out == 7.0)
    if new > 1:
        jg.jgdpa_cache_fwd(**{**kw, "max_q": new - 1}, workspace=ws)
        assert jg.jgdpa_read_device_status(ws) == 6
    for entry in (-1, c.pages, 2 ** 31 - 1, -2 ** 31):
        table = kw["block_table"].clone()
        table[0, 1] = entry
        out, _ = jg.jgdpa_cache_fwd(**{**kw, "block_table": table}, workspace=ws)
        assert jg.jgdpa_read_device_status(ws) == 9
        assert torch.equal(out[off[1]:], good[off[1]:])  # the other request
    out, _ = jg.jgdpa_cache_fwd(**kw, workspace=ws)
    assert jg.jgdpa_read_device_status(ws) == 0 and torch.equal(out, good)


@gpu
def test_mask_narrower_than_a_request_is_refused(jg):
    c = Case(8, [10], [33], 1, 1, 64, 16, "softmax", mask=True)
    kw = c.kwargs()
    ws = torch.empty(jg.jgdpa_cache_fwd_workspace_bytes(1, 1, 64, 33), dtype=torch.uint8, device="cuda")
    jg.jgdpa_cache_fwd(**{**kw, "tree_mask": kw["tree_mask"][:, :1].contiguous()}, workspace=ws)
    assert jg.jgdpa_read_device_status(ws) == 6


@gpu
@pytest.mark.parametrize("act", ["gelu", "softmax"])
@pytest.mark.parametrize("d,new,group", [(128, 1, 4), (64, 6, 4), (32, 1, 2), (128, 30, 2), (64, 60, 4)])
def test_a_wait_that_gives_up_is_reported_and_recovered_from(jg, act, d, new, group):
    c = Case(3, [3000, 900], [new, new], 4, group, d, 64, act, nan=False)
    kw = c.kwargs()
    ws = torch.empty(jg.jgdpa_cache_fwd_workspace_bytes(c.heads, 4, d, new), dtype=torch.uint8, device="cuda")
    good, _ = jg.jgdpa_cache_fwd(**kw, workspace=ws)
    jg.jgdpa_set_wait_limit_ns(1)
    try:
        jg.jgdpa_cache_fwd(**kw, workspace=ws)
        assert jg.jgdpa_read_device_status(ws) in (0, 7)  # (0: every wait was shorter than its first test)
    finally:
        jg.jgdpa_set_wait_limit_ns(0)
    out, _ = jg.jgdpa_cache_fwd(**kw, workspace=ws)
    assert jg.jgdpa_read_device_status(ws) == 0 and torch.equal(out, good)


@gpu
def test_empty_calls(jg):
    c = Case(1, [5], [0], 1, 1, 64, 16, "softmax", extra=2)
    kw = c.kwargs()
    out = torch.full_like(kw["q"], 7.0)
    jg.jgdpa_cache_fwd(**kw, out=out)
    assert torch.all(out == 7.0)
    kw["q"] = kw["q"][:0]
    assert jg.jgdpa_cache_fwd(**kw)[0].shape[0] == 0
    kw = c.kwargs()
    kw.update(block_table=kw["block_table"][:0], q_offsets=i32([0], "cuda"), kv_lens=i32([], "cuda"))
    jg.jgdpa_cache_fwd(**kw)


@gpu
def test_empty_call_with_a_mask(jg):
    kw = Case(1, [5, 40], [3, 2], 1, 1, 64, 16, "softmax", mask=True).kwargs()
    for k in ("q", "tree_mask", "depths"):
        kw[k] = kw[k][:0]
    kw["q_offsets"] = torch.zeros_like(kw["q_offsets"])
    out, lse = jg.jgdpa_cache_fwd(**kw)
    assert out.shape[0] == 0 and lse.shape[1] == 0


@gpu
@pytest.mark.parametrize("ended", [0.0, 0.6])
def test_plan_with_many_pages_back(jg, ended):
    """Far more pages come back than tokens are added."""
    rng = np.random.default_rng(31)
    batch, width = 300, 400
    held = rng.integers(0, width + 1, batch)
    ctx = np.where(rng.random(batch) < ended, 0, np.maximum(0, held * 16 - rng.integers(0, 40, batch)))
    new = np.where(ctx > 0, rng.integers(0, 3, batch), 0)
    new = np.minimum(new, width * 16 - ctx)
    pages = int(held.sum()) + 50
    ids = rng.permutation(pages)
    table = np.full((batch, width), -5)
    at = np.concatenate([[0], np.cumsum(held)])
    for b in range(batch):
        table[b, :held[b]] = ids[at[b]:at[b + 1]]
    free = np.full(pages, -9)
    free[:50] = ids[at[-1]:]
    check_plan(jg, ctx, new, held, table, free, 50, 16, int(new.sum()) + 5)


@gpu
@pytest.mark.parametrize("new", [1, 40])
def test_same_bits_in_graphs_and_on_other_streams(jg, new):
    """Replays of two captured calls, and calls on two streams at once, give
    the bits of a call alone."""
    cs = [Case(20 + i, [9000 - 4000 * i, 17], [new, 2], 2, 4, 64, 64, act, nan=False)
          for i, act in enumerate(("softmax", "gelu"))]
    kws = [c.kwargs() for c in cs]
    alone = [jg.jgdpa_cache_fwd(**kw)[0].clone() for kw in kws]
    streams = [torch.cuda.Stream() for _ in kws]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = [jg.jgdpa_cache_fwd(**kw, stream=s)[0] for kw, s in zip(kws, streams)]
        torch.cuda.synchronize()
        for o, a in zip(outs, alone):
            assert torch.equal(o, a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [jg.jgdpa_cache_fwd(**kw)[0] for kw in kws]
    for _ in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for o, a in zip(outs, alone):
            assert torch.equal(o, a)


# ------------------------------------------------------------ together (GPU)
@gpu
@pytest.mark.parametrize("act", ["gelu", "softmax"])
def test_serving_steps_follow_the_packed_forward(jg, act):
    """Prompts, then single tokens, a rejected draft and requests that end and
    start, through plan, append and attention; at every step each request's
    new rows are those of jgdpa_fwd over its packed history (causal)."""
    rng = np.random.default_rng(12)
    batch, heads, d, page, pool, width = 3, 2, 64, 16, 40, 20
    kc = torch.full((pool, page, heads, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    free, count = torch.arange(pool, dtype=torch.int32, device="cuda"), i32([pool], "cuda")
    held = i32([0] * batch, "cuda")
    bias = 0.1 * torch.randn(heads, 33, device="cuda")
    history = [[torch.zeros(0, heads, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(batch)]
    steps = [([0, 0, 0], [50, 0, 17]), ([50, 0, 17], [1, 33, 1]), ([51, 33, 18], [7, 7, 7]), ([53, 40, 18], [1, 1, 1]),
             ([54, 0, 19], [1, 90, 1]), ([55, 90, 0], [1, 1, 0])]
    for keep, new in steps:
        total = sum(new)
        q, k, v = (torch.from_numpy(rng.standard_normal((total, heads, d), dtype=np.float32)).to(torch.bfloat16).cuda()
                   for _ in range(3))
        slots, q_off, kv, held, count = jg.jgdpa_cache_plan(i32(keep, "cuda"), i32(new, "cuda"), held, table, free, count,
                                                            page, total)
        jg.jgdpa_cache_append(k, v, slots, kc, vc)
        out, _ = jg.jgdpa_cache_fwd(q, kc, vc, table, q_off, kv, act, d ** -0.5, max_q=max(new), bias_table=bias)
        at = 0
        for b in range(batch):
            history[b] = [torch.cat([h[:keep[b]], x[at:at + new[b]]]) for h, x in zip(history[b], (k, v))]
            n = keep[b] + new[b]
            if new[b]:
                # queries of the history's rows are not needed: zeros in front
                full = torch.cat([torch.zeros(keep[b], heads, d, dtype=torch.bfloat16, device="cuda"), q[at:at + new[b]]])
                off = i32([0, n], "cuda")
                want, _ = jg.jgdpa_fwd(full, *history[b], off, off, act, d ** -0.5, bias_table=bias, causal=True)
                want = want[keep[b]:].float()
                # both round P and O to bf16 (u = 2^-8 each of sum |P||V| at most);
                # GELU: jgdpa_fwd's evaluation of act is within 1.2e-3
                x = torch.einsum("qhd,khd->hqk", q[at:at + new[b]].float(), history[b][0].float()) * d ** -0.5
                apart = torch.arange(keep[b], n, device="cuda")[:, None] - torch.arange(n, device="cuda")
                x = (x + bias[:, apart.clamp(-16, 16) + 16]).masked_fill(apart < 0, -torch.inf)
                p = torch.softmax(x, -1) if act == "softmax" else torch.nn.functional.gelu(x).nan_to_num(0.0).abs()
                av = history[b][1].float().abs()
                size = torch.einsum("hqk,khd->qhd", p, av)
                extra = 0 if act == "softmax" else 2.4e-3 * av.sum(0)
                tol = 4 * 2.0 ** -8 * size + 2.0 ** -10 * size + extra
                assert torch.all((out[at:at + new[b]].float() - want).abs() <= tol)
            at += new[b]
    live = [int(h) for h in held.cpu()]
    ids = [int(x) for b, h in enumerate(live) for x in table[b, :h].cpu()] + free[:int(count)].cpu().tolist()
    assert sorted(ids) == list(range(pool))  # no page lost, none twice
