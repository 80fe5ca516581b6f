"""The paged cache held in 4 bits: writes, rows read back, attention over it."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import cache, step as oracle
from tests.test_cache import tree

gpu = pytest.mark.gpu
U = 2.0 ** -8  # half a step of bf16, relative


@pytest.fixture(scope="module")
def jg():
    from jagged_gdpa_gb300 import build as b
    b.build()
    import jagged_gdpa_gb300 as m
    return m


def i32(x, device="cuda"):
    return torch.tensor(np.asarray(x, dtype=np.int64).astype(np.int32), device=device)


def normal(rng, *shape, device="cuda"):
    return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32)).to(torch.bfloat16).to(device)


def empty_cache(pages, heads, page, d, device="cuda"):
    return [torch.zeros(pages, heads, page, n, dtype=t, device=device)
            for n, t in ((d // 2, torch.uint8), (2, torch.bfloat16)) * 2]


class Case:
    """A batch whose cache holds random codes, steps and middles, on the CPU."""

    def __init__(self, seed, ctx, new, kv_heads, group, d, page, act="softmax", bias=0, window=0, mask=False, extra=0,
                 stale=True, middle=0.3):
        rng = np.random.default_rng(seed)
        self.act, self.window, self.d, self.page = act, window, d, page
        self.heads, self.kv_heads, self.scale = kv_heads * group, kv_heads, d ** -0.5
        ctx, new = np.asarray(ctx), np.asarray(new)
        self.new, self.kv = new, ctx + new
        self.off = np.concatenate([[0], np.cumsum(new)])
        need = -(-self.kv // page)
        self.pages = int(need.sum()) + 2
        self.table = np.full((len(ctx), max(1, int(need.max()))), 2 ** 31 - 7)  # entries of no token: no page
        ids = rng.permutation(self.pages)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        total = int(self.off[-1]) + extra
        self.q = normal(rng, total, self.heads, d, device="cpu")
        self.cache = []
        live = torch.zeros(self.pages, page, dtype=torch.bool)
        for b, n in enumerate(self.kv):
            for j in range(n):
                live[self.table[b, j // page], j % page] = True
        for _ in range(2):
            codes = torch.from_numpy(rng.integers(0, 256, (self.pages, kv_heads, page, d // 2), dtype=np.uint8))
            scales = torch.from_numpy(np.stack([rng.uniform(0.1, 0.4, (self.pages, kv_heads, page)),
                                                middle * rng.standard_normal((self.pages, kv_heads, page))], -1)).bfloat16()
            if stale:  # places that hold no token hold anything
                scales.permute(0, 2, 1, 3)[~live] = float("nan")
            self.cache += [codes, scales]
        self.bias = torch.from_numpy((0.5 * rng.standard_normal((self.heads, bias))).astype(np.float32)) if bias else None
        words = -(-int(max(1, new.max())) // 32)
        self.mask, self.depth = tree(rng, new, words) if mask else (None, None)
        if mask and extra:
            self.mask = np.concatenate([self.mask, np.zeros((extra, words), np.int64)])
            self.depth = np.concatenate([self.depth, np.zeros(extra, np.int64)])

    def want(self):
        """(out, lse, size, dot, vsum) as the bf16 cache's oracle gives them, size, dot and vsum from
        |s (c - 8)| + |z| in the values' place: what the kernel's sums add up."""
        f = lambda t: t.double().numpy()  # noqa: E731
        kc, ks, vc, vs = (f(t) for t in self.cache)
        k, v = oracle.values(kc.astype(np.uint8), ks), oracle.values(vc.astype(np.uint8), vs)
        big = [np.abs(s[..., :1] * (oracle.unpack(c.astype(np.uint8)) - 8)) + np.abs(s[..., 1:]) for c, s in ((kc, ks), (vc, vs))]
        rest = (self.table, self.off, self.kv, self.act, self.scale, None if self.bias is None else f(self.bias), self.window,
                self.mask, self.depth)
        turn = lambda x: x.transpose(0, 2, 1, 3)  # noqa: E731
        out, lse, _, _, _ = cache.attend(f(self.q), turn(k), turn(v), *rest)
        _, _, size, _, vsum = cache.attend(f(self.q), turn(k), turn(big[1]), *rest)
        _, _, _, dot, _ = cache.attend(np.abs(f(self.q)), turn(big[0]), turn(v), *rest)
        return out, lse, size, dot, vsum

    def kwargs(self, device="cuda"):
        mask = None if self.mask is None else torch.from_numpy(self.mask.astype(np.uint32).view(np.int32)).to(device)
        names = ("k_codes", "k_scales", "v_codes", "v_scales")
        return dict(q=self.q.to(device), **{n: t.to(device) for n, t in zip(names, self.cache)},
                    block_table=i32(self.table, device), q_offsets=i32(self.off, device), kv_lens=i32(self.kv, device),
                    act=self.act, scale=self.scale, max_q=int(max(1, self.new.max())),
                    bias_table=None if self.bias is None else self.bias.to(device), window=self.window, tree_mask=mask,
                    depths=None if self.depth is None else i32(self.depth, device))


def compare(case, out, lse, want=None):
    """As for the bf16 cache (u = 2^-8): scores are fp32 sums of d exact products and a few
    fp32 roundings of them; P times the step rounds to bf16 (u), P times the middle does not; then O."""
    o, ls, size, dot, vsum = want if want is not None else case.want()
    n = case.off[-1]
    got = out.double().cpu().numpy()[:n]
    o, size, vsum, dot = o[:n], size[:n], vsum[:n], dot[:, :n]
    es = (case.d + 8) * 2.0 ** -23 * dot + 2.0 ** -20
    if case.act == "softmax":
        tol = size * (U + 2.0 ** -12 + 2 * es.T[..., None])
        le = lse.double().cpu().numpy()[:, :n]
        assert np.array_equal(np.isneginf(le), np.isneginf(ls[:, :n]))
        fin = np.isfinite(ls[:, :n])
        assert np.all(np.abs(le[fin] - ls[:, :n][fin]) <= (es + 2.0 ** -20 * np.abs(ls[:, :n]))[fin])
    else:  # GELU's Phi within 1.9e-3 relative, |act'| <= 1.13
        tol = size * (U + 2.0 ** -12 + 2e-3) + vsum * 1.13 * es.T[..., None]
        assert lse is None
    tol = tol + U * (np.abs(o) + tol)
    bad = ~(np.abs(got - o) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size}, worst {np.nanmax(np.abs(got - o) / (tol + 1e-30)):.2f} tolerances"


# ------------------------------------------------------------ the oracle (CPU)
def test_oracle_rows_are_within_half_a_step():
    rng = np.random.default_rng(0)
    x = oracle.bf16(rng.standard_normal((50, 64)) * 3 + rng.standard_normal((50, 1)))
    c, s, z = oracle.quantise(x)
    y = oracle.values(oracle.pack(c), np.stack([s, z], -1).astype(np.float64))
    # half a step; the step itself is rounded (2^-9, at most 8 of them off the middle), and so is the middle
    assert np.all(np.abs(y - x) <= (0.5 + 8 * 2.0 ** -8) * s[:, None] + U * np.abs(z[:, None]) + U * np.abs(x))
    assert np.array_equal(oracle.unpack(oracle.pack(c)), c) and c.min() == 0 and c.max() == 15


def test_oracle_rows_by_hand():
    c, s, z = oracle.quantise(np.array([[0.0, 15.0, 7.4, 7.5], [2.0, 2.0, 2.0, 2.0]]))
    assert c.tolist() == [[0, 15, 7, 8], [8, 8, 8, 8]] and s.tolist() == [1.0, 0.0] and z.tolist() == [8.0, 2.0]


# ------------------------------------------------------------ refusals (CPU)
CACHE = dict(kc=1 << 20, ks=1 << 20, vc=1 << 20, vs=1 << 20, kcs=16 * 4 * 32, kss=16 * 4 * 2, vcs=16 * 4 * 32, vss=16 * 4 * 2,
             pages=8, page=16)


def _fwd_args(**kw):
    a = dict(q=1 << 20, qs=512, **CACHE, table=1 << 20, width=4, off=1 << 20, kv=1 << 20, batch=1, total=4, max_q=4, heads=8,
             kv_heads=4, d=64, act=2, scale=0.125, bias=None, blen=0, window=0, mask=None, words=0, depth=None, out=1 << 20,
             lse=1 << 20, ws=1 << 20, wsb=1 << 30, stream=None)
    a.update(kw)
    a["scale"] = ctypes.c_float(a["scale"])
    return list(a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(d=48), 2), (dict(page=24), 2), (dict(page=8), 2), (dict(pages=0), 1), (dict(pages=1 << 28), 2), (dict(kcs=16 * 4 * 32 - 16), 1),
    (dict(vcs=16 * 4 * 32 + 8), 3), (dict(kss=16 * 4 * 2 + 4), 3), (dict(vss=16), 1), (dict(kc=(1 << 20) + 8), 3), (dict(ks=None), 1),
    (dict(kv_heads=3, kcs=1 << 20, vcs=1 << 20, kss=1 << 20, vss=1 << 20), 1), (dict(kv_heads=0), 1), (dict(act=3), 1), (dict(scale=float("inf")), 1),
    (dict(blen=4, bias=1 << 20), 1), (dict(blen=5), 1), (dict(blen=8191, bias=1 << 20), 2), (dict(window=-1), 1), (dict(words=1), 1),
    (dict(mask=1 << 20), 1), (dict(act=0), 1), (dict(batch=16385), 2), (dict(off=None), 1), (dict(q=None), 1), (dict(qs=504), 1),
    (dict(qs=516), 3), (dict(out=(1 << 20) + 8), 3), (dict(batch=-1), 1), (dict(max_q=-1), 1), (dict(width=1 << 28), 2),
])
def test_fwd_rejects_bad_arguments_without_a_launch(jg, kw, code):
    assert jg.load().jgdpa_cache4_fwd(*_fwd_args(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(k=None), 1), (dict(slots=None), 1), (dict(ks_=248), 1), (dict(ks_=260), 3), (dict(k=(1 << 20) + 8), 3),
    (dict(d=16), 2), (dict(page=12), 2), (dict(pages=0), 1), (dict(kcs=16), 1), (dict(rows=(1 << 31) - 1), 2),
])
def test_rows_reject_bad_arguments_without_a_launch(jg, kw, code):
    a = dict(k=1 << 20, v=1 << 20, ks_=256, vs_=256, slots=1 << 20, rows=3, **CACHE, heads=4, d=64)
    a.update(kw)
    c = [a[n] for n in CACHE]
    assert jg.load().jgdpa_cache4_append(a["k"], a["v"], a["ks_"], a["vs_"], a["slots"], a["rows"], *c, a["heads"], a["d"], None) == code
    assert jg.load().jgdpa_cache4_read(*c, a["heads"], a["d"], a["slots"], a["rows"], a["k"], a["v"], a["ks_"], a["vs_"], None) == code


@pytest.mark.parametrize("field,change,match", [
    ("q", lambda t: t.float(), "q must have dtype"),
    ("q", lambda t: t[:, :, :32], "q must have shape"),
    ("k_codes", lambda t: t[0], "k_codes must be"),
    ("k_codes", lambda t: t.char(), "k_codes must have dtype"),
    ("v_codes", lambda t: t[:-1], "v_codes must have shape"),
    ("k_scales", lambda t: t.float(), "k_scales must have dtype"),
    ("v_scales", lambda t: t[..., :1], "v_scales must have shape"),
    ("k_codes", lambda t: t.transpose(1, 2).contiguous().transpose(1, 2), "contiguous inside"),
    ("v_scales", lambda t: t[:1].expand(t.shape), "must not overlap"),
    ("block_table", lambda t: t.long(), "block_table must have dtype"),
    ("q_offsets", lambda t: t[:-1], "q_offsets must have shape"),
    ("tree_mask", lambda t: t[:, :0], "tree_mask must have columns"),
    ("bias_table", lambda t: t[:-1], "bias_table must have shape"),
    ("q", lambda t: t, "CUDA device"),
])
def test_wrapper_rejects_bad_tensors(jg, field, change, match):
    kw = Case(0, [40, 20], [3, 4], 2, 2, 64, 16, bias=5, mask=True).kwargs("cpu")
    kw[field] = change(kw[field])
    with pytest.raises(ValueError, match=match):
        jg.jgdpa_cache4_fwd(**kw)


def test_wrappers_reject_other_bad_calls(jg):
    kw = Case(0, [40], [3], 2, 2, 64, 16).kwargs("cpu")
    with pytest.raises(ValueError, match="softmax mode only"):
        jg.jgdpa_cache4_fwd(**{**kw, "act": "gelu"}, lse=torch.zeros(4, 3))
    with pytest.raises(ValueError, match="max_q must fit"):
        jg.jgdpa_cache4_fwd(**{**kw, "max_q": 1 << 32})
    four = [kw[n] for n in ("k_codes", "k_scales", "v_codes", "v_scales")]
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k_new must have shape"):
        jg.jgdpa_cache4_append(k, k, i32([0, 1], "cpu"), *four)
    with pytest.raises(ValueError, match="v_new must have dtype"):
        jg.jgdpa_cache4_append(k, k.float(), i32([0, 1, 2], "cpu"), *four)
    with pytest.raises(ValueError, match="k_out must have shape"):
        jg.jgdpa_cache4_read(*four, i32([0, 1], "cpu"), k_out=k)
    with pytest.raises(ValueError, match="slots must have dtype"):
        jg.jgdpa_cache4_read(*four, torch.zeros(3))
    with pytest.raises(ValueError, match="CUDA device"):
        jg.jgdpa_cache4_read(*four, i32([0, 1], "cpu"))


# ------------------------------------------------------------ rows (GPU)
@gpu
@pytest.mark.parametrize("rows,heads,d,page", [(1, 1, 32, 16), (37, 3, 64, 32), (500, 2, 128, 16), (33, 5, 128, 1024), (3000, 8, 64, 128),
                                               (20000, 2, 32, 64)])
def test_rows_there_and_back(jg, rows, heads, d, page):
    rng = np.random.default_rng(rows)
    pages = -(-rows // page) + 2
    pool = [torch.full((pages, 2, heads, page, n), 3, dtype=t, device="cuda") for n, t in ((d // 2, torch.uint8), (2, torch.bfloat16))]
    four = [pool[0][:, 0], pool[1][:, 0], pool[0][:, 1], pool[1][:, 1]]  # K and V interleaved
    wide = 3 * normal(rng, rows, 3, heads, d) + normal(rng, rows, 3, heads, 1)
    wide[0] = 2.5  # one value: a step of 0
    if rows > 3:
        wide[1, :, 0, 1:] = 0.0
        wide[2] *= 2.0 ** -100
        wide[3] *= 2.0 ** 100
    k, v = wide[:, 1], wide[:, 2]
    slots = rng.permutation(pages * page)[:rows]
    if rows > 30:
        slots[7], slots[8] = -1, pages * page
    jg.jgdpa_cache4_append(k, v, i32(slots), *four)
    live = (slots >= 0) & (slots < pages * page)
    at, place = slots[live] // page, slots[live] % page
    for x, codes, scales in ((k, *four[:2]), (v, *four[2:])):
        c, s, z = oracle.quantise(x.float().cpu().numpy()[live])
        assert np.array_equal(codes[at, :, place].cpu().numpy(), oracle.pack(c))
        assert np.array_equal(scales[at, :, place].float().cpu().numpy(), np.stack([s, z], -1))
        written = np.zeros((pages, page), bool)
        written[at, place] = True
        rest = torch.from_numpy(~written).cuda()
        assert torch.all(codes.permute(0, 2, 1, 3)[rest] == 3) and torch.all(scales.permute(0, 2, 1, 3)[rest] == 3)
    out = torch.full((rows, 2, heads, d), 7.0, dtype=torch.bfloat16, device="cuda")
    got = jg.jgdpa_cache4_read(*four, i32(slots), k_out=out[:, 0])
    assert got[0].data_ptr() == out.data_ptr() and torch.all(out[:, 1] == 7.0)
    for y, codes, scales in ((got[0], *four[:2]), (got[1], *four[2:])):
        want = oracle.values(codes[at, :, place].cpu().numpy(), scales[at, :, place].double().cpu().numpy())
        # (the sum rounds to fp32, then to bf16)
        assert np.all(np.abs(y[torch.from_numpy(live)].double().cpu().numpy() - want) <= (U + 2.0 ** -23) * np.abs(want) + 1e-39)
        assert torch.all(y[torch.from_numpy(~live)] == 0)


@gpu
def test_rows_with_infinities_and_nan(jg):
    """They take their own head with them, and no other."""
    rng = np.random.default_rng(1)
    k = normal(rng, 6, 2, 64)
    k[1, 0, 3], k[2, 1, 60], k[3, 0, 0] = float("nan"), float("inf"), -float("inf")
    four = empty_cache(1, 2, 16, 64)
    jg.jgdpa_cache4_append(k, k, i32(range(6)), *four)
    got, _ = jg.jgdpa_cache4_read(*four, i32(range(6)))
    bad = torch.zeros(6, 2, dtype=torch.bool, device="cuda")
    bad[1, 0] = bad[2, 1] = bad[3, 0] = True
    assert torch.equal(~torch.isfinite(got).all(-1), bad) and not torch.isfinite(got[bad]).any()


@gpu
def test_no_rows(jg):
    four = empty_cache(1, 2, 16, 64)
    k = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    jg.jgdpa_cache4_append(k, k, i32([]), *four)
    assert jg.jgdpa_cache4_read(*four, i32([]))[0].shape == (0, 2, 64)
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(jg.jgdpa_cache4_fwd_workspace_bytes(64), dtype=torch.uint8, device="cuda")
    for off, status in (([0, 0], 0), ([0, 2], 6)):
        out, lse = jg.jgdpa_cache4_fwd(q, *four, i32([[0]]), i32(off), i32([5]), "softmax", 1.0, max_q=0, workspace=ws)
        assert out.shape == (0, 4, 64) and jg.jgdpa_read_device_status(ws) == status


# ------------------------------------------------------------ attention (GPU)
@gpu
@pytest.mark.parametrize("act", ["gelu", "silu", "softmax"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("group,new", [(1, 1), (4, 1), (1, 16), (3, 7), (8, 5), (20, 2)])
def test_attention(jg, act, d, group, new):
    rng = np.random.default_rng(d + group)
    c = Case(d + new, rng.integers(0, 300, 6), rng.integers(0, new + 1, 6), 2, group, d, 16, act, extra=2)
    kw = c.kwargs()
    out = torch.full_like(kw["q"], 7.0)
    out, lse = jg.jgdpa_cache4_fwd(**kw, out=out)
    assert torch.all(out[c.off[-1]:] == 7.0)
    compare(c, out, lse)


@gpu
@pytest.mark.parametrize("act", ["gelu", "softmax"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("new,group,bias,window,page,mask", [
    (6, 2, 9, 0, 32, True), (40, 1, 0, 50, 16, True), (33, 1, 257, 7, 64, False), (1, 8, 33, 100, 128, False), (5, 3, 0, 1, 1024, True)])
def test_trees_bias_and_window(jg, act, d, new, group, bias, window, page, mask):
    rng = np.random.default_rng(new)
    c = Case(new + d, rng.integers(0, 250, 4), rng.integers(1, new + 1, 4), 2, group, d, page, act, bias=bias, window=window, mask=mask)
    compare(c, *jg.jgdpa_cache4_fwd(**c.kwargs()))


@gpu
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 160, 161, 513])
def test_lengths_at_block_and_page_borders(jg, d, length):
    for page in (16, 64):
        c = Case(length, [length - 1, 0], [1, 1], 1, 4, d, page)
        compare(c, *jg.jgdpa_cache4_fwd(**c.kwargs()))


@gpu
@pytest.mark.parametrize("act", ["silu", "softmax"])
@pytest.mark.parametrize("new,group,length,d", [(1, 8, 60000, 128), (1, 1, 30000, 64), (20, 1, 9000, 32), (3, 2, 20000, 128)])
def test_long_contexts_are_cut_between_ctas(jg, act, new, group, length, d):
    c = Case(1, [length], [new], 1, group, d, 64, act, stale=False)
    compare(c, *jg.jgdpa_cache4_fwd(**c.kwargs()))


@gpu
@pytest.mark.parametrize("d,new,group", [(64, 1, 4), (32, 3, 1), (128, 2, 9)])
def test_many_requests_per_cta(jg, d, new, group):
    rng = np.random.default_rng(7)
    c = Case(7, rng.integers(0, 30, 1500), rng.integers(0, new + 1, 1500), 1, group, d, 16, "softmax", stale=False)
    compare(c, *jg.jgdpa_cache4_fwd(**c.kwargs()))


@gpu
@pytest.mark.parametrize("d", [32, 64, 128])
def test_every_key_of_a_long_context_counts(jg, d):
    """One key at a time that outweighs all others: the order of keys and columns, through every block."""
    length = 700
    c = Case(2, [length - 1], [1], 1, 1, d, 32, stale=False)
    kw = c.kwargs()
    kw["k_scales"][..., 1] = 0
    keys = list(range(0, length, 37)) + [length - 1]
    rows = torch.stack([kw["v_codes"][c.table[0, j // 32], 0, j % 32] for j in keys]).cpu().numpy()
    scales = torch.stack([kw["v_scales"][c.table[0, j // 32], 0, j % 32] for j in keys]).double().cpu().numpy()
    want = oracle.values(rows, scales)
    for j, v in zip(keys, want):
        codes = kw["k_codes"].clone()
        at = (c.table[0, j // 32], 0, j % 32)
        signs = torch.from_numpy(np.where(np.arange(d) % 3 == 0, 1, 15).astype(np.uint8)).cuda()
        codes[at] = signs[0::2] | (signs[1::2] << 4)
        q = torch.where(torch.arange(d, device="cuda") % 3 == 0, -300.0, 300.0).bfloat16().view(1, 1, d)
        out, _ = jg.jgdpa_cache4_fwd(**{**kw, "q": q, "k_codes": codes})
        assert np.all(np.abs(out.double().cpu().numpy().ravel() - v) <= 4 * U * (np.abs(v) + 8 * 0.4)), j


@gpu
@pytest.mark.parametrize("act", ["gelu", "softmax"])
def test_rows_that_see_nothing(jg, act):
    c = Case(5, [0, 40], [4, 6], 2, 2, 64, 16, act, mask=True)
    c.mask[1] = c.mask[5] = 0  # the first has no context either
    c.mask[2] &= ~(1 << 2)
    out, lse = jg.jgdpa_cache4_fwd(**c.kwargs())
    compare(c, out, lse)
    assert torch.all(out[1] == 0)


@gpu
@pytest.mark.parametrize("value", [float("-inf"), -3.4028e38, 3e38])
@pytest.mark.parametrize("d", [64, 128])
def test_biases_that_hide_keys_or_are_huge(jg, d, value):
    """-inf hides a key (an infinity or NaN there as well); the type's largest stay finite."""
    c = Case(6, [200, 3], [2, 3], 1, 2, d, 16, bias=65)
    c.bias[0, 40:44] = value  # some near keys of head 0
    c.bias[1, 64] = value     # all far keys of head 1
    kw = c.kwargs()
    if value == float("-inf"):
        want = c.want()
        bad = [(0, j) for j in range(150)]  # far keys, which head 1 does not see: head 0 does
        kw2 = c.kwargs()
        for name in ("k_scales", "v_scales"):
            for b, j in bad:
                kw2[name][c.table[b, j // 16], 0, j % 16] = float("nan")
        out, lse = jg.jgdpa_cache4_fwd(**kw2)
        clean, clean_lse = jg.jgdpa_cache4_fwd(**kw)
        compare(c, clean, clean_lse, want)
        assert torch.equal(out[:, 1], clean[:, 1]) and torch.equal(lse[1], clean_lse[1]) and torch.isnan(out[:2, 0]).all()
        return
    out, lse = jg.jgdpa_cache4_fwd(**kw)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    if value < 0:  # as any bias that leaves a key no weight
        mild = c.kwargs()
        mild["bias_table"][mild["bias_table"] == value] = -1e4
        want, want_lse = jg.jgdpa_cache4_fwd(**mild)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        return
    v = oracle.values(c.cache[2].numpy(), c.cache[3].double().numpy())
    for t in range(2):  # ties of the largest: the mean of V over the keys with that bias
        for head, keys in ((0, range(200 + t - 11, 200 + t - 7)), (1, range(0, 200 + t - 31))):
            seen = np.array([v[c.table[0, j // 16], 0, j % 16] for j in keys])
            tol = 2 * U * (np.abs(seen).mean(0) + 0.4 * 8)  # P s, where s (c - 8) is at most 3.2, and O round to bf16
            assert np.all(np.abs(out[t, head].double().cpu().numpy() - seen.mean(0)) <= tol)


@gpu
@pytest.mark.parametrize("act", ["gelu", "softmax"])
@pytest.mark.parametrize("window", [0, 30])
@pytest.mark.parametrize("d", [32, 128])
def test_infinities_reach_only_the_rows_that_see_them(jg, act, window, d):
    c = Case(9, [100, 0, 33], [5, 7, 1], 2, 2, d, 16, act, window=window, mask=True)
    clean, clean_lse = jg.jgdpa_cache4_fwd(**c.kwargs())
    for name in ("k_scales", "v_scales"):
        for b, j in ((0, 3), (0, 99), (0, 102), (1, 4), (2, 33)):
            for what in (float("nan"), float("inf")):
                kw = c.kwargs()
                kw[name][c.table[b, j // 16], 1, j % 16, 1] = what  # head 1's middle
                out, _ = jg.jgdpa_cache4_fwd(**kw)
                ctx = c.kv[b] - c.new[b]
                for r in range(c.off[-1]):
                    t = r - c.off[b]
                    sees = 0 <= t < c.new[b] and (j < ctx or bool(int(c.mask[r][0]) >> (j - ctx) & 1))
                    if sees and window:
                        pos = j if j < ctx else ctx + c.depth[c.off[b] + j - ctx]
                        sees = abs(ctx + c.depth[r] - pos) < window
                    assert torch.equal(out[r, :2], clean[r, :2])
                    if not sees:
                        assert torch.equal(out[r, 2:], clean[r, 2:]), (name, b, j, r)
                    elif name == "v_scales" or what != what:
                        assert not torch.isfinite(out[r, 2:]).all()


@gpu
@pytest.mark.parametrize("up", [False, True])
def test_scores_that_rise_and_fall(jg, up):
    """Maxima that move through the whole context, on steps and middles far larger than usual."""
    c = Case(10, [900], [2], 1, 4, 64, 16, stale=False)
    j = np.arange(902)
    grow = np.where(up, j, j[::-1]) / 30.0
    for t, x in zip(j, grow):
        c.cache[1][c.table[0, t // 16], 0, t % 16] *= float(x)
    compare(c, *jg.jgdpa_cache4_fwd(**c.kwargs()))


@gpu
def test_middles_far_from_zero(jg):
    """Keys and values with a large common part, which 4 bits hold in the middle."""
    c = Case(11, [333, 10], [1, 4], 2, 2, 128, 16, middle=30.0)
    compare(c, *jg.jgdpa_cache4_fwd(**c.kwargs()))


@gpu
def test_strided_queries_and_interleaved_pool(jg):
    c = Case(12, [100, 30], [2, 3], 2, 2, 64, 16, "softmax", bias=9)
    kw = c.kwargs()
    clean, clean_lse = jg.jgdpa_cache4_fwd(**kw)
    wide = torch.randn(c.q.shape[0], 3 * c.heads, 64, device="cuda").to(torch.bfloat16)
    wide[:, c.heads:2 * c.heads] = kw["q"]
    codes, scales = (torch.stack([kw["k_" + n], kw["v_" + n]], 1) for n in ("codes", "scales"))
    out, lse = jg.jgdpa_cache4_fwd(**{**kw, "q": wide[:, c.heads:2 * c.heads], "k_codes": codes[:, 0], "v_codes": codes[:, 1],
                                      "k_scales": scales[:, 0], "v_scales": scales[:, 1]})
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)


@gpu
def test_device_detected_errors_leave_the_outputs(jg):
    c = Case(7, [100, 30], [3, 3], 2, 2, 64, 16, "softmax", stale=False)
    kw = c.kwargs()
    ws = torch.empty(jg.jgdpa_cache4_fwd_workspace_bytes(64), dtype=torch.uint8, device="cuda")
    good, _ = jg.jgdpa_cache4_fwd(**kw, workspace=ws)
    assert jg.jgdpa_read_device_status(ws) == 0
    off, kv = c.off, c.kv
    for change in (dict(q_offsets=[1, off[1], off[2]]), dict(q_offsets=[0, off[2], off[1]]), dict(q_offsets=[0, off[1], off[2] + 1]),
                   dict(kv_lens=[2, kv[1]]), dict(kv_lens=[kv[0], 16 * c.table.shape[1] + 1]), dict(kv_lens=[-5, kv[1]])):
        out = torch.full_like(good, 7.0)
        jg.jgdpa_cache4_fwd(**{**kw, **{k: i32(v) for k, v in change.items()}}, out=out, workspace=ws)
        assert jg.jgdpa_read_device_status(ws) == 6, change
        assert torch.all(out == 7.0)
    for entry in (-1, c.pages, 2 ** 31 - 1, -2 ** 31):
        table = kw["block_table"].clone()
        table[0, 1] = entry
        out, _ = jg.jgdpa_cache4_fwd(**{**kw, "block_table": table}, workspace=ws)
        assert jg.jgdpa_read_device_status(ws) == 9
        assert torch.equal(out[off[1]:], good[off[1]:])  # the other request
    for depth in (-1, 2 ** 31 - 1):
        depths = torch.zeros(6, dtype=torch.int32, device="cuda")
        depths[1] = depth
        jg.jgdpa_cache4_fwd(**{**kw, "depths": depths}, workspace=ws)
        assert jg.jgdpa_read_device_status(ws) == 6
    out, _ = jg.jgdpa_cache4_fwd(**kw, workspace=ws)
    assert jg.jgdpa_read_device_status(ws) == 0 and torch.equal(out, good)


@gpu
def test_same_bits_in_graphs_and_on_other_streams(jg):
    cs = [Case(20 + i, [9000 - 4000 * i, 17], [3, 2], 2, 4, 128 >> i, 64, act, stale=False) for i, act in enumerate(("softmax", "gelu"))]
    kws = [c.kwargs() for c in cs]
    alone = [jg.jgdpa_cache4_fwd(**kw)[0].clone() for kw in kws]
    streams = [torch.cuda.Stream() for _ in kws]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = [jg.jgdpa_cache4_fwd(**kw, stream=s)[0] for kw, s in zip(kws, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(o, a) for o, a in zip(outs, alone))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [jg.jgdpa_cache4_fwd(**kw)[0] for kw in kws]
    for _ in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, a) for o, a in zip(outs, alone))


@gpu
@pytest.mark.parametrize("d", [32, 64, 128])
def test_a_single_key_loses_no_more_than_its_rounding(jg, d):
    """With one key a softmax gives the value that its codes stand for, rounded to bf16 once (half a step, 2^-8 of
    it); of the codes' part, 8 s at most, two bf16 operands lose 2^-16, and fp32 steps less than that again."""
    rng = np.random.default_rng(d)
    n, heads = 40, 2
    pages = [torch.from_numpy(rng.integers(0, 256, (n, heads, 16, d // 2), dtype=np.uint8)).cuda() for _ in range(2)]
    scales = [normal(rng, n, heads, 16, 2) for _ in range(2)]
    out, _ = jg.jgdpa_cache4_fwd(normal(rng, n, heads, d), pages[0], scales[0], pages[1], scales[1], i32(np.arange(n)[:, None]),
                                 i32(np.arange(n + 1)), i32(np.ones(n)), "softmax", 1.0, max_q=1)
    c, sz = pages[1].cpu().numpy()[:, :, 0].astype(np.int64), scales[1].double().cpu().numpy()[:, :, 0]
    v = sz[..., 1:] + sz[..., :1] * (np.stack([c & 15, c >> 4], -1).reshape(n, heads, d) - 8)
    bad = ~(np.abs(out.double().cpu().numpy() - v) <= U * np.abs(v) + 2.0 ** -15 * 8 * np.abs(sz[..., :1]))
    assert not bad.any(), f"{bad.sum()} of {bad.size}"
