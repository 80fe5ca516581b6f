"""Verification of drafted tokens: which rows stay, the next token, where the rows move."""

import numpy as np
import pytest
import torch

from oracle import step as oracle

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def jg():
    from jagged_gdpa_gb300 import build as b
    b.build()
    import jagged_gdpa_gb300 as m
    return m


def i32(x, device="cuda"):
    return torch.tensor(np.asarray(x, dtype=np.int64).astype(np.int32), device=device)


class Case:
    """Requests of `lens` rows; the values of bf16 or fp32 probabilities."""

    def __init__(self, seed, lens, vocab, kind="chain", half=False, draft_half=None, agree=0.7, extra=0):
        rng = np.random.default_rng(seed)
        self.lens, self.vocab = np.asarray(lens), vocab
        self.off = np.concatenate([[0], np.cumsum(lens)])
        total = int(self.off[-1])
        self.extra = extra
        dtype = torch.bfloat16 if half else torch.float32
        logits = 2.0 * rng.standard_normal((total + extra, vocab))
        self.target = torch.softmax(torch.from_numpy(logits), -1).to(dtype)
        self.parents = None
        if kind == "tree":
            self.parents = np.concatenate([[int(rng.integers(0, t)) if t else -7 for t in range(n)] for n in lens]
                                          + [[0] * extra]).astype(np.int64)
        up = np.concatenate([[self.off[b] + (t - 1 if self.parents is None else self.parents[self.off[b] + t]) if t else -1
                              for t in range(n)] for b, n in enumerate(lens)] + [np.zeros(extra)]).astype(np.int64)
        from_row = logits[up]
        self.draft = None
        if kind == "drafts":
            from_row = agree * from_row + (1 - agree) * 3.0 * rng.standard_normal(from_row.shape)
            draft = torch.from_numpy(from_row)
            self.draft = torch.softmax(draft, -1).to(torch.bfloat16 if (half if draft_half is None else draft_half) else torch.float32)
        self.tokens = np.argmax(from_row + rng.gumbel(size=from_row.shape), -1)
        self.uniforms = torch.from_numpy(rng.random(total + extra, dtype=np.float32))
        self.kv = self.lens + rng.integers(0, 100, len(lens))
        self.slots = rng.permutation(5 * (total + extra))[:total + extra]

    def want(self):
        f = lambda t: None if t is None else t.double().numpy()  # noqa: E731
        kept, following, places = oracle.verify(f(self.target), self.tokens, self.off, f(self.uniforms), f(self.draft), self.parents)
        moved = np.full(len(places), -1)
        for b, lo in enumerate(self.off[:-1]):
            for t in range(self.lens[b]):
                if places[lo + t] not in (-1, t):
                    moved[lo + t] = self.slots[lo + places[lo + t]]
        return kept, following, places, self.kv - self.lens + kept, moved

    def kwargs(self, device="cuda"):
        dev = lambda t: None if t is None else t.to(device)  # noqa: E731
        return dict(target_probs=dev(self.target), tokens=i32(self.tokens, device), q_offsets=i32(self.off, device),
                    uniforms=dev(self.uniforms), draft_probs=dev(self.draft),
                    parents=None if self.parents is None else i32(self.parents, device), kv_lens=i32(self.kv, device),
                    slots=i32(self.slots, device))


def check(c, got):
    for name, g, w in zip(("accepted", "next", "places", "keep_lens", "keep_slots"), got, c.want()):
        assert g.cpu().tolist() == list(w), name


# ------------------------------------------------------------ the oracle (CPU)
def test_oracle_chain_keeps_the_targets_distribution():
    """Over many draws of draft and numbers, the first token after the root is distributed as the target's."""
    rng = np.random.default_rng(0)
    p, q = np.array([0.5, 0.2, 0.3, 0.0]), np.array([0.1, 0.6, 0.2, 0.1])
    n, first = 30000, np.zeros(4)
    for _ in range(n):
        x = rng.choice(4, p=q)
        kept, following, _ = oracle.verify(np.array([p, p]), [0, x], [0, 2], rng.random(2), np.array([q, q]))
        first[x if kept[0] == 2 else following[0]] += 1
    assert np.all(np.abs(first / n - p) < 5 * np.sqrt(p * (1 - p) / n) + 1e-12)


def test_oracle_siblings_keep_the_targets_distribution():
    rng = np.random.default_rng(1)
    p = np.array([0.5, 0.2, 0.25, 0.05])
    n, first = 30000, np.zeros(4)
    for _ in range(n):
        kids = rng.integers(0, 4, 3)  # the same token twice, at times
        kept, following, places = oracle.verify(np.tile(p, (4, 1)), [0, *kids], [0, 4], rng.random(4), None, [-1, 0, 0, 0])
        first[kids[int(np.argmax(places[1:] == 1))] if kept[0] == 2 else following[0]] += 1
    assert np.all(np.abs(first / n - p) < 5 * np.sqrt(p * (1 - p) / n) + 1e-12)


def test_oracle_by_hand():
    p = np.array([[0.0, 1.0, 0.0], [0.5, 0.0, 0.5], [1.0, 0.0, 0.0]])
    assert oracle.verify(p, [9, 1, 2], [0, 3], [0.4, 0.9, 0.7])[:2] == ([2], [0])  # 0.7 >= p[1][2]: token 0 is left
    assert oracle.verify(p, [9, 1, 2], [0, 3], [0.4, 0.9, 0.4])[:2] == ([3], [0])
    assert oracle.verify(p, [9, 0, 2], [0, 0, 3], [0.4, 0.0, 0.4])[:2] == ([0, 1], [-1, 1])


# ------------------------------------------------------------ refusals (CPU)
@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), 1), (dict(total=-1), 1), (dict(vocab=0), 1), (dict(th=2), 1), (dict(draft=1 << 20, parents=1 << 20), 1),
    (dict(batch=16385), 2), (dict(ts=99), 1), (dict(draft=1 << 20, ds=99), 1), (dict(target=None), 1), (dict(tokens=None), 1),
    (dict(uniforms=None), 1), (dict(places=None), 1), (dict(off=None), 1), (dict(kv=None), 1), (dict(slots=None), 1),
    (dict(target=(1 << 20) + 2), 3), (dict(tokens=(1 << 20) + 2), 3), (dict(ws=1 << 20, wsb=4), 4), (dict(ts=1 << 40), 2),
])
def test_rejects_bad_arguments_without_a_launch(jg, kw, code):
    a = dict(target=1 << 20, ts=100, th=0, draft=None, ds=100, dh=0, tokens=1 << 20, parents=None, uniforms=1 << 20, off=1 << 20,
             batch=2, total=5, vocab=100, kv=1 << 20, slots=1 << 20, accepted=1 << 21, next=1 << 21, places=1 << 21,
             keep=1 << 21, moved=1 << 21, ws=None, wsb=0, stream=None)
    a.update(kw)
    assert jg.load().jgdpa_verify(*a.values()) == code


@pytest.mark.parametrize("field,change,match", [
    ("target_probs", lambda t: t.half(), "fp32 or bf16"),
    ("target_probs", lambda t: t[0], "target_probs must be"),
    ("target_probs", lambda t: t.t().contiguous().t(), "contiguous inside"),
    ("target_probs", lambda t: t[:1].expand(t.shape), "must not overlap"),
    ("draft_probs", lambda t: t[:, :-1], "draft_probs must have shape"),
    ("tokens", lambda t: t.long(), "tokens must have dtype"),
    ("uniforms", lambda t: t.double(), "uniforms must have dtype"),
    ("parents", lambda t: i32([0] * 5, "cpu"), "parents must be None"),
    ("kv_lens", lambda t: t[:1], "kv_lens must have shape"),
    ("slots", lambda t: t[:1], "slots must have shape"),
    ("q_offsets", lambda t: t[:0], "batch \\+ 1"),
    ("tokens", lambda t: t, "CUDA device"),
])
def test_wrapper_rejects_bad_tensors(jg, field, change, match):
    kw = Case(0, [2, 3], 40, "drafts").kwargs("cpu")
    kw[field] = change(kw[field])
    with pytest.raises(ValueError, match=match):
        jg.jgdpa_verify(**kw)


# ------------------------------------------------------------ against the oracle (GPU)
@gpu
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("kind", ["chain", "drafts", "tree"])
@pytest.mark.parametrize("lens,vocab", [
    ([1], 7), ([5, 1, 0, 9, 2], 1), ([3, 3], 33), ([20, 64, 7], 500), ([4] * 40, 1000), ([2, 6, 1], 4097), ([6, 3], 50001),
    ([1, 0, 2] * 120, 20), ([40], 131072),
])
def test_verify(jg, kind, half, lens, vocab):
    c = Case(len(lens) + vocab, lens, vocab, kind, half, extra=3)
    check(c, jg.jgdpa_verify(**c.kwargs()))


@gpu
@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("kind", ["drafts", "tree"])
def test_many_requests(jg, kind, seed):
    """More requests than SMs, so that a row is one CTA's, and tokens from all over the vocabulary."""
    rng = np.random.default_rng(seed)
    c = Case(seed, rng.integers(0, 9, 400), 700 + seed, kind, agree=0.9)
    check(c, jg.jgdpa_verify(**c.kwargs()))


@gpu
def test_targets_and_drafts_of_different_types_and_padded_rows(jg):
    for half, draft_half in ((False, True), (True, False)):
        c = Case(5, [4, 7], 301, "drafts", half, draft_half)
        kw = c.kwargs()
        check(c, jg.jgdpa_verify(**kw))
        for name in ("target_probs", "draft_probs"):  # slices of wider rows
            wide = torch.full((11, 320), float("nan"), dtype=kw[name].dtype, device="cuda")
            wide[:, 5:306] = kw[name]
            kw[name] = wide[:, 5:306]
        check(c, jg.jgdpa_verify(**kw))
        kept, following, places, lens, moved = jg.jgdpa_verify(**{**kw, "kv_lens": None, "slots": None})
        assert lens is None and moved is None and kept.tolist() == list(c.want()[0])


@gpu
@pytest.mark.parametrize("kind", ["chain", "drafts", "tree"])
def test_numbers_at_the_ends(jg, kind):
    """0 keeps every token that the target may give; the largest below 1 draws the last token with any weight."""
    for u in (0.0, 1 - 2.0 ** -24):
        c = Case(11, [5, 9, 1], 6000, kind)
        c.target[:, -50:] = 0
        c.uniforms.fill_(u)
        check(c, jg.jgdpa_verify(**c.kwargs()))


@gpu
def test_draws_at_the_borders_between_tokens(jg):
    """Weights of 2^-16 each: the sums are exact, and a number that is a border's draws the token behind it."""
    n = 65536
    target = torch.full((512, n), 2.0 ** -16, device="cuda")
    at = torch.randperm(n, generator=torch.Generator().manual_seed(0))[:512]
    at[:3] = torch.tensor([0, 1, n - 1])
    u = (at.double() * 2.0 ** -16).float().cuda()
    off = torch.arange(513, dtype=torch.int32, device="cuda")
    got = jg.jgdpa_verify(target, off[:512], off, u)[1]
    assert torch.equal(got.cpu().long(), at)


@gpu
def test_sums_keep_more_than_fp32_holds(jg):
    """One weight of 1 and a million of 2^-26, which an fp32 sum with the 1 would lose."""
    n = 1 << 20
    target = torch.full((3, n), 2.0 ** -26, device="cuda")
    target[:, 0] = 1.0
    total = 1 + (n - 1) * 2.0 ** -26
    u = torch.tensor([0.5, 1 - 2.0 ** -8, 1 - 2.0 ** -20], device="cuda")
    got = jg.jgdpa_verify(target, i32([0, 0, 0]), i32([0, 1, 2, 3]), u)[1].cpu().tolist()
    for g, x in zip(got, u.double().cpu().tolist()):
        want = 0 if x * total < 1 else int(np.floor((x * total - 1) * 2.0 ** 26)) + 1
        assert g == want


@gpu
def test_rows_that_hold_little_or_nothing(jg):
    """Zeros, negatives, infinities and NaN count nothing; a residual with nothing left falls back to the row."""
    inf, nan = float("inf"), float("nan")
    p = torch.tensor([[0, 0, 0, 0], [nan, -1, 0.25, inf], [0.1, 0.2, 0.3, 0.4], [0.1, 0.2, 0.3, 0.4]])
    u, off, tokens = torch.tensor([0.5, 0.9, 0.99, 0.999]), [0, 1, 2, 4], [0, 0, 0, 1]
    q = torch.full((4, 4), 0.5)  # above the target everywhere
    for draft in (None, q):
        got = jg.jgdpa_verify(p.cuda(), i32(tokens), i32(off), u.cuda(), draft_probs=None if draft is None else draft.cuda())
        want = oracle.verify(p.double().numpy(), tokens, off, u.double().numpy(), None if draft is None else draft.double().numpy())
        assert [g.cpu().tolist() for g in got[:3]] == [list(w) for w in want]
        assert got[1].tolist()[:2] == [-1, 2]


@gpu
def test_siblings_with_the_same_token(jg):
    """A refused token's twin does not stay, and the token is not drawn either."""
    p = torch.zeros(6, 50)
    p[0, 7], p[0, 9], p[0, 11] = 0.5, 0.3, 0.2
    p[1:, 3] = 1.0
    tokens, parents = [0, 7, 7, 9, 7, 11], [0, 0, 0, 0, 0, 0]
    for us in ([0.0, 0.9, 0.0, 0.9, 0.0, 0.5], [0.0, 0.9, 0.0, 0.9, 0.0, 0.999], [0.3, 0.9, 0.0, 0.1, 0.0, 0.0]):
        u = torch.tensor(us)
        got = jg.jgdpa_verify(p.cuda(), i32(tokens), i32([0, 6]), u.cuda(), parents=i32(parents))
        want = oracle.verify(p.double().numpy(), tokens, [0, 6], u.double().numpy(), None, parents)
        assert [g.cpu().tolist() for g in got[:3]] == [list(w) for w in want]


@gpu
def test_longest_requests(jg):
    """1024 rows: a chain that stays whole, a wide root, and one row too many."""
    n, v = 1024, 64
    p = torch.zeros(n, v)
    tokens = np.arange(n) % v
    p[torch.arange(n - 1), torch.from_numpy(tokens[1:])] = 1.0
    p[n - 1, 5] = 1.0
    u = torch.full((n,), 0.5)
    got = jg.jgdpa_verify(p.cuda(), i32(tokens), i32([0, n]), u.cuda())
    assert got[0].tolist() == [n] and got[1].tolist() == [5] and got[2].tolist() == list(range(n))
    wide = torch.full((n + 1, 2000), 1 / 2000)
    u = torch.full((n + 1,), 1 - 2.0 ** -24)
    tokens = np.arange(n + 1)
    got = jg.jgdpa_verify(wide[:n].cuda(), i32(tokens[:n]), i32([0, n]), u[:n].cuda(), parents=i32([0] * n))
    want = oracle.verify(wide[:n].double().numpy(), tokens[:n], [0, n], u[:n].double().numpy(), None, [0] * n)
    assert [g.cpu().tolist() for g in got[:3]] == [list(w) for w in want]
    ws = torch.empty(jg.jgdpa_verify_workspace_bytes(), dtype=torch.uint8, device="cuda")
    got = jg.jgdpa_verify(wide.cuda(), i32(tokens), i32([0, n + 1]), u.cuda(), kv_lens=i32([5000]), workspace=ws)
    assert jg.jgdpa_read_device_status(ws) == 6
    assert got[0].tolist() == [0] and got[1].tolist() == [-1] and torch.all(got[2] == -1) and got[3].tolist() == [5000]


@gpu
def test_device_detected_errors(jg):
    c = Case(3, [3, 4], 100, "tree")
    kw = c.kwargs()
    ws = torch.empty(jg.jgdpa_verify_workspace_bytes(), dtype=torch.uint8, device="cuda")
    check(c, jg.jgdpa_verify(**kw, workspace=ws))
    assert jg.jgdpa_read_device_status(ws) == 0
    for off in ([1, 3, 7], [0, 8, 7], [0, 3, 8], [0, -2, 7], [0, 3, 2 ** 31 - 1]):
        got = jg.jgdpa_verify(**{**kw, "q_offsets": i32(off)}, workspace=ws)
        assert jg.jgdpa_read_device_status(ws) == 6
        assert all(torch.all(g < 10 ** 6) for g in got[:1])
    for field, bad in (("tokens", 100), ("tokens", -1), ("tokens", 2 ** 31 - 1), ("parents", 2), ("parents", -1), ("parents", 2 ** 31 - 1)):
        values = np.array(c.tokens if field == "tokens" else c.parents)
        values[5] = bad  # row 2 of the second request
        d = Case(3, [3, 4], 100, "tree")
        setattr(d, field, values)
        check(d, jg.jgdpa_verify(**{**kw, field: i32(values)}, workspace=ws))
        assert jg.jgdpa_read_device_status(ws) == 6, (field, bad)
    kw["tokens"][0] = -5  # a root's token is not looked at
    check(c, jg.jgdpa_verify(**kw, workspace=ws))
    assert jg.jgdpa_read_device_status(ws) == 0


@gpu
def test_offsets_that_do_not_start_at_0_are_reported(jg):
    p, u = torch.full((3, 10), 0.1, device="cuda"), torch.zeros(3, device="cuda")
    ws = torch.empty(jg.jgdpa_verify_workspace_bytes(), dtype=torch.uint8, device="cuda")
    got = jg.jgdpa_verify(p, i32([0, 0, 0]), i32([3, 3]), u, workspace=ws)  # a request without rows
    assert jg.jgdpa_read_device_status(ws) == 6 and got[0].tolist() == [0]


@gpu
def test_empty_calls(jg):
    p, u = torch.full((3, 10), 0.1, device="cuda"), torch.zeros(3, device="cuda")
    got = jg.jgdpa_verify(p, i32([0, 0, 0]), i32([0]), u, kv_lens=i32([]), slots=i32([1, 2, 3]))
    assert got[0].numel() == got[3].numel() == 0 and torch.all(got[2] == -1) and torch.all(got[4] == -1)
    got = jg.jgdpa_verify(p[:0], i32([]), i32([0, 0]), u[:0], kv_lens=i32([9]))
    assert got[0].tolist() == [0] and got[1].tolist() == [-1] and got[3].tolist() == [9]


@gpu
def test_same_bits_in_graphs_and_on_other_streams(jg):
    cs = [Case(30, [5, 9, 2], 40000, "drafts"), Case(31, [17, 30], 9000, "tree", True)]
    kws = [c.kwargs() for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in kws]
    for _ in range(4):
        outs = [jg.jgdpa_verify(**kw, stream=s) for kw, s in zip(kws, streams)]
        torch.cuda.synchronize()
        for c, o in zip(cs, outs):
            check(c, o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [jg.jgdpa_verify(**kw) for kw in kws]
    for _ in range(2):
        for o in outs:
            for t in o:
                t.fill_(77)
        graph.replay()
        torch.cuda.synchronize()
        for c, o in zip(cs, outs):
            check(c, o)
