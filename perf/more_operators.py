"""Work around the attention calls: norms and rotation of queries and keys, rotated
cache writes, verification of drafted tokens, a cache held in 4 bits.

Each case is one call: `rotate` and `rotate_bwd` are what a training step runs in
front of and behind the packed attention, `write` is a serving step's write into
the paged cache with the rotation on the way, `verify` decides which drafted
tokens stay and draws the next one, `write4` (a write, and the cache read back as
rows for the packed attention) and `attend4` are the cache in 4 bits.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6


def listed():
    """Cases from a server's smallest steps to full training batches."""
    return [
        # a small ranking batch: four short histories, latency
        rotate("rotate b4 d64", batch=4, law="even", lo=1, hi=60, heads=4, kv=4, dim=64, lens=1),
        # the long-tailed training batch
        rotate("rotate long tail d128", batch=64, law="tail", lo=100, hi=16384, heads=8, kv=8, dim=128, lens=2),
        # a causal batch of middling lengths, queries and keys as slices of a fused projection, half the columns rotated
        rotate("back b256 d128 fused", batch=256, law="even", lo=1, hi=1024, heads=8, kv=2, dim=128, lens=3, back=True,
               fused=True, part=2, pairs=True),
        # the long-tailed training batch's backward pass
        rotate("back long tail d128", batch=64, law="tail", lo=100, hi=16384, heads=8, kv=8, dim=128, lens=2, back=True),
        # the decode step of a middling batch
        write("write decode b64", batch=64, new_lo=1, new_hi=1, ctx=131072, heads=32, kv=8, dim=128, page=16, lens=4),
        # prompts admitted in one step, without norms
        write("write prefill r16500", batch=9, new_lo=1000, new_hi=2700, ctx=0, heads=16, kv=4, dim=64, page=64, lens=5,
              norm=False, pairs=True),
        # chains of drafted tokens with the draft model's probabilities
        verify("verify chain b64", batch=64, new_lo=2, new_hi=6, vocab=128000, lens=6, drafts=True),
        # trees of drafted tokens, probabilities in bf16, a small server
        verify("verify tree b8", batch=8, new_lo=8, new_hi=33, vocab=50001, lens=7, tree=True, half=True),
        # a speculative step's rows into the 4-bit cache, some of them rejected
        write4("write4 tree r2047", rows=2047, heads=4, dim=64, page=32, lens=8, skipped=0.3),
        # a prefill step
        write4("write4 prefill r32768", rows=32768, heads=8, dim=128, page=64, lens=9),
        # the decode step of a middling batch, lengths spread evenly
        attend4("one4 b64 softmax d128", batch=64, new_lo=1, new_hi=1, ctx_lo=0, ctx_hi=8192, heads=8, group=4, dim=128,
                page=16, act="softmax", lens=10),
        # trees of drafted tokens over histories, GELU scores with a distance bias
        attend4("tree4 b16 gelu d64", batch=16, new_lo=2, new_hi=16, ctx_lo=100, ctx_hi=6000, heads=8, group=2, dim=64,
                page=32, act="gelu", bias=257, tree=True, lens=11),
    ]


def rotate(name, batch, law, lo, hi, heads, kv, dim, lens, back=False, fused=False, part=1, pairs=False, norm=True):
    return case(name, op="rotate_bwd" if back else "rotate", batch=batch, law=law, lo=lo, hi=hi, heads=heads, kv=kv,
                dim=dim, lens=lens, fused=fused, part=part, pairs=pairs, norm=norm)


def write(name, batch, new_lo, new_hi, ctx, heads, kv, dim, page, lens, norm=True, pairs=False, tree=False):
    return case(name, op="write", batch=batch, new_lo=new_lo, new_hi=new_hi, ctx_lo=0, ctx_hi=ctx, heads=heads, kv=kv,
                dim=dim, page=page, lens=lens, norm=norm, pairs=pairs, tree=tree, part=1)


def verify(name, batch, new_lo, new_hi, vocab, lens, drafts=False, tree=False, half=False):
    return case(name, op="verify", batch=batch, new_lo=new_lo, new_hi=new_hi, ctx_lo=0, ctx_hi=4000, vocab=vocab,
                lens=lens, drafts=drafts, tree=tree, half=half)


def write4(name, rows, heads, dim, page, lens, skipped=0.0):
    return case(name, op="write4", rows=rows, heads=heads, dim=dim, page=page, lens=lens, skipped=skipped)


def attend4(name, batch, new_lo, new_hi, ctx_lo, ctx_hi, heads, group, dim, page, act, lens, bias=0, window=0,
            tree=False):
    return case(name, op="attend4", batch=batch, new_lo=new_lo, new_hi=new_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi,
                heads=heads, group=group, dim=dim, page=page, act=act, lens=lens, bias=bias, window=window, tree=tree)


def case(name, **kw):
    if name:
        kw["name"] = name
    return kw


def spread(rng, lo, hi):
    """An integer of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    lens = rng.randrange(100, 1 << 30)
    kind = rng.choice(("rotate", "rotate_bwd", "write", "verify", "write4", "attend4", "attend4"))
    dim = rng.choice((32, 64, 128))
    if kind in ("rotate", "rotate_bwd"):
        kv, batch = rng.choice((1, 2, 3, 4, 8)), spread(rng, 1, 512)
        heads = kv * rng.choice((1, 1, 2, 4))
        most = max(1, min(16384, (1 << 28) // (batch * heads * dim)))
        return rotate("", batch, rng.choice(("even", "tail")), 1, spread(rng, 1, most), heads, kv, dim, lens,
                      kind == "rotate_bwd", rng.random() < 0.5, rng.choice((1, 1, 2)), rng.random() < 0.4,
                      rng.random() < 0.8)
    if kind == "write":
        kv, batch = rng.choice((1, 2, 4, 5, 8)), spread(rng, 1, 256)
        return write("", batch, 1, spread(rng, 1, min(2048, 16384 // batch)), rng.choice((0, 1000, 131072)),
                     kv * rng.choice((1, 2, 4, 7)), kv, dim, rng.choice((16, 32, 64, 128)), lens, rng.random() < 0.7,
                     rng.random() < 0.4, rng.random() < 0.4)
    if kind == "verify":
        vocab = spread(rng, 100, 160000)
        new = spread(rng, 1, 32)
        batch = spread(rng, 1, max(1, min(256, (1 << 26) // (vocab * new))))
        tree = rng.random() < 0.5
        return verify("", batch, 1, new, vocab, lens, not tree and rng.random() < 0.7, tree, rng.random() < 0.4)
    if kind == "write4":
        return write4("", spread(rng, 1, 32768), spread(rng, 1, 8), dim, rng.choice((16, 32, 64, 128)), lens,
                      rng.choice((0.0, 0.2)))
    batch = spread(rng, 1, 64)
    ctx = spread(rng, 1, min(65536, (1 << 18) // batch))
    return attend4("", batch, 1, spread(rng, 1, 16), ctx // 3 if rng.random() < 0.5 else 0, ctx,
                   rng.choice((1, 2, 4, 5, 8)), rng.choice((1, 2, 3, 4, 7, 8)), dim, rng.choice((16, 32, 64, 128)),
                   rng.choice(("gelu", "silu", "softmax", "softmax")), lens, rng.choice((0, 0, 129, 257)),
                   spread(rng, 16, 4096) if rng.random() < 0.25 else 0, rng.random() < 0.5)


def lengths(case):
    """(tokens kept, tokens added) of each request, or (None, rows) of each segment: the same for every seed."""
    r = np.random.RandomState(case["lens"])
    batch = case["batch"]
    if case["op"].startswith("rotate"):
        if case["law"] == "even":
            return None, r.randint(case["lo"], case["hi"] + 1, batch)
        middle = math.log(max(1.0, math.sqrt(max(1, case["lo"]) * case["hi"])))
        return None, np.clip(np.round(r.lognormal(middle, 1.0, batch)), case["lo"], case["hi"]).astype(np.int64)
    new = r.randint(case["new_lo"], case["new_hi"] + 1, batch)
    return r.randint(case["ctx_lo"], case["ctx_hi"] + 1, batch), new


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).to(DEV)


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)


def weight(g, dim):
    return 1.0 + 0.2 * torch.randn(dim, generator=g, device=DEV)


def frequencies(dim, part):
    n = dim // 2 // part
    return torch.from_numpy((10000.0 ** (-np.arange(n) / n)).astype(np.float32)).to(DEV)


def trees(r, new, most):
    """Parents, depths and who sees whom of random trees of drafted tokens: each but the first continues one before it."""
    batch = len(new)
    up, depth = np.full((batch, most), -1), np.zeros((batch, most), np.int64)
    seen = np.zeros((batch, most, -(-most // 32) * 32), bool)
    at = np.arange(batch)
    for t in range(most):
        if t:
            up[:, t] = (r.rand(batch) * t).astype(np.int64)
            depth[:, t] = depth[at, up[:, t]] + 1
            seen[:, t] = seen[at, up[:, t]]
        seen[:, t, t] = True
    live = np.arange(most)[None] < new[:, None]
    words = seen.shape[2] // 32
    bits = (seen[live].reshape(-1, words, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1)
    return ints(up[live]), ints(depth[live]), torch.from_numpy(bits.astype(np.uint32).view(np.int32)).to(DEV)


def prepare(case, seed):
    r = np.random.RandomState(seed % (1 << 32))
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    op = case["op"]
    if op.startswith("rotate"):
        return prepare_rotate(case, r, g)
    if op == "write4":
        rows, heads, dim, page = case["rows"], case["heads"], case["dim"], case["page"]
        pages = -(-rows // page) + 3
        slots = r.permutation(pages)[: -(-rows // page)]
        slots = (slots[:, None] * page + np.arange(page)).reshape(-1)[:rows]  # whole pages in a shuffled order
        slots = np.where(r.rand(rows) < case["skipped"], -1, slots)
        return {"op": op, "k": normal(g, rows, heads, dim), "v": normal(g, rows, heads, dim), "slots": ints(slots),
                "cache": cache4(g, pages, heads, page, dim), "all": torch.arange(pages * page, dtype=torch.int32, device=DEV)}
    ctx, new = lengths(case)
    order = r.permutation(len(ctx))
    ctx, new = ctx[order], new[order]
    kv, off = ctx + new, np.concatenate([[0], np.cumsum(new)])
    total, most = int(off[-1]), int(new.max())
    up = depth = mask = None
    if case["tree"]:
        up, depth, mask = trees(r, new, most)
    s = {"op": op, "off": ints(off), "kv": ints(kv), "total": total, "most": most, "depth": depth, "mask": mask}
    if op == "verify":
        return {**s, **prepare_verify(case, off, new, up, g)}
    dim, page = case["dim"], case["page"]
    if op == "write":
        heads, kv_heads = case["heads"], case["kv"]
        need = -(-kv // page) - ctx // page  # pages that the new tokens lie in
        pages = int(need.sum()) + 3
        ids, first = r.permutation(pages), np.concatenate([[0], np.cumsum(need)])
        slots = np.concatenate([ids[first[b] + np.arange(ctx[b] % page, ctx[b] % page + new[b]) // page] * page
                                + np.arange(ctx[b], kv[b]) % page for b in range(len(kv))])
        wide = normal(g, total, heads + 2 * kv_heads, dim)  # a fused projection's output
        return {**s, "q": wide[:, :heads], "k": wide[:, heads:heads + kv_heads], "v": wide[:, heads + kv_heads:],
                "slots": ints(slots), "kc": normal(g, pages, page, kv_heads, dim),
                "vc": normal(g, pages, page, kv_heads, dim), "freq": frequencies(dim, case["part"]),
                "qw": weight(g, dim) if case["norm"] else None, "kw": weight(g, dim) if case["norm"] else None,
                "eps": EPS if case["norm"] else None, "pairs": case["pairs"]}
    heads, group = case["heads"], case["group"]
    need = -(-kv // page)
    pages = int(need.sum()) + 3
    table = np.zeros((len(kv), int(need.max())))
    table[np.arange(table.shape[1])[None] < need[:, None]] = r.permutation(pages)[: need.sum()]
    bias = 0.1 * torch.randn(heads * group, case["bias"], generator=g, device=DEV) if case["bias"] else None
    return {**s, "q": normal(g, total, heads * group, dim), "cache": cache4(g, pages, heads, page, dim),
            "table": ints(table), "act": case["act"], "scale": dim ** -0.5, "bias": bias, "window": case["window"]}


def prepare_rotate(case, r, g):
    _, rows = lengths(case)
    rows = rows[r.permutation(len(rows))]
    off = np.concatenate([[0], np.cumsum(rows)])
    heads, kv, dim, total = case["heads"], case["kv"], case["dim"], int(off[-1])
    if case["fused"]:
        wide = normal(g, total, heads + 2 * kv, dim)
        q, k = wide[:, :heads], wide[:, heads:heads + kv]
    else:
        q, k = normal(g, total, heads, dim), normal(g, total, kv, dim)
    s = {"op": case["op"], "q": q, "k": k, "off": ints(off), "freq": frequencies(dim, case["part"]),
         "qw": weight(g, dim) if case["norm"] else None, "kw": weight(g, dim) if case["norm"] else None,
         "eps": EPS if case["norm"] else None, "pairs": case["pairs"]}
    if case["op"] == "rotate_bwd":
        s["dq"], s["dk"] = normal(g, total, heads, dim), normal(g, total, kv, dim)
    return s


def prepare_verify(case, off, new, up, g):
    """Probabilities as a model's softmax gives them, drafted tokens drawn from the draft's, or from the target's own."""
    total, vocab = int(off[-1]), case["vocab"]
    first = torch.from_numpy(np.repeat(off[:-1], new)).to(DEV)
    row = torch.arange(total, device=DEV)
    parent = row - 1 if up is None else first + up.long()
    parent = torch.where(row == first, row, parent)
    logits = 2.0 * torch.randn(total, vocab, generator=g, device=DEV)
    p = torch.softmax(logits, -1)
    q = None
    logits = logits[parent]  # what a row's token was drafted from
    if case["drafts"]:
        logits += 0.7 * torch.randn(total, vocab, generator=g, device=DEV)
        q = torch.softmax(logits, -1)
    logits -= torch.log(torch.empty_like(logits).exponential_(generator=g))
    tokens = logits.argmax(-1).int()
    kind = torch.bfloat16 if case["half"] else torch.float32
    slots = torch.randperm(total, generator=g, device=DEV).int()
    return {"p": p.to(kind), "q": None if q is None else q.to(kind), "tokens": tokens, "up": up, "slots": slots,
            "u": torch.rand(total, generator=g, device=DEV)}


def cache4(g, pages, heads, page, dim):
    """Codes and (step, middle) pairs of keys, and of values, as writes of normal rows leave them."""
    def half():
        codes = torch.randint(0, 256, (pages, heads, page, dim // 2), generator=g, device=DEV, dtype=torch.uint8)
        scales = torch.stack([0.25 + 0.2 * torch.rand(pages, heads, page, generator=g, device=DEV),
                              0.3 * torch.randn(pages, heads, page, generator=g, device=DEV)], -1)
        return codes, scales.bfloat16()
    return *half(), *half()


def run(state):
    s = state
    if own:
        import jagged_gdpa_gb300 as jg
        if s["op"] == "rotate":
            return jg.jgdpa_norm_rotate(s["q"], s["k"], s["off"], s["off"], s["freq"], s["qw"], s["kw"], s["eps"],
                                        interleaved=s["pairs"])
        if s["op"] == "rotate_bwd":
            got = jg.jgdpa_norm_rotate_bwd(s["dq"], s["dk"], s["q"], s["k"], s["off"], s["off"], s["freq"], s["qw"],
                                           s["kw"], s["eps"], interleaved=s["pairs"])
            return [x for x in got if x is not None]
        if s["op"] == "write":
            return jg.jgdpa_cache_append_rotated(s["q"], s["k"], s["v"], s["slots"], s["kc"], s["vc"], s["off"], s["kv"],
                                                 s["freq"], s["qw"], s["kw"], s["eps"], interleaved=s["pairs"],
                                                 depths=s["depth"])
        if s["op"] == "verify":
            return jg.jgdpa_verify(s["p"], s["tokens"], s["off"], s["u"], draft_probs=s["q"], parents=s["up"],
                                   kv_lens=s["kv"], slots=s["slots"])
        if s["op"] == "write4":
            jg.jgdpa_cache4_append(s["k"], s["v"], s["slots"], *s["cache"])
            return jg.jgdpa_cache4_read(*s["cache"], s["all"])
        out, lse = jg.jgdpa_cache4_fwd(s["q"], *s["cache"], s["table"], s["off"], s["kv"], s["act"], s["scale"],
                                       max_q=s["most"], bias_table=s["bias"], window=s["window"], tree_mask=s["mask"],
                                       depths=s["depth"])
        return out if lse is None else (out, lse)
    return {"rotate": plain_rotate, "rotate_bwd": plain_rotate_bwd, "write": plain_write, "verify": plain_verify,
            "write4": plain_write4, "attend4": plain_attend4}[s["op"]](s)


def segment_positions(off, rows):
    row = torch.arange(rows, device=DEV)
    return row - off.long()[torch.searchsorted(off.long(), row, right=True) - 1]


def angles(positions, freq):
    """cos and sin [rows, 1, pairs], the angles in 64 bits: far positions lose them in 32."""
    a = positions.double()[:, None, None] * freq.double()
    return torch.cos(a).float(), torch.sin(a).float()


def turn(x, cos, sin, pairs):
    n = cos.shape[-1]
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if pairs else (x[..., :n], x[..., n:2 * n])
    c, d = a * cos - b * sin, b * cos + a * sin
    both = torch.stack([c, d], -1).flatten(-2) if pairs else torch.cat([c, d], -1)
    return torch.cat([both, x[..., 2 * n:]], -1)


def plain_norm_turn(x, w, eps, cos, sin, pairs):
    h = x.float()
    if eps is not None:
        h = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + eps)
        h = h if w is None else h * w
    return turn(h, cos, sin, pairs).to(x.dtype)


def plain_rotate(s):
    cos, sin = angles(segment_positions(s["off"], len(s["q"])), s["freq"])
    return (plain_norm_turn(s["q"], s["qw"], s["eps"], cos, sin, s["pairs"]),
            plain_norm_turn(s["k"], s["kw"], s["eps"], cos, sin, s["pairs"]))


def plain_rotate_bwd(s):
    cos, sin = angles(segment_positions(s["off"], len(s["q"])), s["freq"])
    grads, weights = [], []
    for x, w, dy in ((s["q"], s["qw"], s["dq"]), (s["k"], s["kw"], s["dk"])):
        g = turn(dy.float(), cos, -sin, s["pairs"])
        if s["eps"] is None:
            grads.append(g.to(x.dtype))
            continue
        x = x.float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"])
        h = x * r
        if w is not None:
            weights.append((g * h).sum((0, 1)))
            g = g * w
        grads.append((r * (g - h * (g * h).mean(-1, keepdim=True))).to(dy.dtype))
    return grads + weights


def plain_write(s):
    off, kv = s["off"].long(), s["kv"].long()
    row = torch.arange(s["total"], device=DEV)
    b = torch.searchsorted(off, row, right=True) - 1
    place = row - off[b]
    at = kv[b] - (off[b + 1] - off[b]) + (place if s["depth"] is None else s["depth"].long())
    cos, sin = angles(at, s["freq"])
    q = plain_norm_turn(s["q"], s["qw"], s["eps"], cos, sin, s["pairs"])
    k = plain_norm_turn(s["k"], s["kw"], s["eps"], cos, sin, s["pairs"])
    live = torch.nonzero(s["slots"] >= 0)[:, 0]
    to = s["slots"][live].long()
    s["kc"].flatten(0, 1)[to] = k[live]
    s["vc"].flatten(0, 1)[to] = s["v"][live]
    return q, s["kc"], s["vc"]


def plain_verify(s):
    p, tokens, u, off, total = s["p"], s["tokens"].long(), s["u"].double(), s["off"].long(), s["total"]
    batch, most = len(off) - 1, s["most"]
    rows = off[1:] - off[:-1]
    t = torch.arange(most, device=DEV)
    live = t < rows[:, None]  # [batch, most]
    at = (off[:-1, None] + t).clamp(max=total - 1)
    up = (t - 1).expand(batch, most) if s["up"] is None else s["up"].long()[at]
    up = torch.where(t > 0, up, 0).clamp(min=0)
    token = tokens[at]
    from_row = at.gather(1, up)
    pt = p[from_row, token].double()
    if s["q"] is not None:
        ok = u[at] * s["q"][at, token].double() < pt
    else:  # what is left of the parent's probability after the children before this one, a token counted once
        before = (up[:, :, None] == up[:, None, :]) & (t[:, None] > t) & (t > 0) & live[:, None, :]
        same = token[:, :, None] == token[:, None, :]
        first = ~(before & same).any(-1)  # the first child with its token
        gone = torch.where(before & first[:, None, :], pt[:, None, :], 0.0).sum(-1)
        ok = first & (u[at] * (1 - gone) < pt)
    ok = ok & live & (t > 0)
    # of a row's accepted children the first; on the path if all its ancestors are
    chosen = ok & ~((up[:, :, None] == up[:, None, :]) & (t[:, None] > t) & ok[:, None, :]).any(-1)
    step = torch.where(chosen, up, most)
    step[:, 0] = 0
    step = torch.cat([step, torch.full_like(step[:, :1], most)], 1)
    place = (step != t.new_tensor(most)).long()
    place[:, 0] = 0
    for _ in range(max(1, most - 1).bit_length()):  # pointer doubling; `most` stands for a row that is not on the path
        place = place + place.gather(1, step)
        step = step.gather(1, step)
    on = (step[:, :most] == 0) & live
    place = place[:, :most]
    kept = on.sum(1)
    last = torch.where(on, place, -1).argmax(1)
    end = at.gather(1, last[:, None])[:, 0]
    rest = p[end].float()
    refused = live & ~ok & (up == last[:, None]) & (t > 0)
    if s["q"] is not None:
        bad = refused & (t == last[:, None] + 1)
        bad_row = torch.where(bad.any(1), at.gather(1, bad.int().argmax(1, keepdim=True))[:, 0], 0)
        rest = torch.where(bad.any(1)[:, None], rest - s["q"][bad_row].float(), rest).clamp(min=0)
    else:
        b, c = torch.nonzero(refused, as_tuple=True)
        rest[b, token[b, c]] = 0.0
    cum = rest.double().cumsum(1)
    drawn = (cum > (u[off[:-1].clamp(max=total - 1)] * cum[:, -1])[:, None]).int().argmax(1)
    where = torch.nonzero(live, as_tuple=True)
    places = torch.where(on, place, -1)[where]
    to = s["slots"][off[:-1, None] + place.clamp(max=most - 1)][where]
    moved = torch.where((places >= 0) & (places != t.expand(batch, most)[where]), to, -1)
    return kept.int(), drawn.int(), places.int(), (s["kv"] - rows + kept).int(), moved.int()


def values(codes, scales):
    """What 4-bit codes stand for: low nibbles are the even columns, (step, middle) of each token and head."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    return scales[..., 1:].float() + scales[..., :1].float() * (c - 8)


def plain_write4(s):
    kc, ks, vc, vs = s["cache"]
    page, live = kc.shape[2], torch.nonzero(s["slots"] >= 0)[:, 0]
    to = s["slots"][live].long()
    for new, codes, scales in ((s["k"], kc, ks), (s["v"], vc, vs)):
        x = new[live].float()
        lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
        step = ((hi - lo) / 15).bfloat16()
        middle = (lo + 8 * step.float()).bfloat16()
        c = torch.where(step > 0, (x - middle.float()) / step.float(), 0.0)
        c = (torch.round(c) + 8).clamp(0, 15).to(torch.uint8)
        codes[to // page, :, to % page] = c[..., 0::2] | (c[..., 1::2] << 4)
        scales[to // page, :, to % page] = torch.cat([step, middle], -1)
    at = s["all"].long()
    return tuple(values(c[at // page, :, at % page], z[at // page, :, at % page]).bfloat16()
                 for c, z in ((kc, ks), (vc, vs)))


def plain_attend4(s):
    q, off, kv, table = s["q"], s["off"].long(), s["kv"].long(), s["table"].long()
    kc, ks, vc, vs = s["cache"]
    batch, most, heads, page, dim = len(kv), s["most"], kc.shape[1], kc.shape[2], 2 * kc.shape[3]
    group = q.shape[1] // heads
    new = off[1:] - off[:-1]
    ctx = kv - new
    t = torch.arange(most, device=DEV)
    row = (off[:-1, None] + t).clamp(max=len(q) - 1)  # [batch, most]
    j = torch.arange(table.shape[1] * page, device=DEV)
    u = j - ctx[:, None]  # [batch, keys]: which of the new tokens a key is
    x = q[row].float().view(batch, most, heads, group, dim).permute(0, 2, 3, 1, 4).reshape(batch, heads, -1, dim)
    k = values(kc[table], ks[table]).permute(0, 2, 4, 1, 3).reshape(batch, heads, dim, len(j))
    x = (x @ k).view(batch, heads, group, most, len(j)) * s["scale"]
    new_at = u.clamp(0, most - 1)
    if s["mask"] is None:
        seen = u[:, None] <= t[:, None]
    else:
        word = s["mask"][row]  # [batch, most, words]
        word = word.gather(2, (new_at // 32)[:, None].expand(batch, most, len(j)))
        seen = (u[:, None] < 0) | ((word >> (new_at % 32)[:, None]) & 1).bool()
    seen = seen & (j < kv[:, None])[:, None]
    depth = t.expand(batch, most) if s["depth"] is None else s["depth"].long()[row]
    apart = (ctx[:, None] + depth)[:, :, None] - torch.where(u < 0, j, ctx[:, None] + depth.gather(1, new_at))[:, None]
    if s["window"]:
        seen = seen & (apart.abs() < s["window"])
    if s["bias"] is not None:
        reach = s["bias"].shape[1] // 2
        bias = s["bias"][:, apart.clamp(-reach, reach) + reach].view(heads, group, batch, most, len(j))
        x = x + bias.permute(2, 0, 1, 3, 4)
    seen = seen[:, None, None]
    if s["act"] == "softmax":
        x = x.masked_fill(~seen, -torch.inf)
        lse = x.logsumexp(-1)
        w = torch.exp(x - lse[..., None].clamp(min=-1e30))
    else:
        w = x * torch.sigmoid(x) if s["act"] == "silu" else x * 0.5 * torch.erfc(-x * 0.5 ** 0.5)
        w = w.masked_fill(~seen, 0.0)
    v = values(vc[table], vs[table]).permute(0, 2, 1, 3, 4).reshape(batch, heads, len(j), dim)
    o = w.view(batch, heads, group * most, len(j)) @ v
    b = torch.searchsorted(off, torch.arange(len(q), device=DEV), right=True) - 1
    at = torch.arange(len(q), device=DEV) - off[b]
    o = o.view(batch, heads, group, most, dim).permute(0, 3, 1, 2, 4)[b, at].reshape(q.shape).to(q.dtype)
    if s["act"] != "softmax":
        return o
    return o, lse.permute(0, 3, 1, 2)[b, at].reshape(len(q), -1).t().contiguous()


def work(case):
    op, dim = case["op"], case.get("dim", 0)
    if op.startswith("rotate"):
        values_of_both = int(lengths(case)[1].sum()) * (case["heads"] + case["kv"]) * dim
        reads = 1 if op == "rotate" or not case["norm"] else 2
        return {"bytes": 2 * values_of_both * (reads + 1) + 4 * case["batch"], "flops": 0}
    if op == "write4":
        pieces = 2 * round(case["rows"] * (1 - case["skipped"])) * case["heads"]
        back = 2 * (-(-case["rows"] // case["page"]) + 3) * case["page"] * case["heads"]
        return {"bytes": (pieces + back) * (2 * dim + dim // 2 + 4) + 4 * case["rows"], "flops": 0}
    ctx, new = lengths(case)
    total, keys = int(new.sum()), ctx + new
    if op == "write":
        return {"bytes": total * (4 * dim * (case["heads"] + 2 * case["kv"]) + 4) + 8 * len(new), "flops": 0}
    if op == "verify":
        wide, both = (2 if case["half"] else 4), (2 if case["drafts"] else 1)
        return {"bytes": wide * both * (len(new) * case["vocab"] + total) + 20 * total + 20 * len(new), "flops": 0}
    if case["window"]:
        keys = np.minimum(ctx, case["window"] - 1) + new
    heads, group = case["heads"], case["group"]
    pairs = int((new * (keys - new) + new * (new + 1) // 2).sum())
    return {"bytes": int(2 * heads * (dim // 2 + 4) * keys.sum() + 4 * heads * dim * group * total
                         + 4 * (-(-(ctx + new) // case["page"])).sum()),
            "flops": 4 * pairs * heads * dim * group}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "verify":
        return None  # whole numbers
    if op.startswith("rotate"):
        lens = (s["off"][1:] - s["off"][:-1]).tolist()
        position = torch.cat([torch.arange(n, device=DEV) for n in lens])
        return exact_rotate(s, position) if op == "rotate" else exact_rotate_bwd(s, position)
    if op == "write":
        off, kv = s["off"].tolist(), s["kv"].tolist()
        inside = [torch.arange(b - a, device=DEV) for a, b in zip(off, off[1:])]
        if s["depth"] is not None:
            inside = s["depth"].long().split([len(i) for i in inside])
        position = torch.cat([n - (b - a) + i for n, a, b, i in zip(kv, off, off[1:], inside)])
        q, k = exact_rotate(s, position)
        live = s["slots"] >= 0
        caches = []
        for new, cache in ((k, s["kc"]), (s["v"].double(), s["vc"])):
            got = cache.double().flatten(0, 1)
            got.index_copy_(0, s["slots"][live].long(), new[live])
            caches.append(got.view(cache.shape))
        return q, *caches
    if op == "write4":  # by the definition's own roundings: fp32 steps, bf16 step and middle
        out = []
        for new, codes, scales in ((s["k"], *s["cache"][:2]), (s["v"], *s["cache"][2:])):
            got = exact_values(codes, scales).transpose(1, 2).flatten(0, 1).contiguous()
            live = s["slots"] >= 0
            x = new[live].double()
            lo = x.min(-1).values[..., None]
            step = ((x.max(-1).values[..., None] - lo).float() / 15).bfloat16().double()
            middle = (lo + 8 * step).float().bfloat16().double()
            c = torch.nan_to_num((x - middle) / step).round().clamp(-8, 7)
            got.index_copy_(0, s["slots"][live].long(), middle + step * c)
            out.append(got)
        return tuple(out)
    return exact_attend4(s)


def exact_rotate(s, position):
    angle = position.double()[:, None] * s["freq"].double()
    turned = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        y = x.double()
        if s["eps"] is not None:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / y.shape[-1] + s["eps"])
            y = y * w.double()
        n = angle.shape[1]
        i, j = torch.arange(n, device=DEV), torch.arange(n, 2 * n, device=DEV)
        if s["pairs"]:
            i, j = 2 * i, 2 * i + 1
        z = torch.complex(y[..., i], y[..., j]) * torch.polar(torch.ones_like(angle), angle)[:, None]
        y[..., i], y[..., j] = z.real, z.imag
        turned.append(y)
    return tuple(turned)


def exact_rotate_bwd(s, position):
    angle = position.double()[:, None] * s["freq"].double()
    n = angle.shape[1]
    i, j = torch.arange(n, device=DEV), torch.arange(n, 2 * n, device=DEV)
    if s["pairs"]:
        i, j = 2 * i, 2 * i + 1
    grads, weights = [], []
    for x, w, dy in ((s["q"], s["qw"], s["dq"]), (s["k"], s["kw"], s["dk"])):
        g = dy.double()
        z = torch.complex(g[..., i], g[..., j]) * torch.polar(torch.ones_like(angle), -angle)[:, None]
        g[..., i], g[..., j] = z.real, z.imag
        if s["eps"] is not None:
            x = x.double()
            size = torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + s["eps"])
            weights.append((g * x / size).sum(0).sum(0))
            g = g * w.double()
            g = g / size - x * ((g * x).sum(-1, keepdim=True) / x.shape[-1]) / size ** 3
        grads.append(g)
    return grads + weights


def exact_values(codes, scales):
    d = torch.empty(*codes.shape[:3], 2 * codes.shape[3], dtype=torch.float64, device=DEV)
    d[..., 0::2], d[..., 1::2] = (codes % 16).double(), (codes // 16).double()
    return (d - 8) * scales[..., 0, None].double() + scales[..., 1, None].double()


def exact_attend4(s):
    off, kv = s["off"].tolist(), s["kv"].tolist()
    kc, ks, vc, vs = s["cache"]
    heads, page, dim = kc.shape[1], kc.shape[2], 2 * kc.shape[3]
    group = s["q"].shape[1] // heads
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["q"].shape[1], len(s["q"]), dtype=torch.float64, device=DEV)
    for b, length in enumerate(kv):
        lo, hi = off[b], off[b + 1]
        ids = s["table"][b, : -(-length // page)].long()
        old = length - (hi - lo)
        tokens = torch.arange(hi - lo, device=DEV)
        sees = torch.ones(hi - lo, length, dtype=torch.bool, device=DEV)
        sees[:, old:] = (tokens[None] <= tokens[:, None] if s["mask"] is None else
                         (s["mask"][lo:hi, tokens // 32] >> (tokens % 32)) & 1 == 1)
        place = torch.arange(length, device=DEV)
        place[old:] = old + (tokens if s["depth"] is None else s["depth"][lo:hi].long())
        apart = place[old:, None] - place[None]
        if s["window"]:
            sees &= apart.abs() < s["window"]
        k, v = (exact_values(c[ids], z[ids]).transpose(0, 1).reshape(heads, -1, dim)[:, :length]
                for c, z in ((kc, ks), (vc, vs)))
        for m in range(heads * group):
            x = s["q"][lo:hi, m].double() @ k[m // group].t() * s["scale"]
            if s["bias"] is not None:
                reach = s["bias"].shape[1] // 2
                x += s["bias"][m].double()[apart.clamp(-reach, reach) + reach]
            if s["act"] == "softmax":
                x = x.masked_fill(~sees, -torch.inf)
                lse[m, lo:hi] = torch.logsumexp(x, 1)
                w = torch.softmax(x, 1)
            else:
                w = (x / (1 + torch.exp(-x)) if s["act"] == "silu" else x * torch.special.ndtr(x)) * sees
            out[lo:hi, m] = w @ v[m // group]
    return (out, lse) if s["act"] == "softmax" else out
