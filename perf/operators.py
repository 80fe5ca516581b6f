"""Work of the paged key/value cache: page plans, cache writes, attention over the cache.

Each case is one call of a serving step: `plan` hands out pages and slots for
the tokens a step adds, `append` writes their keys and values into the pages,
`attend` attends from the new tokens (one per request, or a tree of drafted
ones) over each request's pages.
"""

import numpy as np
import torch

own = False

DEV = "cuda"


def listed():
    """Cases from single decode steps of a few requests to full prefill steps."""
    return [
        # a decode step of a small server: one token for each of 8 requests
        plan("plan decode b8", batch=8, page=16, width=256, new_lo=1, new_hi=1, lens=1),
        # a speculative step: drafted trees, a share of the requests ending or cut back to what was accepted
        plan("plan tree b256", batch=256, page=16, width=1024, new_lo=1, new_hi=64, lens=2, ended=0.1),
        # prompts of 64 requests admitted in one step
        plan("plan prefill b64", batch=64, page=64, width=256, new_lo=100, new_hi=8192, lens=3, fresh=True),
        # the rows of one decode step
        append("append decode r32", rows=32, heads=8, dim=128, page=16, lens=4),
        # drafted trees, keys and values as slices of a fused projection's output, some rows rejected
        append("append tree r2047", rows=2047, heads=4, dim=64, page=32, lens=5, fused=True, skipped=0.3),
        # a prefill step
        append("append prefill r32768", rows=32768, heads=8, dim=128, page=64, lens=6),
        # four users of a ranking model, one candidate each, GELU scores with a distance bias
        attend("one b4 gelu d64", batch=4, new_lo=1, new_hi=1, ctx_lo=16, ctx_hi=1000, heads=8, group=1, dim=64,
               page=16, act="gelu", bias=257, lens=7),
        # the decode step of a middling batch, lengths spread evenly
        attend("one b64 softmax d128", batch=64, new_lo=1, new_hi=1, ctx_lo=0, ctx_hi=8192, heads=8, group=4, dim=128,
               page=16, act="softmax", lens=8),
        # one request with a very long history
        attend("one long softmax d128", batch=1, new_lo=1, new_hi=1, ctx_lo=131071, ctx_hi=131071, heads=8, group=8,
               dim=128, page=64, act="softmax", lens=9),
        # trees of drafted tokens, long-tailed lengths
        attend("tree b32 softmax d128", batch=32, new_lo=8, new_hi=33, ctx_lo=100, ctx_hi=16384, tail=True, heads=8,
               group=4, dim=128, page=32, act="softmax", tree=True, lens=10),
        # many drafted candidates a user against long histories: products bound it
        attend("tree b64 gelu d128", batch=64, new_lo=64, new_hi=64, ctx_lo=1, ctx_hi=8192, heads=4, group=8, dim=128,
               page=64, act="gelu", bias=257, tree=True, lens=11),
        # short drafts under a sliding window, small heads
        attend("draft b128 silu d32 window", batch=128, new_lo=1, new_hi=8, ctx_lo=0, ctx_hi=8000, heads=16, group=1,
               dim=32, page=128, act="silu", window=1024, lens=12),
    ]


def plan(name, batch, page, width, new_lo, new_hi, lens, ended=0.0, fresh=False):
    return case(name, op="plan", batch=batch, page=page, width=width, new_lo=new_lo, new_hi=new_hi, lens=lens,
                ended=ended, fresh=fresh)


def append(name, rows, heads, dim, page, lens, fused=False, skipped=0.0):
    return case(name, op="append", rows=rows, heads=heads, dim=dim, page=page, lens=lens, fused=fused,
                skipped=skipped)


def attend(name, batch, new_lo, new_hi, ctx_lo, ctx_hi, heads, group, dim, page, act, lens, bias=0, window=0,
           tree=False, tail=False):
    return case(name, op="attend", batch=batch, new_lo=new_lo, new_hi=new_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi,
                heads=heads, group=group, dim=dim, page=page, act=act, lens=lens, bias=bias, window=window,
                tree=tree, tail=tail)


def case(name, **kw):
    if name:
        kw["name"] = name
    return kw


def spread(rng, lo, hi):
    """An integer of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(np.exp(rng.uniform(np.log(lo), np.log(hi + 0.49)))))))


def draw(rng):
    lens = rng.randrange(100, 1 << 30)
    kind = rng.choice(("plan", "append", "attend", "attend", "attend"))
    if kind == "plan":
        batch, page, fresh = spread(rng, 1, 1024), rng.choice((16, 32, 64, 128)), rng.random() < 0.3
        most = min(8192, (1 << 18) // batch) if fresh else 64
        width = max(1 + most // page, rng.randrange(4, 1024))
        return plan("", batch, page, width, 1, spread(rng, 1, most), lens, rng.choice((0.0, 0.1, 0.5)), fresh)
    if kind == "append":
        return append("", spread(rng, 1, 32768), spread(rng, 1, 8), rng.choice((32, 64, 128)),
                      rng.choice((16, 32, 64, 128)), lens, rng.random() < 0.5, rng.choice((0.0, 0.2)))
    dim, heads, group = rng.choice((32, 64, 128)), rng.choice((1, 2, 4, 5, 8)), rng.choice((1, 2, 3, 4, 7, 8))
    act = rng.choice(("gelu", "silu", "softmax"))
    batch = spread(rng, 1, 64)
    ctx = spread(rng, 1, min(65536, (1 << 19) // batch))
    new = spread(rng, 1, 64)
    return attend("", batch, 1, new, ctx // 3 if rng.random() < 0.5 else 0, ctx, heads, group, dim,
                  rng.choice((16, 32, 64, 128)), act, lens, rng.choice((0, 0, 129, 257)),
                  spread(rng, 16, 4096) if rng.random() < 0.25 else 0, rng.random() < 0.6, rng.random() < 0.3)


def lengths(case):
    """(tokens kept, tokens added) of each request, the same for every seed up to their order."""
    r = np.random.RandomState(case["lens"])
    batch = case["batch"]
    new = r.randint(case["new_lo"], case["new_hi"] + 1, batch)
    if case["op"] == "plan":
        room = case["width"] * case["page"] - new
        ctx = np.zeros(batch, np.int64) if case["fresh"] else (r.rand(batch) * (room + 1)).astype(np.int64)
        over = r.randint(0, 3, batch)  # pages still held from the drafts of the last step
        held = np.minimum(-(-ctx // case["page"]) + over, case["width"])
        held = np.where(case["fresh"], 0, held)
        gone = r.rand(batch) < case["ended"]
        return np.where(gone, 0, ctx), np.where(gone, 0, new), held
    if case["tail"]:
        mid = np.log(max(2.0, np.sqrt(max(1, case["ctx_lo"]) * case["ctx_hi"])))
        ctx = np.clip(np.round(r.lognormal(mid, 1.0, batch)), case["ctx_lo"], case["ctx_hi"]).astype(np.int64)
    else:
        ctx = r.randint(case["ctx_lo"], case["ctx_hi"] + 1, batch)
    if batch == 1 and not case["tail"]:
        ctx = np.full(1, case["ctx_hi"])
    return ctx, new, None


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).to(DEV)


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)


def prepare(case, seed):
    r = np.random.RandomState(seed % (1 << 32))
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    if case["op"] == "append":
        rows, heads, dim, page = case["rows"], case["heads"], case["dim"], case["page"]
        pages = -(-rows // page) + 3
        slots = r.permutation(pages)[: -(-rows // page)]
        slots = (slots[:, None] * page + np.arange(page)).reshape(-1)[:rows]  # whole pages in a shuffled order
        slots = np.where(r.rand(rows) < case["skipped"], -1, slots)
        wide = normal(g, rows, 3 if case["fused"] else 2, heads, dim)
        k, v = wide[:, -2], wide[:, -1]
        return {"op": "append", "k": k if case["fused"] else k.contiguous(), "v": v if case["fused"] else v.contiguous(),
                "slots": ints(slots), "kc": normal(g, pages, page, heads, dim), "vc": normal(g, pages, page, heads, dim)}
    ctx, new, held = lengths(case)
    order = r.permutation(len(ctx))
    ctx, new = ctx[order], new[order]
    page = case["page"]
    if case["op"] == "plan":
        held = held[order]
        want = -(-(ctx + new) // page)
        pages = int(held.sum() + np.maximum(0, want - held).sum()) + 5
        ids = r.permutation(pages)
        table = np.full((len(ctx), case["width"]), -1)
        at = np.arange(case["width"])[None] < held[:, None]
        table[at] = ids[: held.sum()]
        free = np.full(pages, -1)
        free[: pages - held.sum()] = ids[held.sum():]
        return {"op": "plan", "ctx": ints(ctx), "new": ints(new), "held": ints(held), "table": ints(table),
                "free": ints(free), "count": ints([pages - held.sum()]), "total": int(new.sum()), "page": page}
    heads, group, dim = case["heads"], case["group"], case["dim"]
    kv = ctx + new
    need = -(-kv // page)
    pages = int(need.sum()) + 3
    table = np.zeros((len(kv), int(need.max())))
    table[np.arange(table.shape[1])[None] < need[:, None]] = r.permutation(pages)[: need.sum()]
    off = np.concatenate([[0], np.cumsum(new)])
    total, most = int(off[-1]), int(case["new_hi"])
    depth = mask = None
    if case["tree"]:  # each drafted token but a request's first continues one drafted before it
        words = -(-most // 32)
        depth = np.zeros((len(kv), most), np.int64)
        seen = np.zeros((len(kv), most, words * 32), bool)
        for t in range(most):
            if t:
                up = (r.rand(len(kv)) * t).astype(np.int64)
                depth[:, t] = depth[np.arange(len(kv)), up] + 1
                seen[:, t] = seen[np.arange(len(kv)), up]
            seen[:, t, t] = True
        live = np.arange(most)[None] < new[:, None]
        bits = (seen[live].reshape(total, words, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1)
        mask = torch.from_numpy(bits.astype(np.uint32).view(np.int32)).to(DEV)
        depth = ints(depth[live])
    bias = 0.1 * torch.randn(heads * group, case["bias"], generator=g, device=DEV) if case["bias"] else None
    return {"op": "attend", "q": normal(g, total, heads * group, dim), "kc": normal(g, pages, page, heads, dim),
            "vc": normal(g, pages, page, heads, dim), "table": ints(table), "off": ints(off), "kv": ints(kv),
            "most": most, "act": case["act"], "scale": dim ** -0.5, "bias": bias, "window": case["window"],
            "mask": mask, "depth": depth}


def run(state):
    s = state
    if own:
        import jagged_gdpa_gb300 as jg
        if s["op"] == "plan":
            got = jg.jgdpa_cache_plan(s["ctx"], s["new"], s["held"], s["table"], s["free"], s["count"], s["page"],
                                      s["total"])
            return *got, s["table"], s["free"]
        if s["op"] == "append":
            return jg.jgdpa_cache_append(s["k"], s["v"], s["slots"], s["kc"], s["vc"])
        out, lse = jg.jgdpa_cache_fwd(s["q"], s["kc"], s["vc"], s["table"], s["off"], s["kv"], s["act"], s["scale"],
                                      max_q=s["most"], bias_table=s["bias"], window=s["window"], tree_mask=s["mask"],
                                      depths=s["depth"])
        return out if lse is None else (out, lse)
    return {"plan": plain_plan, "append": plain_append, "attend": plain_attend}[s["op"]](s)


def plain_plan(s):
    page, ctx, held, table, free = s["page"], s["ctx"].long(), s["held"].long(), s["table"], s["free"]
    kv = ctx + s["new"]
    want = (kv + page - 1) // page
    grow, back = (want - held).clamp(min=0), (held - want).clamp(min=0)
    n = s["count"].long()
    top = n + back.sum()
    at = torch.arange(table.shape[1], device=DEV)
    # the stack with the returned pages on it; entries of no interest go behind its end
    place = n + (back.cumsum(0) - back)[:, None] + at - want[:, None]
    place = torch.where((at >= want[:, None]) & (at < held[:, None]), place, free.numel())
    stack = torch.cat([free, free[:1]]).scatter(0, place.reshape(-1), table.reshape(-1))[:-1]
    taken = top - 1 - (grow.cumsum(0) - grow)[:, None] - at + held[:, None]
    fresh = (at >= held[:, None]) & (at < want[:, None])
    table.copy_(torch.where(fresh, stack[torch.where(fresh, taken, 0)], table))
    count = top - grow.sum()
    free.copy_(torch.where(torch.arange(free.numel(), device=DEV) < count, stack, free))
    off = torch.cat([torch.zeros_like(kv[:1]), s["new"].long().cumsum(0)])
    row = torch.arange(s["total"], device=DEV)
    b = torch.searchsorted(off, row, right=True) - 1
    pos = ctx[b] + row - off[b]
    slots = table[b, pos // page].long() * page + pos % page
    return slots.int(), off.int(), kv.int(), want.int(), count.int(), table, free


def plain_append(s):
    kc, vc = s["kc"].flatten(0, 1), s["vc"].flatten(0, 1)
    row = torch.nonzero(s["slots"] >= 0)[:, 0]
    to = s["slots"][row].long()
    kc[to] = s["k"][row]
    vc[to] = s["v"][row]
    return s["kc"], s["vc"]


def plain_attend(s):
    q, off, kv, table = s["q"], s["off"].long(), s["kv"].long(), s["table"].long()
    batch, most, (heads, dim) = len(kv), s["most"], s["kc"].shape[2:]
    group = q.shape[1] // heads
    new = off[1:] - off[:-1]
    ctx = kv - new
    t = torch.arange(most, device=DEV)
    row = (off[:-1, None] + t).clamp(max=len(q) - 1)  # [batch, most]
    j = torch.arange(table.shape[1] * s["kc"].shape[1], device=DEV)
    u = j - ctx[:, None]  # [batch, keys]: which of the new tokens a key is
    x = q[row].float().view(batch, most, heads, group, dim).permute(0, 2, 3, 1, 4).reshape(batch, heads, -1, dim)
    k = s["kc"][table].float().view(batch, len(j), heads, dim).permute(0, 2, 3, 1)
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
        p = torch.exp(x - lse[..., None].clamp(min=-1e30))
    else:
        p = x * torch.sigmoid(x) if s["act"] == "silu" else x * 0.5 * (1 + torch.erf(x * 0.5 ** 0.5))
        p = p.masked_fill(~seen, 0.0)
    v = s["vc"][table].float().view(batch, len(j), heads, dim).masked_fill((j >= kv[:, None])[:, :, None, None], 0.0)
    o = p.view(batch, heads, group * most, len(j)) @ v.transpose(1, 2)
    b = torch.searchsorted(off, torch.arange(len(q), device=DEV), right=True) - 1
    at = torch.arange(len(q), device=DEV) - off[b]
    o = o.view(batch, heads, group, most, dim).permute(0, 3, 1, 2, 4)[b, at].reshape(q.shape).to(q.dtype)
    if s["act"] != "softmax":
        return o
    return o, lse.permute(0, 3, 1, 2)[b, at].reshape(len(q), -1).t().contiguous()


def work(case):
    if case["op"] == "append":
        rows = round(case["rows"] * (1 - case["skipped"]))
        return {"bytes": 8 * rows * case["heads"] * case["dim"] + 4 * case["rows"], "flops": 0}
    ctx, new, held = lengths(case)
    want = -(-(ctx + new) // case["page"])
    if case["op"] == "plan":
        moved = np.abs(want - held).sum()
        return {"bytes": int(4 * (6 * len(ctx) + new.sum() + 3 * moved)), "flops": 0}
    keys = ctx + new if not case["window"] else np.minimum(ctx, case["window"] - 1) + new
    width = case["heads"] * case["dim"]
    pairs = int((new * (keys - new) + new * (new + 1) // 2).sum())
    total, group = int(new.sum()), case["group"]
    return {"bytes": int(4 * width * keys.sum() + 4 * width * group * total + 4 * want.sum()),
            "flops": 4 * pairs * width * group}


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "append":
        both = []
        for new, cache in ((s["k"], s["kc"]), (s["v"], s["vc"])):
            got = cache.double().flatten(0, 1)
            live = s["slots"] >= 0
            got.index_copy_(0, s["slots"][live].long(), new[live].double())
            both.append(got.view(cache.shape))
        return tuple(both)
    off, kv, heads, dim = s["off"].tolist(), s["kv"].tolist(), *s["kc"].shape[2:]
    group, page = s["q"].shape[1] // heads, s["kc"].shape[1]
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
        for h in range(heads):
            k, v = (c[ids, :, h].reshape(-1, dim)[:length].double() for c in (s["kc"], s["vc"]))
            for m in range(h * group, h * group + group):
                x = s["q"][lo:hi, m].double() @ k.t() * s["scale"]
                if s["bias"] is not None:
                    reach = s["bias"].shape[1] // 2
                    x += s["bias"][m].double()[apart.clamp(-reach, reach) + reach]
                if s["act"] == "softmax":
                    x = x.masked_fill(~sees, -torch.inf)
                    lse[m, lo:hi] = torch.logsumexp(x, 1)
                    p = torch.softmax(x, 1)
                else:
                    p = x / (1 + torch.exp(-x)) if s["act"] == "silu" else x * torch.special.ndtr(x)
                    p = p * sees
                out[lo:hi, m] = p @ v
    return (out, lse) if s["act"] == "softmax" else out
