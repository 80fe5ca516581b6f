"""The calls around the attention together, as a server and a training step use them."""

import numpy as np
import pytest
import torch

gpu = pytest.mark.gpu
U = 2.0 ** -8  # half a step of bf16, relative


@pytest.fixture(scope="module")
def jg():
    from jagged_gdpa_gb300 import build as b
    b.build()
    import jagged_gdpa_gb300 as m
    return m


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int64).astype(np.int32), device="cuda")


@gpu
@pytest.mark.parametrize("bits", [16, 4])
def test_speculative_serving(jg, bits):
    """Prompts, then trees of drafted tokens that are verified, moved and continued: what the cache holds
    at the end attends as the packed forward does over the tokens that stayed, rotated at their places."""
    rng = np.random.default_rng(bits)
    batch, heads, kv_heads, d, page, pool, width, vocab = 3, 4, 2, 64, 16, 60, 20, 50
    if bits == 16:
        kc = torch.full((pool, page, kv_heads, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        vc = kc.clone()
    else:
        four = [torch.full((pool, kv_heads, page, n), 255 if t is torch.uint8 else float("nan"), dtype=t, device="cuda")
                for n, t in ((d // 2, torch.uint8), (2, torch.bfloat16)) * 2]
    table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    free, count, held = torch.arange(pool, dtype=torch.int32, device="cuda"), i32([pool]), i32([0] * batch)
    freq = torch.from_numpy((10000.0 ** (-np.arange(32) / 32)).astype(np.float32)).cuda()
    w = torch.from_numpy((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)).cuda()
    ws = torch.empty(jg.jgdpa_norm_rotate_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    history = [[torch.zeros(0, h, d, dtype=torch.bfloat16, device="cuda") for h in (heads, kv_heads, kv_heads)] for _ in range(batch)]
    ctx, sizes = i32([0] * batch), [[20, 1, 33], [5, 7, 1], [6, 2, 9], [4, 4, 4]]
    for step, new in enumerate(sizes):
        total = sum(new)
        q, k, v = (torch.from_numpy(rng.standard_normal((total, h, d), dtype=np.float32)).to(torch.bfloat16).cuda()
                   for h in (heads, kv_heads, kv_heads))
        slots, q_off, kv, held, count = jg.jgdpa_cache_plan(ctx, i32(new), held, table, free, count, page, total)
        mask = parents = depths = None
        if step:  # trees; a prompt is a chain that all stays
            up = [[-1] + [int(rng.integers(0, t)) for t in range(1, n)] for n in new]
            seen, depth = [], []
            for p in up:
                for t, x in enumerate(p):
                    seen.append((seen[len(seen) - t + x] if t else 0) | 1 << t)
                    depth.append(depth[len(depth) - t + x] + 1 if t else 0)
            mask, parents, depths = i32(seen).view(-1, 1), i32(sum(up, [])), i32(depth)

        def write(to):
            if bits == 16:
                return jg.jgdpa_cache_append_rotated(q, k, v, to, kc, vc, q_off, kv, freq, w, w, depths=depths, workspace=ws)[0]
            places = torch.cat([c + (torch.arange(n, device="cuda") if depths is None else depths[o:o + n])
                                for c, n, o in zip(ctx.tolist(), new, q_off.tolist())]).int()
            qr, kr = jg.jgdpa_norm_rotate(q, k, None, None, freq, w, w, q_positions=places, k_positions=places)
            jg.jgdpa_cache4_append(kr, v, to, *four)
            return qr

        qr = write(slots)
        args = (table, q_off, kv, "softmax", d ** -0.5)
        opts = dict(max_q=max(new), tree_mask=mask, depths=depths)
        out, _ = jg.jgdpa_cache_fwd(qr, kc, vc, *args, **opts) if bits == 16 else jg.jgdpa_cache4_fwd(qr, *four, *args, **opts)
        assert torch.isfinite(out).all()
        probs = torch.softmax(torch.from_numpy(rng.standard_normal((total, vocab))).float().cuda(), -1)
        tokens = torch.from_numpy(rng.integers(0, vocab, total).astype(np.int32)).cuda()
        u = torch.from_numpy(rng.random(total, dtype=np.float32)).cuda()
        if step == 0:
            u.zero_()  # everything stays
        else:
            u *= 0.1
        kept, following, places, ctx_next, moves = jg.jgdpa_verify(probs, tokens, q_off, u, parents=parents, kv_lens=kv, slots=slots)
        if step == 0:
            assert kept.tolist() == new
        write(moves)
        o, place = q_off.tolist(), places.tolist()
        for b in range(batch):
            rows = sorted((r for r in range(o[b], o[b + 1]) if place[r] >= 0), key=lambda r: place[r])
            assert [place[r] for r in rows] == list(range(kept.tolist()[b]))
            history[b] = [torch.cat([h, x[rows]]) for h, x in zip(history[b], (q, k, v))]
            assert ctx_next.tolist()[b] == len(history[b][0])
        assert all(0 <= x < vocab for x in following.tolist())
        ctx = ctx_next
    # one more token each, against the packed calls over the whole history
    new, total = [1] * batch, batch
    q, k, v = (torch.from_numpy(rng.standard_normal((total, h, d), dtype=np.float32)).to(torch.bfloat16).cuda()
               for h in (heads, kv_heads, kv_heads))
    slots, q_off, kv, held, count = jg.jgdpa_cache_plan(ctx, i32(new), held, table, free, count, page, total)
    depths = None
    qr = write(slots)
    args = (table, q_off, kv, "softmax", d ** -0.5, 1)
    out, _ = jg.jgdpa_cache_fwd(qr, kc, vc, *args) if bits == 16 else jg.jgdpa_cache4_fwd(qr, *four, *args)
    for b in range(batch):
        hq, hk, hv = (torch.cat([h, x[b:b + 1]]) for h, x in zip(history[b], (q, k, v)))
        off = i32([0, len(hq)])
        hq, hk = jg.jgdpa_norm_rotate(hq, hk, off, off, freq, w, w)
        if bits == 4:  # the same roundings to 4 bits; what the codes stand for is rounded once more for the packed call
            four_b = [torch.zeros(1 + len(hk) // 16, kv_heads, 16, n, dtype=t, device="cuda") for n, t in ((d // 2, torch.uint8), (2, torch.bfloat16)) * 2]
            jg.jgdpa_cache4_append(hk, hv, i32(range(len(hk))), *four_b)
            hk, hv = jg.jgdpa_cache4_read(*four_b, i32(range(len(hk))))
        rep = heads // kv_heads
        hk, hv = hk.repeat_interleave(rep, 1), hv.repeat_interleave(rep, 1)
        want, _ = jg.jgdpa_fwd(hq, hk, hv, off, off, "softmax", d ** -0.5, causal=True)
        x = torch.einsum("hd,khd->hk", hq[-1].float(), hk.float()) * d ** -0.5
        size = torch.einsum("hk,khd->hd", torch.softmax(x, -1), hv.float().abs())
        # P and O rounded on both sides; 4 bits: a score off by u sum |q||k| s, and V by u, on the packed side
        dot = torch.einsum("hd,khd->hk", hq[-1].float().abs(), hk.float().abs()).amax(1, keepdim=True) * d ** -0.5
        tol = (4 * U + 2.0 ** -10 + (0 if bits == 16 else U + 2 * U * dot)) * size
        assert torch.all((out[b].float() - want[-1].float()).abs() <= tol)


@gpu
def test_a_training_step(jg):
    """norm_rotate in front of the packed attention and its backward behind: gradients of queries, keys and
    weights against autograd in 64 bits through the same steps' roundings."""
    rng = np.random.default_rng(3)
    off, heads, d = [0, 70, 71, 200], 2, 64
    x = [torch.from_numpy(rng.standard_normal((200, heads, d), dtype=np.float32)).to(torch.bfloat16).cuda() for _ in range(4)]
    q, k, v, dout = x
    w = [torch.from_numpy((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)).cuda() for _ in range(2)]
    freq = torch.from_numpy((10000.0 ** (-np.arange(32) / 32)).astype(np.float32)).cuda()
    offs = i32(off)
    qr, kr = jg.jgdpa_norm_rotate(q, k, offs, offs, freq, *w)
    out, lse = jg.jgdpa_fwd(qr, kr, v, offs, offs, "softmax", d ** -0.5, causal=True)
    dqr, dkr, dv, _ = jg.jgdpa_bwd(qr, kr, v, out, lse, dout, offs, offs, "softmax", d ** -0.5, causal=True)
    got = jg.jgdpa_norm_rotate_bwd(dqr, dkr, q, k, offs, offs, freq, *w)

    leaves = [t.double().requires_grad_() for t in (q, k, *w)]
    pos = torch.cat([torch.arange(b - a) for a, b in zip(off, off[1:])]).double().cuda()
    c, s = (f(pos[:, None, None] * freq.double()) for f in (torch.cos, torch.sin))

    def turn(x, w):
        h = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
        a, b = h[..., :32], h[..., 32:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    tq, tk = turn(leaves[0], leaves[2]), turn(leaves[1], leaves[3])
    loss = 0
    for a, b in zip(off, off[1:]):
        sc = torch.einsum("qhd,khd->hqk", tq[a:b], tk[a:b]) * d ** -0.5
        sc = sc.masked_fill(torch.ones(b - a, b - a, device="cuda").triu(1).bool(), -torch.inf)
        o = torch.einsum("hqk,khd->qhd", torch.softmax(sc, -1), v[a:b].double())
        loss = loss + (o * dout[a:b].double()).sum()
    loss.backward()
    for g, t in zip(got, leaves):
        # the attention's own bound for its gradients, 2e-2 of the largest
        assert (g.double() - t.grad).abs().max() <= 2e-2 * t.grad.abs().max()
