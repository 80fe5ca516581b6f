"""Norms of queries and keys with the rotation by position: packed rows, their
gradients, and rows on their way into the paged cache."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import step as oracle

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


def f64(t):
    return t.detach().double().cpu().numpy()


def normal(rng, *shape, device="cuda"):
    return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32)).to(torch.bfloat16).to(device)


def freqs(n, device="cuda"):
    return torch.from_numpy((10000.0 ** (-np.arange(n) / n)).astype(np.float32)).to(device)


def weights(rng, d, device="cuda"):
    return torch.from_numpy((1 + 0.3 * rng.standard_normal(d)).astype(np.float32)).to(device)


def pair_size(h, n, interleaved):
    """|a| + |b| of each column's pair (|h| where it has none)."""
    a, b = oracle.pair_columns(n, interleaved)
    size = np.abs(h)
    both = size[..., a] + size[..., b]
    size[..., a] = size[..., b] = both
    return size


def check_rotated(got, x, pos, freq, w, eps, interleaved, rows=None):
    """Within bf16's rounding of the result, and of |a| + |b| of its pair:
    2^-20 for each of sine and cosine (2^-21.1 by the hardware, 2^-22 from the
    angle), and 2^-18 for the norm (a sum of d <= 128 squares in fp32, a reciprocal
    root and three products)."""
    x, w = f64(x), None if w is None else f64(w)
    want = oracle.norm_rotate(x, pos, f64(freq), w, eps, interleaved)
    h = x if eps is None else oracle.norm(x, w, eps)
    tol = U * np.abs(want) + 2.0 ** -17 * pair_size(h, len(freq), interleaved) + 1e-37
    rows = slice(None) if rows is None else rows
    bad = ~(np.abs(f64(got) - want) <= tol)[rows]
    assert not bad.any(), f"{bad.sum()} of {bad.size}"


# ------------------------------------------------------------ the oracle (CPU)
@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_gradients_by_differences_and_autograd(interleaved):
    rng = np.random.default_rng(0)
    x, dy, w = rng.standard_normal((3, 2, 32)), rng.standard_normal((3, 2, 32)), 1 + 0.2 * rng.standard_normal(32)
    pos, freq, eps = [0, 5, 70000], 0.7 ** np.arange(8), 1e-3
    dx, dw, _ = oracle.norm_rotate_bwd(dy, x, pos, freq, w, eps, interleaved)

    def loss(x, w):
        return np.sum(dy * oracle.norm_rotate(x, pos, freq, w, eps, interleaved))

    for at in [(0, 0, 0), (1, 1, 9), (2, 0, 31), (2, 1, 17)]:
        e = np.zeros_like(x)
        e[at] = 1e-6
        assert abs((loss(x + e, w) - loss(x - e, w)) / 2e-6 - dx[at]) < 1e-7
    for i in (0, 8, 31):
        e = np.zeros_like(w)
        e[i] = 1e-6
        assert abs((loss(x, w + e) - loss(x, w - e)) / 2e-6 - dw[i]) < 1e-7
    tx, tw = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    h = tx * torch.rsqrt(tx.square().mean(-1, keepdim=True) + eps) * tw
    a, b = oracle.pair_columns(8, interleaved)
    z = torch.complex(h[..., a], h[..., b]) * torch.polar(torch.ones(3, 1, 8, dtype=torch.float64),
                                                          torch.tensor(np.array(pos)[:, None, None] * freq))
    rest = [c for c in range(32) if c not in a and c not in b]
    y = (z.real * torch.tensor(dy[..., a])).sum() + (z.imag * torch.tensor(dy[..., b])).sum()
    (y + (h[..., rest] * torch.tensor(dy[..., rest])).sum()).backward()
    assert np.allclose(tx.grad.numpy(), dx, atol=1e-12) and np.allclose(tw.grad.numpy(), dw, atol=1e-11)


def test_oracle_rotation_by_hand():
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    quarter = np.array([np.pi / 2])
    assert np.allclose(oracle.rotate(x, [1], quarter, True), [[[-2.0, 1.0, 3.0, 4.0]]])
    assert np.allclose(oracle.rotate(x, [1], np.array([np.pi / 2, np.pi]), False), [[[-3.0, -2.0, 1.0, -4.0]]])


# ------------------------------------------------------------ refusals (CPU)
def _args(**kw):
    a = dict(q=1 << 20, qs=256, qo=1 << 21, qos=256, tq=4, heads=4, q_off=1 << 20, q_pos=None, qw=None, k=1 << 20, ks=128,
             ko=1 << 21, kos=128, tk=4, kv_heads=2, k_off=1 << 20, k_pos=None, kw=None, batch=1, d=64, freq=1 << 20, pairs=32,
             inter=0, norm=1, eps=1e-6, ws=None, wsb=0, stream=None)
    a.update(kw)
    a["eps"] = ctypes.c_float(a["eps"])
    return list(a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(d=48), 2), (dict(pairs=0), 1), (dict(pairs=33), 1), (dict(pairs=12), 2), (dict(inter=2), 1), (dict(norm=2), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(norm=0, qw=1 << 20), 1), (dict(freq=None), 1), (dict(q=None), 1),
    (dict(ko=None), 1), (dict(qs=248), 1), (dict(kos=132), 3), (dict(q=(1 << 20) + 8), 3), (dict(q_off=None), 1),
    (dict(tq=-1), 1), (dict(heads=0), 1), (dict(batch=-1), 1), (dict(tq=1 << 31), 2), (dict(tq=1 << 30), 2),
    (dict(ws=1 << 20, wsb=16), 4), (dict(ws=(1 << 20) + 16, wsb=256), 3), (dict(q_off=(1 << 20) + 2), 3), (dict(ks=1 << 40), 2),
    (dict(batch=2 ** 31 - 1), 2),
])
def test_rejects_bad_arguments_without_a_launch(jg, kw, code):
    assert jg.load().jgdpa_norm_rotate(*_args(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dq_out=None), 1), (dict(q=None), 1), (dict(dq=None), 1), (dict(dqw=1 << 20), 4), (dict(norm=0, dqw=1 << 20), 1),
    (dict(dks=120), 1), (dict(dkw=(1 << 20) + 2, ws=1 << 20, wsb=1 << 30), 3), (dict(pairs=20), 2), (dict(d=16), 2),
])
def test_bwd_rejects_bad_arguments_without_a_launch(jg, kw, code):
    a = dict(dq_out=1 << 20, dqos=256, q=1 << 20, qs=256, dq=1 << 21, dqs=256, tq=4, heads=4, q_off=1 << 20, q_pos=None,
             qw=None, dqw=None, dk_out=1 << 20, dkos=128, k=1 << 20, ks=128, dk=1 << 21, dks=128, tk=4, kv_heads=2,
             k_off=1 << 20, k_pos=None, kw=None, dkw=None, batch=1, d=64, freq=1 << 20, pairs=32, inter=0, norm=1, eps=1e-6,
             ws=None, wsb=0, stream=None)
    a.update(kw)
    a["eps"] = ctypes.c_float(a["eps"])
    got = jg.load().jgdpa_norm_rotate_bwd(*a.values())
    # (a call that needs the number of SMs fails there on a machine without a GPU)
    assert got == code or (code in (3, 4) and got == 5 and not torch.cuda.is_available())


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(k=None), 1), (dict(slots=None), 1), (dict(q=None), 1), (dict(qs=248), 1), (dict(kps=16), 1),
    (dict(page=12), 2), (dict(off=None), 1), (dict(kv=None), 1), (dict(pairs=40), 1), (dict(depths=(1 << 20) + 1), 3),
    (dict(heads=-1), 1), (dict(batch=-1), 1), (dict(norm=0, kw=1 << 20), 1), (dict(d=96), 2),
])
def test_append_rejects_bad_arguments_without_a_launch(jg, kw, code):
    a = dict(q=1 << 20, qs=256, qo=1 << 21, qos=256, heads=4, k=1 << 20, v=1 << 20, ks=128, vs=128, slots=1 << 20, rows=3,
             kc=1 << 20, vc=1 << 20, kps=16 * 128, vps=16 * 128, pages=4, page=16, kv_heads=2, d=64, off=1 << 20, kv=1 << 20,
             depths=None, batch=1, qw=None, kw=None, freq=1 << 20, pairs=32, inter=0, norm=1, eps=1e-6, ws=None, wsb=0,
             stream=None)
    a.update(kw)
    a["eps"] = ctypes.c_float(a["eps"])
    assert jg.load().jgdpa_cache_append_rotated(*a.values()) == code


def _cpu(rng):
    return dict(q=normal(rng, 5, 4, 64, device="cpu"), k=normal(rng, 5, 2, 64, device="cpu"), q_offsets=i32([0, 5], "cpu"),
                kv_offsets=i32([0, 5], "cpu"), inv_freq=freqs(32, "cpu"), q_weight=torch.ones(64), k_weight=torch.ones(64))


@pytest.mark.parametrize("field,change,match", [
    ("q", lambda t: t.float(), "q must have dtype"),
    ("q", lambda t: t[0], "q must be"),
    ("q", lambda t: t.transpose(0, 1).contiguous().transpose(0, 1), "contiguous inside"),
    ("k", lambda t: t[..., :32], "k must have shape"),
    ("k", lambda t: t[:1].expand(5, 2, 64), "must not overlap"),
    ("q_offsets", lambda t: t.long(), "q_offsets must have dtype"),
    ("kv_offsets", lambda t: i32([0, 2, 5], "cpu"), "kv_offsets must have shape"),
    ("inv_freq", lambda t: t[:12], "multiple of 8"),
    ("inv_freq", lambda t: t.double(), "inv_freq must have dtype"),
    ("q_weight", lambda t: t[:32], "q_weight must have shape"),
    ("k_weight", lambda t: t.bfloat16(), "k_weight must have dtype"),
    ("q", lambda t: t, "CUDA device"),
])
def test_wrapper_rejects_bad_tensors(jg, field, change, match):
    kw = _cpu(np.random.default_rng(0))
    kw[field] = change(kw[field])
    with pytest.raises(ValueError, match=match):
        jg.jgdpa_norm_rotate(**kw)


def test_wrappers_reject_other_bad_calls(jg):
    kw = _cpu(np.random.default_rng(0))
    with pytest.raises(ValueError, match="weights belong to a norm"):
        jg.jgdpa_norm_rotate(**kw, eps=None)
    with pytest.raises(ValueError, match="q_positions must have shape"):
        jg.jgdpa_norm_rotate(**kw, q_positions=i32([0], "cpu"))
    with pytest.raises(ValueError, match="q_out must have shape"):
        jg.jgdpa_norm_rotate(**kw, q_out=kw["k"])
    with pytest.raises(ValueError, match="belong to k, which is None"):
        jg.jgdpa_norm_rotate(**{**kw, "k": None})
    with pytest.raises(ValueError, match="q must have shape"):
        jg.jgdpa_norm_rotate_bwd(kw["q"], kw["k"], kw["k"], kw["k"], *list(kw.values())[2:])
    with pytest.raises(ValueError, match="q is required"):
        jg.jgdpa_norm_rotate_bwd(kw["q"], kw["k"], None, None, *list(kw.values())[2:])
    with pytest.raises(ValueError, match="^k_positions must have shape"):
        jg.jgdpa_norm_rotate_bwd(kw["q"], kw["k"], kw["q"], kw["k"], *list(kw.values())[2:], k_positions=i32([0], "cpu"))
    cache = normal(np.random.default_rng(0), 2, 16, 2, 64, device="cpu")
    with pytest.raises(ValueError, match="depths must have dtype"):
        jg.jgdpa_cache_append_rotated(kw["q"], kw["k"], kw["k"], i32(range(5), "cpu"), cache, cache, i32([0, 5], "cpu"),
                                      i32([5], "cpu"), kw["inv_freq"], depths=torch.zeros(5))
    with pytest.raises(ValueError, match="q must have shape"):
        jg.jgdpa_cache_append_rotated(kw["q"][:4], kw["k"], kw["k"], i32(range(5), "cpu"), cache, cache, i32([0, 5], "cpu"),
                                      i32([5], "cpu"), kw["inv_freq"])


# ------------------------------------------------------------ packed rows (GPU)
LENGTHS = {"one": [1], "empty ones": [0, 0, 3, 0, 1, 0, 0], "odd": [37, 1, 130, 5, 64], "many": [2, 0, 1] * 700, "long": [5000, 3]}


@gpu
@pytest.mark.parametrize("lens", list(LENGTHS))
@pytest.mark.parametrize("d,heads,kv_heads,pairs,interleaved,norm", [
    (128, 8, 8, 64, False, True), (128, 3, 1, 16, False, True), (64, 4, 2, 32, True, True), (64, 1, 1, 5, True, False),
    (32, 7, 1, 16, False, False), (32, 2, 2, 8, False, True),
])
def test_forward_and_backward(jg, lens, d, heads, kv_heads, pairs, interleaved, norm):
    rng = np.random.default_rng(3)
    off = np.concatenate([[0], np.cumsum(LENGTHS[lens])])
    rows = int(off[-1])
    koff = np.concatenate([[0], np.cumsum(LENGTHS[lens][::-1])])  # other lengths than the queries'
    x, dy = ([normal(rng, rows, heads, d), normal(rng, rows, kv_heads, d)] for _ in range(2))
    w = [weights(rng, d), weights(rng, d)] if norm else [None, None]
    eps, freq = 1e-5 if norm else None, freqs(pairs)
    offs = [i32(off), i32(koff)]
    got = jg.jgdpa_norm_rotate(*x, *offs, freq, *w, eps, interleaved=interleaved)
    back = jg.jgdpa_norm_rotate_bwd(*dy, *x, *offs, freq, *w, eps, interleaved=interleaved)
    for i, o in enumerate((off, koff)):
        pos = oracle.positions(o, rows)
        check_rotated(got[i], x[i], pos, freq, w[i], eps, interleaved)
        dx, dw, size = oracle.norm_rotate_bwd(f64(dy[i]), f64(x[i]), pos, f64(freq), None if w[i] is None else f64(w[i]), eps,
                                              interleaved)
        # bf16's rounding; the sums over d <= 128 columns and the angles as above
        pair = pair_size(np.abs(f64(dy[i])), pairs, interleaved)
        g = (1 if not norm else np.max(np.abs(f64(w[i]))) / np.sqrt(np.mean(f64(x[i]) ** 2, -1, keepdims=True) + eps))
        tol = U * np.abs(dx) + 2.0 ** -16 * (size + g * pair + (0 if not norm else np.abs(f64(x[i]) * g ** 2) * np.mean(
            pair, -1, keepdims=True))) + 1e-37
        bad = ~(np.abs(f64(back[i]) - dx) <= tol)
        assert not bad.any(), f"{bad.sum()} of {bad.size}"
        if norm:
            # a lane adds at most rows heads / 300 terms in order (rows heads for few), then some 60 sums
            g, h = pair, np.abs(oracle.norm(f64(x[i]), None, eps))
            n = max(64, rows * x[i].shape[1] / 300) + 64
            assert np.all(np.abs(f64(back[2 + i]) - dw) <= (n * 2.0 ** -24 + 2.0 ** -17) * np.sum(g * h, (0, 1)))


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_and_negative_positions(jg, interleaved):
    """As exact as near ones: in fp32 the angle at 2^31 - 1 would be off by some 100 radians."""
    rng = np.random.default_rng(1)
    pos = [0, 1, -1, 2 ** 24 + 1, 123456789, 2 ** 31 - 1, -2 ** 31, 131071]
    q, k, freq = normal(rng, 8, 3, 64), normal(rng, 8, 1, 64), freqs(32)
    freq[3], freq[4] = 0.0, -1.5
    got = jg.jgdpa_norm_rotate(q, k, None, None, freq, eps=None, interleaved=interleaved, q_positions=i32(pos),
                               k_positions=i32(pos[::-1]))
    check_rotated(got[0], q, pos, freq, None, None, interleaved)
    check_rotated(got[1], k, pos[::-1], freq, None, None, interleaved)
    back = jg.jgdpa_norm_rotate_bwd(*got, None, None, None, None, freq, eps=None, interleaved=interleaved, q_positions=i32(pos),
                                    k_positions=i32(pos[::-1]))
    # there and back: two roundings, and the angles' errors twice
    for x, y in ((q, back[0]), (k, back[1])):
        assert np.all(np.abs(f64(x) - f64(y)) <= 3 * U * pair_size(f64(x), 32, interleaved))


@gpu
def test_segments_and_positions_mixed_and_queries_alone(jg):
    rng = np.random.default_rng(2)
    q, k, freq, w = normal(rng, 9, 2, 128), normal(rng, 6, 2, 128), freqs(64), weights(rng, 128)
    off, pos = i32([0, 4, 9]), i32([7, 7, 0, 3, 100000, 2])
    got = jg.jgdpa_norm_rotate(q, k, off, None, freq, w, k_positions=pos)
    check_rotated(got[0], q, oracle.positions([0, 4, 9], 9), freq, w, 1e-6, False)
    check_rotated(got[1], k, pos.cpu().numpy(), freq, None, 1e-6, False)
    alone, none = jg.jgdpa_norm_rotate(q, None, off, None, freq, w)
    assert none is None and torch.equal(alone, got[0])
    dy = normal(rng, 9, 2, 128)
    dq, dk, dw, dkw = jg.jgdpa_norm_rotate_bwd(dy, None, q, None, off, None, freq, w)
    both = jg.jgdpa_norm_rotate_bwd(dy, torch.zeros_like(k), q, k, off, None, freq, w, k_positions=pos)
    assert dk is None and dkw is None and torch.equal(dq, both[0]) and both[3] is None
    assert torch.allclose(dw, both[2], rtol=1e-5, atol=1e-5)  # (summed in another order)


@gpu
@pytest.mark.parametrize("d", [32, 64, 128])
def test_slices_in_place_and_rows_behind_the_last(jg, d):
    """Slices of a fused projection, written in place; rows behind the last segment stay, and count nothing."""
    rng = np.random.default_rng(d)
    off, rows = [0, 11, 11, 30], 37
    wide = normal(rng, rows, 7, d)
    wide[30:] = float("nan")
    q, k = wide[:, :4], wide[:, 4:6]
    w, freq = weights(rng, d), freqs(d // 2)
    dq, dk = normal(rng, rows, 4, d), normal(rng, rows, 2, d)
    dq[30:] = float("nan")
    clean = jg.jgdpa_norm_rotate(q.contiguous(), k.contiguous(), i32(off), i32(off), freq, w, w)
    back = jg.jgdpa_norm_rotate_bwd(dq, dk, q.contiguous(), k.contiguous(), i32(off), i32(off), freq, w, w)
    assert torch.isfinite(back[2]).all() and torch.isfinite(back[3]).all()
    dq2, dk2 = dq.clone(), dk.clone()
    again = jg.jgdpa_norm_rotate_bwd(dq2, dk2, q, k, i32(off), i32(off), freq, w, w, dq=dq2, dk=dk2)
    assert again[0] is dq2 and torch.equal(dq2[:30], back[0][:30]) and torch.equal(dk2[:30], back[1][:30])
    assert torch.isnan(dq2[30:]).all() and torch.equal(dk2[30:], dk[30:]) and torch.equal(again[2], back[2])
    v = wide[:, 6].clone()
    jg.jgdpa_norm_rotate(q, k, i32(off), i32(off), freq, w, w, q_out=q, k_out=k)
    assert torch.equal(q[:30], clean[0][:30]) and torch.equal(k[:30], clean[1][:30])
    assert torch.isnan(wide[30:]).all() and torch.equal(wide[:30, 6], v[:30])


@gpu
def test_bad_offsets_are_reported(jg):
    rng = np.random.default_rng(4)
    q, k, freq = normal(rng, 20, 2, 64), normal(rng, 20, 2, 64), freqs(32)
    ws = torch.empty(jg.jgdpa_norm_rotate_workspace_bytes(64, True), dtype=torch.uint8, device="cuda")
    good = i32([0, 5, 20])
    for off, status in (([0, 5, 20], 0), ([0, 0, 7], 0), ([1, 5, 20], 6), ([0, 21, 20], 6), ([0, 5, 21], 6),
                        ([0, -3, 20], 6), ([2 ** 31 - 1, -2 ** 31, 5], 6)):
        for offs in ((i32(off), good), (good, i32(off))):
            jg.jgdpa_norm_rotate(q, k, *offs, freq, workspace=ws)
            assert jg.jgdpa_read_device_status(ws) == status, off
            jg.jgdpa_norm_rotate_bwd(q, k, q, k, *offs, freq, workspace=ws)
            assert jg.jgdpa_read_device_status(ws) == status, off


@gpu
def test_offsets_of_queries_that_are_beyond_the_keys_are_reported(jg):
    rng = np.random.default_rng(6)
    x, freq, off = normal(rng, 20, 2, 64), freqs(32), i32([0, 5, 20])
    ws = torch.empty(jg.jgdpa_norm_rotate_workspace_bytes(64, True), dtype=torch.uint8, device="cuda")
    for q, k in ((x, x[:19]), (x[:19], x)):
        jg.jgdpa_norm_rotate(q, k, off, off, freq, workspace=ws)
        assert jg.jgdpa_read_device_status(ws) == 6
        jg.jgdpa_norm_rotate_bwd(q, k, q, k, off, off, freq, workspace=ws)
        assert jg.jgdpa_read_device_status(ws) == 6


@gpu
def test_empty_calls(jg):
    freq, w = freqs(32), torch.ones(64, device="cuda")
    none, some = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    q, k = jg.jgdpa_norm_rotate(none, none, i32([0]), i32([0]), freq)
    assert q.shape == k.shape == (0, 2, 64)
    out = torch.full_like(some, 7.0)
    jg.jgdpa_norm_rotate(some, none, i32([0]), i32([0]), freq, q_out=out)  # no segments: no row is any's
    assert torch.all(out == 7.0)
    dq, dk, dqw, dkw = jg.jgdpa_norm_rotate_bwd(some, none, some, none, i32([0, 3]), i32([0, 0]), freq, w, w)
    assert torch.all(dkw == 0) and torch.isfinite(dqw).all()
    got = jg.jgdpa_norm_rotate_bwd(none, none, none, none, i32([0, 0]), i32([0, 0]), freq, w, w)
    assert torch.all(got[2] == 0) and torch.all(got[3] == 0)


@gpu
def test_same_bits_in_graphs_and_on_other_streams(jg):
    rng = np.random.default_rng(5)
    off, freq, w = i32([0, 3000, 3001, 4096]), freqs(64), weights(rng, 128)
    x, dy = ([normal(rng, 4096, 4, 128), normal(rng, 4096, 2, 128)] for _ in range(2))

    def step(stream=None):
        return [*jg.jgdpa_norm_rotate(*x, off, off, freq, w, w, stream=stream),
                *jg.jgdpa_norm_rotate_bwd(*dy, *x, off, off, freq, w, w, stream=stream)]

    alone = [t.clone() for t in step()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        outs = [step(s) for s in streams]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for o in outs for a, b in zip(alone, o))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(2):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, outs))


@gpu
def test_extreme_rows(jg):
    """Zeros (eps keeps them zero), single large entries, and an infinity or NaN that stays in its own head."""
    rng = np.random.default_rng(6)
    q, freq = normal(rng, 6, 2, 64), freqs(32)
    q[0] = 0
    q[1, 0] = 0
    q[1, 0, 5] = 1e10
    q[2, 0, 3], q[3, 1, 40] = float("inf"), float("nan")
    got, _ = jg.jgdpa_norm_rotate(q, None, i32([0, 6]), None, freq)
    assert torch.all(got[0] == 0) and torch.isnan(got[2, 0]).any() and torch.isnan(got[3, 1]).all()
    x = q.clone()
    x[2, 0], x[3, 1] = 1, 1
    clean, _ = jg.jgdpa_norm_rotate(x, None, i32([0, 6]), None, freq)
    for r, h in [(1, 0), (1, 1), (2, 1), (3, 0), (4, 0), (5, 1)]:
        assert torch.equal(got[r, h], clean[r, h])
    check_rotated(clean, x, np.arange(6), freq, None, 1e-6, False)


# ------------------------------------------------------------ on the way to the cache (GPU)
@gpu
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("d,heads,kv_heads,page,interleaved,norm", [
    (128, 8, 2, 16, False, True), (64, 3, 3, 64, True, False), (32, 4, 1, 1024, False, True), (64, 0, 2, 32, False, True),
])
def test_append(jg, d, heads, kv_heads, page, interleaved, norm, tree):
    rng = np.random.default_rng(8)
    ctx, new = np.array([0, 131000, 7, 0, 55]), np.array([20, 1, 0, 3, 9])
    off, kv, total, spare = np.concatenate([[0], np.cumsum(new)]), ctx + new, int(new.sum()), 4
    pos = np.concatenate([np.arange(c, c + n) for c, n in zip(ctx, new)])
    depth = None
    if tree:
        depth = rng.integers(0, 5, total)
        pos = np.repeat(ctx, new) + depth
    pages = -(-total // page) + 2
    slots = rng.permutation(pages * page)[:total + spare]
    slots[2], slots[5] = -1, pages * page
    wide = normal(rng, total + spare, heads + 2 * kv_heads, d)
    q, k, v = wide[:, :heads], wide[:, heads:heads + kv_heads], wide[:, heads + kv_heads:]
    pool = normal(rng, pages, 2, page, kv_heads, d)
    kc, vc = pool[:, 0], pool[:, 1]
    before = pool.clone()
    w = weights(rng, d) if norm else None
    eps, freq = 1e-6 if norm else None, freqs(d // 2)
    ws = torch.empty(jg.jgdpa_norm_rotate_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    q_out = torch.full((total + spare, max(1, heads), d), 7.0, dtype=torch.bfloat16, device="cuda")
    depths = None if depth is None else i32(np.concatenate([depth, [-9] * spare]))
    got, _, _ = jg.jgdpa_cache_append_rotated(q if heads else None, k, v, i32(slots), kc, vc, i32(off), i32(kv), freq,
                                              w if heads else None, w, eps, interleaved=interleaved, depths=depths,
                                              q_out=q_out if heads else None, workspace=ws)
    assert jg.jgdpa_read_device_status(ws) == 0
    if heads:
        check_rotated(got[:total], q[:total], pos, freq, w, eps, interleaved)
        assert torch.all(got[total:] == 7.0)
    written = np.zeros(pages * page, bool)
    live = [r for r in range(total) if 0 <= slots[r] < pages * page]
    rows = torch.stack([kc[s // page, s % page] for s in slots[live]])
    check_rotated(rows, k[live], pos[live], freq, w, eps, interleaved)
    for r in live:
        assert torch.equal(vc[slots[r] // page, slots[r] % page], v[r])
        written[slots[r]] = True
    rest = torch.from_numpy(~written).cuda().view(pages, page)
    for half in range(2):
        assert torch.equal(pool[:, half][rest], before[:, half][rest])


@gpu
def test_append_reports_bad_positions(jg):
    rng = np.random.default_rng(9)
    k, freq = normal(rng, 4, 1, 64), freqs(32)
    kc = normal(rng, 2, 16, 1, 64)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    for off, kv, depths, status in (([0, 4], [4], None, 0), ([0, 4], [3], None, 6), ([0, 5], [9], None, 6), ([1, 4], [9], None, 6),
                                    ([0, 4], [9], [0, 1, 2, -1], 6), ([0, 4], [2 ** 31 - 1], [0, 1, 2, 3], 0),
                                    ([0, 4], [2 ** 31 - 1], [0, 1, 2, 5], 6), ([0, 0], [9], None, 0)):
        jg.jgdpa_cache_append_rotated(None, k, k, i32(range(4)), kc, kc.clone(), i32(off), i32(kv), freq,
                                      depths=None if depths is None else i32(depths), workspace=ws)
        assert jg.jgdpa_read_device_status(ws) == status, (off, kv, depths)


@gpu
def test_append_of_nothing(jg):
    kc = torch.ones(2, 16, 1, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    q, a, b = jg.jgdpa_cache_append_rotated(torch.zeros(0, 3, 64, dtype=torch.bfloat16, device="cuda"), k, k, i32([]), kc, kc,
                                            i32([0, 0]), i32([3]), freqs(32))
    assert q.shape == (0, 3, 64) and torch.all(a == 1)
    k = torch.zeros(2, 1, 64, dtype=torch.bfloat16, device="cuda")
    jg.jgdpa_cache_append_rotated(None, k, k, i32([0, 1]), kc, kc, i32([0]), i32([]), freqs(32))  # no request's rows
    assert torch.all(kc == 1)
