"""The calls around the attention where places pass 32 bits: the last rows of tensors of more than 2^31 elements."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def jg():
    from jagged_gdpa_gb300 import build as b
    b.build()
    import jagged_gdpa_gb300 as m
    return m


@pytest.fixture(autouse=True)
def memory():
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    yield
    torch.cuda.empty_cache()


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int64).astype(np.int32), device="cuda")


def bf(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").bfloat16()


def test_norms_with_rotation(jg):
    """2^24 + 5 rows of a 160-column stride: the last ones as in a tensor of their own."""
    d, rows, n = 64, (1 << 24) + 5, 1000
    wide = torch.zeros(rows, 160, dtype=torch.bfloat16, device="cuda")
    assert wide.numel() > 1 << 31
    wide[-n:] = bf(0, n, 160)
    q, k = wide[:, :128].unflatten(1, (2, d)), wide[:, 96:].unflatten(1, (1, d))
    off, freq, w = [0, 7, rows - n, rows - 3, rows], 1000.0 ** (-torch.arange(32, device="cuda") / 32), torch.rand(d, device="cuda")
    few = [0, n - 3, n]
    got = jg.jgdpa_norm_rotate(q, k, i32(off), i32(off), freq, w, w)
    want = jg.jgdpa_norm_rotate(q[-n:], k[-n:], i32(few), i32(few), freq, w, w)
    assert torch.equal(got[0][-n:], want[0]) and torch.equal(got[1][-n:], want[1])
    back = jg.jgdpa_norm_rotate_bwd(q, k, q, k, i32(off), i32(off), freq, w, w)
    want = jg.jgdpa_norm_rotate_bwd(q[-n:], k[-n:], q[-n:], k[-n:], i32(few), i32(few), freq, w, w)
    assert torch.equal(back[0][-n:], want[0]) and torch.equal(back[1][-n:], want[1])
    # (all other rows are zeros and add nothing; the sums' order differs, each of up to some 2^17 terms a lane)
    for a, b in zip(back[2:], want[2:]):
        assert torch.allclose(a, b, rtol=1e-4, atol=1e-3)


def test_rotated_writes(jg):
    d, heads, page, pages = 128, 4, 64, (1 << 16) + 9
    kc, vc = (torch.zeros(pages, page, heads, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert kc.numel() > 1 << 31
    k, v = bf(1, 70, heads, d), bf(2, 70, heads, d)
    slots = (pages - 2) * page + np.arange(70)
    freq = 1000.0 ** (-torch.arange(64, device="cuda") / 64)
    jg.jgdpa_cache_append_rotated(None, k, v, i32(slots), kc, vc, i32([0, 70]), i32([100]), freq)
    few = [torch.zeros(2, page, heads, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    jg.jgdpa_cache_append_rotated(None, k, v, i32(np.arange(70)), *few, i32([0, 70]), i32([100]), freq)
    assert torch.equal(kc[-2:], few[0]) and torch.equal(vc[-2:], few[1]) and few[0].any()
    assert not kc[:-2].any() and not vc[:-2].any()


@pytest.mark.parametrize("d", [64, 128])
def test_4_bit_cache(jg, d):
    heads, page = 8, 128
    pages = (1 << 32) // (heads * page * d // 2) + 3
    far = [torch.zeros(pages, heads, page, n, dtype=t, device="cuda") for n, t in ((d // 2, torch.uint8), (2, torch.bfloat16)) * 2]
    assert far[0].numel() > 1 << 32
    near = [t[:3].clone() for t in far]
    k, v = bf(3, 3 * page, heads, d), bf(4, 3 * page, heads, d)
    order = torch.randperm(3 * page, generator=torch.Generator().manual_seed(0)).numpy()
    jg.jgdpa_cache4_append(k, v, i32((pages - 3) * page + order), *far)
    jg.jgdpa_cache4_append(k, v, i32(order), *near)
    for a, b in zip(far, near):
        assert torch.equal(a[-3:], b) and not a[:-3].any()
    for a, b in zip(jg.jgdpa_cache4_read(*far, i32((pages - 3) * page + order)), jg.jgdpa_cache4_read(*near, i32(order))):
        assert torch.equal(a, b) and a.any()
    q = bf(5, 3, 2 * heads, d)
    rest = [i32([0, 3]), i32([3 * page - 5]), "softmax", d ** -0.5, 3]
    a, b = (jg.jgdpa_cache4_fwd(q, *four, i32([[first + 2, first, first + 1]]), *rest) for four, first in ((far, pages - 3), (near, 0)))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("half", [False, True])
def test_verification(jg, half):
    vocab, rows = 128001, 17000
    p = torch.zeros(rows, vocab, dtype=torch.bfloat16 if half else torch.float32, device="cuda")
    assert p.numel() > 1 << 31
    p[-5:] = torch.softmax(bf(6, 5, vocab).float() * 2, 1).to(p.dtype)
    draft = p.roll(1, 0)
    off = np.concatenate([np.arange(0, rows - 5, 1000), [rows - 5, rows]])
    tokens, u = i32(np.arange(rows) % vocab), torch.rand(rows, generator=torch.Generator("cuda").manual_seed(7), device="cuda")
    tokens[-5:] = p[-5:].float().argmax(1).int().roll(1)
    for q in (None, draft):
        got = jg.jgdpa_verify(p, tokens, i32(off), u, draft_probs=q)
        want = jg.jgdpa_verify(p[-5:].clone(), tokens[-5:].clone(), i32([0, 5]), u[-5:].clone(),
                               draft_probs=None if q is None else q[-5:].clone())
        assert got[0][-1:].tolist() == want[0].tolist() and got[1][-1:].tolist() == want[1].tolist()
        assert got[2][-5:].tolist() == want[2].tolist() and want[1][0] >= 0
        assert torch.all(got[0][:-1] == 1) and torch.all(got[1][:-1] == -1)
