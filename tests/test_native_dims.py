"""The native calls (csrc/native.cpp) against the wrappers at every head dimension and with every kind of
argument: the same results from both, or both leave the call."""

import numpy as np
import pytest
import torch

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def jg():
    from jagged_gdpa_gb300 import build as b
    b.build()
    import jagged_gdpa_gb300 as m
    return m


@pytest.fixture(scope="module")
def native(jg):
    from jagged_gdpa_gb300 import _lib
    m = _lib._native_calls()
    if isinstance(m, _lib._NoNative):
        pytest.skip("no headers to build it from")
    return m


class Inputs:
    """Two requests of 3 and 5 rows, queries, keys and values as slices of wider rows."""

    def __init__(self, d):
        self.rng = np.random.default_rng(d)
        wide = self.bf(8, 10, d)
        self.q, self.k, self.v = wide[:, :4], wide[:, 4:6], wide[:, 6:8]
        self.off, self.lens = self.i32([0, 3, 8]), self.i32([19, 5])
        self.slots = self.i32([32 + 3, 7, -1, 40, 41, 42, 43, 999])
        self.pos, self.depth = self.i32([5, 0, 7, -2, 100000, 3, 3, 9]), self.i32([0, 1, 1, 0, 1, 2, 2, 3])
        self.w, self.kw = self.f32(d), self.f32(d)
        self.d = d

    def bf(self, *shape):
        return torch.from_numpy(self.rng.standard_normal(shape, dtype=np.float32)).cuda().bfloat16()

    def f32(self, *shape):
        return torch.from_numpy(self.rng.uniform(0.1, 1, shape).astype(np.float32)).cuda()

    def i32(self, x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def freq(self, n):
        return torch.from_numpy((1000.0 ** (-np.arange(n) / n)).astype(np.float32)).cuda()

    def pages(self):
        pool = self.bf(4, 2, 16, 2, self.d)
        return pool[:, 0], pool[:, 1]  # K and V interleaved

    def four(self):
        codes = torch.from_numpy(self.rng.integers(0, 256, (4, 2, 2, 16, self.d // 2), dtype=np.uint8)).cuda()
        scales = self.f32(4, 2, 2, 16, 2).bfloat16()
        return [codes[:, 0], scales[:, 0], codes[:, 1], scales[:, 1]]


def rotations(x):
    d = x.d
    yield [x.q, x.k, x.off, x.off, x.freq(d // 2), x.w, x.kw, 1e-5, False, None, None]
    yield [x.q, x.k, x.off, None, x.freq(8), None, x.kw, 0.0, False, None, x.pos]
    yield [x.q, x.k, None, None, x.freq(3), None, None, None, True, x.pos, x.pos]
    yield [x.q, None, x.off, None, x.freq(8), x.w, None, 1e-5, True, None, None]
    yield [x.q[:0], x.k, x.off[:1], None, x.freq(8), None, None, None, False, None, x.pos]


def calls(name, d):
    """Functions that make one call's positional arguments anew (some are written)."""
    x = Inputs(d)
    if name == "norm_rotate":
        return [lambda a=a: [*a, None, None, None] for a in rotations(x)]
    if name == "norm_rotate_bwd":
        def back(a):
            q, k = a[0].clone(), None if a[1] is None else a[1].clone()
            return [q, k, a[0], a[1], *a[2:], None, None, None, None, None]
        return [lambda a=a: back(a) for a in rotations(x)]
    if name == "cache_append_rotated":
        pool = x.pages()[0]._base

        def append(q, qw, kw, eps, inter, depth, n):
            p = pool.clone()
            return [q, x.k, x.v, x.slots, p[:, 0], p[:, 1], x.off, x.lens, x.freq(n), qw, kw, eps, inter, depth, None, None]
        return [lambda: append(x.q, x.w, x.kw, 1e-5, False, None, d // 2), lambda: append(None, None, x.kw, 1e-5, True, x.depth, 3),
                lambda: append(x.q, None, None, None, False, x.depth, 8)]
    if name == "verify":
        u, tokens = x.f32(8), x.i32([1, 2, 3, 4, 5, 6, 7, 0])
        wide = torch.softmax(x.f32(8, 50) * 5, 1)
        probs, draft, parents = wide[:, :41], torch.softmax(x.f32(8, 41), 1).bfloat16(), x.i32([0, 0, 0, 9, 0, 0, 1, 1])
        return [lambda: [probs, tokens, x.off, u, None, None, None, None, None], lambda: [probs, tokens, x.off, u, draft, None, x.lens, None, None],
                lambda: [draft, tokens, x.off, u, probs, None, None, x.slots, None],
                lambda: [probs.bfloat16(), tokens, x.off, u, None, parents, x.lens, x.slots, None]]
    four = x.four()
    if name == "cache4_append":
        return [lambda: [x.k, x.v, x.slots, *[t.clone() for t in four]], lambda: [x.k, x.v, x.slots, *four]]
    if name == "cache4_read":
        out = x.bf(8, 3, 2, d)
        return [lambda: [*four, x.slots, None, None], lambda: [*four, x.slots, out[:, 0], out[:, 2]]]
    table, bias, mask = x.i32([[1, 2], [3, 0]]), x.f32(4, 33), x.i32([[-1]] * 8)
    return [lambda: [x.q, *four, table, x.off, x.lens, 2, 0.3, 5, None, 0, None, None, None, None, None],
            lambda: [x.q, *four, table, x.off, x.lens, 0, 0.3, 5, bias, 7, mask, x.depth, None, None, None],
            lambda: [x.q, *four, table, x.off, x.lens, 1, 0.3, 5, None, 0, None, x.depth, x.bf(8, 4, d), None, None]]


CALLS = ["norm_rotate", "norm_rotate_bwd", "cache_append_rotated", "verify", "cache4_append", "cache4_read", "cache4_fwd"]


@gpu
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("name", CALLS)
def test_same_results(jg, native, name, d):
    for i, make in enumerate(calls(name, d)):
        got = getattr(native, name)(*make())
        assert type(got) is tuple, i
        got = [None if t is None else t.clone() for t in got]
        want = getattr(jg, "jgdpa_" + name)(*make(), stream=torch.cuda.current_stream())
        assert len(got) == len(want)
        for a, b in zip(got, want):
            assert (a is None) == (b is None), i
            if a is not None:
                assert a.dtype == b.dtype and a.shape == b.shape and torch.equal(a.nan_to_num(77.0), b.nan_to_num(77.0)), i


@gpu
@pytest.mark.parametrize("d", [16, 48, 96, 256])
@pytest.mark.parametrize("name", [n for n in CALLS if n != "verify"])
def test_other_head_dimensions_are_refused(jg, native, name, d):
    for make in calls(name, d):
        got = getattr(native, name)(*make())
        assert got is None or got in (1, 2)
        with pytest.raises((ValueError, jg.JgdpaError)):
            getattr(jg, "jgdpa_" + name)(*make())
        with pytest.raises((ValueError, jg.JgdpaError)):
            getattr(jg, "jgdpa_" + name)(*make(), stream=torch.cuda.current_stream())
