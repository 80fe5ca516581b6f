"""The short way of the Python calls around the attention (csrc/native.cpp): it
takes the plain calls, does what the wrappers do, and leaves everything else to them."""

import numpy as np
import pytest
import torch

gpu = pytest.mark.gpu
CALLS = ["norm_rotate", "norm_rotate_bwd", "cache_append_rotated", "verify", "cache4_append", "cache4_read", "cache4_fwd"]


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


def bf(rng, *shape, device):
    return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32)).to(torch.bfloat16).to(device)


def i32(x, device):
    return torch.tensor(np.asarray(x, dtype=np.int64).astype(np.int32), device=device)


def arguments(name, device="cuda"):
    """A plain call's positional arguments (as the native call takes them), two requests of 3 and 4 rows."""
    rng = np.random.default_rng(0)
    x = lambda heads: bf(rng, 7, heads, 64, device=device)  # noqa: E731
    off, lens = i32([0, 3, 7], device), i32([3, 4], device)
    freq = torch.from_numpy((10000.0 ** (-np.arange(32) / 32)).astype(np.float32)).to(device)
    w = lambda: torch.from_numpy((1 + 0.1 * rng.standard_normal(64)).astype(np.float32)).to(device)  # noqa: E731
    slots = i32([16, 17, 18, 32, 33, 34, 35], device)
    ws = lambda n: torch.zeros(n, dtype=torch.uint8, device=device)  # noqa: E731
    pages = lambda: torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device=device)  # noqa: E731
    codes = lambda: torch.from_numpy(rng.integers(0, 256, (4, 2, 16, 32), dtype=np.uint8)).to(device)  # noqa: E731
    scales = lambda: (0.1 + bf(rng, 4, 2, 16, 2, device=device).abs())  # noqa: E731
    probs = torch.softmax(torch.from_numpy(rng.standard_normal((7, 50)).astype(np.float32)), 1).to(device)
    u = torch.from_numpy(rng.random(7).astype(np.float32)).to(device)
    return {
        "norm_rotate": lambda: [x(4), x(2), off, off, freq, w(), w(), 1e-6, False, None, None, None, None, ws(256)],
        "norm_rotate_bwd": lambda: [x(4), x(2), x(4), x(2), off, off, freq, w(), w(), 1e-6, False, None, None, None, None, None,
                                    None, None],
        "cache_append_rotated": lambda: [x(4), x(2), x(2), slots, pages(), pages(), off, lens, freq, w(), w(), 1e-6, False, None,
                                         None, ws(256)],
        "verify": lambda: [probs, i32([5, 6, 7, 8, 9, 1, 2], device), off, u, None, i32([0, 0, 0, 0, 0, 0, 1], device), lens,
                           slots, ws(256)],
        "cache4_append": lambda: [x(2), x(2), slots, codes(), scales(), codes(), scales()],
        "cache4_read": lambda: [codes(), scales(), codes(), scales(), slots, None, None],
        "cache4_fwd": lambda: [x(4), codes(), scales(), codes(), scales(), i32([[1], [2]], device), off, lens, 2, 0.125, 4, None, 0,
                               None, None, None, None, None],
    }[name]()


@pytest.mark.parametrize("name", CALLS)
def test_leaves_what_is_not_on_the_gpu(native, name):
    args = arguments(name, "cpu")
    f = getattr(native, name)
    assert f(*args) is None
    assert f(*args[:-1]) is None and f() is None and f(*[None] * len(args)) is None and f(*[1] * len(args)) is None


@gpu
@pytest.mark.parametrize("name", CALLS)
def test_same_as_the_wrapper(jg, native, name):
    args, again = arguments(name), arguments(name)
    got = getattr(native, name)(*args)
    assert type(got) is tuple
    want = getattr(jg, "jgdpa_" + name)(*again, stream=torch.cuda.current_stream())
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert (a is None) == (b is None)
        if a is not None:
            assert a.dtype == b.dtype and a.shape == b.shape and a.is_contiguous() and torch.equal(a, b)


@gpu
@pytest.mark.parametrize("name,outs", [("norm_rotate", {11: 0, 12: 1}), ("norm_rotate_bwd", {13: 0, 14: 1, 15: 2, 16: 3}),
                                       ("cache_append_rotated", {14: 0}), ("cache4_read", {5: 0, 6: 1}),
                                       ("cache4_fwd", {15: 0, 16: 1})])
def test_results_that_are_passed(native, name, outs):
    args = arguments(name)
    want = getattr(native, name)(*args)
    for i, r in outs.items():
        args[i] = torch.empty_like(want[r])
    got = getattr(native, name)(*args)
    for i, r in outs.items():
        assert got[r] is args[i] and torch.equal(got[r], want[r])


@gpu
@pytest.mark.parametrize("name", CALLS)
def test_leaves_tensors_that_do_not_fit(jg, native, name):
    """Each tensor in turn with another type, a row too few, on the CPU, and with strides that do not fit."""
    f, good = getattr(native, name), arguments(name)
    assert type(f(*good)) is tuple
    for i, t in enumerate(good):
        if not isinstance(t, torch.Tensor):
            continue
        bad = [t.double(), t.cpu(), t.unsqueeze(0), torch.stack([t, t], -1)[..., 0], "x"]
        if (name, i) not in (("norm_rotate", 0), ("norm_rotate", 1), ("cache4_read", 4), ("cache4_fwd", 0)) and (t.dtype is not torch.uint8 or t.dim() > 1):
            bad.append(t[:-1])  # (any number of rows goes there, a workspace may have any size)
        for b in bad:
            args = list(good)
            args[i] = b
            fits = f(*args) is not None
            assert not fits, (i, getattr(b, "shape", b))


@gpu
def test_parameters_slices_and_other_kinds_of_numbers(jg, native):
    args = arguments("norm_rotate")
    want = native.norm_rotate(*args)
    wide = torch.cat([args[0], args[1]], 1)
    args[0], args[1] = wide[:, :4], wide[:, 4:]
    args[5] = torch.nn.Parameter(args[5])
    got = native.norm_rotate(*args)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and not got[0].requires_grad
    args[7] = 0  # no float: the wrapper's
    assert native.norm_rotate(*args) is None
    assert torch.isfinite(jg.jgdpa_norm_rotate(*args)[0]).all()
    args[1] = args[3] = args[6] = None
    args[7] = 1e-6
    got = native.norm_rotate(*args)
    assert torch.equal(got[0], want[0]) and got[1] is None


@gpu
def test_library_errors_are_raised(jg, native):
    args = arguments("norm_rotate")
    args[13] = torch.zeros(16, dtype=torch.uint8, device="cuda")
    assert native.norm_rotate(*args) == 4
    with pytest.raises(jg.JgdpaError, match="WORKSPACE_TOO_SMALL"):
        jg.jgdpa_norm_rotate(*args)
