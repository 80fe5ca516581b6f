"""Verification of offsets that are not in order: every entry of the results is written, so that no
slot is left to what the memory held."""

import ctypes

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
FILL = 123456789


@pytest.fixture(scope="module")
def jg():
    from jagged_gdpa_gb300 import build as b
    b.build()
    import jagged_gdpa_gb300 as m
    return m


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int64).astype(np.int32), device="cuda")


@pytest.mark.parametrize("vocab", [40, 9000])  # (one CTA per request, and a cluster)
@pytest.mark.parametrize("off", [[1, 3, 7], [7, 7, 7], [0, 8, 7], [0, 3, 8], [0, -2, 7], [0, 3, 2 ** 31 - 1], [-3, 2, 7], [3, 2, 1], [0, 7, 2],
                                 [0, 3, -1], [-2 ** 31, -5, -1], [2 ** 31 - 1] * 3, [9, 8, 8]])
def test_every_entry_is_written(jg, off, vocab):
    rows, batch = 7, 2
    p = torch.full((rows, vocab), 1 / vocab, device="cuda")
    tokens, u = i32([1] * rows), torch.full((rows,), 0.25, device="cuda")
    offsets, lens, slots = i32(off), i32([100, 200]), i32(range(1000, 1000 + rows))
    accepted, following, keep = (torch.full((batch,), FILL, dtype=torch.int32, device="cuda") for _ in range(3))
    places, moved = (torch.full((rows,), FILL, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = torch.zeros(jg.jgdpa_verify_workspace_bytes(), dtype=torch.uint8, device="cuda")
    P = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    rc = jg.load().jgdpa_verify(P(p), vocab, 0, None, vocab, 0, P(tokens), None, P(u), P(offsets), batch, rows, vocab, P(lens), P(slots),
                                P(accepted), P(following), P(places), P(keep), P(moved), P(ws), ws.numel(),
                                ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0 and jg.jgdpa_read_device_status(ws) == 6
    assert torch.all((accepted >= 0) & (accepted <= rows)) and torch.all((following >= -1) & (following < vocab))
    assert torch.all((keep >= 100 - rows) & (keep <= 200))
    assert torch.all((places >= -1) & (places < rows)), places.tolist()
    assert torch.all((moved == -1) | ((moved >= 1000) & (moved < 1000 + rows))), moved.tolist()
