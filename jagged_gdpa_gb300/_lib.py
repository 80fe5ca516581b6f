"""ctypes binding of libjgdpa.so (include/jgdpa.h).

Argument marshalling only: every step of the computation runs in the
library's CUDA kernels.  Tensors are torch tensors on the current CUDA device;
torch supplies device memory and the stream.  If the library is missing the
import fails loudly -- there is no fallback implementation.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libjgdpa.so")
# the same library with GELU/SiLU on the ALU-only polynomial route everywhere
ALU_LIB_PATH = os.path.join(_HERE, "_build", "alu", "libjgdpa.so")

ACT = {"gelu": 0, "silu": 1, "softmax": 2}
STATUS = {
    0: "JGDPA_OK", 1: "JGDPA_ERR_INVALID_ARGUMENT", 2: "JGDPA_ERR_UNSUPPORTED",
    3: "JGDPA_ERR_MISALIGNED", 4: "JGDPA_ERR_WORKSPACE_TOO_SMALL", 5: "JGDPA_ERR_CUDA",
    6: "JGDPA_ERR_BAD_OFFSETS", 7: "JGDPA_ERR_DEVICE_TIMEOUT", 8: "JGDPA_ERR_OUT_OF_PAGES",
    9: "JGDPA_ERR_BAD_PAGE",
}
EXPORTS = ("jgdpa_workspace_bytes", "jgdpa_fwd", "jgdpa_fwd_ex", "jgdpa_bwd", "jgdpa_bwd_ex",
           "jgdpa_ds_scratch_bytes",
           "jgdpa_read_device_status", "jgdpa_status_string", "jgdpa_eval_activation", "jgdpa_fwd_noalloc",
           "jgdpa_set_wait_limit_ns", "jgdpa_shared_q_workspace_bytes", "jgdpa_fwd_shared_q", "jgdpa_bwd_shared_q",
           "jgdpa_cache_plan_workspace_bytes", "jgdpa_cache_plan", "jgdpa_cache_append",
           "jgdpa_cache_fwd_workspace_bytes", "jgdpa_cache_fwd")


class JgdpaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)}")


_libs: dict = {}


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libjgdpa.so (raises if it has not been built).  Each path is
    loaded once; the wrappers below take ``lib=`` to use another build."""
    if path in _libs:
        return _libs[path]
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with jagged_gdpa_gb300.build.build()")
    lib = ctypes.CDLL(path)
    P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.jgdpa_workspace_bytes.argtypes = [i32, i64, i64, i32, i32, ctypes.c_int, i32, i32]
    lib.jgdpa_workspace_bytes.restype = sz
    lib.jgdpa_fwd.argtypes = [P, P, P, P, P, i32, i64, i64, i32, i32, ctypes.c_int, f32, P, i32, i32,
                              P, P, P, sz, P]
    lib.jgdpa_fwd.restype = ctypes.c_int
    lib.jgdpa_fwd_ex.argtypes = lib.jgdpa_fwd.argtypes[:15] + [i32] + lib.jgdpa_fwd.argtypes[15:]
    lib.jgdpa_fwd_ex.restype = ctypes.c_int
    lib.jgdpa_bwd.argtypes = [P, P, P, P, P, P, P, P, i32, i64, i64, i32, i32, ctypes.c_int, f32, P, i32,
                              i32, P, P, P, P, P, sz, P]
    lib.jgdpa_bwd.restype = ctypes.c_int
    lib.jgdpa_bwd_ex.argtypes = (lib.jgdpa_bwd.argtypes[:18] + [i32] + lib.jgdpa_bwd.argtypes[18:-1]
                                 + [P, sz, P, P])
    lib.jgdpa_bwd_ex.restype = ctypes.c_int
    lib.jgdpa_ds_scratch_bytes.argtypes = [P, P, i32, i32, i32]
    lib.jgdpa_ds_scratch_bytes.restype = sz
    lib.jgdpa_read_device_status.argtypes = [P, P]
    lib.jgdpa_read_device_status.restype = ctypes.c_int
    lib.jgdpa_status_string.argtypes = [ctypes.c_int]
    lib.jgdpa_status_string.restype = ctypes.c_char_p
    lib.jgdpa_eval_activation.argtypes = [ctypes.c_int, i32, P, i64, P, P, P]
    lib.jgdpa_eval_activation.restype = ctypes.c_int
    lib.jgdpa_fwd_noalloc.argtypes = [P, P, P, P, P, i32, i64, i64, i32, i32, ctypes.c_int, f32, P, i32, i32,
                                      P, P, P]
    lib.jgdpa_fwd_noalloc.restype = ctypes.c_int
    lib.jgdpa_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    lib.jgdpa_set_wait_limit_ns.restype = None
    lib.jgdpa_shared_q_workspace_bytes.argtypes = [i32, i32, i64, i32, i32, ctypes.c_int, i32, i32]
    lib.jgdpa_shared_q_workspace_bytes.restype = sz
    lib.jgdpa_fwd_shared_q.argtypes = [P, i32, P, P, P, i32, i64, i32, i32, ctypes.c_int, f32, P, i32, i32, i32,
                                       P, P, P, sz, P]
    lib.jgdpa_fwd_shared_q.restype = ctypes.c_int
    lib.jgdpa_bwd_shared_q.argtypes = [P, i32, P, P, P, P, P, P, i32, i64, i32, i32, ctypes.c_int, f32, P, i32,
                                       i32, i32, P, P, P, P, P, sz, P, sz, P, P]
    lib.jgdpa_bwd_shared_q.restype = ctypes.c_int
    lib.jgdpa_cache_plan_workspace_bytes.argtypes = []
    lib.jgdpa_cache_plan_workspace_bytes.restype = sz
    lib.jgdpa_cache_plan.argtypes = [P, P, P, i32, i32, P, i32, P, i32, P, i32, P, P, P, P, P, P, sz, P]
    lib.jgdpa_cache_plan.restype = ctypes.c_int
    lib.jgdpa_cache_append.argtypes = [P, P, i64, i64, P, i32, P, P, i64, i64, i32, i32, i32, i32, P]
    lib.jgdpa_cache_append.restype = ctypes.c_int
    lib.jgdpa_cache_fwd_workspace_bytes.argtypes = [i32, i32, i32, i32]
    lib.jgdpa_cache_fwd_workspace_bytes.restype = sz
    lib.jgdpa_cache_fwd.argtypes = [P, i64, P, P, i64, i64, i32, i32, P, i32, P, P, i32, i64, i32, i32, i32, i32,
                                    ctypes.c_int, f32, P, i32, i32, P, i32, P, P, P, P, sz, P]
    lib.jgdpa_cache_fwd.restype = ctypes.c_int
    _libs[path] = lib
    return lib


def _check(t, name: str, dtype, shape, device=None, optional: bool = False):
    """Raise ValueError unless t is a tensor of this dtype and shape (None
    entries of shape match any size) on `device`.  Run before any pointer is
    taken: the library builds its TMA maps from the shapes it is given, so a
    short tensor would be read past its end."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.dim() != len(shape) or any(w is not None and g != w for g, w in zip(t.shape, shape)):
        want = "[" + ", ".join("*" if w is None else str(w) for w in shape) + "]"
        raise ValueError(f"{name} must have shape {want}, got {list(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _check_common(q, k, v, q_offsets, kv_offsets, bias_table):
    """Shapes and dtypes shared by the forward and backward wrappers; returns
    (total_q, heads, head_dim, total_kv, batch, bias_len)."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a bf16 tensor [total_q, heads, head_dim]")
    total_q, heads, d = q.shape
    _check(q, "q", torch.bfloat16, (None, None, None))
    _check(k, "k", torch.bfloat16, (None, heads, d), q.device)
    total_kv = k.shape[0]
    _check(v, "v", torch.bfloat16, (total_kv, heads, d), q.device)
    _check(q_offsets, "q_offsets", torch.int32, (None,), q.device)
    batch = q_offsets.numel() - 1
    if batch < 0:
        raise ValueError("q_offsets must hold batch + 1 >= 1 entries")
    _check(kv_offsets, "kv_offsets", torch.int32, (batch + 1,), q.device)
    _check(bias_table, "bias_table", torch.float32, (heads, None), q.device, optional=True)
    bias_len = 0 if bias_table is None else int(bias_table.shape[1])
    return total_q, heads, d, total_kv, batch, bias_len


def _check_bytes(t, name: str, device):
    if t is None:
        return
    _check(t, name, torch.uint8, (None,), device)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to libjgdpa must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors passed to libjgdpa must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _events(pass_events):
    """Three torch.cuda.Event (or None) as a C array of cudaEvent_t, or None."""
    if pass_events is None:
        return None
    return (ctypes.c_void_p * 3)(*[None if e is None else e.cuda_event for e in pass_events])


def _stream(stream: Optional[torch.cuda.Stream]):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _rc(rc: int, where: str):
    if rc != 0:
        raise JgdpaError(rc, where)


def _act(act) -> int:
    return ACT[act] if isinstance(act, str) else int(act)


def jgdpa_status_string(code: int, lib=None) -> str:
    return (lib or load()).jgdpa_status_string(int(code)).decode()


def jgdpa_workspace_bytes(batch: int, total_q: int, total_kv: int, heads: int, head_dim: int, act,
                          bias_len: int = 0, for_backward: bool = False, lib=None) -> int:
    return int((lib or load()).jgdpa_workspace_bytes(batch, total_q, total_kv, heads, head_dim, _act(act),
                                                     bias_len, int(bool(for_backward))))


def _workspace(nbytes: int, device, workspace: Optional[torch.Tensor]) -> torch.Tensor:
    if workspace is not None:
        return workspace
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def jgdpa_fwd(q, k, v, q_offsets, kv_offsets, act, scale: float, bias_table=None, causal: bool = False,
              out=None, lse=None, workspace=None, stream=None, window: int = 0, lib=None):
    """Forward pass; returns (out, lse) with lse None unless act == 'softmax'.
    window > 0 takes the sliding-window entry point (jgdpa_fwd_ex).  Shapes
    and dtypes are checked here (ValueError) before the library sees any
    pointer."""
    lib = lib or load()
    total_q, heads, d, total_kv, batch, bias_len = _check_common(q, k, v, q_offsets, kv_offsets, bias_table)
    a = _act(act)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and a == ACT["softmax"]:
        lse = torch.empty((heads, total_q), dtype=torch.float32, device=q.device)
    _check(out, "out", torch.bfloat16, (total_q, heads, d), q.device)
    if a == ACT["softmax"]:
        _check(lse, "lse", torch.float32, (heads, total_q), q.device)
    elif lse is not None:
        raise ValueError("lse is written in softmax mode only; pass None")
    _check_bytes(workspace, "workspace", q.device)
    nbytes = jgdpa_workspace_bytes(batch, total_q, total_kv, heads, d, a, bias_len, False, lib=lib)
    ws = _workspace(nbytes, q.device, workspace)
    head = (_ptr(q), _ptr(k), _ptr(v), _ptr(q_offsets), _ptr(kv_offsets), batch, total_q, total_kv, heads, d,
            a, float(scale), _ptr(bias_table), bias_len, int(bool(causal)))
    tail = (_ptr(out), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream))
    if window:
        rc = lib.jgdpa_fwd_ex(*head, int(window), *tail)
        _rc(rc, "jgdpa_fwd_ex")
    else:
        rc = lib.jgdpa_fwd(*head, *tail)
        _rc(rc, "jgdpa_fwd")
    return out, lse


def jgdpa_ds_scratch_bytes(q_offsets, kv_offsets, heads: int, window: int = 0, lib=None) -> int:
    """Stored-dS scratch bytes for these offsets (copied to the host here)."""
    lib = lib or load()
    qo = q_offsets.detach().to("cpu", torch.int32).contiguous()
    ko = kv_offsets.detach().to("cpu", torch.int32).contiguous()
    return int(lib.jgdpa_ds_scratch_bytes(qo.data_ptr(), ko.data_ptr(), qo.numel() - 1, int(heads), int(window)))


def jgdpa_bwd(q, k, v, out, lse, dout, q_offsets, kv_offsets, act, scale: float, bias_table=None,
              causal: bool = False, dq=None, dk=None, dv=None, dbias=None, want_dbias: bool = True,
              workspace=None, stream=None, ds_scratch=None, pass_events=None, window: int = 0, lib=None):
    """Backward pass; returns (dq, dk, dv, dbias) with dbias None without a bias table.

    ds_scratch: optional uint8 device tensor of at least jgdpa_ds_scratch_bytes
    bytes -- selects the stored-dS backward (jgdpa_bwd_ex).  pass_events:
    optional three torch.cuda.Event (timing enabled, already recorded once),
    recorded before the dK/dV pass, between the passes and after the dQ pass.
    window: the forward's sliding window (jgdpa_bwd_ex); 0 for none.  Shapes
    and dtypes are checked here (ValueError) before the library sees any
    pointer."""
    lib = lib or load()
    total_q, heads, d, total_kv, batch, bias_len = _check_common(q, k, v, q_offsets, kv_offsets, bias_table)
    a = _act(act)
    _check(dout, "dout", torch.bfloat16, (total_q, heads, d), q.device)
    if a == ACT["softmax"]:
        _check(out, "out", torch.bfloat16, (total_q, heads, d), q.device)
        _check(lse, "lse", torch.float32, (heads, total_q), q.device)
    else:
        _check(out, "out", torch.bfloat16, (total_q, heads, d), q.device, optional=True)
        _check(lse, "lse", torch.float32, (heads, total_q), q.device, optional=True)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if dbias is None and bias_len and want_dbias:
        dbias = torch.empty((heads, bias_len), dtype=torch.float32, device=q.device)
    _check(dq, "dq", torch.bfloat16, (total_q, heads, d), q.device)
    _check(dk, "dk", torch.bfloat16, (total_kv, heads, d), q.device)
    _check(dv, "dv", torch.bfloat16, (total_kv, heads, d), q.device)
    if dbias is not None:
        if not bias_len:
            raise ValueError("dbias needs a bias table")
        _check(dbias, "dbias", torch.float32, (heads, bias_len), q.device)
    _check_bytes(workspace, "workspace", q.device)
    _check_bytes(ds_scratch, "ds_scratch", q.device)
    nbytes = jgdpa_workspace_bytes(batch, total_q, total_kv, heads, d, a, bias_len, True, lib=lib)
    ws = _workspace(nbytes, q.device, workspace)
    head = (_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(q_offsets),
            _ptr(kv_offsets), batch, total_q, total_kv, heads, d, a, float(scale),
            _ptr(bias_table), bias_len, int(bool(causal)))
    tail = (_ptr(dq), _ptr(dk), _ptr(dv), _ptr(dbias), _ptr(ws), ws.numel())
    if ds_scratch is None and pass_events is None and not window:
        rc = lib.jgdpa_bwd(*head, *tail, _stream(stream))
        _rc(rc, "jgdpa_bwd")
    else:
        rc = lib.jgdpa_bwd_ex(*head, int(window), *tail, _ptr(ds_scratch),
                              0 if ds_scratch is None else ds_scratch.numel(), _stream(stream),
                              _events(pass_events))
        _rc(rc, "jgdpa_bwd_ex")
    return dq, dk, dv, dbias


def jgdpa_fwd_noalloc(q, k, v, q_offsets, kv_offsets, act, scale: float, bias_table=None,
                      causal: bool = False, out=None, lse=None, stream=None, lib=None):
    """Forward pass using the library's built-in scratch (no workspace
    argument; for callers that cannot allocate device memory at call time).
    out / lse must be passed by such callers; they are created here only for
    convenience when omitted.  Returns (out, lse)."""
    lib = lib or load()
    total_q, heads, d, total_kv, batch, bias_len = _check_common(q, k, v, q_offsets, kv_offsets, bias_table)
    a = _act(act)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and a == ACT["softmax"]:
        lse = torch.empty((heads, total_q), dtype=torch.float32, device=q.device)
    _check(out, "out", torch.bfloat16, (total_q, heads, d), q.device)
    if a == ACT["softmax"]:
        _check(lse, "lse", torch.float32, (heads, total_q), q.device)
    rc = lib.jgdpa_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(q_offsets), _ptr(kv_offsets),
                               q_offsets.numel() - 1, total_q, k.shape[0], heads, d, a, float(scale),
                               _ptr(bias_table), bias_len, int(bool(causal)), _ptr(out), _ptr(lse),
                               _stream(stream))
    _rc(rc, "jgdpa_fwd_noalloc")
    return out, lse


def jgdpa_read_device_status(workspace, stream=None, lib=None) -> int:
    return int((lib or load()).jgdpa_read_device_status(_ptr(workspace), _stream(stream)))


def jgdpa_eval_activation(act, x, path: int = 0, stream=None, lib=None):
    """Device act(x), act'(x) for fp32 x (test hook); path 0 = SFU route, 1 = ALU route."""
    _check(x, "x", torch.float32, (None,))
    y = torch.empty_like(x)
    dy = torch.empty_like(x)
    rc = (lib or load()).jgdpa_eval_activation(_act(act), int(path), _ptr(x), x.numel(), _ptr(y), _ptr(dy),
                                      _stream(stream))
    _rc(rc, "jgdpa_eval_activation")
    return y, dy


def jgdpa_set_wait_limit_ns(limit_ns: int, lib=None) -> None:
    """Test hook: limit of one internal device wait for later launches (0 =
    the default of 2 s)."""
    (lib or load()).jgdpa_set_wait_limit_ns(int(limit_ns))


# ------------------------------------------------------------ shared queries
def jgdpa_shared_q_workspace_bytes(batch: int, n_shared: int, total_kv: int, heads: int, head_dim: int, act,
                                   bias_len: int = 0, for_backward: bool = False, lib=None) -> int:
    return int((lib or load()).jgdpa_shared_q_workspace_bytes(batch, n_shared, total_kv, heads, head_dim,
                                                              _act(act), bias_len, int(bool(for_backward))))


def _check_shared(q, k, v, kv_offsets, bias_table):
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a bf16 tensor [n_shared, heads, head_dim]")
    n_shared, heads, d = q.shape
    _check(q, "q", torch.bfloat16, (None, None, None))
    _check(k, "k", torch.bfloat16, (None, heads, d), q.device)
    total_kv = k.shape[0]
    _check(v, "v", torch.bfloat16, (total_kv, heads, d), q.device)
    _check(kv_offsets, "kv_offsets", torch.int32, (None,), q.device)
    batch = kv_offsets.numel() - 1
    if batch < 0:
        raise ValueError("kv_offsets must hold batch + 1 >= 1 entries")
    _check(bias_table, "bias_table", torch.float32, (heads, None), q.device, optional=True)
    bias_len = 0 if bias_table is None else int(bias_table.shape[1])
    return n_shared, heads, d, total_kv, batch, bias_len


def jgdpa_fwd_shared_q(q, k, v, kv_offsets, act, scale: float, bias_table=None, causal: bool = False,
                       out=None, lse=None, workspace=None, stream=None, window: int = 0, lib=None):
    """Forward with query rows shared by every segment: q is [S, H, d]; out is
    [batch S, H, d] (segment b's rows b S .. b S + S - 1); returns (out, lse)."""
    lib = lib or load()
    n_shared, heads, d, total_kv, batch, bias_len = _check_shared(q, k, v, kv_offsets, bias_table)
    a = _act(act)
    total_q = batch * n_shared
    if out is None:
        out = torch.empty((total_q, heads, d), dtype=q.dtype, device=q.device)
    if lse is None and a == ACT["softmax"]:
        lse = torch.empty((heads, total_q), dtype=torch.float32, device=q.device)
    _check(out, "out", torch.bfloat16, (total_q, heads, d), q.device)
    if a == ACT["softmax"]:
        _check(lse, "lse", torch.float32, (heads, total_q), q.device)
    elif lse is not None:
        raise ValueError("lse is written in softmax mode only; pass None")
    _check_bytes(workspace, "workspace", q.device)
    nbytes = jgdpa_shared_q_workspace_bytes(batch, n_shared, total_kv, heads, d, a, bias_len, False, lib=lib)
    ws = _workspace(nbytes, q.device, workspace)
    rc = lib.jgdpa_fwd_shared_q(_ptr(q), n_shared, _ptr(k), _ptr(v), _ptr(kv_offsets), batch, total_kv, heads, d,
                                a, float(scale), _ptr(bias_table), bias_len, int(bool(causal)), int(window),
                                _ptr(out), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream))
    _rc(rc, "jgdpa_fwd_shared_q")
    return out, lse


def jgdpa_bwd_shared_q(q, k, v, out, lse, dout, kv_offsets, act, scale: float, bias_table=None,
                       causal: bool = False, dq=None, dk=None, dv=None, dbias=None, want_dbias: bool = True,
                       workspace=None, stream=None, ds_scratch=None, window: int = 0, pass_events=None,
                       lib=None):
    """Backward with shared query rows; dq [S, H, d] is the sum over segments.
    pass_events as in jgdpa_bwd.  Returns (dq, dk, dv, dbias)."""
    lib = lib or load()
    n_shared, heads, d, total_kv, batch, bias_len = _check_shared(q, k, v, kv_offsets, bias_table)
    a = _act(act)
    total_q = batch * n_shared
    _check(dout, "dout", torch.bfloat16, (total_q, heads, d), q.device)
    opt = a != ACT["softmax"]
    _check(out, "out", torch.bfloat16, (total_q, heads, d), q.device, optional=opt)
    _check(lse, "lse", torch.float32, (heads, total_q), q.device, optional=opt)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if dbias is None and bias_len and want_dbias:
        dbias = torch.empty((heads, bias_len), dtype=torch.float32, device=q.device)
    _check(dq, "dq", torch.bfloat16, (n_shared, heads, d), q.device)
    _check(dk, "dk", torch.bfloat16, (total_kv, heads, d), q.device)
    _check(dv, "dv", torch.bfloat16, (total_kv, heads, d), q.device)
    if dbias is not None:
        if not bias_len:
            raise ValueError("dbias needs a bias table")
        _check(dbias, "dbias", torch.float32, (heads, bias_len), q.device)
    _check_bytes(workspace, "workspace", q.device)
    _check_bytes(ds_scratch, "ds_scratch", q.device)
    nbytes = jgdpa_shared_q_workspace_bytes(batch, n_shared, total_kv, heads, d, a, bias_len, True, lib=lib)
    ws = _workspace(nbytes, q.device, workspace)
    rc = lib.jgdpa_bwd_shared_q(_ptr(q), n_shared, _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout),
                                _ptr(kv_offsets), batch, total_kv, heads, d, a, float(scale), _ptr(bias_table),
                                bias_len, int(bool(causal)), int(window), _ptr(dq), _ptr(dk), _ptr(dv),
                                _ptr(dbias), _ptr(ws), ws.numel(), _ptr(ds_scratch),
                                0 if ds_scratch is None else ds_scratch.numel(), _stream(stream),
                                _events(pass_events))
    _rc(rc, "jgdpa_bwd_shared_q")
    return dq, dk, dv, dbias


# ------------------------------------------------- paged key/value cache (serving)
# These calls belong to a serving step, where some tens of microseconds of
# Python per call would be what the step waits for: each wrapper first tests
# everything in one pass, and names what is wrong (`_refuse_*`) only if a test fails.
_I32_MAX = (1 << 31) - 1
_i32, _f32, _bf16, _u8 = torch.int32, torch.float32, torch.bfloat16, torch.uint8
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current_raw_stream(index: int) -> int:
    if _raw_stream is not None:
        return _raw_stream(index)
    return torch.cuda.current_stream(index).cuda_stream


class _Alloc:
    """Memory for results and scratch of a call on another stream than the
    current one.  Scratch comes from that stream's own pool, so that it is not
    handed out again before the call's kernels have run; results are known to
    the current stream too."""

    def __init__(self, device, stream):
        self.device, self.stream = device, stream

    def __call__(self, shape, dtype, result=True):
        with torch.cuda.stream(self.stream):
            t = torch.empty(shape, dtype=dtype, device=self.device)
        if result:
            t.record_stream(torch.cuda.current_stream(self.device))
        return t


def _launch_on(stream, device):
    """(cudaStream_t, allocator or None for torch's own) of a call."""
    if stream is None:
        return _current_raw_stream(device.index), None
    if stream == torch.cuda.current_stream(device):
        return stream.cuda_stream, None
    return stream.cuda_stream, _Alloc(device, stream)


def _on_other_device(fn, device, args, kw):
    """Runs a wrapper again with its tensors' device as the current one."""
    with torch.cuda.device(device):
        return fn(*args, **kw)


def _is(t, dtype, shape, index) -> bool:
    """Whether t is a contiguous tensor of this dtype and shape on this CUDA device."""
    return t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous()


def _contiguous(**tensors):
    for name, t in tensors.items():
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _refuse_wide(**numbers):
    """ctypes would cut them to 32 bits without a word."""
    for name, n in numbers.items():
        if not -(1 << 31) <= n < 1 << 31:
            raise ValueError(f"{name} must fit in 32 bits, got {n}")


def _need_cuda(t: torch.Tensor):
    if not t.is_cuda:
        raise ValueError("tensors passed to libjgdpa must be on a CUDA device")


def _page_stride(t: torch.Tensor, page: int, heads: int, d: int) -> int:
    """Elements between the pages of a cache (any multiple of 8 from a page's
    size on), or 0 if its pages are not contiguous inside or overlap."""
    n, stride = t.shape[0], t.stride()
    size = page * heads * d
    if stride[1:] != (heads * d, d, 1) and any(
            k > 1 and a != b for k, a, b in zip((page, heads, d), stride[1:], (heads * d, d, 1))):
        return 0
    if n <= 1:
        return size
    return stride[0] if stride[0] >= size and stride[0] % 8 == 0 else 0


def _row_stride(t: torch.Tensor, heads: int, d: int) -> int:
    """Elements between rows [heads][d] of t (any multiple of 8 from a row's
    size on), or 0 if a row is not contiguous inside or rows overlap."""
    stride = t.stride()
    if t.numel() and (stride[2] != 1 or (heads > 1 and stride[1] != d)):
        return 0
    if t.shape[0] <= 1:
        return heads * d
    return stride[0] if stride[0] >= heads * d and stride[0] % 8 == 0 else 0


def _refuse_cache(k_cache, v_cache):
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be a bf16 tensor [num_pages, page_size, kv_heads, head_dim]")
    _check(k_cache, "k_cache", torch.bfloat16, (None, None, None, None))
    _check(v_cache, "v_cache", torch.bfloat16, k_cache.shape, k_cache.device)
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if not _page_stride(t, *t.shape[1:]):
            raise ValueError(f"{name}: pages must be contiguous inside, must not overlap and lie a multiple of 8 "
                             "elements apart")


def _refuse_rows(t, name, heads, d):
    if not _row_stride(t, heads, d):
        raise ValueError(f"{name}: rows must be contiguous inside, must not overlap and lie a multiple of 8 elements apart")


def jgdpa_cache_plan_workspace_bytes(lib=None) -> int:
    return int((lib or load()).jgdpa_cache_plan_workspace_bytes())


def _refuse_plan(ctx_lens, new_lens, held_pages, block_table, free_pages, free_count, workspace):
    _check(ctx_lens, "ctx_lens", torch.int32, (None,))
    device, batch = ctx_lens.device, ctx_lens.shape[0]
    _check(new_lens, "new_lens", torch.int32, (batch,), device)
    _check(held_pages, "held_pages", torch.int32, (batch,), device)
    _check(block_table, "block_table", torch.int32, (batch, None), device)
    _check(free_pages, "free_pages", torch.int32, (None,), device)
    _check(free_count, "free_count", torch.int32, (1,), device)
    _check_bytes(workspace, "workspace", device)
    _contiguous(ctx_lens=ctx_lens, new_lens=new_lens, held_pages=held_pages, block_table=block_table,
                free_pages=free_pages, workspace=workspace)
    _need_cuda(ctx_lens)


def jgdpa_cache_plan(ctx_lens, new_lens, held_pages, block_table, free_pages, free_count, page_size: int,
                     total_new: int, workspace=None, stream=None, lib=None):
    """Pages and slots for a step's tokens (jgdpa_cache_plan); returns (slots,
    q_offsets, kv_lens, held_pages, free_count), the last two being the new
    counts to pass to the next plan.  block_table and free_pages are updated in
    place.  total_new: rows of slots, at least the sum of new_lens.  workspace:
    where a device-detected error (out of pages) is to be read from."""
    lib = lib or load()
    page_size, total_new = int(page_size), int(total_new)
    if max(page_size, total_new) > _I32_MAX or page_size < -_I32_MAX:
        _refuse_wide(page_size=page_size, total_new=total_new)
    try:
        index, shape = ctx_lens.get_device(), ctx_lens.shape
        batch, width = block_table.shape
        pages = free_pages.shape[0]
        ok = (index >= 0 and _is(ctx_lens, _i32, (batch,), index) and _is(new_lens, _i32, shape, index)
              and _is(held_pages, _i32, shape, index) and _is(block_table, _i32, (batch, width), index)
              and _is(free_pages, _i32, (pages,), index) and _is(free_count, _i32, (1,), index)
              and (workspace is None or _is(workspace, _u8, (workspace.numel(),), index)))
    except (AttributeError, ValueError, IndexError, TypeError):
        ok = False
    if not ok:
        _refuse_plan(ctx_lens, new_lens, held_pages, block_table, free_pages, free_count, workspace)
        raise ValueError("jgdpa_cache_plan: unusable tensors")
    if total_new < 0:
        raise ValueError("total_new must not be negative")
    if max(width, pages) > _I32_MAX:
        _refuse_wide(**{"block_table's width": width, "free_pages' length": pages})
    if index != torch.cuda.current_device():
        return _on_other_device(jgdpa_cache_plan, ctx_lens.device, (ctx_lens, new_lens, held_pages, block_table, free_pages,
                                free_count, page_size, total_new, workspace, stream, lib), {})
    raw, alloc = _launch_on(stream, ctx_lens.device)
    if alloc is None:
        device = ctx_lens.device
        slots = torch.empty(total_new, dtype=_i32, device=device)
        q_offsets = torch.empty(batch + 1, dtype=_i32, device=device)
        kv_lens = torch.empty(batch, dtype=_i32, device=device)
        held = torch.empty(batch, dtype=_i32, device=device)
        count = torch.empty(1, dtype=_i32, device=device)
    else:
        slots, q_offsets, kv_lens, held, count = (alloc(n, _i32) for n in (total_new, batch + 1, batch, batch, 1))
    ws, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    rc = lib.jgdpa_cache_plan(ctx_lens.data_ptr(), new_lens.data_ptr(), held_pages.data_ptr(), batch, page_size,
                              block_table.data_ptr(), width, free_pages.data_ptr(), pages, free_count.data_ptr(),
                              total_new, held.data_ptr(), count.data_ptr(), q_offsets.data_ptr(), kv_lens.data_ptr(),
                              slots.data_ptr(), ws, ws_bytes, raw)
    if rc:
        raise JgdpaError(rc, "jgdpa_cache_plan")
    return slots, q_offsets, kv_lens, held, count


def _refuse_append(k_new, v_new, slots, k_cache, v_cache):
    _refuse_cache(k_cache, v_cache)
    heads, d = k_cache.shape[2:]
    device = k_cache.device
    _check(k_new, "k_new", torch.bfloat16, (None, heads, d), device)
    rows = k_new.shape[0]
    _check(v_new, "v_new", torch.bfloat16, (rows, heads, d), device)
    _check(slots, "slots", torch.int32, (rows,), device)
    _refuse_rows(k_new, "k_new", heads, d)
    _refuse_rows(v_new, "v_new", heads, d)
    _contiguous(slots=slots)
    _need_cuda(k_cache)


def jgdpa_cache_append(k_new, v_new, slots, k_cache, v_cache, stream=None, lib=None):
    """Writes rows of k_new / v_new [total_new, kv_heads, head_dim] (rows may be
    slices of wider ones) to their slots; returns (k_cache, v_cache)."""
    lib = lib or load()
    ks = vs = kps = vps = 0
    try:
        index = k_cache.get_device()
        n, page, heads, d = k_cache.shape
        rows = k_new.shape[0]
        shape = (rows, heads, d)
        if (index >= 0 and k_cache.dtype is _bf16 and v_cache.dtype is _bf16 and v_cache.shape == k_cache.shape
                and v_cache.get_device() == index and k_new.dtype is _bf16 and v_new.dtype is _bf16
                and k_new.shape == shape and v_new.shape == shape and k_new.get_device() == index
                and v_new.get_device() == index and _is(slots, _i32, (rows,), index)):
            kps, vps = _page_stride(k_cache, page, heads, d), _page_stride(v_cache, page, heads, d)
            ks, vs = _row_stride(k_new, heads, d), _row_stride(v_new, heads, d)
    except (AttributeError, ValueError, IndexError, TypeError):
        pass
    if not (ks and vs and kps and vps):
        _refuse_append(k_new, v_new, slots, k_cache, v_cache)
        raise ValueError("jgdpa_cache_append: unusable tensors")
    if max(rows, n) > _I32_MAX:
        _refuse_wide(**{"k_new's rows": rows, "k_cache's pages": n})
    if index != torch.cuda.current_device():
        return _on_other_device(jgdpa_cache_append, k_cache.device, (k_new, v_new, slots, k_cache, v_cache, stream, lib), {})
    rc = lib.jgdpa_cache_append(k_new.data_ptr(), v_new.data_ptr(), ks, vs, slots.data_ptr(), rows, k_cache.data_ptr(),
                                v_cache.data_ptr(), kps, vps, n, page, heads, d,
                                _current_raw_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        raise JgdpaError(rc, "jgdpa_cache_append")
    return k_cache, v_cache


def jgdpa_cache_fwd_workspace_bytes(heads: int, kv_heads: int, head_dim: int, max_q: int, lib=None) -> int:
    _refuse_wide(heads=heads, kv_heads=kv_heads, head_dim=head_dim, max_q=max_q)
    return int((lib or load()).jgdpa_cache_fwd_workspace_bytes(heads, kv_heads, head_dim, max_q))


def _refuse_fwd(q, k_cache, v_cache, block_table, q_offsets, kv_lens, softmax, bias_table, tree_mask, depths, out, lse,
                workspace):
    _refuse_cache(k_cache, v_cache)
    d, device = k_cache.shape[3], k_cache.device
    _check(q, "q", torch.bfloat16, (None, None, d), device)
    total_q, heads = q.shape[0], q.shape[1]
    _check(kv_lens, "kv_lens", torch.int32, (None,), device)
    batch = kv_lens.shape[0]
    _check(q_offsets, "q_offsets", torch.int32, (batch + 1,), device)
    _check(block_table, "block_table", torch.int32, (batch, None), device)
    _check(bias_table, "bias_table", torch.float32, (heads, None), device, optional=True)
    _check(tree_mask, "tree_mask", torch.int32, (total_q, None), device, optional=True)
    _check(depths, "depths", torch.int32, (total_q,), device, optional=True)
    _check(out, "out", torch.bfloat16, (total_q, heads, d), device, optional=True)
    if lse is not None and not softmax:
        raise ValueError("lse is written in softmax mode only; pass None")
    _check(lse, "lse", torch.float32, (heads, total_q), device, optional=True)
    _check_bytes(workspace, "workspace", device)
    for t, name in ((bias_table, "bias_table"), (tree_mask, "tree_mask")):
        if t is not None and t.shape[1] == 0:
            raise ValueError(f"{name} must have columns; pass None for none")
    _refuse_rows(q, "q", heads, d)
    _contiguous(block_table=block_table, q_offsets=q_offsets, kv_lens=kv_lens, bias_table=bias_table,
                tree_mask=tree_mask, depths=depths, out=out, lse=lse, workspace=workspace)
    _need_cuda(k_cache)


def jgdpa_cache_fwd(q, k_cache, v_cache, block_table, q_offsets, kv_lens, act, scale: float, max_q: int,
                    bias_table=None, window: int = 0, tree_mask=None, depths=None, out=None, lse=None,
                    workspace=None, stream=None, lib=None):
    """Attention from new tokens q [total_q, heads, head_dim] over each
    request's pages (jgdpa_cache_fwd); returns (out, lse) with lse None unless
    act == 'softmax'.  max_q: an upper bound of the new tokens per request."""
    lib = lib or load()
    a = _act(act)
    max_q, window = int(max_q), int(window)
    if max(max_q, window) > _I32_MAX or min(max_q, window) < -_I32_MAX:
        _refuse_wide(max_q=max_q, window=window)
    softmax = a == 2
    qs = kps = vps = 0
    bias = mask = depth = None
    bias_len = words = 0
    try:
        index = k_cache.get_device()
        n, page, kv_heads, d = k_cache.shape
        total_q, heads, _ = shape = q.shape
        batch, width = block_table.shape
        ok = (index >= 0 and k_cache.dtype is _bf16 and v_cache.dtype is _bf16 and v_cache.shape == k_cache.shape
              and v_cache.get_device() == index and q.dtype is _bf16 and shape[2] == d and q.get_device() == index
              and _is(block_table, _i32, (batch, width), index) and _is(q_offsets, _i32, (batch + 1,), index)
              and _is(kv_lens, _i32, (batch,), index))
        if ok and bias_table is not None:
            bias, bias_len = bias_table.data_ptr(), bias_table.shape[1]
            ok = bias_len > 0 and _is(bias_table, _f32, (heads, bias_len), index)
        if ok and tree_mask is not None:
            mask, words = tree_mask.data_ptr(), tree_mask.shape[1]
            ok = words > 0 and _is(tree_mask, _i32, (total_q, words), index)
        if ok and depths is not None:
            depth = depths.data_ptr()
            ok = _is(depths, _i32, (total_q,), index)
        if ok and out is not None:
            ok = _is(out, _bf16, shape, index)
        if ok and lse is not None:
            ok = softmax and _is(lse, _f32, (heads, total_q), index)
        if ok and workspace is not None:
            ok = _is(workspace, _u8, (workspace.numel(),), index)
        if ok:
            kps, vps = _page_stride(k_cache, page, kv_heads, d), _page_stride(v_cache, page, kv_heads, d)
            qs = _row_stride(q, heads, d)
    except (AttributeError, ValueError, IndexError, TypeError):
        pass
    if not (qs and kps and vps):
        _refuse_fwd(q, k_cache, v_cache, block_table, q_offsets, kv_lens, softmax, bias_table, tree_mask, depths, out, lse,
                    workspace)
        raise ValueError("jgdpa_cache_fwd: unusable tensors")
    if max(n, width, bias_len) > _I32_MAX:
        _refuse_wide(**{"k_cache's pages": n, "block_table's width": width, "bias_table's length": bias_len})
    if index != torch.cuda.current_device():
        return _on_other_device(jgdpa_cache_fwd, k_cache.device, (q, k_cache, v_cache, block_table, q_offsets, kv_lens, act,
                                scale, max_q, bias_table, window, tree_mask, depths, out, lse, workspace, stream, lib), {})
    device = k_cache.device
    raw, alloc = _launch_on(stream, device)
    if alloc is None:
        if out is None:
            out = torch.empty(shape, dtype=_bf16, device=device)
        if softmax and lse is None:
            lse = torch.empty((heads, total_q), dtype=_f32, device=device)
        if workspace is None:
            workspace = torch.empty(max(256, lib.jgdpa_cache_fwd_workspace_bytes(heads, kv_heads, d, max_q)), dtype=_u8,
                                    device=device)
    else:
        if out is None:
            out = alloc(shape, _bf16)
        if softmax and lse is None:
            lse = alloc((heads, total_q), _f32)
        if workspace is None:
            workspace = alloc(max(256, lib.jgdpa_cache_fwd_workspace_bytes(heads, kv_heads, d, max_q)), _u8, result=False)
    rc = lib.jgdpa_cache_fwd(q.data_ptr(), qs, k_cache.data_ptr(), v_cache.data_ptr(), kps, vps, n, page,
                             block_table.data_ptr(), width, q_offsets.data_ptr(), kv_lens.data_ptr(), batch, total_q,
                             max_q, heads, kv_heads, d, a, float(scale), bias, bias_len, window, mask, words, depth,
                             out.data_ptr(), lse.data_ptr() if lse is not None else None, workspace.data_ptr(),
                             workspace.numel(), raw)
    if rc:
        raise JgdpaError(rc, "jgdpa_cache_fwd")
    return out, lse
