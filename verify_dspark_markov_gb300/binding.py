"""Thin ctypes binding of ``libdspark.so`` (the C ABI in ``include/dspark.h``).

Argument marshalling only: torch tensors supply device memory and the current
stream; every step of the computation runs in the library's CUDA kernels.
There is no CPU fallback: if the library is missing or a CUDA device is absent,
the calls raise.
"""
from __future__ import annotations

import ctypes
import math
import operator
import os
import struct
import threading

import torch

from . import build as _build

OK, EINVAL, ENOSPC, ECUDA, ENOTSUP = 0, -1, -2, -3, -4
BF16, F32 = 0, 1
OP_MARKOV_SAMPLE, OP_VERIFY, OP_ACCEPT_STATS, OP_STS_FIT, OP_RNN_SAMPLE = 0, 1, 2, 3, 4
OP_DISTILL_LOSS, OP_BEAM_SELECT = 5, 6
MAX_REORDER_STATES = 16
REQ_OK, REQ_NONFINITE, REQ_EMPTY, REQ_TIMEOUT, REQ_BAD_POLICY, REQ_BAD_TOKEN = range(6)

EXPORTED = ("dspark_workspace_size", "dspark_markov_sample", "dspark_verify", "dspark_verify_width",
            "dspark_accept_stats", "dspark_accept_stats_grad", "dspark_status_string", "dspark_version",
            "dspark_verify_greedy_noalloc", "dspark_sts_fit", "dspark_rnn_sample", "dspark_markov_launches",
            "dspark_wait_selftest", "dspark_rnn_launches", "dspark_top_logits", "dspark_distill_loss",
            "dspark_distill_grad", "dspark_beam_select", "dspark_beam_reorder")

_lock = threading.Lock()
_lib = None


class DsparkError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {status_string(code)} ({code})")
        self.code = code


def library_path() -> str:
    return _build.LIB


def load(path: str | None = None):
    """Load (but never build) the CUDA library; raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            p = path or _build.LIB
            if not os.path.exists(p):
                raise RuntimeError(f"{p} is missing: build it with "
                                   "verify_dspark_markov_gb300.build.build() first")
            lib = ctypes.CDLL(p)
            P, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
            lib.dspark_workspace_size.argtypes = [i32] * 6
            lib.dspark_workspace_size.restype = sz
            lib.dspark_markov_sample.argtypes = ([P, i32, P, P, P, i32, P, i32, P, P, i32]
                                                 + [P] * 4 + [i32] * 3 + [P] * 6 + [sz, P])
            lib.dspark_markov_sample.restype = i32
            lib.dspark_verify.argtypes = [P, i32, P, P, P, P, P, P, P] + [i32] * 3 + [P] * 4 + [sz, P]
            lib.dspark_verify.restype = i32
            lib.dspark_verify_width.argtypes = ([P, i32, P, P, P, P, P, P, P, P] + [i32] * 3 + [P] * 4
                                                + [sz, P])
            lib.dspark_verify_width.restype = i32
            lib.dspark_accept_stats.argtypes = ([P, P, i32, P, P, P] + [i32] * 3 + [P] * 8
                                                + [sz, P])
            lib.dspark_accept_stats.restype = i32
            lib.dspark_accept_stats_grad.argtypes = ([P, P, i32, P, P, P] + [i32] * 3
                                                     + [ctypes.c_double, P, P, P])
            lib.dspark_accept_stats_grad.restype = i32
            lib.dspark_rnn_sample.argtypes = ([P, i32, P, P, P, i32, P, P, P, P, P, i32, P, P, i32]
                                              + [P] * 4 + [i32] * 3 + [P] * 6 + [sz, P])
            lib.dspark_rnn_sample.restype = i32
            lib.dspark_sts_fit.argtypes = [P, P, P, i32, i32, P, P, P, i32, P, sz, P]
            lib.dspark_sts_fit.restype = i32
            lib.dspark_status_string.argtypes = [i32]
            lib.dspark_status_string.restype = ctypes.c_char_p
            lib.dspark_wait_selftest.argtypes = [i32, i32, i32, P, P, P, P]
            lib.dspark_wait_selftest.restype = i32
            lib.dspark_rnn_launches.argtypes = [i32] * 6
            lib.dspark_rnn_launches.restype = i32
            lib.dspark_markov_launches.argtypes = [i32] * 7
            lib.dspark_markov_launches.restype = i32
            i64, f32 = ctypes.c_int64, ctypes.c_float
            lib.dspark_top_logits.argtypes = [P, i32, i64, i32, i32, i32, f32, P, P, P, P, P]
            lib.dspark_top_logits.restype = i32
            lib.dspark_distill_loss.argtypes = [P, i32, i64, P, i32, P, P, P, f32, i32, i32, i32, P, P, P, P, sz, P]
            lib.dspark_distill_loss.restype = i32
            lib.dspark_distill_grad.argtypes = [P, i32, i64, P, i32, P, P, P, f32, ctypes.c_double, i32, i32, i32,
                                                P, P, P, P]
            lib.dspark_distill_grad.restype = i32
            lib.dspark_beam_select.argtypes = [P, i32, i64, i64, P, P, i32, i32, i32, i32, i32, P, P, P, P, P, sz, P]
            lib.dspark_beam_select.restype = i32
            lib.dspark_beam_reorder.argtypes = [P, i32, P, i32, i32, i32, P]
            lib.dspark_beam_reorder.restype = i32
            lib.dspark_version.argtypes = []
            lib.dspark_version.restype = i32
            _lib = lib
    return _lib


def status_string(code: int) -> str:
    return load().dspark_status_string(int(code)).decode()


def workspace_size(op: int, B: int, gamma: int, V: int, r: int = 0, H: int = 0) -> int:
    return int(load().dspark_workspace_size(op, B, gamma, V, r, H))


def wait_selftest(blocks: int, missing: int, limit_us: int, device=None, stream=None):
    """Blocks meeting at the library's bounded grid barrier, told to expect
    `missing` more arrivals than they make.  Returns (status int32 [blocks],
    waited_ns int64 [blocks]) on the device."""
    dev = torch.device("cuda") if device is None else torch.device(device)
    status = torch.empty((blocks,), dtype=torch.int32, device=dev)
    waited = torch.empty((blocks,), dtype=torch.int64, device=dev)
    ws = torch.empty((256,), dtype=torch.uint8, device=dev)  # set by the call itself
    _check(load().dspark_wait_selftest(blocks, missing, limit_us, _ptr(status), _ptr(waited), _ptr(ws),
                                       _stream(stream)), "dspark_wait_selftest")
    if stream is not None:  # the buffer is in use on that stream until the kernels finish
        ws.record_stream(stream)
    return status, waited


def rnn_launches(dtype: int, B: int, gamma: int, V: int, r: int, conf: bool = False) -> int:
    """Kernels one rnn_sample call with these sizes enqueues on the current device."""
    n = int(load().dspark_rnn_launches(dtype, B, gamma, V, r, int(bool(conf))))
    if n < 0:
        raise ValueError("invalid sizes")
    return n


def markov_launches(dtype: int, B: int, gamma: int, V: int, r: int = 0, policy: bool = True,
                    conf: bool = False) -> int:
    """Kernels one markov_sample call with these sizes enqueues on the current device."""
    n = int(load().dspark_markov_launches(dtype, B, gamma, V, r, int(bool(policy)), int(bool(conf))))
    if n < 0:
        raise ValueError("invalid sizes")
    return n


# ------------------------------------------------------------------ helpers
def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"logits must be bfloat16 or float32, got {t.dtype}")


def _dev(t: torch.Tensor, name: str, dtype=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


class Workspace:
    """A zero-filled device buffer per (device, op); grown on demand.  The
    library leaves it zero-filled after every completed call.  For calls that a
    graph captures, one that an earlier call used: without it the graph fills
    its own at every replay.  keep=False: a buffer made now is for this call
    alone."""

    def __init__(self):
        self._bufs = {}

    def get(self, op: int, nbytes: int, device, keep: bool = True) -> torch.Tensor | None:
        if nbytes == 0:
            return None
        key = (torch.device(device).index, op)
        buf = self._bufs.get(key)
        if buf is None or buf.numel() < nbytes:
            buf = torch.zeros(nbytes, dtype=torch.uint8, device=device)
            if keep:
                self._bufs[key] = buf
        return buf


_default_ws = Workspace()


def _check(code: int, what: str):
    if code != OK:
        raise DsparkError(code, what)


def _policy_ptr(policy):
    """policy: None (all greedy) or an int32 [B, 4] CUDA tensor of packed
    dspark_policy records (float temperature, int top_k, float top_p, int greedy)."""
    if policy is None:
        return None
    _dev(policy, "policy", torch.int32)
    if policy.dim() != 2 or policy.shape[1] != 4:
        raise ValueError("policy must be an int32 [B, 4] tensor of packed records")
    return _ptr(policy)


# ------------------------------------------------------------------ entry points
def rnn_sample(backbone, anchor, U, W, Wi, Wh, bi, bh, h=None, E=None, w_conf=None, policy=None,
               seed=None, request_id=None, pos0=None, workspace: Workspace | None = None, stream=None, out=None):
    """The draft's sequential head in its RNN form over [B, gamma, V] backbone
    logits: U, W bf16 [V, r]; Wi, Wh bf16 [3r, r] (gate rows r, z, n); bi, bh
    fp32 [3r].  Returns dict(proposals, q, q_at_x, conf, status) as
    markov_sample does."""
    _dev(backbone, "backbone")
    B, gamma, V = backbone.shape
    dev = backbone.device
    _dev(anchor, "anchor", torch.int32)
    for t, name in ((U, "U"), (W, "W"), (Wi, "Wi"), (Wh, "Wh")):
        _dev(t, name, torch.bfloat16)
    _dev(bi, "bi", torch.float32)
    _dev(bh, "bh", torch.float32)
    r = U.shape[1]
    if Wi.shape != (3 * r, r) or Wh.shape != (3 * r, r) or bi.shape != (3 * r,) or bh.shape != (3 * r,):
        raise ValueError("Wi, Wh must be [3r, r] and bi, bh [3r]")
    H, h_code = 0, F32
    if h is not None:
        _dev(h, "h")
        h_code = _dtype_code(h)
        H = h.shape[2]
        _dev(E, "E", torch.bfloat16)
        _dev(w_conf, "w_conf", torch.float32)
    if out is None:
        out = dict(proposals=torch.empty((B, gamma), dtype=torch.int32, device=dev),
                   q=(torch.empty((B, gamma, V), dtype=torch.float32, device=dev)
                      if policy is not None else None),
                   q_at_x=torch.empty((B, gamma), dtype=torch.float32, device=dev),
                   conf=(torch.empty((B, gamma), dtype=torch.float32, device=dev)
                         if h is not None else None),
                   status=torch.empty((B,), dtype=torch.int32, device=dev))
    ws_n = workspace_size(OP_RNN_SAMPLE, B, gamma, V, r, H)
    ws = (workspace or _default_ws).get(OP_RNN_SAMPLE, ws_n, dev)
    code = load().dspark_rnn_sample(
        _ptr(backbone), _dtype_code(backbone), _ptr(anchor), _ptr(U), _ptr(W), r, _ptr(Wi), _ptr(Wh), _ptr(bi),
        _ptr(bh), _ptr(h), h_code, _ptr(E), _ptr(w_conf), H, _policy_ptr(policy),
        _ptr(_dev(seed, "seed", torch.int64)), _ptr(_dev(request_id, "request_id", torch.int64)),
        _ptr(_dev(pos0, "pos0", torch.int64)), B, gamma, V, _ptr(out["proposals"]), _ptr(out["q"]),
        _ptr(out["q_at_x"]), _ptr(out["conf"]), _ptr(out["status"]), _ptr(ws), ws_n, _stream(stream))
    _check(code, "dspark_rnn_sample")
    return out


def verify(target, proposals, q=None, q_at_x=None, policy=None, seed=None, request_id=None,
           pos0=None, out=None, workspace: Workspace | None = None, stream=None, width=None):
    """Exact verify of [B, gamma+1, V] target logits against [B, gamma]
    proposals.  Returns (out_tokens [B, gamma+1], num_accepted [B], status [B]).
    width: None, or an int32 [B] CUDA tensor of per-request verify widths
    (0..gamma proposals checked; dspark_verify_width)."""
    _dev(target, "target")
    B, rows, V = target.shape
    gamma = rows - 1
    _dev(proposals, "proposals", torch.int32)
    if width is not None:
        _dev(width, "width", torch.int32)
        if width.shape != (B,):
            raise ValueError(f"width must have shape ({B},), got {tuple(width.shape)}")
    dev = target.device
    if out is None:
        out = (torch.empty((B, rows), dtype=torch.int32, device=dev),
               torch.empty((B,), dtype=torch.int32, device=dev),
               torch.empty((B,), dtype=torch.int32, device=dev))
    # greedy calls (policy None) keep their state on chip and take no workspace
    ws_n = workspace_size(OP_VERIFY, B, gamma, V) if policy is not None else 0
    ws = (workspace or _default_ws).get(OP_VERIFY, ws_n, dev)
    args = [_ptr(target), _dtype_code(target), _ptr(proposals), _ptr(_dev(q, "q", torch.float32)),
            _ptr(_dev(q_at_x, "q_at_x", torch.float32)), _policy_ptr(policy),
            _ptr(_dev(seed, "seed", torch.int64)), _ptr(_dev(request_id, "request_id", torch.int64)),
            _ptr(_dev(pos0, "pos0", torch.int64))]
    tail = [B, gamma, V, _ptr(out[0]), _ptr(out[1]), _ptr(out[2]), _ptr(ws), ws_n, _stream(stream)]
    if width is None:
        code, what = load().dspark_verify(*args, *tail), "dspark_verify"
    else:
        code, what = load().dspark_verify_width(*args, _ptr(width), *tail), "dspark_verify_width"
    _check(code, what)
    return out


def markov_sample(backbone, anchor, U=None, W=None, h=None, E=None, w_conf=None, policy=None,
                  seed=None, request_id=None, pos0=None, workspace: Workspace | None = None,
                  stream=None, out=None):
    """The draft's sequential head over [B, gamma, V] backbone logits.
    Returns dict(proposals, q, q_at_x, conf, status)."""
    _dev(backbone, "backbone")
    B, gamma, V = backbone.shape
    dev = backbone.device
    _dev(anchor, "anchor", torch.int32)
    r = 0 if U is None else U.shape[1]
    if r:
        _dev(U, "U", torch.bfloat16)
        _dev(W, "W", torch.bfloat16)
    H = 0
    h_code = F32
    if h is not None:
        _dev(h, "h")
        h_code = _dtype_code(h)
        H = h.shape[2]
        _dev(E, "E", torch.bfloat16)
        _dev(w_conf, "w_conf", torch.float32)
    if out is None:
        out = dict(proposals=torch.empty((B, gamma), dtype=torch.int32, device=dev),
                   q=(torch.empty((B, gamma, V), dtype=torch.float32, device=dev)
                      if policy is not None else None),
                   q_at_x=torch.empty((B, gamma), dtype=torch.float32, device=dev),
                   conf=(torch.empty((B, gamma), dtype=torch.float32, device=dev)
                         if h is not None else None),
                   status=torch.empty((B,), dtype=torch.int32, device=dev))
    ws_n = workspace_size(OP_MARKOV_SAMPLE, B, gamma, V, r, H) if (policy is not None or r) else 0
    ws = (workspace or _default_ws).get(OP_MARKOV_SAMPLE, ws_n, dev)
    code = load().dspark_markov_sample(
        _ptr(backbone), _dtype_code(backbone), _ptr(anchor), _ptr(U), _ptr(W), r, _ptr(h), h_code,
        _ptr(E), _ptr(w_conf), H, _policy_ptr(policy),
        _ptr(_dev(seed, "seed", torch.int64)), _ptr(_dev(request_id, "request_id", torch.int64)),
        _ptr(_dev(pos0, "pos0", torch.int64)), B, gamma, V,
        _ptr(out["proposals"]), _ptr(out["q"]), _ptr(out["q_at_x"]), _ptr(out["conf"]),
        _ptr(out["status"]), _ptr(ws), ws_n, _stream(stream))
    _check(code, "dspark_markov_sample")
    return out


def accept_stats(draft, target, labels, conf_logits, mask=None, workspace: Workspace | None = None,
                 stream=None, out=None):
    """Acceptance statistics of [N, gamma, V] draft logits against the
    target.  Returns dict(l1, accept, tau, loss_num, report, num_tokens, status)."""
    _dev(draft, "draft")
    _dev(target, "target")
    if draft.shape != target.shape or draft.dtype != target.dtype:
        raise ValueError("draft and target must match in shape and dtype")
    N, gamma, V = draft.shape
    dev = draft.device
    _dev(labels, "labels", torch.int32)
    _dev(conf_logits, "conf_logits", torch.float32)
    _dev(mask, "mask", torch.uint8)
    if out is None:
        out = dict(l1=torch.empty((N, gamma), dtype=torch.float32, device=dev),
                   accept=torch.empty((N, gamma), dtype=torch.float32, device=dev),
                   tau=torch.empty((N,), dtype=torch.float32, device=dev),
                   loss_num=torch.empty((4,), dtype=torch.float64, device=dev),
                   report=torch.empty((2,), dtype=torch.float64, device=dev),
                   num_tokens=torch.empty((1,), dtype=torch.int64, device=dev),
                   status=torch.empty((N,), dtype=torch.int32, device=dev))
    ws_n = workspace_size(OP_ACCEPT_STATS, N, gamma, V)
    ws = (workspace or _default_ws).get(OP_ACCEPT_STATS, ws_n, dev)
    code = load().dspark_accept_stats(
        _ptr(draft), _ptr(target), _dtype_code(draft), _ptr(labels), _ptr(conf_logits), _ptr(mask),
        N, gamma, V, _ptr(out["l1"]), _ptr(out["accept"]), _ptr(out["tau"]), _ptr(out["loss_num"]),
        _ptr(out["report"]), _ptr(out["num_tokens"]), _ptr(out["status"]), _ptr(ws), ws_n,
        _stream(stream))
    _check(code, "dspark_accept_stats")
    return out


def accept_stats_grad(draft, target, labels, conf_logits, mask=None, scale=1.0, stream=None, out=None):
    """Gradient of the statistics' loss 0.1 CE + 0.9 L1 + 1.0 BCE (weighted,
    masked numerators; target and the BCE label held fixed) with respect to
    the draft logits and the confidence logits, times scale.  Returns
    (grad_draft fp32 [N, gamma, V], grad_conf fp32 [N, gamma])."""
    _dev(draft, "draft")
    _dev(target, "target")
    if draft.shape != target.shape or draft.dtype != target.dtype:
        raise ValueError("draft and target must match in shape and dtype")
    N, gamma, V = draft.shape
    dev = draft.device
    _dev(labels, "labels", torch.int32)
    _dev(conf_logits, "conf_logits", torch.float32)
    _dev(mask, "mask", torch.uint8)
    if out is None:
        out = (torch.empty((N, gamma, V), dtype=torch.float32, device=dev),
               torch.empty((N, gamma), dtype=torch.float32, device=dev))
    code = load().dspark_accept_stats_grad(
        _ptr(draft), _ptr(target), _dtype_code(draft), _ptr(labels), _ptr(conf_logits), _ptr(mask),
        N, gamma, V, float(scale), _ptr(out[0]), _ptr(out[1]), _stream(stream))
    _check(code, "dspark_accept_stats_grad")
    return out


def sts_fit(conf_logits, labels, mask=None, max_passes=0, workspace: Workspace | None = None, stream=None,
            out=None):
    """Sequential Temperature Scaling: per block position the inverse
    temperature beta >= 0 of the confidence head, from fp32 [N, gamma]
    confidence logits and accept labels (mask: uint8 [N, gamma] or None);
    max_passes is the pass budget (0: the library's default).
    Returns (beta float64 [gamma], status int32 [gamma], passes int32
    [gamma]: the passes each position's search used)."""
    _dev(conf_logits, "conf_logits", torch.float32)
    _dev(labels, "labels", torch.float32)
    if conf_logits.dim() != 2 or labels.shape != conf_logits.shape:
        raise ValueError("conf_logits and labels must be [N, gamma] tensors of one shape")
    N, gamma = conf_logits.shape
    if mask is not None:
        _dev(mask, "mask", torch.uint8)
        if mask.shape != conf_logits.shape:
            raise ValueError("mask must have the shape of conf_logits")
    dev = conf_logits.device
    if out is None:
        out = (torch.empty((gamma,), dtype=torch.float64, device=dev),
               torch.empty((gamma,), dtype=torch.int32, device=dev),
               torch.empty((gamma,), dtype=torch.int32, device=dev))
    ws_n = workspace_size(OP_STS_FIT, N, gamma, 8)
    ws = (workspace or _default_ws).get(OP_STS_FIT, ws_n, dev)
    code = load().dspark_sts_fit(_ptr(conf_logits), _ptr(labels), _ptr(mask), N, gamma, _ptr(out[0]),
                                 _ptr(out[1]), _ptr(out[2]), int(max_passes), _ptr(ws), ws_n, _stream(stream))
    _check(code, "dspark_sts_fit")
    return out


# ------------------------------------- kept top logits, distillation, beams
def _rows(t: torch.Tensor, name: str):
    """(rows, elements between rows) of a CUDA tensor [.., V] whose last
    dimension is contiguous and whose leading ones have one common stride."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() < 1 or t.shape[-1] < 1:
        raise ValueError(f"{name} must have a last dimension of at least one")
    V = t.shape[-1]
    if t.is_contiguous():
        return t.numel() // V, V
    if t.stride(-1) != 1 and V > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    lead = [(n, s) for n, s in zip(t.shape[:-1], t.stride()[:-1]) if n != 1]
    if any(n == 0 for n, _ in lead):
        return 0, V
    rows, stride = 1, V
    for n, s in reversed(lead):
        if rows == 1:
            stride = s
        elif s != stride * rows:
            raise ValueError(f"the rows of {name} must be evenly spaced")
        rows *= n
    return rows, stride


def _shaped(t, name, dtype, shape, device):
    """The pointer of an optional contiguous CUDA tensor of this type and shape."""
    if t is None:
        return None
    if t.device == device and t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _dev(t, name, dtype)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} is on {t.device}, not {device}")


class _Call:
    """The stream of one call, on the current device.  On a stream other than
    the current one, what the call allocates belongs to that stream, and the
    inputs are recorded on it, so that no block is reused while the call may
    still run."""

    def __init__(self, stream, device):
        current = torch._C._cuda_getDevice()  # torch.cuda.current_device() without its checks; the library launches there
        if device.index != current:
            raise ValueError(f"the tensors are on {device}, not on the current device cuda:{current}")
        self.device = device
        self.ptr = torch._C._cuda_getCurrentRawStream(device.index)  # current_stream() without its object
        self.stream = None
        if stream is not None and stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, not on {device}")
        if stream is not None and stream.cuda_stream != self.ptr:
            self.stream, self.ptr = stream, stream.cuda_stream

    def empty(self, shape, dtype):
        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self.stream):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def workspace(self, workspace, op, nbytes):
        if self.stream is not None and self.stream.cuda_stream != torch._C._cuda_getCurrentRawStream(self.device.index):
            with torch.cuda.stream(self.stream):
                return self.workspace(workspace, op, nbytes)
        # under capture the zero fill of a new buffer runs with the graph: such a
        # buffer is that call's alone, and a graph does not share a default one
        capturing = torch.cuda.is_current_stream_capturing()
        if workspace is None:
            # a default workspace per stream: calls on different streams may overlap
            workspace, op = Workspace() if capturing else _default_ws, (op, self.ptr)
            return workspace.get(op, nbytes, self.device, keep=not capturing)
        buf = workspace.get(op, nbytes, self.device, keep=not capturing)
        if buf is not None and buf.is_cuda:  # a call on another stream may have made it
            buf.record_stream(self.stream or torch.cuda.current_stream(self.device))
        return buf

    def uses(self, *tensors):
        if self.stream is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.stream)


def top_logits(logits, k, temperature=1.0, stream=None, out=None):
    """The k largest logits of each row of [.., V] logits, in (logit
    descending, id ascending) order, with the row's log sum exp at
    `temperature`.  Rows may be of any vocabulary and evenly spaced.  Returns
    dict(values [.., k] of the logits' type, index int32 [.., k], lse fp32
    [..], status int32 [..]); past a row's last finite logit the entries are
    (-inf, -1)."""
    N, stride = _rows(logits, "logits")
    dtype, lead, dev, k = _dtype_code(logits), logits.shape[:-1], logits.device, int(k)
    call = _Call(stream, dev)
    if out is None:
        kept = (*lead, max(k, 0))  # the library refuses a k below 1
        values, index = call.empty(kept, logits.dtype), call.empty(kept, torch.int32)
        lse, status = call.empty(lead, torch.float32), call.empty(lead, torch.int32)
        out = dict(values=values, index=index, lse=lse, status=status)
        ptrs = values.data_ptr(), index.data_ptr(), lse.data_ptr(), status.data_ptr()
    else:
        ptrs = (_shaped(out["values"], "values", logits.dtype, (*lead, k), dev),
                _shaped(out["index"], "index", torch.int32, (*lead, k), dev),
                _shaped(out["lse"], "lse", torch.float32, lead, dev),
                _shaped(out["status"], "status", torch.int32, lead, dev))
    code = load().dspark_top_logits(logits.data_ptr(), dtype, stride, N, logits.shape[-1], k, temperature, *ptrs,
                                    call.ptr)
    _check(code, "dspark_top_logits")
    call.uses(logits, *out.values())
    return out


def _distill_args(draft, values, index, lse, weight, temperature):
    N, stride = _rows(draft, "draft")
    lead, dev = draft.shape[:-1], draft.device
    if index.dim() != draft.dim() or index.shape[:-1] != lead:
        raise ValueError(f"index must have shape {(*lead, 'K')}, got {tuple(index.shape)}")
    return N, index.shape[-1], (draft.data_ptr(), _dtype_code(draft), stride,
                                _shaped(values, "values", values.dtype, index.shape, dev), _dtype_code(values),
                                _shaped(index, "index", torch.int32, index.shape, dev),
                                _shaped(lse, "lse", torch.float32, lead, dev),
                                _shaped(weight, "weight", torch.float32, lead, dev), temperature)


def distill_loss(draft, values, index, lse=None, weight=None, temperature=1.0, workspace: Workspace | None = None,
                 stream=None, out=None):
    """Loss of [.., V] draft logits against a teacher's kept logits (values
    bf16 or fp32, index int32, [.., K]; id -1: an unused entry).  With lse (the
    teacher's log sum exp at `temperature`, fp32 [..]) the teacher's remaining
    mass is one class of its own, without it the kept logits are renormalised.
    weight: fp32 [..] per row (0: the row is not read).  Returns dict(loss
    fp32 [..], loss_num fp32 [2]: the sums of weight * loss and of weight,
    status int32 [..])."""
    N, K, args = _distill_args(draft, values, index, lse, weight, temperature)
    lead, dev = draft.shape[:-1], draft.device
    call = _Call(stream, dev)
    if out is None:
        loss, num = call.empty(lead, torch.float32), call.empty((2,), torch.float32)
        status = call.empty(lead, torch.int32)
        out = dict(loss=loss, loss_num=num, status=status)
        ptrs = loss.data_ptr(), num.data_ptr(), status.data_ptr()
    else:
        ptrs = (_shaped(out["loss"], "loss", torch.float32, lead, dev),
                _shaped(out["loss_num"], "loss_num", torch.float32, (2,), dev),
                _shaped(out["status"], "status", torch.int32, lead, dev))
    ws = call.workspace(workspace, OP_DISTILL_LOSS, 256)
    code = load().dspark_distill_loss(*args, N, draft.shape[-1], K, *ptrs, ws.data_ptr(), ws.numel(), call.ptr)
    _check(code, "dspark_distill_loss")
    call.uses(draft, values, index, lse, weight, *out.values())
    return out


def distill_grad(draft, values, index, lse=None, weight=None, temperature=1.0, scale=1.0, stream=None, out=None):
    """Gradient of scale * sum weight * loss (distill_loss's) with respect to
    the draft logits, with the losses: dict(grad [.., V] of the draft's type,
    loss fp32 [..], status int32 [..])."""
    N, K, args = _distill_args(draft, values, index, lse, weight, temperature)
    lead, dev = draft.shape[:-1], draft.device
    call = _Call(stream, dev)
    if out is None:
        grad, loss = call.empty(draft.shape, draft.dtype), call.empty(lead, torch.float32)
        status = call.empty(lead, torch.int32)
        out = dict(grad=grad, loss=loss, status=status)
        ptrs = grad.data_ptr(), loss.data_ptr(), status.data_ptr()
    else:
        ptrs = (_shaped(out["grad"], "grad", draft.dtype, draft.shape, dev),
                _shaped(out["loss"], "loss", torch.float32, lead, dev),
                _shaped(out["status"], "status", torch.int32, lead, dev))
    code = load().dspark_distill_grad(*args, scale, N, draft.shape[-1], K, *ptrs, call.ptr)
    _check(code, "dspark_distill_grad")
    call.uses(draft, values, index, lse, weight, *out.values())
    return out


def beam_select(logits, scores, m, finished=None, eos=0, workspace: Workspace | None = None, stream=None, out=None):
    """One step of beam search: the m best continuations of [B, W, V] logits'
    beams of fp32 [B, W] scores, each at score + log softmax(logits).  A beam
    whose finished (uint8 [B, W]) is set offers only itself, with token eos; a
    beam of score -inf nothing.  Returns dict(scores fp32, parent int32, token
    int32, each [B, m], status int32 [B]), best first, equal scores by (beam,
    token); unfilled places are (-inf, -1, -1).  out["scores"] may be `scores`."""
    if logits.dim() != 3:
        raise ValueError("logits must be [B, W, V]")
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor")
    B, W, V = logits.shape
    item, row, one = logits.stride()
    if one != 1 and V > 1:
        raise ValueError("logits must be contiguous in the vocabulary")
    dtype, dev, m = _dtype_code(logits), logits.device, int(m)
    call = _Call(stream, dev)
    if out is None:
        shape = (B, max(m, 0))  # the library refuses an m below 1
        score, parent = call.empty(shape, torch.float32), call.empty(shape, torch.int32)
        token, status = call.empty(shape, torch.int32), call.empty((B,), torch.int32)
        out = dict(scores=score, parent=parent, token=token, status=status)
        ptrs = score.data_ptr(), parent.data_ptr(), token.data_ptr(), status.data_ptr()
    else:
        ptrs = (_shaped(out["scores"], "scores", torch.float32, (B, m), dev),
                _shaped(out["parent"], "parent", torch.int32, (B, m), dev),
                _shaped(out["token"], "token", torch.int32, (B, m), dev),
                _shaped(out["status"], "status", torch.int32, (B,), dev))
    lib = load()
    ws_n = lib.dspark_workspace_size(OP_BEAM_SELECT, B, W, 0, m, 0)
    ws = call.workspace(workspace, OP_BEAM_SELECT, ws_n)
    code = lib.dspark_beam_select(
        logits.data_ptr(), dtype, item, row, _shaped(scores, "scores", torch.float32, (B, W), dev),
        _shaped(finished, "finished", torch.uint8, (B, W), dev), eos, B, W, V, m, *ptrs,
        None if ws is None else ws.data_ptr(), ws_n, call.ptr)
    _check(code, "dspark_beam_select")
    call.uses(logits, scores, finished, *out.values())
    return out


_first = operator.itemgetter(0)


def _collapse(dims):
    """Dimensions (size, source stride, target stride), outermost first, as few
    as describe the same elements."""
    out = []
    for n, s, d in dims:
        if n == 1:
            continue
        if out and out[-1][1] == s * n and out[-1][2] == d * n:
            out[-1] = (out[-1][0] * n, s, d)
        else:
            out.append((n, s, d))
    return out


def _state(src, dst, dim, name):
    """The 13 words of one tensor's dspark_state, [outer, B, beams, mid, run]:
    of (sizes, strides) as they are, or folded where that is possible."""
    size, shape, W, M = src.element_size(), src.shape, src.shape[dim + 1], dst.shape[dim + 1]
    if src.is_contiguous() and dst.is_contiguous():
        run = 1
        for n in shape[dim + 2:]:
            run *= n
        run *= size
        item, out_item, B = run * W, run * M, shape[dim]
        return (src.data_ptr(), dst.data_ptr(), run, math.prod(shape[:dim]), 1, item * B, item, run, 0, out_item * B,
                out_item, run, 0)
    ss, ds = src.stride(), dst.stride()
    outer = _collapse([(shape[i], ss[i], ds[i]) for i in range(dim)])
    inner = _collapse([(shape[i], ss[i], ds[i]) for i in range(dim + 2, len(shape))])
    run = inner.pop()[0] if inner and inner[-1][1] == 1 and inner[-1][2] == 1 else 1
    if len(outer) > 1 or len(inner) > 1:
        raise ValueError(f"{name}: at most one strided dimension before the beams' and one before the contiguous run")
    (on, os_, od), (mn, ms, md) = (outer or [(1, 0, 0)])[0], (inner or [(1, 0, 0)])[0]
    return (src.data_ptr(), dst.data_ptr(), run * size, on, mn, os_ * size, ss[dim] * size, ss[dim + 1] * size,
            ms * size, od * size, ds[dim] * size, ds[dim + 1] * size, md * size)


def _extent(t):
    """The bytes [first, last) a tensor's elements lie in."""
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()


def _overlap(a, b):
    """Whether two tensors may share a byte.  Apart are extents that do not
    meet, and tensors that lie in different places within every multiple of
    some stride S (the halves of a double buffer, other positions of a cache):
    dimensions whose stride is a multiple of S do not move them there."""
    (a0, a1), (b0, b1) = _extent(a), _extent(b)
    if a1 <= b0 or b1 <= a0:
        return False
    dims = [[(n, s * t.element_size()) for n, s in zip(t.shape, t.stride()) if n > 1] for t in (a, b)]
    for S in {s for d in dims for _, s in d if s}:
        wide_a, wide_b = (t.element_size() + sum((n - 1) * s for n, s in d if s % S) for t, d in zip((a, b), dims))
        apart = (b0 - a0) % S
        if wide_a <= apart and apart + wide_b <= S:
            return False
    return True


def _overlaps_itself(t):
    """Whether a tensor may cover a byte twice (no slice or permutation does)."""
    span = 1
    for s, n in sorted((s, n) for n, s in zip(t.shape, t.stride()) if n > 1):
        if s < span:
            return True
        span += (n - 1) * s
    return False


def _spans(words, B, W, M):
    """The bytes [first, last) of a dspark_state's source and target, and
    whether the target's strides, each past what the ones after it span, say
    that it covers none of them twice."""
    src, dst, run, on, mn, so, si, sb, sm, to, ti, tb, tm = words
    mid = run + (mn - 1) * tm
    beams = mid + (M - 1) * tb
    item = beams + (B - 1) * ti
    once = (mn == 1 or tm >= run) and (M == 1 or tb >= mid) and (B == 1 or ti >= beams) and (on == 1 or to >= item)
    return (src, src + run + (mn - 1) * sm + (W - 1) * sb + (B - 1) * si + (on - 1) * so), \
        (dst, dst + item + (on - 1) * to), once


def _refuse_overlaps(spans):
    """spans: (first, last, whether it is written, tensor).  What is written
    shares no byte with anything else."""
    spans.sort(key=_first)
    for at, (_, end, written, t) in enumerate(spans):
        for start, _, other_written, other in spans[at + 1:]:
            if start >= end:
                break
            if (written or other_written) and _overlap(t, other):
                raise ValueError("out must not overlap the states, the parents or one another")


def beam_reorder(states, parent, dim=0, stream=None, out=None):
    """The states of the beams a selection kept: for each tensor of `states`
    [.., B, W, ..] (B at `dim`), a tensor [.., B, M, ..] of
    state[.., b, parent[b, j], ..], all in one launch.  parent: int32 [B, M],
    -1 for an unfilled place (zeros).  A tensor may be a view (the filled part
    of a cache) with one strided dimension on either side of the beams'.  out:
    None, or the list of tensors to write, which share no memory with the
    states, the parents or one another."""
    _dev(parent, "parent", torch.int32)
    if parent.dim() != 2:
        raise ValueError("parent must be [B, M]")
    B, M = parent.shape
    dev = parent.device
    call = _Call(stream, dev)
    if out is not None and len(out) != len(states):
        raise ValueError(f"out must hold {len(states)} tensors")
    result, words, spans, W = [], [], [], -1
    for i, t in enumerate(states):
        shape = t.shape
        if t.device != dev:
            raise ValueError(f"states[{i}] must be a CUDA tensor on {dev}")
        if dim >= 0 and W < 0 and len(shape) > dim + 1:
            W = shape[dim + 1]
        if dim < 0 or len(shape) < dim + 2 or shape[dim] != B or shape[dim + 1] != W:
            raise ValueError(f"states[{i}] must have B = {B} and W = {W} at dimensions {dim} and {dim + 1}")
        want = (*shape[:dim + 1], M, *shape[dim + 2:])
        if out is None:
            o = call.empty(want, t.dtype)
        else:
            o = out[i]
            if o.shape != want or o.dtype != t.dtype or o.device != dev:
                raise ValueError(f"out[{i}] must be {t.dtype} {want} on {dev}")
        result.append(o)
        if o.numel():
            if W == 0:
                raise ValueError(f"states[{i}] must have at least one beam")
            state = _state(t, o, dim, f"states[{i}]")
            words += state
            if out is not None:
                read, written, once = _spans(state, B, W, M)
                if not once and _overlaps_itself(o):
                    raise ValueError(f"out[{i}] must not overlap itself")
                spans += (*read, False, t), (*written, True, o)
    if spans:
        at = parent.data_ptr()
        spans.append((at, at + 4 * B * M, False, parent))
        _refuse_overlaps(spans)
    lib, most = load(), 13 * MAX_REORDER_STATES
    for at in range(0, len(words), most):
        part = words[at:at + most]
        code = lib.dspark_beam_reorder(struct.pack(f"{len(part)}q", *part), len(part) // 13, parent.data_ptr(), B, W, M,
                                       call.ptr)
        _check(code, "dspark_beam_reorder")
    call.uses(parent, *states, *result)
    return result
