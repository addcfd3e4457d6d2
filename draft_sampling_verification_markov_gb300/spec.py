"""Thin ctypes binding of libspecmarkov.so (see include/spec_markov.h for the semantics).

Argument marshalling only: every function here passes device pointers, sizes and the current
CUDA stream to the C entry point of the same name and allocates output tensors when the caller
does not supply them. All arithmetic of the hot path runs in the library's CUDA kernels. There is
no fallback: if the library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import build as _build

SPEC_OK = 0
SPEC_F32, SPEC_BF16 = 0, 1
(SPEC_OP_PROPOSE, SPEC_OP_VERIFY_GREEDY, SPEC_OP_VERIFY_REJECTION, SPEC_OP_TV_CONFIDENCE,
 SPEC_OP_SCHEDULE, SPEC_OP_TARGET_STATS, SPEC_OP_MTP_GREEDY, SPEC_OP_ALL) = range(8)
(SPEC_DEV_BAD_TOKEN, SPEC_DEV_NONFINITE, SPEC_DEV_EMPTY_RESIDUAL, SPEC_DEV_BAD_LENGTH,
 SPEC_DEV_TIMEOUT) = 1, 2, 4, 8, 16
SPEC_SCHEDULE_MAX_CANDIDATES = 16384
(SPEC_KCLASS_MARKOV, SPEC_KCLASS_STREAM, SPEC_KCLASS_SELECT, SPEC_KCLASS_OTHER,
 SPEC_KCLASS_PROPOSE) = range(5)
SPEC_NOALLOC_MAX_ROWS = 65536
SPEC_ERR_TOO_LARGE = -7
SPEC_MX_E2M1, SPEC_MX_E4M3 = 0, 1
SPEC_MX_GROUP = 128
SPEC_LOGPROBS_MAX_TOP = 32

_lib = None


class SpecError(RuntimeError):
    def __init__(self, fn, status):
        msg = lib().spec_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{fn} failed with status {status} ({msg})")
        self.status = status


def library_path() -> str:
    return _build.SO


def lib():
    """Load libspecmarkov.so (built in-tree by __graft_entry__.build())."""
    global _lib
    if _lib is None:
        if not os.path.exists(_build.SO):
            raise RuntimeError(f"{_build.SO} is not built; run __graft_entry__.build() first")
        L = ctypes.CDLL(_build.SO)
        vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.spec_abi_version.restype = i
        L.spec_status_string.argtypes = [i]
        L.spec_status_string.restype = ctypes.c_char_p
        L.spec_workspace_bytes.argtypes = [i, i, i, i, i]
        L.spec_workspace_bytes.restype = sz
        L.spec_workspace_init.argtypes = [vp, sz, vp]
        L.spec_device_status.argtypes = [vp, sz, vp, ctypes.POINTER(ctypes.c_uint32), i]
        L.spec_markov_propose.argtypes = [vp, i, vp, vp, i, i, vp, vp, f, i, i, i, vp, vp, vp, vp,
                                          sz, vp]
        L.spec_verify_greedy.argtypes = [vp, i, vp, vp, i, i, i, vp, vp, vp, vp, sz, vp]
        L.spec_mtp_greedy.argtypes = [vp, vp, i, vp, i, i, i, vp, vp, vp, vp, vp, sz, vp]
        L.spec_target_stats.argtypes = [vp, i, f, i, i, vp, vp, sz, vp]
        L.spec_verify_rejection.argtypes = [vp, vp, i, vp, vp, i, i, vp, vp, vp, vp, vp, vp, vp,
                                            f, vp, i, i, i, vp, vp, vp, vp, sz, vp]
        L.spec_tv_confidence.argtypes = [vp, vp, i, vp, vp, i, i, vp, vp, vp, vp, f, i, i, i, vp,
                                         vp, vp, sz, vp]
        L.spec_schedule_prefix.argtypes = [vp, vp, i, i, i, vp, vp, vp, vp, sz, vp]
        L.spec_schedule_topk.argtypes = [vp, vp, i, i, i, vp, vp, vp, vp, vp, vp, sz, vp]
        L.spec_verify_greedy_noalloc.argtypes = [vp, i, vp, vp, i, i, i, vp, vp, vp, vp, vp]
        L.spec_markov_propose_masked.argtypes = [vp, i, vp, vp, i, i, vp, vp, f, i, i, i, vp, vp,
                                                 vp, vp, vp, sz, vp]
        L.spec_markov_propose_target_stats.argtypes = [vp, i, vp, vp, i, i, vp, vp, f, i, i, i,
                                                       vp, vp, vp, vp, vp, vp, sz, vp]
        L.spec_verify_rejection_masked.argtypes = [vp, vp, i, vp, vp, i, i, vp, vp, vp, vp, vp,
                                                   vp, vp, f, vp, i, i, i, vp, vp, vp, vp, vp,
                                                   sz, vp]
        L.spec_tv_confidence_masked.argtypes = [vp, vp, i, vp, vp, i, i, vp, vp, vp, vp, f, i, i,
                                                i, vp, vp, vp, vp, sz, vp]
        L.spec_flat_layout.argtypes = [vp, i, i, vp, vp, vp, vp, sz, vp]
        L.spec_flat_pack.argtypes = [vp, i, vp, vp, i, i, vp, vp, sz, vp]
        L.spec_target_stats_flat.argtypes = [vp, i, f, i, i, i, vp, vp, vp, sz, vp]
        L.spec_verify_greedy_flat.argtypes = [vp, i, vp, vp, vp, i, i, i, vp, vp, vp, vp, sz, vp]
        L.spec_verify_rejection_flat.argtypes = [vp, vp, i, vp, vp, i, i, vp, vp, vp, vp, vp, vp,
                                                 vp, f, vp, vp, i, i, i, vp, vp, vp, vp, vp, sz,
                                                 vp]
        ll = ctypes.c_longlong
        L.spec_mx_code_bytes.argtypes = [i, i, i]
        L.spec_mx_code_bytes.restype = sz
        L.spec_mx_scale_bytes.argtypes = [i, i]
        L.spec_mx_scale_bytes.restype = sz
        L.spec_mx_quantize.argtypes = [vp, i, ll, i, i, i, vp, vp, vp, sz, vp]
        L.spec_mx_dequantize.argtypes = [vp, vp, i, i, i, vp, i, ll, vp, sz, vp]
        L.spec_rmsnorm_mx.argtypes = [vp, ll, vp, ll, i, vp, i, f, i, i, vp, ll, i, vp, vp, vp, sz,
                                      vp]
        L.spec_mx_logits.argtypes = [vp, vp, i, vp, vp, i, i, i, i, vp, i, ll, vp, sz, vp]
        L.spec_token_logprobs.argtypes = [vp, i, ll, vp, f, i, i, i, vp, vp, vp, vp, vp, vp, sz,
                                          vp]
        L.spec_launch_count.restype = ctypes.c_ulonglong
        L.spec_trace_events.argtypes = [i, vp, vp, i]
        L.spec_trace_events.restype = i
        L.spec_trace_count.argtypes = [i]
        L.spec_trace_count.restype = i
        for name in ("spec_workspace_init", "spec_device_status", "spec_markov_propose",
                     "spec_verify_greedy", "spec_target_stats", "spec_verify_rejection",
                     "spec_tv_confidence", "spec_schedule_prefix", "spec_schedule_topk",
                     "spec_verify_greedy_noalloc", "spec_markov_propose_masked",
                     "spec_verify_rejection_masked", "spec_tv_confidence_masked",
                     "spec_markov_propose_target_stats", "spec_mtp_greedy",
                     "spec_flat_layout", "spec_flat_pack", "spec_target_stats_flat",
                     "spec_verify_greedy_flat",
                     "spec_verify_rejection_flat", "spec_mx_quantize", "spec_mx_dequantize",
                     "spec_rmsnorm_mx", "spec_mx_logits", "spec_token_logprobs"):
            getattr(L, name).restype = i
        _lib = L
    return _lib


# ----------------------------------------------------------------------------- marshalling

def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SPEC_F32
    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    raise TypeError(f"logits and weights must be float32 or bfloat16, got {t.dtype}")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libspecmarkov takes device tensors")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _mask(allowed, R, V):
    """Allowed-token bitmask [R, ceil(V/32)] of 32-bit words on the device."""
    if tuple(allowed.shape) != (R, (V + 31) // 32) or allowed.element_size() != 4:
        raise ValueError(f"allowed must be [R, ceil(V/32)] = {(R, (V + 31) // 32)} 32-bit words")
    return allowed


def _check(fn, rc):
    if rc != SPEC_OK:
        raise SpecError(fn, rc)


class Workspace:
    """Caller-owned device workspace (a torch uint8 buffer) for the library's scratch."""

    def __init__(self, nbytes: int = 0, device=None):
        self.device = torch.device(device) if device is not None else torch.device("cuda")
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.buf = None
        self.nbytes = 0
        if nbytes:
            self.reserve(nbytes)

    def reserve(self, nbytes: int, stream=None):
        if self.buf is not None and self.nbytes >= nbytes:
            return
        nbytes = max(int(nbytes), 256)
        self.buf = torch.empty(nbytes + 256, dtype=torch.uint8, device=self.device)
        base = self.buf.data_ptr()
        self._off = (-base) % 256
        self._addr = base + self._off
        self.nbytes = nbytes
        _check("spec_workspace_init", lib().spec_workspace_init(self.ptr, nbytes, _stream(stream)))

    @property
    def ptr(self):
        return ctypes.c_void_p(self.buf.data_ptr() + self._off)

    def for_op(self, op, R, gamma, V, rank, stream=None):
        self.reserve(spec_workspace_bytes(op, R, gamma, V, rank), stream)
        return self.ptr, self.nbytes

    def status(self, clear=True, stream=None) -> int:
        out = ctypes.c_uint32()
        _check("spec_device_status", lib().spec_device_status(self.ptr, self.nbytes,
                                                              _stream(stream),
                                                              ctypes.byref(out), int(clear)))
        return int(out.value)


_default_ws = {}


def default_workspace(device=None) -> Workspace:
    dev = torch.cuda.current_device() if device is None else torch.device(device).index
    if dev not in _default_ws:
        _default_ws[dev] = Workspace(device=torch.device("cuda", dev))
    return _default_ws[dev]


def spec_workspace_bytes(op, R, gamma, V, rank=0) -> int:
    return int(lib().spec_workspace_bytes(op, R, gamma, V, rank))


def spec_abi_version() -> int:
    return int(lib().spec_abi_version())


def _rank_of(W1, rank):
    if rank is not None:
        return int(rank)
    return 0 if W1 is None else int(W1.shape[1])


# ----------------------------------------------------------------------------- entry points

def spec_markov_propose(U, W1, W2, anchors, u_draft, temperature, *, rank=None,
                        draft_tokens=None, draft_logp=None, draft_stats=None, workspace=None,
                        stream=None, want_stats=True, allowed=None):
    """Draft proposal (greedy when u_draft is None or temperature == 0); `allowed` is an
    optional allowed-token bitmask [R, ceil(V/32)] (int32 / uint32 words) for grammar-masked
    drafting. Returns (draft_tokens [R,g] int32, draft_logp [R,g] fp32, draft_stats [R,g,2])."""
    R, gamma, V = U.shape
    rank = _rank_of(W1, rank)
    dev = U.device
    if draft_tokens is None:
        draft_tokens = torch.empty(R, gamma, dtype=torch.int32, device=dev)
    if want_stats and draft_logp is None:
        draft_logp = torch.empty(R, gamma, dtype=torch.float32, device=dev)
    if want_stats and draft_stats is None:
        draft_stats = torch.empty(R, gamma, 2, dtype=torch.float32, device=dev)
    ws = workspace or default_workspace(dev)
    wp, wn = ws.for_op(SPEC_OP_PROPOSE, R, gamma, V, rank, stream)
    wdt = _dt(W1) if W1 is not None else SPEC_BF16
    args = (_ptr(U), _dt(U), _ptr(W1), _ptr(W2), wdt, rank, _ptr(anchors), _ptr(u_draft),
            float(temperature), R, gamma, V, _ptr(draft_tokens), _ptr(draft_logp),
            _ptr(draft_stats))
    if allowed is None:
        rc = lib().spec_markov_propose(*args, wp, wn, _stream(stream))
    else:
        rc = lib().spec_markov_propose_masked(*args, _ptr(_mask(allowed, R, V)), wp, wn,
                                              _stream(stream))
    _check("spec_markov_propose", rc)
    return draft_tokens, draft_logp, draft_stats


def spec_markov_propose_target_stats(U, W1, W2, anchors, u_draft, temperature, target, *,
                                     rank=None, draft_tokens=None, draft_logp=None,
                                     draft_stats=None, target_stats=None, workspace=None,
                                     stream=None):
    """Draft proposal plus the target normalisers of the same window in one call. Returns
    (draft_tokens [R,g] int32, draft_logp [R,g] fp32, draft_stats [R,g,2],
    target_stats [R*(g+1), 2] fp32)."""
    R, gamma, V = U.shape
    rank = _rank_of(W1, rank)
    dev = U.device
    if draft_tokens is None:
        draft_tokens = torch.empty(R, gamma, dtype=torch.int32, device=dev)
    if draft_logp is None:
        draft_logp = torch.empty(R, gamma, dtype=torch.float32, device=dev)
    if draft_stats is None:
        draft_stats = torch.empty(R, gamma, 2, dtype=torch.float32, device=dev)
    if target_stats is None:
        target_stats = torch.empty(R * (gamma + 1), 2, dtype=torch.float32, device=dev)
    ws = workspace or default_workspace(dev)
    wp, wn = ws.for_op(SPEC_OP_PROPOSE, R, gamma, V, rank, stream)
    wdt = _dt(W1) if W1 is not None else SPEC_BF16
    rc = lib().spec_markov_propose_target_stats(
        _ptr(U), _dt(U), _ptr(W1), _ptr(W2), wdt, rank, _ptr(anchors), _ptr(u_draft),
        float(temperature), R, gamma, V, _ptr(draft_tokens), _ptr(draft_logp), _ptr(draft_stats),
        _ptr(target), _ptr(target_stats), wp, wn, _stream(stream))
    _check("spec_markov_propose_target_stats", rc)
    return draft_tokens, draft_logp, draft_stats, target_stats


def spec_mtp_greedy(D, target, lengths=None, *, draft_tokens=None, accept_len=None,
                    out_tokens=None, next_anchor=None, workspace=None, stream=None):
    """MTP/NextN greedy proposal (draft argmax per position) and greedy verification in one
    call. D [R, gamma, V] and target [R, gamma+1, V] of one dtype. Returns (draft_tokens [R,g],
    accept_len [R], out_tokens [R, g+1], next_anchor [R]), all int32."""
    R, rows, V = target.shape
    gamma = rows - 1
    dev = target.device
    if gamma > 0 and (D is None or tuple(D.shape) != (R, gamma, V) or D.dtype != target.dtype):
        raise ValueError("D must be [R, gamma, V] with the target's dtype")
    i32 = dict(dtype=torch.int32, device=dev)
    if draft_tokens is None:
        draft_tokens = torch.empty(R, gamma, **i32)
    if accept_len is None:
        accept_len = torch.empty(R, **i32)
    if out_tokens is None:
        out_tokens = torch.empty(R, gamma + 1, **i32)
    if next_anchor is None:
        next_anchor = torch.empty(R, **i32)
    ws = workspace or default_workspace(dev)
    wp, wn = ws.for_op(SPEC_OP_MTP_GREEDY, R, gamma, V, 0, stream)
    rc = lib().spec_mtp_greedy(_ptr(D), _ptr(target), _dt(target), _ptr(lengths), R, gamma, V,
                               _ptr(draft_tokens), _ptr(accept_len), _ptr(out_tokens),
                               _ptr(next_anchor), wp, wn, _stream(stream))
    _check("spec_mtp_greedy", rc)
    return draft_tokens, accept_len, out_tokens, next_anchor


def spec_verify_greedy(target, draft_tokens, lengths=None, *, accept_len=None, out_tokens=None,
                       next_anchor=None, workspace=None, stream=None):
    R, rows, V = target.shape
    gamma = rows - 1
    dev = target.device
    if accept_len is None:
        accept_len = torch.empty(R, dtype=torch.int32, device=dev)
    if out_tokens is None:
        out_tokens = torch.empty(R, gamma + 1, dtype=torch.int32, device=dev)
    if next_anchor is None:
        next_anchor = torch.empty(R, dtype=torch.int32, device=dev)
    ws = workspace or default_workspace(dev)
    wp, wn = ws.for_op(SPEC_OP_VERIFY_GREEDY, R, gamma, V, 0, stream)
    rc = lib().spec_verify_greedy(_ptr(target), _dt(target), _ptr(draft_tokens), _ptr(lengths), R,
                                  gamma, V, _ptr(accept_len), _ptr(out_tokens), _ptr(next_anchor),
                                  wp, wn, _stream(stream))
    _check("spec_verify_greedy", rc)
    return accept_len, out_tokens, next_anchor


def spec_verify_greedy_noalloc(target, draft_tokens, lengths=None, *, accept_len=None,
                               out_tokens=None, next_anchor=None, device_status=None, stream=None):
    """spec_verify_greedy without a workspace, for callers that cannot allocate device memory
    where they call it: the library's own fixed device scratch stands in for the workspace.
    Output tensors left as None are allocated here by torch (pass them to avoid that);
    `device_status` is an optional int32 device tensor of one element that receives the call's
    SPEC_DEV_* bits."""
    R, rows, V = target.shape
    gamma = rows - 1
    dev = target.device
    if accept_len is None:
        accept_len = torch.empty(R, dtype=torch.int32, device=dev)
    if out_tokens is None:
        out_tokens = torch.empty(R, gamma + 1, dtype=torch.int32, device=dev)
    if next_anchor is None:
        next_anchor = torch.empty(R, dtype=torch.int32, device=dev)
    rc = lib().spec_verify_greedy_noalloc(_ptr(target), _dt(target), _ptr(draft_tokens),
                                          _ptr(lengths), R, gamma, V, _ptr(accept_len),
                                          _ptr(out_tokens), _ptr(next_anchor),
                                          _ptr(device_status), _stream(stream))
    _check("spec_verify_greedy_noalloc", rc)
    return accept_len, out_tokens, next_anchor


def spec_target_stats(target, temperature, *, stats=None, workspace=None, stream=None):
    V = target.shape[-1]
    rows = target.numel() // V
    if stats is None:
        stats = torch.empty(rows, 2, dtype=torch.float32, device=target.device)
    ws = workspace or default_workspace(target.device)
    wp, wn = ws.for_op(SPEC_OP_TARGET_STATS, 1 if rows else 0, max(rows - 1, 0), V, 0, stream)
    rc = lib().spec_target_stats(_ptr(target), _dt(target), float(temperature), rows, V,
                                 _ptr(stats), wp, wn, _stream(stream))
    _check("spec_target_stats", rc)
    return stats


def spec_verify_rejection(target, U, W1, W2, anchors, draft_tokens, draft_logp, draft_stats,
                          u_accept, u_resid, temperature, lengths=None, *, rank=None,
                          target_stats=None, accept_len=None, out_tokens=None, next_anchor=None,
                          workspace=None, stream=None, allowed=None):
    R, gamma, V = U.shape
    rank = _rank_of(W1, rank)
    dev = U.device
    if accept_len is None:
        accept_len = torch.empty(R, dtype=torch.int32, device=dev)
    if out_tokens is None:
        out_tokens = torch.empty(R, gamma + 1, dtype=torch.int32, device=dev)
    if next_anchor is None:
        next_anchor = torch.empty(R, dtype=torch.int32, device=dev)
    ws = workspace or default_workspace(dev)
    wp, wn = ws.for_op(SPEC_OP_VERIFY_REJECTION, R, gamma, V, rank, stream)
    wdt = _dt(W1) if W1 is not None else SPEC_BF16
    args = (_ptr(target), _ptr(U), _dt(U), _ptr(W1), _ptr(W2), wdt, rank, _ptr(anchors),
            _ptr(draft_tokens), _ptr(draft_logp), _ptr(draft_stats), _ptr(target_stats),
            _ptr(u_accept), _ptr(u_resid), float(temperature), _ptr(lengths), R, gamma, V,
            _ptr(accept_len), _ptr(out_tokens), _ptr(next_anchor))
    if allowed is None:
        rc = lib().spec_verify_rejection(*args, wp, wn, _stream(stream))
    else:
        rc = lib().spec_verify_rejection_masked(*args, _ptr(_mask(allowed, R, V)), wp, wn,
                                                _stream(stream))
    _check("spec_verify_rejection", rc)
    return accept_len, out_tokens, next_anchor


def spec_tv_confidence(U, target, W1, W2, anchors, draft_tokens, temperature, *, rank=None,
                       draft_stats=None, target_stats=None, conf=None, survival=None,
                       workspace=None, stream=None, allowed=None):
    R, gamma, V = U.shape
    rank = _rank_of(W1, rank)
    dev = U.device
    if conf is None:
        conf = torch.empty(R, gamma, dtype=torch.float32, device=dev)
    if survival is None:
        survival = torch.empty(R, gamma, dtype=torch.float32, device=dev)
    ws = workspace or default_workspace(dev)
    wp, wn = ws.for_op(SPEC_OP_TV_CONFIDENCE, R, gamma, V, rank, stream)
    wdt = _dt(W1) if W1 is not None else SPEC_BF16
    args = (_ptr(U), _ptr(target), _dt(U), _ptr(W1), _ptr(W2), wdt, rank, _ptr(anchors),
            _ptr(draft_tokens), _ptr(draft_stats), _ptr(target_stats), float(temperature), R,
            gamma, V, _ptr(conf), _ptr(survival))
    if allowed is None:
        rc = lib().spec_tv_confidence(*args, wp, wn, _stream(stream))
    else:
        rc = lib().spec_tv_confidence_masked(*args, _ptr(_mask(allowed, R, V)), wp, wn,
                                             _stream(stream))
    _check("spec_tv_confidence", rc)
    return conf, survival


def spec_schedule_prefix(survival, sps, *, lengths=None, B_out=None, theta_out=None,
                         workspace=None, stream=None, capacity=None, B_opt_out=None):
    """Prefix scheduler. With `capacity` (a [1] int32 device tensor holding a batch size,
    typically the Theta-optimal batch of an earlier step) it is the dynamic top-K selection
    instead of the Theta search; `B_opt_out` ([1] int32, optional) then receives this step's
    Theta-optimal batch size."""
    R, gamma = survival.shape
    dev = survival.device
    if lengths is None:
        lengths = torch.empty(R, dtype=torch.int32, device=dev)
    if B_out is None:
        B_out = torch.empty(1, dtype=torch.int32, device=dev)
    if theta_out is None:
        theta_out = torch.empty(1, dtype=torch.float64, device=dev)
    ws = workspace or default_workspace(dev)
    ws.reserve(256, stream)
    if capacity is None:
        if B_opt_out is not None:
            raise ValueError("B_opt_out is an output of the capacity form")
        rc = lib().spec_schedule_prefix(_ptr(survival), _ptr(sps), sps.numel() - 1, R, gamma,
                                        _ptr(lengths), _ptr(B_out), _ptr(theta_out), ws.ptr,
                                        ws.nbytes, _stream(stream))
    else:
        if capacity.dtype != torch.int32 or capacity.numel() < 1 or capacity.device != dev:
            raise ValueError("capacity must be an int32 tensor on the survival's device")
        if B_opt_out is not None and (B_opt_out.dtype != torch.int32 or B_opt_out.device != dev):
            raise ValueError("B_opt_out must be an int32 tensor on the survival's device")
        rc = lib().spec_schedule_topk(_ptr(survival), _ptr(sps), sps.numel() - 1, R, gamma,
                                      _ptr(capacity), _ptr(lengths), _ptr(B_out),
                                      _ptr(theta_out),
                                      None if B_opt_out is None else _ptr(B_opt_out), ws.ptr,
                                      ws.nbytes, _stream(stream))
    _check("spec_schedule_prefix", rc)
    return lengths, B_out, theta_out


# ----------------------------------------------------------------------------- flattened batch

def _i32_on(t, dev, name):
    if t.dtype != torch.int32 or t.device != dev:
        raise ValueError(f"{name} must be an int32 tensor on {dev}")
    return t


def spec_flat_layout(lengths, gamma, *, offsets=None, row_req=None, row_pos=None, markers=True,
                     workspace=None, stream=None):
    """Packed-row layout of a variable-length verify batch: offsets [R+1] (offsets[R] = B) and,
    with markers=True, the request / position of each of the R*(gamma+1) packed rows (-1 past
    B). Returns (offsets, row_req, row_pos)."""
    R = lengths.shape[0]
    dev = lengths.device
    _i32_on(lengths, dev, "lengths")
    if offsets is None:
        offsets = torch.empty(R + 1, dtype=torch.int32, device=dev)
    if markers and row_req is None:
        row_req = torch.empty(R * (gamma + 1), dtype=torch.int32, device=dev)
    if markers and row_pos is None:
        row_pos = torch.empty(R * (gamma + 1), dtype=torch.int32, device=dev)
    ws = workspace or default_workspace(dev)
    ws.reserve(256, stream)
    rc = lib().spec_flat_layout(_ptr(lengths), R, int(gamma), _ptr(offsets), _ptr(row_req),
                                _ptr(row_pos), ws.ptr, ws.nbytes, _stream(stream))
    _check("spec_flat_layout", rc)
    return offsets, row_req, row_pos


def spec_flat_pack(src, lengths, offsets, *, out=None, workspace=None, stream=None):
    """Rows (r, i <= l_r) of a padded src [R, gamma+1, ...] to packed rows offsets[r] + i of
    out [R*(gamma+1), ...] (allocated when None; rows past B are left as they were)."""
    R, g1 = src.shape[0], src.shape[1]
    dev = src.device
    _i32_on(lengths, dev, "lengths")
    _i32_on(offsets, dev, "offsets")
    row_bytes = src[0, 0].numel() * src.element_size() if src.numel() else 4
    if out is None:
        out = torch.empty((R * g1,) + tuple(src.shape[2:]), dtype=src.dtype, device=dev)
    if out.numel() != src.numel() or out.dtype != src.dtype:
        raise ValueError("out holds R*(gamma+1) rows of src's row shape and dtype")
    ws = workspace or default_workspace(dev)
    ws.reserve(256, stream)
    rc = lib().spec_flat_pack(_ptr(src), int(row_bytes), _ptr(lengths), _ptr(offsets), R,
                              g1 - 1, _ptr(out), ws.ptr, ws.nbytes, _stream(stream))
    _check("spec_flat_pack", rc)
    return out


def spec_target_stats_flat(target, temperature, offsets, gamma, *, stats=None, workspace=None,
                           stream=None):
    """(m, log Z) of the packed target rows b < offsets[R]; target [R*(gamma+1), V]."""
    R = offsets.shape[0] - 1
    V = target.shape[-1]
    dev = target.device
    if target.numel() != R * (gamma + 1) * V:
        raise ValueError("a packed target holds R*(gamma+1) rows")
    _i32_on(offsets, dev, "offsets")
    if stats is None:
        stats = torch.empty(R * (gamma + 1), 2, dtype=torch.float32, device=dev)
    ws = workspace or default_workspace(dev)
    wp, wn = ws.for_op(SPEC_OP_TARGET_STATS, R, gamma, V, 0, stream)
    rc = lib().spec_target_stats_flat(_ptr(target), _dt(target), float(temperature), R,
                                      int(gamma), V, _ptr(offsets), _ptr(stats), wp, wn,
                                      _stream(stream))
    _check("spec_target_stats_flat", rc)
    return stats


def spec_verify_greedy_flat(target, draft_tokens, lengths, offsets, *, accept_len=None,
                            out_tokens=None, next_anchor=None, workspace=None, stream=None):
    """Greedy verify with the target rows packed by spec_flat_layout (target [R*(gamma+1), V])."""
    R, gamma = draft_tokens.shape
    V = target.shape[-1]
    dev = target.device
    if target.numel() != R * (gamma + 1) * V:
        raise ValueError("a packed target holds R*(gamma+1) rows")
    _i32_on(lengths, dev, "lengths")
    _i32_on(offsets, dev, "offsets")
    if accept_len is None:
        accept_len = torch.empty(R, dtype=torch.int32, device=dev)
    if out_tokens is None:
        out_tokens = torch.empty(R, gamma + 1, dtype=torch.int32, device=dev)
    if next_anchor is None:
        next_anchor = torch.empty(R, dtype=torch.int32, device=dev)
    ws = workspace or default_workspace(dev)
    wp, wn = ws.for_op(SPEC_OP_VERIFY_GREEDY, R, gamma, V, 0, stream)
    rc = lib().spec_verify_greedy_flat(_ptr(target), _dt(target), _ptr(draft_tokens),
                                       _ptr(lengths), _ptr(offsets), R, gamma, V,
                                       _ptr(accept_len), _ptr(out_tokens), _ptr(next_anchor),
                                       wp, wn, _stream(stream))
    _check("spec_verify_greedy_flat", rc)
    return accept_len, out_tokens, next_anchor


def spec_verify_rejection_flat(target, U, W1, W2, anchors, draft_tokens, draft_logp,
                               draft_stats, u_accept, u_resid, temperature, lengths, offsets, *,
                               rank=None, target_stats=None, accept_len=None, out_tokens=None,
                               next_anchor=None, workspace=None, stream=None, allowed=None):
    """Rejection verify with the target rows (and target_stats, if given) packed by
    spec_flat_layout; everything else keeps its per-request layout."""
    R, gamma, V = U.shape
    rank = _rank_of(W1, rank)
    dev = U.device
    if target.numel() != R * (gamma + 1) * V:
        raise ValueError("a packed target holds R*(gamma+1) rows")
    _i32_on(lengths, dev, "lengths")
    _i32_on(offsets, dev, "offsets")
    if accept_len is None:
        accept_len = torch.empty(R, dtype=torch.int32, device=dev)
    if out_tokens is None:
        out_tokens = torch.empty(R, gamma + 1, dtype=torch.int32, device=dev)
    if next_anchor is None:
        next_anchor = torch.empty(R, dtype=torch.int32, device=dev)
    ws = workspace or default_workspace(dev)
    wp, wn = ws.for_op(SPEC_OP_VERIFY_REJECTION, R, gamma, V, rank, stream)
    wdt = _dt(W1) if W1 is not None else SPEC_BF16
    mask = None if allowed is None else _mask(allowed, R, V)
    rc = lib().spec_verify_rejection_flat(
        _ptr(target), _ptr(U), _dt(U), _ptr(W1), _ptr(W2), wdt, rank, _ptr(anchors),
        _ptr(draft_tokens), _ptr(draft_logp), _ptr(draft_stats), _ptr(target_stats),
        _ptr(u_accept), _ptr(u_resid), float(temperature), _ptr(lengths), _ptr(offsets), R,
        gamma, V, _ptr(accept_len), _ptr(out_tokens), _ptr(next_anchor), _ptr(mask), wp, wn,
        _stream(stream))
    _check("spec_verify_rejection_flat", rc)
    return accept_len, out_tokens, next_anchor


# ----------------------------------------------------------------------------- vocabulary head
# These calls are short at small batches, so their binding is written for few host operations:
# one allocation a matrix, plain integers for pointers, views made only when they are read.

_DTYPES = {torch.float32: SPEC_F32, torch.bfloat16: SPEC_BF16}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda i: torch.cuda.current_stream(i).cuda_stream)


def _mx_sizes(rows, K, fmt):
    """Bytes of a row of codes, number of scale tiles, 128-element groups of a row."""
    if fmt not in (SPEC_MX_E2M1, SPEC_MX_E4M3):
        raise ValueError("fmt must be SPEC_MX_E2M1 or SPEC_MX_E4M3")
    if K < 1:
        raise ValueError("a block-scaled matrix has at least one column")
    G = -(-K // SPEC_MX_GROUP)
    return G * (SPEC_MX_GROUP // 2 if fmt == SPEC_MX_E2M1 else SPEC_MX_GROUP), -(-rows // 128), G


class MXTensor:
    """A block-scaled [rows, K] matrix: `codes` [rows, Kp / 2] (SPEC_MX_E2M1) or [rows, Kp]
    (SPEC_MX_E4M3) and `scales` [ceil(rows / 128), Kp / 128, 32, 4, 4], both contiguous uint8 on
    the device (Kp = K rounded up to a multiple of 128; the layout is that of
    include/spec_markov.h)."""

    __slots__ = ("rows", "K", "fmt", "device", "_buf", "_codes", "_scales", "_cp", "_sp")

    def __init__(self, codes, scales, fmt, K):
        rows = codes.shape[0]
        width, tiles, G = _mx_sizes(rows, K, fmt)
        if codes.dtype != torch.uint8 or codes.shape != (rows, width) or not codes.is_contiguous():
            raise ValueError(f"codes must be contiguous uint8 [rows, {width}]")
        if (scales.dtype != torch.uint8 or scales.shape != (tiles, G, 32, 4, 4)
                or not scales.is_contiguous()):
            raise ValueError(f"scales must be contiguous uint8 {(tiles, G, 32, 4, 4)}")
        if scales.device != codes.device or not codes.is_cuda:
            raise ValueError("codes and scales must be on one CUDA device")
        self.rows, self.K, self.fmt, self.device = rows, K, fmt, codes.device
        self._buf, self._codes, self._scales = None, codes, scales
        self._cp, self._sp = codes.data_ptr(), scales.data_ptr()

    @classmethod
    def empty(cls, rows, K, fmt, device):
        """An uninitialised [rows, K] matrix for a call to write."""
        width, tiles, G = _mx_sizes(rows, K, fmt)
        q = cls.__new__(cls)
        n = rows * width
        q._buf = buf = torch.empty(n + tiles * G * 512, dtype=torch.uint8, device=device)
        if not buf.is_cuda:
            raise ValueError("libspecmarkov takes device tensors")
        q.rows, q.K, q.fmt, q.device = rows, K, fmt, buf.device
        q._codes = q._scales = None
        q._cp = at = buf.data_ptr()
        q._sp = at + n
        return q

    @property
    def codes(self):
        if self._codes is None:
            width = _mx_sizes(self.rows, self.K, self.fmt)[0]
            self._codes = self._buf[:self.rows * width].view(self.rows, width)
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            width, tiles, G = _mx_sizes(self.rows, self.K, self.fmt)
            self._scales = self._buf[self.rows * width:].view(tiles, G, 32, 4, 4)
        return self._scales

    @property
    def shape(self):
        return self.rows, self.K


def _rows(t, name):
    """(address, rows, width, row stride) of a matrix whose rows are contiguous: two dimensions
    with any row stride, or more dimensions that flatten into evenly spaced rows."""
    if not t.is_cuda:
        raise ValueError("libspecmarkov takes device tensors")
    shape, strides = t.shape, t.stride()
    if not shape:
        raise ValueError(f"{name} must have at least one dimension")
    width = shape[-1]
    if width > 1 and strides[-1] != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    if len(shape) == 2:
        return t.data_ptr(), shape[0], width, strides[0] if shape[0] > 1 else width
    # leading dimensions of more than one index, innermost last
    lead = [(n, st) for n, st in zip(shape[:-1], strides[:-1]) if n != 1]
    rows = 1
    for n, _ in lead:
        rows *= n
    if not lead or rows == 0:
        return t.data_ptr(), rows, width, width
    ld = span = lead[-1][1]
    for n, st in reversed(lead):
        if st != span:
            raise ValueError(f"the rows of {name} must be evenly spaced")
        span = st * n
    return t.data_ptr(), rows, width, ld


def _on(dev, t, name):
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}")


def _dtype_code(dtype):
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"logits and weights must be float32 or bfloat16, got {dtype}")
    return code


_entry = {}  # entry points by name, looked up once


def _launch(name, dev, workspace, stream, *args):
    """Call entry point `name` with args, the status workspace and the stream. The operands'
    device is current meanwhile and its current stream is the default."""
    i = dev.index
    ws = workspace or _default_ws.get(i) or default_workspace(dev)
    if ws.device.index != i:
        raise ValueError(f"the workspace must be on {dev}")
    if torch._C._cuda_getDevice() != i:
        with torch.cuda.device(i):
            return _launch(name, dev, ws, stream, *args)
    if ws.buf is None:
        ws.reserve(256, stream)
    fn = _entry.get(name)
    if fn is None:
        fn = _entry[name] = getattr(lib(), name)
    rc = fn(*args, ws._addr, ws.nbytes, _raw_stream(i) if stream is None else stream.cuda_stream)
    if rc != SPEC_OK:
        raise SpecError(name, rc)


def _on_stream(stream, new, *args, **kw):
    """new(*args), with its memory from the stream that will write it: that of the current one
    could still be in use there, or be given away there while `stream` uses it."""
    if stream is None:
        return new(*args, **kw)
    with torch.cuda.stream(stream):
        return new(*args, **kw)


def _mx_out(out, rows, K, fmt, dev, stream):
    if out is None:
        return _on_stream(stream, MXTensor.empty, rows, K, fmt, dev)
    if out.rows != rows or out.K != K or out.fmt != fmt:
        raise ValueError("out must be an MXTensor of x's rows, width and the given format")
    if out.device != dev:
        raise ValueError(f"out must be on {dev}")
    return out


def spec_mx_quantize(x, fmt=SPEC_MX_E2M1, *, out=None, workspace=None, stream=None):
    """x [rows, K] (or [..., K], evenly spaced rows; bf16 or fp32) as a block-scaled MXTensor of
    `fmt`: SPEC_MX_E2M1 for a vocabulary matrix, SPEC_MX_E4M3 for hidden rows. `out` is an
    MXTensor to write into."""
    ptr, rows, K, ld = _rows(x, "x")
    dt, dev = _dtype_code(x.dtype), x.device
    out = _mx_out(out, rows, K, fmt, dev, stream)
    _launch("spec_mx_quantize", dev, workspace, stream, ptr, dt, ld, rows, K, fmt, out._cp,
            out._sp)
    return out


def spec_mx_dequantize(q, *, dtype=torch.bfloat16, out=None, workspace=None, stream=None):
    """The numbers that the MXTensor q stands for, [rows, K] of `dtype` (bf16 or fp32)."""
    rows, K, dev = q.rows, q.K, q.device
    if out is None:
        dt = _dtype_code(dtype)
        out = _on_stream(stream, torch.empty, rows, K, dtype=dtype, device=dev)
        ptr, ld = out.data_ptr(), K
    else:
        dt = _dtype_code(out.dtype)
        ptr, orows, width, ld = _rows(out, "out")
        if orows != rows or width != K:
            raise ValueError("out must have q's rows and width")
        _on(dev, out, "out")
    _launch("spec_mx_dequantize", dev, workspace, stream, q._cp, q._sp, q.fmt, rows, K, ptr, dt,
            ld)
    return out


def spec_rmsnorm_mx(x, weight, eps=1e-6, *, residual=None, residual_out=None, fmt=SPEC_MX_E4M3,
                    out=None, workspace=None, stream=None):
    """h = x + residual (x without one), then the RMS norm of h's rows times weight [K], block-
    scaled in `fmt`. x, residual [rows, K] (or [..., K], evenly spaced rows) of one dtype.
    Returns (h, MXTensor); h is residual_out (which may be x or residual itself), a new tensor,
    or x when there is no residual."""
    ptr, rows, K, ldx = _rows(x, "x")
    dt, dev = _dtype_code(x.dtype), x.device
    if weight.shape != (K,) or not weight.is_contiguous():
        raise ValueError(f"weight must be contiguous [{K}]")
    rp = op = None
    ldr = ldo = K
    h = x
    if residual is not None:
        if residual.shape != x.shape or residual.dtype != x.dtype:
            raise ValueError("residual must have x's shape and dtype")
        rp, _, _, ldr = _rows(residual, "residual")
        _on(dev, residual, "residual")
        if residual_out is None:
            h = _on_stream(stream, torch.empty, x.shape, dtype=x.dtype, device=dev)
            op = h.data_ptr()
        else:
            h = residual_out
            if h.shape != x.shape or h.dtype != x.dtype:
                raise ValueError("residual_out must have x's shape and dtype")
            op, _, _, ldo = _rows(h, "residual_out")
            _on(dev, h, "residual_out")
    elif residual_out is not None:
        raise ValueError("residual_out is an output of the form with a residual")
    _on(dev, weight, "weight")
    out = _mx_out(out, rows, K, fmt, dev, stream)
    _launch("spec_rmsnorm_mx", dev, workspace, stream, ptr, ldx, rp, ldr, dt, weight.data_ptr(),
            _dtype_code(weight.dtype), eps, rows, K, op, ldo, fmt, out._cp, out._sp)
    return h, out


def spec_mx_logits(a, w, *, dtype=torch.bfloat16, out=None, workspace=None, stream=None):
    """Logits [M, V] (bf16 or fp32) of the MXTensor rows a [M, K] against the vocabulary matrix
    w [V, K]. `out` [M, V] (or [..., V]) may have any even row spacing, for instance one position
    U[:, k] of U [R, gamma, V]."""
    M, V, K, dev = a.rows, w.rows, a.K, a.device
    if K != w.K:
        raise ValueError(f"a has rows of {K} elements, w of {w.K}")
    _on(dev, w, "w")
    if out is None:
        dt = _dtype_code(dtype)
        out = _on_stream(stream, torch.empty, M, V, dtype=dtype, device=dev)
        ptr, ld = out.data_ptr(), V
    else:
        dt = _dtype_code(out.dtype)
        ptr, rows, width, ld = _rows(out, "out")
        if rows != M or width != V:
            raise ValueError(f"out must hold {M} rows of {V}")
        _on(dev, out, "out")
    _launch("spec_mx_logits", dev, workspace, stream, a._cp, a._sp, a.fmt, w._cp, w._sp, w.fmt, M,
            V, K, ptr, dt, ld)
    return out


class TokenLogprobs:
    """Outputs of spec_token_logprobs: logp, rank, entropy [rows], top_ids, top_logp
    [rows, top]; None where not asked for."""

    __slots__ = ("logp", "rank", "entropy", "top_ids", "top_logp")

    def __init__(self, logp=None, rank=None, entropy=None, top_ids=None, top_logp=None):
        self.logp, self.rank, self.entropy = logp, rank, entropy
        self.top_ids, self.top_logp = top_ids, top_logp

    @classmethod
    def empty(cls, rows, top, tokens, device):
        """Uninitialised outputs for a call to write: every field, logp and rank only with
        `tokens`."""
        # tensors of their own: five small allocations take less than two and five views
        f, i, new = torch.float32, torch.int32, torch.empty
        return cls(new(rows, dtype=f, device=device) if tokens else None,
                   new(rows, dtype=i, device=device) if tokens else None,
                   new(rows, dtype=f, device=device),
                   new(rows, top, dtype=i, device=device) if top else None,
                   new(rows, top, dtype=f, device=device) if top else None)

    def _addresses(self, rows, top, dev):
        """Addresses of logp, rank, entropy, top_ids, top_logp (None where not asked for)."""
        out = []
        for name, dt, n in (("logp", torch.float32, rows), ("rank", torch.int32, rows),
                            ("entropy", torch.float32, rows), ("top_ids", torch.int32, rows * top),
                            ("top_logp", torch.float32, rows * top)):
            t = getattr(self, name)
            if t is not None and (t.dtype != dt or t.numel() != n or t.device != dev
                                  or not t.is_contiguous()):
                raise ValueError(f"{name} must hold {n} contiguous elements of {dt} on {dev}")
            out.append(None if t is None else t.data_ptr())
        return out


def spec_token_logprobs(logits, tokens, temperature=1.0, *, top=0, out=None, workspace=None,
                        stream=None):
    """Log-probability and rank of tokens[row] (int32, or None), entropy and the `top` most
    likely tokens under softmax(logits[row] / temperature); logits [rows, V] (or [..., V], evenly
    spaced rows). Rows whose token is -1 are left as they were. `out` is a TokenLogprobs whose
    None fields are not computed."""
    ptr, rows, V, ld = _rows(logits, "logits")
    dt, dev = _dtype_code(logits.dtype), logits.device
    if not 0 <= top <= SPEC_LOGPROBS_MAX_TOP:
        raise ValueError(f"top must be in [0, {SPEC_LOGPROBS_MAX_TOP}]")
    tp = None
    if tokens is not None:
        _i32_on(tokens, dev, "tokens")
        if tokens.numel() != rows or not tokens.is_contiguous():
            raise ValueError(f"tokens must hold {rows} contiguous ids")
        tp = tokens.data_ptr()
    if out is None:
        out = _on_stream(stream, TokenLogprobs.empty, rows, top, tokens is not None, dev)
        lp, rank = (None, None) if tp is None else (out.logp.data_ptr(), out.rank.data_ptr())
        ent = out.entropy.data_ptr()
        ti, tl = (out.top_ids.data_ptr(), out.top_logp.data_ptr()) if top else (None, None)
    else:
        lp, rank, ent, ti, tl = out._addresses(rows, top, dev)
        if tp is None and (lp is not None or rank is not None):
            raise ValueError("logp and rank need tokens")
    _launch("spec_token_logprobs", dev, workspace, stream, ptr, dt, ld, tp, temperature, rows, V,
            top, lp, rank, ent, ti, tl)
    return out


def spec_device_status(workspace=None, clear=True, stream=None) -> int:
    ws = workspace or default_workspace()
    return ws.status(clear=clear, stream=stream)
