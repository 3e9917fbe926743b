"""Thin Python binding of libkda.so (include/kda.h): argument marshalling only.

Every step of the operator runs in the library's CUDA kernels; this module
checks tensor placement/dtype/contiguity, allocates outputs and workspace
with torch when the caller did not pass them, and forwards raw device
pointers plus the current CUDA stream.  There is no CPU fallback: without
the compiled library or a CUDA device every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkda.so")

KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_CUDA, KDA_ERR_TIMEOUT = range(5)
KDA_F32, KDA_BF16 = 0, 1

# Every symbol include/kda.h declares, with (restype, argtypes).
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {
    "kda_status_string": (ctypes.c_char_p, [_i]),
    "kda_version": (_i, []),
    "kda_chunk_fwd_workspace_size": (_sz, [_i] * 7),
    "kda_chunk_fwd_launch_count": (_i, [_i] * 7),
    "kda_chunk_fwd": (_i, [_vp] * 5 + [_f, _vp, _vp, _vp] + [_i] * 7 + [_vp, _sz, _vp]),
    "kda_chunk_fwd_profiled": (_i, [_vp] * 5 + [_f, _vp, _vp, _vp] + [_i] * 7 + [_vp, _sz, _vp, _vp]),
    "kda_chunk_fwd_noalloc": (_i, [_vp] * 5 + [_f, _vp, _vp, _vp] + [_i] * 7 + [_vp]),
    "kda_chunk_fwd_check": (_i, [_vp, _sz, _vp]),
    "kda_chunk_fwd_noalloc_check": (_i, [_vp]),
    "kda_wait_selftest": (_i, [_vp, _sz, _vp]),
    "kda_recurrent_step": (_i, [_vp] * 5 + [_f, _vp, _vp] + [_i] * 5 + [_vp]),
    "kda_chunk_fwd_ex": (_i, [_vp] * 5 + [_f, _vp, _vp, _vp] + [_i] * 9 + [_vp, _sz, _vp]),
    "kda_recurrent_step_ex": (_i, [_vp] * 5 + [_f, _vp, _vp] + [_i] * 7 + [_vp]),
    "kda_backward_workspace_size": (_sz, [_i] * 6),
    "kda_backward": (_i, [_vp] * 5 + [_f] + [_vp] * 9 + [_i] * 7 + [_vp, _sz, _vp]),
    "kda_backward_ex_workspace_size": (_sz, [_i] * 7),
    "kda_backward_ex": (_i, [_vp] * 5 + [_f] + [_vp] * 9 + [_i] * 8 + [_vp, _sz, _vp]),
    "kda_scan_workspace_size": (_sz, [_i] * 5),
    "kda_scan_workspace_size_ex": (_sz, [_i] * 6),
    "kda_scan_checkpoint_size": (_sz, [_i] * 3),
    "kda_scan_fwd": (_i, [_vp] * 4 + [_i] + [_vp] * 3 + [_i] * 6 + [_vp, _sz, _vp]),
    "kda_scan_backward": (_i, [_vp] * 7 + [_i] + [_vp] * 3 + [_i] * 6 + [_vp, _sz, _vp]),
    "kda_scan_backward_ckpt": (_i, [_vp] * 4 + [_i] + [_vp] * 3 + [_i] * 6 + [_vp, _sz, _vp]),
    "kda_scan_step": (_i, [_vp] * 5 + [_i] * 5 + [_vp]),
}

# kda_gate: how the forget gate enters the update (see include/kda.h)
KDA_GATE_CHANNEL, KDA_GATE_HEAD, KDA_GATE_NONE = 0, 1, 2
# kda_prep bits: raw inputs prepared inside the kernels (see include/kda.h)
KDA_PREP_L2NORM_QK, KDA_PREP_GATE_LOGSIGMOID, KDA_PREP_BETA_SIGMOID = 1, 2, 4
KDA_PREP_ALL = KDA_PREP_L2NORM_QK | KDA_PREP_GATE_LOGSIGMOID | KDA_PREP_BETA_SIGMOID
# kda_scan_input: the weight of the input in the elementwise recurrence (1, or 1 - alpha)
KDA_SCAN_INPUT_PLAIN, KDA_SCAN_INPUT_COMPLEMENT = 0, 1


def _gate_kind(g, lead):
    """Gate kind from g's shape: per key channel [*lead, dk] (KDA), per head
    [*lead] (Gated DeltaNet), or None (DeltaNet)."""
    if g is None:
        return KDA_GATE_NONE
    if tuple(g.shape) == tuple(lead):
        return KDA_GATE_HEAD
    return KDA_GATE_CHANNEL

_lib = None


class KDAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def load(path: str = LIB_PATH):
    """Load libkda.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"libkda.so not built at {path}; run gated_delta_rule_67_b200.build.build()")
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load().kda_status_string(int(status)).decode()


def version() -> int:
    return int(load().kda_version())


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return KDA_F32
    if t == torch.bfloat16:
        return KDA_BF16
    raise TypeError(f"unsupported dtype {t}; KDA takes float32 or bfloat16")


def _check_dev(name, x, dtype=None):
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not x.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device (no CPU path exists)")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and x.dtype != dtype:
        raise TypeError(f"{name} has dtype {x.dtype}, expected {dtype}")


def _ptr(x):
    return None if x is None else ctypes.c_void_p(x.data_ptr())


def _stream(stream, device):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _on(device):
    """Makes the tensors' device current for the C call: the library keys its
    per-device set-up (function attributes, the static scratch) by the
    current device, which must own the buffers and the stream."""
    return torch.cuda.device(device)


def kda_chunk_fwd_workspace_size(B, T, H, dk, dv, chunk=64, dtype=torch.bfloat16) -> int:
    return int(load().kda_chunk_fwd_workspace_size(B, T, H, dk, dv, chunk, _dtype_code(dtype)))


def kda_chunk_fwd_launch_count(B, T, H, dk, dv, chunk=64, dtype=torch.bfloat16) -> int:
    """Kernels one kda_chunk_fwd call with these arguments launches (-1: rejected)."""
    return int(load().kda_chunk_fwd_launch_count(B, T, H, dk, dv, chunk, _dtype_code(dtype)))


def kda_chunk_fwd(q, k, v, g, beta, scale=None, initial_state=None, *, chunk=64, o=None, final_state=None,
                  output_final_state=True, workspace=None, stream=None, events=None, prep=0):
    """Chunked KDA prefill.  q,k [B,T,H,dk], v [B,T,H,dv], beta [B,T,H] (fp32 or bf16, CUDA).

    g selects the forget gate: [B,T,H,dk] per key channel (KDA), [B,T,H] one
    per head (Gated DeltaNet), or None (DeltaNet, no forgetting).
    ``prep``: KDA_PREP_* bits; the marked inputs are raw projections prepared
    in the kernels (q, k to unit length; g = logsigmoid(g); beta = sigmoid(beta)).
    Returns (o [B,T,H,dv] in the input dtype, final_state [B,H,dk,dv] fp32 or None).
    ``final_state`` may be ``initial_state`` itself for an in-place update.
    ``events``: optional three recorded torch.cuda.Event objects; the library
    records them before, between and after its kernels (kda_chunk_fwd_profiled,
    per-channel gates only).
    """
    lib = load()
    for name, x in (("q", q), ("k", k), ("v", v), ("beta", beta)):
        _check_dev(name, x, q.dtype)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    gate = _gate_kind(g, (B, T, H))
    if g is not None:
        _check_dev("g", g, q.dtype)
    if k.shape != q.shape or (gate == KDA_GATE_CHANNEL and g.shape != q.shape) or v.shape[:3] != (B, T, H) \
            or beta.shape != (B, T, H):
        raise ValueError("shape mismatch among q, k, v, g, beta")
    if scale is None:
        scale = dk ** -0.5
    code = _dtype_code(q.dtype)
    if initial_state is not None:
        _check_dev("initial_state", initial_state, torch.float32)
        if initial_state.shape != (B, H, dk, dv):
            raise ValueError("initial_state must be [B,H,dk,dv]")
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    _check_dev("o", o, q.dtype)
    if final_state is None and output_final_state:
        final_state = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    if final_state is not None:
        _check_dev("final_state", final_state, torch.float32)
    need = int(lib.kda_chunk_fwd_workspace_size(B, T, H, dk, dv, chunk, code))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale), _ptr(initial_state), _ptr(o),
            _ptr(final_state), B, T, H, dk, dv, chunk, code, _ptr(workspace), ws_bytes, _stream(stream, q.device))
    if gate != KDA_GATE_CHANNEL or prep:
        if events is not None:
            raise ValueError("events are recorded for prepared per-channel-gate inputs only")
        with _on(q.device):
            st = lib.kda_chunk_fwd_ex(*args[:16], gate, int(prep), *args[16:])
    elif events is None:
        with _on(q.device):
            st = lib.kda_chunk_fwd(*args)
    else:
        if len(events) != 3:
            raise ValueError("events must hold three torch.cuda.Event objects")
        handles = (ctypes.c_void_p * 3)(*[ev.cuda_event for ev in events])
        with _on(q.device):
            st = lib.kda_chunk_fwd_profiled(*args, handles)
    if st != KDA_OK:
        raise KDAError(st, "kda_chunk_fwd")
    return o, final_state


def kda_chunk_fwd_noalloc(q, k, v, g, beta, scale=None, initial_state=None, *, chunk=64, o=None,
                          final_state=None, output_final_state=True, stream=None):
    """kda_chunk_fwd using the library's static device scratch instead of a
    workspace: for callers that cannot allocate device memory.  Fits problems
    whose workspace is at most 64 MiB (about 900 chunk-heads, bf16); calls
    overlapping on the GPU race."""
    lib = load()
    for name, x in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta)):
        _check_dev(name, x, q.dtype)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if k.shape != q.shape or g.shape != q.shape or v.shape[:3] != (B, T, H) or beta.shape != (B, T, H):
        raise ValueError("shape mismatch among q, k, v, g, beta")
    if scale is None:
        scale = dk ** -0.5
    if initial_state is not None:
        _check_dev("initial_state", initial_state, torch.float32)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    _check_dev("o", o, q.dtype)
    if final_state is None and output_final_state:
        final_state = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    with _on(q.device):
        st = lib.kda_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale),
                                       _ptr(initial_state), _ptr(o), _ptr(final_state), B, T, H, dk, dv, chunk,
                                       _dtype_code(q.dtype), _stream(stream, q.device))
    if st != KDA_OK:
        raise KDAError(st, "kda_chunk_fwd_noalloc")
    return o, final_state


def kda_chunk_fwd_check(workspace, stream=None) -> int:
    """Status word a bounded on-device wait may have left in ``workspace`` (synchronises)."""
    if workspace is None:
        return KDA_OK
    with _on(workspace.device):
        return int(load().kda_chunk_fwd_check(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                              _stream(stream, workspace.device)))


def kda_chunk_fwd_noalloc_check(device=None, stream=None) -> int:
    """Status word of the static scratch after kda_chunk_fwd_noalloc calls on
    ``device`` (default: the current device); synchronises.  KDA_OK, or
    KDA_ERR_TIMEOUT if a bounded on-device wait of the last call gave up."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with _on(device):
        return int(load().kda_chunk_fwd_noalloc_check(_stream(stream, device)))


def kda_wait_selftest(workspace, stream=None) -> int:
    """Runs the bounded-wait failure path on the device (see include/kda.h); returns the status
    kda_chunk_fwd_check reads afterwards (KDA_ERR_TIMEOUT when the mechanism works)."""
    lib = load()
    nbytes = workspace.numel() * workspace.element_size()
    with _on(workspace.device):
        st = lib.kda_wait_selftest(_ptr(workspace), nbytes, _stream(stream, workspace.device))
    if st != KDA_OK:
        raise KDAError(st, "kda_wait_selftest")
    return kda_chunk_fwd_check(workspace, stream)


def kda_recurrent_step(q, k, v, g, beta, state, scale=None, *, o=None, stream=None, prep=0):
    """One decode step.  q,k [N,H,dk], v [N,H,dv], beta [N,H]; state [N,H,dk,dv] fp32 updated in place.

    g selects the forget gate: [N,H,dk] per key channel (KDA), [N,H] one per
    head (Gated DeltaNet), or None (DeltaNet).  ``prep``: KDA_PREP_* bits as for
    kda_chunk_fwd.  Returns o [N,H,dv] in the input dtype.
    """
    lib = load()
    for name, x in (("q", q), ("k", k), ("v", v), ("beta", beta)):
        _check_dev(name, x, q.dtype)
    _check_dev("state", state, torch.float32)
    N, H, dk = q.shape
    dv = v.shape[-1]
    gate = _gate_kind(g, (N, H))
    if g is not None:
        _check_dev("g", g, q.dtype)
    if k.shape != q.shape or (gate == KDA_GATE_CHANNEL and g.shape != q.shape) or v.shape[:2] != (N, H) \
            or beta.shape != (N, H):
        raise ValueError("shape mismatch among q, k, v, g, beta")
    if state.shape != (N, H, dk, dv):
        raise ValueError("state must be [N,H,dk,dv]")
    if scale is None:
        scale = dk ** -0.5
    if o is None:
        o = torch.empty((N, H, dv), dtype=q.dtype, device=q.device)
    _check_dev("o", o, q.dtype)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale), _ptr(state), _ptr(o), N, H, dk, dv,
            _dtype_code(q.dtype))
    with _on(q.device):
        if gate == KDA_GATE_CHANNEL and not prep:
            st = lib.kda_recurrent_step(*args, _stream(stream, q.device))
        else:
            st = lib.kda_recurrent_step_ex(*args, gate, int(prep), _stream(stream, q.device))
    if st != KDA_OK:
        raise KDAError(st, "kda_recurrent_step")
    return o


def kda_backward(q, k, v, g, beta, grad_o, scale=None, initial_state=None, grad_final_state=None, *,
                 workspace=None, stream=None, want_initial_state_grad=True, prep=0):
    """Gradients of a loss through kda_chunk_fwd (g per key channel [B,T,H,dk],
    per head [B,T,H] or None, as for the forward), given grad_o = dL/do
    [B,T,H,dv] and grad_final_state = dL/dS_T [B,H,dk,dv] fp32 (or None).
    ``prep``: the forward's KDA_PREP_* bits; q, k, g, beta are then the raw
    inputs and the gradients are taken with respect to them.

    Returns a dict: dq, dk, dv, dg (like g; None without a gate), dbeta (input
    dtype) and dS0 = dL/dS_0 fp32 (None if not wanted).
    """
    lib = load()
    for name, x in (("q", q), ("k", k), ("v", v), ("beta", beta), ("grad_o", grad_o)):
        _check_dev(name, x, q.dtype)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    gate = _gate_kind(g, (B, T, H))
    if g is not None:
        _check_dev("g", g, q.dtype)
    if k.shape != q.shape or (gate == KDA_GATE_CHANNEL and g.shape != q.shape) or v.shape[:3] != (B, T, H) \
            or beta.shape != (B, T, H) or grad_o.shape != v.shape:
        raise ValueError("shape mismatch among q, k, v, g, beta, grad_o")
    if scale is None:
        scale = dk ** -0.5
    for name, x in (("initial_state", initial_state), ("grad_final_state", grad_final_state)):
        if x is not None:
            _check_dev(name, x, torch.float32)
            if x.shape != (B, H, dk, dv):
                raise ValueError(f"{name} must be [B,H,dk,dv]")
    code = _dtype_code(q.dtype)
    out = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
               dg=None if g is None else torch.empty_like(g), dbeta=torch.empty_like(beta),
               dS0=torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device) if want_initial_state_grad
               else None)
    need = int(lib.kda_backward_ex_workspace_size(B, T, H, dk, dv, code, int(prep)))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    with _on(q.device):
        st = lib.kda_backward_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale), _ptr(initial_state),
                                 _ptr(grad_o), _ptr(grad_final_state), _ptr(out["dq"]), _ptr(out["dk"]),
                                 _ptr(out["dv"]), _ptr(out["dg"]), _ptr(out["dbeta"]), _ptr(out["dS0"]), B, T, H, dk,
                                 dv, code, gate, int(prep), _ptr(workspace), ws_bytes, _stream(stream, q.device))
    if st != KDA_OK:
        raise KDAError(st, "kda_backward")
    return out


def kda_scan_workspace_size(B, T, D, num_seqs=0, dtype=torch.bfloat16, checkpoint=True) -> int:
    """Bytes of workspace the scan calls need; less where kda_scan_fwd writes no checkpoint.  A call clears the
    workspace's header; kda_chunk_fwd_check(workspace) tells afterwards whether a wait in the kernel gave up."""
    return int(load().kda_scan_workspace_size_ex(B, T, D, num_seqs, _dtype_code(dtype), int(checkpoint)))


def kda_scan_checkpoint_size(B, T, D) -> int:
    """Bytes of the 8-bit activation checkpoint of kda_scan_fwd (its layout: include/kda.h)."""
    return int(load().kda_scan_checkpoint_size(B, T, D))


# The scan calls are short on the device, so their checks are kept short here: one test of everything, and
# only where it fails the one that names the fault.
def _same(name, x, shape, dtype, device):
    if not (isinstance(x, torch.Tensor) and x.dtype is dtype and x.shape == shape and x.device == device
            and x.is_contiguous()):
        _check_dev(name, x, dtype)
        raise ValueError(f"{name} must be {list(shape)} on {device}, not {list(x.shape)} on {x.device}")


def _scan_sizes(x, cu_seqlens):
    """(B, T, D, number of packed sequences) of the [B, T, D] tensor x."""
    if x.dim() != 3:
        raise ValueError("the sequence tensors must be [B,T,D]")
    B, T, D = x.shape
    if cu_seqlens is None:
        return B, T, D, 0
    _check_dev("cu_seqlens", cu_seqlens, torch.int32)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2 or cu_seqlens.device != x.device:
        raise ValueError(f"cu_seqlens must be [num_seqs + 1], num_seqs >= 1, on {x.device}")
    if B != 1:
        raise ValueError("packed sequences (cu_seqlens) need B = 1")
    return B, T, D, cu_seqlens.numel() - 1


def _at(x):
    return None if x is None else x.data_ptr()


# The workspace of a scan call depends on these sizes alone.
@functools.lru_cache(maxsize=1024)
def _scan_need(B, T, D, seqs, code, checkpoint):
    return int(load().kda_scan_workspace_size_ex(B, T, D, seqs, code, checkpoint))


def _state_like(given, shape, device):
    """An fp32 state of `shape`; a state of that shape at hand makes it quicker."""
    return torch.empty(shape, dtype=torch.float32, device=device) if given is None else torch.empty_like(given)


def _scan_on(stream, device, call, *args, **kw):
    """A scan call on ``stream``.  What it allocates is memory of that stream: memory of the current one may still
    be in use by work that the kernel would not wait for.  The results are recorded with the current stream, where
    the caller goes on with them."""
    if stream.device != device:
        raise ValueError(f"stream must belong to {device}, not {stream.device}")
    current = torch.cuda.current_stream(device)
    if stream == current:
        return call(*args, **kw)
    with torch.cuda.stream(stream):
        out = call(*args, **kw)
    for t in out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,):
        if t is not None:
            t.record_stream(current)
    return out


def _scan_call(name, device, args, need=None, workspace=None):
    """One call of the library on the device's current stream.  ``need``: for calls with a workspace, its size."""
    fn = getattr(_lib or load(), name)
    raw = torch._C._cuda_getCurrentRawStream(device.index)
    if torch.cuda.current_device() == device.index:
        st = _scan_launch(fn, args, need, workspace, raw)
    else:
        with _on(device):
            st = _scan_launch(fn, args, need, workspace, raw)
    if st != KDA_OK:
        raise KDAError(st, name)


def _scan_launch(fn, args, need, workspace, raw):
    if need is None:
        return fn(*args, raw)
    if workspace is not None:
        return fn(*args, workspace.data_ptr(), workspace.numel() * workspace.element_size(), raw)
    if not need:
        return fn(*args, None, 0, raw)
    # Memory of the stream that the kernels run on, given back at once: whoever gets it next comes after them there.
    # A tensor for it would take 1.5 us of a short call's 14, this 0.6.
    at = torch._C._cuda_cudaCachingAllocator_raw_alloc(need, raw)
    try:
        return fn(*args, at, need, raw)
    finally:
        torch._C._cuda_cudaCachingAllocator_raw_delete(at)


def _check_scan_workspace(workspace, device):
    _check_dev("workspace", workspace)
    if workspace.device != device:
        raise ValueError(f"workspace must live on {device}")


def kda_scan_fwd(x, g, initial_state=None, *, cu_seqlens=None, input_gate=KDA_SCAN_INPUT_PLAIN, prep=0, h=None,
                 final_state=None, output_final_state=True, checkpoint=None, workspace=None, stream=None):
    """Elementwise gated linear recurrence h_t = alpha_t h_{t-1} + w_t x_t over x, g [B,T,D] (fp32 or bf16, CUDA).

    alpha = exp(g), or sigmoid(g) with ``prep=KDA_PREP_GATE_LOGSIGMOID``; w = 1
    (KDA_SCAN_INPUT_PLAIN) or 1 - alpha (KDA_SCAN_INPUT_COMPLEMENT).  States are [B,D] fp32.
    ``cu_seqlens``: int32 [num_seqs + 1] on the device, packed sequences along the T rows of B = 1
    (states [num_seqs,D]); rows outside every sequence get zeros.
    ``checkpoint``: a uint8 tensor of kda_scan_checkpoint_size(B, T, D) bytes to fill with the 8-bit
    activation checkpoint that kda_scan_backward_ckpt reads.
    Returns (h [B,T,D] in the input dtype, final_state or None); ``final_state`` may be
    ``initial_state`` itself.
    """
    _check_dev("x", x)
    if stream is not None:
        return _scan_on(stream, x.device, kda_scan_fwd, x, g, initial_state, cu_seqlens=cu_seqlens, input_gate=input_gate,
                        prep=prep, h=h, final_state=final_state, output_final_state=output_final_state,
                        checkpoint=checkpoint, workspace=workspace)
    device, dtype, code = x.device, x.dtype, _dtype_code(x.dtype)
    B, T, D, seqs = _scan_sizes(x, cu_seqlens)
    state = (seqs or B, D)
    _same("g", g, x.shape, dtype, device)
    if initial_state is not None:
        _same("initial_state", initial_state, state, torch.float32, device)
    if h is None:
        h = torch.empty_like(x)
    else:
        _same("h", h, x.shape, dtype, device)
    if final_state is not None:
        _same("final_state", final_state, state, torch.float32, device)
    elif output_final_state:
        final_state = _state_like(initial_state, state, device)
    if checkpoint is not None:
        _check_ckpt(checkpoint, x.shape, device)
    if workspace is not None:
        _check_scan_workspace(workspace, device)
    _scan_call("kda_scan_fwd", device,
               (x.data_ptr(), g.data_ptr(), _at(initial_state), _at(cu_seqlens), seqs, h.data_ptr(), _at(final_state),
                _at(checkpoint), B, T, D, code, prep, input_gate),
               _scan_need(B, T, D, seqs, code, checkpoint is not None), workspace)
    return h, final_state


def _check_ckpt(checkpoint, shape, device):
    _check_dev("checkpoint", checkpoint, torch.uint8)
    need = kda_scan_checkpoint_size(*shape)
    if checkpoint.device != device or checkpoint.numel() < need:
        raise ValueError(f"checkpoint must hold {need} bytes on {device}")


def _scan_grads(like, state, given, want_initial_state_grad):
    out = dict(dx=torch.empty_like(like), dg=torch.empty_like(like), dS0=None)
    if want_initial_state_grad:
        out["dS0"] = _state_like(given, state, like.device)
    return out


def kda_scan_backward(x, g, h, grad_h, initial_state=None, grad_final_state=None, *, cu_seqlens=None,
                      input_gate=KDA_SCAN_INPUT_PLAIN, prep=0, workspace=None, stream=None,
                      want_initial_state_grad=True):
    """Gradients of a loss through kda_scan_fwd (same ``prep``, ``input_gate``, ``cu_seqlens``), given its inputs,
    its output h, grad_h = dL/dh and grad_final_state = dL/d final_state (or None).  x may be None for
    KDA_SCAN_INPUT_PLAIN.  Returns a dict: dx, dg (input dtype) and dS0 fp32 (None if not wanted).
    """
    _check_dev("grad_h", grad_h)
    if stream is not None:
        return _scan_on(stream, grad_h.device, kda_scan_backward, x, g, h, grad_h, initial_state, grad_final_state,
                        cu_seqlens=cu_seqlens, input_gate=input_gate, prep=prep, workspace=workspace,
                        want_initial_state_grad=want_initial_state_grad)
    device, dtype, code = grad_h.device, grad_h.dtype, _dtype_code(grad_h.dtype)
    B, T, D, seqs = _scan_sizes(grad_h, cu_seqlens)
    state = (seqs or B, D)
    if x is not None:
        _same("x", x, grad_h.shape, dtype, device)
    elif input_gate == KDA_SCAN_INPUT_COMPLEMENT:
        raise ValueError("x is needed for KDA_SCAN_INPUT_COMPLEMENT")
    _same("g", g, grad_h.shape, dtype, device)
    _same("h", h, grad_h.shape, dtype, device)
    if initial_state is not None:
        _same("initial_state", initial_state, state, torch.float32, device)
    if grad_final_state is not None:
        _same("grad_final_state", grad_final_state, state, torch.float32, device)
    out = _scan_grads(grad_h, state, grad_final_state if grad_final_state is not None else initial_state,
                      want_initial_state_grad)
    if workspace is not None:
        _check_scan_workspace(workspace, device)
    _scan_call("kda_scan_backward", device,
               (_at(x), g.data_ptr(), h.data_ptr(), _at(initial_state), grad_h.data_ptr(), _at(grad_final_state),
                _at(cu_seqlens), seqs, out["dx"].data_ptr(), out["dg"].data_ptr(), _at(out["dS0"]), B, T, D, code, prep,
                input_gate), _scan_need(B, T, D, seqs, code, False), workspace)
    return out


def kda_scan_backward_ckpt(checkpoint, grad_h, grad_final_state=None, *, cu_seqlens=None,
                           input_gate=KDA_SCAN_INPUT_PLAIN, prep=0, workspace=None, stream=None,
                           want_initial_state_grad=True):
    """kda_scan_backward from the 8-bit checkpoint that kda_scan_fwd filled (same sizes, ``prep``, ``input_gate``
    and ``cu_seqlens``) in place of x, g, h and the initial state."""
    _check_dev("grad_h", grad_h)
    if stream is not None:
        return _scan_on(stream, grad_h.device, kda_scan_backward_ckpt, checkpoint, grad_h, grad_final_state,
                        cu_seqlens=cu_seqlens, input_gate=input_gate, prep=prep, workspace=workspace,
                        want_initial_state_grad=want_initial_state_grad)
    device, code = grad_h.device, _dtype_code(grad_h.dtype)
    B, T, D, seqs = _scan_sizes(grad_h, cu_seqlens)
    state = (seqs or B, D)
    if grad_final_state is not None:
        _same("grad_final_state", grad_final_state, state, torch.float32, device)
    _check_ckpt(checkpoint, grad_h.shape, device)
    out = _scan_grads(grad_h, state, grad_final_state, want_initial_state_grad)
    if workspace is not None:
        _check_scan_workspace(workspace, device)
    _scan_call("kda_scan_backward_ckpt", device,
               (checkpoint.data_ptr(), grad_h.data_ptr(), _at(grad_final_state), _at(cu_seqlens), seqs,
                out["dx"].data_ptr(), out["dg"].data_ptr(), _at(out["dS0"]), B, T, D, code, prep, input_gate),
               _scan_need(B, T, D, seqs, code, False), workspace)
    return out


def kda_scan_step(x, g, state, *, input_gate=KDA_SCAN_INPUT_PLAIN, prep=0, h=None, out_state=None, stream=None):
    """One token of the elementwise recurrence for N sequences: x, g [N,D], state [N,D] fp32, updated in place, or
    left and the new one written to ``out_state``.  Returns h [N,D] in the input dtype."""
    _check_dev("x", x)
    if stream is not None:
        return _scan_on(stream, x.device, kda_scan_step, x, g, state, input_gate=input_gate, prep=prep, h=h,
                        out_state=out_state)
    device, code = x.device, _dtype_code(x.dtype)
    if x.dim() != 2:
        raise ValueError("x must be [N,D]")
    if h is None:
        h = torch.empty_like(x)
    else:
        _same("h", h, x.shape, x.dtype, device)
    _same("g", g, x.shape, x.dtype, device)
    _same("state", state, x.shape, torch.float32, device)
    if out_state is None:
        out_state = state
    else:
        _same("out_state", out_state, x.shape, torch.float32, device)
    _scan_call("kda_scan_step", device,
               (x.data_ptr(), g.data_ptr(), state.data_ptr(), out_state.data_ptr(), h.data_ptr(), x.shape[0], x.shape[1],
                code, prep, input_gate))
    return h
