"""Python binding of libspecverify (batched speculative-decoding verification
on MI355X).

Argument marshalling only: every step of verification runs in the HIP kernels
of ``libspecverify.so``; this module checks tensor shapes/dtypes/devices,
allocates outputs and workspace with PyTorch, and passes raw device pointers
and the current HIP stream through the C ABI declared in
``include/spec_verify.h``.  There is no CPU fallback: if the library is not
built, or no GPU is visible, calls raise.

Entry points (same names as the C ABI):

* ``spec_verify_sample(target, draft, draft_tokens, u_accept, u_sample, T)``
* ``spec_verify_greedy(target, draft_tokens)``
* ``spec_verify_tree(target, node_tokens, parents)``
* ``spec_verify_greedy_lmhead``, ``spec_verify_tree_lmhead`` and
  ``spec_verify_sample_lmhead``: the same from the target's hidden states and
  LM head (logits formed on the matrix cores, never written)
* ``spec_commit_tree_kv``, ``spec_ngram_candidates``, ``sv_read_probe``
* over a paged cache (``PagedKV``): ``spec_append_kv_paged`` (norms, rotation
  and cache write of a window), ``spec_attend_paged`` (its attention),
  ``spec_commit_tree_kv_paged``
* ``spec_token_logprobs`` (log probabilities, entropy, alternatives)
* for prompts: ``spec_append_kv_packed`` and ``spec_attend_packed`` (cache write and
  causal attention of packed sequences), ``spec_rms_norm`` (norm with the residual's
  addition, to bf16 or e4m3) and ``spec_linear_e4m3`` (product of e4m3 operands with
  block scales)
"""

from __future__ import annotations

import ctypes
import functools
import os

HERE = os.path.dirname(os.path.abspath(__file__))
# SPECVERIFY_LIB names another build of the library to load (the sanitizer
# build of the host code, for instance); by default the in-tree one.
LIB_PATH = os.environ.get("SPECVERIFY_LIB") or os.path.join(HERE, "libspecverify.so")

SV_OK, SV_ERR_INVALID_ARG, SV_ERR_UNSUPPORTED, SV_ERR_WORKSPACE, SV_ERR_HIP, SV_ERR_SCRATCH = range(6)
SV_NOALLOC_SCRATCH_BYTES = 8 << 20
SV_F32, SV_BF16, SV_E4M3 = 0, 1, 2
SV_MAX_TREE_NODES = 2048
SV_MAX_WINDOW = 64
SV_MAX_TOP = 32
SV_MAX_NORM_COLS = 16384
SV_MAX_LINEAR_K = 131072
SV_MAX_AXES = 4
SCALE_BLOCK = 128
KERNELS = ("rowstats", "accept", "resid_mass", "resid_select", "argmax", "match", "tree",
           "skip_stats", "skip_argmax", "commit", "lmhead", "ngram_count", "ngram_emit",
           "skip_tree", "read_probe", "lmhead_stats", "lmhead_rows", "merge_parts",
           "append_paged", "attend", "attend_join", "commit_paged", "logprob", "logprob_merge",
           "rms_norm", "linear", "linear_join", "append_packed", "attend_packed", "attend_packed_join")

EXPORTS = ("sv_sample_workspace_bytes", "sv_greedy_workspace_bytes", "spec_verify_sample",
           "spec_verify_greedy", "spec_verify_tree", "spec_commit_tree_kv", "sv_status_string",
           "sv_version", "sv_lmhead_workspace_bytes", "spec_verify_greedy_lmhead",
           "spec_verify_tree_lmhead", "sv_ngram_workspace_bytes", "spec_ngram_candidates",
           "sv_read_probe", "sv_read_probe_folds", "sv_trace_begin", "sv_trace_end", "sv_kernel_name",
           "sv_sample_lmhead_workspace_bytes", "spec_verify_sample_lmhead", "spec_verify_sample_noalloc",
           "spec_append_kv_paged", "sv_attend_workspace_bytes", "spec_attend_paged", "spec_commit_tree_kv_paged",
           "sv_token_logprobs_workspace_bytes", "spec_token_logprobs", "spec_rms_norm", "sv_linear_workspace_bytes",
           "spec_linear_e4m3", "spec_append_kv_packed", "sv_attend_packed_workspace_bytes", "spec_attend_packed")


class SpecVerifyError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


class KernelTime(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("ms", ctypes.c_float)]


class _PagedKVStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("dt", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("page_size", ctypes.c_int), ("head_dim", ctypes.c_int)]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libspecverify.so and declare its signatures (no GPU needed)."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run __graft_entry__.build() first")
    lib = ctypes.CDLL(path)
    P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.sv_sample_workspace_bytes.argtypes = [I, I, I, I]
    lib.sv_sample_workspace_bytes.restype = Z
    lib.sv_greedy_workspace_bytes.argtypes = [I, I, I, I]
    lib.sv_greedy_workspace_bytes.restype = Z
    lib.spec_verify_sample.argtypes = [P, P, P, P, P, I, I, I, I, ctypes.c_float, P, P, P, P, P, P, Z, P]
    lib.spec_verify_sample.restype = I
    lib.spec_verify_sample_noalloc.argtypes = [P, P, P, P, P, I, I, I, I, ctypes.c_float, P, P, P, P, P, P]
    lib.spec_verify_sample_noalloc.restype = I
    lib.spec_verify_greedy.argtypes = [P, P, I, I, I, I, P, P, P, P, Z, P]
    lib.spec_verify_greedy.restype = I
    lib.spec_verify_tree.argtypes = [P, P, P, I, I, I, I, P, P, P, P, P, Z, P]
    lib.spec_verify_tree.restype = I
    lib.spec_commit_tree_kv.argtypes = [P, P, I, I, I, I, P, P, P, P, I, P, P]
    lib.spec_commit_tree_kv.restype = I
    lib.sv_ngram_workspace_bytes.argtypes = [I, I]
    lib.sv_ngram_workspace_bytes.restype = Z
    lib.spec_ngram_candidates.argtypes = [P, I, I, P, P, I, I, P, P, P, P, Z, P]
    lib.spec_ngram_candidates.restype = I
    lib.sv_lmhead_workspace_bytes.argtypes = [I, I]
    lib.sv_lmhead_workspace_bytes.restype = Z
    lib.spec_verify_greedy_lmhead.argtypes = [P, P, P, I, I, I, I, P, P, P, P, Z, P]
    lib.spec_verify_greedy_lmhead.restype = I
    lib.spec_verify_tree_lmhead.argtypes = [P, P, P, P, I, I, I, I, P, P, P, P, P, Z, P]
    lib.spec_verify_tree_lmhead.restype = I
    lib.sv_sample_lmhead_workspace_bytes.argtypes = [I, I, I, I, I]
    lib.sv_sample_lmhead_workspace_bytes.restype = Z
    lib.spec_verify_sample_lmhead.argtypes = [P, P, P, P, P, P, I, I, I, I, I, ctypes.c_float, P, P, P, P,
                                              P, P, Z, P]
    lib.spec_verify_sample_lmhead.restype = I
    L, F, KV = ctypes.c_longlong, ctypes.c_float, _PagedKVStruct
    lib.spec_append_kv_paged.argtypes = [P, P, P, L, L, L, P, P, F, P, I, I, I, P, P, P, I, I, I, KV, P, I, P, P, P]
    lib.spec_append_kv_paged.restype = I
    lib.sv_attend_workspace_bytes.argtypes = [I, I, I, I, I, I, I]
    lib.sv_attend_workspace_bytes.restype = Z
    lib.spec_attend_paged.argtypes = [P, L, KV, P, I, P, P, P, I, I, I, F, P, P, P, P, Z, P]
    lib.spec_attend_paged.restype = I
    lib.spec_commit_tree_kv_paged.argtypes = [P, P, I, I, I, I, I, P, I, I, P, P, P, P, I, P, P]
    lib.spec_commit_tree_kv_paged.restype = I
    lib.sv_token_logprobs_workspace_bytes.argtypes = [I, I, I, I]
    lib.sv_token_logprobs_workspace_bytes.restype = Z
    lib.spec_token_logprobs.argtypes = [P, P, I, I, I, F, I, P, P, P, P, P, P, Z, P]
    lib.spec_token_logprobs.restype = I
    lib.spec_rms_norm.argtypes = [P, L, P, P, F, I, I, P, P, I, P, P]
    lib.spec_rms_norm.restype = I
    lib.sv_linear_workspace_bytes.argtypes = [I, I, I, I]
    lib.sv_linear_workspace_bytes.restype = Z
    lib.spec_linear_e4m3.argtypes = [P, L, P, L, P, P, I, I, I, P, I, P, Z, P]
    lib.spec_linear_e4m3.restype = I
    lib.spec_append_kv_packed.argtypes = [P, P, P, L, L, L, P, P, F, P, I, I, I, P, I, P, P, P, I, I, I, KV, P, I, P, P, P]
    lib.spec_append_kv_packed.restype = I
    lib.sv_attend_packed_workspace_bytes.argtypes = [I, I, I, I, I, I, I, I]
    lib.sv_attend_packed_workspace_bytes.restype = Z
    lib.spec_attend_packed.argtypes = [P, L, KV, P, I, P, P, I, I, I, F, P, P, P, P, Z, P]
    lib.spec_attend_packed.restype = I
    lib.sv_read_probe.argtypes = [P, Z, P, P]
    lib.sv_read_probe.restype = I
    lib.sv_read_probe_folds.argtypes = [Z]
    lib.sv_read_probe_folds.restype = Z
    lib.sv_status_string.argtypes = [I]
    lib.sv_status_string.restype = ctypes.c_char_p
    lib.sv_version.argtypes = []
    lib.sv_version.restype = ctypes.c_char_p
    lib.sv_trace_begin.argtypes = [I, ctypes.c_uint]
    lib.sv_trace_begin.restype = I
    lib.sv_trace_end.argtypes = [ctypes.POINTER(KernelTime), I]
    lib.sv_trace_end.restype = I
    lib.sv_kernel_name.argtypes = [I]
    lib.sv_kernel_name.restype = ctypes.c_char_p
    if path == LIB_PATH:
        _lib = lib
    return lib


def status_string(status: int) -> str:
    try:
        return load_library().sv_status_string(status).decode()
    except RuntimeError:
        return "unknown"


def version() -> str:
    return load_library().sv_version().decode()


# ---- helpers -------------------------------------------------------------------

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch

        if not torch.cuda.is_available():
            raise RuntimeError("specverify needs a ROCm GPU; none is visible")
        _torch_module = torch
    return _torch_module


def _dtype_code(t) -> int:
    import torch

    if t.dtype == torch.bfloat16:
        return SV_BF16
    if t.dtype == torch.float32:
        return SV_F32
    raise TypeError(f"logits must be bfloat16 or float32, got {t.dtype}")


def _check(t, name, ndim=None, dtype=None, device=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got shape {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(torch, device, stream):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _call(torch, fn, device, stream, *args):
    """fn(*args, stream) with `device` current.  A call on the current device's
    current stream, the usual one, takes neither a device guard nor a stream
    object (4 us of a call's 16)."""
    if device.index == torch.cuda.current_device():
        if stream is None:
            return fn(*args, torch._C._cuda_getCurrentRawStream(device.index))
        return fn(*args, stream.cuda_stream)
    with torch.cuda.device(device):
        return fn(*args, _stream(torch, device, stream))


def _hold(torch, device, stream, *tensors):
    """The kernels of a call made with ``stream=`` run on that stream, while
    this binding allocates the workspace and outputs on the current one.  When
    the two differ, mark those blocks as in use on ``stream`` so the caching
    allocator hands none of them to another allocation before the call's
    kernels are done with it."""
    if stream is None or stream.cuda_stream == torch.cuda.current_stream(device).cuda_stream:
        return
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _workspace(torch, nbytes, device, workspace):
    if workspace is None:
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    _check(workspace, "workspace", device=device)
    if workspace.numel() * workspace.element_size() < nbytes:
        raise SpecVerifyError(SV_ERR_WORKSPACE, "workspace")
    return workspace


# ---- entry points ----------------------------------------------------------------

def sample_workspace_bytes(B, K, V, dtype_code) -> int:
    return int(load_library().sv_sample_workspace_bytes(B, K, V, dtype_code))


def greedy_workspace_bytes(B, rows_per_req, V, dtype_code) -> int:
    return int(load_library().sv_greedy_workspace_bytes(B, rows_per_req, V, dtype_code))


def spec_verify_sample(target, draft, draft_tokens, u_accept, u_sample, temperature, *,
                       lse=True, status=True, workspace=None, stream=None):
    """Stochastic chain verification.

    target [B,K+1,V] and draft [B,K,V] logits (bf16 or f32, same dtype),
    draft_tokens [B,K] int32, u_accept [B,K] and u_sample [B,K+1] float32 in
    [0,1).  Returns a dict with ``accept_len`` [B], ``tokens`` [B,K+1] and,
    when requested, ``lse_target`` [B,K+1], ``lse_draft`` [B,K], ``status`` [B].
    With lse=False (and K <= 31) the library skips the rows of positions after
    a request's first rejection (same outputs, fewer bytes).
    """
    torch = _torch()
    lib = load_library()
    _check(target, "target", 3)
    dev = target.device
    B, K1, V = target.shape
    K = K1 - 1
    dt = _dtype_code(target)
    if K > 0:
        _check(draft, "draft", 3, target.dtype, dev)
        if tuple(draft.shape) != (B, K, V):
            raise ValueError(f"draft must be [{B},{K},{V}], got {tuple(draft.shape)}")
        _check(draft_tokens, "draft_tokens", 2, torch.int32, dev)
        _check(u_accept, "u_accept", 2, torch.float32, dev)
        if tuple(draft_tokens.shape) != (B, K) or tuple(u_accept.shape) != (B, K):
            raise ValueError("draft_tokens and u_accept must be [B, K]")
    _check(u_sample, "u_sample", 2, torch.float32, dev)
    if tuple(u_sample.shape) != (B, K + 1):
        raise ValueError("u_sample must be [B, K+1]")
    out = dict(accept_len=torch.empty(B, dtype=torch.int32, device=dev),
               tokens=torch.empty((B, K + 1), dtype=torch.int32, device=dev))
    if lse:
        out["lse_target"] = torch.empty((B, K + 1), dtype=torch.float32, device=dev)
        out["lse_draft"] = torch.empty((B, K), dtype=torch.float32, device=dev)
    if status:
        out["status"] = torch.empty(B, dtype=torch.int32, device=dev)
    nbytes = lib.sv_sample_workspace_bytes(B, K, V, dt)
    ws = _workspace(torch, nbytes, dev, workspace)
    with torch.cuda.device(dev):
        rc = lib.spec_verify_sample(
            _ptr(target), _ptr(draft if K > 0 else None), _ptr(draft_tokens if K > 0 else None),
            _ptr(u_accept if K > 0 else None), _ptr(u_sample), B, K, V, dt, float(temperature),
            _ptr(out["accept_len"]), _ptr(out["tokens"]), _ptr(out.get("lse_target")),
            _ptr(out.get("lse_draft")), _ptr(out.get("status")), _ptr(ws),
            ws.numel() * ws.element_size(), _stream(torch, dev, stream))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_sample")
    _hold(torch, dev, stream, ws if workspace is None else None, *out.values())
    return out


def spec_verify_sample_noalloc(target, draft, draft_tokens, u_accept, u_sample, temperature, *,
                               lse=True, status=True, out=None, stream=None):
    """spec_verify_sample through the entry point that allocates nothing: its
    workspace is the library's static scratch of the current device (calls
    that overlap on one device race on it).  ``out`` may hold preallocated
    outputs (the dict spec_verify_sample returns); the binding allocates any
    that are missing.  Returns that dict."""
    torch = _torch()
    lib = load_library()
    _check(target, "target", 3)
    dev = target.device
    B, K1, V = target.shape
    K = K1 - 1
    dt = _dtype_code(target)
    if K > 0:
        _check(draft, "draft", 3, target.dtype, dev)
        if tuple(draft.shape) != (B, K, V):
            raise ValueError(f"draft must be [{B},{K},{V}], got {tuple(draft.shape)}")
        _check(draft_tokens, "draft_tokens", 2, torch.int32, dev)
        _check(u_accept, "u_accept", 2, torch.float32, dev)
        if tuple(draft_tokens.shape) != (B, K) or tuple(u_accept.shape) != (B, K):
            raise ValueError("draft_tokens and u_accept must be [B, K]")
    _check(u_sample, "u_sample", 2, torch.float32, dev)
    if tuple(u_sample.shape) != (B, K + 1):
        raise ValueError("u_sample must be [B, K+1]")
    out = dict(out or {})
    shapes = {"accept_len": ((B,), torch.int32), "tokens": ((B, K + 1), torch.int32)}
    if lse:
        shapes.update(lse_target=((B, K + 1), torch.float32), lse_draft=((B, K), torch.float32))
    if status:
        shapes["status"] = ((B,), torch.int32)
    for name, (shape, dtype) in shapes.items():
        if name in out:
            _check(out[name], name, len(shape), dtype, dev)
            if tuple(out[name].shape) != shape:
                raise ValueError(f"{name} must be {list(shape)}")
        else:
            out[name] = torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.device(dev):
        rc = lib.spec_verify_sample_noalloc(
            _ptr(target), _ptr(draft if K > 0 else None), _ptr(draft_tokens if K > 0 else None),
            _ptr(u_accept if K > 0 else None), _ptr(u_sample), B, K, V, dt, float(temperature),
            _ptr(out["accept_len"]), _ptr(out["tokens"]), _ptr(out.get("lse_target") if lse else None),
            _ptr(out.get("lse_draft") if lse else None), _ptr(out.get("status") if status else None),
            _stream(torch, dev, stream))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_sample_noalloc")
    _hold(torch, dev, stream, *out.values())
    return out


def spec_verify_greedy(target, draft_tokens, *, status=True, workspace=None, stream=None):
    """Greedy chain verification: target [B,K+1,V], draft_tokens [B,K] int32.
    Returns ``accept_len`` [B], ``tokens`` [B,K+1] and ``status`` [B]."""
    torch = _torch()
    lib = load_library()
    _check(target, "target", 3)
    dev = target.device
    B, K1, V = target.shape
    K = K1 - 1
    dt = _dtype_code(target)
    if K > 0:
        _check(draft_tokens, "draft_tokens", 2, torch.int32, dev)
        if tuple(draft_tokens.shape) != (B, K):
            raise ValueError("draft_tokens must be [B, K]")
    out = dict(accept_len=torch.empty(B, dtype=torch.int32, device=dev),
               tokens=torch.empty((B, K + 1), dtype=torch.int32, device=dev))
    if status:
        out["status"] = torch.empty(B, dtype=torch.int32, device=dev)
    ws = _workspace(torch, lib.sv_greedy_workspace_bytes(B, K + 1, V, dt), dev, workspace)
    with torch.cuda.device(dev):
        rc = lib.spec_verify_greedy(
            _ptr(target), _ptr(draft_tokens if K > 0 else None), B, K, V, dt,
            _ptr(out["accept_len"]), _ptr(out["tokens"]), _ptr(out.get("status")), _ptr(ws),
            ws.numel() * ws.element_size(), _stream(torch, dev, stream))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_greedy")
    _hold(torch, dev, stream, ws if workspace is None else None, *out.values())
    return out


def spec_verify_tree(target, node_tokens, parents, *, status=True, workspace=None, stream=None):
    """Greedy tree verification: target [B,N,V], node_tokens [B,N] and
    parents [B,N] int32.  Returns ``accept_len`` [B], ``path`` [B,N],
    ``tokens`` [B,N] and ``status`` [B]."""
    torch = _torch()
    lib = load_library()
    _check(target, "target", 3)
    dev = target.device
    B, N, V = target.shape
    dt = _dtype_code(target)
    _check(node_tokens, "node_tokens", 2, torch.int32, dev)
    _check(parents, "parents", 2, torch.int32, dev)
    if tuple(node_tokens.shape) != (B, N) or tuple(parents.shape) != (B, N):
        raise ValueError("node_tokens and parents must be [B, N]")
    out = dict(accept_len=torch.empty(B, dtype=torch.int32, device=dev),
               path=torch.empty((B, N), dtype=torch.int32, device=dev),
               tokens=torch.empty((B, N), dtype=torch.int32, device=dev))
    if status:
        out["status"] = torch.empty(B, dtype=torch.int32, device=dev)
    ws = _workspace(torch, lib.sv_greedy_workspace_bytes(B, N, V, dt), dev, workspace)
    with torch.cuda.device(dev):
        rc = lib.spec_verify_tree(
            _ptr(target), _ptr(node_tokens), _ptr(parents), B, N, V, dt, _ptr(out["accept_len"]),
            _ptr(out["path"]), _ptr(out["tokens"]), _ptr(out.get("status")), _ptr(ws),
            ws.numel() * ws.element_size(), _stream(torch, dev, stream))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_tree")
    _hold(torch, dev, stream, ws if workspace is None else None, *out.values())
    return out


def _lmhead_operands(torch, hidden, lm_head, lead):
    _check(hidden, "hidden", len(lead) + 1, torch.bfloat16)
    dev = hidden.device
    _check(lm_head, "lm_head", 2, torch.bfloat16, dev)
    D = hidden.shape[-1]
    V = lm_head.shape[0]
    if lm_head.shape[1] != D:
        raise ValueError(f"lm_head must be [V, {D}], got {tuple(lm_head.shape)}")
    return dev, D, V


def spec_verify_greedy_lmhead(hidden, lm_head, draft_tokens, *, status=True, workspace=None,
                              stream=None):
    """Greedy chain verification on the logits hidden @ lm_head.T, which are
    never materialised: hidden [B, K+1, D] bf16, lm_head [V, D] bf16,
    draft_tokens [B, K] int32.  Returns ``accept_len`` [B], ``tokens`` [B, K+1]
    and ``status`` [B]."""
    torch = _torch()
    lib = load_library()
    dev, D, V = _lmhead_operands(torch, hidden, lm_head, (0, 0))
    B, R = hidden.shape[:2]
    K = R - 1
    _check(draft_tokens, "draft_tokens", 2, torch.int32, dev)
    if tuple(draft_tokens.shape) != (B, K):
        raise ValueError(f"draft_tokens must be [{B}, {K}]")
    out = dict(accept_len=torch.empty(B, dtype=torch.int32, device=dev),
               tokens=torch.empty((B, K + 1), dtype=torch.int32, device=dev))
    if status:
        out["status"] = torch.empty(B, dtype=torch.int32, device=dev)
    ws = _workspace(torch, lib.sv_lmhead_workspace_bytes(B * R, V), dev, workspace)
    with torch.cuda.device(dev):
        rc = lib.spec_verify_greedy_lmhead(
            _ptr(hidden), _ptr(lm_head), _ptr(draft_tokens) if K else None, B, K, D, V,
            _ptr(out["accept_len"]), _ptr(out["tokens"]), _ptr(out.get("status")), _ptr(ws),
            ws.numel() * ws.element_size(), _stream(torch, dev, stream))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_greedy_lmhead")
    _hold(torch, dev, stream, ws if workspace is None else None, *out.values())
    return out


def spec_verify_tree_lmhead(hidden, lm_head, node_tokens, parents, *, status=True, workspace=None,
                            stream=None):
    """Greedy tree verification on the logits hidden @ lm_head.T (never
    materialised): hidden [B, N, D] bf16, lm_head [V, D] bf16, node_tokens and
    parents [B, N] int32.  Returns ``accept_len``, ``path``, ``tokens``, ``status``."""
    torch = _torch()
    lib = load_library()
    dev, D, V = _lmhead_operands(torch, hidden, lm_head, (0, 0))
    B, N = hidden.shape[:2]
    _check(node_tokens, "node_tokens", 2, torch.int32, dev)
    _check(parents, "parents", 2, torch.int32, dev)
    if tuple(node_tokens.shape) != (B, N) or tuple(parents.shape) != (B, N):
        raise ValueError("node_tokens and parents must be [B, N]")
    out = dict(accept_len=torch.empty(B, dtype=torch.int32, device=dev),
               path=torch.empty((B, N), dtype=torch.int32, device=dev),
               tokens=torch.empty((B, N), dtype=torch.int32, device=dev))
    if status:
        out["status"] = torch.empty(B, dtype=torch.int32, device=dev)
    ws = _workspace(torch, lib.sv_lmhead_workspace_bytes(B * N, V), dev, workspace)
    with torch.cuda.device(dev):
        rc = lib.spec_verify_tree_lmhead(
            _ptr(hidden), _ptr(lm_head), _ptr(node_tokens), _ptr(parents), B, N, D, V,
            _ptr(out["accept_len"]), _ptr(out["path"]), _ptr(out["tokens"]), _ptr(out.get("status")),
            _ptr(ws), ws.numel() * ws.element_size(), _stream(torch, dev, stream))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_tree_lmhead")
    _hold(torch, dev, stream, ws if workspace is None else None, *out.values())
    return out


def spec_verify_sample_lmhead(hidden, lm_head, draft, draft_tokens, u_accept, u_sample, temperature, *,
                              lse=True, status=True, workspace=None, stream=None):
    """Stochastic chain verification on the target logits hidden @ lm_head.T,
    never materialised: hidden [B, K+1, D] bf16, lm_head [V, D] bf16, draft
    [B, K, V] logits (bf16 or f32), draft_tokens [B, K] int32, u_accept [B, K]
    and u_sample [B, K+1] float32.  Returns what spec_verify_sample returns."""
    torch = _torch()
    lib = load_library()
    dev, D, V = _lmhead_operands(torch, hidden, lm_head, (0, 0))
    B, R = hidden.shape[:2]
    K = R - 1
    dt = SV_BF16
    if K > 0:
        _check(draft, "draft", 3, device=dev)
        dt = _dtype_code(draft)
        if tuple(draft.shape) != (B, K, V):
            raise ValueError(f"draft must be [{B},{K},{V}], got {tuple(draft.shape)}")
        _check(draft_tokens, "draft_tokens", 2, torch.int32, dev)
        _check(u_accept, "u_accept", 2, torch.float32, dev)
        if tuple(draft_tokens.shape) != (B, K) or tuple(u_accept.shape) != (B, K):
            raise ValueError("draft_tokens and u_accept must be [B, K]")
    _check(u_sample, "u_sample", 2, torch.float32, dev)
    if tuple(u_sample.shape) != (B, K + 1):
        raise ValueError("u_sample must be [B, K+1]")
    out = dict(accept_len=torch.empty(B, dtype=torch.int32, device=dev),
               tokens=torch.empty((B, K + 1), dtype=torch.int32, device=dev))
    if lse:
        out["lse_target"] = torch.empty((B, K + 1), dtype=torch.float32, device=dev)
        out["lse_draft"] = torch.empty((B, K), dtype=torch.float32, device=dev)
    if status:
        out["status"] = torch.empty(B, dtype=torch.int32, device=dev)
    ws = _workspace(torch, lib.sv_sample_lmhead_workspace_bytes(B, K, D, V, dt), dev, workspace)
    with torch.cuda.device(dev):
        rc = lib.spec_verify_sample_lmhead(
            _ptr(hidden), _ptr(lm_head), _ptr(draft if K > 0 else None),
            _ptr(draft_tokens if K > 0 else None), _ptr(u_accept if K > 0 else None), _ptr(u_sample),
            B, K, D, V, dt, float(temperature), _ptr(out["accept_len"]), _ptr(out["tokens"]),
            _ptr(out.get("lse_target")), _ptr(out.get("lse_draft")), _ptr(out.get("status")), _ptr(ws),
            ws.numel() * ws.element_size(), _stream(torch, dev, stream))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_sample_lmhead")
    _hold(torch, dev, stream, ws if workspace is None else None, *out.values())
    return out


def spec_ngram_candidates(context, lengths, queries, cap, *, status=True, workspace=None, stream=None):
    """AdaPLD lexical retrieval: context [B, L], lengths [B], queries [B, n]
    (int32 GPU tensors).  Returns ``count`` [B], ``positions`` [B, cap]
    (ascending, -1 padded) and ``status`` [B]."""
    torch = _torch()
    lib = load_library()
    _check(context, "context", 2, torch.int32)
    dev = context.device
    B, L = context.shape
    _check(lengths, "lengths", 1, torch.int32, dev)
    _check(queries, "queries", 2, torch.int32, dev)
    if lengths.shape[0] != B or queries.shape[0] != B:
        raise ValueError("lengths and queries must have B rows")
    n = queries.shape[1]
    out = dict(count=torch.empty(B, dtype=torch.int32, device=dev),
               positions=torch.empty((B, cap), dtype=torch.int32, device=dev))
    if status:
        out["status"] = torch.empty(B, dtype=torch.int32, device=dev)
    ws = _workspace(torch, lib.sv_ngram_workspace_bytes(B, L), dev, workspace)
    with torch.cuda.device(dev):
        rc = lib.spec_ngram_candidates(_ptr(context), B, L, _ptr(lengths), _ptr(queries), n, cap,
                                       _ptr(out["count"]), _ptr(out["positions"]) if cap else None,
                                       _ptr(out.get("status")), _ptr(ws), ws.numel() * ws.element_size(),
                                       _stream(torch, dev, stream))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_ngram_candidates")
    _hold(torch, dev, stream, ws if workspace is None else None, *out.values())
    return out


def spec_commit_tree_kv(kv, tree_base, commit_base, accept_len, path, *, out=None, status=True,
                        stream=None):
    """Move the KV rows of each request's accepted tree path into consecutive
    slots.  kv: [G, B, S, ...] GPU tensor (any dtype; the trailing dimensions
    of one slot form a row of a multiple of 16 bytes); tree_base, commit_base,
    accept_len [B] and path [B, N] int32 (accept_len and path as returned by
    spec_verify_tree).  In place when ``out`` is None, else into ``out`` (same
    shape and dtype as kv).  Returns the per-request status [B] (or None)."""
    torch = _torch()
    lib = load_library()
    if kv is None or kv.dim() < 3:
        raise ValueError("kv must be [G, B, S, ...]")
    _check(kv, "kv")
    dev = kv.device
    G, B, S = kv.shape[:3]
    row_bytes = kv[0, 0, 0].numel() * kv.element_size() if kv.numel() else 0
    dst = kv if out is None else out
    if out is not None:
        _check(out, "out", kv.dim(), kv.dtype, dev)
        if tuple(out.shape) != tuple(kv.shape):
            raise ValueError("out must have the shape of kv")
    for name, t in (("tree_base", tree_base), ("commit_base", commit_base), ("accept_len", accept_len)):
        _check(t, name, 1, torch.int32, dev)
        if t.shape[0] != B:
            raise ValueError(f"{name} must be [B]")
    _check(path, "path", 2, torch.int32, dev)
    if path.shape[0] != B:
        raise ValueError("path must be [B, N]")
    N = path.shape[1]
    st = torch.empty(B, dtype=torch.int32, device=dev) if status else None
    with torch.cuda.device(dev):
        rc = lib.spec_commit_tree_kv(_ptr(kv), _ptr(dst), G, B, S, row_bytes, _ptr(tree_base),
                                     _ptr(commit_base), _ptr(accept_len), _ptr(path), N, _ptr(st),
                                     _stream(torch, dev, stream))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_commit_tree_kv")
    _hold(torch, dev, stream, st)
    return st


# ---- paged cache -----------------------------------------------------------------

class PagedKV:
    """One layer's paged KV cache: the arrays a program keeps, checked once.

    k_pages and v_pages [num_pages, kv_heads, page_size, head_dim], contiguous, bfloat16
    or float8_e4m3fn; the latter with k_scales and v_scales [num_pages, kv_heads,
    page_size] float32.  page_size a power of two in [16, 1024], head_dim 64, 128
    or 256.  The arrays may be slices of one allocation (``kv[layer, 0]``).  A PagedKV
    is fixed once made, and its arrays must keep their storage (no ``resize_``, no
    ``set_``): other arrays take another PagedKV."""

    def __init__(self, k_pages, v_pages, k_scales=None, v_scales=None):
        import torch

        _check(k_pages, "k_pages", 4)
        _check(v_pages, "v_pages", 4, k_pages.dtype, k_pages.device)
        if tuple(v_pages.shape) != tuple(k_pages.shape):
            raise ValueError("v_pages must have the shape of k_pages")
        if k_pages.dtype == torch.bfloat16:
            dt = SV_BF16
            if k_scales is not None or v_scales is not None:
                raise ValueError("a bfloat16 cache has no scales")
        elif k_pages.dtype == torch.float8_e4m3fn:
            dt = SV_E4M3
            for name, s in (("k_scales", k_scales), ("v_scales", v_scales)):
                _check(s, name, 3, torch.float32, k_pages.device)
                if tuple(s.shape) != tuple(k_pages.shape[:3]):
                    raise ValueError(f"{name} must be {list(k_pages.shape[:3])}")
        else:
            raise TypeError(f"pages must be bfloat16 or float8_e4m3fn, got {k_pages.dtype}")
        self.k_pages, self.v_pages, self.k_scales, self.v_scales = k_pages, v_pages, k_scales, v_scales
        self.device = k_pages.device
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = k_pages.shape
        self._c = _PagedKVStruct(k_pages.data_ptr(), v_pages.data_ptr(),
                                 None if k_scales is None else k_scales.data_ptr(),
                                 None if v_scales is None else v_scales.data_ptr(), dt, self.num_pages,
                                 self.kv_heads, self.page_size, self.head_dim)

    def __setattr__(self, name, value):
        # an array put in another's place would leave calls at the old one's address
        if "_c" in self.__dict__:
            raise AttributeError(f"PagedKV.{name} is fixed; make another PagedKV")
        super().__setattr__(name, value)


def _window_rows(torch, t, name, heads, head_dim, dev, lead=None):
    """[B, N, heads, head_dim] bf16 whose heads are consecutive and whose tokens are
    equally far apart (a slice of a projection's output); returns that distance."""
    if t is None or t.dim() != 4:
        raise ValueError(f"{name} must be [B, N, heads, head_dim]")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    B, N, H, D = t.shape
    if D != head_dim or (heads is not None and H != heads) or (lead is not None and (B, N) != lead):
        raise ValueError(f"{name} has shape {tuple(t.shape)}")
    sb, sn, sh, sd = t.stride()
    if (D > 1 and sd != 1) or (H > 1 and sh != D):
        raise ValueError(f"{name}: the heads of a token must be consecutive")
    if N == 1:
        return sb if B > 1 else H * D
    if B > 1 and sb != N * sn:
        raise ValueError(f"{name}: tokens must be equally far apart")
    return sn


def _window_ints(torch, t, name, shape, dev):
    if t is None:
        return
    _check(t, name, len(shape), torch.int32, dev)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")


def _window_out(torch, t, name, shape, dtype, dev):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _check(t, name, len(shape), dtype, dev)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    return t


def spec_append_kv_paged(q, k, v, cache, page_table, base, positions=None, *, q_weight=None, k_weight=None,
                         eps=1e-6, rope=None, interleaved=False, counts=None, q_out=None, status=True,
                         stream=None):
    """Write a window's keys and values into ``cache`` (a PagedKV), with the
    per-head norms (q_weight, k_weight [head_dim] bf16) and the rotation (rope
    [max_pos, rot] float32: rot/2 cosines, rot/2 sines; positions [B, N] int32) of
    queries and keys in the same pass.

    q [B, N, H, head_dim], k and v [B, N, kv_heads, head_dim] bf16, each a
    contiguous tensor or a slice of a projection's output; page_table [B, P],
    base [B] (cached tokens before the window), counts [B] (rows in use) int32.
    Returns ``q`` [B, N, H, head_dim] bf16 (``q_out`` if given; rows behind counts
    are left as they were) and ``status`` [B, N]."""
    torch = _torch()
    lib = load_library()
    dev, D = cache.device, cache.head_dim
    qs = _window_rows(torch, q, "q", None, D, dev)
    B, N, H, _ = q.shape
    ks = _window_rows(torch, k, "k", cache.kv_heads, D, dev, (B, N))
    vs = _window_rows(torch, v, "v", cache.kv_heads, D, dev, (B, N))
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _check(w, name, 1, torch.bfloat16, dev)
            if w.shape[0] != D:
                raise ValueError(f"{name} must be [{D}]")
    rot = max_pos = 0
    if rope is not None:
        _check(rope, "rope", 2, torch.float32, dev)
        max_pos, rot = rope.shape
        if positions is None:
            raise ValueError("positions is required with rope")
    _window_ints(torch, positions, "positions", (B, N), dev)
    _check(page_table, "page_table", 2, torch.int32, dev)
    if page_table.shape[0] != B:
        raise ValueError("page_table must be [B, P]")
    _check(base, "base", 1, torch.int32, dev)
    _window_ints(torch, base, "base", (B,), dev)
    _window_ints(torch, counts, "counts", (B,), dev)
    out = dict(q=_window_out(torch, q_out, "q_out", (B, N, H, D), torch.bfloat16, dev))
    if status:
        out["status"] = torch.empty((B, N), dtype=torch.int32, device=dev)
    rc = _call(
        torch, lib.spec_append_kv_paged, dev, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs,
        _ptr(q_weight), _ptr(k_weight), float(eps), _ptr(rope), rot, max_pos, int(bool(interleaved)),
        _ptr(positions), base.data_ptr(), _ptr(counts), B, N, H, cache._c, page_table.data_ptr(),
        page_table.shape[1], out["q"].data_ptr(),
        _ptr(out.get("status")))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_append_kv_paged")
    _hold(torch, dev, stream, *out.values())
    return out


@functools.lru_cache(maxsize=4096)
def attend_workspace_bytes(B, N, H, kv_heads, head_dim, P, page_size) -> int:
    return int(load_library().sv_attend_workspace_bytes(B, N, H, kv_heads, head_dim, P, page_size))


def spec_attend_paged(q, cache, page_table, base, *, parents=None, counts=None, scale=None, out=None,
                      lse=False, status=True, workspace=None, stream=None):
    """Attention of a window's rows over ``cache`` (a PagedKV that already holds
    the window's own keys and values): one new token, a draft chain, or with
    ``parents`` [B, N] int32 a draft tree.

    q [B, N, H, head_dim] bf16, N <= 64; page_table [B, P], base [B], counts [B]
    int32; scale defaults to head_dim ** -0.5.  Returns ``out`` [B, N, H,
    head_dim] bf16, ``lse`` [B, N, H] float32 (lse=True, or a tensor to write)
    and ``status`` [B].  Rows behind counts are left as they were in ``out`` and
    ``lse``."""
    torch = _torch()
    lib = load_library()
    dev, D = cache.device, cache.head_dim
    qs = _window_rows(torch, q, "q", None, D, dev)
    B, N, H, _ = q.shape
    _check(page_table, "page_table", 2, torch.int32, dev)
    if page_table.shape[0] != B:
        raise ValueError("page_table must be [B, P]")
    P = page_table.shape[1]
    _check(base, "base", 1, torch.int32, dev)
    _window_ints(torch, base, "base", (B,), dev)
    _window_ints(torch, counts, "counts", (B,), dev)
    _window_ints(torch, parents, "parents", (B, N), dev)
    res = dict(out=_window_out(torch, out, "out", (B, N, H, D), torch.bfloat16, dev))
    if lse is not False and lse is not None:
        res["lse"] = _window_out(torch, None if lse is True else lse, "lse", (B, N, H), torch.float32, dev)
    if status:
        res["status"] = torch.empty(B, dtype=torch.int32, device=dev)
    ws = _workspace(torch, attend_workspace_bytes(B, N, H, cache.kv_heads, D, P, cache.page_size), dev, workspace)
    rc = _call(
        torch, lib.spec_attend_paged, dev, stream, q.data_ptr(), qs, cache._c, page_table.data_ptr(), P,
        base.data_ptr(), _ptr(counts), _ptr(parents), B, N, H, float(D ** -0.5 if scale is None else scale),
        res["out"].data_ptr(), _ptr(res.get("lse")), _ptr(res.get("status")), ws.data_ptr(),
        ws.numel() * ws.element_size())
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_attend_paged")
    _hold(torch, dev, stream, ws if workspace is None else None, *res.values())
    return res


def spec_commit_tree_kv_paged(pages, page_table, tree_base, commit_base, accept_len, path, *, scales=None,
                              status=True, stream=None):
    """spec_commit_tree_kv inside a paged cache, in place: pages [G, num_pages,
    kv_heads, page_size, head_dim] (any dtype; rows of 16 * 2^i bytes up to 1024),
    scales [G, num_pages, kv_heads, page_size] float32 moved with the rows,
    page_table [B, P], tree_base, commit_base, accept_len [B] and path [B, N]
    int32.  Returns the per-request status [B] (or None)."""
    torch = _torch()
    lib = load_library()
    _check(pages, "pages", 5)
    dev = pages.device
    G, num_pages, kv_heads, page_size, D = pages.shape
    if scales is not None:
        _check(scales, "scales", 4, torch.float32, dev)
        if tuple(scales.shape) != tuple(pages.shape[:4]):
            raise ValueError(f"scales must be {list(pages.shape[:4])}")
    _check(page_table, "page_table", 2, torch.int32, dev)
    B, P = page_table.shape
    for name, t in (("tree_base", tree_base), ("commit_base", commit_base), ("accept_len", accept_len)):
        _check(t, name, 1, torch.int32, dev)
        if t.shape[0] != B:
            raise ValueError(f"{name} must be [B]")
    _check(path, "path", 2, torch.int32, dev)
    if path.shape[0] != B:
        raise ValueError("path must be [B, N]")
    st = torch.empty(B, dtype=torch.int32, device=dev) if status else None
    rc = _call(
        torch, lib.spec_commit_tree_kv_paged, dev, stream, pages.data_ptr(), _ptr(scales), G, num_pages, kv_heads,
        page_size, D * pages.element_size(), page_table.data_ptr(), P, B, tree_base.data_ptr(),
        commit_base.data_ptr(), accept_len.data_ptr(), path.data_ptr(), path.shape[1], _ptr(st))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_commit_tree_kv_paged")
    _hold(torch, dev, stream, st)
    return st


@functools.lru_cache(maxsize=4096)
def token_logprobs_workspace_bytes(R, V, dtype_code, top_k) -> int:
    return int(load_library().sv_token_logprobs_workspace_bytes(R, V, dtype_code, top_k))


def spec_token_logprobs(logits, tokens=None, *, temperature=1.0, top_k=0, entropy=True, status=True,
                        workspace=None, stream=None):
    """Log probabilities under softmax(logits / temperature): logits [R, V] (bf16
    or f32, contiguous), tokens [R] int32 (a row whose token is -1 is not read).
    Returns ``logprob`` [R] (with tokens), ``entropy`` [R] in nats, ``top_ids`` and
    ``top_logprobs`` [R, top_k] (top_k <= 32, by falling probability, ties to the
    lowest id) and ``status`` [R].  A row that holds NaN or +inf returns NaN."""
    torch = _torch()
    lib = load_library()
    _check(logits, "logits", 2)
    dev = logits.device
    R, V = logits.shape
    dt = _dtype_code(logits)
    _window_ints(torch, tokens, "tokens", (R,), dev)
    out = {}
    if tokens is not None:
        out["logprob"] = torch.empty(R, dtype=torch.float32, device=dev)
    if entropy:
        out["entropy"] = torch.empty(R, dtype=torch.float32, device=dev)
    if top_k:
        out["top_ids"] = torch.empty((R, max(top_k, 0)), dtype=torch.int32, device=dev)
        out["top_logprobs"] = torch.empty((R, max(top_k, 0)), dtype=torch.float32, device=dev)
    if status:
        out["status"] = torch.empty(R, dtype=torch.int32, device=dev)
    ws = _workspace(torch, token_logprobs_workspace_bytes(R, V, dt, top_k), dev, workspace)
    rc = _call(
        torch, lib.spec_token_logprobs, dev, stream, logits.data_ptr(), _ptr(tokens), R, V, dt, float(temperature),
        top_k, _ptr(out.get("logprob")), _ptr(out.get("entropy")), _ptr(out.get("top_ids")),
        _ptr(out.get("top_logprobs")), _ptr(out.get("status")), ws.data_ptr(), ws.numel() * ws.element_size())
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_token_logprobs")
    _hold(torch, dev, stream, ws if workspace is None else None, *out.values())
    return out


# ---- prompts and e4m3 projections --------------------------------------------------

def _matrix(torch, t, name, dtype, dev=None, shape=None):
    """[rows, columns] whose rows are contiguous and equally far apart; returns that
    distance."""
    if t is None or t.dim() != 2:
        raise ValueError(f"{name} must have 2 dimensions")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: rows must be contiguous")
    return t.stride(0) if rows > 1 else cols


def spec_rms_norm(x, weight=None, *, eps=1e-6, residual=None, residual_out=None, e4m3=False, out=None, stream=None):
    """RMS norm of the rows of x [T, D] bf16 (rows contiguous, equally far apart), with
    weight [D] bf16 and the residual's addition: h = x + residual, y = h / sqrt(mean(h^2)
    + eps) * weight.  D a multiple of 8, at most 16384.

    Returns ``out`` [T, D]: y in bf16, or with e4m3=True in float8_e4m3fn beside
    ``scales`` [ceil(D / 128), T] float32, one for each row and 128 columns; and with
    ``residual`` [T, D] bf16, ``residual`` [T, D]: h in bf16 (``residual_out`` if given,
    which may be ``residual`` itself)."""
    torch = _torch()
    lib = load_library()
    xs = _matrix(torch, x, "x", torch.bfloat16)
    dev = x.device
    T, D = x.shape
    if weight is not None:
        _check(weight, "weight", 1, torch.bfloat16, dev)
        if weight.shape[0] != D:
            raise ValueError(f"weight must be [{D}]")
    res = {}
    if residual is not None:
        _check(residual, "residual", 2, torch.bfloat16, dev)
        if residual.shape != (T, D):
            raise ValueError(f"residual must be [{T}, {D}]")
        res["residual"] = (residual.new_empty((T, D)) if residual_out is None else
                           _window_out(torch, residual_out, "residual_out", (T, D), torch.bfloat16, dev))
    elif residual_out is not None:
        raise ValueError("residual_out needs residual")
    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    res["out"] = x.new_empty((T, D), dtype=dt) if out is None else _window_out(torch, out, "out", (T, D), dt, dev)
    if e4m3:
        res["scales"] = x.new_empty((-(-D // SCALE_BLOCK), T), dtype=torch.float32)
    rc = _call(torch, lib.spec_rms_norm, dev, stream, x.data_ptr(), xs, _ptr(residual), _ptr(weight), float(eps), T, D,
               _ptr(res.get("residual")), res["out"].data_ptr(), SV_E4M3 if e4m3 else SV_BF16, _ptr(res.get("scales")))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_rms_norm")
    _hold(torch, dev, stream, *res.values())
    return res


@functools.lru_cache(maxsize=4096)
def linear_workspace_bytes(M, N, K, dtype_code) -> int:
    return int(load_library().sv_linear_workspace_bytes(M, N, K, dtype_code))


def spec_linear_e4m3(x, x_scales, w, w_scales, *, out=None, out_dtype=None, workspace=None, stream=None):
    """x @ w.T of e4m3 operands with a scale for each block of 128: x [M, K]
    float8_e4m3fn (rows contiguous, equally far apart) with x_scales [ceil(K / 128), M]
    float32 (as spec_rms_norm returns them; a slice of columns will do), w [N, K]
    float8_e4m3fn with w_scales [ceil(N / 128), ceil(K / 128)] float32.  K a multiple of
    16.  Returns [M, N] in out_dtype (bfloat16 or float32; bfloat16 by default), or
    ``out``.

    float32 outputs are summed in fp32.  For bfloat16 ones a block's products go through
    the e4m3 matrix instruction, whose sum is within 2^-10 of the sum of its terms'
    magnitudes (an operand below 2^-6 counting as that): small products beside large ones
    that cancel can be lost."""
    torch = _torch()
    lib = load_library()
    e4m3 = torch.float8_e4m3fn
    xs = _matrix(torch, x, "x", e4m3)
    dev = x.device
    M, K = x.shape
    _check(w, "w", 2, e4m3, dev)
    N, blocks = w.shape[0], -(-K // SCALE_BLOCK)
    if w.shape[1] != K:
        raise ValueError(f"w must be [N, {K}], got {list(w.shape)}")
    ss = _matrix(torch, x_scales, "x_scales", torch.float32, dev, (blocks, M))
    _check(w_scales, "w_scales", 2, torch.float32, dev)
    if w_scales.shape != (-(-N // SCALE_BLOCK), blocks):
        raise ValueError(f"w_scales must be [{-(-N // SCALE_BLOCK)}, {blocks}]")
    if out is not None:
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = torch.bfloat16
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"out must be bfloat16 or float32, got {out_dtype}")
    out = x.new_empty((M, N), dtype=out_dtype) if out is None else _window_out(torch, out, "out", (M, N), out_dtype, dev)
    dt = SV_F32 if out_dtype == torch.float32 else SV_BF16
    ws = _workspace(torch, linear_workspace_bytes(M, N, K, dt), dev, workspace)
    rc = _call(torch, lib.spec_linear_e4m3, dev, stream, x.data_ptr(), xs, x_scales.data_ptr(), ss, w.data_ptr(),
               w_scales.data_ptr(), M, N, K, out.data_ptr(), dt,
               ws.data_ptr(), ws.numel() * ws.element_size())
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_linear_e4m3")
    _hold(torch, dev, stream, ws if workspace is None else None, out)
    return out


def _packed_rows(torch, t, name, heads, head_dim, dev, tokens=None):
    """[T, heads, head_dim] bf16 whose heads are consecutive; returns the distance of
    its tokens."""
    if t is None or t.dim() != 3:
        raise ValueError(f"{name} must be [T, heads, head_dim]")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    T, H, D = t.shape
    if D != head_dim or (heads is not None and H != heads) or (tokens is not None and T != tokens):
        raise ValueError(f"{name} has shape {tuple(t.shape)}")
    st, sh, sd = t.stride()
    if (D > 1 and sd != 1) or (H > 1 and sh != D):
        raise ValueError(f"{name}: the heads of a token must be consecutive")
    return st if T > 1 else H * D


def _packed_bounds(torch, page_table, starts, base, dev):
    _check(page_table, "page_table", 2, torch.int32, dev)
    B, P = page_table.shape
    _window_ints(torch, starts, "starts", (B + 1,), dev)
    if starts is None:
        raise ValueError("starts is required")
    _window_ints(torch, base, "base", (B,), dev)
    return B, P


def spec_append_kv_packed(q, k, v, cache, page_table, starts, base=None, positions=None, *, q_weight=None,
                          k_weight=None, eps=1e-6, rope=None, interleaved=False, pair_axis=None, q_out=None,
                          status=True, stream=None):
    """spec_append_kv_paged for packed sequences: q [T, H, head_dim], k and v [T,
    kv_heads, head_dim] bf16 (slices of a projection's output), the tokens of request b
    being starts[b] ... starts[b + 1] - 1 (starts [B + 1] int32, rising), behind base[b]
    cached ones (base [B] int32; None: none).

    positions [T] or [axes, T] int32 (axes <= 4); pair_axis [rot / 2] int32 names the
    axis whose position turns each pair of a head.  Returns ``q`` [T, H, head_dim] bf16
    (``q_out`` if given; tokens outside every request are left as they were) and
    ``status`` [T]."""
    torch = _torch()
    lib = load_library()
    dev, D = cache.device, cache.head_dim
    qs = _packed_rows(torch, q, "q", None, D, dev)
    T, H, _ = q.shape
    ks = _packed_rows(torch, k, "k", cache.kv_heads, D, dev, T)
    vs = _packed_rows(torch, v, "v", cache.kv_heads, D, dev, T)
    B, P = _packed_bounds(torch, page_table, starts, base, dev)
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _check(w, name, 1, torch.bfloat16, dev)
            if w.shape[0] != D:
                raise ValueError(f"{name} must be [{D}]")
    rot = max_pos = 0
    axes = 1
    if rope is not None:
        _check(rope, "rope", 2, torch.float32, dev)
        max_pos, rot = rope.shape
        if positions is None:
            raise ValueError("positions is required with rope")
        axes = positions.shape[0] if positions.dim() == 2 else 1
        _window_ints(torch, positions, "positions", (axes, T) if positions.dim() == 2 else (T,), dev)
        if axes > 1 and pair_axis is None:
            raise ValueError("pair_axis is required with positions of several axes")
        _window_ints(torch, pair_axis, "pair_axis", (rot // 2,), dev)
    res = dict(q=_window_out(torch, q_out, "q_out", (T, H, D), torch.bfloat16, dev))
    if status:
        res["status"] = torch.empty(T, dtype=torch.int32, device=dev)
    rc = _call(
        torch, lib.spec_append_kv_packed, dev, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs,
        _ptr(q_weight), _ptr(k_weight), float(eps), _ptr(rope), rot, max_pos, int(bool(interleaved)),
        _ptr(positions if rope is not None else None), axes, _ptr(pair_axis if rope is not None else None),
        starts.data_ptr(), _ptr(base), T, B, H, cache._c, page_table.data_ptr(), P, res["q"].data_ptr(),
        _ptr(res.get("status")))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_append_kv_packed")
    _hold(torch, dev, stream, *res.values())
    return res


@functools.lru_cache(maxsize=4096)
def attend_packed_workspace_bytes(T, B, H, kv_heads, head_dim, P, page_size, dtype_code) -> int:
    return int(load_library().sv_attend_packed_workspace_bytes(T, B, H, kv_heads, head_dim, P, page_size, dtype_code))


def spec_attend_packed(q, cache, page_table, starts, base=None, *, scale=None, out=None, lse=False, status=True,
                       workspace=None, stream=None):
    """Causal attention of packed sequences over ``cache`` (a PagedKV that already holds
    their keys and values): q [T, H, head_dim] bf16, the tokens of request b being
    starts[b] ... starts[b + 1] - 1 (starts [B + 1] int32), behind base[b] cached ones
    (base [B] int32; None: none).  Token starts[b] + j sees the slots below base[b] + j
    + 1; scale defaults to head_dim ** -0.5.

    Returns ``out`` [T, H, head_dim] bf16, ``lse`` [T, H] float32 (lse=True, or a tensor
    to write) and ``status`` [B].  Rows of tokens outside every request are left as they
    were in ``out`` and ``lse``."""
    torch = _torch()
    lib = load_library()
    dev, D = cache.device, cache.head_dim
    qs = _packed_rows(torch, q, "q", None, D, dev)
    T, H, _ = q.shape
    B, P = _packed_bounds(torch, page_table, starts, base, dev)
    res = dict(out=_window_out(torch, out, "out", (T, H, D), torch.bfloat16, dev))
    if lse is not False and lse is not None:
        res["lse"] = _window_out(torch, None if lse is True else lse, "lse", (T, H), torch.float32, dev)
    if status:
        res["status"] = torch.empty(B, dtype=torch.int32, device=dev)
    ws = _workspace(torch, attend_packed_workspace_bytes(T, B, H, cache.kv_heads, D, P, cache.page_size, cache._c.dt), dev,
                    workspace)
    rc = _call(
        torch, lib.spec_attend_packed, dev, stream, q.data_ptr(), qs, cache._c, page_table.data_ptr(), P,
        starts.data_ptr(), _ptr(base), T, B, H, float(D ** -0.5 if scale is None else scale), res["out"].data_ptr(),
        _ptr(res.get("lse")), _ptr(res.get("status")), ws.data_ptr(), ws.numel() * ws.element_size())
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_attend_packed")
    _hold(torch, dev, stream, ws if workspace is None else None, *res.values())
    return res


def sv_read_probe(buf, *, folds=None, stream=None):
    """Read every byte of the GPU tensor ``buf`` once (a measurement aid: the
    read rate this device reaches).  Returns ``folds`` (int32), entry i the XOR
    of the 32-bit words of the buffer's i-th 16 KB."""
    torch = _torch()
    lib = load_library()
    _check(buf, "buf")
    dev = buf.device
    nbytes = buf.numel() * buf.element_size()
    nf = lib.sv_read_probe_folds(nbytes)
    if folds is None:
        folds = torch.empty(max(nf, 1), dtype=torch.int32, device=dev)
    elif folds.numel() < nf or folds.dtype != torch.int32 or folds.device != dev:
        raise ValueError(f"folds must be int32 on {dev} with at least {nf} entries")
    with torch.cuda.device(dev):
        rc = lib.sv_read_probe(_ptr(buf), nbytes, _ptr(folds), _stream(torch, dev, stream))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "sv_read_probe")
    _hold(torch, dev, stream, folds)
    return folds


# ---- per-kernel timing -----------------------------------------------------------

def trace_begin(capacity: int = 4096, kernels=None) -> None:
    """Time every launch (kernels=None) or only the named kernels."""
    mask = 0
    for k in kernels or ():
        mask |= 1 << KERNELS.index(k)
    rc = load_library().sv_trace_begin(capacity, mask)
    if rc != SV_OK:
        raise SpecVerifyError(rc, "sv_trace_begin")


def trace_end(max_records: int = 1 << 16):
    """Stop tracing; return [(kernel_name, ms), ...] in launch order."""
    lib = load_library()
    recs = (KernelTime * max_records)()
    n = lib.sv_trace_end(recs, max_records)
    return [(lib.sv_kernel_name(recs[i].kernel).decode(), float(recs[i].ms))
            for i in range(min(n, max_records))]
