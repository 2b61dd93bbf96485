"""drafter_sampling_gb300: VocabTrim drafting and speculative verification on
one GB300 GPU (sm_103a).

Thin Python binding over libvt.so (include/vt.h).  Each function below has
the name of the C entry point it calls and only marshals arguments: it checks
tensor devices, dtypes and shapes, allocates outputs and workspace with
PyTorch, and passes raw device pointers and the current CUDA stream.  Every
step of the computation runs in the library's CUDA kernels.

bf16 tensors may be passed as torch.bfloat16 or as int16/uint16 bit patterns.
"""
from __future__ import annotations

import functools

from . import _lib
from ._lib import (VT_BF16, VT_DEV_BAD_DRAFT, VT_DEV_BAD_ID,  # noqa: F401
                   VT_DEV_DUPLICATE_ID, VT_DEV_NONFINITE, VT_DEV_TIMEOUT,
                   VT_DEV_ZERO_RESIDUAL, VT_F32,
                   VtError)

__all__ = ["vt_selftest_wait", "vt_calibrate_topk", "vt_calibrate_top_p", "vt_calibrate_min_count", "vt_trim_head",
           "vt_draft_logits", "vt_draft_step", "vt_draft_topk", "vt_verify", "vt_verify_tree",
           "vt_quantize_head", "vt_draft_logits_fp8", "vt_draft_step_fp8", "vt_draft_topk_fp8",
           "vt_token_logprobs",
           "vt_beam_select", "vt_beam_reorder",
           "vt_distill_loss", "vt_distill_grad", "vt_distill_loss_grad",
           "BlockGraph",
           "workspace_bytes",
           "VtError", "lib"]


def lib():
    """The loaded ctypes library (raises if libvt.so is not built)."""
    return _lib.load()


_TORCH = None
_RAW_STREAM = None  # torch's raw current-stream getter, or False where it has none
_BF16 = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _stream_ptr(stream):
    """The cudaStream_t of `stream`, or of the current device's current
    stream (read without building a torch.cuda.Stream object, which costs a
    few microseconds of host time per call)."""
    global _RAW_STREAM
    torch = _torch()
    if stream is not None:
        return stream.cuda_stream
    if _RAW_STREAM is None:
        _RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", False)
    if _RAW_STREAM:
        return _RAW_STREAM(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _dev(t, name, dtypes, dim=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got {t.dim()}")
    return t


def _bf16_dtypes():
    global _BF16
    if _BF16 is None:
        torch = _torch()
        _BF16 = (torch.bfloat16, torch.int16, torch.uint16)
    return _BF16


def _as_stream(stream, device):
    """`stream` as a torch stream, where it is another object that has the raw one."""
    torch = _torch()
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(stream.cuda_stream, device=device)


def _empty(shape, dtype, device, stream, returned=True):
    """A tensor for a call that runs on `stream`.  Its memory comes from that
    stream's own pool: from the current stream's, it could be a block whose last
    owner's kernels, still running there, write it meanwhile.  Where it is
    returned, the current stream may read it, so its memory is not given to
    another before that stream has passed the point where it is freed."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_as_stream(stream, device)):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _ws(nbytes, device, stream=None):
    return _empty(max(int(nbytes), 256), _torch().uint8, device, stream, returned=False)


def workspace_bytes(kind: str, **kw) -> int:
    L = lib()
    if kind == "calibrate":
        return L.vt_calibrate_topk_workspace_bytes(kw["n"], kw["V"], kw["K"])
    if kind == "select":
        return L.vt_calibrate_select_workspace_bytes(kw["n"], kw["V"])
    if kind == "trim":
        return L.vt_trim_head_workspace_bytes(kw["V"], kw["K"])
    if kind == "draft":
        return L.vt_draft_workspace_bytes(kw["B"], kw["H"], kw["K"])
    if kind == "draft_fp8":
        return L.vt_draft_fp8_workspace_bytes(kw["B"], kw["H"], kw["K"])
    if kind == "draft_topk_fp8":
        return L.vt_draft_topk_fp8_workspace_bytes(kw["B"], kw["H"], kw["K"], kw["k"])
    if kind == "verify":
        return L.vt_verify_workspace_bytes(kw["B"], kw["gamma"], kw["V"], kw["K"])
    if kind == "beam_select":
        return L.vt_beam_select_workspace_bytes(kw["B"], kw["W"], kw["K"], kw["n"])
    raise ValueError(kind)


def vt_calibrate_topk(ids, V: int, K: int, counts=None, topk_ids=None, dev_status=None,
                      workspace=None, stream=None):
    """Token histogram and Top-K (count desc, id asc) of int32 ids.

    Returns (counts uint32-as-int32 [V], topk_ids int32 [K], dev_status int32 [1]).
    """
    torch = _torch()
    _dev(ids, "ids", (torch.int32,), 1)
    dev = ids.device
    n = ids.numel()
    if counts is None:
        counts = _empty(V, torch.int32, dev, stream)
    if topk_ids is None:
        topk_ids = _empty(K, torch.int32, dev, stream)
    if dev_status is None:
        dev_status = _empty(1, torch.int32, dev, stream)
    _dev(counts, "counts", (torch.int32, torch.uint32), 1)
    _dev(topk_ids, "topk_ids", (torch.int32,), 1)
    if counts.numel() != V or topk_ids.numel() != K:
        raise ValueError("counts must have V elements and topk_ids K elements")
    L = lib()
    if workspace is None:
        workspace = _ws(L.vt_calibrate_topk_workspace_bytes(n, V, K), dev, stream)
    st = L.vt_calibrate_topk(ids.data_ptr(), n, V, K, counts.data_ptr(), topk_ids.data_ptr(),
                             dev_status.data_ptr(), workspace.data_ptr(), workspace.numel(),
                             _stream_ptr(stream))
    _lib.check("vt_calibrate_topk", st)
    return counts, topk_ids, dev_status


def _calibrate_select(fn: str, ids, V: int, param, counts, ranked_ids, k_out, dev_status,
                      workspace, stream):
    torch = _torch()
    _dev(ids, "ids", (torch.int32,), 1)
    dev = ids.device
    n = ids.numel()
    if counts is None:
        counts = _empty(V, torch.int32, dev, stream)
    if ranked_ids is None:
        ranked_ids = _empty(V, torch.int32, dev, stream)
    if k_out is None:
        k_out = _empty(1, torch.int32, dev, stream)
    if dev_status is None:
        dev_status = _empty(1, torch.int32, dev, stream)
    _dev(counts, "counts", (torch.int32, torch.uint32), 1)
    _dev(ranked_ids, "ranked_ids", (torch.int32,), 1)
    if counts.numel() != V or ranked_ids.numel() != V:
        raise ValueError("counts and ranked_ids must have V elements")
    L = lib()
    if workspace is None:
        workspace = _ws(L.vt_calibrate_select_workspace_bytes(n, V), dev, stream)
    st = getattr(L, fn)(ids.data_ptr(), n, V, param, counts.data_ptr(), ranked_ids.data_ptr(),
                        k_out.data_ptr(), dev_status.data_ptr(), workspace.data_ptr(),
                        workspace.numel(), _stream_ptr(stream))
    _lib.check(fn, st)
    return counts, ranked_ids, k_out, dev_status


def vt_calibrate_top_p(ids, V: int, P: float, counts=None, ranked_ids=None, k_out=None,
                       dev_status=None, workspace=None, stream=None):
    """Token histogram, full ranking, and K = the smallest ranked prefix whose
    counts reach P of the calibration tokens.  Returns (counts [V], ranked_ids
    [V], k_out int32 [1] on the device, dev_status [1])."""
    return _calibrate_select("vt_calibrate_top_p", ids, V, float(P), counts, ranked_ids, k_out,
                             dev_status, workspace, stream)


def vt_calibrate_min_count(ids, V: int, min_count: int, counts=None, ranked_ids=None, k_out=None,
                           dev_status=None, workspace=None, stream=None):
    """Token histogram, full ranking, and K = the number of ids counted at
    least min_count times.  Returns (counts, ranked_ids, k_out, dev_status)."""
    return _calibrate_select("vt_calibrate_min_count", ids, V, int(min_count), counts,
                             ranked_ids, k_out, dev_status, workspace, stream)


def vt_trim_head(W, topk_ids, W_trim=None, trim_ids=None, inv_map=None, dev_status=None,
                 workspace=None, stream=None):
    """W_trim = W[sorted(topk_ids)], trim_ids (ascending) and inv_map.

    Returns (W_trim [K,H] same dtype as W, trim_ids int32 [K], inv_map int32 [V], dev_status).
    """
    torch = _torch()
    _dev(W, "W", _bf16_dtypes(), 2)
    _dev(topk_ids, "topk_ids", (torch.int32,), 1)
    V, H = W.shape
    K = topk_ids.numel()
    dev = W.device
    if W_trim is None:
        W_trim = _empty((K, H), W.dtype, dev, stream)
    if trim_ids is None:
        trim_ids = _empty(K, torch.int32, dev, stream)
    if inv_map is None:
        inv_map = _empty(V, torch.int32, dev, stream)
    if dev_status is None:
        dev_status = _empty(1, torch.int32, dev, stream)
    _dev(W_trim, "W_trim", _bf16_dtypes(), 2)
    if tuple(W_trim.shape) != (K, H) or trim_ids.numel() != K or inv_map.numel() != V:
        raise ValueError("output shapes do not match (K, H), K and V")
    L = lib()
    if workspace is None:
        workspace = _ws(L.vt_trim_head_workspace_bytes(V, K), dev, stream)
    st = L.vt_trim_head(W.data_ptr(), V, H, topk_ids.data_ptr(), K, W_trim.data_ptr(),
                        trim_ids.data_ptr(), inv_map.data_ptr(), dev_status.data_ptr(),
                        workspace.data_ptr(), workspace.numel(), _stream_ptr(stream))
    _lib.check("vt_trim_head", st)
    return W_trim, trim_ids, inv_map, dev_status


def vt_draft_logits(hidden, W_trim, temperature: float = 1.0, logits=None, workspace=None,
                    stream=None):
    """logits [B, K] fp32 = hidden @ W_trim^T / T."""
    torch = _torch()
    _dev(hidden, "hidden", _bf16_dtypes(), 2)
    _dev(W_trim, "W_trim", _bf16_dtypes(), 2)
    B, H = hidden.shape
    K, H2 = W_trim.shape
    if H2 != H:
        raise ValueError("hidden and W_trim disagree on H")
    if logits is None:
        logits = _empty((B, K), torch.float32, hidden.device, stream)
    if logits.dim() != 2 or logits.shape[0] != B or logits.stride(1) != 1 or logits.shape[1] < K:
        raise ValueError("logits must be [B, >=K] with unit inner stride")
    L = lib()
    if workspace is None:
        workspace = _ws(L.vt_draft_workspace_bytes(B, H, K), hidden.device, stream)
    st = L.vt_draft_logits(hidden.data_ptr(), B, H, W_trim.data_ptr(), K, float(temperature),
                           logits.data_ptr(), logits.stride(0), workspace.data_ptr(),
                           workspace.numel(), _stream_ptr(stream))
    _lib.check("vt_draft_logits", st)
    return logits


def vt_draft_step(hidden, W_trim, trim_ids, uniforms, temperature: float = 1.0, q=None,
                  tokens=None, dev_status=None, workspace=None, stream=None):
    """One drafting step; returns (q [B, K] view, tokens int32 [B] view, dev_status).

    ``q`` may be a strided view such as q_all[:, pos, :] of a contiguous
    [B, gamma, K] tensor (unit inner stride), and ``tokens`` a strided view
    such as tok_all[:, pos] of a [B, gamma] tensor.  temperature == 0 drafts
    greedily (q one-hot); ``uniforms`` may then be None.
    """
    torch = _torch()
    greedy = float(temperature) == 0.0
    _dev(hidden, "hidden", _bf16_dtypes(), 2)
    _dev(W_trim, "W_trim", _bf16_dtypes(), 2)
    _dev(trim_ids, "trim_ids", (torch.int32,), 1)
    if uniforms is not None or not greedy:
        _dev(uniforms, "uniforms", (torch.float32,), 1)
    B, H = hidden.shape
    K = W_trim.shape[0]
    dev = hidden.device
    if q is None:
        q = _empty((B, K), torch.float32, dev, stream)
    if q.dim() != 2 or q.shape[0] != B or q.shape[1] != K or q.stride(1) != 1:
        raise ValueError("q must be [B, K] with unit inner stride")
    if tokens is None:
        tokens = _empty(B, torch.int32, dev, stream)
    if tokens.dim() != 1 or tokens.shape[0] != B or tokens.dtype != torch.int32:
        raise ValueError("tokens must be an int32 vector of B entries (any stride)")
    if dev_status is None:
        dev_status = _empty(1, torch.int32, dev, stream)
    if (uniforms is not None and uniforms.numel() != B) or trim_ids.numel() != K:
        raise ValueError("uniforms must have B and trim_ids K elements")
    L = lib()
    if workspace is None:
        workspace = _ws(L.vt_draft_workspace_bytes(B, H, K), dev, stream)
    st = L.vt_draft_step(hidden.data_ptr(), B, H, W_trim.data_ptr(), trim_ids.data_ptr(), K,
                         uniforms.data_ptr() if uniforms is not None else None,
                         float(temperature), q.data_ptr(), q.stride(0),
                         tokens.data_ptr(), tokens.stride(0), dev_status.data_ptr(),
                         workspace.data_ptr(), workspace.numel(), _stream_ptr(stream))
    _lib.check("vt_draft_step", st)
    return q, tokens, dev_status


def vt_verify(target_logits, q, inv_map, draft_tokens, u_accept, u_resample,
              temperature: float = 1.0, out_tokens=None, out_num_accepted=None,
              out_accept_prob=None, dev_status=None, workspace=None, stream=None,
              want_accept_prob: bool = True):
    """Modified rejection sampling over a batch of drafted blocks.

    target_logits [B, gamma+1, V] float32 or bf16; q [B, gamma, K] float32.
    temperature == 0 verifies greedily (a drafted token is kept iff it is the
    target's highest logit); q, inv_map and the uniforms may then be None.
    Returns (out_tokens [B, gamma+1], out_num_accepted [B], out_accept_prob
    [B, gamma] or None, dev_status [1]).
    """
    torch = _torch()
    if target_logits.dtype == torch.float32:
        dt = VT_F32
    elif target_logits.dtype in _bf16_dtypes():
        dt = VT_BF16
    else:
        raise TypeError("target_logits must be float32 or bf16")
    greedy = float(temperature) == 0.0
    _dev(target_logits, "target_logits", (target_logits.dtype,), 3)
    _dev(draft_tokens, "draft_tokens", (torch.int32,), 2)
    B, R, V = target_logits.shape
    gamma = R - 1
    if tuple(draft_tokens.shape) != (B, gamma):
        raise ValueError("draft_tokens shape does not match target_logits")
    # the sampling rule needs all four; the greedy one reads none (any given
    # one is still checked)
    if not greedy or q is not None:
        _dev(q, "q", (torch.float32,), 3)
        if tuple(q.shape[:2]) != (B, gamma):
            raise ValueError("q shape does not match target_logits")
    if not greedy or inv_map is not None:
        _dev(inv_map, "inv_map", (torch.int32,), 1)
        if inv_map.numel() != V:
            raise ValueError("inv_map must have V entries")
    if not greedy or u_accept is not None:
        _dev(u_accept, "u_accept", (torch.float32,), 2)
        if tuple(u_accept.shape) != (B, gamma):
            raise ValueError("u_accept must be [B, gamma]")
    if not greedy or u_resample is not None:
        _dev(u_resample, "u_resample", (torch.float32,), 2)
        if tuple(u_resample.shape) != (B, R):
            raise ValueError("u_resample must be [B, gamma+1]")
    K = q.shape[2] if q is not None else 1
    ptr = lambda x: x.data_ptr() if x is not None else None
    dev = target_logits.device
    if out_tokens is None:
        out_tokens = _empty((B, R), torch.int32, dev, stream)
    if out_num_accepted is None:
        out_num_accepted = _empty(B, torch.int32, dev, stream)
    if out_accept_prob is None and want_accept_prob:
        out_accept_prob = _empty((B, gamma), torch.float32, dev, stream)
    if dev_status is None:
        dev_status = _empty(1, torch.int32, dev, stream)
    L = lib()
    if workspace is None:
        workspace = _ws(L.vt_verify_workspace_bytes(B, gamma, V, K), dev, stream)
    st = L.vt_verify(target_logits.data_ptr(), dt, B, gamma, V, ptr(q), ptr(inv_map),
                     K, draft_tokens.data_ptr(), ptr(u_accept), ptr(u_resample),
                     float(temperature), out_tokens.data_ptr(), out_num_accepted.data_ptr(),
                     out_accept_prob.data_ptr() if out_accept_prob is not None else None,
                     dev_status.data_ptr(), workspace.data_ptr(), workspace.numel(),
                     _stream_ptr(stream))
    _lib.check("vt_verify", st)
    return out_tokens, out_num_accepted, out_accept_prob, dev_status


def vt_draft_topk(hidden, W_trim, trim_ids, k: int, temperature: float = 1.0, out_ids=None,
                  out_logq=None, dev_status=None, workspace=None, stream=None):
    """The drafter's k best trimmed candidates per row (target ids, best
    first) with log q.  Returns (out_ids int32 [B, k], out_logq [B, k],
    dev_status [1])."""
    torch = _torch()
    _dev(hidden, "hidden", _bf16_dtypes(), 2)
    _dev(W_trim, "W_trim", _bf16_dtypes(), 2)
    _dev(trim_ids, "trim_ids", (torch.int32,), 1)
    B, H = hidden.shape
    K = W_trim.shape[0]
    dev = hidden.device
    if out_ids is None:
        out_ids = _empty((B, k), torch.int32, dev, stream)
    if out_logq is None:
        out_logq = _empty((B, k), torch.float32, dev, stream)
    if dev_status is None:
        dev_status = _empty(1, torch.int32, dev, stream)
    L = lib()
    if workspace is None:
        workspace = _ws(L.vt_draft_topk_workspace_bytes(B, H, K, k), dev, stream)
    st = L.vt_draft_topk(hidden.data_ptr(), B, H, W_trim.data_ptr(), trim_ids.data_ptr(), K, k,
                         float(temperature), out_ids.data_ptr(), out_logq.data_ptr(),
                         dev_status.data_ptr(), workspace.data_ptr(), workspace.numel(),
                         _stream_ptr(stream))
    _lib.check("vt_draft_topk", st)
    return out_ids, out_logq, dev_status


def vt_verify_tree(target_logits, parent, tokens, temperature: float = 0.0, out_tokens=None,
                   out_num_accepted=None, out_path=None, dev_status=None, workspace=None,
                   stream=None, want_path: bool = True):
    """Greedy verification of draft trees: target_logits [B, N+1, V] (row 0
    after the context, row i+1 after node i), parent int32 [B, N] or [N]
    (shared tree; -1 = the context), tokens int32 [B, N].  Returns
    (out_tokens [B, N+1], out_num_accepted [B], out_path [B, N] or None,
    dev_status [1])."""
    torch = _torch()
    if target_logits.dtype == torch.float32:
        dt = VT_F32
    elif target_logits.dtype in _bf16_dtypes():
        dt = VT_BF16
    else:
        raise TypeError("target_logits must be float32 or bf16")
    _dev(target_logits, "target_logits", (target_logits.dtype,), 3)
    _dev(tokens, "tokens", (torch.int32,), 2)
    _dev(parent, "parent", (torch.int32,), None)
    B, R, V = target_logits.shape
    N = R - 1
    if tuple(tokens.shape) != (B, N):
        raise ValueError("tokens must be [B, N] with N + 1 = target_logits.shape[1]")
    if parent.dim() == 1 and parent.numel() == N:
        pstride = 0
    elif parent.dim() == 2 and tuple(parent.shape) == (B, N):
        pstride = N
    else:
        raise ValueError("parent must be [N] or [B, N]")
    dev = target_logits.device
    if out_tokens is None:
        out_tokens = _empty((B, R), torch.int32, dev, stream)
    if out_num_accepted is None:
        out_num_accepted = _empty(B, torch.int32, dev, stream)
    if out_path is None and want_path:
        out_path = _empty((B, N), torch.int32, dev, stream)
    if dev_status is None:
        dev_status = _empty(1, torch.int32, dev, stream)
    L = lib()
    if workspace is None:
        workspace = _ws(L.vt_verify_tree_workspace_bytes(B, N, V), dev, stream)
    st = L.vt_verify_tree(target_logits.data_ptr(), dt, B, N, V, parent.data_ptr(), pstride,
                          tokens.data_ptr(), float(temperature), out_tokens.data_ptr(),
                          out_num_accepted.data_ptr(),
                          out_path.data_ptr() if out_path is not None else None,
                          dev_status.data_ptr(), workspace.data_ptr(), workspace.numel(),
                          _stream_ptr(stream))
    _lib.check("vt_verify_tree", st)
    return out_tokens, out_num_accepted, out_path, dev_status


# Dtype tuples of the arguments below and torch's current-device getter, filled
# at the first call.  These calls take a few microseconds on the GPU, so what
# the binding does per tensor is kept to four attribute reads.
_F32 = _I32 = _FP8 = _U8 = _FLAG = None
_CUR_DEVICE = None
_DEVICES = ()


def _fast():
    global _F32, _I32, _FP8, _U8, _FLAG, _CUR_DEVICE, _DEVICES
    torch = _torch()
    _DEVICES = tuple(torch.device("cuda", i) for i in range(torch.cuda.device_count()))
    _F32, _I32, _U8 = (torch.float32,), (torch.int32,), (torch.uint8,)
    _FLAG = (torch.bool, torch.uint8)
    _CUR_DEVICE = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _bf16_dtypes()
    _FP8 = (torch.float8_e4m3fn, torch.uint8)
    return torch


def _first(t, name):
    """The device index of the leading tensor argument, which has to be the
    current device."""
    torch = _TORCH if _FP8 is not None else _fast()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    cur = _CUR_DEVICE()
    if d != cur:
        raise ValueError(f"{name} is on cuda:{d}, the current device is cuda:{cur}")
    return d


def _arg(t, name, dtypes, shape, dev):
    """A contiguous tensor of the given shape (None: any) on device dev; returns its address."""
    try:
        if (t.get_device() == dev and t.dtype in dtypes and t.is_contiguous() and
                (shape is None or t.shape == shape)):
            return t.data_ptr()
    except AttributeError:
        pass
    _dev(t, name, dtypes)
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on cuda:{dev}")
    raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _new(shape, dtype, dev, stream, returned=True):
    """A tensor on device dev for a call that runs on `stream` (see _empty)."""
    if stream is None:
        return _TORCH.empty(shape, dtype=dtype, device=_DEVICES[dev])
    return _empty(shape, dtype, _DEVICES[dev], stream, returned)


def _on(stream, dev):
    """The raw stream of a call on device dev."""
    if stream is None:
        return _RAW_STREAM(dev) if _RAW_STREAM else _stream_ptr(None)
    if stream.device.index != dev:
        raise ValueError(f"stream is on {stream.device}, the call's tensors on cuda:{dev}")
    return stream.cuda_stream


def _head_fp8(W8, w_scale, dev):
    """(K, H, row stride, addresses) of an e4m3 head and its block scales."""
    if not isinstance(W8, _TORCH.Tensor):
        raise TypeError("W8 must be a torch.Tensor")
    if W8.get_device() != dev:
        raise ValueError(f"W8 must be a CUDA tensor on cuda:{dev}, it is on {W8.device}")
    if W8.dtype not in _FP8:
        raise TypeError(f"W8 has dtype {W8.dtype}, expected one of {_FP8}")
    if W8.dim() != 2 or 0 in W8.shape:
        raise ValueError("W8 must be [K, H]")
    K, H = W8.shape
    ldw, inner = W8.stride()
    if K == 1:
        ldw = (H + 15) // 16 * 16
    ptr = W8.data_ptr()
    if (inner != 1 and H > 1) or ldw < H or ldw % 16 or ptr % 16:
        raise ValueError("W8 must have unit inner stride, a row stride that is a multiple of 16 and "
                         "a 16-byte aligned start")
    return K, H, ldw, ptr, _arg(w_scale, "w_scale", _F32, ((K + 127) // 128, (H + 127) // 128), dev)


def _hidden(hidden, H, dev):
    """(B, address) of hidden states [B, H]."""
    p = _arg(hidden, "hidden", _BF16, None, dev)
    if hidden.dim() != 2:
        raise ValueError("hidden must be [B, H]")
    if hidden.shape[1] != H:
        raise ValueError("hidden and W8 disagree on H")
    return hidden.shape[0], p


def _rows_out(t, name, B, K, dev, wide):
    """(address, row stride) of an fp32 output of B rows and K columns (or
    more, where `wide`), unit inner stride, rows apart."""
    try:
        b, k = t.shape
        ld, inner = t.stride()
        if (t.get_device() == dev and t.dtype in _F32 and b == B and (k == K or (wide and k > K)) and
                (inner == 1 or K == 1) and (ld >= K or B == 1)):
            return t.data_ptr(), ld if B > 1 else k
    except (AttributeError, ValueError):
        pass
    raise ValueError(f"{name} must be a float32 tensor on cuda:{dev}, [{B}, {'>= ' if wide else ''}{K}] "
                     "with unit inner stride")


def _scratch(t, nbytes, dev, stream):
    """(address, bytes) of the workspace given, or of a new one."""
    if t is None:
        t = _new(max(int(nbytes), 256), _U8[0], dev, stream, returned=False)
    p = _arg(t, "workspace", _U8, None, dev)
    return p, t.numel(), t


def vt_quantize_head(W, W8=None, w_scale=None, dev_status=None, stream=None):
    """The head [K, H] (bf16) as e4m3 with one power-of-two scale per block of
    128 x 128.

    Returns (W8 [K, H] float8_e4m3fn, a view whose row stride is a multiple of
    16, w_scale float32 [ceil(K/128), ceil(H/128)], dev_status).
    """
    dev = _first(W, "W")
    wp = _arg(W, "W", _BF16, None, dev)
    if W.dim() != 2 or 0 in W.shape:
        raise ValueError("W must be [K, H]")
    K, H = W.shape
    if W8 is None:
        W8 = _new((K, (H + 15) // 16 * 16), _FP8[0], dev, stream)[:, :H]
    if w_scale is None:
        w_scale = _new(((K + 127) // 128, (H + 127) // 128), _F32[0], dev, stream)
    if dev_status is None:
        dev_status = _new(1, _I32[0], dev, stream)
    K8, H8, ldw, p8, sp = _head_fp8(W8, w_scale, dev)
    if K8 != K or H8 != H:
        raise ValueError("W8 must be [K, H]")
    st = lib().vt_quantize_head(wp, K, H, p8, ldw, sp, _arg(dev_status, "dev_status", _I32, (1,), dev),
                                _on(stream, dev))
    if st:
        _lib.check("vt_quantize_head", st)
    return W8, w_scale, dev_status


def vt_draft_logits_fp8(hidden, W8, w_scale, temperature: float = 1.0, logits=None, workspace=None,
                        stream=None):
    """vt_draft_logits through an e4m3 head (vt_quantize_head); the hidden
    states are quantised inside the call.  w_scale may hold any finite values;
    with 129 to 256 rows (and other even numbers of 128-row chunks), powers of two
    are faster."""
    dev = _first(hidden, "hidden")
    K, H, ldw, p8, sp = _head_fp8(W8, w_scale, dev)
    B, hp = _hidden(hidden, H, dev)
    if logits is None:
        logits = _new((B, K), _F32[0], dev, stream)
    zp, ldz = _rows_out(logits, "logits", B, K, dev, True)
    L = lib()
    ws, n, workspace = _scratch(
        workspace, L.vt_draft_fp8_workspace_bytes(B, H, K) if workspace is None else 0, dev, stream)
    st = L.vt_draft_logits_fp8(hp, B, H, p8, ldw, sp, K, float(temperature), zp, ldz, ws, n,
                               _on(stream, dev))
    if st:
        _lib.check("vt_draft_logits_fp8", st)
    return logits


def vt_draft_step_fp8(hidden, W8, w_scale, trim_ids, uniforms, temperature: float = 1.0, q=None,
                      tokens=None, dev_status=None, workspace=None, stream=None):
    """vt_draft_step through an e4m3 head; returns (q [B, K], tokens int32 [B],
    dev_status).  q and tokens may be strided views as there; temperature == 0
    drafts greedily (uniforms may then be None)."""
    dev = _first(hidden, "hidden")
    K, H, ldw, p8, sp = _head_fp8(W8, w_scale, dev)
    B, hp = _hidden(hidden, H, dev)
    temperature = float(temperature)
    ip = _arg(trim_ids, "trim_ids", _I32, (K,), dev)
    up = None
    if uniforms is not None or temperature != 0.0:
        up = _arg(uniforms, "uniforms", _F32, (B,), dev)
    if q is None:
        q = _new((B, K), _F32[0], dev, stream)
    qp, ldq = _rows_out(q, "q", B, K, dev, False)
    if tokens is None:
        tokens = _new(B, _I32[0], dev, stream)
    if (tokens.get_device() != dev or tokens.dim() != 1 or tokens.shape[0] != B or
            tokens.dtype not in _I32 or (B > 1 and tokens.stride(0) < 1)):
        raise ValueError(f"tokens must be an int32 vector of B entries on cuda:{dev} (any positive stride)")
    if dev_status is None:
        dev_status = _new(1, _I32[0], dev, stream)
    dp = _arg(dev_status, "dev_status", _I32, (1,), dev)
    L = lib()
    ws, n, workspace = _scratch(
        workspace, L.vt_draft_fp8_workspace_bytes(B, H, K) if workspace is None else 0, dev, stream)
    st = L.vt_draft_step_fp8(hp, B, H, p8, ldw, sp, ip, K, up, temperature, qp, ldq, tokens.data_ptr(),
                             tokens.stride(0) if B > 1 else 1, dp, ws, n, _on(stream, dev))
    if st:
        _lib.check("vt_draft_step_fp8", st)
    return q, tokens, dev_status


def vt_draft_topk_fp8(hidden, W8, w_scale, trim_ids, k: int, temperature: float = 1.0, out_ids=None,
                      out_logq=None, dev_status=None, workspace=None, stream=None):
    """vt_draft_topk through an e4m3 head.  Returns (out_ids int32 [B, k],
    out_logq [B, k], dev_status [1])."""
    dev = _first(hidden, "hidden")
    K, H, ldw, p8, sp = _head_fp8(W8, w_scale, dev)
    B, hp = _hidden(hidden, H, dev)
    ip = _arg(trim_ids, "trim_ids", _I32, (K,), dev)
    k = int(k)
    if not 1 <= k <= min(32, K):
        raise ValueError("k must be in [1, min(32, K)]")
    if out_ids is None:
        out_ids = _new((B, k), _I32[0], dev, stream)
    if out_logq is None:
        out_logq = _new((B, k), _F32[0], dev, stream)
    if dev_status is None:
        dev_status = _new(1, _I32[0], dev, stream)
    op = _arg(out_ids, "out_ids", _I32, (B, k), dev)
    lp = _arg(out_logq, "out_logq", _F32, (B, k), dev)
    dp = _arg(dev_status, "dev_status", _I32, (1,), dev)
    L = lib()
    ws, n, workspace = _scratch(
        workspace, L.vt_draft_topk_fp8_workspace_bytes(B, H, K, k) if workspace is None else 0, dev,
        stream)
    st = L.vt_draft_topk_fp8(hp, B, H, p8, ldw, sp, ip, K, k, float(temperature), op, lp, dp, ws, n,
                             _on(stream, dev))
    if st:
        _lib.check("vt_draft_topk_fp8", st)
    return out_ids, out_logq, dev_status


def _logit_rows(logits, name="logits"):
    """(element type, leading shape, rows, row length, row stride) of logits
    [R, V] or [B, R, V]."""
    dt = logits.dtype
    if dt in _F32:
        dt = VT_F32
    elif dt in _BF16:
        dt = VT_BF16
    else:
        raise TypeError(f"{name} must be float32 or bf16")
    full, st = logits.shape, logits.stride()
    if len(full) not in (2, 3) or 0 in full:
        raise ValueError(f"{name} must be [R, V] or [B, R, V]")
    shape, V = full[:-1], full[-1]
    if len(full) == 2:
        R = shape[0]
        ld = st[0] if R > 1 else V
        even = True
    else:
        B, n = shape
        R = B * n
        ld = st[1] if n > 1 else st[0] if B > 1 else V
        even = B == 1 or n == 1 or st[0] == n * ld
    if (st[-1] != 1 and V > 1) or not even or ld < V:
        raise ValueError(f"{name} must have unit inner stride and evenly spaced rows")
    return dt, shape, R, V, ld


def vt_token_logprobs(logits, tokens, k: int = 0, temperature: float = 1.0, out_logp=None,
                      out_entropy=None, out_top_ids=None, out_top_logp=None, dev_status=None,
                      stream=None, want_entropy: bool = True):
    """Log probabilities of given tokens under rows of logits.

    logits [R, V] or [B, R, V], float32 or bf16, unit inner stride and evenly
    spaced rows; tokens int32 of logits' leading shape, contiguous, -1 = row
    not scored.  All tensors are on the current device.
    Returns (logp, entropy or None, top_ids, top_logp, dev_status), logp and
    entropy of tokens' shape, top_ids int32 and top_logp [..., k] (None where
    k == 0): the k best ids, ties to the lower, with their log probabilities.
    """
    dev = _first(logits, "logits")
    dt, shape, R, V, ld = _logit_rows(logits)
    k = int(k)
    if not 0 <= k <= min(32, V):
        raise ValueError("k must be in [0, min(32, V)]")
    tp = _arg(tokens, "tokens", _I32, shape, dev)
    if out_logp is None:
        out_logp = _new(shape, _F32[0], dev, stream)
    lp = _arg(out_logp, "out_logp", _F32, shape, dev)
    ep = ip = pp = None
    if out_entropy is None and want_entropy:
        out_entropy = _new(shape, _F32[0], dev, stream)
    if out_entropy is not None:
        ep = _arg(out_entropy, "out_entropy", _F32, shape, dev)
    if k:
        top = shape + (k,)
        if out_top_ids is None:
            out_top_ids = _new(top, _I32[0], dev, stream)
        if out_top_logp is None:
            out_top_logp = _new(top, _F32[0], dev, stream)
        ip = _arg(out_top_ids, "out_top_ids", _I32, top, dev)
        pp = _arg(out_top_logp, "out_top_logp", _F32, top, dev)
    else:
        out_top_ids = out_top_logp = None
    if dev_status is None:
        dev_status = _new(1, _I32[0], dev, stream)
    dp = _arg(dev_status, "dev_status", _I32, (1,), dev)
    rc = lib().vt_token_logprobs(logits.data_ptr(), dt, R, V, ld, tp, k, float(temperature), lp, ep, ip,
                                 pp, dp, _on(stream, dev))
    if rc:
        _lib.check("vt_token_logprobs", rc)
    return out_logp, out_entropy, out_top_ids, out_top_logp, dev_status


def vt_beam_select(logits, scores, n: int, temperature: float = 1.0, trim_ids=None, done=None,
                   end_id: int = -1, out_scores=None, out_parent=None, out_tokens=None, out_done=None,
                   dev_status=None, workspace=None, stream=None):
    """One step of beam search: the n best continuations of each sequence's beams.

    logits [B, W, K], float32 or bf16, unit inner stride and evenly spaced rows;
    scores float32 [B, W] (-inf: no beam); trim_ids int32 [K] names the indices'
    tokens; done bool or uint8 [B, W] marks beams that have ended with end_id
    (they continue once, as they are).  All tensors are on the current device;
    outputs overlap no input.
    Returns (scores, parent int32, tokens int32, done or None, dev_status), each
    [B, n], best first, ties to the lower beam and index; done where end_id >= 0.
    Missing continuations have score -inf, parent -1 and token -1.  Equal and nearly
    equal beams (within 1e-5) are ordered in 64 bits, for which their rows are read again.
    """
    dev = _first(logits, "logits")
    dt, shape, _, K, ld = _logit_rows(logits)
    if len(shape) != 2:
        raise ValueError("logits must be [B, W, K]")
    B, W = shape
    n, end_id = int(n), int(end_id)
    if not 1 <= n <= 32 or W > 32:
        raise ValueError("n and the number of beams must be in [1, 32]")
    if end_id < -1 or end_id >= 1 << 31:
        raise ValueError("end_id must be a token id, or -1")
    sp = _arg(scores, "scores", _F32, shape, dev)
    tp = gp = op = None
    if trim_ids is not None:
        tp = _arg(trim_ids, "trim_ids", _I32, (K,), dev)
    if (done is not None or out_done is not None) and end_id < 0:
        raise ValueError("done and out_done need end_id")
    if done is not None:
        gp = _arg(done, "done", _FLAG, shape, dev)
    out = (B, n)
    if out_scores is None:
        out_scores = _new(out, _F32[0], dev, stream)
    if out_parent is None:
        out_parent = _new(out, _I32[0], dev, stream)
    if out_tokens is None:
        out_tokens = _new(out, _I32[0], dev, stream)
    if end_id >= 0:
        if out_done is None:
            out_done = _new(out, _FLAG[0], dev, stream)
        op = _arg(out_done, "out_done", _FLAG, out, dev)
    if dev_status is None:
        dev_status = _new(1, _I32[0], dev, stream)
    L = lib()
    ws, nb, workspace = _scratch(
        workspace, L.vt_beam_select_workspace_bytes(B, W, K, n) if workspace is None else 0, dev, stream)
    rc = L.vt_beam_select(logits.data_ptr(), dt, B, W, K, ld, sp, gp, end_id, tp, n, float(temperature),
                          _arg(out_scores, "out_scores", _F32, out, dev),
                          _arg(out_parent, "out_parent", _I32, out, dev),
                          _arg(out_tokens, "out_tokens", _I32, out, dev), op,
                          _arg(dev_status, "dev_status", _I32, (1,), dev), ws, nb, _on(stream, dev))
    if rc:
        _lib.check("vt_beam_select", rc)
    return out_scores, out_parent, out_tokens, out_done, dev_status


def _collapse(shape, strides):
    """(extent, stride) of dimensions that one stride walks through, None where
    none does; extents of 1 fit anywhere."""
    n, st = 1, 0
    for d in range(len(shape) - 1, -1, -1):
        if shape[d] == 1:
            continue
        if n == 1:
            st = strides[d]
        elif strides[d] != st * n:
            return None
        n *= shape[d]
    return n, st


def _tail(shape, st, first):
    """The first dimension, from `first` on, of those at the end that are contiguous."""
    cut = len(shape)
    while cut > first and _collapse(shape[cut - 1:], st[cut - 1:]) in ((_size(shape[cut - 1:]), 1), (1, 0)):
        cut -= 1
    return cut


def _beam_parts(name, shape, st, ost, dim, len_dim):
    """The five extents (outer, B, W, inner, positions), their strides in two tensors
    of this shape (but for W) and these strides, and the row length, in elements, of
    states with their sequences at `dim`."""
    if len_dim is None:  # whole states, in rows as long as both tensors allow
        mid = last = max(_tail(shape, st, dim + 2), _tail(shape, ost, dim + 2))
    else:
        mid, last = len_dim, len_dim + 1
    n = _size(shape[last:])
    steps = []
    for s in (st, ost):
        outer, inner = _collapse(shape[:dim], s[:dim]), _collapse(shape[dim + 2:mid], s[dim + 2:mid])
        row = _collapse(shape[last:], s[last:])
        if outer is None or inner is None or row is None or (n > 1 and row[1] != 1):
            raise ValueError(f"{name} must have contiguous rows, and evenly spaced dimensions before its "
                             "sequences and between its beams and positions")
        steps.append((outer[1], s[dim], s[dim + 1], inner[1], s[len_dim] if len_dim is not None else 0))
    ext = (outer[0], shape[dim], shape[dim + 1], inner[0], shape[len_dim] if len_dim is not None else 1)
    a, b = (tuple(s if e > 1 else 0 for e, s in zip(ext, x)) for x in steps)
    return ext, a, b, n


@functools.lru_cache(maxsize=256)
def _beam_plan(shape, st, oshape, ostr, size, dim, len_dim, n):
    """What vt_beam_reorder passes on of two tensors' layouts (`size` bytes an element): dim
    and the byte strides as the library takes them, extents, bytes of a row and of
    either tensor from its first element to its last."""
    nd = len(shape)
    dim += nd if dim < 0 else 0
    if not 0 <= dim <= nd - 2 or 0 in shape:
        raise ValueError("state must be [..., B, W, ...] with its sequences at dim, and not empty")
    if len_dim is not None:
        len_dim += nd if len_dim < 0 else 0
        if not dim + 2 <= len_dim < nd:
            raise ValueError("len_dim must be a dimension behind the beams")
    if len(oshape) != nd or oshape[:dim + 1] != shape[:dim + 1] or oshape[dim + 2:] != shape[dim + 2:]:
        raise ValueError(f"out must be like state, {list(shape)}, but for its beams, got {list(oshape)}")
    ext, a, b, row = _beam_parts("state", shape, st, ostr, dim, len_dim)
    B, W, slots = ext[1], ext[2], oshape[dim + 1]
    if not 1 <= n <= 32 or W > 32:
        raise ValueError("the slots of parent and the number of beams must be in [1, 32]")
    if n > slots:
        raise ValueError(f"parent has {n} slots, out {slots} beams")
    if W == 1:  # (its slots' stride is out's own)
        b = b[:2] + (ostr[dim + 1] if slots > 1 else 0,) + b[3:]
    if any(s == 0 for s, e in zip(b, (ext[0], B, n, ext[3], ext[4])) if e > 1):
        raise ValueError("out must not be expanded")
    five = _lib._i64 * 5
    span = lambda shape, st: (sum((e - 1) * s for e, s in zip(shape, st)) + 1) * size
    return (B, W, five(*(s * size for s in a)), five(*(s * size for s in b)), ext[0], ext[3], ext[4], row * size,
            span(shape, st), span(oshape, ostr))


def _size(shape):
    n = 1
    for s in shape:
        n *= s
    return n


def vt_beam_reorder(state, parent, out=None, dim: int = 0, lengths=None, len_dim=None, dev_status=None,
                    stream=None):
    """The beams' states follow the beams that were chosen (vt_beam_select's parent).

    state [..., B, W, ...] of any element type, its sequences at dimension dim and
    their beams at dim + 1; parent int32 [B, n], -1: that slot stays as it is.
    With lengths int32 [B], only the first lengths[b] positions along dimension
    len_dim are moved.  Dimensions before dim, and those between dim + 1 and
    len_dim, are evenly spaced; what follows len_dim is contiguous.
    out None (or state itself): in place, n at most W; else a tensor like state, but for
    its number of beams (at least n), that does not overlap it.  Returns (out, dev_status).
    """
    dev = _first(state, "state")
    shape, strides = state.shape, state.stride()
    sp = state.data_ptr()
    if lengths is not None and len_dim is None:
        raise ValueError("lengths needs len_dim")
    pp = _arg(parent, "parent", _I32, None, dev)
    if parent.dim() != 2:
        raise ValueError("parent must be [B, n]")
    pB, n = parent.shape
    if out is None or out is state:
        out, op = state, sp
        plan = _beam_plan(shape, strides, shape, strides, state.element_size(), int(dim), len_dim, n)
    else:
        if not isinstance(out, _TORCH.Tensor) or out.get_device() != dev or out.dtype != state.dtype:
            raise ValueError(f"out must be a tensor of {state.dtype} on cuda:{dev}")
        op, oshape, ostr = out.data_ptr(), out.shape, out.stride()
        plan = _beam_plan(shape, strides, oshape, ostr, state.element_size(), int(dim), len_dim, n)
        if sp < op + plan[9] and op < sp + plan[8] and (op != sp or ostr != strides or oshape != shape):
            raise ValueError("out must be state, or not overlap it")
    B, W, st, ost, outer, inner, positions, row = plan[:8]
    if pB != B:
        raise ValueError(f"parent must be [{B}, n], got {list(parent.shape)}")
    lp = _arg(lengths, "lengths", _I32, (B,), dev) if lengths is not None else None
    if dev_status is None:
        dev_status = _new(1, _I32[0], dev, stream)
    rc = lib().vt_beam_reorder(sp, op, st, ost, outer, B, W, n, inner, positions, row, pp, lp,
                               _arg(dev_status, "dev_status", _I32, (1,), dev), _on(stream, dev))
    if rc:
        _lib.check("vt_beam_reorder", rc)
    return out, dev_status


def _teacher(logits, top_ids, top_logp, inv_map):
    """(device, element type, leading shape, rows, K, stride, addresses and sizes of
    the teacher's list and the map) of a distillation call."""
    dev = _first(logits, "logits")
    dt, shape, R, K, ld = _logit_rows(logits)
    ip = _arg(top_ids, "top_ids", _I32, None, dev)
    full = top_ids.shape
    if full[:-1] != shape or not 1 <= full[-1] <= 128:
        raise ValueError(f"top_ids must be {list(shape)} + [k] with k in [1, 128], got {list(full)}")
    lp = _arg(top_logp, "top_logp", _F32, full, dev)
    mp, V = None, K
    if inv_map is not None:
        mp = _arg(inv_map, "inv_map", _I32, None, dev)
        V = inv_map.numel()
    return dev, dt, shape, R, K, ld, ip, lp, full[-1], mp, V


def _grad_out(out_grad, logits, shape, R, K, dev, stream):
    """(tensor, address, row stride) of the gradient of logits."""
    if out_grad is None:
        out_grad = _new((*shape, K), logits.dtype, dev, stream)
    elif not isinstance(out_grad, _TORCH.Tensor) or out_grad.get_device() != dev or \
            out_grad.dtype != logits.dtype or out_grad.shape != logits.shape:
        raise ValueError(f"out_grad must be a tensor of {logits.dtype} on cuda:{dev}, {[*shape, K]}")
    return out_grad, out_grad.data_ptr(), _logit_rows(out_grad, "out_grad")[4]


def vt_distill_loss(logits, top_ids, top_logp, inv_map=None, rest: bool = True, temperature: float = 1.0,
                    out_loss=None, out_stats=None, dev_status=None, stream=None):
    """Distillation from a teacher's k best ids: the loss of each row of the drafter's logits.

    logits [R, K] or [B, R, K], float32 or bf16, unit inner stride and evenly spaced
    rows; top_ids int32 and top_logp float32 of logits' leading shape + [k], k <= 128, as
    vt_token_logprobs returns them for the target's logits (-1: no entry); inv_map int32 [V]
    (vt_trim_head's) takes the teacher's ids to the drafter's, -1 where it has none.
    rest: what the listed ids leave of either distribution counts as one more outcome; otherwise
    the teacher is renormalised over the ids listed.  Rows with nothing to learn have loss 0.
    Returns (loss, stats, dev_status); stats [..., 5] is what vt_distill_grad needs.  As with every call of
    this package, autograd does not see it: the results carry no graph, whether logits require a
    gradient or not, and the backward pass is vt_distill_grad.
    """
    dev, dt, shape, R, K, ld, ip, lp, k, mp, V = _teacher(logits, top_ids, top_logp, inv_map)
    if out_loss is None:
        out_loss = _new(shape, _F32[0], dev, stream)
    if out_stats is None:
        out_stats = _new((*shape, 5), _F32[0], dev, stream)
    if dev_status is None:
        dev_status = _new(1, _I32[0], dev, stream)
    rc = lib().vt_distill_loss(logits.data_ptr(), dt, R, K, ld, ip, lp, k, mp, V, 1 if rest else 0,
                               float(temperature), _arg(out_loss, "out_loss", _F32, shape, dev),
                               _arg(out_stats, "out_stats", _F32, (*shape, 5), dev),
                               _arg(dev_status, "dev_status", _I32, (1,), dev), _on(stream, dev))
    if rc:
        _lib.check("vt_distill_loss", rc)
    return out_loss, out_stats, dev_status


def vt_distill_grad(logits, top_ids, top_logp, stats, grad_loss=None, inv_map=None,
                    temperature: float = 1.0, out_grad=None, stream=None):
    """The gradient of vt_distill_loss with respect to the logits, from the same arguments and the
    statistics it returned; grad_loss float32 of logits' leading shape (None: 1) is dL/dloss.
    out_grad, of logits' shape and type, may be logits itself.  Returns out_grad, for the caller
    to pass on (torch.autograd.backward(logits, out_grad), or a product with the hidden states)."""
    dev, dt, shape, R, K, ld, ip, lp, k, mp, V = _teacher(logits, top_ids, top_logp, inv_map)
    gp = _arg(grad_loss, "grad_loss", _F32, shape, dev) if grad_loss is not None else None
    out_grad, op, ldg = _grad_out(out_grad, logits, shape, R, K, dev, stream)
    rc = lib().vt_distill_grad(logits.data_ptr(), dt, R, K, ld, ip, lp, k, mp, V, float(temperature),
                               _arg(stats, "stats", _F32, (*shape, 5), dev), gp, op, ldg, _on(stream, dev))
    if rc:
        _lib.check("vt_distill_grad", rc)
    return out_grad


def vt_distill_loss_grad(logits, top_ids, top_logp, grad_loss=None, inv_map=None, rest: bool = True,
                         temperature: float = 1.0, out_loss=None, out_grad=None, out_stats=None,
                         dev_status=None, stream=None):
    """vt_distill_loss and vt_distill_grad in one call: a training step that knows each row's weight
    grad_loss beforehand.  Rows that fit on the chip are read once.  Returns (loss, grad, stats,
    dev_status), none of which autograd knows of (see vt_distill_loss)."""
    dev, dt, shape, R, K, ld, ip, lp, k, mp, V = _teacher(logits, top_ids, top_logp, inv_map)
    gp = _arg(grad_loss, "grad_loss", _F32, shape, dev) if grad_loss is not None else None
    if out_loss is None:
        out_loss = _new(shape, _F32[0], dev, stream)
    if out_stats is None:
        out_stats = _new((*shape, 5), _F32[0], dev, stream)
    if dev_status is None:
        dev_status = _new(1, _I32[0], dev, stream)
    out_grad, op, ldg = _grad_out(out_grad, logits, shape, R, K, dev, stream)
    rc = lib().vt_distill_loss_grad(logits.data_ptr(), dt, R, K, ld, ip, lp, k, mp, V, 1 if rest else 0,
                                    float(temperature), gp, _arg(out_loss, "out_loss", _F32, shape, dev),
                                    _arg(out_stats, "out_stats", _F32, (*shape, 5), dev), op, ldg,
                                    _arg(dev_status, "dev_status", _I32, (1,), dev), _on(stream, dev))
    if rc:
        _lib.check("vt_distill_loss_grad", rc)
    return out_loss, out_grad, out_stats, dev_status


def vt_selftest_wait(which: int, limit: int, flag=None, dev_status=None, stream=None):
    """Runs one of the library's bounded device waits on an object that
    nothing completes (which 0: an mbarrier; 1: the same after one arrival,
    the control; 2: a published flag, int32 [1] on the device) for at most
    `limit` polls.  VT_DEV_TIMEOUT is OR-ed into dev_status (int32 [1],
    zeroed here when not given) when the wait gives up."""
    torch = _torch()
    if dev_status is None:
        dev = flag.device if flag is not None else torch.device("cuda", torch.cuda.current_device())
        dev_status = _empty(1, torch.int32, dev, stream)
        with torch.cuda.stream(_as_stream(stream, dev)):  # zeroed there, ahead of the kernel
            dev_status.zero_()
    _dev(dev_status, "dev_status", (torch.int32,), 1)
    if flag is not None:
        _dev(flag, "flag", (torch.int32, torch.uint32), 1)
    st = lib().vt_selftest_wait(int(which), int(limit),
                                flag.data_ptr() if flag is not None else None,
                                dev_status.data_ptr(), _stream_ptr(stream))
    _lib.check("vt_selftest_wait", st)
    return dev_status


class BlockGraph:
    """One speculative block (gamma drafting steps + verification) captured
    as a CUDA graph by vt_block_graph_create and replayed by launch().

    The tensors are fixed at capture and kept alive by this object; a replay
    reads what they hold when it runs.  Replays may run on any stream: the
    constructor waits until the current stream has no other use of their
    memory, and their memory is not given to another while a stream of torch's
    that launched the graph is at it.  Outputs (q, draft_tokens,
    out_tokens, out_num_accepted, out_accept_prob, dev_status [2]) are
    attributes.  temperature == 0 captures the greedy block (u_draft,
    u_accept and u_resample may then be None).  With w_scale, W_trim is an
    e4m3 head as vt_quantize_head leaves it (vt_block_graph_create_fp8)."""

    def __init__(self, hidden, W_trim, trim_ids, inv_map, target_logits, u_draft=None,
                 u_accept=None, u_resample=None, temperature: float = 1.0,
                 want_accept_prob: bool = True, w_scale=None):
        torch = _torch()
        greedy = float(temperature) == 0.0
        _dev(hidden, "hidden", _bf16_dtypes(), 3)
        fp8 = None
        if w_scale is None:
            _dev(W_trim, "W_trim", _bf16_dtypes(), 2)
        else:
            K8, H8, ldw, p8, sp = _head_fp8(W_trim, w_scale, _first(hidden, "hidden"))
            if H8 != hidden.shape[2]:
                raise ValueError("hidden and W_trim disagree on H")
            if trim_ids.numel() != K8:
                raise ValueError("trim_ids must have K elements")
            fp8 = (p8, ldw, sp)
        _dev(trim_ids, "trim_ids", (torch.int32,), 1)
        _dev(inv_map, "inv_map", (torch.int32,), 1)
        if target_logits.dtype == torch.float32:
            dt = VT_F32
        elif target_logits.dtype in _bf16_dtypes():
            dt = VT_BF16
        else:
            raise TypeError("target_logits must be float32 or bf16")
        _dev(target_logits, "target_logits", (target_logits.dtype,), 3)
        gamma, B, H = hidden.shape
        K = W_trim.shape[0]
        V = target_logits.shape[2]
        if tuple(target_logits.shape[:2]) != (B, gamma + 1) or inv_map.numel() != V:
            raise ValueError("target_logits must be [B, gamma+1, V] and inv_map [V]")
        for name, x, shape in (("u_draft", u_draft, (gamma, B)), ("u_accept", u_accept, (B, gamma)),
                               ("u_resample", u_resample, (B, gamma + 1))):
            if x is None:
                if not greedy:
                    raise ValueError(f"{name} is needed unless temperature == 0")
                continue
            _dev(x, name, (torch.float32,), 2)
            if tuple(x.shape) != shape:
                raise ValueError(f"{name} must be {shape}")
        dev = hidden.device
        self.q = torch.empty((B, gamma, K), dtype=torch.float32, device=dev)
        self.draft_tokens = torch.empty((B, gamma), dtype=torch.int32, device=dev)
        self.out_tokens = torch.empty((B, gamma + 1), dtype=torch.int32, device=dev)
        self.out_num_accepted = torch.empty(B, dtype=torch.int32, device=dev)
        self.out_accept_prob = (torch.empty((B, gamma), dtype=torch.float32, device=dev)
                                if want_accept_prob else None)
        self.dev_status = torch.zeros(2, dtype=torch.int32, device=dev)
        L = lib()
        self.workspace = _ws((L.vt_block_fp8_workspace_bytes if fp8 else L.vt_block_workspace_bytes)(
            B, H, K, V, gamma), dev)
        self._keep = (hidden, W_trim, trim_ids, inv_map, target_logits, u_draft, u_accept,
                      u_resample, w_scale)
        ptr = lambda x: x.data_ptr() if x is not None else None
        d = _lib.BlockDesc(B, H, K, V, gamma, dt, float(temperature), ptr(hidden),
                           None if fp8 else ptr(W_trim),
                           ptr(trim_ids), ptr(inv_map), ptr(u_draft), ptr(target_logits),
                           ptr(u_accept), ptr(u_resample), ptr(self.q), ptr(self.draft_tokens),
                           ptr(self.out_tokens), ptr(self.out_num_accepted),
                           ptr(self.out_accept_prob), ptr(self.dev_status),
                           ptr(self.workspace), self.workspace.numel())
        import ctypes
        h = ctypes.c_void_p()
        if fp8:
            _lib.check("vt_block_graph_create_fp8",
                       L.vt_block_graph_create_fp8(ctypes.byref(d), *fp8, ctypes.byref(h)))
        else:
            _lib.check("vt_block_graph_create",
                       L.vt_block_graph_create(ctypes.byref(d), ctypes.byref(h)))
        self._handle = h
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(dev).synchronize()
        self._known = set()  # raw streams that the allocator knows as users

    def launch(self, stream=None):
        ptr = _stream_ptr(stream)
        if ptr not in self._known:
            self._known.add(ptr)
            s = _TORCH.cuda.current_stream() if stream is None else stream
            # (a stream of the caller's own may not live as long as the tensors)
            own = not isinstance(s, _TORCH.cuda.Stream) or isinstance(s, _TORCH.cuda.ExternalStream)
            for t in () if own else (*self._keep, self.q, self.draft_tokens, self.out_tokens, self.out_num_accepted,
                      self.out_accept_prob, self.dev_status, self.workspace):
                if t is not None:
                    t.record_stream(s)
        _lib.check("vt_block_graph_launch", lib().vt_block_graph_launch(self._handle, ptr))

    def close(self):
        if getattr(self, "_handle", None):
            lib().vt_block_graph_destroy(self._handle)
            self._handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
