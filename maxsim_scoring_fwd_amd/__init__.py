"""MI355X-native late-interaction MaxSim scoring.

Thin Python front end of libmaxsim.so (the C-ABI in include/maxsim.h). The
functions here only marshal arguments: torch tensors supply device memory and
the current HIP stream, and every step of the computation runs in the HIP
kernels of libmaxsim. There is no CPU fallback: if the library is missing or no
gfx950 device is present, the calls raise.

    score(q_i, d_j) summed:  out[b] = sum_i max_j <q_i, d_j>

Beside the scoring it has what the encoder in front of it needs, on the same document
layouts: attention within documents, rotary positions, the norm with the residual's addition,
dropout, the cross entropy over a vocabulary, and the clipping of gradients by their global norm;
and for the index 8-bit and 4-bit vectors.
"""
from __future__ import annotations

import ctypes
import math
import operator
import os
import struct
from array import array

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmaxsim.so")

MAXSIM_BF16, MAXSIM_FP16, MAXSIM_FP32 = 0, 1, 2
_TORCH_DTYPE = {torch.bfloat16: MAXSIM_BF16, torch.float16: MAXSIM_FP16,
                torch.float32: MAXSIM_FP32}

STATUS = {0: "MAXSIM_OK", -1: "MAXSIM_ERR_NULL", -2: "MAXSIM_ERR_SHAPE", -3: "MAXSIM_ERR_DTYPE",
          -4: "MAXSIM_ERR_ALIGN", -5: "MAXSIM_ERR_UNSUPPORTED", -6: "MAXSIM_ERR_LAUNCH",
          -7: "MAXSIM_ERR_DEVICE", -8: "MAXSIM_ERR_SCRATCH"}


class MaxSimError(RuntimeError):
    def __init__(self, status: int, func: str, msg: str):
        super().__init__(f"{func}: {STATUS.get(status, status)} ({msg})")
        self.status = status


# maxsim_attention_desc: q, k and v (address; token, head and document stride), offsets, lengths,
# tokens, documents, prefixes, slopes; nd, heads, key/value heads, d, dtype, causal; cap, scale
_ATTENTION_DESC = struct.Struct("@" + "Pqqq" * 3 + "PPqqPP" + "6i" + "2f")

_lib_handle = None


def lib() -> ctypes.CDLL:
    """The loaded libmaxsim.so with argument types declared."""
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() or "
                              "python -m maxsim_scoring_fwd_amd.build")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        L.maxsim_score.argtypes = [vp, i32, vp, vp, i64, i32, i32, vp, vp]
        L.maxsim_score_fixed.argtypes = [vp, i32, vp, i64, i32, vp, i32, i32, vp, vp]
        L.maxsim_score_i8.argtypes = [vp, vp, i32, vp, vp, vp, i64, i32, i32, vp, vp, vp, vp]
        L.maxsim_pq_tables.argtypes = [vp, i32, i32, vp, i32, i32, i32, vp, vp]
        L.maxsim_score_pq.argtypes = [vp, i32, i32, i32, vp, vp, i64, i32, vp, vp]
        L.maxsim_score_argmax.argtypes = [vp, i32, vp, vp, i64, i32, i32, i32, vp, vp, vp, vp]
        L.maxsim_score_batch.argtypes = [vp, i32, i32, vp, vp, i64, i32, i32, i32, vp, vp]
        L.maxsim_backward.argtypes = [vp, i32, vp, vp, i64, i32, i32, i32, vp, vp, vp, vp, i32,
                                      vp, ctypes.c_size_t, vp]
        L.maxsim_backward_workspace_size.argtypes = [i32, i32, i64]
        L.maxsim_backward_workspace_size.restype = ctypes.c_size_t
        L.maxsim_topk.argtypes = [vp, i64, i32, i32, vp, vp, vp, ctypes.c_size_t, vp]
        L.maxsim_topk_workspace_size.argtypes = [i64, i32, i32]
        L.maxsim_topk_workspace_size.restype = ctypes.c_size_t
        L.maxsim_topk_no_alloc.argtypes = [vp, i64, i32, i32, vp, vp, vp]
        L.maxsim_topk_scratch_bytes.argtypes = []
        L.maxsim_topk_scratch_bytes.restype = ctypes.c_size_t
        f32, f64, sz = ctypes.c_float, ctypes.c_double, ctypes.c_size_t
        L.maxsim_rotary.argtypes = [vp, i64, i32, i32, i64, i64, i32, vp, i32, i32, f32, i32, vp,
                                    i64, vp, vp, i64, i64, vp]
        L.maxsim_attention.argtypes = [vp, vp, vp, vp]
        L.maxsim_attention_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.maxsim_attention_backward_workspace_size.argtypes = [i64, i32]
        L.maxsim_attention_backward_workspace_size.restype = sz
        L.maxsim_clip_grad_norm.argtypes = [vp, vp, vp, vp, i32, f64, vp, vp, sz, vp]
        L.maxsim_clip_grad_norm_workspace_size.argtypes = [i32]
        L.maxsim_clip_grad_norm_workspace_size.restype = sz
        L.maxsim_dropout.argtypes = [vp, i64, i32, f64, vp, i32, vp, vp]
        L.maxsim_rms_norm.argtypes = [vp, i64, vp, i64, i64, i32, i32, vp, i32, f32, f64, vp, i32,
                                      vp, vp, vp, vp]
        L.maxsim_rms_norm_i8.argtypes = [vp, i64, vp, i64, i64, i32, i32, vp, i32, f32, vp, vp, vp,
                                         vp]
        L.maxsim_rms_norm_backward.argtypes = [vp, vp, vp, i64, i64, i32, i32, vp, i32, vp, f64, vp,
                                               i32, vp, vp, vp, vp, sz, vp]
        L.maxsim_linear_cross_entropy.argtypes = [vp, vp, vp, i64, i64, i32, i32, f32, vp, vp, vp,
                                                  sz, vp]
        L.maxsim_linear_cross_entropy_backward.argtypes = [vp, vp, vp, vp, vp, i64, i64, i32, i32,
                                                           f32, vp, vp, vp, sz, vp]
        L.maxsim_rms_norm_backward_workspace_size.argtypes = [i64, i32]
        L.maxsim_linear_cross_entropy_workspace_size.argtypes = [i64, i64, i32, i32]
        L.maxsim_linear_cross_entropy_backward_workspace_size.argtypes = [i64, i64, i32, i32]
        for f in ("rms_norm_backward", "linear_cross_entropy", "linear_cross_entropy_backward"):
            getattr(L, f"maxsim_{f}_workspace_size").restype = sz
        L.maxsim_quantize_mx4.argtypes = [vp, i64, i32, i32, vp, vp, vp]
        L.maxsim_dequantize_mx4.argtypes = [vp, vp, i64, i32, i32, vp, vp]
        L.maxsim_score_mx4.argtypes = [vp, vp, i32, vp, vp, vp, i64, i32, vp, i32, vp, vp]
        L.maxsim_status_string.argtypes = [i32]
        L.maxsim_status_string.restype = ctypes.c_char_p
        L.maxsim_version.argtypes = []
        for f in ("maxsim_score", "maxsim_score_fixed", "maxsim_score_i8", "maxsim_pq_tables",
                  "maxsim_score_pq", "maxsim_version", "maxsim_score_argmax", "maxsim_backward",
                  "maxsim_score_batch", "maxsim_topk", "maxsim_topk_no_alloc", "maxsim_rotary",
                  "maxsim_attention", "maxsim_attention_backward", "maxsim_clip_grad_norm",
                  "maxsim_dropout", "maxsim_rms_norm", "maxsim_rms_norm_i8",
                  "maxsim_rms_norm_backward", "maxsim_linear_cross_entropy",
                  "maxsim_linear_cross_entropy_backward", "maxsim_quantize_mx4",
                  "maxsim_dequantize_mx4", "maxsim_score_mx4"):
            getattr(L, f).restype = ctypes.c_int
        _lib_handle = L
    return _lib_handle


def _check(rc: int, func: str):
    if rc != 0:
        raise MaxSimError(rc, func, lib().maxsim_status_string(rc).decode())


def _dev(t: torch.Tensor | None, name: str):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


# The current stream's handle without a Stream object, a microsecond less a call. Both functions are
# torch's own business: without them the public ones serve.
_RAW_STREAMS = all(hasattr(torch._C, f) for f in ("_cuda_getDevice", "_cuda_getCurrentRawStream"))


def _current_device() -> int:
    return torch._C._cuda_getDevice() if _RAW_STREAMS else torch.cuda.current_device()


def _stream(stream) -> int | None:
    if stream is None:
        if not _RAW_STREAMS:
            return torch.cuda.current_stream().cuda_stream
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _TORCH_DTYPE:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return _TORCH_DTYPE[t.dtype]


def _new(shape, dtype, device, stream) -> torch.Tensor:
    """A new tensor for work on `stream`. It comes from that stream's own memory: a block that the
    current stream has given back may still have work queued on it there, which `stream` would not
    wait for. The caller goes on with it on the current stream: it is not handed out again before
    that one is past it either."""
    if stream is None or device.type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(s):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream())
    return t


def _out(out, n, device, stream, dtype=torch.float32):
    if out is None:
        return _new(n, dtype, device, stream)
    _need(out, "out", dtype, numel=n)
    return out


# Host-side checks of dtypes and shapes. The library takes every type from its arguments
# (the storage dtype from Q, offsets as int64, argmax as int32 ...) and cannot see a
# tensor's dtype, so a mismatch here would make the kernels read past the end of a buffer.
def _need(t, name: str, dtypes, shape=None, numel=None, dim=None):
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if not isinstance(dtypes, (tuple, list)):
        dtypes = (dtypes,)
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must have dtype {' or '.join(str(x) for x in dtypes)}, "
                         f"got {t.dtype}")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got shape {tuple(t.shape)}")
    if shape is not None and t.shape != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must hold {numel} elements, got {t.numel()}")


_FLOAT_STORAGE = tuple(_TORCH_DTYPE)


def _query(Q: torch.Tensor, dim: int = 2) -> None:
    _need(Q, "Q", _FLOAT_STORAGE, dim=dim)


def _docs_like(Q: torch.Tensor, D: torch.Tensor, doc_offsets) -> None:
    """D shares Q's dtype and embedding dimension; [n_docs, nd, d] without offsets, else
    [n_tokens, d] with int64 offsets [n_docs + 1]."""
    _need(D, "D", Q.dtype, dim=2 if doc_offsets is not None else 3)
    if D.shape[-1] != Q.shape[-1]:
        raise ValueError(f"D has d = {D.shape[-1]}, Q has d = {Q.shape[-1]}")
    if doc_offsets is not None:
        _need(doc_offsets, "doc_offsets", torch.int64, dim=1)
        if doc_offsets.numel() < 1:
            raise ValueError("doc_offsets needs n_docs + 1 >= 1 entries")


def maxsim_score(Q: torch.Tensor, D: torch.Tensor, doc_offsets: torch.Tensor,
                 out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """CSR documents. Q [q_len, d], D [n_tokens, d] (same dtype), doc_offsets int64
    [n_docs+1]; returns fp32 scores [n_docs]."""
    _query(Q)
    if doc_offsets is None:
        raise ValueError("maxsim_score needs doc_offsets (use maxsim_score_fixed without)")
    _docs_like(Q, D, doc_offsets)
    n_docs = doc_offsets.numel() - 1
    out = _out(out, n_docs, Q.device, stream)
    _check(lib().maxsim_score(_dev(Q, "Q"), Q.shape[0], _dev(D, "D"),
                              _dev(doc_offsets, "doc_offsets"), n_docs, Q.shape[1],
                              _dtype_code(Q), _dev(out, "out"), _stream(stream)), "maxsim_score")
    return out


def maxsim_score_fixed(Q: torch.Tensor, D: torch.Tensor, doc_lens: torch.Tensor | None = None,
                       out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Fixed-length documents. Q [q_len, d], D [n_docs, nd, d]; doc_lens int32 [n_docs]
    (optional) masks trailing padding tokens. Returns fp32 scores [n_docs]."""
    _query(Q)
    _docs_like(Q, D, None)
    n_docs, nd = D.shape[0], D.shape[1]
    _need(doc_lens, "doc_lens", torch.int32, numel=n_docs)
    out = _out(out, n_docs, Q.device, stream)
    _check(lib().maxsim_score_fixed(_dev(Q, "Q"), Q.shape[0], _dev(D, "D"), n_docs, nd,
                                    _dev(doc_lens, "doc_lens"), Q.shape[1], _dtype_code(Q),
                                    _dev(out, "out"), _stream(stream)), "maxsim_score_fixed")
    return out


def maxsim_score_i8(Q: torch.Tensor, q_scale: torch.Tensor, D: torch.Tensor,
                    d_scale: torch.Tensor, doc_offsets: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, with_token_max: bool = False, stream=None):
    """INT8 x INT8 with per-token fp32 scales. Fixed layout (D [n_docs, nd, d]) when
    doc_offsets is None, else CSR (D [n_tokens, d]). Returns scores, or (scores, tok_max,
    tok_arg) with with_token_max."""
    _need(Q, "Q", torch.int8, dim=2)
    q_len, d = Q.shape
    _need(q_scale, "q_scale", torch.float32, numel=q_len)
    _need(D, "D", torch.int8, dim=2 if doc_offsets is not None else 3)
    if D.shape[-1] != d:
        raise ValueError(f"D has d = {D.shape[-1]}, Q has d = {d}")
    if doc_offsets is None:
        n_docs, nd = D.shape[0], D.shape[1]
    else:
        _need(doc_offsets, "doc_offsets", torch.int64, dim=1)
        n_docs, nd = doc_offsets.numel() - 1, 0
    _need(d_scale, "d_scale", torch.float32, numel=D.numel() // max(d, 1))
    out = _out(out, n_docs, Q.device, stream)
    tm = ta = None
    if with_token_max:
        tm = _new((n_docs, q_len), torch.float32, Q.device, stream)
        ta = _new((n_docs, q_len), torch.int32, Q.device, stream)
    _check(lib().maxsim_score_i8(_dev(Q, "Q"), _dev(q_scale, "q_scale"), q_len, _dev(D, "D"),
                                 _dev(d_scale, "d_scale"), _dev(doc_offsets, "doc_offsets"),
                                 n_docs, nd, d, _dev(out, "out"), _dev(tm, "tok_max"),
                                 _dev(ta, "tok_arg"), _stream(stream)), "maxsim_score_i8")
    return (out, tm, ta) if with_token_max else out


def _docs(D: torch.Tensor, doc_offsets):
    """(n_docs, nd) of fixed documents D [n_docs, nd, d] or CSR tokens D [n_tokens, d]."""
    if doc_offsets is None:
        return D.shape[0], D.shape[1]
    return doc_offsets.numel() - 1, 0


def maxsim_score_argmax(Q: torch.Tensor, D: torch.Tensor, doc_offsets: torch.Tensor | None = None,
                        out=None, tok_max=None, tok_arg=None, stream=None):
    """Scores with per-token maxima and argmax (lowest index on ties). Fixed layout
    (D [n_docs, nd, d]) when doc_offsets is None, else CSR (D [n_tokens, d]). Returns
    (scores fp32 [n_docs], tok_max fp32 [n_docs, q_len], tok_arg int32 [n_docs, q_len])."""
    _query(Q)
    _docs_like(Q, D, doc_offsets)
    q_len, d = Q.shape
    n_docs, nd = _docs(D, doc_offsets)
    out = _out(out, n_docs, Q.device, stream)
    _need(tok_max, "tok_max", torch.float32, shape=(n_docs, q_len))
    _need(tok_arg, "tok_arg", torch.int32, shape=(n_docs, q_len))
    if tok_max is None:
        tok_max = _new((n_docs, q_len), torch.float32, Q.device, stream)
    if tok_arg is None:
        tok_arg = _new((n_docs, q_len), torch.int32, Q.device, stream)
    _check(lib().maxsim_score_argmax(_dev(Q, "Q"), q_len, _dev(D, "D"),
                                     _dev(doc_offsets, "doc_offsets"), n_docs, nd, d,
                                     _dtype_code(Q), _dev(out, "out"), _dev(tok_max, "tok_max"),
                                     _dev(tok_arg, "tok_arg"), _stream(stream)),
           "maxsim_score_argmax")
    return out, tok_max, tok_arg


def maxsim_score_batch(Q: torch.Tensor, D: torch.Tensor, doc_offsets: torch.Tensor | None = None,
                       out=None, stream=None) -> torch.Tensor:
    """Several queries in one pass over the documents. Q [n_q, q_len, d]; fixed documents
    D [n_docs, nd, d] when doc_offsets is None, else CSR D [n_tokens, d]. Returns fp32 scores
    [n_q, n_docs]."""
    _query(Q, dim=3)
    _docs_like(Q, D, doc_offsets)
    n_q, q_len, d = Q.shape
    n_docs, nd = _docs(D, doc_offsets)
    if out is None:
        out = _new((n_q, n_docs), torch.float32, Q.device, stream)
    _need(out, "out", torch.float32, numel=n_q * n_docs)
    _check(lib().maxsim_score_batch(_dev(Q, "Q"), n_q, q_len, _dev(D, "D"),
                                    _dev(doc_offsets, "doc_offsets"), n_docs, nd, d,
                                    _dtype_code(Q), _dev(out, "out"), _stream(stream)),
           "maxsim_score_batch")
    return out


def topk_workspace_size(n: int, rows: int, k: int) -> int:
    """Bytes of workspace maxsim_topk needs."""
    return int(lib().maxsim_topk_workspace_size(n, rows, k))


def maxsim_topk(scores: torch.Tensor, k: int, out_scores=None, out_index=None, workspace=None,
                stream=None):
    """The k best entries of each row of scores ([n] or [rows, n] fp32) by (score
    descending, index ascending). Returns (values, indices) shaped [k] or [rows, k]."""
    _need(scores, "scores", torch.float32)
    if scores.dim() not in (1, 2):
        raise ValueError("scores must be [n] or [rows, n]")
    rows, n = (1, scores.shape[0]) if scores.dim() == 1 else scores.shape
    shape = (k,) if scores.dim() == 1 else (rows, k)
    _need(out_scores, "out_scores", torch.float32, numel=rows * k)
    _need(out_index, "out_index", torch.int32, numel=rows * k)
    _need(workspace, "workspace", torch.uint8)
    if out_scores is None:
        out_scores = _new(shape, torch.float32, scores.device, stream)
    if out_index is None:
        out_index = _new(shape, torch.int32, scores.device, stream)
    need = topk_workspace_size(n, rows, k)
    if workspace is None and need > 0:
        workspace = _new(need, torch.uint8, scores.device, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().maxsim_topk(_dev(scores, "scores"), n, rows, k, _dev(out_scores, "out_scores"),
                             _dev(out_index, "out_index"), _dev(workspace, "workspace"), ws_bytes,
                             _stream(stream)), "maxsim_topk")
    return out_scores, out_index


def maxsim_topk_no_alloc(scores: torch.Tensor, k: int, out_scores: torch.Tensor,
                         out_index: torch.Tensor, stream=None):
    """maxsim_topk with the library's static scratch memory instead of a workspace: the
    library allocates nothing (outputs are the caller's). Calls overlapping on one GPU race."""
    _need(scores, "scores", torch.float32)
    if scores.dim() not in (1, 2):
        raise ValueError("scores must be [n] or [rows, n]")
    rows, n = (1, scores.shape[0]) if scores.dim() == 1 else scores.shape
    _need(out_scores, "out_scores", torch.float32, numel=rows * k)
    _need(out_index, "out_index", torch.int32, numel=rows * k)
    _check(lib().maxsim_topk_no_alloc(_dev(scores, "scores"), n, rows, k,
                                      _dev(out_scores, "out_scores"), _dev(out_index, "out_index"),
                                      _stream(stream)), "maxsim_topk_no_alloc")
    return out_scores, out_index


def topk_scratch_bytes() -> int:
    """Bytes of the static scratch array maxsim_topk_no_alloc uses on each GPU."""
    return int(lib().maxsim_topk_scratch_bytes())


def backward_workspace_size(q_len: int, d: int, n_docs: int) -> int:
    """Bytes of workspace maxsim_backward needs to produce dQ."""
    return int(lib().maxsim_backward_workspace_size(q_len, d, n_docs))


def maxsim_backward(Q: torch.Tensor, D: torch.Tensor, tok_arg: torch.Tensor,
                    grad_out: torch.Tensor, doc_offsets: torch.Tensor | None = None,
                    want_dQ: bool = True, want_dD: bool = True, grad_dtype=torch.float32,
                    dQ=None, dD=None, workspace=None, stream=None):
    """Gradients of sum_b grad_out[b] * score_b from the forward argmax tok_arg. Returns
    (dQ [q_len, d], dD shaped like D), each None when not asked for; grad_dtype is float32
    or the dtype of Q and D."""
    _query(Q)
    _docs_like(Q, D, doc_offsets)
    if grad_dtype not in (torch.float32, Q.dtype):
        raise ValueError("grad_dtype must be float32 or the dtype of Q")
    q_len, d = Q.shape
    n_docs, nd = _docs(D, doc_offsets)
    _need(tok_arg, "tok_arg", torch.int32, shape=(n_docs, q_len))
    _need(grad_out, "grad_out", torch.float32, numel=n_docs)
    _need(dQ, "dQ", grad_dtype, shape=(q_len, d))
    _need(dD, "dD", grad_dtype, shape=tuple(D.shape))
    _need(workspace, "workspace", torch.uint8)
    if want_dQ and dQ is None:
        dQ = _new((q_len, d), grad_dtype, Q.device, stream)
    if want_dD and dD is None:
        dD = _new(D.shape, grad_dtype, Q.device, stream)
    if not want_dQ:
        dQ = None
    if not want_dD:
        dD = None
    ws_bytes = 0
    if dQ is not None:
        ws_bytes = backward_workspace_size(q_len, d, n_docs)
        if workspace is None:
            workspace = _new(max(ws_bytes, 16), torch.uint8, Q.device, stream)
        ws_bytes = workspace.numel() * workspace.element_size()
    else:
        workspace = None
    _check(lib().maxsim_backward(_dev(Q, "Q"), q_len, _dev(D, "D"), _dev(doc_offsets, "doc_offsets"),
                                 n_docs, nd, d, _dtype_code(Q), _dev(tok_arg, "tok_arg"),
                                 _dev(grad_out, "grad_out"), _dev(dQ, "dQ"), _dev(dD, "dD"),
                                 _TORCH_DTYPE[grad_dtype], _dev(workspace, "workspace"), ws_bytes,
                                 _stream(stream)), "maxsim_backward")
    return dQ, dD


class FirstOrderFunction(torch.autograd.Function):
    """Gradients (what `gradients` returns) that depend on `inputs` and have no derivative here:
    with create_graph they are part of the graph, and differentiating them is an error."""

    @staticmethod
    def forward(ctx, name, gradients, *inputs):
        ctx.name = name
        return gradients()

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(f"the gradients of {ctx.name} cannot be differentiated again")


class MaxSimFunction(torch.autograd.Function):
    """Differentiable MaxSim scores: the forward keeps the argmax, the backward turns it
    into dQ and dD with the library's kernels (gradients in the input dtype)."""

    @staticmethod
    def forward(ctx, Q, D, doc_offsets):
        scores, _, tok_arg = maxsim_score_argmax(Q, D, doc_offsets)
        ctx.save_for_backward(Q, D, doc_offsets, tok_arg)
        return scores

    @staticmethod
    def backward(ctx, grad_scores):
        Q, D, doc_offsets, tok_arg = ctx.saved_tensors
        want_dQ, want_dD = ctx.needs_input_grad[:2]

        def gradients():
            return maxsim_backward(Q, D, tok_arg, grad_scores.float().contiguous(), doc_offsets,
                                   want_dQ=want_dQ, want_dD=want_dD, grad_dtype=Q.dtype)
        if torch.is_grad_enabled():
            dQ, dD = FirstOrderFunction.apply("maxsim", gradients, grad_scores, Q, D)
        else:
            dQ, dD = gradients()
        return dQ, dD, None


def maxsim(Q: torch.Tensor, D: torch.Tensor, doc_offsets: torch.Tensor | None = None):
    """Scores [n_docs] that autograd can differentiate with respect to Q and D, once: a gradient of
    the gradients is an error."""
    return MaxSimFunction.apply(Q, D, doc_offsets)


def maxsim_pq_tables(Q: torch.Tensor, C: torch.Tensor, T: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """PQ distance tables T [q_len, M, K] fp32 from Q [q_len, M*dsub] and C [M, K, dsub] fp32."""
    _query(Q)
    _need(C, "C", torch.float32, dim=3)
    M, K, dsub = C.shape
    if Q.shape[1] != M * dsub:
        raise ValueError(f"Q has d = {Q.shape[1]}, the codebook M * dsub = {M * dsub}")
    if T is None:
        T = _new((Q.shape[0], M, K), torch.float32, Q.device, stream)
    _need(T, "T", torch.float32, shape=(Q.shape[0], M, K))
    _check(lib().maxsim_pq_tables(_dev(Q, "Q"), Q.shape[0], _dtype_code(Q), _dev(C, "C"), M, K,
                                  dsub, _dev(T, "T"), _stream(stream)), "maxsim_pq_tables")
    return T


def maxsim_score_pq(T: torch.Tensor, codes: torch.Tensor, doc_offsets: torch.Tensor | None = None,
                    nd: int = 0, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Fused PQ lookup scoring. T [q_len, M, K] fp32, codes uint8 [n_tokens, M]; CSR when
    doc_offsets is given, else fixed documents of nd tokens."""
    _need(T, "T", torch.float32, dim=3)
    q_len, M, K = T.shape
    _need(codes, "codes", torch.uint8, dim=2)
    if codes.shape[1] != M:
        raise ValueError(f"codes have {codes.shape[1]} subspaces, T has M = {M}")
    if doc_offsets is not None:
        _need(doc_offsets, "doc_offsets", torch.int64, dim=1)
    elif nd < 1:
        raise ValueError("fixed documents need nd >= 1")
    n_docs = doc_offsets.numel() - 1 if doc_offsets is not None else codes.shape[0] // max(nd, 1)
    out = _out(out, n_docs, T.device, stream)
    _check(lib().maxsim_score_pq(_dev(T, "T"), q_len, M, K, _dev(codes, "codes"),
                                 _dev(doc_offsets, "doc_offsets"), n_docs, nd, _dev(out, "out"),
                                 _stream(stream)), "maxsim_score_pq")
    return out


# ---- what an encoder in front of the scoring needs ----

def _on(t: torch.Tensor, name: str, at: int) -> int:
    """Address of a tensor of any strides on device number `at`."""
    if t.get_device() == at >= 0:
        return t.data_ptr()
    if at < 0 or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    raise ValueError(f"{name} is on cuda:{t.get_device()}, expected cuda:{at}")


def _at(t: torch.Tensor | None, name: str, at: int):
    """Address of a contiguous tensor on device number `at`, or None."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr() if t.get_device() == at >= 0 else _on(t, name, at)


def _stream_at(stream, at: int) -> int | None:
    """The stream's handle; launches go to the current device, which has to be number `at`."""
    now = _current_device()
    if now != at:
        raise ValueError(f"the tensors are on cuda:{at}, the current device is cuda:{now}")
    if stream is None and _RAW_STREAMS:
        return torch._C._cuda_getCurrentRawStream(at)
    return _stream(stream)


def _like(t: torch.Tensor, stream) -> torch.Tensor:
    """A new contiguous tensor like t, for work on `stream`."""
    if stream is None:
        return torch.empty_like(t, memory_format=torch.contiguous_format)
    return _new(t.shape, t.dtype, t.device, stream)


def _beside(t: torch.Tensor, shape, dtype, stream) -> torch.Tensor:
    """A new tensor on t's device, for work on `stream`."""
    if stream is None:
        # numbers are read faster than a shape
        return t.new_empty(*shape, dtype=dtype) if shape else t.new_empty((), dtype=dtype)
    return _new(shape, dtype, t.device, stream)


_ROTARY_LAYOUT = {"half": 0, "interleaved": 1}


def maxsim_rotary(x: torch.Tensor, freq: torch.Tensor, doc_offsets: torch.Tensor | None = None,
                  positions: torch.Tensor | None = None, layout: str = "half",
                  mscale: float = 1.0, inverse: bool = False, out: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """Rotary positions of x [n_tokens, n_heads, d], whose entries of a head lie side by side.
    The first 2 * len(freq) entries of each head are turned in pairs by position * freq (fp32,
    angle per position) and multiplied by mscale, the others copied. layout: "half" pairs entry
    f with f + len(freq), "interleaved" 2f with 2f + 1. A token's position is positions[t]
    (int32), or its index in its document (doc_offsets int64 [n_docs + 1]), or its index.
    inverse turns by the opposite angle: the gradient of x from the gradient of the result. out
    may be x itself. Returns a tensor shaped like x."""
    _need(x, "x", _FLOAT_STORAGE, dim=3)
    _need(freq, "freq", torch.float32, dim=1)
    n, heads, d = x.shape
    x_token, x_head, x_entry = x.stride()
    half, docs = freq.numel(), 0
    if layout not in _ROTARY_LAYOUT:
        raise ValueError(f"layout must be 'half' or 'interleaved', got {layout!r}")
    if not 1 <= half <= d // 2:
        raise ValueError(f"freq has {half} entries for heads of d = {d}")
    if positions is not None:
        if doc_offsets is not None:
            raise ValueError("give doc_offsets or positions, not both")
        _need(positions, "positions", torch.int32, shape=(n,))
    elif doc_offsets is not None:
        _need(doc_offsets, "doc_offsets", torch.int64, dim=1)
        docs = doc_offsets.numel() - 1
        if docs < 0:
            raise ValueError("doc_offsets needs n_docs + 1 >= 1 entries")
    if x_entry != 1:
        raise ValueError("x needs the entries of a head side by side")
    if out is None:
        out = _like(x, stream)
        out_token, out_head = heads * d, d
    else:
        _need(out, "out", x.dtype, shape=x.shape)
        out_token, out_head, out_entry = out.stride()
        if out_entry != 1:
            raise ValueError("out needs the entries of a head side by side")
    at = x.get_device()
    _check(lib().maxsim_rotary(
        _on(x, "x", at), n, heads, d, x_token, x_head, _TORCH_DTYPE[x.dtype], _at(freq, "freq", at),
        2 * half, _ROTARY_LAYOUT[layout], mscale, 1 if inverse else 0,
        _at(doc_offsets, "doc_offsets", at), docs, _at(positions, "positions", at),
        _on(out, "out", at), out_token, out_head, _stream_at(stream, at)), "maxsim_rotary")
    return out


class RotaryFunction(torch.autograd.Function):
    """Differentiable rotary positions, to any order; freq and the positions are constants."""

    @staticmethod
    def forward(ctx, x, freq, doc_offsets, positions, layout, mscale, inverse):
        ctx.save_for_backward(freq, doc_offsets, positions)
        ctx.layout, ctx.mscale, ctx.inverse = layout, mscale, inverse
        return maxsim_rotary(x, freq, doc_offsets, positions, layout, mscale, inverse)

    @staticmethod
    def backward(ctx, grad):
        freq, doc_offsets, positions = ctx.saved_tensors
        if grad.stride(2) != 1:
            grad = grad.contiguous()
        # with create_graph the gradient is to be differentiated itself: it is linear in grad
        turn = RotaryFunction.apply if torch.is_grad_enabled() else maxsim_rotary
        dx = turn(grad, freq, doc_offsets, positions, ctx.layout, ctx.mscale, not ctx.inverse)
        return dx, None, None, None, None, None, None


def rotary(x: torch.Tensor, freq: torch.Tensor, doc_offsets: torch.Tensor | None = None,
           positions: torch.Tensor | None = None, layout: str = "half",
           mscale: float = 1.0) -> torch.Tensor:
    """maxsim_rotary that autograd can differentiate with respect to x, to any order."""
    return RotaryFunction.apply(x, freq, doc_offsets, positions, layout, mscale, False)


def _attention_refuse(q, k, v, doc_offsets, doc_lens, causal, prefix_lens, slopes):
    """Raises for the first argument of an attention call whose type or shape does not fit."""
    dim = 4 if doc_offsets is None else 3
    _need(q, "q", _FLOAT_STORAGE, dim=dim)
    heads, d = q.shape[-2:]
    for t, name in ((k, "k"), (v, "v")):
        _need(t, name, q.dtype, dim=dim)
        if t.shape[:-2] != q.shape[:-2] or t.shape[-1] != d:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, q has {tuple(q.shape)}")
    kv = k.shape[-2]
    if v.shape[-2] != kv:
        raise ValueError(f"k has {kv} heads, v has {v.shape[-2]}")
    if kv < 1 or heads % kv:
        raise ValueError(f"{heads} query heads cannot share {kv} key/value heads")
    n_docs = q.shape[0]
    if doc_offsets is not None:
        _need(doc_offsets, "doc_offsets", torch.int64, dim=1)
        if doc_offsets.numel() < 1:
            raise ValueError("doc_offsets needs n_docs + 1 >= 1 entries")
        if doc_lens is not None:
            raise ValueError("give doc_offsets or doc_lens, not both")
        n_docs = doc_offsets.numel() - 1
    _need(doc_lens, "doc_lens", torch.int32, shape=(n_docs,))
    if prefix_lens is not None and not causal:
        raise ValueError("prefix_lens needs causal")
    _need(prefix_lens, "prefix_lens", torch.int32, shape=(n_docs,))
    _need(slopes, "slopes", torch.float32, shape=(heads,))
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if t.stride(-1) != 1:
            raise ValueError(f"{name} needs the entries of a head side by side")
        _on(t, name, q.get_device())
    raise ValueError("the arguments of the attention do not fit together")


def _fits(t, dtype, shape) -> bool:
    return t is None or (t.dtype == dtype and t.shape == shape)


def _attention_desc(q, k, v, doc_offsets, doc_lens, causal, prefix_lens, softcap, slopes, scale):
    """(the library's description of an attention call, heads, rows, device number), with the checks
    that the library cannot make: all in one condition, told apart only where it fails."""
    sq, sk, dt, at = q.shape, k.shape, q.dtype, q.get_device()
    tq, tk, tv = q.stride(), k.stride(), v.stride()
    heads, d, kv = sq[-2], sq[-1], sk[-2]
    scale = d ** -0.5 if scale is None else float(scale)
    softcap = float(softcap or 0.0)
    if not 0 < scale < math.inf:
        raise ValueError(f"scale must be positive and finite, got {scale}")
    if not 0 <= softcap < math.inf:
        raise ValueError(f"softcap must be finite and not negative, got {softcap}")
    if doc_offsets is not None:
        docs, nd, rows, dim = doc_offsets.numel() - 1, 0, sq[0], 3
        known = doc_lens is None and docs >= 0 and doc_offsets.dtype == torch.int64 and \
            doc_offsets.dim() == 1
    else:
        docs, nd, dim = sq[0], sq[1], 4
        rows = docs * nd
        known = _fits(doc_lens, torch.int32, (docs,))
    if not (known and dt in _TORCH_DTYPE and k.dtype == dt and v.dtype == dt and len(sq) == dim
            and sk == v.shape and sk[:-2] == sq[:-2] and sk[-1] == d and kv and heads % kv == 0
            and tq[-1] == 1 and tk[-1] == 1 and tv[-1] == 1 and at >= 0 and k.get_device() == at
            and v.get_device() == at and (prefix_lens is None or causal)
            and _fits(prefix_lens, torch.int32, (docs,)) and _fits(slopes, torch.float32, (heads,))):
        _attention_refuse(q, k, v, doc_offsets, doc_lens, causal, prefix_lens, slopes)
    return _ATTENTION_DESC.pack(
        q.data_ptr(), tq[-3], tq[-2], tq[0], k.data_ptr(), tk[-3], tk[-2], tk[0],
        v.data_ptr(), tv[-3], tv[-2], tv[0], _at(doc_offsets, "doc_offsets", at) or 0,
        _at(doc_lens, "doc_lens", at) or 0, rows, docs, _at(prefix_lens, "prefix_lens", at) or 0,
        _at(slopes, "slopes", at) or 0, nd, heads, kv, d, _TORCH_DTYPE[dt], 1 if causal else 0,
        softcap, scale), heads, rows, at


def maxsim_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                     doc_offsets: torch.Tensor | None = None,
                     doc_lens: torch.Tensor | None = None, causal: bool = False,
                     prefix_lens: torch.Tensor | None = None, softcap: float = 0.0,
                     slopes: torch.Tensor | None = None, scale: float | None = None, out=None,
                     lse=None, stream=None):
    """Attention within documents. Packed: q [n_tokens, n_heads, d], k and v [n_tokens,
    n_kv_heads, d] with doc_offsets int64 [n_docs + 1]; fixed: q [n_docs, nd, n_heads, d], k and
    v alike, with optional doc_lens int32 [n_docs] (tokens past a length are padding). Any
    strides with the entries of a head side by side and 16-byte steps. causal: a token sees the
    ones up to itself and those below its document's prefix_lens (int32 [n_docs]); softcap:
    scores become softcap * tanh(score / softcap); slopes (fp32 [n_heads]): slope * |i - j| is
    taken off; scale: d ** -0.5 unless given. Returns (o shaped like q, lse fp32 [n_heads,
    tokens])."""
    desc, heads, rows, at = _attention_desc(q, k, v, doc_offsets, doc_lens, causal, prefix_lens,
                                            softcap, slopes, scale)
    if out is None:
        out = _like(q, stream)
    else:
        _need(out, "out", q.dtype, shape=q.shape)
    if lse is None:
        lse = q.new_empty((heads, rows), dtype=torch.float32) if stream is None else \
            _new((heads, rows), torch.float32, q.device, stream)
    else:
        _need(lse, "lse", torch.float32, shape=(heads, rows))
    _check(lib().maxsim_attention(desc, _at(out, "out", at), _at(lse, "lse", at),
                                  _stream_at(stream, at)), "maxsim_attention")
    return out, lse


def attention_backward_workspace_size(n_tokens: int, n_heads: int) -> int:
    """Bytes of workspace maxsim_attention_backward needs."""
    return int(lib().maxsim_attention_backward_workspace_size(n_tokens, n_heads))


def maxsim_attention_backward(grad_o: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                              v: torch.Tensor, o: torch.Tensor, lse: torch.Tensor,
                              doc_offsets: torch.Tensor | None = None,
                              doc_lens: torch.Tensor | None = None, causal: bool = False,
                              prefix_lens: torch.Tensor | None = None, softcap: float = 0.0,
                              slopes: torch.Tensor | None = None, scale: float | None = None,
                              want_dq: bool = True, want_dkv: bool = True, dq=None, dk=None,
                              dv=None, workspace=None, stream=None):
    """Gradients (dq, dk, dv) of maxsim_attention from its result's gradient grad_o and its
    outputs o and lse; None for what is not wanted. The other arguments are the forward's."""
    desc, heads, rows, at = _attention_desc(q, k, v, doc_offsets, doc_lens, causal, prefix_lens,
                                            softcap, slopes, scale)
    _need(grad_o, "grad_o", q.dtype, shape=q.shape)
    _need(o, "o", q.dtype, shape=q.shape)
    _need(lse, "lse", torch.float32, shape=(heads, rows))
    _need(workspace, "workspace", torch.uint8)

    def grad(g, like, name, want):
        if not want:
            return None
        _need(g, name, like.dtype, shape=like.shape)
        return _like(like, stream) if g is None else g
    dq, dk, dv = grad(dq, q, "dq", want_dq), grad(dk, k, "dk", want_dkv), grad(dv, v, "dv", want_dkv)
    if workspace is None:
        size = attention_backward_workspace_size(rows, heads)
        workspace = q.new_empty(size, dtype=torch.uint8) if stream is None else \
            _new(size, torch.uint8, q.device, stream)
    _check(lib().maxsim_attention_backward(
        desc, _at(o, "o", at), _at(lse, "lse", at), _at(grad_o, "grad_o", at), _at(dq, "dq", at),
        _at(dk, "dk", at), _at(dv, "dv", at), _at(workspace, "workspace", at), workspace.numel(),
        _stream_at(stream, at)), "maxsim_attention_backward")
    return dq, dk, dv


class AttentionFunction(torch.autograd.Function):
    """Differentiable attention: first gradients of q, k and v; the slopes are constants."""

    @staticmethod
    def forward(ctx, q, k, v, doc_offsets, doc_lens, causal, prefix_lens, softcap, slopes, scale):
        o, lse = maxsim_attention(q, k, v, doc_offsets, doc_lens, causal, prefix_lens, softcap,
                                  slopes, scale)
        ctx.save_for_backward(q, k, v, o, lse, doc_offsets, doc_lens, prefix_lens, slopes)
        ctx.causal, ctx.softcap, ctx.scale = causal, softcap, scale
        return o

    @staticmethod
    def backward(ctx, grad):
        q, k, v, o, lse, doc_offsets, doc_lens, prefix_lens, slopes = ctx.saved_tensors
        want_dq = ctx.needs_input_grad[0]
        want_dkv = ctx.needs_input_grad[1] or ctx.needs_input_grad[2]

        def gradients():
            return maxsim_attention_backward(
                grad.contiguous(), q, k, v, o, lse, doc_offsets, doc_lens, ctx.causal, prefix_lens,
                ctx.softcap, slopes, ctx.scale, want_dq=want_dq, want_dkv=want_dkv)
        if torch.is_grad_enabled():
            dq, dk, dv = FirstOrderFunction.apply("attention", gradients, grad, q, k, v)
        else:
            dq, dk, dv = gradients()
        return dq, dk, dv, None, None, None, None, None, None, None


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
              doc_offsets: torch.Tensor | None = None, doc_lens: torch.Tensor | None = None,
              causal: bool = False, prefix_lens: torch.Tensor | None = None,
              softcap: float = 0.0, slopes: torch.Tensor | None = None,
              scale: float | None = None) -> torch.Tensor:
    """maxsim_attention's o, which autograd can differentiate with respect to q, k and v, once: a
    gradient of its gradients is an error."""
    return AttentionFunction.apply(q, k, v, doc_offsets, doc_lens, causal, prefix_lens, softcap,
                                   slopes, scale)


def _must(t, name: str, *a, **k):
    """_need for a tensor that cannot be left out."""
    if t is None:
        raise ValueError(f"{name} must be a torch.Tensor")
    _need(t, name, *a, **k)


def _rows(t: torch.Tensor, name: str):
    """(rows, entries between them) of t [..., d] whose rows lie at one distance from each other."""
    d = t.shape[-1]
    if t.is_contiguous():
        return t.numel() // d, d
    if t.dim() != 2:
        try:
            t = t.view(-1, d)
        except RuntimeError:
            raise ValueError(f"{name} needs rows at one distance from each other") from None
    if t.stride(1) != 1 and d > 1:
        raise ValueError(f"{name} needs the entries of a row side by side")
    return t.shape[0], t.stride(0)


def _chance(dropout: float, rng, call: int) -> float:
    """dropout as a number, with the checks of what belongs to it."""
    if not dropout and rng is None and not call:
        return 0.0
    dropout = float(dropout)
    if not 0 <= dropout <= 1:
        raise ValueError(f"dropout must lie in [0, 1], got {dropout}")
    if dropout and rng is None:
        raise ValueError("dropout needs rng")
    _need(rng, "rng", torch.int64, shape=(2,))
    if not 0 <= call < 1 << 31:
        raise ValueError(f"call must lie in [0, 2^31), got {call}")
    return dropout


def maxsim_dropout(x: torch.Tensor, dropout: float, rng: torch.Tensor, call: int = 0,
                   out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """x / (1 - dropout) where an entry is kept, else 0; x contiguous, of any shape. The mask is made
    from rng (int64 [2] on the device: key and step) and call, and never stored: the same call on a
    gradient of the result is the gradient of x. dropout counts in steps of 2^-16. Raise the step
    from one training step to the next (in place, in a captured one: between replays), and give each
    place that drops a call of its own. out may be x itself."""
    _must(x, "x", _FLOAT_STORAGE)
    if rng is None:
        raise ValueError("dropout needs rng")
    dropout = _chance(dropout, rng, call)
    if out is None:
        out = _like(x, stream)
    else:
        _need(out, "out", x.dtype, shape=x.shape)
    at = x.get_device()
    _check(lib().maxsim_dropout(_at(x, "x", at), x.numel(), _TORCH_DTYPE[x.dtype], dropout,
                                _at(rng, "rng", at), call, _at(out, "out", at),
                                _stream_at(stream, at)), "maxsim_dropout")
    return out


class DropoutFunction(torch.autograd.Function):
    """Differentiable dropout, to any order: it is linear in x."""

    @staticmethod
    def forward(ctx, x, dropout, rng, call):
        ctx.save_for_backward(rng)
        ctx.dropout, ctx.call = dropout, call
        return maxsim_dropout(x, dropout, rng, call)

    @staticmethod
    def backward(ctx, grad):
        drop = DropoutFunction.apply if torch.is_grad_enabled() else maxsim_dropout
        return drop(grad.contiguous(), ctx.dropout, ctx.saved_tensors[0], ctx.call), None, None, None


def dropout(x: torch.Tensor, dropout: float, rng: torch.Tensor, call: int = 0) -> torch.Tensor:
    """maxsim_dropout that autograd can differentiate with respect to x, to any order. Raise the step
    in rng after the backward, which makes the same mask again."""
    return DropoutFunction.apply(x, dropout, rng, call)


def _norm_args(x, weight, residual, eps):
    """(rows, row stride of x, of the residual) of a norm, checked: what most calls are in one
    condition, the others one by one."""
    tensor = torch.Tensor
    if isinstance(x, tensor) and isinstance(weight, tensor):
        shape, dt = x.shape, x.dtype
        if dt in _TORCH_DTYPE and shape and x.is_contiguous() and eps >= 0 and weight.shape == shape[-1:] and \
                (weight.dtype == dt or weight.dtype == torch.float32) and x.numel() and \
                (residual is None or (isinstance(residual, tensor) and residual.dtype == dt and
                                      residual.shape == shape and residual.is_contiguous())):
            return x.numel() // shape[-1], shape[-1], shape[-1]
    _must(x, "x", _FLOAT_STORAGE)
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x needs rows of at least one entry")
    _must(weight, "weight", (x.dtype, torch.float32), shape=x.shape[-1:])
    if not eps >= 0:
        raise ValueError(f"eps must not be negative, got {eps}")
    n, stride = _rows(x, "x")
    if residual is None:
        return n, stride, 0
    _need(residual, "residual", x.dtype, shape=x.shape)
    return n, stride, _rows(residual, "residual")[1]


def maxsim_rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
                    eps: float = 1e-6, dropout: float = 0.0, rng: torch.Tensor | None = None,
                    call: int = 0, out=None, out_h=None, rstd=None, stream=None):
    """h = residual + dropout(x), rounded to x's type (both optional: else h is x), and its root-mean-
    square norm y = h * rstd * weight. x [..., d] and residual alike, rows at one distance from each
    other; weight [d] in x's type or fp32; dropout, rng and call as in maxsim_dropout. Returns (y, h,
    rstd fp32 [...]). out may be x, and out_h the residual, where those are contiguous."""
    n, stride, r_stride = _norm_args(x, weight, residual, eps)
    dropout = _chance(dropout, rng, call)
    dt, at = x.dtype, x.get_device()
    if out is None:
        out = _like(x, stream)
    else:
        _need(out, "out", dt, shape=x.shape)
    h = None
    if residual is not None or dropout:
        if out_h is None:
            h = _like(x, stream)
        else:
            h = out_h
            _need(h, "out_h", dt, shape=x.shape)
    elif out_h is not None:
        raise ValueError("out_h needs a residual or dropout: h is x itself")
    if rstd is None:
        rstd = _beside(x, x.shape[:-1], torch.float32, stream)
    else:
        _need(rstd, "rstd", torch.float32, shape=x.shape[:-1])
    _check(lib().maxsim_rms_norm(
        _on(x, "x", at), stride, None if residual is None else _on(residual, "residual", at),
        r_stride, n, x.shape[-1], _TORCH_DTYPE[dt], _at(weight, "weight", at),
        _TORCH_DTYPE[weight.dtype], eps, dropout, _at(rng, "rng", at), call, _at(out, "out", at),
        _at(h, "out_h", at), _at(rstd, "rstd", at), _stream_at(stream, at)), "maxsim_rms_norm")
    return out, x if h is None else h, rstd


def maxsim_rms_norm_i8(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
                       eps: float = 1e-6, out=None, scale=None, out_h=None, stream=None):
    """maxsim_rms_norm with y in 8 bits, for maxsim_score_i8: returns (codes int8 shaped like x,
    scale fp32 [...], h) with y = codes * scale, scale a row's largest |y| / 127."""
    n, stride, r_stride = _norm_args(x, weight, residual, eps)
    dt, at = x.dtype, x.get_device()
    if out is None:
        out = _beside(x, x.shape, torch.int8, stream)
    else:
        _need(out, "out", torch.int8, shape=x.shape)
    if scale is None:
        scale = _beside(x, x.shape[:-1], torch.float32, stream)
    else:
        _need(scale, "scale", torch.float32, shape=x.shape[:-1])
    h = None
    if residual is not None:
        if out_h is None:
            h = _like(x, stream)
        else:
            h = out_h
            _need(h, "out_h", dt, shape=x.shape)
    elif out_h is not None:
        raise ValueError("out_h needs a residual: h is x itself")
    _check(lib().maxsim_rms_norm_i8(
        _on(x, "x", at), stride, None if residual is None else _on(residual, "residual", at),
        r_stride, n, x.shape[-1], _TORCH_DTYPE[dt], _at(weight, "weight", at),
        _TORCH_DTYPE[weight.dtype], eps, _at(out, "out", at), _at(scale, "scale", at),
        _at(h, "out_h", at), _stream_at(stream, at)), "maxsim_rms_norm_i8")
    return out, scale, x if h is None else h


def rms_norm_backward_workspace_size(n_rows: int, d: int) -> int:
    """Bytes of workspace maxsim_rms_norm_backward needs for the weight's gradient."""
    return int(lib().maxsim_rms_norm_backward_workspace_size(n_rows, d))


def maxsim_rms_norm_backward(grad_y: torch.Tensor, h: torch.Tensor, weight: torch.Tensor,
                             rstd: torch.Tensor, grad_h: torch.Tensor | None = None,
                             dropout: float = 0.0, rng: torch.Tensor | None = None, call: int = 0,
                             want_dx: bool = True, want_dresidual: bool = True,
                             want_dweight: bool = True, dx=None, dresidual=None, dweight=None,
                             workspace=None, stream=None):
    """Gradients (dx, dresidual, dweight) of maxsim_rms_norm, from those of its y and (optionally) h
    and its outputs h and rstd; None for what is not wanted. Without dropout dx and dresidual are
    one tensor, unless two are given."""
    n, stride, _ = _norm_args(h, weight, None, 0.0)
    dropout = _chance(dropout, rng, call)
    dt, at = h.dtype, h.get_device()
    _must(grad_y, "grad_y", dt, shape=h.shape)
    _need(grad_h, "grad_h", dt, shape=h.shape)
    _must(rstd, "rstd", torch.float32, shape=h.shape[:-1])
    _need(dx, "dx", dt, shape=h.shape)
    _need(dresidual, "dresidual", dt, shape=h.shape)
    _need(dweight, "dweight", weight.dtype, shape=weight.shape)
    _need(workspace, "workspace", torch.uint8)
    for t, name in ((grad_y, "grad_y"), (grad_h, "grad_h"), (weight, "weight"), (rstd, "rstd"), (rng, "rng"),
                    (dx, "dx"), (dresidual, "dresidual"), (dweight, "dweight"), (workspace, "workspace")):
        _at(t, name, at)
    _on(h, "h", at)
    return _norm_gradients(grad_y, grad_h, h, n, stride, weight, rstd, dropout, rng, call, want_dx,
                           want_dresidual, want_dweight, dx, dresidual, dweight, workspace, stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _norm_gradients(grad_y, grad_h, h, n, stride, weight, rstd, dropout, rng, call, want_dx, want_dresidual,
                    want_dweight, dx=None, dresidual=None, dweight=None, workspace=None, stream=None):
    """maxsim_rms_norm_backward without its checks."""
    d, size = h.shape[-1], 0
    one = want_dx and want_dresidual and not dropout and (dx is None or dresidual is None)
    if one:
        dx = dresidual = dx if dx is not None else dresidual
    dx, dresidual, dweight = (dx if want_dx else None, dresidual if want_dresidual else None,
                              dweight if want_dweight else None)
    if want_dresidual and dresidual is None:
        dresidual = _like(h, stream)
    if one:
        dx = dresidual
    elif want_dx and dx is None:
        dx = _like(h, stream)
    if want_dweight:
        if dweight is None:
            dweight = _like(weight, stream)
        if workspace is None:
            workspace = _beside(h, (rms_norm_backward_workspace_size(n, d),), torch.uint8, stream)
        size = workspace.numel()
    _check(lib().maxsim_rms_norm_backward(
        grad_y.data_ptr(), _ptr(grad_h), h.data_ptr(), stride, n, d, _TORCH_DTYPE[h.dtype],
        weight.data_ptr(), _TORCH_DTYPE[weight.dtype], rstd.data_ptr(), dropout, _ptr(rng), call,
        None if one else _ptr(dx), _ptr(dresidual), _ptr(dweight), _ptr(workspace), size,
        _stream_at(stream, h.get_device())), "maxsim_rms_norm_backward")
    return dx, dresidual, dweight


class RmsNormFunction(torch.autograd.Function):
    """Differentiable norm: first gradients of x, the residual and the weight."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps, dropout, rng, call):
        y, h, rstd = maxsim_rms_norm(x, weight, residual, eps, dropout, rng, call)
        ctx.save_for_backward(h, weight, rstd, rng)
        ctx.dropout, ctx.call = dropout, call
        ctx.set_materialize_grads(False)
        return y if h is x else (y, h)

    @staticmethod
    def backward(ctx, grad_y, grad_h=None):
        h, weight, rstd, rng = ctx.saved_tensors
        if grad_y is None and grad_h is None:
            return None, None, None, None, None, None, None
        want_dx, want_dw, want_dr = ctx.needs_input_grad[:3]
        n, stride = _rows(h, "h")

        def gradients():
            dy = torch.zeros_like(h, memory_format=torch.contiguous_format) if grad_y is None else grad_y
            return _norm_gradients(dy.contiguous(), None if grad_h is None else grad_h.contiguous(), h, n,
                                   stride, weight, rstd, ctx.dropout, rng, ctx.call, want_dx, want_dr,
                                   want_dw)

        def apart():
            dx, dr, dw = gradients()
            return dx, dr.clone() if dr is dx and dr is not None else dr, dw
        if torch.is_grad_enabled():
            dx, dr, dw = FirstOrderFunction.apply("rms_norm", apart, grad_y, grad_h, h, weight)
        else:
            dx, dr, dw = gradients()
        return dx, dw, dr, None, None, None, None


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
             eps: float = 1e-6, dropout: float = 0.0, rng: torch.Tensor | None = None, call: int = 0):
    """maxsim_rms_norm's (y, h), which autograd can differentiate with respect to x, weight and
    residual, once: a gradient of its gradients is an error. Raise the step in rng after the
    backward, which makes the same mask again."""
    if residual is None and not dropout:
        return RmsNormFunction.apply(x, weight, None, eps, 0.0, None, 0), x
    return RmsNormFunction.apply(x, weight, residual, eps, dropout, rng, call)


def linear_cross_entropy_workspace_size(n_rows: int, vocab: int, d: int, dtype: torch.dtype) -> int:
    """Bytes of workspace maxsim_linear_cross_entropy needs."""
    return int(lib().maxsim_linear_cross_entropy_workspace_size(n_rows, vocab, d, _TORCH_DTYPE[dtype]))


def linear_cross_entropy_backward_workspace_size(n_rows: int, vocab: int, d: int,
                                                 dtype: torch.dtype) -> int:
    """Bytes of workspace maxsim_linear_cross_entropy_backward needs."""
    return int(lib().maxsim_linear_cross_entropy_backward_workspace_size(n_rows, vocab, d,
                                                                         _TORCH_DTYPE[dtype]))


def _loss_args(h, w, labels, scale):
    _must(h, "h", _FLOAT_STORAGE, dim=2)
    _must(w, "w", h.dtype, dim=2)
    if w.shape[1] != h.shape[1]:
        raise ValueError(f"w has d = {w.shape[1]}, h has d = {h.shape[1]}")
    if w.shape[0] < 1:
        raise ValueError("w needs at least one row")
    _must(labels, "labels", torch.int64, shape=h.shape[:1])
    scale = float(scale)
    if not 0 < scale < math.inf:
        raise ValueError(f"scale must be positive and finite, got {scale}")
    return h.shape[0], w.shape[0], h.shape[1], scale, h.get_device()


def maxsim_linear_cross_entropy(h: torch.Tensor, w: torch.Tensor, labels: torch.Tensor,
                                scale: float = 1.0, loss=None, lse=None, workspace=None, stream=None):
    """Softmax cross entropy of the logits scale * h w^T over a vocabulary, which are not kept. h
    [n_rows, d], w [vocab, d] (same type; rows of whole 16 bytes), labels int64 [n_rows]; a row whose
    label lies outside the vocabulary is left out: loss 0, lse -inf, and no work. Returns (loss, lse)
    fp32 [n_rows]."""
    n, vocab, d, scale, at = _loss_args(h, w, labels, scale)
    if loss is None:
        loss = _beside(h, (n,), torch.float32, stream)
    else:
        _need(loss, "loss", torch.float32, shape=(n,))
    if lse is None:
        lse = _beside(h, (n,), torch.float32, stream)
    else:
        _need(lse, "lse", torch.float32, shape=(n,))
    if workspace is None:
        size = linear_cross_entropy_workspace_size(n, vocab, d, h.dtype)
        workspace = _beside(h, (size,), torch.uint8, stream)
    else:
        _need(workspace, "workspace", torch.uint8)
    _check(lib().maxsim_linear_cross_entropy(
        _at(h, "h", at), _at(w, "w", at), _at(labels, "labels", at), n, vocab, d,
        _TORCH_DTYPE[h.dtype], scale, _at(loss, "loss", at), _at(lse, "lse", at),
        _at(workspace, "workspace", at), workspace.numel(), _stream_at(stream, at)),
        "maxsim_linear_cross_entropy")
    return loss, lse


def maxsim_linear_cross_entropy_backward(grad_loss: torch.Tensor, h: torch.Tensor, w: torch.Tensor,
                                         labels: torch.Tensor, lse: torch.Tensor, scale: float = 1.0,
                                         want_dh: bool = True, want_dw: bool = True, dh=None, dw=None,
                                         workspace=None, stream=None):
    """Gradients (dh, dw) of maxsim_linear_cross_entropy's losses from theirs (fp32 [n_rows]) and its
    lse; None for what is not wanted. The vocabulary goes in pieces, of which the workspace holds
    one."""
    n, vocab, d, scale, at = _loss_args(h, w, labels, scale)
    _must(grad_loss, "grad_loss", torch.float32, shape=(n,))
    _must(lse, "lse", torch.float32, shape=(n,))
    if dh is not None:
        _need(dh, "dh", h.dtype, shape=h.shape)
    elif want_dh:
        dh = _like(h, stream)
    if dw is not None:
        _need(dw, "dw", w.dtype, shape=w.shape)
    elif want_dw:
        dw = _like(w, stream)
    _need(workspace, "workspace", torch.uint8)
    if workspace is None:
        size = linear_cross_entropy_backward_workspace_size(n, vocab, d, h.dtype)
        workspace = _beside(h, (size,), torch.uint8, stream)
    dh, dw = dh if want_dh else None, dw if want_dw else None
    _check(lib().maxsim_linear_cross_entropy_backward(
        _at(grad_loss, "grad_loss", at), _at(h, "h", at), _at(w, "w", at), _at(labels, "labels", at),
        _at(lse, "lse", at), n, vocab, d, _TORCH_DTYPE[h.dtype], scale, _at(dh, "dh", at),
        _at(dw, "dw", at), _at(workspace, "workspace", at), workspace.numel(),
        _stream_at(stream, at)), "maxsim_linear_cross_entropy_backward")
    return dh, dw


class LinearCrossEntropyFunction(torch.autograd.Function):
    """Differentiable cross entropy: first gradients of h and w."""

    @staticmethod
    def forward(ctx, h, w, labels, scale):
        loss, lse = maxsim_linear_cross_entropy(h, w, labels, scale)
        ctx.save_for_backward(h, w, labels, lse)
        ctx.scale = scale
        return loss

    @staticmethod
    def backward(ctx, grad):
        h, w, labels, lse = ctx.saved_tensors
        want_dh, want_dw = ctx.needs_input_grad[:2]

        def gradients():
            return maxsim_linear_cross_entropy_backward(grad.contiguous(), h, w, labels, lse,
                                                        ctx.scale, want_dh, want_dw)
        if torch.is_grad_enabled():
            dh, dw = FirstOrderFunction.apply("linear_cross_entropy", gradients, grad, h, w)
        else:
            dh, dw = gradients()
        return dh, dw, None, None


def linear_cross_entropy(h: torch.Tensor, w: torch.Tensor, labels: torch.Tensor,
                         scale: float = 1.0) -> torch.Tensor:
    """maxsim_linear_cross_entropy's losses [n_rows], which autograd can differentiate with respect to
    h and w, once: a gradient of its gradients is an error."""
    return LinearCrossEntropyFunction.apply(h, w, labels, scale)


def clip_grad_norm_workspace_size(n_tensors: int) -> int:
    """Bytes of workspace maxsim_clip_grad_norm needs."""
    return int(lib().maxsim_clip_grad_norm_workspace_size(n_tensors))


_DTYPE_OF = operator.attrgetter("dtype")


def maxsim_clip_grad_norm(grads, max_norm: float, out=None, norm: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Scales a list of gradients (contiguous bf16, fp16 or fp32 tensors, mixed as they come) by
    min(1, max_norm / (norm + 1e-6)), norm their global 2-norm. In place, or into the list `out`
    of tensors like them. Entries of None (parameters without a gradient) are left out. Returns the
    norm before clipping, an fp32 scalar on the device."""
    grads = list(grads)
    outs = grads if out is None else list(out)
    if len(outs) != len(grads):
        raise ValueError(f"out holds {len(outs)} tensors, grads {len(grads)}")
    if not grads:
        raise ValueError("grads must hold at least one tensor")
    max_norm = float(max_norm)
    if not max_norm >= 0:
        raise ValueError(f"max_norm must not be negative, got {max_norm}")
    each = grads if out is None else grads + outs
    # whole lists at a time: an encoder has hundreds of gradients
    try:
        dtypes = set(map(_DTYPE_OF, each))
    except AttributeError:  # some entry is no tensor: those without a gradient are left out
        given = [(g, o) for g, o in zip(grads, outs) if g is not None]
        if len(given) == len(grads):
            raise ValueError("every entry must be a tensor, or None among the gradients") from None
        return maxsim_clip_grad_norm([g for g, _ in given], max_norm,
                                     None if out is None else [o for _, o in given], norm, workspace,
                                     stream)
    if not dtypes <= _TORCH_DTYPE.keys():
        raise ValueError(f"unsupported dtype among {dtypes}")
    if not all(map(torch.Tensor.is_contiguous, each)):
        raise ValueError("every tensor must be contiguous")
    devices = set(map(torch.Tensor.get_device, each))
    if len(devices) != 1 or -1 in devices:
        raise ValueError("every tensor must be a device tensor, all on one device")
    n, at = len(grads), devices.pop()
    code = array("i", [_TORCH_DTYPE[t] for t in map(_DTYPE_OF, grads)])
    numel = array("q", map(torch.Tensor.numel, grads))
    if out is not None and (list(map(_DTYPE_OF, outs)) != list(map(_DTYPE_OF, grads)) or
                            list(map(torch.Tensor.numel, outs)) != list(numel)):
        raise ValueError("out must hold tensors of the gradients' dtypes and sizes")
    ptrs = array("Q", map(torch.Tensor.data_ptr, each))
    if norm is None:
        norm = _new((), torch.float32, grads[0].device, stream)
    else:
        _need(norm, "norm", torch.float32, numel=1)
    if workspace is None:
        workspace = _new(clip_grad_norm_workspace_size(n), torch.uint8, grads[0].device, stream)
    else:
        _need(workspace, "workspace", torch.uint8)
    src = ptrs.buffer_info()[0]
    _check(lib().maxsim_clip_grad_norm(
        src, None if out is None else src + 8 * n, numel.buffer_info()[0], code.buffer_info()[0], n,
        max_norm, _at(norm, "norm", at), _at(workspace, "workspace", at), workspace.numel(),
        _stream_at(stream, at)), "maxsim_clip_grad_norm")
    return norm


def maxsim_quantize_mx4(x: torch.Tensor, codes=None, scales=None, stream=None):
    """Token vectors x [..., d] in microscaled 4-bit floating point: 32 entries share a power of two,
    each is a sign and one of 0, 1/2, 1, 3/2, 2, 3, 4, 6. Returns (codes uint8 [..., d / 2], two
    entries a byte, the first in the low half; scales uint8 [..., d / 32], exponents plus 127)."""
    _must(x, "x", _FLOAT_STORAGE)
    d = x.shape[-1] if x.dim() else 0
    if d < 32 or d % 32:
        raise ValueError(f"x needs rows of whole 32 entries, got shape {tuple(x.shape)}")
    rows = x.shape[:-1]
    if codes is None:
        codes = _beside(x, (*rows, d // 2), torch.uint8, stream)
    else:
        _need(codes, "codes", torch.uint8, shape=(*rows, d // 2))
    if scales is None:
        scales = _beside(x, (*rows, d // 32), torch.uint8, stream)
    else:
        _need(scales, "scales", torch.uint8, shape=(*rows, d // 32))
    at = x.get_device()
    _check(lib().maxsim_quantize_mx4(
        _at(x, "x", at), x.numel() // d, d, _TORCH_DTYPE[x.dtype], _at(codes, "codes", at),
        _at(scales, "scales", at), _stream_at(stream, at)), "maxsim_quantize_mx4")
    return codes, scales


def _mx4(codes, scales, names, dim=None):
    """d of stored vectors, checked."""
    _must(codes, names[0], torch.uint8, dim=dim)
    if not codes.dim() or codes.shape[-1] < 16 or codes.shape[-1] % 16:
        raise ValueError(f"{names[0]} needs rows of whole 16 bytes, got shape {tuple(codes.shape)}")
    _must(scales, names[1], torch.uint8, shape=(*codes.shape[:-1], codes.shape[-1] // 16))
    return codes.shape[-1] * 2


def maxsim_dequantize_mx4(codes: torch.Tensor, scales: torch.Tensor, dtype=torch.float32, out=None,
                          stream=None) -> torch.Tensor:
    """The values [..., d] that codes and scales from maxsim_quantize_mx4 stand for, in dtype."""
    d = _mx4(codes, scales, ("codes", "scales"))
    if dtype not in _TORCH_DTYPE:
        raise ValueError(f"unsupported dtype {dtype}")
    shape = (*codes.shape[:-1], d)
    if out is None:
        out = _beside(codes, shape, dtype, stream)
    else:
        _need(out, "out", dtype, shape=shape)
    at = codes.get_device()
    _check(lib().maxsim_dequantize_mx4(
        _at(codes, "codes", at), _at(scales, "scales", at), out.numel() // d, d, _TORCH_DTYPE[dtype],
        _at(out, "out", at), _stream_at(stream, at)), "maxsim_dequantize_mx4")
    return out


def maxsim_score_mx4(Q: torch.Tensor, q_scale: torch.Tensor, D: torch.Tensor, d_scale: torch.Tensor,
                     doc_offsets: torch.Tensor | None = None, doc_lens: torch.Tensor | None = None,
                     out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Scores of microscaled 4-bit queries and documents (maxsim_quantize_mx4). Q [q_len, d / 2] with
    q_scale [q_len, d / 32]; fixed documents D [n_docs, nd, d / 2] with d_scale alike, of which
    doc_lens (int32 [n_docs]) tokens count, or with doc_offsets CSR D [n_tokens, d / 2]. Returns fp32
    scores [n_docs]."""
    d = _mx4(Q, q_scale, ("Q", "q_scale"), dim=2)
    if _mx4(D, d_scale, ("D", "d_scale"), dim=3 if doc_offsets is None else 2) != d:
        raise ValueError(f"D has d = {2 * D.shape[-1]}, Q has d = {d}")
    if doc_offsets is not None:
        _need(doc_offsets, "doc_offsets", torch.int64, dim=1)
        if doc_offsets.numel() < 1:
            raise ValueError("doc_offsets needs n_docs + 1 >= 1 entries")
        if doc_lens is not None:
            raise ValueError("give doc_offsets or doc_lens, not both")
    n_docs, nd = _docs(D, doc_offsets)
    _need(doc_lens, "doc_lens", torch.int32, shape=(n_docs,))
    out = _out(out, n_docs, Q.device, stream)
    at = Q.get_device()
    at_D, at_scale = _at(D, "D", at), _at(d_scale, "d_scale", at)
    if doc_offsets is not None and not D.numel():
        # documents without a token: an empty tensor has no address, and none is read
        at_D, at_scale = Q.data_ptr(), q_scale.data_ptr()
    _check(lib().maxsim_score_mx4(
        _at(Q, "Q", at), _at(q_scale, "q_scale", at), Q.shape[0], at_D,
        at_scale, _at(doc_offsets, "doc_offsets", at), n_docs, nd,
        _at(doc_lens, "doc_lens", at), d, _at(out, "out", at), _stream_at(stream, at)),
        "maxsim_score_mx4")
    return out


def version() -> int:
    return lib().maxsim_version()


# ---- measurement helpers (include/maxsim_calib.h) ----

def _calib_lib():
    L = lib()
    if not getattr(L, "_calib_bound", False):
        vp = ctypes.c_void_p
        L.maxsim_calib_read.argtypes = [vp, ctypes.c_size_t, ctypes.c_int, vp, vp]
        L.maxsim_calib_copy.argtypes = [vp, vp, ctypes.c_size_t, vp]
        L.maxsim_calib_write.argtypes = [vp, ctypes.c_size_t, ctypes.c_int, ctypes.c_int, vp]
        L.maxsim_calib_write.restype = ctypes.c_int
        L.maxsim_calib_mfma.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, vp, vp, vp]
        L.maxsim_calib_read.restype = ctypes.c_int
        L.maxsim_calib_copy.restype = ctypes.c_int
        L.maxsim_calib_mfma.restype = ctypes.c_int
        L.maxsim_calib_valu.argtypes = [ctypes.c_int, ctypes.c_int, vp, vp, vp]
        L.maxsim_calib_valu.restype = ctypes.c_int
        L.maxsim_calib_mix.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, vp, vp, vp]
        L.maxsim_calib_mix.restype = ctypes.c_int
        L.maxsim_calib_lds.argtypes = [ctypes.c_int, ctypes.c_int, vp, vp, vp]
        L.maxsim_calib_lds.restype = ctypes.c_int
        L._calib_bound = True
    return L


def calib_read(src: torch.Tensor, sink: torch.Tensor, stream=None, wgs_per_cu: int = 1):
    """Stream-read every byte of src (achievable read bandwidth) with wgs_per_cu workgroups
    of 4 waves per CU (0: as many as fit); sink: >= 65536 words."""
    _check(_calib_lib().maxsim_calib_read(_dev(src, "src"), src.numel() * src.element_size(),
                                          int(wgs_per_cu), _dev(sink, "sink"), _stream(stream)),
           "maxsim_calib_read")


def calib_write(dst: torch.Tensor, stream=None, wgs_per_cu: int = 2, contig: bool = True):
    """Stream a fixed pattern into every byte of dst (achievable write bandwidth) with
    wgs_per_cu workgroups of 4 waves per CU (0: as many as fit), each wave writing one
    contiguous range (contig) or blocks dealt in turn."""
    _check(_calib_lib().maxsim_calib_write(_dev(dst, "dst"), dst.numel() * dst.element_size(),
                                           int(wgs_per_cu), int(bool(contig)), _stream(stream)),
           "maxsim_calib_write")


def calib_copy(src: torch.Tensor, dst: torch.Tensor, stream=None):
    """Plain 128-bit copy of src into dst (known traffic for counter scaling)."""
    _check(_calib_lib().maxsim_calib_copy(_dev(src, "src"), _dev(dst, "dst"),
                                          src.numel() * src.element_size(), _stream(stream)),
           "maxsim_calib_copy")


def calib_mfma(kind: int, iters: int, waves_per_simd: int, sink: torch.Tensor, stream=None) -> float:
    """Launch independent MFMA chains (kind 0: 16x16x32 bf16, 1: 32x32x16 bf16, 2: 16x16x64
    int8, 3: 32x32x32 int8); returns the FLOP / integer-op count of the launch."""
    ops = ctypes.c_double(0.0)
    _check(_calib_lib().maxsim_calib_mfma(kind, iters, waves_per_simd, _dev(sink, "sink"),
                                          ctypes.addressof(ops), _stream(stream)),
           "maxsim_calib_mfma")
    return ops.value


def calib_valu(iters: int, waves_per_simd: int, sink: torch.Tensor, stream=None) -> float:
    """Launch independent fp32 FMA chains; returns the FLOP count of the launch."""
    ops = ctypes.c_double(0.0)
    _check(_calib_lib().maxsim_calib_valu(iters, waves_per_simd, _dev(sink, "sink"),
                                          ctypes.addressof(ops), _stream(stream)), "maxsim_calib_valu")
    return ops.value


def calib_mix(valu_per_mfma: int, iters: int, waves_per_simd: int, sink: torch.Tensor,
              stream=None) -> float:
    """Launch int8 MFMA chains with valu_per_mfma independent FMAs per MFMA; returns the
    int8 integer-op count of the launch."""
    ops = ctypes.c_double(0.0)
    _check(_calib_lib().maxsim_calib_mix(valu_per_mfma, iters, waves_per_simd, _dev(sink, "sink"),
                                         ctypes.addressof(ops), _stream(stream)), "maxsim_calib_mix")
    return ops.value


def calib_lds(pattern: int, iters: int, sink: torch.Tensor, stream=None) -> float:
    """Launch the LDS read-rate kernel (0: contiguous, 1: PQ lookups); returns LDS bytes read."""
    b = ctypes.c_double(0.0)
    _check(_calib_lib().maxsim_calib_lds(pattern, iters, _dev(sink, "sink"), ctypes.addressof(b),
                                         _stream(stream)), "maxsim_calib_lds")
    return b.value
