"""Thin Python binding of the C ABI in ``include/nvfp4.h`` (ctypes over ``libnvfp4.so``).

Each ``nvfp4_*`` function here has the name and arguments of the C entry point, with torch
tensors in place of device pointers; it only checks that tensors live on the GPU with the
expected dtype, contiguity and size, passes their pointers and the current torch stream, and
raises ``Nvfp4Error`` on a non-OK status. Every computation runs in the library's HIP kernels;
there is no CPU path. Importing this module fails if the library has not been built
(``python -m block_scale_search_amd.build``).

The convenience wrappers at the end (``diag_hessian``, ``layer_statistics``, ``global_scale``,
``scale_search``, ``scale_search_rules``, ``scale_search_proposal``, ``pack``, ``quantize_activations``, ``gptq``,
``output_error``) allocate outputs and workspaces with torch and call the entry points.
``Matrix`` describes quantised matrices; ``linear``, ``gated`` and their ``_backward`` multiply by them.
``KVCache`` describes a paged key/value cache; the ``kv_*`` wrappers take one and a layer.
"""
from __future__ import annotations

import ctypes
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libnvfp4.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"{_LIB_PATH} is missing: build it with `python -m block_scale_search_amd.build`")
_lib = ctypes.CDLL(_LIB_PATH)

OK, ERR_NULL, ERR_SHAPE, ERR_DTYPE, ERR_ALIGN, ERR_WINDOW, ERR_ARG, ERR_WORKSPACE, ERR_HIP = range(9)
DTYPE_F32, DTYPE_BF16 = 0, 1
MSE, WMSE = 0, 1
GS_AMAX_448, GS_AMAX_256 = 0, 1
ACT_NONE, ACT_SILU, ACT_GELU, ACT_GELU_TANH, ACT_RELU = range(5)

_P, _I64, _I32, _I, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int, ctypes.c_size_t

class SearchRule(ctypes.Structure):
    """``nvfp4_search_rule``: one objective and window with its output pointers."""
    _fields_ = [("objective", ctypes.c_int32), ("lo", ctypes.c_int32), ("hi", ctypes.c_int32),
                ("exhaustive", ctypes.c_int32), ("scales", ctypes.c_void_p),
                ("packed", ctypes.c_void_p), ("loss", ctypes.c_void_p),
                ("offset", ctypes.c_void_p)]


class MatrixStruct(ctypes.Structure):
    """``nvfp4_matrix``."""
    _fields_ = [("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("S", ctypes.c_void_p),
                ("batch", _I64), ("out", _I64), ("in_", _I64), ("stride", _I64)]


class KVCacheStruct(ctypes.Structure):
    """``nvfp4_kv_cache``."""
    _fields_ = [("pages", ctypes.c_void_p), ("layers", _I64), ("layer_stride", _I64),
                ("num_pages", _I64), ("page_stride", _I64), ("heads", _I32), ("head_dim", _I32),
                ("page_size", _I32), ("max_pages", _I32), ("max_slots", _I64),
                ("table", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("refs", ctypes.c_void_p),
                ("S_k", ctypes.c_void_p), ("S_v", ctypes.c_void_p)]


_SIGS = {
    "nvfp4_status_string": ([_I], ctypes.c_char_p),
    "nvfp4_version": ([], ctypes.c_char_p),
    "nvfp4_diag_hessian_workspace_size": ([_I64, _I64, _I64], _SZ),
    "nvfp4_diag_hessian": ([_P, _I, _I64, _I64, _I64, _P, _P, _I, _P, _SZ, _P], _I),
    "nvfp4_diag_hessian_finalize": ([_I, _I64, _I64, _P, _P, _I, _P, _SZ, _P], _I),
    "nvfp4_diag_hessian_batched": ([_P, _I, _P, _I64, _I64, _I64, _I64, _P, _P, _I, _P, _SZ, _P], _I),
    "nvfp4_diag_hessian_chunks_workspace_size": ([_P, _I64, _I64], _SZ),
    "nvfp4_diag_hessian_chunks": ([_P, _I, _P, _I64, _I64, _I64, _P, _P, _I, _P, _SZ, _P], _I),
    "nvfp4_global_scale_workspace_size": ([_I64, _I64, _I64], _SZ),
    "nvfp4_global_scale": ([_P, _I, _I64, _I64, _I64, _I64, _I64, _I, _P, _P, _SZ, _P], _I),
    "nvfp4_layer_statistics_workspace_size": ([_I64, _I64, _I64], _SZ),
    "nvfp4_layer_statistics": ([_P, _I, _I64, _I64, _I64, _P, _P, _I, _P, _I, _I64, _I64, _I, _P,
                                _P, _SZ, _P], _I),
    "nvfp4_scale_search": ([_P, _I, _I64, _I64, _I64, _I64, _I64, _I32, _P, _I64, _I, _I32, _I32, _I,
                            _P, _P, _P, _P, _P, _P], _I),
    "nvfp4_scale_search_rules": ([_P, _I, _I64, _I64, _I64, _I64, _I64, _I32, _P, _I64, _P,
                                  ctypes.POINTER(SearchRule), _I32, _P], _I),
    "nvfp4_scale_search_scored": ([_P, _I, _I64, _I64, _I64, _I64, _I64, _I32, _P, _I64, _I, _I32,
                                   _P, _P, _P], _I),
    "nvfp4_scale_search_proposal": ([_P, _I, _I64, _I64, _I64, _I64, _I64, _I32, _P, _I64, _I,
                                     _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P], _I),
    "nvfp4_pack": ([_P, _I, _I64, _I64, _I64, _I64, _I64, _P, _P, _P, _P], _I),
    "nvfp4_quantize_activations_workspace_size": ([_I64, _I64], _SZ),
    "nvfp4_quantize_activations": ([_P, _I, _I64, _I64, _I64, _I, _P, _I32, _I32, _I, _P, _P, _P,
                                    _P, _SZ, _P], _I),
    "nvfp4_quantize_activations_noalloc": ([_P, _I, _I64, _I64, _I64, _I, _P, _I32, _I32, _I,
                                            _P, _P, _P, _P], _I),
    "nvfp4_gptq_workspace_size": ([_I64, _I64], _SZ),
    "nvfp4_gptq": ([_P, _I, _I64, _I64, _I64, _P, _P, _I, _I32, _I32, _P, _P, _P, _P, _P, _SZ,
                    _P], _I),
    "nvfp4_output_error_workspace_size": ([_I64, _I64, _I64], _SZ),
    "nvfp4_output_error": ([_P, _I, _I64, _I64, _I64, _P, _I, _I64, _I64, _P, _P, _P, _P, _I,
                            _P, _SZ, _P], _I),
    "nvfp4_linear_workspace_size": ([_I, _I64, _I64, _I64, _I64], _SZ),
    "nvfp4_linear": ([_P, _P, _I, _I64, _I64, _P, _P, _I, _P, _I64, _P, _I64, _P, _I64, _P, _SZ, _P], _I),
    "nvfp4_gated_workspace_size": ([_I, _I64, _I64, _I64, _I64], _SZ),
    "nvfp4_gated": ([_P, _P, _P, _I, _I64, _I64, _P, _I, _P, _I64, _P, _I64, _P, _I64, _P, _SZ, _P], _I),
    "nvfp4_linear_backward_workspace_size": ([_I, _I64, _I64, _I64, _I64, _I], _SZ),
    "nvfp4_linear_backward": ([_P, _P, _I, _I64, _I64, _P, _I, _P, _I64, _P, _I64, _P, _P, _I64, _P,
                               _SZ, _P], _I),
    "nvfp4_gated_backward_workspace_size": ([_I, _I64, _I64, _I64, _I64], _SZ),
    "nvfp4_gated_backward": ([_P, _P, _P, _I, _I64, _I64, _P, _I, _P, _I64, _P, _I64, _P, _I64, _P,
                              _I64, _P, _I64, _P, _SZ, _P], _I),
    "nvfp4_kv_page_bytes": ([_I32, _I32, _I32], _SZ),
    "nvfp4_kv_append": ([_P, _I64, _P, _P, _I, _I64, _I64, _I64, _I64, _I64, _P, _P, _I64, _I32,
                         _I32, _P], _I),
    "nvfp4_kv_read": ([_P, _I64, _P, _P, _I, _I64, _P, _P, _I64, _P], _I),
    "nvfp4_kv_attention_workspace_size": ([_P, _I, _I64, _I64, _I64, _I64, _I64], _SZ),
    "nvfp4_kv_attention": ([_P, _I64, _P, _I, _I64, _I64, _I64, _I64, _P, _P, _I64, _I64, _I64,
                            ctypes.c_float, _I, _I64, _P, _I64, _I64, _P, _P, _SZ, _P], _I),
    "nvfp4_kv_pages_workspace_size": ([_P, _I64], _SZ),
    "nvfp4_kv_reserve": ([_P, _P, _P, _I64, _P, _P, _SZ, _P], _I),
    "nvfp4_kv_fork": ([_P, _P, _P, _I64, _P, _P, _SZ, _P], _I),
    "nvfp4_kv_free": ([_P, _P, _I64, _P, _P], _I),
    "nvfp4_kv_compact": ([_P, _P, _P, _SZ, _P], _I),
}
for _name, (_args, _res) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = _res

EXPORTS = tuple(_SIGS)
_KV = {n: getattr(_lib, n) for n in _SIGS if n.startswith("nvfp4_kv_")}


class Nvfp4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_lib.nvfp4_status_string(status).decode()}")


def _check(status: int, where: str) -> None:
    if status != OK:
        raise Nvfp4Error(status, where)


def _run(fname: str, args: tuple, prepare: bool):
    """Call C entry point `fname` with marshalled `args`, or (prepare=True) return a
    zero-argument callable that makes exactly that call; the tensors behind the pointers must
    then stay alive and unchanged in size while the callable is used."""
    f = getattr(_lib, fname)
    if not prepare:
        _check(f(*args), fname)
        return None

    def call():
        _check(f(*args), fname)
    return call


def _dev(t: torch.Tensor | None, name: str, dtypes=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a tensor on the GPU")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    return ctypes.c_void_p(t.data_ptr())


def _wdtype(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return DTYPE_F32
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    raise TypeError(f"unsupported element type {t.dtype} (float32 or bfloat16)")


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _need(t: torch.Tensor, numel: int, name: str):
    if not t.is_contiguous() or t.numel() < numel:
        raise ValueError(f"{name} must be contiguous with at least {numel} elements")


def nvfp4_version() -> str:
    return _lib.nvfp4_version().decode()


def nvfp4_status_string(status: int) -> str:
    return _lib.nvfp4_status_string(status).decode()


def nvfp4_diag_hessian_workspace_size(tokens: int, inp: int, segments: int = 1) -> int:
    return int(_lib.nvfp4_diag_hessian_workspace_size(tokens, inp, segments))


def _i64_array(values):
    return (ctypes.c_int64 * len(values))(*[int(v) for v in values])


def nvfp4_diag_hessian_chunks_workspace_size(tokens, inp: int) -> int:
    t = _i64_array(tokens)
    return int(_lib.nvfp4_diag_hessian_chunks_workspace_size(t, len(tokens), inp))


def nvfp4_diag_hessian_chunks(X_chunks, inp, ldx, h_acc, h, accumulate, workspace, stream=None,
                              prepare=False):
    """h over several token chunks (tensors [tokens_c, in] at separate addresses) in one partial
    launch and one finalize."""
    if not X_chunks:
        raise ValueError("at least one chunk")
    dt = {_wdtype(X) for X in X_chunks}
    if len(dt) != 1:
        raise TypeError("every chunk must have the same element type")
    _need(h_acc, inp, "h_acc")
    if h is not None:
        _need(h, inp, "h")
    ptrs = (ctypes.c_void_p * len(X_chunks))(*[_dev(X, "X").value for X in X_chunks])
    toks = _i64_array([X.shape[0] for X in X_chunks])
    args = (ptrs, dt.pop(), toks, len(X_chunks), inp, ldx, _dev(h_acc, "h_acc", (torch.float64,)),
            _dev(h, "h", (torch.float32,)), int(accumulate), _dev(workspace, "workspace"),
            workspace.numel() * workspace.element_size(), _stream(stream))
    return _run("nvfp4_diag_hessian_chunks", args, prepare)


def nvfp4_global_scale_workspace_size(batch: int, out: int, inp: int) -> int:
    return int(_lib.nvfp4_global_scale_workspace_size(batch, out, inp))


def nvfp4_layer_statistics_workspace_size(tokens: int, inp: int, out: int) -> int:
    return int(_lib.nvfp4_layer_statistics_workspace_size(tokens, inp, out))


def nvfp4_diag_hessian(X, tokens, inp, ldx, h_acc, h, accumulate, workspace, stream=None, prepare=False):
    """h_acc = h = None: deferred mode (row-group sums into the workspace only)."""
    if h_acc is not None:
        _need(h_acc, inp, "h_acc")
    if h is not None:
        _need(h, inp, "h")
    return _run("nvfp4_diag_hessian", (
        _dev(X, "X", (torch.float32, torch.bfloat16)), _wdtype(X), tokens, inp, ldx,
        _dev(h_acc, "h_acc", (torch.float64,)), _dev(h, "h", (torch.float32,)), int(accumulate),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream(stream)), prepare)


def nvfp4_diag_hessian_finalize(X_dtype, tokens, inp, h_acc, h, accumulate, workspace,
                                stream=None, prepare=False):
    """Finalize of deferred nvfp4_diag_hessian calls (X_dtype: torch.bfloat16 or float32)."""
    dt = DTYPE_BF16 if X_dtype == torch.bfloat16 else DTYPE_F32
    return _run("nvfp4_diag_hessian_finalize", (
        dt, tokens, inp, _dev(h_acc, "h_acc", (torch.float64,)), _dev(h, "h", (torch.float32,)),
        int(accumulate), _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream(stream)), prepare)


def nvfp4_diag_hessian_batched(X, seg_offsets, segments, total_tokens, inp, ldx, h_acc, h,
                               accumulate, workspace, stream=None, prepare=False):
    _need(h_acc, segments * inp, "h_acc")
    if h is not None:
        _need(h, segments * inp, "h")
    return _run("nvfp4_diag_hessian_batched", (
        _dev(X, "X", (torch.float32, torch.bfloat16)), _wdtype(X),
        _dev(seg_offsets, "seg_offsets", (torch.int64,)), segments, total_tokens, inp, ldx,
        _dev(h_acc, "h_acc", (torch.float64,)), _dev(h, "h", (torch.float32,)), int(accumulate),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream(stream)), prepare)


def nvfp4_global_scale(W, batch, out, inp, ldw, stride_w, rule, S, workspace, stream=None, prepare=False):
    _need(S, batch, "S")
    return _run("nvfp4_global_scale", (
        _dev(W, "W", (torch.float32, torch.bfloat16)), _wdtype(W), batch, out, inp, ldw, stride_w,
        rule, _dev(S, "S", (torch.float32,)), _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream)), prepare)


def nvfp4_layer_statistics(X, tokens, inp, ldx, h_acc, h, accumulate, W, out, ldw, rule, S,
                           workspace, stream=None, prepare=False):
    _need(h_acc, inp, "h_acc")
    if h is not None:
        _need(h, inp, "h")
    _need(S, 1, "S")
    return _run("nvfp4_layer_statistics", (
        _dev(X, "X", (torch.float32, torch.bfloat16)), _wdtype(X), tokens, inp, ldx,
        _dev(h_acc, "h_acc", (torch.float64,)), _dev(h, "h", (torch.float32,)), int(accumulate),
        _dev(W, "W", (torch.float32, torch.bfloat16)), _wdtype(W), out, ldw, rule,
        _dev(S, "S", (torch.float32,)), _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream)), prepare)


def nvfp4_scale_search(W, batch, out, inp, ldw, stride_w, group_size, h, stride_h, objective,
                       lo, hi, exhaustive, S, scales, packed, loss=None, offset=None, stream=None, prepare=False):
    G = batch * out * (inp // 16)
    _need(scales, G, "scales")
    _need(packed, G * 8, "packed")
    _need(S, batch, "S")
    if loss is not None:
        _need(loss, G, "loss")
    if offset is not None:
        _need(offset, G, "offset")
    return _run("nvfp4_scale_search", (
        _dev(W, "W", (torch.float32, torch.bfloat16)), _wdtype(W), batch, out, inp, ldw, stride_w,
        group_size, _dev(h, "h", (torch.float32,)), stride_h, objective, lo, hi, int(exhaustive),
        _dev(S, "S", (torch.float32,)), _dev(scales, "scales", (torch.uint8,)),
        _dev(packed, "packed", (torch.uint8,)), _dev(loss, "loss", (torch.float32,)),
        _dev(offset, "offset", (torch.int8,)), _stream(stream)), prepare)


def nvfp4_scale_search_rules(W, batch, out, inp, ldw, stride_w, group_size, h, stride_h, S, rules,
                             stream=None, prepare=False):
    """rules: sequence of dicts with keys objective, lo, hi, exhaustive, scales, packed and
    optionally loss, offset (tensors)."""
    G = batch * out * (inp // 16)
    _need(S, batch, "S")
    arr = (SearchRule * len(rules))()
    for k, r in enumerate(rules):
        _need(r["scales"], G, "scales")
        _need(r["packed"], G * 8, "packed")
        loss, offset = r.get("loss"), r.get("offset")
        if loss is not None:
            _need(loss, G, "loss")
        if offset is not None:
            _need(offset, G, "offset")
        p = lambda t, name, dt: None if t is None else _dev(t, name, dt).value
        arr[k] = SearchRule(int(r["objective"]), int(r["lo"]), int(r["hi"]), int(r["exhaustive"]),
                            p(r["scales"], "scales", (torch.uint8,)),
                            p(r["packed"], "packed", (torch.uint8,)),
                            p(loss, "loss", (torch.float32,)), p(offset, "offset", (torch.int8,)))
    call = _run("nvfp4_scale_search_rules", (
        _dev(W, "W", (torch.float32, torch.bfloat16)), _wdtype(W), batch, out, inp, ldw, stride_w,
        group_size, _dev(h, "h", (torch.float32,)), stride_h, _dev(S, "S", (torch.float32,)),
        arr, len(rules), _stream(stream)), prepare)
    if prepare:
        return lambda: (arr, call())[1]     # the closure keeps the rule array alive
    return None


def nvfp4_scale_search_scored(W, batch, out, inp, ldw, stride_w, group_size, h, stride_h,
                              objective, centre_lo, S, count, stream=None, prepare=False):
    _need(S, batch, "S")
    _need(count, 1, "count")
    return _run("nvfp4_scale_search_scored", (
        _dev(W, "W", (torch.float32, torch.bfloat16)), _wdtype(W), batch, out, inp, ldw, stride_w,
        group_size, _dev(h, "h", (torch.float32,)), stride_h, objective, centre_lo,
        _dev(S, "S", (torch.float32,)), _dev(count, "count", (torch.int64,)), _stream(stream)),
        prepare)


def nvfp4_scale_search_proposal(W, batch, out, inp, ldw, stride_w, group_size, h, stride_h,
                                objective, lo, hi, center, incoming, S, scales, packed, loss=None,
                                offset=None, stream=None, prepare=False):
    G = batch * out * (inp // 16)
    _need(scales, G, "scales")
    _need(packed, G * 8, "packed")
    _need(center, G, "center")
    if incoming is not None:
        _need(incoming, G, "incoming")
    _need(S, batch, "S")
    if loss is not None:
        _need(loss, G, "loss")
    if offset is not None:
        _need(offset, G, "offset")
    return _run("nvfp4_scale_search_proposal", (
        _dev(W, "W", (torch.float32, torch.bfloat16)), _wdtype(W), batch, out, inp, ldw, stride_w,
        group_size, _dev(h, "h", (torch.float32,)), stride_h, objective, lo, hi,
        _dev(center, "center", (torch.uint8,)), _dev(incoming, "incoming", (torch.uint8,)),
        _dev(S, "S", (torch.float32,)), _dev(scales, "scales", (torch.uint8,)),
        _dev(packed, "packed", (torch.uint8,)), _dev(loss, "loss", (torch.float32,)),
        _dev(offset, "offset", (torch.int8,)), _stream(stream)), prepare)


def nvfp4_pack(W, batch, out, inp, ldw, stride_w, scales, S, packed, stream=None, prepare=False):
    G = batch * out * (inp // 16)
    _need(scales, G, "scales")
    _need(packed, G * 8, "packed")
    return _run("nvfp4_pack", (
        _dev(W, "W", (torch.float32, torch.bfloat16)), _wdtype(W), batch, out, inp, ldw, stride_w,
        _dev(scales, "scales", (torch.uint8,)), _dev(S, "S", (torch.float32,)),
        _dev(packed, "packed", (torch.uint8,)), _stream(stream)), prepare)


def nvfp4_quantize_activations_workspace_size(tokens: int, inp: int) -> int:
    return int(_lib.nvfp4_quantize_activations_workspace_size(tokens, inp))


def nvfp4_quantize_activations(X, tokens, inp, ldx, objective, h, lo, hi, rule, S_out, scales,
                               packed, workspace, stream=None, prepare=False):
    G = tokens * (inp // 16)
    _need(scales, G, "scales")
    _need(packed, G * 8, "packed")
    return _run("nvfp4_quantize_activations", (
        _dev(X, "X", (torch.float32, torch.bfloat16)), _wdtype(X), tokens, inp, ldx, objective,
        _dev(h, "h", (torch.float32,)), lo, hi, rule, _dev(S_out, "S_out", (torch.float32,)),
        _dev(scales, "scales", (torch.uint8,)), _dev(packed, "packed", (torch.uint8,)),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream(stream)), prepare)


def nvfp4_quantize_activations_noalloc(X, tokens, inp, ldx, objective, h, lo, hi, rule, S_out,
                                       scales, packed, stream=None, prepare=False):
    """nvfp4_quantize_activations without a workspace: the library's own per-GPU scratch (no
    allocation; calls that overlap on one GPU race)."""
    G = tokens * (inp // 16)
    _need(scales, G, "scales")
    _need(packed, G * 8, "packed")
    return _run("nvfp4_quantize_activations_noalloc", (
        _dev(X, "X", (torch.float32, torch.bfloat16)), _wdtype(X), tokens, inp, ldx, objective,
        _dev(h, "h", (torch.float32,)), lo, hi, rule, _dev(S_out, "S_out", (torch.float32,)),
        _dev(scales, "scales", (torch.uint8,)), _dev(packed, "packed", (torch.uint8,)),
        _stream(stream)), prepare)


def nvfp4_gptq_workspace_size(out: int, inp: int) -> int:
    return int(_lib.nvfp4_gptq_workspace_size(out, inp))


def nvfp4_gptq(W, out, inp, ldw, U, h, objective, lo, hi, S, scales, packed, W_final, workspace,
               stream=None, prepare=False):
    _need(scales, out * (inp // 16), "scales")
    _need(packed, out * (inp // 2), "packed")
    _need(U, inp * inp, "U")
    if h is not None:
        _need(h, inp, "h")
    if W_final is not None:
        _need(W_final, out * inp, "W_final")
    return _run("nvfp4_gptq", (
        _dev(W, "W", (torch.float32, torch.bfloat16)), _wdtype(W), out, inp, ldw,
        _dev(U, "U", (torch.float32,)), _dev(h, "h", (torch.float32,)), objective, lo, hi,
        _dev(S, "S", (torch.float32,)), _dev(scales, "scales", (torch.uint8,)),
        _dev(packed, "packed", (torch.uint8,)), _dev(W_final, "W_final", (torch.float32,)),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream(stream)), prepare)


def nvfp4_output_error_workspace_size(tokens: int, out: int, inp: int) -> int:
    return int(_lib.nvfp4_output_error_workspace_size(tokens, out, inp))


def nvfp4_output_error(X, tokens, inp, ldx, W, out, ldw, scales, packed, S, err, accumulate,
                       workspace, stream=None, prepare=False):
    _need(err, out, "err")
    return _run("nvfp4_output_error", (
        _dev(X, "X", (torch.bfloat16,)), DTYPE_BF16, tokens, inp, ldx,
        _dev(W, "W", (torch.float32, torch.bfloat16)), _wdtype(W), out, ldw,
        _dev(scales, "scales", (torch.uint8,)), _dev(packed, "packed", (torch.uint8,)),
        _dev(S, "S", (torch.float32,)), _dev(err, "err", (torch.float64,)), int(accumulate),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream(stream)), prepare)


# --- key/value cache --------------------------------------------------------------------------

KV_DONE, KV_BAD_SLOT, KV_BAD_LENGTH, KV_NO_PAGES = range(4)


def nvfp4_kv_page_bytes(heads: int, head_dim: int, page_size: int) -> int:
    return int(_lib.nvfp4_kv_page_bytes(heads, head_dim, page_size))


class Matrix:
    """``nvfp4_matrix``: codes, scale bytes and global scales of one matrix or a batch, as ``scale_search`` or
    ``gptq`` return them: packed [out, in/2] or [batch, out, in/2] uint8, scales [out, in/16] or
    [batch, out, in/16] uint8, S [batch] float32. Rows are contiguous; the matrices of a batch may lie
    apart (a slice of rows of a larger batch). The tensors are kept, not copied."""

    def __init__(self, packed, scales, S):
        for name, t in (("packed", packed), ("scales", scales)):
            _dev(t, name, (torch.uint8,))
        if packed.dim() not in (2, 3) or scales.dim() != packed.dim():
            raise ValueError("packed and scales must both be 2-D or both 3-D")
        batch = packed.shape[0] if packed.dim() == 3 else 1
        out, half = packed.shape[-2:]
        if half % 8 or tuple(scales.shape) != tuple(packed.shape[:-1]) + (half // 8,):
            raise ValueError("packed must be [.., out, in/2] and scales [.., out, in/16] of the same matrices")
        rows = lambda t: t.stride(-1) == 1 and (out == 1 or t.stride(-2) == t.shape[-1])  # noqa: E731
        if batch * out and half and not (rows(packed) and rows(scales)):
            raise ValueError("rows of packed and scales must be contiguous")
        stride = 2 * packed.stride(0) if batch > 1 else 2 * out * half
        if batch > 1 and 16 * scales.stride(0) != stride:
            raise ValueError("the matrices of packed and of scales must lie equally far apart")
        _dev(S, "S", (torch.float32,))
        _need(S, batch, "S")
        if scales.device != packed.device or S.device != packed.device:
            raise ValueError("packed, scales and S must be on one device")
        self.packed, self.scales, self.S = packed, scales, S
        self.batch, self.out, self.inp = batch, out, 2 * half
        self.device, self.index = packed.device, packed.get_device()
        self.struct = MatrixStruct(packed.data_ptr(), scales.data_ptr(), S.data_ptr(), batch, out, 2 * half,
                                   stride)
        self.ref = ctypes.byref(self.struct)


def _on_device(index: int, f, args: tuple, fname: str, stream, prepare: bool):
    """Calls entry point f with args on `stream` (None: the device's current one), with that device current."""
    s = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if not prepare and torch._C._cuda_getDevice() == index:
        status = f(*args, s)
        if status:
            raise Nvfp4Error(status, fname)
        return None

    def call():
        old = torch._C._cuda_getDevice()
        torch.cuda.set_device(index)
        try:
            _check(f(*args, s), fname)
        finally:
            torch.cuda.set_device(old)
    return call if prepare else call()


def _on(W: Matrix, t, name: str, dtype=None, numel: int | None = None):
    """Address of a tensor on the matrices' device, of this dtype and (contiguous) at least numel elements."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a tensor on the GPU")
    if t.get_device() != W.index:
        raise ValueError(f"{name} must be on the matrices' device {W.device}")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if numel is not None and (not t.is_contiguous() or t.numel() < numel):
        _need(t, numel, name)
    return t.data_ptr()


def _rows(W: Matrix, t, tokens: int, cols: int, dtype, name: str):
    """A row tensor [tokens, cols] with contiguous rows: address and row stride."""
    if t is None:
        return None, cols
    p = _on(W, t, name, dtype)
    if t.dim() != 2 or t.shape[0] != tokens or t.shape[1] != cols or (cols > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be [{tokens}, {cols}] with contiguous rows")
    return p, t.stride(0) if tokens > 1 else max(t.stride(0), cols)


def _segments(W: Matrix, seg_offsets):
    if seg_offsets is not None and seg_offsets.numel() != W.batch + 1:
        raise ValueError(f"seg_offsets must have {W.batch + 1} elements")
    return _on(W, seg_offsets, "seg_offsets", torch.int64, W.batch + 1)


def _space(W: Matrix, t):
    if t is None:
        return None, 0
    return _on(W, t, "workspace", None, 0), t.numel() * t.element_size()


def _dtype_code(dtype) -> int:
    """dtype: torch.bfloat16 or torch.float32."""
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"dtype {dtype} is not supported: torch.bfloat16 or torch.float32")
    return DTYPE_BF16 if dtype == torch.bfloat16 else DTYPE_F32


def nvfp4_linear_workspace_size(dtype, tokens, batch, out, inp) -> int:
    return _lib.nvfp4_linear_workspace_size(_dtype_code(dtype), tokens, batch, out, inp)


def nvfp4_linear(W: Matrix, X, tokens, seg_offsets, bias, activation, residual, Z, Y, workspace, stream=None,
                 prepare=False):
    dt = X.dtype
    x, r = _rows(W, X, tokens, W.inp, None, "X"), _rows(W, residual, tokens, W.out, dt, "residual")
    z, y = _rows(W, Z, tokens, W.out, dt, "Z"), _rows(W, Y, tokens, W.out, dt, "Y")
    return _on_device(W.index, _lib.nvfp4_linear, (
        W.ref, x[0], _dtype_code(dt), tokens, x[1], _segments(W, seg_offsets),
        _on(W, bias, "bias", dt, W.batch * W.out), activation, *r, *z, *y, *_space(W, workspace)),
        "nvfp4_linear", stream, prepare)


def nvfp4_gated_workspace_size(dtype, tokens, batch, out, inp) -> int:
    return _lib.nvfp4_gated_workspace_size(_dtype_code(dtype), tokens, batch, out, inp)


def _pair(W_gate: Matrix, W_up: Matrix):
    if W_up.index != W_gate.index:
        raise ValueError("W_gate and W_up must be on one device")


def nvfp4_gated(W_gate: Matrix, W_up: Matrix, X, tokens, seg_offsets, activation, G, U, H, workspace,
                stream=None, prepare=False):
    _pair(W_gate, W_up)
    W, dt = W_gate, X.dtype
    x, g = _rows(W, X, tokens, W.inp, None, "X"), _rows(W, G, tokens, W.out, dt, "G")
    u, h = _rows(W, U, tokens, W.out, dt, "U"), _rows(W, H, tokens, W.out, dt, "H")
    return _on_device(W.index, _lib.nvfp4_gated, (
        W.ref, W_up.ref, x[0], _dtype_code(dt), tokens, x[1], _segments(W, seg_offsets), activation,
        *g, *u, *h, *_space(W, workspace)), "nvfp4_gated", stream, prepare)


def nvfp4_linear_backward_workspace_size(dtype, tokens, batch, out, inp, with_bias) -> int:
    return _lib.nvfp4_linear_backward_workspace_size(_dtype_code(dtype), tokens, batch, out, inp,
                                                     int(with_bias))


def nvfp4_linear_backward(W: Matrix, dY, tokens, seg_offsets, activation, Z, dZ, dbias, dX, workspace,
                          stream=None, prepare=False):
    dt = dY.dtype
    y, z = _rows(W, dY, tokens, W.out, None, "dY"), _rows(W, Z, tokens, W.out, dt, "Z")
    d, x = _rows(W, dZ, tokens, W.out, dt, "dZ"), _rows(W, dX, tokens, W.inp, dt, "dX")
    return _on_device(W.index, _lib.nvfp4_linear_backward, (
        W.ref, y[0], _dtype_code(dt), tokens, y[1], _segments(W, seg_offsets), activation, *z, *d,
        _on(W, dbias, "dbias", torch.float32, W.batch * W.out), *x, *_space(W, workspace)),
        "nvfp4_linear_backward", stream, prepare)


def nvfp4_gated_backward_workspace_size(dtype, tokens, batch, out, inp) -> int:
    return _lib.nvfp4_gated_backward_workspace_size(_dtype_code(dtype), tokens, batch, out, inp)


def nvfp4_gated_backward(W_gate: Matrix, W_up: Matrix, dH, tokens, seg_offsets, activation, G, U, dG, dU,
                         dX, workspace, stream=None, prepare=False):
    _pair(W_gate, W_up)
    W, dt = W_gate, dH.dtype
    rows = [_rows(W, t, tokens, W.out, dt, name) for t, name in
            ((G, "G"), (U, "U"), (dG, "dG"), (dU, "dU"))]
    h, x = _rows(W, dH, tokens, W.out, None, "dH"), _rows(W, dX, tokens, W.inp, dt, "dX")
    return _on_device(W.index, _lib.nvfp4_gated_backward, (
        W.ref, W_up.ref, h[0], _dtype_code(dt), tokens, h[1], _segments(W, seg_offsets), activation,
        *rows[0], *rows[1], *rows[2], *rows[3], *x, *_space(W, workspace)),
        "nvfp4_gated_backward", stream, prepare)


class KVCache:
    """A paged NVFP4 key/value cache: the tensors behind ``nvfp4_kv_cache`` (kept alive here).

    pages [layers, num_pages, page_bytes] uint8 (records contiguous), table [max_slots, max_pages], lens [max_slots]
    and refs [num_pages] int32 (refs may be None where no page call is made), S_k and S_v
    [layers, heads] float32 (None where only page calls are made). ``KVCache.empty`` allocates a
    cache with no slot in use.

    The cache serves and does not train: no call records a gradient, so outputs never require one, even where
    the rows given do."""

    def __init__(self, pages, table, lens, refs, S_k, S_v, heads: int, head_dim: int,
                 page_size: int):
        record = nvfp4_kv_page_bytes(heads, head_dim, page_size)
        if record == 0:
            raise Nvfp4Error(ERR_SHAPE, "KVCache")
        if pages.dim() != 3 or pages.shape[2] < record or pages.stride(2) != 1:
            raise ValueError(f"pages must be [layers, num_pages, >= {record}] with contiguous records")
        layers, num_pages, _ = pages.shape
        if table.dim() != 2:
            raise ValueError("table must be [max_slots, max_pages]")
        _need(table, table.numel(), "table")
        _need(lens, table.shape[0], "lens")
        if refs is not None:
            _need(refs, num_pages, "refs")
        for name, S in (("S_k", S_k), ("S_v", S_v)):
            if S is not None:
                _need(S, layers * heads, name)
        i32, f32 = (torch.int32,), (torch.float32,)
        p = lambda t, name, dt: None if t is None else _dev(t, name, dt).value  # noqa: E731
        for name, t in (("table", table), ("lens", lens), ("refs", refs), ("S_k", S_k), ("S_v", S_v)):
            if t is not None and t.device != pages.device:
                raise ValueError(f"{name} must be on the pages' device")
        self.pages, self.table, self.lens, self.refs = pages, table, lens, refs
        self.S_k, self.S_v = S_k, S_v
        self.heads, self.head_dim, self.page_size = heads, head_dim, page_size
        self.layers, self.num_pages, self.device = layers, num_pages, pages.device
        self.index = pages.get_device()
        self.sizes = {}                      # workspace bytes by sizes: a pure function of them
        self.struct = KVCacheStruct(
            p(pages, "pages", (torch.uint8,)), layers, pages.stride(0), num_pages, pages.stride(1),
            heads, head_dim, page_size, table.shape[1], table.shape[0], p(table, "table", i32),
            p(lens, "lens", i32), p(refs, "refs", i32), p(S_k, "S_k", f32), p(S_v, "S_v", f32))
        self.ref = ctypes.byref(self.struct)

    @classmethod
    def empty(cls, layers: int, num_pages: int, heads: int, head_dim: int, page_size: int,
              max_slots: int, max_pages: int, S_k, S_v, device="cuda") -> "KVCache":
        record = nvfp4_kv_page_bytes(heads, head_dim, page_size)
        if record == 0:
            raise Nvfp4Error(ERR_SHAPE, "KVCache.empty")
        i32 = dict(dtype=torch.int32, device=device)
        return cls(torch.empty((layers, num_pages, record), dtype=torch.uint8, device=device),
                   torch.full((max_slots, max_pages), -1, **i32), torch.zeros(max_slots, **i32),
                   torch.zeros(num_pages, **i32), S_k, S_v, heads, head_dim, page_size)


def _kv_run(cache: KVCache, fname: str, args: tuple, stream, prepare: bool):
    """Calls a cache entry point with pointers and numbers in `args`, on `stream` (None: the current
    stream of the cache's device), with that device current. (torch's public functions for both take 1.4 us a call,
    these 0.2, where a decode step's calls are bound by the host.)"""
    index = cache.index
    s = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    f = _KV[fname]
    if not prepare and torch._C._cuda_getDevice() == index:
        status = f(cache.ref, *args, s)
        if status:
            raise Nvfp4Error(status, fname)
        return None

    def call():
        old = torch._C._cuda_getDevice()
        torch.cuda.set_device(index)
        try:
            _check(f(cache.ref, *args, s), fname)
        finally:
            torch.cuda.set_device(old)
    return call if prepare else call()


def _kv_ptr(cache: KVCache, t, name: str, dtype=None, numel: int | None = None):
    """Address of a tensor on the cache's device, of this dtype and (contiguous) at least numel elements."""
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.get_device() == cache.index
            and (dtype is None or t.dtype is dtype)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a tensor on the GPU")
        if t.get_device() != cache.index:
            raise ValueError(f"{name} must be on the cache's device {cache.device}")
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if numel is not None and (not t.is_contiguous() or t.numel() < numel):
        _need(t, numel, name)
    return t.data_ptr()


def _kv_rows(cache: KVCache, t, heads, dtype, name):
    """A token tensor [tokens, heads, head_dim] with contiguous rows: address, token and head strides."""
    p = _kv_ptr(cache, t, name, dtype)
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != cache.head_dim or t.stride(2) != 1:
        raise ValueError(f"{name} must be [tokens, {heads}, {cache.head_dim}] with contiguous rows")
    return p, t.stride(0), t.stride(1)


def nvfp4_kv_append(cache: KVCache, layer, K, V, cu_tokens, slots, seqs, lo, hi, stream=None,
                    prepare=False):
    k, skt, skh = _kv_rows(cache, K, cache.heads, None, "K")
    v, svt, svh = _kv_rows(cache, V, cache.heads, K.dtype, "V")
    if V.shape[0] != K.shape[0]:
        raise ValueError("K and V must have the same shape")
    return _kv_run(cache, "nvfp4_kv_append", (
        layer, k, v, _wdtype(K), K.shape[0], skt, skh, svt, svh,
        _kv_ptr(cache, cu_tokens, "cu_tokens", torch.int32, seqs + 1),
        _kv_ptr(cache, slots, "slots", torch.int32, seqs), seqs, lo, hi), stream, prepare)


def nvfp4_kv_read(cache: KVCache, layer, K, V, tokens, cu_tokens, slots, seqs, stream=None,
                  prepare=False):
    numel = tokens * cache.heads * cache.head_dim
    return _kv_run(cache, "nvfp4_kv_read", (
        layer, _kv_ptr(cache, K, "K", None, numel), _kv_ptr(cache, V, "V", K.dtype, numel),
        _wdtype(K), tokens, _kv_ptr(cache, cu_tokens, "cu_tokens", torch.int32, seqs + 1),
        _kv_ptr(cache, slots, "slots", torch.int32, seqs), seqs), stream, prepare)


def nvfp4_kv_attention_workspace_size(cache: KVCache, dtype, tokens, q_heads, seqs, max_q,
                                      max_kv) -> int:
    """dtype: torch.bfloat16 or torch.float32."""
    key = (dtype, tokens, q_heads, seqs, max_q, max_kv)
    size = cache.sizes.get(key)
    if size is None:
        dt = DTYPE_BF16 if dtype == torch.bfloat16 else DTYPE_F32
        size = _lib.nvfp4_kv_attention_workspace_size(cache.ref, dt, tokens, q_heads, seqs, max_q, max_kv)
        if len(cache.sizes) >= 4096:
            cache.sizes.clear()
        cache.sizes[key] = size
    return size


def nvfp4_kv_attention(cache: KVCache, layer, Q, cu_tokens, slots, seqs, max_q, max_kv, scale,
                       causal, window, O, lse, workspace, stream=None, prepare=False):
    q_heads = Q.shape[1] if Q.dim() == 3 else 0
    q, sqt, sqh = _kv_rows(cache, Q, q_heads, None, "Q")
    o, sot, soh = _kv_rows(cache, O, q_heads, Q.dtype, "O")
    tokens = Q.shape[0]
    if O.shape[0] != tokens:
        raise ValueError("O and Q must have the same shape")
    return _kv_run(cache, "nvfp4_kv_attention", (
        layer, q, _wdtype(Q), tokens, q_heads, sqt, sqh,
        _kv_ptr(cache, cu_tokens, "cu_tokens", torch.int32, seqs + 1),
        _kv_ptr(cache, slots, "slots", torch.int32, seqs), seqs, max_q, max_kv, scale, int(causal),
        window, o, sot, soh, _kv_ptr(cache, lse, "lse", torch.float32, tokens * q_heads),
        *_kv_space(cache, workspace)), stream, prepare)


def _kv_space(cache: KVCache, t):
    """Address and bytes of a workspace tensor."""
    if t is None:
        return None, 0
    return _kv_ptr(cache, t, "workspace", None, 0), t.numel() * t.element_size()


def nvfp4_kv_pages_workspace_size(cache: KVCache, n: int) -> int:
    size = cache.sizes.get(n)
    if size is None:
        size = cache.sizes[n] = _lib.nvfp4_kv_pages_workspace_size(cache.ref, n)
    return size


def nvfp4_kv_reserve(cache: KVCache, slots, counts, n, status, workspace, stream=None, prepare=False):
    i32 = torch.int32
    return _kv_run(cache, "nvfp4_kv_reserve", (
        _kv_ptr(cache, slots, "slots", i32, n), _kv_ptr(cache, counts, "counts", i32, n), n,
        _kv_ptr(cache, status, "status", i32, 1), *_kv_space(cache, workspace)), stream, prepare)


def nvfp4_kv_fork(cache: KVCache, parents, children, n, status, workspace, stream=None,
                  prepare=False):
    i32 = torch.int32
    return _kv_run(cache, "nvfp4_kv_fork", (
        _kv_ptr(cache, parents, "parents", i32, n), _kv_ptr(cache, children, "children", i32, n), n,
        _kv_ptr(cache, status, "status", i32, 1), *_kv_space(cache, workspace)), stream, prepare)


def nvfp4_kv_free(cache: KVCache, slots, n, status, stream=None, prepare=False):
    i32 = torch.int32
    return _kv_run(cache, "nvfp4_kv_free", (
        _kv_ptr(cache, slots, "slots", i32, n), n, _kv_ptr(cache, status, "status", i32, 1)),
        stream, prepare)


def nvfp4_kv_compact(cache: KVCache, used, workspace, stream=None, prepare=False):
    return _kv_run(cache, "nvfp4_kv_compact", (
        _kv_ptr(cache, used, "used", torch.int32, 1), *_kv_space(cache, workspace)), stream, prepare)


# --- convenience wrappers (allocate outputs with torch, then call the entry points) ----------

def _bmat(W: torch.Tensor):
    """(batch, out, in, ldw, stride_w) of a [out, in] or [batch, out, in] row-major tensor."""
    if W.dim() == 2:
        if W.stride(1) != 1:
            raise ValueError("W rows must be contiguous")
        return 1, W.shape[0], W.shape[1], W.stride(0), W.shape[0] * W.stride(0)
    if W.dim() == 3:
        if W.stride(2) != 1:
            raise ValueError("W rows must be contiguous")
        return W.shape[0], W.shape[1], W.shape[2], W.stride(1), W.stride(0)
    raise ValueError("W must be 2-D or 3-D")


def diag_hessian(X: torch.Tensor, h_acc: torch.Tensor | None = None, accumulate: bool = False,
                 stream=None):
    """h over X [tokens, in]; returns (h_acc float64 [in], h float32 [in])."""
    T, n = X.shape
    if X.stride(1) != 1:
        raise ValueError("X rows must be contiguous")
    if h_acc is None:
        h_acc = torch.zeros(n, dtype=torch.float64, device=X.device)
    h = torch.empty(n, dtype=torch.float32, device=X.device)
    ws = torch.zeros(max(1, nvfp4_diag_hessian_workspace_size(T, n, 1)), dtype=torch.uint8,
                     device=X.device)
    nvfp4_diag_hessian(X, T, n, X.stride(0), h_acc, h, accumulate, ws, stream)
    return h_acc, h


def diag_hessian_batched(X: torch.Tensor, seg_offsets: torch.Tensor,
                         h_acc: torch.Tensor | None = None, accumulate: bool = False, stream=None):
    """Per-segment h over the routed rows of X; returns (h_acc [E, in] f64, h [E, in] f32)."""
    T, n = X.shape
    E = seg_offsets.numel() - 1
    if h_acc is None:
        h_acc = torch.zeros((E, n), dtype=torch.float64, device=X.device)
    h = torch.empty((E, n), dtype=torch.float32, device=X.device)
    ws = torch.zeros(max(1, nvfp4_diag_hessian_workspace_size(T, n, E)), dtype=torch.uint8,
                     device=X.device)
    nvfp4_diag_hessian_batched(X, seg_offsets, E, T, n, X.stride(0), h_acc, h, accumulate, ws,
                               stream)
    return h_acc, h


def layer_statistics(X: torch.Tensor, W: torch.Tensor, rule: int = GS_AMAX_448,
                     h_acc: torch.Tensor | None = None, accumulate: bool = False, stream=None):
    """h over X [tokens, in] and S of W [out, in]; returns (h_acc f64 [in], h f32 [in], S [1])."""
    T, n = X.shape
    o = W.shape[0]
    if X.stride(1) != 1 or W.stride(1) != 1:
        raise ValueError("X and W rows must be contiguous")
    if h_acc is None:
        h_acc = torch.zeros(n, dtype=torch.float64, device=X.device)
    h = torch.empty(n, dtype=torch.float32, device=X.device)
    S = torch.empty(1, dtype=torch.float32, device=X.device)
    ws = torch.empty(max(16, nvfp4_layer_statistics_workspace_size(T, n, o)), dtype=torch.uint8,
                     device=X.device)
    nvfp4_layer_statistics(X, T, n, X.stride(0), h_acc, h, accumulate, W, o, W.stride(0), rule, S,
                           ws, stream)
    return h_acc, h, S


def global_scale(W: torch.Tensor, rule: int = GS_AMAX_448, stream=None) -> torch.Tensor:
    b, o, n, ldw, sw = _bmat(W)
    S = torch.empty(b, dtype=torch.float32, device=W.device)
    ws = torch.zeros(max(1, nvfp4_global_scale_workspace_size(b, o, n)), dtype=torch.uint8,
                     device=W.device)
    nvfp4_global_scale(W, b, o, n, ldw, sw, rule, S, ws, stream)
    return S


def scale_search(W: torch.Tensor, h: torch.Tensor | None, S: torch.Tensor, objective: int,
                 lo: int = -9, hi: int = 6, exhaustive: bool = False, with_stats: bool = True,
                 stream=None):
    """Scale search + pack over W [out, in] or [batch, out, in]; h [in] or [batch, in]."""
    b, o, n, ldw, sw = _bmat(W)
    shp = (o, n // 16) if W.dim() == 2 else (b, o, n // 16)
    dev = W.device
    scales = torch.empty(shp, dtype=torch.uint8, device=dev)
    packed = torch.empty(shp[:-1] + (n // 2,), dtype=torch.uint8, device=dev)
    loss = torch.empty(shp, dtype=torch.float32, device=dev) if with_stats else None
    offset = torch.empty(shp, dtype=torch.int8, device=dev) if with_stats else None
    stride_h = 0
    if objective == WMSE:
        if h is None:
            raise ValueError("WMSE needs h")
        stride_h = h.stride(0) if h.dim() == 2 else 0
    nvfp4_scale_search(W, b, o, n, ldw, sw, 16, h if objective == WMSE else None, stride_h,
                       objective, lo, hi, exhaustive, S, scales, packed, loss, offset, stream)
    return {"scales": scales, "packed": packed, "loss": loss, "offset": offset}


def scale_search_rules(W: torch.Tensor, h: torch.Tensor | None, S: torch.Tensor, rules,
                       with_stats: bool = True, stream=None) -> list[dict]:
    """Several rules (objective, lo, hi, exhaustive) over W [out, in] or [batch, out, in] in one
    call; returns one output dict per rule, as scale_search would."""
    b, o, n, ldw, sw = _bmat(W)
    shp = (o, n // 16) if W.dim() == 2 else (b, o, n // 16)
    dev = W.device
    outs, specs = [], []
    for objective, lo, hi, exhaustive in rules:
        r = {"scales": torch.empty(shp, dtype=torch.uint8, device=dev),
             "packed": torch.empty(shp[:-1] + (n // 2,), dtype=torch.uint8, device=dev),
             "loss": torch.empty(shp, dtype=torch.float32, device=dev) if with_stats else None,
             "offset": torch.empty(shp, dtype=torch.int8, device=dev) if with_stats else None}
        outs.append(r)
        specs.append(dict(r, objective=objective, lo=lo, hi=hi, exhaustive=exhaustive))
    wmse = any(objective == WMSE for objective, *_ in rules)
    if wmse and h is None:
        raise ValueError("WMSE needs h")
    stride_h = (h.stride(0) if h.dim() == 2 else 0) if wmse else 0
    nvfp4_scale_search_rules(W, b, o, n, ldw, sw, 16, h if wmse else None, stride_h, S, specs,
                             stream)
    return outs


def scale_search_scored(W: torch.Tensor, h: torch.Tensor | None, S: torch.Tensor, objective: int,
                        centre_lo: int = -8, stream=None) -> int:
    """Number of (group, code) candidates the exhaustive search scores on these inputs (centre
    block at base + centre_lo: -8 for scale_search's exhaustive mode, the window's lo when a
    16-code window and the exhaustive rule share one scale_search_rules launch)."""
    b, o, n, ldw, sw = _bmat(W)
    stride_h = 0
    if objective == WMSE:
        if h is None:
            raise ValueError("WMSE needs h")
        stride_h = h.stride(0) if h.dim() == 2 else 0
    count = torch.zeros(1, dtype=torch.int64, device=W.device)
    nvfp4_scale_search_scored(W, b, o, n, ldw, sw, 16, h if objective == WMSE else None, stride_h,
                              objective, centre_lo, S, count, stream)
    return int(count.item())


def scale_search_proposal(W: torch.Tensor, h: torch.Tensor | None, S: torch.Tensor, objective: int,
                          center: torch.Tensor, incoming: torch.Tensor | None = None,
                          lo: int = -4, hi: int = 4, with_stats: bool = True, stream=None):
    """Proposal-centred search + pack: window lo..hi around center[...] (uint8, shaped like the
    scales), the incoming codes (or None) scored first and kept on ties."""
    b, o, n, ldw, sw = _bmat(W)
    shp = (o, n // 16) if W.dim() == 2 else (b, o, n // 16)
    dev = W.device
    scales = torch.empty(shp, dtype=torch.uint8, device=dev)
    packed = torch.empty(shp[:-1] + (n // 2,), dtype=torch.uint8, device=dev)
    loss = torch.empty(shp, dtype=torch.float32, device=dev) if with_stats else None
    offset = torch.empty(shp, dtype=torch.int8, device=dev) if with_stats else None
    stride_h = 0
    if objective == WMSE:
        if h is None:
            raise ValueError("WMSE needs h")
        stride_h = h.stride(0) if h.dim() == 2 else 0
    for name, t in (("center", center), ("incoming", incoming)):
        if t is not None and (tuple(t.shape) != shp or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous uint8 tensor of shape {shp}")
    nvfp4_scale_search_proposal(W, b, o, n, ldw, sw, 16, h if objective == WMSE else None,
                                stride_h, objective, lo, hi, center, incoming, S, scales, packed,
                                loss, offset, stream)
    return {"scales": scales, "packed": packed, "loss": loss, "offset": offset}


def quantize_activations(X: torch.Tensor, objective: int = MSE, lo: int = -3, hi: int = 7,
                         rule: int = GS_AMAX_256, h: torch.Tensor | None = None, stream=None):
    """Dynamic per-tensor S and the scale search + pack of X [tokens, in] in two kernels."""
    T, n = X.shape
    if X.stride(1) != 1:
        raise ValueError("X rows must be contiguous")
    dev = X.device
    S = torch.empty(1, dtype=torch.float32, device=dev)
    scales = torch.empty((T, n // 16), dtype=torch.uint8, device=dev)
    packed = torch.empty((T, n // 2), dtype=torch.uint8, device=dev)
    ws = torch.empty(max(16, nvfp4_quantize_activations_workspace_size(T, n)), dtype=torch.uint8,
                     device=dev)
    nvfp4_quantize_activations(X, T, n, X.stride(0), objective, h if objective == WMSE else None,
                               lo, hi, rule, S, scales, packed, ws, stream)
    return {"S": S, "scales": scales, "packed": packed}


def gptq(W: torch.Tensor, U: torch.Tensor, h: torch.Tensor | None, S: torch.Tensor,
         objective: int = WMSE, lo: int = -9, hi: int = 6, with_final: bool = False, stream=None):
    """GPTQ over W [out, in] with the window search as local quantiser (U: upper factor of the
    damped inverse Hessian, float32 [in, in])."""
    o, n = W.shape
    if W.stride(1) != 1:
        raise ValueError("W rows must be contiguous")
    dev = W.device
    scales = torch.empty((o, n // 16), dtype=torch.uint8, device=dev)
    packed = torch.empty((o, n // 2), dtype=torch.uint8, device=dev)
    W_final = torch.empty((o, n), dtype=torch.float32, device=dev) if with_final else None
    ws = torch.empty(max(16, nvfp4_gptq_workspace_size(o, n)), dtype=torch.uint8, device=dev)
    nvfp4_gptq(W, o, n, W.stride(0), U.contiguous(), h if objective == WMSE else None, objective,
               lo, hi, S, scales, packed, W_final, ws, stream)
    return {"scales": scales, "packed": packed, "W_final": W_final}


def output_error(X: torch.Tensor, W: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                 S: torch.Tensor, err: torch.Tensor | None = None, accumulate: bool = False,
                 stream=None) -> torch.Tensor:
    """Per-row layer-output error err[o] = sum_t (X (W - W_hat)^T)[t, o]^2 (float64 [out])."""
    T, n = X.shape
    o = W.shape[0]
    if X.stride(1) != 1 or W.stride(1) != 1:
        raise ValueError("X and W rows must be contiguous")
    if err is None:
        err = torch.empty(o, dtype=torch.float64, device=X.device)
    ws = torch.empty(max(16, nvfp4_output_error_workspace_size(T, o, n)), dtype=torch.uint8,
                     device=X.device)
    nvfp4_output_error(X, T, n, X.stride(0), W, o, W.stride(0), scales.contiguous(),
                       packed.contiguous(), S, err, accumulate, ws, stream)
    return err


def pack(W: torch.Tensor, scales: torch.Tensor, S: torch.Tensor, stream=None) -> torch.Tensor:
    b, o, n, ldw, sw = _bmat(W)
    packed = torch.empty(scales.shape[:-1] + (n // 2,), dtype=torch.uint8, device=W.device)
    nvfp4_pack(W, b, o, n, ldw, sw, scales, S, packed, stream)
    return packed


def _empty(W: Matrix, shape, dtype, stream):
    """A tensor on the matrices' device that belongs to the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=W.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=W.device)


def linear(W: Matrix, X: torch.Tensor, bias: torch.Tensor | None = None, activation: int = ACT_NONE,
           residual: torch.Tensor | None = None, seg_offsets: torch.Tensor | None = None,
           with_pre: bool = False, stream=None):
    """act(X W^T + bias) + residual of X [tokens, in], bias [batch, out], residual [tokens, out]; returns
    Y [tokens, out], or (Y, Z) with the values before the activation. seg_offsets int64 [batch + 1]: which
    rows belong to which matrix of a batch; rows behind the last are not written. No gradient is
    recorded: linear_backward computes it."""
    T = X.shape[0]
    Y = _empty(W, (T, W.out), X.dtype, stream)
    Z = _empty(W, (T, W.out), X.dtype, stream) if with_pre else None
    need = nvfp4_linear_workspace_size(X.dtype, T, W.batch, W.out, W.inp)
    ws = _empty(W, need, torch.uint8, stream) if need else None
    nvfp4_linear(W, X, T, seg_offsets, bias, activation, residual, Z, Y, ws, stream)
    return (Y, Z) if with_pre else Y


def gated(W_gate: Matrix, W_up: Matrix, X: torch.Tensor, activation: int = ACT_SILU,
          seg_offsets: torch.Tensor | None = None, with_pre: bool = False, stream=None):
    """act(X W_gate^T) * (X W_up^T) of X [tokens, in]; returns H [tokens, out], or (H, G, U) with the two
    products. Rows and gradients as in linear."""
    T, W = X.shape[0], W_gate
    H = _empty(W, (T, W.out), X.dtype, stream)
    G, U = (_empty(W, (T, W.out), X.dtype, stream) if with_pre else None for _ in range(2))
    need = nvfp4_gated_workspace_size(X.dtype, T, W.batch, W.out, W.inp)
    ws = _empty(W, need, torch.uint8, stream) if need else None
    nvfp4_gated(W, W_up, X, T, seg_offsets, activation, G, U, H, ws, stream)
    return (H, G, U) if with_pre else H


def linear_backward(W: Matrix, dY: torch.Tensor, Z: torch.Tensor | None = None, activation: int = ACT_NONE,
                    seg_offsets: torch.Tensor | None = None, with_bias: bool = False, stream=None) -> dict:
    """Gradients of linear from dY [tokens, out] (the residual's is dY itself) and, with an activation, Z:
    dX [tokens, in], dZ [tokens, out] (None without an activation: dY) and dbias float32 [batch, out]
    (None unless asked for)."""
    T = dY.shape[0]
    dX = _empty(W, (T, W.inp), dY.dtype, stream)
    dZ = _empty(W, (T, W.out), dY.dtype, stream) if activation != ACT_NONE else None
    dbias = _empty(W, (W.batch, W.out), torch.float32, stream) if with_bias else None
    need = nvfp4_linear_backward_workspace_size(dY.dtype, T, W.batch, W.out, W.inp, with_bias)
    ws = _empty(W, need, torch.uint8, stream) if need else None
    nvfp4_linear_backward(W, dY, T, seg_offsets, activation, Z, dZ, dbias, dX, ws, stream)
    return {"dX": dX, "dZ": dZ, "dbias": dbias}


def gated_backward(W_gate: Matrix, W_up: Matrix, dH: torch.Tensor, G: torch.Tensor, U: torch.Tensor,
                   activation: int = ACT_SILU, seg_offsets: torch.Tensor | None = None,
                   stream=None) -> dict:
    """Gradients of gated from dH, G and U [tokens, out]: dX [tokens, in], dG and dU [tokens, out]."""
    T, W = dH.shape[0], W_gate
    dX = _empty(W, (T, W.inp), dH.dtype, stream)
    dG, dU = (_empty(W, (T, W.out), dH.dtype, stream) for _ in range(2))
    need = nvfp4_gated_backward_workspace_size(dH.dtype, T, W.batch, W.out, W.inp)
    ws = _empty(W, need, torch.uint8, stream) if need else None
    nvfp4_gated_backward(W, W_up, dH, T, seg_offsets, activation, G, U, dG, dU, dX, ws, stream)
    return {"dX": dX, "dG": dG, "dU": dU}


def _kv_empty(cache: KVCache, shape, dtype, stream):
    """A tensor on the cache's device that belongs to the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=cache.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=cache.device)


def kv_append(cache: KVCache, layer: int, K: torch.Tensor, V: torch.Tensor, cu_tokens: torch.Tensor,
              slots: torch.Tensor | None = None, lo: int = -3, hi: int = 7, stream=None) -> None:
    """Quantise new rows K, V [tokens, heads, head_dim] into the pages of their slots: item i's rows
    cu_tokens[i] .. cu_tokens[i+1] - 1 are the last tokens of slot slots[i] (None: slot i)."""
    nvfp4_kv_append(cache, layer, K, V, cu_tokens, slots, cu_tokens.numel() - 1, lo, hi, stream)


def kv_read(cache: KVCache, layer: int, tokens: int, cu_tokens: torch.Tensor,
            slots: torch.Tensor | None = None, dtype: torch.dtype = torch.bfloat16, stream=None):
    """The cached values of the items' last rows: (K, V), each [tokens, heads, head_dim]; rows behind
    cu_tokens[-1] are not written."""
    shape = (tokens, cache.heads, cache.head_dim)
    K, V = (_kv_empty(cache, shape, dtype, stream) for _ in range(2))
    nvfp4_kv_read(cache, layer, K, V, tokens, cu_tokens, slots, cu_tokens.numel() - 1, stream)
    return K, V


def kv_attention(cache: KVCache, layer: int, Q: torch.Tensor, cu_tokens: torch.Tensor,
                 slots: torch.Tensor | None = None, max_q: int | None = None,
                 max_kv: int | None = None, scale: float | None = None, causal: bool = True,
                 window: int = 0, stream=None):
    """Attention of Q [tokens, q_heads, head_dim] over the cached keys and values; returns
    (out like Q, lse float32 [tokens, q_heads]; rows behind cu_tokens[-1] are not written). max_q and max_kv bound the items' rows and lengths
    (None: all rows, the table's capacity). Tight bounds give faster kernels: a decode step passes
    max_q=1, and a batch of more than 1,024 items always its largest item's rows."""
    T, q_heads, D = Q.shape
    seqs = cu_tokens.numel() - 1
    max_q = T if max_q is None else max_q
    max_kv = cache.table.shape[1] * cache.page_size if max_kv is None else max_kv
    out = _kv_empty(cache, (T, q_heads, D), Q.dtype, stream)
    lse = _kv_empty(cache, (T, q_heads), torch.float32, stream)
    need = nvfp4_kv_attention_workspace_size(cache, Q.dtype, T, q_heads, seqs, max_q, max_kv)
    ws = _kv_empty(cache, need, torch.uint8, stream) if need else None
    nvfp4_kv_attention(cache, layer, Q, cu_tokens, slots, seqs, max_q, max_kv,
                       D ** -0.5 if scale is None else scale, causal, window, out, lse, ws, stream)
    return out, lse


def _pages_space(cache: KVCache, n: int, stream):
    return _kv_empty(cache, max(16, nvfp4_kv_pages_workspace_size(cache, n)), torch.uint8, stream)


def kv_reserve(cache: KVCache, slots: torch.Tensor, counts: torch.Tensor, stream=None) -> torch.Tensor:
    """Room for counts[i] more tokens in slots[i]; returns the device status (KV_DONE, ...) [1]."""
    status = _kv_empty(cache, 1, torch.int32, stream)
    n = slots.numel()
    nvfp4_kv_reserve(cache, slots, counts, n, status, _pages_space(cache, n, stream), stream)
    return status


def kv_fork(cache: KVCache, parents: torch.Tensor, children: torch.Tensor, stream=None) -> torch.Tensor:
    """Empty slots children[i] become copies of parents[i]; returns the device status [1]."""
    status = _kv_empty(cache, 1, torch.int32, stream)
    n = parents.numel()
    nvfp4_kv_fork(cache, parents, children, n, status, _pages_space(cache, n, stream), stream)
    return status


def kv_free(cache: KVCache, slots: torch.Tensor, stream=None) -> torch.Tensor:
    """Empties slots; returns the device status [1]."""
    status = _kv_empty(cache, 1, torch.int32, stream)
    nvfp4_kv_free(cache, slots, slots.numel(), status, stream)
    return status


def kv_compact(cache: KVCache, stream=None) -> torch.Tensor:
    """Moves the used pages to the lowest numbers; returns how many there are, on the device [1]."""
    used = _kv_empty(cache, 1, torch.int32, stream)
    nvfp4_kv_compact(cache, used, _pages_space(cache, 0, stream), stream)
    return used
