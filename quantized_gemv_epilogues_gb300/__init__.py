"""Python binding of the GB300 (sm_103a) decode-MLP library ``libmt.so``.

Argument marshalling only: every call forwards device pointers, sizes and the
current CUDA stream to the C ABI declared in ``include/mt.h``; all work runs in
the library's CUDA kernels.  There is no CPU fallback: importing this package
fails with ImportError when ``libmt.so`` has not been built (build it with
``python -c "import __graft_entry__ as g; g.build()"``).

Calls (same names as the C ABI):

* :func:`mt_add_rmsnorm` -- residual add + RMSNorm, both outputs written.
* :func:`mt_swiglu_gateup` -- gate/up GEMV with the silu(gate) * up epilogue.
* :func:`mt_down_residual` -- down GEMV with the residual added in its epilogue.
* :func:`mt_linear_bias` -- projection GEMV with an optional bias (attention
  q/k/v/o, vocabulary projection).
* :func:`mt_prefill_swiglu_gateup`, :func:`mt_prefill_down_residual`,
  :func:`mt_prefill_linear_bias` -- the same epilogues for many activation
  rows (prefill) on the tcgen05 tensor cores, with a caller-owned workspace
  of :func:`mt_prefill_workspace_bytes` bytes.
* :func:`mt_rope_append` -- per-head RMSNorm and rotary positions (one or
  several axes) of q and k, k and v written to a paged cache.
* :func:`mt_paged_attention` -- attention of each sequence's new tokens over its
  pages, causal, with an optional window and always-visible first tokens
  (workspace of :func:`mt_paged_attention_workspace_bytes` bytes).
* :func:`mt_logit_penalties` -- biases, penalties for repeated tokens and
  allowed-token masks on logits.
* :func:`mt_pack_affine` / :func:`mt_unpack_affine` -- affine group packer.
* :func:`mt_pack_mx` -- MXFP8 / MXFP4 block-scaled packer (E8M0 scales).
* :func:`mt_mlp_plan_create` / :func:`mt_mlp_plan_run` / :func:`mt_mlp_plan_destroy`
  -- the warmed executor: L one-row layers as one persistent kernel.
* :func:`mt_mlp_stack_run_noalloc` -- the same pass without any allocation.

Tensors are ``torch.Tensor`` on the current CUDA device (bf16 activations,
uint8 packed codes, bf16 scales/biases); raw integer device pointers are also
accepted, in which case the sizes given are trusted.
"""
from __future__ import annotations

import ctypes
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmt.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: the CUDA library has not been built "
        "(python -c 'import __graft_entry__ as g; g.build()')")

_lib = ctypes.CDLL(LIB_PATH)

MT_OK, MT_ERR_NULL, MT_ERR_SHAPE, MT_ERR_GROUP, MT_ERR_ALIGN = 0, 1, 2, 3, 4
MT_ERR_FORMAT, MT_ERR_ALIAS, MT_ERR_CUDA, MT_ERR_TIMEOUT, MT_ERR_PAGE = 5, 6, 7, 8, 9
MT_BF16, MT_F32 = 0, 1
MT_W_BF16, MT_W_AFFINE8, MT_W_AFFINE4, MT_W_MXFP8, MT_W_MXFP4 = 0, 1, 2, 3, 4
MT_OPT_PDL, MT_OPT_GEMV, MT_OPT_TEST_BARRIER_EXTRA, MT_OPT_ACT_BITS = 0, 1, 2, 3

MT_ROPE_HALF, MT_ROPE_ADJACENT = 0, 1

_P, _I, _F, _L = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_int64
_SIGS = {
    "mt_add_rmsnorm": (_I, [_P, _P, _P, _F, _P, _P, _I, _I, _I, _P]),
    "mt_swiglu_gateup": (_I, [_P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _P]),
    "mt_down_residual": (_I, [_P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _P]),
    "mt_linear_bias": (_I, [_P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _P]),
    "mt_pack_affine": (_I, [_P, _I, _I, _I, _I, _P, _P, _P, _P]),
    "mt_unpack_affine": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P]),
    "mt_pack_mx": (_I, [_P, _I, _I, _I, _P, _P, _P]),
    "mt_prefill_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I, _I]),
    "mt_prefill_swiglu_gateup": (_I, [_P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _P, ctypes.c_size_t, _P]),
    "mt_prefill_down_residual": (_I, [_P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _P, ctypes.c_size_t, _P]),
    "mt_prefill_linear_bias": (_I, [_P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _P, ctypes.c_size_t, _P]),
    "mt_set_option": (_I, [_I, _I]),
    "mt_get_option": (_I, [_I]),
    "mt_status_string": (ctypes.c_char_p, [_I]),
    "mt_last_cuda_error": (_I, []),
    "mt_device_error": (_I, [_I]),
    "mt_version": (_I, []),
    "mt_mlp_plan_create": (_I, [_P, _I, _I, _I, _I, _I, _F, _P]),
    "mt_mlp_plan_run": (_I, [_P, _P, _P, _P, _P, _P]),
    "mt_mlp_plan_destroy": (_I, [_P]),
    "mt_rope_append": (_I, [_P, _L, _P, _L, _P, _L, _I, _P, _P, _F, _P, _I, _P, _P, _I, _I, _P, _L, _P, _P, _P]),
    "mt_paged_attention_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I, _I, _I]),
    "mt_paged_attention": (_I, [_P, _L, _I, _P, _P, _F, _I, _I, _P, _L, _I, _P, _P, ctypes.c_size_t, _P]),
    "mt_logit_penalties": (_I, [_P, _L, _P, _L, _I, _I, _I, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _I, _P, _L, _P]),
    "mt_mlp_stack_run_noalloc": (_I, [_P, _I, _I, _I, _I, _I, _F, _P, _P, _P, _P]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


class MlpLayer(ctypes.Structure):
    """``mt_mlp_layer``: one layer's device pointers."""
    _fields_ = [(n, _P) for n in ("norm_weight", "Wg", "Wu", "gu_scales", "gu_biases", "Wd",
                                  "d_scales", "d_biases")]


class MlpTrace(ctypes.Structure):
    """``mt_mlp_trace``: optional per-layer outputs (device pointers or NULL)."""
    _fields_ = [(n, _P) for n in ("out_sum", "out_norm", "h", "y")]


class PagedCache(ctypes.Structure):
    """``mt_paged_cache``: K and V pages and their strides in elements."""
    _fields_ = [("k", _P), ("v", _P), ("page_stride", _L), ("token_stride", _L), ("head_stride", _L),
                ("num_pages", _I), ("page_size", _I), ("kv_heads", _I), ("head_dim", _I)]


class PagedBatch(ctypes.Structure):
    """``mt_paged_batch``: one step's sequences, rows and page table."""
    _fields_ = [("q_start", _P), ("kv_len", _P), ("pages", _P), ("pages_ld", _L), ("B", _I), ("T", _I),
                ("max_pages", _I), ("max_q", _I)]


# The two as the calls below pass them: bytes, as building the structures takes 1 us more
_CACHE = struct.Struct("PPqqqiiii").pack
_BATCH = struct.Struct("PPPqiiii").pack


class MTError(RuntimeError):
    def __init__(self, status: int, call: str, what: str | None = None):
        self.status = status
        msg = what or _lib.mt_status_string(status).decode()
        if status == MT_ERR_CUDA:
            msg += f" (cudaError {_lib.mt_last_cuda_error()})"
        super().__init__(f"{call}: {msg}")


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_torch = None  # set by the first call that needs it


def _get_torch():
    global _torch
    import torch
    _torch = torch
    return torch


def _stream(stream):
    if stream is None:
        torch = _torch or _get_torch()
        if torch.cuda.is_initialized():
            # the handle itself: building a Stream object takes 3 us
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(st: int, call: str) -> None:
    if st != MT_OK:
        raise MTError(st, call)


def _rows_cols(t, cols_hint=None):
    if isinstance(t, int):
        raise TypeError("shape arguments are required with raw pointers")
    if t.dim() == 1:
        return 1, t.shape[0]
    return t.shape[0], t.shape[1]


def _odt(t, explicit):
    if explicit is not None:
        return explicit
    import torch
    return MT_F32 if t.dtype == torch.float32 else MT_BF16


def mt_add_rmsnorm(values, residual, weight, eps, out_sum, out_norm, M=None, d=None,
                   norm_dtype=None, stream=None):
    if M is None or d is None:
        M, d = _rows_cols(values)
    nd = _odt(out_norm, norm_dtype) if not isinstance(out_norm, int) else (norm_dtype or MT_BF16)
    _check(_lib.mt_add_rmsnorm(_ptr(values), _ptr(residual), _ptr(weight), float(eps),
                               _ptr(out_sum), _ptr(out_norm), M, d, nd, _stream(stream)),
           "mt_add_rmsnorm")


def mt_swiglu_gateup(x, Wg, Wu, scales, biases, group, out_h, M=None, d=None, f=None, fmt=None,
                     out_dtype=None, stream=None):
    if M is None or d is None:
        M, d = _rows_cols(x)
    if f is None:
        f = _rows_cols(out_h)[1]
    if fmt is None:
        raise TypeError("fmt (MT_W_BF16 / MT_W_AFFINE8 / MT_W_AFFINE4) is required")
    od = _odt(out_h, out_dtype) if not isinstance(out_h, int) else (out_dtype or MT_BF16)
    _check(_lib.mt_swiglu_gateup(_ptr(x), _ptr(Wg), _ptr(Wu), _ptr(scales), _ptr(biases),
                                 int(group), _ptr(out_h), M, d, f, int(fmt), od, _stream(stream)),
           "mt_swiglu_gateup")


def mt_down_residual(h, Wd, scales, biases, group, residual, out_y, M=None, f=None, d=None,
                     fmt=None, out_dtype=None, stream=None):
    if M is None or f is None:
        M, f = _rows_cols(h)
    if d is None:
        d = _rows_cols(out_y)[1]
    if fmt is None:
        raise TypeError("fmt (MT_W_BF16 / MT_W_AFFINE8 / MT_W_AFFINE4) is required")
    od = _odt(out_y, out_dtype) if not isinstance(out_y, int) else (out_dtype or MT_BF16)
    _check(_lib.mt_down_residual(_ptr(h), _ptr(Wd), _ptr(scales), _ptr(biases), int(group),
                                 _ptr(residual), _ptr(out_y), M, f, d, int(fmt), od,
                                 _stream(stream)),
           "mt_down_residual")


def mt_linear_bias(x, W, scales, biases, group, bias, out_y, M=None, K=None, N=None, fmt=None,
                   out_dtype=None, stream=None):
    if M is None or K is None:
        M, K = _rows_cols(x)
    if N is None:
        N = _rows_cols(out_y)[1]
    if fmt is None:
        raise TypeError("fmt (MT_W_BF16 / MT_W_AFFINE8 / MT_W_AFFINE4) is required")
    od = _odt(out_y, out_dtype) if not isinstance(out_y, int) else (out_dtype or MT_BF16)
    _check(_lib.mt_linear_bias(_ptr(x), _ptr(W), _ptr(scales), _ptr(biases), int(group),
                               _ptr(bias), _ptr(out_y), M, K, N, int(fmt), od, _stream(stream)),
           "mt_linear_bias")


def mt_prefill_workspace_bytes(M, K, N, group):
    return int(_lib.mt_prefill_workspace_bytes(int(M), int(K), int(N), int(group)))


def _ws(workspace, M, K, N, group):
    need = mt_prefill_workspace_bytes(M, K, N, group)
    if workspace is None:
        raise TypeError(f"a device workspace of at least {need} bytes is required")
    nbytes = workspace.numel() * workspace.element_size() if not isinstance(workspace, int) else need
    return _ptr(workspace), nbytes


def mt_prefill_swiglu_gateup(x, Wg, Wu, scales, biases, group, out_h, workspace, M=None, d=None, f=None,
                             fmt=None, out_dtype=None, workspace_bytes=None, stream=None):
    if M is None or d is None:
        M, d = _rows_cols(x)
    if f is None:
        f = _rows_cols(out_h)[1]
    if fmt is None:
        raise TypeError("fmt (MT_W_AFFINE8 / MT_W_AFFINE4) is required")
    od = _odt(out_h, out_dtype) if not isinstance(out_h, int) else (out_dtype or MT_BF16)
    wp, wb = _ws(workspace, M, d, f, group)
    _check(_lib.mt_prefill_swiglu_gateup(_ptr(x), _ptr(Wg), _ptr(Wu), _ptr(scales), _ptr(biases), int(group),
                                         _ptr(out_h), M, d, f, int(fmt), od, wp,
                                         workspace_bytes if workspace_bytes is not None else wb, _stream(stream)),
           "mt_prefill_swiglu_gateup")


def mt_prefill_down_residual(h, Wd, scales, biases, group, residual, out_y, workspace, M=None, f=None, d=None,
                             fmt=None, out_dtype=None, workspace_bytes=None, stream=None):
    if M is None or f is None:
        M, f = _rows_cols(h)
    if d is None:
        d = _rows_cols(out_y)[1]
    if fmt is None:
        raise TypeError("fmt (MT_W_AFFINE8 / MT_W_AFFINE4) is required")
    od = _odt(out_y, out_dtype) if not isinstance(out_y, int) else (out_dtype or MT_BF16)
    wp, wb = _ws(workspace, M, f, d, group)
    _check(_lib.mt_prefill_down_residual(_ptr(h), _ptr(Wd), _ptr(scales), _ptr(biases), int(group),
                                         _ptr(residual), _ptr(out_y), M, f, d, int(fmt), od, wp,
                                         workspace_bytes if workspace_bytes is not None else wb, _stream(stream)),
           "mt_prefill_down_residual")


def mt_prefill_linear_bias(x, W, scales, biases, group, bias, out_y, workspace, M=None, K=None, N=None, fmt=None,
                           out_dtype=None, workspace_bytes=None, stream=None):
    if M is None or K is None:
        M, K = _rows_cols(x)
    if N is None:
        N = _rows_cols(out_y)[1]
    if fmt is None:
        raise TypeError("fmt (MT_W_AFFINE8 / MT_W_AFFINE4) is required")
    od = _odt(out_y, out_dtype) if not isinstance(out_y, int) else (out_dtype or MT_BF16)
    wp, wb = _ws(workspace, M, K, N, group)
    _check(_lib.mt_prefill_linear_bias(_ptr(x), _ptr(W), _ptr(scales), _ptr(biases), int(group), _ptr(bias),
                                       _ptr(out_y), M, K, N, int(fmt), od, wp,
                                       workspace_bytes if workspace_bytes is not None else wb, _stream(stream)),
           "mt_prefill_linear_bias")


def mt_pack_affine(W, N, K, group, bits, q, scales, biases, stream=None):
    _check(_lib.mt_pack_affine(_ptr(W), int(N), int(K), int(group), int(bits), _ptr(q),
                               _ptr(scales), _ptr(biases), _stream(stream)), "mt_pack_affine")


def mt_pack_mx(W, N, K, bits, q, scales, stream=None):
    _check(_lib.mt_pack_mx(_ptr(W), int(N), int(K), int(bits), _ptr(q), _ptr(scales), _stream(stream)),
           "mt_pack_mx")


def mt_unpack_affine(q, scales, biases, N, K, group, bits, W, stream=None):
    _check(_lib.mt_unpack_affine(_ptr(q), _ptr(scales), _ptr(biases), int(N), int(K), int(group),
                                 int(bits), _ptr(W), _stream(stream)), "mt_unpack_affine")


def mt_mlp_plan_create(layers, d, f, group, fmt, eps) -> int:
    """Binds L layers (each a mapping with the ``mt_mlp_layer`` field names to
    tensors or device pointers; scale/bias fields may be None for bf16) and
    returns the plan handle (an int)."""
    arr = (MlpLayer * len(layers))()
    for i, ly in enumerate(layers):
        for name, _ in MlpLayer._fields_:
            setattr(arr[i], name, _ptr(ly.get(name)))
    plan = ctypes.c_void_p()
    _check(_lib.mt_mlp_plan_create(arr, len(layers), int(d), int(f), int(group), int(fmt),
                                   float(eps), ctypes.byref(plan)), "mt_mlp_plan_create")
    return plan.value


def mt_mlp_plan_run(plan, values, residual, out_y, trace=None, stream=None) -> None:
    """One pass over the plan's layers.  trace: None or a mapping with some of
    out_sum / out_norm / h / y (tensors [L][.] or device pointers)."""
    tr = None
    if trace is not None:
        tr = MlpTrace(*[_ptr(trace.get(n)) for n, _ in MlpTrace._fields_])
    _check(_lib.mt_mlp_plan_run(plan, _ptr(values), _ptr(residual), _ptr(out_y),
                                ctypes.byref(tr) if tr is not None else None, _stream(stream)),
           "mt_mlp_plan_run")


def mt_mlp_plan_destroy(plan) -> None:
    _check(_lib.mt_mlp_plan_destroy(plan), "mt_mlp_plan_destroy")


def mt_mlp_stack_run_noalloc(layers, d, f, group, fmt, eps, values, residual, out_y,
                             stream=None) -> None:
    """The stack pass with the library's static scratch instead of a plan's
    memory (see include/mt.h)."""
    arr = (MlpLayer * len(layers))()
    for i, ly in enumerate(layers):
        for name, _ in MlpLayer._fields_:
            setattr(arr[i], name, _ptr(ly.get(name)))
    _check(_lib.mt_mlp_stack_run_noalloc(arr, len(layers), int(d), int(f), int(group), int(fmt),
                                         float(eps), _ptr(values), _ptr(residual), _ptr(out_y),
                                         _stream(stream)), "mt_mlp_stack_run_noalloc")


def _on_device(call, **tensors):
    """Refuses tensors whose memory a kernel cannot read: all but the GPU's and
    pinned host memory (which has a device address of its own).  Called where
    not all are the GPU's (asked for each by name: a loop over them takes 2 us)."""
    for name, t in tensors.items():
        if t is not None and not t.is_cuda and t.numel() and not t.is_pinned():
            raise MTError(MT_ERR_NULL, call, f"{name}: a tensor on the GPU is required, this one is in host memory")


def _typed(name, t, dtype, dim):
    if t.dtype is not dtype or t.dim() != dim:
        raise TypeError(f"{name}: a {dim}-dimensional {dtype} tensor is required, got {t.dim()}-dimensional {t.dtype}")


def _flat(name, t, dtype, n=None):
    """Address of a contiguous one-dimensional tensor (of n entries), None for None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.dim() != 1:
        _typed(name, t, dtype, 1)
    if n is not None and t.numel() != n:
        raise ValueError(f"{name}: {n} entries are required")
    if not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor is required")
    return t.data_ptr()


def _head_rows(name, t, dtype, shape):
    """Address and row stride of a [T, H, D] tensor whose heads lie side by side."""
    if t.dtype is not dtype or t.shape != shape:
        _typed(name, t, dtype, 3)
        raise ValueError(f"{name}: shape {tuple(shape)} is required, got {tuple(t.shape)}")
    row, head, one = t.stride()
    T, H, D = shape
    if (one != 1 and D > 1) or (head != D and H > 1):
        raise ValueError(f"{name}: heads must lie side by side in a row")
    return t.data_ptr(), (row if T > 1 else H * D)


def _paged(k_cache, v_cache, pages, q_start, kv_len, T, max_q):
    """The cache and batch arguments and the cache's heads and head size, from tensors: caches [pages, page, heads, dim]
    (any strides with contiguous dim, the same for both), pages int32 [B, n],
    q_start int32 [B + 1], kv_len int32 [B]."""
    bf, i32 = _torch.bfloat16, _torch.int32
    if k_cache.dtype is not bf or v_cache.dtype is not bf or k_cache.dim() != 4:
        _typed("k_cache", k_cache, bf, 4)
        _typed("v_cache", v_cache, bf, 4)
    shape, st = k_cache.shape, k_cache.stride()
    if v_cache.shape != shape or v_cache.stride() != st:
        raise ValueError("k_cache and v_cache must have the same shape and strides")
    n, page, heads, dim = shape
    if st[3] != 1 and dim > 1:
        raise ValueError("k_cache: the last dimension must be contiguous")
    if pages.dtype is not i32 or pages.dim() != 2:
        _typed("pages", pages, i32, 2)
    B, width = pages.shape
    ld, one = pages.stride()
    if one != 1 and width > 1:
        raise ValueError("pages: the last dimension must be contiguous")
    cache = _CACHE(k_cache.data_ptr(), v_cache.data_ptr(), st[0], st[1], st[2], n, page, heads, dim)
    batch = _BATCH(_flat("q_start", q_start, i32, B + 1), _flat("kv_len", kv_len, i32, B), pages.data_ptr(),
                   ld if B > 1 else width, B, T, width, max_q if 0 < max_q < 1 << 31 else 1)
    return cache, batch, heads, dim


def mt_rope_append(q, k, v, positions, inv_freq, q_out, k_cache, v_cache, pages, q_start, kv_len, axis=None,
                   q_norm=None, k_norm=None, eps=1e-6, pairing=MT_ROPE_HALF, stream=None) -> None:
    """Rotary positions of q and k (after an optional per-head RMSNorm), k and v
    written to their cache positions.  q [T, q_heads, dim], k and v [T,
    kv_heads, dim] (bf16, rows at any stride); positions int32 [T] or [n_axes,
    T]; inv_freq float [rot / 2]; axis uint8 [rot / 2] or None (axis 0)."""
    torch = _torch or _get_torch()
    bf = torch.bfloat16
    shape = q.shape
    if len(shape) != 3:
        raise TypeError("q: a 3-dimensional tensor is required")
    T, H, D = shape
    cache, batch, kv_heads, dim = _paged(k_cache, v_cache, pages, q_start, kv_len, T, 1)
    if D != dim:
        raise ValueError(f"the cache's head size is {dim}, q's is {D}")
    kv_shape = (T, kv_heads, D)
    qp, qs = _head_rows("q", q, bf, shape)
    kp, ks = _head_rows("k", k, bf, kv_shape)
    vp, vs = _head_rows("v", v, bf, kv_shape)
    op, os_ = _head_rows("q_out", q_out, bf, shape)
    axes = 1
    if positions.dim() == 2:
        axes = positions.shape[0]
    elif positions.dim() != 1:
        _typed("positions", positions, torch.int32, 2)
    if positions.dtype is not torch.int32 or not positions.is_contiguous() or positions.numel() != axes * T:
        _typed("positions", positions, torch.int32, positions.dim())
        raise ValueError(f"positions: contiguous rows of {T} tokens are required")
    half = inv_freq.numel()
    if not (q.is_cuda and k.is_cuda and v.is_cuda and positions.is_cuda and inv_freq.is_cuda and q_out.is_cuda and k_cache.is_cuda
            and v_cache.is_cuda and pages.is_cuda and q_start.is_cuda and kv_len.is_cuda and (axis is None or axis.is_cuda)
            and (q_norm is None or q_norm.is_cuda) and (k_norm is None or k_norm.is_cuda)):
        _on_device("mt_rope_append", q=q, k=k, v=v, positions=positions, inv_freq=inv_freq, q_out=q_out, k_cache=k_cache,
                   v_cache=v_cache, pages=pages, q_start=q_start, kv_len=kv_len, axis=axis, q_norm=q_norm, k_norm=k_norm)
    _check(_lib.mt_rope_append(qp, qs, kp, ks, vp, vs, H, _flat("q_norm", q_norm, bf, D), _flat("k_norm", k_norm, bf, D), eps,
                               positions.data_ptr(), axes, _flat("inv_freq", inv_freq, torch.float32),
                               _flat("axis", axis, torch.uint8, half), 2 * half, pairing, op, os_,
                               cache, batch, _stream(stream)), "mt_rope_append")


def mt_paged_attention_workspace_bytes(T, B, q_heads, kv_heads, head_dim) -> int:
    return int(_lib.mt_paged_attention_workspace_bytes(int(T), int(B), int(q_heads), int(kv_heads), int(head_dim)))


def mt_paged_attention(q, k_cache, v_cache, pages, q_start, kv_len, max_q, scale, out, workspace, lse=None, window=0,
                       sinks=0, stream=None) -> None:
    """Attention of the new tokens q [T, q_heads, dim] over the paged cache;
    out [T, q_heads, dim] (bf16 or fp32), lse float [T, q_heads] or None,
    window 0 for none.  max_q: the most new tokens of a sequence (a hint)."""
    torch = _torch or _get_torch()
    shape = q.shape
    if len(shape) != 3:
        raise TypeError("q: a 3-dimensional tensor is required")
    T, H, D = shape
    cache, batch, _, dim = _paged(k_cache, v_cache, pages, q_start, kv_len, T, max_q)
    if D != dim:
        raise ValueError(f"the cache's head size is {dim}, q's is {D}")
    qp, qs = _head_rows("q", q, torch.bfloat16, shape)
    f32 = out.dtype is torch.float32
    op, os_ = _head_rows("out", out, torch.float32 if f32 else torch.bfloat16, shape)
    lp = None
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.shape != (T, H) or not lse.is_contiguous():
            _typed("lse", lse, torch.float32, 2)
            raise ValueError(f"lse: a contiguous tensor of shape {(T, H)} is required")
        lp = lse.data_ptr()
    if not workspace.is_contiguous():
        raise ValueError("workspace: a contiguous tensor is required")
    # a C int would take the lower 32 bits of what is wider than any text
    if not -1 < window < 1 << 31:
        window = -1 if window < 0 else 0x7FFFFFFF
    if not -1 < sinks < 1 << 31:
        sinks = -1 if sinks < 0 else 0x7FFFFFFF
    if not (q.is_cuda and k_cache.is_cuda and v_cache.is_cuda and pages.is_cuda and q_start.is_cuda and kv_len.is_cuda and out.is_cuda
            and workspace.is_cuda and (lse is None or lse.is_cuda)):
        _on_device("mt_paged_attention", q=q, k_cache=k_cache, v_cache=v_cache, pages=pages, q_start=q_start, kv_len=kv_len, out=out,
                   workspace=workspace, lse=lse)
    _check(_lib.mt_paged_attention(qp, qs, H, cache, batch, scale, window, sinks, op, os_,
                                   MT_F32 if f32 else MT_BF16, lp, workspace.data_ptr(), workspace.nbytes,
                                   _stream(stream)), "mt_paged_attention")


def mt_logit_penalties(logits, out, history=None, history_start=None, prompt_len=None, repetition=None, presence=None,
                       frequency=None, bias_ids=None, bias_values=None, bias_start=None, allowed=None,
                       stream=None) -> None:
    """Biases, penalties for repeated tokens and allowed-token masks on logits
    [B, V] (bf16 or fp32) into out (which may be logits); ragged int32 history
    and bias lists with [B + 1] starts, allowed int32 [B, words] bits."""
    torch = _torch or _get_torch()
    i32, f32, dt = torch.int32, torch.float32, logits.dtype
    shape = logits.shape
    if (dt is not f32 and dt is not torch.bfloat16) or len(shape) != 2 or out.dtype is not dt:
        _typed("logits", logits, f32 if dt is f32 else torch.bfloat16, 2)
        _typed("out", out, dt, 2)
    B, V = shape
    ld, one = logits.stride()
    out_ld, out_one = out.stride()
    if out.shape != shape or (V > 1 and (one != 1 or out_one != 1)):
        raise ValueError("logits and out must have the same shape and contiguous rows")
    if B == 1:
        ld = out_ld = V
    hist = start = prompt = ids = values = bstart = ap = None
    n_hist = n_bias = ald = 0
    # an empty tensor has no address: a list without entries is no list
    if history is not None:
        n_hist = history.numel()
        hist = _flat("history", history, i32) or None
        start = _flat("history_start", history_start, i32, B + 1) if hist else None
        prompt = _flat("prompt_len", prompt_len, i32, B) if hist else None
    if bias_ids is not None:
        n_bias = bias_ids.numel()
        ids = _flat("bias_ids", bias_ids, i32) or None
        values = _flat("bias_values", bias_values, f32, n_bias) if ids else None
        bstart = _flat("bias_start", bias_start, i32, B + 1) if ids else None
    if allowed is not None:
        if allowed.dtype is not i32 or allowed.dim() != 2:
            _typed("allowed", allowed, i32, 2)
        rows, words = allowed.shape
        ald, one = allowed.stride()
        if rows != B or (words > 1 and one != 1):
            raise ValueError(f"allowed: {B} contiguous rows are required")
        if words * 32 < V:
            raise ValueError(f"allowed: {(V + 31) // 32} words a row are required")
        ap = allowed.data_ptr()
        if B == 1:
            ald = words
    if (B | V | n_hist | n_bias) >> 31:
        raise ValueError("logits and lists of fewer than 2^31 rows, tokens and entries are required")
    if not (logits.is_cuda and out.is_cuda and (hist is None or history.is_cuda) and (start is None or history_start.is_cuda)
            and (prompt is None or prompt_len.is_cuda) and (repetition is None or repetition.is_cuda)
            and (presence is None or presence.is_cuda) and (frequency is None or frequency.is_cuda)
            and (ids is None or bias_ids.is_cuda) and (values is None or bias_values.is_cuda)
            and (bstart is None or bias_start.is_cuda)
            and (allowed is None or allowed.is_cuda)):
        _on_device("mt_logit_penalties", logits=logits, out=out, history=history, history_start=history_start,
                   prompt_len=prompt_len, repetition=repetition, presence=presence, frequency=frequency, bias_ids=bias_ids,
                   bias_values=bias_values, bias_start=bias_start, allowed=allowed)
    _check(_lib.mt_logit_penalties(logits.data_ptr(), ld, out.data_ptr(), out_ld, MT_F32 if dt is f32 else MT_BF16, B, V,
                                   hist, start, prompt, n_hist, _flat("repetition", repetition, f32, B),
                                   _flat("presence", presence, f32, B), _flat("frequency", frequency, f32, B), ids, values,
                                   bstart, n_bias, ap, ald, _stream(stream)), "mt_logit_penalties")


def mt_set_option(opt: int, value: int) -> None:
    _check(_lib.mt_set_option(int(opt), int(value)), "mt_set_option")


def mt_get_option(opt: int) -> int:
    return _lib.mt_get_option(int(opt))


def mt_status_string(status: int) -> str:
    return _lib.mt_status_string(int(status)).decode()


def mt_last_cuda_error() -> int:
    return _lib.mt_last_cuda_error()


def mt_device_error(clear: bool = False) -> int:
    return _lib.mt_device_error(1 if clear else 0)


def mt_version() -> int:
    return _lib.mt_version()


def raw(name: str):
    """The ctypes function of a C-ABI entry point (for tests that call the ABI
    directly with raw pointers)."""
    return getattr(_lib, name)
