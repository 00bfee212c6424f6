"""Python binding of the contextual-sparsity sparse FFN library (libcs.so).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch provides device memory and streams.  The functions carry the
C ABI's names (include/cs.h) and raise :class:`CsError` on a non-OK status.
There is no fallback: if libcs.so is missing, importing the binding's loader
raises.
"""
from __future__ import annotations

import ctypes as C
import importlib.util
import os
import threading

import torch

from . import build as _build

_lock = threading.Lock()
_lib = None

CS_F32, CS_F16, CS_BF16 = 0, 1, 2
CS_SEL_TOPK, CS_SEL_THRESHOLD, CS_SEL_EXACT = 0, 1, 2
CS_STACK_SEQUENTIAL, CS_STACK_LOOKAHEAD = 0, 1
CS_ACT_RELU, CS_ACT_SILU = 0, 1
CS_DEVERR_INDEX, CS_DEVERR_COUNT, CS_DEVERR_TIMEOUT = 0x1, 0x2, 0x4

_TORCH_DT = {torch.float32: CS_F32, torch.float16: CS_F16, torch.bfloat16: CS_BF16}

# every symbol include/cs.h declares
EXPORTS = ["cs_version", "cs_status_string", "cs_last_error", "cs_workspace_size",
           "cs_workspace_init", "cs_get_device_error", "cs_pack_transpose", "cs_predict",
           "cs_select", "cs_sparse_ffn", "cs_exact_ffn", "cs_union_mask", "cs_decode_stack",
           "cs_stack_release", "cs_sparse_ffn_noalloc", "cs_decode_layer", "cs_permute_rows",
           "cs_hot_order", "cs_fit_scratch_size", "cs_fit_predictor", "cs_sparse_attention",
           "cs_decode_attention", "cs_qcache_workspace_size", "cs_qcache_append", "cs_qcache_read",
           "cs_qcache_attention", "cs_qcache_evict", "cs_qcache_trim"]


class CsError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"{msg} (status {status})")
        self.status = status


class _Pred(C.Structure):
    _fields_ = [("d", C.c_int), ("r", C.c_int), ("f", C.c_int), ("dtype", C.c_int),
                ("ld_down", C.c_int), ("ld_up", C.c_int), ("p_down", C.c_void_p),
                ("p_up", C.c_void_p)]


class _Layer(C.Structure):
    _fields_ = [("d", C.c_int), ("f", C.c_int), ("dtype", C.c_int), ("ld", C.c_int),
                ("w_gate", C.c_void_p), ("w_up", C.c_void_p), ("w_down_t", C.c_void_p),
                ("bias", C.c_void_p), ("act", C.c_int)]


class _Attn(C.Structure):
    _fields_ = [("d", C.c_int), ("n_heads", C.c_int), ("d_head", C.c_int), ("dtype", C.c_int),
                ("w_q", C.c_void_p), ("w_o_t", C.c_void_p)]


class _Sel(C.Structure):
    _fields_ = [("mode", C.c_int), ("k", C.c_int), ("tau", C.c_float), ("hot", C.c_int)]


class _QCache(C.Structure):
    _fields_ = [("batch", C.c_int), ("n_heads", C.c_int), ("d_head", C.c_int), ("capacity", C.c_int),
                ("ld_batch", C.c_int64), ("ld_head", C.c_int64), ("k", C.c_void_p), ("v", C.c_void_p),
                ("k_scale", C.c_void_p), ("v_scale", C.c_void_p), ("weight", C.c_void_p), ("pos", C.c_void_p)]


class _Rows(C.Structure):   # cs_head_rows, for callers of the C ABI through lib()
    _fields_ = [("data", C.c_void_p), ("dtype", C.c_int), ("ld_batch", C.c_int64), ("ld_token", C.c_int64),
                ("ld_head", C.c_int64)]


def library_path() -> str:
    return _build.LIB


def lib():
    """Load libcs.so (built by ``build()``); raises if it is missing."""
    global _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise ImportError(f"CUDA library {path} is missing; run "
                                  "contextual_sparsity_sparse_gb300.build.build() first")
            L = C.CDLL(path)
            P, I, S, U = C.c_void_p, C.c_int, C.c_size_t, C.c_uint32
            L.cs_version.restype = C.c_char_p
            L.cs_status_string.argtypes = [I]
            L.cs_status_string.restype = C.c_char_p
            L.cs_last_error.restype = C.c_char_p
            L.cs_workspace_size.argtypes = [I, I, I, I]
            L.cs_workspace_size.restype = S
            L.cs_workspace_init.argtypes = [P, S, P]
            L.cs_get_device_error.argtypes = [P, P, I, C.POINTER(U)]
            L.cs_pack_transpose.argtypes = [P, I, I, I, I, P, I, I, P]
            L.cs_predict.argtypes = [C.POINTER(_Pred), P, I, P, P, S, P]
            L.cs_select.argtypes = [P, I, I, C.POINTER(_Sel), P, P, P, P, S, P]
            L.cs_sparse_ffn.argtypes = [C.POINTER(_Layer), P, I, P, P, P, P, S, P]
            L.cs_exact_ffn.argtypes = [C.POINTER(_Layer), P, P, P, P, P, P, C.c_float, P, S, P]
            L.cs_union_mask.argtypes = [P, I, I, P, P, P, P, S, P]
            L.cs_decode_stack.argtypes = [C.POINTER(_Layer), C.POINTER(_Pred), I, P, C.c_float,
                                          C.POINTER(_Sel), I, P, P, P, S, P, P]
            L.cs_sparse_ffn_noalloc.argtypes = [C.POINTER(_Layer), P, I, P, P, P, P]
            L.cs_decode_layer.argtypes = [C.POINTER(_Layer), C.POINTER(_Pred), P, P, C.POINTER(_Sel),
                                          P, S, P, P, P]
            L.cs_permute_rows.argtypes = [P, I, I, P, I, I, I, P, I, P]
            L.cs_hot_order.argtypes = [P, I, P]
            L.cs_sparse_attention.argtypes = [C.POINTER(_Attn), P, P, P, P, P, I, P, P, S, P]
            L.cs_decode_attention.argtypes = [C.POINTER(_Attn), C.POINTER(_Pred), P, P, C.POINTER(_Sel),
                                              P, P, I, P, S, P, P, P]
            L.cs_fit_scratch_size.argtypes = [I, I, I, I]
            L.cs_fit_scratch_size.restype = S
            L.cs_fit_predictor.argtypes = [C.POINTER(_Layer), C.POINTER(_Pred), P, I, C.c_double, P, S, P]
            QC, HR = C.POINTER(_QCache), C.POINTER(_Rows)
            L.cs_qcache_workspace_size.argtypes = [I] * 6
            L.cs_qcache_workspace_size.restype = S
            L.cs_qcache_append.argtypes = [QC, HR, HR, I, P, P, P, P, P, S, P]
            L.cs_qcache_read.argtypes = [QC, HR, HR, I, P, P, P, S, P]
            L.cs_qcache_attention.argtypes = [QC, HR, I, I, P, P, P, C.c_float, C.c_float, P, HR, P, S, P]
            L.cs_qcache_evict.argtypes = [QC, P, I, I, P, I, I, P, P, S, P]
            L.cs_qcache_trim.argtypes = [QC, P, I, P, I, I, QC, P, S, P]
            for name in ("cs_workspace_init", "cs_get_device_error", "cs_pack_transpose",
                         "cs_predict", "cs_select", "cs_sparse_ffn", "cs_exact_ffn",
                         "cs_union_mask", "cs_decode_stack", "cs_stack_release",
                         "cs_sparse_ffn_noalloc", "cs_decode_layer", "cs_permute_rows", "cs_hot_order",
                         "cs_fit_predictor", "cs_sparse_attention", "cs_decode_attention", "cs_qcache_append",
                         "cs_qcache_read", "cs_qcache_attention", "cs_qcache_evict", "cs_qcache_trim"):
                getattr(L, name).restype = I
            _lib = L
    return _lib


def _check(status):
    if status != 0:
        L = lib()
        raise CsError(status, f"{L.cs_status_string(status).decode()}: {L.cs_last_error().decode()}")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    return t.data_ptr()


def _stream(s):
    if s is None:
        # the current stream's handle itself: building a torch.cuda.Stream around it costs more than a launch
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return s.cuda_stream if hasattr(s, "cuda_stream") else int(s)


def _dt(t):
    return _TORCH_DT[t.dtype]


class Predictor:
    """p_down [r, ld_down], p_up [f, ld_up]; d is the used width of p_down."""

    def __init__(self, p_down, p_up, d=None, r=None):
        self.p_down, self.p_up = p_down, p_up
        self.r, ldd = p_down.shape
        self.f, ldu = p_up.shape
        self.d = int(d if d is not None else ldd)
        if r is not None and r != self.r:
            raise ValueError("r does not match p_down")
        self.c = _Pred(self.d, self.r, self.f, _dt(p_down), ldd, ldu, _ptr(p_down), _ptr(p_up))


class FfnLayer:
    """Neuron-major layer: w_gate, w_up, w_down_t are [f, ld]; d is the used
    width (default ld).  w_up None gives the gate-only ReLU FFN."""

    def __init__(self, w_gate, w_down_t, w_up=None, bias=None, d=None, act=CS_ACT_RELU):
        self.w_gate, self.w_down_t, self.w_up, self.bias = w_gate, w_down_t, w_up, bias
        self.f, ld = w_gate.shape
        self.d = int(d if d is not None else ld)
        self.act = int(act)
        self.c = _Layer(self.d, self.f, _dt(w_gate), ld, _ptr(w_gate), _ptr(w_up), _ptr(w_down_t),
                        _ptr(bias), self.act)


def select_params(mode, k=0, tau=0.0, hot=0):
    """hot: an always-on prefix of neurons for a frequency-sorted layout (a
    multiple of 32); k and tau then apply to the tail (see include/cs.h)."""
    return _Sel(int(mode), int(k), float(tau), int(hot))


class Workspace:
    """Device workspace sized by cs_workspace_size and initialised once."""

    def __init__(self, d, f, r, B=1, device=None, stream=None):
        n = lib().cs_workspace_size(int(d), int(f), int(r), int(B))
        if n == 0:
            raise ValueError("bad workspace dimensions")
        self.nbytes = n
        self.buf = torch.empty(n + 256, dtype=torch.uint8, device=device or "cuda")
        base = self.buf.data_ptr()
        self.ptr = (base + 255) & ~255
        _check(lib().cs_workspace_init(self.ptr, self.nbytes, _stream(stream)))


def cs_version() -> str:
    return lib().cs_version().decode()


def cs_workspace_size(d, f, r, B=1) -> int:
    return int(lib().cs_workspace_size(int(d), int(f), int(r), int(B)))


def cs_get_device_error(ws: Workspace, stream=None, clear=False) -> int:
    v = C.c_uint32(0)
    _check(lib().cs_get_device_error(ws.ptr, _stream(stream), int(bool(clear)), C.byref(v)))
    return v.value


def cs_pack_transpose(src, dst, rows=None, cols=None, stream=None):
    """dst[c, r] = src[r, c] (with dtype conversion).  src [rows, ld_src],
    dst [cols, ld_dst]."""
    rows = src.shape[0] if rows is None else rows
    cols = src.shape[1] if cols is None else cols
    _check(lib().cs_pack_transpose(_ptr(src), _dt(src), int(rows), int(cols), src.shape[1],
                                   _ptr(dst), _dt(dst), dst.shape[1], _stream(stream)))


def cs_predict(pred: Predictor, x, scores, ws: Workspace, stream=None):
    B = x.shape[0] if x.dim() == 2 else 1
    _check(lib().cs_predict(C.byref(pred.c), _ptr(x), B, _ptr(scores), ws.ptr, ws.nbytes,
                            _stream(stream)))


def cs_select(scores, params, idx, count, mask=None, ws: Workspace | None = None, stream=None):
    B, f = (scores.shape if scores.dim() == 2 else (1, scores.shape[0]))
    _check(lib().cs_select(_ptr(scores), B, f, C.byref(params), _ptr(idx), _ptr(count),
                           _ptr(mask), ws.ptr if ws else None, ws.nbytes if ws else 0,
                           _stream(stream)))


def cs_sparse_ffn(layer: FfnLayer, x, idx, count, y, ws: Workspace, stream=None):
    B = x.shape[0] if x.dim() == 2 else 1
    _check(lib().cs_sparse_ffn(C.byref(layer.c), _ptr(x), B, _ptr(idx), _ptr(count), _ptr(y),
                               ws.ptr, ws.nbytes, _stream(stream)))


def cs_sparse_ffn_noalloc(layer: FfnLayer, x, idx, count, y, stream=None):
    """cs_sparse_ffn without a workspace (see include/cs.h): scratch comes from
    a fixed array inside the library, so nothing is allocated."""
    B = x.shape[0] if x.dim() == 2 else 1
    _check(lib().cs_sparse_ffn_noalloc(C.byref(layer.c), _ptr(x), B, _ptr(idx), _ptr(count),
                                       _ptr(y), _stream(stream)))


def cs_exact_ffn(layer: FfnLayer, x, preact, idx, count, y, ws: Workspace, mask=None, stream=None,
                 tau=0.0):
    """tau: the magnitude cut |act(g_j)| > tau (0 with relu: the exact mask g_j > 0)."""
    _check(lib().cs_exact_ffn(C.byref(layer.c), _ptr(x), _ptr(preact), _ptr(idx), _ptr(count),
                              _ptr(mask), _ptr(y), float(tau), ws.ptr, ws.nbytes, _stream(stream)))


def cs_union_mask(masks, f, umask, uidx, ucount, ws: Workspace | None = None, stream=None):
    B = masks.shape[0]
    _check(lib().cs_union_mask(_ptr(masks), B, int(f), _ptr(umask), _ptr(uidx), _ptr(ucount),
                               ws.ptr if ws else None, ws.nbytes if ws else 0, _stream(stream)))


class StackArgs:
    """The layer and predictor arrays of a stack, marshalled once, for
    repeated cs_decode_stack calls."""

    def __init__(self, layers, preds):
        self.L = len(layers)
        self.layers = (_Layer * self.L)(*[l.c for l in layers])
        self.preds = (_Pred * self.L)(*[p.c for p in preds]) if preds is not None else None


def cs_decode_stack(layers, preds, x, resid_scale, params, mode, ws: Workspace, s_main=None,
                    s_pred=None, trace_count=None, trace_idx=None):
    """x_0 -> x_L in place (see include/cs.h).  x may be a CUDA tensor or a
    pinned CPU tensor.  layers may also be a StackArgs (preds then unused)."""
    sa = layers if isinstance(layers, StackArgs) else StackArgs(layers, preds)
    sp = None if s_pred is None else _stream(s_pred)
    d = sa.layers[0].d
    _check(lib().cs_decode_stack(sa.layers, sa.preds, sa.L, _io_ptr(x, d), float(resid_scale), C.byref(params),
                                 int(mode), _stream(s_main), sp, ws.ptr, ws.nbytes,
                                 _ptr(trace_count), _ptr(trace_idx)))


def _io_ptr(t, n):
    """x or y of cs_decode_layer / cs_decode_stack: a CUDA tensor or a pinned CPU tensor, fp32,
    contiguous, holding at least n values (the library itself refuses
    pageable host memory)."""
    if t.dtype != torch.float32 or not t.is_contiguous() or t.numel() < n:
        raise ValueError(f"expected a contiguous fp32 tensor of at least {n} values")
    return t.data_ptr()


def cs_decode_layer(layer: FfnLayer, pred, x, y, params, ws: Workspace, stream=None, idx=None,
                    count=None):
    """One token through one layer: y = FFN(x, select(P(x))) (see include/cs.h).
    x and y may live on the GPU or in pinned host memory."""
    d = layer.c.d
    _check(lib().cs_decode_layer(C.byref(layer.c), C.byref(pred.c) if pred is not None else None,
                                 _io_ptr(x, d), _io_ptr(y, d), C.byref(params), ws.ptr, ws.nbytes,
                                 _stream(stream), _ptr(idx), _ptr(count)))


def cs_permute_rows(src, perm, dst, rows=None, cols=None, stream=None):
    """dst[i, :cols] = src[perm[i], :cols] for i < rows (the frequency-sorted
    layout step; src and dst are 2-D CUDA tensors of one dtype, or 1-D fp32
    vectors such as the bias)."""
    if src.dtype != dst.dtype:
        raise ValueError("src and dst must have the same dtype")
    s2 = src if src.dim() == 2 else src.view(-1, 1)
    d2 = dst if dst.dim() == 2 else dst.view(-1, 1)
    rows = d2.shape[0] if rows is None else int(rows)
    cols = s2.shape[1] if cols is None else int(cols)
    if perm.dtype != torch.int32 or perm.numel() < rows or s2.stride(1) != 1 or d2.stride(1) != 1:
        raise ValueError("perm must be int32 with >= rows entries; rows must be contiguous")
    _check(lib().cs_permute_rows(_ptr(s2), s2.shape[0], s2.stride(0), _ptr(perm), rows, cols, _dt(s2),
                                 _ptr(d2), d2.stride(0), _stream(stream)))


def cs_hot_order(freq):
    """The frequency-sorted neuron order (host): most frequent first, ties by
    lower id.  freq: a sequence or CPU array of f frequencies; returns an
    int32 CPU tensor."""
    fr = torch.as_tensor(freq, dtype=torch.float32).contiguous()
    out = torch.empty(fr.numel(), dtype=torch.int32)
    _check(lib().cs_hot_order(fr.data_ptr(), fr.numel(), out.data_ptr()))
    return out


class AttnLayer:
    """Head-sparse attention weights: w_q and w_o_t are [n_heads * d_head, d]
    CUDA tensors of one dtype (w_o_t is W_o transposed)."""

    def __init__(self, w_q, w_o_t, n_heads):
        if w_q.shape != w_o_t.shape or w_q.dtype != w_o_t.dtype or w_q.shape[0] % int(n_heads):
            raise ValueError("w_q and w_o_t must both be [n_heads * d_head, d] of one dtype")
        self.w_q, self.w_o_t = w_q, w_o_t
        self.n_heads = int(n_heads)
        self.d_head = w_q.shape[0] // self.n_heads
        self.d = w_q.shape[1]
        self.c = _Attn(self.d, self.n_heads, self.d_head, _dt(w_q), _ptr(w_q), _ptr(w_o_t))


def cs_sparse_attention(layer: AttnLayer, x, heads, count, k_cache, v_cache, y, ws: Workspace, stream=None):
    """y = the selected heads' attention over the KV cache (see include/cs.h);
    k_cache / v_cache are [n_heads, seq_len, d_head] CUDA tensors."""
    _check(lib().cs_sparse_attention(C.byref(layer.c), _ptr(x), _ptr(heads), _ptr(count), _ptr(k_cache),
                                     _ptr(v_cache), int(k_cache.shape[1]), _ptr(y), ws.ptr, ws.nbytes,
                                     _stream(stream)))


def cs_decode_attention(layer: AttnLayer, pred, x, y, params, k_cache, v_cache, ws: Workspace, stream=None,
                        heads=None, count=None):
    """One token's head-sparse attention step: the predictor scores the heads,
    the selection picks them, y = their attention over the KV cache (see
    include/cs.h).  x and y may live on the GPU or in pinned host memory;
    k_cache / v_cache are [n_heads, seq_len, d_head] CUDA tensors."""
    d = layer.d
    _check(lib().cs_decode_attention(C.byref(layer.c), C.byref(pred.c), _io_ptr(x, d), _io_ptr(y, d),
                                     C.byref(params), _ptr(k_cache), _ptr(v_cache), int(k_cache.shape[1]),
                                     ws.ptr, ws.nbytes, _stream(stream), _ptr(heads), _ptr(count)))


def cs_fit_predictor(layer: FfnLayer, pred: Predictor, X, lam, stream=None):
    """Overwrite pred's up map with the ridge fit of the layer's gate
    pre-activations onto relu(P_down x) over the calibration inputs X [N, d]
    (see include/cs.h).  Waits for the stream."""
    if X.dtype != torch.float32 or not X.is_cuda or not X.is_contiguous():
        raise ValueError("X must be a contiguous fp32 CUDA tensor [N, d]")
    N = X.shape[0]
    n = lib().cs_fit_scratch_size(layer.d, layer.f, pred.r, N)
    if n == 0:
        raise ValueError("bad fit dimensions")
    buf = torch.empty(n + 256, dtype=torch.uint8, device=X.device)
    ptr = (buf.data_ptr() + 255) & ~255
    _check(lib().cs_fit_predictor(C.byref(layer.c), C.byref(pred.c), _ptr(X), N, float(lam), ptr, n,
                                  _stream(stream)))


QCACHE_GROUP = 64   # channels that share one scale and offset


class QCache:
    """A KV cache held in 4 bits (see include/cs.h): k and v uint8 [batch,
    n_heads, capacity, d_head / 2], k_scale and v_scale fp16 [batch, n_heads,
    capacity, d_head / 64, 2], weight fp32 and pos int32 [batch, n_heads,
    capacity] (either may be None).  The tensors may be views, as long as their
    slots are contiguous, all step alike over sequences and heads, and no
    sequence or head is expanded from another's memory.  For cs_qcache_evict
    alone, weight (and pos) are enough."""

    def __init__(self, k, v, k_scale, v_scale, weight=None, pos=None):
        self.k, self.v, self.k_scale, self.v_scale, self.weight, self.pos = k, v, k_scale, v_scale, weight, pos
        codes = (k, v, k_scale, v_scale)
        if any(t is None for t in codes) != all(t is None for t in codes):
            raise ValueError("k, v, k_scale and v_scale go together")
        some = next((t for t in (k, weight, pos) if t is not None), None)
        if some is None or some.dim() < 3:
            raise ValueError("a cache has codes, or at least weights")
        self.batch, self.n_heads, self.capacity = some.shape[:3]
        self.d_head = 0 if k is None else 2 * k.shape[3]
        lead, groups = tuple(some.shape[:3]), self.d_head // QCACHE_GROUP
        ld = None
        for t, dtype, tail in ((k, torch.uint8, (self.d_head // 2,)), (v, torch.uint8, (self.d_head // 2,)),
                               (k_scale, torch.float16, (groups, 2)), (v_scale, torch.float16, (groups, 2)),
                               (weight, torch.float32, ()), (pos, torch.int32, ())):
            if t is None:
                continue
            if t.dtype != dtype or tuple(t.shape) != lead + tail:
                raise ValueError(f"expected a {dtype} tensor of shape {lead + tail}, got {t.dtype} {tuple(t.shape)}")
            ld = self._slots(t, tail, ld)
        self.ld_batch, self.ld_head = ld
        self.c = _QCache(self.batch, self.n_heads, self.d_head, self.capacity, self.ld_batch, self.ld_head, _ptr(k),
                         _ptr(v), _ptr(k_scale), _ptr(v_scale), _ptr(weight), _ptr(pos))
        self.addr = C.addressof(self.c)

    def _slots(self, t, tail, ld=None):
        """The slots from one sequence and one head of t to the next, which have to be `ld` if that is given."""
        row = 1
        for n, st in zip(reversed(tail), reversed(t.stride()[3:])):
            if st != row and n > 1:
                raise ValueError("a slot's values must be contiguous")
            row *= n
        if self.capacity > 1 and t.stride(2) != row:
            raise ValueError("a head's slots must be contiguous")
        dense = (self.n_heads * self.capacity, self.capacity)
        got = []
        for i, n in ((0, self.batch), (1, self.n_heads)):
            if n > 1 and t.stride(i) % row:
                raise ValueError("a cache tensor must step by whole slots")
            if n > 1 and t.stride(i) == 0:   # a step of 0 would be read as "dense", far past the memory
                raise ValueError("a cache tensor must not be expanded over sequences or heads")
            got.append(t.stride(i) // row if n > 1 else dense[i])
        if ld is not None and tuple(got) != tuple(ld):
            raise ValueError("a cache's tensors must step alike over sequences and heads")
        return tuple(got)

    @classmethod
    def empty(cls, batch, n_heads, capacity, d_head, device="cuda"):
        """A cache of its own, with weights and positions, all slots empty."""
        lead = (int(batch), int(n_heads), int(capacity))
        z = lambda dtype, *tail: torch.zeros(lead + tail, dtype=dtype, device=device)  # noqa: E731
        groups = d_head // QCACHE_GROUP
        return cls(z(torch.uint8, d_head // 2), z(torch.uint8, d_head // 2), z(torch.float16, groups, 2),
                   z(torch.float16, groups, 2), z(torch.float32), z(torch.int32).fill_(-1))


class QCacheWorkspace:
    """Device workspace of the cs_qcache_* calls on caches of this one's sizes,
    with up to n_heads query heads (0: no cs_qcache_attention) and n_q query
    tokens per sequence.  weights=False: for attention that gathers none, whose
    workspace stays small however long the cache.  That of a cache without
    codes serves cs_qcache_evict alone."""

    def __init__(self, cache: QCache, n_heads=None, n_q=1, device=None, stream=None, weights=True):
        heads = cache.n_heads if n_heads is None else int(n_heads)

        def size(capacity, heads):
            return lib().cs_qcache_workspace_size(cache.batch, cache.n_heads, capacity, cache.d_head or QCACHE_GROUP,
                                                  heads, int(n_q))
        if cache.k is None:
            n = size(1, 0)
        elif weights:
            n = size(cache.capacity, heads)
        else:
            n = size(1, heads) and max(size(1, heads), size(cache.capacity, 0))
        if n == 0:
            raise ValueError("no cs_qcache call takes these sizes")
        self.nbytes = n
        some = cache.k if cache.k is not None else cache.weight
        self.buf = torch.empty(n + 256, dtype=torch.uint8, device=device or some.device)
        self.ptr = (self.buf.data_ptr() + 255) & ~255
        _check(lib().cs_workspace_init(self.ptr, self.nbytes, _stream(stream)))


_qcall = None


def _q():
    """The native marshalling of the qcache calls (csrc/qcall.c), bound to libcs.so."""
    global _qcall
    if _qcall is None:
        L = lib()
        spec = importlib.util.spec_from_file_location("_qcall", _build.QCALL)
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
        m.init(torch.float32, torch.float16, torch.bfloat16, torch.int32,
               *(C.cast(getattr(L, f"cs_qcache_{f}"), C.c_void_p).value
                 for f in ("append", "read", "attention", "evict", "trim")))
        _qcall = m
    return _qcall


def cs_qcache_append(cache: QCache, k, v, ws: QCacheWorkspace, start=None, slots=None, n_new=None, pos=None,
                     stream=None):
    """Quantise the new rows k and v [batch, n, n_heads, d_head] into slots
    start[b] + t, or slots[b, h, t] (see include/cs.h)."""
    _check(_q().append(cache.addr, k, v, start, slots, n_new, pos, ws.ptr, ws.nbytes, _stream(stream)))


def cs_qcache_read(cache: QCache, k, v, ws: QCacheWorkspace, start=None, slots=None, stream=None):
    """The values of slots start[b] + t, or slots[b, h, t], into k and v
    [batch, n, n_heads, d_head] (see include/cs.h)."""
    _check(_q().read(cache.addr, k, v, start, slots, ws.ptr, ws.nbytes, _stream(stream)))


def cs_qcache_attention(cache: QCache, q, length, out, ws: QCacheWorkspace, q_pos=None, mask=None, scale=0.0,
                        weight=None, decay=1.0, stream=None):
    """Attention of q [batch, n_q, n_heads, d_head] over the first length[b]
    slots into out (see include/cs.h).  mask: int32 or uint32 [batch,
    ceil(n_heads / 32)], the query heads to compute (cs_select's mask).
    weight: gathers decay * cache.weight + this step's attention per slot; a
    tensor that steps like cache.weight, often cache.weight itself."""
    if mask is not None and (mask.element_size() != 4 or mask.is_floating_point() or not mask.is_contiguous()
                             or tuple(mask.shape) != (cache.batch, -(-q.shape[2] // 32))):
        raise ValueError("mask: expected contiguous 32-bit words [batch, ceil(n_heads / 32)]")
    if weight is not None and weight is not cache.weight:
        if weight.dtype is not torch.float32 or weight.shape != (cache.batch, cache.n_heads, cache.capacity):
            raise ValueError("weight: expected fp32 [batch, n_heads, capacity]")
        if cache.weight is None or weight.stride() != cache.weight.stride():
            cache._slots(weight, (), (cache.ld_batch, cache.ld_head))
    _check(_q().attention(cache.addr, q, length, out, q_pos, _ptr(mask) or 0, scale, _ptr(weight) or 0, decay, ws.ptr,
                          ws.nbytes, _stream(stream)))


def cs_qcache_evict(cache: QCache, length, limit, slots, ws: QCacheWorkspace, next_pos=None, sinks=0, recent=0,
                    stream=None):
    """slots [batch, n_heads, n] = where the next n tokens go when at most
    `limit` slots may be in use (see include/cs.h)."""
    _check(_q().evict(cache.addr, length, limit, slots, next_pos, sinks, recent, ws.ptr, ws.nbytes, _stream(stream)))


def cs_qcache_trim(cache: QCache, length, keep, dst: QCache, ws: QCacheWorkspace, next_pos=None, sinks=0, recent=0,
                   stream=None):
    """Copy each head's `keep` heaviest slots to the front of dst (see
    include/cs.h)."""
    _check(_q().trim(cache.addr, length, keep, dst.addr, next_pos, sinks, recent, ws.ptr, ws.nbytes, _stream(stream)))


def cs_stack_release():
    _check(lib().cs_stack_release())
