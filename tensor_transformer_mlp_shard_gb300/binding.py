"""ctypes binding of libtpmlp (include/tp_mlp.h).

Argument marshalling only: every computation runs in the library's CUDA
kernels.  Besides turning torch tensors into the pointer arrays of the C ABI,
the binding checks what the C side cannot see from raw pointers -- each
buffer's device, dtype, contiguity and shape -- so that no kernel is ever
handed a buffer smaller than the descriptor implies.

There is no fallback: if the library is missing, :func:`lib` raises.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

from . import build as _build

ACT = {"none": 0, "gelu_tanh": 1, "swiglu": 2}
DTYPE = {"f32": 0, "bf16": 1, "fp8": 2}
TORCH_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.bfloat16}  # fp8: bf16 buffers
STATUS = {0: "TP_OK", 1: "TP_ERR_ARG", 2: "TP_ERR_SHAPE", 3: "TP_ERR_UNSUPPORTED", 4: "TP_ERR_CUDA",
          5: "TP_ERR_TIMEOUT", 6: "TP_ERR_INDEX"}
MAX_SHARDS = 16


class TpError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class Desc(ctypes.Structure):
    _fields_ = [("S", ctypes.c_int), ("B", ctypes.c_int), ("H", ctypes.c_int), ("F", ctypes.c_int),
                ("T", ctypes.c_int), ("act", ctypes.c_int), ("dtype", ctypes.c_int), ("has_bias", ctypes.c_int),
                ("residual", ctypes.c_int), ("seq_parallel", ctypes.c_int), ("wgrad_accumulate", ctypes.c_int)]


class LayerDesc(ctypes.Structure):
    _fields_ = [("mlp", Desc), ("dropout_p", ctypes.c_float), ("ln_eps", ctypes.c_float)]


class BlockNormDesc(ctypes.Structure):
    _fields_ = [("S", ctypes.c_int), ("B", ctypes.c_int), ("H", ctypes.c_int), ("T", ctypes.c_int),
                ("dtype", ctypes.c_int), ("residual_f32", ctypes.c_int), ("seq_parallel", ctypes.c_int),
                ("has_block", ctypes.c_int), ("post", ctypes.c_int), ("pre", ctypes.c_int), ("gate", ctypes.c_int),
                ("zero_centered", ctypes.c_int), ("eps", ctypes.c_float), ("residual_scale", ctypes.c_float),
                ("block_scale", ctypes.c_float)]


class AdamWDesc(ctypes.Structure):
    _fields_ = [("n_tensors", ctypes.c_int), ("param_dtype", ctypes.c_int), ("grad_dtype", ctypes.c_int),
                ("state_bits", ctypes.c_int), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_float), ("seed", ctypes.c_uint32)]


class AdamWTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("master", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n", ctypes.c_int64), ("lr_scale", ctypes.c_float),
                ("weight_decay", ctypes.c_float)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int), ("pairs", ctypes.c_int), ("scaling", ctypes.c_int), ("base", ctypes.c_double),
                ("factor", ctypes.c_double), ("original", ctypes.c_double), ("fast", ctypes.c_double),
                ("slow", ctypes.c_double), ("attention_factor", ctypes.c_double)]


class RotaryDesc(ctypes.Structure):
    _fields_ = [("S", ctypes.c_int), ("B", ctypes.c_int), ("T", ctypes.c_int), ("heads", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int),
                ("grouped", ctypes.c_int), ("rope", RopeDesc)]


class PagedDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("heads", ctypes.c_int), ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("dtype", ctypes.c_int), ("grouped", ctypes.c_int), ("page_size", ctypes.c_int),
                ("pages", ctypes.c_int), ("window", ctypes.c_int), ("scale", ctypes.c_float), ("rope", RopeDesc)]


class ProfEntry(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 48), ("launches", ctypes.c_int), ("total_ms", ctypes.c_double),
                ("sm_cycles", ctypes.c_uint64), ("sm_ns", ctypes.c_uint64)]


_lib = None
VP = ctypes.c_void_p
PP = ctypes.POINTER(ctypes.c_void_p)

# exported symbol -> (restype, argtypes)
SIGNATURES = {
    "tp_abi_version": (ctypes.c_int, []),
    "tp_status_str": (ctypes.c_char_p, [ctypes.c_int]),
    "tp_last_error": (ctypes.c_char_p, []),
    "tp_mlp_create": (ctypes.c_int, [ctypes.POINTER(Desc), ctypes.POINTER(VP)]),
    "tp_mlp_destroy": (None, [VP]),
    "tp_mlp_workspace_bytes": (ctypes.c_size_t, [VP]),
    "tp_mlp_fwd": (ctypes.c_int, [VP, PP, PP, PP, PP, VP, PP, PP, PP, VP]),
    "tp_mlp_fwd_ws": (ctypes.c_int, [VP, PP, PP, PP, PP, VP, PP, PP, PP, VP, ctypes.c_size_t, VP]),
    "tp_mlp_set_fp8_history": (ctypes.c_int, [VP, ctypes.c_int]),
    "tp_mlp_fp8_amax": (ctypes.c_int, [VP, VP, ctypes.c_size_t, VP, VP]),
    "tp_layer_fp8_amax": (ctypes.c_int, [VP, VP, ctypes.c_size_t, VP, VP]),
    "tp_mlp_bwd": (ctypes.c_int, [VP, PP, PP, PP, PP, PP, PP, PP, PP, PP, PP, VP, VP, ctypes.c_size_t, VP]),
    "tp_linear_col": (ctypes.c_int, [ctypes.POINTER(Desc), PP, PP, PP, PP, PP, VP]),
    "tp_linear_row": (ctypes.c_int, [ctypes.POINTER(Desc), PP, PP, VP, PP, PP, VP]),
    "tp_linear_col_ws": (ctypes.c_int, [ctypes.POINTER(Desc), PP, PP, PP, PP, PP, VP, ctypes.c_size_t, VP]),
    "tp_linear_row_ws": (ctypes.c_int, [ctypes.POINTER(Desc), PP, PP, VP, PP, PP, VP, ctypes.c_size_t, VP]),
    "tp_linear_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(Desc)]),
    "tp_linear_col_bwd": (ctypes.c_int, [ctypes.POINTER(Desc), PP, PP, PP, PP, PP, PP, VP, ctypes.c_size_t, VP]),
    "tp_linear_row_bwd": (ctypes.c_int, [ctypes.POINTER(Desc), PP, PP, PP, PP, PP, VP, VP, ctypes.c_size_t, VP]),
    "tp_linear_row_bwd_noalloc": (ctypes.c_int, [ctypes.POINTER(Desc), PP, PP, PP, PP, PP, VP, VP]),
    "tp_layer_create": (ctypes.c_int, [ctypes.POINTER(LayerDesc), ctypes.POINTER(VP)]),
    "tp_layer_destroy": (None, [VP]),
    "tp_layer_workspace_bytes": (ctypes.c_size_t, [VP]),
    "tp_layer_set_fp8_history": (ctypes.c_int, [VP, ctypes.c_int]),
    "tp_layer_fwd": (ctypes.c_int, [VP, PP, VP, VP, PP, PP, PP, VP, ctypes.c_uint64, PP, VP, VP, VP, PP, PP, VP,
                                    ctypes.c_size_t, VP]),
    "tp_layer_bwd": (ctypes.c_int, [VP, PP, PP, VP, VP, VP, VP, PP, PP, PP, PP, ctypes.c_uint64, PP, VP, VP, PP,
                                    PP, PP, VP, VP, ctypes.c_size_t, VP]),
    "tp_block_norm_create": (ctypes.c_int, [ctypes.POINTER(BlockNormDesc), ctypes.POINTER(VP)]),
    "tp_block_norm_destroy": (None, [VP]),
    "tp_block_norm_workspace_bytes": (ctypes.c_size_t, [VP]),
    # (their pointer arrays go as packed bytes, cheaper to make than ctypes arrays)
    "tp_block_norm_fwd": (ctypes.c_int, [VP] * 12),
    "tp_block_norm_bwd": (ctypes.c_int, [VP] * 18 + [ctypes.c_size_t, VP]),
    "tp_adamw_create": (ctypes.c_int, [ctypes.POINTER(AdamWDesc), ctypes.POINTER(AdamWTensor), ctypes.POINTER(VP)]),
    "tp_adamw_destroy": (None, [VP]),
    "tp_adamw_set_grads": (ctypes.c_int, [VP, PP]),
    "tp_adamw_ctl_init": (ctypes.c_int, [VP, ctypes.c_int, VP]),
    "tp_adamw_grad_norm": (ctypes.c_int, [VP, ctypes.c_float, ctypes.c_float, VP, VP]),
    "tp_adamw_step": (ctypes.c_int, [VP, ctypes.c_float, ctypes.c_float, ctypes.c_int, VP, VP]),
    "tp_rotary_create": (ctypes.c_int, [ctypes.POINTER(RotaryDesc), ctypes.POINTER(VP)]),
    "tp_rotary_destroy": (None, [VP]),
    "tp_rotary_fwd": (ctypes.c_int, [VP] * 5),
    "tp_rotary_bwd": (ctypes.c_int, [VP] * 5),
    "tp_paged_create": (ctypes.c_int, [ctypes.POINTER(PagedDesc), ctypes.POINTER(VP)]),
    "tp_paged_destroy": (None, [VP]),
    "tp_paged_workspace_bytes": (ctypes.c_size_t, [VP]),
    "tp_paged_append": (ctypes.c_int, [VP] * 4 + [ctypes.c_int, VP, ctypes.c_int, ctypes.c_int] + [VP] * 6),
    "tp_paged_decode": (ctypes.c_int, [VP] * 4 + [ctypes.c_int, VP, ctypes.c_int, ctypes.c_int] + [VP] * 6 +
                        [ctypes.c_size_t, VP]),
    "tp_paged_sync_status": (ctypes.c_int, [VP, VP]),
    "tp_fp8_quantize": (ctypes.c_int, [PP, PP, ctypes.POINTER(ctypes.c_int64), ctypes.c_int, ctypes.c_int, VP, VP]),
    "tp_sync_status": (ctypes.c_int, [VP]),
    "tp_mlp_sync_status": (ctypes.c_int, [VP, VP]),
    "tp_layer_sync_status": (ctypes.c_int, [VP, VP]),
    "tp_mlp_debug_wait_timeout": (ctypes.c_int, [VP, ctypes.c_uint64, VP]),
    "tp_set_wait_limit_ns": (None, [ctypes.c_uint64]),
    "tp_debug_wait_timeout": (ctypes.c_int, [ctypes.c_uint64, VP]),
    "tp_launch_count": (ctypes.c_uint64, []),
    "tp_tail_split_count": (ctypes.c_uint64, []),
    "tp_set_tail_split": (ctypes.c_int, [ctypes.c_int]),
    "tp_set_max_gemm_pairs": (ctypes.c_int, [ctypes.c_int]),
    "tp_set_k_order": (ctypes.c_int, [ctypes.c_int]),
    "tp_set_band_rows": (ctypes.c_int, [ctypes.c_int]),
    "tp_set_launch_overlap": (ctypes.c_int, [ctypes.c_int]),
    "tp_set_tile_mode": (ctypes.c_int, [ctypes.c_int]),
    "tp_set_fused_fwd": (ctypes.c_int, [ctypes.c_int]),
    "tp_prof_enable": (None, [ctypes.c_int]),
    "tp_prof_collect": (ctypes.c_int, [ctypes.POINTER(ProfEntry), ctypes.c_int]),
    "tp_prof_select": (None, [ctypes.c_char_p]),
}


def library_path() -> str:
    return _build.LIB


def lib():
    """Load libtpmlp.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with __graft_entry__.build() "
                               "(the CUDA library is required; there is no fallback)")
        L = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(status: int):
    if status != 0:
        raise TpError(status, lib().tp_last_error().decode(errors="replace"))


# the current stream's handle without a torch.cuda.Stream object around it (0.4 us against 3 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return VP(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return VP(stream.cuda_stream)
    return VP(int(stream))


def _arr(ptrs):
    """Host array of device pointers (None for a missing array)."""
    if ptrs is None:
        return None
    a = (VP * max(1, len(ptrs)))()
    for i, p in enumerate(ptrs):
        a[i] = p
    return ctypes.cast(a, PP)


class _Checker:
    def __init__(self, dtype: str):
        self.dt = TORCH_DTYPE[dtype]

    def tensors(self, name, ts, n, shape, dtype=None):
        dtype = dtype or self.dt
        if ts is None:
            raise ValueError(f"{name}: required")
        if isinstance(ts, torch.Tensor):
            ts = [ts]
        ts = list(ts)
        if len(ts) != n:
            raise ValueError(f"{name}: expected {n} tensors, got {len(ts)}")
        for i, t in enumerate(ts):
            if not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise ValueError(f"{name}[{i}]: must be a CUDA tensor")
            if t.dtype != dtype:
                raise ValueError(f"{name}[{i}]: dtype {t.dtype}, expected {dtype}")
            if not t.is_contiguous():
                raise ValueError(f"{name}[{i}]: must be contiguous")
            if t.numel() != _prod(shape):
                raise ValueError(f"{name}[{i}]: {tuple(t.shape)} has {t.numel()} elements, expected {shape}")
        return [t.data_ptr() for t in ts]

    def optional(self, name, ts, n, shape, dtype=None):
        return None if ts is None else self.tensors(name, ts, n, shape, dtype)


def _prod(shape):
    p = 1
    for s in shape:
        p *= int(s)
    return p


def make_desc(S, B, H, F, T, act="gelu_tanh", dtype="bf16", has_bias=False, residual=False,
              seq_parallel=False, wgrad_accumulate=False) -> Desc:
    return Desc(int(S), int(B), int(H), int(F), int(T), ACT[act], DTYPE[dtype], int(bool(has_bias)),
                int(bool(residual)), int(bool(seq_parallel)), int(bool(wgrad_accumulate)))


class Layout:
    """Buffer shapes implied by a descriptor (see include/tp_mlp.h)."""

    def __init__(self, S, B, H, F, T, act="gelu_tanh", dtype="bf16", has_bias=False, residual=False,
                 seq_parallel=False, wgrad_accumulate=False):
        self.S, self.B, self.H, self.F, self.T = S, B, H, F, T
        self.act, self.dtype = act, dtype
        self.has_bias, self.residual = has_bias, residual
        self.seq_parallel, self.wgrad_accumulate = seq_parallel, wgrad_accumulate
        self.M = S * B
        self.g = 2 if act == "swiglu" else 1
        self.Fs = F // T if T else 0
        self.nx = T if seq_parallel else 1
        self.xrows = self.M // T if seq_parallel else self.M

    def desc(self) -> Desc:
        return make_desc(self.S, self.B, self.H, self.F, self.T, self.act, self.dtype, self.has_bias,
                         self.residual, self.seq_parallel, self.wgrad_accumulate)


class TPMLP(Layout):
    """Handle for one tensor-parallel MLP shape (tp_mlp_create)."""

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        self._d = self.desc()
        h = VP()
        _check(lib().tp_mlp_create(ctypes.byref(self._d), ctypes.byref(h)))
        self._h = h
        self._c = _Checker(self.dtype)

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and _lib is not None:
            _lib.tp_mlp_destroy(h)
            self._h = None

    def workspace_bytes(self) -> int:
        return int(lib().tp_mlp_workspace_bytes(self._h))

    def sync_status(self, stream=None) -> int:
        """Synchronise the stream and return (and clear) this handle's device
        status word (TP_ERR_TIMEOUT when one of its kernels' waits ran out)."""
        return int(lib().tp_mlp_sync_status(self._h, _stream(stream)))

    def debug_wait_timeout(self, limit_ns: int, stream=None):
        """A kernel that waits on a flag nothing sets, reporting its timeout to
        this handle's status word."""
        _check(lib().tp_mlp_debug_wait_timeout(self._h, int(limit_ns), _stream(stream)))

    def set_fp8_history(self, n: int):
        """FP8 delayed scaling over the last n amaxes of every operand (0:
        current scaling).  Clears the history; pass the same workspace to
        every later fwd / bwd."""
        _check(lib().tp_mlp_set_fp8_history(self._h, int(n)))

    FP8_AMAX_NAMES = ("X", "W1", "W2", "A", "dY", "dPre")

    def fp8_amax(self, workspace, stream=None):
        """The per-tensor amaxes the last fwd / bwd recorded in `workspace`, as
        a CUDA float32 tensor in the order of FP8_AMAX_NAMES (dtype "fp8")."""
        ws_ptr, ws_bytes = _workspace(workspace)
        out = torch.empty(len(self.FP8_AMAX_NAMES), dtype=torch.float32, device=workspace.device)
        _check(lib().tp_mlp_fp8_amax(self._h, ws_ptr, ws_bytes, out.data_ptr(), _stream(stream)))
        return out

    def fwd(self, X, W1, b1, W2, b2, Y, pre, A, stream=None, workspace=None):
        """Forward; `workspace` (required for dtype "fp8") must then be passed,
        unchanged, to the following bwd."""
        c, T, H, Fs, g = self._c, self.T, self.H, self.Fs, self.g
        px = c.tensors("X", X, self.nx, (self.xrows, H))
        pw1 = c.tensors("W1", W1, T, (g * Fs, H))
        pw2 = c.tensors("W2", W2, T, (H, Fs))
        pb1 = c.tensors("b1", b1, T, (g * Fs,)) if self.has_bias else None
        pb2 = c.tensors("b2", b2, 1, (H,))[0] if self.has_bias else None
        py = c.tensors("Y", Y, self.nx, (self.xrows, H))
        pp = c.optional("pre", pre, T, (self.M, g * Fs))
        pa = c.tensors("A", A, T, (self.M, Fs))
        if workspace is None:
            _check(lib().tp_mlp_fwd(self._h, _arr(px), _arr(pw1), _arr(pb1), _arr(pw2), pb2, _arr(py), _arr(pp),
                                    _arr(pa), _stream(stream)))
        else:
            ws_ptr, ws_bytes = _workspace(workspace, self.workspace_bytes())
            _check(lib().tp_mlp_fwd_ws(self._h, _arr(px), _arr(pw1), _arr(pb1), _arr(pw2), pb2, _arr(py),
                                       _arr(pp), _arr(pa), ws_ptr, ws_bytes, _stream(stream)))

    def bwd(self, dY, X, W1, W2, pre, A, dX, dW1, db1, dW2, db2, workspace, stream=None):
        c, T, H, Fs, g = self._c, self.T, self.H, self.Fs, self.g
        f32 = torch.float32
        pdy = c.tensors("dY", dY, self.nx, (self.xrows, H))
        px = c.tensors("X", X, self.nx, (self.xrows, H))
        pw1 = c.tensors("W1", W1, T, (g * Fs, H))
        pw2 = c.tensors("W2", W2, T, (H, Fs))
        pp = c.optional("pre", pre, T, (self.M, g * Fs))
        pa = c.tensors("A", A, T, (self.M, Fs))
        pdx = c.tensors("dX", dX, self.nx, (self.xrows, H))
        pdw1 = c.tensors("dW1", dW1, T, (g * Fs, H), f32)
        pdw2 = c.tensors("dW2", dW2, T, (H, Fs), f32)
        pdb1 = c.tensors("db1", db1, T, (g * Fs,), f32) if self.has_bias else None
        pdb2 = c.tensors("db2", db2, 1, (H,), f32)[0] if self.has_bias else None
        nws = self.workspace_bytes()
        ws_ptr, ws_bytes = _workspace(workspace, nws)
        _check(lib().tp_mlp_bwd(self._h, _arr(pdy), _arr(px), _arr(pw1), _arr(pw2), _arr(pp), _arr(pa),
                                _arr(pdx), _arr(pdw1), _arr(pdb1), _arr(pdw2), pdb2, ws_ptr, ws_bytes,
                                _stream(stream)))


class TPLayer(Layout):
    """Handle for the TransformerLayer MLP sub-block
    Y = X + dropout_p(MLP(LayerNorm(X))) (tp_layer_create).  The MLP keyword
    arguments are those of TPMLP (residual must stay False)."""

    def __init__(self, *args, dropout_p: float = 0.0, ln_eps: float = 1e-5, **kw):
        super().__init__(*args, **kw)
        self.dropout_p, self.ln_eps = float(dropout_p), float(ln_eps)
        self._d = LayerDesc(self.desc(), self.dropout_p, self.ln_eps)
        h = VP()
        _check(lib().tp_layer_create(ctypes.byref(self._d), ctypes.byref(h)))
        self._h = h
        self._c = _Checker(self.dtype)

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and _lib is not None:
            _lib.tp_layer_destroy(h)
            self._h = None

    def workspace_bytes(self) -> int:
        return int(lib().tp_layer_workspace_bytes(self._h))

    def sync_status(self, stream=None) -> int:
        """Synchronise the stream and return (and clear) this handle's device
        status word."""
        return int(lib().tp_layer_sync_status(self._h, _stream(stream)))

    FP8_AMAX_NAMES = ("X", "W1", "W2", "A", "dY", "dPre")

    def fp8_amax(self, workspace, stream=None):
        """The per-tensor amaxes of the MLP inside the block, as TPMLP.fp8_amax
        (X: the LayerNorm output, dY: the gradient at the MLP's output)."""
        ws_ptr, ws_bytes = _workspace(workspace)
        out = torch.empty(len(self.FP8_AMAX_NAMES), dtype=torch.float32, device=workspace.device)
        _check(lib().tp_layer_fp8_amax(self._h, ws_ptr, ws_bytes, out.data_ptr(), _stream(stream)))
        return out

    def set_fp8_history(self, n: int):
        """FP8 delayed scaling over the last n amaxes (0: current scaling); as
        TPMLP.set_fp8_history."""
        _check(lib().tp_layer_set_fp8_history(self._h, int(n)))

    def fwd(self, X, gamma, beta, W1, b1, W2, b2, seed, Y, Xn, mean, rstd, pre, A, workspace=None, stream=None):
        c, T, H, Fs, g, M = self._c, self.T, self.H, self.Fs, self.g, self.M
        f32 = torch.float32
        px = c.tensors("X", X, self.nx, (self.xrows, H))
        pg = c.tensors("gamma", gamma, 1, (H,))[0]
        pbt = c.tensors("beta", beta, 1, (H,))[0]
        pw1 = c.tensors("W1", W1, T, (g * Fs, H))
        pw2 = c.tensors("W2", W2, T, (H, Fs))
        pb1 = c.tensors("b1", b1, T, (g * Fs,)) if self.has_bias else None
        pb2 = c.tensors("b2", b2, 1, (H,))[0] if self.has_bias else None
        py = c.tensors("Y", Y, self.nx, (self.xrows, H))
        pxn = c.tensors("Xn", Xn, 1, (M, H))[0]
        pm = c.tensors("mean", mean, 1, (M,), f32)[0]
        pr = c.tensors("rstd", rstd, 1, (M,), f32)[0]
        pp = c.optional("pre", pre, T, (M, g * Fs))
        pa = c.tensors("A", A, T, (M, Fs))
        ws_ptr, ws_bytes = (None, 0) if workspace is None else _workspace(workspace, self.workspace_bytes())
        _check(lib().tp_layer_fwd(self._h, _arr(px), pg, pbt, _arr(pw1), _arr(pb1), _arr(pw2), pb2,
                                  int(seed) & (2 ** 64 - 1), _arr(py), pxn, pm, pr, _arr(pp), _arr(pa), ws_ptr,
                                  ws_bytes, _stream(stream)))

    def bwd(self, dY, X, gamma, Xn, mean, rstd, W1, W2, pre, A, seed, dX, dgamma, dbeta, dW1, db1, dW2, db2,
            workspace, stream=None):
        c, T, H, Fs, g, M = self._c, self.T, self.H, self.Fs, self.g, self.M
        f32 = torch.float32
        pdy = c.tensors("dY", dY, self.nx, (self.xrows, H))
        px = c.tensors("X", X, self.nx, (self.xrows, H))
        pg = c.tensors("gamma", gamma, 1, (H,))[0]
        pxn = c.tensors("Xn", Xn, 1, (M, H))[0]
        pm = c.tensors("mean", mean, 1, (M,), f32)[0]
        pr = c.tensors("rstd", rstd, 1, (M,), f32)[0]
        pw1 = c.tensors("W1", W1, T, (g * Fs, H))
        pw2 = c.tensors("W2", W2, T, (H, Fs))
        pp = c.optional("pre", pre, T, (M, g * Fs))
        pa = c.tensors("A", A, T, (M, Fs))
        pdx = c.tensors("dX", dX, self.nx, (self.xrows, H))
        pdg = c.tensors("dgamma", dgamma, 1, (H,), f32)[0]
        pdb = c.tensors("dbeta", dbeta, 1, (H,), f32)[0]
        pdw1 = c.tensors("dW1", dW1, T, (g * Fs, H), f32)
        pdw2 = c.tensors("dW2", dW2, T, (H, Fs), f32)
        pdb1 = c.tensors("db1", db1, T, (g * Fs,), f32) if self.has_bias else None
        pdb2 = c.tensors("db2", db2, 1, (H,), f32)[0] if self.has_bias else None
        ws_ptr, ws_bytes = _workspace(workspace, self.workspace_bytes())
        _check(lib().tp_layer_bwd(self._h, _arr(pdy), _arr(px), pg, pxn, pm, pr, _arr(pw1), _arr(pw2), _arr(pp),
                                  _arr(pa), int(seed) & (2 ** 64 - 1), _arr(pdx), pdg, pdb, _arr(pdw1), _arr(pdb1),
                                  _arr(pdw2), pdb2, ws_ptr, ws_bytes, _stream(stream)))


def _workspace(workspace, need=None):
    """(pointer, bytes) of a workspace tensor, (None, 0) for None.  The library
    checks the size: the part a call requires can be smaller than the queried
    size `need`, whose end is the optional tail-split scratch."""
    if workspace is None:
        return None, 0
    if not (isinstance(workspace, torch.Tensor) and workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def alloc_workspace(nbytes: int, device="cuda"):
    """A 256-byte aligned byte buffer (torch allocations are 512-aligned)."""
    return torch.empty(max(1, nbytes), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------------------
# single layers
# ---------------------------------------------------------------------------
def linear_col(layout: Layout, X, W, b, out, pre=None, stream=None, workspace=None):
    """Column layer forward; with `workspace` (required for dtype "fp8",
    which then needs it, unchanged, in linear_col_bwd) tp_linear_col_ws."""
    c, T, H, Fs, g = _Checker(layout.dtype), layout.T, layout.H, layout.Fs, layout.g
    d = layout.desc()
    px = c.tensors("X", X, layout.nx, (layout.xrows, H))
    pw = c.tensors("W", W, T, (g * Fs, H))
    pb = c.tensors("b", b, T, (g * Fs,)) if layout.has_bias else None
    po = c.tensors("out", out, T, (layout.M, Fs))
    pp = c.optional("pre", pre, T, (layout.M, g * Fs))
    if workspace is None:
        _check(lib().tp_linear_col(ctypes.byref(d), _arr(px), _arr(pw), _arr(pb), _arr(po), _arr(pp),
                                   _stream(stream)))
    else:
        ws, nws = _workspace(workspace)
        _check(lib().tp_linear_col_ws(ctypes.byref(d), _arr(px), _arr(pw), _arr(pb), _arr(po), _arr(pp), ws, nws,
                                      _stream(stream)))


def linear_row(layout: Layout, X, W, b, R, Y, stream=None, workspace=None):
    """Row layer forward; with `workspace` (required for dtype "fp8", which
    then needs it, unchanged, in linear_row_bwd) tp_linear_row_ws."""
    c, T, H, Fs = _Checker(layout.dtype), layout.T, layout.H, layout.Fs
    d = layout.desc()
    px = c.tensors("X", X, T, (layout.M, Fs))
    pw = c.tensors("W", W, T, (H, Fs))
    pb = c.tensors("b", b, 1, (H,))[0] if layout.has_bias else None
    pr = c.tensors("R", R, layout.nx, (layout.xrows, H)) if layout.residual else None
    py = c.tensors("Y", Y, layout.nx, (layout.xrows, H))
    if workspace is None:
        _check(lib().tp_linear_row(ctypes.byref(d), _arr(px), _arr(pw), pb, _arr(pr), _arr(py), _stream(stream)))
    else:
        ws, nws = _workspace(workspace)
        _check(lib().tp_linear_row_ws(ctypes.byref(d), _arr(px), _arr(pw), pb, _arr(pr), _arr(py), ws, nws,
                                      _stream(stream)))


def linear_workspace_bytes(layout: Layout) -> int:
    d = layout.desc()
    return int(lib().tp_linear_workspace_bytes(ctypes.byref(d)))


def linear_col_bwd(layout: Layout, dOut, X, W, dX, dW, db, workspace=None, stream=None):
    c, T, H, Fs = _Checker(layout.dtype), layout.T, layout.H, layout.Fs
    f32 = torch.float32
    d = layout.desc()
    pdo = c.tensors("dOut", dOut, T, (layout.M, Fs))
    px = c.tensors("X", X, layout.nx, (layout.xrows, H))
    pw = c.tensors("W", W, T, (Fs, H))
    pdx = c.tensors("dX", dX, layout.nx, (layout.xrows, H))
    pdw = c.tensors("dW", dW, T, (Fs, H), f32)
    pdb = c.tensors("db", db, T, (Fs,), f32) if layout.has_bias else None
    ws, nws = _workspace(workspace, linear_workspace_bytes(layout))
    _check(lib().tp_linear_col_bwd(ctypes.byref(d), _arr(pdo), _arr(px), _arr(pw), _arr(pdx), _arr(pdw),
                                   _arr(pdb), ws, nws, _stream(stream)))


def linear_row_bwd(layout: Layout, dY, X, W, dX, dW, db, workspace=None, stream=None):
    c, T, H, Fs = _Checker(layout.dtype), layout.T, layout.H, layout.Fs
    f32 = torch.float32
    d = layout.desc()
    pdy = c.tensors("dY", dY, layout.nx, (layout.xrows, H))
    px = c.tensors("X", X, T, (layout.M, Fs))
    pw = c.tensors("W", W, T, (H, Fs))
    pdx = c.tensors("dX", dX, T, (layout.M, Fs))
    pdw = c.tensors("dW", dW, T, (H, Fs), f32)
    pdb = c.tensors("db", db, 1, (H,), f32)[0] if layout.has_bias else None
    ws, nws = _workspace(workspace, linear_workspace_bytes(layout))
    _check(lib().tp_linear_row_bwd(ctypes.byref(d), _arr(pdy), _arr(px), _arr(pw), _arr(pdx), _arr(pdw), pdb,
                                   ws, nws, _stream(stream)))


def linear_row_bwd_noalloc(layout: Layout, dY, X, W, dX, dW, db, stream=None):
    """tp_linear_row_bwd for callers that cannot allocate device memory: the
    bias-gradient scratch comes from a fixed 4 MiB array inside the library
    instead of a caller workspace (see include/tp_mlp.h for the limits and
    for why overlapping calls race)."""
    c, T, H, Fs = _Checker(layout.dtype), layout.T, layout.H, layout.Fs
    f32 = torch.float32
    d = layout.desc()
    pdy = c.tensors("dY", dY, layout.nx, (layout.xrows, H))
    px = c.tensors("X", X, T, (layout.M, Fs))
    pw = c.tensors("W", W, T, (H, Fs))
    pdx = c.tensors("dX", dX, T, (layout.M, Fs))
    pdw = c.tensors("dW", dW, T, (H, Fs), f32)
    pdb = c.tensors("db", db, 1, (H,), f32)[0] if layout.has_bias else None
    _check(lib().tp_linear_row_bwd_noalloc(ctypes.byref(d), _arr(pdy), _arr(px), _arr(pw), _arr(pdx), _arr(pdw),
                                           pdb, _stream(stream)))


FP8_FORMATS = {"e4m3": 0, "e5m2": 1}


def fp8_quantize(inputs, outputs, fmt: str, amax, stream=None):
    """Quantise one tensor split over bf16 buffers `inputs` into uint8 buffers
    `outputs` (same element counts) with one per-tensor scale; the amax lands
    in the one-element fp32 CUDA tensor `amax`."""
    inputs, outputs = list(inputs), list(outputs)
    if len(inputs) != len(outputs):
        raise ValueError("inputs and outputs differ in length")
    for a, b in zip(inputs, outputs):
        if not (a.is_cuda and b.is_cuda and a.is_contiguous() and b.is_contiguous()):
            raise ValueError("contiguous CUDA tensors required")
        if a.dtype != torch.bfloat16 or b.dtype != torch.uint8 or a.numel() != b.numel():
            raise ValueError("bf16 inputs and uint8 outputs of equal sizes required")
    if not (amax.is_cuda and amax.dtype == torch.float32 and amax.numel() >= 1):
        raise ValueError("amax must be a CUDA float32 tensor")
    n = (ctypes.c_int64 * len(inputs))(*[t.numel() for t in inputs])
    _check(lib().tp_fp8_quantize(_arr([t.data_ptr() for t in inputs]), _arr([t.data_ptr() for t in outputs]), n,
                                 len(inputs), FP8_FORMATS[fmt], amax.data_ptr(), _stream(stream)))


# ---------------------------------------------------------------------------
# block norm
# ---------------------------------------------------------------------------
NORM = {"none": 0, "rms": 1, "layer": 2}
GATE = {"none": 0, "channel": 1, "token": 2, "element": 3}


def _pointer(name, t, n, dtype):
    """Address of a contiguous CUDA tensor of n elements of a type."""
    try:
        if t.dtype is dtype and t.is_cuda and t.is_contiguous() and t.numel() == n:
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    raise ValueError(f"{name}: {tuple(t.shape)} has {t.numel()} elements, expected {n}")


_pack = [struct.Struct("%dP" % k).pack for k in range(MAX_SHARDS + 1)]
_pack1 = _pack[1]


def _pointers(name, ts, count, n, dtype):
    """The addresses of `count` shards (one tensor, or a list), as a C array."""
    if count == 1:
        t = ts[0] if type(ts) is list and len(ts) == 1 else ts
        try:
            if t.dtype is dtype and t.is_cuda and t.is_contiguous() and t.numel() == n:
                return _pack1(t.data_ptr())
        except AttributeError:
            pass
    if ts is None:
        raise ValueError(f"{name}: required")
    if isinstance(ts, torch.Tensor):
        ts = (ts,)
    if len(ts) != count:
        raise ValueError(f"{name}: expected {count} tensors, got {len(ts)}")
    if count == 1:
        return _pack1(_pointer(name, ts[0], n, dtype))
    try:
        ptrs = [t.data_ptr() for t in ts
                if t.dtype is dtype and t.is_cuda and t.is_contiguous() and t.numel() == n]
        if len(ptrs) == count:
            return _pack[count](*ptrs)
    except AttributeError:
        pass
    return _pack[count](*[_pointer(f"{name}[{i}]", t, n, dtype) for i, t in enumerate(ts)])


class TPBlockNorm:
    """Handle for the residual stream between one block and the next
    (tp_block_norm_create):

        Y = residual_scale * X + block_scale * gate * post(F)      N = pre(Y)

    post, pre: "none", "rms" or "layer"; gate: "none", "channel" ([H]), "token"
    ([M]) or "element" ([M, H]).  X and Y are fp32 with residual_f32.  With
    block=False there is no F and no Y: N = pre(X).  Under seq_parallel X, F, Y,
    N, token and element gates and their gradients are lists of T token shards;
    otherwise one tensor each (or a list of one).  An argument that the
    configuration has no use for is None."""

    def __init__(self, S, B, H, T=1, dtype="bf16", post="none", pre="rms", gate="none", block=True,
                 residual_f32=False, seq_parallel=False, zero_centered=False, eps=1e-5, residual_scale=1.0,
                 block_scale=1.0):
        self._d = BlockNormDesc(int(S), int(B), int(H), int(T), DTYPE[dtype], int(bool(residual_f32)),
                                int(bool(seq_parallel)), int(bool(block)), NORM[post], NORM[pre], GATE[gate],
                                int(bool(zero_centered)), float(eps), float(residual_scale), float(block_scale))
        h = VP()
        _check(lib().tp_block_norm_create(ctypes.byref(self._d), ctypes.byref(h)))
        self._h = h
        self.S, self.B, self.H, self.T, self.M = int(S), int(B), int(H), int(T), int(S) * int(B)
        self.dtype, self.post, self.pre, self.gate, self.block = dtype, post, pre, gate, bool(block)
        self.seq_parallel, self.residual_f32 = bool(seq_parallel), bool(residual_f32)
        self.nx = self.T if seq_parallel else 1
        self._act = TORCH_DTYPE[dtype]
        self._res = torch.float32 if residual_f32 else self._act
        rows = self.M // self.nx
        self._n = rows * self.H
        # elements and type of a gate's gradient are those of the gate, but a channel gate's is fp32
        self._gate_n = {"none": 0, "channel": self.H, "token": rows, "element": self._n}[gate]
        self._gate_nx = 1 if gate == "channel" else self.nx
        self._has_post, self._has_pre = post != "none", pre != "none"
        self._post_layer, self._pre_layer = post == "layer", pre == "layer"
        self._fwd, self._bwd = lib().tp_block_norm_fwd, lib().tp_block_norm_bwd

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and _lib is not None:
            _lib.tp_block_norm_destroy(h)
            self._h = None

    def workspace_bytes(self) -> int:
        return int(lib().tp_block_norm_workspace_bytes(self._h))

    def fwd(self, X, F=None, gate=None, post_w=None, post_b=None, pre_w=None, pre_b=None, Y=None, N=None, stats=None,
            stream=None):
        """Forward into Y and N (Y may be X).  stats: an fp32 [M, 4] tensor that
        keeps what the backward needs, or None."""
        n, nx, H, act, res = self._n, self.nx, self.H, self._act, self._res
        x, f, g, y, out = _pointers("X", X, nx, n, res), None, None, None, None
        if self.block:
            f, y = _pointers("F", F, nx, n, act), _pointers("Y", Y, nx, n, res)
            if self._gate_n:
                g = _pointers("gate", gate, self._gate_nx, self._gate_n, act)
        if self._has_pre:
            out = _pointers("N", N, nx, n, act)
        status = self._fwd(
            self._h, x, f, g,
            _pointer("post_w", post_w, H, act) if self._has_post else None,
            _pointer("post_b", post_b, H, act) if self._post_layer else None,
            _pointer("pre_w", pre_w, H, act) if self._has_pre else None,
            _pointer("pre_b", pre_b, H, act) if self._pre_layer else None,
            y, out, None if stats is None else _pointer("stats", stats, 4 * self.M, torch.float32), _stream(stream))
        if status:
            _check(status)

    def bwd(self, dY, dN, Y, F, gate, post_w, post_b, pre_w, stats, dX, dF, dgate, dpost_w, dpost_b, dpre_w, dpre_b,
            workspace=None, stream=None):
        """Backward from dY (None: zero) and dN, with the forward's Y (X without
        a block), F and stats.  dX may be dY.  Parameter gradients are fp32 and
        overwritten; a token or element gate's gradient has the gate's type."""
        n, nx, H, act, res, f32 = self._n, self.nx, self.H, self._act, self._res, torch.float32
        pre, post, pre_l, post_l = self._has_pre, self._has_post, self._pre_layer, self._post_layer
        g = dg = None
        if self._gate_n:
            g = _pointers("gate", gate, self._gate_nx, self._gate_n, act)
            dg = _pointers("dgate", dgate, self._gate_nx, self._gate_n, f32 if self.gate == "channel" else act)
        ws, nws = (None, 0) if workspace is None else _workspace(workspace)
        status = self._bwd(
            self._h,
            None if dY is None else _pointers("dY", dY, nx, n, res),
            _pointers("dN", dN, nx, n, act) if pre else None,
            _pointers("Y", Y, nx, n, res) if pre else None,
            _pointers("F", F, nx, n, act) if post or g is not None else None,
            g,
            _pointer("post_w", post_w, H, act) if post else None,
            _pointer("post_b", post_b, H, act) if post_l else None,
            _pointer("pre_w", pre_w, H, act) if pre else None,
            _pointer("stats", stats, 4 * self.M, f32),
            _pointers("dX", dX, nx, n, res),
            _pointers("dF", dF, nx, n, act) if self.block else None,
            dg,
            _pointer("dpost_w", dpost_w, H, f32) if post else None,
            _pointer("dpost_b", dpost_b, H, f32) if post_l else None,
            _pointer("dpre_w", dpre_w, H, f32) if pre else None,
            _pointer("dpre_b", dpre_b, H, f32) if pre_l else None, ws, nws, _stream(stream))
        if status:
            _check(status)


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------
class TPAdamW:
    """AdamW over a list of tensors (tp_adamw_create): weight shards, biases and
    norm weights, updated in place by one launch.

    params: bf16 (with fp32 `master` copies, made here when not given) or fp32
    CUDA tensors; grads: fp32 or bf16, one for each.  Both are read and written
    where they are at every step (set_grads changes the gradients).  m, v (and
    m_scale, v_scale with state_bits=8) are the states, zeros when not given:
    fp32, or one byte an element (E4M3 codes of m and sqrt(v)) and one fp32
    scale for every 256 elements.  States that are not zero come whole: m with v,
    codes with their scales.  weight_decay and lr_scale: a number, or one
    for each tensor.  steps_done: steps taken before, as grad_norm counts them.
    """

    QBLOCK, CTL_BYTES = 256, 32768

    def __init__(self, params, grads, master=None, m=None, v=None, m_scale=None, v_scale=None, state_bits=32,
                 beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, lr_scale=1.0, seed=0, steps_done=0):
        params, grads = list(params), list(grads)
        if not params:
            raise ValueError("params: at least one tensor required")
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits: {state_bits}, expected 8 or 32")
        half = params[0].dtype == torch.bfloat16
        if not half and params[0].dtype != torch.float32:
            raise ValueError(f"params: dtype {params[0].dtype}, expected bfloat16 or float32")
        dev, sizes = params[0].device, [p.numel() for p in params]
        blocks = [-(-k // self.QBLOCK) for k in sizes]
        f32 = torch.float32

        def own(ts, counts, dtype):
            return [torch.zeros(k, dtype=dtype, device=dev) for k in counts] if ts is None else list(ts)

        self.params = self._each("params", params, sizes, params[0].dtype)
        if half and master is None:
            master = [p.detach().float().contiguous() for p in params]
        self.master = self._each("master", list(master), sizes, f32) if half else None
        m, v, m_scale, v_scale = (None if ts is None else list(ts) for ts in (m, v, m_scale, v_scale))
        if state_bits == 8:
            self._whole("m", m, "m_scale", m_scale)
            self._whole("v", v, "v_scale", v_scale)
        self._whole("m", m, "v", v)
        state = f32 if state_bits == 32 else torch.uint8
        self.m = self._each("m", own(m, sizes, state), sizes, state)
        self.v = self._each("v", own(v, sizes, state), sizes, state)
        self.m_scale = self.v_scale = None
        if state_bits == 8:
            self.m_scale = self._each("m_scale", own(m_scale, blocks, f32), blocks, f32)
            self.v_scale = self._each("v_scale", own(v_scale, blocks, f32), blocks, f32)
        self._sizes = sizes
        self.grads = self._grads(grads, grads[0].dtype if grads else None)
        self.state_bits, self.lr_scale, self.weight_decay = state_bits, lr_scale, weight_decay
        table = (AdamWTensor * len(params))()

        def value(name, x, i):
            if not isinstance(x, (list, tuple)):
                return float(x)
            if len(x) != len(params):
                raise ValueError(f"{name}: expected {len(params)} values, got {len(x)}")
            return float(x[i])

        for i, t in enumerate(table):
            t.param, t.grad = params[i].data_ptr(), grads[i].data_ptr()
            t.master = self.master[i].data_ptr() if half else None
            t.m, t.v = self.m[i].data_ptr(), self.v[i].data_ptr()
            if state_bits == 8:
                t.m_scale, t.v_scale = self.m_scale[i].data_ptr(), self.v_scale[i].data_ptr()
            t.n = sizes[i]
            t.lr_scale, t.weight_decay = value("lr_scale", lr_scale, i), value("weight_decay", weight_decay, i)
        d = AdamWDesc(len(params), DTYPE["bf16" if half else "f32"],
                      DTYPE["bf16" if grads[0].dtype == torch.bfloat16 else "f32"], int(state_bits), float(beta1),
                      float(beta2), float(eps), int(seed) & 0xFFFFFFFF)
        h = VP()
        _check(lib().tp_adamw_create(ctypes.byref(d), table, ctypes.byref(h)))
        self._h = h
        self.ctl = torch.empty(self.CTL_BYTES // 4, dtype=f32, device=dev)
        _check(lib().tp_adamw_ctl_init(self.ctl.data_ptr(), int(steps_done), _stream(None)))
        self._ctl = self.ctl.data_ptr()
        self._norm, self._step = lib().tp_adamw_grad_norm, lib().tp_adamw_step
        self.norm, self.scale = self.ctl[0:1], self.ctl[1:2]
        self.finite, self.steps = self.ctl.view(torch.int32)[2:3], self.ctl.view(torch.int32)[3:4]

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and _lib is not None:
            _lib.tp_adamw_destroy(h)
            self._h = None

    @staticmethod
    def _each(name, ts, counts, dtype):
        if len(ts) != len(counts):
            raise ValueError(f"{name}: expected {len(counts)} tensors, got {len(ts)}")
        for i, (t, n) in enumerate(zip(ts, counts)):
            if not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise ValueError(f"{name}[{i}]: must be a CUDA tensor")
            if t.dtype != dtype:
                raise ValueError(f"{name}[{i}]: dtype {t.dtype}, expected {dtype}")
            if not t.is_contiguous():
                raise ValueError(f"{name}[{i}]: must be contiguous")
            if t.numel() != n:
                raise ValueError(f"{name}[{i}]: {tuple(t.shape)} has {t.numel()} elements, expected {n}")
        return ts

    @staticmethod
    def _whole(name, ts, other, others):
        """Refuses one part of a state whose other part is missing, unless it is zero."""
        if (ts is None) == (others is None):
            return
        if ts is None:
            name, ts, other = other, others, name
        if any(bool(t.any()) for t in ts):
            raise ValueError(f"{other}: required with {name}")

    def _grads(self, grads, dtype):
        if dtype not in (torch.float32, torch.bfloat16):
            raise ValueError(f"grads: dtype {dtype}, expected float32 or bfloat16")
        return self._each("grads", grads, self._sizes, dtype)

    def set_grads(self, grads):
        """Take the gradients from these tensors (same sizes and type) from now on."""
        grads = self._grads(list(grads), self.grads[0].dtype)
        _check(lib().tp_adamw_set_grads(self._h, _arr([g.data_ptr() for g in grads])))
        self.grads = grads

    def grad_norm(self, grad_scale=1.0, max_norm=float("inf"), stream=None):
        """Enqueue the norm of grad_scale * grads and what the next step() takes
        from it: the clip factor, the step count (each call counts one) and
        whether the norm, and its square once clipped, are finite (if not, that
        step changes nothing and none is counted).  Returns the norm as a
        one-element CUDA tensor that the next call overwrites."""
        status = self._norm(self._h, grad_scale, max_norm, self._ctl, _stream(stream))
        if status:
            _check(status)
        return self.norm

    def step(self, lr, step=None, grad_scale=1.0, stream=None):
        """Enqueue one step: number `step` (from 1) on grad_scale * grads, or,
        with step=None, as the last grad_norm() call left it.  A captured step
        keeps the lr of its capture."""
        if step is None:
            status = self._step(self._h, lr, 1.0, 0, self._ctl, _stream(stream))
        else:
            status = self._step(self._h, lr, grad_scale, step, None, _stream(stream))
        if status:
            _check(status)


# ---------------------------------------------------------------------------
# attention around the projections
# ---------------------------------------------------------------------------
_i32, _f32 = torch.int32, torch.float32  # (an attribute of torch takes as long to find as one of a tensor)
ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "parts": 3}


class Rope:
    """How queries and keys turn with their position (tp_rope_desc).

    dim: rotated elements at the start of each head (None: the whole head; 0:
    no rotation); interleaved: pairs (2i, 2i+1) instead of (i, i + dim/2);
    scaling: "none", "linear", "ntk" or "parts" for contexts `factor` times
    longer ("parts" with the length `original` trained on and the turns `fast`
    and `slow` over it); attention_factor: of cosines and sines, None for the
    default (0.1 ln(factor) + 1 with "parts", else 1)."""

    def __init__(self, dim=None, base=10000.0, interleaved=False, scaling="none", factor=1.0, original=0, fast=32.0,
                 slow=1.0, attention_factor=None):
        self.dim, self.base, self.interleaved, self.scaling = dim, base, interleaved, scaling
        self.factor, self.original, self.fast, self.slow = factor, original, fast, slow
        if attention_factor is not None and not attention_factor:
            raise ValueError("attention_factor: 0 leaves no queries and keys")
        self.attention_factor = attention_factor

    def desc(self, head_dim: int) -> RopeDesc:
        return RopeDesc(int(head_dim) if self.dim is None else int(self.dim), int(bool(self.interleaved)),
                        ROPE_SCALING[self.scaling], float(self.base), float(self.factor), float(self.original),
                        float(self.fast), float(self.slow),
                        0.0 if self.attention_factor is None else float(self.attention_factor))


# a C array of an address and those `step`, 2 `step`, ... bytes on (a third of the time of packing a range)
_pack_parts = [eval("lambda a, s: pack(%s)" % ", ".join("a + %d * s" % i for i in range(k)), {"pack": _pack[k]})
               for k in range(MAX_SHARDS + 1)]


def _shards(name, ts, count, n, dtype, dev):
    """The addresses of `count` shards of n elements, a list of tensors or one
    tensor whose equal parts they are, as a C array; all on device `dev`."""
    try:
        if ts.dtype is dtype and ts.get_device() == dev and ts.is_contiguous() and ts.numel() == count * n:
            return _pack1(ts.data_ptr()) if count == 1 else _pack_parts[count](ts.data_ptr(), n * dtype.itemsize)
    except AttributeError:
        pass
    if isinstance(ts, torch.Tensor):
        ts, count, n = [ts], 1, count * n
    out = _pointers(name, ts, count, n, dtype)
    for t in ts:
        if t.get_device() != dev:
            raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{dev}")
    return out


def _vector(name, t, n, dtype, dev):
    """Address of a contiguous tensor of n elements on device `dev`."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and t.numel() == n:
            return t.data_ptr()
    except AttributeError:
        pass
    _pointer(name, t, n, dtype)
    raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{dev}")


def _stream_on(dev, stream):
    return _raw_stream(dev) if stream is None and _raw_stream is not None else _stream(stream)


# (torch.cuda.current_device without its check for a lazy start: a CUDA tensor is at hand)
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


class TPRotary:
    """Handle for the rotation of a QKV tensor's queries and keys
    (tp_rotary_create), in training: M = S*B tokens, T shards [M, (heads + 2
    kv_heads) / T * head_dim] as the QKV column layer leaves them, each a list
    of T tensors or one [T, ...] tensor.  grouped: a shard's columns are, key
    head by key head, its queries, the key and the value; otherwise all
    queries, all keys, all values."""

    def __init__(self, S, B, heads, kv_heads, head_dim, T=1, dtype="bf16", grouped=False, rope=None):
        rope = rope or Rope()
        self._d = RotaryDesc(int(S), int(B), int(T), int(heads), int(kv_heads), int(head_dim), DTYPE[dtype],
                             int(bool(grouped)), rope.desc(head_dim))
        h = VP()
        _check(lib().tp_rotary_create(ctypes.byref(self._d), ctypes.byref(h)))
        self._h = h
        self.M, self.T, self.dtype = int(S) * int(B), int(T), dtype
        self._act = TORCH_DTYPE[dtype]
        self._n = self.M * (int(heads) + 2 * int(kv_heads)) // self.T * int(head_dim)
        self._fwd, self._bwd = lib().tp_rotary_fwd, lib().tp_rotary_bwd

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and _lib is not None:
            _lib.tp_rotary_destroy(h)
            self._h = None

    def _run(self, call, x, x_name, y, y_name, positions, stream):
        dev = _device() if self.M else 0
        px = _shards(x_name, x, self.T, self._n, self._act, dev)
        py = px if y is None else _shards(y_name, y, self.T, self._n, self._act, dev)
        at = None if positions is None else _vector("positions", positions, self.M, _i32, dev)
        status = call(self._h, px, at, py, _stream_on(dev, stream))
        if status:
            _check(status)

    def fwd(self, X, Y=None, positions=None, stream=None):
        """Y = X with its queries and keys turned (None: in place).  positions:
        int32 [M], or None: token m = s*B + b is at position s; a token at a
        negative position is not turned."""
        self._run(self._fwd, X, "X", Y, "Y", positions, stream)

    def bwd(self, dY, dX=None, positions=None, stream=None):
        """dX = the gradient of X from dY (None: in place)."""
        self._run(self._bwd, dY, "dY", dX, "dX", positions, stream)


class TPPagedAttention:
    """Handle for a paged key-value cache and the attention of single tokens
    over it (tp_paged_create).

    The cache of shard i is K_i, V_i: [pages, kv_heads / T, page_size,
    head_dim], of the handle's type, or uint8 with dtype "fp8" (E4M3 codes of
    x * 448 / amax of the key head, from k_amax and v_amax, fp32 [kv_heads];
    everything else is bf16).  X, Q, K, V and O are lists of T tensors or one
    [T, ...] tensor each.  table: int32 [sequences, columns] of pages;
    positions and sequences: int32 [n], a row at a negative position is padding;
    sequences=None: row j is sequence j's.  window: positions that a token sees,
    its own among them (0: all); scale: of the scores (None: head_dim ** -0.5).
    rope: see Rope (None: the whole head, base 10000; Rope(dim=0): none)."""

    def __init__(self, heads, kv_heads, head_dim, page_size, pages, T=1, dtype="bf16", grouped=False, rope=None,
                 window=0, scale=None):
        rope = rope or Rope()
        if scale is not None and not ctypes.c_float(float(scale)).value:
            raise ValueError("scale: 0 (in fp32) leaves no attention")
        self._d = PagedDesc(int(T), int(heads), int(kv_heads), int(head_dim), DTYPE[dtype], int(bool(grouped)),
                            int(page_size), int(pages), int(window), 0.0 if scale is None else float(scale),
                            rope.desc(head_dim))
        h = VP()
        _check(lib().tp_paged_create(ctypes.byref(self._d), ctypes.byref(h)))
        self._h = h
        self.T, self.heads, self.kv_heads, self.head_dim, self.dtype = (int(T), int(heads), int(kv_heads),
                                                                        int(head_dim), dtype)
        self.cache_shape = (int(pages), self.kv_heads // self.T, int(page_size), self.head_dim)
        self.cache_dtype = torch.uint8 if dtype == "fp8" else TORCH_DTYPE[dtype]
        self._act = TORCH_DTYPE[dtype]
        self._cache_n = _prod(self.cache_shape)
        self._q_n = self.heads // self.T * self.head_dim
        self._x_n = (self.heads + 2 * self.kv_heads) // self.T * self.head_dim
        self._append, self._decode = lib().tp_paged_append, lib().tp_paged_decode

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and _lib is not None:
            _lib.tp_paged_destroy(h)
            self._h = None

    def workspace_bytes(self) -> int:
        return int(lib().tp_paged_workspace_bytes(self._h))

    def sync_status(self, stream=None) -> int:
        """Synchronise the stream and return (and clear) this handle's index
        word: TP_ERR_INDEX when a call met a page, sequence or position out of
        range."""
        return int(lib().tp_paged_sync_status(self._h, _stream(stream)))

    def _rows(self, positions, sequences, table, k_amax, v_amax, dev):
        try:
            (n,), (rows, cols) = positions.shape, table.shape
        except (AttributeError, ValueError):
            raise ValueError("positions: must be a CUDA tensor [n], table: one [sequences, columns]") from None
        at = (_vector("positions", positions, n, _i32, dev),
              None if sequences is None else _vector("sequences", sequences, n, _i32, dev), n,
              _vector("table", table, rows * cols, _i32, dev), rows, cols)
        if self.dtype != "fp8":
            return at + (None, None)
        return at + (_vector("k_amax", k_amax, self.kv_heads, _f32, dev),
                     _vector("v_amax", v_amax, self.kv_heads, _f32, dev))

    def append(self, X, positions, table, K, V, Q, sequences=None, k_amax=None, v_amax=None, stream=None):
        """New tokens X [n, (heads + 2 kv_heads) / T * head_dim] a shard: turned
        queries to Q [n, heads / T * head_dim], turned keys and values to the
        slots of their positions.  No two rows name the same slot."""
        dev, T, act = _device(), self.T, self._act
        rows = self._rows(positions, sequences, table, k_amax, v_amax, dev)
        n = rows[2]
        status = self._append(self._h, _shards("X", X, T, n * self._x_n, act, dev), *rows,
                              _shards("Q", Q, T, n * self._q_n, act, dev),
                              _shards("K", K, T, self._cache_n, self.cache_dtype, dev),
                              _shards("V", V, T, self._cache_n, self.cache_dtype, dev), _stream_on(dev, stream))
        if status:
            _check(status)

    def decode(self, Q, positions, table, K, V, O, workspace, sequences=None, k_amax=None, v_amax=None, stream=None):
        """O [n, heads / T * head_dim] a shard (it may be Q) = attention of each
        row's queries over positions max(0, p - window + 1)..p of its sequence;
        zero for padding.  workspace: see alloc_workspace, one for each of the
        calls that may overlap."""
        dev, T, act = _device(), self.T, self._act
        rows = self._rows(positions, sequences, table, k_amax, v_amax, dev)
        n = rows[2]
        ws, nws = _workspace(workspace)
        status = self._decode(self._h, _shards("Q", Q, T, n * self._q_n, act, dev), *rows,
                              _shards("K", K, T, self._cache_n, self.cache_dtype, dev),
                              _shards("V", V, T, self._cache_n, self.cache_dtype, dev),
                              _shards("O", O, T, n * self._q_n, act, dev), ws, nws, _stream_on(dev, stream))
        if status:
            _check(status)


# ---------------------------------------------------------------------------
# status / diagnostics
# ---------------------------------------------------------------------------
def sync_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the status word of the
    calls without a handle (single layers, FP8 quantiser); MLP and sub-block
    handles report through their own sync_status()."""
    return int(lib().tp_sync_status(_stream(stream)))


def set_wait_limit_ns(ns: int):
    lib().tp_set_wait_limit_ns(int(ns))


def debug_wait_timeout(limit_ns: int, stream=None):
    _check(lib().tp_debug_wait_timeout(int(limit_ns), _stream(stream)))


TILE_MODES = {"auto": 0, "single": 1, "pair": 2}


def set_tile_mode(mode: str):
    """GEMM tiling of the bf16 engine: "auto", "single" (128-row tiles, one
    CTA) or "pair" (256-row tiles on a CTA pair)."""
    _check(lib().tp_set_tile_mode(TILE_MODES[mode]))


def set_tail_split(on: bool):
    """Tail split of the pair-tile GEMMs (on by default): the last,
    part-filled round of tiles is cut along K over all CTA pairs."""
    _check(lib().tp_set_tail_split(1 if on else 0))


def set_k_order(alternate: bool):
    """Every other persistent round of the pair GEMMs (row forward, column
    dgrad, weight gradients) walks K backwards (True, the default) so that
    it starts on what the previous round left in L2; False: always forwards."""
    _check(lib().tp_set_k_order(1 if alternate else 0))


def set_launch_overlap(on: bool):
    """Programmatic dependent launch of the pair GEMMs, the block norm, AdamW,
    the rotation and the paged attention (on by default): a kernel's CTAs set up while the previous kernel finishes and wait for it
    before touching memory; False: plain stream order."""
    _check(lib().tp_set_launch_overlap(1 if on else 0))


def set_band_rows(rows: int):
    """Rows of 256-row tiles per raster band of the pair GEMMs' tile order
    (0: the library's choice)."""
    _check(lib().tp_set_band_rows(int(rows)))


def set_max_gemm_pairs(n: int):
    """Upper bound on the CTA pairs of the pair-tile GEMMs (0: all that fit)."""
    _check(lib().tp_set_max_gemm_pairs(int(n)))


def tail_split_count() -> int:
    """GEMM launches since load that split their last round's tiles."""
    return int(lib().tp_tail_split_count())


FUSED_MODES = {"auto": 0, "off": 1, "on": 2}


def set_fused_fwd(mode: str):
    """Forward as one fused kernel for narrow bf16 MLPs (H <= 256): "auto"
    (default) and "on" run it whenever the shape allows it (it measures faster
    than the two GEMMs there), "off" runs the column and row GEMM kernels;
    see include/tp_mlp.h."""
    _check(lib().tp_set_fused_fwd(FUSED_MODES[mode]))


def launch_count() -> int:
    return int(lib().tp_launch_count())


def prof_enable(on: bool = True):
    lib().tp_prof_enable(1 if on else 0)


def prof_select(kernel=None):
    """Time only the launches of `kernel` with events (None: every launch);
    the GEMMs' clock counters keep counting for all kernels."""
    lib().tp_prof_select(kernel.encode() if kernel else None)


def prof_collect(clocks: bool = False):
    """{kernel name: (launches, total device ms)} since the last collect;
    with clocks=True {name: (launches, total ms, SM cycles, SM ns)}, the last
    two summed over the CTAs of GEMM launches (0 for other kernels)."""
    buf = (ProfEntry * 64)()
    n = lib().tp_prof_collect(buf, 64)
    if n < 0:
        raise TpError(4, lib().tp_last_error().decode(errors="replace"))
    if clocks:
        return {buf[i].name.decode(): (buf[i].launches, buf[i].total_ms, buf[i].sm_cycles, buf[i].sm_ns)
                for i in range(n)}
    return {buf[i].name.decode(): (buf[i].launches, buf[i].total_ms) for i in range(n)}


def status_str(s: int) -> str:
    return lib().tp_status_str(int(s)).decode()
