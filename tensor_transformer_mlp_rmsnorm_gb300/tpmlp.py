"""ctypes binding of the tpmlp C ABI (``include/tpmlp.h``).

Argument marshalling only: every step of the sublayer runs in the CUDA
library.  torch supplies device memory and the stream; nothing here computes.
The module raises ``TPMLPError`` if the shared library has not been built --
there is no fallback.

Functions named like the C entry points take torch tensors; ``TPMLP`` wraps a
context together with its workspace.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libtpmlp.so")

OK, ERR_ARG, ERR_SHAPE, ERR_UNSUPPORTED, ERR_ORDER, ERR_CUDA, ERR_TIMEOUT = range(7)
F32, BF16 = 0, 1
SWIGLU, GELU = 0, 1
DBG_SKIP_FWD_REDUCE, DBG_SKIP_BWD_REDUCE, DBG_FORCE_TIMEOUT, DBG_GEMM_SINGLE_CTA = 1, 2, 4, 8
DBG_SKIP_SP_GRAD_SYNC = 16
PREC_BF16, PREC_FP8 = 0, 1

_DTYPES = {"f32": F32, "bf16": BF16}
_ACTS = {"swiglu": SWIGLU, "gelu": GELU}
_TORCH_DTYPE = {F32: torch.float32, BF16: torch.bfloat16}


class TPMLPError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"tpmlp status {status}: {msg}")
        self.status = status


class AttnConfig(ctypes.Structure):
    """tpattn_config."""
    _fields_ = [("max_tokens", ctypes.c_int64), ("hidden", ctypes.c_int64), ("n_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("max_seq", ctypes.c_int32),
                ("max_t", ctypes.c_int32), ("dtype", ctypes.c_int32), ("flags", ctypes.c_int32)]


class ParamSet(ctypes.Structure):
    """tpmlp_param_set: one device float* per parameter (b_1 for GeLU only)."""
    _fields_ = [("norm_w", ctypes.c_void_p), ("w_gate_up", ctypes.c_void_p), ("b_1", ctypes.c_void_p),
                ("w_down", ctypes.c_void_p), ("b_down", ctypes.c_void_p)]


class AttnParamSet(ctypes.Structure):
    """tpattn_param_set: one device float* per attention parameter."""
    _fields_ = [("norm_w", ctypes.c_void_p), ("w_qkv", ctypes.c_void_p), ("w_o", ctypes.c_void_p),
                ("b_o", ctypes.c_void_p)]


class AdamWParams(ctypes.Structure):
    """tpmlp_adamw_params."""
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float), ("max_grad_norm", ctypes.c_float),
                ("step", ctypes.c_int64)]


class Config(ctypes.Structure):
    _fields_ = [("max_tokens", ctypes.c_int64), ("hidden", ctypes.c_int64), ("ffn", ctypes.c_int64),
                ("max_t", ctypes.c_int32), ("dtype", ctypes.c_int32), ("act", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


MAX_ROT_DIM = 256


class RotarySpec(ctypes.Structure):
    """tpattn_rotary."""
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("turn", ctypes.c_uint64 * (MAX_ROT_DIM // 2))]


class QkDesc(ctypes.Structure):
    """tpattn_qk_desc."""
    _fields_ = [("rows", ctypes.c_int64), ("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("positions", ctypes.c_void_p),
                ("seq", ctypes.c_int64), ("q_norm_w", ctypes.c_void_p), ("k_norm_w", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("reserved", ctypes.c_int32)]


class QkParams(ctypes.Structure):
    """tpattn_qk_params."""
    _fields_ = [("rot", ctypes.POINTER(RotarySpec))] + [
        (n, ctypes.c_void_p) for n in ("q_norm_w", "k_norm_w", "dq_norm_w", "dk_norm_w", "master_q", "master_k", "m_q",
                                       "m_k", "v_q", "v_k")] + [("eps", ctypes.c_float), ("reserved", ctypes.c_int32)]


class KvConfig(ctypes.Structure):
    """tpkv_config."""
    _fields_ = [("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32), ("max_batch", ctypes.c_int32),
                ("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("cache_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_vp, _i32, _i64, _u32, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_float
_fp = ctypes.c_void_p  # float* (device)
_SIGNATURES = {
    "tpmlp_create": (_i32, [ctypes.POINTER(Config), _vp, ctypes.POINTER(_vp)]),
    "tpmlp_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(Config)]),
    "tpmlp_bind_workspace": (_i32, [_vp, _vp, ctypes.c_size_t]),
    "tpmlp_set_stream": (_i32, [_vp, _vp]),
    "tpmlp_forward": (_i32, [_vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _f32, _i32, _vp]),
    "tpmlp_mse_loss_grad": (_i32, [_vp, _vp, _vp, _vp, _fp]),
    "tpmlp_backward": (_i32, [_vp, _vp, _vp, _fp, _fp, _fp, _fp, _fp]),
    "tpmlp_bind_master": (_i32, [_vp, _fp, _fp, _fp, _fp, _fp]),
    "tpmlp_sgd_step": (_i32, [_vp, _f32]),
    "tpmlp_bind_adam_state": (_i32, [_vp, ctypes.POINTER(ParamSet), ctypes.POINTER(ParamSet)]),
    "tpmlp_adamw_step": (_i32, [_vp, ctypes.POINTER(AdamWParams), _fp]),
    "tpmlp_set_debug": (_i32, [_vp, _u32, _i32]),
    "tpmlp_set_sequence_parallel": (_i32, [_vp, _i32]),
    "tpmlp_set_update_in_backward": (_i32, [_vp, _i32, _f32]),
    "tpmlp_update_in_epilogue": (_i32, [_vp]),
    "tpmlp_fp8_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(Config)]),
    "tpmlp_bind_fp8_workspace": (_i32, [_vp, _vp, ctypes.c_size_t]),
    "tpmlp_set_precision": (_i32, [_vp, _i32]),
    "tpmlp_sync": (_i32, [_vp]),
    "tpmlp_set_timing": (_i32, [_vp, _i32]),
    "tpmlp_read_kernel_times": (_i32, [_vp, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int64), _i32]),
    "tpmlp_kernel_name": (ctypes.c_char_p, [_i32]),
    "tpmlp_num_kernel_ids": (_i32, []),
    "tpmlp_launch_count": (ctypes.c_uint64, [_vp]),
    "tpmlp_status_string": (ctypes.c_char_p, [_i32]),
    "tpmlp_last_error": (ctypes.c_char_p, [_vp]),
    "tpmlp_destroy": (None, [_vp]),
    "tpmlp_mse_loss_grad_noalloc": (_i32, [_i32, _i64, _vp, _vp, _vp, _fp, _vp]),
    "tpattn_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(AttnConfig)]),
    "tpattn_create": (_i32, [ctypes.POINTER(AttnConfig), _vp, ctypes.POINTER(_vp)]),
    "tpattn_bind_workspace": (_i32, [_vp, _vp, ctypes.c_size_t]),
    "tpattn_forward": (_i32, [_vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _f32, _i32, _vp]),
    "tpattn_backward": (_i32, [_vp, _vp, _vp, _fp, _fp, _fp, _fp]),
    "tpattn_bind_master": (_i32, [_vp, _fp, _fp, _fp, _fp]),
    "tpattn_sgd_step": (_i32, [_vp, _f32]),
    "tpattn_set_update_in_backward": (_i32, [_vp, _i32, _f32]),
    "tpattn_update_in_epilogue": (_i32, [_vp]),
    "tpattn_bind_adam_state": (_i32, [_vp, ctypes.POINTER(AttnParamSet), ctypes.POINTER(AttnParamSet)]),
    "tpattn_adamw_step": (_i32, [_vp, ctypes.POINTER(AdamWParams), _fp]),
    "tpattn_set_fused": (_i32, [_vp, _i32]),
    "tpattn_fused_active": (_i32, [_vp]),
    "tpattn_sync": (_i32, [_vp]),
    "tpattn_set_timing": (_i32, [_vp, _i32]),
    "tpattn_read_kernel_times": (_i32, [_vp, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int64), _i32]),
    "tpattn_kernel_name": (ctypes.c_char_p, [_i32]),
    "tpattn_num_kernel_ids": (_i32, []),
    "tpattn_launch_count": (ctypes.c_uint64, [_vp]),
    "tpattn_last_error": (ctypes.c_char_p, [_vp]),
    "tpattn_destroy": (None, [_vp]),
    "tpattn_rotary_init": (_i32, [ctypes.POINTER(RotarySpec), _i32, _i32, ctypes.POINTER(ctypes.c_double)]),
    "tpattn_qk_rope_forward": (_i32, [ctypes.POINTER(QkDesc), ctypes.POINTER(RotarySpec), _vp, _i64, _vp, _i64, _vp]),
    "tpattn_qk_rope_workspace_bytes": (ctypes.c_size_t, [_i32]),
    "tpattn_qk_rope_backward": (_i32, [ctypes.POINTER(QkDesc), ctypes.POINTER(RotarySpec), _vp, _i64, _vp, _i64, _vp,
                                       _i64, _fp, _fp, _vp, ctypes.c_size_t, _vp]),
    "tpattn_qk_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(AttnConfig)]),
    "tpattn_set_qk": (_i32, [_vp, ctypes.POINTER(QkParams), _vp, ctypes.c_size_t]),
    "tpattn_append_kv": (_i32, [_vp, _vp, _vp, _vp, _i64, _i32]),
    "tpattn_decode": (_i32, [_vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _f32, _i32, _vp, _vp, _i64, _i32, _i32, _i32, _vp]),
    "tpkv_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(KvConfig)]),
    "tpkv_create": (_i32, [ctypes.POINTER(KvConfig), _vp, ctypes.POINTER(_vp)]),
    "tpkv_bind_workspace": (_i32, [_vp, _vp, ctypes.c_size_t]),
    "tpkv_set_stream": (_i32, [_vp, _vp]),
    "tpkv_bind_cache": (_i32, [_vp, _vp, _vp, _i64, _i64, _i64, _fp, _fp]),
    "tpkv_set_rotary": (_i32, [_vp, ctypes.POINTER(RotarySpec), _vp, _vp, _f32]),
    "tpkv_append": (_i32, [_vp, _i64, _i32, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _vp, _i64]),
    "tpkv_decode": (_i32, [_vp, _i32, _vp, _i64, _vp, _i32, _vp, _i64, _i32, _f32, _i32, _i32, _vp, _i64, _fp]),
    "tpkv_sync": (_i32, [_vp]),
    "tpkv_launch_count": (ctypes.c_uint64, [_vp]),
    "tpkv_last_error": (ctypes.c_char_p, [_vp]),
    "tpkv_destroy": (None, [_vp]),
    "tpmlp_fp8_quantize": (_i32, [_vp, _i64, _i64, _vp, _i64, _vp, _i64, _fp, _vp, _vp]),
    "tpmlp_fp8_gemm": (_i32, [_vp, _i64, _vp, _i64, _i64, _i64, _i64, _fp, _fp, _fp, _i64, _vp, _vp]),
}
TPATTN_FUSED_ONLY = 1  # tpattn_config.flags: only the fused attention kernels, no score square
FP8_SCRATCH_BYTES = 4096
NOALLOC_LOSS_MAX_BLOCKS = 1024

_LIB = None


def lib() -> ctypes.CDLL:
    """The loaded C library; raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise TPMLPError(ERR_UNSUPPORTED, f"{LIB_PATH} is missing: build it with "
                             "tensor_transformer_mlp_rmsnorm_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = L
    return _LIB


def _check(status: int, ctx=None):
    if status != OK:
        msg = lib().tpmlp_last_error(ctx).decode(errors="replace")
        raise TPMLPError(status, msg or lib().tpmlp_status_string(status).decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def kernel_names() -> list:
    L = lib()
    return [L.tpmlp_kernel_name(i).decode() for i in range(L.tpmlp_num_kernel_ids())]


def make_config(max_tokens: int, hidden: int, ffn: int, max_t: int = 8, dtype: str = "bf16",
                act: str = "swiglu") -> Config:
    return Config(max_tokens, hidden, ffn, max_t, _DTYPES[dtype], _ACTS[act], 0)


def tpmlp_workspace_bytes(cfg: Config) -> int:
    return int(lib().tpmlp_workspace_bytes(ctypes.byref(cfg)))


def tpmlp_create(cfg: Config, stream=None):
    out = ctypes.c_void_p()
    s = None if stream is None else ctypes.c_void_p(stream)
    _check(lib().tpmlp_create(ctypes.byref(cfg), s, ctypes.byref(out)))
    return out


def tpmlp_mse_loss_grad_noalloc(y, target, dy, loss, stream=None):
    """Loss and gradient without a context or workspace (no device allocation
    by the library); y, target, dy: same dtype and size, loss: one float."""
    dt = {torch.float32: F32, torch.bfloat16: BF16}.get(y.dtype)
    if dt is None or target.dtype != y.dtype or dy.dtype != y.dtype or loss.dtype != torch.float32:
        raise TPMLPError(ERR_ARG, "y/target/dy must share dtype float32 or bfloat16; loss must be float32")
    if target.numel() != y.numel() or dy.numel() != y.numel() or loss.numel() < 1:
        raise TPMLPError(ERR_ARG, "y, target and dy must have the same number of elements")
    for t in (y, target, dy, loss):
        if not t.is_cuda or not t.is_contiguous():
            raise TPMLPError(ERR_ARG, "tensors must be contiguous CUDA tensors")
    s = stream if stream is not None else torch.cuda.current_stream(y.device).cuda_stream
    with torch.cuda.device(y.device):
        _check(lib().tpmlp_mse_loss_grad_noalloc(dt, y.numel(), _ptr(y), _ptr(target), _ptr(dy), _ptr(loss),
                                                 ctypes.c_void_p(s)))
    return loss, dy


def _pitch16(n: int) -> int:
    return (n + 15) // 16 * 16


def fp8_quantize(src, rows_major: bool = True, transposed: bool = True, stream=None):
    """E4M3 codes of a bf16 tensor [rows, cols] with its per-tensor scale
    (tpmlp_fp8_quantize).  Returns (codes [rows, pitch] or None,
    codes_t [cols, pitch] or None, inv_scale [1] float): the pitches are
    rounded up to 16 bytes; columns past cols (rows past rows) are padding."""
    if src.dtype != torch.bfloat16 or src.dim() != 2 or not src.is_contiguous():
        raise TPMLPError(ERR_ARG, "src must be a contiguous 2-D bf16 tensor")
    rows, cols = src.shape
    dev = src.device
    dst = torch.empty(rows, _pitch16(cols), dtype=torch.uint8, device=dev) if rows_major else None
    dst_t = torch.empty(cols, _pitch16(rows), dtype=torch.uint8, device=dev) if transposed else None
    inv = torch.empty(1, dtype=torch.float32, device=dev)
    scratch = torch.empty(FP8_SCRATCH_BYTES, dtype=torch.uint8, device=dev)
    st = (stream or torch.cuda.current_stream(dev)).cuda_stream
    _check(lib().tpmlp_fp8_quantize(_ptr(src), rows, cols, _ptr(dst) if dst is not None else None,
                                    dst.shape[1] if dst is not None else 0,
                                    _ptr(dst_t) if dst_t is not None else None,
                                    dst_t.shape[1] if dst_t is not None else 0, _ptr(inv), _ptr(scratch), st))
    return dst, dst_t, inv


def fp8_gemm(a, b, k: int, inv_a, inv_b, n: int | None = None, stream=None):
    """c = (a b^T) * inv_a * inv_b from E4M3 codes a [M, pitch], b [N, pitch]
    whose first k bytes per row are the operand (tpmlp_fp8_gemm)."""
    M = a.shape[0]
    N = b.shape[0] if n is None else n
    c = torch.empty(M, N, dtype=torch.float32, device=a.device)
    status = torch.zeros(1, dtype=torch.int32, device=a.device)
    st = (stream or torch.cuda.current_stream(a.device)).cuda_stream
    _check(lib().tpmlp_fp8_gemm(_ptr(a), a.shape[1], _ptr(b), b.shape[1], M, N, k, _ptr(inv_a), _ptr(inv_b),
                                _ptr(c), N, _ptr(status), st))
    return c, status


class TPMLP:
    """One context of the sublayer with its caller-owned workspace.

    Methods mirror the C entry points: ``forward``, ``mse_loss_grad``,
    ``backward``, ``bind_master``, ``sgd_step``, ``set_debug``, ``sync``."""

    def __init__(self, max_tokens: int, hidden: int, ffn: int, max_t: int = 8, dtype: str = "bf16",
                 act: str = "swiglu", device=None, stream: torch.cuda.Stream | None = None):
        dev = torch.device(device) if device is not None else torch.device("cuda")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        self.cfg = make_config(max_tokens, hidden, ffn, max_t, dtype, act)
        self.dtype = _TORCH_DTYPE[_DTYPES[dtype]]
        self.act = act
        self.H, self.F = hidden, ffn
        self.stream = stream if stream is not None else torch.cuda.current_stream(self.device)
        with torch.cuda.device(self.device):
            self.ctx = tpmlp_create(self.cfg, self.stream.cuda_stream)
            nbytes = tpmlp_workspace_bytes(self.cfg)
            self.workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.device)
        _check(lib().tpmlp_bind_workspace(self.ctx, _ptr(self.workspace), nbytes), self.ctx)
        self.tokens = 0
        self._fwd = False
        self._loss = torch.zeros(1, dtype=torch.float32, device=self.device)
        self._gn = torch.zeros(1, dtype=torch.float32, device=self.device)
        self._adam = None

    def close(self):
        if getattr(self, "ctx", None):
            lib().tpmlp_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- checks ------------------------------------------------------------
    def _t(self, t, shape, dtype=None, name="tensor"):
        if t is None:
            raise TPMLPError(ERR_ARG, f"{name} is None")
        want = dtype if dtype is not None else self.dtype
        if t.device != self.device or t.dtype != want or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
            raise TPMLPError(ERR_ARG, f"{name}: need contiguous {want} {tuple(shape)} on {self.device}, "
                                      f"got {t.dtype} {tuple(t.shape)} on {t.device}")
        return _ptr(t)

    def _gu_shape(self):
        return (2, self.F, self.H) if self.act == "swiglu" else (self.F, self.H)

    # -- entry points --------------------------------------------------------
    def forward(self, x, norm_w, w_gate_up, w_down, b_down, eps: float, t: int, y=None, b_1=None):
        n = x.shape[0]
        if y is None:
            y = torch.empty_like(x)
        args = (self._t(x, (n, self.H), name="x"), self._t(norm_w, (self.H,), name="norm_w"),
                self._t(w_gate_up, self._gu_shape(), name="w_gate_up"),
                self._t(b_1, (self.F,), name="b_1") if self.act == "gelu" else None,
                self._t(w_down, (self.H, self.F), name="w_down"), self._t(b_down, (self.H,), name="b_down"))
        yp = self._t(y, (n, self.H), name="y")
        self._fwd = False
        _check(lib().tpmlp_forward(self.ctx, n, *args, float(eps), int(t), yp), self.ctx)
        # the library keeps these pointers (backward reads x; the updates write the parameters):
        # hold the tensors until the next forward so that a temporary argument is not freed
        self._fwd_tensors = (x, norm_w, w_gate_up, b_1, w_down, b_down)
        self.tokens = n
        self._fwd = True
        return y

    def _need_forward(self, what):
        if not self._fwd:
            raise TPMLPError(ERR_ORDER, f"{what} before forward")

    def mse_loss_grad(self, y, target, dy=None, loss=None):
        self._need_forward("mse_loss_grad")
        n = self.tokens
        dy = torch.empty_like(y) if dy is None else dy
        loss = self._loss if loss is None else loss
        _check(lib().tpmlp_mse_loss_grad(self.ctx, self._t(y, (n, self.H), name="y"),
                                         self._t(target, (n, self.H), name="target"),
                                         self._t(dy, (n, self.H), name="dy"),
                                         self._t(loss, (1,), torch.float32, "loss")), self.ctx)
        return loss, dy

    def new_grads(self):
        f32 = dict(dtype=torch.float32, device=self.device)
        g = {"norm_w": torch.empty(self.H, **f32), "w_gate_up": torch.empty(self._gu_shape(), **f32),
             "w_down": torch.empty(self.H, self.F, **f32), "b_down": torch.empty(self.H, **f32)}
        if self.act == "gelu":
            g["b_1"] = torch.empty(self.F, **f32)
        return g

    def backward(self, dy, dx=None, grads=None):
        self._need_forward("backward")
        n = self.tokens
        dx = torch.empty_like(dy) if dx is None else dx
        g = self.new_grads() if grads is None else grads
        f32 = torch.float32
        _check(lib().tpmlp_backward(
            self.ctx, self._t(dy, (n, self.H), name="dy"), self._t(dx, (n, self.H), name="dx"),
            self._t(g["norm_w"], (self.H,), f32, "dnorm_w"), self._t(g["w_gate_up"], self._gu_shape(), f32, "dw_gate_up"),
            self._t(g["b_1"], (self.F,), f32, "db_1") if self.act == "gelu" else None,
            self._t(g["w_down"], (self.H, self.F), f32, "dw_down"), self._t(g["b_down"], (self.H,), f32, "db_down")),
            self.ctx)
        # the updates read these gradients later: hold them until the next backward
        self._grads = g
        return dx, g

    def bind_master(self, masters: dict | None):
        f32 = torch.float32
        if masters is None:
            _check(lib().tpmlp_bind_master(self.ctx, None, None, None, None, None), self.ctx)
            self._masters = None
            return
        _check(lib().tpmlp_bind_master(
            self.ctx, self._t(masters["norm_w"], (self.H,), f32, "norm_w"),
            self._t(masters["w_gate_up"], self._gu_shape(), f32, "w_gate_up"),
            self._t(masters["b_1"], (self.F,), f32, "b_1") if self.act == "gelu" else None,
            self._t(masters["w_down"], (self.H, self.F), f32, "w_down"),
            self._t(masters["b_down"], (self.H,), f32, "b_down")), self.ctx)
        self._masters = masters  # keep the tensors alive while bound

    def sgd_step(self, lr: float):
        _check(lib().tpmlp_sgd_step(self.ctx, float(lr)), self.ctx)

    def set_update_in_backward(self, enable: bool, lr: float = 0.0):
        """Have backward apply the SGD update itself (bf16 with bound masters); sgd_step is then not called."""
        _check(lib().tpmlp_set_update_in_backward(self.ctx, int(bool(enable)), float(lr)), self.ctx)

    def update_in_epilogue(self) -> bool:
        """Whether the last backward updated the weight matrices inside their gradient GEMMs' epilogues."""
        return bool(lib().tpmlp_update_in_epilogue(self.ctx))

    def _param_set(self, d: dict, what: str) -> ParamSet:
        f32 = torch.float32
        return ParamSet(self._t(d["norm_w"], (self.H,), f32, f"{what}.norm_w"),
                        self._t(d["w_gate_up"], self._gu_shape(), f32, f"{what}.w_gate_up"),
                        self._t(d["b_1"], (self.F,), f32, f"{what}.b_1") if self.act == "gelu" else None,
                        self._t(d["w_down"], (self.H, self.F), f32, f"{what}.w_down"),
                        self._t(d["b_down"], (self.H,), f32, f"{what}.b_down"))

    def new_adam_state(self):
        """Zeroed first and second moments shaped like the parameters (fp32), bound to this context."""
        m = {k: torch.zeros_like(v) for k, v in self.new_grads().items()}
        v = {k: torch.zeros_like(t) for k, t in m.items()}
        self.bind_adam_state(m, v)
        return m, v

    def bind_adam_state(self, m: dict | None, v: dict | None):
        if m is None and v is None:
            _check(lib().tpmlp_bind_adam_state(self.ctx, None, None), self.ctx)
            self._adam = None
            return
        ms, vs = self._param_set(m, "m"), self._param_set(v, "v")
        _check(lib().tpmlp_bind_adam_state(self.ctx, ctypes.byref(ms), ctypes.byref(vs)), self.ctx)
        self._adam = (m, v)  # keep the tensors alive while bound

    def adamw_step(self, lr: float, step: int, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                   weight_decay: float = 0.1, max_grad_norm: float = 1.0, grad_norm=None):
        """One clipped AdamW update; returns the device float holding the global gradient norm."""
        gn = self._gn if grad_norm is None else grad_norm
        hp = AdamWParams(float(lr), float(beta1), float(beta2), float(eps), float(weight_decay),
                         float(max_grad_norm), int(step))
        _check(lib().tpmlp_adamw_step(self.ctx, ctypes.byref(hp), self._t(gn, (1,), torch.float32, "grad_norm")),
               self.ctx)
        return gn

    def set_precision(self, precision: str):
        """"bf16" or "fp8" GEMM operands; the first switch to FP8 allocates and binds its workspace."""
        prec = {"bf16": PREC_BF16, "fp8": PREC_FP8}[precision]
        if prec == PREC_FP8 and getattr(self, "workspace8", None) is None:
            nbytes = lib().tpmlp_fp8_workspace_bytes(ctypes.byref(self.cfg))
            if nbytes == 0:
                raise TPMLPError(ERR_UNSUPPORTED, "FP8 needs the bf16 dtype")
            self.workspace8 = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
            _check(lib().tpmlp_bind_fp8_workspace(self.ctx, _ptr(self.workspace8), nbytes), self.ctx)
        _check(lib().tpmlp_set_precision(self.ctx, prec), self.ctx)
        self._fwd = False

    def set_sequence_parallel(self, enable: bool):
        _check(lib().tpmlp_set_sequence_parallel(self.ctx, int(bool(enable))), self.ctx)
        self._fwd = False

    def set_debug(self, flags: int, shard: int = 0):
        _check(lib().tpmlp_set_debug(self.ctx, int(flags), int(shard)), self.ctx)

    def sync(self):
        _check(lib().tpmlp_sync(self.ctx), self.ctx)

    def set_timing(self, enable: bool):
        _check(lib().tpmlp_set_timing(self.ctx, 1 if enable else 0), self.ctx)

    def read_kernel_times(self) -> dict:
        n = lib().tpmlp_num_kernel_ids()
        ms = (ctypes.c_float * n)()
        cnt = (ctypes.c_int64 * n)()
        m = lib().tpmlp_read_kernel_times(self.ctx, ms, cnt, n)
        if m < 0:
            raise TPMLPError(ERR_CUDA, "reading kernel times failed")
        names = kernel_names()
        return {names[i]: (float(ms[i]), int(cnt[i])) for i in range(m) if cnt[i] > 0}

    def launch_count(self) -> int:
        return int(lib().tpmlp_launch_count(self.ctx))


def _acheck(status: int, ctx=None):
    if status != OK:
        msg = lib().tpattn_last_error(ctx).decode(errors="replace")
        raise TPMLPError(status, msg or lib().tpmlp_status_string(status).decode())


class TPAttn:
    """The tensor-parallel attention sublayer through the C ABI (tpattn_*):
    bf16 tensors on one CUDA device; the workspace is a torch uint8 tensor.

    Calls run on ``stream`` (torch's current stream at construction unless given; the one that is captured, for calls
    to be replayed from a graph).  Where another one is current at a call, ordering the two is the caller's; the memory
    of what the call uses is not handed out again before the stream is past it."""

    def __init__(self, max_tokens: int, hidden: int, n_heads: int, n_kv_heads: int, head_dim: int,
                 max_seq: int, max_t: int = 8, device=None, stream=None, fused_only: bool = False):
        dev = torch.device(device) if device is not None else torch.device("cuda")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        self.cfg = AttnConfig(max_tokens, hidden, n_heads, n_kv_heads, head_dim, max_seq, max_t, BF16,
                              TPATTN_FUSED_ONLY if fused_only else 0)
        self.H, self.nq, self.nkv, self.d = hidden, n_heads, n_kv_heads, head_dim
        self.W = (n_heads + 2 * n_kv_heads) * head_dim
        self.stream = stream if stream is not None else torch.cuda.current_stream(dev)
        ctx = ctypes.c_void_p()
        with torch.cuda.device(dev), torch.cuda.stream(self.stream):  # the workspace belongs to that stream
            _acheck(lib().tpattn_create(ctypes.byref(self.cfg), self.stream.cuda_stream, ctypes.byref(ctx)))
            self.ctx = ctx
            nbytes = int(lib().tpattn_workspace_bytes(ctypes.byref(self.cfg)))
            self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        _acheck(lib().tpattn_bind_workspace(self.ctx, _ptr(self.workspace), nbytes), self.ctx)
        self._masters = None
        self.tokens = None  # set by forward; the C ABI reports a backward before it

    def close(self):
        if getattr(self, "ctx", None):
            lib().tpattn_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _uses(self, *tensors):
        """Keeps the memory of a call's tensors from reuse until the stream is past the call, where they may belong to
        another stream."""
        if _stream_of(self.device, self.device.index) != self.stream.cuda_stream:
            _record(self.stream, *tensors)

    def _t(self, t, shape, dtype=torch.bfloat16, name="tensor"):
        if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or t.device != self.device:
            raise TPMLPError(ERR_ARG, f"{name}: expected contiguous {dtype} {tuple(shape)} on {self.device}")
        return _ptr(t)

    def forward(self, x, norm_w, w_qkv, w_o, b_o, eps: float, t: int, batch: int, seq: int, y=None):
        y = torch.empty_like(x) if y is None else y
        n = batch * seq
        _acheck(lib().tpattn_forward(self.ctx, batch, seq, self._t(x, (n, self.H), name="x"),
                                     self._t(norm_w, (self.H,), name="norm_w"),
                                     self._t(w_qkv, (self.W, self.H), name="w_qkv"),
                                     self._t(w_o, (self.H, self.nq * self.d), name="w_o"),
                                     self._t(b_o, (self.H,), name="b_o"), float(eps), int(t),
                                     self._t(y, (n, self.H), name="y")), self.ctx)
        self._uses(x, norm_w, w_qkv, w_o, b_o, y)
        # the library keeps these pointers (backward reads x; the updates write the parameters):
        # hold the tensors until the next forward so that a temporary argument is not freed
        self._fwd_tensors = (x, norm_w, w_qkv, w_o, b_o)
        self.params = (norm_w, w_qkv, w_o, b_o)
        self.tokens = n
        self._batch = batch
        return y

    def new_grads(self):
        f = dict(dtype=torch.float32, device=self.device)
        return {"norm_w": torch.empty(self.H, **f), "w_qkv": torch.empty(self.W, self.H, **f),
                "w_o": torch.empty(self.H, self.nq * self.d, **f), "b_o": torch.empty(self.H, **f)}

    def backward(self, dy, dx=None, grads=None):
        dx = torch.empty_like(dy) if dx is None else dx
        g = self.new_grads() if grads is None else grads
        f32 = torch.float32
        n = dy.shape[0] if self.tokens is None else self.tokens
        _acheck(lib().tpattn_backward(self.ctx, self._t(dy, (n, self.H), name="dy"),
                                      self._t(dx, (n, self.H), name="dx"),
                                      self._t(g["norm_w"], (self.H,), f32, "dnorm_w"),
                                      self._t(g["w_qkv"], (self.W, self.H), f32, "dw_qkv"),
                                      self._t(g["w_o"], (self.H, self.nq * self.d), f32, "dw_o"),
                                      self._t(g["b_o"], (self.H,), f32, "db_o")), self.ctx)
        self._uses(dy, dx, *g.values())
        # the updates read these gradients later: hold them until the next backward
        self._grads = g
        return dx, g

    def bind_master(self, m: dict | None):
        if m is None:
            _acheck(lib().tpattn_bind_master(self.ctx, None, None, None, None), self.ctx)
            self._masters = None
            return
        f32 = torch.float32
        _acheck(lib().tpattn_bind_master(self.ctx, self._t(m["norm_w"], (self.H,), f32, "norm_w"),
                                         self._t(m["w_qkv"], (self.W, self.H), f32, "w_qkv"),
                                         self._t(m["w_o"], (self.H, self.nq * self.d), f32, "w_o"),
                                         self._t(m["b_o"], (self.H,), f32, "b_o")), self.ctx)
        self._masters = m
        self._uses(*m.values())

    def sgd_step(self, lr: float):
        _acheck(lib().tpattn_sgd_step(self.ctx, float(lr)), self.ctx)

    def set_update_in_backward(self, enable: bool, lr: float = 0.0):
        """Have backward apply the SGD update itself (needs bound masters); sgd_step is then not called."""
        _acheck(lib().tpattn_set_update_in_backward(self.ctx, int(bool(enable)), float(lr)), self.ctx)

    def update_in_epilogue(self) -> bool:
        """Whether the last backward updated W_qkv and W_o inside their gradient GEMMs' epilogues."""
        return bool(lib().tpattn_update_in_epilogue(self.ctx))

    def _param_set(self, d: dict, what: str) -> AttnParamSet:
        f32 = torch.float32
        return AttnParamSet(self._t(d["norm_w"], (self.H,), f32, f"{what}.norm_w"),
                            self._t(d["w_qkv"], (self.W, self.H), f32, f"{what}.w_qkv"),
                            self._t(d["w_o"], (self.H, self.nq * self.d), f32, f"{what}.w_o"),
                            self._t(d["b_o"], (self.H,), f32, f"{what}.b_o"))

    def new_adam_state(self):
        """Zeroed first and second moments shaped like the parameters (fp32), bound to this context."""
        m = {k: torch.zeros_like(v) for k, v in self.new_grads().items()}
        v = {k: torch.zeros_like(t) for k, t in m.items()}
        self.bind_adam_state(m, v)
        return m, v

    def bind_adam_state(self, m: dict | None, v: dict | None):
        if m is None and v is None:
            _acheck(lib().tpattn_bind_adam_state(self.ctx, None, None), self.ctx)
            self._adam = None
            return
        ms, vs = self._param_set(m, "m"), self._param_set(v, "v")
        _acheck(lib().tpattn_bind_adam_state(self.ctx, ctypes.byref(ms), ctypes.byref(vs)), self.ctx)
        self._adam = (m, v)  # keep the tensors alive while bound
        self._uses(*m.values(), *v.values())

    def adamw_step(self, lr: float, step: int, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                   weight_decay: float = 0.1, max_grad_norm: float = 1.0, grad_norm=None):
        """One clipped AdamW update; returns the device float holding the global gradient norm."""
        if grad_norm is None:
            if getattr(self, "_gn", None) is None:
                with torch.cuda.stream(self.stream):
                    self._gn = torch.zeros(1, dtype=torch.float32, device=self.device)
            grad_norm = self._gn
        hp = AdamWParams(float(lr), float(beta1), float(beta2), float(eps), float(weight_decay),
                         float(max_grad_norm), int(step))
        _acheck(lib().tpattn_adamw_step(self.ctx, ctypes.byref(hp),
                                        self._t(grad_norm, (1,), torch.float32, "grad_norm")), self.ctx)
        self._uses(grad_norm)
        return grad_norm

    def set_qk(self, rotary: Rotary | None = None, q_norm_w=None, k_norm_w=None, eps: float = 1e-6, masters=None,
               moments=None):
        """Rotate queries and keys by position (row % seq) in later forwards and decodes, after the RMS norm of each
        head where bf16 weights are given (tpattn_set_qk).  masters: fp32 (q, k); moments: fp32 AdamW (m_q, m_k, v_q,
        v_k).  Returns the weights' gradient tensors {"q_norm_w", "k_norm_w"} that backward fills (empty without)."""
        d, i = self.d, self.device.index
        p = QkParams()
        p.rot = ctypes.pointer(rotary.spec) if rotary is not None else None
        p.q_norm_w, p.k_norm_w = _vec(q_norm_w, d, _BF, "q_norm_w", i), _vec(k_norm_w, d, _BF, "k_norm_w", i)
        norm = q_norm_w is not None
        grads = {k: torch.empty(d, dtype=_F32T, device=self.device) for k in ("q_norm_w", "k_norm_w")} if norm else {}
        if norm:
            p.dq_norm_w, p.dk_norm_w = grads["q_norm_w"].data_ptr(), grads["k_norm_w"].data_ptr()
        for names, given in ((("master_q", "master_k"), masters), (("m_q", "m_k", "v_q", "v_k"), moments)):
            for name, t in zip(names, given or ()):
                setattr(p, name, _vec(t, d, _F32T, name, i))
        p.eps = float(eps)
        nbytes = int(lib().tpattn_qk_workspace_bytes(ctypes.byref(self.cfg))) if norm else 0
        with torch.cuda.stream(self.stream):  # the rows and sums belong to the stream that its kernels run on
            ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device) if norm else None
        _acheck(lib().tpattn_set_qk(self.ctx, ctypes.byref(p), _ptr(ws), nbytes), self.ctx)
        self._uses(q_norm_w, k_norm_w, *(masters or ()), *(moments or ()), *grads.values())
        self._qk = (rotary, q_norm_w, k_norm_w, masters, moments, grads, ws)  # the context keeps their pointers
        return grads

    def clear_qk(self):
        """Later forwards and decodes neither rotate nor norm."""
        _acheck(lib().tpattn_set_qk(self.ctx, None, None, 0), self.ctx)
        self._qk = None

    def append_kv(self, kv: TPKV, block_table, new_lens=None):
        """Store the last forward's keys and values in a cache, the first new_lens[b] of each sequence (or all)."""
        batch = block_table.shape[0]
        if self.tokens is not None and (batch < 1 or self.tokens % batch or batch != self._batch):
            raise TPMLPError(ERR_SHAPE, "block_table needs a row for each sequence of the last forward")
        tp, ldt, pages = kv._table(block_table, batch)
        _acheck(lib().tpattn_append_kv(self.ctx, kv.ctx, _vec(new_lens, batch, _I32T, "new_lens", self.device.index),
                                       tp, ldt, pages), self.ctx)
        self._uses(block_table, new_lens)
        kv._used_by(self.stream)

    def decode(self, kv: TPKV, x, norm_w, w_qkv, w_o, b_o, eps: float, t: int, past_lens, block_table, window: int = 0,
               sinks: int = 0, y=None):
        """The sublayer for one new token per sequence, appended to the cache at position past_lens[b]
        (tpattn_decode); returns y [batch, H]."""
        n = x.shape[0]
        _int32(t=t, window=window, sinks=sinks)
        y = torch.empty_like(x) if y is None else y
        tp, ldt, pages = kv._table(block_table, n)
        _acheck(lib().tpattn_decode(self.ctx, kv.ctx, n, self._t(x, (n, self.H), name="x"),
                                    self._t(norm_w, (self.H,), name="norm_w"),
                                    self._t(w_qkv, (self.W, self.H), name="w_qkv"),
                                    self._t(w_o, (self.H, self.nq * self.d), name="w_o"),
                                    self._t(b_o, (self.H,), name="b_o"), float(eps), int(t),
                                    _vec(past_lens, n, _I32T, "past_lens", self.device.index), tp, ldt, pages, window,
                                    sinks, self._t(y, (n, self.H), name="y")), self.ctx)
        self._uses(x, norm_w, w_qkv, w_o, b_o, past_lens, block_table, y)
        kv._used_by(self.stream)
        return y

    def sync(self):
        _acheck(lib().tpattn_sync(self.ctx), self.ctx)

    def set_fused(self, enable: bool):
        """Fused attention kernels where the shape allows (the default), or always the unfused path."""
        _acheck(lib().tpattn_set_fused(self.ctx, int(bool(enable))), self.ctx)

    def fused_active(self) -> bool:
        """Whether the last forward ran the fused kernels."""
        return bool(lib().tpattn_fused_active(self.ctx))

    def set_timing(self, enable: bool):
        _acheck(lib().tpattn_set_timing(self.ctx, int(bool(enable))), self.ctx)

    def read_kernel_times(self) -> dict:
        n = lib().tpattn_num_kernel_ids()
        ms = (ctypes.c_float * n)()
        cnt = (ctypes.c_int64 * n)()
        lib().tpattn_read_kernel_times(self.ctx, ms, cnt, n)
        return {lib().tpattn_kernel_name(i).decode(): (float(ms[i]), int(cnt[i])) for i in range(n) if cnt[i]}

    def launch_count(self) -> int:
        return int(lib().tpattn_launch_count(self.ctx))


class Rotary:
    """Position rotation of query and key heads (tpattn_rotary): the first ``rot_dim`` values of a head, as
    pairs (j, j + rot_dim/2), or (2j, 2j + 1) when ``interleaved``; pair j turns by ``inv_freq[j]`` radians per
    position, ``theta ** (-2 j / rot_dim)`` unless given.  Holds no device memory."""

    def __init__(self, rot_dim: int, theta: float = 10000.0, inv_freq=None, interleaved: bool = False):
        freq = [theta ** (-2.0 * j / rot_dim) for j in range(rot_dim // 2)] if inv_freq is None else list(inv_freq)
        if len(freq) != rot_dim // 2:
            raise TPMLPError(ERR_ARG, "inv_freq needs rot_dim / 2 values")
        self.spec = RotarySpec()
        _check(lib().tpattn_rotary_init(ctypes.byref(self.spec), rot_dim, int(bool(interleaved)),
                                        (ctypes.c_double * max(len(freq), 1))(*freq)))
        self.ref = ctypes.byref(self.spec)
        self.rot_dim, self.interleaved = rot_dim, bool(interleaved)


_BF, _F32T, _I32T = torch.bfloat16, torch.float32, torch.int32
# the raw handle of torch's current stream on a device, without a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(device, index: int):
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(device).cuda_stream


def _record(stream, *tensors):
    """Their memory is handed out again only when `stream` is past what it holds now (nothing to do for its own)."""
    for t in tensors:
        if t is not None and t.is_cuda:
            t.record_stream(stream)


def _bad(t, name: str, want: str):
    return TPMLPError(ERR_ARG, f"{name}: need {want}, got {t.dtype} {tuple(t.shape)} with strides {t.stride()} on "
                               f"{t.device}")


_I31 = 1 << 31


def _int32(**values):
    """Refuses whole numbers that ctypes would mask to 32 bits."""
    for name, v in values.items():
        if not -_I31 <= v < _I31:
            raise TPMLPError(ERR_ARG, f"{name} {v} does not fit 32 bits")


def _rows(t, width: int, dtype, name: str, index: int, rows: int = -1):
    """Pointer, row count and row stride of a 2-D tensor on CUDA device `index` whose rows hold at least `width`
    contiguous values."""
    shape = t.shape
    if len(shape) == 2 and t.dtype is dtype and t.get_device() == index and shape[1] >= width:
        n = shape[0]
        ld, inner = t.stride()
        if (rows < 0 or n == rows) and (inner == 1 or shape[1] == 1):
            return t.data_ptr(), n, ld if n > 1 else width
    raise _bad(t, name, f"{'' if rows < 0 else f'{rows} '}{dtype} rows of at least {width} contiguous values on "
                        f"cuda:{index}")


def _vec(t, n: int, dtype, name: str, index: int):
    if t is None:
        return None
    shape = t.shape
    if (len(shape) != 1 or t.dtype is not dtype or shape[0] != n or t.get_device() != index
            or (n > 1 and t.stride(0) != 1)):
        raise _bad(t, name, f"contiguous {dtype} ({n},) on cuda:{index}")
    return t.data_ptr()


def _on_device(index: int, fn, *args):
    """A call without a context, on device `index`."""
    if torch.cuda.current_device() == index:
        status = fn(*args)
    else:
        with torch.cuda.device(index):
            status = fn(*args)
    if status:
        _check(status)


def _qk_desc(n, dtype, index, n_heads, n_kv_heads, head_dim, positions, seq, q_norm_w, k_norm_w, eps) -> QkDesc:
    dt = BF16 if dtype is _BF else F32 if dtype is _F32T else None
    if dt is None:
        raise TPMLPError(ERR_UNSUPPORTED, "rows must be float32 or bfloat16")
    return QkDesc(n, n_heads, n_kv_heads, head_dim, dt, _vec(positions, n, _I32T, "positions", index), seq,
                  _vec(q_norm_w, head_dim, dtype, "q_norm_w", index),
                  _vec(k_norm_w, head_dim, dtype, "k_norm_w", index), eps, 0)


def _cuda_index(t, name: str) -> int:
    index = t.get_device()
    if index < 0:
        raise TPMLPError(ERR_ARG, f"{name} must be a CUDA tensor")
    return index


def qk_norm_rope(x, n_heads: int, n_kv_heads: int, head_dim: int, rotary: Rotary | None = None, positions=None,
                 seq: int = 0, q_norm_w=None, k_norm_w=None, eps: float = 1e-6, out=None, stream=None):
    """RMS norm (where a weight is given) and position rotation of the query and key heads at the start of each
    row of x (tpattn_qk_rope_forward); out may be x.  Positions: int32 per row, or row % seq (seq 0: the row).
    Runs on `stream`, torch's current stream where it is None."""
    if stream is not None:  # what is allocated here belongs to that stream too
        _record(stream, x, positions, q_norm_w, k_norm_w, out)
        with torch.cuda.stream(stream):
            return qk_norm_rope(x, n_heads, n_kv_heads, head_dim, rotary, positions, seq, q_norm_w, k_norm_w, eps, out)
    width, dtype, index = (n_heads + n_kv_heads) * head_dim, x.dtype, _cuda_index(x, "x")
    xp, n, ldx = _rows(x, width, dtype, "x", index)
    if out is None:
        out = x.new_empty((n, width))
    op, _, ldo = _rows(out, width, dtype, "out", index, n)
    d = _qk_desc(n, dtype, index, n_heads, n_kv_heads, head_dim, positions, seq, q_norm_w, k_norm_w, eps)
    _on_device(index, lib().tpattn_qk_rope_forward, d, rotary.spec if rotary is not None else None, xp, ldx, op, ldo,
               _stream_of(x.device, index))
    return out


def qk_norm_rope_backward(dout, x, n_heads: int, n_kv_heads: int, head_dim: int, rotary: Rotary | None = None,
                          positions=None, seq: int = 0, q_norm_w=None, k_norm_w=None, eps: float = 1e-6, dx=None,
                          dq_norm_w=None, dk_norm_w=None, workspace=None, stream=None):
    """Backward of qk_norm_rope: (dx, dq_norm_w, dk_norm_w), the weights' gradients in float32 (None without the
    weight).  x: the forward's input (only read with norm weights, else it may be None); dx may be dout."""
    if stream is not None:  # what is allocated here belongs to that stream too
        _record(stream, dout, x, positions, q_norm_w, k_norm_w, dx, dq_norm_w, dk_norm_w, workspace)
        with torch.cuda.stream(stream):
            return qk_norm_rope_backward(dout, x, n_heads, n_kv_heads, head_dim, rotary, positions, seq, q_norm_w,
                                         k_norm_w, eps, dx, dq_norm_w, dk_norm_w, workspace)
    width, dtype, index = (n_heads + n_kv_heads) * head_dim, dout.dtype, _cuda_index(dout, "dout")
    norm = q_norm_w is not None or k_norm_w is not None
    gp, n, ldg = _rows(dout, width, dtype, "dout", index)
    xp, _, ldx = _rows(x, width, dtype, "x", index, n) if norm else (None, n, 0)
    if dx is None:
        dx = dout.new_empty((n, width))
    dp, _, ldd = _rows(dx, width, dtype, "dx", index, n)
    wp, wbytes = None, 0
    if norm:
        need = lib().tpattn_qk_rope_workspace_bytes(head_dim)
        if workspace is not None:
            if workspace.get_device() != index or not workspace.is_contiguous():
                raise _bad(workspace, "workspace", f"a contiguous tensor on cuda:{index}")
            wp, wbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        else:  # separate tensors: views of one cost more than allocating each
            workspace = torch.empty(need // 4, dtype=_F32T, device=dout.device)
            wp, wbytes = workspace.data_ptr(), need
        if q_norm_w is not None and dq_norm_w is None:
            dq_norm_w = torch.empty(head_dim, dtype=_F32T, device=dout.device)
        if k_norm_w is not None and dk_norm_w is None:
            dk_norm_w = torch.empty(head_dim, dtype=_F32T, device=dout.device)
    d = _qk_desc(n, dtype, index, n_heads, n_kv_heads, head_dim, positions, seq, q_norm_w, k_norm_w, eps)
    _on_device(index, lib().tpattn_qk_rope_backward, d, rotary.spec if rotary is not None else None, xp, ldx, gp, ldg, dp,
               ldd, _vec(dq_norm_w, head_dim, _F32T, "dq_norm_w", index),
               _vec(dk_norm_w, head_dim, _F32T, "dk_norm_w", index), wp, wbytes, _stream_of(dout.device, index))
    return dx, dq_norm_w, dk_norm_w


class TPKV:
    """A paged key/value cache (tpkv_*): append new tokens, attend with one token per sequence.

    ``k_cache`` and ``v_cache``: [pages, n_kv_heads, page_size, head_dim], bfloat16 or float8_e4m3fn, with the same
    strides, the last one 1 (a [pages, page_size, n_kv_heads, head_dim] tensor is passed transposed).  E4M3 codes
    stand for code * inv_scale of their head.  The cache stays the caller's; the context's scratch is a torch
    tensor.  Calls run on ``stream``, or on torch's current stream at each call where it is None; calls that may
    overlap on the GPU need a TPKV each."""

    def __init__(self, k_cache, v_cache, n_heads: int, max_batch: int = 1024, k_inv_scale=None, v_inv_scale=None,
                 stream=None):
        if k_cache.dim() != 4 or k_cache.get_device() < 0:
            raise TPMLPError(ERR_ARG, "k_cache must be a CUDA tensor [pages, n_kv_heads, page_size, head_dim]")
        kinds = {torch.bfloat16: 0, torch.float8_e4m3fn: 1}
        if k_cache.dtype not in kinds:
            raise TPMLPError(ERR_UNSUPPORTED, "the cache must be bfloat16 or float8_e4m3fn")
        if (v_cache.dtype != k_cache.dtype or v_cache.shape != k_cache.shape or v_cache.device != k_cache.device
                or v_cache.stride() != k_cache.stride() or k_cache.stride(3) != 1):
            raise TPMLPError(ERR_ARG, "k_cache and v_cache must agree in type, shape, device and strides, the last 1")
        self.device = dev = k_cache.device
        pages, nkv, page, d = k_cache.shape
        _int32(n_heads=n_heads, max_batch=max_batch)
        self.cfg = KvConfig(pages, page, max_batch, n_heads, nkv, d, kinds[k_cache.dtype], 0)
        self.nq, self.nkv, self.d, self.page_size = n_heads, nkv, d, page
        self.k_cache, self.v_cache = k_cache, v_cache
        self._scales = (k_inv_scale, v_inv_scale)
        self._norm = (None, None)
        self.index = k_cache.get_device()
        self._fixed = stream
        if stream is not None:  # the scratch belongs to the stream that its first use runs on
            with torch.cuda.stream(stream):
                self._create(pages, page, d)
        else:
            self._create(pages, page, d)

    def _create(self, pages: int, page: int, d: int):
        dev, (k_cache, v_cache) = self.device, (self.k_cache, self.v_cache)
        self._stream = _stream_of(dev, self.index)
        ctx = ctypes.c_void_p()
        with torch.cuda.device(dev):
            self._ck(lib().tpkv_create(ctypes.byref(self.cfg), self._stream, ctypes.byref(ctx)))
            self.ctx = ctx
            nbytes = int(lib().tpkv_workspace_bytes(ctypes.byref(self.cfg)))
            self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        self._ck(lib().tpkv_bind_workspace(ctx, self.workspace.data_ptr(), nbytes))
        if self._fixed is not None:
            _record(self._fixed, *self._held())
        f32 = torch.float32
        self._ck(lib().tpkv_bind_cache(ctx, k_cache.data_ptr(), v_cache.data_ptr(), *k_cache.stride()[:3],
                                       _vec(self._scales[0], self.nkv, f32, "k_inv_scale", self.index),
                                       _vec(self._scales[1], self.nkv, f32, "v_inv_scale", self.index)))

    def _ck(self, status: int):
        if status != OK:
            ctx = getattr(self, "ctx", None)
            msg = lib().tpkv_last_error(ctx).decode(errors="replace")
            raise TPMLPError(status, msg or lib().tpmlp_status_string(status).decode())

    def close(self):
        if getattr(self, "ctx", None):
            lib().tpkv_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_stream(self, stream):
        """Run later calls on `stream` (None: torch's current stream at each call)."""
        self._fixed = stream

    def _elsewhere(self) -> bool:
        """Whether torch's current stream is not the fixed one."""
        return self._fixed is not None and _stream_of(self.device, self.index) != self._fixed.cuda_stream

    def _held(self):
        """What the context keeps by pointer."""
        return self.workspace, self.k_cache, self.v_cache, *self._scales, *self._norm

    def _used_by(self, stream):
        """A call of this context ran on `stream`, which need not be the context's own."""
        if stream.cuda_stream != self._stream:
            _record(stream, *self._held())

    def _enter(self):
        s = _stream_of(self.device, self.index)
        if s != self._stream:
            self._ck(lib().tpkv_set_stream(self.ctx, s))
            self._stream = s
            _record(torch.cuda.current_stream(self.device), *self._held())

    def set_rotary(self, rotary: Rotary | None, q_norm_w=None, k_norm_w=None, eps: float = 1e-6):
        """What append does to queries and keys: norm where a bf16 weight is given, then the rotation."""
        self._ck(lib().tpkv_set_rotary(self.ctx, rotary.ref if rotary is not None else None,
                                       _vec(q_norm_w, self.d, _BF, "q_norm_w", self.index),
                                       _vec(k_norm_w, self.d, _BF, "k_norm_w", self.index), float(eps)))
        self._norm = (q_norm_w, k_norm_w)  # the context keeps their pointers
        self._stream = None  # whatever stream is next enters anew, with them

    def _table(self, t, batch: int):
        shape = t.shape
        if (len(shape) != 2 or t.dtype is not _I32T or shape[0] != batch or t.get_device() != self.index
                or (shape[1] > 1 and t.stride(1) != 1) or (batch > 1 and t.stride(0) < shape[1])):
            raise _bad(t, "block_table", f"int32 [{batch}, pages] on cuda:{self.index}, a row of its own for each sequence")
        return t.data_ptr(), t.stride(0) if batch > 1 else shape[1], shape[1]

    def append(self, qkv, past_lens, block_table, cu_rows=None, new_lens=None, q_out=None, transform: bool = True,
               with_queries: bool = True):
        """Store the keys and values of packed rows [Q | K | V] behind each sequence's ``past_lens`` tokens and
        return the normed and rotated queries [rows, n_heads * d] (None without ``with_queries``); see tpkv_append.
        Rows that are no sequence's leave ``q_out`` as it was (undefined where it is made here)."""
        if self._elsewhere():  # what is allocated here belongs to that stream too
            _record(self._fixed, qkv, past_lens, block_table, cu_rows, new_lens, q_out)
            with torch.cuda.stream(self._fixed):
                return self.append(qkv, past_lens, block_table, cu_rows, new_lens, q_out, transform, with_queries)
        index, batch, width = self.index, past_lens.shape[0], self.nq * self.d
        xp, n, ldx = _rows(qkv, width + 2 * self.nkv * self.d, _BF, "qkv", index)
        if q_out is None and with_queries:
            q_out = qkv.new_empty((n, width))
        op, _, ldo = _rows(q_out, width, _BF, "q_out", index, n) if q_out is not None else (None, n, 0)
        tp, ldt, pages = self._table(block_table, batch)
        self._enter()
        status = lib().tpkv_append(self.ctx, n, batch, xp, ldx, _vec(cu_rows, batch + 1, _I32T, "cu_rows", index),
                                   _vec(new_lens, batch, _I32T, "new_lens", index),
                                   _vec(past_lens, batch, _I32T, "past_lens", index), tp, ldt, pages,
                                   1 if transform else 0, op, ldo)
        if status:
            self._ck(status)
        return q_out

    def decode(self, q, lens, block_table, scale: float | None = None, window: int = 0, sinks: int = 0, out=None,
               lse=None, return_lse: bool = False, len_add: int = 0):
        """Attention of one token per sequence over its first ``lens + len_add`` cached tokens; with a window, over
        its last ``window`` tokens and first ``sinks``.  scale: 1 / sqrt(head_dim) unless given.  Returns out
        [batch, n_heads * d], with ``return_lse`` or ``lse`` (out, lse float32 [batch, n_heads]); see tpkv_decode."""
        if self._elsewhere():
            _record(self._fixed, q, lens, block_table, out, lse)
            with torch.cuda.stream(self._fixed):
                return self.decode(q, lens, block_table, scale, window, sinks, out, lse, return_lse, len_add)
        index, width = self.index, self.nq * self.d
        if not (-_I31 <= window < _I31 and -_I31 <= sinks < _I31 and -_I31 <= len_add < _I31):
            _int32(window=window, sinks=sinks, len_add=len_add)
        qp, batch, ldq = _rows(q, width, _BF, "q", index)
        if out is None:
            out = q.new_empty((batch, width))
        op, _, ldo = _rows(out, width, _BF, "out", index, batch)
        if lse is None:
            if return_lse:
                lse = torch.empty((batch, self.nq), dtype=_F32T, device=self.device)
        elif (lse.dtype is not _F32T or tuple(lse.shape) != (batch, self.nq) or lse.get_device() != index
                or not lse.is_contiguous()):
            raise _bad(lse, "lse", f"contiguous float32 {(batch, self.nq)} on cuda:{index}")
        tp, ldt, pages = self._table(block_table, batch)
        self._enter()
        status = lib().tpkv_decode(self.ctx, batch, qp, ldq, _vec(lens, batch, _I32T, "lens", index), len_add, tp,
                                   ldt, pages, self.d ** -0.5 if scale is None else scale, window, sinks, op, ldo,
                                   lse.data_ptr() if lse is not None else None)
        if status:
            self._ck(status)
        return out if lse is None else (out, lse)

    def sync(self):
        """Wait for the stream of the last call; raises where a page or length lay outside the cache."""
        self._ck(lib().tpkv_sync(self.ctx))

    def launch_count(self) -> int:
        return int(lib().tpkv_launch_count(self.ctx))
