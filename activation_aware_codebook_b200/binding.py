"""Thin Python binding of libaaac.so (include/aaac.h).

Argument marshalling only: torch supplies device memory and the current
stream, every step of the fit runs in the library's CUDA kernels.  There is no
CPU fallback: without the built library or a CUDA device every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import os
from typing import Optional, Union

import torch

INT4 = 0
NVFP4 = 1
NVFP4_GS = 2  # NVFP4 with a per-tensor fp32 scale
FREEZE_T0 = 1
FREEZE_T1 = 2
SINGLE_CODEBOOK = 4
CONCURRENT = 8  # grids sized by the layer's weights, for layers fitted side by side
IMPORTANCE_ACCUMULATE = 1
IMPORTANCE_EXACT = 2

STATUS = {0: "AAAC_OK", 1: "AAAC_ERR_INVALID_ARG", 2: "AAAC_ERR_SHAPE", 3: "AAAC_ERR_ALIGN",
          4: "AAAC_ERR_UNSUPPORTED", 5: "AAAC_ERR_CUDA", 6: "AAAC_ERR_WORKSPACE",
          7: "AAAC_ERR_TIMEOUT", 8: "AAAC_ERR_COLLECTIVE"}

# AAAC_CHECKED=1 selects the debugging build with device-side index checks
# (built by `python -m activation_aware_codebook_b200.csrc.build --checks`).
LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)),
                        "libaaac_checked.so" if os.environ.get("AAAC_CHECKED") == "1"
                        else "libaaac.so")

EXPORTS = ("aaac_workspace_size", "aaac_importance", "aaac_init_codebooks", "aaac_fit_layer",
           "aaac_pack", "aaac_last_error", "aaac_version", "aaac_kernel_launches",
           "aaac_fit_layer_fixed_scratch", "aaac_dequant", "aaac_linear",
           "aaac_device_timeouts", "aaac_awq_prescale", "aaac_awq_workspace_size",
           "aaac_awq_fit", "aaac_init_codebooks_sharded", "aaac_fit_layer_sharded",
           "aaac_pack_sharded", "aaac_linear_workspace_size", "aaac_linear_ws",
           "aaac_fit_launch_plan", "aaac_linear_launch_plan", "aaac_inject_fault",
           "aaac_device_checks",
           "aaac_checked_build", "aaac_mx_scale_bytes", "aaac_mx_quantize", "aaac_mx_dequant",
           "aaac_mx_linear", "aaac_mx_workspace_size", "aaac_mx_linear_ws",
           "aaac_mx_launch_plan")


# reduction callback of the row-sharded calls: (user, buf, count, op, stream) -> 0 | error
REDUCE_FN = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                             ctypes.c_int, ctypes.c_void_p)
REDUCE_SUM_I64, REDUCE_MAX_I64, REDUCE_SUM_I32, REDUCE_MAX_I32 = 0, 1, 2, 3


class AaacError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class CConfig(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("g", ctypes.c_int32), ("S", ctypes.c_int32),
                ("iters", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("global_scale", ctypes.c_void_p)]


class CStats(ctypes.Structure):
    _fields_ = [("near_ties", ctypes.c_int64), ("groups_t1", ctypes.c_int64),
                ("empty_cells", ctypes.c_int64), ("dead_groups", ctypes.c_int64),
                ("exact_groups", ctypes.c_int64), ("L", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


STATS_BYTES = ctypes.sizeof(CStats)


@dataclasses.dataclass
class Config:
    fmt: int = INT4
    g: int = 128
    S: int = 128
    iters: int = 20
    flags: int = 0
    # NVFP4_GS: device fp32 [1] holding the per-tensor scale (init_codebooks
    # allocates it on the weights' device when it is None)
    global_scale: Optional[torch.Tensor] = None

    def c(self) -> CConfig:
        gs = self.global_scale.data_ptr() if self.global_scale is not None else None
        return CConfig(self.fmt, self.g, self.S, self.iters, self.flags, gs)

    def ensure_global_scale(self, device) -> None:
        if self.fmt == NVFP4_GS and self.global_scale is None:
            self.global_scale = torch.zeros(1, dtype=torch.float32, device=device)

    @property
    def n(self) -> int:
        return 16 if self.fmt == INT4 else 15


_lib = None


def load(path: str = LIB_PATH):
    """Load libaaac.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libaaac.so not built ({path}); run "
                           "python -m activation_aware_codebook_b200.csrc.build")
    L = ctypes.CDLL(path)
    P, i64, sz, u32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_uint32
    L.aaac_workspace_size.restype = sz
    L.aaac_workspace_size.argtypes = [P, i64, i64, i64]
    L.aaac_importance.restype = ctypes.c_int
    L.aaac_importance.argtypes = [P, i64, i64, i64, u32, P, P, sz, P]
    L.aaac_init_codebooks.restype = ctypes.c_int
    L.aaac_init_codebooks.argtypes = [P, i64, i64, P, P, P, P, sz, P]
    L.aaac_fit_layer.restype = ctypes.c_int
    L.aaac_fit_layer.argtypes = [P, i64, i64, P, P, P, P, P, P, P, sz, P]
    L.aaac_pack.restype = ctypes.c_int
    L.aaac_pack.argtypes = [P, i64, i64, P, P, P, P, P, P, P, P, P, P, sz, P]
    L.aaac_last_error.restype = ctypes.c_char_p
    L.aaac_last_error.argtypes = []
    L.aaac_version.restype = ctypes.c_char_p
    L.aaac_version.argtypes = []
    L.aaac_fit_layer_fixed_scratch.restype = ctypes.c_int
    L.aaac_fit_layer_fixed_scratch.argtypes = [P, i64, i64, P, P, P, P, P, P, P]
    L.aaac_dequant.restype = ctypes.c_int
    L.aaac_dequant.argtypes = [P, P, P, P, i64, i64, P, P, P]
    L.aaac_linear.restype = ctypes.c_int
    L.aaac_linear.argtypes = [P, i64, i64, P, P, P, P, i64, i64, P, P, P]
    L.aaac_device_timeouts.restype = ctypes.c_int
    L.aaac_device_timeouts.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
    L.aaac_kernel_launches.restype = ctypes.c_uint64
    L.aaac_kernel_launches.argtypes = []
    L.aaac_inject_fault.restype = ctypes.c_int
    L.aaac_inject_fault.argtypes = [ctypes.c_char_p]
    L.aaac_device_checks.restype = ctypes.c_int
    L.aaac_device_checks.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
    L.aaac_checked_build.restype = ctypes.c_int
    L.aaac_checked_build.argtypes = []
    L.aaac_fit_launch_plan.restype = ctypes.c_int
    L.aaac_fit_launch_plan.argtypes = [P, i64, i64, i64, ctypes.POINTER(ctypes.c_int32)]
    L.aaac_linear_launch_plan.restype = ctypes.c_int
    L.aaac_linear_launch_plan.argtypes = [P, i64, i64, i64, ctypes.POINTER(ctypes.c_int32)]
    L.aaac_awq_prescale.restype = ctypes.c_int
    L.aaac_awq_prescale.argtypes = [P, i64, i64, P, i64, ctypes.c_int, P, P, P, P]
    L.aaac_awq_workspace_size.restype = sz
    L.aaac_awq_workspace_size.argtypes = [P, i64, i64]
    L.aaac_awq_fit.restype = ctypes.c_int
    L.aaac_awq_fit.argtypes = [P, i64, i64, P, i64, P, P, ctypes.c_int, P, P, P, P, P, P, P, P,
                               P, sz, P]
    L.aaac_linear_workspace_size.restype = sz
    L.aaac_linear_workspace_size.argtypes = [P, i64, i64, i64]
    L.aaac_linear_ws.restype = ctypes.c_int
    L.aaac_linear_ws.argtypes = [P, i64, i64, P, P, P, P, i64, i64, P, P, P, sz, P]
    R = REDUCE_FN
    L.aaac_init_codebooks_sharded.restype = ctypes.c_int
    L.aaac_init_codebooks_sharded.argtypes = [P, i64, i64, i64, P, P, P, R, P, P, sz, P]
    L.aaac_fit_layer_sharded.restype = ctypes.c_int
    L.aaac_fit_layer_sharded.argtypes = [P, i64, i64, i64, P, P, P, P, P, P, R, P, P, sz, P]
    L.aaac_pack_sharded.restype = ctypes.c_int
    L.aaac_pack_sharded.argtypes = [P, i64, i64, i64, P, P, P, P, P, P, P, P, P, R, P, P, sz, P]
    i32 = ctypes.c_int32
    L.aaac_mx_scale_bytes.restype = sz
    L.aaac_mx_scale_bytes.argtypes = [i32, i64, i64, i32]
    L.aaac_mx_quantize.restype = ctypes.c_int
    L.aaac_mx_quantize.argtypes = [P, P, P]
    L.aaac_mx_dequant.restype = ctypes.c_int
    L.aaac_mx_dequant.argtypes = [P, P, i32, i64, P]
    L.aaac_mx_linear.restype = ctypes.c_int
    L.aaac_mx_linear.argtypes = [P, P, P, i32, i64, P]
    L.aaac_mx_workspace_size.restype = sz
    L.aaac_mx_workspace_size.argtypes = [i32, i64, i64, i32, u32]
    L.aaac_mx_linear_ws.restype = ctypes.c_int
    L.aaac_mx_linear_ws.argtypes = [P, i64, P, P, P, i32, i64, P, sz, P]
    L.aaac_mx_launch_plan.restype = ctypes.c_int
    L.aaac_mx_launch_plan.argtypes = [i32, i64, i64, i64, ctypes.POINTER(i32)]
    _lib = L
    return L


def device_checks() -> int:
    """The first failed device-side check of a checked build (0: none)."""
    v = ctypes.c_uint32(0)
    _check(load().aaac_device_checks(ctypes.byref(v)))
    return int(v.value)


def inject_fault(kind: Optional[str]) -> None:
    """Test hook: the next call that would launch work fails on the host
    ("alloc", "launch" or "sync"; None disarms), or, in checked builds, the
    products' device waits run out ("wait"); see aaac_inject_fault."""
    _check(load().aaac_inject_fault(None if kind is None else kind.encode()))


def kernel_launches() -> int:
    """Kernels the library has launched in this process so far."""
    return int(load().aaac_kernel_launches())


def _check(status: int):
    if status != 0:
        raise AaacError(status, load().aaac_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libaaac takes device tensors only")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need_cuda():
    if not torch.cuda.is_available():
        raise RuntimeError("libaaac needs a CUDA device; there is no CPU path")


def workspace_size(cfg: Optional[Config], N: int = 0, K: int = 0, T: int = 0) -> int:
    c = cfg.c() if cfg is not None else None
    return int(load().aaac_workspace_size(ctypes.byref(c) if c is not None else None, N, K, T))


LINEAR_PATHS = {0: "gemv", 1: "cluster", 2: "fused"}


def linear_launch_plan(cfg: Config, M: int, N: int, K: int) -> dict:
    """Host-only: the kernel aaac_linear runs and the cluster kernel's plan."""
    out = (ctypes.c_int32 * 8)()
    _check(load().aaac_linear_launch_plan(ctypes.byref(cfg.c()), M, N, K, out))
    keys = ("path", "cluster", "kblocks", "scale_stride", "choice_stride", "smem16", "smem32",
            "smem_limit")
    d = dict(zip(keys, list(out)))
    d["path"] = LINEAR_PATHS[d["path"]]
    return d


def fit_launch_plan(cfg: Config, N: int, K: int, N_total: Optional[int] = None) -> dict:
    """The fit/pack passes' launch plan for these sizes (host-only query)."""
    out = (ctypes.c_int32 * 5)()
    _check(load().aaac_fit_launch_plan(ctypes.byref(cfg.c()), N, K,
                                       N if N_total is None else N_total, out))
    return dict(blocks=out[0], strips=out[1], items_per_strip=out[2], item_rows=out[3],
                max_items=out[4])


def workspace(cfg: Optional[Config], N: int = 0, K: int = 0, T: int = 0,
              device="cuda") -> torch.Tensor:
    return torch.empty(workspace_size(cfg, N, K, T), dtype=torch.uint8, device=device)


def _bits16(t: torch.Tensor) -> torch.Tensor:
    assert t.dtype in (torch.bfloat16, torch.int16, torch.uint16), t.dtype
    return t.contiguous()


def importance(X: torch.Tensor, I: Optional[torch.Tensor] = None, accumulate: bool = False,
               exact: bool = False, ws: Optional[torch.Tensor] = None, stream=None,
               ncols: Optional[int] = None) -> torch.Tensor:
    """I_k = sum_t X[t,k]^2 (fp32, exact sum rounded once).  X: [T, ldx] bf16."""
    _need_cuda()
    T, ldx = X.shape
    K = ldx if ncols is None else ncols
    if X.stride(1) != 1:
        raise ValueError("X must be row-major")
    ldx = X.stride(0)
    if I is None:
        I = torch.zeros(K, dtype=torch.float32, device=X.device)
    if ws is None:
        ws = workspace(None, 0, K, T, X.device)
    flags = (IMPORTANCE_ACCUMULATE if accumulate else 0) | (IMPORTANCE_EXACT if exact else 0)
    _check(load().aaac_importance(_ptr(X), T, K, ldx, flags, _ptr(I), _ptr(ws), ws.numel(),
                                  _stream(stream)))
    return I


def init_codebooks(W: torch.Tensor, cfg: Config, ws: Optional[torch.Tensor] = None,
                   scales: Optional[torch.Tensor] = None, T: Optional[torch.Tensor] = None,
                   stream=None):
    """Absmax scales and quantile codebooks.  Returns (scales, T[2,16])."""
    _need_cuda()
    W = _bits16(W)
    N, K = W.shape
    sdt = torch.int16 if cfg.fmt == INT4 else torch.uint8
    if scales is None:
        scales = torch.empty(N, K // cfg.g, dtype=sdt, device=W.device)
    if T is None:
        T = torch.empty(2, 16, dtype=torch.float32, device=W.device)
    if ws is None:
        ws = workspace(cfg, N, K, 0, W.device)
    cfg.ensure_global_scale(W.device)
    c = cfg.c()
    _check(load().aaac_init_codebooks(_ptr(W), N, K, ctypes.byref(c), _ptr(scales), _ptr(T),
                                      _ptr(ws), ws.numel(), _stream(stream)))
    return scales, T


def fit_layer(W: torch.Tensor, I: torch.Tensor, scales: torch.Tensor, T: torch.Tensor,
              cfg: Config, ws: Optional[torch.Tensor] = None,
              err_hist: Optional[torch.Tensor] = None, stats: Optional[torch.Tensor] = None,
              stream=None):
    """cfg.iters assign/refine rounds; T [2,16] fp32 is updated in place.
    Returns (T, err_hist[iters] fp64, stats bytes)."""
    _need_cuda()
    W = _bits16(W)
    N, K = W.shape
    if err_hist is None:
        err_hist = torch.zeros(max(cfg.iters, 1), dtype=torch.float64, device=W.device)
    if stats is None:
        stats = torch.zeros(STATS_BYTES, dtype=torch.uint8, device=W.device)
    if ws is None:
        ws = workspace(cfg, N, K, 0, W.device)
    c = cfg.c()
    _check(load().aaac_fit_layer(_ptr(W), N, K, _ptr(I), _ptr(scales), ctypes.byref(c), _ptr(T),
                                 _ptr(err_hist), _ptr(stats), _ptr(ws), ws.numel(),
                                 _stream(stream)))
    return T, err_hist, stats


def fit_layer_fixed_scratch(W: torch.Tensor, I: torch.Tensor, scales: torch.Tensor,
                            T: torch.Tensor, cfg: Config, err_hist: Optional[torch.Tensor] = None,
                            stats: Optional[torch.Tensor] = None, stream=None):
    """fit_layer for callers that cannot allocate: the library's own fixed
    scratch replaces the workspace (see aaac_fit_layer_fixed_scratch)."""
    _need_cuda()
    W = _bits16(W)
    N, K = W.shape
    if err_hist is None:
        err_hist = torch.zeros(max(cfg.iters, 1), dtype=torch.float64, device=W.device)
    if stats is None:
        stats = torch.zeros(STATS_BYTES, dtype=torch.uint8, device=W.device)
    c = cfg.c()
    _check(load().aaac_fit_layer_fixed_scratch(_ptr(W), N, K, _ptr(I), _ptr(scales),
                                               ctypes.byref(c), _ptr(T), _ptr(err_hist),
                                               _ptr(stats), _stream(stream)))
    return T, err_hist, stats


def decode_stats(stats: torch.Tensor) -> dict:
    raw = bytes(stats.cpu().numpy().tobytes())
    s = CStats.from_buffer_copy(raw)
    return {f: getattr(s, f) for f, _ in CStats._fields_ if f != "reserved"}


def pack(W: torch.Tensor, I: torch.Tensor, scales: torch.Tensor, T: torch.Tensor, cfg: Config,
         ws: Optional[torch.Tensor] = None, out: Optional[dict] = None, stream=None) -> dict:
    """bf16 tables, final assign, 4-bit codes, sign-tagged scales, choice bits."""
    _need_cuda()
    W = _bits16(W)
    N, K = W.shape
    dev = W.device
    if out is None:
        nb = (K // cfg.S + 7) // 8
        out = dict(T_bf16=torch.zeros(2, 16, dtype=torch.int16, device=dev),
                   codes=torch.empty(N, K // 2, dtype=torch.uint8, device=dev),
                   scales_tagged=torch.empty_like(scales),
                   choice_bits=(torch.empty(N, nb, dtype=torch.uint8, device=dev)
                                if cfg.S != cfg.g else None),
                   err_final=torch.zeros(1, dtype=torch.float64, device=dev))
    if ws is None:
        ws = workspace(cfg, N, K, 0, dev)
    c = cfg.c()
    _check(load().aaac_pack(_ptr(W), N, K, _ptr(I), _ptr(scales), ctypes.byref(c), _ptr(T),
                            _ptr(out["T_bf16"]), _ptr(out["codes"]), _ptr(out["scales_tagged"]),
                            _ptr(out["choice_bits"]), _ptr(out["err_final"]), _ptr(ws),
                            ws.numel(), _stream(stream)))
    return out


def device_timeouts() -> int:
    """1 when a bounded device wait of the library's kernels has run out since
    the library was loaded on the current device, else 0."""
    v = ctypes.c_uint32(0)
    _check(load().aaac_device_timeouts(ctypes.byref(v)))
    return int(v.value)


def dequant(packed: dict, cfg: Config, N: int, K: int, out: Optional[torch.Tensor] = None,
            stream=None) -> torch.Tensor:
    """bf16 weights of a packed layer (the dict pack() returns), [N, K] bf16 bits (int16)."""
    _need_cuda()
    dev = packed["codes"].device
    if out is None:
        out = torch.empty(N, K, dtype=torch.int16, device=dev)
    c = cfg.c()
    _check(load().aaac_dequant(_ptr(packed["codes"]), _ptr(packed["scales_tagged"]),
                               _ptr(packed.get("choice_bits")), _ptr(packed["T_bf16"]), N, K,
                               ctypes.byref(c), _ptr(out), _stream(stream)))
    return out


def linear_workspace_size(cfg: Config, M: int, N: int, K: int) -> int:
    """Bytes of the workspace that lets linear() dequantise once (0 when the
    fused kernels are used for this token count)."""
    c = cfg.c()
    return int(load().aaac_linear_workspace_size(ctypes.byref(c), M, N, K))


def linear(X: torch.Tensor, packed: dict, cfg: Config, N: int, K: int,
           out: Optional[torch.Tensor] = None, stream=None,
           ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """W4A16 linear on a packed layer: Y[M, N] = X[M, K] @ W_hat^T, fp32.
    With a workspace (linear_workspace_size bytes) large token counts
    dequantise W once and use the TMA-fed tensor-core GEMM."""
    _need_cuda()
    assert X.dtype in (torch.bfloat16, torch.int16, torch.uint16), X.dtype
    if X.stride(1) != 1 or X.stride(0) % 8:
        X = X.contiguous()
    M, ldx = X.shape[0], X.stride(0)
    if out is None:
        out = torch.empty(M, N, dtype=torch.float32, device=X.device)
    c = cfg.c()
    if ws is not None:
        _check(load().aaac_linear_ws(_ptr(X), M, ldx, _ptr(packed["codes"]),
                                     _ptr(packed["scales_tagged"]),
                                     _ptr(packed.get("choice_bits")), _ptr(packed["T_bf16"]), N,
                                     K, ctypes.byref(c), _ptr(out), _ptr(ws), ws.numel(),
                                     _stream(stream)))
        return out
    _check(load().aaac_linear(_ptr(X), M, ldx, _ptr(packed["codes"]),
                              _ptr(packed["scales_tagged"]), _ptr(packed.get("choice_bits")),
                              _ptr(packed["T_bf16"]), N, K, ctypes.byref(c), _ptr(out),
                              _stream(stream)))
    return out


def run_layer(W: torch.Tensor, X: torch.Tensor, cfg: Config, ws: Optional[torch.Tensor] = None,
              stream=None) -> dict:
    """importance -> init -> fit -> pack for one linear, all on the GPU."""
    N, K = W.shape
    if ws is None:
        ws = workspace(cfg, N, K, X.shape[0], W.device)
    I = importance(X, ws=ws, stream=stream)
    scales, T = init_codebooks(W, cfg, ws=ws, stream=stream)
    T_init = T.clone()
    T, err_hist, stats = fit_layer(W, I, scales, T, cfg, ws=ws, stream=stream)
    out = pack(W, I, scales, T, cfg, ws=ws, stream=stream)
    out.update(global_scale=cfg.global_scale)
    out.update(I=I, scales=scales, T_init=T_init, T=T, err_hist=err_hist[:cfg.iters],
               stats=stats)
    return out


def awq_prescale(W: torch.Tensor, I: torch.Tensor, tokens: int, alpha16: int, stream=None):
    """AWQ-style pre-scaling for alpha = alpha16 / 16: (c, I', W') -- the
    per-input-channel scales, the importance of the activations x / c, and
    the rescaled bf16 weights (int16 bits)."""
    _need_cuda()
    W = _bits16(W)
    N, K = W.shape
    dev = W.device
    c = torch.empty(K, dtype=torch.float32, device=dev)
    Is = torch.empty(K, dtype=torch.float32, device=dev)
    Ws = torch.empty(N, K, dtype=torch.int16, device=dev)
    _check(load().aaac_awq_prescale(_ptr(W), N, K, _ptr(I), int(tokens), int(alpha16), _ptr(c),
                                    _ptr(Is), _ptr(Ws), _stream(stream)))
    return c, Is, Ws


def awq_fit(W: torch.Tensor, I: torch.Tensor, tokens: int, cfg: Config, alphas16,
            ws: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Grid search over alpha = j/16 for j in alphas16: pre-scale, fit and
    pack each candidate on the device and keep the first with the lowest
    err_final.  Returns the kept packed layer, c, err_final, the err_final of
    every candidate (err_alpha) and the kept position (best), on the device."""
    _need_cuda()
    W = _bits16(W)
    N, K = W.shape
    dev = W.device
    js = (ctypes.c_int32 * len(alphas16))(*[int(j) for j in alphas16])
    cfg.ensure_global_scale(dev)
    c_cfg = cfg.c()
    if ws is None:
        need = load().aaac_awq_workspace_size(ctypes.byref(c_cfg), N, K)
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    G = K // cfg.g
    sdt = torch.int16 if cfg.fmt == INT4 else torch.uint8
    nb = (K // cfg.S + 7) // 8
    out = dict(c=torch.empty(K, dtype=torch.float32, device=dev),
               T_bf16=torch.zeros(2, 16, dtype=torch.int16, device=dev),
               codes=torch.empty(N, K // 2, dtype=torch.uint8, device=dev),
               scales_tagged=torch.empty(N, G, dtype=sdt, device=dev),
               choice_bits=(torch.empty(N, nb, dtype=torch.uint8, device=dev)
                            if cfg.S != cfg.g else None),
               err_final=torch.zeros(1, dtype=torch.float64, device=dev),
               err_alpha=torch.zeros(len(alphas16), dtype=torch.float64, device=dev),
               best=torch.full((1,), -1, dtype=torch.int32, device=dev))
    _check(load().aaac_awq_fit(_ptr(W), N, K, _ptr(I), int(tokens), ctypes.byref(c_cfg), js,
                               len(alphas16), _ptr(out["c"]), _ptr(out["T_bf16"]),
                               _ptr(out["codes"]), _ptr(out["scales_tagged"]),
                               _ptr(out["choice_bits"]), _ptr(out["err_final"]),
                               _ptr(out["err_alpha"]), _ptr(out["best"]), _ptr(ws), ws.numel(),
                               _stream(stream)))
    return out


# --------------------------------------------------------------------------
# microscaled 4-bit tensors: quantisation, the way back, and the product (no
# backward pass: outputs carry no gradient)
# --------------------------------------------------------------------------
MX_E8M0 = 0  # blocks of 32, power-of-two scales
MX_E4M3 = 1  # blocks of 16, E4M3 scales, a power of two per row
MX_SWIGLU = 1
_MX_TYPES = {torch.bfloat16: 0, torch.float32: 1}


class CMxTensor(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("groups", ctypes.c_int32), ("rows", ctypes.c_int64),
                ("K", ctypes.c_int64), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("row_scale", ctypes.c_void_p), ("offsets", ctypes.c_void_p)]


class CMxSource(ctypes.Structure):
    _fields_ = [("X", ctypes.c_void_p), ("type", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("rows", ctypes.c_int64), ("ldx", ctypes.c_int64), ("index", ctypes.c_void_p)]


def mx_scale_bytes(fmt: int, rows: int, K: int, groups: int = 1) -> int:
    """Bytes of a microscaled tensor's scales (see aaac_mx_tensor)."""
    return int(load().aaac_mx_scale_bytes(fmt, rows, K, groups))


def mx_workspace_size(fmt: int, rows: int, K: int, groups: int = 1, swiglu: bool = False) -> int:
    """Bytes of the workspace in which mx_linear quantises its activations (0
    for the few rows that the product's kernel quantises itself)."""
    return int(load().aaac_mx_workspace_size(fmt, rows, K, groups, MX_SWIGLU if swiglu else 0))


def mx_launch_plan(groups: int, rows: int, N: int, K: int) -> dict:
    """Host-only: the product's plan for these sizes (see aaac_mx_launch_plan)."""
    out = (ctypes.c_int32 * 6)()
    _check(load().aaac_mx_launch_plan(groups, rows, N, K, out))
    return dict(zip(("columns", "split", "ctas", "stages", "tiles", "rows"), list(out)))


class MxTensor:
    """A microscaled 4-bit tensor on the device (aaac_mx_tensor): codes uint8
    [rows, K/2], scales uint8 (mx_scale_bytes of them), row_scale fp32 [rows]
    (MX_E4M3).  Its rows come in `groups` groups: equal ones, or
    offsets[e] : offsets[e + 1] (int32 [groups + 1])."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor,
                 row_scale: Optional[torch.Tensor], fmt: int, groups: int = 1,
                 offsets: Optional[torch.Tensor] = None):
        if codes.dtype != torch.uint8 or codes.dim() != 2 or not codes.is_contiguous():
            raise ValueError("codes must be contiguous uint8 [rows, K/2]")
        rows, half = codes.shape
        # tiles of 128 rows x 4 blocks; every call checks the sizes themselves
        need = (rows // 128 + groups) * -(-half // (64 if fmt == MX_E8M0 else 32)) * 512
        if scales.dtype != torch.uint8 or scales.numel() < need or not scales.is_contiguous():
            raise ValueError(f"scales must be contiguous uint8, {need} bytes")
        if fmt != MX_E4M3:
            row_scale = None
        elif (row_scale is None or row_scale.dtype != torch.float32 or row_scale.numel() < rows
              or not row_scale.is_contiguous()):
            raise ValueError(f"row_scale must be contiguous float32 [{rows}]")
        if offsets is not None:
            _mx_offsets(offsets, groups)
        _mx_on(codes.get_device(), scales, row_scale, offsets)
        self._codes, self._scales, self._row_scale = codes, scales, row_scale
        self._set(fmt, groups, offsets, rows, 2 * half, codes.get_device(), codes.data_ptr(),
                  scales.data_ptr(), None if row_scale is None else row_scale.data_ptr())

    def _set(self, fmt, groups, offsets, rows, K, device, codes, scales, row_scale):
        self.fmt, self.groups, self.offsets = fmt, groups, offsets
        self.rows, self.K, self._device = rows, K, device
        self._c = CMxTensor(fmt, groups, rows, K, codes, scales, row_scale,
                            None if offsets is None else offsets.data_ptr())
        self._ref = ctypes.byref(self._c)

    # A tensor made by empty() keeps its parts in one allocation and cuts them
    # out when they are asked for: decoding asks for none of them.
    @property
    def codes(self) -> torch.Tensor:
        if self._codes is None:
            at, n = self._scale_bytes, self.rows * (self.K // 2)
            self._codes = self._buffer[at:at + n].view(self.rows, self.K // 2)
        return self._codes

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is None:
            self._scales = self._buffer[:self._scale_bytes]
        return self._scales

    @property
    def row_scale(self) -> Optional[torch.Tensor]:
        if self._row_scale is None and self.fmt == MX_E4M3:
            at = self._scale_bytes + self.rows * (self.K // 2)
            self._row_scale = self._buffer[at:at + 4 * self.rows].view(torch.float32)
        return self._row_scale

    @property
    def device(self):
        return torch.device("cuda", self._device)

    @staticmethod
    def empty(fmt: int, rows: int, K: int, groups: int = 1,
              offsets: Optional[torch.Tensor] = None, device="cuda") -> "MxTensor":
        size = _mx_bytes((_lib or load()).aaac_mx_scale_bytes, fmt, rows, K, groups)
        if offsets is not None:
            _mx_offsets(offsets, groups)
        # scales (a multiple of 512 bytes), then codes (of 16 a row), then row scales
        n = rows * (K // 2)
        t = object.__new__(MxTensor)
        t._buffer = b = torch.empty(size + n + 4 * rows, dtype=torch.uint8, device=device)
        t._scale_bytes = size
        t._codes = t._scales = t._row_scale = None
        at = b.data_ptr()
        t._set(fmt, groups, offsets, rows, K, b.get_device(), at + size, at,
               at + size + n if fmt == MX_E4M3 else None)
        return t


def _mx_bytes(size, fmt: int, rows: int, K: int, groups: int) -> int:
    """A size query's answer; its refusal (0) as the error it names."""
    need = size(fmt, rows, K, groups)
    if need == 0:
        raise AaacError(2, load().aaac_last_error().decode())
    return need


def _mx_offsets(offsets: torch.Tensor, groups: int) -> None:
    if (offsets.dtype != torch.int32 or offsets.numel() != groups + 1
            or not offsets.is_contiguous()):
        raise ValueError(f"offsets must be contiguous int32 [{groups + 1}]")


def _mx_on(device: int, *tensors) -> None:
    """Every tensor on CUDA device `device`."""
    if device < 0:
        _need_cuda()
        raise ValueError("libaaac takes device tensors only")
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"tensors on device {t.get_device()} and device {device}")


def _mx_same(device: int, t: "MxTensor") -> None:
    if t._device != device:
        raise ValueError(f"tensors on device {t._device} and device {device}")


def _mx_stream(device: int, stream) -> int:
    """The stream a call runs on.  The library launches on the current device,
    so the tensors have to be there."""
    if device != torch.cuda.current_device():
        raise ValueError(f"tensors on device {device}, but the current device is "
                         f"{torch.cuda.current_device()}")
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(device)


def _on_stream(f, stream, *args):
    """f(*args), its own allocations made on `stream` (the caching allocator
    ties memory to the stream it was allocated on)."""
    with torch.cuda.stream(stream):
        return f(*args)


def _mx_source(X: torch.Tensor, rows: Optional[torch.Tensor], swiglu: bool):
    """(aaac_mx_source, quantised rows, K, the tensor it points into)."""
    kind = _MX_TYPES.get(X.dtype)
    if kind is None or X.dim() != 2:
        raise ValueError("X must be a bfloat16 or float32 matrix")
    n, width = X.shape
    if swiglu and width % 2:
        raise ValueError(f"X has {width} columns, not two halves")
    ldx, step = X.stride()
    at = X.data_ptr()
    # 16-byte aligned rows: 8 bf16 or 4 fp32 values
    if step != 1 or ldx % (4 if kind else 8) or ldx < width or at % 16:
        X = X.contiguous()
        ldx, at = width, X.data_ptr()
    if rows is None:
        index, out_rows = None, n
    else:
        if rows.dtype != torch.int32 or rows.dim() != 1 or not rows.is_contiguous():
            raise ValueError("rows must be contiguous int32 [quantised rows]")
        index, out_rows = rows.data_ptr(), rows.numel()
    if swiglu:
        return CMxSource(at, kind, MX_SWIGLU, n, ldx, index), out_rows, width // 2, X
    return CMxSource(at, kind, 0, n, ldx, index), out_rows, width, X


def _mx_out(out: Optional[torch.Tensor], rows: int, cols: int, dtype, device):
    """(output, its aaac_type, its leading dimension)."""
    if out is None:
        kind = _MX_TYPES.get(dtype)
        if kind is None:
            raise ValueError(f"the output is bfloat16 or float32, not {dtype}")
        return torch.empty((rows, cols), dtype=dtype, device=device), kind, cols
    if (out.shape != (rows, cols) or out.dtype not in _MX_TYPES
            or (cols > 1 and out.stride(1) != 1)):
        raise ValueError(f"out must be a bfloat16 or float32 [{rows}, {cols}] with "
                         "consecutive columns")
    return out, _MX_TYPES[out.dtype], out.stride(0) if rows > 1 else max(out.stride(0), cols)


def mx_quantize(X: torch.Tensor, fmt: int, rows: Optional[torch.Tensor] = None,
                swiglu: bool = False, groups: int = 1,
                offsets: Optional[torch.Tensor] = None, out: Optional[MxTensor] = None,
                stream=None) -> MxTensor:
    """Rows of X (bf16 or fp32 [n, K]) as a microscaled 4-bit tensor.  rows
    (int32) picks the source row of each quantised row (-1: a row of zeros);
    swiglu quantises silu(a) * b of X's two halves [n, 2K]; groups and offsets
    are the rows' groups (see MxTensor)."""
    if stream is not None:
        return _on_stream(_mx_quantize, stream, X, fmt, rows, swiglu, groups, offsets, out, stream)
    return _mx_quantize(X, fmt, rows, swiglu, groups, offsets, out, None)


def _mx_quantize(X, fmt, rows, swiglu, groups, offsets, out, stream):
    src, n, K, X = _mx_source(X, rows, swiglu)
    device = X.get_device()
    if out is None:
        _mx_on(device, rows, offsets)
        out = MxTensor.empty(fmt, n, K, groups, offsets, device)
    else:
        if (out.fmt, out.rows, out.K) != (fmt, n, K):
            raise ValueError(f"out is fmt {out.fmt} [{out.rows}, {out.K}], not {fmt} [{n}, {K}]")
        if (groups not in (1, out.groups)
                or (offsets is not None and offsets is not out.offsets)):
            raise ValueError("out has its own groups and offsets")
        _mx_on(device, rows)
        _mx_same(device, out)
    _check((_lib or load()).aaac_mx_quantize(ctypes.byref(src), out._ref,
                                             _mx_stream(device, stream)))
    return out


def mx_dequant(q: MxTensor, dtype=torch.bfloat16, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """A microscaled tensor's values, bf16 or fp32 [rows, K] (rows of no group are
    not written)."""
    if stream is not None:
        return _on_stream(_mx_dequant, stream, q, dtype, out, stream)
    return _mx_dequant(q, dtype, out, None)


def _mx_dequant(q, dtype, out, stream):
    device = q._device
    out, kind, ld = _mx_out(out, q.rows, q.K, dtype, device)
    _mx_on(device, out)
    _check((_lib or load()).aaac_mx_dequant(q._ref, out.data_ptr(), kind, ld,
                                            _mx_stream(device, stream)))
    return out


def mx_linear(X: Union[torch.Tensor, MxTensor], W: MxTensor, out: Optional[torch.Tensor] = None,
              out_dtype=torch.float32, rows: Optional[torch.Tensor] = None, swiglu: bool = False,
              offsets: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """Y[rows, N] = X @ W^T on the 4-bit tensor cores; with W.groups > 1 each
    group of X's rows (an expert's) meets its own N rows of W.  X is a
    microscaled tensor, or bf16 / fp32 activations that are quantised here as
    mx_quantize does (rows, swiglu and offsets as there; ws: a workspace of
    mx_workspace_size bytes).  Rows of no group are not written: without out
    they hold anything."""
    if isinstance(X, MxTensor):
        if rows is not None or swiglu or offsets is not None or ws is not None:
            raise ValueError("rows, swiglu, offsets and ws go with activations that are not "
                             "quantised yet")
        if stream is not None:
            return _on_stream(_mx_product, stream, X, W, out, out_dtype, stream)
        return _mx_product(X, W, out, out_dtype, None)
    if stream is not None:
        return _on_stream(_mx_linear, stream, X, W, out, out_dtype, rows, swiglu, offsets, ws,
                          stream)
    return _mx_linear(X, W, out, out_dtype, rows, swiglu, offsets, ws, None)


def _mx_product(X, W, out, out_dtype, stream):
    device = X._device
    _mx_same(device, W)
    out, kind, ld = _mx_out(out, X.rows, W.rows // W.groups, out_dtype, device)
    _mx_on(device, out)
    _check((_lib or load()).aaac_mx_linear(X._ref, W._ref, out.data_ptr(), kind, ld,
                                           _mx_stream(device, stream)))
    return out


def _mx_linear(X, W, out, out_dtype, rows, swiglu, offsets, ws, stream):
    src, n, K, X = _mx_source(X, rows, swiglu)
    device = X.get_device()
    if K != W.K:
        raise ValueError(f"X has K={K}, W has K={W.K}")
    if ws is not None and not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    _mx_on(device, rows, offsets, out, ws)
    _mx_same(device, W)
    if offsets is not None:
        _mx_offsets(offsets, W.groups)
    out, kind, ld = _mx_out(out, n, W.rows // W.groups, out_dtype, device)
    lib = _lib or load()
    if ws is None:
        # 0: the product quantises these rows itself (or refuses the sizes below)
        size = lib.aaac_mx_workspace_size(W.fmt, n, K, W.groups, src.flags)
        ws = torch.empty(size, dtype=torch.uint8, device=device) if size else None
    else:
        size = ws.numel() * ws.element_size()
    _check(lib.aaac_mx_linear_ws(ctypes.byref(src), n,
                                 None if offsets is None else offsets.data_ptr(), W._ref,
                                 out.data_ptr(), kind, ld, None if ws is None else ws.data_ptr(), size,
                                 _mx_stream(device, stream)))
    return out


# --------------------------------------------------------------------------
# row-sharded calls (one layer's rows over several processes / GPUs)
# --------------------------------------------------------------------------
class ShardReducer:
    """Adapts a Python all-reduce to the library's callback.  The library
    hands a buffer inside the workspace `ws`; `allreduce(t, op)` receives a
    torch view of it (int64 or int32) and op "sum" or "max", and must combine
    it in place over all shards on the current stream (for example
    torch.distributed.all_reduce with NCCL)."""

    def __init__(self, ws: torch.Tensor, allreduce):
        self.ws, self.allreduce, self.error = ws, allreduce, None

        def cb(user, buf, count, op, stream):
            try:
                off = int(buf) - self.ws.data_ptr()
                esz = 8 if op in (REDUCE_SUM_I64, REDUCE_MAX_I64) else 4
                dt = torch.int64 if esz == 8 else torch.int32
                assert 0 <= off and off + count * esz <= self.ws.numel()
                t = self.ws[off:off + count * esz].view(dt)
                self.allreduce(t, "sum" if op in (REDUCE_SUM_I64, REDUCE_SUM_I32) else "max")
                return 0
            except Exception as e:  # reported by the call as AAAC_ERR_COLLECTIVE
                self.error = e
                return 1

        self.fn = REDUCE_FN(cb)  # kept alive with the reducer

    def check(self, status: int):
        if status == 8 and self.error is not None:
            raise AaacError(status, f"reduce callback failed: {self.error!r}")
        _check(status)


def torch_allreduce(group=None):
    """An allreduce for ShardReducer over torch.distributed (NCCL on GPUs)."""
    import torch.distributed as dist

    def run(t, op):
        dist.all_reduce(t, op=dist.ReduceOp.SUM if op == "sum" else dist.ReduceOp.MAX,
                        group=group)
    return run


def init_codebooks_sharded(W: torch.Tensor, N_total: int, cfg: Config, allreduce,
                           ws: Optional[torch.Tensor] = None, stream=None):
    """init_codebooks over a layer whose rows are split over shards; this
    shard holds W [N, K].  Returns (scales [N, K/g], T [2, 16]); T is the
    whole layer's quantile initialisation on every shard."""
    _need_cuda()
    W = _bits16(W)
    N, K = W.shape
    sdt = torch.int16 if cfg.fmt == INT4 else torch.uint8
    scales = torch.empty(N, K // cfg.g, dtype=sdt, device=W.device)
    T = torch.empty(2, 16, dtype=torch.float32, device=W.device)
    if ws is None:
        ws = workspace(cfg, N, K, 0, W.device)
    cfg.ensure_global_scale(W.device)
    red = ShardReducer(ws, allreduce)
    c = cfg.c()
    red.check(load().aaac_init_codebooks_sharded(_ptr(W), N, K, int(N_total), ctypes.byref(c),
                                                 _ptr(scales), _ptr(T), red.fn, None, _ptr(ws),
                                                 ws.numel(), _stream(stream)))
    return scales, T


def fit_layer_sharded(W: torch.Tensor, N_total: int, I: torch.Tensor, scales: torch.Tensor,
                      T: torch.Tensor, cfg: Config, allreduce, ws: Optional[torch.Tensor] = None,
                      stream=None):
    """fit_layer over a row-sharded layer.  Returns (T, err_hist, stats); every
    shard gets the whole layer's tables, history and counters."""
    _need_cuda()
    W = _bits16(W)
    N, K = W.shape
    err_hist = torch.zeros(max(cfg.iters, 1), dtype=torch.float64, device=W.device)
    stats = torch.zeros(STATS_BYTES, dtype=torch.uint8, device=W.device)
    if ws is None:
        ws = workspace(cfg, N, K, 0, W.device)
    red = ShardReducer(ws, allreduce)
    c = cfg.c()
    red.check(load().aaac_fit_layer_sharded(_ptr(W), N, K, int(N_total), _ptr(I), _ptr(scales),
                                            ctypes.byref(c), _ptr(T), _ptr(err_hist),
                                            _ptr(stats), red.fn, None, _ptr(ws), ws.numel(),
                                            _stream(stream)))
    return T, err_hist, stats


def pack_sharded(W: torch.Tensor, N_total: int, I: torch.Tensor, scales: torch.Tensor,
                 T: torch.Tensor, cfg: Config, allreduce, ws: Optional[torch.Tensor] = None,
                 stream=None) -> dict:
    """pack of this shard's rows; err_final is the whole layer's."""
    _need_cuda()
    W = _bits16(W)
    N, K = W.shape
    dev = W.device
    nb = (K // cfg.S + 7) // 8
    out = dict(T_bf16=torch.zeros(2, 16, dtype=torch.int16, device=dev),
               codes=torch.empty(N, K // 2, dtype=torch.uint8, device=dev),
               scales_tagged=torch.empty_like(scales),
               choice_bits=(torch.empty(N, nb, dtype=torch.uint8, device=dev)
                            if cfg.S != cfg.g else None),
               err_final=torch.zeros(1, dtype=torch.float64, device=dev))
    if ws is None:
        ws = workspace(cfg, N, K, 0, dev)
    red = ShardReducer(ws, allreduce)
    c = cfg.c()
    red.check(load().aaac_pack_sharded(_ptr(W), N, K, int(N_total), _ptr(I), _ptr(scales),
                                       ctypes.byref(c), _ptr(T), _ptr(out["T_bf16"]),
                                       _ptr(out["codes"]), _ptr(out["scales_tagged"]),
                                       _ptr(out["choice_bits"]), _ptr(out["err_final"]),
                                       red.fn, None, _ptr(ws), ws.numel(), _stream(stream)))
    return out
