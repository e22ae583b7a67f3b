"""ctypes binding of the Muon C ABI (``include/muon.h``).

Argument marshalling only: tensors become device pointers, leading dimensions
and dtype codes; every step of the computation runs in the HIP library.  The
library must be built (``newton_schulz_matrix_step_amd._build.build()``); if it
is missing, loading raises instead of falling back to anything else.
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import List, Optional, Sequence

# the in-tree build; MUON_LIBRARY names another build of the same library to load instead
LIB_PATH = os.environ.get("MUON_LIBRARY") or os.path.join(os.path.dirname(os.path.abspath(__file__)),
                                                          "libmuon_mi355x.so")
ABI_VERSION = 7   # the MUON_ABI_VERSION of the header this binding mirrors

MUON_OK = 0
MUON_ERR_INVALID_ARG = 1
MUON_ERR_DTYPE = 2
MUON_ERR_NO_DEVICE = 3
MUON_ERR_OOM = 4
MUON_ERR_HIP = 5

MUON_BF16 = 0
MUON_F32 = 1
MUON_COMPUTE_BF16 = 0
MUON_COMPUTE_FP32 = 1

# layer operators
MUON_ACT8_GROUP = 32       # columns of a row that share one exponent of an 8-bit checkpoint
ACTIVATIONS = {"none": 0, "gelu": 1, "relu_sq": 2}        # muon_activation
W_LAYOUTS = {"in_out": 0, "out_in": 1}                    # muon_weight_layout

MUON_INIT_PROFILE = 0x1
MUON_INIT_FAIL_ALLOC = 0x2
MUON_INIT_DEBUG = 0x4

# kernel roles (muon_role), named as in muon_kernel_stats
ROLE_NAMES = ("momentum_norm", "norm_finalize", "ns_gram", "ns_poly", "ns_axpy", "ns_axpy_update",
              "direct_update", "fill_zero", "adamw", "norm_rescale")


def profile_roles(names) -> int:
    """MUON_INIT_PROFILE_ROLES for the named roles: init flag bits that limit a
    profiling handle's events to those roles."""
    mask = 0
    for nm in names:
        mask |= 1 << ROLE_NAMES.index(nm)
    return (mask & 0x3FF) << 16

EXPORTED_SYMBOLS = (
    "muon_abi_version",
    "muon_init",
    "muon_step",
    "muon_step_noalloc",
    "muon_adamw_step",
    "muon_orthogonalize",
    "muon_layernorm_forward",
    "muon_layernorm_backward",
    "muon_linear_forward",
    "muon_linear_grad_input",
    "muon_linear_grad_weight",
    "muon_act_encode",
    "muon_act_decode",
    "muon_read_norms",
    "muon_kernel_stats_read",
    "muon_kernel_stats_reset",
    "muon_workspace_bytes",
    "muon_destroy",
    "muon_status_str",
    "muon_last_error",
)


class muon_matrix(ctypes.Structure):
    _fields_ = [
        ("param", ctypes.c_void_p),
        ("grad", ctypes.c_void_p),
        ("momentum", ctypes.c_void_p),
        ("update_out", ctypes.c_void_p),
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("ld_param", ctypes.c_int64),
        ("ld_grad", ctypes.c_int64),
        ("ld_mom", ctypes.c_int64),
        ("ld_update", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("block_rows", ctypes.c_int32),
        ("block_cols", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class muon_adamw_tensor(ctypes.Structure):
    _fields_ = [
        ("param", ctypes.c_void_p),
        ("grad", ctypes.c_void_p),
        ("exp_avg", ctypes.c_void_p),
        ("exp_avg_sq", ctypes.c_void_p),
        ("numel", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class muon_adamw_hparams(ctypes.Structure):
    _fields_ = [
        ("lr", ctypes.c_float),
        ("beta1", ctypes.c_float),
        ("beta2", ctypes.c_float),
        ("eps", ctypes.c_float),
        ("weight_decay", ctypes.c_float),
        ("step", ctypes.c_int32),
    ]


class muon_hparams(ctypes.Structure):
    _fields_ = [
        ("lr", ctypes.c_float),
        ("beta", ctypes.c_float),
        ("weight_decay", ctypes.c_float),
        ("eps", ctypes.c_float),
        ("a", ctypes.c_float),
        ("b", ctypes.c_float),
        ("c", ctypes.c_float),
        ("nesterov", ctypes.c_int32),
        ("ns_steps", ctypes.c_int32),
        ("compute", ctypes.c_int32),
        ("coeffs", ctypes.POINTER(ctypes.c_float)),
    ]


class muon_kernel_stats(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 48), ("launches", ctypes.c_int64), ("total_ms", ctypes.c_double)]


class muon_act8(ctypes.Structure):
    _fields_ = [
        ("codes", ctypes.c_void_p),
        ("exponents", ctypes.c_void_p),
        ("ld_codes", ctypes.c_int64),
        ("ld_exponents", ctypes.c_int64),
    ]


class muon_layernorm_args(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("gain", ctypes.c_void_p),
        ("bias", ctypes.c_void_p),
        ("y", ctypes.c_void_p),
        ("mean", ctypes.c_void_p),
        ("rstd", ctypes.c_void_p),
        ("y8", muon_act8),
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("ld_x", ctypes.c_int64),
        ("ld_y", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("param_dtype", ctypes.c_int32),
        ("eps", ctypes.c_float),
        ("reserved", ctypes.c_int32),
    ]


class muon_layernorm_grad_args(ctypes.Structure):
    _fields_ = [
        ("dy", ctypes.c_void_p),
        ("x", ctypes.c_void_p),
        ("gain", ctypes.c_void_p),
        ("mean", ctypes.c_void_p),
        ("rstd", ctypes.c_void_p),
        ("add", ctypes.c_void_p),
        ("dx", ctypes.c_void_p),
        ("dgain", ctypes.c_void_p),
        ("dbias", ctypes.c_void_p),
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("ld_dy", ctypes.c_int64),
        ("ld_x", ctypes.c_int64),
        ("ld_add", ctypes.c_int64),
        ("ld_dx", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("param_dtype", ctypes.c_int32),
        ("accumulate", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class muon_linear_args(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("w", ctypes.c_void_p),
        ("bias", ctypes.c_void_p),
        ("residual", ctypes.c_void_p),
        ("y", ctypes.c_void_p),
        ("z", ctypes.c_void_p),
        ("z8", muon_act8),
        ("rows", ctypes.c_int64),
        ("in_", ctypes.c_int64),
        ("out", ctypes.c_int64),
        ("ld_x", ctypes.c_int64),
        ("ld_w", ctypes.c_int64),
        ("ld_residual", ctypes.c_int64),
        ("ld_y", ctypes.c_int64),
        ("ld_z", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("bias_dtype", ctypes.c_int32),
        ("activation", ctypes.c_int32),
        ("w_layout", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class muon_linear_grad_input_args(ctypes.Structure):
    _fields_ = [
        ("dy", ctypes.c_void_p),
        ("w", ctypes.c_void_p),
        ("z", ctypes.c_void_p),
        ("z8", muon_act8),
        ("add", ctypes.c_void_p),
        ("dx", ctypes.c_void_p),
        ("act_out", ctypes.c_void_p),
        ("rows", ctypes.c_int64),
        ("in_", ctypes.c_int64),
        ("out", ctypes.c_int64),
        ("ld_dy", ctypes.c_int64),
        ("ld_w", ctypes.c_int64),
        ("ld_z", ctypes.c_int64),
        ("ld_add", ctypes.c_int64),
        ("ld_dx", ctypes.c_int64),
        ("ld_act_out", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("activation", ctypes.c_int32),
        ("w_layout", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class muon_linear_grad_weight_args(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("x8", muon_act8),
        ("dy", ctypes.c_void_p),
        ("dw", ctypes.c_void_p),
        ("db", ctypes.c_void_p),
        ("rows", ctypes.c_int64),
        ("in_", ctypes.c_int64),
        ("out", ctypes.c_int64),
        ("ld_x", ctypes.c_int64),
        ("ld_dy", ctypes.c_int64),
        ("ld_dw", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("dw_dtype", ctypes.c_int32),
        ("db_dtype", ctypes.c_int32),
        ("w_layout", ctypes.c_int32),
        ("accumulate", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class MuonError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{status_str(status)}: {msg}" if msg else status_str(status))
        self.status = status


_lib: Optional[ctypes.CDLL] = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the HIP library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"Muon HIP library not built: {path} is missing "
                          "(run newton_schulz_matrix_step_amd._build.build())")
    lib = ctypes.CDLL(path)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.muon_abi_version.restype = ctypes.c_int
    lib.muon_abi_version.argtypes = []
    if lib.muon_abi_version() != ABI_VERSION:
        raise ImportError(f"{path} implements ABI version {lib.muon_abi_version()}, the binding expects "
                          f"{ABI_VERSION}: rebuild the library")
    lib.muon_init.restype = ctypes.c_int
    lib.muon_init.argtypes = [ctypes.POINTER(vp), ctypes.c_int, ctypes.c_uint32]
    lib.muon_step.restype = ctypes.c_int
    lib.muon_step.argtypes = [vp, ctypes.POINTER(muon_matrix), i32, ctypes.POINTER(muon_hparams), vp]
    lib.muon_step_noalloc.restype = ctypes.c_int
    lib.muon_step_noalloc.argtypes = [vp, ctypes.POINTER(muon_matrix), i32, ctypes.POINTER(muon_hparams), vp]
    lib.muon_adamw_step.restype = ctypes.c_int
    lib.muon_adamw_step.argtypes = [vp, ctypes.POINTER(muon_adamw_tensor), i32, ctypes.POINTER(muon_adamw_hparams), vp]
    lib.muon_orthogonalize.restype = ctypes.c_int
    lib.muon_orthogonalize.argtypes = [vp, vp, vp, i64, i64, i64, i64, i32, ctypes.POINTER(muon_hparams), vp]
    for name, st in (("muon_layernorm_forward", muon_layernorm_args),
                     ("muon_layernorm_backward", muon_layernorm_grad_args),
                     ("muon_linear_forward", muon_linear_args),
                     ("muon_linear_grad_input", muon_linear_grad_input_args),
                     ("muon_linear_grad_weight", muon_linear_grad_weight_args)):
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = [vp, ctypes.POINTER(st), vp]
    lib.muon_act_encode.restype = ctypes.c_int
    lib.muon_act_encode.argtypes = [vp, vp, i64, i64, i64, i32, ctypes.POINTER(muon_act8), vp]
    lib.muon_act_decode.restype = ctypes.c_int
    lib.muon_act_decode.argtypes = [vp, ctypes.POINTER(muon_act8), vp, i64, i64, i64, i32, vp]
    lib.muon_read_norms.restype = ctypes.c_int
    lib.muon_read_norms.argtypes = [vp, ctypes.POINTER(ctypes.c_float), i32, vp]
    lib.muon_kernel_stats_read.restype = i32
    lib.muon_kernel_stats_read.argtypes = [vp, ctypes.POINTER(muon_kernel_stats), i32]
    lib.muon_kernel_stats_reset.restype = None
    lib.muon_kernel_stats_reset.argtypes = [vp]
    lib.muon_workspace_bytes.restype = i64
    lib.muon_workspace_bytes.argtypes = [vp]
    lib.muon_destroy.restype = ctypes.c_int
    lib.muon_destroy.argtypes = [vp]
    lib.muon_status_str.restype = ctypes.c_char_p
    lib.muon_status_str.argtypes = [ctypes.c_int]
    lib.muon_last_error.restype = ctypes.c_char_p
    lib.muon_last_error.argtypes = [vp]
    _lib = lib
    return lib


def status_str(status: int) -> str:
    return load().muon_status_str(int(status)).decode()


def _check(handle, status: int) -> None:
    if status != MUON_OK:
        msg = load().muon_last_error(handle).decode() if handle else ""
        raise MuonError(status, msg)


@dataclass
class Hparams:
    lr: float = 0.02
    beta: float = 0.95
    weight_decay: float = 0.0
    eps: float = 1e-7
    a: float = 3.4445
    b: float = -4.7750
    c: float = 2.0315
    nesterov: bool = False
    ns_steps: int = 5
    compute: str = "bf16"      # "bf16" or "fp32"
    coeffs: Optional[Sequence[Sequence[float]]] = None   # per-iteration (a_k, b_k, c_k)

    def to_c(self) -> muon_hparams:
        comp = {"bf16": MUON_COMPUTE_BF16, "fp32": MUON_COMPUTE_FP32}.get(self.compute, -1)
        hp = muon_hparams(self.lr, self.beta, self.weight_decay, self.eps, self.a, self.b, self.c,
                          int(bool(self.nesterov)), int(self.ns_steps), comp, None)
        if self.coeffs is not None:
            flat = [float(v) for t in self.coeffs for v in t]
            if len(flat) != 3 * len(self.coeffs) or len(self.coeffs) < self.ns_steps:
                raise ValueError("coeffs: one (a, b, c) triple per iteration")
            arr = (ctypes.c_float * len(flat))(*flat)
            hp.coeffs = ctypes.cast(arr, ctypes.POINTER(ctypes.c_float))
            hp._coeffs_keepalive = arr   # the array lives as long as the struct
        return hp


@dataclass
class AdamWHparams:
    lr: float = 1e-3
    beta1: float = 0.9
    beta2: float = 0.999
    eps: float = 1e-8
    weight_decay: float = 0.01
    step: int = 1              # 1-based step count of this update

    def to_c(self) -> muon_adamw_hparams:
        return muon_adamw_hparams(self.lr, self.beta1, self.beta2, self.eps, self.weight_decay, int(self.step))


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return MUON_BF16
    if t.dtype == torch.float32:
        return MUON_F32
    return -1


def _ld(t) -> int:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("matrices must be 2-D with unit column stride")
    return int(t.stride(0))


def _stream_ptr(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def muon_abi_version() -> int:
    return int(load().muon_abi_version())


def muon_init(device: int = 0, flags: int = 0) -> int:
    h = ctypes.c_void_p()
    st = load().muon_init(ctypes.byref(h), int(device), int(flags))
    _check(None, st)
    return h.value


def _check_device_tensors(what: str, tensors, device=None):
    """Every tensor a CUDA (HIP) tensor on one device; returns that device."""
    for t in tensors:
        if not getattr(t, "is_cuda", False):
            raise ValueError(f"{what}: tensors must be on the GPU (got one on {t.device})")
        if device is None:
            device = t.device
        elif t.device != device:
            raise ValueError(f"{what}: tensors on {device} and {t.device}")
    return device


def make_matrix(param, grad, momentum, update_out=None, block=(0, 0)) -> muon_matrix:
    """Describe one weight's tensors (device tensors on one device, unit column
    stride); ``block`` = (block_rows, block_cols) cuts it into separately
    orthogonalised blocks (0 = the whole dimension).  The C ABI sees only
    pointers and sizes, so shapes and dtypes are checked here: grad,
    momentum and update_out have param's shape, momentum and update_out are
    float32, param and grad share a dtype."""
    import torch
    ts = [param, grad, momentum] + ([update_out] if update_out is not None else [])
    for t in ts:
        if t.dim() != 2:
            raise ValueError("muon_step: param, grad, momentum and update_out must be 2-D")
    shape = tuple(param.shape)
    for nm, t in (("grad", grad), ("momentum", momentum), ("update_out", update_out)):
        if t is not None and tuple(t.shape) != shape:
            raise ValueError(f"muon_step: {nm} has shape {tuple(t.shape)}, param {shape}")
    if momentum.dtype != torch.float32:
        raise ValueError(f"muon_step: momentum must be float32, got {momentum.dtype}")
    if update_out is not None and update_out.dtype != torch.float32:
        raise ValueError(f"muon_step: update_out must be float32, got {update_out.dtype}")
    _check_device_tensors("muon_step", ts)
    return muon_matrix(
        param.data_ptr(), grad.data_ptr(), momentum.data_ptr(),
        update_out.data_ptr() if update_out is not None else None,
        int(param.shape[0]), int(param.shape[1]),
        _ld(param), _ld(grad), _ld(momentum), _ld(update_out) if update_out is not None else 0,
        _dtype_code(param) if _dtype_code(param) == _dtype_code(grad) else -1,
        int(block[0]), int(block[1]), 0)


def _matrices(params: Sequence, grads: Sequence, moms: Sequence, update_outs: Optional[Sequence] = None,
              blocks: Optional[Sequence] = None):
    """The muon_matrix array of one call."""
    n = len(params)
    if len(grads) != n or len(moms) != n or (update_outs is not None and len(update_outs) != n) or \
            (blocks is not None and len(blocks) != n):
        raise ValueError("params, grads, moms (and update_outs, blocks) must have the same length")
    arr = (muon_matrix * max(n, 1))()
    for i in range(n):
        arr[i] = make_matrix(params[i], grads[i], moms[i], update_outs[i] if update_outs is not None else None,
                             blocks[i] if blocks is not None else (0, 0))
    return arr, n


def muon_step(handle: int, params: Sequence, grads: Sequence, moms: Sequence, hp: Hparams,
              update_outs: Optional[Sequence] = None, stream=None, blocks: Optional[Sequence] = None) -> None:
    """One Muon step over every (param, grad, momentum) triple, on ``stream``;
    ``blocks[i]`` = (block_rows, block_cols) of matrix i, or None for all (0, 0)."""
    arr, n = _matrices(params, grads, moms, update_outs, blocks)
    c_hp = hp.to_c()
    st = load().muon_step(handle, arr, n, ctypes.byref(c_hp), _stream_ptr(stream))
    _check(handle, st)


def muon_step_noalloc(handle: int, params: Sequence, grads: Sequence, moms: Sequence, hp: Hparams,
                      update_outs: Optional[Sequence] = None, stream=None, blocks: Optional[Sequence] = None) -> None:
    """muon_step without any device allocation: the library's static
    per-GPU scratch holds every buffer beyond the caller's tensors."""
    arr, n = _matrices(params, grads, moms, update_outs, blocks)
    c_hp = hp.to_c()
    st = load().muon_step_noalloc(handle, arr, n, ctypes.byref(c_hp), _stream_ptr(stream))
    _check(handle, st)


def make_adamw_tensor(param, grad, exp_avg, exp_avg_sq) -> muon_adamw_tensor:
    """Describe one AdamW tensor (contiguous device tensors of equal size, on one device)."""
    for t in (param, grad, exp_avg, exp_avg_sq):
        if not t.is_contiguous():
            raise ValueError("AdamW tensors must be contiguous")
    n = int(param.numel())
    if any(int(t.numel()) != n for t in (grad, exp_avg, exp_avg_sq)):
        raise ValueError("param, grad, exp_avg and exp_avg_sq must have the same number of elements")
    import torch
    if exp_avg.dtype != torch.float32 or exp_avg_sq.dtype != torch.float32:
        raise ValueError("exp_avg and exp_avg_sq are float32")
    _check_device_tensors("muon_adamw_step", (param, grad, exp_avg, exp_avg_sq))
    return muon_adamw_tensor(param.data_ptr(), grad.data_ptr(), exp_avg.data_ptr(), exp_avg_sq.data_ptr(), n,
                             _dtype_code(param) if _dtype_code(param) == _dtype_code(grad) else -1, 0)


def muon_adamw_step(handle: int, params: Sequence, grads: Sequence, exp_avgs: Sequence, exp_avg_sqs: Sequence,
                    hp: AdamWHparams, stream=None) -> None:
    """One AdamW step over every (param, grad, exp_avg, exp_avg_sq) set, on ``stream``."""
    n = len(params)
    if len(grads) != n or len(exp_avgs) != n or len(exp_avg_sqs) != n:
        raise ValueError("params, grads, exp_avgs and exp_avg_sqs must have the same length")
    arr = (muon_adamw_tensor * max(n, 1))()
    for i in range(n):
        arr[i] = make_adamw_tensor(params[i], grads[i], exp_avgs[i], exp_avg_sqs[i])
    c_hp = hp.to_c()
    _check(handle, load().muon_adamw_step(handle, arr, n, ctypes.byref(c_hp), _stream_ptr(stream)))


def muon_adamw_step_raw(handle: int, arr, n: int, hp: muon_adamw_hparams, stream_ptr: int) -> int:
    """Call with prepared ctypes arguments (the benchmark's inner loop); returns the status."""
    return load().muon_adamw_step(handle, arr, n, ctypes.byref(hp), stream_ptr)


def muon_step_raw(handle: int, arr, n: int, hp: muon_hparams, stream_ptr: int) -> int:
    """Call with prepared ctypes arguments (the benchmark's inner loop); returns the status."""
    return load().muon_step(handle, arr, n, ctypes.byref(hp), stream_ptr)


def muon_orthogonalize(handle: int, inp, out, hp: Hparams, stream=None) -> None:
    """out (float32, inp's shape, same device) = Newton-Schulz(inp)."""
    import torch
    if inp.dim() != 2 or tuple(out.shape) != tuple(inp.shape):
        raise ValueError(f"muon_orthogonalize: out has shape {tuple(out.shape)}, input {tuple(inp.shape)} (2-D)")
    if out.dtype != torch.float32:
        raise ValueError(f"muon_orthogonalize: out must be float32, got {out.dtype}")
    _check_device_tensors("muon_orthogonalize", (inp, out))
    c_hp = hp.to_c()
    st = load().muon_orthogonalize(handle, inp.data_ptr(), out.data_ptr(), int(inp.shape[0]), int(inp.shape[1]),
                                   _ld(inp), _ld(out), _dtype_code(inp), ctypes.byref(c_hp), _stream_ptr(stream))
    _check(handle, st)


# ---- layer operators ----------------------------------------------------------

class Act8:
    """An 8-bit activation checkpoint (``muon_act8``): ``codes`` int8 (rows x
    cols) and ``exponents`` uint8 (rows x ceil(cols / 32)), device tensors with
    unit column stride.  Element (r, c) stands for
    ``codes[r, c] * 2 ** (exponents[r, c // 32] - 127)``."""

    __slots__ = ("codes", "exponents")

    def __init__(self, codes, exponents):
        import torch
        if codes.dtype != torch.int8 or exponents.dtype != torch.uint8:
            raise ValueError(f"Act8: codes must be int8 and exponents uint8, got {codes.dtype} and {exponents.dtype}")
        if codes.dim() != 2 or exponents.dim() != 2:
            raise ValueError("Act8: codes and exponents must be 2-D")
        g = -(-int(codes.shape[1]) // MUON_ACT8_GROUP)
        if tuple(exponents.shape) != (int(codes.shape[0]), g):
            raise ValueError(f"Act8: exponents have shape {tuple(exponents.shape)}, codes {tuple(codes.shape)} need "
                             f"{(int(codes.shape[0]), g)}")
        self.codes = codes
        self.exponents = exponents

    @classmethod
    def empty(cls, rows: int, cols: int, device="cuda") -> "Act8":
        import torch
        return cls(torch.empty(rows, cols, dtype=torch.int8, device=device),
                   torch.empty(rows, -(-cols // MUON_ACT8_GROUP), dtype=torch.uint8, device=device))

    @property
    def shape(self):
        return self.codes.shape

    def _c(self) -> muon_act8:
        return muon_act8(self.codes.data_ptr(), self.exponents.data_ptr(), _ld2(self.codes), _ld2(self.exponents))


_NO_ACT8 = muon_act8()


def _ld2(t) -> int:
    """Leading dimension of a 2-D tensor with unit column stride (a single
    column or row may carry any stride)."""
    if t.dim() != 2:
        raise ValueError("matrices must be 2-D with unit column stride")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("matrices must be 2-D with unit column stride")
    return int(t.stride(0)) if t.shape[0] > 1 else max(int(t.stride(0)), int(t.shape[1]))


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _layer_tensors(what: str, shapes, dtypes):
    """Check named tensors: ``shapes`` (name, tensor or None, expected shape),
    ``dtypes`` groups of (name, tensor or None) that share a storage dtype; all
    on one GPU, which is returned."""
    import torch
    for nm, t, shape in shapes:
        if t is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{what}: {nm} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    for group in dtypes:
        have = [(nm, t) for nm, t in group if t is not None]
        for nm, t in have:
            if t.dtype not in (torch.bfloat16, torch.float32):
                raise ValueError(f"{what}: {nm} must be bfloat16 or float32, got {t.dtype}")
            if t.dtype != have[0][1].dtype:
                raise ValueError(f"{what}: {nm} is {t.dtype}, {have[0][0]} {have[0][1].dtype}")
    flat = []
    for _, t, _ in shapes:
        if isinstance(t, Act8):
            flat += [t.codes, t.exponents]
        elif t is not None:
            flat.append(t)
    for t in flat:
        if t.dim() == 1 and t.numel() > 1 and t.stride(0) != 1:
            raise ValueError(f"{what}: vectors must be contiguous")
    return _check_device_tensors(what, flat)


def _stream_on(stream, device) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return int(stream.cuda_stream)


def _f32_vectors(what: str, **ts):
    import torch
    for nm, t in ts.items():
        if t is not None and t.dtype != torch.float32:
            raise ValueError(f"{what}: {nm} must be float32, got {t.dtype}")


def _code(what: str, table: dict, value: str, name: str) -> int:
    if value not in table:
        raise ValueError(f"{what}: {name} must be one of {sorted(table)}, got {value!r}")
    return table[value]


def muon_layernorm_forward(handle: int, x, gain, bias, y, mean=None, rstd=None, eps: float = 1e-5,
                           y8: Optional[Act8] = None, stream=None) -> None:
    """y = layer norm of x's rows (``bias`` may be None); ``mean``, ``rstd``
    (float32, one per row) and ``y8`` (y's 8-bit checkpoint) are written where given."""
    w = "muon_layernorm_forward"
    if x.dim() != 2:
        raise ValueError(f"{w}: x must be 2-D")
    r, c = (int(v) for v in x.shape)
    _f32_vectors(w, mean=mean, rstd=rstd)
    dev = _layer_tensors(w, [("x", x, (r, c)), ("gain", gain, (c,)), ("bias", bias, (c,)), ("y", y, (r, c)),
                             ("mean", mean, (r,)), ("rstd", rstd, (r,)), ("y8", y8, (r, c))],
                         [[("x", x), ("y", y)], [("gain", gain), ("bias", bias)]])
    a = muon_layernorm_args(x.data_ptr(), gain.data_ptr(), _ptr(bias), y.data_ptr(), _ptr(mean), _ptr(rstd),
                            y8._c() if y8 is not None else _NO_ACT8, r, c, _ld2(x), _ld2(y), _dtype_code(x),
                            _dtype_code(gain), float(eps), 0)
    _check(handle, load().muon_layernorm_forward(handle, ctypes.byref(a), _stream_on(stream, dev)))


def muon_layernorm_backward(handle: int, dy, x, gain, mean, rstd, dx, dgain, dbias=None, add=None,
                            accumulate: bool = False, stream=None) -> None:
    """dx (+ ``add``, which may be ``dx``), dgain and dbias of the layer norm
    from dy; ``accumulate`` adds to dgain and dbias."""
    w = "muon_layernorm_backward"
    if x.dim() != 2:
        raise ValueError(f"{w}: x must be 2-D")
    r, c = (int(v) for v in x.shape)
    _f32_vectors(w, mean=mean, rstd=rstd)
    dev = _layer_tensors(w, [("x", x, (r, c)), ("dy", dy, (r, c)), ("gain", gain, (c,)), ("mean", mean, (r,)),
                             ("rstd", rstd, (r,)), ("dx", dx, (r, c)), ("dgain", dgain, (c,)),
                             ("dbias", dbias, (c,)), ("add", add, (r, c))],
                         [[("x", x), ("dy", dy), ("dx", dx), ("add", add)],
                          [("gain", gain), ("dgain", dgain), ("dbias", dbias)]])
    a = muon_layernorm_grad_args(dy.data_ptr(), x.data_ptr(), gain.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                                 _ptr(add), dx.data_ptr(), dgain.data_ptr(), _ptr(dbias), r, c, _ld2(dy), _ld2(x),
                                 _ld2(add) if add is not None else 0, _ld2(dx), _dtype_code(x), _dtype_code(gain),
                                 int(bool(accumulate)), 0)
    _check(handle, load().muon_layernorm_backward(handle, ctypes.byref(a), _stream_on(stream, dev)))


def _linear_sizes(what: str, w, w_layout: str):
    if w.dim() != 2:
        raise ValueError(f"{what}: the weight must be 2-D")
    _code(what, W_LAYOUTS, w_layout, "w_layout")
    a, b = (int(v) for v in w.shape)
    return (b, a) if w_layout == "out_in" else (a, b)


def muon_linear_forward(handle: int, x, w, y, bias=None, act: str = "none", residual=None, z_out=None,
                        w_layout: str = "in_out", stream=None) -> None:
    """y = act(x W + bias) + residual; ``w`` is (in x out) or, with ``w_layout``
    "out_in", (out x in).  ``residual`` may be ``y``.  ``z_out`` (a tensor or an
    Act8) receives the pre-activation x W + bias."""
    wh = "muon_linear_forward"
    k, n = _linear_sizes(wh, w, w_layout)
    if x.dim() != 2:
        raise ValueError(f"{wh}: x must be 2-D")
    r = int(x.shape[0])
    z8 = z_out if isinstance(z_out, Act8) else None
    z = None if z8 is not None else z_out
    dev = _layer_tensors(wh, [("x", x, (r, k)), ("w", w, w.shape), ("bias", bias, (n,)), ("y", y, (r, n)),
                              ("residual", residual, (r, n)), ("z_out", z_out, (r, n))],
                         [[("x", x), ("w", w), ("y", y), ("residual", residual), ("z_out", z)], [("bias", bias)]])
    a = muon_linear_args(x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(residual), y.data_ptr(), _ptr(z),
                         z8._c() if z8 is not None else _NO_ACT8, r, k, n, _ld2(x), _ld2(w),
                         _ld2(residual) if residual is not None else 0, _ld2(y), _ld2(z) if z is not None else 0,
                         _dtype_code(x), _dtype_code(bias) if bias is not None else MUON_F32,
                         _code(wh, ACTIVATIONS, act, "act"), W_LAYOUTS[w_layout], 0)
    _check(handle, load().muon_linear_forward(handle, ctypes.byref(a), _stream_on(stream, dev)))


def muon_linear_grad_input(handle: int, dy, w, dx, act: str = "none", z=None, act_out=None, add=None,
                           w_layout: str = "in_out", stream=None) -> None:
    """dx = (dy W^T) act'(z) + add: the gradient at the pre-activation ``z`` (a
    tensor or an Act8) behind this layer's input, or at the input itself without
    ``z``.  ``act_out`` receives act(z); ``add`` may be ``dx``."""
    wh = "muon_linear_grad_input"
    k, n = _linear_sizes(wh, w, w_layout)
    if dy.dim() != 2:
        raise ValueError(f"{wh}: dy must be 2-D")
    r = int(dy.shape[0])
    z8 = z if isinstance(z, Act8) else None
    zt = None if z8 is not None else z
    dev = _layer_tensors(wh, [("dy", dy, (r, n)), ("w", w, w.shape), ("dx", dx, (r, k)), ("z", z, (r, k)),
                              ("act_out", act_out, (r, k)), ("add", add, (r, k))],
                         [[("dy", dy), ("w", w), ("dx", dx), ("z", zt), ("act_out", act_out), ("add", add)]])
    a = muon_linear_grad_input_args(dy.data_ptr(), w.data_ptr(), _ptr(zt), z8._c() if z8 is not None else _NO_ACT8,
                                    _ptr(add), dx.data_ptr(), _ptr(act_out), r, k, n, _ld2(dy), _ld2(w),
                                    _ld2(zt) if zt is not None else 0, _ld2(add) if add is not None else 0, _ld2(dx),
                                    _ld2(act_out) if act_out is not None else 0, _dtype_code(dy),
                                    _code(wh, ACTIVATIONS, act, "act"), W_LAYOUTS[w_layout], 0)
    _check(handle, load().muon_linear_grad_input(handle, ctypes.byref(a), _stream_on(stream, dev)))


def muon_linear_grad_weight(handle: int, x, dy, dw, db=None, accumulate: bool = False, w_layout: str = "in_out",
                            stream=None) -> None:
    """dw = x^T dy (stored as the weight is) and db = dy's column sums; ``x`` is
    a tensor or an Act8, ``accumulate`` adds to dw and db."""
    wh = "muon_linear_grad_weight"
    k, n = _linear_sizes(wh, dw, w_layout)
    if dy.dim() != 2:
        raise ValueError(f"{wh}: dy must be 2-D")
    r = int(dy.shape[0])
    x8 = x if isinstance(x, Act8) else None
    xt = None if x8 is not None else x
    dev = _layer_tensors(wh, [("x", x, (r, k)), ("dy", dy, (r, n)), ("dw", dw, dw.shape), ("db", db, (n,))],
                         [[("dy", dy), ("x", xt)], [("dw", dw)], [("db", db)]])
    a = muon_linear_grad_weight_args(_ptr(xt), x8._c() if x8 is not None else _NO_ACT8, dy.data_ptr(), dw.data_ptr(),
                                     _ptr(db), r, k, n, _ld2(xt) if xt is not None else 0, _ld2(dy), _ld2(dw),
                                     _dtype_code(dy), _dtype_code(dw), _dtype_code(db) if db is not None else MUON_F32,
                                     W_LAYOUTS[w_layout], int(bool(accumulate)), 0)
    _check(handle, load().muon_linear_grad_weight(handle, ctypes.byref(a), _stream_on(stream, dev)))


def muon_act_encode(handle: int, x, q: Act8, stream=None) -> None:
    """``q`` = the 8-bit checkpoint of x (2-D, bfloat16 or float32)."""
    w = "muon_act_encode"
    if x.dim() != 2:
        raise ValueError(f"{w}: x must be 2-D")
    dev = _layer_tensors(w, [("x", x, x.shape), ("q", q, x.shape)], [[("x", x)]])
    c = q._c()
    _check(handle, load().muon_act_encode(handle, x.data_ptr(), int(x.shape[0]), int(x.shape[1]), _ld2(x),
                                          _dtype_code(x), ctypes.byref(c), _stream_on(stream, dev)))


def muon_act_decode(handle: int, q: Act8, y, stream=None) -> None:
    """y (bfloat16 or float32) = what the checkpoint ``q`` stands for, exactly."""
    w = "muon_act_decode"
    if y.dim() != 2:
        raise ValueError(f"{w}: y must be 2-D")
    dev = _layer_tensors(w, [("y", y, y.shape), ("q", q, y.shape)], [[("y", y)]])
    c = q._c()
    _check(handle, load().muon_act_decode(handle, ctypes.byref(c), y.data_ptr(), int(y.shape[0]), int(y.shape[1]),
                                          _ld2(y), _dtype_code(y), _stream_on(stream, dev)))


def muon_read_norms(handle: int, n: int, stream=None) -> List[float]:
    buf = (ctypes.c_float * max(n, 1))()
    _check(handle, load().muon_read_norms(handle, buf, int(n), _stream_ptr(stream)))
    return [float(buf[i]) for i in range(n)]


def muon_kernel_stats_read(handle: int) -> dict:
    buf = (muon_kernel_stats * 16)()
    k = load().muon_kernel_stats_read(handle, buf, 16)
    return {buf[i].name.decode(): (int(buf[i].launches), float(buf[i].total_ms)) for i in range(k)}


def muon_kernel_stats_reset(handle: int) -> None:
    load().muon_kernel_stats_reset(handle)


def muon_workspace_bytes(handle: int) -> int:
    return int(load().muon_workspace_bytes(handle))


def muon_destroy(handle: int) -> None:
    _check(None, load().muon_destroy(handle))


def muon_status_str(status: int) -> str:
    return status_str(status)


def muon_last_error(handle: int) -> str:
    return load().muon_last_error(handle).decode()
