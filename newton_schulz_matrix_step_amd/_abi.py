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
        if codes.dtype is not torch.int8 or exponents.dtype is not torch.uint8:
            raise ValueError(f"Act8: codes must be int8 and exponents uint8, got {codes.dtype} and {exponents.dtype}")
        if codes.dim() != 2 or exponents.dim() != 2:
            raise ValueError("Act8: codes and exponents must be 2-D")
        r, c = codes.shape
        want = (r, -(-c // MUON_ACT8_GROUP))
        if exponents.shape != want:
            raise ValueError(f"Act8: exponents have shape {tuple(exponents.shape)}, codes {tuple(codes.shape)} need {want}")
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
        q, e = self.codes, self.exponents
        if q.is_contiguous() and e.is_contiguous():
            c = q.shape[1]
            return muon_act8(q.data_ptr(), e.data_ptr(), c, -(-c // MUON_ACT8_GROUP))
        return muon_act8(q.data_ptr(), e.data_ptr(), _ld2(q), _ld2(e))


_NO_ACT8 = muon_act8()


def _ld2(t) -> int:
    """Leading dimension of a 2-D tensor with unit column stride (a single
    column or row may carry any stride)."""
    if t.dim() != 2:
        raise ValueError("matrices must be 2-D with unit column stride")
    ld, cs = t.stride()
    rows, cols = t.shape
    if cs != 1 and cols > 1:
        raise ValueError("matrices must be 2-D with unit column stride")
    return ld if rows > 1 else max(ld, cols)


class _Torch:
    """What the layer calls need of torch, looked up once."""

    def __init__(self):
        import torch
        self.f32 = torch.float32
        self.codes = {torch.bfloat16: MUON_BF16, torch.float32: MUON_F32}
        self.raw_stream = torch._C._cuda_getCurrentRawStream


_torch: Optional[_Torch] = None


class _Args:
    """Checks of one layer call's tensors (the C ABI sees only pointers and
    sizes) and their marshalling.  The first tensor names the GPU that all
    others must be on.  A contiguous tensor as expected takes the short way
    through each method; the rest of it names what is wrong."""

    __slots__ = ("what", "device", "device_ok", "torch")

    def __init__(self, what: str, t):
        global _torch
        if _torch is None:
            _torch = _Torch()
        self.torch = _torch
        self.what = what
        self.device = t.get_device()   # -1: the host
        self.device_ok = self.device >= 0

    def fail(self, msg: str):
        raise ValueError(f"{self.what}: {msg}")

    def check(self, nm, t, shape, dt, like=None):
        if t.shape != shape:
            self.fail(f"{nm} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if t.dtype is not dt:
            self.fail(f"{nm} is {t.dtype}, {like} {dt}" if like else f"{nm} must be {str(dt)[6:]}, got {t.dtype}")
        if t.get_device() != self.device:
            self.device_ok = False

    def storage(self, nm, t) -> int:
        """muon_dtype of a tensor that may be bfloat16 or float32."""
        c = self.torch.codes.get(t.dtype)
        if c is None:
            self.fail(f"{nm} must be bfloat16 or float32, got {t.dtype}")
        return c

    def matrix(self, nm, t, shape, dt, like):
        """(pointer, leading dimension); (None, 0) for an absent one."""
        if t is None:
            return None, 0
        if t.shape == shape and t.dtype is dt and t.get_device() == self.device and t.is_contiguous():
            return t.data_ptr(), shape[1]
        self.check(nm, t, shape, dt, like)
        return t.data_ptr(), _ld2(t)

    def vector(self, nm, t, n, dt, like=None):
        if t is None:
            return None
        if t.shape == (n,) and t.dtype is dt and t.get_device() == self.device and t.is_contiguous():
            return t.data_ptr()
        self.check(nm, t, (n,), dt, like)
        if n > 1 and t.stride(0) != 1:
            self.fail("vectors must be contiguous")
        return t.data_ptr()

    def act8(self, nm, q, shape):
        if q is None:
            return _NO_ACT8
        if q.codes.shape != shape:
            self.fail(f"{nm} has shape {tuple(q.codes.shape)}, expected {tuple(shape)}")
        if q.codes.get_device() != self.device or q.exponents.get_device() != self.device:
            self.device_ok = False
        return q._c()

    def rows_cols(self, nm, t):
        if t.dim() != 2:
            self.fail(f"{nm} must be 2-D")
        return t.shape

    def stream(self, stream) -> int:
        """The given stream, or the current one of the tensors' GPU.  Called
        last: shapes and dtypes are reported before the device is."""
        if not self.device_ok:
            self.fail("tensors must all be on one GPU")
        return int(stream.cuda_stream) if stream is not None else self.torch.raw_stream(self.device)


def _code(what: str, table: dict, value: str, name: str) -> int:
    if value not in table:
        raise ValueError(f"{what}: {name} must be one of {sorted(table)}, got {value!r}")
    return table[value]


def muon_layernorm_forward(handle: int, x, gain, bias, y, mean=None, rstd=None, eps: float = 1e-5,
                           y8: Optional[Act8] = None, stream=None) -> None:
    """y = layer norm of x's rows (``bias`` may be None); ``mean``, ``rstd``
    (float32, one per row) and ``y8`` (y's 8-bit checkpoint) are written where given."""
    k = _Args("muon_layernorm_forward", x)
    shape = k.rows_cols("x", x)
    r, c = shape
    dt, pdt, f32 = x.dtype, gain.dtype, k.torch.f32
    dc, pc = k.storage("x", x), k.storage("gain", gain)
    px, ldx = k.matrix("x", x, shape, dt, "x")
    py, ldy = k.matrix("y", y, shape, dt, "x")
    a = muon_layernorm_args(px, k.vector("gain", gain, c, pdt), k.vector("bias", bias, c, pdt, "gain"), py,
                            k.vector("mean", mean, r, f32), k.vector("rstd", rstd, r, f32), k.act8("y8", y8, shape),
                            r, c, ldx, ldy, dc, pc, eps, 0)
    _check(handle, load().muon_layernorm_forward(handle, a, k.stream(stream)))


def muon_layernorm_backward(handle: int, dy, x, gain, mean, rstd, dx, dgain, dbias=None, add=None,
                            accumulate: bool = False, stream=None) -> None:
    """dx (+ ``add``, which may be ``dx``), dgain and dbias of the layer norm
    from dy; ``accumulate`` adds to dgain and dbias."""
    k = _Args("muon_layernorm_backward", x)
    shape = k.rows_cols("x", x)
    r, c = shape
    dt, pdt, f32 = x.dtype, gain.dtype, k.torch.f32
    dc, pc = k.storage("x", x), k.storage("gain", gain)
    px, ldx = k.matrix("x", x, shape, dt, "x")
    pdy, lddy = k.matrix("dy", dy, shape, dt, "x")
    pdx, lddx = k.matrix("dx", dx, shape, dt, "x")
    pa, lda = k.matrix("add", add, shape, dt, "x")
    a = muon_layernorm_grad_args(pdy, px, k.vector("gain", gain, c, pdt), k.vector("mean", mean, r, f32),
                                 k.vector("rstd", rstd, r, f32), pa, pdx, k.vector("dgain", dgain, c, pdt, "gain"),
                                 k.vector("dbias", dbias, c, pdt, "gain"), r, c, lddy, ldx, lda, lddx, dc, pc,
                                 1 if accumulate else 0, 0)
    _check(handle, load().muon_layernorm_backward(handle, a, k.stream(stream)))


def _linear_sizes(k: _Args, w, w_layout: str):
    """(in, out, muon_weight_layout) of a weight."""
    a, b = k.rows_cols("the weight", w)
    lay = _code(k.what, W_LAYOUTS, w_layout, "w_layout")
    return (b, a, lay) if lay else (a, b, lay)


def muon_linear_forward(handle: int, x, w, y, bias=None, act: str = "none", residual=None, z_out=None,
                        w_layout: str = "in_out", stream=None) -> None:
    """y = act(x W + bias) + residual; ``w`` is (in x out) or, with ``w_layout``
    "out_in", (out x in).  ``residual`` may be ``y``.  ``z_out`` (a tensor or an
    Act8) receives the pre-activation x W + bias."""
    k = _Args("muon_linear_forward", x)
    i, o, lay = _linear_sizes(k, w, w_layout)
    r = k.rows_cols("x", x)[0]
    dt, dc, ac = x.dtype, k.storage("x", x), _code(k.what, ACTIVATIONS, act, "act")
    z8 = z_out if isinstance(z_out, Act8) else None
    px, ldx = k.matrix("x", x, (r, i), dt, "x")
    pw, ldw = k.matrix("w", w, w.shape, dt, "x")
    py, ldy = k.matrix("y", y, (r, o), dt, "x")
    pr, ldr = k.matrix("residual", residual, (r, o), dt, "x")
    pz, ldz = k.matrix("z_out", None if z8 is not None else z_out, (r, o), dt, "x")
    bc = MUON_F32 if bias is None else k.storage("bias", bias)
    a = muon_linear_args(px, pw, k.vector("bias", bias, o, bias.dtype) if bias is not None else None, pr, py, pz,
                         k.act8("z_out", z8, (r, o)), r, i, o, ldx, ldw, ldr, ldy, ldz, dc, bc, ac, lay, 0)
    _check(handle, load().muon_linear_forward(handle, a, k.stream(stream)))


def muon_linear_grad_input(handle: int, dy, w, dx, act: str = "none", z=None, act_out=None, add=None,
                           w_layout: str = "in_out", stream=None) -> None:
    """dx = (dy W^T) act'(z) + add: the gradient at the pre-activation ``z`` (a
    tensor or an Act8) behind this layer's input, or at the input itself without
    ``z``.  ``act_out`` receives act(z); ``add`` may be ``dx``."""
    k = _Args("muon_linear_grad_input", dy)
    i, o, lay = _linear_sizes(k, w, w_layout)
    r = k.rows_cols("dy", dy)[0]
    dt, dc, ac = dy.dtype, k.storage("dy", dy), _code(k.what, ACTIVATIONS, act, "act")
    z8 = z if isinstance(z, Act8) else None
    pdy, lddy = k.matrix("dy", dy, (r, o), dt, "dy")
    pw, ldw = k.matrix("w", w, w.shape, dt, "dy")
    pdx, lddx = k.matrix("dx", dx, (r, i), dt, "dy")
    pz, ldz = k.matrix("z", None if z8 is not None else z, (r, i), dt, "dy")
    pv, ldv = k.matrix("act_out", act_out, (r, i), dt, "dy")
    pa, lda = k.matrix("add", add, (r, i), dt, "dy")
    a = muon_linear_grad_input_args(pdy, pw, pz, k.act8("z", z8, (r, i)), pa, pdx, pv, r, i, o, lddy, ldw, ldz, lda,
                                    lddx, ldv, dc, ac, lay, 0)
    _check(handle, load().muon_linear_grad_input(handle, a, k.stream(stream)))


def muon_linear_grad_weight(handle: int, x, dy, dw, db=None, accumulate: bool = False, w_layout: str = "in_out",
                            stream=None) -> None:
    """dw = x^T dy (stored as the weight is) and db = dy's column sums; ``x`` is
    a tensor or an Act8, ``accumulate`` adds to dw and db."""
    k = _Args("muon_linear_grad_weight", dy)
    i, o, lay = _linear_sizes(k, dw, w_layout)
    r = k.rows_cols("dy", dy)[0]
    dt, dc, wc = dy.dtype, k.storage("dy", dy), k.storage("dw", dw)
    x8 = x if isinstance(x, Act8) else None
    pdy, lddy = k.matrix("dy", dy, (r, o), dt, "dy")
    px, ldx = k.matrix("x", None if x8 is not None else x, (r, i), dt, "dy")
    pdw, lddw = k.matrix("dw", dw, dw.shape, dw.dtype, "dw")
    bc = MUON_F32 if db is None else k.storage("db", db)
    a = muon_linear_grad_weight_args(px, k.act8("x", x8, (r, i)), pdy, pdw,
                                     k.vector("db", db, o, db.dtype) if db is not None else None, r, i, o, ldx, lddy,
                                     lddw, dc, wc, bc, lay, 1 if accumulate else 0, 0)
    _check(handle, load().muon_linear_grad_weight(handle, a, k.stream(stream)))


def muon_act_encode(handle: int, x, q: Act8, stream=None) -> None:
    """``q`` = the 8-bit checkpoint of x (2-D, bfloat16 or float32)."""
    k = _Args("muon_act_encode", x)
    r, c = k.rows_cols("x", x)
    dc = k.storage("x", x)
    a = k.act8("q", q, x.shape)
    _check(handle, load().muon_act_encode(handle, x.data_ptr(), r, c, _ld2(x), dc, a, k.stream(stream)))


def muon_act_decode(handle: int, q: Act8, y, stream=None) -> None:
    """y (bfloat16 or float32) = what the checkpoint ``q`` stands for, exactly."""
    k = _Args("muon_act_decode", y)
    r, c = k.rows_cols("y", y)
    dc = k.storage("y", y)
    a = k.act8("q", q, y.shape)
    _check(handle, load().muon_act_decode(handle, a, y.data_ptr(), r, c, _ld2(y), dc, k.stream(stream)))


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
