"""learnable_butterfly_rotation_amd -- MI355X (gfx950) learnable butterfly
rotation fused with round-to-nearest group quantization.

Binding over the C ABI of ``libbfly.so`` (include/bfly.h): through ctypes, and
for the norm, the adapters, the clipping and the cache through the native
extension ``_tensors``.  The functions carry the C names; they only check torch tensors
and marshal them into pointers, sizes and the current HIP stream -- every step
of the computation runs in the library's HIP kernels.  There is no CPU fallback: if the library is missing
or no GPU is present the calls raise.

Build the library with ``python -m learnable_butterfly_rotation_amd.build``.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "BflyError", "lib", "library_path", "BFLY_F32", "BFLY_BF16", "BFLY_SYM_ABSMAX",
    "BFLY_ASYM_MINMAX", "bfly_coeff_bytes", "bfly_forward_workspace_bytes", "bfly_prepare",
    "bfly_prepare_hadamard",
    "bfly_forward", "bfly_forward_quant", "bfly_kron_forward", "bfly_kron_forward_wide",
    "bfly_kron_forward_wide_workspace_bytes", "bfly_quant_matmul",
    "bfly_backward", "bfly_backward_workspace_bytes", "bfly_kron_backward",
    "bfly_kron_backward_workspace_bytes", "bfly_calib_config", "bfly_calib_step",
    "bfly_calib_workspace_bytes", "bfly_calib_weight_config", "bfly_calib_step_weight",
    "bfly_calib_step_weight_workspace_bytes", "bfly_status_string",
    "bfly_last_hip_error", "bfly_time_next_forward", "bfly_forward_quant_noalloc",
    "BFLY_Q8_INT8", "BFLY_Q8_E4M3", "bfly_rmsnorm", "bfly_rmsnorm_backward",
    "bfly_rmsnorm_backward_workspace_bytes", "bfly_lora_matmul",
    "bfly_lora_matmul_workspace_bytes", "bfly_grad_clip", "bfly_grad_clip_workspace_bytes",
    "BFLY_KV_BF16", "BFLY_KV_INT8", "BFLY_KV_E4M3", "BFLY_KV_INT4", "bfly_cache_write",
    "bfly_cache_read", "bfly_cache_attention", "bfly_cache_attention_workspace_bytes",
]

BFLY_F32 = 0
BFLY_BF16 = 1
BFLY_SYM_ABSMAX = 0
BFLY_ASYM_MINMAX = 1
BFLY_Q8_INT8 = 0
BFLY_Q8_E4M3 = 1
BFLY_KV_BF16 = 0
BFLY_KV_INT8 = 1
BFLY_KV_E4M3 = 2
BFLY_KV_INT4 = 3

STATUS_NAMES = {0: "BFLY_OK", 1: "BFLY_ERR_NULL", 2: "BFLY_ERR_SIZE", 3: "BFLY_ERR_DTYPE",
                4: "BFLY_ERR_ALIGN", 5: "BFLY_ERR_QUANT", 6: "BFLY_ERR_WORKSPACE",
                7: "BFLY_ERR_UNSUPPORTED", 8: "BFLY_ERR_HIP"}

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libbfly.so")
_lib = None


class BflyError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = "%s: %s (%s)" % (where, STATUS_NAMES.get(status, status), bfly_status_string(status))
        if status == 8:
            msg += ", hipError %d" % bfly_last_hip_error()
        super().__init__(msg)


def lib():
    """The loaded libbfly.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise RuntimeError("libbfly.so is not built: run "
                               "`python -m learnable_butterfly_rotation_amd.build`")
        L = ctypes.CDLL(library_path)
        vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
        L.bfly_coeff_bytes.argtypes = [i32]
        L.bfly_coeff_bytes.restype = sz
        L.bfly_forward_workspace_bytes.argtypes = [i64, i32]
        L.bfly_forward_workspace_bytes.restype = sz
        L.bfly_prepare.argtypes = [vp, i32, vp, sz, vp]
        L.bfly_prepare_hadamard.argtypes = [i32, vp, sz, vp]
        L.bfly_forward.argtypes = [vp, ctypes.c_int, vp, ctypes.c_int, i64, i32, vp, vp, vp, sz,
                                   vp]
        L.bfly_forward_quant.argtypes = [vp, ctypes.c_int, vp, ctypes.c_int, vp, vp, vp, i64, i32,
                                         vp, vp, i32, i32, ctypes.c_int, vp, sz, vp]
        L.bfly_forward_quant_noalloc.argtypes = [vp, ctypes.c_int, vp, ctypes.c_int, vp, vp, vp,
                                                 i64, i32, vp, i32, i32, ctypes.c_int, vp]
        L.bfly_kron_forward.argtypes = [vp, ctypes.c_int, vp, ctypes.c_int, vp, vp, vp, i64, i32,
                                        i32, vp, vp, vp, i32, i32, ctypes.c_int, vp, sz, vp]
        L.bfly_kron_forward_wide.argtypes = [vp, ctypes.c_int, vp, ctypes.c_int, vp, vp, vp, i64,
                                             i32, i32, vp, vp, vp, i32, i32, ctypes.c_int, vp, sz,
                                             vp]
        L.bfly_kron_forward_wide_workspace_bytes.argtypes = [i64, i32, i32]
        L.bfly_kron_forward_wide_workspace_bytes.restype = sz
        L.bfly_quant_matmul.argtypes = [vp, ctypes.c_int, vp, vp, vp, vp, ctypes.c_int, i64, i32,
                                        i32, i32, i32, ctypes.c_int, vp]
        L.bfly_backward.argtypes = [vp, vp, vp, vp, vp, i64, i32, vp, vp, vp, sz, vp]
        L.bfly_backward_workspace_bytes.argtypes = [i64, i32]
        L.bfly_backward_workspace_bytes.restype = sz
        L.bfly_calib_step.argtypes = [vp, i64, i32, vp, vp, vp, i32,
                                      ctypes.POINTER(bfly_calib_config), vp, vp, sz, vp]
        L.bfly_calib_workspace_bytes.argtypes = [i64, i32]
        L.bfly_calib_workspace_bytes.restype = sz
        L.bfly_calib_step_weight.argtypes = [vp, i64, vp, ctypes.c_int, i32, i32, vp, vp, vp, i32,
                                             ctypes.POINTER(bfly_calib_weight_config), vp, vp, sz,
                                             vp]
        L.bfly_calib_step_weight_workspace_bytes.argtypes = [i64, i32, i32]
        L.bfly_calib_step_weight_workspace_bytes.restype = sz
        L.bfly_kron_backward.argtypes = [vp, vp, vp, vp, i64, i32, i32, vp, vp, vp, vp, sz, vp]
        L.bfly_kron_backward_workspace_bytes.argtypes = [i64, i32, i32]
        L.bfly_kron_backward_workspace_bytes.restype = sz
        L.bfly_status_string.argtypes = [ctypes.c_int]
        L.bfly_status_string.restype = ctypes.c_char_p
        L.bfly_last_hip_error.restype = i32
        L.bfly_time_next_forward.argtypes = [vp, vp]
        ci, f32 = ctypes.c_int, ctypes.c_float
        L.bfly_rmsnorm.argtypes = [vp, ci, vp, vp, vp, ci, vp, ci, vp, vp, vp, i64, i32, f32, ci,
                                   i32, vp]
        L.bfly_rmsnorm_backward.argtypes = [vp, ci, vp, ci, vp, vp, vp, vp, ci, vp, i64, i32, vp,
                                            sz, vp]
        L.bfly_rmsnorm_backward_workspace_bytes.argtypes = [i64, i32]
        L.bfly_rmsnorm_backward_workspace_bytes.restype = sz
        L.bfly_lora_matmul.argtypes = [vp, ci, vp, vp, vp, vp, vp, ci, vp, ci, i64, i32, i32, i32,
                                       i32, vp, sz, vp]
        L.bfly_lora_matmul_workspace_bytes.argtypes = [i64, i32, i32, i32]
        L.bfly_lora_matmul_workspace_bytes.restype = sz
        L.bfly_grad_clip.argtypes = [i32, vp, vp, vp, vp, f32, vp, vp, sz, vp]
        L.bfly_grad_clip_workspace_bytes.argtypes = [i32]
        L.bfly_grad_clip_workspace_bytes.restype = sz
        L.bfly_cache_write.argtypes = [vp, i64, vp, i64, ci, vp, i64, vp, vp, vp, vp, i32, i32, i32,
                                       i32, ci, vp]
        L.bfly_cache_read.argtypes = [vp, vp, vp, vp, vp, i64, vp, i64, vp, i64, ci, i32, i32, i32,
                                      i32, ci, vp]
        L.bfly_cache_attention.argtypes = [vp, i64, ci, vp, vp, vp, vp, vp, i32, vp, vp, ci, vp,
                                           i64, i32, i32, i32, i32, i32, ci, f32, i32, i32, vp, sz,
                                           vp]
        L.bfly_cache_attention_workspace_bytes.argtypes = [i64, i32, i32, i32, i32]
        L.bfly_cache_attention_workspace_bytes.restype = sz
        for f in (L.bfly_cache_write, L.bfly_cache_read, L.bfly_cache_attention,
                  L.bfly_rmsnorm, L.bfly_rmsnorm_backward, L.bfly_lora_matmul, L.bfly_grad_clip,
                  L.bfly_prepare, L.bfly_prepare_hadamard, L.bfly_forward, L.bfly_forward_quant,
                  L.bfly_forward_quant_noalloc,
                  L.bfly_kron_forward, L.bfly_kron_forward_wide, L.bfly_quant_matmul,
                  L.bfly_backward,
                  L.bfly_kron_backward, L.bfly_calib_step, L.bfly_calib_step_weight,
                  L.bfly_time_next_forward):
            f.restype = ctypes.c_int
        _lib = L
    return _lib


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

class bfly_calib_config(ctypes.Structure):
    """Settings of bfly_calib_step (include/bfly.h)."""
    _fields_ = [("bits", ctypes.c_int32), ("group", ctypes.c_int32), ("bins", ctypes.c_int32),
                ("lambda_kl", ctypes.c_float), ("lr", ctypes.c_float), ("beta1", ctypes.c_float),
                ("beta2", ctypes.c_float), ("eps", ctypes.c_float)]


class bfly_calib_weight_config(ctypes.Structure):
    """Settings of bfly_calib_step_weight (include/bfly.h)."""
    _fields_ = [("bits", ctypes.c_int32), ("group", ctypes.c_int32), ("mode", ctypes.c_int32),
                ("bins", ctypes.c_int32), ("lambda_kl", ctypes.c_float), ("lr", ctypes.c_float),
                ("beta1", ctypes.c_float), ("beta2", ctypes.c_float), ("eps", ctypes.c_float)]


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _dt(t):
    import torch
    if t.dtype == torch.float32:
        return BFLY_F32
    if t.dtype == torch.bfloat16:
        return BFLY_BF16
    raise TypeError("libbfly takes float32 or bfloat16 rows, got %s" % t.dtype)


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _check(status, where):
    if status != 0:
        raise BflyError(status, where)


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


_extension = _torch = None


def _ext():
    """The extension that takes the tensors of the norm, the adapters, the
    clipping and the cache: it checks that they are contiguous, of the right
    types and shapes and on one GPU, or raises, and gives the library's status."""
    global _extension, _torch
    if _extension is None:
        import importlib
        import torch  # before the extension, which needs its libraries loaded
        try:
            ext = importlib.import_module("._tensors", __name__)
        except ImportError as e:
            raise RuntimeError("the _tensors extension is not built: run "
                               "`python -m learnable_butterfly_rotation_amd.build`") from e
        L = lib()
        ext.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            L.bfly_rmsnorm, L.bfly_rmsnorm_backward, L.bfly_lora_matmul, L.bfly_grad_clip)))
        ext.bind_cache(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            L.bfly_cache_write, L.bfly_cache_read, L.bfly_cache_attention)))
        _torch, _extension = torch, ext
    return _extension


def _call(f, like, stream, *args):
    """The extension's f on a stream: the caller's, or torch's current one of
    the GPU of the tensor `like`, which is made current for the call."""
    device = like.get_device()
    if device < 0:
        raise ValueError("bfly_%s: the tensors have to be on a GPU" % f.__name__)
    if stream is None:
        stream = _torch._C._cuda_getCurrentRawStream(device)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if _torch._C._cuda_getDevice() != device:
        with _torch.cuda.device(device):
            status = f(stream, device, *args)
    else:
        status = f(stream, device, *args)
    if status != 0:
        raise BflyError(status, "bfly_" + f.__name__)


def _scratch(nbytes, like, stream):
    """A uint8 tensor on the GPU of `like` for a call on `stream`, of that
    stream's memory: what used it before and what will use it afterwards is
    then in order with the call, which the current stream's memory, where a
    block is reused as soon as its tensor is gone, would not be."""
    import torch
    if stream is None or like.get_device() < 0:  # the call refuses tensors of the host
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    if isinstance(stream, int):
        stream = (torch.cuda.ExternalStream(stream, device=like.device) if stream
                  else torch.cuda.default_stream(like.device))
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device)


def _table_ws(n, theta, coeffs, workspace, like, stream):
    """The workspace of a forward call: the caller's, or -- when the call
    needs one (angles without a table; n = 8192 always) and none is given --
    a fresh uint8 tensor of bfly_forward_workspace_bytes(rows, n) from
    torch's allocator on the device of `like` (torch supplies the device
    memory; the library allocates none), of the call's stream."""
    if workspace is not None or (n != 8192 and (coeffs is not None or theta is None)):
        return workspace
    return _scratch(max(1, bfly_forward_workspace_bytes(like.shape[0], n)), like, stream)


# ---------------------------------------------------------------------------
# the C ABI, one function per entry point
# ---------------------------------------------------------------------------

def bfly_coeff_bytes(n: int) -> int:
    return lib().bfly_coeff_bytes(n)


def bfly_forward_workspace_bytes(rows: int, n: int) -> int:
    return lib().bfly_forward_workspace_bytes(rows, n)


def bfly_prepare(theta, n: int, coeffs, stream=None) -> None:
    """coeffs (uint8 tensor of >= bfly_coeff_bytes(n) bytes) <- table of theta."""
    _check(lib().bfly_prepare(_ptr(theta), n, _ptr(coeffs), coeffs.numel() * coeffs.element_size(),
                              _stream(stream)), "bfly_prepare")


def bfly_prepare_hadamard(n: int, coeffs, stream=None) -> None:
    """coeffs <- table of H_n = Q(pi/4) D, the orthonormal Walsh-Hadamard matrix."""
    _check(lib().bfly_prepare_hadamard(n, _ptr(coeffs), coeffs.numel() * coeffs.element_size(),
                                       _stream(stream)), "bfly_prepare_hadamard")


def bfly_forward(x, y, theta=None, coeffs=None, workspace=None, stream=None) -> None:
    """y[r] = Q(theta) x[r]; x, y: [rows, n] float32/bfloat16 on the GPU."""
    rows, n = x.shape
    ws = _table_ws(n, theta, coeffs, workspace, x, stream)
    _check(lib().bfly_forward(_ptr(x), _dt(x), _ptr(y), _dt(y), rows, n, _ptr(theta),
                              _ptr(coeffs), _ptr(ws), _nbytes(ws), _stream(stream)),
           "bfly_forward")


def bfly_forward_quant(x, y, codes, scales, zeros=None, theta=None, coeffs=None, bits=4,
                       group=128, mode=BFLY_SYM_ABSMAX, workspace=None, stream=None) -> None:
    """Forward fused with per-group RTN quantization (y may be None)."""
    rows, n = x.shape
    ws = _table_ws(n, theta, coeffs, workspace, x, stream)
    _check(lib().bfly_forward_quant(_ptr(x), _dt(x), _ptr(y), _dt(y) if y is not None else 0,
                                    _ptr(codes), _ptr(scales), _ptr(zeros), rows, n, _ptr(theta),
                                    _ptr(coeffs), bits, group, mode, _ptr(ws), _nbytes(ws),
                                    _stream(stream)),
           "bfly_forward_quant")


def bfly_forward_quant_noalloc(x, y, codes, scales, zeros=None, theta=None, bits=4, group=128,
                               mode=BFLY_SYM_ABSMAX, stream=None) -> None:
    """bfly_forward_quant from angles, its table in the library's fixed
    per-device scratch (no allocation; overlapping calls on one device race)."""
    rows, n = x.shape
    _check(lib().bfly_forward_quant_noalloc(_ptr(x), _dt(x), _ptr(y),
                                            _dt(y) if y is not None else 0, _ptr(codes),
                                            _ptr(scales), _ptr(zeros), rows, n, _ptr(theta), bits,
                                            group, mode, _stream(stream)),
           "bfly_forward_quant_noalloc")


def bfly_kron_forward(x, y, mix, codes=None, scales=None, zeros=None, theta_b=None, coeffs_b=None,
                      bits=4, group=128, mode=BFLY_SYM_ABSMAX, workspace=None, stream=None) -> None:
    """(O kron B) on rows of n = m * nb; mix: [m, m] float32 on the GPU."""
    rows, n = x.shape
    m = mix.shape[0]
    ws = _table_ws(n // m, theta_b, coeffs_b, workspace, x, stream)
    _check(lib().bfly_kron_forward(_ptr(x), _dt(x), _ptr(y), _dt(y) if y is not None else 0,
                                   _ptr(codes), _ptr(scales), _ptr(zeros), rows, m, n // m,
                                   _ptr(theta_b), _ptr(coeffs_b), _ptr(mix), bits, group, mode,
                                   _ptr(ws), _nbytes(ws), _stream(stream)), "bfly_kron_forward")


def bfly_kron_forward_wide_workspace_bytes(rows: int, m: int, nb: int) -> int:
    return lib().bfly_kron_forward_wide_workspace_bytes(rows, m, nb)


def bfly_kron_forward_wide(x, y, mix, workspace, codes=None, scales=None, zeros=None,
                           theta_b=None, coeffs_b=None, bits=4, group=128,
                           mode=BFLY_SYM_ABSMAX, stream=None) -> None:
    """(O kron B) on rows of n = m * nb for m up to 64 (`workspace`: a uint8
    tensor of bfly_kron_forward_wide_workspace_bytes; bf16 rows with nb = 256
    run in one pass, others in two through the workspace)."""
    rows, n = x.shape
    m = mix.shape[0]
    _check(lib().bfly_kron_forward_wide(
        _ptr(x), _dt(x), _ptr(y), _dt(y) if y is not None else 0, _ptr(codes), _ptr(scales),
        _ptr(zeros), rows, m, n // m, _ptr(theta_b), _ptr(coeffs_b), _ptr(mix), bits, group, mode,
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)),
        "bfly_kron_forward_wide")


def bfly_quant_matmul(a, codes, scales, zeros, y, bits=2, group=128, mode=BFLY_ASYM_MINMAX,
                      stream=None) -> None:
    """y = a w^T with w's rows as group codes; a: [rows, k] bfloat16, codes:
    uint8 [n_out, k*bits/8], scales/zeros: float16 [n_out, k/group]."""
    rows, k = a.shape
    n_out = codes.shape[0]
    _check(lib().bfly_quant_matmul(_ptr(a), _dt(a), _ptr(codes), _ptr(scales), _ptr(zeros),
                                   _ptr(y), _dt(y), rows, n_out, k, bits, group, mode,
                                   _stream(stream)), "bfly_quant_matmul")


def bfly_backward_workspace_bytes(rows: int, n: int) -> int:
    return lib().bfly_backward_workspace_bytes(rows, n)


def bfly_backward(x, g, y, dx, dtheta, workspace, theta=None, coeffs=None, stream=None) -> None:
    """y = Q x (optional), dx = Q^T g, dtheta = sum over rows of dL/dtheta."""
    rows, n = x.shape
    _check(lib().bfly_backward(_ptr(x), _ptr(g), _ptr(y), _ptr(dx), _ptr(dtheta), rows, n,
                               _ptr(theta), _ptr(coeffs), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream(stream)),
           "bfly_backward")


def bfly_status_string(status: int) -> str:
    return lib().bfly_status_string(status).decode()


def bfly_last_hip_error() -> int:
    return lib().bfly_last_hip_error()


def bfly_time_next_forward(start_event: int, stop_event: int) -> None:
    """Attach two caller-owned hipEvent_t handles (timing enabled) to the
    next fused forward-kernel dispatch, for kernel-only timing."""
    _check(lib().bfly_time_next_forward(start_event, stop_event), "bfly_time_next_forward")


def bfly_kron_backward_workspace_bytes(rows: int, m: int, nb: int) -> int:
    return lib().bfly_kron_backward_workspace_bytes(rows, m, nb)


def bfly_kron_backward(x, g, dx, dtheta_b, mix, workspace, theta_b=None, coeffs_b=None,
                       stream=None) -> None:
    """dx = (O kron B)^T g and dtheta_b (summed over rows and segments);
    x, g, dx: [rows, m*nb] float32; mix: [m, m] float32 on the GPU."""
    rows, n = x.shape
    m = mix.shape[0]
    _check(lib().bfly_kron_backward(_ptr(x), _ptr(g), _ptr(dx), _ptr(dtheta_b), rows, m, n // m,
                                    _ptr(theta_b), _ptr(coeffs_b), _ptr(mix), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(),
                                    _stream(stream)), "bfly_kron_backward")


def bfly_calib_workspace_bytes(rows: int, n: int) -> int:
    return lib().bfly_calib_workspace_bytes(rows, n)


def bfly_calib_step(x, theta, adam_m, adam_v, step: int, cfg: bfly_calib_config, loss, workspace,
                    stream=None) -> None:
    """One calibration step on rows x ([rows, n] float32): theta, adam_m,
    adam_v ([log2 n, n/2] float32) updated in place; loss [3] float32."""
    rows, n = x.shape
    _check(lib().bfly_calib_step(_ptr(x), rows, n, _ptr(theta), _ptr(adam_m), _ptr(adam_v), step,
                                 ctypes.byref(cfg), _ptr(loss), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream)),
           "bfly_calib_step")


def bfly_calib_step_weight_workspace_bytes(rows: int, out: int, n: int) -> int:
    return lib().bfly_calib_step_weight_workspace_bytes(rows, out, n)


def bfly_calib_step_weight(x, w, theta, adam_m, adam_v, step: int, cfg: bfly_calib_weight_config,
                           loss, workspace, stream=None) -> None:
    """One calibration step with the layer-output loss: x [rows, n] float32,
    w [out, n] float32/bfloat16; theta, adam_m, adam_v updated in place."""
    rows, n = x.shape
    out = w.shape[0]
    _check(lib().bfly_calib_step_weight(_ptr(x), rows, _ptr(w), _dt(w), out, n, _ptr(theta),
                                        _ptr(adam_m), _ptr(adam_v), step, ctypes.byref(cfg),
                                        _ptr(loss), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(),
                                        _stream(stream)), "bfly_calib_step_weight")


# ---------------------------------------------------------------------------
# the norm in front of a layer, adapters beside its product, clipping
# ---------------------------------------------------------------------------

def bfly_rmsnorm(x, weight, eps, y=None, codes=None, scales=None, residual=None, h=None, rstd=None,
                 format=BFLY_Q8_INT8, group=None, stream=None) -> None:
    """h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight per row, and y
    in 8 bits.  x, residual, h: [rows, n] of one type; y: [rows, n] float32 or
    bfloat16; codes: [rows, n] uint8 (or int8 for BFLY_Q8_INT8, float8_e4m3fn
    for BFLY_Q8_E4M3) with scales [rows, n/group] float16 (group None: one
    scale per row); rstd: [rows] float32; weight: [n] or None (ones).  Outputs
    that are None are not computed."""
    _call(_ext().rmsnorm, x, stream, eps, format, group, x, weight, y, codes, scales, residual, h,
          rstd)


def bfly_rmsnorm_backward_workspace_bytes(rows: int, n: int) -> int:
    return lib().bfly_rmsnorm_backward_workspace_bytes(rows, n)


def bfly_rmsnorm_backward(h, weight, rstd, dy, dx, dweight=None, dh=None, workspace=None,
                          stream=None) -> None:
    """dx = dh + dL/dh of y = h rstd weight, dweight = sum over rows of its
    gradient.  h: [rows, n]; dy, dh, dx: [rows, n] of one type; rstd: [rows]
    and dweight: [n] float32; workspace: a uint8 tensor of
    bfly_rmsnorm_backward_workspace_bytes (needed with dweight)."""
    _call(_ext().rmsnorm_backward, h, stream, h, weight, rstd, dy, dx, dweight, dh, workspace)


def bfly_lora_matmul_workspace_bytes(rows: int, n_out: int, k: int, rank: int) -> int:
    return lib().bfly_lora_matmul_workspace_bytes(rows, n_out, k, rank)


def bfly_lora_matmul(x, ids, lora_a, lora_b, scaling, y, workspace, base=None,
                     stream=None) -> None:
    """y = base + scaling[id] * lora_b[id] (lora_a[id] x) per row, id = ids[row]
    (outside [0, adapters): y = base).  x: [rows, k] bfloat16; ids: [rows]
    int32; lora_a: [adapters, rank, k], lora_b: [adapters, n_out, rank]
    bfloat16; scaling: [adapters] float32; base, y: [rows, n_out] float32 or
    bfloat16 (base None: zeros; y may be base); workspace: a uint8 tensor of
    bfly_lora_matmul_workspace_bytes."""
    _call(_ext().lora_matmul, x, stream, x, lora_a, y, ids, lora_b, scaling, base, workspace)


def bfly_grad_clip_workspace_bytes(count: int) -> int:
    return lib().bfly_grad_clip_workspace_bytes(count)


def bfly_grad_clip(grads, max_norm, norm, workspace, outs=None, stream=None) -> None:
    """norm[0] = the 2-norm over all tensors of `grads` (a list; contiguous
    float32 or bfloat16 of any shape), norm[1] = min(1, max_norm / norm[0]),
    and every gradient times norm[1], in place or into `outs`.  norm: [2]
    float32; workspace: a uint8 tensor of bfly_grad_clip_workspace_bytes.  No
    two of the tensors that are written may overlap, nor an output a gradient
    other than its own."""
    _call(_ext().grad_clip, norm, stream, max_norm, norm, workspace, grads, outs)


# ---------------------------------------------------------------------------
# a paged key-value cache in few bits
# ---------------------------------------------------------------------------

def bfly_cache_write(k, v, slots, k_cache, v_cache, k_scales=None, v_scales=None,
                     stream=None) -> None:
    """The keys and values of tokens into their slots (page * page_size +
    place; outside the cache: left out) of a paged cache, quantized.  k, v:
    [tokens, kv_heads, head_dim] of one type, float32 or bfloat16, a token's
    heads contiguous (views into a projection's output are taken as they are);
    slots: [tokens] int32; k_cache, v_cache: [pages, kv_heads, page_size,
    head_dim] bfloat16, int8 or float8_e4m3fn, or uint8 [..., head_dim / 2] for
    two 4-bit codes to a byte; k_scales, v_scales: [pages, kv_heads, page_size]
    float16 (None for bfloat16)."""
    _call(_ext().cache_write, k, stream, k_cache, v_cache, k_scales, v_scales, k, v, slots)


def bfly_cache_read(k_cache, v_cache, slots, k, v, k_scales=None, v_scales=None,
                    stream=None) -> None:
    """k, v <- what the given slots of a cache hold (zeros for a slot outside
    it); the tensors as in bfly_cache_write."""
    _call(_ext().cache_read, k, stream, k_cache, v_cache, k_scales, v_scales, k, v, slots)


def bfly_cache_attention_workspace_bytes(rows: int, heads: int, kv_heads: int, head_dim: int,
                                         max_len: int) -> int:
    """Never falls with rows, heads, head_dim or max_len while kv_heads stays;
    layers that differ in kv_heads take the largest of their sizes."""
    return lib().bfly_cache_attention_workspace_bytes(rows, heads, kv_heads, head_dim, max_len)


def bfly_cache_attention(q, k_cache, v_cache, tables, lens, y, k_scales=None, v_scales=None,
                         scale=None, max_len=None, window=0, lse=None, workspace=None,
                         stream=None) -> None:
    """y = sum_t softmax_t(scale * q . k_t) v_t for one new token per sequence
    over the tokens of a paged cache.  q: [rows, heads, head_dim] float32 or
    bfloat16, a row's heads contiguous; the cache as in bfly_cache_write;
    tables: [rows, width] int32 pages; lens: [rows] int32 tokens (0: y = 0); y:
    [rows, heads, head_dim] float32 or bfloat16; scale None: head_dim ** -0.5;
    max_len: a bound of the lengths (None: what the tables can hold); window:
    only the last so many tokens (0: all); lse: [rows, heads] float32 or None,
    the logarithm of the weights' sum; workspace: a uint8 tensor of
    bfly_cache_attention_workspace_bytes (None: a fresh one)."""
    if workspace is None:
        reach = tables.shape[1] * k_cache.shape[2] if max_len is None else max_len
        nbytes = bfly_cache_attention_workspace_bytes(q.shape[0], q.shape[1], k_cache.shape[1],
                                                      q.shape[2], reach)
        if nbytes:
            workspace = _scratch(nbytes, q, stream)
    _call(_ext().cache_attention, q, stream, scale, max_len, window, k_cache, v_cache, k_scales,
          v_scales, q, tables, lens, y, lse, workspace)
