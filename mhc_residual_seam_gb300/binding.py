"""ctypes binding of libmhcseam (include/mhc_seam.h): argument marshalling only.

Every function has the name of its C entry point and takes torch tensors
(device memory) plus plain numbers; it passes ``data_ptr()`` values and the
CUDA stream handle through, and raises ``MhcError`` on a non-zero status.
There is no fallback: if the library cannot be built or loaded, the first call
raises.
"""
from __future__ import annotations

import ctypes as C
import os
import re

from . import build as _build

MHC_OUT_BF16 = 0
MHC_OUT_MXFP8 = 1
MHC_OUT_FP8_GRID = 2
MHC_DT_BF16, MHC_DT_F16, MHC_DT_F32 = 0, 1, 2
MHC_GATE_NONE, MHC_GATE_CHANNEL, MHC_GATE_TOKEN = 0, 1, 2
MHC_SCORE_SOFTMAX, MHC_SCORE_SIGMOID = 0, 1
MHC_ACT_SILU, MHC_ACT_GELU, MHC_ACT_GELU_TANH, MHC_ACT_RELU = 0, 1, 2, 3
STATUS_NAMES = {
    0: "MHC_OK", -1: "MHC_ERR_NULL", -2: "MHC_ERR_SHAPE", -3: "MHC_ERR_ALIGN", -4: "MHC_ERR_INCOMPLETE_POST",
    -5: "MHC_ERR_WORKSPACE", -6: "MHC_ERR_CAPTURE", -7: "MHC_ERR_TIMEOUT", -8: "MHC_ERR_CUDA", -9: "MHC_ERR_ALIAS",
    -10: "MHC_ERR_CONFIG",
}

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mhc_seam.h")


class MhcError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(code, code)}: {msg}")
        self.code = code


class MhcConfig(C.Structure):
    """mhc_config: zero in a field means the policy decides."""
    _fields_ = [("path", C.c_int), ("block_m", C.c_int), ("cols_per_cta", C.c_int), ("sinkhorn_iters", C.c_int),
                ("amax_floor", C.c_float), ("spin_limit", C.c_longlong), ("projection", C.c_int),
                ("wave_split", C.c_int)]


_lib = None


def lib():
    """Load (building first if needed) the in-tree libmhcseam.so."""
    global _lib
    if _lib is None:
        path = _build.build()
        L = C.CDLL(path)
        P, I64, I = C.c_void_p, C.c_int64, C.c_int
        L.mhc_workspace_bytes.restype = C.c_size_t
        L.mhc_workspace_bytes.argtypes = [I64, I, P]
        L.mhc_workspace_bytes_unshifted.restype = C.c_size_t
        L.mhc_workspace_bytes_unshifted.argtypes = [I64, I, P]
        L.mhc_workspace_init.restype = I
        L.mhc_workspace_init.argtypes = [P, C.c_size_t, P]
        L.mhc_check_status.restype = I
        L.mhc_check_status.argtypes = [P, P]
        L.mhc_packed_fn_bytes.restype = C.c_size_t
        L.mhc_packed_fn_bytes.argtypes = [I]
        L.mhc_pack_fn.restype = I
        L.mhc_pack_fn.argtypes = [P, P, I, P]
        L.mhc_seam.restype = I
        L.mhc_seam.argtypes = [P] * 10 + [C.c_float, I64, I, I] + [P] * 7 + [P, C.c_size_t, P, P]
        L.mhc_seam_unshifted.restype = I
        L.mhc_seam_unshifted.argtypes = [P] * 8 + [C.c_float, I64, I] + [P] * 6 + [C.c_size_t, P, P]
        L.mhc_seam_noalloc.restype = I
        L.mhc_seam_noalloc.argtypes = [P] * 9 + [C.c_float, I64, I, I] + [P] * 7 + [P, P]
        L.mhc_noalloc_check_status.restype = I
        L.mhc_noalloc_check_status.argtypes = [P]
        L.mhc_quant_ue8m0.restype = I
        L.mhc_quant_ue8m0.argtypes = [P, I64, I, C.c_float, P, P, P]
        L.mhc_copy.restype = I
        L.mhc_copy.argtypes = [P, P, C.c_size_t, P]
        F, SZ = C.c_float, C.c_size_t
        L.mhc_embed.restype = I
        L.mhc_embed.argtypes = [P, I, P, I64, I64, I64, F, I64, I, I, I, P, P]
        L.mhc_embed_grad_workspace_bytes.restype = SZ
        L.mhc_embed_grad_workspace_bytes.argtypes = [I64, I64, I]
        L.mhc_embed_grad.restype = I
        L.mhc_embed_grad.argtypes = [P, I, P, I, F, I64, I, I, I64, I64, P, I, P, I, I64, P, SZ, P]
        L.mhc_block_norm.restype = I
        L.mhc_block_norm.argtypes = [P, I64, P, I64, P, P, I, P, F, F, I64, I, I, P, I64, P, I64, P, P, P]
        L.mhc_block_norm_grad_workspace_bytes.restype = SZ
        L.mhc_block_norm_grad_workspace_bytes.argtypes = [I64, I]
        L.mhc_block_norm_grad.restype = I
        L.mhc_block_norm_grad.argtypes = [P] * 6 + [I, P, P, P, F, I64, I, I] + [P] * 6 + [SZ, P]
        L.mhc_route_workspace_bytes.restype = SZ
        L.mhc_route_workspace_bytes.argtypes = [I]
        L.mhc_route.restype = I
        L.mhc_route.argtypes = [P, I64, I, P, I, I, I, I, I, I, F, I64, P, P, P, P, SZ, P]
        L.mhc_route_grad.restype = I
        L.mhc_route_grad.argtypes = [P, P, I64, I, P, I, I, I, I, F, I64, P, I64, P]
        L.mhc_glu_workspace_bytes.restype = SZ
        L.mhc_glu_workspace_bytes.argtypes = [I64, I, I]
        L.mhc_glu.restype = I
        L.mhc_glu.argtypes = [P, I64, P, P, I64, I, I64, I, I, I, P, P, I64, P, SZ, P]
        L.mhc_glu_grad.restype = I
        L.mhc_glu_grad.argtypes = [P, P, P, I64, P, I, I64, I, I, I, P, P, P, I, I, P, SZ, P]
        L.mhc_lora_workspace_bytes.restype = SZ
        L.mhc_lora_workspace_bytes.argtypes = [I64, I]
        L.mhc_lora.restype = I
        L.mhc_lora.argtypes = [P, I64, P, P, P, P, I64, I, I, I, I, I, P, I64, P, I64, P, SZ, P]
        L.mhc_dropout.restype = I
        L.mhc_dropout.argtypes = [P, I64, P, I64, C.c_double, P, I64, I, I, P, I64, P]
        L.mhc_last_launch_count.restype = I
        L.mhc_last_launch_count.argtypes = []
        L.mhc_last_wave_parts.restype = I
        L.mhc_last_wave_parts.argtypes = []
        L.mhc_last_error_string.restype = C.c_char_p
        L.mhc_last_error_string.argtypes = []
        _lib = L
    return _lib


def header_functions() -> list[str]:
    """Names of the entry points the C header declares."""
    src = open(HEADER).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(mhc_[a-z0-9_]+)\s*\(", src)))


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int):
    if rc != 0:
        raise MhcError(rc, lib().mhc_last_error_string().decode())


def _cfg(cfg):
    if cfg is None:
        return None
    if isinstance(cfg, dict):
        cfg = MhcConfig(**cfg)
    return C.byref(cfg)


def mhc_workspace_bytes(T: int, H: int, cfg=None) -> int:
    return int(lib().mhc_workspace_bytes(int(T), int(H), _cfg(cfg)))


def mhc_workspace_init(ws, stream=None) -> None:
    _check(lib().mhc_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def mhc_check_status(ws, stream=None) -> None:
    _check(lib().mhc_check_status(_ptr(ws), _stream(stream)))


def mhc_packed_fn_bytes(H: int) -> int:
    return int(lib().mhc_packed_fn_bytes(int(H)))


def mhc_pack_fn(fn, fn_packed, stream=None) -> None:
    H = fn.shape[0] // 4
    _check(lib().mhc_pack_fn(_ptr(fn), _ptr(fn_packed), H, _stream(stream)))


def mhc_seam(R, Y, post_prev, comb_prev, pre_prev, fn, fn_packed, bias, alpha, gamma, eps: float, out_mode: int,
             residual_out, norm, fp8_codes, e8m0_scales, pre_out, post_out, comb_out, workspace, cfg=None,
             stream=None, T: int | None = None, H: int | None = None) -> None:
    """One seam call; T and H default to R's shape [T, 4, H]."""
    if T is None:
        T = R.shape[0]
    if H is None:
        H = R.shape[-1]
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().mhc_seam(_ptr(R), _ptr(Y), _ptr(post_prev), _ptr(comb_prev), _ptr(pre_prev), _ptr(fn),
                          _ptr(fn_packed), _ptr(bias), _ptr(alpha), _ptr(gamma), float(eps), int(T), int(H),
                          int(out_mode), _ptr(residual_out), _ptr(norm), _ptr(fp8_codes), _ptr(e8m0_scales),
                          _ptr(pre_out), _ptr(post_out), _ptr(comb_out), _ptr(workspace), ws_bytes, _cfg(cfg),
                          _stream(stream)))


def mhc_seam_unshifted(R, Y, post_prev, comb_prev, fn, fn_packed, bias, alpha, eps: float, residual_out, x_out,
                       pre_out, post_out, comb_out, workspace, cfg=None, stream=None, T: int | None = None,
                       H: int | None = None) -> None:
    """One seam call in the unshifted ordering (x with the fresh pre, no norm);
    T and H default to R's shape [T, 4, H]."""
    if T is None:
        T = R.shape[0]
    if H is None:
        H = R.shape[-1]
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().mhc_seam_unshifted(_ptr(R), _ptr(Y), _ptr(post_prev), _ptr(comb_prev), _ptr(fn), _ptr(fn_packed),
                                    _ptr(bias),
                                    _ptr(alpha), float(eps), int(T), int(H), _ptr(residual_out), _ptr(x_out),
                                    _ptr(pre_out), _ptr(post_out), _ptr(comb_out), _ptr(workspace), ws_bytes,
                                    _cfg(cfg), _stream(stream)))


def mhc_workspace_bytes_unshifted(T: int, H: int, cfg=None) -> int:
    return int(lib().mhc_workspace_bytes_unshifted(int(T), int(H), _cfg(cfg)))


def mhc_seam_noalloc(R, Y, post_prev, comb_prev, pre_prev, fn, bias, alpha, gamma, eps: float, out_mode: int,
                     residual_out, norm, fp8_codes, e8m0_scales, pre_out, post_out, comb_out, cfg=None,
                     stream=None, T: int | None = None, H: int | None = None) -> None:
    """mhc_seam on the split path with the library's own static scratch, for
    callers that cannot allocate device memory (no workspace argument)."""
    if T is None:
        T = R.shape[0]
    if H is None:
        H = R.shape[-1]
    _check(lib().mhc_seam_noalloc(_ptr(R), _ptr(Y), _ptr(post_prev), _ptr(comb_prev), _ptr(pre_prev), _ptr(fn),
                                  _ptr(bias), _ptr(alpha), _ptr(gamma), float(eps), int(T), int(H), int(out_mode),
                                  _ptr(residual_out), _ptr(norm), _ptr(fp8_codes), _ptr(e8m0_scales),
                                  _ptr(pre_out), _ptr(post_out), _ptr(comb_out), _cfg(cfg), _stream(stream)))


def mhc_noalloc_check_status(stream=None) -> None:
    _check(lib().mhc_noalloc_check_status(_stream(stream)))


def mhc_quant_ue8m0(x, codes, scales, amax_floor: float = 0.0, stream=None) -> None:
    rows, H = x.shape
    _check(lib().mhc_quant_ue8m0(_ptr(x), rows, H, float(amax_floor), _ptr(codes), _ptr(scales), _stream(stream)))


def mhc_copy(src, dst, nbytes: int | None = None, stream=None) -> None:
    if nbytes is None:
        nbytes = src.numel() * src.element_size()
    _check(lib().mhc_copy(_ptr(src), _ptr(dst), int(nbytes), _stream(stream)))


def mhc_last_launch_count() -> int:
    return int(lib().mhc_last_launch_count())


def mhc_last_wave_parts() -> int:
    return int(lib().mhc_last_wave_parts())


def mhc_last_error_string() -> str:
    return lib().mhc_last_error_string().decode()


# ------------------------------------------- the operators around the seam --
# Pointers carry no type or shape, so these functions check the tensors'
# before they pass the pointers on (MHC_ERR_CONFIG for a type or a tensor that is
# not on the GPU, MHC_ERR_SHAPE for a shape or a stride).  They are written to cost
# a few microseconds of Python per call: messages are put together only for a
# refusal.
_DTYPES: dict = {}
_F32 = _I32 = _I64 = _U64 = _raw_stream = _device = None


def _ops():
    """The library, with this section's constants and the stream lookup set up."""
    global _F32, _I32, _I64, _U64, _raw_stream, _device
    if _F32 is None:
        import torch
        _DTYPES.update({torch.bfloat16: MHC_DT_BF16, torch.float16: MHC_DT_F16, torch.float32: MHC_DT_F32})
        # the current stream's handle without a Stream object around it
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _device = getattr(torch._C, "_cuda_getDevice", None)
        _I64, _U64 = torch.int64, torch.uint64
        _F32, _I32 = torch.float32, torch.int32
    return lib()


def _where(stream):
    if stream is None and _raw_stream is not None and _device is not None:
        return _raw_stream(_device())
    return _stream(stream)


def _refuse(t, name: str, want: str, dtype=None):
    if not t.is_cuda:
        raise MhcError(-10, f"{name} is not on the GPU")
    if dtype is not None and t.dtype != dtype:
        raise MhcError(-10, f"{name} must be {dtype}, not {t.dtype}")
    raise MhcError(-2, f"{name} must be {want}, not {tuple(t.shape)} with strides {t.stride()}")


def _dtype(t, name: str) -> int:
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise MhcError(-10, f"{name} is {t.dtype}, not bf16, fp16 or fp32")
    return d


def _dense(t, shape, dtype, name: str):
    """The address of ``t``, a dense tensor of this shape and type, or None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        _refuse(t, name, f"dense, of shape {shape}", dtype)
    return t.data_ptr()


def _vec(t, n: int, dtype, name: str):
    """The address of ``t``, a dense vector of n elements of this type, or None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.dim() != 1 or t.numel() != n or not t.is_cuda or not t.is_contiguous():
        _refuse(t, name, f"a dense vector of {n}", dtype)
    return t.data_ptr()


def _pitch(t, T: int, H: int, dtype, name: str) -> int:
    """The row stride of a [T, H] matrix with dense rows (H for None)."""
    if t is None:
        return H
    if t.dtype is not dtype or t.shape != (T, H) or not t.is_cuda:
        _refuse(t, name, f"[{T}, {H}]", dtype)
    rows, cols = t.stride()
    if cols != 1 and H > 1:
        _refuse(t, name, f"[{T}, {H}] with dense rows")
    return rows if T > 1 else H


def _ids(ids):
    import torch
    size = 8 if ids.dtype == torch.int64 else 4
    if (size == 4 and ids.dtype != _I32) or ids.dim() != 1 or not ids.is_cuda or not ids.is_contiguous():
        _refuse(ids, "ids", "a dense vector", ids.dtype if ids.dtype in (torch.int64, _I32) else torch.int64)
    return ids.data_ptr(), size


def _space(ws):
    if ws is None:
        return None, 0
    if not ws.is_cuda or not ws.is_contiguous():
        _refuse(ws, "workspace", "dense")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def mhc_embed(ids, table, out, scale: float = 1.0, first_id: int = 0, stream=None) -> None:
    """Rows of ``table`` [V, H] into ``out`` [T, H] or [T, streams, H]."""
    L = _ops()
    (V, H), dt, shape = table.shape, table.dtype, out.shape
    p, size = _ids(ids)
    T = ids.shape[0]
    S = shape[1] if len(shape) == 3 else 1
    o = _dense(out, (T, S, H) if len(shape) == 3 else (T, H), dt, "out")
    rc = L.mhc_embed(p, size, table.data_ptr(), _pitch(table, V, H, dt, "table"), V, first_id, scale, T, H, S,
                     _dtype(table, "table"), o, _where(stream))
    if rc:
        _check(rc)


def mhc_embed_grad_workspace_bytes(T: int, V: int, H: int) -> int:
    return int(lib().mhc_embed_grad_workspace_bytes(int(T), int(V), int(H)))


def mhc_embed_grad(ids, dout, dtable, workspace, scale: float = 1.0, first_id: int = 0, padding_id: int | None = None,
                   accumulate: bool = False, stream=None) -> None:
    """The gradient of mhc_embed by its table: ``dout`` [T, H] or [T, streams, H]
    into ``dtable`` [V, H] (fp32 or dout's type)."""
    L = _ops()
    (V, H), dt, shape = dtable.shape, dout.dtype, dout.shape
    p, size = _ids(ids)
    T = ids.shape[0]
    S = shape[1] if len(shape) == 3 else 1
    d = _dense(dout, (T, S, H) if len(shape) == 3 else (T, H), dt, "dout")
    pad = None if padding_id is None else C.byref(C.c_int64(padding_id))
    ws, n = _space(workspace)
    rc = L.mhc_embed_grad(p, size, d, _dtype(dout, "dout"), scale, T, H, S, V, first_id, pad, int(accumulate),
                          dtable.data_ptr(), _dtype(dtable, "dtable"), _pitch(dtable, V, H, dtable.dtype, "dtable"), ws, n,
                          _where(stream))
    if rc:
        _check(rc)


def _gate(gate, gate_mode: int, T: int, H: int, dtype):
    if gate is None:
        return None
    return _vec(gate, T, _F32, "gate") if gate_mode == MHC_GATE_TOKEN else _vec(gate, H, dtype, "gate")


def mhc_block_norm(y, r, gamma_post, gate, gamma_pre, r_out, norm, rstd_post, rstd_pre, gate_mode: int = MHC_GATE_NONE,
                   res_scale: float = 1.0, eps: float = 1e-6, stream=None) -> None:
    """Norm after a block, gate, residual add and norm before the next block;
    y, r, r_out and norm are [T, H] (rows may be strided)."""
    L = _ops()
    x = y if r is None else r
    if x is None:
        raise MhcError(-1, "y or r is required")
    (T, H), dt = x.shape, x.dtype
    rc = L.mhc_block_norm(
        None if y is None else y.data_ptr(), _pitch(y, T, H, dt, "y"),
        None if r is None else r.data_ptr(), _pitch(r, T, H, dt, "r"),
        _vec(gamma_post, H, dt, "gamma_post"), _gate(gate, gate_mode, T, H, dt), gate_mode,
        _vec(gamma_pre, H, dt, "gamma_pre"), res_scale, eps, T, H, _dtype(x, "r"),
        None if r_out is None else r_out.data_ptr(), _pitch(r_out, T, H, dt, "r_out"),
        None if norm is None else norm.data_ptr(), _pitch(norm, T, H, dt, "norm"),
        _vec(rstd_post, T, _F32, "rstd_post"), _vec(rstd_pre, T, _F32, "rstd_pre"), _where(stream))
    if rc:
        _check(rc)


def mhc_block_norm_grad_workspace_bytes(T: int, H: int) -> int:
    return int(lib().mhc_block_norm_grad_workspace_bytes(int(T), int(H)))


def mhc_block_norm_grad(dr_out, dnorm, y, r_out, gamma_post, gate, gamma_pre, rstd_post, rstd_pre, dy, dr, dgamma_post,
                        dgate, dgamma_pre, workspace, gate_mode: int = MHC_GATE_NONE, res_scale: float = 1.0,
                        stream=None) -> None:
    """The gradient of mhc_block_norm; all matrices are dense [T, H], the
    weights' gradients fp32."""
    L = _ops()
    x = dy if dr is None else dr
    if x is None:
        raise MhcError(-1, "dy or dr is required")
    shape, dt = x.shape, x.dtype
    T, H = shape
    ws, n = _space(workspace)
    rc = L.mhc_block_norm_grad(
        _dense(dr_out, shape, dt, "dr_out"), _dense(dnorm, shape, dt, "dnorm"), _dense(y, shape, dt, "y"),
        _dense(r_out, shape, dt, "r_out"), _vec(gamma_post, H, dt, "gamma_post"), _gate(gate, gate_mode, T, H, dt),
        gate_mode, _vec(gamma_pre, H, dt, "gamma_pre"), _vec(rstd_post, T, _F32, "rstd_post"),
        _vec(rstd_pre, T, _F32, "rstd_pre"), res_scale, T, H, _dtype(x, "dr"), _dense(dy, shape, dt, "dy"),
        _dense(dr, shape, dt, "dr"), _vec(dgamma_post, H, _F32, "dgamma_post"),
        _vec(dgate, T if gate_mode == MHC_GATE_TOKEN else H, _F32, "dgate"),
        _vec(dgamma_pre, H, _F32, "dgamma_pre"), ws, n, _where(stream))
    if rc:
        _check(rc)


def mhc_route_workspace_bytes(E: int) -> int:
    return int(lib().mhc_route_workspace_bytes(int(E)))


def mhc_route(logits, bias, indices, weights, counts=None, workspace=None, score: int = MHC_SCORE_SIGMOID,
              groups: int = 1, top_groups: int = 1, renorm: bool = True, scale: float = 1.0, stream=None) -> None:
    """The k best experts of each row of ``logits`` [T, E]: ``indices`` [T, k]
    int32, ``weights`` [T, k] fp32 and, where given, the experts' ``counts``."""
    L = _ops()
    T, E = logits.shape
    k = indices.shape[-1]
    ws, n = _space(workspace)
    rc = L.mhc_route(logits.data_ptr(), _pitch(logits, T, E, logits.dtype, "logits"), _dtype(logits, "logits"),
                     _vec(bias, E, _F32, "bias"), score, E, groups, top_groups, k, int(renorm), scale, T,
                     _dense(indices, (T, k), _I32, "indices"), _dense(weights, (T, k), _F32, "weights"),
                     _vec(counts, E, _I32, "counts"), ws, n, _where(stream))
    if rc:
        _check(rc)


def mhc_route_grad(dweights, logits, indices, dlogits, score: int = MHC_SCORE_SIGMOID, renorm: bool = True,
                   scale: float = 1.0, stream=None) -> None:
    """The gradient of mhc_route's weights by the logits."""
    L = _ops()
    (T, E), dt = logits.shape, logits.dtype
    k = indices.shape[-1]
    rc = L.mhc_route_grad(_dense(dweights, (T, k), _F32, "dweights"), logits.data_ptr(), _pitch(logits, T, E, dt, "logits"),
                          _dtype(logits, "logits"), _dense(indices, (T, k), _I32, "indices"), score, E, k, int(renorm), scale,
                          T, dlogits.data_ptr(), _pitch(dlogits, T, E, dt, "dlogits"), _where(stream))
    if rc:
        _check(rc)


def mhc_glu_workspace_bytes(T: int, H: int, F: int) -> int:
    return int(lib().mhc_glu_workspace_bytes(int(T), int(H), int(F)))


def _addend(add, T: int, N: int, dtype) -> int:
    """The row stride of what is added to [T, N]: 0 where one row serves every token."""
    if add is None:
        return 0
    if add.dim() == 2 and T > 1 and add.shape[0] == T and add.stride(0) == 0:
        _pitch(add[:1], 1, N, dtype, "add")
        return 0
    return _pitch(add, T, N, dtype, "add")


def mhc_glu(x, w, h, workspace, add=None, gu=None, act: int = MHC_ACT_SILU, stream=None) -> None:
    """act(x Wg^T + add_g) * (x Wu^T + add_u) into ``h`` [T, F], of ``x`` [T, H] and ``w``
    [2F, H] (the gate's rows first); ``add`` [T, 2F] may be one row expanded to all tokens."""
    L = _ops()
    (T, H), dt = x.shape, x.dtype
    F = w.shape[0] // 2
    ws, n = _space(workspace)
    rc = L.mhc_glu(x.data_ptr(), _pitch(x, T, H, dt, "x"), _dense(w, (2 * F, H), dt, "w"), None if add is None else add.data_ptr(),
                   _addend(add, T, 2 * F, dt), act, T, H, F, _dtype(x, "x"), _dense(gu, (T, 2 * F), dt, "gu"), h.data_ptr(),
                   _pitch(h, T, F, dt, "h"), ws, n, _where(stream))
    if rc:
        _check(rc)


def mhc_glu_grad(dh, gu, x, w, dgu, dx, dw, workspace, act: int = MHC_ACT_SILU, accumulate: bool = False, stream=None) -> None:
    """The gradient of mhc_glu: ``dgu`` [T, 2F], ``dx`` [T, H] and ``dw`` [2F, H] (fp32 or x's
    type) from ``dh`` [T, F] and the kept ``gu``; dx and dw may be None."""
    L = _ops()
    (T, F), dt = dh.shape, dh.dtype
    H = x.shape[1] if x is not None else w.shape[1] if w is not None else 8
    ws, n = _space(workspace)
    rc = L.mhc_glu_grad(_dense(dh, (T, F), dt, "dh"), _dense(gu, (T, 2 * F), dt, "gu"), None if x is None else x.data_ptr(),
                        _pitch(x, T, H, dt, "x"), _dense(w, (2 * F, H), dt, "w"), act, T, H, F, _dtype(dh, "dh"),
                        _dense(dgu, (T, 2 * F), dt, "dgu"), _dense(dx, (T, H), dt, "dx"),
                        None if dw is None else _dense(dw, (2 * F, H), dw.dtype, "dw"), MHC_DT_F32 if dw is None else _dtype(dw, "dw"),
                        int(accumulate), ws, n, _where(stream))
    if rc:
        _check(rc)


def mhc_lora_workspace_bytes(T: int, R: int) -> int:
    return int(lib().mhc_lora_workspace_bytes(int(T), int(R)))


def mhc_lora(x, a, b, index, out, workspace, scale=None, base=None, stream=None) -> None:
    """base + scale[i] * b[i] @ (a[i] @ x[t]), i = index[t], into ``out`` [T, N]: of ``x``
    [T, H], ``a`` [n, R, H] and ``b`` [n, N, R]; out may be base."""
    L = _ops()
    (T, H), dt = x.shape, x.dtype
    n, N, R = b.shape
    ws, size = _space(workspace)
    rc = L.mhc_lora(x.data_ptr(), _pitch(x, T, H, dt, "x"), _dense(a, (n, R, H), dt, "a"), _dense(b, (n, N, R), dt, "b"),
                    _vec(index, T, _I32, "index"), _vec(scale, n, _F32, "scale"), T, H, N, R, n, _dtype(x, "x"),
                    None if base is None else base.data_ptr(), _pitch(base, T, N, dt, "base"), out.data_ptr(),
                    _pitch(out, T, N, dt, "out"), ws, size, _where(stream))
    if rc:
        _check(rc)


def mhc_dropout(y, out, seed, r=None, p: float = 0.1, stream=None) -> None:
    """Dropout of ``y`` [T, H] and the residual add of ``r``, into ``out`` (rows may be
    strided).  ``seed`` is an int64 (or uint64) tensor of two on the GPU: the key and the
    call's number.  The gradient by y is this call on the gradient of out, without r."""
    L = _ops()
    (T, H), dt = y.shape, y.dtype
    if seed.dtype is not _I64 and seed.dtype is not _U64:
        _refuse(seed, "seed", "a dense vector of 2", _I64)
    rc = L.mhc_dropout(y.data_ptr(), _pitch(y, T, H, dt, "y"), None if r is None else r.data_ptr(), _pitch(r, T, H, dt, "r"),
                       p, _vec(seed, 2, seed.dtype, "seed"), T, H, _dtype(y, "y"), out.data_ptr(),
                       _pitch(out, T, H, dt, "out"), _where(stream))
    if rc:
        _check(rc)


# ----------------------------------------------------------- allocation ----
def alloc_outputs(T: int, H: int, out_mode: int, device, cfg=None, unshifted: bool = False) -> dict:
    """Output tensors and an initialised workspace for one seam call (with
    ``unshifted``, for mhc_seam_unshifted: ``norm`` then receives x)."""
    import torch
    o = {
        "residual_out": torch.empty((T, 4, H), dtype=torch.bfloat16, device=device),
        "norm": torch.empty((T, H), dtype=torch.bfloat16, device=device),
        # mxfp8: e4m3 codes; fp8_grid: the bf16 grid (written through the same argument)
        "fp8_codes": (torch.empty((T, H), dtype=torch.uint8, device=device) if out_mode == MHC_OUT_MXFP8 else
                      torch.empty((T, H), dtype=torch.bfloat16, device=device) if out_mode == MHC_OUT_FP8_GRID
                      else None),
        "e8m0_scales": torch.empty((T, H // 32), dtype=torch.uint8, device=device) if out_mode == MHC_OUT_MXFP8 else None,
        "pre_out": torch.empty((T, 4), dtype=torch.float32, device=device),
        "post_out": torch.empty((T, 4), dtype=torch.float32, device=device),
        "comb_out": torch.empty((T, 4, 4), dtype=torch.float32, device=device),
    }
    nbytes = mhc_workspace_bytes_unshifted(T, H, cfg) if unshifted else mhc_workspace_bytes(T, H, cfg)
    o["workspace"] = torch.empty((nbytes + 15) // 16 * 16, dtype=torch.uint8, device=device)
    mhc_workspace_init(o["workspace"])
    return o
