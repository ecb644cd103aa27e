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
# before they pass the pointers on (MHC_ERR_CONFIG for a type, MHC_ERR_SHAPE
# for a shape or a stride).
_DTYPES: dict = {}


def _dtype(t) -> int:
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.bfloat16: MHC_DT_BF16, torch.float16: MHC_DT_F16, torch.float32: MHC_DT_F32})
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise MhcError(-10, f"{t.dtype} is not bf16, fp16 or fp32")
    return d


def _need(ok: bool, msg: str, code: int = -2) -> None:
    if not ok:
        raise MhcError(code, msg)


def _dense(t, shape, dtype, name: str) -> None:
    """``t`` is None or a dense tensor of this shape and type."""
    if t is not None:
        _need(t.is_cuda, f"{name} is not on the GPU", -10)
        _need(t.dtype == dtype, f"{name} must be {dtype}", -10)
        _need(tuple(t.shape) == shape and t.is_contiguous(), f"{name} must be dense, of shape {shape}")


def _rows(t, T: int, H: int, dtype, name: str) -> int:
    """The row stride of a [T, H] matrix with dense rows (H for None)."""
    if t is None:
        return H
    _need(t.is_cuda, f"{name} is not on the GPU", -10)
    _need(t.dtype == dtype, f"{name} must be {dtype}", -10)
    _need(t.dim() == 2 and t.shape[0] == T and t.shape[1] == H and (t.stride(1) == 1 or H == 1),
          f"{name} must be [{T}, {H}] with dense rows")
    return t.stride(0) if T > 1 else max(H, t.stride(0) // 8 * 8)


def _id_bytes(ids) -> int:
    import torch
    _need(ids.is_cuda, "ids is not on the GPU", -10)
    _need(ids.dtype in (torch.int32, torch.int64), "ids must be int32 or int64", -10)
    _need(ids.dim() == 1 and ids.is_contiguous(), "ids must be a dense vector")
    return ids.element_size()


def mhc_embed(ids, table, out, scale: float = 1.0, first_id: int = 0, stream=None) -> None:
    """Rows of ``table`` [V, H] into ``out`` [T, H] or [T, streams, H]."""
    T, (V, H) = ids.shape[0], table.shape
    S = out.shape[1] if out.dim() == 3 else 1
    _dense(out, (T, S, H) if out.dim() == 3 else (T, H), table.dtype, "out")
    _check(lib().mhc_embed(_ptr(ids), _id_bytes(ids), _ptr(table), _rows(table, V, H, table.dtype, "table"), V,
                           int(first_id), float(scale), T, H, S, _dtype(table), _ptr(out), _stream(stream)))


def mhc_embed_grad_workspace_bytes(T: int, V: int, H: int) -> int:
    return int(lib().mhc_embed_grad_workspace_bytes(int(T), int(V), int(H)))


def mhc_embed_grad(ids, dout, dtable, workspace, scale: float = 1.0, first_id: int = 0, padding_id: int | None = None,
                   accumulate: bool = False, stream=None) -> None:
    """The gradient of mhc_embed by its table: ``dout`` [T, H] or [T, streams, H]
    into ``dtable`` [V, H] (fp32 or dout's type)."""
    T, (V, H) = ids.shape[0], dtable.shape
    S = dout.shape[1] if dout.dim() == 3 else 1
    _dense(dout, (T, S, H) if dout.dim() == 3 else (T, H), dout.dtype, "dout")
    pad = None if padding_id is None else C.byref(C.c_int64(padding_id))
    _check(lib().mhc_embed_grad(_ptr(ids), _id_bytes(ids), _ptr(dout), _dtype(dout), float(scale), T, H, S, V,
                                int(first_id), pad, int(accumulate), _ptr(dtable), _dtype(dtable),
                                _rows(dtable, V, H, dtable.dtype, "dtable"), _ptr(workspace), _bytes(workspace),
                                _stream(stream)))


def _bytes(t) -> int:
    if t is None:
        return 0
    _need(t.is_cuda and t.is_contiguous(), "workspace must be dense and on the GPU", -10)
    return t.numel() * t.element_size()


def _gate(gate, gate_mode: int, T: int, H: int, dtype) -> None:
    import torch
    if gate is not None:
        token = gate_mode == MHC_GATE_TOKEN
        _dense(gate, (T,) if token else (H,), torch.float32 if token else dtype, "gate")


def mhc_block_norm(y, r, gamma_post, gate, gamma_pre, r_out, norm, rstd_post, rstd_pre, gate_mode: int = MHC_GATE_NONE,
                   res_scale: float = 1.0, eps: float = 1e-6, stream=None) -> None:
    """Norm after a block, gate, residual add and norm before the next block;
    y, r, r_out and norm are [T, H] (rows may be strided)."""
    import torch
    (T, H), dt = r.shape, r.dtype
    _gate(gate, gate_mode, T, H, dt)
    for t, n in ((gamma_post, "gamma_post"), (gamma_pre, "gamma_pre")):
        _dense(t, (H,), dt, n)
    for t, n in ((rstd_post, "rstd_post"), (rstd_pre, "rstd_pre")):
        _dense(t, (T,), torch.float32, n)
    _check(lib().mhc_block_norm(_ptr(y), _rows(y, T, H, dt, "y"), _ptr(r), _rows(r, T, H, dt, "r"), _ptr(gamma_post),
                                _ptr(gate), gate_mode, _ptr(gamma_pre), float(res_scale), float(eps), T, H, _dtype(r),
                                _ptr(r_out), _rows(r_out, T, H, dt, "r_out"), _ptr(norm), _rows(norm, T, H, dt, "norm"),
                                _ptr(rstd_post), _ptr(rstd_pre), _stream(stream)))


def mhc_block_norm_grad_workspace_bytes(T: int, H: int) -> int:
    return int(lib().mhc_block_norm_grad_workspace_bytes(int(T), int(H)))


def mhc_block_norm_grad(dr_out, dnorm, y, r_out, gamma_post, gate, gamma_pre, rstd_post, rstd_pre, dy, dr, dgamma_post,
                        dgate, dgamma_pre, workspace, gate_mode: int = MHC_GATE_NONE, res_scale: float = 1.0,
                        stream=None) -> None:
    """The gradient of mhc_block_norm; all matrices are dense [T, H], the
    weights' gradients fp32."""
    import torch
    (T, H), dt, f32 = dr.shape, dr.dtype, torch.float32
    _gate(gate, gate_mode, T, H, dt)
    for t, n in ((dr_out, "dr_out"), (dnorm, "dnorm"), (y, "y"), (r_out, "r_out"), (dy, "dy"), (dr, "dr")):
        _dense(t, (T, H), dt, n)
    for t, n in ((gamma_post, "gamma_post"), (gamma_pre, "gamma_pre")):
        _dense(t, (H,), dt, n)
    for t, n in ((rstd_post, "rstd_post"), (rstd_pre, "rstd_pre")):
        _dense(t, (T,), f32, n)
    for t, n in ((dgamma_post, "dgamma_post"), (dgamma_pre, "dgamma_pre")):
        _dense(t, (H,), f32, n)
    _dense(dgate, (T,) if gate_mode == MHC_GATE_TOKEN else (H,), f32, "dgate")
    _check(lib().mhc_block_norm_grad(_ptr(dr_out), _ptr(dnorm), _ptr(y), _ptr(r_out), _ptr(gamma_post), _ptr(gate),
                                     gate_mode, _ptr(gamma_pre), _ptr(rstd_post), _ptr(rstd_pre), float(res_scale), T,
                                     H, _dtype(dr), _ptr(dy), _ptr(dr), _ptr(dgamma_post), _ptr(dgate),
                                     _ptr(dgamma_pre), _ptr(workspace), _bytes(workspace), _stream(stream)))


def mhc_route_workspace_bytes(E: int) -> int:
    return int(lib().mhc_route_workspace_bytes(int(E)))


def mhc_route(logits, bias, indices, weights, counts=None, workspace=None, score: int = MHC_SCORE_SIGMOID,
              groups: int = 1, top_groups: int = 1, renorm: bool = True, scale: float = 1.0, stream=None) -> None:
    """The k best experts of each row of ``logits`` [T, E]: ``indices`` [T, k]
    int32, ``weights`` [T, k] fp32 and, where given, the experts' ``counts``."""
    import torch
    (T, E), k = logits.shape, indices.shape[-1]
    _dense(bias, (E,), torch.float32, "bias")
    _dense(indices, (T, k), torch.int32, "indices")
    _dense(weights, (T, k), torch.float32, "weights")
    _dense(counts, (E,), torch.int32, "counts")
    _check(lib().mhc_route(_ptr(logits), _pitch(logits, T, E, "logits"), _dtype(logits), _ptr(bias), score, E, groups,
                           top_groups, k, int(renorm), float(scale), T, _ptr(indices), _ptr(weights), _ptr(counts),
                           _ptr(workspace), _bytes(workspace), _stream(stream)))


def _pitch(t, T: int, E: int, name: str) -> int:
    """The row stride of a [T, E] matrix with dense rows, of any alignment."""
    _need(t.is_cuda, f"{name} is not on the GPU", -10)
    _need(t.dim() == 2 and t.shape[0] == T and t.shape[1] == E and (t.stride(1) == 1 or E == 1),
          f"{name} must be [{T}, {E}] with dense rows")
    return t.stride(0) if T > 1 else E


def mhc_route_grad(dweights, logits, indices, dlogits, score: int = MHC_SCORE_SIGMOID, renorm: bool = True,
                   scale: float = 1.0, stream=None) -> None:
    """The gradient of mhc_route's weights by the logits."""
    import torch
    (T, E), k = logits.shape, indices.shape[-1]
    _dense(dweights, (T, k), torch.float32, "dweights")
    _dense(indices, (T, k), torch.int32, "indices")
    _need(dlogits.dtype == logits.dtype, "dlogits must have logits' type", -10)
    _check(lib().mhc_route_grad(_ptr(dweights), _ptr(logits), _pitch(logits, T, E, "logits"), _dtype(logits),
                                _ptr(indices), score, E, k, int(renorm), float(scale), T, _ptr(dlogits),
                                _pitch(dlogits, T, E, "dlogits"), _stream(stream)))


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
