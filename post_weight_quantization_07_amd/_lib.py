"""ctypes binding of libgptq.so (include/gptq.h).

Argument marshalling only: every step of the solve runs in the HIP library.
Tensors must live on the current HIP device; PyTorch supplies device memory
and the current stream.  Loading fails loudly when the library is missing.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import c_float, c_int32, c_int64, c_size_t, c_void_p
from dataclasses import dataclass
from typing import Mapping, Optional

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgptq.so")

GPTQ_OK, GPTQ_ERR_INVALID_ARG, GPTQ_ERR_NOT_SPD, GPTQ_ERR_HIP, GPTQ_ERR_WORKSPACE, GPTQ_ERR_TOO_LARGE = range(6)
GPTQ_F32, GPTQ_BF16, GPTQ_I8 = 0, 1, 2

EXPORTS = ("gptq_config_validate", "gptq_status_string", "gptq_hessian_workspace_size",
           "gptq_hessian_accumulate", "gptq_prepare_workspace_size", "gptq_prepare_hinv",
           "gptq_workspace_size", "gptq_quantize_layer", "gptq_pack", "gptq_dequant_workspace_size",
           "gptq_dequant_matmul", "gptq_dequant_order", "gptq_dequant_ordered_workspace_size",
           "gptq_dequant_matmul_ordered", "gptq_dequant_scratch_bytes", "gptq_dequant_noalloc_need",
           "gptq_dequant_matmul_noalloc", "gptq_quantize_tokens", "gptq_integer_weight",
           "gptq_integer_workspace_size", "gptq_integer_matmul", "gptq_integer_linear",
           "gptq_integer_gated_workspace_size", "gptq_integer_gated", "gptq_norm_tokens", "gptq_cache_write",
           "gptq_cache_read", "gptq_attention_workspace_size", "gptq_cache_attention", "gptq_cache_attention_scores",
           "gptq_phase_timing", "gptq_phase_count", "gptq_phase_name",
           "gptq_phase_read")


class GptqError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_lib().gptq_status_string(status).decode()} (status {status})")


class NotPositiveDefinite(GptqError):
    """The damped Hessian failed a Cholesky pivot; retry with a larger damp_percent."""


class NonFiniteHessian(GptqError):
    """diag(H) holds a NaN or an infinity: the calibration inputs are not finite."""


class _CConfig(ctypes.Structure):
    _fields_ = [("bits", c_int32), ("group_size", c_int32), ("damp_percent", c_float),
                ("desc_act", c_int32), ("static_groups", c_int32), ("sym", c_int32),
                ("block_size", c_int32)]


class _CCache(ctypes.Structure):
    _fields_ = [("n_pages", c_int64), ("page_size", c_int32), ("n_kv_heads", c_int32), ("head_dim", c_int32),
                ("bits", c_int32), ("k_codes", c_void_p), ("v_codes", c_void_p), ("k_scales", c_void_p),
                ("v_scales", c_void_p)]


class _CLayer(ctypes.Structure):
    _fields_ = [("w", c_void_p), ("scales", c_void_p), ("offsets", c_void_p), ("bias", c_void_p)]


class _CScores(ctypes.Structure):
    _fields_ = [("cap", c_float), ("slopes", c_void_p), ("prefix_lens", c_void_p)]


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                              "or python -m post_weight_quantization_07_amd.build")
        lib = ctypes.CDLL(LIB_PATH)
        vp, i64, sz = c_void_p, c_int64, c_size_t
        cfgp, cachep = ctypes.POINTER(_CConfig), ctypes.POINTER(_CCache)
        layerp, scoresp = ctypes.POINTER(_CLayer), ctypes.POINTER(_CScores)
        sig = {
            "gptq_config_validate": (c_int32, [cfgp]),
            "gptq_status_string": (ctypes.c_char_p, [c_int32]),
            "gptq_hessian_workspace_size": (sz, [i64, i64, c_int32]),
            "gptq_hessian_accumulate": (c_int32, [vp, i64, vp, c_int32, i64, i64, vp, sz, vp]),
            "gptq_prepare_workspace_size": (sz, [i64]),
            "gptq_prepare_hinv": (c_int32, [vp, i64, i64, cfgp, vp, vp, vp, vp, sz, vp]),
            "gptq_workspace_size": (sz, [i64, i64, cfgp]),
            "gptq_quantize_layer": (c_int32, [vp, c_int32, i64, i64, vp, vp, cfgp, vp, vp, vp, vp, vp, vp,
                                              vp, sz, vp]),
            "gptq_pack": (c_int32, [vp, i64, i64, c_int32, vp, vp]),
            "gptq_dequant_workspace_size": (sz, [i64, i64, i64]),
            "gptq_dequant_matmul": (c_int32, [vp, c_int32, i64, i64, vp, vp, vp, vp, c_int32, i64, c_int32, vp, vp,
                                              sz, vp]),
            "gptq_dequant_order": (c_int32, [vp, vp, c_int32, i64, i64, vp, vp, vp, vp]),
            "gptq_dequant_ordered_workspace_size": (sz, [i64, i64, i64]),
            "gptq_dequant_matmul_ordered": (c_int32, [vp, c_int32, i64, i64, vp, vp, vp, vp, vp, c_int32, i64,
                                                      c_int32, vp, vp, sz, vp]),
            "gptq_dequant_scratch_bytes": (sz, []),
            "gptq_dequant_noalloc_need": (sz, [i64, c_int32, i64, c_int32, i64]),
            "gptq_dequant_matmul_noalloc": (c_int32, [vp, c_int32, i64, i64, vp, vp, vp, vp, c_int32, i64, c_int32,
                                                      vp, vp]),
            "gptq_quantize_tokens": (c_int32, [vp, c_int32, i64, i64, i64, vp, vp, vp, vp]),
            "gptq_integer_weight": (c_int32, [vp, vp, c_int32, i64, i64, vp, vp, vp]),
            "gptq_integer_workspace_size": (sz, [i64, c_int32, i64, i64]),
            "gptq_integer_matmul": (c_int32, [vp, c_int32, vp, vp, i64, i64, i64, vp, vp, vp, i64, vp, c_int32, vp, sz,
                                              vp]),
            "gptq_integer_linear": (c_int32, [vp, c_int32, vp, vp, i64, i64, i64, layerp, i64, c_int32, vp, c_int32, i64, vp,
                                              c_int32, vp, sz, vp]),
            "gptq_integer_gated_workspace_size": (sz, [i64, c_int32, i64, i64]),
            "gptq_integer_gated": (c_int32, [vp, c_int32, vp, vp, i64, i64, i64, layerp, layerp, i64, c_int32, vp, c_int32, vp,
                                             sz, vp]),
            "gptq_norm_tokens": (c_int32, [vp, c_int32, i64, i64, i64, vp, c_int32, i64, vp, c_int32, c_float, vp, i64, vp,
                                           c_int32, vp, vp, vp, vp]),
            "gptq_cache_write": (c_int32, [cachep, vp, vp, c_int32, i64, i64, i64, vp, vp]),
            "gptq_cache_read": (c_int32, [cachep, vp, i64, vp, vp, c_int32, vp]),
            "gptq_attention_workspace_size": (sz, [cachep, i64, c_int32, c_int32, i64]),
            "gptq_cache_attention": (c_int32, [cachep, vp, c_int32, i64, i64, c_int32, vp, i64, vp, vp, c_int32, c_float,
                                               vp, i64, vp, sz, vp]),
            "gptq_cache_attention_scores": (c_int32, [cachep, vp, c_int32, i64, i64, c_int32, vp, i64, vp, vp, c_int32, c_float,
                                                      scoresp, vp, i64, vp, sz, vp]),
            "gptq_phase_timing": (c_int32, [c_int32]),
            "gptq_phase_count": (c_int32, []),
            "gptq_phase_name": (ctypes.c_char_p, [c_int32]),
            "gptq_phase_read": (c_int32, [vp, vp, c_int32]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
    return _LIB


def phase_timing(enable: bool) -> None:
    """Switch the library's per-phase launch timing on (clearing the record) or off."""
    _check(_lib().gptq_phase_timing(1 if enable else 0), "gptq_phase_timing")


def phase_read() -> dict:
    """{phase name: (summed ms, launches)} of the launches recorded since timing was switched on."""
    lib = _lib()
    n = int(lib.gptq_phase_count())
    ms = (c_float * n)()
    cnt = (c_int32 * n)()
    _check(lib.gptq_phase_read(ctypes.cast(ms, c_void_p), ctypes.cast(cnt, c_void_p), n), "gptq_phase_read")
    return {lib.gptq_phase_name(i).decode(): (float(ms[i]), int(cnt[i])) for i in range(n)}


def library_path() -> str:
    _lib()
    return LIB_PATH


# --------------------------------------------------------------------------
# configuration: the field names and defaults of BaseQuantizeConfig
# (AutoGPTQ examples walkthrough, section 1.4; OLMo quick-start, section 三)
# --------------------------------------------------------------------------

@dataclass
class QuantizeConfig:
    bits: int = 4
    group_size: int = -1
    damp_percent: float = 0.01
    desc_act: bool = True
    static_groups: bool = False
    sym: bool = True
    block_size: int = 128

    def __post_init__(self):
        if self.bits not in (2, 3, 4, 8):
            raise ValueError(f"bits must be one of [2, 3, 4, 8], got {self.bits}")
        if not (self.group_size == -1 or self.group_size > 0):
            raise ValueError(f"group_size must be -1 or > 0, got {self.group_size}")
        if not (0 < self.damp_percent < 1):
            raise ValueError(f"damp_percent must be in (0, 1), got {self.damp_percent}")
        st = _lib().gptq_config_validate(ctypes.byref(self._c()))
        if st != GPTQ_OK:
            raise ValueError(f"configuration rejected by the solver (block_size must be 128; a group "
                             f"must divide 128 or be a multiple of it): {self}")

    def _c(self) -> _CConfig:
        return _CConfig(int(self.bits), int(self.group_size), float(self.damp_percent), int(bool(self.desc_act)),
                        int(bool(self.static_groups)), int(bool(self.sym)), int(self.block_size))

    def n_groups(self, d_in: int) -> int:
        return 1 if self.group_size == -1 else -(-d_in // self.group_size)


# --------------------------------------------------------------------------
# marshalling helpers
# --------------------------------------------------------------------------

def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(st: int, what: str):
    if st != GPTQ_OK:
        raise GptqError(st, what)


def _dev(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous and on the GPU")


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return GPTQ_BF16
    if t.dtype == torch.float32:
        return GPTQ_F32
    raise ValueError(f"unsupported dtype {t.dtype}: expected bfloat16 or float32")


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _ws_bytes(ws: Optional[torch.Tensor]) -> int:
    """The bytes of a workspace, of any dtype.  One whose elements do not lie one
    behind the other (a strided or an expanded view) has no such size."""
    if ws is None:
        return 0
    if not ws.is_contiguous():
        raise ValueError("a workspace must be contiguous")
    return ws.numel() * ws.element_size()


# --------------------------------------------------------------------------
# the four calls of the C ABI
# --------------------------------------------------------------------------

def gptq_hessian_workspace_size(d_in: int, n_tokens: int, dtype: torch.dtype) -> int:
    code = GPTQ_BF16 if dtype == torch.bfloat16 else GPTQ_F32
    return int(_lib().gptq_hessian_workspace_size(d_in, n_tokens, code))


def gptq_hessian_accumulate(S: torch.Tensor, X: torch.Tensor, ws: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """S += X^T X for X [n_tokens, d_in] (rows may be strided)."""
    if X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be 2-D with unit column stride")
    _dev(S)
    if not X.is_cuda:
        raise ValueError("X must be on the GPU")
    n, d = X.shape
    if S.shape != (d, d) or S.dtype != torch.float32:
        raise ValueError("S must be float32 [d_in, d_in]")
    code = _dtype_code(X)
    need = gptq_hessian_workspace_size(d, n, X.dtype)
    if ws is None:
        ws = _workspace(need, X.device)
    _check(_lib().gptq_hessian_accumulate(_ptr(S), d, _ptr(X), code, n, X.stride(0), _ptr(ws), _ws_bytes(ws),
                                          _stream(stream)), "gptq_hessian_accumulate")
    return S


def gptq_prepare_workspace_size(d_in: int) -> int:
    return int(_lib().gptq_prepare_workspace_size(d_in))


def gptq_prepare_hinv(S: torch.Tensor, n_total: int, cfg: QuantizeConfig, U: Optional[torch.Tensor] = None,
                      perm: Optional[torch.Tensor] = None, info: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None, stream=None, check: bool = True):
    """S -> H in place; returns (U, perm, info).  With check=True the stream is
    synchronised and a failed pivot raises NotPositiveDefinite."""
    _dev(S)
    d = S.shape[0]
    dev = S.device
    U = torch.empty((d, d), dtype=torch.float32, device=dev) if U is None else U
    perm = torch.empty(d, dtype=torch.int32, device=dev) if perm is None else perm
    info = torch.empty(1, dtype=torch.int32, device=dev) if info is None else info
    if ws is None:
        ws = _workspace(gptq_prepare_workspace_size(d), dev)
    _check(_lib().gptq_prepare_hinv(_ptr(S), d, int(n_total), ctypes.byref(cfg._c()), _ptr(U), _ptr(perm),
                                    _ptr(info), _ptr(ws), _ws_bytes(ws), _stream(stream)), "gptq_prepare_hinv")
    if check:
        k = int(info.item())
        if k == -1:
            raise NonFiniteHessian(GPTQ_ERR_NOT_SPD, "gptq_prepare_hinv: diag(H) is not finite (NaN or infinity "
                                   "in the calibration inputs)")
        if k != 0:
            raise NotPositiveDefinite(GPTQ_ERR_NOT_SPD, "gptq_prepare_hinv: the damped Hessian's trailing block is "
                                      f"not positive definite from sweep position {k - 1}")
    return U, perm, info


def gptq_workspace_size(d_out: int, d_in: int, cfg: QuantizeConfig) -> int:
    return int(_lib().gptq_workspace_size(d_out, d_in, ctypes.byref(cfg._c())))


def gptq_quantize_layer(W: torch.Tensor, U: torch.Tensor, perm: Optional[torch.Tensor], cfg: QuantizeConfig,
                        want_q: bool = True, want_loss: bool = True, out: Optional[dict] = None,
                        ws: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Column sweep; returns codes (uint8, original order), scales, zeros, g_idx
    and optionally Q (dequantized) and row_loss."""
    _dev(W, U, perm)
    d_out, d_in = W.shape
    dev = W.device
    ng = cfg.n_groups(d_in)
    o = dict(out) if out else {}
    o.setdefault("codes", torch.empty((d_out, d_in), dtype=torch.uint8, device=dev))
    o.setdefault("scales", torch.empty((ng, d_out), dtype=torch.float32, device=dev))
    o.setdefault("zeros", torch.empty((ng, d_out), dtype=torch.int32, device=dev))
    o.setdefault("g_idx", torch.empty(d_in, dtype=torch.int32, device=dev))
    if want_q:
        o.setdefault("Q", torch.empty((d_out, d_in), dtype=torch.float32, device=dev))
    if want_loss:
        o.setdefault("row_loss", torch.empty(d_out, dtype=torch.float32, device=dev))
    if ws is None:
        ws = _workspace(gptq_workspace_size(d_out, d_in, cfg), dev)
    _check(_lib().gptq_quantize_layer(_ptr(W), _dtype_code(W), d_out, d_in, _ptr(U), _ptr(perm),
                                      ctypes.byref(cfg._c()), _ptr(o["codes"]), _ptr(o["scales"]),
                                      _ptr(o["zeros"]), _ptr(o["g_idx"]), _ptr(o.get("Q")),
                                      _ptr(o.get("row_loss")), _ptr(ws), _ws_bytes(ws), _stream(stream)),
           "gptq_quantize_layer")
    return o


def gptq_pack(codes: torch.Tensor, bits: int, qweight: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    _dev(codes)
    d_out, d_in = codes.shape
    if qweight is None:
        qweight = torch.empty((d_in * bits // 32, d_out), dtype=torch.int32, device=codes.device)
    _check(_lib().gptq_pack(_ptr(codes), d_out, d_in, int(bits), _ptr(qweight), _stream(stream)), "gptq_pack")
    return qweight


def gptq_dequant_workspace_size(m: int, d_in: int, d_out: int) -> int:
    return int(_lib().gptq_dequant_workspace_size(m, d_in, d_out))


def gptq_dequant_matmul(x: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                        g_idx: torch.Tensor, bits: int, y: Optional[torch.Tensor] = None,
                        ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y [m, d_out] fp32 = x [m, d_in] (bf16 or fp32) times the transpose of the
    weights dequantized from qweight / scales / zeros / g_idx."""
    _dev(x, qweight, scales, zeros, g_idx)
    if x.dim() != 2 or not x.is_contiguous():
        raise ValueError("gptq_dequant_matmul: x must be a contiguous [m, d_in] matrix")
    m, d_in = x.shape
    d_out = qweight.shape[1]
    n_groups = scales.shape[0]
    if (qweight.shape[0] * 32 != d_in * bits or scales.shape != (n_groups, d_out) or zeros.shape != (n_groups, d_out)
            or g_idx.shape != (d_in,) or qweight.dtype != torch.int32 or scales.dtype != torch.float32
            or zeros.dtype != torch.int32 or g_idx.dtype != torch.int32):
        raise ValueError("gptq_dequant_matmul: qweight / scales / zeros / g_idx do not match x and bits")
    if y is None:
        y = torch.empty((m, d_out), dtype=torch.float32, device=x.device)
    if ws is None:
        need = gptq_dequant_workspace_size(m, d_in, d_out)
        ws = _workspace(need, x.device) if need > 0 else None
    _check(_lib().gptq_dequant_matmul(_ptr(x), _dtype_code(x), m, d_in, _ptr(qweight.contiguous()),
                                      _ptr(scales.contiguous()), _ptr(zeros.contiguous()), _ptr(g_idx.contiguous()),
                                      int(bits), d_out, n_groups, _ptr(y), _ptr(ws), _ws_bytes(ws),
                                      _stream(stream)),
           "gptq_dequant_matmul")
    return y


def gptq_dequant_scratch_bytes() -> int:
    return int(_lib().gptq_dequant_scratch_bytes())


def gptq_dequant_noalloc_need(m: int, dtype: torch.dtype, d_in: int, bits: int, d_out: int) -> int:
    code = GPTQ_BF16 if dtype == torch.bfloat16 else GPTQ_F32
    return int(_lib().gptq_dequant_noalloc_need(m, code, d_in, bits, d_out))


def gptq_dequant_matmul_noalloc(x: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                                g_idx: torch.Tensor, bits: int, y: torch.Tensor, stream=None) -> torch.Tensor:
    """gptq_dequant_matmul with the library's fixed scratch buffer instead of a
    workspace: the call itself allocates nothing (y is the caller's)."""
    _dev(x, qweight, scales, zeros, g_idx, y)
    if x.dim() != 2:
        raise ValueError("gptq_dequant_matmul_noalloc: x must be a contiguous [m, d_in] matrix")
    m, d_in = x.shape
    d_out = qweight.shape[1]
    n_groups = scales.shape[0]
    if (qweight.shape[0] * 32 != d_in * bits or scales.shape != (n_groups, d_out) or zeros.shape != (n_groups, d_out)
            or g_idx.shape != (d_in,) or y.shape != (m, d_out) or qweight.dtype != torch.int32
            or scales.dtype != torch.float32 or zeros.dtype != torch.int32 or g_idx.dtype != torch.int32
            or y.dtype != torch.float32):
        raise ValueError("gptq_dequant_matmul_noalloc: tensors do not match x and bits")
    _check(_lib().gptq_dequant_matmul_noalloc(_ptr(x), _dtype_code(x), m, d_in, _ptr(qweight), _ptr(scales),
                                              _ptr(zeros), _ptr(g_idx), int(bits), d_out, n_groups, _ptr(y),
                                              _stream(stream)),
           "gptq_dequant_matmul_noalloc")
    return y


def gptq_dequant_order(qweight: torch.Tensor, g_idx: torch.Tensor, bits: int, stream=None):
    """An act-order layer put in group order for the dequantizing product:
    returns (qweight_sorted, g_idx_sorted, order), order[j] = the original
    input channel at sorted position j (a stable sort of the channels by
    group), the codes repacked in that order."""
    _dev(qweight, g_idx)
    d_in = g_idx.shape[0]
    d_out = qweight.shape[1]
    if (g_idx.dim() != 1 or qweight.dim() != 2 or qweight.shape[0] * 32 != d_in * bits
            or qweight.dtype != torch.int32 or g_idx.dtype != torch.int32):
        raise ValueError("gptq_dequant_order: qweight / g_idx do not match bits")
    q_out = torch.empty_like(qweight)
    g_out = torch.empty_like(g_idx)
    order = torch.empty_like(g_idx)
    _check(_lib().gptq_dequant_order(_ptr(qweight.contiguous()), _ptr(g_idx.contiguous()), int(bits), d_in, d_out,
                                     _ptr(q_out), _ptr(g_out), _ptr(order), _stream(stream)),
           "gptq_dequant_order")
    return q_out, g_out, order


def gptq_dequant_ordered_workspace_size(m: int, d_in: int, d_out: int) -> int:
    return int(_lib().gptq_dequant_ordered_workspace_size(m, d_in, d_out))


def gptq_dequant_matmul_ordered(x: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                                g_idx: torch.Tensor, order: torch.Tensor, bits: int, y: Optional[torch.Tensor] = None,
                                ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """gptq_dequant_matmul on a layer reordered by gptq_dequant_order; x is
    given in the original channel order."""
    _dev(x, qweight, scales, zeros, g_idx, order)
    if x.dim() != 2 or not x.is_contiguous():
        raise ValueError("gptq_dequant_matmul_ordered: x must be a contiguous [m, d_in] matrix")
    m, d_in = x.shape
    d_out = qweight.shape[1]
    n_groups = scales.shape[0]
    if (qweight.shape[0] * 32 != d_in * bits or scales.shape != (n_groups, d_out) or zeros.shape != (n_groups, d_out)
            or g_idx.shape != (d_in,) or order.shape != (d_in,) or qweight.dtype != torch.int32
            or scales.dtype != torch.float32 or zeros.dtype != torch.int32 or g_idx.dtype != torch.int32
            or order.dtype != torch.int32):
        raise ValueError("gptq_dequant_matmul_ordered: tensors do not match x and bits")
    if y is None:
        y = torch.empty((m, d_out), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = _workspace(gptq_dequant_ordered_workspace_size(m, d_in, d_out), x.device)
    _check(_lib().gptq_dequant_matmul_ordered(_ptr(x), _dtype_code(x), m, d_in, _ptr(qweight.contiguous()),
                                              _ptr(scales.contiguous()), _ptr(zeros.contiguous()),
                                              _ptr(g_idx.contiguous()), _ptr(order.contiguous()), int(bits), d_out,
                                              n_groups, _ptr(y), _ptr(ws), _ws_bytes(ws), _stream(stream)),
           "gptq_dequant_matmul_ordered")
    return y


# --------------------------------------------------------------------------
# serving: the product in 8-bit integers, the quantized cache, its attention
# --------------------------------------------------------------------------

_TYPE = {torch.float32: GPTQ_F32, torch.bfloat16: GPTQ_BF16}


def _on_device(what: str, *ts) -> int:
    """The index of the current device, on which every given tensor has to lie."""
    dev = ts[0].get_device()
    for t in ts:
        if t is not None and t.get_device() != dev:
            dev = -1
    if dev < 0 or dev != torch._C._cuda_getDevice():  # torch.cuda.current_device() without its initialization
        raise ValueError(f"{what}: the tensors must be on the current GPU")
    return dev


def _on_stream(stream):
    """The context in which `stream` is the current one: what a call allocates
    (outputs, workspace, laid-out copies) then belongs to the stream that uses it."""
    if not isinstance(stream, torch.cuda.Stream):
        raw = _stream(stream)
        stream = torch.cuda.ExternalStream(raw) if raw else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _raw_stream(dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev)


def _row_stride(x: torch.Tensor) -> int:
    """Of a matrix; that of a single row says nothing.  (One below the row's
    length, as of an expanded row, is refused by the library.)"""
    return x.stride(0) if x.shape[0] > 1 else x.shape[1]


def _type_code(what: str, dtype: torch.dtype) -> int:
    code = _TYPE.get(dtype)
    if code is None:
        raise ValueError(f"{what}: unsupported dtype {dtype}: expected bfloat16 or float32")
    return code


def gptq_quantize_tokens(x: torch.Tensor, codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                         sums: Optional[torch.Tensor] = None, stream=None):
    """The 8-bit codes of the rows of x [m, d_in] (bf16 or fp32; rows may be
    strided): (codes int8 [m, d_in], scales fp32 [m], sums int32 [m]), the sums
    being those of a row's codes.  gptq_integer_matmul takes the three in x's place."""
    if stream is not None:
        with _on_stream(stream):
            return gptq_quantize_tokens(x, codes, scales, sums)
    what = "gptq_quantize_tokens"
    if x.dim() != 2 or (x.stride(1) != 1 and x.shape[1] > 1):
        raise ValueError(f"{what}: x must be 2-D with unit column stride")
    code = _type_code(what, x.dtype)
    dev = _on_device(what, x, codes, scales, sums)
    m, d = x.shape

    def place(t, shape, dtype):
        if t is None:
            return x.new_empty(shape, dtype=dtype)
        if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
            raise ValueError(f"{what}: codes, scales and sums must be contiguous int8 [m, d_in], float32 [m] and "
                             "int32 [m]")
        return t
    codes, scales, sums = place(codes, (m, d), torch.int8), place(scales, (m,), torch.float32), place(sums, (m,), torch.int32)
    _check(_lib().gptq_quantize_tokens(x.data_ptr(), code, m, d, _row_stride(x), codes.data_ptr(), scales.data_ptr(),
                                       sums.data_ptr(), _raw_stream(dev)), what)
    return codes, scales, sums


def gptq_integer_weight(qweight: torch.Tensor, zeros: torch.Tensor, bits: int, stream=None):
    """A layer with one group per output channel laid out for
    gptq_integer_matmul: (w int8 [d_out, d_in], offsets int32 [d_out]) with
    W = scale (w - offset).  zeros: [d_out] or [1, d_out] int32."""
    if stream is not None:
        with _on_stream(stream):
            return gptq_integer_weight(qweight, zeros, bits)
    what = "gptq_integer_weight"
    dev = _on_device(what, qweight, zeros)
    if bits not in (2, 3, 4, 8) or qweight.dim() != 2 or (qweight.shape[0] * 32) % bits != 0:
        raise ValueError(f"{what}: qweight does not match bits")
    d_in, d_out = qweight.shape[0] * 32 // bits, qweight.shape[1]
    if qweight.dtype != torch.int32 or zeros.dtype != torch.int32 or zeros.numel() != d_out or zeros.shape[-1] != d_out:
        raise ValueError(f"{what}: qweight and zeros must be int32 [d_in * bits / 32, d_out] and [d_out]: "
                         "the layer needs one group per output channel")
    w = torch.empty((d_out, d_in), dtype=torch.int8, device=qweight.device)
    offsets = torch.empty(d_out, dtype=torch.int32, device=qweight.device)
    _check(_lib().gptq_integer_weight(_ptr(qweight.contiguous()), _ptr(zeros.contiguous()), int(bits), d_in, d_out,
                                      _ptr(w), _ptr(offsets), _raw_stream(dev)), what)
    return w, offsets


def gptq_integer_workspace_size(m: int, dtype: torch.dtype, d_in: int, d_out: int) -> int:
    """dtype: of x (int8: codes)."""
    code = GPTQ_I8 if dtype == torch.int8 else _type_code("gptq_integer_workspace_size", dtype)
    return int(_lib().gptq_integer_workspace_size(m, code, d_in, d_out))


ACTIVATIONS = {None: 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}  # gptq_activation


def _activation(what: str, name: Optional[str]) -> int:
    if name not in ACTIVATIONS:
        raise ValueError(f"{what}: unknown activation {name!r}: expected one of {[a for a in ACTIVATIONS if a]} or None")
    return ACTIVATIONS[name]


def _integer_codes(what: str, x, offsets: bool):
    """Codes, scales and sums that a product in integers takes as x."""
    x, x_scales, x_sums = x
    m = x.shape[0]
    if (x.dtype != torch.int8 or x_scales.shape != (m,) or x_scales.dtype != torch.float32
            or not x_scales.is_contiguous() or (x_sums is not None and (x_sums.shape != (m,)
                                                or x_sums.dtype != torch.int32 or not x_sums.is_contiguous()))):
        raise ValueError(f"{what}: expected the codes, scales and sums of gptq_quantize_tokens")
    if offsets and x_sums is None:
        raise ValueError(f"{what}: a layer with offsets needs the sums of the codes")
    return x, x_scales, x_sums


def _integer_layer_ok(what: str, d_in: int, d_out: int, w, w_scales, offsets, bias) -> None:
    if (w.shape != (d_out, d_in) or w.dtype != torch.int8 or not w.is_contiguous() or w_scales.numel() != d_out
            or w_scales.dtype != torch.float32 or not w_scales.is_contiguous()):
        raise ValueError(f"{what}: w and w_scales must be contiguous int8 [d_out, d_in] and float32 [d_out]")
    if offsets is not None and (offsets.shape != (d_out,) or offsets.dtype != torch.int32 or not offsets.is_contiguous()):
        raise ValueError(f"{what}: offsets must be contiguous int32 [d_out]")
    if bias is not None and (bias.shape != (d_out,) or bias.dtype != torch.float32 or not bias.is_contiguous()):
        raise ValueError(f"{what}: a bias must be contiguous float32 [d_out]")


def _integer_y(what: str, m: int, d_out: int, y: torch.Tensor) -> int:
    """The type code of a y that the caller gives."""
    if y.shape != (m, d_out) or not y.is_contiguous():
        raise ValueError(f"{what}: y must be contiguous [m, d_out]")
    return _type_code(what, y.dtype)


def gptq_integer_matmul(x, w: torch.Tensor, w_scales: torch.Tensor, offsets: Optional[torch.Tensor] = None,
                        out_dtype: torch.dtype = torch.float32, y: Optional[torch.Tensor] = None,
                        ws: Optional[torch.Tensor] = None, stream=None, bias: Optional[torch.Tensor] = None,
                        activation: Optional[str] = None, residual: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [m, d_out] = act(x W^T + bias) + residual in 8-bit integers, W = w_scales
    (w - offsets) as laid out by gptq_integer_weight (offsets None: all zero).  x
    is [m, d_in] bf16 or fp32 (rows may be strided), quantized per token on the
    way, or what gptq_quantize_tokens or gptq_norm_tokens returned for it; y may not
    lie over codes or over up to four tokens.
    bias: fp32 [d_out]; activation: "relu", "gelu", "gelu_tanh" or "silu"; residual:
    [m, d_out] bf16 or fp32 (rows may be strided), which y may be itself.  They
    are applied to the sums in fp32 (gptq_integer_linear of the C ABI)."""
    if stream is not None:
        with _on_stream(stream):
            return gptq_integer_matmul(x, w, w_scales, offsets, out_dtype, y, ws, None, bias, activation, residual)
    what = "gptq_integer_matmul"
    x_scales = x_sums = None
    if isinstance(x, tuple):
        x, x_scales, x_sums = _integer_codes(what, x, offsets is not None)
        code = GPTQ_I8
    else:
        code = _type_code(what, x.dtype)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError(f"{what}: x must be 2-D with unit column stride")
    act = 0 if activation is None else _activation(what, activation)
    dev = _on_device(what, x, w, w_scales, offsets, x_scales, x_sums, y, ws, bias, residual)
    m, d_in = x.shape
    d_out = w.shape[0]
    _integer_layer_ok(what, d_in, d_out, w, w_scales, offsets, bias)
    rt = ldr = 0
    if residual is not None:
        rt = _type_code(what, residual.dtype)
        if residual.shape != (m, d_out) or (residual.stride(1) != 1 and d_out > 1):
            raise ValueError(f"{what}: residual must be [m, d_out] with unit column stride")
        ldr = _row_stride(residual)
    if y is None:
        yt = _type_code(what, out_dtype)
        y = x.new_empty((m, d_out), dtype=out_dtype)
    else:
        yt = _integer_y(what, m, d_out, y)
    lib = _lib()
    if ws is None:
        need = lib.gptq_integer_workspace_size(m, code, d_in, d_out)
        if need:
            ws = torch.empty(need, dtype=torch.uint8, device=x.device)
    if bias is None and act == 0 and residual is None:
        st = lib.gptq_integer_matmul(x.data_ptr(), code, _ptr(x_scales), _ptr(x_sums), m, d_in, _row_stride(x),
                                     w.data_ptr(), w_scales.data_ptr(), _ptr(offsets), d_out, y.data_ptr(), yt, _ptr(ws),
                                     _ws_bytes(ws), _raw_stream(dev))
    else:
        layer = _CLayer(w.data_ptr(), w_scales.data_ptr(), _ptr(offsets), _ptr(bias))
        st = lib.gptq_integer_linear(x.data_ptr(), code, _ptr(x_scales), _ptr(x_sums), m, d_in, _row_stride(x), layer, d_out,
                                     act, _ptr(residual), rt, ldr, y.data_ptr(), yt, _ptr(ws), _ws_bytes(ws),
                                     _raw_stream(dev))
    _check(st, what)
    return y


def gptq_integer_gated_workspace_size(m: int, dtype: torch.dtype, d_in: int, d_out: int) -> int:
    """dtype: of x (int8: codes)."""
    code = GPTQ_I8 if dtype == torch.int8 else _type_code("gptq_integer_gated_workspace_size", dtype)
    return int(_lib().gptq_integer_gated_workspace_size(m, code, d_in, d_out))


def gptq_integer_gated(x, gate: Mapping[str, torch.Tensor], up: Mapping[str, torch.Tensor],
                       activation: Optional[str] = "silu", out_dtype: torch.dtype = torch.float32,
                       y: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y [m, d_out] = act(x G^T + bias_g) * (x U^T + bias_u) in 8-bit integers, both
    products in one kernel.  gate, up: layers as checkpoint.integer_layer gives
    them ("w", "scales" and optionally "offsets"), and optionally a "bias" (fp32
    [d_out]); x and activation as for gptq_integer_matmul."""
    if stream is not None:
        with _on_stream(stream):
            return gptq_integer_gated(x, gate, up, activation, out_dtype, y, ws)
    what = "gptq_integer_gated"
    (gw, gs, go, gb), (uw, us, uo, ub) = ((t["w"], t["scales"], t.get("offsets"), t.get("bias")) for t in (gate, up))
    x_scales = x_sums = None
    if isinstance(x, tuple):
        x, x_scales, x_sums = _integer_codes(what, x, go is not None or uo is not None)
        code = GPTQ_I8
    else:
        code = _type_code(what, x.dtype)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError(f"{what}: x must be 2-D with unit column stride")
    act = _activation(what, activation)
    dev = _on_device(what, x, gw, gs, go, gb, uw, us, uo, ub, x_scales, x_sums, y, ws)
    m, d_in = x.shape
    d_out = gw.shape[0]
    _integer_layer_ok(what, d_in, d_out, gw, gs, go, gb)
    _integer_layer_ok(what, d_in, d_out, uw, us, uo, ub)
    if y is None:
        yt = _type_code(what, out_dtype)
        y = x.new_empty((m, d_out), dtype=out_dtype)
    else:
        yt = _integer_y(what, m, d_out, y)
    lib = _lib()
    if ws is None:
        need = lib.gptq_integer_gated_workspace_size(m, code, d_in, d_out)
        if need:
            ws = torch.empty(need, dtype=torch.uint8, device=x.device)
    g = _CLayer(gw.data_ptr(), gs.data_ptr(), _ptr(go), _ptr(gb))
    u = _CLayer(uw.data_ptr(), us.data_ptr(), _ptr(uo), _ptr(ub))
    _check(lib.gptq_integer_gated(x.data_ptr(), code, _ptr(x_scales), _ptr(x_sums), m, d_in, _row_stride(x), g, u, d_out, act,
                                  y.data_ptr(), yt, _ptr(ws), _ws_bytes(ws), _raw_stream(dev)), what)
    return y


def gptq_norm_tokens(x: torch.Tensor, weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                     eps: float = 1e-6, dtype: torch.dtype = torch.int8, total: Optional[torch.Tensor] = None,
                     y: Optional[torch.Tensor] = None, stream=None):
    """The root-mean-square norm of the rows of h = x + residual, times weight:
    returns (rows, total).  x [m, d] and residual (None: h = x) are bf16 or fp32,
    rows may be strided; weight [d] bf16 or fp32 (None: ones).
    rows, for dtype int8: (codes, scales, sums) as gptq_quantize_tokens returns
    them, which the products in integers take as x; for bfloat16 or float32: y
    [m, d].  y given beside codes: it is written too.  total: h in the residual's type
    (x itself without a residual), written to the given tensor, which may be the
    residual or x, or to a new one."""
    if stream is not None:
        with _on_stream(stream):
            return gptq_norm_tokens(x, weight, residual, eps, dtype, total, y)
    what = "gptq_norm_tokens"
    if x.dim() != 2 or (x.stride(1) != 1 and x.shape[1] > 1):
        raise ValueError(f"{what}: x must be 2-D with unit column stride")
    m, d = x.shape
    xt = _type_code(what, x.dtype)
    rt = wt = yt = ldr = lds = 0
    dev = _on_device(what, x, weight, residual, total, y)
    if weight is not None:
        wt = _type_code(what, weight.dtype)
        if weight.shape != (d,) or (weight.stride(0) != 1 and d > 1):
            raise ValueError(f"{what}: weight must be [d], contiguous")
    if residual is None:
        if total is not None:
            raise ValueError(f"{what}: without a residual there is no total to write")
    else:
        rt = _type_code(what, residual.dtype)
        if residual.shape != (m, d) or (residual.stride(1) != 1 and d > 1):
            raise ValueError(f"{what}: residual must be like x, with unit column stride")
        if total is None:
            total = torch.empty((m, d), dtype=residual.dtype, device=x.device)
        elif total.shape != (m, d) or total.dtype != residual.dtype or (total.stride(1) != 1 and d > 1):
            raise ValueError(f"{what}: total must be like the residual, with unit column stride")
        ldr, lds = _row_stride(residual), _row_stride(total)
    codes = scales = sums = None
    if dtype == torch.int8:
        codes = x.new_empty((m, d), dtype=torch.int8)
        scales, sums = x.new_empty(m, dtype=torch.float32), x.new_empty(m, dtype=torch.int32)
    elif y is None:
        y = x.new_empty((m, d), dtype=dtype)
    if y is not None:
        yt = _type_code(what, y.dtype)
        if y.shape != (m, d) or not y.is_contiguous() or (codes is None and y.dtype != dtype):
            raise ValueError(f"{what}: y must be contiguous [m, d]" + ("" if codes is not None else f" {dtype}"))
    _check(_lib().gptq_norm_tokens(x.data_ptr(), xt, m, d, _row_stride(x), _ptr(residual), rt, ldr, _ptr(weight), wt, eps,
                                   _ptr(total), lds, _ptr(y), yt, _ptr(codes), _ptr(scales), _ptr(sums), _raw_stream(dev)),
           what)
    return (y if codes is None else (codes, scales, sums)), (x if residual is None else total)


class QuantizedCache:
    """A paged key/value cache in 8- or 4-bit codes (gptq_cache of the C ABI)
    over the caller's tensors: codes [n_pages, n_kv_heads, page_size,
    head_dim * bits / 8] (int8 for 8 bits, uint8 for 4), scales [n_pages,
    n_kv_heads, page_size] fp32, all contiguous and on one GPU."""

    def __init__(self, k_codes: torch.Tensor, v_codes: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
                 bits: int = 8):
        what = "QuantizedCache"
        if bits not in (4, 8):
            raise ValueError(f"{what}: bits must be 4 or 8, got {bits}")
        if k_codes.dim() != 4:
            raise ValueError(f"{what}: codes must be [n_pages, n_kv_heads, page_size, head_dim * bits / 8]")
        n_pages, n_kv, page, width = k_codes.shape
        dtype = torch.int8 if bits == 8 else torch.uint8
        for t in (k_codes, v_codes):
            if t.shape != k_codes.shape or t.dtype != dtype or not t.is_contiguous() or not t.is_cuda:
                raise ValueError(f"{what}: k_codes and v_codes must be alike: contiguous {dtype} on the GPU")
        for t in (k_scales, v_scales):
            if t.shape != (n_pages, n_kv, page) or t.dtype != torch.float32 or not t.is_contiguous():
                raise ValueError(f"{what}: scales must be contiguous float32 [n_pages, n_kv_heads, page_size]")
        if any(t.get_device() != k_codes.get_device() for t in (v_codes, k_scales, v_scales)):
            raise ValueError(f"{what}: the tensors must be on one GPU")
        if page not in (16, 32, 64, 128, 256):
            raise ValueError(f"{what}: page_size must be 16, 32, 64, 128 or 256, got {page}")
        self.head_dim = width * 8 // bits
        if self.head_dim % 16 != 0 or not 16 <= self.head_dim <= 256:
            raise ValueError(f"{what}: head_dim must be a multiple of 16 up to 256, got {self.head_dim}")
        if n_pages < 1 or n_kv < 1:
            raise ValueError(f"{what}: a cache needs a page and a head")
        self.n_pages, self.n_kv_heads, self.page_size, self.bits = n_pages, n_kv, page, bits
        self.k_codes, self.v_codes, self.k_scales, self.v_scales = k_codes, v_codes, k_scales, v_scales
        self.device = k_codes.device
        self._index = k_codes.get_device()
        self._c = _CCache(n_pages, page, n_kv, self.head_dim, bits, k_codes.data_ptr(), v_codes.data_ptr(),
                          k_scales.data_ptr(), v_scales.data_ptr())
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, bits: int = 8,
              device="cuda:0") -> "QuantizedCache":
        """A cache of zeros."""
        if bits not in (4, 8):
            raise ValueError(f"QuantizedCache: bits must be 4 or 8, got {bits}")
        if head_dim % 16 != 0 or not 16 <= head_dim <= 256:
            raise ValueError(f"QuantizedCache: head_dim must be a multiple of 16 up to 256, got {head_dim}")
        shape = (n_pages, n_kv_heads, page_size)
        dtype = torch.int8 if bits == 8 else torch.uint8
        codes = [torch.full((*shape, head_dim * bits // 8), 0 if bits == 8 else 0x88, dtype=dtype, device=device)
                 for _ in range(2)]
        scales = [torch.zeros(shape, dtype=torch.float32, device=device) for _ in range(2)]
        return cls(*codes, *scales, bits)

    def _here(self, what: str, *ts) -> int:
        dev = _on_device(what, *ts)
        if dev != self._index:
            raise ValueError(f"{what}: the cache is on cuda:{self._index}, not on the current GPU")
        return dev


def _heads_together(t: torch.Tensor) -> bool:
    """Of [tokens, heads, head_dim]: a token's heads lie one behind the other.  The
    stride of a single head, and any of no tokens, says nothing."""
    n, heads, hd = t.shape
    return n == 0 or (t.stride(2) == 1 and (heads == 1 or t.stride(1) == hd))


def _slots(what: str, slots: torch.Tensor) -> int:
    if slots.dim() != 1 or slots.dtype != torch.int64 or not slots.is_contiguous():
        raise ValueError(f"{what}: slots must be a contiguous int64 vector")
    return slots.shape[0]


def gptq_cache_write(cache: QuantizedCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
    """Quantize k, v [n, n_kv_heads, head_dim] (bf16 or fp32; tokens may be
    strided, as in a slice of a fused projection) into the cache's slots
    (page * page_size + offset; int64 [n], different from each other; one
    outside the cache is skipped)."""
    if stream is not None:
        with _on_stream(stream):
            return gptq_cache_write(cache, k, v, slots)
    what = "gptq_cache_write"
    n = _slots(what, slots)
    code = _type_code(what, k.dtype)
    heads, hd = cache.n_kv_heads, cache.head_dim
    shape = (n, heads, hd)
    if k.shape != shape or v.shape != shape or k.dtype != v.dtype or not _heads_together(k) or not _heads_together(v):
        raise ValueError(f"{what}: k and v must be [n, {heads}, {hd}] of one dtype, heads contiguous")
    dev = cache._here(what, k, v, slots)
    ldk, ldv = (k.stride(0), v.stride(0)) if n > 1 else (heads * hd, heads * hd)
    _check(_lib().gptq_cache_write(cache._ref, k.data_ptr(), v.data_ptr(), code, n, ldk, ldv, slots.data_ptr(),
                                   _raw_stream(dev)), what)


def gptq_cache_read(cache: QuantizedCache, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                    k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None, stream=None):
    """The values held in the given slots: (k, v), each [n, n_kv_heads,
    head_dim]; zeros for a slot outside the cache."""
    if stream is not None:
        with _on_stream(stream):
            return gptq_cache_read(cache, slots, dtype, k, v)
    what = "gptq_cache_read"
    n = _slots(what, slots)
    shape = (n, cache.n_kv_heads, cache.head_dim)
    code = _type_code(what, dtype if k is None else k.dtype)
    k = torch.empty(shape, dtype=dtype, device=slots.device) if k is None else k
    v = torch.empty_like(k) if v is None else v
    if k.shape != shape or v.shape != shape or k.dtype != v.dtype or not k.is_contiguous() or not v.is_contiguous():
        raise ValueError(f"{what}: k and v must be contiguous [n, n_kv_heads, head_dim] of one dtype")
    dev = cache._here(what, slots, k, v)
    _check(_lib().gptq_cache_read(cache._ref, slots.data_ptr(), n, k.data_ptr(), v.data_ptr(), code,
                                  _raw_stream(dev)), what)
    return k, v


def gptq_attention_workspace_size(cache: QuantizedCache, n_tokens: int, n_heads: int, n_seq: int,
                                  pages_per_seq: int) -> int:
    return int(_lib().gptq_attention_workspace_size(cache._ref, n_tokens, n_heads, n_seq, pages_per_seq))


def gptq_cache_attention(q: torch.Tensor, cache: QuantizedCache, page_table: torch.Tensor, q_starts: torch.Tensor,
                         kv_lens: torch.Tensor, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                         ws: Optional[torch.Tensor] = None, stream=None, cap: Optional[float] = None,
                         slopes: Optional[torch.Tensor] = None, prefix_lens: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Causal attention of the new tokens q [n_tokens, n_heads, head_dim] bf16
    over the cache, which holds their keys and values already.  Sequence i owns
    the tokens q_starts[i] .. q_starts[i + 1] - 1 (int32 [n_seq + 1]), has
    kv_lens[i] keys (int32 [n_seq]) and its pages in page_table[i] (int32
    [n_seq, pages_per_seq]).  scale: 1 / sqrt(head_dim) unless given.  Rows of
    out outside the sequences are left as they were.
    cap: scores s become cap tanh(s / cap), 2^-20 <= cap <= 2^20.  slopes: fp32
    [n_heads]; slope |a - j| is then taken off the score of key j for the token
    at place a.  prefix_lens: int32 [n_seq]; every token of a sequence sees that
    many first keys (gptq_cache_attention_scores of the C ABI)."""
    if stream is not None:
        with _on_stream(stream):
            return gptq_cache_attention(q, cache, page_table, q_starts, kv_lens, scale, out, ws, None, cap, slopes, prefix_lens)
    what = "gptq_cache_attention"
    hd = cache.head_dim
    if q.dim() != 3 or q.shape[2] != hd or q.dtype != torch.bfloat16:
        raise ValueError(f"{what}: q must be bfloat16 [n_tokens, n_heads, {hd}]")
    n, heads = q.shape[0], q.shape[1]
    if heads < 1 or heads % cache.n_kv_heads != 0:
        raise ValueError(f"{what}: {heads} query heads do not divide over {cache.n_kv_heads} key heads")
    if not _heads_together(q):
        raise ValueError(f"{what}: the heads of a token must be contiguous in q")
    if (page_table.dim() != 2 or page_table.dtype != torch.int32 or not page_table.is_contiguous()
            or kv_lens.dtype != torch.int32 or q_starts.dtype != torch.int32 or not kv_lens.is_contiguous()
            or not q_starts.is_contiguous() or kv_lens.shape != (page_table.shape[0],)
            or q_starts.shape != (page_table.shape[0] + 1,)):
        raise ValueError(f"{what}: page_table, q_starts and kv_lens must be contiguous int32 [n_seq, pages_per_seq], "
                         "[n_seq + 1] and [n_seq]")
    width = heads * hd
    if out is None:
        out = q.new_empty((n, heads, hd))
    elif out.shape != q.shape or out.dtype != torch.bfloat16 or not _heads_together(out):
        raise ValueError(f"{what}: out must be bfloat16 like q, the heads of a token contiguous")
    if slopes is not None and (slopes.shape != (heads,) or slopes.dtype != torch.float32 or not slopes.is_contiguous()):
        raise ValueError(f"{what}: slopes must be contiguous float32 [n_heads]")
    if prefix_lens is not None and (prefix_lens.shape != kv_lens.shape or prefix_lens.dtype != torch.int32
                                    or not prefix_lens.is_contiguous()):
        raise ValueError(f"{what}: prefix_lens must be contiguous int32 [n_seq]")
    if cap is not None and not 2.0 ** -20 <= cap <= 2.0 ** 20:
        raise ValueError(f"{what}: cap must lie in [2^-20, 2^20], got {cap}")
    dev = cache._here(what, q, page_table, q_starts, kv_lens, out, ws, slopes, prefix_lens)
    n_seq, pages = page_table.shape
    ldq, ldo = (q.stride(0), out.stride(0)) if n > 1 else (width, width)
    lib = _lib()
    if ws is None:
        need = lib.gptq_attention_workspace_size(cache._ref, n, heads, n_seq, pages)
        if need:
            ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    scale = hd ** -0.5 if scale is None else scale
    if cap is None and slopes is None and prefix_lens is None:
        st = lib.gptq_cache_attention(cache._ref, q.data_ptr(), GPTQ_BF16, n, ldq, heads, page_table.data_ptr(), pages,
                                      q_starts.data_ptr(), kv_lens.data_ptr(), n_seq, scale, out.data_ptr(), ldo, _ptr(ws),
                                      _ws_bytes(ws), _raw_stream(dev))
    else:
        scores = _CScores(cap or 0.0, _ptr(slopes), _ptr(prefix_lens))
        st = lib.gptq_cache_attention_scores(cache._ref, q.data_ptr(), GPTQ_BF16, n, ldq, heads, page_table.data_ptr(), pages,
                                             q_starts.data_ptr(), kv_lens.data_ptr(), n_seq, scale, scores, out.data_ptr(),
                                             ldo, _ptr(ws), _ws_bytes(ws), _raw_stream(dev))
    _check(st, what)
    return out
