"""Python binding of libosc (include/osc.h): OSC W4A4 linear layers on MI355X (gfx950).

Argument marshalling only.  Every step runs in the HIP kernels of libosc.so;
there is no CPU fallback: importing this package fails loudly when the library
has not been built (``python w4a4_outlier_split_amd/build.py``).

Device buffers are torch tensors on a ROCm device (their ``data_ptr()`` is
passed through); table slices ``L`` are host arrays (numpy int32 or anything
``numpy.asarray`` accepts) or None.  ``stream=None`` means torch's current
stream on the current device.  A non-OK status raises :class:`OscError`.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np
# torch first: its HIP runtime must be the process's only one.  libosc's dependency on
# libamdhip64.so.7 then resolves to the runtime torch has already loaded; a second copy
# loaded ahead of torch does not see the device.
import torch  # noqa: F401

_HERE = os.path.dirname(os.path.abspath(__file__))
# OSC_LIBRARY names another build of the same library (the host-sanitizer build of the tests)
LIB_PATH = os.environ.get("OSC_LIBRARY") or os.path.join(_HERE, "_build", "libosc.so")

OSC_MXFP4 = 0
OSC_MXFP8 = 1
OSC_FP6P = 2  # G = 16 pairs: E3M2 codes, one E8M0 scale per 32 channels
OSC_Y_BF16 = 0
OSC_Y_F32 = 1
OSC_MAX_GROUPS = 1024
OSC_MAX_CHANNELS = 3
OSC_MAX_REQUESTS = 4096
OSC_MAX_TREE = 256    # nodes of a request's tree of drafted tokens
OSC_MAX_TOP = 64      # alternatives of osc_logprobs
OSC_MAX_LAYERS = 128  # layers of one osc_tree_commit

STATUS = {0: "OSC_OK", 1: "OSC_E_NULL", 2: "OSC_E_SHAPE", 3: "OSC_E_TABLE", 4: "OSC_E_ALIGN",
          5: "OSC_E_FORMAT", 6: "OSC_E_DEVICE"}

EXPORTS = ("osc_pack_weights", "osc_quant_act", "osc_gemm", "osc_gemm_fp8", "osc_build_table",
           "osc_pack_weights_multi", "osc_quant_act_multi", "osc_gemm_multi", "osc_build_table_multi",
           "osc_swiglu_quant", "osc_swiglu", "osc_linear_decode", "osc_gemm_fp6p", "osc_rmsnorm_quant",
           "osc_rmsnorm", "osc_page_plan", "osc_qkv_append", "osc_attn_workspace", "osc_attn_paged", "osc_tree_plan",
           "osc_attn_tree_workspace", "osc_attn_tree", "osc_logprobs_workspace", "osc_logprobs", "osc_tree_accept",
           "osc_tree_commit", "osc_status_str", "osc_last_device_error")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libosc.so is not built ({LIB_PATH}); run python w4a4_outlier_split_amd/build.py")

_lib = ctypes.CDLL(LIB_PATH)
_P = ctypes.c_void_p
_I = ctypes.c_int
_D = ctypes.c_double
_F = ctypes.c_float
_L = ctypes.c_int64
_lib.osc_pack_weights.argtypes = [_P, _I, _I, _I, _P, _I, _P, _P, _P, _P]
_lib.osc_quant_act.argtypes = [_P, _I, _I, _I, _P, _I, _P, _P, _P, _P]
_lib.osc_gemm.argtypes = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _I, _P]
_lib.osc_gemm_fp8.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _I, _P]
_lib.osc_build_table.argtypes = [_P, _I, _I, _I, _D, _D, _P, _P, _P, _P]
_lib.osc_pack_weights_multi.argtypes = [_P, _I, _I, _I, _P, _I, _I, _P, _P, _P, _P]
_lib.osc_quant_act_multi.argtypes = [_P, _I, _I, _I, _P, _I, _I, _P, _P, _P, _P]
_lib.osc_gemm_multi.argtypes = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _I, _P]
_lib.osc_build_table_multi.argtypes = [_P, _I, _I, _I, _D, _D, _I, _P, _P, _P, _P]
_lib.osc_swiglu_quant.argtypes = [_P, _I, _I, _I, _P, _I, _I, _P, _P, _P, _P]
_lib.osc_swiglu.argtypes = [_P, _I, _I, _P, _P]
_lib.osc_linear_decode.argtypes = [_P, _I, _I, _I, _P, _I, _P, _P, _P, _I, _P, _I, _P]
_lib.osc_gemm_fp6p.argtypes = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _I, _P]
_lib.osc_rmsnorm_quant.argtypes = [_P, _P, _P, _I, _I, _F, _I, _P, _I, _I, _P, _P, _P, _P, _P]
_lib.osc_rmsnorm.argtypes = [_P, _P, _P, _I, _I, _F, _P, _P, _P]
_lib.osc_page_plan.argtypes = [_P, _P, _I, _I, _I, _P, _I, _P, _I, _P, _I, _P, _P, _P, _P, _P, _P]
_lib.osc_qkv_append.argtypes = [_P, _I, _I, _I, _I, _P, _P, _F, _P, _I, _P, _P, _P, _P, _P, _I, _I, _P]
_lib.osc_attn_workspace.argtypes = [_I, _I, _I, _I, _I, _I, _I, _P]
_lib.osc_attn_paged.argtypes = [_P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _F, _P, _P, _L, _P]
_lib.osc_tree_plan.argtypes = [_P, _P, _P, _I, _I, _I, _P, _P, _P]
_lib.osc_attn_tree_workspace.argtypes = [_I, _I, _I, _I, _I, _I, _I, _I, _P]
_lib.osc_attn_tree.argtypes = [_P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _I, _F, _P, _P, _L, _P]
_lib.osc_logprobs_workspace.argtypes = [_I, _I, _I, _P]
_lib.osc_logprobs.argtypes = [_P, _I, _I, _I, _I, _F, _P, _I, _I, _P, _P, _P, _P, _P, _L, _P]
_lib.osc_tree_accept.argtypes = [_P, _P, _P, _I, _P, _P, _I, _P, _I, _I, _I, _P, _P, _P, _P]
_lib.osc_tree_commit.argtypes = [_P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _I, _I, _I, _P]
for _f in EXPORTS[:-2]:
    getattr(_lib, _f).restype = _I
_lib.osc_status_str.argtypes = [_I]
_lib.osc_status_str.restype = ctypes.c_char_p
_lib.osc_last_device_error.argtypes = []
_lib.osc_last_device_error.restype = ctypes.c_char_p


def code_bytes(rows: int, H: int, fmt: int) -> int:
    """Bytes of a tiled code buffer (QX / QW) for ``rows`` rows of H channels."""
    return rows * (H // 2 if fmt == OSC_MXFP4 else H if fmt == OSC_MXFP8 else 3 * H // 4)


def scale_bytes(rows: int, H: int, G: int, fmt: int = OSC_MXFP4) -> int:
    """Bytes of a tiled E8M0 scale buffer (SX / SW): one per row and group (per pair of 16-groups
    for OSC_FP6P)."""
    return rows * (H // 32 if fmt == OSC_FP6P else H // G)


def side_elems(rows: int, H: int, G: int, m: int = 1) -> int:
    """bf16 elements of a tiled B / W_L buffer: m*K compensation columns in panels of 32, the
    last one padded."""
    return rows * ((m * (H // G) + 31) // 32) * 32


class OscError(RuntimeError):
    def __init__(self, status: int, call: str, detail: str = ""):
        self.status = status
        msg = f"{call}: {osc_status_str(status)}"
        if detail:
            msg += f" ({detail})"
        if status == 6:
            msg += f" ({_lib.osc_last_device_error().decode()})"
        super().__init__(msg)


def osc_status_str(status: int) -> str:
    return _lib.osc_status_str(int(status)).decode()


def _ptr(t) -> Optional[int]:
    """Device pointer of a tensor (or an int address), None for None."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _table(L):
    if L is None:
        return None, None
    arr = np.ascontiguousarray(np.asarray(L), dtype=np.int32)
    return arr, arr.ctypes.data_as(ctypes.c_void_p)


# the current stream's handle without a Stream object around it (2.7 us a call), where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> Optional[int]:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, call: str) -> None:
    if status != 0:
        raise OscError(status, call)


def osc_pack_weights(W, N: int, H: int, G: int, L, wfmt: int, QW, SW, WL, stream=None) -> None:
    keep, lp = _table(L)
    _check(_lib.osc_pack_weights(_ptr(W), N, H, G, lp, wfmt, _ptr(QW), _ptr(SW), _ptr(WL), _stream(stream)),
           "osc_pack_weights")


def osc_quant_act(X, S: int, H: int, G: int, L, afmt: int, QX, SX, B, stream=None) -> None:
    keep, lp = _table(L)
    _check(_lib.osc_quant_act(_ptr(X), S, H, G, lp, afmt, _ptr(QX), _ptr(SX), _ptr(B), _stream(stream)),
           "osc_quant_act")


def osc_gemm(QX, SX, B, QW, SW, WL, S: int, N: int, H: int, G: int, Y, yt: int, stream=None) -> None:
    _check(_lib.osc_gemm(_ptr(QX), _ptr(SX), _ptr(B), _ptr(QW), _ptr(SW), _ptr(WL), S, N, H, G, _ptr(Y), yt,
                         _stream(stream)), "osc_gemm")


def osc_gemm_fp8(QX8, SX, QW, SW, wfmt: int, S: int, N: int, H: int, G: int, Y, yt: int, stream=None) -> None:
    _check(_lib.osc_gemm_fp8(_ptr(QX8), _ptr(SX), _ptr(QW), _ptr(SW), wfmt, S, N, H, G, _ptr(Y), yt,
                             _stream(stream)), "osc_gemm_fp8")


def osc_build_table(Xcal, R: int, H: int, G: int, alpha: float, rho: float, L, hits, events, stream=None) -> None:
    _check(_lib.osc_build_table(_ptr(Xcal), R, H, G, float(alpha), float(rho), _ptr(L), _ptr(hits), _ptr(events),
                                _stream(stream)), "osc_build_table")


# ---- several protected channels per group (L: m entries per group, [K, m] or flat K*m)

def osc_pack_weights_multi(W, N: int, H: int, G: int, L, m: int, wfmt: int, QW, SW, WL, stream=None) -> None:
    keep, lp = _table(L)
    _check(_lib.osc_pack_weights_multi(_ptr(W), N, H, G, lp, m, wfmt, _ptr(QW), _ptr(SW), _ptr(WL),
                                       _stream(stream)), "osc_pack_weights_multi")


def osc_quant_act_multi(X, S: int, H: int, G: int, L, m: int, afmt: int, QX, SX, B, stream=None) -> None:
    keep, lp = _table(L)
    _check(_lib.osc_quant_act_multi(_ptr(X), S, H, G, lp, m, afmt, _ptr(QX), _ptr(SX), _ptr(B), _stream(stream)),
           "osc_quant_act_multi")


def osc_swiglu_quant(GU, S: int, F: int, G: int, L, m: int, afmt: int, QX, SX, B, stream=None) -> None:
    """GU: [S, 2F] bf16 (gate | up) -> the tiled quantized h = silu(gate) * up (W2's input)."""
    keep, lp = _table(L)
    _check(_lib.osc_swiglu_quant(_ptr(GU), S, F, G, lp, m, afmt, _ptr(QX), _ptr(SX), _ptr(B), _stream(stream)),
           "osc_swiglu_quant")


def osc_gemm_fp6p(QX, SX, B, QW, SW, WL, S: int, N: int, H: int, m: int, Y, yt: int, stream=None) -> None:
    """G = 16 on E3M2 pairs (operands from the quant / pack calls with fmt OSC_FP6P, G = 16)."""
    _check(_lib.osc_gemm_fp6p(_ptr(QX), _ptr(SX), _ptr(B), _ptr(QW), _ptr(SW), _ptr(WL), S, N, H, m, _ptr(Y), yt,
                              _stream(stream)), "osc_gemm_fp6p")


def osc_linear_decode(X, S: int, H: int, G: int, L, m: int, QW, SW, WL, N: int, Y, yt: int, stream=None) -> None:
    """S <= 32: quantization of X fused into the GEMM; Y equals quant_act_multi + gemm_multi."""
    keep, lp = _table(L)
    _check(_lib.osc_linear_decode(_ptr(X), S, H, G, lp, m, _ptr(QW), _ptr(SW), _ptr(WL), N, _ptr(Y), yt,
                                  _stream(stream)), "osc_linear_decode")


def osc_swiglu(GU, S: int, F: int, Hout, stream=None) -> None:
    """GU: [S, 2F] bf16 (gate | up) -> Hout [S, F] bf16 = silu(gate) * up."""
    _check(_lib.osc_swiglu(_ptr(GU), S, F, _ptr(Hout), _stream(stream)), "osc_swiglu")


def osc_gemm_multi(QX, SX, B, QW, SW, WL, S: int, N: int, H: int, G: int, m: int, Y, yt: int, stream=None) -> None:
    _check(_lib.osc_gemm_multi(_ptr(QX), _ptr(SX), _ptr(B), _ptr(QW), _ptr(SW), _ptr(WL), S, N, H, G, m, _ptr(Y),
                               yt, _stream(stream)), "osc_gemm_multi")


def osc_build_table_multi(Xcal, R: int, H: int, G: int, alpha: float, rho: float, m: int, L, hits, events,
                          stream=None) -> None:
    _check(_lib.osc_build_table_multi(_ptr(Xcal), R, H, G, float(alpha), float(rho), m, _ptr(L), _ptr(hits),
                                      _ptr(events), _stream(stream)), "osc_build_table_multi")


# ---- between the projections: norm, paged cache, attention

_BF16 = (torch.bfloat16, torch.int16, torch.uint16)  # the values or their bits
_I32 = (torch.int32,)
_F32 = (torch.float32,)


def _at(call: str, dev: int, t, need: int, types=None) -> Optional[int]:
    """Address of a tensor (or an address, or None) of which the call reads or writes ``need`` contiguous
    bytes on the current device ``dev``; types: those that the elements may have, None for plain bytes."""
    if t is None or type(t) is int:
        return t
    if t.get_device() != dev:
        raise OscError(2, call, f"a tensor on {t.device}, the current device is cuda:{dev}")
    if types is not None and t.dtype not in types:
        raise OscError(5, call, f"a tensor of {t.dtype} where {types[0]} is read or written")
    if not t.is_contiguous() or t.nbytes < need:
        raise OscError(2, call, f"a tensor of {t.nbytes} bytes, strides {tuple(t.stride())}, where {need} contiguous "
                                "bytes are needed")
    return t.data_ptr()


def osc_rmsnorm_quant(X, RES, W, S: int, H: int, eps: float, G: int, L, m: int, afmt: int, RES_OUT, QX, SX, B,
                      stream=None) -> None:
    """r = X + RES to RES_OUT (both None: r = X); the RMS norm of r, quantized as osc_quant_act_multi."""
    c = "osc_rmsnorm_quant"
    keep, lp = _table(L)
    n = 2 * S * H
    g = max(G, 1)  # the library refuses a group size it does not have
    if keep is not None and keep.size < H // g * m:
        raise OscError(3, c, f"{keep.size} table entries for {H // g} groups of {m}")
    d = torch.cuda.current_device()
    _check(_lib.osc_rmsnorm_quant(_at(c, d, X, n, _BF16), _at(c, d, RES, n, _BF16), _at(c, d, W, 2 * H, _BF16),
                                  S, H, eps, G, lp, m, afmt, _at(c, d, RES_OUT, n, _BF16), _at(c, d, QX, code_bytes(S, H, afmt)),
                                  _at(c, d, SX, scale_bytes(S, H, g, afmt)), _at(c, d, B, 2 * side_elems(S, H, g, m), _BF16),
                                  _stream(stream)), c)


def osc_rmsnorm(X, RES, W, S: int, H: int, eps: float, RES_OUT, Y, stream=None) -> None:
    """The same norm written out: Y [S, H] bf16."""
    c = "osc_rmsnorm"
    n = 2 * S * H
    d = torch.cuda.current_device()
    _check(_lib.osc_rmsnorm(_at(c, d, X, n, _BF16), _at(c, d, RES, n, _BF16), _at(c, d, W, 2 * H, _BF16),
                            S, H, eps, _at(c, d, RES_OUT, n, _BF16), _at(c, d, Y, n, _BF16), _stream(stream)), c)


def osc_page_plan(CTX, NEW, R: int, page: int, NP: int, FREE, F: int, HEAD, T: int, TABLE, MB: int, CU, KV, SLOT, POS, USED,
                  stream=None) -> None:
    """Page tables and slot maps of one step from request lengths (all int32 device tensors)."""
    c = "osc_page_plan"
    d = torch.cuda.current_device()
    _check(_lib.osc_page_plan(_at(c, d, CTX, 4 * R, _I32), _at(c, d, NEW, 4 * R, _I32), R, page, NP,
                              _at(c, d, FREE, 4 * F, _I32), F, _at(c, d, HEAD, 4, _I32), T, _at(c, d, TABLE, 4 * R * MB, _I32), MB,
                              _at(c, d, CU, 4 * R + 4, _I32), _at(c, d, KV, 4 * R, _I32), _at(c, d, SLOT, 4 * T, _I32),
                              _at(c, d, POS, 4 * T, _I32), _at(c, d, USED, 4, _I32), _stream(stream)), c)


def osc_qkv_append(QKV, S: int, HQ: int, HKV: int, D: int, WQ, WK, eps: float, CS, P: int, POS, SLOT, Q, KC, VC, NP: int,
                   page: int, stream=None) -> None:
    """QKV rows [S, (HQ + 2 HKV) D]: normed and rotated queries to Q, keys and values to their slots."""
    c = "osc_qkv_append"
    d = torch.cuda.current_device()
    n = 2 * NP * HKV * page * D
    _check(_lib.osc_qkv_append(_at(c, d, QKV, 2 * S * (HQ + 2 * HKV) * D, _BF16), S, HQ, HKV, D,
                               _at(c, d, WQ, 2 * D, _BF16), _at(c, d, WK, 2 * D, _BF16), eps, _at(c, d, CS, 4 * P * D, _F32), P,
                               _at(c, d, POS, 4 * S, _I32), _at(c, d, SLOT, 4 * S, _I32), _at(c, d, Q, 2 * S * HQ * D, _BF16),
                               _at(c, d, KC, n, _BF16), _at(c, d, VC, n, _BF16), NP, page, _stream(stream)), c)


def osc_attn_workspace(S: int, R: int, HQ: int, HKV: int, D: int, page: int, MB: int) -> int:
    """Bytes of the workspace that osc_attn_paged needs at these sizes."""
    n = _L(0)
    _check(_lib.osc_attn_workspace(S, R, HQ, HKV, D, page, MB, ctypes.byref(n)), "osc_attn_workspace")
    return n.value


def osc_attn_paged(Q, KC, VC, S: int, R: int, HQ: int, HKV: int, D: int, page: int, MB: int, NP: int, TABLE, CU, KV,
                   scale: float, O, WS, stream=None) -> None:
    """Causal attention of the new tokens of R requests over the paged cache; WS: a tensor (or the
    address) of at least osc_attn_workspace bytes, or None where that is 0."""
    c = "osc_attn_paged"
    d = torch.cuda.current_device()
    n, q = 2 * NP * HKV * page * D, 2 * S * HQ * D
    # the caller of an address answers for its bytes, as everywhere
    ws = 0 if WS is None else osc_attn_workspace(S, R, HQ, HKV, D, page, MB) if type(WS) is int else WS.nbytes
    _check(_lib.osc_attn_paged(_at(c, d, Q, q, _BF16), _at(c, d, KC, n, _BF16), _at(c, d, VC, n, _BF16), S, R, HQ, HKV, D, page,
                               MB, NP, _at(c, d, TABLE, 4 * R * MB, _I32), _at(c, d, CU, 4 * R + 4, _I32), _at(c, d, KV, 4 * R, _I32),
                               scale, _at(c, d, O, q, _BF16), _at(c, d, WS, 0), ws, _stream(stream)), c)


# ---- steps with drafted tokens

_U64 = (torch.uint64, torch.int64)  # bit masks


def osc_tree_plan(PARENT, CU, CTX, R: int, T: int, N: int, POS, MASK, stream=None) -> None:
    """Positions POS [T] and masks MASK [T, ceil(N / 64)] (64-bit) of the nodes of R requests' trees of at most N nodes."""
    c = "osc_tree_plan"
    d = torch.cuda.current_device()
    _check(_lib.osc_tree_plan(_at(c, d, PARENT, 4 * T, _I32), _at(c, d, CU, 4 * R + 4, _I32), _at(c, d, CTX, 4 * R, _I32), R, T, N,
                              _at(c, d, POS, 4 * T, _I32), _at(c, d, MASK, 8 * T * ((N + 63) // 64), _U64), _stream(stream)), c)


def osc_attn_tree_workspace(S: int, R: int, HQ: int, HKV: int, D: int, page: int, MB: int, N: int) -> int:
    """Bytes of the workspace that osc_attn_tree needs at these sizes."""
    n = _L(0)
    _check(_lib.osc_attn_tree_workspace(S, R, HQ, HKV, D, page, MB, N, ctypes.byref(n)), "osc_attn_tree_workspace")
    return n.value


def osc_attn_tree(Q, KC, VC, S: int, R: int, HQ: int, HKV: int, D: int, page: int, MB: int, NP: int, TABLE, CU, KV, MASK, N: int,
                  scale: float, O, WS, stream=None) -> None:
    """Attention of R requests' trees over the paged cache: each token sees its request's context and the new keys in its
    MASK [S, ceil(N / 64)] (64-bit); WS: a tensor (or the address) of at least osc_attn_tree_workspace bytes."""
    c = "osc_attn_tree"
    d = torch.cuda.current_device()
    n, q = 2 * NP * HKV * page * D, 2 * S * HQ * D
    ws = 0 if WS is None else osc_attn_tree_workspace(S, R, HQ, HKV, D, page, MB, N) if type(WS) is int else WS.nbytes
    _check(_lib.osc_attn_tree(_at(c, d, Q, q, _BF16), _at(c, d, KC, n, _BF16), _at(c, d, VC, n, _BF16), S, R, HQ, HKV, D, page, MB, NP,
                              _at(c, d, TABLE, 4 * R * MB, _I32), _at(c, d, CU, 4 * R + 4, _I32), _at(c, d, KV, 4 * R, _I32),
                              _at(c, d, MASK, 8 * S * ((N + 63) // 64), _U64), N, scale, _at(c, d, O, q, _BF16), _at(c, d, WS, 0), ws,
                              _stream(stream)), c)


def osc_logprobs_workspace(S: int, V: int, K: int) -> int:
    """Bytes of the workspace that osc_logprobs needs at these sizes."""
    n = _L(0)
    _check(_lib.osc_logprobs_workspace(S, V, K, ctypes.byref(n)), "osc_logprobs_workspace")
    return n.value


def osc_logprobs(X, xt: int, S: int, V: int, ld: int, scale: float, ID, M: int, K: int, LP, ENT, TOPV, TOPI, WS, stream=None) -> None:
    """Of S rows of V logits (X: rows of ld, bf16 or fp32 by xt), p = softmax(scale x): log p of the tokens ID [S, M] to LP, the
    entropy to ENT [S] (or None), the K most likely tokens' log p and ids to TOPV and TOPI [S, K]; WS: a tensor (or the
    address) of at least osc_logprobs_workspace bytes, or None where that is 0."""
    c = "osc_logprobs"
    d = torch.cuda.current_device()
    ws = 0 if WS is None else osc_logprobs_workspace(S, V, K) if type(WS) is int else WS.nbytes
    f32 = xt == OSC_Y_F32
    need = max(0, (S - 1) * ld + V) * (4 if f32 else 2) if S > 0 else 0
    if M == 0:
        ID = LP = None
    if K == 0:
        TOPV = TOPI = None
    _check(_lib.osc_logprobs(_at(c, d, X, need, _F32 if f32 else _BF16), xt, S, V, ld, scale, _at(c, d, ID, 4 * S * M, _I32), M, K,
                             _at(c, d, LP, 4 * S * M, _F32), _at(c, d, ENT, 4 * S, _F32), _at(c, d, TOPV, 4 * S * K, _F32),
                             _at(c, d, TOPI, 4 * S * K, _I32), _at(c, d, WS, 0), ws, _stream(stream)), c)


def osc_tree_accept(TOKEN, PARENT, CHOICE, ldc: int, SLOT, POS, P: int, CU, R: int, T: int, N: int, ACC, PATH, NEXT, stream=None) -> None:
    """The path of each tree along the chosen tokens CHOICE [T, ldc] (column 0): its length ACC [R], its nodes PATH [R, N], the token
    behind it NEXT [R]."""
    c = "osc_tree_accept"
    d = torch.cuda.current_device()
    t, r = 4 * T, 4 * R
    _check(_lib.osc_tree_accept(_at(c, d, TOKEN, t, _I32), _at(c, d, PARENT, t, _I32), _at(c, d, CHOICE, max(0, t * ldc - 4 * (ldc - 1)), _I32),
                                ldc, _at(c, d, SLOT, t, _I32), _at(c, d, POS, t if P > 0 else 0, _I32), P, _at(c, d, CU, r + 4, _I32), R, T, N,
                                _at(c, d, ACC, r, _I32), _at(c, d, PATH, r * N, _I32), _at(c, d, NEXT, r, _I32), _stream(stream)), c)


class LayerCaches:
    """The layers' caches of osc_tree_commit, KC and VC of each (tensors, or addresses), checked once and kept.  All have the
    same heads and pages: a tensor of four dimensions is [NP, HKV, page, D] or [NP, HKV, D, page], NP or more, any other is taken as its bytes."""

    def __init__(self, KC, VC, NP: int, HKV: int, D: int, page: int):
        c = "LayerCaches"
        self.KC, self.VC, self.NP, self.HKV, self.D, self.page = list(KC), list(VC), NP, HKV, D, page
        self.layers = len(self.KC)
        if len(self.VC) != self.layers or self.layers > OSC_MAX_LAYERS:
            raise OscError(2, c, f"{self.layers} layers of keys, {len(self.VC)} of values, at most {OSC_MAX_LAYERS}")
        n = 2 * NP * HKV * page * D
        held = [t for t in self.KC + self.VC if t is not None and type(t) is not int]
        for ts, block in ((self.KC, (HKV, page, D)), (self.VC, (HKV, D, page))):
            for t in ts:
                if t is not None and type(t) is not int and t.dim() == 4 and tuple(t.shape[1:]) != block:
                    raise OscError(2, c, f"a cache of shape {tuple(t.shape)} among those of {block} a page")
        self.device = held[0].get_device() if held else None
        at = lambda ts: (_P * max(1, self.layers))(*[_at(c, self.device, t, n, _BF16) for t in ts])
        self._kc, self._vc = at(self.KC), at(self.VC)


def osc_tree_commit(caches: LayerCaches, SLOT, CU, ACC, PATH, R: int, T: int, N: int, stream=None) -> None:
    """Keys and values of each path's nodes to the slots behind the context, in all layers."""
    c = "osc_tree_commit"
    d = torch.cuda.current_device()
    if caches.device is not None and caches.device != d:
        raise OscError(2, c, f"caches on cuda:{caches.device}, the current device is cuda:{d}")
    _check(_lib.osc_tree_commit(caches._kc, caches._vc, caches.layers, caches.NP, caches.HKV, caches.D, caches.page, _at(c, d, SLOT, 4 * T, _I32),
                                _at(c, d, CU, 4 * R + 4, _I32), _at(c, d, ACC, 4 * R, _I32), _at(c, d, PATH, 4 * R * N, _I32), R, T, N,
                                _stream(stream)), c)
