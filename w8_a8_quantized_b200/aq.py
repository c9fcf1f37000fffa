"""Thin Python binding of libaq's C ABI (include/aq.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of libaq.so.  PyTorch provides device memory and the current CUDA
stream.  There is no CPU fallback: if libaq.so is missing the first call
raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libaq.so")

AQ_OK = 0
AQ_F32, AQ_BF16 = 0, 1
AQ_WEIGHTS_BF16, AQ_WEIGHTS_EXACT = 0x100, 0x200  # how aq_linear_backward takes the weights
AQ_PHASE_DECODE, AQ_PHASE_PREFILL = 0, 1
BUF_NAMES = ("bitmap", "row_off4", "row_off8", "tile_idx", "w4", "w8", "scales")
EXPORTED = ("aq_status_str", "aq_packed_sizes", "aq_pack_metadata", "aq_pack", "aq_quant_act",
            "aq_workspace_bytes", "aq_linear_decode", "aq_linear_prefill", "aq_debug_tile_partials",
            "aq_linear_group", "aq_group_workspace_bytes", "aq_workspace_status", "aq_linear_decode_noalloc",
            "aq_quantize_weights", "aq_paper_packed_bytes", "aq_expanded_bytes", "aq_expand_int8",
            "aq_linear_prefill_expanded", "aq_act_group_rows", "aq_quant_act_groups", "aq_measure_i8_peak",
            "aq_debug_linear_stalled", "aq_pack_tiles", "aq_paper_quant_act", "aq_paper_linear",
            "aq_debug_paper_partials", "aq_lora_apply", "aq_lora_backward", "aq_lora_workspace_bytes",
            "aq_silu_mul_quant", "aq_silu_mul_backward", "aq_linear_backward", "aq_linear_backward_workspace_bytes",
            "aq_debug_lora_backward_stalled", "aq_debug_linear_backward_stalled")


class AqError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {lib().aq_status_str(status).decode()} ({status})")


AQ_SCALES_ROW_FP16, AQ_SCALES_TILE_FP32 = 0, 1


class AqPackedStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("N", "K", "bN", "bK", "R", "C", "T4", "T8")] + \
               [(n, ctypes.c_void_p) for n in BUF_NAMES] + [("scale_kind", ctypes.c_int32)]


class AqLoraStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("N", "K", "L", "R", "max_rank")] + \
               [(n, ctypes.c_void_p) for n in ("a", "bt", "off", "scale")]


_lib = None


def lib():
    """Load libaq.so once and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run `python -m w8_a8_quantized_b200.build` "
                           "(this package has no CPU fallback)")
    L = ctypes.CDLL(LIB_PATH)
    c_int, c_void_p, c_size_t = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    P = ctypes.POINTER(AqPackedStruct)
    L.aq_status_str.restype = ctypes.c_char_p
    L.aq_status_str.argtypes = [c_int]
    L.aq_packed_sizes.restype = c_int
    L.aq_packed_sizes.argtypes = [c_int, c_int, c_int, c_int, c_int, ctypes.POINTER(c_size_t)]
    L.aq_pack_metadata.restype = c_int
    L.aq_pack_metadata.argtypes = [c_void_p, c_int, c_int, c_void_p, c_void_p, c_void_p, c_void_p,
                                   ctypes.POINTER(ctypes.c_int32)]
    L.aq_pack.restype = c_int
    L.aq_pack.argtypes = [c_void_p, c_void_p, c_void_p, c_int, c_int, c_int, c_int, P, c_void_p]
    L.aq_pack_tiles.restype = c_int
    L.aq_pack_tiles.argtypes = [c_void_p, c_void_p, c_void_p, c_int, c_int, c_int, c_int, P, c_void_p]
    L.aq_paper_quant_act.restype = c_int
    L.aq_paper_quant_act.argtypes = [c_void_p, c_int, c_int, c_int, c_void_p, c_void_p, c_void_p, c_void_p]
    L.aq_paper_linear.restype = c_int
    L.aq_paper_linear.argtypes = [P, c_void_p, c_void_p, c_int, c_void_p, c_void_p, c_void_p, c_int, c_void_p]
    L.aq_debug_paper_partials.restype = c_int
    L.aq_debug_paper_partials.argtypes = [P, c_void_p, c_int, c_void_p, c_void_p]
    L.aq_quant_act.restype = c_int
    L.aq_paper_packed_bytes.restype = c_int
    L.aq_paper_packed_bytes.argtypes = [c_int, c_int, c_int, c_int, c_int, ctypes.POINTER(c_size_t)]
    L.aq_expanded_bytes.restype = c_size_t
    L.aq_expanded_bytes.argtypes = [P]
    L.aq_expand_int8.restype = c_int
    L.aq_expand_int8.argtypes = [P, c_void_p, c_size_t, P, c_void_p]
    L.aq_linear_prefill_expanded.restype = c_int
    L.aq_linear_prefill_expanded.argtypes = [P, c_void_p, c_void_p, c_int, c_void_p, c_void_p, c_int, c_int, c_void_p,
                                             c_size_t, c_void_p, c_size_t, c_void_p]
    L.aq_act_group_rows.restype = c_int
    L.aq_act_group_rows.argtypes = [c_int]
    L.aq_quant_act_groups.restype = c_int
    L.aq_quant_act_groups.argtypes = [c_void_p, c_int, c_int, c_int, c_void_p, c_void_p, c_void_p]
    L.aq_quantize_weights.restype = c_int
    L.aq_quantize_weights.argtypes = [c_void_p, c_int, c_int, c_int, c_int, c_int, c_int, c_void_p, c_int,
                                      c_void_p, c_void_p, c_void_p]
    L.aq_quant_act.argtypes = [c_void_p, c_int, c_int, c_int, c_void_p, c_void_p, c_void_p]
    L.aq_workspace_bytes.restype = c_size_t
    L.aq_workspace_bytes.argtypes = [c_int, c_int, P]
    for f in (L.aq_linear_decode, L.aq_linear_prefill):
        f.restype = c_int
        f.argtypes = [P, c_void_p, c_void_p, c_int, c_void_p, c_void_p, c_int, c_int, c_void_p, c_size_t,
                      c_void_p]
    L.aq_debug_tile_partials.restype = c_int
    L.aq_debug_tile_partials.argtypes = [P, c_void_p, c_int, c_int, c_void_p, c_void_p, c_size_t, c_void_p]
    L.aq_linear_group.restype = c_int
    L.aq_linear_group.argtypes = [c_int, ctypes.POINTER(P), c_int, c_void_p, c_int, c_int, ctypes.POINTER(c_void_p),
                                  ctypes.POINTER(c_void_p), ctypes.POINTER(c_int), c_int, c_void_p, c_size_t,
                                  c_void_p]
    L.aq_group_workspace_bytes.restype = c_size_t
    L.aq_group_workspace_bytes.argtypes = [c_int, c_int, ctypes.POINTER(P), c_int]
    L.aq_linear_decode_noalloc.restype = c_int
    L.aq_linear_decode_noalloc.argtypes = [P, c_void_p, c_void_p, c_int, c_void_p, c_void_p, c_int, c_int, c_void_p]
    L.aq_debug_linear_stalled.restype = c_int
    L.aq_debug_linear_stalled.argtypes = [P, c_void_p, c_void_p, c_int, c_int, c_void_p, c_int, c_void_p, c_size_t,
                                          ctypes.c_ulonglong, c_int, c_void_p]
    L.aq_measure_i8_peak.restype = c_int
    L.aq_measure_i8_peak.argtypes = [c_int, ctypes.POINTER(ctypes.c_double), c_void_p]
    L.aq_workspace_status.restype = c_int
    L.aq_workspace_status.argtypes = [c_void_p, c_void_p, ctypes.POINTER(c_int)]
    A = ctypes.POINTER(AqLoraStruct)
    L.aq_lora_apply.restype = c_int
    L.aq_lora_apply.argtypes = [A, c_void_p, c_int, c_void_p, c_int, c_void_p, c_int, c_void_p, c_int, c_int, c_void_p,
                                c_void_p, c_size_t, c_void_p]
    L.aq_lora_backward.restype = c_int
    L.aq_lora_backward.argtypes = [A, c_void_p, c_int, c_void_p, c_int, c_void_p, c_void_p, c_int, c_void_p, c_void_p,
                                   c_void_p, c_void_p, c_int, c_void_p, c_int, c_int, c_void_p, c_size_t, c_void_p]
    L.aq_lora_workspace_bytes.restype = c_size_t
    L.aq_lora_workspace_bytes.argtypes = [A, c_int, c_int]
    L.aq_silu_mul_quant.restype = c_int
    L.aq_silu_mul_quant.argtypes = [c_void_p, c_int, c_void_p, c_int, c_int, c_int] + [c_void_p] * 7
    L.aq_silu_mul_backward.restype = c_int
    L.aq_silu_mul_backward.argtypes = [c_void_p, c_int, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_int, c_void_p,
                                       c_int, c_void_p, c_int, c_void_p]
    L.aq_linear_backward.restype = c_int
    L.aq_linear_backward.argtypes = [P, c_void_p, c_int, c_int, c_void_p, c_int, c_void_p, c_int, c_int, c_void_p,
                                     c_size_t, c_void_p]
    L.aq_linear_backward_workspace_bytes.restype = c_size_t
    L.aq_linear_backward_workspace_bytes.argtypes = [c_int, P]
    L.aq_debug_lora_backward_stalled.restype = c_int
    L.aq_debug_lora_backward_stalled.argtypes = [A, c_void_p, c_int, c_void_p, c_int, c_void_p, c_void_p, c_int, c_void_p,
                                                 c_void_p, c_void_p, c_void_p, c_int, c_int, c_void_p, c_size_t, c_int,
                                                 ctypes.c_ulonglong, c_int, c_void_p]
    L.aq_debug_linear_backward_stalled.restype = c_int
    L.aq_debug_linear_backward_stalled.argtypes = [P, c_void_p, c_int, c_int, c_void_p, c_int, c_int, c_void_p, c_size_t,
                                                   ctypes.c_ulonglong, c_int, c_void_p]
    _lib = L
    return L


def _check(rc: int, what: str):
    if rc != AQ_OK:
        raise AqError(rc, what)


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _need(t: torch.Tensor, name: str, dtype, device=None):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def aq_packed_sizes(N: int, K: int, bN: int, bK: int, T4: int) -> dict:
    out = (ctypes.c_size_t * 7)()
    _check(lib().aq_packed_sizes(N, K, bN, bK, T4, out), "aq_packed_sizes")
    return dict(zip(BUF_NAMES, [int(v) for v in out]))


def aq_paper_packed_bytes(R: int, C: int, T4: int, bN: int, bK: int) -> int:
    """Storage of one packed projection as eq. 18 accounts it (FP32 scale per tile)."""
    out = ctypes.c_size_t()
    _check(lib().aq_paper_packed_bytes(R, C, T4, bN, bK, ctypes.byref(out)), "aq_paper_packed_bytes")
    return int(out.value)


class PackedWeights:
    """Device buffers of one packed projection plus the C struct describing them."""

    def __init__(self, N: int, K: int, bN: int, bK: int, T4: int, device):
        sizes = aq_packed_sizes(N, K, bN, bK, T4)
        self.device = torch.device(device)
        self.buffers = {n: torch.empty(max(s, 16), dtype=torch.uint8, device=self.device) for n, s in sizes.items()}
        self.sizes = sizes
        if self.device.type == "cuda":
            _report(self.buffers["w4"].device.index)
        self.struct = AqPackedStruct(N=N, K=K, bN=bN, bK=bK, R=N // bN, C=K // bK, T4=T4, T8=0)
        for n in BUF_NAMES:
            setattr(self.struct, n, self.buffers[n].data_ptr())

    N = property(lambda s: s.struct.N)
    K = property(lambda s: s.struct.K)
    bN = property(lambda s: s.struct.bN)
    bK = property(lambda s: s.struct.bK)
    R = property(lambda s: s.struct.R)
    C = property(lambda s: s.struct.C)
    T4 = property(lambda s: s.struct.T4)
    T8 = property(lambda s: s.struct.T8)

    @property
    def nbytes(self) -> int:
        """Bytes of the packed representation (all seven buffers)."""
        return sum(self.sizes.values())

    def host_buffers(self) -> dict:
        return {n: self.buffers[n][: self.sizes[n]].cpu().numpy() for n in BUF_NAMES}


def aq_pack(codes: torch.Tensor, scales: torch.Tensor, pmap: torch.Tensor, bN: int, bK: int) -> PackedWeights:
    """codes int8 [N][K], scales float16 [N][C], pmap uint8 [R][C] (1 = INT4), all on one CUDA device."""
    _need(codes, "codes", torch.int8)
    dev = codes.device
    _need(scales, "scales", torch.float16, dev)
    _need(pmap, "pmap", torch.uint8, dev)
    N, K = codes.shape
    T4 = aq_int4_tiles(pmap)
    if scales.dim() != 2 or scales.shape[0] != N or pmap.dim() != 2 or pmap.shape[0] * bN != N or \
            pmap.shape[1] * bK != K or scales.shape[1] != pmap.shape[1]:
        raise ValueError("codes [N][K], scales [N][C] and pmap [R][C] do not agree with the tile shape")
    w = PackedWeights(N, K, bN, bK, T4, dev)
    with torch.cuda.device(dev):
        _check(lib().aq_pack(codes.data_ptr(), scales.data_ptr(), pmap.data_ptr(), N, K, bN, bK,
                             ctypes.byref(w.struct), _stream(dev)), "aq_pack")
    return w


def aq_pack_tiles(codes: torch.Tensor, tile_scales: torch.Tensor, pmap: torch.Tensor, bN: int,
                  bK: int = 64) -> PackedWeights:
    """Paper-exact packing: codes int8 [N][K], tile_scales float32 [R][C] (one
    scale per whole tile), pmap uint8 [R][C] (1 = INT4), bK = 64."""
    _need(codes, "codes", torch.int8)
    dev = codes.device
    _need(tile_scales, "tile_scales", torch.float32, dev)
    _need(pmap, "pmap", torch.uint8, dev)
    N, K = codes.shape
    if pmap.dim() != 2 or pmap.shape[0] * bN != N or pmap.shape[1] * bK != K or \
            tuple(tile_scales.shape) != tuple(pmap.shape):
        raise ValueError("codes [N][K], tile_scales [R][C] and pmap [R][C] do not agree with the tile shape")
    T4 = aq_int4_tiles(pmap)
    w = PackedWeights(N, K, bN, bK, T4, dev)
    with torch.cuda.device(dev):
        _check(lib().aq_pack_tiles(codes.data_ptr(), tile_scales.data_ptr(), pmap.data_ptr(), N, K, bN, bK,
                                   ctypes.byref(w.struct), _stream(dev)), "aq_pack_tiles")
    return w


def aq_paper_quant_act(x: torch.Tensor, v: torch.Tensor = None):
    """Paper-exact activation preparation: x bf16 [M][ldx], v float32 [K/64][64][64]
    (V_c blocks; None = identity) -> (xq int8 [M'][K], sx float32 [M'/b_M][K/64])."""
    if x.dtype != torch.bfloat16 or not x.is_cuda or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D bf16 CUDA tensor with unit inner stride")
    M, K = x.shape
    if v is not None:
        _need(v, "v", torch.float32, x.device)
        if tuple(v.shape) != (K // 64, 64, 64):
            raise ValueError("v must be float32 [K/64][64][64]")
    bM = int(lib().aq_act_group_rows(M))
    Mp = -(-M // bM) * bM
    xq = torch.empty((Mp, K), dtype=torch.int8, device=x.device)
    sx = torch.empty((Mp // bM, max(K // 64, 1)), dtype=torch.float32, device=x.device)
    with torch.cuda.device(x.device):
        _check(lib().aq_paper_quant_act(x.data_ptr(), M, K, x.stride(0), v.data_ptr() if v is not None else None,
                                        xq.data_ptr(), sx.data_ptr(), _stream(x.device)), "aq_paper_quant_act")
    return xq, sx


def _paper_operands(w: PackedWeights, xq: torch.Tensor, M: int) -> int:
    """Check the paper-exact layer's codes against the packed weights: the kernel
    reads xq as [M'][K] (M' = M rounded up to whole row groups); returns the
    number of activation row groups M' / b_M."""
    if w.struct.scale_kind != AQ_SCALES_TILE_FP32:
        raise ValueError("w must be packed by aq_pack_tiles (per-tile fp32 scales)")
    _need(xq, "xq", torch.int8, w.device)
    bM = int(lib().aq_act_group_rows(M)) if M >= 1 else 0
    if bM == 0:
        raise ValueError("M must be at least 1")
    Mp = -(-M // bM) * bM
    if xq.dim() != 2 or xq.shape[1] != w.K or xq.shape[0] < Mp:
        raise ValueError(f"xq must be [>= {Mp}][{w.K}] (M = {M} padded to whole row groups), got {tuple(xq.shape)}")
    return Mp // bM


def aq_paper_linear(w: PackedWeights, xq: torch.Tensor, sx: torch.Tensor, M: int, u: torch.Tensor = None,
                    bias: torch.Tensor = None, out: torch.Tensor = None) -> torch.Tensor:
    """Paper-exact layer (eq. 19, then Y = Y~ U): w from aq_pack_tiles, (xq, sx)
    from aq_paper_quant_act, u float32 [R][bN][bN] (None = identity), bias
    float32 [N] -> y float32 [M][N]."""
    dev = w.device
    groups = _paper_operands(w, xq, M)
    _need(sx, "sx", torch.float32, dev)
    if sx.numel() < groups * w.C:
        raise ValueError(f"sx must hold [{groups}][{w.C}] group scales, got {sx.numel()} values")
    if u is not None:
        _need(u, "u", torch.float32, dev)
        if tuple(u.shape) != (w.R, w.bN, w.bN):
            raise ValueError("u must be float32 [R][bN][bN]")
    if bias is not None:
        _need(bias, "bias", torch.float32, dev)
        if bias.numel() != w.N:
            raise ValueError("bias must have N elements")
    if out is None:
        out = torch.empty((M, w.N), dtype=torch.float32, device=dev)
    _need(out, "out", torch.float32, dev)
    if out.dim() != 2 or out.shape[0] < M or out.shape[1] < w.N or out.stride(1) != 1:
        raise ValueError("out must be float32 [>= M][>= N] with unit inner stride")
    with torch.cuda.device(dev):
        _check(lib().aq_paper_linear(ctypes.byref(w.struct), xq.data_ptr(), sx.data_ptr(), M,
                                     u.data_ptr() if u is not None else None,
                                     bias.data_ptr() if bias is not None else None, out.data_ptr(), out.stride(0),
                                     _stream(dev)), "aq_paper_linear")
    return out


def aq_debug_paper_partials(w: PackedWeights, xq: torch.Tensor, M: int) -> torch.Tensor:
    """Exact integer tile products of the paper-exact layer: int32 [M][N][K/64]."""
    dev = w.device
    _paper_operands(w, xq, M)
    P = torch.zeros((M, w.N, w.C), dtype=torch.int32, device=dev)
    with torch.cuda.device(dev):
        _check(lib().aq_debug_paper_partials(ctypes.byref(w.struct), xq.data_ptr(), M, P.data_ptr(), _stream(dev)),
               "aq_debug_paper_partials")
    return P


def aq_int4_tiles(pmap: torch.Tensor) -> int:
    """INT4 tile count of a precision map (uint8 [R][C], 1 = INT4), as the library's
    host-side metadata builder counts it; it rejects labels other than 0 and 1."""
    if pmap.dim() != 2 or pmap.dtype != torch.uint8:
        raise ValueError("pmap must be a 2-D uint8 tensor")
    R, C = pmap.shape
    host = np.ascontiguousarray(pmap.cpu().numpy())
    T = R * C
    bitmap = np.zeros(max((T + 7) // 8, 1), np.uint8)
    off4, off8 = np.zeros(R + 1, np.int32), np.zeros(R + 1, np.int32)
    idx = np.zeros(max(T, 1), np.int32)
    t4 = ctypes.c_int32(0)
    p = lambda a: a.ctypes.data_as(ctypes.c_void_p)
    _check(lib().aq_pack_metadata(p(host), R, C, p(bitmap), p(off4), p(off8), p(idx), ctypes.byref(t4)),
           "aq_pack_metadata")
    return int(t4.value)


def aq_quantize_weights(w: torch.Tensor, pmap: torch.Tensor, bN: int, bK: int = 128, search: bool = True,
                        codes: torch.Tensor = None, scales: torch.Tensor = None):
    """Float weights w (float32 or bfloat16, [N][ldw] with unit inner stride) and
    labels pmap uint8 [R][C] (1 = INT4) -> (codes int8 [N][K], scales float16
    [N][C]) for aq_pack.  K = pmap.shape[1] * bK; search selects eq. 7's scale
    search over eq. 6's endpoint scale."""
    if w.dim() != 2 or not w.is_cuda or w.stride(1) != 1 or w.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("w must be a 2-D float32 or bfloat16 CUDA tensor with unit inner stride")
    dev = w.device
    _need(pmap, "pmap", torch.uint8, dev)
    N, K = w.shape[0], pmap.shape[1] * bK
    if codes is None:
        codes = torch.empty((N, K), dtype=torch.int8, device=dev)
    if scales is None:
        scales = torch.empty((N, pmap.shape[1]), dtype=torch.float16, device=dev)
    _need(codes, "codes", torch.int8, dev)
    _need(scales, "scales", torch.float16, dev)
    wdtype = AQ_F32 if w.dtype == torch.float32 else AQ_BF16
    _check(lib().aq_quantize_weights(w.data_ptr(), wdtype, N, K, w.stride(0), bN, bK, pmap.data_ptr(),
                                     int(bool(search)), codes.data_ptr(), scales.data_ptr(), _stream(dev)),
           "aq_quantize_weights")
    return codes, scales


def aq_quantize_and_pack(w: torch.Tensor, pmap: torch.Tensor, bN: int, bK: int = 128,
                         search: bool = True) -> PackedWeights:
    """Float weights -> packed tile format: aq_quantize_weights then aq_pack."""
    codes, scales = aq_quantize_weights(w, pmap, bN, bK, search)
    return aq_pack(codes, scales, pmap, bN, bK)


def aq_quant_act(x: torch.Tensor, xq: torch.Tensor = None, sx: torch.Tensor = None, K: int = None):
    """x bf16 [M][ldx] -> (xq int8 [M][K], sx float32 [M]) on x's stream."""
    if x.dtype != torch.bfloat16 or not x.is_cuda or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D bf16 CUDA tensor with unit inner stride")
    M = x.shape[0]
    K = x.shape[1] if K is None else K
    if xq is None:
        xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
    if sx is None:
        sx = torch.empty((M,), dtype=torch.float32, device=x.device)
    _need(xq, "xq", torch.int8, x.device)
    _need(sx, "sx", torch.float32, x.device)
    if xq.dim() != 2 or xq.shape[0] < M or xq.shape[1] != K or sx.numel() < M or x.shape[1] < K:
        raise ValueError("xq must be [M][K] and sx hold M scales, with K <= x.shape[1]")
    with torch.cuda.device(x.device):
        _check(lib().aq_quant_act(x.data_ptr(), M, K, x.stride(0), xq.data_ptr(), sx.data_ptr(),
                                  _stream(x.device)), "aq_quant_act")
    return xq, sx


def aq_quant_act_groups(x: torch.Tensor, K: int = None):
    """Paper-form activation quantization: x bf16 [M][ldx] -> (xq int8 [M'][K],
    sx float32 [M'/b_M][K/64]) with one scale per 64 features x b_M rows."""
    if x.dtype != torch.bfloat16 or not x.is_cuda or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D bf16 CUDA tensor with unit inner stride")
    M = x.shape[0]
    K = x.shape[1] if K is None else K
    bM = int(lib().aq_act_group_rows(M))
    Mp = -(-M // bM) * bM
    xq = torch.empty((Mp, K), dtype=torch.int8, device=x.device)
    sx = torch.empty((Mp // bM, K // 64), dtype=torch.float32, device=x.device)
    _check(lib().aq_quant_act_groups(x.data_ptr(), M, K, x.stride(0), xq.data_ptr(), sx.data_ptr(),
                                     _stream(x.device)), "aq_quant_act_groups")
    return xq, sx


def aq_workspace_bytes(phase: int, M: int, w: PackedWeights) -> int:
    return int(lib().aq_workspace_bytes(phase, M, ctypes.byref(w.struct)))


_ws_cache = {}

# The adapter and gradient calls' own workspaces report their errors to a header of their device as well,
# which outlives them: {device index: (that header, the header that such a workspace starts with)}.
_WS_HEADER = 256
_reports, _reports_lock = {}, threading.Lock()


def _report(index: int):
    r = _reports.get(index)
    if r is None:
        with _reports_lock, torch.cuda.device(index), torch.inference_mode(False):
            r = _reports.get(index)
            if r is None:
                if torch.cuda.is_current_stream_capturing():
                    raise RuntimeError("make the Adapters or PackedWeights before the capture begins")
                head = torch.zeros(_WS_HEADER, dtype=torch.uint8, device="cuda")
                first = np.zeros(_WS_HEADER, np.uint8)
                first[16:24] = np.frombuffer(head.data_ptr().to_bytes(8, "little"), np.uint8)
                r = head, torch.from_numpy(first).to(head.device)
                torch.cuda.current_stream().synchronize()  # both are there for every stream
                _reports[index] = r
    return r


def workspace(phase: int, M: int, w: PackedWeights) -> torch.Tensor:
    """A zero-initialised workspace big enough for (phase, M, w), cached per device."""
    need = aq_workspace_bytes(phase, M, w)
    if need == 0:
        raise ValueError("invalid arguments for a workspace")
    key = (w.device, phase)
    ws = _ws_cache.get(key)
    if ws is None or ws.numel() < need:
        ws = torch.zeros(max(need, 1 << 20), dtype=torch.uint8, device=w.device)
        _ws_cache[key] = ws
    return ws


def _linear_operands(w, xq, sx, bias, out, out_dtype):
    """Check the operands of a linear call against the packed weights (shapes the
    kernels read and write through raw pointers); allocate `out` if absent."""
    _need(xq, "xq", torch.int8, w.device)
    _need(sx, "sx", torch.float32, w.device)
    if xq.dim() != 2 or xq.shape[1] != w.K:
        raise ValueError(f"xq must be [M][{w.K}], got {tuple(xq.shape)}")
    M = xq.shape[0]
    if M < 1 or sx.numel() < M:
        raise ValueError(f"sx must hold at least M = {M} token scales")
    if out is None:
        out = torch.empty((M, w.N), dtype=out_dtype, device=w.device)
    if out.dtype not in (torch.float32, torch.bfloat16) or out.dim() != 2 or out.stride(1) != 1 or \
            out.device != w.device:
        raise ValueError("out must be a 2-D float32 or bfloat16 tensor on the weights' device, unit inner stride")
    if out.shape[0] < M or out.shape[1] < w.N:
        raise ValueError(f"out must be at least [{M}][{w.N}], got {tuple(out.shape)}")
    if bias is not None:
        _need(bias, "bias", torch.float32, w.device)
        if bias.numel() < w.N:
            raise ValueError(f"bias must hold N = {w.N} values")
    return M, out


def _linear(fn, name, phase, w, xq, sx, bias, out, out_dtype, ws):
    M, out = _linear_operands(w, xq, sx, bias, out, out_dtype)
    ydt = AQ_F32 if out.dtype == torch.float32 else AQ_BF16
    if ws is None:
        ws = workspace(phase, M, w)
    with torch.cuda.device(w.device):
        _check(fn(ctypes.byref(w.struct), xq.data_ptr(), sx.data_ptr(), M,
                  bias.data_ptr() if bias is not None else None, out.data_ptr(), ydt, out.stride(0),
                  ws.data_ptr(), ws.numel(), _stream(w.device)), name)
    return out


def aq_linear_decode(w: PackedWeights, xq, sx, bias=None, out=None, out_dtype=torch.float32, ws=None):
    """Decode-phase y = sx * sum_j sw * (xq q^T)_j (+ bias) for 1 <= M <= 64 tokens."""
    return _linear(lib().aq_linear_decode, "aq_linear_decode", AQ_PHASE_DECODE, w, xq, sx, bias, out, out_dtype, ws)


def aq_linear_prefill(w: PackedWeights, xq, sx, bias=None, out=None, out_dtype=torch.float32, ws=None):
    """Prefill-phase y (tensor-core INT8 path), any M >= 1."""
    return _linear(lib().aq_linear_prefill, "aq_linear_prefill", AQ_PHASE_PREFILL, w, xq, sx, bias, out, out_dtype,
                   ws)


def aq_expanded_bytes(w: PackedWeights) -> int:
    """Bytes of the all-INT8 copy of w made by the long-prefill variant."""
    return int(lib().aq_expanded_bytes(ctypes.byref(w.struct)))


class ExpandedWeights:
    """The all-INT8 copy of a packed projection (long-prefill variant); shares w's scales."""

    def __init__(self, w: PackedWeights, buf: torch.Tensor = None):
        need = aq_expanded_bytes(w)
        if need == 0:
            raise ValueError("invalid packed weights")
        self.source, self.device = w, w.device
        self.buf = torch.empty(need + 256, dtype=torch.uint8, device=w.device) if buf is None else buf
        off = (-self.buf.data_ptr()) % 256  # the library wants a 256-byte aligned buffer
        self.base = self.buf[off:off + need]
        self.struct = AqPackedStruct()
        _check(lib().aq_expand_int8(ctypes.byref(w.struct), self.base.data_ptr(), need, ctypes.byref(self.struct),
                                    _stream(w.device)), "aq_expand_int8")

    N = property(lambda s: s.struct.N)
    K = property(lambda s: s.struct.K)
    R = property(lambda s: s.struct.R)
    C = property(lambda s: s.struct.C)
    T4 = property(lambda s: s.struct.T4)
    T8 = property(lambda s: s.struct.T8)

    def host_buffers(self) -> dict:
        """Bitmap, offsets, tile table and INT8 payload as host arrays (scales: the source's)."""
        st, R, C, bN = self.struct, self.R, self.C, self.struct.bN
        T = R * C
        def view(ptr, nbytes):
            o = ptr - self.base.data_ptr()
            return self.base[o:o + nbytes].cpu().numpy()
        return {"bitmap": view(st.bitmap, (T + 7) // 8), "row_off4": view(st.row_off4, 4 * (R + 1)).view(np.int32),
                "row_off8": view(st.row_off8, 4 * (R + 1)).view(np.int32),
                "tile_idx": view(st.tile_idx, 4 * T).view(np.int32),
                "w8": view(st.w8, T * bN * 128).view(np.int8).reshape(T, bN, 128)}


def aq_linear_prefill_expanded(w: PackedWeights, xq, sx, bias=None, out=None, out_dtype=torch.float32, ws=None,
                               tmp=None):
    """aq_linear_prefill through the long-prefill variant: expand to an INT8 copy in
    `tmp` (uint8, >= aq_expanded_bytes(w) + 256), then the pure INT8 GEMM."""
    need = aq_expanded_bytes(w)
    if tmp is None:
        tmp = torch.empty(need + 256, dtype=torch.uint8, device=w.device)
    off = (-tmp.data_ptr()) % 256
    if tmp.numel() - off < need:
        raise ValueError("tmp is too small")
    L = lib()
    def fn(wp, xqp, sxp, M, bp, yp, ydt, ldy, wsp, wsn, st):
        return L.aq_linear_prefill_expanded(wp, xqp, sxp, M, bp, yp, ydt, ldy, wsp, wsn, tmp.data_ptr() + off,
                                            tmp.numel() - off, st)
    return _linear(fn, "aq_linear_prefill_expanded", AQ_PHASE_PREFILL, w, xq, sx, bias, out, out_dtype, ws)


def aq_linear_decode_noalloc(w: PackedWeights, xq, sx, bias=None, out=None, out_dtype=torch.float32):
    """aq_linear_decode without a workspace, for callers that cannot allocate device
    memory: the library's fixed 4 MiB device scratch is used instead (calls that
    overlap on the GPU must not share it).  `out` must be preallocated by callers
    that cannot allocate; it is allocated here only for convenience."""
    M, out = _linear_operands(w, xq, sx, bias, out, out_dtype)
    # the library resolves its scratch array on the CURRENT device: make it the weights' device
    with torch.cuda.device(w.device):
        _check(lib().aq_linear_decode_noalloc(ctypes.byref(w.struct), xq.data_ptr(), sx.data_ptr(), M,
                                              bias.data_ptr() if bias is not None else None, out.data_ptr(),
                                              AQ_F32 if out.dtype == torch.float32 else AQ_BF16, out.stride(0),
                                              _stream(w.device)), "aq_linear_decode_noalloc")
    return out


class Group:
    """Projections sharing one input (q/k/v or gate/up), run by aq_linear_group."""

    def __init__(self, weights, phase: int, M: int):
        self.weights = list(weights)
        self.phase, self.M = phase, M
        G = len(self.weights)
        P = ctypes.POINTER(AqPackedStruct)
        self._w = (P * G)(*[ctypes.pointer(w.struct) for w in self.weights])
        need = int(lib().aq_group_workspace_bytes(phase, M, self._w, G))
        if need == 0:
            raise ValueError("invalid projection group")
        self.ws = torch.zeros(need, dtype=torch.uint8, device=self.weights[0].device)

    def __call__(self, x: torch.Tensor, outs, bias=None, ws=None):
        """x bf16 [M][ldx]; outs: one float32 or bfloat16 [M][N_g] tensor per member."""
        G = len(self.weights)
        dev = self.weights[0].device
        if x.dtype != torch.bfloat16 or x.device != dev or x.dim() != 2 or x.stride(1) != 1:
            raise ValueError("x must be a 2-D bf16 tensor on the weights' device with unit inner stride")
        if x.shape[0] != self.M or x.shape[1] < self.weights[0].K or len(outs) != G:
            raise ValueError("token count, input width or number of outputs does not match the group")
        for o, w in zip(outs, self.weights):
            if o.dim() != 2 or o.shape[0] < self.M or o.shape[1] < w.N:
                raise ValueError(f"each output must be at least [M][N] = [{self.M}][{w.N}]")
        if bias is not None and (len(bias) != G or any(b is not None and (b.dtype != torch.float32 or
                                                                       b.device != dev or b.numel() < w.N or
                                                                       not b.is_contiguous())
                                                      for b, w in zip(bias, self.weights))):
            raise ValueError("bias must hold one contiguous float32 [N] tensor (or None) per member")
        dt = outs[0].dtype
        if dt not in (torch.float32, torch.bfloat16) or any(o.dtype != dt or o.device != dev or o.stride(1) != 1
                                                             for o in outs):
            raise ValueError("outputs must share one dtype (float32 or bfloat16) on the weights' device")
        ys = (ctypes.c_void_p * G)(*[o.data_ptr() for o in outs])
        lds = (ctypes.c_int * G)(*[o.stride(0) for o in outs])
        bs = None
        if bias is not None:
            bs = (ctypes.c_void_p * G)(*[b.data_ptr() if b is not None else None for b in bias])
        ws = self.ws if ws is None else ws
        ydt = AQ_F32 if dt == torch.float32 else AQ_BF16
        with torch.cuda.device(dev):
            _check(lib().aq_linear_group(self.phase, self._w, G, x.data_ptr(), x.stride(0), self.M, bs, ys, lds,
                                         ydt, ws.data_ptr(), ws.numel(), _stream(dev)), "aq_linear_group")
        return outs


# ------------------------------------------------------------------ adapters, gated activation, gradients
#
# These calls stand outside autograd, as the linear calls do: results carry no graph, whatever the
# inputs require; a training step calls the backward entries itself.

AQ_LORA_MAX_RANK = 256


_F32, _BF16 = torch.float32, torch.bfloat16
# the current stream's handle without building a stream object (2 us a call), and the cheaper forms of two queries
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)


def _rows(t: torch.Tensor, name: str, dtypes, device, M: int, width: int) -> int:
    """Check a 2-D [>= M][>= width] tensor with unit inner stride whose rows the
    kernels read or write; returns its leading dimension (a single row's stride
    says nothing: its width rounded up stands in)."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
        raise TypeError(f"{name} must be a {' or '.join(str(d) for d in dtypes)} tensor")
    if t.device != device:
        raise ValueError(f"{name} must live on {device}")
    stride = t.stride()
    if len(stride) == 2 and stride[1] == 1:
        rows, cols = t.shape
        if rows >= M and cols >= width:
            if rows == 1:
                return -(-cols // 16) * 16
            if stride[0] >= width:
                return stride[0]
    raise ValueError(f"{name} must be [>= {M}][>= {width}] with unit inner stride and rows that do not overlap")


def _lead(t: torch.Tensor, name: str, device=None, width: int = 0):
    """_rows of the 2-D bf16 tensor that sets a call's sizes: its rows, columns, leading
    dimension and device."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _BF16 or t.dim() != 2:
        raise TypeError(f"{name} must be a 2-D torch.bfloat16 tensor")
    dev = t.device
    if dev.type != "cuda" or (device is not None and dev != device):
        raise ValueError(f"{name} must live on {device or 'a CUDA device'}")
    rows, cols = t.shape
    ld, inner = t.stride()
    if inner != 1 or cols < width or (ld < cols and rows > 1):
        raise ValueError(f"{name} must be [M][>= {width}] with unit inner stride and rows that do not overlap")
    return rows, cols, ld if rows > 1 else -(-cols // 16) * 16, dev


def _exact(t: torch.Tensor, name: str, dtype, device, shape):
    """_need, with a shape; one pass over what is right, the messages where it is not."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device and t.is_contiguous()):
        _need(t, name, dtype, device)
    if t.shape != shape:
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {list(t.shape)}")


_shapes = {}


def _new(rows: int, cols: int, dtype, device) -> torch.Tensor:
    """An uninitialised [rows][cols] tensor ([rows] for cols 0).  Made like a kept tensor of
    that shape that has no storage, which is 1 us cheaper than torch.empty."""
    key = rows, cols, dtype, device.index
    like = _shapes.get(key)
    if like is None:
        if len(_shapes) >= 4096:
            _shapes.clear()
        with torch.inference_mode(False):
            like = torch.empty((rows, cols) if cols else (rows,), dtype=dtype, device=device)
        like.untyped_storage().resize_(0)
        _shapes[key] = like
    return torch.empty_like(like)


def _call(fn, name: str, device, *args):
    """fn(*args, stream) with `device` current, on its current stream."""
    index = device.index
    if _current_device() == index:
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
    if rc != AQ_OK:
        raise AqError(rc, name)


_NO_WS = 16  # workspace bytes of a call that does not touch its workspace


class Adapters:
    """Low-rank adapters of one N x K projection, laid out for aq_lora_apply.

    a bf16 [R][K] and bt bf16 [R][N] hold the adapters' rows one after another
    (adapter l: ranks[l] rows of A_l, and as many columns of B_l); they are used in
    place, so an optimizer may update them.  scales: one factor per adapter."""

    def __init__(self, a: torch.Tensor, bt: torch.Tensor, ranks, scales):
        _need(a, "a", torch.bfloat16)
        _need(bt, "bt", torch.bfloat16, a.device)
        self.ranks, self.scales = [int(r) for r in ranks], [float(s) for s in scales]
        if a.dim() != 2 or bt.dim() != 2 or a.shape[0] != bt.shape[0] or a.shape[0] != sum(self.ranks):
            raise ValueError("a [R][K] and bt [R][N] must hold sum(ranks) rows")
        if len(self.ranks) != len(self.scales) or min(self.ranks, default=-1) < 0 or max(self.ranks, default=0) < 1:
            raise ValueError("one rank >= 0 and one scale per adapter, not all ranks 0")
        if max(self.ranks) > AQ_LORA_MAX_RANK:
            raise ValueError(f"ranks above {AQ_LORA_MAX_RANK} are not supported")
        self.a, self.bt, self.device = a, bt, a.device
        _report(a.device.index)
        off = np.concatenate([[0], np.cumsum(self.ranks)]).astype(np.int32)
        self.off = torch.from_numpy(off).to(self.device)
        self.scale = torch.tensor(self.scales, dtype=torch.float32, device=self.device)
        self.struct = AqLoraStruct(N=bt.shape[1], K=a.shape[1], L=len(self.ranks), R=a.shape[0],
                                   max_rank=max(self.ranks), a=a.data_ptr(), bt=bt.data_ptr(),
                                   off=self.off.data_ptr(), scale=self.scale.data_ptr())
        self.ref = ctypes.byref(self.struct)
        self.N, self.K, self.L, self.R, self.max_rank = (getattr(self.struct, n) for n in ("N", "K", "L", "R", "max_rank"))
        self.ws_bytes = {}  # workspace bytes by (tokens, backward): a function of the sizes alone
        self.no_ws = torch.empty(_NO_WS, dtype=torch.uint8, device=self.device)  # for calls that touch no workspace

    @classmethod
    def from_pairs(cls, pairs, scales) -> "Adapters":
        """From (A [r][K], B [N][r]) bf16 pairs on one CUDA device."""
        return cls(torch.cat([a for a, _ in pairs]).contiguous(), torch.cat([b.t() for _, b in pairs]).contiguous(),
                   [a.shape[0] for a, _ in pairs], scales)

    def split(self, da: torch.Tensor, dbt: torch.Tensor):
        """Views of aq_lora_backward's gradients per adapter: (dA [r][K], dB [N][r]) pairs."""
        return [(x, y.t()) for x, y in zip(da.split(self.ranks), dbt.split(self.ranks))]


def aq_lora_workspace_bytes(ad: Adapters, M: int, backward: bool) -> int:
    return int(lib().aq_lora_workspace_bytes(ctypes.byref(ad.struct), M, int(bool(backward))))


_thread = threading.local()  # .ws: a thread's workspaces, gone with it


def _new_ws(need: int, device) -> torch.Tensor:
    """A workspace whose header is ready; the rest of it needs no clearing."""
    first = _report(device.index)[1]
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    ws[:_WS_HEADER].copy_(first)
    return ws


def _stream_ws(tag: str, need: int, device) -> torch.Tensor:
    """A workspace of the current stream and thread, kept and grown on demand (threads
    may take turns on a stream between one call's launches: autograd runs backward
    passes in a thread of its own); a call that is captured into a graph gets its own,
    so that graphs share none."""
    if _capturing():
        return _new_ws(need, device)
    kept = getattr(_thread, "ws", None)
    if kept is None:
        kept = _thread.ws = {}
    key = device.index, tag, _raw_stream(device.index)
    ws = kept.get(key)
    if ws is None or ws.numel() < need:
        ws = kept[key] = _new_ws(need, device)
    return ws


def _own_ws(tag: str, need: int, device) -> torch.Tensor:
    if need == 0:
        raise ValueError("invalid arguments for a workspace")
    if _current_device() == device.index:
        return _stream_ws(tag, need, device)
    with torch.cuda.device(device):
        return _stream_ws(tag, need, device)


def _lora_ws(ad: Adapters, M: int, backward: int, ws):
    """The call's workspace: the caller's or the stream's; none to speak of for a
    decode batch."""
    if ws is not None:
        _need(ws, "ws", torch.uint8, ad.device)
        return ws
    need = ad.ws_bytes.get((M, backward))
    if need is None:
        need = ad.ws_bytes[M, backward] = aq_lora_workspace_bytes(ad, M, backward)
    if need == _NO_WS:
        return ad.no_ws
    return _own_ws("lora", need, ad.device)


def aq_lora_apply(ad: Adapters, x: torch.Tensor, ids: torch.Tensor, y: torch.Tensor = None, s: torch.Tensor = None,
                  out: torch.Tensor = None, out_dtype=torch.float32, ws: torch.Tensor = None) -> torch.Tensor:
    """y + scale_l B_l A_l x per token, l = ids[m] (none outside [0, L)): x bf16 [M][K],
    ids int32 [M], y float32 or bfloat16 [M][N] (None: the adapters' part alone, in
    out_dtype).  out may be y.  s float32 [M][max_rank] receives the products that
    aq_lora_backward takes."""
    dev, N = ad.device, ad.N
    M, _, ldx, _ = _lead(x, "x", dev, ad.K)
    _exact(ids, "ids", torch.int32, dev, (M,))
    ldy = 0
    if y is not None:
        ldy, out_dtype = _rows(y, "y", (_F32, _BF16), dev, M, N), y.dtype
    if out is None:
        if out_dtype is not _F32 and out_dtype is not _BF16:
            raise TypeError("out_dtype must be torch.float32 or torch.bfloat16")
        out, ldo = _new(M, N, out_dtype, dev), N
    else:
        ldo = _rows(out, "out", (_F32, _BF16) if y is None else (out_dtype,), dev, M, N)
    if s is not None:
        _exact(s, "s", _F32, dev, (M, ad.max_rank))
    ws = _lora_ws(ad, M, 0, ws)
    _call(lib().aq_lora_apply, "aq_lora_apply", dev, ad.ref, x.data_ptr(), ldx, ids.data_ptr(), M,
          None if y is None else y.data_ptr(), ldy, out.data_ptr(), ldo, AQ_F32 if out.dtype == _F32 else AQ_BF16,
          None if s is None else s.data_ptr(), ws.data_ptr(), ws.numel())
    return out


def aq_lora_backward(ad: Adapters, dy: torch.Tensor, ids: torch.Tensor, s: torch.Tensor, x: torch.Tensor,
                     sx: torch.Tensor = None, add: torch.Tensor = None, dx: torch.Tensor = None, want_dx: bool = True,
                     dx_dtype=torch.bfloat16, da: torch.Tensor = None, dbt: torch.Tensor = None,
                     ws: torch.Tensor = None):
    """Gradients of aq_lora_apply -> (da float32 [R][K], dbt float32 [R][N], dx [M][K] or
    None).  dy bf16 [M][N]; s as the forward call wrote it; x the activations'
    8-bit checkpoint (int8 codes with token scales sx, as aq_quant_act made them)
    or bf16 (sx None).  dx = add + the adapters' part, in add's dtype (dx_dtype
    without add); dx may be add."""
    dev, N, K, R = ad.device, ad.N, ad.K, ad.R
    M, _, ldd, _ = _lead(dy, "dy", dev, N)
    _exact(ids, "ids", torch.int32, dev, (M,))
    _exact(s, "s", _F32, dev, (M, ad.max_rank))
    ldx = _rows(x, "x", (_BF16,) if sx is None else (torch.int8,), dev, M, K)
    if sx is not None:
        _need(sx, "sx", torch.float32, dev)
        if sx.numel() < M:
            raise ValueError(f"sx must hold M = {M} token scales")
    ldadd = lddx = 0
    if add is not None:
        ldadd, dx_dtype = _rows(add, "add", (_F32, _BF16), dev, M, K), add.dtype
    if dx is None and (want_dx or add is not None):
        if dx_dtype is not _F32 and dx_dtype is not _BF16:
            raise TypeError("dx_dtype must be torch.float32 or torch.bfloat16")
        dx, lddx = _new(M, K, dx_dtype, dev), K
    elif dx is not None:
        lddx = _rows(dx, "dx", (_F32, _BF16) if add is None else (dx_dtype,), dev, M, K)
    if da is None:
        da = _new(R, K, _F32, dev)
    else:
        _exact(da, "da", _F32, dev, (R, K))
    if dbt is None:
        dbt = _new(R, N, _F32, dev)
    else:
        _exact(dbt, "dbt", _F32, dev, (R, N))
    ws = _lora_ws(ad, M, 1, ws)
    _call(lib().aq_lora_backward, "aq_lora_backward", dev, ad.ref, dy.data_ptr(), ldd, ids.data_ptr(), M, s.data_ptr(),
          x.data_ptr(), ldx, None if sx is None else sx.data_ptr(), da.data_ptr(), dbt.data_ptr(),
          None if add is None else add.data_ptr(), ldadd, None if dx is None else dx.data_ptr(), lddx,
          AQ_F32 if dx is not None and dx.dtype == _F32 else AQ_BF16, ws.data_ptr(), ws.numel())
    return da, dbt, dx


AQ_GATED_GROUP = 128  # features per scale of a gated checkpoint


def aq_silu_mul_quant(gate: torch.Tensor, up: torch.Tensor, keep: bool = False, hq: torch.Tensor = None,
                      sh: torch.Tensor = None):
    """silu(gate) * up, quantized per token to INT8: gate, up bf16 [M][F]
    -> (hq int8 [M][F], sh float32 [M]), the down projection's input.  keep=True
    appends the 8-bit checkpoints of gate and up for aq_silu_mul_backward: (..., gq
    int8 [M][F], gs float32 [M][ceil(F/128)], uq, us)."""
    M, F, ldg, dev = _lead(gate, "gate")
    m, f, ldu, _ = _lead(up, "up", dev)
    if m != M or f != F:
        raise ValueError("gate and up must have one shape")
    if hq is None:
        hq = _new(M, F, torch.int8, dev)
    else:
        _exact(hq, "hq", torch.int8, dev, (M, F))
    if sh is None:
        sh = _new(M, 0, _F32, dev)
    else:
        _exact(sh, "sh", _F32, dev, (M,))
    kept, ptrs = (), (None,) * 4
    if keep:
        groups = -(-F // AQ_GATED_GROUP)
        kept = tuple(_new(M, n, t, dev) for n, t in ((F, torch.int8), (groups, _F32)) * 2)
        ptrs = tuple(t.data_ptr() for t in kept)
    _call(lib().aq_silu_mul_quant, "aq_silu_mul_quant", dev, gate.data_ptr(), ldg, up.data_ptr(), ldu, M, F,
          hq.data_ptr(), sh.data_ptr(), *ptrs)
    return (hq, sh) + kept


def aq_silu_mul_backward(dh: torch.Tensor, gq: torch.Tensor, gs: torch.Tensor, uq: torch.Tensor, us: torch.Tensor,
                         dgate: torch.Tensor = None, dup: torch.Tensor = None):
    """Gradients of silu(gate) * up from its 8-bit checkpoints: dh bf16 [M][F] ->
    (dgate, dup) bf16 [M][F].  dgate or dup may be dh."""
    M, F, ldd, dev = _lead(dh, "dh")
    groups = -(-F // AQ_GATED_GROUP)
    _exact(gq, "gq", torch.int8, dev, (M, F))
    _exact(uq, "uq", torch.int8, dev, (M, F))
    _exact(gs, "gs", _F32, dev, (M, groups))
    _exact(us, "us", _F32, dev, (M, groups))
    if dgate is None:
        dgate, ldg = _new(M, F, _BF16, dev), F
    else:
        ldg = _rows(dgate, "dgate", (_BF16,), dev, M, F)
    if dup is None:
        dup, ldu = _new(M, F, _BF16, dev), F
    else:
        ldu = _rows(dup, "dup", (_BF16,), dev, M, F)
    _call(lib().aq_silu_mul_backward, "aq_silu_mul_backward", dev, dh.data_ptr(), ldd, gq.data_ptr(), gs.data_ptr(),
          uq.data_ptr(), us.data_ptr(), M, F, dgate.data_ptr(), ldg, dup.data_ptr(), ldu)
    return dgate, dup


def aq_linear_backward_workspace_bytes(M: int, w: PackedWeights) -> int:
    return int(lib().aq_linear_backward_workspace_bytes(M, ctypes.byref(w.struct)))


_WEIGHTS = {None: 0, _F32: AQ_WEIGHTS_EXACT, _BF16: AQ_WEIGHTS_BF16}


def aq_linear_backward(w: PackedWeights, dy: torch.Tensor, add: torch.Tensor = None, out: torch.Tensor = None,
                       out_dtype=torch.bfloat16, ws: torch.Tensor = None, weights=None) -> torch.Tensor:
    """Input gradient of a packed projection: dx = add + dy W (W dequantized), dy bf16
    [M][N] -> [M][K] in add's dtype (out_dtype without add).  out may be add.  A float32
    result takes the dequantized weights exactly, a bfloat16 one rounded to bfloat16 (a third
    of the products, 1.4 times the rounding error); weights = torch.float32 or
    torch.bfloat16 takes the one or the other for either."""
    dev, K = w.device, w.K
    if weights not in _WEIGHTS:
        raise TypeError("weights must be None, torch.float32 or torch.bfloat16")
    M, _, ldd, _ = _lead(dy, "dy", dev, w.N)
    ldadd = 0
    if add is not None:
        ldadd, out_dtype = _rows(add, "add", (_F32, _BF16), dev, M, K), add.dtype
    if out is None:
        if out_dtype is not _F32 and out_dtype is not _BF16:
            raise TypeError("out_dtype must be torch.float32 or torch.bfloat16")
        out, ldo = _new(M, K, out_dtype, dev), K
    else:
        ldo = _rows(out, "out", (_F32, _BF16) if add is None else (out_dtype,), dev, M, K)
    if ws is not None:
        _need(ws, "ws", torch.uint8, dev)
    else:
        sizes = w.__dict__.setdefault("backward_ws_bytes", {})  # by token count: a function of the sizes alone
        need = sizes.get(M)
        if need is None:
            need = sizes[M] = aq_linear_backward_workspace_bytes(M, w)
        ws = _own_ws("backward", need, dev)
    _call(lib().aq_linear_backward, "aq_linear_backward", dev, ctypes.byref(w.struct), dy.data_ptr(), ldd, M,
          None if add is None else add.data_ptr(), ldadd, out.data_ptr(), ldo,
          (AQ_F32 if out.dtype == _F32 else AQ_BF16) + _WEIGHTS[weights], ws.data_ptr(), ws.numel())
    return out


def aq_debug_tile_partials(w: PackedWeights, xq: torch.Tensor, phase: int, ws=None) -> torch.Tensor:
    """Exact INT32 tile products P[M][N][C] computed by the `phase` data path."""
    _need(xq, "xq", torch.int8, w.device)
    if xq.dim() != 2 or xq.shape[1] != w.K:
        raise ValueError(f"xq must be [M][{w.K}]")
    M = xq.shape[0]
    P = torch.zeros((M, w.N, w.C), dtype=torch.int32, device=w.device)
    if ws is None:
        ws = workspace(AQ_PHASE_PREFILL, M, w)
    with torch.cuda.device(w.device):
        _check(lib().aq_debug_tile_partials(ctypes.byref(w.struct), xq.data_ptr(), M, phase, P.data_ptr(),
                                            ws.data_ptr(), ws.numel(), _stream(w.device)), "aq_debug_tile_partials")
    return P


def aq_debug_linear_stalled(w: PackedWeights, xq, sx, phase: int, ws: torch.Tensor, wait_ns: int = 20_000_000,
                            stop_after: int = 1) -> torch.Tensor:
    """Run the tensor-core linear kernel with a stage that never fills (test of the
    bounded waits): returns the (unspecified) output; the error lands in `ws`."""
    M, out = _linear_operands(w, xq, sx, None, None, torch.float32)
    with torch.cuda.device(w.device):
        _check(lib().aq_debug_linear_stalled(ctypes.byref(w.struct), xq.data_ptr(), sx.data_ptr(), M, phase,
                                             out.data_ptr(), out.stride(0), ws.data_ptr(), ws.numel(), wait_ns,
                                             stop_after, _stream(w.device)), "aq_debug_linear_stalled")
    return out


def aq_debug_lora_backward_stalled(ad: Adapters, dy, ids, s, x, sx, kernel: int, ws: torch.Tensor = None,
                                   wait_ns: int = 20_000_000, stop_after: int = 1):
    """aq_lora_backward with a stage of one of its kernels (0 contraction, 1 expansion, 2
    weight gradients) that never fills: returns the (unspecified) gradients; the error
    lands in `ws`.  Contiguous tensors, as aq_lora_backward checks them."""
    M = dy.shape[0]
    ws = _lora_ws(ad, M, 1, ws)
    da, dbt = _new(ad.R, ad.K, _F32, ad.device), _new(ad.R, ad.N, _F32, ad.device)
    dx = _new(M, ad.K, _BF16, ad.device)
    for t, name, dtype, shape in ((dy, "dy", _BF16, (M, ad.N)), (ids, "ids", torch.int32, (M,)),
                                  (s, "s", _F32, (M, ad.max_rank)),
                                  (x, "x", _BF16 if sx is None else torch.int8, (M, ad.K))):
        _exact(t, name, dtype, ad.device, shape)
    if sx is not None:
        _exact(sx, "sx", _F32, ad.device, (M,))
    _call(lib().aq_debug_lora_backward_stalled, "aq_debug_lora_backward_stalled", ad.device, ad.ref, dy.data_ptr(), ad.N,
          ids.data_ptr(), M, s.data_ptr(), x.data_ptr(), ad.K, None if sx is None else sx.data_ptr(), da.data_ptr(),
          dbt.data_ptr(), dx.data_ptr(), ad.K, AQ_BF16, ws.data_ptr(), ws.numel(), kernel, wait_ns, stop_after)
    return da, dbt, dx


def aq_debug_linear_backward_stalled(w: PackedWeights, dy, ws: torch.Tensor = None, out_dtype=torch.bfloat16,
                                     wait_ns: int = 20_000_000, stop_after: int = 1) -> torch.Tensor:
    """aq_linear_backward with a weight producer that stops: returns the (unspecified)
    result; the error lands in `ws`."""
    M = dy.shape[0]
    _exact(dy, "dy", _BF16, w.device, (M, w.N))
    if ws is None:
        ws = _own_ws("backward", aq_linear_backward_workspace_bytes(M, w), w.device)
    out = _new(M, w.K, out_dtype, w.device)
    _call(lib().aq_debug_linear_backward_stalled, "aq_debug_linear_backward_stalled", w.device, ctypes.byref(w.struct),
          dy.data_ptr(), w.N, M, out.data_ptr(), w.K, AQ_F32 if out_dtype == _F32 else AQ_BF16, ws.data_ptr(),
          ws.numel(), wait_ns, stop_after)
    return out


def aq_workspace_status(ws: torch.Tensor):
    """Synchronise; return (status, info) of the kernel error word of a workspace and clear it."""
    info = ctypes.c_int(0)
    rc = lib().aq_workspace_status(ws.data_ptr(), _stream(ws.device), ctypes.byref(info))
    if rc not in (AQ_OK, -7):
        _check(rc, "aq_workspace_status")
    return rc, info.value


def aq_measure_i8_peak(iters: int = 20000, device=None) -> float:
    """Measured dense INT8 tensor-core rate of the device in TOPS (tcgen05 loop on
    shared-memory operands; a measurement helper, not part of the layer)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    tops = ctypes.c_double(0.0)
    with torch.cuda.device(dev):
        _check(lib().aq_measure_i8_peak(iters, ctypes.byref(tops), _stream(dev)), "aq_measure_i8_peak")
    return float(tops.value)


def check_all_workspaces():
    """Raise if a call on a workspace that was left out recorded a kernel error: also
    one of a thread that has ended, or of a replayed graph.  Waits for the devices."""
    for index in list(_reports):
        torch.cuda.synchronize(index)
    for ws in list(_ws_cache.values()) + [head for head, _ in list(_reports.values())]:
        rc, info = aq_workspace_status(ws)
        if rc != AQ_OK:
            raise AqError(rc, f"kernel wait gave up (info {info})")
