"""Python binding of the block-scaled GEMM library for MI355X (gfx950).

Every function here only marshals torch tensors (device memory and streams) into
the C ABI declared in ``include/bsg.h`` and raises on a non-zero status; every
step of the computation runs in the library's HIP kernels.  There is no fallback:
if ``libbsg.so`` is missing or cannot be loaded, every call raises.

    D = gemm_bf16(A, B)                         # bf16 [M,K] x bf16 [N,K] -> bf16 [M,N]
    D = gemm_fp8_blockscaled(A, sfa, B, sfb)    # e4m3 with UE8M0 1x128 / 128x128 scales
    D = gemm_fp4_blockscaled(A, sfa, B, sfb)    # e2m1 (2 per byte) with UE8M0 1x32 scales
    D = m_grouped_gemm_fp8(A, sfa, B, sfb, offsets)
    D = m_grouped_gemm_bf16(A, B, offsets) / m_grouped_gemm_fp4(A, sfa, B, sfb, offsets, K=K)
    D = m_grouped_gemm_fp8_masked(A, sfa, B, sfb, masked_m)   # A [G, max_m, K], counts on the GPU
    P = pack_ue8m0_scales(sf)                   # uint8 [mn, kb] -> int16 [ceil(kb/2), mn]
    sf = unpack_ue8m0_scales(P, mn, kb)
    P = ensure_packed(sf, mn, kb)               # reuse if already packed, else pack
    Q, P = quantize_fp8_per_token(X)            # bf16 [M,K] -> e4m3 + packed 1x128 scales
    Q, P = quantize_fp4_per_token(X)            # bf16 [M,K] -> e2m1 (2/byte) + packed 1x32 scales
    Q, P = swiglu_quantize_fp8(H, inter)        # silu(H[:, :I]) * H[:, I:2I] -> e4m3 + scales
    D = moe_ffn_fp8(A, sfa, W13, sfw13, W2, sfw2, offsets)   # grouped up, SwiGLU, grouped down
    moe_ffn_fp8_noalloc(A, sfa, W13, sfw13, W2, sfw2, offsets, out=D)   # no workspace, no allocation
    L = mqa_logits(fmt, Q, sfq, K, sfk, W, ks, ke, S)  # sum_h w * max(0, q_h . k) in key windows
    plan = sort_tokens(ids, G, align=128)       # expert ids [T, k] -> rows grouped by expert
    A = moe_dispatch_bf16(X, plan)              # token rows -> their experts' rows
    A, sfa = moe_dispatch_fp8(X, plan)          # the same, quantised on the way (also _fp4)
    D = moe_combine(Y, plan, W)                 # sum_j w * experts' row, back in token order
    dY, dW = moe_combine_backward(dD, Y, plan, W)
    D = lora_add_bf16(X, A, B, plan, scale, base)  # base + s_g B_g (A_g x), an adapter per token
    D = gemm_bf16_act(A, B, bias, act, residual)       # residual + f(A B^T + bias); also _fp8, _fp4
    dA, dB, dbias = gemm_bf16_act_backward(dD, A, B, preact, act)
    H = gemm_bf16_glu(X, W13, act)              # f(X Wg^T) * (X Wu^T), W13 = [Wg; Wu]
    dX, dW13 = gemm_bf16_glu_backward(dH, X, W13, preact, act)

No function records an autograd graph: the results are detached whatever their inputs
require, and training calls the gradients' functions itself (from a
torch.autograd.Function, say).
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbsg.so")
BINDING_PATH = os.path.join(_HERE, "_binding.so")

BSG_OK = 0
BSG_ERR_INVALID_ARG = 1
BSG_ERR_UNSUPPORTED_SHAPE = 2
BSG_ERR_MISALIGNED = 3
BSG_ERR_HIP = 4

SCALE_RULES = {"ceil": 0, "ocp_mx": 1}
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}

_lock = threading.Lock()
_lib = None

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32

EXPORTS = {
    "gemm_bf16": [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _i64, _vp],
    "gemm_fp8_blockscaled": [_vp, _i64, _vp, _i64, _i32, _vp, _i64, _vp, _i64, _i32, _vp, _i64,
                             _i64, _i64, _i64, _vp],
    "gemm_fp4_blockscaled": [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64,
                             _i64, _i64, _i64, _vp],
    "m_grouped_gemm_fp8": [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64,
                           _vp, _i32, _i64, _i64, _i64, _vp],
    "m_grouped_gemm_bf16": [_vp, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _i32, _i64, _i64, _i64, _vp],
    "m_grouped_gemm_fp4": [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64,
                           _vp, _i32, _i64, _i64, _i64, _vp],
    "m_grouped_gemm_fp8_masked": [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _vp,
                                  _i64, _vp, _i32, _i64, _i64, _i64, _vp],
    "pack_ue8m0_scales": [_vp, _i64, _i64, _i64, _vp, _i64, _vp],
    "unpack_ue8m0_scales": [_vp, _i64, _i64, _i64, _vp, _i64, _vp],
    "pack_ue8m0_scales_f32": [_vp, _i64, _i64, _i64, _vp, _i64, _vp, _vp],
    "quantize_fp8_per_token": [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _i32, _vp],
    "quantize_fp4_per_token": [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _i32, _vp],
    "swiglu_quantize_fp8": [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _i32, _vp],
    "moe_ffn_fp8": [_vp, _i64, _vp, _i64,
                    _vp, _i64, _i64, _vp, _i64, _i64,
                    _vp, _i64, _i64, _vp, _i64, _i64,
                    _vp, _i32, _i64, _i64, _i64,
                    _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32, _vp],
    "mqa_logits_fp8": [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64,
                       _i64, _i64, _i32, _i64, _i64, _vp],
    "mqa_logits_fp4": [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64,
                       _i64, _i64, _i32, _i64, _i64, _vp],
    "moe_ffn_fp8_noalloc": [_vp, _i64, _vp, _i64,
                            _vp, _i64, _i64, _vp, _i64, _i64,
                            _vp, _i64, _i64, _vp, _i64, _i64,
                            _vp, _i32, _i64, _i64, _i64,
                            _vp, _i64, _i32, _vp],
    "sort_tokens": [_vp, _i64, _i64, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _i64, _vp, _i64,
                    _vp],
    "moe_dispatch_bf16": [_vp, _i64, _vp, _vp, _i64, _i32, _i64, _i64, _vp, _i64, _vp],
    "moe_dispatch_fp8": [_vp, _i64, _vp, _vp, _i64, _i32, _i64, _i64, _vp, _i64, _vp, _i64, _i32,
                         _vp],
    "moe_dispatch_fp4": [_vp, _i64, _vp, _vp, _i64, _i32, _i64, _i64, _vp, _i64, _vp, _i64, _i32,
                         _vp],
    "moe_combine": [_vp, _i64, _vp, _vp, _i64, _i64, _i32, _i64, _i64, _vp, _i64, _vp],
    "moe_combine_backward": [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _i32, _i64, _i64,
                             _vp, _i64, _vp, _i64, _vp],
    "lora_add_bf16": [_vp, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _i64,
                      _vp, _i64, _vp, _i64, _i64, _i32, _i64, _i64, _i32, _vp, _i64, _vp],
    "gemm_bf16_act": [_vp, _i64, _vp, _i64, _vp, _i32, _vp, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _i64,
                      _vp, _i64, _vp],
    "gemm_fp8_act": [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32, _vp, _i32, _vp, _i64, _vp, _i64,
                     _i64, _i64, _i64, _vp, _i64, _vp],
    "gemm_fp4_act": [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i32, _vp, _i64, _vp, _i64,
                     _i64, _i64, _i64, _vp, _i64, _vp],
    "gemm_bf16_act_backward": [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32, _vp, _i64, _vp, _i64, _vp,
                               _i64, _i64, _i64, _vp, _i64, _vp],
    "gemm_bf16_glu": [_vp, _i64, _vp, _i64, _i32, _vp, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _i64, _vp],
    "gemm_bf16_glu_backward": [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32, _vp, _i64, _vp, _i64,
                               _i64, _i64, _i64, _vp, _i64, _vp],
}
# functions that return a number of bytes, not a status
SIZES = {
    "sort_tokens_workspace": [_i64, _i32],
    "lora_add_workspace": [_i64, _i64, _i32, _i64, _i64, _i32],
    "gemm_bf16_act_workspace": [_i64, _i64, _i64],
    "gemm_fp8_act_workspace": [_i64, _i64, _i64],
    "gemm_fp4_act_workspace": [_i64, _i64, _i64],
    "gemm_bf16_act_backward_workspace": [_i64, _i64, _i64],
    "gemm_bf16_glu_workspace": [_i64, _i64, _i64],
    "gemm_bf16_glu_backward_workspace": [_i64, _i64, _i64],
}


class BsgError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")


def lib() -> ctypes.CDLL:
    """The loaded libbsg.so; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with "
                    "`python -m block_scaled_precision_05_amd.build` (hipcc, gfx950)")
            l = ctypes.CDLL(LIB_PATH)
            for name, argtypes in EXPORTS.items():
                f = getattr(l, name)
                f.argtypes = argtypes
                f.restype = ctypes.c_int
            for name, argtypes in SIZES.items():
                f = getattr(l, name)
                f.argtypes = argtypes
                f.restype = _i64
            l.bsg_status_string.argtypes = [ctypes.c_int]
            l.bsg_status_string.restype = ctypes.c_char_p
            _lib = l
        return _lib


def status_string(status: int) -> str:
    return lib().bsg_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != BSG_OK:
        raise BsgError(fn, status)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t: torch.Tensor | None) -> int:
    return 0 if t is None else t.data_ptr()


def _mat(t: torch.Tensor, name: str) -> int:
    """Leading dimension of a 2-D tensor whose rows are contiguous."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _dev(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("all tensors must live on the GPU")


def _bytes_u8(t: torch.Tensor) -> torch.Tensor:
    return t.view(torch.uint8) if t.dtype != torch.uint8 else t


def _out(out, M, N, device):
    if out is None:
        return torch.empty((M, N), dtype=torch.bfloat16, device=device)
    if out.dtype != torch.bfloat16 or out.shape[0] < M or out.shape[1] < N:
        raise ValueError("out must be a bfloat16 tensor of at least [M, N]")
    return out


def gemm_bf16(A: torch.Tensor, B: torch.Tensor, out: torch.Tensor | None = None, stream=None):
    """D[M,N] = A[M,K] @ B[N,K]^T, bf16 in, fp32 accumulate, bf16 out."""
    _dev(A, B, out)
    if A.dtype != torch.bfloat16 or B.dtype != torch.bfloat16:
        raise TypeError("A and B must be bfloat16")
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K:
        raise ValueError("K mismatch")
    D = _out(out, M, N, A.device)
    _check("gemm_bf16", lib().gemm_bf16(_ptr(A), _mat(A, "A"), _ptr(B), _mat(B, "B"), _ptr(D),
                                        _mat(D, "out"), M, N, K, _stream(stream)))
    return D


def _packed(sf: torch.Tensor, name: str) -> int:
    if sf.dtype != torch.int16:
        raise TypeError(f"{name} must be packed int16 scales (see ensure_packed)")
    return _mat(sf, name)


def gemm_fp8_blockscaled(A, sfa, B, sfb, out=None, stream=None, sfb_gran_mn: int = 128):
    """FP8 e4m3 GEMM with UE8M0 scales: sfa packed int16 [ceil(K/256), >=M] (1x128
    per row of A); sfb packed int16 [ceil(K/256), >=ceil(N/128)] (128x128 blocks of
    B, sfb_gran_mn = 128) or [ceil(K/256), >=N] (one per row of B per 128-wide
    K-block, sfb_gran_mn = 1).  A and B are float8_e4m3fn or uint8 codes."""
    _dev(A, sfa, B, sfb, out)
    A, B = _bytes_u8(A), _bytes_u8(B)
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K:
        raise ValueError("K mismatch")
    D = _out(out, M, N, A.device)
    _check("gemm_fp8_blockscaled", lib().gemm_fp8_blockscaled(
        _ptr(A), _mat(A, "A"), _ptr(sfa), _packed(sfa, "sfa"), 1, _ptr(B), _mat(B, "B"),
        _ptr(sfb), _packed(sfb, "sfb"), sfb_gran_mn, _ptr(D), _mat(D, "out"), M, N, K,
        _stream(stream)))
    return D


def gemm_fp4_blockscaled(A, sfa, B, sfb, K: int | None = None, out=None, stream=None):
    """FP4 e2m1 GEMM: A uint8 [M, K/2] and B uint8 [N, K/2] hold two values per
    byte (even K index in the low nibble); sfa / sfb packed int16 [ceil(K/64), >=M]
    / [.., >=N] (one UE8M0 byte per row per 32-wide K-block)."""
    _dev(A, sfa, B, sfb, out)
    A, B = _bytes_u8(A), _bytes_u8(B)
    M = A.shape[0]
    N = B.shape[0]
    if K is None:
        K = 2 * A.shape[1]
    if A.shape[1] * 2 < K or B.shape[1] * 2 < K:
        raise ValueError("K larger than the operands")
    D = _out(out, M, N, A.device)
    _check("gemm_fp4_blockscaled", lib().gemm_fp4_blockscaled(
        _ptr(A), _mat(A, "A"), _ptr(sfa), _packed(sfa, "sfa"), _ptr(B), _mat(B, "B"), _ptr(sfb),
        _packed(sfb, "sfb"), _ptr(D), _mat(D, "out"), M, N, K, _stream(stream)))
    return D


def m_grouped_gemm_fp8(A, sfa, B, sfb, offsets, out=None, stream=None):
    """M-grouped FP8 GEMM.  A e4m3 [M_total, K]; B e4m3 [G, N, K]; sfa packed int16
    [ceil(K/256), >=M_total]; sfb packed int16 [G, ceil(K/256), >=ceil(N/128)];
    offsets int32 [G+1] on the GPU (rows [off[g], off[g+1]) use expert g).  Rows
    outside [off[0], off[G]) of ``out`` are left untouched."""
    _dev(A, sfa, B, sfb, offsets, out)
    A, B = _bytes_u8(A), _bytes_u8(B)
    if B.dim() != 3 or sfb.dim() != 3:
        raise ValueError("B must be [G, N, K] and sfb [G, kp, ld]")
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous():
        raise TypeError("offsets must be a contiguous int32 vector")
    G, N, K = B.shape
    if offsets.numel() != G + 1:
        raise ValueError("offsets must have G+1 entries")
    M = A.shape[0]
    if A.shape[1] != K:
        raise ValueError("K mismatch")
    if B.stride(2) != 1 or sfb.stride(2) != 1 or sfb.dtype != torch.int16:
        raise ValueError("B and sfb must be contiguous along their last dimension")
    D = _out(out, M, N, A.device)
    _check("m_grouped_gemm_fp8", lib().m_grouped_gemm_fp8(
        _ptr(A), _mat(A, "A"), _ptr(sfa), _packed(sfa, "sfa"), _ptr(B), B.stride(1), B.stride(0),
        _ptr(sfb), sfb.stride(1), sfb.stride(0), _ptr(D), _mat(D, "out"), _ptr(offsets), G, M, N,
        K, _stream(stream)))
    return D


def _offsets_check(offsets, G):
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous():
        raise TypeError("offsets must be a contiguous int32 vector")
    if offsets.numel() != G + 1:
        raise ValueError("offsets must have G+1 entries")


def m_grouped_gemm_bf16(A, B, offsets, out=None, stream=None):
    """M-grouped BF16 GEMM.  A bf16 [M_total, K]; B bf16 [G, N, K]; offsets int32
    [G+1] on the GPU.  Rows outside [off[0], off[G]) of ``out`` are left untouched."""
    _dev(A, B, offsets, out)
    if A.dtype != torch.bfloat16 or B.dtype != torch.bfloat16:
        raise TypeError("A and B must be bfloat16")
    if B.dim() != 3 or B.stride(2) != 1:
        raise ValueError("B must be [G, N, K], contiguous along K")
    G, N, K = B.shape
    _offsets_check(offsets, G)
    M = A.shape[0]
    if A.shape[1] != K:
        raise ValueError("K mismatch")
    D = _out(out, M, N, A.device)
    _check("m_grouped_gemm_bf16", lib().m_grouped_gemm_bf16(
        _ptr(A), _mat(A, "A"), _ptr(B), B.stride(1), B.stride(0), _ptr(D), _mat(D, "out"),
        _ptr(offsets), G, M, N, K, _stream(stream)))
    return D


def m_grouped_gemm_fp4(A, sfa, B, sfb, offsets, K: int | None = None, out=None, stream=None):
    """M-grouped FP4 GEMM.  A uint8 [M_total, K/2]; B uint8 [G, N, K/2] (two e2m1
    values per byte, even K index in the low nibble); sfa packed int16
    [ceil(K/64), >=M_total]; sfb packed int16 [G, ceil(K/64), >=N]; offsets int32
    [G+1] on the GPU."""
    _dev(A, sfa, B, sfb, offsets, out)
    A, B = _bytes_u8(A), _bytes_u8(B)
    if B.dim() != 3 or sfb.dim() != 3:
        raise ValueError("B must be [G, N, K/2] and sfb [G, kp, ld]")
    G, N, kb = B.shape
    K = 2 * kb if K is None else K
    _offsets_check(offsets, G)
    M = A.shape[0]
    if A.shape[1] * 2 < K or kb * 2 < K:
        raise ValueError("K larger than the operands")
    if B.stride(2) != 1 or sfb.stride(2) != 1 or sfb.dtype != torch.int16:
        raise ValueError("B and sfb must be contiguous along their last dimension")
    D = _out(out, M, N, A.device)
    _check("m_grouped_gemm_fp4", lib().m_grouped_gemm_fp4(
        _ptr(A), _mat(A, "A"), _ptr(sfa), _packed(sfa, "sfa"), _ptr(B), B.stride(1), B.stride(0),
        _ptr(sfb), sfb.stride(1), sfb.stride(0), _ptr(D), _mat(D, "out"), _ptr(offsets), G, M, N,
        K, _stream(stream)))
    return D


def m_grouped_gemm_fp8_masked(A, sfa, B, sfb, masked_m, out=None, stream=None):
    """Masked M-grouped FP8 GEMM.  A e4m3 [G, max_m, K]; B e4m3 [G, N, K]; sfa packed
    int16 [ceil(K/256), >=G*max_m] over the G*max_m rows; sfb packed int16
    [G, ceil(K/256), >=ceil(N/128)]; masked_m int32 [G] on the GPU.  Returns D bf16
    [G, max_m, N]; rows r >= masked_m[g] of expert g are left untouched."""
    _dev(A, sfa, B, sfb, masked_m, out)
    A, B = _bytes_u8(A), _bytes_u8(B)
    if A.dim() != 3 or B.dim() != 3 or sfb.dim() != 3:
        raise ValueError("A must be [G, max_m, K], B [G, N, K] and sfb [G, kp, ld]")
    if masked_m.dtype != torch.int32 or masked_m.dim() != 1 or not masked_m.is_contiguous():
        raise TypeError("masked_m must be a contiguous int32 vector")
    G, max_m, K = A.shape
    N = B.shape[1]
    if B.shape[0] != G or B.shape[2] != K or masked_m.numel() != G:
        raise ValueError("A, B and masked_m disagree on G or K")
    if A.stride(2) != 1 or A.stride(0) != max_m * A.stride(1):
        raise ValueError("A's experts must be stacked rows of one [G*max_m, K] matrix")
    if B.stride(2) != 1 or sfb.stride(2) != 1 or sfb.dtype != torch.int16:
        raise ValueError("B and sfb must be contiguous along their last dimension")
    if out is None:
        out = torch.empty((G, max_m, N), dtype=torch.bfloat16, device=A.device)
    if out.dtype != torch.bfloat16 or out.dim() != 3 or out.stride(2) != 1 or \
            out.stride(0) != max_m * out.stride(1) or out.shape[1] != max_m or out.shape[2] < N:
        raise ValueError("out must be bfloat16 [G, max_m, >=N] stacked rows")
    _check("m_grouped_gemm_fp8_masked", lib().m_grouped_gemm_fp8_masked(
        _ptr(A), A.stride(1), _ptr(sfa), _packed(sfa, "sfa"), _ptr(B), B.stride(1), B.stride(0),
        _ptr(sfb), sfb.stride(1), sfb.stride(0), _ptr(out), out.stride(1), _ptr(masked_m), G,
        max_m, N, K, _stream(stream)))
    return out


# hipStreamLegacy: the legacy default stream as a non-NULL handle (the pack and
# unpack entry points read a NULL stream as "host pointers").
_HIP_STREAM_LEGACY = 1


def _pack_stream(tensors, stream) -> int:
    """NULL (host path) when every tensor lives in host memory; otherwise the
    device stream, with the default stream passed as hipStreamLegacy."""
    on_gpu = [t.is_cuda for t in tensors if t is not None]
    if not any(on_gpu):
        if stream is not None:
            raise ValueError("host tensors are packed synchronously: pass no stream")
        return 0
    if not all(on_gpu):
        raise ValueError("sf and the packed array must both live on the GPU or both on the host")
    s = _stream(stream)
    return s if s else _HIP_STREAM_LEGACY


def pack_ue8m0_scales(sf: torch.Tensor, ld_packed: int | None = None, out=None, stream=None):
    """uint8 (or float8_e8m0fnu) [mn, kb] -> packed int16 [ceil(kb/2), ld_packed].
    GPU tensors are packed by a kernel on ``stream``; host tensors on the calling
    thread (the C entry point's NULL-stream path)."""
    sf = _bytes_u8(sf)
    mn, kb = sf.shape
    ldp = mn if ld_packed is None else int(ld_packed)
    if out is None:
        out = torch.empty(((kb + 1) // 2, ldp), dtype=torch.int16, device=sf.device)
    st = _pack_stream((sf, out), stream)
    _check("pack_ue8m0_scales", lib().pack_ue8m0_scales(_ptr(sf), mn, kb, _mat(sf, "sf"),
                                                        _ptr(out), _mat(out, "out"), st))
    return out


def pack_ue8m0_scales_f32(sf: torch.Tensor, ld_packed: int | None = None, out=None, stream=None):
    """fp32 [mn, kb] holding powers of two 2^e (-127 <= e <= 127) -> packed int16
    [ceil(kb/2), ld_packed], exactly; raises ValueError if any value has no UE8M0
    code (the library counts them; for GPU tensors reading the count back
    synchronises the stream)."""
    if sf.dtype != torch.float32 or sf.dim() != 2:
        raise TypeError("sf must be a 2-D float32 tensor")
    mn, kb = sf.shape
    ldp = mn if ld_packed is None else int(ld_packed)
    if out is None:
        out = torch.empty(((kb + 1) // 2, ldp), dtype=torch.int16, device=sf.device)
    count = torch.zeros(1, dtype=torch.int32, device=sf.device)
    st = _pack_stream((sf, out, count), stream)
    _check("pack_ue8m0_scales_f32", lib().pack_ue8m0_scales_f32(
        _ptr(sf), mn, kb, _mat(sf, "sf"), _ptr(out), _mat(out, "out"), _ptr(count), st))
    bad = int(count.item())
    if bad:
        raise ValueError(f"{bad} scale factors are not powers of two in [2^-127, 2^127]: "
                         "UE8M0 cannot represent them (rounding scales is the quantiser's job)")
    return out


def unpack_ue8m0_scales(packed: torch.Tensor, mn: int, kb: int, out=None, stream=None):
    """packed int16 [ceil(kb/2), >=mn] -> uint8 [mn, kb] (on the GPU or, for host
    tensors, on the calling thread)."""
    if out is None:
        out = torch.empty((mn, kb), dtype=torch.uint8, device=packed.device)
    st = _pack_stream((packed, out), stream)
    _check("unpack_ue8m0_scales", lib().unpack_ue8m0_scales(_ptr(packed), mn, kb,
                                                            _packed(packed, "packed"), _ptr(out),
                                                            _mat(out, "out"), st))
    return out


def is_packed(sf: torch.Tensor, mn: int, kb: int) -> bool:
    """True if ``sf`` already has the packed layout: int16 [ceil(kb/2), >=mn] with
    unit stride along MN."""
    return (sf.dtype == torch.int16 and sf.dim() == 2 and sf.shape[0] == (kb + 1) // 2
            and sf.shape[1] >= mn and (sf.shape[1] <= 1 or sf.stride(1) == 1))


def ensure_packed(sf: torch.Tensor, mn: int, kb: int, stream=None) -> torch.Tensor:
    """Reuse-or-convert, decided on every call: an already packed tensor is
    returned as it is; UE8M0 bytes ([mn, kb] uint8 or float8_e8m0fnu) are packed,
    and fp32 powers of two ([mn, kb]) converted exactly and packed (anything else
    in fp32 raises: UE8M0 cannot hold it), on the GPU for GPU tensors.  The pages describe this helper and note the conversion costs
    time when it is needed ("DeepGEMM-Ascend cobre quantas operacoes no Ascend
    950?", section "Fatores de escala FP8 e o formato UE8M0 no Ascend")."""
    if is_packed(sf, mn, kb):
        return sf
    if sf.dtype in (torch.uint8, torch.float8_e8m0fnu) and sf.dim() == 2 and \
            tuple(sf.shape) == (mn, kb):
        return pack_ue8m0_scales(sf, stream=stream if sf.is_cuda else None)
    if sf.dtype == torch.float32 and sf.dim() == 2 and tuple(sf.shape) == (mn, kb):
        return pack_ue8m0_scales_f32(sf, stream=stream if sf.is_cuda else None)
    raise TypeError(
        f"scales must be packed int16 [{(kb + 1) // 2}, >={mn}], UE8M0 bytes [{mn}, {kb}] or "
        f"fp32 powers of two [{mn}, {kb}]; got {sf.dtype} {tuple(sf.shape)}")


def _quantize(fn: str, X, rule, q_cols, gk, out, sf_out, ld_sf, stream):
    _dev(X, out, sf_out)
    if X.dtype != torch.bfloat16:
        raise TypeError("X must be bfloat16")
    if rule not in SCALE_RULES:
        raise ValueError(f"rule must be one of {sorted(SCALE_RULES)}")
    M, K = X.shape
    kp = (K // gk + 1) // 2
    ld = M if ld_sf is None else int(ld_sf)
    Q = torch.empty((M, q_cols(K)), dtype=torch.uint8, device=X.device) if out is None \
        else _bytes_u8(out)
    P = torch.empty((kp, ld), dtype=torch.int16, device=X.device) if sf_out is None else sf_out
    _check(fn, getattr(lib(), fn)(_ptr(X), _mat(X, "X"), _ptr(Q), _mat(Q, "out"), _ptr(P),
                                  _packed(P, "sf_out"), M, K, SCALE_RULES[rule], _stream(stream)))
    return Q, P


def quantize_fp8_per_token(X, rule: str = "ceil", out=None, sf_out=None, ld_sf=None, stream=None):
    """bf16 [M, K] -> (e4m3 codes uint8 [M, K], packed int16 scales [ceil(K/256), ld_sf])
    with one UE8M0 scale per row per 128-wide K-block; ``rule`` is "ceil" (no
    clipping) or "ocp_mx".  The scales are ready to pass as ``sfa``."""
    return _quantize("quantize_fp8_per_token", X, rule, lambda K: K, 128, out, sf_out, ld_sf,
                     stream)


def quantize_fp4_per_token(X, rule: str = "ceil", out=None, sf_out=None, ld_sf=None, stream=None):
    """bf16 [M, K] -> (e2m1 codes uint8 [M, K/2], even K index in the low nibble;
    packed int16 scales [ceil(K/64), ld_sf]), one UE8M0 scale per row per 32-wide
    K-block."""
    return _quantize("quantize_fp4_per_token", X, rule, lambda K: K // 2, 32, out, sf_out, ld_sf,
                     stream)


def swiglu_quantize_fp8(H, inter: int, rule: str = "ceil", out=None, sf_out=None, ld_sf=None,
                        stream=None):
    """bf16 H [M, >=2*inter] (gate in columns [0, inter), up in [inter, 2*inter)) ->
    (e4m3 codes uint8 [M, inter], packed int16 scales [ceil(inter/256), ld_sf]) of
    y = silu(gate) * up, one UE8M0 scale per row per 128 columns."""
    _dev(H, out, sf_out)
    if H.dtype != torch.bfloat16:
        raise TypeError("H must be bfloat16")
    if rule not in SCALE_RULES:
        raise ValueError(f"rule must be one of {sorted(SCALE_RULES)}")
    M = H.shape[0]
    kp = (inter // 128 + 1) // 2
    ld = M if ld_sf is None else int(ld_sf)
    Q = torch.empty((M, inter), dtype=torch.uint8, device=H.device) if out is None \
        else _bytes_u8(out)
    P = torch.empty((kp, ld), dtype=torch.int16, device=H.device) if sf_out is None else sf_out
    _check("swiglu_quantize_fp8", lib().swiglu_quantize_fp8(
        _ptr(H), _mat(H, "H"), _ptr(Q), _mat(Q, "out"), _ptr(P), _packed(P, "sf_out"), M, inter,
        SCALE_RULES[rule], _stream(stream)))
    return Q, P


def moe_ffn_fp8(A, sfa, W13, sfw13, W2, sfw2, offsets, rule: str = "ceil", out=None,
                workspace=None, stream=None):
    """MoE FFN core: grouped up-projection (W13 [G, 2*inter, hidden]), SwiGLU + FP8
    requantisation, grouped down-projection (W2 [G, hidden, inter]); A e4m3
    [M_total, hidden] with packed scales; offsets int32 [G+1] on the GPU.  Returns
    D bf16 [M_total, hidden].  ``workspace`` may pass the (Y, sfy) buffers (e4m3
    uint8 [M_total, >=inter] and packed int16 [ceil(inter/256), >=M_total]); they
    are allocated here otherwise.  The bf16 up-projection output H is never formed."""
    _dev(A, sfa, W13, sfw13, W2, sfw2, offsets, out)
    A, W13, W2 = _bytes_u8(A), _bytes_u8(W13), _bytes_u8(W2)
    if W13.dim() != 3 or W2.dim() != 3 or sfw13.dim() != 3 or sfw2.dim() != 3:
        raise ValueError("W13, W2 and their scales must be [G, rows, cols]")
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous():
        raise TypeError("offsets must be a contiguous int32 vector")
    G, two_i, hidden = W13.shape
    inter = two_i // 2
    if W2.shape[0] != G or W2.shape[1] != hidden or W2.shape[2] != inter or two_i != 2 * inter:
        raise ValueError("W2 must be [G, hidden, inter] for W13 [G, 2*inter, hidden]")
    M = A.shape[0]
    if workspace is None:
        Y = torch.empty((M, inter), dtype=torch.uint8, device=A.device)
        sfy = torch.empty(((inter // 128 + 1) // 2, M), dtype=torch.int16, device=A.device)
    else:
        Y, sfy = workspace
    D = _out(out, M, hidden, A.device)
    for t, n in ((W13, "W13"), (W2, "W2"), (sfw13, "sfw13"), (sfw2, "sfw2")):
        if t.stride(2) != 1:
            raise ValueError(f"{n} must be contiguous along its last dimension")
    _check("moe_ffn_fp8", lib().moe_ffn_fp8(
        _ptr(A), _mat(A, "A"), _ptr(sfa), _packed(sfa, "sfa"),
        _ptr(W13), W13.stride(1), W13.stride(0), _ptr(sfw13), sfw13.stride(1), sfw13.stride(0),
        _ptr(W2), W2.stride(1), W2.stride(0), _ptr(sfw2), sfw2.stride(1), sfw2.stride(0),
        _ptr(offsets), G, M, hidden, inter,
        0, 0, _ptr(Y), _mat(_bytes_u8(Y), "Y"), _ptr(sfy), _packed(sfy, "sfy"),
        _ptr(D), _mat(D, "out"), SCALE_RULES[rule], _stream(stream)))
    return D


def moe_ffn_fp8_noalloc(A, sfa, W13, sfw13, W2, sfw2, offsets, out, rule: str = "ceil",
                        stream=None):
    """moe_ffn_fp8 without a workspace: the library keeps Y and its scales in a fixed
    64 MiB device array (one per GPU), so the call allocates nothing; ``out`` (bf16
    [M_total, hidden]) must be given.  Calls that overlap on one GPU race on that
    array."""
    _dev(A, sfa, W13, sfw13, W2, sfw2, offsets, out)
    A, W13, W2 = _bytes_u8(A), _bytes_u8(W13), _bytes_u8(W2)
    if W13.dim() != 3 or W2.dim() != 3 or sfw13.dim() != 3 or sfw2.dim() != 3:
        raise ValueError("W13, W2 and their scales must be [G, rows, cols]")
    _offsets_check(offsets, W13.shape[0])
    G, two_i, hidden = W13.shape
    M = A.shape[0]
    if out.dtype != torch.bfloat16 or out.shape[0] < M or out.shape[1] < hidden:
        raise ValueError("out must be a bfloat16 tensor of at least [M_total, hidden]")
    for t, n in ((W13, "W13"), (W2, "W2"), (sfw13, "sfw13"), (sfw2, "sfw2")):
        if t.stride(2) != 1:
            raise ValueError(f"{n} must be contiguous along its last dimension")
    _check("moe_ffn_fp8_noalloc", lib().moe_ffn_fp8_noalloc(
        _ptr(A), _mat(A, "A"), _ptr(sfa), _packed(sfa, "sfa"),
        _ptr(W13), W13.stride(1), W13.stride(0), _ptr(sfw13), sfw13.stride(1), sfw13.stride(0),
        _ptr(W2), W2.stride(1), W2.stride(0), _ptr(sfw2), sfw2.stride(1), sfw2.stride(0),
        _ptr(offsets), G, M, hidden, two_i // 2, _ptr(out), _mat(out, "out"),
        SCALE_RULES[rule], _stream(stream)))
    return out


def mqa_logits(fmt: str, Q, sfq, K, sfk, W, ks, ke, S: int, q_per_group: int | None = None,
               group_rows: int = 0, out=None, stream=None):
    """MQA logits (fmt "fp8" or "fp4"): L[t][s] = sum_h W[t][h] * max(0, q[t][h] . k[s])
    for ks[t] <= s < ke[t], -inf for the other s < S.  Q: codes [T*H, 128] (fp8) or
    [T*H, 64] (fp4, two per byte) with packed scales sfq over its rows; K: codes over
    the key rows with packed scales sfk; W float32 [T, H]; ks, ke int32 [T] on the GPU.
    Query t reads key group t // q_per_group (default: one group), whose key s is
    row g * group_rows + s of K.  Returns float32 [T, S]."""
    _dev(Q, sfq, K, sfk, W, ks, ke, out)
    if fmt not in ("fp8", "fp4"):
        raise ValueError("fmt must be 'fp8' or 'fp4'")
    Q, K = _bytes_u8(Q), _bytes_u8(K)
    if W.dtype != torch.float32 or ks.dtype != torch.int32 or ke.dtype != torch.int32:
        raise TypeError("W must be float32 and ks, ke int32")
    T, H = W.shape
    if Q.shape[0] != T * H:
        raise ValueError("Q must hold T*H rows")
    per = T if q_per_group is None else int(q_per_group)
    if out is None:
        out = torch.empty((T, S), dtype=torch.float32, device=Q.device)
    fn = lib().mqa_logits_fp8 if fmt == "fp8" else lib().mqa_logits_fp4
    _check("mqa_logits_" + fmt, fn(
        _ptr(Q), _mat(Q, "Q"), _ptr(sfq), _packed(sfq, "sfq"), _ptr(K), _mat(K, "K"), _ptr(sfk),
        _packed(sfk, "sfk"), _ptr(W), _mat(W, "W"), _ptr(ks), _ptr(ke), _ptr(out), _mat(out, "out"),
        T, S, H, max(per, 1), int(group_rows), _stream(stream)))
    return out


# The calls below are short (a decode step's combine runs 4 us on the GPU), so their
# host side is kept short too: on the current stream a call first goes to the compiled
# marshalling, which takes it whole or returns None; what it leaves (empty tensors, other
# streams and devices, every wrong argument) is checked and called here.
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


_DENSE = tuple(n + w for n in ("gemm_bf16_act", "gemm_fp8_act", "gemm_fp4_act", "gemm_bf16_act_backward",
                               "gemm_bf16_glu", "gemm_bf16_glu_backward") for w in ("", "_workspace"))
_native_lock = threading.Lock()
_native_module = None


def _native():
    """The compiled marshalling of these operators' usual calls (csrc/binding.cpp), on the
    loaded libbsg.so."""
    global _native_module
    if _native_module is None:
        if not os.path.exists(BINDING_PATH):
            raise RuntimeError(
                f"{BINDING_PATH} is missing: build it with "
                "`python -m block_scaled_precision_05_amd.build`")
        from . import _binding
        with _native_lock:
            _binding.init(TokenSort, {n: ctypes.cast(getattr(lib(), n), _vp).value
                                      for n in ("sort_tokens", "sort_tokens_workspace", "moe_dispatch_bf16",
                                                "moe_dispatch_fp8", "moe_dispatch_fp4", "moe_combine",
                                                "moe_combine_backward", "lora_add_bf16",
                                                "lora_add_workspace") + _DENSE})
            _native_module = _binding
    return _native_module


def _launch(t, stream, body):
    """body(stream handle) with t's device current (launches and allocations go there) and,
    for a stream given by the caller, with that stream current, so that buffers allocated
    for the call belong to it."""
    index = t.get_device()
    if stream is None:
        if index == _current_device():
            return body(_raw_stream(index))
        with torch.cuda.device(index):
            return body(_raw_stream(index))
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=t.device)
    elif stream.device != t.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
    with torch.cuda.device(index), torch.cuda.stream(stream):
        return body(stream.cuda_stream)


def _one_gpu(first, *ts):
    index = first.get_device()
    for t in ts:
        if t is not None and t.get_device() != index:
            raise ValueError("all tensors must live on the same GPU")
    if index < 0:
        raise ValueError("all tensors must live on the GPU")


def _ld(t, name, dtype, rows, cols):
    """Leading dimension of a [rows, cols] tensor of that type with contiguous rows."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or t.shape != (rows, cols):
        raise ValueError(f"{name} must be [{rows}, {cols}], got {list(t.shape)}")
    ld, step = t.stride()
    if step == 1 and ld >= cols:
        return ld
    if t.numel() == 0:      # an empty tensor's strides mean nothing
        return cols
    return _mat(t, name)


class TokenSort(NamedTuple):
    """The plan of sort_tokens.  The operators below take it, or any four such tensors."""
    offsets: torch.Tensor    # int32 [G+1] row ranges of the groups; masked layout: counts [G]
    row_of: torch.Tensor     # int32 [T, k] row of each pair, -1 without one
    pair_of: torch.Tensor    # int32 [rows] pair t*k + j in a row; -1 padding, -2 no group's row
    row_group: torch.Tensor  # int32 [rows] group of a row that holds a pair, -1 elsewhere


def sort_tokens(ids, G: int, align: int = 1, cap: int = 0, out: TokenSort | None = None,
                workspace=None, stream=None) -> TokenSort:
    """Stable sort of token-expert pairs by expert.  ids int32 [T, k] (values outside
    [0, G) have no row).  Contiguous layout (cap = 0): every group's count is rounded up
    to a multiple of ``align`` rows and plan.offsets are the M-grouped GEMMs' offsets;
    masked layout (cap > 0): group g owns rows g*cap .., keeps its first cap pairs, and
    plan.offsets are the masked GEMM's counts.  ``out`` may pass a plan's four tensors
    (rows at least T*k + min(G, T*k)*(align-1), or G*cap), ``workspace`` a contiguous
    tensor of at least sort_tokens_workspace(T*k, G) bytes."""
    if stream is None:
        r = (_native_module or _native()).sort_tokens(ids, G, align, cap) if out is workspace is None \
            else None
        if r is not None:
            return r
    if ids.dtype != torch.int32 or ids.dim() != 2:
        raise TypeError("ids must be an int32 tensor [T, k]")
    T, k = ids.shape
    ld = _ld(ids, "ids", torch.int32, T, k)
    n = T * k
    if align < 1 or cap < 0 or G < 0:
        raise ValueError("align must be at least 1, cap and G not negative")
    heads = G if cap else G + 1
    if out is None:
        rows = G * cap if cap else (n + min(G, n) * (align - 1) if G else 0)
        _one_gpu(ids, workspace)
    else:
        out = TokenSort(*out)
        _one_gpu(ids, workspace, *out)
        rows = out.pair_of.numel()
        for t in out:
            if t.dtype != torch.int32 or not t.is_contiguous():
                raise TypeError("out must hold contiguous int32 tensors")
        if out.offsets.numel() != heads or out.row_of.shape != ids.shape or \
                out.row_group.numel() != rows:
            raise ValueError("out must hold offsets [G+1] (masked: [G]), row_of [T, k] and "
                             "pair_of, row_group [rows]")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    L = lib()

    def body(st):
        plan, ws, size = out, workspace, 0
        if plan is None:
            # one allocation, cut into the plan's four tensors
            o, r, p, g = torch.empty(heads + n + 2 * rows, dtype=torch.int32,
                                     device=ids.device).split_with_sizes((heads, n, rows, rows))
            plan = TokenSort(o, r.view(T, k), p, g)
        if ws is None:
            need = L.sort_tokens_workspace(n, G)
            if need:
                ws = torch.empty(need // 4, dtype=torch.int32, device=ids.device)
        if ws is not None:
            size = ws.numel() * ws.element_size()
        _check("sort_tokens", L.sort_tokens(
            ids.data_ptr(), ld, T, k, G, align, cap, plan[0].data_ptr(), plan[1].data_ptr(),
            plan[2].data_ptr(), plan[3].data_ptr(), rows, _ptr(ws), size, st))
        return plan
    return _launch(ids, stream, body)


def _plan(plan, *ts):
    """A plan's row_of, pair_of and row_group, T, k and rows, checked against the other
    operands' device."""
    offsets, row_of, pair_of, row_group = plan
    _one_gpu(row_of, pair_of, row_group, offsets, *ts)
    for t in (row_of, pair_of, row_group):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise TypeError("the plan must hold contiguous int32 tensors")
    rows = pair_of.numel()
    if row_of.dim() != 2 or pair_of.dim() != 1 or row_group.numel() != rows:
        raise ValueError("the plan must hold row_of [T, k] and pair_of, row_group [rows]")
    T, k = row_of.shape
    return row_of, pair_of, row_group, T, k, rows


def _width(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {list(t.shape)}")
    return t.shape[1]


def moe_dispatch_bf16(X, plan, out=None, stream=None):
    """bf16 X [T, H] -> bf16 [rows, H]: row plan.row_of[t, j] is token t's row; padding
    rows are zero and rows of no group (pair_of -2) keep what ``out`` held (they are
    uninitialised in a tensor allocated here).  The gradient with respect to X is
    moe_combine(gradient, plan)."""
    if stream is None:
        r = (_native_module or _native()).moe_dispatch_bf16(X, plan, out)
        if r is not None:
            return r
    row_of, pair_of, _, T, k, rows = _plan(plan, X, out)
    H = _width(X, "X")
    ldx = _ld(X, "X", torch.bfloat16, T, H)
    ldo = H if out is None else _ld(out, "out", torch.bfloat16, rows, H)

    def body(st):
        D = torch.empty((rows, H), dtype=torch.bfloat16, device=X.device) if out is None else out
        _check("moe_dispatch_bf16", lib().moe_dispatch_bf16(
            X.data_ptr(), ldx, row_of.data_ptr(), pair_of.data_ptr(), T, k, rows, H,
            D.data_ptr(), ldo, st))
        return D
    return _launch(X, stream, body)


def _dispatch_quant(fn, X, plan, rule, per, gk, out, sf_out, stream):
    if stream is None:
        r = (_native_module or _native()).moe_dispatch_quantized(
            per == 2, X, plan, SCALE_RULES.get(rule, -1), out, sf_out)
        if r is not None:
            return r
    row_of, pair_of, _, T, k, rows = _plan(plan, X, out, sf_out)
    H = _width(X, "X")
    ldx = _ld(X, "X", torch.bfloat16, T, H)
    if rule not in SCALE_RULES:
        raise ValueError(f"rule must be one of {sorted(SCALE_RULES)}")
    kp = (H // gk + 1) // 2
    ldq, ld_sf = H // per, rows
    if out is not None:
        out = _bytes_u8(out)
        ldq = _ld(out, "out", torch.uint8, rows, H // per)
    if sf_out is not None:
        ld_sf = _packed(sf_out, "sf_out")
        if sf_out.shape[0] != kp or sf_out.shape[1] < rows:
            raise ValueError(f"sf_out must be packed int16 [{kp}, >={rows}]")

    def body(st):
        Q = torch.empty((rows, ldq), dtype=torch.uint8, device=X.device) if out is None else out
        P = torch.empty((kp, rows), dtype=torch.int16, device=X.device) if sf_out is None else sf_out
        _check(fn, getattr(lib(), fn)(
            X.data_ptr(), ldx, row_of.data_ptr(), pair_of.data_ptr(), T, k, rows, H,
            Q.data_ptr(), ldq, P.data_ptr(), ld_sf, SCALE_RULES[rule], st))
        return Q, P
    return _launch(X, stream, body)


def moe_dispatch_fp8(X, plan, rule: str = "ceil", out=None, sf_out=None, stream=None):
    """bf16 X [T, H] -> (e4m3 codes uint8 [rows, H], packed int16 scales [ceil(H/256), rows])
    in the groups' rows: quantize_fp8_per_token's codes and scales, each token quantised
    once and written to its k rows.  Padding rows are a quantised zero row; rows of no
    group are left as they were."""
    return _dispatch_quant("moe_dispatch_fp8", X, plan, rule, 1, 128, out, sf_out, stream)


def moe_dispatch_fp4(X, plan, rule: str = "ceil", out=None, sf_out=None, stream=None):
    """bf16 X [T, H] -> (e2m1 codes uint8 [rows, H/2], packed int16 scales [ceil(H/64), rows])
    in the groups' rows, as moe_dispatch_fp8 with quantize_fp4_per_token's format."""
    return _dispatch_quant("moe_dispatch_fp4", X, plan, rule, 2, 32, out, sf_out, stream)


def moe_combine(Y, plan, weights=None, out=None, stream=None):
    """out[t] = sum_j weights[t, j] * Y[plan.row_of[t, j]] (bf16 [T, H], fp32 sums, rounded
    once); weights float32 [T, k], or None for ones (the gradient of the dispatch).  A
    pair without a row adds nothing."""
    if stream is None:
        r = (_native_module or _native()).moe_combine(Y, plan, weights, out)
        if r is not None:
            return r
    row_of, _, _, T, k, rows = _plan(plan, Y, weights, out)
    H = _width(Y, "Y")
    ldy = _ld(Y, "Y", torch.bfloat16, rows, H)
    ldw = k if weights is None else _ld(weights, "weights", torch.float32, T, k)
    ldo = H if out is None else _ld(out, "out", torch.bfloat16, T, H)

    def body(st):
        D = torch.empty((T, H), dtype=torch.bfloat16, device=Y.device) if out is None else out
        _check("moe_combine", lib().moe_combine(
            Y.data_ptr(), ldy, row_of.data_ptr(), _ptr(weights), ldw, T, k, rows, H,
            D.data_ptr(), ldo, st))
        return D
    return _launch(Y, stream, body)


def moe_combine_backward(dout, Y, plan, weights=None, need_weights: bool = True, out=None,
                         stream=None):
    """Gradients of moe_combine: (dY bf16 [rows, H], dW float32 [T, k]) from dout bf16
    [T, H].  Padding rows of dY are zero, rows of no group keep what ``out`` held.  With
    need_weights False dW is None and Y is not read (it may be None)."""
    if stream is None:
        r = (_native_module or _native()).moe_combine_backward(
            dout, Y, plan, weights, out) if need_weights else None
        if r is not None:
            return r
    row_of, pair_of, _, T, k, rows = _plan(plan, dout, Y, weights, out)
    H = _width(dout, "dout")
    ldd = _ld(dout, "dout", torch.bfloat16, T, H)
    if need_weights and Y is None:
        raise ValueError("the weights' gradient needs Y")
    ldy = 0 if Y is None else _ld(Y, "Y", torch.bfloat16, rows, H)
    ldw = k if weights is None else _ld(weights, "weights", torch.float32, T, k)
    ldo = H if out is None else _ld(out, "out", torch.bfloat16, rows, H)

    def body(st):
        dY = torch.empty((rows, H), dtype=torch.bfloat16, device=dout.device) if out is None else out
        dW = torch.empty((T, k), dtype=torch.float32, device=dout.device) if need_weights else None
        _check("moe_combine_backward", lib().moe_combine_backward(
            dout.data_ptr(), ldd, _ptr(Y), ldy, row_of.data_ptr(), pair_of.data_ptr(),
            _ptr(weights), ldw, T, k, rows, H, dY.data_ptr(), ldo, _ptr(dW), k, st))
        return dY, dW
    return _launch(dout, stream, body)


def lora_add_bf16(X, A, B, plan, scale=None, base=None, out=None, workspace=None, stream=None):
    """out[t] = base[t] + scale[g] * B[g] (A[g] x_t) for token t of adapter g, base[t] for a
    token without one.  X bf16 [T, K]; A bf16 [G, r, K] and B bf16 [G, N, r] (r a multiple
    of 8, at most 128; lower ranks padded with zeros); plan of sort_tokens(ids [T, 1], G,
    align) with align a multiple of 16; scale float32 [G] or None; base bf16 [T, N] or
    None (zeros).  ``out`` may be ``base`` (in place).  ``workspace`` may pass a 16-byte
    aligned contiguous tensor of at least lora_add_workspace(T, rows, G, N, K, r) bytes."""
    if stream is None:
        r = (_native_module or _native()).lora_add_bf16(
            X, A, B, plan, scale, base, out) if workspace is None else None
        if r is not None:
            return r
    row_of, pair_of, row_group, T, k, rows = _plan(plan, X, A, B, scale, base, out, workspace)
    offsets = plan[0]
    if k != 1:
        raise ValueError("a token takes one adapter: the plan must come from ids [T, 1]")
    if A.dtype != torch.bfloat16 or B.dtype != torch.bfloat16:
        raise TypeError("A and B must be bfloat16")
    if A.dim() != 3 or B.dim() != 3:
        raise ValueError("A must be [G, r, K] and B [G, N, r]")
    G, r, K = A.shape
    N = B.shape[1]
    if B.shape != (G, N, r):
        raise ValueError("A and B disagree on the adapters or the rank")
    _offsets_check(offsets, G)
    sa, sb = A.stride(), B.stride()
    if (K > 1 and sa[2] != 1) or (r > 1 and sb[2] != 1):
        raise ValueError("A and B must be contiguous along their last dimension")
    ldx = _ld(X, "X", torch.bfloat16, T, K)
    ld_base = 0 if base is None else _ld(base, "base", torch.bfloat16, T, N)
    ldo = N if out is None else _ld(out, "out", torch.bfloat16, T, N)
    if scale is not None and (scale.dtype != torch.float32 or scale.shape != (G,) or
                              not scale.is_contiguous()):
        raise TypeError("scale must be a contiguous float32 vector [G]")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    L = lib()

    def body(st):
        D = torch.empty((T, N), dtype=torch.bfloat16, device=X.device) if out is None else out
        ws, size = workspace, 0
        if ws is None:
            need = L.lora_add_workspace(T, rows, G, N, K, r)
            if need:
                ws = torch.empty(need, dtype=torch.uint8, device=X.device)
        if ws is not None:
            size = ws.numel() * ws.element_size()
        _check("lora_add_bf16", L.lora_add_bf16(
            X.data_ptr(), ldx, A.data_ptr(), sa[1], sa[0], B.data_ptr(), sb[1], sb[0],
            _ptr(scale), offsets.data_ptr(), row_of.data_ptr(), pair_of.data_ptr(),
            row_group.data_ptr(), rows,
            _ptr(base), ld_base, D.data_ptr(), ldo, T, G, N, K, r, _ptr(ws), size, st))
        return D
    return _launch(X, stream, body)


# Dense products with work in their epilogues, and their gradients.

def _act(act):
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}")
    return ACTIVATIONS[act]


def _space(workspace, need, device):
    """(tensor, its bytes) of a call's workspace, allocated when none was given."""
    if workspace is None:
        if not need:
            return None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace, workspace.numel() * workspace.element_size()


def _epilogue(M, N, bias, residual, out, preact=None):
    """Leading dimensions of the residual, the output and the pre-activation."""
    if bias is not None:
        if bias.dtype != torch.bfloat16:
            raise TypeError(f"bias must be {torch.bfloat16}, got {bias.dtype}")
        if bias.shape != (N,) or not bias.is_contiguous():
            raise ValueError(f"bias must be a contiguous vector [{N}]")
    ldr = 0 if residual is None else _ld(residual, "residual", torch.bfloat16, M, N)
    ldd = N if out is None else _ld(out, "out", torch.bfloat16, M, N)
    ldz = 0 if preact is None else _ld(preact, "preact", torch.bfloat16, M, N)
    return ldr, ldd, ldz


def gemm_bf16_act(A, B, bias=None, act: str = "none", residual=None, out=None, preact=None, workspace=None,
                  stream=None):
    """D = residual + f(A B^T + bias): A bf16 [M, K], B bf16 [N, K], bias bf16 [N] or None,
    act one of "none", "relu", "silu", "gelu", "gelu_tanh", residual bf16 [M, N] or None
    (``out`` may be the residual: added in place).  ``preact`` (bf16 [M, N]), where given,
    receives A B^T + bias, which gemm_bf16_act_backward takes.  Sums are fp32, each output
    rounded once.  ``workspace`` may pass a 16-byte aligned contiguous tensor of at least
    gemm_bf16_act_workspace(M, N, K) bytes."""
    if stream is None and workspace is None:
        r = (_native_module or _native()).gemm_bf16_act(A, B, bias, ACTIVATIONS.get(act, -1), residual, out, preact)
        if r is not None:
            return r
    _one_gpu(A, B, bias, residual, out, preact, workspace)
    M, K = A.shape[0], _width(A, "A")
    N = B.shape[0]
    lda, ldb = _ld(A, "A", torch.bfloat16, M, K), _ld(B, "B", torch.bfloat16, N, K)
    code = _act(act)
    ldr, ldd, ldz = _epilogue(M, N, bias, residual, out, preact)
    L = lib()

    def body(st):
        D = torch.empty((M, N), dtype=torch.bfloat16, device=A.device) if out is None else out
        ws, size = _space(workspace, L.gemm_bf16_act_workspace(M, N, K), A.device)
        _check("gemm_bf16_act", L.gemm_bf16_act(
            A.data_ptr(), lda, B.data_ptr(), ldb, _ptr(bias), code, _ptr(residual), ldr, D.data_ptr(), ldd,
            _ptr(preact), ldz, M, N, K, _ptr(ws), size, st))
        return D
    return _launch(A, stream, body)


def _act_scaled(fn, A, sfa, B, sfb, gran, bias, act, residual, K, out, workspace, stream):
    _one_gpu(A, sfa, B, sfb, bias, residual, out, workspace)
    A, B = _bytes_u8(A), _bytes_u8(B)
    M, N = A.shape[0], B.shape[0]
    lda, ldb = _mat(A, "A"), _mat(B, "B")
    ld_sfa, ld_sfb = _packed(sfa, "sfa"), _packed(sfb, "sfb")
    gk = 128 if fn == "gemm_fp8_act" else 32
    kp = (K // gk + 1) // 2
    rows_b = N if gran == 1 else (N + 127) // 128
    if sfa.shape[0] < kp or sfa.shape[1] < M or sfb.shape[0] < kp or sfb.shape[1] < rows_b:
        raise ValueError(f"sfa must be packed int16 [{kp}, >={M}] and sfb [{kp}, >={rows_b}]")
    code = _act(act)
    ldr, ldd, _ = _epilogue(M, N, bias, residual, out)
    L = lib()

    def body(st):
        D = torch.empty((M, N), dtype=torch.bfloat16, device=A.device) if out is None else out
        ws, size = _space(workspace, getattr(L, fn + "_workspace")(M, N, K), A.device)
        scales = (B.data_ptr(), ldb, sfb.data_ptr(), ld_sfb) + ((gran,) if fn == "gemm_fp8_act" else ())
        _check(fn, getattr(L, fn)(
            A.data_ptr(), lda, sfa.data_ptr(), ld_sfa, *scales, _ptr(bias), code, _ptr(residual), ldr,
            D.data_ptr(), ldd, M, N, K, _ptr(ws), size, st))
        return D
    return _launch(A, stream, body)


def gemm_fp8_act(A, sfa, B, sfb, bias=None, act: str = "none", residual=None, out=None, workspace=None,
                 stream=None, sfb_gran_mn: int = 128):
    """gemm_bf16_act on the operands of gemm_fp8_blockscaled (e4m3 codes with packed UE8M0
    scales; sfb per 128x128 block of B, or per row with sfb_gran_mn = 1), without preact."""
    if stream is None and workspace is None:
        r = (_native_module or _native()).gemm_scaled_act(
            False, A, sfa, B, sfb, sfb_gran_mn, bias, ACTIVATIONS.get(act, -1), residual, out)
        if r is not None:
            return r
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[1]:
        raise ValueError("A must be [M, K] and B [N, K]")
    return _act_scaled("gemm_fp8_act", A, sfa, B, sfb, sfb_gran_mn, bias, act, residual, A.shape[1], out,
                       workspace, stream)


def gemm_fp4_act(A, sfa, B, sfb, bias=None, act: str = "none", residual=None, K: int | None = None, out=None,
                 workspace=None, stream=None):
    """gemm_bf16_act on the operands of gemm_fp4_blockscaled (e2m1 codes, two per byte, with
    packed 1x32 scales on both), without preact."""
    if stream is None and workspace is None and K is None:
        r = (_native_module or _native()).gemm_scaled_act(
            True, A, sfa, B, sfb, 1, bias, ACTIVATIONS.get(act, -1), residual, out)
        if r is not None:
            return r
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A must be [M, K/2] and B [N, K/2]")
    K = 2 * A.shape[1] if K is None else K
    if A.shape[1] * 2 < K or B.shape[1] * 2 < K:
        raise ValueError("K larger than the operands")
    return _act_scaled("gemm_fp4_act", A, sfa, B, sfb, 1, bias, act, residual, K, out, workspace, stream)


def gemm_bf16_act_backward(dout, A, B, preact=None, act: str = "none", need=(True, True, True), workspace=None,
                           stream=None):
    """Gradients of gemm_bf16_act: (dA bf16 [M, K], dB bf16 [N, K], dbias float32 [N]) from
    dout bf16 [M, N] and the forward call's ``preact`` (with act "none" not read, may be
    None).  The residual's gradient is dout itself.  ``need`` tells which of the three are
    computed, the others are None.  ``workspace`` may pass at least
    gemm_bf16_act_backward_workspace(M, N, K) bytes."""
    if stream is None and workspace is None:
        r = (_native_module or _native()).gemm_bf16_act_backward(
            dout, A, B, preact, ACTIVATIONS.get(act, -1), *need)
        if r is not None:
            return r
    _one_gpu(dout, A, B, preact, workspace)
    M, K = A.shape[0], _width(A, "A")
    N = B.shape[0]
    lda, ldb = _ld(A, "A", torch.bfloat16, M, K), _ld(B, "B", torch.bfloat16, N, K)
    ldd = _ld(dout, "dout", torch.bfloat16, M, N)
    code = _act(act)
    if preact is None and code:
        raise ValueError(f"the gradient of {act} needs preact")
    ldz = 0 if preact is None else _ld(preact, "preact", torch.bfloat16, M, N)
    need_a, need_b, need_bias = need
    L = lib()

    def body(st):
        dA = torch.empty((M, K), dtype=torch.bfloat16, device=A.device) if need_a else None
        dB = torch.empty((N, K), dtype=torch.bfloat16, device=A.device) if need_b else None
        dbias = torch.empty(N, dtype=torch.float32, device=A.device) if need_bias else None
        ws, size = _space(workspace, L.gemm_bf16_act_backward_workspace(M, N, K), A.device)
        _check("gemm_bf16_act_backward", L.gemm_bf16_act_backward(
            dout.data_ptr(), ldd, _ptr(preact), ldz, A.data_ptr(), lda, B.data_ptr(), ldb, code, _ptr(dA), K,
            _ptr(dB), K, _ptr(dbias), M, N, K, _ptr(ws), size, st))
        return dA, dB, dbias
    return _launch(A, stream, body)


def _glu_sizes(X, W13):
    M, K = X.shape[0], _width(X, "X")
    two_i = W13.shape[0]
    if two_i % 2:
        raise ValueError("W13 must be [2*inter, K]: gate rows, then up rows")
    return M, two_i // 2, K, _ld(X, "X", torch.bfloat16, M, K), _ld(W13, "W13", torch.bfloat16, two_i, K)


def gemm_bf16_glu(X, W13, act: str = "silu", out=None, preact=None, workspace=None, stream=None):
    """H = f(X Wg^T) * (X Wu^T), the gated block's first half: X bf16 [M, K], W13 bf16
    [2*inter, K] (gate rows, then up rows), H bf16 [M, inter].  ``preact`` (bf16 [M,
    2*inter]), where given, receives both projections, which gemm_bf16_glu_backward takes.
    ``workspace`` may pass at least gemm_bf16_glu_workspace(M, inter, K) bytes."""
    if stream is None and workspace is None:
        r = (_native_module or _native()).gemm_bf16_glu(X, W13, ACTIVATIONS.get(act, -1), out, preact)
        if r is not None:
            return r
    _one_gpu(X, W13, out, preact, workspace)
    M, inter, K, ldx, ldw = _glu_sizes(X, W13)
    code = _act(act)
    ldh = inter if out is None else _ld(out, "out", torch.bfloat16, M, inter)
    ldz = 0 if preact is None else _ld(preact, "preact", torch.bfloat16, M, 2 * inter)
    L = lib()

    def body(st):
        H = torch.empty((M, inter), dtype=torch.bfloat16, device=X.device) if out is None else out
        ws, size = _space(workspace, L.gemm_bf16_glu_workspace(M, inter, K), X.device)
        _check("gemm_bf16_glu", L.gemm_bf16_glu(
            X.data_ptr(), ldx, W13.data_ptr(), ldw, code, H.data_ptr(), ldh, _ptr(preact), ldz, M, inter, K,
            _ptr(ws), size, st))
        return H
    return _launch(X, stream, body)


def gemm_bf16_glu_backward(dout, X, W13, preact, act: str = "silu", need=(True, True), workspace=None,
                           stream=None):
    """Gradients of gemm_bf16_glu: (dX bf16 [M, K], dW13 bf16 [2*inter, K]) from dout bf16
    [M, inter] and the forward call's ``preact``.  ``need`` tells which of the two are
    computed.  ``workspace`` may pass at least gemm_bf16_glu_backward_workspace(M, inter, K)
    bytes."""
    if stream is None and workspace is None:
        r = (_native_module or _native()).gemm_bf16_glu_backward(
            dout, X, W13, preact, ACTIVATIONS.get(act, -1), *need)
        if r is not None:
            return r
    _one_gpu(dout, X, W13, preact, workspace)
    M, inter, K, ldx, ldw = _glu_sizes(X, W13)
    ldd = _ld(dout, "dout", torch.bfloat16, M, inter)
    ldz = _ld(preact, "preact", torch.bfloat16, M, 2 * inter)
    code = _act(act)
    need_x, need_w = need
    L = lib()

    def body(st):
        dX = torch.empty((M, K), dtype=torch.bfloat16, device=X.device) if need_x else None
        dW = torch.empty((2 * inter, K), dtype=torch.bfloat16, device=X.device) if need_w else None
        ws, size = _space(workspace, L.gemm_bf16_glu_backward_workspace(M, inter, K), X.device)
        _check("gemm_bf16_glu_backward", L.gemm_bf16_glu_backward(
            dout.data_ptr(), ldd, preact.data_ptr(), ldz, X.data_ptr(), ldx, W13.data_ptr(), ldw, code,
            _ptr(dX), K, _ptr(dW), K, M, inter, K, _ptr(ws), size, st))
        return dX, dW
    return _launch(X, stream, body)
