"""B200 (sm_100a) FP8 NT GEMM with fine-grained scaling: dense, M-grouped contiguous and M-grouped masked.

Thin ctypes binding over ``libdg.so`` (the C ABI in ``include/dg.h``).  This module only marshals
arguments: it checks dtypes/shapes of the torch tensors, passes raw device pointers and the current CUDA
stream, and turns a negative status into ``DGError``.  Every step of the GEMM runs in the library's CUDA
kernels; there is no fallback of any kind.

Operands follow the NT convention of the DeepGEMM family ("Interfaces / Notices" of the DeepGEMM-for-PPU
README): ``lhs = (a, sfa)`` with ``a`` [M, K] e4m3 and ``sfa`` fp32 [K/128, tma_aligned(M)] (MN-major, one
scale per row and 128-K block); ``rhs = (b, sfb)`` with ``b`` [N, K] e4m3 (grouped: [G, N, K]) and ``sfb``
fp32 [ceil(N/128), K/128] (grouped: [G, ...]), one scale per 128x128 block.  Scales must be powers of two
unless ``set_fp32_scale_promotion(True)`` is in force (any finite fp32 scales, promoted per 128-K block).
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdg.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "dg.h")

DG_OK = 0
STATUS_NAMES = {0: "DG_OK", -1: "DG_ERR_INVALID_ARG", -2: "DG_ERR_ALIGNMENT", -3: "DG_ERR_UNSUPPORTED",
                -4: "DG_ERR_CUDA", -5: "DG_ERR_DEVICE_TIMEOUT", -6: "DG_ERR_BAD_GROUP",
                -7: "DG_ERR_BAD_SCALE"}


class DGError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m moe_grouped_gemm_03_b200.build` "
                      "(or __graft_entry__.build()); there is no non-CUDA implementation")

_lib = ctypes.CDLL(LIB_PATH)


class _NoBinding:
    """In the place of _rowwise where it cannot be loaded: the GEMMs do without it, every call of the others raises."""

    def __init__(self, error):
        self._error = error

    def __getattr__(self, name):
        raise ImportError(f"{os.path.join(_HERE, '_rowwise.so')} cannot be loaded ({self._error}): build it against the "
                          "installed torch with __graft_entry__.build()")


try:
    from . import _rowwise  # noqa: E402  (the binding of the row-wise operators, linked to libdg.so)
except ImportError as _e:
    _rowwise = _NoBinding(str(_e))
else:
    _rowwise.set_error(DGError)
_P = ctypes.c_void_p
_I = ctypes.c_int
_LL = ctypes.c_longlong
_F = ctypes.c_float

_SIGNATURES = {
    "dg_get_m_alignment_for_contiguous_layout": (_I, []),
    "dg_set_m_alignment_for_contiguous_layout": (_I, [_I]),
    "dg_get_tma_aligned_size": (_I, [_I, _I]),
    "dg_set_num_sms": (_I, [_I]),
    "dg_get_num_sms": (_I, []),
    "dg_num_tiles": (_LL, [_LL, _LL, _I, _I]),
    "dg_select_block_n": (_I, [_LL, _I, _I]),
    "dg_fp8_gemm_nt": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P]),
    "dg_m_grouped_fp8_gemm_nt_contiguous": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "dg_m_grouped_fp8_gemm_nt_masked": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "dg_m_grouped_fp8_gemm_nt_nopad": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "dg_m_grouped_fp8_gemm_nn_contiguous": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "dg_m_grouped_fp8_fp4_gemm_nt_contiguous": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "dg_m_grouped_fp8_fp4_gemm_nt_masked": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "dg_k_grouped_fp8_gemm_nt_contiguous": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P]),
    "dg_fp8_gemm_nt_noalloc": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P]),
    "dg_moe_m_total_bound": (_LL, [_LL, _I]),
    "dg_moe_sort_contiguous": (_I, [_P, _I, _I, _I, _I, _I, _P, _P, _P, _P]),
    "dg_moe_sort_nopad": (_I, [_P, _I, _I, _I, _I, _P, _P, _P]),
    "dg_moe_sort_masked": (_I, [_P, _I, _I, _I, _I, _I, _P, _P, _P]),
    "dg_moe_permute": (_I, [_P, _I, _P, _I, _I, _I, _I, _I, _P, _P, _P]),
    "dg_moe_unpermute": (_I, [_P, _I, _P, _P, _I, _I, _I, _I, _P, _P]),
    "dg_moe_unpermute_backward": (_I, [_P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P]),
    "dg_swiglu": (_I, [_P, _I, _I, _I, _P, _P, _P, _I, _P, _P, _P]),
    "dg_swiglu_backward": (_I, [_P, _P, _I, _I, _I, _P, _P, _P, _I, _P, _P, _P]),
    "dg_rms_norm": (_I, [_P, _I, _P, _I, _F, _I, _I, _P, _I, _P, _P, _P]),
    "dg_rms_norm_backward": (_I, [_P, _P, _P, _I, _I, _P, _I, _P, _I, _I, _P, _P, _P]),
    "dg_residual_rms_norm": (_I, [_P, _I, _P, _I, _P, _P, _P, _I, _I, _F, _F, _I, _I, _P, _P, _P, _P, _P, _P]),
    "dg_residual_rms_norm_backward": (_I, [_P, _P, _P, _I, _P, _I, _P, _P, _P, _I, _I, _F, _P, _P, _I, _I, _P, _P, _P,
                                           _P, _P, _P]),
    "dg_set_cta_pair_policy": (_I, [_I]),
    "dg_set_swap_policy": (_I, [_I]),
    "dg_set_fp32_scale_promotion": (_I, [_I]),
    "dg_get_fp32_scale_promotion": (_I, []),
    "dg_debug_bounded_wait": (_I, [ctypes.c_ulonglong, _I]),
    "dg_debug_clock_record": (_I, [_I]),
    "dg_debug_clock_read": (_I, [_P, _I]),
    "dg_last_error": (ctypes.c_char_p, []),
    "dg_check_device_error": (_I, [_P]),
}
for _name, (_res, _args) in _SIGNATURES.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def lib() -> ctypes.CDLL:
    """The loaded C library (raw entry points with the names of include/dg.h)."""
    return _lib


def header_symbols():
    """Names of the functions include/dg.h declares."""
    with open(HEADER_PATH) as f:
        return re.findall(r"^DG_EXPORT[^(]*?\b(dg_\w+)\(", f.read(), flags=re.M)


def last_error() -> str:
    return _lib.dg_last_error().decode()


def _check(status: int):
    if status != DG_OK:
        raise DGError(status, last_error())


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


_FP8_TYPES = (torch.uint8, torch.float8_e4m3fn)


def _need(cond: bool, what) -> None:
    """Raise DG_ERR_INVALID_ARG when cond is false; `what` is the message or a callable that builds it (messages
    are only formatted on failure, which keeps a passing check cheap)."""
    if not cond:
        raise DGError(-1, what() if callable(what) else what)


def _check_operand(name, t, dims, dtypes):
    if isinstance(t, torch.Tensor) and t.dim() == dims and t.dtype in dtypes and t.is_cuda and t.is_contiguous():
        return
    _need(isinstance(t, torch.Tensor), lambda: f"{name} must be a torch.Tensor")
    _need(t.dim() == dims, lambda: f"{name} must have {dims} dims, got {tuple(t.shape)}")
    _need(t.dtype in dtypes, lambda: f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    _need(t.is_contiguous(), lambda: f"{name} must be contiguous")
    _need(t.is_cuda, lambda: f"{name} must be a CUDA tensor")


# ------------------------------------------------------------------------------------------------ utilities
def get_m_alignment_for_contiguous_layout() -> int:
    return _lib.dg_get_m_alignment_for_contiguous_layout()


def get_mk_alignment_for_contiguous_layout() -> int:
    """The MATE wrapper's name for get_m_alignment_for_contiguous_layout (same value)."""
    return _lib.dg_get_m_alignment_for_contiguous_layout()


def set_m_alignment_for_contiguous_layout(alignment: int) -> int:
    """128 (default) or 256: the per-segment M padding the contiguous calls expect from here on."""
    rc = _lib.dg_set_m_alignment_for_contiguous_layout(int(alignment))
    _check(rc if rc < 0 else DG_OK)
    return rc


def get_tma_aligned_size(mn: int, element_size: int) -> int:
    return _lib.dg_get_tma_aligned_size(mn, element_size)


def get_mn_major_tma_aligned_tensor(sf: torch.Tensor) -> torch.Tensor:
    """Per-row scales [M, K/128] (masked layout: [G, M, K/128]) -> the layout the GEMMs take for sfa: fp32,
    MN-major and TMA-aligned, [K/128, tma_aligned(M)] (or [G, K/128, tma_aligned(M)]), contiguous, on the same
    device; the padding columns hold 1.0.  ("Utilities" and "Notices" of the DeepGEMM-for-PPU README: the LHS
    scale factor tensor is TMA-aligned and transposed.)  Input preparation by a tensor copy, outside any GEMM
    call."""
    _need(isinstance(sf, torch.Tensor) and sf.dim() in (2, 3), "sf must be a [M, K/128] or [G, M, K/128] tensor")
    x = sf.unsqueeze(0) if sf.dim() == 2 else sf
    G, M, nkb = x.shape
    out = torch.ones((G, nkb, get_tma_aligned_size(M, 4)), dtype=torch.float32, device=sf.device)
    out[:, :, :M] = x.transpose(1, 2)
    return out[0] if sf.dim() == 2 else out


get_col_major_tma_aligned_tensor = get_mn_major_tma_aligned_tensor  # the pages' other name for it


def set_num_sms(n: int) -> int:
    return _lib.dg_set_num_sms(n)


def get_num_sms() -> int:
    return _lib.dg_get_num_sms()


def num_tiles(M: int, N: int, block_m: int, block_n: int) -> int:
    return _lib.dg_num_tiles(M, N, block_m, block_n)


def select_block_n(num_m_blocks: int, N: int, num_sms: int) -> int:
    return _lib.dg_select_block_n(num_m_blocks, N, num_sms)


def set_cta_pair_policy(policy: int) -> int:
    """-1: library decides; 0: single-CTA 128-row tiles only; 1: 2-CTA 256-row tiles wherever possible."""
    return _lib.dg_set_cta_pair_policy(policy)


def set_swap_policy(policy: int) -> int:
    """-1: library decides; 0: never; 1: swapped operands (B's rows on the MMA's M side, a group's tokens on its
    N side) wherever supported."""
    return _lib.dg_set_swap_policy(policy)


def set_fp32_scale_promotion(enable: bool) -> bool:
    """False (default): scales must be powers of two (applied as UE8M0 exponents by the block-scaled MMA; others
    are reported as DG_ERR_BAD_SCALE by check_device_error).  True: any finite fp32 scales, applied by fp32
    promotion of every 128-K block's partial product (W4A8: of every 32-K sub-block's), on every call."""
    return bool(_lib.dg_set_fp32_scale_promotion(1 if enable else 0))


def get_fp32_scale_promotion() -> bool:
    return bool(_lib.dg_get_fp32_scale_promotion())


def debug_bounded_wait(limit_ns: int = 0, drop_first_stage: bool = False) -> None:
    """Testing aid: set the in-kernel wait limit (0 = default 2 s) and, optionally, make the next GEMM launch
    leave one operand stage unloaded so a wait runs out and DG_ERR_DEVICE_TIMEOUT is recorded."""
    _check(_lib.dg_debug_bounded_wait(int(limit_ns), 1 if drop_first_stage else 0))


def debug_clock_record(enable: bool) -> None:
    """Measurement aid: while on, every GEMM launch's first CTA adds its SM cycles and nanoseconds to a per-device
    accumulator (dg_debug_clock_record)."""
    _lib.dg_debug_clock_record(1 if enable else 0)


def debug_clock_read(reset: bool = True):
    """(cycles, nanoseconds, launches) recorded on the current device since the last reset (dg_debug_clock_read);
    cycles / nanoseconds is the mean SM clock of those launches in GHz."""
    out = (ctypes.c_ulonglong * 3)()
    _check(_lib.dg_debug_clock_read(ctypes.cast(out, _P), 1 if reset else 0))
    return int(out[0]), int(out[1]), int(out[2])


def check_device_error(stream=None) -> None:
    """Synchronise the stream and raise if a kernel recorded a device-side error since the last check."""
    s = _stream() if stream is None else stream
    _check(_lib.dg_check_device_error(s))


# ------------------------------------------------------------------------------------------------ GEMMs
def fp8_gemm_nt(lhs: Tuple[torch.Tensor, torch.Tensor], rhs: Tuple[torch.Tensor, torch.Tensor],
                out: torch.Tensor) -> None:
    """out[M, N] = bf16(lhs @ rhs^T) with fine-grained scales (dense)."""
    a, sfa = lhs
    b, sfb = rhs
    _check_operand("a", a, 2, _FP8_TYPES)
    _check_operand("b", b, 2, _FP8_TYPES)
    _check_operand("sfa", sfa, 2, (torch.float32,))
    _check_operand("sfb", sfb, 2, (torch.float32,))
    _check_operand("out", out, 2, (torch.bfloat16,))
    M, K = a.shape
    N = b.shape[0]
    _need(b.shape[1] == K and tuple(out.shape) == (M, N), "shape mismatch between a, b and out")
    _need(sfa.shape == (K // 128, get_tma_aligned_size(M, 4)), lambda: f"sfa must be [{K // 128}, {get_tma_aligned_size(M, 4)}]")
    _need(sfb.shape == ((N + 127) // 128, K // 128), "sfb must be [ceil(N/128), K/128]")
    _check(_lib.dg_fp8_gemm_nt(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(out), M, N, K, _stream()))


def fp8_gemm_nt_noalloc(lhs: Tuple[torch.Tensor, torch.Tensor], rhs: Tuple[torch.Tensor, torch.Tensor],
                        out: torch.Tensor) -> None:
    """Same as fp8_gemm_nt but allocates no device memory: the packed scales go to the library's fixed 16 MiB
    buffer (for callers that may not allocate during the call, e.g. under a global-mode stream capture).
    Calls overlapping on the GPU share that buffer and race; calls on one stream are safe."""
    a, sfa = lhs
    b, sfb = rhs
    _check_operand("a", a, 2, _FP8_TYPES)
    _check_operand("b", b, 2, _FP8_TYPES)
    _check_operand("sfa", sfa, 2, (torch.float32,))
    _check_operand("sfb", sfb, 2, (torch.float32,))
    _check_operand("out", out, 2, (torch.bfloat16,))
    M, K = a.shape
    N = b.shape[0]
    _need(b.shape[1] == K and tuple(out.shape) == (M, N), "shape mismatch between a, b and out")
    _need(sfa.shape == (K // 128, get_tma_aligned_size(M, 4)), lambda: f"sfa must be [{K // 128}, {get_tma_aligned_size(M, 4)}]")
    _need(sfb.shape == ((N + 127) // 128, K // 128), "sfb must be [ceil(N/128), K/128]")
    _check(_lib.dg_fp8_gemm_nt_noalloc(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(out), M, N, K, _stream()))


def m_grouped_fp8_gemm_nt_contiguous(lhs, rhs, out: torch.Tensor, m_indices: torch.Tensor) -> None:
    """Contiguous layout: out[m] = lhs[m] @ rhs[m_indices[m]]^T; rows with m_indices == -1 are untouched."""
    a, sfa = lhs
    b, sfb = rhs
    _check_operand("a", a, 2, _FP8_TYPES)
    _check_operand("b", b, 3, _FP8_TYPES)
    _check_operand("sfa", sfa, 2, (torch.float32,))
    _check_operand("sfb", sfb, 3, (torch.float32,))
    _check_operand("out", out, 2, (torch.bfloat16,))
    _check_operand("m_indices", m_indices, 1, (torch.int32,))
    M, K = a.shape
    G, N, _ = b.shape
    _need(b.shape[2] == K and tuple(out.shape) == (M, N) and m_indices.shape[0] == M, "shape mismatch")
    _need(sfa.shape == (K // 128, get_tma_aligned_size(M, 4)), "sfa must be [K/128, tma_aligned(M)]")
    _need(sfb.shape == (G, (N + 127) // 128, K // 128), "sfb must be [G, ceil(N/128), K/128]")
    _check(_lib.dg_m_grouped_fp8_gemm_nt_contiguous(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(out),
                                                    _ptr(m_indices), M, N, K, G, _stream()))


def m_grouped_fp8_gemm_nt_masked(lhs, rhs, out: torch.Tensor, masked_m: torch.Tensor, expected_m: int) -> None:
    """Masked layout: out[g, :masked_m[g]] = lhs[g, :masked_m[g]] @ rhs[g]^T; other rows are untouched."""
    a, sfa = lhs
    b, sfb = rhs
    _check_operand("a", a, 3, _FP8_TYPES)
    _check_operand("b", b, 3, _FP8_TYPES)
    _check_operand("sfa", sfa, 3, (torch.float32,))
    _check_operand("sfb", sfb, 3, (torch.float32,))
    _check_operand("out", out, 3, (torch.bfloat16,))
    _check_operand("masked_m", masked_m, 1, (torch.int32,))
    G, M_max, K = a.shape
    N = b.shape[1]
    _need(b.shape[0] == G and b.shape[2] == K and tuple(out.shape) == (G, M_max, N) and masked_m.shape[0] == G,
          "shape mismatch")
    _need(sfa.shape == (G, K // 128, get_tma_aligned_size(M_max, 4)), "sfa must be [G, K/128, tma_aligned(M_max)]")
    _need(sfb.shape == (G, (N + 127) // 128, K // 128), "sfb must be [G, ceil(N/128), K/128]")
    _check(_lib.dg_m_grouped_fp8_gemm_nt_masked(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(out), _ptr(masked_m),
                                                G, M_max, N, K, int(expected_m), _stream()))


def m_grouped_fp8_gemm_nn_contiguous(lhs, rhs, out: torch.Tensor, m_indices: torch.Tensor) -> None:
    """Contiguous layout with rhs = (b [G, K, N], sfb [G, K/128, ceil(N/128)]): out = lhs @ rhs[g] per group."""
    a, sfa = lhs
    b, sfb = rhs
    _check_operand("a", a, 2, _FP8_TYPES)
    _check_operand("b", b, 3, _FP8_TYPES)
    _check_operand("sfa", sfa, 2, (torch.float32,))
    _check_operand("sfb", sfb, 3, (torch.float32,))
    _check_operand("out", out, 2, (torch.bfloat16,))
    _check_operand("m_indices", m_indices, 1, (torch.int32,))
    M, K = a.shape
    G, _, N = b.shape
    _need(b.shape[1] == K and tuple(out.shape) == (M, N) and m_indices.shape[0] == M, "shape mismatch")
    _need(sfa.shape == (K // 128, get_tma_aligned_size(M, 4)), "sfa must be [K/128, tma_aligned(M)]")
    _need(sfb.shape == (G, K // 128, (N + 127) // 128), "sfb must be [G, K/128, ceil(N/128)]")
    _check(_lib.dg_m_grouped_fp8_gemm_nn_contiguous(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(out),
                                                    _ptr(m_indices), M, N, K, G, _stream()))


def k_grouped_fp8_gemm_nt_contiguous(lhs, rhs, out: torch.Tensor, ks, ks_tensor: torch.Tensor,
                                     c: Optional[torch.Tensor] = None) -> None:
    """K-grouped (recipe (1, 1, 128)): lhs = (a [M, sum ks], sfa [sum ks/128, tma_aligned(M)]), rhs = (b [N, sum ks],
    sfb [sum ks/128, tma_aligned(N)]); out fp32 [G, M, N] = c + per-group products (c None, another tensor, or out)."""
    a, sfa = lhs
    b, sfb = rhs
    _check_operand("a", a, 2, _FP8_TYPES)
    _check_operand("b", b, 2, _FP8_TYPES)
    _check_operand("sfa", sfa, 2, (torch.float32,))
    _check_operand("sfb", sfb, 2, (torch.float32,))
    _check_operand("out", out, 3, (torch.float32,))
    _check_operand("ks_tensor", ks_tensor, 1, (torch.int32,))
    ks = [int(k) for k in ks]
    G = len(ks)
    M, Kt = a.shape
    N = b.shape[0]
    _need(b.shape[1] == Kt and sum(ks) == Kt and tuple(out.shape) == (G, M, N) and ks_tensor.shape[0] == G,
          "shape mismatch")
    _need(sfa.shape == (Kt // 128, get_tma_aligned_size(M, 4)), "sfa must be [sum ks/128, tma_aligned(M)]")
    _need(sfb.shape == (Kt // 128, get_tma_aligned_size(N, 4)), "sfb must be [sum ks/128, tma_aligned(N)]")
    if c is not None:
        _check_operand("c", c, 3, (torch.float32,))
        _need(tuple(c.shape) == (G, M, N), "c must be [G, M, N]")
    ks_host = (ctypes.c_int * G)(*ks)
    _check(_lib.dg_k_grouped_fp8_gemm_nt_contiguous(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(out), _ptr(c),
                                                    ctypes.cast(ks_host, ctypes.c_void_p), _ptr(ks_tensor), G, M,
                                                    N, _stream()))


def m_grouped_fp8_fp4_gemm_nt_contiguous(lhs, rhs, out: torch.Tensor, m_indices: torch.Tensor) -> None:
    """W4A8 contiguous layout: rhs = (b packed E2M1 uint8 [G, N, K/2], sfb [G, K/32, tma_aligned(N)]), one B
    scale per (row, 32-K block); lhs and out as for m_grouped_fp8_gemm_nt_contiguous."""
    a, sfa = lhs
    b, sfb = rhs
    _check_operand("a", a, 2, _FP8_TYPES)
    _check_operand("b", b, 3, (torch.uint8,))
    _check_operand("sfa", sfa, 2, (torch.float32,))
    _check_operand("sfb", sfb, 3, (torch.float32,))
    _check_operand("out", out, 2, (torch.bfloat16,))
    _check_operand("m_indices", m_indices, 1, (torch.int32,))
    M, K = a.shape
    G, N, half_k = b.shape
    _need(half_k * 2 == K and tuple(out.shape) == (M, N) and m_indices.shape[0] == M, "shape mismatch")
    _need(sfa.shape == (K // 128, get_tma_aligned_size(M, 4)), "sfa must be [K/128, tma_aligned(M)]")
    _need(sfb.shape == (G, K // 32, get_tma_aligned_size(N, 4)), "sfb must be [G, K/32, tma_aligned(N)]")
    _check(_lib.dg_m_grouped_fp8_fp4_gemm_nt_contiguous(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(out),
                                                        _ptr(m_indices), M, N, K, G, _stream()))


def m_grouped_fp8_fp4_gemm_nt_masked(lhs, rhs, out: torch.Tensor, masked_m: torch.Tensor, expected_m: int) -> None:
    """W4A8 masked layout: rhs = (b packed E2M1 uint8 [G, N, K/2], sfb [G, K/32, tma_aligned(N)]); lhs, out and
    masked_m as for m_grouped_fp8_gemm_nt_masked."""
    a, sfa = lhs
    b, sfb = rhs
    _check_operand("a", a, 3, _FP8_TYPES)
    _check_operand("b", b, 3, (torch.uint8,))
    _check_operand("sfa", sfa, 3, (torch.float32,))
    _check_operand("sfb", sfb, 3, (torch.float32,))
    _check_operand("out", out, 3, (torch.bfloat16,))
    _check_operand("masked_m", masked_m, 1, (torch.int32,))
    G, M_max, K = a.shape
    N = b.shape[1]
    _need(b.shape[0] == G and b.shape[2] * 2 == K and tuple(out.shape) == (G, M_max, N) and masked_m.shape[0] == G,
          "shape mismatch")
    _need(sfa.shape == (G, K // 128, get_tma_aligned_size(M_max, 4)), "sfa must be [G, K/128, tma_aligned(M_max)]")
    _need(sfb.shape == (G, K // 32, get_tma_aligned_size(N, 4)), "sfb must be [G, K/32, tma_aligned(N)]")
    _check(_lib.dg_m_grouped_fp8_fp4_gemm_nt_masked(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(out), _ptr(masked_m),
                                                    G, M_max, N, K, int(expected_m), _stream()))


def m_grouped_fp8_gemm_nt_nopad(lhs, rhs, out: torch.Tensor, counts: torch.Tensor) -> None:
    """No-padding layout: group g's rows are off_g .. off_g + counts[g] - 1 (off_g = sum of the earlier counts);
    out rows of group g = lhs rows of group g @ rhs[g]^T; rows past sum(counts) are untouched."""
    a, sfa = lhs
    b, sfb = rhs
    _check_operand("a", a, 2, _FP8_TYPES)
    _check_operand("b", b, 3, _FP8_TYPES)
    _check_operand("sfa", sfa, 2, (torch.float32,))
    _check_operand("sfb", sfb, 3, (torch.float32,))
    _check_operand("out", out, 2, (torch.bfloat16,))
    _check_operand("counts", counts, 1, (torch.int32,))
    M, K = a.shape
    G, N, _ = b.shape
    _need(b.shape[2] == K and tuple(out.shape) == (M, N) and counts.shape[0] == G, "shape mismatch")
    _need(sfa.shape[0] == K // 128 and sfa.shape[1] == get_tma_aligned_size(M, 4),
          "sfa must be [K/128, tma_aligned(M_total)]")
    _need(sfb.shape == (G, (N + 127) // 128, K // 128), "sfb must be [G, ceil(N/128), K/128]")
    _check(_lib.dg_m_grouped_fp8_gemm_nt_nopad(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(out), _ptr(counts),
                                               M, N, K, G, _stream()))


# --------------------------------------------------------------------------- dispatch, combine, SwiGLU and norms
# Checked and called in _rowwise (csrc/rowwise_binding.cpp): contiguous CUDA tensors on the current device, on whose current
# stream the calls run; DGError for anything else, ImportError if _rowwise.so is missing or of another torch.
def get_m_total_bound(num_slots: int, num_groups: int) -> int:
    """Rows the contiguous layout needs at most for num_slots routed slots and num_groups groups (the size of m_indices,
    and of the GEMM's operands, when the counts are known on the device only)."""
    n = _lib.dg_moe_m_total_bound(int(num_slots), int(num_groups))
    _check(int(n) if n < 0 else DG_OK)
    return n


def moe_sort_contiguous(topk_ids: torch.Tensor, row_of_slot: torch.Tensor, m_indices: torch.Tensor,
                        counts: torch.Tensor) -> None:
    """Rows of the routed slots in the contiguous layout.  topk_ids [T, k] (int32 or int64; -1: no row) -> row_of_slot
    int32 [T, k] (-1: none), m_indices int32 [M_total] as m_grouped_fp8_gemm_nt_contiguous takes it (M_total:
    get_m_total_bound, or any multiple of the alignment that has room), counts int32 [G] rows of each group."""
    _rowwise.moe_sort_contiguous(topk_ids, row_of_slot, m_indices, counts)


def moe_sort_nopad(topk_ids: torch.Tensor, row_of_slot: torch.Tensor, counts: torch.Tensor) -> None:
    """Rows of the routed slots in the no-padding layout: row_of_slot int32 [T, k], counts int32 [G] as
    m_grouped_fp8_gemm_nt_nopad takes them."""
    _rowwise.moe_sort_nopad(topk_ids, row_of_slot, counts)


def moe_sort_masked(topk_ids: torch.Tensor, row_of_slot: torch.Tensor, masked_m: torch.Tensor, m_max: int) -> None:
    """Rows of the routed slots in the masked layout (row g * m_max + i): row_of_slot int32 [T, k], masked_m int32 [G] as
    m_grouped_fp8_gemm_nt_masked takes it.  Slots past m_max of their group get no row (DG_ERR_BAD_GROUP)."""
    _rowwise.moe_sort_masked(topk_ids, row_of_slot, masked_m, m_max)


def moe_permute(x: torch.Tensor, row_of_slot: torch.Tensor, out) -> None:
    """Dispatch: out[row_of_slot[t, s]] = x[t].  x [T, H] bf16 or fp32; out [rows, H] or [G, M_max, H] of x's type, or the
    pair (e4m3, sfa) that a grouped GEMM takes as lhs.  Rows without a slot are left as they were.  The gradient of x is
    moe_unpermute of the rows' gradient without weights."""
    _rowwise.moe_permute(x, row_of_slot, out)


def moe_unpermute(rows: torch.Tensor, row_of_slot: torch.Tensor, out: torch.Tensor,
                  weights: Optional[torch.Tensor] = None) -> None:
    """Combine: out[t] = sum_s weights[t, s] * rows[row_of_slot[t, s]] over the slots with a row, summed in fp32 in the
    slots' order.  rows [R, H] or [G, M_max, H], out [T, H] of the same type; weights fp32 [T, k], None for 1."""
    _rowwise.moe_unpermute(rows, row_of_slot, out, weights)


def moe_unpermute_backward(d_out: torch.Tensor, rows: torch.Tensor, row_of_slot: torch.Tensor, weights: torch.Tensor,
                           d_rows, d_weights: torch.Tensor) -> None:
    """Gradient of moe_unpermute: d_rows[row_of_slot[t, s]] = weights[t, s] * d_out[t] (shaped as rows and of their type,
    or the pair (e4m3, sf)), d_weights[t, s] = <d_out[t], rows[row_of_slot[t, s]]> fp32 (0 for a slot without a row)."""
    _rowwise.moe_unpermute_backward(d_out, rows, row_of_slot, weights, d_rows, d_weights)


def swiglu(gate_up: torch.Tensor, out, m_indices: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
           masked_m: Optional[torch.Tensor] = None) -> None:
    """out = silu(g) * u on the rows that the groups own, gate_up [R, 2 I] = [g | u] (masked: [G, M_max, 2 I]); out [R, I]
    of the same type, or the pair (e4m3, sfa) that the next grouped GEMM takes as lhs.  m_indices, counts or masked_m as
    the GEMM that wrote gate_up took it; none: every row.  Other rows are left as they were."""
    _rowwise.swiglu(None, gate_up, out, m_indices, counts, masked_m)


def swiglu_backward(d_out: torch.Tensor, gate_up: torch.Tensor, d_gate_up, m_indices: Optional[torch.Tensor] = None,
                    counts: Optional[torch.Tensor] = None, masked_m: Optional[torch.Tensor] = None) -> None:
    """Gradient of swiglu: d_gate_up [R, 2 I] = [d_g | d_u] (gate_up's type, or the pair (e4m3, sf) for the data-gradient
    GEMM) from d_out [R, I] and the forward's gate_up, on the same rows."""
    if d_out is None:
        raise DGError(-1, "d_out must be a torch.Tensor")
    _rowwise.swiglu(d_out, gate_up, d_gate_up, m_indices, counts, masked_m)


def rms_norm(x: torch.Tensor, weight: torch.Tensor, out, eps: float = 1e-6, rstd: Optional[torch.Tensor] = None) -> None:
    """out = x * r * weight, r = 1 / sqrt(mean(x^2) + eps) in each row.  x [T, H] bf16 or fp32; weight [H] bf16 or fp32;
    out [T, H] bf16 (fp32 with an fp32 x), or the pair (e4m3, sfa) that fp8_gemm_nt takes as lhs.  rstd fp32 [T] keeps r
    for rms_norm_backward."""
    _rowwise.rms_norm(x, weight, out, eps, rstd)


def rms_norm_backward(d_out: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor, d_x: torch.Tensor,
                      d_weight: torch.Tensor, d_skip: Optional[torch.Tensor] = None) -> None:
    """Gradient of rms_norm: d_x [T, H] of x's type, plus d_skip (the gradient that reaches x past the norm; may be d_x
    itself), and d_weight fp32 [H].  d_out [T, H] of the forward's output type before quantisation."""
    _rowwise.rms_norm_backward(d_out, x, weight, rstd, d_x, d_weight, d_skip)


def residual_rms_norm(x: torch.Tensor, y: torch.Tensor, x_out: torch.Tensor, weight: Optional[torch.Tensor] = None, out=None,
                      weight_post: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, alpha: float = 1.0,
                      eps: float = 1e-6, rstd: Optional[torch.Tensor] = None,
                      rstd_post: Optional[torch.Tensor] = None) -> None:
    """The norms between two blocks: n = y * r_y * weight_post (n = y without weight_post), x_out = x + alpha * gate * n,
    out = x_out * r_x * weight (weight and out go together).  x and x_out [T, H] bf16 or fp32 (x_out may be x); y [T, H] and
    out bf16 (fp32 with an fp32 x), out also the pair (e4m3, sfa); weight and weight_post [H], gate [H] (one type, bf16 or
    fp32) or [T, H] (y's type).  rstd and rstd_post fp32 [T] keep r_x and r_y for residual_rms_norm_backward."""
    _rowwise.residual_rms_norm(x, y, x_out, weight, out, weight_post, gate, alpha, eps, rstd, rstd_post)


def residual_rms_norm_backward(d_x_out: Optional[torch.Tensor], y: torch.Tensor, d_x: torch.Tensor, d_y: torch.Tensor,
                               d_out: Optional[torch.Tensor] = None, x_out: Optional[torch.Tensor] = None,
                               weight: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                               weight_post: Optional[torch.Tensor] = None, rstd_post: Optional[torch.Tensor] = None,
                               gate: Optional[torch.Tensor] = None, alpha: float = 1.0,
                               d_weight: Optional[torch.Tensor] = None, d_weight_post: Optional[torch.Tensor] = None,
                               d_gate: Optional[torch.Tensor] = None) -> None:
    """Gradient of residual_rms_norm.  Comes in: d_x_out (x's type; None: 0) and, with weight, d_out (y's type); x_out as
    the forward stored it, y, the parameters, rstd and rstd_post.  Goes out: d_x (x's type; may be d_x_out), d_y (y's type),
    d_weight and d_weight_post fp32 [H], d_gate fp32 [H] for a gate [H], or of y's type for a gate [T, H]."""
    _rowwise.residual_rms_norm_backward(d_x_out, y, d_x, d_y, d_out, x_out, weight, rstd, weight_post, rstd_post, gate, alpha,
                                        d_weight, d_weight_post, d_gate)


__all__ = [
    "DGError", "fp8_gemm_nt", "fp8_gemm_nt_noalloc", "m_grouped_fp8_gemm_nt_contiguous", "m_grouped_fp8_gemm_nt_masked",
    "m_grouped_fp8_gemm_nt_nopad", "m_grouped_fp8_gemm_nn_contiguous", "k_grouped_fp8_gemm_nt_contiguous",
    "m_grouped_fp8_fp4_gemm_nt_contiguous", "m_grouped_fp8_fp4_gemm_nt_masked",
    "get_m_alignment_for_contiguous_layout", "set_m_alignment_for_contiguous_layout", "get_tma_aligned_size", "set_num_sms", "get_num_sms", "num_tiles",
    "get_m_total_bound", "moe_sort_contiguous", "moe_sort_nopad", "moe_sort_masked", "moe_permute", "moe_unpermute",
    "moe_unpermute_backward", "swiglu", "swiglu_backward", "rms_norm", "rms_norm_backward", "residual_rms_norm",
    "residual_rms_norm_backward",
    "select_block_n", "set_cta_pair_policy", "check_device_error", "lib", "header_symbols", "last_error",
]
