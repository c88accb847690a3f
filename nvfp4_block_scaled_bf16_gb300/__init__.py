"""GB300 (sm_103a) NVFP4 / MXFP4 block-scaled GEMM library -- Python binding of libnvfp4.so.

Thin ctypes marshalling over the C ABI in include/nvfp4.h: each function here has the name of
the C entry point it calls, takes torch CUDA tensors, allocates missing outputs with
torch.empty, checks what the library cannot see behind a bare pointer (device, dtype,
contiguity, size of every buffer), and passes raw pointers and the current CUDA stream.  All
arithmetic runs in the library's CUDA kernels; there is no CPU fallback.  Importing fails if
libnvfp4.so is missing (build it with ``python nvfp4_block_scaled_bf16_gb300/build.py``).
"""
from __future__ import annotations

import ctypes
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libnvfp4.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"{_LIB_PATH} is not built: run `python nvfp4_block_scaled_bf16_gb300/build.py`")
_lib = ctypes.CDLL(_LIB_PATH)

_i64, _u32, _int, _vp, _sz = ctypes.c_int64, ctypes.c_uint32, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
_f32 = ctypes.c_float

FLAG_PDL = 1 << 0
FLAG_SF_SM103 = 1 << 2
FLAG_DEBUG_TIMEOUT = 1 << 8
FLAG_DEBUG_SKIP_FIRST_LOAD = 1 << 9

STATUS = {0: "NVFP4_OK", 1: "NVFP4_ERR_INVALID_ARG", 2: "NVFP4_ERR_MISALIGNED",
          3: "NVFP4_ERR_UNSUPPORTED_SHAPE", 4: "NVFP4_ERR_UNSUPPORTED_DEVICE", 5: "NVFP4_ERR_CUDA",
          6: "NVFP4_ERR_TIMEOUT"}


class PlanT(ctypes.Structure):
    _fields_ = [("swap_ab", _int), ("tile_m", _int), ("tile_n", _int), ("splits", _int),
                ("stages", _int), ("ctas", _int), ("dp_tiles", _int), ("sk_tiles", _int)]


_SIGS = {
    "nvfp4_last_error": (ctypes.c_char_p, []),
    "nvfp4_sf_bytes": (_sz, [_i64, _i64, _int]),
    "mxfp4_grouped_sf_bytes": (_sz, [_i64, _int, _i64]),
    "nvfp4_quantize": (_int, [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _u32, _vp]),
    "mxfp4_quantize": (_int, [_vp, _i64, _i64, _i64, _vp, _int, _vp, _vp, _sz, _u32, _vp]),
    "nvfp4_gemm_plan": (_int, [_i64, _i64, _i64, ctypes.POINTER(PlanT)]),
    "nvfp4_gemm_workspace_size": (_int, [_i64, _i64, _i64, ctypes.POINTER(_sz)]),
    "nvfp4_gemm": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _u32, _vp]),
    "nvfp4_gemm_noalloc": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _u32, _vp]),
    "nvfp4_quantize_gemm": (_int, [_vp, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _u32, _vp]),
    "nvfp4_gated_gemm": (_int, [_vp, _vp, _vp, _vp, _vp, _int, _vp, _i64, _i64, _i64, _vp, _sz, _u32, _vp]),
    "nvfp4_gated_gemm_backward": (_int, [_vp, _vp, _vp, _vp, _vp, _int, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _u32,
                                         _vp]),
    "mxfp4_grouped_gemm": (_int, [_vp, _vp, _vp, _int, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _u32, _vp]),
    "sf_swizzle": (_int, [_vp, _vp, _i64, _i64, _int, _vp]),
    "nvfp4_sf_convert_layout": (_int, [_vp, _vp, _i64, _i64, _int, _vp]),
    "moe_sort_workspace_size": (_sz, [_i64, _int]),
    "moe_sort_by_expert": (_int, [_vp, _i64, _int, _int, _vp, _vp, _vp, _vp, _sz, _u32, _vp]),
    "moe_gather_rows": (_int, [_vp, _i64, _i64, _i64, _vp, _i64, _vp, _u32, _vp]),
    "nvfp4_quantize_experts": (_int, [_vp, _i64, _i64, _i64, _vp, _int, _vp, _vp, _vp, _sz, _u32, _vp]),
    "nvfp4_gather_quantize_experts": (_int, [_vp, _i64, _i64, _i64, _vp, _i64, _vp, _int, _vp, _vp, _vp, _sz, _u32,
                                             _vp]),
    "nvfp4_silu_mul_quantize_experts": (_int, [_vp, _i64, _i64, _i64, _vp, _int, _vp, _vp, _vp, _sz, _u32, _vp]),
    "nvfp4_grouped_gemm": (_int, [_vp, _vp, _vp, _int, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _u32, _vp]),
    "moe_combine": (_int, [_vp, _i64, _vp, _vp, _i64, _int, _i64, _vp, _u32, _vp]),
    "block_norm": (_int, [_vp, _int, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _f32, _f32, _f32, _vp, _i64, _vp, _i64,
                          _i64, _i64, _u32, _vp]),
    "block_norm_quantize": (_int, [_vp, _int, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _f32, _f32, _f32, _vp, _i64, _vp,
                                   _vp, _vp, _i64, _i64, _u32, _vp]),
    "block_norm_backward_workspace_size": (_sz, [_i64, _i64]),
    "block_norm_backward": (_int, [_vp, _i64, _vp, _i64, _vp, _int, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _f32, _f32,
                                   _f32, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _u32, _vp]),
    "sample_tokens": (_int, [_vp, _int, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _u32, _vp]),
    "fp8_padded_rows": (_i64, [_i64, _int]),
    "fp8_quantize": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _i64, _vp, _int, _vp, _vp, _vp, _vp, _u32, _vp]),
    "fp8_quantize_weight": (_int, [_vp, _int, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _u32, _vp]),
    "fp8_gemm": (_int, [_vp, _vp, _vp, _vp, _int, _vp, _int, _int, _i64, _i64, _i64, _u32, _vp]),
    "fp8_grouped_gemm": (_int, [_vp, _vp, _vp, _int, _vp, _vp, _vp, _int, _i64, _i64, _i64, _u32, _vp]),
    "fp8_grouped_weight_grad": (_int, [_vp, _vp, _vp, _vp, _vp, _int, _vp, _int, _int, _i64, _i64, _i64, _u32, _vp]),
    "moe_combine_backward": (_int, [_vp, _i64, _vp, _i64, _vp, _vp, _i64, _int, _i64, _vp, _vp, _u32, _vp]),
    "moe_gather_backward": (_int, [_vp, _i64, _vp, _i64, _int, _i64, _vp, _u32, _vp]),
    "nvfp4_check_status": (_int, [_vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

lib = _lib  # raw ctypes handle (tests call entry points through it directly)
LIB_PATH = _LIB_PATH


class NVFP4Error(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"{STATUS.get(code, code)}: {message}")
        self.code = code


def last_error() -> str:
    return _lib.nvfp4_last_error().decode()


def _check(code: int) -> None:
    if code != 0:
        raise NVFP4Error(code, last_error())


# The pointers and the stream go to ctypes as plain integers (its argument types make them void *), and
# the device and stream are asked of torch's C layer: a small call spends its time here, not on the GPU.
# (Where that layer lacks them, in a torch without CUDA for one, the public functions stand in.)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda device: torch.cuda.current_stream(device).cuda_stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        return _raw_stream(_current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check_device(t, name):
    """The library launches on the current CUDA device; every tensor must live there."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    cur = _current_device()
    if t.get_device() != cur:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{cur}")


def _need(t, dtype, name, dim=None):
    _check_device(t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions")


def _room(t, dtype, name, numel):
    """A buffer the kernels read or write `numel` elements of, densely from its first element (the
    library sees only the pointer, so its size is checked here)."""
    _need(t, dtype, name)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} elements, needs {numel}")


def _on(stream):
    """A context in which the caching allocator and torch's own kernels use the launch stream."""
    return torch.cuda.stream(stream if stream is None or isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream))


def _capturing(stream) -> bool:
    """Whether the launch stream is being captured into a graph."""
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    with _on(stream):
        return torch.cuda.is_current_stream_capturing()


def _contig(t, stream):
    """`t` with dense rows.  A copy is made on the launch stream, so that the caching allocator
    cannot hand its memory out again before that stream's kernel has read it."""
    if t.is_contiguous():
        return t
    if stream is None:
        return t.contiguous()
    with _on(stream):
        return t.contiguous()


def _scratch(nbytes: int, device, stream):
    """An uninitialised uint8 workspace that belongs to the launch stream (see _contig)."""
    if stream is None:
        return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)
    with _on(stream):
        return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def sf_bytes(rows: int, k: int, sf_vec: int = 16) -> int:
    """Bytes of a 128x4-swizzled scale buffer: round_up(rows,128) * round_up(k/sf_vec, 4)."""
    return int(_lib.nvfp4_sf_bytes(rows, k, sf_vec))


def grouped_sf_bytes(total_rows: int, experts: int, k: int) -> int:
    return int(_lib.mxfp4_grouped_sf_bytes(total_rows, experts, k))


def nvfp4_gemm_plan(m: int, n: int, k: int) -> dict:
    p = PlanT()
    _check(_lib.nvfp4_gemm_plan(m, n, k, ctypes.byref(p)))
    return {f: getattr(p, f) for f, _ in PlanT._fields_}


def gemm_workspace_size(m: int, n: int, k: int) -> int:
    """Bytes of workspace nvfp4_gemm needs for (m, n, k) on the current device."""
    v = _sz(0)
    _check(_lib.nvfp4_gemm_workspace_size(m, n, k, ctypes.byref(v)))
    return int(v.value)


def gemm_workspace(nbytes: int, device=None) -> torch.Tensor:
    """A zero-filled uint8 workspace of at least nbytes (the library needs it zero before first use)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


_ws_cache: dict = {}


def _default_workspace(nbytes: int, device: torch.device, stream) -> torch.Tensor:
    """A workspace for a product that was given none: one zeroed buffer per device and launch stream, grown
    on demand.  It is made on that stream, so its zero fill comes before the kernel and what it
    replaces is not handed out before the stream is done with it.  A call under graph capture gets a
    buffer of the graph's, zeroed by every replay."""
    if _capturing(stream):
        with _on(stream):
            ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
            ws[:4096].zero_()      # the counters, one per split tile (at most one tile per two SMs); partials need no zero
            return ws
    key = (device, _stream(stream))
    ws = _ws_cache.get(key)
    if ws is None or ws.numel() < nbytes:
        with _on(stream):
            ws = _ws_cache[key] = gemm_workspace(nbytes, device)
    return ws


def nvfp4_quantize(x, gs, q=None, sf=None, flags: int = 0, stream=None):
    """bf16 [m, k] -> (packed e2m1 uint8 [m, k/2], swizzled e4m3 scales uint8 [sf_bytes])."""
    _need(x, torch.bfloat16, "x", 2)
    _need(gs, torch.float32, "gs")
    if x.stride(1) != 1:
        raise ValueError("x rows must be contiguous")
    m, k = x.shape
    if q is None:
        q = torch.empty((m, k // 2), dtype=torch.uint8, device=x.device)
    if sf is None:
        sf = torch.empty(sf_bytes(m, k, 16), dtype=torch.uint8, device=x.device)
    _room(q, torch.uint8, "q", m * (k // 2))
    _room(sf, torch.uint8, "sf", sf_bytes(m, k, 16))
    _check(_lib.nvfp4_quantize(_ptr(x), m, k, x.stride(0), _ptr(gs), _ptr(q), _ptr(sf), flags, _stream(stream)))
    return q, sf


def mxfp4_quantize(x, row_offsets=None, q=None, sf=None, flags: int = 0, stream=None):
    """bf16 [t, k] -> (packed e2m1 [t, k/2], ue8m0 scales); grouped per expert with row_offsets [E+1]."""
    _need(x, torch.bfloat16, "x", 2)
    if x.stride(1) != 1:
        raise ValueError("x rows must be contiguous")
    t, k = x.shape
    experts = 0
    if row_offsets is not None:
        _need(row_offsets, torch.int64, "row_offsets", 1)
        experts = row_offsets.numel() - 1
    need = grouped_sf_bytes(t, experts, k) if row_offsets is not None else sf_bytes(t, k, 32)
    if q is None:
        q = torch.empty((t, k // 2), dtype=torch.uint8, device=x.device)
    if sf is None:
        sf = torch.zeros(need, dtype=torch.uint8, device=x.device)
    _room(q, torch.uint8, "q", t * (k // 2))
    _room(sf, torch.uint8, "sf", 0)            # its capacity goes to the library, which checks it
    _check(_lib.mxfp4_quantize(_ptr(x), t, k, x.stride(0), _ptr(row_offsets), experts, _ptr(q), _ptr(sf),
                               sf.numel(), flags, _stream(stream)))
    return q, sf


def nvfp4_gemm(a, sfa, b, sfb, alpha, d=None, flags: int = 0, stream=None, workspace=None):
    """D[m, n] = bf16(alpha * deq(a) @ deq(b)^T); a [m, k/2], b [n, k/2] packed uint8.

    workspace: zero-filled uint8 CUDA tensor of at least gemm_workspace_size(m, n, k) bytes
    (the library leaves it zero after each call); None uses one that the calls on a stream share."""
    _need(a, torch.uint8, "a", 2)
    _need(b, torch.uint8, "b", 2)
    _need(sfa, torch.uint8, "sfa")
    _need(sfb, torch.uint8, "sfb")
    _need(alpha, torch.float32, "alpha")
    m, kh = a.shape
    n = b.shape[0]
    if b.shape[1] != kh:
        raise ValueError("a and b disagree on K")
    for t_, name in ((a, "a"), (b, "b")):
        if not t_.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if sfa.numel() < sf_bytes(m, 2 * kh) or sfb.numel() < sf_bytes(n, 2 * kh):
        raise ValueError("scale buffers are too small")
    if d is None:
        d = torch.empty((m, n), dtype=torch.bfloat16, device=a.device)
    _room(d, torch.bfloat16, "d", m * n)
    if workspace is None and m > 0:
        need = gemm_workspace_size(m, n, 2 * kh)
        if need:
            workspace = _default_workspace(need, a.device, stream)
    if workspace is not None:
        _room(workspace, torch.uint8, "workspace", 0)   # the library checks its size
    _check(_lib.nvfp4_gemm(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(alpha), _ptr(d), m, n, 2 * kh,
                           _ptr(workspace), 0 if workspace is None else workspace.numel(), flags,
                           _stream(stream)))
    return d


def nvfp4_quantize_gemm(x, gs, b, sfb, alpha, d=None, flags: int = 0, stream=None):
    """nvfp4_gemm(*nvfp4_quantize(x, gs), b, sfb, alpha) in one kernel (1 <= m <= 256): x bf16
    [m, k] with contiguous rows, b [n, k/2] packed uint8; bit-identical to the two calls."""
    _need(x, torch.bfloat16, "x", 2)
    _need(gs, torch.float32, "gs")
    _need(b, torch.uint8, "b", 2)
    _need(sfb, torch.uint8, "sfb")
    _need(alpha, torch.float32, "alpha")
    if x.stride(1) != 1:
        raise ValueError("x rows must be contiguous")
    if not b.is_contiguous():
        raise ValueError("b must be contiguous")
    m, k = x.shape
    n = b.shape[0]
    if b.shape[1] * 2 != k:
        raise ValueError("x and b disagree on K")
    if sfb.numel() < sf_bytes(n, k):
        raise ValueError("sfb is too small")
    if d is None:
        d = torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    _room(d, torch.bfloat16, "d", m * n)
    _check(_lib.nvfp4_quantize_gemm(_ptr(x), x.stride(0), _ptr(gs), _ptr(b), _ptr(sfb), _ptr(alpha), _ptr(d), m, n, k,
                                    None, 0, flags, _stream(stream)))
    return d


def nvfp4_gemm_noalloc(a, sfa, b, sfb, alpha, d=None, flags: int = 0, stream=None):
    """nvfp4_gemm with the library's static split-K scratch instead of a workspace (never
    allocates on the device beyond the output when d is None).  Not for concurrent use."""
    _need(a, torch.uint8, "a", 2)
    _need(b, torch.uint8, "b", 2)
    _need(sfa, torch.uint8, "sfa")
    _need(sfb, torch.uint8, "sfb")
    _need(alpha, torch.float32, "alpha")
    m, kh = a.shape
    n = b.shape[0]
    if b.shape[1] != kh:
        raise ValueError("a and b disagree on K")
    for t_, name in ((a, "a"), (b, "b")):
        if not t_.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if sfa.numel() < sf_bytes(m, 2 * kh) or sfb.numel() < sf_bytes(n, 2 * kh):
        raise ValueError("scale buffers are too small")
    if d is None:
        d = torch.empty((m, n), dtype=torch.bfloat16, device=a.device)
    _room(d, torch.bfloat16, "d", m * n)
    _check(_lib.nvfp4_gemm_noalloc(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(alpha), _ptr(d), m, n, 2 * kh,
                                   flags, _stream(stream)))
    return d


ACTIVATIONS = {"silu": 0, "gelu_tanh": 1}   # NVFP4_ACT_*


def interleave_gate_up(gate, up):
    """The gate and the up weight [inter, ...] as one [2 inter, ...] matrix whose rows alternate in
    groups of 16, gate rows first: what nvfp4_gated_gemm reads once quantised (inter % 16 == 0).
    Done once per weight."""
    if gate.shape != up.shape or gate.shape[0] % 16:
        raise ValueError(f"gate and up must agree and have a multiple of 16 rows, got {tuple(gate.shape)} and {tuple(up.shape)}")
    groups = (gate.shape[0] // 16, 16) + tuple(gate.shape[1:])
    return torch.stack((gate.reshape(groups), up.reshape(groups)), dim=1).reshape(2 * gate.shape[0], *gate.shape[1:])


def _gated_operands(a, sfa, b, sfb, alpha, activation, workspace, stream):
    """Checks what the gated products share: (m, inter, k, activation, workspace)."""
    _need(a, torch.uint8, "a", 2)
    _need(b, torch.uint8, "b", 2)
    m, kh = a.shape
    n, kb = b.shape
    if kb != kh:
        raise ValueError("a and b disagree on K")
    if n % 2:
        raise ValueError("b must hold as many gate rows as up rows")
    if not a.is_contiguous() or not b.is_contiguous():
        raise ValueError("a and b must be contiguous")
    _room(sfa, torch.uint8, "sfa", sf_bytes(m, 2 * kh))
    _room(sfb, torch.uint8, "sfb", sf_bytes(n, 2 * kh))
    _room(alpha, torch.float32, "alpha", 2)
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
    if workspace is None and m > 0 and n > 0:
        need = gemm_workspace_size(m, n, 2 * kh)
        if need:
            workspace = _default_workspace(need, a.device, stream)
    if workspace is not None:
        _room(workspace, torch.uint8, "workspace", 0)   # the library checks its size
    return m, n // 2, 2 * kh, ACTIVATIONS[activation], workspace


def nvfp4_gated_gemm(a, sfa, b, sfb, alpha, activation: str = "silu", h=None, flags: int = 0, stream=None,
                     workspace=None):
    """h[m, inter] = bf16(act(alpha[0] * a @ gate^T) * (alpha[1] * a @ up^T)): both projections, the
    activation and the product in one kernel.

    a [m, k/2] packed, b [2 inter, k/2] packed with gate and up rows alternating in groups of 16
    (interleave_gate_up), alpha fp32 [2], activation "silu" or "gelu_tanh"; workspace as nvfp4_gemm."""
    m, inter, k, act, workspace = _gated_operands(a, sfa, b, sfb, alpha, activation, workspace, stream)
    if h is None:
        h = a.new_empty((m, inter), dtype=torch.bfloat16)
    else:
        _room(h, torch.bfloat16, "h", m * inter)
    _check(_lib.nvfp4_gated_gemm(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(alpha), act, _ptr(h), m, inter, k,
                                 _ptr(workspace), 0 if workspace is None else workspace.numel(), flags, _stream(stream)))
    return h


def nvfp4_gated_gemm_backward(a, sfa, b, sfb, alpha, dh, activation: str = "silu", dgu=None, h=None, flags: int = 0,
                              stream=None, workspace=None):
    """The gradients of nvfp4_gated_gemm's two products given dh, the gradient of h (bf16 [m, inter]).

    Returns (dgu, h): dgu bf16 [m, 2 inter] in the row order of b, and the forward result, both
    computed again from the packed operands."""
    m, inter, k, act, workspace = _gated_operands(a, sfa, b, sfb, alpha, activation, workspace, stream)
    _need(dh, torch.bfloat16, "dh", 2)
    if tuple(dh.shape) != (m, inter):
        raise ValueError(f"dh must have shape {(m, inter)}, got {tuple(dh.shape)}")
    dh = _contig(dh, stream)
    if dgu is None:
        dgu = torch.empty((m, 2 * inter), dtype=torch.bfloat16, device=a.device)
    if h is None:
        h = torch.empty((m, inter), dtype=torch.bfloat16, device=a.device)
    _room(dgu, torch.bfloat16, "dgu", m * 2 * inter)
    _room(h, torch.bfloat16, "h", m * inter)
    _check(_lib.nvfp4_gated_gemm_backward(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(alpha), act, _ptr(dh), _ptr(dgu),
                                          _ptr(h), m, inter, k, _ptr(workspace),
                                          0 if workspace is None else workspace.numel(), flags, _stream(stream)))
    return dgu, h


def mxfp4_grouped_gemm(a, sfa, row_offsets, b, sfb, alpha=None, d=None, flags: int = 0, stream=None):
    """Per expert e: D[rows of e] = bf16(alpha * deq(A_e) @ deq(B_e)^T); b [E, n, k/2]."""
    _need(a, torch.uint8, "a", 2)
    _need(b, torch.uint8, "b", 3)
    _need(row_offsets, torch.int64, "row_offsets", 1)
    t, kh = a.shape
    experts, n, kb = b.shape
    if kb != kh or row_offsets.numel() != experts + 1:
        raise ValueError("shape mismatch")
    if not b.is_contiguous():
        raise ValueError("b must be contiguous")
    _need(sfa, torch.uint8, "sfa")
    _room(sfb, torch.uint8, "sfb", experts * sf_bytes(n, 2 * kh, 32))
    if alpha is not None:
        _room(alpha, torch.float32, "alpha", 1)
    if d is None:
        d = torch.empty((t, n), dtype=torch.bfloat16, device=a.device)
    _room(d, torch.bfloat16, "d", t * n)
    _check(_lib.mxfp4_grouped_gemm(_ptr(a), _ptr(sfa), _ptr(row_offsets), experts, _ptr(b), _ptr(sfb),
                                   _ptr(alpha), _ptr(d), t, n, 2 * kh, flags, _stream(stream)))
    return d


def sf_swizzle(src, rows: int, cols: int, to_swizzled: bool = True, dst=None, stream=None):
    """Row-major scale bytes [rows, cols] <-> 128x4 swizzled buffer."""
    padded = (-(-rows // 128) * 128) * (-(-cols // 4) * 4)
    _room(src, torch.uint8, "src", rows * cols if to_swizzled else padded)
    if dst is None:
        dst = torch.empty(padded if to_swizzled else rows * cols, dtype=torch.uint8, device=src.device)
    _room(dst, torch.uint8, "dst", padded if to_swizzled else rows * cols)
    _check(_lib.sf_swizzle(_ptr(src), _ptr(dst), rows, cols, 1 if to_swizzled else 0, _stream(stream)))
    return dst


def sf_convert_layout(src, rows: int, cols: int, to_sm103: bool = True, dst=None, stream=None):
    """Swizzled NVFP4 scale buffer: 128x4 ("SM100") layout <-> SM103 layout."""
    padded = (-(-rows // 128) * 128) * (-(-cols // 4) * 4)
    _room(src, torch.uint8, "src", padded)
    if dst is None:
        dst = torch.empty_like(src)
    _room(dst, torch.uint8, "dst", padded)
    _check(_lib.nvfp4_sf_convert_layout(_ptr(src), _ptr(dst), rows, cols, 1 if to_sm103 else 0, _stream(stream)))
    return dst


# ---------------------------------------------------------------- MoE steps (NVFP4)
def expert_sf_bytes(total_rows: int, experts: int, k: int) -> int:
    """Grouped NVFP4 scale buffer bound: (round_up(t,128) + 128 E) * round_up(k/16, 4)."""
    return (-(-total_rows // 128) * 128 + 128 * experts) * (-(-(k // 16) // 4) * 4)


def moe_sort_workspace_size(num_tokens: int, num_experts: int) -> int:
    return int(_lib.moe_sort_workspace_size(num_tokens, num_experts))


def moe_sort_by_expert(topk_ids, num_experts: int, out=None, workspace=None, flags: int = 0, stream=None):
    """int32 [T, topk] expert ids -> (row_offsets int64 [E+1], src_rows int32 [T*topk],
    pos int32 [T, topk]); stable: (token, slot) order inside an expert.  `out` may pass the
    three output tensors to fill."""
    _need(topk_ids, torch.int32, "topk_ids", 2)
    topk_ids = _contig(topk_ids, stream)
    T, topk = topk_ids.shape
    dv = topk_ids.device
    if out is None:
        out = (torch.empty(num_experts + 1, dtype=torch.int64, device=dv),
               torch.empty(T * topk, dtype=torch.int32, device=dv),
               torch.empty((T, topk), dtype=torch.int32, device=dv))
    ro, src, pos = out
    _room(ro, torch.int64, "row_offsets", num_experts + 1)
    _room(src, torch.int32, "src_rows", T * topk)
    _room(pos, torch.int32, "pos", T * topk)
    if workspace is None:
        workspace = torch.empty(max(1, moe_sort_workspace_size(T, num_experts) // 4), dtype=torch.int32, device=dv)
    _room(workspace, torch.int32, "workspace", 0)        # its size in bytes goes to the library
    _check(_lib.moe_sort_by_expert(_ptr(topk_ids), T, topk, num_experts, _ptr(ro), _ptr(src), _ptr(pos),
                                   _ptr(workspace), workspace.numel() * 4, flags, _stream(stream)))
    return ro, src, pos


def moe_gather_rows(x, src_rows, out=None, flags: int = 0, stream=None):
    """out[r] = x[src_rows[r]] (bf16 rows)."""
    _need(x, torch.bfloat16, "x", 2)
    _need(src_rows, torch.int32, "src_rows", 1)
    if x.stride(1) != 1:
        raise ValueError("x rows must be contiguous")
    T, h = x.shape
    rows = src_rows.numel()
    if out is None:
        out = torch.empty((rows, h), dtype=torch.bfloat16, device=x.device)
    if not src_rows.is_contiguous():
        raise ValueError("src_rows must be contiguous")
    _room(out, torch.bfloat16, "out", rows * h)
    _check(_lib.moe_gather_rows(_ptr(x), T, h, x.stride(0), _ptr(src_rows), rows, _ptr(out), flags, _stream(stream)))
    return out


def nvfp4_quantize_experts(x, row_offsets, gs, q=None, sf=None, flags: int = 0, stream=None):
    """bf16 [t, k] (rows by expert) -> (packed e2m1 [t, k/2], grouped e4m3 scales); gs fp32 [E]."""
    _need(x, torch.bfloat16, "x", 2)
    _need(row_offsets, torch.int64, "row_offsets", 1)
    _need(gs, torch.float32, "gs", 1)
    t, k = x.shape
    experts = row_offsets.numel() - 1
    if q is None:
        q = torch.empty((t, k // 2), dtype=torch.uint8, device=x.device)
    if sf is None:
        sf = torch.empty(expert_sf_bytes(t, experts, k), dtype=torch.uint8, device=x.device)
    _room(row_offsets, torch.int64, "row_offsets", experts + 1)
    _room(gs, torch.float32, "gs", experts)
    _room(q, torch.uint8, "q", t * (k // 2))
    _room(sf, torch.uint8, "sf", 0)            # its capacity goes to the library, which checks it
    _check(_lib.nvfp4_quantize_experts(_ptr(x), t, k, x.stride(0), _ptr(row_offsets), experts, _ptr(gs), _ptr(q),
                                       _ptr(sf), sf.numel(), flags, _stream(stream)))
    return q, sf


def nvfp4_gather_quantize_experts(x, src_rows, row_offsets, gs, q=None, sf=None, flags: int = 0, stream=None):
    """Row r of the result quantises x[src_rows[r]]: moe_gather_rows + nvfp4_quantize_experts in one launch."""
    _need(x, torch.bfloat16, "x", 2)
    _need(src_rows, torch.int32, "src_rows", 1)
    _need(row_offsets, torch.int64, "row_offsets", 1)
    _need(gs, torch.float32, "gs", 1)
    if x.stride(1) != 1:
        raise ValueError("x rows must be contiguous")
    if not src_rows.is_contiguous():
        raise ValueError("src_rows must be contiguous")
    tokens, k = x.shape
    rows = src_rows.numel()
    experts = row_offsets.numel() - 1
    if q is None:
        q = torch.empty((rows, k // 2), dtype=torch.uint8, device=x.device)
    if sf is None:
        sf = torch.empty(expert_sf_bytes(rows, experts, k), dtype=torch.uint8, device=x.device)
    _room(row_offsets, torch.int64, "row_offsets", experts + 1)
    _room(gs, torch.float32, "gs", experts)
    _room(q, torch.uint8, "q", rows * (k // 2))
    _room(sf, torch.uint8, "sf", 0)            # its capacity goes to the library, which checks it
    _check(_lib.nvfp4_gather_quantize_experts(_ptr(x), tokens, k, x.stride(0), _ptr(src_rows), rows,
                                              _ptr(row_offsets), experts, _ptr(gs), _ptr(q), _ptr(sf), sf.numel(),
                                              flags, _stream(stream)))
    return q, sf


def nvfp4_silu_mul_quantize_experts(x, row_offsets, gs, q=None, sf=None, flags: int = 0, stream=None):
    """bf16 [t, 2I] = [gate | up] -> NVFP4 of h = bf16(silu(gate) * up): (q [t, I/2], grouped scales)."""
    _need(x, torch.bfloat16, "x", 2)
    _need(row_offsets, torch.int64, "row_offsets", 1)
    _need(gs, torch.float32, "gs", 1)
    t, w = x.shape
    inter = w // 2
    experts = row_offsets.numel() - 1
    if q is None:
        q = torch.empty((t, inter // 2), dtype=torch.uint8, device=x.device)
    if sf is None:
        sf = torch.empty(expert_sf_bytes(t, experts, inter), dtype=torch.uint8, device=x.device)
    _room(row_offsets, torch.int64, "row_offsets", experts + 1)
    _room(gs, torch.float32, "gs", experts)
    _room(q, torch.uint8, "q", t * (inter // 2))
    _room(sf, torch.uint8, "sf", 0)
    _check(_lib.nvfp4_silu_mul_quantize_experts(_ptr(x), t, inter, x.stride(0), _ptr(row_offsets), experts, _ptr(gs),
                                                _ptr(q), _ptr(sf), sf.numel(), flags, _stream(stream)))
    return q, sf


def nvfp4_grouped_gemm(a, sfa, row_offsets, b, sfb, alpha=None, d=None, flags: int = 0, stream=None):
    """Per expert e: D[rows of e] = bf16(alpha[e] * deq(A_e) @ deq(B_e)^T); b [E, n, k/2], alpha fp32 [E]."""
    _need(a, torch.uint8, "a", 2)
    _need(b, torch.uint8, "b", 3)
    _need(row_offsets, torch.int64, "row_offsets", 1)
    t, kh = a.shape
    experts, n, kb = b.shape
    if kb != kh or row_offsets.numel() != experts + 1 or (alpha is not None and alpha.numel() != experts):
        raise ValueError("shape mismatch")
    if not b.is_contiguous():
        raise ValueError("b must be contiguous")
    _need(sfa, torch.uint8, "sfa")
    _room(sfb, torch.uint8, "sfb", experts * sf_bytes(n, 2 * kh, 16))
    if alpha is not None:
        _room(alpha, torch.float32, "alpha", experts)
    if d is None:
        d = torch.empty((t, n), dtype=torch.bfloat16, device=a.device)
    _room(d, torch.bfloat16, "d", t * n)
    _check(_lib.nvfp4_grouped_gemm(_ptr(a), _ptr(sfa), _ptr(row_offsets), experts, _ptr(b), _ptr(sfb), _ptr(alpha),
                                   _ptr(d), t, n, 2 * kh, flags, _stream(stream)))
    return d


def moe_combine(y, pos, weights, out=None, flags: int = 0, stream=None):
    """out[t] = bf16(sum_j weights[t, j] * y[pos[t, j]]) (fp32, slot order)."""
    _need(y, torch.bfloat16, "y", 2)
    _need(pos, torch.int32, "pos", 2)
    _need(weights, torch.float32, "weights", 2)
    if not y.is_contiguous():
        raise ValueError("y must be contiguous")
    rows, h = y.shape
    T, topk = pos.shape
    if tuple(weights.shape) != (T, topk):
        raise ValueError(f"weights must have shape {(T, topk)}, got {tuple(weights.shape)}")
    pos, weights = _contig(pos, stream), _contig(weights, stream)
    if out is None:
        out = torch.empty((T, h), dtype=torch.bfloat16, device=y.device)
    _room(out, torch.bfloat16, "out", T * h)
    _check(_lib.moe_combine(_ptr(y), rows, _ptr(pos), _ptr(weights), T, topk, h, _ptr(out),
                            flags, _stream(stream)))
    return out


# ---------------------------------------------------------------- norms around a decoder block
_STREAM_TYPES = {torch.bfloat16: 0, torch.float32: 1}   # NVFP4_DTYPE_*


def _rows(t, dtype, name, m, n, dev):
    """A [m, n] operand on device `dev` with contiguous rows at any row stride; returns the stride."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.dim() == 2):
        _need(t, dtype, name, 2)
        raise ValueError(f"{name} is on another device")
    ld, step = t.stride()
    if t.shape != (m, n):
        raise ValueError(f"{name} must have shape {(m, n)}, got {tuple(t.shape)}")
    if step != 1 and n > 1:
        raise ValueError(f"{name} rows must be contiguous")
    return ld if m > 1 else max(n, ld)


def _vector(t, dtype, name, n, dev):
    """A contiguous [n] vector on device `dev` (None: absent)."""
    if t is None:
        return
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.dim() == 1):
        _need(t, dtype, name, 1)
        raise ValueError(f"{name} is on another device")
    if t.numel() != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {n}")


def _block_operands(x, w_pre, y, w_post, gate, stream):
    """Checks what the forward and backward norms share:
    (x_type, m, n, device index, row strides of x, y and gate, gate)."""
    _check_device(x, "x")
    xt = _STREAM_TYPES.get(x.dtype)
    if xt is None:
        raise TypeError(f"x must be bfloat16 or float32, got {x.dtype}")
    if x.dim() != 2:
        raise ValueError("x must have 2 dimensions")
    m, n = x.shape
    dev = x.get_device()
    ldx = _rows(x, x.dtype, "x", m, n, dev)
    _vector(w_pre, torch.bfloat16, "w_pre", n, dev)
    if y is None:
        if w_post is not None or gate is not None:
            raise ValueError("w_post and gate belong to y")
        return xt, m, n, dev, ldx, 0, 0, None
    ldy = _rows(y, torch.bfloat16, "y", m, n, dev)
    _vector(w_post, torch.bfloat16, "w_post", n, dev)
    ldg = 0
    if gate is not None:
        if isinstance(gate, torch.Tensor) and gate.dim() == 2:
            ldg = _rows(gate, torch.bfloat16, "gate", m, n, dev)
            if ldg < n:      # rows expanded from one: a gate per token still, with a gradient per token
                gate = _contig(gate, stream)
                ldg = n
        else:
            _vector(gate, torch.bfloat16, "gate", n, dev)
    return xt, m, n, dev, ldx, ldy, ldg, gate


def _stream_out(x, y, x_out, m, n, dev):
    """x_out (made where it is missing) and its row stride."""
    if y is None:
        if x_out is not None:
            raise ValueError("x_out belongs to y")
        return None, 0
    if x_out is None:
        return x.new_empty((m, n)), n
    return x_out, _rows(x_out, x.dtype, "x_out", m, n, dev)


def block_norm(x, w_pre=None, y=None, w_post=None, gate=None, residual_scale: float = 1.0, eps: float = 1e-6,
               weight_offset: float = 0.0, x_out=None, h=None, flags: int = 0, stream=None):
    """The RMS norm after a block (w_post), its gate, the residual sum and the norm before the next
    block (w_pre), one pass: r = x + residual_scale * gate * norm(y), h = norm(r).

    x bf16 or fp32 [m, n], y bf16 [m, n] or None (h = norm(x) only), weights bf16 [n] or None, gate
    bf16 [n] or [m, n] or None.  Returns (x_out, h): the stream in x's type (x itself without y) and
    bf16 [m, n] (None without w_pre).  x_out may be x."""
    xt, m, n, dev, ldx, ldy, ldg, gate = _block_operands(x, w_pre, y, w_post, gate, stream)
    x_out, ldo = _stream_out(x, y, x_out, m, n, dev)
    ldh = n
    if w_pre is None:
        if h is not None:
            raise ValueError("h belongs to w_pre")
    elif h is None:
        h = x.new_empty((m, n), dtype=torch.bfloat16)
    else:
        ldh = _rows(h, torch.bfloat16, "h", m, n, dev)
    _check(_lib.block_norm(_ptr(x), xt, ldx, _ptr(y), ldy, _ptr(w_post), _ptr(gate), ldg, _ptr(w_pre), residual_scale,
                           eps, weight_offset, _ptr(x_out), ldo, _ptr(h), ldh, m, n, flags, _stream(stream)))
    return (x if y is None else x_out), h


def block_norm_quantize(x, w_pre, gs, y=None, w_post=None, gate=None, residual_scale: float = 1.0, eps: float = 1e-6,
                        weight_offset: float = 0.0, x_out=None, q=None, sf=None, flags: int = 0, stream=None):
    """block_norm whose h is quantised on the way out: (x_out, q, sf) with q and sf equal to
    nvfp4_quantize(h, gs)."""
    xt, m, n, dev, ldx, ldy, ldg, gate = _block_operands(x, w_pre, y, w_post, gate, stream)
    if w_pre is None:
        raise ValueError("w_pre is needed")
    _room(gs, torch.float32, "gs", 1)
    x_out, ldo = _stream_out(x, y, x_out, m, n, dev)
    need = sf_bytes(m, n // 16 * 16, 16)
    if q is None:
        q = x.new_empty((m, n // 2), dtype=torch.uint8)
    else:
        _room(q, torch.uint8, "q", m * (n // 2))
    if sf is None:
        sf = x.new_empty(need, dtype=torch.uint8)
    else:
        _room(sf, torch.uint8, "sf", need)
    _check(_lib.block_norm_quantize(_ptr(x), xt, ldx, _ptr(y), ldy, _ptr(w_post), _ptr(gate), ldg, _ptr(w_pre),
                                    residual_scale, eps, weight_offset, _ptr(x_out), ldo, _ptr(gs), _ptr(q), _ptr(sf),
                                    m, n, flags, _stream(stream)))
    return (x if y is None else x_out), q, sf


def block_norm_backward_workspace_size(m: int, n: int) -> int:
    return int(_lib.block_norm_backward_workspace_size(m, n))


def block_norm_backward(dh, dx_out, x_out, w_pre=None, y=None, w_post=None, gate=None, residual_scale: float = 1.0,
                        eps: float = 1e-6, weight_offset: float = 0.0, workspace=None, flags: int = 0, stream=None):
    """Backward pass of block_norm: dh the gradient of h (None without w_pre), dx_out the gradient that
    reaches x_out from elsewhere (None: zero), x_out the stream the forward pass returned.

    Returns (dx, dy, dw_pre, dw_post, dgate): dx in x_out's type, dy bf16, the weights' gradients fp32 [n],
    dgate fp32 [n] for a gate per channel or bf16 [m, n] for a gate per token; None for what was absent."""
    xt, m, n, dev, ldr, ldy, ldg, gate = _block_operands(x_out, w_pre, y, w_post, gate, stream)
    if (dh is None) != (w_pre is None):
        raise ValueError("dh and w_pre: give both or neither")
    lddh = 0 if dh is None else _rows(dh, torch.bfloat16, "dh", m, n, dev)
    lddr = 0 if dx_out is None else _rows(dx_out, x_out.dtype, "dx_out", m, n, dev)

    def new(shape, dtype, wanted):
        return x_out.new_empty(shape, dtype=dtype) if wanted else None

    dx = x_out.new_empty((m, n))
    dy = new((m, n), torch.bfloat16, y is not None)
    dw_pre = new(n, torch.float32, w_pre is not None)
    dw_post = new(n, torch.float32, w_post is not None)
    dgate = new((m, n), torch.bfloat16, True) if ldg else new(n, torch.float32, gate is not None)
    if workspace is None:
        # made on the launch stream, so that its memory is not handed out before that stream is done with it
        workspace = _scratch(block_norm_backward_workspace_size(m, n), x_out.device, stream)
    _room(workspace, torch.uint8, "workspace", 0)      # the library checks its size
    _check(_lib.block_norm_backward(_ptr(dh), lddh, _ptr(dx_out), lddr, _ptr(x_out), xt, ldr, _ptr(y), ldy, _ptr(w_post),
                                    _ptr(gate), ldg, _ptr(w_pre), residual_scale, eps, weight_offset, _ptr(dx), n,
                                    _ptr(dy), n, _ptr(dw_pre), _ptr(dw_post), _ptr(dgate), n if ldg else 0, m, n,
                                    _ptr(workspace), workspace.numel(), flags, _stream(stream)))
    return dx, dy, dw_pre, dw_post, dgate


# ---------------------------------------------------------------- draw of the next token
def sample_tokens(logits, uniform, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None, logprobs=None,
                  flags: int = 0, stream=None):
    """One token per row of logits (bf16 or fp32 [rows, vocab], any row stride) from uniform, fp32 [rows]
    in [0, 1).  temperature, top_p, min_p fp32 [rows] and top_k int32 [rows], each None for off; a
    temperature <= 0 takes the largest logit.  Ties go to the lowest index; the result does not depend on
    how the work is split.

    Returns (tokens int32 [rows], logprobs fp32 [rows]): -1 where a row holds nothing but -inf and NaN;
    the log-probability is the one among the tokens the filters kept."""
    _check_device(logits, "logits")
    lt = _STREAM_TYPES.get(logits.dtype)
    if lt is None:
        raise TypeError(f"logits must be bfloat16 or float32, got {logits.dtype}")
    if logits.dim() != 2:
        raise ValueError("logits must have 2 dimensions")
    rows, vocab = logits.shape
    dev = logits.get_device()
    ld = _rows(logits, logits.dtype, "logits", rows, vocab, dev)
    if uniform is None:
        raise TypeError("uniform is needed")
    _vector(uniform, torch.float32, "uniform", rows, dev)
    _vector(temperature, torch.float32, "temperature", rows, dev)
    _vector(top_k, torch.int32, "top_k", rows, dev)
    _vector(top_p, torch.float32, "top_p", rows, dev)
    _vector(min_p, torch.float32, "min_p", rows, dev)
    if tokens is None:
        tokens = logits.new_empty(rows, dtype=torch.int32)
    else:
        _vector(tokens, torch.int32, "tokens", rows, dev)
    if logprobs is None:
        logprobs = logits.new_empty(rows, dtype=torch.float32)
    else:
        _vector(logprobs, torch.float32, "logprobs", rows, dev)
    _check(_lib.sample_tokens(_ptr(logits), lt, ld, _ptr(uniform), _ptr(temperature), _ptr(top_k),
                              _ptr(top_p), _ptr(min_p), _ptr(tokens), _ptr(logprobs), rows, vocab, flags, _stream(stream)))
    return tokens, logprobs


# ---------------------------------------------------------------- 8-bit products with a scale per block of 128
E4M3 = torch.float8_e4m3fn


def _type_of(t, name):
    """NVFP4_DTYPE_* of a bf16 or fp32 tensor."""
    xt = _STREAM_TYPES.get(t.dtype)
    if xt is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    return xt


def _dense(t, dtype, name, shape, dev):
    """A contiguous tensor of this type and shape on device `dev`."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return
    _need(t, dtype, name)
    if t.get_device() != dev:
        raise ValueError(f"{name} is on another device")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _is(t, dtype, dim, dev):
    """Whether `t` is a contiguous tensor of this type on device `dev` (one test for a small call; where it fails,
    _need and the others say why)."""
    return isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.dim() == dim and t.is_contiguous()


def _made(t, dtype, name, shape, dev, stream):
    """The output tensor `t`, or a new one (made for the launch stream, so that its memory belongs to it: see _contig)."""
    if t is not None:
        _dense(t, dtype, name, shape, dev.index if dev.index is not None else -1)
        return t
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with _on(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def fp8_padded_rows(rows: int, experts: int = 0) -> int:
    """Columns of fp8_quantize's transposed codes: round_up(rows, 128) + 128 * experts."""
    return int(_lib.fp8_padded_rows(rows, experts))


def fp8_quantize(x, src_rows=None, row_offsets=None, rows: bool = True, transpose: bool = False, q=None, sf=None, qt=None,
                 sft=None, flags: int = 0, stream=None):
    """e4m3 codes of x (bf16 or fp32 [n, k], k % 16 == 0) with one fp32 scale per block of 128.

    Along the rows (rows=True): q [m, k], sf [ceil(k/128), m].  Along the columns and transposed
    (transpose=True): qt [k, P], sft [P/128, k] with P = fp8_padded_rows(m, experts); with row_offsets (int64
    [E+1]) each expert's rows begin at a multiple of 128 there, and rows past the last expert's are not quantised (q and
    sf stay as they were there; new ones hold whatever their memory held).  src_rows (int32 [m]): row r of the result is
    x[src_rows[r]] (without it m = n).  Returns (q, sf), (qt, sft) or (q, sf, qt, sft); x is read once."""
    if _is(x, torch.bfloat16, 2, _current_device()):
        xt, (n, k) = 0, x.shape
        ldx = k
    else:
        _check_device(x, "x")
        xt = _type_of(x, "x")
        if x.dim() != 2:
            raise ValueError("x must have 2 dimensions")
        n, k = x.shape
        ldx = _rows(x, x.dtype, "x", n, k, x.get_device())
    dev = x.device
    m, experts = n, 0
    src_p = ro_p = q_p = sf_p = qt_p = sft_p = None
    if src_rows is not None:
        _need(src_rows, torch.int32, "src_rows", 1)
        if not src_rows.is_contiguous():
            raise ValueError("src_rows must be contiguous")
        m = src_rows.numel()
        src_p = src_rows.data_ptr()
    if row_offsets is not None:
        if not transpose:
            raise ValueError("row_offsets belong to transpose")
        _need(row_offsets, torch.int64, "row_offsets", 1)
        if not row_offsets.is_contiguous() or row_offsets.numel() < 2:
            raise ValueError("row_offsets must be contiguous and hold at least two entries")
        experts = row_offsets.numel() - 1
        ro_p = row_offsets.data_ptr()
    if rows:
        q = _made(q, E4M3, "q", (m, k), dev, stream)
        sf = _made(sf, torch.float32, "sf", (-(-k // 128), m), dev, stream)
        q_p, sf_p = q.data_ptr(), sf.data_ptr()
    elif not transpose:
        raise ValueError("rows or transpose: one at least")
    elif q is not None or sf is not None:
        raise ValueError("q and sf belong to rows")
    if transpose:
        p = -(-m // 128) + experts
        qt = _made(qt, E4M3, "qt", (k, 128 * p), dev, stream)
        sft = _made(sft, torch.float32, "sft", (p, k), dev, stream)
        qt_p, sft_p = qt.data_ptr(), sft.data_ptr()
    elif qt is not None or sft is not None:
        raise ValueError("qt and sft belong to transpose")
    _check(_lib.fp8_quantize(x.data_ptr(), xt, n, k, ldx, src_p, m, ro_p, experts, q_p, sf_p, qt_p, sft_p, flags,
                             _stream(stream)))
    return (q, sf, qt, sft) if rows and transpose else (q, sf) if rows else (qt, sft)


def fp8_quantize_weight(w, transpose: bool = False, q=None, sf=None, qt=None, sft=None, flags: int = 0, stream=None):
    """e4m3 codes of one weight or several (bf16 or fp32 [n, k] or [E, n, k], contiguous rows) with one fp32 scale
    per 128 x 128 block: (q, sf [.., ceil(n/128), ceil(k/128)]), and with transpose the same codes and scales
    transposed: (q, sf, qt, sft)."""
    _check_device(w, "w")
    wt = _type_of(w, "w")
    if w.dim() not in (2, 3):
        raise ValueError("w must have 2 or 3 dimensions")
    n, k = w.shape[-2:]
    lead = tuple(w.shape[:-2])
    matrices = lead[0] if lead else 1
    if lead:
        if not w.is_contiguous():
            raise ValueError("w must be contiguous")
        ldw = k
    else:
        ldw = _rows(w, w.dtype, "w", n, k, w.get_device())
    nb, kb, dev = -(-n // 128), -(-k // 128), w.device
    q, sf = _made(q, E4M3, "q", lead + (n, k), dev, stream), _made(sf, torch.float32, "sf", lead + (nb, kb), dev, stream)
    if transpose:
        qt = _made(qt, E4M3, "qt", lead + (k, n), dev, stream)
        sft = _made(sft, torch.float32, "sft", lead + (kb, nb), dev, stream)
    elif qt is not None or sft is not None:
        raise ValueError("qt and sft belong to transpose")
    _check(_lib.fp8_quantize_weight(w.data_ptr(), wt, matrices, n, k, ldw, q.data_ptr(), sf.data_ptr(), _ptr(qt), _ptr(sft),
                                    flags, _stream(stream)))
    return (q, sf, qt, sft) if transpose else (q, sf)


def _codes(a, da, b, db):
    """Checks a product's codes; returns their device."""
    dev = _current_device()
    if not (_is(a, E4M3, da, dev) and _is(b, E4M3, db, dev)):
        _need(a, E4M3, "a", da)
        _need(b, E4M3, "b", db)
        raise ValueError("a and b must be contiguous")
    return dev


def _product_out(d, out_dtype, accumulate, shape, dev, stream):
    """(d, its NVFP4_DTYPE_*)."""
    if d is not None:
        out_dtype = d.dtype if isinstance(d, torch.Tensor) else None
    elif accumulate:
        raise ValueError("accumulate needs d")
    dt = _STREAM_TYPES.get(out_dtype)
    if dt is None:
        raise TypeError(f"the result must be bfloat16 or float32, got {out_dtype}")
    return _made(d, out_dtype, "d", shape, dev, stream), dt


def fp8_gemm(a, sfa, b, sfb, block_b: int = 128, out_dtype=torch.bfloat16, d=None, accumulate: bool = False, flags: int = 0,
             stream=None):
    """D[m, n] = deq(a) @ deq(b)^T; a [m, k] and b [n, k] e4m3, sfa fp32 [ceil(k/128), m] (fp8_quantize), sfb
    fp32 [ceil(n/128), ceil(k/128)] (block_b=128, fp8_quantize_weight) or [ceil(k/128), n] (block_b=1,
    fp8_quantize).  D is bf16 or fp32; accumulate adds to an fp32 d."""
    dev = _codes(a, 2, b, 2)
    m, k = a.shape
    n, kb = b.shape
    if kb != k:
        raise ValueError("a and b disagree on K")
    if block_b not in (1, 128):
        raise ValueError(f"block_b must be 1 or 128, got {block_b}")
    kb = -(-k // 128)
    _dense(sfa, torch.float32, "sfa", (kb, m), dev)
    _dense(sfb, torch.float32, "sfb", (-(-n // 128), kb) if block_b == 128 else (kb, n), dev)
    d, dt = _product_out(d, out_dtype, accumulate, (m, n), a.device, stream)
    _check(_lib.fp8_gemm(a.data_ptr(), sfa.data_ptr(), b.data_ptr(), sfb.data_ptr(), block_b, d.data_ptr(), dt,
                         1 if accumulate else 0, m, n, k, flags, _stream(stream)))
    return d


def fp8_grouped_gemm(a, sfa, row_offsets, b, sfb, out_dtype=torch.bfloat16, d=None, flags: int = 0, stream=None):
    """Per expert e: D[rows of e] = deq(A_e) @ deq(B_e)^T; a e4m3 [t, k] with its rows sorted by expert (sfa
    [ceil(k/128), t]), b e4m3 [E, n, k] (sfb [E, ceil(n/128), ceil(k/128)]), D bf16 or fp32.  Rows past the last
    expert's stay as they were (in a new D: whatever its memory held)."""
    dev = _codes(a, 2, b, 3)
    t, k = a.shape
    experts, n, kb = b.shape
    if kb != k:
        raise ValueError("a and b disagree on K")
    kb = -(-k // 128)
    _dense(row_offsets, torch.int64, "row_offsets", (experts + 1,), dev)
    _dense(sfa, torch.float32, "sfa", (kb, t), dev)
    _dense(sfb, torch.float32, "sfb", (experts, -(-n // 128), kb), dev)
    d, dt = _product_out(d, out_dtype, False, (t, n), a.device, stream)
    _check(_lib.fp8_grouped_gemm(a.data_ptr(), sfa.data_ptr(), row_offsets.data_ptr(), experts, b.data_ptr(), sfb.data_ptr(),
                                 d.data_ptr(), dt, t, n, k, flags, _stream(stream)))
    return d


def fp8_grouped_weight_grad(a, sfa, b, sfb, row_offsets, out_dtype=torch.bfloat16, d=None, accumulate: bool = False,
                            flags: int = 0, stream=None):
    """Per expert e: D[e] = deq(a)[:, rows of e] @ deq(b)[:, rows of e]^T, the gradient of its weight; a e4m3 [n, P]
    (of the output's gradient) and b e4m3 [k, P] (of the input) with sfa [P/128, n], sfb [P/128, k], as
    fp8_quantize(transpose=True) gives them under the same row_offsets.  D [E, n, k] bf16 or fp32; accumulate adds
    to an fp32 d."""
    dev = _codes(a, 2, b, 2)
    if not _is(row_offsets, torch.int64, 1, dev):
        _need(row_offsets, torch.int64, "row_offsets", 1)
        raise ValueError("row_offsets must be contiguous")
    n, p = a.shape
    k, pb = b.shape
    if pb != p:
        raise ValueError("a and b disagree on the rows")
    experts = row_offsets.numel() - 1
    _dense(sfa, torch.float32, "sfa", (p // 128, n), dev)
    _dense(sfb, torch.float32, "sfb", (p // 128, k), dev)
    d, dt = _product_out(d, out_dtype, accumulate, (experts, n, k), a.device, stream)
    _check(_lib.fp8_grouped_weight_grad(a.data_ptr(), sfa.data_ptr(), b.data_ptr(), sfb.data_ptr(), row_offsets.data_ptr(),
                                        experts, d.data_ptr(), dt, 1 if accumulate else 0, p, n, k, flags, _stream(stream)))
    return d


# ---------------------------------------------------------------- gradients of the MoE steps
def moe_combine_backward(dout, y, pos, weights, dy=None, dweights=None, flags: int = 0, stream=None):
    """Gradients of moe_combine: (dy bf16 [rows, h], dweights fp32 [T, topk]) with dy[pos[t, j]] = weights[t, j] *
    dout[t] and dweights[t, j] = dout[t] . y[pos[t, j]].  Rows of dy that no slot names stay as they were (in a
    new dy: whatever its memory held); no row may be named twice (moe_sort_by_expert's pos names none twice)."""
    cur = _current_device()
    if not (_is(y, torch.bfloat16, 2, cur) and _is(pos, torch.int32, 2, cur) and _is(weights, torch.float32, 2, cur)):
        _need(y, torch.bfloat16, "y", 2)
        _need(pos, torch.int32, "pos", 2)
        _need(weights, torch.float32, "weights", 2)
        if not y.is_contiguous():
            raise ValueError("y must be contiguous")
        pos, weights = _contig(pos, stream), _contig(weights, stream)
    rows, h = y.shape
    T, topk = pos.shape
    dev = y.device
    ldo = _rows(dout, torch.bfloat16, "dout", T, h, cur)
    if weights.shape != (T, topk):
        raise ValueError(f"weights must have shape {(T, topk)}, got {tuple(weights.shape)}")
    dy = _made(dy, torch.bfloat16, "dy", (rows, h), dev, stream)
    dweights = _made(dweights, torch.float32, "dweights", (T, topk), dev, stream)
    _check(_lib.moe_combine_backward(dout.data_ptr(), ldo, y.data_ptr(), rows, pos.data_ptr(), weights.data_ptr(), T, topk, h,
                                     dy.data_ptr(), dweights.data_ptr(), flags, _stream(stream)))
    return dy, dweights


def moe_gather_backward(dxs, pos, dx=None, flags: int = 0, stream=None):
    """Gradient of moe_gather_rows under moe_sort_by_expert's src_rows: dx[t] = bf16(sum_j dxs[pos[t, j]]) (fp32, slot
    order)."""
    cur = _current_device()
    if not (_is(dxs, torch.bfloat16, 2, cur) and _is(pos, torch.int32, 2, cur)):
        _need(dxs, torch.bfloat16, "dxs", 2)
        _need(pos, torch.int32, "pos", 2)
        if not dxs.is_contiguous():
            raise ValueError("dxs must be contiguous")
        pos = _contig(pos, stream)
    rows, h = dxs.shape
    T, topk = pos.shape
    dx = _made(dx, torch.bfloat16, "dx", (T, h), dxs.device, stream)
    _check(_lib.moe_gather_backward(dxs.data_ptr(), rows, pos.data_ptr(), T, topk, h, dx.data_ptr(), flags, _stream(stream)))
    return dx


def check_status(stream=None) -> None:
    """Raise NVFP4Error(TIMEOUT) if a kernel gave up a bounded wait since the last check."""
    _check(_lib.nvfp4_check_status(_stream(stream)))
