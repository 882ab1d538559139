"""Gated Hyena cascade operator on NVIDIA B200 (sm_100a).

Thin Python binding over the C ABI in include/hyena.h: every function below
only checks and marshals torch tensors (device memory and streams) into raw
pointers and sizes and calls the CUDA library; all arithmetic happens in the
library's kernels.  There is no CPU path.

    y = x3 * (h_c * (x1 * x2)) + Dskip * (x1 * x2)

with h_c either an explicit short FIR (hcs 7 taps / hcm 128 taps,
``short_conv``) or the long modal filter h_c[t] = sum_n R[c,n] exp(a[c,n] t)
(hcl, ``modal_long_conv``).  Layout [B, L, D] bf16, channel-contiguous; a row
stride ld >= D is allowed, so x1, x2, x3 may be views of one [B, L, 3D]
projection output.  The ``*_packed`` variants read the three inputs from one
[B, L, >= 3D] projection buffer whose rows hold channel groups of ``group``
channels as [x1 | x2 | x3] (group = 1: per-channel triples x1_c x2_c x3_c).
The ``*_complex`` variants take complex modes (poles and residues as [D, N, 2]
fp32 pairs; h_c[t] = Re sum_n R p^t), and the ``*_decode`` functions advance
the modal state or the FIR window by one generated token.

Around the mixers: ``gated_recurrence`` (a modal filter of one mode whose pole
depends on the token), ``rms_norm`` and ``rms_norm_fp8``, the 8-bit projections
``fp8_quantize`` and ``fp8_matmul``, and the gated feed-forward block
``gated_ffn`` (with ``gated_ffn_backward``) and ``gated_ffn_fp8``.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

from ._lib import HyenaError, check, lib  # noqa: F401

__all__ = [
    "FfnGrads",
    "FfnWorkspace",
    "HyenaError",
    "MatmulWorkspace",
    "ModalWorkspace",
    "NormGrads",
    "RecurrenceGrads",
    "RecurrenceWorkspace",
    "fp8_matmul",
    "fp8_quantize",
    "gated_ffn",
    "gated_ffn_backward",
    "gated_ffn_fp8",
    "gated_recurrence",
    "gated_recurrence_backward",
    "gated_recurrence_decode",
    "last_launch_count",
    "modal_decode",
    "modal_decode_complex",
    "modal_decode_complex_packed",
    "modal_decode_packed",
    "modal_long_conv",
    "modal_long_conv_complex",
    "modal_long_conv_complex_packed",
    "HostWorkspace",
    "modal_long_conv_host",
    "modal_prepare",
    "modal_long_conv_prepared",
    "short_conv_host",
    "modal_long_conv_packed",
    "modal_state_init",
    "recurrence_unit_states",
    "rms_norm",
    "rms_norm_backward",
    "rms_norm_fp8",
    "short_conv",
    "short_conv_packed",
    "short_conv_dft",
    "short_decode",
    "short_decode_packed",
    "workspace_check",
    "workspace_size",
]

MAX_MODES = 64
MAX_COMPLEX_MODES = 32
MAX_TAPS = 128
RECURRENCE_UNIT = 64
MAX_NORM_WIDTH = 16384
PRODUCT_HEADER = 4096  # bytes of a product's workspace that have to be zero at first
ACTIVATIONS = {"silu": 1, "gelu": 2, "gelu_tanh": 3, "identity": 4}


_torch_module = None  # imported by the first call; a statement in each costs it 0.1 us every time
_BF16 = _F32 = _E4M3 = None  # its types, likewise


def _torch():
    global _torch_module, _BF16, _F32, _E4M3
    if _torch_module is None:
        import torch
        _BF16, _F32, _E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
        _torch_module = torch
    return _torch_module


def _stream(stream):
    torch = _torch()
    if stream is None:
        # the current stream of the current device; torch's raw query skips
        # building a Stream object (3.5 us of a ~19 us decode call)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t):
    # a plain integer: ctypes converts it through the entry point's c_void_p
    # argument type (None is NULL)
    return None if t is None else t.data_ptr()


def _bld(x, name):
    """[B, L, D] bf16 view with unit channel stride -> (B, L, D, ld)."""
    torch = _torch()
    if x.dtype != torch.bfloat16 or x.dim() != 3 or not x.is_cuda:
        raise ValueError(f"{name} must be a 3-D bf16 CUDA tensor [B, L, D]")
    B, L, D = x.shape
    if x.stride(2) != 1:
        raise ValueError(f"{name} must be channel-contiguous")
    ld = x.stride(1) if L > 1 else (x.stride(0) // max(L, 1) if B > 1 else D)
    if B > 1 and L > 0 and x.stride(0) != L * ld:
        raise ValueError(f"{name}: batch stride must equal L * row stride")
    return B, L, D, ld


def _same_ld(*xs):
    lds = {x[3] for x in xs}
    if len(lds) != 1:
        raise ValueError("x1, x2, x3 must share one row stride")


def _f32(t, shape, name, allow_none=True):
    if t is None:
        if allow_none:
            return None
        raise ValueError(f"{name} is required")
    torch = _torch()
    if t.dtype is not torch.float32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp32 tensor of shape {tuple(shape)}")
    return t


def _current(stream):
    """Makes a given stream (a torch Stream or a raw handle) the current one, so
    that what the call allocates belongs to it as well."""
    torch = _torch()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _zeroed(n, device, stream, clear=None):
    """n bytes of device memory, the first `clear` (None: all) zero, taken and
    cleared on one stream (the given one, else the device's current one): taken on
    another, they may be a block that work still pending there writes to after the
    clearing."""
    torch = _torch()
    if getattr(device, "type", None) == "cuda" and device.index == torch.cuda.current_device():
        device = None  # the usual case, of a tensor's device
    if device is not None or stream is not None:
        if device is None and isinstance(stream, torch.cuda.Stream):
            device = stream.device
        with torch.cuda.device(device):
            here = torch.cuda.current_device()
            with torch.cuda.stream(None) if stream is None else _current(stream):
                if torch.cuda.current_device() != here:
                    raise ValueError("the stream belongs to another device")
                return _zeroed(n, None, None, clear)
    buf = torch.empty(n, dtype=torch.uint8, device="cuda")
    check("hyena_modal_workspace_init",
          lib().hyena_modal_workspace_init(_ptr(buf), n if clear is None else clear, _stream(None)))
    return buf


def last_launch_count() -> int:
    """Kernels/memsets enqueued by the most recent call on this thread."""
    return int(lib().hyena_last_launch_count())


def workspace_size(B: int, D: int, N: int) -> int:
    return int(lib().hyena_modal_long_conv_workspace_size(B, D, N))


class ModalWorkspace:
    """Device workspace for modal_long_conv, zero-filled once at creation."""

    def __init__(self, B: int, D: int, N: int, device=None, stream=None):
        n = workspace_size(B, D, N)
        if n == 0:
            raise ValueError("invalid workspace shape")
        self.nbytes = n
        self.buf = _zeroed(n, device, stream)

    def fits(self, B: int, D: int, N: int) -> bool:
        return workspace_size(B, D, N) <= self.nbytes


def workspace_check(ws: ModalWorkspace, stream=None) -> None:
    """Synchronise and raise if a bounded device wait of an earlier call ran out."""
    check("hyena_workspace_check", lib().hyena_workspace_check(_ptr(ws.buf), _stream(stream)))


def modal_state_init(state, stream=None):
    """Zero a [B, D, N] fp32 modal state (start of chunked prefill)."""
    B, D, N = state.shape
    _f32(state, (B, D, N), "state", allow_none=False)
    check("hyena_modal_state_init", lib().hyena_modal_state_init(_ptr(state), B, D, N, _stream(stream)))
    return state


def modal_long_conv(x1, x2, x3, log_poles, residues, Dskip=None, y=None, state_in=None,
                    state_out=None, workspace: ModalWorkspace | None = None, stream=None):
    """Long modal-form Hyena filter (hcl) with fused gates.

    x1, x2, x3: [B, L, D] bf16 (views sharing a row stride); log_poles,
    residues: [D, N] fp32; Dskip: [D] fp32 or None; state_in/state_out:
    [B, D, N] fp32 or None (may be the same tensor).  Returns y ([B, L, D]
    bf16, allocated if not given).
    """
    torch = _torch()
    s1, s2, s3 = _bld(x1, "x1"), _bld(x2, "x2"), _bld(x3, "x3")
    _same_ld(s1, s2, s3)
    B, L, D, ld = s1
    if s2[:3] != (B, L, D) or s3[:3] != (B, L, D):
        raise ValueError("x1, x2, x3 shapes differ")
    Dn, N = log_poles.shape
    if Dn != D:
        raise ValueError("log_poles must be [D, N]")
    _f32(log_poles, (D, N), "log_poles", False)
    _f32(residues, (D, N), "residues", False)
    _f32(Dskip, (D,), "Dskip")
    _f32(state_in, (B, D, N), "state_in")
    _f32(state_out, (B, D, N), "state_out")
    if y is None:
        y = torch.empty((B, L, D), dtype=torch.bfloat16, device=x1.device)
    yB, yL, yD, ld_y = _bld(y, "y")
    if (yB, yL, yD) != (B, L, D):
        raise ValueError("y shape differs from x")
    if workspace is None:
        workspace = ModalWorkspace(B, D, N, device=x1.device, stream=stream)
    rc = lib().hyena_modal_long_conv(_ptr(x1), _ptr(x2), _ptr(x3), ld, _ptr(log_poles), _ptr(residues),
                                     _ptr(Dskip), _ptr(y), ld_y, _ptr(state_in), _ptr(state_out),
                                     B, L, D, N, _ptr(workspace.buf), workspace.nbytes, _stream(stream))
    check("hyena_modal_long_conv", rc)
    return y


def modal_prepare(log_poles, residues, Dskip, workspace: ModalWorkspace, B: int = 1, stream=None):
    """Form the coefficient table of a real-mode filter in ``workspace`` once,
    for the chunks of one sequence that follow (modal_long_conv_prepared)."""
    D, N = log_poles.shape
    _f32(log_poles, (D, N), "log_poles", False)
    _f32(residues, (D, N), "residues", False)
    _f32(Dskip, (D,), "Dskip")
    rc = lib().hyena_modal_prepare(_ptr(log_poles), _ptr(residues), _ptr(Dskip), B, D, N, _ptr(workspace.buf),
                                   workspace.nbytes, _stream(stream))
    check("hyena_modal_prepare", rc)


def modal_long_conv_prepared(x1, x2, x3, N: int, workspace: ModalWorkspace, y=None, state_in=None, state_out=None,
                             stream=None):
    """modal_long_conv with the table of the last modal_prepare on ``workspace``
    (the same bits as modal_long_conv with those parameters)."""
    torch = _torch()
    s1, s2, s3 = _bld(x1, "x1"), _bld(x2, "x2"), _bld(x3, "x3")
    _same_ld(s1, s2, s3)
    B, L, D, ld = s1
    if s2[:3] != (B, L, D) or s3[:3] != (B, L, D):
        raise ValueError("x1, x2, x3 shapes differ")
    _f32(state_in, (B, D, N), "state_in")
    _f32(state_out, (B, D, N), "state_out")
    if y is None:
        y = torch.empty((B, L, D), dtype=torch.bfloat16, device=x1.device)
    yB, yL, yD, ld_y = _bld(y, "y")
    if (yB, yL, yD) != (B, L, D):
        raise ValueError("y shape differs from x")
    rc = lib().hyena_modal_long_conv_prepared(_ptr(x1), _ptr(x2), _ptr(x3), ld, _ptr(y), ld_y, _ptr(state_in),
                                              _ptr(state_out), B, L, D, N, _ptr(workspace.buf), workspace.nbytes,
                                              _stream(stream))
    check("hyena_modal_long_conv_prepared", rc)
    return y


def _host_bld(x, name):
    """[B, L, D] bf16 (or int16 bits) host tensor with unit channel stride ->
    (B, L, D, ld)."""
    torch = _torch()
    if x.dtype not in (torch.bfloat16, torch.int16) or x.dim() != 3 or x.is_cuda:
        raise ValueError(f"{name} must be a 3-D bf16 host tensor [B, L, D]")
    B, L, D = x.shape
    if x.stride(2) != 1:
        raise ValueError(f"{name} must be channel-contiguous")
    ld = x.stride(1) if L > 1 else (x.stride(0) // max(L, 1) if B > 1 else D)
    if B > 1 and L > 0 and x.stride(0) != L * ld:
        raise ValueError(f"{name}: batch stride must equal L * row stride")
    return B, L, D, ld


class HostWorkspace:
    """Device workspace of modal_long_conv_host (the scan's workspace, two
    staging slots of `chunk` tokens and the carried state), zero-filled once."""

    def __init__(self, B: int, D: int, N: int, chunk: int = 2048, device=None, stream=None):
        n = int(lib().hyena_modal_host_workspace_size(B, D, N, chunk))
        if n == 0:
            raise ValueError("invalid host-workspace shape (chunk must be a positive multiple of 128)")
        self.nbytes, self.chunk = n, chunk
        self.buf = _zeroed(n, device, stream)


def modal_long_conv_host(x1, x2, x3, log_poles, residues, Dskip=None, y=None, state_in=None,
                         state_out=None, workspace: HostWorkspace | None = None, stream=None):
    """modal_long_conv with x1, x2, x3 and y in host memory ([B, L, D] bf16
    host tensors, pinned for overlapped copies): the sequence is streamed
    through the device in chunks of ``workspace.chunk`` tokens with the copies
    in both directions overlapping the scan.  Parameters and state are device
    tensors.  Returns y (a host tensor, allocated pinned if not given); it is
    valid once ``stream`` has been synchronised."""
    torch = _torch()
    s1, s2, s3 = _host_bld(x1, "x1"), _host_bld(x2, "x2"), _host_bld(x3, "x3")
    _same_ld(s1, s2, s3)
    B, L, D, ld = s1
    if s2[:3] != (B, L, D) or s3[:3] != (B, L, D):
        raise ValueError("x1, x2, x3 shapes differ")
    Dn, N = log_poles.shape
    if Dn != D:
        raise ValueError("log_poles must be [D, N]")
    _f32(log_poles, (D, N), "log_poles", False)
    _f32(residues, (D, N), "residues", False)
    _f32(Dskip, (D,), "Dskip")
    _f32(state_in, (B, D, N), "state_in")
    _f32(state_out, (B, D, N), "state_out")
    if y is None:
        y = torch.empty((B, L, D), dtype=torch.bfloat16).pin_memory()
    yB, yL, yD, ld_y = _host_bld(y, "y")
    if (yB, yL, yD) != (B, L, D):
        raise ValueError("y shape differs from x")
    if workspace is None:
        workspace = HostWorkspace(B, D, N, device=log_poles.device, stream=stream)
    rc = lib().hyena_modal_long_conv_host(_ptr(x1), _ptr(x2), _ptr(x3), ld, _ptr(log_poles), _ptr(residues),
                                          _ptr(Dskip), _ptr(y), ld_y, _ptr(state_in), _ptr(state_out),
                                          B, L, D, N, workspace.chunk, _ptr(workspace.buf), workspace.nbytes,
                                          _stream(stream))
    check("hyena_modal_long_conv_host", rc)
    return y


def short_conv_host(x1, x2, x3, taps, Dskip=None, y=None, hist_in=None, hist_out=None, chunk=2048,
                    workspace=None, stream=None):
    """short_conv with x1, x2, x3 and y in host memory ([B, L, D] bf16 host
    tensors, pinned for overlapped copies), streamed through the device in
    chunks with the FIR window carried.  taps [D, K] bf16, Dskip, hist_in and
    hist_out ([B, K-1, D] fp32) are device tensors; ``workspace`` is a device
    uint8 tensor of at least short_host_workspace_size bytes (allocated if
    not given).  Returns y, valid once ``stream`` has been synchronised."""
    torch = _torch()
    s1, s2, s3 = _host_bld(x1, "x1"), _host_bld(x2, "x2"), _host_bld(x3, "x3")
    _same_ld(s1, s2, s3)
    B, L, D, ld = s1
    if s2[:3] != (B, L, D) or s3[:3] != (B, L, D):
        raise ValueError("x1, x2, x3 shapes differ")
    if taps.dtype != torch.bfloat16 or taps.dim() != 2 or taps.shape[0] != D or not taps.is_contiguous():
        raise ValueError("taps must be a contiguous [D, K] bf16 tensor")
    K = taps.shape[1]
    _f32(Dskip, (D,), "Dskip")
    _f32(hist_in, (B, K - 1, D), "hist_in")
    _f32(hist_out, (B, K - 1, D), "hist_out")
    if y is None:
        y = torch.empty((B, L, D), dtype=torch.bfloat16).pin_memory()
    yB, yL, yD, ld_y = _host_bld(y, "y")
    if (yB, yL, yD) != (B, L, D):
        raise ValueError("y shape differs from x")
    need = int(lib().hyena_short_host_workspace_size(B, D, K, chunk))
    if need == 0:
        raise ValueError("invalid host-workspace shape")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=taps.device)
    rc = lib().hyena_short_conv_host(_ptr(x1), _ptr(x2), _ptr(x3), ld, _ptr(taps), _ptr(Dskip), _ptr(y), ld_y,
                                     _ptr(hist_in), _ptr(hist_out), B, L, D, K, chunk, _ptr(workspace),
                                     workspace.numel(), _stream(stream))
    check("hyena_short_conv_host", rc)
    return y


def _bd(x, name):
    """One token per batch row: [B, D] or [B, 1, D] bf16 with unit channel
    stride -> (B, D, ld), element (b, c) at b * ld + c."""
    torch = _torch()
    sh = x.shape  # one query each of shape and strides: this runs once per tensor per token
    if x.dtype is not torch.bfloat16 or not x.is_cuda or len(sh) not in (2, 3) or (len(sh) == 3 and sh[1] != 1):
        raise ValueError(f"{name} must be a bf16 CUDA tensor [B, D] or [B, 1, D]")
    st = x.stride()
    if st[-1] != 1:
        raise ValueError(f"{name} must have unit channel stride")
    return sh[0], sh[-1], st[0]


def modal_decode(x1, x2, x3, log_poles, residues, Dskip, state, y=None, stream=None):
    """One generated token through the long modal filter: advances ``state``
    ([B, D, N] fp32, in place) and returns y ([B, D] or [B, 1, D] like x1).
    Equals ``modal_long_conv`` on a one-token sequence with state_in =
    state_out = state, bit for bit."""
    torch = _torch()
    (B, D, ld), b2, b3 = _bd(x1, "x1"), _bd(x2, "x2"), _bd(x3, "x3")
    if b2 != (B, D, ld) or b3 != (B, D, ld):
        raise ValueError("x1, x2, x3 must share shape and row stride")
    Dn, N = log_poles.shape
    if Dn != D:
        raise ValueError("log_poles must be [D, N]")
    _f32(log_poles, (D, N), "log_poles", False)
    _f32(residues, (D, N), "residues", False)
    _f32(Dskip, (D,), "Dskip")
    _f32(state, (B, D, N), "state", False)
    if y is None:
        y = torch.empty_like(x1, memory_format=torch.contiguous_format)
    yB, yD, ld_y = _bd(y, "y")
    if (yB, yD) != (B, D):
        raise ValueError("y shape differs from x")
    rc = lib().hyena_modal_decode(_ptr(x1), _ptr(x2), _ptr(x3), ld, _ptr(log_poles), _ptr(residues), _ptr(Dskip),
                                  _ptr(y), ld_y, _ptr(state), B, D, N, _stream(stream))
    check("hyena_modal_decode", rc)
    return y


def short_decode(x1, x2, x3, taps, Dskip, hist, y=None, stream=None):
    """One generated token through an explicit FIR: advances the window
    ``hist`` ([B, K-1, D] fp32, in place; None when K = 1) and returns y.
    Equals ``short_conv`` on a one-token sequence with hist_in = hist_out =
    hist, bit for bit."""
    torch = _torch()
    (B, D, ld), b2, b3 = _bd(x1, "x1"), _bd(x2, "x2"), _bd(x3, "x3")
    if b2 != (B, D, ld) or b3 != (B, D, ld):
        raise ValueError("x1, x2, x3 must share shape and row stride")
    if taps.dtype != torch.bfloat16 or taps.dim() != 2 or taps.shape[0] != D or not taps.is_contiguous():
        raise ValueError("taps must be a contiguous bf16 [D, K] tensor")
    K = taps.shape[1]
    _f32(Dskip, (D,), "Dskip")
    if K > 1:
        _f32(hist, (B, K - 1, D), "hist", False)
    if y is None:
        y = torch.empty_like(x1, memory_format=torch.contiguous_format)
    yB, yD, ld_y = _bd(y, "y")
    if (yB, yD) != (B, D):
        raise ValueError("y shape differs from x")
    rc = lib().hyena_short_decode(_ptr(x1), _ptr(x2), _ptr(x3), ld, _ptr(taps), _ptr(Dskip), _ptr(y), ld_y,
                                  _ptr(hist) if K > 1 else None, B, D, K, _stream(stream))
    check("hyena_short_decode", rc)
    return y


def short_conv(x1, x2, x3, taps, Dskip=None, y=None, hist_in=None, hist_out=None, stream=None):
    """Explicit short Hyena FIR (hcs/hcm) with fused gates.

    taps: [D, K] bf16 in lag order (taps[c, k] multiplies v[t-k]);
    hist_in/hist_out: [B, K-1, D] fp32 or None (may be the same tensor).
    """
    return _short_conv("hyena_short_conv", x1, x2, x3, taps, Dskip, y, hist_in, hist_out, stream)


def short_conv_dft(x1, x2, x3, taps, Dskip=None, y=None, hist_in=None, hist_out=None, stream=None):
    """short_conv computed on the tensor cores as overlap-save DFT-as-GEMM
    (hyena_short_conv_dft): the same arguments; results agree with short_conv
    to tf32 rounding.  The first call on a device copies the DFT tables with a
    synchronous copy (make it before any CUDA graph capture).
    """
    return _short_conv("hyena_short_conv_dft", x1, x2, x3, taps, Dskip, y, hist_in, hist_out, stream)


def _short_conv(entry, x1, x2, x3, taps, Dskip, y, hist_in, hist_out, stream):
    torch = _torch()
    s1, s2, s3 = _bld(x1, "x1"), _bld(x2, "x2"), _bld(x3, "x3")
    _same_ld(s1, s2, s3)
    B, L, D, ld = s1
    if s2[:3] != (B, L, D) or s3[:3] != (B, L, D):
        raise ValueError("x1, x2, x3 shapes differ")
    if taps.dtype != torch.bfloat16 or taps.dim() != 2 or taps.shape[0] != D or not taps.is_contiguous():
        raise ValueError("taps must be a contiguous bf16 [D, K] tensor")
    K = taps.shape[1]
    _f32(Dskip, (D,), "Dskip")
    _f32(hist_in, (B, K - 1, D), "hist_in")
    _f32(hist_out, (B, K - 1, D), "hist_out")
    if y is None:
        y = torch.empty((B, L, D), dtype=torch.bfloat16, device=x1.device)
    yB, yL, yD, ld_y = _bld(y, "y")
    if (yB, yL, yD) != (B, L, D):
        raise ValueError("y shape differs from x")
    rc = getattr(lib(), entry)(_ptr(x1), _ptr(x2), _ptr(x3), ld, _ptr(taps), _ptr(Dskip), _ptr(y), ld_y,
                               _ptr(hist_in), _ptr(hist_out), B, L, D, K, _stream(stream))
    check(entry, rc)
    return y


# ---------------------------------------------------------------- packed inputs

def _packed(xp, D, decode=False):
    """Projection buffer [B, L, W] (decode: [B, W] or [B, 1, W]) with W >= 3D
    and unit element stride -> (B, L, ld)."""
    if decode:
        B, W, ld = _bd(xp, "xp")
        L = 1
    else:
        B, L, W, ld = _bld(xp, "xp")
    if W < 3 * D:
        raise ValueError(f"xp rows hold {W} values, fewer than 3 D = {3 * D}")
    return B, L, ld


def modal_long_conv_packed(xp, group, log_poles, residues, Dskip=None, y=None, state_in=None,
                           state_out=None, workspace: ModalWorkspace | None = None, stream=None):
    """``modal_long_conv`` with x1, x2, x3 read from one projection buffer xp
    ([B, L, W >= 3D] bf16) in channel groups of ``group`` (x_k of channel c at
    column 3 group (c // group) + (k-1) group + c % group).  D is taken from
    log_poles ([D, N])."""
    torch = _torch()
    D, N = log_poles.shape
    B, L, ld = _packed(xp, D)
    _f32(log_poles, (D, N), "log_poles", False)
    _f32(residues, (D, N), "residues", False)
    _f32(Dskip, (D,), "Dskip")
    _f32(state_in, (B, D, N), "state_in")
    _f32(state_out, (B, D, N), "state_out")
    if y is None:
        y = torch.empty((B, L, D), dtype=torch.bfloat16, device=xp.device)
    yB, yL, yD, ld_y = _bld(y, "y")
    if (yB, yL, yD) != (B, L, D):
        raise ValueError("y must be [B, L, D]")
    if workspace is None:
        workspace = ModalWorkspace(B, D, N, device=xp.device, stream=stream)
    rc = lib().hyena_modal_long_conv_packed(_ptr(xp), ld, int(group), _ptr(log_poles), _ptr(residues),
                                            _ptr(Dskip), _ptr(y), ld_y, _ptr(state_in), _ptr(state_out),
                                            B, L, D, N, _ptr(workspace.buf), workspace.nbytes, _stream(stream))
    check("hyena_modal_long_conv_packed", rc)
    return y


def short_conv_packed(xp, group, taps, Dskip=None, y=None, hist_in=None, hist_out=None, stream=None):
    """``short_conv`` with x1, x2, x3 read from one projection buffer xp in
    channel groups of ``group`` (see ``modal_long_conv_packed``).  D is taken
    from taps ([D, K])."""
    torch = _torch()
    if taps.dtype != torch.bfloat16 or taps.dim() != 2 or not taps.is_contiguous():
        raise ValueError("taps must be a contiguous bf16 [D, K] tensor")
    D, K = taps.shape
    B, L, ld = _packed(xp, D)
    _f32(Dskip, (D,), "Dskip")
    _f32(hist_in, (B, K - 1, D), "hist_in")
    _f32(hist_out, (B, K - 1, D), "hist_out")
    if y is None:
        y = torch.empty((B, L, D), dtype=torch.bfloat16, device=xp.device)
    yB, yL, yD, ld_y = _bld(y, "y")
    if (yB, yL, yD) != (B, L, D):
        raise ValueError("y must be [B, L, D]")
    rc = lib().hyena_short_conv_packed(_ptr(xp), ld, int(group), _ptr(taps), _ptr(Dskip), _ptr(y), ld_y,
                                       _ptr(hist_in), _ptr(hist_out), B, L, D, K, _stream(stream))
    check("hyena_short_conv_packed", rc)
    return y


def modal_decode_packed(xp, group, log_poles, residues, Dskip, state, y=None, stream=None):
    """``modal_decode`` with the token's x1, x2, x3 read from one projection
    row per batch row (xp [B, W] or [B, 1, W], W >= 3D) in channel groups of
    ``group``."""
    torch = _torch()
    D, N = log_poles.shape
    B, _, ld = _packed(xp, D, decode=True)
    _f32(log_poles, (D, N), "log_poles", False)
    _f32(residues, (D, N), "residues", False)
    _f32(Dskip, (D,), "Dskip")
    _f32(state, (B, D, N), "state", False)
    if y is None:
        y = torch.empty((B, D), dtype=torch.bfloat16, device=xp.device)
    yB, yD, ld_y = _bd(y, "y")
    if (yB, yD) != (B, D):
        raise ValueError("y must be [B, D] or [B, 1, D]")
    rc = lib().hyena_modal_decode_packed(_ptr(xp), ld, int(group), _ptr(log_poles), _ptr(residues), _ptr(Dskip),
                                         _ptr(y), ld_y, _ptr(state), B, D, N, _stream(stream))
    check("hyena_modal_decode_packed", rc)
    return y


def short_decode_packed(xp, group, taps, Dskip, hist, y=None, stream=None):
    """``short_decode`` with the token's x1, x2, x3 read from one projection
    row per batch row in channel groups of ``group``."""
    torch = _torch()
    if taps.dtype != torch.bfloat16 or taps.dim() != 2 or not taps.is_contiguous():
        raise ValueError("taps must be a contiguous bf16 [D, K] tensor")
    D, K = taps.shape
    B, _, ld = _packed(xp, D, decode=True)
    _f32(Dskip, (D,), "Dskip")
    if K > 1:
        _f32(hist, (B, K - 1, D), "hist", False)
    if y is None:
        y = torch.empty((B, D), dtype=torch.bfloat16, device=xp.device)
    yB, yD, ld_y = _bd(y, "y")
    if (yB, yD) != (B, D):
        raise ValueError("y must be [B, D] or [B, 1, D]")
    rc = lib().hyena_short_decode_packed(_ptr(xp), ld, int(group), _ptr(taps), _ptr(Dskip), _ptr(y), ld_y,
                                         _ptr(hist) if K > 1 else None, B, D, K, _stream(stream))
    check("hyena_short_decode_packed", rc)
    return y


# ---------------------------------------------------------------- complex modes

def _cpar(poles, residues):
    """poles, residues fp32 [D, N, 2] (real, imaginary) -> (D, N)."""
    if poles.dim() != 3 or poles.shape[2] != 2:
        raise ValueError("poles must be a [D, N, 2] fp32 tensor")
    D, N, _ = poles.shape
    _f32(poles, (D, N, 2), "poles", False)
    _f32(residues, (D, N, 2), "residues", False)
    return D, N


def modal_long_conv_complex(x1, x2, x3, poles, residues, Dskip=None, y=None, state_in=None,
                            state_out=None, workspace: ModalWorkspace | None = None, stream=None):
    """Long modal filter with complex modes, h[t] = Re sum_n R_n p_n^t, with
    fused gates.  poles, residues: [D, N, 2] fp32 (real, imaginary);
    state_in/state_out: [B, D, N, 2] fp32 or None.  The workspace is that of
    2N real modes."""
    torch = _torch()
    s1, s2, s3 = _bld(x1, "x1"), _bld(x2, "x2"), _bld(x3, "x3")
    _same_ld(s1, s2, s3)
    B, L, D, ld = s1
    if s2[:3] != (B, L, D) or s3[:3] != (B, L, D):
        raise ValueError("x1, x2, x3 shapes differ")
    Dp, N = _cpar(poles, residues)
    if Dp != D:
        raise ValueError("poles must be [D, N, 2]")
    _f32(Dskip, (D,), "Dskip")
    _f32(state_in, (B, D, N, 2), "state_in")
    _f32(state_out, (B, D, N, 2), "state_out")
    if y is None:
        y = torch.empty((B, L, D), dtype=torch.bfloat16, device=x1.device)
    yB, yL, yD, ld_y = _bld(y, "y")
    if (yB, yL, yD) != (B, L, D):
        raise ValueError("y shape differs from x")
    if workspace is None:
        workspace = ModalWorkspace(B, D, 2 * N, device=x1.device, stream=stream)
    rc = lib().hyena_modal_long_conv_complex(_ptr(x1), _ptr(x2), _ptr(x3), ld, _ptr(poles), _ptr(residues),
                                             _ptr(Dskip), _ptr(y), ld_y, _ptr(state_in), _ptr(state_out),
                                             B, L, D, N, _ptr(workspace.buf), workspace.nbytes, _stream(stream))
    check("hyena_modal_long_conv_complex", rc)
    return y


def modal_decode_complex(x1, x2, x3, poles, residues, Dskip, state, y=None, stream=None):
    """One generated token through the complex-mode filter: advances
    ``state`` ([B, D, N, 2] fp32, in place); equals ``modal_long_conv_complex``
    on a one-token sequence bit for bit."""
    torch = _torch()
    (B, D, ld), b2, b3 = _bd(x1, "x1"), _bd(x2, "x2"), _bd(x3, "x3")
    if b2 != (B, D, ld) or b3 != (B, D, ld):
        raise ValueError("x1, x2, x3 must share shape and row stride")
    Dp, N = _cpar(poles, residues)
    if Dp != D:
        raise ValueError("poles must be [D, N, 2]")
    _f32(Dskip, (D,), "Dskip")
    _f32(state, (B, D, N, 2), "state", False)
    if y is None:
        y = torch.empty_like(x1, memory_format=torch.contiguous_format)
    yB, yD, ld_y = _bd(y, "y")
    if (yB, yD) != (B, D):
        raise ValueError("y shape differs from x")
    rc = lib().hyena_modal_decode_complex(_ptr(x1), _ptr(x2), _ptr(x3), ld, _ptr(poles), _ptr(residues),
                                          _ptr(Dskip), _ptr(y), ld_y, _ptr(state), B, D, N, _stream(stream))
    check("hyena_modal_decode_complex", rc)
    return y


def modal_long_conv_complex_packed(xp, group, poles, residues, Dskip=None, y=None, state_in=None,
                                   state_out=None, workspace: ModalWorkspace | None = None, stream=None):
    """``modal_long_conv_complex`` with x1, x2, x3 read from one projection
    buffer xp in channel groups of ``group`` (see ``modal_long_conv_packed``)."""
    torch = _torch()
    D, N = _cpar(poles, residues)
    B, L, ld = _packed(xp, D)
    _f32(Dskip, (D,), "Dskip")
    _f32(state_in, (B, D, N, 2), "state_in")
    _f32(state_out, (B, D, N, 2), "state_out")
    if y is None:
        y = torch.empty((B, L, D), dtype=torch.bfloat16, device=xp.device)
    yB, yL, yD, ld_y = _bld(y, "y")
    if (yB, yL, yD) != (B, L, D):
        raise ValueError("y must be [B, L, D]")
    if workspace is None:
        workspace = ModalWorkspace(B, D, 2 * N, device=xp.device, stream=stream)
    rc = lib().hyena_modal_long_conv_complex_packed(_ptr(xp), ld, int(group), _ptr(poles), _ptr(residues),
                                                    _ptr(Dskip), _ptr(y), ld_y, _ptr(state_in), _ptr(state_out),
                                                    B, L, D, N, _ptr(workspace.buf), workspace.nbytes,
                                                    _stream(stream))
    check("hyena_modal_long_conv_complex_packed", rc)
    return y


def modal_decode_complex_packed(xp, group, poles, residues, Dskip, state, y=None, stream=None):
    """``modal_decode_complex`` with the token's x1, x2, x3 read from one
    projection row per batch row in channel groups of ``group``."""
    torch = _torch()
    D, N = _cpar(poles, residues)
    B, _, ld = _packed(xp, D, decode=True)
    _f32(Dskip, (D,), "Dskip")
    _f32(state, (B, D, N, 2), "state", False)
    if y is None:
        y = torch.empty((B, D), dtype=torch.bfloat16, device=xp.device)
    yB, yD, ld_y = _bd(y, "y")
    if (yB, yD) != (B, D):
        raise ValueError("y must be [B, D] or [B, 1, D]")
    rc = lib().hyena_modal_decode_complex_packed(_ptr(xp), ld, int(group), _ptr(poles), _ptr(residues),
                                                 _ptr(Dskip), _ptr(y), ld_y, _ptr(state), B, D, N, _stream(stream))
    check("hyena_modal_decode_complex_packed", rc)
    return y


# ------------------------------------------------------------ gated recurrence

def _here(x, *others):
    """The current stream's handle, once x and the given tensors (None: absent)
    are known to be on the current device: the call launches there."""
    C = _torch()._C
    dev = x.get_device()
    if dev < 0 or dev != C._cuda_getDevice():
        raise ValueError("tensors must be on the current CUDA device")
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError("all tensors must be on one CUDA device")
    return C._cuda_getCurrentRawStream(dev)


def _like(x, shape, st, ld, name):
    """Row stride of a bf16 [B, L, D] tensor of the given shape, as _bld (the
    device is checked by _here); the usual case, the stride of a tensor whose
    row stride ld is known, is settled by comparing."""
    if x.dtype is not _torch().bfloat16 or x.shape != shape:
        raise ValueError(f"{name} must be a bf16 CUDA tensor of shape {tuple(shape)}")
    xst = x.stride()
    if xst == st:
        return ld
    if xst[2] != 1:
        raise ValueError(f"{name} must be channel-contiguous")
    B, L, D = shape
    if L > 1:
        if B > 1 and xst[0] != L * xst[1]:
            raise ValueError(f"{name}: batch stride must equal L * row stride")
        return xst[1]
    return xst[0] if B > 1 and L == 1 else D


def _opt(t):
    return None if t is None else t.data_ptr()


def _reset(t, B, L):
    torch = _torch()
    if t is not None and (t.dtype not in (torch.bool, torch.uint8) or tuple(t.shape) != (B, L)
                          or not t.is_contiguous()):
        raise ValueError(f"reset must be a contiguous bool or uint8 tensor of shape {(B, L)}")
    return t


class RecurrenceWorkspace:
    """Device workspace of gated_recurrence and its backward for sequences up
    to L tokens, zero-filled once at creation."""

    def __init__(self, B: int, L: int, D: int, device=None, stream=None):
        n = int(lib().hyena_gated_recurrence_workspace_size(B, L, D))
        if n == 0:
            raise ValueError("invalid workspace shape")
        self.nbytes = n
        self.buf = _zeroed(n, device, stream)


def recurrence_unit_states(B: int, L: int, D: int, device=None):
    """An uninitialised buffer for gated_recurrence's ``unit_states``: the
    state before each unit of RECURRENCE_UNIT tokens."""
    torch = _torch()
    return torch.empty((B, -(-L // RECURRENCE_UNIT), D), dtype=torch.float32, device=device or "cuda")


def gated_recurrence(x1, x2, x3, gate, log_rate, Dskip=None, reset=None, normalize=True, y=None, state_in=None,
                     state_out=None, unit_states=None, workspace: RecurrenceWorkspace | None = None, stream=None):
    """Gated linear recurrence: s_t = a_t s_{t-1} + w_t v_t with v = x1 x2 and
    a_t = exp(log_rate sigmoid(gate_t)) (0 where reset_t), y = x3 s + Dskip v;
    w = sqrt(1 - a^2) with ``normalize``, else 1.

    x1, x2, x3 ([B, L, D] bf16, one row stride), gate ([B, L, D] bf16);
    log_rate, Dskip: [D] fp32; reset: [B, L] bool or uint8 or None;
    state_in/state_out: [B, D] fp32 or None (may be the same tensor);
    unit_states: from recurrence_unit_states, filled for the backward call.
    Returns y ([B, L, D] bf16, allocated if not given).

    A device wait that ran out leaves NaN and is reported by workspace_check;
    a call without a ``workspace`` uses one of its own, so that the NaN are all
    that shows it.
    """
    if stream is not None:
        with _current(stream):
            return gated_recurrence(x1, x2, x3, gate, log_rate, Dskip, reset, normalize, y, state_in, state_out,
                                    unit_states, workspace)
    torch = _torch()
    shape, st = x1.shape, x1.stride()
    if len(shape) != 3:
        raise ValueError("x1 must be a 3-D bf16 CUDA tensor [B, L, D]")
    B, L, D = shape
    ld = _like(x1, shape, None, 0, "x1")
    if _like(x2, shape, st, ld, "x2") != ld or _like(x3, shape, st, ld, "x3") != ld:
        raise ValueError("x1, x2, x3 must share one row stride")
    ld_g = _like(gate, shape, st, ld, "gate")
    _f32(log_rate, (D,), "log_rate", False)
    _f32(Dskip, (D,), "Dskip")
    _reset(reset, B, L)
    _f32(state_in, (B, D), "state_in")
    _f32(state_out, (B, D), "state_out")
    _f32(unit_states, (B, -(-L // RECURRENCE_UNIT), D), "unit_states")
    here = _here(x1, x2, x3, gate, log_rate, Dskip, reset, y, state_in, state_out, unit_states,
                 None if workspace is None else workspace.buf)
    if y is None:
        y, ld_y = torch.empty_like(x1, memory_format=torch.contiguous_format), D
    else:
        ld_y = _like(y, shape, st, ld, "y")
    if workspace is None:
        workspace = RecurrenceWorkspace(B, L, D)
    rc = lib().hyena_gated_recurrence(x1.data_ptr(), x2.data_ptr(), x3.data_ptr(), ld, gate.data_ptr(), ld_g,
                                      log_rate.data_ptr(), _opt(Dskip), _opt(reset), 1 if normalize else 0,
                                      y.data_ptr(), ld_y, _opt(state_in), _opt(state_out), _opt(unit_states),
                                      B, L, D, workspace.buf.data_ptr(), workspace.nbytes, here)
    check("hyena_gated_recurrence", rc)
    return y


class RecurrenceGrads(NamedTuple):
    """Gradients of gated_recurrence (dDskip is None without Dskip)."""
    dx1: object
    dx2: object
    dx3: object
    dgate: object
    dlog_rate: object
    dDskip: object
    dstate_in: object


def gated_recurrence_backward(dy, x1, x2, x3, gate, log_rate, Dskip, unit_states, reset=None, normalize=True,
                              dstate_out=None, dx1=None, dx2=None, dx3=None, dgate=None, dstate_in=None,
                              workspace: RecurrenceWorkspace | None = None, stream=None) -> RecurrenceGrads:
    """Gradients of ``gated_recurrence`` from dy ([B, L, D] bf16) and, if
    given, the gradient of its last state (dstate_out, [B, D] fp32), with the
    forward call's inputs and the unit_states it filled.  dx1, dx2, dx3
    (sharing a row stride), dgate and dstate_in are allocated if not given."""
    if stream is not None:
        with _current(stream):
            return gated_recurrence_backward(dy, x1, x2, x3, gate, log_rate, Dskip, unit_states, reset, normalize,
                                             dstate_out, dx1, dx2, dx3, dgate, dstate_in, workspace)
    torch = _torch()
    shape, st = x1.shape, x1.stride()
    if len(shape) != 3:
        raise ValueError("x1 must be a 3-D bf16 CUDA tensor [B, L, D]")
    B, L, D = shape
    ld = _like(x1, shape, None, 0, "x1")
    if _like(x2, shape, st, ld, "x2") != ld or _like(x3, shape, st, ld, "x3") != ld:
        raise ValueError("x1, x2, x3 must share one row stride")
    ld_g, ld_dy = _like(gate, shape, st, ld, "gate"), _like(dy, shape, st, ld, "dy")
    _f32(log_rate, (D,), "log_rate", False)
    _f32(Dskip, (D,), "Dskip")
    _reset(reset, B, L)
    _f32(unit_states, (B, -(-L // RECURRENCE_UNIT), D), "unit_states", False)
    _f32(dstate_out, (B, D), "dstate_out")
    _f32(dstate_in, (B, D), "dstate_in")
    here = _here(x1, x2, x3, gate, dy, log_rate, Dskip, reset, unit_states, dstate_out, dx1, dx2, dx3, dgate,
                 dstate_in, None if workspace is None else workspace.buf)
    dense = torch.contiguous_format
    if dx1 is None and dx2 is None and dx3 is None:
        dx1, dx2, dx3 = (torch.empty_like(x1, memory_format=dense) for _ in range(3))
        ld_dx = D
    elif dx1 is None or dx2 is None or dx3 is None:
        raise ValueError("give all of dx1, dx2, dx3 or none")
    else:
        ld_dx = _like(dx1, shape, st, ld, "dx1")
        if _like(dx2, shape, st, ld, "dx2") != ld_dx or _like(dx3, shape, st, ld, "dx3") != ld_dx:
            raise ValueError("dx1, dx2, dx3 must share one row stride")
    if dgate is None:
        dgate, ld_dg = torch.empty_like(x1, memory_format=dense), D
    else:
        ld_dg = _like(dgate, shape, st, ld, "dgate")
    if dstate_in is None:
        dstate_in = unit_states.new_empty((B, D))
    dlog_rate = torch.empty_like(log_rate)
    dDskip = None if Dskip is None else torch.empty_like(Dskip)
    if workspace is None:
        workspace = RecurrenceWorkspace(B, L, D)
    rc = lib().hyena_gated_recurrence_backward(
        dy.data_ptr(), ld_dy, x1.data_ptr(), x2.data_ptr(), x3.data_ptr(), ld, gate.data_ptr(), ld_g,
        log_rate.data_ptr(), _opt(Dskip), _opt(reset), 1 if normalize else 0, unit_states.data_ptr(),
        _opt(dstate_out), dx1.data_ptr(), dx2.data_ptr(), dx3.data_ptr(), ld_dx, dgate.data_ptr(), ld_dg,
        dlog_rate.data_ptr(), _opt(dDskip), dstate_in.data_ptr(), B, L, D, workspace.buf.data_ptr(),
        workspace.nbytes, here)
    check("hyena_gated_recurrence_backward", rc)
    return RecurrenceGrads(dx1, dx2, dx3, dgate, dlog_rate, dDskip, dstate_in)


def gated_recurrence_decode(x1, x2, x3, gate, log_rate, Dskip, state, normalize=True, y=None, stream=None):
    """One generated token through the gated recurrence: advances ``state``
    ([B, D] fp32, in place) and returns y ([B, D] or [B, 1, D] like x1).
    Equals ``gated_recurrence`` on a one-token sequence with state_in =
    state_out = state, bit for bit."""
    if stream is not None:
        with _current(stream):
            return gated_recurrence_decode(x1, x2, x3, gate, log_rate, Dskip, state, normalize, y)
    torch = _torch()
    B, D, ld = _bd(x1, "x1")
    shape, st, bf16 = x1.shape, x1.stride(), x1.dtype
    for t, name in ((x2, "x2"), (x3, "x3"), (gate, "gate")):
        if t.dtype is not bf16 or t.shape != shape:
            raise ValueError(f"{name} must be a bf16 CUDA tensor of x1's shape")
    if (x2.stride() != st or x3.stride() != st) and (_bd(x2, "x2")[2] != ld or _bd(x3, "x3")[2] != ld):
        raise ValueError("x1, x2, x3 must share one row stride")
    ld_g = ld if gate.stride() == st else _bd(gate, "gate")[2]
    _f32(log_rate, (D,), "log_rate", False)
    _f32(Dskip, (D,), "Dskip")
    _f32(state, (B, D), "state", False)
    here = _here(x1, x2, x3, gate, log_rate, Dskip, state, y)
    if y is None:
        y, ld_y = torch.empty_like(x1, memory_format=torch.contiguous_format), D
    else:
        yB, yD, ld_y = _bd(y, "y")
        if (yB, yD) != (B, D):
            raise ValueError("y shape differs from x")
    rc = lib().hyena_gated_recurrence_decode(x1.data_ptr(), x2.data_ptr(), x3.data_ptr(), ld, gate.data_ptr(), ld_g,
                                             log_rate.data_ptr(), _opt(Dskip), 1 if normalize else 0, y.data_ptr(),
                                             ld_y, state.data_ptr(), B, D, here)
    check("hyena_gated_recurrence_decode", rc)
    return y


# -------------------------------------------------------------------- RMS norm

def _rows(x, name, dtypes):
    """[M, D] or [B, L, D] tensor with unit channel stride and evenly spaced
    rows -> (rows, D, ld); the device is checked by _here."""
    sh, st = x.shape, x.stride()
    if x.dtype not in dtypes or len(sh) not in (2, 3):
        raise ValueError(f"{name} must be a CUDA tensor [rows, D] or [B, L, D] of type {' or '.join(map(str, dtypes))}")
    if st[-1] != 1:
        raise ValueError(f"{name} must be channel-contiguous")
    if len(sh) == 2:
        M, D = sh
        return M, D, st[0] if M > 1 else D
    B, L, D = sh
    ld = st[1] if L > 1 else (st[0] if B > 1 else D)
    if B > 1 and L > 1 and st[0] != L * ld:
        raise ValueError(f"{name}: batch stride must equal L * row stride")
    return B * L, D, ld


def _new_codes(x, width):
    """(codes, row stride) for x's rows, `width` a row: a stride of whole 16 bytes,
    as the products ask of their operands."""
    sh = x.shape
    if width % 16 == 0 and width == sh[-1]:  # half the time of the other way
        torch = _torch()
        return torch.empty_like(x, dtype=_E4M3, memory_format=torch.contiguous_format), width
    ld = (width + 15) & ~15
    q = x.new_empty((*sh[:-1], ld), dtype=_E4M3)
    return (q if ld == width else q[..., :width]), ld


def _weight(t, D):
    """hyena_dtype_t of a norm weight."""
    torch = _torch()
    if (t.dtype is not torch.float32 and t.dtype is not torch.bfloat16) or t.shape != (D,) or not t.is_contiguous():
        raise ValueError(f"weight must be a contiguous fp32 or bf16 tensor of shape {(D,)}")
    return _dtype_code(t)


def _dtype_code(t):
    """hyena_dtype_t of a tensor (bf16 or fp32)."""
    return 1 if t.dtype is _torch().bfloat16 else 2


def _norm_inputs(x, weight, residual, residual_out, rstd):
    """Checks what both forms of the norm take -> (rows, D, ld_x, weight type,
    ld_r, residual type)."""
    torch = _torch()
    M, D, ld = _rows(x, "x", (torch.bfloat16,))
    wt = _weight(weight, D)
    _f32(rstd, (M,), "rstd")
    ld_r, kind = 0, 1
    if residual is not None:
        rM, rD, ld_r = _rows(residual, "residual", (torch.bfloat16, torch.float32))
        if rM != M or rD != D:
            raise ValueError("residual shape differs from x")
        kind = _dtype_code(residual)
        if residual_out is not None and (
                residual_out.dtype is not residual.dtype or residual_out.shape != residual.shape
                or (residual_out.stride() != residual.stride()
                    and _rows(residual_out, "residual_out", (residual.dtype,))[2] != ld_r)):
            raise ValueError("residual_out must have the residual's type, shape and row stride")
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    return M, D, ld, wt, ld_r, kind


def rms_norm(x, weight, eps=1e-6, residual=None, residual_out=None, y=None, rstd=None, stream=None):
    """Root-mean-square norm of each row of h = x + residual (or x), times
    weight.  x: [rows, D] or [B, L, D] bf16; weight: [D] fp32 or bf16;
    residual, residual_out: bf16 or fp32 (residual_out receives h, and may be
    the residual itself); rstd: [rows] fp32 or None, filled for the backward
    call.  Returns y (bf16, allocated if not given)."""
    if stream is not None:
        with _current(stream):
            return rms_norm(x, weight, eps, residual, residual_out, y, rstd)
    torch = _torch()
    M, D, ld, wt, ld_r, kind = _norm_inputs(x, weight, residual, residual_out, rstd)
    here = _here(x, weight, residual, residual_out, y, rstd)
    if y is None:
        y, ld_y = torch.empty_like(x, memory_format=torch.contiguous_format), D
    else:
        yM, yD, ld_y = _rows(y, "y", (torch.bfloat16,))
        if yM != M or yD != D:
            raise ValueError("y shape differs from x")
    rc = lib().hyena_rms_norm(x.data_ptr(), ld, _opt(residual), _opt(residual_out), ld_r, kind, weight.data_ptr(), wt,
                              eps, y.data_ptr(), ld_y, _opt(rstd), M, D, here)
    check("hyena_rms_norm", rc)
    return y


def rms_norm_fp8(x, weight, eps=1e-6, residual=None, residual_out=None, group=0, q=None, scales=None, rstd=None,
                 stream=None):
    """``rms_norm`` with an 8-bit output: returns (q, scales) with y ~ q scale,
    q float8_e4m3fn of x's shape and one fp32 scale per row (group = 0, shape
    [rows, 1]) or per 128 channels (group = 128, [rows, ceil(D / 128)]).  An
    allocated q has its rows at multiples of 16 bytes, as ``fp8_matmul`` takes
    them: it is contiguous where D is a multiple of 16."""
    if stream is not None:
        with _current(stream):
            return rms_norm_fp8(x, weight, eps, residual, residual_out, group, q, scales, rstd)
    torch = _torch()
    M, D, ld, wt, ld_r, kind = _norm_inputs(x, weight, residual, residual_out, rstd)
    if group not in (0, 128):
        raise ValueError("group must be 0 (one scale per row) or 128")
    here = _here(x, weight, residual, residual_out, q, scales, rstd)
    if q is None:
        q, ld_q = _new_codes(x, D)
    else:
        qM, qD, ld_q = _rows(q, "q", (torch.float8_e4m3fn,))
        if qM != M or qD != D:
            raise ValueError("q shape differs from x")
    want = (M, 1 if group == 0 else -(-D // 128))
    if scales is None:
        scales = x.new_empty(want, dtype=torch.float32)
    else:
        _f32(scales, want, "scales")
    rc = lib().hyena_rms_norm_fp8(x.data_ptr(), ld, _opt(residual), _opt(residual_out), ld_r, kind,
                                  weight.data_ptr(), wt, eps, q.data_ptr(), ld_q, scales.data_ptr(), group,
                                  _opt(rstd), M, D, here)
    check("hyena_rms_norm_fp8", rc)
    return q, scales


class NormGrads(NamedTuple):
    """Gradients of rms_norm: of x, of the residual and of the weight (fp32).
    The gradient of a bf16 residual is dx itself."""
    dx: object
    dresidual: object
    dweight: object


def rms_norm_backward(dy, h, weight, rstd, dresidual_out=None, dx=None, dresidual=None, workspace=None,
                      stream=None) -> NormGrads:
    """Gradients of ``rms_norm`` (and of ``rms_norm_fp8``, its rounding passed
    straight through) from dy (bf16), with h the forward call's residual_out
    (or its x) and the rstd it filled; dresidual_out: the gradient of
    residual_out, of h's type, or None.  dx (bf16) and, for an fp32 residual,
    dresidual (fp32; may be dresidual_out) are allocated if not given;
    ``workspace``: a uint8 tensor of rms_norm_backward_workspace_size bytes."""
    if stream is not None:
        with _current(stream):
            return rms_norm_backward(dy, h, weight, rstd, dresidual_out, dx, dresidual, workspace)
    torch = _torch()
    M, D, ld_dy = _rows(dy, "dy", (torch.bfloat16,))
    hM, hD, ld_h = _rows(h, "h", (torch.bfloat16, torch.float32))
    if hM != M or hD != D:
        raise ValueError("h shape differs from dy")
    wt, ht = _weight(weight, D), _dtype_code(h)
    _f32(rstd, (M,), "rstd", False)
    if workspace is not None and (workspace.dtype is not torch.uint8 or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous uint8 tensor")
    here = _here(dy, h, weight, rstd, dresidual_out, dx, dresidual, workspace)
    if dx is None:
        dx, ld_dx = torch.empty_like(dy, memory_format=torch.contiguous_format), D
    else:
        xM, xD, ld_dx = _rows(dx, "dx", (torch.bfloat16,))
        if xM != M or xD != D:
            raise ValueError("dx shape differs from dy")
    ld_r = ld_dr = 0
    if dresidual_out is not None:
        rM, rD, ld_r = _rows(dresidual_out, "dresidual_out", (h.dtype,))
        if rM != M or rD != D:
            raise ValueError("dresidual_out shape differs from dy")
    if ht == 1:
        if dresidual is not None:
            raise ValueError("the gradient of a bf16 residual is dx: give no dresidual")
    elif dresidual is None:
        dresidual, ld_dr = torch.empty_like(h, memory_format=torch.contiguous_format), D
    else:
        rM, rD, ld_dr = _rows(dresidual, "dresidual", (h.dtype,))
        if rM != M or rD != D:
            raise ValueError("dresidual shape differs from dy")
    dweight = rstd.new_empty(D)
    if workspace is None:
        need = int(lib().hyena_rms_norm_backward_workspace_size(M, D))
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dy.device)
    rc = lib().hyena_rms_norm_backward(dy.data_ptr(), ld_dy, h.data_ptr(), ld_h, ht, weight.data_ptr(), wt,
                                       rstd.data_ptr(), _opt(dresidual_out), ld_r, dx.data_ptr(), ld_dx,
                                       _opt(dresidual), ld_dr, dweight.data_ptr(), M, D, workspace.data_ptr(),
                                       workspace.nbytes, here)
    check("hyena_rms_norm_backward", rc)
    return NormGrads(dx, dx if ht == 1 else dresidual, dweight)


# ----------------------------------------- 8-bit products, feed-forward block

def _act(name):
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}")
    return code


def _matrix(t, name, dtype):
    """(rows, width, row stride) of a weight with unit stride within a row."""
    sh, st = t.shape, t.stride()
    if t.dtype is not dtype or len(sh) != 2 or st[1] != 1:
        kind = "e4m3" if dtype is _E4M3 else "bf16"
        raise ValueError(f"{name} must be a {kind} CUDA tensor [rows, width], contiguous within its rows")
    rows, width = sh
    return rows, width, st[0] if rows > 1 else max(st[0], width)


def _pair(a, b, names, dtype, D):
    """Two weights [F, D] of one shape and row stride -> (F, row stride)."""
    F, width, ld = _matrix(a, names[0], dtype)
    if width != D:
        raise ValueError(f"weights must be of shape [F, {D}]")
    if b.dtype is not dtype or b.shape != a.shape or b.stride() != a.stride() and _matrix(b, names[1], dtype)[2] != ld:
        raise ValueError(f"{names[1]} must have the type, shape and row stride of {names[0]}")
    return F, ld


def _codes(x, x_scales, name):
    """Codes [M, K] or [B, L, K] with scales [M, 1] or [M, ceil(K / 128)] ->
    (M, K, ld, group)."""
    M, K, ld = _rows(x, name, (_E4M3,))
    if M == 1:  # no second row: any stride will do
        ld = -(-K // 16) * 16
    groups = -(-K // 128)
    sh = x_scales.shape
    if len(sh) != 2 or sh[0] != M or (sh[1] != 1 and sh[1] != groups) or x_scales.dtype is not _F32 \
            or not x_scales.is_contiguous():
        raise ValueError(f"{name}'s scales must be a contiguous fp32 tensor of shape {(M, 1)} or {(M, groups)}")
    return M, K, ld, 0 if sh[1] == 1 else 128  # one scale a row; the same thing where a row is one group


def _weight_scales(t, N, K, name):
    if t.dtype is not _F32 or t.shape != (-(-N // 128), -(-K // 128)) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp32 tensor of shape {(-(-N // 128), -(-K // 128))}")


def _out_rows(t, M, width, dtype, name):
    """Row stride of a given [M, width] (or [B, L, width]) tensor."""
    tM, tW, ld = _rows(t, name, (dtype,))
    if tM != M or tW != width:
        raise ValueError(f"{name} must be of shape [..., {width}] with {M} rows")
    return ld


def _kept(gate, up, M, F):
    """(row stride, hyena_dtype_t) of the two kept products."""
    torch = _torch()
    if gate is None or up is None:
        raise ValueError("give both of gate and up or neither")
    gM, gF, ld = _rows(gate, "gate", (torch.bfloat16, torch.float32))
    if gM != M or gF != F or _out_rows(up, M, F, gate.dtype, "up") != ld:
        raise ValueError(f"gate and up must be of shape [..., {F}] with {M} rows, of one type and row stride")
    return ld, _dtype_code(gate)


class MatmulWorkspace:
    """Device workspace of fp8_matmul for up to M rows, N outputs and K channels,
    its header zero-filled once at creation; for calls in order on one stream."""

    def __init__(self, M: int, N: int, K: int, device=None, stream=None):
        n = int(lib().hyena_fp8_matmul_workspace_size(M, N, K))
        if n == 0:
            raise ValueError("invalid workspace shape")
        self.nbytes = n
        self.buf = _zeroed(n, device, stream, PRODUCT_HEADER)


class FfnWorkspace:
    """Device workspace of gated_ffn and gated_ffn_fp8 for up to M rows (with
    ``backward``, of gated_ffn_backward too), its header zero-filled once at
    creation; for calls in order on one stream."""

    def __init__(self, M: int, D: int, F: int, backward: bool = False, device=None, stream=None):
        n = int(lib().hyena_gated_ffn_workspace_size(M, D, F, 1 if backward else 0))
        if n == 0:
            raise ValueError("invalid workspace shape")
        self.nbytes = n
        self.buf = _zeroed(n, device, stream, PRODUCT_HEADER)


def fp8_quantize(x, block=1, q=None, scales=None, stream=None):
    """e4m3 codes of x ([rows, D] or [B, L, D], bf16 or fp32) with one fp32 scale
    per row and 128 channels (block = 1, scales [rows, ceil(D / 128)]:
    activations) or per 128 rows x 128 channels (block = 128, scales
    [ceil(rows / 128), ceil(D / 128)]: weights): returns (q, scales) with
    x ~ q scale, q float8_e4m3fn of x's shape.  An allocated q has its rows at
    multiples of 16 bytes, as the products take them: it is contiguous where D
    is a multiple of 16."""
    if stream is not None:
        with _current(stream):
            return fp8_quantize(x, block, q, scales)
    torch = _torch()
    M, D, ld = _rows(x, "x", (torch.bfloat16, torch.float32))
    if block not in (1, 128):
        raise ValueError("block must be 1 (rows of activations) or 128 (blocks of a weight)")
    here = _here(x, q, scales)
    if q is None:
        q, ld_q = _new_codes(x, D)
    else:
        qM, qD, ld_q = _rows(q, "q", (torch.float8_e4m3fn,))
        if qM != M or qD != D:
            raise ValueError("q shape differs from x")
    want = (M if block == 1 else -(-M // 128), -(-D // 128))
    if scales is None:
        scales = x.new_empty(want, dtype=torch.float32)
    else:
        _f32(scales, want, "scales")
    rc = lib().hyena_fp8_quantize(x.data_ptr(), ld, _dtype_code(x), q.data_ptr(), ld_q, scales.data_ptr(), block, M, D,
                                  here)
    check("hyena_fp8_quantize", rc)
    return q, scales


def fp8_matmul(x, x_scales, weight, weight_scales, y=None, dtype=None, workspace: MatmulWorkspace | None = None,
               stream=None):
    """x weight^T of e4m3 tensors with scales, summed in fp32: x [M, K] or
    [B, L, K] with x_scales [M, 1] or [M, ceil(K / 128)] (as rms_norm_fp8 and
    fp8_quantize leave them), weight [N, K] with weight_scales
    [ceil(N / 128), ceil(K / 128)] (fp8_quantize with block = 128).  Returns y
    ([..., N], bf16 or the given dtype bf16 or fp32, allocated if not given).
    Row strides of x and weight: multiples of 16, whatever K (the calls that make
    codes allocate them so).

    A device wait that ran out leaves NaN and is reported by workspace_check; a
    call without a ``workspace`` uses one of its own."""
    if stream is not None:
        with _current(stream):
            return fp8_matmul(x, x_scales, weight, weight_scales, y, dtype, workspace)
    torch = _torch()
    M, K, ld, group = _codes(x, x_scales, "x")
    N, Kw, ld_w = _matrix(weight, "weight", _E4M3)
    if Kw != K:
        raise ValueError(f"weight must be [N, {K}]")
    _weight_scales(weight_scales, N, K, "weight_scales")
    here = _here(x, x_scales, weight, weight_scales, y, None if workspace is None else workspace.buf)
    if y is None:
        if dtype is None:
            dtype = torch.bfloat16
        elif dtype is not torch.bfloat16 and dtype is not torch.float32:
            raise ValueError("dtype must be bf16 or fp32")
        y, ld_y = x.new_empty((*x.shape[:-1], N), dtype=dtype), N
    else:
        if dtype not in (None, y.dtype) or y.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("y must be bf16 or fp32, and of the given dtype")
        ld_y = _out_rows(y, M, N, y.dtype, "y")
    if workspace is None:
        workspace = MatmulWorkspace(M, N, K)
    rc = lib().hyena_fp8_matmul(x.data_ptr(), ld, x_scales.data_ptr(), group, weight.data_ptr(), ld_w,
                                weight_scales.data_ptr(), y.data_ptr(), ld_y, _dtype_code(y), M, N, K,
                                workspace.buf.data_ptr(), workspace.nbytes, here)
    check("hyena_fp8_matmul", rc)
    return y


def gated_ffn(x, gate_weight, up_weight, activation="silu", y=None, gate_out=None, up_out=None,
              workspace: FfnWorkspace | None = None, stream=None):
    """Gated feed-forward block up to its down projection: y = act(x Wg^T) (x Wu^T).
    x: [M, D] or [B, L, D] bf16; gate_weight, up_weight: [F, D] bf16 with one
    row stride; activation: silu, gelu, gelu_tanh or identity; gate_out,
    up_out: [M, F] (or [B, L, F]), both bf16 or both fp32, or None: the two
    products, kept for the gradient (in bf16 its error is 3.0e-3 of its norm, in
    fp32 2.3e-3, of which 1.7e-3 is its own rounding).  Returns y ([..., F] bf16, allocated if
    not given)."""
    if stream is not None:
        with _current(stream):
            return gated_ffn(x, gate_weight, up_weight, activation, y, gate_out, up_out, workspace)
    torch = _torch()
    act = _act(activation)
    M, D, ld = _rows(x, "x", (torch.bfloat16,))
    F, ld_w = _pair(gate_weight, up_weight, ("gate_weight", "up_weight"), _BF16, D)
    here = _here(x, gate_weight, up_weight, y, gate_out, up_out, None if workspace is None else workspace.buf)
    if y is None:
        y, ld_y = x.new_empty((*x.shape[:-1], F)), F
    else:
        ld_y = _out_rows(y, M, F, torch.bfloat16, "y")
    ld_g, kind = (0, 1) if gate_out is None and up_out is None else _kept(gate_out, up_out, M, F)
    if workspace is None:
        workspace = FfnWorkspace(M, D, F)
    rc = lib().hyena_gated_ffn(x.data_ptr(), ld, gate_weight.data_ptr(), up_weight.data_ptr(), ld_w, act, y.data_ptr(),
                               ld_y, _opt(gate_out), _opt(up_out), ld_g, kind, M, D, F, workspace.buf.data_ptr(),
                               workspace.nbytes, here)
    check("hyena_gated_ffn", rc)
    return y


def gated_ffn_fp8(x, x_scales, gate_weight, gate_scales, up_weight, up_scales, activation="silu", fp8_out=False,
                  y=None, q=None, scales=None, workspace: FfnWorkspace | None = None, stream=None):
    """``gated_ffn`` of e4m3 operands with scales as in ``fp8_matmul``.  Returns
    y ([..., F] bf16), or with ``fp8_out`` (q, scales): y's codes with one scale
    per row and 128 of its values, as the down projection by ``fp8_matmul``
    takes them (an allocated q with its rows at multiples of 16 bytes)."""
    if stream is not None:
        with _current(stream):
            return gated_ffn_fp8(x, x_scales, gate_weight, gate_scales, up_weight, up_scales, activation, fp8_out, y,
                                 q, scales, workspace)
    torch = _torch()
    e4m3 = torch.float8_e4m3fn
    act = _act(activation)
    M, D, ld, group = _codes(x, x_scales, "x")
    F, ld_w = _pair(gate_weight, up_weight, ("gate_weight", "up_weight"), e4m3, D)
    _weight_scales(gate_scales, F, D, "gate_scales")
    _weight_scales(up_scales, F, D, "up_scales")
    here = _here(x, x_scales, gate_weight, gate_scales, up_weight, up_scales, y, q, scales,
                 None if workspace is None else workspace.buf)
    ld_y = ld_q = 0
    if fp8_out:
        if y is not None:
            raise ValueError("y is the bf16 output: give q and scales with fp8_out")
        if q is None:
            q, ld_q = _new_codes(x, F)
        else:
            ld_q = _out_rows(q, M, F, e4m3, "q")
            if M == 1:  # no second row: any stride will do
                ld_q = (F + 15) & ~15
        want = (M, -(-F // 128))
        if scales is None:
            scales = x_scales.new_empty(want)
        else:
            _f32(scales, want, "scales")
    else:
        if q is not None or scales is not None:
            raise ValueError("q and scales are the output of fp8_out")
        if y is None:
            y, ld_y = torch.empty((*x.shape[:-1], F), dtype=torch.bfloat16, device=x.device), F
        else:
            ld_y = _out_rows(y, M, F, torch.bfloat16, "y")
    if workspace is None:
        workspace = FfnWorkspace(M, D, F)
    rc = lib().hyena_gated_ffn_fp8(x.data_ptr(), ld, x_scales.data_ptr(), group, gate_weight.data_ptr(),
                                   gate_scales.data_ptr(), up_weight.data_ptr(), up_scales.data_ptr(), ld_w, act,
                                   _opt(y), ld_y, _opt(q), ld_q, _opt(scales), M, D, F, workspace.buf.data_ptr(),
                                   workspace.nbytes, here)
    check("hyena_gated_ffn_fp8", rc)
    return (q, scales) if fp8_out else y


class FfnGrads(NamedTuple):
    """Gradients of gated_ffn: of x and of the two weights (bf16)."""
    dx: object
    dgate_weight: object
    dup_weight: object


def gated_ffn_backward(dy, x, gate_weight, up_weight, gate, up, activation="silu", dx=None, dgate_weight=None,
                       dup_weight=None, workspace: FfnWorkspace | None = None, stream=None) -> FfnGrads:
    """Gradients of ``gated_ffn`` from dy ([..., F] bf16), the forward call's
    inputs and the gate and up products it kept.  dx and the weights' gradients
    (bf16, written not added to; one row stride; in no input's place) are
    allocated if not given; ``workspace``: an FfnWorkspace made with backward = True."""
    if stream is not None:
        with _current(stream):
            return gated_ffn_backward(dy, x, gate_weight, up_weight, gate, up, activation, dx, dgate_weight,
                                      dup_weight, workspace)
    torch = _torch()
    b = torch.bfloat16
    act = _act(activation)
    M, D, ld = _rows(x, "x", (b,))
    F, ld_w = _pair(gate_weight, up_weight, ("gate_weight", "up_weight"), b, D)
    ld_dy = _out_rows(dy, M, F, b, "dy")
    ld_g, kind = _kept(gate, up, M, F)
    here = _here(dy, x, gate_weight, up_weight, gate, up, dx, dgate_weight, dup_weight,
                 None if workspace is None else workspace.buf)
    if dx is None:
        dx, ld_dx = torch.empty_like(x, memory_format=torch.contiguous_format), D
    else:
        ld_dx = _out_rows(dx, M, D, b, "dx")
    if dgate_weight is None and dup_weight is None:
        dgate_weight, dup_weight, ld_dw = x.new_empty((F, D)), x.new_empty((F, D)), D
    elif dgate_weight is None or dup_weight is None:
        raise ValueError("give both of dgate_weight and dup_weight or neither")
    else:
        if dgate_weight.shape != (F, D):
            raise ValueError(f"dgate_weight must be of shape {(F, D)}")
        ld_dw = _pair(dgate_weight, dup_weight, ("dgate_weight", "dup_weight"), b, D)[1]
    if workspace is None:
        workspace = FfnWorkspace(M, D, F, backward=True)
    rc = lib().hyena_gated_ffn_backward(dy.data_ptr(), ld_dy, x.data_ptr(), ld, gate_weight.data_ptr(),
                                        up_weight.data_ptr(), ld_w, gate.data_ptr(), up.data_ptr(), ld_g, kind, act,
                                        dx.data_ptr(), ld_dx, dgate_weight.data_ptr(), dup_weight.data_ptr(), ld_dw,
                                        M, D, F, workspace.buf.data_ptr(), workspace.nbytes, here)
    check("hyena_gated_ffn_backward", rc)
    return FfnGrads(dx, dgate_weight, dup_weight)
