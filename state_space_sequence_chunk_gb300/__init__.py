"""GB300-native (sm_103a) Mamba-2 SSD chunked-scan forward pass.

A thin ctypes binding over the C ABI in ``include/ssd.h`` (``_lib/libssd.so``,
built in-tree by :mod:`state_space_sequence_chunk_gb300.build`).  The Python
side only marshals arguments: it allocates outputs and workspace with torch,
passes raw device pointers and torch's current CUDA stream, and turns status
codes into exceptions.  Every step of the computation runs in the library's
CUDA kernels; there is no CPU or PyTorch fallback -- if the library is missing,
the calls raise.

Entry points (same names as the C ABI):

* :func:`ssd_fwd` -- the whole forward pass, ``(y, final_state)``.
* :func:`ssd_chunk_cumsum`, :func:`ssd_fwd_pass_state`,
  :func:`ssd_compute_out` -- the three steps one at a time.
* :func:`ssd_fwd_workspace_bytes`, :func:`ssd_intermediate_bytes`.
* :func:`linattn_fwd`, :func:`linattn_bwd`, :func:`linattn_step` -- linear
  attention with a decay for each head: prompts, their gradient, single tokens.
* :func:`block_norm_fwd`, :func:`block_norm_bwd` -- the norms before and after a
  block with its gate and residual scale, and their gradient.
* :func:`short_conv_fwd`, :func:`short_conv_bwd`, :func:`short_conv_step` -- the
  depthwise causal convolution over packed rows: prompts, gradient, single tokens.
* :func:`selscan_fwd`, :func:`selscan_bwd`, :func:`selscan_step` -- the selective
  scan, with a decay for every state of every channel: the same three.

None of these is recorded by autograd: what they return is cut from the graph, also of
inputs that require a gradient.  A training step calls the ``_bwd`` functions, from an
``autograd.Function`` for instance (``examples/linear_attention_block.py`` has one for each pair).
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libssd.so")

SSD_F32, SSD_BF16 = 0, 1
STATUS = {0: "SSD_OK", 1: "SSD_ERR_NULL", 2: "SSD_ERR_SHAPE", 3: "SSD_ERR_DTYPE",
          4: "SSD_ERR_ALIGN", 5: "SSD_ERR_WORKSPACE", 6: "SSD_ERR_ARCH", 7: "SSD_ERR_CUDA",
          8: "SSD_ERR_ALIAS", 9: "SSD_ERR_TIMEOUT"}
EXPORTS = ["ssd_abi_version", "ssd_status_string", "ssd_fwd_workspace_bytes",
           "ssd_intermediate_bytes", "ssd_fwd", "ssd_chunk_cumsum", "ssd_fwd_pass_state",
           "ssd_fwd_pass_state_scratch_bytes", "ssd_compute_out", "ssd_fwd_noalloc",
           "ssd_take_device_errors", "ssd_debug_withhold_handoffs", "ssd_step",
           "ssd_causal_conv1d", "ssd_gdn_chunk_fwd_h", "ssd_gdn_chunk_fwd_o",
           "ssd_fwd_host_staging_bytes", "ssd_fwd_host", "ssd_linattn_workspace_bytes",
           "ssd_linattn_fwd", "ssd_linattn_bwd", "ssd_linattn_step", "ssd_block_norm_fwd",
           "ssd_block_norm_bwd_workspace_bytes", "ssd_block_norm_bwd", "ssd_short_conv_fwd",
           "ssd_short_conv_bwd_workspace_bytes", "ssd_short_conv_bwd", "ssd_short_conv_step",
           "ssd_selscan_workspace_bytes", "ssd_selscan_fwd", "ssd_selscan_bwd", "ssd_selscan_step"]
GATES = {None: 0, "silu": 1, "sigmoid": 2}
ACTIVATIONS = {None: 0, "silu": 1}
SELSCAN_CHUNK = 16


class SSDError(RuntimeError):
    """A non-OK status returned by the library."""

    def __init__(self, code: int, message: str):
        super().__init__(f"{STATUS.get(code, code)}: {message}")
        self.code = code


class ConvDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("dim", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("width", ctypes.c_int64), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class GdnDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int64),
                ("kdim", ctypes.c_int64), ("vdim", ctypes.c_int64), ("chunk", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class LinattnDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in
                ("nseqs", "tokens", "nheads", "ngroups", "kdim", "vdim", "q_stride", "k_stride",
                 "v_stride", "max_seqlen")] + [("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class NormDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("tokens", "width", "ngroups", "y_stride", "z_stride")] + [
        ("gate", ctypes.c_int32), ("eps", ctypes.c_float), ("dtype", ctypes.c_int32),
        ("rdtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class ShortConvDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("nseqs", "tokens", "dim", "width", "x_stride")] + [
        ("activation", ctypes.c_int32), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class SelscanDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in
                ("nseqs", "tokens", "dim", "dstate", "ngroups", "x_stride", "dt_stride", "z_stride",
                 "B_stride", "C_stride", "max_seqlen")] + [
        ("dt_softplus", ctypes.c_int32), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("nheads", ctypes.c_int64), ("headdim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("chunk_size", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


_lock = threading.Lock()
_lib = None


def load_library(path: str = LIB_PATH):
    """Load libssd.so (cached).  Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(
                f"CUDA library not found at {path}; build it with "
                "`python -m state_space_sequence_chunk_gb300.build` (or __graft_entry__.build())")
        lib = ctypes.CDLL(path)
        vp, dp = ctypes.c_void_p, ctypes.POINTER(Dims)
        sz = ctypes.c_size_t
        lib.ssd_abi_version.argtypes, lib.ssd_abi_version.restype = [], ctypes.c_int
        lib.ssd_status_string.argtypes, lib.ssd_status_string.restype = [ctypes.c_int], ctypes.c_char_p
        lib.ssd_fwd_workspace_bytes.argtypes, lib.ssd_fwd_workspace_bytes.restype = [dp], sz
        lib.ssd_intermediate_bytes.argtypes = [dp, ctypes.POINTER(sz), ctypes.POINTER(sz)]
        lib.ssd_intermediate_bytes.restype = ctypes.c_int
        lib.ssd_fwd.argtypes = [dp] + [vp] * 10 + [sz, vp]
        lib.ssd_fwd.restype = ctypes.c_int
        lib.ssd_chunk_cumsum.argtypes = [dp] + [vp] * 5
        lib.ssd_chunk_cumsum.restype = ctypes.c_int
        lib.ssd_fwd_pass_state.argtypes = [dp] + [vp] * 8 + [sz, vp]
        lib.ssd_fwd_pass_state_scratch_bytes.argtypes = [dp]
        lib.ssd_fwd_pass_state_scratch_bytes.restype = sz
        lib.ssd_fwd_pass_state.restype = ctypes.c_int
        lib.ssd_compute_out.argtypes = [dp] + [vp] * 9
        lib.ssd_compute_out.restype = ctypes.c_int
        lib.ssd_debug_withhold_handoffs.argtypes = [ctypes.c_int]
        lib.ssd_debug_withhold_handoffs.restype = ctypes.c_int
        lib.ssd_take_device_errors.argtypes = []
        lib.ssd_take_device_errors.restype = ctypes.c_uint
        lib.ssd_fwd_noalloc.argtypes = [dp] + [vp] * 10
        lib.ssd_fwd_noalloc.restype = ctypes.c_int
        lib.ssd_step.argtypes = [dp] + [vp] * 9
        lib.ssd_step.restype = ctypes.c_int
        lib.ssd_causal_conv1d.argtypes = [ctypes.POINTER(ConvDims)] + [vp] * 5
        lib.ssd_causal_conv1d.restype = ctypes.c_int
        lib.ssd_gdn_chunk_fwd_h.argtypes = [ctypes.POINTER(GdnDims)] + [vp] * 9
        lib.ssd_gdn_chunk_fwd_h.restype = ctypes.c_int
        lib.ssd_gdn_chunk_fwd_o.argtypes = [ctypes.POINTER(GdnDims)] + [vp] * 7
        lib.ssd_gdn_chunk_fwd_o.restype = ctypes.c_int
        lib.ssd_fwd_host_staging_bytes.argtypes = [dp, ctypes.c_int]
        lib.ssd_fwd_host_staging_bytes.restype = sz
        lib.ssd_fwd_host.argtypes = [dp] + [vp] * 10 + [sz, ctypes.c_int, ctypes.POINTER(vp)]
        lib.ssd_fwd_host.restype = ctypes.c_int
        la, nd, f32, i64 = ctypes.POINTER(LinattnDims), ctypes.POINTER(NormDims), ctypes.c_float, ctypes.c_int64
        lib.ssd_linattn_workspace_bytes.argtypes = [la, ctypes.c_int]
        lib.ssd_linattn_workspace_bytes.restype = sz
        lib.ssd_linattn_fwd.argtypes = [la] + [vp] * 4 + [f32] + [vp] * 5 + [sz, vp]
        lib.ssd_linattn_fwd.restype = ctypes.c_int
        lib.ssd_linattn_bwd.argtypes = [la] + [vp] * 5 + [f32] + [vp] * 8 + [sz, vp]
        lib.ssd_linattn_bwd.restype = ctypes.c_int
        lib.ssd_linattn_step.argtypes = [la] + [vp] * 4 + [f32, vp, vp, i64, vp, vp]
        lib.ssd_linattn_step.restype = ctypes.c_int
        lib.ssd_block_norm_fwd.argtypes = [nd] + [vp] * 11
        lib.ssd_block_norm_fwd.restype = ctypes.c_int
        lib.ssd_block_norm_bwd_workspace_bytes.argtypes = [nd]
        lib.ssd_block_norm_bwd_workspace_bytes.restype = sz
        lib.ssd_block_norm_bwd.argtypes = [nd] + [vp] * 17 + [sz, vp]
        lib.ssd_block_norm_bwd.restype = ctypes.c_int
        cd, sd = ctypes.POINTER(ShortConvDims), ctypes.POINTER(SelscanDims)
        lib.ssd_short_conv_fwd.argtypes = [cd] + [vp] * 8
        lib.ssd_short_conv_fwd.restype = ctypes.c_int
        lib.ssd_short_conv_bwd_workspace_bytes.argtypes = [cd]
        lib.ssd_short_conv_bwd_workspace_bytes.restype = sz
        lib.ssd_short_conv_bwd.argtypes = [cd] + [vp] * 12 + [sz, vp]
        lib.ssd_short_conv_bwd.restype = ctypes.c_int
        lib.ssd_short_conv_step.argtypes = [cd] + [vp] * 5 + [i64, vp, vp]
        lib.ssd_short_conv_step.restype = ctypes.c_int
        lib.ssd_selscan_workspace_bytes.argtypes = [sd, ctypes.c_int]
        lib.ssd_selscan_workspace_bytes.restype = sz
        lib.ssd_selscan_fwd.argtypes = [sd] + [vp] * 14 + [sz, vp]
        lib.ssd_selscan_fwd.restype = ctypes.c_int
        lib.ssd_selscan_bwd.argtypes = [sd] + [vp] * 22 + [sz, vp]
        lib.ssd_selscan_bwd.restype = ctypes.c_int
        lib.ssd_selscan_step.argtypes = [sd] + [vp] * 10 + [i64, vp, vp]
        lib.ssd_selscan_step.restype = ctypes.c_int
        _lib = lib
        return lib


def _check(code: int):
    if code != 0:
        msg = load_library().ssd_status_string(code).decode()
        raise SSDError(code, msg)


def dims_for(x: torch.Tensor, B: torch.Tensor, chunk_size: int) -> Dims:
    """ssd_dims for x [b, L, H, P] and B [b, L, G, N]."""
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be [b, L, H, P] and B [b, L, G, N]")
    if x.dtype == torch.bfloat16:
        dt_code = SSD_BF16
    elif x.dtype == torch.float32:
        dt_code = SSD_F32
    else:
        raise TypeError(f"x must be float32 or bfloat16, got {x.dtype}")
    b, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    return Dims(b, L, H, P, N, G, int(chunk_size), dt_code, 0)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors must be contiguous CUDA tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def ssd_take_device_errors() -> int:
    """Read and clear the kernels' device-side error bits (0 = no bounded wait
    ever gave up).  Synchronises the device."""
    return int(load_library().ssd_take_device_errors())


def ssd_debug_withhold_handoffs(on: bool) -> None:
    """Test hook for failure detection: with ``on``, fwd_pass_state launches skip
    their range hand-offs, so the receiving CTAs' bounded waits give up and the
    launch ends early with error bit 0 set (see ``ssd_take_device_errors``)."""
    _check(load_library().ssd_debug_withhold_handoffs(1 if on else 0))


def ssd_fwd_workspace_bytes(dims: Dims) -> int:
    return int(load_library().ssd_fwd_workspace_bytes(ctypes.byref(dims)))


def ssd_intermediate_bytes(dims: Dims):
    g, h = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load_library().ssd_intermediate_bytes(ctypes.byref(dims), ctypes.byref(g), ctypes.byref(h)))
    return g.value, h.value


def ssd_fwd(x, dt, A, B, C, D=None, init_state=None, chunk_size: int = 256,
            return_final_state: bool = True, workspace=None, out=None, final_out=None):
    """The whole SSD forward pass on x's device and torch's current stream.

    x [b, L, H, P] and B, C [b, L, G, N] share one dtype (float32 or bfloat16);
    dt [b, L, H], A [H], D [H], init_state [b, H, P, N] are float32.
    Returns ``(y, final_state)`` (final_state None unless requested).
    ``workspace`` (uint8 CUDA tensor), ``out`` and ``final_out`` may be given
    to reuse buffers.
    """
    lib = load_library()
    dims = dims_for(x, B, chunk_size)
    y = out if out is not None else torch.empty_like(x)
    fin = None
    if return_final_state:
        fin = final_out if final_out is not None else torch.empty(
            (x.shape[0], x.shape[2], x.shape[3], B.shape[3]), dtype=torch.float32, device=x.device)
    nbytes = int(lib.ssd_fwd_workspace_bytes(ctypes.byref(dims)))
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=x.device)
    _check(lib.ssd_fwd(ctypes.byref(dims), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                       _ptr(init_state), _ptr(y), _ptr(fin), _ptr(workspace),
                       ctypes.c_size_t(workspace.numel()), _stream()))
    return y, fin


def _host_ptr(t):
    if t is None:
        return None
    if t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors must be contiguous host (CPU) tensors")
    return ctypes.c_void_p(t.data_ptr())


_copy_streams = {}


def ssd_fwd_host_staging_bytes(dims: Dims, nslices: int) -> int:
    return int(load_library().ssd_fwd_host_staging_bytes(ctypes.byref(dims), int(nslices)))


def ssd_fwd_host(x, dt, A, B, C, D=None, init_state=None, chunk_size: int = 256,
                 return_final_state: bool = True, nslices: int = None, staging=None, out=None,
                 final_out=None, device=None):
    """ssd_fwd on HOST tensors (pinned, for the copies to overlap): the batch is
    cut into ``nslices`` slices whose host-device copies overlap the other
    slices' computation.  The compute runs on torch's current stream of
    ``device`` (default: the current CUDA device); two copy streams are kept
    per device.  Returns host tensors ``(y, final_state)``; they are complete
    once that stream has reached the end of the call (synchronise it before
    reading them).  ``staging`` (uint8 CUDA tensor) may be given to reuse it.
    """
    lib = load_library()
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    dims = dims_for(x, B, chunk_size)
    b = x.shape[0]
    if nslices is None:
        nslices = max(1, min(b, 4))
    y = out if out is not None else torch.empty(x.shape, dtype=x.dtype, pin_memory=True)
    fin = None
    if return_final_state:
        fin = final_out if final_out is not None else torch.empty(
            (b, x.shape[2], x.shape[3], B.shape[3]), dtype=torch.float32, pin_memory=True)
    if b == 0:
        return y, fin
    nbytes = ssd_fwd_host_staging_bytes(dims, nslices)
    if staging is None:
        staging = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        if dev.index not in _copy_streams:
            _copy_streams[dev.index] = (torch.cuda.Stream(dev), torch.cuda.Stream(dev))
        s_in, s_out = _copy_streams[dev.index]
        streams = (ctypes.c_void_p * 3)(torch.cuda.current_stream(dev).cuda_stream,
                                        s_in.cuda_stream, s_out.cuda_stream)
        _check(lib.ssd_fwd_host(ctypes.byref(dims), _host_ptr(x), _host_ptr(dt), _host_ptr(A),
                                _host_ptr(B), _host_ptr(C), _host_ptr(D), _host_ptr(init_state),
                                _host_ptr(y), _host_ptr(fin), _ptr(staging),
                                ctypes.c_size_t(staging.numel()), int(nslices), streams))
    return y, fin


def ssd_chunk_cumsum(dt, A, chunk_size: int, x_dtype=torch.bfloat16):
    """Step 1: returns ``(Gcs, dtT)``, both [b, H, Lp] float32."""
    lib = load_library()
    b, L, H = dt.shape
    dims = Dims(b, L, H, 16, 16, 1, int(chunk_size),
                SSD_BF16 if x_dtype == torch.bfloat16 else SSD_F32, 0)
    nc = (L + chunk_size - 1) // chunk_size
    Gcs = torch.empty((b, H, nc * chunk_size), dtype=torch.float32, device=dt.device)
    dtT = torch.empty_like(Gcs)
    _check(lib.ssd_chunk_cumsum(ctypes.byref(dims), _ptr(dt), _ptr(A), _ptr(Gcs), _ptr(dtT),
                                _stream()))
    return Gcs, dtT


def ssd_fwd_pass_state(x, B, Gcs, dtT, init_state=None, chunk_size: int = 256,
                       return_final_state: bool = True, scratch=None):
    """Step 2: returns ``(hiddens [b, H, nc, N, P] in x.dtype, final_state)``;
    hiddens[b, h, c] is the chunk-start state transposed.  ``scratch`` (uint8
    device tensor of at least ssd_fwd_pass_state_scratch_bytes) is allocated
    here when not given."""
    lib = load_library()
    dims = dims_for(x, B, chunk_size)
    b, L, H, P = x.shape
    N = B.shape[3]
    nc = (L + chunk_size - 1) // chunk_size
    hid = torch.empty((b, H, nc, N, P), dtype=x.dtype, device=x.device)
    fin = torch.empty((b, H, P, N), dtype=torch.float32, device=x.device) if return_final_state else None
    need = int(lib.ssd_fwd_pass_state_scratch_bytes(ctypes.byref(dims)))
    if scratch is None and need > 0:
        scratch = torch.empty(need, dtype=torch.uint8, device=x.device)
    nbytes = 0 if scratch is None else scratch.numel() * scratch.element_size()
    _check(lib.ssd_fwd_pass_state(ctypes.byref(dims), _ptr(x), _ptr(B), _ptr(Gcs), _ptr(dtT),
                                  _ptr(init_state), _ptr(hid), _ptr(fin), _ptr(scratch), nbytes,
                                  _stream()))
    return hid, fin


def ssd_compute_out(x, B, C, Gcs, dtT, hiddens, D=None, chunk_size: int = 256):
    """Step 3: returns y [b, L, H, P] in x.dtype."""
    lib = load_library()
    dims = dims_for(x, B, chunk_size)
    y = torch.empty_like(x)
    _check(lib.ssd_compute_out(ctypes.byref(dims), _ptr(x), _ptr(B), _ptr(C), _ptr(Gcs), _ptr(dtT),
                               _ptr(hiddens), _ptr(D), _ptr(y), _stream()))
    return y


def _gdn_dims(k, vdim, chunk, *tensors):
    if k.dim() != 4:
        raise ValueError("k must be a [B, T, H, K] tensor")
    for t in (k,) + tensors:
        if t is not None and t.dtype != torch.float32:
            raise TypeError(f"the Gated DeltaNet kernels take float32 tensors, got {t.dtype}")
    B, T, H, K = k.shape
    return GdnDims(B, T, H, K, vdim, int(chunk), SSD_F32, 0)


def gdn_chunk_fwd_h(k, w, u, g, h0=None, chunk: int = 64, return_final_state: bool = True):
    """Gated DeltaNet state recurrence over chunks: returns ``(h [B, H, NT, K, V],
    v_new [B, T, H, V], final_state [B, H, K, V] or None)``; all fp32."""
    lib = load_library()
    d = _gdn_dims(k, u.shape[3], chunk, w, u, g, h0)
    B, T, H, K = k.shape
    V = u.shape[3]
    NT = -(-T // chunk)
    h = torch.empty((B, H, NT, K, V), dtype=torch.float32, device=k.device)
    v_new = torch.empty_like(u)
    fin = torch.empty((B, H, K, V), dtype=torch.float32, device=k.device) if return_final_state else None
    _check(lib.ssd_gdn_chunk_fwd_h(ctypes.byref(d), _ptr(k), _ptr(w), _ptr(u), _ptr(g), _ptr(h0),
                                   _ptr(h), _ptr(v_new), _ptr(fin), _stream()))
    return h, v_new, fin


def gdn_chunk_fwd_o(q, k, v_new, h, g, chunk: int = 64):
    """Gated DeltaNet chunk outputs: returns o [B, T, H, V] (fp32)."""
    lib = load_library()
    d = _gdn_dims(k, v_new.shape[3], chunk, q, v_new, h, g)
    o = torch.empty_like(v_new)
    _check(lib.ssd_gdn_chunk_fwd_o(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v_new), _ptr(h), _ptr(g),
                                   _ptr(o), _stream()))
    return o


def causal_conv1d(x, weight, bias=None):
    """Depthwise causal conv1d: x [b, dim, L] (bf16 or fp32), weight [dim, W] fp32,
    bias [dim] fp32 or None; returns out [b, dim, L] in x.dtype."""
    lib = load_library()
    if x.dim() != 3 or weight.dim() != 2:
        raise ValueError("x must be [b, dim, L] and weight [dim, W]")
    code = SSD_BF16 if x.dtype == torch.bfloat16 else SSD_F32
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"x must be float32 or bfloat16, got {x.dtype}")
    b, dim, L = x.shape
    d = ConvDims(b, dim, L, weight.shape[1], code, 0)
    out = torch.empty_like(x)
    _check(lib.ssd_causal_conv1d(ctypes.byref(d), _ptr(x), _ptr(weight), _ptr(bias), _ptr(out),
                                 _stream()))
    return out


def ssd_step(x, dt, A, B, C, D, state):
    """Token-by-token recurrence over x's L tokens (decode): updates ``state``
    [b, H, P, N] fp32 in place and returns y [b, L, H, P] in x.dtype."""
    lib = load_library()
    dims = dims_for(x, B, 64)
    y = torch.empty_like(x)
    _check(lib.ssd_step(ctypes.byref(dims), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                        _ptr(state), _ptr(y), _stream()))
    return y


def ssd_fwd_noalloc(x, dt, A, B, C, D=None, init_state=None, chunk_size: int = 256,
                    out=None, final_out=None):
    """ssd_fwd without a workspace argument, for callers that cannot allocate
    device memory: the library uses its own fixed 32 MiB device scratch array.

    The caller passes every input and output buffer (``out`` for y and, if the
    final state is wanted, ``final_out``); nothing is allocated here when both
    are given.  Problems needing more scratch than the fixed array raise
    SSD_ERR_WORKSPACE.  Calls on one device share the array, so calls that
    overlap on the GPU must be serialised by the caller.
    """
    lib = load_library()
    dims = dims_for(x, B, chunk_size)
    y = out if out is not None else torch.empty_like(x)
    _check(lib.ssd_fwd_noalloc(ctypes.byref(dims), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C),
                               _ptr(D), _ptr(init_state), _ptr(y), _ptr(final_out), _stream()))
    return y, final_out


# The calls below are often made for a single token, where the host's work is
# most of their time: pointers go as plain integers, and a contiguous tensor's
# rows need no further look.
_DTYPE_CODE = {torch.bfloat16: SSD_BF16, torch.float32: SSD_F32}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_int() -> int:
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _dtype_code(t: torch.Tensor, name: str) -> int:
    code = _DTYPE_CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return code


def _typed(t, name: str, dtype, shape):
    """t, checked: None passes, else dtype and shape have to be these."""
    if t is not None:
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t


def _addr(t):
    """Address of a contiguous CUDA tensor (None passes)."""
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors must be contiguous CUDA tensors")
    return t.data_ptr()


def _rows(t, inner: int):
    """Address and row stride of a tensor [rows, ...] whose rows are contiguous
    (`inner` elements each) and evenly spaced.  Rows that share memory, as a tensor
    expanded over its rows has them, are refused: the library reads a stride of 0 as
    contiguous rows, which lie past the end of such a tensor's one."""
    if not t.is_cuda:
        raise ValueError("tensors must be CUDA tensors")
    if t.is_contiguous():
        return t.data_ptr(), inner
    want = 1
    for n, s in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if n != 1 and s != want:
            raise ValueError("each row (all dimensions but the first) must be contiguous")
        want *= n
    if t.shape[0] > 1 and t.stride(0) < inner:
        raise ValueError("rows must not share memory (a tensor expanded over its rows needs .contiguous())")
    return t.data_ptr(), (t.stride(0) if t.shape[0] > 1 else inner)


def _linattn_dims(q, k, v, log_decay, nseqs, max_seqlen):
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q and k must be [tokens, G, K] and v [tokens, H, V]")
    T, G, K = q.shape
    H, V = v.shape[1:]
    dt = q.dtype
    _typed(k, "k", dt, (T, G, K))
    _typed(v, "v", dt, (T, H, V))
    _typed(log_decay, "log_decay", torch.float32, (H,))
    (qp, qs), (kp, ks), (vp, vs) = _rows(q, G * K), _rows(k, G * K), _rows(v, H * V)
    d = LinattnDims(nseqs, T, H, G, K, V, qs, ks, vs, max_seqlen, _dtype_code(q, "q"), 0)
    return d, qp, kp, vp


def _linattn_nseqs(cu_seqlens, nseqs):
    if cu_seqlens is None:
        return int(nseqs)
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be a 1-D int32 tensor of nseqs + 1 values")
    return cu_seqlens.numel() - 1


def _linattn_workspace(lib, d, backward, workspace, device):
    need = int(lib.ssd_linattn_workspace_bytes(ctypes.byref(d), backward))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    return workspace, 0 if workspace is None else workspace.numel() * workspace.element_size()


def linattn_fwd(q, k, v, log_decay, cu_seqlens=None, scale: float = None, init_state=None,
                nseqs: int = 1, max_seqlen: int = 0, return_final_state: bool = True,
                workspace=None, out=None, final_out=None):
    """Linear attention with a decay for each head: S_t = exp(log_decay[h]) S_{t-1} +
    v_t k_t^T, o_t = scale S_t q_t (scale: K**-0.5 if not given).

    q, k [tokens, G, K] and v [tokens, H, V] share one dtype (bfloat16 or float32)
    and hold the sequences one after another: ``cu_seqlens`` (int32, nseqs + 1) says
    where each begins, or without it they are ``nseqs`` of equal length.  Their rows
    may be slices of a wider tensor's.  log_decay [H] and init_state
    [nseqs, H, V, K] are float32.  ``max_seqlen`` (0: not known) spares the
    preparations for long sequences where there are none (12 prompts of 16384 tokens
    in all, 32 heads of 128 x 128: 154 us with it, 219 without).
    Returns ``(o [tokens, H, V], final_state [nseqs, H, V, K] float32 or None)``.
    """
    lib = _lib or load_library()
    n = _linattn_nseqs(cu_seqlens, nseqs)
    d, qp, kp, vp = _linattn_dims(q, k, v, log_decay, n, max_seqlen)
    T, H, V = v.shape
    K = q.shape[2]
    _typed(init_state, "init_state", torch.float32, (n, H, V, K))
    o = _typed(out, "out", q.dtype, (T, H, V))
    if o is None:
        o = torch.empty((T, H, V), dtype=q.dtype, device=q.device)
    fin = None
    if return_final_state:
        fin = _typed(final_out, "final_out", torch.float32, (n, H, V, K))
        if fin is None:
            fin = torch.empty((n, H, V, K), dtype=torch.float32, device=q.device)
    workspace, nbytes = _linattn_workspace(lib, d, 0, workspace, q.device)
    _check(lib.ssd_linattn_fwd(ctypes.byref(d), qp, kp, vp, _addr(log_decay),
                               K ** -0.5 if scale is None else float(scale), _addr(cu_seqlens),
                               _addr(init_state), _addr(o), _addr(fin), _addr(workspace), nbytes, _stream_int()))
    return o, fin


def linattn_bwd(q, k, v, dout, log_decay, cu_seqlens=None, scale: float = None, init_state=None,
                dfinal_state=None, nseqs: int = 1, max_seqlen: int = 0, workspace=None):
    """The gradient of linattn_fwd from dout [tokens, H, V] and dfinal_state (None: 0).
    Returns ``(dq, dk, dv, dinit_state)``; dinit_state is None without an init_state."""
    lib = _lib or load_library()
    n = _linattn_nseqs(cu_seqlens, nseqs)
    d, qp, kp, vp = _linattn_dims(q, k, v, log_decay, n, max_seqlen)
    T, H, V = v.shape
    K = q.shape[2]
    _typed(dout, "dout", q.dtype, (T, H, V))
    _typed(init_state, "init_state", torch.float32, (n, H, V, K))
    _typed(dfinal_state, "dfinal_state", torch.float32, (n, H, V, K))
    new = lambda shape, dt: torch.empty(shape, dtype=dt, device=q.device)
    dq, dk, dv = new(q.shape, q.dtype), new(k.shape, q.dtype), new(v.shape, q.dtype)
    d0 = None if init_state is None else new((n, H, V, K), torch.float32)
    workspace, nbytes = _linattn_workspace(lib, d, 1, workspace, q.device)
    _check(lib.ssd_linattn_bwd(ctypes.byref(d), qp, kp, vp, _addr(dout), _addr(log_decay),
                               K ** -0.5 if scale is None else float(scale), _addr(cu_seqlens),
                               _addr(init_state), _addr(dfinal_state), _addr(dq), _addr(dk), _addr(dv),
                               _addr(d0), _addr(workspace), nbytes, _stream_int()))
    return dq, dk, dv, d0


def linattn_step(q, k, v, log_decay, cache, slots=None, scale: float = None, out=None):
    """Linear attention for one more token of each row's stream: q, k [b, G, K],
    v [b, H, V]; ``cache`` [nslots, H, V, K] float32 holds the states and is updated
    in place; ``slots`` [b] int32 says which is whose (row b's slot is b without it;
    a negative one marks a row without a stream, whose output is 0).
    Returns o [b, H, V]."""
    lib = _lib or load_library()
    d, qp, kp, vp = _linattn_dims(q, k, v, log_decay, q.shape[0], 0)
    b, H, V = v.shape
    K = q.shape[2]
    _typed(cache, "cache", torch.float32, (cache.shape[0], H, V, K))
    _typed(slots, "slots", torch.int32, (b,))
    o = _typed(out, "out", q.dtype, (b, H, V))
    if o is None:
        o = torch.empty((b, H, V), dtype=q.dtype, device=q.device)
    _check(lib.ssd_linattn_step(ctypes.byref(d), qp, kp, vp, _addr(log_decay),
                                K ** -0.5 if scale is None else float(scale), _addr(slots), _addr(cache),
                                cache.shape[0], _addr(o), _stream_int()))
    return o


def _norm_dims(r, y, z, w_post, alpha, w_pre, gate, ngroups, eps):
    if gate not in GATES:
        raise ValueError(f"gate must be one of {list(GATES)}, got {gate!r}")
    if y.dim() != 2:
        raise ValueError("y must be [tokens, width]")
    T, D = y.shape
    if tuple(r.shape) != (T, D):
        raise ValueError(f"r must be {[T, D]}, got {list(r.shape)}")
    if gate is not None and z is None:
        raise ValueError("a gate needs z")
    _typed(z, "z", y.dtype, (T, D))
    for name, w in (("w_post", w_post), ("alpha", alpha), ("w_pre", w_pre)):
        _typed(w, name, torch.float32, (D,))
    yp, ys = _rows(y, D)
    zp, zs = (None, 0) if z is None or gate is None else _rows(z, D)
    d = NormDims(T, D, int(ngroups), ys, zs, GATES[gate], float(eps), _dtype_code(y, "y"),
                 _dtype_code(r, "r"), 0)
    return d, yp, zp


def block_norm_fwd(r, y, w_pre, z=None, w_post=None, alpha=None, gate=None, ngroups: int = 1,
                   eps: float = 1e-5, return_rstd: bool = False, r_out=None, out=None):
    """The norm after a block (y in ``ngroups`` groups of columns), its gate
    (``"silu"`` or ``"sigmoid"`` of z, or None), the residual scale ``alpha`` and the
    norm before the next block:
    r_out = r + alpha w_post gate(z) rmsnorm(y), n = w_pre rmsnorm(r_out).

    y, z and n [tokens, width] share one dtype; r and r_out may be float32 beside
    bfloat16.  The weights are float32 [width].  Rows of y and z may be slices.
    ``r_out`` may be r.  Returns ``(r_out, n)``, with ``return_rstd`` also the pair
    of factors that block_norm_bwd needs."""
    lib = _lib or load_library()
    d, yp, zp = _norm_dims(r, y, z, w_post, alpha, w_pre, gate, ngroups, eps)
    T, D = y.shape
    ro = _typed(r_out, "r_out", r.dtype, (T, D))
    if ro is None:
        ro = torch.empty((T, D), dtype=r.dtype, device=y.device)
    n = _typed(out, "out", y.dtype, (T, D))
    if n is None:
        n = torch.empty((T, D), dtype=y.dtype, device=y.device)
    rstd = None
    if return_rstd:
        rstd = (torch.empty((T, int(ngroups)), dtype=torch.float32, device=y.device),
                torch.empty((T,), dtype=torch.float32, device=y.device))
    _check(lib.ssd_block_norm_fwd(ctypes.byref(d), _addr(r), yp, zp, _addr(w_post), _addr(alpha),
                                  _addr(w_pre), _addr(ro), _addr(n), _addr(rstd[0]) if rstd else None,
                                  _addr(rstd[1]) if rstd else None, _stream_int()))
    return (ro, n, rstd) if return_rstd else (ro, n)


def block_norm_bwd(r, y, w_pre, dr_out, dn, rstd, z=None, w_post=None, alpha=None, gate=None,
                   ngroups: int = 1, eps: float = 1e-5, workspace=None):
    """The gradient of block_norm_fwd (same inputs, and its ``rstd``) from dr_out and
    dn.  Returns a dict: dr, dy, dz (None without a gate), dw_pre, dw_post and
    dalpha (None where the weight is None)."""
    lib = _lib or load_library()
    d, yp, zp = _norm_dims(r, y, z, w_post, alpha, w_pre, gate, ngroups, eps)
    T, D = y.shape
    _typed(dr_out, "dr_out", r.dtype, (T, D))
    _typed(dn, "dn", y.dtype, (T, D))
    _typed(rstd[0], "rstd[0]", torch.float32, (T, int(ngroups)))
    _typed(rstd[1], "rstd[1]", torch.float32, (T,))
    new = lambda t: torch.empty((T, D), dtype=t.dtype, device=t.device)
    col = lambda w: None if w is None else torch.empty((D,), dtype=torch.float32, device=y.device)
    g = {"dr": new(r), "dy": new(y), "dz": None if gate is None else new(z), "dw_pre": col(w_pre),
         "dw_post": col(w_post), "dalpha": col(alpha)}
    need = int(lib.ssd_block_norm_bwd_workspace_bytes(ctypes.byref(d)))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=y.device)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.ssd_block_norm_bwd(ctypes.byref(d), _addr(r), yp, zp, _addr(w_post), _addr(alpha),
                                  _addr(w_pre), _addr(dr_out), _addr(dn), _addr(rstd[0]), _addr(rstd[1]),
                                  _addr(g["dr"]), _addr(g["dy"]), _addr(g["dz"]), _addr(g["dw_post"]),
                                  _addr(g["dalpha"]), _addr(g["dw_pre"]), _addr(workspace), nbytes,
                                  _stream_int()))
    return g


# The calls below launch on the current device: operands of another one, or of the host,
# are refused where their addresses are taken.
def _here(t, dev):
    """Address of a contiguous tensor on device `dev` (None passes)."""
    if t is None:
        return None
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError("tensors must be contiguous CUDA tensors on the current device")
    return t.data_ptr()


def _at(t, name, dtype, shape, dev):
    """_typed and _here in one: a call's operands are many, and each test costs."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        return _here(_typed(t, name, dtype, shape), dev)
    return t.data_ptr()


def _rows_at(t, name, dtype, shape, inner, dev):
    """_rows, of a tensor of this dtype and shape on device `dev`."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _typed(t, name, dtype, shape)
        raise ValueError("tensors must be CUDA tensors on the current device")
    if t.is_contiguous():
        return t.data_ptr(), inner
    return _rows(t, inner)


def _stream_of(dev) -> int:
    return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream


def _seqs(cu_seqlens, nseqs):
    if cu_seqlens is None:
        return int(nseqs)
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be a 1-D int32 tensor of nseqs + 1 values")
    return cu_seqlens.numel() - 1


def _space(need: int, workspace, device):
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    return workspace, 0 if workspace is None else workspace.numel() * workspace.element_size()


def _out(t, name, dtype, shape, device, dev):
    """The caller's output, checked, or a new one, and its address."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=device)
        return t, t.data_ptr()
    return t, _at(t, name, dtype, shape, dev)


def _ptrs(g):
    """Addresses of new outputs."""
    return (None if t is None else t.data_ptr() for t in g.values())


def _short_conv_dims(x, weight, bias, activation, nseqs, dev):
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x must be [tokens, dim] and weight [dim, width]")
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {list(ACTIVATIONS)}, got {activation!r}")
    T, D = x.shape
    W = weight.shape[1]
    wp, bp = _at(weight, "weight", torch.float32, (D, W), dev), _at(bias, "bias", torch.float32, (D,), dev)
    xp, xs = _rows_at(x, "x", x.dtype, x.shape, D, dev)
    return ShortConvDims(nseqs, T, D, W, xs, act, _dtype_code(x, "x"), 0), T, D, W, (xp, wp, bp)


def short_conv_fwd(x, weight, bias=None, activation=None, cu_seqlens=None, init_state=None,
                   nseqs: int = 1, return_final_state: bool = True, out=None, final_out=None):
    """Depthwise causal convolution over the rows of packed sequences:
    out_t = act(bias + sum_k weight[:, k] x_{t - W + 1 + k}), ``activation`` None or "silu".

    x [tokens, dim] (bfloat16 or float32; its rows may be slices of a wider tensor's) holds
    the sequences one after another: ``cu_seqlens`` (int32, nseqs + 1) says where each
    begins, or without it they are ``nseqs`` of equal length.  weight [dim, W] and bias
    [dim] are float32.  init_state [nseqs, W - 1, dim] in x's dtype holds the rows before
    each sequence, oldest first (0 without it).
    Returns ``(out [tokens, dim], final_state [nseqs, W - 1, dim] or None)``.
    """
    lib = _lib or load_library()
    n = _seqs(cu_seqlens, nseqs)
    dev = torch.cuda.current_device()
    d, T, D, W, args = _short_conv_dims(x, weight, bias, activation, n, dev)
    state = (n, W - 1, D)
    ip = _at(init_state, "init_state", x.dtype, state, dev)
    o, op = _out(out, "out", x.dtype, (T, D), x.device, dev)
    fin, fp = _out(final_out, "final_out", x.dtype, state, x.device, dev) if return_final_state else (None, None)
    _check(lib.ssd_short_conv_fwd(ctypes.byref(d), *args, _here(cu_seqlens, dev), ip, op, fp, _stream_of(dev)))
    return o, fin


def short_conv_bwd(x, weight, dout, bias=None, activation=None, cu_seqlens=None, init_state=None,
                   dfinal_state=None, nseqs: int = 1, workspace=None):
    """The gradient of short_conv_fwd from dout [tokens, dim] and dfinal_state (None: 0).
    Returns a dict: dx, dweight, dbias (None without a bias) and dinit_state (None without
    an init_state)."""
    lib = _lib or load_library()
    n = _seqs(cu_seqlens, nseqs)
    dev = torch.cuda.current_device()
    d, T, D, W, args = _short_conv_dims(x, weight, bias, activation, n, dev)
    state = (n, W - 1, D)
    ip = _at(init_state, "init_state", x.dtype, state, dev)
    gp, fp = _at(dout, "dout", x.dtype, (T, D), dev), _at(dfinal_state, "dfinal_state", x.dtype, state, dev)
    new = lambda shape, dt: torch.empty(shape, dtype=dt, device=x.device)
    g = {"dx": new((T, D), x.dtype), "dweight": new((D, W), torch.float32),
         "dbias": None if bias is None else new((D,), torch.float32),
         "dinit_state": None if init_state is None else new(state, x.dtype)}
    workspace, nbytes = _space(lib.ssd_short_conv_bwd_workspace_bytes(ctypes.byref(d)), workspace, x.device)
    _check(lib.ssd_short_conv_bwd(ctypes.byref(d), *args, _here(cu_seqlens, dev), ip, gp, fp, *_ptrs(g),
                                  _here(workspace, dev), nbytes, _stream_of(dev)))
    return g


def short_conv_step(x, weight, cache, bias=None, activation=None, slots=None, out=None):
    """The same convolution for one more token of each row's stream: x [b, dim]; ``cache``
    [nslots, W - 1, dim] in x's dtype holds each stream's last rows (short_conv_fwd's final
    states) and is moved up by one in place; ``slots`` [b] int32 says which is whose (row
    b's slot is b without it; a negative one marks a row without a stream, whose output is
    0; no slot may occur twice).  Returns out [b, dim]."""
    lib = _lib or load_library()
    dev = torch.cuda.current_device()
    d, b, D, W, args = _short_conv_dims(x, weight, bias, activation, x.shape[0], dev)
    n = cache.shape[0]
    cp, sp = _at(cache, "cache", x.dtype, (n, W - 1, D), dev), _at(slots, "slots", torch.int32, (b,), dev)
    o, op = _out(out, "out", x.dtype, (b, D), x.device, dev)
    _check(lib.ssd_short_conv_step(ctypes.byref(d), *args, sp, cp, n, op, _stream_of(dev)))
    return o


def _selscan_dims(x, dt, A, B, C, D, z, dt_bias, dt_softplus, nseqs, max_seqlen, dev):
    if x.dim() != 2 or A.dim() != 2 or B.dim() != 3:
        raise ValueError("x must be [tokens, dim], A [dim, N], B and C [tokens, G, N]")
    T, W = x.shape
    N, G = A.shape[1], B.shape[1]
    kind, rows, mix, f32 = x.dtype, (T, W), (T, G, N), torch.float32
    xp, xs = _rows_at(x, "x", kind, rows, W, dev)
    tp, ts = _rows_at(dt, "dt", kind, rows, W, dev)
    zp, zs = (None, 0) if z is None else _rows_at(z, "z", kind, rows, W, dev)
    Bp, Bs = _rows_at(B, "B", kind, mix, G * N, dev)
    Cp, Cs = _rows_at(C, "C", kind, mix, G * N, dev)
    Ap, Dp, bp = _at(A, "A", f32, (W, N), dev), _at(D, "D", f32, (W,), dev), _at(dt_bias, "dt_bias", f32, (W,), dev)
    d = SelscanDims(nseqs, T, W, N, G, xs, ts, zs, Bs, Cs, max_seqlen, 1 if dt_softplus else 0,
                    _dtype_code(x, "x"), 0)
    return d, T, W, N, (xp, tp, Ap, Bp, Cp, Dp, zp, bp)


def selscan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus: bool = False,
                cu_seqlens=None, init_state=None, nseqs: int = 1, max_seqlen: int = 0,
                return_final_state: bool = True, return_states: bool = False, workspace=None,
                out=None, final_out=None):
    """The selective state space scan: with delta = softplus(dt + dt_bias) (or dt + dt_bias),
    h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t and y_t = (C_t . h_t + D x_t) silu(z_t),
    with N states and decays for each channel.

    x, dt, z [tokens, dim] and B, C [tokens, G, N] share one dtype (bfloat16 or float32) and
    hold the sequences one after another: ``cu_seqlens`` (int32, nseqs + 1) says where each
    begins, or without it they are ``nseqs`` of equal length.  Channel d reads group
    d // (dim // G) of B and C.  Rows may be slices of a wider tensor's; those of B and C
    need no alignment.  A [dim, N], D, dt_bias [dim] and init_state [nseqs, dim, N] are
    float32; D, z and dt_bias may be None.  ``max_seqlen`` (0: not known) spares the
    preparations for long sequences where there are none: without it any sequence may be as
    long as all of the tokens (12 prompts of 16384 tokens in all, 5120 channels: 627 us
    instead of 447).
    Returns ``(y [tokens, dim], final_state [nseqs, dim, N] float32 or None)``, with
    ``return_states`` also the states on the way that selscan_bwd needs,
    [tokens // SELSCAN_CHUNK + nseqs, dim, N] float32.
    """
    lib = _lib or load_library()
    n = _seqs(cu_seqlens, nseqs)
    dev = torch.cuda.current_device()
    d, T, W, N, args = _selscan_dims(x, dt, A, B, C, D, z, dt_bias, dt_softplus, n, max_seqlen, dev)
    state = (n, W, N)
    ip = _at(init_state, "init_state", torch.float32, state, dev)
    y, yp = _out(out, "out", x.dtype, (T, W), x.device, dev)
    fin, fp = _out(final_out, "final_out", torch.float32, state, x.device, dev) if return_final_state else (None, None)
    states = torch.empty((T // SELSCAN_CHUNK + n, W, N), dtype=torch.float32, device=x.device) if return_states else None
    workspace, nbytes = _space(lib.ssd_selscan_workspace_bytes(ctypes.byref(d), 0), workspace, x.device)
    _check(lib.ssd_selscan_fwd(ctypes.byref(d), *args, _here(cu_seqlens, dev), ip, yp, fp, _here(states, dev),
                               _here(workspace, dev), nbytes, _stream_of(dev)))
    return (y, fin, states) if return_states else (y, fin)


def selscan_bwd(x, dt, A, B, C, dout, states, D=None, z=None, dt_bias=None, dt_softplus: bool = False,
                cu_seqlens=None, dfinal_state=None, nseqs: int = 1, max_seqlen: int = 0,
                return_dinit: bool = False, workspace=None):
    """The gradient of selscan_fwd (same inputs, and its ``states``) from dout [tokens, dim] and
    dfinal_state (None: 0).  Returns a dict: dx, ddt, dA, dB, dC, dD, dz and ddt_bias (each None
    where the input is None) and dinit_state (None unless ``return_dinit``)."""
    lib = _lib or load_library()
    n = _seqs(cu_seqlens, nseqs)
    dev = torch.cuda.current_device()
    d, T, W, N, args = _selscan_dims(x, dt, A, B, C, D, z, dt_bias, dt_softplus, n, max_seqlen, dev)
    sp = _at(states, "states", torch.float32, (T // SELSCAN_CHUNK + n, W, N), dev)
    gp, fp = _at(dout, "dout", x.dtype, (T, W), dev), _at(dfinal_state, "dfinal_state", torch.float32, (n, W, N), dev)
    like = lambda t: None if t is None else torch.empty(t.shape, dtype=t.dtype, device=x.device)
    g = {"dx": like(x), "ddt": like(dt), "dA": like(A), "dB": like(B), "dC": like(C), "dD": like(D), "dz": like(z),
         "ddt_bias": like(dt_bias),
         "dinit_state": torch.empty((n, W, N), dtype=torch.float32, device=x.device) if return_dinit else None}
    workspace, nbytes = _space(lib.ssd_selscan_workspace_bytes(ctypes.byref(d), 1), workspace, x.device)
    _check(lib.ssd_selscan_bwd(ctypes.byref(d), *args, _here(cu_seqlens, dev), sp, gp, fp, *_ptrs(g),
                               _here(workspace, dev), nbytes, _stream_of(dev)))
    return g


def selscan_step(x, dt, A, B, C, cache, D=None, z=None, dt_bias=None, dt_softplus: bool = False,
                 slots=None, out=None):
    """The selective scan for one more token of each row's stream: x, dt, z [b, dim],
    B, C [b, G, N]; ``cache`` [nslots, dim, N] float32 holds the states and is updated in
    place; ``slots`` as for short_conv_step.  Returns y [b, dim]."""
    lib = _lib or load_library()
    dev = torch.cuda.current_device()
    d, b, W, N, args = _selscan_dims(x, dt, A, B, C, D, z, dt_bias, dt_softplus, x.shape[0], 0, dev)
    n = cache.shape[0]
    cp, sp = _at(cache, "cache", torch.float32, (n, W, N), dev), _at(slots, "slots", torch.int32, (b,), dev)
    y, yp = _out(out, "out", x.dtype, (b, W), x.device, dev)
    _check(lib.ssd_selscan_step(ctypes.byref(d), *args, sp, cp, n, yp, _stream_of(dev)))
    return y
