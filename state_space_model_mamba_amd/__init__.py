"""Python binding of libssd, the MI355X (gfx950) Mamba-2 SSD prefill scan and
O(1) cached decode step.

Argument marshalling only: every step of the computation runs in the HIP
kernels of ``libssd.so`` (C ABI in ``include/ssd.h``).  PyTorch provides device
memory and the stream.  There is no fallback: if the library is missing, or a
call fails, an exception is raised.

Functions keep the C names (each call also takes dt_softplus=True, dt_bias=[H]
to pass u instead of dt; the step size is then softplus(u + dt_bias) in the kernels):
    ssd_state_init(state, src=None)
    ssd_chunk_scan_workspace_size(...)
    ssd_chunk_scan(x, dt, A, B, C, D, chunk, initial_state=None, ...) -> (y, final_state)
    ssd_decode_step(x, dt, A, B, C, D, state, y=None) -> y
    ssd_decode_steps(x, dt, A, B, C, D, state, y=None) -> y   (S steps in one launch)
    ssd_chunk_scan_timed(...) -> (y, final_state, [(kernel, ms), ...])
    ssd_chunk_scan_noalloc(x, dt, A, B, C, D, chunk, ...) -> (y, final_state)  (no workspace)
    ssd_chunk_scan_varlen(x, dt, A, B, C, D, cu_seqlens, chunk, ...) -> (y, final_states)
    ssd_gdn_decode_step(q, k, v, g, beta, state, o=None) -> o   (Gated DeltaNet step)
    ssd_gdn_decode_steps(q, k, v, g, beta, state, o=None) -> o  (S steps in one launch)
and the attention layers of hybrid stacks:
    ssd_linattn_chunk_scan(q, k, v, log_decay, initial_state=None, ...) -> (o, final_state)
    ssd_linattn_chunk_scan_varlen(q, k, v, log_decay, cu_seqlens, ...) -> (o, final_states)
    ssd_linattn_decode_step(q, k, v, log_decay, state, o=None) -> o
    ssd_attn_prefill(q, k, v, cu_seqlens, kv_starts=None, kv_lens=None, ...) -> o
    ssd_attn_decode_step(q, k, v, k_cache, v_cache, lengths, ...) -> o  (cache appended in place)
with the norm and rotation of the latter's queries and keys, and a paged cache of its own:
    ssd_attn_qk_norm_rope(q, k, positions, inv_freq=None, q_weight=None, ...) -> (q_out, k_out)
    ssd_attn_paged_append(q, k, v, k_pages, v_pages, block_table, lengths, ...) -> q_out
    ssd_attn_paged_gather(k_pages, v_pages, block_table, cu_seqlens, ...) -> (k, v)
    ssd_attn_paged_decode_step(q, k_pages, v_pages, block_table, lengths, ...) -> o
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(PKG, "libssd.so")

SSD_F32, SSD_BF16 = 0, 1
SSD_PAGES_IO, SSD_PAGES_4BIT = 0, 1
SSD_DT_SOFTPLUS = 1            # ssd_dims.flags: dt holds u, the step size is softplus(u + dt_bias)
STATUS = {0: "SSD_OK", 1: "SSD_ERR_NULL", 2: "SSD_ERR_SHAPE", 3: "SSD_ERR_UNSUPPORTED",
          4: "SSD_ERR_ALIAS", 5: "SSD_ERR_WORKSPACE", 6: "SSD_ERR_DEVICE", 7: "SSD_ERR_ALIGNMENT"}
EXPORTS = ("ssd_status_string", "ssd_version", "ssd_state_init", "ssd_chunk_scan_workspace_size",
           "ssd_chunk_scan", "ssd_decode_step", "ssd_decode_steps", "ssd_chunk_scan_timed",
           "ssd_chunk_scan_varlen_workspace_size", "ssd_chunk_scan_varlen",
           "ssd_gdn_decode_step", "ssd_gdn_decode_steps", "ssd_chunk_scan_noalloc",
           "ssd_linattn_chunk_scan_workspace_size", "ssd_linattn_chunk_scan",
           "ssd_linattn_chunk_scan_varlen_workspace_size", "ssd_linattn_chunk_scan_varlen",
           "ssd_linattn_decode_step", "ssd_attn_prefill", "ssd_attn_decode_workspace_size",
           "ssd_attn_decode_step", "ssd_attn_qk_norm_rope", "ssd_attn_paged_append",
           "ssd_attn_paged_gather", "ssd_attn_paged_decode_workspace_size",
           "ssd_attn_paged_decode_step")
NOALLOC_SCRATCH_BYTES = 96 << 20   # SSD_NOALLOC_SCRATCH_BYTES of include/ssd.h


class SsdError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} failed: {msg}")
        self.code = code


class SsdDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("nheads", ctypes.c_int64), ("headdim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("chunk", ctypes.c_int64), ("io_dtype", ctypes.c_int32),
                ("flags", ctypes.c_int32), ("dt_bias", ctypes.c_void_p)]


class SsdGdnDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("qk_heads", ctypes.c_int64),
                ("v_heads", ctypes.c_int64), ("dk", ctypes.c_int64), ("dv", ctypes.c_int64),
                ("io_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_lib = None


def load(path: str | None = None):
    """Load libssd.so (built in-tree by ``state_space_model_mamba_amd.build``)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIBRARY
    if not os.path.exists(p):
        raise RuntimeError(f"libssd not built: {p} is missing "
                           "(run `python -m state_space_model_mamba_amd.build`)")
    lib = ctypes.CDLL(p)
    vp, fp, i64p = ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t)
    dims = ctypes.POINTER(SsdDims)
    lib.ssd_status_string.argtypes = [ctypes.c_int]
    lib.ssd_status_string.restype = ctypes.c_char_p
    lib.ssd_version.argtypes = []
    lib.ssd_version.restype = ctypes.c_int
    lib.ssd_state_init.argtypes = [dims, fp, fp, vp]
    lib.ssd_state_init.restype = ctypes.c_int
    lib.ssd_chunk_scan_workspace_size.argtypes = [dims, i64p]
    lib.ssd_chunk_scan_workspace_size.restype = ctypes.c_int
    lib.ssd_chunk_scan.argtypes = [dims] + [vp] * 10 + [ctypes.c_size_t, vp]
    lib.ssd_chunk_scan.restype = ctypes.c_int
    lib.ssd_chunk_scan_timed.argtypes = ([dims] + [vp] * 10 + [ctypes.c_size_t, vp] +
                                         [ctypes.POINTER(ctypes.c_float),
                                          ctypes.POINTER(ctypes.c_char_p),
                                          ctypes.POINTER(ctypes.c_int)])
    lib.ssd_chunk_scan_timed.restype = ctypes.c_int
    lib.ssd_chunk_scan_noalloc.argtypes = [dims] + [vp] * 10
    lib.ssd_chunk_scan_noalloc.restype = ctypes.c_int
    lib.ssd_decode_step.argtypes = [dims] + [vp] * 9
    lib.ssd_decode_step.restype = ctypes.c_int
    lib.ssd_decode_steps.argtypes = [dims, ctypes.c_int64] + [vp] * 9
    lib.ssd_decode_steps.restype = ctypes.c_int
    cu = ctypes.POINTER(ctypes.c_int64)
    lib.ssd_chunk_scan_varlen_workspace_size.argtypes = [dims, cu, i64p]
    lib.ssd_chunk_scan_varlen_workspace_size.restype = ctypes.c_int
    lib.ssd_chunk_scan_varlen.argtypes = [dims, cu] + [vp] * 10 + [ctypes.c_size_t, vp]
    lib.ssd_chunk_scan_varlen.restype = ctypes.c_int
    lib.ssd_gdn_decode_step.argtypes = [ctypes.POINTER(SsdGdnDims)] + [vp] * 8
    lib.ssd_gdn_decode_step.restype = ctypes.c_int
    lib.ssd_gdn_decode_steps.argtypes = [ctypes.POINTER(SsdGdnDims), ctypes.c_int64] + [vp] * 8
    lib.ssd_gdn_decode_steps.restype = ctypes.c_int
    lin, att, sz = ctypes.POINTER(SsdLinattnDims), ctypes.POINTER(SsdAttnDims), ctypes.c_size_t
    pag, rope = ctypes.POINTER(SsdPagedDims), ctypes.POINTER(SsdQkRope)
    for name, args in (
            ("ssd_linattn_chunk_scan_workspace_size", [lin, i64p]),
            ("ssd_linattn_chunk_scan", [lin] + [vp] * 8 + [sz, vp]),
            ("ssd_linattn_chunk_scan_varlen_workspace_size", [lin, cu, i64p]),
            ("ssd_linattn_chunk_scan_varlen", [lin, cu] + [vp] * 8 + [sz, vp]),
            ("ssd_linattn_decode_step", [lin] + [vp] * 7),
            ("ssd_attn_prefill", [att] + [cu] * 3 + [vp] * 5),
            ("ssd_attn_decode_workspace_size", [att, i64p]),
            ("ssd_attn_decode_step", [att] + [vp] * 8 + [sz, vp]),
            ("ssd_attn_qk_norm_rope", [pag, rope] + [vp] * 5),
            ("ssd_attn_paged_append", [pag, rope] + [vp] * 13),
            ("ssd_attn_paged_gather", [pag] + [vp] * 10),
            ("ssd_attn_paged_decode_workspace_size", [pag, i64p]),
            ("ssd_attn_paged_decode_step", [pag] + [vp] * 9 + [sz, vp])):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = ctypes.c_int
    if path is None:
        _lib = lib
    return lib


def _check(fn: str, rc: int):
    if rc != 0:
        msg = load().ssd_status_string(rc).decode()
        raise SsdError(fn, rc, msg)


def _ptr(t):
    """A tensor's device address as an int (ctypes passes it as void*), or NULL."""
    return None if t is None else t.data_ptr()


def _current_raw_stream(di):
    """The current stream's handle on device `di`, without building a Stream object."""
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return get(di) if get is not None else torch.cuda.current_stream(di).cuda_stream


def _stream(stream, di):
    """hipStream_t of `stream`, or of device `di`'s current stream."""
    return _current_raw_stream(di) if stream is None else stream.cuda_stream


_HERE = contextlib.nullcontext()   # (holds nothing: one for all calls)


def _on(stream):
    """Allocation context of a call: the caller's stream when one is given (the
    current stream is the allocator's default otherwise), so that blocks
    allocated for the call are not handed to other work while its kernels run."""
    return _HERE if stream is None else torch.cuda.stream(stream)


def _io_dtype(t, names="x/B/C"):
    if t.dtype == torch.bfloat16:
        return SSD_BF16
    if t.dtype == torch.float32:
        return SSD_F32
    raise TypeError(f"{names} must be bfloat16 or float32, got {t.dtype}")


def _need(name, t, di, dtype=None, shape=None, optional=False):
    """Checks that a tensor argument can be handed to the kernels as a plain
    device pointer: a contiguous tensor on GPU `di` of the stated dtype and
    shape.  A host tensor would hand a host address to a kernel, and a strided
    view or a wrong dtype would be read as something else, so each raises here
    instead.  (One combined test on the common path: small decode calls are
    bound by host time.)"""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    try:
        ok = (t.get_device() == di and (dtype is None or t.dtype == dtype) and t.is_contiguous()
              and (shape is None or t.shape == shape))
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}") from None
    if not ok:
        if t.get_device() != di:
            raise ValueError(f"{name} is on {t.device}, expected cuda:{di}")
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _device_of(t):
    """The device index of the first tensor argument, which must be a GPU tensor."""
    di = t.get_device()
    if di < 0:
        raise ValueError(f"arguments must be device (HIP) tensors, got one on {t.device}")
    return di


def _bias_check(di, H, dt_softplus, dt_bias):
    if dt_softplus:
        _need("dt_bias", dt_bias, di, torch.float32, (H,), optional=True)


def make_dims(batch, seqlen, nheads, headdim, dstate, ngroups, chunk, io_dtype,
              dt_softplus=False, dt_bias=None) -> SsdDims:
    """ssd_dims; with dt_softplus the dt arguments hold u and the step size is
    softplus(u + dt_bias[h]) (dt_bias: a [H] fp32 device tensor or None)."""
    flags = SSD_DT_SOFTPLUS if dt_softplus else 0
    bias = dt_bias.data_ptr() if (dt_softplus and dt_bias is not None) else None
    return SsdDims(batch, seqlen, nheads, headdim, dstate, ngroups, chunk, io_dtype, flags, bias)


def ssd_chunk_scan_workspace_size(batch, seqlen, nheads, headdim, dstate, ngroups, chunk,
                                  io_dtype=SSD_BF16) -> int:
    d = make_dims(batch, seqlen, nheads, headdim, dstate, ngroups, chunk, io_dtype)
    n = ctypes.c_size_t(0)
    _check("ssd_chunk_scan_workspace_size",
           load().ssd_chunk_scan_workspace_size(ctypes.byref(d), ctypes.byref(n)))
    return int(n.value)


def ssd_state_init(state, src=None, stream=None):
    """state [B, H, P, N] fp32 <- src (or zeros)."""
    dev = _device_of(state)
    _need("state", state, dev, torch.float32)
    if state.dim() != 4:
        raise ValueError(f"state must be [B, H, P, N], got shape {tuple(state.shape)}")
    b, h, p, n = state.shape
    _need("src", src, dev, torch.float32, state.shape, optional=True)
    d = make_dims(b, 0, h, p, n, 1, 1, SSD_F32)
    _check("ssd_state_init", load().ssd_state_init(ctypes.byref(d), _ptr(state), _ptr(src),
                                                   _stream(stream, dev)))
    return state


def _scan_args(x, dt, A, B, C, D, chunk, initial_state, y, final_state, workspace,
               dt_softplus=False, dt_bias=None, stream=None, need_workspace=True):
    dev = _device_of(x)
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be [B, L, H, P] and B, C [B, L, G, N]")
    bsz, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    io = _io_dtype(x)
    f32 = torch.float32
    _need("x", x, dev, x.dtype)
    _need("dt", dt, dev, f32, (bsz, L, H))
    _need("A", A, dev, f32, (H,))
    _need("B", B, dev, x.dtype, (bsz, L, G, N))
    _need("C", C, dev, x.dtype, (bsz, L, G, N))
    _need("D", D, dev, f32, (H,))
    _need("initial_state", initial_state, dev, f32, (bsz, H, P, N), optional=True)
    _need("y", y, dev, x.dtype, x.shape, optional=True)
    _need("final_state", final_state, dev, f32, (bsz, H, P, N), optional=True)
    _need("workspace", workspace, dev, optional=True)
    _bias_check(dev, H, dt_softplus, dt_bias)
    d = make_dims(bsz, L, H, P, N, G, chunk, io, dt_softplus, dt_bias)
    need = ssd_chunk_scan_workspace_size(bsz, L, H, P, N, G, chunk, io) if need_workspace else 0
    # outputs and workspace come from the allocator on the call's own stream, so
    # that their blocks are not handed to other work while the kernels run
    with _on(stream):
        if y is None:
            y = torch.empty_like(x)
        if final_state is None:
            final_state = torch.empty((bsz, H, P, N), dtype=f32, device=dev)
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = [ctypes.byref(d), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
            _ptr(initial_state), _ptr(y), _ptr(final_state), _ptr(workspace), ws_bytes]
    return args, y, final_state, workspace


def ssd_chunk_scan(x, dt, A, B, C, D, chunk, initial_state=None, y=None, final_state=None,
                   workspace=None, stream=None, dt_softplus=False, dt_bias=None):
    """Prefill over x[B, L, H, P]; returns (y, final_state)."""
    args, y, fs, ws = _scan_args(x, dt, A, B, C, D, chunk, initial_state, y, final_state,
                                 workspace, dt_softplus, dt_bias, stream)
    _check("ssd_chunk_scan", load().ssd_chunk_scan(*args, _stream(stream, x.get_device())))
    return y, fs


def ssd_chunk_scan_noalloc(x, dt, A, B, C, D, chunk, initial_state=None, y=None,
                           final_state=None, stream=None, dt_softplus=False, dt_bias=None):
    """ssd_chunk_scan with the library's own per-device scratch array as its
    workspace (nothing is allocated by the library; pass y and final_state to
    allocate nothing here either).  Calls that overlap in time on one device
    race on the scratch array.  Returns (y, final_state)."""
    args, y, fs, _ = _scan_args(x, dt, A, B, C, D, chunk, initial_state, y, final_state, None,
                                dt_softplus, dt_bias, stream, need_workspace=False)
    _check("ssd_chunk_scan_noalloc",
           load().ssd_chunk_scan_noalloc(*args[:10], _stream(stream, x.get_device())))
    return y, fs


def ssd_chunk_scan_timed(x, dt, A, B, C, D, chunk, initial_state=None, y=None, final_state=None,
                         workspace=None, stream=None, dt_softplus=False, dt_bias=None):
    """As ssd_chunk_scan, synchronously, also returning [(kernel name, ms), ...]."""
    args, y, fs, ws = _scan_args(x, dt, A, B, C, D, chunk, initial_state, y, final_state,
                                 workspace, dt_softplus, dt_bias, stream)
    cap = 8
    ms = (ctypes.c_float * cap)()
    names = (ctypes.c_char_p * cap)()
    n = ctypes.c_int(cap)
    _check("ssd_chunk_scan_timed", load().ssd_chunk_scan_timed(
        *args, _stream(stream, x.get_device()), ms, names, ctypes.byref(n)))
    return y, fs, [(names[i].decode(), float(ms[i])) for i in range(n.value)]


def ssd_decode_step(x, dt, A, B, C, D, state, y=None, stream=None, dt_softplus=False,
                    dt_bias=None):
    """One decode step: x[B, H, P], B/C[B, G, N], state[B, H, P, N] updated in place; returns y."""
    dev = _device_of(x)
    if x.dim() != 3 or B.dim() != 3:
        raise ValueError("x must be [B, H, P] and B, C [B, G, N]")
    bsz, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    f32 = torch.float32
    _need("x", x, dev, x.dtype)
    _need("dt", dt, dev, f32, (bsz, H))
    _need("A", A, dev, f32, (H,))
    _need("B", B, dev, x.dtype, (bsz, G, N))
    _need("C", C, dev, x.dtype, (bsz, G, N))
    _need("D", D, dev, f32, (H,))
    _need("state", state, dev, f32, (bsz, H, P, N))
    _need("y", y, dev, x.dtype, x.shape, optional=True)
    _bias_check(dev, H, dt_softplus, dt_bias)
    d = make_dims(bsz, 1, H, P, N, G, 1, _io_dtype(x), dt_softplus, dt_bias)
    if y is None:
        with _on(stream):
            y = torch.empty_like(x)
    _check("ssd_decode_step", load().ssd_decode_step(
        ctypes.byref(d), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(state),
        _ptr(y), _stream(stream, dev)))
    return y


def ssd_decode_steps(x, dt, A, B, C, D, state, y=None, stream=None, dt_softplus=False,
                     dt_bias=None):
    """S decode steps in one launch: x[S, B, H, P], dt[S, B, H], B/C[S, B, G, N];
    state[B, H, P, N] updated in place (read and written once); returns y[S, B, H, P]."""
    dev = _device_of(x)
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be [S, B, H, P] and B, C [S, B, G, N]")
    nsteps, bsz, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    f32 = torch.float32
    _need("x", x, dev, x.dtype)
    _need("dt", dt, dev, f32, (nsteps, bsz, H))
    _need("A", A, dev, f32, (H,))
    _need("B", B, dev, x.dtype, (nsteps, bsz, G, N))
    _need("C", C, dev, x.dtype, (nsteps, bsz, G, N))
    _need("D", D, dev, f32, (H,))
    _need("state", state, dev, f32, (bsz, H, P, N))
    _need("y", y, dev, x.dtype, x.shape, optional=True)
    _bias_check(dev, H, dt_softplus, dt_bias)
    d = make_dims(bsz, 1, H, P, N, G, 1, _io_dtype(x), dt_softplus, dt_bias)
    if y is None:
        with _on(stream):
            y = torch.empty_like(x)
    _check("ssd_decode_steps", load().ssd_decode_steps(
        ctypes.byref(d), ctypes.c_int64(nsteps), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C),
        _ptr(D), _ptr(state), _ptr(y), _stream(stream, dev)))
    return y


def _cu_array(cu_seqlens):
    import numpy as np
    cu = np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int64))
    return cu, cu.ctypes.data_as(ctypes.POINTER(ctypes.c_int64))


def ssd_chunk_scan_varlen_workspace_size(cu_seqlens, nheads, headdim, dstate, ngroups, chunk,
                                         io_dtype=SSD_BF16) -> int:
    cu, cup = _cu_array(cu_seqlens)
    d = make_dims(len(cu) - 1, int(cu[-1]), nheads, headdim, dstate, ngroups, chunk, io_dtype)
    n = ctypes.c_size_t(0)
    _check("ssd_chunk_scan_varlen_workspace_size",
           load().ssd_chunk_scan_varlen_workspace_size(ctypes.byref(d), cup, ctypes.byref(n)))
    return int(n.value)


def ssd_chunk_scan_varlen(x, dt, A, B, C, D, cu_seqlens, chunk, initial_states=None, y=None,
                          final_states=None, workspace=None, stream=None, dt_softplus=False,
                          dt_bias=None):
    """Prefill of a packed batch: x[T, H, P], dt[T, H], B/C[T, G, N]; sequence i is
    tokens cu_seqlens[i] .. cu_seqlens[i+1]-1 (a host sequence of S + 1 offsets).
    Returns (y[T, H, P], final_states[S, H, P, N])."""
    dev = _device_of(x)
    if x.dim() != 3 or B.dim() != 3:
        raise ValueError("x must be [T, H, P] and B, C [T, G, N]")
    T, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    cu, cup = _cu_array(cu_seqlens)
    nseq = len(cu) - 1
    io = _io_dtype(x)
    f32 = torch.float32
    _need("x", x, dev, x.dtype)
    _need("dt", dt, dev, f32, (T, H))
    _need("A", A, dev, f32, (H,))
    _need("B", B, dev, x.dtype, (T, G, N))
    _need("C", C, dev, x.dtype, (T, G, N))
    _need("D", D, dev, f32, (H,))
    _need("initial_states", initial_states, dev, f32, (nseq, H, P, N), optional=True)
    _need("y", y, dev, x.dtype, x.shape, optional=True)
    _need("final_states", final_states, dev, f32, (nseq, H, P, N), optional=True)
    _need("workspace", workspace, dev, optional=True)
    _bias_check(dev, H, dt_softplus, dt_bias)
    d = make_dims(nseq, T, H, P, N, G, chunk, io, dt_softplus, dt_bias)
    need = ssd_chunk_scan_varlen_workspace_size(cu, H, P, N, G, chunk, io)
    with _on(stream):
        if y is None:
            y = torch.empty_like(x)
        if final_states is None:
            final_states = torch.empty((nseq, H, P, N), dtype=f32, device=dev)
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("ssd_chunk_scan_varlen", load().ssd_chunk_scan_varlen(
        ctypes.byref(d), cup, _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
        _ptr(initial_states), _ptr(y), _ptr(final_states), _ptr(workspace), ws_bytes,
        _stream(stream, dev)))
    return y, final_states


def ssd_gdn_decode_step(q, k, v, g, beta, state, o=None, stream=None):
    """One Gated DeltaNet decode step: q, k [B, Hk, dk], v [B, Hv, dv], g, beta [B, Hv]
    fp32, state [B, Hv, dk, dv] fp32 updated in place; returns o [B, Hv, dv]."""
    dev = _device_of(q)
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k must be [B, Hk, dk] and v [B, Hv, dv]")
    bsz, Hk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    f32 = torch.float32
    _need("q", q, dev, q.dtype)
    _need("k", k, dev, q.dtype, q.shape)
    _need("v", v, dev, q.dtype)
    _need("g", g, dev, f32, (bsz, Hv))
    _need("beta", beta, dev, f32, (bsz, Hv))
    _need("state", state, dev, f32, (bsz, Hv, dk, dv))
    _need("o", o, dev, q.dtype, v.shape, optional=True)
    d = SsdGdnDims(bsz, Hk, Hv, dk, dv, _io_dtype(q, "q/k/v"), 0)
    if o is None:
        with _on(stream):
            o = torch.empty_like(v)
    _check("ssd_gdn_decode_step", load().ssd_gdn_decode_step(
        ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state), _ptr(o),
        _stream(stream, dev)))
    return o


def ssd_gdn_decode_steps(q, k, v, g, beta, state, o=None, stream=None):
    """S Gated DeltaNet steps in one launch: q, k [S, B, Hk, dk], v [S, B, Hv, dv],
    g, beta [S, B, Hv]; state [B, Hv, dk, dv] read and written once; returns o [S, B, Hv, dv]."""
    dev = _device_of(q)
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k must be [S, B, Hk, dk] and v [S, B, Hv, dv]")
    nsteps, bsz, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    f32 = torch.float32
    _need("q", q, dev, q.dtype)
    _need("k", k, dev, q.dtype, q.shape)
    _need("v", v, dev, q.dtype)
    _need("g", g, dev, f32, (nsteps, bsz, Hv))
    _need("beta", beta, dev, f32, (nsteps, bsz, Hv))
    _need("state", state, dev, f32, (bsz, Hv, dk, dv))
    _need("o", o, dev, q.dtype, v.shape, optional=True)
    d = SsdGdnDims(bsz, Hk, Hv, dk, dv, _io_dtype(q, "q/k/v"), 0)
    if o is None:
        with _on(stream):
            o = torch.empty_like(v)
    _check("ssd_gdn_decode_steps", load().ssd_gdn_decode_steps(
        ctypes.byref(d), ctypes.c_int64(nsteps), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
        _ptr(state), _ptr(o), _stream(stream, dev)))
    return o


# --------------------------------------------------------------------------
# Linear attention and softmax attention
# --------------------------------------------------------------------------
class SsdLinattnDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("qk_heads", ctypes.c_int64), ("v_heads", ctypes.c_int64),
                ("dk", ctypes.c_int64), ("dv", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("scale", ctypes.c_float),
                ("io_dtype", ctypes.c_int32)]


class SsdAttnDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("q_rows", ctypes.c_int64),
                ("kv_rows", ctypes.c_int64), ("q_heads", ctypes.c_int64),
                ("kv_heads", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("scale", ctypes.c_float),
                ("io_dtype", ctypes.c_int32)]


def _offsets(name, x, n=None):
    """A host sequence of offsets or lengths as int64: (array, pointer)."""
    a, p = _cu_array(x)
    if a.ndim != 1 or (len(a) < 1 if n is None else len(a) != n):
        raise ValueError(f"{name} must hold " + ("S + 1 offsets" if n is None else "one entry per sequence"))
    return a, p


# (the plain query: the tensors at hand have initialised the device)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _guard(di):
    """The tensors' device as the current one for a call's launches."""
    return _HERE if _current_device() == di else torch.cuda.device(di)


def _row_stride(name, t, di, dtype, shape):
    """Checks a [tokens.., heads, dim] argument whose tokens may lie further apart
    than its heads need (a slice of one projection), and returns the distance
    between tokens in elements."""
    width = shape[-1] * shape[-2]
    try:
        ok = t.get_device() == di and t.dtype == dtype and t.shape == shape
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}") from None
    if ok and t.is_contiguous():
        return width
    if not ok:
        if t.get_device() != di:
            raise ValueError(f"{name} is on {t.device}, expected cuda:{di}")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    st = t.stride()
    if st[-1] != 1 or (shape[-2] > 1 and st[-2] != shape[-1]):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    row = width
    if len(shape) == 4 and shape[0] > 1 and shape[1] > 1:
        row = st[1]
        if st[0] != shape[1] * row:
            raise ValueError(f"{name}: consecutive tokens must lie evenly spaced over the batch")
    elif len(shape) == 4:
        row = st[1] if shape[1] > 1 else st[0] if shape[0] > 1 else width
    elif shape[0] > 1:
        row = st[0]
    if row < width:
        raise ValueError(f"{name}: tokens overlap")
    return row


def _empty_rows(t):
    """An uninitialised contiguous tensor like `t` (which may be a strided slice)."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty_like(
        t, memory_format=torch.contiguous_format)


def _linattn_dims(q, k, v, lead, batch, seqlen, scale, dev):
    """dims of a linear-attention call whose tokens have `lead` leading dimensions."""
    if q.dim() != lead + 2 or v.dim() != lead + 2:
        want = (("[T, Hk, dk]", "[T, Hv, dv]"), ("[B, L, Hk, dk]", "[B, L, Hv, dv]"))[lead - 1]
        raise ValueError(f"q, k must be {want[0]} and v {want[1]}")
    shp, vshp, dtype = q.shape, v.shape, q.dtype
    if vshp[:lead] != shp[:lead]:
        raise ValueError(f"v has shape {tuple(vshp)}, which does not go with q {tuple(shp)}")
    return SsdLinattnDims(batch, seqlen, shp[-2], vshp[-2], shp[-1], vshp[-1],
                          _row_stride("q", q, dev, dtype, shp),
                          _row_stride("k", k, dev, dtype, shp),
                          _row_stride("v", v, dev, dtype, vshp), scale, _io_dtype(q, "q/k/v"))


def _linattn_scan(fn, lead, q, k, v, log_decay, cu_seqlens, initial_state, o, final_state, workspace,
                  scale, stream):
    lib = load()
    dev = _device_of(q)
    if lead == 1:
        cu, cup = _offsets("cu_seqlens", cu_seqlens)
        nseq = len(cu) - 1
    else:
        nseq = q.shape[0]
    d = _linattn_dims(q, k, v, lead, nseq, q.shape[lead - 1], scale, dev)
    f32 = torch.float32
    state = (nseq, d.v_heads, d.dk, d.dv)
    _need("log_decay", log_decay, dev, f32, (d.v_heads,))
    _need("initial_state", initial_state, dev, f32, state, optional=True)
    _need("o", o, dev, q.dtype, v.shape, optional=True)
    _need("final_state", final_state, dev, f32, state, optional=True)
    _need("workspace", workspace, dev, optional=True)
    args = (ctypes.byref(d),) if lead == 2 else (ctypes.byref(d), cup)
    need = 0
    if workspace is None:
        n = ctypes.c_size_t(0)
        _check(fn + "_workspace_size", getattr(lib, fn + "_workspace_size")(*args, ctypes.byref(n)))
        need = n.value
    with _guard(dev):
        if o is None or final_state is None or need > 0:
            with _on(stream):
                if o is None:
                    o = _empty_rows(v)
                if final_state is None:
                    final_state = log_decay.new_empty(state)
                if need > 0:
                    workspace = torch.empty(need, dtype=torch.uint8, device=v.device)
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        _check(fn, getattr(lib, fn)(*args, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                    log_decay.data_ptr(), _ptr(initial_state), o.data_ptr(),
                                    final_state.data_ptr(), _ptr(workspace), ws_bytes,
                                    _stream(stream, dev)))
    return o, final_state


def ssd_linattn_chunk_scan_workspace_size(batch, seqlen, qk_heads, v_heads, dk, dv,
                                          io_dtype=SSD_BF16) -> int:
    d = SsdLinattnDims(batch, seqlen, qk_heads, v_heads, dk, dv, 0, 0, 0, 1.0, io_dtype)
    n = ctypes.c_size_t(0)
    _check("ssd_linattn_chunk_scan_workspace_size",
           load().ssd_linattn_chunk_scan_workspace_size(ctypes.byref(d), ctypes.byref(n)))
    return int(n.value)


def ssd_linattn_chunk_scan(q, k, v, log_decay, initial_state=None, o=None, final_state=None,
                           workspace=None, scale=1.0, stream=None):
    """Linear attention with one decay per head over prompts: q, k [B, L, Hk, dk],
    v [B, L, Hv, dv], log_decay [Hv] fp32; returns (o [B, L, Hv, dv], final_state
    [B, Hv, dk, dv] fp32).  q, k and v may be slices of one projection."""
    return _linattn_scan("ssd_linattn_chunk_scan", 2, q, k, v, log_decay, None, initial_state, o,
                         final_state, workspace, scale, stream)


def ssd_linattn_chunk_scan_varlen_workspace_size(cu_seqlens, qk_heads, v_heads, dk, dv,
                                                 io_dtype=SSD_BF16) -> int:
    cu, cup = _offsets("cu_seqlens", cu_seqlens)
    d = SsdLinattnDims(len(cu) - 1, int(cu[-1]), qk_heads, v_heads, dk, dv, 0, 0, 0, 1.0, io_dtype)
    n = ctypes.c_size_t(0)
    _check("ssd_linattn_chunk_scan_varlen_workspace_size",
           load().ssd_linattn_chunk_scan_varlen_workspace_size(ctypes.byref(d), cup, ctypes.byref(n)))
    return int(n.value)


def ssd_linattn_chunk_scan_varlen(q, k, v, log_decay, cu_seqlens, initial_states=None, o=None,
                                  final_states=None, workspace=None, scale=1.0, stream=None):
    """ssd_linattn_chunk_scan of a packed batch: q, k [T, Hk, dk], v [T, Hv, dv];
    sequence i is tokens cu_seqlens[i] .. cu_seqlens[i+1]-1 (a host sequence of
    S + 1 offsets).  Returns (o [T, Hv, dv], final_states [S, Hv, dk, dv])."""
    return _linattn_scan("ssd_linattn_chunk_scan_varlen", 1, q, k, v, log_decay, cu_seqlens,
                         initial_states, o, final_states, workspace, scale, stream)


def ssd_linattn_decode_step(q, k, v, log_decay, state, o=None, scale=1.0, stream=None):
    """One linear-attention decode step: q, k [B, Hk, dk], v [B, Hv, dv], state
    [B, Hv, dk, dv] fp32 updated in place; returns o [B, Hv, dv]."""
    dev = _device_of(q)
    d = _linattn_dims(q, k, v, 1, q.shape[0], 1, scale, dev)
    f32 = torch.float32
    _need("log_decay", log_decay, dev, f32, (d.v_heads,))
    _need("state", state, dev, f32, (d.batch, d.v_heads, d.dk, d.dv))
    _need("o", o, dev, q.dtype, v.shape, optional=True)
    with _guard(dev):
        if o is None:
            with _on(stream):
                o = _empty_rows(v)
        _check("ssd_linattn_decode_step", load().ssd_linattn_decode_step(
            ctypes.byref(d), q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
            state.data_ptr(), o.data_ptr(), _stream(stream, dev)))
    return o


def _attn_scale(scale, D):
    return max(D, 1) ** -0.5 if scale is None else scale


def ssd_attn_prefill(q, k, v, cu_seqlens, kv_starts=None, kv_lens=None, scale=None, o=None,
                     stream=None):
    """Causal softmax attention over packed prompts: q [T, Hq, D], k, v [Tk, Hkv, D];
    sequence i has queries cu_seqlens[i] .. cu_seqlens[i+1]-1 and, unless kv_starts
    and kv_lens are None (the prompts' own rows), kv_lens[i] keys from row
    kv_starts[i] on, the last query seeing them all (host sequences).  scale
    defaults to 1 / sqrt(D).  Returns o [T, Hq, D]."""
    dev = _device_of(q)
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q must be [T, Hq, D] and k, v [Tk, Hkv, D]")
    T, Hq, D = q.shape
    Tk, Hkv, _ = k.shape
    qs = _row_stride("q", q, dev, q.dtype, q.shape)
    ks = _row_stride("k", k, dev, q.dtype, (Tk, Hkv, D))
    vs = _row_stride("v", v, dev, q.dtype, (Tk, Hkv, D))
    _need("o", o, dev, q.dtype, q.shape, optional=True)
    cu, cup = _offsets("cu_seqlens", cu_seqlens)
    st, stp = (None, None) if kv_starts is None else _offsets("kv_starts", kv_starts, len(cu) - 1)
    kl, klp = (None, None) if kv_lens is None else _offsets("kv_lens", kv_lens, len(cu) - 1)
    d = SsdAttnDims(len(cu) - 1, T, Tk, Hq, Hkv, D, qs, ks, vs,
                    _attn_scale(scale, D), _io_dtype(q, "q/k/v"))
    with _guard(dev):
        if o is None:
            with _on(stream):
                o = _empty_rows(q)
        _check("ssd_attn_prefill", load().ssd_attn_prefill(
            ctypes.byref(d), cup, stp, klp, _ptr(q), _ptr(k), _ptr(v), _ptr(o),
            _stream(stream, dev)))
    return o


def ssd_attn_decode_workspace_size(batch, cache_rows, q_heads, kv_heads, head_dim,
                                   io_dtype=SSD_BF16) -> int:
    d = SsdAttnDims(batch, 0, cache_rows, q_heads, kv_heads, head_dim, 0, 0, 0, 1.0, io_dtype)
    n = ctypes.c_size_t(0)
    _check("ssd_attn_decode_workspace_size",
           load().ssd_attn_decode_workspace_size(ctypes.byref(d), ctypes.byref(n)))
    return int(n.value)


def ssd_attn_decode_step(q, k, v, k_cache, v_cache, lengths, scale=None, o=None, workspace=None,
                         stream=None):
    """One softmax-attention decode step: k, v [B, Hkv, D] are written to row
    lengths[b] of k_cache, v_cache [B, M, Hkv, D], and q [B, Hq, D] attends rows
    0 .. lengths[b].  lengths [B] int32 is a device tensor and is left as it is; a
    length outside [0, M) marks an unused slot (o[b] = 0, cache untouched).
    Returns o [B, Hq, D]."""
    dev = _device_of(q)
    if q.dim() != 3 or k.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("q must be [B, Hq, D], k, v [B, Hkv, D] and the caches [B, M, Hkv, D]")
    B, Hq, D = q.shape
    Hkv, M = k.shape[1], k_cache.shape[1]
    qs = _row_stride("q", q, dev, q.dtype, q.shape)
    ks = _row_stride("k", k, dev, q.dtype, (B, Hkv, D))
    vs = _row_stride("v", v, dev, q.dtype, (B, Hkv, D))
    _need("k_cache", k_cache, dev, q.dtype, (B, M, Hkv, D))
    _need("v_cache", v_cache, dev, q.dtype, (B, M, Hkv, D))
    _need("lengths", lengths, dev, torch.int32, (B,))
    _need("o", o, dev, q.dtype, q.shape, optional=True)
    _need("workspace", workspace, dev, optional=True)
    lib = load()
    d = SsdAttnDims(B, 0, M, Hq, Hkv, D, qs, ks, vs, _attn_scale(scale, D),
                    _io_dtype(q, "q/k/v"))
    need = 0
    if workspace is None:
        n = ctypes.c_size_t(0)
        _check("ssd_attn_decode_workspace_size",
               lib.ssd_attn_decode_workspace_size(ctypes.byref(d), ctypes.byref(n)))
        need = n.value
    with _guard(dev):
        if o is None or need > 0:
            with _on(stream):
                if o is None:
                    o = _empty_rows(q)
                if need > 0:
                    workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        _check("ssd_attn_decode_step", lib.ssd_attn_decode_step(
            ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache),
            _ptr(lengths), _ptr(o), _ptr(workspace), ws_bytes, _stream(stream, dev)))
    return o


# --------------------------------------------------------------------------
# Norm and rotation of queries and keys, paged caches
# --------------------------------------------------------------------------
class SsdPagedDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("rows", ctypes.c_int64),
                ("q_heads", ctypes.c_int64), ("kv_heads", ctypes.c_int64),
                ("head_dim", ctypes.c_int64), ("num_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("max_pages", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("q_out_stride", ctypes.c_int64),
                ("k_out_stride", ctypes.c_int64), ("scale", ctypes.c_float),
                ("io_dtype", ctypes.c_int32), ("page_format", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class SsdQkRope(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("eps", ctypes.c_float), ("reserved", ctypes.c_int32)]


def _rope(dev, T, D, positions, inv_freq, q_weight, k_weight, eps, interleaved):
    f32 = torch.float32
    rot, fp, qp, kp, pp = 0, None, None, None, None
    if inv_freq is not None:
        _need("inv_freq", inv_freq, dev, f32)
        if inv_freq.dim() != 1:
            raise ValueError(f"inv_freq must be [rot_dim / 2], got shape {tuple(inv_freq.shape)}")
        rot, fp = 2 * inv_freq.shape[0], inv_freq.data_ptr()
    if q_weight is not None:
        _need("q_weight", q_weight, dev, f32, (D,))
        qp = q_weight.data_ptr()
    if k_weight is not None:
        _need("k_weight", k_weight, dev, f32, (D,))
        kp = k_weight.data_ptr()
    if positions is not None:
        _need("positions", positions, dev, torch.int32, (T,))
        pp = positions.data_ptr()
    return SsdQkRope(fp, qp, kp, pp, rot, int(interleaved), eps, 0)


def _out_rows(name, t, like, dev, stream):
    """An output of rows like `like`, given or new: (tensor, distance between its rows)."""
    if t is not None:
        return t, _row_stride(name, t, dev, like.dtype, like.shape)
    if stream is None:
        return _empty_rows(like), 0
    with _on(stream):
        return _empty_rows(like), 0


def _host_rows(name, x, n=None):
    """_offsets with the array's address."""
    import numpy as np
    a = np.ascontiguousarray(x, dtype=np.int64)
    if a.ndim != 1 or (len(a) < 1 if n is None else len(a) != n):
        raise ValueError(f"{name} must hold " + ("B + 1 offsets" if n is None else "one entry per sequence"))
    return a, a.__array_interface__["data"][0]


def _pages(dev, k_pages, v_pages, block_table, k_scales, v_scales, io, D=None, Hkv=None, B=None):
    """Checks a paged cache of input type `io`; returns (page_format, num_pages, Hkv, page_size,
    D, B, max_pages)."""
    if not (isinstance(k_pages, torch.Tensor) and isinstance(block_table, torch.Tensor)):
        raise TypeError("k_pages and block_table must be torch.Tensors, got "
                        f"{type(k_pages).__name__} and {type(block_table).__name__}")
    if k_pages.dim() != 4 or block_table.dim() != 2:
        raise ValueError("pages must be [num_pages, Hkv, page_size, D] (D / 2 bytes in 4 bits) and "
                         "block_table [B, max_pages]")
    q4 = k_scales is not None or v_scales is not None
    n, h, p, width = k_pages.shape
    d = 2 * width if q4 else width
    dtype = torch.uint8 if q4 else io
    _need("k_pages", k_pages, dev, dtype)
    if (D is not None and d != D) or (Hkv is not None and h != Hkv):
        raise ValueError(f"k_pages has shape {tuple(k_pages.shape)}, which does not go with "
                         f"{Hkv if Hkv is not None else h} key heads of {D if D is not None else d}")
    _need("v_pages", v_pages, dev, dtype, k_pages.shape)
    if q4:
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            _need(name, t, dev, torch.float16, (n, h, p, d // 64, 2))
    _need("block_table", block_table, dev, torch.int32, None if B is None else (B, block_table.shape[1]))
    return (SSD_PAGES_4BIT if q4 else SSD_PAGES_IO, n, h, p, d, block_table.shape[0], block_table.shape[1])


def ssd_attn_qk_norm_rope(q, k, positions=None, inv_freq=None, q_weight=None, k_weight=None, eps=1e-6,
                          interleaved=False, q_out=None, k_out=None, stream=None):
    """Norms every head of q [T, Hq, D] and k [T, Hkv, D] (x w / sqrt(mean(x^2) + eps) for the
    weights that are given, [D] fp32) and rotates its first 2 len(inv_freq) values by
    positions [T] int32 times inv_freq (fp32), pairing value i with i + len(inv_freq), or
    neighbours with interleaved.  q and k may be slices of one projection, and q_out and
    k_out may be q and k.  Returns (q_out, k_out)."""
    dev = _device_of(q)
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q must be [T, Hq, D] and k [T, Hkv, D]")
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    if inv_freq is not None and positions is None:
        raise ValueError("positions is required with inv_freq")
    qs, ks = _row_stride("q", q, dev, q.dtype, q.shape), _row_stride("k", k, dev, q.dtype, (T, Hkv, D))
    io = _io_dtype(q, "q/k")
    rope = _rope(dev, T, D, positions, inv_freq, q_weight, k_weight, eps, interleaved)
    with _guard(dev):
        q_out, qos = _out_rows("q_out", q_out, q, dev, stream)
        k_out, kos = _out_rows("k_out", k_out, k, dev, stream)
        d = SsdPagedDims(0, T, Hq, Hkv, D, 0, 0, 0, qs, ks, 0, qos, kos, 1.0, io, 0, 0)
        _check("ssd_attn_qk_norm_rope", load().ssd_attn_qk_norm_rope(
            ctypes.byref(d), ctypes.byref(rope), q.data_ptr(), k.data_ptr(), q_out.data_ptr(),
            k_out.data_ptr(), _stream(stream, dev)))
    return q_out, k_out


def ssd_attn_paged_append(q, k, v, k_pages, v_pages, block_table, lengths, cu_seqlens=None, k_scales=None,
                          v_scales=None, positions=None, inv_freq=None, q_weight=None, k_weight=None,
                          eps=1e-6, interleaved=False, q_out=None, k_out=None, stream=None):
    """Norms and rotates q [T, Hq, D] (returned as q_out; None: no queries) and k [T, Hkv, D] as
    ssd_attn_qk_norm_rope does, and appends k and v [T, Hkv, D] to a paged cache: k_pages,
    v_pages [num_pages, Hkv, page_size, D] of the input type, or with k_scales, v_scales
    [num_pages, Hkv, page_size, D / 64, 2] float16 the 4-bit codes [.., D / 2] uint8.  Token j
    of sequence b becomes row lengths[b] + j, line r % page_size of page block_table[b, r //
    page_size]; that row is its position unless positions is given.  cu_seqlens: a host
    sequence of B + 1 offsets, None for one token per sequence.  block_table [B, max_pages] and
    lengths [B] are int32 device tensors, left as they are.  Tokens whose row has no page are
    not stored.  k_out, if given, receives the keys as ssd_attn_prefill takes them."""
    dev = _device_of(k)
    if k.dim() != 3 or (q is not None and q.dim() != 3):
        raise ValueError("q must be [T, Hq, D] and k, v [T, Hkv, D]")
    T, Hkv, D = k.shape
    Hq = Hkv if q is None else q.shape[1]
    dt = k.dtype
    io = _io_dtype(k, "q/k/v")
    if cu_seqlens is None:
        B, cup = T, None
    else:
        cu, cup = _host_rows("cu_seqlens", cu_seqlens)
        B = len(cu) - 1
    qs = 0 if q is None else _row_stride("q", q, dev, dt, (T, Hq, D))
    ks, vs = _row_stride("k", k, dev, dt, k.shape), _row_stride("v", v, dev, dt, k.shape)
    fmt, n, _, p, _, _, m = _pages(dev, k_pages, v_pages, block_table, k_scales, v_scales, dt, D, Hkv, B)
    _need("lengths", lengths, dev, torch.int32, (B,))
    rope = _rope(dev, T, D, positions, inv_freq, q_weight, k_weight, eps, interleaved)
    if q is None and q_out is not None:
        raise ValueError("q_out needs q")
    kos = 0 if k_out is None else _row_stride("k_out", k_out, dev, dt, k.shape)
    with _guard(dev):
        qos = 0
        if q is not None:
            q_out, qos = _out_rows("q_out", q_out, q, dev, stream)
        d = SsdPagedDims(B, T, Hq, Hkv, D, n, p, m, qs, ks, vs, qos, kos, 1.0, io, fmt, 0)
        _check("ssd_attn_paged_append", load().ssd_attn_paged_append(
            ctypes.byref(d), ctypes.byref(rope), cup, _ptr(q), k.data_ptr(), v.data_ptr(), k_pages.data_ptr(),
            v_pages.data_ptr(), _ptr(k_scales), _ptr(v_scales), block_table.data_ptr(), lengths.data_ptr(),
            _ptr(q_out), _ptr(k_out), _stream(stream, dev)))
    return q_out


def ssd_attn_paged_gather(k_pages, v_pages, block_table, cu_seqlens, starts=None, k_scales=None, v_scales=None,
                          dtype=None, k=None, v=None, stream=None):
    """Rows starts[b] .. (None: 0 ..) of every sequence's pages as packed rows cu_seqlens[b] ..
    cu_seqlens[b+1]-1 (host sequences), which ssd_attn_prefill attends with kv_starts =
    cu_seqlens[:-1]: returns (k, v) [T, Hkv, D].  dtype: the values' type of 4-bit pages
    (bfloat16 unless given).  Rows on no page are 0."""
    dev = _device_of(k_pages)
    if k_scales is None and v_scales is None:
        dt = k_pages.dtype
        if dtype is not None and dtype != dt:
            raise TypeError(f"rows of {dt} pages are {dt}, not {dtype}")
    else:
        dt = torch.bfloat16 if dtype is None else dtype
    cu, cup = _host_rows("cu_seqlens", cu_seqlens)
    B, T = len(cu) - 1, int(cu[-1])
    st, stp = (None, None) if starts is None else _host_rows("starts", starts, B)
    fmt, n, Hkv, p, D, _, m = _pages(dev, k_pages, v_pages, block_table, k_scales, v_scales, dt, B=B)
    io = SSD_BF16 if dt == torch.bfloat16 else SSD_F32 if dt == torch.float32 else None
    if io is None:
        raise TypeError(f"pages and rows must be bfloat16 or float32, got {dt}")
    d = SsdPagedDims(B, T, Hkv, Hkv, D, n, p, m, 0, 0, 0, 0, 0, 1.0, io, fmt, 0)
    with _guard(dev):
        with _on(stream):
            if k is None:
                k = k_pages.new_empty((max(T, 0), Hkv, D), dtype=dt)
            else:
                _need("k", k, dev, dt, (T, Hkv, D))
            if v is None:
                v = torch.empty_like(k)
            else:
                _need("v", v, dev, dt, (T, Hkv, D))
        _check("ssd_attn_paged_gather", load().ssd_attn_paged_gather(
            ctypes.byref(d), cup, stp, k_pages.data_ptr(), v_pages.data_ptr(), _ptr(k_scales), _ptr(v_scales),
            block_table.data_ptr(), k.data_ptr(), v.data_ptr(), _stream(stream, dev)))
    return k, v


def ssd_attn_paged_decode_workspace_size(batch, q_heads, kv_heads, head_dim, num_pages, page_size, max_pages,
                                         io_dtype=SSD_BF16, page_format=SSD_PAGES_IO) -> int:
    d = SsdPagedDims(batch, 0, q_heads, kv_heads, head_dim, num_pages, page_size, max_pages, 0, 0, 0, 0, 0, 1.0,
                     io_dtype, page_format, 0)
    n = ctypes.c_size_t(0)
    _check("ssd_attn_paged_decode_workspace_size",
           load().ssd_attn_paged_decode_workspace_size(ctypes.byref(d), ctypes.byref(n)))
    return int(n.value)


def ssd_attn_paged_decode_step(q, k_pages, v_pages, block_table, lengths, k_scales=None, v_scales=None,
                               scale=None, o=None, workspace=None, stream=None):
    """Softmax attention of one token per sequence over a paged cache (see
    ssd_attn_paged_append, which has stored the token's own key and value): q [B, Hq, D]
    attends rows 0 .. lengths[b].  A length outside [0, max_pages page_size) marks an unused
    slot (o[b] = 0); rows on no page are not attended.  scale defaults to 1 / sqrt(D).
    Returns o [B, Hq, D]."""
    dev = _device_of(q)
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, D]")
    B, Hq, D = q.shape
    io = _io_dtype(q, "q")
    qs = _row_stride("q", q, dev, q.dtype, q.shape)
    fmt, n, Hkv, p, _, _, m = _pages(dev, k_pages, v_pages, block_table, k_scales, v_scales, q.dtype, D, None, B)
    _need("lengths", lengths, dev, torch.int32, (B,))
    _need("o", o, dev, q.dtype, q.shape, optional=True)
    _need("workspace", workspace, dev, optional=True)
    lib = load()
    d = SsdPagedDims(B, 0, Hq, Hkv, D, n, p, m, qs, 0, 0, 0, 0, _attn_scale(scale, D), io, fmt, 0)
    need = 0
    if workspace is None:
        size = ctypes.c_size_t(0)
        _check("ssd_attn_paged_decode_workspace_size",
               lib.ssd_attn_paged_decode_workspace_size(ctypes.byref(d), ctypes.byref(size)))
        need = size.value
    with _guard(dev):
        if o is None or need > 0:
            with _on(stream):
                if o is None:
                    o = _empty_rows(q)
                if need > 0:
                    workspace = lengths.new_empty(need // 4)
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        _check("ssd_attn_paged_decode_step", lib.ssd_attn_paged_decode_step(
            ctypes.byref(d), q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), _ptr(k_scales), _ptr(v_scales),
            block_table.data_ptr(), lengths.data_ptr(), o.data_ptr(), _ptr(workspace), ws_bytes,
            _stream(stream, dev)))
    return o
