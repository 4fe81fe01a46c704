"""Binding of the operators around the recurrence: the short causal convolution, the selective
state space scan, and the verification and commit of drafted tokens.

As in :mod:`api`, this module only checks tensors, allocates outputs and workspaces and passes raw
pointers and the stream; the work is in the library's CUDA kernels.  Every call is asynchronous
and leaves its workspace in ``<function>.last_workspace`` for :func:`read_device_status`.

Results carry no history of PyTorch's autograd, whether or not the inputs require gradients: a training
program makes a forward and a backward call one node (``examples/recurrent_training.py`` has both nodes of
its block).
"""
from __future__ import annotations

import ctypes

import torch

from . import api
from .api import KDA_FLAG_CUDA_CORE_PATH, KdaDesc, KdaError, _dt, _need, _shape

_P = ctypes.c_void_p
_I32, _I64 = ctypes.c_int32, ctypes.c_int64
STATUS_WORKSPACE_BYTES = 256


class KdaConvDesc(ctypes.Structure):
    """Mirror of ``kda_conv_desc_t`` in include/kda.h."""
    _fields_ = [("num_seqs", _I32), ("total_tokens", _I64), ("channels", _I32), ("width", _I32),
                ("dtype", ctypes.c_int), ("silu", _I32), ("x_pitch", _I64), ("num_slots", _I64),
                ("slot_stride_elems", _I64)]


class KdaSsmInputs(ctypes.Structure):
    """Mirror of ``kda_ssm_inputs_t`` in include/kda.h."""
    _fields_ = [("x", _P), ("x_pitch", _I64), ("dt", _P), ("dt_pitch", _I64), ("b", _P),
                ("b_pitch", _I64), ("c", _P), ("c_pitch", _I64), ("a_log", _P), ("dt_bias", _P),
                ("d", _P)]


class KdaGatedDesc(ctypes.Structure):
    """Mirror of ``kda_gated_desc_t`` in include/kda.h."""
    _fields_ = [("num_seqs", _I32), ("total_tokens", _I64), ("channels", _I32), ("dtype", ctypes.c_int),
                ("x_pitch", _I64), ("r_pitch", _I64), ("i_pitch", _I64), ("num_slots", _I64),
                ("slot_stride_elems", _I64)]


class KdaSampleDesc(ctypes.Structure):
    """Mirror of ``kda_sample_desc_t`` in include/kda.h."""
    _fields_ = [("num_rows", _I32), ("vocab", _I32), ("dtype", ctypes.c_int), ("logits_pitch", _I64),
                ("noise_pitch", _I64), ("temperature", ctypes.c_float), ("top_k", _I32),
                ("top_p", ctypes.c_float), ("min_p", ctypes.c_float)]


_lib = None


def _load():
    global _lib
    if _lib is None:
        lib = api.load()
        size, desc, conv = ctypes.c_size_t, ctypes.POINTER(KdaDesc), ctypes.POINTER(KdaConvDesc)
        ins, gated = ctypes.POINTER(KdaSsmInputs), ctypes.POINTER(KdaGatedDesc)
        draw = ctypes.POINTER(KdaSampleDesc)
        for name, args, res in (
                ("kda_causal_conv", [conv, *[_P] * 9, size, _P], ctypes.c_int),
                ("kda_causal_conv_decode",
                 [conv, *[_P] * 7, _I64, _I32, ctypes.c_int, _P, _P, size, _P], ctypes.c_int),
                ("kda_causal_conv_backward", [conv, _P, _I64, *[_P] * 11, size, _P], ctypes.c_int),
                ("kda_causal_conv_backward_workspace_size", [conv], size),
                ("kda_ssm_scan", [desc, ins, *[_P] * 6, size, _P], ctypes.c_int),
                ("kda_ssm_scan_workspace_size", [desc], size),
                ("kda_ssm_decode",
                 [desc, ins, *[_P] * 4, _I64, _I32, ctypes.c_int, _P, _P, size, _P], ctypes.c_int),
                ("kda_gated_scan", [gated, *[_P] * 11, size, _P], ctypes.c_int),
                ("kda_gated_scan_workspace_size", [gated], size),
                ("kda_gated_scan_backward", [gated, _P, _I64, *[_P] * 14, size, _P], ctypes.c_int),
                ("kda_gated_scan_backward_workspace_size", [gated], size),
                ("kda_gated_decode",
                 [gated, *[_P] * 8, _I64, _I32, ctypes.c_int, _P, _P, size, _P], ctypes.c_int),
                ("kda_sample", [draw, *[_P] * 8, size, _P], ctypes.c_int),
                ("kda_sample_probs", [draw, *[_P] * 7, size, _P], ctypes.c_int),
                ("kda_verify_draft", [_I32, _I64, _I32, *[_P] * 9, size, _P], ctypes.c_int),
                ("kda_verify_draft_marked",
                 [_I32, _I64, _I32, *[_P] * 8, ctypes.c_uint32, _P, size, _P], ctypes.c_int),
                ("kda_commit_draft",
                 [_I32, ctypes.c_int, _I64, _P, _I64, _I32, _P, _P, _I64, _I64, _P, _P, size, _P],
                 ctypes.c_int)):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, res
        _lib = lib
    return _lib


def _p(t):
    return None if t is None else t.data_ptr()


# The checks below sit on the host path of every call, a good part of a small call's time: each
# asks the expected case in one expression and leaves the finding of what is wrong to the slow
# path behind it.

def _plain(t, name, dtype, shape):
    """``t`` is a contiguous tensor of ``dtype`` and ``shape``."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.is_contiguous()):
        _need(t, name, dtype, cuda=False)
        _shape(t, name, shape)


def _rows(t, name, shape, dtype):
    """``t`` has ``dtype`` and ``shape``, each row (the trailing dimensions) packed and no two rows
    overlapping; returns the elements between rows."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape:
        st = t.stride()
        if shape[0] < 2:
            pass
        elif len(st) == 2:
            if st[1] == 1 and st[0] >= shape[1]:
                return st[0]
        elif st[2] == 1 and st[1] == shape[2] and st[0] >= shape[1] * shape[2]:
            return st[0]
    return _rows_slow(t, name, shape, dtype)


def _rows_slow(t, name, shape, dtype):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    _shape(t, name, shape)
    row = 1
    for i in range(t.dim() - 1, 0, -1):
        if t.shape[i] > 1 and t.stride(i) != row:
            raise ValueError(f"the rows of {name} must be contiguous")
        row *= t.shape[i]
    if t.shape[0] > 1 and t.stride(0) < row:
        raise ValueError(f"the rows of {name} must not overlap")
    return t.stride(0) if t.shape[0] > 1 else row  # the stride of a single row says nothing


def _cuda(*tensors):
    """Every tensor of the call, a given workspace among them, lives on one CUDA device, the current one:
    the library launches there, and a stream's handle of 0 means that device's default stream."""
    dev = None
    for t in tensors:
        if t is not None:
            i = t.get_device()
            if i < 0:
                raise ValueError("every tensor of the call must live on a CUDA device")
            if dev is None:
                dev = i
            elif i != dev:
                raise ValueError(f"the call's tensors must share one device, got cuda:{dev} and cuda:{i}")
    if dev != torch.cuda.current_device():
        raise ValueError(f"the call's tensors live on cuda:{dev}, which must be the current device "
                         "(torch.cuda.device)")


def _activation(activation):
    if activation is None:
        return 0
    if activation != "silu":
        raise ValueError(f"activation must be None or 'silu', got {activation!r}")
    return 1


def _num_seqs(cu_seqlens):
    if not (isinstance(cu_seqlens, torch.Tensor) and cu_seqlens.dtype is torch.int32
            and cu_seqlens.dim() == 1 and cu_seqlens.is_contiguous()):
        _need(cu_seqlens, "cu_seqlens", torch.int32, cuda=False)
        _shape(cu_seqlens, "cu_seqlens", (None,))
    n = cu_seqlens.shape[0] - 1
    if n < 0:
        raise ValueError("cu_seqlens needs at least one element")
    return n


def _step_cache(cache, name, N, max_steps, row, dtype):
    """Row pitch of a step cache: [requests, ...] with max_steps packed rows each."""
    if not isinstance(cache, torch.Tensor) or cache.dtype != dtype:
        raise TypeError(f"{name} must be a tensor of {dtype}")
    if cache.dim() < 2 or cache.shape[0] < N:
        raise ValueError(f"{name} must hold {N} requests, got {list(cache.shape)}")
    if cache.is_contiguous():
        packed = pitch = cache.numel() // cache.shape[0] if cache.shape[0] else 0
    else:
        packed = 1
        for i in range(cache.dim() - 1, 0, -1):
            if cache.shape[i] > 1 and cache.stride(i) != packed:
                raise ValueError(f"the requests of {name} must be contiguous")
            packed *= cache.shape[i]
        pitch = cache.stride(0) if cache.shape[0] > 1 else packed
    if N > 0 and (packed < max_steps * row or pitch < packed):
        raise ValueError(f"{name} must hold {max_steps} states of {row} elements a request")
    return max(pitch, max_steps * row)


def _state_pool(state, name, dims, slot_stride):
    """Pool of [slots, *dims], packed, or a buffer of shape[0] slots slot_stride elements apart."""
    if not (isinstance(state, torch.Tensor) and state.is_contiguous()):
        _need(state, name, cuda=False)
    if slot_stride == 0:
        if state.shape[1:] != dims:
            _shape(state, name, (None, *dims))
        if state.shape[0] == 0:
            raise ValueError(f"{name} has no slots")
        return
    row = 1
    for d in dims:
        row *= d
    if slot_stride < row or state.dim() < 1 or state.shape[0] == 0 or \
            state.numel() < (state.shape[0] - 1) * slot_stride + row:
        raise ValueError(f"{name} is too small for its slots of pitch {slot_stride}")


def _stream(stream, device):
    if stream is None:  # the handle alone: torch.cuda.current_stream() builds an object, 2 us of a call's 20
        return torch._C._cuda_getCurrentRawStream(device.index)
    if stream.device_index != device.index:
        raise ValueError(f"the stream belongs to cuda:{stream.device_index}, the call's tensors to {device}")
    return stream.cuda_stream


def _empty(stream, shape, dtype, device):
    """An uninitialised tensor that belongs to the call's stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _workspace(stream, given, size, device):
    """The given workspace if it holds a status word, else a new one of ``size`` bytes."""
    if given is not None:
        if not given.is_contiguous():
            raise ValueError("workspace must be contiguous")
        if given.numel() * given.element_size() >= STATUS_WORKSPACE_BYTES:
            return given, given.numel() * given.element_size()
    return _empty(stream, size, torch.uint8, device), size


def _done(rc, what, owner, workspace):
    if rc != 0:
        raise KdaError(rc, what)
    owner.last_workspace = workspace


# ------------------------------------------------------------------------ short convolution

def check_conv_args(x, weight, *, bias=None, cu_seqlens=None, state=None, state_indices=None,
                    final_state=None, out=None, slot_stride=0, token=False):
    """Checks of a convolution call (host only); returns (N, T, channels, width, x's pitch)."""
    if not isinstance(x, torch.Tensor) or x.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("x must be a bfloat16 or float32 tensor")
    if x.dim() != 2 or x.shape[1] < 1:
        raise ValueError(f"x must have shape [T, channels], got {list(x.shape)}")
    dtype = x.dtype
    T, ch = x.shape
    pitch = _rows(x, "x", (T, ch), dtype)
    width = weight.shape[1] if isinstance(weight, torch.Tensor) and weight.dim() == 2 else 0
    _plain(weight, "weight", dtype, (ch, width))
    if not 2 <= width <= 4:
        raise ValueError(f"weight must have 2 to 4 taps, got {width}")
    if bias is not None:
        _plain(bias, "bias", dtype, (ch,))
    N = T if cu_seqlens is None else _num_seqs(cu_seqlens)
    if state_indices is not None:
        _plain(state_indices, "state_indices", torch.int32, (N,))
    if token or state_indices is not None:
        if state is None:
            raise ValueError("pool mode needs the pool in `state`")
        _state_pool(state, "state", (width - 1, ch), slot_stride)
        if state.dtype is not dtype:
            raise TypeError(f"state must be {dtype}, got {state.dtype}")
        if final_state is not None and final_state is not state:
            raise ValueError("pool mode updates the pool: final_state must be None or the pool")
    else:
        if state is not None:
            _plain(state, "state", dtype, (N, width - 1, ch))
        if final_state is not None:
            _plain(final_state, "final_state", dtype, (N, width - 1, ch))
    if out is not None:
        _plain(out, "out", dtype, (T, ch))
    return N, T, ch, width, pitch


def causal_conv(x, weight, cu_seqlens, *, bias=None, activation=None, state=None,
                state_indices=None, final_state=None, output_final_state=True, slot_stride=0,
                out=None, workspace=None, stream=None):
    """Short causal depthwise convolution of packed sequences (kda_causal_conv).  Returns
    ``(y, final)``.

    x [T, Ch] bf16 or fp32, its rows at any pitch (a slice of a projection); weight [Ch, W], W = 2..4;
    bias [Ch] or None; activation "silu" or None; cu_seqlens [N+1] int32.  A state is the last W-1
    inputs, [W-1, Ch], oldest first.  Pool mode (``state_indices`` [N] int32): ``state`` is the pool
    [num_slots, W-1, Ch], updated in place and returned as ``final``.  Dense mode: ``state`` is
    [N, W-1, Ch] or None (zeros); ``final`` is ``final_state`` or a new tensor, or None when
    ``output_final_state`` is False.
    """
    N, T, ch, width, pitch = check_conv_args(
        x, weight, bias=bias, cu_seqlens=cu_seqlens, state=state, state_indices=state_indices,
        final_state=final_state, out=out, slot_stride=slot_stride)
    _cuda(x, weight, bias, cu_seqlens, state, state_indices, final_state, out, workspace)
    silu = _activation(activation)
    lib, dev = _load(), x.device
    pool = state_indices is not None
    if pool:
        final_state = state
    elif final_state is None and output_final_state:
        final_state = _empty(stream, (N, width - 1, ch), x.dtype, dev)
    if out is None:
        out = _empty(stream, (T, ch), x.dtype, dev)
    ws, nws = _workspace(stream, workspace, STATUS_WORKSPACE_BYTES, dev)
    d = KdaConvDesc(N, T, ch, width, _dt(x.dtype), silu, pitch, state.shape[0] if pool else 0,
                    slot_stride)
    rc = lib.kda_causal_conv(ctypes.byref(d), _p(x), _p(weight), _p(bias), _p(cu_seqlens), _p(state),
                             _p(state_indices), _p(final_state), _p(out), _p(ws), nws,
                             _stream(stream, dev))
    _done(rc, "kda_causal_conv", causal_conv, ws)
    return out, final_state


def _conv_token(x, weight, cu_seqlens, state, state_indices, bias, activation, cache, max_steps,
                update_state, slot_stride, out, workspace, stream, owner):
    N, T, ch, width, pitch = check_conv_args(x, weight, bias=bias, cu_seqlens=cu_seqlens, state=state,
                                             state_indices=state_indices, out=out,
                                             slot_stride=slot_stride, token=True)
    _cuda(x, weight, bias, cu_seqlens, state, state_indices, cache, out, workspace)
    silu = _activation(activation)
    cpitch = 0
    if cache is not None:
        cpitch = _step_cache(cache, "cache", N, max_steps, (width - 1) * ch, x.dtype)
    lib, dev = _load(), x.device
    if out is None:
        out = _empty(stream, (T, ch), x.dtype, dev)
    ws, nws = _workspace(stream, workspace, STATUS_WORKSPACE_BYTES, dev)
    d = KdaConvDesc(N, T, ch, width, _dt(x.dtype), silu, pitch, state.shape[0], slot_stride)
    rc = lib.kda_causal_conv_decode(ctypes.byref(d), _p(x), _p(weight), _p(bias), _p(cu_seqlens),
                                    _p(state), _p(state_indices), _p(cache), cpitch, max_steps,
                                    1 if update_state else 0, _p(out), _p(ws), nws,
                                    _stream(stream, dev))
    _done(rc, "kda_causal_conv_decode", owner, ws)
    return out


def causal_conv_decode(x, weight, state, state_indices=None, *, bias=None, activation=None,
                       slot_stride=0, out=None, workspace=None, stream=None):
    """The convolution of one new token a row (kda_causal_conv_decode), updating the pool ``state``
    [num_slots, W-1, Ch] in place.  x [N, Ch].  Returns y [N, Ch]."""
    return _conv_token(x, weight, None, state, state_indices, bias, activation, None, 1, True,
                       slot_stride, out, workspace, stream, causal_conv_decode)


def _steps(cu_seqlens, max_steps, stream):
    if max_steps is not None:
        return int(max_steps)
    if _num_seqs(cu_seqlens) < 1:
        return 1
    with torch.cuda.stream(stream):  # after what the call's stream has still to write (None: the current one)
        return max(1, int((cu_seqlens[1:] - cu_seqlens[:-1]).max().item()))


def causal_conv_draft(x, weight, cu_seqlens, state, state_indices=None, *, bias=None,
                      activation=None, cache=None, max_steps=None, update_state=False,
                      slot_stride=0, out=None, workspace=None, stream=None):
    """The convolution of drafted tokens, as :func:`decode_draft`: request n's tokens
    cu_seqlens[n] .. cu_seqlens[n+1]-1 follow pool slot n; ``cache`` [N, steps, W-1, Ch] gets the state
    after each.  ``max_steps`` (the most tokens of a request) is read from the device if not given.
    Returns y [T, Ch]."""
    return _conv_token(x, weight, cu_seqlens, state, state_indices, bias, activation, cache,
                       _steps(cu_seqlens, max_steps, stream), update_state, slot_stride, out, workspace,
                       stream, causal_conv_draft)


def causal_conv_backward(dy, x, weight, cu_seqlens, *, bias=None, activation=None, state=None, dfinal=None,
                         workspace=None, stream=None):
    """The derivatives of a loss by the inputs of a dense :func:`causal_conv` (kda_causal_conv_backward), from
    those by y (``dy`` [T, Ch], rows at any pitch) and by the final states (``dfinal`` [N, W-1, Ch] or None).
    Returns ``(dx, dweight, dbias, dstate)``: dx and dstate in x's type, dweight [Ch, W] and dbias [Ch] fp32;
    dbias None without ``bias``, dstate None without ``state``.

    x, weight, cu_seqlens, bias, activation and state as the forward call had them.
    """
    N, T, ch, width, pitch = check_conv_args(x, weight, bias=bias, cu_seqlens=cu_seqlens, state=state)
    dy_pitch = _rows(dy, "dy", (T, ch), x.dtype)
    if dfinal is not None:
        _plain(dfinal, "dfinal", x.dtype, (N, width - 1, ch))
    _cuda(dy, x, weight, cu_seqlens, bias, state, dfinal, workspace)
    silu = _activation(activation)
    lib, dev = _load(), x.device
    dx = _empty(stream, (T, ch), x.dtype, dev)
    dweight = _empty(stream, (ch, width), torch.float32, dev)
    dbias = None if bias is None else _empty(stream, (ch,), torch.float32, dev)
    dstate = None if state is None else _empty(stream, (N, width - 1, ch), x.dtype, dev)
    d = KdaConvDesc(N, T, ch, width, _dt(x.dtype), silu, pitch, 0, 0)
    size = lib.kda_causal_conv_backward_workspace_size(ctypes.byref(d))
    ws, nws = _workspace(stream, workspace, max(size, STATUS_WORKSPACE_BYTES), dev)
    rc = lib.kda_causal_conv_backward(ctypes.byref(d), _p(dy), dy_pitch, _p(x), _p(weight), _p(bias),
                                      _p(cu_seqlens), _p(state), _p(dfinal), _p(dx), _p(dweight), _p(dbias),
                                      _p(dstate), _p(ws), nws, _stream(stream, dev))
    _done(rc, "kda_causal_conv_backward", causal_conv_backward, ws)
    return dx, dweight, dbias, dstate


# ------------------------------------------------------------------------ state space scan

def check_ssm_args(x, dt, A_log, B, C, *, D=None, dt_bias=None, cu_seqlens=None, state=None,
                   state_indices=None, final_state=None, out=None, slot_stride=0, token=False):
    """Checks of a scan call (host only); returns (N, T, H, G, K, V, pitches of x, dt, B, C)."""
    if not isinstance(x, torch.Tensor) or x.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("x must be a bfloat16 or float32 tensor")
    if x.dim() != 3 or not isinstance(B, torch.Tensor) or B.dim() != 3:
        raise ValueError("x must have shape [T, H, V] and B [T, G, K]")
    dtype = x.dtype
    T, H, V = x.shape
    _, G, K = B.shape
    if G == 0 or H == 0 or H % G != 0:
        raise ValueError(f"the head count {H} must be a multiple of the group count {G}")
    pitches = (_rows(x, "x", (T, H, V), dtype), _rows(dt, "dt", (T, H), dtype),
               _rows(B, "B", (T, G, K), dtype), _rows(C, "C", (T, G, K), dtype))
    _plain(A_log, "A_log", torch.float32, (H,))
    if dt_bias is not None:
        _plain(dt_bias, "dt_bias", torch.float32, (H,))
    if D is not None:
        _plain(D, "D", torch.float32, (H,))
    N = T if cu_seqlens is None else _num_seqs(cu_seqlens)
    if state_indices is not None:
        _plain(state_indices, "state_indices", torch.int32, (N,))
    if token or state_indices is not None:
        if state is None:
            raise ValueError("pool mode needs the pool in `state`")
        _state_pool(state, "state", (H, K, V), slot_stride)
        if final_state is not None and final_state is not state:
            raise ValueError("pool mode updates the pool: final_state must be None or the pool")
    else:
        if state is not None:
            _plain(state, "state", state.dtype, (N, H, K, V))
        if final_state is not None:
            want = final_state.dtype if state is None else state.dtype
            _plain(final_state, "final_state", want, (N, H, K, V))
    if out is not None:
        _plain(out, "out", dtype, (T, H, V))
    return N, T, H, G, K, V, pitches


def _ssm_inputs(x, dt, A_log, B, C, D, dt_bias, pitches):
    px, pd, pb, pc = pitches
    return KdaSsmInputs(_p(x), px, _p(dt), pd, _p(B), pb, _p(C), pc, _p(A_log), _p(dt_bias), _p(D))


def ssm_desc(N, T, H, G, K, V, qkv_dtype, state_dtype=torch.float32, num_slots=0, slot_stride=0,
             flags=0):
    """Descriptor of a scan call (scale and chunk size are not used)."""
    return KdaDesc(N, T, G, H, K, V, _dt(qkv_dtype), _dt(state_dtype), 0.0, 64, num_slots,
                   slot_stride, flags)


def ssm_scan_workspace_size(desc: KdaDesc) -> int:
    return int(_load().kda_ssm_scan_workspace_size(ctypes.byref(desc)))


def ssm_scan(x, dt, A_log, B, C, cu_seqlens, *, D=None, dt_bias=None, state=None,
             state_indices=None, final_state=None, output_final_state=True, slot_stride=0, out=None,
             workspace=None, stream=None, cuda_core_path=False):
    """Selective state space scan of packed sequences (kda_ssm_scan).  Returns ``(y, final)``.

    x [T, H, V], dt [T, H], B and C [T, G, K], bf16 or fp32 (one dtype), token rows at any pitch (x, B
    and C at 16-byte aligned ones); A_log, dt_bias, D [H] fp32 (the last two or None); cu_seqlens
    [N+1] int32.  K and V are 64 or 128; head h uses group h // (H // G).  States are [H, K, V], fp32 or
    bf16; pool and dense mode as in :func:`chunk_prefill`.
    """
    N, T, H, G, K, V, pitches = check_ssm_args(
        x, dt, A_log, B, C, D=D, dt_bias=dt_bias, cu_seqlens=cu_seqlens, state=state,
        state_indices=state_indices, final_state=final_state, out=out, slot_stride=slot_stride)
    _cuda(x, dt, A_log, B, C, D, dt_bias, cu_seqlens, state, state_indices, final_state, out, workspace)
    lib, dev = _load(), x.device
    pool = state_indices is not None
    sdt = state.dtype if state is not None else (
        final_state.dtype if final_state is not None else torch.float32)
    if pool:
        final_state = state
    elif final_state is None and output_final_state:
        final_state = _empty(stream, (N, H, K, V), sdt, dev)
    if out is None:
        out = _empty(stream, (T, H, V), x.dtype, dev)
    d = ssm_desc(N, T, H, G, K, V, x.dtype, sdt, state.shape[0] if pool else 0, slot_stride,
                 KDA_FLAG_CUDA_CORE_PATH if cuda_core_path else 0)
    size = lib.kda_ssm_scan_workspace_size(ctypes.byref(d))
    ws, nws = _workspace(stream, workspace, max(size, STATUS_WORKSPACE_BYTES), dev)
    ins = _ssm_inputs(x, dt, A_log, B, C, D, dt_bias, pitches)
    rc = lib.kda_ssm_scan(ctypes.byref(d), ctypes.byref(ins), _p(cu_seqlens), _p(state),
                          _p(state_indices), _p(final_state), _p(out), _p(ws), nws, _stream(stream, dev))
    _done(rc, "kda_ssm_scan", ssm_scan, ws)
    return out, final_state


def _ssm_token(x, dt, A_log, B, C, cu_seqlens, pool, state_indices, D, dt_bias, cache, max_steps,
               update_pool, slot_stride, out, workspace, stream, owner):
    N, T, H, G, K, V, pitches = check_ssm_args(
        x, dt, A_log, B, C, D=D, dt_bias=dt_bias, cu_seqlens=cu_seqlens, state=pool,
        state_indices=state_indices, out=out, slot_stride=slot_stride, token=True)
    _cuda(x, dt, A_log, B, C, D, dt_bias, cu_seqlens, pool, state_indices, cache, out, workspace)
    cpitch = 0
    if cache is not None:
        cpitch = _step_cache(cache, "cache", N, max_steps, H * K * V, pool.dtype)
    lib, dev = _load(), x.device
    if out is None:
        out = _empty(stream, (T, H, V), x.dtype, dev)
    ws, nws = _workspace(stream, workspace, STATUS_WORKSPACE_BYTES, dev)
    d = ssm_desc(N, T, H, G, K, V, x.dtype, pool.dtype, pool.shape[0], slot_stride)
    ins = _ssm_inputs(x, dt, A_log, B, C, D, dt_bias, pitches)
    rc = lib.kda_ssm_decode(ctypes.byref(d), ctypes.byref(ins), _p(cu_seqlens), _p(pool),
                            _p(state_indices), _p(cache), cpitch, max_steps, 1 if update_pool else 0,
                            _p(out), _p(ws), nws, _stream(stream, dev))
    _done(rc, "kda_ssm_decode", owner, ws)
    return out


def ssm_decode(x, dt, A_log, B, C, pool, state_indices=None, *, D=None, dt_bias=None, slot_stride=0,
               out=None, workspace=None, stream=None):
    """One scan step a row (kda_ssm_decode), updating ``pool`` [num_slots, H, K, V] in place; x
    [N, H, V], dt [N, H], B and C [N, G, K].  Returns y [N, H, V]."""
    return _ssm_token(x, dt, A_log, B, C, None, pool, state_indices, D, dt_bias, None, 1, True,
                      slot_stride, out, workspace, stream, ssm_decode)


def ssm_decode_draft(x, dt, A_log, B, C, cu_seqlens, pool, state_indices=None, *, D=None,
                     dt_bias=None, cache=None, max_steps=None, update_pool=False, slot_stride=0,
                     out=None, workspace=None, stream=None):
    """Scan steps of drafted tokens, as :func:`decode_draft`; ``cache`` [N, steps, H, K, V] gets the
    state after each.  Returns y [T, H, V]."""
    return _ssm_token(x, dt, A_log, B, C, cu_seqlens, pool, state_indices, D, dt_bias, cache,
                      _steps(cu_seqlens, max_steps, stream), update_pool, slot_stride, out, workspace, stream,
                      ssm_decode_draft)


# ------------------------------------------------------------------------ gated linear recurrence

CARRY_ROWS = 48  # KDA_GATED_CARRY_ROWS


def check_gated_args(x, r, A_log, *, i=None, cu_seqlens=None, state=None, state_indices=None,
                     final_state=None, out=None, slot_stride=0, token=False):
    """Checks of a gated recurrence's call (host only); returns (N, T, channels, pitches of x, r, i)."""
    if not isinstance(x, torch.Tensor) or x.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("x must be a bfloat16 or float32 tensor")
    if x.dim() != 2 or x.shape[1] < 1:
        raise ValueError(f"x must have shape [T, channels], got {list(x.shape)}")
    dtype = x.dtype
    T, ch = x.shape
    pitches = (_rows(x, "x", (T, ch), dtype), _rows(r, "r", (T, ch), dtype),
               ch if i is None else _rows(i, "i", (T, ch), dtype))
    _plain(A_log, "A_log", torch.float32, (ch,))
    N = T if cu_seqlens is None else _num_seqs(cu_seqlens)
    if state_indices is not None:
        _plain(state_indices, "state_indices", torch.int32, (N,))
    if token or state_indices is not None:
        if state is None:
            raise ValueError("pool mode needs the pool in `state`")
        _state_pool(state, "state", (ch,), slot_stride)
        if state.dtype is not torch.float32:
            raise TypeError(f"state must be float32, got {state.dtype}")
        if final_state is not None and final_state is not state:
            raise ValueError("pool mode updates the pool: final_state must be None or the pool")
    else:
        if state is not None:
            _plain(state, "state", torch.float32, (N, ch))
        if final_state is not None:
            _plain(final_state, "final_state", torch.float32, (N, ch))
    if out is not None:
        _plain(out, "out", dtype, (T, ch))
    return N, T, ch, pitches


def _gated_desc(N, T, ch, dtype, pitches, num_slots=0, slot_stride=0):
    return KdaGatedDesc(N, T, ch, _dt(dtype), *pitches, num_slots, slot_stride)


def gated_scan(x, r, A_log, cu_seqlens, *, i=None, state=None, state_indices=None, final_state=None,
               output_final_state=True, output_carries=False, slot_stride=0, out=None, workspace=None,
               stream=None):
    """Gated linear recurrence of packed sequences (kda_gated_scan), per channel
    ``h = a h + sqrt(1 - a^2) sigmoid(i) x`` with ``a = exp(-exp(A_log) sigmoid(r))``.  Returns
    ``(y, final)``, with ``output_carries`` ``(y, final, carries)``.

    x, r and i [T, Ch] bf16 or fp32 (one dtype), their rows at any pitch; i None: x enters whole; A_log
    [Ch] fp32; cu_seqlens [N+1] int32.  States are [Ch] fp32; pool and dense mode as in
    :func:`causal_conv`.  ``carries`` [ceil(T / 48), Ch] fp32 is what :func:`gated_scan_backward` wants of
    the forward pass.  A sequence's first row counts like any other: where a model lets x enter it whole, it is
    divided by sqrt(1 - a^2) beforehand.
    """
    N, T, ch, pitches = check_gated_args(
        x, r, A_log, i=i, cu_seqlens=cu_seqlens, state=state, state_indices=state_indices,
        final_state=final_state, out=out, slot_stride=slot_stride)
    _cuda(x, r, A_log, cu_seqlens, i, state, state_indices, final_state, out, workspace)
    lib, dev = _load(), x.device
    pool = state_indices is not None
    if pool:
        final_state = state
    elif final_state is None and output_final_state:
        final_state = _empty(stream, (N, ch), torch.float32, dev)
    if out is None:
        out = _empty(stream, (T, ch), x.dtype, dev)
    carries = None
    if output_carries:
        carries = _empty(stream, ((T + CARRY_ROWS - 1) // CARRY_ROWS, ch), torch.float32, dev)
    d = _gated_desc(N, T, ch, x.dtype, pitches, state.shape[0] if pool else 0, slot_stride)
    size = lib.kda_gated_scan_workspace_size(ctypes.byref(d))
    ws, nws = _workspace(stream, workspace, max(size, STATUS_WORKSPACE_BYTES), dev)
    rc = lib.kda_gated_scan(ctypes.byref(d), _p(x), _p(r), _p(i), _p(A_log), _p(cu_seqlens), _p(state),
                            _p(state_indices), _p(final_state), _p(out), _p(carries), _p(ws), nws,
                            _stream(stream, dev))
    _done(rc, "kda_gated_scan", gated_scan, ws)
    return (out, final_state, carries) if output_carries else (out, final_state)


def gated_scan_backward(dy, x, r, A_log, cu_seqlens, carries, *, i=None, state=None, dfinal=None,
                        workspace=None, stream=None):
    """The derivatives of a loss by the inputs of a dense :func:`gated_scan` (kda_gated_scan_backward), from
    those by y (``dy`` [T, Ch], rows at any pitch) and by the final states (``dfinal`` [N, Ch] fp32 or None).
    Returns ``(dx, dr, di, dA_log, dstate)``: di None without i, dA_log [Ch] fp32, dstate [N, Ch] fp32 or
    None without ``state``.

    x, r, A_log, cu_seqlens, i and state as the forward call had them, carries as it returned them.
    """
    N, T, ch, pitches = check_gated_args(x, r, A_log, i=i, cu_seqlens=cu_seqlens, state=state)
    dy_pitch = _rows(dy, "dy", (T, ch), x.dtype)
    _plain(carries, "carries", torch.float32, ((T + CARRY_ROWS - 1) // CARRY_ROWS, ch))
    if dfinal is not None:
        _plain(dfinal, "dfinal", torch.float32, (N, ch))
    _cuda(dy, x, r, A_log, cu_seqlens, carries, i, state, dfinal, workspace)
    lib, dev = _load(), x.device
    dx, dr = (_empty(stream, (T, ch), x.dtype, dev) for _ in range(2))
    di = None if i is None else _empty(stream, (T, ch), x.dtype, dev)
    da_log = _empty(stream, (ch,), torch.float32, dev)
    dstate = None if state is None else _empty(stream, (N, ch), torch.float32, dev)
    d = _gated_desc(N, T, ch, x.dtype, pitches)
    size = lib.kda_gated_scan_backward_workspace_size(ctypes.byref(d))
    ws, nws = _workspace(stream, workspace, max(size, STATUS_WORKSPACE_BYTES), dev)
    rc = lib.kda_gated_scan_backward(ctypes.byref(d), _p(dy), dy_pitch, _p(x), _p(r), _p(i), _p(A_log),
                                     _p(cu_seqlens), _p(carries), _p(state), _p(dfinal), _p(dx), _p(dr),
                                     _p(di), _p(da_log), _p(dstate), _p(ws), nws, _stream(stream, dev))
    _done(rc, "kda_gated_scan_backward", gated_scan_backward, ws)
    return dx, dr, di, da_log, dstate


def _gated_token(x, r, A_log, cu_seqlens, pool, state_indices, i, cache, max_steps, update_pool, slot_stride,
                 out, workspace, stream, owner):
    N, T, ch, pitches = check_gated_args(x, r, A_log, i=i, cu_seqlens=cu_seqlens, state=pool,
                                         state_indices=state_indices, out=out, slot_stride=slot_stride,
                                         token=True)
    _cuda(x, r, A_log, i, cu_seqlens, pool, state_indices, cache, out, workspace)
    cpitch = 0
    if cache is not None:
        cpitch = _step_cache(cache, "cache", N, max_steps, ch, torch.float32)
    lib, dev = _load(), x.device
    if out is None:
        out = _empty(stream, (T, ch), x.dtype, dev)
    ws, nws = _workspace(stream, workspace, STATUS_WORKSPACE_BYTES, dev)
    d = _gated_desc(N, T, ch, x.dtype, pitches, pool.shape[0], slot_stride)
    rc = lib.kda_gated_decode(ctypes.byref(d), _p(x), _p(r), _p(i), _p(A_log), _p(cu_seqlens), _p(pool),
                              _p(state_indices), _p(cache), cpitch, max_steps, 1 if update_pool else 0, _p(out),
                              _p(ws), nws, _stream(stream, dev))
    _done(rc, "kda_gated_decode", owner, ws)
    return out


def gated_decode(x, r, A_log, pool, state_indices=None, *, i=None, slot_stride=0, out=None, workspace=None,
                 stream=None):
    """One step of the gated recurrence a row (kda_gated_decode), updating ``pool`` [num_slots, Ch] fp32 in
    place; x, r and i [N, Ch].  Returns y [N, Ch]."""
    return _gated_token(x, r, A_log, None, pool, state_indices, i, None, 1, True, slot_stride, out, workspace,
                        stream, gated_decode)


def gated_decode_draft(x, r, A_log, cu_seqlens, pool, state_indices=None, *, i=None, cache=None,
                       max_steps=None, update_pool=False, slot_stride=0, out=None, workspace=None,
                       stream=None):
    """Steps of the gated recurrence of drafted tokens, as :func:`decode_draft`; ``cache`` [N, steps, Ch]
    fp32 gets the state after each.  Returns y [T, Ch]."""
    return _gated_token(x, r, A_log, cu_seqlens, pool, state_indices, i, cache,
                        _steps(cu_seqlens, max_steps, stream), update_pool, slot_stride, out, workspace, stream,
                        gated_decode_draft)


# ------------------------------------------------------------------------ draw of tokens

def _param(value, name, n, dtype, off):
    """A parameter of each row ([n] tensor), or of all (a number; None: ``off``): (tensor, number)."""
    if isinstance(value, torch.Tensor):
        _plain(value, name, dtype, (n,))
        return value, off
    if value is None:
        return None, off
    if isinstance(value, bool) or not isinstance(value, (int,) if dtype is torch.int32 else (int, float)):
        raise TypeError(f"{name} must be a number or a tensor of {dtype}, got {value!r}")
    if value != value or (dtype is torch.int32 and not -2 ** 31 <= value < 2 ** 31):
        raise ValueError(f"{name} must be a number within its type, got {value!r}")
    return None, value


def _draw_args(logits, temperature, top_k, top_p, min_p):
    """Checks of a draw's call (host only); returns (rows, vocab, parameters' tensors, descriptor)."""
    if not isinstance(logits, torch.Tensor) or logits.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("logits must be a bfloat16 or float32 tensor")
    if logits.dim() != 2 or logits.shape[1] < 1:
        raise ValueError(f"logits must have shape [rows, vocab], got {list(logits.shape)}")
    n, vocab = logits.shape
    pitch = _rows(logits, "logits", (n, vocab), logits.dtype)
    t, t_all = _param(temperature, "temperature", n, torch.float32, 1.0)
    k, k_all = _param(top_k, "top_k", n, torch.int32, 0)
    p, p_all = _param(top_p, "top_p", n, torch.float32, 1.0)
    m, m_all = _param(min_p, "min_p", n, torch.float32, 0.0)
    if t_all < 0:
        raise ValueError(f"temperature must not be negative, got {t_all!r}")
    return n, vocab, (t, k, p, m), KdaSampleDesc(n, vocab, _dt(logits.dtype), pitch, vocab, t_all, k_all, p_all,
                                                 m_all)


def sample(logits, noise, *, temperature=None, top_k=None, top_p=None, min_p=None, out=None, workspace=None,
           stream=None):
    """A token a row from logits and given random numbers (kda_sample).  Returns int32 [rows].

    logits [rows, vocab] bf16 or fp32, noise [rows, vocab] fp32 ~ Exp(1), rows of both at any pitch; each
    parameter a number for all rows, or a tensor of one a row (top_k int32, the others fp32).  The first
    top_k entries by value (then index), of these the first whose probabilities sum up to top_p, and of
    these those of at least min_p of the largest one's probability stand; of them the one with the largest
    probability over noise is drawn.  Temperature 0: the largest.  -1 for a row with nothing to draw from.
    """
    n, vocab, params, d = _draw_args(logits, temperature, top_k, top_p, min_p)
    d.noise_pitch = _rows(noise, "noise", (n, vocab), torch.float32)
    if out is not None:
        _plain(out, "out", torch.int32, (n,))
    _cuda(logits, noise, *params, out, workspace)
    lib, dev = _load(), logits.device
    if out is None:
        out = _empty(stream, (n,), torch.int32, dev)
    ws, nws = _workspace(stream, workspace, STATUS_WORKSPACE_BYTES, dev)
    rc = lib.kda_sample(ctypes.byref(d), _p(logits), _p(noise), *map(_p, params), _p(out), _p(ws), nws,
                        _stream(stream, dev))
    _done(rc, "kda_sample", sample, ws)
    return out


def sample_probs(logits, *, temperature=None, top_k=None, top_p=None, min_p=None, out=None, workspace=None,
                 stream=None):
    """The probabilities that :func:`sample` draws with (kda_sample_probs), [rows, vocab] fp32, 0 for entries
    that do not stand: what :func:`verify_draft` wants of the target and of the draft."""
    n, vocab, params, d = _draw_args(logits, temperature, top_k, top_p, min_p)
    if out is not None:
        _plain(out, "out", torch.float32, (n, vocab))
    _cuda(logits, *params, out, workspace)
    lib, dev = _load(), logits.device
    if out is None:
        out = _empty(stream, (n, vocab), torch.float32, dev)
    ws, nws = _workspace(stream, workspace, STATUS_WORKSPACE_BYTES, dev)
    rc = lib.kda_sample_probs(ctypes.byref(d), _p(logits), *map(_p, params), _p(out), _p(ws), nws,
                              _stream(stream, dev))
    _done(rc, "kda_sample_probs", sample_probs, ws)
    return out


# ------------------------------------------------------------------------ drafted tokens

def verify_draft(tokens, target_probs, draft_probs, accept_u, noise, cu_seqlens, *,
                 num_accepted=None, next_token=None, mark_skipped=None, workspace=None, stream=None):
    """Drafted tokens against the target's probabilities from given random numbers
    (kda_verify_draft).  Returns ``(num_accepted, next_token)``, int32 [N].

    tokens [T] int32: for each request its last sampled token, then the drafted ones; target_probs
    [T, vocab] fp32, row t following token t; draft_probs the same of the draft, or None for drafts
    made without drawing; accept_u [T] fp32 in [0, 1); noise [N, vocab] fp32 ~ Exp(1); cu_seqlens
    [N+1] int32.  num_accepted counts the tokens of a request that stand, the first among them: the
    step that :func:`commit_draft` keeps.  A request that is skipped (a drafted token outside the
    vocabulary, bad lengths: see the status word) gets 0 and -1 in outputs made here; outputs given
    (``num_accepted``, ``next_token`` [N] int32) keep what they hold for it, unless ``mark_skipped``
    is True.
    """
    if not isinstance(target_probs, torch.Tensor) or target_probs.dim() != 2:
        raise ValueError("target_probs must have shape [T, vocab]")
    T, vocab = target_probs.shape
    if vocab == 0:
        raise ValueError("target_probs has no entries")
    _plain(tokens, "tokens", torch.int32, (T,))
    _plain(target_probs, "target_probs", torch.float32, (T, vocab))
    if draft_probs is not None:
        _plain(draft_probs, "draft_probs", torch.float32, (T, vocab))
    _plain(accept_u, "accept_u", torch.float32, (T,))
    N = _num_seqs(cu_seqlens)
    _plain(noise, "noise", torch.float32, (N, vocab))
    if num_accepted is not None:
        _plain(num_accepted, "num_accepted", torch.int32, (N,))
    if next_token is not None:
        _plain(next_token, "next_token", torch.int32, (N,))
    _cuda(tokens, target_probs, draft_probs, accept_u, noise, cu_seqlens, num_accepted, next_token, workspace)
    lib, dev = _load(), tokens.device
    flags = 3 if mark_skipped else 0  # KDA_VERIFY_MARK_COUNT, KDA_VERIFY_MARK_TOKEN
    if num_accepted is None:
        num_accepted = _empty(stream, (N,), torch.int32, dev)
        flags |= 1
    if next_token is None:
        next_token = _empty(stream, (N,), torch.int32, dev)
        flags |= 2
    ws, nws = _workspace(stream, workspace, STATUS_WORKSPACE_BYTES, dev)
    rc = lib.kda_verify_draft_marked(N, T, vocab, _p(tokens), _p(target_probs), _p(draft_probs),
                                     _p(accept_u), _p(noise), _p(cu_seqlens), _p(num_accepted),
                                     _p(next_token), flags, _p(ws), nws, _stream(stream, dev))
    _done(rc, "kda_verify_draft", verify_draft, ws)
    return num_accepted, next_token


def commit_draft(cache, num_accepted, pool, state_indices=None, *, slot_stride=0, workspace=None,
                 stream=None):
    """Copies each request's state after its accepted tokens, ``cache[n, num_accepted[n] - 1]``, into
    its slot of ``pool`` (kda_commit_draft); nothing for a count of 0.  cache [N, steps, *row] of any
    step cache (rows packed, requests at any pitch); pool [num_slots, *row], or with ``slot_stride`` a
    buffer of pool.shape[0] slots that many elements apart, as the draft steps take it.  Returns the
    pool."""
    if not (isinstance(pool, torch.Tensor) and pool.is_contiguous()):
        _need(pool, "pool", cuda=False)
    shape = pool.shape
    if len(shape) < 1 or shape[0] == 0 or pool.numel() == 0 or (len(shape) < 2 and slot_stride == 0):
        raise ValueError(f"pool must have shape [num_slots, *row], got {list(shape)}")
    if not isinstance(cache, torch.Tensor) or cache.dim() < 3 or cache.shape[1] == 0 or \
            (slot_stride == 0 and cache.shape[2:] != shape[1:]):
        raise ValueError("cache must have shape [N, steps, *row] with the pool's rows")
    if not isinstance(num_accepted, torch.Tensor) or num_accepted.dim() != 1:
        raise TypeError("num_accepted must be an int32 tensor of one dimension")
    N, steps, row = num_accepted.shape[0], cache.shape[1], cache.shape[2:].numel()
    if slot_stride != 0:
        _state_pool(pool, "pool", cache.shape[2:], slot_stride)
    _plain(num_accepted, "num_accepted", torch.int32, (N,))
    pitch = _step_cache(cache, "cache", N, steps, row, pool.dtype)
    if state_indices is not None:
        _plain(state_indices, "state_indices", torch.int32, (N,))
    _cuda(cache, num_accepted, pool, state_indices, workspace)
    lib, dev = _load(), pool.device
    ws, nws = _workspace(stream, workspace, STATUS_WORKSPACE_BYTES, dev)
    rc = lib.kda_commit_draft(N, _dt(pool.dtype), row, _p(cache), pitch, steps, _p(num_accepted),
                              _p(pool), shape[0], slot_stride, _p(state_indices), _p(ws), nws,
                              _stream(stream, dev))
    _done(rc, "kda_commit_draft", commit_draft, ws)
    return pool
