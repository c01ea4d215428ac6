"""Binding of the calls around the recurrence: the short convolution, the
selective scan and the 8-bit state cache (``include/kda.h``).

As in ``_native``: argument checks, output and workspace allocation with
torch, raw pointers and torch's current stream; the work is in ``libkda.so``.
Token matrices may be column ranges of wider ones (rows of unit-stride
elements); weights and states are contiguous.
"""
from __future__ import annotations

import ctypes

import torch

from ._native import KDA_BF16, KDA_F32, KDA_OK, KdaError, SsmIo, _host_cu, load

_ACTS = {None: 0, "none": 0, "silu": 1}
_FORMATS = {torch.int8: 0, torch.float8_e4m3fn: 1}


def _dtype(t, name):
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_F32
    raise TypeError("%s must be float32 or bfloat16, got %s" % (name, t.dtype))


def _act(activation):
    if activation not in _ACTS:
        raise ValueError("activation must be \"silu\" or None, got %r" % (activation,))
    return _ACTS[activation]


def _rows(t, shape, dtype, name):
    """A token matrix: `shape` with dense rows; returns its row stride."""
    if t.shape != shape:
        raise ValueError("%s must have shape %s (got %s)" % (name, tuple(shape), tuple(t.shape)))
    if t.dtype != dtype:
        raise ValueError("%s must be %s (got %s)" % (name, dtype, t.dtype))
    width = shape[1] if len(shape) == 2 else shape[1] * shape[2]
    if t.is_contiguous():
        return width
    st = t.stride()
    if (shape[-1] != 1 and st[-1] != 1) or \
            (len(shape) == 3 and shape[1] != 1 and st[1] != shape[2]):
        raise ValueError("%s must have dense rows (strides %s)" % (name, st))
    # (a single row's stride is whatever torch left there)
    return st[0] if shape[0] > 1 else max(width, st[0])


def _dense(t, shape, dtype, name):
    if t is None:
        return
    if t.shape != shape:
        raise ValueError("%s must have shape %s (got %s)" % (name, tuple(shape), tuple(t.shape)))
    if t.dtype != dtype:
        raise ValueError("%s must be %s (got %s)" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _device(first, *ts):
    """The device of all tensors (None among `ts` left out)."""
    at = first.get_device()
    if at < 0:
        raise ValueError("KDA tensors must live on a HIP device")
    for t in ts:
        if t is not None and t.get_device() != at:
            if t.get_device() < 0:
                raise ValueError("KDA tensors must live on a HIP device")
            raise ValueError("all KDA tensors must be on one device")
    return first.device


def _count(n, name):
    """A count that the library takes in 32 bits (ctypes would wrap it)."""
    if n > 0x7fffffff:
        raise ValueError("%s must be below 2^31 (got %d)" % (name, n))
    return n


def _like(x):
    """A dense output of x's shape, type and device."""
    return torch.empty_like(x) if x.is_contiguous() else \
        torch.empty(x.shape, dtype=x.dtype, device=x.device)


def _p(t):
    return None if t is None else t.data_ptr()


def _call(name, dev, *args):
    """``name`` of the library with `args` and the current stream of `dev`,
    which is made the current device while the call runs; raises on a status."""
    fn = getattr(load(), name)
    # (torch.cuda.current_stream builds a Stream object: 2.8 us against 0.1)
    stream = torch._C._cuda_getCurrentRawStream(dev.index)
    if dev.index == torch.cuda.current_device():
        st = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, stream)
    if st != KDA_OK:
        raise KdaError(st, name)


def _slots(slots, count, name="slots"):
    if slots is None:
        return
    if slots.dtype != torch.int32 or slots.shape != (count,) or not slots.is_contiguous():
        raise ValueError("%s must be contiguous int32 [%d]" % (name, count))


def _pools(initial, final, count, slots, tail, dtype):
    """Checks prompt state buffers; returns their slice count."""
    num = count
    for t, name in ((initial, "initial_state"), (final, "final_state")):
        if t is None:
            continue
        num = t.shape[0] if slots is not None and t.dim() > 0 else count
        _dense(t, (num,) + tail, dtype, name)
    if initial is not None and final is not None and initial.shape != final.shape:
        raise ValueError("initial_state and final_state must have one shape")
    return _count(num, "the number of state slices")


def _bounds(cu_seqlens, T):
    cu = _host_cu(cu_seqlens, T)
    if int(cu[-1]) != T:
        raise ValueError("cu_seqlens[-1] must equal the number of tokens")
    return cu


def _workspace(workspace, nbytes, dev):
    if nbytes == 0:
        return None
    if workspace is None or workspace.numel() < nbytes:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous uint8")
    return workspace


def short_conv(x, weight, bias=None, cu_seqlens=None, initial_state=None,
               output_final_state: bool = True, activation="silu", slots=None, y=None,
               final_state=None, workspace=None):
    """Short causal depthwise convolution over packed sequences
    (``kda_short_conv``).

    x ``[T, D]``, weight ``[D, W]``, bias ``[D]`` or None, all of one dtype;
    ``activation`` "silu" or None.  initial_state, final_state ``[N, W - 1,
    D]`` of x's dtype (oldest input first); with ``slots`` (int32 ``[N]`` on
    the device) they are pools of any number of slices, and final_state is
    written only if it is passed.  Returns ``(y, final_state or None)``.
    """
    T, D = x.shape
    W = weight.shape[-1]
    code = _dtype(x, "x")
    dt = x.dtype
    xs = _rows(x, (T, D), dt, "x")
    _dense(weight, (D, W), dt, "weight")
    _dense(bias, (D,), dt, "bias")
    act = _act(activation)
    cu = _bounds(cu_seqlens, T)
    n = cu.size - 1
    _slots(slots, n)
    pool = _pools(initial_state, final_state, n, slots, (W - 1, D), dt)
    ys = D if y is None else _rows(y, (T, D), dt, "y")
    dev = _device(x, weight, bias, initial_state, final_state, slots, y, workspace)
    if y is None:
        y = _like(x)
    if final_state is None and output_final_state and slots is None:
        final_state = torch.empty((n, W - 1, D), dtype=dt, device=dev)
    lib = load()
    ws = _workspace(workspace, lib.kda_short_conv_workspace_size(n), dev)
    _call("kda_short_conv", dev, n, cu.ctypes.data, D, W, code, _p(x), xs, _p(weight), _p(bias), act,
          _p(initial_state), _p(final_state), _p(slots), pool, _p(y), ys,
          _p(ws), 0 if ws is None else ws.numel())
    return y, final_state


def short_conv_step(state, x, weight, bias=None, activation="silu", slots=None, y=None):
    """The convolution for one token per row (``kda_short_conv_step``): x
    ``[N, D]``, state ``[N, W - 1, D]`` (or a pool of slices with ``slots``)
    shifted in place.  Rows whose slot is out of range are skipped, their
    output left as it was.  ``y`` may be x.  Returns y."""
    N, D = x.shape
    W = weight.shape[-1]
    code = _dtype(x, "x")
    dt = x.dtype
    xs = _rows(x, (N, D), dt, "x")
    _dense(weight, (D, W), dt, "weight")
    _dense(bias, (D,), dt, "bias")
    act = _act(activation)
    _slots(slots, N)
    pool = _count(N, "the number of rows")
    if slots is not None:
        pool = _count(state.shape[0], "the number of state slices")
    _dense(state, (pool, W - 1, D), dt, "state")
    ys = D if y is None else _rows(y, (N, D), dt, "y")
    dev = _device(x, weight, bias, state, slots, y)
    if y is None:
        y = _like(x)
    _call("kda_short_conv_step", dev, N, D, W, code, _p(x), xs, _p(weight), _p(bias), act,
          _p(state), _p(slots), pool, _p(y), ys)
    return y


def _ssm_io(x, delta, A, B, C, D, z, delta_bias, delta_softplus, y):
    """The scan's argument block, checked; y still to be filled in if None."""
    rows, ch = x.shape
    code = _dtype(x, "x")
    dt = x.dtype
    if A.dim() != 2 or B.dim() != 3:
        raise ValueError("A must be [D, N] and B, C [rows, G, N]")
    N, G = A.shape[1], B.shape[1]
    if G < 1 or ch % G != 0:
        raise ValueError("the number of channels must be a multiple of B's groups")
    f32 = torch.float32
    io = SsmIo()
    io.x_stride = _rows(x, (rows, ch), dt, "x")
    io.delta_stride = _rows(delta, (rows, ch), dt, "delta")
    io.B_stride = _rows(B, (rows, G, N), dt, "B")
    io.C_stride = _rows(C, (rows, G, N), dt, "C")
    if z is not None:
        io.z_stride = _rows(z, (rows, ch), dt, "z")
    _dense(A, (ch, N), f32, "A")
    _dense(D, (ch,), f32, "D")
    _dense(delta_bias, (ch,), f32, "delta_bias")
    io.y_stride = ch if y is None else _rows(y, (rows, ch), dt, "y")
    io.x, io.delta, io.B, io.C, io.z = _p(x), _p(delta), _p(B), _p(C), _p(z)
    io.A, io.D_skip, io.delta_bias = _p(A), _p(D), _p(delta_bias)
    io.delta_softplus = 1 if delta_softplus else 0
    return io, rows, ch, N, G, code


def selective_scan(x, delta, A, B, C, D=None, z=None, delta_bias=None,
                   delta_softplus: bool = True, cu_seqlens=None, initial_state=None,
                   output_final_state: bool = True, split_hint: int = 0, slots=None, y=None,
                   final_state=None, workspace=None):
    """Selective state space scan over packed sequences
    (``kda_selective_scan``).

    x, delta and the optional gate z ``[T, D]``, B and C ``[T, G, N]``, of one
    dtype; A ``[D, N]``, the optional skip D ``[D]`` and delta_bias ``[D]`` in
    fp32.  initial_state, final_state ``[N_seqs, D, N]`` fp32; with ``slots``
    (int32 on the device) they are pools of any number of slices, and
    final_state is written only if it is passed.  ``split_hint``: as in
    include/kda.h.  Returns ``(y, final_state or None)``.
    """
    io, T, ch, N, G, code = _ssm_io(x, delta, A, B, C, D, z, delta_bias, delta_softplus, y)
    cu = _bounds(cu_seqlens, T)
    n = cu.size - 1
    split = _count(int(split_hint), "split_hint")
    _slots(slots, n)
    pool = _pools(initial_state, final_state, n, slots, (ch, N), torch.float32)
    dev = _device(x, delta, A, B, C, D, z, delta_bias, initial_state, final_state, slots, y,
                  workspace)
    if y is None:
        y = _like(x)
    io.y = _p(y)
    if final_state is None and output_final_state and slots is None:
        final_state = torch.empty((n, ch, N), dtype=torch.float32, device=dev)
    lib = load()
    cup = cu.ctypes.data
    ws = _workspace(workspace, lib.kda_selective_scan_workspace_size(n, cup, ch, N, G, split), dev)
    _call("kda_selective_scan", dev, n, cup, ch, N, G, code, ctypes.byref(io), _p(initial_state),
          _p(final_state), _p(slots), pool, split, _p(ws),
          0 if ws is None else ws.numel())
    return y, final_state


def selective_scan_step(state, x, delta, A, B, C, D=None, z=None, delta_bias=None,
                        delta_softplus: bool = True, slots=None, y=None):
    """The scan for one token per row (``kda_selective_scan_step``): the
    arguments of ``selective_scan`` with one row per sequence, state ``[rows,
    D, N]`` fp32 (or a pool of slices with ``slots``) updated in place.  Rows
    whose slot is out of range are skipped, their output left as it was.
    Returns y."""
    io, rows, ch, N, G, code = _ssm_io(x, delta, A, B, C, D, z, delta_bias, delta_softplus, y)
    _slots(slots, rows)
    pool = _count(rows, "the number of rows")
    if slots is not None:
        pool = _count(state.shape[0], "the number of state slices")
    _dense(state, (pool, ch, N), torch.float32, "state")
    dev = _device(x, delta, A, B, C, D, z, delta_bias, state, slots, y)
    if y is None:
        y = _like(x)
    io.y = _p(y)
    _call("kda_selective_scan_step", dev, rows, ch, N, G, code, ctypes.byref(io), _p(state),
          _p(slots), pool)
    return y


def _cache_args(state, codes, scales, src, dst, store):
    if codes.dtype not in _FORMATS:
        raise TypeError("codes must be int8 or float8_e4m3fn, got %s" % codes.dtype)
    if state.dim() < 2 or codes.dim() != state.dim() or codes.shape[1:] != state.shape[1:]:
        raise ValueError("state [items, ..., L] and codes [slots, ..., L] must agree past the "
                         "first dimension")
    _dense(state, state.shape, torch.float32, "state")
    _dense(codes, codes.shape, codes.dtype, "codes")
    _dense(scales, codes.shape[:-1], torch.float32, "scales")
    items = _count(state.shape[0], "the number of states")
    held = _count(codes.shape[0], "the number of slots")
    n_from, n_to = (items, held) if store else (held, items)
    n = items
    if src is not None or dst is not None:
        n = _count(src.numel() if src is not None else dst.numel(), "the number of entries")
    elif held < n:
        raise ValueError("codes hold %d slots for %d states" % (held, n))
    _slots(src, n, "src")
    _slots(dst, n, "dst")
    L = _count(state.shape[-1], "the row length")
    R = 1
    for v in state.shape[1:-1]:
        R *= v
    if R * L == 0:
        n = 0
    return n, max(R, 1), max(L, 1), _FORMATS[codes.dtype], n_from, n_to


def state_store(state, codes, scales, src=None, dst=None):
    """Quantise fp32 states into an 8-bit cache (``kda_state_store``).

    state ``[items, ..., L]`` fp32, codes ``[slots, ..., L]`` int8 or
    float8_e4m3fn, scales ``[slots, ...]`` fp32 (one per row of L values).
    Item ``src[i]`` goes to slot ``dst[i]`` (int32 on the device; None: i);
    as many items move as the tables have entries, without tables all of
    ``state``.  Pairs with an entry out of range are skipped.  Slots that are
    not named keep what they hold."""
    n, R, L, fmt, n_from, n_to = _cache_args(state, codes, scales, src, dst, True)
    dev = _device(state, codes, scales, src, dst)
    _call("kda_state_store", dev, n, R, L, fmt, _p(state), _p(src), n_from, _p(codes),
          _p(scales), _p(dst), n_to)


def state_load(codes, scales, state, src=None, dst=None):
    """Read states back from an 8-bit cache (``kda_state_load``): slot
    ``src[i]`` of codes and scales becomes item ``dst[i]`` of state; shapes and
    entries as in ``state_store``.  Returns state."""
    n, R, L, fmt, n_from, n_to = _cache_args(state, codes, scales, src, dst, False)
    dev = _device(state, codes, scales, src, dst)
    _call("kda_state_load", dev, n, R, L, fmt, _p(codes), _p(scales), _p(src), n_from,
          _p(state), _p(dst), n_to)
    return state
