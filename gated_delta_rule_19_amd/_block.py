"""Binding of a decoder block's calls beside the KDA layer: the decayed
attention, the block norm, beam selection and state reordering
(``include/kda.h``).

As in ``_recurrent``: argument checks, output and workspace allocation with
torch, raw pointers and torch's current stream; the work is in ``libkda.so``.
"""
from __future__ import annotations

import ctypes

import torch

from ._native import DecayIo, NormIo, load
from ._recurrent import (_bounds, _call, _count, _dense, _device, _dtype, _p, _pools, _rows,
                         _slots, _workspace)

_ORDERS = {"score": 0, "rows": 1}
_MAX_STATES = 32


def _new(like, shape, dtype):
    """A dense output on like's device (torch makes one of like's shape in 1.15
    us, one from a shape in 1.65)."""
    if like.shape == shape and like.is_contiguous():
        return torch.empty_like(like, dtype=dtype)
    return torch.empty(shape, dtype=dtype, device=like.device)


def _decay_io(q, k, v, g, scale, o):
    """The attention's argument block, checked; o still to be filled in if None."""
    for x, name in ((q, "q"), (k, "k"), (v, "v")):
        if x.dim() != 3:
            raise ValueError("%s must be [tokens, heads, size] (got %s)" % (name, tuple(x.shape)))
    rows, Hq, dk = q.shape
    Hk, (_, Hv, dv) = k.shape[1], v.shape
    if g.dim() not in (1, 2):
        raise ValueError("g must be [tokens, H] or [H] (got %s)" % (tuple(g.shape),))
    H = _count(g.shape[-1], "the number of heads")
    code = _dtype(q, "q")
    dt = q.dtype
    for few, name in ((Hq, "q"), (Hk, "k"), (Hv, "v")):
        if few < 1 or H % few != 0:
            raise ValueError("the decay's %d heads must be a multiple of %s's %d" % (H, name, few))
    qs = _rows(q, (rows, Hq, dk), dt, "q")
    ks = _rows(k, (rows, Hk, dk), dt, "k")
    vs = _rows(v, (rows, Hv, dv), dt, "v")
    gs = 0
    if g.dim() == 2:
        gs = _rows(g, (rows, H), torch.float32, "g")
    else:
        _dense(g, (H,), torch.float32, "g")
    os = H * dv if o is None else _rows(o, (rows, H, dv), dt, "o")
    # (in one go: a field set by name costs more than the checks)
    io = DecayIo(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), None, qs, ks, vs, gs, os,
                 Hq, Hk, Hv, _count(dk, "q's size"), _count(dv, "v's size"), float(scale))
    return io, rows, H, dk, dv, code


def decay_attention(q, k, v, g, scale: float = 1.0, cu_seqlens=None, initial_state=None,
                    output_final_state: bool = True, split_hint: int = 0, slots=None, o=None,
                    final_state=None, workspace=None):
    """Linear attention with one decay a head over packed sequences
    (``kda_decay_attention``): ``S_t = exp(g_t) S_{t-1} + k_t v_t^T``,
    ``o_t = scale S_t^T q_t``.

    q ``[T, Hq, dk]``, k ``[T, Hk, dk]``, v ``[T, Hv, dv]`` of one dtype; g
    ``[T, H]`` or ``[H]`` fp32, the natural logarithm of the decay; Hq, Hk and
    Hv each divide H (shared heads).  initial_state, final_state ``[N, H, dk,
    dv]`` fp32; with ``slots`` (int32 ``[N]`` on the device) they are pools of
    any number of slices, and final_state is written only if it is passed.
    ``split_hint``: as in include/kda.h.  Returns ``(o [T, H, dv], final_state
    or None)``.
    """
    io, T, H, dk, dv, code = _decay_io(q, k, v, g, scale, o)
    cu = _bounds(cu_seqlens, T)
    n = cu.size - 1
    split = _count(int(split_hint), "split_hint")
    _slots(slots, n)
    pool = _pools(initial_state, final_state, n, slots, (H, dk, dv), torch.float32)
    dev = _device(q, k, v, g, initial_state, final_state, slots, o, workspace)
    if o is None:
        o = _new(v, (T, H, dv), q.dtype)
    io.o = _p(o)
    if final_state is None and output_final_state and slots is None:
        final_state = torch.empty((n, H, dk, dv), dtype=torch.float32, device=dev)
    cup = cu.ctypes.data
    ws = _workspace(workspace, load().kda_decay_attention_workspace_size(n, cup, H, dk, dv, code,
                                                                         split), dev)
    _call("kda_decay_attention", dev, n, cup, H, code, ctypes.byref(io), _p(initial_state),
          _p(final_state), _p(slots), pool, split, _p(ws), 0 if ws is None else ws.numel())
    return o, final_state


def decay_attention_step(state, q, k, v, g, scale: float = 1.0, slots=None, o=None):
    """The attention for one token per row (``kda_decay_attention_step``): the
    arguments of ``decay_attention`` with one row per sequence, state ``[rows,
    H, dk, dv]`` fp32 (or a pool of slices with ``slots``) updated in place.
    Rows whose slot is out of range are skipped, their output left as it was.
    Returns o."""
    io, rows, H, dk, dv, code = _decay_io(q, k, v, g, scale, o)
    _slots(slots, rows)
    pool = _count(rows, "the number of rows")
    if slots is not None:
        pool = _count(state.shape[0], "the number of state slices")
    _dense(state, (pool, H, dk, dv), torch.float32, "state")
    dev = _device(q, k, v, g, state, slots, o)
    if o is None:
        o = _new(v, (rows, H, dv), q.dtype)
    io.o = _p(o)
    _call("kda_decay_attention_step", dev, rows, H, code, ctypes.byref(io), _p(state), _p(slots),
          pool)
    return o


def block_norm(x, weight=None, eps: float = 1e-6, residual=None, scale=1.0, gate=None,
               post_weight=None, post_eps: float = 1e-6, residual_out=None, y=None):
    """Norm after a block, its gate and scaled residual, and the norm before
    the next block (``kda_block_norm``)::

        u = rmsnorm(x) * post_weight     (post_weight None: u = x)
        u = u * sigmoid(gate)            (gate None: not gated)
        r = residual + scale * u         (residual None: r = scale * u)
        y = rmsnorm(r) * weight          (weight None: no y)

    x, gate and y ``[rows, D]`` of one dtype, residual and r ``[rows, D]`` of
    residual's dtype (x's without one); weights fp32 ``[D]``; scale a number
    or fp32 ``[D]``.  Weights and a scale ``[D]`` start at multiples of 16
    bytes: others (slices of larger parameters, for instance) are refused.
    ``residual_out`` (it may be residual itself) and ``y`` take the outputs.
    Returns ``(r, y or None)``; r is not written where neither residual nor
    residual_out is given and y is formed: then ``(None, y)``.
    """
    if x.dim() != 2:
        raise ValueError("x must be [rows, D] (got %s)" % (tuple(x.shape),))
    rows, D = x.shape
    code = _dtype(x, "x")
    dt = x.dtype
    if y is not None and weight is None:
        raise ValueError("y needs weight")
    rdt = residual.dtype if residual is not None else \
        residual_out.dtype if residual_out is not None else dt
    rcode = code if rdt == dt else _dtype(
        residual if residual is not None else residual_out, "residual")
    shape = (rows, D)
    xs = _rows(x, shape, dt, "x")
    gs = rs = ros = ys = 0
    if gate is not None:
        gs = _rows(gate, shape, dt, "gate")
    if residual is not None:
        rs = _rows(residual, shape, rdt, "residual")
    per_channel = isinstance(scale, torch.Tensor)
    f32 = torch.float32
    _dense(post_weight, (D,), f32, "post_weight")
    _dense(weight, (D,), f32, "weight")
    if per_channel:
        _dense(scale, (D,), f32, "scale")
    dev = _device(x, gate, residual, residual_out, y, post_weight, weight,
                  scale if per_channel else None)
    if residual_out is not None:
        ros = _rows(residual_out, shape, rdt, "residual_out")
    elif residual is not None or weight is None:
        residual_out = _new(x, shape, rdt)
        ros = D
    if y is not None:
        ys = _rows(y, shape, dt, "y")
    elif weight is not None:
        y = _new(x, shape, dt)
        ys = D
    # (in one go: a field set by name costs more than the checks)
    io = NormIo(x.data_ptr(), _p(gate), _p(residual), _p(residual_out), _p(y), xs, gs, rs, ros, ys,
                _p(post_weight), _p(weight), scale.data_ptr() if per_channel else None,
                float(post_eps), float(eps), 0.0 if per_channel else float(scale), rcode)
    _call("kda_block_norm", dev, _count(rows, "the number of rows"), _count(D, "the row length"),
          code, ctypes.byref(io))
    return residual_out, y


def beam_select(logits, scores, beams=None, finished=None, eos: int = -1, order: str = "score",
                workspace=None):
    """The best continuations over beams and vocabulary
    (``kda_beam_select``).

    logits ``[B, W, V]`` (rows of unit-stride elements, evenly spaced), scores
    fp32 ``[B, W]``: the beams' log-probabilities; finished bool ``[B, W]`` or
    None; ``eos`` the token that finishes a beam, -1 for none.  Returns
    ``(scores fp32, parents int32, tokens int32, finished bool)``, each ``[B,
    beams]`` (beams None: W), best first with ``order="score"``; with
    ``"rows"`` the best continuation of beam w is in row w (where there is
    one) and the others fill the rows left, so that ``state_reorder`` moves
    as few states as possible.  Values are compared in 64 bits, in which the
    logarithm of a beam's sum is good to some 2^-23, and equal ones taken by
    the lower ``w * V + v``.
    """
    if logits.dim() != 3:
        raise ValueError("logits must be [batch, beams, vocabulary] (got %s)"
                         % (tuple(logits.shape),))
    B, W, V = logits.shape
    code = _dtype(logits, "logits")
    if order not in _ORDERS:
        raise ValueError("order must be one of %s, got %r" % (sorted(_ORDERS), order))
    K = W if beams is None else _count(int(beams), "beams")
    stride = V
    if not logits.is_contiguous() and logits.numel() > 0:
        sb, sw, sv = logits.stride()
        stride = sw if W > 1 else sb if B > 1 else V
        if (V > 1 and sv != 1) or (B > 1 and W > 1 and sb != W * sw) or stride < V:
            raise ValueError("logits must have evenly spaced dense rows (strides %s)"
                             % (logits.stride(),))
    _dense(scores, (B, W), torch.float32, "scores")
    _dense(finished, (B, W), torch.bool, "finished")
    dev = _device(logits, scores, finished, workspace)
    args = (_count(B, "the batch"), W, _count(V, "the vocabulary"), K, code)
    ws = _workspace(workspace, load().kda_beam_select_workspace_size(*args), dev)
    shape = (B, K)
    out = _new(scores, shape, torch.float32)
    parents = _new(scores, shape, torch.int32)
    tokens = _new(scores, shape, torch.int32)
    done = _new(scores, shape, torch.bool)
    _call("kda_beam_select", dev, *args, _p(logits), stride, _p(scores), _p(finished),
          _count(int(eos), "eos"), _ORDERS[order], _p(out), _p(parents), _p(tokens), _p(done),
          _p(ws), 0 if ws is None else ws.numel())
    return out, parents, tokens, done


def state_reorder(states, parents, slots=None):
    """Reorder states in place after a beam selection
    (``kda_state_reorder``): row r of group b becomes what row ``parents[b,
    r]`` of the group was.

    states: a tensor, or a list of up to 32, each ``[slices, ...]``
    contiguous, of any dtype; parents int32 ``[groups, K]``; slots int32
    ``[groups, K]``, the slice of each row (None: ``b * K + r``).  Rows whose
    slice, or whose parent's, is out of range stay as they are.  Returns
    states."""
    many = [states] if isinstance(states, torch.Tensor) else list(states)
    if len(many) > _MAX_STATES:
        raise ValueError("at most %d states in one call (got %d)" % (_MAX_STATES, len(many)))
    if parents.dim() != 2 or parents.dtype != torch.int32 or not parents.is_contiguous():
        raise ValueError("parents must be contiguous int32 [groups, K]")
    _dense(slots, parents.shape, torch.int32, "slots")
    groups, K = parents.shape
    n = len(many)
    at, size, held = (ctypes.c_void_p * n)(), (ctypes.c_int64 * n)(), (ctypes.c_int32 * n)()
    for i, s in enumerate(many):
        if s.dim() < 1 or not s.is_contiguous():
            raise ValueError("states must be contiguous [slices, ...]")
        held[i] = _count(s.shape[0], "the number of state slices")
        if slots is None and held[i] < groups * K:
            raise ValueError("a state holds %d slices for %d rows" % (held[i], groups * K))
        at[i] = s.data_ptr()
        size[i] = s.numel() // max(1, s.shape[0]) * s.element_size()
    dev = _device(parents, slots, *many)
    _call("kda_state_reorder", dev, _count(groups, "the number of groups"), K, _p(parents),
          _p(slots), n, at, size, held)
    return states
