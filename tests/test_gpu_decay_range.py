"""Decayed attention on the GPU where infinities, NaN and the ends of fp32's
range meet the chunks: prompts are held to the recurrence, infinities by sign,
NaN as NaN, everything else by the bounds of ``block_ref``."""
import numpy as np
import pytest
import torch

import block_ref as ref
import gated_delta_rule_19_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")


def inputs(T, H, dk, dv, dtype, seed):
    """Positive q and k, so that an infinity keeps its sign in every sum."""
    g = torch.Generator().manual_seed(seed)
    q = (torch.rand(T, H, dk, generator=g) * dk ** -0.5 + 0.01).to(dtype)
    k = (torch.rand(T, H, dk, generator=g) * dk ** -0.5 + 0.01).to(dtype)
    v = torch.randn(T, H, dv, generator=g).to(dtype)
    return q, k, v, -0.1 * torch.rand(T, H, generator=g)


def held(name, got, want, tol):
    got, fine = ref.f64(got), torch.isfinite(want)
    bad = torch.where(fine, ~((got - want).abs() <= tol), (got != want) & ~(got.isnan() & want.isnan()))
    if bad.any():
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError("%s: %d of %d off; first at %s: %r, expected %r +- %.3g" % (
            name, int(bad.sum()), bad.numel(), at, float(got[at]), float(want[at]), float(tol[at])))


def compare(q, k, v, g, cu=None, init=None, split=0):
    """Prompt and single tokens against the recurrence."""
    cu = [0, q.shape[0]] if cu is None else cu
    ro, otol, rf, ftol = ref.decay_attention(ref.f64(q), ref.f64(k), ref.f64(v), ref.f64(g), 1.0, cu, ref.f64(init),
                                             q.dtype)
    dev = [x.to(DEV) for x in (q, k, v, g)]
    o, fin = kda.decay_attention(*dev, cu_seqlens=cu, initial_state=None if init is None else init.to(DEV),
                                 split_hint=split)
    torch.cuda.synchronize()
    held("o", o, ro, otol)
    held("final state", fin, rf, ftol)
    S = torch.zeros_like(fin) if init is None else init.to(DEV)
    for i in range(len(cu) - 1):
        for t in range(cu[i], cu[i + 1]):
            kda.decay_attention_step(S[i:i + 1], *(x[t:t + 1] for x in dev))
    torch.cuda.synchronize()
    held("state of the steps", S, rf, ftol)
    return o, fin


# (streams take bf16 heads of multiples of 8; others, fp32 and cuts the chunk kernel)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk", [1, 8, 37, 100, 104, 130])
@pytest.mark.parametrize("split", [1, 3])
def test_an_infinite_value_keeps_its_sign(dk, split, dtype):
    """Rows of the state that pad dk to whole tiles do not turn an infinity
    into a NaN for the tokens behind it."""
    print("decay infinite value", dk, split, dtype, flush=True)
    q, k, v, g = inputs(260, 2, dk, 24, dtype, dk)
    v[30, 0, 5] = INF
    v[200, 1, 23] = -INF
    o, fin = compare(q, k, v, g, split=split)
    assert (o[30:, 0, 5] == INF).all() and (o[200:, 1, 23] == -INF).all()
    assert (fin[0, 0, :, 5] == INF).all() and (fin[0, 1, :, 23] == -INF).all()
