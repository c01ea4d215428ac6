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


WAYS = [(dk, split, dtype) for dtype in (F32, BF16) for dk in (100, 104, 128, 200) for split in (1, 3)]


@pytest.mark.parametrize("dk,split,dtype", WAYS)
def test_an_infinite_state_outlasts_decays(dk, split, dtype):
    """Decays that underflow over a chunk and over a segment leave an infinite
    state infinite; one of 0 makes it NaN, as the product does."""
    print("decay infinite state", dk, split, dtype, flush=True)
    q, k, v, g = inputs(260, 3, dk, 40, dtype, dk + 1)
    g[:] = -2.0
    g[150, 2] = -INF
    init = torch.randn(1, 3, dk, 40, generator=torch.Generator().manual_seed(1))
    init[0, 0, 3, 7] = INF
    init[0, 1, dk - 1, 39] = -INF
    init[0, 2, 0, 0] = INF
    o, fin = compare(q, k, v, g, init=init, split=split)
    assert (o[:, 0, 7] == INF).all() and (o[:, 1, 39] == -INF).all()
    assert (o[:150, 2, 0] == INF).all() and o[150:, 2, 0].isnan().all() and torch.isfinite(o[:, 2, 1:]).all()


@pytest.mark.parametrize("dk,split,dtype", WAYS)
def test_growth_within_the_range_of_fp32(dk, split, dtype):
    """Decays above 1 whose product over a chunk passes fp32, on a state that
    begins at 0 and stays within it."""
    print("decay growth", dk, split, dtype, flush=True)
    q, k, v, g = inputs(260, 2, dk, 40, dtype, dk + 2)
    v *= 2.0 ** -26
    g[70:138, 0] = 1.5
    k[70:100, 0] = 0.0
    g[190:200, 1] = 4.0
    o, fin = compare(q, k, v, g, split=split)
    assert torch.isfinite(o).all() and torch.isfinite(fin).all() and fin[0, 0].abs().max() > 1e25
    # ... and one that stays 0
    k.zero_()
    g[64:192] = 1.5
    o, fin = compare(q, k, v, g, split=split)
    assert (o == 0).all() and (fin == 0).all()


@pytest.mark.parametrize("dk,split,dtype", WAYS)
def test_an_infinite_query_takes_the_signs_of_the_state(dk, split, dtype):
    print("decay infinite query", dk, split, dtype, flush=True)
    q, k, v, g = inputs(260, 2, dk, 40, dtype, dk + 3)
    q[0, 0, 1] = INF
    q[77, 0, 3] = INF
    q[255, 1, dk - 1] = -INF
    q[130, 1, 0] = float("nan")
    o, fin = compare(q, k, v, g, split=split)
    assert (o[77, 0].abs() == INF).all() and (o[255, 1].abs() == INF).all() and o[130, 1].isnan().all()
    assert torch.isfinite(fin).all() and torch.isfinite(o[131:255]).all()


@pytest.mark.parametrize("dk,split,dtype", WAYS)
def test_infinities_and_nan_in_every_input(dk, split, dtype):
    print("decay infinities", dk, split, dtype, flush=True)
    q, k, v, g = inputs(260, 4, dk, 40, dtype, dk + 4)
    k[100, 0, 5] = INF
    k[101, 0, 6] = float("nan")
    v[20, 1, 3] = -INF
    v[21, 1, 3] = INF
    v[64, 1, 8] = float("nan")
    g[200, 2] = float("nan")
    v[259, 3, 1] = INF
    cu = [0, 0, 130, 260]
    compare(q, k, v, g, cu=cu, split=split)
    # an infinite decay above 1 (a cut could not tell whose sign it takes)
    if split == 1:
        g[90, 3] = INF
        compare(q, k, v, g, cu=cu)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_products_beyond_fp32_that_meet_small_values(dtype):
    """Scores q . k that overflow, where k v and S q do not."""
    print("decay large scores", dtype, flush=True)
    q, k, v, g = inputs(100, 1, 64, 32, dtype, 5)
    q *= 2.0 ** 70
    k *= 2.0 ** 64
    v *= 2.0 ** -80
    compare(q, k, v, g)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_decay_of_nan_beside_infinities(dtype):
    """An infinity in front of the NaN, in the same chunk, is still held to the
    recurrence."""
    print("decay nan and infinity", dtype, flush=True)
    for split in (1, 3):
        q, k, v, g = inputs(260, 3, 64, 40, dtype, 6)
        g[90, :] = float("nan")
        v[70, 0, 1] = INF
        k[80, 1, 2] = INF
        v[100, 2, 3] = INF
        o, fin = compare(q, k, v, g, split=split)
        assert torch.isfinite(o[:90, 2]).all() and o[90:].isnan().all() and (o[70:90, 0, 1] == INF).all()
