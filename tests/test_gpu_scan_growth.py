"""Selective scan whose states grow (A > 0, or negative steps): a segment's
growth may pass the largest fp32 number where no state does.  Cut and uncut
calls against the 64-bit recurrence."""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_19_amd as kda
from gated_delta_rule_19_amd import _native as nat
import recurrent_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
U = ref.U


def pairs_of(cu, D, N, G, split):
    """Segment pairs of a call, from its workspace: each holds the end states
    of blocks of 64 channels (16 a channel and lane group, or N) and a sum of
    steps."""
    a = np.ascontiguousarray(cu, dtype=np.int64)
    size = nat.load().kda_selective_scan_workspace_size(len(cu) - 1, a.ctypes.data, D, N, G, split)
    blocks = G * ((D // G + 63) // 64)
    rows = 16 * (1 if N <= 16 else 2 if N <= 32 else 4 if N <= 64 else 8)
    for kind, held in (("row", rows), ("lane", N)):
        if size % (256 * blocks * (held + 1)) == 0:
            return kind, size // (256 * blocks * (held + 1))
    raise AssertionError("a workspace of %d bytes" % size)


def scan64(x, delta, A, B, C, init, segment, dtype):
    """The recurrence of one sequence (G = 1, steps as given) and its bound.

    As in recurrent_ref.scan a step's decay is off by |delta A| (U + 3 U) and
    2 U, its input by 3 U, a sum by U.  A segment's decay is the exponential of
    a sum of its steps: the sum, of steps of one sign, is off by a rounding of
    at most itself for each of its tokens and for each of the at most 64
    segments of a run, which the exponential turns into as many U of |A sum|.
    That is what as many U of every step's own |delta A| come to.  (With
    growth |A sum| exp(A sum) is no longer below 1, so the bound of a decaying
    scan does not hold.)  2 E: the entry state is a product of its own."""
    T, D = x.shape
    N = A.shape[1]
    h = np.zeros((D, N)) if init is None else init.copy()
    E = np.zeros((D, N))
    y, ytol = np.zeros((T, D)), np.zeros((T, D))
    for t in range(T):
        arg = delta[t][:, None] * A
        a = np.exp(arg)
        inp = (delta[t] * x[t])[:, None] * B[t]
        hold = a * h
        E = a * E + np.abs(hold) * (np.abs(arg) * (4 + segment + 64) * U + 3 * U) + np.abs(inp) * 3 * U
        h = hold + inp
        E = E + U * np.abs(h)
        term = C[t] * h
        y[t] = term.sum(1)
        ytol[t] = (np.abs(C[t]) * 2 * E).sum(1) + (N + 3) * U * np.abs(term).sum(1)
    return y, ytol + ref.HALF[dtype] * np.abs(y) + 1e-37, h, 2 * E + 1e-37


def run(x, delta, A, B, C, init, split, dtype, name):
    on = lambda t: None if t is None else t.to(DEV)
    T, D = x.shape
    N = A.shape[1]
    kind, pairs = pairs_of([0, T], D, N, 1, split)
    segment = T if pairs == 0 else T // pairs
    y, fin = kda.selective_scan(on(x), on(delta), on(A), on(B.unsqueeze(1)), on(C.unsqueeze(1)),
                                delta_softplus=False,
                                initial_state=None if init is None else on(init.unsqueeze(0)),
                                split_hint=split)
    torch.cuda.synchronize()
    ry, yt, rf, ft = scan64(*(ref.f64(t) for t in (x, delta, A, B, C, init)), segment, dtype)
    assert np.isfinite(ry).all() and np.isfinite(rf).all()
    print("  segments of", segment, kind, flush=True)
    ref.check("%s y" % name, y, ry, yt)
    ref.check("%s final state" % name, fin[0], rf, ft)
    return pairs


def inputs(T, D, N, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    f = lambda *s: torch.randn(s, generator=g)
    x, B, C = f(T, D).to(dtype), f(T, N).to(dtype), f(T, N).to(dtype)
    delta = (0.1 * torch.exp(0.2 * f(T, D))).to(dtype)
    return x, delta, B, C


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N", [3, 13, 16, 20, 65])
def test_nothing_grows_to_nothing(N, dtype, sign):
    """Zeros until 60 tokens before the end: the state of every segment before
    is 0 however much it would have grown.  Rates whose growth passes an fp32
    over a segment, over a run of segments only, and not at all."""
    print("scan growth from zero", N, dtype, sign, flush=True)
    T, D = 3000, 66
    x, delta, B, C = inputs(T, D, N, dtype, 400 + N)
    x[:-60] = 0
    A = torch.tensor([6.0, 3.0, 0.5, 0.0, -2.0, 1e-3, 8.0]).repeat(N)[:N].repeat(D, 1).contiguous()
    A = A * (1 + 0.01 * torch.arange(D)[:, None] / D)
    cuts = [run(x, sign * delta, sign * A, B, C, None, split, dtype, "growth")
            for split in (0, 1, 4, 30)]
    assert cuts[0] > 8 and cuts[1] == 0 and cuts[2] == 3 and cuts[3] > 20


@pytest.mark.parametrize("N", [5, 16, 20])
def test_a_small_state_grows_by_more_than_the_largest_number(N):
    """An initial state of some 1e-30 that grows by e^100 within one middle
    segment, or over all of them: what comes out is some 1e13."""
    print("scan growth of a small state", N, flush=True)
    T, D = 700, 66
    x, delta, B, C = inputs(T, D, N, F32, 420 + N)
    g = torch.Generator().manual_seed(430)
    init = 1e-30 * (1 + torch.rand((D, N), generator=g))
    x[:] = 0
    A = torch.ones(D, N)
    for name, lo, hi in (("in one segment", 250, 330), ("over all", 0, T)):
        d = torch.full_like(delta, 1e-4)
        d[lo:hi] = 100.0 / (hi - lo)
        for split in (1, 4, 20):
            run(x, d, A, B, C, init, split, F32, name)


def test_growth_past_every_number_is_infinite():
    """A state that does pass the largest number, cut or not."""
    print("scan growth to infinity", flush=True)
    T, D, N = 700, 64, 16
    x, delta, B, C = inputs(T, D, N, F32, 440)
    x = x.abs() + 0.1
    B = B.abs() + 0.1
    C = C.abs() + 0.1
    A = torch.full((D, N), 8.0)
    for split in (1, 4, 20):
        y, fin = kda.selective_scan(*(t.to(DEV) for t in (x, delta, A, B.unsqueeze(1), C.unsqueeze(1))),
                                    delta_softplus=False, split_hint=split)
        torch.cuda.synchronize()
        assert torch.isposinf(fin).all() and torch.isposinf(y[-1]).all()
