"""Beam selection over many beams and large vocabularies: the chosen, and that
candidates with different values are ranked at once, not one after the other."""
import pytest
import torch

import block_ref as ref
import gated_delta_rule_19_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def case(B, W, V, dtype, spread, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, W, V, generator=g) * 2.5).to(dtype), -10 + spread * torch.randn(B, W, generator=g)


@pytest.mark.parametrize("W,K,V,dtype", [(16, 32, 200000, F32), (16, 16, 60000, F32), (64, 64, 20000, BF16),
                                         (5, 64, 50000, F32), (1, 64, 200000, F32), (64, 33, 8193, F32)])
def test_chosen(W, K, V, dtype):
    print("wide beams", W, K, V, dtype, flush=True)
    for spread in (0.3, 2.0, 30.0):
        logits, scores = case(1, W, V, dtype, spread, W + K)
        if spread == 30.0:
            scores[0, 1:] = -float("inf")  # as in a first step
        got = kda.beam_select(logits.to(DEV), scores.to(DEV), beams=K)
        torch.cuda.synchronize()
        want = ref.beam_select(logits, scores, K)
        assert torch.equal(got[1].cpu(), want[1]) and torch.equal(got[2].cpu(), want[2])


def took(logits, scores, K):
    """The fastest of some runs, in ms on the GPU."""
    logits, scores, best = logits.to(DEV), scores.to(DEV), float("inf")
    for _ in range(6):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(5):
            kda.beam_select(logits, scores, beams=K)
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) / 5)
    return best


@pytest.mark.parametrize("W,K,odd_W,odd_K,V,dtype", [(16, 32, 16, 20, 200000, F32), (64, 64, 50, 50, 128001, BF16)])
def test_a_power_of_two_costs_what_its_neighbours_do(W, K, odd_W, odd_K, V, dtype):
    print("wide beams, time", W, K, V, dtype, flush=True)
    ms = took(*case(1, W, V, dtype, 0.3, 1), K)
    near = took(*case(1, odd_W, V, dtype, 0.3, 2), odd_K)
    # (candidates and logits are up to 1.7 times as many)
    assert ms < 4 * near, (ms, near)
