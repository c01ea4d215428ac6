"""Accuracy of the block norm's parts where the general bound of ``block_ref``
is wide: the gate far from 0."""
import pytest
import torch

import block_ref as ref
import gated_delta_rule_19_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24
INF = float("inf")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gates_far_from_zero(dtype):
    """u sigmoid(gate) in fp32 to 8 U wherever the gate is: exponential and
    reciprocal 2 U each, one each for its argument's remainder, the sum with 1,
    the product with u and the scale.  Below 2^-126 fp32's numbers are 2^-149
    apart, whatever their size: half of that more."""
    print("norm gate", dtype, flush=True)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(40, 1002, generator=g).to(dtype)
    gate = ((torch.rand(40, 1002, generator=g) - 0.5) * 170).to(dtype)
    out = torch.empty(40, 1002, device=DEV)
    r, y = kda.block_norm(x.to(DEV), gate=gate.to(DEV), residual_out=out)
    torch.cuda.synchronize()
    want = ref.f64(x) * torch.sigmoid(ref.f64(gate))
    assert y is None and r is out
    ref.check("r", r, want, 8 * U * want.abs() + 2.0 ** -150)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gates_at_the_ends(dtype):
    print("norm gate ends", dtype, flush=True)
    gate = torch.tensor([[-INF, -1e30, -200.0, 200.0, 1e30, INF, float("nan"), 0.0]], dtype=dtype)
    r, _ = kda.block_norm(torch.full((1, 8), 3.0, dtype=dtype, device=DEV), gate=gate.to(DEV))
    torch.cuda.synchronize()
    r = r[0].tolist()
    assert r[:6] == [0, 0, 0, 3, 3, 3] and r[6] != r[6] and r[7] == 1.5


def test_small_sums_beside_a_large_one():
    """A square of 2^24 and fifteen of 1 far from each other: added to the large
    one by one, each would be lost in its rounding.  Joined first, at most one
    is: 2^-24 of the mean; and root, division and two products half a step each."""
    print("norm sums", flush=True)
    D = 65536
    x = torch.zeros(2, D)
    x[:, 0] = 4096.0
    x[1, [256 * i for i in range(1, 16)]] = 1.0
    r, y = kda.block_norm(x.to(DEV), torch.ones(D, device=DEV), eps=0.0)
    torch.cuda.synchronize()
    want = ref.f64(x) / ref.f64(x).square().mean(-1, keepdim=True).sqrt()
    ref.check("y", y, want, 5 * U * want.abs())
    assert y[1, 0] < y[0, 0]
