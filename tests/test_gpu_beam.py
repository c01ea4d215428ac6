"""Beam selection and state reordering on the GPU, against the definitions."""
import numpy as np
import pytest
import torch

import block_ref as ref
import gated_delta_rule_19_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
NINF = -float("inf")


def run(logits, scores, K, finished=None, eos=-1, order="score"):
    out = kda.beam_select(logits.to(DEV), scores.to(DEV), beams=K,
                          finished=None if finished is None else finished.to(DEV), eos=eos, order=order)
    torch.cuda.synchronize()
    return [x.cpu() for x in out]


def compare(logits, scores, K, finished=None, eos=-1, order="score"):
    got = run(logits, scores, K, finished, eos, order)
    want = ref.beam_select(logits, scores, K, finished, eos, order)
    assert torch.equal(got[1], want[1]), (got[1], want[1])
    assert torch.equal(got[2], want[2]), (got[2], want[2])
    assert torch.equal(got[3], want[3])
    fine = torch.isfinite(want[0])
    assert torch.equal(got[0][~fine].double(), want[0][~fine])
    # lse is off by some 2^-23 of its sum's terms, the value is rounded once
    tol = 2.0 ** -22 + 2.0 ** -24 * want[0][fine].abs()
    assert ((got[0].double()[fine] - want[0][fine]).abs() <= tol).all()
    return got


def random_case(B, W, V, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, W, V, generator=g) * 2.5).to(dtype), -10 + 2 * torch.randn(B, W, generator=g)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 100, 4095, 4096, 4097, 8191, 8192, 8193, 20011, 50000])
def test_vocabularies(V, dtype):
    print("beam vocabulary", V, dtype, flush=True)
    logits, scores = random_case(3, 4, V, dtype, V)
    compare(logits, scores, min(4, 4 * V))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("W,K", [(1, 1), (1, 4), (2, 3), (4, 8), (8, 8), (5, 16), (16, 32), (33, 33), (64, 64), (1, 64)])
@pytest.mark.parametrize("order", ["score", "rows"])
def test_beams(W, K, order, dtype):
    print("beams", W, K, order, dtype, flush=True)
    logits, scores = random_case(2, W, 9001, dtype, W * 100 + K)
    compare(logits, scores, K, order=order)


def test_fewer_beams_than_before():
    print("fewer beams", flush=True)
    logits, scores = random_case(4, 8, 1000, F32, 3)
    compare(logits, scores, 3)


@pytest.mark.parametrize("order", ["score", "rows"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_finished_beams(order, dtype):
    print("finished beams", order, dtype, flush=True)
    logits, scores = random_case(6, 5, 3000, dtype, 4)
    done = torch.rand(6, 5, generator=torch.Generator().manual_seed(5)) < 0.4
    done[0] = True          # all of a batch
    done[1] = False
    logits[2, :, 7] = 30.0  # a batch whose live beams all finish now
    compare(logits, scores, 5, done, 7, order)
    got = run(logits[:1], scores[:1], 5, done[:1], 7)
    assert (got[2] == 7).all() and torch.equal(got[0][0], scores[0].sort(descending=True)[0])


def test_finished_beam_alone():
    """One candidate above -inf, and places left to fill."""
    print("finished beam alone", flush=True)
    logits, scores = random_case(1, 1, 50, F32, 6)
    for eos in (0, 2, 49):
        compare(logits, scores, 4, torch.tensor([[True]]), eos)
        compare(logits, scores, 4, torch.tensor([[True]]), eos, "rows")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_masked_tokens(dtype):
    """Rows with few or no tokens left, more beams than tokens, whole parts
    masked."""
    print("beam masks", dtype, flush=True)
    logits, scores = random_case(5, 4, 30000, dtype, 7)
    keep = logits.clone()
    logits[:] = NINF
    logits[0, 1, 29999] = 1.0                      # one token of one beam
    logits[1, :, [5, 20000]] = keep[1, :, [5, 20000]]
    logits[2, 0] = keep[2, 0]                      # one beam open
    logits[3] = keep[3]
    logits[3, :, :16384] = NINF                    # whole parts
    # batch 4: nothing at all
    for K in (4, 9):
        got = compare(logits, scores, K)
        assert got[2][4].tolist() == list(range(K)) and (got[0][4] == NINF).all()
    compare(logits, scores, 4, order="rows")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_beams_without_value(dtype):
    print("beams without value", dtype, flush=True)
    logits, scores = random_case(4, 3, 9000, dtype, 8)
    scores[0, 1] = NINF                            # as in a first step
    scores[0, 2] = NINF
    scores[1, 0] = float("nan")
    scores[1, 1] = float("inf")
    logits[2, 0, 8999] = float("nan")
    logits[2, 1, 3] = float("inf")
    logits[3, :, 100] = float("nan")               # no beam left
    logits[3, 2] = NINF
    logits[3, 2, 10] = float("nan")
    compare(logits, scores, 3)
    compare(logits, scores, 5, order="rows")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [100, 8192, 20000])
def test_ties(V, dtype):
    """Equal logits and equal beams: the lower beam, then the lower token."""
    print("beam ties", V, dtype, flush=True)
    logits = torch.zeros(3, 4, V, dtype=dtype)
    logits[1] = -0.0
    logits[1, :, ::3] = 0.0
    logits[2, :, V // 2:] = 1.0
    scores = torch.full((3, 4), -1.0)
    compare(logits, scores, 4)
    compare(logits, scores, 64)
    compare(logits, scores, 8, order="rows")


def test_many_equal_values_over_many_beams():
    """More candidates at the threshold than the merge holds at once."""
    print("beam equal values", flush=True)
    logits = torch.zeros(1, 64, 40000, dtype=F32)
    scores = torch.full((1, 64), -2.0)
    got = compare(logits, scores, 64)
    assert (got[1] == 0).all() and got[2][0].tolist() == list(range(64))
    scores[0, :] = -torch.arange(64).flip(0).float()
    compare(logits, scores, 40)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sorted_logits(dtype):
    print("beam sorted logits", dtype, flush=True)
    base = torch.linspace(-20, 20, 30000)
    logits = torch.stack([base, base.flip(0), base.roll(4000)]).to(dtype).view(1, 3, -1)
    compare(logits, torch.tensor([[-1.0, -1.5, -2.0]]), 16)


def test_extreme_logits():
    print("beam extreme logits", flush=True)
    logits, scores = random_case(2, 2, 5000, F32, 9)
    logits[0] *= 1e37
    logits[1] *= 1e-30
    got = run(logits, scores, 2)
    assert got[1][0].tolist() == ref.beam_select(logits[:1], scores[:1], 2)[1][0].tolist()
    # all but equal: within a beam the logits themselves decide
    top = logits[1].max(-1).values.argmax()
    assert got[2][1, 0] == logits[1, got[1][1, 0]].argmax() and top >= 0


def test_strided_rows():
    print("beam strides", flush=True)
    for dtype in (F32, BF16):
        logits, scores = random_case(2, 3, 5001, dtype, 10)
        buf = torch.full((2, 3, 5011), 100.0, dtype=dtype, device=DEV)
        buf[:, :, 3:5004] = logits.to(DEV)
        out = kda.beam_select(buf[:, :, 3:5004], scores.to(DEV))
        torch.cuda.synchronize()
        want = ref.beam_select(logits, scores, 3)
        assert torch.equal(out[1].cpu(), want[1]) and torch.equal(out[2].cpu(), want[2])


def test_rows_keep_their_place():
    print("beam rows", flush=True)
    logits, scores = random_case(40, 6, 500, F32, 11)
    got = run(logits, scores, 6, order="rows")
    for b in range(40):
        for r in range(6):
            p = int(got[1][b, r])
            assert got[1][b, p] == p  # a beam that goes on does so in its row


# ---- reordering -------------------------------------------------------------------

def tables(G, K, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, K, (G, K), generator=g, dtype=torch.int32)


@pytest.mark.parametrize("K", [1, 2, 3, 4, 5, 8, 13, 16, 17, 33, 64])
@pytest.mark.parametrize("shape,dtype", [((3, 1001), BF16), ((2, 64, 32), F32), ((1,), F32), ((7,), torch.int8),
                                         ((5, 3), torch.float8_e4m3fn), ((20000,), F32)])
def test_reorder(K, shape, dtype):
    print("reorder", K, shape, dtype, flush=True)
    G = 3
    state = torch.randint(-100, 100, (G * K,) + shape, dtype=torch.int32,
                          generator=torch.Generator().manual_seed(K))
    state = state.to(torch.int8).view(dtype) if dtype.itemsize == 1 else state.to(dtype)
    parents = tables(G, K, K + 1)
    if K > 1:
        parents[1] = torch.arange(K).roll(1)       # a cycle
        parents[2] = K - 1                         # one parent for all
    d = state.to(DEV)
    assert kda.state_reorder(d, parents.to(DEV)) is d
    torch.cuda.synchronize()
    raw = lambda x: x.view(torch.int8) if dtype.itemsize == 1 else x
    assert torch.equal(raw(d.cpu()), ref.reorder(raw(state), parents))


def test_reorder_slots_and_padding():
    print("reorder slots", flush=True)
    state = torch.randn(9, 50, generator=torch.Generator().manual_seed(1))
    parents = torch.tensor([[1, 0, -1], [2, 2, 0], [0, 7, 1]], dtype=torch.int32)
    slots = torch.tensor([[8, 3, 0], [-1, 5, 1], [2, 4, 9]], dtype=torch.int32)
    d = state.to(DEV)
    kda.state_reorder(d, parents.to(DEV), slots=slots.to(DEV))
    torch.cuda.synchronize()
    assert torch.equal(d.cpu(), ref.reorder(state, parents, slots))


def test_reorder_several_states_of_odd_alignment():
    print("reorder several states", flush=True)
    parents, G, K = tables(4, 5, 2), 4, 5
    slots = torch.randperm(25, generator=torch.Generator().manual_seed(3))[:20].int().view(4, 5)
    made = [torch.randn(25, 2, 64, 64), torch.randn(25, 3, 101).to(BF16), torch.randn(30, 17),
            torch.randint(-9, 9, (25, 33), dtype=torch.int8), torch.randn(25, 0), torch.randn(40, 1)]
    dev = []
    for i, s in enumerate(made):  # at odd element offsets
        buf = torch.zeros(s.numel() + 3, dtype=s.dtype, device=DEV)
        dev.append(buf[i % 3: i % 3 + s.numel()].view(s.shape))
        dev[-1].copy_(s)
    kda.state_reorder(dev, parents.to(DEV), slots=slots.to(DEV))
    torch.cuda.synchronize()
    for d, s in zip(dev, made):
        assert torch.equal(d.cpu(), ref.reorder(s, parents, slots))


def test_reorder_offsets_past_32_bits():
    print("reorder offsets past 32 bits", flush=True)
    state = torch.empty((40, 1 << 27), dtype=torch.int8, device=DEV)  # 5 GiB
    state[38], state[39] = 3, 5
    parents = torch.tensor([[1, 0]], dtype=torch.int32, device=DEV)
    kda.state_reorder(state, parents, slots=torch.tensor([[38, 39]], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert (state[38] == 5).all() and (state[39] == 3).all()


def test_nothing_to_do():
    print("beam nothing", flush=True)
    out = kda.beam_select(torch.empty(0, 2, 10, device=DEV), torch.empty(0, 2, device=DEV))
    assert [tuple(x.shape) for x in out] == [(0, 2)] * 4
    s = torch.randn(3, 4, device=DEV)
    keep = s.clone()
    kda.state_reorder(s, torch.empty((0, 3), dtype=torch.int32, device=DEV))
    kda.state_reorder([], torch.zeros((1, 3), dtype=torch.int32, device=DEV))
    assert torch.equal(s, keep)
