"""8-bit state cache on the GPU: codes and scales equal the definition's bit
for bit, and so does what is read back."""
import numpy as np
import pytest
import torch

import gated_delta_rule_19_amd as kda
import recurrent_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
KINDS = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def rows(shape, seed):
    g = torch.Generator().manual_seed(seed)
    size = torch.exp(4 * torch.randn(shape[:-1] + (1,), generator=g))
    return torch.randn(shape, generator=g) * size


def bits(t):
    return t.cpu().view(torch.int8) if t.dtype != torch.int8 else t.cpu()


def pool(slots, shape, kind):
    codes = torch.full((slots,) + shape, 77, dtype=torch.int8, device=DEV).view(kind)
    scales = torch.full((slots,) + shape[:-1], -3.0, device=DEV)
    return codes, scales


def same(a, b):
    """Equal, with NaN equal to NaN."""
    return torch.equal(torch.nan_to_num(a, nan=1e30), torch.nan_to_num(b, nan=1e30)) and \
        torch.equal(torch.isnan(a), torch.isnan(b))


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("L", [1, 2, 3, 4, 13, 16, 31, 64, 65, 96, 100, 128, 129, 200, 250, 255, 256])
def test_row_lengths(L, kind):
    print("cache row length", L, kind, flush=True)
    dt = KINDS[kind]
    x = rows((3, 37, L), 10 + L)
    codes, scales = pool(5, (37, L), dt)
    dst = torch.tensor([4, 0, 2], dtype=torch.int32, device=DEV)
    kda.state_store(x.to(DEV), codes, scales, dst=dst)
    rc, rs = ref.quantise(x, dt)
    torch.cuda.synchronize()
    at = [4, 0, 2]
    assert torch.equal(bits(codes)[at], bits(rc)) and torch.equal(scales.cpu()[at], rs)
    assert (bits(codes)[[1, 3]] == 77).all() and (scales[[1, 3]] == -3).all()
    back = torch.full((4, 37, L), 9.0, device=DEV)
    src = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    out = kda.state_load(codes, scales, back, src=src,
                         dst=torch.tensor([3, 1, 0], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    want = rc.float() * rs[..., None]
    assert out is back
    assert torch.equal(back.cpu()[[3, 1, 0]], want[[1, 2, 0]]) and (back[2] == 9).all()


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("R", [1, 2, 15, 16, 17, 500])
def test_row_counts_and_kda_states(R, kind):
    print("cache rows", R, kind, flush=True)
    dt = KINDS[kind]
    x = rows((2, R, 128), 30 + R)
    codes, scales = pool(2, (R, 128), dt)
    kda.state_store(x.to(DEV), codes, scales)
    back = kda.state_load(codes, scales, torch.empty_like(x, device=DEV))
    rc, rs = ref.quantise(x, dt)
    torch.cuda.synchronize()
    assert torch.equal(bits(codes), bits(rc)) and torch.equal(scales.cpu(), rs)
    assert torch.equal(back.cpu(), rc.float() * rs[..., None])


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("L", [13, 128])
def test_special_rows(L, kind):
    """Zero rows, subnormal rows, the largest values, infinities and NaN."""
    print("cache special rows", L, kind, flush=True)
    dt = KINDS[kind]
    x = rows((1, 12, L), 50)
    x[0, 0] = 0.0
    x[0, 1] = 0.0
    x[0, 1, 3] = -1e-44          # a subnormal
    x[0, 2] = 1.1754944e-38      # the smallest normal
    x[0, 3] *= 3e38 / x[0, 3].abs().max()
    x[0, 4, 5] = float("inf")
    x[0, 5, 2] = float("nan")
    x[0, 6, L - 1] = -float("inf")
    x[0, 7] = -0.0
    x[0, 8] = torch.finfo(torch.float32).max
    codes, scales = pool(1, (12, L), dt)
    kda.state_store(x.to(DEV), codes, scales)
    back = kda.state_load(codes, scales, torch.empty_like(x, device=DEV))
    rc, rs = ref.quantise(x, dt)
    torch.cuda.synchronize()
    assert same(scales.cpu(), rs)
    assert torch.equal(codes.cpu().float(), rc.float())
    assert torch.isnan(back[0, [4, 5, 6]]).all()
    assert (back[0, [0, 7]] == 0).all()
    assert torch.isfinite(back[0, [0, 1, 2, 3, 7, 8, 9, 10, 11]]).all()


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_every_code_reads_back(kind):
    print("cache codes", kind, flush=True)
    dt = KINDS[kind]
    codes = torch.arange(-128, 128, dtype=torch.int32).to(torch.int8).view(dt).reshape(1, 2, 128)
    scales = torch.tensor([[0.37, 2.0 ** -126]])
    for L in (128, 64):
        c = codes.view(torch.int8).reshape(1, -1, L).view(dt)
        s = scales.repeat_interleave(128 // L, dim=1).contiguous()
        back = kda.state_load(c.to(DEV), s.to(DEV), torch.empty(c.shape, device=DEV))
        torch.cuda.synchronize()
        assert same(back.cpu(), c.float() * s[..., None])


def test_ties_round_to_even():
    print("cache ties", flush=True)
    x = torch.arange(-127, 128).float().repeat(1, 1, 1)
    x = torch.cat([x, torch.arange(-126.5, 127.0, 1.0).view(1, 1, -1), torch.full((1, 1, 1), 127.0)], -1)
    for at in range(0, 510, 255):  # rows whose amax is 127: the scale is 1
        row = torch.cat([x[..., at:at + 255], torch.full((1, 1, 1), 127.0)], -1)
        codes, scales = pool(1, (1, 256), torch.int8)
        kda.state_store(row.to(DEV), codes, scales)
        torch.cuda.synchronize()
        assert scales.item() == 1.0
        assert torch.equal(codes.cpu(), torch.round(row).to(torch.int8))


def test_unaligned_buffers():
    """State and codes at odd element offsets run the narrow loads."""
    print("cache unaligned", flush=True)
    x = rows((2, 9, 128), 60)
    for kind in KINDS.values():
        buf = torch.zeros(x.numel() + 3, device=DEV)
        st = buf[3:].view(2, 9, 128)
        st.copy_(x)
        raw = torch.zeros(x.numel() + 1, dtype=torch.int8, device=DEV)
        codes = raw[1:].view(2, 9, 128).view(kind)
        scales = torch.zeros((2, 9), device=DEV)
        kda.state_store(st, codes, scales)
        out = torch.zeros(x.numel() + 1, device=DEV)[1:].view(2, 9, 128)
        kda.state_load(codes, scales, out)
        rc, rs = ref.quantise(x, kind)
        torch.cuda.synchronize()
        assert torch.equal(bits(codes), bits(rc)) and torch.equal(scales.cpu(), rs)
        assert torch.equal(out.cpu(), rc.float() * rs[..., None])
        assert raw[0] == 0 and (buf[:3] == 0).all()


def test_padding_entries_are_skipped():
    print("cache padding", flush=True)
    x = rows((4, 5, 16), 70)
    codes, scales = pool(3, (5, 16), torch.int8)
    src = torch.tensor([3, -1, 0, 4, 1], dtype=torch.int32, device=DEV)
    dst = torch.tensor([1, 2, 3, 0, -7], dtype=torch.int32, device=DEV)
    kda.state_store(x.to(DEV), codes, scales, src=src, dst=dst)
    torch.cuda.synchronize()
    rc, rs = ref.quantise(x[3:], torch.int8)
    assert torch.equal(codes.cpu()[1:2], rc) and torch.equal(scales.cpu()[1:2], rs)
    assert (codes[[0, 2]] == 77).all() and (scales[[0, 2]] == -3).all()
    back = torch.full((2, 5, 16), 9.0, device=DEV)
    kda.state_load(codes, scales, back, src=torch.tensor([1, 3, 0], dtype=torch.int32, device=DEV),
                   dst=torch.tensor([1, 0, 2], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert torch.equal(back.cpu()[1:], rc.float() * rs[..., None]) and (back[0] == 9).all()


def test_offsets_past_32_bits():
    """The last slot of a pool of more than 2^31 codes, from and to the last
    item of more than 2^31 fp32 values."""
    print("cache offsets past 32 bits", flush=True)
    R, L, slots = 12288, 128, 1400
    codes = torch.empty((slots, R, L), dtype=torch.int8, device=DEV)
    scales = torch.empty((slots, R), device=DEV)
    x = rows((1, R, L), 80)
    many = torch.empty((slots, R, L), device=DEV)
    many[-1:] = x
    last = torch.tensor([slots - 1], dtype=torch.int32, device=DEV)
    kda.state_store(many, codes, scales, src=last, dst=last)
    rc, rs = ref.quantise(x, torch.int8)
    torch.cuda.synchronize()
    assert torch.equal(codes[-1:].cpu(), rc) and torch.equal(scales[-1:].cpu(), rs)
    many[-1:] = 0
    kda.state_load(codes, scales, many, src=last, dst=last)
    torch.cuda.synchronize()
    assert torch.equal(many[-1:].cpu(), rc.float() * rs[..., None])
