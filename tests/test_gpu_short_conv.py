"""Short convolution on the GPU against the 64-bit form, elementwise within
the bound of its roundings; states (copied, never rounded) bit for bit."""
import numpy as np
import pytest
import torch

import gated_delta_rule_19_amd as kda
import recurrent_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def case(lengths, D, W, dtype, seed, bias=True, state=True, act="silu"):
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)
    c = dict(x=rand((int(cu[-1]), D), dtype, seed), w=rand((D, W), dtype, seed + 1, 0.5),
             b=rand((D,), dtype, seed + 2) if bias else None, cu=cu, act=act,
             s=rand((len(lengths), W - 1, D), dtype, seed + 3) if state else None)
    return c


def on(t):
    return None if t is None else t.to(DEV)


def reference(c):
    return ref.conv(ref.f64(c["x"]), ref.f64(c["w"]), ref.f64(c["b"]), c["cu"], ref.f64(c["s"]),
                    c["act"] is not None, c["x"].dtype)


def compare(c, y, fin):
    ry, tol, rf = reference(c)
    ref.check("y", y, ry, tol)
    assert np.array_equal(ref.f64(fin), rf)


LENGTHS = {
    "one": [1], "short": [2], "tile": [64], "odd": [131],
    "mixed": [0, 1, 2, 3, 0, 64, 65, 7, 200, 0],
    "many": [(i * 7) % 13 for i in range(120)],       # past the inline table
    "table_edge": [3] * 64, "table_edge1": [3] * 65, "parts": [2] * 321,
    "none": [0, 0],
}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lens", sorted(LENGTHS))
def test_lengths(lens, dtype):
    print("conv lengths", lens, dtype, flush=True)
    c = case(LENGTHS[lens], 48, 4, dtype, 10)
    y, fin = kda.short_conv(on(c["x"]), on(c["w"]), on(c["b"]), cu_seqlens=c["cu"],
                            initial_state=on(c["s"]))
    torch.cuda.synchronize()
    compare(c, y, fin)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("W", [2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("D", [1, 7, 64, 520])
def test_widths_and_channels(D, W, dtype):
    print("conv width", W, "channels", D, dtype, flush=True)
    c = case([5, 1, 90], D, W, dtype, 20 + W, bias=D != 64, state=W % 2 == 0,
             act="silu" if D != 7 else None)
    y, fin = kda.short_conv(on(c["x"]), on(c["w"]), on(c["b"]), cu_seqlens=c["cu"],
                            initial_state=on(c["s"]), activation=c["act"])
    torch.cuda.synchronize()
    compare(c, y, fin)


@pytest.mark.parametrize("off", [0, 1, 8])
def test_column_ranges_and_alignment(off):
    """x and y as column ranges of one wide buffer; nothing else is touched."""
    print("conv columns", off, flush=True)
    c = case([40, 3], 64, 4, BF16, 30)
    wide = torch.full((43, 200), 7.0, dtype=BF16, device=DEV)
    x, y = wide[:, off:off + 64], wide[:, 100 + off:164 + off]
    x.copy_(c["x"])
    out, fin = kda.short_conv(x, on(c["w"]), on(c["b"]), cu_seqlens=c["cu"],
                              initial_state=on(c["s"]), y=y)
    torch.cuda.synchronize()
    assert out is y
    compare(c, y, fin)
    assert torch.equal(x.cpu(), c["x"])
    keep = torch.ones(200, dtype=torch.bool)
    keep[off:off + 64] = keep[100 + off:164 + off] = False
    assert (wide[:, keep.to(DEV)] == 7).all()


def test_in_place_state_and_resume():
    """A prompt in two calls with the state updated in place equals one call."""
    print("conv resume", flush=True)
    c = case([100, 2, 31], 72, 4, BF16, 40)
    x, w, b, s = (on(c[k]) for k in ("x", "w", "b", "s"))
    cut = [0, 50, 51, 70]  # tokens of the first call
    first = torch.cat([x[0:50], x[100:101], x[102:121]])
    rest = torch.cat([x[50:100], x[101:102], x[121:133]])
    y1, f1 = kda.short_conv(first, w, b, cu_seqlens=cut, initial_state=s, final_state=s)
    assert f1 is s
    y2, _ = kda.short_conv(rest, w, b, cu_seqlens=[0, 50, 51, 63], initial_state=s, final_state=s)
    torch.cuda.synchronize()
    y = torch.empty_like(x)
    y[0:50], y[100:101], y[102:121] = y1[0:50], y1[50:51], y1[51:70]
    y[50:100], y[101:102], y[121:133] = y2[0:50], y2[50:51], y2[51:63]
    compare(c, y, s)


def test_slots_pick_slices_and_padding_keeps_out():
    print("conv slots", flush=True)
    c = case([5, 9, 3, 0], 40, 4, F32, 50)
    pool = rand((7, 3, 40), F32, 55).to(DEV)
    before = pool.clone()
    slots = torch.tensor([6, -1, 2, 99], dtype=torch.int32, device=DEV)
    y, fin = kda.short_conv(on(c["x"]), on(c["w"]), on(c["b"]), cu_seqlens=c["cu"],
                            initial_state=pool, final_state=pool, slots=slots)
    torch.cuda.synchronize()
    assert fin is pool
    c["s"] = torch.stack([before[6], torch.zeros_like(before[0]), before[2],
                          torch.zeros_like(before[0])]).cpu()
    ry, tol, rf = reference(c)
    ref.check("y", y, ry, tol)
    assert np.array_equal(ref.f64(pool[6]), rf[0]) and np.array_equal(ref.f64(pool[2]), rf[2])
    for i in (0, 1, 3, 4, 5):
        assert torch.equal(pool[i], before[i])
    # a pool that is only read: no final state comes back
    _, none = kda.short_conv(on(c["x"]), on(c["w"]), cu_seqlens=c["cu"], initial_state=pool,
                             slots=slots)
    assert none is None


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_nonfinite_stays_in_its_sequence_and_channel(value):
    print("conv nonfinite", value, flush=True)
    c = case([6, 8, 5], 64, 4, F32, 60)
    x = on(c["x"]).clone()
    x[8, 5] = value  # sequence 1, token 2
    clean, _ = kda.short_conv(on(c["x"]), on(c["w"]), on(c["b"]), cu_seqlens=c["cu"])
    y, _ = kda.short_conv(x, on(c["w"]), on(c["b"]), cu_seqlens=c["cu"])
    torch.cuda.synchronize()
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[8:12, 5] = True
    assert torch.equal(y[~hit], clean[~hit])
    if value != value:
        assert torch.isnan(y[hit]).all()
    else:
        # silu of +inf is inf, of -inf the limit's NaN-free 0 or a NaN of 0 * inf
        assert not torch.equal(y[hit], clean[hit])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,D,W", [(1, 1, 2), (1, 512, 4), (3, 100, 3), (17, 520, 4), (5, 96, 8)])
def test_step(rows, D, W, dtype):
    print("conv step", rows, D, W, dtype, flush=True)
    pool = rand((rows + 4, W - 1, D), dtype, 70).to(DEV)
    before = pool.clone()
    x, w, b = rand((rows, D), dtype, 71), rand((D, W), dtype, 72), rand((D,), dtype, 73)
    perm = torch.randperm(rows + 4, generator=torch.Generator().manual_seed(74))[:rows]
    y = kda.short_conv_step(pool, on(x), on(w), on(b), slots=perm.to(torch.int32).to(DEV))
    torch.cuda.synchronize()
    ry, tol, rs = ref.conv_step(ref.f64(x), ref.f64(before[perm.to(DEV)]), ref.f64(w), ref.f64(b),
                                True, dtype)
    ref.check("y", y, ry, tol)
    assert np.array_equal(ref.f64(pool[perm.to(DEV)]), rs)
    rest = [i for i in range(rows + 4) if i not in perm.tolist()]
    assert torch.equal(pool[rest], before[rest])


def test_step_skips_padding_rows_and_runs_in_place():
    print("conv step padding", flush=True)
    st = rand((3, 3, 64), BF16, 80).to(DEV)
    before = st.clone()
    x = rand((4, 64), BF16, 81).to(DEV)
    keep = x.clone()
    w = rand((64, 4), BF16, 82).to(DEV)
    slots = torch.tensor([2, -1, 3, 0], dtype=torch.int32, device=DEV)
    y = kda.short_conv_step(st, x, w, slots=slots, activation=None, y=x)
    torch.cuda.synchronize()
    assert y is x
    assert torch.equal(x[1:3], keep[1:3])
    assert torch.equal(st[1], before[1])
    at = [2, 0]
    ry, tol, rs = ref.conv_step(ref.f64(keep[[0, 3]]), ref.f64(before[at]), ref.f64(w), None, False, BF16)
    ref.check("y", x[[0, 3]], ry, tol)
    assert np.array_equal(ref.f64(st[at]), rs)


def test_steps_continue_a_prompt():
    """A prompt, then token by token from its final state: the outputs of the
    whole prompt, bit for bit (the same sums in the same order)."""
    print("conv prompt then steps", flush=True)
    c = case([70, 20], 96, 4, BF16, 90)
    x, w, b = (on(c[k]) for k in ("x", "w", "b"))
    whole, fin = kda.short_conv(x, w, b, cu_seqlens=c["cu"])
    _, st = kda.short_conv(torch.cat([x[:60], x[70:80]]), w, b, cu_seqlens=[0, 60, 70])
    for i in range(10):
        y = kda.short_conv_step(st, torch.stack([x[60 + i], x[80 + i]]), w, b)
        assert torch.equal(y, torch.stack([whole[60 + i], whole[80 + i]]))
    assert torch.equal(st, fin)


def test_offsets_past_32_bits():
    """The last columns of a matrix of more than 2^31 elements, and a late
    slice of a pool of more than 2^31 elements."""
    print("conv offsets past 32 bits", flush=True)
    T, stride = 60000, 36864
    wide = torch.empty((T, stride), dtype=BF16, device=DEV)
    x = wide[:, -64:]
    g = torch.Generator(device=DEV).manual_seed(100)
    x.copy_(torch.randn((T, 64), device=DEV, generator=g))
    w = rand((64, 4), BF16, 101).to(DEV)
    y, fin = kda.short_conv(x, w)
    small, fin2 = kda.short_conv(x.contiguous(), w)
    assert torch.equal(y, small) and torch.equal(fin, fin2) and torch.equal(fin[0], x[-3:])
    del wide
    D, slots = 36864, 20000
    pool = torch.empty((slots, 3, D), dtype=BF16, device=DEV)
    last = rand((1, 3, D), BF16, 102).to(DEV)
    pool[-1:] = last
    w = rand((D, 4), BF16, 103).to(DEV)
    xt = rand((1, D), BF16, 104).to(DEV)
    y = kda.short_conv_step(pool, xt, w, slots=torch.tensor([slots - 1], dtype=torch.int32, device=DEV))
    y2 = kda.short_conv_step(last, xt, w)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(pool[-1:], last)


@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("dtype,D", [(F32, 7), (BF16, 13)])
@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
def test_infinities_go_where_the_formula_takes_them(value, dtype, D, act):
    """An infinite input in a channel of a whole vector and in one of the
    rest: each sum it enters is infinite with the sign of its weight; silu
    keeps +inf and makes NaN (-inf * 0) of -inf.  A prompt and its steps."""
    print("conv infinities", value, dtype, D, act, flush=True)
    c = case([6, 8, 5], D, 4, dtype, 110, state=False, act=act)
    c["w"] = torch.where(c["w"] == 0, torch.ones_like(c["w"]), c["w"])
    clean, cfin = kda.short_conv(on(c["x"]), on(c["w"]), on(c["b"]), cu_seqlens=c["cu"], activation=act)
    c["x"] = c["x"].clone()
    for d in (2, D - 1):
        c["x"][8, d] = value  # sequence 1, token 2
    y, fin = kda.short_conv(on(c["x"]), on(c["w"]), on(c["b"]), cu_seqlens=c["cu"], activation=act)
    torch.cuda.synchronize()
    want = ref.f64(clean).copy()
    for d in (2, D - 1):
        for j in range(4):  # the input is the weight's of the token j later
            s = np.sign(ref.f64(c["w"])[d, 3 - j]) * value
            want[8 + j, d] = s if act is None or s > 0 else np.nan
    assert np.array_equal(ref.f64(y), want, equal_nan=True)
    assert np.array_equal(ref.f64(fin), ref.f64(cfin))
    _, st = kda.short_conv(on(c["x"][6:8]), on(c["w"]), on(c["b"]), activation=act)
    for t in range(8, 14):
        y1 = kda.short_conv_step(st, on(c["x"][t:t + 1]), on(c["w"]), on(c["b"]), activation=act)
        assert np.array_equal(ref.f64(y1)[0], want[t], equal_nan=True)
