"""Selective scan on the GPU against the 64-bit recurrence, elementwise within
the bound that follows its roundings step by step."""
import numpy as np
import pytest
import torch

import gated_delta_rule_19_amd as kda
import recurrent_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def case(lengths, D, N, G, dtype, seed, gate=True, skip=True, bias=True, state=True, softplus=True,
         slow=False):
    g = torch.Generator().manual_seed(seed)
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)
    T = int(cu[-1])
    f = lambda *s: torch.randn(s, generator=g)
    step = torch.exp(torch.rand((D,), generator=g) * 4.6 - 6.9)  # 0.001 .. 0.1
    if slow:
        step = step * 0.02
    c = dict(x=f(T, D).to(dtype), A=-torch.arange(1.0, N + 1) * torch.exp(0.1 * f(D, N)),
             B=f(T, G, N).to(dtype), C=f(T, G, N).to(dtype), D=f(D) if skip else None,
             z=f(T, D).to(dtype) if gate else None, cu=cu, softplus=softplus,
             s=f(len(lengths), D, N) if state else None)
    if softplus:
        c["delta"] = (0.5 * f(T, D)).to(dtype)
        c["bias"] = step + torch.log(-torch.expm1(-step)) if bias else None
    else:
        c["delta"] = (step * torch.exp(0.3 * f(T, D))).to(dtype)
        c["bias"] = step * 0.1 if bias else None
    return c


def on(t):
    return None if t is None else t.to(DEV)


def args(c):
    return dict(x=on(c["x"]), delta=on(c["delta"]), A=on(c["A"]), B=on(c["B"]), C=on(c["C"]),
                D=on(c["D"]), z=on(c["z"]), delta_bias=on(c["bias"]), delta_softplus=c["softplus"])


def reference(c, fold=2.0):
    return ref.scan(*(ref.f64(c[k]) for k in ("x", "delta", "A", "B", "C", "D", "z", "bias")),
                    c["softplus"], c["cu"], ref.f64(c["s"]), c["x"].dtype, fold)


def compare(c, y, fin):
    ry, yt, rf, ft = reference(c)
    ref.check("y", y, ry, yt)
    ref.check("final state", fin, rf, ft)


def run(c, **kw):
    y, fin = kda.selective_scan(**args(c), cu_seqlens=c["cu"], initial_state=on(c["s"]), **kw)
    torch.cuda.synchronize()
    return y, fin


LENGTHS = {
    "one": [1], "two": [2], "tile": [32], "past": [33], "odd": [131], "long": [1000],
    "mixed": [0, 1, 2, 3, 0, 64, 65, 7, 200, 0], "many": [(i * 7) % 13 for i in range(120)],
    "edge": [3] * 65, "none": [0, 0],
}


@pytest.mark.parametrize("split", [0, 1, 3])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lens", sorted(LENGTHS))
def test_lengths(lens, dtype, split):
    print("scan lengths", lens, dtype, split, flush=True)
    c = case(LENGTHS[lens], 70, 16, 1, dtype, 10)
    compare(c, *run(c, split_hint=split))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 8, 13, 16, 17, 32, 48, 63, 64, 65, 128])
def test_state_counts(N, dtype):
    print("scan states", N, dtype, flush=True)
    c = case([37, 70], 66, N, 2, dtype, 20 + N)
    for split in (1, 2):
        compare(c, *run(c, split_hint=split))


@pytest.mark.parametrize("D,G", [(1, 1), (3, 3), (64, 1), (65, 1), (128, 4), (390, 2), (130, 13)])
def test_channels_and_groups(D, G):
    print("scan channels", D, "groups", G, flush=True)
    c = case([41, 6], D, 16, G, F32, 40 + D)
    compare(c, *run(c))


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("softplus,bias", [(True, False), (False, True), (False, False)])
def test_options(gate, skip, softplus, bias):
    print("scan options", gate, skip, softplus, bias, flush=True)
    for dtype in (F32, BF16):
        c = case([50, 9], 64, 8, 1, dtype, 50, gate=gate, skip=skip, softplus=softplus, bias=bias,
                 state=gate)
        compare(c, *run(c, split_hint=2))


@pytest.mark.parametrize("split", [0, 7, 50])
def test_long_memory_across_segments(split):
    """Slow decay: the entry state of every segment matters to its end."""
    print("scan long memory", split, flush=True)
    c = case([3000, 1700], 64, 16, 1, F32, 60, slow=True)
    compare(c, *run(c, split_hint=split))


def test_softplus_over_its_range():
    """delta's argument from far below 0 (delta underflows to it) to far
    above (delta is the argument), around 20 and around 0."""
    print("scan softplus range", flush=True)
    c = case([64], 64, 4, 1, F32, 70, bias=False, state=False)
    lin = torch.cat([torch.linspace(-100, 100, 2048), torch.linspace(-1, 1, 1024),
                     torch.linspace(19, 21, 1024)])
    c["delta"] = lin.reshape(64, 64).contiguous()
    compare(c, *run(c))


def test_extreme_decays_and_growth():
    """A of size 0 (a plain sum), large negative (no memory), positive."""
    print("scan extreme decays", flush=True)
    c = case([90], 64, 4, 1, F32, 80)
    c["A"] = torch.tensor([0.0, -1e4, 0.5, -1e-6]).repeat(64, 1)
    for split in (1, 2):
        compare(c, *run(c, split_hint=split))


def test_column_ranges_and_alignment():
    """Every token matrix as a column range of one projection's output, at odd
    element offsets; y too, and nothing else is written."""
    print("scan columns", flush=True)
    D, N, G, T = 70, 5, 2, 43
    for dtype in (F32, BF16):
        c = case([40, 3], D, N, G, dtype, 90)
        wide = torch.full((T, 5 * 71 + 2 * G * N + 9), 7.0, dtype=dtype, device=DEV)
        a = args(c)
        at = 1
        used = []
        for k in ("x", "delta", "z", "y", "B", "C"):
            w = G * N if k in "BC" else D
            view = wide[:, at:at + w]
            if k != "y":
                view.copy_(a[k].reshape(T, w))
            a[k] = view.view(T, G, N) if k in "BC" else view
            used.append((at, at + w))
            at += w + 1
        keep = wide.clone()
        y, fin = kda.selective_scan(**a, cu_seqlens=c["cu"], initial_state=on(c["s"]))
        torch.cuda.synchronize()
        compare(c, y, fin)
        lo, hi = used[3]
        assert torch.equal(wide[:, :lo], keep[:, :lo]) and torch.equal(wide[:, hi:], keep[:, hi:])


def test_in_place_state_and_resume():
    print("scan resume", flush=True)
    c = case([300, 2, 31], 70, 16, 1, F32, 100)
    s = on(c["s"])
    a = args(c)
    first = list(range(0, 150)) + [300] + list(range(302, 321))
    rest = list(range(150, 300)) + [301] + list(range(321, 333))
    y = torch.empty_like(a["x"])
    for rows, cu in ((first, [0, 150, 151, 170]), (rest, [0, 150, 151, 163])):
        b = dict(a)
        for k in ("x", "delta", "B", "C", "z"):
            b[k] = a[k][rows]
        out, fin = kda.selective_scan(**b, cu_seqlens=cu, initial_state=s, final_state=s, split_hint=3)
        assert fin is s
        y[rows] = out
    torch.cuda.synchronize()
    compare(c, y, s)


def test_slots_pick_slices_and_padding_keeps_out():
    print("scan slots", flush=True)
    for split in (1, 4):
        c = case([150, 90, 3, 0], 40, 16, 1, F32, 110)
        pool = torch.randn((7, 40, 16), generator=torch.Generator().manual_seed(111)).to(DEV)
        before = pool.clone()
        slots = torch.tensor([6, -1, 2, 99], dtype=torch.int32, device=DEV)
        y, fin = kda.selective_scan(**args(c), cu_seqlens=c["cu"], initial_state=pool,
                                    final_state=pool, slots=slots, split_hint=split)
        torch.cuda.synchronize()
        zero = torch.zeros_like(before[0])
        c["s"] = torch.stack([before[6], zero, before[2], zero]).cpu()
        ry, yt, rf, ft = reference(c)
        ref.check("y", y, ry, yt)
        ref.check("final", pool[[6, 2]], rf[[0, 2]], ft[[0, 2]])
        for i in (0, 1, 3, 4, 5):
            assert torch.equal(pool[i], before[i])


@pytest.mark.parametrize("split", [1, 3])
def test_nonfinite_stays_where_the_formula_takes_it(split):
    """A NaN input spoils its channel from its token on, in its sequence only;
    one in B spoils its state in every channel."""
    print("scan nonfinite", split, flush=True)
    c = case([100, 210, 64], 64, 8, 2, F32, 120, state=False)
    clean, cfin = run(c, split_hint=split)
    d = dict(c, x=c["x"].clone())
    d["x"][130, 5] = float("nan")
    y, fin = run(d, split_hint=split)
    hit = torch.zeros_like(clean, dtype=torch.bool)
    hit[130:310, 5] = True
    assert torch.isnan(y[hit]).all() and torch.equal(y[~hit], clean[~hit])
    assert torch.isnan(fin[1, 5]).all()
    fin[1, 5] = cfin[1, 5]
    assert torch.equal(fin, cfin)
    d = dict(c, B=c["B"].clone())
    d["B"][99, 1, 3] = float("inf")  # the last token of sequence 0, group 1
    y, fin = run(d, split_hint=split)
    hit[:] = False
    hit[99, 32:] = True
    assert not torch.isfinite(y[hit]).any() and torch.equal(y[~hit], clean[~hit])
    bad = torch.zeros_like(fin, dtype=torch.bool)
    bad[0, 32:, 3] = True
    assert not torch.isfinite(fin[bad]).any() and torch.equal(fin[~bad], cfin[~bad])


def test_repeats_bit_for_bit_and_rows_do_not_depend_on_the_batch():
    print("scan repeats", flush=True)
    c = case([257, 64], 130, 16, 1, BF16, 130)
    y, fin = run(c, split_hint=4)
    y2, fin2 = run(c, split_hint=4)
    assert torch.equal(y, y2) and torch.equal(fin, fin2)
    d = {k: (v[257:] if k in ("x", "delta", "B", "C", "z") else v) for k, v in c.items()}
    d.update(cu=np.array([0, 64]), s=c["s"][1:])
    y3, fin3 = run(d, split_hint=1)
    y4, fin4 = run(c, split_hint=1)
    assert torch.equal(y3, y4[257:]) and torch.equal(fin3, fin4[1:])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,D,N,G", [(1, 1, 1, 1), (1, 64, 16, 1), (3, 70, 13, 2), (9, 260, 16, 4),
                                        (2, 66, 65, 1), (2, 66, 128, 3), (5, 33, 6, 3), (2, 40, 64, 1)])
def test_step(rows, D, N, G, dtype):
    print("scan step", rows, D, N, G, dtype, flush=True)
    c = case([1] * rows, D, N, G, dtype, 140, gate=rows != 3, skip=rows != 2, bias=rows != 5)
    pool = torch.randn((rows + 4, D, N), generator=torch.Generator().manual_seed(141)).to(DEV)
    before = pool.clone()
    perm = torch.randperm(rows + 4, generator=torch.Generator().manual_seed(142))[:rows]
    y = kda.selective_scan_step(pool, **args(c), slots=perm.to(torch.int32).to(DEV))
    torch.cuda.synchronize()
    c["s"] = before.cpu()[perm]
    ry, yt, rf, ft = reference(c, 1.0)
    # (the step's sum over the states runs over lanes: as many roundings)
    ref.check("y", y, ry, yt)
    ref.check("state", pool[perm.to(DEV)], rf, ft)
    rest = [i for i in range(rows + 4) if i not in perm.tolist()]
    assert torch.equal(pool[rest], before[rest])


def test_step_skips_padding_rows():
    print("scan step padding", flush=True)
    c = case([1] * 4, 64, 16, 1, BF16, 150)
    pool = torch.randn((3, 64, 16), generator=torch.Generator().manual_seed(151)).to(DEV)
    before = pool.clone()
    y = torch.full((4, 64), 7.0, dtype=BF16, device=DEV)
    slots = torch.tensor([2, -5, 3, 0], dtype=torch.int32, device=DEV)
    out = kda.selective_scan_step(pool, **args(c), slots=slots, y=y)
    torch.cuda.synchronize()
    assert out is y and (y[1:3] == 7).all() and torch.equal(pool[1], before[1])
    c["s"] = torch.stack([before[2], before[0], before[0], before[0]]).cpu()
    ry, yt, rf, ft = reference(c, 1.0)
    ref.check("y", y[[0, 3]], ry[[0, 3]], yt[[0, 3]])
    ref.check("state", pool[[2, 0]], rf[[0, 3]], ft[[0, 3]])


def test_steps_continue_a_prompt():
    print("scan prompt then steps", flush=True)
    c = case([90, 20], 70, 16, 1, F32, 160)
    a = args(c)
    rows = list(range(80)) + list(range(90, 100))
    b = {k: (v[rows] if k in ("x", "delta", "B", "C", "z") else v) for k, v in a.items()}
    y = torch.empty_like(a["x"])
    out, st = kda.selective_scan(**b, cu_seqlens=[0, 80, 90], initial_state=on(c["s"]))
    y[rows] = out
    for i in range(10):
        r = [80 + i, 100 + i]
        b = {k: (v[r] if k in ("x", "delta", "B", "C", "z") else v) for k, v in a.items()}
        y[r] = kda.selective_scan_step(st, **b)
    torch.cuda.synchronize()
    compare(c, y, st)


def test_offsets_past_32_bits():
    print("scan offsets past 32 bits", flush=True)
    T, stride = 60000, 36864
    wide = torch.empty((T, stride), dtype=BF16, device=DEV)
    c = case([T], 64, 4, 1, BF16, 170, gate=False, state=False)
    a = args(c)
    x = wide[:, -64:]
    x.copy_(a["x"])
    y, fin = kda.selective_scan(**dict(a, x=x))
    y2, fin2 = kda.selective_scan(**a)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(fin, fin2)
    del wide
    D, slots = 12288, 12000
    pool = torch.empty((slots, D, 16), device=DEV)
    c = case([1], D, 16, 1, BF16, 171)
    a = args(c)
    pool[-1:] = on(c["s"])
    last = on(c["s"])
    y = kda.selective_scan_step(pool, **a, slots=torch.tensor([slots - 1], dtype=torch.int32, device=DEV))
    y2 = kda.selective_scan_step(last, **a)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(pool[-1:], last)


@pytest.mark.parametrize("name,lengths,D,N,G", [
    ("many short prompts of many channels", [1 + i % 5 for i in range(300)], 1024, 16, 1),
    ("few states, many prompts", [7] * 100, 512, 3, 2),
    ("many states, one long prompt", [2100, 40], 64, 20, 1),
    ("all states, one long prompt", [1030], 32, 128, 2),
    ("one long prompt", [4000], 128, 16, 1),
])
def test_automatic_choice_at_its_edges(name, lengths, D, N, G):
    """Shapes for which the call picks each of its kernels and cuts by itself."""
    print("scan", name, flush=True)
    for dtype in (F32, BF16):
        c = case(lengths, D, N, G, dtype, 180)
        compare(c, *run(c))


@pytest.mark.parametrize("N", [16, 20])
def test_many_cut_sequences(N):
    """More sequences than the inline table, several of them cut, others not."""
    print("scan many cut sequences", N, flush=True)
    c = case([(i * 53) % 300 for i in range(90)], 66, N, 1, F32, 190)
    compare(c, *run(c, split_hint=6))


@pytest.mark.parametrize("lens", [[37], [100, 3, 70]])
@pytest.mark.parametrize("split", [1, 3])
def test_infinite_rates_forget(lens, split):
    """A = -inf drops the state at every token, as any very large rate does,
    also at lengths that end inside a tile."""
    print("scan infinite rates", lens, split, flush=True)
    c = case(lens, 66, 16, 1, F32, 200)
    c["A"][:, 3] = -1e30
    c["A"][5] = -1e30
    y, fin = run(c, split_hint=split)
    c["A"][:, 3] = -float("inf")
    c["A"][5] = -float("inf")
    y2, fin2 = run(c, split_hint=split)
    assert torch.isfinite(y).all() and torch.equal(y, y2) and torch.equal(fin, fin2)


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_nonfinite_states_stay_in_their_slice(value):
    """An infinite or NaN initial state spoils its own channel of its own
    sequence, whose final state keeps it, and nothing else."""
    print("scan nonfinite state", value, flush=True)
    for split in (1, 3):
        c = case([90, 41, 130], 66, 16, 1, F32, 210)
        clean, cfin = run(c, split_hint=split)
        c["s"] = c["s"].clone()
        c["s"][1, 7, 2] = value
        y, fin = run(c, split_hint=split)
        hit = torch.zeros_like(y, dtype=torch.bool)
        hit[90:131, 7] = True
        assert torch.equal(y[~hit], clean[~hit]) and not torch.isfinite(y[hit]).any()
        assert not torch.isfinite(fin[1, 7, 2])
        fin[1, 7, 2] = cfin[1, 7, 2]
        assert torch.equal(fin, cfin)


def test_rows_past_the_last_sequence_are_left_alone():
    """Through the C ABI: buffers longer than the packed tokens."""
    print("scan rows past the end", flush=True)
    import ctypes
    from gated_delta_rule_19_amd import _native as nat
    c = case([45, 20], 70, 16, 1, BF16, 220)
    a = args(c)
    want, _ = run(c, split_hint=1)
    y = torch.full((80, 70), 7.0, dtype=BF16, device=DEV)
    io = nat.SsmIo()
    for k, t, w in (("x", a["x"], 70), ("delta", a["delta"], 70), ("z", a["z"], 70), ("y", y, 70),
                    ("B", a["B"], 16), ("C", a["C"], 16)):
        setattr(io, k, t.data_ptr())
        setattr(io, k + "_stride", w)
    io.A, io.D_skip, io.delta_bias = (a[k].data_ptr() for k in ("A", "D", "delta_bias"))
    io.delta_softplus = 1
    cu = np.ascontiguousarray(c["cu"])
    s = on(c["s"])
    st = nat.load().kda_selective_scan(2, cu.ctypes.data, 70, 16, 1, nat.KDA_BF16, ctypes.byref(io),
                                       s.data_ptr(), None, None, 2, 1, None, 0,
                                       torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == nat.KDA_OK
    assert torch.equal(y[:65], want) and (y[65:] == 7).all()


def test_long_prompt_of_few_channels():
    """20000 tokens of 1536 channels, which the call cuts on its own; the
    recurrence and its bound (as in recurrent_ref.scan) in 64 bits on the
    device."""
    print("scan long prompt", flush=True)
    T, D, N = 20000, 1536, 16
    c = case([T], D, N, 1, F32, 230, gate=False, skip=False)
    a = args(c)
    y, fin = kda.selective_scan(**a, initial_state=on(c["s"]))
    U = ref.U
    x, A, B, C = (a[k].double() for k in ("x", "A", "B", "C"))
    lin = a["delta"].double() + a["delta_bias"].double()
    d = torch.logaddexp(lin, torch.zeros_like(lin))
    rd = torch.where(lin > 0, torch.full_like(lin, 16 * U), U * (3 * lin.abs() + 12))
    h = on(c["s"])[0].double()
    E = torch.zeros_like(h)
    worst = torch.zeros((), dtype=torch.float64, device=DEV)
    for t in range(T):
        dt_, r = d[t][:, None], rd[t][:, None]
        arg = dt_ * A
        decay = torch.exp(arg)
        hold, inp = decay * h, (d[t] * x[t])[:, None] * B[t]
        E = decay * E + hold.abs() * (arg.abs() * (r + 3 * U) + 2 * U) + inp.abs() * (r + 2 * U)
        h = hold + inp
        E = E + U * h.abs()
        term = C[t] * h
        v = term.sum(1)
        # (2 E: the cut; N + 3 roundings of the sum; the output's own)
        tol = (C[t].abs() * E * 2).sum(1) + (N + 3) * U * term.abs().sum(1) + U * v.abs() + 1e-37
        worst = torch.maximum(worst, ((y[t].double() - v).abs() / tol).max())
    assert worst.item() <= 1
    assert ((fin[0].double() - h).abs() <= 2 * E + 1e-37).all()


def infinite(lens, N, seed, skip, what, at):
    """A case of positive terms with one infinite input: every sum that it
    enters is infinite, none is the difference of two."""
    c = case(lens, 66, N, 1, F32, seed, skip=skip)
    for k in ("x", "B", "C", "s", "D"):
        if c[k] is not None:
            c[k] = c[k].abs()
    c["z"] = c["z"].abs() + 0.1
    c[what] = c[what].clone()
    c[what][at, 5] = float("inf")
    return c


def same_classes(name, got, want, tol):
    """Infinities where the reference has them, the others within the bound."""
    got = ref.f64(got)
    inf = np.isinf(want)
    assert inf.any() and not np.isnan(want).any()
    assert np.array_equal(got[inf], want[inf]), name
    ref.check(name, np.where(inf, 0.0, got), np.where(inf, 0.0, want), np.where(inf, 0.0, tol))


@pytest.mark.parametrize("what", ["x", "delta"])
@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("N", [1, 3, 5, 8, 12, 16, 20, 40, 65, 128])
def test_infinite_inputs_stay_infinite(N, skip, what):
    """Without a skip, and with state counts that fill no register, lane or
    tile: what is not there adds no 0 * inf."""
    print("scan infinite inputs", N, skip, what, flush=True)
    for lens, at in (([90, 41, 130], 100), ([230], 17), ([230], 100)):
        c = infinite(lens, N, 240 + N, skip, what, at)
        ry, yt, rf, ft = reference(c)
        for split in (1, 4):
            y, fin = run(c, split_hint=split)
            same_classes("y", y, ry, yt)
            same_classes("final state", fin, rf, ft)


@pytest.mark.parametrize("what", ["x", "delta"])
@pytest.mark.parametrize("N", [1, 3, 5, 12, 16, 20, 65, 67, 127, 128])
def test_infinite_inputs_of_a_step(N, what):
    print("scan step infinite inputs", N, what, flush=True)
    for skip in (False, True):
        c = infinite([1] * 5, N, 260 + N, skip, what, 3)
        ry, yt, rf, ft = reference(c, fold=1.0)
        state = on(c["s"]).clone()
        y = kda.selective_scan_step(state, **args(c))
        torch.cuda.synchronize()
        same_classes("y", y, ry, yt)
        same_classes("state", state, rf, ft)


@pytest.mark.parametrize("N", [16, 20])
@pytest.mark.parametrize("split", [1, 4])
def test_steps_whose_sum_passes_the_largest_number(N, split):
    """A rate of 0 keeps its state over any finite step, also over a segment
    whose steps add up to more than an fp32 holds."""
    print("scan large steps", N, split, flush=True)
    c = case([300], 66, N, 1, F32, 280, softplus=False, bias=False)
    c["A"][:, 2] = 0.0
    for t in (100, 110, 200):
        c["delta"][t, 5] = 2e38
        c["x"][t, 5] = 0.0
    compare(c, *run(c, split_hint=split))


@pytest.mark.parametrize("N", range(1, 17))
def test_every_state_count_of_one_lane(N):
    """split_hint > 1 and many sequences: all states of a channel in a lane,
    in a kernel of their own for each count."""
    print("scan lane states", N, flush=True)
    for dtype in (F32, BF16):
        c = case([70, 150, 33], 66, N, 2, dtype, 290 + N)
        compare(c, *run(c, split_hint=2))


@pytest.mark.parametrize("N", [4, 16])
def test_infinite_states_outlast_a_segment(N):
    """The decay over a segment, not that of a step, underflows: what is
    infinite before it is infinite after it, cut or not."""
    print("scan infinite states over segments", N, flush=True)
    for at in (17, 100):
        c = infinite([700], N, 320, False, "x", at)
        c["bias"] = None
        c["A"] = -1.0 - 3.0 * torch.rand((66, N), generator=torch.Generator().manual_seed(321))
        ry, yt, rf, ft = reference(c)
        for split in (1, 5, 21):
            y, fin = run(c, split_hint=split)
            same_classes("y", y, ry, yt)
            same_classes("final state", fin, rf, ft)


def cut_of_row_kernel(c, D, N, G):
    """Whether the call by itself runs the row kernel in segments: its
    workspace holds 16 end states and a sum of steps for every segment pair
    and channel (the lane kernel's N and one)."""
    from gated_delta_rule_19_amd import _native as nat
    cu = np.ascontiguousarray(c["cu"])
    size = nat.load().kda_selective_scan_workspace_size(len(cu) - 1, cu.ctypes.data, D, N, G, 0)
    pair = 256 * G * ((D // G + 63) // 64)
    return size > 0 and size % (17 * pair) == 0 and size % ((N + 1) * pair) != 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,G", [(5, 1), (5, 2), (13, 1), (13, 2), (12, 1)])
def test_cut_row_kernel_of_few_states(N, G, dtype):
    """A long prompt of few channels with states that do not fill 16 lanes."""
    print("scan cut row kernel", N, G, dtype, flush=True)
    c = case([3000], 66, N, G, dtype, 330 + N)
    assert cut_of_row_kernel(c, 66, N, G)
    compare(c, *run(c))
    slow = case([3000], 66, N, G, dtype, 331 + N, slow=True, skip=False)
    compare(slow, *run(slow))


@pytest.mark.parametrize("what", ["x", "delta"])
@pytest.mark.parametrize("N", [5, 12, 13])
def test_infinite_inputs_of_the_cut_row_kernel(N, what):
    """In the first segment, a middle one and the last."""
    print("scan cut row kernel, infinite", N, what, flush=True)
    for at in (17, 1500, 2990):
        c = infinite([3000], N, 340 + N, False, what, at)
        assert cut_of_row_kernel(c, 66, N, 1)
        ry, yt, rf, ft = reference(c)
        y, fin = run(c)
        same_classes("y", y, ry, yt)
        same_classes("final state", fin, rf, ft)


@pytest.mark.parametrize("N", [5, 13])
def test_nan_of_the_cut_row_kernel_stays_in_its_channel(N):
    print("scan cut row kernel, NaN", N, flush=True)
    c = case([3000], 66, N, 1, F32, 350 + N)
    assert cut_of_row_kernel(c, 66, N, 1)
    clean, cfin = run(c)
    for at in (17, 1500, 2990):
        d = dict(c, x=c["x"].clone())
        d["x"][at, 5] = float("nan")
        y, fin = run(d)
        hit = torch.zeros_like(clean, dtype=torch.bool)
        hit[at:, 5] = True
        assert torch.isnan(y[hit]).all() and torch.equal(y[~hit], clean[~hit])
        assert torch.isnan(fin[0, 5]).all()
        fin[0, 5] = cfin[0, 5]
        assert torch.equal(fin, cfin)


@pytest.mark.parametrize("softplus", [False, True])
@pytest.mark.parametrize("N", [5, 16, 65, 67])
def test_infinite_rates_of_a_step(N, softplus):
    """A = -inf drops the state at every step but one of 0, which keeps it: as
    in a prompt of one token, and as any very large rate."""
    print("scan step infinite rates", N, softplus, flush=True)
    c = case([1] * 4, 66, N, 1, F32, 360 + N, softplus=softplus, bias=False)
    c["delta"][1] = -300.0 if softplus else 0.0  # (its softplus underflows)
    c["delta"][2, ::2] = -300.0 if softplus else 0.0
    c["A"][:, 3] = -1e30
    c["A"][5] = -1e30
    out = []
    for rate in (-1e30, -float("inf")):
        c["A"][:, 3] = rate
        c["A"][5] = rate
        state = on(c["s"]).clone()
        y = kda.selective_scan_step(state, **args(c))
        py, pfin = run(c)
        out.append((y, state, py, pfin))
    assert all(torch.isfinite(t).all() for t in out[0])
    assert all(torch.equal(a, b) for a, b in zip(*out))
    assert torch.equal(out[1][1][1, 5], on(c["s"])[1, 5])  # a step of 0 keeps the state
    c["A"][:, 3] = -1e30
    c["A"][5] = -1e30
    ry, yt, rf, ft = reference(c, 1.0)
    ref.check("y", out[1][0], ry, yt)
    ref.check("state", out[1][1], rf, ft)
