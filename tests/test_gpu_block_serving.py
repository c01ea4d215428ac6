"""The decayed attention, the block norm, beam selection and state reordering
as a server uses them: a beam search over a small model, in graphs, on streams
of their own, and the attention at the sizes where it changes its way of
working."""
import numpy as np
import pytest
import torch

import block_ref as ref
import gated_delta_rule_19_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def f(g, *shape):
    return torch.randn(shape, device=DEV, generator=g)


# ---- the attention's ways of working ------------------------------------------------

def attention(lengths, H, dk, dv, dtype, seed, bad=(), shift=0, split=0, Hq=None):
    """One call against the 64-bit form; `bad`: tokens whose k holds an
    infinity (the outputs before them in their sequence stay what they are)."""
    cu = [0] + np.cumsum(lengths).tolist()
    T, N = cu[-1], len(lengths)
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g)
    Hq = Hq or H
    # (elements in front, so that rows start at an odd element where shift is 1)
    q, k, v = (torch.cat([torch.zeros(shift), (rand(T * h * d) * s)]).to(dtype)
               for h, d, s in ((Hq, dk, 1.0), (H, dk, dk ** -0.5), (H, dv, 1.0)))
    gl = -torch.rand(T, H, generator=g) * 0.3
    init = rand(N, H, dk, dv)
    dq, dk_, dv_ = (x.to(DEV)[shift:].view(T, h, d) for x, h, d in ((q, Hq, dk), (k, H, dk), (v, H, dv)))
    q, k, v = dq.cpu(), dk_.cpu(), dv_.cpu()
    for t in bad:
        dk_[t, 0, 0] = float("inf")
    o, fin = kda.decay_attention(dq, dk_, dv_, gl.to(DEV), scale=dk ** -0.5, cu_seqlens=cu,
                                 initial_state=init.to(DEV), split_hint=split)
    torch.cuda.synchronize()
    want, otol, wfin, ftol = ref.decay_attention(ref.f64(q), ref.f64(k), ref.f64(v), ref.f64(gl), dk ** -0.5, cu,
                                                 ref.f64(init), dtype)
    o, fin = o.cpu(), fin.cpu()
    for n in range(N):
        hit = [t for t in bad if cu[n] <= t < cu[n + 1]]
        end = min(hit) if hit else cu[n + 1]
        ref.check("o", o[cu[n]:end], want[cu[n]:end], otol[cu[n]:end])
        clean = slice(1, None) if hit else slice(None)  # (only head 0 meets it)
        ref.check("o behind", o[end:cu[n + 1], clean], want[end:cu[n + 1], clean], otol[end:cu[n + 1], clean])
        ref.check("state", fin[n, clean], wfin[n, clean], ftol[n, clean])
        if hit:
            assert not torch.isfinite(o[end:cu[n + 1], 0].float()).all(-1).any()
            assert not torch.isfinite(fin[n, 0, 0]).any()


MANY = [1, 64, 0, 65, 200, 63, 128] * 10  # with 4 heads of 128: more workgroups than CUs


@pytest.mark.parametrize("bad", [False, True])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lengths,H,dk,dv", [
    ([300, 129, 0, 1, 200], 3, 128, 128), ([300, 129, 0, 1, 200], 3, 64, 96), ([257], 2, 120, 8),
    (MANY, 4, 128, 128), (MANY, 4, 64, 72), (MANY, 8, 32, 48), ([700] + [40] * 60, 5, 104, 128),
    ([150, 70], 2, 200, 160),
])
def test_ways_of_working(lengths, H, dk, dv, dtype, shift, bad):
    print("ways", len(lengths), H, dk, dv, dtype, shift, bad, flush=True)
    cu = np.cumsum(lengths)
    at = [int(cu[0]) - 1] if not bad else [int(cu[0]) * 3 // 4, int(cu[-1]) - 2]
    attention(lengths, H, dk, dv, dtype, 1, at if bad else (), shift)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lengths,H,dk,dv,Hq", [([2200], 1, 128, 128, 1), ([1500, 40, 1400], 2, 64, 64, 1),
                                               ([1290], 1, 200, 40, 1), ([1300], 2, 40, 130, 2)])
def test_long_sequences_are_cut(lengths, H, dk, dv, Hq, dtype):
    print("cut", lengths, H, dk, dv, dtype, flush=True)
    cu = np.concatenate([[0], np.cumsum(lengths)])
    size = kda._native.load().kda_decay_attention_workspace_size(
        len(lengths), cu.astype(np.int64).ctypes.data, H, dk, dv, int(dtype == BF16), 0)
    assert size > 0
    attention(lengths, H, dk, dv, dtype, 2, Hq=Hq)
    # an infinity in a middle segment
    attention(lengths, H, dk, dv, dtype, 3, bad=[700], Hq=Hq)


def test_splits_of_one_prompt_agree():
    """Any cut gives the uncut result, up to the roundings of both."""
    print("splits", flush=True)
    T, H, d = 1000, 3, 128
    g = gen(5)
    q, k, v = f(g, T, H, d).to(BF16), (f(g, T, H, d) * d ** -0.5).to(BF16), f(g, T, H, d).to(BF16)
    gl = -torch.rand(T, H, device=DEV, generator=g) * 0.1
    o1, s1 = kda.decay_attention(q, k, v, gl, split_hint=1)
    _, otol, _, ftol = ref.decay_attention(ref.f64(q), ref.f64(k), ref.f64(v), ref.f64(gl), 1.0, [0, T], None, BF16)
    for split in (2, 3, 5, 16, 1000):
        o, s = kda.decay_attention(q, k, v, gl, split_hint=split)
        ref.check("o", o, ref.f64(o1), 2 * otol)
        ref.check("state", s, ref.f64(s1), 2 * ftol)


# ---- graphs and streams ---------------------------------------------------------------

class Block:
    """One call of each, its inputs in place."""

    def __init__(self, lengths, H, dk, dv, D, W, K, V, dtype, seed):
        g = gen(seed)
        self.cu = [0] + np.cumsum(lengths).tolist()
        T, n = self.cu[-1], len(lengths)
        self.q, self.k, self.v = f(g, T, H, dk).to(dtype), (f(g, T, H, dk) * dk ** -0.5).to(dtype), f(g, T, H, dv).to(dtype)
        self.g = -torch.rand(T, H, device=DEV, generator=g)
        self.state = f(g, n, H, dk, dv)
        self.x, self.gate, self.res = (f(g, T, D).to(dtype) for _ in range(3))
        self.w, self.post = f(g, D), f(g, D)
        self.logits, self.scores = f(g, 2, W, V).to(dtype), f(g, 2, W)
        self.pool = f(g, 2 * K, H, dk, dv)
        self.sq = f(g, 2 * K, H, dk).to(dtype)
        self.sv = f(g, 2 * K, H, dv).to(dtype)
        self.sg = -torch.rand(2 * K, H, device=DEV, generator=g)
        self.K = K

    def tensors(self):
        return [t for t in vars(self).values() if isinstance(t, torch.Tensor)]

    def go(self, split=0, ws=None):
        o, fin = kda.decay_attention(self.q, self.k, self.v, self.g, cu_seqlens=self.cu, initial_state=self.state,
                                     final_state=self.state, split_hint=split, workspace=ws)
        r, y = kda.block_norm(self.x, self.w, residual=self.res, gate=self.gate, post_weight=self.post, scale=0.5)
        s, parents, tokens, done = kda.beam_select(self.logits, self.scores, beams=self.K)
        kda.state_reorder(self.pool, parents % self.K)
        so = kda.decay_attention_step(self.pool, self.sq, self.sq, self.sv, self.sg)
        return [o, fin, r, y, s, parents, tokens, done, so, self.pool]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lengths,split", [([70, 5, 0], 0), ([3] * 64, 1), ([i % 90 for i in range(200)], 0),
                                           ([900, 64, 1], 3), ([700] + [2] * 70, 4)])
def test_captured_calls_replay_equal_eager(lengths, split, dtype):
    """Each replay on new inputs equals the eager calls, with eager calls of
    other shapes between the replays."""
    print("captured block", len(lengths), split, dtype, flush=True)
    shape = (lengths, 2, 64, 72, 300, 3, 4, 5001, dtype)
    b = Block(*shape, seed=1)
    b.go(split)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b.go(split)
    for rep in range(4):
        new = Block(*shape, seed=10 + rep)
        for a, c in zip(b.tensors(), new.tensors()):
            a.copy_(c)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        other = Block([130, 1], 1, 40, 40, 64, 2, 2, 100, dtype, seed=20 + rep).go(2)
        assert all(torch.isfinite(t.float()).all() for t in other)
        want = new.go(split)
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(got, want)):
            assert torch.equal(x, y), (rep, i)


def test_two_graphs_share_a_workspace():
    """Two graphs of other shapes with one workspace, replayed in turn."""
    print("shared workspace", flush=True)
    kinds = [(([900] + [7] * 70), 2, 64, 64), ([i % 40 for i in range(100)] + [800], 3, 32, 40)]
    blocks = [Block(l, H, dk, dv, 64, 2, 2, 100, BF16, seed=i) for i, (l, H, dk, dv) in enumerate(kinds)]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    outs, graphs = [], []
    for b in blocks:
        b.go(3, ws)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(b.go(3, ws))
        graphs.append(gr)
    for rep in range(3):
        for i, (l, H, dk, dv) in enumerate(kinds):
            new = Block(l, H, dk, dv, 64, 2, 2, 100, BF16, seed=30 + 2 * rep + i)
            for a, c in zip(blocks[i].tensors(), new.tensors()):
                a.copy_(c)
            graphs[i].replay()
            want = new.go(3)
            torch.cuda.synchronize()
            for x, y in zip(outs[i], want):
                assert torch.equal(x, y)


def test_two_streams_at_once():
    """The same calls on two streams with different inputs, in flight
    together, equal the calls run alone."""
    print("two streams", flush=True)
    make = lambda i: Block([1400, 3, 700] + [9] * 66, 3, 128, 128, 1000, 4, 5, 40000, BF16, seed=40 + i)
    alone = [[t.clone() for t in make(i).go()] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        blocks = [make(i) for i in range(2)]
        torch.cuda.synchronize()
        both = []
        for s, b in zip(streams, blocks):
            with torch.cuda.stream(s):
                both.append(b.go())
        torch.cuda.synchronize()
        for got, want in zip(both, alone):
            for x, y in zip(got, want):
                assert torch.equal(x, y)


def test_arrays_side_by_side_in_one_buffer():
    """States, outputs and parameters that touch without overlapping are
    accepted, and each call writes its own only."""
    print("side by side", flush=True)
    rows, H, d, D = 5, 2, 32, 64
    b = Block([2, 3], H, d, d, D, 2, 2, 100, F32, seed=50)
    sizes = dict(q=rows * H * d, o=rows * H * d, k=rows * H * d, g=rows * H, state=rows * H * d * d, v=rows * H * d,
                 y=rows * D, x=rows * D, r=rows * D, w=D)
    arena = torch.full((sum(-(-n // 4) * 4 for n in sizes.values()),), 7.0, device=DEV)
    t, at = {}, 0
    for name, n in sizes.items():
        t[name] = arena[at:at + n]
        at += -(-n // 4) * 4
    shaped = {n: t[n].view(rows, H, d) for n in "qkvo"}
    for n in "qkv":
        shaped[n].copy_(getattr(b, n))
    t["g"].view(rows, H).copy_(b.g)
    t["x"].view(rows, D).copy_(b.x)
    t["w"].copy_(b.w)
    state = t["state"].view(rows, H, d, d)
    state.copy_(f(gen(51), rows, H, d, d))
    s0 = state.clone()
    before = arena.clone()
    want = kda.decay_attention_step(s0, b.q, b.k, b.v, b.g)
    _, wy = kda.block_norm(b.x, b.w, residual=b.x)
    o = kda.decay_attention_step(state, shaped["q"], shaped["k"], shaped["v"], t["g"].view(rows, H), o=shaped["o"])
    kda.block_norm(t["x"].view(rows, D), t["w"], residual=t["x"].view(rows, D), residual_out=t["r"].view(rows, D),
                   y=t["y"].view(rows, D))
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(state, s0)
    assert torch.equal(t["y"].view(rows, D), wy) and torch.equal(t["r"].view(rows, D), 2 * b.x)
    for n in ("q", "k", "v", "g", "x", "w"):
        lo = t[n].storage_offset()
        assert torch.equal(t[n], before[lo:lo + t[n].numel()])


# ---- a beam search -----------------------------------------------------------------------

class Model:
    """A block of convolution, decayed attention and norms between an
    embedding and logits, fp32; beside it a KDA layer fed from tables of its
    own, whose states the beams take along."""

    V, D, H, DK, DV, WIDTH = 300, 64, 2, 24, 40, 4

    def __init__(self):
        g = gen(60)
        H, dk, dv, D = self.H, self.DK, self.DV, self.D
        self.embed = f(g, self.V, D)
        self.norm_in = 1 + 0.1 * f(g, D)
        self.C = 2 * H * dk + H * dv
        self.proj = f(g, D, self.C) * D ** -0.5
        self.conv = f(g, self.C, self.WIDTH) * 0.5
        self.decay = -torch.tensor([0.05, 0.4], device=DEV)
        self.out = f(g, H * dv, D) * (H * dv) ** -0.5
        self.gate = f(g, D, D) * D ** -0.5
        self.post, self.norm_out = 1 + 0.1 * f(g, D), 1 + 0.1 * f(g, D)
        self.head = f(g, D, self.V) * 1.5 * D ** -0.5
        kq = lambda: torch.nn.functional.normalize(f(g, self.V, 2, 128), dim=-1).to(BF16)
        self.kda_q, self.kda_k, self.kda_v = kq(), kq(), f(g, self.V, 2, 128).to(BF16)
        self.kda_g = -torch.rand(self.V, 2, 128, device=DEV, generator=g)
        self.kda_beta = torch.rand(self.V, 2, device=DEV, generator=g)

    def parts(self, c):
        n = self.H * self.DK
        return (c[:, :n].unflatten(1, (self.H, self.DK)), c[:, n:2 * n].unflatten(1, (self.H, self.DK)),
                c[:, 2 * n:].unflatten(1, (self.H, self.DV)))

    def head_of(self, x, o):
        _, y = kda.block_norm(o.flatten(1) @ self.out, self.norm_out, residual=x, gate=x @ self.gate,
                              post_weight=self.post, scale=0.7)
        return y @ self.head

    def prompt(self, tokens, cu, conv, state):
        """Logits of all tokens; the states after each sequence into the pools."""
        x = self.embed[tokens]
        _, h = kda.block_norm(x, self.norm_in)
        c, _ = kda.short_conv(h @ self.proj, self.conv, cu_seqlens=cu, initial_state=conv, final_state=conv)
        q, k, v = self.parts(c)
        o, _ = kda.decay_attention(q, k, v, self.decay, cu_seqlens=cu, initial_state=state, final_state=state)
        return self.head_of(x, o)

    def step(self, tokens, conv, state):
        x = self.embed[tokens]
        _, h = kda.block_norm(x, self.norm_in)
        q, k, v = self.parts(kda.short_conv_step(conv, h @ self.proj, self.conv))
        return self.head_of(x, kda.decay_attention_step(state, q, k, v, self.decay))

    def kda_step(self, tokens, state):
        cast = lambda t: t[tokens].contiguous()
        return kda.decode_step(state, cast(self.kda_q), cast(self.kda_k), cast(self.kda_v), cast(self.kda_g).to(BF16),
                               cast(self.kda_beta).to(BF16))

    def pools(self, n):
        return (torch.zeros(n, self.WIDTH - 1, self.C, device=DEV),
                torch.zeros(n, self.H, self.DK, self.DV, device=DEV),
                torch.zeros(n, 2, 128, 128, device=DEV))


@pytest.mark.parametrize("order", ["score", "rows"])
def test_beam_search(order):
    """Prompts, then 9 tokens of beam search: the states that follow the beams
    are those of running each chosen sequence alone, the scores the sums of
    its log-probabilities.

    The bound: prompts and steps, and products over other batches, round in
    another order.  A logit passes three products of at most 80 terms, two
    norms and the sums over 30 tokens, a state less: under 1000 roundings of
    2^-24 of the sums' largest magnitudes, which stay below 16 times the
    result's largest here (the sums' terms add up like squares do)."""
    print("beam search", order, flush=True)
    m = Model()
    B, W, eos, steps = 2, 3, 7, 9
    prompts = [torch.randint(0, m.V, (n,), device=DEV, generator=gen(61 + n)) for n in (13, 5)]
    conv, state, deep = m.pools(B * W)
    cu = [0] + np.cumsum([len(p) for p in prompts for _ in range(W)]).tolist()
    logits = m.prompt(torch.cat([p for p in prompts for _ in range(W)]), cu, conv, state)
    logits = logits[torch.tensor(cu[1:], device=DEV) - 1]
    for b, p in enumerate(prompts):
        for t in p:
            m.kda_step(t.expand(W), deep[b * W:(b + 1) * W])
    scores = torch.full((B, W), -float("inf"), device=DEV)
    scores[:, 0] = 0.0  # the beams of a prompt are one at first
    done = torch.zeros(B, W, dtype=torch.bool, device=DEV)
    seqs = [[[] for _ in range(W)] for _ in range(B)]
    for i in range(steps):
        if i == 3:  # (a beam ends on its way)
            logits.view(B, W, m.V)[:, 0, eos] += 6.0
            bumped = [seqs[b][0] for b in range(B)]
        before = (logits.clone(), scores.clone(), done.clone())
        scores, parents, tokens, done = kda.beam_select(logits.view(B, W, m.V), scores, finished=done, eos=eos,
                                                        order=order)
        want = ref.beam_select(before[0].cpu().view(B, W, m.V), before[1].cpu(), W, before[2].cpu(), eos, order)
        assert torch.equal(parents.cpu(), want[1]) and torch.equal(tokens.cpu(), want[2])
        assert torch.equal(done.cpu(), want[3])
        kda.state_reorder([conv, state, deep], parents)
        chosen, par = tokens.cpu(), parents.cpu()
        seqs = [[seqs[b][par[b, w]] + [int(chosen[b, w])] for w in range(W)] for b in range(B)]
        flat = tokens.view(-1).long()
        logits = m.step(flat, conv, state)
        m.kda_step(flat, deep)
    assert done.any() and not done.all()

    # each chosen sequence alone
    full = [torch.cat([prompts[b], torch.tensor(seqs[b][w], device=DEV)]) for b in range(B) for w in range(W)]
    cu = [0] + np.cumsum([len(t) for t in full]).tolist()
    c1, s1, d1 = m.pools(B * W)
    lg = m.prompt(torch.cat(full), cu, c1, s1)
    for r, t in enumerate(full):
        for tok in t:
            m.kda_step(tok.view(1), d1[r:r + 1])
    torch.cuda.synchronize()
    assert torch.equal(deep, d1)  # (the same call row by row: bit for bit)
    rel = 16 * 1000 * U
    assert (conv - c1).abs().max() <= rel * c1.abs().max()
    assert (state - s1).abs().max() <= rel * s1.abs().max()
    last = lg[torch.tensor(cu[1:], device=DEV) - 1]
    assert (logits - last).abs().max() <= rel * last.abs().max()
    for b in range(B):
        for w in range(W):
            row = lg[cu[b * W + w]:cu[b * W + w + 1]].double().cpu()
            total, n = 0.0, len(prompts[b])
            for i, tok in enumerate(seqs[b][w]):
                x = row[n - 1 + i].clone()
                if i == 3 and seqs[b][w][:3] == bumped[b]:
                    x[eos] += 6.0
                total += float(x[tok] - torch.logsumexp(x, 0))
                if tok == eos:
                    break
            assert abs(float(scores[b, w]) - total) <= steps * 2 * rel * float(row.abs().max())


# ---- calls at the edge of what is documented ----------------------------------------------

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("split", [1, 4])
def test_states_in_place_and_in_pools(split, dtype):
    """final_state in initial_state's place, in slots of a pool, some of them
    out of range: the same as with buffers of their own, and no other slice
    changes.  Cut or not."""
    print("in place", split, dtype, flush=True)
    cu, H, dk, dv = [0, 500, 500, 577, 900], 3, 64, 40
    g = gen(90)
    q, k, v = f(g, 900, H, dk).to(dtype), (f(g, 900, H, dk) * dk ** -0.5).to(dtype), f(g, 900, H, dv).to(dtype)
    gl = -torch.rand(900, H, device=DEV, generator=g) * 0.05
    pool = f(g, 6, H, dk, dv)
    slots = torch.tensor([4, 1, 9, 0], dtype=torch.int32, device=DEV)
    init = pool[[4, 1, 0, 0]].clone()
    init[2] = 0  # (a slot out of range: from nothing)
    o, fin = kda.decay_attention(q, k, v, gl, cu_seqlens=cu, initial_state=init, split_hint=split)
    before = pool.clone()
    o2, _ = kda.decay_attention(q, k, v, gl, cu_seqlens=cu, initial_state=pool, final_state=pool, slots=slots,
                                split_hint=split)
    torch.cuda.synchronize()
    assert torch.equal(o, o2)
    for s, n in ((4, 0), (1, 1), (0, 3)):
        assert torch.equal(pool[s], fin[n])
    assert torch.equal(pool[[2, 3, 5]], before[[2, 3, 5]])


def test_logits_below_the_normal_numbers_keep_their_order():
    """Within a beam the logits' own order decides, where 64-bit values are
    equal too."""
    print("denormal logits", flush=True)
    for dtype, unit in ((F32, 2.0 ** -149), (BF16, 2.0 ** -133)):
        x = torch.full((1, 1, 9000), -1.0, dtype=dtype)
        at = torch.tensor([8999, 17, 4096, 5000, 0])
        x[0, 0, at] = (torch.tensor([5.0, 4.0, 3.0, 0.0, -1.0], dtype=torch.float64) * unit).to(dtype)
        x[0, 0, 40] = -0.0  # (as 0: the lower token goes first)
        _, _, tokens, _ = kda.beam_select(x.to(DEV), torch.zeros(1, 1, device=DEV), beams=6)
        assert tokens[0].tolist() == [8999, 17, 4096, 40, 5000, 0]


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_masks_of_the_lowest_value(dtype):
    """A few tokens allowed, the others at the type's lowest value, over many
    parts: these tie, and the first of them follow the allowed ones."""
    print("lowest masks", dtype, flush=True)
    V = 40000
    x = torch.full((2, 3, V), torch.finfo(dtype).min, dtype=dtype)
    g = torch.Generator().manual_seed(91)
    for b in range(2):
        for w in range(3):
            x[b, w, torch.randperm(V, generator=g)[:2 + w]] = torch.randn(2 + w, generator=g).to(dtype)
    scores = torch.tensor([[0.0, -1.0, -2.0], [-3.0, -0.5, 0.0]])
    for K in (3, 8, 64):
        got = kda.beam_select(x.to(DEV), scores.to(DEV), beams=K)
        want = ref.beam_select(x, scores, K)
        assert torch.equal(got[1].cpu(), want[1]) and torch.equal(got[2].cpu(), want[2])


def test_the_same_parent_for_every_row_and_every_kind_of_state():
    """One parent for all rows, states of every type and of a byte a slice,
    beams of every count the reordering has its own way for."""
    print("one parent", flush=True)
    for K in (1, 2, 4, 5, 8, 9, 16, 17, 32, 33, 64):
        g = gen(92 + K)
        states = [f(g, 2 * K, 3, 7), f(g, 2 * K, 130).to(BF16), torch.randint(-9, 9, (2 * K, 1), device=DEV, generator=g).to(torch.int8),
                  f(g, 2 * K, 33).to(torch.float8_e4m3fn).view(torch.int8), torch.zeros(2 * K, 0, device=DEV)]
        parents = torch.randint(0, K, (2, 1), device=DEV, generator=g, dtype=torch.int32).expand(2, K).contiguous()
        want = [ref.reorder(s.cpu(), parents.cpu()) for s in states]
        kda.state_reorder(states, parents)
        torch.cuda.synchronize()
        for s, w in zip(states, want):
            assert torch.equal(s.cpu(), w)


def test_empty_and_single_rows_of_a_batch():
    """Sequences without tokens only, a step of one row, a norm of one column."""
    print("smallest", flush=True)
    state = f(gen(95), 3, 2, 8, 8)
    e = torch.empty(0, 2, 8, device=DEV)
    o, fin = kda.decay_attention(e, e, e, torch.empty(0, 2, device=DEV), cu_seqlens=[0, 0, 0, 0], initial_state=state)
    assert o.shape == (0, 2, 8) and torch.equal(fin, state)
    x = torch.tensor([[3.0], [-2.0], [0.0]], device=DEV)
    r, y = kda.block_norm(x, torch.ones(1, device=DEV), eps=0.0, residual=torch.zeros_like(x))
    assert r.view(-1).tolist() == [3.0, -2.0, 0.0] and y[:2].view(-1).tolist() == [1.0, -1.0] and torch.isnan(y[2, 0])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lengths,split", [([150, 70], 1), ([150, 70], 2), ([60] * 90, 1)])
def test_a_decay_of_nan_spoils_what_follows_it_only(lengths, split, dtype):
    """Prompts and single tokens: the outputs before it, other heads and other
    sequences stay what they are."""
    print("nan decay", len(lengths), split, dtype, flush=True)
    cu = [0] + np.cumsum(lengths).tolist()
    T, H, d, at = cu[-1], 4, 64, 37
    g = gen(97)
    q, k, v = f(g, T, H, d).to(dtype), (f(g, T, H, d) * d ** -0.5).to(dtype), f(g, T, H, d).to(dtype)
    gl = -torch.rand(T, H, device=DEV, generator=g) * 0.1
    clean, cfin = kda.decay_attention(q, k, v, gl, cu_seqlens=cu, split_hint=split)
    bad = gl.clone()
    bad[at, 0] = float("nan")
    o, fin = kda.decay_attention(q, k, v, bad, cu_seqlens=cu, split_hint=split)
    end = cu[1]
    torch.cuda.synchronize()
    assert torch.equal(o[:at], clean[:at]) and torch.equal(o[:, 1:], clean[:, 1:]) and torch.equal(o[end:], clean[end:])
    assert torch.isnan(o[at:end, 0].float()).all()
    assert torch.isnan(fin[0, 0]).all()
    assert torch.equal(fin[0, 1:], cfin[0, 1:]) and torch.equal(fin[1:], cfin[1:])

    state = f(g, 3, H, d, d)
    want = state.clone()
    rows = slice(at - 1, at + 2)
    wo = kda.decay_attention_step(want, q[rows], k[rows], v[rows], gl[rows])
    so = kda.decay_attention_step(state, q[rows], k[rows], v[rows], bad[rows])
    torch.cuda.synchronize()
    assert torch.isnan(so[1, 0].float()).all() and torch.isnan(state[1, 0]).all()
    so[1, 0], state[1, 0] = wo[1, 0], want[1, 0]
    assert torch.equal(so, wo) and torch.equal(state, want)
