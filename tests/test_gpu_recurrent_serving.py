"""The calls around the recurrence as a server uses them together: prompt,
states parked in the 8-bit cache and read back, then token by token; in
graphs, and on streams of their own."""
import numpy as np
import pytest
import torch

import gated_delta_rule_19_amd as kda
import oracle
import recurrent_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def f(g, *shape):
    return torch.randn(shape, device=DEV, generator=g)


class Mixer:
    """A selective-scan layer's recurrent part: convolution, then scan.  The
    projections in front are random columns of one matrix."""

    def __init__(self, D, N, G, W, dtype, seed):
        g = gen(seed)
        self.D, self.N, self.G, self.W, self.dt = D, N, G, W, dtype
        self.w = f(g, D, W).mul_(0.5).to(dtype)
        self.b = f(g, D).mul_(0.1).to(dtype)
        self.A = -torch.arange(1.0, N + 1, device=DEV) * torch.exp(0.1 * f(g, D, N))
        self.skip = f(g, D)
        self.bias = f(g, D) - 3
        self.width = 3 * D + 2 * G * N

    def parts(self, p):
        D, n = self.D, self.G * self.N
        at = [0, D, 2 * D, 3 * D, 3 * D + n, 3 * D + 2 * n]
        x, z, dl, B, C = (p[:, a:b] for a, b in zip(at[:-1], at[1:]))
        return x, z, dl, B.view(-1, self.G, self.N), C.view(-1, self.G, self.N)

    def prompt(self, p, cu, conv, ssm, slots):
        x, z, dl, B, C = self.parts(p)
        xc, _ = kda.short_conv(x, self.w, self.b, cu_seqlens=cu, initial_state=conv,
                               final_state=conv, slots=slots)
        y, _ = kda.selective_scan(xc, dl, self.A, B, C, D=self.skip, z=z, delta_bias=self.bias,
                                  cu_seqlens=cu, initial_state=ssm, final_state=ssm, slots=slots)
        return y

    def step(self, p, conv, ssm, slots, y=None):
        x, z, dl, B, C = self.parts(p)
        xc = kda.short_conv_step(conv, x, self.w, self.b, slots=slots)
        return kda.selective_scan_step(ssm, xc, dl, self.A, B, C, D=self.skip, z=z,
                                       delta_bias=self.bias, slots=slots, y=y)

    def plain(self, p, cu, conv, ssm):
        """The same in 64 bits (x rounded to its type between the two, as
        the calls do), with the scan's own error bound."""
        x, z, dl, B, C = (ref.f64(t) for t in self.parts(p))
        y, tol, fin = ref.conv(x, ref.f64(self.w), ref.f64(self.b), cu, conv, True, self.dt)
        return y, tol, fin, (z, dl, B, C)


def test_prompt_cache_and_steps_together():
    """fp32 end to end: prompts of uneven length into pools, the states parked
    in int8 and read back into other slots, then 6 tokens each.  Every stage
    is held to the 64-bit form of its own inputs."""
    print("serving run", flush=True)
    m = Mixer(96, 16, 2, 4, F32, 1)
    lengths = [65, 1, 0, 130]
    cu = np.concatenate([[0], np.cumsum(lengths)])
    slots = torch.tensor([3, 0, 5, 1], dtype=torch.int32, device=DEV)
    conv = torch.zeros((6, 3, 96), device=DEV)
    ssm = torch.zeros((6, 96, 16), device=DEV)
    p = f(gen(2), int(cu[-1]), m.width)
    y = m.prompt(p, cu, conv, ssm, slots)
    torch.cuda.synchronize()

    x, z, dl, B, C = m.parts(p)
    xc, _ = kda.short_conv(x, m.w, m.b, cu_seqlens=cu)
    cy, ctol, cfin = ref.conv(ref.f64(x), ref.f64(m.w), ref.f64(m.b), cu, None, True, F32)
    ref.check("conv", xc, cy, ctol)
    assert np.array_equal(ref.f64(conv[slots.long()]), cfin)
    sy, ytol, sfin, ftol = ref.scan(ref.f64(xc), ref.f64(dl), ref.f64(m.A), ref.f64(B), ref.f64(C),
                                    ref.f64(m.skip), ref.f64(z), ref.f64(m.bias), True, cu, None, F32, 2.0)
    ref.check("scan", y, sy, ytol)
    ref.check("scan state", ssm[slots.long()], sfin, ftol)

    # park, clear, and read back into other slots
    codes = torch.zeros((9, 96, 16), dtype=torch.int8, device=DEV)
    scales = torch.zeros((9, 96), device=DEV)
    cache = torch.tensor([8, 2, 4, 0], dtype=torch.int32, device=DEV)
    kda.state_store(ssm, codes, scales, src=slots, dst=cache)
    want_c, want_s = ref.quantise(ssm[slots.long()].cpu(), torch.int8)
    ssm.zero_()
    back = torch.tensor([1, 2, 3, 4], dtype=torch.int32, device=DEV)
    kda.state_load(codes, scales, ssm, src=cache, dst=back)
    conv[back.long()] = conv[slots.long()]
    torch.cuda.synchronize()
    assert torch.equal(ssm[back.long()].cpu(), want_c.float() * want_s[..., None])

    for i in range(6):
        p1 = f(gen(10 + i), 4, m.width)
        x, z, dl, B, C = m.parts(p1)
        c0, s0 = ref.f64(conv[back.long()]), ref.f64(ssm[back.long()])
        xr, xt, c1 = ref.conv_step(ref.f64(x), c0, ref.f64(m.w), ref.f64(m.b), True, F32)
        y = m.step(p1, conv, ssm, back)
        torch.cuda.synchronize()
        assert np.array_equal(ref.f64(conv[back.long()]), c1)
        # the scan from the convolution's outputs as the kernel rounds them
        tmp = torch.tensor(c0, dtype=F32, device=DEV)
        xc = kda.short_conv_step(tmp, x, m.w, m.b)
        ref.check("step conv", xc, xr, xt)
        sy, ytol, s1, ftol = ref.scan(ref.f64(xc), ref.f64(dl), ref.f64(m.A), ref.f64(B), ref.f64(C),
                                      ref.f64(m.skip), ref.f64(z), ref.f64(m.bias), True, [0, 1, 2, 3, 4],
                                      s0, F32)
        ref.check("step scan", y, sy, ytol)
        ref.check("step state", ssm[back.long()], s1, ftol)


@pytest.mark.parametrize("kind,step", [(torch.int8, 0.5 / 127), (torch.float8_e4m3fn, 2.0 ** -4)])
def test_kda_layer_with_convolutions_and_parked_states(kind, step):
    """q, k and v through their convolutions into the gated prefill; its
    checkpoint states parked in the cache; a decode step from what is read
    back, against the oracle from the very same state."""
    print("kda layer run", kind, flush=True)
    H, W, T = 3, 4, 150
    D = H * 128
    g = gen(30)
    qkv = f(g, T, 3 * D).to(BF16)
    w = [f(g, D, W).mul_(0.5).to(BF16) for _ in range(3)]
    A_log, zg = f(g, H) * 0.3, f(g, T, H, 128).to(BF16)
    beta = torch.sigmoid(f(g, T, H)).to(BF16)
    cu = [0, 130, 150]
    outs, convs = [], []
    for i in range(3):
        o, s = kda.short_conv(qkv[:, i * D:(i + 1) * D], w[i], cu_seqlens=cu)
        outs.append(o.view(T, H, 128))
        convs.append(s)
    kw = dict(A_log=A_log, qk_norm_eps=1e-6)
    o, fin, ck, pos = None, None, None, None
    o, fin = kda.chunk_prefill_gated(*outs, zg, beta, cu_seqlens=cu, **kw)
    torch.cuda.synchronize()
    assert torch.isfinite(o.float()).all()

    codes = torch.zeros((5, H, 128, 128), dtype=torch.int8, device=DEV).view(kind)
    scales = torch.zeros((5, H, 128), device=DEV)
    at = torch.tensor([4, 1], dtype=torch.int32, device=DEV)
    kda.state_store(fin, codes, scales, dst=at)
    state = kda.state_load(codes, scales, torch.empty_like(fin), src=at)
    torch.cuda.synchronize()
    # half a code step of the row's largest value (e4m3: of the value, or of
    # the smallest normal's step)
    amax = fin.abs().amax(-1, keepdim=True)
    tol = amax * step if kind == torch.int8 else torch.maximum(fin.abs() * step, amax / 448 * 2.0 ** -10)
    assert ((state - fin).abs() <= tol * (1 + 2.0 ** -20)).all()

    x1 = f(g, 2, 3 * D).to(BF16)
    q, k, v = (kda.short_conv_step(convs[i], x1[:, i * D:(i + 1) * D], w[i]).view(2, H, 128)
               for i in range(3))
    z1, b1 = f(g, 2, H, 128).to(BF16), torch.sigmoid(f(g, 2, H)).to(BF16)
    before = state.clone()
    o1 = kda.decode_step_gated(state, q, k, v, z1, b1, **kw)
    torch.cuda.synchronize()
    ql, kl = (oracle.l2_normalize(t, 1e-6) for t in (q, k))
    gl = oracle.gate_log_decay(z1, A_log, -5.0)
    o_ref, s_ref = oracle.decode_step(before.cpu().double().numpy(), ql, kl, v, gl, b1)
    err = np.max(np.abs(ref.f64(o1) - o_ref)) / np.max(np.abs(o_ref))
    assert err <= 1e-2
    assert np.max(np.abs(ref.f64(state) - s_ref)) <= 1e-4 * np.max(np.abs(s_ref))


@pytest.mark.parametrize("nseq", [3, 64, 200])
def test_captured_prompts_replay_equal_eager(nseq):
    """Prompt calls in a graph, inline and workspace tables, cut sequences:
    each replay on new inputs equals the eager call, with eager calls of other
    shapes between the replays."""
    print("captured prompts", nseq, flush=True)
    m = Mixer(70, 16, 1, 4, BF16, 40)
    lengths = [(i * 37) % 150 for i in range(nseq)]
    cu = np.concatenate([[0], np.cumsum(lengths)])
    T = int(cu[-1])
    p = torch.zeros((T, m.width), dtype=BF16, device=DEV)
    conv = torch.zeros((nseq, 3, 70), dtype=BF16, device=DEV)
    ssm = torch.zeros((nseq, 70, 16), device=DEV)
    codes = torch.zeros((nseq, 70, 16), dtype=torch.int8, device=DEV)
    scales = torch.zeros((nseq, 70), device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = m.prompt(p, cu, conv, ssm, None)
        kda.state_store(ssm, codes, scales)
    for rep in range(4):
        g = gen(50 + rep)
        p.copy_(f(g, T, m.width))
        c0, s0 = f(g, nseq, 3, 70).to(BF16), f(g, nseq, 70, 16)
        conv.copy_(c0)
        ssm.copy_(s0)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, conv, ssm, codes, scales)]
        other = m.prompt(p[:37], [0, 30, 37], c0[:2].clone(), s0[:2].clone(), None)
        assert torch.isfinite(other.float()).all()
        want_y = m.prompt(p, cu, c0, s0, None)
        wc, ws = torch.zeros_like(codes), torch.zeros_like(scales)
        kda.state_store(s0, wc, ws)
        torch.cuda.synchronize()
        for a, b in zip(got, (want_y, c0, s0, wc, ws)):
            assert torch.equal(a, b)


def test_captured_steps_replay_equal_eager():
    print("captured steps", flush=True)
    m = Mixer(130, 13, 1, 3, F32, 60)
    p = torch.zeros((5, m.width), device=DEV)
    slots = torch.tensor([4, 0, -1, 2, 7], dtype=torch.int32, device=DEV)
    conv, ssm = f(gen(61), 6, 2, 130), f(gen(62), 6, 130, 13)
    c0, s0 = conv.clone(), ssm.clone()
    y = torch.zeros((5, 130), device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.step(p, conv, ssm, slots, y=y)
    for rep in range(5):
        p.copy_(f(gen(70 + rep), 5, m.width))
        slots.copy_(torch.tensor([[4, 0, -1, 2, 7], [1, 2, 3, 4, 5]][rep % 2], dtype=torch.int32))
        graph.replay()
        want = torch.zeros_like(y)
        if rep:
            want.copy_(last)
        m.step(p, c0, s0, slots, y=want)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(conv, c0) and torch.equal(ssm, s0)
        last = want


def test_two_streams_at_once():
    """The same calls on two streams with different inputs, in flight
    together, equal the calls run alone."""
    print("two streams", flush=True)
    m = Mixer(256, 16, 1, 4, BF16, 80)
    cu = np.concatenate([[0], np.cumsum([700] * 2 + [9] * 70)])
    T = int(cu[-1])
    n = len(cu) - 1
    ps = [f(gen(81 + i), T, m.width).to(BF16) for i in range(2)]

    def go(p):
        conv = torch.zeros((n, 3, 256), dtype=BF16, device=DEV)
        ssm = torch.zeros((n, 256, 16), device=DEV)
        y = m.prompt(p, cu, conv, ssm, None)
        codes = torch.zeros((n, 256, 16), dtype=torch.int8, device=DEV)
        scales = torch.zeros((n, 256), device=DEV)
        kda.state_store(ssm, codes, scales)
        return y, conv, ssm, codes, scales

    alone = [go(p) for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    both = []
    for _ in range(3):
        for s, p in zip(streams, ps):
            with torch.cuda.stream(s):
                both.append(go(p))
    torch.cuda.synchronize()
    for i, got in enumerate(both):
        for a, b in zip(got, alone[i % 2]):
            assert torch.equal(a, b)


def test_arrays_side_by_side_in_one_buffer():
    """States, outputs and parameters that touch without overlapping are
    accepted, and each call writes its own only."""
    print("side by side", flush=True)
    D, N, W, rows = 64, 16, 4, 5
    m = Mixer(D, N, 1, W, F32, 120)
    p = f(gen(121), rows, m.width)
    x, z, dl, B, C = m.parts(p)
    sizes = dict(conv=rows * 3 * D, xc=rows * D, ssm=rows * D * N, y=rows * D, A=D * N, skip=D,
                 bias=D, w=D * W, b=D, back=rows * D * N, scales=rows * D, codes=rows * D * N // 4)
    arena = torch.full((sum(sizes.values()),), 7.0, device=DEV)
    v, at = {}, 0
    for k, n in sizes.items():
        v[k] = arena[at:at + n]
        at += n
    shape = dict(conv=(rows, 3, D), xc=(rows, D), ssm=(rows, D, N), y=(rows, D), A=(D, N), w=(D, W),
                 back=(rows, D, N), scales=(rows, D))
    v = {k: t.view(shape[k]) if k in shape else t for k, t in v.items()}
    codes = v["codes"].view(torch.int8).view(rows, D, N)
    for k, t in (("A", m.A), ("skip", m.skip), ("bias", m.bias), ("w", m.w), ("b", m.b)):
        v[k].copy_(t)
    c0, s0 = f(gen(122), rows, 3, D), f(gen(123), rows, D, N)
    v["conv"].copy_(c0)
    v["ssm"].copy_(s0)
    want = m.step(p, c0, s0, None)
    kda.short_conv_step(v["conv"], x, v["w"], v["b"], y=v["xc"])
    y = kda.selective_scan_step(v["ssm"], v["xc"], dl, v["A"], B, C, D=v["skip"], z=z,
                                delta_bias=v["bias"], y=v["y"])
    kda.state_store(v["ssm"], codes, v["scales"])
    kda.state_load(codes, v["scales"], v["back"])
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(v["conv"], c0) and torch.equal(v["ssm"], s0)
    assert torch.equal(v["A"], m.A) and torch.equal(v["bias"], m.bias) and torch.equal(v["w"], m.w)
    qc, qs = ref.quantise(s0.cpu(), torch.int8)
    assert torch.equal(codes.cpu(), qc) and torch.equal(v["scales"].cpu(), qs)
    assert torch.equal(v["back"].cpu(), qc.float() * qs[..., None])
    kda.short_conv(x, v["w"], v["b"], initial_state=v["conv"][:1], final_state=v["conv"][:1], y=v["xc"])
    kda.selective_scan(v["xc"], dl, v["A"], B, C, D=v["skip"], delta_bias=v["bias"],
                       initial_state=v["ssm"][:1], final_state=v["ssm"][:1], y=v["y"])
    torch.cuda.synchronize()
    assert torch.equal(v["conv"][1:], c0[1:]) and torch.equal(v["ssm"][1:], s0[1:])
    assert torch.equal(v["A"], m.A) and torch.equal(v["bias"], m.bias) and torch.equal(v["w"], m.w)
