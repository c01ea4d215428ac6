"""Operators around a decoder block with recurrent mixers: what is timed, and
their plain forms.

Five calls that follow each other when such a model answers with beams:

- ``block_norm``: the norm after a block, its gate and scaled residual, and
  the norm in front of the next block;
- ``decay_attention`` / ``decay_attention_step``: linear attention with one
  decay a head, for packed prompts and for single tokens;
- ``beam_select``: the best continuations over beams and vocabulary;
- ``state_reorder``: the recurrent states that follow the chosen beams.

``own`` chooses between the plain form (elementary torch operations, 32-bit;
64-bit where candidates are ordered) and the library's calls.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EOS = 2


# ---------------------------------------------------------------- cases

def listed():
    return [
        # The benchmark's prefill shape: one long prompt, 96 heads.
        {"name": "attn_8192x96x128_bf16", "op": "attn", "seqs": 1, "tokens": 8192, "H": 96,
         "Hq": 96, "Hk": 96, "Hv": 96, "dk": 128, "dv": 128, "type": "bf16", "state": False},
        # The benchmark's long context on few heads: the sequence has to be cut.
        {"name": "attn_131072x12x128_bf16", "op": "attn", "seqs": 1, "tokens": 131072, "H": 12,
         "Hq": 12, "Hk": 12, "Hv": 12, "dk": 128, "dv": 128, "type": "bf16", "state": False},
        # Packed resumed prompts, fp32, shared key and value heads, sizes that divide nothing.
        {"name": "attn_37seqs_9001x10x100_f32", "op": "attn", "seqs": 37, "tokens": 9001, "H": 10,
         "Hq": 10, "Hk": 5, "Hv": 5, "dk": 100, "dv": 72, "type": "f32", "state": True},
        # The benchmark's decode batch.
        {"name": "step_256x96x128_bf16", "op": "step", "rows": 256, "H": 96, "Hq": 96, "Hk": 96,
         "Hv": 96, "dk": 128, "dv": 128, "type": "bf16", "slots": 256},
        # A few users decoding, shared heads, odd sizes: latency.
        {"name": "step_3x10x100_f32", "op": "step", "rows": 3, "H": 10, "Hq": 10, "Hk": 5,
         "Hv": 5, "dk": 100, "dv": 72, "type": "f32", "slots": 7},
        # One user with four beams: latency.
        {"name": "beam_1x4x32000_f32", "op": "beam", "batch": 1, "W": 4, "K": 4, "V": 32000,
         "type": "f32", "finished": False, "order": "score"},
        # A batch of users with eight beams each over a large vocabulary of odd
        # size, some beams finished.
        {"name": "beam_64x8x128001_bf16", "op": "beam", "batch": 64, "W": 8, "K": 8, "V": 128001,
         "type": "bf16", "finished": True, "order": "rows"},
        # The 96-head states of 32 users with four beams, of which two survive.
        {"name": "reorder_32x4x96x128x128_f32", "op": "reorder", "batch": 32, "K": 4, "live": 2,
         "R": 12288, "L": 128, "type": "f32", "slots": 128, "order": "rows"},
        # Convolution states of a few users, an odd number of channels.
        {"name": "reorder_3x5x3x1001_bf16", "op": "reorder", "batch": 3, "K": 5, "live": 2,
         "R": 3, "L": 1001, "type": "bf16", "slots": 20, "order": "score"},
        # A decode step of one user between two blocks: latency.
        {"name": "norm_1x12288_bf16", "op": "norm", "rows": 1, "D": 12288, "type": "bf16",
         "post": True, "gate": False, "stream": "bf16", "pre": True},
        # A full prompt between two blocks, 96 heads of 128.
        {"name": "norm_8192x12288_bf16", "op": "norm", "rows": 8192, "D": 12288, "type": "bf16",
         "post": True, "gate": True, "stream": "bf16", "pre": True},
        # fp32, an odd width, a residual stream without a norm after the block.
        {"name": "norm_20000x1002_f32", "op": "norm", "rows": 20000, "D": 1002, "type": "f32",
         "post": False, "gate": True, "stream": "f32", "pre": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng, most):
    """Heads of the decay, q, k and v: all alike, shared k and v, or shared q and k."""
    share = rng.choice([1, 1, 2, 4])
    few = _log_int(rng, 1, max(1, most // share))
    H = few * share
    return rng.choice([(H, H, few, few), (H, few, few, H)])


def draw(rng):
    op = rng.choice(["attn", "attn", "step", "beam", "beam", "reorder", "norm"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    size = [16, 37, 64, 64, 96, 100, 128, 128, 128, 256]
    if op == "attn":
        H, Hq, Hk, Hv = _heads(rng, 96)
        dk, dv = rng.choice(size), rng.choice(size)
        most = 600000000 if kind == "f32" else 12000000000
        tokens = min(_log_int(rng, 16, 131072), most // (H * dk * dv))
        return {"op": op, "seqs": min(tokens, _log_int(rng, 1, 60)), "tokens": tokens, "H": H,
                "Hq": Hq, "Hk": Hk, "Hv": Hv, "dk": dk, "dv": dv, "type": kind,
                "state": rng.random() < 0.5}
    if op == "step":
        H, Hq, Hk, Hv = _heads(rng, 96)
        rows = _log_int(rng, 1, 256)
        return {"op": op, "rows": rows, "H": H, "Hq": Hq, "Hk": Hk, "Hv": Hv,
                "dk": rng.choice(size), "dv": rng.choice(size), "type": kind,
                "slots": rows + rng.randint(0, 20)}
    if op == "beam":
        W, batch = _log_int(rng, 1, 16), _log_int(rng, 1, 64)
        K = rng.choice([W, W, 2 * W])
        return {"op": op, "batch": batch, "W": W, "K": K,
                "V": max(100, min(_log_int(rng, 1000, 200000), 60000000 // (W * batch))),
                "type": kind, "finished": rng.random() < 0.5,
                "order": rng.choice(["score", "rows"])}
    if op == "reorder":
        K, batch = _log_int(rng, 2, 16), _log_int(rng, 1, 32)
        L = rng.choice([128, 128, 16, 64, 13])
        return {"op": op, "batch": batch, "K": K, "live": rng.randint(1, K - 1),
                "R": max(1, min(_log_int(rng, 3, 12288), 190000000 // (L * K * batch))), "L": L,
                "type": kind, "slots": batch * K + rng.randint(0, 20),
                "order": rng.choice(["score", "rows"])}
    D = _log_int(rng, 64, 16384)
    rows = _log_int(rng, 1, min(100000, 100000000 // D))
    return {"op": op, "rows": rows, "D": D, "type": kind, "post": rng.random() < 0.5,
            "gate": rng.random() < 0.5, "stream": rng.choice(["f32", kind]),
            "pre": rng.random() < 0.8}


# ---------------------------------------------------------------- inputs

def _lengths(tokens, seqs, seed):
    """`seqs` lengths that sum to `tokens`, uneven, some of them possibly 0."""
    if seqs == 1:
        return [tokens]
    r = np.random.default_rng(seed + 17)
    cuts = np.sort(r.integers(0, tokens + 1, size=seqs - 1))
    return np.diff(np.concatenate([[0], cuts, [tokens]])).tolist()


def _slots(rows, pool, seed):
    """`rows` different slots of a pool, in no order."""
    r = np.random.default_rng(seed + 29)
    return torch.tensor(r.permutation(pool)[:rows].astype(np.int32), device=DEV)


def _parents(case, seed):
    """Which row of its group each row continues: `live` rows have all
    children; ordered by rows each of them keeps its own."""
    r = np.random.default_rng(seed + 41)
    out = np.zeros((case["batch"], case["K"]), np.int32)
    for b in range(case["batch"]):
        perm = r.permutation(case["K"])
        live = perm[:case["live"]]
        rest = np.resize(r.permutation(live), case["K"] - case["live"])
        if case["order"] == "rows":
            out[b, live] = live
            out[b, perm[case["live"]:]] = rest
        else:
            out[b] = r.permutation(np.concatenate([live, rest]))
    return torch.tensor(out, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    f = dict(device=DEV, generator=g)
    op = case["op"]
    dt = TYPES[case["type"]]
    s = {"case": case}
    if op in ("attn", "step"):
        H, dk, dv = case["H"], case["dk"], case["dv"]
        rows = case["tokens"] if op == "attn" else case["rows"]
        # keys of about unit length, as after their norm
        s["q"] = torch.randn((rows, case["Hq"], dk), **f).mul_(dk ** -0.5).to(dt)
        s["k"] = torch.randn((rows, case["Hk"], dk), **f).mul_(dk ** -0.5).to(dt)
        s["v"] = torch.randn((rows, case["Hv"], dv), **f).to(dt)
        # memories of about 3 to 2000 tokens, varying from token to token
        head = torch.exp(-torch.rand((H,), **f) * math.log(700.0)) * 0.35
        s["g"] = -head * torch.exp(0.5 * torch.randn((rows, H), **f))
        if op == "step":
            s["slots"] = _slots(rows, case["slots"], seed)
            s["state"] = torch.randn((case["slots"], H, dk, dv), **f)
        else:
            s["cu"] = np.concatenate(
                [[0], np.cumsum(_lengths(rows, case["seqs"], seed))]).astype(np.int64)
            if case["state"]:
                s["state"] = torch.randn((case["seqs"], H, dk, dv), **f)
        return s
    if op == "beam":
        B, W, V = case["batch"], case["W"], case["V"]
        s["logits"] = torch.randn((B, W, V), **f).mul_(2.5).to(dt)
        # banned tokens
        banned = torch.randint(0, V, (V // 50 + 1,), **f)
        s["logits"][:, :, banned] = -math.inf
        s["scores"] = -20.0 + 2.0 * torch.randn((B, W), **f)
        s["finished"] = torch.rand((B, W), **f) < 0.15 if case["finished"] else None
        return s
    if op == "reorder":
        s["parents"] = _parents(case, seed)
        s["slots"] = _slots(case["batch"] * case["K"], case["slots"], seed).view(case["batch"], -1)
        s["state"] = torch.randn((case["slots"], case["R"], case["L"]), **f).to(dt)
        return s
    rows, D = case["rows"], case["D"]
    s["x"] = torch.randn((rows, D), **f).to(dt)
    s["gate"] = torch.randn((rows, D), **f).to(dt) if case["gate"] else None
    s["residual"] = (3.0 * torch.randn((rows, D), **f)).to(TYPES[case["stream"]])
    s["scale"] = 0.2 + 0.1 * torch.randn((D,), **f)
    s["post"] = 1.0 + 0.1 * torch.randn((D,), **f) if case["post"] else None
    s["pre"] = 1.0 + 0.1 * torch.randn((D,), **f) if case["pre"] else None
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return OWN[op](s)
    return PLAIN[op](s)


def _kda():
    import gated_delta_rule_19_amd as kda
    return kda


def _own_attn(s):
    o, final = _kda().decay_attention(s["q"], s["k"], s["v"], s["g"], cu_seqlens=s["cu"],
                                      initial_state=s.get("state"))
    return {"o": o, "final": final}


def _own_step(s):
    o = _kda().decay_attention_step(s["state"], s["q"], s["k"], s["v"], s["g"], slots=s["slots"])
    return {"o": o, "state": s["state"]}


def _own_beam(s):
    c = s["case"]
    scores, parents, tokens, finished = _kda().beam_select(
        s["logits"], s["scores"], beams=c["K"], finished=s["finished"], eos=EOS, order=c["order"])
    return {"scores": scores, "parents": parents, "tokens": tokens, "finished": finished}


def _own_reorder(s):
    _kda().state_reorder(s["state"], s["parents"], slots=s["slots"])
    return {"state": s["state"]}


def _own_norm(s):
    r, y = _kda().block_norm(s["x"], post_weight=s["post"], gate=s["gate"], residual=s["residual"],
                             scale=s["scale"], weight=s["pre"])
    return {"residual": r, "y": y} if y is not None else {"residual": r}


# ---------------------------------------------------------------- plain forms

def _wide(x, H):
    """[rows, few, d] to one row of d for each of H heads, 32-bit."""
    return x.float().repeat_interleave(H // x.shape[1], dim=1)


def _plain_attn(s):
    """Chunks of 64 tokens: scores within a chunk, states between chunks, and
    a doubling of runs of chunks for the states that enter them."""
    C = 64
    H, dk, dv = s["case"]["H"], s["case"]["dk"], s["case"]["dv"]
    cu = s["cu"]
    lens = np.diff(cu)
    per = (lens + C - 1) // C
    first = np.cumsum(per) - per             # each sequence's first chunk
    n = int(per.sum())
    seq = np.repeat(np.arange(len(lens)), per)
    start = cu[seq] + C * (np.arange(n) - first[seq])
    tok = torch.as_tensor(start[:, None] + np.arange(C), device=DEV)
    real = tok < torch.as_tensor(cu[seq + 1], device=DEV)[:, None]
    tok = torch.where(real, tok, 0)

    def chunks(x):  # [T, heads, d] to [n, H, C, d], zeros past a sequence's end
        x = _wide(x, H)[tok] * real[..., None, None]
        return x.transpose(1, 2).contiguous()

    q, k, v = chunks(s["q"]), chunks(s["k"]), chunks(s["v"])
    G = (s["g"].double()[tok] * real[..., None]).cumsum(1).transpose(1, 2)  # [n, H, C]
    low = torch.ones((C, C), dtype=torch.bool, device=DEV).tril()
    A = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, -math.inf).float())
    A *= torch.matmul(q, k.transpose(2, 3))
    o = torch.matmul(A, v)
    del A
    last = G[..., -1:]
    local = torch.matmul((k * torch.exp((last - G).float())[..., None]).transpose(2, 3), v)
    a = torch.exp(last.float())[..., None]                              # [n, H, 1, 1]
    state = s.get("state")
    if state is None:
        state = torch.zeros((len(lens), H, dk, dv), device=DEV)
    full = torch.as_tensor(np.flatnonzero(per), device=DEV)
    head = torch.as_tensor(first[per > 0], device=DEV)
    tail = torch.as_tensor((first + per - 1)[per > 0], device=DEV)
    local[head] += a[head] * state[full]
    a[head] = 0  # nothing passes from one sequence to the next
    run_ = 1
    while run_ < per.max():
        local[run_:] += a[run_:] * local[:-run_]
        a[run_:] *= a[:-run_].clone()
        run_ *= 2
    final = state.clone()
    final[full] = local[tail]
    enter = torch.cat([local[:1], local[:-1]])
    enter[head] = state[full]
    del local
    o += torch.matmul(q * torch.exp(G.float())[..., None], enter)
    return {"o": o.transpose(1, 2)[real].to(s["q"].dtype), "final": final}


def _plain_step(s):
    H = s["case"]["H"]
    at = s["slots"].long()
    S = s["state"][at] * torch.exp(s["g"])[..., None, None]
    S += _wide(s["k"], H)[..., None] * _wide(s["v"], H)[..., None, :]
    s["state"][at] = S
    o = (S * _wide(s["q"], H)[..., None]).sum(-2)
    return {"o": o.to(s["q"].dtype), "state": s["state"]}


def _plain_beam(s):
    c = s["case"]
    B, W, V, K = c["batch"], c["W"], c["V"], c["K"]
    x = s["logits"].double()
    top = x.amax(-1, keepdim=True)
    lse = top + torch.log(torch.exp(x - top).sum(-1, keepdim=True))
    cand = s["scores"].double()[..., None] + (x - lse)
    cand = torch.where(torch.isnan(cand), -math.inf, cand)
    done = s["finished"]
    if done is None:
        done = torch.zeros((B, W), dtype=torch.bool, device=DEV)
    keep = torch.full((V,), -math.inf, dtype=torch.float64, device=DEV)
    keep[EOS] = 0
    cand = torch.where(done[..., None], s["scores"].double()[..., None] + keep, cand)
    best, at = torch.sort(cand.view(B, W * V), dim=1, descending=True, stable=True)
    best, at = best[:, :K], at[:, :K]
    parents, tokens = at // V, at % V
    if c["order"] == "rows":
        # the first child of a beam to the beam's row, the others to the rows left, in order
        same = parents[:, :, None] == parents[:, None, :]
        stays = ~(same & torch.ones((K, K), dtype=torch.bool, device=DEV).tril(-1)).any(-1)
        taken = torch.zeros((B, K), dtype=torch.bool, device=DEV)
        taken.scatter_(1, parents, True)
        spare = torch.argsort(taken.to(torch.int8), dim=1, stable=True)  # free rows first, in order
        nth = torch.cumsum((~stays).long(), 1) - 1
        row = torch.where(stays, parents, torch.gather(spare, 1, nth.clamp(min=0)))
        back = torch.argsort(row, dim=1)
        best, parents, tokens = (torch.gather(v, 1, back) for v in (best, parents, tokens))
    finished = torch.gather(done, 1, parents) | (tokens == EOS)
    return {"scores": best.float(), "parents": parents.int(), "tokens": tokens.int(),
            "finished": finished}


def _plain_reorder(s):
    at = s["slots"].long()
    src = torch.gather(at, 1, s["parents"].long())
    s["state"][at.view(-1)] = s["state"][src.view(-1)]
    return {"state": s["state"]}


def _rms(x):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)


def _plain_norm(s):
    u = s["x"].float()
    if s["post"] is not None:
        u = _rms(u) * s["post"]
    if s["gate"] is not None:
        u = u / (1 + torch.exp(-s["gate"].float()))
    r = s["residual"].float() + s["scale"] * u
    out = {"residual": r.to(s["residual"].dtype)}
    if s["pre"] is not None:
        out["y"] = (_rms(r) * s["pre"]).to(s["x"].dtype)
    return out


OWN = {"attn": _own_attn, "step": _own_step, "beam": _own_beam, "reorder": _own_reorder,
       "norm": _own_norm}
PLAIN = {"attn": _plain_attn, "step": _plain_step, "beam": _plain_beam, "reorder": _plain_reorder,
         "norm": _plain_norm}


# ---------------------------------------------------------------- work and 64 bits

def work(case):
    op = case["op"]
    es = 2 if case["type"] == "bf16" else 4
    if op in ("attn", "step"):
        H, dk, dv = case["H"], case["dk"], case["dv"]
        rows = case.get("tokens") or case["rows"]
        states = 2 * rows if op == "step" else case["seqs"] * (2 if case["state"] else 1)
        return {"bytes": rows * (es * ((case["Hq"] + case["Hk"]) * dk + (case["Hv"] + H) * dv)
                                 + 4 * H) + 4 * states * H * dk * dv,
                "flops": 4 * rows * H * dk * dv}
    if op == "beam":
        n = case["batch"] * case["W"]
        return {"bytes": n * (case["V"] * es + 5) + case["batch"] * case["K"] * 13,
                "flops": 3 * n * case["V"]}
    if op == "reorder":
        K, live = case["K"], case["live"]
        moved = K - live
        read = min(live, moved)
        if case["order"] == "score":  # a row in K keeps its place by chance
            moved, read = K - 1, live
        return {"bytes": case["batch"] * (read + moved) * case["R"] * case["L"] * es, "flops": 0}
    rs = 2 if case["stream"] == "bf16" else 4
    per = es * (1 + case["gate"] + case["pre"]) + 2 * rs
    return {"bytes": case["D"] * (case["rows"] * per + 12),
            "flops": case["D"] * case["rows"] * 12}


def _exact_steps(s):
    """The attention token by token in 64 bits, all sequences beside each other."""
    c = s["case"]
    H, dk, dv = c["H"], c["dk"], c["dv"]
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    decay = torch.exp(s["g"].double())
    of = {n: torch.arange(H, device=DEV) // (H // c["H" + n]) for n in "qkv"}
    o = torch.empty((q.shape[0], H, dv), dtype=torch.float64, device=DEV)

    def step(S, rows):
        S = S * decay[rows].unsqueeze(-1).unsqueeze(-1)
        S += k[rows][:, of["k"]].unsqueeze(-1) * v[rows][:, of["v"]].unsqueeze(-2)
        o[rows] = (q[rows][:, of["q"]].unsqueeze(-1) * S).sum(-2)
        return S

    if c["op"] == "step":
        at = s["slots"].long()
        out = s["state"].double()
        out[at] = step(out[at], torch.arange(q.shape[0], device=DEV))
        return o, out
    cu = s["cu"]
    lens = np.diff(cu)
    order = np.argsort(-lens, kind="stable")  # sequences that end first come last
    where = torch.as_tensor(order, device=DEV)
    out = s["state"].double() if "state" in s else torch.zeros(
        (len(lens), H, dk, dv), dtype=torch.float64, device=DEV)
    S = out[where]
    begin = torch.as_tensor(cu[:-1][order], device=DEV)
    alive = [int(n) for n in np.searchsorted(-lens[order], -np.arange(lens.max()), side="left")]
    for t, live in enumerate(alive):
        S[:live] = step(S[:live], begin[:live] + t)
    out[where] = S
    return o, out


def _exact_beam(s):
    c = s["case"]
    V, K = c["V"], c["K"]
    scores, parents, tokens, finished = [], [], [], []
    for b in range(c["batch"]):
        lp = torch.log_softmax(s["logits"][b].double(), dim=-1)
        lp += s["scores"][b].double().unsqueeze(-1)
        done = [] if s["finished"] is None else s["finished"][b].nonzero().flatten().tolist()
        for w in done:
            lp[w] = -math.inf
            lp[w, EOS] = s["scores"][b, w].double()
        flat = lp.flatten()
        least = torch.topk(flat, K).values[-1]
        cand = [(-val, at) for val, at in zip(flat[flat >= least].tolist(),
                                              (flat >= least).nonzero().flatten().tolist())]
        cand = sorted(cand)[:K]
        if c["order"] == "rows":
            rows, late = [None] * K, []
            for item in cand:
                w = item[1] // V
                if rows[w] is None:
                    rows[w] = item
                else:
                    late.append(item)
            cand = [late.pop(0) if r is None else r for r in rows]
        scores.append([-v for v, _ in cand])
        parents.append([at // V for _, at in cand])
        tokens.append([at % V for _, at in cand])
        finished.append([at // V in done or at % V == EOS for _, at in cand])
    f = dict(device=DEV)
    return {"scores": torch.tensor(scores, dtype=torch.float64, **f),
            "parents": torch.tensor(parents, dtype=torch.int32, **f),
            "tokens": torch.tensor(tokens, dtype=torch.int32, **f),
            "finished": torch.tensor(finished, dtype=torch.bool, **f)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("attn", "step"):
        o, state = _exact_steps(s)
        return {"o": o, "final" if op == "attn" else "state": state}
    if op == "beam":
        return _exact_beam(s)
    if op == "reorder":
        out = s["state"].double()
        for row, near in zip(s["slots"].tolist(), s["parents"].tolist()):
            for to, source in zip(row, near):
                out[to] = s["state"][row[source]].double()
        return {"state": out}
    u = s["x"].double()
    if s["post"] is not None:
        u = u / torch.sqrt(u.square().mean(-1, keepdim=True) + 1e-6) * s["post"].double()
    if s["gate"] is not None:
        u = u * torch.sigmoid(s["gate"].double())
    r = s["residual"].double() + s["scale"].double() * u
    if s["pre"] is None:
        return {"residual": r}
    y = r / torch.sqrt(r.square().mean(-1, keepdim=True) + 1e-6) * s["pre"].double()
    return {"residual": r, "y": y}
