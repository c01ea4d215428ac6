"""Recurrent-layer serving operators: what is timed, and their plain forms.

Six calls, in three groups that are used together when a hybrid model with
recurrent mixers is served:

- ``short_conv`` / ``short_conv_step``: the short causal depthwise
  convolution in front of the recurrence, for packed prompts and for single
  tokens;
- ``selective_scan`` / ``selective_scan_step``: the selective state space scan
  (a diagonal recurrence with N states per channel), for packed prompts and
  for single tokens;
- ``state_store`` / ``state_load``: a pool of recurrent states held in 8 bits,
  quantised row by row as they are written, and read back.

``own`` chooses between the plain form (elementary torch operations, 32-bit)
and the library's calls.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
CODES = {"int8": (torch.int8, 127.0), "e4m3": (torch.float8_e4m3fn, 448.0)}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One user decoding: the q, k and v channels of 96 heads through the
        # convolution; only the call's latency counts.
        {"name": "conv_step_1x36864_bf16", "op": "conv_step", "rows": 1, "D": 36864, "W": 4,
         "type": "bf16", "slots": 8},
        # The decode batch of the benchmark (256 sequences) on the same channels.
        {"name": "conv_step_256x36864_bf16", "op": "conv_step", "rows": 256, "D": 36864, "W": 4,
         "type": "bf16", "slots": 300},
        # A full prompt of the benchmark's prefill, q, k and v channels.
        {"name": "conv_8192x36864_bf16", "op": "conv", "seqs": 1, "tokens": 8192, "D": 36864,
         "W": 4, "type": "bf16", "silu": True, "state": False},
        # A packed batch of resumed prompts of uneven length, fp32, 12 heads.
        {"name": "conv_64seqs_20000x1536_f32", "op": "conv", "seqs": 64, "tokens": 20000,
         "D": 1536, "W": 3, "type": "f32", "silu": False, "state": True},
        # A short prompt: latency again.
        {"name": "scan_256x1536_bf16", "op": "scan", "seqs": 1, "tokens": 256, "D": 1536, "N": 16,
         "G": 1, "type": "bf16", "gate": True, "state": False},
        # An ordinary long prompt of one sequence.
        {"name": "scan_8192x8192_bf16", "op": "scan", "seqs": 1, "tokens": 8192, "D": 8192,
         "N": 16, "G": 1, "type": "bf16", "gate": True, "state": False},
        # The long-context prompt of the benchmark: few channels, many tokens.
        {"name": "scan_131072x1536_bf16", "op": "scan", "seqs": 1, "tokens": 131072, "D": 1536,
         "N": 16, "G": 1, "type": "bf16", "gate": True, "state": False},
        # Packed resumed prompts, fp32, with sizes that divide nothing.
        {"name": "scan_37seqs_9001x1002_f32", "op": "scan", "seqs": 37, "tokens": 9001, "D": 1002,
         "N": 13, "G": 2, "type": "f32", "gate": False, "state": True},
        # A few users decoding, odd sizes.
        {"name": "scan_step_3x1002_f32", "op": "scan_step", "rows": 3, "D": 1002, "N": 13, "G": 2,
         "type": "f32", "gate": False, "slots": 7},
        # The benchmark's decode batch.
        {"name": "scan_step_256x12288_bf16", "op": "scan_step", "rows": 256, "D": 12288, "N": 16,
         "G": 1, "type": "bf16", "gate": True, "slots": 300},
        # 64 checkpoints of a 96-head KDA layer parked in the prefix cache.
        {"name": "store_64x12288x128_e4m3", "op": "store", "rows": 64, "R": 12288, "L": 128,
         "codes": "e4m3", "slots": 80},
        # Scan states of a batch taken back out of it.
        {"name": "load_250x8192x16_int8", "op": "load", "rows": 250, "R": 8192, "L": 16,
         "codes": "int8", "slots": 300},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_step", "conv", "scan", "scan", "scan_step", "store", "load"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op == "conv_step":
        rows = _log_int(rng, 1, 256)
        return {"op": op, "rows": rows, "D": _log_int(rng, 200, 36864), "W": rng.choice([2, 3, 4, 4]),
                "type": kind, "slots": rows + rng.randint(0, 50)}
    if op == "conv":
        tokens = _log_int(rng, 16, 60000)
        return {"op": op, "seqs": min(tokens, _log_int(rng, 1, 100)), "tokens": tokens,
                "D": min(_log_int(rng, 200, 36864), 150000000 // tokens), "W": rng.choice([2, 3, 4, 4]),
                "type": kind, "silu": rng.random() < 0.7, "state": rng.random() < 0.5}
    if op == "scan":
        tokens = _log_int(rng, 16, 131072)
        G = rng.choice([1, 1, 2, 4])
        return {"op": op, "seqs": min(tokens, _log_int(rng, 1, 60)), "tokens": tokens,
                "D": G * max(1, min(_log_int(rng, 200, 12288), 67000000 // tokens) // G),
                "N": rng.choice([16, 16, 8, 5, 13]), "G": G, "type": kind,
                "gate": rng.random() < 0.6, "state": rng.random() < 0.5}
    if op == "scan_step":
        rows = _log_int(rng, 1, 256)
        G = rng.choice([1, 1, 2, 4])
        return {"op": op, "rows": rows, "D": G * (_log_int(rng, 200, 12288) // G),
                "N": rng.choice([16, 16, 8, 5, 13]), "G": G, "type": kind,
                "gate": rng.random() < 0.6, "slots": rows + rng.randint(0, 50)}
    L = rng.choice([128, 128, 16, 64, 13])
    rows = _log_int(rng, 1, 64)
    return {"op": op, "rows": rows, "R": _log_int(rng, 500, 12288), "L": L,
            "codes": rng.choice(["int8", "e4m3"]), "slots": rows + rng.randint(0, 20)}


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


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    f = dict(device=DEV, generator=g)
    op = case["op"]
    s = {"case": case}
    if op in ("store", "load"):
        dt, qmax = CODES[case["codes"]]
        rows, R, L, pool = case["rows"], case["R"], case["L"], case["slots"]
        s["slots"] = _slots(rows, pool, seed)
        # rows of a state decay at different rates: their sizes differ
        size = torch.exp(torch.randn((rows, R, 1), **f))
        state = torch.randn((rows, R, L), **f) * size * 0.1
        s["codes"] = torch.zeros((pool, R, L), dtype=torch.int8, device=DEV).view(dt)
        s["scales"] = torch.zeros((pool, R), device=DEV)
        if op == "store":
            s["state"] = state
        else:
            scale = state.abs().amax(-1) / qmax
            q = state / scale[..., None]
            q = torch.round(q).to(torch.int8) if dt == torch.int8 else q.to(dt)
            at = s["slots"].long()
            s["codes"].view(torch.int8)[at] = q.view(torch.int8)
            s["scales"][at] = scale
            s["state"] = torch.zeros((rows, R, L), device=DEV)
        return s

    dt = TYPES[case["type"]]
    D = case["D"]
    if "tokens" in case:
        rows = case["tokens"]
        cu = np.concatenate([[0], np.cumsum(_lengths(rows, case["seqs"], seed))])
        s["cu"] = cu.astype(np.int64)
    else:
        rows = case["rows"]
        s["slots"] = _slots(rows, case["slots"], seed)
    if op.startswith("conv"):
        W = case["W"]
        s["x"] = torch.randn((rows, D), **f).to(dt)
        s["weight"] = (torch.rand((D, W), **f) * 2 - 1).mul_(W ** -0.5).to(dt)
        s["bias"] = (torch.randn((D,), **f) * 0.1).to(dt)
        if op == "conv_step":
            s["state"] = torch.randn((case["slots"], W - 1, D), **f).to(dt)
        elif case["state"]:
            s["state"] = torch.randn((case["seqs"], W - 1, D), **f).to(dt)
        return s

    N, G = case["N"], case["G"]
    s["x"] = torch.randn((rows, D), **f).to(dt)
    s["delta"] = (torch.randn((rows, D), **f) * 0.5).to(dt)
    # B and C are parts of one projection's output
    bc = torch.randn((rows, 2 * G * N), **f).to(dt)
    s["B"] = bc[:, : G * N].view(rows, G, N)
    s["C"] = bc[:, G * N:].view(rows, G, N)
    s["A"] = -torch.arange(1, N + 1, device=DEV) * torch.exp(0.1 * torch.randn((D, N), **f))
    s["D"] = torch.ones((D,), device=DEV)
    # step sizes spread between 0.001 and 0.1
    step = torch.exp(torch.rand((D,), **f) * math.log(100.0) + math.log(1e-3))
    s["bias"] = step + torch.log(-torch.expm1(-step))
    s["z"] = torch.randn((rows, D), **f).to(dt) if case["gate"] else None
    if op == "scan_step":
        s["state"] = torch.randn((case["slots"], D, N), **f) * 0.3
    elif case["state"]:
        s["state"] = torch.randn((case["seqs"], D, N), **f) * 0.3
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


def _own_conv(s):
    y, final = _kda().short_conv(s["x"], s["weight"], s["bias"], cu_seqlens=s["cu"],
                                 initial_state=s.get("state"),
                                 activation="silu" if s["case"]["silu"] else None)
    return {"y": y, "final": final}


def _own_conv_step(s):
    y = _kda().short_conv_step(s["state"], s["x"], s["weight"], s["bias"], activation="silu",
                               slots=s["slots"])
    return {"y": y, "state": s["state"]}


def _own_scan(s):
    y, final = _kda().selective_scan(s["x"], s["delta"], s["A"], s["B"], s["C"], D=s["D"],
                                     z=s["z"], delta_bias=s["bias"], delta_softplus=True,
                                     cu_seqlens=s["cu"], initial_state=s.get("state"))
    return {"y": y, "final": final}


def _own_scan_step(s):
    y = _kda().selective_scan_step(s["state"], s["x"], s["delta"], s["A"], s["B"], s["C"],
                                   D=s["D"], z=s["z"], delta_bias=s["bias"],
                                   delta_softplus=True, slots=s["slots"])
    return {"y": y, "state": s["state"]}


def _own_store(s):
    _kda().state_store(s["state"], s["codes"], s["scales"], dst=s["slots"])
    return {"codes": s["codes"], "scales": s["scales"]}


def _own_load(s):
    _kda().state_load(s["codes"], s["scales"], s["state"], src=s["slots"])
    return {"state": s["state"]}


# ---------------------------------------------------------------- plain forms

def _silu(x):
    return x / (1 + torch.exp(-x))


def _softplus(x):
    return torch.where(x > 20, x, torch.log1p(torch.exp(torch.clamp(x, max=20.0))))


def _starts(cu, T):
    """On the device: sequence bounds, and each token's sequence."""
    cu = torch.as_tensor(cu, device=DEV)
    seq = torch.searchsorted(cu, torch.arange(T, device=DEV), right=True) - 1
    return cu, seq


def _plain_conv(s):
    x, w = s["x"], s["weight"].float()
    T, D = x.shape
    W = w.shape[1]
    cu, seq = _starts(s["cu"], T)
    n = cu.numel() - 1
    state = s.get("state")
    if state is None:
        state = torch.zeros((n, W - 1, D), dtype=x.dtype, device=DEV)
    # every position before a sequence's start is a row of its state
    rows = torch.cat([state.reshape(n * (W - 1), D), x])
    base = n * (W - 1)

    def at(pos, sq):
        before = pos - cu[sq]
        return torch.where(before >= 0, base + pos, (sq + 1) * (W - 1) + before)

    t = torch.arange(T, device=DEV)
    acc = s["bias"].float().expand(T, D)
    for j in range(W):
        acc = acc + w[:, j] * rows[at(t - (W - 1) + j, seq)].float()
    if s["case"]["silu"]:
        acc = _silu(acc)
    sq = torch.arange(n, device=DEV)[:, None]
    last = cu[1:, None] - (W - 1) + torch.arange(W - 1, device=DEV)
    return {"y": acc.to(x.dtype), "final": rows[at(last, sq)]}


def _plain_conv_step(s):
    x, w = s["x"], s["weight"].float()
    at = s["slots"].long()
    win = torch.cat([s["state"][at], x[:, None]], dim=1)
    acc = (win.float() * w.t()).sum(1) + s["bias"].float()
    s["state"][at] = win[:, 1:]
    return {"y": _silu(acc).to(x.dtype), "state": s["state"]}


def _wide(v, D):
    """[rows, G, N] to one row of N for each channel."""
    return v.float().repeat_interleave(D // v.shape[1], dim=1)


def _scan_out(s, y):
    y = y + s["D"] * s["x"].float()
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return y.to(s["x"].dtype)


def _plain_scan(s):
    x = s["x"]
    T, D = x.shape
    cu, seq = _starts(s["cu"], T)
    n = cu.numel() - 1
    state = s.get("state")
    if state is None:
        state = torch.zeros((n, D, s["case"]["N"]), device=DEV)
    delta = _softplus(s["delta"].float() + s["bias"])
    a = torch.exp(delta[..., None] * s["A"])
    h = (delta * x.float())[..., None] * _wide(s["B"], D)
    full = (cu[1:] > cu[:-1]).nonzero()[:, 0]
    first = cu[full]
    h[first] += a[first] * state[full]
    a[first] = 0  # nothing passes from one sequence to the next
    # (a, h) of a run of tokens: doubled until every run reaches its start
    longest = int(np.max(np.diff(s["cu"])))
    k = 1
    while k < longest:
        h[k:] += a[k:] * h[:-k]
        a[k:] *= a[:-k].clone()
        k *= 2
    final = state.clone()
    final[full] = h[cu[1:][full] - 1]
    del a
    h *= _wide(s["C"], D)
    return {"y": _scan_out(s, h.sum(-1)), "final": final}


def _plain_scan_step(s):
    x = s["x"]
    D = x.shape[1]
    at = s["slots"].long()
    delta = _softplus(s["delta"].float() + s["bias"])
    h = s["state"][at] * torch.exp(delta[..., None] * s["A"])
    h = h + (delta * x.float())[..., None] * _wide(s["B"], D)
    s["state"][at] = h
    return {"y": _scan_out(s, (h * _wide(s["C"], D)).sum(-1)), "state": s["state"]}


def _plain_store(s):
    dt, qmax = CODES[s["case"]["codes"]]
    x = s["state"]
    amax = x.abs().amax(-1)
    scale = torch.maximum(amax / torch.full_like(amax, qmax), torch.full_like(amax, 2.0 ** -126))
    q = x * (torch.ones_like(scale) / scale)[..., None]
    ok = torch.isfinite(amax)
    q = torch.where(ok[..., None], q, 0.0)
    scale = torch.where(ok, scale, math.nan)
    q = torch.round(q).to(torch.int8) if dt == torch.int8 else q.to(dt)
    at = s["slots"].long()
    s["codes"].view(torch.int8)[at] = q.view(torch.int8)
    s["scales"][at] = scale
    return {"codes": s["codes"], "scales": s["scales"]}


def _plain_load(s):
    at = s["slots"].long()
    codes = s["codes"].view(torch.int8)[at].view(s["codes"].dtype)
    torch.mul(codes.float(), s["scales"][at][..., None], out=s["state"])
    return {"state": s["state"]}


OWN = {"conv": _own_conv, "conv_step": _own_conv_step, "scan": _own_scan,
       "scan_step": _own_scan_step, "store": _own_store, "load": _own_load}
PLAIN = {"conv": _plain_conv, "conv_step": _plain_conv_step, "scan": _plain_scan,
         "scan_step": _plain_scan_step, "store": _plain_store, "load": _plain_load}


# ---------------------------------------------------------------- work and 64 bits

def work(case):
    op = case["op"]
    if op in ("store", "load"):
        rows = case["rows"] * case["R"]
        return {"bytes": rows * (5 * case["L"] + 4), "flops": 2 * rows * case["L"]}
    es = 2 if case["type"] == "bf16" else 4
    D = case["D"]
    rows = case.get("tokens") or case["rows"]
    if op.startswith("conv"):
        W = case["W"]
        states = 2 * rows if op == "conv_step" else case["seqs"] * (2 if case["state"] else 1)
        return {"bytes": es * D * (2 * rows + states * (W - 1) + W + 1), "flops": 2 * W * rows * D}
    N, G = case["N"], case["G"]
    states = 2 * rows if op == "scan_step" else case["seqs"] * (2 if case["state"] else 1)
    return {"bytes": es * rows * ((4 if case["gate"] else 3) * D + 2 * G * N)
            + 4 * D * N * states + 4 * D * (N + 2),
            "flops": 7 * rows * D * N}


def _exact_steps(s):
    """The scan token by token in 64 bits, all sequences beside each other."""
    x, D, N = s["x"].double(), s["case"]["D"], s["case"]["N"]
    lin = s["delta"].double() + s["bias"].double()
    delta = torch.logaddexp(lin, torch.zeros_like(lin))
    A = s["A"].double()
    z = s["z"]
    head = torch.arange(D, device=DEV) // (D // s["case"]["G"])
    y = torch.empty_like(x)

    def step(h, rows):
        d = delta[rows]
        h = h * torch.exp(d.unsqueeze(-1) * A)
        h += (d * x[rows]).unsqueeze(-1) * s["B"][rows].double()[:, head]
        y[rows] = torch.einsum("rdn,rdn->rd", h, s["C"][rows].double()[:, head])
        return h

    if s["case"]["op"] == "scan_step":
        at = s["slots"].long()
        out = s["state"].double()
        out[at] = step(out[at], torch.arange(x.shape[0], device=DEV))
    else:
        cu = s["cu"]
        lens = np.diff(cu)
        order = np.argsort(-lens, kind="stable")  # sequences that end first come last
        out = s["state"].double() if "state" in s else torch.zeros(
            (len(lens), D, N), dtype=torch.float64, device=DEV)
        h = out[torch.as_tensor(order, device=DEV)]
        begin = torch.as_tensor(cu[:-1][order], device=DEV)
        alive = [int(v) for v in np.searchsorted(-lens[order], -np.arange(lens.max()), side="left")]
        for t, live in enumerate(alive):
            h[:live] = step(h[:live], begin[:live] + t)
        out[torch.as_tensor(order, device=DEV)] = h
    y += s["D"].double() * x
    if z is not None:
        y *= z.double() * torch.sigmoid(z.double())
    return y, out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "store":
        amax = s["state"].double().abs().amax(-1)
        scales = s["scales"].double()
        scales[s["slots"].long()] = amax / CODES[case["codes"]][1]
        return {"codes": None, "scales": scales}
    if op == "load":
        at = s["slots"].long()
        codes = s["codes"].view(torch.int8)[at].view(s["codes"].dtype)
        return {"state": codes.double() * s["scales"].double()[at].unsqueeze(-1)}
    if op.startswith("scan"):
        y, state = _exact_steps(s)
        return {"y": y, "final" if op == "scan" else "state": state}

    x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
    W = case["W"]

    def window(seq):  # [W-1 + len, D] to [len, D]
        out = b + w[:, W - 1] * seq[W - 1:]
        for back in range(1, W):
            out += w[:, W - 1 - back] * seq[W - 1 - back: seq.shape[0] - back]
        return out

    if op == "conv_step":
        at = s["slots"].long()
        past = s["state"].double()
        full = torch.cat([past[at], x.unsqueeze(1)], dim=1)
        y = b + torch.einsum("rwd,dw->rd", full, w)
        past[at] = full[:, 1:]
        return {"y": y * torch.sigmoid(y), "state": past}
    ys, ends = [], []
    for n in range(case["seqs"]):
        past = s["state"][n].double() if "state" in s else torch.zeros(
            (W - 1, case["D"]), dtype=torch.float64, device=DEV)
        seq = torch.cat([past, x[s["cu"][n]: s["cu"][n + 1]]])
        ys.append(window(seq))
        ends.append(seq[seq.shape[0] - (W - 1):])
    y = torch.cat(ys)
    if case["silu"]:
        y = y * torch.sigmoid(y)
    return {"y": y, "final": torch.stack(ends)}
