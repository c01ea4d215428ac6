"""Plain 64-bit forms of the decayed attention, the block norm, beam selection
and state reordering, with error bounds that follow the kernels' roundings
(include/kda.h): U = 2^-24 for an fp32 operation, HALF for one rounding to an
element type.
"""
import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64)


def _heads(x, H):
    return x.repeat_interleave(H // x.shape[1], dim=1)


def decay_attention(q, k, v, g, scale, cu, init, dtype):
    """o, its bound, the final states and theirs (all 64-bit, on the CPU).

    Beside S runs A, the same sums of absolute values, and E, the bound of
    the state's error.  A step's decay is off by U (2 |g| + 4) relative (its
    argument in fp32, log2(e) and the exponential) and each step adds a few
    roundings, which the decay carries on.  A chunk adds up to 64 decayed
    products at once: 64 U of A where the steps' own bound is carried away by
    the decay; 80 U with the products' own.  bf16 only: the update's operand
    is split into three bf16 parts, which leave 2^-24 of it, one U more.

    o: fp32 sums over dk and a chunk: (dk + 80) U of sum |q| A, and with bf16
    half a step each of the scores and of the state that enters (their sum
    with |q| A at most), and of o.
    """
    T = q.shape[0]
    H, dk, dv = g.shape[-1], q.shape[2], v.shape[2]
    q, k, v = _heads(q, H), _heads(k, H), _heads(v, H)
    if g.dim() == 1:
        g = g.expand(T, H)
    n = len(cu) - 1
    o, otol = torch.zeros(T, H, dv, dtype=torch.float64), torch.zeros(T, H, dv, dtype=torch.float64)
    fin = torch.zeros(n, H, dk, dv, dtype=torch.float64) if init is None else init.clone()
    ftol = torch.zeros_like(fin)
    for i in range(n):
        S = fin[i]
        A, E = S.abs(), torch.zeros_like(S)
        for t in range(cu[i], cu[i + 1]):
            a = torch.exp(g[t])[:, None, None]
            E = a * (E + U * (2 * g[t].abs().clamp(max=150)[:, None, None] + 4) * A)
            outer = k[t][:, :, None] * v[t][:, None, :]
            S = a * S + outer
            A = a * A + outer.abs()
            E = E + 4 * U * A
            o[t] = scale * (q[t][:, :, None] * S).sum(1)
            mag = (q[t].abs()[:, :, None] * A).sum(1)
            err = (q[t].abs()[:, :, None] * E).sum(1) * 2 + (dk + 80) * U * mag
            if dtype == torch.bfloat16:
                err = err + 1.01 * HALF[dtype] * mag
            otol[t] = abs(scale) * err + HALF[dtype] * (o[t].abs() + abs(scale) * err)
        fin[i] = S
        ftol[i] = 2 * E + 80 * U * A
    return o, otol + 1e-37, fin, ftol + 1e-37


def block_norm(x, weight, eps, residual, scale, gate, post_weight, post_eps, dtype, rdtype):
    """r, its bound, y or None and its bound.

    A mean of D squares summed lane by lane (at most 64 + 11 deep here) is off
    by 80 U, its root by half of that, with the division and the products 46 U
    relative.  The gate: the argument times log2(e) (2 U of it), exponential
    and reciprocal 2 U each, 2 more."""
    D = x.shape[1]
    u = x.clone()
    rel = torch.zeros_like(u)
    if post_weight is not None:
        u = u / torch.sqrt(u.square().mean(-1, keepdim=True) + post_eps) * post_weight
        rel = rel + 46 * U
    if gate is not None:
        sig = torch.sigmoid(gate)
        u = u * sig
        rel = rel + U * (8 + 2 * gate.abs() * (1 - sig))
    u = scale * u
    rel = rel + 2 * U
    r = u if residual is None else residual + u
    err = u.abs() * rel + U * r.abs()
    rtol = err + HALF[rdtype] * r.abs()
    if weight is None:
        return r, rtol + 1e-37, None, None
    root = torch.sqrt(r.square().mean(-1, keepdim=True) + eps)
    y = r / root * weight
    # the mean moves by at most 2 |r| err / D summed: its root by that over 2 root^2
    moved = (r.abs() * err).sum(-1, keepdim=True) / D / root.square()
    ytol = err / root * weight.abs() + y.abs() * (moved + 46 * U)
    return r, rtol + 1e-37, y, ytol + HALF[dtype] * (y.abs() + ytol) + 1e-37


def beam_select(logits, scores, K, finished=None, eos=-1, order="score"):
    """scores, parents, tokens, finished by the definition, one batch at a
    time; logits as they are, values in 64 bits."""
    B, W, V = logits.shape
    x = logits.double()
    out = [[], [], [], []]
    for b in range(B):
        cand = torch.full((W, V), -np.inf, dtype=torch.float64)
        for w in range(W):
            s = float(scores[b, w])
            if not np.isfinite(s):
                continue
            if finished is not None and finished[b, w]:
                cand[w, eos] = s
                continue
            row = x[b, w]
            top = row.max()
            lse = top + torch.log(torch.exp(row - top).sum())
            if torch.isfinite(lse):
                cand[w] = s + (row - lse)
        flat = cand.flatten().numpy()
        pick = np.argsort(-flat, kind="stable")[:K]
        sel = [(flat[i], int(i) // V, int(i) % V) for i in pick]
        if order == "rows":
            rows, late = [None] * K, []
            for c in sel:
                if rows[c[1]] is None:
                    rows[c[1]] = c
                else:
                    late.append(c)
            sel = [late.pop(0) if c is None else c for c in rows]
        out[0].append([c[0] for c in sel])
        out[1].append([c[1] for c in sel])
        out[2].append([c[2] for c in sel])
        out[3].append([bool((finished is not None and finished[b, c[1]]) or c[2] == eos)
                       for c in sel])
    return (torch.tensor(out[0], dtype=torch.float64).view(B, K),
            torch.tensor(out[1], dtype=torch.int32).view(B, K),
            torch.tensor(out[2], dtype=torch.int32).view(B, K),
            torch.tensor(out[3], dtype=torch.bool).view(B, K))


def reorder(state, parents, slots=None):
    """A copy of `state` reordered."""
    G, K = parents.shape
    if slots is None:
        slots = torch.arange(G * K, dtype=torch.int32).view(G, K)
    out = state.clone()
    n = state.shape[0]
    for b in range(G):
        for r in range(K):
            p = int(parents[b, r])
            if not 0 <= p < K:
                continue
            to, src = int(slots[b, r]), int(slots[b, p])
            if 0 <= to < n and 0 <= src < n:
                out[to] = state[src]
    return out


def check(name, got, want, tol):
    """`got` within `tol` of `want` everywhere."""
    got = f64(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    bad = ~((got - want).abs() <= tol)
    if bad.any():
        far = torch.where(bad, (got - want).abs() / tol, torch.tensor(-1.0, dtype=torch.float64))
        at = np.unravel_index(int(torch.nan_to_num(far, nan=np.inf).argmax()), got.shape)
        raise AssertionError("%s: %d of %d beyond the bound; at %s got %r, expected %r +- %.3g" % (
            name, int(bad.sum()), bad.numel(), at, float(got[at]), float(want[at]), float(tol[at])))
