"""Plain 64-bit forms of the short convolution, the selective scan and the
8-bit state cache, with error bounds that follow the kernels' roundings.

Each form returns its result and, beside it, an elementwise bound on how far
a kernel may be from it that rounds where include/kda.h says it does: fp32
arithmetic (U = 2^-24 a rounding; 2 U for the hardware's exponential and
reciprocal), one rounding of the output to its type (HALF).
"""
import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def _sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


# silu(s) in fp32, relative: the argument times log2(e) (constant and product:
# 2 U of it, which the exponential turns into 2 U |s|), the exponential 2 U,
# the sum 1 U, the reciprocal 2 U, the product 1 U
def _silu_rel(s):
    return U * (2 * np.abs(s) + 6)


def conv(x, weight, bias, cu, init, act, dtype):
    """y, its bound, and the final state ([N, W - 1, D])."""
    T, D = x.shape
    W = weight.shape[1]
    y = np.zeros((T, D))
    tol = np.zeros((T, D))
    fin = np.zeros((len(cu) - 1, W - 1, D))
    for n in range(len(cu) - 1):
        a, b = cu[n], cu[n + 1]
        past = np.zeros((W - 1, D)) if init is None else init[n]
        rows = np.concatenate([past, x[a:b]])
        fin[n] = rows[rows.shape[0] - (W - 1):]
        s = np.zeros((b - a, D)) + (0.0 if bias is None else bias)
        mag = np.abs(s)
        for j in range(W):
            s = s + weight[:, j] * rows[j: j + b - a]
            mag = mag + np.abs(weight[:, j] * rows[j: j + b - a])
        out, err = _activate(s, (W + 1) * U * mag, act)
        y[a:b] = out
        tol[a:b] = err + HALF[dtype] * np.abs(out) + 1e-37
    return y, tol, fin


def _activate(s, err, act):
    if not act:
        return s, err
    out = s * _sigmoid(s)
    # |silu'| <= 1.1
    return out, 1.1 * err + _silu_rel(s) * np.abs(out)


def conv_step(x, state, weight, bias, act, dtype):
    """y [N, D], its bound, and the shifted state."""
    rows = np.concatenate([state, x[:, None]], axis=1)
    b = 0.0 if bias is None else bias
    prod = rows * weight.T[None]
    s = prod.sum(1) + b
    mag = np.abs(prod).sum(1) + np.abs(b)
    out, err = _activate(s, (weight.shape[1] + 1) * U * mag, act)
    return out, err + HALF[dtype] * np.abs(out) + 1e-37, rows[:, 1:]


def scan(x, delta, A, B, C, D, z, bias, softplus, cu, init, dtype, fold=1.0):
    """y, its bound, the final states and theirs.

    The bound follows the recurrence.  With rd the relative error of delta,
    a step's decay is off by |delta A| (rd + 3 U) (its argument: A log2(e) and
    the product) plus 2 U (the exponential), its input by (rd + 2 U), and the
    sum by U; what is there is carried on by the decay.  ``fold`` = 2 where
    the call may cut the sequence: a segment's decay is the exponential of a
    sum of n delta, off by n U |A sum| exp(A sum) <= n U, as much as the n
    steps' own decays together.
    """
    T, ch = x.shape
    N = A.shape[1]
    head = np.arange(ch) // (ch // B.shape[1])
    lin = delta + (0.0 if bias is None else bias)
    if softplus:
        d = np.logaddexp(lin, 0.0)
        # the sum is off by U |lin| (twice: inputs are exact, one rounding),
        # softplus' = sigmoid; its own evaluation: exponential of |lin|
        # (2 |lin| + 2 U on e, which enters log1p(e) at most in proportion),
        # 2 + e, reciprocal, products and series: 10 U
        rd = U * (3 * np.abs(lin) + 12)
        rd = np.where(lin > 0, U * 16, rd)
    else:
        d = lin
        rd = np.full_like(d, U)
    nseq = len(cu) - 1
    y = np.zeros((T, ch))
    ytol = np.zeros((T, ch))
    fin = np.zeros((nseq, ch, N)) if init is None else init.copy()
    ftol = np.zeros((nseq, ch, N))
    for n in range(nseq):
        h = fin[n]
        E = ftol[n]
        for t in range(cu[n], cu[n + 1]):
            dt_, r = d[t][:, None], rd[t][:, None]
            with np.errstate(over="ignore", invalid="ignore"):
                a = np.exp(dt_ * A)
                inp = dt_ * x[t][:, None] * B[t][head]
                hold = a * h
                E = a * E + np.abs(hold) * (np.abs(dt_ * A) * (r + 3 * U) + 2 * U) \
                    + np.abs(inp) * (r + 2 * U)
                h = hold + inp
                E = E + U * np.abs(h)
                term = C[t][head] * h
                v = term.sum(1)
                e = (np.abs(C[t][head]) * E * fold).sum(1) + (N + 3) * U * np.abs(term).sum(1)
                if D is not None:
                    v = v + D * x[t]
                    e = e + U * (np.abs(D * x[t]) + np.abs(v))
                if z is not None:
                    gate = z[t] * _sigmoid(z[t])
                    v = v * gate
                    e = e * np.abs(gate) + np.abs(v) * (_silu_rel(z[t]) + U)
            y[t] = v
            ytol[t] = e
        fin[n] = h
        ftol[n] = E
    return y, ytol + HALF[dtype] * np.abs(y) + 1e-37, fin, ftol * fold + 1e-37


def quantise(state, kind):
    """codes (int8 values, or the fp32 values e4m3 holds) and scales, by the
    definition, in fp32 where it says fp32."""
    x = state.numpy().astype(np.float32)
    qmax = np.float32(127 if kind == torch.int8 else 448)
    with np.errstate(all="ignore"):
        amax = np.max(np.abs(x), axis=-1)
        ok = np.isfinite(amax)
        scale = np.maximum(amax / qmax, np.float32(2.0 ** -126))
        top = np.float32(np.finfo(np.float32).max / qmax)
        while not np.isfinite(top * qmax):
            top = np.nextafter(top, np.float32(0))
        scale = np.minimum(scale, top)
        q = x * (np.float32(1) / scale)[..., None]
    q = np.where(ok[..., None], q, np.float32(0))
    scale = np.where(ok, scale, np.float32(np.nan)).astype(np.float32)
    if kind == torch.int8:
        return torch.from_numpy(np.rint(q).astype(np.int8)), torch.from_numpy(scale)
    return torch.from_numpy(q.astype(np.float32)).to(kind), torch.from_numpy(scale)


def check(name, got, ref, tol):
    """`got` within `tol` of `ref` everywhere."""
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    bad = ~(np.abs(got - ref) <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(got - ref) / tol, -1)), got.shape)
        raise AssertionError("%s: %d of %d beyond the bound; at %s got %r, expected %r +- %.3g" % (
            name, bad.sum(), bad.size, i, got[i], ref[i], tol[i]))
