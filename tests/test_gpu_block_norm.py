"""Block norm on the GPU against its 64-bit form."""
import pytest
import torch

import block_ref as ref
import gated_delta_rule_19_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def make(rows, D, dtype, rdtype, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    return dict(x=n(rows, D).to(dtype), gate=(2 * n(rows, D)).to(dtype), residual=(3 * n(rows, D)).to(rdtype),
                scale=0.5 + 0.2 * n(D), post_weight=1 + 0.1 * n(D), weight=1 + 0.1 * n(D))


def compare(a, eps=1e-6, post_eps=1e-5, **kw):
    """`a` without the arguments that are None; what is in kw goes to the call as it is."""
    on = {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in a.items() if v is not None}
    r, y = kda.block_norm(eps=eps, post_eps=post_eps, **on, **kw)
    torch.cuda.synchronize()
    scale = 1.0 if a.get("scale") is None else a["scale"]
    rdt = a["residual"].dtype if a.get("residual") is not None else \
        kw["residual_out"].dtype if kw.get("residual_out") is not None else a["x"].dtype
    rr, rtol, ry, ytol = ref.block_norm(
        ref.f64(a["x"]), ref.f64(a.get("weight")), eps, ref.f64(a.get("residual")),
        ref.f64(scale) if isinstance(scale, torch.Tensor) else scale, ref.f64(a.get("gate")),
        ref.f64(a.get("post_weight")), post_eps, a["x"].dtype, rdt)
    if r is not None:
        assert r.dtype == rdt
        ref.check("r", r, rr, rtol)
    if ry is not None:
        assert y.dtype == a["x"].dtype
        ref.check("y", y, ry, ytol)
    return r, y


@pytest.mark.parametrize("dtype,rdtype", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("D", [1, 2, 7, 8, 9, 63, 64, 65, 128, 500, 512, 513, 1002, 1024, 1025, 2047, 2048, 2049,
                               4099, 12288, 20000, 32768, 32769, 65536])
def test_widths(D, dtype, rdtype):
    print("norm width", D, dtype, rdtype, flush=True)
    compare(make(5, D, dtype, rdtype, D))


@pytest.mark.parametrize("rows", [1, 2, 3, 31, 32, 33, 257])
def test_rows(rows):
    print("norm rows", rows, flush=True)
    for D in (40, 300, 3001):
        compare(make(rows, D, BF16, F32, rows))


@pytest.mark.parametrize("dtype,rdtype", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("D", [300, 3001])
@pytest.mark.parametrize("without", [(), ("gate",), ("residual",), ("scale",), ("post_weight",), ("weight",),
                                     ("gate", "post_weight"), ("gate", "residual", "scale"),
                                     ("gate", "post_weight", "residual", "scale"), ("weight", "residual"),
                                     ("weight", "residual", "scale", "gate", "post_weight")])
def test_parts(without, D, dtype, rdtype):
    print("norm parts", without, D, dtype, flush=True)
    a = make(4, D, dtype, rdtype, 3)
    for n in without:
        a[n] = None
    r, y = compare(a)
    assert (r is None) == (a["residual"] is None and a["weight"] is not None)
    assert (y is None) == (a["weight"] is None)


def test_scale_number_and_residual_out_alone():
    print("norm scale number", flush=True)
    a = make(4, 130, BF16, F32, 4)
    a["scale"] = -0.125
    compare(a)
    a["residual"] = None
    out = torch.empty(4, 130, device=DEV)
    r, _ = compare(a, residual_out=out)
    assert r is out


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [100, 2000, 5000])
def test_in_place(D, dtype):
    print("norm in place", D, dtype, flush=True)
    a = make(6, D, dtype, dtype, 5)
    want_r, want_y = compare(a)
    on = {k: v.to(DEV) for k, v in a.items()}
    x, res, gate = on["x"].clone(), on["residual"].clone(), on["gate"].clone()
    r, y = kda.block_norm(**{**on, "x": x, "residual": res}, post_eps=1e-5, residual_out=res, y=x)
    assert r is res and y is x and torch.equal(r, want_r) and torch.equal(y, want_y)
    r, y = kda.block_norm(**{**on, "gate": gate}, post_eps=1e-5, y=gate)
    assert torch.equal(y, want_y)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides_and_alignment(dtype):
    print("norm strides", dtype, flush=True)
    for D in (90, 700, 2500):
        a = make(7, D, dtype, F32, 6)
        wide = torch.full((7, 2 * D + 3), 9.0, dtype=dtype, device=DEV)
        wide[:, 1:1 + D] = a["x"].to(DEV)
        wide[:, 1 + D:1 + 2 * D] = a["gate"].to(DEV)
        out = torch.full((7, D + 9), 9.0, dtype=dtype, device=DEV)
        rout = torch.full((7, D + 1), 9.0, device=DEV)
        on = {k: v.to(DEV) for k, v in a.items()}
        r, y = kda.block_norm(wide[:, 1:1 + D], weight=on["weight"], residual=on["residual"], scale=on["scale"],
                              gate=wide[:, 1 + D:1 + 2 * D], post_weight=on["post_weight"], post_eps=1e-5,
                              y=out[:, 5:5 + D], residual_out=rout[:, 1:])
        want_r, want_y = compare(a)
        assert torch.equal(r, want_r) and torch.equal(y, want_y)
        assert (out[:, :5] == 9).all() and (out[:, 5 + D:] == 9).all() and (rout[:, 0] == 9).all()
        assert (wide[:, 0] == 9).all() and (wide[:, 1 + 2 * D:] == 9).all()


def test_special_rows():
    """Zero rows, one infinite or NaN element: nothing leaves its row."""
    print("norm special rows", flush=True)
    for D in (64, 3001):
        a = make(6, D, F32, F32, 7)
        clean_r, clean_y = compare(a)
        b = {k: v.clone() for k, v in a.items()}
        b["x"][1] = 0
        b["x"][2, 5] = float("nan")
        b["x"][3, 7] = float("inf")
        b["residual"][4, 1] = -float("inf")
        r, y = kda.block_norm(**{k: v.to(DEV) for k, v in b.items()}, post_eps=1e-5)
        for i in (0, 5):
            assert torch.equal(r[i], clean_r[i]) and torch.equal(y[i], clean_y[i])
        assert torch.isfinite(y[1]).all() and torch.equal(r[1].cpu(), b["residual"][1])
        assert torch.isnan(r[2]).all() and torch.isnan(r[3, 7])
        assert (torch.isfinite(r[4]).sum() == D - 1) and torch.isnan(y[4, 1]) and (y[4, 2:] == 0).all()
    z = torch.zeros(2, 40, device=DEV)
    r, y = kda.block_norm(z, weight=torch.ones(40, device=DEV), post_weight=torch.ones(40, device=DEV))
    assert (y == 0).all()


def test_offsets_past_32_bits():
    print("norm offsets past 32 bits", flush=True)
    rows, D = 70000, 32768  # 2.3e9 elements
    x = torch.zeros((rows, D), dtype=BF16, device=DEV)
    a = make(1, D, BF16, BF16, 8)
    x[-1:] = a["x"].to(DEV)
    w = a["weight"].to(DEV)
    _, y = kda.block_norm(x, weight=w)
    _, one = kda.block_norm(a["x"].to(DEV), weight=w)
    assert torch.equal(y[-1:], one) and (y[:5] == 0).all()


def test_no_rows():
    print("norm no rows", flush=True)
    r, y = kda.block_norm(torch.empty(0, 8, device=DEV), weight=torch.ones(8, device=DEV))
    assert r is None and y.shape == (0, 8)
