"""CPU tests of the short convolution, the selective scan and the state cache:
what the C ABI and the binding refuse (before anything reaches a device), and
the 64-bit forms of the GPU tests against closed forms."""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_19_amd as kda
from gated_delta_rule_19_amd import _native as nat
import recurrent_ref as ref

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
F32, BF16 = nat.KDA_F32, nat.KDA_BF16
PTR = 0x7F0000000000  # never dereferenced: every call below is refused


@pytest.fixture(scope="module")
def lib():
    return nat.load()


def cu_ptr(*bounds):
    a = np.array(bounds, dtype=np.int64)
    return a, a.ctypes.data_as(ctypes.POINTER(ctypes.c_int64))


# ---- C ABI: short convolution ----------------------------------------------------

def conv(lib, cu=(0, 5), D=64, W=4, dt=BF16, x=PTR, xs=64, w=PTR + (1 << 20), b=None, act=1,
         init=None, fin=None, slots=None, num_slots=1, y=PTR + (1 << 24), ys=64, ws=None, wsb=0,
         n=None):
    keep, p = cu_ptr(*cu)
    return lib.kda_short_conv(len(cu) - 1 if n is None else n, p, D, W, dt, x, xs, w, b, act, init,
                              fin, slots, num_slots, y, ys, ws, wsb, None)


@pytest.mark.parametrize("status,kw", [
    (UNSUPPORTED, dict(dt=7)),
    (UNSUPPORTED, dict(W=1)),
    (UNSUPPORTED, dict(W=9)),
    (INVALID, dict(D=0)),
    (INVALID, dict(act=2)),
    (INVALID, dict(n=-1)),
    (INVALID, dict(cu=(1, 5))),
    (INVALID, dict(cu=(0, 5, 4))),
    (INVALID, dict(cu=(0, 1 << 31))),
    (INVALID, dict(x=None)),
    (INVALID, dict(x=PTR + 1)),
    (INVALID, dict(xs=63)),
    (INVALID, dict(w=None)),
    (INVALID, dict(w=PTR + 2)),
    (INVALID, dict(b=PTR + 8)),
    (INVALID, dict(y=None)),
    (INVALID, dict(ys=63)),
    (INVALID, dict(y=PTR)),                            # y on x
    (INVALID, dict(y=PTR + 2)),                        # interleaved by one column
    (INVALID, dict(xs=128, ys=128, y=PTR + 2 * 63)),   # one shared column
    (INVALID, dict(xs=128, ys=127, y=PTR + 2 * 64)),   # other pitch: ranges meet
    (INVALID, dict(fin=PTR + (1 << 28) + 8)),
    (INVALID, dict(slots=PTR + 2)),
    (INVALID, dict(cu=(0, 2, 5), fin=PTR + (1 << 28), num_slots=1)),
    (INVALID, dict(init=PTR + (1 << 28), fin=PTR + (1 << 28) + 16)),
    (WORKSPACE, dict(cu=tuple(range(80)))),
    (WORKSPACE, dict(cu=tuple(range(80)), ws=PTR, wsb=64)),
    (INVALID, dict(cu=tuple(range(80)), ws=PTR + 16, wsb=1 << 20)),
])
def test_short_conv_refuses(lib, status, kw):
    assert conv(lib, **kw) == status


def test_short_conv_of_no_sequences_is_a_no_op(lib):
    assert conv(lib, cu=(0,), x=None, y=None) == OK


def test_short_conv_workspace(lib):
    assert lib.kda_short_conv_workspace_size(0) == 0
    assert lib.kda_short_conv_workspace_size(64) == 0
    assert lib.kda_short_conv_workspace_size(65) >= 66 * 32
    assert lib.kda_short_conv_workspace_size(-1) == 0


@pytest.mark.parametrize("status,kw", [
    (UNSUPPORTED, dict(W=0)), (UNSUPPORTED, dict(dt=3)), (INVALID, dict(N=-1)),
    (INVALID, dict(state=None)), (INVALID, dict(state=PTR + (1 << 28) + 4)),
    (INVALID, dict(num_slots=2)), (INVALID, dict(num_slots=-1, slots=PTR)),
    (INVALID, dict(x=None)), (INVALID, dict(y=PTR, ys=65)), (INVALID, dict(y=PTR + 2)),
    (INVALID, dict(weight=None)),
])
def test_short_conv_step_refuses(lib, status, kw):
    a = dict(N=3, D=64, W=4, dt=BF16, x=PTR, xs=64, weight=PTR + (1 << 20), bias=None, act=0,
             state=PTR + (1 << 28), slots=None, num_slots=3, y=PTR + (1 << 24), ys=64, stream=None)
    a.update(kw)
    assert lib.kda_short_conv_step(*a.values()) == status
    a.update(N=0)
    if "N" not in kw and status == INVALID and set(kw) <= {"state", "x", "y", "ys", "weight"}:
        assert lib.kda_short_conv_step(*a.values()) == OK  # nothing to do


# ---- C ABI: selective scan --------------------------------------------------------

def ssm_io(**kw):
    a = dict(x=PTR, delta=PTR + (1 << 24), B=PTR + (2 << 24), C=PTR + (3 << 24), z=None,
             y=PTR + (4 << 24), x_stride=64, delta_stride=64, B_stride=16, C_stride=16,
             z_stride=0, y_stride=64, A=PTR + (5 << 24), D_skip=None, delta_bias=None,
             delta_softplus=1, reserved=0)
    a.update(kw)
    return nat.SsmIo(**a)


@pytest.mark.parametrize("status,io,kw", [
    (UNSUPPORTED, {}, dict(dt=2)),
    (UNSUPPORTED, {}, dict(N=129)),
    (INVALID, {}, dict(N=0)),
    (INVALID, {}, dict(D=0)),
    (INVALID, {}, dict(G=3)),
    (INVALID, {}, dict(G=0)),
    (INVALID, {}, dict(split=-1)),
    (INVALID, {}, dict(cu=(0, 3, 2))),
    (INVALID, dict(reserved=1), {}),
    (INVALID, dict(delta_softplus=2), {}),
    (INVALID, dict(x=None), {}),
    (INVALID, dict(delta=None), {}),
    (INVALID, dict(B=None), {}),
    (INVALID, dict(C=PTR + 1), {}),
    (INVALID, dict(A=None), {}),
    (INVALID, dict(A=PTR + 4), {}),
    (INVALID, dict(D_skip=PTR + 4), {}),
    (INVALID, dict(x_stride=63), {}),
    (INVALID, dict(B_stride=15), {}),
    (INVALID, dict(z=PTR + (6 << 24), z_stride=63), {}),
    (INVALID, dict(y=PTR), {}),
    (INVALID, dict(y=PTR + (3 << 24)), {}),
    (INVALID, dict(z=PTR + (4 << 24) + 2, z_stride=64), {}),
    (INVALID, {}, dict(fin=PTR + (7 << 24) + 4)),
    (INVALID, {}, dict(fin=PTR + (7 << 24), num_slots=0)),
    (INVALID, {}, dict(init=PTR + (7 << 24), fin=PTR + (7 << 24) + 64)),
    (INVALID, {}, dict(slots=PTR + 1)),
    (WORKSPACE, {}, dict(cu=(0, 4096), split=8, wsb=0)),
    (WORKSPACE, {}, dict(cu=(0, 4096), split=8, ws=None)),
    (INVALID, {}, dict(cu=(0, 4096), split=8, ws=PTR + (8 << 24) + 64)),
])
def test_selective_scan_refuses(lib, status, io, kw):
    a = dict(cu=(0, 5), D=64, N=16, G=1, dt=BF16, init=None, fin=None, slots=None, num_slots=1,
             split=0, ws=PTR + (8 << 24), wsb=1 << 24)
    a.update(kw)
    keep, p = cu_ptr(*a["cu"])
    blk = ssm_io(**io)
    assert lib.kda_selective_scan(len(a["cu"]) - 1, p, a["D"], a["N"], a["G"], a["dt"],
                                  ctypes.byref(blk), a["init"], a["fin"], a["slots"],
                                  a["num_slots"], a["split"], a["ws"], a["wsb"], None) == status


def test_selective_scan_refuses_a_null_block_and_bad_bounds(lib):
    keep, p = cu_ptr(0, 5)
    assert lib.kda_selective_scan(1, p, 64, 16, 1, BF16, None, None, None, None, 1, 0, PTR,
                                  1 << 24, None) == INVALID
    assert lib.kda_selective_scan_workspace_size(1, p, 64, 129, 1, 0) == 0
    assert lib.kda_selective_scan_workspace_size(1, p, 64, 16, 1, -1) == 0
    keep2, p2 = cu_ptr(0, -5)
    assert lib.kda_selective_scan_workspace_size(1, p2, 64, 16, 1, 0) == 0


def test_selective_scan_workspace_grows_with_the_cut(lib):
    keep, p = cu_ptr(0, 4096)
    one = lib.kda_selective_scan_workspace_size(1, p, 64, 16, 1, 1)
    # seven transition pairs more: end states [64, 16] and sums [64] each
    assert lib.kda_selective_scan_workspace_size(1, p, 64, 16, 1, 8) >= one + 7 * 64 * 17 * 4


@pytest.mark.parametrize("status,io,kw", [
    (UNSUPPORTED, {}, dict(N=200)), (INVALID, {}, dict(rows=-1)), (INVALID, {}, dict(state=None)),
    (INVALID, {}, dict(state=PTR + (7 << 24) + 8)), (INVALID, {}, dict(num_slots=2)),
    (INVALID, dict(x=None), {}), (INVALID, dict(y=PTR), {}), (INVALID, dict(C_stride=3), {}),
])
def test_selective_scan_step_refuses(lib, status, io, kw):
    a = dict(rows=3, D=64, N=16, G=1, dt=BF16, state=PTR + (7 << 24), slots=None, num_slots=3)
    a.update(kw)
    blk = ssm_io(**io)
    args = (a["D"], a["N"], a["G"], a["dt"], ctypes.byref(blk), a["state"], a["slots"],
            a["num_slots"], None)
    assert lib.kda_selective_scan_step(a["rows"], *args) == status


# ---- C ABI: state cache -------------------------------------------------------------

@pytest.mark.parametrize("status,kw", [
    (UNSUPPORTED, dict(format=2)), (UNSUPPORTED, dict(L=257)), (INVALID, dict(L=0)),
    (INVALID, dict(R=0)), (INVALID, dict(n=-1)), (INVALID, dict(num_a=1)),
    (INVALID, dict(num_b=1)), (INVALID, dict(a=None)), (INVALID, dict(c=None)),
    (INVALID, dict(sc=None)), (INVALID, dict(sc=PTR + 2)), (INVALID, dict(src=PTR + 2)),
    (INVALID, dict(n=1 << 30, R=1 << 31, num_a=1 << 30, num_b=1 << 30)),
])
def test_state_cache_refuses(lib, status, kw):
    a = dict(n=2, R=8, L=16, format=0, a=PTR, src=None, num_a=2, c=PTR + (1 << 24),
             sc=PTR + (2 << 24), dst=None, num_b=2)
    a.update(kw)
    assert lib.kda_state_store(a["n"], a["R"], a["L"], a["format"], a["a"], a["src"], a["num_a"],
                               a["c"], a["sc"], a["dst"], a["num_b"], None) == status
    assert lib.kda_state_load(a["n"], a["R"], a["L"], a["format"], a["c"], a["sc"], a["src"],
                              a["num_a"], a["a"], a["dst"], a["num_b"], None) == status


def test_state_cache_refuses_a_grid_that_passes_64_bits(lib):
    n, R, L = (1 << 31) - 1, 1 << 31, 255
    for fmt in (0, 1):
        assert lib.kda_state_store(n, R, L, fmt, PTR, None, n, PTR + (1 << 24), PTR + (2 << 24),
                                   None, n, None) == INVALID
        assert lib.kda_state_load(n, R, L, fmt, PTR + (1 << 24), PTR + (2 << 24), None, n, PTR,
                                  None, n, None) == INVALID


def test_state_cache_of_no_items_is_a_no_op(lib):
    assert lib.kda_state_store(0, 8, 16, 0, None, None, 0, None, None, None, 0, None) == OK
    assert lib.kda_state_load(0, 8, 16, 1, None, None, None, 0, None, None, 0, None) == OK


# ---- C ABI: what a call writes lies apart from everything else it is given ---------
# (81 sequences and no workspace: a call whose arguments pass is then refused
# for that, before anything is enqueued)

CU80 = tuple(range(0, 160, 2)) + (160,)
FAR = PTR + (1 << 28)


@pytest.mark.parametrize("status,kw", [
    (WORKSPACE, {}),
    (INVALID, dict(w=PTR + (1 << 24) + 128)),                    # y on the weights
    (INVALID, dict(w=PTR + (1 << 24) - 64 * 4 * 2 + 16)),        # their end
    (WORKSPACE, dict(w=PTR + (1 << 24) - 64 * 4 * 2)),           # right in front of y
    (WORKSPACE, dict(w=PTR + (1 << 24) + 160 * 64 * 2)),         # right behind it
    (INVALID, dict(w=PTR + (1 << 24) + 160 * 64 * 2 - 16)),
    (INVALID, dict(b=PTR + (1 << 24) + 256)),
    (INVALID, dict(init=PTR + (1 << 24) + 256, num_slots=80)),
    (INVALID, dict(fin=PTR + (1 << 24) - 80 * 3 * 64 * 2 + 16, num_slots=80)),
    (WORKSPACE, dict(fin=PTR + (1 << 24) - 80 * 3 * 64 * 2, num_slots=80)),
    (INVALID, dict(slots=PTR + (1 << 24) + 4)),
    (INVALID, dict(fin=PTR + 256, num_slots=80)),                # final state on x
    (INVALID, dict(init=PTR + 256, fin=PTR + 256, num_slots=80)),
    (WORKSPACE, dict(init=PTR + 256, num_slots=80)),             # both only read
    (INVALID, dict(fin=PTR + (1 << 20), num_slots=80)),          # on the weights
    (INVALID, dict(b=FAR, fin=FAR, num_slots=80)),
    (INVALID, dict(slots=FAR + 8, fin=FAR, num_slots=80)),
    # rows of 64 columns in a buffer of 128: between them there is room for 128 bytes
    (WORKSPACE, dict(xs=128, ys=128, b=PTR + (1 << 24) + 128)),
    (WORKSPACE, dict(xs=128, ys=128, b=PTR + (1 << 24) + 256 * 159 - 128)),
    (INVALID, dict(xs=128, ys=128, b=PTR + (1 << 24) + 128 - 16)),
    (INVALID, dict(xs=128, ys=128, b=PTR + (1 << 24) + 128 + 16)),
    (WORKSPACE, dict(xs=128, ys=128, b=PTR + (1 << 24) + 256 * 159 + 128)),
    (INVALID, dict(b=FAR, ws=FAR, wsb=1 << 20)),                 # workspace on the bias
    (INVALID, dict(ws=PTR + (1 << 24), wsb=1 << 20)),            # workspace on y
    (INVALID, dict(ws=PTR, wsb=1 << 20)),                        # on x
    (INVALID, dict(ws=PTR + (1 << 20), wsb=1 << 20)),            # on the weights
    (INVALID, dict(ws=FAR, wsb=1 << 20, init=FAR, num_slots=80)),
    (INVALID, dict(ws=FAR, wsb=1 << 20, fin=FAR, num_slots=80)),
    # sizes that pass 64 bits: a pool's, and the distance of the last rows
    (INVALID, dict(cu=(0,) * 81, D=(1 << 31) - 1, fin=FAR, num_slots=(1 << 31) - 1, b=FAR + (1 << 40))),
    (INVALID, dict(cu=tuple(i * ((1 << 30) - 1) for i in range(1024)), num_slots=1023, dt=F32,
                   xs=1 << 22, ys=(1 << 22) - 1)),
])
def test_short_conv_refuses_overlaps(lib, status, kw):
    a = dict(cu=CU80, num_slots=80)
    a.update(kw)
    assert conv(lib, **a) == status


@pytest.mark.parametrize("kw", [
    dict(y=PTR + (1 << 20)), dict(y=FAR + 64), dict(bias=PTR + (1 << 24)),
    dict(slots=PTR + (1 << 24)), dict(x=FAR + 128), dict(weight=FAR), dict(bias=FAR + 16),
    dict(slots=FAR + 4), dict(x=FAR, y=FAR),
    dict(state=PTR + (1 << 24) - 3 * 3 * 64 * 2 + 16), dict(y=PTR, x=PTR, bias=PTR + 64),
])
def test_short_conv_step_refuses_overlaps(lib, kw):
    a = dict(N=3, D=64, W=4, dt=BF16, x=PTR, xs=64, weight=PTR + (1 << 20), bias=None, act=0,
             state=FAR, slots=None, num_slots=3, y=PTR + (1 << 24), ys=64, stream=None)
    a.update(kw)
    assert lib.kda_short_conv_step(*a.values()) == INVALID


@pytest.mark.parametrize("store,load,kw", [
    (INVALID, INVALID, dict(c=PTR + 2 * 8 * 16 * 4 - 1)),            # codes on the states' end
    (INVALID, INVALID, dict(a=PTR + (1 << 24) + 2 * 8 * 16 - 4)),    # states on the codes' end
    (INVALID, INVALID, dict(sc=PTR + 64)),                           # scales on the states
    (INVALID, None, dict(sc=PTR + (1 << 24) + 128)),                 # scales on the codes
    (INVALID, None, dict(sc=PTR + (1 << 24) - 60)),
    (INVALID, None, dict(src=PTR + (1 << 24))),                      # tables on what is written
    (INVALID, None, dict(dst=PTR + (2 << 24) + 60)),
    (None, INVALID, dict(src=PTR + 4)),
    (None, INVALID, dict(dst=PTR)),
    (INVALID, INVALID, dict(num_a=(1 << 31) - 1, num_b=(1 << 31) - 1, R=1 << 31, n=0x7fffffff,
                            L=256)),
])
def test_state_cache_refuses_overlaps(lib, store, load, kw):
    a = dict(n=2, R=8, L=16, format=0, a=PTR, src=None, num_a=2, c=PTR + (1 << 24),
             sc=PTR + (2 << 24), dst=None, num_b=2)
    a.update(kw)
    if store is not None:
        assert lib.kda_state_store(a["n"], a["R"], a["L"], a["format"], a["a"], a["src"],
                                   a["num_a"], a["c"], a["sc"], a["dst"], a["num_b"], None) == store
    if load is not None:
        assert lib.kda_state_load(a["n"], a["R"], a["L"], a["format"], a["c"], a["sc"], a["src"],
                                  a["num_b"], a["a"], a["dst"], a["num_a"], None) == load


# (a cut of 7 pairs and no workspace: refused for that where the arguments pass)
POOL, WS, Y = PTR + (7 << 24), PTR + (8 << 24), PTR + (4 << 24)


@pytest.mark.parametrize("status,io,kw", [
    (WORKSPACE, {}, {}),
    (INVALID, dict(A=Y + 64), {}),
    (WORKSPACE, dict(A=Y + 4096 * 64 * 2), {}),
    (INVALID, dict(A=Y - 64 * 16 * 4 + 16), {}),
    (WORKSPACE, dict(A=Y - 64 * 16 * 4), {}),
    (INVALID, dict(D_skip=Y + 4096 * 64 * 2 - 16), {}),
    (INVALID, dict(delta_bias=Y), {}),
    (INVALID, dict(y_stride=128, delta_bias=Y + 128), {}),       # 256 bytes in a gap of 128
    (WORKSPACE, dict(y_stride=192, delta_bias=Y + 128), {}),     # in one of 256
    (INVALID, {}, dict(init=Y)),
    (INVALID, {}, dict(fin=Y + 4096 * 64 * 2 - 16)),
    (WORKSPACE, {}, dict(fin=Y + 4096 * 64 * 2)),
    (INVALID, {}, dict(slots=Y + 8)),
    (WORKSPACE, {}, dict(init=PTR)),                             # both only read
    (INVALID, {}, dict(fin=PTR)),                                # final state on x
    (INVALID, {}, dict(fin=PTR + (1 << 24))),                    # delta
    (INVALID, {}, dict(fin=PTR + (2 << 24))),                    # B
    (INVALID, {}, dict(fin=PTR + (3 << 24))),                    # C
    (INVALID, dict(z=POOL, z_stride=64), dict(fin=POOL)),
    (INVALID, {}, dict(fin=PTR + (5 << 24))),                    # A
    (INVALID, dict(D_skip=POOL + 16), dict(fin=POOL)),
    (INVALID, dict(delta_bias=POOL + 64), dict(init=POOL, fin=POOL)),
    (INVALID, {}, dict(slots=POOL + 4, fin=POOL)),
    (INVALID, {}, dict(ws=Y, wsb=1 << 24)),
    (INVALID, {}, dict(ws=PTR, wsb=1 << 24)),
    (INVALID, {}, dict(ws=PTR + (2 << 24), wsb=1 << 24)),
    (INVALID, {}, dict(ws=PTR + (5 << 24), wsb=1 << 24)),
    (INVALID, {}, dict(ws=POOL, wsb=1 << 24, init=POOL)),
    (INVALID, {}, dict(ws=POOL, wsb=1 << 24, fin=POOL)),
])
def test_selective_scan_refuses_overlaps(lib, status, io, kw):
    a = dict(init=None, fin=None, slots=None, ws=None, wsb=0)
    a.update(kw)
    keep, p = cu_ptr(0, 4096)
    blk = ssm_io(**io)
    assert lib.kda_selective_scan(1, p, 64, 16, 1, BF16, ctypes.byref(blk), a["init"], a["fin"],
                                  a["slots"], 1, 8, a["ws"], a["wsb"], None) == status


@pytest.mark.parametrize("io,kw", [
    (dict(A=Y), {}), (dict(D_skip=Y + 16), {}), (dict(delta_bias=Y), {}), ({}, dict(state=Y)),
    ({}, dict(slots=Y)), (dict(x=POOL), {}), (dict(delta=POOL + 64), {}), (dict(B=POOL), {}),
    (dict(C=POOL), {}), (dict(z=POOL, z_stride=64), {}), (dict(A=POOL), {}),
    (dict(D_skip=POOL), {}), (dict(delta_bias=POOL), {}), ({}, dict(slots=POOL)),
])
def test_selective_scan_step_refuses_overlaps(lib, io, kw):
    a = dict(state=POOL, slots=None)
    a.update(kw)
    blk = ssm_io(**io)
    assert lib.kda_selective_scan_step(3, 64, 16, 1, BF16, ctypes.byref(blk), a["state"],
                                       a["slots"], 3, None) == INVALID


# ---- binding ---------------------------------------------------------------------------

bf, f32 = torch.bfloat16, torch.float32


def z(*shape, dtype=bf):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("name,kw", [
    ("weight", dict(weight=z(63, 4))), ("weight", dict(weight=z(64, 4, dtype=f32))),
    ("weight", dict(weight=z(4, 64).t())), ("bias", dict(bias=z(63))),
    ("initial_state", dict(initial_state=z(2, 3, 64))),
    ("initial_state", dict(initial_state=z(1, 3, 64, dtype=f32))),
    ("final_state", dict(final_state=z(1, 2, 64))), ("y", dict(y=z(9, 64))),
    ("y", dict(y=z(64, 10).t())), ("slots", dict(slots=torch.zeros(1, dtype=torch.int64))),
    ("slots", dict(slots=torch.zeros(2, dtype=torch.int32))),
    ("cu_seqlens", dict(cu_seqlens=[0, 9])),
    ("one shape", dict(slots=torch.zeros(1, dtype=torch.int32), initial_state=z(4, 3, 64),
                       final_state=z(5, 3, 64))),
    ("HIP device", {}),
])
def test_short_conv_binding_rejects(name, kw):
    a = dict(x=z(10, 64), weight=z(64, 4))
    a.update(kw)
    with pytest.raises((ValueError, TypeError), match=name):
        kda.short_conv(a.pop("x"), a.pop("weight"), **a)


def test_short_conv_binding_rejects_types_and_activations():
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        kda.short_conv(z(10, 64, dtype=torch.float16), z(64, 4, dtype=torch.float16))
    with pytest.raises(ValueError, match="activation"):
        kda.short_conv(z(10, 64), z(64, 4), activation="relu")


@pytest.mark.parametrize("name,kw", [
    ("state", dict(state=z(3, 2, 64))), ("state", dict(state=z(3, 3, 64, dtype=f32))),
    ("weight", dict(weight=z(64, 4)[:, ::2])), ("HIP device", {}),
])
def test_short_conv_step_binding_rejects(name, kw):
    a = dict(state=z(3, 3, 64), x=z(3, 64), weight=z(64, 4))
    a.update(kw)
    with pytest.raises((ValueError, TypeError), match=name):
        kda.short_conv_step(**a)


def scan_args():
    return dict(x=z(10, 64), delta=z(10, 64), A=z(64, 5, dtype=f32), B=z(10, 2, 5), C=z(10, 2, 5))


@pytest.mark.parametrize("name,kw", [
    ("delta", dict(delta=z(10, 63))), ("delta", dict(delta=z(10, 64, dtype=f32))),
    ("A", dict(A=z(64, 5))), ("A", dict(A=z(5, 64, dtype=f32).t())), ("A must", dict(A=z(64, dtype=f32))),
    ("B", dict(B=z(10, 2, 4))), ("multiple", dict(B=z(10, 3, 5))), ("C", dict(C=z(10, 1, 5))),
    ("dense rows", dict(B=z(10, 5, 2).transpose(1, 2))),
    ("D must", dict(D=z(63, dtype=f32))), ("delta_bias", dict(delta_bias=z(64))),
    ("z must", dict(z=z(10, 32))), ("y must", dict(y=z(10, 64, dtype=f32))),
    ("initial_state", dict(initial_state=z(1, 64, 4, dtype=f32))),
    ("final_state", dict(final_state=z(1, 64, 5))), ("HIP device", {}),
])
def test_selective_scan_binding_rejects(name, kw):
    a = scan_args()
    a.update(kw)
    with pytest.raises((ValueError, TypeError), match=name):
        kda.selective_scan(**a)


@pytest.mark.parametrize("name,kw", [
    ("state", dict(state=z(9, 64, 5, dtype=f32))), ("state", dict(state=z(10, 64, 5))),
    ("slots", dict(slots=torch.zeros(9, dtype=torch.int32))), ("HIP device", {}),
])
def test_selective_scan_step_binding_rejects(name, kw):
    a = dict(scan_args(), state=z(10, 64, 5, dtype=f32))
    a.update(kw)
    with pytest.raises((ValueError, TypeError), match=name):
        kda.selective_scan_step(**a)


@pytest.mark.parametrize("name,kw", [
    ("int8 or", dict(codes=z(3, 4, 8, dtype=torch.uint8))),
    ("agree", dict(codes=z(3, 4, 7, dtype=torch.int8))),
    ("scales", dict(scales=z(3, 5, dtype=f32))), ("scales", dict(scales=z(3, 4))),
    ("state", dict(state=z(2, 4, 8))), ("contiguous", dict(state=z(2, 8, 4, dtype=f32).transpose(1, 2))),
    ("src", dict(src=torch.zeros(2, dtype=torch.int64))),
    ("dst", dict(src=torch.zeros(2, dtype=torch.int32), dst=torch.zeros(3, dtype=torch.int32))),
    ("HIP device", {}),
])
def test_state_cache_binding_rejects(name, kw):
    a = dict(state=z(2, 4, 8, dtype=f32), codes=z(3, 4, 8, dtype=torch.int8),
             scales=z(3, 4, dtype=f32))
    a.update(kw)
    with pytest.raises((ValueError, TypeError), match=name):
        kda.state_store(**a)
    with pytest.raises((ValueError, TypeError), match=name):
        kda.state_load(**a)


@pytest.mark.parametrize("items", [4, 100])
def test_state_cache_without_tables_moves_every_state_or_refuses(items):
    """Fewer slots than states: no state may be dropped, or left unread."""
    a = dict(state=z(items, 4, 8, dtype=f32), codes=z(3, 4, 8, dtype=torch.int8),
             scales=z(3, 4, dtype=f32))
    with pytest.raises(ValueError, match="3 slots"):
        kda.state_store(**a)
    with pytest.raises(ValueError, match="3 slots"):
        kda.state_load(**a)


def far(*shape, dtype=bf):
    """A shape without memory."""
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("call", [
    lambda n: kda.state_store(far(n, 1, dtype=f32), far(n, 1, dtype=torch.int8), far(n, dtype=f32)),
    lambda n: kda.state_load(far(n, 1, dtype=torch.int8), far(n, dtype=f32), far(n, 1, dtype=f32)),
    lambda n: kda.state_store(far(1, n, dtype=f32), far(1, n, dtype=torch.int8), far(1, dtype=f32)),
    lambda n: kda.state_store(far(4, 1, dtype=f32), far(n, 1, dtype=torch.int8), far(n, dtype=f32),
                              dst=far(4, dtype=torch.int32)),
    lambda n: kda.short_conv_step(far(n, 1, 1), far(n, 1), far(1, 2)),
    lambda n: kda.short_conv_step(far(n, 1, 1), far(3, 1), far(1, 2), slots=far(3, dtype=torch.int32)),
    lambda n: kda.short_conv_step(far(3, 1, 1), far(n, 1), far(1, 2), slots=far(n, dtype=torch.int32)),
    lambda n: kda.short_conv(far(3, 1), far(1, 2), initial_state=far(n, 1, 1),
                             slots=far(1, dtype=torch.int32)),
    lambda n: kda.selective_scan_step(far(n, 1, 1, dtype=f32), far(n, 1), far(n, 1),
                                      far(1, 1, dtype=f32), far(n, 1, 1), far(n, 1, 1)),
    lambda n: kda.selective_scan_step(far(n, 1, 1, dtype=f32), far(3, 1), far(3, 1),
                                      far(1, 1, dtype=f32), far(3, 1, 1), far(3, 1, 1),
                                      slots=far(3, dtype=torch.int32)),
    lambda n: kda.selective_scan(far(3, 1), far(3, 1), far(1, 1, dtype=f32), far(3, 1, 1),
                                 far(3, 1, 1), final_state=far(n, 1, 1, dtype=f32),
                                 slots=far(1, dtype=torch.int32)),
    lambda n: kda.selective_scan(far(3, 1), far(3, 1), far(1, 1, dtype=f32), far(3, 1, 1),
                                 far(3, 1, 1), split_hint=n),
])
def test_counts_past_31_bits_are_refused(call):
    """The library counts in 32 bits, and 2^32 + 5 must not pass for 5."""
    for n in ((1 << 31), (1 << 32) + 5):
        with pytest.raises(ValueError, match="2\\^31"):
            call(n)


# ---- the 64-bit forms -------------------------------------------------------------------

def test_conv_form_is_a_correlation():
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((9, 3)), rng.standard_normal((3, 4))
    y, _, fin = ref.conv(x, w, None, [0, 9], None, False, torch.float32)
    for d in range(3):
        full = np.convolve(x[:, d], w[d, ::-1])[:9]
        np.testing.assert_allclose(y[:, d], full, rtol=1e-12)
    np.testing.assert_array_equal(fin[0], x[6:])
    # two halves with the state between them are the whole
    y1, _, f1 = ref.conv(x[:2], w, None, [0, 2], None, True, torch.float32)
    y2, _, f2 = ref.conv(x[2:], w, None, [0, 7], f1, True, torch.float32)
    yw, _, fw = ref.conv(x, w, None, [0, 9], None, True, torch.float32)
    np.testing.assert_allclose(np.concatenate([y1, y2]), yw, rtol=1e-12)
    np.testing.assert_array_equal(f2, fw)


def test_scan_form_closed_cases():
    # one state, constant step: a geometric series
    T = 6
    one = np.ones((T, 1))
    A = np.array([[-0.5]])
    y, _, fin, _ = ref.scan(one, one, A, np.ones((T, 1, 1)), np.ones((T, 1, 1)), None, None, None,
                            False, [0, T], None, torch.float32)
    a = np.exp(-0.5)
    np.testing.assert_allclose(y[:, 0], [(1 - a ** (t + 1)) / (1 - a) for t in range(T)], rtol=1e-12)
    np.testing.assert_allclose(fin[0, 0, 0], y[-1, 0], rtol=1e-12)
    # no input: the state only decays
    h0 = np.array([[[2.0]]])
    y, _, fin, _ = ref.scan(0 * one, one, A, np.ones((T, 1, 1)), np.ones((T, 1, 1)), None, None, None,
                            False, [0, T], h0, torch.float32)
    np.testing.assert_allclose(fin[0, 0, 0], 2 * a ** T, rtol=1e-12)


def test_quantise_form_is_within_half_a_step():
    g = torch.Generator().manual_seed(3)
    x = torch.randn((50, 7, 33), generator=g)
    for kind, rel in ((torch.int8, 0.0), (torch.float8_e4m3fn, 2.0 ** -4)):
        codes, scale = ref.quantise(x, kind)
        back = codes.double() * scale.double()[..., None]
        # int8: half a step of the scale; e4m3: half a step of the value, or
        # half of its subnormal step 2^-9
        step = scale.double()[..., None] * (0.5 if kind == torch.int8 else 2.0 ** -10)
        tol = torch.maximum(step.expand_as(x), rel * x.double().abs()) * (1 + 2.0 ** -20)
        assert ((back - x.double()).abs() <= tol).all()
