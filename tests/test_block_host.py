"""CPU tests of the decayed attention, the block norm, beam selection and
state reordering: what the C ABI and the binding refuse (before anything
reaches a device), and the 64-bit forms of the GPU tests against closed
forms."""
import ctypes

import numpy as np
import pytest
import torch

import block_ref as ref
import gated_delta_rule_19_amd as kda
from gated_delta_rule_19_amd import _native as nat

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
F32, BF16 = nat.KDA_F32, nat.KDA_BF16
PTR = 0x7F0000000000  # never dereferenced: every call below is refused, or does nothing
M = 1 << 24


@pytest.fixture(scope="module")
def lib():
    return nat.load()


def cu_ptr(*bounds):
    a = np.array(bounds, dtype=np.int64)
    return a, a.ctypes.data_as(ctypes.POINTER(ctypes.c_int64))


# ---- C ABI: decayed attention ----------------------------------------------------

def decay_io(**kw):
    a = dict(q=PTR, k=PTR + M, v=PTR + 2 * M, g=PTR + 3 * M, o=PTR + 4 * M, q_stride=64, k_stride=64,
             v_stride=128, g_stride=4, o_stride=128, Hq=4, Hk=4, Hv=4, dk=16, dv=32, scale=1.0)
    a.update(kw)
    return nat.DecayIo(**a)


BAD_IO = [
    (UNSUPPORTED, dict(dk=257)), (UNSUPPORTED, dict(dv=257)), (INVALID, dict(dk=0)), (INVALID, dict(dv=0)),
    (INVALID, dict(Hq=3)), (INVALID, dict(Hk=0)), (INVALID, dict(Hv=8)), (INVALID, dict(Hk=-4)),
    (INVALID, dict(q=None)), (INVALID, dict(k=None)), (INVALID, dict(v=None)), (INVALID, dict(g=None)),
    (INVALID, dict(o=None)), (INVALID, dict(q=PTR + 1)), (INVALID, dict(g=PTR + 3 * M + 2)),
    (INVALID, dict(q_stride=63)), (INVALID, dict(k_stride=63)), (INVALID, dict(v_stride=127)),
    (INVALID, dict(o_stride=127)), (INVALID, dict(g_stride=3)), (INVALID, dict(g_stride=-4)),
    (INVALID, dict(q_stride=(1 << 22) + 1)), (INVALID, dict(g_stride=(1 << 22) + 1)),
    (INVALID, dict(o=PTR)), (INVALID, dict(o=PTR + M + 2)), (INVALID, dict(o=PTR + 3 * M)),
    (INVALID, dict(o=PTR + 2 * M, o_stride=256)),      # other pitch: ranges meet
    (INVALID, dict(o=PTR + 3 * M - 8, g_stride=0)),    # on the decays of all tokens
]


@pytest.mark.parametrize("status,io,kw", [(s, d, {}) for s, d in BAD_IO] + [
    (UNSUPPORTED, {}, dict(dt=2)),
    (INVALID, {}, dict(H=0)),
    (INVALID, {}, dict(split=-1)),
    (INVALID, {}, dict(cu=(0, 3, 2))),
    (INVALID, {}, dict(cu=(1, 5))),
    (INVALID, {}, dict(cu=(0, 1 << 30))),
    (INVALID, {}, dict(fin=PTR + 5 * M + 4)),
    (INVALID, {}, dict(init=PTR + 5 * M + 8)),
    (INVALID, {}, dict(fin=PTR + 5 * M, num_slots=0)),
    (INVALID, {}, dict(init=PTR + 5 * M, slots=PTR + 6 * M, num_slots=-1)),
    (INVALID, {}, dict(init=PTR + 5 * M, fin=PTR + 5 * M + 64)),
    (INVALID, {}, dict(fin=PTR)),
    (INVALID, {}, dict(init=PTR + 4 * M)),             # o on the initial state
    (INVALID, {}, dict(slots=PTR + 1)),
    (INVALID, {}, dict(slots=PTR + 4 * M)),            # o on the slots
    (WORKSPACE, {}, dict(cu=(0, 4096), split=8, wsb=0)),
    (WORKSPACE, {}, dict(cu=(0, 4096), split=8, ws=None)),
    (WORKSPACE, {}, dict(cu=tuple(range(80)), ws=None, num_slots=79)),
    (INVALID, {}, dict(cu=(0, 4096), split=8, ws=PTR + 8 * M + 64)),
    (INVALID, {}, dict(cu=(0, 4096), split=8, ws=PTR + 4 * M)),   # the workspace on o
])
def test_decay_attention_refuses(lib, status, io, kw):
    a = dict(cu=(0, 5), H=4, dt=BF16, init=None, fin=None, slots=None, num_slots=1, split=0, ws=PTR + 8 * M,
             wsb=M)
    a.update(kw)
    keep, p = cu_ptr(*a["cu"])
    assert lib.kda_decay_attention(len(a["cu"]) - 1, p, a["H"], a["dt"], ctypes.byref(decay_io(**io)), a["init"],
                                   a["fin"], a["slots"], a["num_slots"], a["split"], a["ws"], a["wsb"],
                                   None) == status


def test_decay_attention_of_nothing(lib):
    keep, p = cu_ptr(0)
    none = dict(q=None, k=None, v=None, g=None, o=None)
    assert lib.kda_decay_attention(0, p, 4, F32, ctypes.byref(decay_io(**none)), None, None, None, 0, 0, None, 0,
                                   None) == OK
    assert lib.kda_decay_attention(0, p, 4, F32, None, None, None, None, 0, 0, None, 0, None) == INVALID
    assert lib.kda_decay_attention_step(0, 4, F32, ctypes.byref(decay_io(**none)), None, None, 0, None) == OK


def test_decay_attention_workspace(lib):
    keep, p = cu_ptr(0, 4096)
    size = lib.kda_decay_attention_workspace_size
    assert size(1, p, 4, 64, 64, BF16, 1) == 0
    for dt, dk, dv in ((BF16, 64, 64), (F32, 128, 100), (BF16, 100, 129), (F32, 256, 1)):
        # seven pairs more: a state in whole tiles and a double a head each
        assert size(1, p, 4, dk, dv, dt, 8) >= 7 * 4 * (dk * dv * 4 + 8)
    assert size(1, p, 4, 257, 64, BF16, 8) == 0 and size(1, p, 0, 64, 64, BF16, 8) == 0
    assert size(1, p, 4, 64, 64, 5, 8) == 0 and size(1, p, 4, 64, 64, BF16, -1) == 0
    keep2, p2 = cu_ptr(0, -5)
    assert size(1, p2, 4, 64, 64, BF16, 0) == 0
    keep3, p3 = cu_ptr(*range(66))
    assert size(65, p3, 4, 64, 64, BF16, 1) > 0  # the sequences' table
    # one long sequence of one head is cut by itself
    keep4, p4 = cu_ptr(0, 1 << 20)
    assert size(1, p4, 1, 128, 128, BF16, 0) > 0 and size(1, p4, 1, 128, 128, F32, 0) > 0


def test_a_long_sequence_among_many_short_ones_is_cut(lib):
    """... and a batch of many equal ones is not."""
    size = lib.kda_decay_attention_workspace_size
    keep, p = cu_ptr(*np.concatenate([[0], np.cumsum([20000] + [30] * 300)]))
    keep2, p2 = cu_ptr(*range(0, 64 * 501, 500))
    for dt in (F32, BF16):
        assert size(301, p, 2, 128, 128, dt, 0) >= size(301, p, 2, 128, 128, dt, 8)
        assert size(64, p2, 16, 128, 128, dt, 0) == 0


@pytest.mark.parametrize("status,io,kw", [(s, d, {}) for s, d in BAD_IO] + [
    (UNSUPPORTED, {}, dict(dt=9)), (INVALID, {}, dict(rows=-1)), (INVALID, {}, dict(state=None)),
    (INVALID, {}, dict(state=PTR + 5 * M + 8)), (INVALID, {}, dict(num_slots=2)),
    (INVALID, {}, dict(state=PTR)), (INVALID, {}, dict(slots=PTR + 2)),
    (INVALID, {}, dict(slots=PTR + 5 * M)),            # the table in the states
    (INVALID, {}, dict(rows=1 << 24, num_slots=1 << 24)),  # (the outputs would meet)
])
def test_decay_attention_step_refuses(lib, status, io, kw):
    a = dict(rows=3, H=4, dt=BF16, state=PTR + 5 * M, slots=None, num_slots=3)
    a.update(kw)
    assert lib.kda_decay_attention_step(a["rows"], a["H"], a["dt"], ctypes.byref(decay_io(**io)), a["state"],
                                        a["slots"], a["num_slots"], None) == status


# ---- C ABI: block norm --------------------------------------------------------------

@pytest.mark.parametrize("status,io,kw", [
    (UNSUPPORTED, {}, dict(dt=2)), (UNSUPPORTED, {}, dict(D=65537)), (INVALID, {}, dict(D=0)),
    (INVALID, {}, dict(rows=-1)),
    (UNSUPPORTED, dict(residual_dt=7), {}),
    (INVALID, dict(y=None, residual_out=None), {}),
    (INVALID, dict(weight=None), {}),
    (INVALID, dict(x=None), {}), (INVALID, dict(x=PTR + 1), {}), (INVALID, dict(x_stride=63), {}),
    (INVALID, dict(gate_stride=63), {}), (INVALID, dict(residual=PTR + 2 * M + 2), {}),
    (INVALID, dict(residual_stride=63), {}), (INVALID, dict(residual_out_stride=63), {}),
    (INVALID, dict(y_stride=63), {}), (INVALID, dict(y_stride=(1 << 22) + 1), {}),
    (INVALID, dict(weight=PTR + 5 * M + 4), {}), (INVALID, dict(scale=PTR + 6 * M + 8), {}),
    (INVALID, dict(post_weight=PTR + 7 * M + 4), {}),
    (INVALID, dict(y=PTR + 2), {}),                                    # y beside x by one element
    (INVALID, dict(y=PTR, x_stride=128), {}),                          # x's place, another stride
    (INVALID, dict(residual_out=PTR), {}),                             # x's place, another type
    (INVALID, dict(residual_out=PTR + 2 * M + 4), {}),
    (INVALID, dict(y=PTR + 2 * M), {}),                                # y on the residual
    (INVALID, dict(y=PTR + 5 * M), {}),                                # y on the weight
    (INVALID, dict(y=PTR + 3 * M), {}),                                # y on residual_out
    (INVALID, dict(residual_out=PTR + 6 * M), {}),                     # on the scale
])
def test_block_norm_refuses(lib, status, io, kw):
    a = dict(rows=3, D=64, dt=BF16)
    a.update(kw)
    b = dict(x=PTR, gate=PTR + M, residual=PTR + 2 * M, residual_out=PTR + 3 * M, y=PTR + 4 * M, x_stride=64,
             gate_stride=64, residual_stride=64, residual_out_stride=64, y_stride=64, post_weight=PTR + 7 * M,
             weight=PTR + 5 * M, scale=PTR + 6 * M, post_eps=1e-6, eps=1e-6, scale_all=1.0, residual_dt=F32)
    b.update(io)
    assert lib.kda_block_norm(a["rows"], a["D"], a["dt"], ctypes.byref(nat.NormIo(**b)), None) == status


def test_block_norm_of_nothing(lib):
    assert lib.kda_block_norm(0, 64, BF16, ctypes.byref(nat.NormIo()), None) == OK
    assert lib.kda_block_norm(1, 64, BF16, None, None) == INVALID


# ---- C ABI: beams -------------------------------------------------------------------

def beam(lib, **kw):
    a = dict(B=2, W=4, V=100, K=4, dt=F32, logits=PTR, stride=100, scores=PTR + M, finished=PTR + 2 * M, eos=3,
             order=0, out=PTR + 3 * M, parents=PTR + 4 * M, tokens=PTR + 5 * M, done=PTR + 6 * M, ws=PTR + 7 * M,
             wsb=M)
    a.update(kw)
    return lib.kda_beam_select(*a.values(), None)


@pytest.mark.parametrize("status,kw", [
    (UNSUPPORTED, dict(dt=4)), (UNSUPPORTED, dict(W=65)), (UNSUPPORTED, dict(K=65)), (INVALID, dict(W=0)),
    (INVALID, dict(K=0)), (INVALID, dict(V=0)), (INVALID, dict(B=-1)), (INVALID, dict(W=1, V=3)),
    (INVALID, dict(order=2)), (INVALID, dict(order=1, K=3)), (INVALID, dict(eos=-2)), (INVALID, dict(eos=100)),
    (INVALID, dict(eos=-1)),                            # finished beams without a token for them
    (INVALID, dict(logits=None)), (INVALID, dict(logits=PTR + 2)), (INVALID, dict(stride=99)),
    (INVALID, dict(stride=(1 << 31) + 1)), (INVALID, dict(scores=None)), (INVALID, dict(scores=PTR + M + 1)),
    (INVALID, dict(out=None)), (INVALID, dict(parents=None)), (INVALID, dict(tokens=None)),
    (INVALID, dict(done=None)), (INVALID, dict(out=PTR + 3 * M + 2)), (INVALID, dict(tokens=PTR + 5 * M + 1)),
    (INVALID, dict(out=PTR)), (INVALID, dict(out=PTR + M)), (INVALID, dict(done=PTR + 2 * M)),
    (INVALID, dict(parents=PTR + 3 * M + 28)), (INVALID, dict(ws=PTR)), (INVALID, dict(ws=PTR + 7 * M + 8)),
    (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(wsb=8)),
])
def test_beam_select_refuses(lib, status, kw):
    assert beam(lib, **kw) == status


def test_beam_select_of_nothing(lib):
    assert beam(lib, B=0, logits=None, scores=None, out=None, ws=None) == OK
    size = lib.kda_beam_select_workspace_size
    assert size(0, 4, 100, 4, F32) == 0 and size(2, 65, 100, 4, F32) == 0 and size(2, 4, 100, 4, 7) == 0
    # a part's K candidates and its sum, for 16 KB of logits each
    assert size(2, 4, 40960, 8, F32) >= 2 * 4 * 10 * (8 * 8 + 16)
    assert size(2, 4, 40960, 8, BF16) >= 2 * 4 * 5 * (8 * 8 + 16)


def reorder(lib, groups=2, K=3, parents=PTR, slots=None, states=(PTR + M, PTR + 2 * M), size=(16, 8), held=(6, 6),
            n=None):
    count = len(states)
    return lib.kda_state_reorder(groups, K, parents, slots, count if n is None else n,
                                 (ctypes.c_void_p * max(1, count))(*states),
                                 (ctypes.c_int64 * max(1, count))(*size),
                                 (ctypes.c_int32 * max(1, count))(*held), None)


@pytest.mark.parametrize("status,kw", [
    (UNSUPPORTED, dict(K=65)), (UNSUPPORTED, dict(n=33)), (INVALID, dict(K=0)), (INVALID, dict(groups=-1)),
    (INVALID, dict(n=-1)), (INVALID, dict(parents=None)), (INVALID, dict(parents=PTR + 1)),
    (INVALID, dict(slots=PTR + 2)), (INVALID, dict(size=(-1, 8))), (INVALID, dict(size=((1 << 46) + 1, 8))),
    (INVALID, dict(held=(5, 6))), (INVALID, dict(held=(-1, 6), slots=PTR + 4 * M)),
    (INVALID, dict(states=(None, PTR))), (INVALID, dict(states=(PTR + M, PTR + M + 95))),
    (INVALID, dict(states=(PTR, PTR + 2 * M))), (INVALID, dict(slots=PTR + 2 * M + 8)),
    (INVALID, dict(groups=1 << 30, K=64, held=(1 << 30,) * 2)),
])
def test_state_reorder_refuses(lib, status, kw):
    assert reorder(lib, **kw) == status


def test_state_reorder_of_nothing(lib):
    assert reorder(lib, groups=0, parents=None) == OK
    assert reorder(lib, states=(), size=(), held=(), parents=None) == OK
    assert reorder(lib, size=(0, 0), states=(None, None)) == OK
    assert reorder(lib, K=1, held=(2, 2)) == OK                       # one row a group: nothing to move
    assert reorder(lib, K=1, held=(1, 2)) == INVALID


# ---- binding ------------------------------------------------------------------------

def z(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("kw", [
    dict(q=z(5, 16)), dict(g=z(5, 4, 1)), dict(k=z(4, 2, 16)), dict(v=z(5, 3, 32)), dict(k=z(5, 2, 8)),
    dict(q=z(5, 2, 16, dtype=torch.float16)), dict(k=z(5, 2, 16, dtype=torch.bfloat16)),
    dict(g=z(5, 4, dtype=torch.bfloat16)), dict(g=z(4, 4)), dict(o=z(5, 4, 16)), dict(q=z(5, 2, 32)[:, :, ::2]),
    dict(cu_seqlens=[0, 4]), dict(cu_seqlens=[1, 5]), dict(initial_state=z(2, 4, 16, 32)),
    dict(initial_state=z(1, 4, 16, 32, dtype=torch.bfloat16)), dict(final_state=z(1, 4, 32, 16)),
    dict(slots=torch.zeros(2, dtype=torch.int32)), dict(slots=torch.zeros(1, dtype=torch.int64)),
    dict(workspace=z(4)),
])
def test_decay_attention_binding_refuses(kw):
    a = dict(q=z(5, 2, 16), k=z(5, 2, 16), v=z(5, 4, 32), g=z(5, 4))
    a.update(kw)
    with pytest.raises((ValueError, TypeError)):
        kda.decay_attention(**a)


@pytest.mark.parametrize("kw", [
    dict(state=z(4, 4, 16, 32)), dict(state=z(5, 4, 16, 32, dtype=torch.bfloat16)),
    dict(state=z(5, 4, 32, 16).transpose(2, 3)), dict(o=z(5, 4, 31)), dict(slots=torch.zeros(4, dtype=torch.int32)),
    dict(v=z(5, 3, 32)),
])
def test_decay_attention_step_binding_refuses(kw):
    a = dict(state=z(5, 4, 16, 32), q=z(5, 2, 16), k=z(5, 2, 16), v=z(5, 4, 32), g=z(5, 4))
    a.update(kw)
    with pytest.raises((ValueError, TypeError)):
        kda.decay_attention_step(**a)


@pytest.mark.parametrize("kw", [
    dict(x=z(64)), dict(x=z(3, 64, dtype=torch.float16)), dict(gate=z(3, 63)), dict(residual=z(2, 64)),
    dict(weight=z(63)), dict(weight=z(64, dtype=torch.bfloat16)), dict(post_weight=z(65)), dict(scale=z(63)),
    dict(y=z(3, 64), weight=None), dict(y=z(3, 64, dtype=torch.bfloat16)), dict(residual_out=z(3, 65)),
    dict(residual=z(3, 64, dtype=torch.float64)), dict(x=z(3, 128)[:, ::2]),
    dict(residual=z(3, 64), residual_out=z(3, 64, dtype=torch.bfloat16)),
])
def test_block_norm_binding_refuses(kw):
    a = dict(x=z(3, 64), weight=z(64))
    a.update(kw)
    with pytest.raises((ValueError, TypeError)):
        kda.block_norm(**a)


@pytest.mark.parametrize("kw", [
    dict(logits=z(4, 100)), dict(logits=z(2, 4, 100, dtype=torch.float16)), dict(scores=z(2, 3)),
    dict(scores=z(2, 4, dtype=torch.bfloat16)), dict(finished=torch.zeros(2, 4, dtype=torch.uint8), eos=0),
    dict(order="best"), dict(logits=z(2, 4, 200)[:, :, ::2]), dict(logits=z(4, 2, 100).transpose(0, 1)),
])
def test_beam_select_binding_refuses(kw):
    a = dict(logits=z(2, 4, 100), scores=z(2, 4))
    a.update(kw)
    with pytest.raises((ValueError, TypeError)):
        kda.beam_select(**a)


@pytest.mark.parametrize("kw", [
    dict(states=[z(6, 4)] * 33), dict(parents=torch.zeros(2, 3, dtype=torch.int64)),
    dict(parents=torch.zeros(6, dtype=torch.int32)), dict(states=z(5, 4)), dict(states=z(4, 6).t()),
    dict(slots=torch.zeros(3, 2, dtype=torch.int32)),
    dict(parents=torch.zeros(3, 2, dtype=torch.int32).t()),
])
def test_state_reorder_binding_refuses(kw):
    a = dict(states=z(6, 4), parents=torch.zeros(2, 3, dtype=torch.int32))
    a.update(kw)
    with pytest.raises((ValueError, TypeError)):
        kda.state_reorder(**a)


# ---- the 64-bit forms against closed forms --------------------------------------------

def test_attention_form_against_the_sum_over_tokens():
    """o_t = scale sum_j exp(g_{j+1} + .. + g_t) (q_t . k_j) v_j, and the same
    with exp(g_1 + .. + g_t) S_0 for a state that enters."""
    g = torch.Generator().manual_seed(1)
    T, H, dk, dv = 9, 4, 3, 5
    q, k, v = (torch.randn(T, h, d, generator=g, dtype=torch.float64) for h, d in ((2, dk), (1, dk), (4, dv)))
    gl = -torch.rand(T, H, generator=g, dtype=torch.float64)
    init = torch.randn(2, H, dk, dv, generator=g, dtype=torch.float64)
    cu = [0, 4, 9]
    o, otol, fin, _ = ref.decay_attention(q, k, v, gl, 0.5, cu, init, torch.float32)
    for n in range(2):
        for h in range(H):
            for t in range(cu[n], cu[n + 1]):
                run = torch.exp(gl[cu[n]:t + 1, h].sum()) * init[n, h]
                for j in range(cu[n], t + 1):
                    run = run + torch.exp(gl[j + 1:t + 1, h].sum()) * torch.outer(k[j, 0], v[j, h])
                want = 0.5 * q[t, h // 2] @ run
                assert (o[t, h] - want).abs().max() < 1e-12
            assert (fin[n, h] - run).abs().max() < 1e-12
    assert (otol > 0).all()


def test_norm_form_in_closed_form():
    x = torch.full((1, 4), 3.0, dtype=torch.float64)
    one = torch.ones(4, dtype=torch.float64)
    r, _, y, _ = ref.block_norm(x, 2 * one, 0.0, 5 * x, 2.0, 0 * x, one, 0.0, torch.float32, torch.float32)
    assert torch.allclose(r, 15 + torch.ones_like(x)) and torch.allclose(y, 2 * torch.ones_like(x))
    r, _, y, _ = ref.block_norm(x, None, 0.0, None, 2.0, None, None, 0.0, torch.float32, torch.float32)
    assert torch.equal(r, 2 * x) and y is None


def test_beam_form_by_hand():
    ninf = -float("inf")
    logits = torch.tensor([[[0.0, 0.0], [np.log(3.0), 0.0], [ninf, ninf]]])
    s, p, t, d = ref.beam_select(logits, torch.tensor([[0.0, 0.0, 5.0]]), 6, None, -1)
    assert p[0].tolist() == [1, 0, 0, 1, 2, 2] and t[0].tolist() == [0, 0, 1, 1, 0, 1]
    assert torch.allclose(s[0, :4].exp(), torch.tensor([0.75, 0.5, 0.5, 0.25], dtype=torch.float64))
    assert torch.isinf(s[0, 4:]).all() and not d.any()
    s, p, t, d = ref.beam_select(logits, torch.tensor([[0.0, 0.0, -0.1]]), 3, torch.tensor([[False, False, True]]), 1,
                                 "rows")
    assert p[0].tolist() == [0, 1, 2] and t[0].tolist() == [0, 0, 1] and d[0].tolist() == [False, False, True]


def test_reorder_form_by_hand():
    state = torch.arange(6.0).view(6, 1)
    parents = torch.tensor([[1, 0, 0], [2, 7, -1]], dtype=torch.int32)
    assert ref.reorder(state, parents).view(-1).tolist() == [1, 0, 0, 5, 4, 5]
    slots = torch.tensor([[5, 4, 3], [2, 1, 9]], dtype=torch.int32)
    assert ref.reorder(state, parents, slots).view(-1).tolist() == [0, 1, 2, 5, 5, 4]


def test_workspace_covers_rows_at_any_place(lib):
    """A prompt that runs uncut where its rows start at multiples of 16 bytes,
    and in segments where they do not: what is asked for holds both."""
    keep, p = cu_ptr(0, 1024)
    size = lib.kda_decay_attention_workspace_size
    assert size(1, p, 32, 128, 128, BF16, 0) >= size(1, p, 32, 128, 128, BF16, 3) > 0
    assert size(1, p, 32, 128, 128, BF16, 1) == 0
