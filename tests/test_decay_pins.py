"""CPU checks of the decay attention, the group norm and AdamW: the fp64 oracle
against what the operators mean, and refusals of the C ABI before any launch."""
import ctypes
import math

import numpy as np
import pytest

from oracle import decay as ref
from oracle import q8 as ref8
from oracle import train as ref_t
from sub_linear_memory_gb300 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    from sub_linear_memory_gb300 import binding

    return binding.raw()


def draw(seed=0, t=11, hq=4, hk=2, dk=3, dv=5, n=3):
    r = np.random.RandomState(seed)
    q, k, v, do = (r.randn(t, h, w) for h, w in ((hq, dk), (hk, dk), (hk, dv), (hq, dv)))
    return q, k, v, do, -r.rand(hk), r.randn(n, hk, dk, dv), r.randn(n, hk, dk, dv)


CU = [0, 4, 4, 10]


def test_recurrence_is_the_decayed_sum():
    q, k, v, _, g, s0, _ = draw()
    o, ends = ref.forward(q, k, v, g, CU, 0.7, s0)
    for i, (a, b) in enumerate(zip(CU, CU[1:])):
        for h in range(4):
            lam = math.exp(g[h // 2])
            for t in range(a, b):
                y = lam ** (t + 1 - a) * q[t, h] @ s0[i, h // 2]
                for j in range(a, t + 1):
                    y = y + lam ** (t - j) * (q[t, h] @ k[j, h // 2]) * v[j, h // 2]
                assert np.allclose(o[t, h], 0.7 * y, rtol=1e-12, atol=1e-12)
    assert np.array_equal(ends[1], s0[1])  # an empty sequence hands its state on
    assert not o[10].any()


def test_gradients_against_differences():
    q, k, v, do, g, s0, g_in = draw(1)

    def loss(q, k, v, s0):
        o, ends = ref.forward(q, k, v, g, CU, 0.7, s0)
        return (o * do).sum() + (ends * g_in).sum()

    grads = ref.backward(q, k, v, g, CU, do, 0.7, s0, g_in)
    args = [q, k, v, s0]
    r = np.random.RandomState(2)
    for i, grad in enumerate(grads):
        for _ in range(12):
            at = tuple(r.randint(n) for n in args[i].shape)
            ends = []
            for step in (1e-5, -1e-5):
                moved = [x.copy() for x in args]
                moved[i][at] += step
                ends.append(loss(*moved))
            assert abs((ends[0] - ends[1]) / 2e-5 - grad[at]) <= 1e-8 * (1 + abs(grad[at]))


def test_group_norm_gradients_against_differences():
    r = np.random.RandomState(3)
    x, z, dy = r.randn(3, 3, 12)
    gamma, beta = r.randn(2, 12)
    grads = ref_t.group_norm_bwd(dy, x, gamma, beta, 3, z, 1e-3)
    args = [x, z, gamma, beta]
    for i, grad in enumerate(grads):
        for at in np.ndindex(args[i].shape):
            ends = []
            for step in (1e-5, -1e-5):
                moved = [a.copy() for a in args]
                moved[i][at] += step
                ends.append((dy * ref_t.group_norm(moved[0], moved[2], moved[3], 3, moved[1], 1e-3)).sum())
            assert abs((ends[0] - ends[1]) / 2e-5 - grad[at]) <= 1e-8 * (1 + abs(grad[at]))


def test_rounding_at_random_is_to_a_neighbour_and_right_in_the_mean():
    r = np.random.RandomState(4)
    x = r.randn(128) * np.exp(3 * r.randn(128))
    total = np.zeros(128)
    draws = 4096
    for bits in np.arange(draws) * (65536 // draws):
        held, scales = ref_t.held_at_random(x, np.full(128, bits))
        total += held
        e = 2.0 ** (int(scales[0]) - 127)
        a, c = np.abs(x) / e, np.abs(held) / e
        lo = np.searchsorted(ref8.E4M3, a, side="right") - 1
        assert np.all((c == ref8.E4M3[lo]) | (c == ref8.E4M3[np.minimum(lo + 1, 126)]))
    # evenly spread bits: the mean is off by at most one part in 4096 of a step of 1/8
    step = np.maximum(np.abs(x) / 8, e * 2.0 ** -9)
    assert np.all(np.abs(total / draws - x) <= step / draws * 1.001)


def test_a_step_of_adamw_by_hand():
    # first step: m / (1 - b1) = g, sqrt(v / (1 - b2)) = |g|
    m, v = ref_t.moments(np.array([-3.0]), np.zeros(1), np.zeros(1), (0.9, 0.99))
    p = ref_t.weight(np.array([2.0]), m, v, 1, 0.1, (0.9, 0.99), 0.0, 0.5)
    assert np.allclose(p, 2.0 + 0.1 - 0.1 * 0.5 * 2.0, rtol=1e-14)


# ---- refusals ----------------------------------------------------------------

def shape(**kw):
    from sub_linear_memory_gb300 import decay

    s = dict(tokens=8, seqs=2, heads=2, groups=2, dk=16, dv=8, places=2, q_row=64, k_row=32, v_row=16, o_row=32,
             dq_row=64, dk_row=32, dv_row=16)
    s.update(kw)
    return decay.Shape(*(s[n] for n, _ in decay.Shape._fields_))


P = [ctypes.c_void_p(4096 * (i + 1)) for i in range(16)]
BIG = 1 << 40


def fwd(lib, s, cu=P[4], state=P[5], slots=None, q=P[0], g=P[3], o=P[6], ws=P[7], n=BIG):
    return lib.slim_decay_fwd(q, P[1], P[2], g, cu, state, state, slots, o, ctypes.byref(s), 1.0, ws, n, None)


@pytest.mark.parametrize("want, kw, args", [
    (1, dict(tokens=-1), {}), (1, dict(seqs=-1), {}), (1, dict(groups=0), {}), (1, dict(dk=0), {}), (1, dict(dv=0), {}),
    (2, dict(dk=257), {}), (2, dict(dv=300), {}), (2, dict(groups=65), {}),
    (1, dict(q_row=63), {}), (1, dict(k_row=31), {}), (1, dict(v_row=15), {}), (1, dict(o_row=31), {}),
    (1, dict(places=3), {}), (1, dict(tokens=9), dict(cu=None)), (1, {}, dict(q=None)), (1, {}, dict(g=None)),
    (1, {}, dict(o=P[1])), (2, {}, dict(q=ctypes.c_void_p(4097))), (2, {}, dict(cu=ctypes.c_void_p(4098))),
    (2, {}, dict(state=ctypes.c_void_p(4098))), (3, {}, dict(ws=None)), (3, {}, dict(n=100)),
    (2, {}, dict(ws=ctypes.c_void_p(4096 + 128)))])
def test_attn_refuses(lib, want, kw, args):
    assert fwd(lib, shape(**kw), **args) == want


def bwd(lib, s, d_o=P[5], g_in=P[7], g_out=P[8], outs=(P[9], P[10], P[11]), n=BIG):
    return lib.slim_decay_bwd(P[0], P[1], P[2], P[3], P[4], d_o, P[6], g_in, g_out, *outs, ctypes.byref(s), 1.0, P[12], n, None)


@pytest.mark.parametrize("want, kw, args", [
    (1, {}, dict(d_o=None)), (1, {}, dict(g_out=P[7])), (1, {}, dict(g_out=P[6])), (1, {}, dict(outs=(P[9], P[9], P[11]))),
    (1, {}, dict(outs=(P[5], P[10], P[11]))), (1, dict(dq_row=63), {}), (1, dict(dk_row=31), {}), (1, dict(dv_row=15), {}),
    (1, dict(places=1), {}), (3, {}, dict(n=8)), (2, {}, dict(outs=(ctypes.c_void_p(4097), P[10], P[11])))])
def test_attn_bwd_refuses(lib, want, kw, args):
    assert bwd(lib, shape(**kw), **args) == want


@pytest.mark.parametrize("want, kw, state, slots", [
    (1, {}, P[4], None), (1, dict(places=8), None, None), (2, dict(dk=257, places=8), P[4], None),
    (1, dict(q_row=60, places=8), P[4], None), (1, dict(tokens=-3), P[4], P[5]), (2, {}, ctypes.c_void_p(4097), P[5])])
def test_step_refuses(lib, want, kw, state, slots):
    assert lib.slim_decay_step(P[0], P[1], P[2], P[3], state, slots, P[6], ctypes.byref(shape(**kw)), 1.0, None) == want


def test_nothing_to_do(lib):
    assert fwd(lib, shape(seqs=0, places=0), q=None, ws=None) == 0
    assert fwd(lib, shape(heads=0), q=None, ws=None) == 0
    assert lib.slim_decay_step(*[None] * 7, ctypes.byref(shape(tokens=0, places=0)), 1.0, None) == 0
    assert lib.slim_decay_workspace_bytes(ctypes.byref(shape(tokens=8000)), 0, 1) > lib.slim_decay_workspace_bytes(
        ctypes.byref(shape(tokens=0)), 0, 0) > 0
    assert lib.slim_decay_workspace_bytes(ctypes.byref(shape(dk=0)), 0, 0) == 0
    assert lib.slim_decay_workspace_bytes(ctypes.byref(shape(tokens=9)), 1, 0) == 0


@pytest.mark.parametrize("want, rows, cols, groups, eps, x, gate, y", [
    (1, -1, 8, 2, 0.0, P[0], P[3], P[4]), (1, 4, 0, 1, 0.0, P[0], P[3], P[4]), (1, 4, 9, 2, 0.0, P[0], P[3], P[4]),
    (1, 4, 8, 0, 0.0, P[0], P[3], P[4]), (2, 4, 16392, 2, 0.0, P[0], P[3], P[4]), (1, 4, 8, 2, -1.0, P[0], P[3], P[4]),
    (1, 4, 8, 2, math.nan, P[0], P[3], P[4]), (1, 4, 8, 2, 0.0, None, P[3], P[4]), (1, 4, 8, 2, 0.0, P[0], P[3], P[0]),
    (1, 4, 8, 2, 0.0, P[0], P[4], P[4]), (2, 4, 8, 2, 0.0, ctypes.c_void_p(4097), P[3], P[4]), (0, 0, 8, 2, 0.0, None, None, None)])
def test_group_norm_refuses(lib, want, rows, cols, groups, eps, x, gate, y):
    from sub_linear_memory_gb300 import norm  # noqa: F401  (argument types)

    assert lib.slim_group_norm(x, P[1], P[2], gate, cols, eps, y, rows, cols, groups, None) == want


@pytest.mark.parametrize("want, dx, dgate, gate, ws, n", [
    (1, P[5], None, P[4], P[9], BIG), (1, P[5], P[6], None, P[9], BIG), (1, P[0], P[6], P[4], P[9], BIG),
    (1, P[5], P[5], P[4], P[9], BIG), (3, P[5], P[6], P[4], None, 0), (3, P[5], P[6], P[4], P[9], 8),
    (2, P[5], P[6], P[4], ctypes.c_void_p(4104), BIG), (1, None, P[6], P[4], P[9], BIG)])
def test_group_norm_bwd_refuses(lib, want, dx, dgate, gate, ws, n):
    from sub_linear_memory_gb300 import norm  # noqa: F401

    assert lib.slim_group_norm_bwd(P[0], P[1], P[2], P[3], gate, 8, 0.0, dx, dgate, 8, P[7], P[8], ws, n, 4, 8, 2, None) == want


@pytest.mark.parametrize("want, change, entry", [
    (1, dict(bits=16), {}), (1, dict(beta1=1.0), {}), (1, dict(beta2=-0.1), {}), (1, dict(eps=-1e-8), {}),
    (1, dict(beta1=math.nan), {}), (1, {}, dict(n=-1)), (1, {}, dict(param=None)), (1, {}, dict(m=None)), (1, dict(bits=8), {}),
    (2, {}, dict(param=4097)), (2, {}, dict(grad=4098)), (2, {}, dict(n=1 << 41)),
    (2, dict(bits=8), dict(m_scales=4096, v_scales=4096, m=4104))])
def test_adamw_refuses(lib, want, change, entry):
    from sub_linear_memory_gb300 import optim

    t = (optim._Tensor * 1)()
    for k, x in dict(dict(param=4096, grad=8192, m=12288, v=16384, n=4), **entry).items():
        setattr(t[0], k, x)
    o = optim._Options(1e-3, 1e-8, 0.0, 32, 0.9, 0.99, 0, None)
    for k, x in change.items():
        setattr(o, k, x)
    assert lib.slim_adamw_f32(t, 1, ctypes.byref(o), P[0], None) == want


def test_adamw_needs_a_count_and_options(lib):
    from sub_linear_memory_gb300 import optim

    o = optim._Options(1e-3, 1e-8, 0.0, 32, 0.9, 0.99, 0, None)
    assert lib.slim_adamw_f32(None, 0, ctypes.byref(o), None, None) == 1
    assert lib.slim_adamw_f32(None, 0, None, P[0], None) == 1
    assert lib.slim_adamw_f32(None, 2, ctypes.byref(o), P[0], None) == 1


def test_group_norm_refuses_gates_whose_rows_overlap(lib):
    from sub_linear_memory_gb300 import norm  # noqa: F401

    assert lib.slim_group_norm(P[0], P[1], P[2], P[3], 7, 0.0, P[4], 4, 8, 2, None) == 1
    for rows in ((7, 8), (8, 7)):
        assert lib.slim_group_norm_bwd(P[0], P[1], P[2], P[3], P[4], rows[0], 0.0, P[5], P[6], rows[1], P[7], P[8], P[9], BIG, 4, 8, 2,
                                       None) == 1
