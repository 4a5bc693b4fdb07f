"""GPU parity of the group norm with a gate with fp64 (oracle/train.py).

Tolerances, element by element: storing as bf16 2^-8 of the value; fp32
arithmetic a unit 2^-24 of the terms for each of a few dozen operations (the
exponential and the reciprocal among them), and for each addition in sequence
of the group's sums (at most 64 for a lane and 5 between lanes, but 512 where a
group is wider than 1024 columns).  The terms: of n (|x| + |mean|) rstd, whose
relative error grows with a mean far from 0.
"""
import numpy as np
import pytest
import torch

from oracle import train as ref
from sub_linear_memory_gb300 import inputs

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
STORE = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def norm():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from sub_linear_memory_gb300 import norm

    return norm


def np64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def draw(shape, slot, dtype=F32, scale=1.0):
    return inputs.gaussian(shape, 7300, slot, scale=scale, dtype=dtype).cuda()


def make(rows, cols, dtype, gate=True, offset=0.0):
    x = (draw((rows, cols), 0) + offset).to(dtype)
    return (draw((rows, cols), 1, dtype), x, 1 + 0.3 * draw((cols,), 2), draw((cols,), 3),
            draw((rows, cols), 4, dtype, 2.0) if gate else None)


def check(norm, rows, cols, groups, dtype, gate=True, offset=0.0, eps=1e-5):
    dy, x, gamma, beta, z = make(rows, cols, dtype, gate, offset)
    y = norm.group_norm(x, gamma, beta, groups, z, eps)
    got = norm.group_norm_bwd(dy, x, gamma, beta, groups, z, eps)
    torch.cuda.synchronize()
    hx, hg, hb, hdy = np64(x), np64(gamma), np64(beta), np64(dy)
    hz = np64(z) if gate else None
    width = cols // groups
    u = 2.0 ** -24 * (40 + (64 if width <= 1024 else width // 32 + 8))
    v = hx.reshape(rows, groups, width)
    rstd = 1 / np.sqrt(v.var(2, keepdims=True) + eps)
    n_mag = ((np.abs(v) + np.abs(v).mean(2, keepdims=True)) * rstd).reshape(rows, cols)
    s = 1 / (1 + np.exp(-hz)) if gate else np.ones_like(hx)
    opened = np.abs(hz * s) if gate else s
    y_mag = n_mag * np.abs(hg) + np.abs(hb)
    want = ref.group_norm(hx, hg, hb, groups, hz, eps)
    # the exponent's rounding: |z| units of e^-z
    rough = u * (1 + (np.abs(hz) / 8 if gate else 0))
    store = STORE[dtype]
    assert np.all(np.abs(np64(y) - want) <= store * np.abs(want) + rough * y_mag * opened)
    dx, dgate, dgamma, dbeta = ref.group_norm_bwd(hdy, hx, hg, hb, groups, hz, eps)
    d_mag = np.abs(hdy) * opened
    if gate:
        assert np.all(np.abs(np64(got[1]) - dgate) <= store * np.abs(dgate) + rough * np.abs(hdy) * y_mag * (1 + np.abs(hz)))
    else:
        assert got[1] is None
    h = (d_mag * np.abs(hg)).reshape(v.shape)
    nm = n_mag.reshape(v.shape)
    dx_mag = (rstd * (h + h.mean(2, keepdims=True) + nm * (h * nm).mean(2, keepdims=True))).reshape(rows, cols)
    assert np.all(np.abs(np64(got[0]) - dx) <= store * np.abs(dx) + 3 * rough * dx_mag)
    # a column's sum: at most a thousand additions in sequence
    for g, w, m in ((got[2], dgamma, d_mag * n_mag), (got[3], dbeta, d_mag)):
        assert np.all(np.abs(np64(g) - w) <= (m * (rough + 2.0 ** -24 * 1000)).sum(0) + 2.0 ** -24 * np.abs(w))


SIZES = [(1, 64, 1), (3, 1024, 16), (130, 512, 8), (7, 768, 6), (5, 40, 5), (9, 24, 8), (20, 1000, 8), (33, 77, 7), (2, 1, 1),
         (4, 6, 6), (11, 1024, 4), (6, 2048, 4), (5, 2048, 2), (3, 4096, 2), (2, 16384, 1), (4, 1536, 12), (3, 3000, 2), (600, 256, 2),
         (17, 8, 1), (2500, 48, 3), (70, 130, 1), (10, 1002, 2)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("rows, cols, groups", SIZES)
def test_forward_and_backward(norm, rows, cols, groups, gate, dtype):
    check(norm, rows, cols, groups, dtype, gate)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_mean_far_from_zero(norm, dtype):
    check(norm, 40, 512, 8, dtype, offset=50.0)


def test_misaligned_rows(norm):
    """Tensors that do not start on 16 bytes go element by element, with the same result."""
    dy, x, gamma, beta, z = make(50, 512, BF16)
    shift = lambda t: torch.cat([t.flatten()[:1], t.flatten()])[1:].view(t.shape)
    moved = [shift(t) for t in (dy, x, z)]
    assert all(t.data_ptr() % 16 for t in moved)
    y = norm.group_norm(moved[1], gamma, beta, 8, moved[2])
    want = ref.group_norm(np64(x), np64(gamma), np64(beta), 8, np64(z))
    assert np.all(np.abs(np64(y) - want) <= 2.0 ** -8 * np.abs(want) + 1e-5)
    a, b = norm.group_norm_bwd(moved[0], moved[1], gamma, beta, 8, moved[2]), norm.group_norm_bwd(dy, x, gamma, beta, 8, z)
    for s, t in zip(a, b):
        assert np.linalg.norm(np64(s) - np64(t)) <= 4e-3 * np.linalg.norm(np64(t))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols, groups, pitch", [(512, 8, 1536), (96, 2, 200), (100, 4, 303), (2048, 1, 2056)])
def test_gates_whose_rows_lie_apart(norm, cols, groups, pitch, dtype):
    dy, x, gamma, beta, z = make(33, cols, dtype)
    rows = draw((33, pitch), 9, dtype)
    rows[:, 8:8 + cols] = z
    out = rows.clone()
    apart = rows[:, 8:8 + cols]
    y, same = norm.group_norm(x, gamma, beta, groups, apart), norm.group_norm(x, gamma, beta, groups, z)
    assert np.linalg.norm(np64(y) - np64(same)) <= (4e-3 if dtype == BF16 else 1e-6) * np.linalg.norm(np64(same))
    want = norm.group_norm_bwd(dy, x, gamma, beta, groups, z)
    got = norm.group_norm_bwd(dy, x, gamma, beta, groups, apart, dgate=out[:, 8:8 + cols])
    for a, b in zip(got, want):  # an odd pitch takes another kernel, whose sums run in another order
        assert np.linalg.norm(np64(a) - np64(b)) <= (4e-3 if dtype == BF16 else 1e-6) * np.linalg.norm(np64(b))
    assert torch.equal(out[:, :8], rows[:, :8]) and torch.equal(out[:, 8 + cols:], rows[:, 8 + cols:])


def test_equal_columns_and_eps(norm):
    """A group of equal values has no variance: n = 0, and with eps = 0 the result is NaN, as 0 times infinity is."""
    x = torch.full((2, 64), 3.0, dtype=BF16, device="cuda")
    gamma, beta = torch.ones(64, device="cuda"), torch.arange(64.0, device="cuda")
    assert torch.equal(norm.group_norm(x, gamma, beta, 1).float(), beta.bfloat16().float().expand(2, 64))
    assert norm.group_norm(x, gamma, beta, 1, eps=0.0).isnan().all()


def test_one_groups_nan_stays_in_it(norm):
    dy, x, gamma, beta, z = make(6, 256, BF16)
    clean = norm.group_norm(x, gamma, beta, 4, z)
    x[2, 70] = float("nan")
    y = norm.group_norm(x, gamma, beta, 4, z)
    assert y[2, 64:128].isnan().all()
    y[2, 64:128] = clean[2, 64:128]
    assert torch.equal(y, clean)


def test_no_rows_and_the_same_every_time(norm):
    dy, x, gamma, beta, z = make(0, 64, BF16)
    assert norm.group_norm(x, gamma, beta, 2, z).shape == (0, 64)
    out = norm.group_norm_bwd(dy, x, gamma, beta, 2, z)
    assert not out[2].any() and not out[3].any()
    dy, x, gamma, beta, z = make(3000, 512, BF16)
    first, again = (norm.group_norm_bwd(dy, x, gamma, beta, 8, z) for _ in range(2))
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = norm.group_norm_bwd(dy, x, gamma, beta, 8, z)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, held))


def test_refusals(norm):
    dy, x, gamma, beta, z = make(4, 64, BF16)
    bad = [lambda: norm.group_norm(x.t(), gamma, beta, 2), lambda: norm.group_norm(x.half(), gamma, beta, 2),
           lambda: norm.group_norm(x, gamma[:3], beta, 2), lambda: norm.group_norm(x, gamma, beta.bfloat16(), 2),
           lambda: norm.group_norm(x, gamma, beta, 3), lambda: norm.group_norm(x, gamma, beta, 0),
           lambda: norm.group_norm(x, gamma, beta, 2, z.float()), lambda: norm.group_norm(x, gamma, beta, 2, z[:2]),
           lambda: norm.group_norm(x.cpu(), gamma, beta, 2), lambda: norm.group_norm_bwd(dy[:1], x, gamma, beta, 2)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail("call %d was taken" % i)
    from sub_linear_memory_gb300 import binding

    with pytest.raises(binding.SlimError):
        norm.group_norm(x, gamma, beta, 2, z, out=x)
