"""GPU parity of AdamW with fp64 (oracle/train.py).

Tolerances: fp32 arithmetic, a unit 2^-24 of the terms for each of a few
operations (p: 8 of them, and the update's dozen; moments: 4).  8-bit states:
a code may differ by one step where fp64 and fp32 fall on the two sides of the
random threshold, which a value within 2^-20 of it can; they are counted (at
most one in ten thousand, and one), and the rest are equal.
"""
import numpy as np
import pytest
import torch

from oracle import q8 as ref8
from oracle import train as ref
from sub_linear_memory_gb300 import inputs

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
BETAS, EPS, LR, WD = (0.9, 0.99), 1e-8, 1e-2, 0.1
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def optim():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from sub_linear_memory_gb300 import optim

    return optim


def np64(t):
    return t.detach().to("cpu", torch.float64).numpy().reshape(-1)


def draw(shape, slot, dtype=F32, scale=1.0):
    return inputs.gaussian(shape, 7400, slot, scale=scale, dtype=dtype).cuda()


SIZES = [[(5,)], [(128,), (1,), (4096,), (3, 43)], [(64, 129), (4097,), (127,), (12345,), (0,), (2, 2)], [(7,)] * 60, [(20000,)] + [(33,)] * 520]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "%d_tensors" % len(s))
def test_states_in_32_bits(optim, sizes, dtype):
    params = [draw(s, i) for i, s in enumerate(sizes)]
    grads = [draw(s, 1000 + i, dtype, 1e-2) for i, s in enumerate(sizes)]
    opt = optim.AdamW(params, LR, BETAS, EPS, WD)
    b, lr, wd, eps = BETAS, float(np.float32(LR)), float(np.float32(WD)), float(np.float32(EPS))
    ref_p = [np64(p) for p in params]
    ref_m, ref_v = [np.zeros_like(p) for p in ref_p], [np.zeros_like(p) for p in ref_p]
    for t in (1, 2, 3):
        opt.step(grads)
        for i, g in enumerate(grads):
            ref_m[i], ref_v[i] = ref.moments(np64(g), ref_m[i], ref_v[i], b)
            ref_p[i] = ref.weight(ref_p[i], ref_m[i], ref_v[i], t, lr, b, eps, wd)
        grads = [g.flip(0) * 0.5 for g in grads]
    torch.cuda.synchronize()
    assert opt.count.tolist() == [3, 0]
    for i, g in enumerate(grads):
        top = np.abs(ref_m[i]) + 0.1 * np.max(np.abs(np64(g)), initial=0.0)
        assert np.all(np.abs(np64(opt.m[i]) - ref_m[i]) <= 12 * U * top)
        assert np.all(np.abs(np64(opt.v[i]) - ref_v[i]) <= 12 * U * np.abs(ref_v[i]))
        # three updates of at most 3 lr each, a dozen units of their terms (m's relative to top), and p's own roundings
        assert np.all(np.abs(np64(params[i]) - ref_p[i]) <= 24 * U * np.abs(ref_p[i]) + 3 * 40 * U * 10 * lr)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("sizes", SIZES[:4], ids=lambda s: "%d_tensors" % len(s))
def test_states_in_8_bits(optim, sizes, dtype):
    from sub_linear_memory_gb300 import q8

    seed = 0x123456789ABCDEF
    params = [draw(s, i) for i, s in enumerate(sizes)]
    opt = optim.AdamW(params, LR, BETAS, EPS, WD, bits=8, seed=seed)
    b, lr, wd, eps = BETAS, float(np.float32(LR)), float(np.float32(WD)), float(np.float32(EPS))
    wrong = total = 0
    for t in (1, 2):
        grads = [draw(s, 1000 * t + i, F32, 1e-2) for i, s in enumerate(sizes)]
        grads = [(g * torch.exp(3 * draw(g.shape, 5000 + i))).to(dtype) for i, g in enumerate(grads)]
        p0 = [np64(p) for p in params]
        m0, r0 = ([np64(q8.dequantize(s, F32)) for s in states] for states in (opt.m, opt.v))
        opt.step(grads)
        torch.cuda.synchronize()
        for i, g in enumerate(grads):
            m, v = ref.moments(np64(g), m0[i], r0[i] ** 2, b)
            want = ref.weight(p0[i], m, v, t, lr, b, eps, wd)
            rate = (np.abs(m0[i]) * b[0] + np.abs(np64(g)) * (1 - b[0])) / (np.sqrt(v / (1 - b[1] ** t)) + eps) / (1 - b[0] ** t)
            assert np.all(np.abs(np64(params[i]) - want) <= 16 * U * (np.abs(p0[i]) + lr * rate))
            for state, x, half in ((opt.m[i], m, 0), (opt.v[i], np.sqrt(v), 1)):
                bits = ref.random16(x.size, i, t, seed)[half]
                held, scales = ref.held_at_random(x, bits, half == 1)
                nb = -(-x.size // 128)
                got_scales = state.scales.cpu().numpy().reshape(-1)
                got = np64(q8.dequantize(state, F32))
                # A block's scale may differ where its largest value lies on the border of two, 448 times a power of
                # two, but for the fp32 roundings: a bf16 gradient of 17.5 alone has the root sqrt(0.01) 17.5 = 1.75 =
                # 448 / 256, and fp32's 0.01 lies below it.  Its root takes half of v's four units, and rounds once.
                same = np.repeat(got_scales[:nb] == scales, 128)[:x.size]
                tops = np.abs(np.pad(x, (0, -x.size % 128))).reshape(-1, 128).max(1)[got_scales[:nb] != scales]
                border = 448 * 2.0 ** np.round(np.log2(np.maximum(tops, 1e-300) / 448))
                assert np.all(np.abs(tops - border) <= 4 * U * border)
                wrong += int((got != held)[same].sum())
                total += x.size
                assert np.all(np.abs(got - held) <= np.maximum(np.abs(held) * 0.25, 2.0 ** -8 * np.repeat(2.0 ** (scales.astype(float) - 127), 128)[:x.size]))
                assert np.all(got_scales[nb:] == 127) and not state.codes.view(torch.uint8)[:, x.size:].any()
                if half:
                    assert np.all((got > 0) | (x == 0))
    assert wrong <= 1 + total * 1e-4


def test_roundings_at_random_keep_small_changes(optim):
    """A second moment that should grow by 0.1% a step does, in the mean, though a code's step is a hundred times that."""
    n = 1 << 16
    p = torch.zeros(n, device="cuda")
    opt = optim.AdamW([p], 0.0, (0.9, 0.999), EPS, 0.0, bits=8, seed=5)
    from sub_linear_memory_gb300 import q8

    start = torch.full((n,), 0.9, device="cuda")
    start[::128] = 7.0  # the block's largest stays what it is: one scale throughout
    held = q8.quantize(start.view(1, n))
    opt = optim.AdamW([p], 0.0, (0.9, 0.999), EPS, 0.0, bits=8, seed=5, v=[held])
    r0 = q8.dequantize(opt.v[0], F32).view(-1)
    g = r0 * 2 ** 0.5
    g[::128] = r0[::128]
    for _ in range(20):
        opt.step([g])
    r = q8.dequantize(opt.v[0], F32).view(-1)
    pick = torch.arange(n, device="cuda") % 128 != 0
    # v -> v + (1 - b2)(2 v0 - v): after 20 steps v / v0 = 2 - 0.999^20.  The mean of r^2 also gains the variance of
    # its roundings, at most a quarter of a squared step (1/16 here) a step, and its sample mean is off by 4 / sqrt(n) of a step.
    want = (2 - 0.999 ** 20) ** 0.5
    mean = float((r[pick] / r0[pick]).double().mean())
    step = 0.0625 / 0.875
    assert want - 4 * step / n ** 0.5 - 0.01 * (want - 1) - step ** 2 / 8 <= mean <= want + 4 * step / n ** 0.5 + step ** 2 * 20 * 0.001


def test_a_captured_step_goes_on_counting(optim):
    """Replays of one graph are the steps that calls would have made, under the rate of that moment."""
    for bits in (8, 32):
        lr = torch.full((1,), LR, device="cuda")
        a, b = ([draw((300,), 1), draw((1000,), 2)] for _ in range(2))
        grads = [draw((300,), 3), draw((1000,), 4)]
        one, two = optim.AdamW(a, lr, BETAS, bits=bits, seed=9), optim.AdamW(b, lr, BETAS, bits=bits, seed=9)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            two.step(grads)
        for k in range(4):
            lr.fill_(LR / (k + 1))
            one.step(grads)
            graph.replay()
        torch.cuda.synchronize()
        assert one.count.tolist() == two.count.tolist() == [4, 0]
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_tensors_without_gradient_and_alignment(optim):
    base = draw((3001,), 0)
    params = [base[1:1000], base[1000:1700].clone(), base[1701:3001]]  # 4, 16 and 4 bytes off
    grads = [draw((1001,), 1, BF16)[2:], None, draw((1301,), 2, BF16)[1:]]
    kept = [p.clone() for p in params]
    opt = optim.AdamW(params, LR, BETAS, bits=8)
    opt.step(grads)
    other = [p.clone() for p in kept]
    plain = optim.AdamW(other, LR, BETAS, bits=8)
    plain.step([g if g is None else g.clone() for g in grads])
    torch.cuda.synchronize()
    assert torch.equal(params[1], kept[1]) and not opt.m[1].codes.view(torch.uint8).any()
    assert all(torch.equal(x, y) for x, y in zip(params, other))
    assert base[0] == draw((3001,), 0)[0] and base[1700] == draw((3001,), 0)[1700]
    opt.step([None] * 3)
    assert opt.count.tolist() == [2, 0]


def test_a_gradient_that_is_not_finite(optim):
    """It takes its own element (its own block of the 8-bit states), as a plain step does, and no other."""
    for bits in (8, 32):
        p = draw((400,), 0)
        clean = p.clone()
        g = draw((400,), 1)
        optim.AdamW([clean], LR, BETAS, bits=bits).step([g])
        g[200] = float("nan")
        opt = optim.AdamW([p], LR, BETAS, bits=bits)
        opt.step([g])
        assert p[200].isnan()
        p[200] = clean[200]
        assert torch.equal(p, clean)
        if bits == 8:
            assert opt.m[0].scales[0, :4].tolist()[1] == 255


def test_refusals(optim):
    from sub_linear_memory_gb300 import q8

    p, g = draw((64,), 0), draw((64,), 1)
    make = lambda **kw: optim.AdamW([p], **kw)
    bad = [lambda: optim.AdamW([]), lambda: optim.AdamW([p.cpu()]), lambda: optim.AdamW([p.bfloat16()]), lambda: optim.AdamW([p[::2]]),
           lambda: optim.AdamW([p, p]), lambda: optim.AdamW([p, p[10:20]]), lambda: make(bits=16), lambda: make(betas=(1.0, 0.9)),
           lambda: make(betas=(0.9, -0.1)), lambda: make(eps=-1.0), lambda: make(seed=-1), lambda: make(m=[]),
           lambda: make(m=[draw((3,), 2)]), lambda: make(m=[p]), lambda: make(bits=8, m=[draw((64,), 2)]),
           lambda: make(bits=8, v=[q8.empty(1, 65)]), lambda: make().step([]), lambda: make().step([g.half()]),
           lambda: make().step([g[:10]]), lambda: make().step([g.cpu()]), lambda: optim.AdamW([p, draw((4,), 3)]).step([g, draw((4,), 3, BF16)]),
           lambda: make(lr=torch.zeros(1)).step([g]), lambda: make(lr=torch.zeros(2, device="cuda")).step([g])]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail("call %d was taken" % i)


def test_codes_are_those_of_elementary_operations(optim):
    """The moments formed in fp32 by one rounded operation after another, and rounded at random: every code the same."""
    from sub_linear_memory_gb300 import q8

    n, seed = 40000, 77
    p, g = draw((n,), 0), draw((n,), 1) * torch.exp(2 * draw((n,), 2))
    opt = optim.AdamW([p], LR, BETAS, EPS, WD, bits=8, seed=seed)
    for t in (1, 2, 3):
        m, r = (q8.dequantize(s, F32).view(-1) for s in (opt.m[0], opt.v[0]))
        m = m * BETAS[0] + g * (1 - BETAS[0])
        v = r.square() * BETAS[1] + g * g * (1 - BETAS[1])
        opt.step([g])
        torch.cuda.synchronize()
        bits = ref.random16(n, 0, t, seed)
        for state, x, half in ((opt.m[0], m, 0), (opt.v[0], v.sqrt(), 1)):
            held, scales = ref.held_at_random(np64(x), bits[half], half == 1)
            assert np.array_equal(state.scales.cpu().numpy().reshape(-1)[:scales.size], scales)
            # fp32's sum with 2^-6, below the normal codes, may round across the threshold
            assert (np64(q8.dequantize(state, F32)) != held).mean() <= 1e-4
