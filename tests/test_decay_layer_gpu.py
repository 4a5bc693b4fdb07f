"""The decay attention, the group norm and AdamW together: a layer's training
step and its serving against the same layer in fp64, and steps of its weights.

Bars as for the Performer layer: an e4m3 rounding is a relative rms of 2.6%,
and a chain of n of them sqrt(n) times that: at most 6 on the way forward
(6.4%), 12 on the way back to a gradient (9%); the bars are twice that.  A
wrong term is off by its own size.
"""
import numpy as np
import pytest
import torch

from oracle import lm
from sub_linear_memory_gb300 import inputs

pytestmark = pytest.mark.gpu

LENGTHS = [130, 1, 0, 200, 75]
T = sum(LENGTHS)
HEADS, KV, D, FF = 4, 2, 64, 512
DM = HEADS * D
LOGS = [-0.2, -0.01]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def draw(shape, slot, scale=1.0, dtype=torch.float32):
    return inputs.gaussian(shape, 7500, slot, scale=scale, dtype=dtype)


def weights():
    return {"win": draw(((2 * HEADS + 2 * KV) * D, DM), 1, DM ** -0.5), "wo": draw((DM, DM), 2, DM ** -0.5),
            "w1": draw((FF, DM), 3, DM ** -0.5), "w2": draw((DM, FF), 4, FF ** -0.5), "g1": 1 + 0.1 * draw((DM,), 5),
            "g2": 1 + 0.1 * draw((DM,), 6), "gn": 1 + 0.1 * draw((DM,), 7), "bn": 0.1 * draw((DM,), 8)}


def make(w):
    from sub_linear_memory_gb300.layer8 import DecayLayer8

    return DecayLayer8(HEADS, KV, torch.tensor(LOGS, device="cuda"), **{k: v.cuda() for k, v in w.items()})


def cu():
    return torch.tensor(np.cumsum([0] + LENGTHS), dtype=torch.int32, device="cuda")


def reference(w, x, r, dh=None, df=None):
    """The layer in fp64, its gradients by autograd, with the attention's quadratic form."""
    t = {k: v.double().requires_grad_(True) for k, v in w.items()}
    x = x.double().requires_grad_(True)
    norm = lambda h, g: h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-5) * g
    h = x + r.double()
    q, k, v, z = (norm(h, t["g1"]) @ t["win"].t()).split((DM, KV * D, KV * D, DM), 1)
    lam = torch.tensor(LOGS).double().exp()
    outs, a = [], 0
    for n in LENGTHS:
        heads = lambda y, m: y[a:a + n].view(n, m, D).transpose(0, 1)
        qs, ks, vs = heads(q, HEADS), heads(k, KV).repeat_interleave(2, 0), heads(v, KV).repeat_interleave(2, 0)
        i = torch.arange(n).double()
        dec = torch.tril(lam.repeat_interleave(2)[:, None, None] ** (i[:, None] - i).clamp(min=0))
        outs.append((((qs @ ks.transpose(1, 2)) * dec @ vs) * D ** -0.5).transpose(0, 1).reshape(n, DM))
        a += n
    o = torch.cat(outs).view(T, HEADS, D)
    c = o - o.mean(2, keepdim=True)
    gn = (c / torch.sqrt((c * c).mean(2, keepdim=True) + 1e-5)).view(T, DM) * t["gn"] + t["bn"]
    h2 = h + (gn * z * torch.sigmoid(z)) @ t["wo"].t()
    f = lm.gelu(norm(h2, t["g2"]) @ t["w1"].t()) @ t["w2"].t()
    if dh is None:
        return h2.detach(), f.detach()
    ((h2 * dh.double()).sum() + (f * df.double()).sum()).backward()
    return h2.detach(), f.detach(), x.grad, {k: v.grad for k, v in t.items()}


def rel(got, want):
    got, want = got.detach().double().cpu(), want.double().cpu()
    return float((got - want).norm() / want.norm())


def rows():
    bf = lambda slot, scale=1.0: draw((T, DM), slot, scale, torch.bfloat16)
    return bf(10), bf(11, 0.5), bf(12, 1e-3), bf(13, 1e-3)


def test_training_step():
    from sub_linear_memory_gb300 import binding

    w = weights()
    x, r, dh, df = rows()
    layer = make(w)
    (h2, f), kept = layer.forward(x.cuda(), r.cuda(), cu())
    dx, grads = layer.backward(dh.cuda(), df.cuda(), kept)
    binding.sync_status()
    h2_ref, f_ref, dx_ref, grads_ref = reference(w, x, r, dh, df)
    assert rel(h2, h2_ref) <= 0.13 and rel(f, f_ref) <= 0.13
    assert rel(dx, dx_ref) <= 0.18
    assert set(grads) == set(grads_ref)
    for name, want in grads_ref.items():
        assert grads[name].shape == want.shape and rel(grads[name], want) <= 0.18, name


def test_serving():
    """Prompts in two windows and tokens one by one, states in a cache, give the forward's rows: the same
    roundings, but for sums in another order."""
    from sub_linear_memory_gb300 import binding

    layer = make(weights())
    b, length = 3, 140
    x, r = draw((b, length, DM), 20, 1.0, torch.bfloat16).cuda(), draw((b, length, DM), 21, 0.5, torch.bfloat16).cuda()
    ends = lambda n: torch.arange(b + 1, dtype=torch.int32, device="cuda") * n
    part = lambda t, i, j: t[:, i:j].reshape(b * (j - i), DM).contiguous()
    (h2, f), _ = layer.forward(part(x, 0, length), part(r, 0, length), ends(length))
    cache = torch.zeros((7, KV, D, D), device="cuda")
    slots = torch.tensor([6, 0, 3], dtype=torch.int32, device="cuda")
    for i, j in ((0, 100), (100, 137)):
        got = layer.prefill(part(x, i, j), part(r, i, j), ends(j - i), cache, slots)
        for a, want in zip(got, (h2, f)):
            assert rel(a, want.view(b, length, DM)[:, i:j].reshape(-1, DM)) <= 0.05
    for i in range(137, length):
        got = layer.decode(x[:, i].contiguous(), r[:, i].contiguous(), cache, slots)
        for a, want in zip(got, (h2, f)):
            assert rel(a, want.view(b, length, DM)[:, i]) <= 0.05
    binding.sync_status()
    assert not cache[[1, 2, 4, 5]].any()


@pytest.mark.parametrize("bits", [8, 32])
def test_steps_of_the_weights(bits):
    """Gradients into AdamW, new weights into the layer: the weights are those of the plain formula on the same
    gradients (8-bit moments: whose first two steps they cannot tell apart by more than a code's step, 1/8 of an
    update), and the layer goes on with them."""
    from sub_linear_memory_gb300 import binding, optim

    w = {k: v.cuda() for k, v in weights().items()}
    layer = make(w)
    x, r, dh, df = (t.cuda() for t in rows())
    names = list(w)
    lr, betas = 1e-3, (0.9, 0.99)
    opt = optim.AdamW([w[n] for n in names], lr=lr, betas=betas, weight_decay=0.0, bits=bits)
    want = {n: w[n].double().clone() for n in names}
    m, v = {n: 0.0 for n in names}, {n: 0.0 for n in names}
    outs = []
    for t in (1, 2):
        (_, f), kept = layer.forward(x, r, cu())
        outs.append(f)
        _, grads = layer.backward(dh, df, kept)
        opt.step([grads[n] for n in names])
        layer.load(**{n: w[n] for n in layer.NAMES})
        for n in names:
            g = grads[n].double()
            m[n], v[n] = betas[0] * m[n] + (1 - betas[0]) * g, betas[1] * v[n] + (1 - betas[1]) * g * g
            want[n] -= lr * (m[n] / (1 - betas[0] ** t)) / ((v[n] / (1 - betas[1] ** t)).sqrt() + 1e-8)
    binding.sync_status()
    for n in names:
        off = (w[n].double() - want[n]).abs()
        tiny = 2.0 ** -22 * want[n].abs() + lr * 1e-4
        assert bool((off <= tiny + (0.5 * lr if bits == 8 else 0)).all()), n
        assert float((off / lr).square().mean()) <= (0.125 ** 2 if bits == 8 else 1e-6), n
    assert torch.isfinite(outs[1].float()).all() and not torch.equal(outs[0], outs[1])


def test_no_rows():
    from sub_linear_memory_gb300 import binding

    layer = make(weights())
    none = torch.empty((0, DM), dtype=torch.bfloat16, device="cuda")
    ends = torch.zeros(3, dtype=torch.int32, device="cuda")
    (h2, f), kept = layer.forward(none, none, ends)
    dx, grads = layer.backward(none, none, kept)
    state = draw((2, KV, D, D), 30).cuda()
    before = state.clone()
    layer.prefill(none, none, ends, state)
    layer.decode(none, none, state[:0])
    binding.sync_status()
    assert h2.shape == f.shape == dx.shape == (0, DM) and torch.equal(state, before)
    assert all(not g.any() for g in grads.values())
