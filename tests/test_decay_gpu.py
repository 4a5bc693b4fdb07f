"""GPU parity of the decay attention with the fp64 recurrence (oracle/decay.py).

Tolerances, element by element, from what each step may round.  With A the same
result formed from magnitudes (an upper bound on the sum of its terms'
magnitudes):
  * storing as bf16: 2^-8 of the value;
  * bf16 rows: the weighted score, or the state, is rounded to bf16 before its
    product: 2^-8 A;
  * fp32 sums: one unit 2^-24 of A for each addition in sequence (at most 600:
    the columns, the rows of a tile, the tiles and shares), and the same for
    the powers of lambda; states of bf16 rows, whose weighted rows enter as two
    bf16 numbers, 2^-16 A besides.
In the 2-norm, where roundings of random size and sign add up as their root
mean square, 1/sqrt(3) of the largest: sqrt(2/3) 2^-8 for two of them in bf16,
which leaves 2^-8; 2e-6 in fp32, and 2^-17 for states of bf16 rows.
"""
import numpy as np
import pytest
import torch

from oracle import decay as ref
from oracle import rel_l2
from sub_linear_memory_gb300 import inputs

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def decay():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from sub_linear_memory_gb300 import decay

    return decay


def sync():
    from sub_linear_memory_gb300 import binding

    binding.sync_status()


def np64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def draw(shape, slot, dtype=F32, scale=1.0):
    return inputs.gaussian(shape, 7200, slot, scale=scale, dtype=dtype).cuda()


def close(got, want, size, dtype, state=False):
    got, two = np64(got), 2.0 ** -24 * 600
    bf = dtype == BF16
    tol = size * (two + (2.0 ** -16 if state else 2.0 ** -8 if bf else 0)) + (0 if state or not bf else 2.0 ** -8 * np.abs(want))
    off = np.abs(got - want)
    assert np.all(off <= tol), "%g over the bound" % np.max(off / np.maximum(tol, 1e-300))
    if want.size > 64 and np.linalg.norm(want) > 0:
        assert rel_l2(got, want) <= (2.0 ** -17 if state and bf else 2e-6 if state or not bf else 2.0 ** -8)


LOGS = {1: [-0.02], 2: [-0.3, -0.004], 3: [-1.5, -0.03, 0.0], 4: [-40.0, -0.2, -0.01, -0.0002]}


class Case:
    def __init__(self, lengths, hk, group, dk, dv, dtype, gap=(0, 0), fused=False, state=True, scale=0.3):
        self.lengths, self.dtype, self.scale = lengths, dtype, scale
        t = sum(lengths) + sum(gap)
        self.cu = [gap[0] + sum(lengths[:i]) for i in range(len(lengths) + 1)]
        hq = hk * group
        widths = (hq * dk, hk * dk, hk * dv)
        if fused:
            rows = draw((t, sum(widths)), 0, dtype)
            q, k, v = rows.split(widths, 1)
        else:
            q, k, v = (draw((t, w), i, dtype) for i, w in enumerate(widths))
        self.q, self.k, self.v = q.view(t, hq, dk), k.view(t, hk, dk), v.view(t, hk, dv)
        self.do = draw((t, hq, dv), 4, dtype)
        self.log = torch.tensor(LOGS[hk], dtype=F32, device="cuda")
        n = len(lengths)
        self.s0 = draw((n, hk, dk, dv), 5) if state else None
        self.g_in = draw((n, hk, dk, dv), 6) if state else None
        self.cu_gpu = torch.tensor(self.cu, dtype=torch.int32, device="cuda")

    def host(self, absolute=False):
        f = (lambda x: None if x is None else np.abs(np64(x))) if absolute else (lambda x: None if x is None else np64(x))
        return f(self.q), f(self.k), f(self.v), np64(self.log), self.cu, f(self.do), f(self.s0), f(self.g_in)

    def check_forward(self, decay, use_cu=True):
        end = torch.empty_like(self.s0) if self.s0 is not None else torch.empty(
            (len(self.lengths),) + (self.k.shape[1], self.k.shape[2], self.v.shape[2]), device="cuda")
        kw = dict(cu_seqlens=self.cu_gpu) if use_cu else dict(seqs=len(self.lengths))
        out = torch.full((self.q.shape[0], self.q.shape[1], self.v.shape[2]), 7.0, dtype=self.dtype, device="cuda")
        o = decay.attn(self.q, self.k, self.v, self.log, scale=self.scale, state_in=self.s0, state_out=end, out=out, **kw)
        sync()
        inside = slice(self.cu[0], self.cu[-1])
        (o_ref, e_ref), (o_mag, e_mag) = (ref.forward(*self.host(a)[:5], self.scale, self.host(a)[6]) for a in (False, True))
        close(o[inside], o_ref[inside], o_mag[inside], self.dtype)
        close(end, e_ref, e_mag, self.dtype, state=True)
        assert (o[:self.cu[0]] == 7).all() and (o[self.cu[-1]:] == 7).all()

    def check_backward(self, decay, use_cu=True):
        g_out = torch.empty_like(self.s0) if self.s0 is not None else None
        kw = dict(cu_seqlens=self.cu_gpu) if use_cu else dict(seqs=len(self.lengths))
        out = [torch.full_like(x, 7.0, memory_format=torch.contiguous_format) for x in (self.q, self.k, self.v)]
        got = decay.attn_bwd(self.q, self.k, self.v, self.log, self.do, scale=self.scale, state_in=self.s0, g_in=self.g_in,
                             g_out=g_out, out=out, **kw)
        sync()
        want, size = (ref.backward(*self.host(a)[:6], self.scale, *self.host(a)[6:]) for a in (False, True))
        inside = slice(self.cu[0], self.cu[-1])
        for g, w, m in zip(got, want, size):
            close(g[inside], w[inside], m[inside], self.dtype)
            assert (g[:self.cu[0]] == 7).all() and (g[self.cu[-1]:] == 7).all()
        if g_out is not None:
            close(g_out, want[3], size[3], self.dtype, state=True)


# lengths, key-value heads, group, dk, dv, further arguments
CASES = {
    "one_token": ([1], 1, 1, 64, 64, {}),
    "a_tile": ([128], 2, 1, 64, 64, {}),
    "a_tile_and_one": ([129], 2, 1, 64, 64, {}),
    "ragged_64": ([1, 0, 127, 130, 64, 3, 400], 2, 2, 64, 64, {}),
    "ragged_128": ([255, 1, 0, 31, 300], 2, 3, 128, 128, {}),
    "gaps": ([40, 200], 2, 1, 64, 64, dict(gap=(3, 130))),
    "fused_rows": ([77, 140, 9], 3, 2, 64, 64, dict(fused=True)),
    "fused_rows_128": ([260, 19], 1, 4, 128, 128, dict(fused=True)),
    "no_state": ([300, 45], 2, 1, 64, 64, dict(state=False)),
    "no_state_128": ([300, 45], 2, 2, 128, 128, dict(state=False)),
    "odd_widths": ([70, 5, 131], 2, 2, 40, 24, {}),
    "narrow": ([33, 100], 3, 1, 1, 7, {}),
    "wide": ([90, 41], 1, 2, 160, 256, {}),
    "strong_decay": ([200, 150], 4, 1, 64, 64, {}),
    "odd_rows": ([100, 37], 1, 1, 65, 64, dict(fused=True)),
    "long": ([2000], 2, 1, 64, 64, {}),
    "long_128": ([1500, 700], 1, 2, 128, 128, {}),
    "many_query_heads_64": ([140, 300, 20], 1, 9, 64, 64, {}),
    "seven_query_heads_64": ([260, 129], 1, 7, 64, 64, {}),
    "many_query_heads_128": ([140, 300], 1, 5, 128, 128, {}),
    "group_of_four_128": ([290, 1, 128], 2, 4, 128, 128, dict(gap=(1, 2))),
    "group_of_four_64": ([290, 1, 128], 2, 4, 64, 64, dict(gap=(1, 2))),
}


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("name", CASES)
def test_forward(decay, name, dtype):
    *args, kw = CASES[name]
    Case(*args, dtype, **kw).check_forward(decay)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("name", CASES)
def test_backward(decay, name, dtype):
    *args, kw = CASES[name]
    Case(*args, dtype, **kw).check_backward(decay)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n, length, d", [(3, 50, 64), (2, 300, 128), (5, 128, 64), (4, 1, 64), (2, 0, 64)])
def test_sequences_of_one_length(decay, n, length, d, dtype):
    c = Case([length] * n, 2, 2, d, d, dtype)
    c.check_forward(decay, use_cu=False)
    c.check_backward(decay, use_cu=False)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128, 24])
def test_many_short_sequences(decay, d, dtype):
    r = np.random.RandomState(1)
    c = Case([int(n) for n in r.randint(0, 9, 300)], 2, 1, d, d, dtype)
    c.check_forward(decay)
    c.check_backward(decay)


def test_no_decay_and_full_decay(decay):
    """log_decay of 0 or more keeps everything, -inf keeps the row alone."""
    c = Case([300], 2, 1, 64, 64, BF16)
    c.log.copy_(torch.tensor([0.5, -float("inf")]))
    c.check_forward(decay)
    c.check_backward(decay)


def test_prompt_by_windows_and_tokens(decay):
    """A prompt in two windows and then token by token, states in a cache."""
    t, hk, d = 200, 2, 64
    c = Case([t, t], hk, 2, d, d, F32, state=False)
    whole = torch.empty((2, hk, d, d), device="cuda")
    o = decay.attn(c.q, c.k, c.v, c.log, c.cu_gpu, c.scale, state_out=whole)
    cache = torch.full((5, hk, d, d), 3.0, device="cuda")
    slots = torch.tensor([4, 1], dtype=torch.int32, device="cuda")
    cache[slots.long()] = 0
    seq = lambda x, a, b: torch.cat([x[a:b], x[t + a:t + b]]).contiguous()
    cu = lambda n: torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    parts = []
    for a, b in ((0, 130), (130, 190)):
        parts.append(decay.attn(seq(c.q, a, b), seq(c.k, a, b), seq(c.v, a, b), c.log, cu(b - a), c.scale, cache, cache, slots).view(2, b - a, 2 * hk, d))
    for a in range(190, t):
        parts.append(decay.step(seq(c.q, a, a + 1), seq(c.k, a, a + 1), seq(c.v, a, a + 1), c.log, cache, slots, c.scale).view(2, 1, 2 * hk, d))
    sync()
    got = torch.cat(parts, 1).view(2 * t, 2 * hk, d)
    assert rel_l2(np64(got), np64(o)) <= 2e-6
    assert rel_l2(np64(cache[slots.long()]), np64(whole)) <= 2e-6
    assert (cache[[0, 2, 3]] == 3).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("long", [False, True])
def test_slots_that_name_no_place_or_anothers(decay, dtype, long):
    lengths = [20, 30, 25, 700 if long else 11, 5]
    c = Case(lengths, 2, 1, 64, 64, dtype)
    c.s0 = draw((7, 2, 64, 64), 5)
    slots = torch.tensor([3, -1, 3, 6, 7], dtype=torch.int32, device="cuda")
    cache = c.s0.clone()
    o = decay.attn(c.q, c.k, c.v, c.log, c.cu_gpu, c.scale, cache, cache, slots)
    sync()
    start = np.zeros((5, 2, 64, 64))
    start[0], start[3] = np64(c.s0)[3], np64(c.s0)[6]
    o_ref, e_ref = ref.forward(*c.host()[:5], c.scale, start)
    o_mag, e_mag = ref.forward(*c.host(True)[:5], c.scale, np.abs(start))
    close(o, o_ref, o_mag, dtype)
    for place, seq in ((3, 0), (6, 3)):
        close(cache[place], e_ref[seq], e_mag[seq], dtype, state=True)
    assert torch.equal(cache[[0, 1, 2, 4, 5]], c.s0[[0, 1, 2, 4, 5]])


STEPS = [(1, 1, 1, 64, 64), (5, 2, 3, 128, 128), (33, 4, 1, 64, 64), (3, 2, 2, 40, 24), (2, 1, 9, 7, 130), (4, 1, 64, 256, 256),
         (2, 3, 4, 5, 1), (3, 1, 8, 130, 6)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n, hk, group, dk, dv", STEPS)
def test_step(decay, n, hk, group, dk, dv, dtype):
    c = Case([1] * n, hk, group, dk, dv, dtype, fused=dk % 2 == 0)
    state = c.s0.clone()
    o = decay.step(c.q, c.k, c.v, c.log, state, scale=c.scale)
    sync()
    (o_ref, e_ref), (o_mag, e_mag) = (ref.forward(*c.host(a)[:5], c.scale, c.host(a)[6]) for a in (False, True))
    close(o, o_ref, o_mag, dtype)
    # one product and one sum, in fp32: lambda's and their roundings
    assert np.all(np.abs(np64(state) - e_ref) <= 4 * 2.0 ** -24 * e_mag)


def test_step_slots(decay):
    c = Case([1] * 6, 2, 2, 64, 64, BF16)
    cache = draw((9, 2, 64, 64), 8)
    before = cache.clone()
    slots = torch.tensor([8, 2, -1, 9, 2, 0], dtype=torch.int32, device="cuda")
    o = decay.step(c.q, c.k, c.v, c.log, cache, slots, c.scale)
    sync()
    for row, place in ((0, 8), (1, 2), (5, 0)):
        one = [x[row:row + 1] for x in (c.q, c.k, c.v)]
        state = before[place:place + 1].clone()
        assert torch.equal(decay.step(*one, c.log, state, scale=c.scale), o[row:row + 1])
        assert torch.equal(state[0], cache[place])
    assert not o[2:5].any()
    rest = [1, 3, 4, 5, 6, 7]
    assert torch.equal(cache[rest], before[rest])


@pytest.mark.parametrize("d", [64, 128, 24])
def test_the_rows_behind_a_sequence_do_not_matter(decay, d):
    """NaN and infinities in another sequence's rows, or in none's, change nothing."""
    c = Case([50, 90, 140], 2, 2, d, d, BF16, gap=(5, 40))
    run = lambda: [decay.attn(c.q, c.k, c.v, c.log, c.cu_gpu, c.scale, c.s0)] + list(
        decay.attn_bwd(c.q, c.k, c.v, c.log, c.do, c.cu_gpu, c.scale, c.s0, c.g_in))
    clean = run()
    for a, b in ((0, c.cu[0]), (c.cu[1], c.cu[2]), (c.cu[3], c.q.shape[0])):
        for x, bad in zip((c.q, c.k, c.v, c.do), (float("nan"), float("inf"), float("nan"), -float("inf"))):
            x[a:b] = bad
    dirty = run()
    sync()
    for a, b in ((c.cu[0], c.cu[1]), (c.cu[2], c.cu[3])):
        for x, y in zip(clean, dirty):
            assert torch.isfinite(x[a:b]).all() and torch.equal(x[a:b], y[a:b])


@pytest.mark.parametrize("d", [64, 128, 24])
def test_the_same_every_time_and_in_a_graph_on_another_stream(decay, d):
    c = Case([300, 64, 500], 2, 2, d, d, BF16)
    end, g_out = torch.empty_like(c.s0), torch.empty_like(c.s0)

    def run():
        o = decay.attn(c.q, c.k, c.v, c.log, c.cu_gpu, c.scale, c.s0, end)
        return [o, *decay.attn_bwd(c.q, c.k, c.v, c.log, c.do, c.cu_gpu, c.scale, c.s0, c.g_in, g_out), end, g_out]

    first = [x.clone() for x in run()]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for x in outs:
        x.zero_()
    graph.replay()
    sync()
    assert all(torch.equal(x, y) for x, y in zip(first, outs))
    # other lengths in the same rows: the graph reads them when it runs
    c.cu_gpu.copy_(torch.tensor([10, 11, 200, 864], dtype=torch.int32))
    graph.replay()
    again = run()
    sync()
    assert all(torch.equal(x[10:], y[10:]) for x, y in zip(again[:4], outs[:4]))


def test_two_calls_at_once(decay):
    """Each call has a workspace of its own."""
    cases = [Case([900, 100], 2, 1, 64, 64, BF16), Case([400, 600], 2, 1, 64, 64, BF16)]
    one = lambda c: decay.attn_bwd(c.q, c.k, c.v, c.log, c.do, c.cu_gpu, c.scale)
    want = [[x.clone() for x in one(c)] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [None, None]
    for _ in range(5):
        for i, (c, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                got[i] = one(c)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for w, g in zip(want, got) for x, y in zip(w, g))


def test_lengths_outside_the_rows_are_kept_inside(decay):
    c = Case([50, 60], 2, 1, 64, 64, BF16)
    o = decay.attn(c.q, c.k, c.v, c.log, c.cu_gpu, c.scale)
    beyond = torch.tensor([-7, 50, 4000], dtype=torch.int32, device="cuda")
    assert torch.equal(decay.attn(c.q, c.k, c.v, c.log, beyond, c.scale), o)


def test_refusals(decay):
    c = Case([20, 30], 2, 2, 16, 8, BF16)
    args = (c.q, c.k, c.v, c.log)
    bad = [
        lambda: decay.attn(c.q[:, :3], c.k, c.v, c.log),
        lambda: decay.attn(c.q.half(), c.k, c.v, c.log),
        lambda: decay.attn(c.q, c.k.float(), c.v, c.log),
        lambda: decay.attn(c.q, c.k[:10], c.v, c.log),
        lambda: decay.attn(c.q.transpose(1, 2).contiguous().transpose(1, 2), c.k, c.v, c.log),
        lambda: decay.attn(c.q, c.k, c.v, c.log.double()),
        lambda: decay.attn(c.q, c.k, c.v, c.log[:1]),
        lambda: decay.attn(*args, cu_seqlens=c.cu_gpu.long()),
        lambda: decay.attn(*args, cu_seqlens=c.cu_gpu.cpu()),
        lambda: decay.attn(*args, seqs=3),
        lambda: decay.attn(*args, seqs=0),
        lambda: decay.attn(*args, c.cu_gpu, state_in=c.s0[:1]),
        lambda: decay.attn(*args, c.cu_gpu, state_in=c.s0.bfloat16()),
        lambda: decay.attn(*args, c.cu_gpu, state_in=c.s0, state_out=draw((3, 2, 16, 8), 1), slots=torch.zeros(2, dtype=torch.int32, device="cuda")),
        lambda: decay.attn(*args, c.cu_gpu, state_in=c.s0, slots=torch.zeros(3, dtype=torch.int32, device="cuda")),
        lambda: decay.attn(*args, c.cu_gpu, out=torch.empty_like(c.q)),
        lambda: decay.attn_bwd(*args, c.do[:, :2], c.cu_gpu),
        lambda: decay.attn_bwd(*args, c.do, c.cu_gpu, out=(c.q, torch.empty_like(c.k), torch.empty_like(c.q))),
        lambda: decay.step(*args, c.s0),
        lambda: decay.step(*args, c.s0, slots=torch.zeros(50, dtype=torch.int64, device="cuda")),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail("call %d was taken" % i)
    from sub_linear_memory_gb300 import binding

    with pytest.raises(binding.SlimError):
        decay.attn(c.q, c.k, draw((50, 2, 16), 9, BF16), c.log, out=c.q)
    with pytest.raises(binding.SlimError):
        decay.attn_bwd(*args, c.do, c.cu_gpu, g_in=c.g_in, g_out=c.g_in)
    with pytest.raises(binding.SlimError):
        decay.attn(draw((4, 2, 257), 9, BF16), draw((4, 2, 257), 9, BF16), draw((4, 2, 8), 9, BF16), c.log)
