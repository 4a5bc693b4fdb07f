"""Decay attention, group norm with a gate, and AdamW, as they are measured.

The mixing part of a layer whose linear attention forgets, and the update of its weights:

``attn``   linear attention with a decay lambda_h = exp(g_h) for each key-value head over packed
           sequences, with grouped query heads: S_t = lambda S_(t-1) + k_t v_t^T, o_t = scale q_t^T S_t;
           ``train`` is the same with its gradients, ``step`` the form for one token of each sequence;
``norm``   group norm of each row's heads, times the SiLU of a gate, and its gradients;
``adamw``  one AdamW step over many tensors, states in 32 bits or in the 8-bit form (e4m3 codes, a
           power-of-two scale for each 128 values).  There the second moment is held as its root r,
           and both are rounded up or down at random: element i of tensor k takes the word i % 4 of
           Philox4x32-10 with counter (i / 4, k, 0, step) and the seed as key, its low 16 bits for m
           and its high 16 for r.  r > 0 is never rounded to 0.

Values held in 8 bits are returned as bf16, which holds each exactly.  Rows are tokens, columns are
heads * d (1024 for 16 heads of 64, 1536 for 12 heads of 128).
"""
import math
import random

import torch

own = False

EPS = 1e-5
CHUNK = 256
BLOCK = 128
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
LR, BETAS, ADAM_EPS, DECAY = 1e-3, (0.9, 0.95), 1e-8, 0.1


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # one short prompt, its state kept for the tokens that follow: latency
        dict(name="attn_short", op="attn", seqs=1, tokens=17, heads=16, groups=1, d=64, dv=64, dtype="bf16", state=True),
        # prompts of many lengths packed into one call, grouped heads, each going on from a cached state
        dict(name="attn_packed", op="attn", seqs=37, tokens=24001, heads=4, groups=3, d=128, dv=128, dtype="bf16", state=True),
        # one document of 2^20 tokens, 8 heads
        dict(name="attn_l1m", op="attn", seqs=1, tokens=1 << 20, heads=8, groups=1, d=64, dv=64, dtype="bf16", state=True),
        # training on 2 sequences of 32768 tokens, 16 heads of 64
        dict(name="train_l32k", op="train", seqs=2, tokens=65536, heads=16, groups=1, d=64, dv=64, dtype="bf16", state=False),
        # the same tokens as documents of many lengths, 12 query heads of 128 on 4 key-value heads
        dict(name="train_packed", op="train", seqs=61, tokens=65536, heads=4, groups=3, d=128, dv=128, dtype="bf16", state=False),
        # a small model in fp32 at odd sizes, trained in windows: the state's gradient too
        dict(name="train_ragged_f32", op="train", seqs=5, tokens=4099, heads=3, groups=2, d=40, dv=24, dtype="fp32", state=True),
        # one token of each of 128 sequences
        dict(name="step_tokens", op="step", seqs=128, heads=16, groups=1, d=64, dv=64, dtype="bf16", slots=0),
        # the same with grouped heads of 128, states in a cache of 200 places
        dict(name="step_slots", op="step", seqs=129, heads=4, groups=3, d=128, dv=128, dtype="bf16", slots=200),
        # the norm of 128 tokens' heads
        dict(name="norm_tokens", op="norm", rows=128, cols=1024, groups=16, dtype="bf16", gate=True, train=False),
        # training on 2 sequences of 32768 tokens
        dict(name="norm_train_l32k", op="norm", rows=65536, cols=1024, groups=16, dtype="bf16", gate=True, train=True),
        # the weights of four layers (d_model 1024, d_ff 4096), states in 8 bits
        dict(name="adamw8_layers", op="adamw", tensors=32, largest=1 << 22, bits=8, dtype="fp32"),
        # a small model's tensors at odd sizes, bf16 gradients, states in 32 bits
        dict(name="adamw32_ragged", op="adamw", tensors=19, largest=66001, bits=32, dtype="bf16"),
    ]


MOST_TOKEN_HEADS = 1 << 21  # query-head rows of 64 columns
MOST_ELEMENTS = 65536 * 1024
MOST_WEIGHTS = 1 << 25


def _log_size(rng, lo, hi, step=1):
    x = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, x // step * step if x >= step else x))


def draw(rng):
    op = rng.choice(["attn", "attn", "train", "train", "step", "norm", "norm", "adamw", "adamw"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op in ("attn", "train", "step"):
        d = rng.choice([64, 64, 128, 128, 0])
        d, dv = (d, d) if d else (rng.randint(8, 160), rng.randint(8, 160))
        case = dict(op=op, heads=rng.randint(1, 8), groups=rng.choice([1, 1, 2, 3, 4]), d=d, dv=dv, dtype=dtype)
        if op == "step":
            case["seqs"] = _log_size(rng, 1, 512)
            case["slots"] = rng.choice([0, case["seqs"] + rng.randint(1, 64)])
            return case
        slow = dtype == "fp32" or d != dv or d % 64
        most = MOST_TOKEN_HEADS // (case["heads"] * case["groups"]) * 64 // max(d, dv) // (16 if slow else 4)
        case["tokens"] = _log_size(rng, 1, most)
        case["seqs"] = min(case["tokens"], _log_size(rng, 1, 100))
        case["state"] = rng.random() < 0.5
        return case
    if op == "norm":
        while True:
            groups, width = _log_size(rng, 1, 64), _log_size(rng, 8, 512, rng.choice([1, 8, 32]))
            rows = _log_size(rng, 1, 65536)
            if groups * width <= 8192 and rows * groups * width <= MOST_ELEMENTS:
                return dict(op=op, rows=rows, cols=groups * width, groups=groups, dtype=dtype, gate=rng.random() < 0.8,
                            train=rng.random() < 0.6)
    while True:
        case = dict(op=op, tensors=_log_size(rng, 1, 60), largest=_log_size(rng, 1, 1 << 23), bits=rng.choice([8, 32]), dtype=dtype)
        if sum(_tensor_sizes(case)) <= MOST_WEIGHTS:
            return case


def _lengths(case):
    """Lengths of a case's sequences, whole numbers that add up to its tokens: equal, or spread as documents are."""
    n, tokens = case["seqs"], case["tokens"]
    if n == 1 or (n == 2 and tokens % 2 == 0):
        return [tokens // n] * n
    rng = random.Random(tokens * 131 + n)
    share = [math.exp(rng.gauss(0, 1.2)) for _ in range(n)]
    cuts, total, run_ = [0], sum(share), 0.0
    for s in share[:-1]:
        run_ += s
        cuts.append(int(tokens * run_ / total))
    cuts.append(tokens)
    return [b - a for a, b in zip(cuts, cuts[1:])]


def _tensor_sizes(case):
    """Elements of a case's tensors: a layer's eight again and again (four matrices, four vectors), or a spread of sizes."""
    n, top = case["tensors"], case["largest"]
    if top == 1 << 22:
        return [(1 << 22, 1 << 20, 1 << 22, 1 << 22, 1024, 1024, 1024, 1024)[i % 8] for i in range(n)]
    rng = random.Random(top * 17 + n)
    return [top] + [max(1, int(top * math.exp(-rng.uniform(0, 6)))) for _ in range(n - 1)]


def _spans(case):
    """Where each tensor lies in one buffer that holds them all, every one on a place of its own of whole
    groups of four blocks, and the buffer's size."""
    spans, at = [], 0
    for n in _tensor_sizes(case):
        spans.append((at, at + n))
        at += -(-n // (4 * BLOCK)) * 4 * BLOCK
    return spans, at


def _held_parts(stored, spans):
    """The codes and scales of each tensor in those of the buffer."""
    codes, scales = stored
    up = lambda b, a: a + -(-(b - a) // BLOCK) * BLOCK
    return [(codes[:, a:up(b, a)], scales[:, a // BLOCK:a // BLOCK + -(-(b - a) // (4 * BLOCK)) * 4]) for a, b in spans]


def work(case):
    op = case["op"]
    size = 4 if case["dtype"] == "fp32" else 2
    if op == "adamw":
        n = sum(_tensor_sizes(case))
        held = 2 * 2 * (1 + 1 / BLOCK) if case["bits"] == 8 else 2 * 2 * 4  # both moments in and out
        return {"bytes": n * (size + 8 + held), "flops": 15.0 * n}
    if op == "norm":
        n = case["rows"] * case["cols"]
        arrays = 3 if case["gate"] else 2  # x (and the gate) in, y out
        moved, flops = arrays * size * n + 8 * case["cols"], 12.0 * n
        if case["train"]:  # dy, x (and the gate) in, dx (and the gate's gradient) out
            moved, flops = moved + (5 if case["gate"] else 3) * size * n + 12 * case["cols"], flops + 25.0 * n
        return {"bytes": moved, "flops": flops}
    heads, q_heads, d, dv = case["heads"], case["heads"] * case["groups"], case["d"], case["dv"]
    per_state = heads * d * dv
    if op == "step":
        n = case["seqs"]
        moved = n * (8 * per_state + size * (q_heads * (d + dv) + heads * (d + dv)))
        return {"bytes": moved, "flops": n * (3.0 * per_state + 2.0 * q_heads * d * dv)}
    tokens = case["tokens"]
    rows_in = tokens * size * (q_heads * d + heads * (d + dv))
    moved, flops = rows_in + tokens * size * q_heads * dv, 2.0 * tokens * d * dv * (heads + q_heads)
    if case["state"]:
        moved += 8 * case["seqs"] * per_state
    if op == "train":
        moved += 2 * rows_in + tokens * size * q_heads * dv  # q, k, v and the output's gradient in, dq, dk, dv out
        flops += 2.0 * tokens * d * dv * (2 * q_heads + 3 * heads)
        if case["state"]:
            moved += 12 * case["seqs"] * per_state
    return {"bytes": moved, "flops": flops}


# ---- inputs ----------------------------------------------------------------

def _power(e):
    """2^e in fp32 for integers -126 <= e <= 127, by its bits (exp2 may round)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _blocks(x):
    """A flat fp32 tensor as rows of 128, the last one filled with zeros, and each row's exponent: the smallest
    e in [-117, 120] with every magnitude at most 448 * 2^e."""
    nb = -(-x.numel() // BLOCK)
    pad = torch.zeros(nb * BLOCK, dtype=torch.float32, device=x.device)
    pad[:x.numel()] = x
    t = pad.view(nb, BLOCK)
    top = t.abs().amax(dim=1).contiguous()
    return t, (((top.view(torch.int32) + 0x1FFFFF) >> 23) - 135).clamp(-117, 120)


def _stored(values, e):
    """codes [1, 128 * blocks] and scales [1, 4 * ceil(blocks / 4)] of scaled values that are e4m3 numbers."""
    nb = e.numel()
    scales = torch.full((1, -(-nb // 4) * 4), 127, dtype=torch.uint8, device=e.device)
    scales[0, :nb] = (e + 127).to(torch.uint8)
    return values.to(torch.float8_e4m3fn).view(1, nb * BLOCK), scales


def _quantized(x):
    t, e = _blocks(x)
    return _stored(t * _power(-e)[:, None], e)


def _values(codes, scales, n, dtype=torch.float32):
    """The values that codes and scales stand for (plain form)."""
    nb = codes.shape[1] // BLOCK
    s = _power(scales[0, :nb].to(torch.int32) - 127)
    return (codes.reshape(nb, BLOCK).to(torch.float32) * s[:, None]).view(-1)[:n].to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")
    op, dtype = case["op"], DTYPES[case["dtype"]]
    state = {"case": case}
    if op == "adamw":
        # moments as after some steps, of gradients whose sizes differ from element to element
        spans, total = _spans(case)
        level = torch.zeros(total, device="cuda")
        for a, b in spans:
            level[a:b] = 1e-3 * torch.exp(randn(b - a))
        state.update(count=20, seed=seed, p=0.03 * randn(total) * (level > 0), g=(level * randn(total)).to(dtype))
        m, v = 0.3 * level * randn(total), (level * (1 + 0.1 * randn(total))).square()
        if case["bits"] == 8:
            state["m"], state["v"] = _quantized(m), _quantized(v.sqrt())
        else:
            state["m"], state["v"] = m, v
        return state
    if op == "norm":
        rows, cols = case["rows"], case["cols"]
        level = torch.exp(0.5 * randn(rows, case["groups"], 1))  # heads differ in size, and have a mean of their own
        x = level * (randn(rows, case["groups"], cols // case["groups"]) + 0.3 * randn(rows, case["groups"], 1))
        state.update(x=x.view(rows, cols).to(dtype), gamma=1 + 0.2 * randn(cols), beta=0.1 * randn(cols))
        state["gate"] = (1.5 * randn(rows, cols)).to(dtype) if case["gate"] else None
        if case["train"]:
            state["dy"] = (1e-3 * randn(rows, cols)).to(dtype)
        return state
    heads, q_heads, d, dv, seqs = case["heads"], case["heads"] * case["groups"], case["d"], case["dv"], case["seqs"]
    rows = seqs if op == "step" else case["tokens"]
    # what one projection gives: q, k and v of a token beside one another
    qkv = randn(rows, q_heads * d + heads * (d + dv)).to(dtype)
    state["q"] = qkv[:, :q_heads * d].view(rows, q_heads, d)
    state["k"] = qkv[:, q_heads * d:q_heads * d + heads * d].view(rows, heads, d)
    state["v"] = qkv[:, q_heads * d + heads * d:].view(rows, heads, dv)
    state["scale"] = d ** -0.5
    # lambda from 3/4 to 1 - 2^-12
    away = torch.linspace(2, 12, heads, dtype=torch.float64) if heads > 1 else torch.tensor([7.0], dtype=torch.float64)
    state["log_decay"] = torch.log1p(-(2.0 ** -away)).to(torch.float32).cuda()
    if op == "step":
        places = case["slots"] or seqs
        state["state"] = randn(places, heads, d, dv)
        state["slots"] = torch.randperm(places, generator=g, device="cuda")[:seqs].to(torch.int32) if case["slots"] else None
        return state
    state["lengths"] = _lengths(case)
    state["cu_seqlens"] = torch.tensor([0] + state["lengths"]).cumsum(0).to(torch.int32).cuda()
    state["state"] = randn(seqs, heads, d, dv) if case["state"] else None
    if op == "train":
        state["do"] = (1e-3 * randn(rows, q_heads, dv)).to(dtype)
        state["g_in"] = 1e-3 * randn(seqs, heads, d, dv) if case["state"] else None
    return state


# ---- one pass --------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(state):
    from sub_linear_memory_gb300 import decay, norm, optim, q8

    case = state["case"]
    op = case["op"]
    if op == "adamw":
        spans, total = _spans(case)
        eight = case["bits"] == 8
        if "optimizer" not in state:  # as a user's program does, once
            parts = lambda t: [t[a:b] for a, b in spans]
            held = lambda t: [q8.Q8(*h, b - a) for h, (a, b) in zip(_held_parts(t, spans), spans)] if eight else parts(t)
            state["optimizer"] = optim.AdamW(parts(state["p"]), lr=LR, betas=BETAS, eps=ADAM_EPS, weight_decay=DECAY, bits=case["bits"],
                                             seed=state["seed"], m=held(state["m"]), v=held(state["v"]), count=state["count"])
            state["grads"] = parts(state["g"])
        state["optimizer"].step(state["grads"])
        m, v = (q8.dequantize(q8.Q8(*state[k], total)).view(-1) if eight else state[k] for k in "mv")
        return {"p": state["p"], "m": m, "v": v}
    if op == "norm":
        args = (state["x"], state["gamma"], state["beta"], case["groups"], state["gate"], EPS)
        out = {"y": norm.group_norm(*args)}
        if case["train"]:
            out["dx"], out["dgate"], out["dgamma"], out["dbeta"] = norm.group_norm_bwd(state["dy"], *args)
        return out
    qkv = (state["q"], state["k"], state["v"], state["log_decay"])
    if op == "step":
        return {"o": decay.step(*qkv, state["state"], slots=state["slots"], scale=state["scale"]), "state": state["state"]}
    s, kw = state["state"], dict(cu_seqlens=state["cu_seqlens"], scale=state["scale"])
    if op == "attn":
        return {"o": decay.attn(*qkv, state_in=s, state_out=s, **kw), "state": s}
    out = {}
    if s is not None:
        out["state"], out["dstate"] = torch.empty_like(s), torch.empty_like(s)
    out["o"] = decay.attn(*qkv, state_in=s, state_out=out.get("state"), **kw)
    out["dq"], out["dk"], out["dv"] = decay.attn_bwd(*qkv, state["do"], state_in=s, g_in=state["g_in"], g_out=out.get("dstate"), **kw)
    return out


def _mix(a, b, c, log_decay, start):
    """out_i = sum over j <= i of lambda^(i-j) (a_i . b_j) c_j + lambda^(i+1) a_i start, and the state after the last row.

    a [H, Ga, L, x], b [H, Gb, L, x], c [H, Gb, L, y], start [H, x, y]; Ga or Gb is 1, and the Gb products are added."""
    h, ga, length, x = a.shape
    gb, y = b.shape[1], c.shape[3]
    n = -(-length // CHUNK)
    pad = lambda t: torch.nn.functional.pad(t, (0, 0, 0, n * CHUNK - length)).view(h, t.shape[1], n, CHUNK, t.shape[3])
    a, b, c = pad(a), pad(b), pad(c)
    g = log_decay.double()
    at = torch.arange(CHUNK, device=a.device, dtype=torch.float64)
    apart = at[:, None] - at
    within = torch.where(apart >= 0, torch.exp(g[:, None, None] * apart.clamp(min=0)), 0.0).float()
    ahead = torch.exp(g[:, None] * (CHUNK - 1 - at)).float()
    since = torch.exp(g[:, None] * (at + 1)).float()
    gained = ((b * ahead[:, None, None, :, None]).transpose(3, 4) @ c).sum(1)  # [H, n, x, y]
    # states before each chunk, and behind the last row, which ends the last chunk early
    carried, before, over = start.double(), [], torch.exp(g * CHUNK)[:, None, None]
    for i in range(n):
        before.append(carried)
        if i < n - 1:
            carried = carried * over + gained[:, i]
    rest = length - (n - 1) * CHUNK
    tail = (b[:, :, -1, :rest] * torch.exp(g[:, None] * (rest - 1 - at[:rest])).float()[:, None, :, None]).transpose(2, 3) @ c[:, :, -1, :rest]
    end = carried * torch.exp(g * rest)[:, None, None] + tail.sum(1)
    before = torch.stack(before, 1).float()[:, None]  # [H, 1, n, x, y]
    out = ((a @ b.transpose(3, 4)) * within[:, None, None]) @ c
    if gb > 1:
        out = out.sum(1, keepdim=True)
    out = out + (a @ before) * since[:, None, None, :, None]
    return out.view(h, ga, n * CHUNK, y)[:, :, :length], end.float()


def _grouped(t, heads):
    """[L, heads * G, x] -> [heads, G, L, x] in fp32."""
    return t.float().view(t.shape[0], heads, -1, t.shape[2]).permute(1, 2, 0, 3)


def _rows(t, dtype):
    """[heads, G, L, x] -> [L, heads * G, x]."""
    return t.permute(2, 0, 1, 3).reshape(t.shape[2], -1, t.shape[3]).to(dtype)


def _run_plain(state):
    case = state["case"]
    op = case["op"]
    if op == "adamw":
        return _adamw_plain(state)
    if op == "norm":
        return _norm_plain(state)
    dtype, heads, scale, g = DTYPES[case["dtype"]], case["heads"], state["scale"], state["log_decay"]
    if op == "step":
        at = state["slots"].long() if state["slots"] is not None else slice(None)
        q = state["q"].float().view(case["seqs"], heads, case["groups"], case["d"])
        s = state["state"][at] * torch.exp(g.double()).float()[None, :, None, None]
        s = s + state["k"].float()[..., None] * state["v"].float()[:, :, None, :]
        state["state"][at] = s
        return {"o": ((q @ s) * scale).reshape(case["seqs"], -1, case["dv"]).to(dtype), "state": state["state"]}
    outs = {k: [] for k in (("o", "dq", "dk", "dv") if op == "train" else ("o",))}
    ends, dstarts, first = [], [], 0
    for i, length in enumerate(state["lengths"]):
        q, k, v = (_grouped(state[t][first:first + length], heads) for t in "qkv")
        start = state["state"][i] if state["state"] is not None else torch.zeros(heads, case["d"], case["dv"], device=q.device)
        o, end = _mix(q, k, v, g, start)
        outs["o"].append(_rows(o * scale, dtype))
        ends.append(end)
        if op == "train":
            do = _grouped(state["do"][first:first + length], heads)
            ahead = state["g_in"][i] / scale if state["g_in"] is not None else torch.zeros_like(start)
            turn = lambda t: t.flip(2)
            dq, _ = _mix(do, v, k, g, start.transpose(1, 2))
            # behind a row the state has not yet forgotten for that row: the gradient that comes from later rows has one decay less
            less = torch.exp(-g.double()).float()[:, None, None]
            dv, dstart = _mix(turn(k), turn(q), turn(do), g, ahead * less)
            dk, _ = _mix(turn(v), turn(do), turn(q), g, (ahead * less).transpose(1, 2))
            for name, t in (("dq", dq), ("dk", turn(dk)), ("dv", turn(dv))):
                outs[name].append(_rows(t * scale, dtype))
            dstarts.append(dstart * torch.exp(g.double()).float()[:, None, None] * scale)
        first += length
    out = {k: torch.cat(t) for k, t in outs.items()}
    if state["state"] is not None:
        out["state"] = torch.stack(ends)
        if op == "train":
            out["dstate"] = torch.stack(dstarts)
        else:
            state["state"].copy_(out["state"])
    elif op == "attn":
        out["state"] = None
    return out


def _norm_plain(state):
    case = state["case"]
    dtype, shape = DTYPES[case["dtype"]], (case["rows"], case["groups"], -1)
    x = state["x"].float().view(shape)
    mean = x.mean(2, keepdim=True)
    centred = x - mean
    rstd = torch.rsqrt(centred.square().mean(2, keepdim=True) + EPS)
    n = (centred * rstd).view(case["rows"], -1)
    y = n * state["gamma"] + state["beta"]
    z = state["gate"].float() if state["gate"] is not None else None
    s = 1 / (1 + torch.exp(-z)) if z is not None else None
    out = {"y": (y * z * s if z is not None else y).to(dtype)}
    if case["train"]:
        dy = state["dy"].float()
        dn = dy * z * s if z is not None else dy
        out["dgate"] = (dy * y * s * (1 + z * (1 - s))).to(dtype) if z is not None else None
        out["dgamma"], out["dbeta"] = (dn.double() * n).sum(0).float(), dn.sum(0, dtype=torch.float64).float()
        h, nv = (dn * state["gamma"]).view(shape), n.view(shape)
        dx = rstd * (h - h.mean(2, keepdim=True) - nv * (h * nv).mean(2, keepdim=True))
        out["dx"] = dx.view(case["rows"], -1).to(dtype)
    return out


def _philox(first, tensor, step, seed):
    """Words of Philox4x32-10 (Salmon et al., SC 2011) for counters (first + i, tensor, 0, step): int64 [n, 4]."""
    mask = 0xFFFFFFFF
    c = [first, torch.full_like(first, tensor), torch.zeros_like(first), torch.full_like(first, step)]
    k0, k1 = seed & mask, (seed >> 32) & mask
    high = lambda m, t: (((t >> 16) * m + (((t & 0xFFFF) * m) >> 16)) >> 16) & mask  # of a 32 x 32 bit product
    for r in range(10):
        h0, l0 = high(0xD2511F53, c[0]), (c[0] * 0xD2511F53) & mask
        h1, l1 = high(0xCD9E8D57, c[2]), (c[2] * 0xCD9E8D57) & mask
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & mask, (k1 + 0xBB67AE85) & mask
    return torch.stack(c, 1)


def _rounded_at_random(x, bits16):
    """codes and scales of x with each value rounded up with the probability of its place between two codes."""
    t, e = _blocks(x)
    w = t.abs() * _power(-e)[:, None]
    small = w < 2.0 ** -6  # equal steps there: as between 2^-6 and 2^-5
    r = torch.zeros_like(t, dtype=torch.int32).view(-1)
    r[:x.numel()] = (bits16 << 4).to(torch.int32)
    w = torch.where(small, w + 2.0 ** -6, w)
    w = ((w.view(torch.int32) + r.view_as(t)) & ~0xFFFFF).view(torch.float32)
    w = torch.where(small, w - 2.0 ** -6, w).clamp(max=448)
    return w, t, e


def _adamw_plain(state):
    b1, b2 = BETAS
    state["count"] += 1
    t = state["count"]
    c1, c2 = 1 - b1 ** t, 1 - b2 ** t
    eight = state["case"]["bits"] == 8
    spans, total = _spans(state["case"])
    for k, (first, last) in enumerate(spans):
        n, g, p = last - first, state["g"][first:last].float(), state["p"][first:last]
        if eight:
            held = [_held_parts(state[s], spans)[k] for s in "mv"]
            m, v = _values(*held[0], n), _values(*held[1], n).square()
        else:
            m, v = state["m"][first:last], state["v"][first:last]
        m1, v1 = m * b1 + g * (1 - b1), v * b2 + g * g * (1 - b2)
        p.mul_(1 - LR * DECAY)
        p.sub_(m1 / ((v1 / c2).sqrt() + ADAM_EPS) * (LR / c1))
        if eight:
            words = _philox(torch.arange(-(-n // 4), device=p.device), k, t, state["seed"]).view(-1)[:n]
            w, x, e = _rounded_at_random(m1, words & 0xFFFF)
            r, y, f = _rounded_at_random(v1.sqrt(), words >> 16)
            new = _stored(torch.copysign(w, x), e), _stored(torch.where(y > 0, r.clamp(min=2.0 ** -9), r), f)
            for old, now in zip(held, new):
                old[0].copy_(now[0])
                old[1].copy_(now[1])
        else:
            m.copy_(m1)
            v.copy_(v1)
    m, v = (_values(*state[s], total, torch.bfloat16) if eight else state[s] for s in "mv")
    return {"p": state["p"], "m": m, "v": v}


# ---- the same in 64 bits, from the definitions --------------------------------

def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "adamw":
        return _exact_adamw(state)
    if op == "norm":
        return _exact_norm(state)
    heads, groups, scale = case["heads"], case["groups"], state["scale"]
    lam = torch.exp(state["log_decay"].double())
    q, k, v = (state[t].double() for t in "qkv")
    if op == "step":
        at = state["slots"].long() if state["slots"] is not None else torch.arange(case["seqs"], device=q.device)
        s = state["state"].double()
        s[at] = lam[:, None, None] * s[at] + torch.einsum("nhi,nhj->nhij", k, v)
        read = s[at].repeat_interleave(groups, 1)
        return {"o": scale * torch.einsum("nhi,nhij->nhj", q, read), "state": s}
    g = state["log_decay"].double().repeat_interleave(groups)
    k, v = k.repeat_interleave(groups, 1), v.repeat_interleave(groups, 1)  # every query head with its own copy
    o, dq, dk, dv, ends, dstarts = torch.zeros(q.shape[0], q.shape[1], case["dv"], dtype=torch.float64, device=q.device), [], [], [], [], []
    if op == "train":
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    step, first = 384, 0
    for i, length in enumerate(state["lengths"]):
        s = torch.zeros(heads * groups, case["d"], case["dv"], dtype=torch.float64, device=q.device)
        if state["state"] is not None:
            s = state["state"][i].double().repeat_interleave(groups, 0)
        kept = []
        spans = [slice(a, min(a + step, first + length)) for a in range(first, first + length, step)]
        for at in spans:
            n = at.stop - at.start
            j = torch.arange(n, dtype=torch.float64, device=q.device)
            dec = torch.tril(torch.exp(g[:, None, None] * (j[:, None] - j).clamp(min=0)))
            kept.append((s, dec, j))
            o[at] = torch.einsum("hij,jhd->ihd", torch.einsum("ihd,jhd->hij", q[at], k[at]) * dec, v[at])
            o[at] += torch.einsum("ihd,hde->ihe", q[at], s) * torch.exp(g * (j[:, None] + 1))[:, :, None]
            s = s * torch.exp(g * n)[:, None, None] + torch.einsum("jhd,jhe->hde", k[at] * torch.exp(g * (n - 1 - j[:, None]))[:, :, None], v[at])
            kept[-1] = (kept[-1][0], None, None) if op == "train" else None
        ends.append(s[::groups])
        if op != "train":
            first += length
            continue
        do = state["do"].double()
        # the gradient with respect to the state behind the rows done: of each query head's copy
        back = torch.zeros_like(s)
        if state["g_in"] is not None:
            back[::groups] = state["g_in"][i].double() / scale  # one copy has it all: only the sum over a group counts
        for at, (s, _, _) in zip(reversed(spans), reversed(kept)):
            n = at.stop - at.start
            j = torch.arange(n, dtype=torch.float64, device=q.device)
            dec = torch.tril(torch.exp(g[:, None, None] * (j[:, None] - j).clamp(min=0)))
            to_end, from_start = torch.exp(g * (n - 1 - j[:, None]))[:, :, None], torch.exp(g * (j[:, None] + 1))[:, :, None]
            da = torch.einsum("ihd,jhd->hij", do[at], v[at]) * dec
            pa = torch.einsum("ihd,jhd->hij", q[at], k[at]) * dec
            dq[at] = torch.einsum("hij,jhd->ihd", da, k[at]) + torch.einsum("ihe,hde->ihd", do[at], s) * from_start
            dk[at] = torch.einsum("hij,ihd->jhd", da, q[at]) + torch.einsum("jhe,hde->jhd", v[at], back) * to_end
            dv[at] = torch.einsum("hij,ihe->jhe", pa, do[at]) + torch.einsum("jhd,hde->jhe", k[at], back) * to_end
            back = back * torch.exp(g * n)[:, None, None] + torch.einsum("ihd,ihe->hde", q[at] * from_start, do[at])
        dstarts.append(scale * back.view(heads, groups, case["d"], case["dv"]).sum(1))
        first += length
    out = {"o": scale * o}
    if state["state"] is not None:
        out["state"] = torch.stack(ends)
    if op == "train":
        shared = lambda t: t.view(t.shape[0], heads, groups, -1).sum(2)
        out.update(dq=scale * dq, dk=scale * shared(dk), dv=scale * shared(dv))
        if state["state"] is not None:
            out["dstate"] = torch.stack(dstarts)
    return out


def _exact_norm(state):
    case = state["case"]
    parts = lambda t: t.view(case["rows"], case["groups"], -1)
    x = parts(state["x"].double())
    var, mean = torch.var_mean(x, dim=2, unbiased=False, keepdim=True)
    root = 1 / torch.sqrt(var + EPS)
    n = ((x - mean) * root).reshape(case["rows"], -1)
    gamma, y = state["gamma"].double(), n * state["gamma"].double() + state["beta"].double()
    open_, slope = 1.0, None
    if state["gate"] is not None:
        z = state["gate"].double()
        s = torch.sigmoid(z)
        open_, slope = z * s, s + z * s * (1 - s)
    out = {"y": y * open_}
    if case["train"]:
        dy = state["dy"].double()
        out["dgate"] = dy * y * slope if slope is not None else None
        out["dgamma"], out["dbeta"] = (dy * open_ * n).sum(0), (dy * open_).sum(0)
        h, nv = parts(dy * open_ * gamma), parts(n)
        out["dx"] = (root * (h - h.mean(2, keepdim=True) - nv * (h * nv).mean(2, keepdim=True))).reshape(case["rows"], -1)
    return out


def _exact_read(codes, scales, n):
    """Stored values bit by bit: sign, four exponent bits (bias 7), three fraction bits, times 2^(scale - 127)."""
    raw = codes.view(torch.uint8).view(-1)[:n].to(torch.int32)
    exponent, fraction = (raw >> 3) & 15, (raw & 7).double()
    size = torch.where(exponent == 0, fraction / 512, torch.ldexp(1 + fraction / 8, exponent - 7))
    block = torch.arange(n, device=codes.device) // BLOCK
    return torch.ldexp(torch.where(raw >= 128, -size, size), scales.view(-1)[block].to(torch.int32) - 127)


def _exact_held(x, bits16, never_zero):
    """x as the 8-bit form holds it, each magnitude rounded down to a step after bits16 / 2^16 of a step was added."""
    out = x.clone()
    for rows in range(0, x.numel(), 1 << 22):
        part = x[rows:rows + (1 << 22)]
        n = part.numel()
        pad = torch.nn.functional.pad(part.abs(), (0, -n % BLOCK)).view(-1, BLOCK)
        f, p = torch.frexp(pad.amax(1, keepdim=True))
        e = torch.where(f == 0, torch.full_like(p, -117), (p - 9 + (f > 0.875)).clamp(-117, 120))
        w = torch.ldexp(pad, -e)
        step = (torch.frexp(w)[1] - 1).clamp(min=-6) - 3
        add = torch.nn.functional.pad(bits16[rows:rows + (1 << 22)], (0, -n % BLOCK)).view(-1, BLOCK).double() / 65536
        w = torch.ldexp(torch.floor(torch.ldexp(w, -step) + add), step).clamp(max=448)
        if never_zero:
            w = torch.where(pad > 0, w.clamp(min=2.0 ** -9), w)
        out[rows:rows + (1 << 22)] = torch.copysign(torch.ldexp(w, e).view(-1)[:n], part)
    return out


def _exact_adamw(state):
    b1, b2 = BETAS
    t = state["count"] + 1
    eight = state["case"]["bits"] == 8
    spans, total = _spans(state["case"])
    p, g = state["p"].double(), state["g"].double()
    if eight:
        m, v = _exact_read(*state["m"], total), _exact_read(*state["v"], total) ** 2
    else:
        m, v = state["m"].double(), state["v"].double()
    m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g ** 2
    p = p - LR * (m / (1 - b1 ** t) / (torch.sqrt(v / (1 - b2 ** t)) + ADAM_EPS) + DECAY * p)
    if eight:
        v = torch.sqrt(v)
        for k, (first, last) in enumerate(spans):
            n = last - first
            words = _philox(torch.arange(-(-n // 4), device=p.device), k, t, state["seed"]).view(-1)[:n]
            m[first:last] = _exact_held(m[first:last], words & 0xFFFF, False)
            v[first:last] = _exact_held(v[first:last], words >> 16, True)
    return {"p": p, "m": m, "v": v}
