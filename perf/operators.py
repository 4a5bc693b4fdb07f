"""The 8-bit layer operators, as they are measured.

Around the causal linear attention a layer has a norm with the residual's addition, dense
projections, an activation, and the rows that the backward pass needs of each.  These
cases run the library's 8-bit forms of them: ``rms_norm`` (residual + root-mean-square
norm, output in 8 bits, backward from an 8-bit or a full checkpoint), ``matmul`` (8-bit
products with a scale for each block of 128) and the 8-bit checkpoints and their use
(``gelu`` / ``gelu_bwd``, ``quantize``, ``wgrad``).

An 8-bit tensor is e4m3 codes and power-of-two scales, one for each row (or each 128 rows
of a weight) and each 128 columns: value = code * 2^(scale - 127), with the smallest
exponent e in [-117, 120] for which the block's largest magnitude is at most 448 * 2^e; a
block with an infinity or a NaN has scale 255 and is NaN throughout.  Codes of a row are
padded with zeros to whole blocks, scales to groups of four.  Values held in 8 bits are
returned as bf16, which holds every code * 2^e exactly.

Rows are tokens (batch * length), columns are heads * d (1024 for 16 heads of 64, 1536
for 12 heads of 128) or the feed-forward width of four times that.
"""
import math

import torch

own = False

BLOCK = 128
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # one decode step of 128 sequences: the norm before the projections
        dict(name="norm_tokens", op="norm", rows=128, cols=1024, dtype="bf16", train=False, checkpoint=False),
        # training on 2 sequences of 32768: forward, and backward from the 8-bit checkpoint
        dict(name="norm_train_l32k", op="norm", rows=65536, cols=1024, dtype="bf16", train=True, checkpoint=True),
        # a ragged batch at a width that is no multiple of the block, fp32 rows kept in full
        dict(name="norm_train_ragged", op="norm", rows=4099, cols=1000, dtype="fp32", train=True, checkpoint=False),
        # one token through the feed-forward block's second projection
        dict(name="matmul_one_token", op="matmul", rows=1, n=1024, k=4096, dtype="bf16"),
        # one decode step of 128 sequences through the first one
        dict(name="matmul_tokens", op="matmul", rows=128, n=4096, k=1024, dtype="bf16"),
        # the first projection over 2 sequences of 32768
        dict(name="matmul_l32k", op="matmul", rows=65536, n=4096, k=1024, dtype="bf16"),
        # odd sizes in every direction, fp32 result (logits)
        dict(name="matmul_ragged_f32", op="matmul", rows=4099, n=1001, k=1336, dtype="fp32"),
        # data gradient of the output projection, 4 sequences of 16384, 12 heads of 128:
        # the gradient is put into 8 bits and multiplied with the transposed weight
        dict(name="dgrad_elu16k", op="dgrad", rows=65536, n=1536, k=1536, dtype="bf16"),
        # weight gradient of the second projection from the 8-bit checkpoint of its input
        dict(name="wgrad_l32k", op="wgrad", rows=65536, n=1024, k=4096),
        # the same for a ragged batch of a small model
        dict(name="wgrad_ragged", op="wgrad", rows=5003, n=264, k=520),
        # the activation between the projections, forward and backward from its checkpoint
        dict(name="gelu_train_l32k", op="gelu", rows=65536, cols=4096, dtype="bf16"),
        dict(name="gelu_train_ragged", op="gelu", rows=777, cols=1001, dtype="fp32"),
    ]


MOST_MACS = 65536 * 4096 * 1024
MOST_ELEMENTS = 65536 * 1024


def _log_size(rng, lo, hi, step=1):
    x = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, x // step * step if x >= step else x))


def draw(rng):
    op = rng.choice(["norm", "norm", "matmul", "matmul", "dgrad", "wgrad", "gelu"])
    even = rng.random() < 0.5  # whole blocks, or any size
    width = lambda hi: _log_size(rng, 16, hi, 128 if even else 8 if rng.random() < 0.5 else 1)
    while True:
        if op in ("norm", "gelu"):
            case = dict(op=op, rows=_log_size(rng, 1, 65536), cols=width(8192), dtype=rng.choice(["bf16", "bf16", "fp32"]))
            if op == "norm":
                case["train"] = rng.random() < 0.6
                case["checkpoint"] = bool(case["train"] and rng.random() < 0.6)
            if case["rows"] * case["cols"] <= MOST_ELEMENTS:
                return case
        else:
            case = dict(op=op, rows=_log_size(rng, 1, 65536), n=width(4096), k=width(4096))
            if op != "wgrad":
                case["dtype"] = "fp32" if op == "matmul" and rng.random() < 0.3 else "bf16"
            if case["rows"] * case["n"] * case["k"] <= MOST_MACS // 2:
                return case


def work(case):
    op, rows = case["op"], case["rows"]
    size = 4 if case.get("dtype") == "fp32" else 2
    q = lambda r, c: r * c + r * -(-c // BLOCK)  # codes and scales
    if op == "norm":
        cols = case["cols"]
        # x and the residual in, their sum and the 8-bit rows out
        moved, flops = 3 * size * rows * cols + q(rows, cols) + 4 * cols, 7.0 * rows * cols
        if case["train"]:
            # dy, the gradient of the sum and the kept rows in, the gradient of the sum and of gamma out
            moved += 3 * size * rows * cols + 4 * rows + 8 * cols
            moved += 2 * q(rows, cols) if case["checkpoint"] else size * rows * cols
            flops += 9.0 * rows * cols
        return {"bytes": moved, "flops": flops}
    if op == "gelu":
        cols = case["cols"]
        # z in, a and the checkpoint out; da and the checkpoint in, dz out
        return {"bytes": 3 * size * rows * cols + 3 * q(rows, cols), "flops": 60.0 * rows * cols}
    n, k = case["n"], case["k"]
    if op == "matmul":
        return {"bytes": q(rows, k) + q(n, k) + size * rows * n, "flops": 2.0 * rows * n * k}
    if op == "dgrad":
        return {"bytes": 2 * rows * n + q(k, n) + 2 * rows * k, "flops": 2.0 * rows * n * k}
    return {"bytes": 2 * rows * n + q(rows, k) + 4 * n * k, "flops": 2.0 * rows * n * k}


# ---- inputs ----------------------------------------------------------------

def _power(e):
    """2^e in fp32 for integers -126 <= e <= 127, by its bits (exp2 may round)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantized(x, block_rows=1):
    """codes [rows, 128 * blocks] e4m3 and scales [groups, 4 * ceil(blocks / 4)] uint8 of a finite x."""
    rows, cols = x.shape
    nb, groups = -(-cols // BLOCK), -(-rows // block_rows)
    pad = torch.zeros((groups * block_rows, nb * BLOCK), dtype=torch.float32, device=x.device)
    pad[:rows, :cols] = x
    t = pad.view(groups, block_rows, nb, BLOCK)
    top = t.abs().amax(dim=(1, 3)).contiguous()
    # the bits of a float are its exponent over its fraction: carry where the fraction is over 1.75
    e = (((top.view(torch.int32) + 0x1FFFFF) >> 23) - 135).clamp(-117, 120)
    codes = (t * _power(-e)[:, None, :, None]).to(torch.float8_e4m3fn)
    codes = codes.view(groups * block_rows, nb * BLOCK)[:rows].contiguous()
    scales = torch.full((groups, -(-nb // 4) * 4), 127, dtype=torch.uint8, device=x.device)
    scales[:, :nb] = (e + 127).to(torch.uint8)
    return codes, scales


def _values(codes, scales, cols, block_rows=1, dtype=torch.float32):
    """The values that codes and scales stand for (plain form)."""
    rows, width = codes.shape
    s = _power(scales[:, :width // BLOCK].to(torch.int32) - 127)
    if block_rows > 1:
        s = s.repeat_interleave(block_rows, 0)[:rows]
    return (codes.to(torch.float32).view(rows, -1, BLOCK) * s[:, :, None]).view(rows, width)[:, :cols].to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")
    op, rows = case["op"], case["rows"]
    dtype = DTYPES[case.get("dtype", "bf16")]
    state = {"case": case}

    def stream(cols):  # residual-stream rows: a few channels and a few tokens are much larger
        x = randn(rows, cols)
        x *= 1 + 15 * (torch.rand(cols, generator=g, device="cuda") > 0.99)
        x *= torch.exp(0.5 * randn(rows, 1))
        return x

    if op == "norm":
        cols = case["cols"]
        state.update(x=stream(cols).to(dtype), res=(0.5 * randn(rows, cols)).to(dtype), gamma=1 + 0.2 * randn(cols))
        if case["train"]:
            state.update(dy=(1e-3 * randn(rows, cols)).to(dtype), dres=(1e-3 * randn(rows, cols)).to(dtype))
    elif op == "gelu":
        cols = case["cols"]
        state.update(z=(1.5 * randn(rows, cols)).to(dtype), da=(1e-3 * randn(rows, cols)).to(dtype))
    elif op == "matmul":
        n, k = case["n"], case["k"]
        x = stream(k)
        x *= torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
        state["a"] = _quantized(x)
        state["w"] = _quantized(randn(n, k) * k ** -0.5, BLOCK)
    elif op == "dgrad":
        n, k = case["n"], case["k"]
        state["dy"] = (1e-3 * randn(rows, n) * torch.exp(0.5 * randn(rows, 1))).to(dtype)
        state["wt"] = _quantized(randn(k, n) * k ** -0.5, BLOCK)  # the transposed weight, kept beside it
    else:
        n, k = case["n"], case["k"]
        state["dy"] = (1e-3 * randn(rows, n)).to(torch.bfloat16)
        state["x"] = _quantized(torch.relu(randn(rows, k)) + 0.1 * randn(rows, k))
    return state


# ---- one pass --------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(state):
    from sub_linear_memory_gb300 import q8

    case = state["case"]
    op = case["op"]
    if op == "norm":
        h, y, rstd, h8 = q8.rms_norm(state["x"], state["gamma"], res=state["res"], eps=EPS, checkpoint=case["checkpoint"])
        out = {"h": h, "y": q8.dequantize(y)}
        if case["train"]:
            kept = h8 if case["checkpoint"] else h
            out["dh"], out["dgamma"] = q8.rms_norm_bwd(state["dy"], kept, rstd, state["gamma"], dres=state["dres"])
        return out
    if op == "gelu":
        a, z8 = q8.gelu(state["z"])
        return {"a": q8.dequantize(a), "dz": q8.gelu_bwd(state["da"], z8)}
    if op == "matmul":
        return q8.matmul(q8.Q8(*state["a"], case["k"]), q8.Q8(*state["w"], case["k"], BLOCK), dtype=DTYPES[case["dtype"]])
    if op == "dgrad":
        return q8.matmul(q8.quantize(state["dy"]), q8.Q8(*state["wt"], case["n"], BLOCK))
    return q8.wgrad(state["dy"], q8.Q8(*state["x"], case["k"]))


def _gelu_cdf(z):
    """The normal distribution function, by erfc so that the far left keeps its digits."""
    return 0.5 * torch.special.erfc(z * -math.sqrt(0.5))


def _run_plain(state):
    case = state["case"]
    op = case["op"]
    if op == "norm":
        dtype, cols = DTYPES[case["dtype"]], case["cols"]
        h = (state["x"].float() + state["res"].float()).to(dtype)
        hf = h.float()
        rstd = torch.rsqrt(hf.square().mean(1, keepdim=True) + EPS)
        y = _values(*_quantized(hf * rstd * state["gamma"]), cols, dtype=torch.bfloat16)
        out = {"h": h, "y": y}
        if case["train"]:
            kept = _values(*_quantized(hf), cols) if case["checkpoint"] else hf
            dy, xhat = state["dy"].float(), kept * rstd
            g = dy * state["gamma"]
            dh = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True)) + state["dres"].float()
            out["dh"], out["dgamma"] = dh.to(dtype), (dy * xhat).sum(0)
        return out
    if op == "gelu":
        dtype, cols = DTYPES[case["dtype"]], case["cols"]
        z = state["z"].float()
        a = _values(*_quantized(z * _gelu_cdf(z)), cols, dtype=torch.bfloat16)
        kept = _values(*_quantized(z), cols)
        slope = _gelu_cdf(kept) + kept * torch.exp(-0.5 * kept * kept) * (0.5 / math.pi) ** 0.5
        return {"a": a, "dz": (state["da"].float() * slope).to(dtype)}
    if op == "matmul":
        a = _values(*state["a"], case["k"])
        w = _values(*state["w"], case["k"], BLOCK)
        return (a @ w.t()).to(DTYPES[case["dtype"]])
    if op == "dgrad":
        dy = _values(*_quantized(state["dy"].float()), case["n"])
        wt = _values(*state["wt"], case["n"], BLOCK)
        return (dy @ wt.t()).to(torch.bfloat16)
    return state["dy"].float().t() @ _values(*state["x"], case["k"])


# ---- the same in 64 bits, from the definitions --------------------------------

def _times_power(x, e):
    """x * 2^e in fp64, the power by its bits."""
    return x * ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_held(x):
    """x (fp64, finite) as the 8-bit form holds it, one scale for each row and 128 columns."""
    out = torch.empty_like(x)
    for c in range(0, x.shape[1], BLOCK):
        b = x[:, c:c + BLOCK]
        m, p = torch.frexp(b.abs().amax(1, keepdim=True))  # m in [1/2, 1): at most 448 * 2^e = 0.875 * 2^(e + 9)
        e = (p - 9 + (m > 0.875)).clamp(-117, 120)
        e = torch.where(m == 0, torch.full_like(e, -117), e)
        v = _times_power(b, -e)
        step = (torch.frexp(v)[1] - 1).clamp(min=-6) - 3  # three fraction bits
        out[:, c:c + BLOCK] = _times_power(torch.round(_times_power(v, -step)), step + e)
    return out


def _exact_stored(codes, scales, cols, block_rows=1):
    """The values of stored codes, read bit by bit: sign, four exponent bits (bias 7), three fraction bits."""
    raw = codes.view(torch.uint8).to(torch.int32)
    exponent, fraction = (raw >> 3) & 15, (raw & 7).double()
    size = torch.where(exponent == 0, fraction / 512, _times_power(1 + fraction / 8, exponent - 7))
    value = torch.where(raw >= 128, -size, size)
    row = torch.arange(codes.shape[0], device=codes.device) // block_rows
    col = torch.arange(codes.shape[1], device=codes.device) // BLOCK
    return _times_power(value, scales.to(torch.int32)[row][:, col] - 127)[:, :cols]


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    normal = lambda z: torch.special.erfc(-z / math.sqrt(2.0)) / 2
    if op == "norm":
        h = (state["x"].double() + state["res"].double()).to(DTYPES[case["dtype"]]).double()
        gamma = state["gamma"].double()
        root = 1 / torch.sqrt((h * h).sum(1, keepdim=True) / case["cols"] + EPS)
        out = {"h": h, "y": _exact_held(h * root * gamma)}
        if case["train"]:
            n = (_exact_held(h) if case["checkpoint"] else h) * root
            dy = state["dy"].double()
            along = (dy * gamma * n).sum(1, keepdim=True) / case["cols"]
            out["dh"] = (dy * gamma - n * along) * root + state["dres"].double()
            out["dgamma"] = (dy * n).sum(0)
        return out
    if op == "gelu":
        z = state["z"].double()
        kept = _exact_held(z)
        slope = normal(kept) + kept * torch.exp(-kept * kept / 2) / math.sqrt(2 * math.pi)
        return {"a": _exact_held(z * normal(z)), "dz": state["da"].double() * slope}
    if op == "matmul":
        return _exact_stored(*state["a"], case["k"]) @ _exact_stored(*state["w"], case["k"], BLOCK).t()
    if op == "dgrad":
        return _exact_held(state["dy"].double()) @ _exact_stored(*state["wt"], case["n"], BLOCK).t()
    return state["dy"].double().t() @ _exact_stored(*state["x"], case["k"])
