"""GPU tests of the 8-bit products on every way through their kernels: few rows
with k in one CTA or over a cluster, many output tiles, whole and cut tiles of
the weight gradient, every code and scale.  References in fp64; those of large
matrices are formed on the GPU (library products)."""
import pytest
import torch

from sub_linear_memory_gb300 import inputs

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
STORE = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def q8():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from sub_linear_memory_gb300 import q8

    return q8


def sync():
    from sub_linear_memory_gb300 import binding

    binding.sync_status()


def draw(shape, slot, dtype=F32, scale=1.0):
    return inputs.gaussian(shape, 7700, slot, device="cuda", scale=scale, dtype=dtype)


def check_matmul(q8, a, w, dtype):
    """Each of the additions of 32 columns in sequence cuts off at most a unit
    2^-23 of the terms' magnitudes (128 of them in one sum of an fp32 result),
    16 units within one instruction, half a unit for each 4096 columns."""
    out = q8.matmul(a, w, dtype=dtype)
    sync()
    av, wv = q8.dequantize(a, F32).double(), q8.dequantize(w, F32).double()
    want, size = av @ wv.t(), av.abs() @ wv.abs().t()
    units = min(a.cols / 32, 128 if dtype == F32 else 1e9) + a.cols / 8192 + 16
    bound = STORE[dtype] * want.abs() + units * 2.0 ** -23 * size
    err = (out.double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    assert torch.equal(q8.matmul(a, w, dtype=dtype), out)
    return out


def pair(q8, rows, n, k, seed):
    a = draw((rows, k), seed) * torch.exp(draw((rows, 1), seed + 1))
    return q8.quantize(a), q8.pack_weight(draw((n, k), seed + 2, scale=k ** -0.5), transpose=False)[0]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows, n, k", [(33, 264, 1300), (64, 1001, 4096), (100, 1001, 1336), (128, 1024, 4096),
                                        (128, 10001, 4096), (5, 40, 131072), (3, 10240, 23000), (127, 8, 2000),
                                        (65, 520, 1025), (64, 4096, 1024)])
def test_matmul_of_few_rows(q8, rows, n, k, dtype):
    check_matmul(q8, *pair(q8, rows, n, k, 10), dtype)


@pytest.mark.parametrize("rows, n, k", [(5, 260, 1300), (47, 260, 1300), (64, 260, 700), (128, 260, 1300),
                                        (3, 10260, 1300)])
def test_matmul_of_few_rows_scales_of_every_block(q8, rows, n, k):
    """Blocks whose scales differ by many powers of two, in both operands, and
    one block alone deciding each result (an exact product)."""
    a, w = torch.zeros((rows, k)), torch.zeros((n, k))
    r, c = torch.arange(rows), torch.arange(n)
    blocks = -(-k // 128)
    at = [min(b * 128 + 5 * b, k - 1) for b in range(blocks)]
    for b, kk in enumerate(at):
        a[:, kk] = torch.exp2(((r * 7 + b * 3) % 23 - 11).float())
        w[:, kk] = torch.exp2(((c // 128 * 5 + b * 4) % 17 - 8).float())
    qw = q8.pack_weight(w.cuda(), transpose=False)[0]
    check_matmul(q8, q8.quantize(a.cuda()), qw, F32)
    wv = q8.dequantize(qw, F32)
    for kk in at:
        only = torch.zeros_like(a)
        only[:, kk] = a[:, kk]
        out = q8.matmul(q8.quantize(only.cuda()), qw, dtype=F32)
        sync()
        assert torch.equal(out, only[:, kk:kk + 1].cuda() * wv[:, kk][None])


def all_codes(q8, rows, first, step):
    """rows x 254 columns: every code but the NaNs, under the scales 2^first, 2^(first + step), ..."""
    codes = torch.arange(256, dtype=torch.uint8)
    raw = torch.zeros((rows, 256), dtype=torch.uint8)
    raw[:, :254] = codes[(codes & 127) != 127]
    scales = torch.full((rows, 4), 127, dtype=torch.uint8)
    e = (first + step * torch.arange(rows)) % 236 - 117  # -117 ... 118
    scales[:, 0], scales[:, 1] = (e + 127).to(torch.uint8), (e.flip(0) + 127).to(torch.uint8)
    return q8.Q8(raw.view(torch.float8_e4m3fn).cuda(), scales.cuda(), 254)


@pytest.mark.parametrize("rows", [60, 300])
def test_matmul_of_every_code_and_scale(q8, rows):
    """With the identity for a weight the values come through unchanged."""
    a = all_codes(q8, rows, 0, 7)
    one = q8.pack_weight(torch.eye(254, device="cuda"), transpose=False)[0]
    out = q8.matmul(a, one, dtype=F32)
    sync()
    assert torch.equal(out, q8.dequantize(a, F32))


def test_wgrad_of_every_code_and_scale(q8):
    """Subnormal codes too: one row of dy is 1 for each row of x, so dw is x."""
    x = all_codes(q8, 236, 0, 1)
    dw = q8.wgrad(torch.eye(236, dtype=BF16, device="cuda"), x)
    sync()
    assert torch.equal(dw, q8.dequantize(x, F32))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows, n, k", [(300, 264, 700), (2600, 1040, 300), (300, 1033, 9000)])
def test_nonfinite_blocks_through_whole_tiles(q8, rows, n, k, dtype):
    """A block with a NaN or an infinity makes its own row of the result NaN (of
    a weight: the 128 columns of its block), and nothing else."""
    a, w = draw((rows, k), 30), draw((n, k), 31)
    a[7, k - 1], a[rows - 1, 3] = float("nan"), float("-inf")
    w[200, 130] = float("inf")
    out = q8.matmul(q8.quantize(a), q8.pack_weight(w, transpose=False)[0], dtype=dtype)
    sync()
    want = torch.zeros((rows, n), dtype=torch.bool, device="cuda")
    want[[7, rows - 1]] = True
    want[:, 128:256] = True
    assert torch.equal(out.isnan(), want) and bool(out[~want].isfinite().all())


# (rows, n, k) in tiles of 256 x 256 for 76 pairs: several whole tiles a pair and cut
# ones of one step; a wave and few cut tiles; rows of dy off 16 bytes; a wave and
# cut tiles whose ends the left-over pairs share; long whole tiles; cut tiles alone
@pytest.mark.parametrize("rows, n, k", [(70, 4096, 4096), (1500, 2304, 2304), (1301, 2311, 2600), (3200, 2304, 3584),
                                        (5000, 4608, 1536), (40000, 2304, 2304), (9000, 1800, 1300), (6000, 768, 2816)])
def test_wgrad_of_many_tiles(q8, rows, n, k):
    """Terms of one sign.  An accumulator takes 80 additions, which cut off half
    a unit 2^-23 of a partial sum that is half of the whole on average (20
    units, 16 within an instruction); the sums of those are rounded to nearest,
    half a unit for each accumulator (1280 rows) and each part of a tile (32 at
    most)."""
    dy = draw((rows, n), 40, BF16).abs()
    x = q8.quantize(draw((rows, k), 41).abs() * torch.exp(draw((rows, 1), 42)))
    dw = q8.wgrad(dy, x)
    sync()
    want = dy.double().t() @ q8.dequantize(x, F32).double()
    units = 20 + 16 + rows / 2560 + 16
    err = float(((dw.double() - want).abs() / want).max()) * 2 ** 23
    assert err <= units, (err, units)
    assert torch.equal(q8.wgrad(dy, x), dw)
    acc = torch.full_like(dw, 0.25)
    q8.wgrad(dy, x, dw=acc, accumulate=True)
    sync()
    assert bool(((acc.double() - 0.25 - want).abs() <= (units + 1) * 2.0 ** -23 * (want + 0.25)).all())
