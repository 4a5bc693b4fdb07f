"""GPU tests of the 8-bit layer operators at the ends of their ranges, against
fp64: values past what fp32 can square, long sums, many tiles."""
import numpy as np
import pytest
import torch

from oracle import q8 as ref
from sub_linear_memory_gb300 import inputs

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def q8():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from sub_linear_memory_gb300 import q8

    return q8


def sync():
    from sub_linear_memory_gb300 import binding

    binding.sync_status()


def np64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def draw(shape, slot, dtype=F32, scale=1.0):
    return inputs.gaussian(shape, 7500, slot, scale=scale, dtype=dtype).cuda()


# ---- norm: sums of squares past fp32's range ----------------------------------

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", [40, 264, 1000, 1024, 3001, 16384])
def test_rms_norm_past_fp32_range(q8, cols, dtype):
    """Rows of finite values whose squares overflow have rstd = 0 and y = 0, an
    infinity is NaN in its own block, a NaN in its whole row; a row whose
    1 / rms is finite but not its square is normed as any other."""
    x = draw((9, cols), 1, dtype)
    x[1] = 1e20
    x[2, cols // 2] = -2e19  # one square that overflows
    x[3] = 1.7e19 * cols ** -0.25  # the sum alone overflows
    x[4, cols - 1] = float("inf")
    x[5, 3] = float("nan")
    tiny = torch.where(draw((cols,), 2) < 0, -1e-20, 1e-20)
    x[6] = tiny.to(dtype)
    gamma = 1 + 0.1 * draw((cols,), 3)
    for checkpoint in (False, True):
        h, y, rstd, h8 = q8.rms_norm(x, gamma, eps=0.0, checkpoint=checkpoint)
        sync()
        v, r = np64(q8.dequantize(y)), np64(rstd)
        over = [1, 2] if cols < 16 else [1, 2, 3]
        assert np.all(r[over] == 0) and np.all(v[over] == 0)
        own = np.arange(cols) // 128 == (cols - 1) // 128
        assert r[4] == 0 and np.isnan(v[4][own]).all() and np.all(v[4][~own] == 0)
        assert np.isnan(r[5]) and np.isnan(v[5]).all()
        # squares of 1e-40 are held to 2^-150, 2^-17 of themselves, and so is their mean
        h64 = np64(x[6])
        assert abs(r[6] * np.sqrt((h64 * h64).mean()) - 1) <= 2.0 ** -16
        want = h64 / np.sqrt((h64 * h64).mean()) * np64(gamma)
        step = 2.0 ** (np64(y.scales[6:7].double())[0, np.arange(cols) // 128] - 127 - 10)
        assert np.all(np.abs(v[6] - want) <= np.maximum(np.abs(want) * 2.0 ** -4, step) * (1 + 2.0 ** -14))
        # the rows beside them are untouched
        rest = [0, 7, 8]
        assert torch.equal(rstd[rest], q8.rms_norm(x[rest], gamma, eps=0.0)[2])
        if checkpoint:
            dh, dgamma = q8.rms_norm_bwd(draw((9, cols), 4, dtype), h8, torch.where(rstd.isnan(), 0, rstd), gamma)
            sync()
            assert torch.isfinite(dh[[0, 1, 2, 3, 7, 8]]).all()
    # the same without eps in the row's way
    r = q8.rms_norm(x, gamma, eps=1e-5)[2]
    sync()
    assert np.all(np64(r)[over] == 0) and abs(float(r[6]) - 1e-5 ** -0.5) < 1e-3
    assert float(q8.rms_norm(x, gamma, eps=float("inf"))[2][0]) == 0


# ---- products: long sums ------------------------------------------------------

def values_on_gpu(q8, q):
    return q8.dequantize(q, F32).double()


# (rows, n, k): the kernel for few rows with k in one CTA and over a cluster, and
# the whole-tile kernel with several tiles a pair, rows of out on and off 16 bytes
@pytest.mark.parametrize("rows, n, k", [(3, 10240, 4096), (3, 10240, 23000), (5, 264, 131072), (128, 1001, 131072),
                                        (50, 10001, 8200), (130, 264, 4096), (130, 264, 131072), (300, 1033, 16777),
                                        (20000, 512, 8200), (2433, 1033, 9000)])
def test_matmul_long_sums_are_not_truncated(q8, rows, n, k):
    """Operands of one sign, so that what each addition cuts off adds up: at most
    128 additions in one accumulator, which lose half a unit 2^-23 of a partial
    sum that is half of the whole on average; then one rounding to nearest for
    each 4096 columns, and 16 units for those within an instruction."""
    g = torch.Generator(device="cuda").manual_seed(7600 + rows)
    a = q8.quantize(torch.randn((rows, k), generator=g, device="cuda").abs())
    w = q8.pack_weight(torch.randn((n, k), generator=g, device="cuda").abs(), transpose=False)[0]
    buf = torch.full((rows * n + 512,), 7.0, device="cuda")
    out = buf[256:256 + rows * n].view(rows, n)
    q8.matmul(a, w, out=out)
    sync()
    assert torch.all(buf[:256] == 7) and torch.all(buf[256 + rows * n:] == 7)
    want = values_on_gpu(q8, a) @ values_on_gpu(q8, w).t()
    units = min(k / 32, 128) / 4 + k / 8192 + 16
    err = float(((out.double() - want).abs() / want).max()) * 2 ** 23
    assert err <= units, (err, units)
    assert torch.equal(q8.matmul(a, w, dtype=F32), out)


# ---- GeLU: the normal distribution function near 0 --------------------------------

def test_gelu_slope_near_zero(q8):
    """Phi(z) + z phi(z) in fp32 at every code with |z| <= 1 under 16 scales.
    Phi is 1/2 + z P: within 3e-8 of Phi(-|z|) by its fit, half a unit 2^-25 of
    P <= 0.4 and of the last step before it, and half a unit of the sum: 1.25 *
    2^-24.  phi: two units 2^-23 of the hardware's exponential and one each of
    the square, the exponent and the product."""
    codes = torch.arange(256, dtype=torch.uint8)
    codes = codes[(codes & 127) != 127]  # without the NaNs
    raw = torch.zeros((16, 256), dtype=torch.uint8)
    raw[:, :254] = codes
    scales = torch.full((16, 4), 127, dtype=torch.uint8)
    scales[:, :2] = 127 - 1 - torch.arange(16, dtype=torch.uint8)[:, None]
    z8 = q8.Q8(raw.view(torch.float8_e4m3fn).cuda(), scales.cuda(), 254)
    dz = q8.gelu_bwd(torch.ones((16, 254), device="cuda"), z8)
    sync()
    z = np64(q8.dequantize(z8, F32))
    near = np.abs(z) <= 1
    assert near.sum() > 2000
    want = ref.gelu_slope(z)
    bound = 1.25 * 2.0 ** -24 + np.abs(z) * np.exp(-0.5 * z * z) * 0.4 * 5 * 2.0 ** -23 + 2.0 ** -24 * np.abs(want)
    assert np.all((np.abs(np64(dz) - want) <= bound)[near]), float((np.abs(np64(dz) - want) / bound)[near].max())
