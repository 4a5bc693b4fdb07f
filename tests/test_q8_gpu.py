"""GPU parity of the 8-bit layer operators with the fp64 oracle (oracle/q8.py).

Tolerances, element by element, are sums of what each step may round:
  * storing as bf16: 2^-8 of the value; as e4m3: 2^-4 of the value, or half the
    subnormal step 2^(e - 10) of the block's scale 2^e; codes and scales of a
    matrix that is quantized as it is are exact;
  * fp32 arithmetic: a few units (2^-24 of the terms) for each operation;
  * sums on the tensor cores: one unit 2^-23 of the sum of magnitudes for each
    of the additions in sequence (one for each 32 columns of e4m3, or 16 rows
    of bf16), and 16 for those within one instruction.
"""
import numpy as np
import pytest
import torch

from oracle import q8 as ref
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


def np64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def draw(shape, slot, dtype=F32, scale=1.0):
    return inputs.gaussian(shape, 7100, slot, scale=scale, dtype=dtype).cuda()


def stored(q):
    """(code values, scale bytes) of a Q8, as the oracle holds them."""
    return np64(q.codes.to(torch.float32)), q.scales.cpu().numpy()


def same_q8(q, codes, scales):
    got_c, got_s = stored(q)
    assert np.array_equal(got_s, scales)
    assert np.array_equal(got_c, codes, equal_nan=True)


def check_held(q, y, arith=4e-7):
    """A Q8 of computed values y (fp64): the smallest scales, codes within half a step."""
    codes, scales = stored(q)
    nb = -(-q.cols // 128)
    assert np.all(scales[:, nb:] == 127) and np.all(codes[:, q.cols:] == 0)
    pad = np.zeros((y.shape[0], nb * 128))
    pad[:, :q.cols] = y
    top = np.abs(pad).reshape(y.shape[0], nb, 128).max(2)
    e = scales[:, :nb].astype(int) - 127
    assert np.all(top <= 448 * 2.0 ** e * (1 + arith))
    assert np.all((top > 448 * 2.0 ** (e - 1) * (1 - arith)) | (e == -117))
    step = 2.0 ** (np.repeat(e, 128, 1)[:, :q.cols] - 10.0)
    v = ref.values(codes, scales, q.cols)
    assert np.all(np.abs(v - y) <= np.maximum(np.abs(y) * (2.0 ** -4), step) * (1 + 1e-5) + arith * np.abs(y))


SHAPES = [(1, 1), (1, 128), (3, 129), (5, 1000), (130, 256), (7, 77), (64, 8)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows, cols", SHAPES)
def test_quantize_and_dequantize_are_exact(q8, rows, cols, dtype):
    x = (draw((rows, cols), 1) * torch.exp(6 * draw((rows, 1), 2))).to(dtype)
    x[rows // 2, : cols // 2] = 0
    q = q8.quantize(x)
    sync()
    codes, scales = ref.quantize(np64(x))
    same_q8(q, codes, scales)
    v = ref.values(codes, scales, cols)
    assert np.array_equal(np64(q8.dequantize(q)), v)
    assert np.array_equal(np64(q8.dequantize(q, F32)), v)


def test_quantize_extremes(q8):
    """Zeros, the type's largest and smallest values, scale borders, infinities and NaNs."""
    x = torch.zeros((9, 300))
    x[1] = 3.3e38
    x[2] = 1e-38
    x[3] = 448.0
    x[4] = torch.nextafter(torch.tensor(448.0), torch.tensor(500.0))
    x[5, 7] = float("inf")
    x[6, 200] = float("-inf")
    x[7, 299] = float("nan")
    x[8, ::2] = -(2.0 ** -149)
    for dtype in (F32, BF16):
        y = x.to(dtype).cuda()
        q = q8.quantize(y)
        sync()
        codes, scales = ref.quantize(np64(y))
        same_q8(q, codes, scales)
        assert np.array_equal(np64(q8.dequantize(q, F32)), ref.values(codes, scales, 300), equal_nan=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n, k", [(1, 1), (128, 128), (129, 127), (300, 264), (8, 1000), (257, 16)])
def test_pack_weight(q8, n, k, dtype):
    w = (draw((n, k), 3) * torch.exp(draw((n, 1), 4))).to(dtype)
    q, qt = q8.pack_weight(w)
    sync()
    codes, scales = ref.quantize(np64(w), 128)
    same_q8(q, codes, scales)
    v = ref.values(codes, scales, k, 128)
    assert np.array_equal(np64(q8.dequantize(q)), v)
    assert np.array_equal(np64(q8.dequantize(qt)), v.T)
    tc, ts = ref.quantize(np64(w).T, 128)
    same_q8(qt, tc, ts)
    only, none = q8.pack_weight(w, transpose=False)
    assert none is None and torch.equal(only.codes.view(torch.uint8), q.codes.view(torch.uint8))


NORM_SHAPES = [(1, 1), (3, 8), (9, 129), (65, 264), (33, 520), (17, 1000), (5, 1024), (6, 1528), (4, 2048), (3, 3080),
               (3, 4096), (2, 6000), (2, 8192), (2, 12001), (2, 16384), (2500, 24)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows, cols", NORM_SHAPES)
def test_rms_norm(q8, rows, cols, dtype):
    x, res = draw((rows, cols), 5, dtype, 3.0), draw((rows, cols), 6, dtype)
    gamma, eps = 1 + 0.2 * draw((cols,), 7), 1e-5
    for r in (res, None):
        h, y, rstd, h8 = q8.rms_norm(x, gamma, res=r, eps=eps, checkpoint=True)
        sync()
        hh = x if r is None else (x.float() + r.float()).to(dtype)
        assert torch.equal(h, hh) and (r is not None or h is x)
        y64, rstd64 = ref.rms_norm(np64(hh), np64(gamma), eps)
        # the sum of squares: at most cols / 32 + 10 additions in sequence, all of one sign
        tol = (cols / 64 + 16) * 2.0 ** -24
        assert np.all(np.abs(np64(rstd) - rstd64) <= tol * rstd64)
        check_held(y, y64, arith=tol + 2e-7)
        same_q8(h8, *ref.quantize(np64(hh)))
        assert q8.rms_norm(x, gamma, res=r, eps=eps)[3] is None


def test_rms_norm_in_place_and_zero_rows(q8):
    from sub_linear_memory_gb300 import binding

    x, res, gamma = draw((12, 520), 5, BF16), draw((12, 520), 6, BF16), 1 + draw((520,), 7, scale=0.1)
    h, y, rstd, _ = q8.rms_norm(x, gamma, res=res)
    y2 = q8.empty(12, 520)
    buf = x.clone()
    st = torch.cuda.current_stream().cuda_stream
    assert binding.raw().slim_q8_rms_norm(buf.data_ptr(), res.data_ptr(), gamma.data_ptr(), 1e-5, buf.data_ptr(), None,
                                          y2.codes.data_ptr(), y2.scales.data_ptr(), None, None, 12, 520, st) == 0
    sync()
    assert torch.equal(buf, h)
    assert torch.equal(y2.codes.view(torch.uint8), y.codes.view(torch.uint8)) and torch.equal(y2.scales, y.scales)
    z = torch.zeros((3, 200), dtype=BF16, device="cuda")
    _, y, rstd, _ = q8.rms_norm(z, torch.ones(200, device="cuda"))
    sync()
    assert torch.all(q8.dequantize(y) == 0) and torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=1e-6)
    # an infinity or a NaN reaches its own row only
    x = draw((4, 300), 8)
    x[1, 5], x[2, 250] = float("inf"), float("nan")
    v = np64(q8.dequantize(q8.rms_norm(x, torch.ones(300, device="cuda"))[1]))
    sync()
    assert np.isnan(v[1, :128]).all() and np.isnan(v[2]).all() and np.isfinite(v[[0, 3]]).all()
    empty = torch.empty((0, 64), device="cuda")
    assert q8.rms_norm(empty, torch.ones(64, device="cuda"))[1].rows == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kept", ["full", "8bit"])
@pytest.mark.parametrize("rows, cols", NORM_SHAPES)
def test_rms_norm_bwd(q8, rows, cols, kept, dtype):
    h, gamma = draw((rows, cols), 9, dtype, 2.0), 1 + 0.2 * draw((cols,), 10)
    dy, dres = draw((rows, cols), 11, dtype, 1e-3), draw((rows, cols), 12, dtype, 1e-3)
    _, rstd64 = ref.rms_norm(np64(h), np64(gamma), 1e-5)
    rstd = torch.tensor(rstd64, dtype=F32, device="cuda")
    keep = q8.quantize(h) if kept == "8bit" else h
    k64 = ref.held(np64(h)) if kept == "8bit" else np64(h)
    for r in (dres, None):
        dh, dgamma = q8.rms_norm_bwd(dy, keep, rstd, gamma, dres=r)
        sync()
        r64 = None if r is None else np64(r)
        dh64, dg64 = ref.rms_norm_bwd(np64(dy), k64, np64(rstd), np64(gamma), r64)
        n, g = np.abs(k64) * np64(rstd)[:, None], np.abs(np64(dy) * np64(gamma))
        # magnitudes of the terms; the mean is a sum as in the forward
        terms = np64(rstd)[:, None] * (g + n * (g * n).mean(1, keepdims=True) * (1 + cols / 64 + 16))
        if r is not None:
            terms = terms + np.abs(r64)
        assert np.all(np.abs(np64(dh) - dh64) <= STORE[dtype] * np.abs(dh64) + 8 * 2.0 ** -24 * terms)
        # dgamma: rows are summed at most `rows` in sequence
        bound = (np.abs(np64(dy)) * n).sum(0) * 2.0 ** -24 * (min(rows, 64) + 64)
        assert np.all(np.abs(np64(dgamma) - dg64) <= bound)
    # the order of the sums is fixed
    again = q8.rms_norm_bwd(dy, keep, rstd, gamma, dres=None)
    assert torch.equal(again[0], dh) and torch.equal(again[1], dgamma)


def test_rms_norm_bwd_many_rows_and_none(q8):
    rows, cols = 40001, 136
    h, dy, gamma = draw((rows, cols), 13, BF16), draw((rows, cols), 14, BF16, 1e-3), 1 + 0.1 * draw((cols,), 15)
    _, rstd64 = ref.rms_norm(np64(h), np64(gamma), 1e-5)
    rstd = torch.tensor(rstd64, dtype=F32, device="cuda")
    dh, dgamma = q8.rms_norm_bwd(dy, h, rstd, gamma)
    sync()
    dh64, dg64 = ref.rms_norm_bwd(np64(dy), np64(h), np64(rstd), np64(gamma))
    assert np.linalg.norm(np64(dgamma) - dg64) <= 2e-6 * np.linalg.norm(dg64)
    assert np.linalg.norm(np64(dh) - dh64) <= 2.0 ** -8 * np.linalg.norm(dh64)
    none = torch.empty((0, cols), dtype=BF16, device="cuda")
    dh, dgamma = q8.rms_norm_bwd(none, none, torch.empty(0, device="cuda"), gamma)
    sync()
    assert dh.shape == (0, cols) and torch.all(dgamma == 0)


# |GeLU|: the distribution function to 2e-7 of its value (fp32 exp of a squared
# argument of up to 100 loses more far in the left tail: 2^-24 of the exponent)
def gelu_tol(z):
    return 4e-7 + 2.0 ** -24 * z * z


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows, cols", SHAPES)
def test_gelu(q8, rows, cols, dtype):
    z = draw((rows, cols), 16, dtype, 2.0)
    z[0, : min(cols, 9)] = torch.tensor([0.0, 5.0, -5.0, 9.0, -9.0, 1e-3, -1e-30, 30.0, -0.5])[: min(cols, 9)].to(dtype)
    a, z8 = q8.gelu(z)
    sync()
    z64 = np64(z)
    same_q8(z8, *ref.quantize(z64))
    check_held(a, ref.gelu(z64), arith=float(gelu_tol(np.minimum(np.abs(z64), 14.0)).max()))
    da = draw((rows, cols), 17, dtype, 1e-3)
    dz, dz8 = q8.gelu_bwd(da, z8, quantized=True)
    sync()
    kept = ref.held(z64)
    dz64 = np64(da) * ref.gelu_slope(kept)
    # Phi(z) and z phi(z) cancel near z = -0.75: errors are of the larger term
    size = np.abs(np64(da)) * (ref.cdf(kept) + np.abs(kept) * np.exp(-0.5 * kept * kept) * 0.4) * gelu_tol(kept)
    assert np.all(np.abs(np64(dz) - dz64) <= STORE[dtype] * np.abs(dz64) * 1.001 + size)
    same_q8(dz8, *ref.quantize(np64(dz)))
    assert torch.equal(q8.gelu_bwd(da, z8), dz)
    assert q8.gelu(z, checkpoint=False)[1] is None


def test_gelu_far_tails_and_nonfinite(q8):
    z = torch.zeros((4, 256), device="cuda")
    z[0, :128] = torch.linspace(-13, -3, 128)  # a block of the left tail alone keeps its digits
    z[1, 0], z[2, 130] = float("inf"), float("nan")
    z[3] = 1e30
    a, z8 = q8.gelu(z)
    sync()
    tail = np.linspace(-13, -3, 128).astype(np.float32).astype(np.float64)[None]
    part = q8.Q8(a.codes[:1, :128].contiguous(), torch.cat([a.scales[:1, :1], a.scales[:1, 2:3].repeat(1, 3)], 1), 128)
    check_held(part, ref.gelu(tail), arith=float(gelu_tol(tail).max()) * 2)
    v = np64(q8.dequantize(a))
    assert np.isnan(v[1, :128]).all() and np.isnan(v[2, 128:]).all() and np.isfinite(v[3]).all()
    dz = np64(q8.gelu_bwd(torch.ones_like(z), z8))
    assert np.isnan(dz[1, :128]).all() and np.isnan(dz[2, 128:]).all() and np.isfinite(dz[3]).all()
    assert np.isfinite(dz[1, 128:]).all()


def pair(q8, rows, n, k, seed):
    a = draw((rows, k), 20 + seed, F32) * torch.exp(draw((rows, 1), 30 + seed))
    w = draw((n, k), 40 + seed, F32, k ** -0.5)
    return q8.quantize(a), q8.pack_weight(w, transpose=False)[0]


def check_matmul(q8, a, w, dtype):
    out = q8.matmul(a, w, dtype=dtype)
    sync()
    av = ref.values(*stored(a), a.cols)
    wv = ref.values(*stored(w), w.cols, 128)
    want = av @ wv.T
    size = np.abs(av) @ np.abs(wv).T
    steps = -(-a.cols // 32) + 16
    err = np.abs(np64(out) - want)
    assert np.all(err <= STORE[dtype] * np.abs(want) + steps * 2.0 ** -23 * size), float(
        (err / np.maximum(size, 1e-300)).max())
    return out


MM_SHAPES = [(1, 1, 1), (1, 128, 128), (1, 1024, 4096), (3, 264, 136), (16, 8, 520), (17, 130, 1000), (100, 1001, 640),
             (128, 256, 384), (129, 512, 1024), (200, 72, 2056), (515, 392, 640), (300, 1536, 512), (1, 40, 8192)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows, n, k", MM_SHAPES)
def test_matmul(q8, rows, n, k, dtype):
    a, w = pair(q8, rows, n, k, 0)
    out = check_matmul(q8, a, w, dtype)
    assert torch.equal(q8.matmul(a, w, dtype=dtype), out)


# output tiles enough for the persistent kernel: ragged in each direction, rows of
# out on and off 16 bytes, one block of k to many
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows, n, k", [(2560, 1024, 1024), (9728, 256, 128), (2433, 1033, 700), (1300, 2056, 392),
                                        (5000, 520, 1928), (257, 9999, 264), (12000, 1001, 136), (3000, 1536, 4000),
                                        (20001, 1033, 520), (40000, 640, 1160), (300, 8, 256), (300, 24, 1500),
                                        (129, 1, 40), (66, 100, 1024), (128, 4099, 1000)])
def test_matmul_many_tiles(q8, rows, n, k, dtype):
    a, w = pair(q8, rows, n, k, 2)
    out = check_matmul(q8, a, w, dtype)
    assert torch.equal(q8.matmul(a, w, dtype=dtype), out)


@pytest.mark.parametrize("rows, n, k", [(130, 260, 1300), (2433, 1033, 1300)])
def test_matmul_scales_of_every_block(q8, rows, n, k):
    """Blocks whose scales differ by many powers of two, in both operands, and
    one block alone deciding each result (an exact product)."""
    a = torch.zeros((rows, k))
    w = torch.zeros((n, k))
    r, c = torch.arange(rows), torch.arange(n)
    for b in range(11):
        kk = min(b * 128 + 5 * b, k - 1)
        a[:, kk] = torch.exp2(((r * 7 + b * 3) % 23 - 11).float())
        w[:, kk] = torch.exp2(((c // 128 * 5 + b * 4) % 17 - 8).float())
    qa, qw = q8.quantize(a.cuda()), q8.pack_weight(w.cuda(), transpose=False)[0]
    check_matmul(q8, qa, qw, F32)
    for b in (0, 3, 4, 7, 10):
        only = torch.zeros_like(a)
        kk = min(b * 128 + 5 * b, k - 1)
        only[:, kk] = a[:, kk]
        out = q8.matmul(q8.quantize(only.cuda()), qw, dtype=F32)
        sync()
        wv = q8.dequantize(qw, F32).cpu()
        assert torch.equal(out.cpu(), only[:, kk:kk + 1] * wv[:, kk][None])


def test_matmul_nan_and_empty(q8):
    a, w = draw((40, 300), 50), draw((70, 300), 51)
    a[7, 299] = float("nan")
    out = np64(q8.matmul(q8.quantize(a), q8.pack_weight(w)[0]))
    sync()
    assert np.isnan(out[7]).all() and np.isfinite(np.delete(out, 7, 0)).all()
    z = q8.matmul(q8.quantize(draw((5, 0), 1)), q8.pack_weight(draw((6, 0), 1))[0], dtype=F32)
    sync()
    assert z.shape == (5, 6) and torch.all(z == 0)
    assert q8.matmul(q8.quantize(draw((0, 64), 1)), q8.pack_weight(draw((6, 64), 1))[0]).shape == (0, 6)


@pytest.mark.parametrize("rows, n, k", [(131, 203, 260), (2433, 1035, 260), (2433, 1040, 260)])
def test_matmul_writes_inside_its_output_only(q8, rows, n, k):
    a, w = pair(q8, rows, n, k, 1)
    for dtype in (BF16, F32):
        buf = torch.full((rows * n + 512,), 7.0, dtype=dtype, device="cuda")
        out = buf[256:256 + rows * n].view(rows, n)
        q8.matmul(a, w, out=out)
        sync()
        assert torch.all(buf[:256] == 7) and torch.all(buf[256 + rows * n:] == 7)
        assert torch.equal(out, q8.matmul(a, w, dtype=dtype))


WG_SHAPES = [(1, 1, 1), (64, 128, 256), (63, 8, 128), (130, 264, 520), (1000, 200, 129), (700, 131, 300), (4096, 16, 64),
             (5000, 384, 640)]


@pytest.mark.parametrize("rows, n, k", WG_SHAPES)
def test_wgrad(q8, rows, n, k):
    dy = draw((rows, n), 60, BF16, 1e-3)
    x = q8.quantize(draw((rows, k), 61) * torch.exp(2 * draw((rows, 1), 62)))
    dw = q8.wgrad(dy, x)
    sync()
    xv = ref.values(*stored(x), k)
    want, size = np64(dy).T @ xv, np.abs(np64(dy)).T @ np.abs(xv)
    tol = (-(-rows // 16) + 16) * 2.0 ** -23
    err = np.abs(np64(dw) - want)
    assert np.all(err <= tol * size), float((err / np.maximum(size, 1e-300)).max())
    assert torch.equal(q8.wgrad(dy, x), dw)
    acc = torch.full_like(dw, 0.25)
    q8.wgrad(dy, x, dw=acc, accumulate=True)
    sync()
    assert np.all(np.abs(np64(acc) - 0.25 - want) <= tol * size + 2.0 ** -23)


def test_wgrad_scale_range_nan_and_empty(q8):
    """Every exponent of the scales (past bf16's range in one factor), NaN blocks, no rows."""
    es = list(range(-117, 90, 9)) + [7, 8, 9]
    rows = len(es)
    x = torch.zeros((rows, 130))
    for i, e in enumerate(es):
        x[i, :128] = 400.0 * 2.0 ** e
        x[i, 1:100] *= torch.linspace(-1, 1, 99)
        x[i, 128:] = 2.0 ** min(e, 20)
    q = q8.quantize(x.cuda())
    dy = torch.zeros((rows, rows), dtype=BF16)
    dy[torch.arange(rows), torch.arange(rows)] = 1.0
    dw = q8.wgrad(dy.cuda(), q)
    sync()
    # one term to each result: exact, but for what is below fp32's normal range
    want = ref.values(*stored(q), 130)
    assert np.all(np.abs(np64(dw) - want) <= 2.0 ** -126)
    x[3, 5] = float("inf")
    dw = np64(q8.wgrad(torch.ones((rows, 9), dtype=BF16, device="cuda"), q8.quantize(x.cuda())))
    sync()
    assert np.isnan(dw[:, :128]).all() and np.isfinite(dw[:, 128:]).all()
    none = q8.quantize(torch.empty((0, 40), device="cuda"))
    dw = q8.wgrad(torch.empty((0, 24), dtype=BF16, device="cuda"), none)
    sync()
    assert dw.shape == (24, 40) and torch.all(dw == 0)
    keep = torch.ones((24, 40), device="cuda")
    q8.wgrad(torch.empty((0, 24), dtype=BF16, device="cuda"), none, dw=keep, accumulate=True)
    assert torch.all(keep == 1)


def test_other_stream_and_graph(q8):
    """On another stream than the inputs' own, and captured into a graph and replayed on new inputs."""
    x, gamma = draw((300, 512), 70, BF16), 1 + 0.1 * draw((512,), 71)
    w, wt = q8.pack_weight(draw((256, 512), 72, BF16, 0.05))
    dy = draw((300, 256), 73, BF16)

    def step():
        h, y, rstd, h8 = q8.rms_norm(x, gamma, checkpoint=True)
        out = q8.matmul(y, w)
        dh, dgamma = q8.rms_norm_bwd(q8.matmul(q8.quantize(dy), wt), h8, rstd, gamma)
        return out, dh, dgamma, q8.wgrad(dy, y)

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    x.copy_(draw((300, 512), 74, BF16))
    graph.replay()
    torch.cuda.synchronize()
    want = step()
    sync()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_offsets_past_32_bits(q8):
    """Matrices of more than 2^31 elements: the last rows, and an odd width's."""
    rows, cols = 70001, 32768
    x = torch.empty((rows, cols), dtype=BF16, device="cuda").uniform_(-3, 3)
    q = q8.quantize(x)
    last = np64(x[-2:])
    codes, scales = ref.quantize(last)
    assert np.array_equal(np64(q.codes[-2:].float()), codes)
    assert np.array_equal(q.scales[-2:].cpu().numpy(), scales)
    x = q8.dequantize(q)
    sync()
    assert np.array_equal(np64(x[-2:]), ref.values(codes, scales, cols))
    dz = q8.gelu_bwd(x, q)
    sync()
    held = ref.values(codes, scales, cols)
    assert np.all(np.abs(np64(dz[-2:]) - held * ref.gelu_slope(held)) <= 2.0 ** -8 * np.abs(held * 1.2) + 1e-5)
    del x, q, dz
    rows, n, k = 262200, 8200, 128
    a = q8.quantize(torch.randn((rows, k), device="cuda"))
    w = q8.pack_weight(torch.randn((n, k), device="cuda"), transpose=False)[0]
    out = q8.matmul(a, w)
    sync()
    av = ref.values(*stored(q8.Q8(a.codes[-3:], a.scales[-3:], k)), k)
    want = av @ ref.values(*stored(w), k, 128).T
    assert np.all(np.abs(np64(out[-3:]) - want) <= 2.0 ** -8 * np.abs(want) + 1e-4)
    dw = q8.wgrad(out, a)
    sync()
    dw64 = torch.zeros((8, k), dtype=torch.float64, device="cuda")
    values = q8.dequantize(a, F32)
    for r in range(0, rows, 65536):
        dw64 += out[r:r + 65536, -8:].double().t() @ values[r:r + 65536].double()
    assert np.linalg.norm(np64(dw[-8:]) - np64(dw64)) <= 2e-6 * np.linalg.norm(np64(dw64))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", [264, 1001])
def test_gradients_in_place(q8, cols, dtype):
    """dz may be da; dh may be dy or dres (aligned rows and rows that start anywhere)."""
    from sub_linear_memory_gb300 import binding

    rows, st = 37, torch.cuda.current_stream().cuda_stream
    f = "" if dtype == BF16 else "_f32"
    z, da = draw((rows, cols), 80, dtype, 2.0), draw((rows, cols), 81, dtype)
    z8 = q8.quantize(z)
    want, buf = q8.gelu_bwd(da, z8), da.clone()
    call = getattr(binding.raw(), "slim_q8_gelu_bwd" + f)
    assert call(buf.data_ptr(), z8.codes.data_ptr(), z8.scales.data_ptr(), buf.data_ptr(), None, None, rows, cols, st) == 0
    sync()
    assert torch.equal(buf, want)
    gamma, rstd = 1 + 0.1 * draw((cols,), 82), torch.rand(rows, device="cuda") + 0.5
    dres = draw((rows, cols), 83, dtype)
    want, _ = q8.rms_norm_bwd(da, z8, rstd, gamma, dres=dres)
    call = getattr(binding.raw(), "slim_q8_rms_norm_bwd" + f)
    for over in ("dy", "dres"):
        dy, dr = da.clone(), dres.clone()
        out = dy if over == "dy" else dr
        assert call(dy.data_ptr(), None, z8.codes.data_ptr(), z8.scales.data_ptr(), rstd.data_ptr(), gamma.data_ptr(),
                    dr.data_ptr(), out.data_ptr(), None, None, 0, rows, cols, st) == 0
        sync()
        assert torch.equal(out, want)
