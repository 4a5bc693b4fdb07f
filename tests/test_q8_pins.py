"""CPU checks of the 8-bit layer operators: the fp64 oracle against what the
format and the formulas fix, and the entry points' refusals on the host (no
GPU work)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import q8 as ref
from sub_linear_memory_gb300 import build

vp = ctypes.c_void_p
P = vp(4096)  # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    build.build()
    from sub_linear_memory_gb300 import q8  # noqa: F401  (signatures)
    from sub_linear_memory_gb300 import binding

    return binding.raw()


# ---- the oracle ---------------------------------------------------------------

def test_codes_are_the_e4m3_numbers():
    raw = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(raw, ref.E4M3)


def test_rounding_is_that_of_the_e4m3_cast():
    """Random values, every midpoint between neighbours and its neighbours."""
    rng = np.random.default_rng(3)
    mid = 0.5 * (ref.E4M3[1:] + ref.E4M3[:-1])
    v = np.concatenate([rng.normal(0, 100, 4000).clip(-448, 448), mid, -mid, mid * (1 + 1e-6), mid * (1 - 1e-6)])
    v = v.astype(np.float32)
    cast = torch.tensor(v).to(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(ref.round_e4m3(v.astype(np.float64)), cast)


@pytest.mark.parametrize("amax, e", [(448.0, 0), (np.nextafter(np.float32(448), np.float32(500)), 1), (1.75, -8),
                                     (1.0, -8), (0.0, -117), (2.0 ** -140, -117), (3.4e38, 120), (896.0, 1)])
def test_exponent_is_the_smallest_that_fits(amax, e):
    assert ref.exponent(float(amax)) == e


def test_held_values_are_bf16_numbers_within_half_a_step():
    rng = np.random.default_rng(4)
    x = rng.normal(size=(7, 300)) * np.exp(3 * rng.normal(size=(7, 1)))
    v = ref.held(x)
    assert np.array_equal(torch.tensor(v).to(torch.bfloat16).to(torch.float64).numpy(), v)
    _, s = ref.quantize(x)
    floor = 2.0 ** (np.repeat(s[:, :3].astype(float), 128, 1)[:, :300] - 127 - 10)  # half the subnormal step
    assert np.all(np.abs(v - x) <= np.maximum(np.abs(x) * 2.0 ** -4, floor))


def test_nonfinite_elements_make_their_block_nan_only():
    x = np.ones((2, 256))
    x[0, 3], x[1, 200] = np.inf, np.nan
    v = ref.held(x)
    assert np.isnan(v[0, :128]).all() and np.isnan(v[1, 128:]).all()
    assert np.isfinite(v[0, 128:]).all() and np.isfinite(v[1, :128]).all()


def test_norm_and_gelu_gradients_match_differences():
    rng = np.random.default_rng(5)
    h, gamma, dy = rng.normal(size=(3, 10)), rng.normal(size=10), rng.normal(size=(3, 10))
    eps, d = 1e-5, 1e-6
    y, rstd = ref.rms_norm(h, gamma, eps)
    dh, dgamma = ref.rms_norm_bwd(dy, h, rstd, gamma)
    f = lambda h, g: float((ref.rms_norm(h, g, eps)[0] * dy).sum())
    for i in range(3):
        for j in range(10):
            up, dn = h.copy(), h.copy()
            up[i, j] += d
            dn[i, j] -= d
            assert abs((f(up, gamma) - f(dn, gamma)) / (2 * d) - dh[i, j]) < 1e-7 * max(1, abs(dh[i, j]) * 10)
    for j in range(10):
        up, dn = gamma.copy(), gamma.copy()
        up[j] += d
        dn[j] -= d
        assert abs((f(h, up) - f(h, dn)) / (2 * d) - dgamma[j]) < 1e-7
    z = np.linspace(-6, 6, 101)
    assert np.abs((ref.gelu(z + d) - ref.gelu(z - d)) / (2 * d) - ref.gelu_slope(z)).max() < 1e-8


# ---- sizes and refusals ---------------------------------------------------------

def test_buffer_sizes(lib):
    assert lib.slim_q8_codes_bytes(3, 130) == 3 * 256
    assert lib.slim_q8_scales_bytes(3, 130, 1) == 3 * 4
    assert lib.slim_q8_scales_bytes(129, 1000, 128) == 2 * 8
    assert lib.slim_q8_codes_bytes(0, 130) == lib.slim_q8_codes_bytes(3, -1) == 0
    assert lib.slim_q8_scales_bytes(3, 130, 64) == 0
    assert lib.slim_q8_codes_bytes(1 << 20, 1 << 14) == 1 << 34  # past 32 bits
    # workspaces: bounded, whatever the number of rows
    assert lib.slim_q8_rms_norm_bwd_workspace_bytes(1 << 20, 1024) == lib.slim_q8_rms_norm_bwd_workspace_bytes(
        1 << 24, 1024) > 0
    assert lib.slim_q8_wgrad_workspace_bytes(1 << 20, 1024, 4096) == lib.slim_q8_wgrad_workspace_bytes(
        1 << 24, 1024, 4096) > 0
    assert lib.slim_q8_rms_norm_bwd_workspace_bytes(8, 16385) == 0


def calls(lib):
    """name -> a call with one argument replaced: call(**{argument: value})."""
    def make(fn, **default):
        return lambda **kw: fn(*{**default, **kw}.values(), None)

    out = {}
    for f in ("", "_f32"):
        out["quantize" + f] = make(getattr(lib, "slim_q8_quantize" + f), x=P, codes=P, scales=P, rows=2, cols=130)
        out["dequantize" + f] = make(getattr(lib, "slim_q8_dequantize" + f), codes=P, scales=P, x=P, rows=2, cols=130,
                                     block_rows=1)
        out["pack_weight" + f] = make(getattr(lib, "slim_q8_pack_weight" + f), x=P, codes=P, scales=P, codes_t=P,
                                      scales_t=P, rows=2, cols=130)
        out["rms_norm" + f] = make(getattr(lib, "slim_q8_rms_norm" + f), x=P, res=P, gamma=P, eps=1e-5, h=P, rstd=P,
                                   codes=P, scales=P, h_codes=P, h_scales=P, rows=2, cols=130)
        out["rms_norm_bwd" + f] = make(getattr(lib, "slim_q8_rms_norm_bwd" + f), x=P, h=None, codes=P, scales=P,
                                       rstd=P, gamma=P, dres=P, dh=P, dgamma=P, ws=P, ws_bytes=1 << 20, rows=2,
                                       cols=130)
        out["gelu" + f] = make(getattr(lib, "slim_q8_gelu" + f), x=P, codes=P, scales=P, z_codes=P, z_scales=P, rows=2,
                               cols=130)
        out["gelu_bwd" + f] = make(getattr(lib, "slim_q8_gelu_bwd" + f), x=P, codes=P, scales=P, dz=P, dz_codes=P,
                                   dz_scales=P, rows=2, cols=130)
        out["matmul" + f] = make(getattr(lib, "slim_q8_matmul" + f), codes=P, scales=P, b_codes=P, b_scales=P, x=P,
                                 rows=2, n=8, cols=130)
    out["wgrad"] = make(lib.slim_q8_wgrad, x=P, codes=P, scales=P, dw=P, accumulate=0, ws=P, ws_bytes=1 << 30, rows=2,
                        n=8, cols=130)
    return out


NAMES = [b + f for b in ("quantize", "dequantize", "pack_weight", "rms_norm", "rms_norm_bwd", "gelu", "gelu_bwd",
                         "matmul") for f in ("", "_f32")] + ["wgrad"]
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.mark.parametrize("name", NAMES)
def test_bad_arguments_are_refused_before_any_launch(lib, name):
    call = calls(lib)[name]
    assert call(rows=-1) == INVALID
    assert call(cols=-1) == INVALID
    for null in ("x", "codes", "scales"):
        assert call(**{null: None}) == INVALID, null
    assert call(codes=vp(4096 + 8)) == UNSUPPORTED
    assert call(scales=vp(4096 + 2)) == UNSUPPORTED
    assert call(x=vp(4097)) == UNSUPPORTED
    assert call(rows=(1 << 31) - 1, cols=4096) == UNSUPPORTED  # 2^31 blocks and more


def test_other_refusals(lib):
    c = calls(lib)
    assert c["dequantize"](block_rows=64) == INVALID
    assert c["pack_weight"](codes_t=None) == INVALID  # scales_t without codes_t
    assert c["rms_norm"](gamma=None) == INVALID
    assert c["rms_norm"](eps=-1.0) == INVALID
    assert c["rms_norm"](eps=float("nan")) == INVALID
    assert c["rms_norm"](cols=0) == INVALID
    assert c["rms_norm"](cols=16385) == UNSUPPORTED
    assert c["rms_norm"](h_scales=None) == INVALID
    assert c["rms_norm_bwd"](h=P) == INVALID  # both kept forms
    assert c["rms_norm_bwd"](codes=None, scales=None) == INVALID  # neither
    assert c["rms_norm_bwd"](cols=0) == INVALID
    assert c["rms_norm_bwd"](cols=16385) == UNSUPPORTED
    assert c["rms_norm_bwd"](ws=None) == WORKSPACE
    assert c["rms_norm_bwd"](ws_bytes=16) == WORKSPACE
    assert c["rms_norm_bwd"](ws=vp(4096 + 4)) == UNSUPPORTED
    assert c["rms_norm_bwd"](rstd=None) == INVALID
    assert c["gelu_bwd"](dz=None) == INVALID
    assert c["gelu_bwd"](dz_codes=None) == INVALID
    assert c["matmul"](b_codes=None) == INVALID
    assert c["matmul"](n=-1) == INVALID
    assert c["matmul"](cols=131073) == UNSUPPORTED
    assert c["wgrad"](dw=None) == INVALID
    assert c["wgrad"](rows=4096, ws_bytes=16) == WORKSPACE
    assert c["wgrad"](rows=4096, ws=None) == WORKSPACE
    assert c["wgrad"](rows=4096, ws=vp(4096 + 4)) == UNSUPPORTED
    assert c["wgrad"](n=-1) == INVALID


@pytest.mark.parametrize("name", NAMES)
def test_nothing_to_write_is_a_no_op(lib, name):
    c = calls(lib)[name]
    none = {k: None for k in ("x", "codes", "scales")}
    if name == "wgrad":
        assert c(n=0, **none) == 0  # no rows: dw is zeroed, on the GPU
    elif name.startswith("rms_norm_bwd"):
        assert c(rows=0, dgamma=None, **none) == 0
    else:
        assert c(rows=0, **none) == 0
        if "norm" not in name and "matmul" not in name:
            assert c(cols=0, **none) == 0


def test_python_checks():
    build.build()
    from sub_linear_memory_gb300 import q8

    cpu = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        q8.quantize(cpu)
    bad = q8.Q8(torch.zeros(2, 128, dtype=torch.float8_e4m3fn), torch.zeros(2, 4, dtype=torch.uint8), 8)
    for call in (lambda: q8.dequantize(bad), lambda: q8.matmul(bad, bad), lambda: q8.gelu_bwd(cpu, bad),
                 lambda: q8.wgrad(cpu, bad), lambda: q8.rms_norm(cpu, cpu[0]),
                 lambda: q8.rms_norm_bwd(cpu, bad, cpu[0], cpu[0]), lambda: q8.pack_weight(cpu), lambda: q8.gelu(cpu)):
        with pytest.raises(ValueError):
            call()


def test_register_shares_hold_without_spills(tmp_path):
    """The weight gradient's warpgroups trade registers (setmaxnreg): each role
    has to fit its share, so the kernel must compile without spills."""
    import os
    import shutil
    import subprocess

    nvcc = os.environ.get("NVCC", "nvcc")
    if shutil.which(nvcc) is None:
        pytest.skip("no nvcc")
    src = os.path.join(build.CSRC, "q8_wgrad.cu")
    out = subprocess.run([nvcc, *build.ARCH, *build.FLAGS, "-Xptxas", "-v", "-c", src, "-o", str(tmp_path / "w.o")],
                         capture_output=True, text=True, check=True)
    spills = [line for line in (out.stdout + out.stderr).splitlines() if "spill stores" in line]
    assert spills and all("0 bytes spill stores, 0 bytes spill loads" in line for line in spills)
