"""gemv_nvfp4 with SiLU at float32's digits, and several passes over a weight that clusters share.

SiLU alone: the weight has one value in each row, so an output is one product and no sum hides what SiLU's own
rounding does. v = SiLU(x) is within 2^-21 of itself in float32 (expf 2^-22, the sum 2^-24, the reciprocal
2^-23, the product 2^-24; where 1 + e^-x passes 2^126 it is 0, off by less than 2^-119). Its two f16 parts
leave 2^-22 of it, or 2^-39 of the largest of its 128 columns where the second part has no bits left (1.01 times
that, since the largest is rounded to bf16 before it chooses the power of two).
Adding the two products in the tensor core costs 2^-23, the factors (block scale, row, per-tensor scale)
2^-24 each: 2^-21 + 2^-22 + 2^-23 + 3 2^-24 < 2^-20 (1 + 1/8 + ...) in all, 2^-19 with a half to spare."""
import numpy as np
import pytest
import torch

import epilogues_nvfp4_quantize_b200 as ep
from oracle import layer_ops as lo
from gpu_util import device, nvfp4_from_arrays

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def silu64(x):
    with np.errstate(over="ignore"):
        return x / (1.0 + np.exp(-x))


def one_value_per_row(K, seed):
    """An NVFP4 weight of K rows, row n with one value, at column n; and these values without G."""
    r = np.random.default_rng(seed)
    codes, scales = np.zeros((K, K), np.uint8), np.full((K, K // 16), 0x38, np.uint8)  # scale 1
    i = np.arange(K)
    codes[i, i] = np.where(r.random(K) < 0.5, 2, 13)  # +1 and -3
    scales[i, i // 16] = np.where(r.random(K) < 0.5, 0x38, 0x41)  # 1 and 2.25
    w = np.where(codes[i, i] == 2, 1.0, -3.0) * np.where(scales[i, i // 16] == 0x38, 1.0, 2.25)
    return codes, scales, w


@pytest.mark.parametrize("M", [1, 2, 3, 8, 13, 16, 19])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("K,spread", [(64, 3.0), (256, 30.0), (1024, 8.0), (2112, 60.0)])
def test_silu_has_float32_digits(M, dtype, K, spread):
    codes, scales, w = one_value_per_row(K, K)
    G = np.float32(0.37)
    r = np.random.default_rng(M + K)
    x = torch.from_numpy(np.clip(r.standard_normal((M, K)) * spread, -86, 86)).to(TYPES[dtype])
    D = torch.empty(M, K, device=device())
    ep.gemv_nvfp4(x.to(device()), nvfp4_from_arrays(codes, scales, G), D, silu=True)
    v = silu64(x.double().numpy())
    ref = v * w * float(G)
    # the largest |v| of each value's 128 columns
    pad = np.zeros((M, -(-K // 128) * 128))
    pad[:, :K] = np.abs(v)
    top = np.repeat(pad.reshape(M, -1, 128).max(2), 128, 1)[:, :K]
    tol = 2.0 ** -19 * np.abs(ref) + (1.01 * 2.0 ** -39 * top + 2.0 ** -119) * np.abs(w) * float(G)
    err = np.abs(D.double().cpu().numpy() - ref)
    assert (err <= tol).all(), f"{int((err > tol).sum())} of {err.size}, worst {np.max(err / tol):.3g} of the tolerance"


@pytest.mark.parametrize("M", [1, 2, 5, 16])
def test_infinities_nan_and_the_largest_values_through_silu(M):
    K, N = 256, 130
    B = nvfp4_from_arrays(np.full((N, K), 2, np.uint8), np.full((N, K // 16), 0x38, np.uint8), 1.0)  # all +1
    x = torch.linspace(-20, 20, M * K).view(M, K).to(torch.bfloat16).to(device())
    D, plain = torch.empty(2, M, N, device=device())
    ep.gemv_nvfp4(x, B, plain, silu=True)
    for value, holds in ((float("inf"), lambda d: d == float("inf")), (float("nan"), torch.isnan),
                         (float("-inf"), torch.isnan),  # -inf / inf
                         (3e38, lambda d: (d - float(torch.tensor(3e38).bfloat16())).abs() <= 2.0 ** -19 * 3e38)):
        for row in {0, M - 1}:
            y = x.clone()
            y[row, 200] = value
            ep.gemv_nvfp4(y, B, D, silu=True)
            others = torch.arange(M, device=device()) != row
            assert bool(holds(D[row]).all()), (value, row)
            assert torch.equal(D[others], plain[others]), (value, row)


def weight(N, K, seed):
    r = np.random.default_rng(seed)
    return r.integers(0, 16, (N, K)).astype(np.uint8), r.integers(0x20, 0x50, (N, K // 16)).astype(np.uint8), np.float32(1e-3)


def check_against_the_form(M, N, K, silu, out):
    """Tolerance: products are exact (SiLU's within 2^-20 as above). A step of 128 columns adds at most 16
    instructions' sums one after another, steps, warps and CTAs K / 128 + 24 more in float32, each off by at
    most 2^-23 of sum |x w|; factors and bias 2^-22; then half a step of the output's type."""
    arrays = weight(N, K, N + K)
    r = np.random.default_rng(M)
    x = torch.from_numpy(r.standard_normal((M, K)) * 2).to(torch.bfloat16)
    bias = r.standard_normal(N).astype(np.float32)
    B, xd, bd = nvfp4_from_arrays(*arrays), x.to(device()), torch.from_numpy(bias).to(device())
    D, E = torch.empty(2, M, N, dtype=TYPES[out], device=device())
    ep.gemv_nvfp4(xd, B, D, bias=bd, silu=silu)
    ep.gemv_nvfp4(xd, B, E, bias=bd, silu=silu)
    assert torch.equal(D, E), "the same inputs give the same bits"
    ref, size = lo.gemv(x.double().numpy(), *arrays, bias=bias, silu=silu)
    err = (K / 128 + 40) * 2.0 ** -23 * size + 2.0 ** -22 * (np.abs(ref) + np.abs(bias)) + (2.0 ** -20 * size if silu else 0)
    tol = err + torch.finfo(TYPES[out]).eps / 2 * (np.abs(ref) + err)
    d = np.abs(D.double().cpu().numpy() - ref)
    assert (d <= tol).all(), f"{int((d > tol).sum())} of {d.size}, worst {np.max(d / tol):.3g} of the tolerance"
    assert ep.read_device_status() == 0


@pytest.mark.parametrize("M", [17, 33, 40])
@pytest.mark.parametrize("N,K,silu,out", [(9000, 4096, False, "f32"), (4099, 4096, True, "f32"), (2300, 12288, False, "bf16"),
                                          (2300, 12288, True, "f32")])
def test_several_passes_with_several_rounds_of_joins(M, N, K, silu, out):
    check_against_the_form(M, N, K, silu, out)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 16])
@pytest.mark.parametrize("N,K,out", [(20011, 4096, "f32"), (9001, 6208, "f16")])
def test_silu_of_few_rows_with_several_rounds_of_joins(M, N, K, out):
    check_against_the_form(M, N, K, True, out)


@pytest.mark.parametrize("M,K", [(2, 32768), (7, 32768), (8, 32768), (9, 10240), (16, 10304), (12, 16384), (20, 30016)])
def test_silu_of_long_rows(M, K):
    """Where two f16 for each of 16 or 8 rows do not fit in a cluster, fewer rows are taken at a time."""
    check_against_the_form(M, 300, K, True, "f32")


def test_more_passes_than_a_grid_has_rows():
    """4 rows at a time and 65536 passes: the passes' second dimension."""
    M, N, K = 4 * 65535 + 6, 16, 32768
    B = nvfp4_from_arrays(*weight(N, K, 1))
    base = torch.randn(8, K, generator=torch.Generator().manual_seed(1)).bfloat16().to(device())
    want = torch.empty(8, N, device=device())
    ep.gemv_nvfp4(base, B, want, silu=True)
    x = base.repeat((M + 7) // 8, 1)[:M]
    D = torch.full((M + 1, N), 7.0, device=device())
    ep.gemv_nvfp4(x, B, D[:M], silu=True)
    torch.cuda.synchronize()
    i = torch.arange(M, device=device()) % 8
    assert torch.equal(D[:M], want[i]) and bool((D[M] == 7.0).all())
    del x, base
    torch.cuda.empty_cache()


@pytest.mark.parametrize("silu", [False, True])
def test_rows_near_the_smallest_bf16(silu):
    """Rows of magnitude 2^-108 to 2^-133. Below float32's smallest normal number a sum's step is 2^-149; SiLU may be
    off by 2^-119 for each column."""
    N, K = 130, 320
    arrays = (*weight(N, K, 4)[:2], np.float32(1.0))
    r = np.random.default_rng(5)
    xv = r.standard_normal((5, K)) * 2.0 ** np.array([[-108.0], [-113], [-120], [-126], [-131]])
    x = torch.from_numpy(xv).to(torch.bfloat16)
    D = torch.empty(5, N, device=device())
    ep.gemv_nvfp4(x.to(device()), nvfp4_from_arrays(*arrays), D, silu=silu)
    ref, size = lo.gemv(x.double().numpy(), *arrays, silu=silu)
    tol = (K / 128 + 40) * 2.0 ** -23 * size + (K / 16 + 64) * 2.0 ** -149
    if silu:
        _, weights = lo.gemv(np.ones((1, K)), *arrays)
        tol = tol + 2.0 ** -20 * size + 2.0 ** -119 * weights
    err = np.abs(D.double().cpu().numpy() - ref)
    assert (err <= tol).all(), f"worst {np.max(err / tol):.3g} of the tolerance"
    assert silu or float(np.abs(ref[-1]).max()) > 0
