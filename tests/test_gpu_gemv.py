"""gemv_nvfp4 on the GPU against the float64 form (oracle/layer_ops.py).

Tolerance. The weights are exact in f16 and so are bf16 activations down to 2^-28 of their row's
largest (2^-39 of it below that), so products are exact; what is left is float32 sums. One warp adds
16 products per instruction, at most K / 16 of them one after another, then at most 16 warps and 8
CTAs; each addition is off by at most 2^-23 of sum |x w| (2^-24 if it rounds, 2^-23 if it truncates).
With the scale, the row factor and the bias: (K / 16 + 48) 2^-23 sum |x w| + 2^-22 (|y| + |bias|), then
half a step of the output's type. SiLU's result is rounded to f16, half a step of each term (2^-11),
and SiLU in float32 is itself off by a few 2^-24 (1 + |x|) of it, for |x| < 100 covered by 1.02."""
import numpy as np
import pytest
import torch

import epilogues_nvfp4_quantize_b200 as ep
from oracle import layer_ops as lo
from gpu_util import device, nvfp4_from_arrays

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def weight(N, K, seed, zero_blocks=True):
    r = np.random.default_rng(seed)
    codes = r.integers(0, 16, (N, K)).astype(np.uint8)
    scales = r.integers(0x20, 0x50, (N, K // 16)).astype(np.uint8)
    if zero_blocks:
        scales[r.random((N, K // 16)) < 0.05] = 0
        scales[0, 0], scales[-1, -1] = 0x7E, 0x01  # the largest and the smallest E4M3 value
    return codes, scales, np.float32(0.0037 / np.sqrt(K))


def check(x, B, arrays, out, bias=None, silu=False, ld_extra=0):
    M, K = x.shape
    N = arrays[0].shape[0]
    buf = torch.full((M + 2, N + ld_extra + 3), 7.0, dtype=TYPES[out], device=device())
    D = buf[1:M + 1, 1:N + 1]
    b = None if bias is None else torch.from_numpy(bias).to(device())
    ep.gemv_nvfp4(x, B, D, bias=b, silu=silu)
    torch.cuda.synchronize()
    got = D.double().cpu().numpy()
    xf = x.double().cpu().numpy()
    ref, size = lo.gemv(xf, *arrays, bias=bias, silu=silu)
    half = torch.finfo(TYPES[out]).eps / 2
    err = (K / 16 + 48) * 2.0 ** -23 * size + 2.0 ** -22 * (np.abs(ref) + (0 if bias is None else np.abs(bias)))
    if silu:
        err += 1.02 * 2.0 ** -11 * size
    tol = err + half * (np.abs(ref) + err) + (2.0 ** -25 if out == "f16" else 0.0)  # f16's subnormal step
    over = np.abs(got - ref) > tol
    assert not over.any(), f"{int(over.sum())} of {over.size}, worst {np.max(np.abs(got - ref) / tol):.3g} of the tolerance"
    edge = torch.ones_like(buf, dtype=torch.bool)
    edge[1:M + 1, 1:N + 1] = False
    assert bool((buf[edge] == 7.0).all()), "written outside D"


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 40])
@pytest.mark.parametrize("N,K", [(128, 64), (1, 64), (130, 192), (1000, 1024)])
def test_row_counts_and_ragged_widths(M, N, K):
    arrays = weight(N, K, M + N + K)
    r = np.random.default_rng(M)
    x = torch.from_numpy(r.standard_normal((M, K))).to(torch.bfloat16).to(device())
    check(x, nvfp4_from_arrays(*arrays), arrays, "bf16")


@pytest.mark.parametrize("N,K", [(2304, 4096), (4099, 12288), (64, 32768), (6000, 2112), (40000, 128)])
@pytest.mark.parametrize("M,x,out,silu,bias", [(1, "bf16", "f32", False, True), (3, "bf16", "bf16", True, True),
                                               (8, "f16", "f16", False, False), (13, "f16", "f32", False, True),
                                               (16, "bf16", "f16", True, False)])
def test_types_activation_bias(N, K, M, x, out, silu, bias):
    arrays = weight(N, K, N + K)
    r = np.random.default_rng(N + M)
    xv = r.standard_normal((M, K))
    xv[:, :: max(1, K // 8)] *= 20.0
    b = r.standard_normal(N).astype(np.float32) if bias else None
    check(torch.from_numpy(xv).to(TYPES[x]).to(device()), nvfp4_from_arrays(*arrays), arrays, out, b, silu)


@pytest.mark.parametrize("M,N,K", [(1, 20011, 4096), (2, 33000, 2048), (5, 20011, 4096), (13, 20011, 4096), (16, 9000, 8192)])
def test_many_strips_per_cluster(M, N, K):
    """Several rounds of joins across the CTAs that share K, the last one not full."""
    arrays = weight(N, K, N + K)
    r = np.random.default_rng(M + N)
    x = torch.from_numpy(r.standard_normal((M, K))).to(torch.bfloat16).to(device())
    B = nvfp4_from_arrays(*arrays)
    check(x, B, arrays, "f32", r.standard_normal(N).astype(np.float32))
    D, E = torch.empty(2, M, N, device=device())
    for _ in range(3):
        ep.gemv_nvfp4(x, B, D), ep.gemv_nvfp4(x, B, E)
        assert torch.equal(D, E), "the same inputs give the same bits"


def test_rows_of_very_different_size_and_strides():
    N, K = 256, 1024
    arrays = weight(N, K, 5)
    r = np.random.default_rng(6)
    size = 10.0 ** np.array([[-30.0], [-8], [0], [9], [25], [0]])
    xv = r.standard_normal((6, K)) * size
    xv[5] = 0.0  # an all-zero row
    wide = torch.zeros(6, K + 64, dtype=torch.bfloat16, device=device())
    wide[:, 8:K + 8] = torch.from_numpy(xv).to(torch.bfloat16).to(device())
    x = wide[:, 8:K + 8]
    check(x, nvfp4_from_arrays(*arrays), arrays, "f32", ld_extra=5)


def test_wide_range_within_a_row():
    """Values over 2^60 within a row: those below 2^-28 of the largest may be off by 2^-39 of it,
    which the sums' tolerance covers."""
    N, K = 130, 256
    arrays = weight(N, K, 8)
    r = np.random.default_rng(9)
    xv = r.standard_normal((2, K)) * 2.0 ** r.integers(-40, 20, (2, K))
    check(torch.from_numpy(xv).to(torch.bfloat16).to(device()), nvfp4_from_arrays(*arrays), arrays, "f32")


def test_infinities_and_nan_stay_in_their_row():
    N, K = 200, 192
    arrays = weight(N, K, 10, zero_blocks=False)
    arrays[0][:, 5] = 2  # a weight of +1 in every row where x is infinite
    r = np.random.default_rng(11)
    x = torch.from_numpy(r.standard_normal((4, K)) * 1e30).to(torch.bfloat16).to(device())
    x[0, 5] = float("inf")
    x[2, 7] = float("nan")
    B = nvfp4_from_arrays(*arrays)
    D = torch.empty(4, N, dtype=torch.float32, device=device())
    ep.gemv_nvfp4(x, B, D)
    assert bool((D[0] == float("inf")).all()) and bool(torch.isnan(D[2]).all())
    assert bool(torch.isfinite(D[1]).all()) and bool(torch.isfinite(D[3]).all())
    clean = x.clone()
    clean[0], clean[2] = 0, 0
    E = torch.empty_like(D)
    ep.gemv_nvfp4(clean, B, E)
    assert torch.equal(D[1], E[1]) and torch.equal(D[3], E[3])


def test_quantised_weight_other_stream_and_graph():
    """A weight packed by nvfp4_quantize; on a side stream and from a captured graph the bits are
    those of the plain call."""
    N, K, M = 1536, 1024, 4
    g = torch.Generator().manual_seed(3)
    w = (torch.randn(N, K, generator=g) / 32).to(torch.bfloat16).to(device())
    x = torch.randn(M, K, generator=g).to(torch.bfloat16).to(device())
    B = ep.nvfp4_quantize(w, ep.NVFP4Tensor.empty(N, K, device()))
    D = torch.empty(M, N, dtype=torch.bfloat16, device=device())
    ep.gemv_nvfp4(x, B, D, silu=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    D2, D3 = torch.zeros_like(D), torch.zeros_like(D)
    ep.gemv_nvfp4(x, B, D2, silu=True, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.gemv_nvfp4(x, B, D3, silu=True)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(D, D2) and torch.equal(D, D3)
    assert ep.read_device_status() == 0
