"""rope_axes on the GPU against the float64 form (oracle/layer_ops.py).

Tolerance. The reduced angle is at most pi and rounded to float32 in units of pi (2^-25 pi, about
1e-7), sincospif is off by about 2 steps (2^-23): cos and sin by less than 4.4e-7. With the two
products and their sum, an element is off by at most 2^-20 (|u| + |v|) of its pair, then half a step
of the output's type."""
import numpy as np
import pytest
import torch

import epilogues_nvfp4_quantize_b200 as ep
from oracle import layer_ops as lo
from gpu_util import device

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def inputs(rows, heads, hd, pairs, dtype, far=0, fraction=False, seed=0):
    g = torch.Generator().manual_seed(seed + rows + hd)
    x = torch.randn(rows, heads, hd, generator=g).to(TYPES[dtype]).to(device())
    pos = torch.randint(0, 200, (rows, len(pairs)), generator=g) + far
    pos = (pos.float() * 0.75 - 20.5) if fraction else pos.int()
    return x, pos.to(device()), ep.rope_frequencies(pairs, device=device())


def check(y, x, pos, freqs, pairs, interleaved, inverse=False):
    xf = x.double().cpu().numpy()
    ref = lo.rope(xf, pos.double().cpu().numpy(), freqs.cpu().numpy(), pairs, interleaved, inverse)
    n = sum(pairs)
    i = np.arange(n)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, n + i)
    size = np.zeros_like(xf)
    size[..., a] = size[..., b] = np.abs(xf[..., a]) + np.abs(xf[..., b])
    err = 2.0 ** -20 * size
    tol = err + torch.finfo(x.dtype).eps / 2 * (np.abs(ref) + err) + (2.0 ** -25 if x.dtype == torch.float16 else 0)
    got = y.double().cpu().numpy()
    d = np.abs(got - ref)
    assert np.array_equal(got[..., 2 * n:], xf[..., 2 * n:]), "elements past the pairs"
    assert not (d > tol).any(), f"{int((d > tol).sum())} of {d.size}, worst {np.max(d / tol):.3g} of the tolerance"


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("rows,heads,hd,pairs", [
    (1, 1, 8, [4]), (1, 1, 8, [1]), (5, 3, 64, [32]), (77, 2, 64, [8, 12, 12]), (33, 5, 96, [16, 8, 8]),
    (130, 24, 128, [16, 24, 24]), (3, 1, 256, [30, 1, 1, 64]), (19, 2, 256, [3, 50]), (2, 40, 1024, [200, 312]),
    (9, 300, 16, [3, 2])])
def test_layouts(dtype, interleaved, rows, heads, hd, pairs):
    x, pos, freqs = inputs(rows, heads, hd, pairs, dtype)
    check(ep.rope_axes(x, pos, freqs, pairs, interleaved=interleaved), x, pos, freqs, pairs, interleaved)


@pytest.mark.parametrize("interleaved", [True, False])
def test_many_rows_per_block(interleaved):
    """Enough rows that a CTA holds several, with a last one that is not full."""
    pairs = [4, 6, 6]
    x, pos, freqs = inputs(20011, 2, 64, pairs, "bf16")
    check(ep.rope_axes(x, pos, freqs, pairs, interleaved=interleaved), x, pos, freqs, pairs, interleaved)


@pytest.mark.parametrize("far,fraction", [(1 << 20, False), (2 ** 31 - 300, False), (1 << 20, True), (-5000, False)])
def test_far_positions(far, fraction):
    pairs = [32, 32]
    x, pos, freqs = inputs(40, 2, 128, pairs, "f32", far, fraction)
    check(ep.rope_axes(x, pos, freqs, pairs), x, pos, freqs, pairs, True)


@pytest.mark.parametrize("interleaved", [True, False])
def test_heads_inside_a_qkv_buffer_in_place_and_transposed(interleaved):
    rows, heads, hd, pairs = 50, 4, 128, [16, 24, 20]
    _, pos, freqs = inputs(rows, heads, hd, pairs, "bf16")
    qkv = torch.randn(rows, 3 * heads * hd, device=device()).bfloat16()
    before = qkv.clone()
    qk = qkv[:, :2 * heads * hd].view(rows, 2 * heads, hd)
    out = torch.zeros(2 * heads, rows, hd, dtype=torch.bfloat16, device=device())
    ep.rope_axes(qk, pos, freqs, pairs, out.transpose(0, 1), interleaved=interleaved)
    check(out.transpose(0, 1), qk, pos, freqs, pairs, interleaved)
    ep.rope_axes(qk, pos, freqs, pairs, qk, interleaved=interleaved)
    assert torch.equal(qk, out.transpose(0, 1))
    assert torch.equal(qkv[:, 2 * heads * hd:], before[:, 2 * heads * hd:])
    # positions as columns of a wider table
    table = torch.zeros(rows, 7, dtype=torch.int32, device=device())
    table[:, 2:5] = pos
    src = before[:, :2 * heads * hd].view(rows, 2 * heads, hd)
    assert torch.equal(ep.rope_axes(src, table[:, 2:5], freqs, pairs, interleaved=interleaved), qk)


def test_elements_past_the_pairs_keep_infinities_and_nan():
    pairs = [5]
    x, pos, freqs = inputs(4, 2, 64, pairs, "bf16")
    x[..., 10:] = float("inf")
    x[..., 11] = float("nan")
    for inter in (True, False):
        y = ep.rope_axes(x, pos, freqs, pairs, interleaved=inter)
        assert bool(torch.isfinite(y[..., :10]).all())
        assert torch.equal(torch.isnan(y[..., 10:]), torch.isnan(x[..., 10:])) and bool((y[..., 12:] == float("inf")).all())


@pytest.mark.parametrize("interleaved", [True, False])
def test_gradient_is_the_opposite_rotation(interleaved):
    pairs = [10, 22]
    x, pos, freqs = inputs(30, 3, 80, pairs, "f32")
    x.requires_grad_(True)
    dy = torch.randn(30, 80, 3, device=device()).transpose(1, 2)  # a gradient with another order
    y = ep.RopeAxes.apply(x, pos, freqs, pairs, interleaved)
    check(y.detach(), x.detach(), pos, freqs, pairs, interleaved)
    y.backward(dy)
    check(x.grad, dy, pos, freqs, pairs, interleaved, inverse=True)
    # against differences of the forward pass: sum(dy (y(x + e) - y(x - e))) / 2 = sum(x.grad e)
    e = torch.randn_like(x.detach())
    with torch.no_grad():
        up = ep.rope_axes(x + e, pos, freqs, pairs, interleaved=interleaved)
        down = ep.rope_axes(x - e, pos, freqs, pairs, interleaved=interleaved)
    want = float((dy.double() * (up.double() - down.double())).sum()) / 2
    got = float((x.grad.double() * e.double()).sum())
    size = float((dy.abs().double() * (x.detach().abs() + e.abs()).double()).sum())
    assert abs(got - want) <= 2.0 ** -18 * size


def test_other_stream_and_graph():
    pairs = [16, 16]
    x, pos, freqs = inputs(64, 4, 64, pairs, "bf16")
    want = ep.rope_axes(x, pos, freqs, pairs)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = torch.zeros_like(x)
    ep.rope_axes(x, pos, freqs, pairs, y, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    made = ep.rope_axes(x, pos, freqs, pairs, stream=s)
    s.synchronize()
    assert torch.equal(made, want)
    at = made.data_ptr()
    owners = [g["stream"] for g in torch.cuda.memory_snapshot() if g["address"] <= at < g["address"] + g["total_size"]]
    assert owners == [s.cuda_stream]  # its memory is the stream's own
    z = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.rope_axes(x, pos, freqs, pairs, z)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(z, want)
    assert ep.read_device_status() == 0
