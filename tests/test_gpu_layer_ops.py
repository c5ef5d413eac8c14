"""The operators between a layer's GEMMs together, as a DiT layer uses them: modulation vectors from a
few-row product, the first norm into the QKV projection's NVFP4 operand, rotary positions on its Q and
K heads, the branch added with its gate and the second norm, the FFN; every stage against its float64
form on what the stage before really produced. The same step replayed from a captured graph; the
training operators chained under autograd; offsets past 32 bits; two calls at once."""
import numpy as np
import pytest
import torch

import epilogues_nvfp4_quantize_b200 as ep
from oracle import layer_ops as lo
from oracle import nvfp4_oracle as o
import workloads as wk
from gpu_util import REL_TOL, assert_close, device, quantize_gpu, read_nvfp4

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy()


class Layer:
    """One layer's buffers and its step: M tokens in two images of different size, width D."""

    def __init__(self, M=256, D=512, heads=4, hd=128, nh=512):
        dev = device()
        T = ep.NVFP4Tensor
        g = torch.Generator().manual_seed(0)
        rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.M, self.D, self.heads, self.hd, self.nh = M, D, heads, hd, nh
        pack = lambda n, k, s, **kw: ep.nvfp4_quantize(wk.weights(n, k, 1 / np.sqrt(k), seed=s).to(dev), T.empty(n, k, dev), **kw)  # noqa: E731
        self.Wm = pack(6 * D, D, 1)
        self.Wq, self.Wo = pack(3 * heads * hd, D, 2), pack(D, heads * hd, 3)
        self.Wu, self.Wd = pack(2 * nh, D, 4, interleave=True), pack(D, nh, 5)
        self.bias_m = (0.1 * rn(6 * D)).to(dev)
        self.cond = rn(2, D).bfloat16().to(dev)
        self.x0 = (rn(M, D) * 1.5).bfloat16().to(dev)
        self.x = self.x0.clone()
        self.offsets = torch.tensor([0, 100, M], dtype=torch.int32, device=dev)
        self.w_heads = (1 + 0.1 * rn(2 * heads * hd)).to(dev)
        self.pairs = [16, 24, 24]
        self.freqs = ep.rope_frequencies(self.pairs, device=dev)
        self.pos = torch.stack([torch.zeros(M), torch.arange(M) // 16, torch.arange(M) % 16], 1).int().to(dev)
        bf = dict(dtype=torch.bfloat16, device=dev)
        self.mod = torch.empty(2, 6 * D, **bf)
        self.h1, self.h2, self.a, self.f = T.empty(M, D, dev), T.empty(M, D, dev), T.empty(M, heads * hd, dev), T.empty(M, nh, dev)
        for t, s in ((self.h1, 0.004), (self.h2, 0.004), (self.a, 0.003), (self.f, 0.004)):
            t.gscale.fill_(s)
        self.qkv, self.attn, self.down = torch.empty(M, 3 * heads * hd, **bf), torch.empty(M, D, **bf), torch.empty(M, D, **bf)

    def m(self, i):
        return self.mod[:, i * self.D:(i + 1) * self.D]

    def step(self):
        n = 2 * self.heads * self.hd
        ep.gemv_nvfp4(self.cond, self.Wm, self.mod, bias=self.bias_m, silu=True)
        ep.residual_norm(self.x, hq=self.h1, scale=self.m(0), shift=self.m(1), offsets=self.offsets)
        ep.gemm_nvfp4_rmsnorm(self.h1, self.Wq, self.w_heads, self.hd, n, 1e-6, self.qkv)
        qk = self.qkv[:, :n].view(self.M, 2 * self.heads, self.hd)
        ep.rope_axes(qk, self.pos, self.freqs, self.pairs, qk)
        # (the attention itself is not this library's: V stands for its output)
        ep.nvfp4_quantize(self.qkv[:, n:], self.a, compute_amax=False)
        ep.gemm_nvfp4_plain(self.a, self.Wo, self.attn)
        ep.residual_norm(self.x, hq=self.h2, y=self.attn, x_out=self.x, gate=self.m(2), scale=self.m(3), shift=self.m(4),
                         offsets=self.offsets)
        ep.gemm_nvfp4_swiglu(self.h2, self.Wu, None, self.f)
        ep.gemm_nvfp4_plain(self.f, self.Wd, self.down)
        ep.residual_norm(self.x, y=self.down, x_out=self.x, gate=self.m(5), norm=None, offsets=self.offsets)


def _values(t):
    q, s, G, _ = read_nvfp4(t)
    return o.dequantize(q, s, G).astype(np.float64)


def test_a_layer_stage_by_stage():
    L = Layer()
    n, D = 2 * L.heads * L.hd, L.D
    b = lo.sequences(L.M, 2, L.offsets.tolist())
    ep.gemv_nvfp4(L.cond, L.Wm, L.mod, bias=L.bias_m, silu=True)
    q, s, G, _ = read_nvfp4(L.Wm)
    ref, size = lo.gemv(f64(L.cond), q, s, G, f64(L.bias_m), silu=True)
    # SiLU's rounding to f16 on every term, then the output's
    assert (np.abs(f64(L.mod) - ref) <= 2.0 ** -11 * 1.02 * size + 2.0 ** -8 * np.abs(ref) + 2.0 ** -16).all()

    ep.residual_norm(L.x, hq=L.h1, scale=L.m(0), shift=L.m(1), offsets=L.offsets)
    h = torch.empty(L.M, D, dtype=torch.bfloat16, device=device())
    ep.residual_norm(L.x, h, scale=L.m(0), shift=L.m(1), offsets=L.offsets)
    want = quantize_gpu(h.cpu(), G=L.h1.gscale.item())
    assert torch.equal(want.codes, L.h1.codes) and torch.equal(want.sf, L.h1.sf)
    href = lo.modulated_norm(f64(L.x), b, "layer", None, f64(L.m(0)), f64(L.m(1)))
    assert (np.abs(f64(h) - href) <= 2.0 ** -8 * np.abs(href) + 2.0 ** -16).all()

    ep.gemm_nvfp4_rmsnorm(L.h1, L.Wq, L.w_heads, L.hd, n, 1e-6, L.qkv)
    c = _values(L.h1) @ _values(L.Wq).T
    heads = c[:, :n].reshape(L.M, 2 * L.heads, L.hd)
    heads = heads / np.sqrt((heads ** 2).mean(-1, keepdims=True) + 1e-6)
    c[:, :n] = heads.reshape(L.M, n) * f64(L.w_heads)
    assert_close(f64(L.qkv), c, "QKV")

    before = f64(L.qkv)
    qk = L.qkv[:, :n].view(L.M, 2 * L.heads, L.hd)
    ep.rope_axes(qk, L.pos, L.freqs, L.pairs, qk)
    ref = lo.rope(before[:, :n].reshape(L.M, 2 * L.heads, L.hd), f64(L.pos), f64(L.freqs), L.pairs)
    assert (np.abs(f64(qk) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * np.abs(before).max()).all()
    assert np.array_equal(f64(L.qkv)[:, n:], before[:, n:])

    ep.nvfp4_quantize(L.qkv[:, n:], L.a, compute_amax=False)
    ep.gemm_nvfp4_plain(L.a, L.Wo, L.attn)
    xr = lo.residual(f64(L.x), f64(L.attn), b, f64(L.m(2)))
    ep.residual_norm(L.x, hq=L.h2, y=L.attn, x_out=L.x, gate=L.m(2), scale=L.m(3), shift=L.m(4), offsets=L.offsets)
    assert (np.abs(f64(L.x) - xr) <= 2.0 ** -8 * np.abs(xr) + 2.0 ** -18).all()
    ep.gemm_nvfp4_swiglu(L.h2, L.Wu, None, L.f)
    ep.gemm_nvfp4_plain(L.f, L.Wd, L.down)
    assert_close(f64(L.down), _values(L.f) @ _values(L.Wd).T, "down")
    xr = lo.residual(f64(L.x), f64(L.down), b, f64(L.m(5)))
    ep.residual_norm(L.x, y=L.down, x_out=L.x, gate=L.m(5), norm=None, offsets=L.offsets)
    assert (np.abs(f64(L.x) - xr) <= 2.0 ** -8 * np.abs(xr) + 2.0 ** -18).all()
    assert REL_TOL == 2e-2 and ep.read_device_status() == 0


def test_a_layer_replayed_from_a_graph():
    L = Layer()
    L.step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (L.mod, L.qkv, L.attn, L.down, L.x, L.h1.codes, L.h2.codes, L.f.codes)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            L.step()
    for t in (L.mod, L.qkv, L.attn, L.down):
        t.zero_()
    for _ in range(3):
        L.x.copy_(L.x0)
        graph.replay()
    torch.cuda.synchronize()
    got = (L.mod, L.qkv, L.attn, L.down, L.x, L.h1.codes, L.h2.codes, L.f.codes)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert ep.read_device_status() == 0


def test_training_operators_together():
    """x, y -> residual norm -> fake quantisation (gradient passes through) -> rotary heads -> loss."""
    rows, heads, hd, pairs = 64, 4, 64, [12, 20]
    cols = heads * hd
    g = torch.Generator().manual_seed(4)
    rn = lambda *s: torch.randn(*s, generator=g).to(device())  # noqa: E731
    x = rn(rows, cols).requires_grad_(True)
    y = (rn(rows, cols)).bfloat16().requires_grad_(True)
    gate, scale, shift = ((0.5 * rn(2, cols)).requires_grad_(True) for _ in range(3))
    pos = torch.randint(0, 64, (rows, 2), generator=g).int().to(device())
    freqs = ep.rope_frequencies(pairs, device=device())
    cx, cq = rn(rows, cols), rn(rows, heads, hd).bfloat16()
    x_out, h = ep.ResidualNorm.apply(x, y, gate, scale, shift)
    q = ep.FakeQuantizeSTE.apply(h)
    r = ep.RopeAxes.apply(q.view(rows, heads, hd), pos, freqs, pairs)
    ((x_out * cx).sum() + (r * cq).float().sum()).backward()
    # the gradient of h: the loss's, turned back and rounded to bf16
    dh = torch.from_numpy(lo.rope(f64(cq), f64(pos), f64(freqs), pairs, inverse=True)).reshape(rows, cols)
    b = lo.sequences(rows, 2)
    ref = lo.residual_norm_backward(f64(x_out), b, 2, f64(cx), f64(dh.bfloat16()), f64(y), f64(gate), scale=f64(scale))
    slack = lo.residual_norm_backward(f64(x_out), b, 2, None, f64(dh.abs()), f64(y), f64(gate), scale=f64(scale))
    for t, k in ((x, "dx"), (gate, "dgate"), (scale, "dscale"), (shift, "dshift"), (y, "dy")):
        # dh may round the other way where its float32 value lies next to a midpoint: a step of bf16 on it
        tol = 1024 * U * ref["size_" + k] + 2.0 ** -7 * slack["size_" + k] * 0.02 + (2.0 ** -8 * np.abs(ref[k]) if k == "dy" else 0)
        assert (np.abs(f64(t.grad) - ref[k]) <= tol).all(), k


def test_a_training_step_captured_and_replayed():
    """Forward and backward of the operators together in one graph: replays give the eager step's bits,
    for the inputs that are in the buffers then."""
    rows, heads, hd, pairs = 96, 4, 64, [12, 20]
    cols = heads * hd
    g = torch.Generator().manual_seed(5)
    rn = lambda *s: torch.randn(*s, generator=g).to(device())  # noqa: E731
    x, y, c = rn(rows, cols), rn(rows, cols).bfloat16(), rn(rows, heads, hd).bfloat16()
    gate, scale, shift = (0.5 * rn(3, cols) for _ in range(3))
    w, w_post = 1 + 0.1 * rn(cols), 1 + 0.1 * rn(cols)
    offsets = torch.tensor([0, 30, 30, 90], dtype=torch.int32, device=device())
    pos = torch.randint(0, 64, (rows, 2), generator=g).int().to(device())
    freqs = ep.rope_frequencies(pairs, device=device())

    def step():
        leaves = [t.detach().requires_grad_(True) for t in (x, y, gate, scale, shift, w, w_post)]
        x_out, h = ep.ResidualNorm.apply(*leaves, "layer", True, 1.0, 1e-6, offsets)
        r = ep.RopeAxes.apply(h.view(rows, heads, hd), pos, freqs, pairs)
        return [x_out.detach(), r.detach()] + list(torch.autograd.grad([x_out, r], leaves, [x.detach(), c]))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (6, 7):
        g.manual_seed(seed)
        x.copy_(rn(rows, cols)), y.copy_(rn(rows, cols)), scale.copy_(rn(3, cols))
        want = step()
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert ep.read_device_status() == 0


def test_offsets_past_32_bits():
    """Rows 2^31 elements apart: every operator's addresses in 64 bits."""
    pitch = 2 ** 31
    big = torch.empty(2 * pitch + 4096, dtype=torch.bfloat16, device=device())
    cols = 1024
    view = big.as_strided((3, cols), (pitch, 1))
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, cols, generator=g).bfloat16().to(device())
    view.copy_(x)
    h, h2 = torch.empty_like(x), torch.empty_like(x)
    ep.residual_norm(view, h)
    ep.residual_norm(x, h2)
    assert torch.equal(h, h2)
    stats = torch.empty(3, 4, device=device())
    ep.residual_norm(view, h, stats=stats)
    dx, dx2 = torch.empty_like(x), torch.empty_like(x)
    ep.residual_norm_backward(view, stats, dh=h, dx=dx)
    ep.residual_norm_backward(x, stats, dh=h, dx=dx2)
    assert torch.equal(dx, dx2)
    pairs = [64]
    pos, freqs = torch.arange(3, dtype=torch.int32, device=device())[:, None], ep.rope_frequencies(pairs, device=device())
    heads = big.as_strided((3, 8, 128), (pitch, 128, 1))
    assert torch.equal(ep.rope_axes(heads, pos, freqs, pairs), ep.rope_axes(x.view(3, 8, 128), pos, freqs, pairs))
    W = quantize_gpu(wk.weights(256, cols, 1 / 32, seed=1))
    d, d2 = torch.empty(3, 256, dtype=torch.bfloat16, device=device()), big.as_strided((3, 256), (pitch, 1), 2048)
    ep.gemv_nvfp4(view, W, d)
    ep.gemv_nvfp4(x, W, d2)
    assert torch.equal(d, d2)
    del big, view, heads, d2
    torch.cuda.empty_cache()


def test_a_weight_of_more_than_2_to_the_32_bytes():
    """A vocabulary-sized weight: 2^18 + 65 rows of 32768 (4.3 GB of codes); the last rows' products
    are those of a small weight made of them."""
    N, K = 2 ** 18 + 65, 32768
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=device())
    sf = torch.randint(0x20, 0x40, (ep.sf_bytes(N, K),), dtype=torch.uint8, device=device())
    B = ep.NVFP4Tensor(codes, sf, torch.full((1,), 1e-4, device=device()), N, K)
    x = torch.randn(2, K, device=device()).bfloat16()
    D = torch.empty(2, N, device=device())
    ep.gemv_nvfp4(x, B, D)
    first = N // 128 * 128  # the last row tile, whole
    tail = ep.NVFP4Tensor(codes[first:].contiguous(), sf[first // 128 * (K // 64) * 512:].contiguous(), B.gscale, N - first, K)
    E = torch.empty(2, N - first, device=device())
    ep.gemv_nvfp4(x, tail, E)
    # another split of K among warps and CTAs: float32 sums in another order
    size = x.abs().float().sum(1, keepdim=True) * 6 * 0.25 * 1e-4  # E4M3 codes below 0x40 are below 2
    assert bool(((D[:, first:] - E).abs() <= 8 * size * (K / 128 + 48) * 2.0 ** -24).all())
    assert bool(torch.isfinite(D).all()) and float(D[:, first:].std()) > 0
    del codes, sf, B, D
    torch.cuda.empty_cache()


def test_two_calls_at_once():
    """The same inputs on two streams at once, each with its own outputs and workspace."""
    g = torch.Generator().manual_seed(2)
    rows, cols = 2000, 1024
    x, y = (torch.randn(rows, cols, generator=g).bfloat16().to(device()) for _ in range(2))
    gate = torch.randn(1, cols, generator=g).bfloat16().to(device())
    w = torch.ones(cols, device=device())
    W = quantize_gpu(wk.weights(2048, cols, 1 / 32, seed=1))
    pairs = [32, 32]
    pos, freqs = torch.randint(0, 99, (rows, 2), generator=g).int().to(device()), ep.rope_frequencies(pairs, device=device())

    def buffers():
        z = lambda *s, **k: torch.zeros(*s, device=device(), **k)  # noqa: E731
        bf = dict(dtype=torch.bfloat16)
        return dict(xo=z(rows, cols, **bf), h=z(rows, cols, **bf), st=z(rows, 4), dx=z(rows, cols, **bf), dg=z(1, cols),
                    dw=z(cols), D=z(4, 2048), r=z(rows, 8, 128, **bf),
                    ws=torch.empty(ep.residual_norm_workspace_bytes(rows, cols, 1), dtype=torch.uint8, device=device()))

    def run(b, stream=None):
        for _ in range(10):
            ep.residual_norm(x, b["h"], y=y, x_out=b["xo"], gate=gate, w=w, stats=b["st"], stream=stream)
            ep.residual_norm_backward(b["xo"], b["st"], dx_out=x, dh=b["h"], y=y, gate=gate, w=w, dx=b["dx"], dgate=b["dg"],
                                      dw=b["dw"], workspace=b["ws"], stream=stream)
            ep.gemv_nvfp4(x[:4], W, b["D"], silu=True, stream=stream)
            ep.rope_axes(b["h"].view(rows, 8, 128), pos, freqs, pairs, b["r"], stream=stream)

    one, two, three = buffers(), buffers(), buffers()
    run(one)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    run(two, s)
    run(three, t)
    torch.cuda.synchronize()
    for k in one:
        if k != "ws":
            assert torch.equal(one[k], two[k]) and torch.equal(one[k], three[k]), k
    assert ep.read_device_status() == 0
