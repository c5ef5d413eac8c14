"""Layouts that the operators between the GEMMs are given in real programs: views that start between 16-byte
boundaries, single rows of wider buffers. What needs no GPU is tested on the CPU."""
import pytest
import torch

import epilogues_nvfp4_quantize_b200 as ep
from epilogues_nvfp4_quantize_b200 import _lib
from gpu_util import device

BF = torch.bfloat16


def at_offset(t, n):
    """A contiguous copy of t that starts n elements into its buffer."""
    buf = torch.empty(t.numel() + n, dtype=t.dtype, device=t.device)
    out = buf[n:].view(t.shape)
    out.copy_(t)
    assert out.is_contiguous() and out.data_ptr() % 16 == n * t.element_size() % 16
    return out


# ---- views that start between 16-byte boundaries ------------------------------------------
def test_a_contiguous_view_off_a_16_byte_boundary_is_copied():
    t = at_offset(torch.arange(512, dtype=torch.float32).to(BF).view(8, 64), 1)
    got = _lib._rows_of_16_bytes(t)
    assert got.data_ptr() % 16 == 0 and got.is_contiguous() and torch.equal(got, t)
    one = at_offset(torch.arange(64, dtype=torch.float32).view(1, 64), 1)
    got = _lib._rows_of_16_bytes(one)
    assert got.data_ptr() % 16 == 0 and torch.equal(got, one)
    heads = at_offset(torch.arange(512, dtype=torch.float32).view(4, 2, 64), 3)
    got = _lib._aligned(heads)
    assert got.data_ptr() % 16 == 0 and torch.equal(got, heads)
    w = at_offset(torch.arange(64, dtype=torch.float32), 1)
    got = _lib._aligned(w)
    assert got.data_ptr() % 16 == 0 and torch.equal(got, w)


def test_what_can_be_read_as_it_is_is_not_copied():
    t = torch.zeros(8, 80, dtype=BF)
    for v in (t, t[:, :64], t[:1, 8:72], t[::2]):
        assert _lib._rows_of_16_bytes(v) is v
    h = torch.zeros(4, 3, 64, dtype=BF)
    for v in (h, h[:, :2], h.transpose(0, 1), h[:, :1].expand(4, 3, 64)):
        assert _lib._aligned(v) is v
    for v in (t[:, ::2], t[:1].expand(8, 80), t[:, 1:65], torch.zeros(8, 68, dtype=BF)[:, :64]):
        got = _lib._rows_of_16_bytes(v)
        assert got is not v and got.is_contiguous() and got.data_ptr() % 16 == 0 and torch.equal(got, v)


@pytest.mark.gpu
@pytest.mark.parametrize("stream", [BF, torch.float32])
def test_residual_norm_gradients_off_a_16_byte_boundary(stream):
    """The gradient that torch.cat hands back starts wherever its part did."""
    rows, cols, B = 24, 128, 2
    g = torch.Generator().manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=g).to(device())  # noqa: E731
    base = dict(x=rn(rows, cols).to(stream), y=rn(rows, cols).to(BF), gate=rn(B, cols), scale=rn(B, cols), shift=rn(B, cols),
                w=rn(cols), w_post=rn(cols))
    cx, ch = rn(rows * cols).to(stream), rn(rows * cols).to(BF)

    def run(shifted):
        leaves = [t.clone().requires_grad_(True) for t in base.values()]
        # as inputs, views at odd offsets; the gradients come back through cat
        given = [torch.cat([t.new_zeros(1), t.flatten()])[1:].view(t.shape) for t in leaves] if shifted else leaves
        x_out, h = ep.ResidualNorm.apply(*given, "layer", True)
        if shifted:
            assert any(t.data_ptr() % 16 for t in given)
            flat = [torch.cat([t.new_zeros(1), t.flatten()])[1:] for t in (x_out, h)]
        else:
            flat = [x_out.flatten(), h.flatten()]
        grads = torch.autograd.grad(flat, leaves, [cx, ch])
        return [x_out.detach(), h.detach(), *grads]

    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, torch.float16, torch.float32])
def test_rope_gradient_off_a_16_byte_boundary(dtype):
    rows, heads, hd, pairs = 20, 3, 64, [12, 20]
    g = torch.Generator().manual_seed(2)
    x = torch.randn(rows, heads, hd, generator=g).to(dtype).to(device())
    c = torch.randn(rows * heads * hd, generator=g).to(dtype).to(device())
    pos = torch.randint(0, 50, (rows, 2), generator=g).int().to(device())
    freqs = ep.rope_frequencies(pairs, device=device())

    def run(shifted):
        leaf = x.clone().requires_grad_(True)
        given = torch.cat([leaf.new_zeros(1), leaf.flatten()])[1:].view(x.shape) if shifted else leaf
        r = ep.RopeAxes.apply(given, pos, freqs, pairs)
        flat = torch.cat([r.new_zeros(1), r.flatten()])[1:] if shifted else r.flatten()
        return r.detach(), torch.autograd.grad(flat, leaf, c)[0]

    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)


# ---- single rows of buffers with any pitch --------------------------------------------------
def one_row(t, pitch):
    """The values of t (1 x n) as a row of a buffer whose rows are `pitch` elements apart."""
    return torch.empty_strided(t.shape, (pitch, 1), dtype=t.dtype, device=t.device).copy_(t)


def test_one_row_has_no_pitch():
    for dtype in (BF, torch.float32):
        t = one_row(torch.zeros(1, 64, dtype=dtype), 101)
        assert t.stride() == (101, 1)
        assert _lib._matrix(t, "t", (1, 64), dtype) == (t.data_ptr(), 64)
        packed, _ = _lib._norm_inputs(t, None, None, t, t, None, None, "layer", False, 1.0, 1e-6, None, None)
        fields = _lib._NORM_INPUTS.unpack(packed)
        assert fields[:3] == (1, 64, 1) and [v for v in fields if v == 101] == []
    two = torch.zeros(2, 72, dtype=BF)[:, :64]
    assert _lib._matrix(two, "t", (2, 64), BF)[1] == 72


@pytest.mark.gpu
def test_operators_on_one_row_of_an_odd_pitch():
    K, N, cols = 256, 200, 512
    g = torch.Generator().manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    W = ep.nvfp4_quantize((rn(N, K) / 16).to(BF).to(device()), ep.NVFP4Tensor.empty(N, K, device()))
    x = rn(1, K).to(BF).to(device())
    D, E = torch.zeros(1, N, dtype=BF, device=device()), one_row(torch.zeros(1, N, dtype=BF, device=device()), N + 1)
    ep.gemv_nvfp4(x, W, D)
    ep.gemv_nvfp4(one_row(x, K + 5), W, E)
    assert torch.equal(D, E)

    s = rn(1, cols).to(BF).to(device())
    y, dxo, dh, gate, scale, shift = (rn(1, cols).to(BF).to(device()) for _ in range(6))

    def run(lay):
        new = lambda dtype=BF: lay(torch.zeros(1, cols, dtype=dtype, device=device()))  # noqa: E731
        a = {k: lay(v) for k, v in dict(y=y, gate=gate, scale=scale).items()}
        xo, h, stats = new(), new(), torch.zeros(1, 4, device=device())
        ep.residual_norm(lay(s), h, x_out=xo, shift=lay(shift), stats=stats, **a)
        d = dict(dx=new(), dy=new(), dgate=new(torch.float32), dscale=new(torch.float32), dshift=new(torch.float32))
        ep.residual_norm_backward(xo, stats, dx_out=lay(dxo), dh=lay(dh), **a, **d)
        return [xo, h, stats, *d.values()]

    for a, b in zip(run(lambda t: one_row(t, cols + 3)), run(lambda t: t)):
        assert torch.equal(a, b)


# ---- buffers that hold less memory than they have values --------------------------------------
def test_buffers_of_repeated_or_scattered_values_are_refused(monkeypatch):
    u8 = torch.uint8
    codes, sf, G = torch.zeros(8, 32, dtype=u8), torch.zeros(512, dtype=u8), torch.ones(1)
    assert _lib._nvfp4(_lib.NVFP4Tensor(codes, sf, G, 8, 64)).rows == 8
    for bad in ((codes[:1].expand(8, 32), sf, G), (torch.zeros(8, 64, dtype=u8)[:, :32], sf, G),
                (codes, sf[:1].expand(512), G), (codes, torch.zeros(1024, dtype=u8)[::2], G)):
        with pytest.raises(ValueError, match="contiguous"):
            _lib._nvfp4(_lib.NVFP4Tensor(*bad, 8, 64))
    with pytest.raises(ValueError, match="float32"):
        _lib._nvfp4(_lib.NVFP4Tensor(codes, sf, G.double(), 8, 64))

    need = ep.residual_norm_workspace_bytes(4, 64, 1)
    x, stats, dw = torch.zeros(4, 64), torch.zeros(4, 4), torch.zeros(64)
    monkeypatch.setattr(_lib, "_same_device", lambda *t: 0)
    monkeypatch.setattr(_lib, "_call", lambda *a: None)
    call = lambda ws: ep.residual_norm_backward(x, stats, dx_out=x, dh=x.to(BF), dw=dw, workspace=ws)  # noqa: E731
    call(torch.empty(need, dtype=u8))
    for bad in (torch.empty(need - 1, dtype=u8), torch.empty(1, dtype=u8).expand(need), torch.empty(2 * need, dtype=u8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            call(bad)

    need = ep.quantize_workspace_bytes()
    for bad in (torch.empty(1, dtype=u8).expand(need), torch.empty(2 * need, dtype=u8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            _lib._workspace(bad, True, "cpu")


# ---- rope_axes' own result in a graph -------------------------------------------------------
def test_a_new_result_of_rope_axes_carries_its_gradient(monkeypatch):
    calls = []
    monkeypatch.setattr(_lib, "_same_device", lambda *t: 0)
    monkeypatch.setattr(_lib, "_call", lambda *a: calls.append(a))
    x, pos = torch.zeros(4, 2, 32), torch.zeros(4, 1, dtype=torch.int32)
    freqs = ep.rope_frequencies([16], device="cpu")
    assert not ep.rope_axes(x, pos, freqs, [16]).requires_grad
    x.requires_grad_(True)
    for inverse in (False, True):
        r = ep.rope_axes(x, pos, freqs, [16], interleaved=False, inverse=inverse)
        assert r.requires_grad
        r.backward(torch.ones_like(r))
        forward, backward = calls[-2:]
        assert forward[17:19] == (False, inverse) and backward[17:19] == (False, not inverse)
    with torch.no_grad():
        assert not ep.rope_axes(x, pos, freqs, [16]).requires_grad
    y = torch.zeros(4, 2, 32)
    assert ep.rope_axes(x, pos, freqs, [16], y) is y and not y.requires_grad  # written to, no graph


@pytest.mark.gpu
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("stream", ["current", "object", "handle"])
def test_gradient_through_a_new_result_of_rope_axes(inverse, stream):
    rows, heads, hd, pairs = 33, 2, 64, [12, 16]
    g = torch.Generator().manual_seed(4)
    x, c = (torch.randn(rows, heads, hd, generator=g).to(device()) for _ in range(2))
    pos = torch.randint(0, 90, (rows, 2), generator=g).int().to(device())
    freqs = ep.rope_frequencies(pairs, device=device())
    want = ep.rope_axes(x, pos, freqs, pairs, torch.empty_like(x), inverse=inverse)
    dx = ep.rope_axes(c, pos, freqs, pairs, torch.empty_like(c), inverse=not inverse)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    leaf = x.clone().requires_grad_(True)
    torch.cuda.synchronize()
    r = ep.rope_axes(leaf, pos, freqs, pairs, inverse=inverse,
                     stream=dict(current=None, object=s, handle=s.cuda_stream)[stream])
    torch.cuda.synchronize()
    r.backward(c)
    torch.cuda.synchronize()
    assert torch.equal(r.detach(), want) and torch.equal(leaf.grad, dx)


# ---- a call without anything to compute -----------------------------------------------------
def test_residual_norm_without_a_branch_and_a_norm_is_refused(monkeypatch):
    monkeypatch.setattr(_lib, "_same_device", lambda *t: 0)
    monkeypatch.setattr(_lib, "_call", lambda *a: None)
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="branch"):
        ep.ResidualNorm.apply(x, None, None, None, None, None, None, None)
    assert ep.ResidualNorm.apply(x, x.to(BF), None, None, None, None, None, None).shape == (4, 64)
    assert ep.ResidualNorm.apply(x).shape == (4, 64)
