"""residual_norm and its gradient on the GPU against the float64 form (oracle/layer_ops.py).

Tolerances, u = 2^-24 (half a step of float32) and H half a step of the output's type
(finfo.eps / 2). A row's sum goes through at most 64 additions one after another (16 to 32 values per
thread, 5 + 5 levels of shuffles), so a mean of magnitudes is off by at most 64 u of it and a mean of
squares by 64 u relative; rsqrt and the products around it add a few u: a reciprocal root is off by
at most 40 u relative (half of the sum's 64, plus 8).
- x': alpha x + gate y~ with y~ = y rstd_y w_post: 48 u (|alpha x| + |gate y~|), then H.
- h, from the stored x': n is off by 40 u |n| + rstd (64 u mean|x'| + 2 u |x'|); the modulation adds
  4 u of each of its terms; then H.
- Gradients: with xhat, rstd off as above, T is off by at most 256 u of the sum of its terms'
  magnitudes (the forms' "size"), plus what xhat's own error does where a mean is large; dy likewise,
  512 u with the branch's norm on top. Sums over a sequence's rows add the rows of a piece one after
  another (at most rows / 64 + 1 here) and at most 256 pieces in eights: (rows / 64 + 300) u on top."""
import numpy as np
import pytest
import torch

import epilogues_nvfp4_quantize_b200 as ep
from oracle import layer_ops as lo
from gpu_util import device, read_nvfp4, quantize_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def half(t):
    return torch.finfo(t.dtype).eps / 2


def within(got, ref, err, h, what):
    tol = err + h * (np.abs(ref) + err) + 1e-38
    d = np.abs(f64(got) - ref)
    over = ~(d <= tol)
    assert not over.any(), f"{what}: {int(over.sum())} of {over.size} over, worst {np.nanmax(d / tol):.3g} of the tolerance"


def make(rows, cols, B, stream="bf16", mod="bf16", offsets=None, branch=True, post=False, norm="layer", w=False,
         mods=("gate", "scale", "shift"), seed=0, mean=0.3, alpha=1.0):
    g = torch.Generator().manual_seed(seed + rows + cols)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = device()
    wide = rn(rows, cols + 16) * 2 + mean  # the stream is a slice of wider rows
    m = (rn(B, 3 * cols) * 0.5).to(TYPES[mod]).to(d)
    a = dict(y=(rn(rows, cols) * 1.5).bfloat16().to(d) if branch else None, residual_scale=alpha, norm=norm,
             post_norm=post, w=(1 + 0.2 * rn(cols)).to(d) if w else None,
             w_post=(1 + 0.2 * rn(cols)).to(d) if post and w else None,
             offsets=None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=d))
    for i, name in enumerate(("shift", "scale", "gate")):
        a[name] = m[:, i * cols:(i + 1) * cols] if name in mods else None
    if not branch:
        a["gate"] = None
    if norm is None:
        a["scale"] = a["shift"] = a["w"] = None
    return wide.to(TYPES[stream]).to(d)[:, 8:cols + 8], a, lo.sequences(rows, B, offsets)


def check_forward(x, a, b, hq=False):
    rows, cols = x.shape
    B = len(set(b[b >= 0])) if a["offsets"] is None else a["offsets"].numel() - 1
    x_out = torch.full((rows, cols + 8), 3.0, dtype=x.dtype, device=device())[:, :cols]
    h = torch.full((rows, cols), 5.0, dtype=torch.bfloat16, device=device()) if a["norm"] else None
    stats = torch.full((rows, 4), -1.0, device=device())
    q = None
    if hq:
        q = ep.NVFP4Tensor.empty(rows, cols, device())
        q.codes.fill_(0xAB), q.sf.fill_(0xCD), q.gscale.fill_(0.003)
    ep.residual_norm(x, h, q, x_out=x_out, stats=stats, batches=None if a["offsets"] is not None else B, **a)
    torch.cuda.synchronize()
    live = b >= 0
    p = {k: f64(a[k]) for k in ("y", "gate", "w", "w_post", "scale", "shift")}
    if p["y"] is None:
        assert torch.equal(x_out[live], x[live])
    else:
        ref = lo.residual(f64(x), p["y"], b, p["gate"], a["post_norm"], p["w_post"], a["residual_scale"])
        size = np.abs(a["residual_scale"] * f64(x)) + np.abs(
            (1.0 if p["gate"] is None else p["gate"][np.maximum(b, 0)]) * lo.branch(p["y"], a["post_norm"], p["w_post"]))
        within(x_out[live], ref[live], 48 * U * size[live], half(x), "x_out")
    if (~live).any():
        assert bool((x_out[~live] == 3.0).all()) and bool((stats[~live] == -1.0).all())
        assert h is None or bool((h[~live] == 5.0).all())
    z = f64(x_out)
    if h is None:
        return x_out, stats
    n = lo.modulated_norm(z, b, a["norm"], p["w"])
    ref = lo.modulated_norm(z, b, a["norm"], p["w"], p["scale"], p["shift"])
    mean, rstd = lo.stats(z, a["norm"])
    wv = 1.0 if p["w"] is None else np.abs(p["w"])
    one = 1.0 + (0.0 if p["scale"] is None else p["scale"][np.maximum(b, 0)])
    sh = 0.0 if p["shift"] is None else np.abs(p["shift"][np.maximum(b, 0)])
    e_n = 40 * U * np.abs(n) + wv * rstd * (64 * U * np.abs(z).mean(1, keepdims=True) + 2 * U * np.abs(z))
    err = e_n * np.abs(one) + 4 * U * (np.abs(n) * (1 + np.abs(one - 1)) + sh) + 0 * z
    within(h[live], ref[live], err[live], half(h), "h")
    within(stats[live][:, 1:2], rstd[live],
           (40 * U * rstd + rstd ** 2 * 64 * U * np.abs(z).mean(1, keepdims=True))[live], 0, "rstd")
    if q is not None:
        # the codes and scales are those of nvfp4_quantize on the bf16 output, rows without a
        # sequence untouched, padding scales 0
        codes, scales, G, buf = read_nvfp4(q)
        ref_q = quantize_gpu(h.cpu(), G=G)
        rc, rs, _, rbuf = read_nvfp4(ref_q)
        assert np.array_equal(codes[live], rc[live]) and np.array_equal(scales[live], rs[live])
        if (~live).any():
            assert (q.codes.cpu().numpy()[~live] == 0xAB).all()
            assert (scales[~live] == 0xCD).all()
        elif rows % 128:
            assert np.array_equal(buf, rbuf)
    return x_out, stats


CASES = [
    # rows, cols, sequences, options
    (1, 8, 1, dict()),
    (5, 64, 1, dict(norm="rms", w=True)),
    (130, 256, 2, dict(post=True, w=True, norm="rms", alpha=0.8)),
    (33, 264, 3, dict(stream="f32", mod="f32", post=True)),
    (64, 1024, 4, dict(mod="f32", branch=False)),
    (9, 1032, 1, dict(mods=("gate",))),
    (12, 2568, 4, dict(stream="f32", w=True, norm="rms", mods=("shift",))),
    (7, 4096, 7, dict(post=True, w=True)),
    (3, 5120, 1, dict(stream="f32", mods=())),
    (2, 16384, 1, dict(post=True, w=True, norm="rms")),
    (6, 8200, 2, dict(stream="f32", mod="f32")),
    (20, 512, 1, dict(norm=None, post=True, w=True, alpha=0.5)),
    (50, 320, 5, dict(offsets=[0, 10, 10, 31, 44, 47], w=True)),
    (40, 1088, 3, dict(offsets=[2, 2, 20, 39], stream="f32", post=True)),
    (16, 128, 2, dict(offsets=[0, 0, 0])),  # no row has a sequence
]


@pytest.mark.parametrize("rows,cols,B,opt", CASES)
def test_forward(rows, cols, B, opt):
    x, a, b = make(rows, cols, B, **opt)
    check_forward(x, a, b, hq=a["norm"] is not None and cols % 64 == 0)


# enough rows that a CTA walks several of them
MANY_ROWS = [
    (1000, 4096, 2, dict(post=True, w=True, alpha=0.8)),
    (913, 4096, 1, dict(stream="f32", mod="f32", norm="rms", w=True)),
    (4201, 1024, 1, dict(branch=False)),
    (7200, 64, 3, dict(post=True, mod="f32")),
    (7400, 8, 1, dict(mods=())),
    (1500, 2568, 4, dict(offsets=[0, 1, 1, 1100, 1490], stream="f32", post=True, w=True, norm="rms")),
    (2500, 2048, 3, dict(offsets=[3, 900, 2400, 2500], w=True)),
    (501, 8200, 1, dict(post=True)),
    (502, 16384, 2, dict(stream="f32", w=True)),
    (940, 4032, 2, dict(norm=None, post=True, w=True, alpha=0.5)),
    (940, 3968, 5, dict(norm=None)),
    (1600, 256, 1600, dict(post=True, w=True)),  # a modulation vector for each row
    (1600, 9000, 1600, dict(mod="f32")),
]


@pytest.mark.parametrize("rows,cols,B,opt", MANY_ROWS)
def test_forward_many_rows(rows, cols, B, opt):
    x, a, b = make(rows, cols, B, **opt)
    check_forward(x, a, b, hq=a["norm"] is not None and cols % 64 == 0)


@pytest.mark.parametrize("stream", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(300, 4096), (257, 1024), (128, 192)])
def test_forward_with_nvfp4_output(stream, rows, cols):
    x, a, b = make(rows, cols, 1, stream=stream, seed=9)
    check_forward(x, a, b, hq=True)


def test_large_mean_and_tiny_spread_keep_their_digits():
    """A mean 1000 times the spread: the centred second pass keeps rstd to the tolerance of the
    mean itself; a constant row has rstd eps^-1/2 and h = shift."""
    x, a, b = make(16, 2048, 1, stream="f32", mod="f32", branch=False, mean=2000.0)
    check_forward(x, a, b)
    h = torch.empty(16, 2048, dtype=torch.bfloat16, device=device())
    ep.residual_norm(torch.full((16, 2048), 4.0, device=device()), h, scale=a["scale"], shift=a["shift"])
    assert torch.equal(h, a["shift"].bfloat16().expand(16, -1))


def test_in_place_other_stream_and_graph():
    x, a, b = make(257, 1536, 1, post=True, w=True)
    h = torch.empty(257, 1536, dtype=torch.bfloat16, device=device())
    xo = torch.empty_like(h)
    ep.residual_norm(x, h, x_out=xo, **a)
    torch.cuda.synchronize()
    x2, h2 = x.clone(), torch.zeros_like(h)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ep.residual_norm(x2, h2, x_out=x2, stream=s, **a)
    s.synchronize()
    assert torch.equal(x2, xo) and torch.equal(h2, h)
    x3, h3 = x.clone(), torch.zeros_like(h)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.residual_norm(x3, h3, x_out=x3, **a)
    x3.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(x3, xo) and torch.equal(h3, h)


def grads(x_out, stats, a, b, B, dxo, dh, only=None):
    rows, cols = x_out.shape
    d = device()
    out = dict(dx=torch.full_like(x_out, 3.0, memory_format=torch.contiguous_format))
    if a["y"] is not None:
        out["dy"] = torch.full_like(a["y"], 3.0)
        out["dgate"] = torch.full((B, cols), 3.0, device=d)
        if a["post_norm"]:
            out["dw_post"] = torch.full((cols,), 3.0, device=d)
    if a["norm"]:
        out["dscale"], out["dshift"] = torch.full((2, B, cols), 3.0, device=d)
        out["dw"] = torch.full((cols,), 3.0, device=d)
    if only is not None:
        out = {k: v for k, v in out.items() if k in only}
    args = {k: v for k, v in a.items() if k not in ("shift",)}
    ep.residual_norm_backward(x_out, stats, dx_out=dxo, dh=dh, batches=None if a["offsets"] is not None else B, **args, **out)
    torch.cuda.synchronize()
    return out


def check_gradient(x_out, a, b, B, dxo, dh, got):
    p = {k: f64(a[k]) for k in ("y", "gate", "w", "w_post", "scale")}
    ref = lo.residual_norm_backward(f64(x_out), b, B, f64(dxo), f64(dh), p["y"], p["gate"], a["post_norm"],
                                    p["w_post"], a["residual_scale"], a["norm"], p["w"], p["scale"])
    live = b >= 0
    rows = x_out.shape[0]
    # dscale and dw: xhat = (x' - mean) rstd is off by rstd (64 u mean|x'| + 2 u |x'|) besides its 40 u |xhat|
    # (as h above), and a sum over rows by |dh w| or |dh (1 + scale)| times that; where a sequence has one
    # row and x' is next to its mean, that is more than any multiple of u |dh xhat|
    extra = {}
    if dh is not None:
        z = f64(x_out)[live]
        d = np.abs(f64(dh)[live]) * lo.stats(f64(x_out), a["norm"])[1][live] * (
            64 * U * np.abs(z).mean(1, keepdims=True) + 2 * U * np.abs(z))
        extra["dscale"] = np.zeros((B, z.shape[1]))
        np.add.at(extra["dscale"], b[live], d * (1.0 if p["w"] is None else np.abs(p["w"])))
        extra["dw"] = (d * (1.0 if p["scale"] is None else np.abs(1 + p["scale"][b[live]]))).sum(0)
    for k, t in got.items():
        if k in ("dx", "dy"):
            within(t[live], ref[k][live], (256 if k == "dx" else 512) * U * ref["size_" + k][live], half(t), k)
            assert bool((t[~live] == 3.0).all()), f"{k}: rows without a sequence"
        elif k in ref:
            within(t, ref[k], (512 + rows / 64 + 300) * U * ref["size_" + k] + extra.get(k, 0.0), U, k)
        else:  # no dh: the norm contributes nothing
            assert bool((t == 0).all()), k


GRAD_CASES = [c for c in CASES if c[1] <= 8200] + [
    (700, 640, 2, dict(post=True, w=True)),
    (1000, 96, 1, dict(stream="f32", mod="f32", norm="rms", w=True)),
    (3000, 72, 3, dict(offsets=[0, 1, 2900, 2950], post=True, w=True, stream="f32")),
    (64, 64, 64, dict(post=True, w=True)),  # a modulation vector for each row
    (3, 16384, 1, dict(post=True, w=True, norm="rms")),
    (2400, 256, 2400, dict(w=True, stream="f32")),
    (400, 5120, 4, dict(offsets=[1, 1, 200, 260, 390], post=True, w=True)),  # clusters that walk several rows
    (290, 8200, 2, dict(stream="f32", mod="f32", w=True)),
    (129, 16384, 3, dict(stream="f32", post=True, w=True, norm="rms")),
]


@pytest.mark.parametrize("rows,cols,B,opt", GRAD_CASES)
def test_gradient(rows, cols, B, opt):
    x, a, b = make(rows, cols, B, **opt)
    g = torch.Generator().manual_seed(7)
    dxo = torch.randn(rows, cols, generator=g).to(x.dtype).to(device())
    dh = torch.randn(rows, cols, generator=g).bfloat16().to(device()) if a["norm"] else None
    x_out = torch.zeros(rows, cols, dtype=x.dtype, device=device())
    stats = torch.zeros(rows, 4, device=device())
    nb = None if a["offsets"] is not None else B
    ep.residual_norm(x, torch.empty_like(x, dtype=torch.bfloat16, memory_format=torch.contiguous_format) if a["norm"] else None,
                     x_out=x_out, stats=stats, batches=nb, **a)
    got = grads(x_out, stats, a, b, B, dxo, dh)
    check_gradient(x_out, a, b, B, dxo, dh, got)
    again = grads(x_out, stats, a, b, B, dxo, dh)
    assert all(torch.equal(got[k], again[k]) for k in got), "the same inputs give the same bits"
    # either gradient alone, and a part of the outputs
    if dh is not None:
        part = grads(x_out, stats, a, b, B, None, dh, only=("dx", "dshift"))
        check_gradient(x_out, a, b, B, None, dh, part)
        if a["y"] is not None:
            part = grads(x_out, stats, a, b, B, dxo, None, only=("dy", "dgate", "dscale"))
            check_gradient(x_out, a, b, B, dxo, None, part)


@pytest.mark.parametrize("rows,cols", [(60, 256), (1500, 512), (200, 5120)])
def test_what_stands_in_rows_without_a_sequence_reaches_nothing(rows, cols):
    """NaN and infinities in the rows in front of the first and behind the last sequence: outputs and
    gradients are those of the same call with zeros there, the parameters' among them."""
    off = [3, rows // 2, rows // 2, rows - 7]
    x, a, b = make(rows, cols, 3, offsets=off, post=True, w=True)
    live = torch.from_numpy(b >= 0).to(device())[:, None]

    def run(fill):
        put = lambda t: torch.where(live, t, torch.full_like(t, fill))  # noqa: E731
        c = dict(a, y=put(a["y"]))
        g = torch.Generator().manual_seed(3)
        dxo, dh = (put(torch.randn(rows, cols, generator=g).bfloat16().to(device())) for _ in range(2))
        h = torch.full((rows, cols), 5.0, dtype=torch.bfloat16, device=device())
        xo, stats = put(torch.zeros_like(h)), put(torch.zeros(rows, 1, device=device())).expand(rows, 4).contiguous()
        ep.residual_norm(put(x), h, x_out=xo, stats=stats, **c)
        out = grads(xo, stats, c, b, 3, dxo, dh)
        return [t for k, t in out.items()] + [h, torch.where(live, xo, torch.zeros_like(xo))]

    want = run(0.0)
    for fill in (float("nan"), float("inf")):
        assert all(torch.equal(p, q) for p, q in zip(run(fill), want))
    assert all(bool(torch.isfinite(t).all()) for t in want)


def test_gradient_in_place():
    x, a, b = make(40, 512, 2, post=True, w=True)
    xo, stats = torch.empty(40, 512, dtype=x.dtype, device=device()), torch.empty(40, 4, device=device())
    ep.residual_norm(x, torch.empty_like(xo), x_out=xo, stats=stats, batches=2, **a)
    dxo, dh = torch.randn_like(xo), torch.randn_like(xo)
    want = grads(xo, stats, a, b, 2, dxo, dh, only=("dx", "dy"))
    args = {k: v for k, v in a.items() if k != "shift"}
    d1, d2 = dxo.clone(), dh.clone()
    ep.residual_norm_backward(xo, stats, dx_out=d1, dh=d2, dx=d1, dy=d2, batches=2, **args)
    assert torch.equal(d1, want["dx"]) and torch.equal(d2, want["dy"])


def test_autograd_function_against_the_form_and_broadcast_inputs():
    rows, cols, B = 48, 256, 3
    x, a, b = make(rows, cols, B, stream="f32", mod="f32", post=True, w=True)
    leaf = lambda t: t.detach().clone().requires_grad_(True)  # noqa: E731
    xs, y, w, wp = leaf(x), leaf(a["y"]), leaf(a["w"]), leaf(a["w_post"])
    gate = leaf(a["gate"][:1])  # one gate for all sequences
    scale, shift = leaf(a["scale"]), leaf(a["shift"])
    x_out, h = ep.ResidualNorm.apply(xs, y, gate.expand(B, cols), scale, shift, w, wp, "layer", True, 0.7)
    cx, ch = torch.randn(rows, 1, device=device()), torch.randn(rows, cols, device=device()).bfloat16()
    (x_out * cx).sum().add((h.float() * ch.float()).sum()).backward()
    ref = lo.residual_norm_backward(f64(x_out), b, B, np.broadcast_to(f64(cx), (rows, cols)), f64(ch), f64(y),
                                    np.broadcast_to(f64(gate), (B, cols)), True, f64(wp), 0.7, "layer", f64(w), f64(scale))
    within(xs.grad, ref["dx"], 256 * U * ref["size_dx"], U, "dx")
    within(y.grad, ref["dy"], 512 * U * ref["size_dy"], half(y), "dy")
    within(gate.grad, ref["dgate"].sum(0, keepdims=True), 820 * U * ref["size_dgate"].sum(0, keepdims=True), U, "dgate")
    for t, k in ((scale, "dscale"), (shift, "dshift"), (w, "dw"), (wp, "dw_post")):
        within(t.grad, ref[k], 820 * U * ref["size_" + k], U, k)


@pytest.mark.parametrize("which", ["no branch", "no norm", "only h used", "only x_out used"])
def test_autograd_function_parts(which):
    rows, cols = 10, 128
    x, a, b = make(rows, cols, 1, stream="f32", mod="f32", branch=which != "no branch")
    leaf = lambda t: None if t is None else t.detach().clone().requires_grad_(True)  # noqa: E731
    xs, y, gate, scale, shift = (leaf(t) for t in (x, a["y"], a["gate"], a["scale"], a["shift"]))
    norm = None if which == "no norm" else "layer"
    if norm is None:
        scale = shift = None
    out = ep.ResidualNorm.apply(xs, y, gate, scale, shift, None, None, norm)
    c = torch.randn(rows, cols, device=device()).bfloat16()
    x_out, h = out if isinstance(out, tuple) else (None, out) if which == "no branch" else (out, None)
    use_x, use_h = which in ("no norm", "only x_out used"), which in ("no branch", "only h used")
    ((x_out if use_x else h).float() * c.float()).sum().backward()
    z = f64(xs) if x_out is None else f64(x_out)
    ref = lo.residual_norm_backward(z, b, 1, f64(c) if use_x else None, f64(c) if use_h else None, f64(y), f64(gate),
                                    norm=norm, scale=f64(scale))
    within(xs.grad, ref["dx"], 256 * U * ref["size_dx"], U, "dx")
    if y is not None:
        within(y.grad, ref["dy"], 512 * U * ref["size_dy"], half(y), "dy")
    if use_h:
        within(shift.grad, ref["dshift"], 820 * U * ref["size_dshift"], U, "dshift")
    elif norm is not None:
        assert bool((shift.grad == 0).all())


def test_a_workspace_belongs_to_the_stream_of_its_call(monkeypatch):
    x, a, b = make(100, 512, 2, post=True, w=True)
    xo, stats = torch.empty(100, 512, dtype=x.dtype, device=device()), torch.empty(100, 4, device=device())
    ep.residual_norm(x, torch.empty_like(xo), x_out=xo, stats=stats, batches=2, **a)
    dh = torch.randn_like(xo)
    want = torch.empty(2, 512, device=device())
    args = {k: v for k, v in a.items() if k != "shift"}
    ep.residual_norm_backward(xo, stats, dh=dh, batches=2, dgate=want, **args)
    torch.cuda.synchronize()
    made_on, empty = [], torch.empty

    def spy(*p, **k):
        made_on.append(torch.cuda.current_stream().cuda_stream)
        return empty(*p, **k)

    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):  # an object, and a plain handle
        got = torch.zeros_like(want)
        torch.cuda.synchronize()
        monkeypatch.setattr(torch, "empty", spy)
        ep.residual_norm_backward(xo, stats, dh=dh, batches=2, dgate=got, stream=stream, **args)
        monkeypatch.undo()
        s.synchronize()
        assert torch.equal(got, want)
    assert made_on == [s.cuda_stream] * 2
    assert torch.cuda.current_stream().cuda_stream != s.cuda_stream


def test_gradient_from_a_graph():
    x, a, b = make(100, 512, 2, post=True, w=True)
    xo, stats = torch.empty(100, 512, dtype=x.dtype, device=device()), torch.empty(100, 4, device=device())
    ep.residual_norm(x, torch.empty_like(xo), x_out=xo, stats=stats, batches=2, **a)
    dxo, dh = torch.randn_like(xo), torch.randn_like(xo)
    want = grads(xo, stats, a, b, 2, dxo, dh)
    out = {k: torch.zeros_like(v) for k, v in want.items()}
    ws = torch.empty(ep.residual_norm_workspace_bytes(100, 512, 2), dtype=torch.uint8, device=device())
    args = {k: v for k, v in a.items() if k != "shift"}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.residual_norm_backward(xo, stats, dx_out=dxo, dh=dh, batches=2, workspace=ws, **args, **out)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[k], want[k]) for k in want)
    with pytest.raises(ValueError, match="workspace"):
        ep.residual_norm_backward(xo, stats, dx_out=dxo, dh=dh, batches=2, workspace=ws[:-4], **args, **out)
    assert ep.read_device_status() == 0
