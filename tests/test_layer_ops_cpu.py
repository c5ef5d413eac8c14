"""The float64 forms of the operators between a layer's GEMMs (oracle/layer_ops.py) against
independent statements and finite differences, and the operators' argument checks (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import epilogues_nvfp4_quantize_b200 as ep
from epilogues_nvfp4_quantize_b200 import _lib
from oracle import layer_ops as lo
from oracle import nvfp4_oracle as o

INVALID, SHAPE, MISALIGNED = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from epilogues_nvfp4_quantize_b200.build import build
    build()
    return ep.load()


# ---- the float64 forms -----------------------------------------------------------------
def test_gemv_form_against_loops():
    r = np.random.default_rng(0)
    codes, scales = r.integers(0, 16, (5, 64)), r.integers(1, 0x7F, (5, 4))
    x, bias = r.standard_normal((3, 64)), r.standard_normal(5)
    levels = [0, .5, 1, 1.5, 2, 3, 4, 6]
    ref = np.zeros((3, 5))
    for m in range(3):
        for n in range(5):
            for k in range(64):
                c = int(codes[n, k])
                s = torch.tensor([int(scales[n, k // 16])], dtype=torch.uint8).view(torch.float8_e4m3fn).double().item()
                v = x[m, k] / (1 + np.exp(-x[m, k]))
                ref[m, n] += v * levels[c & 7] * (-1 if c & 8 else 1) * s * 0.01
    got, _ = lo.gemv(x, codes.astype(np.uint8), scales.astype(np.uint8), 0.01, bias, silu=True)
    assert np.allclose(got, ref + bias, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("norm,post,ragged", [("layer", False, False), ("rms", True, True), ("layer", True, True),
                                              ("rms", False, False), (None, True, False)])
def test_norm_gradient_form_against_differences(norm, post, ragged):
    r = np.random.default_rng(1)
    rows, cols, B = 7, 8, 3 if ragged else 1
    off = [0, 3, 3, 5] if ragged else None
    b = lo.sequences(rows, B, off)
    p = dict(x=r.standard_normal((rows, cols)), y=r.standard_normal((rows, cols)), gate=r.standard_normal((B, cols)),
             scale=r.standard_normal((B, cols)), shift=r.standard_normal((B, cols)), w=1 + r.standard_normal(cols),
             w_post=1 + r.standard_normal(cols))
    gx, gh = r.standard_normal((rows, cols)), r.standard_normal((rows, cols))
    live = (b >= 0)[:, None]
    wp = lambda q: q["w_post"] if post else None  # noqa: E731

    def loss(q):
        z = lo.residual(q["x"], q["y"], b, q["gate"], post, wp(q), 0.7)
        v = gx * z
        if norm is not None:
            v = v + gh * lo.modulated_norm(z, b, norm, q["w"], q["scale"], q["shift"])
        return float((v * live).sum())

    z = lo.residual(p["x"], p["y"], b, p["gate"], post, wp(p), 0.7)
    g = lo.residual_norm_backward(z, b, B, gx, gh if norm else None, p["y"], p["gate"], post, wp(p), 0.7, norm,
                                  p["w"] if norm else None, p["scale"] if norm else None)
    names = ["x", "y", "gate"] + (["w_post"] if post else []) + (["scale", "shift", "w"] if norm else [])
    for name in names:
        for at in np.ndindex(p[name].shape):
            diff = []
            for step in (1e-5, -1e-5):
                q = dict(p, **{name: p[name].copy()})
                q[name][at] += step
                diff.append(loss(q))
            want = (diff[0] - diff[1]) / 2e-5
            got = g["d" + name][at]
            if name in ("x", "y") and b[at[0]] < 0:
                continue  # rows without a sequence are not part of the op
            assert abs(got - want) <= 1e-6 * max(1.0, abs(want)) * 10, (name, at, got, want)


def test_rope_form_keeps_lengths_and_inverts():
    r = np.random.default_rng(2)
    x = r.standard_normal((6, 2, 32))
    pos, pairs = r.integers(0, 1000, (6, 3)), [3, 5, 6]
    freqs = ep.rope_frequencies(pairs, device="cpu").numpy()
    for inter in (True, False):
        y = lo.rope(x, pos, freqs, pairs, inter)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        assert np.array_equal(y[..., 28:], x[..., 28:])
        assert np.allclose(lo.rope(y, pos, freqs, pairs, inter, inverse=True), x)
        # scores of a pair of rows depend on the difference of their positions only
        s0 = (lo.rope(x, pos, freqs, pairs, inter) * lo.rope(x[::-1], pos + 7, freqs, pairs, inter)).sum()
        s1 = (lo.rope(x, pos + 100, freqs, pairs, inter) * lo.rope(x[::-1], pos + 107, freqs, pairs, inter)).sum()
        assert abs(s0 - s1) < 1e-9
    # one pair by hand
    y = lo.rope(np.array([[[1.0, 2.0, 5.0, 6.0]]]), np.array([[2]]), np.array([0.3]), [1])
    c, s = np.cos(0.6), np.sin(0.6)
    assert np.allclose(y[0, 0], [c - 2 * s, s + 2 * c, 5, 6])


def test_rope_frequencies():
    f = ep.rope_frequencies([4, 2], 100.0, device="cpu")
    assert f.dtype == torch.float64
    assert np.allclose(f.numpy(), [1, 100 ** -.25, 100 ** -.5, 100 ** -.75, 1, 0.1])


# ---- argument checks of the C entry points ----------------------------------------------
def _t(rows=256, cols=128, codes=16, sf=16, g=16):
    return _lib._Tensor(codes, sf, g, rows, cols)


def test_gemv_argument_checks(lib):
    def call(x=16, xt=0, M=1, ldx=128, act=0, B=None, bias=None, ot=0, D=16, ldd=256):
        return lib.gemv_nvfp4(x, xt, M, ldx, act, B or _t(), bias, ot, D, ldd, None)

    assert call(x=None) == INVALID and call(D=None) == INVALID
    assert call(xt=2) == INVALID and call(xt=-1) == INVALID and call(ot=3) == INVALID
    assert call(act=1) == INVALID  # ReLU belongs to the pointwise epilogue
    assert call(B=_t(codes=0)) == INVALID
    assert call(M=0) == SHAPE and call(M=524281) == SHAPE and call(B=_t(rows=0)) == SHAPE and call(B=_t(cols=0)) == SHAPE
    assert call(B=_t(cols=96), ldx=96) == SHAPE and call(B=_t(cols=32768 + 64), ldx=40000) == SHAPE
    assert call(ldx=120) == INVALID and call(ldd=255) == INVALID
    assert call(x=24) == MISALIGNED and call(ldx=132) == MISALIGNED
    assert call(B=_t(codes=8)) == MISALIGNED and call(B=_t(sf=8)) == MISALIGNED and call(bias=18) == MISALIGNED
    assert call(D=17) == MISALIGNED and call(D=18, ot=2) == MISALIGNED


NORM_FIELDS = ("rows cols batches offsets stream_dtype mod_dtype norm post_norm residual_scale eps x ldx y ldy gate "
               "ldgate scale ldscale shift ldshift w_post w").split()
GRAD_FIELDS = "dx_out lddxo dh lddh dx lddx dy lddy dgate lddgate dscale lddscale dshift lddshift dw dw_post".split()


def _norm(**k):
    a = dict(rows=4, cols=64, batches=2, norm=1, residual_scale=1.0, eps=1e-6, x=16, ldx=64)
    a.update(k)
    assert set(a) <= set(NORM_FIELDS)
    return _lib._NORM_INPUTS.pack(*(a.get(f) or 0 for f in NORM_FIELDS))


def test_residual_norm_argument_checks(lib):
    def call(x_out=None, ldxo=64, h=16, ldh=64, hq=None, stats=None, **k):
        return lib.residual_norm(_norm(**k), x_out, ldxo, h, ldh, None if hq is None else ctypes.pointer(hq), stats,
                                 None)

    assert lib.residual_norm(None, None, 0, 16, 64, None, None, None) == INVALID
    assert call(x=None) == INVALID and call(h=None) == INVALID
    assert call(stream_dtype=1) == INVALID and call(mod_dtype=1) == INVALID and call(norm=3) == INVALID
    assert call(post_norm=2) == INVALID and call(eps=0.0) == INVALID and call(eps=float("inf")) == INVALID
    assert call(eps=float("nan")) == INVALID
    # parts of a branch without a branch, norm parameters without a norm
    assert call(gate=16, ldgate=64) == INVALID and call(residual_scale=0.5) == INVALID and call(post_norm=1) == INVALID
    assert call(y=16, ldy=64, w_post=16) == INVALID
    assert call(norm=0, x_out=16, h=None, scale=16, ldscale=64) == INVALID
    assert call(norm=0, x_out=16) == INVALID  # h without a norm
    assert call(rows=0) == SHAPE and call(cols=0) == SHAPE and call(cols=60, ldx=64) == SHAPE
    assert call(cols=16392, ldx=16392) == SHAPE and call(batches=0) == SHAPE and call(batches=3) == SHAPE
    assert call(ldx=56) == INVALID and call(ldh=56) == INVALID and call(x_out=32, ldxo=56) == INVALID
    assert call(x_out=16, ldxo=128) == INVALID  # in place with another pitch
    assert call(scale=16, ldscale=32) == INVALID
    assert call(x=24) == MISALIGNED and call(ldx=68) == MISALIGNED and call(h=24) == MISALIGNED
    assert call(scale=8, ldscale=64) == MISALIGNED and call(shift=16, ldshift=68) == MISALIGNED
    assert call(w=8) == MISALIGNED and call(stats=8) == MISALIGNED and call(offsets=2) == MISALIGNED
    assert call(hq=_t(4, 32)) == INVALID and call(hq=_t(4, 64, codes=8)) == MISALIGNED
    assert call(cols=72, ldx=72, ldh=72, hq=_t(4, 72)) == SHAPE  # NVFP4 output: cols % 64


def test_residual_norm_backward_argument_checks(lib):
    def call(stats=16, ws=16, i=None, **k):
        g = dict(dx_out=16, lddxo=64, dh=16, lddh=64, dx=16, lddx=64)
        g.update(k)
        assert set(g) <= set(GRAD_FIELDS)
        packed = _lib._NORM_GRADS.pack(*(g.get(f) or 0 for f in GRAD_FIELDS))
        return lib.residual_norm_backward(_norm(**(i or {})), stats, packed, ws, None)

    assert lib.residual_norm_backward(_norm(), 16, None, 16, None) == INVALID
    assert call(stats=None) == INVALID and call(dx_out=None, dh=None) == INVALID and call(dx=None) == INVALID
    assert call(i=dict(norm=0)) == INVALID  # dh without a norm
    assert call(dy=16, lddy=64) == INVALID and call(dgate=16, lddgate=64) == INVALID  # no branch
    assert call(dw_post=16, i=dict(y=16, ldy=64)) == INVALID
    assert call(dscale=16, lddscale=64, ws=None) == INVALID
    # in place with another pitch
    assert call(dx=16, lddx=128) == INVALID
    assert call(dx=None, dy=16, lddy=128, i=dict(y=32, ldy=64)) == INVALID
    assert call(dx=None, dy=32, lddy=128, i=dict(y=32, ldy=64)) == INVALID
    assert call(lddx=56) == INVALID and call(dshift=16, lddshift=56) == INVALID
    assert call(dx=24) == MISALIGNED and call(dh=24) == MISALIGNED and call(lddxo=68) == MISALIGNED
    assert call(ws=8, dscale=16, lddscale=64) == MISALIGNED and call(dw=18) == MISALIGNED
    assert lib.residual_norm_workspace_bytes(0, 64, 1) == -1
    assert lib.residual_norm_workspace_bytes(16, 64, 2) > 0


def test_rope_argument_checks(lib):
    def call(x=16, dt=0, rows=4, heads=2, hd=64, xs=(128, 64), pos=16, pf=0, ldpos=2, axes=2, pairs=(16, 16), fr=16,
             inter=1, inv=0, y=32, ys=(128, 64)):
        return lib.rope_axes(x, dt, rows, heads, hd, xs[0], xs[1], pos, pf, ldpos, axes,
                             (ctypes.c_int32 * 4)(*pairs), fr, inter, inv, y, ys[0], ys[1], None)

    for k in ("x", "y", "pos", "fr"):
        assert call(**{k: None}) == INVALID
    assert call(dt=3) == INVALID and call(inter=2) == INVALID and call(inv=2) == INVALID and call(pf=2) == INVALID
    assert call(rows=0) == SHAPE and call(heads=0) == SHAPE and call(hd=60) == SHAPE and call(hd=1032) == SHAPE
    assert call(axes=0) == SHAPE and call(axes=5) == SHAPE and call(pairs=(16, 0)) == SHAPE
    assert call(pairs=(16, 17)) == SHAPE and call(ldpos=1) == INVALID
    assert call(ys=(64, 64)) == INVALID and call(ys=(128, 32)) == INVALID and call(ys=(0, 64)) == INVALID
    assert call(ys=(128, -64)) == INVALID and call(xs=(-128, 64)) == INVALID
    assert call(y=16, ys=(256, 64)) == INVALID  # in place with other strides
    assert call(x=24) == MISALIGNED and call(y=40) == MISALIGNED and call(xs=(132, 64)) == MISALIGNED
    assert call(ys=(132, 64)) == MISALIGNED and call(fr=20) == MISALIGNED and call(pos=18) == MISALIGNED


# ---- argument checks of the Python calls -------------------------------------------------
def test_python_calls_refuse_wrong_tensors(lib):
    bf = torch.bfloat16
    B = _lib.NVFP4Tensor(torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), torch.ones(1), 8, 64)
    x, D = torch.zeros(2, 64, dtype=bf), torch.zeros(2, 8, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        ep.gemv_nvfp4(x, B, D)
    for bad in (x.float(), x[:, ::2], x[:, :32], x[0]):
        with pytest.raises(ValueError):
            ep.gemv_nvfp4(bad, B, D)
    for bad in (D.double(), D[:1], torch.zeros(8, 2, dtype=bf).t()):
        with pytest.raises(ValueError):
            ep.gemv_nvfp4(x, B, bad)
    with pytest.raises(ValueError):
        ep.gemv_nvfp4(x, B, D, bias=torch.zeros(8, dtype=bf))

    for codes, sf in ((B.codes[:7], B.sf), (B.codes, B.sf[:256])):  # the second is an MXFP4 tensor's
        with pytest.raises(ValueError, match="too small"):
            _lib._nvfp4(_lib.NVFP4Tensor(codes, sf, B.gscale, 8, 64))
    assert _lib._nvfp4(B).rows == 8

    h = torch.zeros(2, 64, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        ep.residual_norm(x, h)

    def norm_inputs(**k):
        a = dict(x=x, y=None, gate=None, scale=None, shift=None, w=None, w_post=None, norm="layer", post_norm=False,
                 residual_scale=1.0, eps=1e-6, offsets=None, batches=None)
        a.update(k)
        return _lib._norm_inputs(**a)

    assert norm_inputs()[1] == (1, 64)
    mod = torch.zeros(2, 192, dtype=bf)
    packed, shape = norm_inputs(y=x, gate=mod[:, :64], scale=mod[:, 64:128], shift=mod[:, 128:])
    a = dict(zip(NORM_FIELDS, _lib._NORM_INPUTS.unpack(packed)))
    assert shape == (2, 64) and (a["batches"], a["ldgate"], a["mod_dtype"]) == (2, 192, 0)
    for bad in (dict(x=x.half()), dict(x=x[0]), dict(norm="group"), dict(y=x.float()), dict(y=x[:, :32]),
                dict(scale=mod[:, :32]), dict(scale=mod[:, :64], shift=mod[:, :64].float()), dict(scale=mod[:, :64].half()),
                dict(w=torch.zeros(64, dtype=bf)), dict(w_post=torch.zeros(32)),
                dict(offsets=torch.zeros(3)), dict(offsets=torch.zeros(1, dtype=torch.int32)),
                dict(offsets=torch.zeros(3, dtype=torch.int32), batches=3)):
        with pytest.raises(ValueError):
            norm_inputs(**bad)

    q = torch.zeros(4, 2, 32)
    pos, fr = torch.zeros(4, 1, dtype=torch.int32), torch.zeros(16, dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        ep.rope_axes(q, pos, fr, [16])
    for args in ((q.double(), pos, fr, [16]), (q[0], pos, fr, [16]), (q, pos.long(), fr, [16]), (q, pos[:2], fr, [16]),
                 (q, pos, fr.float(), [16]), (q, pos, fr, [8]), (q, pos, fr, [8, 8]), (q, pos, fr, [16], q.half())):
        with pytest.raises(ValueError):
            ep.rope_axes(*args)


def test_oracle_dequantize_is_what_the_gemv_form_uses():
    q, s, G = o.quantize(np.random.default_rng(3).standard_normal((4, 32)).astype(np.float32))
    y, _ = lo.gemv(np.eye(32), q, s, G)
    assert np.allclose(y.T, o.dequantize(q, s, G), rtol=1e-6)
