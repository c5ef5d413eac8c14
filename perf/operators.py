"""Operators around the NVFP4 GEMMs of a transformer layer, as they are measured.

- ``gemv``: a few rows (the conditioning vectors of a batch of images, or the tokens of a
  decoding step) times an NVFP4 weight: 4-bit values with a scale per group of 16.
- ``norm``: the residual stream between two blocks: the branch's output normalised, gated and
  added to the stream, and the next block's input normalised and modulated; its gradient
  (``norm_grad``); and with an NVFP4 output, followed by the projection that reads it
  (``norm_proj``).
- ``rope``: rotary positions with one to three axes (time, height, width) on the heads of Q and K.

Each case is one call. ``own`` picks the framework's kernels or the plain form in elementary
torch operations.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
LARGEST_WEIGHT = 24576 * 4096
LARGEST_ROWS = 16384 * 4096
LARGEST_HEADS = 14091 * 24 * 128


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def listed():
    return [
        # a timestep embedding's projection of a small model: latency is all there is
        dict(name="gemv_one", op="gemv", M=1, K=1024, N=1024, x="bf16", out="bf16", silu=False, bias=True),
        # the six modulation vectors of a layer for an image and its unconditional twin
        dict(name="gemv_modulation", op="gemv", M=2, K=4096, N=24576, x="bf16", out="bf16", silu=True, bias=True),
        # the down projection for a handful of tokens, an output width that no tile divides
        dict(name="gemv_tokens", op="gemv", M=13, K=12288, N=4099, x="f16", out="f32", silu=False, bias=False),
        # the first norm of a layer on the tokens of a thumbnail: no branch to add yet
        dict(name="norm_first", op="norm", M=256, D=1024, batches=1, ragged=False, stream="bf16", mod="bf16",
             branch=False, post=False, norm="layer"),
        # a layer's middle on one 1K image: branch added with its gate, LayerNorm, modulation
        dict(name="norm_image", op="norm", M=4096, D=4096, batches=2, ragged=False, stream="bf16", mod="bf16",
             branch=True, post=False, norm="layer"),
        # images of several sizes packed behind one another, a float32 stream, norms on both sides
        dict(name="norm_packed", op="norm", M=6021, D=2568, batches=5, ragged=True, stream="f32", mod="f32",
             branch=True, post=True, norm="rms"),
        # one training step's gradient of the same op for packed images
        dict(name="norm_grad_packed", op="norm_grad", M=1531, D=2048, batches=3, ragged=True, stream="f32",
             mod="f32", branch=True, post=True, norm="rms"),
        # and for a batch of 1K images at full width
        dict(name="norm_grad_batch", op="norm_grad", M=16384, D=4096, batches=4, ragged=False, stream="bf16",
             mod="bf16", branch=True, post=False, norm="layer"),
        # the norm hands its NVFP4 output to the projection that follows
        dict(name="norm_proj", op="norm_proj", M=1024, D=2048, N=2048, batches=1, ragged=False, stream="bf16",
             mod="bf16", branch=True, post=False, norm="layer"),
        # the tokens of a prompt, one axis, far positions
        dict(name="rope_text", op="rope", M=77, H=16, hd=64, axes="32", type="f32", interleaved=False, far=True,
             fraction=False, inverse=False, swap=False),
        # Q and K heads of one 1K image inside the QKV buffer, three axes
        dict(name="rope_image", op="rope", M=4096, H=24, hd=256, axes="16,56,56", type="bf16", interleaved=True,
             far=False, fraction=False, inverse=False, swap=False),
        # the gradient through the rotation for a video, heads outermost on the way out
        dict(name="rope_video_grad", op="rope", M=14091, H=24, hd=128, axes="16,24,24", type="f16",
             interleaved=True, far=False, fraction=True, inverse=True, swap=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemv", "norm", "norm_grad", "norm_proj", "rope"])
    if op == "gemv":
        K = 64 * _log(rng, 1, 256)
        N = min(_log(rng, 16, 24576), LARGEST_WEIGHT // K)
        silu = rng.random() < 0.5
        return dict(op=op, M=_log(rng, 1, 40), K=K, N=N, x=rng.choice(["bf16", "f16"]),
                    out=rng.choice(["bf16", "f16"] if silu else ["bf16", "f16", "f32"]), silu=silu,
                    bias=rng.random() < 0.5)
    if op == "norm" or op == "norm_grad":
        D = 8 * _log(rng, 8, 1024)
        M = min(_log(rng, 1, 16384), LARGEST_ROWS // D)
        ragged = rng.random() < 0.5
        batches = rng.randint(1, 6) if ragged else rng.choice([b for b in (1, 2, 3, 4, 8) if M % b == 0])
        branch = op == "norm_grad" or rng.random() < 0.7
        return dict(op=op, M=M, D=D, batches=batches, ragged=ragged, stream=rng.choice(["bf16", "f32"]),
                    mod=rng.choice(["bf16", "f32"]), branch=branch, post=branch and rng.random() < 0.5,
                    norm=rng.choice(["layer", "rms"]))
    if op == "norm_proj":
        return dict(op=op, M=128 * _log(rng, 1, 16), D=256 * _log(rng, 1, 16), N=256 * _log(rng, 1, 16),
                    batches=1, ragged=False, stream=rng.choice(["bf16", "f32"]), mod=rng.choice(["bf16", "f32"]),
                    branch=rng.random() < 0.7, post=False, norm=rng.choice(["layer", "rms"]))
    hd = rng.choice([64, 128, 256])
    H = rng.randint(1, 40)
    M = min(_log(rng, 1, 16384), LARGEST_HEADS // (H * hd))
    n = rng.randint(1, 3)
    left, axes = hd // 2, []
    for i in range(n):  # pairs of each axis; what is left over is not rotated
        axes.append(left if n == 1 else rng.randint(1, left - (n - 1 - i)))
        left -= axes[-1]
    return dict(op=op, M=M, H=H, hd=hd, axes=",".join(map(str, axes)), type=rng.choice(["bf16", "f16", "f32"]),
                interleaved=rng.random() < 0.5, far=rng.random() < 0.3, fraction=rng.random() < 0.3,
                inverse=rng.random() < 0.5, swap=rng.random() < 0.5)


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _pack_nvfp4(w):
    """Codes, block scales in the tensor-core layout and per-tensor scale of a weight (rows x cols)."""
    rows, cols = w.shape
    G = w.abs().amax().float() / 2688.0
    blocks = w.float().view(rows, cols // 16, 16)
    s = (blocks.abs().amax(2) / (6.0 * G)).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = s.float() * G
    v = blocks / torch.where(d > 0, d, torch.ones_like(d))[..., None]
    v = torch.where(d[..., None] > 0, v, torch.zeros_like(v))
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    code = torch.bucketize(v.abs(), mids).to(torch.uint8) + 8 * (v < 0).to(torch.uint8)
    code = code.view(rows, cols // 2, 2)
    codes = (code[..., 0] + 16 * code[..., 1]).contiguous()
    pad = (rows + 127) // 128 * 128
    sb = torch.zeros(pad, cols // 16, dtype=torch.uint8, device=w.device)
    sb[:rows] = s.view(torch.uint8)
    sf = sb.view(pad // 128, 4, 32, cols // 64, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)
    return codes, sf, G.reshape(1)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    s = dict(case=case)
    if case["op"] == "gemv":
        M, K, N = case["M"], case["K"], case["N"]
        x = rn(M, K)
        x[:, torch.randint(0, K, (max(1, K // 1000),), generator=g, device=DEV)] *= 20.0  # outlier channels
        s["x"] = x.to(TYPES[case["x"]])
        s["codes"], s["sf"], s["g"] = _pack_nvfp4((rn(N, K) / math.sqrt(K)).bfloat16())
        s["bias"] = rn(N) * 0.1 if case["bias"] else None
        s["out"] = torch.zeros(M, N, dtype=TYPES[case["out"]], device=DEV)
        return s
    if case["op"] == "rope":
        M, H, hd, T = case["M"], case["H"], case["hd"], TYPES[case["type"]]
        axes = [int(a) for a in case["axes"].split(",")]
        s["axes"] = axes
        s["freqs"] = torch.cat([10000.0 ** (-torch.arange(n, dtype=torch.float64) / n) for n in axes]).to(DEV)
        # the heads sit in a wider row, as Q and K do beside V
        s["x"] = rn(M, H + max(1, H // 2), hd).to(T)[:, :H]
        side = max(1, round(M ** (1 / len(axes))))
        i = torch.arange(M, device=DEV)
        pos = torch.stack([(i // side ** (len(axes) - 1 - k)) % (side if k else M) for k in range(len(axes))], 1)
        if case["far"]:
            pos = pos + torch.randint(0, 1 << 20, (1, len(axes)), generator=g, device=DEV)
        s["pos"] = (pos.float() * 0.75 - 0.5) if case["fraction"] else pos.int()
        s["out"] = (torch.zeros(H, M, hd, dtype=T, device=DEV).transpose(0, 1) if case["swap"]
                    else torch.zeros(M, H, hd, dtype=T, device=DEV))
        return s
    M, D, B = case["M"], case["D"], case["batches"]
    ST, MT = TYPES[case["stream"]], TYPES[case["mod"]]
    if case["ragged"]:  # packed sequences, some rows behind the last one
        cuts = torch.randint(0, M + 1, (B + 1,), generator=g, device=DEV).sort().values
        cuts[0] = 0
        cuts[-1] = M - min(M - 1, M // 50)
        s["offsets"] = torch.minimum(cuts, cuts[-1]).int()
    else:
        s["offsets"] = None
    s["x"] = (rn(M, D) * 2 + 0.3).to(ST)
    # shift, scale and gate are slices of one modulation output
    mod = (rn(B, 3 * D) * 0.3).to(MT)
    s["shift"], s["scale"], s["gate"] = mod[:, :D], mod[:, D:2 * D], mod[:, 2 * D:]
    s["w"] = 1 + 0.1 * rn(D) if case["norm"] == "rms" else None
    s["y"] = (rn(M, D) * 1.5).bfloat16() if case["branch"] else None
    s["w_post"] = 1 + 0.1 * rn(D) if case["post"] else None
    s["alpha"] = 0.9 if case["post"] else 1.0
    if not case["branch"]:
        s["gate"] = None
    if case["op"] == "norm_grad":  # x is the stream after the addition, as the forward pass left it
        s["dx_out"] = rn(M, D).to(ST)
        s["dh"] = rn(M, D).bfloat16()
        xd, yd = s["x"].double(), s["y"].double()
        mean = xd.mean(1) if case["norm"] == "layer" else torch.zeros(M, device=DEV, dtype=torch.float64)
        rstd = ((xd - mean[:, None]).square().mean(1) + 1e-6).rsqrt()
        s["stats"] = torch.stack([mean, rstd, (yd.square().mean(1) + 1e-6).rsqrt(), torch.zeros_like(mean)], 1).float()
        s["dx"], s["dy"] = torch.zeros_like(s["x"]), torch.zeros_like(s["y"])
        s["dmod"] = torch.zeros(3, B, D, device=DEV)
        s["dw"] = torch.zeros(D, device=DEV) if s["w"] is not None else None
        s["dw_post"] = torch.zeros(D, device=DEV) if case["post"] else None
        return s
    s["x_out"] = torch.zeros_like(s["x"]) if case["branch"] else None
    if case["op"] == "norm":
        s["h"] = torch.zeros(M, D, dtype=torch.bfloat16, device=DEV)
        return s
    N = case["N"]
    s["codes"], s["sf"], s["g"] = _pack_nvfp4((rn(N, D) / math.sqrt(D)).bfloat16())
    s["h_codes"] = torch.zeros(M, D // 2, dtype=torch.uint8, device=DEV)
    s["h_sf"] = torch.zeros(M * D // 16, dtype=torch.uint8, device=DEV)
    s["h_g"] = torch.full((1,), 7.93714 / 2688.0, device=DEV)  # calibrated: no round number
    s["out"] = torch.zeros(M, N, dtype=torch.bfloat16, device=DEV)
    return s


# ---------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------
_LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _weight(codes, sf, rows, cols):
    """The values of NVFP4 codes and block scales, without the per-tensor scale, in 32 bits."""
    lut = torch.tensor(_LEVELS, device=codes.device)
    v = torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], 2).view(rows, cols // 16, 16)
    s = sf.view(-1, cols // 64, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, cols // 16)[:rows]
    return (v * s.contiguous().view(torch.float8_e4m3fn).float()[..., None]).view(rows, cols)


def _plain_gemv(s):
    x = s["x"].float()
    if s["case"]["silu"]:
        x = x / (1 + torch.exp(-x))
    y = x @ _weight(s["codes"], s["sf"], s["case"]["N"], s["case"]["K"]).t() * s["g"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["out"].dtype)


def _plain_batch(s):
    """The sequence of each row, and whether it has one."""
    M, B = s["case"]["M"], s["case"]["batches"]
    r = torch.arange(M, device=DEV)
    if s["offsets"] is None:
        return r // (M // B), None
    b = torch.searchsorted(s["offsets"], r.int(), right=True) - 1
    return b.clamp(max=B - 1), (b < B)[:, None]


def _plain_norm(s):
    b, live = _plain_batch(s)
    x = s["x"].float()
    x_out = None
    if s["y"] is not None:
        y = s["y"].float()
        if s["w_post"] is not None:
            y = y * torch.rsqrt(y.square().mean(1, keepdim=True) + 1e-6) * s["w_post"]
        x_out = (s["alpha"] * x + s["gate"].float()[b] * y).to(s["x"].dtype)
        x = x_out.float()  # the norm reads the stream as it is stored
    if s["case"]["norm"] == "layer":
        x = x - x.mean(1, keepdim=True)
    h = x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)
    if s["w"] is not None:
        h = h * s["w"]
    h = h * (1 + s["scale"].float()[b]) + s["shift"].float()[b]
    if live is not None:
        h = torch.where(live, h, 0.0)
        x_out = None if x_out is None else torch.where(live, x_out, torch.zeros_like(x_out))
    return x_out, h


def _plain_grad(s):
    b, live = _plain_batch(s)
    B, st = s["case"]["batches"], s["stats"]
    dh, dxo = s["dh"].float(), s["dx_out"].float()
    xhat = (s["x"].float() - st[:, 0:1]) * st[:, 1:2]
    yhat = s["y"].float()
    if s["w_post"] is not None:
        yhat = yhat * st[:, 2:3]
    one = 1 + s["scale"].float()[b]
    w = s["w"] if s["w"] is not None else 1.0
    d = dh * one * w
    dn = d - xhat * (d * xhat).mean(1, keepdim=True)
    if s["case"]["norm"] == "layer":
        dn = dn - d.mean(1, keepdim=True)
    t = dxo + st[:, 1:2] * dn
    gate, wp = s["gate"].float()[b], s["w_post"] if s["w_post"] is not None else 1.0
    e = t * gate * wp
    dy = e if s["w_post"] is None else st[:, 2:3] * (e - yhat * (e * yhat).mean(1, keepdim=True))
    dx = s["alpha"] * t
    if live is not None:
        zero = torch.zeros((), device=DEV)
        dx, dy, dh, t = (torch.where(live, v, zero) for v in (dx, dy, dh, t))
    rows = [dh, dh * xhat * w, t * yhat * wp]  # shift, scale, gate
    pick = torch.nn.functional.one_hot(b, B).double().t()
    dmod = torch.stack([(pick @ v.double()) for v in rows]).float()
    dw = (dh * one * xhat).double().sum(0).float() if s["w"] is not None else None
    dwp = (t * gate * yhat).double().sum(0).float() if s["w_post"] is not None else None
    return dict(dx=dx.to(s["x"].dtype), dy=dy.bfloat16(), dmod=dmod, dw=dw, dw_post=dwp)


def _plain_proj(s):
    case = s["case"]
    x_out, h = _plain_norm(s)
    h = h.bfloat16().float()  # what is quantised is the bf16 value
    blocks = h.view(case["M"], -1, 16)
    sc = (blocks.abs().amax(2) / (6.0 * s["h_g"])).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    d = (sc * s["h_g"])[..., None]
    v = torch.where(d > 0, blocks / torch.where(d > 0, d, torch.ones_like(d)), torch.zeros_like(blocks))
    a = v.abs()
    a = torch.where(a < 2, torch.round(2 * a) / 2, torch.where(a < 4, torch.round(a), 2 * torch.round(a / 2)))
    v = a.clamp(max=6.0) * torch.sign(v)
    hq = (v * sc[..., None]).view(case["M"], -1)
    out = hq @ _weight(s["codes"], s["sf"], case["N"], case["D"]).t() * (s["h_g"] * s["g"])
    return x_out, out.bfloat16()


def _plain_rope(s):
    x, case = s["x"].float(), s["case"]
    axis = torch.cat([torch.full((n,), k, dtype=torch.long) for k, n in enumerate(s["axes"])]).to(DEV)
    a = s["pos"].double()[:, axis] * s["freqs"]
    c, sn = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    if case["inverse"]:
        sn = -sn
    n = axis.numel()
    out = x.clone()
    if case["interleaved"]:
        p, q = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        out[..., 0:2 * n:2], out[..., 1:2 * n:2] = p * c - q * sn, p * sn + q * c
    else:
        p, q = x[..., :n], x[..., n:2 * n]
        out[..., :n], out[..., n:2 * n] = p * c - q * sn, p * sn + q * c
    return out.to(s["x"].dtype)


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------
def _own(s):
    import epilogues_nvfp4_quantize_b200 as ep
    case, op = s["case"], s["case"]["op"]
    if op == "gemv":
        B = ep.NVFP4Tensor(s["codes"], s["sf"], s["g"], case["N"], case["K"])
        return ep.gemv_nvfp4(s["x"], B, s["out"], bias=s["bias"], silu=case["silu"])
    if op == "rope":
        return ep.rope_axes(s["x"], s["pos"], s["freqs"], s["axes"], s["out"], interleaved=case["interleaved"],
                            inverse=case["inverse"])
    if op == "norm_grad":
        ep.residual_norm_backward(
            s["x"], s["stats"], dx_out=s["dx_out"], dh=s["dh"], y=s["y"], gate=s["gate"], post_norm=case["post"],
            w_post=s["w_post"], residual_scale=s["alpha"], norm=case["norm"], w=s["w"], scale=s["scale"],
            offsets=s["offsets"], dx=s["dx"], dy=s["dy"], dshift=s["dmod"][0], dscale=s["dmod"][1],
            dgate=s["dmod"][2], dw=s["dw"], dw_post=s["dw_post"])
        return {k: s[k] for k in ("dx", "dy", "dmod", "dw", "dw_post")}
    same = dict(y=s["y"], x_out=s["x_out"], gate=s["gate"], post_norm=case["post"], w_post=s["w_post"],
                residual_scale=s["alpha"], norm=case["norm"], w=s["w"], scale=s["scale"], shift=s["shift"], eps=1e-6,
                offsets=s["offsets"])
    if op == "norm":
        ep.residual_norm(s["x"], h=s["h"], **same)
        return s["x_out"], s["h"]
    A = ep.NVFP4Tensor(s["h_codes"], s["h_sf"], s["h_g"], case["M"], case["D"])
    B = ep.NVFP4Tensor(s["codes"], s["sf"], s["g"], case["N"], case["D"])
    ep.residual_norm(s["x"], hq=A, **same)
    return s["x_out"], ep.gemm_nvfp4_plain(A, B, s["out"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "gemv":
        return _plain_gemv(state)
    if op == "rope":
        return _plain_rope(state)
    if op == "norm_grad":
        return _plain_grad(state)
    if op == "norm_proj":
        return _plain_proj(state)
    x_out, h = _plain_norm(state)
    return x_out, h.bfloat16()


# ---------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def work(case):
    if case["op"] == "gemv":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": N * K * 9 // 16 + M * K * 2 + M * N * _SIZE[case["out"]] + 4 * N * case["bias"],
                "flops": 2 * M * N * K}
    if case["op"] == "rope":
        M, H, hd, n = case["M"], case["H"], case["hd"], len(case["axes"].split(","))
        return {"bytes": 2 * M * H * hd * _SIZE[case["type"]] + 4 * M * n, "flops": 3 * M * H * hd}
    M, D, B = case["M"], case["D"], case["batches"]
    st, md = _SIZE[case["stream"]], _SIZE[case["mod"]]
    vectors = 4 * D * ((case["norm"] == "rms") + case["post"])
    if case["op"] == "norm_grad":  # x, y, dx_out, dh and the statistics in; dx, dy and the vectors' gradients out
        return {"bytes": M * D * (3 * st + 3 * 2) + 16 * M + B * D * (2 * md + 12) + 2 * vectors,
                "flops": 30 * M * D}
    own_out = 9 / 16 if case["op"] == "norm_proj" else 2
    n = {"bytes": M * D * (st + case["branch"] * (2 + st) + own_out) + B * D * md * (2 + case["branch"]) + vectors,
         "flops": 14 * M * D}
    if case["op"] == "norm_proj":
        N = case["N"]
        n["bytes"] += M * D * 9 / 16 + N * D * 9 / 16 + 2 * M * N
        n["flops"] += 2 * M * N * D
    return n


# ---------------------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------------------
def _exact_values(codes, sf, G, rows, cols):
    """Value of element (r, c): level(code) * scale(block) * G."""
    byte = codes.repeat_interleave(2, 1)
    odd = torch.arange(cols, device=DEV) % 2 == 1
    code = torch.where(odd, byte // 16, byte % 16).to(torch.int32)
    e, m = (code // 2) % 4, (code % 2).double()
    mag = torch.where(e == 0, m / 2, torch.pow(2.0, (e - 1).double()) * (1 + m / 2))
    val = torch.where(code >= 8, -mag, mag)
    r, k = torch.arange(rows, device=DEV)[:, None], torch.arange(cols // 16, device=DEV)[None, :]
    at = ((r // 128) * (cols // 64) + k // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + k % 4
    b = sf[at].to(torch.int32)
    e, m = b // 8, (b % 8).double()
    scale = torch.where(e == 0, m / 512, torch.pow(2.0, (e - 7).double()) * (1 + m / 8))
    return val * scale.repeat_interleave(16, 1) * G.double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemv":
        x = s["x"].double()
        if case["silu"]:
            x = x * torch.sigmoid(x)
        out = []
        for n0 in range(0, case["N"], 4096):  # in pieces of the output
            n1 = min(case["N"], n0 + 4096)
            whole = torch.zeros(n1 - n0, case["K"], dtype=torch.float64, device=DEV)
            whole += _exact_values(s["codes"][n0:n1], s["sf"][n0 * (case["K"] // 16):], s["g"], n1 - n0, case["K"])
            out.append(x @ whole.t())
        y = torch.cat(out, 1)
        return y if s["bias"] is None else y + s["bias"].double()
    if op == "rope":
        x, out = s["x"].double(), s["x"].double().clone()
        at = 0
        for k, n in enumerate(s["axes"]):
            for j in range(n):
                p = at + j
                a = s["pos"][:, k].double() * s["freqs"][p] * (-1 if case["inverse"] else 1)
                i0, i1 = (2 * p, 2 * p + 1) if case["interleaved"] else (p, p + sum(s["axes"]))
                z = torch.complex(x[..., i0], x[..., i1]) * torch.polar(torch.ones_like(a), a)[:, None]
                out[..., i0], out[..., i1] = z.real, z.imag
            at += n
        return out
    M, D, B = case["M"], case["D"], case["batches"]
    off = s["offsets"].tolist() if s["offsets"] is not None else [i * (M // B) for i in range(B + 1)]
    if op == "norm_grad":
        # gradients by automatic differentiation of the definition, around the stored stream
        dx, dy = torch.zeros(M, D, dtype=torch.float64, device=DEV), torch.zeros(M, D, dtype=torch.float64, device=DEV)
        dmod = torch.zeros(3, B, D, dtype=torch.float64, device=DEV)
        one = torch.ones(D, dtype=torch.float64, device=DEV)
        w = (s["w"].double() if s["w"] is not None else one.clone()).requires_grad_(True)
        wp = (s["w_post"].double() if case["post"] else one.clone()).requires_grad_(True)
        dw, dwp = torch.zeros_like(one), torch.zeros_like(one)
        for b in range(B):
            for r0 in range(off[b], off[b + 1], 2048):
                r = slice(r0, min(off[b + 1], r0 + 2048))
                y, gate, scale, shift = (v.double().clone().requires_grad_(True)
                                         for v in (s["y"][r], s["gate"][b], s["scale"][b], s["shift"][b]))
                z = s["x"][r].double().clone().requires_grad_(True)  # the stream after the addition
                c = z - z.mean(1, keepdim=True) if case["norm"] == "layer" else z
                h = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-6) * w * (1 + scale) + shift
                gz, gs, gh, gw = torch.autograd.grad(h, (z, scale, shift, w), s["dh"][r].double())
                t = s["dx_out"][r].double() + gz
                u = y / torch.sqrt((y * y).mean(1, keepdim=True) + 1e-6) * wp if case["post"] else y * wp
                gy, gg, gwp = torch.autograd.grad(gate * u, (y, gate, wp), t)
                dx[r], dy[r] = s["alpha"] * t, gy
                dmod[0, b] += gh
                dmod[1, b] += gs
                dmod[2, b] += gg
                dw += gw
                dwp += gwp
        return dict(dx=dx, dy=dy, dmod=dmod, dw=dw if s["w"] is not None else None, dw_post=dwp if case["post"] else None)
    x_out = torch.zeros(M, D, dtype=torch.float64, device=DEV)
    h = torch.zeros(M, D, dtype=torch.float64, device=DEV)
    for b in range(B):
        r = slice(off[b], off[b + 1])
        z = s["x"][r].double()
        if case["branch"]:
            y = s["y"][r].double()
            if case["post"]:
                y = y / torch.sqrt((y * y).mean(1, keepdim=True) + 1e-6) * s["w_post"].double()
            z = s["alpha"] * z + s["gate"][b].double() * y
            x_out[r] = z
            z = z.to(s["x"].dtype).double()  # the stored stream
        c = z - z.mean(1, keepdim=True) if case["norm"] == "layer" else z
        n = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-6)
        n = n * s["w"].double() if s["w"] is not None else n
        h[r] = n * (1 + s["scale"][b].double()) + s["shift"][b].double()
    x_out = x_out if case["branch"] else None
    if op == "norm":
        return x_out, h
    G = s["h_g"].double()
    blocks = h.bfloat16().double().view(M, D // 16, 16)
    sc = (blocks.abs().amax(2) / (6 * G)).clamp(max=448).float().to(torch.float8_e4m3fn).double()
    lv = torch.tensor(_LEVELS[:8], dtype=torch.float64, device=DEV)
    q = torch.empty_like(blocks)
    for r0 in range(0, M, 256):  # the nearest level, the lower one's neighbour with the even code at a tie
        v = blocks[r0:r0 + 256] / torch.where(sc[r0:r0 + 256] > 0, sc[r0:r0 + 256] * G, torch.ones_like(G))[..., None]
        far = (v.abs().clamp(max=6)[..., None] - lv).abs()
        far[..., 1::2] += 1e-13
        q[r0:r0 + 256] = lv[far.argmin(-1)] * torch.sign(v)
    A = (q * (sc * G)[..., None]).view(M, D)
    return x_out, A @ _exact_values(s["codes"], s["sf"], s["g"], case["N"], D).t()
