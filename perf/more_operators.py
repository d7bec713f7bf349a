"""Workloads of a layer around the FP8 weights and of the tensors that are not
such weights: the linear layer in E4M3 (quantizer of its activations, forward
product, both gradients), layer norm with its gradient, and AdamW over many
tensors with states in 32 or in 8 bits.

own = False runs each operator in its plain form (elementary torch, 32 bits or
more); own = True calls blockwise_fp8_zero_amd.  A FP8 weight is a uint8 tensor
of E4M3 codes (rows, cols) and a float32 grid (ceil(rows/128), ceil(cols/128)):
value = code * grid of its 128x128 tile.
"""
import math
import random

import numpy as np
import torch

own = False

T = 128
BLOCK = 256  # elements that share the scales of 8-bit optimizer states
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
HP = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
STEP = 11
EPS = 1e-5
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # generation: one token through a square projection, bf16 in and out
        dict(name="linear_one", kind="linear", tokens=1, rows=4096, cols=4096, x="bf16", out="bf16"),
        # a batch of generated tokens through the up projection
        dict(name="linear_few", kind="linear", tokens=64, rows=11008, cols=4096, x="bf16", out="bf16"),
        # a prompt through the down projection
        dict(name="linear_prompt", kind="linear", tokens=2048, rows=4096, cols=11008, x="bf16", out="bf16"),
        # a ragged weight in training: rows off 16-byte boundaries, edge tiles on every side
        dict(name="linear_train_odd", kind="train", tokens=1013, rows=1544, cols=1001, x="f32", out="f32", pow2=True),
        # a training microbatch through the up projection: forward and both gradients, quantization included
        dict(name="linear_train_batch", kind="train", tokens=8192, rows=11008, cols=4096, x="bf16", out="bf16", pow2=False),
        # generation: the norm of one token
        dict(name="norm_one", kind="norm", tokens=1, dim=4096, x="bf16", param="f32", grad=False),
        # a batch of prompts
        dict(name="norm_batch", kind="norm", tokens=32768, dim=4096, x="bf16", param="f32", grad=False),
        # odd rows in 32 bits, forward and gradients
        dict(name="norm_grad_odd", kind="norm", tokens=3001, dim=1001, x="f32", param="f32", grad=True),
        # a training batch, forward and gradients
        dict(name="norm_grad_batch", kind="norm", tokens=32768, dim=4096, x="bf16", param="f32", grad=True),
        # the norm weights and biases of a model: many vectors, where launches count
        dict(name="adamw_vectors", kind="adamw", count=65, lo=4096, hi=4096, vectors=True, param="f32", grad="f32", bits=32, order=0, clip=True),
        # a ragged model's matrices and vectors, gradients as the backward pass left them, 8-bit states
        dict(name="adamw_ragged_8bit", kind="adamw", count=40, lo=129, hi=7168, vectors=False, param="f32", grad="mixed", bits=8, order=3, clip=True),
        # a token table kept in 32 bits
        dict(name="adamw_table", kind="adamw", count=1, lo=16384, hi=16384, vectors=False, param="f32", grad="bf16", bits=32, order=1, clip=False),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["linear", "linear", "train", "norm", "norm", "adamw"])

    def width(hi):
        return _spread(rng, 64, hi) if rng.random() < 0.5 else 64 * _spread(rng, 2, hi // 64)

    if kind == "linear":
        return dict(kind=kind, tokens=_spread(rng, 1, 8192), rows=width(11008), cols=width(11008), x=rng.choice(["bf16", "bf16", "f32", "f16"]),
                    out=rng.choice(["bf16", "bf16", "f32", "f16"]))
    if kind == "train":
        return dict(kind=kind, tokens=_spread(rng, 1, 8192), rows=width(8192), cols=width(4096), x=rng.choice(["bf16", "bf16", "f32"]),
                    out=rng.choice(["bf16", "f32"]), pow2=rng.random() < 0.5)
    if kind == "norm":
        x = rng.choice(["bf16", "bf16", "f16", "f32"])
        return dict(kind=kind, tokens=_spread(rng, 1, 16384), dim=width(8192), x=x, param=rng.choice(["f32", x]), grad=rng.random() < 0.6)
    lo = _spread(rng, 16, 500)
    return dict(kind=kind, count=_spread(rng, 1, 200), lo=lo, hi=_spread(rng, lo, 1500), vectors=rng.random() < 0.3, param=rng.choice(["f32", "f32", "bf16"]),
                grad=rng.choice(["f32", "bf16", "mixed"]), bits=rng.choice([8, 32]), order=rng.randrange(1 << 20), clip=rng.random() < 0.5)


# ---- inputs ------------------------------------------------------------------


def _shapes(c):
    """(rows, cols, gradient type) of each tensor of an adamw case."""
    r = random.Random(c["order"])
    out = []
    for k in range(c["count"]):
        h, w = _spread(r, c["lo"], c["hi"]), _spread(r, c["lo"], c["hi"])
        if c["vectors"] or k % 5 == 4:
            w = 1  # a norm's or a bias's vector
        out.append((h, w, ("f32" if k % 2 else "bf16") if c["grad"] == "mixed" else c["grad"]))
    return out


def _normal(shape, gen, std, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(dtype)


def _fp8_weight(rows, cols, gen, std):
    """E4M3 codes and tile scales of a normal weight, one scale per tile."""
    hb, wb = -(-rows // T), -(-cols // T)
    grid = (torch.rand((hb, wb), generator=gen, device="cuda") * 0.5 + 0.75) * (std * 4.5 / 448)
    up = grid.repeat_interleave(T, 0)[:rows].repeat_interleave(T, 1)[:, :cols]
    return (_normal((rows, cols), gen, std) / up).clamp_(-448, 448).to(E4M3).view(torch.uint8), grid


def _activations(tokens, dim, gen, dtype):
    """Hidden states: a few features are far larger than the others."""
    x = torch.randn((tokens, dim), generator=gen, device="cuda")
    x *= torch.where(torch.rand(dim, generator=gen, device="cuda") < 0.01, 20.0, 1.0)
    return x.to(dtype)


def _upstream(tokens, dim, gen, dtype):
    """Gradients of outputs: tokens differ in size, some (padding) have none."""
    size = torch.exp(torch.randn((tokens, 1), generator=gen, device="cuda")) * 1e-3
    size = torch.where(torch.rand((tokens, 1), generator=gen, device="cuda") < 0.03, 0.0, size)
    return (torch.randn((tokens, dim), generator=gen, device="cuda") * size).to(dtype)


def _places(c, per):
    """Where each tensor's values lie in a buffer of them all, one for every
    `per` elements: tensors start on multiples of 256 elements."""
    at = np.cumsum([0] + [-(-h * w // BLOCK) * BLOCK for h, w, _ in _shapes(c)]) // per
    return at.tolist()


def _slots(c, per, dtype, s, name, values):
    """Views, one for each tensor, of a buffer s[name] that holds them all."""
    at = _places(c, per)
    s[name] = torch.zeros(at[-1], dtype=dtype, device="cuda")
    views = [s[name][a:a + x.numel()].view(x.shape) for a, x in zip(at, values)]
    [v.copy_(x) for v, x in zip(views, values)]
    return views


def _warm_states(n, gen, bits):
    """Moments after some steps; in 8 bits their codes and block scales."""
    m, r = _normal((n,), gen, 3e-4), _normal((n,), gen, 1e-3).abs_()
    if bits == 32:
        return m, r.square_(), None, None
    (mc, ms), (rc, rs) = _plain_blocks(m), _plain_blocks(r, True)
    return mc, rc, ms, rs


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case=c)
    if c["kind"] in ("linear", "train"):
        n, rows, cols = c["tokens"], c["rows"], c["cols"]
        s["x"] = _activations(n, cols, gen, TYPES[c["x"]])
        s["weight"], s["grid"] = _fp8_weight(rows, cols, gen, 1.0 / math.sqrt(cols))
        s["y"] = torch.empty((n, rows), dtype=TYPES[c["out"]], device="cuda")
        if c["kind"] == "train":
            s["dy"] = _upstream(n, rows, gen, TYPES[c["x"]])
            s["dx"] = torch.empty((n, cols), dtype=TYPES[c["out"]], device="cuda")
            s["dweight"] = torch.empty((rows, cols), device="cuda")
    elif c["kind"] == "norm":
        n, d, x, p = c["tokens"], c["dim"], TYPES[c["x"]], TYPES[c["param"]]
        s["x"] = (_activations(n, d, gen, torch.float32) + _normal((n, 1), gen, 0.5)).to(x)
        s["weight"] = (1.0 + _normal((d,), gen, 0.2)).to(p)
        s["bias"] = _normal((d,), gen, 0.1, p)
        s["y"] = torch.empty((n, d), dtype=x, device="cuda")
        s["mean"], s["rstd"] = (torch.empty(n, device="cuda") for _ in range(2))
        if c["grad"]:
            s["dy"] = _upstream(n, d, gen, x)
            s["dx"] = torch.empty((n, d), dtype=x, device="cuda")
            s["dweight"], s["dbias"] = (torch.empty(d, device="cuda") for _ in range(2))
    else:
        shapes = _shapes(c)
        s["params"] = _slots(c, 1, TYPES[c["param"]], s, "flat", [_normal((h, w), gen, 0.02) for h, w, _ in shapes])
        s["grads"] = [_normal((h, w), gen, 1e-3, TYPES[t]) for h, w, t in shapes]
        states = list(zip(*[_warm_states(h * w, gen, c["bits"]) for h, w, _ in shapes]))
        kept = torch.float32 if c["bits"] == 32 else torch.uint8
        s["m"], s["v"] = (_slots(c, 1, kept, s, "flat_" + name, values) for name, values in zip("mv", states))
        s["m_scale"] = s["v_scale"] = [None] * len(shapes)
        if c["bits"] == 8:
            s["m_scale"], s["v_scale"] = (_slots(c, BLOCK, torch.float32, s, "flat_" + name, values)
                                          for name, values in zip(("m_scale", "v_scale"), states[2:]))
        s["coef"] = torch.full((1,), 0.37, device="cuda") if c["clip"] else None
    if own:
        import blockwise_fp8_zero_amd as bfz
        s["bfz"] = bfz
        if c["kind"] == "linear":
            s["work"] = bfz.linear_workspace(n, s["weight"], s["x"].dtype)
        if c["kind"] == "train":
            s["work"] = bfz.linear_workspace(n, s["weight"])
            s["xc"], s["xs"] = bfz.quantize_buffers(n, cols, tiles=True)
            s["dc"], s["ds"] = bfz.quantize_buffers(n, rows, tiles=True)
        if c["kind"] == "norm" and c["grad"]:
            s["work"] = bfz.layer_norm_workspace(n, d)
        if c["kind"] == "adamw":
            s["list"] = bfz.AdamWList(s["params"], s["m"], s["v"], s["m_scale"], s["v_scale"], grads=s["grads"])
            s["hp"] = bfz.AdamW(step=STEP, **HP)
    return s


# ---- one pass ----------------------------------------------------------------


def run(s):
    kind = s["case"]["kind"]
    return (OWN if own else PLAIN)[kind](s)


def _own_linear(s):
    s["bfz"].linear(s["x"], s["weight"], s["grid"], s["y"], s["work"])
    return s["y"]


def _own_train(s):
    bfz, pow2 = s["bfz"], s["case"]["pow2"]
    bfz.quantize(s["x"], s["xc"], s["xs"], tiles=True, pow2=pow2)
    bfz.linear(s["xc"], s["weight"], s["grid"], s["y"], s["work"], scales=s["xs"], tiles=True)
    bfz.quantize(s["dy"], s["dc"], s["ds"], tiles=True, pow2=pow2)
    bfz.linear_grad_input(s["dc"], s["weight"], s["grid"], s["dx"], s["work"], scales=s["ds"], tiles=True)
    bfz.linear_grad_weight(s["dc"], s["ds"], s["xc"], s["xs"], s["dweight"], s["work"])
    return dict(y=s["y"], dx=s["dx"], dweight=s["dweight"], x=s["xc"].view(E4M3), x_grid=s["xs"], dy=s["dc"].view(E4M3), dy_grid=s["ds"])


def _own_norm(s):
    bfz = s["bfz"]
    bfz.layer_norm(s["x"], s["weight"], s["bias"], s["y"], eps=EPS, mean=s["mean"], rstd=s["rstd"])
    if not s["case"]["grad"]:
        return s["y"], s["mean"], s["rstd"]
    bfz.layer_norm_grad(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"], s["work"])
    return s["y"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"]


def _own_adamw(s):
    s["list"].step(s["hp"], grad_scale=s["coef"])
    return _adamw_out(s)


def _adamw_out(s):
    if s["case"]["bits"] == 32:
        return dict(params=s["flat"], m=s["flat_m"], v=s["flat_v"])
    return dict(params=s["flat"], m=s["flat_m"].view(E4M3), v=s["flat_v"].view(E4M3), m_scale=s["flat_m_scale"], v_scale=s["flat_v_scale"])


OWN = dict(linear=_own_linear, train=_own_train, norm=_own_norm, adamw=_own_adamw)


def _scale(amax, pow2=False):
    """448 times it holds amax; 1 for nothing but zeros."""
    if pow2:
        mantissa, exponent = torch.frexp(amax)  # amax = mantissa 2^exponent, mantissa in [0.5, 1); 448 = 0.875 * 2^9
        scale = torch.ldexp(torch.ones_like(amax), exponent - 9 + (mantissa > 0.875).int())
    else:
        scale = amax / torch.full_like(amax, 448.0)  # by a tensor: by a number torch multiplies with the reciprocal
    return torch.where(amax == 0, torch.ones_like(amax), scale)


def _encode(quotient):
    return quotient.clamp(-448, 448).to(E4M3)


def _plain_rows(x):
    """Codes (n, d) and scales (ceil(d/128), n) of groups of 128 columns."""
    n, d = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -d % T)).view(n, -1, T)
    scale = _scale(x.abs().amax(2))
    return _encode(x / scale[:, :, None]).view(n, -1)[:, :d], scale.t()


def _plain_tiles(x, pow2):
    """Codes (n, d) and the grid of their 128x128 tiles."""
    n, d = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -d % T, 0, -n % T))
    h, w = x.shape
    x = x.view(h // T, T, w // T, T)
    scale = _scale(x.abs().amax(dim=(1, 3)), pow2)
    return _encode(x / scale[:, None, :, None]).view(h, w)[:n, :d], scale


def _plain_blocks(x, positive=False):
    """Codes and scales of blocks of 256 elements of a vector; positive: what
    is above zero stays above zero."""
    n = x.numel()
    x = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)
    scale = _scale(x.abs().amax(1))
    codes = _encode(x / scale[:, None]).view(torch.uint8)
    if positive:
        codes = torch.where((codes == 0) & (x > 0), torch.ones_like(codes), codes)
    return codes.view(-1)[:n].clone(), scale


def _tile_values(codes, grid):
    up = grid.repeat_interleave(T, 1)[:, :codes.shape[1]].repeat_interleave(T, 0)[:codes.shape[0]]
    return codes.view(E4M3).float() * up


def _plain_linear(s):
    codes, scales = _plain_rows(s["x"])
    x = codes.float() * scales.t().repeat_interleave(T, 1)[:, :codes.shape[1]]
    s["y"].copy_(x @ _tile_values(s["weight"], s["grid"]).t())
    return s["y"]


def _plain_train(s):
    pow2, w = s["case"]["pow2"], _tile_values(s["weight"], s["grid"])
    xc, xs = _plain_tiles(s["x"], pow2)
    dc, ds = _plain_tiles(s["dy"], pow2)
    x, dy = _tile_values(xc, xs), _tile_values(dc, ds)
    s["y"].copy_(x @ w.t())
    s["dx"].copy_(dy @ w)
    s["dweight"].copy_(dy.t() @ x)
    return dict(y=s["y"], dx=s["dx"], dweight=s["dweight"], x=xc, x_grid=xs, dy=dc, dy_grid=ds)


def _plain_norm(s):
    x, w = s["x"].float(), s["weight"].float()
    mean = x.mean(1, keepdim=True)
    x = x - mean
    rstd = 1.0 / torch.sqrt(x.square().mean(1, keepdim=True) + EPS)
    x = x * rstd
    s["y"].copy_(x * w + s["bias"].float())
    s["mean"].copy_(mean[:, 0])
    s["rstd"].copy_(rstd[:, 0])
    if not s["case"]["grad"]:
        return s["y"], s["mean"], s["rstd"]
    dy = s["dy"].float()
    g = dy * w
    s["dx"].copy_((g - g.mean(1, keepdim=True) - x * (g * x).mean(1, keepdim=True)) * rstd)
    s["dweight"].copy_((dy * x).sum(0))
    s["dbias"].copy_(dy.sum(0))
    return s["y"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"]


def _block_values(codes, scale):
    return codes.view(E4M3).float() * scale.repeat_interleave(BLOCK)[:codes.numel()]


def _plain_adamw(s):
    b1, b2, lr = HP["beta1"], HP["beta2"], HP["lr"]
    for k, (p, g) in enumerate(zip(s["params"], s["grads"])):
        g = g.float().view(-1)
        if s["coef"] is not None:
            g = g * s["coef"]
        if s["case"]["bits"] == 8:
            m, v = _block_values(s["m"][k], s["m_scale"][k]), _block_values(s["v"][k], s["v_scale"][k]).square_()
        else:
            m, v = s["m"][k], s["v"][k]
        m = m * b1 + g * (1 - b1)
        v = v * b2 + (g * g) * (1 - b2)
        root = v.sqrt()
        den = root / torch.full_like(root, math.sqrt(1 - b2 ** STEP)) + HP["eps"]
        x = p.float().view(-1)
        x = x - (m / den) * (lr / (1 - b1 ** STEP))
        x = x - x * (lr * HP["weight_decay"])
        p.copy_(x.view(p.shape))
        if s["case"]["bits"] == 8:
            for (codes, scale), names in ((_plain_blocks(m), ("m", "m_scale")), (_plain_blocks(root, True), ("v", "v_scale"))):
                s[names[0]][k].copy_(codes)
                s[names[1]][k].copy_(scale)
        else:
            s["m"][k].copy_(m)
            s["v"][k].copy_(v)
    return _adamw_out(s)


PLAIN = dict(linear=_plain_linear, train=_plain_train, norm=_plain_norm, adamw=_plain_adamw)


# ---- what a pass cannot do without --------------------------------------------


def work(case):
    c = case
    if c["kind"] in ("linear", "train"):
        n, o, i = c["tokens"], c["rows"], c["cols"]
        e, f = SIZE[c["x"]], SIZE[c["out"]]
        weight = o * i + 4 * (-(-o // T)) * (-(-i // T))
        once = n * i * e + weight + n * o * f
        if c["kind"] == "linear":
            return dict(bytes=once, flops=2 * n * o * i)
        # codes are written, for the caller, and both gradients
        return dict(bytes=once + n * (o + i) + n * o * e + n * i * f + 4 * o * i, flops=6 * n * o * i)
    if c["kind"] == "norm":
        n, d, e = c["tokens"], c["dim"], SIZE[c["x"]]
        moved = 2 * n * d * e + 8 * n + 2 * d * SIZE[c["param"]]
        return dict(bytes=moved + ((2 * n * d * e + 8 * d) if c["grad"] else 0), flops=(20 if c["grad"] else 8) * n * d)
    total = {t: sum(h * w for h, w, g in _shapes(c) if g == t) for t in ("f32", "bf16")}
    n = total["f32"] + total["bf16"]
    state = 16.0 if c["bits"] == 32 else 4.0 + 16.0 / BLOCK
    return dict(bytes=int(n * (2 * SIZE[c["param"]] + state)) + 4 * total["f32"] + 2 * total["bf16"], flops=20 * n)


# ---- the same from the definitions, in 64 bits ---------------------------------


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return EXACT[case["kind"]](s, case)


def _exact_quantized(x, rows, pow2):
    """Values, scales of quantized x: the scale is a 32-bit number and so is
    the quotient that is rounded to E4M3, both rounded once from 64 bits."""
    n, d = x.shape
    x = x.double()
    value = torch.empty_like(x)
    hb = n if rows else (n + T - 1) // T
    scales = torch.empty((hb, (d + T - 1) // T), dtype=torch.float64, device="cuda")
    for j in range(scales.shape[1]):
        part = x[:, j * T:(j + 1) * T]
        top = part.abs().max(1).values
        if not rows:
            top = torch.stack([t.max() for t in top.split(T)])
        sc = torch.exp2(torch.ceil(torch.log2(top / 448))) if pow2 else (top / 448).float().double()
        sc[top == 0] = 1
        scales[:, j] = sc
        each = (sc if rows else sc.repeat_interleave(T)[:n])[:, None]
        q = (part / each).float()
        value[:, j * T:(j + 1) * T] = torch.clamp(q, min=-448, max=448).to(E4M3).double() * each
    return value, scales


def _exact_weight(s):
    r, k = (torch.arange(z, device="cuda") // T for z in s["weight"].shape)
    return s["weight"].view(E4M3).to(torch.float64) * s["grid"].double()[r][:, k]


def _exact_linear(s, c):
    x, _ = _exact_quantized(s["x"], True, False)
    return torch.matmul(x, _exact_weight(s).T)


def _exact_train(s, c):
    w = _exact_weight(s)
    x, xs = _exact_quantized(s["x"], False, c["pow2"])
    dy, ds = _exact_quantized(s["dy"], False, c["pow2"])
    return dict(y=torch.matmul(x, w.T), dx=torch.matmul(dy, w), dweight=torch.matmul(dy.T, x), x=None, x_grid=xs, dy=None, dy_grid=ds)


def _exact_norm(s, c):
    n, d = c["tokens"], c["dim"]
    w, b = s["weight"].double(), s["bias"].double()
    shape = dict(dtype=torch.float64, device="cuda")
    y, dx = torch.empty((n, d), **shape), torch.empty((n, d), **shape)
    mean, rstd, dw, db = torch.empty(n, **shape), torch.empty(n, **shape), torch.zeros(d, **shape), torch.zeros(d, **shape)
    for a in range(0, n, 4096):
        at = slice(a, a + 4096)
        x = s["x"][at].double()
        mean[at] = x.sum(1) / d
        var = ((x - mean[at, None]) ** 2).sum(1) / d
        rstd[at] = (var + EPS) ** -0.5
        h = (x - mean[at, None]) * rstd[at, None]
        y[at] = torch.addcmul(b, h, w)
        if c["grad"]:
            dy = s["dy"][at].double()
            up = dy * w
            c1, c2 = up.sum(1, keepdim=True) / d, (up * h).sum(1, keepdim=True) / d
            dx[at] = (up - c1 - h * c2) * rstd[at, None]
            dw += torch.einsum("td,td->d", dy, h)
            db += dy.sum(0)
    return (y, mean, rstd, dx, dw, db) if c["grad"] else (y, mean, rstd)


def _exact_adamw(s, c):
    b1, b2, lr, coef = HP["beta1"], HP["beta2"], HP["lr"], (float(s["coef"]) if c["clip"] else 1.0)
    names = ("params", "m", "v") if c["bits"] == 32 else ("params", "m", "v", "m_scale", "v_scale")
    out = {name: s["flat" if name == "params" else "flat_" + name].double() for name in names if c["bits"] == 32 or name not in ("m", "v")}
    start = 0
    for k, (p, g) in enumerate(zip(s["params"], s["grads"])):
        g, p64 = g.double().flatten() * coef, p.double().flatten()
        n = g.numel()
        m, v = s["m"][k], s["v"][k]
        if c["bits"] == 8:
            at = torch.arange(n, device="cuda") // BLOCK
            m = m.view(E4M3).to(torch.float64) * s["m_scale"][k].double()[at]
            v = (v.view(E4M3).to(torch.float64) * s["v_scale"][k].double()[at]) ** 2
        m = b1 * m.double() + (1 - b1) * g
        v = b2 * v.double() + (1 - b2) * g ** 2
        mhat, vhat = m / (1 - b1 ** STEP), v / (1 - b2 ** STEP)
        out["params"][start:start + n] = (p64 - lr * mhat / (vhat ** 0.5 + HP["eps"])) * (1 - lr * HP["weight_decay"])
        if c["bits"] == 32:
            out["m"][start:start + n], out["v"][start:start + n] = m, v
        else:
            for x, name in ((m, "m_scale"), (v ** 0.5, "v_scale")):
                whole = n // BLOCK * BLOCK
                top = [x[:whole].view(-1, BLOCK).abs().max(1).values] if whole else []
                top = torch.cat(top + ([x[whole:].abs().max().view(1)] if whole < n else []))
                out[name][start // BLOCK:start // BLOCK + len(top)] = torch.where(top > 0, top / 448, torch.ones_like(top))
        start += (n + BLOCK - 1) // BLOCK * BLOCK
    return {name: out.get(name) for name in names}


EXACT = dict(linear=_exact_linear, train=_exact_train, norm=_exact_norm, adamw=_exact_adamw)
