"""Workloads of the training operators around the FP8 weights: the global
gradient norm with its clipping (alone, and inside the optimizer step), the
token embedding with its gradient, and the vocabulary cross entropy with its
gradient.

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
TILE = T * T
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "fp8": 1}
HP = dict(lr=1e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
STEP = 11


def listed():
    return [
        # one small weight: what the norm costs as a launch, not as a read
        dict(name="norm_small", kind="norm", count=1, lo=256, hi=384, types="f32", order=0, max_norm=1.0, write=False),
        # all gradients of a ragged model, half of them bf16, clipped into the float32 buffers the step reads
        dict(name="norm_clip_ragged", kind="norm", count=40, lo=129, hi=4200, types="mixed", order=3, max_norm=1.0, write=True),
        # one layer of the dense model on one rank: norm of the shard, then the step that clips as it reads
        dict(name="clip_step_layer", kind="step", hidden=4096, inner=11008, layers=1, max_norm=1.0),
        # a vector-sized model part: the clipped step where launches count
        dict(name="clip_step_small", kind="step", hidden=512, inner=1000, layers=2, max_norm=0.5),
        # generation reads one row of a FP8 table
        dict(name="embed_one", kind="embed", tokens=1, vocab=32768, dim=4096, table="fp8", out="bf16", scaled=True),
        # a training batch reads its rows of a FP8 table
        dict(name="embed_batch", kind="embed", tokens=32768, vocab=131072, dim=4096, table="fp8", out="bf16", scaled=True),
        # a small batch adds its rows onto the gradient that the tied head left there
        dict(name="embed_grad_tied", kind="embed_grad", tokens=3001, vocab=50001, dim=1000, dout="f32", add=True),
        # the gradient of a whole table from a training batch, rows without a token included
        dict(name="embed_grad_batch", kind="embed_grad", tokens=32768, vocab=131072, dim=4096, dout="bf16", add=False),
        # one scored token: the head's weights are read once
        dict(name="loss_one", kind="loss", tokens=1, vocab=32768, dim=4096, weight="fp8", grad=False),
        # scoring a prompt, without gradients
        dict(name="loss_prompt", kind="loss", tokens=2048, vocab=131072, dim=4096, weight="fp8", grad=False),
        # odd sizes, bf16 weights, loss and gradients
        dict(name="loss_grad_odd", kind="loss", tokens=1013, vocab=50001, dim=1000, weight="bf16", grad=True),
        # a training microbatch on the FP8 head, loss and gradients
        dict(name="loss_grad_batch", kind="loss", tokens=8192, vocab=131072, dim=4096, weight="fp8", grad=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "step", "embed", "embed_grad", "loss", "loss"])
    if kind == "norm":
        lo = _spread(rng, 16, 1000)
        return dict(kind=kind, count=_spread(rng, 1, 300), lo=lo, hi=_spread(rng, lo, 4000), types=rng.choice(["f32", "bf16", "mixed"]),
                    order=rng.randrange(1 << 20), max_norm=rng.choice([0.1, 1.0, 1e6]), write=rng.random() < 0.5)
    if kind == "step":
        return dict(kind=kind, hidden=_spread(rng, 100, 4096), inner=_spread(rng, 100, 11008), layers=1, max_norm=rng.choice([0.1, 1.0, 1e6]))
    dim = _spread(rng, 64, 4096) if rng.random() < 0.5 else 64 * _spread(rng, 1, 64)
    vocab = _spread(rng, 1000, 131072)
    if kind == "embed":
        return dict(kind=kind, tokens=_spread(rng, 1, 32768), vocab=vocab, dim=dim, table=rng.choice(["fp8", "bf16", "f32"]),
                    out=rng.choice(["bf16", "f16", "f32"]), scaled=rng.random() < 0.7)
    if kind == "embed_grad":
        return dict(kind=kind, tokens=_spread(rng, 1, 32768), vocab=vocab, dim=dim, dout=rng.choice(["bf16", "f32"]), add=rng.random() < 0.5)
    return dict(kind=kind, tokens=_spread(rng, 1, 4096), vocab=vocab, dim=dim, weight=rng.choice(["fp8", "bf16"]), grad=rng.random() < 0.6)


# ---- inputs ------------------------------------------------------------------


def _tensors(c):
    """(rows, cols, type) of each gradient of a norm case."""
    r = random.Random(c["order"])
    out = []
    for k in range(c["count"]):
        h, w = (c["lo"], c["hi"]) if c["count"] == 1 else (_spread(r, c["lo"], c["hi"]), _spread(r, c["lo"], c["hi"]))
        if k % 7 == 6:
            w = 1  # a norm's or a bias's vector
        out.append((h, w, ("f32" if k % 2 else "bf16") if c["types"] == "mixed" else c["types"]))
    return out


def _dims(c):
    return ([(1, c["hidden"], c["hidden"])] * 4 + [(1, c["hidden"], c["inner"])] * 2 + [(1, c["inner"], c["hidden"])]) * c["layers"]


def _normal(shape, gen, std, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(dtype)


def _ids(n, vocab, gen, ignored):
    """Token ids as text has them (the k-th most frequent about 1/k as often
    as the first), a few of them -1: padding, or a target left out."""
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    ids = ((vocab + 1.0) ** u).to(torch.int64).sub_(1).clamp_(0, vocab - 1)
    ids = (ids * 7919 + 13) % vocab  # frequent ids lie anywhere in the table
    return torch.where(torch.rand(n, generator=gen, device="cuda") < ignored, -1, ids)


def _fp8_weight(rows, cols, gen, std):
    """E4M3 codes and tile scales of a normal weight, one scale per tile."""
    hb, wb = -(-rows // T), -(-cols // T)
    grid = torch.rand((hb, wb), generator=gen, device="cuda") * 0.5 + 0.75
    grid = grid * (std * 4.5 / 448)
    up = grid.repeat_interleave(T, 1)[:, :cols].contiguous()
    codes = torch.empty((rows, cols), dtype=torch.uint8, device="cuda")
    step = 8192
    for r0 in range(0, rows, step):
        r1 = min(rows, r0 + step)
        w = _normal((r1 - r0, cols), gen, std) / up[r0 // T:-(-r1 // T)].repeat_interleave(T, 0)[:r1 - r0]
        codes[r0:r1] = w.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, grid


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case=c)
    if c["kind"] == "norm":
        s["grads"] = [_normal((h, w), gen, 1e-3, TYPES[t]) for h, w, t in _tensors(c)]
        if c["write"]:  # one flat float32 buffer, each gradient on a 256-byte boundary of it
            at = np.cumsum([0] + [-(-g.numel() // 64) * 64 for g in s["grads"]])
            s["flat"] = torch.zeros(int(at[-1]), device="cuda")
            s["outs"] = [s["flat"][a:a + g.numel()].view(g.shape) for a, g in zip(at.tolist(), s["grads"])]
        s["norm"], s["coef"] = (torch.empty(1, device="cuda") for _ in range(2))
    elif c["kind"] == "step":
        dims = _dims(c)
        q = sum(E * (-(-H // T)) * (-(-W // T)) for E, H, W in dims)
        s["dims"], s["q"] = dims, q
        s["grads"] = [_normal(d, gen, 1e-3) for d in dims]
        stride = 3 * TILE + 1024  # [master | m | v] of a tile and a gap
        s["state"] = torch.zeros((q, stride), device="cuda")
        s["master"], s["m"], s["v"] = (s["state"][:, k * TILE:(k + 1) * TILE] for k in range(3))
        s["master"].copy_(_tiles([_normal(d, gen, 0.02) for d in dims]))
        s["m"].copy_(_tiles([_normal(d, gen, 1e-3) for d in dims]))
        s["v"].copy_(_tiles([_normal(d, gen, 1e-3).square_() for d in dims]))
        s["codes"] = torch.empty(q * TILE, dtype=torch.uint8, device="cuda")
        s["scale_inv"] = torch.empty(q, device="cuda")
        s["fp8"] = [torch.zeros(d, dtype=torch.uint8, device="cuda") for d in dims]
        s["grid"] = [torch.zeros((E, -(-H // T), -(-W // T)), device="cuda") for E, H, W in dims]
        s["norm"], s["coef"] = (torch.empty(1, device="cuda") for _ in range(2))
    elif c["kind"] == "embed":
        s["ids"] = _ids(c["tokens"], c["vocab"], gen, 0.01 if c["tokens"] > 100 else 0.0)
        if c["table"] == "fp8":
            s["table"], s["grid"] = _fp8_weight(c["vocab"], c["dim"], gen, 0.02)
        else:
            s["table"], s["grid"] = _normal((c["vocab"], c["dim"]), gen, 0.02, TYPES[c["table"]]), None
        s["scale"] = math.sqrt(c["dim"]) if c["scaled"] else 1.0
        s["out"] = torch.empty((c["tokens"], c["dim"]), dtype=TYPES[c["out"]], device="cuda")
    elif c["kind"] == "embed_grad":
        s["ids"] = _ids(c["tokens"], c["vocab"], gen, 0.01 if c["tokens"] > 100 else 0.0)
        s["dout"] = _normal((c["tokens"], c["dim"]), gen, 1e-3, TYPES[c["dout"]])
        s["scale"] = math.sqrt(c["dim"])
        s["dtable"] = _normal((c["vocab"], c["dim"]), gen, 1e-2) if c["add"] else torch.empty((c["vocab"], c["dim"]), device="cuda")
    else:
        s["hidden"] = _normal((c["tokens"], c["dim"]), gen, 1.0, torch.bfloat16)
        s["targets"] = _ids(c["tokens"], c["vocab"], gen, 0.02 if c["tokens"] > 100 else 0.0)
        std = 1.3 / math.sqrt(c["dim"])  # logits of a spread that trained heads have
        if c["weight"] == "fp8":
            s["weight"], s["grid"] = _fp8_weight(c["vocab"], c["dim"], gen, std)
        else:
            s["weight"], s["grid"] = _normal((c["vocab"], c["dim"]), gen, std, torch.bfloat16), None
        s["loss"], s["lse"] = (torch.empty(c["tokens"], device="cuda") for _ in range(2))
        if c["grad"]:
            s["dloss"] = torch.full((c["tokens"],), 1.0 / c["tokens"], device="cuda")
            s["dhidden"] = torch.empty_like(s["hidden"])
            s["dweight"] = torch.empty((c["vocab"], c["dim"]), dtype=torch.bfloat16, device="cuda")
    if own:
        import blockwise_fp8_zero_amd as bfz
        s["bfz"] = bfz
        if c["kind"] in ("norm", "step"):
            s["work"] = bfz.norm_workspace()
        if c["kind"] == "step":
            s["plan"] = bfz.Plan(s["dims"])
            s["hp"] = bfz.AdamW(step=STEP, **HP)
        if c["kind"] == "embed_grad":
            s["work"] = bfz.embed_grad_workspace(c["tokens"], c["dim"])
        if c["kind"] == "loss":
            s["work"] = bfz.vocab_loss_workspace(c["tokens"], c["vocab"], c["dim"], weight_dtype=s["weight"].dtype, grad=c["grad"])
    return s


# ---- one pass ----------------------------------------------------------------


def run(s):
    kind = s["case"]["kind"]
    return (OWN if own else PLAIN)[kind](s)


def _own_norm(s):
    bfz, c = s["bfz"], s["case"]
    bfz.grad_norm(s["grads"], s["norm"], s["work"], max_norm=c["max_norm"], coef=s["coef"])
    if not c["write"]:
        return s["norm"], s["coef"]
    bfz.clip_grads(s["grads"], s["coef"], s["outs"])
    return s["norm"], s["coef"], s["flat"]


def _own_step(s):
    bfz = s["bfz"]
    bfz.shard_grad_norm(s["plan"], s["grads"], s["norm"], s["work"], max_norm=s["case"]["max_norm"], coef=s["coef"])
    bfz.fold_adamw_fp8_step_unpack(s["plan"], s["grads"], s["master"], s["m"], s["v"], s["codes"], s["scale_inv"], s["fp8"], s["grid"],
                                   s["hp"], grad_scale=s["coef"])
    return _step_out(s)


def _own_embed(s):
    s["bfz"].embed(s["ids"], s["table"], s["out"], scale=s["scale"], grid=s["grid"])
    return s["out"]


def _own_embed_grad(s):
    s["bfz"].embed_grad(s["ids"], s["dout"], s["dtable"], s["work"], scale=s["scale"], accumulate=s["case"]["add"])
    return s["dtable"]


def _own_loss(s):
    bfz = s["bfz"]
    bfz.vocab_loss(s["hidden"], s["weight"], s["targets"], s["loss"], s["lse"], s["work"], grid=s["grid"])
    if not s["case"]["grad"]:
        return s["loss"], s["lse"]
    bfz.vocab_loss_grad(s["hidden"], s["weight"], s["targets"], s["lse"], s["dloss"], s["dhidden"], s["dweight"], s["work"], grid=s["grid"])
    return s["loss"], s["lse"], s["dhidden"], s["dweight"]


def _step_out(s):
    return dict(norm=s["norm"], coef=s["coef"], master=s["master"], m=s["m"], v=s["v"], codes=s["codes"].view(torch.float8_e4m3fn),
                scale_inv=s["scale_inv"], fp8=[x.view(torch.float8_e4m3fn) for x in s["fp8"]], grid=s["grid"])


OWN = dict(norm=_own_norm, step=_own_step, embed=_own_embed, embed_grad=_own_embed_grad, loss=_own_loss)


def _tiles(weights):
    """(tiles, 16384): the weights' 128x128 tiles, zero padded, in the order
    (weight, expert, tile row, tile column)."""
    def one(w):
        E, H, W = w.shape
        w = torch.nn.functional.pad(w, (0, -W % T, 0, -H % T))
        return w.view(E, -(-H // T), T, -(-W // T), T).transpose(2, 3).reshape(-1, TILE)
    return torch.cat([one(w) for w in weights])


def _untile(tiles, dims):
    n = np.cumsum([0] + [E * (-(-H // T)) * (-(-W // T)) for E, H, W in dims]).tolist()
    return [tiles[a:b].view(E, -(-H // T), -(-W // T), T, T).transpose(2, 3).reshape(E, -(-H // T) * T, -(-W // T) * T)[:, :H, :W]
            for a, b, (E, H, W) in zip(n, n[1:], dims)]


def _norm_and_coef(grads, max_norm):
    norm = torch.stack([g.double().square().sum() for g in grads]).sum().sqrt().view(1)
    return norm, (max_norm / (norm + 1e-6)).clamp(max=1.0)


def _plain_norm(s):
    norm, coef = _norm_and_coef(s["grads"], s["case"]["max_norm"])
    s["norm"].copy_(norm)
    s["coef"].copy_(coef)
    if not s["case"]["write"]:
        return s["norm"], s["coef"]
    [o.copy_(g.float() * s["coef"]) for o, g in zip(s["outs"], s["grads"])]
    return s["norm"], s["coef"], s["flat"]


def _plain_step(s):
    norm, coef = _norm_and_coef(s["grads"], s["case"]["max_norm"])
    s["norm"].copy_(norm)
    s["coef"].copy_(coef)
    b1, b2, lr = HP["beta1"], HP["beta2"], HP["lr"]
    g = _tiles(s["grads"]) * s["coef"]
    m = s["m"] * b1 + g * (1 - b1)
    v = s["v"] * b2 + (g * g) * (1 - b2)
    den = v.sqrt() / math.sqrt(1 - b2 ** STEP) + HP["eps"]
    p = s["master"] - (m / den) * (lr / (1 - b1 ** STEP))
    p = p - p * (lr * HP["weight_decay"])
    s["master"].copy_(p)
    s["m"].copy_(m)
    s["v"].copy_(v)
    amax = p.abs().amax(1)
    scale = torch.where(amax == 0, torch.ones_like(amax), amax / 448.0)
    s["scale_inv"].copy_(scale)
    codes = (p / scale[:, None]).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    s["codes"].copy_(codes.view(-1))
    [d.copy_(x) for d, x in zip(s["fp8"], _untile(codes, s["dims"]))]
    n = np.cumsum([0] + [x.numel() for x in s["grid"]]).tolist()
    [d.copy_(scale[a:b].view(d.shape)) for d, a, b in zip(s["grid"], n, n[1:])]
    return _step_out(s)


def _plain_embed(s):
    ids, table = s["ids"], s["table"]
    row = ids.clamp(min=0)
    x = table[row]
    if s["grid"] is not None:
        x = x.view(torch.float8_e4m3fn).float() * s["grid"][row // T].repeat_interleave(T, 1)[:, :table.shape[1]]
    x = torch.where((ids >= 0)[:, None], x.float() * s["scale"], 0.0)
    s["out"].copy_(x)
    return s["out"]


def _plain_embed_grad(s):
    ids, d = s["ids"], s["dtable"]
    if not s["case"]["add"]:
        d.zero_()
    x = torch.where((ids >= 0)[:, None], s["dout"].float() * s["scale"], 0.0)
    return d.index_add_(0, ids.clamp(min=0), x)


def _values(weight, grid):
    if grid is None:
        return weight.float()
    up = grid.repeat_interleave(T, 1)[:, :weight.shape[1]].repeat_interleave(T, 0)[:weight.shape[0]]
    return weight.view(torch.float8_e4m3fn).float() * up


def _plain_loss(s):
    h, w, t = s["hidden"].float(), _values(s["weight"], s["grid"]), s["targets"]
    kept, t = t >= 0, t.clamp(min=0)
    z = h @ w.t()
    top = z.amax(1, keepdim=True)
    lse = (z - top).exp_().sum(1).log() + top[:, 0]
    s["lse"].copy_(lse)
    s["loss"].copy_(torch.where(kept, lse - z.gather(1, t[:, None])[:, 0], 0.0))
    if not s["case"]["grad"]:
        return s["loss"], s["lse"]
    g = torch.where(kept, s["dloss"], 0.0)[:, None]
    dz = z.sub_(lse[:, None]).exp_().mul_(g)
    dz.scatter_add_(1, t[:, None], -g)
    s["dhidden"].copy_(dz @ w)
    s["dweight"].copy_(dz.t() @ h)
    return s["loss"], s["lse"], s["dhidden"], s["dweight"]


PLAIN = dict(norm=_plain_norm, step=_plain_step, embed=_plain_embed, embed_grad=_plain_embed_grad, loss=_plain_loss)


# ---- what a pass cannot do without --------------------------------------------


def _distinct(tokens, vocab):
    k = np.arange(vocab, dtype=np.float64)
    p = np.log((k + 2) / (k + 1)) / math.log(vocab + 1)
    return float((1 - (1 - p) ** tokens).sum())


def work(case):
    c = case
    if c["kind"] == "norm":
        n = sum(h * w for h, w, _ in _tensors(c))
        read = sum(h * w * SIZE[t] for h, w, t in _tensors(c))
        return dict(bytes=read + (4 * n if c["write"] else 0), flops=(3 if c["write"] else 2) * n)
    if c["kind"] == "step":
        n = sum(E * H * W for E, H, W in _dims(c))
        # gradient; master, m and v read and written; codes written in both orders
        return dict(bytes=n * (4 + 24 + 2), flops=20 * n)
    n, d, V = c["tokens"], c["dim"], c["vocab"]
    if c["kind"] == "embed":
        return dict(bytes=8 * n + _distinct(n, V) * d * SIZE[c["table"]] + n * d * SIZE[c["out"]], flops=n * d)
    if c["kind"] == "embed_grad":
        rows = _distinct(n, V) * 2 if c["add"] else V
        return dict(bytes=8 * n + n * d * SIZE[c["dout"]] + rows * d * 4, flops=n * d)
    weight = V * d * SIZE[c["weight"]] + (-(-V // T)) * (-(-d // T)) * 4 * (c["weight"] == "fp8")
    return dict(bytes=16 * n + 2 * n * d + weight + ((4 * n + 2 * n * d + 2 * V * d) if c["grad"] else 0), flops=(8 if c["grad"] else 2) * n * V * d)


# ---- the same from the definitions, in 64 bits ---------------------------------


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return EXACT[case["kind"]](s, case)


def _exact_norm(s, c):
    norm = math.sqrt(sum(float(torch.dot(x, x)) for x in (g.double().flatten() for g in s["grads"])))
    coef = min(1.0, c["max_norm"] / (norm + 1e-6))
    out = [np.array([norm]), np.array([coef])]
    if c["write"]:
        flat = s["flat"].double()
        at = 0
        for g in s["grads"]:
            flat[at:at + g.numel()] = g.double().flatten() * coef
            at += (g.numel() + 63) // 64 * 64
        out.append(flat)
    return tuple(out)


def _exact_step(s, c):
    norm = math.sqrt(sum(float((g.double() ** 2).sum()) for g in s["grads"]))
    coef = min(1.0, c["max_norm"] / (norm + 1e-6))
    b1, b2 = HP["beta1"], HP["beta2"]
    out = {k: torch.empty((s["q"], TILE), dtype=torch.float64, device="cuda") for k in ("master", "m", "v")}
    scale = torch.ones(s["q"], dtype=torch.float64, device="cuda")
    grids, slot = [], 0
    for (E, H, W), g in zip(s["dims"], s["grads"]):
        cells = torch.ones((E, (H + T - 1) // T, (W + T - 1) // T), dtype=torch.float64, device="cuda")
        for e in range(E):
            for i in range(cells.shape[1]):
                band = torch.zeros((T, cells.shape[2] * T), dtype=torch.float64, device="cuda")
                rows = g[e, i * T:(i + 1) * T]
                band[:rows.shape[0], :W] = rows.double() * coef
                at = slice(slot, slot + cells.shape[2])
                x = band.view(T, -1, T).permute(1, 0, 2).reshape(-1, TILE)
                m = b1 * s["m"][at].double() + (1 - b1) * x
                v = b2 * s["v"][at].double() + (1 - b2) * x * x
                mhat, vhat = m / (1 - b1 ** STEP), v / (1 - b2 ** STEP)
                p = s["master"][at].double() - HP["lr"] * mhat / (vhat.sqrt() + HP["eps"])
                p = p * (1 - HP["lr"] * HP["weight_decay"])
                top = p.abs().max(1).values
                cells[e, i] = torch.where(top > 0, top / 448, torch.ones_like(top))
                scale[at] = cells[e, i]
                out["master"][at], out["m"][at], out["v"][at] = p, m, v
                slot += cells.shape[2]
        grids.append(cells)
    return dict(norm=np.array([norm]), coef=np.array([coef]), codes=None, scale_inv=scale, fp8=[None] * len(grids), grid=grids, **out)


def _exact_weight(s, r0, r1):
    w = s["weight"] if "weight" in s else s["table"]
    if s["grid"] is None:
        return w[r0:r1].double()
    r = torch.arange(r0, r1, device="cuda") // T
    k = torch.arange(w.shape[1], device="cuda") // T
    return w[r0:r1].view(torch.float8_e4m3fn).to(torch.float64) * s["grid"].double()[r][:, k]


def _exact_embed(s, c):
    ids = s["ids"].cpu()
    out = torch.zeros((c["tokens"], c["dim"]), dtype=torch.float64, device="cuda")
    for r0 in range(0, c["vocab"], 16384):
        r1 = min(c["vocab"], r0 + 16384)
        at = torch.nonzero((ids >= r0) & (ids < r1))[:, 0]
        if len(at):
            out[at.cuda()] = s["scale"] * _exact_weight(s, r0, r1)[(ids[at] - r0).cuda()]
    return out


def _exact_embed_grad(s, c):
    d = s["dtable"].double() if c["add"] else torch.zeros((c["vocab"], c["dim"]), dtype=torch.float64, device="cuda")
    order = torch.argsort(s["ids"])
    ids, rows = s["ids"][order], s["dout"][order].double()
    ids, rows = ids[ids >= 0], rows[ids >= 0]
    rank = torch.arange(len(ids), device="cuda") - torch.searchsorted(ids, ids)  # the k-th of its token
    for k in range(0, int(rank.max()) + 1 if len(ids) else 0):
        pick = torch.nonzero(rank >= k)[:, 0] if k == 64 else torch.nonzero(rank == k)[:, 0]
        if k < 64:
            d[ids[pick]] += s["scale"] * rows[pick]
            continue
        for t in ids[pick].unique().tolist():  # what is left: a few frequent tokens
            d[t] += s["scale"] * rows[pick][ids[pick] == t].sum(0)
        break
    return d


def _exact_loss(s, c):
    n, V = c["tokens"], c["vocab"]
    w = _exact_weight(s, 0, V)
    loss, lse = (torch.zeros(n, dtype=torch.float64, device="cuda") for _ in range(2))
    dh = torch.zeros((n, c["dim"]), dtype=torch.float64, device="cuda")
    dw = torch.zeros((V, c["dim"]), dtype=torch.float64, device="cuda") if c["grad"] else None
    for a in range(0, n, 1024):
        h, t = s["hidden"][a:a + 1024].double(), s["targets"][a:a + 1024]
        z = h @ w.T
        lse[a:a + 1024] = torch.logsumexp(z, 1)
        kept = torch.nonzero(t >= 0)[:, 0]
        loss[a + kept] = lse[a + kept] - z[kept, t[kept]]
        if c["grad"]:
            p = torch.softmax(z, 1)
            p[kept, t[kept]] -= 1
            up = torch.zeros(len(t), dtype=torch.float64, device="cuda")
            up[kept] = s["dloss"][a + kept].double()
            p *= up[:, None]
            dh[a:a + 1024] = p @ w
            dw += p.T @ h
    return (loss, lse, dh, dw) if c["grad"] else (loss, lse)


EXACT = dict(norm=_exact_norm, step=_exact_step, embed=_exact_embed, embed_grad=_exact_embed_grad, loss=_exact_loss)
