"""AdamW over many tensors on the GPU.  Every operation is one binary32 rounding
in a stated order, so parameters and states have to equal the same operations
done in 64 bits and rounded to 32 after each (exact for +, -, *, /, sqrt:
rounding twice from 53 to 24 bits gives the one rounding), and codes and scales
the quantizer's definition."""
import math
import sys

import pytest
import torch

import blockwise_fp8_zero_amd as bfz

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
HP = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=3)


def _say(*a):
    print("[gpu-adamw-list]", *a, flush=True)
    sys.stdout.flush()


def r(x):
    """One rounding to binary32."""
    return x.float().double()


def f32(x):
    return float(torch.tensor(x, dtype=torch.float64).float())


def blocks(x, n):
    pad = torch.zeros(-(-n // 256) * 256, dtype=torch.float64, device=x.device)
    pad[:n] = x
    return pad.view(-1, 256)


def encode(x, positive):
    """Codes and scales of a vector (float64 of binary32 values)."""
    n = x.numel()
    b = blocks(x, n)
    top = b.abs().amax(1)
    s = (top / 448).float().double()
    s = torch.where(s == 0, torch.full_like(s, 2.0 ** -149), s)
    s = torch.where(top == 0, torch.ones_like(s), s)
    c = (b / s[:, None]).float().clamp(-448, 448).to(E4M3).view(torch.uint8)
    if positive:
        c = torch.where((b > 0) & (c == 0), torch.ones_like(c), c)
    return c.reshape(-1)[:n], s.float()


def decode(codes, scale):
    n = codes.numel()
    return r(codes.view(-1).contiguous().view(E4M3).to(torch.float64) * scale.double().repeat_interleave(256)[:n])


def want(p, g, m, v, hp, factor=None):
    """p', m', sqrt(v'), v' of vectors in float64 of binary32 values."""
    b1, b2, t = hp["beta1"], hp["beta2"], hp["step"]
    g = g.double()
    if factor is not None:
        g = r(g * factor)
    m = r(r(f32(b1) * m) + r(f32(1 - b1) * g))
    v = r(r(f32(b2) * v) + r(f32(1 - b2) * r(g * g)))
    root = r(v.sqrt())
    den = r(r(root / f32(math.sqrt(1 - b2 ** t))) + f32(hp["eps"]))
    p = r(p.double() - r(f32(hp["lr"] / (1 - b1 ** t)) * r(m / den)))
    if hp["weight_decay"] != 0:
        p = r(p - r(f32(hp["lr"] * hp["weight_decay"]) * p))
    return p, m, root, v


def _tensors(sizes, param, grad, bits, gen):
    def normal(n, std):
        return torch.randn(n, generator=gen, device="cuda") * std

    params = [normal(n, 0.02).to(param) for n in sizes]
    grads = [normal(n, 1e-3).to(g) for n, g in zip(sizes, grad)]
    m, v, ms, vs = bfz.adamw_states(params, bits)
    for k, n in enumerate(sizes):
        a, b = normal(n, 3e-4), normal(n, 1e-3).abs()
        if bits == 32:
            m[k].copy_(a)
            v[k].copy_(b * b)
        else:
            for codes, scale, x, positive in ((m, ms, a, False), (v, vs, b, True)):
                c, s = encode(x.double(), positive)
                codes[k].copy_(c)
                scale[k].copy_(s)
    return params, grads, m, v, ms, vs


def _check(params, before, grads, hp, bits, m, v, ms, vs, factor=None):
    for k, p in enumerate(params):
        p0, m0, v0, ms0, vs0 = before[k]
        if bits == 8:
            m0, v0 = decode(m0, ms0), decode(v0, vs0)
            v0 = r(v0 * v0)
        wp, wm, wr, wv = want(p0.view(-1), grads[k].view(-1), m0.double().view(-1), v0.double().view(-1), hp, factor)
        assert torch.equal(p.view(-1), wp.to(p.dtype)), k
        if bits == 32:
            assert torch.equal(m[k].view(-1).double(), wm) and torch.equal(v[k].view(-1).double(), wv), k
        else:
            for codes, scale, x, positive in ((m, ms, wm, False), (v, vs, wr, True)):
                c, s = encode(x, positive)
                assert torch.equal(scale[k], s) and torch.equal(codes[k].view(-1), c), (k, positive)


def _copies(params, m, v, ms, vs):
    return [tuple(None if z is None else z.clone() for z in zs) for zs in zip(params, m, v, ms, vs)]


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("param", [F32, BF16, F16])
@pytest.mark.parametrize("sizes", [[1], [256], [257, 1, 0, 4095, 4097], [5000] * 130 + [3, 100000]])
def test_steps(bits, param, sizes):
    _say(bits, param, len(sizes))
    gen = torch.Generator(device="cuda").manual_seed(len(sizes) + bits)
    grad = [(F32, BF16, F16)[k % 3] for k in range(len(sizes))]
    params, grads, m, v, ms, vs = _tensors(sizes, param, grad, bits, gen)
    opt = bfz.AdamWList(params, m, v, ms, vs, grads=grads)
    factor = torch.full((1,), 0.37, device="cuda")
    for step, scale in ((3, None), (4, factor)):
        hp = dict(HP, step=step, weight_decay=0.1 if scale is None else 0.0)
        before = _copies(params, m, v, ms, vs)
        opt.step(hp, grad_scale=scale)
        _check(params, before, grads, hp, bits, m, v, ms, vs, None if scale is None else float(factor))


@pytest.mark.parametrize("bits", [8, 32])
def test_alignment_and_neighbours(bits):
    """Tensors at any element of larger buffers; the elements between them stay."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    sizes, at = [700, 300, 4100, 9], [1, 704, 1009, 5200]
    plain = _tensors(sizes, F32, [F32, BF16, F32, F16], bits, gen)
    bufs = [torch.full((6000,), 7, dtype=plain[j][0].dtype, device="cuda") for j in (0, 2, 3)]
    params, m, v = ([b[a:a + n] for a, n in zip(at, sizes)] for b in bufs)
    for views, values in zip((params, m, v), (plain[0], plain[2], plain[3])):
        [a.copy_(b) for a, b in zip(views, values)]
    grads, ms, vs = plain[1], plain[4], plain[5]
    before = _copies(params, m, v, ms, vs)
    bfz.AdamWList(params, m, v, ms, vs).step(HP, grads=grads)
    _check(params, before, grads, HP, bits, m, v, ms, vs)
    for b in bufs:
        for a, n in zip(at, sizes):
            b[a:a + n] = 7
        assert bool((b == 7).all())


def test_extremes_of_states():
    """Blocks of zeros, of subnormal and of huge moments, a root far below its
    block's largest; a NaN gradient stays in its element."""
    n = 256 * 7
    p = torch.zeros(n, device="cuda")
    g = torch.zeros(n, device="cuda")
    g[256:512] = torch.randn(256, device="cuda") * 1e-22    # g g underflows
    g[512:768] = torch.randn(256, device="cuda") * 1e18
    g[768:1024] = 1e-9
    g[800] = 1.0                                            # all others far below it
    g[1024:1280] = torch.randn(256, device="cuda") * 1e-38
    g[1280:] = torch.randn(n - 1280, device="cuda")
    m, v, ms, vs = bfz.adamw_states([p], bits=8)
    hp = dict(HP, step=1)
    before = _copies([p], m, v, ms, vs)
    opt = bfz.AdamWList([p], m, v, ms, vs)
    opt.step(hp, grads=[g])
    _check([p], before, [g], hp, 8, m, v, ms, vs)
    assert bool((v[0][768:1024] > 0).all())  # no positive root became zero
    g2 = g.clone()
    g2[1300] = float("nan")
    before = _copies([p], m, v, ms, vs)
    twin = [z.clone() for z in (p, m[0], v[0], ms[0], vs[0])]
    bfz.AdamWList([twin[0]], [twin[1]], [twin[2]], [twin[3]], [twin[4]]).step(dict(hp, step=2), grads=[g2])
    opt.step(dict(hp, step=2), grads=[g])
    assert bool(twin[0][1300].isnan()) and int(twin[0].isnan().sum()) == 1
    far = torch.ones(n, dtype=torch.bool, device="cuda")
    far[1280:1536] = False
    assert torch.equal(twin[0][far], p[far]) and torch.equal(twin[1][far], m[0][far]) and torch.equal(twin[2][far], v[0][far])
    assert int(twin[1].view(E4M3).float().isnan().sum()) == 1


@pytest.mark.parametrize("bits", [8, 32])
def test_graph_stream_and_repeats(bits):
    gen = torch.Generator(device="cuda").manual_seed(6)
    sizes = [4096] * 60 + [12345]
    params, grads, m, v, ms, vs = _tensors(sizes, F32, [BF16] * 61, bits, gen)
    opt = bfz.AdamWList(params, m, v, ms, vs, grads=grads)
    factor = torch.full((1,), 0.5, device="cuda")
    hp = bfz.AdamW(**HP)
    state = [z for zs in (params, m, v, ms, vs) for z in zs if z is not None]
    start = [z.clone() for z in state]

    def reset():
        [a.copy_(b) for a, b in zip(state, start)]

    opt.step(hp, grad_scale=factor)
    first = [z.clone() for z in state]
    side = torch.cuda.Stream()
    reset()
    side.wait_stream(torch.cuda.current_stream())
    opt.step(hp, grad_scale=factor, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, state))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(hp, grad_scale=factor)
    for _ in range(3):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, state))


def test_matches_the_fp8_step():
    """On whole tiles the update is the one of adamw_fp8_step, bit for bit."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    n = 3 * 16384
    (p,), (g,), (m,), (v,), _, _ = _tensors([n], F32, [F32], 32, gen)
    master, mm, vv = p.clone(), m.clone(), v.clone()
    codes, scale = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty(3, device="cuda")
    bfz.adamw_fp8_step(master, g, mm, vv, codes, scale, HP)
    bfz.AdamWList([p], [m], [v], grads=[g]).step(HP)
    assert torch.equal(p, master) and torch.equal(m, mm) and torch.equal(v, vv)
