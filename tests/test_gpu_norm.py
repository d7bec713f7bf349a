"""Gradient norm and clipping on the GPU: against 64-bit sums, bit for bit
between runs, and inside the step against a step on clipped gradients.

Tolerances: sumsq is a binary64 sum of n exact squares in a tree, off by at
most (log2(n) + chunk depth) half steps of 2^-53 -- 1e-12 is above it for
every n here; norm and coef are that rounded once to binary32 (2^-24) after a
binary64 square root and division."""
import math
import sys

import numpy as np
import pytest
import torch

import blockwise_fp8_zero_amd as bfz

pytestmark = pytest.mark.gpu
F32 = 2.0 ** -24 * 1.01


def _say(*a):
    print("[gpu-norm]", *a, flush=True)
    sys.stdout.flush()


def _one(v=float("nan"), dtype=torch.float32):
    return torch.full((1,), v, dtype=dtype, device="cuda")


def _norm(grads, max_norm=1.0, work=None):
    norm, coef, sumsq = _one(), _one(), _one(dtype=torch.float64)
    bfz.grad_norm(grads, norm, bfz.norm_workspace() if work is None else work, max_norm=max_norm, coef=coef, sumsq=sumsq)
    return norm.item(), coef.item(), sumsq.item()


def _want(grads, max_norm=1.0):
    s = math.fsum(float(np.sum(g.double().cpu().numpy().ravel() ** 2)) for g in grads)
    n = math.sqrt(s)
    return n, min(1.0, max_norm / (n + 1e-6)), s


def _check(got, want):
    assert abs(got[2] - want[2]) <= 1e-12 * want[2], (got, want)
    for g, w in zip(got[:2], want[:2]):
        assert abs(g - w) <= F32 * abs(w) + 1e-45, (got, want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", [1, 2, 7, 255, 4095, 4097, 65537, 1000003])
def test_norm_of_one_tensor(n, dtype):
    _say(n, dtype)
    torch.manual_seed(n)
    x = (torch.randn(n + 9, device="cuda") * 0.3).to(dtype)
    for off in (0, 1, 3, 5):
        g = [x[off:off + n]]
        _check(_norm(g, 0.25), _want(g, 0.25))


@pytest.mark.parametrize("count", [0, 1, 95, 96, 97, 193])
def test_norm_of_lists(count):
    _say("list of", count)
    rng = np.random.default_rng(count)
    types = [torch.float32, torch.bfloat16, torch.float16]
    grads = [(torch.randn(int(rng.integers(0, 6000)), device="cuda")).to(types[k % 3]) for k in range(count)]
    work = bfz.norm_workspace()
    got = _norm(grads, 3.0, work)
    if count == 0:
        assert got == (0.0, 1.0, 0.0)
        return
    _check(got, _want(grads, 3.0))
    assert got == _norm(grads, 3.0, work)  # the workspace comes back as it was, the bits too
    _check(_norm([g.view(-1) for g in grads] + [torch.empty(0, device="cuda")], None, work)[:1] + (1.0,) + got[2:],
           _want(grads, math.inf))


def test_norm_of_a_long_list_element():
    """More chunks than workgroups: a workgroup walks several."""
    g = [torch.full((90_000_001,), 1e-3, device="cuda"), torch.full((70_000_003,), -2.0, dtype=torch.bfloat16, device="cuda")]
    x = float(torch.tensor(1e-3, dtype=torch.float32))
    want = 90_000_001 * x * x + 70_000_003 * 4.0
    got = _norm(g, 1.0)
    assert abs(got[2] - want) <= 1e-12 * want
    assert got == _norm(g, 1.0)


def test_norm_range_and_specials():
    big = [torch.full((1000,), 2.0 ** 100, device="cuda")]
    _check(_norm(big), _want(big))
    small = [torch.full((1000,), 2.0 ** -130, device="cuda")]  # subnormal binary32
    got, want = _norm(small), _want(small)
    assert abs(got[2] - want[2]) <= 1e-12 * want[2] and got[1] == 1.0
    x = torch.randn(5000, device="cuda")
    x[4321] = float("inf")
    assert _norm([x])[:2] == (float("inf"), 0.0)
    x[17] = float("nan")
    assert all(math.isnan(v) for v in _norm([x]))
    z = [torch.zeros(300, device="cuda")]
    assert _norm(z) == (0.0, 1.0, 0.0)


def test_masked_ends_do_not_leak():
    """NaN right before and after an unaligned range is not read into it."""
    x = torch.full((5003,), float("nan"), device="cuda")
    x[3:5001] = 0.5
    _check(_norm([x[3:5001]]), _want([x[3:5001]]))
    y = torch.full((5003,), float("nan"), dtype=torch.bfloat16, device="cuda")
    y[5:4998] = 0.5
    _check(_norm([y[5:4998]]), _want([y[5:4998]]))


@pytest.mark.parametrize("dims,D", [([(1, 256, 384)], 1), ([(2, 130, 257), (1, 129, 128), (1, 1, 1), (1, 300, 1000)], 3),
                                    ([(1, 40, 50 + k) for k in range(70)], 4), ([(1, 128, 128)], 5)])
def test_shard_norms_add_up(dims, D):
    _say(dims[:3], D)
    torch.manual_seed(1)
    for off in (0, 1):
        base = [torch.randn(E * H * W + 4, device="cuda") for E, H, W in dims]
        grads = [b[off:off + E * H * W] for b, (E, H, W) in zip(base, dims)]
        work, total = bfz.norm_workspace(), 0.0
        for rank in range(D):
            plan = bfz.Plan(dims, D, rank)
            s = _one(dtype=torch.float64)
            bfz.shard_grad_norm(plan, grads, None, work, sumsq=s)
            t = plan.table()
            want = 0.0
            for p, e, i, j, r, c in t[t[:, 0] >= 0]:
                E, H, W = dims[p]
                tile = grads[p].view(E, H, W)[e, 128 * i:128 * i + r, 128 * j:128 * j + c].double()
                want += float((tile * tile).sum())
            assert abs(s.item() - want) <= 1e-12 * want, (rank, s.item(), want)
            total += s.item()
        want = _want(grads, 2.0)
        assert abs(total - want[2]) <= 2e-12 * want[2]
        norm, coef = _one(), _one()
        bfz.clip_coef(_one(total, torch.float64), 2.0, norm, coef)
        _check((norm.item(), coef.item(), total), (want[0], want[1], total))


@pytest.mark.parametrize("src", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dst", [torch.float32, torch.bfloat16, torch.float16])
def test_clip_rounds_once(src, dst):
    torch.manual_seed(3)
    coef = _one(0.37)
    for n, off in ((1, 0), (1000, 0), (4096, 1), (70001, 3), (8191, 4)):
        g = (torch.randn(n + 8, device="cuda") * 2).to(src)[off:off + n]
        out = torch.full((n + 8,), -7.0, device="cuda").to(dst)
        bfz.clip_grads([g], coef, [out[off:off + n]])
        want = (g.float() * coef).to(dst)
        assert torch.equal(out[off:off + n], want), (n, off)
        assert bool((out[:off] == -7).all()) and bool((out[off + n:] == -7).all())


def test_clip_in_place_and_lists():
    torch.manual_seed(4)
    grads = [torch.randn(50 + 3 * k, device="cuda") for k in range(200)]
    want = [g * 0.5 for g in grads]
    bfz.clip_grads(grads, _one(0.5))
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
    bfz.clip_grads(grads, _one(1.0))
    assert all(torch.equal(a, b) for a, b in zip(grads, want))


@pytest.mark.parametrize("dims", [[(1, 256, 384)], [(2, 130, 257), (1, 129, 200), (1, 300, 1000)]])
def test_clipped_steps_match_steps_on_clipped_gradients(dims):
    _say("clipped steps", dims)
    torch.manual_seed(5)
    plan = bfz.Plan(dims)
    q = plan.shard_tiles
    coef = _one(0.123)
    grads = [torch.randn(d, device="cuda") for d in dims]
    clipped = [g * coef for g in grads]
    tiles, tiles_c = torch.zeros(q * 16384, device="cuda"), torch.zeros(q * 16384, device="cuda")
    bfz.pack_shard(plan, grads, tiles)
    bfz.pack_shard(plan, clipped, tiles_c)
    init = torch.randn(q * 16384, device="cuda")
    hp = bfz.AdamW(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=3)

    def run(kind, gs, tile_g, **kw):
        st = [torch.zeros(q * 16384, device="cuda") for _ in range(3)]
        bfz.pack_shard(plan, [init[:E * H * W].view(E, H, W) if E * H * W <= init.numel() else None for E, H, W in dims], st[0])
        codes = torch.zeros(q * 16384, dtype=torch.uint8, device="cuda")
        sc = torch.zeros(q, device="cuda")
        f8 = [torch.zeros(d, dtype=torch.uint8, device="cuda") for d in dims]
        gr = [torch.zeros(E, -(-H // 128), -(-W // 128), device="cuda") for E, H, W in dims]
        t8 = [torch.zeros(E, W, H, dtype=torch.uint8, device="cuda") for E, H, W in dims]
        tg = [torch.zeros(E, W, -(-H // 128), device="cuda") for E, H, W in dims]
        if kind == "tile":
            bfz.adamw_fp8_step(*st[:1], tile_g, *st[1:], codes, sc, hp, **kw)
        elif kind == "fold":
            bfz.fold_adamw_fp8_step(plan, gs, *st, codes, sc, hp, **kw)
        elif kind == "unpack":
            bfz.fold_adamw_fp8_step_unpack(plan, gs, *st, codes, sc, f8, gr, hp, **kw)
        else:
            bfz.fold_adamw_fp8_step_unpack_t(plan, gs, *st, codes, sc, f8, gr, t8, tg, hp, **kw)
        return st + [codes, sc] + f8 + gr + t8 + tg

    for kind in ("tile", "fold", "unpack", "t"):
        a = run(kind, grads, tiles, grad_scale=coef)
        b = run(kind, clipped, tiles_c)
        for k, (x, y) in enumerate(zip(a, b)):
            assert torch.equal(x, y), (kind, k)


def test_norm_and_clip_in_a_graph():
    torch.manual_seed(6)
    grads = [torch.randn(300, 500, device="cuda"), torch.randn(70001, device="cuda").to(torch.bfloat16)]
    outs = [torch.zeros(g.shape, device="cuda") for g in grads]
    norm, coef, work = _one(), _one(), bfz.norm_workspace()

    def step():
        bfz.grad_norm(grads, norm, work, max_norm=1.0, coef=coef)
        bfz.clip_grads(grads, coef, outs)

    step()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    for k in range(4):
        for g in grads:
            g.mul_(1.5)
        step()
        torch.cuda.synchronize()
        want = [norm.clone(), coef.clone()] + [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        norm.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, [norm, coef] + outs)), k
