"""Vocabulary cross entropy and its gradient on the GPU against the formulas in
64 bits, and the gradient against differences.

Tolerances, from the roundings (u = 2^-24):
  a logit is a binary32 sum of d products, rescaled d / 128 times:
      ez = (d + 2 d/128 + 4) u sum|h w|
  lse: the largest ez of the row, exponentials of arguments off by 2u|z - top|
      and 4u each, sums of at most 32 + slots/64 + 16 steps, the final log
  loss: that and the target's ez
  dz is rounded to bf16 (2^-8 of itself) after p's own error, then summed in
      binary32 over V (dh) or n (dw) terms, the output rounded once more."""
import sys

import pytest
import torch

import blockwise_fp8_zero_amd as bfz

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def _say(*a):
    print("[gpu-vocab-loss]", *a, flush=True)
    sys.stdout.flush()


def _weight(V, d, kind, std=None):
    std = std or 1.5 / d ** 0.5
    if kind == "bf16":
        w = (torch.randn(V, d, device="cuda") * std).to(torch.bfloat16)
        return w, None, w.double()
    codes = (torch.randn(V, d, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    grid = (torch.rand(-(-V // 128), -(-d // 128), device="cuda") + 0.5) * (std / 100)
    return codes.view(torch.uint8), grid, _value(codes, grid)


def _value(codes, grid):
    V, d = codes.shape
    up = grid.double().repeat_interleave(128, 0)[:V].repeat_interleave(128, 1)[:, :d]
    return codes.view(torch.float8_e4m3fn).to(torch.float64) * up


def _case(n, V, d, kind):
    torch.manual_seed(n + 7 * V + d)
    h = torch.randn(n, d, device="cuda").to(torch.bfloat16)
    w, grid, value = _weight(V, d, kind)
    t = torch.randint(0, V, (n,), device="cuda")
    if n > 4:
        t[1], t[3] = -100, V
    return h, w, grid, value, t


def _run(h, w, grid, t, dloss=None, dw_type=torch.bfloat16, base=None):
    n, d = h.shape
    V = w.shape[0]
    work = bfz.vocab_loss_workspace(n, V, d, weight_dtype=w.dtype, grad=dloss is not None)
    work.fill_(0xFF)  # NaN wherever something unwritten is read
    loss, lse = (torch.full((n,), float("nan"), device="cuda") for _ in range(2))
    bfz.vocab_loss(h, w, t, loss, lse, work, grid=grid)
    if dloss is None:
        return loss, lse
    work.fill_(0xFF)
    dh = torch.full((n, d), float("nan"), device="cuda").to(torch.bfloat16)
    dw = base.clone() if base is not None else torch.full((V, d), float("nan"), device="cuda").to(dw_type)
    bfz.vocab_loss_grad(h, w, t, lse, dloss, dh, dw, work, grid=grid, accumulate=base is not None)
    return loss, lse, dh, dw


def _check(h, value, t, got, dloss=None, base=None):
    n, d = h.shape
    V = value.shape[0]
    hd = h.double()
    z = hd @ value.t()
    ez = ((d + d / 64 + 4) * U * (hd.abs() @ value.abs().t())).amax(1)
    keep = (t >= 0) & (t < V)
    tt = t.clamp(0, V - 1).long()
    lse = torch.logsumexp(z, 1)
    loss = torch.where(keep, lse - z.gather(1, tt[:, None])[:, 0], 0.0)
    span = z.amax(1) - z.amin(1)
    steps = 32 + V / 32 / 64 + 16
    elog = ez + (4 * span + 8 + steps) * U + 4 * U * lse.abs()
    for name, a, b, e in (("lse", got[1], lse, elog), ("loss", got[0], loss, elog + ez + 2 * U * loss.abs())):
        bad = (a.double() - b).abs() > e
        assert not bool((bad | torch.isnan(a)).any()), (name, a[bad][:4], b[bad][:4], e[bad][:4])
    assert bool((got[0][~keep] == 0).all())
    if dloss is None:
        return
    up = torch.where(keep, dloss.double(), 0.0)
    dz = (z - lse[:, None]).exp() * up[:, None]
    ep = dz.abs() * (ez + elog + 8 * U)[:, None]  # of p, before the subtraction
    dz.scatter_add_(1, tt[:, None], -up[:, None])
    edz = 2.0 ** -8 * dz.abs() + 1.01 * ep + 2.0 ** -133
    for name, a, b, e, terms, adds in (("dh", got[2], dz @ value, edz @ value.abs(), V, dz.abs() @ value.abs()),
                                       ("dw", got[3], dz.t() @ hd, edz.t() @ hd.abs(), n, dz.abs().t() @ hd.abs())):
        e = e + (terms + V / 64) * U * adds
        if name == "dw" and base is not None:
            b = b + base.double()
        e = e + HALF[a.dtype] * (b.abs() + e) + 2.0 ** -133
        bad = (a.double() - b).abs() > e
        assert not bool((bad | torch.isnan(a)).any()), (name, int(bad.sum()), a[bad][:4], b[bad][:4], e[bad][:4])


SIZES = [(1, 1, 1), (1, 300, 64), (5, 257, 100), (7, 1000, 16), (64, 256, 128), (65, 1000, 72), (128, 511, 192), (129, 700, 130),
         (130, 513, 1000), (256, 1024, 256), (257, 3000, 320), (300, 9000, 64), (3, 40000, 48),
         (16, 5000, 200), (17, 600, 136), (15, 127, 520), (600, 2500, 512)]


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("n,V,d", SIZES)
def test_loss(n, V, d, kind):
    _say("loss", n, V, d, kind)
    h, w, grid, value, t = _case(n, V, d, kind)
    got = _run(h, w, grid, t)
    _check(h, value, t, got)
    again = _run(h, w, grid, t.int())
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("dw_type", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("n,V,d", SIZES)
def test_loss_grad(n, V, d, kind, dw_type):
    _say("grad", n, V, d, kind, dw_type)
    h, w, grid, value, t = _case(n, V, d, kind)
    dloss = torch.rand(n, device="cuda") + 0.1
    got = _run(h, w, grid, t, dloss, dw_type)
    _check(h, value, t, got, dloss)
    again = _run(h, w, grid, t, dloss, dw_type)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    base = torch.randn(V, d, device="cuda").to(dw_type)
    _check(h, value, t, _run(h, w, grid, t, dloss, dw_type, base), dloss, base)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_pieces(kind):
    """More rows than one piece holds, and a ragged last one."""
    n, V, d = 8200, 33333, 72
    _say("pieces", n, V, d, kind)
    h, w, grid, value, t = _case(n, V, d, kind)
    dloss = torch.full((n,), 1.0 / n, device="cuda")
    _check(h, value, t, _run(h, w, grid, t, dloss, torch.float32), dloss)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_strides_and_alignment(kind):
    torch.manual_seed(11)
    n, V, d = 70, 600, 128
    esize = 2 if kind == "bf16" else 1
    for hld, hoff, wld, woff in ((136, 0, 144, 16), (129, 0, 128, 0), (136, 3, 130, 0), (136, 8, 144, 5)):
        _say("strides", kind, hld, hoff, wld, woff)
        hb = torch.full((n * hld + 16,), float("nan"), device="cuda").to(torch.bfloat16)
        h = torch.as_strided(hb, (n, d), (hld, 1), hoff)
        h.copy_(torch.randn(n, d, device="cuda"))
        w0, grid, value = _weight(V, d, kind)
        wb = torch.full((V * wld + 32,), 0x7F, dtype=torch.uint8, device="cuda") if esize == 1 else \
            torch.full((V * wld + 32,), float("nan"), device="cuda").to(torch.bfloat16)
        w = torch.as_strided(wb, (V, d), (wld, 1), woff)
        w.copy_(w0)
        t = torch.randint(0, V, (n,), device="cuda")
        dloss = torch.rand(n, device="cuda")
        work = bfz.vocab_loss_workspace(n, V, d, weight_dtype=w.dtype)
        loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        bfz.vocab_loss(h, w, t, loss, lse, work, grid=grid)
        dhb = torch.full((n * 131 + 8,), 3.0, device="cuda").to(torch.bfloat16)
        dwb = torch.full((V * 133 + 8,), 3.0, device="cuda")
        dh, dw = torch.as_strided(dhb, (n, d), (131, 1), 1), torch.as_strided(dwb, (V, d), (133, 1), 2)
        bfz.vocab_loss_grad(h, w, t, lse, dloss, dh, dw, work, grid=grid)
        _check(h.contiguous(), value, t, (loss, lse, dh.contiguous(), dw.contiguous()), dloss)
        for buf, view in ((dhb, (n, d, 131, 1)), (dwb, (V, d, 133, 2))):
            rest = torch.ones_like(buf, dtype=torch.bool)
            torch.as_strided(rest, view[:2], (view[2], 1), view[3]).fill_(False)
            assert bool((buf[rest] == 3).all())


def test_uneven_tile_scales():
    """All-zero tiles (scale 1), tiny and subnormal scales, jumps both ways."""
    torch.manual_seed(12)
    n, V, d = 40, 700, 900
    h, codes, grid, _, t = _case(n, V, d, "fp8")
    grid[:, 1] = 1.0
    codes[:, 128:256] = 0
    grid[0, 2] = 2.0 ** -149
    grid[1, 0] = 1e-30
    grid[2, 3] *= 1e-6
    grid[3, 4] *= 30
    grid[4, :] = 2.0 ** -140
    value = _value(codes, grid)
    dloss = torch.rand(n, device="cuda")
    _check(h, value, t, _run(h, codes, grid, t, dloss), dloss)


def test_large_logits_and_nan():
    torch.manual_seed(13)
    n, V, d = 20, 500, 64
    h, w, grid, value, t = _case(n, V, d, "bf16")
    big = (w.float() * 200).to(torch.bfloat16)
    bigv = big.double()
    dloss = torch.ones(n, device="cuda")
    got = _run(h, big, None, t, dloss)
    assert bool(torch.isfinite(got[0]).all())
    _check(h, bigv, t, got, dloss)
    h[2, 5] = float("nan")  # spoils its own token only
    loss, lse = _run(h, w, None, t)
    rest = torch.arange(n, device="cuda") != 2
    assert bool(torch.isnan(lse[2])) and bool(torch.isfinite(lse[rest]).all())


def test_one_side_only_and_empty():
    h, w, grid, value, t = _case(50, 400, 96, "fp8")
    dloss = torch.rand(50, device="cuda")
    loss, lse, dh, dw = _run(h, w, grid, t, dloss)
    work = bfz.vocab_loss_workspace(50, 400, 96)
    dh2, dw2 = torch.zeros_like(dh), torch.zeros_like(dw)
    bfz.vocab_loss_grad(h, w, t, lse, dloss, dh2, None, work, grid=grid)
    bfz.vocab_loss_grad(h, w, t, lse, dloss, None, dw2, work, grid=grid)
    assert torch.equal(dh, dh2) and torch.equal(dw, dw2)
    empty = torch.zeros(0, device="cuda")
    bfz.vocab_loss(h[:0], w, t[:0], empty, empty, work, grid=grid)
    bfz.vocab_loss_grad(h[:0], w, t[:0], empty, empty, h[:0], dw2, work, grid=grid)
    assert bool((dw2 == 0).all())
    none = torch.full_like(t, -1)
    loss, lse, dh, dw = _run(h, w, grid, none, dloss)
    assert bool((loss == 0).all()) and bool((dh == 0).all()) and bool((dw == 0).all())


def test_a_workspace_serves_smaller_batches():
    V, d = 5000, 128
    h, w, grid, value, t = _case(2000, V, d, "fp8")
    dloss = torch.rand(2000, device="cuda")
    work = bfz.vocab_loss_workspace(2000, V, d)
    for n in (1, 16, 17, 300, 1999):
        want = _run(h[:n], w, grid, t[:n], dloss[:n])
        work.fill_(0xFF)
        loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        dh, dw = torch.empty_like(h[:n]), torch.empty(V, d, device="cuda", dtype=torch.bfloat16)
        bfz.vocab_loss(h[:n], w, t[:n], loss, lse, work, grid=grid)
        bfz.vocab_loss_grad(h[:n], w, t[:n], lse, dloss[:n], dh, dw, work, grid=grid)
        assert all(torch.equal(a, b) for a, b in zip(want, (loss, lse, dh, dw))), n


def test_gradient_against_differences():
    """(L(h + e x) - L(h - e x)) / 2e along random bf16-exact directions, in
    64 bits from the formula, against <dh, x> of the kernel: off by the
    gradient's own tolerance (2^-7 of sum|dh x|) and e^2 of curvature."""
    torch.manual_seed(14)
    n, V, d = 33, 777, 96
    h, w, grid, value, t = _case(n, V, d, "fp8")
    t = t.clamp(0, V - 1)
    dloss = torch.rand(n, device="cuda")
    _, _, dh, dw = _run(h, w, grid, t, dloss, torch.float32)

    def total(hh, ww):
        z = hh @ ww.t()
        return float((dloss.double() * (torch.logsumexp(z, 1) - z.gather(1, t[:, None])[:, 0])).sum())

    hd, e = h.double(), 1e-4
    for k in range(3):
        x, y = torch.randn_like(hd), torch.randn_like(value) * 0.1
        for a, b, g in ((lambda q: total(hd + q * x, value), dh, x), (lambda q: total(hd, value + q * y), dw, y)):
            diff = (a(e) - a(-e)) / (2 * e)
            want = float((b.double() * g).sum())
            lim = 2.0 ** -7 * float((b.double() * g).norm()) * 4 + 1e-5
            assert abs(diff - want) <= lim, (k, diff, want, lim)


def test_past_32_bits():
    """Weight and gradient offsets past 2^32 elements."""
    V, d, n = 1_060_000, 4096, 2
    _say("past 32 bits")
    codes = torch.zeros(V, d, dtype=torch.uint8, device="cuda")
    codes[V - 1].fill_(0x38)  # 1.0
    codes[5].fill_(0x30)      # 0.5
    grid = torch.full((-(-V // 128), d // 128), 1.0, device="cuda")
    grid[-1] = 1.0 / 512
    grid[0] = 1.0 / 256
    h = torch.ones(n, d, device="cuda").to(torch.bfloat16)
    t = torch.tensor([V - 1, 5], device="cuda")
    dloss = torch.ones(n, device="cuda")
    loss, lse, dh, dw = _run(h, codes, grid, t, dloss)
    # z: 8 at both rows, 0 at the other V - 2
    want = float(torch.log(torch.tensor(2 * torch.e ** 8 + V - 2, dtype=torch.float64)))
    assert float((lse.double() - want).abs().max()) < 1e-5 and float((loss.double() - (want - 8)).abs().max()) < 1e-5
    p = torch.e ** (8 - want)
    for row, expect in ((V - 1, 2 * p - 1), (5, 2 * p - 1), (V - 2, 2 * torch.e ** -want), (600_000, 2 * torch.e ** -want)):
        got = dw[row].double()
        assert float((got - expect).abs().max()) <= 3 * 2.0 ** -8 * abs(expect) + 2.0 ** -8 * p, (row, got[:3], expect)
    del dw
    torch.cuda.empty_cache()


def test_in_a_graph_and_on_a_side_stream():
    torch.manual_seed(15)
    n, V, d = 200, 3000, 256
    h, w, grid, value, t = _case(n, V, d, "fp8")
    dloss = torch.rand(n, device="cuda")
    work = bfz.vocab_loss_workspace(n, V, d)
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    dh, dw = torch.empty_like(h), torch.empty(V, d, device="cuda")
    outs = [loss, lse, dh, dw]

    def step():
        bfz.vocab_loss(h, w, t, loss, lse, work, grid=grid)
        bfz.vocab_loss_grad(h, w, t, lse, dloss, dh, dw, work, grid=grid)

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    for k in range(4):
        h.copy_(torch.randn(n, d, device="cuda"))
        step()
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), k
