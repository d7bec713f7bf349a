"""Token embedding and its gradient on the GPU against 64-bit references.

Tolerances: a looked-up value passes two binary32 roundings (scale * tile
scale, then the product) and one to its own type; a gradient of c terms is a
binary32 sum, off by at most c * 2^-24 of the terms' absolute sum, then scaled
(one rounding) and rounded to its type, and added to the old value where it
accumulates (one more)."""
import sys

import pytest
import torch

import blockwise_fp8_zero_amd as bfz

pytestmark = pytest.mark.gpu
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}
U = 2.0 ** -24


def _say(*a):
    print("[gpu-embedding]", *a, flush=True)
    sys.stdout.flush()


def _fp8(V, d):
    codes = (torch.randn(V, d, device="cuda") * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
    grid = torch.rand(-(-V // 128), -(-d // 128), device="cuda") * 1e-3 + 1e-4
    up = grid.double().repeat_interleave(128, 0)[:V].repeat_interleave(128, 1)[:, :d]
    return codes.view(torch.uint8), grid, codes.to(torch.float64) * up


def _near(got, want, rel, tiny):
    err = (got.double() - want).abs()
    lim = rel * want.abs() + tiny
    bad = err > lim
    assert not bool(bad.any()), (err[bad][:4], want[bad][:4])


@pytest.mark.parametrize("out_type", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("table_type", ["fp8", torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V,d,n", [(1, 1, 1), (300, 128, 5), (257, 1000, 33), (1000, 4096, 70), (129, 130, 2), (200, 4097, 9)])
def test_embed(table_type, out_type, V, d, n):
    _say(table_type, out_type, V, d, n)
    torch.manual_seed(V + d)
    grid = None
    if table_type == "fp8":
        table, grid, value = _fp8(V, d)
    else:
        table = torch.randn(V, d, device="cuda").to(table_type)
        value = table.double()
    ids = torch.randint(0, V, (n,), device="cuda")
    if n > 4:
        ids[1], ids[3] = -1, V
    out = torch.full((n, d), 9.0, device="cuda").to(out_type)
    scale = 0.8125 * d ** 0.5
    bfz.embed(ids, table, out, scale=scale, grid=grid)
    keep = (ids >= 0) & (ids < V)
    s32 = float(torch.tensor(scale, dtype=torch.float32))
    want = torch.where(keep[:, None], value[ids.clamp(0, V - 1)] * s32, 0.0)
    _near(out, want, HALF[out_type] + 3 * U, TINY[out_type])
    out2 = torch.full((n, d), 9.0, device="cuda").to(out_type)
    bfz.embed(ids.int(), table, out2, scale=scale, grid=grid)
    assert torch.equal(out, out2)


def test_embed_strides_and_alignment():
    torch.manual_seed(2)
    V, d, n = 300, 256, 40
    ids = torch.randint(0, V, (n,), device="cuda")
    for off, ldt, ldo in ((0, 256, 256), (0, 272, 264), (1, 257, 259), (8, 300, 260), (4, 260, 300)):
        tab = torch.randn(V * ldt + 16, device="cuda").to(torch.bfloat16)
        table = torch.as_strided(tab, (V, d), (ldt, 1), off)
        buf = torch.full((n * ldo + 16,), 5.0, device="cuda")
        out = torch.as_strided(buf, (n, d), (ldo, 1), off)
        rest = torch.ones_like(buf, dtype=torch.bool)
        torch.as_strided(rest, (n, d), (ldo, 1), off).fill_(False)
        bfz.embed(ids, table, out, scale=2.0)
        assert torch.equal(out, table.float()[ids] * 2.0), (off, ldt, ldo)
        assert bool((buf[rest] == 5).all())
    codes, grid, value = _fp8(V, 300)
    for off in (0, 1, 4, 8, 16):
        out = torch.empty(n, 256, device="cuda")
        sub = torch.as_strided(torch.cat([codes.view(-1), codes.view(-1)[:64]]), (V, 256), (300, 1), off)
        g2 = grid[:, :2].contiguous()
        bfz.embed(ids, sub, out, grid=g2)
        val = sub.contiguous().view(torch.float8_e4m3fn).to(torch.float64)
        val = val * g2.double().repeat_interleave(128, 0)[:V].repeat_interleave(128, 1)
        _near(out, val[ids], 3 * U, 2.0 ** -149)


def _grad_want(ids, dout, V, scale, base):
    keep = (ids >= 0) & (ids < V)
    rows, at = dout.double()[keep], ids[keep]
    s = torch.zeros(V, dout.shape[1], dtype=torch.float64, device="cuda").index_add_(0, at, rows)
    a = torch.zeros_like(s).index_add_(0, at, rows.abs())
    c = torch.zeros(V, dtype=torch.float64, device="cuda").index_add_(0, at, torch.ones(len(at), dtype=torch.float64, device="cuda"))
    want = s * scale + (base.double() if base is not None else 0.0)
    err = (c[:, None] + 2) * U * a * abs(scale)
    return want, err, c > 0


def _grad_case(ids, dout, V, dtype, accumulate, scale=3.25):
    n, d = dout.shape
    base = torch.randn(V, d, device="cuda").to(dtype) if accumulate else None
    dt = base.clone() if accumulate else torch.full((V, d), float("nan"), device="cuda").to(dtype)
    work = bfz.embed_grad_workspace(n, d)
    work.fill_(0xA5)
    bfz.embed_grad(ids, dout, dt, work, scale=scale, accumulate=accumulate)
    want, err, hit = _grad_want(ids, dout, V, scale, base)
    got = dt.double()
    assert bool(torch.isfinite(got).all())
    lim = err + (HALF[dtype] + 2 * U) * (want.abs() + err) + TINY[dtype]
    bad = (got - want).abs() > lim
    assert not bool(bad.any()), (int(bad.sum()), got[bad][:4], want[bad][:4])
    if accumulate:
        assert torch.equal(dt[~hit], base[~hit])
    dt2 = base.clone() if accumulate else torch.zeros_like(dt)
    bfz.embed_grad(ids, dout, dt2, work, scale=scale, accumulate=accumulate)
    assert torch.equal(dt, dt2)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 63, 2048, 2049, 5000, 16384, 40001])
def test_embed_grad_counts(n, accumulate):
    _say("n", n, accumulate)
    torch.manual_seed(n)
    V, d = 700, 136
    ids = (torch.rand(n, device="cuda") ** 3 * (V + 20)).long() - 10  # some outside
    _grad_case(ids, torch.randn(n, d, device="cuda"), V, torch.float32, accumulate)


@pytest.mark.parametrize("src", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dst", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V,d", [(1, 1), (50, 130), (333, 1025), (20, 4100)])
def test_embed_grad_types(src, dst, V, d):
    _say(src, dst, V, d)
    torch.manual_seed(d)
    ids = torch.randint(-1, V + 1, (300,), device="cuda", dtype=torch.int32)
    _grad_case(ids.long(), torch.randn(300, d, device="cuda").to(src), V, dst, False)
    _grad_case(ids.long(), torch.randn(300, d, device="cuda").to(src), V, dst, True)


@pytest.mark.parametrize("kind", ["one", "none", "ends", "distinct", "descending"])
def test_embed_grad_patterns(kind):
    _say(kind)
    torch.manual_seed(7)
    V, d, n = 33000, 64, 33000
    ids = {"one": torch.full((n,), 5, device="cuda"), "none": torch.full((n,), -3, device="cuda"),
           "ends": torch.where(torch.rand(n, device="cuda") < 0.5, 0, V - 1), "distinct": torch.randperm(V, device="cuda"),
           "descending": torch.arange(n - 1, -1, -1, device="cuda") // 40}[kind]
    _grad_case(ids, torch.randn(n, d, device="cuda"), V, torch.float32, False)
    _grad_case(ids, torch.randn(n, d, device="cuda"), V, torch.float32, True)


def test_embed_grad_many_runs():
    """More tokens than one merge joins."""
    torch.manual_seed(8)
    n, V = 600_011, 5000
    ids = (torch.rand(n, device="cuda") ** 2 * V).long()
    _grad_case(ids, torch.randn(n, 8, device="cuda"), V, torch.float32, False)


def test_embed_grad_strides_and_empty():
    torch.manual_seed(9)
    V, d, n = 90, 100, 77
    ids = torch.randint(0, V, (n,), device="cuda")
    buf = torch.randn(n * 131 + 8, device="cuda")
    dout = torch.as_strided(buf, (n, d), (131, 1), 3)
    tab = torch.full((V * 120 + 8,), 4.0, device="cuda")
    dt = torch.as_strided(tab, (V, d), (120, 1), 4)
    work = bfz.embed_grad_workspace(n, d)
    bfz.embed_grad(ids, dout, dt, work)
    want, err, _ = _grad_want(ids, dout.contiguous(), V, 1.0, None)
    assert bool(((dt.double() - want).abs() <= err + 3 * U * want.abs()).all())
    rest = torch.ones_like(tab, dtype=torch.bool)
    torch.as_strided(rest, (V, d), (120, 1), 4).fill_(False)
    assert bool((tab[rest] == 4).all())
    bfz.embed_grad(ids[:0], dout[:0], dt, work)
    assert bool((dt == 0).all())
    out = torch.empty(0, d, device="cuda")
    bfz.embed(ids[:0], dt, out)


def test_embed_grad_workspace_serves_smaller_batches():
    torch.manual_seed(11)
    V, d = 400, 60
    ids = torch.randint(0, V, (20000,), device="cuda")
    dout = torch.randn(20000, d, device="cuda")
    work = bfz.embed_grad_workspace(20000, d)
    for n in (1, 500, 9000, 16383, 16384, 20000):
        a, b = torch.empty(V, d, device="cuda"), torch.empty(V, d, device="cuda")
        bfz.embed_grad(ids[:n], dout[:n], a, work)
        bfz.embed_grad(ids[:n], dout[:n], b, bfz.embed_grad_workspace(n, d))
        assert torch.equal(a, b), n


def test_embed_past_32_bits():
    """Row offsets past 2^32 elements, both ways."""
    V, d = 1_100_000, 4096
    table = torch.zeros(V, d, dtype=torch.uint8, device="cuda")
    table[V - 1].fill_(0x38)  # 1.0
    grid = torch.ones(-(-V // 128), d // 128, device="cuda")
    grid[-1] = 2.5
    ids = torch.tensor([V - 1, 0, V - 1, V], device="cuda")
    out = torch.empty(4, d, device="cuda")
    bfz.embed(ids, table, out, grid=grid)
    assert bool((out[0] == 2.5).all()) and bool((out[2] == 2.5).all()) and bool((out[[1, 3]] == 0).all())
    del table
    dt = torch.zeros(V, d, device="cuda")
    bfz.embed_grad(ids, torch.ones(4, d, device="cuda"), dt, bfz.embed_grad_workspace(4, d), accumulate=True)
    assert bool((dt[V - 1] == 2).all()) and bool((dt[0] == 1).all()) and float(dt[V - 2].abs().max()) == 0


def test_embedding_in_a_graph_and_on_a_side_stream():
    torch.manual_seed(10)
    V, d, n = 900, 512, 3000
    codes, grid, _ = _fp8(V, d)
    ids = torch.randint(0, V, (n,), device="cuda")
    dout = torch.randn(n, d, device="cuda")
    out, dt = torch.empty(n, d, device="cuda"), torch.empty(V, d, device="cuda")
    work = bfz.embed_grad_workspace(n, d)

    def step():
        bfz.embed(ids, codes, out, grid=grid)
        bfz.embed_grad(ids, dout, dt, work)

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    for k in range(4):
        ids.copy_(torch.randint(-1, V, (n,), device="cuda"))
        step()
        torch.cuda.synchronize()
        want = out.clone(), dt.clone()
        out.zero_()
        dt.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(dt, want[1]), k
