"""GPU checks of the products with 4-bit group-quantized weights and of the gated
block (forward and backward) against the plain 64-bit forms of tests/linear_ref.py,
element by element within bounds that count roundings: token counts from one to
several tiles, odd widths, groups that divide nothing, float32 and bfloat16,
symmetric and affine weights, empty groups and rows, non-finite tokens, side
streams, unaligned views, graphs, and gradients against differences."""
import pytest
import torch

import linear_ref as ref
from conftest import log

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lin(fqlib):
    from fake_quant_amd import linear
    return linear


# (m, n, k, group)
SHAPES = [
    (1, 1, 1, 1), (1, 64, 64, 32), (3, 5, 7, 3), (2, 17, 130, 64), (1, 4096, 512, 128), (1, 257, 4100, 128),
    (5, 100, 333, 32), (8, 48, 1024, 256), (9, 70, 96, 96), (17, 33, 256, 128), (16, 128, 128, 128),
    (31, 95, 640, 64), (33, 40, 200, 48), (48, 272, 2048, 128), (64, 64, 512, 512), (65, 130, 1000, 64),
    (130, 300, 641, 32), (200, 520, 768, 1000), (257, 264, 384, 128), (300, 1030, 264, 128), (513, 130, 136, 64),
]


def sides(n, k, group, scheme, seed):
    w = ref.weight(n, k, group, scheme, seed)
    return ref.to(w, "cuda"), ref.dense(w, k, group)


@pytest.mark.parametrize("m,n,k,group", SHAPES)
@pytest.mark.parametrize("dtype,scheme", [(BF, "sym"), (BF, "affine"), (F, "affine"), (F, "sym")])
def test_matmul(lin, m, n, k, group, dtype, scheme):
    log(f"matmul {m} {n} {k} group {group} {dtype} {scheme}")
    w, wd = sides(n, k, group, scheme, m + n)
    x = ref.tokens(m, k, dtype, k)
    y = lin.w4_matmul(x.cuda(), w, group)
    torch.cuda.synchronize()
    assert y.dtype == dtype
    ref.assert_within(y, *ref.matmul(x, wd), "y")


@pytest.mark.parametrize("m,n,k,group", SHAPES)
@pytest.mark.parametrize("dtype,scheme,act,save", [(BF, "sym", "silu", True), (BF, "affine", "gelu", False),
                                                   (F, "affine", "silu", True), (F, "sym", "gelu", False)])
def test_gated(lin, m, n, k, group, dtype, scheme, act, save):
    log(f"gated {m} {n} {k} group {group} {dtype} {scheme} {act} save={save}")
    (wg, gd), (wu, ud) = sides(n, k, group, scheme, m + n), sides(n, k, group, scheme, m + n + 1)
    x = ref.tokens(m, k, dtype, k)
    out = lin.w4_gated(x.cuda(), wg, wu, group, act, save=save)
    torch.cuda.synchronize()
    want, bound = ref.gated(x, gd, ud, act)
    for name, o, w_, b in zip("hgu", out if save else (out,), want, bound):
        ref.assert_within(o, w_, b, name)


@pytest.mark.parametrize("m,n,k,group", SHAPES)
@pytest.mark.parametrize("scheme,dw_dtype", [("sym", F), ("affine", BF)])
def test_matmul_backward(lin, m, n, k, group, scheme, dw_dtype):
    log(f"matmul backward {m} {n} {k} group {group} {scheme} {dw_dtype}")
    w, wd = sides(n, k, group, scheme, m + n)
    x, dy = ref.tokens(m, k, BF, k), ref.tokens(m, n, BF, n, 1e-3)
    got = lin.w4_matmul_backward(dy.cuda(), x.cuda(), w, group, dw_dtype=dw_dtype)
    torch.cuda.synchronize()
    want, bound = ref.matmul_backward(dy, x, wd, dw_dtype)
    for name, o, w_, b in zip(("dx", "dw"), got, want, bound):
        ref.assert_within(o, w_, b, name)


@pytest.mark.parametrize("m,n,k,group", SHAPES)
@pytest.mark.parametrize("scheme,act,dw_dtype", [("sym", "silu", BF), ("affine", "gelu", F)])
def test_gated_backward(lin, m, n, k, group, scheme, act, dw_dtype):
    log(f"gated backward {m} {n} {k} group {group} {scheme} {act} {dw_dtype}")
    (wg, gd), (wu, ud) = sides(n, k, group, scheme, m + n), sides(n, k, group, scheme, m + n + 1)
    x, dh = ref.tokens(m, k, BF, k), ref.tokens(m, n, BF, n, 1e-3)
    g, u = ref.tokens(m, n, BF, n + 1, 2.0), ref.tokens(m, n, BF, n + 2)
    got = lin.w4_gated_backward(dh.cuda(), x.cuda(), g.cuda(), u.cuda(), wg, wu, group, act, dw_dtype=dw_dtype)
    torch.cuda.synchronize()
    want, bound = ref.gated_backward(dh, x, g, u, gd, ud, act, dw_dtype)
    for name, o, w_, b in zip(("dx", "dwg", "dwu"), got, want, bound):
        ref.assert_within(o, w_, b, name)


@pytest.mark.parametrize("sigma", [1e-30, 1e-8, 1e6, 1e25])
def test_gradient_range(lin, sigma):
    """Gradients far from 1, beside rows that are 2^20 times smaller."""
    m, n, k, group = 70, 200, 192, 64
    (wg, gd), (wu, ud) = sides(n, k, group, "affine", 1), sides(n, k, group, "affine", 2)
    x, dh = ref.tokens(m, k, BF, 3), ref.tokens(m, n, BF, 4, sigma)
    dh[::3] *= 2.0 ** -20
    g, u = ref.tokens(m, n, BF, 5, 2.0), ref.tokens(m, n, BF, 6)
    log(f"gradient range {sigma}")
    got = lin.w4_gated_backward(dh.cuda(), x.cuda(), g.cuda(), u.cuda(), wg, wu, group)
    got2 = lin.w4_matmul_backward(dh.cuda(), x.cuda(), wg, group)
    torch.cuda.synchronize()
    want, bound = ref.gated_backward(dh, x, g, u, gd, ud, "silu", BF)
    for name, o, w_, b in zip(("dx", "dwg", "dwu"), got, want, bound):
        ref.assert_within(o, w_, b, name)
    for name, o, w_, b in zip(("dx", "dw"), got2, *ref.matmul_backward(dh, x, gd, F)):
        ref.assert_within(o, w_, b, name)


@pytest.mark.parametrize("m", [1, 7, 40, 200, 300])
@pytest.mark.parametrize("group", [32, 128, 48])
@pytest.mark.parametrize("dtype", [BF, F])
def test_nonfinite_tokens(lin, m, group, dtype):
    """Inf and NaN in one token's row stay in that row; an infinity meets a zero weight as NaN."""
    n, k = 150, 512
    w, wd = sides(n, k, group, "sym", 9)
    (wu, ud) = sides(n, k, group, "sym", 10)
    x = ref.tokens(m, k, dtype, 11)
    bad = (m - 1) // 2
    x[bad, 70] = float("inf")
    log(f"nonfinite m={m} group={group} {dtype}")
    y = lin.w4_matmul(x.cuda(), w, group)
    ref.assert_within(y, *ref.matmul(x, wd), "inf")
    x[bad, 70] = 1.0
    x[bad, k - 1] = float("nan")
    y, h = lin.w4_matmul(x.cuda(), w, group), lin.w4_gated(x.cuda(), w, wu, group)
    ref.assert_within(y, *ref.matmul(x, wd), "nan")
    assert bool(torch.isnan(h[bad]).all()) and int(torch.isnan(h).sum()) == n


def test_nonfinite_gradients(lin):
    """A token whose gradient is NaN spoils its own dx row and every dw, and no other dx row."""
    m, n, k, group = 140, 96, 256, 64
    (wg, _), (wu, _) = sides(n, k, group, "sym", 1), sides(n, k, group, "affine", 2)
    x, dh = ref.tokens(m, k, BF, 3).cuda(), ref.tokens(m, n, BF, 4).cuda()
    g, u = ref.tokens(m, n, BF, 5).cuda(), ref.tokens(m, n, BF, 6).cuda()
    dh[77] = float("nan")
    for dx in (lin.w4_gated_backward(dh, x, g, u, wg, wu, group)[0], lin.w4_matmul_backward(dh, x, wg, group)[0]):
        assert bool(torch.isnan(dx[77]).all()) and int(torch.isnan(dx).sum()) == k


@pytest.mark.parametrize("dtype", [BF, F])
def test_no_tokens(lin, dtype):
    w, _ = sides(48, 96, 32, "sym", 1)
    x = torch.empty(0, 96, dtype=dtype, device="cuda")
    assert lin.w4_matmul(x, w, 32).shape == (0, 48)
    assert all(t.shape == (0, 48) for t in lin.w4_gated(x, w, w, 32, save=True))
    if dtype == BF:
        dy = torch.empty(0, 48, dtype=BF, device="cuda")
        dx, dw = lin.w4_matmul_backward(dy, x, w, 32)
        assert dx.shape == (0, 96) and dw.shape == (48, 96) and not bool(dw.any())
        dx, a, b = lin.w4_gated_backward(dy, x, dy, dy, w, w, 32)
        assert dx.shape == (0, 96) and not bool(a.any()) and not bool(b.any())


@pytest.mark.parametrize("m", [1, 20, 140])
def test_unaligned_views(lin, m):
    """Codes at an odd address, x and y two bytes off a 16-byte border."""
    n, k, group = 130, 384, 128
    w, wd = sides(n, k, group, "affine", 3)
    x = ref.tokens(m, k, BF, 4)
    store = torch.empty(n * k // 2 + 1, dtype=torch.uint8, device="cuda")
    store[1:] = w["codes"].reshape(-1)
    w["codes"] = store[1:].view(n, k // 2)
    xs = torch.empty(m * k + 1, dtype=BF, device="cuda")
    xs[1:] = x.reshape(-1).cuda()
    y = lin.w4_matmul(xs[1:].view(m, k), w, group)
    ref.assert_within(y, *ref.matmul(x, wd), "y")
    dys = torch.empty(m * n + 1, dtype=BF, device="cuda")
    dy = ref.tokens(m, n, BF, 5)
    dys[1:] = dy.reshape(-1).cuda()
    got = lin.w4_matmul_backward(dys[1:].view(m, n), xs[1:].view(m, k), w, group)
    for name, o, w_, b in zip(("dx", "dw"), got, *ref.matmul_backward(dy, x, wd, F)):
        ref.assert_within(o, w_, b, name)


@pytest.mark.parametrize("m", [1, 300])
def test_parts_and_streams(lin, m):
    """One output at a time, on a stream of its own, gives the bits that both together give."""
    n, k, group = 200, 320, 64
    (wg, _), (wu, _) = sides(n, k, group, "sym", 1), sides(n, k, group, "sym", 2)
    x, dh = ref.tokens(m, k, BF, 3).cuda(), ref.tokens(m, n, BF, 4).cuda()
    g, u = ref.tokens(m, n, BF, 5).cuda(), ref.tokens(m, n, BF, 6).cuda()
    both = lin.w4_matmul_backward(dh, x, wg, group)
    three = lin.w4_gated_backward(dh, x, g, u, wg, wu, group)
    h = lin.w4_gated(x, wg, wu, group)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        dx = lin.w4_matmul_backward(dh, x, wg, group, want_dw=False)[0]
        dw = lin.w4_matmul_backward(dh, x, wg, group, want_dx=False)[1]
        dx3 = lin.w4_gated_backward(dh, x, g, u, wg, wu, group, want_dw=False)[0]
        dw3 = lin.w4_gated_backward(dh, x, g, u, wg, wu, group, want_dx=False)[1:]
        h2 = lin.w4_gated(x, wg, wu, group, save=True)[0]
    s.synchronize()
    for a, b in zip((dx, dw, dx3, *dw3, h2), (*both, *three, h)):
        assert torch.equal(a.view(torch.int16 if a.dtype == BF else torch.int32),
                           b.view(torch.int16 if b.dtype == BF else torch.int32))


@pytest.mark.parametrize("m", [1, 150])
def test_graph(lin, m):
    """Captured and replayed on new inputs, with eager work between the replays."""
    n, k, group = 136, 260, 32
    w, wd = sides(n, k, group, "affine", 1)
    x, dh = ref.tokens(m, k, BF, 3).cuda(), ref.tokens(m, n, BF, 4).cuda()

    def step():
        h, g, u = lin.w4_gated(x, w, w, group, "gelu", save=True)
        return (h, *lin.w4_gated_backward(dh, x, g, u, w, w, group, "gelu"), lin.w4_matmul(x, w, group))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(4):
        x.copy_(ref.tokens(m, k, BF, 20 + seed))
        dh.copy_(ref.tokens(m, n, BF, 30 + seed))
        graph.replay()
        torch.cuda.synchronize()
        held = [t.clone() for t in out]
        for a, b in zip(held, step()):
            assert torch.equal(a, b)


def test_against_differences(lin):
    """<gradient, direction> against central differences of the 64-bit forward form."""
    m, n, k, group = 40, 72, 160, 32
    (wg, gd), (wu, ud) = sides(n, k, group, "affine", 1), sides(n, k, group, "affine", 2)
    x, dh = ref.tokens(m, k, BF, 3), ref.tokens(m, n, BF, 4)
    xd, d = x.double(), dh.double()
    g, u = (xd @ gd.T).to(BF), (xd @ ud.T).to(BF)
    got = [t.double().cpu() for t in lin.w4_gated_backward(dh.cuda(), x.cuda(), g.cuda(), u.cuda(), wg, wu, group,
                                                           "silu", dw_dtype=F)]
    want, bound = ref.gated_backward(dh, x, g, u, gd, ud, "silu", F)

    def loss(x_, g_, u_):
        return float((ref.act(x_ @ g_.T, "silu") * (x_ @ u_.T) * d).sum())

    gen = torch.Generator().manual_seed(7)
    for i, t in enumerate((xd, gd, ud)):
        v = torch.randn(t.shape, generator=gen, dtype=torch.float64)
        e = 1e-5
        args = [xd, gd, ud]
        lo, hi = list(args), list(args)
        lo[i], hi[i] = t - e * v, t + e * v
        diff = (loss(*hi) - loss(*lo)) / (2 * e)
        # the kernel reads g and u rounded to bfloat16: dg = dh u act'(g) and du = dh act(g) move by
        # at most (|g| max|act''| + max|act'|) |u| 2^-8 and max|act'| |g| 2^-8 of |dh|; the differences' own error is h^2
        G, U = (xd @ gd.T).abs(), (xd @ ud.T).abs()
        mg = d.abs() * U * (ref.CURVE_MAX * G + ref.SLOPE_MAX) * 2.0 ** -8
        mu = d.abs() * ref.SLOPE_MAX * G * 2.0 ** -8
        moved = (mg @ gd.abs() + mu @ ud.abs(), mg.T @ xd.abs(), mu.T @ xd.abs())[i]
        slack = float(((bound[i] + 1.01 * moved) * v.abs()).sum()) + 1e-6 * abs(diff)
        assert abs(float((got[i] * v).sum()) - diff) <= slack, i
        # and the 64-bit formula itself, which has no such slack, on unrounded g and u
        dg, du = d * (xd @ ud.T) * ref.slope(xd @ gd.T, "silu"), d * ref.act(xd @ gd.T, "silu")
        exact = (dg @ gd + du @ ud, dg.T @ xd, du.T @ xd)[i]
        assert abs(float((exact * v).sum()) - diff) <= 1e-6 * float((exact * v).abs().sum())
