"""GPU checks of the 4-bit products at sizes that take each kernel's variants: tiles of
256 and 128 token rows, few-token blocks beyond one, contractions split over
workgroups and joined, pairs of weights of which one has zero-points, and views that
start off 16-byte borders.  Bounds as in tests/linear_ref.py."""
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


def sides(n, k, group, scheme, seed):
    w = ref.weight(n, k, group, scheme, seed)
    return ref.to(w, "cuda"), ref.dense(w, k, group)


# (m, n, k, group): few tokens in several blocks, 128-row tiles, 256-row tiles, odd widths of each
FORWARD = [(513, 264, 384, 128), (700, 130, 1000, 64), (1030, 1000, 96, 96), (2100, 2000, 264, 32), (2049, 2050, 129, 64),
           (8300, 1000, 200, 64), (8193, 1025, 77, 32), (14400, 70, 128, 128), (300, 12000, 72, 32)]


@pytest.mark.parametrize("m,n,k,group", FORWARD)
@pytest.mark.parametrize("dtype,scheme", [(BF, "affine"), (F, "sym")])
def test_matmul(lin, m, n, k, group, dtype, scheme):
    log(f"matmul {m} {n} {k} group {group} {dtype} {scheme}")
    w, wd = sides(n, k, group, scheme, m + n)
    x = ref.tokens(m, k, dtype, k)
    y = lin.w4_matmul(x.cuda(), w, group)
    torch.cuda.synchronize()
    ref.assert_within(y, *ref.matmul(x, wd), "y")


@pytest.mark.parametrize("m,n,k,group", [(5, 100, 300, 64), (600, 70, 260, 32), (2100, 1000, 264, 32), (8300, 500, 130, 64),
                                         (8200, 513, 77, 32)])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("first", ["sym", "affine"])
def test_gated_mixed(lin, m, n, k, group, dtype, first):
    """One weight with zero-points, the other without."""
    log(f"gated {m} {n} {k} group {group} {dtype} {first} first")
    second = "affine" if first == "sym" else "sym"
    (wg, gd), (wu, ud) = sides(n, k, group, first, m + n), sides(n, k, group, second, m + n + 1)
    x = ref.tokens(m, k, dtype, k)
    out = lin.w4_gated(x.cuda(), wg, wu, group, "gelu", save=True)
    torch.cuda.synchronize()
    want, bound = ref.gated(x, gd, ud, "gelu")
    for name, o, w_, b in zip("hgu", out, want, bound):
        ref.assert_within(o, w_, b, name)


# split over the contraction for dx, for dw, for both, for neither; 256-row tiles for dx, for dw
BACKWARD = [(70, 1100, 264, 64), (2000, 70, 130, 32), (1100, 1100, 136, 64), (40, 2050, 77, 32), (200, 4200, 1000, 128),
            (8300, 72, 1000, 64), (8193, 129, 1027, 64), (1000, 520, 6000, 32)]


@pytest.mark.parametrize("m,n,k,group", BACKWARD)
@pytest.mark.parametrize("scheme,dw_dtype", [("affine", F), ("sym", BF)])
def test_matmul_backward(lin, m, n, k, group, scheme, dw_dtype):
    log(f"matmul backward {m} {n} {k} group {group} {scheme} {dw_dtype}")
    w, wd = sides(n, k, group, scheme, m + n)
    x, dy = ref.tokens(m, k, BF, k), ref.tokens(m, n, BF, n, 1e-3)
    got = lin.w4_matmul_backward(dy.cuda(), x.cuda(), w, group, dw_dtype=dw_dtype)
    torch.cuda.synchronize()
    want, bound = ref.matmul_backward(dy, x, wd, dw_dtype)
    for name, o, w_, b in zip(("dx", "dw"), got, want, bound):
        ref.assert_within(o, w_, b, name)


@pytest.mark.parametrize("m,n,k,group", BACKWARD)
@pytest.mark.parametrize("first,act,dw_dtype", [("sym", "silu", BF), ("affine", "gelu", F)])
def test_gated_backward(lin, m, n, k, group, first, act, dw_dtype):
    log(f"gated backward {m} {n} {k} group {group} {first} first {act} {dw_dtype}")
    second = "affine" if first == "sym" else "sym"
    (wg, gd), (wu, ud) = sides(n, k, group, first, m + n), sides(n, k, group, second, m + n + 1)
    x, dh = ref.tokens(m, k, BF, k), ref.tokens(m, n, BF, n, 1e-3)
    g, u = ref.tokens(m, n, BF, n + 1, 2.0), ref.tokens(m, n, BF, n + 2)
    got = lin.w4_gated_backward(dh.cuda(), x.cuda(), g.cuda(), u.cuda(), wg, wu, group, act, dw_dtype=dw_dtype)
    torch.cuda.synchronize()
    want, bound = ref.gated_backward(dh, x, g, u, gd, ud, act, dw_dtype)
    for name, o, w_, b in zip(("dx", "dwg", "dwu"), got, want, bound):
        ref.assert_within(o, w_, b, name)


def test_same_bits_twice(lin):
    """Split and joined sums do not depend on the order in which workgroups end."""
    m, n, k, group = 1100, 1100, 136, 64
    (wg, _), (wu, _) = sides(n, k, group, "sym", 1), sides(n, k, group, "affine", 2)
    x, dh = ref.tokens(m, k, BF, 3).cuda(), ref.tokens(m, n, BF, 4).cuda()
    g, u = ref.tokens(m, n, BF, 5).cuda(), ref.tokens(m, n, BF, 6).cuda()
    first = lin.w4_gated_backward(dh, x, g, u, wg, wu, group, dw_dtype=F)
    for _ in range(3):
        for a, b in zip(first, lin.w4_gated_backward(dh, x, g, u, wg, wu, group, dw_dtype=F)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("m", [600, 2100])
def test_graph(lin, m):
    """Captured with its workspaces and replayed on new inputs, with eager work between the replays."""
    n, k, group = 1030, 260, 32
    w, _ = sides(n, k, group, "affine", 1)
    x, dh = ref.tokens(m, k, BF, 3).cuda(), ref.tokens(m, n, BF, 4).cuda()

    def step():
        h, g, u = lin.w4_gated(x, w, w, group, "silu", save=True)
        return (h, *lin.w4_gated_backward(dh, x, g, u, w, w, group, "silu"), *lin.w4_matmul_backward(dh, x, w, group))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(3):
        x.copy_(ref.tokens(m, k, BF, 20 + seed))
        dh.copy_(ref.tokens(m, n, BF, 30 + seed))
        graph.replay()
        torch.cuda.synchronize()
        held = [t.clone() for t in out]
        for a, b in zip(held, step()):
            assert torch.equal(a, b)


def test_unaligned_views_of_many_tokens(lin):
    m, n, k, group = 2100, 2000, 136, 64
    w, wd = sides(n, k, group, "affine", 3)
    x = ref.tokens(m, k, BF, 4)
    xs = torch.empty(m * k + 1, dtype=BF, device="cuda")
    xs[1:] = x.reshape(-1).cuda()
    y = lin.w4_matmul(xs[1:].view(m, k), w, group)
    ref.assert_within(y, *ref.matmul(x, wd), "y")


def test_nonfinite_tokens_of_tiles(lin):
    """An infinity and a NaN in two tokens' rows stay in those rows of the tile."""
    m, n, k, group = 2100, 2000, 136, 64
    w, wd = sides(n, k, group, "affine", 9)
    for dtype in (BF, F):
        x = ref.tokens(m, k, dtype, 11)
        x[2099, 135] = float("inf")
        x[130, 0] = float("nan")
        log(f"nonfinite tile {dtype}")
        y = lin.w4_matmul(x.cuda(), w, group)
        ref.assert_within(y, *ref.matmul(x, wd), "y")


@pytest.mark.parametrize("ratio", [2.0 ** -10, 2.0 ** -20, 2.0 ** 12])
def test_uneven_scales(lin, ratio):
    """Groups and rows of a weight far from the others', and tokens far from each other."""
    m, n, k, group = 70, 300, 256, 64
    ws = []
    for seed in (1, 2):
        w = ref.weight(n, k, group, "affine", seed)
        w["scale"][:, 1] *= ratio
        w["scale"][::3] *= ratio
        ws.append((ref.to(w, "cuda"), ref.dense(w, k, group)))
    (wg, gd), (wu, ud) = ws
    x, dh = ref.tokens(m, k, BF, 3), ref.tokens(m, n, BF, 4, 1e-3)
    dh[::2] *= ratio
    g, u = ref.tokens(m, n, BF, 5, 2.0), ref.tokens(m, n, BF, 6)
    log(f"uneven scales {ratio}")
    got = lin.w4_gated_backward(dh.cuda(), x.cuda(), g.cuda(), u.cuda(), wg, wu, group)
    want, bound = ref.gated_backward(dh, x, g, u, gd, ud, "silu", BF)
    for name, o, w_, b in zip(("dx", "dwg", "dwu"), got, want, bound):
        ref.assert_within(o, w_, b, name)


def test_long_rows(lin):
    """Tokens of more than 16384 values of g and u."""
    m, n, k, group = 5, 17000, 64, 32
    (wg, gd), (wu, ud) = sides(n, k, group, "sym", 1), sides(n, k, group, "affine", 2)
    x, dh = ref.tokens(m, k, BF, 3), ref.tokens(m, n, BF, 4, 1e-3)
    g, u = ref.tokens(m, n, BF, 5, 2.0), ref.tokens(m, n, BF, 6)
    log("long rows")
    got = lin.w4_gated_backward(dh.cuda(), x.cuda(), g.cuda(), u.cuda(), wg, wu, group)
    want, bound = ref.gated_backward(dh, x, g, u, gd, ud, "silu", BF)
    for name, o, w_, b in zip(("dx", "dwg", "dwu"), got, want, bound):
        ref.assert_within(o, w_, b, name)
