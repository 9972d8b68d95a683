"""GPU checks of the 4-bit products where offsets pass 32 bits: weights of more than
4 GiB of codes, outputs of more than 2^31 elements.  Sampled rows and columns, at the
ends and in the middle, against the 64-bit forms of tests/linear_ref.py."""
import pytest
import torch

import linear_ref as ref
from conftest import log

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def lin(fqlib):
    from fake_quant_amd import linear
    return linear


def big_weight(n, k, group, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.empty((n, k // 2), dtype=torch.uint8, device="cuda")
    for part in codes.split(1 << 15):
        part.random_(0, 256, generator=gen)
    scale = torch.rand(n, k // group, generator=gen, device="cuda") / 64
    zp = torch.randint(-8, 8, (n, k // group), generator=gen, device="cuda", dtype=torch.int32)
    return dict(codes=codes, scale=scale, zp=zp)


def rows_of(w, rows):
    return {name: t[rows].contiguous() for name, t in w.items()}


@pytest.mark.parametrize("m", [3, 40])
def test_codes_beyond_4_gib(lin, m):
    n, k, group = 270_001, 32768, 128
    w = big_weight(n, k, group, 1)
    x, dy = ref.tokens(m, k, BF, 2), ref.tokens(m, n, BF, 3, 1e-3)
    log(f"large weight m={m}")
    y = lin.w4_matmul(x.cuda(), w, group)
    dx, dw = lin.w4_matmul_backward(dy.cuda(), x.cuda(), w, group, dw_dtype=BF)
    torch.cuda.synchronize()
    rows = torch.tensor([0, 1, n // 2, n - 17, n - 2, n - 1])
    wd = ref.dense(rows_of(w, rows.cuda()), k, group)
    ref.assert_within(y[:, rows.cuda()], *ref.matmul(x, wd), "y")
    (_, dw_want), (_, dw_bound) = ref.matmul_backward(dy[:, rows], x, wd, BF)
    ref.assert_within(dw[rows.cuda()], dw_want, dw_bound, "dw")
    # 32 columns of dx at each end, summed over all rows
    for c0 in (0, k - 32):
        part = dict(codes=w["codes"][:, c0 // 2:c0 // 2 + 16].contiguous(), scale=w["scale"][:, c0 // group:c0 // group + 1],
                    zp=w["zp"][:, c0 // group:c0 // group + 1])
        cols = ref.dense(part, 32, group)
        (dx_want, _), (dx_bound, _) = ref.matmul_backward(dy, x[:, c0:c0 + 32], cols, BF)
        ref.assert_within(dx[:, c0:c0 + 32], dx_want, dx_bound, "dx")


def test_outputs_beyond_2_31(lin):
    m, n, k, group = 70_001, 32_776, 64, 32
    (wg, gd), (wu, ud) = ((ref.to(w, "cuda"), ref.dense(w, k, group))
                          for w in (ref.weight(n, k, group, "affine", s) for s in (1, 2)))
    x = ref.tokens(m, k, BF, 4)
    log("large outputs")
    rows = torch.tensor([0, 1, m // 2, 65_535, 65_536, m - 2, m - 1])
    y = lin.w4_matmul(x.cuda(), wg, group)[rows.cuda()]
    h = lin.w4_gated(x.cuda(), wg, wu, group)[rows.cuda()]
    torch.cuda.synchronize()
    ref.assert_within(y, *ref.matmul(x[rows], gd), "y")
    want, bound = ref.gated(x[rows], gd, ud, "silu")
    ref.assert_within(h, want[0], bound[0], "h")
