"""Plain 64-bit forms of the 4-bit group-quantized products, on the CPU, and how
far a kernel's outputs may be from them.

Bounds count roundings.  A value rounded to a type is off by at most
``finfo(type).eps / 2`` of itself (bfloat16 2^-8, float32 2^-24).  A sum of c
binary32 terms of magnitude S = sum |term| is off by at most c * 2^-23 * S in any
order: one rounding a term, of up to one step (a matrix instruction may truncate
inside).  A float32 x enters as three bfloat16 parts, so its sums have 3 k terms;
eight roundings more cover the group scales and their sum.
"""
import math

import numpy as np
import torch

U_BF16 = 2.0 ** -8
U_STEP = 2.0 ** -23
TINY = 1e-37


def unit(dtype):
    return torch.finfo(dtype).eps / 2


def dense(w, k, group):
    """float64 [n, k] of a stored weight dict (tensors on any device)."""
    b = w["codes"].cpu().numpy().view(np.uint8)
    q = np.empty((b.shape[0], b.shape[1] * 2), np.int64)
    q[:, 0::2], q[:, 1::2] = b >> 4, b & 15
    q = np.where(q > 7, q - 16, q)[:, :k].astype(np.float64)
    col = np.arange(k) // group
    if w.get("zp") is not None:
        q = q - w["zp"].cpu().numpy().astype(np.float64)[:, col]
    return torch.from_numpy(q * w["scale"].cpu().numpy().astype(np.float64)[:, col])


def act(g, name):
    if name == "silu":
        return g * torch.sigmoid(g)
    return 0.5 * g * torch.special.erfc(-g / math.sqrt(2.0))


def slope(g, name):
    if name == "silu":
        s = torch.sigmoid(g)
        return s * (1 + g * (1 - s))
    return 0.5 * torch.special.erfc(-g / math.sqrt(2.0)) + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def sum_bound(a, b, terms):
    """c * 2^-23 * |a| |b|^T for a [i, l], b [j, l]."""
    return terms * U_STEP * (a.abs() @ b.abs().T)


def matmul(x, wd):
    """(y, bound) in float64 for x of its own type."""
    xd = x.double().cpu()
    y = xd @ wd.T
    return y, sum_bound(xd, wd, 3 * xd.shape[1] + 8) + unit(x.dtype) * y.abs() + TINY


# |silu'| and |gelu'| stay under 1.13; act and act' are evaluated to a few steps
# (under 2^-20 of themselves), where gelu's tail multiplies the rounding of its
# argument by g^2.
SLOPE_MAX = 1.13
CURVE_MAX = 0.8  # |act''| of both


def act_error(g, name):
    return 2.0 ** -20 * (1 + (g * g if name == "gelu" else 0)) * act(g, name).abs()


def gated(x, gd, ud, name):
    """(h, g, u) and their bounds."""
    xd = x.double().cpu()
    g, u = xd @ gd.T, xd @ ud.T
    t = 3 * xd.shape[1] + 8
    eg, eu = sum_bound(xd, gd, t), sum_bound(xd, ud, t)
    h = act(g, name) * u
    r = unit(x.dtype)
    eh = (SLOPE_MAX * eg + act_error(g, name)) * (u.abs() + eu) + act(g, name).abs() * eu
    return (h, g, u), (eh + r * h.abs() + r * eh + TINY, eg + r * g.abs() + TINY, eu + r * u.abs() + TINY)


def matmul_backward(dy, x, wd, dw_dtype):
    """(dx, dw) and bounds: dx's sums hold W rounded to bfloat16, dw's exact products."""
    dyd, xd = dy.double().cpu(), x.double().cpu()
    m, n = dyd.shape
    dx, dw = dyd @ wd, dyd.T @ xd
    edx = sum_bound(dyd, wd.T, n + 8) * (1 + U_BF16) + U_BF16 * (dyd.abs() @ wd.abs())
    edw = sum_bound(dyd.T, xd.T, m + 8)
    return (dx, dw), (edx + U_BF16 * (dx.abs() + edx) + TINY, edw + unit(dw_dtype) * (dw.abs() + edw) + TINY)


def gated_backward(dh, x, g, u, gd, ud, name, dw_dtype):
    """(dx, dwg, dwu) and bounds: every dg, du and W is off by at most a bfloat16
    rounding (and the act's own error) where a sum reads it."""
    d, xd, gg, uu = (t.double().cpu() for t in (dh, x, g, u))
    m, n = d.shape
    dg, du = d * uu * slope(gg, name), d * act(gg, name)
    # act' may cancel to near 0, so its error is taken against 1.13 and not itself
    eg = 2.0 ** -20 * (d * uu).abs() * SLOPE_MAX * (1 + gg * gg) + U_BF16 * dg.abs() + TINY
    eu = d.abs() * act_error(gg, name) + U_BF16 * du.abs() + TINY
    dx, dwg, dwu = dg @ gd + du @ ud, dg.T @ xd, du.T @ xd
    mag = dg.abs() @ gd.abs() + du.abs() @ ud.abs()
    edx = eg @ gd.abs() + eu @ ud.abs() + U_BF16 * 1.01 * mag + (2 * n + 8) * U_STEP * 1.01 * mag
    r = unit(dw_dtype)

    def dw_bound(dw, dv, ev):
        e = ev.T @ xd.abs() + (m + 8) * U_STEP * 1.01 * (dv.abs().T @ xd.abs())
        return e + r * (dw.abs() + e) + TINY

    return (dx, dwg, dwu), (edx + U_BF16 * (dx.abs() + edx) + TINY, dw_bound(dwg, dg, eg), dw_bound(dwu, du, eu))


def assert_within(got, want, bound, what):
    """Elementwise: NaN and Inf where the 64-bit form has them, elsewhere within the bound."""
    got = got.double().cpu()
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)}"
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN places"
    inf = ~fine & ~torch.isnan(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities"
    err = (got - want).abs()[fine]
    over = err > bound[fine]
    if bool(over.any()):
        i = int(torch.nonzero(over)[0, 0])
        raise AssertionError(f"{what}: {int(over.sum())} of {over.numel()} outside, first: got {got[fine][i]}, "
                             f"want {want[fine][i]}, bound {bound[fine][i]}")


def quantize(w, group, scheme):
    """Weight dict (CPU) by the rules of group calibration: min / max, ties to even."""
    n, k = w.shape
    ng = -(-k // group)
    p = torch.cat([w.double(), torch.zeros(n, ng * group - k, dtype=torch.float64)], 1).view(n, ng, group)
    if scheme == "sym":
        scale, zp = p.abs().amax(2) / 7, torch.zeros(n, ng, dtype=torch.float64)
    else:
        lo, hi = p.amin(2).clamp(max=0), p.amax(2).clamp(min=0)
        scale = (hi - lo) / 15
        zp = torch.nan_to_num(torch.round(-8 - lo / scale)).clamp(-8, 7)
    q = torch.nan_to_num(torch.round(p / scale[..., None])) + zp[..., None]
    q = q.clamp(-7 if scheme == "sym" else -8, 7).view(n, ng * group)[:, :k].long() & 15
    if k % 2:
        q = torch.cat([q, torch.zeros(n, 1, dtype=q.dtype)], 1)
    return dict(codes=(q[:, 0::2] * 16 + q[:, 1::2]).to(torch.uint8), scale=scale.float().contiguous(),
                zp=None if scheme == "sym" else zp.to(torch.int32).contiguous())


def weight(n, k, group, scheme, seed):
    gen = torch.Generator().manual_seed(seed)
    w = torch.randn(n, k, generator=gen) * torch.exp(torch.randn(n, 1, generator=gen) * 0.5) / math.sqrt(k)
    w[n // 2, : min(group, k)] = 0.0  # a group without a range: scale 0
    return quantize(w, group, scheme)


def tokens(m, c, dtype, seed, sigma=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(m, c, generator=gen) * sigma
    x[:, ::97] *= 10
    if m > 2:
        x[m // 2] = 0.0  # a row that holds nothing
    return x.to(dtype)


def to(w, device):
    return {n: None if t is None else t.to(device) for n, t in w.items()}
