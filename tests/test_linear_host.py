"""Host-side checks of include/fq_linear.h and its binding (no GPU, nothing is
launched): exported names, constants, and every refusal before anything is
enqueued."""
import ctypes
import os
import re

import pytest
import torch

from conftest import ROOT

HEADER = os.path.join(ROOT, "include", "fq_linear.h")
P = 0x10000  # a non-null, well-aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lin():
    if not os.path.exists(os.path.join(ROOT, "fake_quant_amd", "libfq.so")):
        from fake_quant_amd import build
        build.build()
    from fake_quant_amd import linear
    return linear


def test_exports_and_constants(lin):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    assert sorted(lin.EXPORTS) == sorted(set(re.findall(r"\b(fql_w4_[a-z0-9_]+)\s*\(", text)))
    assert re.search(r"FQL_SILU = (\d+)", text).group(1) == str(lin.SILU)
    assert re.search(r"FQL_GELU = (\d+)", text).group(1) == str(lin.GELU)


def weights(lin):
    good = lin.W4(P, P, P)
    bad = [lin.W4(None, P, None), lin.W4(P, None, None), lin.W4(P, P + 2, None), lin.W4(P, P, P + 1)]
    return ctypes.byref(good), [ctypes.byref(b) for b in bad] + [None]


SIZES = [(-1, 8, 8, 8), (4, 0, 8, 8), (4, 8, 0, 8), (4, 8, 8, 0), (4, -1, 8, 8), (1 << 31, 8, 8, 8), (4, 1 << 31, 8, 8),
         (4, 8, 1 << 31, 8)]


def test_matmul_refusals(lin):
    f, (w, bad) = lin._lib.fql_w4_matmul, weights(lin)
    big = 1 << 40
    assert f(P, 2, 4, 8, 64, 32, w, P, P, big, None) == lin.E_UNSUPPORTED
    for m, n, k, g in SIZES:
        assert f(P, 1, m, n, k, g, w, P, P, big, None) == lin.E_INVALID, (m, n, k, g)
    for b in bad:
        assert f(P, 1, 4, 8, 64, 32, b, P, P, big, None) == lin.E_INVALID
    assert f(None, 1, 4, 8, 64, 32, w, P, P, big, None) == lin.E_INVALID
    assert f(P, 1, 4, 8, 64, 32, w, None, P, big, None) == lin.E_INVALID
    assert f(P + 1, 1, 4, 8, 64, 32, w, P, P, big, None) == lin.E_INVALID
    assert f(P, 0, 4, 8, 64, 32, w, P + 2, P, big, None) == lin.E_INVALID
    assert f(None, 1, 0, 8, 64, 32, w, None, None, 0, None) == lin.OK  # no tokens: nothing to do


def test_gated_refusals(lin):
    f, (w, bad) = lin._lib.fql_w4_gated, weights(lin)
    big = 1 << 40
    assert f(P, 3, 4, 8, 64, 32, 0, w, w, P, None, None, P, big, None) == lin.E_UNSUPPORTED
    assert f(P, 1, 4, 8, 64, 32, 2, w, w, P, None, None, P, big, None) == lin.E_UNSUPPORTED
    for m, n, k, g in SIZES:
        assert f(P, 1, m, n, k, g, 0, w, w, P, None, None, P, big, None) == lin.E_INVALID
    for b in bad:
        assert f(P, 1, 4, 8, 64, 32, 0, b, w, P, None, None, P, big, None) == lin.E_INVALID
        assert f(P, 1, 4, 8, 64, 32, 0, w, b, P, None, None, P, big, None) == lin.E_INVALID
    assert f(P, 1, 4, 8, 64, 32, 0, w, w, None, None, None, P, big, None) == lin.E_INVALID
    assert f(P, 1, 4, 8, 64, 32, 0, w, w, P, P, None, P, big, None) == lin.E_INVALID  # g without u
    assert f(P, 1, 4, 8, 64, 32, 0, w, w, P, P + 1, P, P, big, None) == lin.E_INVALID
    assert f(None, 1, 0, 8, 64, 32, 0, w, w, None, None, None, None, 0, None) == lin.OK


def test_backward_refusals(lin):
    f, (w, bad) = lin._lib.fql_w4_matmul_backward, weights(lin)
    big = 1 << 40
    assert f(P, P, 0, 4, 8, 64, 32, w, P, P, 0, P, big, None) == lin.E_UNSUPPORTED  # float32 activations
    assert f(P, P, 1, 4, 8, 64, 32, w, P, P, 2, P, big, None) == lin.E_UNSUPPORTED
    for m, n, k, g in SIZES:
        assert f(P, P, 1, m, n, k, g, w, P, P, 0, P, big, None) == lin.E_INVALID
    for b in bad:
        assert f(P, P, 1, 4, 8, 64, 32, b, P, P, 0, P, big, None) == lin.E_INVALID
    assert f(P, P, 1, 4, 8, 64, 32, w, None, None, 0, P, big, None) == lin.E_INVALID
    assert f(None, P, 1, 4, 8, 64, 32, w, P, P, 0, P, big, None) == lin.E_INVALID
    assert f(P, None, 1, 4, 8, 64, 32, w, P, P, 0, P, big, None) == lin.E_INVALID
    assert f(P, P, 1, 4, 8, 64, 32, w, P, P + 2, 0, P, big, None) == lin.E_INVALID
    f = lin._lib.fql_w4_gated_backward
    assert f(P, P, P, P, 0, 4, 8, 64, 32, 0, w, w, P, P, P, 1, P, big, None) == lin.E_UNSUPPORTED
    assert f(P, P, P, P, 1, 4, 8, 64, 32, 5, w, w, P, P, P, 1, P, big, None) == lin.E_UNSUPPORTED
    for m, n, k, g in SIZES:
        assert f(P, P, P, P, 1, m, n, k, g, 0, w, w, P, P, P, 1, P, big, None) == lin.E_INVALID
    for b in bad:
        assert f(P, P, P, P, 1, 4, 8, 64, 32, 0, w, b, P, P, P, 1, P, big, None) == lin.E_INVALID
        assert f(P, P, P, P, 1, 4, 8, 64, 32, 0, b, w, P, P, P, 1, P, big, None) == lin.E_INVALID
    assert f(P, P, P, P, 1, 4, 8, 64, 32, 0, w, w, P, P, None, 1, P, big, None) == lin.E_INVALID
    assert f(P, P, P, P, 1, 4, 8, 64, 32, 0, w, w, None, None, None, 1, P, big, None) == lin.E_INVALID
    for miss in range(4):
        a = [P] * 4
        a[miss] = None
        assert f(*a, 1, 4, 8, 64, 32, 0, w, w, P, P, P, 1, P, big, None) == lin.E_INVALID


def test_workspace_refusals(lin):
    """A call that needs a workspace refuses a missing, short or misaligned one."""
    w, _ = weights(lin)
    m, n, k, g = 70, 96, 72, 32
    need = lin.fql_w4_matmul_workspace_bytes(0, m, n, k, g)
    if need:
        for ws, b in ((None, need), (P, need - 1), (P + 8, need)):
            assert lin._lib.fql_w4_matmul(P, 0, m, n, k, g, w, P, ws, b, None) == lin.E_INVALID
    need = lin.fql_w4_gated_workspace_bytes(0, m, n, k, g)
    if need:
        for ws, b in ((None, need), (P, need - 1), (P + 8, need)):
            assert lin._lib.fql_w4_gated(P, 0, m, n, k, g, 0, w, w, P, None, None, ws, b, None) == lin.E_INVALID
    need = lin.fql_w4_matmul_backward_workspace_bytes(m, n, k, g)
    if need:
        for ws, b in ((None, need), (P, need - 1), (P + 8, need)):
            assert lin._lib.fql_w4_matmul_backward(P, P, 1, m, n, k, g, w, P, P, 0, ws, b, None) == lin.E_INVALID
    need = lin.fql_w4_gated_backward_workspace_bytes(m, n, k, g)
    if need:
        for ws, b in ((None, need), (P, need - 1), (P + 8, need)):
            assert lin._lib.fql_w4_gated_backward(P, P, P, P, 1, m, n, k, g, 0, w, w, P, P, P, 1, ws, b,
                                                  None) == lin.E_INVALID
    for bad in SIZES:
        assert lin.fql_w4_matmul_workspace_bytes(1, *bad) == 0 and lin.fql_w4_gated_workspace_bytes(0, *bad) == 0
        assert lin.fql_w4_matmul_backward_workspace_bytes(*bad) == 0
        assert lin.fql_w4_gated_backward_workspace_bytes(*bad) == 0


def cpu_weight(n=8, k=64, group=32):
    return dict(codes=torch.zeros(n, (k + 1) // 2, dtype=torch.uint8), scale=torch.ones(n, -(-k // group)),
                zp=torch.zeros(n, -(-k // group), dtype=torch.int32))


def test_helper_refusals(lin):
    from fake_quant_amd.fq import FqError
    x, w = torch.zeros(4, 64), cpu_weight()

    def refused(status, fn, *a, **kw):
        with pytest.raises(FqError) as e:
            fn(*a, **kw)
        assert e.value.status == status, e.value

    refused(lin.E_INVALID, lin.w4_matmul, x, w, 32)  # not on a GPU
    refused(lin.E_INVALID, lin.w4_matmul, x[0], w, 32)
    refused(lin.E_INVALID, lin.w4_matmul, x, w, 0)
    refused(lin.E_UNSUPPORTED, lin.w4_matmul, x.half(), w, 32)
    refused(lin.E_DIM, lin.w4_matmul, x, w, 64)
    refused(lin.E_DIM, lin.w4_matmul, x, cpu_weight(k=66), 32)
    refused(lin.E_UNSUPPORTED, lin.w4_matmul, x, dict(w, scale=w["scale"].double()), 32)
    refused(lin.E_DIM, lin.w4_gated, x, w, cpu_weight(n=9), 32)
    refused(lin.E_UNSUPPORTED, lin.w4_gated, x, w, w, 32, "relu")
    refused(lin.E_DIM, lin.w4_matmul_backward, torch.zeros(4, 9), x, w, 32)
    refused(lin.E_DIM, lin.w4_matmul_backward, torch.zeros(4, 8).bfloat16(), x, w, 32)
    refused(lin.E_UNSUPPORTED, lin.w4_matmul_backward, torch.zeros(4, 8), x, w, 32, dw_dtype=torch.float16)
    d = torch.zeros(4, 8)
    refused(lin.E_DIM, lin.w4_gated_backward, d, x, d, torch.zeros(3, 8), w, w, 32)


def test_workspace_refusals_of_tiles(lin):
    """Sizes whose kernels need a workspace, beyond test_workspace_refusals."""
    w, _ = weights(lin)
    m, n, k, g = 2100, 2000, 72, 32
    calls = [
        (lin.fql_w4_matmul_workspace_bytes(0, m, n, k, g),
         lambda ws, b: lin._lib.fql_w4_matmul(P, 0, m, n, k, g, w, P, ws, b, None)),
        (lin.fql_w4_matmul_workspace_bytes(1, m, n, 77, g),
         lambda ws, b: lin._lib.fql_w4_matmul(P, 1, m, n, 77, g, w, P, ws, b, None)),
        (lin.fql_w4_gated_workspace_bytes(0, m, n, k, g),
         lambda ws, b: lin._lib.fql_w4_gated(P, 0, m, n, k, g, 0, w, w, P, None, None, ws, b, None)),
        (lin.fql_w4_matmul_backward_workspace_bytes(m, 77, k, g),
         lambda ws, b: lin._lib.fql_w4_matmul_backward(P, P, 1, m, 77, k, g, w, P, P, 0, ws, b, None)),
        (lin.fql_w4_gated_backward_workspace_bytes(m, n, k, g),
         lambda ws, b: lin._lib.fql_w4_gated_backward(P, P, P, P, 1, m, n, k, g, 0, w, w, P, P, P, 1, ws, b, None)),
    ]
    for need, call in calls:
        assert need > 0 and need % 16 == 0
        for ws, b in ((None, need), (P, need - 1), (P + 8, need)):
            assert call(ws, b) == lin.E_INVALID
