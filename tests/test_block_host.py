"""Argument checks of the dense operators of a block (linear map, block norm, few tokens) that need no GPU: every refusal comes back as a
status before any device work, and the workspace functions are pure functions of the sizes."""
import ctypes

import pytest
import torch

import token_dispatch_grouped_route_amd as moe

NULL, SHAPE, WORKSPACE, ALIGN, DEVICE = -1, -2, -4, -5, -7
A, B, C, D, E = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000   # addresses that no check reads through


def linear(dtype=0, bdtype=0, odtype=0, act=0, M=4, N=32, K=64, x=A, ldx=64, w=B, ldw=32, by_column=0, bias=C, res=C, ldr=32, y=D, ldy=32, z=E, ldz=32, ws=A, n=1 << 30):
    return moe.lib().moe_linear_forward(dtype, bdtype, odtype, act, M, N, K, x, ldx, w, ldw, by_column, bias, res, ldr, y, ldy, z, ldz, ws, n, None)


def linear_bwd(dtype=0, bdtype=0, odtype=0, act=3, M=4, N=32, K=64, dy=A, lddy=32, x=A, ldx=64, w=B, ldw=32, by_column=0, z=C, ldz=32, dx=D, lddx=64, dw=E, lddw=32,
               db=D + 4096, ws=A, n=1 << 30):
    return moe.lib().moe_linear_backward(dtype, bdtype, odtype, act, M, N, K, dy, lddy, x, ldx, w, ldw, by_column, z, ldz, dx, lddx, dw, lddw, db, ws, n, None)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), SHAPE), (dict(dtype=1), SHAPE), (dict(odtype=1), SHAPE), (dict(bdtype=3), SHAPE), (dict(act=5), SHAPE), (dict(act=-1), SHAPE), (dict(M=-1), SHAPE),
    (dict(M=(1 << 24) + 1), SHAPE), (dict(N=0), SHAPE), (dict(N=(1 << 20) + 1, ldw=1 << 21, ldy=1 << 21, ldr=1 << 21, ldz=1 << 21), SHAPE), (dict(K=0), SHAPE),
    (dict(M=1 << 24, N=1 << 20, ldw=1 << 20, ldy=1 << 20, ldr=1 << 20, ldz=1 << 20), SHAPE), (dict(ldx=63), SHAPE), (dict(ldw=31), SHAPE), (dict(by_column=1), SHAPE),
    (dict(ldy=31), SHAPE), (dict(ldr=31), SHAPE), (dict(ldz=31), SHAPE), (dict(act=4, ldw=64), SHAPE), (dict(x=None), NULL), (dict(w=None), NULL), (dict(y=None), NULL),
    (dict(ws=None, K=8192, ldx=8192), NULL), (dict(y=A), SHAPE), (dict(y=B), SHAPE), (dict(z=A), SHAPE), (dict(z=D), SHAPE), (dict(z=C), SHAPE), (dict(res=D, ldr=40), SHAPE), (dict(x=A + 1), ALIGN),
    (dict(w=B + 1), ALIGN), (dict(bias=C + 1), ALIGN), (dict(bdtype=2, bias=C + 2), ALIGN), (dict(odtype=2, y=D + 2), ALIGN), (dict(odtype=2, res=C + 2), ALIGN), (dict(ws=A + 64), ALIGN), (dict(n=8, K=8192, ldx=8192), WORKSPACE),
])
def test_linear_refusals(bad, status):
    assert linear(**bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), SHAPE), (dict(act=5), SHAPE), (dict(lddy=31), SHAPE), (dict(ldx=63), SHAPE), (dict(ldw=31), SHAPE), (dict(lddw=31), SHAPE), (dict(lddx=63), SHAPE), (dict(ldz=31), SHAPE),
    (dict(dx=None, dw=None, db=None), NULL), (dict(dy=None), NULL), (dict(x=None), NULL), (dict(w=None), NULL), (dict(z=None), NULL), (dict(ws=None), NULL),
    (dict(dx=A), SHAPE), (dict(dw=B), SHAPE), (dict(dx=C), SHAPE), (dict(db=B), SHAPE), (dict(dx=D + 1), ALIGN), (dict(dw=E + 1), ALIGN), (dict(z=C + 1), ALIGN), (dict(ws=A + 8), ALIGN), (dict(n=8), WORKSPACE),
    (dict(M=1 << 24, K=1 << 20, ldx=1 << 20, lddx=1 << 20), SHAPE),
])
def test_linear_backward_refusals(bad, status):
    assert linear_bwd(**bad) == status


def test_linear_without_rows():
    assert linear(M=0, x=None, y=None, ws=None) == 0
    assert linear_bwd(M=0, dw=None, db=None, dy=None, x=None, ws=None) == 0


def test_linear_workspace():
    f = moe.lib().moe_linear_workspace_bytes
    for bad in ((5, 4, 32, 64), (0, -1, 32, 64), (0, 4, 0, 64), (0, 4, 32, 0), (0, 1 << 24, 1 << 20, 64)):
        assert f(*bad, 0) == 0 and f(*bad, 1) == 0
    for M, N, K in ((0, 32, 64), (1, 4096, 7168), (48, 7168, 2048), (8192, 4096, 7168), (1003, 1407, 2049), (1 << 24, 128, 128)):
        for act, C in ((0, N), (4, 2 * N)):
            assert f(act, M, N, K, 0) % 256 == 0 and f(act, M, N, K, 0) > 0
            assert f(act, M, N, K, 1) >= 2 * M * C
    with pytest.raises(moe.MoeError):
        moe.linear_workspace_bytes(4, 0, 64)


def test_binding_refuses_host_tensors():
    x = torch.ones(2, 64, dtype=torch.bfloat16)
    for call in (lambda: moe.linear(x, x.t()), lambda: moe.linear_forward(x, x.t()), lambda: moe.linear_backward(x, x, x.t()), lambda: moe.linear_forward(None, x)):
        with pytest.raises(moe.MoeError):
            call()


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real")
def test_without_a_gpu_valid_calls_report_the_device():
    assert linear() == DEVICE and linear_bwd() == DEVICE
    assert linear(res=D) == DEVICE and linear(by_column=1, ldw=64) == DEVICE and linear(act=4, ldw=64, ldz=64) == DEVICE


def block(kind=1, parts=3, dtype=0, sdtype=0, wdtype=0, rows=6, cols=64, x=A, ldx=64, b=B, ldb=64, w1=C, c1=None, gate=C, gate_rows=2, w2=C, c2=None, eps=1e-5, r=D, ldr=64, n=E, ldn=64,
          stats=(None, A, None, A)):
    return moe.lib().moe_block_norm_forward(kind, parts, dtype, sdtype, wdtype, rows, cols, x, ldx, b, ldb, 1.0, 1.0, w1, c1, gate, gate_rows, w2, c2, eps, r, ldr, n, ldn, *stats, None)


def block_bwd(kind=1, parts=3, dtype=0, sdtype=0, wdtype=0, rows=6, cols=64, dr=A, lddr=64, dn=A, lddn=64, r=B, ldr=64, b=B, ldb=64, w1=C, c1=None, gate=C, gate_rows=2, w2=C,
              stats=(None, A, None, A), dx=D, lddx=64, db=E, lddb=64, vec=(D + 4096, D + 8192, None, E + 4096, None), ws=A, size=1 << 24):
    return moe.lib().moe_block_norm_backward(kind, parts, dtype, sdtype, wdtype, rows, cols, dr, lddr, dn, lddn, r, ldr, b, ldb, 1.0, 1.0, w1, c1, gate, gate_rows, w2, *stats, dx, lddx, db,
                                             lddb, *vec, ws, size, None)


@pytest.mark.parametrize("bad,status", [
    (dict(kind=2), SHAPE), (dict(parts=4), SHAPE), (dict(dtype=3), SHAPE), (dict(sdtype=1), SHAPE), (dict(wdtype=1), SHAPE), (dict(rows=-1), SHAPE), (dict(cols=0), SHAPE),
    (dict(cols=32769, ldx=40000, ldb=40000, ldr=40000, ldn=40000), SHAPE), (dict(ldx=63), SHAPE), (dict(ldb=63), SHAPE), (dict(ldr=63), SHAPE), (dict(ldn=63), SHAPE), (dict(eps=-1.0), SHAPE),
    (dict(eps=float("nan")), SHAPE), (dict(c1=A), SHAPE), (dict(c2=A), SHAPE), (dict(parts=2), SHAPE), (dict(parts=1), SHAPE), (dict(gate_rows=4), SHAPE), (dict(gate_rows=0), SHAPE),
    (dict(gate=None), SHAPE), (dict(x=None), NULL), (dict(b=None), NULL), (dict(r=None), NULL), (dict(n=None), NULL), (dict(r=B), SHAPE), (dict(n=A), SHAPE), (dict(n=B), SHAPE), (dict(n=D), SHAPE),
    (dict(r=A, ldr=72), SHAPE), (dict(x=A + 1), ALIGN), (dict(gate=C + 1), ALIGN), (dict(w2=C + 1), ALIGN), (dict(sdtype=2, x=A + 2), ALIGN), (dict(stats=(None, A + 2, None, A)), ALIGN),
])
def test_block_norm_refusals(bad, status):
    assert block(**bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(parts=4), SHAPE), (dict(lddr=63), SHAPE), (dict(lddn=63), SHAPE), (dict(ldr=63), SHAPE), (dict(ldb=63), SHAPE), (dict(lddx=63), SHAPE), (dict(lddb=63), SHAPE),
    (dict(parts=1, w2=None), SHAPE), (dict(parts=2, w1=None), SHAPE), (dict(vec=(D, D, A, None, None)), SHAPE), (dict(gate=None, gate_rows=0), SHAPE),
    (dict(dx=None, db=None, vec=(None,) * 5), NULL), (dict(dr=None, dn=None), NULL), (dict(r=None), NULL), (dict(b=None), NULL), (dict(stats=(None, None, None, A)), NULL),
    (dict(stats=(None, A, None, None)), NULL), (dict(kind=0), NULL), (dict(ws=None), NULL), (dict(dx=A), SHAPE), (dict(db=B), SHAPE), (dict(db=D), SHAPE), (dict(ws=A + 64), ALIGN),
    (dict(dx=D + 1), ALIGN), (dict(vec=(D + 1, None, None, None, None)), ALIGN), (dict(size=64), WORKSPACE),
])
def test_block_norm_backward_refusals(bad, status):
    assert block_bwd(**bad) == status


def test_block_norm_without_rows():
    assert block(rows=0, x=None, b=None, r=None, n=None) == 0
    assert block_bwd(rows=0, dr=None, dn=None, r=None, b=None, vec=(None,) * 5, ws=None) == 0


def test_block_norm_workspace():
    f = moe.lib().moe_block_norm_workspace_bytes
    assert f(3, 6, 64, 0) == 0 and f(0, -1, 64, 0) == 0 and f(0, 6, 0, 0) == 0 and f(0, 6, 32769, 0) == 0 and f(0, 6, 64, 4) == 0 and f(0, 6, 64, -1) == 0
    for dtype in (0, 1, 2):
        for cols in (1, 63, 64, 2048, 7168, 8192, 8193, 32768):
            for rows in (0, 1, 16, 17, 1003, 8192, 65536, 10 ** 7):
                n = f(dtype, rows, cols, 0)
                wide = 16 * rows if cols < 8 or cols > 8192 else 0
                assert n > 0 and n % 256 == 0 and n <= wide + 4 * 4 * (2100 * max(cols, 512) + 512)   # a bound that the rows do not move, but for their means
                # a gate of few rows has partial sums of its own, one of many is written as it is
                assert f(dtype, rows, cols, 1) >= n and f(dtype, rows, cols, rows) <= n + 4 * 4 * 2100 * max(cols, 512)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real")
def test_block_norm_without_a_gpu():
    assert block() == DEVICE and block_bwd() == DEVICE and block(r=A) == DEVICE


def few(s, x=A, idx=A, tw=A, w1=B, w2=B, ws=C, n=1 << 30, y=D):
    return moe.lib().moe_forward_few(ctypes.byref(s) if s is not None else None, x, idx, tw, w1, w2, ws, n, y, None)


def test_forward_few_refusals():
    shape = lambda: moe.make_shape(4, 256, 128, 8, 8, 2, block_m=64)
    assert few(None) == NULL
    for bad, status in [(dict(x=None), NULL), (dict(idx=None), NULL), (dict(tw=None), NULL), (dict(w1=None), NULL), (dict(w2=None), NULL), (dict(ws=None), NULL), (dict(y=None), NULL),
                        (dict(ws=C + 64), ALIGN), (dict(w2=B + 8), ALIGN), (dict(x=A + 2), ALIGN), (dict(idx=A + 2), ALIGN), (dict(y=D + 8), ALIGN), (dict(n=64), WORKSPACE)]:
        assert few(shape(), **bad) == status, bad
    for change in (dict(T=2049), dict(train=1), dict(H=100), dict(k=33), dict(EL=0), dict(H=32768 + 128), dict(I=32768 + 128), dict(T=-1), dict(e_lo=1)):
        t = shape()
        for f, v in change.items():
            setattr(t, f, v)
        assert few(t) == SHAPE and moe.lib().moe_few_workspace_bytes(ctypes.byref(t)) == 0
    assert moe.few_workspace_bytes(shape()) >= 8 * (128 * 2 + 256 * 4)
    with pytest.raises(moe.MoeError):
        moe.few_workspace_bytes(moe.make_shape(2049, 256, 128, 8, 8, 2, block_m=64))
    if not torch.cuda.is_available():
        assert few(shape()) == DEVICE
