"""Argument checks of the operators around the expert layer (row norm, router, 4-bit products) that
need no GPU: every refusal comes back as a status before any device work, and the workspace functions
are pure functions of the sizes."""
import ctypes

import pytest
import torch

import token_dispatch_grouped_route_amd as moe

NULL, SHAPE, WORKSPACE, ALIGN, DEVICE = -1, -2, -4, -5, -7
A, B, C = 0x10000, 0x20000, 0x30000   # addresses that no check reads through


def norm_fwd(kind=0, dtype=0, wdtype=0, rows=4, cols=64, x=A, ldx=64, w=B, b=B, eps=1e-5, y=C, ldy=64, mean=A, rstd=A):
    return moe.lib().moe_norm_forward(kind, dtype, wdtype, rows, cols, x, ldx, w, b, eps, y, ldy, mean, rstd, None)


def norm_bwd(kind=0, dtype=0, wdtype=0, rows=4, cols=64, dy=A, lddy=64, x=A, ldx=64, w=B, mean=B, rstd=B, dx=C, lddx=64, dw=C, db=C, ws=A, n=1 << 20):
    return moe.lib().moe_norm_backward(kind, dtype, wdtype, rows, cols, dy, lddy, x, ldx, w, mean, rstd, dx, lddx, dw, db, ws, n, None)


@pytest.mark.parametrize("bad,status", [
    (dict(kind=2), SHAPE), (dict(dtype=3), SHAPE), (dict(wdtype=1), SHAPE), (dict(rows=-1), SHAPE), (dict(cols=0), SHAPE), (dict(cols=32769, ldx=40000, ldy=40000), SHAPE),
    (dict(ldx=63), SHAPE), (dict(ldy=63), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(kind=1), SHAPE),
    (dict(x=None), NULL), (dict(y=None), NULL), (dict(y=A), SHAPE), (dict(x=A + 1), ALIGN), (dict(y=C + 1), ALIGN), (dict(w=B + 1), ALIGN),
    (dict(mean=A + 2), ALIGN), (dict(rstd=A + 2), ALIGN), (dict(ldx=1 << 62), SHAPE), (dict(dtype=2, wdtype=0), SHAPE),
])
def test_norm_forward_refusals(bad, status):
    assert norm_fwd(**bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(kind=1), SHAPE), (dict(dx=None, dw=None, db=None), NULL), (dict(mean=None), NULL), (dict(rstd=None), NULL), (dict(dy=None), NULL),
    (dict(x=None), NULL), (dict(dx=A), SHAPE), (dict(lddx=63), SHAPE), (dict(lddy=1), SHAPE), (dict(ws=None), NULL), (dict(ws=A + 128), ALIGN),
    (dict(n=100), WORKSPACE), (dict(dw=C + 1), ALIGN), (dict(rows=-3), SHAPE),
])
def test_norm_backward_refusals(bad, status):
    assert norm_bwd(**bad) == status


def test_norm_without_rows_is_no_work():
    assert norm_fwd(rows=0, x=None, y=None) == 0
    assert norm_bwd(rows=0, x=None, dy=None, mean=None, rstd=None, dw=None, db=None) == 0


def test_norm_workspace():
    f = moe.lib().moe_norm_workspace_bytes
    assert f(3, 10, 64) == 0 and f(0, -1, 64) == 0 and f(0, 10, 0) == 0 and f(0, 10, 32769) == 0
    assert f(0, 0, 64) > 0
    for dtype in (0, 1, 2):
        for cols in (1, 64, 2048, 7168, 32768):
            sizes = [f(dtype, rows, cols) for rows in (1, 8, 9, 1000, 10 ** 5, 10 ** 9)]
            assert sizes == sorted(sizes) and all(s % 512 == 0 and s > 0 for s in sizes)
            assert sizes[0] >= 2 * 4 * cols and sizes[-1] == sizes[-2]   # a bound that the rows do not move


def route(dtype=2, T=4, E=64, k=8, logits=A, ld=64, bias=B, score=0, renorm=1, n_group=1, topk_group=1, scale=1.0, idx=C, w=C):
    return moe.lib().moe_route_topk(dtype, T, E, k, logits, ld, bias, score, renorm, n_group, topk_group, scale, idx, w, None)


def route_bwd(dtype=2, T=4, E=64, k=8, logits=A, ld=64, idx=B, dw=B, score=0, renorm=1, scale=1.0, out=C, ldd=64):
    return moe.lib().moe_route_topk_backward(dtype, T, E, k, logits, ld, idx, dw, score, renorm, scale, out, ldd, None)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=3), SHAPE), (dict(T=-1), SHAPE), (dict(T=(1 << 25) + 1), SHAPE), (dict(E=0), SHAPE), (dict(E=1025, ld=1025), SHAPE), (dict(k=0), SHAPE), (dict(k=33), SHAPE),
    (dict(E=4, k=5), SHAPE), (dict(ld=63), SHAPE), (dict(score=2), SHAPE), (dict(n_group=0), SHAPE), (dict(n_group=17), SHAPE), (dict(n_group=3), SHAPE),
    (dict(n_group=4, topk_group=5), SHAPE), (dict(n_group=4, topk_group=0), SHAPE), (dict(logits=None), NULL), (dict(idx=None), NULL), (dict(w=None), NULL),
    (dict(logits=A + 2), ALIGN), (dict(bias=B + 2), ALIGN), (dict(idx=C + 1), ALIGN),
])
def test_route_refusals(bad, status):
    assert route(**bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(k=33), SHAPE), (dict(T=(1 << 25) + 1), SHAPE), (dict(ldd=63), SHAPE), (dict(score=-1), SHAPE), (dict(idx=None), NULL), (dict(dw=None), NULL), (dict(out=None), NULL),
    (dict(out=A), SHAPE), (dict(out=C + 2), ALIGN),
])
def test_route_backward_refusals(bad, status):
    assert route_bwd(**bad) == status


def test_route_without_tokens_is_no_work():
    assert route(T=0, logits=None, idx=None, w=None) == 0
    assert route_bwd(T=0, logits=None, idx=None, dw=None, out=None) == 0


def quantize(wdtype=2, dtype=0, E=2, K=256, N=64, group=64, w=A, codes=B, scales=C, zeros=None):
    return moe.lib().moe_w4_quantize(wdtype, dtype, E, K, N, group, w, codes, scales, zeros, None)


def linear(dtype=0, M=2, N=64, K=256, group=64, x=A, ldx=256, codes=B, scales=C, zeros=None, y=C, ldy=64):
    return moe.lib().moe_w4_linear(dtype, M, N, K, group, x, ldx, codes, scales, zeros, y, ldy, None)


@pytest.mark.parametrize("bad,status", [
    (dict(wdtype=3), SHAPE), (dict(dtype=2), SHAPE), (dict(E=0), SHAPE), (dict(group=16), SHAPE), (dict(group=96, K=288), SHAPE), (dict(K=200), SHAPE),
    (dict(K=65536), SHAPE), (dict(N=0), SHAPE), (dict(N=(1 << 28) + 1), SHAPE), (dict(w=None), NULL), (dict(codes=None), NULL), (dict(scales=None), NULL), (dict(codes=B + 8), ALIGN), (dict(zeros=B + 4), ALIGN),
])
def test_quantize_refusals(bad, status):
    assert quantize(**bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), SHAPE), (dict(M=-1), SHAPE), (dict(M=(1 << 20) + 1), SHAPE), (dict(M=1 << 20, N=2049, ldy=2049), SHAPE), (dict(N=0), SHAPE), (dict(group=48), SHAPE), (dict(K=0), SHAPE), (dict(ldx=255), SHAPE),
    (dict(ldy=63), SHAPE), (dict(x=None), NULL), (dict(codes=None), NULL), (dict(y=None), NULL), (dict(x=A + 8), ALIGN), (dict(ldx=260), ALIGN),
    (dict(scales=C + 2), ALIGN), (dict(y=C + 1), ALIGN),
])
def test_linear_refusals(bad, status):
    assert linear(**bad) == status


def forward(s, dtype=0, group=128, x=A, idx=A, tw=A, w1=B, s1=B, z1=None, w2=B, s2=B, z2=None, ws=C, n=1 << 30, y=A):
    return moe.lib().moe_forward_w4(ctypes.byref(s) if s is not None else None, dtype, group, x, idx, tw, w1, s1, z1, w2, s2, z2, ws, n, y, None)


def test_forward_w4_refusals():
    s = moe.make_shape(4, 256, 128, 8, 8, 2, block_m=64)
    assert forward(None) == NULL
    for bad, status in [(dict(dtype=2), SHAPE), (dict(group=256), SHAPE), (dict(group=24), SHAPE), (dict(x=None), NULL), (dict(idx=None), NULL), (dict(w1=None), NULL),
                        (dict(s2=None), NULL), (dict(ws=None), NULL), (dict(y=None), NULL), (dict(ws=C + 64), ALIGN), (dict(w2=B + 4), ALIGN), (dict(z1=B + 8), ALIGN),
                        (dict(x=A + 2), ALIGN), (dict(n=64), WORKSPACE)]:
        assert forward(s, **bad) == status, bad
    for change in (dict(T=2049), dict(train=1), dict(H=100), dict(k=33), dict(EL=0)):
        t = moe.make_shape(4, 256, 128, 8, 8, 2, block_m=64)
        for f, v in change.items():
            setattr(t, f, v)
        assert forward(t) == SHAPE and moe.lib().moe_w4_workspace_bytes(ctypes.byref(t)) == 0
    assert moe.w4_workspace_bytes(s) >= 8 * (128 * 2 + 256 * 4)
    t = moe.make_shape(2048, 256, 128, 8, 8, 2, block_m=64)
    assert moe.w4_workspace_bytes(t) >= 4096 * (128 * 2 + 256 * 4)
    with pytest.raises(moe.MoeError):
        moe.w4_workspace_bytes(moe.make_shape(2049, 256, 128, 8, 8, 2, block_m=64))


def test_binding_refuses_host_tensors():
    x = torch.ones(2, 64)
    for call in (lambda: moe.norm_forward(x), lambda: moe.route_topk(x, 2), lambda: moe.w4_quantize(x.t().contiguous()),
                 lambda: moe.w4_linear(x, x, x), lambda: moe.layer_norm(x), lambda: moe.router(x, 2), lambda: moe.norm_forward(None)):
        with pytest.raises(moe.MoeError):
            call()


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real")
def test_without_a_gpu_valid_calls_report_the_device():
    assert norm_fwd() == DEVICE and norm_bwd() == DEVICE and route() == DEVICE and route_bwd() == DEVICE
    assert quantize() == DEVICE and linear() == DEVICE
    assert forward(moe.make_shape(4, 256, 128, 8, 8, 2, block_m=64)) == DEVICE


def test_route_choice_by_score_is_a_flag_of_the_score():
    for good in (0x100, 0x101):
        assert route(T=0, score=good, logits=None, idx=None, w=None) == 0
        assert route_bwd(T=0, score=good, logits=None, idx=None, dw=None, out=None) == 0
    for bad in (0x102, 0x200, 0x301, -1):
        assert route(score=bad) == SHAPE and route_bwd(score=bad) == SHAPE
