"""The linear map's backward where the kept z is infinite.  z is kept in the operands' type, so a finite z beyond fp16's range
(65504) is kept as infinity; the slope there is the activation's limit: 1 or 0, never NaN."""
import pytest
import torch

import token_dispatch_grouped_route_amd as moe

pytestmark = pytest.mark.gpu
INF = float("inf")


def identity(n, by_column):
    w = torch.eye(n, device="cuda").half()
    return w.t() if by_column else w


@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
def test_slope_at_infinity(act):
    z = torch.tensor([INF, -INF, 65504.0, -65504.0, 129.0, -129.0, 127.0, -127.0], device="cuda").half().repeat(5, 1)
    dy = torch.arange(1, 6, device="cuda").half()[:, None].expand(5, 8).contiguous()
    for by_column in (False, True):
        # W is the identity, so dx is dz: dy where z is positive, else 0 (the slopes at |z| >= 127 are 1 and 0 to within 2^-100)
        dx, _, db = moe.linear_backward(dy, torch.zeros_like(z), identity(8, by_column), z, act=act, bias=True)
        want = torch.where(z > 0, dy, 0)
        assert torch.equal(dx.abs(), want), (act, dx)
        assert torch.equal(db.abs(), want.sum(0))


def test_swiglu_at_infinity():
    gate = torch.tensor([INF, -INF, -65504.0, -129.0, -127.0, 129.0, 2.0, 0.0], device="cuda").half().repeat(3, 1)
    up = torch.full_like(gate, 0.5)
    dy = torch.ones_like(gate)
    # the bias's gradient is the sum of dz over the rows, column by column (in dx an infinite dz meets the zeros of W)
    db = moe.linear_backward(dy, torch.zeros(3, 16, device="cuda").half(), identity(16, False), torch.cat((gate, up), 1), act="swiglu", bias=True)[2]
    assert (db[[0, 5]] == 3 * 0.5).all()                           # up times the slope 1
    assert not db[1:5].any() and not db[9:13].any()                # slope and silu are 0
    assert db[8] == INF                                            # silu(inf) = inf: dup follows the z that was kept
    assert torch.isfinite(db[[5, 6, 7, 13, 14, 15]]).all()


@pytest.mark.parametrize("act", [None, "relu", "gelu", "silu"])
def test_map_beyond_fp16(act):
    """z reaches 2^17, y is fp32: the gradients are dy's where z is positive, all finite."""
    M, K, N = 40, 64, 48
    x = torch.full((M, K), 128.0, device="cuda").half()
    x[::2] *= -1
    w = torch.full((K, N), 16.0, device="cuda").half().requires_grad_()   # z = +-2^17
    x.requires_grad_()
    y = moe.linear(x, w, act=act, out_dtype=torch.float32)
    assert (y[1::2] == 2.0 ** 17).all()
    y.backward(torch.full_like(y, 2.0 ** -6))
    slope = (x.detach() > 0).double() if act else torch.ones(M, K, device="cuda", dtype=torch.float64)
    # powers of two and sums below 2^11 of them: exact in fp32 and fp16
    assert torch.equal(x.grad.double(), slope * (N * 16.0 * 2.0 ** -6))
    assert torch.equal(w.grad.double(), ((x.detach().double() * slope).sum(0)[:, None] * 2.0 ** -6).expand(K, N))


def test_nan_stays():
    z = torch.full((2, 8), float("nan"), device="cuda").half()
    for act in ("gelu", "silu"):
        dx, _, _ = moe.linear_backward(torch.ones_like(z), torch.zeros_like(z), identity(8, False), z, act=act)
        assert torch.isnan(dx).all()
