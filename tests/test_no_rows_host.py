"""Backward passes over no rows where only gradients of rows are wanted: an empty tensor's address is NULL, so every gradient is
NULL, and there is nothing to do.  Needs no GPU: the calls end before any device work."""
import token_dispatch_grouped_route_amd as moe

OK, NULL, SHAPE = 0, -1, -2
A = 0x10000   # an address that no check reads through


def linear_bwd(M, act=0, dy=None, x=None, w=A, z=None, dx=None, dw=None, db=None, ws=None, n=0, lddx=64):
    return moe.lib().moe_linear_backward(0, 0, 0, act, M, 32, 64, dy, 32, x, 64, w, 64, 0, z, 64, dx, lddx, dw, 64, db, ws, n, None)


def test_linear_backward():
    for act in range(5):
        assert linear_bwd(0, act) == OK
        assert linear_bwd(0, act, w=None) == OK
    assert linear_bwd(1, dy=A, x=A) == NULL          # rows, but no gradient is asked for
    assert linear_bwd(0, dw=A) == NULL               # zeros for dw need a workspace
    assert linear_bwd(0, 5) == SHAPE and linear_bwd(-1) == SHAPE
