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


def block_bwd(rows, parts=3, dr=None, dn=None, b=None, stats=(None, None, None, None), dx=None, db=None, vec=(None,) * 5, ws=None, n=0, w=A, gate_rows=0):
    w1, w2 = (w if parts & 1 else None), (w if parts & 2 else None)
    return moe.lib().moe_block_norm_backward(1, parts, 0, 0, 0, rows, 64, dr, 64, dn, 64, dr, 64, b, 64, 1.0, 1.0, w1, None, w if gate_rows else None, gate_rows, w2, *stats, dx, 64,
                                             db, 64, *vec, ws, n, None)


def test_block_norm_backward():
    for parts in range(4):
        for gate_rows in (0, 1, 2):
            assert block_bwd(0, parts, gate_rows=gate_rows) == OK
    assert block_bwd(2, dr=A, dn=A, b=A, stats=(None, A, None, A)) == NULL   # rows, but no gradient is asked for
    assert block_bwd(0, vec=(None, A, None, None, None)) == NULL            # zeros for a vector need a workspace
    assert block_bwd(0, 4) == SHAPE and block_bwd(-1) == SHAPE


def norm_bwd(rows, kind=0, dy=None, x=None, w=A, mean=None, rstd=None, dx=None, dw=None, db=None, ws=None, n=0):
    return moe.lib().moe_norm_backward(kind, 0, 0, rows, 64, dy, 64, x, 64, w, mean, rstd, dx, 64, dw, db, ws, n, None)


def test_norm_backward():
    for kind in (0, 1):
        assert norm_bwd(0, kind) == OK and norm_bwd(0, kind, w=None) == OK
    assert norm_bwd(2, dy=A, x=A, mean=A, rstd=A) == NULL   # rows, but no gradient is asked for
    assert norm_bwd(0, dw=A) == NULL                        # zeros for dweight need a workspace
    assert norm_bwd(0, 2) == SHAPE and norm_bwd(-1) == SHAPE and norm_bwd(0, 1, db=A) == SHAPE
