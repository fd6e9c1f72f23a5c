"""Argument checks of the sandwich norm, its gradients, the balance loss and
the router's gradient that come before any CUDA call (no GPU needed)."""
import ctypes

import pytest

from moe_expert_grouped_split_gb300 import binding as B
from moe_expert_grouped_split_gb300.build import build

OK, INVALID, UNSUPPORTED = 0, -1, -5
P = 4096  # a 16-byte aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    build()
    return B.lib()


def how(pre=P, post=P, gate=P, row_offsets=P, n_groups=3, block_scale=1.0, residual_scale=1.0, eps=1e-6):
    return B.dwdp_sandwich(pre, post, gate, row_offsets, n_groups, block_scale, residual_scale, eps)


COMMON = ("pre", "post", "gate", "row_offsets", "n_groups", "block_scale", "residual_scale", "eps")


def norm(lib, x=P, x_stride=64, residual=P, rows=4, H=64, residual_out=P, out=P, codes=P, row_scale=P, x_codes=P,
         x_scale=P, h_codes=P, h_scale=P, rstd=P, **common):
    return lib.dwdp_sandwich_norm(ctypes.byref(how(**common)), x, x_stride, residual, rows, H, residual_out, out, codes,
                                  row_scale, x_codes, x_scale, h_codes, h_scale, rstd, None)


def grad(lib, x=P, x_stride=64, x_scale=P, h=P, h_scale=P, rstd=P, dout=P, dres=P, rows=4, H=64, dx=P, dresidual=P,
         dpost=P, dpre=P, dgate=P, ws=P, ws_bytes=1 << 30, **common):
    return lib.dwdp_sandwich_norm_grad(ctypes.byref(how(**common)), x, x_stride, x_scale, h, h_scale, rstd, dout, dres,
                                       rows, H, dx, dresidual, dpost, dpre, dgate, ws, ws_bytes, None)


SHARED = [
    (dict(rows=-1), INVALID), (dict(rows=1 << 31), INVALID), (dict(H=0), UNSUPPORTED), (dict(H=60), UNSUPPORTED),
    (dict(H=32776, x_stride=32776), UNSUPPORTED), (dict(x_stride=56), INVALID), (dict(x_stride=68), INVALID), (dict(x_stride=-64), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(eps=1e-31), INVALID),
    (dict(block_scale=float("inf")), INVALID), (dict(residual_scale=float("nan")), INVALID),
    (dict(n_groups=0), INVALID), (dict(n_groups=-1), INVALID), (dict(n_groups=B.MAX_GATES + 1), UNSUPPORTED),
    (dict(gate=None), INVALID), (dict(gate=None, n_groups=0), INVALID), (dict(gate=None, row_offsets=None), INVALID),
    (dict(row_offsets=None), INVALID),
    (dict(pre=P + 2), INVALID), (dict(post=P + 8), INVALID), (dict(gate=P + 4), INVALID),
    (dict(row_offsets=P + 4), INVALID), (dict(x=P + 2), INVALID), (dict(rstd=P + 8), INVALID), (dict(x=None), INVALID)]


@pytest.mark.parametrize("bad, code", SHARED + [
    (dict(codes=None), INVALID), (dict(row_scale=None), INVALID), (dict(x_codes=None), INVALID),
    (dict(x_scale=None), INVALID), (dict(h_codes=None), INVALID), (dict(h_scale=None), INVALID),
    (dict(out=None), INVALID), (dict(pre=None), INVALID), (dict(pre=None, out=None), INVALID),
    (dict(pre=None, out=None, codes=None, row_scale=None, residual_out=None), INVALID),
    (dict(residual=P + 8), INVALID), (dict(residual_out=P + 8), INVALID), (dict(out=P + 2), INVALID),
    (dict(codes=P + 1), INVALID), (dict(row_scale=P + 4), INVALID), (dict(x_codes=P + 8), INVALID),
    (dict(x_scale=P + 4), INVALID), (dict(h_codes=P + 8), INVALID), (dict(h_scale=P + 4), INVALID)], ids=str)
def test_sandwich_norm_refuses(lib, bad, code):
    assert norm(lib, **bad) == code
    assert B.dwdp_last_error(None)


@pytest.mark.parametrize("bad, code", SHARED + [
    (dict(h=None), INVALID), (dict(h=None, h_scale=None), INVALID), (dict(dout=None), INVALID),
    (dict(rstd=None), INVALID), (dict(pre=None), INVALID), (dict(pre=None, dpre=None), INVALID),
    (dict(pre=None, dpre=None, h=None, h_scale=None), INVALID),
    (dict(pre=None, dpre=None, h=None, h_scale=None, dout=None, dres=None), INVALID),
    (dict(post=None), INVALID), (dict(gate=None, row_offsets=None, n_groups=0), INVALID),
    (dict(ws=None), INVALID), (dict(ws_bytes=100), INVALID), (dict(ws=P + 8), INVALID),
    (dict(x_scale=P + 4), INVALID), (dict(h=P + 8), INVALID), (dict(h_scale=P + 4), INVALID),
    (dict(dout=P + 8), INVALID), (dict(dres=P + 2), INVALID), (dict(dx=P + 8), INVALID),
    (dict(dresidual=P + 8), INVALID), (dict(dpost=P + 4), INVALID), (dict(dpre=P + 4), INVALID),
    (dict(dgate=P + 4), INVALID)], ids=str)
def test_sandwich_norm_grad_refuses(lib, bad, code):
    assert grad(lib, **bad) == code
    assert B.dwdp_last_error(None)


def test_calls_that_have_nothing_to_do(lib):
    nothing = dict(x=None, residual=None, residual_out=None, out=None, codes=None, row_scale=None, x_codes=None,
                   x_scale=None, h_codes=None, h_scale=None, rstd=None)
    assert norm(lib, rows=0, **nothing) == OK
    assert grad(lib, dx=None, dresidual=None, dpost=None, dpre=None, dgate=None, ws=None) == OK
    assert grad(lib, rows=0, dpost=None, dpre=None, dgate=None, ws=None) == OK


def test_no_structure(lib):
    assert lib.dwdp_sandwich_norm(None, P, 64, P, 4, 64, P, P, None, None, None, None, None, None, None, None) == INVALID


def test_workspaces(lib):
    for bad in ((-1, 64), (1 << 31, 64), (4, 0), (4, 60), (4, 32776)):
        assert B.dwdp_sandwich_grad_workspace_bytes(*bad) == 0
    for H in (8, 512, 7168, 8192, 32768):
        last = 0
        for rows in (0, 1, 17, 151, 153, 8192, (1 << 31) - 1):
            n = B.dwdp_sandwich_grad_workspace_bytes(rows, H)
            assert max(256, last) <= n <= 1 << 27
            last = n
    for bad in ((-1, 8, 1), ((1 << 30) + 1, 8, 1), (4, 0, 1), (4, 1025, 1), (4, 8, 0)):
        assert B.dwdp_balance_workspace_bytes(*bad) == 0
    for E in (1, 7, 64, 256, 1024):
        for T in (0, 1, 1000, 65536, 1 << 20):
            assert 256 <= B.dwdp_balance_workspace_bytes(T, E, 3) <= 1 << 28


def test_calls_without_a_context(lib):
    sc = B.scoring()
    assert lib.dwdp_balance_loss(None, P, P, 4, None, 1, ctypes.byref(sc), P, P, P, P, P, 1 << 20, None) == INVALID
    assert lib.dwdp_route_scored_grad(None, P, P, P, 4, None, 1, ctypes.byref(sc), P, P, P, P, 0, None) == INVALID


def test_biased_gradient_without_a_context(lib):
    sc = B.scoring()
    assert lib.dwdp_route_scored_biased_grad(None, P, P, P, P, 4, None, 1, ctypes.byref(sc), P, P, P, P, 0, None) == INVALID
