"""Argument checks of the calls around the expert layer that come before any
CUDA call (no GPU needed)."""
import ctypes

import pytest

from moe_expert_grouped_split_gb300 import binding as B
from moe_expert_grouped_split_gb300.build import build

INVALID, UNSUPPORTED = -1, -5
P = 4096  # a 16-byte aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    build()
    return B.lib()


def norm(lib, x=P, x_stride=64, residual=P, residual_out=P, weight=P, eps=1e-6, rows=4, H=64, out=P, codes=P,
         row_scale=P):
    return lib.dwdp_add_rmsnorm(x, x_stride, residual, residual_out, weight, eps, rows, H, out, codes, row_scale, None)


@pytest.mark.parametrize("bad, code", [
    (dict(rows=-1), INVALID), (dict(rows=1 << 31), INVALID),
    (dict(H=0), UNSUPPORTED), (dict(H=60), UNSUPPORTED), (dict(H=32776, x_stride=32776), UNSUPPORTED),
    (dict(x_stride=56), INVALID), (dict(x_stride=68), INVALID), (dict(x_stride=-64), INVALID),
    (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(residual=None), INVALID), (dict(residual_out=None), INVALID),
    (dict(codes=None), INVALID), (dict(row_scale=None), INVALID),
    (dict(x=None), INVALID), (dict(weight=None), INVALID), (dict(out=None), INVALID),
    (dict(x=P + 2), INVALID), (dict(residual=P + 8), INVALID), (dict(residual_out=P + 8), INVALID),
    (dict(weight=P + 4), INVALID), (dict(out=P + 2), INVALID), (dict(codes=P + 1), INVALID),
    (dict(row_scale=P + 4), INVALID)], ids=str)
def test_add_rmsnorm_refuses(lib, bad, code):
    assert norm(lib, **bad) == code
    assert B.dwdp_last_error(None)


def test_add_rmsnorm_of_no_rows_reads_nothing(lib):
    assert norm(lib, rows=0, x=None, weight=None, out=None) == 0


def test_lora_workspace(lib):
    for bad in ((-1, 64, 64, 16), (4, 60, 64, 16), (4, 64, 0, 16), (4, 64, 64, 0), (4, 64, 64, 12),
                (4, 64, 64, 136), (4, (1 << 20) + 8, 64, 16), (4, 64, (1 << 20) + 8, 16), ((1 << 30) + 1, 64, 64, 16)):
        assert B.dwdp_lora_workspace_bytes(*bad) == 0
    last = 0
    for T in (0, 1, 17, 128, 129, 8192, 100000):
        n = B.dwdp_lora_workspace_bytes(T, 7168, 7168, 16)
        assert n >= max(256, last)
        last = n


def test_calls_without_a_context(lib):
    how = B.scoring()
    out = B.dwdp_route_out()
    assert lib.dwdp_route_scored(None, P, 4, P, None, ctypes.byref(how), ctypes.byref(out), P, 1 << 20, None) == INVALID
    assert lib.dwdp_lora_add(None, P, 64, 4, 64, 64, P, P, P, 1, 16, P, P, 64, P, 64, P, 1 << 20, None) == INVALID
    assert lib.dwdp_moe_layer_codes(None, 0, 0, P, P, 4, ctypes.byref(out), P, P, 1 << 20, None) == INVALID
