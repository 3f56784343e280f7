"""The operators around the sync on the CPU: the library exports what
include/ddp_train.h declares, every declaration is documented, and bad
arguments are refused before anything touches a GPU."""

import ctypes
import os
import re

import pytest

from conftest import ROOT

rar = pytest.importorskip("ring_all_reduce_ddp_amd")

HEADER = os.path.join(ROOT, "include", "ddp_train.h")


def declarations():
    """(name, the text before its declaration)."""
    text = open(HEADER).read()
    body = text[text.index('extern "C" {'):]
    out, prev = [], 0
    for m in re.finditer(r"^(?:int|void) (ddp_[a-z0-9_]+)\s*\([^;]*\)\s*;", body, flags=re.M | re.S):
        out.append((m.group(1), body[prev:m.start()]))
        prev = m.end()
    return out


def test_exports_every_declared_symbol():
    names = [n for n, _ in declarations()]
    assert len(names) == len(set(names)) and "ddp_grads_norm" in names
    lib = ctypes.CDLL(rar.LIB_PATH)
    assert [n for n in names if not hasattr(lib, n)] == []


def test_every_declaration_has_a_comment():
    assert [n for n, before in declarations() if "/*" not in before] == []


def refused(status, match):
    msg = rar.lib.ddp_last_error().decode()
    assert status == rar.DDP_EINVAL and match in msg, (status, msg)


def test_grads_arguments():
    lib = rar.lib
    out = ctypes.c_void_p(1)
    one = (ctypes.c_void_p * 1)(0x1000)
    n1 = (ctypes.c_int64 * 1)(4)
    refused(lib.ddp_grads_create(one, n1, 1, 0, None), "out is NULL")
    refused(lib.ddp_grads_create(one, n1, 1, 7, ctypes.byref(out)), "dtype")
    assert out.value is None
    refused(lib.ddp_grads_create(one, n1, -1, 0, ctypes.byref(out)), "negative")
    refused(lib.ddp_grads_create(None, n1, 1, 0, ctypes.byref(out)), "array is NULL")
    refused(lib.ddp_grads_create(one, (ctypes.c_int64 * 1)(-3), 1, 0, ctypes.byref(out)), "numels[0]")
    refused(lib.ddp_grads_create((ctypes.c_void_p * 1)(0x1001), n1, 1, 0, ctypes.byref(out)), "aligned")
    refused(lib.ddp_grads_create((ctypes.c_void_p * 1)(None), n1, 1, 0, ctypes.byref(out)), "grads[0] is NULL")
    refused(lib.ddp_grads_norm(None, 0, None, None), "grads is NULL")
    refused(lib.ddp_grads_clip(None, None, 1.0, None, None), "grads is NULL")
    lib.ddp_grads_free(None)


def test_adamw_arguments():
    lib = rar.lib
    out = ctypes.c_void_p(1)
    refused(lib.ddp_adamw_create(None, None, None, None, None, None, None, None), "out is NULL")
    refused(lib.ddp_adamw_create(None, None, None, None, None, None, None, ctypes.byref(out)), "grads is NULL")
    assert out.value is None
    refused(lib.ddp_adamw_step(None, 1e-3, 0.9, 0.99, 1e-8, 0.0, 0.0, None, None), "opt is NULL")
    lib.ddp_adamw_free(None)


A = 0x100000      # addresses that are never read: the refusals come first
FAR = 1 << 30



def forward_args(**change):
    """ddp_linear_forward on 4 x 8 outputs of 16 inputs, fp32, with everything asked for."""
    a = dict(x=A, ldx=16, w=A + FAR, ldw=16, bias=A + 2 * FAR, residual=A + 3 * FAR, ldr=8, y=A + 4 * FAR, ldy=8,
             z=A + 5 * FAR, ldz=8, M=4, N=8, K=16, dtype=0, act=1, workspace=A + 6 * FAR, workspace_bytes=FAR, stream=None)
    assert set(change) <= set(a)
    a.update(change)
    return list(a.values())


@pytest.mark.parametrize("change, match", [
    (dict(dtype=9), "unknown dtype"), (dict(act=-1), "unknown activation"), (dict(act=99), "unknown activation"),
    (dict(M=-1), "M, N and K"), (dict(N=-1), "M, N and K"), (dict(K=1 << 31), "M, N and K"),
    (dict(x=None), "x"), (dict(w=None), "w"), (dict(y=None), "y"),
    (dict(x=A + 2), "x is not aligned"), (dict(bias=A + 2 * FAR + 1), "bias is not aligned"),
    (dict(ldx=15), "leading dimension of x"), (dict(ldw=15), "leading dimension of w"), (dict(ldy=7), "leading dimension of y"),
    (dict(ldz=7), "leading dimension of z"), (dict(ldr=7), "leading dimension of residual"),
    (dict(ldw=(1 << 30) + 1), "over 2^22"), (dict(ldx=1 << 62), "over 2^22"),
    (dict(y=A + 16), "y overlaps x"), (dict(z=A + 4 * FAR), "overlaps"), (dict(residual=A + 4 * FAR + 4), "overlaps"),
    (dict(residual=A + 4 * FAR, ldr=9), "overlaps"), (dict(y=A + FAR + 508), "y overlaps w"),
])
def test_linear_forward_arguments(change, match):
    refused(rar.lib.ddp_linear_forward(*forward_args(**change)), match)


def test_linear_forward_of_nothing():
    assert rar.lib.ddp_linear_forward(*forward_args(M=0, x=None, y=None)) == rar.DDP_OK
    assert rar.lib.ddp_linear_forward(*forward_args(N=0, w=None, y=None)) == rar.DDP_OK


def backward_input_args(**change):
    a = dict(dz=A, lddz=8, w=A + FAR, ldw=16, z=A + 2 * FAR, ldz=16, add=A + 3 * FAR, ldadd=16, dx=A + 4 * FAR, lddx=16,
             M=4, N=8, K=16, dtype=0, act=1, workspace=A + 6 * FAR, workspace_bytes=FAR, stream=None)
    assert set(change) <= set(a)
    a.update(change)
    return list(a.values())


@pytest.mark.parametrize("change, match", [
    (dict(dtype=-1), "unknown dtype"), (dict(act=99), "unknown activation"), (dict(M=-1), "M, N and K"),
    (dict(z=None), "needs z"), (dict(dz=None), "dz"), (dict(w=None), "w"), (dict(dx=None), "dx"),
    (dict(lddz=7), "leading dimension of dz"), (dict(lddx=15), "leading dimension of dx"), (dict(ldadd=15), "leading dimension of add"),
    (dict(dx=A), "dx overlaps dz"), (dict(dx=A + 2 * FAR), "dx overlaps z"), (dict(dx=A + 3 * FAR + 4), "dx overlaps add"),
])
def test_linear_backward_input_arguments(change, match):
    refused(rar.lib.ddp_linear_backward_input(*backward_input_args(**change)), match)


def backward_weight_args(**change):
    a = dict(dz=A, lddz=8, x=A + FAR, ldx=16, dw=A + 2 * FAR, lddw=16, db=A + 3 * FAR, M=4, N=8, K=16, dtype=0,
             grad_dtype=0, accumulate=0, workspace=A + 6 * FAR, workspace_bytes=FAR, stream=None)
    assert set(change) <= set(a)
    a.update(change)
    return list(a.values())


@pytest.mark.parametrize("change, match", [
    (dict(dtype=5), "unknown dtype"), (dict(grad_dtype=1), "grad_dtype"), (dict(accumulate=2), "accumulate"),
    (dict(K=-1), "M, N and K"), (dict(dz=None), "dz"), (dict(x=None), "x"), (dict(dw=None), "dw"),
    (dict(dw=A + FAR), "dw overlaps x"), (dict(db=A + 2 * FAR + 8), "overlaps"), (dict(lddw=15), "leading dimension of dw"),
    (dict(workspace=None), "workspace needs"), (dict(workspace_bytes=3), "workspace needs"),
    (dict(workspace=A + 6 * FAR + 8), "16-byte aligned"), (dict(workspace=A + 2 * FAR), "overlaps"),
])
def test_linear_backward_weight_arguments(change, match):
    refused(rar.lib.ddp_linear_backward_weight(*backward_weight_args(**change)), match)


@pytest.mark.parametrize("change, match", [
    (dict(dtype=2), "unknown dtype"), (dict(act=99), "unknown activation"), (dict(N=-1), "M, N and K"),
    (dict(dy=None), "dy"), (dict(z=None), "z"), (dict(dz=None), "dz"), (dict(lddy=7), "leading dimension of dy"),
    (dict(dz=A + 4), "dz overlaps dy"), (dict(dz=A + FAR), "dz overlaps z"),
])
def test_act_backward_arguments(change, match):
    a = dict(dy=A, lddy=8, z=A + FAR, ldz=8, dz=A + 2 * FAR, lddz=8, M=4, N=8, dtype=0, act=1, stream=None)
    assert set(change) <= set(a)
    a.update(change)
    refused(rar.lib.ddp_act_backward(*a.values()), match)


def test_linear_workspace_arguments():
    lib, out = rar.lib, ctypes.c_int64(7)
    refused(lib.ddp_linear_workspace(0, 1, 1, 1, 0, None), "bytes is NULL")
    refused(lib.ddp_linear_workspace(3, 1, 1, 1, 0, ctypes.byref(out)), "direction")
    refused(lib.ddp_linear_workspace(0, -1, 1, 1, 0, ctypes.byref(out)), "M, N and K")
    refused(lib.ddp_linear_workspace(0, 1, 1, 1, 4, ctypes.byref(out)), "dtype")
    assert out.value == 0


@pytest.mark.parametrize("change, overlaps", [
    # y (4 x 8, of fp32) beside the residual, z and x in one buffer with rows of 32 and 40 elements
    (dict(y=A, ldy=32, residual=A + 32, ldr=32), False), (dict(y=A + 32, ldy=32, residual=A, ldr=32), False),
    (dict(y=A, ldy=32, residual=A + 28, ldr=32), True), (dict(y=A + 28, ldy=32, residual=A, ldr=32), True),
    (dict(y=A, ldy=32, z=A + 96, ldz=32), False), (dict(y=A, ldy=32, z=A + 100, ldz=32), True),
    (dict(y=A + 100, ldy=32, z=A, ldz=32), True), (dict(y=A, ldy=32, z=A + 128 + 32, ldz=32), False),
    (dict(y=A, ldy=32, z=A + 128 - 4, ldz=32), True), (dict(y=A + 64, ldy=40, x=A, ldx=40), False),
    (dict(y=A + 60, ldy=40, x=A, ldx=40), True), (dict(y=A, ldy=32, z=A + 32, ldz=33), True),
    # the bias, one row, in the gap behind y's columns
    (dict(y=A, ldy=32, bias=A + 128 + 64), False), (dict(y=A, ldy=32, bias=A + 128 + 100), True),
    (dict(y=A, ldy=32, bias=A + 128 + 28), True),
])
def test_column_blocks_of_one_buffer_do_not_overlap(change, overlaps):
    """On addresses of no allocation, which is what a call without overlap is refused for."""
    base = dict(x=A + 7 * FAR)
    status = rar.lib.ddp_linear_forward(*forward_args(**{**base, **change}))
    refused(status, "overlaps" if overlaps else "not inside a device allocation")


def test_linear_tiling():
    lib, tile, parts = rar.lib, ctypes.c_int32(7), ctypes.c_int32(7)
    out = ctypes.byref(tile), ctypes.byref(parts)
    refused(lib.ddp_linear_tiling(0, 1, 1, 1, 0, 0, None, out[1]), "output is NULL")
    refused(lib.ddp_linear_tiling(0, 1, 1, 1, 0, 0, out[0], None), "output is NULL")
    refused(lib.ddp_linear_tiling(-1, 1, 1, 1, 0, 0, *out), "direction")
    refused(lib.ddp_linear_tiling(0, 1, 1, 1, 0, 2, *out), "direct must be")
    refused(lib.ddp_linear_tiling(0, 1, -1, 1, 0, 1, *out), "M, N and K")
    refused(lib.ddp_linear_tiling(0, 1, 1, 1, 3, 1, *out), "dtype")
    assert (tile.value, parts.value) == (0, 0)
    assert rar.linear_tiling(rar.LINEAR_FORWARD, 1, 4096, 4096, "bf16")[0] == 0
    for dtype, direct, wide in (("bf16", True, 256), ("bf16", False, 128), ("fp32", True, 128), ("fp32", False, 128)):
        for direction in range(3):
            assert rar.linear_tiling(direction, 8192, 8192, 8192, dtype, direct) == (wide, 1)
