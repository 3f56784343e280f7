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
