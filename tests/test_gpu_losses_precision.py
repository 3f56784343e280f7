"""The gradients of the losses where the data is bf16 (include/ddp_train.h): dz meets
the products in two terms, so that a gradient is off by its own rounding and next to nothing else.

Tolerances are those of test_gpu_losses.py with dz off by b^2 (b = 2^-8) for every output, and fp32 sums of
twice as many terms."""

import math

import pytest
import torch

from test_gpu_linear import B, U, close, gen, matrix
from test_gpu_losses import TINY, Case

pytestmark = pytest.mark.gpu


def check(c, dx, dw, grads, old):
    e_dz = (c.e_dz + B * B * c.dz.abs() + TINY) * c.counts[:, None]
    tol = e_dz @ c.w64.abs() + 2 * (2 * c.v + 8) * U * (c.dz.abs() @ c.w64.abs())
    close(dx, c.dz @ c.w64, tol, "bf16", "dx")
    want = c.dz.t() @ c.x64
    tol = e_dz.t() @ c.x64.abs() + 2 * (2 * c.m + 2) * U * (c.dz.abs().t() @ c.x64.abs())
    if old is not None:
        want = want + old
        tol = tol + U * want.abs()
    close(dw, want, tol, grads, "dw")


# M, V, K, pad, shift: tiles of 32, 64, 128 and 256, direct loads and others, rows shorter than 16 bytes, sums in parts, pieces
SIZES = [(33, 64, 96, 0, 0), (33, 200, 71, 3, 1), (7, 90, 4, 0, 0), (300, 257, 264, 8, 0), (300, 257, 263, 3, 1), (700, 2000, 520, 0, 0),
         (3841, 16, 2056, 0, 0), (2500, 1500, 1001, 0, 0), (20, 20000, 40, 0, 0), (40000, 9003, 24, 0, 0)]


@pytest.mark.parametrize("grads", ["bf16", "fp32"])
@pytest.mark.parametrize("top", [0, 9])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_gradients_are_off_by_their_own_rounding(size, top, grads):
    m, v, k, pad, shift = size
    c = Case(m, v, k, "bf16", top=top, temperature=2.0 if top else 1.0, ignored=0.1, pad=pad, shift=shift)
    loss, lse = c.forward()
    c.formulas()
    accumulate = m % 2 == 0
    dw = matrix(gen(9), v, k, grads, pad, shift=shift)
    old = dw.double() if accumulate else None
    if not accumulate:
        dw.fill_(math.nan)
    dx = c.backward(lse, dw=dw, accumulate=accumulate)
    check(c, dx, dw, grads, old)


def test_dx_alone():
    c = Case(130, 300, 72, "bf16", ignored=0.2)
    _, lse = c.forward()
    c.formulas()
    dx = c.backward(lse)
    e_dz = (c.e_dz + B * B * c.dz.abs() + TINY) * c.counts[:, None]
    close(dx, c.dz @ c.w64, e_dz @ c.w64.abs() + 2 * (2 * c.v + 8) * U * (c.dz.abs() @ c.w64.abs()), "bf16", "dx")
