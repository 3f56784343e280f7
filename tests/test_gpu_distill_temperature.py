"""Distillation at the ends of the temperatures that are allowed, against 64 bits.

Tolerances are those of test_gpu_losses.py, and one more: at small T the probabilities reach below fp32's smallest
normal number, 2^-126, where an exponential may be any subnormal number near it or 0. So p is off by 2^-126 more, and dz by
|slope| times that. (fp32 counts its own subnormals of the result in close() already, 2^-149.)"""

import pytest
import torch

from test_gpu_losses import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("temperature", [2.0 ** -20, 2.0 ** -7, 2.0 ** 10, 2.0 ** 20])
def test_ends(temperature, dtype):
    c = Case(70, 300, 72, dtype, top=5, temperature=temperature, ignored=0.2)
    loss, lse = c.forward()
    c.formulas()
    c.check_forward(loss, lse)
    c.e_dz += 2.0 ** -126 * torch.where(c.counts, c.dloss.double().abs() * c.t, 0.0)[:, None]
    dw = torch.empty(300, 72, device="cuda")
    dx = c.backward(lse, dw=dw)
    c.check_backward(dx, dw, "fp32")
