"""Temperatures at which the distillation's T^2 or logits / T would leave fp32 are refused."""

import pytest

from test_more_operators_cpu import A, DISTILL_FORWARD, FAR, args, rar, refused

DISTILL_BACKWARD = dict(x=A, ldx=16, w=A + FAR, ldw=16, ids=A + 2 * FAR, ld_ids=3, teacher=A + 5 * FAR, ld_teacher=3, teacher_dtype=0,
                        temperature=2.0, lse=A + 3 * FAR, dloss=A + 4 * FAR, dx=A + 7 * FAR, lddx=16, dw=A + 8 * FAR, lddw=16, M=4, V=8, K=16,
                        C=3, dtype=1, grad_dtype=0, accumulate=0, workspace=A + 6 * FAR, workspace_bytes=FAR, stream=None)


@pytest.mark.parametrize("temperature", [3e38, 2.0 ** 64, 2.0 ** 20 * 1.001, 2.0 ** -20 * 0.999, 1e-10, 1e-30])
def test_refused(temperature):
    refused(rar.lib.ddp_distill_forward(*args(DISTILL_FORWARD, dict(temperature=temperature))), "temperature must lie in [2^-20, 2^20]")
    refused(rar.lib.ddp_distill_backward(*args(DISTILL_BACKWARD, dict(temperature=temperature))), "temperature must lie in [2^-20, 2^20]")


@pytest.mark.parametrize("temperature", [2.0 ** 20, 2.0 ** -20, 1.0])
def test_not_refused_for_it(temperature):
    """The next refusal is that of the workspace."""
    refused(rar.lib.ddp_distill_forward(*args(DISTILL_FORWARD, dict(temperature=temperature, workspace_bytes=0))), "workspace needs")
    refused(rar.lib.ddp_distill_backward(*args(DISTILL_BACKWARD, dict(temperature=temperature, workspace_bytes=0))), "workspace needs")
