"""The experts' layers and the losses on the CPU: bad arguments are refused
before anything touches a GPU."""

import ctypes

import pytest

rar = pytest.importorskip("ring_all_reduce_ddp_amd")

A = 0x100000      # addresses that are never read: the refusals come first
FAR = 1 << 30


def refused(status, match):
    msg = rar.lib.ddp_last_error().decode()
    assert status == rar.DDP_EINVAL and match in msg, (status, msg)


def args(base, change):
    assert set(change) <= set(base)
    return list({**base, **change}.values())


EXPERTS_FORWARD = dict(x=A, ldx=16, w=A + FAR, ldw=16, bias=A + 2 * FAR, offsets=A + 3 * FAR, y=A + 4 * FAR, ldy=8, z=A + 5 * FAR, ldz=8,
                       T=4, E=3, N=8, K=16, dtype=0, act=1, workspace=A + 6 * FAR, workspace_bytes=FAR, stream=None)


@pytest.mark.parametrize("change, match", [
    (dict(dtype=9), "unknown dtype"), (dict(act=99), "unknown activation"), (dict(T=-1), "M, N and K"), (dict(N=-1), "M, N and K"),
    (dict(E=0), "E must"), (dict(E=65537), "E must"), (dict(K=0), "K must"), (dict(E=65536, N=1 << 15), "E * N"),
    (dict(x=None), "x"), (dict(w=None), "w"), (dict(y=None), "y"), (dict(offsets=None), "offsets"),
    (dict(offsets=A + 3 * FAR + 4), "offsets is not aligned"), (dict(w=A + FAR + 2), "w is not aligned"),
    (dict(ldx=15), "leading dimension of x"), (dict(ldw=15), "leading dimension of w"), (dict(ldz=7), "leading dimension of z"),
    (dict(y=A + 16), "y overlaps x"), (dict(z=A + 4 * FAR), "overlaps"), (dict(y=A + 3 * FAR + 24), "y overlaps offsets"),
    (dict(y=A + FAR + 3 * 8 * 16 * 4 - 4), "y overlaps w"),
])
def test_experts_forward(change, match):
    refused(rar.lib.ddp_experts_forward(*args(EXPERTS_FORWARD, change)), match)


EXPERTS_INPUT = dict(dz=A, lddz=8, w=A + FAR, ldw=16, offsets=A + 3 * FAR, z=A + 2 * FAR, ldz=16, dx=A + 4 * FAR, lddx=16, T=4, E=3, N=8,
                     K=16, dtype=0, act=1, workspace=A + 6 * FAR, workspace_bytes=FAR, stream=None)


@pytest.mark.parametrize("change, match", [
    (dict(dtype=-1), "unknown dtype"), (dict(z=None), "needs z"), (dict(dz=None), "dz"), (dict(dx=None), "dx"), (dict(offsets=None), "offsets"),
    (dict(lddz=7), "leading dimension of dz"), (dict(lddx=15), "leading dimension of dx"), (dict(dx=A), "dx overlaps dz"),
    (dict(dx=A + 2 * FAR), "dx overlaps z"),
])
def test_experts_backward_input(change, match):
    refused(rar.lib.ddp_experts_backward_input(*args(EXPERTS_INPUT, change)), match)


EXPERTS_WEIGHT = dict(dz=A, lddz=8, x=A + FAR, ldx=16, offsets=A + 3 * FAR, dw=A + 2 * FAR, lddw=16, db=A + 5 * FAR, T=4, E=3, N=8, K=16,
                      dtype=1, grad_dtype=0, accumulate=0, workspace=A + 6 * FAR, workspace_bytes=FAR, stream=None)


@pytest.mark.parametrize("change, match", [
    (dict(grad_dtype=7), "grad_dtype"), (dict(dtype=0, grad_dtype=1), "grad_dtype"), (dict(accumulate=2), "accumulate"),
    (dict(workspace_bytes=0), "workspace needs"), (dict(workspace=None), "workspace needs"), (dict(workspace=A + 6 * FAR + 8), "16-byte"),
    (dict(dw=A), "dw overlaps dz"), (dict(db=A + 2 * FAR + 4), "overlaps"), (dict(workspace=A + 2 * FAR), "overlaps"),
    (dict(offsets=None), "offsets"), (dict(lddw=15), "leading dimension of dw"),
])
def test_experts_backward_weight(change, match):
    refused(rar.lib.ddp_experts_backward_weight(*args(EXPERTS_WEIGHT, change)), match)


def test_nothing_to_do():
    lib = rar.lib
    assert lib.ddp_experts_forward(*args(EXPERTS_FORWARD, dict(T=0, x=None, y=None, z=None))) == rar.DDP_OK
    assert lib.ddp_experts_backward_input(*args(EXPERTS_INPUT, dict(T=0, dz=None, dx=None))) == rar.DDP_OK
    assert lib.ddp_experts_backward_weight(*args(EXPERTS_WEIGHT, dict(N=0, dw=None))) == rar.DDP_OK
    assert lib.ddp_cross_entropy_forward(*args(ENTROPY_FORWARD, dict(M=0, x=None, loss=None))) == rar.DDP_OK
    assert lib.ddp_cross_entropy_backward(*args(ENTROPY_BACKWARD, dict(dx=None, dw=None))) == rar.DDP_OK


ENTROPY_FORWARD = dict(x=A, ldx=16, w=A + FAR, ldw=16, targets=A + 2 * FAR, loss=A + 3 * FAR, lse=A + 4 * FAR, M=4, V=8, K=16, dtype=0,
                       workspace=A + 6 * FAR, workspace_bytes=FAR, stream=None)
ENTROPY_BACKWARD = dict(x=A, ldx=16, w=A + FAR, ldw=16, targets=A + 2 * FAR, lse=A + 3 * FAR, dloss=A + 4 * FAR, dx=A + 5 * FAR, lddx=16,
                        dw=A + 7 * FAR, lddw=16, M=4, V=8, K=16, dtype=1, grad_dtype=0, accumulate=0, workspace=A + 8 * FAR,
                        workspace_bytes=FAR, stream=None)


@pytest.mark.parametrize("change, match", [
    (dict(dtype=5), "unknown dtype"), (dict(M=-1), "M, N and K"), (dict(V=0), "V and K"), (dict(K=0), "V and K"),
    (dict(M=(1 << 20) + 1), "2^20"), (dict(K=(1 << 21) + 1), "2^21"), (dict(M=1 << 20, K=4097), "2^32"),
    (dict(M=1 << 13, V=1 << 30), "M * V"),
    (dict(x=None), "x"), (dict(w=None), "w"), (dict(targets=None), "targets"), (dict(loss=None), "loss"), (dict(lse=None), "lse"),
    (dict(targets=A + 2 * FAR + 4), "targets is not aligned"), (dict(ldx=15), "leading dimension of x"), (dict(ldw=15), "leading dimension of w"),
    (dict(workspace_bytes=16), "workspace needs"), (dict(workspace=None), "workspace needs"),
    (dict(lse=A + 3 * FAR + 12), "overlaps"), (dict(loss=A), "loss overlaps x"), (dict(workspace=A + FAR), "overlaps"),
])
def test_cross_entropy_forward(change, match):
    refused(rar.lib.ddp_cross_entropy_forward(*args(ENTROPY_FORWARD, change)), match)


@pytest.mark.parametrize("change, match", [
    (dict(grad_dtype=3), "grad_dtype"), (dict(dtype=0, grad_dtype=1), "grad_dtype"), (dict(accumulate=-1), "accumulate"),
    (dict(lse=None), "lse"), (dict(dloss=None), "dloss"), (dict(dx=A), "dx overlaps x"), (dict(dw=A + FAR), "dw overlaps w"),
    (dict(dx=A + 3 * FAR), "dx overlaps lse"), (dict(lddx=15), "leading dimension of dx"), (dict(lddw=15), "leading dimension of dw"),
    (dict(workspace_bytes=64), "workspace needs"),
])
def test_cross_entropy_backward(change, match):
    refused(rar.lib.ddp_cross_entropy_backward(*args(ENTROPY_BACKWARD, change)), match)


DISTILL_FORWARD = dict(x=A, ldx=16, w=A + FAR, ldw=16, ids=A + 2 * FAR, ld_ids=3, teacher=A + 5 * FAR, ld_teacher=3, teacher_dtype=0,
                       temperature=2.0, loss=A + 3 * FAR, lse=A + 4 * FAR, M=4, V=8, K=16, C=3, dtype=0, workspace=A + 6 * FAR,
                       workspace_bytes=FAR, stream=None)


@pytest.mark.parametrize("change, match", [
    (dict(C=0), "C must"), (dict(C=1025), "C must"), (dict(temperature=0.0), "temperature"), (dict(temperature=-1.0), "temperature"),
    (dict(temperature=float("inf")), "temperature"), (dict(temperature=float("nan")), "temperature"), (dict(temperature=1e-45), "temperature"),
    (dict(teacher_dtype=4), "teacher_dtype"), (dict(ids=None), "ids"), (dict(teacher=None), "teacher"), (dict(ld_ids=2), "leading dimension of ids"),
    (dict(ld_teacher=2), "leading dimension of teacher"), (dict(dtype=5), "unknown dtype"), (dict(loss=A + 2 * FAR), "loss overlaps ids"),
    (dict(workspace_bytes=0), "workspace needs"),
])
def test_distill_forward(change, match):
    refused(rar.lib.ddp_distill_forward(*args(DISTILL_FORWARD, change)), match)


def test_workspaces():
    lib, n = rar.lib, ctypes.c_int64(7)
    refused(lib.ddp_experts_workspace(9, 4, 3, 8, 16, 0, ctypes.byref(n)), "direction")
    refused(lib.ddp_experts_workspace(0, 4, 3, 8, 16, 0, None), "bytes is NULL")
    assert n.value == 0 and lib.ddp_experts_workspace(0, 4, 3, 8, 16, 0, ctypes.byref(n)) == rar.DDP_OK and n.value == 0
    n.value = 7
    refused(lib.ddp_experts_workspace(1, 4, 0, 8, 16, 0, ctypes.byref(n)), "E must")
    assert n.value == 0
    refused(lib.ddp_cross_entropy_workspace(2, 4, 8, 16, 0, 0, ctypes.byref(n)), "direction")
    refused(lib.ddp_cross_entropy_workspace(0, 4, 8, 16, 0, 0, None), "bytes is NULL")
    refused(lib.ddp_distill_workspace(0, 4, 8, 16, 0, 0, 0, ctypes.byref(n)), "C must")
    # without the logits: 8192 rows of 128000 columns would be 2 GiB in bf16, and 4 GiB in fp32
    assert rar.cross_entropy_workspace(rar.LOSS_FORWARD, 8192, 128000, 4096, "bf16") < 1 << 28
    assert rar.cross_entropy_workspace(rar.LOSS_BACKWARD, 8192, 128000, 4096, "bf16", "bf16") < 1 << 29
    assert rar.cross_entropy_workspace(rar.LOSS_BACKWARD, 8192, 128000, 4096, "bf16", "fp32") < 3 << 28
    with pytest.raises(ValueError):
        rar.distill_workspace(rar.LOSS_FORWARD, 4, 8, 16, 0, "fp32")


def test_tilings():
    lib, n, piece = rar.lib, [ctypes.c_int32(7) for _ in range(3)], ctypes.c_int64(7)
    out = [ctypes.byref(x) for x in n]
    refused(lib.ddp_experts_tiling(3, 4, 3, 8, 16, 0, 1, *out), "direction")
    refused(lib.ddp_experts_tiling(0, 4, 3, 8, 16, 0, 2, *out), "direct must be")
    refused(lib.ddp_experts_tiling(0, 4, 0, 8, 16, 0, 1, *out), "E must")
    refused(lib.ddp_experts_tiling(0, 4, 3, 8, 16, 0, 1, None, *out[1:]), "output is NULL")
    refused(lib.ddp_loss_tiling(4, 4, 8, 16, 0, 0, 1, *out, ctypes.byref(piece)), "product")
    refused(lib.ddp_loss_tiling(0, 4, 8, 16, 0, 0, 3, *out, ctypes.byref(piece)), "direct must be")
    refused(lib.ddp_loss_tiling(0, 4, 0, 16, 0, 0, 1, *out, ctypes.byref(piece)), "V and K")
    refused(lib.ddp_loss_tiling(0, 4, 8, 16, 0, 0, 1, *out, None), "output is NULL")
    assert [x.value for x in n] == [0, 0, 0] and piece.value == 0
    assert rar.experts_tiling(rar.LINEAR_FORWARD, 1 << 17, 8, 4096, 4096, "bf16") == (256, 256, 1)
    assert rar.loss_tiling(rar.LOSS_Z, 8192, 128000, 4096, "bf16") == (256, 256, 1, 128000)
    # the vocabulary in pieces of whole tiles
    assert rar.loss_tiling(rar.LOSS_Z_AGAIN, 8192, 128000, 4096, "bf16", "fp32") == (256, 256, 1, 16128)
    assert rar.loss_tiling(rar.LOSS_DW, 8192, 128000, 4096, "bf16", "fp32")[:3] == (256, 256, 1)
