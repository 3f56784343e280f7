"""Python binding of libddp_ring.so: the bucketed ring all-reduce of DDP
gradients over N virtual ranks on one MI355X.

The functions have the names of the C entry points in include/ddp_ring.h (the
operators around the sync, of include/ddp_train.h, drop the ddp_ prefix) and
only marshal arguments: torch tensors become device pointers, dtypes become
DDP_FP32 / DDP_BF16, and the stream defaults to torch's current stream. Every
step of the computation runs in the library's HIP kernels; there is no other
code path. The library is loaded on first use; every call fails with an
ImportError naming the build command if it has not been built
(python -m ring_all_reduce_ddp_amd.build).

PyTorch is used for device memory and streams only. It is imported before the
library is loaded so that both use the single HIP runtime that torch ships.
"""

import ctypes
import functools
import os
import sys

import torch  # noqa: F401  (loads the HIP runtime the library binds to)

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libddp_ring.so")

DDP_OK = 0
DDP_EINVAL = -1
DDP_EHIP = -2
DDP_ENORESOURCE = -3
DDP_ETIMEOUT = -4
DDP_ENOMEM = -5
DDP_FP32 = 0
DDP_BF16 = 1
DDP_RS = 0
DDP_AG = 1
DDP_MAX_RANKS = 64
VARIANTS = {"fused": 0, "steps": 1, "persistent": 2, "view": 3}

_STATUS_NAMES = {DDP_EINVAL: "DDP_EINVAL", DDP_EHIP: "DDP_EHIP", DDP_ENORESOURCE: "DDP_ENORESOURCE",
                 DDP_ETIMEOUT: "DDP_ETIMEOUT", DDP_ENOMEM: "DDP_ENOMEM"}


class DDPError(RuntimeError):
    """A non-zero status from the library, with ddp_last_error()'s message."""

    def __init__(self, status, message):
        super().__init__(f"{_STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m ring_all_reduce_ddp_amd.build` (hipcc, gfx950)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    f64 = ctypes.c_double
    pp = ctypes.POINTER(ctypes.c_void_p)
    sig = {
        "ddp_last_error": (ctypes.c_char_p, []),
        "ddp_bucket_plan": (ctypes.c_int, [ctypes.POINTER(i64), i32, i32, i64, i64, i32,
                                           ctypes.POINTER(vp)]),
        "ddp_bucket_plan_ex": (ctypes.c_int, [ctypes.POINTER(i64), i32, i32, i32, i64, i64, i32,
                                              ctypes.POINTER(vp)]),
        "ddp_plan_free": (None, [vp]),
        "ddp_plan_num_buckets": (ctypes.c_int, [vp, ctypes.POINTER(i32)]),
        "ddp_plan_bucket": (ctypes.c_int, [vp, i32, ctypes.POINTER(i64), ctypes.POINTER(i32)]),
        "ddp_plan_member": (ctypes.c_int, [vp, i32, i32, ctypes.POINTER(i32), ctypes.POINTER(i64),
                                           ctypes.POINTER(i64)]),
        "ddp_plan_grad_arena": (ctypes.c_int, [vp, ctypes.POINTER(i64), ctypes.POINTER(i64)]),
        "ddp_plan_arena_map": (ctypes.c_int, [vp, vp, i64]),
        "bucket_pack": (ctypes.c_int, [vp, i32, pp, pp, i32, vp]),
        "bucket_unpack_scale": (ctypes.c_int, [vp, i32, pp, pp, i32, f32, vp]),
        "ring_allreduce_step": (ctypes.c_int, [pp, i32, i64, i32, i32, i32, vp]),
        "ring_allreduce_persistent": (ctypes.c_int, [pp, i32, i64, i32, i32, vp]),
        "ring_allreduce_persistent_ex": (ctypes.c_int, [pp, i32, i64, i32, i32, i32, i64, ctypes.c_uint32, vp]),
        "ring_allreduce_persistent_noalloc": (ctypes.c_int, [pp, i32, i64, i32, i32, vp]),
        "ddp_persistent_test_hook": (ctypes.c_int, [ctypes.c_uint32, i64]),
        "ddp_persistent_grid": (ctypes.c_int, [i32, i64, i32, ctypes.POINTER(i32), ctypes.POINTER(i32)]),
        "ddp_persistent_status": (ctypes.c_int, [vp]),
        "ring_allreduce_fused": (ctypes.c_int, [pp, i32, i64, i32, vp]),
        "bucket_allreduce_view": (ctypes.c_int, [vp, i32, pp, i32, f32, vp]),
        "ring_reduce_scatter_fused": (ctypes.c_int, [pp, pp, i32, i64, i32, f32, vp]),
        "ddp_sync": (ctypes.c_int, [vp, pp, pp, i32, i32, f32, vp]),
        "ddp_reducer_create": (ctypes.c_int, [vp, pp, pp, i32, i32, f32, i64, vp, ctypes.POINTER(vp)]),
        "ddp_reducer_free": (None, [vp]),
        "ddp_reducer_prepare": (ctypes.c_int, [vp]),
        "ddp_reducer_mark_ready": (ctypes.c_int, [vp, i32, vp]),
        "ddp_reducer_finalize": (ctypes.c_int, [vp, vp]),
        "ddp_synthetic_backward": (ctypes.c_int, [pp, pp, i32, i64, i32, i32, i32, vp]),
        "ddp_synthetic_backward_pass": (ctypes.c_int, [vp, pp, pp, i32, i32, i32, vp, vp]),
        "ddp_count_mismatches": (ctypes.c_int, [pp, i32, i64, i32, vp, vp]),
        "ddp_copy_probe": (ctypes.c_int, [vp, vp, i64, vp]),
        "ddp_device_alloc": (ctypes.c_int, [i64, i32, ctypes.POINTER(vp)]),
        "ddp_device_free": (ctypes.c_int, [vp]),
        "ddp_grads_create": (ctypes.c_int, [pp, ctypes.POINTER(i64), i32, i32, ctypes.POINTER(vp)]),
        "ddp_grads_free": (None, [vp]),
        "ddp_grads_norm": (ctypes.c_int, [vp, i32, vp, vp]),
        "ddp_grads_clip": (ctypes.c_int, [vp, vp, f32, vp, vp]),
        "ddp_adamw_create": (ctypes.c_int, [vp, pp, pp, pp, pp, ctypes.POINTER(ctypes.c_uint8), vp,
                                            ctypes.POINTER(vp)]),
        "ddp_adamw_free": (None, [vp]),
        "ddp_adamw_step": (ctypes.c_int, [vp, f64, f64, f64, f64, f64, f64, vp, vp]),
        "ddp_linear_workspace": (ctypes.c_int, [i32, i64, i64, i64, i32, ctypes.POINTER(i64)]),
        "ddp_linear_tiling": (ctypes.c_int, [i32, i64, i64, i64, i32, i32, ctypes.POINTER(i32), ctypes.POINTER(i32)]),
        "ddp_linear_forward": (ctypes.c_int, [vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, i64, i64, i64, i64,
                                              i32, i32, vp, i64, vp]),
        "ddp_linear_backward_input": (ctypes.c_int, [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, i64, i64, i64,
                                                     i32, i32, vp, i64, vp]),
        "ddp_linear_backward_weight": (ctypes.c_int, [vp, i64, vp, i64, vp, i64, vp, i64, i64, i64, i32, i32, i32,
                                                      vp, i64, vp]),
        "ddp_experts_workspace": (ctypes.c_int, [i32, i64, i64, i64, i64, i32, ctypes.POINTER(i64)]),
        "ddp_experts_tiling": (ctypes.c_int, [i32, i64, i64, i64, i64, i32, i32, *[ctypes.POINTER(i32)] * 3]),
        "ddp_loss_tiling": (ctypes.c_int, [i32, i64, i64, i64, i32, i32, i32, *[ctypes.POINTER(i32)] * 3, ctypes.POINTER(i64)]),
        "ddp_experts_forward": (ctypes.c_int, [vp, i64, vp, i64, vp, vp, vp, i64, vp, i64, i64, i64, i64, i64, i32, i32, vp, i64, vp]),
        "ddp_experts_backward_input": (ctypes.c_int, [vp, i64, vp, i64, vp, vp, i64, vp, i64, i64, i64, i64, i64, i32, i32,
                                                      vp, i64, vp]),
        "ddp_experts_backward_weight": (ctypes.c_int, [vp, i64, vp, i64, vp, vp, i64, vp, i64, i64, i64, i64, i32, i32, i32,
                                                       vp, i64, vp]),
        "ddp_cross_entropy_workspace": (ctypes.c_int, [i32, i64, i64, i64, i32, i32, ctypes.POINTER(i64)]),
        "ddp_cross_entropy_forward": (ctypes.c_int, [vp, i64, vp, i64, vp, vp, vp, i64, i64, i64, i32, vp, i64, vp]),
        "ddp_cross_entropy_backward": (ctypes.c_int, [vp, i64, vp, i64, vp, vp, vp, vp, i64, vp, i64, i64, i64, i64, i32, i32, i32,
                                                      vp, i64, vp]),
        "ddp_distill_workspace": (ctypes.c_int, [i32, i64, i64, i64, i32, i32, i32, ctypes.POINTER(i64)]),
        "ddp_distill_forward": (ctypes.c_int, [vp, i64, vp, i64, vp, i64, vp, i64, i32, f32, vp, vp, i64, i64, i64, i32, i32,
                                               vp, i64, vp]),
        "ddp_distill_backward": (ctypes.c_int, [vp, i64, vp, i64, vp, i64, vp, i64, i32, f32, vp, vp, vp, i64, vp, i64, i64, i64, i64,
                                                i32, i32, i32, i32, vp, i64, vp]),
        "ddp_act_backward": (ctypes.c_int, [vp, i64, vp, i64, vp, i64, i64, i64, i32, i32, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


_lib = None


def _get_lib():
    global _lib
    if _lib is None:
        _lib = _load()
    return _lib


def __getattr__(name):
    # `ring_all_reduce_ddp_amd.lib` is the ctypes handle, loaded on first access.
    if name == "lib":
        return _get_lib()
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


def _check(status):
    if status != DDP_OK:
        msg = _get_lib().ddp_last_error()
        raise DDPError(status, msg.decode() if msg else "")


# ---------------------------------------------------------------- marshalling helpers

_TORCH_DTYPES = {torch.float32: DDP_FP32, torch.bfloat16: DDP_BF16}
_NAMED_DTYPES = {"fp32": DDP_FP32, "bf16": DDP_BF16, DDP_FP32: DDP_FP32, DDP_BF16: DDP_BF16}


def dtype_code(dtype):
    if dtype in _TORCH_DTYPES:
        return _TORCH_DTYPES[dtype]
    if dtype in _NAMED_DTYPES:
        return _NAMED_DTYPES[dtype]
    raise ValueError(f"unsupported dtype {dtype!r}")


def _ptr(x):
    if isinstance(x, torch.Tensor):
        return x.data_ptr()
    return int(x)


def _ptr_array(xs):
    return (ctypes.c_void_p * len(xs))(*[_ptr(x) for x in xs])


def _stream(stream):
    if stream is None:
        # torch.cuda.current_stream() without making its Stream object (3 us of a small call)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _ring_args(bufs, count, dtype):
    """(pointer array, N, count, dtype code) from tensors or raw pointers."""
    n = len(bufs)
    if isinstance(bufs[0], torch.Tensor):
        t0 = bufs[0]
        if dtype is None:
            dtype = t0.dtype
        if count is None:
            count = t0.numel()
        for t in bufs:
            if not t.is_contiguous() or t.numel() < count or t.dtype != t0.dtype:
                raise ValueError("rank buffers must be contiguous tensors of one dtype holding count elements")
    if count is None or dtype is None:
        raise ValueError("count and dtype are required for raw pointers")
    return _ptr_array(bufs), n, int(count), dtype_code(dtype)


# ---------------------------------------------------------------- planner

class Plan:
    """A bucket plan (see ddp_bucket_plan). Owns the library's handle."""

    def __init__(self, handle, n_params, dtype, world_size):
        self._h = handle
        self.n_params = n_params
        self.dtype = dtype
        self.comm_dtype = dtype
        self.world_size = world_size

    @property
    def handle(self):
        return self._h

    def free(self):
        if self._h:
            _get_lib().ddp_plan_free(self._h)
            self._h = None

    def __del__(self, _finalizing=sys.is_finalizing):
        # Never while the interpreter shuts down: freeing a plan's device
        # tables calls into the HIP runtime, which may already be going away
        # (the process's memory is returned anyway). The check is bound at
        # definition: module globals such as `sys` may already be None here.
        if _finalizing():
            return
        try:
            self.free()
        except Exception:
            pass

    @property
    def num_buckets(self):
        n = ctypes.c_int32()
        _check(_get_lib().ddp_plan_num_buckets(self._h, ctypes.byref(n)))
        return n.value

    def bucket(self, b):
        """(padded_numel, [(param_index, offset, numel), ...]) of bucket b."""
        padded, nm = ctypes.c_int64(), ctypes.c_int32()
        _check(_get_lib().ddp_plan_bucket(self._h, b, ctypes.byref(padded), ctypes.byref(nm)))
        members = []
        for i in range(nm.value):
            p, off, m = ctypes.c_int32(), ctypes.c_int64(), ctypes.c_int64()
            _check(_get_lib().ddp_plan_member(self._h, b, i, ctypes.byref(p), ctypes.byref(off), ctypes.byref(m)))
            members.append((p.value, off.value, m.value))
        return padded.value, members

    def buckets(self):
        """All buckets as dicts {"members": [...], "padded_numel": int}."""
        out = []
        for b in range(self.num_buckets):
            padded, members = self.bucket(b)
            out.append({"members": members, "padded_numel": padded})
        return out

    def arena_map(self):
        """The in-place sync's per-vector arena map, as a numpy uint16 array."""
        import numpy as np
        n, _ = self.grad_arena()
        v = 16 // (4 if self.dtype == DDP_FP32 else 2)
        out = np.empty(n // v, dtype=np.uint16)
        _check(_get_lib().ddp_plan_arena_map(self._h, out.ctypes.data_as(ctypes.c_void_p), len(out)))
        return out

    def grad_arena(self):
        """(arena_numel, [offset of parameter p in elements])."""
        n = ctypes.c_int64()
        offs = (ctypes.c_int64 * max(self.n_params, 1))()
        _check(_get_lib().ddp_plan_grad_arena(self._h, ctypes.byref(n), offs))
        return n.value, list(offs[:self.n_params])


def ddp_bucket_plan(param_numels, dtype="fp32", cap_bytes=25 * 1024 * 1024,
                    first_bucket_bytes=1024 * 1024, world_size=1):
    numels = (ctypes.c_int64 * max(len(param_numels), 1))(*[int(m) for m in param_numels])
    h = ctypes.c_void_p()
    _check(_get_lib().ddp_bucket_plan(numels, len(param_numels), dtype_code(dtype), int(cap_bytes),
                                      int(first_bucket_bytes), int(world_size), ctypes.byref(h)))
    return Plan(h.value, len(param_numels), dtype_code(dtype), int(world_size))


def ddp_bucket_plan_ex(param_numels, grad_dtype="fp32", comm_dtype="bf16", cap_bytes=25 * 1024 * 1024,
                       first_bucket_bytes=1024 * 1024, world_size=1):
    numels = (ctypes.c_int64 * max(len(param_numels), 1))(*[int(m) for m in param_numels])
    h = ctypes.c_void_p()
    _check(_get_lib().ddp_bucket_plan_ex(numels, len(param_numels), dtype_code(grad_dtype),
                                         dtype_code(comm_dtype), int(cap_bytes), int(first_bucket_bytes),
                                         int(world_size), ctypes.byref(h)))
    plan = Plan(h.value, len(param_numels), dtype_code(grad_dtype), int(world_size))
    plan.comm_dtype = dtype_code(comm_dtype)
    return plan


# ---------------------------------------------------------------- kernels

def bucket_pack(plan, b, grad_arenas, bucket_bufs, stream=None):
    _check(_get_lib().bucket_pack(plan.handle, b, _ptr_array(grad_arenas), _ptr_array(bucket_bufs),
                           len(bucket_bufs), _stream(stream)))


def bucket_unpack_scale(plan, b, bucket_bufs, grad_arenas, scale, stream=None):
    _check(_get_lib().bucket_unpack_scale(plan.handle, b, _ptr_array(bucket_bufs), _ptr_array(grad_arenas),
                                   len(bucket_bufs), float(scale), _stream(stream)))


def ring_allreduce_step(bufs, step, phase, count=None, dtype=None, stream=None):
    ptrs, n, count, dt = _ring_args(bufs, count, dtype)
    _check(_get_lib().ring_allreduce_step(ptrs, n, count, dt, int(step), int(phase), _stream(stream)))


def ring_allreduce_stepwise(bufs, count=None, dtype=None, stream=None):
    """The whole all-reduce as 2(N-1) ring_allreduce_step launches, in order."""
    n = len(bufs)
    for phase in (DDP_RS, DDP_AG):
        for s in range(n - 1):
            ring_allreduce_step(bufs, s, phase, count, dtype, stream)


def ring_allreduce_persistent(bufs, n_steps=None, count=None, dtype=None, stream=None):
    ptrs, n, count, dt = _ring_args(bufs, count, dtype)
    if n_steps is None:
        n_steps = 2 * (n - 1)
    _check(_get_lib().ring_allreduce_persistent(ptrs, n, count, dt, int(n_steps), _stream(stream)))


def ring_allreduce_persistent_ex(bufs, n_steps=None, max_blocks=0, timeout_us=10_000_000,
                                 extra_arrivals=0, count=None, dtype=None, stream=None):
    ptrs, n, count, dt = _ring_args(bufs, count, dtype)
    if n_steps is None:
        n_steps = 2 * (n - 1)
    _check(_get_lib().ring_allreduce_persistent_ex(ptrs, n, count, dt, int(n_steps), int(max_blocks),
                                            int(timeout_us), int(extra_arrivals), _stream(stream)))


def ring_allreduce_persistent_noalloc(bufs, n_steps=None, count=None, dtype=None, stream=None):
    """ring_allreduce_persistent with its barrier words in the library's fixed
    device array instead of an allocation (calls on one GPU must not overlap)."""
    ptrs, n, count, dt = _ring_args(bufs, count, dtype)
    if n_steps is None:
        n_steps = 2 * (n - 1)
    _check(_get_lib().ring_allreduce_persistent_noalloc(ptrs, n, count, dt, int(n_steps), _stream(stream)))


def ddp_persistent_test_hook(extra_arrivals=0, timeout_us=0):
    """Tests of the time-out path only: later default persistent launches
    expect extra_arrivals more blocks and give up after timeout_us (0 resets)."""
    _check(_get_lib().ddp_persistent_test_hook(int(extra_arrivals), int(timeout_us)))


def ddp_persistent_grid(n, count, dtype="fp32"):
    """(grid, compute units) the persistent launch would use."""
    g, cu = ctypes.c_int32(), ctypes.c_int32()
    _check(_get_lib().ddp_persistent_grid(int(n), int(count), dtype_code(dtype), ctypes.byref(g), ctypes.byref(cu)))
    return g.value, cu.value


def ddp_persistent_status(stream=None):
    _check(_get_lib().ddp_persistent_status(_stream(stream)))


def ring_allreduce_fused(bufs, count=None, dtype=None, stream=None):
    ptrs, n, count, dt = _ring_args(bufs, count, dtype)
    _check(_get_lib().ring_allreduce_fused(ptrs, n, count, dt, _stream(stream)))


def bucket_allreduce_view(plan, b, grad_arenas, scale, stream=None):
    _check(_get_lib().bucket_allreduce_view(plan.handle, b, _ptr_array(grad_arenas), len(grad_arenas),
                                     float(scale), _stream(stream)))


def ring_reduce_scatter_fused(bufs, shards, scale=1.0, count=None, dtype=None, stream=None):
    """shards[c] receives chunk c of the ring sum (times scale); None for an
    empty chunk."""
    ptrs, n, count, dt = _ring_args(bufs, count, dtype)
    sh = (ctypes.c_void_p * n)(*[None if x is None else _ptr(x) for x in shards])
    _check(_get_lib().ring_reduce_scatter_fused(ptrs, sh, n, count, dt, float(scale), _stream(stream)))


def ddp_sync(plan, grad_arenas, bucket_bufs=None, *, scale, variant="fused", stream=None):
    """bucket_bufs: list over buckets of lists over ranks (or a flat list,
    bucket-major); None for the "view" variant, which uses no bucket buffers.
    scale: the fp32 multiplier of the copy back, chosen by the caller (1/N
    for DDP's mean)."""
    n = len(grad_arenas)
    if bucket_bufs is None:
        bufs = None
    else:
        flat = [x for row in bucket_bufs for x in row] if isinstance(bucket_bufs[0], (list, tuple)) \
            else list(bucket_bufs)
        bufs = _ptr_array(flat)
    _check(_get_lib().ddp_sync(plan.handle, _ptr_array(grad_arenas), bufs, n, VARIANTS[variant], float(scale),
                        _stream(stream)))


class Reducer:
    """Launches each bucket's sync as soon as its last gradient is marked
    ready, on `comm_stream` (see ddp_reducer_* in include/ddp_ring.h).
    bucket_bufs: list over buckets of lists over ranks; None for "view".
    scale: the fp32 multiplier of each bucket's copy back (1/N for DDP's
    mean), chosen by the caller."""

    def __init__(self, plan, grad_arenas, bucket_bufs=None, *, scale, variant="view", comm_stream=None,
                 comm_max_blocks=0):
        n = len(grad_arenas)
        self.plan = plan   # the plan must outlive the reducer
        if bucket_bufs is None:
            bufs = None
        else:
            flat = [x for row in bucket_bufs for x in row] if isinstance(bucket_bufs[0], (list, tuple)) \
                else list(bucket_bufs)
            bufs = _ptr_array(flat)
        h = ctypes.c_void_p()
        _check(_get_lib().ddp_reducer_create(plan.handle, _ptr_array(grad_arenas), bufs, n, VARIANTS[variant],
                                             float(scale), int(comm_max_blocks),
                                             _stream(comm_stream), ctypes.byref(h)))
        self._h = h.value

    def prepare(self):
        _check(_get_lib().ddp_reducer_prepare(self._h))

    def mark_ready(self, param, stream=None):
        _check(_get_lib().ddp_reducer_mark_ready(self._h, int(param), _stream(stream)))

    def finalize(self, stream=None):
        _check(_get_lib().ddp_reducer_finalize(self._h, _stream(stream)))

    def free(self):
        if self._h:
            _get_lib().ddp_reducer_free(self._h)
            self._h = None

    def __del__(self, _finalizing=sys.is_finalizing):
        if _finalizing():   # as for Plan: no HIP calls during shutdown
            return
        try:
            self.free()
        except Exception:
            pass


def ddp_synthetic_backward(srcs, dsts, work, lds_kib=0, numel=None, dtype=None, stream=None):
    """dsts[r][:numel] = srcs[r][:numel] after `work` FMAs per element (a
    stand-in for the backward kernels that produce gradients)."""
    ptrs, n, numel, dt = _ring_args(srcs, numel, dtype)
    _check(_get_lib().ddp_synthetic_backward(ptrs, _ptr_array(dsts), n, numel, dt, int(work), int(lds_kib),
                                             _stream(stream)))


def ddp_synthetic_backward_pass(plan, src_arenas, grad_arenas, work, reducer=None, lds_kib=0, stream=None):
    """One synthetic backward over the plan's parameters in reverse order,
    marking each gradient ready on `reducer` (if given) as it is produced."""
    _check(_get_lib().ddp_synthetic_backward_pass(plan.handle, _ptr_array(src_arenas), _ptr_array(grad_arenas),
                                                  len(grad_arenas), int(work), int(lds_kib),
                                                  None if reducer is None else reducer._h, _stream(stream)))


def ddp_count_mismatches(bufs, out, count=None, dtype=None, stream=None):
    """Enqueues the count into `out` (a device int64/uint64 tensor of one element)."""
    ptrs, n, count, dt = _ring_args(bufs, count, dtype)
    _check(_get_lib().ddp_count_mismatches(ptrs, n, count, dt, ctypes.c_void_p(_ptr(out)), _stream(stream)))


DDP_ALLOC_CONTIGUOUS = 1

_TORCH_TYPESTR = {torch.float32: "<f4", torch.bfloat16: "<V2", torch.uint8: "|u1"}


class DeviceBuffer:
    """Device memory from ddp_device_alloc, owned by this object (freed by
    free() or when it is collected). `ptr` is the device address; tensor()
    gives a torch view of it (the buffer must outlive the view)."""

    def __init__(self, ptr, nbytes, contiguous):
        self.ptr = ptr
        self.nbytes = nbytes
        self.contiguous = contiguous

    def tensor(self, dtype=torch.float32, numel=None, offset_bytes=0):
        """A 1-D tensor of `numel` elements at ptr + offset_bytes (no copy)."""
        esize = torch.empty((), dtype=dtype).element_size()
        if numel is None:
            numel = (self.nbytes - offset_bytes) // esize
        if self.ptr is None or offset_bytes < 0 or offset_bytes % esize or offset_bytes + numel * esize > self.nbytes:
            raise ValueError("the view does not fit in the buffer")
        # bfloat16 has no array-interface type string: view the bytes, then reinterpret
        view_dtype = dtype if dtype in (torch.float32, torch.uint8) else torch.uint8
        n = numel if view_dtype is dtype else numel * esize

        class _Iface:
            __cuda_array_interface__ = {"shape": (n,), "typestr": _TORCH_TYPESTR[view_dtype],
                                        "data": (self.ptr + offset_bytes, False), "version": 2}
        t = torch.as_tensor(_Iface(), device=torch.device("cuda", torch.cuda.current_device()))
        return t if view_dtype is dtype else t.view(dtype)

    def free(self):
        if self.ptr is not None:
            _check(_get_lib().ddp_device_free(ctypes.c_void_p(self.ptr)))
            self.ptr = None

    def __del__(self, _finalizing=sys.is_finalizing):
        if _finalizing():
            return
        try:
            self.free()
        except Exception:
            pass


def device_alloc(nbytes, contiguous=True):
    """nbytes of device memory on the current device (ddp_device_alloc);
    contiguous=True asks for physically contiguous memory."""
    p = ctypes.c_void_p()
    _check(_get_lib().ddp_device_alloc(int(nbytes), DDP_ALLOC_CONTIGUOUS if contiguous else 0, ctypes.byref(p)))
    return DeviceBuffer(p.value, int(nbytes), bool(contiguous))


def ddp_copy_probe(dst, src, nbytes=None, stream=None):
    if nbytes is None:
        nbytes = src.numel() * src.element_size()
    _check(_get_lib().ddp_copy_probe(ctypes.c_void_p(_ptr(dst)), ctypes.c_void_p(_ptr(src)), int(nbytes),
                              _stream(stream)))


# ---------------------------------------------------------------- around the sync (ddp_train.h)

NORMS = {"l2": 0, "max": 1}


def _empty(shape, dtype, stream):
    """Memory that belongs to `stream` (None: the current one)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device="cuda")
    with torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))):
        return torch.empty(shape, dtype=dtype, device="cuda")


def _device_tensors(tensors, dtype, numels, what):
    tensors = list(tensors)
    if numels is not None and len(tensors) != len(numels):
        raise ValueError(f"{what}: {len(tensors)} tensors for {len(numels)} gradients")
    for i, t in enumerate(tensors):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous() or t.dtype != dtype:
            raise ValueError(f"{what}[{i}] must be a contiguous {dtype} tensor on the GPU")
        if numels is not None and t.numel() != numels[i]:
            raise ValueError(f"{what}[{i}] has {t.numel()} elements, its gradient {numels[i]}")
    return tensors


class GradSet:
    """A set of gradient tensors at fixed places (views of a gradient arena,
    or any others of one dtype on one device): their global norm, and clipping
    (see ddp_grads_* in include/ddp_train.h). Keeps the tensors alive."""

    def __init__(self, tensors):
        tensors = list(tensors)
        dtype = tensors[0].dtype if tensors else torch.float32
        self.dtype = dtype_code(dtype)
        self.tensors = _device_tensors(tensors, dtype, None, "grads")
        self.numels = [t.numel() for t in self.tensors]
        n = len(self.tensors)
        numels = (ctypes.c_int64 * max(n, 1))(*self.numels)
        h = ctypes.c_void_p()
        _check(_get_lib().ddp_grads_create(_ptr_array(self.tensors), numels, n, self.dtype, ctypes.byref(h)))
        self._h = h.value

    def norm(self, kind="l2", out=None, stream=None):
        """The norm, as a float32 device tensor of one element (`out` if given)."""
        if out is None:
            out = _empty((), torch.float32, stream)
        elif out.dtype != torch.float32 or out.numel() != 1:
            raise ValueError("out must hold one float32")
        _check(_get_lib().ddp_grads_norm(self._h, NORMS[kind], out.data_ptr(), _stream(stream)))
        return out

    def clip(self, max_norm, norm, into=None, stream=None):
        """Scales the gradients by min(1, max_norm / (norm + 1e-6)), in place
        or into another GradSet; `norm` is a float32 device tensor."""
        if norm.dtype != torch.float32 or norm.numel() != 1:
            raise ValueError("norm must hold one float32")
        if into is not None and not into._h:   # NULL would mean in place
            raise ValueError("into is freed")
        _check(_get_lib().ddp_grads_clip(self._h, None if into is None else into._h, float(max_norm),
                                         norm.data_ptr(), _stream(stream)))

    def free(self):
        if self._h:
            _get_lib().ddp_grads_free(self._h)
            self._h = None

    def __del__(self, _finalizing=sys.is_finalizing):
        if _finalizing():   # as for Plan: no HIP calls during shutdown
            return
        try:
            self.free()
        except Exception:
            pass


class AdamW:
    """AdamW on fp32 parameters whose gradients are the GradSet `grads` (see
    ddp_adamw_* in include/ddp_train.h). params, exp_avg, exp_avg_sq: float32
    tensors, one per gradient; steps: an int64 device tensor of one element,
    the steps done; params_bf16: tensors that receive the rounded weights;
    decay: per tensor, whether weight decay applies (None: to all). The
    tensors are updated in place and kept alive."""

    def __init__(self, grads, params, exp_avg, exp_avg_sq, steps, params_bf16=None, decay=None):
        if steps.dtype != torch.int64 or steps.numel() != 1:
            raise ValueError("steps must hold one int64")
        n = len(grads.numels)
        if decay is not None and len(decay) != n:
            raise ValueError(f"decay: {len(decay)} entries for {n} gradients")
        self.grads = grads   # the set must outlive the optimizer
        self.params = _device_tensors(params, torch.float32, grads.numels, "params")
        self.exp_avg = _device_tensors(exp_avg, torch.float32, grads.numels, "exp_avg")
        self.exp_avg_sq = _device_tensors(exp_avg_sq, torch.float32, grads.numels, "exp_avg_sq")
        self.params_bf16 = None if params_bf16 is None else \
            _device_tensors(params_bf16, torch.bfloat16, grads.numels, "params_bf16")
        self.steps = steps
        flags = None if decay is None else (ctypes.c_uint8 * max(n, 1))(*[1 if d else 0 for d in decay])
        h = ctypes.c_void_p()
        _check(_get_lib().ddp_adamw_create(grads._h, _ptr_array(self.params), _ptr_array(self.exp_avg),
                                           _ptr_array(self.exp_avg_sq),
                                           None if params_bf16 is None else _ptr_array(self.params_bf16), flags,
                                           steps.data_ptr(), ctypes.byref(h)))
        self._h = h.value

    def step(self, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, max_norm=None, norm=None, stream=None):
        """One step. With `norm` (a float32 device tensor) and max_norm the
        gradients count as clipped, and a norm that is not finite skips it."""
        if (norm is None) != (max_norm is None):
            raise ValueError("norm and max_norm go together")
        if norm is not None and (norm.dtype != torch.float32 or norm.numel() != 1):
            raise ValueError("norm must hold one float32")
        _check(_get_lib().ddp_adamw_step(self._h, float(lr), float(betas[0]), float(betas[1]), float(eps),
                                         float(weight_decay), 0.0 if max_norm is None else float(max_norm),
                                         None if norm is None else norm.data_ptr(), _stream(stream)))

    def free(self):
        if self._h:
            _get_lib().ddp_adamw_free(self._h)
            self._h = None

    def __del__(self, _finalizing=sys.is_finalizing):
        if _finalizing():   # as for Plan: no HIP calls during shutdown
            return
        try:
            self.free()
        except Exception:
            pass


ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
LINEAR_FORWARD, LINEAR_BACKWARD_INPUT, LINEAR_BACKWARD_WEIGHT = 0, 1, 2


def linear_workspace(direction, m, n, k, dtype):
    """Bytes of scratch that a linear call of these sizes needs."""
    return _linear_workspace(int(direction), int(m), int(n), int(k), dtype_code(dtype))


def linear_tiling(direction, m, n, k, dtype, direct=True):
    """(tile, parts): the side of the square tiles that a product of these
    sizes is cut into (0: a few rows, without tiles) and the parts of its sum;
    direct: the operands' rows are whole, aligned 16-byte chunks (see
    ddp_linear_tiling in include/ddp_train.h)."""
    tile, parts = ctypes.c_int32(), ctypes.c_int32()
    _check(_get_lib().ddp_linear_tiling(int(direction), int(m), int(n), int(k), dtype_code(dtype), 1 if direct else 0,
                                        ctypes.byref(tile), ctypes.byref(parts)))
    return tile.value, parts.value


@functools.lru_cache(maxsize=4096)
def _linear_workspace(direction, m, n, k, code):
    b = ctypes.c_int64()
    _check(_get_lib().ddp_linear_workspace(direction, m, n, k, code, ctypes.byref(b)))
    return b.value


def _matrix(t, rows, cols, dtype, what):
    """(pointer, leading dimension) of a rows x cols matrix; (None, cols) for None."""
    if t is None:
        return None, cols
    if t.dtype is not dtype or t.shape != (rows, cols) or not t.is_cuda:
        raise ValueError(f"{what} must be a {rows} x {cols} matrix of {dtype} on the GPU")
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"the rows of {what} must be contiguous")
    return t.data_ptr(), (ld if rows > 1 else max(cols, 1))


def _vector(t, n, dtype, what):
    if t is None:
        return None
    if not t.is_cuda or t.numel() != n or t.dim() != 1 or not t.is_contiguous() or t.dtype != dtype:
        raise ValueError(f"{what} must be a contiguous vector of {n} {dtype} on the GPU")
    return t.data_ptr()


def _scratch(nbytes, workspace, stream):
    """The caller's workspace, or torch memory that belongs to the stream."""
    if workspace is None:
        if not nbytes:
            return None, (0, None)
        workspace = _empty(nbytes, torch.uint8, stream)
        return workspace, (nbytes, workspace.data_ptr())
    if not workspace.is_cuda or not workspace.is_contiguous():   # else it spans more, or less, than its elements
        raise ValueError("workspace must be a contiguous tensor on the GPU")
    return workspace, (workspace.numel() * workspace.element_size(), workspace.data_ptr())


def _result(out, rows, cols, dtype, stream):
    return _empty((rows, cols), dtype, stream) if out is None else out


def linear_forward(x, w, bias=None, residual=None, act="none", keep=False, out=None, z=None, workspace=None, stream=None):
    """act(x w^T + bias) + residual; with keep=True (or a matrix z to fill)
    the pair (y, z), z = x w^T + bias as the backward pass takes it (see
    ddp_linear_forward in include/ddp_train.h)."""
    m, k = x.shape
    n, dt = w.shape[0], x.dtype
    code = dtype_code(dt)
    y = _result(out, m, n, dt, stream)
    if keep and z is None:
        z = _result(None, m, n, dt, stream)
    xp, ldx = _matrix(x, m, k, dt, "x")
    wp, ldw = _matrix(w, n, k, dt, "w")
    rp, ldr = _matrix(residual, m, n, dt, "residual")
    yp, ldy = _matrix(y, m, n, dt, "out")
    zp, ldz = _matrix(z, m, n, dt, "z")
    ws, (nbytes, p) = _scratch(_linear_workspace(LINEAR_FORWARD, m, n, k, code), workspace, stream)
    _check(_get_lib().ddp_linear_forward(xp, ldx, wp, ldw, _vector(bias, n, dt, "bias"), rp, ldr, yp, ldy, zp, ldz,
                                         m, n, k, code, ACTIVATIONS[act], p, nbytes, _stream(stream)))
    return y if z is None else (y, z)


def linear_backward_input(dz, w, act="none", z=None, add=None, out=None, workspace=None, stream=None):
    """(dz w) * act'(z) + add: the gradient of the layer's input, through the
    activation of the layer before it (see ddp_linear_backward_input)."""
    m, n = dz.shape
    k, dt = w.shape[1], dz.dtype
    code = dtype_code(dt)
    dx = _result(out, m, k, dt, stream)
    gp, ldg = _matrix(dz, m, n, dt, "dz")
    wp, ldw = _matrix(w, n, k, dt, "w")
    zp, ldz = _matrix(z, m, k, dt, "z")
    ap, lda = _matrix(add, m, k, dt, "add")
    op, ldo = _matrix(dx, m, k, dt, "out")
    ws, (nbytes, p) = _scratch(_linear_workspace(LINEAR_BACKWARD_INPUT, m, n, k, code), workspace, stream)
    _check(_get_lib().ddp_linear_backward_input(gp, ldg, wp, ldw, zp, ldz, ap, lda, op, ldo, m, n, k, code,
                                                ACTIVATIONS[act], p, nbytes, _stream(stream)))
    return dx


def linear_backward_weight(dz, x, dw, db=None, accumulate=False, workspace=None, stream=None):
    """dw (+)= dz^T x and db (+)= the sum of dz's rows, into tensors of the
    data's dtype or float32, e.g. views of a gradient arena (see
    ddp_linear_backward_weight)."""
    m, n = dz.shape
    k, dt, gt = x.shape[1], dz.dtype, dw.dtype
    code = dtype_code(dt)
    gp, ldg = _matrix(dz, m, n, dt, "dz")
    xp, ldx = _matrix(x, m, k, dt, "x")
    wp, ldw = _matrix(dw, n, k, gt, "dw")
    bp = _vector(db, n, gt, "db")
    ws, (nbytes, p) = _scratch(_linear_workspace(LINEAR_BACKWARD_WEIGHT, m, n, k, code), workspace, stream)
    _check(_get_lib().ddp_linear_backward_weight(gp, ldg, xp, ldx, wp, ldw, bp, m, n, k, code, dtype_code(gt),
                                                 1 if accumulate else 0, p, nbytes, _stream(stream)))


def act_backward(dy, z, act, out=None, stream=None):
    """dy * act'(z), element by element; out may be dy."""
    m, n = dy.shape
    dt = dy.dtype
    dz = _result(out, m, n, dt, stream)
    yp, ldy = _matrix(dy, m, n, dt, "dy")
    zp, ldz = _matrix(z, m, n, dt, "z")
    op, ldo = _matrix(dz, m, n, dt, "out")
    _check(_get_lib().ddp_act_backward(yp, ldy, zp, ldz, op, ldo, m, n, dtype_code(dt), ACTIVATIONS[act], _stream(stream)))
    return dz


def _offsets(t, n, what="offsets"):
    if not t.is_cuda or t.dtype != torch.int64 or t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous vector of {n} int64 on the GPU")
    return t.data_ptr()


def _expert_matrices(t, e, n, k, dtype, what):
    """(pointer, leading dimension) of e matrices n x k whose rows follow each other at one pitch."""
    if t.dtype is not dtype or t.shape != (e, n, k) or not t.is_cuda:
        raise ValueError(f"{what} must be {e} matrices {n} x {k} of {dtype} on the GPU")
    group, ld, step = t.stride()
    if (step != 1 and k > 1) or (e > 1 and n > 1 and group != n * ld):
        raise ValueError(f"the rows of {what} must be contiguous and evenly spaced")
    if n <= 1:
        ld = group if e > 1 else max(k, 1)
    return t.data_ptr(), ld


def _expert_vectors(t, e, n, dtype, what):
    if t is None:
        return None
    if not t.is_cuda or t.shape != (e, n) or not t.is_contiguous() or t.dtype != dtype:
        raise ValueError(f"{what} must be a contiguous {e} x {n} matrix of {dtype} on the GPU")
    return t.data_ptr()


@functools.lru_cache(maxsize=4096)
def _experts_workspace(direction, t, e, n, k, code):
    b = ctypes.c_int64()
    _check(_get_lib().ddp_experts_workspace(direction, t, e, n, k, code, ctypes.byref(b)))
    return b.value


def experts_workspace(direction, t, e, n, k, dtype):
    """Bytes of scratch that an experts' call of these sizes needs (direction
    LINEAR_FORWARD, LINEAR_BACKWARD_INPUT or LINEAR_BACKWARD_WEIGHT)."""
    return _experts_workspace(int(direction), int(t), int(e), int(n), int(k), dtype_code(dtype))


def experts_tiling(direction, t, e, n, k, dtype, direct=True):
    """(rows, columns, parts): the tiles that a direction's products are cut
    into and the parts of their sums (see ddp_experts_tiling)."""
    out = [ctypes.c_int32() for _ in range(3)]
    _check(_get_lib().ddp_experts_tiling(int(direction), int(t), int(e), int(n), int(k), dtype_code(dtype), 1 if direct else 0,
                                         *(ctypes.byref(o) for o in out)))
    return tuple(o.value for o in out)


def experts_forward(x, w, offsets, bias=None, act="none", keep=False, out=None, z=None, workspace=None, stream=None):
    """act(x_i w_e^T + bias_e) over rows sorted by expert: expert e has the rows
    offsets[e] to offsets[e + 1] (int64, on the GPU) of x and the matrix w[e].
    With keep=True (or a matrix z to fill) the pair (y, z). Rows of no expert
    stay as they are in out and z, and are undefined in new ones (see
    ddp_experts_forward in include/ddp_train.h)."""
    t, k = x.shape
    e, n = w.shape[0], w.shape[1]
    dt = x.dtype
    code = dtype_code(dt)
    y = _result(out, t, n, dt, stream)
    if keep and z is None:
        z = _result(None, t, n, dt, stream)
    xp, ldx = _matrix(x, t, k, dt, "x")
    wp, ldw = _expert_matrices(w, e, n, k, dt, "w")
    yp, ldy = _matrix(y, t, n, dt, "out")
    zp, ldz = _matrix(z, t, n, dt, "z")
    ws, (nbytes, p) = _scratch(_experts_workspace(LINEAR_FORWARD, t, e, n, k, code), workspace, stream)
    _check(_get_lib().ddp_experts_forward(xp, ldx, wp, ldw, _expert_vectors(bias, e, n, dt, "bias"), _offsets(offsets, e + 1),
                                          yp, ldy, zp, ldz, t, e, n, k, code, ACTIVATIONS[act], p, nbytes, _stream(stream)))
    return y if z is None else (y, z)


def experts_backward_input(dz, w, offsets, act="none", z=None, out=None, workspace=None, stream=None):
    """(dz_i w_e) * act'(z_i) (see ddp_experts_backward_input)."""
    t, n = dz.shape
    e, k = w.shape[0], w.shape[2]
    dt = dz.dtype
    dx = _result(out, t, k, dt, stream)
    gp, ldg = _matrix(dz, t, n, dt, "dz")
    wp, ldw = _expert_matrices(w, e, n, k, dt, "w")
    zp, ldz = _matrix(z, t, k, dt, "z")
    op, ldo = _matrix(dx, t, k, dt, "out")
    code = dtype_code(dt)
    ws, (nbytes, p) = _scratch(_experts_workspace(LINEAR_BACKWARD_INPUT, t, e, n, k, code), workspace, stream)
    _check(_get_lib().ddp_experts_backward_input(gp, ldg, wp, ldw, _offsets(offsets, e + 1), zp, ldz, op, ldo, t, e, n, k, code,
                                                 ACTIVATIONS[act], p, nbytes, _stream(stream)))
    return dx


def experts_backward_weight(dz, x, offsets, dw, db=None, accumulate=False, workspace=None, stream=None):
    """dw[e] (+)= dz_i^T x_i and db[e] (+)= dz_i, summed over each expert's
    rows, into tensors of the data's dtype or float32, e.g. views of a gradient
    arena (see ddp_experts_backward_weight)."""
    t, n = dz.shape
    e, k = dw.shape[0], x.shape[1]
    dt, gt = dz.dtype, dw.dtype
    code = dtype_code(dt)
    gp, ldg = _matrix(dz, t, n, dt, "dz")
    xp, ldx = _matrix(x, t, k, dt, "x")
    wp, ldw = _expert_matrices(dw, e, n, k, gt, "dw")
    bp = _expert_vectors(db, e, n, gt, "db")
    ws, (nbytes, p) = _scratch(_experts_workspace(LINEAR_BACKWARD_WEIGHT, t, e, n, k, code), workspace, stream)
    _check(_get_lib().ddp_experts_backward_weight(gp, ldg, xp, ldx, _offsets(offsets, e + 1), wp, ldw, bp, t, e, n, k, code,
                                                  dtype_code(gt), 1 if accumulate else 0, p, nbytes, _stream(stream)))


LOSS_FORWARD, LOSS_BACKWARD = 0, 1


@functools.lru_cache(maxsize=4096)
def _loss_workspace(direction, m, v, k, top, code, grad_code):
    b = ctypes.c_int64()
    if top:
        _check(_get_lib().ddp_distill_workspace(direction, m, v, k, top, code, grad_code, ctypes.byref(b)))
    else:
        _check(_get_lib().ddp_cross_entropy_workspace(direction, m, v, k, code, grad_code, ctypes.byref(b)))
    return b.value


def cross_entropy_workspace(direction, m, v, k, dtype, grad_dtype=None):
    """Bytes of scratch that a cross entropy call of these sizes needs
    (direction LOSS_FORWARD or LOSS_BACKWARD)."""
    code = dtype_code(dtype)
    return _loss_workspace(int(direction), int(m), int(v), int(k), 0, code, code if grad_dtype is None else dtype_code(grad_dtype))


def distill_workspace(direction, m, v, k, top, dtype, grad_dtype=None):
    """Bytes of scratch that a distillation call of these sizes needs."""
    code = dtype_code(dtype)
    if int(top) < 1:
        raise ValueError("a row has at least one entry")
    return _loss_workspace(int(direction), int(m), int(v), int(k), int(top), code,
                           code if grad_dtype is None else dtype_code(grad_dtype))


LOSS_Z, LOSS_Z_AGAIN, LOSS_DX, LOSS_DW = 0, 1, 2, 3


def loss_tiling(product, m, v, k, dtype, grad_dtype=None, direct=True):
    """(rows, columns, parts, piece): the tiles that a loss's product (LOSS_Z,
    LOSS_Z_AGAIN, LOSS_DX or LOSS_DW) is cut into, the parts of its sums, and the
    columns of the vocabulary that it takes at a time (see ddp_loss_tiling)."""
    out, piece = [ctypes.c_int32() for _ in range(3)], ctypes.c_int64()
    code = dtype_code(dtype)
    _check(_get_lib().ddp_loss_tiling(int(product), int(m), int(v), int(k), code, code if grad_dtype is None else dtype_code(grad_dtype),
                                      1 if direct else 0, *(ctypes.byref(o) for o in out), ctypes.byref(piece)))
    return (*(o.value for o in out), piece.value)


def _row_values(t, m, what, stream):
    """A float32 vector of m elements, made if it is None."""
    t = _empty((m,), torch.float32, stream) if t is None else t
    return t, _vector(t, m, torch.float32, what)


def _entries(ids, teacher, m):
    """Arguments of a teacher's entries: (ids, ld, logits, ld, logits' dtype, entries a row)."""
    c = ids.shape[1] if ids.dim() == 2 else 0
    if c < 1:
        raise ValueError("ids must be a matrix with at least one entry a row")
    ip, ldi = _matrix(ids, m, c, torch.int64, "ids")
    tp, ldt = _matrix(teacher, m, c, teacher.dtype, "teacher")
    return ip, ldi, tp, ldt, dtype_code(teacher.dtype), c


def _loss_shapes(x, w):
    """(m, v, k, dtype, its code, x's and w's arguments)."""
    m, k = x.shape
    v, dt = w.shape[0], x.dtype
    xp, ldx = _matrix(x, m, k, dt, "x")
    wp, ldw = _matrix(w, v, k, dt, "w")
    return m, v, k, dt, dtype_code(dt), (xp, ldx, wp, ldw)


def _gradients(dx, dw, m, v, k, dt):
    """Arguments of dx and dw (None: not wanted), and the code of dw's dtype."""
    op, ldo = _matrix(dx, m, k, dt, "out")
    gt = dt if dw is None else dw.dtype
    gp, ldg = _matrix(dw, v, k, gt, "dw")
    return (op, ldo, gp, ldg), dtype_code(gt)


def cross_entropy_forward(x, w, targets, loss=None, lse=None, workspace=None, stream=None):
    """(loss, lse) of every row of z = x w^T with an int64 target a row
    (negative: the row does not count), float32, without a matrix of z (see
    ddp_cross_entropy_forward in include/ddp_train.h)."""
    m, v, k, dt, code, xw = _loss_shapes(x, w)
    loss, lossp = _row_values(loss, m, "loss", stream)
    lse, lsep = _row_values(lse, m, "lse", stream)
    ws, (nbytes, p) = _scratch(_loss_workspace(LOSS_FORWARD, m, v, k, 0, code, code), workspace, stream)
    _check(_get_lib().ddp_cross_entropy_forward(*xw, _vector(targets, m, torch.int64, "targets"), lossp, lsep, m, v, k, code,
                                                p, nbytes, _stream(stream)))
    return loss, lse


def cross_entropy_backward(x, w, targets, lse, dloss, dw=None, accumulate=False, out=None, need_dx=True, workspace=None, stream=None):
    """dx (None with need_dx=False), with dw (+)= the gradient of w where a
    tensor is given: the gradients of sum(dloss * loss); lse as
    cross_entropy_forward gave it (see ddp_cross_entropy_backward)."""
    m, v, k, dt, code, xw = _loss_shapes(x, w)
    dx = _result(out, m, k, dt, stream) if need_dx else None
    grads, grad_code = _gradients(dx, dw, m, v, k, dt)
    ws, (nbytes, p) = _scratch(_loss_workspace(LOSS_BACKWARD, m, v, k, 0, code, grad_code), workspace, stream)
    _check(_get_lib().ddp_cross_entropy_backward(*xw, _vector(targets, m, torch.int64, "targets"),
                                                 _vector(lse, m, torch.float32, "lse"), _vector(dloss, m, torch.float32, "dloss"),
                                                 *grads, m, v, k, code, grad_code, 1 if accumulate else 0, p, nbytes,
                                                 _stream(stream)))
    return dx


def distill_forward(x, w, ids, teacher, temperature=1.0, loss=None, lse=None, workspace=None, stream=None):
    """(loss, lse) of every row: temperature^2 times the divergence of
    softmax(x w^T / temperature) from the softmax of a teacher's logits /
    temperature at `ids` (int64; negative, or a logit of -inf: left out). See
    ddp_distill_forward in include/ddp_train.h."""
    m, v, k, dt, code, xw = _loss_shapes(x, w)
    entries = _entries(ids, teacher, m)
    loss, lossp = _row_values(loss, m, "loss", stream)
    lse, lsep = _row_values(lse, m, "lse", stream)
    ws, (nbytes, p) = _scratch(_loss_workspace(LOSS_FORWARD, m, v, k, entries[5], code, code), workspace, stream)
    _check(_get_lib().ddp_distill_forward(*xw, *entries[:5], float(temperature), lossp, lsep, m, v, k, entries[5], code, p, nbytes,
                                          _stream(stream)))
    return loss, lse


def distill_backward(x, w, ids, teacher, lse, dloss, temperature=1.0, dw=None, accumulate=False, out=None, need_dx=True,
                     workspace=None, stream=None):
    """The gradients of sum(dloss * loss), as cross_entropy_backward gives
    them (see ddp_distill_backward)."""
    m, v, k, dt, code, xw = _loss_shapes(x, w)
    entries = _entries(ids, teacher, m)
    dx = _result(out, m, k, dt, stream) if need_dx else None
    grads, grad_code = _gradients(dx, dw, m, v, k, dt)
    ws, (nbytes, p) = _scratch(_loss_workspace(LOSS_BACKWARD, m, v, k, entries[5], code, grad_code), workspace, stream)
    _check(_get_lib().ddp_distill_backward(*xw, *entries[:5], float(temperature), _vector(lse, m, torch.float32, "lse"),
                                           _vector(dloss, m, torch.float32, "dloss"), *grads, m, v, k, entries[5], code, grad_code,
                                           1 if accumulate else 0, p, nbytes, _stream(stream)))
    return dx
