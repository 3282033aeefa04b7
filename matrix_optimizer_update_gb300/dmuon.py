"""ctypes binding of the C ABI in include/dmuon.h.

Argument marshalling only: every step of the update runs in the library's
CUDA kernels. PyTorch is used by callers for device memory and streams; the
functions here take plain integers (device addresses, stream handles).

Loading fails loudly (``DmuonError``) when the shared library has not been
built: there is no fallback implementation.
"""

from __future__ import annotations

import ctypes
import json
import os
from array import array
from dataclasses import dataclass

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdmuon.so")

OK = 0
ERR_INVALID_ARG = -1
ERR_UNSUPPORTED = -2
ERR_WORKSPACE = -3
ERR_CUDA = -4
ERR_NOT_BOUND = -5
ERR_DEVICE = -6

F32 = 0
BF16 = 1
DTYPE = {"f32": F32, "bf16": BF16}

FLAG_CAPTURE_UPDATE = 0x1
FLAG_GRAM_NS = 0x2
FLAG_TUNE = 0x4
FLAG_PAIR_TILES = 0x8
FLAG_EPILOGUE_AX = 0x10
FLAG_STATIC_TILES = 0x20
FLAG_DEBUG_CHECKS = 0x40
FLAG_ONE_SM_TILES = 0x80
DEV_NONFINITE_NORM = 0x1
DEV_WAIT_TIMEOUT = 0x2

KIND_MOMENTUM, KIND_GRAM, KIND_POLY, KIND_GEMM, KIND_UPDATE0, KIND_SYMM, KIND_NORM = range(7)
KIND_NAMES = {0: "momentum", 1: "gram", 2: "poly", 3: "gemm", 4: "update0", 5: "symm", 6: "norm"}

# every symbol include/dmuon.h declares
EXPORTS = (
    "dmuon_plan", "dmuon_plan_workspace_bytes", "dmuon_plan_bind", "dmuon_step",
    "dmuon_set_weight_events", "dmuon_read_device_status", "dmuon_read_update", "dmuon_plan_describe",
    "dmuon_profile_begin", "dmuon_profile_end", "dmuon_profile_cta_times", "dmuon_read_cta_times",
    "dmuon_plan_costs", "dmuon_launch_count",
    "dmuon_selftest_wait_timeout", "dmuon_momentum_norm_noalloc", "dmuon_assign_owners", "dmuon_adamw_flat",
    "dmuon_head_create", "dmuon_head_workspace_bytes", "dmuon_head_scores_workspace_bytes", "dmuon_head_bind",
    "dmuon_head_xent", "dmuon_head_xent_backward", "dmuon_head_xent_backward_loss", "dmuon_head_distill", "dmuon_head_distill_backward",
    "dmuon_head_logprobs", "dmuon_head_logprobs_backward",
    "dmuon_head_read_device_status", "dmuon_head_destroy",
    "dmuon_route_workspace_bytes", "dmuon_route_sort", "dmuon_route_dispatch", "dmuon_route_combine",
    "dmuon_route_combine_backward",
    "dmuon_experts_workspace_bytes", "dmuon_experts_forward", "dmuon_experts_read_device_status",
    "dmuon_clip_workspace_bytes", "dmuon_grad_norm", "dmuon_grad_clip",
    "dmuon_plan_destroy", "dmuon_last_error", "dmuon_version",
)


class DmuonError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"dmuon status {status}: {msg}")
        self.status = status


class Shape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class Dtypes(ctypes.Structure):
    _fields_ = [("param", ctypes.c_int32), ("grad", ctypes.c_int32),
                ("momentum", ctypes.c_int32), ("compute", ctypes.c_int32)]


_lib = None


def lib():
    """Load libdmuon.so (once). Raises DmuonError if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise DmuonError(ERR_CUDA, f"{LIB_PATH} is not built; run python -m matrix_optimizer_update_gb300.build")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, u32, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32,
                                  ctypes.c_float, ctypes.c_size_t)
    sig = {
        "dmuon_plan": (i32, [ctypes.POINTER(Shape), i32, i32, ctypes.POINTER(f32), i32, f32, Dtypes, u32,
                             ctypes.POINTER(vp)]),
        "dmuon_plan_workspace_bytes": (i32, [vp, ctypes.POINTER(sz)]),
        "dmuon_plan_bind": (i32, [vp, vp, sz, vp]),
        "dmuon_step": (i32, [vp, ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(vp), f32, f32, i32, vp]),
        "dmuon_set_weight_events": (i32, [vp, vp, vp]),
        "dmuon_read_device_status": (i32, [vp, vp, ctypes.POINTER(u32)]),
        "dmuon_read_update": (i32, [vp, i32, vp, vp]),
        "dmuon_plan_describe": (i32, [vp, ctypes.c_char_p, sz, ctypes.POINTER(sz)]),
        "dmuon_profile_begin": (i32, [vp, i32]),
        "dmuon_profile_end": (i32, [vp, ctypes.POINTER(i32), ctypes.POINTER(f32), ctypes.POINTER(ctypes.c_double),
                                    i32, ctypes.POINTER(i32)]),
        "dmuon_profile_cta_times": (i32, [vp, i32]),
        "dmuon_read_cta_times": (i32, [vp, i32, ctypes.POINTER(ctypes.c_uint64), i32, ctypes.POINTER(i32), vp]),
        "dmuon_plan_costs": (i32, [vp, ctypes.POINTER(ctypes.c_double), i32]),
        "dmuon_launch_count": (i32, [vp, ctypes.POINTER(i64)]),
        "dmuon_selftest_wait_timeout": (i32, [vp, i64, vp, ctypes.POINTER(u32)]),
        "dmuon_momentum_norm_noalloc": (i32, [vp, vp, vp, vp, i64, i64, i32, i32, f32, i32, f32, vp]),
        "dmuon_assign_owners": (i32, [ctypes.POINTER(Shape), i32, i32, ctypes.POINTER(ctypes.c_double), i32,
                                      ctypes.POINTER(i32), ctypes.POINTER(ctypes.c_double)]),
        "dmuon_adamw_flat": (i32, [vp, vp, vp, vp, i64, i32, i32, f32, f32, f32, f32, f32, i32, vp]),
        "dmuon_head_create": (i32, [i64, i64, i64, i32, ctypes.POINTER(vp)]),
        "dmuon_head_workspace_bytes": (i32, [vp, ctypes.POINTER(sz)]),
        "dmuon_head_scores_workspace_bytes": (i32, [vp, ctypes.POINTER(sz)]),
        "dmuon_head_bind": (i32, [vp, vp, sz, vp]),
        "dmuon_head_xent": (i32, [vp, vp, i64, vp, i64, vp, i64, vp, vp, vp]),
        "dmuon_head_xent_backward": (i32, [vp, vp, i64, vp, i64, vp, i64, vp, vp, vp, i64, vp, i64, vp]),
        "dmuon_head_xent_backward_loss": (i32, [vp, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, i64, vp, i64, vp]),
        "dmuon_head_distill": (i32, [vp, vp, i64, vp, i64, vp, vp, i32, f32, i64, vp, vp, vp]),
        "dmuon_head_distill_backward": (i32, [vp, vp, i64, vp, i64, vp, vp, i32, f32, i64, vp, vp, vp, i64, vp, i64,
                                              vp]),
        "dmuon_head_logprobs": (i32, [vp, vp, i64, vp, i64, vp, f32, i32, i64, vp, vp, vp, vp, vp, vp]),
        "dmuon_head_logprobs_backward": (i32, [vp, vp, i64, vp, i64, vp, f32, i64, vp, vp, vp, vp, vp, vp, i64, vp, i64,
                                               vp]),
        "dmuon_head_read_device_status": (i32, [vp, vp, ctypes.POINTER(u32)]),
        "dmuon_head_destroy": (None, [vp]),
        "dmuon_route_workspace_bytes": (i32, [i64, i32, i32, ctypes.POINTER(sz)]),
        "dmuon_route_sort": (i32, [vp, i64, i32, i32, vp, vp, vp, vp, sz, vp]),
        "dmuon_route_dispatch": (i32, [vp, i64, vp, vp, i64, i32, i64, i32, vp, vp]),
        "dmuon_route_combine": (i32, [vp, vp, vp, i64, i32, i64, i32, vp, i64, vp]),
        "dmuon_route_combine_backward": (i32, [vp, i64, vp, vp, vp, vp, i64, i32, i64, i32, vp, vp, vp]),
        "dmuon_experts_workspace_bytes": (i32, [i64, i32, i32, i64, i64, ctypes.POINTER(sz)]),
        "dmuon_experts_forward": (i32, [vp, i64, vp, vp, i64, i32, i32, i64, i64, vp, vp, vp, vp, i64, vp, sz, vp]),
        "dmuon_experts_read_device_status": (i32, [vp, vp, ctypes.POINTER(u32)]),
        "dmuon_clip_workspace_bytes": (i32, [ctypes.POINTER(sz)]),
        "dmuon_grad_norm": (i32, [vp, vp, vp, i32, vp, vp, sz, vp]),
        "dmuon_grad_clip": (i32, [vp, vp, vp, vp, i32, f32, vp, vp, sz, vp]),
        "dmuon_plan_destroy": (None, [vp]),
        "dmuon_last_error": (ctypes.c_char_p, []),
        "dmuon_version": (i32, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def _check(st: int):
    if st != OK:
        raise DmuonError(st, lib().dmuon_last_error().decode())


def _ptr_array(ptrs):
    arr = (ctypes.c_void_p * len(ptrs))()
    for i, p in enumerate(ptrs):
        arr[i] = int(p)
    return arr


def dmuon_version() -> int:
    return lib().dmuon_version()


def dmuon_plan(shapes, ns_steps=5, coeffs=(3.4445, -4.7750, 2.0315), eps=1e-7,
               param="bf16", grad="bf16", compute="bf16", flags=0) -> "Plan":
    """Build a plan (host only). ``coeffs`` is one (a, b, c) or ns_steps triples."""
    n = len(shapes)
    sh = (Shape * max(n, 1))(*[Shape(int(r), int(c)) for r, c in shapes])
    flat = []
    if coeffs is not None and len(coeffs) and isinstance(coeffs[0], (tuple, list)):
        for t in coeffs:
            flat.extend(t)
        triples = len(coeffs)
    elif coeffs is not None:
        flat = list(coeffs)
        triples = 1
    else:
        triples = 0
    cf = (ctypes.c_float * max(len(flat), 1))(*flat) if flat else None
    dt = Dtypes(DTYPE[param], DTYPE[grad], F32, DTYPE[compute])
    h = ctypes.c_void_p()
    _check(lib().dmuon_plan(sh if n else None, n, ns_steps, cf, triples, eps, dt, flags, ctypes.byref(h)))
    return Plan(h, list(shapes), ns_steps)


class Plan:
    """Owns a ``dmuon_plan_t`` handle; thin wrappers over the C calls."""

    def __init__(self, handle, shapes, ns_steps):
        self._h = handle
        self.shapes = shapes
        self.ns_steps = ns_steps
        self._ptr_cache = None

    @property
    def handle(self):
        return self._h

    def workspace_bytes(self) -> int:
        n = ctypes.c_size_t()
        _check(lib().dmuon_plan_workspace_bytes(self._h, ctypes.byref(n)))
        return n.value

    def bind(self, d_workspace: int, nbytes: int, stream: int = 0):
        _check(lib().dmuon_plan_bind(self._h, ctypes.c_void_p(d_workspace), nbytes, ctypes.c_void_p(stream)))

    def step(self, params, grads, momenta, lr, mu, nesterov, stream: int = 0):
        key = (tuple(params), tuple(grads), tuple(momenta))
        if self._ptr_cache is None or self._ptr_cache[0] != key:
            self._ptr_cache = (key, _ptr_array(params), _ptr_array(grads), _ptr_array(momenta))
        _, pa, ga, ma = self._ptr_cache
        _check(lib().dmuon_step(self._h, pa, ga, ma, float(lr), float(mu), int(bool(nesterov)),
                                ctypes.c_void_p(stream)))

    def set_weight_events(self, wait_before_write: int = 0, after_write: int = 0):
        """cudaEvent_t handles (ints, 0 = none): see dmuon_set_weight_events."""
        _check(lib().dmuon_set_weight_events(self._h, ctypes.c_void_p(wait_before_write or None),
                                             ctypes.c_void_p(after_write or None)))

    def read_device_status(self, stream: int = 0) -> int:
        b = ctypes.c_uint32()
        _check(lib().dmuon_read_device_status(self._h, ctypes.c_void_p(stream), ctypes.byref(b)))
        return b.value

    def read_update(self, mat: int, d_dst: int, stream: int = 0):
        _check(lib().dmuon_read_update(self._h, mat, ctypes.c_void_p(d_dst), ctypes.c_void_p(stream)))

    def describe(self) -> dict:
        need = ctypes.c_size_t()
        _check(lib().dmuon_plan_describe(self._h, None, 0, ctypes.byref(need)))
        buf = ctypes.create_string_buffer(need.value)
        _check(lib().dmuon_plan_describe(self._h, buf, need.value, ctypes.byref(need)))
        return json.loads(buf.value.decode())

    def profile_begin(self, max_launches: int):
        _check(lib().dmuon_profile_begin(self._h, max_launches))

    def profile_end(self, cap: int):
        kinds = (ctypes.c_int32 * cap)()
        ms = (ctypes.c_float * cap)()
        work = (ctypes.c_double * cap)()
        n = ctypes.c_int32()
        _check(lib().dmuon_profile_end(self._h, kinds, ms, work, cap, ctypes.byref(n)))
        k = min(n.value, cap)
        return [(kinds[i], ms[i], work[i]) for i in range(k)]

    def profile_cta_times(self, enable: bool = True):
        _check(lib().dmuon_profile_cta_times(self._h, int(bool(enable))))

    def read_cta_times(self, launch: int, stream: int = 0):
        """[(start_ns, end_ns)] per CTA of launch `launch` of the last recorded step."""
        n = ctypes.c_int32()
        _check(lib().dmuon_read_cta_times(self._h, launch, None, 0, ctypes.byref(n), ctypes.c_void_p(stream)))
        if n.value == 0:
            return []
        buf = (ctypes.c_uint64 * (2 * n.value))()
        _check(lib().dmuon_read_cta_times(self._h, launch, buf, n.value, ctypes.byref(n), ctypes.c_void_p(stream)))
        return [(buf[2 * i], buf[2 * i + 1]) for i in range(n.value)]

    def costs(self):
        """Measured per-matrix cost (ms) of a tuned plan."""
        n = len(self.shapes)
        out = (ctypes.c_double * n)()
        _check(lib().dmuon_plan_costs(self._h, out, n))
        return list(out)

    def launch_count(self) -> int:
        c = ctypes.c_int64()
        _check(lib().dmuon_launch_count(self._h, ctypes.byref(c)))
        return c.value

    def destroy(self):
        if self._h is not None and self._h.value:
            lib().dmuon_plan_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def dmuon_selftest_wait_timeout(d_scratch: int, limit_ns: int, stream: int = 0) -> int:
    b = ctypes.c_uint32()
    _check(lib().dmuon_selftest_wait_timeout(ctypes.c_void_p(d_scratch), int(limit_ns), ctypes.c_void_p(stream),
                                             ctypes.byref(b)))
    return b.value


def dmuon_momentum_norm_noalloc(grad: int, momentum: int, u_out: int, s_out: int, rows: int, cols: int,
                                grad_dtype="bf16", u_dtype="bf16", mu=0.95, nesterov=True, eps=1e-7, stream: int = 0):
    """Momentum + normalisation pass of one matrix with no workspace (see include/dmuon.h)."""
    _check(lib().dmuon_momentum_norm_noalloc(ctypes.c_void_p(grad), ctypes.c_void_p(momentum), ctypes.c_void_p(u_out),
                                             ctypes.c_void_p(s_out), int(rows), int(cols), DTYPE[grad_dtype],
                                             DTYPE[u_dtype], float(mu), int(bool(nesterov)), float(eps),
                                             ctypes.c_void_p(stream)))


def dmuon_assign_owners(shapes, n_ranks, ns_steps=5, costs=None):
    """Owner rank per matrix and the predicted load per rank (host only)."""
    n = len(shapes)
    sh = (Shape * max(n, 1))(*[Shape(int(r), int(c)) for r, c in shapes])
    cs = (ctypes.c_double * n)(*costs) if costs is not None else None
    own = (ctypes.c_int32 * max(n, 1))()
    load = (ctypes.c_double * max(n_ranks, 1))()
    _check(lib().dmuon_assign_owners(sh if n else None, n, ns_steps, cs, n_ranks, own, load))
    return list(own)[:n], list(load)[:n_ranks]


def dmuon_adamw_flat(param: int, grad: int, exp_avg: int, exp_avg_sq: int, n: int, param_dtype="bf16",
                     grad_dtype="bf16", lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1,
                     stream: int = 0):
    """One AdamW step over a flat buffer (see include/dmuon.h)."""
    _check(lib().dmuon_adamw_flat(ctypes.c_void_p(param), ctypes.c_void_p(grad), ctypes.c_void_p(exp_avg),
                                  ctypes.c_void_p(exp_avg_sq), int(n), DTYPE[param_dtype], DTYPE[grad_dtype],
                                  float(lr), float(beta1), float(beta2), float(eps), float(weight_decay), int(step),
                                  ctypes.c_void_p(stream)))


@dataclass
class Muon:
    """Convenience holder: a plan plus its torch-allocated workspace.

    ``params``, ``grads`` and ``momenta`` are lists of CUDA tensors (one per
    matrix, contiguous, 16-byte aligned). Only memory and the stream come
    from torch; the step itself is ``dmuon_step``.
    """

    plan: Plan
    workspace: object  # torch.Tensor (uint8, cuda)

    @classmethod
    def create(cls, shapes, *, ns_steps=5, coeffs=(3.4445, -4.7750, 2.0315), eps=1e-7, param="bf16",
               grad="bf16", compute="bf16", flags=0, device=None, stream=None):
        import torch
        plan = dmuon_plan(shapes, ns_steps, coeffs, eps, param, grad, compute, flags)
        nbytes = plan.workspace_bytes()
        ws = torch.empty(nbytes + 1024, dtype=torch.uint8, device=device or "cuda")
        base = ws.data_ptr()
        aligned = (base + 1023) // 1024 * 1024
        s = stream if stream is not None else torch.cuda.current_stream()
        plan.bind(aligned, nbytes, s.cuda_stream)
        return cls(plan, ws)

    def step(self, params, grads, momenta, *, lr, mu=0.95, nesterov=True, stream=None):
        import torch
        s = stream if stream is not None else torch.cuda.current_stream()
        self.plan.step([t.data_ptr() for t in params] if not isinstance(params[0], int) else params,
                       [t.data_ptr() for t in grads] if not isinstance(grads[0], int) else grads,
                       [t.data_ptr() for t in momenta] if not isinstance(momenta[0], int) else momenta,
                       lr, mu, nesterov, s.cuda_stream)


# --------------------------------------------------------------------------
# losses of the language-model head, and routing to experts
# --------------------------------------------------------------------------

_torch = None


def _t():
    """torch, imported by the first call that takes tensors."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _refuse(msg: str):
    raise DmuonError(ERR_INVALID_ARG, msg)


def _current_device() -> int:
    return _torch._C._cuda_getDevice()


def _here(device) -> int:
    """The raw handle of a device's current stream (the object torch.cuda.current_stream() makes costs more than
    a small call)."""
    return _torch._C._cuda_getCurrentRawStream(device)


def _elsewhere(t, device, name):
    """Refuse a tensor of another device than the object's, which a caller's check has found."""
    if device is None:
        raise DmuonError(ERR_NOT_BOUND, "head is not bound")
    if t.is_cuda and t.get_device() != device:
        _refuse(f"{name} is on cuda:{t.get_device()}, what takes it on cuda:{device}")


def _rows(t, dim, dtype, name, device, rows=None):
    """A matrix on the object's device whose rows lie contiguous (any row pitch); returns that pitch."""
    shape = t.shape
    if not (t.get_device() == device and t.dtype == dtype and len(shape) == 2 and shape[1] == dim and
            (rows is None or shape[0] == rows) and (dim <= 1 or t.stride(1) == 1)):
        _elsewhere(t, device, name)
        _refuse(f"{name} must be a CUDA {dtype} tensor of shape [{'rows' if rows is None else rows}, {dim}] "
                "with contiguous rows")
    return t.stride(0) if shape[0] > 1 else -(-dim // 8) * 8


def _flat(t, shape, dtype, name, device):
    """The address of a contiguous tensor on the object's device."""
    if not (t.get_device() == device and t.dtype == dtype and t.shape == shape and t.is_contiguous()):
        _elsewhere(t, device, name)
        _refuse(f"{name} must be a contiguous CUDA {dtype} tensor of shape {list(shape)}")
    return t.data_ptr()


def _run(owner, call, stream, *tensors, scratch=None):
    """Run ``call(handle)`` on the device of ``owner`` and on ``stream`` (None: the current one): what it allocates
    belongs to that stream. ``scratch``, the owner's workspace, and what a call with a stream of its own is given
    stay alive until the stream is done with them; other tensors on the current stream are the caller's to keep."""
    device, current = owner.device, _current_device()
    if stream is None:
        if current != device:
            _refuse(f"the operator is on cuda:{device}, the current device is cuda:{current}")
        handle = _here(device)
        if scratch is not None and handle != owner.home:
            scratch.record_stream(_t().cuda.current_stream(device))
        return call(handle)
    if stream.device_index != device:
        _refuse(f"the operator is on cuda:{device}, the stream on cuda:{stream.device_index}")
    for t in (*tensors, scratch):
        if t is not None:
            t.record_stream(stream)
    if current == device and stream.cuda_stream == _here(device):
        return call(stream.cuda_stream)
    with _t().cuda.stream(stream):
        return call(stream.cuda_stream)


@dataclass
class Logprobs:
    """What Head.logprobs returns of each token (see include/dmuon.h)."""

    logp: object      # [tokens] fp32: the target's log probability, 0 where there is no target
    entropy: object   # [tokens] fp32
    lse: object       # [tokens] fp32
    top_ids: object   # [tokens, top] int64, likeliest first; None where none were asked for
    top_logp: object  # [tokens, top] fp32; None where none were asked for


class Head:
    """Losses of a language model's head with their gradients, without the logits.

    One object per (max_tokens, vocab, dim, max_top), with its workspace from
    torch; one call uses it at a time. ``hidden`` is [tokens, dim] and
    ``weight`` [vocab, dim], both bf16 with rows that start on 16 bytes;
    losses, log sums and their gradients are fp32 [tokens]. All of them lie on
    the device the head is bound on, which is the current one or the stream's.
    See include/dmuon.h for the formulas.
    """

    def __init__(self, handle, max_tokens, vocab, dim, max_top):
        self._h = handle
        self.max_tokens, self.vocab, self.dim, self.max_top = max_tokens, vocab, dim, max_top
        self.workspace = None
        self.device = None  # index of the device it is bound on
        self.home = 0       # raw handle of the stream the workspace was allocated on

    @classmethod
    def create(cls, max_tokens, vocab, dim, *, max_top=0, alternatives=True, device=None, stream=None):
        """``alternatives=False``: no room beside what the losses need, up to half the workspace; ``logprobs`` with
        ``top`` then takes smaller pieces of the vocabulary, one after another."""
        h = ctypes.c_void_p()
        _check(lib().dmuon_head_create(int(max_tokens), int(vocab), int(dim), int(max_top), ctypes.byref(h)))
        self = cls(h, int(max_tokens), int(vocab), int(dim), int(max_top))
        nbytes = self.workspace_bytes(alternatives)
        ws = _t().empty(nbytes + 1024, dtype=_t().uint8, device=device or "cuda")
        here = _here(ws.get_device())
        s = here if stream is None else stream.cuda_stream
        if s != here:
            ws.record_stream(stream)
        self.bind((ws.data_ptr() + 1023) // 1024 * 1024, nbytes, s)
        self.workspace, self.home = ws, here
        return self

    def workspace_bytes(self, alternatives=False) -> int:
        """What ``bind`` needs at least, or with room for the logits that alternatives are chosen from."""
        n = ctypes.c_size_t()
        size = lib().dmuon_head_scores_workspace_bytes if alternatives else lib().dmuon_head_workspace_bytes
        _check(size(self._h, ctypes.byref(n)))
        return n.value

    def bind(self, d_workspace: int, nbytes: int, stream: int = 0):
        _check(lib().dmuon_head_bind(self._h, ctypes.c_void_p(d_workspace), nbytes, ctypes.c_void_p(stream)))
        _t()
        self.device = _current_device()

    def _inputs(self, hidden, weight):
        bf16 = _t().bfloat16
        lh = _rows(hidden, self.dim, bf16, "hidden", self.device)
        lw = _rows(weight, self.dim, bf16, "weight", self.device, self.vocab)
        return hidden.data_ptr(), lh, weight.data_ptr(), lw

    def _teacher(self, top_ids, top_logits, tokens):
        top = top_ids.shape[-1]
        ids = _flat(top_ids, (tokens, top), _t().int64, "top_ids", self.device)
        return ids, _flat(top_logits, (tokens, top), _t().float32, "top_logits", self.device), top

    def _forward(self, fn, hidden, args, stream, *tensors):
        n = hidden.shape[0]

        def call(s):
            empty, f32 = _t().empty, _t().float32
            loss = empty(n, dtype=f32, device=hidden.device)
            lse = empty(n, dtype=f32, device=hidden.device)
            _check(fn(self._h, *args, n, loss.data_ptr(), lse.data_ptr(), s))
            return loss, lse

        return _run(self, call, stream, hidden, *tensors, scratch=self.workspace)

    def _backward(self, fn, hidden, weight, args, lse, grad_loss, dhidden, dweight, stream, *tensors, loss=None):
        n = hidden.shape[0]
        f32, dev = _t().float32, self.device
        args += (n, _flat(lse, (n,), f32, "lse", dev))
        if loss is not None:
            args += (_flat(loss, (n,), f32, "loss", dev),)
            tensors += (loss,)
        args += (_flat(grad_loss, (n,), f32, "grad_loss", dev),)

        def call(s):
            dh, ph, lh = self._grad(hidden, dhidden, "dhidden")
            dw, pw, lw = self._grad(weight, dweight, "dweight")
            _check(fn(self._h, *args, ph, lh, pw, lw, s))
            return dh, dw

        given = self._given(hidden, weight, dhidden, dweight)
        return _run(self, call, stream, hidden, weight, lse, grad_loss, *tensors, *given, scratch=self.workspace)

    def _given(self, hidden, weight, dhidden, dweight):
        """The gradients that the caller wants written into tensors of its own, checked."""
        given = []
        for like, want, name in ((hidden, dhidden, "dhidden"), (weight, dweight, "dweight")):
            if want is not None and not isinstance(want, bool):
                _rows(want, self.dim, _t().bfloat16, name, self.device, like.shape[0])
                given.append(want)
        return given

    def _grad(self, like, want, name):
        """The gradient of ``like`` (made where True, left out where False or None), its address and pitch."""
        if want is False or want is None:
            return None, None, 0
        rows, dim = like.shape[0], self.dim
        if want is True:
            if dim % 8 == 0:
                want = _t().empty(rows, dim, dtype=like.dtype, device=like.device)
                return want, want.data_ptr(), dim
            want = _t().empty(rows, -(-dim // 8) * 8, dtype=like.dtype, device=like.device)[:, :dim]
        return want, want.data_ptr(), _rows(want, dim, _t().bfloat16, name, self.device, rows)

    def xent(self, hidden, weight, targets, *, stream=None):
        """(loss, lse) per token; targets int64, one outside the vocabulary does not count."""
        y = _flat(targets, hidden.shape[:1], _t().int64, "targets", self.device)
        return self._forward(lib().dmuon_head_xent, hidden, (*self._inputs(hidden, weight), y), stream, weight, targets)

    def xent_backward(self, hidden, weight, targets, lse, grad_loss, *, loss=None, dhidden=True, dweight=True,
                      stream=None):
        """(dhidden, dweight) of sum(grad_loss * loss). Either may be a tensor to write into, or False. With ``loss``
        as xent returned it, the gradients of tokens predicted with near certainty are exact too."""
        y = _flat(targets, hidden.shape[:1], _t().int64, "targets", self.device)
        fn = lib().dmuon_head_xent_backward if loss is None else lib().dmuon_head_xent_backward_loss
        return self._backward(fn, hidden, weight, (*self._inputs(hidden, weight), y), lse, grad_loss, dhidden, dweight,
                              stream, targets, loss=loss)

    def distill(self, hidden, weight, top_ids, top_logits, temperature=1.0, *, stream=None):
        """(loss, lse) per token against a teacher's top logits; ids int64 and logits fp32, both [tokens, top]."""
        lists = self._teacher(top_ids, top_logits, hidden.shape[0])
        return self._forward(lib().dmuon_head_distill, hidden,
                             (*self._inputs(hidden, weight), *lists, float(temperature)), stream, weight, top_ids,
                             top_logits)

    def distill_backward(self, hidden, weight, top_ids, top_logits, temperature, lse, grad_loss, *, dhidden=True,
                         dweight=True, stream=None):
        """(dhidden, dweight) of sum(grad_loss * loss), as xent_backward."""
        lists = self._teacher(top_ids, top_logits, hidden.shape[0])
        return self._backward(lib().dmuon_head_distill_backward, hidden, weight,
                              (*self._inputs(hidden, weight), *lists, float(temperature)), lse, grad_loss, dhidden,
                              dweight, stream, top_ids, top_logits)

    def logprobs(self, hidden, weight, targets=None, *, top=0, temperature=1.0, stream=None) -> Logprobs:
        """Log probability of each token's target (int64; one outside the vocabulary, or None: no target), entropy of
        the distribution, and the ``top`` (up to 32) likeliest entries with their log probabilities."""
        n, dev, top = hidden.shape[0], self.device, int(top)
        y = None if targets is None else _flat(targets, hidden.shape[:1], _t().int64, "targets", dev)
        args = (*self._inputs(hidden, weight), y, float(temperature), top, n)

        def call(s):
            empty, f32, place = _t().empty, _t().float32, hidden.device
            out = [empty(n, dtype=f32, device=place) for _ in range(3)]
            ids = values = None
            if top > 0:
                ids, values = empty((n, top), dtype=_t().int64, device=place), empty((n, top), dtype=f32, device=place)
            _check(lib().dmuon_head_logprobs(self._h, *args, *[t.data_ptr() for t in out],
                                             None if ids is None else ids.data_ptr(),
                                             None if values is None else values.data_ptr(), s))
            return Logprobs(*out, ids, values)

        return _run(self, call, stream, hidden, weight, targets, scratch=self.workspace)

    def logprobs_backward(self, hidden, weight, targets, scores, grad_logp=None, grad_entropy=None, *, temperature=1.0,
                          dhidden=True, dweight=True, stream=None):
        """(dhidden, dweight) of sum(grad_logp * logp + grad_entropy * entropy); ``scores`` as logprobs returned them
        for the same inputs; a gradient that is None is zeros. Either result may be a tensor to write into, or False."""
        f32, dev, shape = _t().float32, self.device, hidden.shape[:1]
        y = None if targets is None else _flat(targets, shape, _t().int64, "targets", dev)
        logp, entropy = _flat(scores.logp, shape, f32, "logp", dev), _flat(scores.entropy, shape, f32, "entropy", dev)
        lse = _flat(scores.lse, shape, f32, "lse", dev)
        gl = None if grad_logp is None else _flat(grad_logp, shape, f32, "grad_logp", dev)
        ge = None if grad_entropy is None else _flat(grad_entropy, shape, f32, "grad_entropy", dev)
        args = (*self._inputs(hidden, weight), y, float(temperature), shape[0], logp, entropy, lse, gl, ge)
        given = self._given(hidden, weight, dhidden, dweight)

        def call(s):
            dh, ph, lh = self._grad(hidden, dhidden, "dhidden")
            dw, pw, lw = self._grad(weight, dweight, "dweight")
            _check(lib().dmuon_head_logprobs_backward(self._h, *args, ph, lh, pw, lw, s))
            return dh, dw

        return _run(self, call, stream, hidden, weight, targets, scores.logp, scores.entropy, scores.lse, grad_logp,
                    grad_entropy, *given, scratch=self.workspace)

    def read_device_status(self, stream: int = 0) -> int:
        b = ctypes.c_uint32()
        _check(lib().dmuon_head_read_device_status(self._h, ctypes.c_void_p(stream), ctypes.byref(b)))
        return b.value

    def destroy(self):
        if self._h is not None and self._h.value:
            lib().dmuon_head_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


@dataclass
class Route:
    """Rows of the assignments in expert order (see include/dmuon.h)."""

    dest: object     # [tokens, top] int32: the assignment's row, -1 when dropped
    source: object   # [tokens * top] int32: the row's assignment, -1 for rows not in use
    offsets: object  # [experts + 1] int32: the experts' first rows


class Router:
    """Tokens to experts and back, for up to ``max_tokens`` tokens with ``top`` experts each.

    Holds the sort's scratch (torch-allocated; one sort uses it at a time).
    Rows are bf16 or fp32, weights fp32 [tokens, top]. All of them lie on the
    scratch's device, which is the current one or the stream's.
    """

    def __init__(self, max_tokens, top, experts, workspace):
        self.max_tokens, self.top, self.experts, self.workspace = max_tokens, top, experts, workspace
        _t()
        self.device = workspace.get_device()
        self.home = _here(self.device)  # raw handle of the stream the workspace was allocated on

    @classmethod
    def create(cls, max_tokens, top, experts, *, device=None):
        n = ctypes.c_size_t()
        _check(lib().dmuon_route_workspace_bytes(int(max_tokens), int(top), int(experts), ctypes.byref(n)))
        return cls(int(max_tokens), int(top), int(experts),
                   _t().empty(n.value, dtype=_t().uint8, device=device or "cuda"))

    def sort(self, expert_ids, *, stream=None) -> Route:
        """Order the assignments by expert; expert_ids int64 [tokens, top], one outside 0..experts-1 is dropped."""
        t, top = expert_ids.shape[0], self.top
        if t > self.max_tokens:
            _refuse(f"expert_ids has {t} tokens, more than max_tokens ({self.max_tokens})")
        ids = _flat(expert_ids, (t, top), _t().int64, "expert_ids", self.device)

        def call(s):
            empty, i32, dev = _t().empty, _t().int32, expert_ids.device
            dest = empty((t, top), dtype=i32, device=dev)
            source = empty(t * top, dtype=i32, device=dev)
            offsets = empty(self.experts + 1, dtype=i32, device=dev)
            ws = self.workspace
            _check(lib().dmuon_route_sort(ids, t, top, self.experts, dest.data_ptr(), source.data_ptr(),
                                          offsets.data_ptr(), ws.data_ptr(), ws.numel(), s))
            return Route(dest, source, offsets)

        return _run(self, call, stream, expert_ids, scratch=self.workspace)

    def _kind(self, t, name):
        if t.dim() == 2:
            if t.dtype == _t().bfloat16:
                return BF16
            if t.dtype == _t().float32:
                return F32
        _refuse(f"{name} must be a bf16 or fp32 matrix")

    def _route(self, route, tokens):
        i32 = _t().int32
        return (_flat(route.dest, (tokens, self.top), i32, "route.dest", self.device),
                _flat(route.source, (tokens * self.top,), i32, "route.source", self.device))

    def dispatch(self, x, route, *, stream=None):
        """xs [tokens * top, dim]: x's rows in expert order, zeros in rows not in use."""
        kind = self._kind(x, "x")
        t, dim = x.shape
        ld = _rows(x, dim, x.dtype, "x", self.device)
        dest, source = self._route(route, t)

        def call(s):
            xs = _t().empty((t * self.top, dim), dtype=x.dtype, device=x.device)
            _check(lib().dmuon_route_dispatch(x.data_ptr(), ld, dest, source, t, self.top, dim, kind, xs.data_ptr(), s))
            return xs

        return _run(self, call, stream, x, route.dest, route.source)

    def combine(self, ys, weights, route, *, stream=None):
        """y [tokens, dim]: the sum of each token's expert rows, times weights (fp32 [tokens, top], or None: 1)."""
        kind = self._kind(ys, "ys")
        t, dim = route.dest.shape[0], ys.shape[1]
        dest, _ = self._route(route, t)
        rows = _flat(ys, (t * self.top, dim), ys.dtype, "ys", self.device)
        w = None if weights is None else _flat(weights, (t, self.top), _t().float32, "weights", self.device)

        def call(s):
            y = _t().empty((t, dim), dtype=ys.dtype, device=ys.device)
            _check(lib().dmuon_route_combine(rows, w, dest, t, self.top, dim, kind, y.data_ptr(), dim, s))
            return y

        return _run(self, call, stream, ys, weights, route.dest)

    def combine_backward(self, dy, ys, weights, route, *, stream=None):
        """(dys, dweights) of combine."""
        kind = self._kind(ys, "ys")
        t, dim = route.dest.shape[0], ys.shape[1]
        dest, source = self._route(route, t)
        rows = _flat(ys, (t * self.top, dim), ys.dtype, "ys", self.device)
        w = _flat(weights, (t, self.top), _t().float32, "weights", self.device)
        ld = _rows(dy, dim, ys.dtype, "dy", self.device, t)

        def call(s):
            dys = _t().empty_like(ys)
            dw = _t().empty_like(weights)
            _check(lib().dmuon_route_combine_backward(dy.data_ptr(), ld, rows, w, dest, source, t, self.top, dim, kind,
                                                      dys.data_ptr(), dw.data_ptr(), s))
            return dys, dw

        return _run(self, call, stream, dy, ys, weights, route.dest, route.source)

    def dispatch_backward(self, dxs, route, *, stream=None):
        """dx [tokens, dim]: the gradient of dispatch, the sum of each token's rows of dxs."""
        return self.combine(dxs, None, route, stream=stream)


class Experts:
    """A mixture's experts for a few tokens, from the router's ids and weights to the layer's output.

    For up to ``max_tokens`` tokens with ``top`` experts each (together at most
    2048 assignments), beside ``Router``, which serves many tokens and training.
    Holds the scratch of a call (torch-allocated; one call uses it at a time).
    All tensors lie on the scratch's device, which is the current one or the
    stream's. See include/dmuon.h for the formulas.
    """

    def __init__(self, max_tokens, top, experts, dim, inner, workspace):
        self.max_tokens, self.top, self.experts, self.dim, self.inner = max_tokens, top, experts, dim, inner
        self.workspace = workspace
        _t()
        self.device = workspace.get_device()
        self.home = _here(self.device)  # raw handle of the stream the workspace was allocated on

    @classmethod
    def create(cls, max_tokens, top, experts, dim, inner, *, device=None):
        sizes = int(max_tokens), int(top), int(experts), int(dim), int(inner)
        n = ctypes.c_size_t()
        _check(lib().dmuon_experts_workspace_bytes(*sizes, ctypes.byref(n)))
        return cls(*sizes, _t().empty(n.value, dtype=_t().uint8, device=device or "cuda"))

    def forward(self, x, expert_ids, weights, up, down, *, gate=None, stream=None):
        """y [tokens, dim] of x [tokens, dim]; expert_ids int64 and weights fp32 [tokens, top], an id outside
        0..experts-1 adds nothing; up and gate bf16 [experts, inner, dim], down [experts, dim, inner]."""
        bf16, dev, dim = _t().bfloat16, self.device, self.dim
        t = x.shape[0]
        if t > self.max_tokens:
            _refuse(f"x has {t} tokens, more than max_tokens ({self.max_tokens})")
        ld = _rows(x, dim, bf16, "x", dev)
        ids = _flat(expert_ids, (t, self.top), _t().int64, "expert_ids", dev)
        w = _flat(weights, (t, self.top), _t().float32, "weights", dev)
        wide = (self.experts, self.inner, dim)
        pu = _flat(up, wide, bf16, "up", dev)
        pg = None if gate is None else _flat(gate, wide, bf16, "gate", dev)
        pd = _flat(down, (self.experts, dim, self.inner), bf16, "down", dev)

        def call(s):
            y = _t().empty((t, dim), dtype=bf16, device=x.device)
            ws = self.workspace
            _check(lib().dmuon_experts_forward(x.data_ptr(), ld, ids, w, t, self.top, self.experts, dim, self.inner, pu,
                                               pg, pd, y.data_ptr(), dim, ws.data_ptr(), ws.numel(), s))
            return y

        return _run(self, call, stream, x, expert_ids, weights, up, down, gate, scratch=self.workspace)

    def read_device_status(self, stream: int = 0) -> int:
        """The status of the last call that had tokens."""
        b = ctypes.c_uint32()
        _check(lib().dmuon_experts_read_device_status(self.workspace.data_ptr(), ctypes.c_void_p(stream), ctypes.byref(b)))
        return b.value


_KINDS = {}


def _kinds():
    """The library's type of a torch type."""
    if not _KINDS:
        _KINDS.update({_t().bfloat16: BF16, _t().float32: F32})
    return _KINDS


def _at(a):
    """The address of an array's elements."""
    return a.buffer_info()[0]


class GradClip:
    """The global norm of many gradient tensors, and their clipping.

    Holds the sums' scratch (torch-allocated; one call uses it at a time).
    Gradients are contiguous bf16 or fp32 tensors on the scratch's device, which
    is the current one or the stream's. See include/dmuon.h.
    """

    def __init__(self, workspace):
        self.workspace = workspace
        _t()
        self.device = workspace.get_device()
        self.home = _here(self.device)  # raw handle of the stream the workspace was allocated on

    @classmethod
    def create(cls, *, device=None):
        n = ctypes.c_size_t()
        _check(lib().dmuon_clip_workspace_bytes(ctypes.byref(n)))
        return cls(_t().empty(n.value, dtype=_t().uint8, device=device or "cuda"))

    def _table(self, tensors, name):
        """Arrays of the tensors' addresses, element counts and types."""
        kinds, device = _kinds(), self.device
        types = []
        for t in tensors:
            kind = kinds.get(t.dtype)
            if kind is None:
                _refuse(f"{name} must be bf16 or fp32 tensors")
            if t.get_device() != device or not t.is_contiguous():
                _elsewhere(t, device, name)
                _refuse(f"{name} must be contiguous CUDA tensors")
            types.append(kind)
        return (array("Q", [t.data_ptr() for t in tensors]), array("q", [t.numel() for t in tensors]), array("i", types))

    def norm(self, grads, *, stream=None):
        """The 2-norm over all elements of all tensors: an fp32 tensor without dimensions."""
        grads = list(grads)
        ptrs, counts, types = self._table(grads, "grads")

        def call(s):
            norm = _t().empty((), dtype=_t().float32, device=self.workspace.device)
            ws = self.workspace
            _check(lib().dmuon_grad_norm(_at(ptrs), _at(counts), _at(types), len(grads), norm.data_ptr(), ws.data_ptr(),
                                         ws.numel(), s))
            return norm

        return _run(self, call, stream, *grads, scratch=self.workspace)

    def clip(self, grads, max_norm, *, out=None, stream=None):
        """Scale the gradients by min(1, max_norm / norm), in place or into the tensors ``out``; returns the norm
        before that, as ``norm`` does. A norm that is not finite clips nothing."""
        grads = list(grads)
        ptrs, counts, types = self._table(grads, "grads")
        to, results = ptrs, []
        if out is not None:
            results = list(out)
            to, counts_to, types_to = self._table(results, "out")
            if counts_to != counts or types_to != types or any(a.shape != b.shape for a, b in zip(results, grads)):
                _refuse("out must have the gradients' shapes and types")

        def call(s):
            norm = _t().empty((), dtype=_t().float32, device=self.workspace.device)
            ws = self.workspace
            _check(lib().dmuon_grad_clip(_at(ptrs), _at(to), _at(counts), _at(types), len(grads), float(max_norm),
                                         norm.data_ptr(), ws.data_ptr(), ws.numel(), s))
            return norm

        return _run(self, call, stream, *grads, *results, scratch=self.workspace)
