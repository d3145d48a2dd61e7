"""Python binding of libvsa.so (argument marshalling only).

Every step of the forward pass runs in the library's CUDA kernels; PyTorch
only provides device memory and the current stream. There is no CPU path:
calls raise if the library is not built or the tensors are not on an
sm_100 CUDA device.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(HERE, "libvsa.so")

STATUS = {0: "VSA_OK", 1: "VSA_ERR_INVALID_ARG", 2: "VSA_ERR_SHAPE", 3: "VSA_ERR_UNSUPPORTED",
          4: "VSA_ERR_ALIGN", 5: "VSA_ERR_CUDA", 6: "VSA_ERR_TIMEOUT", 7: "VSA_ERR_DEVICE"}

EXPORTED = ["vsa_workspace_bytes", "vsa_workspace_layout", "vsa_plan", "vsa_run", "vsa_run_fixed_idx",
            "vsa_forward", "vsa_check", "vsa_plan_destroy", "vsa_status_string", "vsa_set_wait_limit_ns",
            "vsa_set_debug_stall", "vsa_set_stage_timing", "vsa_stage_times", "vsa_kernels_per_run",
            "vsa_forward_noalloc", "vsa_set_cube_major_copies", "vsa_run_host", "vsa_measure_l2_read",
            "vsa_run_train", "vsa_backward_workspace_bytes", "vsa_run_backward", "vsa_backward_stage_times",
            "vsa_stage_times_history", "vsa_backward_stage_times_history",
            "vsa_rope", "vsa_rope_backward", "vsa_qk_norm_rope", "vsa_qk_norm_rope_backward_workspace_bytes",
            "vsa_qk_norm_rope_backward", "vsa_linear_workspace_bytes", "vsa_linear",
            "vsa_linear_backward_workspace_bytes", "vsa_linear_backward", "vsa_linear_check", "vsa_linear_set_limits"]

TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
ROPE_MAX_PAIRS, ROPE_MAX_AXES = 128, 4
ACTIVATIONS = {None: 0, "silu": 1, "gelu": 2, "gelu_tanh": 3}


class VSAError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        super().__init__(f"{what}: {STATUS.get(code, code)}" if what else STATUS.get(code, str(code)))


class Config(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("heads", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("W", ctypes.c_int), ("D", ctypes.c_int), ("topk", ctypes.c_int), ("top_p", ctypes.c_float),
                ("kmin", ctypes.c_int), ("kmax", ctypes.c_int)]


class WorkspaceLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("q_cube", "k_cube", "v_cube", "q_pool", "k_pool", "v_pool",
                                               "o_coarse", "s_coarse", "pool_split", "p_split", "cnt", "order",
                                               "err", "total")]


class Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("heads", ctypes.c_int), ("s_b", ctypes.c_longlong),
                ("s_h", ctypes.c_longlong), ("s_n", ctypes.c_longlong)]


class RotationSpec(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_int), ("interleaved", ctypes.c_int), ("axes", ctypes.c_int),
                ("axis", ctypes.c_int * ROPE_MAX_PAIRS), ("freq", ctypes.c_double * ROPE_MAX_PAIRS)]


class Positions(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("H", ctypes.c_int), ("W", ctypes.c_int), ("origin", ctypes.c_int * 3),
                ("list", ctypes.c_void_p), ("list_type", ctypes.c_int), ("list_batch", ctypes.c_longlong)]


class RopeSizes(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int), ("B", ctypes.c_int), ("N", ctypes.c_int), ("D", ctypes.c_int)]


class LinearSizes(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int), ("B", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int),
                ("F", ctypes.c_int)]


# The same structs as bytes: packing one costs a tenth of filling a ctypes structure.
_pack_heads = struct.Struct("@Piqqq").pack
_pack_positions = struct.Struct("@6iPiq").pack
_pack_rope_sizes = struct.Struct("@4i").pack
_pack_linear_sizes = struct.Struct("@5i").pack

_lib = None
_projection = None


def load():
    """Loads libvsa.so and declares its signatures (no GPU needed)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(lib_path):
        raise RuntimeError(f"{lib_path} is not built; run: python -m trainable_block_sparse_cube_b200.build")
    L = ctypes.CDLL(lib_path)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L.vsa_workspace_bytes.argtypes = [ctypes.POINTER(Config)]
    L.vsa_workspace_bytes.restype = sz
    L.vsa_workspace_layout.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(WorkspaceLayout)]
    L.vsa_workspace_layout.restype = i32
    L.vsa_plan.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(Config), vp, sz]
    L.vsa_plan.restype = i32
    L.vsa_run.argtypes = [vp] * 10
    L.vsa_run.restype = i32
    L.vsa_run_fixed_idx.argtypes = [vp] * 12
    L.vsa_run_host.argtypes = [vp] * 10
    L.vsa_run_host.restype = i32
    L.vsa_run_fixed_idx.restype = i32
    L.vsa_forward.argtypes = [vp] * 5 + [i32] * 7 + [ctypes.c_float, vp, vp, vp]
    L.vsa_forward.restype = i32
    L.vsa_check.argtypes = [vp]
    L.vsa_check.restype = i32
    L.vsa_plan_destroy.argtypes = [vp]
    L.vsa_plan_destroy.restype = None
    L.vsa_status_string.argtypes = [i32]
    L.vsa_status_string.restype = ctypes.c_char_p
    L.vsa_set_wait_limit_ns.argtypes = [vp, ctypes.c_uint64]
    L.vsa_set_wait_limit_ns.restype = i32
    L.vsa_set_debug_stall.argtypes = [vp, i32]
    L.vsa_set_debug_stall.restype = i32
    L.vsa_set_cube_major_copies.argtypes = [vp, i32]
    L.vsa_set_cube_major_copies.restype = i32
    L.vsa_set_stage_timing.argtypes = [vp, i32]
    L.vsa_set_stage_timing.restype = i32
    L.vsa_stage_times.argtypes = [vp, ctypes.POINTER(ctypes.c_float)]
    L.vsa_stage_times.restype = i32
    L.vsa_stage_times_history.argtypes = [vp, ctypes.POINTER(ctypes.c_float), i32, ctypes.POINTER(ctypes.c_int)]
    L.vsa_stage_times_history.restype = i32
    L.vsa_kernels_per_run.argtypes = []
    L.vsa_kernels_per_run.restype = i32
    L.vsa_forward_noalloc.argtypes = [vp] * 5 + [i32] * 7 + [ctypes.c_float, vp, vp, vp]
    L.vsa_forward_noalloc.restype = i32
    L.vsa_run_train.argtypes = [vp] * 12
    L.vsa_run_train.restype = i32
    L.vsa_backward_workspace_bytes.argtypes = [ctypes.POINTER(Config)]
    L.vsa_backward_workspace_bytes.restype = sz
    L.vsa_run_backward.argtypes = [vp, vp, sz] + [vp] * 16
    L.vsa_run_backward.restype = i32
    L.vsa_backward_stage_times.argtypes = [vp, ctypes.POINTER(ctypes.c_float)]
    L.vsa_backward_stage_times.restype = i32
    L.vsa_backward_stage_times_history.argtypes = [vp, ctypes.POINTER(ctypes.c_float), i32, ctypes.POINTER(ctypes.c_int)]
    L.vsa_backward_stage_times_history.restype = i32
    L.vsa_measure_l2_read.argtypes = [vp, sz, i32, vp, vp]
    L.vsa_measure_l2_read.restype = i32
    H, F = ctypes.POINTER(Heads), ctypes.POINTER
    what = [F(RopeSizes), F(RotationSpec), F(Positions)]
    L.vsa_rope.argtypes = what + [H] * 4 + [vp]
    L.vsa_rope.restype = i32
    L.vsa_rope_backward.argtypes = what + [H] * 4 + [vp]
    L.vsa_rope_backward.restype = i32
    L.vsa_qk_norm_rope.argtypes = what + [H, H, vp, vp, ctypes.c_float, H, H, vp]
    L.vsa_qk_norm_rope.restype = i32
    L.vsa_qk_norm_rope_backward_workspace_bytes.argtypes = [i32]
    L.vsa_qk_norm_rope_backward_workspace_bytes.restype = sz
    L.vsa_qk_norm_rope_backward.argtypes = what + [H, H, vp, vp, ctypes.c_float, H, H, H, H, vp, vp, vp, sz, vp]
    L.vsa_qk_norm_rope_backward.restype = i32
    L.vsa_linear_workspace_bytes.argtypes = [F(LinearSizes)]
    L.vsa_linear_workspace_bytes.restype = sz
    L.vsa_linear.argtypes = [F(LinearSizes), H, vp, ctypes.c_longlong, vp, i32, H, H, H, vp, sz, vp]
    L.vsa_linear.restype = i32
    L.vsa_linear_backward_workspace_bytes.argtypes = [F(LinearSizes), i32]
    L.vsa_linear_backward_workspace_bytes.restype = sz
    L.vsa_linear_backward.argtypes = [F(LinearSizes), H, vp, ctypes.c_longlong, H, i32, H, H, vp, vp, vp, sz, vp]
    L.vsa_linear_backward.restype = i32
    L.vsa_linear_check.argtypes = [vp]
    L.vsa_linear_check.restype = i32
    L.vsa_linear_set_limits.argtypes = [ctypes.c_uint64, i32]
    L.vsa_linear_set_limits.restype = i32
    _lib = L
    return L


def _load_projection():
    """The projection side's functions with untyped pointers, to be called with packed structs."""
    global _projection
    if _projection is None:
        load()
        L = ctypes.CDLL(lib_path)
        vp, i32, sz, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_longlong
        for name, args in (("vsa_rope", [vp] * 8), ("vsa_rope_backward", [vp] * 8),
                           ("vsa_qk_norm_rope", [vp] * 7 + [ctypes.c_float] + [vp] * 3),
                           ("vsa_qk_norm_rope_backward", [vp] * 7 + [ctypes.c_float] + [vp] * 7 + [sz, vp]),
                           ("vsa_linear", [vp] * 3 + [i64, vp, i32] + [vp] * 4 + [sz, vp]),
                           ("vsa_linear_backward", [vp] * 3 + [i64, vp, i32] + [vp] * 5 + [sz, vp])):
            getattr(L, name).argtypes = args
        L.vsa_qk_norm_rope_backward_workspace_bytes.argtypes = [i32]
        L.vsa_linear_workspace_bytes.argtypes = [vp]
        L.vsa_linear_backward_workspace_bytes.argtypes = [vp, i32]
        for name in ("vsa_qk_norm_rope_backward_workspace_bytes", "vsa_linear_workspace_bytes",
                     "vsa_linear_backward_workspace_bytes"):
            getattr(L, name).restype = sz
        _projection = L
    return _projection


def _check(code: int, what: str):
    if code != 0:
        raise VSAError(code, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _address(t):
    return None if t is None else t.data_ptr()


def _stream():
    # what torch.cuda.current_stream().cuda_stream gives, without building the Stream object (3 us)
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _need(t, name, dtype, shape):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def make_config(B, heads, T, H, W, D, topk=0, top_p=0.0, kmin=0, kmax=0) -> Config:
    return Config(B, heads, T, H, W, D, topk, top_p, kmin, kmax)


def workspace_bytes(cfg: Config) -> int:
    return int(load().vsa_workspace_bytes(ctypes.byref(cfg)))


def workspace_layout(cfg: Config) -> WorkspaceLayout:
    lay = WorkspaceLayout()
    _check(load().vsa_workspace_layout(ctypes.byref(cfg), ctypes.byref(lay)), "vsa_workspace_layout")
    return lay


class Plan:
    """A plan with its device workspace (a torch uint8 tensor it owns)."""

    def __init__(self, B, heads, T, H, W, D, topk=0, top_p=0.0, kmin=0, kmax=0, device=None):
        L = load()
        self.cfg = make_config(B, heads, T, H, W, D, topk, top_p, kmin, kmax)
        self.B, self.heads, self.T, self.H, self.W, self.D = B, heads, T, H, W, D
        self.N = T * H * W
        self.C = self.N // 64
        self.kcap = topk if topk > 0 else kmax
        nbytes = L.vsa_workspace_bytes(ctypes.byref(self.cfg))
        if nbytes == 0:
            raise VSAError(L.vsa_workspace_layout(ctypes.byref(self.cfg), ctypes.byref(WorkspaceLayout())) or 1,
                           "invalid configuration")
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.layout = workspace_layout(self.cfg)
        h = ctypes.c_void_p()
        _check(L.vsa_plan(ctypes.byref(h), ctypes.byref(self.cfg), _ptr(self.workspace), nbytes), "vsa_plan")
        self._h = h

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and _lib is not None:
            _lib.vsa_plan_destroy(h)
            self._h = None

    # ------------------------------------------------------------ helpers
    def _inputs(self, q, k, v, gate_c, gate_f):
        BHND = (self.B, self.heads, self.N, self.D)
        for t, n in ((q, "q"), (k, "k"), (v, "v")):
            _need(t, n, torch.bfloat16, BHND)
        for t, n in ((gate_c, "gate_c"), (gate_f, "gate_f")):
            _need(t, n, torch.float32, BHND[:3])

    def run(self, q, k, v, gate_c, gate_f, out=None, idx=None, cnt=None):
        """Whole forward pass. Returns (out, idx, cnt); enqueued on the current stream."""
        self._inputs(q, k, v, gate_c, gate_f)
        dev = q.device
        out = torch.empty_like(q) if out is None else out
        idx = torch.empty((self.B, self.heads, self.C, self.kcap), dtype=torch.int32, device=dev) if idx is None else idx
        cnt = torch.empty((self.B, self.heads, self.C), dtype=torch.int32, device=dev) if cnt is None else cnt
        _check(load().vsa_run(self._h, _ptr(q), _ptr(k), _ptr(v), _ptr(gate_c), _ptr(gate_f), _ptr(out), _ptr(idx),
                              _ptr(cnt), _stream()), "vsa_run")
        return out, idx, cnt

    def run_train(self, q, k, v, gate_c, gate_f):
        """Forward pass that also saves the backward pass's inputs. Returns
        (out, idx, cnt, o_fine, lse); enqueued on the current stream."""
        self._inputs(q, k, v, gate_c, gate_f)
        dev = q.device
        out = torch.empty_like(q)
        o_fine = torch.empty(q.shape, dtype=torch.float32, device=dev)
        lse = torch.empty((self.B, self.heads, self.N), dtype=torch.float32, device=dev)
        idx = torch.empty((self.B, self.heads, self.C, self.kcap), dtype=torch.int32, device=dev)
        cnt = torch.empty((self.B, self.heads, self.C), dtype=torch.int32, device=dev)
        _check(load().vsa_run_train(self._h, _ptr(q), _ptr(k), _ptr(v), _ptr(gate_c), _ptr(gate_f), _ptr(out),
                                    _ptr(idx), _ptr(cnt), _ptr(o_fine), _ptr(lse), _stream()), "vsa_run_train")
        return out, idx, cnt, o_fine, lse

    def run_backward(self, q, k, v, gate_c, gate_f, idx, cnt, o_fine, lse, dout):
        """Gradients of the gated output with the selection held fixed.
        Returns (dq, dk, dv, dgate_c, dgate_f); enqueued on the current stream.
        The backward workspace is allocated (once) by this plan."""
        self._inputs(q, k, v, gate_c, gate_f)
        BHND = (self.B, self.heads, self.N, self.D)
        _need(idx, "idx", torch.int32, (self.B, self.heads, self.C, self.kcap))
        if cnt is not None:
            _need(cnt, "cnt", torch.int32, (self.B, self.heads, self.C))
        _need(o_fine, "o_fine", torch.float32, BHND)
        _need(lse, "lse", torch.float32, BHND[:3])
        _need(dout, "dout", torch.bfloat16, BHND)
        L = load()
        if getattr(self, "bwd_workspace", None) is None:
            nb = L.vsa_backward_workspace_bytes(ctypes.byref(self.cfg))
            self.bwd_workspace = torch.empty(nb, dtype=torch.uint8, device=q.device)
        dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
        dgc, dgf = torch.empty_like(gate_c), torch.empty_like(gate_f)
        _check(L.vsa_run_backward(self._h, _ptr(self.bwd_workspace), self.bwd_workspace.numel(), _ptr(q), _ptr(k),
                                  _ptr(v), _ptr(gate_c), _ptr(gate_f), _ptr(idx), _ptr(cnt), _ptr(o_fine), _ptr(lse),
                                  _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dgc), _ptr(dgf), _stream()),
               "vsa_run_backward")
        return dq, dk, dv, dgc, dgf

    def backward_stage_times_history(self, max_runs):
        """[(gather + coarse, prep + lists + coarse backward, dq, dk/dv) ms] of the last timed backward calls."""
        ms = (ctypes.c_float * (4 * max_runs))()
        n = ctypes.c_int(0)
        _check(load().vsa_backward_stage_times_history(self._h, ms, int(max_runs), ctypes.byref(n)),
               "vsa_backward_stage_times_history")
        return [tuple(float(x) for x in ms[4 * i: 4 * i + 4]) for i in range(n.value)]

    def backward_stage_times(self):
        """Device ms of (gather + coarse, prep + lists + coarse backward, dq, dk/dv) of the last timed backward."""
        ms = (ctypes.c_float * 4)()
        _check(load().vsa_backward_stage_times(self._h, ms), "vsa_backward_stage_times")
        return tuple(float(x) for x in ms)

    def run_host(self, q, k, v, gate_c, gate_f, out, idx, cnt=None):
        """Forward pass on host tensors (pinned for overlapped copies): inputs are
        copied in and out/idx/cnt written back by the library; enqueued on the
        current stream (synchronise it before reading the results)."""
        BHND = (self.B, self.heads, self.N, self.D)
        for t, n, dt, sh in ((q, "q", torch.bfloat16, BHND), (k, "k", torch.bfloat16, BHND),
                             (v, "v", torch.bfloat16, BHND), (gate_c, "gate_c", torch.float32, BHND[:3]),
                             (gate_f, "gate_f", torch.float32, BHND[:3]), (out, "out", torch.bfloat16, BHND),
                             (idx, "idx", torch.int32, (self.B, self.heads, self.C, self.kcap)),
                             (cnt, "cnt", torch.int32, (self.B, self.heads, self.C))):
            if t is None and n == "cnt":
                continue
            if not isinstance(t, torch.Tensor) or t.is_cuda or t.dtype != dt or tuple(t.shape) != tuple(sh) \
                    or not t.is_contiguous():
                raise ValueError(f"{n} must be a contiguous host tensor of {dt} and shape {tuple(sh)}")
        _check(load().vsa_run_host(self._h, _ptr(q), _ptr(k), _ptr(v), _ptr(gate_c), _ptr(gate_f), _ptr(out),
                                   _ptr(idx), _ptr(cnt), _stream()), "vsa_run_host")
        return out, idx, cnt

    def run_fixed_idx(self, q, k, v, gate_c, gate_f, idx, cnt=None, want_out=True, want_coarse=False,
                      want_fine=False):
        """Forward pass on a given selection. Returns (out, coarse, fine) (None where not requested)."""
        self._inputs(q, k, v, gate_c, gate_f)
        dev = q.device
        _need(idx, "idx", torch.int32, (self.B, self.heads, self.C, self.kcap))
        if cnt is not None:
            _need(cnt, "cnt", torch.int32, (self.B, self.heads, self.C))
        out = torch.empty_like(q) if want_out else None
        oc = torch.empty((self.B, self.heads, self.C, self.D), dtype=torch.float32, device=dev) if want_coarse else None
        of = torch.empty((self.B, self.heads, self.N, self.D), dtype=torch.float32, device=dev) if want_fine else None
        _check(load().vsa_run_fixed_idx(self._h, _ptr(q), _ptr(k), _ptr(v), _ptr(gate_c), _ptr(gate_f), _ptr(idx),
                                        _ptr(cnt), _ptr(out), _ptr(oc), _ptr(of), _stream()), "vsa_run_fixed_idx")
        return out, oc, of

    def check(self):
        """Synchronises and raises VSAError if a device-side error was recorded."""
        _check(load().vsa_check(self._h), "vsa_check")

    def set_wait_limit_ns(self, ns: int):
        _check(load().vsa_set_wait_limit_ns(self._h, int(ns)), "vsa_set_wait_limit_ns")

    def set_debug_stall(self, on: bool):
        _check(load().vsa_set_debug_stall(self._h, 1 if on else 0), "vsa_set_debug_stall")

    def set_cube_major_copies(self, on: bool):
        """Also write the cube-major copy of q into the workspace (k and v are always copied)."""
        _check(load().vsa_set_cube_major_copies(self._h, 1 if on else 0), "vsa_set_cube_major_copies")

    def set_stage_timing(self, on):
        """True (or a run count n >= 1): record stage events of the next runs,
        keeping the last n (1 for True); False/0 switches timing off."""
        n = int(on) if not isinstance(on, bool) else (1 if on else 0)
        _check(load().vsa_set_stage_timing(self._h, n), "vsa_set_stage_timing")

    def stage_times(self):
        """Device ms of (gather+pool, coarse, fine) of the last timed run."""
        ms = (ctypes.c_float * 3)()
        _check(load().vsa_stage_times(self._h, ms), "vsa_stage_times")
        return tuple(float(x) for x in ms)

    def stage_times_history(self, max_runs):
        """[(gather+pool, coarse, fine) ms] of the last timed runs, oldest first."""
        ms = (ctypes.c_float * (3 * max_runs))()
        n = ctypes.c_int(0)
        _check(load().vsa_stage_times_history(self._h, ms, int(max_runs), ctypes.byref(n)), "vsa_stage_times_history")
        return [tuple(float(x) for x in ms[3 * i: 3 * i + 3]) for i in range(n.value)]

    # ------------------------------------------------------------ workspace views
    def workspace_view(self, region: str, dtype, shape):
        off = getattr(self.layout, region)
        nbytes = torch.empty((), dtype=dtype).element_size()
        for s in shape:
            nbytes *= s
        return self.workspace[off: off + nbytes].view(dtype).view(*shape)

    def cube_major(self, which: str):
        return self.workspace_view(f"{which}_cube", torch.bfloat16, (self.B * self.heads, self.C, 64, self.D))

    def pooled(self, which: str):
        return self.workspace_view(f"{which}_pool", torch.float32, (self.B * self.heads, self.C, self.D))


def measure_l2_read(buf, passes, status):
    """Enqueues the L2 -> SM bulk-copy read of the uint8 CUDA tensor `buf`
    (`passes` times) on the current stream; `status` is a zeroed int32 CUDA
    tensor (bit 0 set if a bounded wait gave up)."""
    _need(buf, "buf", torch.uint8, tuple(buf.shape))
    _need(status, "status", torch.int32, tuple(status.shape))
    _check(load().vsa_measure_l2_read(_ptr(buf), buf.numel(), int(passes), _ptr(status), _stream()),
           "vsa_measure_l2_read")


def forward(q, k, v, gate_c, gate_f, T, H, W, topk=0, top_p=0.0, out=None, idx=None):
    """One-call form (library-owned plan cache). Returns (out, idx)."""
    B, heads, N, D = q.shape
    if N != T * H * W:
        raise ValueError("N must equal T*H*W")
    C = N // 64
    kcap = topk if topk > 0 else min(128, C)
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.bfloat16, (B, heads, N, D))
    for t, n in ((gate_c, "gate_c"), (gate_f, "gate_f")):
        _need(t, n, torch.float32, (B, heads, N))
    out = torch.empty_like(q) if out is None else out
    idx = torch.empty((B, heads, C, kcap), dtype=torch.int32, device=q.device) if idx is None else idx
    _check(load().vsa_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(gate_c), _ptr(gate_f), B, heads, T, H, W, D, topk,
                              ctypes.c_float(top_p), _ptr(out), _ptr(idx), _stream()), "vsa_forward")
    return out, idx


# ---------------------------------------------------------------- the projection side
class Rotation:
    """How the channels of a head turn with a token's positions.

    ``sections``: rotated channels of each axis (even; one to four axes, in
    order; together at most D, the remaining channels are not rotated). Pair i
    of an axis' n channels turns by position * scale * base**(-2i/n); with
    ``shared`` the pairs of all axes are numbered through and share one table,
    base**(-2j/sum). ``scale``: factor on each axis' positions (default 1).
    Pairs are channels (2j, 2j+1) if ``interleaved``, else (j, j + rot/2) of the
    rot = sum(sections) rotated channels, and then rot is a multiple of 16.
    """

    def __init__(self, D, sections, base=10000.0, scale=None, interleaved=True, shared=False):
        self.D, self.sections = int(D), tuple(int(n) for n in sections)
        self.interleaved, self.axes, self.rot = bool(interleaved), len(self.sections), sum(self.sections)
        if not 1 <= self.axes <= ROPE_MAX_AXES or any(n < 0 or n % 2 for n in self.sections):
            raise ValueError(f"sections must be one to {ROPE_MAX_AXES} even numbers, got {self.sections}")
        if not 0 <= self.rot <= min(self.D, 2 * ROPE_MAX_PAIRS):
            raise ValueError(f"sections {self.sections} do not fit into {self.D} channels")
        if not self.interleaved and self.rot % 16:
            raise ValueError("pairs (j, j + rot/2) need sections that add up to a multiple of 16")
        if not base > 0:
            raise ValueError("base must be positive")
        scale = (1.0,) * self.axes if scale is None else tuple(float(x) for x in scale)
        if len(scale) != self.axes:
            raise ValueError("scale must have one factor for each axis")
        self.spec = RotationSpec(self.rot, int(self.interleaved), self.axes)
        j = 0
        for a, n in enumerate(self.sections):
            for i in range(n // 2):
                self.spec.axis[j] = a
                self.spec.freq[j] = scale[a] * float(base) ** (-2.0 * j / self.rot if shared else -2.0 * i / n)
                j += 1
        self._packed = bytes(self.spec)


def _elsewhere(device):
    """Whether another device than the tensors' is current (the call then starts again on theirs)."""
    return torch._C._cuda_getDevice() != device.index


def _need_heads(t, name, like=None, dtype=None, device=None):
    """Checks for a CUDA tensor [B, heads, N, D] of any strides whose channels are contiguous; its packed view."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    shape, s = t.shape, t.stride()
    if len(s) != 4:
        raise ValueError(f"{name} must have shape [B, heads, N, D], got {tuple(shape)}")
    if t.dtype is not dtype and (dtype is not None or t.dtype not in TYPES):
        raise ValueError(f"{name} must be {dtype or 'bfloat16, float16 or float32'}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not {device}")
    if like is not None and shape != like:
        raise ValueError(f"{name} must have shape {tuple(like)}, got {tuple(shape)}")
    if s[3] != 1 and shape[3] > 1:
        raise ValueError(f"{name} must have contiguous channels")
    return _pack_heads(t.data_ptr(), shape[1], s[0], s[1], s[2])


def _where(rotation, grid, origin, positions, B, N, device):
    if (grid is None) == (positions is None):
        raise ValueError("give either grid or positions")
    if grid is not None:
        if rotation.axes != 3 or len(grid) != 3 or len(origin) != 3:
            raise ValueError("a grid and its origin have three numbers (T, H, W), and the rotation three axes")
        if any(not -2 ** 31 <= o < 2 ** 31 for o in origin):
            raise ValueError("origin must fit into 32 bits")
        if N != grid[0] * grid[1] * grid[2]:
            raise ValueError(f"N = {N} must equal T*H*W of grid {tuple(grid)}")
        return _pack_positions(*grid, *origin, 0, 0, 0)
    p, axes = positions, rotation.axes
    if not isinstance(p, torch.Tensor) or not p.is_cuda or p.device != device:
        raise ValueError(f"positions must be a CUDA tensor on {device}")
    if p.dtype not in (torch.int32, torch.float32):
        raise ValueError(f"positions must be int32 or float32, got {p.dtype}")
    shape, s = p.shape, p.stride()
    if len(s) not in (2, 3) or shape[-2:] != (N, axes) or (len(s) == 3 and shape[0] not in (1, B)):
        raise ValueError(f"positions must have shape [{N}, {axes}] or [{B}, {N}, {axes}], got {tuple(shape)}")
    if N and ((axes > 1 and s[-1] != 1) or (N > 1 and s[-2] != axes)):
        raise ValueError("positions must be contiguous")
    return _pack_positions(0, 0, 0, 0, 0, 0, p.data_ptr() or 16, 0 if p.dtype == torch.int32 else 1,
                           s[0] if len(s) == 3 and shape[0] > 1 else 0)


def _sizes(q, k, rotation, names=("q", "k")):
    """(B, N, D, packed sizes, packed q, packed k)"""
    hq = _need_heads(q, names[0])
    B, _, N, D = q.shape
    if rotation.D != D:
        raise ValueError(f"the rotation is for {rotation.D} channels, {names[0]} has {D}")
    hk = None
    if k is not None:
        hk = _need_heads(k, names[1], None, q.dtype, q.device)
        s = k.shape
        if s[0] != B or s[2] != N or s[3] != D:
            raise ValueError(f"{names[1]} must have shape [{B}, heads, {N}, {D}], got {tuple(s)}")
    return B, N, D, _pack_rope_sizes(TYPES[q.dtype], B, N, D), hq, hk


def _need_weight(w, name, D, device):
    if w is not None:
        _need(w, name, torch.float32, (D,))
        if w.device != device:
            raise ValueError(f"{name} is on {w.device}, not {device}")


def _output(t, o, name, like_input=False):
    """The given output, checked, or a new one (contiguous, or in its input's order of dimensions), and its view."""
    if t is None:
        if o is not None:
            raise ValueError(f"{name} has no input")
        return None, None
    if o is None:
        o = torch.empty_like(t) if like_input else torch.empty_like(t, memory_format=torch.contiguous_format)
        s = o.stride()
        return o, _pack_heads(o.data_ptr(), o.shape[1], s[0], s[1], s[2])
    return o, _need_heads(o, name, t.shape, t.dtype, t.device)


def rope(q, k, rotation, grid=None, origin=(0, 0, 0), positions=None, q_out=None, k_out=None):
    """Rotary positions with several axes on q and k ([B, heads, N, D], any strides; k may be None or have
    another number of heads). Tokens lie on the raster ``grid`` (T, H, W) from ``origin`` on, or at
    ``positions`` ([N, axes] or [B, N, axes], int32 or float32). Returns (q_out, k_out), contiguous unless
    given; an output may be its input. Enqueued on the current stream. Like every call here it leaves no trace for
    autograd, also where an input requires a gradient: rope_backward gives it."""
    B, N, _, sizes, hq, hk = _sizes(q, k, rotation)
    device = q.device
    where = _where(rotation, grid, origin, positions, B, N, device)
    if _elsewhere(device):
        with torch.cuda.device(device):
            return rope(q, k, rotation, grid, origin, positions, q_out, k_out)
    q_out, oq = _output(q, q_out, "q_out")
    k_out, ok = _output(k, k_out, "k_out")
    _check(_load_projection().vsa_rope(sizes, rotation._packed, where, hq, hk, oq, ok, _stream()), "vsa_rope")
    return q_out, k_out


def rope_backward(dq_out, dk_out, rotation, grid=None, origin=(0, 0, 0), positions=None, dq=None, dk=None):
    """Gradients of rope's inputs from those of its outputs (dk_out may be None): (dq, dk), contiguous unless
    given. Enqueued on the current stream."""
    B, N, _, sizes, hq, hk = _sizes(dq_out, dk_out, rotation, ("dq_out", "dk_out"))
    device = dq_out.device
    where = _where(rotation, grid, origin, positions, B, N, device)
    if _elsewhere(device):
        with torch.cuda.device(device):
            return rope_backward(dq_out, dk_out, rotation, grid, origin, positions, dq, dk)
    dq, oq = _output(dq_out, dq, "dq")
    dk, ok = _output(dk_out, dk, "dk")
    _check(_load_projection().vsa_rope_backward(sizes, rotation._packed, where, hq, hk, oq, ok, _stream()),
           "vsa_rope_backward")
    return dq, dk


def qk_norm_rope(q, k, q_weight, k_weight, rotation, grid=None, origin=(0, 0, 0), positions=None, eps=1e-6,
                 q_out=None, k_out=None):
    """RMS norm of every head's queries and keys (weights [D] fp32 or None) and the rotation of ``rope`` in one
    pass; arguments, outputs and stream as there."""
    B, N, D, sizes, hq, hk = _sizes(q, k, rotation)
    device = q.device
    where = _where(rotation, grid, origin, positions, B, N, device)
    _need_weight(q_weight, "q_weight", D, device)
    _need_weight(k_weight, "k_weight", D, device)
    if _elsewhere(device):
        with torch.cuda.device(device):
            return qk_norm_rope(q, k, q_weight, k_weight, rotation, grid, origin, positions, eps, q_out, k_out)
    q_out, oq = _output(q, q_out, "q_out")
    k_out, ok = _output(k, k_out, "k_out")
    _check(_load_projection().vsa_qk_norm_rope(sizes, rotation._packed, where, hq, hk, _address(q_weight),
                                               _address(k_weight), eps, oq, ok, _stream()), "vsa_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_backward(q, k, q_weight, k_weight, dq_out, dk_out, rotation, grid=None, origin=(0, 0, 0),
                          positions=None, eps=1e-6, dq=None, dk=None):
    """Gradients of qk_norm_rope from its inputs (nothing is saved) and the gradients of its outputs. Returns
    (dq, dk, dq_weight, dk_weight): dq and dk in the order of dimensions that q and k are stored in unless
    given, the weights' in fp32 (None where the weight is None). Enqueued on the current stream."""
    B, N, D, sizes, hq, hk = _sizes(q, k, rotation)
    device = q.device
    where = _where(rotation, grid, origin, positions, B, N, device)
    _need_weight(q_weight, "q_weight", D, device)
    _need_weight(k_weight, "k_weight", D, device)
    gq = _need_heads(dq_out, "dq_out", q.shape, q.dtype, device)
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out must be given together")
    gk = None if k is None else _need_heads(dk_out, "dk_out", k.shape, q.dtype, device)
    if _elsewhere(device):
        with torch.cuda.device(device):
            return qk_norm_rope_backward(q, k, q_weight, k_weight, dq_out, dk_out, rotation, grid, origin, positions,
                                         eps, dq, dk)
    L = _load_projection()
    dq, oq = _output(q, dq, "dq", like_input=True)
    dk, ok = _output(k, dk, "dk", like_input=True)
    dwq = None if q_weight is None else torch.empty_like(q_weight)
    dwk = None if k is None or k_weight is None else torch.empty_like(k_weight)
    nb = L.vsa_qk_norm_rope_backward_workspace_bytes(D)
    ws = q.new_empty(nb // q.element_size())
    _check(L.vsa_qk_norm_rope_backward(sizes, rotation._packed, where, hq, hk, _address(q_weight), _address(k_weight),
                                       eps, gq, gk, oq, ok, _address(dwq), _address(dwk), ws.data_ptr(), nb,
                                       _stream()), "vsa_qk_norm_rope_backward")
    return dq, dk, dwq, dwk


def _need_rows(t, name, dtype=None, device=None, shape=None):
    """Checks for a 16-bit CUDA tensor [B, N, channels] or [B, heads, N, D] whose channels are contiguous; its
    packed view as rows."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype and (dtype is not None or t.dtype not in (torch.bfloat16, torch.float16)):
        raise ValueError(f"{name} must be {dtype or 'bfloat16 or float16'}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not {device}")
    size, s = t.shape, t.stride()
    if shape is not None and size != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(size)}")
    if len(s) not in (3, 4):
        raise ValueError(f"{name} must have shape [B, N, channels] or [B, heads, N, D], got {tuple(size)}")
    if s[-1] != 1 and size[-1] > 1:
        raise ValueError(f"{name} must have contiguous channels")
    if len(s) == 3:
        return _pack_heads(t.data_ptr(), 1, s[0], 0, s[1])
    return _pack_heads(t.data_ptr(), size[1], s[0], s[1], s[2])


def _linear_sizes(x, weight, activation):
    """(B, N, F, packed sizes, packed x)"""
    hx = _need_rows(x, "x")
    shape = x.shape
    B, N, K = shape if len(shape) == 3 else (shape[0], shape[2], shape[1] * shape[3])
    if not isinstance(weight, torch.Tensor) or not weight.is_cuda or weight.device != x.device:
        raise ValueError(f"weight must be a CUDA tensor on {x.device}")
    if weight.dtype is not x.dtype:
        raise ValueError(f"weight must be {x.dtype}, got {weight.dtype}")
    if weight.dim() != 2 or weight.shape[1] != K:
        raise ValueError(f"weight must have shape [F, {K}], got {tuple(weight.shape)}")
    if weight.stride(1) != 1:
        raise ValueError("weight must have contiguous rows")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {list(ACTIVATIONS)}, got {activation!r}")
    F = weight.shape[0]
    return B, N, F, _pack_linear_sizes(TYPES[x.dtype], B, N, K, F), hx


def linear(x, weight, bias=None, activation=None, residual=None, heads=None, out=None, z=None):
    """act(x weight^T + bias) + residual. x is [B, N, K], or [B, heads, N, D] in the attention's layout (rows of
    K = heads * D channels, D a multiple of 64 if heads > 1), of any strides with contiguous channels; weight
    [F, K]; bias [F] fp32; activation None, "silu", "gelu" or "gelu_tanh". Returns [B, N, F], or
    [B, heads, N, F / heads] if ``heads`` is given; ``residual``, ``out`` and ``z`` (which receives
    x weight^T + bias for linear_backward) have that shape. out may be the residual. Enqueued on the current
    stream. The result has no autograd history, whatever x and weight require: linear_backward gives the gradients."""
    B, N, F, sizes, hx = _linear_sizes(x, weight, activation)
    device, dtype = x.device, x.dtype
    if bias is not None:
        _need_weight(bias, "bias", F, device)
    if heads is None:
        shape = (B, N, F)
    elif heads < 1 or F % heads:
        raise ValueError(f"{F} channels do not split into {heads} heads")
    else:
        shape = (B, heads, N, F // heads)
    hr = None if residual is None else _need_rows(residual, "residual", dtype, device, shape)
    hz = None if z is None else _need_rows(z, "z", dtype, device, shape)
    ho = None if out is None else _need_rows(out, "out", dtype, device, shape)
    if _elsewhere(device):
        with torch.cuda.device(device):
            return linear(x, weight, bias, activation, residual, heads, out, z)
    L = _load_projection()
    if out is None:
        out = x.new_empty(shape)
        ho = _pack_heads(out.data_ptr(), 1, N * F, 0, F) if heads is None else \
            _pack_heads(out.data_ptr(), heads, N * F, N * shape[3], shape[3])
    nb = L.vsa_linear_workspace_bytes(sizes)
    ws = x.new_empty(nb // 2) if nb else None
    _check(L.vsa_linear(sizes, hx, weight.data_ptr(), weight.stride(0), _address(bias), ACTIVATIONS[activation], hr, hz,
                        ho, _address(ws), nb, _stream()), "vsa_linear")
    return out


def linear_backward(x, weight, dout, z=None, activation=None, bias=False, dx=None, want=(True, True)):
    """Gradients of linear from that of its output (whose shape dout has): (dx, dweight, dbias). z is what linear
    stored, needed with an activation; dbias (fp32) is None unless ``bias``; ``want`` switches dx and dweight
    off. dx is in the order of dimensions that x is stored in unless given; it overlaps no other argument. The
    residual's gradient is dout. Enqueued on the current stream."""
    B, N, F, sizes, hx = _linear_sizes(x, weight, activation)
    device, dtype = x.device, x.dtype
    hg = _need_rows(dout, "dout", dtype, device)
    s = dout.shape
    if (s if len(s) == 3 else (s[0], s[2], s[1] * s[3])) != (B, N, F):
        raise ValueError(f"dout must have shape [{B}, {N}, {F}] or [{B}, heads, {N}, D], got {tuple(s)}")
    hz = None if activation is None else _need_rows(z, "z", dtype, device, s)
    hd = None if dx is None else _need_rows(dx, "dx", dtype, device, x.shape)
    if _elsewhere(device):
        with torch.cuda.device(device):
            return linear_backward(x, weight, dout, z, activation, bias, dx, want)
    L = _load_projection()
    if not want[0]:
        dx = hd = None
    elif dx is None:
        dx = torch.empty_like(x)
        hd = _need_rows(dx, "dx")
    dw = torch.empty_like(weight, memory_format=torch.contiguous_format) if want[1] else None
    db = x.new_empty(F, dtype=torch.float32) if bias else None
    nb = L.vsa_linear_backward_workspace_bytes(sizes, ACTIVATIONS[activation])
    ws = x.new_empty(nb // 2) if nb else None
    _check(L.vsa_linear_backward(sizes, hx, weight.data_ptr(), weight.stride(0), hz, ACTIVATIONS[activation], hg, hd,
                                 _address(dw), _address(db), _address(ws), nb, _stream()), "vsa_linear_backward")
    return dx, dw, db


def linear_check(device=None):
    """Synchronises the current stream of the device and raises VSAError if a wait inside a linear product that was
    enqueued on it, or captured into a graph, gave up since this stream's last check. Not while it is captured."""
    with torch.cuda.device(device):
        _check(load().vsa_linear_check(_stream()), "vsa_linear_check")
