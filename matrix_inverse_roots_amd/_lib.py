"""ctypes binding of include/dash.h.  Argument marshalling only; all work runs in libdash.so.

Each ``dash_*`` function mirrors the C call of the same name.  Device buffers are torch tensors
(contiguous, on the GPU); sizes are passed explicitly as in the C ABI.  ``stream=None`` means
torch's current HIP stream on the tensors' device.
"""
from __future__ import annotations

import ctypes
import operator
import os
import sys

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libdash.so")

DASH_OK, DASH_ERR_INVALID_ARG, DASH_ERR_SHAPE, DASH_ERR_WORKSPACE, DASH_ERR_UNSUPPORTED, DASH_ERR_DEVICE = range(6)
DASH_FP32, DASH_FP16, DASH_BF16, DASH_FP32_SPLIT, DASH_FP32_SPLIT16 = 0, 1, 2, 3, 4
DASH_SCALE_FROBENIUS, DASH_SCALE_POWER = 0, 1
(DASH_OP_SCALE, DASH_OP_NDB, DASH_OP_CN, DASH_OP_CHEB, DASH_OP_APPLY, DASH_OP_STATS, DASH_OP_EVD,
 DASH_OP_ROUTED) = range(8)
DASH_MX_E2M1, DASH_MX_E4M3 = 0, 1


class DashError(RuntimeError):
    def __init__(self, call: str, status: int):
        self.status = status
        super().__init__("%s failed: %s (status %d)" % (call, dash_status_string(status), status))


class DashMat(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("ld", ctypes.c_int64)]


class DashVec(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("len", ctypes.c_int64)]


class DashTensor(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("ld", ctypes.c_int64), ("type", ctypes.c_int)]


_lib = None
_torch_module = None
_Tensor = ()  # torch.Tensor
_dtypes = {}  # element types by the names that _Args.ptr takes
_precs = {}  # dash_prec by element type


def _torch_loaded():
    """Whether the program has torch (only then can an argument be a tensor); takes it up if so."""
    return sys.modules.get("torch") is not None and _torch() is not None


def _torch():
    """torch, imported at the first call that needs it."""
    global _torch_module, _Tensor
    if _torch_module is None:
        import torch

        _dtypes.update(float32=torch.float32, int32=torch.int32, uint8=torch.uint8)
        _precs.update({torch.float32: DASH_FP32, torch.float16: DASH_FP16, torch.bfloat16: DASH_BF16})
        _Tensor = torch.Tensor
        _torch_module = torch
    return _torch_module


def library() -> ctypes.CDLL:
    """Load libdash.so (raises if it has not been built: there is no fallback path)."""
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise ImportError("libdash.so is not built; run `python -m matrix_inverse_roots_amd.build`")
        lib = ctypes.CDLL(library_path)
        vp, i32, i64, f32, f64, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                                      ctypes.c_double, ctypes.c_size_t)
        st = ctypes.c_int
        sig = {
            "dash_stack": (st, [ctypes.POINTER(DashMat), i32, i32, vp, vp]),
            "dash_unstack": (st, [vp, i32, ctypes.POINTER(DashMat), i32, vp]),
            "dash_update_stats": (st, [vp, i64, i32, f32, vp, vp]),
            "dash_update_stats_prec": (st, [vp, i64, i32, f32, st, vp, vp]),
            "dash_update_stats_ws": (st, [vp, i64, i32, f32, st, vp, vp, sz, vp]),
            "dash_scale": (st, [vp, i64, i32, st, st, i32, i32, vp, ctypes.c_uint64, vp, vp, sz, vp]),
            "dash_start_vectors": (st, [i32, i32, ctypes.c_uint64, vp, vp]),
            "dash_inverse_root_ndb": (st, [vp, vp, i64, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]),
            "dash_inverse_root_ndb_prec": (st, [vp, vp, i64, i32, i32, i32, st, vp, vp, vp, vp, vp, sz, vp]),
            "dash_inverse_root_cn": (st, [vp, vp, i64, i32, i32, i32, st, vp, vp, vp, vp, sz, vp]),
            "dash_inverse_root_ndb_half": (st, [vp, vp, i64, i32, i32, i32, i32, vp, vp, vp, vp, sz, vp]),
            "dash_inverse_root_ndb_lowp": (st, [vp, vp, i64, i32, i32, i32, st, i32, vp, vp, vp, vp, sz, vp]),
            "dash_inverse_root_ndb_adaptive": (st, [vp, vp, i64, i32, i32, i32, f32, vp, vp, vp, vp, vp, vp, sz,
                                                    vp]),
            "dash_inverse_root_cn_adaptive": (st, [vp, vp, i64, i32, i32, i32, f32, st, vp, vp, vp, vp, vp, sz, vp]),
            "dash_inverse_root_cheb": (st, [vp, vp, i64, i32, i32, f64, f64, vp, vp, vp, sz, vp]),
            "dash_inverse_root_cheb_prec": (st, [vp, vp, i64, i32, i32, f64, f64, st, vp, vp, vp, sz, vp]),
            "dash_inverse_root_evd": (st, [vp, i64, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]),
            "dash_inverse_root_evd_prec": (st, [vp, i64, i32, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]),
            "dash_apply": (st, [vp, vp, vp, i64, i32, vp, vp, sz, vp]),
            "dash_apply_prec": (st, [vp, vp, vp, i64, i32, st, vp, vp, sz, vp]),
            "dash_inverse_root_cheb_blocks": (st, [vp, vp, i64, i32, i32, f64, vp, f32, f64, st, vp, vp, vp, vp, sz,
                                                   vp]),
            "dash_spectrum_min": (st, [vp, vp, i64, i32, f64, i32, i32, vp, vp, vp, sz, vp]),
            "dash_residual_probe": (st, [vp, vp, i64, i32, i32, vp, vp, vp, sz, vp]),
            "dash_inverse_root_routed": (st, [vp, vp, i64, i32, i32, f64, f64, i32, i32, vp, f32, i32, st, vp, vp, vp,
                                              vp, vp, vp, sz, vp]),
            "dash_scale_noalloc": (st, [vp, i64, i32, st, st, i32, i32, vp, ctypes.c_uint64, vp, vp]),
            "dash_noalloc_scratch_bytes": (sz, []),
            "dash_stack_vec": (st, [ctypes.POINTER(DashVec), i32, i32, vp, vp]),
            "dash_unstack_vec": (st, [vp, i32, ctypes.POINTER(DashVec), i32, vp]),
            "dash_update_stats_vec": (st, [vp, i64, i32, f32, vp, vp]),
            "dash_inverse_sqrt_ndb": (st, [vp, vp, i64, i32, i32, st, vp, vp, vp, vp, sz, vp]),
            "dash_apply_vec": (st, [vp, vp, i64, i32, vp, vp]),
            "dash_mx_quantize": (st, [vp, st, i64, i64, i64, i64, st, vp, vp, vp, vp, vp, vp]),
            "dash_mx_dequantize": (st, [vp, vp, vp, i64, i64, i64, st, st, i64, vp, vp]),
            "dash_update_stats_mx": (st, [vp, vp, vp, vp, i64, i32, st, f32, vp, vp]),
            "dash_apply_mx": (st, [vp, vp, vp, vp, vp, vp, vp, i64, i32, st, vp, vp, sz, vp]),
            "dash_grad_stack_mx": (st, [vp, st, i64, vp, vp, st, i64, i64, i64, i32, i32, vp, vp, sz, vp]),
            "dash_grad_stack_mx_workspace": (st, [i64, i64, i64, st, ctypes.POINTER(sz)]),
            "dash_rmsnorm": (st, [vp, i64, vp, i64, st, vp, st, i64, i64, f32, vp, i64, vp, i64, st, vp, vp, vp, vp]),
            "dash_rmsnorm_backward": (st, [vp, i64, vp, i64, vp, i64, st, vp, st, vp, i64, i64, vp, i64, vp, i32, vp, sz,
                                           vp]),
            "dash_rmsnorm_backward_workspace": (st, [i64, i64, ctypes.POINTER(sz)]),
            "dash_grad_norm": (st, [ctypes.POINTER(DashTensor), i32, vp, vp, vp, sz, vp]),
            "dash_grad_norm_workspace": (st, [ctypes.POINTER(DashTensor), i32, ctypes.POINTER(sz)]),
            "dash_grad_clip": (st, [ctypes.POINTER(DashTensor), i32, vp, f32, vp]),
            "dash_stack_clip": (st, [ctypes.POINTER(DashMat), i32, i32, vp, f32, vp, vp]),
            "dash_workspace_size": (st, [st, i64, i32, st, i32, ctypes.POINTER(sz)]),
            "dash_solver_products": (i64, [st, i32, i32]),
            "dash_flops": (f64, [st, i64, i32, st, i32, i32]),
            "dash_status_string": (ctypes.c_char_p, [st]),
            "dash_abi_version": (i32, []),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


class _Args:
    """Host-side checks of one call's tensor arguments before their pointers reach the library.

    A torch tensor must be a contiguous GPU tensor of the expected dtype, on the same device as the
    call's other tensors, with at least as many elements as the call touches; a violation raises
    ValueError and nothing is enqueued.  ``None`` is NULL.  Plain integers and objects that only
    expose ``data_ptr()`` pass through unchecked as raw device addresses (the ABI tests use them).
    """

    __slots__ = ("call", "device", "index")

    def __init__(self, call: str):
        self.call = call
        self.device = None
        self.index = None  # of that device

    def _tensor(self, t, name):
        if _torch_module is None and not _torch_loaded():  # (raw addresses need no torch)
            return False
        if not isinstance(t, _Tensor):
            return False
        index = t.get_device()
        if index != self.index or index < 0:  # the call's first tensor, or one elsewhere
            if index < 0:
                raise ValueError("%s: %s must be a GPU tensor, got one on %s" % (self.call, name, t.device))
            if self.device is not None:
                raise ValueError("%s: %s is on %s, the call's other tensors on %s" % (self.call, name, t.device,
                                                                                      self.device))
            self.device, self.index = t.device, index
        return True

    def ptr(self, t, name, dtype="float32", numel=0):
        """Pointer of tensor argument `name` of `dtype` ('float32', 'int32', 'uint8' or None for any) holding
        at least `numel` elements."""
        if t is None or t.__class__ is int:
            return t
        if (t.__class__ is _Tensor and t.get_device() == self.index) or self._tensor(t, name):
            want = _dtypes.get(dtype)
            if want is not None and t.dtype != want:
                raise ValueError("%s: %s must be %s, got %s" % (self.call, name, dtype, t.dtype))
            if not t.is_contiguous():
                raise ValueError("%s: %s must be contiguous" % (self.call, name))
            if t.numel() < numel:
                raise ValueError("%s: %s holds %d elements, the call touches %d" % (self.call, name, t.numel(),
                                                                                     int(numel)))
        elif isinstance(t, int):
            return t
        return t.data_ptr()

    def ws(self, t):
        """Workspace tensor: any dtype, contiguous, on the call's device; its byte size is checked by
        the library against dash_workspace_size."""
        if t is None or isinstance(t, int):
            return t
        if self._tensor(t, "ws") and not t.is_contiguous():
            raise ValueError("%s: ws must be contiguous" % self.call)
        return t.data_ptr()

    def mats(self, ts, name):
        """dash_mat descriptors of 2-D fp32 GPU matrices with unit column stride."""
        arr = (DashMat * len(ts))()
        for i, t in enumerate(ts):
            if self._tensor(t, "%s[%d]" % (name, i)):
                import torch

                if t.dim() != 2 or t.dtype != torch.float32 or t.stride(1) != 1:
                    raise ValueError("%s: %s[%d] must be a 2-D float32 matrix with unit column stride"
                                     % (self.call, name, i))
            arr[i].ptr = t.data_ptr()
            arr[i].rows, arr[i].cols = t.shape
            arr[i].ld = t.stride(0)
        return arr

    def rows(self, t, name, N, rows, cols, type, ld):
        """(pointer, dash_prec type, row pitch) of N row-major matrices of rows x cols, one after the
        other: a tensor [rows, cols] (N = 1) or [N, rows, cols] of float32, float16 or bfloat16 with unit
        column stride and matrices rows * pitch apart, or a raw pointer with type and ld given."""
        if t is None or t.__class__ is int or not ((t.__class__ is _Tensor and t.get_device() == self.index) or
                                                   self._tensor(t, name)):
            p = t if t is None or isinstance(t, int) else t.data_ptr()
            return p, DASH_FP32 if type is None else type, cols if ld is None else ld
        have = _precs.get(t.dtype)
        if have is None or type not in (None, have):
            raise ValueError("%s: %s must be float32, float16 or bfloat16, got %s" % (self.call, name, t.dtype))
        shape = t.shape
        if N == 1 and ld is None and shape == (rows, cols):  # (the usual matrix, by the shortest way)
            pitch, step = t.stride()
            if step == 1 and (pitch >= cols or rows == 1):
                return t.data_ptr(), have, pitch if pitch >= cols else cols
        shape = tuple(shape)
        if shape != (N, rows, cols) and (N != 1 or shape != (rows, cols)):
            raise ValueError("%s: %s must be [%d, %d, %d], got %s" % (self.call, name, N, rows, cols, shape))
        if t.numel() == 0:
            return t.data_ptr(), have, cols
        pitch = t.stride(-2) if rows > 1 else max(cols, t.stride(-2) if N == 1 else t.stride(0))
        if (cols > 1 and t.stride(-1) != 1) or pitch < cols or (N > 1 and t.stride(0) != rows * pitch):
            raise ValueError("%s: %s must be row-major with unit column stride" % (self.call, name))
        if ld not in (None, pitch):
            raise ValueError("%s: %s has a row pitch of %d, not %d" % (self.call, name, pitch, ld))
        return t.data_ptr(), have, pitch

    def vector(self, t, name, n, type):
        """(pointer, dash_prec type) of a contiguous vector of at least n elements of float32, float16 or
        bfloat16; a raw pointer takes type."""
        if t is None or t.__class__ is int or not self._tensor(t, name):
            return t if t is None or isinstance(t, int) else t.data_ptr(), DASH_FP32 if type is None else type
        have = _precs.get(t.dtype)
        if have is None or type not in (None, have):
            raise ValueError("%s: %s must be float32, float16 or bfloat16, got %s" % (self.call, name, t.dtype))
        return self.ptr(t, name, None, n), have

    def codes(self, codes, scales, name, N, rows, cols, fmt):
        """Pointers of the codes and scale bytes of N microscaled matrices of rows x cols."""
        n = N * rows * -(-cols // 32)
        return (self.ptr(codes, name, "uint8", n * (32 if fmt == DASH_MX_E4M3 else 16)),
                self.ptr(scales, name + "_scales" if name else "scales", "uint8", n))

    def vecs(self, ts, name):
        """dash_vec descriptors of contiguous 1-D fp32 GPU vectors."""
        arr = (DashVec * len(ts))()
        for i, t in enumerate(ts):
            if self._tensor(t, "%s[%d]" % (name, i)):
                import torch

                if t.dim() != 1 or t.dtype != torch.float32 or not t.is_contiguous():
                    raise ValueError("%s: %s[%d] must be a contiguous 1-D float32 vector" % (self.call, name, i))
            arr[i].ptr = t.data_ptr()
            arr[i].len = t.shape[0]
        return arr

    def tensors(self, ts, name):
        """dash_tensor descriptors of GPU gradients: contiguous ones of any shape, or matrices with unit column
        stride, of float32, float16 or bfloat16; a GradList's own."""
        if isinstance(ts, GradList):
            # (1000 tensors 35 us, which a call's kernels hide; shapes and strides as well would be 100 more)
            if ts._at and list(map(_Tensor.data_ptr, ts.tensors)) != ts._at:
                ts._differs(ts._at, _Tensor.data_ptr, self.call, "memory")
            if ts.index is not None:
                if self.index not in (None, ts.index):
                    raise ValueError("%s: %s is on %s, the call's other tensors on %s" % (self.call, name, ts.device,
                                                                                          self.device))
                self.device, self.index = ts.device, ts.index
            return ts.array
        arr = (DashTensor * len(ts))()
        for i, t in enumerate(ts):
            if not self._tensor(t, "%s[%d]" % (name, i)):
                raise ValueError("%s: %s[%d] must be a tensor" % (self.call, name, i))
            have = _precs.get(t.dtype)
            if have is None:
                raise ValueError("%s: %s[%d] must be float32, float16 or bfloat16, got %s" % (self.call, name, i, t.dtype))
            if t.is_contiguous():
                rows, cols = 1, t.numel()
                ld = cols
            elif t.dim() == 2 and (t.stride(1) == 1 or t.shape[1] == 1) and (t.shape[0] == 1 or
                                                                              t.stride(0) >= t.shape[1]):
                rows, cols = t.shape
                ld = t.stride(0) if rows > 1 else cols
            else:
                raise ValueError("%s: %s[%d] must be contiguous, or a matrix with unit column stride"
                                 % (self.call, name, i))
            arr[i] = (t.data_ptr(), rows, cols, ld, have)
        return arr

    def stream(self, stream):
        if stream is not None:
            return stream if isinstance(stream, int) else stream.cuda_stream
        if self.device is None:
            return _torch().cuda.current_stream(None).cuda_stream
        return _torch_module._C._cuda_getCurrentRawStream(self.index)  # (current_stream(device) without its object)

    def run(self, fn, *args):
        """fn(*args) with the tensors' device current, as a launch on that device's default stream needs;
        raises DashError on a non-OK status."""
        if self.device is None or self.index == _torch_module._C._cuda_getDevice():
            status = fn(*args)
        else:
            with _torch_module.cuda.device(self.device):
                status = fn(*args)
        if status != DASH_OK:
            raise DashError(self.call, status)


class GradList:
    """The gradients of a model, described once for many calls (dash_grad_norm, dash_grad_clip, dash_stack_clip).
    It stands for the tensors as they are when it is made, and keeps their memory.  A call raises ValueError once one of
    them lies elsewhere (another .data, set_, a storage that was resized), dash_stack_clip also once one has more or
    fewer elements; they need a new list then, as does a gradient that gets another tensor.  Other changes of shape
    within the same memory are not looked for: the list goes on standing for what it was made of."""

    __slots__ = ("tensors", "array", "device", "index", "_held", "_at", "_sizes", "_mats", "_tiles")

    def __init__(self, tensors):
        self.tensors = tuple(tensors)
        a = _Args("grad_list")
        self.array = a.tensors(self.tensors, "tensors")
        self.device, self.index = a.device, a.index
        self._held = tuple(t.detach() for t in self.tensors)  # (which no change of a tensor's own memory reaches)
        self._at = [t.data_ptr() for t in self._held]
        self._sizes = [t.numel() for t in self._held]
        self._mats = None
        self._tiles = (0, 0)  # a block size, and the tiles of that size

    def __len__(self):
        return len(self.tensors)

    def _differs(self, then, now, call, what):
        i = [now(t) == s for t, s in zip(self.tensors, then)].index(False)
        raise ValueError("%s: grads[%d] has other %s than when the list was made" % (call, i, what))

    def mats(self, call, B):
        """(dash_mat descriptors, tiles of B x B)"""
        if self._at and list(map(_Tensor.numel, self.tensors)) != self._sizes:
            self._differs(self._sizes, _Tensor.numel, call, "sizes")
        if self._mats is None:
            self._mats = _Args(call).mats(self._held, "grads")
        if self._tiles[0] != B:  # (300 weights 25 us)
            self._tiles = (B, _tiles([t.shape for t in self._held], B))
        return self._mats, self._tiles[1]


def _check(name, status):
    if status != DASH_OK:
        raise DashError(name, status)


def _nbytes(t):
    if t is None or isinstance(t, int):
        return 0
    return t.numel() * t.element_size()


def _prec_of(dtype):
    """The dash_prec of a torch element type."""
    _torch()
    if dtype not in _precs:
        raise ValueError("dtype must be torch.float32, torch.float16 or torch.bfloat16, got %s" % (dtype,))
    return _precs[dtype]


def _tiles(shapes, B):
    return sum((-(-r // B)) * (-(-c // B)) for r, c in shapes) if B > 0 else 0


def dash_status_string(status: int) -> str:
    return library().dash_status_string(status).decode()


def dash_abi_version() -> int:
    return library().dash_abi_version()


def dash_solver_products(op: int, iters1: int, iters2: int = 0) -> int:
    return library().dash_solver_products(op, iters1, iters2)


def dash_flops(op: int, N: int, B: int, prec: int = DASH_FP32, a1: int = 0, a2: int = 0) -> float:
    return library().dash_flops(op, N, B, prec, a1, a2)


def dash_workspace_size(op: int, N: int, B: int, prec: int = DASH_FP32, k_or_degree: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check("dash_workspace_size", library().dash_workspace_size(op, N, B, prec, k_or_degree, ctypes.byref(out)))
    return out.value


def workspace(op: int, N: int, B: int, prec: int = DASH_FP32, k_or_degree: int = 0, device="cuda"):
    """A byte tensor of the size dash_workspace_size reports (None when no workspace is needed)."""
    import torch

    n = dash_workspace_size(op, N, B, prec, k_or_degree)
    if n == 0:
        return None
    return torch.empty(n, dtype=torch.uint8, device=device)


def dash_stack(grads, B: int, G_stack, stream=None):
    a = _Args("dash_stack")
    arr = a.mats(grads, "grads")
    n = _tiles([tuple(t.shape) for t in grads], B) * B * B
    _check("dash_stack", library().dash_stack(arr, len(grads), B, a.ptr(G_stack, "G_stack", numel=n), a.stream(stream)))


def dash_unstack(U_stack, B: int, outs, stream=None):
    a = _Args("dash_unstack")
    arr = a.mats(outs, "outs")
    n = _tiles([tuple(t.shape) for t in outs], B) * B * B
    _check("dash_unstack", library().dash_unstack(a.ptr(U_stack, "U_stack", numel=n), B, arr, len(outs),
                                                  a.stream(stream)))


def dash_update_stats(G_stack, NG: int, B: int, beta: float, A, stream=None):
    a = _Args("dash_update_stats")
    _check("dash_update_stats",
           library().dash_update_stats(a.ptr(G_stack, "G_stack", numel=NG * B * B), NG, B, beta,
                                       a.ptr(A, "A", numel=2 * NG * B * B), a.stream(stream)))


def dash_update_stats_prec(G_stack, NG: int, B: int, beta: float, prec: int, A, stream=None):
    a = _Args("dash_update_stats_prec")
    _check("dash_update_stats_prec",
           library().dash_update_stats_prec(a.ptr(G_stack, "G_stack", numel=NG * B * B), NG, B, beta, prec,
                                            a.ptr(A, "A", numel=2 * NG * B * B), a.stream(stream)))


def dash_update_stats_ws(G_stack, NG: int, B: int, beta: float, prec: int, A, ws=None, stream=None):
    a = _Args("dash_update_stats_ws")
    _check("dash_update_stats_ws",
           library().dash_update_stats_ws(a.ptr(G_stack, "G_stack", numel=NG * B * B), NG, B, beta, prec,
                                          a.ptr(A, "A", numel=2 * NG * B * B), a.ws(ws), _nbytes(ws),
                                          a.stream(stream)))


def dash_scale(A, N: int, B: int, how: int, prec: int, k: int, steps: int, V0, s, ws=None, stream=None, seed: int = 0):
    """V0 None with power iteration: the start pool drawn on the device from seed."""
    a = _Args("dash_scale")
    vn = B * k if how == DASH_SCALE_POWER else 0
    _check("dash_scale", library().dash_scale(a.ptr(A, "A", numel=N * B * B), N, B, how, prec, k, steps,
                                              a.ptr(V0, "V0", numel=vn), seed, a.ptr(s, "s", numel=N), a.ws(ws),
                                              _nbytes(ws), a.stream(stream)))


def dash_start_vectors(B: int, k: int, seed: int, V0, stream=None):
    a = _Args("dash_start_vectors")
    _check("dash_start_vectors", library().dash_start_vectors(B, k, seed, a.ptr(V0, "V0", numel=B * k),
                                                              a.stream(stream)))


def dash_scale_noalloc(A, N: int, B: int, how: int, prec: int, k: int, steps: int, V0, s, stream=None,
                       seed: int = 0):
    """dash_scale with the library's own scratch: no workspace argument, nothing allocated."""
    a = _Args("dash_scale_noalloc")
    vn = B * k if how == DASH_SCALE_POWER else 0
    _check("dash_scale_noalloc",
           library().dash_scale_noalloc(a.ptr(A, "A", numel=N * B * B), N, B, how, prec, k, steps,
                                        a.ptr(V0, "V0", numel=vn), seed, a.ptr(s, "s", numel=N),
                                        a.stream(stream)))


def dash_noalloc_scratch_bytes() -> int:
    return library().dash_noalloc_scratch_bytes()


def dash_spectrum_min(A, s, N: int, B: int, hi: float, k: int, steps: int, V0, lam_min, ws=None, stream=None):
    a = _Args("dash_spectrum_min")
    _check("dash_spectrum_min",
           library().dash_spectrum_min(a.ptr(A, "A", numel=N * B * B), a.ptr(s, "s", numel=N), N, B, hi, k, steps,
                                       a.ptr(V0, "V0", numel=B * k), a.ptr(lam_min, "lam_min", numel=N), a.ws(ws),
                                       _nbytes(ws), a.stream(stream)))


def dash_residual_probe(A, X, N: int, B: int, k: int, V0, r, ws=None, stream=None):
    a = _Args("dash_residual_probe")
    _check("dash_residual_probe",
           library().dash_residual_probe(a.ptr(A, "A", numel=N * B * B), a.ptr(X, "X", numel=N * B * B), N, B, k,
                                         a.ptr(V0, "V0", numel=B * k), a.ptr(r, "r", numel=N), a.ws(ws),
                                         _nbytes(ws), a.stream(stream)))


def _solver_ptrs(a, A, s, X, N, B):
    return a.ptr(A, "A", numel=N * B * B), a.ptr(s, "s", numel=N), a.ptr(X, "X", numel=N * B * B)


def dash_inverse_root_ndb(A, s, N: int, B: int, iters1: int, iters2: int, X, sqrt_out=None, monitor=None,
                          status=None, ws=None, stream=None):
    a = _Args("dash_inverse_root_ndb")
    pA, ps, pX = _solver_ptrs(a, A, s, X, N, B)
    _check("dash_inverse_root_ndb",
           library().dash_inverse_root_ndb(pA, ps, N, B, iters1, iters2, pX, a.ptr(sqrt_out, "sqrt_out", numel=N * B * B),
                                           a.ptr(monitor, "monitor", numel=N * (iters1 + iters2)),
                                           a.ptr(status, "status", "int32", N), a.ws(ws), _nbytes(ws),
                                           a.stream(stream)))


def dash_inverse_root_ndb_prec(A, s, N: int, B: int, iters1: int, iters2: int, prec: int, X, sqrt_out=None,
                               monitor=None, status=None, ws=None, stream=None):
    a = _Args("dash_inverse_root_ndb_prec")
    pA, ps, pX = _solver_ptrs(a, A, s, X, N, B)
    _check("dash_inverse_root_ndb_prec",
           library().dash_inverse_root_ndb_prec(pA, ps, N, B, iters1, iters2, prec, pX,
                                                a.ptr(sqrt_out, "sqrt_out", numel=N * B * B),
                                                a.ptr(monitor, "monitor", numel=N * (iters1 + iters2)),
                                                a.ptr(status, "status", "int32", N), a.ws(ws), _nbytes(ws),
                                                a.stream(stream)))


def dash_inverse_root_cn(A, s, N: int, B: int, p: int, iters: int, prec: int, X, monitor=None, status=None,
                         ws=None, stream=None):
    a = _Args("dash_inverse_root_cn")
    pA, ps, pX = _solver_ptrs(a, A, s, X, N, B)
    _check("dash_inverse_root_cn",
           library().dash_inverse_root_cn(pA, ps, N, B, p, iters, prec, pX, a.ptr(monitor, "monitor", numel=N * iters),
                                          a.ptr(status, "status", "int32", N), a.ws(ws), _nbytes(ws),
                                          a.stream(stream)))


def dash_inverse_root_ndb_half(A, s, N: int, B: int, iters1: int, iters2: int, refine: int, X, monitor=None,
                               status=None, ws=None, stream=None):
    a = _Args("dash_inverse_root_ndb_half")
    pA, ps, pX = _solver_ptrs(a, A, s, X, N, B)
    _check("dash_inverse_root_ndb_half",
           library().dash_inverse_root_ndb_half(pA, ps, N, B, iters1, iters2, refine, pX,
                                                a.ptr(monitor, "monitor", numel=N * (iters1 + iters2)),
                                                a.ptr(status, "status", "int32", N), a.ws(ws), _nbytes(ws),
                                                a.stream(stream)))


def dash_inverse_root_ndb_lowp(A, s, N: int, B: int, iters1: int, iters2: int, prec: int, refine: int, X,
                               monitor=None, status=None, ws=None, stream=None):
    a = _Args("dash_inverse_root_ndb_lowp")
    pA, ps, pX = _solver_ptrs(a, A, s, X, N, B)
    _check("dash_inverse_root_ndb_lowp",
           library().dash_inverse_root_ndb_lowp(pA, ps, N, B, iters1, iters2, prec, refine, pX,
                                                a.ptr(monitor, "monitor", numel=N * (iters1 + iters2)),
                                                a.ptr(status, "status", "int32", N), a.ws(ws), _nbytes(ws),
                                                a.stream(stream)))


def dash_inverse_root_ndb_adaptive(A, s, N: int, B: int, max_iters1: int, max_iters2: int, tol: float, X, monitor,
                                   sqrt_out=None, steps=None, status=None, ws=None, stream=None):
    a = _Args("dash_inverse_root_ndb_adaptive")
    pA, ps, pX = _solver_ptrs(a, A, s, X, N, B)
    _check("dash_inverse_root_ndb_adaptive",
           library().dash_inverse_root_ndb_adaptive(pA, ps, N, B, max_iters1, max_iters2, tol, pX,
                                                    a.ptr(sqrt_out, "sqrt_out", numel=N * B * B),
                                                    a.ptr(monitor, "monitor", numel=N * (max_iters1 + max_iters2)),
                                                    a.ptr(steps, "steps", "int32", 2 * N),
                                                    a.ptr(status, "status", "int32", N), a.ws(ws), _nbytes(ws),
                                                    a.stream(stream)))


def dash_inverse_root_cn_adaptive(A, s, N: int, B: int, p: int, max_iters: int, tol: float, prec: int, X, monitor,
                                  steps=None, status=None, ws=None, stream=None):
    a = _Args("dash_inverse_root_cn_adaptive")
    pA, ps, pX = _solver_ptrs(a, A, s, X, N, B)
    _check("dash_inverse_root_cn_adaptive",
           library().dash_inverse_root_cn_adaptive(pA, ps, N, B, p, max_iters, tol, prec, pX,
                                                   a.ptr(monitor, "monitor", numel=N * max_iters),
                                                   a.ptr(steps, "steps", "int32", N),
                                                   a.ptr(status, "status", "int32", N), a.ws(ws), _nbytes(ws),
                                                   a.stream(stream)))


def dash_inverse_root_cheb(A, s, N: int, B: int, degree: int, lo: float, hi: float, X, status=None, ws=None,
                           stream=None):
    a = _Args("dash_inverse_root_cheb")
    pA, ps, pX = _solver_ptrs(a, A, s, X, N, B)
    _check("dash_inverse_root_cheb",
           library().dash_inverse_root_cheb(pA, ps, N, B, degree, lo, hi, pX, a.ptr(status, "status", "int32", N),
                                            a.ws(ws), _nbytes(ws), a.stream(stream)))


def dash_inverse_root_cheb_prec(A, s, N: int, B: int, degree: int, lo: float, hi: float, prec: int, X, status=None,
                                ws=None, stream=None):
    a = _Args("dash_inverse_root_cheb_prec")
    pA, ps, pX = _solver_ptrs(a, A, s, X, N, B)
    _check("dash_inverse_root_cheb_prec",
           library().dash_inverse_root_cheb_prec(pA, ps, N, B, degree, lo, hi, prec, pX,
                                                 a.ptr(status, "status", "int32", N), a.ws(ws), _nbytes(ws),
                                                 a.stream(stream)))


def dash_inverse_root_cheb_blocks(A, s, N: int, B: int, degree: int, floor: float, lam_min, theta: float, hi: float,
                                  prec: int, X, lo_out=None, status=None, ws=None, stream=None):
    a = _Args("dash_inverse_root_cheb_blocks")
    pA, ps, pX = _solver_ptrs(a, A, s, X, N, B)
    _check("dash_inverse_root_cheb_blocks",
           library().dash_inverse_root_cheb_blocks(pA, ps, N, B, degree, floor, a.ptr(lam_min, "lam_min", numel=N),
                                                   theta, hi, prec, pX, a.ptr(lo_out, "lo_out", numel=N),
                                                   a.ptr(status, "status", "int32", N), a.ws(ws), _nbytes(ws),
                                                   a.stream(stream)))


def dash_inverse_root_routed(A, s, N: int, B: int, degree: int, floor: float, hi: float, k: int, est_steps: int, V0,
                             tol: float, cn_iters: int, prec: int, X, lam_min=None, resid=None, route=None,
                             status=None, ws=None, stream=None):
    a = _Args("dash_inverse_root_routed")
    pA, ps, pX = _solver_ptrs(a, A, s, X, N, B)
    _check("dash_inverse_root_routed",
           library().dash_inverse_root_routed(pA, ps, N, B, degree, floor, hi, k, est_steps,
                                              a.ptr(V0, "V0", numel=B * k), tol, cn_iters, prec, pX,
                                              a.ptr(lam_min, "lam_min", numel=N), a.ptr(resid, "resid", numel=N),
                                              a.ptr(route, "route", "int32", N), a.ptr(status, "status", "int32", N),
                                              a.ws(ws), _nbytes(ws), a.stream(stream)))


def dash_inverse_root_evd(A, N: int, B: int, max_sweeps: int, refine: int, X, eigvals=None, sweeps=None, status=None,
                          ws=None, stream=None):
    a = _Args("dash_inverse_root_evd")
    _check("dash_inverse_root_evd",
           library().dash_inverse_root_evd(a.ptr(A, "A", numel=N * B * B), N, B, max_sweeps, refine,
                                           a.ptr(X, "X", numel=N * B * B), a.ptr(eigvals, "eigvals", numel=N * B),
                                           a.ptr(sweeps, "sweeps", "int32", N), a.ptr(status, "status", "int32", N),
                                           a.ws(ws), _nbytes(ws), a.stream(stream)))


def dash_inverse_root_evd_prec(A, N: int, B: int, max_sweeps: int, refine: int, prec: int, X, eigvals=None,
                               sweeps=None, status=None, ws=None, stream=None):
    a = _Args("dash_inverse_root_evd_prec")
    _check("dash_inverse_root_evd_prec",
           library().dash_inverse_root_evd_prec(a.ptr(A, "A", numel=N * B * B), N, B, max_sweeps, refine, prec,
                                                a.ptr(X, "X", numel=N * B * B),
                                                a.ptr(eigvals, "eigvals", numel=N * B),
                                                a.ptr(sweeps, "sweeps", "int32", N),
                                                a.ptr(status, "status", "int32", N), a.ws(ws), _nbytes(ws),
                                                a.stream(stream)))


def dash_apply(XL, XR, G_stack, NG: int, B: int, U_stack, ws=None, stream=None):
    a = _Args("dash_apply")
    n = NG * B * B
    _check("dash_apply", library().dash_apply(a.ptr(XL, "XL", numel=n), a.ptr(XR, "XR", numel=n),
                                              a.ptr(G_stack, "G_stack", numel=n), NG, B,
                                              a.ptr(U_stack, "U_stack", numel=n), a.ws(ws), _nbytes(ws),
                                              a.stream(stream)))


def dash_apply_prec(XL, XR, G_stack, NG: int, B: int, prec: int, U_stack, ws=None, stream=None):
    a = _Args("dash_apply_prec")
    n = NG * B * B
    _check("dash_apply_prec",
           library().dash_apply_prec(a.ptr(XL, "XL", numel=n), a.ptr(XR, "XR", numel=n),
                                     a.ptr(G_stack, "G_stack", numel=n), NG, B, prec,
                                     a.ptr(U_stack, "U_stack", numel=n), a.ws(ws), _nbytes(ws), a.stream(stream)))


def _pieces(lens, B):
    return sum(-(-n // B) for n in lens) if B > 0 else 0


def dash_stack_vec(grads, B: int, g_pieces, stream=None):
    """The pieces of B (the last zero-padded) of 1-D gradients into g_pieces[P, B]."""
    a = _Args("dash_stack_vec")
    arr = a.vecs(grads, "grads")
    n = _pieces([t.shape[0] for t in grads], B) * B
    _check("dash_stack_vec", library().dash_stack_vec(arr, len(grads), B, a.ptr(g_pieces, "g_pieces", numel=n),
                                                      a.stream(stream)))


def dash_unstack_vec(u_pieces, B: int, outs, stream=None):
    a = _Args("dash_unstack_vec")
    arr = a.vecs(outs, "outs")
    n = _pieces([t.shape[0] for t in outs], B) * B
    _check("dash_unstack_vec", library().dash_unstack_vec(a.ptr(u_pieces, "u_pieces", numel=n), B, arr, len(outs),
                                                          a.stream(stream)))


def dash_update_stats_vec(g_pieces, P: int, B: int, beta: float, L, stream=None):
    a = _Args("dash_update_stats_vec")
    _check("dash_update_stats_vec",
           library().dash_update_stats_vec(a.ptr(g_pieces, "g_pieces", numel=P * B), P, B, beta,
                                           a.ptr(L, "L", numel=P * B * B), a.stream(stream)))


def dash_inverse_sqrt_ndb(A, s, N: int, B: int, iters: int, prec: int, X, monitor=None, status=None, ws=None,
                          stream=None):
    a = _Args("dash_inverse_sqrt_ndb")
    pA, ps, pX = _solver_ptrs(a, A, s, X, N, B)
    _check("dash_inverse_sqrt_ndb",
           library().dash_inverse_sqrt_ndb(pA, ps, N, B, iters, prec, pX, a.ptr(monitor, "monitor", numel=N * iters),
                                           a.ptr(status, "status", "int32", N), a.ws(ws), _nbytes(ws),
                                           a.stream(stream)))


def dash_apply_vec(X, g_pieces, P: int, B: int, u_pieces, stream=None):
    a = _Args("dash_apply_vec")
    _check("dash_apply_vec",
           library().dash_apply_vec(a.ptr(X, "X", numel=P * B * B), a.ptr(g_pieces, "g_pieces", numel=P * B), P, B,
                                    a.ptr(u_pieces, "u_pieces", numel=P * B), a.stream(stream)))


def mx_buffers(N: int, rows: int, cols: int, fmt: int, device="cuda"):
    """(codes, scales): uint8 tensors [N, rows, bytes of a row] and [N, rows, groups] for N microscaled
    matrices of rows x cols."""
    if fmt not in (DASH_MX_E2M1, DASH_MX_E4M3):
        raise ValueError("mx_buffers: fmt must be DASH_MX_E2M1 or DASH_MX_E4M3, got %s" % (fmt,))
    torch = _torch()
    g = -(-cols // 32)
    return (torch.empty((N, rows, g * (32 if fmt == DASH_MX_E4M3 else 16)), dtype=torch.uint8, device=device),
            torch.empty((N, rows, g), dtype=torch.uint8, device=device))


def dash_mx_quantize(src, N: int, rows: int, cols: int, fmt: int, codes=None, scales=None, codes_t=None, scales_t=None,
                     diag=None, type=None, ld=None, stream=None):
    """src: a tensor [N, rows, cols] (or [rows, cols]); its element type and row pitch are taken from it
    (a raw pointer takes type and ld)."""
    a = _Args("dash_mx_quantize")
    p, prec, pitch = a.rows(src, "src", N, rows, cols, type, ld)
    c = a.codes(codes, scales, "codes", N, rows, cols, fmt)
    ct = a.codes(codes_t, scales_t, "codes_t", N, cols, rows, fmt)
    a.run(library().dash_mx_quantize, p, prec, N, rows, cols, pitch, fmt, *c, *ct, a.ptr(diag, "diag", numel=N * rows),
          a.stream(stream))


def dash_mx_dequantize(codes, scales, N: int, rows: int, cols: int, fmt: int, dst, diag=None, type=None, ld=None,
                       stream=None):
    """dst: a tensor [N, rows, cols] (or [rows, cols]) of the wanted element type."""
    a = _Args("dash_mx_dequantize")
    c = a.codes(codes, scales, "codes", N, rows, cols, fmt)
    p, prec, pitch = a.rows(dst, "dst", N, rows, cols, type, ld)
    a.run(library().dash_mx_dequantize, *c, a.ptr(diag, "diag", numel=N * rows), N, rows, cols, fmt, prec, pitch, p,
          a.stream(stream))


def dash_update_stats_mx(codes, scales, codes_t, scales_t, NG: int, B: int, fmt: int, beta: float, A, stream=None):
    a = _Args("dash_update_stats_mx")
    c = a.codes(codes, scales, "codes", NG, B, B, fmt)
    ct = a.codes(codes_t, scales_t, "codes_t", NG, B, B, fmt)
    a.run(library().dash_update_stats_mx, *c, *ct, NG, B, fmt, beta, a.ptr(A, "A", numel=2 * NG * B * B),
          a.stream(stream))


def dash_apply_mx(XL, XL_scales, XR, XR_scales, G_stack, NG: int, B: int, fmt: int, U_stack, XL_diag=None, XR_diag=None,
                  ws=None, stream=None):
    a = _Args("dash_apply_mx")
    n = NG * B * B
    cl = a.codes(XL, XL_scales, "XL", NG, B, B, fmt)
    cr = a.codes(XR, XR_scales, "XR", NG, B, B, fmt)
    a.run(library().dash_apply_mx, *cl, a.ptr(XL_diag, "XL_diag", numel=NG * B), *cr,
          a.ptr(XR_diag, "XR_diag", numel=NG * B), a.ptr(G_stack, "G_stack", numel=n), NG, B, fmt,
          a.ptr(U_stack, "U_stack", numel=n), a.ws(ws), _nbytes(ws), a.stream(stream))


def dash_grad_stack_mx_workspace(T: int, out_features: int, in_features: int, type: int) -> int:
    out = ctypes.c_size_t(0)
    _check("dash_grad_stack_mx_workspace",
           library().dash_grad_stack_mx_workspace(T, out_features, in_features, type, ctypes.byref(out)))
    return out.value


def grad_stack_mx_workspace(T, out_features: int, in_features: int, dtype, device="cuda"):
    """A byte tensor of the size dash_grad_stack_mx_workspace reports for dY of torch type `dtype` (None
    when no workspace is needed).  T: a token count, or several (any iterable) whose calls share the
    workspace: a smaller count can need more than a larger one, so it holds the largest size of all."""
    torch = _torch()
    try:
        counts = [operator.index(T)]
    except TypeError:
        counts = [operator.index(t) for t in T]
    prec = _prec_of(dtype)
    n = max(dash_grad_stack_mx_workspace(t, out_features, in_features, prec) for t in counts)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def dash_grad_stack_mx(dY, codes, scales, fmt: int, T: int, out_features: int, in_features: int, B: int, G_stack,
                       accumulate: bool = False, type=None, ldy=None, ws=None, stream=None):
    """dY: a tensor [T, out_features]; its element type and row pitch are taken from it (a raw pointer
    takes type and ldy)."""
    a = _Args("dash_grad_stack_mx")
    p, prec, pitch = a.rows(dY, "dY", 1, T, out_features, type, ldy)
    c = a.codes(codes, scales, "codes", 1, T, in_features, fmt)
    n = _tiles([(out_features, in_features)], B) * B * B
    a.run(library().dash_grad_stack_mx, p, prec, pitch, *c, fmt, T, out_features, in_features, B, int(bool(accumulate)),
          a.ptr(G_stack, "G_stack", numel=n), a.ws(ws), _nbytes(ws), a.stream(stream))


def dash_rmsnorm(x, T: int, n: int, eps: float, res=None, gain=None, h=None, y=None, fmt: int = DASH_MX_E4M3, codes=None,
                 scales=None, rstd=None, type=None, gain_type=None, ldx=None, ldr=None, ldh=None, ldy=None, stream=None):
    """x, res, h and y: tensors [T, n]; their element type and row pitches are taken from them (raw pointers
    take type and the pitches), gain's from it."""
    a = _Args("dash_rmsnorm")
    px, prec, pitch = a.rows(x, "x", 1, T, n, type, ldx)
    pr, _, pitch_r = a.rows(res, "res", 1, T, n, prec, ldr)
    pg, gprec = a.vector(gain, "gain", n, gain_type)
    ph, _, pitch_h = a.rows(h, "h", 1, T, n, prec, ldh)
    py, _, pitch_y = a.rows(y, "y", 1, T, n, prec, ldy)
    c = a.codes(codes, scales, "", 1, T, n, fmt)
    a.run(library().dash_rmsnorm, px, pitch, pr, pitch_r, prec, pg, gprec, T, n, eps, ph, pitch_h, py, pitch_y, fmt, *c,
          a.ptr(rstd, "rstd", numel=T), a.stream(stream))


def dash_rmsnorm_backward_workspace(T: int, n: int) -> int:
    out = ctypes.c_size_t(0)
    _check("dash_rmsnorm_backward_workspace", library().dash_rmsnorm_backward_workspace(T, n, ctypes.byref(out)))
    return out.value


def rmsnorm_backward_workspace(T: int, n: int, device="cuda"):
    """A byte tensor of the size dash_rmsnorm_backward_workspace reports (None when no workspace is needed); it
    serves calls of fewer rows too."""
    torch = _torch()
    size = dash_rmsnorm_backward_workspace(T, n)
    return torch.empty(size, dtype=torch.uint8, device=device) if size else None


def dash_rmsnorm_backward(dy, h, rstd, T: int, n: int, dx, gain=None, dh=None, dgain=None, accumulate: bool = False,
                          type=None, gain_type=None, lddy=None, ldh=None, lddh=None, lddx=None, ws=None, stream=None):
    """dy, h, dh and dx: tensors [T, n], as dash_rmsnorm's."""
    a = _Args("dash_rmsnorm_backward")
    py, prec, pitch_y = a.rows(dy, "dy", 1, T, n, type, lddy)
    ph, _, pitch_h = a.rows(h, "h", 1, T, n, prec, ldh)
    pd, _, pitch_d = a.rows(dh, "dh", 1, T, n, prec, lddh)
    px, _, pitch_x = a.rows(dx, "dx", 1, T, n, prec, lddx)
    pg, gprec = a.vector(gain, "gain", n, gain_type)
    a.run(library().dash_rmsnorm_backward, py, pitch_y, ph, pitch_h, pd, pitch_d, prec, pg, gprec,
          a.ptr(rstd, "rstd", numel=T), T, n, px, pitch_x, a.ptr(dgain, "dgain", numel=n), int(bool(accumulate)),
          a.ws(ws), _nbytes(ws), a.stream(stream))


def grad_list(tensors) -> GradList:
    """Describes gradients (contiguous tensors of any shape, or matrices with unit column stride; float32, float16
    or bfloat16) once, for a program whose gradients keep their buffers from step to step."""
    return GradList(tensors)


def dash_grad_norm_workspace(grads) -> int:
    out = ctypes.c_size_t(0)
    _check("dash_grad_norm_workspace",
           library().dash_grad_norm_workspace(_Args("dash_grad_norm_workspace").tensors(grads, "grads"), len(grads),
                                              ctypes.byref(out)))
    return out.value


def grad_norm_workspace(grads, device="cuda"):
    """A byte tensor of the size dash_grad_norm_workspace reports for these gradients (None for none)."""
    torch = _torch()
    size = dash_grad_norm_workspace(grads)
    return torch.empty(size, dtype=torch.uint8, device=device) if size else None


def dash_grad_norm(grads, norm, norms=None, ws=None, stream=None):
    """grads: tensors, or a grad_list of them."""
    a = _Args("dash_grad_norm")
    arr = a.tensors(grads, "grads")
    a.run(library().dash_grad_norm, arr, len(grads), a.ptr(norm, "norm", numel=1), a.ptr(norms, "norms", numel=len(grads)),
          a.ws(ws), _nbytes(ws), a.stream(stream))


def dash_grad_clip(grads, norm, max_norm: float, stream=None):
    """grads: tensors, or a grad_list of them; norm: what dash_grad_norm wrote."""
    a = _Args("dash_grad_clip")
    arr = a.tensors(grads, "grads")
    a.run(library().dash_grad_clip, arr, len(grads), a.ptr(norm, "norm", numel=1), max_norm, a.stream(stream))


def dash_stack_clip(grads, B: int, norm, max_norm: float, G_stack, stream=None):
    """grads: matrices as dash_stack's, or a grad_list of them."""
    a = _Args("dash_stack_clip")
    if isinstance(grads, GradList):
        a.tensors(grads, "grads")  # (the call's device)
        arr, tiles = grads.mats(a.call, B)
    else:
        arr, tiles = a.mats(grads, "grads"), _tiles([t.shape for t in grads], B)
    n = tiles * B * B
    a.run(library().dash_stack_clip, arr, len(grads), B, a.ptr(norm, "norm", numel=1), max_norm,
          a.ptr(G_stack, "G_stack", numel=n), a.stream(stream))
