"""Hierarchical (pyramid) top-K key-block selection + causal block-sparse attention on B200.

Thin ctypes binding over ``lib/libpyr.so`` (the C ABI declared in
``include/pyr.h``). Functions here only marshal arguments: torch tensors give
device pointers and the current CUDA stream; every step of the computation
runs in the library's sm_100a kernels. There is no CPU fallback: the library
is loaded on first use and every call raises ImportError if it is missing;
every call needs CUDA tensors.

    pyr_build(shape, K, pyr)                  key pyramid (mean pooling)
    pyr_update(shape, K, pyr, from_pos)       refresh the nodes over rewritten key positions
    pyr_select(shape, Q, pyr, idx, gap)       coarse-to-fine LogSumExp top-K
    pyr_select_ex(shape, Q, pyr, idx, gap, opts)
                                              the same with the PHAROS variants (per-head budget,
                                              confidence fallback, cross-level guidance) and a trace
    bsa_forward(shape, Q, K, V, idx, O, lse)  causal block-sparse attention
    phba_state_build(shape, M, Ks, V, A, W, PK, PV, workspace)
                                              PHBA prefix states (gated slot recurrence, chunkwise)
    phba_forward(shape, Q, K, V, idx, O, lse, Qs, M, PK, PV)
                                              block-sparse attention over tokens and state slots
    dense_forward(shape, Q, K, V, O, lse)     dense causal attention
    bsa_route_invert(shape, idx, offset, rho) routes in block-major form (for the backward)
    bsa_backward(shape, Q, K, V, O, lse, dO, idx, offset, rho, delta, dQ, dK, dV)
                                              gradients of the block-sparse attention
    forward(Q, K, V, b, topk, cap)            allocate outputs and run all three
    rope_spec(d, rot, base, layout, scaling)  rotary positions: the frequencies of a head's pairs
    rope_apply(spec, Q, K, Qo, Ko, pos)       rotate queries and keys (inverse=True: the gradient)
    packed_shape(S, T, Hq, Hkv, d, dtype), packed_plan(shape, cu)
                                              sequences of different lengths on one token axis
    packed_forward(shape, Q, K, V, plan, O, lse)
                                              causal attention of every packed sequence
    packed_backward(shape, Q, K, V, plan, O, lse, dO, delta, dQ, dK, dV)
                                              its gradients
    tree_shape(B, Hq, Hkv, N, T, d, dtype)
    tree_forward(shape, Q, K, V, lens, parent, O, lse, workspace)
                                              drafted token trees over a cache (one token: ragged decode)
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libpyr.so")

PYR_OK, PYR_EINVAL, PYR_EUNSUPPORTED, PYR_ECUDA, PYR_ETIMEOUT, PYR_EBADIDX, PYR_EBADSEQ = range(7)
PYR_F32, PYR_BF16 = 0, 1
PYR_TREE_ROOT, PYR_TREE_ABSENT = -1, -2

ABI_SYMBOLS = ("pyr_num_levels", "pyr_num_nodes", "pyr_num_qblocks", "pyr_pyramid_elems", "pyr_build", "pyr_means",
               "pyr_update",
               "pyr_select", "pyr_select_ex", "pyr_select_trace_levels", "pyr_select_trace_width", "bsa_forward",
               "dense_forward", "bsa_forward_host", "pyr_host_workspace_bytes", "bsa_route_invert", "bsa_backward",
               "bsa_backward_noalloc", "pyr_selftest_wait", "pyr_strerror", "phba_state_elems",
               "phba_state_workspace_bytes", "phba_state_build", "phba_forward", "rope_spec_init", "rope_apply",
               "packed_plan_elems", "packed_plan", "packed_forward", "packed_backward", "tree_workspace_bytes",
               "tree_forward")


class PyrShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "Hq", "Hkv", "N", "Nq", "q_offset", "d", "b", "topk", "cap",
                                             "dtype")]

    def __repr__(self):
        return "PyrShape(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


class PyrSelectOpts(ctypes.Structure):
    _fields_ = [("budget", ctypes.c_void_p), ("fcf_tau", ctypes.c_float), ("fcf_extra", ctypes.c_int),
                ("rcg_lambda", ctypes.c_float), ("trace", ctypes.c_void_p)]


class PyrView(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch", ctypes.c_int64), ("head", ctypes.c_int64),
                ("row", ctypes.c_int64)]


class RopeSpec(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int), ("rot", ctypes.c_int), ("layout", ctypes.c_int), ("reserved", ctypes.c_int),
                ("scale", ctypes.c_double), ("freq", ctypes.c_double * 64)]


class PackedShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("S", "T", "Hq", "Hkv", "d", "dtype")]


class TreeShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "Hq", "Hkv", "N", "T", "d", "dtype")]


class PyrError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {strerror(code)} (status {code})")


def _load_lib():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"libpyr.so is missing at {LIB_PATH}; build it with `python -m hierarchical_block_sparse_pyr_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    sp = ctypes.POINTER(PyrShape)
    vp = ctypes.c_void_p
    lib.pyr_num_levels.argtypes = [sp]
    lib.pyr_num_levels.restype = ctypes.c_int
    lib.pyr_num_nodes.argtypes = [sp]
    lib.pyr_num_nodes.restype = ctypes.c_int64
    lib.pyr_num_qblocks.argtypes = [sp]
    lib.pyr_num_qblocks.restype = ctypes.c_int64
    lib.pyr_pyramid_elems.argtypes = [sp]
    lib.pyr_pyramid_elems.restype = ctypes.c_size_t
    lib.pyr_build.argtypes = [sp, vp, vp, vp, vp]
    lib.pyr_build.restype = ctypes.c_int
    lib.pyr_means.argtypes = [sp, vp, vp, vp, vp]
    lib.pyr_means.restype = ctypes.c_int
    lib.pyr_update.argtypes = [sp, vp, vp, ctypes.c_int, vp, vp]
    lib.pyr_update.restype = ctypes.c_int
    lib.pyr_select.argtypes = [sp, vp, vp, vp, vp, vp, vp]
    lib.pyr_select.restype = ctypes.c_int
    lib.pyr_select_ex.argtypes = [sp, vp, vp, ctypes.POINTER(PyrSelectOpts), vp, vp, vp, vp]
    lib.pyr_select_ex.restype = ctypes.c_int
    lib.pyr_select_trace_levels.argtypes = [sp]
    lib.pyr_select_trace_levels.restype = ctypes.c_int
    lib.pyr_select_trace_width.argtypes = [sp]
    lib.pyr_select_trace_width.restype = ctypes.c_int
    lib.bsa_forward.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.bsa_forward.restype = ctypes.c_int
    lib.dense_forward.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp]
    lib.dense_forward.restype = ctypes.c_int
    lib.bsa_forward_host.argtypes = [sp, vp, vp, vp, vp, vp, ctypes.c_int, vp, ctypes.c_size_t, vp, vp]
    lib.bsa_forward_host.restype = ctypes.c_int
    lib.pyr_host_workspace_bytes.argtypes = [sp, ctypes.c_int, ctypes.c_int]
    lib.pyr_host_workspace_bytes.restype = ctypes.c_size_t
    lib.bsa_route_invert.argtypes = [sp, vp, vp, vp, vp, vp]
    lib.bsa_route_invert.restype = ctypes.c_int
    lib.bsa_backward.argtypes = [sp] + [vp] * 15
    lib.bsa_backward.restype = ctypes.c_int
    lib.bsa_backward_noalloc.argtypes = [sp] + [vp] * 14
    lib.bsa_backward_noalloc.restype = ctypes.c_int
    lib.phba_state_elems.argtypes = [sp, ctypes.c_int]
    lib.phba_state_elems.restype = ctypes.c_size_t
    lib.phba_state_workspace_bytes.argtypes = [sp, ctypes.c_int]
    lib.phba_state_workspace_bytes.restype = ctypes.c_size_t
    lib.phba_state_build.argtypes = [sp, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp, vp]
    lib.phba_state_build.restype = ctypes.c_int
    lib.phba_forward.argtypes = [sp, vp, vp, vp, vp, vp, ctypes.c_int, vp, vp, vp, vp, vp, vp]
    lib.phba_forward.restype = ctypes.c_int
    vw, ps, ts = vp, ctypes.POINTER(PackedShape), ctypes.POINTER(TreeShape)  # (vw: a PyrView's address)
    i, dbl = ctypes.c_int, ctypes.c_double
    lib.rope_spec_init.argtypes = [ctypes.POINTER(RopeSpec), i, i, i, dbl, i, dbl, i]
    lib.rope_apply.argtypes = [ctypes.POINTER(RopeSpec), i, i, i, i, i, vw, vw, vp, ctypes.c_int64, i, vw, vw, i, vp,
                               vp]
    lib.packed_plan_elems.argtypes = [ps]
    lib.packed_plan_elems.restype = ctypes.c_size_t
    lib.packed_plan.argtypes = [ps, vp, vp, vp, vp]
    lib.packed_forward.argtypes = [ps, vw, vw, vw, vp, vw, vp, vp, vp]
    lib.packed_backward.argtypes = [ps, vw, vw, vw, vp, vw, vp, vw, vp, vw, vw, vw, vp, vp]
    lib.tree_workspace_bytes.argtypes = [ts]
    lib.tree_workspace_bytes.restype = ctypes.c_size_t
    lib.tree_forward.argtypes = [ts, vw, vw, vw, vp, vp, vw, vp, vp, ctypes.c_size_t, vp, vp]
    for fn in (lib.rope_spec_init, lib.rope_apply, lib.packed_plan, lib.packed_forward, lib.packed_backward,
               lib.tree_forward):
        fn.restype = i
    lib.pyr_selftest_wait.argtypes = [vp, vp]
    lib.pyr_selftest_wait.restype = ctypes.c_int
    lib.pyr_strerror.argtypes = [ctypes.c_int]
    lib.pyr_strerror.restype = ctypes.c_char_p
    return lib


_lib_handle = None


def _L():
    """The loaded libpyr (loaded once, on first use)."""
    global _lib_handle
    if _lib_handle is None:
        _lib_handle = _load_lib()
    return _lib_handle


def strerror(code: int) -> str:
    return _L().pyr_strerror(code).decode()


def make_shape(B, Hq, Hkv, N, Nq, q_offset, d, b, topk, cap, dtype) -> PyrShape:
    if isinstance(dtype, torch.dtype):
        dtype = {torch.float32: PYR_F32, torch.bfloat16: PYR_BF16}[dtype]
    return PyrShape(B, Hq, Hkv, N, Nq, q_offset, d, b, topk, cap, dtype)


def shape_of(w) -> PyrShape:
    """PyrShape from any object with fields B, Hq, Hkv, N, Nq, q_offset, d, b, topk, cap, dtype."""
    return make_shape(w.B, w.Hq, w.Hkv, w.N, w.Nq, w.q_offset, w.d, w.b, w.topk, w.cap, w.dtype)


def num_levels(s: PyrShape) -> int:
    return _L().pyr_num_levels(ctypes.byref(s))


def num_nodes(s: PyrShape) -> int:
    return _L().pyr_num_nodes(ctypes.byref(s))


def num_qblocks(s: PyrShape) -> int:
    return _L().pyr_num_qblocks(ctypes.byref(s))


def pyramid_elems(s: PyrShape) -> int:
    """bf16 values of the pyr buffer: B * Hkv * P * 2 * d."""
    return _L().pyr_pyramid_elems(ctypes.byref(s))


def _dev(t, name, nullable=False):
    if t is None:
        if nullable:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _check(rc, what):
    if rc != PYR_OK:
        raise PyrError(rc, what)


def pyr_build(s: PyrShape, K, pyr, status=None, stream=None):
    _check(_L().pyr_build(ctypes.byref(s), _dev(K, "K"), _dev(pyr, "pyr"), _dev(status, "status", True),
                          _stream(stream)), "pyr_build")


def pyr_means(s: PyrShape, pyr, means, status=None, stream=None):
    """fp32 node means [B, Hkv, P, d] (means, written) from a pyramid's (hi, lo) pairs."""
    _check(_L().pyr_means(ctypes.byref(s), _dev(pyr, "pyr"), _dev(means, "means"), _dev(status, "status", True),
                          _stream(stream)), "pyr_means")


def pyr_update(s: PyrShape, K, pyr, from_pos: int, status=None, stream=None):
    _check(_L().pyr_update(ctypes.byref(s), _dev(K, "K"), _dev(pyr, "pyr"), int(from_pos), _dev(status, "status", True),
                           _stream(stream)), "pyr_update")


def pyr_select(s: PyrShape, Q, pyr, idx, gap=None, status=None, stream=None):
    _check(_L().pyr_select(ctypes.byref(s), _dev(Q, "Q"), _dev(pyr, "pyr"), _dev(idx, "idx"),
                           _dev(gap, "gap", True), _dev(status, "status", True), _stream(stream)), "pyr_select")


def select_trace_levels(s: PyrShape) -> int:
    return _L().pyr_select_trace_levels(ctypes.byref(s))


def select_trace_width(s: PyrShape) -> int:
    return _L().pyr_select_trace_width(ctypes.byref(s))


def new_trace(s: PyrShape, device="cuda"):
    """A trace buffer [B, Hkv, nqb, levels, width] int32 for pyr_select_ex."""
    return torch.empty((s.B, s.Hkv, num_qblocks(s), select_trace_levels(s), select_trace_width(s)),
                       dtype=torch.int32, device=device)


def pyr_select_ex(s: PyrShape, Q, pyr, idx, gap=None, budget=None, fcf_tau: float = 0.0, fcf_extra: int = 0,
                  rcg_lambda: float = 0.0, trace=None, status=None, stream=None):
    """pyr_select with the PHAROS variants: budget (int32 CUDA tensor [B, Hkv], DBA), fcf_tau / fcf_extra
    (FCF), rcg_lambda (RCG), and an optional trace buffer (new_trace)."""
    o = PyrSelectOpts(_dev(budget, "budget", True), float(fcf_tau), int(fcf_extra), float(rcg_lambda),
                      _dev(trace, "trace", True))
    _check(_L().pyr_select_ex(ctypes.byref(s), _dev(Q, "Q"), _dev(pyr, "pyr"), ctypes.byref(o), _dev(idx, "idx"),
                              _dev(gap, "gap", True), _dev(status, "status", True), _stream(stream)),
           "pyr_select_ex")


def bsa_forward(s: PyrShape, Q, K, V, idx, O, lse=None, status=None, stream=None):
    _check(_L().bsa_forward(ctypes.byref(s), _dev(Q, "Q"), _dev(K, "K"), _dev(V, "V"), _dev(idx, "idx"), _dev(O, "O"),
                            _dev(lse, "lse", True), _dev(status, "status", True), _stream(stream)), "bsa_forward")


def phba_state_elems(s: PyrShape, M: int) -> int:
    return _L().phba_state_elems(ctypes.byref(s), int(M))


def phba_state_workspace_bytes(s: PyrShape, M: int) -> int:
    return _L().phba_state_workspace_bytes(ctypes.byref(s), int(M))


class PhbaStates:
    """Device buffers of the PHBA prefix states (PK, PV [B, Hkv, nb, M, d]) and the build workspace."""

    def __init__(self, s: PyrShape, M: int, device="cuda"):
        nb = (s.N + s.b - 1) // s.b
        dt = torch.float32 if s.dtype == PYR_F32 else torch.bfloat16
        self.M = M
        self.PK = torch.empty((s.B, s.Hkv, nb, M, s.d), dtype=dt, device=device)
        self.PV = torch.empty_like(self.PK)
        self.workspace = torch.empty(phba_state_workspace_bytes(s, M), dtype=torch.uint8, device=device)


def phba_state_build(s: PyrShape, M: int, Ks, V, A, W, PK, PV, workspace, status=None, stream=None):
    """Prefix states of every key block: A (retention), W (write) fp32 CUDA tensors [B, Hkv, N, M]."""
    _check(_L().phba_state_build(ctypes.byref(s), int(M), _dev(Ks, "Ks"), _dev(V, "V"), _dev(A, "A"), _dev(W, "W"),
                                 _dev(PK, "PK"), _dev(PV, "PV"), _dev(workspace, "workspace"),
                                 workspace.numel() * workspace.element_size(), _dev(status, "status", True),
                                 _stream(stream)), "phba_state_build")


def phba_forward(s: PyrShape, Q, K, V, idx, O, lse=None, Qs=None, M: int = 0, PK=None, PV=None, status=None,
                 stream=None):
    """bsa_forward over the tokens and the M slots of the prefix states (Qs: the state query, None = Q)."""
    _check(_L().phba_forward(ctypes.byref(s), _dev(Q, "Q"), _dev(K, "K"), _dev(V, "V"), _dev(idx, "idx"),
                             _dev(Qs, "Qs", True), int(M), _dev(PK, "PK", M == 0), _dev(PV, "PV", M == 0),
                             _dev(O, "O"), _dev(lse, "lse", True), _dev(status, "status", True), _stream(stream)),
           "phba_forward")


def dense_forward(s: PyrShape, Q, K, V, O, lse=None, status=None, stream=None):
    _check(_L().dense_forward(ctypes.byref(s), _dev(Q, "Q"), _dev(K, "K"), _dev(V, "V"), _dev(O, "O"),
                              _dev(lse, "lse", True), _dev(status, "status", True), _stream(stream)),
           "dense_forward")


def _host(t, name, nullable=False):
    if t is None:
        if nullable:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor) or t.device.type != "cpu":
        raise TypeError(f"{name} must be a CPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def host_workspace_bytes(s: PyrShape, units_per_chunk: int = 0, with_lse: bool = False) -> int:
    return _L().pyr_host_workspace_bytes(ctypes.byref(s), int(units_per_chunk), int(bool(with_lse)))


def bsa_forward_host(s: PyrShape, Q, K, V, O, lse=None, units_per_chunk: int = 0, workspace=None, status=None,
                     stream=None):
    """The whole forward path for host (CPU, ideally pinned) Q, K, V; writes host O and lse.

    workspace: a CUDA uint8 tensor of at least host_workspace_bytes(s, units_per_chunk, lse is not None)
    bytes. The results are ready once `stream` (default: the current stream) has been synchronised."""
    _check(_L().bsa_forward_host(ctypes.byref(s), _host(Q, "Q"), _host(K, "K"), _host(V, "V"), _host(O, "O"),
                                 _host(lse, "lse", True), int(units_per_chunk), _dev(workspace, "workspace"),
                                 workspace.numel() * workspace.element_size(), _dev(status, "status", True),
                                 _stream(stream)), "bsa_forward_host")


def bsa_route_invert(s: PyrShape, idx, offset, rho, status=None, stream=None):
    _check(_L().bsa_route_invert(ctypes.byref(s), _dev(idx, "idx"), _dev(offset, "offset"), _dev(rho, "rho"),
                                 _dev(status, "status", True), _stream(stream)), "bsa_route_invert")


def bsa_backward(s: PyrShape, Q, K, V, O, lse, dO, idx, offset, rho, delta, dQ, dK, dV, status=None, stream=None):
    args = [_dev(t, n) for t, n in ((Q, "Q"), (K, "K"), (V, "V"), (O, "O"), (lse, "lse"), (dO, "dO"), (idx, "idx"),
                                    (offset, "offset"), (rho, "rho"), (delta, "delta"), (dQ, "dQ"), (dK, "dK"),
                                    (dV, "dV"))]
    _check(_L().bsa_backward(ctypes.byref(s), *args, _dev(status, "status", True), _stream(stream)), "bsa_backward")


def bsa_backward_noalloc(s: PyrShape, Q, K, V, O, lse, dO, idx, offset, rho, dQ, dK, dV, status=None,
                         stream=None):
    """bsa_backward without the delta workspace: the library keeps it in a fixed device array."""
    args = [_dev(t, n) for t, n in ((Q, "Q"), (K, "K"), (V, "V"), (O, "O"), (lse, "lse"), (dO, "dO"), (idx, "idx"),
                                    (offset, "offset"), (rho, "rho"), (dQ, "dQ"), (dK, "dK"), (dV, "dV"))]
    _check(_L().bsa_backward_noalloc(ctypes.byref(s), *args, _dev(status, "status", True), _stream(stream)),
           "bsa_backward_noalloc")


# ---- strided operands: rotary positions, packed prompts, drafted trees ------------------------------------

_DTYPES = {torch.float32: PYR_F32, torch.bfloat16: PYR_BF16}


def _dtype_code(dtype):
    if isinstance(dtype, torch.dtype):
        if dtype not in _DTYPES:
            raise TypeError(f"dtype must be float32 or bfloat16, not {dtype}")
        return _DTYPES[dtype]
    return _int32(dtype, "dtype")


_TORCH_DTYPES = {v: k for k, v in _DTYPES.items()}
_VIEW_ARRAYS = {n: ctypes.c_int64 * (4 * n) for n in range(1, 9)}


def _refuse(t, name, shape, dtype, device):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, the call's is {dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on another device than the other operands")
    raise ValueError(f"the elements of a row of {name} must be adjacent")


def _views(dtype, device, *operands):
    """pyr_views of (tensor, name, shape) operands, tensors [batch, head, row, d] or [head, row, d] of any
    strides with adjacent elements: the array that holds them and its address (32 bytes a view)."""
    td = _TORCH_DTYPES.get(dtype)
    vals = []
    for t, name, shape in operands:
        if not isinstance(t, torch.Tensor) or t.dtype is not td or t.shape != shape or t.get_device() != device or \
                device < 0:
            _refuse(t, name, shape, td, device)
        st = t.stride()
        if st[-1] != 1:
            _refuse(t, name, shape, td, device)
        vals += (t.data_ptr(), *st[:3]) if len(st) == 4 else (t.data_ptr(), 0, st[0], st[1])
    arr = _VIEW_ARRAYS[len(operands)](*vals)
    return arr, ctypes.addressof(arr)


def _device_of(t):
    return t.get_device() if isinstance(t, torch.Tensor) else -1


def _plain(t, name, dtype, need, device):
    """Pointer of a contiguous tensor of one dtype (None: NULL) of the shape `need` (a tuple), or of at least `need`
    elements in any shape (an int: buffers)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must have dtype {dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on another device than the other operands")
    if need.__class__ is tuple:
        if t.shape != need or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous with shape {need}, not {tuple(t.shape)}")
    elif not t.is_contiguous() or t.numel() < need:
        raise ValueError(f"{name} must be contiguous with at least {need} elements")
    return t.data_ptr()


def _need(t, name, dtype, need, device):
    if t is None:
        raise ValueError(f"{name} is required")
    return _plain(t, name, dtype, need, device)


def _int32(x, name):
    """x as the library's 32-bit integer; ctypes would wrap one that does not fit."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} = {x} does not fit in 32 bits")
    return x


def _call(fn, what, device, stream, *args):
    """fn(*args, stream) with the operands' device current; stream None: that device's current stream."""
    if torch.cuda.current_device() != device:
        with torch.cuda.device(device):
            return _call(fn, what, device, stream, *args)
    rc = fn(*args, torch.cuda.current_stream(device).cuda_stream if stream is None else _stream(stream))
    if rc:
        raise PyrError(rc, what)


def _torch_stream(stream, device):
    """A stream argument (None, a torch stream, a raw handle) as a torch stream or None, for allocations."""
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else torch.cuda.default_stream(device)


_ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
_ROPE_SCALINGS = {None: 0, "none": 0, "linear": 1, "ntk": 2, "yarn": 3}


def rope_spec(d: int, rot: int = None, base: float = 10000.0, layout: str = "half", scaling: str = None,
              factor: float = 1.0, trained: int = 0) -> RopeSpec:
    """Rotary frequencies: the first `rot` elements of a head of d (all by default) turn in pairs (i, i + rot/2)
    ("half") or (2i, 2i + 1) ("interleaved"), pair i by base^(-2i/rot) radians per position. scaling None,
    "linear", "ntk" or "yarn" stretches them by `factor` ("yarn" takes the trained length). The result's
    fields freq (radians per position) and scale may be rewritten for any other schedule."""
    if layout not in _ROPE_LAYOUTS or scaling not in _ROPE_SCALINGS:
        raise ValueError(f"unknown layout {layout!r} or scaling {scaling!r}")
    spec = RopeSpec()
    _check(_L().rope_spec_init(ctypes.byref(spec), _int32(d, "d"), _int32(d if rot is None else rot, "rot"),
                               _ROPE_LAYOUTS[layout], float(base), _ROPE_SCALINGS[scaling], float(factor),
                               _int32(trained, "trained")), "rope_spec")
    return spec


def rope_apply(spec: RopeSpec, Q, K, Qo, Ko, pos=None, pos_offset: int = 0, inverse: bool = False, status=None,
               stream=None):
    """Rotate Q [B, Hq, N, d] into Qo and K [B, Hkv, N, d] into Ko (any strides; in place with Qo is Q, Ko is K;
    either pair may be None). pos: int32 [B, N] or [N]; None: row n is at pos_offset + n. inverse: the
    transposed rotation, which turns the outputs' gradients into the inputs'."""
    first = Q if Q is not None else K
    if not isinstance(first, torch.Tensor) or first.dim() != 4 or not first.is_cuda:
        raise TypeError("Q or K must be a CUDA tensor [B, H, N, d]")
    if (Q is None) != (Qo is None) or (K is None) != (Ko is None):
        raise ValueError("Q and Qo, and K and Ko, come in pairs")
    B, _, N, d = first.shape
    if d != spec.d:
        raise ValueError(f"the spec is for d = {spec.d}, not {d}")
    _int32(B, "B")
    _int32(N, "N")
    dt, dev = _dtype_code(first.dtype), first.get_device()
    operands, heads = [], [0, 0]
    for i, (x, y, name) in enumerate(((Q, Qo, "Q"), (K, Ko, "K"))):
        if x is None:
            continue
        if not isinstance(x, torch.Tensor) or x.dim() != 4 or x.shape[1] < 1:
            raise ValueError(f"{name} must be [B, H, N, d]")
        heads[i] = _int32(x.shape[1], "heads")
        shape = (B, heads[i], N, d)
        operands += ((x, name, shape), (y, name + "o", shape))
    arr, v = _views(dt, dev, *operands)
    q, qo = (v, v + 32) if Q is not None else (None, None)
    v += 64 if Q is not None else 0
    k, ko = (v, v + 32) if K is not None else (None, None)
    stride = 0
    p = _plain(pos, "pos", torch.int32, 0, dev)
    if pos is not None:
        if pos.shape != (B, N) and pos.shape != (N,):
            raise ValueError("pos must be [B, N] or [N]")
        stride = N if pos.dim() == 2 else 0
    _call(_L().rope_apply, "rope_apply", dev, stream, ctypes.byref(spec), B, heads[0], heads[1], N, dt, q, k, p, stride,
          _int32(pos_offset, "pos_offset"), qo, ko, int(bool(inverse)), _plain(status, "status", torch.int32, 1, dev))


def packed_shape(S: int, T: int, Hq: int, Hkv: int, d: int, dtype) -> PackedShape:
    """S sequences on a token axis of T tokens (the last sequence may end before T)."""
    return PackedShape(_int32(S, "S"), _int32(T, "T"), _int32(Hq, "Hq"), _int32(Hkv, "Hkv"), _int32(d, "d"),
                       _dtype_code(dtype))


def packed_plan_elems(s: PackedShape) -> int:
    return _L().packed_plan_elems(ctypes.byref(s))


def _plan_words(s):
    """packed_plan_elems, asked of the library once per shape and its values."""
    key = (s.S, s.T, s.Hq, s.Hkv, s.d, s.dtype)
    known = getattr(s, "_words", None)
    if known is None or known[0] != key:
        known = s._words = (key, packed_plan_elems(s))
    return known[1]


def packed_plan(s: PackedShape, cu, plan=None, status=None, stream=None):
    """The work list of sequences [cu[i], cu[i+1]) (int32 CUDA tensor [S + 1]); it serves every packed_forward
    and packed_backward of this shape and these boundaries. Returns plan (allocated if None, as memory of the
    stream that writes it: another stream's user waits for that stream and keeps the plan until it is done)."""
    dev = _device_of(cu)
    c = _need(cu, "cu", torch.int32, (s.S + 1,), dev)
    n = packed_plan_elems(s)
    if plan is None:
        with torch.cuda.stream(_torch_stream(stream, dev)):
            plan = torch.empty(max(n, 1), dtype=torch.int32, device=cu.device)
    _call(_L().packed_plan, "packed_plan", dev, stream, ctypes.byref(s), c,
          _need(plan, "plan", torch.int32, n, dev), _plain(status, "status", torch.int32, 1, dev))
    return plan


def packed_forward(s: PackedShape, Q, K, V, plan, O, lse=None, status=None, stream=None):
    """Causal attention inside every packed sequence: Q, O [Hq, T, d], K, V [Hkv, T, d] (any strides), lse fp32
    [Hq, T]. Tokens outside the sequences are neither used nor written."""
    dev = _device_of(Q)
    q, kv = (s.Hq, s.T, s.d), (s.Hkv, s.T, s.d)
    arr, v = _views(s.dtype, dev, (Q, "Q", q), (K, "K", kv), (V, "V", kv), (O, "O", q))
    _call(_L().packed_forward, "packed_forward", dev, stream, ctypes.byref(s), v, v + 32, v + 64,
          _need(plan, "plan", torch.int32, _plan_words(s), dev), v + 96,
          _plain(lse, "lse", torch.float32, (s.Hq, s.T), dev), _plain(status, "status", torch.int32, 1, dev))


def packed_backward(s: PackedShape, Q, K, V, plan, O, lse, dO, delta, dQ, dK, dV, status=None, stream=None):
    """Gradients of packed_forward for dO, from its O and lse: dQ, dK, dV (views like Q, K, V), with delta an
    fp32 workspace [Hq, T]."""
    dev = _device_of(Q)
    q, kv = (s.Hq, s.T, s.d), (s.Hkv, s.T, s.d)
    arr, v = _views(s.dtype, dev, (Q, "Q", q), (K, "K", kv), (V, "V", kv), (O, "O", q), (dO, "dO", q), (dQ, "dQ", q),
                    (dK, "dK", kv), (dV, "dV", kv))
    n = (s.Hq, s.T)
    _call(_L().packed_backward, "packed_backward", dev, stream, ctypes.byref(s), v, v + 32, v + 64,
          _need(plan, "plan", torch.int32, _plan_words(s), dev), v + 96, _need(lse, "lse", torch.float32, n, dev),
          v + 128, _need(delta, "delta", torch.float32, n, dev), v + 160, v + 192, v + 224,
          _plain(status, "status", torch.int32, 1, dev))


def tree_shape(B: int, Hq: int, Hkv: int, N: int, T: int, d: int, dtype) -> TreeShape:
    """T drafted tokens of each of B sequences over caches of N rows."""
    return TreeShape(_int32(B, "B"), _int32(Hq, "Hq"), _int32(Hkv, "Hkv"), _int32(N, "N"), _int32(T, "T"),
                     _int32(d, "d"), _dtype_code(dtype))


def tree_workspace_bytes(s: TreeShape) -> int:
    return _L().tree_workspace_bytes(ctypes.byref(s))


def tree_forward(s: TreeShape, Q, K, V, lens, parent, O, lse=None, workspace=None, status=None, stream=None):
    """Attention of drafted tokens: Q, O [B, Hq, T, d], caches K, V [B, Hkv, N, d] (any strides), lens int32 [B]
    context lengths, parent int32 [B, T] (None: a chain), lse fp32 [B, Hq, T]; the drafted tokens' keys and
    values are in the cache rows lens[b] + t. workspace: a CUDA uint8 tensor of tree_workspace_bytes(s) bytes."""
    dev = _device_of(Q)
    q, kv = (s.B, s.Hq, s.T, s.d), (s.B, s.Hkv, s.N, s.d)
    arr, v = _views(s.dtype, dev, (Q, "Q", q), (K, "K", kv), (V, "V", kv), (O, "O", q))
    w = _need(workspace, "workspace", torch.uint8, 0, dev)
    _call(_L().tree_forward, "tree_forward", dev, stream, ctypes.byref(s), v, v + 32, v + 64,
          _need(lens, "lens", torch.int32, (s.B,), dev), _plain(parent, "parent", torch.int32, (s.B, s.T), dev), v + 96,
          _plain(lse, "lse", torch.float32, (s.B, s.Hq, s.T), dev), w, workspace.numel(),
          _plain(status, "status", torch.int32, 1, dev))


def selftest_wait(status, stream=None):
    """Launch the bounded-wait self-test; status (int32 CUDA tensor) reads PYR_ETIMEOUT afterwards."""
    _check(_L().pyr_selftest_wait(_dev(status, "status"), _stream(stream)), "pyr_selftest_wait")


class Buffers:
    """Device buffers of one forward pass (allocated by torch, owned by the caller)."""

    def __init__(self, s: PyrShape, device="cuda"):
        self.shape = s
        nqb = num_qblocks(s)
        dt = torch.float32 if s.dtype == PYR_F32 else torch.bfloat16
        # each node mean x is stored as the bf16 pair (hi, lo) = (RN(x), RN(x - hi))
        self.pyr = torch.empty((s.B, s.Hkv, num_nodes(s), 2, s.d), dtype=torch.bfloat16, device=device)
        self.idx = torch.empty((s.B, s.Hkv, nqb, s.topk), dtype=torch.int32, device=device)
        self.gap = torch.empty((s.B, s.Hkv, nqb), dtype=torch.float32, device=device)
        self.O = torch.empty((s.B, s.Hq, s.Nq, s.d), dtype=dt, device=device)
        self.lse = torch.empty((s.B, s.Hq, s.Nq), dtype=torch.float32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)


class BackwardBuffers:
    """Device buffers of one backward pass (allocated by torch, owned by the caller)."""

    def __init__(self, s: PyrShape, device="cuda"):
        self.shape = s
        nqb = num_qblocks(s)
        nb = (s.N + s.b - 1) // s.b
        dt = torch.float32 if s.dtype == PYR_F32 else torch.bfloat16
        self.offset = torch.empty((s.B * s.Hkv, nb + 1), dtype=torch.int32, device=device)
        self.rho = torch.empty((s.B * s.Hkv, nqb * s.topk), dtype=torch.int32, device=device)
        self.delta = torch.empty((s.B, s.Hq, s.Nq), dtype=torch.float32, device=device)
        self.dQ = torch.empty((s.B, s.Hq, s.Nq, s.d), dtype=dt, device=device)
        self.dK = torch.empty((s.B, s.Hkv, s.N, s.d), dtype=dt, device=device)
        self.dV = torch.empty((s.B, s.Hkv, s.N, s.d), dtype=dt, device=device)


def run_backward(s: PyrShape, Q, K, V, dO, fwd: "Buffers", bwd: BackwardBuffers, stream=None):
    """Enqueue route inversion and the gradients of the forward pass held in fwd."""
    bsa_route_invert(s, fwd.idx, bwd.offset, bwd.rho, fwd.status, stream)
    bsa_backward(s, Q, K, V, fwd.O, fwd.lse, dO, fwd.idx, bwd.offset, bwd.rho, bwd.delta, bwd.dQ, bwd.dK, bwd.dV,
                 fwd.status, stream)
    return bwd


def pyramid_means(s: PyrShape, pyr: torch.Tensor, stream=None) -> torch.Tensor:
    """Allocate and fill the fp32 node means [B, Hkv, P, d] of a pyramid (pyr_means)."""
    means = torch.empty((s.B, s.Hkv, num_nodes(s), s.d), dtype=torch.float32, device=pyr.device)
    pyr_means(s, pyr, means, stream=stream)
    return means


def run(s: PyrShape, Q, K, V, buf: Buffers, stream=None, with_gap=True):
    """Enqueue the whole path (pyramid, selection, attention) into buf."""
    pyr_build(s, K, buf.pyr, buf.status, stream)
    pyr_select(s, Q, buf.pyr, buf.idx, buf.gap if with_gap else None, buf.status, stream)
    bsa_forward(s, Q, K, V, buf.idx, buf.O, buf.lse, buf.status, stream)
    return buf


def forward(Q, K, V, b: int, topk: int, cap: int, q_offset: int = 0):
    """Allocate outputs and run pyramid + selection + block-sparse attention.

    Q: [B, Hq, Nq, d]; K, V: [B, Hkv, N, d] CUDA tensors (fp32 or bf16).
    Returns (O, lse, idx, gap); raises PyrError on a host-side error or on a
    device-side status (read after synchronising the current stream).
    """
    B, Hq, Nq, d = Q.shape
    N, Hkv = K.shape[2], K.shape[1]
    s = make_shape(B, Hq, Hkv, N, Nq, q_offset, d, b, topk, cap, Q.dtype)
    buf = run(s, Q, K, V, Buffers(s, Q.device))
    torch.cuda.current_stream().synchronize()
    code = int(buf.status.item())
    if code:
        raise PyrError(code, "device")
    return buf.O, buf.lse, buf.idx, buf.gap
