"""Python binding of libar.so: argument marshalling only.

Every step of a collective runs in the library's HIP kernels; PyTorch only
supplies device memory (tensors) and the stream.  The entry points keep the
C names (``include/ar.h``):

    comm = Comm(nranks, max_bytes_per_rank, max_line_bytes_per_rank)
    comm.allreduce(send, recv, algo="ring", proto="simple", chunk_bytes=0)   # or "auto"
    comm.reduce_scatter(send, recv, ...)
    comm.allgather(send, recv, ...)
    plan_bytes(nranks, op, count, dtype, algo, proto, ...)
    select(nranks, op, count, dtype, algo="auto", proto="auto", max_line_bytes_per_rank=0)
    gated_ffn(x, w_gate, w_up, w_down, act="silu")                           # + gated_ffn_backward
    linear_cross_entropy(x, w, target)                                       # + linear_cross_entropy_backward

``send`` / ``recv`` are lists of N contiguous CUDA (HIP) tensors on the
communicator's device.  If the library is missing it is built once with hipcc;
if that fails every call raises -- there is no CPU fallback.
"""

import ctypes
import functools
import os

HERE = os.path.dirname(os.path.abspath(__file__))
# AR_LIBRARY points at another build of the same library (measurements only).
LIB_PATH = os.environ.get("AR_LIBRARY") or os.path.join(HERE, "libar.so")

OPS = {"allreduce": 0, "reduce_scatter": 1, "allgather": 2}
ALGOS = {"oneshot": 0, "twoshot": 1, "ring": 2, "tree": 3}
PROTOS = {"simple": 0, "ll": 1, "ll128": 2}
ALGO_AUTO, PROTO_AUTO = 4, 3  # AR_ALGO_AUTO / AR_PROTO_AUTO: the library picks (ar_select)
DTYPES = {"f32": 0, "bf16": 1, "i32": 2}
ESIZE = {"f32": 4, "bf16": 2, "i32": 4}
ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}

STATUS = {
    0: "AR_OK", 1: "AR_ERR_INVALID", 2: "AR_ERR_UNSUPPORTED", 3: "AR_ERR_NOMEM",
    4: "AR_ERR_TOO_LARGE", 5: "AR_ERR_HIP", 6: "AR_ERR_TIMEOUT", 7: "AR_ERR_BROKEN",
}

# Every symbol include/ar.h declares.
SYMBOLS = (
    "ar_comm_create", "ar_comm_destroy", "ar_comm_check", "ar_comm_reset",
    "ar_comm_workspace_bytes", "ar_comm_set_max_workgroups", "ar_allreduce", "ar_allreduce_rmsnorm", "ar_reduce_scatter", "ar_allgather",
    "ar_plan_bytes", "ar_select", "ar_debug_inject", "ar_debug_state", "ar_status_string",
    "ar_allreduce_noalloc", "ar_debug_calls", "ar_stream_ceiling",
    "ar_gated_ffn_workspace", "ar_gated_ffn", "ar_gated_ffn_backward",
    "ar_linear_cross_entropy_workspace", "ar_linear_cross_entropy", "ar_linear_cross_entropy_backward",
)


class CallRecord(ctypes.Structure):
    """ar_call_record (include/ar.h)."""
    _fields_ = [("seq", ctypes.c_uint64), ("op", ctypes.c_int32), ("algo", ctypes.c_int32),
                ("proto", ctypes.c_int32), ("dtype", ctypes.c_int32), ("nranks", ctypes.c_int32),
                ("in_place", ctypes.c_int32), ("grid", ctypes.c_uint32), ("batch", ctypes.c_uint32),
                ("counter_free", ctypes.c_uint32), ("by_die", ctypes.c_uint32), ("count", ctypes.c_uint64),
                ("ntasks", ctypes.c_uint64), ("tile_bytes", ctypes.c_uint64)]


class ARError(RuntimeError):
    def __init__(self, status, what=""):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)} ({_lib().ar_status_string(status).decode()})")


_LIB = None


def _declare(lib):
    P, S, I, U64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_uint64
    PP = ctypes.POINTER(ctypes.c_void_p)
    lib.ar_comm_create.argtypes = [I, S, S, ctypes.POINTER(P)]
    lib.ar_comm_destroy.argtypes = [P]
    lib.ar_comm_check.argtypes = [P, P, ctypes.POINTER(I), ctypes.POINTER(I)]
    lib.ar_comm_reset.argtypes = [P, P]
    lib.ar_comm_workspace_bytes.argtypes = [P]
    lib.ar_comm_workspace_bytes.restype = S
    lib.ar_comm_set_max_workgroups.argtypes = [P, ctypes.c_uint]
    lib.ar_allreduce_rmsnorm.argtypes = [P, PP, PP, PP, P, S, S, ctypes.c_float, I, P]
    for name in ("ar_allreduce", "ar_reduce_scatter", "ar_allgather"):
        getattr(lib, name).argtypes = [P, PP, PP, S, I, I, I, S, P]
    lib.ar_allreduce_noalloc.argtypes = [I, PP, PP, S, I, I, I, S, P]
    lib.ar_debug_calls.argtypes = [P, ctypes.POINTER(CallRecord), I, ctypes.POINTER(I)]
    lib.ar_stream_ceiling.argtypes = [I, PP, I, PP, S, P, I, I, I, P]
    lib.ar_plan_bytes.argtypes = [I, I, S, I, I, I, S, I, ctypes.POINTER(U64), ctypes.POINTER(U64),
                                  ctypes.POINTER(U64), ctypes.POINTER(U64)]
    lib.ar_select.argtypes = [I, I, S, I, I, I, S, ctypes.POINTER(I), ctypes.POINTER(I),
                              ctypes.POINTER(ctypes.c_double)]
    lib.ar_debug_inject.argtypes = [P, I, I, U64]
    lib.ar_debug_state.argtypes = [P, P, ctypes.POINTER(U64), I]
    lib.ar_gated_ffn_workspace.argtypes = [I, S, S, S, I, I]
    lib.ar_gated_ffn.argtypes = [I] + [PP] * 7 + [S, S, S, I, I, P, S, P]
    lib.ar_gated_ffn_backward.argtypes = [I] + [PP] * 11 + [S, S, S, I, I, P, S, P]
    lib.ar_linear_cross_entropy_workspace.argtypes = [I, S, S, S, I, I, S]
    lib.ar_linear_cross_entropy.argtypes = [I, PP, PP, P, PP, PP, S, S, S, I, P, S, P]
    lib.ar_linear_cross_entropy_backward.argtypes = [I, P, PP, PP, P, PP, PP, PP, S, S, S, I, S, P, S, P]
    lib.ar_status_string.argtypes = [I]
    lib.ar_status_string.restype = ctypes.c_char_p
    for name in SYMBOLS:
        if name in ("ar_gated_ffn_workspace", "ar_linear_cross_entropy_workspace"):
            getattr(lib, name).restype = S
        elif name not in ("ar_comm_workspace_bytes", "ar_status_string"):
            getattr(lib, name).restype = I
    return lib


def _lib():
    """Load libar.so (building it first if it is not there)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            from .build import build
            build()
        _LIB = _declare(ctypes.CDLL(LIB_PATH))
    return _LIB


def library():
    return _lib()


def _check(status, what):
    if status != 0:
        raise ARError(status, what)


def _algo(name):
    return ALGO_AUTO if name == "auto" else ALGOS[name]


def _proto(name):
    return PROTO_AUTO if name == "auto" else PROTOS[name]


_TORCH = None
_DT_NAMES = None  # torch dtype -> "f32" / "bf16" / "i32"


def _torch():
    global _TORCH, _DT_NAMES
    if _TORCH is None:
        import torch

        _DT_NAMES = {torch.float32: "f32", torch.bfloat16: "bf16", torch.int32: "i32"}
        _TORCH = torch
    return _TORCH


def _dtype_name(t):
    _torch()
    name = _DT_NAMES.get(t.dtype)
    if name is None:
        raise TypeError(f"unsupported tensor dtype {t.dtype}")
    return name


def _ptrs(tensors, nranks, device):
    if len(tensors) != nranks:
        raise ValueError(f"need {nranks} rank buffers, got {len(tensors)}")
    for t in tensors:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("rank buffers must be contiguous device tensors")
        if t.device.index != device:
            raise ValueError("rank buffers must live on the communicator's device")
    return (ctypes.c_void_p * nranks)(*[t.data_ptr() for t in tensors])


def _sizes(tensors, want, what):
    for i, t in enumerate(tensors):
        if t.numel() != want:
            raise ValueError(f"{what}[{i}] holds {t.numel()} elements; the call needs {want}")


def _marshal(tensors, nranks, dtype, want, device):
    """Pointer array of `nranks` rank tensors that all pass the checks keeping
    a kernel inside them (dtype, element count, device, contiguity), in one
    pass of cheap attribute reads; None if any fails (then `_rank_buffers`
    names the failure).  Small calls are bound by this host work."""
    if len(tensors) != nranks:
        return None
    ptrs = []
    for t in tensors:
        if t.dtype is not dtype or t.numel() != want or t.get_device() != device or not t.is_contiguous():
            return None
        ptrs.append(t.data_ptr())
    return (ctypes.c_void_p * nranks)(*ptrs)


def _rank_buffers(send, recv, nranks, device, n_send, n_recv):
    """(dtype name, send pointers, recv pointers) of a call, or the first
    failed check as an exception: dtypes, then element counts, then device
    and layout."""
    dt = _dtype_name(send[0])
    dtype = send[0].dtype
    s = _marshal(send, nranks, dtype, n_send, device)
    r = _marshal(recv, nranks, dtype, n_recv, device)
    if s is not None and r is not None:
        return dt, s, r
    for t in list(send) + list(recv):
        if _dtype_name(t) != dt:
            raise TypeError("all rank buffers must share one dtype")
    _sizes(send, n_send, "send")
    _sizes(recv, n_recv, "recv")
    _ptrs(send, nranks, device)
    _ptrs(recv, nranks, device)
    raise ValueError("rank buffers failed the device check")  # not reached: _ptrs names the failure


def _stream_handle(stream, device=None):
    torch = _torch()
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    if device is not None:  # the raw handle without building a Stream object
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(device))
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


class Comm:
    """N simulated ranks on the current device with a workspace allocated once."""

    def __init__(self, nranks: int, max_bytes_per_rank: int, max_line_bytes_per_rank: int = 0):
        import torch

        self.nranks = nranks
        self.device = torch.cuda.current_device()
        self._h = ctypes.c_void_p()
        _check(_lib().ar_comm_create(nranks, max_bytes_per_rank, max_line_bytes_per_rank,
                                     ctypes.byref(self._h)), "ar_comm_create")

    def close(self):
        if self._h:
            _check(_lib().ar_comm_destroy(self._h), "ar_comm_destroy")
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            if self._h:
                _lib().ar_comm_destroy(self._h)
        except Exception:
            pass

    @property
    def workspace_bytes(self) -> int:
        return _lib().ar_comm_workspace_bytes(self._h)

    def set_max_workgroups(self, max_workgroups: int):
        """Workgroup budget of later calls (0: the default, up to 3 per CU)."""
        _check(_lib().ar_comm_set_max_workgroups(self._h, max_workgroups), "ar_comm_set_max_workgroups")

    def _call(self, name, send, recv, count, algo, proto, chunk_bytes, stream, n_send, n_recv):
        """n_send / n_recv: the elements every send / recv buffer must hold.
        The C ABI sees only pointers, so a shorter tensor would let the kernel
        read or write past it: sizes are checked here, before any launch."""
        dt, s, r = _rank_buffers(send, recv, self.nranks, self.device, n_send, n_recv)
        status = getattr(_lib(), name)(self._h, s, r, count, DTYPES[dt], _algo(algo), _proto(proto),
                                       chunk_bytes, _stream_handle(stream, self.device))
        _check(status, name)

    def allreduce_rmsnorm(self, send, out, weight, eps=1e-6, residual=None, stream=None):
        """out[r] = RMSNorm(sum of send[0..N-1] (+ residual[r])) * weight, row by row.

        send / out / residual: N contiguous [rows, hidden] device tensors
        (residual updated in place, or None); weight: [hidden]."""
        fast = self._rmsnorm_buffers(send, out, weight, residual)
        if fast is not None:  # every check passed in one cheap pass
            dt, rows, hidden, s, o, res = fast
            status = _lib().ar_allreduce_rmsnorm(self._h, s, o, res, ctypes.c_void_p(weight.data_ptr()), rows,
                                                 hidden, float(eps), DTYPES[dt], _stream_handle(stream, self.device))
            _check(status, "ar_allreduce_rmsnorm")
            return out
        dt = _dtype_name(send[0])
        for t in list(send) + list(out) + list(residual or []) + [weight]:
            if _dtype_name(t) != dt:
                raise TypeError("all buffers must share one dtype")
        if send[0].dim() != 2:
            raise ValueError("rank buffers must be [rows, hidden]")
        rows, hidden = send[0].shape
        for what, ts in (("send", send), ("out", out), ("residual", residual or [])):
            for i, t in enumerate(ts):
                if tuple(t.shape) != (rows, hidden):
                    raise ValueError(f"{what}[{i}] has shape {tuple(t.shape)}; the call needs {(rows, hidden)}")
        if weight.numel() != hidden or not weight.is_contiguous() or not weight.is_cuda:
            raise ValueError("weight must be a contiguous device vector of `hidden` elements")
        s, o = _ptrs(send, self.nranks, self.device), _ptrs(out, self.nranks, self.device)
        res = _ptrs(residual, self.nranks, self.device) if residual is not None else None
        status = _lib().ar_allreduce_rmsnorm(self._h, s, o, res, ctypes.c_void_p(weight.data_ptr()), rows, hidden,
                                             float(eps), DTYPES[dt], _stream_handle(stream))
        _check(status, "ar_allreduce_rmsnorm")
        return out

    def _rmsnorm_buffers(self, send, out, weight, residual):
        """(dtype name, rows, hidden, pointer arrays) of a fused call whose
        buffers all pass its checks (one dtype, [rows, hidden] contiguous
        on the communicator's device, weight [hidden]), else None."""
        _torch()
        dt = _DT_NAMES.get(send[0].dtype)
        if dt is None or send[0].dim() != 2:
            return None
        dtype, shape = send[0].dtype, send[0].shape
        rows, hidden = shape
        n, dev = self.nranks, self.device
        ptrs = []
        for ts in (send, out) + ((residual,) if residual is not None else ()):
            if len(ts) != n:
                return None
            p = []
            for t in ts:
                if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
                    return None
                p.append(t.data_ptr())
            ptrs.append((ctypes.c_void_p * n)(*p))
        if (weight.dtype is not dtype or weight.numel() != hidden or weight.get_device() != dev
                or not weight.is_contiguous()):
            return None
        return dt, rows, hidden, ptrs[0], ptrs[1], ptrs[2] if residual is not None else None

    def allreduce(self, send, recv=None, algo="ring", proto="simple", chunk_bytes=0, stream=None):
        """recv[r] = sum of send[0..N-1]; recv=None runs in place."""
        recv = send if recv is None else recv
        count = send[0].numel()
        self._call("ar_allreduce", send, recv, count, algo, proto, chunk_bytes, stream, count, count)
        return recv

    def reduce_scatter(self, send, recv, algo="ring", proto="simple", chunk_bytes=0, stream=None):
        """send[i] holds N*recvcount elements; recv[r] receives slice r of the sum."""
        count = recv[0].numel()
        self._call("ar_reduce_scatter", send, recv, count, algo, proto, chunk_bytes, stream, self.nranks * count,
                   count)
        return recv

    def allgather(self, send, recv, algo="ring", proto="simple", chunk_bytes=0, stream=None):
        """recv[r] = send[0] | send[1] | ... | send[N-1]."""
        count = send[0].numel()
        self._call("ar_allgather", send, recv, count, algo, proto, chunk_bytes, stream, count,
                   self.nranks * count)
        return recv

    def check(self, stream=None):
        """Synchronize and return (status name, rank, step) of a latched error."""
        rank, step = ctypes.c_int(-1), ctypes.c_int(-1)
        st = _lib().ar_comm_check(self._h, _stream_handle(stream), ctypes.byref(rank), ctypes.byref(step))
        return STATUS.get(st, st), rank.value, step.value

    def reset(self, stream=None):
        _check(_lib().ar_comm_reset(self._h, _stream_handle(stream)), "ar_comm_reset")

    def debug_state(self, stream=None):
        """Device control block: see ar_debug_state in include/ar.h."""
        out = (ctypes.c_uint64 * 10)()
        _check(_lib().ar_debug_state(self._h, _stream_handle(stream), out, 10), "ar_debug_state")
        keys = ("timeouts", "flag_index", "seen", "awaited", "epoch_then", "tasks_done", "calls", "ticket",
                "done", "abort")
        return dict(zip(keys, list(out)))

    def debug_calls(self, max_calls=16):
        """The communicator's most recent calls (ar_debug_calls), oldest first."""
        recs = (CallRecord * max_calls)()
        n = ctypes.c_int()
        _check(_lib().ar_debug_calls(self._h, recs, max_calls, ctypes.byref(n)), "ar_debug_calls")
        names = ({v: k for k, v in OPS.items()}, {v: k for k, v in ALGOS.items()}, {v: k for k, v in PROTOS.items()},
                 {v: k for k, v in DTYPES.items()})
        out = []
        for r in recs[:n.value]:
            d = {f: getattr(r, f) for f, _ in CallRecord._fields_}
            d["op"], d["algo"], d["proto"], d["dtype"] = (names[0][r.op], names[1][r.algo], names[2][r.proto],
                                                          names[3][r.dtype])
            out.append(d)
        return out

    def inject(self, rank: int, step: int, timeout_us: int = 0):
        _check(_lib().ar_debug_inject(self._h, rank, step, timeout_us), "ar_debug_inject")


def allreduce_noalloc(send, recv=None, algo="ring", proto="simple", chunk_bytes=0, stream=None):
    """ar_allreduce_noalloc: recv[r] = sum of send[0..N-1] with N = len(send),
    on the current device, with no communicator and no device allocation
    (Simple only, at most 1 GiB per rank).  recv=None runs in place."""
    import torch

    recv = send if recv is None else recv
    n = len(send)
    count = send[0].numel()
    dev = torch.cuda.current_device()
    dt, s, r = _rank_buffers(send, recv, n, dev, count, count)
    _check(_lib().ar_allreduce_noalloc(n, s, r, count, DTYPES[dt], _algo(algo), _proto(proto), chunk_bytes,
                                       _stream_handle(stream, dev)), "ar_allreduce_noalloc")
    return recv


# ---- operators of a tensor-parallel layer ----
# Small calls are bound by this host work: pointer array types are made once,
# workspace sizes are kept by shape, checks are one pass of attribute reads.

_PTRS = [ctypes.c_void_p * n for n in range(9)]


@functools.lru_cache(maxsize=256)
def _ffn_workspace(n, rows, hidden, inter, dt, backward):
    return _lib().ar_gated_ffn_workspace(n, rows, hidden, inter, DTYPES[dt], backward)


@functools.lru_cache(maxsize=256)
def _xent_workspace(n, rows, hidden, vocab, dt, backward, piece):
    return _lib().ar_linear_cross_entropy_workspace(n, rows, hidden, vocab, DTYPES[dt], backward, piece)


def _layer_ranks(first, what):
    """(rank count, device index, dtype name) of a layer call, from its first
    list of rank tensors; the current device is the call's device."""
    n = len(first)
    if not 1 <= n <= 8:
        raise ValueError(f"{what} holds {n} rank buffers; a call has 1 to 8 ranks")
    return n, first[0].get_device(), _dtype_name(first[0])


def _layer_list(ts, n, shapes, dtype, device, what):
    """Pointer array of N rank tensors after their checks; `shapes` is one
    shape for all ranks or a list of N."""
    if len(ts) != n:
        raise ValueError(f"{what} holds {len(ts)} rank buffers; the call needs {n}")
    ptrs = []
    same = not isinstance(shapes, list)
    for i, t in enumerate(ts):
        shape = shapes if same else shapes[i]
        if t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
            if t.dtype is not dtype:
                raise TypeError(f"{what}[{i}] is {t.dtype}; the call needs {dtype}")
            if t.shape != shape:
                raise ValueError(f"{what}[{i}] has shape {tuple(t.shape)}; the call needs {tuple(shape)}")
            raise ValueError(f"{what}[{i}] must be a contiguous tensor on the call's device")
        ptrs.append(t.data_ptr())
    return _PTRS[n](*ptrs)


def _layer_vector(t, rows, dtype, device, what):
    if t.dtype is not dtype:
        raise TypeError(f"{what} is {t.dtype}; the call needs {dtype}")
    if t.dim() != 1 or t.numel() != rows or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous vector of {rows} elements on the call's device")
    return ctypes.c_void_p(t.data_ptr())


def _on_device(device, stream):
    """The call's tensors must be device tensors on the current device, and its
    stream one of that device (the workspace goes back to the device's memory
    pool of that stream)."""
    torch = _TORCH
    if device < 0:
        raise ValueError("rank buffers must be contiguous device tensors")
    if stream is not None and stream.device_index != device:
        raise ValueError("stream must be a stream of the rank buffers' device")
    if device != torch.cuda.current_device():
        raise ValueError("rank buffers must live on the current device")


class _Scratch:
    """Memory a call makes for itself (workspace, results the caller gave no
    buffers for), allocated for the stream the call runs on."""

    def __init__(self, stream, device):
        self.stream, self.device = stream, device

    def empty(self, shape, dtype):
        torch = _TORCH
        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self.stream):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def ranks(self, n, shape, dtype):
        """N rank buffers of one shape, each a tensor of its own: views of one
        allocation would keep each other alive, be saved together, and count
        as one tensor's views in autograd."""
        return [self.empty(shape, dtype) for _ in range(n)]

    def workspace(self, nbytes):
        ws = self.empty((nbytes,), _TORCH.uint8)
        return ws, ctypes.c_void_p(ws.data_ptr())


def _ffn_weights(x, w_gate, w_up, w_down):
    """(n, device, dtype, dtype name, rows, hidden, inter, pointer arrays of the four)"""
    n, device, dt = _layer_ranks(x, "x")
    dtype = x[0].dtype
    if x[0].dim() != 2:
        raise ValueError("x must be [rows, hidden] on every rank")
    rows, hidden = x[0].shape
    if len(w_gate) != n or w_gate[0].dim() != 2:
        raise ValueError(f"w_gate must be {n} matrices [inter, hidden]")
    inter = w_gate[0].shape[0]
    ptrs = [_layer_list(x, n, (rows, hidden), dtype, device, "x"),
            _layer_list(w_gate, n, (inter, hidden), dtype, device, "w_gate"),
            _layer_list(w_up, n, (inter, hidden), dtype, device, "w_up"),
            _layer_list(w_down, n, (hidden, inter), dtype, device, "w_down")]
    return n, device, dtype, dt, rows, hidden, inter, ptrs


def _act(name):
    if name not in ACTS:
        raise ValueError(f"act must be one of {', '.join(ACTS)}; got {name!r}")
    return ACTS[name]


def gated_ffn(x, w_gate, w_up, w_down, out=None, gate=None, up=None, act="silu", stream=None):
    """ar_gated_ffn: out[r] = (act(x[r] w_gate[r]^T) * (x[r] w_up[r]^T)) w_down[r]^T,
    rank r's partial sum of a gated feed-forward block split over N = len(x)
    ranks (``Comm.allreduce`` or ``Comm.allreduce_rmsnorm`` over ``out`` completes it).

    x[r]: [rows, hidden]; w_gate[r], w_up[r]: [inter, hidden]; w_down[r]:
    [hidden, inter]; out[r]: [rows, hidden], allocated when None.  gate, up:
    None, or N fp32 tensors [rows, inter] that receive the two projections for
    ``gated_ffn_backward``.  act: "silu", "gelu" or "gelu_tanh".  Runs on the
    current device; fp32 and bf16.  Every matrix is contiguous and starts on a
    16-byte boundary (rows cut out of a tensor of odd width may not: ARError
    AR_ERR_INVALID)."""
    a = _act(act)
    n, device, dtype, dt, rows, hidden, inter, ptrs = _ffn_weights(x, w_gate, w_up, w_down)
    f32 = _torch().float32
    if (gate is None) != (up is None):
        raise ValueError("gate and up are given together or not at all")
    g = _layer_list(gate, n, (rows, inter), f32, device, "gate") if gate is not None else None
    u = _layer_list(up, n, (rows, inter), f32, device, "up") if up is not None else None
    o = _layer_list(out, n, (rows, hidden), dtype, device, "out") if out is not None else None
    _on_device(device, stream)
    scratch = _Scratch(stream, device)
    if out is None:
        out = scratch.ranks(n, (rows, hidden), dtype)
        o = _PTRS[n](*[t.data_ptr() for t in out])
    nbytes = _ffn_workspace(n, rows, hidden, inter, dt, 0)
    ws, ws_ptr = scratch.workspace(nbytes)
    _check(_lib().ar_gated_ffn(n, *ptrs, o, g, u, rows, hidden, inter, a, DTYPES[dt], ws_ptr, nbytes,
                               _stream_handle(stream, device)), "ar_gated_ffn")
    return out


def gated_ffn_backward(dout, x, w_gate, w_up, w_down, gate, up, dx=None, dw_gate=None, dw_up=None, dw_down=None,
                       act="silu", stream=None):
    """ar_gated_ffn_backward: (dx, dw_gate, dw_up, dw_down), lists of N tensors.

    dout[r]: [rows, hidden], the gradient of the block's output; gate, up:
    what ``gated_ffn`` stored.  dx[r] is rank r's partial sum (``Comm.allreduce``
    completes it).  Results the caller gives no tensors for are allocated;
    given ones are overwritten."""
    a = _act(act)
    n, device, dtype, dt, rows, hidden, inter, ptrs = _ffn_weights(x, w_gate, w_up, w_down)
    f32 = _torch().float32
    d = _layer_list(dout, n, (rows, hidden), dtype, device, "dout")
    g = _layer_list(gate, n, (rows, inter), f32, device, "gate")
    u = _layer_list(up, n, (rows, inter), f32, device, "up")
    results = [("dx", dx, (rows, hidden)), ("dw_gate", dw_gate, (inter, hidden)), ("dw_up", dw_up, (inter, hidden)),
               ("dw_down", dw_down, (hidden, inter))]
    given = [_layer_list(t, n, shape, dtype, device, what) if t is not None else None for what, t, shape in results]
    _on_device(device, stream)
    scratch = _Scratch(stream, device)
    outs = []
    for i, (_, t, shape) in enumerate(results):
        if t is None:
            t = scratch.ranks(n, shape, dtype)
            given[i] = _PTRS[n](*[v.data_ptr() for v in t])
        outs.append(t)
    nbytes = _ffn_workspace(n, rows, hidden, inter, dt, 1)
    ws, ws_ptr = scratch.workspace(nbytes)
    _check(_lib().ar_gated_ffn_backward(n, d, *ptrs, g, u, *given, rows, hidden, inter, a, DTYPES[dt], ws_ptr, nbytes,
                                        _stream_handle(stream, device)), "ar_gated_ffn_backward")
    return tuple(outs)


def vocab_shards(vocab, nranks):
    """Vocabulary rows each rank holds: blocks of ceil(vocab / nranks)."""
    b = -(-vocab // nranks)
    return [min((r + 1) * b, vocab) - min(r * b, vocab) for r in range(nranks)]


def _xent_inputs(x, w, target):
    """(n, device, dtype, dtype name, rows, hidden, vocab, shards, pointers of x, w and target)"""
    torch = _torch()
    n, device, dt = _layer_ranks(x, "x")
    dtype = x[0].dtype
    if x[0].dim() != 2:
        raise ValueError("x must be [rows, hidden] on every rank")
    rows, hidden = x[0].shape
    if len(w) != n or any(t.dim() != 2 for t in w):
        raise ValueError(f"w must be {n} matrices [shard, hidden]")
    vocab = sum(t.shape[0] for t in w)
    shards = vocab_shards(vocab, n)
    ptrs = [_layer_list(x, n, (rows, hidden), dtype, device, "x"),
            _layer_list(w, n, [(v, hidden) for v in shards], dtype, device, "w"),
            _layer_vector(target, rows, torch.int64, device, "target")]
    return n, device, dtype, dt, rows, hidden, vocab, shards, ptrs


def linear_cross_entropy(x, w, target, loss=None, lse=None, stream=None):
    """ar_linear_cross_entropy: (loss, lse), lists of N fp32 vectors [rows].

    The softmax cross entropy of logits x W^T against `target`, without the
    logits, the vocabulary split over N = len(x) ranks: w[r] holds rank r's
    ``vocab_shards(vocab, N)[r]`` rows of W [vocab, hidden]; x[r]: [rows,
    hidden], the same on every rank; target: one int64 vector [rows]; rows whose
    target is outside [0, vocab) have loss 0.  Every rank receives the whole
    loss = lse - logit of the target, and lse, which the backward pass needs.
    Every matrix is contiguous and starts on a 16-byte boundary (a shard cut out of
    a W of odd width may not: ARError AR_ERR_INVALID)."""
    torch = _torch()
    n, device, _, dt, rows, hidden, vocab, _, ptrs = _xent_inputs(x, w, target)
    given = [_layer_list(t, n, (rows,), torch.float32, device, what) if t is not None else None
             for what, t in (("loss", loss), ("lse", lse))]
    _on_device(device, stream)
    scratch = _Scratch(stream, device)
    outs = []
    for i, t in enumerate((loss, lse)):
        if t is None:
            t = scratch.ranks(n, (rows,), torch.float32)
            given[i] = _PTRS[n](*[v.data_ptr() for v in t])
        outs.append(t)
    nbytes = _xent_workspace(n, rows, hidden, vocab, dt, 0, 0)
    ws, ws_ptr = scratch.workspace(nbytes)
    _check(_lib().ar_linear_cross_entropy(n, *ptrs, *given, rows, hidden, vocab, DTYPES[dt], ws_ptr, nbytes,
                                          _stream_handle(stream, device)), "ar_linear_cross_entropy")
    return tuple(outs)


def linear_cross_entropy_backward(grad_loss, x, w, target, lse, dx=None, dw=None, piece=0, stream=None):
    """ar_linear_cross_entropy_backward: (dx, dw), lists of N tensors shaped
    like x and w.

    grad_loss: fp32 vector [rows], the gradient of each row's loss; lse: what
    ``linear_cross_entropy`` returned.  dx[r] is rank r's partial sum
    (``Comm.allreduce`` completes it).  `piece`: vocabulary rows of each rank
    worked on at a time (at least 256; 0: chosen by the library), which caps the
    workspace."""
    torch = _torch()
    n, device, dtype, dt, rows, hidden, vocab, shards, ptrs = _xent_inputs(x, w, target)
    if piece < 0:
        raise ValueError("piece must not be negative")
    gl = _layer_vector(grad_loss, rows, torch.float32, device, "grad_loss")
    z = _layer_list(lse, n, (rows,), torch.float32, device, "lse")
    results = [("dx", dx, [(rows, hidden)] * n), ("dw", dw, [(v, hidden) for v in shards])]
    given = [_layer_list(t, n, shapes, dtype, device, what) if t is not None else None for what, t, shapes in results]
    _on_device(device, stream)
    scratch = _Scratch(stream, device)
    outs = []
    for i, (_, t, shapes) in enumerate(results):
        if t is None:
            t = [scratch.empty(shape, dtype) for shape in shapes]
            given[i] = _PTRS[n](*[v.data_ptr() for v in t])
        outs.append(t)
    nbytes = _xent_workspace(n, rows, hidden, vocab, dt, 1, piece)
    ws, ws_ptr = scratch.workspace(nbytes)
    _check(_lib().ar_linear_cross_entropy_backward(n, gl, *ptrs, z, *given, rows, hidden, vocab, DTYPES[dt], piece,
                                                   ws_ptr, nbytes, _stream_handle(stream, device)),
           "ar_linear_cross_entropy_backward")
    return tuple(outs)


def stream_ceiling(src, dst, sink=None, nt_loads=False, nt_stores=False, unroll=8, wg_per_cu=0, stream=None):
    """ar_stream_ceiling: one streaming pass reading every tensor of `src`
    and writing every tensor of `dst` (all contiguous device tensors of the
    same byte size; a measurement aid), plain or non-temporal."""
    tensors = list(src) + list(dst)
    nbytes = tensors[0].numel() * tensors[0].element_size()
    for t in tensors:
        if not t.is_cuda or not t.is_contiguous() or t.numel() * t.element_size() != nbytes:
            raise ValueError("streams must be contiguous device tensors of one byte size")
    s = (ctypes.c_void_p * max(1, len(src)))(*[t.data_ptr() for t in src])
    d = (ctypes.c_void_p * max(1, len(dst)))(*[t.data_ptr() for t in dst])
    _check(_lib().ar_stream_ceiling(len(src), s, len(dst), d, nbytes,
                                    ctypes.c_void_p(sink.data_ptr() if sink is not None else 0),
                                    int(nt_loads) | 2 * int(nt_stores), unroll, wg_per_cu, _stream_handle(stream)),
           "ar_stream_ceiling")


def select(nranks, op, count, dtype, algo="auto", proto="auto", max_line_bytes_per_rank=0):
    """The library's choice for a call: (algo, proto, predicted_us)."""
    a, p, t = ctypes.c_int(), ctypes.c_int(), ctypes.c_double()
    _check(_lib().ar_select(nranks, OPS[op], count, DTYPES[dtype], _algo(algo), _proto(proto),
                            max_line_bytes_per_rank, ctypes.byref(a), ctypes.byref(p), ctypes.byref(t)),
           "ar_select")
    names_a = {v: k for k, v in ALGOS.items()}
    names_p = {v: k for k, v in PROTOS.items()}
    return names_a[a.value], names_p[p.value], t.value


def plan_bytes(nranks, op, count, dtype, algo, proto, chunk_bytes=0, in_place=False):
    """Host-side byte accounting of one call (no GPU needed)."""
    rd, wr, nt = ctypes.c_uint64(), ctypes.c_uint64(), ctypes.c_uint64()
    link = (ctypes.c_uint64 * nranks)()
    _check(_lib().ar_plan_bytes(nranks, OPS[op], count, DTYPES[dtype], ALGOS[algo], PROTOS[proto],
                                chunk_bytes, int(in_place), ctypes.byref(rd), ctypes.byref(wr), link,
                                ctypes.byref(nt)), "ar_plan_bytes")
    return {"read": rd.value, "write": wr.value, "hbm": rd.value + wr.value,
            "link": list(link), "ntasks": nt.value}
