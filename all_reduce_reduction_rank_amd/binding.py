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
    qk_norm_rope(q, k, q_weight, k_weight, pos, freq)                        # + qk_norm_rope_backward
    cache = KVCache.empty(nranks, pages, kv_heads, head_dim, page=64)
    cache_write(cache, k, v, table, first, start)                            # + cache_read
    cache_attention(q, cache, table, first, length)

``send`` / ``recv`` are lists of N contiguous CUDA (HIP) tensors on the
communicator's device.  If the library is missing it is built once with hipcc;
if that fails every call raises -- there is no CPU fallback.
"""

import ctypes
import functools
import importlib
import os
import warnings

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
    "ar_qk_norm_rope", "ar_qk_norm_rope_workspace", "ar_qk_norm_rope_backward",
    "ar_cache_write", "ar_cache_read", "ar_cache_attention_workspace", "ar_cache_attention",
)


class CallRecord(ctypes.Structure):
    """ar_call_record (include/ar.h)."""
    _fields_ = [("seq", ctypes.c_uint64), ("op", ctypes.c_int32), ("algo", ctypes.c_int32),
                ("proto", ctypes.c_int32), ("dtype", ctypes.c_int32), ("nranks", ctypes.c_int32),
                ("in_place", ctypes.c_int32), ("grid", ctypes.c_uint32), ("batch", ctypes.c_uint32),
                ("counter_free", ctypes.c_uint32), ("by_die", ctypes.c_uint32), ("count", ctypes.c_uint64),
                ("ntasks", ctypes.c_uint64), ("tile_bytes", ctypes.c_uint64)]


class CacheRecord(ctypes.Structure):
    """ar_kv_cache (include/ar.h)."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("pages", ctypes.c_size_t), ("page", ctypes.c_size_t), ("kv_heads", ctypes.c_size_t),
                ("head_dim", ctypes.c_size_t), ("nranks", ctypes.c_int)]


class PagedRows(ctypes.Structure):
    """ar_paged_rows (include/ar.h)."""
    _fields_ = [("table", ctypes.c_void_p), ("first", ctypes.c_void_p), ("at", ctypes.c_void_p),
                ("table_stride", ctypes.c_size_t), ("width", ctypes.c_size_t), ("seqs", ctypes.c_size_t),
                ("rows", ctypes.c_size_t)]


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
    # (pointer arrays as ctypes arrays or as bytes)
    F, C, R = ctypes.c_float, ctypes.POINTER(CacheRecord), ctypes.POINTER(PagedRows)
    lib.ar_qk_norm_rope.argtypes = [I, P, S, P, S, P, P, P, P, P, P, S, S, S, S, S, I, F, I, P]
    lib.ar_qk_norm_rope_workspace.argtypes = [I, S, S, S, S]
    lib.ar_qk_norm_rope_backward.argtypes = ([I, P, P, P, S, P, S, P, P, P, P, P, S, P, S, P, P, S, S, S, S, S, I, F, I,
                                              P, S, P])
    lib.ar_cache_write.argtypes = [C, P, S, P, S, R, I, P]
    lib.ar_cache_read.argtypes = [C, P, P, R, I, P]
    lib.ar_cache_attention_workspace.argtypes = [C, S, S, S, S, S, S, I]
    lib.ar_cache_attention.argtypes = [C, P, S, R, P, P, S, F, I, S, S, I, P, S, P]
    lib.ar_status_string.argtypes = [I]
    lib.ar_status_string.restype = ctypes.c_char_p
    for name in SYMBOLS:
        if name.endswith("_workspace"):
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
_MARSHAL = None  # the checks of the attention operators' tensors in C++ (csrc/marshal.cpp), where built
_DT_NAMES = None  # torch dtype -> "f32" / "bf16" / "i32"


def _compiled_checks():
    """csrc/marshal.cpp's module, or None: the same checks run in Python."""
    from .build import checks_built_for
    try:
        found = importlib.import_module("._marshal", __package__)
    except ModuleNotFoundError:
        return None
    except ImportError as e:
        warnings.warn(f"_marshal.so does not load, the checks run in Python: {e}", RuntimeWarning, stacklevel=4)
        return None
    mark = getattr(found, "BUILT_FOR", "something else")
    if mark != checks_built_for():
        warnings.warn(f"_marshal.so was built for {mark}, the checks run in Python", RuntimeWarning, stacklevel=4)
        return None
    return found


def _torch():
    global _TORCH, _DT_NAMES, _MARSHAL
    if _TORCH is None:
        import torch

        _MARSHAL = _compiled_checks()
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


def _head_list(ts, n, rows, width, dtype, device, what):
    """(pointer array, stride) of N rank tensors [rows, heads, head_dim] whose
    rows are contiguous and all the same distance apart (views of a wider
    matrix are fine); `width` = (heads, head_dim) or None for the first one's."""
    if _MARSHAL is not None and width is not None and len(ts) == n:
        found = _MARSHAL.rows(ts, dtype, device, rows, *width)
        if found is not None:
            return found
    if len(ts) != n:
        raise ValueError(f"{what} holds {len(ts)} rank buffers; the call needs {n}")
    first = ts[0]
    if first.dim() != 3:
        raise ValueError(f"{what} must be [rows, heads, head_dim] on every rank")
    shape = (rows, *(width or first.shape[1:]))
    dim = shape[2]
    strides = first.stride()
    ptrs = []
    for i, t in enumerate(ts):
        if t.dtype is not dtype or t.shape != shape or t.get_device() != device or t.stride() != strides:
            if t.dtype is not dtype:
                raise TypeError(f"{what}[{i}] is {t.dtype}; the call needs {dtype}")
            if t.shape != shape:
                raise ValueError(f"{what}[{i}] has shape {tuple(t.shape)}; the call needs {tuple(shape)}")
            raise ValueError(f"{what}[{i}] must lie on the call's device with the strides of {what}[0]")
        ptrs.append(t.data_ptr())
    if rows and shape[1] and (strides[2] != 1 or (shape[1] > 1 and strides[1] != dim)):
        raise ValueError(f"{what} must have each row's heads side by side (strides {strides})")
    # (the stride of a single row is arbitrary)
    return _PTRS[n](*ptrs), strides[0] if rows > 1 else shape[1] * dim


def _rank_list(ts, n, shape, dtype, device, what):
    """``_layer_list`` of one shape, in C++ where that is built."""
    if _MARSHAL is not None and len(ts) == n:
        found = _MARSHAL.contiguous(ts, dtype, device, shape)
        if found is not None:
            return found
    return _layer_list(ts, n, shape, dtype, device, what)


def _shared_vector(t, n, dtype, device, what):
    """``_layer_vector``, in C++ where that is built."""
    if _MARSHAL is not None:
        found = _MARSHAL.vector(t, dtype, device, n)
        if found is not None:
            return found
    return _layer_vector(t, n, dtype, device, what)


def _rope_inputs(q, k, q_weight, k_weight, pos, freq):
    """(n, device, dtype, name, sizes, pointers and strides) of a qk_norm_rope call."""
    torch = _torch()
    n, device, dt = _layer_ranks(q, "q")
    dtype = q[0].dtype
    if q[0].dim() != 3:
        raise ValueError("q must be [rows, heads, head_dim] on every rank")
    rows, heads, dim = q[0].shape
    qp, qs = _head_list(q, n, rows, (heads, dim), dtype, device, "q")
    kp, ks, kw, kv = None, 0, None, 0
    if (k is None) != (k_weight is None):
        raise ValueError("k and k_weight are given together or not at all")
    if k is not None:
        kp, ks = _head_list(k, n, rows, (k[0].shape[1] if k[0].dim() == 3 else 0, dim), dtype, device, "k")
        kv = k[0].shape[1]
        kw = _shared_vector(k_weight, dim, dtype, device, "k_weight")
    rot = 0 if freq is None else 2 * freq.numel()
    if rot and pos is None:
        raise ValueError("freq needs pos")
    args = [_shared_vector(q_weight, dim, dtype, device, "q_weight"), kw,
            _shared_vector(pos, rows, torch.int64, device, "pos") if rot else None,
            _shared_vector(freq, rot // 2, torch.float32, device, "freq") if rot else None]
    return n, device, dtype, dt, (rows, heads, kv, dim, rot), (qp, qs, kp, ks), args


def qk_norm_rope(q, k, q_weight, k_weight, pos, freq, eps=1e-6, pairs=False, q_out=None, k_out=None, stream=None):
    """ar_qk_norm_rope: (q_out, k_out), lists of N = len(q) tensors: each head of
    each row over its root mean square, times its weight, its first
    2 * len(freq) values turned by the angles pos * freq (halves together, or
    with `pairs` neighbours).

    q[r]: [rows, heads, head_dim], k[r]: [rows, kv_heads, head_dim], each row's
    heads side by side (views of one projection's result are fine);
    q_weight, k_weight: [head_dim], aligned to 16 bytes; pos: int64 [rows]; freq: fp32
    [rot / 2] (None: no rotation).  k and k_weight None: queries alone, k_out is None.  q_out,
    k_out: contiguous, allocated when None.  head_dim 64, 128 or 256; fp32 and bf16."""
    n, device, dtype, dt, (rows, heads, kv, dim, rot), x, shared = _rope_inputs(q, k, q_weight, k_weight, pos, freq)
    qo = _rank_list(q_out, n, (rows, heads, dim), dtype, device, "q_out") if q_out is not None else None
    if k is None and k_out is not None:
        raise ValueError("k_out needs k")
    ko = _rank_list(k_out, n, (rows, kv, dim), dtype, device, "k_out") if k_out is not None else None
    _on_device(device, stream)
    scratch = _Scratch(stream, device)
    if qo is None:
        q_out = scratch.ranks(n, (rows, heads, dim), dtype)
        qo = _PTRS[n](*[t.data_ptr() for t in q_out])
    if ko is None and k is not None:
        k_out = scratch.ranks(n, (rows, kv, dim), dtype)
        ko = _PTRS[n](*[t.data_ptr() for t in k_out])
    _check(_lib().ar_qk_norm_rope(n, *x, *shared, qo, ko, rows, heads, kv, dim, rot, bool(pairs), eps, DTYPES[dt],
                                  _stream_handle(stream, device)), "ar_qk_norm_rope")
    return q_out, k_out


@functools.lru_cache(maxsize=256)
def _rope_workspace(n, rows, heads, kv, dim):
    return _lib().ar_qk_norm_rope_workspace(n, rows, heads, kv, dim)


def qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, pos, freq, eps=1e-6, pairs=False, dq=None, dk=None,
                          dq_weight=None, dk_weight=None, stream=None):
    """ar_qk_norm_rope_backward: (dq, dk, dq_weight, dk_weight), lists of N tensors.

    dq_out, dk_out: the gradients of ``qk_norm_rope``'s results, contiguous; the
    rest as there.  dq, dk may be views of one matrix (the projection's gradient).
    dq_weight[r], dk_weight[r] are rank r's partial sums (``Comm.allreduce``
    completes them).  Results the caller gives no tensors for are allocated;
    given ones are overwritten."""
    n, device, dtype, dt, (rows, heads, kv, dim, rot), x, shared = _rope_inputs(q, k, q_weight, k_weight, pos, freq)
    if k is None and not dk_out is dk is dk_weight is None:
        raise ValueError("dk_out, dk and dk_weight need k")
    go = [_rank_list(dq_out, n, (rows, heads, dim), dtype, device, "dq_out"),
          _rank_list(dk_out, n, (rows, kv, dim), dtype, device, "dk_out") if k is not None else None]
    given = [_head_list(dq, n, rows, (heads, dim), dtype, device, "dq") if dq is not None else None,
             _head_list(dk, n, rows, (kv, dim), dtype, device, "dk") if dk is not None else None]
    sums = [_rank_list(t, n, (dim,), dtype, device, what) if t is not None else None
            for what, t in (("dq_weight", dq_weight), ("dk_weight", dk_weight))]
    _on_device(device, stream)
    scratch = _Scratch(stream, device)
    outs, weights = [dq, dk], [dq_weight, dk_weight]
    for i, width in enumerate((heads, kv)):
        if i == 1 and k is None:
            given[i] = (None, 0)
            continue
        if given[i] is None:
            outs[i] = scratch.ranks(n, (rows, width, dim), dtype)
            given[i] = (_PTRS[n](*[t.data_ptr() for t in outs[i]]), width * dim)
        if sums[i] is None:
            weights[i] = scratch.ranks(n, (dim,), dtype)
            sums[i] = _PTRS[n](*[t.data_ptr() for t in weights[i]])
    nbytes = _rope_workspace(n, rows, heads, kv, dim)
    ws, ws_ptr = scratch.workspace(nbytes)
    _check(_lib().ar_qk_norm_rope_backward(n, *go, *x, *shared, *given[0], *given[1], *sums, rows, heads, kv, dim, rot,
                                           bool(pairs), eps, DTYPES[dt], ws_ptr, nbytes, _stream_handle(stream, device)),
           "ar_qk_norm_rope_backward")
    return outs[0], outs[1], weights[0], weights[1]


class KVCache:
    """ar_kv_cache: the 8-bit key/value cache of N ranks, held as lists of N
    uint8 tensors: ``k`` [pages, kv_heads, page, head_dim] and ``v`` [pages,
    kv_heads, head_dim, page] (e4m3 codes), ``k_scale`` and ``v_scale`` [pages,
    kv_heads] (a code c stands for value(c) * 2^(scale - 127)).

    ``KVCache(k, v, k_scale, v_scale)`` takes tensors of the caller's;
    ``KVCache.empty(nranks, pages, kv_heads, head_dim, page=64)`` allocates
    them on the current device (contents unset: a page counts from its first
    write on)."""

    def __init__(self, k, v, k_scale, v_scale):
        torch = _torch()
        n = len(k)
        if not 1 <= n <= 8:
            raise ValueError(f"k holds {n} rank buffers; a cache has 1 to 8 ranks")
        if k[0].dim() != 4:
            raise ValueError("k must be [pages, kv_heads, page, head_dim] on every rank")
        pages, kv, page, dim = k[0].shape
        self.device = k[0].get_device()
        self.nranks, self.pages, self.kv_heads, self.page, self.head_dim = n, pages, kv, page, dim
        self.k, self.v, self.k_scale, self.v_scale = tuple(k), tuple(v), tuple(k_scale), tuple(v_scale)
        shapes = (("k", self.k, (pages, kv, page, dim)), ("v", self.v, (pages, kv, dim, page)),
                  ("k_scale", self.k_scale, (pages, kv)), ("v_scale", self.v_scale, (pages, kv)))
        # kept alive beside the record, which holds their addresses
        self._ptrs = [_layer_list(ts, n, shape, torch.uint8, self.device, what) for what, ts, shape in shapes]
        self.record = CacheRecord(*[ctypes.cast(p, ctypes.c_void_p) for p in self._ptrs], pages, page, kv, dim, n)

    @classmethod
    def empty(cls, nranks, pages, kv_heads, head_dim, page=64):
        torch = _torch()

        def make(*shape):
            return [torch.empty(shape, dtype=torch.uint8, device="cuda") for _ in range(nranks)]
        return cls(make(pages, kv_heads, page, head_dim), make(pages, kv_heads, head_dim, page), make(pages, kv_heads),
                   make(pages, kv_heads))


def _paged_rows(cache, table, first, at, rows, what):
    """ar_paged_rows of a call's sequences."""
    if _MARSHAL is not None:
        found = _MARSHAL.sequences(table, first, at, cache.device)
        if found is not None:
            return PagedRows(*found, rows)
    torch = _TORCH
    for name, t, dim in (("table", table, 2), ("first", first, 1), (what, at, 1)):
        if t.dtype is not torch.int32:
            raise TypeError(f"{name} is {t.dtype}; the call needs {torch.int32}")
        if t.dim() != dim or t.get_device() != cache.device or (t.stride(-1) != 1 and t.shape[-1] > 1):
            raise ValueError(f"{name} must be an int32 tensor of {dim} dimension{'s' * (dim > 1)} on the cache's device, its last one contiguous")
    seqs, width = table.shape
    if first.shape[0] != seqs + 1 or at.shape[0] != seqs:
        raise ValueError(f"table names {seqs} sequences, so first has {seqs + 1} entries and {what} {seqs}; "
                         f"got {first.shape[0]} and {at.shape[0]}")
    stride = table.stride(0) if seqs > 1 else width
    if stride < width:
        raise ValueError("table must not repeat or overlap its rows")
    return PagedRows(table.data_ptr(), first.data_ptr(), at.data_ptr(), stride, width, seqs, rows)


def cache_write(cache, k, v, table, first, start, stream=None):
    """ar_cache_write: stores new keys and values in the cache's pages.

    k[r], v[r]: [rows, kv_heads, head_dim], each row's heads side by side (views
    of one projection's result are fine); table: int32 [seqs, width], the pages
    of each sequence in order (a view of a wider table is fine); first: int32
    [seqs + 1], sequence s has the rows first[s] .. first[s + 1] - 1; start:
    int32 [seqs], the position of its first row.  fp32 and bf16.  A page must
    belong to one sequence of the call; one that grows may change its scale,
    which rounds its smallest earlier values again."""
    n, device, dt = _layer_ranks(k, "k")
    _cache_ranks(cache, n, device, "k")
    if k[0].dim() != 3:
        raise ValueError("k must be [rows, kv_heads, head_dim] on every rank")
    rows, width, dtype = k[0].shape[0], (cache.kv_heads, cache.head_dim), k[0].dtype
    kp, ks = _head_list(k, n, rows, width, dtype, device, "k")
    vp, vs = _head_list(v, n, rows, width, dtype, device, "v")
    paged = _paged_rows(cache, table, first, start, rows, "start")
    _on_device(device, stream)
    _check(_lib().ar_cache_write(cache.record, kp, ks, vp, vs, paged, DTYPES[dt], _stream_handle(stream, device)),
           "ar_cache_write")


def _cache_ranks(cache, n, device, what):
    if n != cache.nranks:
        raise ValueError(f"{what} holds {n} rank buffers; the cache has {cache.nranks}")
    if device != cache.device:
        raise ValueError(f"{what} and the cache must live on one device")


def cache_read(cache, table, first, start, k, v, stream=None):
    """ar_cache_read: (k, v) filled with tokens read back from the cache.

    k[r], v[r]: contiguous [rows, kv_heads, head_dim], fp32 or bf16 (exact but at
    the ends of the range, ar.h); rows first[s] .. first[s + 1] - 1 receive the tokens of sequence s from
    position start[s] on, zeros where the table names no page."""
    n, device, dt = _layer_ranks(k, "k")
    _cache_ranks(cache, n, device, "k")
    if k[0].dim() != 3:
        raise ValueError("k must be [rows, kv_heads, head_dim] on every rank")
    shape, dtype = (k[0].shape[0], cache.kv_heads, cache.head_dim), k[0].dtype
    kp = _rank_list(k, n, shape, dtype, device, "k")
    vp = _rank_list(v, n, shape, dtype, device, "v")
    paged = _paged_rows(cache, table, first, start, shape[0], "start")
    _on_device(device, stream)
    _check(_lib().ar_cache_read(cache.record, kp, vp, paged, DTYPES[dt], _stream_handle(stream, device)), "ar_cache_read")
    return k, v


@functools.lru_cache(maxsize=1024)
def _attention_workspace(n, pages, page, kv, dim, seqs, rows, width, heads, window, max_rows, dt):
    ptr = ctypes.cast(_PTRS[n](*[16] * n), ctypes.c_void_p)  # the sizes do not depend on the buffers
    rec = CacheRecord(ptr, ptr, ptr, ptr, pages, page, kv, dim, n)
    return _lib().ar_cache_attention_workspace(rec, seqs, rows, width, heads, window, max_rows, DTYPES[dt])


def cache_attention(q, cache, table, first, length, scale=None, causal=True, window=0, max_rows=0, out=None, lse=None,
                    stream=None):
    """ar_cache_attention: out[r] = softmax(scale q k^T) v over the cache, lists
    of N tensors [rows, heads, head_dim].

    q[r]: [rows, heads, head_dim], each row's heads side by side; heads a
    multiple of the cache's kv_heads (head h reads key/value head
    h // (heads // kv_heads)); table, first as for ``cache_write``; length:
    int32 [seqs], the cached tokens of each sequence, those of its own rows
    among them: the last row stands at position length - 1.  causal False:
    every row sees all of them (an encoder's states).  window: with causal, a row
    sees the last `window` positions up to its own (0: all).  scale: 1 /
    sqrt(head_dim) when None.  max_rows: the rows the longest sequence is expected to
    have (0: the mean of the call counts); it chooses the kernel, and with bf16 whether the
    softmax weights enter the product with v in two bf16 terms (up to 96 rows of a key
    head) or in one.  lse: None, or N fp32 tensors
    [rows, heads] that receive the log of the softmax denominators.  Rows that
    see nothing have out 0 and lse minus infinity."""
    n, device, dt = _layer_ranks(q, "q")
    _cache_ranks(cache, n, device, "q")
    dtype = q[0].dtype
    if q[0].dim() != 3:
        raise ValueError("q must be [rows, heads, head_dim] on every rank")
    rows, heads, dim = q[0].shape
    qp, qs = _head_list(q, n, rows, (heads, cache.head_dim), dtype, device, "q")
    if heads < 1 or heads % cache.kv_heads:
        raise ValueError(f"heads must be a multiple of the cache's {cache.kv_heads} kv_heads; got {heads}")
    if window < 0 or max_rows < 0:
        raise ValueError("window and max_rows must not be negative")
    if window and not causal:
        raise ValueError("window needs causal")
    op = _rank_list(out, n, (rows, heads, dim), dtype, device, "out") if out is not None else None
    lp = _rank_list(lse, n, (rows, heads), _TORCH.float32, device, "lse") if lse is not None else None
    paged = _paged_rows(cache, table, first, length, rows, "length")
    _on_device(device, stream)
    scratch = _Scratch(stream, device)
    if out is None:
        out = scratch.ranks(n, (rows, heads, dim), dtype)
        op = _PTRS[n](*[t.data_ptr() for t in out])
    nbytes = _attention_workspace(n, cache.pages, cache.page, cache.kv_heads, dim, paged.seqs, rows, paged.width, heads,
                                  window, max_rows, dt)
    ws, ws_ptr = scratch.workspace(nbytes) if nbytes else (None, None)
    _check(_lib().ar_cache_attention(cache.record, qp, qs, paged, op, lp, heads,
                                     dim ** -0.5 if scale is None else scale, bool(causal), window, max_rows, DTYPES[dt],
                                     ws_ptr, nbytes, _stream_handle(stream, device)), "ar_cache_attention")
    return out


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
