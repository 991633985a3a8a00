"""Python binding of the simulated-communicator library ``libsimcomm.so`` (C ABI: include/simcomm.h).

Argument marshalling only: tensors become device pointers and the current CUDA stream becomes the
stream handle; every step of every collective runs in the library's CUDA kernels. There is no
fallback: without the built library (``python -m collective_communication_primitives_b200.build``)
creating a communicator raises.
"""
import ctypes
import math
import os
import struct

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsimcomm.so")

STATUS = {0: "COLL_OK", 1: "COLL_ERR_INVALID_ARG", 2: "COLL_ERR_UNSUPPORTED", 3: "COLL_ERR_CUDA",
          4: "COLL_ERR_TIMEOUT", 5: "COLL_ERR_ABORTED", 6: "COLL_ERR_OVERFLOW", 7: "COLL_ERR_INTERNAL"}
OK, INVALID_ARG, UNSUPPORTED, CUDA, TIMEOUT, ABORTED, OVERFLOW, INTERNAL = range(8)
DTYPES = {"int32": 0, "fp32": 1, "bf16": 2}
OPS = {"sum": 0, "min": 1, "max": 2, "avg": 3}
ALGOS = {"direct": 0, "ring": 1, "rd": 2, "hd": 3, "tree": 4, "dbtree": 5, "ll": 6, "rd_ll": 7, "tree_ll": 8,
         "dbtree_ll": 9}

PARALLEL = {"column": 0, "row": 1}

_lib = None


class SimCommError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


class _Bufs(ctypes.Structure):
    _fields_ = [("send", ctypes.POINTER(ctypes.c_void_p)), ("recv", ctypes.POINTER(ctypes.c_void_p))]


class IpcHandle(ctypes.Structure):
    """sim_ipc_handle_t: 64 opaque bytes naming a shareable device buffer."""
    _fields_ = [("reserved", ctypes.c_ubyte * 64)]


class TraceRecord(ctypes.Structure):
    """sim_comm_trace_record_t: one traced call."""
    _fields_ = [("seq", ctypes.c_ulonglong), ("coll", ctypes.c_char_p), ("p", ctypes.c_int), ("dtype", ctypes.c_int),
                ("op", ctypes.c_int), ("root", ctypes.c_int), ("algo", ctypes.c_int), ("status", ctypes.c_int),
                ("n", ctypes.c_ulonglong), ("launches", ctypes.c_uint), ("device_ms", ctypes.c_float)]


def load_library(path=LIB_PATH):
    """Load libsimcomm.so and declare its signatures. Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m collective_communication_primitives_b200.build`"
                           " (there is no fallback path)")
    L = ctypes.CDLL(path)
    vp, sz, i32, ll = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_longlong
    llp = ctypes.POINTER(ctypes.c_longlong)
    st = ctypes.c_int
    L.sim_comm_create.argtypes = [i32]
    L.sim_comm_create.restype = vp
    L.sim_comm_create_rank.argtypes = [i32, i32]
    L.sim_comm_create_rank.restype = vp
    L.sim_comm_rank.argtypes = [vp]
    L.sim_comm_rank.restype = i32
    L.sim_ipc_alloc.argtypes = [sz, ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(IpcHandle)]
    L.sim_ipc_free.argtypes = [vp]
    L.sim_ipc_open.argtypes = [ctypes.POINTER(IpcHandle), ctypes.POINTER(ctypes.c_void_p)]
    L.sim_ipc_close.argtypes = [vp]
    for name in ("sim_ipc_alloc", "sim_ipc_free", "sim_ipc_open", "sim_ipc_close"):
        getattr(L, name).restype = ctypes.c_int
    L.sim_comm_destroy.argtypes = [vp]
    L.sim_comm_destroy.restype = st
    L.sim_comm_size.argtypes = [vp]
    L.sim_comm_size.restype = i32
    L.sim_comm_last_error.argtypes = []
    L.sim_comm_last_error.restype = ctypes.c_char_p
    L.coll_status_string.argtypes = [st]
    L.coll_status_string.restype = ctypes.c_char_p
    L.sim_comm_set_option.argtypes = [vp, ctypes.c_char_p, ll]
    L.sim_comm_set_option.restype = st
    L.sim_comm_get_option.argtypes = [vp, ctypes.c_char_p, llp]
    L.sim_comm_get_option.restype = st
    L.sim_comm_get_async_error.argtypes = [vp, ctypes.POINTER(ctypes.c_int)]
    L.sim_comm_get_async_error.restype = st
    L.sim_comm_abort.argtypes = [vp]
    L.sim_comm_abort.restype = st
    L.sim_comm_reset.argtypes = [vp]
    L.sim_comm_reset.restype = st
    L.sim_comm_launch_count.argtypes = [vp, ctypes.POINTER(ctypes.c_ulonglong)]
    L.sim_comm_launch_count.restype = st
    L.sim_comm_trace_read.argtypes = [vp, ctypes.POINTER(TraceRecord), i32, ctypes.POINTER(ctypes.c_int)]
    L.sim_comm_trace_read.restype = st
    L.coll_allreduce.argtypes = [vp, _Bufs, sz, i32, i32, i32, vp]
    L.coll_reduce.argtypes = [vp, _Bufs, sz, i32, i32, i32, i32, vp]
    L.coll_broadcast.argtypes = [vp, _Bufs, sz, i32, i32, i32, vp]
    L.coll_reduce_scatter.argtypes = [vp, _Bufs, sz, i32, i32, i32, vp]
    L.coll_allgather.argtypes = [vp, _Bufs, sz, i32, i32, vp]
    L.coll_alltoall.argtypes = [vp, _Bufs, sz, i32, i32, vp]
    L.coll_alltoallv.argtypes = [vp, _Bufs, vp, llp, llp, i32, i32, vp, vp]
    L.coll_scatter.argtypes = [vp, _Bufs, sz, i32, i32, i32, vp]
    L.coll_gather.argtypes = [vp, _Bufs, sz, i32, i32, i32, vp]
    L.coll_allreduce_ring_noalloc.argtypes = [i32, _Bufs, sz, i32, i32, vp, vp]
    L.sim_hbm_probe.argtypes = [i32, vp, vp, sz, i32, vp]
    pp = ctypes.POINTER(ctypes.c_void_p)
    L.coll_moe_dispatch.argtypes = [vp, pp, pp, sz, i32, sz, i32, i32, pp, sz, pp, vp, vp, vp]
    L.coll_moe_combine.argtypes = [vp, pp, sz, pp, pp, pp, pp, sz, i32, sz, i32, i32, pp, vp]
    pa = vp  # a HOST array of pointers, given as the bytes of SimComm._tensors
    L.coll_moe_route.argtypes = [vp, pa, sz, i32, i32, i32, i32, pa, pa, vp]
    L.coll_moe_route_backward.argtypes = [vp, pa, pa, pa, sz, i32, i32, i32, i32, pa, vp]
    L.coll_linear_w4.argtypes = [vp, pa, pa, pa, sz, sz, sz, i32, i32, i32, pa, vp]
    L.coll_moe_layer.argtypes = [vp, pa, pa, pa, pa, sz, i32, sz, sz, i32, i32, i32, pa, pa, pa, pa, i32, pa, vp]
    L.coll_logprobs.argtypes = [vp, pa, sz, vp, sz, sz, i32, pa, pa, pa, i32, pa, pa, vp]
    L.coll_logprobs_backward.argtypes = [vp, pa, sz, vp, sz, sz, i32, pa, pa, vp, vp, pa, sz, vp]
    for name in ("coll_moe_route", "coll_moe_route_backward", "coll_linear_w4", "coll_moe_layer", "coll_logprobs",
                 "coll_logprobs_backward"):
        getattr(L, name).restype = st
    for name in ("coll_allreduce", "coll_reduce", "coll_broadcast", "coll_reduce_scatter", "coll_allgather",
                 "coll_alltoall", "coll_alltoallv", "coll_scatter", "coll_gather", "coll_allreduce_ring_noalloc",
                 "coll_moe_dispatch", "coll_moe_combine", "sim_hbm_probe"):
        getattr(L, name).restype = st
    _lib = L
    return L


def _ptr(x):
    """Device address of a tensor (or an int address, or None -> NULL)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


_NAMES = {}  # torch's types, once torch is there


def _dtype_of(t):
    if not _NAMES:
        import torch
        _NAMES.update({torch.int32: "int32", torch.float32: "fp32", torch.bfloat16: "bf16"})
    if t.dtype not in _NAMES:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return _NAMES[t.dtype]


def _stream(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


class SimComm:
    """A communicator of p logical ranks on the current CUDA device (or, with `rank`, the rank view
    that the process of that rank holds when every rank is its own process)."""

    def __init__(self, p, rank=None):
        self._L = load_library()
        h = self._L.sim_comm_create(int(p)) if rank is None else self._L.sim_comm_create_rank(int(p), int(rank))
        if not h:
            raise SimCommError(CUDA if rank is None else INVALID_ARG, self._L.sim_comm_last_error().decode())
        self._h = ctypes.c_void_p(h)
        self.p = int(p)
        self.rank = None if rank is None else int(rank)
        import torch
        self._torch = torch
        self._device = torch.cuda.current_device()
        self._pack = struct.Struct(f"{self.p}P").pack

    # -- lifecycle ---------------------------------------------------------------------------------
    def close(self):
        if getattr(self, "_h", None):
            self._L.sim_comm_destroy(self._h)
            self._h = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check(self, status):
        if status != OK:
            raise SimCommError(status, self._L.sim_comm_last_error().decode())

    def set_option(self, key, value):
        self._check(self._L.sim_comm_set_option(self._h, key.encode(), int(value)))

    def get_option(self, key):
        v = ctypes.c_longlong()
        self._check(self._L.sim_comm_get_option(self._h, key.encode(), ctypes.byref(v)))
        return v.value

    def async_error(self):
        s = ctypes.c_int()
        self._check(self._L.sim_comm_get_async_error(self._h, ctypes.byref(s)))
        return s.value

    def abort(self):
        self._check(self._L.sim_comm_abort(self._h))

    def reset(self):
        self._check(self._L.sim_comm_reset(self._h))

    def launch_count(self):
        v = ctypes.c_ulonglong()
        self._check(self._L.sim_comm_launch_count(self._h, ctypes.byref(v)))
        return v.value

    def trace_read(self, cap=4096):
        """The traced calls not read yet (option "trace" = 1), oldest first, as dicts with the fields of
        sim_comm_trace_record_t (coll decoded to str). Waits for their events."""
        buf = (TraceRecord * cap)()
        got = ctypes.c_int()
        self._check(self._L.sim_comm_trace_read(self._h, buf, cap, ctypes.byref(got)))
        out = []
        for r in buf[:got.value]:
            d = {name: getattr(r, name) for name, _ in TraceRecord._fields_}
            d["coll"] = d["coll"].decode()
            out.append(d)
        return out

    # -- marshalling -------------------------------------------------------------------------------
    def _bufs(self, sends, recvs):
        p = self.p
        s = (ctypes.c_void_p * p)(*[_ptr(x) for x in sends])
        r = (ctypes.c_void_p * p)(*[_ptr(x) for x in recvs])
        self._keep = (s, r)
        return _Bufs(ctypes.cast(s, ctypes.POINTER(ctypes.c_void_p)), ctypes.cast(r, ctypes.POINTER(ctypes.c_void_p)))

    @staticmethod
    def _resolve(dtype, tensors):
        if dtype is not None:
            return DTYPES[dtype]
        for t in tensors:
            if t is not None and not isinstance(t, int):
                return DTYPES[_dtype_of(t)]
        raise ValueError("dtype is needed when only raw pointers are given")

    # -- collectives (n follows include/simcomm.h: the per-rank FULL buffer) -----------------------
    def allreduce(self, sends, recvs, op="sum", algo="direct", n=None, dtype=None, stream=None):
        n = sends[0].numel() if n is None else n
        self._check(self._L.coll_allreduce(self._h, self._bufs(sends, recvs), n, self._resolve(dtype, list(sends) + list(recvs)),
                                           OPS[op], ALGOS[algo], _stream(stream)))

    def reduce(self, sends, recvs, root, op="sum", algo="direct", n=None, dtype=None, stream=None):
        n = sends[0].numel() if n is None else n
        self._check(self._L.coll_reduce(self._h, self._bufs(sends, recvs), n, self._resolve(dtype, list(sends) + list(recvs)), OPS[op],
                                        int(root), ALGOS[algo], _stream(stream)))

    def broadcast(self, sends, recvs, root, algo="direct", n=None, dtype=None, stream=None):
        n = recvs[0].numel() if n is None else n
        self._check(self._L.coll_broadcast(self._h, self._bufs(sends, recvs), n, self._resolve(dtype, list(sends) + list(recvs)),
                                           int(root), ALGOS[algo], _stream(stream)))

    def reduce_scatter(self, sends, recvs, op="sum", algo="direct", n=None, dtype=None, stream=None):
        n = sends[0].numel() if n is None else n
        self._check(self._L.coll_reduce_scatter(self._h, self._bufs(sends, recvs), n, self._resolve(dtype, list(sends) + list(recvs)),
                                                OPS[op], ALGOS[algo], _stream(stream)))

    def allgather(self, sends, recvs, algo="direct", n=None, dtype=None, stream=None):
        n = recvs[0].numel() if n is None else n
        self._check(self._L.coll_allgather(self._h, self._bufs(sends, recvs), n, self._resolve(dtype, list(sends) + list(recvs)),
                                           ALGOS[algo], _stream(stream)))

    def alltoall(self, sends, recvs, algo="direct", n=None, dtype=None, stream=None):
        n = sends[0].numel() if n is None else n
        self._check(self._L.coll_alltoall(self._h, self._bufs(sends, recvs), n, self._resolve(dtype, list(sends) + list(recvs)),
                                          ALGOS[algo], _stream(stream)))

    def scatter(self, sends, recvs, root, algo="direct", n=None, dtype=None, stream=None):
        """n: the root's full buffer (p blocks); only sends[root] is read."""
        n = sends[root].numel() if n is None else n
        self._check(self._L.coll_scatter(self._h, self._bufs(sends, recvs), n,
                                         self._resolve(dtype, list(sends) + list(recvs)), int(root), ALGOS[algo],
                                         _stream(stream)))

    def gather(self, sends, recvs, root, algo="direct", n=None, dtype=None, stream=None):
        """n: the root's full buffer (p blocks); only recvs[root] is written."""
        n = recvs[root].numel() if n is None else n
        self._check(self._L.coll_gather(self._h, self._bufs(sends, recvs), n,
                                        self._resolve(dtype, list(sends) + list(recvs)), int(root), ALGOS[algo],
                                        _stream(stream)))

    def alltoallv(self, sends, recvs, counts, send_cap=None, recv_cap=None, algo="direct", recv_counts=None,
                  dtype=None, stream=None):
        """counts: device int64 [p][p] tensor (c[i][j] elements from i to j). Capacities default to the
        buffers' sizes."""
        p = self.p
        send_cap = [sends[i].numel() for i in range(p)] if send_cap is None else send_cap
        recv_cap = [recvs[j].numel() for j in range(p)] if recv_cap is None else recv_cap
        sc = (ctypes.c_longlong * p)(*[int(x) for x in send_cap])
        rc = (ctypes.c_longlong * p)(*[int(x) for x in recv_cap])
        self._check(self._L.coll_alltoallv(self._h, self._bufs(sends, recvs), ctypes.c_void_p(_ptr(counts)), sc, rc,
                                           self._resolve(dtype, list(sends) + list(recvs)), ALGOS[algo], _stream(stream),
                                           ctypes.c_void_p(_ptr(recv_counts)) if recv_counts is not None else None))

    # -- MoE dispatch / combine ----------------------------------------------------------------------
    def _parr(self, tensors):
        """HOST array of p device pointers (None when tensors is None)."""
        if tensors is None:
            return None
        a = (ctypes.c_void_p * self.p)(*[_ptr(t) for t in tensors])
        self._keep_moe = getattr(self, "_keep_moe", [])[-16:] + [a]
        return ctypes.cast(a, ctypes.POINTER(ctypes.c_void_p))

    def moe_dispatch(self, x, topk_idx, experts, recv, route_pos=None, expert_counts=None, recv_counts=None,
                     dtype=None, stream=None):
        """x[i]: [T][H] token rows; topk_idx[i]: [T][k] int32 expert ids; recv[j]: [cap][H]. Optional
        outputs: route_pos[i] [T][k] int32, expert_counts [p][E] int64, recv_counts [p] int64."""
        T, k = topk_idx[0].shape
        H = x[0].shape[1] if x[0].dim() == 2 else x[0].numel() // max(T, 1)
        cap = recv[0].shape[0]
        self._check(self._L.coll_moe_dispatch(
            self._h, self._parr(x), self._parr(topk_idx), T, k, H, int(experts),
            self._resolve(dtype, list(x) + list(recv)), self._parr(recv), cap, self._parr(route_pos),
            ctypes.c_void_p(_ptr(expert_counts)) if expert_counts is not None else None,
            ctypes.c_void_p(_ptr(recv_counts)) if recv_counts is not None else None, _stream(stream)))

    def moe_combine(self, y, topk_idx, route_pos, topk_weight, experts, out, residual=None, dtype=None,
                    stream=None):
        """out[i][t] = residual[i][t] + Σ_s w[i][t][s] * y[owner][route_pos[i][t][s]] (fp32, slot order)."""
        T, k = topk_idx[0].shape
        H = out[0].shape[1]
        self._check(self._L.coll_moe_combine(
            self._h, self._parr(y), y[0].shape[0], self._parr(topk_idx), self._parr(route_pos),
            self._parr(topk_weight), self._parr(residual), T, k, H, int(experts),
            self._resolve(dtype, list(y) + list(out)), self._parr(out), _stream(stream)))


    # -- router, products with sharded weights, log probabilities ------------------------------------
    def _tensors(self, what, tensors, dtype, shape, row=None, one=False):
        """HOST array of the ranks' device pointers (its bytes), after checking that every tensor is where and what
        the kernels take it for: on the communicator's device, of `dtype` (a torch dtype) and `shape`, or flat
        with as many elements (a whole number: so many of any shape), contiguous (or, with `row` = (ld,
        columns), rows at that distance). A rank view's entries of other ranks may be None or addresses.
        `one`: a single tensor, its address."""
        if tensors is None:
            return None
        dev = self._device
        vector = isinstance(shape, int)
        if not one:
            try:  # the usual call in one sweep; anything else takes the slow way, which says what is wrong
                if vector:
                    out = [t.data_ptr() for t in tensors
                           if t.dtype is dtype and t.get_device() == dev and t.numel() == shape and t.is_contiguous()]
                else:
                    out = [t.data_ptr() for t in tensors
                           if t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous()]
            except AttributeError:
                out = ()
            if len(out) == self.p == len(tensors) and (row is None or row[0] == row[1]):
                return self._pack(*out)
        out, numel = [], shape if vector else math.prod(shape)
        for t in ((tensors,) if one else tensors):
            if t is None or isinstance(t, int):
                if self.rank is None:
                    raise TypeError(f"{what}: a tensor for every rank is needed")
                out.append(t or 0)
                continue
            if t.dtype is not dtype:
                raise TypeError(f"{what}: {t.dtype}, not {dtype}")
            if t.get_device() != dev:
                raise ValueError(f"{what}: on {t.device}, not on the communicator's device")
            if t.numel() != numel or not (vector or t.shape == shape or t.dim() == 1 and row is None):
                raise ValueError(f"{what}: shape {tuple(t.shape)}, {shape} is wanted")
            if row is not None and t.shape[0] > 1:
                if t.stride(1) != 1 or t.stride(0) != row[0]:
                    raise ValueError(f"{what}: strides {t.stride()} do not fit the call")
            elif not t.is_contiguous():
                raise ValueError(f"{what}: not contiguous")
            out.append(t.data_ptr())
        if one:
            return out[0]
        if len(out) != self.p:
            raise ValueError(f"{what}: {len(out)} entries for {self.p} ranks")
        return self._pack(*out)

    def _launch_stream(self, stream):
        """The stream's handle; by default the current stream of the communicator's device."""
        if stream is None:
            return self._torch._C._cuda_getCurrentRawStream(self._device)
        return stream if isinstance(stream, int) else stream.cuda_stream

    def _own(self, tensors):
        """A tensor of this handle's own ranks, whose shape and type stand for all."""
        return tensors[0 if self.rank is None else self.rank]

    def moe_route(self, logits, topk_idx, topk_weight, normalise=True, stream=None):
        """Softmax over logits[i] [T][E] (fp32 or bf16), the k best experts of every token into topk_idx[i]
        [T][k] int32 and their weights (shares of the k when `normalise`) into topk_weight[i] [T][k] fp32:
        what moe_dispatch, moe_combine and moe_layer take."""
        torch = self._torch
        x = self._own(logits)
        T, E = x.shape
        k = self._own(topk_idx).shape[1]
        self._check(self._L.coll_moe_route(
            self._h, self._tensors("logits", logits, x.dtype, (T, E)), T, k, E, DTYPES[_dtype_of(x)], 1 if normalise else 0,
            self._tensors("topk_idx", topk_idx, torch.int32, (T, k)),
            self._tensors("topk_weight", topk_weight, torch.float32, (T, k)), self._launch_stream(stream)))

    def moe_route_backward(self, logits, topk_idx, grad_weight, grad_logits, normalise=True, stream=None):
        """Gradient of moe_route's scores into grad_logits[i] [T][E] (of the scores' type), from grad_weight[i]
        [T][k] fp32, the gradient of its weights."""
        torch = self._torch
        x = self._own(logits)
        T, E = x.shape
        k = self._own(topk_idx).shape[1]
        self._check(self._L.coll_moe_route_backward(
            self._h, self._tensors("logits", logits, x.dtype, (T, E)),
            self._tensors("topk_idx", topk_idx, torch.int32, (T, k)),
            self._tensors("grad_weight", grad_weight, torch.float32, (T, k)), T, k, E, DTYPES[_dtype_of(x)],
            1 if normalise else 0, self._tensors("grad_logits", grad_logits, x.dtype, (T, E)), self._launch_stream(stream)))

    def linear_w4(self, x, w, scale, out, parallel="row", stream=None):
        """out = x W^T for few tokens, W of 4-bit weights (q - 8) * scale: w[r] uint8 [N_r][K_r/2] (element 2i in
        the low half of byte i), scale[r] bf16 [N_r][K_r/group], x[r] bf16 [T][K_r]. parallel "column": the
        ranks hold rows of W and out[r] is [T][N/p]; "row": they hold columns, the partial products are summed
        and every out[r] is [T][N]. out fp32 or bf16."""
        torch = self._torch
        if parallel not in PARALLEL:
            raise ValueError(f"parallel must be one of {sorted(PARALLEL)}")
        o = self._own(out)
        T, K = self._own(x).shape
        N = self._own(w).shape[0]
        groups = self._own(scale).shape[1]
        if groups < 1 or K % groups:
            raise ValueError(f"scale: {groups} groups do not divide rows of {K}")
        row = parallel == "row"
        self._check(self._L.coll_linear_w4(
            self._h, self._tensors("x", x, torch.bfloat16, (T, K)), self._tensors("w", w, torch.uint8, (N, K // 2)),
            self._tensors("scale", scale, torch.bfloat16, (N, groups)), T, N if row else N * self.p,
            K * self.p if row else K, K // groups, PARALLEL[parallel], DTYPES[_dtype_of(o)],
            self._tensors("out", out, o.dtype, (T, N)), self._launch_stream(stream)))

    def moe_layer(self, x, topk_idx, topk_weight, experts, w_up, w_down, out, up_scale=None, down_scale=None,
                  residual=None, stream=None):
        """A whole expert layer for a few tokens: out[i][t] = residual[i][t] + sum_s w[i][t][s] * D_e (silu(G_e x) *
        (U_e x)). x, residual, out bf16 [T][H]; w_up[j] [E/p][2F][H] (G's rows, then U's) and w_down[j]
        [E/p][H][F] bf16, or, with up_scale [E/p][2F][H/group] and down_scale [E/p][H][F/group] (bf16), 4-bit:
        uint8 with half as many columns."""
        torch = self._torch
        T, H = self._own(x).shape
        k = self._own(topk_idx).shape[1]
        el, rows = self._own(w_up).shape[:2]
        F = rows // 2
        q4 = up_scale is not None
        if q4 != (down_scale is not None) or rows != 2 * F or el * self.p != experts:
            raise ValueError("w_up must be [experts / p][2 F][...], and both scales or none be given")
        group, wt, per, su, sd = 0, torch.bfloat16, 1, None, None
        if q4:
            groups = self._own(up_scale).shape[2]
            if groups < 1 or H % groups or F % (H // groups):
                raise ValueError(f"up_scale: {groups} groups do not fit rows of {H} and {F}")
            group, wt, per = H // groups, torch.uint8, 2  # weights to an element
            su = self._tensors("up_scale", up_scale, torch.bfloat16, (el, rows, groups))
            sd = self._tensors("down_scale", down_scale, torch.bfloat16, (el, H, F // group))
        self._check(self._L.coll_moe_layer(
            self._h, self._tensors("x", x, torch.bfloat16, (T, H)),
            self._tensors("topk_idx", topk_idx, torch.int32, (T, k)),
            self._tensors("topk_weight", topk_weight, torch.float32, (T, k)),
            self._tensors("residual", residual, torch.bfloat16, (T, H)), T, k, H, F, int(experts), 1 if q4 else 0, group,
            self._tensors("w_up", w_up, wt, (el, rows, H // per)), su, self._tensors("w_down", w_down, wt, (el, H, F // per)), sd, DTYPES["bf16"],
            self._tensors("out", out, torch.bfloat16, (T, H)), self._launch_stream(stream)))

    def logprobs(self, logits, tokens, vocab, logprob, entropy=None, lse=None, top_idx=None, top_logprob=None,
                 stream=None):
        """Log probabilities of `tokens` (int32 [R], -1: none) under rows of scores whose `vocab` columns are
        sharded over the ranks: logits[r] [R][m], m = ceil(vocab / p), fp32 or bf16, rows at any distance. Every
        rank gets logprob[r], entropy[r], lse[r] fp32 [R] and the n best columns and their log probabilities
        in top_idx[r] int32 and top_logprob[r] fp32 [R][n]."""
        torch = self._torch
        x = self._own(logits)
        R, m = x.shape
        if m != -(-int(vocab) // self.p):
            raise ValueError(f"logits: {m} columns per rank for a vocabulary of {vocab} on {self.p} ranks")
        ld = x.stride(0) if R > 1 else m
        f = torch.float32
        n = 0 if top_idx is None else self._own(top_idx).shape[1]
        if (top_idx is None) != (top_logprob is None):
            raise ValueError("top_idx and top_logprob go together")
        self._check(self._L.coll_logprobs(
            self._h, self._tensors("logits", logits, x.dtype, (R, m), row=(ld, m)), ld,
            self._tensors("tokens", tokens, torch.int32, R, one=True), R, int(vocab), DTYPES[_dtype_of(x)],
            self._tensors("logprob", logprob, f, R), self._tensors("entropy", entropy, f, R),
            self._tensors("lse", lse, f, R), n, self._tensors("top_idx", top_idx, torch.int32, (R, n)),
            self._tensors("top_logprob", top_logprob, f, (R, n)), self._launch_stream(stream)))

    def logprobs_backward(self, logits, tokens, vocab, lse, grad_logprob, grad_logits, entropy=None,
                          grad_entropy=None, stream=None):
        """Gradient of logprobs' scores into grad_logits[r] [R][m] (of the scores' type, zeros in padding
        columns), from grad_logprob and grad_entropy (fp32 [R], the latter with `entropy`) and the forward
        call's lse[r] and entropy[r]."""
        torch = self._torch
        x, g = self._own(logits), self._own(grad_logits)
        R, m = x.shape
        if m != -(-int(vocab) // self.p):
            raise ValueError(f"logits: {m} columns per rank for a vocabulary of {vocab} on {self.p} ranks")
        ld, ldg = (x.stride(0), g.stride(0)) if R > 1 else (m, m)
        f = torch.float32
        if grad_entropy is not None and entropy is None:
            raise ValueError("grad_entropy needs entropy")
        self._check(self._L.coll_logprobs_backward(
            self._h, self._tensors("logits", logits, x.dtype, (R, m), row=(ld, m)), ld,
            self._tensors("tokens", tokens, torch.int32, R, one=True), R, int(vocab), DTYPES[_dtype_of(x)],
            self._tensors("lse", lse, f, R), self._tensors("entropy", entropy, f, R),
            self._tensors("grad_logprob", grad_logprob, f, R, one=True),
            None if grad_entropy is None else self._tensors("grad_entropy", grad_entropy, f, R, one=True),
            self._tensors("grad_logits", grad_logits, x.dtype, (R, m), row=(ldg, m)), ldg, self._launch_stream(stream)))


def allreduce_ring_noalloc(sends, recvs, op="sum", n=None, dtype=None, status=None, stream=None):
    """Ring AllReduce on the library's static scratch: no communicator, no allocation (for callers
    that cannot allocate device memory; see include/simcomm.h). `status` is an optional device int32
    tensor that receives the call's asynchronous status."""
    L = load_library()
    p = len(sends)
    n = sends[0].numel() if n is None else n
    s = (ctypes.c_void_p * p)(*[_ptr(x) for x in sends])
    r = (ctypes.c_void_p * p)(*[_ptr(x) for x in recvs])
    bufs = _Bufs(ctypes.cast(s, ctypes.POINTER(ctypes.c_void_p)), ctypes.cast(r, ctypes.POINTER(ctypes.c_void_p)))
    dt = SimComm._resolve(dtype, list(sends) + list(recvs))
    rc = L.coll_allreduce_ring_noalloc(p, bufs, n, dt, OPS[op], ctypes.c_void_p(_ptr(status)) if status is not None
                                       else None, _stream(stream))
    if rc != OK:
        raise SimCommError(rc, L.sim_comm_last_error().decode())


PROBES = {"load": 0, "store": 1, "copy": 2, "bulk_store": 3, "bulk_fanout": 4}


def hbm_probe(kind, dst, src, nbytes, ctas_per_sm, stream=None):
    """One HBM access-pattern probe (sim_hbm_probe): `kind` in PROBES; dst/src device tensors (or None
    where the kind does not use them), nbytes a multiple of 16 KiB (bulk_fanout: of 32 KiB, and dst
    holds 8 * nbytes)."""
    L = load_library()
    rc = L.sim_hbm_probe(PROBES[kind], ctypes.c_void_p(_ptr(dst)) if dst is not None else None,
                         ctypes.c_void_p(_ptr(src)) if src is not None else None, nbytes, ctas_per_sm,
                         _stream(stream))
    if rc != OK:
        raise SimCommError(rc, L.sim_comm_last_error().decode())
