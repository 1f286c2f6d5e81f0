"""Thin ctypes binding of the C ABI in include/lbq.h (argument marshalling only).

Every function keeps the C name and hands torch tensors' device pointers and the
current CUDA stream to liblbq.so; all arithmetic runs in the library's kernels. With
`stream=` a call runs on that stream, and the tensors it makes itself (outputs, a
workspace) are that stream's: order them as any tensor made there before another stream
reads them. No call records a gradient: outputs are plain tensors, and the calls that
compute gradients (lbq_expert_combine_grad, lbq_expert_combine) are called as they are.
Importing this module fails loudly when the library has not been built: there
is no fallback path.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from dataclasses import dataclass

import torch

LBQ_TERN5, LBQ_SIGN1, LBQ_Q2RHT, LBQ_Q4G32, LBQ_Q4G128 = 1, 2, 3, 5, 6
FORMATS = {"tern": LBQ_TERN5, "sign": LBQ_SIGN1, "q2": LBQ_Q2RHT, "q4g32": LBQ_Q4G32,
           "q4g128": LBQ_Q4G128}

LBQ_OK, LBQ_ERR_ARG, LBQ_ERR_SHAPE, LBQ_ERR_ALIGN, LBQ_ERR_FORMAT, LBQ_ERR_CUDA, \
    LBQ_ERR_WORKSPACE, LBQ_ERR_DEVICE_WAIT = range(8)

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "liblbq.so")
EXPORTS = ("lbq_status_string", "lbq_packed_layout", "lbq_pack", "lbq_unpack", "lbq_rht_signs",
           "lbq_hadamard", "lbq_workspace_bytes", "lbq_gemv", "lbq_gemm", "lbq_gemv_noalloc", "lbq_device_fault",
           "lbq_selftest_wait", "lbq_read_probe", "lbq_gemv_batch_workspace_bytes", "lbq_gemv_batch",
           "lbq_last_cuda_error", "lbq_last_cuda_error_string", "lbq_gemv_f32", "lbq_gemv_batch_plan",
           "lbq_expert_sort", "lbq_expert_dispatch", "lbq_expert_combine", "lbq_expert_combine_grad",
           "lbq_expert_workspace_bytes", "lbq_expert_gemm")
LBQ_MAX_EXPERTS = 1024
LBQ_BATCH_MAX = 256
LBQ_BATCH_MAX_CTAS = 192
LBQ_NOALLOC_SCRATCH_BYTES = 4 << 20


class lbq_weights(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("reserved", ctypes.c_int32), ("K", ctypes.c_int64),
                ("N", ctypes.c_int64), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("code_stride", ctypes.c_int64), ("scale_stride", ctypes.c_int64)]


class lbq_product(ctypes.Structure):
    _fields_ = [("w", lbq_weights), ("x", ctypes.c_void_p), ("D", ctypes.c_void_p),
                ("y", ctypes.c_void_p)]


class LbqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        extra = ""
        if status == LBQ_ERR_CUDA:
            extra = f": {_lib.lbq_last_cuda_error_string().decode()} ({_lib.lbq_last_cuda_error()})"
        super().__init__(f"{where}: {lbq_status_string(status)} (status {status}){extra}")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m bit_weight_only_ternary_b200.build` (needs nvcc)")
    lib = ctypes.CDLL(LIB_PATH)
    p, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    W = ctypes.POINTER(lbq_weights)
    sig = {
        "lbq_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "lbq_packed_layout": (ctypes.c_int, [i32, i64, i64, p, p, p, p]),
        "lbq_pack": (ctypes.c_int, [i32, p, i64, i64, p, p, p]),
        "lbq_unpack": (ctypes.c_int, [W, p, p, p]),
        "lbq_rht_signs": (ctypes.c_int, [ctypes.c_uint64, i64, p, p]),
        "lbq_hadamard": (ctypes.c_int, [p, p, i64, i64, p, p]),
        "lbq_workspace_bytes": (sz, [W, i64]),
        "lbq_gemv": (ctypes.c_int, [W, p, p, p, p, sz, p]),
        "lbq_gemv_f32": (ctypes.c_int, [W, p, p, p, p, sz, p]),
        "lbq_gemm": (ctypes.c_int, [W, p, i64, p, p, p, sz, p]),
        "lbq_gemv_noalloc": (ctypes.c_int, [W, p, p, p, p]),
        "lbq_device_fault": (ctypes.c_int, [p]),
        "lbq_selftest_wait": (ctypes.c_int, [p]),
        "lbq_read_probe": (ctypes.c_int, [p, sz, p, p]),
        "lbq_gemv_batch_workspace_bytes": (sz, [ctypes.POINTER(lbq_product), i32]),
        "lbq_gemv_batch": (ctypes.c_int, [ctypes.POINTER(lbq_product), i32, p, sz, p]),
        "lbq_gemv_batch_plan": (ctypes.c_int, [ctypes.POINTER(lbq_product), i32, i32, p, p, p]),
        "lbq_expert_sort": (ctypes.c_int, [p, i32, i64, i32, i32, p, p, p, p]),
        "lbq_expert_dispatch": (ctypes.c_int, [p, i64, i64, p, i32, p, i64, p, p]),
        "lbq_expert_combine": (ctypes.c_int, [p, i64, i64, p, i64, i32, p, p, p]),
        "lbq_expert_combine_grad": (ctypes.c_int, [p, p, i64, i64, p, i64, i32, p, p, p, p]),
        "lbq_expert_workspace_bytes": (sz, [W, i32, i64]),
        "lbq_expert_gemm": (ctypes.c_int, [W, i32, p, i64, p, p, i32, i64, p, p, sz, p]),
        "lbq_last_cuda_error": (i32, []),
        "lbq_last_cuda_error_string": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    return lib


_lib = _load()


def lib():
    return _lib


def lbq_status_string(status: int) -> str:
    return _lib.lbq_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != LBQ_OK:
        raise LbqError(status, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _current_raw_stream() -> int:
    """The handle of torch's current stream (without building a Stream object, which takes
    longer than the launch of a small product, where this torch allows it)."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(torch.cuda.current_device()) if raw else torch.cuda.current_stream().cuda_stream


def _stream(stream):
    if stream is None:
        return _current_raw_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_HERE = contextlib.nullcontext()


def _on(stream):
    """A context for the memory that a call makes itself (outputs, workspaces): taken from
    and filled in the order of the stream that the call runs on, not of torch's current
    one, with which nothing orders it."""
    if stream is None:
        return _HERE
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)
        # (0 and 1 name the default stream, and 0 to ExternalStream a new one)
        stream = torch.cuda.default_stream() if handle in (0, 1) else torch.cuda.ExternalStream(handle)
    return torch.cuda.stream(stream)


def lbq_packed_layout(fmt: int, K: int, N: int):
    """-> (code_stride bytes, scale_stride elements, code_bytes, scale_bytes)."""
    cs, ss = ctypes.c_int64(), ctypes.c_int64()
    cb, sb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(_lib.lbq_packed_layout(fmt, K, N, ctypes.byref(cs), ctypes.byref(ss), ctypes.byref(cb),
                                  ctypes.byref(sb)), "lbq_packed_layout")
    return cs.value, ss.value, cb.value, sb.value


@dataclass
class PackedWeights:
    """A packed matrix in the library's group-of-four row order: codes uint8
    [ceil(N/4)][4 * code_stride] and (sign, 2-bit) fp16 scales [ceil(N/4)][4 * scale_stride]."""
    fmt: int
    K: int
    N: int
    codes: torch.Tensor
    scales: torch.Tensor | None

    def desc(self) -> lbq_weights:
        return lbq_weights(self.fmt, 0, self.K, self.N, self.codes.data_ptr(),
                           None if self.scales is None else self.scales.data_ptr(),
                           self.codes.stride(0) // 4,
                           0 if self.scales is None else self.scales.stride(0) // 4)

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + (0 if self.scales is None else 2 * self.scales.numel())


def lbq_pack(fmt: int, W: torch.Tensor, stream=None) -> PackedWeights:
    """Quantise + pack fp32 W [N][K] (device) into freshly allocated device buffers."""
    assert W.is_cuda and W.dtype == torch.float32 and W.is_contiguous() and W.dim() == 2
    N, K = W.shape
    cs, ss, cb, sb = lbq_packed_layout(fmt, K, N)
    G = (N + 3) // 4  # rows are stored in groups of four
    with _on(stream):
        codes = torch.empty((G, 4 * cs), dtype=torch.uint8, device=W.device)
        scales = torch.empty((G, 4 * ss), dtype=torch.int16, device=W.device) if ss else None
    # (torch's allocations are 256-byte aligned, as the scales' TMA rows require)
    _check(_lib.lbq_pack(fmt, _ptr(W), K, N, _ptr(codes), _ptr(scales), _stream(stream)),
           "lbq_pack")
    return PackedWeights(fmt, K, N, codes, scales)


def lbq_unpack(pw: PackedWeights, stream=None):
    """-> (int8 codes [N][K], fp32 block scales [N][K/blk]) on the device."""
    blk = 32 if pw.fmt in (LBQ_Q2RHT, LBQ_Q4G32) else 128
    with _on(stream):
        out = torch.empty((pw.N, pw.K), dtype=torch.int8, device=pw.codes.device)
        sc = torch.empty((pw.N, pw.K // blk), dtype=torch.float32, device=pw.codes.device)
    d = pw.desc()
    _check(_lib.lbq_unpack(ctypes.byref(d), _ptr(out), _ptr(sc), _stream(stream)), "lbq_unpack")
    return out, sc


def lbq_rht_signs(seed: int, K: int, device="cuda", stream=None) -> torch.Tensor:
    with _on(stream):
        D = torch.empty(K, dtype=torch.int8, device=device)
    _check(_lib.lbq_rht_signs(ctypes.c_uint64(seed), K, _ptr(D), _stream(stream)), "lbq_rht_signs")
    return D


def lbq_hadamard(x: torch.Tensor, D: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """fp32 x' = H D x / sqrt(512) per 512-block for bf16 x [M][K] (or [K])."""
    x2 = x if x.dim() == 2 else x.view(1, -1)
    M, K = x2.shape
    if out is None:
        with _on(stream):
            out = torch.empty((M, K), dtype=torch.float32, device=x.device)
    _check(_lib.lbq_hadamard(_ptr(x2), _ptr(D), M, K, _ptr(out), _stream(stream)), "lbq_hadamard")
    return out.view(x.shape)


def lbq_device_fault() -> int:
    """Code of a bounded in-kernel wait that gave up since the last query (0: none)."""
    code = ctypes.c_uint32()
    st = _lib.lbq_device_fault(ctypes.byref(code))
    if st != LBQ_ERR_DEVICE_WAIT:
        _check(st, "lbq_device_fault")
    return code.value


def lbq_selftest_wait(stream=None) -> None:
    """Enqueues the kernel whose bounded wait runs out on purpose (fault code 11)."""
    _check(_lib.lbq_selftest_wait(_stream(stream)), "lbq_selftest_wait")


def lbq_workspace_bytes(pw: PackedWeights, M: int = 1) -> int:
    d = pw.desc()
    return int(_lib.lbq_workspace_bytes(ctypes.byref(d), M))


def workspace_for(pw: PackedWeights, M: int = 1, device=None) -> torch.Tensor | None:
    """A zero-filled workspace of lbq_workspace_bytes(pw, M) bytes (None if 0)."""
    n = lbq_workspace_bytes(pw, M)
    if n == 0:
        return None
    return torch.zeros(((n + 15) // 16) * 16, dtype=torch.uint8,
                       device=device or pw.codes.device)


def lbq_gemv(pw: PackedWeights, x: torch.Tensor, D=None, y=None, workspace=None,
             stream=None) -> torch.Tensor:
    """bf16 y [N] = W_hat x for bf16 x [K] (device)."""
    if y is None:
        with _on(stream):
            y = torch.empty(pw.N, dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        with _on(stream):
            workspace = workspace_for(pw, 1, x.device)
    d = pw.desc()
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.lbq_gemv(ctypes.byref(d), _ptr(x), _ptr(D), _ptr(y), _ptr(workspace), wsb,
                         _stream(stream)), "lbq_gemv")
    return y


def lbq_gemv_f32(pw: PackedWeights, x: torch.Tensor, D=None, y=None, workspace=None,
                 stream=None) -> torch.Tensor:
    """fp32 y [N] = W_hat x for bf16 x [K] (device), without the final bf16 rounding."""
    if y is None:
        with _on(stream):
            y = torch.empty(pw.N, dtype=torch.float32, device=x.device)
    if workspace is None:
        with _on(stream):
            workspace = workspace_for(pw, 1, x.device)
    d = pw.desc()
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.lbq_gemv_f32(ctypes.byref(d), _ptr(x), _ptr(D), _ptr(y), _ptr(workspace), wsb,
                             _stream(stream)), "lbq_gemv_f32")
    return y


def lbq_gemm(pw: PackedWeights, X: torch.Tensor, D=None, Y=None, workspace=None,
             stream=None) -> torch.Tensor:
    """bf16 Y [M][N] = X W_hat^T for bf16 X [M][K] (device)."""
    M = X.shape[0]
    if Y is None:
        with _on(stream):
            Y = torch.empty((M, pw.N), dtype=torch.bfloat16, device=X.device)
    if workspace is None:
        with _on(stream):
            workspace = workspace_for(pw, M, X.device)
    d = pw.desc()
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.lbq_gemm(ctypes.byref(d), _ptr(X), M, _ptr(D), _ptr(Y), _ptr(workspace), wsb,
                         _stream(stream)), "lbq_gemm")
    return Y


def lbq_gemv_noalloc(pw: PackedWeights, x: torch.Tensor, D=None, y=None,
                     stream=None) -> torch.Tensor:
    """lbq_gemv for callers that cannot allocate device memory: the library's own fixed
    scratch array replaces the workspace (see include/lbq.h). Only `y` is allocated
    here, and only when the caller passes none."""
    if y is None:
        with _on(stream):
            y = torch.empty(pw.N, dtype=torch.bfloat16, device=x.device)
    d = pw.desc()
    _check(_lib.lbq_gemv_noalloc(ctypes.byref(d), _ptr(x), _ptr(D), _ptr(y), _stream(stream)),
           "lbq_gemv_noalloc")
    return y


def lbq_read_probe(buf: torch.Tensor, sink: torch.Tensor, nbytes: int | None = None,
                   stream=None) -> None:
    """Reads nbytes (default: all) of a device tensor once, XOR-folding the words into
    sink (an int32 device tensor): the plain read-stream rate, a bandwidth denominator."""
    n = buf.numel() * buf.element_size() if nbytes is None else int(nbytes)
    _check(_lib.lbq_read_probe(_ptr(buf), n, _ptr(sink), _stream(stream)), "lbq_read_probe")


class ProductList:
    """A host array of lbq_product records for lbq_gemv_batch, built once from
    (packed weights, x, D or None, y) tuples; the tensors must outlive its use."""

    def __init__(self, items):
        self.items = list(items)
        self.arr = (lbq_product * len(self.items))()
        for i, (pw, x, D, y) in enumerate(self.items):
            self.arr[i].w = pw.desc()
            self.arr[i].x = x.data_ptr()
            self.arr[i].D = None if D is None else D.data_ptr()
            self.arr[i].y = y.data_ptr()

    def __len__(self):
        return len(self.items)


def lbq_gemv_batch_plan(arr, n: int, ctas: int):
    """The schedule one launch of lbq_gemv_batch gives a list of one format (host only):
    (pieces per product, CTA boundaries [ctas + 1], total unit-slices). `arr` is a
    ctypes array of lbq_product (ProductList.arr, or records built by hand)."""
    pieces = (ctypes.c_int32 * n)()
    bound = (ctypes.c_int64 * (ctas + 1))()
    total = ctypes.c_int64()
    _check(_lib.lbq_gemv_batch_plan(arr, n, ctas, pieces, bound, ctypes.byref(total)),
           "lbq_gemv_batch_plan")
    return list(pieces), list(bound), int(total.value)


def lbq_gemv_batch_workspace_bytes(plist: ProductList) -> int:
    return int(_lib.lbq_gemv_batch_workspace_bytes(plist.arr, len(plist)))


def lbq_gemv_batch(plist: ProductList, workspace=None, stream=None) -> None:
    """Every product of the list (independent batch-1 products, see include/lbq.h), one
    launch per format present and LBQ_BATCH_MAX products of it. The workspace's first
    64 KB must be zero when it is first used (workspace_for_batch gives such a buffer)."""
    if workspace is None:
        with _on(stream):
            workspace = workspace_for_batch(plist)
    wsb = workspace.numel() * workspace.element_size()
    _check(_lib.lbq_gemv_batch(plist.arr, len(plist), _ptr(workspace), wsb, _stream(stream)),
           "lbq_gemv_batch")


def workspace_for_batch(plist: ProductList, device=None) -> torch.Tensor:
    n = lbq_gemv_batch_workspace_bytes(plist)
    if n == 0:
        _check(LBQ_ERR_ARG, "lbq_gemv_batch_workspace_bytes")
    dev = device or plist.items[0][1].device
    return torch.zeros(((n + 15) // 16) * 16, dtype=torch.uint8, device=dev)


def _args(where: str, *specs):
    """The expert calls take dense tensors of one type on the current device: anything
    else is refused here (the C call sees pointers only). specs: (tensor or None, dtype,
    shape or None)."""
    dev = torch.cuda.current_device()
    for t, dtype, shape in specs:
        if t is None:
            continue
        if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
            _check(LBQ_ERR_ARG, where)
        if shape is not None and t.shape != shape:
            _check(LBQ_ERR_SHAPE, where)


@dataclass
class ExpertWeights:
    """E packed K x N matrices of one 4-bit format: codes uint8 [E][ceil(N/4)][4 *
    code_stride], scales fp16 (as int16) [E][ceil(N/4)][4 * scale_stride]. Both are dense:
    the matrices lie behind one another (a choice of experts, codes[::2], is copied first:
    codes[::2].contiguous())."""
    fmt: int
    K: int
    N: int
    E: int
    codes: torch.Tensor
    scales: torch.Tensor

    def desc(self) -> lbq_weights:
        """The C call's descriptor. Raises LbqError unless both tensors are of the shape
        above, dense, and of one-byte and two-byte values: it takes a pointer to expert 0
        and finds the others by these sizes."""
        for t, size in ((self.codes, 1), (self.scales, 2)):
            if t.dim() != 3 or t.shape[0] != self.E or t.shape[1] != (self.N + 3) // 4 or t.shape[2] % 4:
                _check(LBQ_ERR_SHAPE, "ExpertWeights")
            if t.element_size() != size or not t.is_contiguous():
                _check(LBQ_ERR_ARG, "ExpertWeights")
        return lbq_weights(self.fmt, 0, self.K, self.N, self.codes.data_ptr(),
                           self.scales.data_ptr(), self.codes.shape[2] // 4,
                           self.scales.shape[2] // 4)


def pack_experts(fmt: int, W: torch.Tensor, stream=None) -> ExpertWeights:
    """lbq_pack of every expert's fp32 matrix, W [E][N][K] (device), behind one another."""
    assert W.is_cuda and W.dtype == torch.float32 and W.is_contiguous() and W.dim() == 3
    E, N, K = W.shape
    cs, ss, _, _ = lbq_packed_layout(fmt, K, N)
    if ss == 0:
        _check(LBQ_ERR_FORMAT, "pack_experts")
    G = (N + 3) // 4
    with _on(stream):
        codes = torch.empty((E, G, 4 * cs), dtype=torch.uint8, device=W.device)
        scales = torch.empty((E, G, 4 * ss), dtype=torch.int16, device=W.device)
    for e in range(E):
        _check(_lib.lbq_pack(fmt, _ptr(W[e]), K, N, _ptr(codes[e]), _ptr(scales[e]),
                             _stream(stream)), "lbq_pack")
    return ExpertWeights(fmt, K, N, E, codes, scales)


def lbq_expert_sort(expert: torch.Tensor, E: int, offsets=None, rows=None, slots=None, stream=None):
    """expert int32 or int64 [T][topk] -> (offsets int32 [E+1], rows int32 [T][topk], slots
    int32 [T*topk]): a stable sort of the slots by expert (ids outside 0..E-1 left out)."""
    T, topk = expert.shape
    _args("lbq_expert_sort", (expert, torch.int64 if expert.dtype is torch.int64 else torch.int32, None),
          (offsets, torch.int32, (E + 1,)), (rows, torch.int32, (T, topk)), (slots, torch.int32, (T * topk,)))
    with _on(stream):
        if offsets is None:
            offsets = torch.empty(E + 1, dtype=torch.int32, device=expert.device)
        if rows is None:
            rows = torch.empty((T, topk), dtype=torch.int32, device=expert.device)
        if slots is None:
            slots = torch.empty(T * topk, dtype=torch.int32, device=expert.device)
    _check(_lib.lbq_expert_sort(_ptr(expert), expert.element_size(), T, topk, E, _ptr(offsets),
                                _ptr(rows), _ptr(slots), _stream(stream)), "lbq_expert_sort")
    return offsets, rows, slots


def lbq_expert_dispatch(X: torch.Tensor, rows: torch.Tensor, weights=None, out=None,
                        stream=None) -> torch.Tensor:
    """out[rows[t][j]] = (weights[t][j] *) X[t] for bf16 X [T][K]; out [R][K], by default
    R = T * topk (rows behind the last sorted one are then uninitialised)."""
    T, K = X.shape
    topk = rows.shape[1]
    _args("lbq_expert_dispatch", (X, torch.bfloat16, None), (rows, torch.int32, (T, topk)),
          (weights, torch.float32, (T, topk)),
          (out, torch.bfloat16, None if out is None else (out.shape[0], K)))
    if out is None:
        with _on(stream):
            out = torch.empty((T * topk, K), dtype=torch.bfloat16, device=X.device)
    _check(_lib.lbq_expert_dispatch(_ptr(X), T, K, _ptr(rows), topk, _ptr(weights), out.shape[0],
                                    _ptr(out), _stream(stream)), "lbq_expert_dispatch")
    return out


def lbq_expert_combine(Y: torch.Tensor, rows: torch.Tensor, weights=None, out=None,
                       stream=None) -> torch.Tensor:
    """bf16 out [T][N]: out[t] = sum_j (weights[t][j] *) Y[rows[t][j]] for bf16 Y [R][N]."""
    R, N = Y.shape
    T, topk = rows.shape
    _args("lbq_expert_combine", (Y, torch.bfloat16, None), (rows, torch.int32, None),
          (weights, torch.float32, (T, topk)), (out, torch.bfloat16, (T, N)))
    if out is None:
        with _on(stream):
            out = torch.empty((T, N), dtype=torch.bfloat16, device=Y.device)
    _check(_lib.lbq_expert_combine(_ptr(Y), R, N, _ptr(rows), T, topk, _ptr(weights), _ptr(out),
                                   _stream(stream)), "lbq_expert_combine")
    return out


def lbq_expert_combine_grad(dout: torch.Tensor, Y: torch.Tensor, rows: torch.Tensor,
                            weights: torch.Tensor, dY=None, dweights=None, stream=None):
    """The gradients of lbq_expert_combine: (dY bf16 [R][N], dweights fp32 [T][topk]). Rows
    of dY that no slot names are left as they were (uninitialised in a new dY)."""
    R, N = Y.shape
    T, topk = rows.shape
    _args("lbq_expert_combine_grad", (Y, torch.bfloat16, None), (dout, torch.bfloat16, (T, N)),
          (rows, torch.int32, None), (weights, torch.float32, (T, topk)), (dY, torch.bfloat16, (R, N)),
          (dweights, torch.float32, (T, topk)))
    with _on(stream):
        if dY is None:
            dY = torch.empty((R, N), dtype=torch.bfloat16, device=Y.device)
        if dweights is None:
            dweights = torch.empty((T, topk), dtype=torch.float32, device=Y.device)
    _check(_lib.lbq_expert_combine_grad(_ptr(dout), _ptr(Y), R, N, _ptr(rows), T, topk,
                                        _ptr(weights), _ptr(dY), _ptr(dweights), _stream(stream)),
           "lbq_expert_combine_grad")
    return dY, dweights


def lbq_expert_workspace_bytes(ew: ExpertWeights, R: int) -> int:
    d = ew.desc()
    return int(_lib.lbq_expert_workspace_bytes(ctypes.byref(d), ew.E, R))


def workspace_for_experts(ew: ExpertWeights, R: int, device=None) -> torch.Tensor | None:
    """A zero-filled workspace of lbq_expert_workspace_bytes(ew, R) bytes (None if 0)."""
    n = lbq_expert_workspace_bytes(ew, R)
    if n == 0:
        return None
    return torch.zeros(((n + 15) // 16) * 16, dtype=torch.uint8, device=device or ew.codes.device)


def lbq_expert_gemm(ew: ExpertWeights, X: torch.Tensor, offsets: torch.Tensor, slots=None,
                    topk: int = 1, Y=None, workspace=None, stream=None) -> torch.Tensor:
    """bf16 Y [R][N]: row r of expert e is W_hat_e X[slots[r] // topk] (X[r] with slots None)
    for offsets[e] <= r < offsets[e+1]; other rows are left as they were."""
    T = X.shape[0]
    w = "lbq_expert_gemm"
    R = Y.shape[0] if Y is not None else (T if slots is None else slots.shape[0])
    _args(w, (X, torch.bfloat16, (T, ew.K)), (offsets, torch.int32, (ew.E + 1,)), (slots, torch.int32, (R,)),
          (Y, torch.bfloat16, (R, ew.N)))
    dev = X.get_device()
    if ew.codes.get_device() != dev or ew.scales.get_device() != dev:
        _check(LBQ_ERR_ARG, w)
    if workspace is not None and (workspace.get_device() != dev or not workspace.is_contiguous()):
        _check(LBQ_ERR_ARG, w)
    d = ew.desc()
    if Y is None:
        with _on(stream):
            Y = torch.empty((R, ew.N), dtype=torch.bfloat16, device=X.device)
    if workspace is None:
        with _on(stream):
            workspace = workspace_for_experts(ew, R, X.device)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.lbq_expert_gemm(ctypes.byref(d), ew.E, _ptr(X), T, _ptr(offsets), _ptr(slots), topk,
                                R, _ptr(Y), _ptr(workspace), wsb, _stream(stream)),
           "lbq_expert_gemm")
    return Y
