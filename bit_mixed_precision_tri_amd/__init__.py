"""Python binding of libtri, the gfx950 ternary linear layer.

The functions named ``tri_*`` mirror the C ABI in ``include/tri.h`` one to one:
they only marshal arguments (device pointers of torch tensors, the current HIP
stream) and raise ``TriError`` on a negative status.  All the work runs in the
library's HIP kernels; there is no fallback of any kind -- if ``libtri.so`` is
missing, every call raises.  The helpers at the end (``pack``, ``unpack``,
``quantize``, ``linear``) allocate their outputs with torch and then call the same
entry points.
"""
import collections
import ctypes
import functools
import os
import struct

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libtri.so")

TRI_FMT_2BIT = 0
TRI_FMT_1P6BIT = 1
TRI_OK, TRI_EINVAL, TRI_EALIGN, TRI_EHIP = 0, -1, -2, -3
TRI_ALGO_AUTO, TRI_ALGO_GEMV, TRI_ALGO_SMALLM, TRI_ALGO_GEMM = 0, 1, 2, 3
ALGO_NAMES = {TRI_ALGO_GEMV: "gemv", TRI_ALGO_SMALLM: "smallm", TRI_ALGO_GEMM: "gemm"}

_lib = None


class TriGlue(ctypes.Structure):
    """tri_glue of include/tri.h."""
    _fields_ = [("norm_gain", ctypes.c_void_p), ("norm", ctypes.c_int), ("norm_eps", ctypes.c_float),
                ("pair", ctypes.c_int), ("residual", ctypes.c_void_p)]


class TriHeads(ctypes.Structure):
    """tri_heads of include/tri.h."""
    _fields_ = [("X", ctypes.c_void_p), ("Y", ctypes.c_void_p), ("gain", ctypes.c_void_p), ("x_stride", ctypes.c_int64),
                ("y_stride", ctypes.c_int64), ("heads", ctypes.c_int)]


class TriRotary(ctypes.Structure):
    """tri_rotary of include/tri.h."""
    _fields_ = [("table", ctypes.c_void_p), ("rows", ctypes.c_int64), ("dims", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("norm", ctypes.c_int), ("eps", ctypes.c_float)]


class TriCache(ctypes.Structure):
    """tri_cache of include/tri.h."""
    _fields_ = [("K", ctypes.c_void_p), ("V", ctypes.c_void_p), ("K_scale", ctypes.c_void_p), ("V_scale", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("heads", ctypes.c_int), ("dim", ctypes.c_int), ("page", ctypes.c_int),
                ("fmt", ctypes.c_int)]


class TriSequences(ctypes.Structure):
    """tri_sequences of include/tri.h."""
    _fields_ = [("offsets", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("table", ctypes.c_void_p), ("B", ctypes.c_int64),
                ("width", ctypes.c_int64), ("max_new", ctypes.c_int64), ("max_len", ctypes.c_int64)]


class TriError(RuntimeError):
    def __init__(self, code, what):
        super().__init__("%s failed: %s (%d)" % (what, status_string(code), code))
        self.code = code


def lib():
    """The loaded libtri.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libtri.so is not built (%s); run __graft_entry__.build()" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        i64, p, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
        L.tri_row_bytes.argtypes = [i64, i32]
        L.tri_row_bytes.restype = i64
        for name in ("tri_pack2", "tri_pack16"):
            getattr(L, name).argtypes = [p, i64, i64, p, p]
            getattr(L, name).restype = i32
        L.tri_unpack.argtypes = [p, i64, i64, i32, p, p]
        L.tri_unpack.restype = i32
        L.tri_quantize_workspace_bytes.argtypes = [i64, i64]
        L.tri_quantize_workspace_bytes.restype = i64
        L.tri_quantize.argtypes = [p, i64, i64, i32, p, p, p, i64, p]
        L.tri_quantize.restype = i32
        L.tri_quantize_noalloc.argtypes = [p, i64, i64, i32, p, p, p]
        L.tri_quantize_noalloc.restype = i32
        L.tri_linear.argtypes = [p, p, ctypes.c_float, i64, i64, i64, i32, p, p]
        L.tri_linear.restype = i32
        L.tri_linear_algo.argtypes = [p, p, ctypes.c_float, i64, i64, i64, i32, p, i32, p]
        L.tri_linear_algo.restype = i32
        L.tri_linear_grouped.argtypes = [p, p, p, i64, p, i64, i32, p, i32, p]
        L.tri_linear_grouped.restype = i32
        L.tri_linear_fused.argtypes = [p, p, p, i64, p, i64, i32, p, i32, ctypes.POINTER(TriGlue), p]
        L.tri_linear_fused.restype = i32
        L.tri_select_algo.argtypes = [i64, i64, i64, i32]
        L.tri_select_algo.restype = i32
        L.tri_status_string.argtypes = [i32]
        L.tri_status_string.restype = ctypes.c_char_p
        L.tri_probe_read.argtypes = [p, i64, p, p]
        L.tri_probe_read.restype = i32
        L.tri_probe_copy.argtypes = [p, p, i64, p]
        L.tri_probe_copy.restype = i32
        L.tri_probe_empty.argtypes = [i64, i32, p, p]
        L.tri_probe_empty.restype = i32
        L.tri_probe_rows.argtypes = [p, p, i64, i64, i32, i32, p, p]
        L.tri_probe_rows.restype = i32
        L.tri_probe_stream.argtypes = [p, i64, i32, i32, p, p]
        L.tri_probe_stream.restype = i32
        L.tri_int4_bytes.argtypes = [i64, i64, i32, i32]
        L.tri_int4_bytes.restype = i64
        L.tri_int4_pack.argtypes = [p, p, p, i64, i64, i32, p, p]
        L.tri_int4_unpack.argtypes = [p, i64, i64, i32, i32, p, p, p, p]
        L.tri_int4_quantize.argtypes = [p, i64, i64, i32, i32, p, p]
        L.tri_int4_linear.argtypes = [p, p, i64, i64, i64, i32, i32, p, p, p]
        L.tri_experts_route_workspace_bytes.argtypes = [i64, i32, i32]
        L.tri_experts_route_workspace_bytes.restype = i64
        L.tri_experts_route.argtypes = [p, i32, i64, i32, i32, i32, p, p, p, p, p, p, i64, p]
        L.tri_experts_linear.argtypes = [p, i64, p, p, i64, p, p, i32, i64, i64, i32, p, p]
        L.tri_experts_pair.argtypes = [p, i64, p, p, i64, p, p, p, p, i32, i64, i64, i32, p, p]
        L.tri_experts_combine.argtypes = [p, i64, p, p, p, i64, i32, i64, p, p]
        L.tri_heads_rotate.argtypes = [p, i32, i64, i32, p, p, p]
        L.tri_cache_append.argtypes = [p, p, i64, p, i64, p, i64, p, p, p, p]
        L.tri_cache_attend_workspace_bytes.argtypes = [p, p, i64, i32, i64, i64]
        L.tri_cache_attend_workspace_bytes.restype = i64
        L.tri_cache_attend.argtypes = [p, p, i64, p, i64, i32, ctypes.c_float, i64, i64, p, i64, p, i64, p]
        for name in ("tri_int4_pack", "tri_int4_unpack", "tri_int4_quantize", "tri_int4_linear", "tri_experts_route",
                     "tri_experts_linear", "tri_experts_pair", "tri_experts_combine", "tri_heads_rotate", "tri_cache_append",
                     "tri_cache_attend"):
            getattr(L, name).restype = i32
        _lib = L
    return _lib


def status_string(code):
    return lib().tri_status_string(int(code)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr() if hasattr(t, "data_ptr") else int(t))


def _stream(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(rc, what):
    if rc != TRI_OK:
        raise TriError(rc, what)
    return rc


# ---------------------------------------------------------------- the C ABI, one to one

def tri_row_bytes(K, fmt):
    return int(lib().tri_row_bytes(int(K), int(fmt)))


def tri_pack2(W, N, K, Wp, stream=None):
    return _check(lib().tri_pack2(_ptr(W), int(N), int(K), _ptr(Wp), _stream(stream)), "tri_pack2")


def tri_pack16(W, N, K, Wp, stream=None):
    return _check(lib().tri_pack16(_ptr(W), int(N), int(K), _ptr(Wp), _stream(stream)), "tri_pack16")


def tri_unpack(Wp, N, K, fmt, W, stream=None):
    return _check(lib().tri_unpack(_ptr(Wp), int(N), int(K), int(fmt), _ptr(W), _stream(stream)), "tri_unpack")


def tri_quantize_workspace_bytes(N, K):
    return int(lib().tri_quantize_workspace_bytes(int(N), int(K)))


def tri_quantize(W, N, K, fmt, Wp, scale_out, workspace, workspace_bytes, stream=None):
    return _check(lib().tri_quantize(_ptr(W), int(N), int(K), int(fmt), _ptr(Wp), _ptr(scale_out), _ptr(workspace),
                                     int(workspace_bytes), _stream(stream)), "tri_quantize")


def tri_quantize_noalloc(W, N, K, fmt, Wp, scale_out, stream=None):
    return _check(lib().tri_quantize_noalloc(_ptr(W), int(N), int(K), int(fmt), _ptr(Wp), _ptr(scale_out),
                                             _stream(stream)), "tri_quantize_noalloc")


def tri_linear(X, Wp, scale, M, N, K, fmt, Y, stream=None):
    return _check(lib().tri_linear(_ptr(X), _ptr(Wp), float(scale), int(M), int(N), int(K), int(fmt), _ptr(Y),
                                   _stream(stream)), "tri_linear")


def tri_linear_algo(X, Wp, scale, M, N, K, fmt, Y, algo, stream=None):
    return _check(lib().tri_linear_algo(_ptr(X), _ptr(Wp), float(scale), int(M), int(N), int(K), int(fmt), _ptr(Y),
                                        int(algo), _stream(stream)), "tri_linear_algo")


TRI_MAX_GROUPS = 4
TRI_QUANTIZE_SCRATCH_BYTES = 16384


def tri_linear_grouped(X, Wps, scales, M, Ns, K, fmt, Ys, stream=None):
    """Wps, scales, Ns, Ys: sequences of G entries (device tensors / floats / ints)."""
    G = len(Wps)
    if not (len(scales) == len(Ns) == len(Ys) == G):
        raise ValueError("tri_linear_grouped: Wps, scales, Ns and Ys must have the same length")
    wp = (ctypes.c_void_p * max(G, 1))(*[_ptr(w).value for w in Wps])
    sc = (ctypes.c_float * max(G, 1))(*[float(v) for v in scales])
    nn = (ctypes.c_int64 * max(G, 1))(*[int(v) for v in Ns])
    yy = (ctypes.c_void_p * max(G, 1))(*[_ptr(y).value for y in Ys])
    return _check(lib().tri_linear_grouped(_ptr(X), wp, sc, int(M), nn, int(K), int(fmt), yy, int(G),
                                           _stream(stream)), "tri_linear_grouped")


def tri_linear_fused(X, Wps, scales, M, Ns, K, fmt, Ys, norm=False, gain=None, eps=1e-5, pair=False,
                     residuals=None, stream=None):
    """tri_linear_grouped with a decode block's glue: y_g = scales[g] * x' W_g^T (x' = rmsnorm(X) if norm);
    Ys[g] = fp16(residuals[g] + y_g), or with pair (two matrices, gate then up) Ys[0] = fp16(residuals[0] +
    silu(y_0) * y_1).  residuals: None or a sequence of G entries (tensor or None); Ys[1] may be None with pair."""
    G = len(Wps)
    if not (len(scales) == len(Ns) == len(Ys) == G) or (residuals is not None and len(residuals) != G):
        raise ValueError("tri_linear_fused: per-matrix sequences must have the same length")
    wp = (ctypes.c_void_p * max(G, 1))(*[_ptr(w).value for w in Wps])
    sc = (ctypes.c_float * max(G, 1))(*[float(v) for v in scales])
    nn = (ctypes.c_int64 * max(G, 1))(*[int(v) for v in Ns])
    yy = (ctypes.c_void_p * max(G, 1))(*[None if y is None else _ptr(y).value for y in Ys])
    rr = None
    if residuals is not None:
        rr = (ctypes.c_void_p * max(G, 1))(*[None if r is None else _ptr(r).value for r in residuals])
    glue = TriGlue(None if gain is None else _ptr(gain).value, 1 if norm else 0, float(eps), 1 if pair else 0,
                   None if rr is None else ctypes.cast(rr, ctypes.c_void_p).value)
    return _check(lib().tri_linear_fused(_ptr(X), wp, sc, int(M), nn, int(K), int(fmt), yy, int(G),
                                         ctypes.byref(glue), _stream(stream)), "tri_linear_fused")


TRI_MAX_EXPERTS, TRI_MAX_TOPK = 256, 16
TRI_F16, TRI_F32 = 0, 1


def tri_int4_bytes(N, K, group, zeros):
    return int(lib().tri_int4_bytes(int(N), int(K), int(group), 1 if zeros else 0))


def tri_int4_pack(Q, S, Z, N, K, group, Wp, stream=None):
    return _check(lib().tri_int4_pack(_ptr(Q), _ptr(S), _ptr(Z), int(N), int(K), int(group), _ptr(Wp),
                                      _stream(stream)), "tri_int4_pack")


def tri_int4_unpack(Wp, N, K, group, zeros, Q, S, Z, stream=None):
    return _check(lib().tri_int4_unpack(_ptr(Wp), int(N), int(K), int(group), 1 if zeros else 0, _ptr(Q), _ptr(S),
                                        _ptr(Z), _stream(stream)), "tri_int4_unpack")


def tri_int4_quantize(W, N, K, group, zeros, Wp, stream=None):
    return _check(lib().tri_int4_quantize(_ptr(W), int(N), int(K), int(group), 1 if zeros else 0, _ptr(Wp),
                                          _stream(stream)), "tri_int4_quantize")


def tri_int4_linear(X, Wp, M, N, K, group, zeros, residual, Y, stream=None):
    return _check(lib().tri_int4_linear(_ptr(X), _ptr(Wp), int(M), int(N), int(K), int(group), 1 if zeros else 0,
                                        _ptr(residual), _ptr(Y), _stream(stream)), "tri_int4_linear")


def tri_experts_route_workspace_bytes(T, E, topk):
    return int(lib().tri_experts_route_workspace_bytes(int(T), int(E), int(topk)))


def tri_experts_route(logits, dtype, T, E, topk, renorm, ids, weights, offsets, rows, pos, workspace, workspace_bytes,
                      stream=None):
    return _check(lib().tri_experts_route(_ptr(logits), int(dtype), int(T), int(E), int(topk), 1 if renorm else 0,
                                          _ptr(ids), _ptr(weights), _ptr(offsets), _ptr(rows), _ptr(pos),
                                          _ptr(workspace), int(workspace_bytes), _stream(stream)), "tri_experts_route")


def tri_experts_linear(X, T, offsets, rows, R, Wp, scale, E, N, K, fmt, Y, stream=None):
    return _check(lib().tri_experts_linear(_ptr(X), int(T), _ptr(offsets), _ptr(rows), int(R), _ptr(Wp), _ptr(scale),
                                           int(E), int(N), int(K), int(fmt), _ptr(Y), _stream(stream)),
                  "tri_experts_linear")


def tri_experts_pair(X, T, offsets, rows, R, Wp, scale, Wp_up, scale_up, E, N, K, fmt, Y, stream=None):
    return _check(lib().tri_experts_pair(_ptr(X), int(T), _ptr(offsets), _ptr(rows), int(R), _ptr(Wp), _ptr(scale),
                                         _ptr(Wp_up), _ptr(scale_up), int(E), int(N), int(K), int(fmt), _ptr(Y),
                                         _stream(stream)), "tri_experts_pair")


def tri_experts_combine(Z, R, pos, weights, residual, T, topk, N, Y, stream=None):
    return _check(lib().tri_experts_combine(_ptr(Z), int(R), _ptr(pos), _ptr(weights), _ptr(residual), int(T),
                                            int(topk), int(N), _ptr(Y), _stream(stream)), "tri_experts_combine")


TRI_KV_INT8, TRI_KV_E4M3 = 0, 1


def _ref(struct):
    return None if struct is None else ctypes.addressof(struct)


def tri_heads_rotate(heads, T, dim, rot, positions, stream=None):
    """heads: a sequence of TriHeads; rot: a TriRotary."""
    G = len(heads)
    hs = (TriHeads * max(G, 1))(*heads)
    return _check(lib().tri_heads_rotate(_ref(hs), G, int(T), int(dim), _ref(rot), _ptr(positions), _stream(stream)),
                  "tri_heads_rotate")


def tri_cache_append(cache, seqs, T, K, k_stride, V, v_stride, rot=None, k_gain=None, queries=None, stream=None):
    """cache: a TriCache; seqs: a TriSequences; rot: a TriRotary or None; queries: a TriHeads or None."""
    return _check(lib().tri_cache_append(_ref(cache), _ref(seqs), int(T), _ptr(K), int(k_stride), _ptr(V), int(v_stride),
                                         _ref(rot), _ptr(k_gain), _ref(queries), _stream(stream)), "tri_cache_append")


def tri_cache_attend_workspace_bytes(cache, seqs, T, heads, window=0, sinks=0):
    return int(lib().tri_cache_attend_workspace_bytes(_ref(cache), _ref(seqs), int(T), int(heads), int(window), int(sinks)))


def tri_cache_attend(cache, seqs, T, Q, q_stride, heads, scale, window, sinks, O, o_stride, workspace, workspace_bytes,
                     stream=None):
    return _check(lib().tri_cache_attend(_ref(cache), _ref(seqs), int(T), _ptr(Q), int(q_stride), int(heads), float(scale),
                                         int(window), int(sinks), _ptr(O), int(o_stride), _ptr(workspace),
                                         int(workspace_bytes), _stream(stream)), "tri_cache_attend")


def tri_select_algo(M, N, K, fmt):
    return int(lib().tri_select_algo(int(M), int(N), int(K), int(fmt)))


def tri_status_string(code):
    return status_string(code)


def tri_probe_read(src, nbytes, sink, stream=None):
    return _check(lib().tri_probe_read(_ptr(src), int(nbytes), _ptr(sink), _stream(stream)), "tri_probe_read")


def tri_probe_copy(src, dst, nbytes, stream=None):
    return _check(lib().tri_probe_copy(_ptr(src), _ptr(dst), int(nbytes), _stream(stream)), "tri_probe_copy")


def tri_probe_empty(workgroups, threads, sink, stream=None):
    return _check(lib().tri_probe_empty(int(workgroups), int(threads), _ptr(sink), _stream(stream)), "tri_probe_empty")


def tri_probe_rows(X, Wp, N, K, fmt, waves, Y, stream=None):
    return _check(lib().tri_probe_rows(_ptr(X), _ptr(Wp), int(N), int(K), int(fmt), int(waves), _ptr(Y),
                                       _stream(stream)), "tri_probe_rows")


def tri_probe_stream(src, nbytes, workgroups, unroll, sink, stream=None):
    return _check(lib().tri_probe_stream(_ptr(src), int(nbytes), int(workgroups), int(unroll), _ptr(sink),
                                         _stream(stream)), "tri_probe_stream")


# ---------------------------------------------------------------- allocating helpers

_torch = None


def _load_torch():
    global _torch
    import torch
    _torch = torch
    return torch


def _new(shape, dtype, device, stream, result=True):
    """An uninitialised tensor for a call on `stream`.  A stream that the caller named writes it without waiting for the
    current one, so its memory comes from that stream's own pool: the current stream's pool hands out memory that kernels
    queued there may still use.  A result is not reused, either, before the current stream is done with it, where the
    caller reads it after the two were ordered."""
    torch = _torch or _load_torch()
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else stream
    if handle is None or handle == torch._C._cuda_getCurrentRawStream(device.index):
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(torch.cuda.ExternalStream(handle, device=device)):
        t = torch.empty(shape, dtype=dtype, device=device)
    if result:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def pack(W, fmt, stream=None):
    """Pack a (N, K) int8 CUDA tensor; returns a new (N, row_bytes) uint8 tensor."""
    import torch
    N, K = W.shape
    assert W.dtype == torch.int8 and W.is_cuda and W.is_contiguous()
    Wp = _new((N, tri_row_bytes(K, fmt)), torch.uint8, W.device, stream)
    (tri_pack2 if fmt == TRI_FMT_2BIT else tri_pack16)(W, N, K, Wp, stream)
    return Wp


def unpack(Wp, K, fmt, stream=None):
    """Unpack a (N, row_bytes) uint8 CUDA tensor; returns a new (N, K) int8 tensor."""
    import torch
    N = Wp.shape[0]
    assert Wp.dtype == torch.uint8 and Wp.is_cuda and Wp.is_contiguous()
    assert Wp.shape[1] == tri_row_bytes(K, fmt)
    W = _new((N, K), torch.int8, Wp.device, stream)
    tri_unpack(Wp, N, K, fmt, W, stream)
    return W


def quantize(W, fmt, stream=None):
    """Quantise a (N, K) float32 CUDA tensor of latent weights; returns (packed weights as a new
    (N, row_bytes) uint8 tensor, the scale as a new 1-element float32 tensor on the device)."""
    import torch
    N, K = W.shape
    assert W.dtype == torch.float32 and W.is_cuda and W.is_contiguous()
    Wp = _new((N, tri_row_bytes(K, fmt)), torch.uint8, W.device, stream)
    scale = _new(1, torch.float32, W.device, stream)
    nbytes = tri_quantize_workspace_bytes(N, K)
    ws = _new(max(nbytes, 16), torch.uint8, W.device, stream, result=False)
    tri_quantize(W, N, K, fmt, Wp, scale, ws, nbytes, stream)
    return Wp, scale


def linear(X, Wp, scale, K, fmt, algo=TRI_ALGO_AUTO, out=None, stream=None):
    """Y = fp16(scale * X @ W.T) for a (M, K) fp16 CUDA tensor X and packed weights Wp."""
    import torch
    M = X.shape[0]
    N = Wp.shape[0]
    assert X.dtype == torch.float16 and X.is_cuda and X.is_contiguous() and X.shape[1] == K
    assert Wp.dtype == torch.uint8 and Wp.is_contiguous() and Wp.shape[1] == tri_row_bytes(K, fmt)
    Y = out if out is not None else _new((M, N), torch.float16, X.device, stream)
    if algo == TRI_ALGO_AUTO:
        tri_linear(X, Wp, scale, M, N, K, fmt, Y, stream)
    else:
        tri_linear_algo(X, Wp, scale, M, N, K, fmt, Y, algo, stream)
    return Y


# The helpers below take the tensors' device (whichever device is current) and its current stream, or `stream` (ordering
# that stream behind what writes their inputs, and whoever reads their results behind it, is the caller's); they raise
# ValueError for tensors of another type, shape, device or layout than they name.

def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _launch(name, device, stream, *args):
    """The entry point `name` on `device` (an ordinal) with the stream appended."""
    torch = _torch
    if device != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return _launch(name, device, stream, *args)
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(device)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    rc = getattr(_lib or lib(), name)(*args, stream)
    if rc:
        raise TriError(rc, name)


def _plain(t, dtype, device):
    """Whether tensor `t` is of `dtype`, contiguous and on `device`."""
    return t.dtype is dtype and t.get_device() == device and t.is_contiguous()


def _tensors(device, dtype, **named):
    """Every named tensor (None is left out) is of `dtype`, contiguous and on `device`."""
    for name, t in named.items():
        if t is not None and not _plain(t, dtype, device):
            raise ValueError("%s must be a contiguous %s tensor on device %d" % (name, dtype, device))


@functools.lru_cache(maxsize=4096)
def _int4_nbytes(N, K, group, zeros):
    return tri_int4_bytes(N, K, group, zeros)


@functools.lru_cache(maxsize=4096)
def _route_nbytes(T, E, topk):
    return tri_experts_route_workspace_bytes(T, E, topk)


@functools.lru_cache(maxsize=4096)
def _row_nbytes(K, fmt):
    return tri_row_bytes(K, fmt)


def int4_pack(Q, S, group, Z=None, stream=None):
    """Lay out 4-bit codes Q (N, K) uint8 with group scales S (N, ceil(K/group)) float16 and, optionally, zero points
    Z of S's shape uint8 (8 everywhere without); returns a new uint8 tensor for int4_linear."""
    torch = _torch or _load_torch()
    _need(Q.is_cuda and Q.dim() == 2 and Q.numel() > 0, "Q must be an (N, K) tensor on the GPU")
    (N, K), dev = Q.shape, Q.get_device()
    _tensors(dev, torch.uint8, Q=Q, Z=Z)
    _tensors(dev, torch.float16, S=S)
    nbytes = tri_int4_bytes(N, K, group, Z is not None)
    _need(nbytes > 0, "group must be 32, 64 or 128 (and the matrix below 2^22 tiles)")
    shape = (N, -(-K // group))
    _need(S.shape == shape and (Z is None or Z.shape == shape), "S and Z must be (N, ceil(K/group))")
    Wp = _new(nbytes, torch.uint8, Q.device, stream)
    _launch("tri_int4_pack", dev, stream, Q.data_ptr(), S.data_ptr(), None if Z is None else Z.data_ptr(), N, K, group,
            Wp.data_ptr())
    return Wp


def int4_unpack(Wp, N, K, group, zeros=False, stream=None):
    """The codes, scales and zero points (None where zeros is false) of a packed 4-bit matrix."""
    torch = _torch or _load_torch()
    _need(Wp.is_cuda, "Wp must be on the GPU")
    dev = Wp.get_device()
    _tensors(dev, torch.uint8, Wp=Wp)
    nbytes = tri_int4_bytes(N, K, group, zeros)
    _need(nbytes > 0 and Wp.numel() == nbytes, "Wp does not hold tri_int4_bytes(N, K, group, zeros) bytes")
    shape = (N, -(-K // group))
    Q = _new((N, K), torch.uint8, Wp.device, stream)
    S = _new(shape, torch.float16, Wp.device, stream)
    Z = _new(shape, torch.uint8, Wp.device, stream) if zeros else None
    _launch("tri_int4_unpack", dev, stream, Wp.data_ptr(), N, K, group, 1 if zeros else 0, Q.data_ptr(), S.data_ptr(),
            None if Z is None else Z.data_ptr())
    return Q, S, Z


def int4_quantize(W, group, zeros=False, stream=None):
    """Quantise an (N, K) float32 tensor to 4-bit codes with group scales (and zero points), laid out for int4_linear."""
    torch = _torch or _load_torch()
    _need(W.is_cuda and W.dim() == 2 and W.numel() > 0, "W must be an (N, K) tensor on the GPU")
    (N, K), dev = W.shape, W.get_device()
    _tensors(dev, torch.float32, W=W)
    nbytes = tri_int4_bytes(N, K, group, zeros)
    _need(nbytes > 0, "group must be 32, 64 or 128 (and the matrix below 2^22 tiles)")
    Wp = _new(nbytes, torch.uint8, W.device, stream)
    _launch("tri_int4_quantize", dev, stream, W.data_ptr(), N, K, group, 1 if zeros else 0, Wp.data_ptr())
    return Wp


def int4_linear(X, Wp, N, group, zeros=False, residual=None, out=None, stream=None):
    """Y = fp16(residual + X @ W.T) for an (M, K) fp16 tensor X and a packed 4-bit matrix of N rows.  `residual` may be
    `out` itself."""
    torch = _torch or _load_torch()
    half, dev, shape = torch.float16, X.get_device(), X.shape
    if not (len(shape) == 2 and dev >= 0 and shape[0] > 0 and X.dtype is half and X.is_contiguous()):
        raise ValueError("X must be a contiguous (M, K) float16 tensor on the GPU")
    M, K = shape
    if not (Wp.dtype is torch.uint8 and Wp.get_device() == dev and Wp.is_contiguous() and
            Wp.numel() == _int4_nbytes(N, K, group, zeros)):
        raise ValueError("Wp must be a contiguous uint8 tensor on X's device of tri_int4_bytes(N, K, group, zeros) bytes for "
                         "X's width")
    Y = _new((M, N), half, X.device, stream) if out is None else out
    res = None
    if residual is not None:
        _need(residual.shape == (M, N) and _plain(residual, half, dev),
              "residual must be a contiguous (M, N) float16 tensor on X's device")
        res = residual.data_ptr()
    if not (Y.shape == (M, N) and Y.dtype is half and Y.get_device() == dev and Y.is_contiguous()):
        raise ValueError("out must be a contiguous (M, N) float16 tensor on X's device")
    _launch("tri_int4_linear", dev, stream, X.data_ptr(), Wp.data_ptr(), M, N, K, group, 1 if zeros else 0, res,
            Y.data_ptr())
    return Y


class Routing(collections.namedtuple("Routing", "ids weights offsets rows pos")):
    """What experts_route gives: ids, weights and pos (T, topk), offsets (E + 1), rows (T * topk)."""


def experts_route(logits, topk, renorm=True, workspace=None, out=None, stream=None):
    """The top-k experts of every row of (T, E) float16 or float32 logits, their weights, and the order of the (token,
    expert) pairs by expert, as a Routing (the tensors of `out`, if it is given).  `workspace`: a uint8 tensor of at
    least tri_experts_route_workspace_bytes(T, E, topk) bytes; allocated where it is None."""
    torch = _torch or _load_torch()
    dtype, dev, shape = logits.dtype, logits.get_device(), logits.shape
    _need(dev >= 0 and len(shape) == 2 and (dtype is torch.float16 or dtype is torch.float32) and logits.is_contiguous(),
          "logits must be a contiguous (T, E) float16 or float32 tensor on the GPU")
    T, E = shape
    need = _route_nbytes(T, E, topk)
    _need(need >= 0, "1 <= E <= %d, 1 <= topk <= min(E, %d) and T * topk < 2^31 are taken" % (TRI_MAX_EXPERTS, TRI_MAX_TOPK))
    i32 = torch.int32
    if out is None:
        out = Routing(*(_new(sh, torch.float32 if i == 1 else i32, logits.device, stream)
                        for i, sh in enumerate(((T, topk), (T, topk), (E + 1,), (T * topk,), (T, topk)))))
    ids, weights, offsets, rows, pos = out
    _need(_plain(ids, i32, dev) and _plain(weights, torch.float32, dev) and _plain(offsets, i32, dev) and
          _plain(rows, i32, dev) and _plain(pos, i32, dev) and ids.shape == weights.shape == pos.shape == (T, topk) and
          offsets.shape == (E + 1,) and rows.shape == (T * topk,),
          "out: ids, weights, pos (T, topk), offsets (E + 1), rows (T * topk); int32, the weights float32")
    if workspace is None and need > 0:
        workspace = _new(need, torch.uint8, logits.device, stream, result=False)
    ws, nbytes = None, 0
    if workspace is not None:
        _need(_plain(workspace, torch.uint8, dev), "workspace must be a contiguous uint8 tensor on the logits' device")
        ws, nbytes = workspace.data_ptr(), workspace.numel()
    _launch("tri_experts_route", dev, stream, logits.data_ptr(), TRI_F16 if dtype is torch.float16 else TRI_F32, T, E, topk,
            1 if renorm else 0, ids.data_ptr(), weights.data_ptr(), offsets.data_ptr(), rows.data_ptr(), pos.data_ptr(), ws,
            nbytes)
    return out


def _experts(name, X, offsets, rows, mats, K, fmt, out, stream):
    torch = _torch or _load_torch()
    half, i32, dev, shape = torch.float16, torch.int32, X.get_device(), X.shape
    _need(dev >= 0 and len(shape) == 2 and shape[1] == K and shape[0] > 0 and _plain(X, half, dev),
          "X must be a contiguous (T, K) float16 tensor on the GPU")
    T, wshape = shape[0], mats[0][0].shape
    _need(len(wshape) == 3 and wshape[2] == _row_nbytes(K, fmt), "weights must be (E, N, tri_row_bytes(K, fmt))")
    E, N = wshape[0], wshape[1]
    _need(_plain(offsets, i32, dev) and offsets.shape == (E + 1,), "offsets must be a contiguous (E + 1) int32 tensor on X's device")
    R, rp = T, None
    if rows is not None:
        _need(_plain(rows, i32, dev) and rows.dim() == 1, "rows must be a contiguous one-dimensional int32 tensor on X's device")
        R, rp = rows.shape[0], rows.data_ptr()
    Y = out if out is not None else _new((R, N), half, X.device, stream)
    _need(_plain(Y, half, dev) and Y.dim() == 2 and Y.shape[0] >= R and Y.shape[1] == N,
          "out must be a contiguous (R, N) float16 tensor on X's device")
    args = []
    for W, scale in mats:
        _need(_plain(W, torch.uint8, dev) and W.shape == wshape and _plain(scale, torch.float32, dev) and scale.numel() == E,
              "weights must be contiguous (E, N, tri_row_bytes(K, fmt)) uint8 tensors, scales (E) float32, on X's device")
        args += [W.data_ptr(), scale.data_ptr()]
    _launch(name, dev, stream, X.data_ptr(), T, offsets.data_ptr(), rp, R, *args, E, N, K, fmt, Y.data_ptr())
    return Y


def experts_linear(X, offsets, rows, Wp, scale, K, fmt, out=None, stream=None):
    """Y[r] = fp16(scale[e] * X[rows[r]] @ W_e.T) for the places r of expert e, offsets[e] <= r < offsets[e + 1] (rows
    None: X[r]).  Wp: (E, N, row_bytes) uint8, scale: (E) float32 on the device, offsets, rows: as experts_route gives
    them.  Rows of a new Y behind offsets[E] are not written; those of `out` stay as they are."""
    return _experts("tri_experts_linear", X, offsets, rows, ((Wp, scale),), K, fmt, out, stream)


def experts_pair(X, offsets, rows, Wp_gate, scale_gate, Wp_up, scale_up, K, fmt, out=None, stream=None):
    """experts_linear with two matrices per expert: Y[r] = fp16(silu(gate) * up)."""
    return _experts("tri_experts_pair", X, offsets, rows, ((Wp_gate, scale_gate), (Wp_up, scale_up)), K, fmt, out, stream)


def experts_combine(Z, pos, weights, residual=None, out=None, stream=None):
    """Y[t] = fp16(residual[t] + sum_j weights[t, j] * Z[pos[t, j]]); pairs with pos outside Z are left out.  `residual`
    may be `out` itself."""
    torch = _torch or _load_torch()
    half, dev, shape, pshape = torch.float16, Z.get_device(), Z.shape, pos.shape
    if not (len(shape) == 2 and dev >= 0 and shape[0] > 0 and Z.dtype is half and Z.is_contiguous()):
        raise ValueError("Z must be a contiguous (R, N) float16 tensor on the GPU")
    if not (len(pshape) == 2 and pos.dtype is torch.int32 and pos.get_device() == dev and pos.is_contiguous() and
            weights.shape == pshape and weights.dtype is torch.float32 and weights.get_device() == dev and
            weights.is_contiguous()):
        raise ValueError("pos must be a contiguous (T, topk) int32 tensor on Z's device, weights a float32 one like it")
    (R, N), (T, topk) = shape, pshape
    Y = _new((T, N), half, Z.device, stream) if out is None else out
    res = None
    if residual is not None:
        if not (residual.shape == (T, N) and residual.dtype is half and residual.get_device() == dev and
                residual.is_contiguous()):
            raise ValueError("residual must be a contiguous (T, N) float16 tensor on Z's device")
        res = residual.data_ptr()
    if not (Y.shape == (T, N) and Y.dtype is half and Y.get_device() == dev and Y.is_contiguous()):
        raise ValueError("out must be a contiguous (T, N) float16 tensor on Z's device")
    _launch("tri_experts_combine", dev, stream, Z.data_ptr(), R, pos.data_ptr(), weights.data_ptr(), res, T, topk, N,
            Y.data_ptr())
    return Y


def experts_mlp(X, logits, topk, gate, up, down, fmt, renorm=True, residual=None, stream=None):
    """A gated MLP of experts: for every row of X, the weighted sum over its top-k experts of
    down(silu(gate(x)) * up(x)), plus `residual`.  gate, up and down are (packed weights, scales) as experts_pair and
    experts_linear take them, logits (T, E) as experts_route takes them.  Four launches or a few more, no waiting."""
    torch = _torch or _load_torch()
    (T, hidden), inner = X.shape, gate[0].shape[1]
    _need(logits.dim() == 2 and logits.shape[0] == T, "logits must have a row for every row of X")
    r = experts_route(logits, topk, renorm=renorm, stream=stream)
    H = _new((T * topk, inner), torch.float16, X.device, stream, result=False)
    Z = _new((T * topk, down[0].shape[1]), torch.float16, X.device, stream, result=False)
    experts_pair(X, r.offsets, r.rows, *gate, *up, hidden, fmt, out=H, stream=stream)
    experts_linear(H, r.offsets, None, *down, inner, fmt, out=Z, stream=stream)
    return experts_combine(Z, r.pos, r.weights, residual=residual, stream=stream)


# ---------------------------------------------------------------- heads and the 8-bit cache

def rotary_table(rows, dims, base=10000.0, device="cuda"):
    """Cosines and sines of positions 0 .. rows-1 for `dims` rotated values, a (rows, dims / 2, 2) float32 tensor: angle
    p * base^(-2 i / dims), taken in 64 bits."""
    torch = _torch or _load_torch()
    freq = base ** (-torch.arange(0, dims, 2, device=device, dtype=torch.float64) / dims)
    angle = torch.arange(rows, device=device, dtype=torch.float64)[:, None] * freq
    return torch.stack([torch.cos(angle), torch.sin(angle)], -1).float()


class Rotary:
    """How heads are normalised and rotated (tri_rotary); made once and kept.  table: as rotary_table gives it, or None (no
    rotation); gains: None, or the norm's fp16 gains of the sets of heads it will be used on, (queries, keys) for
    cache_append, each (dim) or None."""

    def __init__(self, table, gains=None, norm=True, eps=1e-5, interleaved=False):
        torch = _torch or _load_torch()
        if table is not None:
            _need(table.is_cuda and table.dim() == 3 and table.shape[0] > 0 and table.shape[2] == 2 and
                  table.dtype is torch.float32 and table.is_contiguous(),
                  "table must be a contiguous (rows, dims / 2, 2) float32 tensor on the GPU")
        self.table, self.gains, self.norm = table, None if gains is None else tuple(gains), bool(norm)
        for g in self.gains or ():
            _need(g is None or (g.is_cuda and g.dtype is torch.float16 and g.dim() == 1 and g.is_contiguous()),
                  "gains must be contiguous (dim) float16 tensors on the GPU")
        self._device = None if table is None else table.get_device()
        self._gains = [(0, 0, 0) if g is None else (g.data_ptr(), g.shape[0], g.get_device()) for g in self.gains or ()]
        rows, half = (0, 0) if table is None else table.shape[:2]
        self.struct = TriRotary(None if table is None else table.data_ptr(), rows, 2 * half, 1 if interleaved else 0,
                                1 if norm else 0, eps)
        self._ref = ctypes.addressof(self.struct)

    def _gain(self, i, n, dim, device):
        """The gain of set i of n as an address (0: none), checked."""
        if self._device != device and self._device is not None:
            raise ValueError("the rotation's table must be on the heads' device")
        if self.gains is None:
            return 0
        _need(len(self._gains) == n, "gains must be one for each set of heads")
        ptr, size, dev = self._gains[i]
        _need(ptr == 0 or (size == dim and dev == device), "gains must be (dim) tensors on the heads' device")
        return ptr


class KVCache:
    """The pages of an 8-bit cache (tri_cache): codes K (pages, heads, page, dim) and V (pages, heads, dim, page), uint8,
    scales (pages, heads) float32.  KVCache.empty makes a new one."""

    def __init__(self, K, V, K_scale, V_scale, fmt):
        torch = _torch or _load_torch()
        _need(K.is_cuda and K.dim() == 4, "K must be a (pages, heads, page, dim) tensor on the GPU")
        (pages, heads, page, dim), dev = K.shape, K.get_device()
        _need(dim in (64, 128, 256) and page in (16, 32, 64, 128), "dim must be 64, 128 or 256, page 16, 32, 64 or 128")
        _need(fmt in (TRI_KV_INT8, TRI_KV_E4M3), "fmt must be TRI_KV_INT8 or TRI_KV_E4M3")
        _need(V.shape == (pages, heads, dim, page) and K_scale.shape == V_scale.shape == (pages, heads),
              "V must be (pages, heads, dim, page), the scales (pages, heads)")
        _tensors(dev, torch.uint8, K=K, V=V)
        _tensors(dev, torch.float32, K_scale=K_scale, V_scale=V_scale)
        self.K, self.V, self.K_scale, self.V_scale, self.fmt = K, V, K_scale, V_scale, fmt
        self.pages, self.heads, self.page, self.dim, self.device = pages, heads, page, dim, dev
        self.struct = TriCache(K.data_ptr(), V.data_ptr(), K_scale.data_ptr(), V_scale.data_ptr(), pages, heads, dim, page, fmt)
        self._ref = ctypes.addressof(self.struct)

    @classmethod
    def empty(cls, pages, heads, dim, page=64, fmt=TRI_KV_INT8, device="cuda"):
        torch = _torch or _load_torch()
        K = torch.zeros((pages, heads, page, dim), dtype=torch.uint8, device=device)
        scales = torch.ones((2, pages, heads), dtype=torch.float32, device=device)
        return cls(K, torch.zeros((pages, heads, dim, page), dtype=torch.uint8, device=device), scales[0], scales[1], fmt)


class Sequences:
    """A batch of sequences with new tokens (tri_sequences): offsets (B + 1), lens (B) and table (B, width), int32 on the
    device, read when a call runs (so a step may change them in place, inside a captured graph as well).  max_new: the most
    new tokens of a sequence; max_len: the most tokens, new ones included (all that the table has room for, if None)."""

    def __init__(self, offsets, lens, table, max_new, max_len=None):
        torch = _torch or _load_torch()
        _need(table.is_cuda and table.dim() == 2 and table.numel() > 0, "table must be a (B, width) tensor on the GPU")
        (B, width), dev = table.shape, table.get_device()
        _tensors(dev, torch.int32, offsets=offsets, lens=lens, table=table)
        _need(offsets.shape == (B + 1,) and lens.shape == (B,), "offsets must be (B + 1), lens (B)")
        _need(max_new > 0 and (max_len is None or max_len > 0), "max_new and max_len must be at least 1")
        self.offsets, self.lens, self.table, self.device = offsets, lens, table, dev
        # a struct for every size of a page: calls of several threads on several caches may share the sequences
        self.structs = {page: TriSequences(offsets.data_ptr(), lens.data_ptr(), table.data_ptr(), B, width, max_new,
                                           min(page * width, (1 << 31) - 129) if max_len is None else max_len)
                        for page in (16, 32, 64, 128)}
        self._refs = {page: ctypes.addressof(s) for page, s in self.structs.items()}

    def _fit(self, cache):
        """The struct's address for a call on `cache`."""
        if self.device != cache.device:
            raise ValueError("the sequences must be on the cache's device")
        return self._refs[cache.page]


_pack_heads = struct.Struct("PPPqqi4x").pack     # tri_heads


def _heads_of(x, what, dim, device, T, heads):
    """Address and token stride of a (T, heads, dim) float16 tensor whose tokens may lie apart."""
    if (x.is_contiguous() and x.dtype is _torch.float16 and x.get_device() == device and x.shape == (T, heads, dim) and
            heads > 0):                          # (the usual case, in half the time)
        return x.data_ptr(), heads * dim
    shape, stride = x.shape, x.stride()
    if not (shape == (T, heads, dim) and x.dtype is _torch.float16 and x.get_device() == device and stride[2] == 1 and
            (stride[1] == dim or heads == 1) and heads > 0):
        raise ValueError("%s must be a (T, heads, dim) float16 tensor on device %d whose heads lie one after another" %
                         (what, device))
    return x.data_ptr(), stride[0] if T > 1 else heads * dim


def heads_rotate(xs, rotary, positions, out=None, stream=None):
    """The heads of every (T, heads, dim) float16 tensor of `xs` (queries and keys, of the same T tokens) normalised and
    rotated by their tokens' positions (T) int32, in one launch; returns a tuple of new tensors, or `out`, which may be `xs`
    itself.  Rows of a token whose position is outside the rotation's table are not written."""
    torch = _torch or _load_torch()
    _need(0 < len(xs) <= TRI_MAX_GROUPS and xs[0].dim() == 3 and xs[0].is_cuda, "xs must be 1 to 4 (T, heads, dim) tensors on the GPU")
    (T, _, dim), dev = xs[0].shape, xs[0].get_device()
    _need(_plain(positions, torch.int32, dev) and positions.shape == (T,), "positions must be a contiguous (T) int32 tensor on the heads' device")
    if out is None:
        out = tuple(_new(tuple(x.shape), torch.float16, x.device, stream) for x in xs)
    _need(len(out) == len(xs), "out must have a tensor for each of xs")
    hs = b""
    for i, x in enumerate(xs):
        _need(x.dim() == 3, "xs must be 1 to 4 (T, heads, dim) tensors on the GPU")
        H = x.shape[1]
        xp, xst = _heads_of(x, "xs", dim, dev, T, H)
        yp, yst = _heads_of(out[i], "out", dim, dev, T, H)
        hs += _pack_heads(xp, yp, rotary._gain(i, len(xs), dim, dev), xst, yst, H)
    _launch("tri_heads_rotate", dev, stream, hs, len(xs), T, dim, rotary._ref, positions.data_ptr())
    return tuple(out)


def cache_append(cache, seqs, K, V, rotary=None, Q=None, out=None, stream=None):
    """Round the new tokens' keys and values (T, heads, dim) to 8 bits, into the pages of their sequences.  With `rotary`, keys
    are normalised and rotated first; the queries Q (T, query heads, dim), if given, too, in the same launch: they are returned,
    in a new tensor or in `out`, which may be Q itself."""
    torch = _torch or _load_torch()
    dim, dev = cache.dim, cache.device
    T = K.shape[0]
    kp, ks = _heads_of(K, "K", dim, dev, T, cache.heads)
    vp, vs = _heads_of(V, "V", dim, dev, T, cache.heads)
    rot = gain = q = None
    if rotary is not None:
        rot, gain = rotary._ref, rotary._gain(1, 2, dim, dev)
    if Q is not None:
        _need(rotary is not None and Q.dim() == 3, "queries are (T, heads, dim), and taken with a rotation only")
        H = Q.shape[1]
        if out is None:
            out = _new(tuple(Q.shape), torch.float16, Q.device, stream)
        qp, qs = _heads_of(Q, "Q", dim, dev, T, H)
        op, os_ = _heads_of(out, "out", dim, dev, T, H)
        q = _pack_heads(qp, op, rotary._gain(0, 2, dim, dev), qs, os_, H)
    else:
        _need(out is None, "out is for queries")
    _launch("tri_cache_append", dev, stream, cache._ref, seqs._fit(cache), T, kp, ks, vp, vs, rot, gain or None, q)
    return out


def cache_attend_workspace_bytes(cache, seqs, T, heads, window=0, sinks=0):
    """What cache_attend needs as workspace for T new tokens of `heads` query heads (0: none)."""
    seqs._fit(cache)
    need = tri_cache_attend_workspace_bytes(cache.struct, seqs.structs[cache.page], T, heads, window, sinks)
    _need(need >= 0, "sizes that tri_cache_attend does not take")
    return need


def cache_attend(cache, seqs, Q, scale=None, window=0, sinks=0, workspace=None, out=None, stream=None):
    """Causal attention of the new tokens' queries Q (T, query heads, dim) over their sequences in the cache, where
    cache_append has put their own keys and values.  window > 0: a token sees the last `window` positions and the first
    `sinks`.  scale: dim ** -0.5 if None.  Returns (T, query heads, dim), a new tensor (rows of no sequence are not written) or
    `out`.  `workspace`: a uint8 tensor of at least cache_attend_workspace_bytes; allocated where it is None and needed."""
    torch = _torch or _load_torch()
    dim, dev = cache.dim, cache.device
    _need(Q.dim() == 3 and Q.shape[0] > 0, "Q must be a (T, heads, dim) tensor")
    T, H, _ = Q.shape
    qp, qs = _heads_of(Q, "Q", dim, dev, T, H)
    O = _new(tuple(Q.shape), torch.float16, Q.device, stream) if out is None else out
    op, os_ = _heads_of(O, "out", dim, dev, T, H)
    sref = seqs._fit(cache)
    ws, nbytes = None, 0
    if workspace is None:
        nbytes = _lib.tri_cache_attend_workspace_bytes(cache._ref, sref, T, H, window, sinks) if _lib else \
            cache_attend_workspace_bytes(cache, seqs, T, H, window, sinks)
        if nbytes > 0:
            workspace = _new(nbytes, torch.uint8, Q.device, stream, result=False)
    if workspace is not None:
        _need(_plain(workspace, torch.uint8, dev), "workspace must be a contiguous uint8 tensor on the cache's device")
        ws, nbytes = workspace.data_ptr(), workspace.numel()
    _launch("tri_cache_attend", dev, stream, cache._ref, sref, T, qp, qs, H, dim ** -0.5 if scale is None else scale, window,
            sinks, op, os_, ws, max(nbytes, 0))
    return O
