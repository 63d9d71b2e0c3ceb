"""B200 (sm_100a) W4A16: 4-bit weight-only quantised linear layers with 16-bit activations.

Thin Python binding of the C ABI in include/w4a16.h.  The functions below carry the C
names, check each tensor's dtype and size, and marshal arguments: PyTorch provides
device memory, streams and output allocation; every step of the computation runs in
the library's CUDA kernels
(bit_weight_only_w4_b200/_lib/libw4a16.so, built in-tree by
``python -m bit_weight_only_w4_b200.build``).  There is no CPU fallback: if the library
is missing or a call fails, an exception is raised.

    qweight, scales, zeros = w4_quantize_pack(W, s, group_size=128)
    Y = w4a16_gemm(X, qweight, scales, zeros, group_size=128, s_inv=s_inv)

Calls run on the current stream, or on the one passed as ``stream``.  What they allocate comes
from that stream's pool, as under ``torch.cuda.stream(stream)``; their inputs have to be ready
on it.
"""
import contextlib
import ctypes
import os
import struct
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libw4a16.so")

W4_OK, W4_ERR_INVALID_ARG, W4_ERR_UNSUPPORTED, W4_ERR_CUDA, W4_ERR_TIMEOUT, W4_ERR_DEVICE_ARG = range(6)
W4_F16, W4_BF16, W4_F32 = 0, 1, 2
W4_FP4_NVFP4, W4_FP4_MXFP4 = 0, 1
FP4_BLOCK = {W4_FP4_NVFP4: 16, W4_FP4_MXFP4: 32}
W4_ACT_NONE, W4_ACT_RELU, W4_ACT_SILU, W4_ACT_GELU, W4_ACT_GELU_TANH = range(5)
W4_ROPE_PLAIN, W4_ROPE_LINEAR, W4_ROPE_BASE, W4_ROPE_BANDS, W4_ROPE_RAMP = range(5)
_ACTIVATIONS = {None: W4_ACT_NONE, "none": W4_ACT_NONE, "relu": W4_ACT_RELU, "silu": W4_ACT_SILU,
                "gelu": W4_ACT_GELU, "gelu_tanh": W4_ACT_GELU_TANH}
_ROPE_SCALINGS = {None: W4_ROPE_PLAIN, "plain": W4_ROPE_PLAIN, "linear": W4_ROPE_LINEAR,
                  "base": W4_ROPE_BASE, "bands": W4_ROPE_BANDS, "ramp": W4_ROPE_RAMP}

_lib = None
_lib_lock = threading.Lock()


class W4Error(RuntimeError):
    """A library call returned a status other than W4_OK."""

    def __init__(self, status, what):
        self.status = status
        super().__init__(f"{what}: {w4_status_string(status)}")


def lib():
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lib_lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"W4A16 CUDA library not found at {LIB_PATH}; build it with "
                "`python -m bit_weight_only_w4_b200.build` (nvcc, sm_100a)")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32, u64, sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32,
                                 ctypes.c_uint64, ctypes.c_size_t)
        st = ctypes.c_int
        L.w4_quantize_pack.argtypes = [vp, st, i64, i64, vp, i32, i32, vp, vp, vp, vp, vp]
        L.w4_quantize_pack.restype = st
        L.w4a16_gemm.argtypes = [vp, st, i64, i64, i64, vp, vp, vp, vp, i32, vp, vp, st, vp, sz, vp]
        L.w4a16_gemm.restype = st
        L.w4a16_gemm_noalloc.argtypes = [vp, st, i64, i64, i64, vp, vp, vp, vp, i32, vp, vp, st, vp]
        L.w4a16_gemm_noalloc.restype = st
        L.w4a16_workspace_bytes.argtypes = [i64, i64, i64, i32]
        L.w4a16_workspace_bytes.restype = sz
        L.w4_unpack_canonical.argtypes = [vp, i64, i64, vp, vp]
        L.w4_unpack_canonical.restype = st
        L.w4_check_device_error.argtypes = []
        L.w4_check_device_error.restype = st
        L.w4_stream_capture_id.argtypes = [vp, ctypes.POINTER(u64)]
        L.w4_stream_capture_id.restype = st
        L.w4_set_wait_limit_ns.argtypes = [u64]
        L.w4_set_wait_limit_ns.restype = st
        L.w4_selftest_noalloc_scratch.argtypes = [i32, ctypes.POINTER(u64)]
        L.w4_selftest_noalloc_scratch.restype = st
        L.w4_selftest_expired_wait.argtypes = [vp]
        L.w4_selftest_expired_wait.restype = st
        L.w4_status_string.argtypes = [st]
        L.w4_status_string.restype = ctypes.c_char_p
        L.w4_actorder_perm.argtypes = [vp, i64, i32, vp, vp]
        L.w4_actorder_perm.restype = st
        L.w4_quantize_pack_perm.argtypes = [vp, st, i64, i64, vp, i32, i32, vp, vp, vp, vp, vp]
        L.w4_quantize_pack_perm.restype = st
        L.w4a16_gemm_perm.argtypes = [vp, st, i64, i64, i64, vp, vp, vp, vp, i32, vp, vp, st, vp, sz, vp]
        L.w4a16_gemm_perm.restype = st
        L.w4a16_workspace_bytes_perm.argtypes = [i64, i64, i64, i32]
        L.w4a16_workspace_bytes_perm.restype = sz
        L.w4_awq_search.argtypes = [vp, st, i64, i64, vp, st, i64, i32, i32, i32, vp, vp, vp, vp, sz, vp]
        L.w4_awq_search.restype = st
        L.w4_awq_search_workspace_bytes.argtypes = [i64, i64, i64, i32, i32, i32]
        L.w4_awq_search_workspace_bytes.restype = sz
        L.w4_fp4_quantize_pack.argtypes = [vp, st, i64, i64, st, vp, vp, vp, vp]
        L.w4_fp4_quantize_pack.restype = st
        L.w4a16_fp4_gemm.argtypes = [vp, st, i64, i64, i64, vp, vp, vp, st, vp, st, vp, sz, vp]
        L.w4a16_fp4_gemm.restype = st
        L.w4a16_fp4_workspace_bytes.argtypes = [i64, i64, i64, st]
        L.w4a16_fp4_workspace_bytes.restype = sz
        L.w4a16_gemm_chain.argtypes = [ctypes.POINTER(ChainLayer), i32, i64, st, st, vp, sz, vp]
        L.w4a16_gemm_chain.restype = st
        L.w4a16_chain_workspace_bytes.argtypes = [i64]
        L.w4a16_chain_workspace_bytes.restype = sz
        L.w4a16_gemm_epi.argtypes = [vp, st, i64, i64, i64, vp, vp, vp, vp, vp, i32, vp,
                                     ctypes.POINTER(Epilogue), vp, st, vp, sz, vp]
        L.w4a16_gemm_epi.restype = st
        f32, f64 = ctypes.c_float, ctypes.c_double
        L.w4_rope.argtypes = [vp, st, i64, i32, i32, i64, i64, vp, vp, i32, f32, i32, vp, i64, i64, vp]
        L.w4_rope.restype = st
        L.w4_rope_freqs.argtypes = [i32, f64, st, f64, f64, f64, f64, ctypes.POINTER(f64), ctypes.POINTER(f32)]
        L.w4_rope_freqs.restype = st
        L.w4_prompt_attention.argtypes = [vp, st, vp, sz, vp]   # w4_attention: an Attention by reference, or its bytes
        L.w4_prompt_attention.restype = st
        L.w4_prompt_attention_workspace_bytes.argtypes = [i32, i32, i32, i32, i64, i64]
        L.w4_prompt_attention_workspace_bytes.restype = sz
        _lib = L
    return _lib


class ChainLayer(ctypes.Structure):
    """w4_chain_layer of include/w4a16.h."""
    _fields_ = [("X", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("qweight", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p), ("s_inv", ctypes.c_void_p),
                ("Y", ctypes.c_void_p), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("group_size", ctypes.c_int32)]


class Epilogue(ctypes.Structure):
    """w4_epilogue of include/w4a16.h."""
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("ldr", ctypes.c_int64),
                ("ldy", ctypes.c_int64), ("bias_dtype", ctypes.c_int), ("residual_dtype", ctypes.c_int),
                ("activation", ctypes.c_int), ("gated", ctypes.c_int32)]


class Attention(ctypes.Structure):
    """w4_attention of include/w4a16.h."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("Q", "K", "V", "O", "lse", "cu_seqlens_q", "cu_seqlens_k")]
                + [(n, ctypes.c_int64) for n in ("q_tokens", "k_tokens", "q_token_stride", "q_head_stride",
                                                 "k_token_stride", "k_head_stride", "v_token_stride",
                                                 "v_head_stride", "o_token_stride", "o_head_stride")]
                + [(n, ctypes.c_int32) for n in ("batch", "heads", "kv_heads", "head_dim")]
                + [("scale", ctypes.c_float), ("causal", ctypes.c_int32)])


_ATTENTION = struct.Struct("@7P10q4ifi")   # the same, packed
assert _ATTENTION.size == ctypes.sizeof(Attention)


# ---------------------------------------------------------------- marshalling helpers
def _torch():
    import torch
    return torch


def _dtype_code(dt):
    torch = _torch()
    if dt == torch.float16:
        return W4_F16
    if dt == torch.bfloat16:
        return W4_BF16
    if dt == torch.float32:
        return W4_F32
    raise TypeError(f"unsupported dtype {dt}")


def _ptr(t):
    # c_void_p arguments take a plain int (or None for NULL)
    return None if t is None else t.data_ptr()


def _stream_handle(stream, device):
    # the current stream's handle without building a torch.cuda.Stream (a call per layer and token)
    return stream.cuda_stream if stream is not None else _torch()._C._cuda_getCurrentRawStream(device.index)


_sizes = {}


def _workspace_size(index, fn, *args):
    """What a w4_*_workspace_bytes function of the library says for these sizes on device
    `index`, remembered (it depends on nothing else)."""
    key = (index, fn.__name__, args)
    need = _sizes.get(key)
    if need is None:
        if len(_sizes) >= 4096:
            _sizes.clear()
        need = _sizes[key] = _on_device(index, fn, *args)
    return need


def _on_device(index, fn, *args):
    """fn(*args) with CUDA device `index` current (the common case: it is already)."""
    torch = _torch()
    if torch._C._cuda_getDevice() == index:
        return fn(*args)
    with torch.cuda.device(index):
        return fn(*args)


def _allocating_on(stream, device):
    """Context in which tensors come from the pool of `stream` (None: of the current stream)."""
    if stream is None:
        return contextlib.nullcontext()
    torch = _torch()
    if not isinstance(stream, torch.cuda.Stream):   # any object with a cuda_stream handle
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    return torch.cuda.stream(stream)


def _new(like, shape, dtype, stream):
    """An uninitialised output on `like`'s device of a call on `stream`: from that stream's
    pool, whose memory no work queued on another stream still reads or writes.  The current
    stream, where the caller will read it, keeps it until its work is done."""
    if stream is None:
        return like.new_empty(shape) if dtype is like.dtype else like.new_empty(shape, dtype=dtype)
    with _allocating_on(stream, like.device):
        t = like.new_empty(shape, dtype=dtype)
    t.record_stream(_torch().cuda.current_stream(like.device))
    return t


def _check(status, what):
    if status != W4_OK:
        raise W4Error(status, what)


def _need_cuda(*tensors):
    dev = None
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors (there is no CPU path)")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("tensors are on different devices")
    return dev


def _expect(t, name, dtypes, shape=None, numel=None):
    """Refuse a tensor of the wrong dtype or size before its pointer reaches the library,
    which sees only the pointer and would read past a short buffer."""
    if t is None:
        return
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must hold {numel} elements, not {t.numel()}")


def _matrix(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix, not of shape {tuple(t.shape)}")
    return t.shape


def _groups(K, group_size):
    if group_size <= 0 or K % group_size != 0:
        raise ValueError(f"group_size {group_size} must divide K = {K}")
    return K // group_size


def _f16s():
    torch = _torch()
    return (torch.float16, torch.bfloat16)


def _words():
    torch = _torch()
    return (torch.int32, torch.uint32)


class _DeviceGuard:
    def __init__(self, device):
        self.device = device

    def __enter__(self):
        torch = _torch()
        self.prev = torch.cuda.current_device()
        self.switch = self.prev != self.device.index
        if self.switch:
            torch.cuda.set_device(self.device)

    def __exit__(self, *exc):
        if self.switch:
            _torch().cuda.set_device(self.prev)


# ---------------------------------------------------------------- C ABI, same names
def w4_status_string(status):
    return lib().w4_status_string(int(status)).decode()


def w4a16_workspace_bytes(M, N, K, group_size):
    return int(lib().w4a16_workspace_bytes(int(M), int(N), int(K), int(group_size)))


def w4_actorder_perm(g_idx, group_size, perm=None, stream=None):
    """perm int32 [K]: the channels sorted by g_idx (ties in channel order), for packing
    act-order weights with contiguous groups (every group must hold group_size channels;
    otherwise w4_check_device_error() reports W4_ERR_DEVICE_ARG)."""
    torch = _torch()
    if g_idx.dim() != 1:
        raise ValueError("g_idx must be a vector")
    K = g_idx.shape[0]
    _expect(g_idx, "g_idx", (torch.int32,))
    _expect(perm, "perm", (torch.int32,), numel=K)
    dev = _need_cuda(g_idx, perm)
    if perm is None:
        perm = _new(g_idx, K, torch.int32, stream)
    with _DeviceGuard(dev):
        st = lib().w4_actorder_perm(_ptr(g_idx), K, int(group_size), _ptr(perm), _stream_handle(stream, dev))
    _check(st, "w4_actorder_perm")
    return perm


def w4_awq_search(W, X, group_size=128, symmetric=False, n_grid=20, stream=None):
    """AWQ's scale search on the calibration rows X [M,K] for W [N,K] (both CUDA, fp16 or
    bf16): candidates s = m^a / geomean(m^a), m the mean |X| per channel, a = j / n_grid.
    Returns (best j, its exponent a, host float64 losses [n_grid], s_best float32 [K] on
    the device).  Synchronous."""
    torch = _torch()
    N, K = _matrix(W, "W")
    M, KX = _matrix(X, "X")
    if KX != K:
        raise ValueError(f"X has {KX} channels, W has {K}")
    _expect(W, "W", _f16s())
    _expect(X, "X", _f16s())
    dev = _need_cuda(W, X)
    s_best = _new(W, K, torch.float32, stream)
    losses = (ctypes.c_double * int(n_grid))()
    best = ctypes.c_int32(-1)
    with _DeviceGuard(dev):
        need = lib().w4_awq_search_workspace_bytes(M, N, K, int(group_size), int(bool(symmetric)), int(n_grid))
        if need == 0:
            raise ValueError("w4_awq_search: unsupported sizes")
        # a buffer of its own: the search writes over the front of its workspace, where the
        # cached GEMM workspace keeps the zero-filled split-K slots
        with _allocating_on(stream, dev):
            ws = torch.zeros(need, dtype=torch.uint8, device=dev)
        st = lib().w4_awq_search(_ptr(W), _dtype_code(W.dtype), N, K, _ptr(X), _dtype_code(X.dtype), M,
                                 int(group_size), int(bool(symmetric)), int(n_grid), _ptr(s_best),
                                 ctypes.addressof(losses), ctypes.addressof(best), _ptr(ws),
                                 ws.numel() * ws.element_size(), _stream_handle(stream, dev))
    _check(st, "w4_awq_search")
    import numpy as np
    return best.value, best.value / n_grid, np.array(losses[:], dtype=np.float64), s_best


def w4_quantize_pack(W, s=None, group_size=128, symmetric=False, g_idx=None,
                     qweight=None, scales=None, zeros=None, stream=None, perm=None):
    """AWQ scaling + group-wise RTN INT4 + packing of W [N,K] (fp16/bf16, CUDA).

    With perm (from w4_actorder_perm; g_idx then None) column k of the packed matrix is
    channel perm[k] and groups are contiguous.  Returns (qweight uint32-as-int32 [N*K/8]
    device layout, scales fp16 [G,N], zeros fp16 [G,N] or None when symmetric)."""
    torch = _torch()
    N, K = _matrix(W, "W")
    G = _groups(K, group_size)
    if perm is not None and g_idx is not None:
        raise ValueError("pass g_idx or perm, not both")
    _expect(W, "W", _f16s())
    _expect(s, "s", (torch.float32,), numel=K)
    _expect(g_idx, "g_idx", (torch.int32,), numel=K)
    _expect(perm, "perm", (torch.int32,), numel=K)
    _expect(qweight, "qweight", _words(), numel=N * K // 8)
    _expect(scales, "scales", (torch.float16,), shape=(G, N))
    _expect(zeros, "zeros", (torch.float16,), shape=(G, N))
    dev = _need_cuda(W, s, g_idx, qweight, scales, zeros, perm)
    if qweight is None:
        qweight = _new(W, N * K // 8, torch.int32, stream)
    if scales is None:
        scales = _new(W, (G, N), torch.float16, stream)
    if zeros is None and not symmetric:
        zeros = _new(W, (G, N), torch.float16, stream)
    with _DeviceGuard(dev):
        if perm is not None:
            st = lib().w4_quantize_pack_perm(_ptr(W), _dtype_code(W.dtype), N, K, _ptr(s), int(group_size),
                                             int(bool(symmetric)), _ptr(perm), _ptr(qweight),
                                             _ptr(scales), _ptr(zeros), _stream_handle(stream, dev))
        else:
            st = lib().w4_quantize_pack(_ptr(W), _dtype_code(W.dtype), N, K, _ptr(s), int(group_size),
                                        int(bool(symmetric)), _ptr(g_idx), _ptr(qweight),
                                        _ptr(scales), _ptr(zeros), _stream_handle(stream, dev))
    _check(st, "w4_quantize_pack")
    return qweight, scales, zeros


_ws_cache = {}      # (device index, stream handle): the buffer of eager calls on that stream
_ws_captured = {}   # (device index, stream handle): (capture, the buffer of the calls it recorded)
_ws_lock = threading.Lock()


def _capture_id(index, handle):
    """The number of the capture that records the stream's work, 0 while none does."""
    out = ctypes.c_uint64()
    _check(_on_device(index, lib().w4_stream_capture_id, handle, ctypes.byref(out)), "w4_stream_capture_id")
    return out.value


def workspace_for(device, nbytes, stream=None):
    """A scratch buffer of at least nbytes on `device`, zero-filled where the kernels want it
    so, for a call on `stream` (default: the current one) that passes no workspace of its own.

    Calls on one stream share a buffer: they follow one another on the GPU, also where it is
    outgrown and its memory goes back to that stream's pool.  Calls that a graph capture
    records share one that belongs to the graph (allocated within the capture, its split-K slots
    zeroed by every replay), and no later call takes that one.  So graphs may be replayed beside
    each other and beside eager calls (a layer sequence, w4a16_gemm_chain, wants the GPU's SMs to
    itself all the same)."""
    torch = _torch()
    device = torch.device(device)
    index = torch.cuda.current_device() if device.index is None else device.index
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    return _scratch(torch, device, index, handle, nbytes, stream)


def _scratch(torch, device, index, handle, nbytes, stream):
    key = (index, handle)
    buf = _ws_cache.get(key)
    # the common case, at little cost: an eager call on the current stream
    if buf is not None and buf.numel() >= nbytes and stream is None and torch._C._cuda_getDevice() == index \
            and not torch._C._cuda_isCurrentStreamCapturing():
        return buf
    capture = _capture_id(index, handle)
    with _ws_lock:
        if capture:
            owner, buf = _ws_captured.get(key, (0, None))
            if owner != capture:
                buf = None
        else:
            buf = _ws_cache.get(key)
        if buf is not None and buf.numel() >= nbytes:
            return buf
        nbytes = max(nbytes, 1 << 20)
        with _allocating_on(stream, device):
            if capture:
                # only the slots have to be zero (the activations behind them may be large)
                buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
                buf[:_workspace_size(index, lib().w4a16_workspace_bytes, 1, 16, 64, 64) or nbytes].zero_()
                _ws_captured[key] = (capture, buf)
            else:
                _ws_cache[key] = buf = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        return buf


_DTYPES = None


def _dtypes():
    """(float16, bfloat16, float32, int32, uint32), looked up once."""
    global _DTYPES
    if _DTYPES is None:
        torch = _torch()
        _DTYPES = (torch.float16, torch.bfloat16, torch.float32, torch.int32, torch.uint32)
    return _DTYPES


def _gemm_args(X, qweight, scales, zeros, group_size, g_idx, s_inv, Y, perm=None):
    """Shapes and dtypes of a GEMM call; returns (M, K, N), N taken from the scales.  A
    well-formed call passes one combined test (the decode path is called per token and
    per layer); any failure goes through the per-tensor checks, which name the culprit."""
    f16, bf16, f32, i32, u32 = _dtypes()
    xs, ss = X.shape, scales.shape
    if len(xs) == 2 and len(ss) == 2 and group_size > 0 and xs[1] % group_size == 0:
        M, K = xs
        N = ss[1]
        if ((X.dtype is f16 or X.dtype is bf16)
                and (qweight.dtype is i32 or qweight.dtype is u32) and qweight.numel() == N * K // 8
                and scales.dtype is f16 and ss[0] == K // group_size
                and (zeros is None or (zeros.dtype is f16 and zeros.shape == ss))
                and (g_idx is None or (g_idx.dtype is i32 and g_idx.numel() == K))
                and (s_inv is None or (s_inv.dtype is f32 and s_inv.numel() == K))
                and (perm is None or (perm.dtype is i32 and perm.numel() == K))
                and (Y is None or ((Y.dtype is f16 or Y.dtype is bf16 or Y.dtype is f32)
                                   and Y.shape == (M, N)))):
            return M, K, N
    _gemm_args_checked(X, qweight, scales, zeros, group_size, g_idx, s_inv, Y, perm)
    raise ValueError("inconsistent GEMM arguments")


def _gemm_args_checked(X, qweight, scales, zeros, group_size, g_idx, s_inv, Y, perm=None):
    torch = _torch()
    M, K = _matrix(X, "X")
    G = _groups(K, group_size)
    N = _matrix(scales, "scales")[1]
    _expect(X, "X", _f16s())
    _expect(qweight, "qweight", _words(), numel=N * K // 8)
    _expect(scales, "scales", (torch.float16,), shape=(G, N))
    _expect(zeros, "zeros", (torch.float16,), shape=(G, N))
    _expect(g_idx, "g_idx", (torch.int32,), numel=K)
    _expect(s_inv, "s_inv", (torch.float32,), numel=K)
    _expect(Y, "Y", _f16s() + (torch.float32,), shape=(M, N))
    _expect(perm, "perm", (torch.int32,), numel=K)


def w4a16_gemm(X, qweight, scales, zeros, group_size=128, g_idx=None, s_inv=None,
               out_dtype=None, Y=None, workspace=None, stream=None, perm=None):
    """Y[M,N] = (X * s_inv)[M,K] @ dequant(qweight, scales, zeros, g_idx)^T on the GPU.

    With perm, the weights were packed with that permutation (w4_quantize_pack(perm=...))
    and the activation columns are gathered through it (w4a16_gemm_perm).

    Without `workspace`, the calls on a stream share one cached zero-filled buffer, and those
    of a graph capture one that belongs to the graph (workspace_for).  A workspace of the
    caller's, torch.zeros(w4a16_workspace_bytes(...), dtype=torch.uint8, device=...), must not be
    shared by calls that may run at once (unordered streams, graphs replayed beside others)."""
    torch = _torch()
    M, K, N = _gemm_args(X, qweight, scales, zeros, group_size, g_idx, s_inv, Y, perm)
    if perm is not None and g_idx is not None:
        raise ValueError("pass g_idx or perm, not both")
    dev = _need_cuda(X, qweight, scales, zeros, g_idx, s_inv, Y, workspace, perm)
    out_dtype = out_dtype or X.dtype
    if Y is None:
        Y = _new(X, (M, N), out_dtype, stream)
    handle = _stream_handle(stream, dev)
    with _DeviceGuard(dev):
        if workspace is None and M > 0:
            size = lib().w4a16_workspace_bytes if perm is None else lib().w4a16_workspace_bytes_perm
            need = _workspace_size(dev.index, size, M, N, K, int(group_size))
            if need > 0:
                workspace = _scratch(torch, dev, dev.index, handle, need, stream)
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        if perm is not None:
            st = lib().w4a16_gemm_perm(_ptr(X), _dtype_code(X.dtype), M, N, K, _ptr(qweight), _ptr(scales),
                                       _ptr(zeros), _ptr(perm), int(group_size), _ptr(s_inv), _ptr(Y),
                                       _dtype_code(Y.dtype), _ptr(workspace), ws_bytes, handle)
        else:
            st = lib().w4a16_gemm(_ptr(X), _dtype_code(X.dtype), M, N, K, _ptr(qweight), _ptr(scales),
                                  _ptr(zeros), _ptr(g_idx), int(group_size), _ptr(s_inv), _ptr(Y),
                                  _dtype_code(Y.dtype), _ptr(workspace), ws_bytes, handle)
    _check(st, "w4a16_gemm_perm" if perm is not None else "w4a16_gemm")
    return Y


def w4a16_gemm_noalloc(X, qweight, scales, zeros, group_size=128, g_idx=None, s_inv=None,
                       out_dtype=None, Y=None, stream=None):
    """w4a16_gemm without a workspace, for callers that cannot allocate device memory at
    the point of the call: the library's fixed per-device scratch is used instead.  Only
    Y is allocated here, and only when not passed in."""
    torch = _torch()
    M, K, N = _gemm_args(X, qweight, scales, zeros, group_size, g_idx, s_inv, Y)
    dev = _need_cuda(X, qweight, scales, zeros, g_idx, s_inv, Y)
    out_dtype = out_dtype or X.dtype
    if Y is None:
        Y = _new(X, (M, N), out_dtype, stream)
    with _DeviceGuard(dev):
        st = lib().w4a16_gemm_noalloc(_ptr(X), _dtype_code(X.dtype), M, N, K, _ptr(qweight),
                                      _ptr(scales), _ptr(zeros), _ptr(g_idx), int(group_size),
                                      _ptr(s_inv), _ptr(Y), _dtype_code(Y.dtype),
                                      _stream_handle(stream, dev))
    _check(st, "w4a16_gemm_noalloc")
    return Y


def _fp4_format(fmt):
    if fmt in ("nvfp4", W4_FP4_NVFP4):
        return W4_FP4_NVFP4
    if fmt in ("mxfp4", W4_FP4_MXFP4):
        return W4_FP4_MXFP4
    raise ValueError(f"unknown FP4 format {fmt!r} (nvfp4 or mxfp4)")


def w4_fp4_quantize_pack(W, fmt="nvfp4", qweight=None, block_scales=None, tensor_scale=None,
                         stream=None):
    """Quantise W [N,K] (fp16/bf16) to NVFP4 or MXFP4.  Returns (qweight int32 [N*K/8]
    in the device layout, block_scales uint8 [K/B, N], tensor_scale fp32 [1] or None)."""
    torch = _torch()
    f = _fp4_format(fmt)
    B = FP4_BLOCK[f]
    _matrix(W, "W")
    _expect(W, "W", _f16s())
    N, K = W.shape
    if K % B != 0:
        raise ValueError(f"K = {K} must be a multiple of the block ({B})")
    _expect(qweight, "qweight", _words(), numel=N * K // 8)
    _expect(block_scales, "block_scales", (torch.uint8,), shape=(K // B, N))
    _expect(tensor_scale, "tensor_scale", (torch.float32,), numel=1)
    dev = _need_cuda(W, qweight, block_scales, tensor_scale)
    if qweight is None:
        qweight = _new(W, N * K // 8, torch.int32, stream)
    if block_scales is None:
        block_scales = _new(W, (K // B, N), torch.uint8, stream)
    if f == W4_FP4_NVFP4 and tensor_scale is None:
        tensor_scale = _new(W, 1, torch.float32, stream)
    if f == W4_FP4_MXFP4:
        tensor_scale = None
    with _DeviceGuard(dev):
        st = lib().w4_fp4_quantize_pack(_ptr(W), _dtype_code(W.dtype), N, K, f, _ptr(qweight),
                                        _ptr(block_scales), _ptr(tensor_scale), _stream_handle(stream, dev))
    _check(st, "w4_fp4_quantize_pack")
    return qweight, block_scales, tensor_scale


def w4a16_fp4_workspace_bytes(M, N, K, fmt="nvfp4"):
    return int(lib().w4a16_fp4_workspace_bytes(int(M), int(N), int(K), _fp4_format(fmt)))


def w4a16_fp4_gemm(X, qweight, block_scales, tensor_scale=None, fmt="nvfp4", out_dtype=None, Y=None,
                   workspace=None, stream=None):
    """Y = X @ What^T with NVFP4 / MXFP4 weights from w4_fp4_quantize_pack (fp16 X)."""
    torch = _torch()
    f = _fp4_format(fmt)
    B = FP4_BLOCK[f]
    _matrix(X, "X")
    _expect(X, "X", _f16s())
    M, K = X.shape
    if K % B != 0:
        raise ValueError(f"K = {K} must be a multiple of the block ({B})")
    N = block_scales.shape[1]
    _expect(qweight, "qweight", _words(), numel=N * K // 8)
    _expect(block_scales, "block_scales", (torch.uint8,), shape=(K // B, N))
    _expect(tensor_scale, "tensor_scale", (torch.float32,), numel=1)
    _expect(Y, "Y", (torch.float16, torch.bfloat16, torch.float32), shape=(M, N))
    dev = _need_cuda(X, qweight, block_scales, tensor_scale, Y, workspace)
    out_dtype = out_dtype or (Y.dtype if Y is not None else X.dtype)
    if Y is None:
        Y = _new(X, (M, N), out_dtype, stream)
    with _DeviceGuard(dev):
        need = w4a16_fp4_workspace_bytes(M, N, K, f) if M > 0 else 0
        if workspace is None and need > 0:
            workspace = _scratch(torch, dev, dev.index, _stream_handle(stream, dev), need, stream)
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        st = lib().w4a16_fp4_gemm(_ptr(X), _dtype_code(X.dtype), M, N, K, _ptr(qweight), _ptr(block_scales),
                                  _ptr(tensor_scale), f, _ptr(Y), _dtype_code(Y.dtype), _ptr(workspace),
                                  ws_bytes, _stream_handle(stream, dev))
    _check(st, "w4a16_fp4_gemm")
    return Y


def w4a16_chain_workspace_bytes(M):
    return int(lib().w4a16_chain_workspace_bytes(int(M)))


def w4a16_gemm_chain(layers, workspace=None, stream=None):
    """Run a list of small-batch GEMMs (M <= 8) in order, in one persistent launch per 32
    layers.  Each layer is a dict with X, qweight, scales, zeros, group_size, s_inv and Y
    (X [M,K] may be a view of an earlier layer's Y: rows may be further apart than K,
    elements must be contiguous).  Layer l+1 reads its X only after every earlier output
    is stored.  Outputs are written into the given Y tensors; returns the list of Ys.  The CTAs
    of a launch wait for one another, so no other work may hold SMs meanwhile: such a wait ends
    after the wait limit, and w4_check_device_error() reports it."""
    torch = _torch()
    n = len(layers)
    if n == 0:
        return []
    arr = (ChainLayer * n)()
    M = None
    act = None
    out = None
    devs = []
    for i, d in enumerate(layers):
        X, Y = d["X"], d["Y"]
        qw, sc, zr, s_inv = d["qweight"], d["scales"], d.get("zeros"), d.get("s_inv")
        g = int(d.get("group_size", 128))
        if X.dim() != 2 or Y.dim() != 2 or X.stride(1) != 1 or not Y.is_contiguous():
            raise ValueError(f"layer {i}: X must be a 2-D row-strided view, Y a contiguous matrix")
        m, K = X.shape
        N = Y.shape[1]
        if M is None:
            M, act, out = m, X.dtype, Y.dtype
        if m != M or Y.shape[0] != M or X.dtype != act or Y.dtype != out:
            raise ValueError(f"layer {i}: every layer has the same M, activation and output dtype")
        _expect(qw, "qweight", _words(), numel=N * K // 8)
        G = _groups(K, g)
        _expect(sc, "scales", _f16s(), shape=(G, N))
        _expect(zr, "zeros", _f16s(), shape=(G, N))
        _expect(s_inv, "s_inv", (torch.float32,), numel=K)
        if not X.is_cuda:
            raise ValueError("all tensors must be CUDA tensors (there is no CPU path)")
        devs += [Y, qw, sc, zr, s_inv]
        arr[i] = ChainLayer(_ptr(X), X.stride(0), _ptr(qw), _ptr(sc), _ptr(zr), _ptr(s_inv), _ptr(Y),
                            N, K, g)
    dev = _need_cuda(*devs, workspace)
    if any(d["X"].device != dev for d in layers):
        raise ValueError("tensors are on different devices")
    with _DeviceGuard(dev):
        need = w4a16_chain_workspace_bytes(M)
        if workspace is None and need > 0:
            workspace = _scratch(torch, dev, dev.index, _stream_handle(stream, dev), need, stream)
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        st = lib().w4a16_gemm_chain(arr, n, M, _dtype_code(act), _dtype_code(out), _ptr(workspace),
                                    ws_bytes, _stream_handle(stream, dev))
    _check(st, "w4a16_gemm_chain")
    return [d["Y"] for d in layers]


def w4_unpack_canonical(qweight, N, K, out=None, stream=None):
    torch = _torch()
    _expect(qweight, "qweight", _words(), numel=N * K // 8)
    _expect(out, "out", _words(), numel=N * K // 8)
    dev = _need_cuda(qweight, out)
    if out is None:
        out = _new(qweight, (N, K // 8), torch.int32, stream)
    with _DeviceGuard(dev):
        st = lib().w4_unpack_canonical(_ptr(qweight), int(N), int(K), _ptr(out),
                                       _stream_handle(stream, dev))
    _check(st, "w4_unpack_canonical")
    return out


def w4_check_device_error():
    """Synchronise the current device and raise if a kernel reported an error.  After a
    timeout the library zeroes its allocation-free scratch again, and this binding zeroes
    its cached workspaces of the current device (a kernel that gave up a wait may have left
    split-K flags in either; the workspaces of graphs are zeroed by every replay)."""
    st = lib().w4_check_device_error()
    if st == W4_ERR_TIMEOUT:
        torch = _torch()
        with _ws_lock:
            for (index, _), buf in _ws_cache.items():
                if index == torch.cuda.current_device():
                    buf.zero_()
            torch.cuda.synchronize()
    _check(st, "w4_check_device_error")


def w4_set_wait_limit_ns(ns):
    _check(lib().w4_set_wait_limit_ns(int(ns)), "w4_set_wait_limit_ns")


def w4_selftest_expired_wait(stream=None):
    torch = _torch()
    dev = torch.device("cuda", torch.cuda.current_device())
    _check(lib().w4_selftest_expired_wait(_stream_handle(stream, dev)), "w4_selftest_expired_wait")


# ---------------------------------------------------------------- around the projections
def gated_rows(F, device=None):
    """Row order of gated weights for w4a16_gemm_epi(gated=True): an index into the rows of
    [gate; up] ([2F, K], F a multiple of 8) that puts them in alternating blocks of 8, e.g.
    w4_quantize_pack(torch.cat([W_gate, W_up])[gated_rows(F)]); a bias is ordered the same."""
    torch = _torch()
    if F % 8 != 0:
        raise ValueError(f"F = {F} must be a multiple of 8")
    f = torch.arange(F, device=device).view(-1, 1, 8)
    return torch.cat([f, f + F], 1).reshape(-1)


def _rows_of(t, name, rows, cols):
    """The row stride of a [rows, cols] matrix whose elements are contiguous within rows
    (rows may be further apart)."""
    if t.dtype not in _dtypes()[:3]:
        raise TypeError(f"{name} must be torch.float16, torch.bfloat16 or torch.float32, not {t.dtype}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must have shape {(rows, cols)}, not {tuple(t.shape)}")
    ld, one = t.stride()
    if (cols > 1 and one != 1) or (rows > 1 and ld < cols):
        raise ValueError(f"{name}: elements of a row must be contiguous, and rows must not overlap")
    return ld if rows > 1 else cols


def w4a16_gemm_epi(X, qweight, scales, zeros, group_size=128, bias=None, activation=None, gated=False,
                   residual=None, g_idx=None, s_inv=None, out_dtype=None, Y=None, workspace=None,
                   stream=None, perm=None):
    """w4a16_gemm with an epilogue in the same kernel, applied in fp32 before the one rounding:

        t = (X * s_inv) @ dequant(...)^T + bias
        Y = act(t) + residual                        [M, N]
        Y = act(t_gate) * t_up + residual            [M, N/2], gated

    activation: None, "relu", "silu", "gelu" (erf) or "gelu_tanh".  gated: the packed rows (and
    bias) are in the order of gated_rows().  residual and Y may be row-strided views (rows on
    16-byte boundaries); residual may be Y itself.  Workspace rules as w4a16_gemm."""
    torch = _torch()
    M, K, N = _gemm_args(X, qweight, scales, zeros, group_size, g_idx, s_inv, None, perm)
    if perm is not None and g_idx is not None:
        raise ValueError("pass g_idx or perm, not both")
    act = _ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"unknown activation {activation!r} ({', '.join(k for k in _ACTIVATIONS if k)})")
    if bias is not None:
        _expect(bias, "bias", _dtypes()[:3], numel=N)
    index = X.get_device()
    for t in (X, qweight, scales, zeros, g_idx, s_inv, bias, workspace, perm):
        if t is not None and (t.get_device() != index or index < 0 or not t.is_contiguous()):
            _need_cuda(X, qweight, scales, zeros, g_idx, s_inv, bias, workspace, perm)   # names the reason
    n_out = N // 2 if gated else N
    xt = X.dtype
    if Y is None:
        yt = out_dtype or xt
        Y = _new(X, (M, n_out), yt, stream)
        ldy = n_out
    else:
        yt = Y.dtype
        if out_dtype is not None and out_dtype != yt:
            raise TypeError(f"Y is {yt}, out_dtype {out_dtype}")
        ldy = _rows_of(Y, "Y", M, n_out)
    ldr = 0 if residual is None else _rows_of(residual, "residual", M, n_out)
    if Y.get_device() != index or (residual is not None and residual.get_device() != index):
        raise ValueError("tensors are on different devices")
    e = Epilogue(_ptr(bias), _ptr(residual), ldr, ldy, 0 if bias is None else _dtype_code(bias.dtype),
                 0 if residual is None else _dtype_code(residual.dtype), act, 1 if gated else 0)
    L = lib()
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if workspace is None and M > 0:
        need = _workspace_size(index, L.w4a16_workspace_bytes if perm is None else L.w4a16_workspace_bytes_perm,
                               M, N, K, group_size)
        if need > 0:
            workspace = _scratch(torch, X.device, index, handle, need, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = _on_device(index, L.w4a16_gemm_epi, X.data_ptr(), _dtype_code(xt), M, N, K, qweight.data_ptr(),
                    scales.data_ptr(), _ptr(zeros), _ptr(g_idx), _ptr(perm), group_size, _ptr(s_inv), e, Y.data_ptr(),
                    _dtype_code(yt), _ptr(workspace), ws_bytes, handle)
    if st:
        raise W4Error(st, "w4a16_gemm_epi")
    return Y


def _heads_of(t, name):
    """(shape, strides) of a [tokens, heads, head_dim] CUDA tensor (a view with contiguous
    head elements)."""
    shape, strides = t.shape, t.stride()
    if len(shape) != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim], not of shape {tuple(shape)}")
    if strides[2] != 1 and shape[2] > 1:
        raise ValueError(f"{name}: elements of a head must be contiguous")
    return shape, strides


def _cuda_index(*tensors):
    """The index of the one CUDA device that the tensors (or None) are on."""
    index = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError("tensors are on different devices")
    if index < 0:
        raise ValueError("all tensors must be CUDA tensors (there is no CPU path)")
    return index


def w4_rope_freqs(rot_dim, theta=10000.0, scaling=None, factor=1.0, context=8192, lo=1.0, hi=4.0, device=None):
    """(inv_freq float64 [rot_dim/2], mscale) for w4_rope: theta^(-2i/rot_dim), stretched for
    contexts longer than `context` by scaling = "linear", "base", "bands" or "ramp" (see
    include/w4a16.h).  Computed on the host and copied to `device` (default: the current CUDA
    device): once per model."""
    torch = _torch()
    code = _ROPE_SCALINGS.get(scaling)
    if code is None:
        raise ValueError(f"unknown scaling {scaling!r} ({', '.join(k for k in _ROPE_SCALINGS if k)})")
    rot_dim = int(rot_dim)
    out = (ctypes.c_double * max(1, rot_dim // 2))()
    mscale = ctypes.c_float()
    _check(lib().w4_rope_freqs(rot_dim, float(theta), code, float(factor), float(context), float(lo), float(hi),
                               out, ctypes.byref(mscale)), "w4_rope_freqs")
    freqs = torch.tensor(out[:], dtype=torch.float64)
    return freqs.to(device if device is not None else "cuda"), mscale.value


def w4_rope(X, positions, inv_freq, interleaved=False, mscale=1.0, Y=None, stream=None):
    """Rotary positions on X [tokens, heads, head_dim] (fp16, bf16 or fp32; any view with
    contiguous head elements, e.g. the query and key heads of a fused projection's output):
    the first 2 * len(inv_freq) elements of each head are rotated by positions[t] *
    inv_freq[i], as pairs (i, i + len(inv_freq)) or, interleaved, (2i, 2i+1).  positions int32
    [tokens], inv_freq float64.  Y=X rotates in place; without Y a new tensor is returned."""
    torch = _torch()
    shape, sx = _heads_of(X, "X")
    T, H, D = shape
    if positions.dtype is not torch.int32 or positions.shape != (T,) or not positions.is_contiguous():
        _expect(positions, "positions", (torch.int32,), shape=(T,))
        raise ValueError("positions must be contiguous")
    if inv_freq.dtype is not torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        _expect(inv_freq, "inv_freq", (torch.float64,))
        raise ValueError("inv_freq must be a contiguous vector")
    rot = 2 * inv_freq.shape[0]
    if rot > D or rot == 0:
        raise ValueError(f"inv_freq must hold 1 .. {D // 2} frequencies, not {rot // 2}")
    xt = X.dtype
    if Y is None:
        index = _cuda_index(X, positions, inv_freq)
        Y = _new(X, shape, xt, stream)
        sy = (H * D, D)
    else:
        index = _cuda_index(X, positions, inv_freq, Y)
        ys, sy = _heads_of(Y, "Y")
        if Y.dtype is not xt or ys != shape:
            _expect(Y, "Y", (xt,), shape=shape)
    st = _on_device(index, lib().w4_rope, X.data_ptr(), _dtype_code(xt), T, H, D, sx[0], sx[1], positions.data_ptr(),
                    inv_freq.data_ptr(), rot, mscale, 1 if interleaved else 0, Y.data_ptr(), sy[0], sy[1],
                    torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream)
    if st:
        raise W4Error(st, "w4_rope")
    return Y


def w4_prompt_attention_workspace_bytes(batch, heads, kv_heads, head_dim, q_tokens, k_tokens):
    return int(lib().w4_prompt_attention_workspace_bytes(int(batch), int(heads), int(kv_heads), int(head_dim),
                                                         int(q_tokens), int(k_tokens)))


def w4_prompt_attention(Q, K, V, cu_seqlens=None, cu_seqlens_k=None, causal=True, scale=None, O=None,
                        return_lse=False, workspace=None, stream=None):
    """Softmax attention of packed sequences: Q [q_tokens, heads, head_dim], K and V
    [k_tokens, kv_heads, head_dim] (fp16 or bf16; views with contiguous head elements and
    strides of multiples of 8, e.g. slices of a fused projection's output), heads a multiple
    of kv_heads.  cu_seqlens int32 [batch+1]: the sequences' bounds in Q, cu_seqlens_k those in
    K and V when keys precede the queries; without them one sequence.  causal aligns the last
    query with the last key.  scale defaults to head_dim^-0.5.

    Returns O [q_tokens, heads, head_dim] (rows behind the last sequence are not written), and
    with return_lse also lse float32 [q_tokens, heads].

    Where a call needs scratch (w4_prompt_attention_workspace_bytes) and passes none, it is
    allocated for this call on the stream it runs on."""
    torch = _torch()
    (Tq, H, D), sq = _heads_of(Q, "Q")
    ks, sk = _heads_of(K, "K")
    vs, sv = _heads_of(V, "V")
    dt = Q.dtype
    if dt is not torch.float16 and dt is not torch.bfloat16:
        raise TypeError(f"Q must be torch.float16 or torch.bfloat16, not {dt}")
    if K.dtype is not dt or V.dtype is not dt:
        raise TypeError("Q, K and V must have one dtype")
    if ks != vs or ks[2] != D:
        raise ValueError(f"K and V must be [k_tokens, kv_heads, {D}], not {tuple(ks)} and {tuple(vs)}")
    Tk, Hk = ks[0], ks[1]
    batch = 1
    if cu_seqlens is not None:
        batch = cu_seqlens.shape[0] - 1 if cu_seqlens.dim() == 1 else -1
    for cu, name in ((cu_seqlens, "cu_seqlens"), (cu_seqlens_k, "cu_seqlens_k")):
        if cu is not None:
            if cu.dtype is not torch.int32:
                raise TypeError(f"{name} must be torch.int32, not {cu.dtype}")
            if cu_seqlens is None or batch < 0 or cu.shape != (batch + 1,) or not cu.is_contiguous():
                raise ValueError(f"{name} must be a contiguous vector of batch+1 bounds, cu_seqlens_k with a "
                                 "cu_seqlens of the same length")
    if scale is None:
        scale = D ** -0.5 if D > 0 else 1.0   # (heads without elements are refused by the library)
    index = _cuda_index(Q, K, V, cu_seqlens, cu_seqlens_k, O, workspace)
    if workspace is not None and not workspace.is_contiguous():   # (an expanded one holds less than it counts)
        raise ValueError("workspace must be contiguous")
    if O is None:
        O = _new(Q, (Tq, H, D), dt, stream)
        so = (H * D, D)
    else:
        os_, so = _heads_of(O, "O")
        if O.dtype is not dt or os_ != (Tq, H, D):
            _expect(O, "O", (dt,), shape=(Tq, H, D))
    lse = _new(Q, (Tq, H), torch.float32, stream) if return_lse else None
    # w4_attention, packed at once (a ctypes structure of 24 fields takes longer to fill)
    a = _ATTENTION.pack(Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), 0 if lse is None else lse.data_ptr(),
                        0 if cu_seqlens is None else cu_seqlens.data_ptr(),
                        0 if cu_seqlens_k is None else cu_seqlens_k.data_ptr(), Tq, Tk, sq[0], sq[1], sk[0], sk[1],
                        sv[0], sv[1], so[0], so[1], batch, H, Hk, D, scale,
                        1 if causal else 0)
    L = lib()
    if workspace is None:
        need = _workspace_size(index, L.w4_prompt_attention_workspace_bytes, batch, H, Hk, D, Tq, Tk)
        if need > 0:
            with _allocating_on(stream, Q.device):   # its next use is ordered behind this call
                workspace = Q.new_empty(need, dtype=torch.uint8)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = _on_device(index, L.w4_prompt_attention, a, _dtype_code(dt), _ptr(workspace), ws_bytes,
                    torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream)
    if st:
        raise W4Error(st, "w4_prompt_attention")
    return (O, lse) if return_lse else O
