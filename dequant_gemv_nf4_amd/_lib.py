"""ctypes binding of libnf4.so.  Argument marshalling only: shapes and dtypes are
checked here so that errors name the Python argument; everything else (the
library's own checks, every kernel) happens behind the C ABI."""
import ctypes
import os

import torch  # loaded first so libnf4 binds to the HIP runtime torch already uses

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libnf4.so")

GROUP = 64
MAX_M = 32
MAX_K = 32768
PACK_NONFINITE = 1
PACK_SCALE_OVERFLOW = 2
EMBED_BAD_ID = 1
MX_BLOCK = 32
MOE_MAX_E = 512
MOE_BAD_ID = 1
LOSS_BAD_TARGET = 1
MOE_MLP_MAX_T = 64

_STATUS = {0: "NF4_OK", -1: "NF4_EINVAL", -2: "NF4_EALIGN", -3: "NF4_ERANGE",
           -4: "NF4_EDEVICE", -5: "NF4_ELAUNCH"}

_lib = None


class NF4Error(RuntimeError):
    def __init__(self, func, status, msg):
        super().__init__(f"{func}: {_STATUS.get(status, status)} ({msg})")
        self.status = status


def lib_path() -> str:
    return _LIB_PATH


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is not built; run __graft_entry__.build() "
                          "or python dequant_gemv_nf4_amd/build.py")
    L = ctypes.CDLL(_LIB_PATH)
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    L.nf4_pack.argtypes = [vp, i64, i64, vp, vp, vp, vp]
    L.nf4_unpack.argtypes = [vp, vp, i64, i64, vp, vp]
    L.nf4_gemv.argtypes = [vp, vp, i64, i64, vp, vp, vp]
    L.nf4_gemm_smallm.argtypes = [vp, vp, i64, i64, vp, i64, vp, vp]
    L.nf4_gemm_prefill.argtypes = [vp, vp, i64, i64, vp, i64, vp, vp]
    L.nf4_gemm_smallm_ws.argtypes = [vp, vp, i64, i64, vp, i64, vp, vp, i64, vp]
    L.nf4_gemm_smallm_workspace_bytes.argtypes = [i64, i64, i64]
    L.nf4_gemm_smallm_workspace_bytes.restype = ctypes.c_int64
    L.nf4_gemm_smallm_noalloc.argtypes = [vp, vp, i64, i64, vp, i64, vp, vp]
    L.nf4_gemm_smallm_noalloc.restype = ctypes.c_int
    L.nf4_gemm_smallm_noalloc_max_bytes.argtypes = []
    L.nf4_gemm_smallm_noalloc_max_bytes.restype = ctypes.c_int64
    L.nf4_gemm_prefill_ws.argtypes = [vp, vp, i64, i64, vp, i64, vp, vp, i64, vp]
    L.nf4_gemm_prefill_workspace_bytes.argtypes = [i64, i64, i64]
    L.nf4_gemm_prefill_workspace_bytes.restype = ctypes.c_int64
    L.nf4_embed.argtypes = [vp, vp, i64, i64, vp, i64, vp, vp, vp]
    L.nf4_ring_create.argtypes = [ctypes.POINTER(ctypes.c_void_p), vp, vp, i64, vp, vp]
    L.nf4_ring_gemm.argtypes = [vp, vp, vp, i64, i64, vp, i64, vp]
    L.nf4_ring_destroy.argtypes = [vp]
    L.nf4_ring_slot_bytes.argtypes = [i64, i64]
    L.nf4_ring_slot_bytes.restype = ctypes.c_int64
    ci = ctypes.c_int
    L.nf4_mx_pack.argtypes = [vp, ci, i64, i64, vp, vp, vp, vp]
    L.nf4_mx_unpack.argtypes = [vp, vp, i64, i64, vp, ci, vp]
    L.nf4_mx_gemm.argtypes = [vp, vp, i64, i64, vp, i64, vp, ci, vp]
    L.nf4_mx_gemm_packed.argtypes = [vp, vp, i64, i64, vp, vp, i64, vp, ci, vp]
    L.nf4_mx_gemm_grouped.argtypes = [vp, vp, i64, i64, i64, vp, vp, i64, vp, ci, vp]
    L.nf4_mx_gemm_grouped_grad.argtypes = [vp, vp, i64, i64, i64, vp, vp, i64, vp, ci, vp]
    L.nf4_moe_sort.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp, vp]
    L.nf4_moe_gather.argtypes = [vp, ci, vp, i64, i64, i64, vp, vp]
    L.nf4_moe_combine.argtypes = [vp, ci, vp, vp, i64, i64, i64, vp, vp]
    L.nf4_moe_combine_grad.argtypes = [vp, vp, ci, vp, vp, i64, i64, i64, vp, vp, vp]
    L.nf4_mx_linear.argtypes = [vp, vp, i64, i64, vp, i64, vp, ci, ci, vp, vp, ci, vp, vp]
    L.nf4_mx_linear_grad.argtypes = [vp, vp, i64, i64, vp, vp, ci, i64, vp, vp, vp, ci, vp, i64, vp]
    L.nf4_mx_linear_grad_workspace_bytes.argtypes = [i64, i64, i64]
    L.nf4_mx_linear_grad_workspace_bytes.restype = i64
    L.nf4_mx_cross_entropy.argtypes = [vp, vp, i64, i64, vp, vp, i64, vp, vp, vp, vp, ci, vp, i64, vp, vp]
    L.nf4_mx_cross_entropy_workspace_bytes.argtypes = [i64, i64, i64, ci]
    L.nf4_mx_cross_entropy_workspace_bytes.restype = i64
    L.nf4_moe_mlp.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, vp, vp, i64, i64, ci, vp, vp, ci, vp, i64, vp]
    L.nf4_moe_mlp_workspace_bytes.argtypes = [i64, i64, i64, ci, i64, i64]
    L.nf4_moe_mlp_workspace_bytes.restype = i64
    for f in (L.nf4_mx_linear, L.nf4_mx_linear_grad, L.nf4_mx_cross_entropy, L.nf4_moe_mlp):
        f.restype = ci
    for f in (L.nf4_mx_pack, L.nf4_mx_unpack, L.nf4_mx_gemm, L.nf4_mx_gemm_packed,
              L.nf4_mx_gemm_grouped, L.nf4_mx_gemm_grouped_grad, L.nf4_moe_sort,
              L.nf4_moe_gather, L.nf4_moe_combine, L.nf4_moe_combine_grad):
        f.restype = ci
    for f in (L.nf4_ring_create, L.nf4_ring_gemm, L.nf4_ring_destroy):
        f.restype = ctypes.c_int
    for f in (L.nf4_pack, L.nf4_unpack, L.nf4_gemv, L.nf4_gemm_smallm, L.nf4_gemm_smallm_ws,
              L.nf4_gemm_prefill, L.nf4_gemm_prefill_ws, L.nf4_embed):
        f.restype = ctypes.c_int
    L.nf4_codebook.argtypes = [ctypes.POINTER(ctypes.c_float)]
    L.nf4_codebook.restype = None
    L.nf4_strerror.argtypes = [ctypes.c_int]
    L.nf4_strerror.restype = ctypes.c_char_p
    _lib = L
    return L


def _check(func, status):
    if status != 0:
        raise NF4Error(func, status, _load().nf4_strerror(status).decode())


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(device, stream):
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _torch_stream(device, stream):
    """`stream` (a torch stream or a raw handle) as a torch stream of `device`."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = _stream(device, stream).value
    if not handle:  # a null handle makes torch take a stream of its pool
        return torch.cuda.default_stream(device)
    return torch.cuda.ExternalStream(handle, device=device)


def _empty(shape, dtype, device, stream):
    """An output of a call on `stream` (None: the current one), from that stream's
    memory: a block of another stream may still be in use by work queued there, and
    would be handed out again there while this stream still writes it.  So `stream=`
    is as a call under torch.cuda.stream(stream): outputs are its own, and inputs made
    elsewhere have to be ready on it and be kept (Tensor.record_stream) until it has
    used them."""
    if stream is None or torch.device(device).type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_torch_stream(device, stream)):
        return torch.empty(shape, dtype=dtype, device=device)


def _read(status, stream):
    """The value of a status word that a call on `stream` wrote (waits for it)."""
    if stream is None:
        return int(status.item())
    with torch.cuda.stream(_torch_stream(status.device, stream)):
        return int(status.item())


def _run(func, tensors, args, stream):
    """Call func(*args, stream) of the library on the tensors' device: `stream`, or that
    device's current one.  Small calls take less time than their marshalling, so
    the device is switched only where it is another one, and pointers and the
    stream go over as plain integers."""
    index = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"{func}: tensors on different devices: " + ", ".join(
                str(t.device) for t in tensors if t is not None))
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(index)
    else:
        stream = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    f = getattr(_lib or _load(), func)
    if torch.cuda.current_device() == index:
        status = f(*args, stream)
    else:
        with torch.cuda.device(index):
            status = f(*args, stream)
    if status:
        _check(func, status)


def _need(t, name, dtypes, ndim=None):
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and t.is_contiguous()
            and (ndim is None or t.dim() in ndim)):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() not in ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, has {t.dim()}")


_U16 = (torch.int16, torch.uint16)
_BF16 = (torch.bfloat16, torch.int16, torch.uint16)


def nf4_pack(W, codes, scales, dev_status=None, stream=None):
    """Quantize fp32 W [N][K] into codes uint8 [N][K/2] and scales (fp16 bits) [N][K/64]."""
    _need(W, "W", (torch.float32,), (2,))
    N, K = W.shape
    _need(codes, "codes", (torch.uint8,))
    _need(scales, "scales", _U16 + (torch.float16,))
    if dev_status is not None:
        _need(dev_status, "dev_status", (torch.int32,))
    with torch.cuda.device(W.device):
        _check("nf4_pack", _load().nf4_pack(_ptr(W), N, K, _ptr(codes), _ptr(scales),
                                            _ptr(dev_status), _stream(W.device, stream)))


def nf4_unpack(codes, scales, W_out, stream=None):
    """Dequantize to fp32 W_out [N][K] = fp32(L[c] * s)."""
    _need(W_out, "W_out", (torch.float32,), (2,))
    N, K = W_out.shape
    _need(codes, "codes", (torch.uint8,))
    _need(scales, "scales", _U16 + (torch.float16,))
    with torch.cuda.device(W_out.device):
        _check("nf4_unpack", _load().nf4_unpack(_ptr(codes), _ptr(scales), N, K, _ptr(W_out),
                                                _stream(W_out.device, stream)))


def _nk(codes, scales, K):
    N = codes.shape[0]
    if codes.numel() != N * K // 2:
        raise ValueError(f"codes has {codes.numel()} bytes, expected N*K/2 = {N * K // 2}")
    if scales.numel() != N * (K // GROUP):
        raise ValueError(f"scales has {scales.numel()} entries, expected N*K/64")
    return N


def nf4_gemv(codes, scales, x, y, stream=None):
    """y [N] (fp32) = dequant(codes, scales) . x, x bf16 [K]."""
    _need(codes, "codes", (torch.uint8,), (2,))
    _need(scales, "scales", _U16 + (torch.float16,))
    _need(x, "x", _BF16)
    _need(y, "y", (torch.float32,))
    K = x.numel()
    N = _nk(codes, scales, K)
    if y.numel() != N:
        raise ValueError("y must have N elements")
    with torch.cuda.device(x.device):
        _check("nf4_gemv", _load().nf4_gemv(_ptr(codes), _ptr(scales), N, K, _ptr(x), _ptr(y),
                                            _stream(x.device, stream)))


def nf4_gemm_smallm(codes, scales, X, Y, stream=None):
    """Y [M][N] (fp32) = X . dequant(codes, scales)^T, X bf16 [M][K], 1 <= M <= 32."""
    _need(codes, "codes", (torch.uint8,), (2,))
    _need(scales, "scales", _U16 + (torch.float16,))
    _need(X, "X", _BF16, (1, 2))
    _need(Y, "Y", (torch.float32,))
    M, K = (1, X.shape[0]) if X.dim() == 1 else X.shape
    N = _nk(codes, scales, K)
    if Y.numel() != M * N:
        raise ValueError("Y must have M*N elements")
    with torch.cuda.device(X.device):
        _check("nf4_gemm_smallm", _load().nf4_gemm_smallm(_ptr(codes), _ptr(scales), N, K,
                                                          _ptr(X), M, _ptr(Y),
                                                          _stream(X.device, stream)))


def smallm_workspace_bytes(N, K, M):
    """Bytes of workspace nf4_gemm_smallm_ws needs for (N, K, M); 0 = no split."""
    n = _load().nf4_gemm_smallm_workspace_bytes(int(N), int(K), int(M))
    if n < 0:
        raise ValueError(f"invalid shape N={N} K={K} M={M}")
    return int(n)


def nf4_gemm_smallm_ws(codes, scales, X, Y, workspace, stream=None):
    """nf4_gemm_smallm with a device workspace (uint8 tensor, counters zeroed
    before its first use; or None when smallm_workspace_bytes is 0)."""
    _need(codes, "codes", (torch.uint8,), (2,))
    _need(scales, "scales", _U16 + (torch.float16,))
    _need(X, "X", _BF16, (1, 2))
    _need(Y, "Y", (torch.float32,))
    M, K = (1, X.shape[0]) if X.dim() == 1 else X.shape
    N = _nk(codes, scales, K)
    if Y.numel() != M * N:
        raise ValueError("Y must have M*N elements")
    nbytes = 0
    if workspace is not None:
        _need(workspace, "workspace", (torch.uint8,))
        nbytes = workspace.numel()
    with torch.cuda.device(X.device):
        _check("nf4_gemm_smallm_ws", _load().nf4_gemm_smallm_ws(
            _ptr(codes), _ptr(scales), N, K, _ptr(X), M, _ptr(Y), _ptr(workspace), nbytes,
            _stream(X.device, stream)))


def noalloc_max_bytes():
    """Size of the library-owned scratch behind nf4_gemm_smallm_noalloc."""
    return int(_load().nf4_gemm_smallm_noalloc_max_bytes())


def nf4_gemm_smallm_noalloc(codes, scales, X, Y, stream=None):
    """nf4_gemm_smallm_ws with the library's own per-device scratch instead of a
    workspace: no allocation anywhere in the call.  Calls that overlap on one GPU
    race on that scratch."""
    _need(codes, "codes", (torch.uint8,), (2,))
    _need(scales, "scales", _U16 + (torch.float16,))
    _need(X, "X", _BF16, (1, 2))
    _need(Y, "Y", (torch.float32,))
    M, K = (1, X.shape[0]) if X.dim() == 1 else X.shape
    N = _nk(codes, scales, K)
    if Y.numel() != M * N:
        raise ValueError("Y must have M*N elements")
    with torch.cuda.device(X.device):
        _check("nf4_gemm_smallm_noalloc", _load().nf4_gemm_smallm_noalloc(
            _ptr(codes), _ptr(scales), N, K, _ptr(X), M, _ptr(Y), _stream(X.device, stream)))


# one workspace per (device, stream): calls sharing one must not overlap, and
# calls on one stream never do
_workspaces = {}
# Workspaces replaced by a larger one stay allocated for the life of the
# process: a HIP graph captured earlier still holds their address, and work
# already enqueued may still use them.  (Each replacement at least doubles the
# size, so the kept ones add up to less than the current one.)
_retired = []


def workspace_for(device, nbytes, stream=None):
    """A zero-initialised workspace of at least nbytes for calls on `stream`
    (default: the current stream) of `device`, kept and reused.  A new one is
    allocated and zeroed on that stream, so the zeroing is ordered before the
    call that receives it."""
    device = torch.device(device)
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    handle = _stream(device, stream).value
    key = (device.index, handle)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        size = max(nbytes, 1 << 16, 2 * ws.numel() if ws is not None else 0)
        ts = torch.cuda.current_stream(device) if stream is None else _torch_stream(device, stream)
        with torch.cuda.device(device), torch.cuda.stream(ts):
            new = torch.zeros(size, dtype=torch.uint8, device=device)
        if ws is not None:
            _retired.append(ws)
        _workspaces[key] = ws = new
    return ws


def nf4_gemm_prefill(codes, scales, X, Y, stream=None):
    """Y [M][N] (fp32) = X . dequant(codes, scales)^T, X bf16 [M][K], any M >= 1
    (M * K < 2^30), on the large-tile MFMA kernel."""
    _need(codes, "codes", (torch.uint8,), (2,))
    _need(scales, "scales", _U16 + (torch.float16,))
    _need(X, "X", _BF16, (1, 2))
    _need(Y, "Y", (torch.float32,))
    M, K = (1, X.shape[0]) if X.dim() == 1 else X.shape
    N = _nk(codes, scales, K)
    if Y.numel() != M * N:
        raise ValueError("Y must have M*N elements")
    with torch.cuda.device(X.device):
        _check("nf4_gemm_prefill", _load().nf4_gemm_prefill(_ptr(codes), _ptr(scales), N, K,
                                                            _ptr(X), M, _ptr(Y),
                                                            _stream(X.device, stream)))


def prefill_workspace_bytes(N, K, M):
    """Bytes of workspace nf4_gemm_prefill_ws needs for (N, K, M); 0 = no split."""
    n = _load().nf4_gemm_prefill_workspace_bytes(int(N), int(K), int(M))
    if n < 0:
        raise ValueError(f"invalid shape N={N} K={K} M={M}")
    return int(n)


def nf4_gemm_prefill_ws(codes, scales, X, Y, workspace, stream=None):
    """nf4_gemm_prefill with a device workspace (uint8 tensor, counters zeroed
    before its first use; or None when prefill_workspace_bytes is 0)."""
    _need(codes, "codes", (torch.uint8,), (2,))
    _need(scales, "scales", _U16 + (torch.float16,))
    _need(X, "X", _BF16, (1, 2))
    _need(Y, "Y", (torch.float32,))
    M, K = (1, X.shape[0]) if X.dim() == 1 else X.shape
    N = _nk(codes, scales, K)
    if Y.numel() != M * N:
        raise ValueError("Y must have M*N elements")
    nbytes = 0
    if workspace is not None:
        _need(workspace, "workspace", (torch.uint8,))
        nbytes = workspace.numel()
    with torch.cuda.device(X.device):
        _check("nf4_gemm_prefill_ws", _load().nf4_gemm_prefill_ws(
            _ptr(codes), _ptr(scales), N, K, _ptr(X), M, _ptr(Y), _ptr(workspace), nbytes,
            _stream(X.device, stream)))


def nf4_embed(codes, scales, K, ids, out, dev_status=None, stream=None):
    """out bf16 [T][K] = rows ids (int64 [T]) of dequant(codes, scales), rounded once."""
    _need(codes, "codes", (torch.uint8,), (2,))
    _need(scales, "scales", _U16 + (torch.float16,))
    _need(ids, "ids", (torch.int64,), (1,))
    _need(out, "out", _BF16, (2,))
    N = _nk(codes, scales, K)
    T = ids.numel()
    if tuple(out.shape) != (T, K):
        raise ValueError(f"out must be [T={T}][K={K}]")
    if dev_status is not None:
        _need(dev_status, "dev_status", (torch.int32,))
    with torch.cuda.device(codes.device):
        _check("nf4_embed", _load().nf4_embed(_ptr(codes), _ptr(scales), N, K, _ptr(ids), T,
                                              _ptr(out), _ptr(dev_status),
                                              _stream(codes.device, stream)))


def ring_slot_bytes(N, K):
    """Device bytes one CopyRing slot needs for an N x K packed matrix."""
    return int(_load().nf4_ring_slot_bytes(N, K))


class Ring:
    """CopyRing (nf4_ring_*): products over packed matrices in pinned host memory,
    streamed through two device slots of `slot_bytes` each.  Copies run on their
    own stream, products on `compute_stream` (default: the current stream)."""

    def __init__(self, slot_bytes, device, compute_stream=None, copy_stream=None):
        self.device = torch.device(device)
        self.slots = [torch.empty(slot_bytes, dtype=torch.uint8, device=self.device)
                      for _ in range(2)]
        self.compute_stream = compute_stream or torch.cuda.current_stream(self.device)
        self.copy_stream = copy_stream or torch.cuda.Stream(self.device)
        self._ring = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check("nf4_ring_create", _load().nf4_ring_create(
                ctypes.byref(self._ring), _ptr(self.slots[0]), _ptr(self.slots[1]), slot_bytes,
                ctypes.c_void_p(self.compute_stream.cuda_stream),
                ctypes.c_void_p(self.copy_stream.cuda_stream)))
        self._keep = []  # host buffers of enqueued copies, held until close()

    def gemm(self, host_codes, host_scales, X, Y):
        """Y [M][N] fp32 = X bf16 [M][K] . dequant(host_codes, host_scales)^T."""
        for t, n in ((host_codes, "host_codes"), (host_scales, "host_scales")):
            if t.device.type != "cpu" or not t.is_pinned() or not t.is_contiguous():
                raise ValueError(f"{n} must be a contiguous pinned host tensor")
        _need(X, "X", _BF16, (1, 2))
        _need(Y, "Y", (torch.float32,))
        M, K = (1, X.shape[0]) if X.dim() == 1 else X.shape
        N = _nk(host_codes, host_scales, K)
        if Y.numel() != M * N:
            raise ValueError("Y must have M*N elements")
        self._keep.append((host_codes, host_scales))
        with torch.cuda.device(self.device):
            _check("nf4_ring_gemm", _load().nf4_ring_gemm(
                self._ring, _ptr(host_codes), _ptr(host_scales), N, K, _ptr(X), M, _ptr(Y)))

    def close(self):
        if self._ring:
            with torch.cuda.device(self.device):
                st = _load().nf4_ring_destroy(self._ring)
            self._ring = ctypes.c_void_p()
            self._keep.clear()
            _check("nf4_ring_destroy", st)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def nf4_codebook():
    """The library's 16 fp32 NF4 levels (host call, no GPU needed)."""
    out = (ctypes.c_float * 16)()
    _load().nf4_codebook(out)
    return [float(v) for v in out]


# ---- allocation conveniences (torch allocates; the library is then called) ----
def empty_packed(N, K, device, stream=None):
    codes = _empty((N, K // 2), torch.uint8, device, stream)
    scales = _empty((N, K // GROUP), torch.int16, device, stream)
    return codes, scales


def pack(W, stream=None, check=True):
    """Allocate and fill (codes, scales) for W; with check=True raise on flagged groups."""
    N, K = W.shape
    codes, scales = empty_packed(N, K, W.device, stream)
    status = _empty(1, torch.int32, W.device, stream) if check else None
    nf4_pack(W, codes, scales, status, stream)
    if check:
        st = _read(status, stream)
        if st:
            raise ValueError(f"nf4_pack flagged groups: status bits {st:#x}")
    return codes, scales


def unpack(codes, scales, K, stream=None):
    W = _empty((codes.shape[0], K), torch.float32, codes.device, stream)
    nf4_unpack(codes, scales, W, stream)
    return W


def gemv(codes, scales, x, stream=None):
    y = _empty(codes.shape[0], torch.float32, x.device, stream)
    nf4_gemv(codes, scales, x, y, stream)
    return y


def embed(codes, scales, K, ids, stream=None):
    out = _empty((ids.numel(), K), torch.bfloat16, codes.device, stream)
    nf4_embed(codes, scales, K, ids, out, None, stream)
    return out


def gemm(codes, scales, X, stream=None):
    """Y = X . dequant(codes, scales)^T for any M: up to MAX_M rows on the
    small-batch kernels (with a kept workspace where K splits over workgroups),
    beyond that on the prefill tiles."""
    M = 1 if X.dim() == 1 else X.shape[0]
    Y = _empty((M, codes.shape[0]), torch.float32, X.device, stream)
    if M <= MAX_M:
        need = smallm_workspace_bytes(codes.shape[0], X.shape[-1], M)
        if need:
            nf4_gemm_smallm_ws(codes, scales, X, Y, workspace_for(X.device, need, stream), stream)
        else:
            nf4_gemm_smallm(codes, scales, X, Y, stream)
    else:
        need = prefill_workspace_bytes(codes.shape[0], X.shape[-1], M)
        if need:
            nf4_gemm_prefill_ws(codes, scales, X, Y, workspace_for(X.device, need, stream), stream)
        else:
            nf4_gemm_prefill(codes, scales, X, Y, stream)
    return Y


# ---- MXFP4 and experts ----
_DTYPE = {torch.float32: 0, torch.bfloat16: 1}
_FLOATS = tuple(_DTYPE)
_U8 = (torch.uint8,)
_I32 = (torch.int32,)
_F32 = (torch.float32,)


def _addr(t):
    return None if t is None else t.data_ptr()


def _mx_matrix(codes, scales, what="codes", ndim=2):
    """The sizes (.., N, K) of a packed MXFP4 matrix (a stack of them: ndim 3)."""
    _need(codes, what, _U8, (ndim,))
    _need(scales, "scales" if what == "codes" else "xscales", _U8, (ndim,))
    *lead, half = codes.shape
    if half % (MX_BLOCK // 2) or list(scales.shape) != lead + [half // (MX_BLOCK // 2)]:
        raise ValueError(f"{what} {tuple(codes.shape)} needs scales [..., K/{MX_BLOCK}] with "
                         f"K = {2 * half}, got {tuple(scales.shape)}")
    return lead + [2 * half]


def nf4_mx_pack(W, codes, scales, dev_status=None, stream=None):
    """Quantise W [N][K] (fp32 or bf16) into MXFP4 codes uint8 [N][K/2] and scales
    uint8 [N][K/32]."""
    _need(W, "W", _FLOATS, (2,))
    N, K = W.shape
    if _mx_matrix(codes, scales) != [N, K]:
        raise ValueError(f"codes must be [N][K/2] for W {tuple(W.shape)}")
    if dev_status is not None:
        _need(dev_status, "dev_status", _I32)
    _run("nf4_mx_pack", (W, codes, scales, dev_status),
         (W.data_ptr(), _DTYPE[W.dtype], N, K, codes.data_ptr(), scales.data_ptr(),
          _addr(dev_status)), stream)


def nf4_mx_unpack(codes, scales, W_out, stream=None):
    """W_out [N][K] (fp32 or bf16) = the values of a packed MXFP4 matrix."""
    _need(W_out, "W_out", _FLOATS, (2,))
    N, K = W_out.shape
    if _mx_matrix(codes, scales) != [N, K]:
        raise ValueError(f"W_out must be [N][K], has {tuple(W_out.shape)}")
    _run("nf4_mx_unpack", (codes, scales, W_out),
         (codes.data_ptr(), scales.data_ptr(), N, K, W_out.data_ptr(), _DTYPE[W_out.dtype]), stream)


def nf4_mx_gemm(codes, scales, X, Y, stream=None):
    """Y [M][N] (fp32 or bf16) = X . dequant(codes, scales)^T, X bf16 [M][K], any M >= 1."""
    N, K = _mx_matrix(codes, scales)
    _need(X, "X", _BF16, (1, 2))
    _need(Y, "Y", _FLOATS)
    M = 1 if X.dim() == 1 else X.shape[0]
    if X.shape[-1] != K:
        raise ValueError(f"X has {X.shape[-1]} columns, the matrix K = {K}")
    if Y.numel() != M * N:
        raise ValueError("Y must have M*N elements")
    _run("nf4_mx_gemm", (X, codes, scales, Y),
         (codes.data_ptr(), scales.data_ptr(), N, K, X.data_ptr(), M, Y.data_ptr(),
          _DTYPE[Y.dtype]), stream)


def nf4_mx_gemm_packed(codes, scales, xcodes, xscales, Y, stream=None):
    """Y [M][N] (fp32 or bf16) = dequant(xcodes, xscales) . dequant(codes, scales)^T."""
    N, K = _mx_matrix(codes, scales)
    M, KX = _mx_matrix(xcodes, xscales, "xcodes")
    _need(Y, "Y", _FLOATS)
    if KX != K:
        raise ValueError(f"xcodes has K = {KX}, codes K = {K}")
    if Y.numel() != M * N:
        raise ValueError("Y must have M*N elements")
    _run("nf4_mx_gemm_packed", (codes, scales, xcodes, xscales, Y),
         (codes.data_ptr(), scales.data_ptr(), N, K, xcodes.data_ptr(), xscales.data_ptr(), M,
          Y.data_ptr(), _DTYPE[Y.dtype]), stream)


def _grouped(func, codes, scales, rows, name, grad, offsets, out, out_name, stream):
    E, N, K = _mx_matrix(codes, scales, ndim=3)
    width, out_width = (N, K) if grad else (K, N)
    _need(rows, name, _BF16, (2,))
    _need(offsets, "offsets", _I32, (1,))
    _need(out, out_name, _FLOATS, (2,))
    R = rows.shape[0]
    if rows.shape[1] != width:
        raise ValueError(f"{name} must be [R][{width}], has {tuple(rows.shape)}")
    if tuple(out.shape) != (R, out_width):
        raise ValueError(f"{out_name} must be [{R}][{out_width}], has {tuple(out.shape)}")
    if offsets.numel() != E + 1:
        raise ValueError(f"offsets must have E + 1 = {E + 1} entries")
    _run(func, (rows, codes, scales, offsets, out),
         (codes.data_ptr(), scales.data_ptr(), E, N, K, rows.data_ptr(), offsets.data_ptr(), R,
          out.data_ptr(), _DTYPE[out.dtype]), stream)


def nf4_mx_gemm_grouped(codes, scales, X, offsets, Y, stream=None):
    """Y [R][N] (fp32 or bf16): rows offsets[e] .. offsets[e+1]-1 of X bf16 [R][K]
    times expert e's packed matrix, codes [E][N][K/2], scales [E][N][K/32]; rows from
    offsets[E] on are zero.  offsets: int32 [E+1] on the device."""
    _grouped("nf4_mx_gemm_grouped", codes, scales, X, "X", False, offsets, Y, "Y", stream)


def nf4_mx_gemm_grouped_grad(codes, scales, dY, offsets, dX, stream=None):
    """dX [R][K] (fp32 or bf16): the gradient of nf4_mx_gemm_grouped in its rows,
    from dY bf16 [R][N], N % 8 == 0."""
    _grouped("nf4_mx_gemm_grouped_grad", codes, scales, dY, "dY", True, offsets, dX, "dX", stream)


def nf4_moe_sort(experts, num_experts, offsets, order, place, dev_status=None, stream=None):
    """Sort the slots of experts (int64 [T][topk], -1: none) by expert: offsets int32
    [E+1], order int32 [T*topk] (slot of each row), place int32 [T][topk] (row of
    each slot; ~ marks slots without an expert, which come last)."""
    _need(experts, "experts", (torch.int64,), (2,))
    _need(offsets, "offsets", _I32, (1,))
    _need(order, "order", _I32, (1,))
    _need(place, "place", _I32, (2,))
    T, topk = experts.shape
    if offsets.numel() != num_experts + 1:
        raise ValueError(f"offsets must have E + 1 = {num_experts + 1} entries")
    if order.numel() != T * topk or place.shape != experts.shape:
        raise ValueError(f"order must have {T * topk} entries and place the shape of experts")
    if dev_status is not None:
        _need(dev_status, "dev_status", _I32)
    _run("nf4_moe_sort", (experts, offsets, order, place, dev_status),
         (experts.data_ptr(), T, topk, int(num_experts), offsets.data_ptr(), order.data_ptr(),
          place.data_ptr(), _addr(dev_status)), stream)


def _rows(place, per_token, per_row, weights=()):
    """(T, topk, H, dtype) of a row operator.  per_token and per_row: (name, tensor)
    pairs of one dtype, [T][H] and [T*topk][H]; weights: pairs of fp32 [T][topk]."""
    _need(place, "place", _I32, (2,))
    T, topk = place.shape
    first, ref = per_token[0]
    for pairs, n in ((per_token, T), (per_row, T * topk)):
        for name, t in pairs:
            _need(t, name, _FLOATS, (2,))
            rows, H = t.shape
            if rows != n or H != ref.shape[1]:
                raise ValueError(f"{name} must be [{n}][{ref.shape[1]}], has {tuple(t.shape)}")
            if t.dtype != ref.dtype:
                raise TypeError(f"{name} has dtype {t.dtype}, {first} {ref.dtype}")
    for name, t in weights:
        _need(t, name, _F32, (2,))
        if t.shape != place.shape:
            raise ValueError(f"{name} must have the shape of place, {tuple(place.shape)}")
    return T, topk, ref.shape[1], _DTYPE[ref.dtype]


def nf4_moe_gather(X, place, out, stream=None):
    """out [T*topk][H]: row place[t][j] = X[t], zeros for slots without an expert."""
    T, topk, H, dtype = _rows(place, (("X", X),), (("out", out),))
    _run("nf4_moe_gather", (X, place, out),
         (X.data_ptr(), dtype, place.data_ptr(), T, topk, H, out.data_ptr()), stream)


def nf4_moe_combine(Y, place, weights, out, stream=None):
    """out [T][H] = sum_j weights[t][j] * Y[place[t][j]] (weights None: plain sum)."""
    T, topk, H, dtype = _rows(place, (("out", out),), (("Y", Y),),
                              () if weights is None else (("weights", weights),))
    _run("nf4_moe_combine", (Y, place, weights, out),
         (Y.data_ptr(), dtype, place.data_ptr(), _addr(weights), T, topk, H, out.data_ptr()), stream)


def nf4_moe_combine_grad(dOut, Y, place, weights, dY, dweights, stream=None):
    """dY [T*topk][H] and dweights fp32 [T][topk] of nf4_moe_combine from dOut [T][H]."""
    T, topk, H, dtype = _rows(place, (("dOut", dOut),), (("Y", Y), ("dY", dY)),
                              (("weights", weights), ("dweights", dweights)))
    _run("nf4_moe_combine_grad", (dOut, Y, place, weights, dY, dweights),
         (dOut.data_ptr(), Y.data_ptr(), dtype, place.data_ptr(), weights.data_ptr(), T, topk, H,
          dY.data_ptr(), dweights.data_ptr()), stream)


def mx_pack(W, stream=None, check=True):
    """Allocate and fill MXFP4 (codes, scales) for W; with check=True raise on blocks
    that hold NaN or infinity (a host synchronisation)."""
    _need(W, "W", _FLOATS, (2,))
    N, K = W.shape
    if K % MX_BLOCK:
        raise ValueError(f"each block of {MX_BLOCK} along K needs scales of its own: K = {K}")
    dev = W.device
    codes = _empty((N, K // 2), torch.uint8, dev, stream)
    scales = _empty((N, K // MX_BLOCK), torch.uint8, dev, stream)
    status = _empty(1, torch.int32, dev, stream) if check else None
    _run("nf4_mx_pack", (W,), (W.data_ptr(), _DTYPE[W.dtype], N, K, codes.data_ptr(),
                               scales.data_ptr(), _addr(status)), stream)
    if check:
        st = _read(status, stream)
        if st:
            raise ValueError(f"nf4_mx_pack flagged blocks: status bits {st:#x}")
    return codes, scales


def mx_unpack(codes, scales, dtype=torch.float32, stream=None):
    W = _empty((codes.shape[0], 2 * codes.shape[1]), dtype, codes.device, stream)
    nf4_mx_unpack(codes, scales, W, stream)
    return W


def mx_gemm(codes, scales, X, out_dtype=torch.float32, stream=None):
    """Y [M][N] = X . dequant(codes, scales)^T for any M (a vector X: Y [N])."""
    shape = (X.shape[0], codes.shape[0]) if X.dim() == 2 else (codes.shape[0],)
    Y = _empty(shape, out_dtype, X.device, stream)
    nf4_mx_gemm(codes, scales, X, Y, stream)
    return Y


def mx_gemm_packed(codes, scales, xcodes, xscales, out_dtype=torch.float32, stream=None):
    Y = _empty((xcodes.shape[0], codes.shape[0]), out_dtype, codes.device, stream)
    nf4_mx_gemm_packed(codes, scales, xcodes, xscales, Y, stream)
    return Y


def mx_gemm_grouped(codes, scales, X, offsets, out_dtype=torch.float32, stream=None):
    Y = _empty((X.shape[0], codes.shape[1]), out_dtype, X.device, stream)
    nf4_mx_gemm_grouped(codes, scales, X, offsets, Y, stream)
    return Y


def mx_gemm_grouped_grad(codes, scales, dY, offsets, out_dtype=torch.float32, stream=None):
    dX = _empty((dY.shape[0], 2 * codes.shape[2]), out_dtype, dY.device, stream)
    nf4_mx_gemm_grouped_grad(codes, scales, dY, offsets, dX, stream)
    return dX


def moe_sort(experts, num_experts, stream=None, check=False):
    """(offsets, order, place) of experts int64 [T][topk]; see nf4_moe_sort.  An id that is
    neither -1 nor in [0, num_experts) counts as -1; with check=True it raises (a host
    synchronisation, so not under capture)."""
    _need(experts, "experts", (torch.int64,), (2,))
    dev = experts.device
    offsets = _empty(num_experts + 1, torch.int32, dev, stream)
    order = _empty(experts.numel(), torch.int32, dev, stream)
    place = _empty(experts.shape, torch.int32, dev, stream)
    status = _empty(1, torch.int32, dev, stream) if check else None
    T, topk = experts.shape
    _run("nf4_moe_sort", (experts,), (experts.data_ptr(), T, topk, int(num_experts), offsets.data_ptr(),
                                      order.data_ptr(), place.data_ptr(), _addr(status)), stream)
    if check:
        st = _read(status, stream)
        if st:
            raise ValueError(f"nf4_moe_sort flagged expert ids: status bits {st:#x}")
    return offsets, order, place


def moe_gather(X, place, stream=None):
    out = _empty((place.numel(), X.shape[-1]), X.dtype, X.device, stream)
    nf4_moe_gather(X, place, out, stream)
    return out


def moe_combine(Y, place, weights=None, stream=None):
    out = _empty((place.shape[0], Y.shape[-1]), Y.dtype, Y.device, stream)
    nf4_moe_combine(Y, place, weights, out, stream)
    return out


def moe_combine_grad(dOut, Y, place, weights, stream=None):
    """(dY, dweights) of moe_combine."""
    dY = _empty(Y.shape, Y.dtype, Y.device, stream)
    dw = _empty(place.shape, torch.float32, Y.device, stream)
    nf4_moe_combine_grad(dOut, Y, place, weights, dY, dw, stream)
    return dY, dw


# ---- fused forms of the MXFP4 products ----
ACTS = {None: 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4, "swiglu": 5, "geglu": 6}
GATED_ACTS = ("swiglu", "geglu")


def _act(act, N):
    """(the library's number of `act`, columns that it makes of N)."""
    if act not in ACTS:
        raise ValueError(f"act is {act!r}, expected one of {tuple(ACTS)}")
    if act not in GATED_ACTS:
        return ACTS[act], N
    if N % 2:
        raise ValueError(f"{act} gates one half of the rows with the other: N = {N} is odd")
    return ACTS[act], N // 2


def _like(t, name, shape, dtypes):
    _need(t, name, dtypes)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, has {tuple(t.shape)}")


# The conveniences below check what the caller gave and allocate the rest in the right
# shape, so each operator's call is in one function, without a second round of checks: for
# one token they take longer than the kernel.
def _linear_sizes(codes, scales, X, bias, act, residual, out_dtype):
    """(N, K, number of the act, leading sizes, columns of Y)."""
    N, K = _mx_matrix(codes, scales)
    number, cols = _act(act, N)
    _need(X, "X", _BF16, (1, 2))
    *lead, width = X.shape
    if width != K:
        raise ValueError(f"X has {width} columns, the matrix K = {K}")
    if bias is not None:
        _like(bias, "bias", (N,), _FLOATS)
    if residual is not None:
        _like(residual, "residual", (*lead, cols), (out_dtype,))
    return N, K, number, lead, cols


def _linear(codes, scales, N, K, X, lead, bias, number, residual, Y, Z, stream):
    _run("nf4_mx_linear", (X, codes, scales, Y, bias, residual, Z),
         (codes.data_ptr(), scales.data_ptr(), N, K, X.data_ptr(), lead[0] if lead else 1,
          _addr(bias), 0 if bias is None else _DTYPE[bias.dtype], number, _addr(residual),
          Y.data_ptr(), _DTYPE[Y.dtype], _addr(Z)), stream)


def nf4_mx_linear(codes, scales, X, Y, bias=None, act=None, residual=None, Z=None, stream=None):
    """Y [M][N] ([M][N/2] for a gated act; fp32 or bf16) = act(X . dequant(codes, scales)^T +
    bias) + residual; Z bf16 [M][N], if given, receives what the activation is taken of."""
    _need(Y, "Y", _FLOATS)
    N, K, number, lead, cols = _linear_sizes(codes, scales, X, bias, act, residual, Y.dtype)
    _like(Y, "Y", (*lead, cols), _FLOATS)
    if Z is not None:
        _like(Z, "Z", (*lead, N), _BF16)
    _linear(codes, scales, N, K, X, lead, bias, number, residual, Y, Z, stream)


def mx_linear(codes, scales, X, bias=None, act=None, residual=None, out_dtype=torch.bfloat16,
              keep_z=False, stream=None):
    """act(X . dequant(codes, scales)^T + bias) + residual for any number of rows; with keep_z
    (that, Z) for mx_linear_grad.  act: None, "relu", "silu", "gelu", "gelu_tanh", or "swiglu"
    and "geglu", where the matrix's first half of rows gates its second."""
    N, K, number, lead, cols = _linear_sizes(codes, scales, X, bias, act, residual, out_dtype)
    if out_dtype not in _DTYPE:
        raise TypeError(f"out_dtype is {out_dtype}, expected one of {_FLOATS}")
    Y = _empty((*lead, cols), out_dtype, X.device, stream)
    Z = _empty((*lead, N), torch.bfloat16, X.device, stream) if keep_z else None
    _linear(codes, scales, N, K, X, lead, bias, number, residual, Y, Z, stream)
    return (Y, Z) if keep_z else Y


def mx_linear_grad_workspace_bytes(N, K, M):
    """Bytes of workspace nf4_mx_linear_grad needs for (N, K, M); 0 = none."""
    n = _load().nf4_mx_linear_grad_workspace_bytes(int(N), int(K), int(M))
    if n < 0:
        raise ValueError(f"invalid shape N={N} K={K} M={M}")
    return int(n)


def _linear_grad_sizes(codes, scales, dY, Z, act):
    N, K = _mx_matrix(codes, scales)
    number, cols = _act(act, N)
    _need(dY, "dY", _BF16, (1, 2))
    *lead, width = dY.shape
    if width != cols:
        raise ValueError(f"dY has {width} columns, expected {cols}")
    if Z is not None or act is not None:
        _like(Z, "Z", (*lead, N), _BF16)
    return N, K, number, lead


def _linear_grad(codes, scales, N, K, dY, lead, Z, number, dZ, dbias, dX, workspace, stream):
    _run("nf4_mx_linear_grad", (dY, codes, scales, Z, dX, dZ, dbias, workspace),
         (codes.data_ptr(), scales.data_ptr(), N, K, dY.data_ptr(), _addr(Z), number,
          lead[0] if lead else 1, _addr(dZ), _addr(dbias), dX.data_ptr(), _DTYPE[dX.dtype],
          _addr(workspace), 0 if workspace is None else workspace.numel()), stream)


def nf4_mx_linear_grad(codes, scales, dY, Z, act, dX, dZ=None, dbias=None, workspace=None, stream=None):
    """dX [M][K] (fp32 or bf16), dZ bf16 [M][N] and dbias fp32 [N] of nf4_mx_linear from dY
    bf16 [M][N] ([M][N/2] gated) and the Z that it kept; N % 8 == 0.  Z and dZ may be None
    without an activation.  workspace: uint8, mx_linear_grad_workspace_bytes(N, K, M)."""
    N, K, number, lead = _linear_grad_sizes(codes, scales, dY, Z, act)
    _like(dX, "dX", (*lead, K), _FLOATS)
    if dZ is not None or act is not None:
        _like(dZ, "dZ", (*lead, N), _BF16)
    if dbias is not None:
        _like(dbias, "dbias", (N,), _F32)
    if workspace is not None:
        _need(workspace, "workspace", _U8)
    _linear_grad(codes, scales, N, K, dY, lead, Z, number, dZ, dbias, dX, workspace, stream)


def mx_linear_grad(codes, scales, dY, Z=None, act=None, out_dtype=torch.bfloat16, bias_grad=False,
                   stream=None):
    """(dX, dZ, dbias) of mx_linear; dbias is None unless bias_grad, dZ is dY itself without an
    activation.  The residual's gradient is dY."""
    N, K, number, lead = _linear_grad_sizes(codes, scales, dY, Z, act)
    if out_dtype not in _DTYPE:
        raise TypeError(f"out_dtype is {out_dtype}, expected one of {_FLOATS}")
    dev = dY.device
    dX = _empty((*lead, K), out_dtype, dev, stream)
    dZ = None if act is None else _empty((*lead, N), torch.bfloat16, dev, stream)
    dbias = _empty((N,), torch.float32, dev, stream) if bias_grad else None
    need = _load().nf4_mx_linear_grad_workspace_bytes(N, K, lead[0] if lead else 1)
    ws = _empty((need,), torch.uint8, dev, stream) if need > 0 else None
    _linear_grad(codes, scales, N, K, dY, lead, Z, number, dZ, dbias, dX, ws, stream)
    return dX, dY if act is None else dZ, dbias


def mx_cross_entropy_workspace_bytes(N, K, M, grad=False):
    """Bytes of workspace nf4_mx_cross_entropy needs for (N, K, M), with or without gradient."""
    n = _load().nf4_mx_cross_entropy_workspace_bytes(int(N), int(K), int(M), int(grad))
    if n < 0:
        raise ValueError(f"invalid shape N={N} K={K} M={M}")
    return int(n)


def _loss_sizes(codes, scales, X, targets, dloss):
    N, K = _mx_matrix(codes, scales)
    _need(X, "X", _BF16, (2,))
    M, width = X.shape
    if width != K:
        raise ValueError(f"X has {width} columns, the matrix K = {K}")
    _like(targets, "targets", (M,), (torch.int64,))
    if dloss is not None:
        _like(dloss, "dloss", (M,), _F32)
    return N, K, M


def _loss(codes, scales, N, K, X, targets, M, loss, lse, dloss, dX, workspace, dev_status, stream):
    _run("nf4_mx_cross_entropy", (X, codes, scales, targets, loss, lse, dloss, dX, workspace, dev_status),
         (codes.data_ptr(), scales.data_ptr(), N, K, X.data_ptr(), targets.data_ptr(), M,
          loss.data_ptr(), lse.data_ptr(), _addr(dloss), _addr(dX), 0 if dX is None else _DTYPE[dX.dtype],
          _addr(workspace), 0 if workspace is None else workspace.numel(), _addr(dev_status)), stream)


def nf4_mx_cross_entropy(codes, scales, X, targets, loss, lse, dloss=None, dX=None, workspace=None,
                         dev_status=None, stream=None):
    """loss and lse fp32 [M] of the logits X . dequant(codes, scales)^T (X bf16 [M][K]) at
    targets int64 [M], negative ones ignored; with dloss fp32 [M] the gradient dX [M][K]
    (fp32 or bf16).  workspace: uint8, mx_cross_entropy_workspace_bytes(N, K, M, dX is given)."""
    N, K, M = _loss_sizes(codes, scales, X, targets, dloss)
    _like(loss, "loss", (M,), _F32)
    _like(lse, "lse", (M,), _F32)
    if (dX is None) != (dloss is None):
        raise ValueError("dX and dloss are given together")
    if dX is not None:
        _like(dX, "dX", (M, K), _FLOATS)
    if workspace is not None:
        _need(workspace, "workspace", _U8)
    if dev_status is not None:
        _need(dev_status, "dev_status", _I32)
    _loss(codes, scales, N, K, X, targets, M, loss, lse, dloss, dX, workspace, dev_status, stream)


def mx_cross_entropy(codes, scales, X, targets, dloss=None, out_dtype=torch.bfloat16, stream=None,
                     check=False):
    """(loss, lse) of each row, or with the losses' gradients dloss (loss, lse, dX).  A target
    below 0 is ignored, and so is one of N or more; with check=True the latter raises (a host
    synchronisation, so not under capture)."""
    N, K, M = _loss_sizes(codes, scales, X, targets, dloss)
    if out_dtype not in _DTYPE:
        raise TypeError(f"out_dtype is {out_dtype}, expected one of {_FLOATS}")
    dev = X.device
    need = _load().nf4_mx_cross_entropy_workspace_bytes(N, K, M, 0 if dloss is None else 1)
    loss = _empty((M,), torch.float32, dev, stream)
    lse = _empty((M,), torch.float32, dev, stream)
    dX = None if dloss is None else _empty((M, K), out_dtype, dev, stream)
    ws = _empty((max(need, 0),), torch.uint8, dev, stream)
    status = _empty(1, torch.int32, dev, stream) if check else None
    _loss(codes, scales, N, K, X, targets, M, loss, lse, dloss, dX, ws, status, stream)
    if check:
        st = _read(status, stream)
        if st:
            raise ValueError(f"nf4_mx_cross_entropy flagged targets: status bits {st:#x}")
    return (loss, lse) if dX is None else (loss, lse, dX)


def _mlp_sizes(codes1, scales1, codes2, scales2, act, X, experts, weights, residual, out_dtype):
    """(E, H, I, number of the act, T, topk) of an expert layer."""
    E, N1, H = _mx_matrix(codes1, scales1, ndim=3)
    E2, H2, I = _mx_matrix(codes2, scales2, ndim=3)
    number, cols = _act(act, N1)
    if E2 != E or H2 != H or I != cols:
        raise ValueError(f"codes1 {tuple(codes1.shape)} with act {act!r} needs codes2 of [E={E}][H={H}]"
                         f"[I/2={cols // 2}], got {tuple(codes2.shape)}")
    _need(X, "X", _BF16, (2,))
    T, width = X.shape
    if width != H:
        raise ValueError(f"X has {width} columns, the matrices H = {H}")
    if T > MOE_MLP_MAX_T:
        raise ValueError(f"moe_mlp takes up to {MOE_MLP_MAX_T} tokens, got {T}; sort the tokens (moe_sort) "
                         "and use the grouped products")
    _need(experts, "experts", (torch.int64,), (2,))
    rows, topk = experts.shape
    if rows != T:
        raise ValueError(f"experts must be [T={T}][topk], has {tuple(experts.shape)}")
    _like(weights, "weights", (T, topk), _F32)
    if residual is not None:
        _like(residual, "residual", (T, H), (out_dtype,))
    return E, H, I, number, T, topk


def moe_mlp_workspace_bytes(E, H, I, T, topk, act="swiglu"):
    """Bytes of workspace nf4_moe_mlp needs."""
    n = _load().nf4_moe_mlp_workspace_bytes(int(E), int(H), int(I), _act(act, 2)[0], int(T), int(topk))
    if n < 0:
        raise ValueError(f"invalid sizes E={E} H={H} I={I} T={T} topk={topk}")
    return int(n)


def _mlp(codes1, scales1, codes2, scales2, sizes, X, experts, weights, residual, out, workspace, stream):
    E, H, I, number, T, topk = sizes
    _run("nf4_moe_mlp", (X, codes1, scales1, codes2, scales2, experts, weights, residual, out, workspace),
         (codes1.data_ptr(), scales1.data_ptr(), codes2.data_ptr(), scales2.data_ptr(), E, H, I,
          X.data_ptr(), experts.data_ptr(), weights.data_ptr(), T, topk, number, _addr(residual),
          out.data_ptr(), _DTYPE[out.dtype], _addr(workspace),
          0 if workspace is None else workspace.numel()), stream)


def nf4_moe_mlp(codes1, scales1, codes2, scales2, X, experts, weights, out, act="swiglu", residual=None,
                workspace=None, stream=None):
    """out [T][H] (fp32 or bf16) = sum_j weights[t][j] W2[e] act(W1[e] X[t]) + residual[t] with e =
    experts[t][j] (int64; none outside [0, E)), X bf16 [T][H], at most MOE_MLP_MAX_T tokens; W1
    packed [E][2 I][H] ([E][I][H] for an act that does not gate), W2 packed [E][H][I].
    workspace: uint8, moe_mlp_workspace_bytes(E, H, I, T, topk, act)."""
    _need(out, "out", _FLOATS)
    sizes = _mlp_sizes(codes1, scales1, codes2, scales2, act, X, experts, weights, residual, out.dtype)
    _like(out, "out", X.shape, _FLOATS)
    if workspace is not None:
        _need(workspace, "workspace", _U8)
    _mlp(codes1, scales1, codes2, scales2, sizes, X, experts, weights, residual, out, workspace, stream)


def moe_mlp(codes1, scales1, codes2, scales2, X, experts, weights, act="swiglu", residual=None,
            out_dtype=torch.bfloat16, stream=None):
    """A whole layer of experts for up to MOE_MLP_MAX_T tokens; see nf4_moe_mlp."""
    sizes = _mlp_sizes(codes1, scales1, codes2, scales2, act, X, experts, weights, residual, out_dtype)
    if out_dtype not in _DTYPE:
        raise TypeError(f"out_dtype is {out_dtype}, expected one of {_FLOATS}")
    E, H, I, number, T, topk = sizes
    out = _empty((T, H), out_dtype, X.device, stream)
    need = _load().nf4_moe_mlp_workspace_bytes(E, H, I, number, T, topk)
    ws = _empty((max(need, 0),), torch.uint8, X.device, stream)
    _mlp(codes1, scales1, codes2, scales2, sizes, X, experts, weights, residual, out, ws, stream)
    return out
