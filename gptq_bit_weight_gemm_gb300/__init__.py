"""GB300 (sm_103a) GPTQ mixed-precision GEMM -- Python binding of the C ABI (include/gptq.h).

Argument marshalling only: every step of the computation runs in the CUDA library
``_lib/libgptq_gb300.so`` (built in-tree by ``build.py``).  PyTorch supplies device memory
and streams.  There is no fallback: if the library is missing or the device is not a GB300
(sm_103), calls raise ``GPTQError``.

Operations (page "增强 vLLM 对 GPTQv2 格式的支持：分析与实现", sections "LLM 的权重量化",
"从 GPTQv1 到 GPTQv2", "调整细节：根据格式选择处理方式"):

  gemm(A, qweight, qzeros, scales, g_idx, bits, group, fmt)  -> C = A @ dequant(W)
  dequant(qweight, qzeros, scales, g_idx, K, bits, group, fmt, dtype) -> W [K, N]
  quantize_rtn(W, bits, group, g_idx, sym, fmt)              -> (qweight, qzeros, scales)
  repack_zeros_v1_to_v2(qzeros_v1, N, bits)                  (host memory)
  prepack_act_order(qweight, g_idx, K, N, bits, group)      (host memory) -> (qweight', perm)
  prepack_act_order_device(qweight, g_idx, K, N, bits, group) (device memory) -> (qweight', perm)
  gemm_perm(A, perm, qweight', qzeros, scales, bits, group) -> A[:, perm] @ dequant(W'), M <= 32
  prepack_interleave(qweight, K, N, bits)                    (host memory) -> qweight in the decode
                                                             kernel's interleaved layout
  gemm_interleaved(A, qweight_il, qzeros, scales, perm, N, bits, group) -> the decode GEMM on it
  gemm_grouped(A, offsets, qweight[E], qzeros[E], scales[E], bits, group, max_m)
                                                             -> rows of expert e times W_e
  device_status(stream)                                      -> GPTQ_DEV_* bits

Beside the GEMMs, the rest of a decode step (include/gptq_serving.h):

  paged_attention(q, k_cache, v_cache, block_table, seq_lens) -> attention of one new token per sequence
                                                             (with k_new, v_new: appended first)
  moe_layer(x, router, up, down, topk, bits, group)          -> router, experts on packed weights and sum
  sample(logits, uniform, temperature, top_k, top_p, min_p)  -> (token, log probability) of each row

Every call on the device runs on `stream` (None: the current one).  With a stream that is not the current
one, the caller has its inputs ready there; what the call allocates (outputs, workspaces) belongs to it.
"""
import contextlib
import ctypes
import os
import re

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_lib", "libgptq_gb300.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "gptq.h")
SERVING_HEADER = os.path.join(os.path.dirname(HERE), "include", "gptq_serving.h")

F16, BF16, F32 = 0, 1, 2
V1, V2 = 1, 2
DEV_TIMEOUT, DEV_GIDX_RANGE, DEV_SCALE_OVERFLOW, DEV_EXPERT_ROWS, DEV_GIDX_GROUPS = 0x1, 0x2, 0x4, 0x8, 0x10
DEV_PAGE_RANGE, DEV_SEQ_LEN, DEV_NO_TOKEN = 0x20, 0x40, 0x80
DECODE_MAX_M = 32

_STATUS = {0: "GPTQ_OK", -1: "GPTQ_ERR_ARG", -2: "GPTQ_ERR_SHAPE", -3: "GPTQ_ERR_ALIGN",
           -4: "GPTQ_ERR_WORKSPACE", -5: "GPTQ_ERR_ZERO_OVERFLOW", -6: "GPTQ_ERR_CUDA",
           -7: "GPTQ_ERR_UNSUPPORTED", -8: "GPTQ_ERR_DEVICE"}


class GPTQError(RuntimeError):
    def __init__(self, code, what=""):
        self.code = code
        msg = "%s (%d)" % (_STATUS.get(code, "unknown"), code)
        try:
            msg = lib().gptq_strerror(code).decode()
        except Exception:
            pass
        super().__init__("%s%s" % (what + ": " if what else "", msg))


_lib = None

_P, _I, _SZ, _F, _LL = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float, ctypes.c_longlong
_Strides = _LL * 9
_SIGNATURES = {
    "gptq_dequant": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P]),
    "gptq_gemm": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "gptq_gemm_host": (_I, [_P, _P, _I, _I, _I, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _SZ, _P]),
    "gptq_host_plan_create": (_I, [ctypes.POINTER(ctypes.c_void_p), _P, _P, _I, _I, _I, _P, _P, _P, _P, _I, _I, _I,
                                   _I, _P, _P, _P, _SZ, _P]),
    "gptq_host_plan_run": (_I, [_P]),
    "gptq_host_plan_destroy": (_I, [_P]),
    "gptq_gemm_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
    "gptq_gemm_act_order_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
    "gptq_repack_zeros_v1_to_v2": (_I, [_P, _P, _I, _I, _I]),
    "gptq_quantize_rtn": (_I, [_P, _I, _I, _I, _I, _P, _I, _I, _P, _P, _P, _P]),
    "gptq_get_device_status": (_I, [_P, ctypes.POINTER(ctypes.c_uint)]),
    "gptq_strerror": (ctypes.c_char_p, [_I]),
    "gptq_selftest_wait_timeout": (_I, [ctypes.c_ulonglong, _P, _P]),
    "gptq_prepack_act_order": (_I, [_P, _P, _I, _I, _I, _I, _P, _P]),
    "gptq_prepack_act_order_device": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _P, _SZ, _P]),
    "gptq_prepack_act_order_device_workspace_size": (_SZ, [_I, _I, _I]),
    "gptq_gemm_perm": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "gptq_gemm_perm_workspace_size": (_SZ, [_I, _I]),
    "gptq_gemm_perm_noalloc": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P]),
    "gptq_gemm_grouped": (_I, [_P, _I, _I, _I, _P, _I, _I, _P, _P, _P, _I, _I, _I, _I, _P, _P]),
    "gptq_prepack_interleave": (_I, [_P, _I, _I, _I, _P]),
    "gptq_gemm_interleaved": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "gptq_paged_attention_workspace_size": (_SZ, [_I, _I, _I]),
    "gptq_paged_attention": (_I, [_P, _I, _I, _I, _P, _P, _I, _I, _I, _I, ctypes.POINTER(_LL), _P, _I, _P, _P, _P, _F, _I,
                                  _P, _P, _P, _SZ, _P]),
    "gptq_moe_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
    "gptq_moe": (_I, [_P, _I, _I, _I, _I, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _SZ, _P]),
    "gptq_sample": (_I, [_P, _I, _I, _LL, _I, _P, _P, _P, _P, _P, _P, _P, _P]),
}


def lib():
    """The loaded C library (ctypes).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("GPTQ CUDA library not built (%s): run "
                               "`python -c 'import __graft_entry__ as g; g.build()'`" % LIB_PATH)
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def header_functions(header=HEADER):
    """Names of the functions include/gptq.h (or another header) declares."""
    with open(header) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:int|size_t|const char\s*\*)\s+(gptq_\w+)\s*\(", text, re.M)))


def selftest_wait_timeout(limit_ns=50_000_000, stream=None):
    """Run the bounded-wait self-test; returns (waited_out, status bits)."""
    torch = _torch()
    with _on(stream):
        flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    _check(lib().gptq_selftest_wait_timeout(int(limit_ns), _ptr(flag), _stream(stream)),
           "gptq_selftest_wait_timeout")
    status = device_status(stream)
    return int(flag.item()), status


def _check(rc, what):
    if rc != 0:
        raise GPTQError(rc, what)


def _torch():
    import torch
    return torch


def _dtype_code(t):
    torch = _torch()
    if t.dtype == torch.float16:
        return F16
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError("activations must be float16 or bfloat16, got %s" % t.dtype)


def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _on(stream):
    """Within it, what a call allocates belongs to the stream that the call runs on: a fill precedes the
    kernels, and memory that is released when the call returns is not handed out to another stream
    while they use it."""
    return contextlib.nullcontext() if stream is None else _torch().cuda.stream(stream)


def _new(stream, like, shape, dtype=None):
    """An output for the caller, of like's device and (unless given) type.  The caller's current stream
    may use it as well."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with _on(stream):
        t = like.new_empty(shape, dtype=dtype)
    here = _torch().cuda.current_stream()
    if here != stream:
        t.record_stream(here)
    return t


def gemm(A, qweight, qzeros, scales, g_idx=None, *, bits, group, fmt=V2, out=None, workspace=None,
         sort_rows=True, stream=None):
    """C[M, N] = A[M, K] @ dequant(qweight, qzeros, scales, g_idx).  When no
    workspace is given one is allocated here: act-order (g_idx) with sort_rows, where the shape
    qualifies, takes act_order_workspace_size(...) bytes (rows sorted by group on the device);
    otherwise bf16 activations take workspace_size(...) bytes."""
    torch = _torch()
    M, K = A.shape
    N = qweight.shape[1]
    if out is None:
        out = _new(stream, A, (M, N))
    if workspace is None and M > 0:
        size = act_order_workspace_size(M, K, N, bits, group) if (g_idx is not None and sort_rows) else 0
        if size == 0 and A.dtype == torch.bfloat16:
            size = workspace_size(M, K, N, bits, group)
        if size:
            with _on(stream):
                workspace = torch.empty(size, dtype=torch.uint8, device=A.device)
    ws_ptr = _ptr(workspace, name="workspace") if workspace is not None else None
    ws_len = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = lib().gptq_gemm(_ptr(A, name="A"), M, K, _dtype_code(A),
                         _ptr(qweight, torch.int32, "qweight"), _ptr(qzeros, torch.int32, "qzeros"),
                         _ptr(scales, torch.float16, "scales"), _ptr(g_idx, torch.int32, "g_idx"),
                         N, bits, group, fmt, _ptr(out, A.dtype, "out"), ws_ptr, ws_len, _stream(stream))
    _check(rc, "gptq_gemm")
    return out


class HostGemm:
    """gptq_gemm_host prepared once, for a loop that reruns one problem on the same host and device
    buffers (only the contents of A_host change between calls): calling the object takes A_host
    [M, K] (a CPU tensor, page-locked for the direct path) into A_dev, computes C = A @ dequant(W)
    and returns C_host (a CPU tensor) once it holds the result.  On a named stream the call is
    captured into a CUDA graph (gptq_host_plan_create, which runs it once) and each call replays
    the graph; on the default stream each call is one gptq_gemm_host call with the arguments
    marshalled here.  The staging buffers and the workspace belong to the caller and must outlive
    the object (as for gemm, a bf16 prefill needs workspace_size(...) bytes)."""

    def __init__(self, A_host, A_dev, qweight, qzeros, scales, g_idx=None, *, bits, group, C_dev, C_host,
                 fmt=V2, workspace=None, stream=None):
        torch = _torch()
        M, K = A_host.shape
        N = qweight.shape[1]
        for t, name in ((A_host, "A_host"), (C_host, "C_host")):
            if t.is_cuda or not t.is_contiguous():
                raise ValueError("%s must be a contiguous CPU tensor" % name)
        if A_dev.dtype != A_host.dtype or C_dev.dtype != A_host.dtype or C_host.dtype != A_host.dtype:
            raise TypeError("A_host, A_dev, C_dev and C_host must share A's dtype")
        if A_dev.numel() < M * K or C_dev.numel() < M * N or C_host.numel() < M * N:
            raise ValueError("staging buffers smaller than the problem")
        ws_ptr = _ptr(workspace, name="workspace") if workspace is not None else None
        ws_len = workspace.numel() * workspace.element_size() if workspace is not None else 0
        # the tensors stay referenced for as long as the object can be called
        self._keep = (A_host, A_dev, qweight, qzeros, scales, g_idx, C_dev, C_host, workspace)
        self._args = (ctypes.c_void_p(A_host.data_ptr()), _ptr(A_dev, name="A_dev"), M, K, _dtype_code(A_host),
                      _ptr(qweight, torch.int32, "qweight"), _ptr(qzeros, torch.int32, "qzeros"),
                      _ptr(scales, torch.float16, "scales"), _ptr(g_idx, torch.int32, "g_idx"), N, bits, group,
                      fmt, _ptr(C_dev, name="C_dev"), ctypes.c_void_p(C_host.data_ptr()), ws_ptr, ws_len,
                      _stream(stream))
        self.C_host = C_host
        self._plan = None
        if self._args[-1].value:
            # a named stream: the call is captured once (gptq_host_plan_create, which also runs it
            # once) and each call replays the capture
            h = ctypes.c_void_p()
            _check(lib().gptq_host_plan_create(ctypes.byref(h), *self._args), "gptq_host_plan_create")
            self._plan = h
            self._run = lib().gptq_host_plan_run
        else:
            self._fn = lib().gptq_gemm_host

    def __call__(self):
        if self._plan is not None:
            _check(self._run(self._plan), "gptq_host_plan_run")
        else:
            _check(self._fn(*self._args), "gptq_gemm_host")
        return self.C_host

    def close(self):
        """Release the captured plan (also done when the object is collected)."""
        if getattr(self, "_plan", None) is not None and _lib is not None:
            lib().gptq_host_plan_destroy(self._plan)
        self._plan = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def gemm_host(A_host, A_dev, qweight, qzeros, scales, g_idx=None, *, bits, group, C_dev, C_host, fmt=V2,
              workspace=None, stream=None):
    """One gptq_gemm_host call: returns C_host holding C = A @ dequant(W) (HostGemm prepares the
    call for a loop over the same buffers)."""
    torch = _torch()
    M, K = A_host.shape
    N = qweight.shape[1]
    for t, name in ((A_host, "A_host"), (C_host, "C_host")):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("%s must be a contiguous CPU tensor" % name)
    if A_dev.dtype != A_host.dtype or C_dev.dtype != A_host.dtype or C_host.dtype != A_host.dtype:
        raise TypeError("A_host, A_dev, C_dev and C_host must share A's dtype")
    if A_dev.numel() < M * K or C_dev.numel() < M * N or C_host.numel() < M * N:
        raise ValueError("staging buffers smaller than the problem")
    ws_ptr = _ptr(workspace, name="workspace") if workspace is not None else None
    ws_len = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = lib().gptq_gemm_host(ctypes.c_void_p(A_host.data_ptr()), _ptr(A_dev, name="A_dev"), M, K,
                              _dtype_code(A_host), _ptr(qweight, torch.int32, "qweight"),
                              _ptr(qzeros, torch.int32, "qzeros"), _ptr(scales, torch.float16, "scales"),
                              _ptr(g_idx, torch.int32, "g_idx"), N, bits, group, fmt, _ptr(C_dev, name="C_dev"),
                              ctypes.c_void_p(C_host.data_ptr()), ws_ptr, ws_len, _stream(stream))
    _check(rc, "gptq_gemm_host")
    return C_host


def dequant(qweight, qzeros, scales, g_idx=None, *, K, bits, group, fmt=V2, dtype=None, out=None,
            stream=None):
    """W[K, N] = RN((q - zero) * scale) in `dtype` (float16 default)."""
    torch = _torch()
    dtype = torch.float16 if dtype is None else dtype
    N = qweight.shape[1]
    if out is None:
        out = _new(stream, qweight, (K, N), dtype)
    code = F16 if dtype == torch.float16 else BF16
    rc = lib().gptq_dequant(_ptr(qweight, torch.int32, "qweight"), _ptr(qzeros, torch.int32, "qzeros"),
                            _ptr(scales, torch.float16, "scales"), _ptr(g_idx, torch.int32, "g_idx"),
                            K, N, bits, group, fmt, code, _ptr(out, dtype, "out"), _stream(stream))
    _check(rc, "gptq_dequant")
    return out


def quantize_rtn(W, *, bits, group, g_idx=None, sym=False, fmt=V2, out=None, stream=None):
    """Round-to-nearest checkpoint of fp32 weights W [K, N]: (qweight, qzeros, scales), written
    into `out` = (qweight, qzeros, scales) when given."""
    torch = _torch()
    K, N = W.shape
    G = 1 if group == -1 else K // group
    if out is not None:
        qweight, qzeros, scales = out
    else:
        qweight = _new(stream, W, (K * bits // 32, N), torch.int32)
        qzeros = _new(stream, W, (G, N * bits // 32), torch.int32)
        scales = _new(stream, W, (G, N), torch.float16)
    if (tuple(qweight.shape) != (K * bits // 32, N) or tuple(qzeros.shape) != (G, N * bits // 32)
            or tuple(scales.shape) != (G, N)):
        raise ValueError("quantize_rtn: output buffers of the wrong shape")
    rc = lib().gptq_quantize_rtn(_ptr(W, torch.float32, "W"), K, N, bits, group,
                                 _ptr(g_idx, torch.int32, "g_idx"), int(bool(sym)), fmt,
                                 _ptr(qweight), _ptr(qzeros), _ptr(scales), _stream(stream))
    _check(rc, "gptq_quantize_rtn")
    return qweight, qzeros, scales


def repack_zeros_v1_to_v2(qzeros_v1, N, bits):
    """Host repack of v1 qzeros (numpy int32 [G, N*bits/32]) into a new v2 array."""
    src = np.ascontiguousarray(qzeros_v1, dtype=np.int32)
    out = np.empty_like(src)
    G = src.shape[0]
    rc = lib().gptq_repack_zeros_v1_to_v2(src.ctypes.data_as(_P), out.ctypes.data_as(_P), G, N, bits)
    _check(rc, "gptq_repack_zeros_v1_to_v2")
    return out


def prepack_act_order(qweight, g_idx, *, K, N, bits, group):
    """Host: sort an act-order checkpoint's rows by group.  qweight (numpy int32 [K*bits/32, N])
    and g_idx (numpy int32 [K]) -> (qweight_out, perm), with A @ W == A[:, perm] @ W_out."""
    qw = np.ascontiguousarray(qweight, dtype=np.int32)
    gi = np.ascontiguousarray(g_idx, dtype=np.int32)
    out = np.empty_like(qw)
    perm = np.empty(K, dtype=np.int32)
    rc = lib().gptq_prepack_act_order(qw.ctypes.data_as(_P), gi.ctypes.data_as(_P), K, N, bits, group,
                                      out.ctypes.data_as(_P), perm.ctypes.data_as(_P))
    _check(rc, "gptq_prepack_act_order")
    return out, perm


def prepack_act_order_device_workspace_size(K, bits, group):
    return int(lib().gptq_prepack_act_order_device_workspace_size(K, bits, group))


def prepack_act_order_device(qweight, g_idx, *, K, N, bits, group, workspace=None, stream=None):
    """Device: sort an act-order checkpoint's rows by group on `stream` (asynchronous).  qweight
    (int32 [K*bits/32, N]) and g_idx (int32 [K]) on the device -> (qweight_out, perm) on the
    device, bit-identical to prepack_act_order.  A g_idx whose groups are not all of `group` rows
    leaves both unwritten and sets DEV_GIDX_GROUPS in the device status word."""
    torch = _torch()
    ws_bytes = prepack_act_order_device_workspace_size(K, bits, group)
    if ws_bytes == 0:
        raise GPTQError(-2, "gptq_prepack_act_order_device")
    if workspace is None:
        with _on(stream):
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=qweight.device)
    out = _new(stream, qweight, qweight.shape)
    perm = _new(stream, qweight, (K,))
    rc = lib().gptq_prepack_act_order_device(_ptr(qweight, torch.int32, "qweight"), _ptr(g_idx, torch.int32, "g_idx"),
                                             K, N, bits, group, _ptr(out, torch.int32, "qweight_out"),
                                             _ptr(perm, torch.int32, "perm"), _ptr(workspace, name="workspace"),
                                             workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "gptq_prepack_act_order_device")
    return out, perm


def gemm_perm_workspace_size(M, K):
    return int(lib().gptq_gemm_perm_workspace_size(M, K))


def gemm_perm(A, perm, qweight, qzeros, scales, *, bits, group, fmt=V2, out=None, workspace=None,
              stream=None):
    """C[M, N] = A[:, perm] @ dequant(prepacked qweight), M <= 32.  For M > 1 a workspace of
    gemm_perm_workspace_size(M, K) bytes is used (allocated here when not given)."""
    torch = _torch()
    M, K = A.shape
    N = qweight.shape[1]
    if out is None:
        out = _new(stream, A, (M, N))
    ws_bytes = gemm_perm_workspace_size(M, K)
    if ws_bytes and workspace is None:
        with _on(stream):
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=A.device)
    ws_ptr = _ptr(workspace, name="workspace") if ws_bytes else None
    ws_len = workspace.numel() * workspace.element_size() if ws_bytes else 0
    rc = lib().gptq_gemm_perm(_ptr(A, name="A"), M, K, _dtype_code(A), _ptr(perm, torch.int32, "perm"),
                              _ptr(qweight, torch.int32, "qweight"), _ptr(qzeros, torch.int32, "qzeros"),
                              _ptr(scales, torch.float16, "scales"), N, bits, group, fmt,
                              _ptr(out, A.dtype, "out"), ws_ptr, ws_len, _stream(stream))
    _check(rc, "gptq_gemm_perm")
    return out


def prepack_interleave(qweight, *, K, N, bits):
    """Host: qweight (numpy int32 [K*bits/32, N]) in the decode kernel's interleaved layout."""
    qw = np.ascontiguousarray(qweight, dtype=np.int32)
    out = np.empty(qw.size, dtype=np.int32)
    rc = lib().gptq_prepack_interleave(qw.ctypes.data_as(_P), K, N, bits, out.ctypes.data_as(_P))
    _check(rc, "gptq_prepack_interleave")
    return out


def gemm_interleaved(A, qweight_il, qzeros, scales, perm=None, *, N, bits, group, fmt=V2, out=None,
                     workspace=None, stream=None):
    """C[M, N] = A @ dequant(W) (A[:, perm] @ ... with perm) for an interleaved qweight, M <= 32."""
    torch = _torch()
    M, K = A.shape
    if out is None:
        out = _new(stream, A, (M, N))
    ws_bytes = gemm_perm_workspace_size(M, K) if perm is not None else 0
    if ws_bytes and workspace is None:
        with _on(stream):
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=A.device)
    ws_ptr = _ptr(workspace, name="workspace") if ws_bytes else None
    ws_len = workspace.numel() * workspace.element_size() if ws_bytes else 0
    rc = lib().gptq_gemm_interleaved(_ptr(A, name="A"), M, K, _dtype_code(A), _ptr(perm, torch.int32, "perm"),
                                     _ptr(qweight_il, torch.int32, "qweight_il"), _ptr(qzeros, torch.int32, "qzeros"),
                                     _ptr(scales, torch.float16, "scales"), N, bits, group, fmt,
                                     _ptr(out, A.dtype, "out"), ws_ptr, ws_len, _stream(stream))
    _check(rc, "gptq_gemm_interleaved")
    return out


def gemm_grouped(A, offsets, qweight, qzeros, scales, *, bits, group, max_m, fmt=V2, out=None,
                 stream=None):
    """Mixture-of-experts GEMM: rows [offsets[e], offsets[e+1]) of A [rows, K] times expert e's
    weight, into the same rows of C [rows, N].  qweight [E, K*bits/32, N], qzeros
    [E, G, N*bits/32], scales [E, G, N] fp16; offsets [E+1] int32 on the device; every expert
    has at most max_m (<= 32) rows."""
    torch = _torch()
    rows, K = A.shape
    E, _, N = qweight.shape
    if out is None:
        out = _new(stream, A, (rows, N))
    rc = lib().gptq_gemm_grouped(_ptr(A, name="A"), rows, K, _dtype_code(A),
                                 _ptr(offsets, torch.int32, "offsets"), E, max_m,
                                 _ptr(qweight, torch.int32, "qweight"), _ptr(qzeros, torch.int32, "qzeros"),
                                 _ptr(scales, torch.float16, "scales"), N, bits, group, fmt,
                                 _ptr(out, A.dtype, "out"), _stream(stream))
    _check(rc, "gptq_gemm_grouped")
    return out


def workspace_size(M, K, N, bits, group):
    return int(lib().gptq_gemm_workspace_size(M, K, N, bits, group))


def act_order_workspace_size(M, K, N, bits, group):
    return int(lib().gptq_gemm_act_order_workspace_size(M, K, N, bits, group))


def device_status(stream=None):
    """Synchronize `stream`, read and clear the device status word (GPTQ_DEV_* bits)."""
    v = ctypes.c_uint(0)
    _check(lib().gptq_get_device_status(_stream(stream), ctypes.byref(v)), "gptq_get_device_status")
    return int(v.value)


def strerror(code):
    return lib().gptq_strerror(code).decode()


# ------------------------------------------------------------------ the rest of a decode step
# A decode step is tens of these calls, some of a few microseconds on the GPU, so each checks its
# tensors in one expression (attribute reads, about 0.1 us each) and calls the library; only where the
# expression fails are they looked at one by one, to say what is wrong.
class _Runtime:
    """What the calls below use of torch, looked up once."""

    def __init__(self):
        torch = _torch()
        self.int32, self.float32, self.float16 = torch.int32, torch.float32, torch.float16
        self.codes = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}
        self.lib = lib()
        raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
        if raw is None or device is None:
            self.stream = lambda: torch.cuda.current_stream().cuda_stream
        else:
            torch.cuda.init()
            self.stream = lambda: raw(device())


_rt = None


def _runtime():
    global _rt
    if _rt is None:
        _rt = _Runtime()
    return _rt


def _look(t, dtype, shape, name):
    """Raises what is wrong with a tensor that should be a contiguous CUDA tensor of this type and shape."""
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have the shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _address(t, dtype, shape, name):
    if not (t.is_cuda and t.dtype == dtype and t.shape == shape and t.is_contiguous()):
        _look(t, dtype, shape, name)
    return t.data_ptr()


def _buffer(nbytes, zeroed, what):
    if nbytes == 0:
        raise GPTQError(-2, what)
    make = _torch().zeros if zeroed else _torch().empty
    return make(nbytes, dtype=_torch().uint8, device="cuda")


def _workspace(t):
    """(address, bytes) of a workspace tensor."""
    if not (t.is_cuda and t.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return t.data_ptr(), t.nbytes


def paged_attention_workspace_size(heads, kv_heads, head_dim):
    return int(lib().gptq_paged_attention_workspace_size(heads, kv_heads, head_dim))


def paged_attention_workspace(heads, kv_heads, head_dim):
    """A workspace for paged_attention with these heads (zeroed, as its first use needs): kept by the
    caller and given to one call after the other on one stream, whatever their batch and lengths."""
    return _buffer(paged_attention_workspace_size(heads, kv_heads, head_dim), True, "gptq_paged_attention_workspace_size")


def _look_rows(t, dtype, shape, name):
    """Raises what is wrong with [batch, heads, dim] rows that should be contiguous within a sequence."""
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have the shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    stride = t.stride()
    if stride[2] != 1 or (shape[1] > 1 and stride[1] != shape[2]):
        raise ValueError("%s: the heads of a sequence must be contiguous" % name)


def _look_cache(t, dtype, shape, name):
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape or t.stride()[3] != 1:
        raise ValueError("%s must be [pages, page_size, kv_heads, dim] = %s with contiguous rows" % (name, tuple(shape)))


def paged_attention(q, k_cache, v_cache, block_table, seq_lens, *, scale=None, window=0, k_new=None, v_new=None,
                    out=None, lse=None, workspace=None, stream=None):
    """Attention of one new token of each sequence over a paged cache: q [batch, heads, dim],
    k_cache / v_cache [pages, page_size, kv_heads, dim] (views in any order of the first three, the
    last contiguous), block_table [batch, width] int32, seq_lens [batch] int32 -> out [batch, heads,
    dim].  k_new / v_new [batch, kv_heads, dim] are written to slot seq_lens - 1 first.  window > 0:
    only the last `window` keys.  scale: dim ** -0.5 where not given.  lse [batch, heads] fp32 takes
    the log of each row's exponential sum.  A workspace (paged_attention_workspace) is made here
    when none is given."""
    rt = _rt or _runtime()
    batch, heads, dim = shape = q.shape
    pages, page_size, kv_heads, _ = cache_shape = k_cache.shape
    dtype, i32 = q.dtype, rt.int32
    code = rt.codes.get(dtype, F32)
    if code == F32:
        raise TypeError("q must be float16 or bfloat16, got %s" % dtype)
    table_shape, lens_shape = block_table.shape, seq_lens.shape
    qs, ks, vs = q.stride(), k_cache.stride(), v_cache.stride()
    if not (q.is_cuda and qs[2] == 1 and (qs[1] == dim or heads == 1)):
        _look_rows(q, dtype, shape, "q")
    if not (k_cache.is_cuda and v_cache.is_cuda and k_cache.dtype == dtype and v_cache.dtype == dtype
            and v_cache.shape == cache_shape and cache_shape[3] == dim and ks[3] == 1 and vs[3] == 1):
        for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
            _look_cache(t, dtype, (pages, page_size, kv_heads, dim), name)
    if not (block_table.is_cuda and seq_lens.is_cuda and block_table.dtype == i32 and seq_lens.dtype == i32
            and len(table_shape) == 2 and table_shape[0] == batch and len(lens_shape) == 1 and lens_shape[0] == batch
            and block_table.is_contiguous() and seq_lens.is_contiguous()):
        if len(table_shape) != 2:
            raise ValueError("block_table must be [batch, width]")
        _look(block_table, i32, (batch, table_shape[1]), "block_table")
        _look(seq_lens, i32, (batch,), "seq_lens")
    kn = vn = None
    kn_stride = vn_stride = 0
    if k_new is not None or v_new is not None:
        if k_new is None or v_new is None:
            raise ValueError("k_new and v_new go together")
        new_shape = (batch, kv_heads, dim)
        ns, nv = k_new.stride(), v_new.stride()
        if not (k_new.is_cuda and v_new.is_cuda and k_new.dtype == dtype and v_new.dtype == dtype and k_new.shape == new_shape
                and v_new.shape == new_shape and ns[2] == 1 and nv[2] == 1 and ns[1] == dim and nv[1] == dim):
            _look_rows(k_new, dtype, new_shape, "k_new")
            _look_rows(v_new, dtype, new_shape, "v_new")
        kn, vn, kn_stride, vn_stride = k_new.data_ptr(), v_new.data_ptr(), ns[0], nv[0]
    if out is None:
        out = q.new_empty(shape) if stream is None else _new(stream, q, shape)
        out_ptr = out.data_ptr()
    else:
        out_ptr = _address(out, dtype, shape, "out")
    lse_ptr = None if lse is None else _address(lse, rt.float32, (batch, heads), "lse")
    if workspace is None:
        with _on(stream):
            workspace = paged_attention_workspace(heads, kv_heads, dim)
    ws, ws_bytes = _workspace(workspace)
    strides = _Strides(qs[0], kn_stride, vn_stride, ks[0], ks[1], ks[2], vs[0], vs[1], vs[2])
    rc = rt.lib.gptq_paged_attention(q.data_ptr(), batch, heads, code, k_cache.data_ptr(), v_cache.data_ptr(), pages, page_size,
                                     kv_heads, dim, strides, block_table.data_ptr(), table_shape[1], seq_lens.data_ptr(), kn, vn,
                                     dim ** -0.5 if scale is None else scale, window, out_ptr, lse_ptr, ws, ws_bytes,
                                     rt.stream() if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "gptq_paged_attention")
    return out


def moe_workspace_size(tokens, hidden, inter, experts, topk):
    return int(lib().gptq_moe_workspace_size(tokens, hidden, inter, experts, topk))


def moe_workspace(tokens, hidden, inter, experts, topk):
    """A workspace for moe_layer of this shape or any smaller one: kept by the caller and given to one
    call after the other on one stream."""
    return _buffer(moe_workspace_size(tokens, hidden, inter, experts, topk), False, "gptq_moe_workspace_size")


def moe_layer(x, router, up, down, *, topk, bits, group, fmt=V2, renormalize=True, out=None, workspace=None,
              return_routing=False, stream=None):
    """The mixture-of-experts layer for up to 32 tokens x [tokens, hidden]: the `topk` experts of the
    largest softmax(router x) (router [experts, hidden], equal ones by index), their weights
    renormalised over the chosen (renormalize), and the weighted sum of down(silu(gate x) * up x)
    over them.  up = (qweight [E, hidden*bits/32, 2*inter], qzeros, scales) holds the gate in its
    first `inter` columns, down = (qweight [E, inter*bits/32, hidden], qzeros, scales); layouts as
    for gemm_grouped.  Returns out [tokens, hidden], or (out, ids, weights) with return_routing.  A
    workspace (moe_workspace) is made here when none is given."""
    rt = _rt or _runtime()
    tokens, hidden = shape = x.shape
    experts = router.shape[0]
    uq, uz, us = up
    dq, dz, ds = down
    inter = uq.shape[2] // 2
    dtype, i32, f16 = x.dtype, rt.int32, rt.float16
    code = rt.codes.get(dtype, F32)
    if code == F32:
        raise TypeError("x must be float16 or bfloat16, got %s" % dtype)
    Gu, Gd = (1, 1) if group == -1 else (hidden // max(1, group), inter // max(1, group))
    if not (x.is_cuda and router.is_cuda and router.dtype == dtype and router.shape == (experts, hidden)
            and x.is_contiguous() and router.is_contiguous()):
        _look(x, dtype, shape, "x")
        _look(router, dtype, (experts, hidden), "router")
    if not (uq.is_cuda and uz.is_cuda and us.is_cuda and dq.is_cuda and dz.is_cuda and ds.is_cuda
            and uq.dtype == i32 and uz.dtype == i32 and us.dtype == f16 and dq.dtype == i32 and dz.dtype == i32 and ds.dtype == f16
            and uq.shape == (experts, hidden * bits // 32, 2 * inter) and uz.shape == (experts, Gu, inter * bits // 16)
            and us.shape == (experts, Gu, 2 * inter) and dq.shape == (experts, inter * bits // 32, hidden)
            and dz.shape == (experts, Gd, hidden * bits // 32) and ds.shape == (experts, Gd, hidden)
            and uq.is_contiguous() and uz.is_contiguous() and us.is_contiguous()
            and dq.is_contiguous() and dz.is_contiguous() and ds.is_contiguous()):
        for weight, K, N, G, name in ((up, hidden, 2 * inter, Gu, "up"), (down, inter, hidden, Gd, "down")):
            _look(weight[0], i32, (experts, K * bits // 32, N), name + " qweight")
            _look(weight[1], i32, (experts, G, N * bits // 32), name + " qzeros")
            _look(weight[2], f16, (experts, G, N), name + " scales")
    if out is None:
        out = x.new_empty(shape) if stream is None else _new(stream, x, shape)
        out_ptr = out.data_ptr()
    else:
        out_ptr = _address(out, dtype, shape, "out")
    ids = weights = ids_ptr = weights_ptr = None
    if return_routing:
        ids, weights = _new(stream, x, (tokens, topk), i32), _new(stream, x, (tokens, topk), rt.float32)
        ids_ptr, weights_ptr = ids.data_ptr(), weights.data_ptr()
    ws = ws_bytes = 0
    if workspace is None and tokens > 0:
        with _on(stream):
            workspace = moe_workspace(tokens, hidden, inter, experts, topk)
    if workspace is not None:
        ws, ws_bytes = _workspace(workspace)
    rc = rt.lib.gptq_moe(x.data_ptr(), tokens, hidden, inter, code, router.data_ptr(), experts, topk, 1 if renormalize else 0,
                         uq.data_ptr(), uz.data_ptr(), us.data_ptr(), dq.data_ptr(), dz.data_ptr(), ds.data_ptr(), bits, group,
                         fmt, out_ptr, ids_ptr, weights_ptr, ws, ws_bytes, rt.stream() if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "gptq_moe")
    return (out, ids, weights) if return_routing else out


def sample(logits, uniform, *, temperature=None, top_k=None, top_p=None, min_p=None, out=None, stream=None):
    """One token for each row of logits [batch, vocab] (float16, bfloat16 or float32; rows may be
    strided) from uniform [batch] fp32 in [0, 1), with [batch] settings (temperature, top_p, min_p
    fp32; top_k int32; None: off) -> (token [batch] int32, logprob [batch] fp32), written into `out` =
    (token, logprob) when given.  Among the kept tokens the first, in index order, whose cumulated
    probability exceeds the uniform number."""
    rt = _rt or _runtime()
    batch, vocab = logits.shape
    code = rt.codes.get(logits.dtype)
    if code is None:
        raise TypeError("logits must be float16, bfloat16 or float32, got %s" % logits.dtype)
    row, col = logits.stride()
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor")
    if col != 1 and vocab > 1:
        raise ValueError("logits: a row must be contiguous")
    f32, one = rt.float32, (batch,)
    u_ptr = _address(uniform, f32, one, "uniform")
    t_ptr = None if temperature is None else _address(temperature, f32, one, "temperature")
    k_ptr = None if top_k is None else _address(top_k, rt.int32, one, "top_k")
    p_ptr = None if top_p is None else _address(top_p, f32, one, "top_p")
    m_ptr = None if min_p is None else _address(min_p, f32, one, "min_p")
    if out is None:
        token, logprob = _new(stream, uniform, one, rt.int32), _new(stream, uniform, one)
        token_ptr, logprob_ptr = token.data_ptr(), logprob.data_ptr()
    else:
        token, logprob = out
        token_ptr, logprob_ptr = _address(token, rt.int32, one, "token"), _address(logprob, f32, one, "logprob")
    rc = rt.lib.gptq_sample(logits.data_ptr(), batch, vocab, row if batch > 1 else vocab, code, u_ptr, t_ptr, k_ptr, p_ptr, m_ptr,
                            token_ptr, logprob_ptr, rt.stream() if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "gptq_sample")
    return token, logprob
