"""Small-M FP8 block-scaled linear layer for GB300 (sm_103a).

Thin Python binding over the C ABI of ``lib/libfp8bs.so`` (declared in
``include/fp8bs.h``).  This module only marshals arguments: torch tensors
provide device memory and the current CUDA stream; every step of the layer
runs in the library's CUDA kernels.  There is no fallback: if the library is
missing or a call fails, a RuntimeError says why.

Entry points (same names as the C ABI):

* ``fp8_quant_act(x)`` -> (xq, xs): per-token, per-128 E4M3 cast of bf16 X.
* ``fp8_quant_weight_blocks(w, tiled=False)`` -> (wq, ws): 128x128-block
  E4M3 weights, row-major or one contiguous 16 KB run per block.
* ``fp8_blockscaled_gemm(aq, as_, wq, ws)`` -> Y bf16 (M up to 512).
* ``fp8_blockscaled_gemm_fused(x, wq, ws)`` -> Y bf16 (cast fused in).
* ``fp8_blockscaled_gemm_fused_greedy(x, wq, ws)`` -> (token, logit, Y):
  the same plus the greedy next-token choice (M up to 64).
* ``speculative_verify(logits, sample_u, draft, accept_u)`` -> (tokens,
  accepted, probs): drafted tokens against the target's logits, and the next one.
* ``bf16_pack_weights_tiled(w)``, ``bf16_gemm_ref(x, w)`` -> Y bf16 (the
  16-bit output-layer baseline).
* ``fp8_mx_quant_weights(w)``, ``fp8_mx_quant_act(x)``, ``fp8_mx_gemm(...)``:
  the native block-scaled (MX) variant, one UE8M0 scale per 32 K.
* ``fp8_rmsnorm_quant_act(x, gamma, eps, residual)``, ``fp8_mx_rmsnorm_quant_act``
  -> (xq, scales, residual_out, y): residual's addition, RMS norm and 8-bit cast.
* ``moe_route(x, wr, top_k)`` -> (ids, weights), ``fp8_moe_experts(x, ids,
  weights, w13, s13, w2, s2)`` -> Y and ``fp8_moe_layer(x, wr, top_k, w13, s13,
  w2, s2)`` -> (Y, ids, weights): a mixture-of-experts layer (M up to 64).
* ``fp4_quant_weights(w, fmt)``, ``fp4_quant_act(x, fmt)``, ``fp4_gemm(...)``,
  ``fp4_gemm_fused(x, ...)``, ``fp4_dequant_weights(...)``: microscaled 4-bit
  weights and activations (FP4_NV or FP4_MX).
* ``fp8_blockscaled_gemm_workspace_size``, ``make_workspace``,
  ``workspace_status``, ``split_plan``, ``gemm_schedule``, ``fused_route``:
  workspace and schedule queries.
"""
import contextlib
import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "lib", "libfp8bs.so")
DEBUG_LIB_PATH = os.path.join(PKG, "lib", "libfp8bs_debug.so")

FLAG_OVERLAP_PREV = 1
FLAG_WEIGHTS_TILED = 2
FLAG_PROLOGUE_CAST = 4
F32, BF16 = 0, 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
FP4_NV, FP4_MX = 0, 1  # 4-bit formats: 16-wide E4M3 scales and fp32 row scales; 32-wide powers of two

_lib = None


class Fp8bsError(RuntimeError):
    def __init__(self, fn, code, text):
        super().__init__("%s failed: %s (status %d)" % (fn, text, code))
        self.code = code


_loaded = {}


def lib():
    """The active copy of the library: libfp8bs.so, or libfp8bs_debug.so
    inside ``with debug_library():``.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        _lib = _load(LIB_PATH)
    return _lib


@contextlib.contextmanager
def debug_library():
    """Route every call of this module to libfp8bs_debug.so (the FP8BS_DEBUG
    build, with device-side bounds checks) inside the ``with`` block."""
    global _lib
    prev = lib()
    _lib = _load(DEBUG_LIB_PATH)
    try:
        yield _lib
    finally:
        _lib = prev


def _load(path):
    if path in _loaded:
        return _loaded[path]
    if not os.path.exists(path):
        raise RuntimeError("%s is not built (expected at %s); run "
                           "`python -c \"import __graft_entry__ as g; g.build()\"`" % (os.path.basename(path), path))
    L = ctypes.CDLL(path)
    vp, i, u, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint, ctypes.c_size_t
    L.fp8bs_status_string.restype = ctypes.c_char_p
    L.fp8bs_status_string.argtypes = [i]
    sigs = {
        "fp8_quant_act": [vp, i, i, i, vp, vp, u, vp],
        "fp8_quant_weight_blocks": [vp, i, i, i, vp, vp, vp],
        "fp8_quant_weight_blocks_tiled": [vp, i, i, i, vp, vp, vp],
        "bf16_pack_weights_tiled": [vp, i, i, vp, vp],
        "fp8_blockscaled_gemm_workspace_size": [i, i, i, ctypes.POINTER(sz)],
        "fp8_blockscaled_gemm": [vp, vp, vp, vp, vp, i, i, i, vp, sz, u, vp],
        "fp8_blockscaled_gemm_fused": [vp, i, vp, vp, vp, i, i, i, vp, sz, u, vp],
        "fp8_blockscaled_gemm_fused_greedy": [vp, i, vp, vp, vp, i, i, i, vp, vp, vp, sz, u, vp],
        "bf16_gemm_ref_workspace_size": [i, i, i, ctypes.POINTER(sz)],
        "bf16_gemm_ref": [vp, vp, vp, i, i, i, vp, sz, u, vp],
        "fp8bs_workspace_status": [vp, i, ctypes.POINTER(i)],
        "fp8bs_split_plan": [i, i, i, i, i, ctypes.POINTER(i), ctypes.POINTER(ctypes.c_longlong),
                             ctypes.POINTER(ctypes.c_longlong), ctypes.POINTER(ctypes.c_longlong)],
        "fp8bs_gemm_schedule": [i, i, i, i, ctypes.POINTER(i), ctypes.POINTER(i), ctypes.POINTER(i),
                                ctypes.POINTER(ctypes.c_longlong), ctypes.POINTER(i)],
        "fp8bs_fused_route": [i, i, i, i, ctypes.c_uint, ctypes.POINTER(i)],
        "fp8bs_testhook_gemm_stall": [vp, vp, vp, vp, vp, i, i, i, vp, sz, i, ctypes.c_ulonglong, vp],
        "fp8bs_testhook_kernel_runs": [i, i, ctypes.POINTER(ctypes.c_ulonglong)],
        "fp8bs_testhook_gemm_fused_sms": [vp, i, vp, vp, vp, i, i, i, vp, sz, u, i, vp],
        "fp8bs_testhook_workspace_size_sms": [i, i, i, i, ctypes.POINTER(sz)],
        "fp8bs_testhook_debug_bad_tile": [vp, vp, vp, vp, vp, i, i, i, vp, sz, i, ctypes.c_ulonglong, vp],
        "fp8_blockscaled_gemm_fused_noalloc": [vp, i, vp, vp, vp, i, i, i, u, vp],
        "fp8_mx_quant_weights": [vp, i, i, i, vp, vp, vp],
        "fp8_mx_quant_act": [vp, i, i, i, vp, vp, u, vp],
        "fp8_mx_gemm_workspace_size": [i, i, i, ctypes.POINTER(sz)],
        "speculative_verify_workspace_size": [i, i, i, ctypes.POINTER(sz)],
        "speculative_verify": [vp, i, i, vp, vp, vp, i, vp, vp, vp, i, i, i, vp, vp, vp, vp, sz, u, vp],
        "fp8_rmsnorm_quant_act": [vp, i, vp, i, vp, i, vp, i, ctypes.c_float, i, i, vp, vp, vp, u, vp],
        "fp8_mx_rmsnorm_quant_act": [vp, i, vp, i, vp, i, vp, i, ctypes.c_float, i, i, vp, vp, vp, u, vp],
        "fp8bs_testhook_fp4_stall": [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, vp, sz, i, ctypes.c_ulonglong, vp],
        "fp8bs_testhook_moe_stall": [vp, i, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp, sz, u, i, i,
                                     ctypes.c_ulonglong, vp],
        "moe_route_workspace_size": [i, i, ctypes.POINTER(sz)],
        "moe_route": [vp, i, vp, i, i, i, i, i, i, vp, vp, vp, sz, u, vp],
        "fp8_moe_workspace_size": [i, i, i, i, i, ctypes.POINTER(sz)],
        "fp8_moe_experts": [vp, i, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp, sz, u, vp],
        "fp8_moe_layer": [vp, i, vp, i, i, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp, sz, u, vp],
        "moe_route_grouped": [vp, i, vp, i, vp, i, i, i, i, i, i, i, i, i, ctypes.c_float, vp, vp, vp, sz, u, vp],
        "fp8_moe_layer_grouped": [vp, i, vp, i, vp, i, i, i, i, i, ctypes.c_float, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i,
                                  vp, sz, u, vp],
        "fp4_quant_weights": [vp, i, i, i, i, vp, vp, vp, vp],
        "fp4_dequant_weights": [vp, vp, vp, i, i, i, vp, i, vp],
        "fp4_quant_act": [vp, i, i, i, i, vp, vp, vp, u, vp],
        "fp4_gemm_workspace_size": [i, i, i, i, ctypes.POINTER(sz)],
        "fp4_gemm": [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, vp, sz, u, vp],
        "fp4_gemm_fused": [vp, i, vp, vp, vp, vp, i, i, i, i, vp, sz, u, vp],
        "fp8_mx_gemm": [vp, vp, vp, vp, vp, i, i, i, vp, sz, u, vp],
    }
    for name, args in sigs.items():
        f = getattr(L, name)
        f.restype = i
        f.argtypes = args
    L.fp8bs_testhook_debug_build.restype = i
    L.fp8bs_testhook_debug_build.argtypes = []
    _loaded[path] = L
    return L


def status_string(code):
    return lib().fp8bs_status_string(int(code)).decode()


def _check(fn, code):
    if code != 0:
        raise Fp8bsError(fn, code, status_string(code))


# ---------------------------------------------------------------- helpers
_torch_module = None


def _torch():
    """torch, imported at the first call that needs it."""
    global _torch_module, _bf16, _f32, _i32, _u8, _empty
    if _torch_module is None:
        import torch
        _bf16, _f32, _i32, _u8, _empty = torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.empty
        _torch_module = torch
    return _torch_module


# The helpers below run on every call: an eager decode pass makes hundreds of
# them per step, and their host time is on the critical path whenever the
# layers are short (measured: 17.3 us a fused call with the stream taken from
# torch.cuda.current_stream() and the device from t.device, 10.1 us as here,
# 4.8 us of it in the library).
_raw_stream = None


def _stream():
    """The current CUDA stream of the current device, as an integer handle."""
    global _raw_stream
    if _raw_stream is not None:
        return _raw_stream[0](_raw_stream[1]())
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    device = getattr(torch._C, "_cuda_getDevice", None)
    if raw is not None and device is not None:
        stream = raw(torch.cuda.current_device())  # (this initialises CUDA)
        _raw_stream = (raw, device)
        return stream
    return torch.cuda.current_stream().cuda_stream


def _ptr(t):
    """Device address of a tensor (the c_void_p arguments take integers)."""
    return t.data_ptr() if t is not None else None


def _need(t, dtype, name, ndim=2):
    torch = _torch()
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and t.dim() == ndim:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (there is no CPU path)" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.dim() != ndim:
        raise ValueError("%s must be %d-D" % (name, ndim))


def _rows_contiguous(t, name):
    if t.stride(-1) != 1:
        raise ValueError("%s must have unit stride along K" % name)


# ---------------------------------------------------------------- entry points
def scales_shape(M, K):
    """Shape of the activation scales for M tokens: (M, K/128) token-major up
    to 16 tokens, (K/128, M) K-block-major above."""
    kg = max(K // 128, 0)
    return (M, kg) if M <= 16 else (kg, M)


def fp8_quant_act(x, xq=None, xs=None, flags=0):
    """bf16 X [M, K] (row stride may exceed K) -> (xq uint8 [M,K], xs fp32 of
    scales_shape(M, K))."""
    torch = _torch()
    _need(x, torch.bfloat16, "x")
    _rows_contiguous(x, "x")
    M, K = x.shape
    if xq is None:
        xq = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    if xs is None:
        xs = torch.empty(scales_shape(M, K), dtype=torch.float32, device=x.device)
    _check("fp8_quant_act", lib().fp8_quant_act(_ptr(x), M, K, x.stride(0), _ptr(xq), _ptr(xs), flags, _stream()))
    return xq, xs


def fp8_quant_weight_blocks(w, wq=None, ws=None, tiled=False):
    """fp32 or bf16 W [N, K] -> (wq, ws fp32 [ceil(N/128), K/128]).

    wq is uint8 [N, K] row-major, or with ``tiled=True`` uint8
    [ceil(N/128) * K/128, 128, 128]: one contiguous 128x128 block per weight
    tile (rows past N zero), for the GEMMs' tiled-weight mode."""
    torch = _torch()
    if w.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("w must be float32 or bfloat16")
    _need(w, w.dtype, "w")
    if not w.is_contiguous():
        raise ValueError("w must be contiguous")
    N, K = w.shape
    if wq is None:
        shape = (((N + 127) // 128) * max(K // 128, 0), 128, 128) if tiled else (N, K)
        wq = torch.empty(shape, dtype=torch.uint8, device=w.device)
    if ws is None:
        ws = torch.empty(((N + 127) // 128, max(K // 128, 0)), dtype=torch.float32, device=w.device)
    wt = BF16 if w.dtype == torch.bfloat16 else F32
    fn = lib().fp8_quant_weight_blocks_tiled if tiled else lib().fp8_quant_weight_blocks
    _check("fp8_quant_weight_blocks", fn(_ptr(w), wt, N, K, _ptr(wq), _ptr(ws), _stream()))
    return wq, ws


def bf16_pack_weights_tiled(w, wt=None):
    """bf16 W [N, K] -> bf16 [ceil(N/128) * K/64, 128, 64], one contiguous
    128x64 tile per block (rows past N zero), for bf16_gemm_ref(tiled)."""
    torch = _torch()
    _need(w, torch.bfloat16, "w")
    if not w.is_contiguous():
        raise ValueError("w must be contiguous")
    N, K = w.shape
    if wt is None:
        wt = torch.empty((((N + 127) // 128) * max(K // 64, 0), 128, 64), dtype=torch.bfloat16, device=w.device)
    _check("bf16_pack_weights_tiled", lib().bf16_pack_weights_tiled(_ptr(w), N, K, _ptr(wt), _stream()))
    return wt


def _weight_dims(wq, K, n, what):
    """(N, flag) of a row-major [N,K] or tiled [tiles,128,*] weight operand."""
    if wq.dim() == 2:
        if wq.shape[1] != K:
            raise ValueError("operand shapes do not agree")
        return wq.shape[0], 0
    if wq.dim() == 3 and wq.shape[1] == 128:
        if n is None:
            raise ValueError("%s is tiled: pass n= (the number of weight rows)" % what)
        if wq.numel() != ((int(n) + 127) // 128) * 128 * K:
            raise ValueError("tiled %s does not hold ceil(n/128)*128*K elements" % what)
        return int(n), FLAG_WEIGHTS_TILED
    raise ValueError("%s must be [N, K] or tiled [tiles, 128, *]" % what)


def fp8_blockscaled_gemm_workspace_size(M, N, K):
    n = ctypes.c_size_t(0)
    _check("fp8_blockscaled_gemm_workspace_size", lib().fp8_blockscaled_gemm_workspace_size(M, N, K, ctypes.byref(n)))
    return n.value


def bf16_gemm_ref_workspace_size(M, N, K):
    n = ctypes.c_size_t(0)
    _check("bf16_gemm_ref_workspace_size", lib().bf16_gemm_ref_workspace_size(M, N, K, ctypes.byref(n)))
    return n.value


def make_workspace(nbytes, device=None):
    """A zero-filled, 256-byte aligned device workspace of ``nbytes``."""
    torch = _torch()
    return torch.zeros(nbytes, dtype=torch.uint8, device=device or "cuda")


def fp8_blockscaled_gemm(aq, as_, wq, ws, y=None, workspace=None, flags=0, n=None):
    """Y[M,N] bf16 from pre-quantised operands (wq row-major, or tiled with
    n= the number of weight rows)."""
    torch = _torch()
    _need(aq, torch.uint8, "aq")
    _need(as_, torch.float32, "as_")
    _need(wq, torch.uint8, "wq", ndim=wq.dim() if wq.dim() in (2, 3) else 2)
    _need(ws, torch.float32, "ws")
    for t, nm in ((aq, "aq"), (as_, "as_"), (wq, "wq"), (ws, "ws")):
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % nm)
    M, K = aq.shape
    N, tf = _weight_dims(wq, K, n, "wq")
    flags |= tf
    if tuple(as_.shape) != scales_shape(M, K) or tuple(ws.shape) != ((N + 127) // 128, K // 128):
        raise ValueError("operand shapes do not agree")
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=aq.device)
    if workspace is None:
        workspace = make_workspace(fp8_blockscaled_gemm_workspace_size(M, N, K), aq.device)
    _check("fp8_blockscaled_gemm",
           lib().fp8_blockscaled_gemm(_ptr(aq), _ptr(as_), _ptr(wq), _ptr(ws), _ptr(y), M, N, K,
                                      _ptr(workspace), workspace.numel(), flags, _stream()))
    return y


def fp8_blockscaled_gemm_fused(x, wq, ws, y=None, workspace=None, flags=0, n=None):
    """Y[M,N] bf16 from bf16 activations (row stride may exceed K); wq
    row-major, or tiled with n= the number of weight rows."""
    torch = _torch()
    _need(x, torch.bfloat16, "x")
    _rows_contiguous(x, "x")
    _need(wq, torch.uint8, "wq", ndim=wq.dim() if wq.dim() in (2, 3) else 2)
    _need(ws, torch.float32, "ws")
    M, K = x.shape
    N, tf = _weight_dims(wq, K, n, "wq")
    flags |= tf
    if tuple(ws.shape) != ((N + 127) // 128, K // 128):
        raise ValueError("operand shapes do not agree")
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = make_workspace(fp8_blockscaled_gemm_workspace_size(M, N, K), x.device)
    _check("fp8_blockscaled_gemm_fused",
           lib().fp8_blockscaled_gemm_fused(_ptr(x), x.stride(0), _ptr(wq), _ptr(ws), _ptr(y), M, N, K,
                                            _ptr(workspace), workspace.numel(), flags, _stream()))
    return y


def fp8_blockscaled_gemm_fused_greedy(x, wq, ws, y=None, store_y=True, token=None, logit=None, workspace=None,
                                      flags=0, n=None):
    """The fused layer plus the greedy next-token choice per token row:
    returns (token int32 [M], logit fp32 [M], y bf16 [M,N] or None).  With
    ``store_y=False`` the logits are not written (y must then be None)."""
    torch = _torch()
    _need(x, torch.bfloat16, "x")
    _rows_contiguous(x, "x")
    _need(wq, torch.uint8, "wq", ndim=wq.dim() if wq.dim() in (2, 3) else 2)
    _need(ws, torch.float32, "ws")
    M, K = x.shape
    N, tf = _weight_dims(wq, K, n, "wq")
    flags |= tf
    if tuple(ws.shape) != ((N + 127) // 128, K // 128):
        raise ValueError("operand shapes do not agree")
    if not store_y and y is not None:
        raise ValueError("store_y=False takes no y")
    if store_y and y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    if token is None:
        token = torch.empty((M,), dtype=torch.int32, device=x.device)
    if logit is None:
        logit = torch.empty((M,), dtype=torch.float32, device=x.device)
    _need(token, torch.int32, "token", ndim=1)
    _need(logit, torch.float32, "logit", ndim=1)
    if token.numel() < M or logit.numel() < M:
        raise ValueError("token and logit need M entries")
    if workspace is None:
        workspace = make_workspace(fp8_blockscaled_gemm_workspace_size(M, N, K), x.device)
    _check("fp8_blockscaled_gemm_fused_greedy",
           lib().fp8_blockscaled_gemm_fused_greedy(_ptr(x), x.stride(0), _ptr(wq), _ptr(ws),
                                                   _ptr(y) if y is not None else None, M, N, K, _ptr(token),
                                                   _ptr(logit), _ptr(workspace), workspace.numel(), flags,
                                                   _stream()))
    return token, logit, y


def bf16_gemm_ref(x, w, y=None, workspace=None, flags=0, n=None):
    """Y[M,N] bf16 = X bf16 [M,K] . W bf16 [N,K]^T (fp32 accumulation); w
    row-major, or tiled (bf16_pack_weights_tiled) with n= the weight rows."""
    torch = _torch()
    _need(x, torch.bfloat16, "x")
    _need(w, torch.bfloat16, "w", ndim=w.dim() if w.dim() in (2, 3) else 2)
    if not (x.is_contiguous() and w.is_contiguous()):
        raise ValueError("x and w must be contiguous")
    M, K = x.shape
    N, tf = _weight_dims(w, K, n, "w")
    flags |= tf
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = make_workspace(bf16_gemm_ref_workspace_size(M, N, K), x.device)
    _check("bf16_gemm_ref",
           lib().bf16_gemm_ref(_ptr(x), _ptr(w), _ptr(y), M, N, K, _ptr(workspace), workspace.numel(),
                               flags, _stream()))
    return y


# ---------------------------------------------------------------- MX variant
def fp8_mx_quant_weights(w, wq=None, ws_atoms=None):
    """fp32 or bf16 W [N, K] -> (wq uint8 [ceil(N/128) * K/128, 128, 128]
    tiled codes, ws_atoms uint8 [ceil(N/128) * K/128, 512] scale atoms):
    one power-of-two (UE8M0) scale per 32 K per row (include/fp8bs.h)."""
    torch = _torch()
    if w.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("w must be float32 or bfloat16")
    _need(w, w.dtype, "w")
    if not w.is_contiguous():
        raise ValueError("w must be contiguous")
    N, K = w.shape
    tiles = ((N + 127) // 128) * max(K // 128, 0)
    if wq is None:
        wq = torch.empty((tiles, 128, 128), dtype=torch.uint8, device=w.device)
    if ws_atoms is None:
        ws_atoms = torch.empty((tiles, 512), dtype=torch.uint8, device=w.device)
    wt = BF16 if w.dtype == torch.bfloat16 else F32
    _check("fp8_mx_quant_weights", lib().fp8_mx_quant_weights(_ptr(w), wt, N, K, _ptr(wq), _ptr(ws_atoms), _stream()))
    return wq, ws_atoms


def fp8_mx_quant_act(x, xq=None, xs_atoms=None, flags=0):
    """bf16 X [M, K] (M <= 512; row stride may exceed K) -> (xq uint8 [M, K],
    xs_atoms uint8 [ceil(M/128) * K/128, 512]: atom (token tile, K block))."""
    torch = _torch()
    _need(x, torch.bfloat16, "x")
    _rows_contiguous(x, "x")
    M, K = x.shape
    if xq is None:
        xq = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    if xs_atoms is None:
        xs_atoms = torch.empty((((M + 127) // 128) * max(K // 128, 0), 512), dtype=torch.uint8, device=x.device)
    _check("fp8_mx_quant_act", lib().fp8_mx_quant_act(_ptr(x), M, K, x.stride(0), _ptr(xq), _ptr(xs_atoms), flags,
                                                      _stream()))
    return xq, xs_atoms


def fp8_mx_gemm_workspace_size(M, N, K):
    n = ctypes.c_size_t(0)
    _check("fp8_mx_gemm_workspace_size", lib().fp8_mx_gemm_workspace_size(M, N, K, ctypes.byref(n)))
    return n.value


def fp8_mx_gemm(aq, as_atoms, wq, ws_atoms, n, y=None, workspace=None, flags=0):
    """Y[M, n] bf16 from MX operands (fp8_mx_quant_act / fp8_mx_quant_weights;
    n = the number of weight rows)."""
    torch = _torch()
    _need(aq, torch.uint8, "aq")
    _need(as_atoms, torch.uint8, "as_atoms")
    _need(wq, torch.uint8, "wq", ndim=3)
    _need(ws_atoms, torch.uint8, "ws_atoms")
    M, K = aq.shape
    N = int(n)
    tiles = ((N + 127) // 128) * (K // 128)
    if (wq.numel() != tiles * 16384 or ws_atoms.numel() != tiles * 512 or
            as_atoms.numel() != ((M + 127) // 128) * (K // 128) * 512):
        raise ValueError("operand shapes do not agree")
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=aq.device)
    if workspace is None:
        workspace = make_workspace(fp8_mx_gemm_workspace_size(M, N, K), aq.device)
    _check("fp8_mx_gemm", lib().fp8_mx_gemm(_ptr(aq), _ptr(as_atoms), _ptr(wq), _ptr(ws_atoms), _ptr(y), M, N, K,
                                            _ptr(workspace), workspace.numel(), flags, _stream()))
    return y


# ------------------------------------------------- expert and 4-bit layers
# Each tensor is checked and turned into its address in one short call: a
# decode step makes many of these calls, and between kernel launches every
# attribute that Python reads costs a tenth of a microsecond or more.  So what
# is no tensor is found out by the attribute it lacks.
def _tensors(**named):
    """TypeError for the first argument that is no tensor."""
    for name, t in named.items():
        if not isinstance(t, _torch().Tensor):
            raise TypeError("%s must be a torch.Tensor" % name)


def _addr(t, dtype, numel, name):
    """Address of a contiguous CUDA tensor of that type and number of elements."""
    try:
        if t.dtype is dtype and t.is_cuda and t.is_contiguous() and t.numel() == numel:
            return t.data_ptr()
    except AttributeError:
        pass
    _tensors(**{name: t})
    _need(t, dtype, name, t.dim())
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    raise ValueError("operand shapes do not agree (%s has %d elements, not %d)" % (name, t.numel(), numel))


def _act(x):
    """(M, K, row stride, address) of bf16 activations [M, K]."""
    if _torch_module is None:
        _torch()
    try:
        if x.dtype is not _bf16 or not x.is_cuda or x.dim() != 2:
            _need(x, _bf16, "x")
    except AttributeError:
        _need(x, _bf16, "x")
        raise
    M, K = x.shape
    ld, unit = x.stride()
    if unit != 1:
        raise ValueError("x must have unit stride along K")
    if M == 1:
        ld = K  # one row: whatever its stride says
    elif ld > 0x7fffffff:
        raise ValueError("x's row stride does not fit in 32 bits")
    return M, K, ld, x.data_ptr()


def _matrix(w, name):
    """(rows, K, dtype code, address) of a contiguous fp32 or bf16 matrix."""
    if _torch_module is None:
        _torch()
    try:
        t = w.dtype
    except AttributeError:
        _tensors(**{name: w})
        raise
    if t is not _bf16 and t is not _f32:
        _tensors(**{name: w})
        raise TypeError("%s must be float32 or bfloat16" % name)
    if not w.is_cuda or w.dim() != 2:
        _need(w, t, name)
    if not w.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    rows, K = w.shape
    return rows, K, BF16 if t is _bf16 else F32, w.data_ptr()


def _out(t, shape, dtype, device, name):
    """(tensor, address) of an output: `t` checked (that shape, contiguous), or a new one."""
    if t is None:
        t = _empty(shape, dtype=dtype, device=device)
        return t, t.data_ptr()
    try:
        if t.dtype is dtype and t.is_cuda and t.shape == shape and t.is_contiguous():
            return t, t.data_ptr()
    except AttributeError:
        pass
    _need(t, dtype, name, len(shape))
    raise ValueError("%s must be contiguous of shape %s" % (name, shape))


def _work(workspace):
    """(address, bytes) of a workspace."""
    try:
        if workspace.dtype is _u8 and workspace.is_cuda and workspace.is_contiguous():
            return workspace.data_ptr(), workspace.numel()
    except AttributeError:
        pass
    raise TypeError("workspace must be a contiguous CUDA tensor of bytes (make_workspace)")


# ----------------------------------- norm and cast, drafted tokens, scored routing
# As above, one short call a tensor; these also take the device: the kernels run
# on the current one's current stream, so x has to lie there and the rest with it.
_device_now = None


def _first_use():
    """torch, and how to ask for the current device."""
    global _device_now
    torch = _torch()
    torch.cuda.is_available() and torch.cuda.current_device()  # (this initialises CUDA)
    _device_now = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _home(t, name):
    """The device number of a call's first tensor, which is the current device."""
    if _device_now is None:
        _first_use()
    d = t.get_device()
    if d != _device_now():
        raise ValueError("%s is on device %d, which is not the current one" % (name, d))
    return d


def _rows(t, name):
    """(shape, row stride, address) of a bf16 matrix with unit stride along K."""
    try:
        if t.dtype is _bf16 and t.is_cuda:
            shape = t.shape
            ld, unit = t.stride()
            if unit == 1 and 0 <= ld <= 0x7fffffff:
                return shape, ld if shape[0] != 1 else shape[1], t.data_ptr()
            if unit == 1 and shape[0] == 1:
                return shape, shape[1], t.data_ptr()
    except (AttributeError, ValueError):
        pass
    _need(t, _bf16, name)
    if t.stride(1) != 1:
        raise ValueError("%s must have unit stride along K" % name)
    raise ValueError("%s's row stride does not fit in 32 bits" % name)


def _in(t, dtype, numel, name, d):
    """Address of a contiguous input of that type and number of elements on device d."""
    try:
        if t.dtype is dtype and t.get_device() == d and t.is_contiguous() and t.numel() == numel:
            return t.data_ptr()
    except AttributeError:
        pass
    _addr(t, dtype, numel, name)
    raise ValueError("%s must be on device %d, as the first argument" % (name, d))


def _there(t, name, d):
    if t.get_device() != d:
        raise ValueError("%s must be on device %d, as the first argument" % (name, d))


def _make(t, shape, dtype, dev, name, d):
    """(tensor, address) of an output: `t` checked, or a new one."""
    if t is None:
        t = _empty(shape, dtype=dtype, device=dev)
        return t, t.data_ptr()
    r = _out(t, shape, dtype, dev, name)
    _there(t, name, d)
    return r


def _rmsnorm(mx, x, gamma, eps, residual, residual_out, y, store_y, xq, scales, flags):
    if _device_now is None:
        _first_use()
    bf = False
    try:  # the usual call, in as few reads as it takes; anything else is looked at one by one
        shape = x.shape
        M, K = shape
        ldx, unit = x.stride()
        d = x.get_device()
        bf = gamma.dtype is _bf16
        usual = (x.dtype is _bf16 and unit == 1 and ldx <= 0x7fffffff and d >= 0 and d == _device_now() and
                 (bf or gamma.dtype is _f32) and gamma.get_device() == d and gamma.is_contiguous() and gamma.numel() == K)
    except (AttributeError, ValueError):
        usual = False
    if usual:
        xp, gp = x.data_ptr(), gamma.data_ptr()
        if M == 1:
            ldx = K
    else:
        shape, ldx, xp = _rows(x, "x")
        M, K = shape
        d = _home(x, "x")
        _tensors(gamma=gamma)
        if not bf and gamma.dtype is not _f32:
            raise TypeError("gamma must be float32 or bfloat16")
        gp = _in(gamma, _bf16 if bf else _f32, K, "gamma", d)
    dev = x.device
    rp = op = yp = None
    ldr = ldo = 0
    if residual is not None:
        rshape, ldr, rp = _rows(residual, "residual")
        if rshape != shape:
            raise ValueError("residual must have shape %s" % (tuple(shape),))
        _there(residual, "residual", d)
        if residual_out is None:
            residual_out = _empty(shape, dtype=_bf16, device=dev)
            ldo, op = K, residual_out.data_ptr()
        else:
            oshape, ldo, op = _rows(residual_out, "residual_out")
            if oshape != shape:
                raise ValueError("residual_out must have shape %s" % (tuple(shape),))
            _there(residual_out, "residual_out", d)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if store_y or y is not None:
        y, yp = _make(y, shape, _bf16, dev, "y", d)
    if xq is None:
        xq = _empty(shape, dtype=_u8, device=dev)
        qp = xq.data_ptr()
    else:
        xq, qp = _make(xq, shape, _u8, dev, "xq", d)
    if mx:
        sshape, sdtype, call = ((M + 127) // 128 * (K // 128), 512), _u8, lib().fp8_mx_rmsnorm_quant_act
    else:
        sshape, sdtype, call = (M, K // 128) if M <= 16 else (K // 128, M), _f32, lib().fp8_rmsnorm_quant_act
    if scales is None:
        scales = _empty(sshape, dtype=sdtype, device=dev)
        sp = scales.data_ptr()
    else:
        scales, sp = _make(scales, sshape, sdtype, dev, "xs_atoms" if mx else "xs", d)
    code = call(xp, ldx, rp, ldr, op, ldo, gp, 1 if bf else 0, eps, M, K, yp, qp, sp, flags, _stream())
    if code:
        _check("fp8_mx_rmsnorm_quant_act" if mx else "fp8_rmsnorm_quant_act", code)
    return xq, scales, residual_out, y


def fp8_rmsnorm_quant_act(x, gamma, eps=1e-6, residual=None, residual_out=None, y=None, store_y=False, xq=None, xs=None,
                          flags=0):
    """RMS norm of h = x + residual (bf16 [M, K], row strides may exceed K; h =
    x without a residual) with weights gamma (fp32 or bf16 [K]), and its E4M3
    cast: (xq uint8 [M, K], xs fp32 of scales_shape(M, K), residual_out = h bf16
    [M, K] or None, y = the norm's bf16 values [M, K], None without
    ``store_y``).  residual_out=residual adds in place."""
    return _rmsnorm(False, x, gamma, eps, residual, residual_out, y, store_y, xq, xs, flags)


def fp8_mx_rmsnorm_quant_act(x, gamma, eps=1e-6, residual=None, residual_out=None, y=None, store_y=False, xq=None,
                             xs_atoms=None, flags=0):
    """The same with the MX cast (M <= 512): (xq, xs_atoms uint8 [ceil(M/128) *
    K/128, 512], residual_out, y)."""
    return _rmsnorm(True, x, gamma, eps, residual, residual_out, y, store_y, xq, xs_atoms, flags)


def speculative_verify_workspace_size(B, L, V):
    n = ctypes.c_size_t(0)
    _check("speculative_verify_workspace_size", lib().speculative_verify_workspace_size(B, L, V, ctypes.byref(n)))
    return n.value


def _logit_rows(t, rows, V, dtypes, name):
    """(row stride, address) of rows with unit stride along the vocabulary."""
    try:
        if t.dtype in dtypes and t.is_cuda and t.shape == (rows, V):
            ld, unit = t.stride()
            if unit == 1 or V == 1:
                if rows <= 1:
                    return V, t.data_ptr()
                if V <= ld <= 0x7fffffff:
                    return ld, t.data_ptr()
    except AttributeError:
        pass
    _tensors(**{name: t})
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s" % (name, " or ".join(str(d) for d in dtypes)))
    _need(t, t.dtype, name)
    if t.shape != (rows, V):
        raise ValueError("%s must have shape (%d, %d)" % (name, rows, V))
    if t.stride(1) != 1:
        raise ValueError("%s must have unit stride along the vocabulary" % name)
    raise ValueError("%s's rows overlap, or their stride does not fit in 32 bits" % name)


def speculative_verify(logits, sample_u, draft=None, accept_u=None, draft_probs=None, draft_len=None, temperature=None,
                       tokens=None, accepted=None, probs=None, workspace=None, flags=0):
    """Drafted tokens against the target's logits (include/fp8bs.h has the
    rule): logits bf16 or fp32 [B * (L + 1), V] as the output layer writes them (row
    stride may exceed V), sample_u fp32 [B], draft int32 [B, L], accept_u fp32 [B,
    L], draft_probs fp32 [B * L, V] or None (the draft is certain of its tokens),
    draft_len int32 [B] or None (L each), temperature fp32 [B] or None (1) ->
    (tokens int32 [B, L + 1]: the accepted ones, the next one, then -1; accepted
    int32 [B]; probs fp32 [B, L + 1]: the target's probabilities of those tokens).
    Without a draft one token is drawn from each row."""
    if _torch_module is None:
        _torch()
    try:
        B = sample_u.numel()
        V = logits.shape[-1]
        d = _home(logits, "logits") if logits.is_cuda else -1
    except AttributeError:
        _tensors(logits=logits, sample_u=sample_u)
        raise
    L, dp, ap, qp, np_, tp, ldq = 0, None, None, None, None, None, 0
    if draft is not None:
        _need(draft, _i32, "draft")
        L = draft.shape[1]
    elif accept_u is not None or draft_probs is not None or draft_len is not None:
        raise ValueError("accept_u, draft_probs and draft_len need a draft")
    ldl, lp = _logit_rows(logits, B * (L + 1), V, (_bf16, _f32), "logits")
    if L:
        dp, ap = _in(draft, _i32, B * L, "draft", d), _in(accept_u, _f32, B * L, "accept_u", d)
        if draft_len is not None:
            np_ = _in(draft_len, _i32, B, "draft_len", d)
        if draft_probs is not None:
            ldq, qp = _logit_rows(draft_probs, B * L, V, (_f32,), "draft_probs")
            _there(draft_probs, "draft_probs", d)
    sp = _in(sample_u, _f32, B, "sample_u", d)
    if temperature is not None:
        tp = _in(temperature, _f32, B, "temperature", d)
    dev = logits.device
    tokens, op = _make(tokens, (B, L + 1), _i32, dev, "tokens", d)
    accepted, cp = _make(accepted, (B,), _i32, dev, "accepted", d)
    probs, pp = _make(probs, (B, L + 1), _f32, dev, "probs", d)
    if workspace is None:
        workspace = make_workspace(speculative_verify_workspace_size(B, L, V), dev)
    wsp, wsn = _work(workspace)
    _there(workspace, "workspace", d)
    code = lib().speculative_verify(lp, BF16 if logits.dtype is _bf16 else F32, ldl, dp, np_, qp, ldq, ap, sp, tp, B, L, V, op,
                                    cp, pp, wsp, wsn, flags, _stream())
    if code:
        _check("speculative_verify", code)
    return tokens, accepted, probs


def moe_route_workspace_size(M, E):
    n = ctypes.c_size_t(0)
    _check("moe_route_workspace_size", lib().moe_route_workspace_size(M, E, ctypes.byref(n)))
    return n.value


def fp8_moe_workspace_size(M, H, I, E, top_k):
    n = ctypes.c_size_t(0)
    _check("fp8_moe_workspace_size", lib().fp8_moe_workspace_size(M, H, I, E, top_k, ctypes.byref(n)))
    return n.value


def _experts(w13, s13, w2, s2, H, E):
    """(I, flag, addresses of w13, s13, w2, s2) of E experts' weights: w13 [E,
    2I, H] and w2 [E, H, I], or both tiled [tiles, 128, 128]."""
    kg = H // 128
    flag = None
    try:
        shape13, shape2 = w13.shape, w2.shape
        if E >= 1 and s2.dim() == 2 and s13.dim() == 2:
            rows2, rows = s2.shape  # rows: 128-row tiles of I
            tiles = E * rows * kg
            if tiles >= 1 and rows2 == E * kg and s13.shape == (2 * E * rows, kg):
                I = rows * 128
                if shape13 == (2 * tiles, 128, 128) and shape2 == (tiles, 128, 128):
                    flag = FLAG_WEIGHTS_TILED
                elif shape13 == (E, 2 * I, H) and shape2 == (E, H, I):
                    flag = 0
    except AttributeError:
        pass
    if flag is None:
        _tensors(w13=w13, s13=s13, w2=w2, s2=s2)
        raise ValueError("operand shapes do not agree")
    return (I, flag, _addr(w13, _u8, 2 * tiles * 16384, "w13"), _addr(s13, _f32, 2 * tiles, "s13"),
            _addr(w2, _u8, tiles * 16384, "w2"), _addr(s2, _f32, tiles, "s2"))


def moe_route(x, wr, top_k, renormalize=True, ids=None, weights=None, workspace=None, flags=0):
    """The experts of each token: x bf16 [M, H] (row stride may exceed H), wr
    fp32 or bf16 [E, H] -> (ids int32 [M, top_k] by descending logit, weights
    fp32 [M, top_k], softmax over the chosen or, with renormalize=False, over
    all experts)."""
    M, H, ldx, xp = _act(x)
    E, Hr, wt, wrp = _matrix(wr, "wr")
    if H != Hr:
        raise ValueError("operand shapes do not agree")
    ids, idp = _out(ids, (M, top_k), _i32, x.device, "ids")
    weights, wp = _out(weights, (M, top_k), _f32, x.device, "weights")
    if workspace is None:
        workspace = make_workspace(moe_route_workspace_size(M, E), x.device)
    wsp, wsn = _work(workspace)
    _check("moe_route", lib().moe_route(xp, ldx, wrp, wt, M, H, E, top_k, 1 if renormalize else 0, idp, wp,
                                        wsp, wsn, flags, _stream()))
    return ids, weights


def fp8_moe_experts(x, ids, weights, w13, s13, w2, s2, experts=None, y=None, workspace=None, flags=0):
    """Y bf16 [M, H] of the experts that ids int32 [M, top_k] names, weighted
    by weights fp32 [M, top_k] (an id outside [0, experts) is skipped); w13
    [experts, 2I, H] and w2 [experts, H, I] E4M3 row-major, or both tiled
    (fp8_quant_weight_blocks of the matrices with the experts' rows stacked)
    with experts= given; s13, s2 their block scales."""
    M, H, ldx, xp = _act(x)
    if experts is None:
        _tensors(w13=w13)
        if w13.dim() != 3 or w13.shape[2] != H:
            raise ValueError("w13 is tiled: pass experts= (the number of experts)")
        experts = w13.shape[0]
    E = int(experts)
    I, tf, w13p, s13p, w2p, s2p = _experts(w13, s13, w2, s2, H, E)
    try:
        bad = ids.dim() != 2 or ids.shape[0] != M or ids.shape != weights.shape
    except AttributeError:
        _tensors(ids=ids, weights=weights)
        raise
    if bad:
        _tensors(weights=weights)
        raise ValueError("operand shapes do not agree")
    k = ids.shape[1]
    idp, wp = _addr(ids, _i32, M * k, "ids"), _addr(weights, _f32, M * k, "weights")
    y, yp = _out(y, (M, H), _bf16, x.device, "y")
    if workspace is None:
        workspace = make_workspace(fp8_moe_workspace_size(M, H, I, E, k), x.device)
    wsp, wsn = _work(workspace)
    _check("fp8_moe_experts", lib().fp8_moe_experts(xp, ldx, idp, wp, w13p, s13p, w2p, s2p, yp, M, H, I, E, k, wsp, wsn,
                                                    flags | tf, _stream()))
    return y


def fp8_moe_layer(x, wr, top_k, w13, s13, w2, s2, renormalize=True, y=None, ids=None, weights=None, workspace=None,
                  flags=0):
    """The whole layer, moe_route and fp8_moe_experts in three kernels: (y
    bf16 [M, H], ids int32 [M, top_k], weights fp32 [M, top_k]); w13 and w2 as
    in fp8_moe_experts, row-major or tiled."""
    M, H, ldx, xp = _act(x)
    E, Hr, wt, wrp = _matrix(wr, "wr")
    if H != Hr:
        raise ValueError("operand shapes do not agree")
    I, tf, w13p, s13p, w2p, s2p = _experts(w13, s13, w2, s2, H, E)
    dev = x.device
    y, yp = _out(y, (M, H), _bf16, dev, "y")
    ids, idp = _out(ids, (M, top_k), _i32, dev, "ids")
    weights, wp = _out(weights, (M, top_k), _f32, dev, "weights")
    if workspace is None:
        workspace = make_workspace(fp8_moe_workspace_size(M, H, I, E, top_k), dev)
    wsp, wsn = _work(workspace)
    _check("fp8_moe_layer", lib().fp8_moe_layer(xp, ldx, wrp, wt, 1 if renormalize else 0, w13p, s13p, w2p, s2p,
                                                yp, idp, wp, M, H, I, E, top_k, wsp, wsn, flags | tf, _stream()))
    return y, ids, weights


def _scores(x, wr, bias):
    """(M, K, row stride, address of x; E, dtype code, address of wr; address of bias; device)."""
    M, H, ldx, xp = _act(x)
    d = _home(x, "x")
    E, Hr, wt, wrp = _matrix(wr, "wr")
    if H != Hr:
        raise ValueError("operand shapes do not agree")
    _there(wr, "wr", d)
    return M, H, ldx, xp, E, wt, wrp, None if bias is None else _in(bias, _f32, E, "bias", d), d


def moe_route_grouped(x, wr, top_k, bias=None, scoring=SCORE_SIGMOID, groups=1, top_groups=1, group_best=2,
                      renormalize=True, scale=1.0, ids=None, weights=None, workspace=None, flags=0):
    """The experts of each token by scores, bias and groups (include/fp8bs.h has
    the rule): x bf16 [M, H] (row stride may exceed H), wr fp32 or bf16 [E, H], bias
    fp32 [E] or None -> (ids int32 [M, top_k] by descending score plus bias, weights
    fp32 [M, top_k]: the scores, over their sum with ``renormalize``, times
    scale).  Workspace of moe_route_workspace_size."""
    M, H, ldx, xp, E, wt, wrp, bp, d = _scores(x, wr, bias)
    dev = x.device
    ids, idp = _make(ids, (M, top_k), _i32, dev, "ids", d)
    weights, wp = _make(weights, (M, top_k), _f32, dev, "weights", d)
    if workspace is None:
        workspace = make_workspace(moe_route_workspace_size(M, E), dev)
    wsp, wsn = _work(workspace)
    _there(workspace, "workspace", d)
    _check("moe_route_grouped", lib().moe_route_grouped(xp, ldx, wrp, wt, bp, M, H, E, top_k, scoring, groups, top_groups,
                                                        group_best, 1 if renormalize else 0, scale, idp, wp, wsp, wsn,
                                                        flags, _stream()))
    return ids, weights


def fp8_moe_layer_grouped(x, wr, top_k, w13, s13, w2, s2, bias=None, scoring=SCORE_SIGMOID, groups=1, top_groups=1,
                          group_best=2, renormalize=True, scale=1.0, y=None, ids=None, weights=None, workspace=None,
                          flags=0):
    """The whole layer, moe_route_grouped and fp8_moe_experts in three kernels:
    (y bf16 [M, H], ids int32 [M, top_k], weights fp32 [M, top_k]); w13 and w2 as in
    fp8_moe_experts, row-major or tiled."""
    M, H, ldx, xp, E, wt, wrp, bp, d = _scores(x, wr, bias)
    I, tf, w13p, s13p, w2p, s2p = _experts(w13, s13, w2, s2, H, E)
    dev = x.device
    y, yp = _make(y, (M, H), _bf16, dev, "y", d)
    ids, idp = _make(ids, (M, top_k), _i32, dev, "ids", d)
    weights, wp = _make(weights, (M, top_k), _f32, dev, "weights", d)
    if workspace is None:
        workspace = make_workspace(fp8_moe_workspace_size(M, H, I, E, top_k), dev)
    wsp, wsn = _work(workspace)
    for t, name in ((w13, "w13"), (s13, "s13"), (w2, "w2"), (s2, "s2"), (workspace, "workspace")):
        _there(t, name, d)
    _check("fp8_moe_layer_grouped",
           lib().fp8_moe_layer_grouped(xp, ldx, wrp, wt, bp, scoring, groups, top_groups, group_best,
                                       1 if renormalize else 0, scale, w13p, s13p, w2p, s2p, yp, idp, wp, M, H, I, E,
                                       top_k, wsp, wsn, flags | tf, _stream()))
    return y, ids, weights


def _fp4_tiles(N, K):
    return ((N + 127) // 128) * ((K + 255) // 256)


def _fp4_atoms(fmt):
    """Scale atoms per 128 rows and 256 K."""
    if fmt != FP4_NV and fmt != FP4_MX:
        raise ValueError("fmt must be FP4_NV or FP4_MX")
    return 4 if fmt == FP4_NV else 2


def _fp4_weights(wq, ws_atoms, w_rows, N, K, fmt):
    """Addresses of packed 4-bit weights (w_rows may be None: all 1, FP4_MX only)."""
    if _torch_module is None:
        _torch()
    tiles = _fp4_tiles(N, K)
    return (_addr(wq, _u8, tiles * 16384, "wq"), _addr(ws_atoms, _u8, tiles * _fp4_atoms(fmt) * 512, "ws_atoms"),
            None if w_rows is None else _addr(w_rows, _f32, N, "w_rows"))


def fp4_quant_weights(w, fmt=FP4_NV, wq=None, ws_atoms=None, w_rows=None):
    """fp32 or bf16 W [N, K] (K % 32 == 0) -> (wq uint8 [ceil(N/128) *
    ceil(K/256), 128, 128] tiled codes, two to a byte, ws_atoms uint8 [tiles *
    4 or 2, 512] scale atoms, w_rows fp32 [N] row scales, None for FP4_MX unless
    given (then all 1))."""
    N, K, wt, wp = _matrix(w, "w")
    tiles, dev = _fp4_tiles(N, K), w.device
    atoms = tiles * _fp4_atoms(fmt)
    wq, qp = _out(wq, (tiles, 128, 128), _u8, dev, "wq")
    ws_atoms, ap = _out(ws_atoms, (atoms, 512), _u8, dev, "ws_atoms")
    rp = None
    if fmt == FP4_NV or w_rows is not None:
        w_rows, rp = _out(w_rows, (N,), _f32, dev, "w_rows")
    _check("fp4_quant_weights", lib().fp4_quant_weights(wp, wt, N, K, fmt, qp, ap, rp, _stream()))
    return wq, ws_atoms, w_rows


def fp4_dequant_weights(wq, ws_atoms, w_rows, n, k, fmt=FP4_NV, w=None, dtype=None):
    """The values [n, k] (fp32, or bf16 with dtype=torch.bfloat16) that packed
    4-bit weights stand for (w_rows None: all 1, FP4_MX only)."""
    N, K = int(n), int(k)
    qp, ap, rp = _fp4_weights(wq, ws_atoms, w_rows, N, K, fmt)
    if dtype is None:
        if w is not None:
            _tensors(w=w)
        dtype = _f32 if w is None else w.dtype
    if dtype is not _f32 and dtype is not _bf16:
        raise TypeError("w must be float32 or bfloat16")
    w, op = _out(w, (N, K), dtype, wq.device, "w")
    _check("fp4_dequant_weights", lib().fp4_dequant_weights(qp, ap, rp, N, K, fmt, op, BF16 if dtype is _bf16 else F32,
                                                            _stream()))
    return w


def fp4_quant_act(x, fmt=FP4_NV, xq=None, xs_atoms=None, x_rows=None, flags=0):
    """bf16 X [M, K] (M <= 512, K % 32 == 0; row stride may exceed K) -> (xq
    uint8 [M, ceil(K/256) * 128], xs_atoms uint8 [ceil(M/128) * ceil(K/256) *
    4 or 2, 512], x_rows fp32 [M], None for FP4_MX unless given)."""
    M, K, ldx, xp = _act(x)
    kt, dev = (K + 255) // 256, x.device
    atoms = (M + 127) // 128 * kt * _fp4_atoms(fmt)
    xq, qp = _out(xq, (M, kt * 128), _u8, dev, "xq")
    xs_atoms, ap = _out(xs_atoms, (atoms, 512), _u8, dev, "xs_atoms")
    rp = None
    if fmt == FP4_NV or x_rows is not None:
        x_rows, rp = _out(x_rows, (M,), _f32, dev, "x_rows")
    _check("fp4_quant_act", lib().fp4_quant_act(xp, M, K, ldx, fmt, qp, ap, rp, flags, _stream()))
    return xq, xs_atoms, x_rows


def fp4_gemm_workspace_size(M, N, K, fmt=FP4_NV):
    n = ctypes.c_size_t(0)
    _check("fp4_gemm_workspace_size", lib().fp4_gemm_workspace_size(M, N, K, fmt, ctypes.byref(n)))
    return n.value


def fp4_gemm(aq, as_atoms, a_rows, wq, ws_atoms, w_rows, n, k, fmt=FP4_NV, y=None, workspace=None, flags=0):
    """Y[M, n] bf16 from 4-bit operands (fp4_quant_act / fp4_quant_weights;
    n = the number of weight rows, k = the unpadded K)."""
    try:
        M, N, K = aq.shape[0], int(n), int(k)
    except AttributeError:
        _tensors(aq=aq)
        raise
    kt = (K + 255) // 256
    if _torch_module is None:
        _torch()
    aqp = _addr(aq, _u8, M * kt * 128, "aq")
    qp, ap, rp = _fp4_weights(wq, ws_atoms, w_rows, N, K, fmt)
    asp = _addr(as_atoms, _u8, (M + 127) // 128 * kt * _fp4_atoms(fmt) * 512, "as_atoms")
    arp = None if a_rows is None else _addr(a_rows, _f32, M, "a_rows")
    y, yp = _out(y, (M, N), _bf16, aq.device, "y")
    if workspace is None:
        workspace = make_workspace(fp4_gemm_workspace_size(M, N, K, fmt), aq.device)
    wsp, wsn = _work(workspace)
    _check("fp4_gemm", lib().fp4_gemm(aqp, asp, arp, qp, ap, rp, yp, M, N, K, fmt, wsp, wsn, flags,
                                      _stream()))
    return y


def fp4_gemm_fused(x, wq, ws_atoms, w_rows, n, fmt=FP4_NV, y=None, workspace=None, flags=0):
    """Y[M, n] bf16 from bf16 activations (row stride may exceed K) and packed
    4-bit weights: the cast into the workspace, then the product."""
    M, K, ldx, xp = _act(x)
    N = int(n)
    qp, ap, rp = _fp4_weights(wq, ws_atoms, w_rows, N, K, fmt)
    y, yp = _out(y, (M, N), _bf16, x.device, "y")
    if workspace is None:
        workspace = make_workspace(fp4_gemm_workspace_size(M, N, K, fmt), x.device)
    wsp, wsn = _work(workspace)
    _check("fp4_gemm_fused", lib().fp4_gemm_fused(xp, ldx, qp, ap, rp, yp, M, N, K, fmt, wsp, wsn, flags,
                                                  _stream()))
    return y


def workspace_status(workspace, clear=False):
    """Device-side failure word of a workspace (synchronises the device)."""
    code = ctypes.c_int(0)
    rc = lib().fp8bs_workspace_status(_ptr(workspace), 1 if clear else 0, ctypes.byref(code))
    if rc not in (0, 7):
        _check("fp8bs_workspace_status", rc)
    return code.value


def split_plan(N, K, bf16=False, num_sms=0, cta=-1):
    """(ctas, units, unit_begin, unit_end) of the K-split schedule."""
    c = ctypes.c_int(0)
    u = ctypes.c_longlong(0)
    b = ctypes.c_longlong(0)
    e = ctypes.c_longlong(0)
    _check("fp8bs_split_plan", lib().fp8bs_split_plan(N, K, 1 if bf16 else 0, num_sms, cta, ctypes.byref(c),
                                                      ctypes.byref(u), ctypes.byref(b), ctypes.byref(e)))
    return c.value, u.value, (b.value if cta >= 0 else None), (e.value if cta >= 0 else None)


def fused_route(M, N, K, num_sms=0, flags=0):
    """'prologue' when fp8_blockscaled_gemm_fused casts the activations in the
    GEMM kernel's prologue for this shape and flags (FLAG_PROLOGUE_CAST, where
    the cache fits), 'separate' when it runs the cast as its own kernel first."""
    v = ctypes.c_int(0)
    _check("fp8bs_fused_route", lib().fp8bs_fused_route(M, N, K, num_sms, flags, ctypes.byref(v)))
    return "prologue" if v.value else "separate"


def gemm_schedule(M, N, K, num_sms=0):
    """dict(npad, token_tiles, ctas, units, split) the FP8 GEMMs use for M tokens."""
    v = [ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0), ctypes.c_longlong(0), ctypes.c_int(0)]
    _check("fp8bs_gemm_schedule", lib().fp8bs_gemm_schedule(M, N, K, num_sms, *[ctypes.byref(a) for a in v]))
    return dict(npad=v[0].value, token_tiles=v[1].value, ctas=v[2].value, units=v[3].value, split=bool(v[4].value))
