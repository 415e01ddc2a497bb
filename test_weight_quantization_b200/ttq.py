"""ctypes binding of libttq (include/ttq.h): same call names, marshalling only.

Every function takes torch tensors that already live on a CUDA device,
passes their device pointers and the current torch stream to the C ABI, and
raises :class:`TTQError` on a non-OK status. No step of the computation runs
in Python; if ``libttq.so`` is missing or cannot be loaded, importing this
module raises, so there is no silent fallback.

Paper: "TTQ: Activation-Aware Test-Time Quantization to Accelerate LLM
Inference On The Fly" (TTQ review, section "Proposed method", bullets 1-7).
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)),
                         "libttq.so")

TTQ_OK = 0
DEVERR_TIMEOUT = 0x1
DEVERR_FP16_RANGE = 0x2
DEVERR_INDEX = 0x4

_DTYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


class TTQError(RuntimeError):
    pass


def _load() -> ctypes.CDLL:
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"{_LIB_PATH} is missing: build it with "
            "`python -m test_weight_quantization_b200.build`")
    lib = ctypes.CDLL(_LIB_PATH)
    P, I64, I, F, SZ = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                        ctypes.c_float, ctypes.c_size_t)
    sig = {
        "ttq_act_stats": [P, I, I64, I64, I64, F, I, P, P],
        "ttq_awq_scales": [P, I64, I64, P, P, P, P],
        "ttq_act_stats_scales": [P, I, I64, I64, I64, I, I64, P, P, P, P, P,
                                 P],
        "ttq_quantize_rtn_grouped": [P, I, I64, I64, I64, P, I, I, P, P, P, P],
        "ttq_w_lowbit_gemm_workspace_size": [I64, I64, I],
        "ttq_w_lowbit_gemm": [P, I, I64, I64, I64, P, P, P, P, I64, I, I, P, P,
                              I, P, I, I64, P, SZ, P],
        "ttq_prepare_activations": [P, I, I64, I64, I64, P, I, P, I, P, P, P],
        "ttq_w_lowbit_gemm_prepared": [P, P, I64, I64, P, P, P, I64, I, I, P,
                                       I, I, P, I, I64, P],
        "ttq_lowrank_add": [P, I, I64, I64, I64, P, P, I, I64, P, I, I64, P],
        "ttq_unpack_codes": [P, I64, I64, I, P, P],
        "ttq_status_string": [I],
        "ttq_device_error": [I],
        "ttq_abi_version": [],
        "ttq_codes_ld": [I64, I],
        "ttq_groups_ld": [I64, I],
        "ttq_selftest_bounded_wait": [I, P, P],
        "ttq_channel_moment_total": [P, I64, I64, P, P],
        "ttq_awq_scales_sharded": [P, I64, I64, I64, P, P, P, P, P],
        "ttq_projection_stats_rows": [I64, I64, I64, I],
        "ttq_w_lowbit_gemm_prepared_stats": [P, P, I64, I64, P, P, P, I64, I,
                                             I, P, I, I, P, I, I64, F, P,
                                             I64, P],
        "ttq_stats_reduce": [P, I64, I64, I, P, P],
        "ttq_quantize_gemm_prepared": [P, I, I64, P, P, P, I64, I64, I64, I,
                                       I, P, I, I, P, I, I64, P, P, P, P],
        "ttq_lowrank_factors_workspace_size": [I64, I64, I],
        "ttq_lowrank_factors": [P, I64, I64, I64, P, P, I, I, P, P, P, SZ, P],
        "ttq_lowrank_residual": [P, I64, I64, I64, P, P, I, P, I64, P],
        "ttq_moe_route": [P, I, I64, I64, I64, P, I, I64, I64, P, I, I, I, F,
                          P, P, P],
        "ttq_moe_lowbit_workspace_size": [I64, I64, I64, I],
        "ttq_moe_lowbit": [P, I, I64, I64, I64, P, P, I, I64, P, P, P, P, I64,
                           P, P, P, P, I, I, I, P, I, I64, P, SZ, P],
        "ttq_adapters_plan_size": [I64, I64],
        "ttq_adapters_plan": [P, I64, I64, P, I64, P],
        "ttq_adapters_add": [P, I, I64, I64, I64, P, P, P, I64, I, I64, P,
                             I64, P, I, I64, P, I64, P],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = I
    lib.ttq_status_string.restype = ctypes.c_char_p
    lib.ttq_w_lowbit_gemm_workspace_size.restype = SZ
    lib.ttq_codes_ld.restype = I64
    lib.ttq_groups_ld.restype = I64
    lib.ttq_projection_stats_rows.restype = I64
    lib.ttq_lowrank_factors_workspace_size.restype = SZ
    lib.ttq_moe_lowbit_workspace_size.restype = SZ
    lib.ttq_adapters_plan_size.restype = I64
    return lib


_lib = _load()

# Names the C ABI exports (include/ttq.h).
EXPORTS = ("ttq_act_stats", "ttq_awq_scales", "ttq_act_stats_scales",
           "ttq_quantize_rtn_grouped",
           "ttq_w_lowbit_gemm_workspace_size", "ttq_w_lowbit_gemm",
           "ttq_prepare_activations", "ttq_w_lowbit_gemm_prepared",
           "ttq_lowrank_add", "ttq_unpack_codes", "ttq_status_string",
           "ttq_device_error", "ttq_abi_version", "ttq_codes_ld",
           "ttq_groups_ld", "ttq_selftest_bounded_wait",
           "ttq_channel_moment_total", "ttq_awq_scales_sharded",
           "ttq_projection_stats_rows", "ttq_w_lowbit_gemm_prepared_stats",
           "ttq_stats_reduce", "ttq_quantize_gemm_prepared",
           "ttq_lowrank_factors_workspace_size", "ttq_lowrank_factors",
           "ttq_lowrank_residual", "ttq_moe_route",
           "ttq_moe_lowbit_workspace_size", "ttq_moe_lowbit",
           "ttq_adapters_plan_size", "ttq_adapters_plan", "ttq_adapters_add")


class _Params(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int), ("group", ctypes.c_int),
                ("alpha", ctypes.c_float), ("lambda_", ctypes.c_float),
                ("p", ctypes.c_float)]


@dataclass(frozen=True)
class TTQParams:
    """Fixed per-layer hyperparameters (Proposed method, bullet 4)."""
    bits: int = 4
    group: int = 128
    alpha: float = 0.5
    lam: float = 0.1
    p: float = 2.0


def _check(status: int, what: str) -> None:
    if status != TTQ_OK:
        raise TTQError(f"{what}: {_lib.ttq_status_string(status).decode()}")


# The current stream's handle and the current device without building the
# objects of torch.cuda (0.1 us instead of 3.4 us per call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream() -> int:
    if _raw_stream is None or _raw_device is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(_raw_device())


def _dev(t: torch.Tensor, name: str) -> None:
    """A CUDA tensor on the current device (the one the call launches on)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TTQError(f"{name} must be a CUDA tensor")
    cur = torch.cuda.current_device() if _raw_device is None \
        else _raw_device()
    if t.get_device() != cur:
        raise TTQError(f"{name} is on {t.device}; the call launches on "
                       f"cuda:{cur}")


def _code(t: torch.Tensor, name: str) -> int:
    """The ttq_dtype of a floating tensor."""
    if t.dtype not in _DTYPE:
        raise TTQError(f"{name} must be float32, bfloat16 or float16, not "
                       f"{t.dtype}")
    return _DTYPE[t.dtype]


def _rows(t: torch.Tensor, name: str) -> int:
    """Row pitch (elements) of a 2D tensor whose rows are contiguous."""
    _dev(t, name)
    if t.dim() != 2 or t.stride(1) != 1:
        raise TTQError(f"{name} must be 2D with contiguous rows")
    return t.stride(0)


_CODE_DTYPES = (torch.int32, torch.uint32)


def _buf(t: torch.Tensor, name: str, dtypes, rows: int,
         cols: int | None = None) -> None:
    """A dense device buffer: at least ``rows`` entries ([rows] vector), or
    at least ``rows`` rows of exactly ``cols`` entries."""
    _dev(t, name)
    if t.dtype is dtypes:  # the usual case, first
        shape = t.shape
        if ((len(shape) == 1 and shape[0] >= rows) if cols is None else
                (len(shape) == 2 and shape[0] >= rows and shape[1] == cols)) \
                and t.is_contiguous():
            return
    dtypes = dtypes if isinstance(dtypes, tuple) else (dtypes,)
    if t.dtype not in dtypes:
        raise TTQError(f"{name} must be {' or '.join(map(str, dtypes))}, "
                       f"not {t.dtype}")
    if cols is None:
        ok = t.dim() == 1 and t.numel() >= rows
        want = f"[{rows}]"
    else:
        ok = t.dim() == 2 and t.shape[0] >= rows and t.shape[1] == cols
        want = f"[{rows}, {cols}]"
    if not ok or not t.is_contiguous():
        raise TTQError(f"{name} must be a dense buffer of shape {want}, got "
                       f"{tuple(t.shape)} with strides {t.stride()}")


def _packed(codes, delta, zero, N: int, K: int, bits: int, group: int):
    """Codes, delta and zero of an [N, K] weight in the packed layout."""
    cl, gl = codes_ld(K, bits), groups_ld(K, group)
    if cl <= 0 or gl <= 0:
        raise TTQError(f"no packed layout for K={K}, bits={bits}, "
                       f"group={group}")
    _buf(codes, "codes", _CODE_DTYPES, N, cl)
    _buf(delta, "delta", torch.float32, N, gl)
    _buf(zero, "zero", torch.uint8, N, gl)


def _out(Y: torch.Tensor, name: str, T: int, N: int) -> int:
    """An output [T, N] with contiguous rows; returns its row pitch."""
    ld = _rows(Y, name)
    _code(Y, name)
    if tuple(Y.shape) != (T, N):
        raise TTQError(f"{name} must have shape ({T}, {N}), got "
                       f"{tuple(Y.shape)}")
    return ld


def _factors(A, B, N: int, K: int, dtype) -> int:
    """The low-rank factors A [r, K] and B [N, r] (both or neither);
    returns r."""
    if (A is None) != (B is None):
        raise TTQError("A and B come together")
    if A is None:
        return 0
    r = A.shape[0] if A.dim() == 2 else -1
    _buf(A, "A", dtype, r, K)
    _buf(B, "B", dtype, N, r)
    if B.shape[0] != N:
        raise TTQError(f"B must have {N} rows, got {B.shape[0]}")
    return r


def _ptr(t):
    return None if t is None else t.data_ptr()


def abi_version() -> int:
    return int(_lib.ttq_abi_version())


@functools.lru_cache(maxsize=4096)
def codes_ld(K: int, bits: int) -> int:
    """Row pitch (uint32 words) of the packed codes."""
    return int(_lib.ttq_codes_ld(K, bits))


@functools.lru_cache(maxsize=4096)
def groups_ld(K: int, group: int) -> int:
    """Row pitch (entries) of delta and zero."""
    return int(_lib.ttq_groups_ld(K, group))


def device_error(clear: bool = True) -> int:
    """Sticky device error bits (synchronising read)."""
    return int(_lib.ttq_device_error(1 if clear else 0))


def selftest_bounded_wait(arrive: bool) -> tuple[bool, int]:
    """Runs the kernels' bounded wait on a barrier that completes (arrive)
    or never does. Returns (whether the wait completed, the device error
    bits, which are cleared). Synchronises the device."""
    out = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    _check(_lib.ttq_selftest_bounded_wait(1 if arrive else 0, out.data_ptr(),
                                          _stream()),
           "ttq_selftest_bounded_wait")
    torch.cuda.synchronize()
    done = int(out.item())
    if done not in (0, 1):
        raise TTQError(f"ttq_selftest_bounded_wait wrote {done}")
    return done == 1, device_error(clear=True)


def act_stats(X: torch.Tensor, p: float = 2.0, out: torch.Tensor | None = None,
              accumulate: bool = False) -> torch.Tensor:
    """Step 1: out[j] (+)= sum_t |X[t, j]|^p, fp32 [K]."""
    ldx = _rows(X, "X")
    T, K = X.shape
    if out is None:
        out = torch.empty(K, dtype=torch.float32, device=X.device)
    _buf(out, "out", torch.float32, K)
    _check(_lib.ttq_act_stats(X.data_ptr(), _code(X, "X"), T, K, ldx,
                              float(p), 1 if accumulate else 0,
                              out.data_ptr(), _stream()), "ttq_act_stats")
    return out


def awq_scales(sums: torch.Tensor, T_total: int, alpha: float = 0.5,
               lam: float = 0.1, p: float = 2.0, s=None, inv_s=None):
    """Step 2: (s, inv_s) fp32 [K] from the channel sums."""
    _buf(sums, "sums", torch.float32, 0)
    K = sums.shape[0]
    s = torch.empty(K, dtype=torch.float32, device=sums.device) if s is None \
        else s
    inv_s = torch.empty_like(s) if inv_s is None else inv_s
    _buf(s, "s", torch.float32, K)
    _buf(inv_s, "inv_s", torch.float32, K)
    prm = _Params(0, 0, alpha, lam, p)
    _check(_lib.ttq_awq_scales(sums.data_ptr(), int(T_total), K,
                               ctypes.addressof(prm), s.data_ptr(),
                               inv_s.data_ptr(), _stream()), "ttq_awq_scales")
    return s, inv_s


def channel_moment_total(sums: torch.Tensor, T_total: int,
                         out: torch.Tensor | None = None) -> torch.Tensor:
    """sum_j sums[j] / T_total of one shard's channels, fp64 [1] on the
    device (the shard's part of the shrinkage mean)."""
    _buf(sums, "sums", torch.float32, 0)
    K = sums.shape[0]
    out = torch.empty(1, dtype=torch.float64, device=sums.device) \
        if out is None else out
    _buf(out, "out", torch.float64, 1)
    _check(_lib.ttq_channel_moment_total(sums.data_ptr(), int(T_total), K,
                                         out.data_ptr(), _stream()),
           "ttq_channel_moment_total")
    return out


def awq_scales_sharded(sums: torch.Tensor, T_total: int, K_total: int,
                       total: torch.Tensor, alpha: float = 0.5,
                       lam: float = 0.1, p: float = 2.0, s=None, inv_s=None):
    """Step 2 of one shard of the input channels: (s, inv_s) fp32 [K] with
    the shrinkage mean total / K_total, total being the fp64 [1] sum of every
    shard's channel_moment_total."""
    _buf(sums, "sums", torch.float32, 0)
    _buf(total, "total", torch.float64, 1)
    K = sums.shape[0]
    s = torch.empty(K, dtype=torch.float32, device=sums.device) if s is None \
        else s
    inv_s = torch.empty_like(s) if inv_s is None else inv_s
    _buf(s, "s", torch.float32, K)
    _buf(inv_s, "inv_s", torch.float32, K)
    prm = _Params(0, 0, alpha, lam, p)
    _check(_lib.ttq_awq_scales_sharded(sums.data_ptr(), int(T_total), K,
                                       int(K_total), ctypes.addressof(prm),
                                       total.data_ptr(), s.data_ptr(),
                                       inv_s.data_ptr(), _stream()),
           "ttq_awq_scales_sharded")
    return s, inv_s


def new_counter(device=None) -> torch.Tensor:
    """A zeroed device word for act_stats_scales (one per concurrent
    stream; each call leaves it zero again)."""
    return torch.zeros(1, dtype=torch.int32, device=device or "cuda")


def act_stats_scales(X: torch.Tensor, counter: torch.Tensor,
                     alpha: float = 0.5, lam: float = 0.1, p: float = 2.0,
                     sums=None, s=None, inv_s=None, accumulate: bool = False,
                     T_total: int | None = None):
    """Steps 1 and 2 in one launch: (sums, s, inv_s), each fp32 [K]."""
    ldx = _rows(X, "X")
    _buf(counter, "counter", _CODE_DTYPES, 1)
    T, K = X.shape
    f32 = dict(dtype=torch.float32, device=X.device)
    sums = torch.empty(K, **f32) if sums is None else sums
    s = torch.empty(K, **f32) if s is None else s
    inv_s = torch.empty(K, **f32) if inv_s is None else inv_s
    for t, name in ((sums, "sums"), (s, "s"), (inv_s, "inv_s")):
        _buf(t, name, torch.float32, K)
    prm = _Params(0, 0, alpha, lam, p)
    _check(_lib.ttq_act_stats_scales(
        X.data_ptr(), _code(X, "X"), T, K, ldx, 1 if accumulate else 0,
        int(T if T_total is None else T_total), ctypes.addressof(prm),
        sums.data_ptr(), s.data_ptr(), inv_s.data_ptr(), counter.data_ptr(),
        _stream()), "ttq_act_stats_scales")
    return sums, s, inv_s


def quantize_rtn_grouped(W: torch.Tensor, s: torch.Tensor | None, bits: int,
                         group: int, codes=None, delta=None, zero=None):
    """Step 3: packed codes [N, codes_ld] u32 (held as int32), delta
    [N, groups_ld] fp32, zero [N, groups_ld] u8 (see ttq.h for the layout)."""
    ldw = _rows(W, "W")
    N, K = W.shape
    dev = W.device
    if codes is None:
        codes = torch.empty((N, codes_ld(K, bits)), dtype=torch.int32,
                            device=dev)
    if delta is None:
        delta = torch.empty((N, groups_ld(K, group)), dtype=torch.float32,
                            device=dev)
    if zero is None:
        zero = torch.empty((N, groups_ld(K, group)), dtype=torch.uint8,
                           device=dev)
    if s is not None:
        _buf(s, "s", torch.float32, K)
    _packed(codes, delta, zero, N, K, bits, group)
    _check(_lib.ttq_quantize_rtn_grouped(
        W.data_ptr(), _code(W, "W"), N, K, ldw, _ptr(s), bits, group,
        codes.data_ptr(), delta.data_ptr(), zero.data_ptr(), _stream()),
        "ttq_quantize_rtn_grouped")
    return codes, delta, zero


def workspace_size(T: int, K: int, r: int = 0) -> int:
    return int(_lib.ttq_w_lowbit_gemm_workspace_size(T, K, r))


def w_lowbit_gemm(X: torch.Tensor, inv_s: torch.Tensor, codes: torch.Tensor,
                  delta: torch.Tensor, zero: torch.Tensor, N: int, bits: int,
                  group: int, A: torch.Tensor | None = None,
                  B: torch.Tensor | None = None,
                  out: torch.Tensor | None = None, out_dtype=None,
                  workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Step 4: Y = (X diag(inv_s)) W_hat^T [+ (X A^T) B^T], [T, N]."""
    ldx = _rows(X, "X")
    T, K = X.shape
    r = _factors(A, B, N, K, X.dtype)
    _buf(inv_s, "inv_s", torch.float32, K)
    _packed(codes, delta, zero, N, K, bits, group)
    if out is None:
        out = torch.empty((T, N), dtype=out_dtype or X.dtype, device=X.device)
    ldy = _out(out, "out", T, N)
    need = workspace_size(T, K, r)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
    _dev(workspace, "workspace")
    if not workspace.is_contiguous():
        raise TTQError("workspace must be contiguous")
    _check(_lib.ttq_w_lowbit_gemm(
        X.data_ptr(), _code(X, "X"), T, K, ldx, inv_s.data_ptr(),
        codes.data_ptr(), delta.data_ptr(), zero.data_ptr(), N, bits, group,
        _ptr(A), _ptr(B), r, out.data_ptr(), _code(out, "out"), ldy,
        workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _stream()), "ttq_w_lowbit_gemm")
    return out


def prepare_activations(X: torch.Tensor, inv_s: torch.Tensor, bits: int,
                        A: torch.Tensor | None = None, Xs=None, U=None):
    """Activation side of step 4: Xs = fp16(X diag(inv_s)) [T, K] (channels
    ordered for `bits`-bit codes, see ttq.h) and, with low-rank factors,
    U = fp16(X A^T) zero-padded to [T, 64]."""
    ldx = _rows(X, "X")
    T, K = X.shape
    r = 0
    if A is not None:
        r = A.shape[0] if A.dim() == 2 else -1
        _buf(A, "A", X.dtype, r, K)
    _buf(inv_s, "inv_s", torch.float32, K)
    if Xs is None:
        Xs = torch.empty((T, K), dtype=torch.float16, device=X.device)
    _buf(Xs, "Xs", torch.float16, T, K)
    if r and U is None:
        U = torch.empty((T, 64), dtype=torch.float16, device=X.device)
    if r:
        _buf(U, "U", torch.float16, T, 64)
    _check(_lib.ttq_prepare_activations(
        X.data_ptr(), _code(X, "X"), T, K, ldx, inv_s.data_ptr(), bits,
        _ptr(A), r, Xs.data_ptr(), _ptr(U) if r else None, _stream()),
        "ttq_prepare_activations")
    return Xs, (U if r else None)


def w_lowbit_gemm_prepared(Xs: torch.Tensor, U: torch.Tensor | None,
                           codes: torch.Tensor, delta: torch.Tensor,
                           zero: torch.Tensor, N: int, bits: int, group: int,
                           B: torch.Tensor | None = None,
                           out: torch.Tensor | None = None,
                           out_dtype=torch.bfloat16) -> torch.Tensor:
    """The projection on prepared operands (one kernel launch; one or two
    tokens run on CUDA cores, more on tensor cores)."""
    _dev(Xs, "Xs")
    if Xs.dim() != 2:
        raise TTQError("Xs must be 2D")
    T, K = Xs.shape
    _buf(Xs, "Xs", torch.float16, T, K)
    r = 0
    if B is not None:
        r = B.shape[1] if B.dim() == 2 else -1
        _buf(B, "B", B.dtype, N, r)
        _code(B, "B")
        if B.shape[0] != N:
            raise TTQError(f"B must have {N} rows, got {B.shape[0]}")
        if U is None:
            raise TTQError("a low-rank projection needs U")
        _buf(U, "U", torch.float16, T, 64)
    _packed(codes, delta, zero, N, K, bits, group)
    if out is None:
        out = torch.empty((T, N), dtype=out_dtype, device=Xs.device)
    ldy = _out(out, "out", T, N)
    _check(_lib.ttq_w_lowbit_gemm_prepared(
        Xs.data_ptr(), _ptr(U) if r else None, T, K, codes.data_ptr(),
        delta.data_ptr(), zero.data_ptr(), N, bits, group, _ptr(B),
        _code(B, "B") if r else 0, r, out.data_ptr(), _code(out, "out"),
        ldy, _stream()), "ttq_w_lowbit_gemm_prepared")
    return out


def quantize_gemm_prepared(W: torch.Tensor, s: torch.Tensor, Xs: torch.Tensor,
                           U: torch.Tensor | None, bits: int, group: int,
                           B: torch.Tensor | None = None,
                           out: torch.Tensor | None = None,
                           out_dtype=torch.bfloat16, store_codes: bool = True,
                           codes=None, delta=None, zero=None):
    """Steps 3 and 4 in one launch (the projection quantizes the bf16 W
    itself): Y [T, N], and (codes, delta, zero) of the quantized weights
    unless store_codes is False (then None)."""
    ldw = _rows(W, "W")
    N, K = W.shape
    _buf(s, "s", torch.float32, K)
    _dev(Xs, "Xs")
    T = Xs.shape[0]
    _buf(Xs, "Xs", torch.float16, T, K)
    r = 0
    if B is not None:
        r = B.shape[1] if B.dim() == 2 else -1
        _buf(B, "B", B.dtype, N, r)
        if B.shape[0] != N:
            raise TTQError(f"B must have {N} rows, got {B.shape[0]}")
        if U is None:
            raise TTQError("a low-rank projection needs U")
        _buf(U, "U", torch.float16, T, 64)
    if store_codes:
        dev = W.device
        cl, gl = codes_ld(K, bits), groups_ld(K, group)
        codes = torch.zeros((N, cl), dtype=torch.int32, device=dev) \
            if codes is None else codes
        delta = torch.zeros((N, gl), dtype=torch.float32, device=dev) \
            if delta is None else delta
        zero = torch.zeros((N, gl), dtype=torch.uint8, device=dev) \
            if zero is None else zero
        _packed(codes, delta, zero, N, K, bits, group)
    if out is None:
        out = torch.empty((T, N), dtype=out_dtype, device=Xs.device)
    ldy = _out(out, "out", T, N)
    _check(_lib.ttq_quantize_gemm_prepared(
        W.data_ptr(), _code(W, "W"), ldw, s.data_ptr(), Xs.data_ptr(),
        _ptr(U) if r else None, T, K, N, bits, group, _ptr(B),
        _code(B, "B") if r else 0, r, out.data_ptr(), _code(out, "out"), ldy,
        _ptr(codes) if store_codes else None,
        _ptr(delta) if store_codes else None,
        _ptr(zero) if store_codes else None, _stream()),
        "ttq_quantize_gemm_prepared")
    return out, ((codes, delta, zero) if store_codes else None)


def projection_stats_rows(T: int, N: int, K: int, bits: int) -> int:
    """Partial rows the fused output statistic needs (0: none for T)."""
    return int(_lib.ttq_projection_stats_rows(T, N, K, bits))


def w_lowbit_gemm_prepared_stats(Xs: torch.Tensor, U: torch.Tensor | None,
                                 codes: torch.Tensor, delta: torch.Tensor,
                                 zero: torch.Tensor, N: int, bits: int,
                                 group: int, B: torch.Tensor | None = None,
                                 p: float = 2.0, out: torch.Tensor | None = None,
                                 out_dtype=torch.bfloat16,
                                 stats: torch.Tensor | None = None):
    """The projection on prepared operands plus the partial statistic of its
    stored output: (Y [T, N], stats [rows, N] fp32); stats_reduce adds the
    rows into the next layer's channel sums."""
    _dev(Xs, "Xs")
    if Xs.dim() != 2:
        raise TTQError("Xs must be 2D")
    T, K = Xs.shape
    _buf(Xs, "Xs", torch.float16, T, K)
    rows = projection_stats_rows(T, N, K, bits)
    if rows == 0:
        raise TTQError(f"no fused statistic for T = {T} (prefill only)")
    r = 0
    if B is not None:
        r = B.shape[1] if B.dim() == 2 else -1
        _buf(B, "B", B.dtype, N, r)
        _code(B, "B")
        if B.shape[0] != N:
            raise TTQError(f"B must have {N} rows, got {B.shape[0]}")
        if U is None:
            raise TTQError("a low-rank projection needs U")
        _buf(U, "U", torch.float16, T, 64)
    _packed(codes, delta, zero, N, K, bits, group)
    if out is None:
        out = torch.empty((T, N), dtype=out_dtype, device=Xs.device)
    ldy = _out(out, "out", T, N)
    if stats is None:
        stats = torch.empty((rows, N), dtype=torch.float32, device=Xs.device)
    _buf(stats, "stats", torch.float32, rows, N)
    if stats.shape[0] != rows:
        raise TTQError(f"stats must have {rows} rows")
    _check(_lib.ttq_w_lowbit_gemm_prepared_stats(
        Xs.data_ptr(), _ptr(U) if r else None, T, K, codes.data_ptr(),
        delta.data_ptr(), zero.data_ptr(), N, bits, group, _ptr(B),
        _code(B, "B") if r else 0, r, out.data_ptr(), _code(out, "out"),
        ldy, float(p), stats.data_ptr(), rows, _stream()),
        "ttq_w_lowbit_gemm_prepared_stats")
    return out, stats


def stats_reduce(partials: torch.Tensor, out: torch.Tensor | None = None,
                 accumulate: bool = False) -> torch.Tensor:
    """out[n] (+)= sum_i partials[i][n], fp32 [N]."""
    _dev(partials, "partials")
    if partials.dim() != 2:
        raise TTQError("partials must be 2D")
    P, N = partials.shape
    _buf(partials, "partials", torch.float32, P, N)
    if out is None:
        out = torch.empty(N, dtype=torch.float32, device=partials.device)
    _buf(out, "out", torch.float32, N)
    _check(_lib.ttq_stats_reduce(partials.data_ptr(), P, N, int(accumulate),
                                 out.data_ptr(), _stream()),
           "ttq_stats_reduce")
    return out


def lowrank_add(X: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                Y: torch.Tensor) -> torch.Tensor:
    """Y += (X A^T) B^T in place."""
    ldx = _rows(X, "X")
    T, K = X.shape
    _dev(B, "B")
    N = B.shape[0]
    r = _factors(A, B, N, K, X.dtype)
    ldy = _out(Y, "Y", T, N)
    _check(_lib.ttq_lowrank_add(X.data_ptr(), _code(X, "X"), T, K, ldx,
                                A.data_ptr(), B.data_ptr(), r, N, Y.data_ptr(),
                                _code(Y, "Y"), ldy, _stream()),
           "ttq_lowrank_add")
    return Y


def lowrank_factors_workspace_size(N: int, K: int, r: int) -> int:
    return int(_lib.ttq_lowrank_factors_workspace_size(N, K, r))


def lowrank_factors(W: torch.Tensor, s: torch.Tensor, omega: torch.Tensor,
                    iters: int = 1, workspace: torch.Tensor | None = None):
    """Per-prompt low-rank factors (B [N, r], A [r, K], bf16) of the bf16
    weight W for the scales s, from the probe vectors omega [r, K] (fp32):
    randomized subspace iteration on W diag(s), B = Q, A = Q^T W."""
    ldw = _rows(W, "W")
    N, K = W.shape
    if W.dtype != torch.bfloat16:
        raise TTQError("W must be bfloat16")
    _buf(s, "s", torch.float32, K)
    if omega.dim() != 2 or omega.shape[1] != K:
        raise TTQError(f"omega must be [r, {K}], got {tuple(omega.shape)}")
    r = omega.shape[0]
    _buf(omega, "omega", torch.float32, r, K)
    need = lowrank_factors_workspace_size(N, K, r)
    if need == 0:
        raise TTQError(f"no factor workspace for N={N}, K={K}, r={r}")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=W.device)
    _buf(workspace, "workspace", torch.uint8, need)
    B = torch.empty((N, r), dtype=torch.bfloat16, device=W.device)
    A = torch.empty((r, K), dtype=torch.bfloat16, device=W.device)
    _check(_lib.ttq_lowrank_factors(W.data_ptr(), N, K, ldw, s.data_ptr(),
                                    omega.data_ptr(), r, int(iters),
                                    B.data_ptr(), A.data_ptr(),
                                    workspace.data_ptr(), workspace.numel(),
                                    _stream()), "ttq_lowrank_factors")
    return B, A


def lowrank_residual(W: torch.Tensor, B: torch.Tensor, A: torch.Tensor,
                     out: torch.Tensor | None = None) -> torch.Tensor:
    """R = bf16(W - B A) (bf16 W [N, K], B [N, r], A [r, K])."""
    ldw = _rows(W, "W")
    N, K = W.shape
    if W.dtype != torch.bfloat16:
        raise TTQError("W must be bfloat16")
    r = _factors(A, B, N, K, torch.bfloat16)
    if out is None:
        out = torch.empty((N, K), dtype=torch.bfloat16, device=W.device)
    ldr = _out(out, "out", N, K)
    if out.dtype != torch.bfloat16:
        raise TTQError("out must be bfloat16")
    _check(_lib.ttq_lowrank_residual(W.data_ptr(), N, K, ldw, B.data_ptr(),
                                     A.data_ptr(), r, out.data_ptr(), ldr,
                                     _stream()), "ttq_lowrank_residual")
    return out


_SCORE = {"softmax": 0, "sigmoid": 1}
_ACT = {"silu": 0, "gelu": 1}


def _named(table: dict, value, name: str) -> int:
    if value not in table:
        raise TTQError(f"{name} must be one of {', '.join(table)}, not "
                       f"{value!r}")
    return table[value]


def moe_route(X: torch.Tensor, W: torch.Tensor, top_k: int,
              bias: torch.Tensor | None = None, score: str = "softmax",
              renormalize: bool = True, scaling: float = 1.0,
              ids: torch.Tensor | None = None,
              weights: torch.Tensor | None = None):
    """Each token's top_k experts of the router W [E, K]: (ids int32, weights
    fp32), both [T, top_k], the best expert first. ``score`` is "softmax" or
    "sigmoid"; ``bias`` [E] fp32 takes part in the choice only."""
    ldx, ldw = _rows(X, "X"), _rows(W, "W")
    T, K = X.shape
    E = W.shape[0]
    if W.shape[1] != K:
        raise TTQError(f"W must have {K} columns, got {W.shape[1]}")
    if bias is not None:
        _buf(bias, "bias", torch.float32, E)
    if ids is None:
        ids = X.new_empty((T, top_k), dtype=torch.int32)
    else:
        _buf(ids, "ids", torch.int32, T, top_k)
    if weights is None:
        weights = X.new_empty((T, top_k), dtype=torch.float32)
    else:
        _buf(weights, "weights", torch.float32, T, top_k)
    _check(_lib.ttq_moe_route(
        X.data_ptr(), _code(X, "X"), T, K, ldx, W.data_ptr(), _code(W, "W"),
        E, ldw, _ptr(bias), int(top_k), _named(_SCORE, score, "score"),
        1 if renormalize else 0, float(scaling), ids.data_ptr(),
        weights.data_ptr(), _stream()), "ttq_moe_route")
    return ids, weights


@functools.lru_cache(maxsize=4096)
def moe_lowbit_workspace_size(T: int, K: int, I: int, top_k: int) -> int:
    return int(_lib.ttq_moe_lowbit_workspace_size(T, K, I, top_k))


def moe_lowbit(X: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor,
               inv_s: torch.Tensor, up, inv_s_mid: torch.Tensor, down,
               bits: int, group: int, act: str = "silu",
               out: torch.Tensor | None = None, out_dtype=None,
               workspace: torch.Tensor | None = None) -> torch.Tensor:
    """A mixture-of-experts layer on packed experts for up to 64 tokens:
    Y[t] = sum_i weights[t, i] D_e (act(G_e x) * (U_e x) * inv_s_mid[e]),
    e = ids[t, i], x = X[t] * inv_s. ``up`` is (codes, delta, zero) of the E
    stacked [2I, K] weights (gate rows first), ``down`` of the E stacked
    [K, I] weights, both from quantize_rtn_grouped; inv_s_mid is [E, I]
    fp32. A negative id is no expert. ``act`` is "silu" or "gelu" (tanh)."""
    ldx = _rows(X, "X")
    T, K = X.shape
    _dev(inv_s_mid, "inv_s_mid")
    if inv_s_mid.dim() != 2:
        raise TTQError("inv_s_mid must be [E, I]")
    E, I = inv_s_mid.shape
    _buf(inv_s_mid, "inv_s_mid", torch.float32, E, I)
    _dev(ids, "ids")
    if ids.dim() != 2:
        raise TTQError("ids must be [T, top_k]")
    top_k = ids.shape[1]
    _buf(ids, "ids", torch.int32, T, top_k)
    _buf(weights, "weights", torch.float32, T, top_k)
    _buf(inv_s, "inv_s", torch.float32, K)
    _packed(*up, E * 2 * I, K, bits, group)
    _packed(*down, E * K, I, bits, group)
    if out is None:
        out = X.new_empty((T, K), dtype=out_dtype or X.dtype)
        ldy = K
    else:
        ldy = _out(out, "out", T, K)
    need = moe_lowbit_workspace_size(T, K, I, top_k)
    if workspace is None:
        workspace = X.new_empty(max(need, 16), dtype=torch.uint8)
    else:
        _buf(workspace, "workspace", torch.uint8, need)
    _check(_lib.ttq_moe_lowbit(
        X.data_ptr(), _code(X, "X"), T, K, ldx, ids.data_ptr(),
        weights.data_ptr(), top_k, E, inv_s.data_ptr(), up[0].data_ptr(),
        up[1].data_ptr(), up[2].data_ptr(), I, inv_s_mid.data_ptr(),
        down[0].data_ptr(), down[1].data_ptr(), down[2].data_ptr(), bits,
        group, _named(_ACT, act, "act"), out.data_ptr(), _code(out, "out"),
        ldy, workspace.data_ptr(), workspace.numel(), _stream()),
        "ttq_moe_lowbit")
    return out


@functools.lru_cache(maxsize=4096)
def _plan_size(T: int, L: int) -> int:
    return int(_lib.ttq_adapters_plan_size(T, L))


def adapters_plan(index: torch.Tensor, L: int,
                  plan: torch.Tensor | None = None) -> torch.Tensor:
    """Groups a batch's tokens by adapter: ``index`` [T] int32 is each
    token's adapter of L, negative for none. The plan (int32) serves every
    adapters_add of the batch."""
    _buf(index, "index", torch.int32, 0)
    T = index.shape[0]
    need = _plan_size(T, int(L))
    if need <= 0:
        raise TTQError(f"no adapter plan for T={T}, L={L}")
    if plan is None:
        plan = torch.empty(need, dtype=torch.int32, device=index.device)
    _buf(plan, "plan", torch.int32, need)
    _check(_lib.ttq_adapters_plan(index.data_ptr(), T, int(L),
                                  plan.data_ptr(), plan.numel(), _stream()),
           "ttq_adapters_plan")
    return plan


def adapters_add(X: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                 plan: torch.Tensor, Y: torch.Tensor,
                 scale: torch.Tensor | None = None,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """Y + scale[a] (X A_a^T) B_a^T of each token's adapter a, in place unless
    ``out`` is given. A [L, r, K], B [L, N, r], scale [L] fp32; ``plan`` from
    adapters_plan for this batch and L."""
    ldx = _rows(X, "X")
    T, K = X.shape
    for t, name in ((A, "A"), (B, "B")):
        _dev(t, name)
        if t.dim() != 3 or not t.is_contiguous() or t.dtype != X.dtype:
            raise TTQError(f"{name} must be a dense 3D {X.dtype} tensor")
    L, r, N = A.shape[0], A.shape[1], B.shape[1]
    if tuple(A.shape) != (L, r, K) or tuple(B.shape) != (L, N, r):
        raise TTQError(f"A must be [L, r, {K}] and B [L, N, r], got "
                       f"{tuple(A.shape)} and {tuple(B.shape)}")
    if scale is not None:
        _buf(scale, "scale", torch.float32, L)
    ldy = ldo = _out(Y, "Y", T, N)
    if out is None:
        out = Y
    else:
        ldo = _out(out, "out", T, N)
    if out.dtype != Y.dtype:
        raise TTQError(f"out must be {Y.dtype}, got {out.dtype}")
    _buf(plan, "plan", torch.int32, max(_plan_size(T, L), 1))
    _check(_lib.ttq_adapters_add(
        X.data_ptr(), _code(X, "X"), T, K, ldx, A.data_ptr(), B.data_ptr(),
        _ptr(scale), L, r, N, plan.data_ptr(), plan.numel(), Y.data_ptr(),
        _code(Y, "Y"), ldy, out.data_ptr(), ldo, _stream()),
        "ttq_adapters_add")
    return out


def unpack_codes(codes: torch.Tensor, K: int, bits: int) -> torch.Tensor:
    """One uint8 per weight, [N, K]."""
    _dev(codes, "codes")
    N = codes.shape[0]
    _buf(codes, "codes", _CODE_DTYPES, N, codes_ld(K, bits))
    q = torch.empty((N, K), dtype=torch.uint8, device=codes.device)
    _check(_lib.ttq_unpack_codes(codes.data_ptr(), N, K, bits, q.data_ptr(),
                                 _stream()), "ttq_unpack_codes")
    return q


class TTQLinear:
    """One linear layer run the TTQ way: per prompt, statistics and scales
    (one launch) -> quantize -> low-bit projection (+ optional static
    low-rank term).

    ``W`` is the stored weight ([N, K], or the residual W - B A when ``A`` and
    ``B`` are given). Buffers are allocated once per (T) and reused; the
    layer's arrival counter makes concurrent use of one layer object on
    several streams unsafe (use one object per stream).
    """

    def __init__(self, W: torch.Tensor, params: TTQParams, A=None, B=None):
        self.W, self.A, self.B, self.prm = W, A, B, params
        N, K = W.shape
        dev = W.device
        self.sums = torch.empty(K, dtype=torch.float32, device=dev)
        self.s = torch.empty(K, dtype=torch.float32, device=dev)
        self.inv_s = torch.empty(K, dtype=torch.float32, device=dev)
        self.counter = new_counter(dev)
        self.codes = torch.empty((N, codes_ld(K, params.bits)),
                                 dtype=torch.int32, device=dev)
        gl = groups_ld(K, params.group)
        self.delta = torch.empty((N, gl), dtype=torch.float32, device=dev)
        self.zero = torch.empty((N, gl), dtype=torch.uint8, device=dev)
        self._ws = None

    def calibrate(self, X: torch.Tensor) -> None:
        """Online statistics and quantization from this prompt's input."""
        p = self.prm
        act_stats_scales(X, self.counter, p.alpha, p.lam, p.p, self.sums,
                         self.s, self.inv_s)
        quantize_rtn_grouped(self.W, self.s, p.bits, p.group, self.codes,
                             self.delta, self.zero)

    def project(self, X: torch.Tensor, out: torch.Tensor | None = None,
                adapters: "tuple[AdapterBank, torch.Tensor] | None" = None):
        """The projection of X; with ``adapters`` (a bank and the batch's
        plan) each token's adapter is added to it."""
        T, K = X.shape
        r = 0 if self.A is None else self.A.shape[0]
        need = workspace_size(T, K, r)
        if self._ws is None or self._ws.numel() < need:
            self._ws = torch.empty(need, dtype=torch.uint8, device=X.device)
        Y = w_lowbit_gemm(X, self.inv_s, self.codes, self.delta, self.zero,
                          self.W.shape[0], self.prm.bits, self.prm.group,
                          self.A, self.B, out=out, workspace=self._ws)
        if adapters is not None:
            bank, plan = adapters
            bank.add(X, plan, Y)
        return Y

    def __call__(self, X: torch.Tensor, out: torch.Tensor | None = None,
                 adapters: "tuple[AdapterBank, torch.Tensor] | None" = None):
        self.calibrate(X)
        return self.project(X, out, adapters)


class AdapterBank:
    """The low-rank adapters of one layer: A [L, r, K], B [L, N, r] (an
    adapter of a lower rank padded with zeros) and scale [L] fp32. One plan
    per batch serves the banks of all layers with L adapters."""

    def __init__(self, A: torch.Tensor, B: torch.Tensor,
                 scale: torch.Tensor | None = None):
        self.A, self.B, self.scale = A, B, scale

    def plan(self, index: torch.Tensor) -> torch.Tensor:
        """The batch's plan from each token's adapter (negative: none)."""
        return adapters_plan(index, self.A.shape[0])

    def add(self, X: torch.Tensor, plan: torch.Tensor, Y: torch.Tensor,
            out: torch.Tensor | None = None) -> torch.Tensor:
        return adapters_add(X, self.A, self.B, plan, Y, self.scale, out)


class TTQMoE:
    """A mixture-of-experts layer run the TTQ way.

    ``prompt(X)``: statistics and scales of the layer's input, shared by all
    experts, and every expert's gate and up weights quantized by them; then,
    expert by expert, its tokens' projection, the statistics and scales of
    its own intermediate activations, and its down weight quantized by those.
    An expert that meets no token of the prompt keeps scales of 1 for its
    down weight. ``decode(X)`` runs up to 64 tokens on the packed experts:
    the router and the whole layer, without a copy to the host.

    ``router`` [E, K], ``W_up`` [E, 2I, K] (gate rows first), ``W_down``
    [E, K, I]. One object serves one stream at a time.
    """

    def __init__(self, router: torch.Tensor, W_up: torch.Tensor,
                 W_down: torch.Tensor, params: TTQParams, top_k: int,
                 act: str = "silu", score: str = "softmax",
                 bias: torch.Tensor | None = None, renormalize: bool = True,
                 scaling: float = 1.0):
        E, K, I = W_down.shape
        if tuple(W_up.shape) != (E, 2 * I, K) or \
                tuple(router.shape) != (E, K):
            raise TTQError(f"router must be [E, K] and W_up [E, 2I, K] for "
                           f"W_down {tuple(W_down.shape)}, got "
                           f"{tuple(router.shape)} and {tuple(W_up.shape)}")
        _named(_ACT, act, "act")
        _named(_SCORE, score, "score")
        self.router, self.W_up, self.W_down = router, W_up, W_down
        self.prm, self.top_k, self.act = params, top_k, act
        self.route_args = dict(bias=bias, score=score,
                               renormalize=renormalize, scaling=scaling)
        f32 = dict(dtype=torch.float32, device=W_up.device)
        self.sums = torch.empty(K, **f32)
        self.s, self.inv_s = torch.empty(K, **f32), torch.empty(K, **f32)
        self.sums_mid = torch.empty(I, **f32)
        self.s_mid = torch.ones(E, I, **f32)
        self.inv_s_mid = torch.ones(E, I, **f32)
        self.counter = new_counter(W_up.device)
        self.up = self._packed_buffers(E * 2 * I, K)
        self.down = self._packed_buffers(E * K, I)
        self._ws = None

    def _packed_buffers(self, N: int, K: int):
        dev, gl = self.W_up.device, groups_ld(K, self.prm.group)
        return (torch.empty((N, codes_ld(K, self.prm.bits)),
                            dtype=torch.int32, device=dev),
                torch.empty((N, gl), dtype=torch.float32, device=dev),
                torch.empty((N, gl), dtype=torch.uint8, device=dev))

    def route(self, X: torch.Tensor):
        """(ids, weights) of the tokens' experts."""
        return moe_route(X, self.router, self.top_k, **self.route_args)

    def prompt(self, X: torch.Tensor) -> torch.Tensor:
        """Quantizes the experts for this prompt and runs it, [T, K]."""
        p = self.prm
        E, K, I = self.W_down.shape
        act_stats_scales(X, self.counter, p.alpha, p.lam, p.p, self.sums,
                         self.s, self.inv_s)
        quantize_rtn_grouped(self.W_up.view(E * 2 * I, K), self.s, p.bits,
                             p.group, *self.up)
        ids, weights = self.route(X)
        # the experts' tokens: one read of the choices by the host
        order = torch.argsort(ids.view(-1), stable=True)
        counts = torch.bincount(ids.view(-1).long(), minlength=E).tolist()
        Y = torch.zeros(X.shape, dtype=torch.float32, device=X.device)
        self.s_mid.fill_(1.0)
        self.inv_s_mid.fill_(1.0)
        f = torch.nn.functional
        at = 0
        for e, n in enumerate(counts):
            slots = order[at:at + n]
            at += n
            down = tuple(b[e * K:(e + 1) * K] for b in self.down)
            h = None
            if n:
                t = slots // self.top_k
                up = tuple(b[e * 2 * I:(e + 1) * 2 * I] for b in self.up)
                gu = w_lowbit_gemm(X[t], self.inv_s, *up, 2 * I, p.bits,
                                   p.group, out_dtype=torch.float32)
                g = f.silu(gu[:, :I]) if self.act == "silu" else \
                    f.gelu(gu[:, :I], approximate="tanh")
                h = (g * gu[:, I:]).to(X.dtype)
                act_stats_scales(h, self.counter, p.alpha, p.lam, p.p,
                                 self.sums_mid, self.s_mid[e],
                                 self.inv_s_mid[e])
            quantize_rtn_grouped(self.W_down[e], self.s_mid[e], p.bits,
                                 p.group, *down)
            if n:
                y = w_lowbit_gemm(h, self.inv_s_mid[e], *down, K, p.bits,
                                  p.group, out_dtype=torch.float32)
                Y.index_add_(0, t, y * weights.view(-1)[slots][:, None])
        return Y.to(X.dtype)

    def decode(self, X: torch.Tensor,
               out: torch.Tensor | None = None) -> torch.Tensor:
        """Up to 64 tokens on the experts the last prompt quantized."""
        T, K = X.shape
        ids, weights = self.route(X)
        need = moe_lowbit_workspace_size(T, K, self.inv_s_mid.shape[1],
                                         self.top_k)
        if self._ws is None or self._ws.numel() < need:
            self._ws = torch.empty(max(need, 16), dtype=torch.uint8,
                                   device=X.device)
        return moe_lowbit(X, ids, weights, self.inv_s, self.up,
                          self.inv_s_mid, self.down, self.prm.bits,
                          self.prm.group, act=self.act, out=out,
                          workspace=self._ws)

    def __call__(self, X: torch.Tensor) -> torch.Tensor:
        return self.prompt(X)
