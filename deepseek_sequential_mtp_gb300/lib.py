"""Thin ctypes binding of libmtp (include/mtp.h).

Argument marshalling only: every step of the hot path runs in the library's
CUDA kernels.  PyTorch supplies device memory and the current stream.  The
binding raises if the library is missing or a call returns an error; there
is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmtp.so")

MTP_F32, MTP_BF16 = 0, 1
DEN = {"fixed": 0, "masked_mean": 1, "sum": 2, "global": 3, "weighted_pair": 4}
LOGITS_STATUS = {0: "ok", 1: "empty", 2: "invalid_logits", 3: "invalid_param"}
VERIFY_STATUS = {0: "ok", 1: "invalid_draft", 2: "zero_residual", 3: "invalid_probs",
                 4: "invalid_budget"}


class MtpError(RuntimeError):
    pass


class Dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("d", ctypes.c_int),
                ("n_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("ffn", ctypes.c_int),
                ("V", ctypes.c_int), ("D", ctypes.c_int), ("eps", ctypes.c_float),
                ("rope_base", ctypes.c_float), ("dtype", ctypes.c_int)]


_PP = ctypes.POINTER(ctypes.c_void_p)
_WEIGHT_LISTS = ("hnorm", "enorm", "eh_proj", "attn_norm", "wq", "wk", "wv", "wo",
                 "ffn_norm", "w_gate", "w_up", "w_down")


class Weights(ctypes.Structure):
    _fields_ = [("embed", ctypes.c_void_p), ("head", ctypes.c_void_p),
                ("out_norm", ctypes.c_void_p)] + [(k, _PP) for k in _WEIGHT_LISTS]


class Grads(ctypes.Structure):
    _fields_ = [("embed", ctypes.c_void_p), ("head", ctypes.c_void_p), ("out_norm", ctypes.c_void_p),
                ("h0", ctypes.c_void_p)] + [(k, _PP) for k in _WEIGHT_LISTS]


FP8_LINEAR_MAPS = ("eh_proj", "wq", "wk", "wv", "wo", "w_gate", "w_up", "w_down")


class Fp8Matrix(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


class BlockFp8(ctypes.Structure):
    _fields_ = [(k, Fp8Matrix) for k in FP8_LINEAR_MAPS]


class Int4Matrix(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("zero", ctypes.c_void_p)]


class BlockInt4(ctypes.Structure):
    _fields_ = [(k, Int4Matrix) for k in FP8_LINEAR_MAPS] + [("group", ctypes.c_int)]


class DraftExt(ctypes.Structure):
    _fields_ = [("fp8", ctypes.POINTER(BlockFp8)), ("int4", ctypes.POINTER(BlockInt4)),
                ("prefix_k", ctypes.c_void_p), ("prefix_v", ctypes.c_void_p), ("prefix_len", ctypes.c_int)]


class PrefixDims(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int) for k in ("R", "L", "n_heads", "n_kv_heads", "head_dim", "P", "T", "causal")] + \
               [("scale", ctypes.c_float)] + \
               [(k, ctypes.c_longlong) for k in ("q_stride_r", "q_stride_t", "q_stride_h", "prefix_stride_t",
                                                 "prefix_stride_h", "kv_stride_r", "kv_stride_t", "kv_stride_h")]


class LogitsParams(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("temperature", "repetition", "frequency", "presence", "hist",
                                               "hist_len", "prompt_len", "draft", "bias_ids", "bias", "mask")] + \
               [("hist_cap", ctypes.c_int), ("n_bias", ctypes.c_int)]


_lib = None


def load() -> ctypes.CDLL:
    """Load libmtp.so (built by ``__graft_entry__.build()``); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise MtpError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, u64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint64, ctypes.c_size_t
    lib.mtp_status_string.restype = ctypes.c_char_p
    lib.mtp_status_string.argtypes = [i32]
    lib.mtp_abi_version.restype = i32
    lib.mtp_check_errors.restype = i32
    lib.mtp_check_errors.argtypes = [vp, ctypes.POINTER(ctypes.c_uint)]
    lib.spec_verify.restype = i32
    lib.spec_verify.argtypes = [i32, i32, i32, vp, vp, vp, u64, u64, vp, vp, vp, vp, vp, vp, vp]
    lib.mtp_gemm_bf16.restype = i32
    lib.mtp_gemm_bf16.argtypes = [i32, i32, i32, vp, vp, vp, vp]
    lib.mtp_chain_workspace_bytes.restype = sz
    lib.mtp_chain_workspace_bytes.argtypes = [ctypes.POINTER(Dims)]
    lib.mtp_chain_forward.restype = i32
    lib.mtp_chain_forward.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(Weights),
                                      vp, vp, vp, vp, vp, vp, sz, vp]
    lib.mtp_chain_loss.restype = i32
    lib.mtp_chain_loss.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(Weights),
                                   vp, vp, vp, vp, ctypes.c_float, i32, i32,
                                   vp, vp, vp, vp, vp, sz, vp]
    lib.mtp_loss_assemble_weighted.restype = i32
    lib.mtp_loss_assemble_weighted.argtypes = [i32, vp, ctypes.c_double, ctypes.POINTER(ctypes.c_float),
                                               ctypes.c_float, i32, i32, vp, vp]
    lib.mtp_loss_assemble.restype = i32
    lib.mtp_loss_assemble.argtypes = [i32, vp, ctypes.c_double, ctypes.c_float, i32, i32, vp, vp]
    lib.mtp_profile_kernel.restype = i32
    lib.mtp_profile_kernel.argtypes = [i32, vp, i32, ctypes.POINTER(ctypes.c_int)]
    lib.mtp_draft_workspace_bytes.restype = sz
    lib.mtp_draft_workspace_bytes.argtypes = [ctypes.POINTER(Dims)]
    lib.mtp_draft_round_workspace_bytes.restype = sz
    lib.mtp_draft_round_workspace_bytes.argtypes = [ctypes.POINTER(Dims), i32]
    lib.mtp_draft_round.restype = i32
    lib.mtp_draft_round.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(Weights), vp, vp, vp, vp, vp, vp, i32,
                                    ctypes.c_uint64, ctypes.c_uint64, vp, vp, vp, vp, sz, vp]
    lib.mtp_draft_step.restype = i32
    lib.mtp_draft_step.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(Weights), vp, vp, vp, vp, vp, vp,
                                   u64, u64, vp, vp, vp, vp, sz, vp]
    lib.mtp_draft_round_fp8.restype = i32
    lib.mtp_draft_round_fp8.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(Weights), ctypes.POINTER(BlockFp8),
                                        vp, vp, vp, vp, vp, vp, i32, ctypes.c_uint64, ctypes.c_uint64, vp, vp, vp,
                                        vp, sz, vp]
    lib.mtp_draft_round_ext_workspace_bytes.restype = sz
    lib.mtp_draft_round_ext_workspace_bytes.argtypes = [ctypes.POINTER(Dims), i32, i32]
    lib.mtp_draft_round_ext.restype = i32
    lib.mtp_draft_round_ext.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(Weights), ctypes.POINTER(DraftExt),
                                        vp, vp, vp, vp, vp, vp, i32, ctypes.c_uint64, ctypes.c_uint64, vp, vp, vp,
                                        vp, sz, vp]
    lib.mtp_gemm_decode_bf16.restype = i32
    lib.mtp_gemm_decode_bf16.argtypes = [i32, i32, i32, vp, vp, vp, vp]
    lib.mtp_gemm_f32acc.restype = i32
    lib.mtp_gemm_f32acc.argtypes = [i32, i32, i32, vp, i32, i32, vp, i32, i32, vp, i32, i32, vp]
    lib.mtp_gemm_fp8w_workspace_bytes.restype = sz
    lib.mtp_gemm_fp8w_workspace_bytes.argtypes = [i32]
    lib.mtp_gemm_fp8w.restype = i32
    lib.mtp_gemm_fp8w.argtypes = [i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
    lib.mtp_chain_grad_workspace_bytes.restype = sz
    lib.mtp_chain_grad_workspace_bytes.argtypes = [ctypes.POINTER(Dims)]
    lib.mtp_chain_loss_grad.restype = i32
    lib.mtp_chain_loss_grad.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(Weights), vp, vp, vp, vp,
                                        ctypes.c_float, i32, i32, ctypes.POINTER(ctypes.c_float), vp, vp,
                                        ctypes.POINTER(Grads), vp, sz, vp]
    lib.mtp_diag_verify_starved.restype = i32
    lib.mtp_diag_verify_starved.argtypes = [i32, i32, i32, vp, vp, vp, u64, u64, vp, vp, vp, vp,
                                            ctypes.c_longlong, vp]
    lib.mtp_gemm_int4w.restype = i32
    lib.mtp_gemm_int4w.argtypes = [i32, i32, i32, i32, vp, ctypes.POINTER(Int4Matrix), vp, i32, vp]
    lib.mtp_prefix_attention_workspace_bytes.restype = sz
    lib.mtp_prefix_attention_workspace_bytes.argtypes = [ctypes.POINTER(PrefixDims)]
    lib.mtp_prefix_attention.restype = i32
    lib.mtp_prefix_attention.argtypes = [ctypes.POINTER(PrefixDims)] + [vp] * 9 + [sz, vp]
    lib.mtp_logits_probs.restype = i32
    lib.mtp_logits_probs.argtypes = [i32, i32, i32, i32, vp, ctypes.c_longlong, ctypes.POINTER(LogitsParams), vp, vp,
                                     vp]
    lib.mtp_kernel_launches.restype = ctypes.c_ulonglong
    lib.mtp_kernel_launches.argtypes = []
    _lib = lib
    return lib


def _check(status: int, what: str):
    if status != 0:
        msg = load().mtp_status_string(status).decode()
        raise MtpError(f"{what}: {msg} (status {status})")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# the current stream's handle without the object around it (3 us of a small call), and the
# current device's number without the check for a first use, where torch has them
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream=None):
    if stream is None and _raw_stream is not None:
        return _raw_stream(_current_device())
    return (stream if stream is not None else torch.cuda.current_stream()).cuda_stream


def _need(t: torch.Tensor, name: str, dtype: torch.dtype):
    if not t.is_cuda:
        raise MtpError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise MtpError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise MtpError(f"{name} must be contiguous")


def _arg(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, shape, device):
    """Address of an optional dense argument of the given type, shape and device (None = null)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        _need(t, name, dtype)
        if tuple(t.shape) != tuple(shape):
            raise MtpError(f"{name} must be {list(shape)}, got {list(t.shape)}")
        raise MtpError(f"{name} is on {t.device}, not on {device}")
    return t.data_ptr()


def _launch_device(t: torch.Tensor, stream):
    """The device of a call's tensors; it has to be the current one, and the stream's."""
    dev = t.device
    if dev.type != "cuda" or dev.index != _current_device() or (
            stream is not None and stream.device != dev):
        raise MtpError(f"the tensors are on {dev}: make it the current device and use a stream of it")
    return dev


def _empty(shape, dtype, device, stream):
    """An output or workspace whose memory belongs to the launching stream."""
    if stream is None or stream == torch.cuda.current_stream():
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def check_errors(stream=None) -> int:
    """Synchronise and return the device error bits (raises if any is set)."""
    flags = ctypes.c_uint(0)
    st = load().mtp_check_errors(_stream(stream), ctypes.byref(flags))
    if st != 0:
        raise MtpError(f"device error word 0x{flags.value:x} ({load().mtp_status_string(st).decode()})")
    return flags.value


# --------------------------------------------------------------------------
# spec_verify
# --------------------------------------------------------------------------
def spec_verify(p: torch.Tensor, q: torch.Tensor, draft: torch.Tensor, seed: int, offset: int,
                eos: Optional[torch.Tensor] = None, remaining: Optional[torch.Tensor] = None,
                out: Optional[dict] = None, stream=None) -> dict:
    """Exact speculative verification (include/mtp.h: spec_verify)."""
    R, gamma = draft.shape
    V = p.shape[-1]
    _need(p, "p", torch.float32)
    _need(q, "q", torch.float32)
    _need(draft, "draft", torch.int32)
    if p.shape != (R, gamma + 1, V) or q.shape != (R, gamma, V):
        raise MtpError("p must be [R, gamma+1, V] and q [R, gamma, V]")
    for name, t in (("eos", eos), ("remaining", remaining)):
        if t is not None:
            _need(t, name, torch.int32)
    if out is None:
        out = {k: torch.empty(R, dtype=torch.int32, device=p.device)
               for k in ("accepted", "next_token", "n_emit", "status")}
    st = load().spec_verify(R, gamma, V, _ptr(p), _ptr(q), _ptr(draft),
                            int(seed) & (2**64 - 1), int(offset) & (2**64 - 1),
                            _ptr(eos), _ptr(remaining), _ptr(out["accepted"]),
                            _ptr(out["next_token"]), _ptr(out["n_emit"]), _ptr(out["status"]),
                            _stream(stream))
    _check(st, "spec_verify")
    return out


def verify_starved(p: torch.Tensor, q: torch.Tensor, draft: torch.Tensor, seed: int, offset: int,
                   wait_limit_cycles: int, stream=None) -> dict:
    """spec_verify with a producer that issues no copy, so every row sweep's
    bounded wait runs out (include/mtp.h: mtp_diag_verify_starved)."""
    R, gamma = draft.shape
    V = p.shape[-1]
    _need(p, "p", torch.float32)
    _need(q, "q", torch.float32)
    _need(draft, "draft", torch.int32)
    out = {k: torch.empty(R, dtype=torch.int32, device=p.device)
           for k in ("accepted", "next_token", "n_emit", "status")}
    st = load().mtp_diag_verify_starved(R, gamma, V, _ptr(p), _ptr(q), _ptr(draft),
                                        int(seed) & (2**64 - 1), int(offset) & (2**64 - 1),
                                        _ptr(out["accepted"]), _ptr(out["next_token"]), _ptr(out["n_emit"]),
                                        _ptr(out["status"]), int(wait_limit_cycles), _stream(stream))
    _check(st, "mtp_diag_verify_starved")
    return out


# --------------------------------------------------------------------------
# Logits to probability rows
# --------------------------------------------------------------------------
def logits_probs(logits: torch.Tensor, temperature=None, hist=None, hist_len=None, prompt_len=None, draft=None,
                 repetition=None, frequency=None, presence=None, bias_ids=None, bias=None, mask=None,
                 out: Optional[dict] = None, stream=None) -> dict:
    """Probability rows from logits [R, L, V] (f32 or bf16; rows may be a fixed
    distance apart) under each request's penalties, biases, grammar mask and
    temperature (include/mtp.h: mtp_logits_probs).  Returns {"p": [R, L, V]
    float32, "status": [R, L] int32}; ``out`` may supply them, and out["p"] may
    be the float32 logits themselves."""
    if logits.dim() != 3:
        raise MtpError("logits must be [R, L, V]")
    R, L, V = logits.shape
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise MtpError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    dev = _launch_device(logits, stream)
    sr, sl, sv = logits.stride()
    ld = sl if L > 1 else sr if R > 1 else V
    if R * L > 0 and ((V > 1 and sv != 1) or (R > 1 and L > 1 and sr != L * ld) or ld < V):
        raise MtpError("logits must have dense rows a fixed distance apart")
    prm = LogitsParams()
    f32, i32 = torch.float32, torch.int32
    prm.temperature = _arg(temperature, "temperature", f32, (R,), dev)
    prm.repetition = _arg(repetition, "repetition", f32, (R,), dev)
    prm.frequency = _arg(frequency, "frequency", f32, (R,), dev)
    prm.presence = _arg(presence, "presence", f32, (R,), dev)
    if hist is not None:
        if hist.dim() != 2:
            raise MtpError("hist must be [R, capacity]")
        prm.hist_cap = hist.shape[1]
        prm.hist = _arg(hist, "hist", i32, (R, prm.hist_cap), dev)
        prm.hist_len = _arg(hist_len, "hist_len", i32, (R,), dev)
        prm.prompt_len = _arg(prompt_len, "prompt_len", i32, (R,), dev)
    elif hist_len is not None or prompt_len is not None:
        raise MtpError("hist_len and prompt_len need hist")
    if draft is not None:
        prm.draft = _arg(draft, "draft", i32, (R, L - 1), dev)
    if (bias_ids is None) != (bias is None):
        raise MtpError("bias_ids and bias come together")
    if bias_ids is not None:
        if bias_ids.dim() != 2:
            raise MtpError("bias_ids must be [R, n]")
        prm.n_bias = bias_ids.shape[1]
        prm.bias_ids = _arg(bias_ids, "bias_ids", i32, (R, prm.n_bias), dev)
        prm.bias = _arg(bias, "bias", f32, (R, prm.n_bias), dev)
    prm.mask = _arg(mask, "mask", i32, (R, L, (V + 31) // 32), dev)
    if out is None:
        out = {"p": _empty((R, L, V), f32, dev, stream), "status": _empty((R, L), i32, dev, stream)}
    else:
        _arg(out["p"], "out['p']", f32, (R, L, V), dev)
        _arg(out["status"], "out['status']", i32, (R, L), dev)
    st = load().mtp_logits_probs(R, L, V, MTP_F32 if logits.dtype == f32 else MTP_BF16, logits.data_ptr(), ld,
                                 ctypes.byref(prm), out["p"].data_ptr(), out["status"].data_ptr(), _stream(stream))
    _check(st, "mtp_logits_probs")
    return out


# --------------------------------------------------------------------------
# GEMM diagnostic
# --------------------------------------------------------------------------
def gemm_bf16(A: torch.Tensor, B: torch.Tensor, C: Optional[torch.Tensor] = None, stream=None):
    """C = A · B^T on the library's tcgen05 GEMM core (bf16 in/out, fp32 accumulate)."""
    _need(A, "A", torch.bfloat16)
    _need(B, "B", torch.bfloat16)
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K:
        raise MtpError("A and B must share K")
    if C is None:
        C = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _check(load().mtp_gemm_bf16(M, N, K, _ptr(A), _ptr(B), _ptr(C), _stream(stream)), "mtp_gemm_bf16")
    return C


# --------------------------------------------------------------------------
# Chain
# --------------------------------------------------------------------------
def make_dims(cfg) -> Dims:
    return Dims(cfg.B, cfg.T, cfg.d, cfg.n_heads, cfg.head_dim, cfg.ffn, cfg.V, cfg.D,
                cfg.eps, cfg.rope_base, MTP_BF16 if cfg.dtype == "bf16" else MTP_F32)


class ChainWeights:
    """Holds the ctypes views of a weight dict (see synth.make_weights); the lists
    named in ``without`` are not read and may be missing."""

    def __init__(self, weights: dict, D: int, without=()):
        self._keep = []
        self.struct = Weights()
        self.struct.embed = weights["embed"].data_ptr()
        self.struct.head = weights["head"].data_ptr()
        self.struct.out_norm = weights["out_norm"].data_ptr()
        for k in _WEIGHT_LISTS:
            if k in without:
                continue
            lst = weights[k]
            if len(lst) != D:
                raise MtpError(f"weights[{k!r}] must have D={D} entries")
            arr = (ctypes.c_void_p * D)(*[t.data_ptr() for t in lst])
            self._keep.append(arr)
            setattr(self.struct, k, ctypes.cast(arr, _PP))


class Fp8Block:
    """ctypes view of the FP8 linear maps of one module: fp8[name] = (q, scale)
    with q uint8 [n, K] e4m3 codes and scale float32 [ceil(n/128), ceil(K/128)]."""

    def __init__(self, fp8: dict):
        self.fp8 = fp8
        self.struct = BlockFp8()
        for name in FP8_LINEAR_MAPS:
            q, sc = fp8[name]
            _need(q, name + ".q", torch.uint8)
            _need(sc, name + ".scale", torch.float32)
            nb, kb = -(-q.shape[0] // 128), -(-q.shape[1] // 128)
            if tuple(sc.shape) != (nb, kb):
                raise MtpError(f"{name}.scale must be [{nb}, {kb}]")
            m = getattr(self.struct, name)
            m.q = q.data_ptr()
            m.scale = sc.data_ptr()


class Int4Block:
    """ctypes view of the 4-bit linear maps of one module: int4[name] = (q, scale,
    zero or None) as _int4_matrix takes them, all on one GPU."""

    def __init__(self, int4: dict, group: int, cfg):
        d, f = cfg.d, cfg.ffn
        device = int4[FP8_LINEAR_MAPS[0]][0].device
        if device.type != "cuda":
            raise MtpError("4-bit weights must be CUDA tensors")
        self.int4 = int4
        self.struct = BlockInt4()
        self.struct.group = int(group)
        shapes = {"eh_proj": (d, 2 * d), "w_gate": (f, d), "w_up": (f, d), "w_down": (d, f)}
        for name in FP8_LINEAR_MAPS:
            q, sc, z = int4[name]
            n, k = shapes.get(name, (d, d))
            if tuple(q.shape) != (n, k // 2):
                raise MtpError(f"{name}.q must be [{n}, {k // 2}]")
            setattr(self.struct, name, _int4_matrix(name, q, sc, z, int(group), device))


def gemm_decode_bf16(x: torch.Tensor, w: torch.Tensor, out: torch.Tensor, stream=None):
    """out[R, N] += x[R, K] @ w[N, K]^T for R <= 32 tokens (mtp_gemm_decode_bf16)."""
    _need(x, "x", torch.bfloat16)
    _need(w, "w", torch.bfloat16)
    _need(out, "out", torch.float32)
    R, K = x.shape
    N = w.shape[0]
    if w.shape[1] != K or tuple(out.shape) != (R, N):
        raise MtpError("gemm_decode_bf16: x [R, K], w [N, K], out [R, N]")
    _check(load().mtp_gemm_decode_bf16(R, N, K, _ptr(x), _ptr(w), _ptr(out), _stream(stream)), "mtp_gemm_decode_bf16")
    return out


def gemm_f32acc(A: torch.Tensor, B: torch.Tensor, out: torch.Tensor, a_mn=False, b_mn=False, splits=1, stream=None):
    """out += A' B'^T (mtp_gemm_f32acc): A' = A ([M, K]) or, with a_mn, A^T of a
    [K, M] tensor; B' = B ([N, K]) or, with b_mn, B^T of a [K, N] tensor."""
    _need(A, "A", torch.bfloat16)
    _need(B, "B", torch.bfloat16)
    _need(out, "out", torch.float32)
    M = A.shape[1] if a_mn else A.shape[0]
    K = A.shape[0] if a_mn else A.shape[1]
    N = B.shape[1] if b_mn else B.shape[0]
    if (B.shape[0] if b_mn else B.shape[1]) != K or tuple(out.shape) != (M, N):
        raise MtpError("gemm_f32acc: inconsistent shapes")
    _check(load().mtp_gemm_f32acc(M, N, K, _ptr(A), A.shape[1], int(a_mn), _ptr(B), B.shape[1], int(b_mn), _ptr(out),
                                  out.shape[1], int(splits), _stream(stream)), "mtp_gemm_f32acc")
    return out


def gemm_fp8w(x: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, out: torch.Tensor, stream=None, ws=None):
    """out[R, N] += x~[R, K] @ W^T, W = e4m3(q) * block scales, x~ the two-term
    e4m3 form of x (mtp_gemm_fp8w)."""
    _need(x, "x", torch.bfloat16)
    _need(q, "q", torch.uint8)
    _need(scale, "scale", torch.float32)
    _need(out, "out", torch.float32)
    R, K = x.shape
    N = q.shape[0]
    if q.shape[1] != K or tuple(out.shape) != (R, N):
        raise MtpError("gemm_fp8w: x [R, K], q [N, K], out [R, N]")
    if ws is None:
        ws = torch.empty(max(16, int(load().mtp_gemm_fp8w_workspace_bytes(K))), dtype=torch.uint8, device=x.device)
    _check(load().mtp_gemm_fp8w(R, N, K, _ptr(x), _ptr(q), _ptr(scale), _ptr(out), _ptr(ws), ws.numel(),
                                _stream(stream)), "mtp_gemm_fp8w")
    return out


def _int4_matrix(name: str, q, scale, zero, group: int, device) -> Int4Matrix:
    """ctypes view of one 4-bit matrix: q uint8 [N, K/2], scale bf16 and zero
    uint8 (or None) [N, ceil(K/group)]."""
    if q.dim() != 2 or group < 1:
        raise MtpError(f"{name}.q must be [N, K/2] and the group positive")
    shape = (q.shape[0], (2 * q.shape[1] + group - 1) // group)
    m = Int4Matrix()
    m.q = _arg(q, name + ".q", torch.uint8, q.shape, device)
    m.scale = _arg(scale, name + ".scale", torch.bfloat16, shape, device)
    m.zero = _arg(zero, name + ".zero", torch.uint8, shape, device)
    return m


def gemm_int4w(x: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, zero: Optional[torch.Tensor] = None,
               group: int = 128, out: Optional[torch.Tensor] = None, accumulate: bool = False, stream=None):
    """out[R, N] = x[R, K] @ W^T (added to ``out`` if ``accumulate``) with W =
    (code - zero) * scale in groups of ``group`` along K, two codes per byte of
    q [N, K/2] (include/mtp.h: mtp_gemm_int4w)."""
    dev = _launch_device(x, stream)
    m = _int4_matrix("w", q, scale, zero, group, dev)
    _need(x, "x", torch.bfloat16)
    N = q.shape[0]
    if x.dim() != 2 or x.shape[1] != 2 * q.shape[1]:
        raise MtpError("gemm_int4w: x [R, K], q [N, K/2]")
    R, K = x.shape
    if out is None:
        if accumulate:
            raise MtpError("gemm_int4w: accumulate needs out")
        out = _empty((R, N), torch.float32, dev, stream)
    else:
        _arg(out, "out", torch.float32, (R, N), dev)
    _check(load().mtp_gemm_int4w(R, N, K, group, x.data_ptr(), ctypes.byref(m), out.data_ptr(), int(accumulate),
                                 _stream(stream)), "mtp_gemm_int4w")
    return out


def _check_chain_inputs(cfg, tokens, seg, pos, h0, weights):
    dt = torch.bfloat16 if cfg.dtype == "bf16" else torch.float32
    for name, t in (("tokens", tokens), ("seg", seg), ("pos", pos)):
        _need(t, name, torch.int32)
        if tuple(t.shape) != (cfg.B, cfg.T):
            raise MtpError(f"{name} must be [B, T]")
    _need(h0, "h0", dt)
    for k, v in weights.items():
        for t in (v if isinstance(v, (list, tuple)) else [v]):
            _need(t, k, dt)
    return dt


def chain_workspace_bytes(cfg) -> int:
    dims = make_dims(cfg)
    return int(load().mtp_chain_workspace_bytes(ctypes.byref(dims)))


class Chain:
    """Reusable call state (dims, weight views, workspace) for one shape."""

    def __init__(self, cfg, weights: dict, device="cuda"):
        self.cfg = cfg
        self.dims = make_dims(cfg)
        self.w = ChainWeights(weights, cfg.D)
        self.weights = weights
        nbytes = chain_workspace_bytes(cfg)
        if nbytes == 0:
            raise MtpError("invalid chain dimensions")
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=device)

    def loss_grad(self, tokens, seg, pos, h0, grads: dict, lam=None, den="fixed", with_main=True,
                  depth_weights=None, out=None, stream=None):
        """Training step (include/mtp.h: mtp_chain_loss_grad): losses as
        ``loss`` and the gradients added into ``grads`` (fp32 tensors keyed as
        the weights, plus "h0"; per-depth entries are lists; missing keys are
        not computed)."""
        cfg = self.cfg
        _check_chain_inputs(cfg, tokens, seg, pos, h0, self.weights)
        if not hasattr(self, "gws"):
            nbytes = int(load().mtp_chain_grad_workspace_bytes(ctypes.byref(self.dims)))
            if nbytes == 0:
                raise MtpError("the training step does not support these dimensions")
            self.gws = torch.empty(nbytes, dtype=torch.uint8, device=h0.device)
        dev = h0.device
        if out is None:
            out = {"sums_counts": torch.empty(2 * (cfg.D + 1), dtype=torch.float64, device=dev),
                   "losses": torch.empty(cfg.D + 2, dtype=torch.float32, device=dev)}
        g = Grads()
        keep = []
        for k in ("embed", "head", "out_norm", "h0"):
            t = grads.get(k)
            if t is not None:
                _need(t, f"grads[{k!r}]", torch.float32)
                setattr(g, k, t.data_ptr())
        for k in _WEIGHT_LISTS:
            lst = grads.get(k)
            if lst is not None:
                arr = (ctypes.c_void_p * cfg.D)(*[t.data_ptr() for t in lst])
                keep.append(arr)
                setattr(g, k, ctypes.cast(arr, _PP))
        w = None
        if depth_weights is not None:
            w = (ctypes.c_float * cfg.D)(*[float(x) for x in depth_weights])
        st = load().mtp_chain_loss_grad(ctypes.byref(self.dims), ctypes.byref(self.w.struct),
                                        _ptr(tokens), _ptr(seg), _ptr(pos), _ptr(h0),
                                        float(cfg.lam if lam is None else lam), DEN[den], int(with_main), w,
                                        _ptr(out["sums_counts"]), _ptr(out["losses"]), ctypes.byref(g),
                                        _ptr(self.gws), self.gws.numel(), _stream(stream))
        _check(st, "mtp_chain_loss_grad")
        return out

    def forward(self, tokens, seg, pos, h0, h_out=None, stream=None):
        cfg = self.cfg
        dt = _check_chain_inputs(cfg, tokens, seg, pos, h0, self.weights)
        if h_out is None:
            h_out = torch.empty((cfg.D, cfg.B, cfg.T, cfg.d), dtype=dt, device=h0.device)
        st = load().mtp_chain_forward(ctypes.byref(self.dims), ctypes.byref(self.w.struct),
                                      _ptr(tokens), _ptr(seg), _ptr(pos), _ptr(h0), _ptr(h_out),
                                      _ptr(self.ws), self.ws.numel(), _stream(stream))
        _check(st, "mtp_chain_forward")
        return h_out

    def loss(self, tokens, seg, pos, h0, lam=None, den="fixed", with_main=True,
             row_loss=False, h_out=None, out=None, stream=None):
        cfg = self.cfg
        _check_chain_inputs(cfg, tokens, seg, pos, h0, self.weights)
        dev = h0.device
        if out is None:
            out = {"sums_counts": torch.empty(2 * (cfg.D + 1), dtype=torch.float64, device=dev),
                   "losses": torch.empty(cfg.D + 2, dtype=torch.float32, device=dev)}
            if row_loss:
                out["row_loss"] = torch.empty((cfg.D + 1, cfg.B, cfg.T), dtype=torch.float32, device=dev)
        st = load().mtp_chain_loss(ctypes.byref(self.dims), ctypes.byref(self.w.struct),
                                   _ptr(tokens), _ptr(seg), _ptr(pos), _ptr(h0),
                                   float(cfg.lam if lam is None else lam), DEN[den], int(with_main),
                                   _ptr(out["sums_counts"]), _ptr(out["losses"]),
                                   _ptr(out.get("row_loss")), _ptr(h_out),
                                   _ptr(self.ws), self.ws.numel(), _stream(stream))
        _check(st, "mtp_chain_loss")
        if h_out is not None:
            out["h"] = h_out
        return out


# --------------------------------------------------------------------------
# Loss assembly (data-parallel callers) and measurement hooks
# --------------------------------------------------------------------------
def loss_assemble(sums_counts: torch.Tensor, D: int, n_positions: float, lam: float, den="fixed",
                  with_main=True, losses: Optional[torch.Tensor] = None, stream=None,
                  depth_weights=None) -> torch.Tensor:
    """L, L_main, L^(1..D) from (already all-reduced) per-term sums and counts
    under reduction ``den`` (include/mtp.h: mtp_den) with per-depth weights
    (a sequence of D floats; None = lam / D each)."""
    _need(sums_counts, "sums_counts", torch.float64)
    if losses is None:
        losses = torch.empty(D + 2, dtype=torch.float32, device=sums_counts.device)
    w = None
    if depth_weights is not None:
        if len(depth_weights) != D:
            raise MtpError("depth_weights must hold D values")
        w = (ctypes.c_float * D)(*[float(x) for x in depth_weights])
    _check(load().mtp_loss_assemble_weighted(D, _ptr(sums_counts), float(n_positions), w, float(lam), DEN[den],
                                             int(with_main), _ptr(losses), _stream(stream)),
           "mtp_loss_assemble_weighted")
    return losses


KERNEL_CLASSES = {"head_ce_gemm": 0, "gate_up_gemm": 1, "down_gemm": 2, "qkv_gemm": 3, "o_gemm": 4,
                  "proj_gemm": 5, "attention": 6, "spec_verify": 7, "prologue": 8}


class KernelTimer:
    """Arms the library's event hook for one kernel class: CUDA events are
    recorded on the launching stream around each launch of that class."""

    def __init__(self, kernel_class: str, max_launches: int):
        self.cls = KERNEL_CLASSES[kernel_class]
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(2 * max_launches)]
        for e in self.events:  # CUDA creates the events on first record
            e.record()
        self._handles = (ctypes.c_void_p * (2 * max_launches))(*[e.cuda_event for e in self.events])
        self.recorded = ctypes.c_int(0)
        self.max = max_launches

    def arm(self):
        _check(load().mtp_profile_kernel(self.cls, self._handles, self.max, ctypes.byref(self.recorded)),
               "mtp_profile_kernel")

    @staticmethod
    def disarm_all():
        for c in KERNEL_CLASSES.values():
            load().mtp_profile_kernel(c, None, 0, None)

    def durations_ms(self):
        n = self.recorded.value
        return [self.events[2 * i].elapsed_time(self.events[2 * i + 1]) for i in range(n)]


def kernel_launches() -> int:
    return int(load().mtp_kernel_launches())


# --------------------------------------------------------------------------
# Draft step (decode-shaped MTP proposal)
# --------------------------------------------------------------------------
class _Draft:
    """Call state of a draft round of ``gamma`` steps for one shape: dims, weight
    views, workspace.  ``rows`` is the outputs' leading shape."""

    def __init__(self, cfg, weights: dict, gamma: int, rows: tuple, device, fp8, int4, int4_group, prefix_len):
        self.cfg = cfg
        self.gamma = int(gamma)
        self.rows = rows
        self.prefix_len = int(prefix_len)
        self.dims = Dims(cfg.R, cfg.ctx, cfg.d, cfg.n_heads, cfg.head_dim, cfg.ffn, cfg.V, 1, cfg.eps,
                         cfg.rope_base, MTP_BF16)
        if fp8 is not None and int4 is not None:
            raise MtpError("a module has its linear maps in FP8 or in 4 bits, not both")
        # maps in another form replace the weight dict's, which are neither read nor kept
        without = FP8_LINEAR_MAPS if fp8 is not None or int4 is not None else ()
        self.weights = {k: v for k, v in weights.items() if k not in without}
        d, f = cfg.d, cfg.ffn
        shapes = {"embed": (cfg.V, d), "head": (cfg.V, d), "out_norm": (d,), "hnorm": (d,), "enorm": (d,),
                  "attn_norm": (d,), "ffn_norm": (d,), "eh_proj": (d, 2 * d), "wq": (d, d), "wk": (d, d),
                  "wv": (d, d), "wo": (d, d), "w_gate": (f, d), "w_up": (f, d), "w_down": (d, f)}
        for name, shape in shapes.items():
            t = self.weights.get(name, ())
            for m in t if isinstance(t, (list, tuple)) else (t,):
                _arg(m, f"weights[{name!r}]", torch.bfloat16, shape, self.weights["embed"].device)
        self.w = ChainWeights(self.weights, 1, without)
        self.f8 = Fp8Block(fp8) if fp8 is not None else None
        self.i4 = Int4Block(int4, int4_group, cfg) if int4 is not None else None
        nbytes = int(load().mtp_draft_round_ext_workspace_bytes(ctypes.byref(self.dims), self.gamma, self.prefix_len))
        if nbytes == 0:
            raise MtpError("invalid draft-step dimensions or gamma")
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        blocks = [b[FP8_LINEAR_MAPS[0]][0] for b in (fp8, int4) if b is not None]
        if any(t.device != self.ws.device for t in (self.weights["embed"], *blocks)):
            raise MtpError(f"the weights and the draft step ({self.ws.device}) must be on one device")

    def __call__(self, parent_hidden, frontier, pos, kv_k, kv_v, ctx_len, seed, offset,
                 out=None, h_out=None, stream=None, prefix_k=None, prefix_v=None):
        cfg, g = self.cfg, self.gamma
        dev = _launch_device(parent_hidden, stream)
        if self.ws.device != dev:
            raise MtpError(f"the draft step was built on {self.ws.device}, its inputs are on {dev}")
        bf16, i32, f32 = torch.bfloat16, torch.int32, torch.float32
        rows = [_arg(t, name, dtype, shape, dev) for t, name, dtype, shape in (
            (parent_hidden, "parent_hidden", bf16, (cfg.R, cfg.d)), (frontier, "frontier", i32, (cfg.R,)),
            (pos, "pos", i32, (cfg.R,)), (kv_k, "kv_k", bf16, (cfg.R, cfg.ctx, cfg.d)),
            (kv_v, "kv_v", bf16, (cfg.R, cfg.ctx, cfg.d)), (ctx_len, "ctx_len", i32, (cfg.R,)))]
        h = _arg(h_out, "h_out", bf16, (*self.rows, cfg.d), dev)
        ext = None
        if self.i4 is not None or self.prefix_len > 0:
            ext = DraftExt()
            if self.f8 is not None:
                ext.fp8 = ctypes.pointer(self.f8.struct)
            if self.i4 is not None:
                ext.int4 = ctypes.pointer(self.i4.struct)
            if self.prefix_len > 0:
                for name, t in (("prefix_k", prefix_k), ("prefix_v", prefix_v)):
                    if t is None:
                        raise MtpError(f"{name} is missing")
                    _arg(t, name, bf16, (self.prefix_len, cfg.d), dev)
                ext.prefix_k, ext.prefix_v, ext.prefix_len = prefix_k.data_ptr(), prefix_v.data_ptr(), self.prefix_len
        if self.prefix_len == 0 and (prefix_k is not None or prefix_v is not None):
            raise MtpError("prefix rows were given to a draft step built with prefix_len = 0")
        if out is None:
            out = {"q": _empty((*self.rows, cfg.V), f32, dev, stream), "y": _empty(self.rows, i32, dev, stream)}
        q = _arg(out["q"], "out['q']", f32, (*self.rows, cfg.V), dev)
        y = _arg(out["y"], "out['y']", i32, self.rows, dev)
        if stream is not None:
            self.ws.record_stream(stream)  # allocated on another one
        rest = (int(seed) & (2**64 - 1), int(offset) & (2**64 - 1), q, y, h, self.ws.data_ptr(), self.ws.numel(),
                _stream(stream))
        dims, w = ctypes.byref(self.dims), ctypes.byref(self.w.struct)
        if ext is not None:
            _check(load().mtp_draft_round_ext(dims, w, ctypes.byref(ext), *rows, g, *rest), "mtp_draft_round_ext")
        elif self.f8 is not None:
            _check(load().mtp_draft_round_fp8(dims, w, ctypes.byref(self.f8.struct), *rows, g, *rest),
                   "mtp_draft_round_fp8")
        elif len(self.rows) == 1:
            _check(load().mtp_draft_step(dims, w, *rows, *rest), "mtp_draft_step")
        else:
            _check(load().mtp_draft_round(dims, w, *rows, g, *rest), "mtp_draft_round")
        if h_out is not None:
            out["h"] = h_out
        return out


class DraftStep(_Draft):
    """Reusable call state of mtp_draft_step for one shape (see synth.DraftConfig).
    The module's linear maps may be in FP8 (``fp8``) or in 4 bits (``int4``:
    name -> (q, scale, zero or None), groups of ``int4_group``; ``weights`` need not
    hold the bf16 maps then), and the caches
    may begin with ``prefix_len`` rows that all requests share, passed to each
    call as prefix_k and prefix_v [prefix_len, d] (mtp_draft_round_ext).  A call
    takes parent_hidden [R, d], frontier, pos, ctx_len [R] and kv_k, kv_v [R, ctx, d]
    on the step's device and returns {"q": [R, V] float32, "y": [R] int32} and,
    where h_out [R, d] is given, "h"; ``out`` may supply them.  Calls of one object
    share its workspace and must not overlap."""

    def __init__(self, cfg, weights: dict, device="cuda", fp8: Optional[dict] = None, int4: Optional[dict] = None,
                 int4_group: int = 128, prefix_len: int = 0):
        super().__init__(cfg, weights, 1, (cfg.R,), device, fp8, int4, int4_group, prefix_len)


class DraftRound(_Draft):
    """Reusable call state of mtp_draft_round: gamma recurrent draft steps of
    one module for one shape (see synth.DraftConfig).  As DraftStep, with outputs
    [R, gamma, V], [R, gamma] and h_out [R, gamma, d]."""

    def __init__(self, cfg, weights: dict, gamma: int, device="cuda", fp8: Optional[dict] = None,
                 int4: Optional[dict] = None, int4_group: int = 128, prefix_len: int = 0):
        super().__init__(cfg, weights, gamma, (cfg.R, int(gamma)), device, fp8, int4, int4_group, prefix_len)


# --------------------------------------------------------------------------
# Attention over a shared prefix
# --------------------------------------------------------------------------
_DENSE = {n: (0,) * (n - 1) for n in range(1, 9)}


def _strides(t: torch.Tensor, name: str):
    """Strides of all dimensions but the last, which has to be dense; 0 for those
    of a dense tensor, and (of no consequence) for those of one element."""
    if t.is_contiguous():
        return _DENSE[t.dim()]
    if t.stride(-1) != 1:
        raise MtpError(f"{name} must be dense in its last dimension")
    if any(n > 1 and s == 0 for n, s in zip(t.shape, t.stride())):
        raise MtpError(f"{name} must not be expanded")
    return [0 if n == 1 else s for n, s in zip(t.shape[:-1], t.stride()[:-1])]


def _pair(k, v, name: str, dims: int, device):
    """Strides (None: dense) of keys and values of one shape and layout, the last dimension dense."""
    for t in (k, v):
        if t.dim() != dims or t.dtype is not torch.bfloat16 or t.device != device:
            raise MtpError(f"{name}_k and {name}_v must be bfloat16 tensors of {dims} dimensions on {device}")
    if k.shape == v.shape and k.is_contiguous() and v.is_contiguous():
        return None
    strides = _strides(k, name + "_k")
    if k.shape != v.shape or strides != _strides(v, name + "_v"):
        raise MtpError(f"{name}_k and {name}_v must have the same shape and strides")
    return strides


def prefix_attention(q: torch.Tensor, prefix_k: torch.Tensor, prefix_v: torch.Tensor,
                     kv_k: Optional[torch.Tensor] = None, kv_v: Optional[torch.Tensor] = None,
                     ctx_len: Optional[torch.Tensor] = None, causal: bool = True, scale: Optional[float] = None,
                     out: Optional[dict] = None, ws: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Attention of q [R, L, H, hd] over a prefix [P, Hkv, hd] that all requests
    share and each request's own cache [R, T, Hkv, hd] of ctx_len[r] rows, the
    last L of them the new tokens' own (include/mtp.h: mtp_prefix_attention).
    Any strides that are multiples of 8 with a dense last dimension will do.
    Returns {"o": bfloat16 [R, L, H, hd], "lse": float32 [R, L, H]}; ``out`` may
    supply them."""
    if q.dim() != 4 or q.dtype != torch.bfloat16:
        raise MtpError("q must be bfloat16 [R, L, H, hd]")
    dev = _launch_device(q, stream)
    R, L, H, hd = q.shape
    prefix_strides = _pair(prefix_k, prefix_v, "prefix", 3, dev)
    P, Hkv = prefix_k.shape[0], prefix_k.shape[1]
    if prefix_k.shape[2] != hd:
        raise MtpError("prefix_k must be [P, Hkv, hd]")
    d = PrefixDims(R, L, H, Hkv, hd, P, 0, int(causal), 0.0 if scale is None else float(scale))
    if scale is not None and not 0.0 < scale < 3e38:
        raise MtpError("scale must be positive and finite")
    if not q.is_contiguous():
        d.q_stride_r, d.q_stride_t, d.q_stride_h = _strides(q, "q")
    if prefix_strides is not None:
        d.prefix_stride_t, d.prefix_stride_h = prefix_strides
    if (kv_k is None) != (kv_v is None):
        raise MtpError("kv_k and kv_v come together")
    if kv_k is not None:
        kv_strides = _pair(kv_k, kv_v, "kv", 4, dev)
        if kv_k.shape[0] != R or tuple(kv_k.shape[2:]) != (Hkv, hd):
            raise MtpError("kv_k must be [R, T, Hkv, hd]")
        d.T = kv_k.shape[1]
        if kv_strides is not None:
            d.kv_stride_r, d.kv_stride_t, d.kv_stride_h = kv_strides
    elif ctx_len is not None:
        raise MtpError("ctx_len needs kv_k and kv_v")
    ctx = _arg(ctx_len, "ctx_len", torch.int32, (R,), dev)
    if out is None:
        out = {"o": _empty((R, L, H, hd), torch.bfloat16, dev, stream), "lse": _empty((R, L, H), torch.float32, dev, stream)}
    else:
        _arg(out["o"], "out['o']", torch.bfloat16, (R, L, H, hd), dev)
        _arg(out["lse"], "out['lse']", torch.float32, (R, L, H), dev)
    lib = load()
    if ws is None:
        ws = _empty(int(lib.mtp_prefix_attention_workspace_bytes(ctypes.byref(d))), torch.uint8, dev, stream)
    elif ws.device != dev or not ws.is_contiguous():
        raise MtpError(f"ws must be a contiguous tensor on {dev}")
    st = lib.mtp_prefix_attention(ctypes.byref(d), q.data_ptr(), prefix_k.data_ptr(), prefix_v.data_ptr(),
                                  kv_k.data_ptr() if d.T > 0 else None, kv_v.data_ptr() if d.T > 0 else None, ctx,
                                  out["o"].data_ptr(), out["lse"].data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(),
                                  _stream(stream))
    _check(st, "mtp_prefix_attention")
    return out
