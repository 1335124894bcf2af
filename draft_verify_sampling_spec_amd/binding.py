"""ctypes binding of ``libspec_verify.so`` (argument marshalling only).

Every function of the C ABI (include/spec_verify.h) is exposed under its own
name; ``SpecVerify`` wraps a context for torch tensors. Tensors are passed as
raw device pointers and the current torch stream as the HIP stream; all work
runs in the library's kernels. There is no fallback: if the library is not
built, ``load()`` raises.

torch is imported before the library is opened so that the library binds to
the HIP runtime torch already loaded (one runtime per process).
"""
from __future__ import annotations

import ctypes
import functools
import math
import os

import torch

from .build import LIB_PATH

SV_OK = 0
SV_ERR_NULL = -1
SV_ERR_ARG = -2
SV_ERR_DTYPE = -3
SV_ERR_ALIGN = -4
SV_ERR_HIP = -5
SV_ERR_NOMEM = -6
SV_ERR_STATE = -7
SV_ERR_TOO_BIG = -8

SV_DTYPE_F32 = 0
SV_DTYPE_BF16 = 1

SV_FLAG_BAD_BUDGET = 0x1
SV_FLAG_BAD_TOKEN = 0x2
SV_FLAG_SYNC_TIMEOUT = 0x4
SV_FLAG_BAD_LENGTH = 0x8
SV_FLAG_BAD_PAGE = 0x10
SV_FLAG_NO_PAGES = 0x20
SV_FLAG_BAD_PARENT = 0x40
SV_FLAG_NO_PREFIX = 0x80

SV_MAX_BATCH = 16384
SV_MAX_K = 32
SV_MAX_VOCAB = 1 << 20
SV_NOALLOC_SCRATCH_BYTES = 16 << 20
SV_MAX_HEADS = 256
SV_MAX_PAGE = 4096
SV_MAX_CONTEXT = 1 << 24
SV_MAX_HIDDEN = 65536
SV_MAX_STRIDE = 2147483647
SV_MAX_GROUPS = 512

EXPORTED = (
    "spec_verify_init",
    "spec_verify_run",
    "spec_verify_run_ex",
    "spec_verify_run_noalloc",
    "spec_verify_check_args",
    "spec_verify_status",
    "spec_verify_philox_words",
    "spec_verify_timing",
    "spec_verify_timing_read",
    "spec_budget_schedule",
    "spec_head_stats",
    "spec_head_workspace_bytes",
    "spec_verify_hidden",
    "spec_verify_hidden_workspace_bytes",
    "spec_markov_draft",
    "spec_markov_draft_workspace_bytes",
    "spec_verify_cache_bytes",
    "spec_verify_cache_write",
    "spec_verify_cache_read",
    "spec_verify_pages_plan",
    "spec_verify_pages_plan_workspace_bytes",
    "spec_verify_cache_write_rotated",
    "spec_verify_attention",
    "spec_verify_attention_workspace_bytes",
    "spec_verify_attention_sinks",
    "spec_verify_attention_sinks_workspace_bytes",
    "spec_verify_attention_shared",
    "spec_verify_attention_shared_workspace_bytes",
    "spec_head_quantize",
    "spec_head_logits",
    "spec_verify_free",
    "spec_verify_strerror",
    "spec_verify_chunks",
)

_lib = None

_vp = ctypes.c_void_p
_i = ctypes.c_int


def _declare(lib):
    lib.spec_verify_init.argtypes = [ctypes.POINTER(_vp), _i, _i, _i, _i, _i]
    lib.spec_verify_init.restype = _i
    lib.spec_verify_run.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, ctypes.c_float,
                                    ctypes.c_uint64, _vp, _vp, _vp, _vp, _vp]
    lib.spec_verify_run.restype = _i
    lib.spec_verify_run_ex.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, ctypes.c_float,
                                       ctypes.c_uint64, ctypes.c_int64, _vp, _vp, _vp, _vp, _vp]
    lib.spec_verify_run_ex.restype = _i
    lib.spec_verify_run_noalloc.argtypes = [_i, _i, _vp, _vp, _vp, _vp, _i, _i, ctypes.c_float,
                                            ctypes.c_uint64, ctypes.c_int64, _vp, _vp, _vp, _vp,
                                            _vp, _vp]
    lib.spec_verify_run_noalloc.restype = _i
    lib.spec_verify_check_args.argtypes = [_i, _i, _i, _i, _vp, _vp, _vp, _vp, _i, _i,
                                           ctypes.c_float, _vp, _vp, _vp, _vp]
    lib.spec_verify_check_args.restype = _i
    lib.spec_verify_status.argtypes = [_vp, ctypes.POINTER(ctypes.c_uint32)]
    lib.spec_verify_status.restype = _i
    lib.spec_verify_philox_words.argtypes = [ctypes.c_uint64, _i, _i, _vp, _vp]
    lib.spec_verify_philox_words.restype = _i
    lib.spec_verify_free.argtypes = [_vp]
    lib.spec_verify_free.restype = None
    lib.spec_verify_strerror.argtypes = [_i]
    lib.spec_verify_strerror.restype = ctypes.c_char_p
    lib.spec_verify_chunks.argtypes = [_i, _i]
    lib.spec_verify_chunks.restype = _i
    lib.spec_head_stats.argtypes = [_vp, _vp, _i, _i, _i, _vp, ctypes.c_float, _vp, _vp, _vp,
                                    _vp, _vp, ctypes.c_size_t, _vp]
    lib.spec_head_stats.restype = _i
    lib.spec_head_workspace_bytes.argtypes = [_i, _i]
    lib.spec_head_workspace_bytes.restype = ctypes.c_size_t
    lib.spec_verify_hidden.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, ctypes.c_float,
                                       ctypes.c_uint64, _vp, _vp, _vp, _vp, _vp, _vp,
                                       ctypes.c_size_t, _vp]
    lib.spec_verify_hidden.restype = _i
    lib.spec_verify_hidden_workspace_bytes.argtypes = [_i, _i, _i]
    lib.spec_verify_hidden_workspace_bytes.restype = ctypes.c_size_t
    lib.spec_markov_draft.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp,
                                      ctypes.c_size_t, _vp]
    lib.spec_markov_draft.restype = _i
    lib.spec_markov_draft_workspace_bytes.argtypes = [_i, _i]
    lib.spec_markov_draft_workspace_bytes.restype = ctypes.c_size_t
    lib.spec_budget_schedule.argtypes = [_vp, _i, _i, _i, ctypes.c_float, _vp, _vp]
    lib.spec_budget_schedule.restype = _i
    lib.spec_verify_cache_bytes.argtypes = [_i, _i, _i, _i]
    lib.spec_verify_cache_bytes.restype = ctypes.c_size_t
    lib.spec_verify_cache_write.argtypes = [_vp, _vp, _i, ctypes.c_int64, ctypes.c_int64, _vp,
                                            _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp]
    lib.spec_verify_cache_write.restype = _i
    lib.spec_verify_cache_read.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i,
                                           _vp, _vp, _vp, _vp]
    lib.spec_verify_cache_read.restype = _i
    lib.spec_verify_pages_plan.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i,
                                           _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
    lib.spec_verify_pages_plan.restype = _i
    lib.spec_verify_pages_plan_workspace_bytes.argtypes = [_i, _i, _i]
    lib.spec_verify_pages_plan_workspace_bytes.restype = ctypes.c_size_t
    lib.spec_verify_cache_write_rotated.argtypes = [
        _vp, _vp, _vp, _i, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, _vp, _vp, ctypes.c_int64,
        _vp, _i, _i, ctypes.c_float, _vp, _vp, _i, ctypes.c_float, _i, _i, _i, _i, _i, _vp, _vp, _vp,
        _vp, _vp]
    lib.spec_verify_cache_write_rotated.restype = _i
    lib.spec_verify_attention.argtypes = [_vp, ctypes.c_int64, _vp, _vp, _vp, _vp, _i, _i, _i, _i,
                                          _i, _i, _i, _i, ctypes.c_float, _i, _vp, _vp, _vp,
                                          ctypes.c_size_t, _vp]
    lib.spec_verify_attention.restype = _i
    lib.spec_verify_attention_sinks.argtypes = [
        _vp, ctypes.c_int64, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, ctypes.c_float, _i, _i,
        _vp, _vp, _vp, ctypes.c_size_t, _vp]
    lib.spec_verify_attention_sinks.restype = _i
    lib.spec_verify_attention_sinks_workspace_bytes.argtypes = [_i] * 9
    lib.spec_verify_attention_sinks_workspace_bytes.restype = ctypes.c_size_t
    lib.spec_verify_attention_shared.argtypes = [
        _vp, ctypes.c_int64, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _i,
        ctypes.c_float, _vp, _vp, _vp, ctypes.c_size_t, _vp]
    lib.spec_verify_attention_shared.restype = _i
    lib.spec_verify_attention_shared_workspace_bytes.argtypes = [_i] * 8
    lib.spec_verify_attention_shared_workspace_bytes.restype = ctypes.c_size_t
    lib.spec_verify_attention_workspace_bytes.argtypes = [_i, _i, _i, _i, _i, _i, _i, _i]
    lib.spec_verify_attention_workspace_bytes.restype = ctypes.c_size_t
    lib.spec_head_quantize.argtypes = [_vp, _i, _i, _i, _i, _vp, _vp, _vp]
    lib.spec_head_quantize.restype = _i
    lib.spec_head_logits.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp]
    lib.spec_head_logits.restype = _i
    lib.spec_verify_timing.argtypes = [_vp, _i]
    lib.spec_verify_timing.restype = _i
    lib.spec_verify_timing_read.argtypes = [_vp, ctypes.POINTER(_i), ctypes.POINTER(ctypes.c_double)]
    lib.spec_verify_timing_read.restype = _i


def load(path: str | None = None):
    """Open the built library (once per process)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is not built; run `python -m draft_verify_sampling_spec_amd.build`")
    lib = ctypes.CDLL(path)
    _declare(lib)
    _lib = lib
    return lib


# ---- the C functions under their own names ------------------------------------

def spec_verify_strerror(code: int) -> str:
    return load().spec_verify_strerror(int(code)).decode()


def spec_verify_chunks(vocab: int, dtype: int) -> int:
    return load().spec_verify_chunks(int(vocab), int(dtype))


def spec_verify_check_args(max_batch, max_k, vocab, dtype, target, draft, tokens, budgets,
                           B, K, temperature, out_tokens, out_num_accepted,
                           out_p_draft=None, out_q_draft=None) -> int:
    """Host-only argument check; pointer arguments are ints (addresses) or None."""
    return load().spec_verify_check_args(
        max_batch, max_k, vocab, dtype, target, draft, tokens, budgets, B, K,
        ctypes.c_float(temperature), out_tokens, out_num_accepted, out_p_draft, out_q_draft)


def spec_verify_init(device: int, max_batch: int, max_k: int, vocab: int, dtype: int):
    """Returns (status, ctx handle or None)."""
    ctx = _vp()
    rc = load().spec_verify_init(ctypes.byref(ctx), device, max_batch, max_k, vocab, dtype)
    return rc, (ctx.value if rc == SV_OK else None)


def spec_verify_run(ctx, target, draft, tokens, budgets, B, K, temperature, seed,
                    out_tokens, out_num_accepted, out_p_draft, out_q_draft, stream) -> int:
    return load().spec_verify_run(ctx, target, draft, tokens, budgets, B, K,
                                  ctypes.c_float(temperature), ctypes.c_uint64(seed),
                                  out_tokens, out_num_accepted, out_p_draft, out_q_draft,
                                  stream)


def spec_verify_run_ex(ctx, target, draft, tokens, budgets, B, K, temperature, seed,
                       request_base, out_tokens, out_num_accepted, out_p_draft, out_q_draft,
                       stream) -> int:
    return load().spec_verify_run_ex(ctx, target, draft, tokens, budgets, B, K,
                                     ctypes.c_float(temperature), ctypes.c_uint64(seed),
                                     ctypes.c_int64(request_base), out_tokens, out_num_accepted,
                                     out_p_draft, out_q_draft, stream)


def spec_verify_run_noalloc(vocab, dtype, target, draft, tokens, budgets, B, K, temperature,
                            seed, request_base, out_tokens, out_num_accepted, out_p_draft,
                            out_q_draft, out_status, stream) -> int:
    return load().spec_verify_run_noalloc(vocab, dtype, target, draft, tokens, budgets, B, K,
                                          ctypes.c_float(temperature), ctypes.c_uint64(seed),
                                          ctypes.c_int64(request_base), out_tokens,
                                          out_num_accepted, out_p_draft, out_q_draft, out_status,
                                          stream)


def spec_verify_status(ctx):
    """Returns (status, flags)."""
    flags = ctypes.c_uint32(0)
    rc = load().spec_verify_status(ctx, ctypes.byref(flags))
    return rc, flags.value


def spec_verify_philox_words(seed: int, B: int, P: int, out_words, stream) -> int:
    return load().spec_verify_philox_words(ctypes.c_uint64(seed), B, P, out_words, stream)


def spec_budget_schedule(confidences, B: int, K: int, n_total: int, tau: float, out_budgets,
                         stream) -> int:
    return load().spec_budget_schedule(confidences, B, K, n_total, ctypes.c_float(tau),
                                       out_budgets, stream)


def spec_verify_timing(ctx, enable: bool) -> int:
    return load().spec_verify_timing(ctx, 1 if enable else 0)


def spec_verify_timing_read(ctx):
    """Returns (status, [launches of pass 0, pass 1], [total ms of pass 0, pass 1])."""
    counts = (_i * 2)()
    total = (ctypes.c_double * 2)()
    rc = load().spec_verify_timing_read(ctx, counts, total)
    return rc, [counts[0], counts[1]], [total[0], total[1]]


def spec_verify_free(ctx) -> None:
    load().spec_verify_free(ctx)


# ---- torch convenience ----------------------------------------------------------

def _check(rc: int, what: str):
    if rc != SV_OK:
        raise RuntimeError(f"{what}: {spec_verify_strerror(rc)} ({rc})")


def _stream_handle(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


_DTYPES = {torch.float32: SV_DTYPE_F32, torch.bfloat16: SV_DTYPE_BF16}


class SpecVerify:
    """A verify context bound to one device, vocabulary and logit dtype."""

    def __init__(self, device, max_batch: int, max_k: int, vocab: int,
                 dtype: torch.dtype = torch.bfloat16):
        if dtype not in _DTYPES:
            raise ValueError(f"logits must be float32 or bfloat16, not {dtype}")
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError("SpecVerify needs a GPU device")
        self.max_batch, self.max_k, self.vocab, self.dtype = max_batch, max_k, vocab, dtype
        idx = self.device.index if self.device.index is not None else torch.cuda.current_device()
        rc, ctx = spec_verify_init(idx, max_batch, max_k, vocab, _DTYPES[dtype])
        _check(rc, "spec_verify_init")
        self._ctx = ctx

    def close(self):
        if getattr(self, "_ctx", None):
            spec_verify_free(self._ctx)
            self._ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _tensor(self, t, name, dtype, shape):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.device != self.device and not (t.device.type == "cuda" and self.device.index is None):
            raise ValueError(f"{name} is on {t.device}, context on {self.device}")
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()

    def run(self, target, draft, tokens, budgets, temperature: float, seed: int,
            out_tokens=None, out_num_accepted=None, out_p=None, out_q=None,
            want_probs: bool = True, stream=None, request_base: int = 0):
        """Verify a batch. Returns (tokens [B,K+1], n_accepted [B], p_x, q_x).

        p_x/q_x are None unless ``want_probs`` (or output buffers are given).
        ``request_base``: index of row 0 in the whole batch (its Philox
        counter). Enqueued on ``stream`` (default: the current torch stream),
        not waited for; device-side problems (a bad budget or token) only
        show in ``status()``, which waits.
        """
        if target.dim() != 3:
            raise ValueError("target logits must be [B, K+1, V]")
        B, K1, V = target.shape
        K = K1 - 1
        if V != self.vocab:
            raise ValueError(f"vocabulary {V} != context vocabulary {self.vocab}")
        temperature = float(temperature)
        if not math.isfinite(temperature) or temperature < 0:
            raise ValueError("temperature must be finite and >= 0")
        t_ptr = self._tensor(target, "target", self.dtype, (B, K + 1, V))
        d_ptr = None
        if draft is not None:
            d_ptr = self._tensor(draft, "draft", self.dtype, (B, K, V))
        elif temperature > 0 and K > 0:
            raise ValueError("sampled verification needs drafter logits")
        x_ptr = self._tensor(tokens, "tokens", torch.int32, (B, K))
        k_ptr = self._tensor(budgets, "budgets", torch.int32, (B,))
        dev = target.device
        if out_tokens is None:
            out_tokens = torch.empty(B, K + 1, dtype=torch.int32, device=dev)
        if out_num_accepted is None:
            out_num_accepted = torch.empty(B, dtype=torch.int32, device=dev)
        if want_probs and out_p is None:
            out_p = torch.empty(B, K, dtype=torch.float32, device=dev)
        if want_probs and out_q is None:
            out_q = torch.empty(B, K, dtype=torch.float32, device=dev)
        ot = self._tensor(out_tokens, "out_tokens", torch.int32, (B, K + 1))
        on = self._tensor(out_num_accepted, "out_num_accepted", torch.int32, (B,))
        op = self._tensor(out_p, "out_p", torch.float32, (B, K)) if out_p is not None else None
        oq = self._tensor(out_q, "out_q", torch.float32, (B, K)) if out_q is not None else None
        s = stream.cuda_stream if stream is not None else _stream_handle(dev)
        rc = spec_verify_run_ex(self._ctx, t_ptr, d_ptr, x_ptr, k_ptr, B, K, temperature,
                                int(seed) & 0xFFFFFFFFFFFFFFFF, int(request_base), ot, on, op, oq,
                                s)
        _check(rc, "spec_verify_run_ex")
        return out_tokens, out_num_accepted, out_p, out_q

    def status(self) -> int:
        rc, flags = spec_verify_status(self._ctx)
        _check(rc, "spec_verify_status")
        return flags

    def timing(self, enable: bool) -> None:
        """Start (True) or stop and discard (False) per-pass event timing."""
        _check(spec_verify_timing(self._ctx, enable), "spec_verify_timing")

    def pass_times(self):
        """Launch counts and summed milliseconds of the streaming pass and the
        draw pass recorded since the last read (waits for them)."""
        rc, counts, total = spec_verify_timing_read(self._ctx)
        _check(rc, "spec_verify_timing_read")
        return counts, total


def verify_noalloc(target, draft, tokens, budgets, temperature: float, seed: int,
                   request_base: int = 0, out_tokens=None, out_num_accepted=None, out_p=None,
                   out_q=None, out_status=None, stream=None):
    """One verify call through the allocation-free entry point (the library's
    static scratch; no context). Tensors as for ``SpecVerify.run``; outputs
    not given are allocated here with torch (a caller that cannot allocate
    passes them all). Returns (tokens, n_accepted, p_x, q_x, status [1])."""
    if target.dim() != 3 or target.dtype not in _DTYPES:
        raise ValueError("target logits must be a float32 or bfloat16 [B, K+1, V] tensor")
    B, K1, V = target.shape
    K = K1 - 1
    dev = target.device
    mats = [(target, target.dtype, (B, K + 1, V)), (tokens, torch.int32, (B, K)),
            (budgets, torch.int32, (B,))]
    if draft is not None:
        mats.append((draft, target.dtype, (B, K, V)))
    for t, dt, shape in mats:
        if t.dtype != dt or tuple(t.shape) != shape or not t.is_contiguous() or t.device != dev:
            raise ValueError(f"expected a contiguous {dt} tensor of shape {shape} on {dev}")
    if out_tokens is None:
        out_tokens = torch.empty(B, K + 1, dtype=torch.int32, device=dev)
    if out_num_accepted is None:
        out_num_accepted = torch.empty(B, dtype=torch.int32, device=dev)
    if out_p is None:
        out_p = torch.empty(B, K, dtype=torch.float32, device=dev)
    if out_q is None:
        out_q = torch.empty(B, K, dtype=torch.float32, device=dev)
    if out_status is None:
        out_status = torch.empty(1, dtype=torch.int32, device=dev)
    s = stream.cuda_stream if stream is not None else _stream_handle(dev)
    with torch.cuda.device(dev):
        rc = spec_verify_run_noalloc(V, _DTYPES[target.dtype], target.data_ptr(),
                                     None if draft is None else draft.data_ptr(),
                                     tokens.data_ptr(), budgets.data_ptr(), B, K,
                                     float(temperature), int(seed) & 0xFFFFFFFFFFFFFFFF,
                                     int(request_base), out_tokens.data_ptr(),
                                     out_num_accepted.data_ptr(), out_p.data_ptr(),
                                     out_q.data_ptr(), out_status.data_ptr(), s)
    _check(rc, "spec_verify_run_noalloc")
    return out_tokens, out_num_accepted, out_p, out_q, out_status


def philox_words(seed: int, B: int, P: int, device="cuda") -> torch.Tensor:
    """The device generator's blocks for counters (b, i, 0, 0): [B, P, 4] int64."""
    out = torch.empty(B * P * 4, dtype=torch.int32, device=device)
    rc = spec_verify_philox_words(int(seed) & 0xFFFFFFFFFFFFFFFF, B, P, out.data_ptr(),
                                  _stream_handle(out.device))
    _check(rc, "spec_verify_philox_words")
    return out.view(B, P, 4).to(torch.int64) & 0xFFFFFFFF


def schedule_budgets(confidences: torch.Tensor, n_total: int, tau: float = 0.0,
                     out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Per-request verify budgets (int32 [B]) from per-position confidences
    (float32 [B, K], contiguous, on the GPU): the N largest gains above tau.
    Enqueued on ``stream`` (default: the current torch stream)."""
    if confidences.dim() != 2 or confidences.dtype != torch.float32:
        raise ValueError("confidences must be a float32 [B, K] tensor")
    if not confidences.is_cuda or not confidences.is_contiguous():
        raise ValueError("confidences must be a contiguous GPU tensor")
    B, K = confidences.shape
    if out is None:
        out = torch.empty(B, dtype=torch.int32, device=confidences.device)
    elif out.dtype != torch.int32 or out.shape != (B,) or not out.is_contiguous() \
            or out.device != confidences.device:
        raise ValueError("out must be a contiguous int32 [B] tensor on the same device")
    s = stream.cuda_stream if stream is not None else _stream_handle(confidences.device)
    rc = spec_budget_schedule(confidences.data_ptr(), B, K, int(n_total), float(tau),
                              out.data_ptr(), s)
    _check(rc, "spec_budget_schedule")
    return out


def spec_head_workspace_bytes(R: int, V: int) -> int:
    return int(load().spec_head_workspace_bytes(int(R), int(V)))


def spec_head_stats(hidden, weight, R, H, V, tokens, temperature, out_max, out_sumexp, out_ztok,
                    out_argmax, workspace, workspace_bytes, stream) -> int:
    return load().spec_head_stats(hidden, weight, R, H, V, tokens, ctypes.c_float(temperature),
                                  out_max, out_sumexp, out_ztok, out_argmax, workspace,
                                  ctypes.c_size_t(workspace_bytes), stream)


def head_stats(hidden: torch.Tensor, weight: torch.Tensor, tokens: torch.Tensor | None,
               temperature: float, stream=None):
    """Row statistics of hidden @ weight^T (bf16 [R, H] and [V, H], contiguous,
    on the GPU): (max, exp-sum, token logit, first argmax) as tensors [R].
    Allocates its outputs and scratch with torch; enqueued on ``stream``."""
    if hidden.dtype != torch.bfloat16 or weight.dtype != torch.bfloat16:
        raise ValueError("hidden and weight must be bfloat16")
    if hidden.dim() != 2 or weight.dim() != 2 or hidden.shape[1] != weight.shape[1]:
        raise ValueError("hidden [R, H] and weight [V, H] must share H")
    if not (hidden.is_cuda and weight.is_cuda and hidden.is_contiguous() and weight.is_contiguous()):
        raise ValueError("hidden and weight must be contiguous GPU tensors")
    R, H = hidden.shape
    V = weight.shape[0]
    dev = hidden.device
    out_m = torch.empty(R, dtype=torch.float32, device=dev)
    out_s = torch.empty(R, dtype=torch.float32, device=dev)
    out_z = torch.empty(R, dtype=torch.float32, device=dev)
    out_a = torch.empty(R, dtype=torch.int32, device=dev)
    nbytes = spec_head_workspace_bytes(max(R, 1), V)
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
    tp = 0
    if tokens is not None:
        if tokens.dtype != torch.int32 or tokens.shape != (R,) or not tokens.is_contiguous():
            raise ValueError("tokens must be a contiguous int32 [R] tensor")
        tp = tokens.data_ptr()
    s = stream.cuda_stream if stream is not None else _stream_handle(dev)
    rc = spec_head_stats(hidden.data_ptr(), weight.data_ptr(), R, H, V, tp or None,
                         float(temperature), out_m.data_ptr(), out_s.data_ptr(), out_z.data_ptr(),
                         out_a.data_ptr(), ws.data_ptr(), ws.numel(), s)
    _check(rc, "spec_head_stats")
    return out_m, out_s, out_z, out_a


def spec_verify_hidden_workspace_bytes(B: int, K: int, V: int) -> int:
    return int(load().spec_verify_hidden_workspace_bytes(int(B), int(K), int(V)))


def spec_verify_hidden(target_hidden, draft_hidden, head, draft_tokens, budgets, B, K, H, V,
                       temperature, seed, out_tokens, out_num_accepted, out_p, out_q,
                       out_status, workspace, workspace_bytes, stream) -> int:
    return load().spec_verify_hidden(target_hidden, draft_hidden, head, draft_tokens, budgets,
                                     B, K, H, V, ctypes.c_float(temperature),
                                     ctypes.c_uint64(seed), out_tokens, out_num_accepted, out_p,
                                     out_q, out_status, workspace,
                                     ctypes.c_size_t(workspace_bytes), stream)


class HiddenVerify:
    """Verify steps from hidden states through the shared head, for one
    batch shape (B, K, V) on one device. Holds the library's workspace
    (torch-allocated) across calls; outputs are fresh tensors per call."""

    def __init__(self, device, B: int, K: int, V: int):
        self.device = torch.device(device)
        self.B, self.K, self.V = int(B), int(K), int(V)
        nbytes = spec_verify_hidden_workspace_bytes(max(self.B, 1), self.K, self.V)
        if nbytes == 0:
            raise ValueError(f"bad shape B={B} K={K} V={V}")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=self.device)

    def run(self, target_hidden: torch.Tensor, draft_hidden: torch.Tensor | None,
            head: torch.Tensor, tokens: torch.Tensor, budgets: torch.Tensor,
            temperature: float, seed: int, stream=None):
        """(tokens [B, K+1], n_accepted [B], p_x [B, K], q_x [B, K], status [1])."""
        B, K, V = self.B, self.K, self.V
        if target_hidden.dim() != 3 or target_hidden.shape[:2] != (B, K + 1):
            raise ValueError("target_hidden must be [B, K+1, H]")
        H = int(target_hidden.shape[2])
        if head.shape != (V, H):
            raise ValueError("head must be [V, H]")
        greedy = float(temperature) == 0.0
        mats = [target_hidden, head] + ([] if draft_hidden is None else [draft_hidden])
        for m in mats:
            if m.dtype != torch.bfloat16 or not m.is_contiguous() or m.device != self.device:
                raise ValueError("hidden states and head must be contiguous bf16 on the device")
        if draft_hidden is not None and draft_hidden.shape != (B, K, H):
            raise ValueError("draft_hidden must be [B, K, H]")
        if not greedy and K > 0 and draft_hidden is None:
            raise ValueError("sampled verification needs draft_hidden")
        for t, shape in ((tokens, (B, K)), (budgets, (B,))):
            if t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous():
                raise ValueError(f"expected a contiguous int32 tensor of shape {shape}")
        dev = self.device
        out_tok = torch.empty((B, K + 1), dtype=torch.int32, device=dev)
        out_n = torch.empty(B, dtype=torch.int32, device=dev)
        out_p = torch.empty((B, K), dtype=torch.float32, device=dev)
        out_q = torch.empty((B, K), dtype=torch.float32, device=dev)
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        s = stream.cuda_stream if stream is not None else _stream_handle(dev)
        rc = spec_verify_hidden(target_hidden.data_ptr(),
                                None if draft_hidden is None else draft_hidden.data_ptr(),
                                head.data_ptr(), tokens.data_ptr() if K > 0 else None,
                                budgets.data_ptr(), B, K, H, V, float(temperature),
                                int(seed) & 0xFFFFFFFFFFFFFFFF, out_tok.data_ptr(),
                                out_n.data_ptr(), out_p.data_ptr(), out_q.data_ptr(),
                                status.data_ptr(), self.workspace.data_ptr(),
                                self.workspace.numel(), s)
        _check(rc, "spec_verify_hidden")
        return out_tok, out_n, out_p, out_q, status


def spec_markov_draft_workspace_bytes(B: int, V: int) -> int:
    return int(load().spec_markov_draft_workspace_bytes(int(B), int(V)))


def spec_markov_draft(base_logits, markov_a, markov_b, prev_tokens, B, K, r, V, out_logits,
                      out_tokens, out_status, workspace, workspace_bytes, stream) -> int:
    return load().spec_markov_draft(base_logits, markov_a, markov_b, prev_tokens, B, K, r, V,
                                    out_logits, out_tokens, out_status, workspace,
                                    ctypes.c_size_t(workspace_bytes), stream)


class MarkovDraft:
    """Drafted blocks through the low-rank Markov head, for one batch shape
    (B, K, V) on one device. Holds the library's workspace (torch-allocated)
    across calls; outputs are fresh tensors per call unless given."""

    def __init__(self, device, B: int, K: int, V: int):
        self.device = torch.device(device)
        self.B, self.K, self.V = int(B), int(K), int(V)
        nbytes = spec_markov_draft_workspace_bytes(max(self.B, 1), self.V)
        if nbytes == 0:
            raise ValueError(f"bad shape B={B} V={V}")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=self.device)

    def run(self, base_logits: torch.Tensor, markov_a: torch.Tensor, markov_b: torch.Tensor,
            prev_tokens: torch.Tensor, out_logits=None, out_tokens=None, stream=None):
        """(drafter logits bf16 [B, K, V], drafted tokens int32 [B, K], status int32 [1])."""
        B, K, V = self.B, self.K, self.V
        if base_logits.shape != (B, K, V):
            raise ValueError("base_logits must be [B, K, V]")
        if markov_a.dim() != 2 or markov_a.shape[0] != V or markov_b.shape != markov_a.shape:
            raise ValueError("markov_a and markov_b must both be [V, r]")
        r = int(markov_a.shape[1])
        for m in (base_logits, markov_a, markov_b):
            if m.dtype != torch.bfloat16 or not m.is_contiguous() or m.device != self.device:
                raise ValueError("logits and Markov factors must be contiguous bf16 on the device")
        if (prev_tokens.dtype != torch.int32 or prev_tokens.shape != (B,)
                or not prev_tokens.is_contiguous() or prev_tokens.device != self.device):
            raise ValueError(f"prev_tokens must be a contiguous int32 tensor of shape ({B},)")
        dev = self.device
        if out_logits is None:
            out_logits = torch.empty((B, K, V), dtype=torch.bfloat16, device=dev)
        if out_tokens is None:
            out_tokens = torch.empty((B, K), dtype=torch.int32, device=dev)
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        s = stream.cuda_stream if stream is not None else _stream_handle(dev)
        rc = spec_markov_draft(base_logits.data_ptr(), markov_a.data_ptr(), markov_b.data_ptr(),
                               prev_tokens.data_ptr(), B, K, r, V, out_logits.data_ptr(),
                               out_tokens.data_ptr(), status.data_ptr(),
                               self.workspace.data_ptr(), self.workspace.numel(), s)
        _check(rc, "spec_markov_draft")
        return out_logits, out_tokens, status


# ---- the paged 4-bit cache and the 8-bit head --------------------------------------

def spec_verify_cache_bytes(num_pages: int, kv_heads: int, head_dim: int, page_size: int) -> int:
    return int(load().spec_verify_cache_bytes(int(num_pages), int(kv_heads), int(head_dim),
                                              int(page_size)))


def spec_verify_cache_write(keys, values, dtype, key_stride, value_stride, page_table, ctx_lens,
                            budgets, B, T, kv_heads, head_dim, page_size, max_pages, num_pages,
                            cache, out_status, stream) -> int:
    return load().spec_verify_cache_write(keys, values, dtype, key_stride, value_stride,
                                          page_table, ctx_lens, budgets, B, T, kv_heads, head_dim,
                                          page_size, max_pages, num_pages, cache, out_status,
                                          stream)


def spec_verify_cache_read(cache, page_table, starts, lens, B, T, kv_heads, head_dim, page_size,
                           max_pages, num_pages, dtype, out_keys, out_values, out_status,
                           stream) -> int:
    return load().spec_verify_cache_read(cache, page_table, starts, lens, B, T, kv_heads,
                                         head_dim, page_size, max_pages, num_pages, dtype,
                                         out_keys, out_values, out_status, stream)


def spec_verify_pages_plan(page_table, page_refs, ctx_lens, budgets, parents, prefix_lens, B, T,
                           page_size, max_pages, num_pages, window, sinks, out_starts, out_slots,
                           out_positions, out_status, workspace, workspace_bytes, stream) -> int:
    return load().spec_verify_pages_plan(page_table, page_refs, ctx_lens, budgets, parents,
                                         prefix_lens, B, T, page_size, max_pages, num_pages, window,
                                         sinks, out_starts, out_slots, out_positions, out_status,
                                         workspace, workspace_bytes, stream)


def spec_verify_pages_plan_workspace_bytes(B: int, max_pages: int, num_pages: int) -> int:
    return int(load().spec_verify_pages_plan_workspace_bytes(int(B), int(max_pages),
                                                             int(num_pages)))


def spec_verify_cache_write_rotated(queries, keys, values, dtype, query_stride, key_stride,
                                    value_stride, slots, positions, tokens, inv_freq, rot,
                                    interleaved, factor, q_norm, k_norm, norm_dtype, eps, q_heads,
                                    kv_heads, head_dim, page_size, num_pages, cache, out_queries,
                                    out_keys, out_status, stream) -> int:
    return load().spec_verify_cache_write_rotated(
        queries, keys, values, dtype, query_stride, key_stride, value_stride, slots, positions,
        tokens, inv_freq, rot, interleaved, factor, q_norm, k_norm, norm_dtype, eps, q_heads,
        kv_heads, head_dim, page_size, num_pages, cache, out_queries, out_keys, out_status, stream)


def spec_verify_attention(queries, query_stride, cache, page_table, ctx_lens, budgets, B, K,
                          q_heads, kv_heads, head_dim, page_size, max_pages, num_pages, scale,
                          window, out, out_status, workspace, workspace_bytes, stream) -> int:
    return load().spec_verify_attention(queries, query_stride, cache, page_table, ctx_lens,
                                        budgets, B, K, q_heads, kv_heads, head_dim, page_size,
                                        max_pages, num_pages, scale, window, out, out_status,
                                        workspace, workspace_bytes, stream)


def spec_verify_attention_workspace_bytes(B: int, K: int, q_heads: int, kv_heads: int,
                                          head_dim: int, page_size: int, max_pages: int,
                                          window: int = 0) -> int:
    return int(load().spec_verify_attention_workspace_bytes(
        int(B), int(K), int(q_heads), int(kv_heads), int(head_dim), int(page_size),
        int(max_pages), int(window)))


def spec_verify_attention_sinks(queries, query_stride, cache, page_table, ctx_lens, budgets, B, K,
                                q_heads, kv_heads, head_dim, page_size, max_pages, num_pages,
                                scale, window, sinks, out, out_status, workspace, workspace_bytes,
                                stream) -> int:
    return load().spec_verify_attention_sinks(queries, query_stride, cache, page_table, ctx_lens,
                                              budgets, B, K, q_heads, kv_heads, head_dim,
                                              page_size, max_pages, num_pages, scale, window,
                                              sinks, out, out_status, workspace, workspace_bytes,
                                              stream)


def spec_verify_attention_sinks_workspace_bytes(B: int, K: int, q_heads: int, kv_heads: int,
                                                head_dim: int, page_size: int, max_pages: int,
                                                window: int, sinks: int) -> int:
    return int(load().spec_verify_attention_sinks_workspace_bytes(
        int(B), int(K), int(q_heads), int(kv_heads), int(head_dim), int(page_size),
        int(max_pages), int(window), int(sinks)))


def spec_verify_attention_shared(queries, query_stride, cache, page_table, ctx_lens, budgets,
                                 groups, shared_lens, B, K, G, q_heads, kv_heads, head_dim,
                                 page_size, max_pages, num_pages, scale, out, out_status, workspace,
                                 workspace_bytes, stream) -> int:
    return load().spec_verify_attention_shared(queries, query_stride, cache, page_table, ctx_lens,
                                               budgets, groups, shared_lens, B, K, G, q_heads,
                                               kv_heads, head_dim, page_size, max_pages, num_pages,
                                               scale, out, out_status, workspace, workspace_bytes,
                                               stream)


def spec_verify_attention_shared_workspace_bytes(B: int, K: int, G: int, q_heads: int,
                                                 kv_heads: int, head_dim: int, page_size: int,
                                                 max_pages: int) -> int:
    return int(load().spec_verify_attention_shared_workspace_bytes(
        int(B), int(K), int(G), int(q_heads), int(kv_heads), int(head_dim), int(page_size),
        int(max_pages)))


def spec_head_quantize(src, dtype, rows, H, block_rows, out_codes, out_scales, stream) -> int:
    return load().spec_head_quantize(src, dtype, rows, H, block_rows, out_codes, out_scales, stream)


def spec_head_logits(h_codes, h_scales, w_codes, w_scales, R, H, V, dtype, out, stream) -> int:
    return load().spec_head_logits(h_codes, h_scales, w_codes, w_scales, R, H, V, dtype, out,
                                   stream)


# A serving step makes these calls for every layer, so what they cost on the
# host counts: arguments are checked without building messages, the stream and
# device are read through torch's own accessors, and the C function is called
# directly. A call for another stream, or from another current device, enters
# torch's context for it and calls itself: tensors that torch allocates inside
# belong to that stream, so that one freed when the call returns is not handed
# out again before the stream is done with it.

# A torch build without GPU support has no such accessors and still imports this.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


# A function of the shapes alone, for every layer and step: the last shapes' sizes.
_attention_bytes = functools.lru_cache(maxsize=1024)(spec_verify_attention_workspace_bytes)
_sinks_bytes = functools.lru_cache(maxsize=1024)(spec_verify_attention_sinks_workspace_bytes)
_shared_bytes = functools.lru_cache(maxsize=1024)(spec_verify_attention_shared_workspace_bytes)


def _need(t, name, dtype, shape, index):
    """The address of a contiguous tensor of exactly this type, shape and GPU."""
    if isinstance(t, torch.Tensor):
        if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
            return t.data_ptr()
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on "
                         f"cuda:{index}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    raise TypeError(f"{name} must be a torch.Tensor")


def _other_stream(stream, index):
    if stream.device.index != index:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
    return torch.cuda.stream(stream)


def _ready(index):
    """Waits for what a constructor enqueued, so that calls on any stream find it
    done (not in a capture, which cannot wait and replays it in order)."""
    with torch.cuda.device(index):
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream().synchronize()


def _token_stride(t, name, index):
    """Elements between tokens of a [B, T, heads, head_dim] tensor whose heads
    are contiguous and whose requests follow each other."""
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the cache on cuda:{index}")
    B, T, heads, dim = t.shape
    if t.is_contiguous():
        return heads * dim
    sb, st, sh, sd = t.stride()
    stride = st if T > 1 else sb if B > 1 else heads * dim
    if (sd != 1 or (heads > 1 and sh != dim) or (B > 1 and T > 1 and sb != T * stride)
            or stride < heads * dim):
        raise ValueError(f"{name} must have contiguous heads and evenly spaced tokens, got "
                         f"strides {t.stride()}")
    return stride


class BlockCache:
    """A target layer's paged 4-bit key/value cache on one device: writing
    blocks (or prompts), reading tokens back, and the attention of drafted
    blocks over it. Holds the pool (torch-allocated, and ready on every stream,
    unless given: uint8 [num_pages, kv_heads, page_size / 32, 34 head_dim];
    ``pool`` may be replaced by another of that shape between calls); the page
    table and the lengths are the caller's.

    ``status`` (int32 [1] on the device, or None) collects SV_FLAG_* bits;
    nothing clears it. Calls are enqueued on ``stream`` (default: the current
    torch stream) and not waited for."""

    def __init__(self, device, num_pages: int, kv_heads: int, head_dim: int, page_size: int = 64,
                 pool: torch.Tensor | None = None):
        device = torch.device(device)
        if device.type != "cuda":
            raise ValueError("BlockCache needs a GPU device")
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        self.device, self._index = device, device.index
        self.num_pages, self.kv_heads = int(num_pages), int(kv_heads)
        self.head_dim, self.page_size = int(head_dim), int(page_size)
        if spec_verify_cache_bytes(num_pages, kv_heads, head_dim, page_size) == 0:
            raise ValueError(f"bad cache geometry: {num_pages} pages of {page_size} tokens, "
                             f"{kv_heads} heads of {head_dim}")
        self.pool = torch.zeros(self._pool_shape(), dtype=torch.uint8, device=device) \
            if pool is None else pool
        self._pool_ptr()
        # For calls whose plan has no parts, which leave their 256 bytes alone.
        self._no_parts = torch.empty(256, dtype=torch.uint8, device=device)
        if pool is None:
            _ready(self._index)

    def _pool_shape(self):
        return self.num_pages, self.kv_heads, self.page_size // 32, 34 * self.head_dim

    def _pool_ptr(self):
        # At every call: ``pool`` may be another tensor, or have other storage, by then.
        return _need(self.pool, "pool", torch.uint8, self._pool_shape(), self._index)

    def _table(self, page_table, B):
        shape = page_table.shape
        if len(shape) != 2 or shape[0] != B or shape[1] < 1:
            raise ValueError(f"page_table must be [{B}, max_pages], got {tuple(shape)}")
        return _need(page_table, "page_table", torch.int32, shape, self._index), shape[1]

    def write(self, keys, values, page_table, ctx_lens, budgets=None, status=None, stream=None):
        """Quantise [B, T, kv_heads, head_dim] keys and values (float32 or
        bfloat16; slices of a fused projection's rows are fine) into positions
        ctx_lens[b] .. ctx_lens[b] + budgets[b] of every request."""
        index = self._index
        if stream is not None:
            with _other_stream(stream, index):
                return self.write(keys, values, page_table, ctx_lens, budgets, status)
        if _current_device() != index:
            with torch.cuda.device(index):
                return self.write(keys, values, page_table, ctx_lens, budgets, status)
        shape = keys.shape
        if len(shape) != 4 or shape[2] != self.kv_heads or shape[3] != self.head_dim:
            raise ValueError(f"keys must be [B, T, {self.kv_heads}, {self.head_dim}]")
        dtype = _DTYPES.get(keys.dtype)
        if values.shape != shape or values.dtype is not keys.dtype or dtype is None:
            raise ValueError("keys and values must share their shape and be float32 or bfloat16")
        B, T = shape[0], shape[1]
        ks = _token_stride(keys, "keys", index)
        vs = _token_stride(values, "values", index)
        table, width = self._table(page_table, B)
        rc = load().spec_verify_cache_write(
            keys.data_ptr(), values.data_ptr(), dtype, ks, vs, table,
            _need(ctx_lens, "ctx_lens", torch.int32, (B,), index),
            None if budgets is None else _need(budgets, "budgets", torch.int32, (B,), index),
            B, T, self.kv_heads, self.head_dim, self.page_size, width, self.num_pages,
            self._pool_ptr(),
            None if status is None else _need(status, "status", torch.int32, (1,), index),
            _raw_stream(index))
        if rc != SV_OK:
            _check(rc, "spec_verify_cache_write")

    def write_rotated(self, queries, keys, values, slots, positions, inv_freq=None, q_norm=None,
                      k_norm=None, eps: float = 1e-6, interleaved: bool = False,
                      factor: float = 1.0, out=None, out_keys=None, status=None, stream=None):
        """Normalise (weights q_norm, k_norm [head_dim], float32 or bfloat16;
        None: not) and rotate (inv_freq float32 [rot / 2], rot a multiple of 16;
        None: not) the queries [B, T, q_heads, head_dim] and keys [B, T, kv_heads,
        head_dim] of a step, float32 or bfloat16, at ``positions`` int32 [B, T];
        returns the queries (bfloat16), and quantises keys and values into the
        cache at ``slots`` int32 [B, T] (both from ``PageTables.plan``). Pairs are
        the channels i and i + rot / 2, or with ``interleaved`` 2 i and 2 i + 1;
        cosine and sine are multiplied by ``factor``. ``out_keys``, if given,
        receives the rotated keys in bfloat16. Tokens with a negative slot are
        skipped: ``out`` keeps its values there (a fresh one is zero)."""
        index = self._index
        if stream is not None:
            with _other_stream(stream, index):
                return self.write_rotated(queries, keys, values, slots, positions, inv_freq, q_norm,
                                          k_norm, eps, interleaved, factor, out, out_keys, status)
        if _current_device() != index:
            with torch.cuda.device(index):
                return self.write_rotated(queries, keys, values, slots, positions, inv_freq, q_norm,
                                          k_norm, eps, interleaved, factor, out, out_keys, status)
        shape, kv = queries.shape, keys.shape
        if len(shape) != 4 or shape[3] != self.head_dim or shape[2] % self.kv_heads != 0 \
                or kv != (shape[0], shape[1], self.kv_heads, self.head_dim) or values.shape != kv:
            raise ValueError(f"queries must be [B, T, q_heads, {self.head_dim}] and keys and values "
                             f"[B, T, {self.kv_heads}, {self.head_dim}]")
        dtype = _DTYPES.get(queries.dtype)
        if dtype is None or keys.dtype is not queries.dtype or values.dtype is not queries.dtype:
            raise ValueError("queries, keys and values must share their type, float32 or bfloat16")
        B, T, heads, dim = shape
        rot = 0
        if inv_freq is not None:
            rot = 2 * inv_freq.numel()
            if rot % 16 != 0 or rot > dim:
                raise ValueError(f"inv_freq must have a multiple of 8 entries, at most {dim // 2}, "
                                 f"got {inv_freq.numel()}")
            inv_freq = _need(inv_freq, "inv_freq", torch.float32, (rot // 2,), index)
        norms, norm_dtype = [None, None], 0
        for i, w in enumerate((q_norm, k_norm)):
            if w is not None:
                code = _DTYPES.get(w.dtype)
                if code is None or (norms[0] is not None and code != norm_dtype):
                    raise ValueError("q_norm and k_norm must share their type, float32 or bfloat16")
                norm_dtype = code
                norms[i] = _need(w, "k_norm" if i else "q_norm", w.dtype, (dim,), index)
        if out is None:
            out = torch.zeros(shape, dtype=torch.bfloat16, device=self.device)
        rc = load().spec_verify_cache_write_rotated(
            queries.data_ptr(), keys.data_ptr(), values.data_ptr(), dtype,
            _token_stride(queries, "queries", index), _token_stride(keys, "keys", index),
            _token_stride(values, "values", index), _need(slots, "slots", torch.int32, (B, T), index),
            _need(positions, "positions", torch.int32, (B, T), index), B * T, inv_freq, rot,
            1 if interleaved else 0, factor, norms[0], norms[1], norm_dtype, eps, heads,
            self.kv_heads, dim, self.page_size, self.num_pages, self._pool_ptr(),
            _need(out, "out", torch.bfloat16, shape, index),
            None if out_keys is None else _need(out_keys, "out_keys", torch.bfloat16, kv, index),
            None if status is None else _need(status, "status", torch.int32, (1,), index),
            _raw_stream(index))
        if rc != SV_OK:
            _check(rc, "spec_verify_cache_write_rotated")
        return out

    def read(self, page_table, starts, lens, length: int, dtype=torch.bfloat16, out=None,
             status=None, stream=None):
        """The keys and values [B, length, kv_heads, head_dim] of positions
        starts[b] .. starts[b] + lens[b] - 1 (starts None: 0). Rows behind
        lens[b] are left as ``out`` (a pair of tensors) holds them; fresh
        outputs are zero there."""
        index = self._index
        if stream is not None:
            with _other_stream(stream, index):
                return self.read(page_table, starts, lens, length, dtype, out, status)
        if _current_device() != index:
            with torch.cuda.device(index):
                return self.read(page_table, starts, lens, length, dtype, out, status)
        B, T = lens.shape[0], int(length)
        shape = (B, T, self.kv_heads, self.head_dim)
        table, width = self._table(page_table, B)
        if out is not None:
            dtype = out[0].dtype
        code = _DTYPES.get(dtype)
        if code is None:
            raise ValueError(f"values are read as float32 or bfloat16, not {dtype}")
        if out is None:
            out = tuple(torch.zeros(shape, dtype=dtype, device=self.device) for _ in range(2))
        rc = load().spec_verify_cache_read(
            self._pool_ptr(), table,
            None if starts is None else _need(starts, "starts", torch.int32, (B,), index),
            _need(lens, "lens", torch.int32, (B,), index), B, T, self.kv_heads, self.head_dim,
            self.page_size, width, self.num_pages, code,
            _need(out[0], "out keys", dtype, shape, index),
            _need(out[1], "out values", dtype, shape, index),
            None if status is None else _need(status, "status", torch.int32, (1,), index),
            _raw_stream(index))
        if rc != SV_OK:
            _check(rc, "spec_verify_cache_read")
        return out[0], out[1]

    def attend(self, queries, page_table, ctx_lens, budgets=None, scale: float | None = None,
               window: int = 0, out=None, status=None, stream=None, sinks: int = 0):
        """Attention of the blocks' rows, bfloat16 [B, K+1, q_heads, head_dim]
        (a slice of a fused projection's rows is fine), over the cache, which
        already holds the blocks' own tokens. ``scale`` None: head_dim ** -0.5.
        Under a ``window`` a row sees that many positions up to its own, and the
        first ``sinks`` ones.
        Rows behind budgets[b] and empty slots are left as ``out`` holds them;
        a fresh output is zero there."""
        index = self._index
        if stream is not None:
            with _other_stream(stream, index):
                return self.attend(queries, page_table, ctx_lens, budgets, scale, window, out,
                                   status, sinks=sinks)
        if _current_device() != index:
            with torch.cuda.device(index):
                return self.attend(queries, page_table, ctx_lens, budgets, scale, window, out,
                                   status, sinks=sinks)
        shape = queries.shape
        if len(shape) != 4 or queries.dtype is not torch.bfloat16 or shape[3] != self.head_dim \
                or shape[1] < 1:
            raise ValueError(f"queries must be bfloat16 [B, K+1, q_heads, {self.head_dim}]")
        if not 0 <= window <= 0x7fffffff:                   # ctypes would cut it to 32 bits
            raise ValueError(f"window must be 0..2^31 - 1, got {window}")
        B, T, heads, dim = shape
        stride = _token_stride(queries, "queries", index)
        table, width = self._table(page_table, B)
        if not 0 <= sinks <= 0x7fffffff:
            raise ValueError(f"sinks must be 0..2^31 - 1, got {sinks}")
        if sinks and window:
            nbytes = _sinks_bytes(max(B, 1), T - 1, heads, self.kv_heads, dim, self.page_size, width,
                                  window, sinks)
            call, seen = load().spec_verify_attention_sinks, (window, sinks)
        else:
            nbytes = _attention_bytes(max(B, 1), T - 1, heads, self.kv_heads, dim, self.page_size,
                                      width, window)
            call, seen = load().spec_verify_attention, (window,)
        if nbytes == 0:
            raise ValueError(f"bad attention shape: B={B} K={T - 1} q_heads={heads} kv_heads="
                             f"{self.kv_heads} window={window} max_pages={width}")
        if out is None:
            out = torch.zeros(shape, dtype=torch.bfloat16, device=self.device)
        workspace = self._no_parts if nbytes == 256 else torch.empty(
            nbytes, dtype=torch.uint8, device=self.device)
        rc = call(
            queries.data_ptr(), stride, self._pool_ptr(), table,
            _need(ctx_lens, "ctx_lens", torch.int32, (B,), index),
            None if budgets is None else _need(budgets, "budgets", torch.int32, (B,), index),
            B, T - 1, heads, self.kv_heads, dim, self.page_size, width, self.num_pages,
            dim ** -0.5 if scale is None else scale, *seen,
            _need(out, "out", torch.bfloat16, shape, index),
            None if status is None else _need(status, "status", torch.int32, (1,), index),
            workspace.data_ptr(), nbytes, _raw_stream(index))
        if rc != SV_OK:
            _check(rc, "spec_verify_attention")
        return out

    def attend_shared(self, queries, page_table, ctx_lens, groups, shared_lens, budgets=None,
                      scale: float | None = None, out=None, status=None, stream=None):
        """``attend`` (without a window) for requests that share a prefix:
        ``groups`` int32 [B], the group of every request (outside 0 .. G - 1:
        none), ``shared_lens`` int32 [G], the tokens from position 0 on that all
        requests of a group have in common. Their keys and values are read and
        multiplied once for all rows of the group, through the page table row of
        its first request. Pays from about 64 requests behind 2,000 tokens, or 32
        blocks behind 8,000, on; ``attend`` is faster below."""
        index = self._index
        if stream is not None:
            with _other_stream(stream, index):
                return self.attend_shared(queries, page_table, ctx_lens, groups, shared_lens,
                                          budgets, scale, out, status)
        if _current_device() != index:
            with torch.cuda.device(index):
                return self.attend_shared(queries, page_table, ctx_lens, groups, shared_lens,
                                          budgets, scale, out, status)
        shape = queries.shape
        if len(shape) != 4 or queries.dtype is not torch.bfloat16 or shape[3] != self.head_dim \
                or shape[1] < 1:
            raise ValueError(f"queries must be bfloat16 [B, K+1, q_heads, {self.head_dim}]")
        if shared_lens.dim() != 1 or shared_lens.shape[0] > SV_MAX_GROUPS:
            raise ValueError(f"shared_lens must be [G], G up to {SV_MAX_GROUPS}, got "
                             f"{tuple(shared_lens.shape)}")
        B, T, heads, dim = shape
        G = shared_lens.shape[0]
        stride = _token_stride(queries, "queries", index)
        table, width = self._table(page_table, B)
        nbytes = _shared_bytes(max(B, 1), T - 1, G, heads, self.kv_heads, dim, self.page_size, width)
        if nbytes == 0:
            raise ValueError(f"bad attention shape: B={B} K={T - 1} q_heads={heads} kv_heads="
                             f"{self.kv_heads} max_pages={width}")
        if out is None:
            out = torch.zeros(shape, dtype=torch.bfloat16, device=self.device)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        rc = load().spec_verify_attention_shared(
            queries.data_ptr(), stride, self._pool_ptr(), table,
            _need(ctx_lens, "ctx_lens", torch.int32, (B,), index),
            None if budgets is None else _need(budgets, "budgets", torch.int32, (B,), index),
            _need(groups, "groups", torch.int32, (B,), index),
            _need(shared_lens, "shared_lens", torch.int32, (G,), index),
            B, T - 1, G, heads, self.kv_heads, dim, self.page_size, width, self.num_pages,
            dim ** -0.5 if scale is None else scale,
            _need(out, "out", torch.bfloat16, shape, index),
            None if status is None else _need(status, "status", torch.int32, (1,), index),
            workspace.data_ptr(), nbytes, _raw_stream(index))
        if rc != SV_OK:
            _check(rc, "spec_verify_attention_shared")
        return out


class PageTables:
    """Which pages of a pool every slot of a batch holds: ``table`` (int32 [B,
    max_pages], -1 where there is none) and ``refs`` (int32 [num_pages], how many
    entries hold each page), both on the device and changed by ``plan`` only.
    One object serves the caches of all layers, whose pools it numbers alike.
    ``table`` and ``refs`` may be given to go on from a state of their own; a
    table alone has its pages counted. What is made here is ready on every stream.

    Calls are enqueued on ``stream`` (default: the current torch stream) and not
    waited for; ``status`` as in ``BlockCache``."""

    def __init__(self, device, B: int, max_pages: int, num_pages: int, page_size: int = 64,
                 table: torch.Tensor | None = None, refs: torch.Tensor | None = None):
        device = torch.device(device)
        if device.type != "cuda":
            raise ValueError("PageTables needs a GPU device")
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        self.device, self._index = device, device.index
        self.B, self.max_pages = int(B), int(max_pages)
        self.num_pages, self.page_size = int(num_pages), int(page_size)
        self._bytes = spec_verify_pages_plan_workspace_bytes(max(self.B, 1), max_pages, num_pages)
        if self._bytes == 0 or self.B < 0 or self.num_pages * self.page_size >= 1 << 31 \
                or spec_verify_cache_bytes(num_pages, 1, 64, page_size) == 0 \
                or self.max_pages * self.page_size > SV_MAX_CONTEXT:
            raise ValueError(f"bad page tables: {B} rows of {max_pages} pages out of {num_pages} "
                             f"of {page_size} tokens")
        self.table = torch.full((self.B, self.max_pages), -1, dtype=torch.int32, device=device) \
            if table is None else table
        self.refs = torch.zeros(self.num_pages, dtype=torch.int32, device=device) \
            if refs is None else refs
        self._state()
        if table is not None and refs is None:
            held = table[(table >= 0) & (table < self.num_pages)]
            self.refs.copy_(torch.bincount(held, minlength=self.num_pages))
        # For small tables, whose plan leaves its 256 bytes alone.
        self._unused = torch.empty(256, dtype=torch.uint8, device=device)
        if table is None or refs is None:
            _ready(self._index)

    def _state(self):
        return (_need(self.table, "table", torch.int32, (self.B, self.max_pages), self._index),
                _need(self.refs, "refs", torch.int32, (self.num_pages,), self._index))

    def plan(self, ctx_lens, budgets=None, length: int = 1, window: int = 0, sinks: int = 0,
             parents=None, prefix_lens=None, out=None, status=None, stream=None):
        """One step: gives back the pages that a request no longer needs for
        positions 0 .. ctx_lens[b] + budgets[b] (budgets None: length - 1; under a
        ``window`` the first ``sinks`` positions and those of the window), takes
        what is missing from the parent's row (whole pages of prefix_lens[b]
        tokens and in front of ctx_lens[b]; SV_FLAG_NO_PREFIX in ``status`` if that
        lacks one) or from the free pages. Returns
        (starts int32 [B]: ctx_lens, -1 where the request cannot run; slots int32
        [B, length] and positions int32 [B, length] of its tokens, -1 behind its
        budget)."""
        index = self._index
        if stream is not None:
            with _other_stream(stream, index):
                return self.plan(ctx_lens, budgets, length, window, sinks, parents, prefix_lens, out,
                                 status)
        if _current_device() != index:
            with torch.cuda.device(index):
                return self.plan(ctx_lens, budgets, length, window, sinks, parents, prefix_lens, out,
                                 status)
        B, T = self.B, int(length)
        if not 1 <= T <= SV_MAX_CONTEXT or not 0 <= window <= 0x7fffffff or not 0 <= sinks <= 0x7fffffff:
            raise ValueError(f"length must be 1..2^24, window and sinks 0..2^31 - 1, got {length}, "
                             f"{window}, {sinks}")
        if parents is not None and prefix_lens is None:
            raise ValueError("parents need prefix_lens")
        if out is None:
            device = self.device
            out = (torch.empty_strided((B,), (1,), dtype=torch.int32, device=device),
                   torch.empty_strided((B, T), (T, 1), dtype=torch.int32, device=device),
                   torch.empty_strided((B, T), (T, 1), dtype=torch.int32, device=device))
        workspace = self._unused if self._bytes == 256 else torch.empty_strided(
            (self._bytes,), (1,), dtype=torch.uint8, device=self.device)
        table, refs = self._state()
        rows = (B,)
        rc = load().spec_verify_pages_plan(
            table, refs, _need(ctx_lens, "ctx_lens", torch.int32, rows, index),
            None if budgets is None else _need(budgets, "budgets", torch.int32, rows, index),
            None if parents is None else _need(parents, "parents", torch.int32, rows, index),
            None if parents is None else _need(prefix_lens, "prefix_lens", torch.int32, rows, index),
            B, T, self.page_size, self.max_pages, self.num_pages, window, sinks,
            _need(out[0], "out starts", torch.int32, rows, index),
            _need(out[1], "out slots", torch.int32, (B, T), index),
            _need(out[2], "out positions", torch.int32, (B, T), index),
            None if status is None else _need(status, "status", torch.int32, (1,), index),
            workspace.data_ptr(), self._bytes, _raw_stream(index))
        if rc != SV_OK:
            _check(rc, "spec_verify_pages_plan")
        return out[0], out[1], out[2]


def head_quantize(x: torch.Tensor, block_rows: int = 1, out=None, stream=None):
    """Quantise float32 or bfloat16 [rows, H] (contiguous, on the GPU) to
    8 bits: (codes float8_e4m3fn [rows, Hp], scales float8_e8m0fnu
    [ceil(rows / block_rows), Hp / 128]), Hp = H rounded up to 128, zeros
    behind H. block_rows 1 for hidden states, 128 for a head."""
    index = x.get_device()
    code = _DTYPES.get(x.dtype)
    if code is None or index < 0 or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 or bfloat16 [rows, H] GPU tensor")
    if stream is not None:
        with _other_stream(stream, index):
            return head_quantize(x, block_rows, out)
    if _current_device() != index:
        with torch.cuda.device(index):
            return head_quantize(x, block_rows, out)
    if block_rows != 1 and block_rows != 128:
        raise ValueError("block_rows must be 1 or 128")
    rows, H = x.shape
    blocks = -(-H // 128)
    codes, scales = (rows, blocks * 128), (-(-rows // block_rows), blocks)
    if out is None:                     # empty_strided costs the host less than empty
        device = x.device
        out = (torch.empty_strided(codes, (blocks * 128, 1), dtype=torch.float8_e4m3fn, device=device),
               torch.empty_strided(scales, (blocks, 1), dtype=torch.float8_e8m0fnu, device=device))
    rc = load().spec_head_quantize(
        x.data_ptr(), code, rows, H, block_rows,
        _need(out[0], "out codes", torch.float8_e4m3fn, codes, index),
        _need(out[1], "out scales", torch.float8_e8m0fnu, scales, index), _raw_stream(index))
    if rc != SV_OK:
        _check(rc, "spec_head_quantize")
    return out[0], out[1]


def head_logits(h_codes: torch.Tensor, h_scales: torch.Tensor, w_codes: torch.Tensor,
                w_scales: torch.Tensor, dtype=torch.float32, out=None, stream=None):
    """Logits [R, V] (float32 or bfloat16) of quantised states (block_rows 1)
    under a quantised head (block_rows 128)."""
    index = h_codes.get_device()
    if index < 0:
        raise ValueError("h_codes must be a GPU tensor")
    if stream is not None:
        with _other_stream(stream, index):
            return head_logits(h_codes, h_scales, w_codes, w_scales, dtype, out)
    if _current_device() != index:
        with torch.cuda.device(index):
            return head_logits(h_codes, h_scales, w_codes, w_scales, dtype, out)
    h_shape, w_shape = h_codes.shape, w_codes.shape
    if len(h_shape) != 2 or len(w_shape) != 2 or h_shape[1] != w_shape[1] \
            or h_shape[1] % 128 != 0 or h_shape[1] == 0:
        raise ValueError("h_codes [R, Hp] and w_codes [V, Hp] must share Hp, a multiple of 128")
    R, H = h_shape
    V = w_shape[0]
    e4m3, e8m0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    if out is not None:
        dtype = out.dtype
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"logits are float32 or bfloat16, not {dtype}")
    if out is None:
        out = torch.empty_strided((R, V), (V, 1), dtype=dtype, device=h_codes.device)
    rc = load().spec_head_logits(
        _need(h_codes, "h_codes", e4m3, h_shape, index),
        _need(h_scales, "h_scales", e8m0, (R, H // 128), index),
        _need(w_codes, "w_codes", e4m3, w_shape, index),
        _need(w_scales, "w_scales", e8m0, (-(-V // 128), H // 128), index), R, H, V, code,
        _need(out, "out", dtype, (R, V), index), _raw_stream(index))
    if rc != SV_OK:
        _check(rc, "spec_head_logits")
    return out
