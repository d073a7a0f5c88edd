"""ctypes binding of libdspark (include/dspark.h).

Argument marshalling only: every step of the hot path runs in the library's
CUDA kernels.  The low-level functions carry the C names (``dspark_*``) and
take torch tensors (device memory, caller-owned) plus an optional CUDA
stream; the convenience wrappers below them allocate the outputs.  There is no
CPU fallback: if the compiled library is missing, loading raises.
"""

from __future__ import annotations

import ctypes
import os
from array import array
from dataclasses import dataclass
from operator import attrgetter
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libdspark.so")
# the same library with the draft kernel's device-side offset checks compiled in
DEBUG_LIB_PATH = os.path.join(_HERE, "_build", "libdspark_debug.so")

STATUS = {
    0: "DSPARK_OK", 1: "DSPARK_ERR_INVALID_ARG", 2: "DSPARK_ERR_UNSUPPORTED",
    3: "DSPARK_ERR_CUDA", 4: "DSPARK_ERR_TIMEOUT", 5: "DSPARK_ERR_DEVICE_OOB",
    6: "DSPARK_ERR_NO_DEVICE", 7: "DSPARK_ERR_CTX_POISONED", 8: "DSPARK_ERR_CAPACITY",
}
OK, INVALID_ARG, UNSUPPORTED, CUDA, TIMEOUT, DEVICE_OOB, NO_DEVICE, POISONED, CAPACITY = range(9)

# Functions declared in include/dspark.h (checked against the header by the tests).
EXPORTS = (
    "dspark_ctx_create", "dspark_ctx_destroy", "dspark_ctx_reset", "dspark_get_status",
    "dspark_debug_set", "dspark_debug_refuse_next_launch", "dspark_debug_trace", "dspark_strerror",
    "dspark_abi_version", "dspark_last_launch_count",
    "dspark_markov_draft", "dspark_gated_draft", "dspark_gate", "dspark_selector_scores",
    "dspark_selector_walk", "dspark_confidence", "dspark_markov_logits",
    "dspark_markov_draft_noalloc", "dspark_verify", "dspark_schedule", "dspark_accept_label",
    "dspark_sts_fit", "dspark_rnn_draft", "dspark_rnn_logits", "dspark_verify_probs",
    "dspark_distill", "dspark_rnn_scan", "dspark_rnn_scan_grad", "dspark_embed",
    "dspark_embed_grad", "dspark_clip_grads", "dspark_linear", "dspark_linear_grad",
)


class DSparkError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)} ({strerror(code)})")


class ConfArgs(ctypes.Structure):
    _fields_ = [
        ("h", ctypes.c_void_p), ("w", ctypes.c_void_p), ("bias", ctypes.c_float),
        ("d", ctypes.c_int), ("with_markov", ctypes.c_int), ("threshold", ctypes.c_float),
        ("conf", ctypes.c_void_p), ("cumprod", ctypes.c_void_p), ("verify_len", ctypes.c_void_p),
        ("tau", ctypes.c_void_p),
    ]


_libs = {}


def load(path: str = LIB_PATH):
    """Load libdspark.so (or its checked twin); raise if it has not been built."""
    if path in _libs:
        return _libs[path]
    if not os.path.exists(path):
        raise RuntimeError(f"{os.path.basename(path)} not found at {path}: build it first "
                           "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    P, I, F, U64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_uint64
    I64 = ctypes.c_int64
    sig = {
        "dspark_ctx_create": [ctypes.POINTER(P), I, I, I, I],
        "dspark_ctx_destroy": [P],
        "dspark_ctx_reset": [P, P],
        "dspark_get_status": [P, ctypes.POINTER(I)],
        "dspark_debug_set": [P, I, I],
        "dspark_debug_refuse_next_launch": [P],
        "dspark_debug_trace": [P, P, ctypes.c_int64],
        "dspark_strerror": [I],
        "dspark_abi_version": [],
        "dspark_last_launch_count": [P],
        "dspark_markov_draft": [P, P, P, P, P, I, I, I, I, F, U64, P, P, P, P],
        "dspark_gated_draft": [P, P, P, P, P, P, P, I, I, I, I, I, F, U64, P, P, P, P],
        "dspark_gate": [P, P, P, I, I, I, P, P],
        "dspark_selector_scores": [P, P, P, P, P, P, P, I, I, I, I, I, I, P, P, P, P],
        "dspark_selector_walk": [P, P, P, P, P, I, I, I, I, I, F, U64, P, P, P, P],
        "dspark_confidence": [P, P, P, P, P, P, F, I, I, I, I, I, I, F, P, P, P, P, P],
        "dspark_markov_logits": [P, P, P, P, P, P, P, I, I, I, I, I, F, P, P, P],
        "dspark_markov_draft_noalloc": [P, P, P, P, I, I, I, I, F, U64, P, P, P, P],
        "dspark_verify": [P, P, P, P, P, P, P, P, I, P, P, P, I, I, I, I, F, F, U64, P, P, P, P],
        "dspark_schedule": [P, P, I, I, P, I, P, P, P],
        "dspark_accept_label": [P, P, P, P, P, P, P, P, I, P, P, I, I, I, I, F, F, P, P],
        "dspark_sts_fit": [P, P, P, I, I, F, F, P, P, P],
        "dspark_rnn_draft": [P, P, P, P, P, P, P, P, I, I, I, I, I, F, U64, P, P, P, P],
        "dspark_rnn_logits": [P, P, P, P, P, P, P, P, I, I, I, I, I, F, P, P, P],
        "dspark_verify_probs": [P, P, P, P, P, I, P, P, P, P, I, I, I, P, P, P, P],
        "dspark_distill": [P, P, I, I64, P, P, I, P, P, I64, I, F, F, F, P, P, P, I64, P],
        "dspark_rnn_scan": [P, P, P, P, I, I64, I64, I64, P, P, I64, I64, I, P, P, P],
        "dspark_rnn_scan_grad": [P, P, P, P, P, P, I, I64, I64, I64, P, P, P, I64, I64, I, P, P,
                                 I64, I64, P, P, P],
        "dspark_embed": [P, P, I, I64, P, I64, I, I, F, P, I, I64, P],
        "dspark_embed_grad": [P, P, P, I, I64, I64, I, I, F, I, P, I, I64, P],
        "dspark_clip_grads": [P, P, P, P, I, F, P, P, P],
        "dspark_linear": [P, P, I64, P, I64, P, I, P, I, I64, I64, I, I, P, I, I64, P, I64, P,
                          ctypes.POINTER(I64), P],
        "dspark_linear_grad": [P, P, I64, P, I64, P, I, I64, I, P, I, I64, I64, I, I, P, I, I64, P,
                               I, I64, P, P, ctypes.POINTER(I64), P],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_char_p if name == "dspark_strerror" else ctypes.c_int
    _libs[path] = lib
    return lib


def strerror(code: int) -> str:
    try:
        return load().dspark_strerror(int(code)).decode()
    except RuntimeError:
        return "library not loaded"


# ----------------------------------------------------------------- marshalling
_BF16 = (torch.bfloat16, torch.int16, torch.uint16)


def _ptr(t: Optional[torch.Tensor], dtypes=None, name: str = "tensor"):
    """Address of a contiguous CUDA tensor (None passes through)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name}: must live in CUDA device memory")
    return t.data_ptr()


def _rows(t: Optional[torch.Tensor], dtype, name: str):
    """Address and row distance (elements) of a [..., D] tensor whose last dimension is
    contiguous and whose rows are evenly spaced (a slice of a wider contiguous tensor)."""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype} is not {dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must live in CUDA device memory")
    if t.is_contiguous() and t.dim() > 0:
        return t.data_ptr(), t.shape[-1]
    shape, strides = t.shape, t.stride()
    if t.dim() == 0 or (shape[-1] > 1 and strides[-1] != 1):
        raise ValueError(f"{name}: the last dimension must be contiguous")
    ld = step = None
    for i in range(len(shape) - 2, -1, -1):
        if shape[i] == 1:
            continue
        if ld is None:
            ld = strides[i]
        elif strides[i] != step:
            raise ValueError(f"{name}: rows must be evenly spaced")
        step = strides[i] * shape[i]
    return t.data_ptr(), shape[-1] if ld is None else ld


_DTYPE = {torch.float32: 0, torch.bfloat16: 1}  # dspark_dtype


def _dtype(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype not in _DTYPE:
        raise TypeError(f"{name}: dtype {t.dtype} not in {tuple(_DTYPE)}")
    return _DTYPE[t.dtype]


_ACT = {None: 0, "sigmoid": 1, "tanh": 2, "relu": 3, "silu": 4, "gelu": 5}  # dspark_act


def _act(name) -> int:
    if name not in _ACT:
        raise ValueError(f"act: {name!r} not in {tuple(_ACT)}")
    return _ACT[name]


def _shape(t: Optional[torch.Tensor], shape, name: str):
    if t is not None and t.shape != shape:  # (a torch.Size is a tuple)
        raise ValueError(f"{name}: shape {tuple(t.shape)} is not {tuple(shape)}")


# The handle that torch.cuda.current_stream(device).cuda_stream gives, without making the object
# (some 1 us a call); a torch without this call makes it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream(stream, device):
    if stream is None:
        index = device if isinstance(device, int) else device.index
        if index is None:
            index = torch.cuda.current_device()
        return _raw_stream(index)
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _empty(stream, shape, dtype, device, returned=True):
    """A tensor for a call's work on `stream` (None: the current one), of memory that was last used
    there: what torch's allocator hands out for another stream may still be in use by work queued on
    that one, which the call's does not wait for.  The caller's current stream, which may read what is
    `returned`, is recorded, so that the memory goes back when its work so far is done too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _check(code: int, where: str):
    if code != OK:
        raise DSparkError(code, where)


class Context:
    """A dspark_ctx: per-device scratch for B_max requests, K_max positions, V_max tokens."""

    def __init__(self, device: int = 0, B_max: int = 128, V_max: int = 151936, K_max: int = 16,
                 checked: bool = False):
        # checked: run through libdspark_debug.so, whose draft kernel checks its on-chip
        # offsets (a failed check is reported as DSPARK_ERR_DEVICE_OOB)
        self.lib = load(DEBUG_LIB_PATH if checked else LIB_PATH)
        self.device = device
        self.B_max, self.V_max, self.K_max = B_max, V_max, K_max
        h = ctypes.c_void_p()
        _check(self.lib.dspark_ctx_create(ctypes.byref(h), device, B_max, V_max, K_max),
               "dspark_ctx_create")
        self.handle = h

    def close(self):
        if getattr(self, "handle", None):
            torch.cuda.synchronize(self.device)
            self.lib.dspark_ctx_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def reset(self, stream=None):
        _check(self.lib.dspark_ctx_reset(self.handle, _stream(stream, self.device)),
               "dspark_ctx_reset")

    def status(self) -> int:
        v = ctypes.c_int(0)
        _check(self.lib.dspark_get_status(self.handle, ctypes.byref(v)), "dspark_get_status")
        return v.value

    def debug_set(self, cta: int = -1, timeout_ms: int = 0):
        _check(self.lib.dspark_debug_set(self.handle, cta, timeout_ms), "dspark_debug_set")

    def refuse_next_launch(self):
        """The next draft or long-row distillation launch is refused by the CUDA runtime (a test
        aid)."""
        _check(self.lib.dspark_debug_refuse_next_launch(self.handle),
               "dspark_debug_refuse_next_launch")

    def trace_next(self, buf: Optional[torch.Tensor]):
        """Record the next draft launch's phase stamps into buf (int64, >= grid * K * 8)."""
        if buf is None:
            _check(self.lib.dspark_debug_trace(self.handle, None, 0), "dspark_debug_trace")
            return
        _check(self.lib.dspark_debug_trace(self.handle, _ptr(buf, (torch.int64,), "trace"),
                                           buf.numel()), "dspark_debug_trace")

    @property
    def last_launches(self) -> int:
        return int(self.lib.dspark_last_launch_count(self.handle))


@dataclass
class Confidence:
    """Inputs and outputs of the confidence head (dspark_conf_args)."""
    h: torch.Tensor            # [B, K, d] bf16
    w: torch.Tensor            # [d + r] (with_markov) or [d] bf16
    bias: float = 0.0
    with_markov: bool = True
    threshold: float = 0.3
    conf: Optional[torch.Tensor] = None       # out [B, K] fp32
    cumprod: Optional[torch.Tensor] = None    # out [B, K] fp32
    verify_len: Optional[torch.Tensor] = None  # out [B] int32
    tau: Optional[torch.Tensor] = None         # [K] fp32 STS temperatures (None: all 1)

    def allocate(self, B: int, K: int, stream=None):
        dev = self.h.device
        if self.conf is None:
            self.conf = _empty(stream, (B, K), torch.float32, dev)
        if self.cumprod is None:
            self.cumprod = _empty(stream, (B, K), torch.float32, dev)
        if self.verify_len is None:
            self.verify_len = _empty(stream, (B,), torch.int32, dev)
        return self

    def struct(self) -> ConfArgs:
        return ConfArgs(_ptr(self.h, _BF16, "conf.h"), _ptr(self.w, _BF16, "conf.w"),
                        float(self.bias), int(self.h.shape[-1]), int(bool(self.with_markov)),
                        float(self.threshold), _ptr(self.conf, (torch.float32,), "conf.conf"),
                        _ptr(self.cumprod, (torch.float32,), "conf.cumprod"),
                        _ptr(self.verify_len, (torch.int32,), "conf.verify_len"),
                        _ptr(self.tau, (torch.float32,), "conf.tau"))


def _conf_ref(conf: Optional[Confidence]):
    return None if conf is None else ctypes.byref(conf.struct())


# ------------------------------------------------------- C-named entry points
def dspark_markov_draft(ctx: Context, U, W1, W2, anchors, B, K, V, r, temperature, seed,
                        tokens, logprobs, conf: Optional[Confidence] = None, stream=None):
    code = ctx.lib.dspark_markov_draft(
        ctx.handle, _ptr(U, (torch.float32,), "U"), _ptr(W1, _BF16, "W1"),
        _ptr(W2, _BF16, "W2"), _ptr(anchors, (torch.int32,), "anchors"), B, K, V, r,
        float(temperature), int(seed) & (2 ** 64 - 1), _ptr(tokens, (torch.int32,), "tokens"),
        _ptr(logprobs, (torch.float32,), "logprobs"), _conf_ref(conf), _stream(stream, ctx.device))
    _check(code, "dspark_markov_draft")


def dspark_gated_draft(ctx: Context, U, W1, W2, anchors, h, Wg, d, B, K, V, r, temperature,
                       seed, tokens, logprobs, conf: Optional[Confidence] = None, stream=None):
    code = ctx.lib.dspark_gated_draft(
        ctx.handle, _ptr(U, (torch.float32,), "U"), _ptr(W1, _BF16, "W1"),
        _ptr(W2, _BF16, "W2"), _ptr(anchors, (torch.int32,), "anchors"), _ptr(h, _BF16, "h"),
        _ptr(Wg, _BF16, "Wg"), d, B, K, V, r, float(temperature), int(seed) & (2 ** 64 - 1),
        _ptr(tokens, (torch.int32,), "tokens"), _ptr(logprobs, (torch.float32,), "logprobs"),
        _conf_ref(conf), _stream(stream, ctx.device))
    _check(code, "dspark_gated_draft")


def dspark_rnn_draft(ctx: Context, U, W1, W2, anchors, h, Wa, Wg, d, B, K, V, r, temperature,
                     seed, tokens, logprobs, conf: Optional[Confidence] = None, stream=None):
    code = ctx.lib.dspark_rnn_draft(
        ctx.handle, _ptr(U, (torch.float32,), "U"), _ptr(W1, _BF16, "W1"),
        _ptr(W2, _BF16, "W2"), _ptr(anchors, (torch.int32,), "anchors"), _ptr(h, _BF16, "h"),
        _ptr(Wa, _BF16, "Wa"), _ptr(Wg, _BF16, "Wg"), d, B, K, V, r, float(temperature),
        int(seed) & (2 ** 64 - 1), _ptr(tokens, (torch.int32,), "tokens"),
        _ptr(logprobs, (torch.float32,), "logprobs"), _conf_ref(conf), _stream(stream, ctx.device))
    _check(code, "dspark_rnn_draft")


def dspark_rnn_logits(ctx: Context, U, W1, W2, prev_tokens, h, Wa, Wg, d, B, K, V, r, temperature,
                      logits, lse, stream=None):
    code = ctx.lib.dspark_rnn_logits(
        ctx.handle, _ptr(U, (torch.float32,), "U"), _ptr(W1, _BF16, "W1"), _ptr(W2, _BF16, "W2"),
        _ptr(prev_tokens, (torch.int32,), "prev_tokens"), _ptr(h, _BF16, "h"),
        _ptr(Wa, _BF16, "Wa"), _ptr(Wg, _BF16, "Wg"), d, B, K, V, r, float(temperature),
        _ptr(logits, (torch.float32,), "logits"), _ptr(lse, (torch.float32,), "lse"),
        _stream(stream, ctx.device))
    _check(code, "dspark_rnn_logits")


def dspark_gate(ctx: Context, h, Wg, M, d, r, H, stream=None):
    code = ctx.lib.dspark_gate(ctx.handle, _ptr(h, _BF16, "h"), _ptr(Wg, _BF16, "Wg"), M, d, r,
                               _ptr(H, (torch.float32,), "H"), _stream(stream, ctx.device))
    _check(code, "dspark_gate")


def dspark_selector_scores(ctx: Context, U, A, Bt, anchors, h, Wg, d, B, K, V, r, topk, cand,
                           cand_U, scores, stream=None):
    code = ctx.lib.dspark_selector_scores(
        ctx.handle, _ptr(U, (torch.float32,), "U"), _ptr(A, _BF16, "A"), _ptr(Bt, _BF16, "Bt"),
        _ptr(anchors, (torch.int32,), "anchors"), _ptr(h, _BF16, "h"), _ptr(Wg, _BF16, "Wg"), d,
        B, K, V, r, topk, _ptr(cand, (torch.int32,), "cand"),
        _ptr(cand_U, (torch.float32,), "cand_U"), _ptr(scores, (torch.float32,), "scores"),
        _stream(stream, ctx.device))
    _check(code, "dspark_selector_scores")


def dspark_selector_walk(ctx: Context, cand, scores, anchors, A, B, K, V, r, topk, temperature,
                         seed, tokens, logprobs, conf: Optional[Confidence] = None, stream=None):
    code = ctx.lib.dspark_selector_walk(
        ctx.handle, _ptr(cand, (torch.int32,), "cand"), _ptr(scores, (torch.float32,), "scores"),
        _ptr(anchors, (torch.int32,), "anchors"), _ptr(A, _BF16, "A"), B, K, V, r, topk,
        float(temperature), int(seed) & (2 ** 64 - 1), _ptr(tokens, (torch.int32,), "tokens"),
        _ptr(logprobs, (torch.float32,), "logprobs"), _conf_ref(conf), _stream(stream, ctx.device))
    _check(code, "dspark_selector_walk")


def dspark_confidence(ctx: Context, h, W1, anchors, tokens, w, bias, with_markov, B, K, d, r, V,
                      threshold, tau, conf, cumprod, verify_len, stream=None):
    code = ctx.lib.dspark_confidence(
        ctx.handle, _ptr(h, _BF16, "h"), _ptr(W1, _BF16, "W1"),
        _ptr(anchors, (torch.int32,), "anchors"), _ptr(tokens, (torch.int32,), "tokens"),
        _ptr(w, _BF16, "w"), float(bias), int(bool(with_markov)), B, K, d, r, V, float(threshold),
        _ptr(tau, (torch.float32,), "tau"), _ptr(conf, (torch.float32,), "conf"), _ptr(cumprod, (torch.float32,), "cumprod"),
        _ptr(verify_len, (torch.int32,), "verify_len"), _stream(stream, ctx.device))
    _check(code, "dspark_confidence")


def dspark_markov_logits(ctx: Context, U, W1, W2, prev_tokens, h, Wg, d, B, K, V, r,
                         temperature, logits, lse, stream=None):
    code = ctx.lib.dspark_markov_logits(
        ctx.handle, _ptr(U, (torch.float32,), "U"), _ptr(W1, _BF16, "W1"), _ptr(W2, _BF16, "W2"),
        _ptr(prev_tokens, (torch.int32,), "prev_tokens"), _ptr(h, _BF16, "h"),
        _ptr(Wg, _BF16, "Wg"), d, B, K, V, r, float(temperature),
        _ptr(logits, (torch.float32,), "logits"), _ptr(lse, (torch.float32,), "lse"),
        _stream(stream, ctx.device))
    _check(code, "dspark_markov_logits")


def dspark_verify(ctx: Context, P, U, W1, W2, anchors, h, Wg, d, tokens, draft_logprobs, ell,
                  B, K, V, r, draft_temperature, target_temperature, seed, n_acc, next_token,
                  accept_prob, stream=None):
    code = ctx.lib.dspark_verify(
        ctx.handle, _ptr(P, (torch.float32,), "P"), _ptr(U, (torch.float32,), "U"),
        _ptr(W1, _BF16, "W1"), _ptr(W2, _BF16, "W2"), _ptr(anchors, (torch.int32,), "anchors"),
        _ptr(h, _BF16, "h"), _ptr(Wg, _BF16, "Wg"), d, _ptr(tokens, (torch.int32,), "tokens"),
        _ptr(draft_logprobs, (torch.float32,), "draft_logprobs"), _ptr(ell, (torch.int32,), "ell"),
        B, K, V, r, float(draft_temperature), float(target_temperature), int(seed) & (2 ** 64 - 1),
        _ptr(n_acc, (torch.int32,), "n_acc"), _ptr(next_token, (torch.int32,), "next_token"),
        _ptr(accept_prob, (torch.float32,), "accept_prob"), _stream(stream, ctx.device))
    _check(code, "dspark_verify")


def dspark_accept_label(ctx: Context, P, U, W1, W2, anchors, h, Wg, d, tokens, draft_logprobs,
                        B, K, V, r, draft_temperature, target_temperature, label, stream=None):
    code = ctx.lib.dspark_accept_label(
        ctx.handle, _ptr(P, (torch.float32,), "P"), _ptr(U, (torch.float32,), "U"),
        _ptr(W1, _BF16, "W1"), _ptr(W2, _BF16, "W2"), _ptr(anchors, (torch.int32,), "anchors"),
        _ptr(h, _BF16, "h"), _ptr(Wg, _BF16, "Wg"), d, _ptr(tokens, (torch.int32,), "tokens"),
        _ptr(draft_logprobs, (torch.float32,), "draft_logprobs"), B, K, V, r,
        float(draft_temperature), float(target_temperature), _ptr(label, (torch.float32,), "label"),
        _stream(stream, ctx.device))
    _check(code, "dspark_accept_label")


def dspark_sts_fit(ctx: Context, conf, label, N, K, tau_lo, tau_hi, tau, loss, stream=None):
    code = ctx.lib.dspark_sts_fit(
        ctx.handle, _ptr(conf, (torch.float32,), "conf"), _ptr(label, (torch.float32,), "label"),
        N, K, float(tau_lo), float(tau_hi), _ptr(tau, (torch.float32,), "tau"),
        _ptr(loss, (torch.float32,), "loss"), _stream(stream, ctx.device))
    _check(code, "dspark_sts_fit")


def dspark_schedule(ctx: Context, a, R, K, sps, ell, theta, stream=None):
    code = ctx.lib.dspark_schedule(
        ctx.handle, _ptr(a, (torch.float32,), "a"), R, K, _ptr(sps, (torch.float32,), "sps"),
        int(sps.numel()), _ptr(ell, (torch.int32,), "ell"), _ptr(theta, (torch.float32,), "theta"),
        _stream(stream, ctx.device))
    _check(code, "dspark_schedule")


def dspark_verify_probs(ctx: Context, P, Q, cand, cand_q, m, tokens, u_accept, u_draw, ell, B, K,
                        V, n_acc, next_token, accept_prob, stream=None):
    f32, i32 = (torch.float32,), (torch.int32,)
    code = ctx.lib.dspark_verify_probs(
        ctx.handle, _ptr(P, f32, "P"), _ptr(Q, f32, "Q"), _ptr(cand, i32, "cand"),
        _ptr(cand_q, f32, "cand_q"), m, _ptr(tokens, i32, "tokens"),
        _ptr(u_accept, f32, "u_accept"), _ptr(u_draw, f32, "u_draw"), _ptr(ell, i32, "ell"), B, K,
        V, _ptr(n_acc, i32, "n_acc"), _ptr(next_token, i32, "next_token"),
        _ptr(accept_prob, f32, "accept_prob"), _stream(stream, ctx.device))
    _check(code, "dspark_verify_probs")


def dspark_distill(ctx: Context, logits, teacher_ids, teacher_logits, k, teacher_rest, row_weight,
                   N, V, temperature, alpha_kl, alpha_tv, loss, tv, grad, stream=None):
    f32 = (torch.float32,)
    dtype = _dtype(logits, "logits")
    p, ld = _rows(logits, logits.dtype, "logits")
    pg, ld_grad = _rows(grad, logits.dtype, "grad")
    code = ctx.lib.dspark_distill(
        ctx.handle, p, dtype, ld, _ptr(teacher_ids, (torch.int32,), "teacher_ids"),
        _ptr(teacher_logits, f32, "teacher_logits"), k, _ptr(teacher_rest, f32, "teacher_rest"),
        _ptr(row_weight, f32, "row_weight"), N, V, float(temperature), float(alpha_kl),
        float(alpha_tv), _ptr(loss, f32, "loss"), _ptr(tv, f32, "tv"), pg, ld_grad,
        _stream(stream, ctx.device))
    _check(code, "dspark_distill")


def dspark_rnn_scan(ctx: Context, za, zg, e, s0, reset, N, L, D, s, s_last, stream=None):
    f32 = (torch.float32,)
    dtype = _dtype(e, "e")
    pa, ld_za = _rows(za, e.dtype, "za")
    pg, ld_zg = _rows(zg, e.dtype, "zg")
    pe, ld_e = _rows(e, e.dtype, "e")
    code = ctx.lib.dspark_rnn_scan(
        ctx.handle, pa, pg, pe, dtype, ld_za, ld_zg, ld_e, _ptr(s0, f32, "s0"),
        _ptr(reset, (torch.uint8, torch.bool), "reset"), N, L, D, _ptr(s, (e.dtype,), "s"),
        _ptr(s_last, f32, "s_last"), _stream(stream, ctx.device))
    _check(code, "dspark_rnn_scan")


def dspark_rnn_scan_grad(ctx: Context, za, zg, e, s, ds, s0, reset, ds_last, N, L, D, dza, dzg, de,
                         ds0, stream=None):
    f32 = (torch.float32,)
    dtype = _dtype(e, "e")
    pa, ld_za = _rows(za, e.dtype, "za")
    pg, ld_zg = _rows(zg, e.dtype, "zg")
    pe, ld_e = _rows(e, e.dtype, "e")
    pda, ld_dza = _rows(dza, e.dtype, "dza")
    pdg, ld_dzg = _rows(dzg, e.dtype, "dzg")
    code = ctx.lib.dspark_rnn_scan_grad(
        ctx.handle, pa, pg, pe, _ptr(s, (e.dtype,), "s"), _ptr(ds, (e.dtype,), "ds"), dtype, ld_za,
        ld_zg, ld_e, _ptr(s0, f32, "s0"), _ptr(reset, (torch.uint8, torch.bool), "reset"),
        _ptr(ds_last, f32, "ds_last"), N, L, D, pda, pdg, ld_dza, ld_dzg,
        _ptr(de, (e.dtype,), "de"), _ptr(ds0, f32, "ds0"), _stream(stream, ctx.device))
    _check(code, "dspark_rnn_scan_grad")


def dspark_embed(ctx: Context, table, ids, N, V, D, scale, out, stream=None):
    p, ld = _rows(table, table.dtype, "table")
    po, ldo = _rows(out, out.dtype, "out")
    code = ctx.lib.dspark_embed(
        ctx.handle, p, _dtype(table, "table"), ld, _ptr(ids, (torch.int32,), "ids"), N, V, D,
        float(scale), po, _dtype(out, "out"), ldo, _stream(stream, ctx.device))
    _check(code, "dspark_embed")


def dspark_embed_grad(ctx: Context, ids, de, N, V, D, scale, accumulate, grad, stream=None):
    p, ld = _rows(de, de.dtype, "de")
    pg, ldg = _rows(grad, grad.dtype, "grad")
    code = ctx.lib.dspark_embed_grad(
        ctx.handle, _ptr(ids, (torch.int32,), "ids"), p, _dtype(de, "de"), ld, N, V, D,
        float(scale), int(bool(accumulate)), pg, _dtype(grad, "grad"), ldg,
        _stream(stream, ctx.device))
    _check(code, "dspark_embed_grad")


def _tensor_list(ts, name: str):
    """Addresses, element counts and dtypes of a list of contiguous CUDA tensors, for C."""
    try:
        dtypes = list(map(_DTYPE.get, map(attrgetter("dtype"), ts)))
        contiguous = all(map(torch.Tensor.is_contiguous, ts))
        pointers, numel = list(map(torch.Tensor.data_ptr, ts)), list(map(torch.Tensor.numel, ts))
    except (AttributeError, TypeError):
        raise TypeError(f"{name}: expected torch.Tensors") from None
    if None in dtypes:
        raise TypeError(f"{name}: dtype {ts[dtypes.index(None)].dtype} not in {tuple(_DTYPE)}")
    if not contiguous:
        raise ValueError(f"{name}: must be contiguous")
    if not all(map(attrgetter("is_cuda"), ts)):
        raise ValueError(f"{name}: must live in CUDA device memory")
    return array("Q", pointers), array("q", numel), array("i", dtypes)


def _each_once(pointers, numel, name: str):
    """No tensor (that has elements) is listed twice: both of its places would scale it at one time."""
    if len(set(pointers)) != len(pointers):
        used = [p for p, n in zip(pointers, numel) if n > 0]
        if len(set(used)) != len(used):
            raise ValueError(f"{name}: the same tensor twice")


def dspark_clip_grads(ctx: Context, grads, max_norm, out, norm, stream=None):
    """grads and out: lists of contiguous tensors (out None: only the norm)."""
    src, numel, dtypes = _tensor_list(grads, "grads")
    dst = None
    if out is grads:
        dst = src
    elif out is not None:
        dst, n, dt = _tensor_list(out, "out")
        if n != numel or dt != dtypes:
            raise ValueError("out: other sizes or types than the gradients'")
    if dst is not None:
        _each_once(dst, numel, "grads" if out is grads else "out")
    address = lambda a: None if a is None else a.buffer_info()[0]  # noqa: E731
    code = ctx.lib.dspark_clip_grads(ctx.handle, address(src), address(numel), address(dtypes),
                                     len(src), float(max_norm), address(dst),
                                     _ptr(norm, (torch.float32,), "norm"),
                                     _stream(stream, ctx.device))
    _check(code, "dspark_clip_grads")


def _with_workspace(call, workspace, likely: int, device, stream, where: str):
    """call(address, bytes) -> status.  Without a workspace of the caller's, `likely` bytes of one (0:
    none) or what the call then asks for come from torch's allocator, for the call's stream alone."""
    given = workspace is not None
    if not given and likely > 0:
        workspace = _empty(stream, (likely,), torch.uint8, device, returned=False)
    size = ctypes.c_int64(0 if workspace is None else workspace.numel() * workspace.element_size())
    code = call(_ptr(workspace, None, "workspace"), ctypes.byref(size))
    if code == CAPACITY and not given:
        workspace = _empty(stream, (size.value,), torch.uint8, device, returned=False)
        code = call(workspace.data_ptr(), ctypes.byref(size))
    _check(code, where)


def _copy_bytes(rows: int, cols: int) -> int:
    """Of a bf16 matrix with rows on 16-byte boundaries, as the linear layers copy one."""
    return (rows * ((cols + 7) & ~7) * 2 + 255) & ~255


def dspark_linear(ctx: Context, x, W, bias, act, residual, M, K, N, y, pre, workspace=None,
                  stream=None):
    """workspace None: allocated where the call needs one."""
    px, ld_x = _rows(x, torch.bfloat16, "x")
    pw, ld_w = _rows(W, torch.bfloat16, "W")
    dtype = _dtype(y, "y")
    py, ld_y = _rows(y, y.dtype, "y")
    pp, ld_pre = _rows(pre, y.dtype, "pre")
    pr, ld_r, rdt = None, 0, 0
    if residual is not None:
        rdt = _dtype(residual, "residual")
        pr, ld_r = _rows(residual, residual.dtype, "residual")
    pb, a, s = _ptr(bias, (torch.float32,), "bias"), _act(act), _stream(stream, ctx.device)
    likely = 0
    if (px or 0) & 15 or ld_x & 7:
        likely += _copy_bytes(M, K)
    if (pw or 0) & 15 or ld_w & 7:
        likely += _copy_bytes(K, N)
    _with_workspace(
        lambda p, size: ctx.lib.dspark_linear(ctx.handle, px, ld_x, pw, ld_w, pb, a, pr, rdt, ld_r,
                                              M, K, N, py, dtype, ld_y, pp, ld_pre, p, size, s),
        workspace, likely, x.device, stream, "dspark_linear")


def dspark_linear_grad(ctx: Context, x, W, dy, act, pre, M, K, N, dx, dW, dbias, workspace=None,
                       stream=None):
    """workspace None: allocated where the call needs one."""
    px, ld_x = _rows(x, torch.bfloat16, "x")
    pw, ld_w = _rows(W, torch.bfloat16, "W")
    ydt = _dtype(dy, "dy")
    py, ld_dy = _rows(dy, dy.dtype, "dy")
    rows = []
    for t, name in ((pre, "pre"), (dx, "dx"), (dW, "dW")):
        if t is None:
            rows.append((None, 0, 0))
        else:
            dt = _dtype(t, name)
            rows.append((*_rows(t, t.dtype, name), dt))
    (pp, ld_p, pdt), (pdx, ld_dx, xdt), (pdw, ld_dw, wdt) = rows
    pb, a, s = _ptr(dbias, (torch.float32,), "dbias"), _act(act), _stream(stream, ctx.device)
    likely = 0
    if dW is not None and ((px or 0) & 15 or ld_x & 7):
        likely += _copy_bytes(M, K)
    if dx is not None and ((pw or 0) & 15 or ld_w & 7):
        likely += _copy_bytes(K, N)
    if (dx is not None or dW is not None) and (a or ydt == 0 or (py or 0) & 15 or ld_dy & 7):
        likely += (1 if not a and ydt else 3) * _copy_bytes(M, N)
    _with_workspace(
        lambda p, size: ctx.lib.dspark_linear_grad(
            ctx.handle, px, ld_x, pw, ld_w, py, ydt, ld_dy, a, pp, pdt, ld_p, M, K, N, pdx, xdt,
            ld_dx, pdw, wdt, ld_dw, pb, p, size, s),
        workspace, likely, dy.device, stream, "dspark_linear_grad")


def dspark_markov_draft_noalloc(U, W1, W2, anchors, B, K, V, r, temperature, seed, tokens,
                                logprobs, device_status=None, stream=None):
    """Context-free draft that allocates no device memory (scratch compiled into the library).

    For callers that may not allocate device memory themselves; the current CUDA
    device must hold every tensor.  Calls that overlap on the GPU race on the
    shared scratch.  device_status: optional int32 device tensor receiving the
    launch's device status.
    """
    lib = load()
    code = lib.dspark_markov_draft_noalloc(
        _ptr(U, (torch.float32,), "U"), _ptr(W1, _BF16, "W1"), _ptr(W2, _BF16, "W2"),
        _ptr(anchors, (torch.int32,), "anchors"), B, K, V, r, float(temperature),
        int(seed) & (2 ** 64 - 1), _ptr(tokens, (torch.int32,), "tokens"),
        _ptr(logprobs, (torch.float32,), "logprobs"),
        _ptr(device_status, (torch.int32,), "device_status"),
        _stream(stream, U.device))
    _check(code, "dspark_markov_draft_noalloc")


# ------------------------------------------------------ allocating wrappers
# With `stream`, the outputs that a wrapper makes (and its workspace) are that stream's memory; they may
# be read on it, or on the caller's current stream once that waits for it.  Inputs must be ready on it,
# and stay in use until its work is done, as with any torch call on another stream.
def _rank(W1) -> int:
    return 0 if W1 is None else int(W1.shape[1])


def markov_draft(ctx: Context, U, W1, W2, anchors, *, temperature=1.0, seed=0, h=None, Wg=None,
                 conf: Optional[Confidence] = None, stream=None) -> dict:
    """Vanilla (h, Wg None) or gated draft; returns tokens and logprobs [B, K]."""
    B, K, V = U.shape
    r = _rank(W1)
    tokens = _empty(stream, (B, K), torch.int32, U.device)
    logprobs = _empty(stream, (B, K), torch.float32, U.device)
    if conf is not None:
        conf.allocate(B, K, stream)
    if h is None and Wg is None:
        dspark_markov_draft(ctx, U, W1, W2, anchors, B, K, V, r, temperature, seed, tokens,
                            logprobs, conf, stream)
    else:
        dspark_gated_draft(ctx, U, W1, W2, anchors, h, Wg, int(h.shape[-1]), B, K, V, r,
                           temperature, seed, tokens, logprobs, conf, stream)
    out = dict(tokens=tokens, logprobs=logprobs)
    if conf is not None:
        out.update(conf=conf.conf, cumprod=conf.cumprod, verify_len=conf.verify_len)
    return out


def gate(ctx: Context, h, Wg, stream=None) -> torch.Tensor:
    d, r = Wg.shape
    M = h.numel() // d
    H = _empty(stream, (*h.shape[:-1], r), torch.float32, h.device)
    dspark_gate(ctx, h, Wg, M, d, r, H, stream)
    return H


def selector_scores(ctx: Context, U, A, Bt, anchors, *, topk=16, h=None, Wg=None,
                    stream=None) -> dict:
    B, K, V = U.shape
    r = int(A.shape[1])
    cand = _empty(stream, (B, K, topk), torch.int32, U.device)
    cand_U = _empty(stream, (B, K, topk), torch.float32, U.device)
    scores = _empty(stream, (B, K, topk, topk), torch.float32, U.device)
    d = 0 if h is None else int(h.shape[-1])
    dspark_selector_scores(ctx, U, A, Bt, anchors, h, Wg, d, B, K, V, r, topk, cand, cand_U,
                           scores, stream)
    return dict(cand=cand, cand_U=cand_U, scores=scores)


def selector_walk(ctx: Context, cand, scores, anchors, *, V, A=None, temperature=1.0, seed=0,
                  conf: Optional[Confidence] = None, stream=None) -> dict:
    B, K, topk = cand.shape
    r = 0 if A is None else int(A.shape[1])
    tokens = _empty(stream, (B, K), torch.int32, cand.device)
    logprobs = _empty(stream, (B, K), torch.float32, cand.device)
    if conf is not None:
        conf.allocate(B, K, stream)
    dspark_selector_walk(ctx, cand, scores, anchors, A, B, K, V, r, topk, temperature, seed,
                         tokens, logprobs, conf, stream)
    out = dict(tokens=tokens, logprobs=logprobs)
    if conf is not None:
        out.update(conf=conf.conf, cumprod=conf.cumprod, verify_len=conf.verify_len)
    return out


def confidence(ctx: Context, h, W1, anchors, tokens, w, *, V, bias=0.0, with_markov=True,
               threshold=0.3, tau=None, stream=None) -> dict:
    B, K, d = h.shape
    r = _rank(W1) if with_markov else 0
    conf = _empty(stream, (B, K), torch.float32, h.device)
    cum = _empty(stream, (B, K), torch.float32, h.device)
    vl = _empty(stream, (B,), torch.int32, h.device)
    dspark_confidence(ctx, h, W1 if with_markov else None, anchors, tokens, w, bias, with_markov,
                      B, K, d, r, V, threshold, tau, conf, cum, vl, stream)
    return dict(conf=conf, cumprod=cum, verify_len=vl)


def verify(ctx: Context, P, U, W1, W2, anchors, tokens, draft_logprobs, *, draft_temperature,
           target_temperature, seed=0, ell=None, h=None, Wg=None, stream=None) -> dict:
    """Speculative verification of drafted tokens [B, K] against target logits P [B, K+1, V]."""
    B, K, V = U.shape
    r = _rank(W1)
    n_acc = _empty(stream, (B,), torch.int32, U.device)
    next_token = _empty(stream, (B,), torch.int32, U.device)
    accept_prob = _empty(stream, (B, K), torch.float32, U.device)
    d = 0 if h is None else int(h.shape[-1])
    dspark_verify(ctx, P, U, W1, W2, anchors, h, Wg, d, tokens, draft_logprobs, ell, B, K, V, r,
                  draft_temperature, target_temperature, seed, n_acc, next_token, accept_prob,
                  stream)
    return dict(n_acc=n_acc, next_token=next_token, accept_prob=accept_prob)


def accept_label(ctx: Context, P, U, W1, W2, anchors, tokens, draft_logprobs=None, *,
                 draft_temperature, target_temperature, h=None, Wg=None, stream=None):
    """Acceptance label 1 - TV(draft, target) [B, K] of drafted tokens [B, K]."""
    B, K, V = U.shape
    r = _rank(W1)
    label = _empty(stream, (B, K), torch.float32, U.device)
    d = 0 if h is None else int(h.shape[-1])
    dspark_accept_label(ctx, P, U, W1, W2, anchors, h, Wg, d, tokens, draft_logprobs, B, K, V, r,
                        draft_temperature, target_temperature, label, stream)
    return label


def sts_fit(ctx: Context, conf, label, *, tau_lo=1.0 / 64, tau_hi=64.0, stream=None) -> dict:
    """Sequential temperature scaling: temperatures [K] from raw confidences and labels [N, K]."""
    N, K = conf.shape
    tau = _empty(stream, (K,), torch.float32, conf.device)
    loss = _empty(stream, (K,), torch.float32, conf.device)
    dspark_sts_fit(ctx, conf, label, N, K, tau_lo, tau_hi, tau, loss, stream)
    return dict(tau=tau, loss=loss)


def schedule(ctx: Context, a, sps, stream=None) -> dict:
    """Greedy load-aware verify lengths: survival a [R, K], SPS(B) table [>= R (K+1) + 1]."""
    R, K = a.shape
    ell = _empty(stream, (R,), torch.int32, a.device)
    theta = _empty(stream, (1,), torch.float32, a.device)
    dspark_schedule(ctx, a, R, K, sps, ell, theta, stream)
    return dict(ell=ell, theta=theta)


def rnn_draft(ctx: Context, U, W1, W2, anchors, h, Wa, *, Wg=None, temperature=1.0, seed=0,
              conf: Optional[Confidence] = None, stream=None) -> dict:
    """The RNN head's draft (decay gate from Wa, input gate from Wg or 1); returns tokens and
    logprobs [B, K] (and the confidence head's outputs when conf is given)."""
    B, K, V = U.shape
    r = _rank(W1)
    tokens = _empty(stream, (B, K), torch.int32, U.device)
    logprobs = _empty(stream, (B, K), torch.float32, U.device)
    if conf is not None:
        conf.allocate(B, K, stream)
    dspark_rnn_draft(ctx, U, W1, W2, anchors, h, Wa, Wg, int(h.shape[-1]), B, K, V, r,
                     temperature, seed, tokens, logprobs, conf, stream)
    out = dict(tokens=tokens, logprobs=logprobs)
    if conf is not None:
        out.update(conf=conf.conf, cumprod=conf.cumprod, verify_len=conf.verify_len)
    return out


def rnn_logits(ctx: Context, U, W1, W2, prev_tokens, h, Wa, *, Wg=None, temperature=1.0,
               stream=None) -> dict:
    """The RNN head's teacher-forced logits [B, K, V] and LSE [B, K]."""
    B, K, V = U.shape
    r = _rank(W1)
    logits = _empty(stream, (B, K, V), torch.float32, U.device)
    lse = _empty(stream, (B, K), torch.float32, U.device)
    dspark_rnn_logits(ctx, U, W1, W2, prev_tokens, h, Wa, Wg, int(h.shape[-1]), B, K, V, r,
                      temperature, logits, lse, stream)
    return dict(logits=logits, lse=lse)


def markov_logits(ctx: Context, U, W1, W2, prev_tokens, *, temperature=1.0, h=None, Wg=None,
                  stream=None) -> dict:
    B, K, V = U.shape
    r = _rank(W1)
    logits = _empty(stream, (B, K, V), torch.float32, U.device)
    lse = _empty(stream, (B, K), torch.float32, U.device)
    d = 0 if h is None else int(h.shape[-1])
    dspark_markov_logits(ctx, U, W1, W2, prev_tokens, h, Wg, d, B, K, V, r, temperature, logits,
                         lse, stream)
    return dict(logits=logits, lse=lse)


def verify_probs(ctx: Context, P, tokens, u_accept, u_draw, *, Q=None, cand=None, cand_q=None,
                 ell=None, stream=None) -> dict:
    """Accept-or-correct of drafted tokens [B, K] against target probabilities P [B, K+1, V] from
    uniforms u_accept [B, K] and u_draw [B]; the draft's probabilities are Q [B, K, V], or cand_q
    on the candidates cand [B, K, m]."""
    B, K = tokens.shape
    V = P.shape[-1]
    m = 0 if cand is None else int(cand.shape[-1])
    _shape(P, (B, K + 1, V), "P")
    _shape(Q, (B, K, V), "Q")
    _shape(cand, (B, K, m), "cand")
    _shape(cand_q, (B, K, m), "cand_q")
    _shape(u_accept, (B, K), "u_accept")
    _shape(u_draw, (B,), "u_draw")
    _shape(ell, (B,), "ell")
    n_acc = _empty(stream, (B,), torch.int32, P.device)
    next_token = _empty(stream, (B,), torch.int32, P.device)
    accept_prob = _empty(stream, (B, K), torch.float32, P.device)
    dspark_verify_probs(ctx, P, Q, cand, cand_q, m, tokens, u_accept, u_draw, ell, B, K, V, n_acc,
                        next_token, accept_prob, stream)
    return dict(n_acc=n_acc, next_token=next_token, accept_prob=accept_prob)


def distill(ctx: Context, logits, teacher_ids, teacher_logits, *, teacher_rest=None,
            row_weight=None, temperature=1.0, alpha_kl=0.1, alpha_tv=0.9, grad=True,
            stream=None) -> dict:
    """Loss of student logits [..., V] (fp32 or bf16, rows evenly spaced) against a teacher's top
    logits [..., k], and its gradient: grad True allocates it, a tensor (logits itself, say)
    receives it, False leaves it out.  Returns loss and tv [...], and grad [..., V]."""
    lead, V = logits.shape[:-1], int(logits.shape[-1])
    k = int(teacher_ids.shape[-1])
    _shape(teacher_ids, (*lead, k), "teacher_ids")
    _shape(teacher_logits, (*lead, k), "teacher_logits")
    _shape(teacher_rest, lead, "teacher_rest")
    _shape(row_weight, lead, "row_weight")
    N = lead.numel()
    loss = _empty(stream, lead, torch.float32, logits.device)
    tv = _empty(stream, lead, torch.float32, logits.device)
    if grad is True:
        grad = _empty(stream, (*lead, V), logits.dtype, logits.device)
    elif grad is False:
        grad = None
    _shape(grad, (*lead, V), "grad")
    dspark_distill(ctx, logits, teacher_ids, teacher_logits, k, teacher_rest, row_weight, N, V,
                   temperature, alpha_kl, alpha_tv, loss, tv, grad, stream)
    out = dict(loss=loss, tv=tv)
    if grad is not None:
        out["grad"] = grad
    return out


def rnn_scan(ctx: Context, za, zg, e, *, s0=None, reset=None, stream=None) -> dict:
    """States of the RNN head over given sequences: s_t = sigmoid(za_t) s_{t-1} + sigmoid(zg_t) e_t
    (zg None: 1), tensors [N, L, D] in fp32 or bf16; returns s [N, L, D] and s_last [N, D] fp32."""
    N, L, D = e.shape
    _shape(za, e.shape, "za")
    _shape(zg, e.shape, "zg")
    _shape(s0, (N, D), "s0")
    _shape(reset, (N, L), "reset")
    s = _empty(stream, (N, L, D), e.dtype, e.device)
    s_last = _empty(stream, (N, D), torch.float32, e.device)
    dspark_rnn_scan(ctx, za, zg, e, s0, reset, N, L, D, s, s_last, stream)
    return dict(s=s, s_last=s_last)


def rnn_scan_grad(ctx: Context, za, zg, e, s, ds, *, s0=None, ds_last=None, reset=None,
                  stream=None) -> dict:
    """Gradients of rnn_scan from ds [N, L, D] (of s) and ds_last [N, D] (of s_last).  Returns
    dza and dzg (the two halves of one [N, L, 2 D] tensor; dzg only with zg), de, and ds0 [N, D]."""
    N, L, D = e.shape
    _shape(za, e.shape, "za")
    _shape(zg, e.shape, "zg")
    _shape(s, e.shape, "s")
    _shape(ds, e.shape, "ds")
    _shape(s0, (N, D), "s0")
    _shape(ds_last, (N, D), "ds_last")
    _shape(reset, (N, L), "reset")
    dz = _empty(stream, (N, L, D if zg is None else 2 * D), e.dtype, e.device)
    dza, dzg = dz[..., :D], None if zg is None else dz[..., D:]
    de = _empty(stream, (N, L, D), e.dtype, e.device)
    ds0 = _empty(stream, (N, D), torch.float32, e.device)
    dspark_rnn_scan_grad(ctx, za, zg, e, s, ds, s0, reset, ds_last, N, L, D, dza, dzg, de, ds0,
                         stream)
    out = dict(dza=dza, de=de, ds0=ds0)
    if zg is not None:
        out["dzg"] = dzg
    return out


def embed(ctx: Context, table, ids, *, scale=1.0, dtype=None, out=None, stream=None) -> torch.Tensor:
    """scale * table[ids] [..., D] for ids [...] (negative: zeros), of the table's type or `dtype`
    (fp32, bf16); out receives it."""
    V, D = table.shape
    if out is None:
        out = _empty(stream, (*ids.shape, D), dtype or table.dtype, table.device)
    _shape(out, (*ids.shape, D), "out")
    dspark_embed(ctx, table, ids, ids.numel(), V, D, scale, out, stream)
    return out


def embed_grad(ctx: Context, ids, de, V=None, *, scale=1.0, dtype=torch.float32, grad=None,
               accumulate=False, stream=None) -> torch.Tensor:
    """Gradient [V, D] of embed's table from de [..., D]: per token, scale times the sum of its
    rows.  grad receives it (with accumulate: is added to)."""
    D = de.shape[-1]
    _shape(de, (*ids.shape, D), "de")
    if grad is None:
        if accumulate or V is None:
            raise ValueError("embed_grad: accumulate needs grad, and a new gradient V")
        grad = _empty(stream, (V, D), dtype, de.device)
    _shape(grad, (grad.shape[0] if V is None else V, D), "grad")
    dspark_embed_grad(ctx, ids, de, ids.numel(), grad.shape[0], D, scale, accumulate, grad, stream)
    return grad


def grad_norm(ctx: Context, grads, stream=None) -> torch.Tensor:
    """The norm of all tensors of a list together (fp32 scalar on the device)."""
    norm = _empty(stream, (), torch.float32, torch.device("cuda", ctx.device))
    dspark_clip_grads(ctx, list(grads), 0.0, None, norm, stream)
    return norm


def clip_grads(ctx: Context, grads, max_norm, *, out=None, stream=None) -> torch.Tensor:
    """Scale a list of gradients (fp32, bf16) to a common norm of at most max_norm, in place or
    into the tensors of out; returns their norm before (fp32 scalar on the device).  A tensor that
    several parameters share is listed once."""
    norm = _empty(stream, (), torch.float32, torch.device("cuda", ctx.device))
    grads = list(grads)
    dspark_clip_grads(ctx, grads, max_norm, grads if out is None else list(out), norm, stream)
    return norm


def linear(ctx: Context, x, W, *, bias=None, act=None, residual=None, dtype=None, out=None,
           pre=False, workspace=None, stream=None) -> dict:
    """act(x W + bias) + residual for x [..., K] and W [K, N] in bf16 (rows evenly spaced), act None,
    "sigmoid", "tanh", "relu", "silu" or "gelu".  Returns y [..., N] (of `dtype`, x's by default;
    out receives it and may be the residual) and, with pre, x W + bias in y's type."""
    K, N = W.shape
    lead = x.shape[:-1]
    _shape(x, (*lead, K), "x")
    _shape(bias, (N,), "bias")
    _shape(residual, (*lead, N), "residual")
    y = _empty(stream, (*lead, N), dtype or x.dtype, x.device) if out is None else out
    _shape(y, (*lead, N), "out")
    if pre is True:
        pre = _empty(stream, (*lead, N), y.dtype, x.device)
    elif pre is False:
        pre = None
    _shape(pre, (*lead, N), "pre")
    dspark_linear(ctx, x, W, bias, act, residual, lead.numel(), K, N, y, pre, workspace, stream)
    out = dict(y=y)
    if pre is not None:
        out["pre"] = pre
    return out


def linear_grad(ctx: Context, x, W, dy, *, act=None, pre=None, dx=True, dW=True, dbias=False,
                workspace=None, stream=None) -> dict:
    """Gradients of linear from dy [..., N] (fp32 or bf16; pre as linear returned it, where there
    is an activation).  dx [..., K] in x's type, dW [K, N] and dbias [N] in fp32: True allocates, a
    tensor receives (dx, dW of either type), False leaves out."""
    K, N = W.shape
    lead = dy.shape[:-1]
    _shape(x, (*lead, K), "x")
    _shape(dy, (*lead, N), "dy")
    _shape(pre, (*lead, N), "pre")
    given = dict(dx=(dx, (*lead, K), x.dtype), dW=(dW, (K, N), torch.float32), dbias=(dbias, (N,), torch.float32))
    out = {}
    for name, (want, shape, dtype) in given.items():
        if want is True:
            out[name] = _empty(stream, shape, dtype, dy.device)
        elif want is not False:
            _shape(want, shape, name)
            out[name] = want
    dspark_linear_grad(ctx, x, W, dy, act, pre, lead.numel(), K, N, out.get("dx"), out.get("dW"),
                       out.get("dbias"), workspace, stream)
    return out
