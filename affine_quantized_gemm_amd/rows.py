"""What lies between the products and the cache in a decoder's step: the gated block, rotary positions, log probabilities.

Argument checks and marshalling only; every step runs in the HIP kernels of
``libqmm.so`` (``qmm_gated``, ``qmm_rotary``, ``qmm_log_probs`` and the
gradients in ``include/qmm.h``, where the formulas and contracts are).
None of them records itself for torch's autograd: the ``_backward`` calls (and
``rotary`` with ``inverse``) are the gradients.
"""

from __future__ import annotations

import ctypes
import math
from typing import NamedTuple

import torch

from . import (_DT, _as_stream, _lib, QMM_ERR_UNSUPPORTED, QmmError, _check, _check_quantized, _dev, _dt, _expect,
               _same_device)

ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}  # qmm_act
PAIRS = {"halves": 0, "adjacent": 1}                      # qmm_pairs
LOG_PROBS_ZEROED_BYTES = 65536                            # QMM_LOG_PROBS_ZEROED_BYTES
LOG_PROBS_WORKSPACE_BYTES = 65536 + 1024 * 66 * 8         # QMM_LOG_PROBS_WORKSPACE_BYTES
_CODES, _GROUPS = (4, 6, 8), (32, 64, 128)
_INTS = (torch.int32, torch.int64)


class _On:
    """The device and stream of a call on t: t's device, its current stream unless one is given."""

    __slots__ = ("device", "stream", "raw", "back")

    def __init__(self, t: torch.Tensor, stream):
        if not t.is_cuda:
            raise ValueError("the operands must be GPU tensors")
        self.device, self.stream = t.device, stream
        self.back = None

    def __enter__(self):
        index = self.device.index
        now = torch.cuda.current_device()
        if now != index:  # (a kernel goes to the current device)
            torch.cuda.set_device(index)
            self.back = now
        self.raw = torch._C._cuda_getCurrentRawStream(index) if self.stream is None else \
            int(getattr(self.stream, "cuda_stream", self.stream))
        return self

    def __exit__(self, *_):
        if self.back is not None:
            torch.cuda.set_device(self.back)

    def new(self, shape, dtype):
        """A tensor of this call, of the memory of the stream it runs on."""
        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self.torch_stream()):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def torch_stream(self):
        return _as_stream(self.stream, self.device)


def _fits(t, shape, dtype, index):
    """Whether a GPU tensor is as expected; where one is not, the checks that name the fault are run (they take 1 to 2 us
    an operand, this 0.4, and a small call's kernel runs 5)."""
    return isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype and t.get_device() == index and t.is_contiguous()


def _key(table, name, what):
    if name not in table:
        raise ValueError(f"{what} is {name!r}, expected one of {tuple(table)}")
    return table[name]


def _out(on, out, name, shape, dtype):
    if out is None:
        return on.new(shape, dtype)
    _expect(out, name, shape, (dtype,))
    _dev(out, name)
    if out.device != on.device:
        raise ValueError(f"{name} is on {out.device}, expected {on.device}")
    return out


# ---- gated block ----

def _check_gated(x, wq, scales, biases, bits, group_size):
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D [M, K], got shape {tuple(x.shape)}")
    dt = _dt(x.dtype)
    if wq.dim() != 2 or wq.shape[0] % 2:
        raise ValueError(f"wq must be 2-D [2F, K*bits/32], got shape {tuple(wq.shape)}")
    M, K = x.shape
    # (what the library refuses of bits and group_size, it refuses itself)
    if bits in _CODES and group_size in _GROUPS and K % group_size == 0:
        rows, index = wq.shape[0], x.get_device()
        groups = (rows, K // group_size)
        if (index >= 0 and x.is_contiguous() and _fits(wq, (rows, K * bits // 32), torch.int32, index)
                and _fits(scales, groups, x.dtype, index) and _fits(biases, groups, x.dtype, index)):
            return dt, M, rows // 2, K
    _check_quantized(x.dtype, wq, scales, biases, wq.shape[0], K, bits, group_size)
    for t, n in ((x, "x"), (wq, "wq"), (scales, "scales"), (biases, "biases")):
        _dev(t, n)
    _same_device(x, (wq, "wq"), (scales, "scales"), (biases, "biases"))
    return dt, M, wq.shape[0] // 2, K


def gated(x: torch.Tensor, wq: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor, bits: int, group_size: int,
          act: str = "silu", out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """h [M, F] = act(x . Wg^T) * (x . Wu^T): x [M, K], wq [2F, K*bits/32] (and scales, biases) of both, the gate's rows
    first (:func:`quantize` of a [2F, K] matrix).  ``act``: "silu", "gelu", "gelu_tanh" or "relu"."""
    dt, M, F, K = _check_gated(x, wq, scales, biases, bits, group_size)
    a = _key(ACTS, act, "act")
    with _On(x, stream) as on:
        out = _out(on, out, "out", (M, F), x.dtype)
        _check(_lib.qmm_gated(dt, bits, group_size, a, M, F, K, x.data_ptr(), wq.data_ptr(), scales.data_ptr(),
                              biases.data_ptr(), out.data_ptr(), on.raw), "qmm_gated")
    return out


def gated_backward_workspace_bytes(dtype, bits: int, group_size: int, M: int, F: int, K: int) -> int:
    """Bytes of workspace :func:`gated_backward` needs (0: none)."""
    n = int(_lib.qmm_gated_backward_workspace_bytes(_dt(dtype), bits, group_size, M, F, K))
    if n < 0:
        raise QmmError(n, "qmm_gated_backward_workspace_bytes")
    return n


def gated_backward(x: torch.Tensor, wq: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor, bits: int,
                   group_size: int, grad: torch.Tensor, act: str = "silu", grad_gate_up: torch.Tensor | None = None,
                   out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """(grad_x [M, K], grad_gate_up [M, 2F]) of :func:`gated` for grad [M, F] of its result: the gradients of x and of
    the two products x . [Wg; Wu]^T.  The weights are constants."""
    dt, M, F, K = _check_gated(x, wq, scales, biases, bits, group_size)
    a = _key(ACTS, act, "act")
    _expect(grad, "grad", (M, F), (x.dtype,))
    _dev(grad, "grad")
    _same_device(x, (grad, "grad"))
    need = gated_backward_workspace_bytes(x.dtype, bits, group_size, M, F, K)
    with _On(x, stream) as on:
        grad_gate_up = _out(on, grad_gate_up, "grad_gate_up", (M, 2 * F), x.dtype)
        out = _out(on, out, "out", (M, K), x.dtype)
        if workspace is None and need > 0:
            # (a temporary's block goes back to the caching allocator, which hands it out again in stream order)
            workspace = on.new((need,), torch.uint8)
        elif workspace is not None:
            _dev(workspace, "workspace")
            _same_device(x, (workspace, "workspace"))
        _check(_lib.qmm_gated_backward(dt, bits, group_size, a, M, F, K, x.data_ptr(), wq.data_ptr(), scales.data_ptr(),
                                       biases.data_ptr(), grad.data_ptr(), grad_gate_up.data_ptr(), out.data_ptr(),
                                       None if workspace is None else workspace.data_ptr(),
                                       0 if workspace is None else workspace.numel() * workspace.element_size(), on.raw),
               "qmm_gated_backward")
    return out, grad_gate_up


# ---- rotary positions ----

def rotary(x: torch.Tensor, positions: torch.Tensor, freq: torch.Tensor, sections=None, pairs: str = "halves",
           inverse: bool = False, scale: float = 1.0, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """x [rows, heads, head_dim] with every head's pairs turned by positions * freq (radians).

    ``positions`` [rows], or [axes, rows] with ``sections``, the numbers of
    consecutive pairs of each axis (int32 or int64); ``freq`` fp32
    [rotary_dim / 2], rotary_dim up to head_dim (values behind it stay).
    ``pairs``: "halves", (p, p + rotary_dim / 2), or "adjacent", (2p, 2p + 1).
    ``inverse`` turns back, which is also the gradient's map.  ``scale``
    multiplies the turned values.  x's rows and heads may be strided; ``out``
    may be x."""
    if x.dim() != 3:
        raise ValueError(f"x must be 3-D [rows, heads, head_dim], got shape {tuple(x.shape)}")
    dt = _dt(x.dtype)
    rows, heads, dim = x.shape
    if dim and x.stride(2) != 1:
        raise ValueError("x's last axis must be contiguous")
    axes = 1 if sections is None else len(sections)
    if _fits(positions, (rows,) if sections is None else (axes, rows), torch.int64, x.get_device()):
        pass
    elif sections is None or (axes == 1 and positions.dim() == 1):
        _expect(positions, "positions", (rows,), _INTS)
    else:
        _expect(positions, "positions", (axes, rows), _INTS)
    if rows > 1 and positions.stride(-1) != 1:
        raise ValueError("positions' last axis must be contiguous")
    if freq.dim() != 1:
        raise ValueError(f"freq must be 1-D [rotary_dim / 2], got shape {tuple(freq.shape)}")
    if not _fits(freq, freq.shape, torch.float32, x.get_device()):
        _expect(freq, "freq", tuple(freq.shape), (torch.float32,))
        _dev(freq, "freq")
        _same_device(x, (freq, "freq"))
    _same_device(x, (positions, "positions"))
    if sections is None:
        cuts = None
    else:
        if not 1 <= axes <= 4 or any(int(n) < 0 for n in sections) or sum(int(n) for n in sections) != freq.numel():
            raise ValueError(f"sections {tuple(sections)}: 1 to 4 axes, together the {freq.numel()} pairs of freq")
        cuts = (ctypes.c_int32 * axes)(*[int(n) for n in sections])
    kind = _key(PAIRS, pairs, "pairs")
    with _On(x, stream) as on:
        if out is None:
            out = on.new((rows, heads, dim), x.dtype)
        else:
            _expect(out, "out", (rows, heads, dim), (x.dtype,))
            _same_device(x, (out, "out"))
            if dim and out.stride(2) != 1:
                raise ValueError("out's last axis must be contiguous")
        xr, xh, _ = x.stride()
        outr, outh, _ = out.stride()
        _check(_lib.qmm_rotary(dt, rows, heads, dim, 2 * freq.numel(), kind, 1 if inverse else 0, scale, x.data_ptr(), xr, xh,
                               positions.data_ptr(), 1 if positions.dtype is torch.int64 else 0,
                               positions.stride(0) if positions.dim() == 2 else 0, axes, cuts, freq.data_ptr(),
                               out.data_ptr(), outr, outh, on.raw), "qmm_rotary")
    return out


# ---- log probabilities ----

class LogProbs(NamedTuple):
    lse: torch.Tensor                 # fp32 [rows]: ln sum exp of the scaled logits
    entropy: torch.Tensor             # fp32 [rows], nats
    tokens: torch.Tensor | None       # fp32, the given tokens' log probabilities, their shape
    top_values: torch.Tensor | None   # fp32 [rows, top], likeliest first
    top_ids: torch.Tensor | None      # int64 [rows, top]


_spaces: dict[tuple[int, int], torch.Tensor] = {}  # (device, stream): the workspace kept for its calls


def _zeroed(device):
    return torch.zeros((LOG_PROBS_WORKSPACE_BYTES,), dtype=torch.uint8, device=device)


def log_probs_workspace(device="cuda") -> torch.Tensor:
    """A workspace for :func:`log_probs` calls of any sizes (one per stream, or per captured graph)."""
    return _zeroed(device)


def _own_space(on):
    """The workspace of a call that was not given one: kept for the stream; in a call that is being captured one of its
    own, whose counters are zeroed in the graph."""
    if on.stream is not None:
        with torch.cuda.stream(on.torch_stream()):  # its state of capture, its memory
            return _space_here(on)
    return _space_here(on)


def _space_here(on):
    if torch.cuda.is_current_stream_capturing():
        own = torch.empty((LOG_PROBS_WORKSPACE_BYTES,), dtype=torch.uint8, device=on.device)
        own[:LOG_PROBS_ZEROED_BYTES].zero_()
        return own
    kept = _spaces.get((on.device.index, on.raw))
    if kept is None:
        kept = _spaces[(on.device.index, on.raw)] = _zeroed(on.device)
    return kept


def _check_logits(logits, tokens, scale):
    """(dt, rows, vocab, stride, given) of a call."""
    if logits.dim() != 2:
        raise ValueError(f"logits must be 2-D [rows, vocab], got shape {tuple(logits.shape)}")
    dt = _dt(logits.dtype)
    if not logits.is_cuda:
        raise ValueError("logits must be a GPU tensor")
    rows, vocab = logits.shape
    if vocab > 1 and logits.stride(1) != 1:
        raise ValueError("logits' last axis must be contiguous")
    if not (math.isfinite(scale) and scale > 0):
        raise ValueError(f"scale {scale}: a finite number above 0")
    given = 0
    if tokens is not None:
        if tokens.dim() not in (1, 2):
            raise ValueError(f"tokens must be [rows] or [rows, n], got shape {tuple(tokens.shape)}")
        given = 1 if tokens.dim() == 1 else tokens.shape[1]
        shape = (rows,) if tokens.dim() == 1 else (rows, given)
        if not _fits(tokens, shape, torch.int64, logits.get_device()):
            _expect(tokens, "tokens", shape, _INTS)
            _dev(tokens, "tokens")
            _same_device(logits, (tokens, "tokens"))
    return dt, rows, vocab, logits.stride(0), given


def log_probs(logits: torch.Tensor, tokens: torch.Tensor | None = None, top: int = 0, scale: float = 1.0,
              workspace: torch.Tensor | None = None, stream=None) -> LogProbs:
    """Log probabilities under softmax(scale * logits), logits [rows, vocab] (rows may be strided, -infinity bars a token).

    ``tokens`` [rows] or [rows, n] (int32 or int64; an id outside the
    vocabulary, padding, gets 0); ``top``: so many of the likeliest tokens (up
    to 64), of equal logits the lowest id first.  ``scale`` is the inverse
    temperature (2^-100 to 2^100).  ``workspace``: from :func:`log_probs_workspace` (default: one
    kept for the stream)."""
    dt, rows, vocab, stride, given = _check_logits(logits, tokens, scale)
    if not 0 <= top <= min(64, vocab):
        raise QmmError(QMM_ERR_UNSUPPORTED, f"top={top} of {vocab} tokens")
    with _On(logits, stream) as on:
        lse, entropy = on.new((rows,), torch.float32), on.new((rows,), torch.float32)
        lp = None if tokens is None else on.new(tuple(tokens.shape), torch.float32)
        values = ids = None
        if top:
            values, ids = on.new((rows, top), torch.float32), on.new((rows, top), torch.int64)
        if workspace is not None:
            _dev(workspace, "workspace")
            _same_device(logits, (workspace, "workspace"))
        elif _lib.qmm_log_probs_needs_workspace(rows, vocab) == 1:
            workspace = _own_space(on)
        _check(_lib.qmm_log_probs(dt, rows, vocab, scale, logits.data_ptr(), stride,
                                  None if tokens is None else tokens.data_ptr(),
                                  1 if tokens is not None and tokens.dtype is torch.int64 else 0, given, top, lse.data_ptr(),
                                  entropy.data_ptr(), None if lp is None else lp.data_ptr(),
                                  None if values is None else values.data_ptr(), None if ids is None else ids.data_ptr(),
                                  None if workspace is None else workspace.data_ptr(),
                                  0 if workspace is None else workspace.numel() * workspace.element_size(), on.raw),
               "qmm_log_probs")
    return LogProbs(lse, entropy, lp, values, ids)


def log_probs_backward(logits: torch.Tensor, tokens: torch.Tensor | None, lse: torch.Tensor,
                       entropy: torch.Tensor | None, grad_tokens: torch.Tensor | None,
                       grad_entropy: torch.Tensor | None = None, grad_lse: torch.Tensor | None = None,
                       scale: float = 1.0, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient [rows, vocab] of sum grad_tokens * tokens + grad_entropy * entropy + grad_lse * lse for the logits, with
    ``lse`` and ``entropy`` as :func:`log_probs` returned them.  The likeliest tokens' log probabilities have theirs as
    given tokens.  ``out`` may be the logits."""
    dt, rows, vocab, stride, given = _check_logits(logits, tokens, scale)
    if (tokens is None) != (grad_tokens is None):
        raise ValueError("tokens and grad_tokens go together")
    if grad_entropy is not None and entropy is None:
        raise ValueError("grad_entropy needs the entropy")
    named = [(lse, "lse", (rows,)), (entropy, "entropy", (rows,)), (grad_entropy, "grad_entropy", (rows,)),
             (grad_lse, "grad_lse", (rows,))]
    if grad_tokens is not None:
        named.append((grad_tokens, "grad_tokens", tuple(tokens.shape)))
    for t, n, shape in named:
        if t is not None:
            _expect(t, n, shape, (torch.float32,))
            _dev(t, n)
            _same_device(logits, (t, n))
        elif n == "lse":
            raise ValueError("lse must be a tensor")
    ptr = lambda t: None if t is None else t.data_ptr()
    with _On(logits, stream) as on:
        if out is None:
            out = on.new((rows, vocab), logits.dtype)
        else:
            _expect(out, "out", (rows, vocab), (logits.dtype,))
            _same_device(logits, (out, "out"))
            if vocab > 1 and out.stride(1) != 1:
                raise ValueError("out's last axis must be contiguous")
        _check(_lib.qmm_log_probs_backward(dt, rows, vocab, scale, logits.data_ptr(), stride, ptr(tokens),
                                           1 if tokens is not None and tokens.dtype is torch.int64 else 0, given, ptr(lse),
                                           ptr(entropy), ptr(grad_tokens), ptr(grad_entropy), ptr(grad_lse), out.data_ptr(),
                                           out.stride(0), on.raw), "qmm_log_probs_backward")
    return out
