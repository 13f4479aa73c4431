"""Training objectives: device buffers (allocated with torch) around libvsf's
loss and router calls, as ``step.ShardStep`` is around the shard step.

TokenLogprobs   log probability of each token under its row of logits
PolicyLoss      clipped policy loss with a KL term, and the logits' gradient
PreferenceLoss  loss of (chosen, rejected) pairs, and the logits' gradient
Router          top-k choice, gates, per-expert counts, balance loss; gradient

An object owns its workspace and its outputs, sized for the largest call
(`tokens` rows); a call returns views of the outputs, which the next call of
the same object overwrites, on the object's stream, whose memory they are. As
everywhere in the library nothing is synchronised: a caller that works on
another stream orders the two itself, and keeps inputs and outputs (or
record_stream()s them) until the other stream is done with them. The object's
device has to be the current one. The formulas stand at the C functions in
include/vsf.h.
"""
from __future__ import annotations

import torch

from . import vsf as V

_DTYPES = {torch.bfloat16: V.VSF_BF16, torch.float32: V.VSF_FP32}


class _Objective:
    """The device, the stream and the checks of arguments."""

    def __init__(self, tokens: int, width: int, dtype, device, stream):
        if dtype not in _DTYPES:
            raise ValueError(f"logits are bfloat16 or float32, not {dtype}")
        if tokens < 0 or width < 1:
            raise ValueError(f"sizes out of range: {tokens} tokens, rows of {width}")
        self.tokens, self.width, self.dtype = int(tokens), int(width), dtype
        self._vdt = _DTYPES[dtype]
        device = torch.device("cuda" if device is None else device)
        self._index = torch.cuda.current_device()
        if device.type != "cuda" or device.index not in (None, self._index):
            raise ValueError(f"device: the current one (cuda:{self._index}), not {device}")
        self.device = torch.device("cuda", self._index)
        self.stream = stream if stream is not None else torch.cuda.current_stream(self.device)
        self._st = self.stream.cuda_stream

    def _new(self, *shape, dtype=torch.float32):
        # Memory of the object's own stream: a block of the caller's could still
        # be in use there while it is prepared here, or be handed out again there
        # while the last call runs.
        with torch.cuda.stream(self.stream):
            return torch.empty(*shape, dtype=dtype, device=self.device)

    def _workspace(self, nbytes: int):
        if not nbytes:
            raise ValueError("sizes out of range")
        self.workspace = self._new(nbytes, dtype=torch.uint8)
        self._ws, self._ws_bytes = self.workspace.data_ptr(), nbytes
        V.vsf_objective_workspace_init(self._ws, nbytes, self._st)

    def _rows(self, x, what: str):
        """Checks rows of logits (or their gradient); their number and stride."""
        shape = x.shape
        if x.dtype is not self.dtype or len(shape) != 2 or shape[1] != self.width \
                or shape[0] > self.tokens or x.get_device() != self._index:
            raise ValueError(f"{what}: expected {self.dtype} [<= {self.tokens}, {self.width}] on "
                             f"{self.device}, got {x.dtype} {tuple(shape)} on {x.device}")
        rows, cols = shape
        ld, unit = x.stride()
        if unit != 1 and cols > 1:
            raise ValueError(f"{what}: the elements of a row must be adjacent (stride {unit})")
        if ld < cols:
            if rows > 1:
                raise ValueError(f"{what}: rows overlap (stride {ld}, {cols} elements)")
            ld = cols
        return rows, ld

    def _vec(self, x, n: int, dtype, what: str):
        """Checks a contiguous vector of n elements; its address (None: none)."""
        if x is None:
            return None
        if x.dtype is not dtype or x.numel() != n or x.get_device() != self._index \
                or not x.is_contiguous():
            raise ValueError(f"{what}: expected {n} contiguous {dtype} on {self.device}, got "
                             f"{x.dtype} {tuple(x.shape)} on {x.device}")
        return x.data_ptr()

    def _first(self, buf, n: int):
        """The first n rows of an output of the object's own."""
        return buf if n == self.tokens else buf[:n]

    def device_error(self) -> int:
        """The device error word (0: no wait ran out, every target in range, the
        workspace this object's alone)."""
        return int(self.workspace[:4].view(torch.int32).item())


class TokenLogprobs(_Objective):
    """logp[t] = ln softmax(inv_temperature * logits[t])[targets[t]]; 0 where
    the target is negative. targets: int64."""

    def __init__(self, tokens: int, vocab: int, *, dtype=torch.bfloat16,
                 inv_temperature: float = 1.0, device=None, stream=None):
        super().__init__(tokens, vocab, dtype, device, stream)
        self.inv_temperature = inv_temperature
        self._workspace(V.vsf_objective_workspace_bytes(self.tokens))
        self.logp = self._new(self.tokens)
        self._logp = self.logp.data_ptr()

    def __call__(self, logits, targets):
        n, ld = self._rows(logits, "logits")
        V.vsf_token_logprobs(logits.data_ptr(), self._vdt, n, self.width, ld,
                             self._vec(targets, n, torch.int64, "targets"), self.inv_temperature,
                             self._logp, self._ws, self._ws_bytes, self._st)
        return self._first(self.logp, n)


class _LogitsLoss(_Objective):
    def _outputs(self, pairs: int, stats: int, with_grad: bool):
        self._workspace(V.vsf_objective_workspace_bytes(self.tokens, pairs))
        self.stats = self._new(stats)
        self.logp = self._new(self.tokens)
        self._out = self.stats.data_ptr(), self.logp.data_ptr()
        self.grad = None
        # The gradient's rows lie as far apart, modulo 16 bytes, as the logits',
        # so that both go in wide pieces.
        self._step = 16 // self.dtype.itemsize
        self._views = {}
        if with_grad:
            self._buffer = self._new(self.tokens * (self.width + self._step - 1), dtype=self.dtype)
            self._grad_at = self._buffer.data_ptr()
            self.grad = self._view(-self.width % self._step)

    def _view(self, pad: int):
        if pad not in self._views:
            self._views[pad] = self._buffer.as_strided((self.tokens, self.width),
                                                       (self.width + pad, 1))
        return self._views[pad]

    def _grad(self, n: int, ld: int, grad):
        """The gradient's tensor, address and row stride of a call."""
        if grad is not None:
            rows, grad_ld = self._rows(grad, "grad")
            if rows != n:
                raise ValueError(f"grad: {rows} rows, logits have {n}")
            return grad, grad.data_ptr(), grad_ld
        if self.grad is None:
            return None, None, self.width
        pad = (ld - self.width) % self._step
        self.grad = self._view(pad)  # (the attribute shows what the call writes)
        return self._first(self.grad, n), self._grad_at, self.width + pad


class PolicyLoss(_LogitsLoss):
    """Clipped policy loss with a KL term. A call returns (stats, logp, grad):
    stats = [loss, policy term, KL term, sum of the live weights]. grad is the
    object's own buffer, or the tensor given (the logits themselves to write
    in place); with_grad=False and no tensor given: loss only, grad None."""

    def __init__(self, tokens: int, vocab: int, *, dtype=torch.bfloat16, clip_low: float = 0.2,
                 clip_high: float = 0.2, kl_beta: float = 0.0, inv_temperature: float = 1.0,
                 scale: float = 1.0, mean: bool = True, with_grad: bool = True, device=None,
                 stream=None):
        super().__init__(tokens, vocab, dtype, device, stream)
        self.hp = V.make_policy_hparams(clip_low, clip_high, kl_beta, inv_temperature, scale, mean)
        self._outputs(0, 4, with_grad)

    def __call__(self, logits, targets, old_logp, advantages, ref_logp=None, weights=None,
                 grad=None):
        n, ld = self._rows(logits, "logits")
        grad, g, grad_ld = self._grad(n, ld, grad)
        f32 = torch.float32
        stats, logp = self._out
        V.vsf_policy_loss(logits.data_ptr(), self._vdt, n, self.width, ld,
                          self._vec(targets, n, torch.int64, "targets"),
                          self._vec(old_logp, n, f32, "old_logp"),
                          self._vec(ref_logp, n, f32, "ref_logp"),
                          self._vec(advantages, n, f32, "advantages"),
                          self._vec(weights, n, f32, "weights"), self.hp, stats, logp, g,
                          grad_ld, self._ws, self._ws_bytes, self._st)
        return self.stats, self._first(self.logp, n), grad


class PreferenceLoss(_LogitsLoss):
    """Preference loss of `pairs` pairs: sequences 0..pairs-1 are the chosen
    ones, pairs..2*pairs-1 the rejected ones, sequence s at rows
    [seq_starts[s], seq_starts[s+1]) (int64). A call returns (stats, rewards,
    logp, grad): stats = [loss, mean of beta h], rewards = beta D_s."""

    KINDS = {"sigmoid": V.VSF_PREF_SIGMOID, "squared": V.VSF_PREF_SQUARED}

    def __init__(self, pairs: int, tokens: int, vocab: int, *, dtype=torch.bfloat16,
                 kind: str = "sigmoid", beta: float = 0.1, smoothing: float = 0.0,
                 margin: float = 0.0, average: bool = False, inv_temperature: float = 1.0,
                 scale: float = 1.0, with_grad: bool = True, device=None, stream=None):
        super().__init__(tokens, vocab, dtype, device, stream)
        if kind not in self.KINDS:
            raise ValueError(f"kind: one of {sorted(self.KINDS)}, not {kind!r}")
        if pairs < 1:
            raise ValueError(f"pairs: at least 1, not {pairs}")
        self.pairs = int(pairs)
        self.hp = V.make_preference_hparams(beta, smoothing, margin, inv_temperature, scale,
                                            self.KINDS[kind], average)
        self._outputs(self.pairs, 2, with_grad)
        self.rewards = self._new(2 * self.pairs)
        self._rewards = self.rewards.data_ptr()

    def __call__(self, logits, targets, seq_starts, ref_logp=None, weights=None, grad=None):
        n, ld = self._rows(logits, "logits")
        grad, g, grad_ld = self._grad(n, ld, grad)
        f32 = torch.float32
        stats, logp = self._out
        V.vsf_preference_loss(logits.data_ptr(), self._vdt, n, self.width, ld,
                              self._vec(targets, n, torch.int64, "targets"),
                              self._vec(ref_logp, n, f32, "ref_logp"),
                              self._vec(weights, n, f32, "weights"),
                              self._vec(seq_starts, 2 * self.pairs + 1, torch.int64,
                                        "seq_starts"),
                              self.pairs, self.hp, stats, self._rewards, logp, g, grad_ld,
                              self._ws, self._ws_bytes, self._st)
        return self.stats, self.rewards, self._first(self.logp, n), grad


class Router(_Objective):
    """A mixture-of-experts router. forward returns (idx [T, top_k] int32,
    gates [T, top_k] fp32, counts [E] int32, balance loss fp32 scalar);
    backward the logits' gradient from the gates' gradient (None: none) and
    loss_scale times the balance loss, for the last forward call, whose choices
    and counts it reads. `calls` counts the forward calls: a program that may
    make another one in between (a second micro-batch, activations computed
    again) keeps the number and gives it to backward as `call`, which refuses
    if it is not the last one's any more."""

    SCORES = {"softmax": V.VSF_SCORE_SOFTMAX, "sigmoid": V.VSF_SCORE_SIGMOID}

    def __init__(self, tokens: int, experts: int, top_k: int, *, dtype=torch.bfloat16,
                 score: str = "softmax", renorm: bool = True, route_scale: float = 1.0,
                 balance: float = 0.0, sequences: int = 1, device=None, stream=None):
        super().__init__(tokens, experts, dtype, device, stream)
        if score not in self.SCORES:
            raise ValueError(f"score: one of {sorted(self.SCORES)}, not {score!r}")
        self.top_k, self.sequences = int(top_k), int(sequences)
        self.hp = V.make_route_hparams(top_k, self.SCORES[score], renorm, route_scale, balance)
        self._workspace(V.vsf_route_workspace_bytes(self.width, self.sequences))
        i32 = torch.int32
        self.idx = self._new(self.tokens, self.top_k, dtype=i32)
        self.gates = self._new(self.tokens, self.top_k)
        self.counts = self._new(self.width, dtype=i32)
        self.loss = self._new(())
        self.seq_counts = self._new(self.sequences, self.width, dtype=i32)
        self.seq_coef = self._new(self.sequences)
        self._out = [t.data_ptr() for t in (self.idx, self.gates, self.counts, self.loss,
                                            self.seq_counts, self.seq_coef)]
        self.grad = None  # made by the first backward
        self.calls, self._rows_routed = 0, None

    def _args(self, logits, live, seq_starts):
        n, ld = self._rows(logits, "logits")
        if seq_starts is None and self.sequences != 1:
            raise ValueError(f"seq_starts: needed for {self.sequences} sequences")
        return (n, ld, self._vec(live, n, torch.uint8, "live"),
                self._vec(seq_starts, self.sequences + 1, torch.int64, "seq_starts"))

    def forward(self, logits, bias=None, live=None, seq_starts=None):
        n, ld, lv, starts = self._args(logits, live, seq_starts)
        V.vsf_route(logits.data_ptr(), self._vdt, n, self.width, ld,
                    self._vec(bias, self.width, torch.float32, "bias"), lv, starts,
                    self.sequences, self.hp, *self._out, self._ws, self._ws_bytes, self._st)
        self.calls += 1
        self._rows_routed = n
        return self._first(self.idx, n), self._first(self.gates, n), self.counts, self.loss

    def backward(self, logits, d_gates=None, live=None, seq_starts=None, loss_scale: float = 1.0,
                 grad=None, call: int | None = None):
        n, ld, lv, starts = self._args(logits, live, seq_starts)
        if n != self._rows_routed:
            raise ValueError(f"backward: {n} tokens, the last forward call had {self._rows_routed}")
        if call is not None and call != self.calls:
            raise ValueError(f"backward of forward call {call}: call {self.calls} has followed it")
        if grad is None:
            if self.grad is None:
                self.grad = self._new(self.tokens, self.width, dtype=self.dtype)
            grad, grad_ld = self._first(self.grad, n), self.width
        else:
            rows, grad_ld = self._rows(grad, "grad")
            if rows != n:
                raise ValueError(f"grad: {rows} rows, logits have {n}")
        V.vsf_route_grad(logits.data_ptr(), self._vdt, n, self.width, ld, lv, starts,
                         self.sequences, self.hp, self._out[0],
                         self._vec(d_gates, n * self.top_k, torch.float32, "d_gates"),
                         *self._out[4:], loss_scale,
                         grad.data_ptr(), grad_ld, self._st)
        return grad
