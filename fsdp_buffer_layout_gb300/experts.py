"""A mixture-of-experts layer between ``objectives.Router`` and the losses: device
buffers (allocated with torch) around libvsf's expert calls.

Dispatch      tokens sorted by expert, their rows in that order, the experts'
              outputs combined with the gates; both gradients
ExpertLinear  the products of sorted rows with their experts' weights; the
              gradients of rows and weights

As for the objects of ``objectives``: an object owns its outputs, sized for the
largest call; a call returns views of them, which the next call of the same
object overwrites, on the object's stream, whose memory they are. Nothing is
synchronised. Every output may also be given by the caller (`out` and its
like), so that several micro-batches keep theirs. The formulas stand at the C
functions in include/vsf.h.

Rows behind the last one that holds a choice (rows from starts[-1] on) are left
as they were, in the object's outputs and in given ones. The object's hold
zeros there at first, and after that what earlier calls with more choices left:
a call's result is the first starts[-1] rows alone. The calls here go by that.
What a program computes over whole arrays in between (a bias' gradient
d_y.sum(0), a largest absolute value) has to leave the others out, for instance
by torch.where(source[:, None] >= 0, d_y, 0), which waits for nothing.
"""
from __future__ import annotations

import torch

from . import vsf as V
from .objectives import _Objective


class _Rows(_Objective):
    def _check(self, x, rows: int, width: int, what: str) -> int:
        """Checks a matrix of exactly `rows` rows; its row stride."""
        shape = x.shape
        if x.dtype is not self.dtype or len(shape) != 2 or shape[0] != rows or shape[1] != width \
                or x.get_device() != self._index:
            raise ValueError(f"{what}: expected {self.dtype} [{rows}, {width}] on {self.device}, got "
                             f"{x.dtype} {tuple(shape)} on {x.device}")
        ld, unit = x.stride()
        if unit != 1 and width > 1:
            raise ValueError(f"{what}: the elements of a row must be adjacent (stride {unit})")
        if rows <= 1:  # (no stride to speak of)
            return self._padded(width)
        if ld < width:
            raise ValueError(f"{what}: rows overlap (stride {ld}, {width} elements)")
        return ld

    def _padded(self, width: int) -> int:
        step = 16 // self.dtype.itemsize
        return -(-width // step) * step

    def _matrix(self, *shape, zero: bool = True):
        """An output whose rows start on 16-byte boundaries."""
        with torch.cuda.stream(self.stream):
            make = torch.zeros if zero else torch.empty
            return make(*shape[:-1], self._padded(shape[-1]), dtype=self.dtype,
                        device=self.device)[..., :shape[-1]]

    def _output(self, given, own, rows: int, width: int, what: str):
        """The first rows of an output of the object's own, or of the one given;
        its address and row stride."""
        if given is not None:
            ld = self._check(given, rows, width, what)
            return given, given.data_ptr(), ld
        if own is None:
            raise ValueError(f"{what}: none of the object's own (with_grad=False) and none given")
        ld = self._padded(width)
        if rows != own.shape[0]:
            own = own[:rows]
        return own, own.data_ptr(), ld


class Dispatch(_Rows):
    """Tokens to their experts and back, for idx of ``Router.forward``.

    sort(idx) -> (starts [E + 1], source [T top_k], place [T, top_k]), int32;
    the other calls go by the last sort. gather(x) -> rows [T top_k, hidden] in
    the experts' order; combine(y, gates) -> out [T, hidden];
    combine_backward(d_out, y, gates) -> (d_y, d_gates [T, top_k] fp32);
    gather_backward(d_rows) -> d_x. `calls` counts the sorts: a program that may
    sort again in between keeps the number and gives it as `call` to the other
    calls, which refuse if it is not the last one's any more. With
    with_grad=False there are no buffers for gradients: give them, or leave the
    backward calls alone."""

    def __init__(self, tokens: int, experts: int, top_k: int, hidden: int, *, dtype=torch.bfloat16,
                 with_grad: bool = True, device=None, stream=None):
        super().__init__(tokens, hidden, dtype, device, stream)
        self.experts, self.top_k = int(experts), int(top_k)
        nbytes = V.vsf_expert_sort_workspace_bytes(self.tokens, self.top_k, self.experts)
        if not nbytes:
            raise ValueError(f"sizes out of range: {tokens} tokens, {top_k} of {experts} experts")
        self.workspace = self._new(nbytes, dtype=torch.uint8)
        i32, n = torch.int32, self.tokens * self.top_k
        self.starts = self._new(self.experts + 1, dtype=i32)
        self.source = self._new(n, dtype=i32)
        self.place = self._new(self.tokens, self.top_k, dtype=i32)
        self.rows = self._matrix(n, self.width)
        self.out = self._matrix(self.tokens, self.width)
        self.d_y = self.d_gates = self.d_x = None
        if with_grad:
            self.d_y = self._matrix(n, self.width)
            self.d_gates = self._new(self.tokens, self.top_k)
            self.d_x = self._matrix(self.tokens, self.width)
        self._at = [t.data_ptr() for t in (self.starts, self.source, self.place, self.workspace)]
        self._bytes = nbytes
        self.calls, self._n = 0, None

    def _sorted(self, call) -> int:
        if self._n is None:
            raise ValueError("sort first")
        if call is not None and call != self.calls:
            raise ValueError(f"of sort {call}: sort {self.calls} has followed it")
        return self._n

    def sort(self, idx):
        shape = idx.shape
        if len(shape) != 2 or shape[0] > self.tokens or shape[1] != self.top_k:
            raise ValueError(f"idx: expected [<= {self.tokens}, {self.top_k}], got {tuple(shape)}")
        n = shape[0]
        at = self._vec(idx, n * self.top_k, torch.int32, "idx")
        V.vsf_expert_sort(at, n, self.top_k, self.experts, *self._at, self._bytes, self._st)
        self.calls += 1
        self._n = n
        if n == self.tokens:
            return self.starts, self.source, self.place
        return self.starts, self.source[:n * self.top_k], self.place[:n]

    def gather(self, x, out=None, call: int | None = None):
        n = self._sorted(call)
        ld = self._check(x, n, self.width, "x")
        out, at, out_ld = self._output(out, self.rows, n * self.top_k, self.width, "out")
        V.vsf_expert_gather(x.data_ptr(), self._vdt, n, self.width, ld, self._at[2], self.top_k, at,
                            out_ld, self._st)
        return out

    def _combine(self, y, gates, out, own, call, what):
        n = self._sorted(call)
        ld = self._check(y, n * self.top_k, self.width, what)
        out, at, out_ld = self._output(out, own, n, self.width, "out")
        g = self._vec(gates, n * self.top_k, torch.float32, "gates")
        V.vsf_expert_combine(y.data_ptr(), self._vdt, n, self.width, ld, self._at[2], g, self.top_k,
                             at, out_ld, self._st)
        return out

    def combine(self, y, gates, out=None, call: int | None = None):
        return self._combine(y, gates, out, self.out, call, "y")

    def gather_backward(self, d_rows, out=None, call: int | None = None):
        return self._combine(d_rows, None, out, self.d_x, call, "d_rows")

    def combine_backward(self, d_out, y, gates, d_y=None, d_gates=None, call: int | None = None):
        n = self._sorted(call)
        k = self.top_k
        ld = self._check(d_out, n, self.width, "d_out")
        y_ld = self._check(y, n * k, self.width, "y")
        d_y, at, d_ld = self._output(d_y, self.d_y, n * k, self.width, "d_y")
        if gates is None:
            raise ValueError("gates: needed")
        if d_gates is None:
            if self.d_gates is None:
                raise ValueError("d_gates: none of the object's own (with_grad=False) and none given")
            d_gates = self._first(self.d_gates, n)
        V.vsf_expert_combine_grad(d_out.data_ptr(), self._vdt, n, self.width, ld, y.data_ptr(), y_ld,
                                  self._at[2], self._vec(gates, n * k, torch.float32, "gates"), k,
                                  at, d_ld,
                                  self._vec(d_gates, n * k, torch.float32, "d_gates"), self._st)
        return d_y, d_gates

    def device_error(self) -> int:
        """Always 0: these calls have no wait that could run out, and whatever
        their indexes hold is checked."""
        return 0


class ExpertLinear(_Rows):
    """y[r] = weight[e] x[r] for the rows r of expert e, as Dispatch.sort's starts
    give them; bfloat16, accumulated in fp32. `rows` is the most rows of a call
    (tokens * top_k), weight [experts, out_features, in_features].

    forward(x, weight, starts) -> y; backward_input(d_y, weight, starts) -> d_x;
    backward_weight(d_y, x, starts) -> d_weight (zeros for experts without a
    row). Rows of every tensor start on 16-byte boundaries (strides of whole 8
    elements); the sizes themselves may be odd."""

    def __init__(self, rows: int, experts: int, out_features: int, in_features: int, *,
                 with_grad: bool = True, device=None, stream=None):
        super().__init__(rows, in_features, torch.bfloat16, device, stream)
        if experts < 1 or out_features < 1:
            raise ValueError(f"sizes out of range: {experts} experts, {out_features} features")
        self.experts, self.out_features = int(experts), int(out_features)
        self.in_features = self.width
        with torch.cuda.stream(self.stream):
            self.workspace = torch.zeros(16, dtype=torch.uint8, device=self.device)
        self._ws = self.workspace.data_ptr()
        self.y = self._matrix(self.tokens, self.out_features)
        self.d_x = self.d_weight = None
        if with_grad:
            self.d_x = self._matrix(self.tokens, self.in_features)
            self.d_weight = self._matrix(self.experts, self.out_features, self.in_features, zero=False)

    def _weight(self, w, what: str):
        """Checks weights (or their gradient); strides of rows and experts."""
        shape = (self.experts, self.out_features, self.in_features)
        if w.dtype is not self.dtype or tuple(w.shape) != shape or w.get_device() != self._index:
            raise ValueError(f"{what}: expected {self.dtype} {shape} on {self.device}, got {w.dtype} "
                             f"{tuple(w.shape)} on {w.device}")
        stride, ld, unit = w.stride()
        if unit != 1 and shape[2] > 1:
            raise ValueError(f"{what}: the elements of a row must be adjacent (stride {unit})")
        if shape[1] == 1:
            ld = self._padded(shape[2])
        return ld, stride

    def _rows_of(self, x, width: int, what: str):
        if x.dim() != 2 or x.shape[0] > self.tokens:
            raise ValueError(f"{what}: expected [<= {self.tokens}, {width}], got {tuple(x.shape)}")
        return x.shape[0], self._check(x, x.shape[0], width, what)

    def _starts(self, starts):
        return self._vec(starts, self.experts + 1, torch.int32, "starts")

    def forward(self, x, weight, starts, out=None):
        n, ld = self._rows_of(x, self.in_features, "x")
        w_ld, w_stride = self._weight(weight, "weight")
        out, at, out_ld = self._output(out, self.y, n, self.out_features, "out")
        V.vsf_expert_product(x.data_ptr(), n, self.in_features, ld, weight.data_ptr(), self.experts,
                             self.out_features, w_ld, w_stride, self._starts(starts), at, out_ld,
                             self._ws, self._st)
        return out

    def backward_input(self, d_y, weight, starts, out=None):
        n, ld = self._rows_of(d_y, self.out_features, "d_y")
        w_ld, w_stride = self._weight(weight, "weight")
        out, at, out_ld = self._output(out, self.d_x, n, self.in_features, "out")
        V.vsf_expert_product_input_grad(d_y.data_ptr(), n, self.out_features, ld, weight.data_ptr(),
                                        self.experts, self.in_features, w_ld, w_stride,
                                        self._starts(starts), at, out_ld, self._ws, self._st)
        return out

    def backward_weight(self, d_y, x, starts, out=None):
        n, ld = self._rows_of(d_y, self.out_features, "d_y")
        x_ld = self._check(x, n, self.in_features, "x")
        if out is None:
            if self.d_weight is None:
                raise ValueError("out: none of the object's own (with_grad=False) and none given")
            out = self.d_weight
        w_ld, w_stride = self._weight(out, "out")
        V.vsf_expert_product_weight_grad(d_y.data_ptr(), n, self.out_features, ld, x.data_ptr(),
                                         self.in_features, x_ld, self.experts, self._starts(starts),
                                         out.data_ptr(), w_ld, w_stride, self._ws, self._st)
        return out
