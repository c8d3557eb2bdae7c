"""Device-resident DeepSeekMoE layer: uploads weights once, owns the workspaces,
and calls ``moe_forward`` on each batch and ``moe_backward`` for its gradient.
Memory management only; the layer's arithmetic is entirely in libmoe's kernels.

For an e4m3 layer the bf16 master weights are uploaded and block-quantised on
the device by ``moe_quantize_weights_128x128`` (128 x 128 blocks, §3.3 of the
"DeepSeek-V3 Technical Report" page); the master copy is then released.
"""
from __future__ import annotations

import contextlib
import math

import numpy as np
import torch

from . import (MOE_BF16, MOE_E4M3, MOE_F32, MOE_WS_FORWARD, MOE_WS_PERMUTE, MoeShape, make_gate_rule, make_shape,
               moe_backward, moe_backward_workspace_bytes, moe_combine, moe_dequantize_mx4, moe_ffn_mx4_workspace_bytes,
               moe_forward, moe_gate, moe_gate_backward, moe_grouped_ffn_mx4, moe_grouped_product, moe_grouped_product_dw,
               moe_grouped_product_dx, moe_grouped_product_int8, moe_orthogonalize, moe_orthogonalize_workspace_bytes,
               moe_permute, moe_quantize_int8, moe_quantize_mx4, moe_quantize_weights_128x128, moe_transpose_expert_weights,
               moe_workspace_bytes)
from . import _stream as _raw


def to_device(a: np.ndarray, device="cuda") -> torch.Tensor:
    """numpy float32 / bf16 bits (uint16) / int32 / uint8 -> device tensor of the same storage."""
    if a.dtype == np.uint16:
        return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).to(device).view(torch.bfloat16)
    return torch.from_numpy(np.ascontiguousarray(a)).to(device)


def to_host(t: torch.Tensor) -> np.ndarray:
    """Inverse of to_device: bf16 comes back as uint16 bit patterns, e4m3 as uint8 codes."""
    t = t.detach()
    if t.dtype == torch.bfloat16:
        return t.view(torch.int16).cpu().numpy().view(np.uint16)
    if t.dtype == torch.float8_e4m3fn:
        return t.view(torch.uint8).cpu().numpy()
    return t.cpu().numpy()


def quantize_weights_128x128(w: torch.Tensor, stream=None):
    """[n, rows, cols] bf16/fp32 device tensor -> (e4m3 codes uint8, fp32 scales [n, rows/128, cols/128])."""
    n, rows, cols = w.shape
    q = torch.empty((n, rows, cols), dtype=torch.uint8, device=w.device)
    s = torch.empty((n, rows // 128, cols // 128), dtype=torch.float32, device=w.device)
    dt = MOE_BF16 if w.dtype == torch.bfloat16 else MOE_F32
    moe_quantize_weights_128x128(n, rows, cols, dt, w, q, s, stream)
    return q, s


def _torch_stream(stream, device) -> torch.cuda.Stream:
    """The torch stream of what the entry points take as one (a torch stream, a handle, None)."""
    if stream is None:
        return torch.cuda.current_stream(device)
    if isinstance(stream, int):
        return torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
    if stream.device != torch.device(device):
        raise ValueError("a stream of %s expected, not of %s" % (device, stream.device))
    return stream


def _on(stream, device):
    """What is allocated inside belongs to `stream`: once dropped, its memory is reused behind that stream's work alone."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(_torch_stream(stream, device))


def _float_type(t: torch.Tensor) -> int:
    if t.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("bf16 or fp32 expected, not %s" % t.dtype)
    return MOE_BF16 if t.dtype == torch.bfloat16 else MOE_F32


def _row_stride(t: torch.Tensor) -> int:
    """Elements from row to row of a matrix whose rows are contiguous and do not overlap."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < t.shape[1]):
        raise ValueError("a matrix of contiguous rows expected, not strides %s" % (t.stride(),))
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _check(name, t, device, dtypes, shape, dense=True):
    """The entry points take bare pointers: refuses a tensor that is not what the kernels will read or write."""
    if t.device != device or t.dtype not in dtypes or t.shape != shape or (dense and not t.is_contiguous()):
        raise ValueError("%s: %s%s of %s on %s expected, not %s of %s on %s" % (
            name, "contiguous " if dense else "", list(shape), " or ".join(map(str, dtypes)), device, list(t.shape), t.dtype,
            t.device))


def _on_gpu(*tensors):
    if any(not t.is_cuda or t.device != tensors[0].device for t in tensors):
        raise ValueError("tensors on one GPU expected, not on %s" % ", ".join(str(t.device) for t in tensors))


def quantize_mx4(x: torch.Tensor, stream=None):
    """bf16/fp32 device tensor [..., cols] whose rows are contiguous and evenly spaced -> MX4
    (codes [..., 64 R], scales [..., 4 R]), uint8, R = ceil(cols / 128)."""
    _on_gpu(x)
    cols = x.shape[-1]
    rows = x.view(-1, cols) if x.numel() else x.reshape(0, cols)
    runs = -(-cols // 128)
    with _on(stream, x.device):
        q = torch.empty(x.shape[:-1] + (64 * runs,), dtype=torch.uint8, device=x.device)
        s = torch.empty(x.shape[:-1] + (4 * runs,), dtype=torch.uint8, device=x.device)
    moe_quantize_mx4(rows.shape[0], cols, _float_type(x), rows, _row_stride(rows), q, s, stream)
    return q, s


def dequantize_mx4(q: torch.Tensor, s: torch.Tensor, cols: int, dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """The values [..., cols] that MX4 codes and scales stand for (exact in bf16 and fp32)."""
    _on_gpu(q, s)
    if cols <= 0 or q.dtype != torch.uint8 or s.dtype != torch.uint8:
        raise ValueError("uint8 codes and scales of rows of at least one value expected")
    runs = -(-cols // 128)
    if q.shape[-1] != 64 * runs or s.shape != q.shape[:-1] + (4 * runs,) or not (q.is_contiguous() and s.is_contiguous()):
        raise ValueError("codes [..., %d] and scales [..., %d], contiguous, expected" % (64 * runs, 4 * runs))
    with _on(stream, q.device):
        y = torch.empty(q.shape[:-1] + (cols,), dtype=dtype, device=q.device)
    moe_dequantize_mx4(y.numel() // cols, cols, q, s, _float_type(y), y, cols, stream)
    return y


# ---- products of experts ------------------------------------------------------------------------
# Autograd does not record these calls, also where an input requires a gradient: gradients are calls of their own.


@contextlib.contextmanager
def _at(stream, device):
    """`device` and `stream` (its current one if None) are the current ones inside."""
    with torch.cuda.device(device), torch.cuda.stream(_torch_stream(stream, device)):
        yield


def _batch(offsets, gather, n, rows, device):
    """Checks the experts' bounds and the rows' tokens; the number of rows."""
    _check("offsets", offsets, device, (torch.int32,), (n + 1,))
    if gather is None:
        return rows
    _check("gather", gather, device, (torch.int32,), (gather.numel(),))
    return gather.numel()


def _out(name, out, shape, dtype, device, *inputs):
    if dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("%s: bf16 or fp32 expected, not %s" % (name, dtype))
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _check(name, out, device, (dtype,), shape, dense=False)
    _apart(name, out, *inputs)
    return out


def _place(t):
    """First byte, bytes of a row, bytes from row to row and the byte behind the last of a matrix of rows or a dense tensor."""
    size = t.element_size()
    rows, cols, ld = (1, t.numel(), t.numel()) if t.is_contiguous() else (*t.shape, _row_stride(t))
    return t.data_ptr(), cols * size, ld * size, t.data_ptr() + ((rows - 1) * ld + cols) * size


def _apart(name, out, *inputs):
    """Refuses a result over an input: kernels write it while they still read.  Columns of one buffer beside each other are
    apart."""
    first, width, step, end = _place(out)
    for t in inputs:
        at, w, ld, behind = _place(t)
        if not out.numel() or not t.numel() or first >= behind or at >= end:
            continue
        # rows at multiples of `every`: apart where the one's columns lie in the gap behind the other's
        every = math.gcd(step, ld)
        if w <= (first - at) % every <= every - width:
            continue
        raise ValueError("%s shares memory with an input" % name)


def grouped_product(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, gather: torch.Tensor = None,
                    dtype=torch.bfloat16, out: torch.Tensor = None, stream=None) -> torch.Tensor:
    """y[r] = w[e] x[gather[r]] for the rows offsets[e] <= r < offsets[e + 1] of expert e.

    x [tokens][in] bf16 (rows may be padded), w [n][out][in] bf16, offsets [n + 1] and gather [rows] int32 (None: a row for
    each token), all on one GPU; y [rows][out] bf16 or fp32.  Rows from offsets[n] on are left as they were; out shares no memory
    with the inputs.  Autograd does not record it: grouped_product_dx and grouped_product_dw are its gradients."""
    _on_gpu(x, w, offsets)
    n, cout, cin = w.shape
    _check("x", x, w.device, (torch.bfloat16,), (x.shape[0], cin), dense=False)
    _check("w", w, w.device, (torch.bfloat16,), w.shape)
    rows = _batch(offsets, gather, n, x.shape[0], w.device)
    with _at(stream, w.device):
        y = _out("out", out, (rows, cout), dtype, w.device, x, w)
        moe_grouped_product(n, offsets, rows, gather, cin, cout, x, _row_stride(x), w, _float_type(y), y, _row_stride(y))
    return y


def grouped_product_dx(dy: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, dtype=torch.bfloat16,
                       out: torch.Tensor = None, stream=None) -> torch.Tensor:
    """The gradient of grouped_product at the rows of x: dx[r] = w[e]^T dy[r], [rows][in], from dy [rows][out] bf16.  A token's
    gradient is the sum of its rows'."""
    _on_gpu(dy, w, offsets)
    n, cout, cin = w.shape
    _check("dy", dy, w.device, (torch.bfloat16,), (dy.shape[0], cout), dense=False)
    _check("w", w, w.device, (torch.bfloat16,), w.shape)
    rows = _batch(offsets, None, n, dy.shape[0], w.device)
    with _at(stream, w.device):
        dx = _out("out", out, (rows, cin), dtype, w.device, dy, w)
        moe_grouped_product_dx(n, offsets, rows, cin, cout, dy, _row_stride(dy), w, _float_type(dx), dx, _row_stride(dx))
    return dx


def grouped_product_dw(x: torch.Tensor, dy: torch.Tensor, offsets: torch.Tensor, gather: torch.Tensor = None,
                       dtype=torch.float32, add_to: torch.Tensor = None, stream=None) -> torch.Tensor:
    """The gradient of grouped_product at w: dw[e] = the sum over the expert's rows of dy[r] x[gather[r]]^T, [n][out][in].
    add_to: an fp32 gradient that the sums are added to, in place."""
    _on_gpu(x, dy, offsets)
    n, cin, cout = offsets.numel() - 1, x.shape[1], dy.shape[1]
    _check("x", x, x.device, (torch.bfloat16,), (x.shape[0], cin), dense=False)
    rows = _batch(offsets, gather, n, x.shape[0], x.device)
    _check("dy", dy, x.device, (torch.bfloat16,), (rows, cout), dense=False)
    with _at(stream, x.device):
        if add_to is not None:
            _check("add_to", add_to, x.device, (torch.float32,), (n, cout, cin))
        dw = _out("dw", add_to, (n, cout, cin), torch.float32 if add_to is not None else dtype, x.device, x, dy)
        moe_grouped_product_dw(n, offsets, rows, gather, cin, cout, x, _row_stride(x), dy, _row_stride(dy), _float_type(dw),
                               dw, add_to is not None)
    return dw


def quantize_int8(x: torch.Tensor, stream=None):
    """bf16/fp32 device tensor [..., cols] whose rows are contiguous and evenly spaced -> (codes [..., 128 R] int8 with zeros
    behind the last value, scales [...] fp32), R = ceil(cols / 128): a scale a token, or for weights one an output channel."""
    _on_gpu(x)
    cols = x.shape[-1]
    rows = x.view(-1, cols) if x.numel() else x.reshape(0, cols)
    with _at(stream, x.device):
        q = torch.empty(x.shape[:-1] + (-(-cols // 128) * 128,), dtype=torch.int8, device=x.device)
        s = torch.empty(x.shape[:-1], device=x.device)
        moe_quantize_int8(rows.shape[0], cols, _float_type(x), rows, _row_stride(rows), q, s)
    return q, s


def grouped_product_int8(x: torch.Tensor, x_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor, cols: int,
                         offsets: torch.Tensor, gather: torch.Tensor = None, dtype=torch.bfloat16,
                         out: torch.Tensor = None, stream=None) -> torch.Tensor:
    """grouped_product of quantize_int8's tokens x [tokens][128 R], x_scales [tokens] and weights w [n][out][128 R], w_scales
    [n][out], of `cols` values a row.  It has no gradient."""
    _on_gpu(x, x_scales, w, w_scales, offsets)
    n, cout = w_scales.shape
    run = -(-cols // 128) * 128
    _check("x", x, w.device, (torch.int8,), (x.shape[0], run))
    _check("x_scales", x_scales, w.device, (torch.float32,), (x.shape[0],))
    _check("w", w, w.device, (torch.int8,), (n, cout, run))
    _check("w_scales", w_scales, w.device, (torch.float32,), (n, cout))
    rows = _batch(offsets, gather, n, x.shape[0], w.device)
    with _at(stream, w.device):
        y = _out("out", out, (rows, cout), dtype, w.device, x, x_scales, w, w_scales)
        moe_grouped_product_int8(n, offsets, rows, gather, cols, cout, x, x_scales, w, w_scales, _float_type(y), y,
                                 _row_stride(y))
    return y


NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)


def orthogonalize(g: torch.Tensor, steps: int = 5, coefficients=None, eps: float = 1e-7, scale: float = 1.0,
                  out: torch.Tensor = None, stream=None) -> torch.Tensor:
    """scale times the matrices g [..., rows, cols] (bf16 or fp32, contiguous) brought near their nearest orthogonal ones by
    Newton-Schulz steps, bf16.  coefficients: (a, b, c) for all steps or a list of them (default NEWTON_SCHULZ).  out may be g in
    bf16; otherwise they share no memory."""
    _on_gpu(g)
    _check("g", g, g.device, (torch.bfloat16, torch.float32), g.shape)
    rows, cols = g.shape[-2:]
    n = g.numel() // max(1, rows * cols)
    c = [tuple(v) for v in coefficients] if coefficients is not None and not isinstance(coefficients[0], (int, float)) \
        else [tuple(coefficients or NEWTON_SCHULZ)] * steps
    if len(c) != steps or any(len(v) != 3 for v in c):
        raise ValueError("three coefficients for each of %d steps expected" % steps)
    with _at(stream, g.device):
        if out is None:
            out = torch.empty(g.shape, dtype=torch.bfloat16, device=g.device)
        _check("out", out, g.device, (torch.bfloat16,), g.shape)
        if n == 0:
            return out
        ws = torch.empty(moe_orthogonalize_workspace_bytes(n, rows, cols), dtype=torch.uint8, device=g.device)
        moe_orthogonalize(n, rows, cols, _float_type(g), g, steps, [x for v in c for x in v], eps, scale, out, ws)
    return out


class MoeLayer:
    def __init__(self, shape: MoeShape, gate_w, bias, routed_w, shared_w=None, routed_s=None, shared_s=None):
        self.shape = shape
        self.gate_w = gate_w
        self.bias = bias
        self.routed_w = tuple(routed_w)
        self.shared_w = tuple(shared_w) if shared_w is not None else None
        self.routed_s = tuple(routed_s) if routed_s is not None else None
        self.shared_s = tuple(shared_s) if shared_s is not None else None
        self._ws = None
        self._ws_T = -1
        self._bws = None
        self._bws_T = -1
        self._wt = None

    @classmethod
    def from_host(cls, shape: MoeShape, gate_w, bias, wg, wu, wd, swg=None, swu=None, swd=None, device="cuda"):
        """Upload host master weights (numpy); quantise them on the device when
        the shape's expert dtype is e4m3."""
        g = to_device(gate_w, device)
        b = to_device(np.asarray(bias, np.float32), device)
        fp8 = shape.w_dtype == MOE_E4M3

        def up(ws):
            if ws[0] is None:
                return None, None
            if not fp8:
                return tuple(to_device(w, device) for w in ws), None
            qs, ss = [], []
            for w in ws:
                dw = to_device(w, device)
                q, s = quantize_weights_128x128(dw)
                del dw
                qs.append(q)
                ss.append(s)
            return tuple(qs), tuple(ss)

        rw, rs = up((wg, wu, wd))
        sw, ss = up((swg, swu, swd))
        torch.cuda.synchronize()
        return cls(shape, g, b, rw, sw, rs, ss)

    def workspace(self, T: int) -> torch.Tensor:
        if self._ws is None or self._ws_T != T:
            self.shape.T = T
            n = moe_workspace_bytes(self.shape, MOE_WS_FORWARD)
            self._ws = torch.empty(max(n, 256), dtype=torch.uint8, device=self.gate_w.device)
            self._ws_T = T
        return self._ws

    def forward(self, u: torch.Tensor, out: torch.Tensor = None, topk_idx=None, topk_w=None, counts=None,
                scores=None, stream=None) -> torch.Tensor:
        T = u.shape[0]
        ws = self.workspace(T)
        self.shape.T = T
        if out is None:
            out = torch.empty((T, self.shape.d), dtype=u.dtype, device=u.device)
        moe_forward(self.shape, u, self.gate_w, self.bias, self.routed_w, self.routed_s, self.shared_w,
                    self.shared_s, out, topk_idx, topk_w, counts, scores, ws, stream)
        return out

    # ---- backward -----------------------------------------------------------

    def transposed_weights(self, stream=None):
        """(routed, shared) transposed copies ((W_down^T [n, I, d], [W_gate^T | W_up^T] [n, d, 2I]),
        e4m3 block scales or None) that the backward reads; built on first use.  Call
        drop_transposed() after changing the weights."""
        if self._wt is None:
            d, I = self.shape.d, self.shape.inter
            fp8 = self.shape.w_dtype == MOE_E4M3

            def tr(ws, ss):
                if ws is None:
                    return None, None
                wg, wu, wd = ws
                n = wg.shape[0]
                wdt = torch.empty((n, I, d), dtype=wd.dtype, device=wd.device)
                wgut = torch.empty((n, d, 2 * I), dtype=wg.dtype, device=wg.device)
                st = None
                if fp8:
                    st = (torch.empty((n, I // 128, d // 128), dtype=torch.float32, device=wd.device),
                          torch.empty((n, d // 128, 2 * I // 128), dtype=torch.float32, device=wd.device))
                moe_transpose_expert_weights(self.shape, n, ws, ss, (wdt, wgut), st, stream)
                return (wdt, wgut), st

            self._wt = (tr(self.routed_w, self.routed_s), tr(self.shared_w, self.shared_s))
        return self._wt

    def drop_transposed(self):
        self._wt = None

    def backward(self, u: torch.Tensor, dout: torch.Tensor, du: torch.Tensor = None, dgate_w=None, d_routed_w=None,
                 d_shared_w=None, dtopk_w=None, stream=None) -> torch.Tensor:
        """Gradients for the most recent forward(u) (its workspace holds the saved
        activations, so no other forward may run in between).  du is returned;
        dgate_w [N_r, d] fp32, d_routed_w / d_shared_w (dW_gate, dW_up, dW_down) and
        dtopk_w [T, K] fp32 are filled when given."""
        T = u.shape[0]
        if self._ws is None or self._ws_T != T:
            raise ValueError("backward needs the workspace of a forward call on the same batch")
        (rt, rts), (st, sts) = self.transposed_weights(stream)
        self.shape.T = T
        if self._bws is None or self._bws_T != T:
            n = moe_backward_workspace_bytes(self.shape)
            self._bws = torch.empty(max(n, 256), dtype=torch.uint8, device=u.device)
            self._bws_T = T
        if du is None:
            du = torch.empty((T, self.shape.d), dtype=u.dtype, device=u.device)
        moe_backward(self.shape, u, self.gate_w, self.routed_w, self.routed_s, rt, rts, self.shared_w, self.shared_s,
                     st, sts, self._ws, dout, du, dgate_w, d_routed_w, d_shared_w, dtopk_w, self._bws, stream)
        return du


class Mx4Experts:
    """The routed and shared experts of a layer in MX4, behind a gate whose logits the caller computes:
    choice and weights (moe_gate), dispatch (moe_permute), rounding of the tokens (moe_quantize_mx4), the
    experts (moe_grouped_ffn_mx4, the shared ones as further experts over all tokens) and moe_combine.

    w_gate, w_up [n][inter][d], w_down [n][d][inter] are bf16 or fp32 device tensors of the n_routed experts
    and then the n_shared ones; they are rounded once and not kept.  rule: make_gate_rule's keywords beside T,
    n_experts and topk.  d has to be a multiple of 128, inter may be any size.

    Buffers hold the largest batch so far and are shared by all calls: calls on different streams have to be ordered by
    the caller, as for every workspace, and topk_idx, topk_w and counts hold the last call's choice.  A call's results
    belong to its stream.  A captured call uses the buffers of its time, which the layer keeps from then on: running the
    largest batch before capturing keeps one set."""

    def __init__(self, w_gate, w_up, w_down, topk, n_shared=0, stream=None, **rule):
        _on_gpu(w_gate, w_up, w_down)
        n, self.inter, self.d = w_gate.shape
        if w_up.shape != w_gate.shape or w_down.shape != (n, self.d, self.inter) or not 0 <= n_shared < n:
            raise ValueError("w_gate and w_up [n][inter][d], w_down [n][d][inter] expected, and fewer shared experts than n")
        self.n_routed, self.n_shared, self.topk, self.rule = n - n_shared, n_shared, topk, rule
        w = [quantize_mx4(x, stream) for x in (w_gate, w_up, w_down)]
        self.codes, self.scales = [q for q, _ in w], [s for _, s in w]
        self.device = w_gate.device
        self._T, self._capacity, self._held, self._captured, self._kept = -1, 0, None, False, []
        self._streams = {_raw(stream)}     # those that own the weights and buffers or were recorded on them

    def _gate_rule(self, logits):
        _check("logits", logits, self.device, (torch.float32, torch.bfloat16), (self._T, self.n_routed), dense=False)
        return make_gate_rule(self._T, self.n_routed, self.topk,
                              logits="bf16" if _float_type(logits) == MOE_BF16 else "fp32", **self.rule)

    def _use(self, stream):
        """Before work on `stream`: weights and buffers that are dropped later are not reused before it has ended."""
        if _raw(stream) not in self._streams:
            for t in self.codes + self.scales + [t for held in self._kept + [self._held or ()] for t in held]:
                t.record_stream(_torch_stream(stream, t.device))
            self._streams.add(_raw(stream))

    def _buffers(self, T, stream):
        """Buffers for T tokens on `stream`."""
        K, Nr, Ns, runs = self.topk, self.n_routed, self.n_shared, -(-self.d // 128)
        device = self.device
        self._use(stream)
        if T > self._capacity or self._held is None:
            # the old ones are released before the larger ones are taken, unless a graph may hold their addresses
            if self._captured:
                self._kept.append(self._held)
            self._T, self._capacity, self._held = -1, 0, None
            self.topk_idx = self.topk_w = self.counts = self._offsets = self._tokens = self._inv = None
            self._xq = self._xs = self._y = self._ws = self._pws = None
            shape = make_shape(T, self.d, Nr, Ns, 1, 1, K, 128)
            with _on(stream, device):
                new = lambda n, dtype: torch.empty(n, dtype=dtype, device=device)  # noqa: E731
                rows = T * (K + Ns)
                self._held = (new((T, K), torch.int32), new((T, K), torch.float32), new((Nr,), torch.int32),
                              new((Nr + Ns + 1,), torch.int32), new((rows,), torch.int32), new((T * K,), torch.int32),
                              new((T, 64 * runs), torch.uint8), new((T, 4 * runs), torch.uint8),
                              new((rows, self.d), torch.bfloat16),
                              new((moe_ffn_mx4_workspace_bytes(rows, self.inter),), torch.uint8),
                              new((max(256, moe_workspace_bytes(shape, MOE_WS_PERMUTE)),), torch.uint8))
            self._capacity, self._streams = T, {_raw(stream)}
        if T != self._T:
            idx, w, counts, offsets, tokens, inv, xq, xs, y, ws, pws = self._held
            rows = T * (K + Ns)
            # dispatch reads the choice's sizes of it, the combine d as well, neither the experts' inner size
            self._shape = make_shape(T, self.d, Nr, Ns, 1, 1, K, 128)
            self.topk_idx, self.topk_w, self.counts, self._offsets = idx[:T], w[:T], counts, offsets
            self._tokens, self._inv, self._xq, self._xs = tokens[:rows], inv[:T * K], xq[:T], xs[:T]
            self._y, self._ws, self._pws = y[:rows], ws, pws
        with _on(stream, device):
            self._captured = self._captured or torch.cuda.is_current_stream_capturing()
        if Ns and T:
            # the shared experts' rows follow the routed ones'.  Their bounds and tokens stay from one batch to the next of
            # its size; once a call has been captured every call writes them, as replays may come between any two
            with _on(stream, device):
                if T != self._T or self._captured:
                    torch.arange(T * K, T * (K + Ns) + 1, T, out=self._offsets[Nr:])
                    for j in range(Ns):
                        torch.arange(T, out=self._tokens[T * (K + j):T * (K + j + 1)])
        self._T = T

    def forward(self, u: torch.Tensor, logits: torch.Tensor, bias: torch.Tensor = None, out: torch.Tensor = None,
                scores: torch.Tensor = None, stream=None) -> torch.Tensor:
        """u [T][d] bf16, logits [T][n_routed] fp32 or bf16 (rows of either may be padded); the choice stays in
        topk_idx, topk_w and counts.  bias [n_routed] fp32; out [T][d] bf16 and scores [T][n_routed] fp32 contiguous."""
        T, fp32 = u.shape[0], (torch.float32,)
        _check("u", u, self.device, (torch.bfloat16,), (T, self.d), dense=False)
        _check("logits", logits, self.device, (torch.float32, torch.bfloat16), (T, self.n_routed), dense=False)
        if bias is not None:
            _check("bias", bias, self.device, fp32, (self.n_routed,))
        if scores is not None:
            _check("scores", scores, self.device, fp32, (T, self.n_routed))
        if out is not None:
            _check("out", out, self.device, (torch.bfloat16,), (T, self.d))
        u_ld, logits_ld = _row_stride(u), _row_stride(logits)
        if out is None:
            with _on(stream, self.device):
                out = torch.empty((T, self.d), dtype=u.dtype, device=self.device)
        self._buffers(T, stream)
        if T == 0:
            with _on(stream, self.device):
                self.counts.zero_()
            return out
        moe_gate(self._gate_rule(logits), logits, logits_ld, bias, scores, self.topk_idx, self.topk_w, stream)
        moe_permute(self._shape, self.topk_idx, None, self.counts, self._offsets, self._tokens, self._inv, None, None,
                    self._pws, stream)
        moe_quantize_mx4(T, self.d, MOE_BF16, u, u_ld, self._xq, self._xs, stream)
        moe_grouped_ffn_mx4(self.n_routed + self.n_shared, self._offsets, T * (self.topk + self.n_shared), self._tokens,
                            self.d, self.inter, self._xq, self._xs, self.codes, self.scales, self._y, self._ws, stream)
        shared = self._y[T * self.topk:] if self.n_shared else None
        moe_combine(self._shape, self._y, self._inv, self.topk_w, shared, None, out, stream)
        return out

    def gate_gradient(self, logits: torch.Tensor, dtopk_w: torch.Tensor, dscores: torch.Tensor = None,
                      stream=None) -> torch.Tensor:
        """dL/dlogits of the most recent forward's choice, from dL/dtopk_w [T][topk] and (optional) dL/dscores
        [T][n_routed], fp32 of any strides (what is not contiguous, as an expanded mean's gradient, is copied)."""
        rule = self._gate_rule(logits)
        _check("dtopk_w", dtopk_w, self.device, (torch.float32,), (self._T, self.topk), dense=False)
        if dscores is not None:
            _check("dscores", dscores, self.device, (torch.float32,), (self._T, self.n_routed), dense=False)
        ld = _row_stride(logits)
        self._use(stream)
        with _on(stream, self.device):
            dtopk_w = dtopk_w.contiguous()
            dscores = None if dscores is None else dscores.contiguous()
            dlogits = torch.empty(logits.shape, dtype=logits.dtype, device=self.device)
        moe_gate_backward(rule, logits, ld, self.topk_idx, self.topk_w, dtopk_w, dscores, dlogits,
                          self.n_routed, stream)
        return dlogits
