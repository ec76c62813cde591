"""The trainable frame around the tensor product: the embedding that makes the
first node features, the per-irrep norm and gated residual around a block, and
the AdamW step over a network's parameters.

As in the rest of the binding, this marshals torch CUDA tensors into the C ABI
and the current torch stream; the computation runs in the library's kernels.
"""
from __future__ import annotations

import ctypes
import functools
import operator

import numpy as np
import torch

from . import BF16, F16, F32, F64, CgtpError, _AdamwArgs, _check, _need, _Rows, _stream, lib

_TYPES = {torch.float32: F32, torch.float64: F64, torch.bfloat16: BF16, torch.float16: F16}
_NONE = _Rows(None, 0)

# The small calls here are as long as their Python: the raw stream spares a
# Stream object a call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on():
    """The current stream's handle."""
    return _stream() if _raw_stream is None else _raw_stream(_device())


_facts = operator.attrgetter("shape", "dtype", "is_cuda")


def _at(t):
    return None if t is None else t.data_ptr()


def _type(dtype) -> int:
    if dtype not in _TYPES:
        raise CgtpError(f"unsupported dtype {dtype}")
    return _TYPES[dtype]


def _rows(t, name, dtype, n, width):
    """Rows of a tensor, which may lie further apart than they are wide."""
    if t is None:
        return _NONE
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise CgtpError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise CgtpError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != (n, width):
        raise CgtpError(f"{name} has shape {tuple(t.shape)}, expected {(n, width)}")
    step, inner = t.stride()
    if inner != 1 and width != 1:
        raise CgtpError(f"{name} must have contiguous rows")
    return _Rows(t.data_ptr(), step if n > 1 else width)


def _scratch(nbytes, device):
    return torch.empty(max(256, nbytes), dtype=torch.uint8, device=device)


# ------------------------------------------------------------- embedding --

def _index(index):
    if not isinstance(index, torch.Tensor) or not index.is_cuda:
        raise CgtpError("index must be a CUDA tensor")
    if index.dtype not in (torch.int32, torch.int64) or index.dim() != 1:
        raise CgtpError(f"index must be a row of int32 or int64, got {index.dtype} of "
                        f"{index.dim()} dimensions")
    if not index.is_contiguous():
        raise CgtpError("index must be contiguous")
    return index.element_size() * 8


def embed_forward(index, table, scale: float = 1.0, out=None):
    """out[n] = scale * table[index[n]].  index [N] int32 or int64 (negative:
    padding, a zero row); table [V, D] fp32, fp64, bfloat16 or binary16.  ``out``
    [N, D] may be a block of wider rows, such as the scalar channels of a
    feature row; the rest of those rows is left as it is."""
    bits = _index(index)
    _need(table, "table", table.dtype)
    if table.dim() != 2:
        raise CgtpError(f"table has {table.dim()} dimensions, expected 2")
    n, (v, d) = index.shape[0], table.shape
    if out is None:
        out = torch.empty(n, d, dtype=table.dtype, device=table.device)
        o, step = out.data_ptr(), d
    else:
        o = _rows(out, "out", table.dtype, n, d)
        o, step = o.data, o.stride
    _check(lib().cgtp_embed_forward(_type(table.dtype), bits, n, v, d, index.data_ptr(),
                                    table.data_ptr(), float(scale), o, step, _on()))
    return out


@functools.lru_cache(maxsize=256)
def _embed_workspace(ty, n, v, d) -> int:
    nb = ctypes.c_size_t()
    _check(lib().cgtp_embed_backward_workspace(ty, n, v, d, ctypes.byref(nb)))
    return nb.value


def embed_backward(index, grad_out, n_rows: int, scale: float = 1.0, out=None, workspace=None):
    """The gradient of embed_forward's table [n_rows, D]: scale times the sum of
    the rows of grad_out [N, D] at each index, zero rows where there is none.
    Deterministic."""
    bits = _index(index)
    n = index.shape[0]
    if not isinstance(grad_out, torch.Tensor) or grad_out.dim() != 2:
        raise CgtpError("grad_out must be a tensor of rows")
    d = grad_out.shape[1]
    g = _rows(grad_out, "grad_out", grad_out.dtype, n, d)
    if out is None:
        out = torch.empty(n_rows, d, dtype=grad_out.dtype, device=grad_out.device)
    else:
        _need(out, "out", grad_out.dtype, (n_rows, d))
    ty = _type(grad_out.dtype)
    if workspace is None:
        nb = _embed_workspace(ty, n, n_rows, d)
        workspace = _scratch(nb, grad_out.device) if nb else None
    nws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().cgtp_embed_backward(ty, bits, n, n_rows, d, index.data_ptr(), g.data, g.stride,
                                     float(scale), out.data_ptr(), _at(workspace), nws, _on()))
    return out


def embed_device_status() -> int:
    """1 if an index past the table was met since the last query, then cleared
    (synchronous)."""
    c = ctypes.c_int()
    _check(lib().cgtp_embed_device_status(ctypes.byref(c)))
    return c.value


# ---------------------------------------------- norms and gated residuals --

class IrrepsNorm:
    """Equivariant RMS norm of feature rows (``irreps``), alone and fused with
    the gate, the residual scale and the next norm after a block:

        norm(b) = b * weight / sqrt(mean over the irrep of b^2 + eps)
        h = x + scale * sigmoid(gate) * norm(b)
        y = norm(h) with next_weight

    ``weight``, ``scale``, ``next_weight`` [channels] hold one value per irrep
    and channel (fp32; fp64 for fp64 rows), ``gate`` [n, channels] one per row
    too; ``None`` is 1.  Rows are stored in ``dtype`` (fp32, fp64, bfloat16,
    binary16) and may lie further apart than they are wide.  "Dx0e" is the plain
    RMS norm of rows of D."""

    def __init__(self, irreps: str, eps: float = 1e-5, dtype=torch.float32):
        self.irreps, self.eps, self.dtype = irreps, float(eps), dtype
        self.wdtype = torch.float64 if dtype == torch.float64 else torch.float32
        h = ctypes.c_void_p()
        _check(lib().cgtp_norm_create(ctypes.byref(h), irreps.encode(), self.eps, _type(dtype)))
        self._h = h
        a, b, c = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_size_t()
        _check(lib().cgtp_norm_info(h, ctypes.byref(a), ctypes.byref(b)))
        _check(lib().cgtp_norm_workspace(h, ctypes.byref(c)))
        self.dim, self.channels, self.workspace_bytes = a.value, b.value, c.value

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None:
            lib().cgtp_norm_destroy(h)
            self._h = None

    def _w(self, t, name):
        if t is None:
            return None
        _need(t, name, self.wdtype, (self.channels,))
        return t.data_ptr()

    def _in(self, t, name, n):
        return _rows(t, name, self.dtype, n, self.dim)

    def _new(self, like, n, width):
        """New rows, and their description."""
        t = like.new_empty((n, width))
        return t, _Rows(t.data_ptr(), width)

    def _space(self, workspace, device):
        if workspace is None:
            workspace = _scratch(self.workspace_bytes, device)
        return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()

    def forward(self, x, weight=None, out=None):
        """y = norm(x)."""
        n = x.shape[0]
        xr = self._in(x, "x", n)
        if out is None:
            out, o = self._new(x, n, self.dim)
        else:
            o = self._in(out, "out", n)
        _check(lib().cgtp_norm_forward(self._h, n, xr, self._w(weight, "weight"), o, _on()))
        return out

    def backward(self, x, grad_out, weight=None, need=(True, True), workspace=None):
        """(grad_x, grad_weight); an entry is None where ``need`` is False."""
        n = x.shape[0]
        xr, gr = self._in(x, "x", n), self._in(grad_out, "grad_out", n)
        w = self._w(weight, "weight")
        gx, o = self._new(x, n, self.dim) if need[0] else (None, _NONE)
        gw, ws, nws = None, None, 0
        if need[1]:
            gw = torch.empty(self.channels, dtype=self.wdtype, device=x.device)
            workspace, ws, nws = self._space(workspace, x.device)
        _check(lib().cgtp_norm_backward(self._h, n, xr, w, gr, o, _at(gw), ws, nws, _on()))
        return gx, gw

    def residual_forward(self, x, b, weight=None, gate=None, scale=None, next_weight=None,
                         norm_next: bool = True, out=None):
        """(h, y): the residual stream after a block with output ``b`` and, unless
        ``norm_next`` is False (then None), its norm.  ``out``: (h, y) to write;
        h may be x or b."""
        n = b.shape[0]
        br, xr = self._in(b, "b", n), self._in(x, "x", n)
        if out is None:
            h, hr = self._new(b, n, self.dim)
            y, yr = self._new(b, n, self.dim) if norm_next else (None, _NONE)
        else:
            h, y = out
            hr, yr = self._in(h, "h", n), self._in(y, "y", n)
        _check(lib().cgtp_residual_forward(
            self._h, n, xr, br, self._w(weight, "weight"),
            _rows(gate, "gate", self.dtype, n, self.channels), self._w(scale, "scale"),
            self._w(next_weight, "next_weight"), hr, yr, _on()))
        return h, y

    def residual_backward(self, b, h, grad_h, grad_y=None, weight=None, gate=None, scale=None,
                          next_weight=None, need=(True,) * 6, workspace=None):
        """(grad_x, grad_b, grad_gate, grad_weight, grad_scale, grad_next_weight)
        for the cotangents of residual_forward's h and y (either may be None);
        ``h`` as it returned it (None without grad_y).  Entries not in ``need``
        and those of absent arguments (gate; next_weight without grad_y) are
        None."""
        n = b.shape[0]
        br, hr = self._in(b, "b", n), self._in(h, "h", n)
        ghr, gyr = self._in(grad_h, "grad_h", n), self._in(grad_y, "grad_y", n)
        zr = _rows(gate, "gate", self.dtype, n, self.channels)
        none = (None, _NONE)
        gx, gxr = self._new(b, n, self.dim) if need[0] else none
        gb, gbr = self._new(b, n, self.dim) if need[1] else none
        gz, gzr = self._new(b, n, self.channels) if need[2] and gate is not None else none
        sums = [need[3], need[4], need[5] and grad_y is not None]
        gw = gs = gn = ws = None
        nws = 0
        if any(sums):
            gw, gs, gn = (torch.empty(self.channels, dtype=self.wdtype, device=b.device)
                          if wanted else None for wanted in sums)
            workspace, ws, nws = self._space(workspace, b.device)
        _check(lib().cgtp_residual_backward(
            self._h, n, br, hr, self._w(weight, "weight"), zr, self._w(scale, "scale"),
            self._w(next_weight, "next_weight"), ghr, gyr, gxr, gbr, gzr, _at(gw), _at(gs),
            _at(gn), ws, nws, _on()))
        return gx, gb, gz, gw, gs, gn


# ----------------------------------------------------------------- AdamW --

class AdamW:
    """AdamW over a list of parameter tensors, updated in place, one launch per
    64 tensors.  Parameters of one dtype: fp32 (gradients fp32, bfloat16 or
    binary16), fp64, bfloat16 or binary16.

    ``state_bits=8`` holds the moments in one byte each (``m``, ``v``) with one
    exponent byte per 256 elements (``m_exp``, ``v_exp``), rounded
    stochastically from ``seed``; ``state_values()`` gives what they stand for.
    ``copy_dtype`` keeps the parameters' 16-bit copies in ``copies`` (one tensor
    per parameter, for plans with 16-bit weights).  ``m``, ``v``, ``copy`` are
    flat: parameter i's elements start at ``first[i]``.  ``step_count`` is the
    number of steps taken; it and the state tensors are all there is to save."""

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 0.01, state_bits: int = 32, copy_dtype=None, seed: int = 0):
        self.params = list(params)
        if not self.params:
            raise CgtpError("no parameters")
        self.dtype, self.device = self.params[0].dtype, self.params[0].device
        for i, p in enumerate(self.params):
            _need(p, f"parameter {i}", self.dtype)
        _type(self.dtype)
        if state_bits not in (8, 32) or (state_bits == 8 and self.dtype == torch.float64):
            raise CgtpError(f"state_bits {state_bits} is not supported for {self.dtype}")
        if copy_dtype not in (None, torch.bfloat16, torch.float16) or (
                copy_dtype is not None and self.dtype == torch.float64):
            raise CgtpError(f"copy_dtype {copy_dtype} is not supported for {self.dtype}")
        self.lr, self.betas, self.eps = float(lr), (float(betas[0]), float(betas[1])), float(eps)
        self.weight_decay, self.state_bits, self.seed = float(weight_decay), state_bits, int(seed)
        self.step_count = 0
        n = len(self.params)
        # cgtp_adamw_tensor rows: parameter, gradient, length; filled in by step()
        self._table = np.zeros((n, 3), dtype=np.int64)
        self._shapes = [p.shape for p in self.params]
        self._want = {}  # what a step expects of its tensors, by dtype
        self._table[:, 2] = [p.numel() for p in self.params]
        numel = (ctypes.c_int64 * n)(*self._table[:, 2].tolist())
        first, total = (ctypes.c_int64 * n)(), ctypes.c_int64()
        _check(lib().cgtp_adamw_layout(n, numel, first, ctypes.byref(total)))
        self.first, self.total = list(first), total.value
        state = torch.uint8 if state_bits == 8 else (
            torch.float64 if self.dtype == torch.float64 else torch.float32)
        zeros = lambda k, t: torch.zeros(max(k, 1), dtype=t, device=self.device)[:k]  # noqa: E731
        self.m, self.v = zeros(self.total, state), zeros(self.total, state)
        self.m_exp = self.v_exp = None
        if state_bits == 8:
            self.m_exp, self.v_exp = (zeros(self.total // 256, torch.uint8) for _ in range(2))
        self.copy, self.copies, self._copy_type = None, None, F32
        if copy_dtype is not None:
            self.copy, self._copy_type = zeros(self.total, copy_dtype), _type(copy_dtype)
            self.copies = [self.copy[a:a + p.numel()].view(p.shape)
                           for a, p in zip(self.first, self.params)]
            for c, p in zip(self.copies, self.params):
                c.copy_(p)

    def _check_tensors(self, what, tensors, dtype):
        want = self._want.get(dtype)
        if want is None:
            want = self._want[dtype] = [(shape, dtype, True) for shape in self._shapes]
        if list(map(_facts, tensors)) != want or not all(map(torch.Tensor.is_contiguous, tensors)):
            raise CgtpError(f"the {what}s must be contiguous CUDA tensors of {dtype} with the "
                            "shapes that the parameters were given with")

    def step(self, grads, lr=None):
        """One step for the gradients (in the order of the parameters); ``lr``
        replaces the rate for this step."""
        if len(grads) != len(self.params):
            raise CgtpError(f"{len(grads)} gradients for {len(self.params)} parameters")
        gtype, table, params = grads[0].dtype, self._table, self.params
        self._check_tensors("parameter", params, self.dtype)
        self._check_tensors("gradient", grads, gtype)
        table[:, 0] = list(map(torch.Tensor.data_ptr, params))
        table[:, 1] = list(map(torch.Tensor.data_ptr, grads))
        args = _AdamwArgs(self.lr if lr is None else float(lr), *self.betas, self.eps,
                          self.weight_decay, self.step_count + 1, self.seed)
        _check(lib().cgtp_adamw_step(_type(self.dtype), _type(gtype), self.state_bits, len(grads),
                                     table.ctypes.data, self.m.data_ptr(), self.v.data_ptr(),
                                     _at(self.m_exp), _at(self.v_exp), _at(self.copy),
                                     self._copy_type, ctypes.byref(args), _on()))
        self.step_count += 1

    def state_values(self, dtype=torch.bfloat16):
        """(m, v), flat, as the values that 8-bit states stand for: exact in
        bfloat16 and in fp32."""
        if self.state_bits != 8:
            raise CgtpError("state_values() is for 8-bit states")
        m, v = (torch.empty(self.total, dtype=dtype, device=self.device) for _ in range(2))
        _check(lib().cgtp_adamw_values(self.total, self.m.data_ptr(), self.m_exp.data_ptr(),
                                       self.v.data_ptr(), self.v_exp.data_ptr(), _type(dtype),
                                       m.data_ptr(), v.data_ptr(), _on()))
        return m, v
