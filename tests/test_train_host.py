"""Host-side checks of the training operators' entry points (no GPU needed):
argument errors return before any launch, layouts and sizes are as documented."""
import ctypes

import numpy as np
import pytest

import clebsch_gordan_tensor_gb300 as cg
import torch
from tests import train_reference as R

A = 0x100000  # stands for device memory: every call here returns before using it


def rows(p, stride):
    return cg._Rows(p, stride)


def test_embed_argument_errors():
    L = cg.lib()
    call = lambda t=0, bits=32, n=4, v=5, d=8, i=A, tab=A, out=A, st=8: L.cgtp_embed_forward(  # noqa: E731
        t, bits, n, v, d, i, tab, 1.0, out, st, None)
    assert call(n=0) == 0
    assert [call(t=4), call(bits=16), call(n=-1), call(n=1 << 31), call(v=-1), call(d=0),
            call(st=7), call(i=None), call(tab=None), call(out=None), call(i=A + 2),
            call(tab=A + 2), call(out=A + 1), call(t=1, tab=A + 4), call(t=2, out=A + 1)] == [1] * 15
    n = ctypes.c_size_t()
    assert L.cgtp_embed_backward_workspace(0, 0, 5, 8, ctypes.byref(n)) == 0 and n.value == 0
    assert L.cgtp_embed_backward_workspace(0, 100, 5, 8, ctypes.byref(n)) == 0 and n.value == 0
    assert L.cgtp_embed_backward_workspace(0, 3000, 5, 8, ctypes.byref(n)) == 0 and n.value > 48000
    back = lambda n_=3000, ws=A, nb=n.value, g=A, out=A, st=8: L.cgtp_embed_backward(  # noqa: E731
        0, 32, n_, 5, 8, A, g, st, 1.0, out, ws, nb, None)
    assert [back(ws=None), back(ws=A + 16), back(nb=n.value - 1), back(g=None), back(out=None),
            back(st=-1)] == [1] * 6
    assert L.cgtp_embed_backward(0, 32, 4, 0, 8, A, A, 8, 1.0, None, None, 0, None) == 0
    assert L.cgtp_embed_device_status(None) == 1


def test_norm_handles_and_argument_errors():
    L = cg.lib()
    h = ctypes.c_void_p()
    make = lambda s, eps=1e-5, t=0: L.cgtp_norm_create(ctypes.byref(h), s, eps, t)  # noqa: E731
    assert make(b"8x0e", t=4) == 1 and make(b"8x0e", eps=0.0) == 1 and make(b"8x0e", eps=-1.0) == 1
    assert make(b"8x0e", eps=float("nan")) == 1 and make(b"8x0q") == 2 and make(b"8x7e") == 2
    assert make(None) == 2 and make(b"+".join([b"1x0e"] * 33)) == 4
    assert make(b"+".join([b"1x0e"] * 32)) == 0
    L.cgtp_norm_destroy(h)
    assert make(b"2000000000x0e") == 4
    assert make(b"4x0e+3x1o+2x2e") == 0
    d, c, w = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_size_t()
    assert L.cgtp_norm_info(h, ctypes.byref(d), ctypes.byref(c)) == 0
    assert (d.value, c.value) == (4 + 9 + 10, 9)
    assert L.cgtp_norm_workspace(h, ctypes.byref(w)) == 0 and w.value > 0
    ok, none = rows(A, 23), rows(None, 0)
    f = lambda n=5, x=ok, wt=A, y=rows(2 * A, 23): L.cgtp_norm_forward(h, n, x, wt, y, None)  # noqa: E731
    assert f(n=0) == 0
    assert [f(n=-1), f(x=none), f(y=none), f(wt=A + 2), f(x=rows(A + 2, 23)),
            f(y=rows(2 * A, 22)), f(x=rows(A, -1))] == [1] * 7
    out = lambda k: rows((2 + k) * A, 23)  # noqa: E731
    g = lambda b=ok, hh=ok, gh=ok, gy=ok, gx=out(0), gb=out(1), gw=5 * A, ws=A, nb=w.value: \
        L.cgtp_residual_backward(h, 5, b, hh, None, none, None, None, gh, gy, gx, gb, none, gw,
                                 None, None, ws, nb, None)  # noqa: E731
    assert [g(b=none), g(hh=none), g(gh=none, gy=none), g(gx=rows(A, 23)), g(gb=rows(A, 23)),
            g(ws=None), g(ws=A + 128), g(nb=w.value - 1)] == [1] * 8
    assert L.cgtp_residual_forward(h, 5, none, ok, None, none, None, None, out(0), out(0), None) == 1
    assert L.cgtp_norm_destroy(h) == 0 and L.cgtp_norm_destroy(None) == 0
    assert L.cgtp_norm_forward(None, 1, ok, None, ok, None) == 1


def test_adamw_layout_and_argument_errors():
    L = cg.lib()
    numel = (ctypes.c_int64 * 4)(1, 0, 256, 257)
    first, total = (ctypes.c_int64 * 4)(), ctypes.c_int64()
    assert L.cgtp_adamw_layout(4, numel, first, ctypes.byref(total)) == 0
    assert list(first) == [0, 256, 256, 512] and total.value == 1024
    numel[0] = -1
    assert L.cgtp_adamw_layout(4, numel, first, ctypes.byref(total)) == 1
    assert L.cgtp_adamw_layout(0, None, None, ctypes.byref(total)) == 0 and total.value == 0

    def step(p=0, g=0, bits=32, n=1, param=A, grad=A, count=10, m=A, exp=A, copy=None, ct=2,
             **args):
        t = cg._AdamwTensor(param, grad, count)
        a = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1, seed=0)
        a.update(args)
        return L.cgtp_adamw_step(p, g, bits, n, ctypes.byref(t), m, A, exp, A, copy, ct,
                                 ctypes.byref(cg._AdamwArgs(**a)), None)

    assert step(n=0) == 0 and step(count=0) == 0
    assert [step(p=4), step(g=9), step(bits=16), step(n=-1), step(param=None), step(grad=None),
            step(param=A + 2), step(grad=A + 1), step(count=-1), step(m=None), step(m=A + 16),
            step(bits=8, exp=None), step(copy=A, ct=0), step(copy=A + 2), step(eps=0.0),
            step(beta1=1.0), step(beta2=-0.1), step(step=0), step(lr=float("inf")),
            step(weight_decay=float("nan"))] == [1] * 20
    assert [step(p=2, g=0), step(p=0, g=1), step(p=1, g=0), step(p=1, g=1, bits=8),
            step(p=1, g=1, copy=A)] == [4] * 5
    v = lambda total=256, t=0, m=A: L.cgtp_adamw_values(total, m, A, A, A, t, A, A, None)  # noqa: E731
    assert v(total=0) == 0 and [v(total=100), v(t=1), v(m=None), v(m=A + 4)] == [1] * 4


@pytest.mark.parametrize("dtype", [2, 3])
def test_other_entry_points_refuse_16bit_types(dtype):
    L = cg.lib()
    h = ctypes.c_void_p()
    assert L.cgtp_plan_create(ctypes.byref(h), b"4x0e", b"0e", b"4x0e", None, 0, dtype, 0, 0) == 1
    assert L.cgtp_linear_create(ctypes.byref(h), b"4x0e", b"4x0e", None, 0, dtype) == 1
    assert L.cgtp_uvw_create(ctypes.byref(h), b"4x0e", b"0e", b"4x0e", dtype) == 1
    assert L.cgtp_sh_forward(2, dtype, 4, A, A, None) == 1
    assert L.cgtp_edge_forces(dtype, 1, 1, A, A, A, A, A, None) == 1


def test_irreps_norm_sizes():
    norm = cg.IrrepsNorm("64x0e+64x1o+64x2e", dtype=torch.bfloat16)
    assert (norm.dim, norm.channels, norm.wdtype) == (576, 192, torch.float32)
    with pytest.raises(cg.CgtpError):
        cg.IrrepsNorm("64x0e", dtype=torch.int32)


def test_reference_rounding_is_unbiased_and_on_the_grid():
    """The tests' own 8-bit definition: over all 16-bit noises the mean of the
    rounded values is the value, and a value on the grid stays."""
    x = np.zeros(256)
    x[0], x[1] = 1.7, 0.3
    u = (np.arange(4096) + 0.5) / 4096
    got = np.array([R.code_value(*R.encode(x, 4, np.full(256, k)), 4)[1] for k in u])
    assert abs(got.mean() - 0.3) < 0.3 / 16 / 4096 * 2
    assert set(got) == {0.28125, 0.3125}
    y = R.code_value(*R.encode(x, 5, np.full(256, 0.3)), 5)
    again = R.code_value(*R.encode(y, 5, np.full(256, 0.999)), 5)
    assert np.array_equal(y, again)
