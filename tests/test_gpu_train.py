"""GPU tests of the training operators (embedding, per-irrep norm and gated
residual, AdamW) against plain 64-bit implementations."""
import numpy as np
import pytest

from tests import train_reference as R
from tests.gpu_util import need_gpu, torch

pytestmark = pytest.mark.gpu

F32, F64, BF16, F16 = torch.float32, torch.float64, torch.bfloat16, torch.float16
TYPES = [F32, F64, BF16, F16]
name = lambda t: str(t).replace("torch.", "")  # noqa: E731


def _cg():
    need_gpu()
    import clebsch_gordan_tensor_gb300 as cg
    return cg


def _rows(gen, n, d, dtype, pad=0, shift=0):
    """Random rows; pad: columns of wider rows, shift: the first column taken."""
    t = torch.randn(n, d + pad + shift, generator=gen, dtype=F64).to(dtype).cuda()
    return t[:, shift:shift + d]


# ------------------------------------------------------------- embedding --

EMBED = [  # n, v, d, pad, shift
    (29, 119, 32, 480, 0), (1, 1, 1, 0, 0), (1, 5, 64, 0, 0), (0, 7, 8, 0, 0), (300, 10, 33, 0, 0),
    (1000, 3, 64, 0, 0), (5000, 119, 16, 3, 0), (513, 700, 130, 0, 1), (2049, 70000, 24, 0, 0),
    (4096, 2, 256, 0, 0), (70, 4, 1000, 8, 0), (64, 1000, 2056, 0, 0), (6000, 300, 40, 0, 0),
    (1024, 119, 64, 0, 0), (1025, 119, 64, 0, 0), (1000, 40000, 100, 4, 0), (3, 60000, 260, 0, 0),
    (7, 256, 8, 0, 0), (2000, 255, 8, 0, 0), (2000, 65535, 8, 0, 0), (2000, 65536, 4, 0, 0),
]


def _index(n, v, kind, seed):
    rng = np.random.default_rng(seed)
    i = rng.integers(0, max(1, v), n)
    if n > 10:
        i[n // 2:] = np.where(rng.random(n - n // 2) < 0.7, v // 2, i[n // 2:])  # one row is hot
        i[rng.random(n) < 0.05] = -1
        i[3] = -(2 ** 31) + 5
    return torch.from_numpy(i).to(kind).cuda()


@pytest.mark.parametrize("dtype", TYPES, ids=name)
@pytest.mark.parametrize("case", EMBED, ids=lambda c: "-".join(map(str, c)))
def test_embed_forward(case, dtype):
    cg = _cg()
    n, v, d, pad, shift = case
    gen = torch.Generator().manual_seed(n + d)
    for kind in (torch.int32, torch.int64):
        idx = _index(n, v, kind, d)
        table = _rows(gen, v, d, dtype)
        wide = torch.full((n, d + pad + shift), 3.0, dtype=dtype, device="cuda")
        out = wide[:, shift:shift + d]
        assert cg.embed_forward(idx, table, 1.75, out=out) is out
        ref = torch.zeros(n, d, dtype=F64)
        i = idx.cpu().long()
        ref[i >= 0] = table.cpu().double()[i[i >= 0]] * 1.75
        R.assert_rounded(out, ref, dtype, "out", sums=0)
        rest = torch.cat([wide[:, :shift], wide[:, shift + d:]], 1)
        assert (rest == 3.0).all()  # the rest of wider rows stays
    assert cg.embed_device_status() == 0


@pytest.mark.parametrize("dtype", TYPES, ids=name)
@pytest.mark.parametrize("case", EMBED, ids=lambda c: "-".join(map(str, c)))
def test_embed_backward(case, dtype):
    cg = _cg()
    n, v, d, pad, shift = case
    gen = torch.Generator().manual_seed(n + d)
    g = _rows(gen, n, d, dtype, pad, shift)
    for kind in (torch.int32, torch.int64):
        idx = _index(n, v, kind, d)
        out = torch.full((v, d), 9.0, dtype=dtype, device="cuda")
        assert cg.embed_backward(idx, g, v, 0.3, out=out) is out
        R.assert_rounded(out, R.embed_grad(idx.cpu(), g.cpu(), v, 0.3), dtype, "grad_table")
        again = cg.embed_backward(idx, g, v, 0.3)
        assert torch.equal(out, again)  # the order of the sums is fixed
    assert cg.embed_device_status() == 0


def test_embed_backward_is_the_adjoint_of_forward():
    cg = _cg()
    gen = torch.Generator().manual_seed(5)
    idx = _index(3000, 50, torch.int32, 1)
    table, g = _rows(gen, 50, 48, F64), _rows(gen, 3000, 48, F64)
    a = (cg.embed_forward(idx, table, 0.7) * g).sum()
    b = (table * cg.embed_backward(idx, g, 50, 0.7)).sum()
    assert abs((a - b).item()) <= 1e-11 * g.abs().sum().item()


def test_embed_out_of_range_indices_read_nothing_and_are_reported():
    cg = _cg()
    gen = torch.Generator().manual_seed(6)
    table, g = _rows(gen, 10, 64, F32), _rows(gen, 40, 64, F32)
    idx = torch.arange(40, device="cuda", dtype=torch.int64)
    idx[39] = 2 ** 40
    assert cg.embed_device_status() == 0
    out = cg.embed_forward(idx, table)
    assert torch.equal(out[:10], table) and (out[10:] == 0).all()
    assert cg.embed_device_status() == 1 and cg.embed_device_status() == 0
    gt = cg.embed_backward(idx, g, 10)
    assert torch.equal(gt, g[:10])
    assert cg.embed_device_status() == 1 and cg.embed_device_status() == 0


def test_embed_gradient_of_broadcast_rows():
    cg = _cg()
    idx = _index(500, 7, torch.int32, 2)
    g = torch.randn(1, 24, device="cuda").expand(500, 24)
    R.assert_rounded(cg.embed_backward(idx, g, 7), R.embed_grad(idx.cpu(), g.cpu(), 7, 1.0), F32, "g")


def test_embed_large_n_matches_sorted_sums():
    """More positions than one chunk's run: a row that takes most of them."""
    cg = _cg()
    n, v, d = 200_000, 6, 20
    gen = torch.Generator().manual_seed(3)
    idx = (torch.rand(n, generator=gen) ** 6 * v).int()
    g = torch.randn(n, d, generator=gen)
    ref = torch.stack([g.double()[idx == k].sum(0) for k in range(v)])
    R.assert_rounded(cg.embed_backward(idx.cuda(), g.cuda(), v), ref, F32, "g")


# ---------------------------------------------- norms and gated residuals --

NORM = [  # n, irreps, pad, shift
    (29, "32x0e+32x1o+32x2e+32x3o", 0, 0), (1, "1x0e", 0, 0), (7, "5x0e+3x1o+2x2e", 0, 0),
    (0, "8x0e+8x1o", 0, 0), (33, "64x0e+64x1o+64x2e", 64, 0), (50, "64x0e+64x1o+64x2e", 3, 1),
    (3, "4096x0e", 0, 0), (5, "1000x0e", 0, 0), (2, "8192x0e", 0, 0), (2, "9000x0e", 0, 0),
    (2, "8193x0e", 0, 0), (3, "600x1o", 0, 0), (2, "2056x1o+2056x0e", 0, 0), (3, "260x3o", 0, 0),
    (2, "1100x2e", 0, 0), (9, "16x4e+8x5o+4x6e", 0, 0), (4, "300x6e", 0, 0),
    (257, "128x0e+128x1o+128x2e", 0, 0), (130, "20x0e+12x1o+4x0o", 0, 0), (11, "700x0e+33x1o", 0, 0),
    (700, "2x0e+2x1o", 0, 0),
]


def _problem(case, dtype, seed=0):
    n, irreps, pad, shift = case
    gen = torch.Generator().manual_seed(seed + n)
    blocks = R.parse(irreps)
    d, ch = sum(m * (2 * l + 1) for m, l in blocks), sum(m for m, _ in blocks)
    w = F64 if dtype == F64 else F32
    q = {k: _rows(gen, n, d, dtype, pad, shift) for k in ("x", "b", "gh", "gy")}
    q["gate"] = (1.5 * _rows(gen, n, ch, dtype, pad, shift).double()).to(dtype)
    for k in ("weight", "scale", "next_weight"):
        q[k] = (1 + 0.3 * torch.randn(ch, generator=gen, dtype=F64)).to(w).cuda()
    if n > 4:
        q["b"][2] = 0  # a row with nothing in it
        q["x"][3] = 0
    return q, irreps


@pytest.mark.parametrize("dtype", TYPES, ids=name)
@pytest.mark.parametrize("case", NORM, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}-{c[3]}")
def test_norm(case, dtype):
    cg = _cg()
    q, irreps = _problem(case, dtype)
    norm = cg.IrrepsNorm(irreps, eps=1e-5, dtype=dtype)
    y = norm.forward(q["b"], q["weight"])
    x = q["b"].cpu().double().requires_grad_()
    w = q["weight"].cpu().double().requires_grad_()
    ref = R.norm(x, w, irreps, 1e-5)
    R.assert_rounded(y, ref, dtype, "y")
    gx, gw = norm.backward(q["b"], q["gh"], q["weight"])
    rx, rw = torch.autograd.grad(ref, (x, w), q["gh"].cpu().double())
    R.assert_rounded(gx, rx, dtype, "grad_x",
                     terms=R.norm_grad_terms(x, q["gh"].cpu().double(), w, irreps, 1e-5))
    R.assert_rounded(gw, rw, norm.wdtype, "grad_weight")
    plain = norm.forward(q["b"])
    R.assert_rounded(plain, R.norm(x, None, irreps, 1e-5), dtype, "y without a weight")
    gx2, none = norm.backward(q["b"], q["gh"], q["weight"], need=(True, False))
    assert none is None and torch.equal(gx2, gx)


@pytest.mark.parametrize("dtype", TYPES, ids=name)
@pytest.mark.parametrize("case", NORM, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}-{c[3]}")
def test_residual(case, dtype):
    cg = _cg()
    q, irreps = _problem(case, dtype)
    norm = cg.IrrepsNorm(irreps, eps=1e-3, dtype=dtype)
    h, y = norm.residual_forward(q["x"], q["b"], q["weight"], q["gate"], q["scale"],
                                 q["next_weight"])
    r = {k: v.cpu().double() for k, v in q.items()}
    leaves = [r[k].requires_grad_() for k in ("x", "b", "gate", "weight", "scale")]
    ref = R.residual(r["x"], r["b"], r["weight"], r["gate"], r["scale"], irreps, 1e-3)
    R.assert_rounded(h, ref, dtype, "h")
    hs = h.cpu().double().requires_grad_()  # y and its gradient go by h as it is stored
    w2 = r["next_weight"].requires_grad_()
    yr = R.norm(hs, w2, irreps, 1e-3)
    R.assert_rounded(y, yr, dtype, "y")
    got = norm.residual_backward(q["b"], h, q["gh"], q["gy"], q["weight"], q["gate"], q["scale"],
                                 q["next_weight"])
    gh, g2 = torch.autograd.grad(yr, (hs, w2), r["gy"])
    gh = gh + r["gh"]
    gx, gb, gz, gw, gs = torch.autograd.grad(ref, leaves, gh)
    terms = {"grad_x": R.norm_grad_terms(hs, r["gy"], w2, irreps, 1e-3),
             "grad_b": R.norm_grad_terms(r["b"], gh.abs() * R.per_component(
                 r["scale"].detach().abs(), irreps), r["weight"], irreps, 1e-3)}
    for k, a, e, t in (("grad_x", got[0], gx, dtype), ("grad_b", got[1], gb, dtype),
                       ("grad_gate", got[2], gz, dtype), ("grad_weight", got[3], gw, norm.wdtype),
                       ("grad_scale", got[4], gs, norm.wdtype),
                       ("grad_next_weight", got[5], g2, norm.wdtype)):
        R.assert_rounded(a, e, t, k, terms=terms.get(k, 0.0))
    again = norm.residual_backward(q["b"], h, q["gh"], q["gy"], q["weight"], q["gate"], q["scale"],
                                   q["next_weight"])
    assert all(torch.equal(a, e) for a, e in zip(got, again))


@pytest.mark.parametrize("left_out", ["x", "gate", "scale", "weight", "next_weight", "gh", "gy"])
def test_residual_with_an_argument_left_out(left_out):
    cg = _cg()
    q, irreps = _problem((37, "16x0e+16x1o+8x2e", 0, 0), F64)
    q[left_out] = None
    norm = cg.IrrepsNorm(irreps, eps=1e-5, dtype=F64)
    h, y = norm.residual_forward(q["x"], q["b"], q["weight"], q["gate"], q["scale"],
                                 q["next_weight"], norm_next=q["gy"] is not None)
    assert (y is None) == (q["gy"] is None)
    r = {k: None if v is None else v.cpu().requires_grad_() for k, v in q.items()}
    ref = R.residual(r["x"], r["b"], r["weight"], r["gate"], r["scale"], irreps, 1e-5)
    R.assert_rounded(h, ref, F64, "h")
    loss = 0 if r["gh"] is None else (ref * r["gh"].detach()).sum()
    if r["gy"] is not None:
        yr = R.norm(ref, r["next_weight"], irreps, 1e-5)
        R.assert_rounded(y, yr, F64, "y")
        loss = loss + (yr * r["gy"].detach()).sum()
    got = norm.residual_backward(q["b"], h if q["gy"] is not None else None, q["gh"], q["gy"],
                                 q["weight"], q["gate"], q["scale"], q["next_weight"])
    keys = ["x", "b", "gate", "weight", "scale", "next_weight"]
    want = [r[k] for k in keys if r[k] is not None]
    grads = dict(zip([k for k in keys if r[k] is not None],
                     torch.autograd.grad(loss, want, allow_unused=True)))
    for k, g in zip(keys, got):
        if grads.get(k) is not None:
            R.assert_rounded(g, grads[k], F64, "gradient of " + k)


def test_residual_gradient_against_differences():
    """The fp64 kernels' own forward, along random directions: a step of 1e-5
    leaves a relative truncation of about 1e-10 and a rounding of about 1e-11."""
    cg = _cg()
    q, irreps = _problem((23, "6x0e+5x1o+4x2e", 0, 0), F64)
    norm = cg.IrrepsNorm(irreps, eps=1e-2, dtype=F64)

    def loss(p):
        h, y = norm.residual_forward(p["x"], p["b"], p["weight"], p["gate"], p["scale"],
                                     p["next_weight"])
        return (h * q["gh"]).sum() + (y * q["gy"]).sum()

    h, _ = norm.residual_forward(q["x"], q["b"], q["weight"], q["gate"], q["scale"],
                                 q["next_weight"])
    grads = norm.residual_backward(q["b"], h, q["gh"], q["gy"], q["weight"], q["gate"], q["scale"],
                                   q["next_weight"])
    for k, g in zip(("x", "b", "gate", "weight", "scale", "next_weight"), grads):
        d = torch.randn_like(q[k])
        up, down = ({**q, k: q[k] + s * 1e-5 * d} for s in (1, -1))
        slope = (loss(up) - loss(down)).item() / 2e-5
        assert abs(slope - (g * d).sum().item()) <= 1e-7 * (g * d).abs().sum().item(), k


def test_norm_commutes_with_rotations():
    cg = _cg()
    from scipy.spatial.transform import Rotation
    order = [1, 2, 0]  # an l = 1 block's components are (y, z, x)
    D1 = torch.from_numpy(Rotation.random(random_state=3).as_matrix()[np.ix_(order, order)])
    mul, n = 8, 12
    turn = lambda t: torch.einsum("ij,njk->nik", D1, t.view(n, 3, mul)).reshape(n, -1)  # noqa: E731
    gen = torch.Generator().manual_seed(1)
    b = torch.randn(n, 3 * mul, generator=gen, dtype=F64)
    w = torch.rand(mul, generator=gen, dtype=F64).cuda()
    gate = torch.randn(n, mul, generator=gen, dtype=F64).cuda()
    norm = cg.IrrepsNorm(f"{mul}x1o", dtype=F64)
    y0, _ = norm.residual_forward(None, b.cuda(), w, gate, norm_next=False)
    y1, _ = norm.residual_forward(None, turn(b).cuda(), w, gate, norm_next=False)
    assert (y1.cpu() - turn(y0.cpu())).abs().max() < 1e-12


def test_residual_in_place_and_in_broadcast_rows():
    cg = _cg()
    q, irreps = _problem((40, "16x0e+16x1o", 0, 0), F32)
    norm = cg.IrrepsNorm(irreps)
    args = (q["weight"], q["gate"], q["scale"], q["next_weight"])
    h, y = norm.residual_forward(q["x"], q["b"], *args)
    x = q["x"].clone()
    y2 = torch.empty_like(y)
    norm.residual_forward(x, q["b"], *args, out=(x, y2))
    assert torch.equal(x, h) and torch.equal(y2, y)
    one = q["gate"][:1].expand(40, -1)  # one gate for all rows
    h1, y1 = norm.residual_forward(q["x"], q["b"], q["weight"], one, q["scale"], q["next_weight"])
    h2, y2 = norm.residual_forward(q["x"], q["b"], q["weight"], one.contiguous(), q["scale"],
                                   q["next_weight"])
    assert torch.equal(h1, h2) and torch.equal(y1, y2)


def test_norm_keeps_infinities_and_nan_to_their_rows():
    cg = _cg()
    q, irreps = _problem((40, "16x0e+16x1o", 0, 0), F32)
    norm = cg.IrrepsNorm(irreps)
    clean = norm.residual_forward(q["x"], q["b"], q["weight"], q["gate"], q["scale"])[1]
    q["b"][7, 3] = float("nan")
    q["b"][8, 20] = float("inf")
    got = norm.residual_forward(q["x"], q["b"], q["weight"], q["gate"], q["scale"])[1]
    keep = [i for i in range(40) if i not in (7, 8)]
    assert torch.equal(got[keep], clean[keep])
    assert torch.isnan(got[7, :16]).all() and torch.equal(got[7, 16:], clean[7, 16:])
    assert torch.equal(got[8, :16], clean[8, :16]) and torch.isnan(got[8, 20])


# ----------------------------------------------------------------- AdamW --

HYPER = dict(lr=3e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)


def _np(t):
    return t.detach().cpu().double().numpy().reshape(-1)


def _params(sizes, dtype, gtype, seed=0, shift=0):
    gen = torch.Generator().manual_seed(seed)
    def make(k, t, size):
        buf = (size * torch.randn(k + shift, generator=gen)).to(t).cuda()
        return buf[shift:]
    return [make(k, dtype, 0.5) for k in sizes], [
        [make(k, gtype, 10.0 ** -(i % 4)) for i, k in enumerate(sizes)] for _ in range(3)]


SIZES = [(1,), (255, 256, 257), (7, 0, 1024, 3000, 1), (70_000,), tuple(range(1, 140))]


@pytest.mark.parametrize("types", [(F32, F32), (F64, F64), (BF16, BF16), (F16, F16), (F32, BF16),
                                   (F32, F16)], ids=lambda t: f"{name(t[0])}-{name(t[1])}")
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("shift", [0, 1])
def test_adamw_32bit_states(types, sizes, shift):
    cg = _cg()
    dtype, gtype = types
    params, grads = _params(sizes, dtype, gtype, shift=shift)
    opt = cg.AdamW(params, state_bits=32, **HYPER)
    work = np.float64 if dtype == F64 else np.float32
    state = [[np.zeros(k, work) for k in sizes] for _ in range(2)]
    for t, gs in enumerate(grads, 1):
        before = [_np(p).astype(work) for p in params]
        opt.step(gs)
        for i, k in enumerate(sizes):
            if k == 0:
                continue
            ref, state[0][i], state[1][i] = R.adamw(before[i], _np(gs[i]).astype(work), state[0][i],
                                                    state[1][i], HYPER["lr"], *HYPER["betas"],
                                                    HYPER["eps"], HYPER["weight_decay"], t)
            # one rounding of the parameter, and 1e-5 of a step's size (lr)
            tol = 1.001 * R.UNIT[dtype] * np.abs(ref) + (1e-12 if dtype == F64 else 4e-8) * (
                np.abs(ref) + HYPER["lr"])
            if dtype == F16:
                tol = tol + 2.0 ** -25
            assert (np.abs(_np(params[i]) - ref) <= tol + 1e-5 * HYPER["lr"] * (dtype != F64)).all()
            at = opt.first[i]
            # the recursions' products are rounded apart: equal to the bit
            assert np.array_equal(opt.m[at:at + k].cpu().numpy(), state[0][i])
            assert np.array_equal(opt.v[at:at + k].cpu().numpy(), state[1][i])
    assert opt.step_count == 3


@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16), (F16, F16), (F32, BF16)],
                         ids=lambda t: f"{name(t[0])}-{name(t[1])}")
@pytest.mark.parametrize("sizes", SIZES[:4], ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("shift", [0, 1])
def test_adamw_8bit_states(types, sizes, shift):
    """The codes equal the definition's to the bit, from states that are on the
    grid (each step starts from the codes of the one before)."""
    cg = _cg()
    dtype, gtype = types
    seed = (5 << 32) + 77
    params, grads = _params(sizes, dtype, gtype, shift=shift)
    opt = cg.AdamW(params, state_bits=8, seed=seed, **HYPER)
    for t, gs in enumerate(grads, 1):
        before = [_np(p).astype(np.float32) for p in params]
        was_m, was_v = (R.code_value(c.cpu(), e.cpu(), b) for c, e, b in
                        ((opt.m, opt.m_exp, 4), (opt.v, opt.v_exp, 5)))
        opt.step(gs)
        got_m, got_v = (c.cpu().numpy() for c in (opt.m, opt.v))
        em, ev = opt.m_exp.cpu().numpy(), opt.v_exp.cpu().numpy()
        val_m, val_v = opt.state_values(F32)
        assert np.array_equal(_np(val_m), R.code_value(got_m, em, 4))
        assert np.array_equal(_np(val_v), R.code_value(got_v, ev, 5))
        for a, b in zip(opt.state_values(), (val_m, val_v)):
            assert torch.equal(a.float(), b)  # bfloat16 holds the values exactly
        for i, k in enumerate(sizes):
            if k == 0:
                continue
            at, end = opt.first[i], opt.first[i] + -(-k // 256) * 256
            ref, m, v = R.adamw(before[i], _np(gs[i]).astype(np.float32),
                                was_m[at:at + k].astype(np.float32),
                                was_v[at:at + k].astype(np.float32), HYPER["lr"], *HYPER["betas"],
                                HYPER["eps"], HYPER["weight_decay"], t)
            tol = 1.001 * R.UNIT[dtype] * np.abs(ref) + 4e-8 * (np.abs(ref) + HYPER["lr"]) \
                + 1e-5 * HYPER["lr"] + (2.0 ** -25 if dtype == F16 else 0)
            # m / sqrt(v) can exceed 1 here (v rounds): the step's size is its own scale
            step = np.abs(ref - before[i] * (1 - HYPER["lr"] * HYPER["weight_decay"]))
            assert (np.abs(_np(params[i]) - ref) <= tol + 1e-5 * step).all()
            um, uv = R.noise(seed, t, i, k) if k < 5000 else (None, None)
            if um is None:
                continue
            cm, xm = R.encode(R.pad256(m), 4, R.pad256(um))
            cv, xv = R.encode(R.pad256(v), 5, R.pad256(uv))
            assert np.array_equal(em[at // 256:end // 256], xm)
            assert np.array_equal(ev[at // 256:end // 256], xv)
            assert np.array_equal(got_m[at:end], cm) and np.array_equal(got_v[at:end], cv)


def test_adamw_8bit_rounding_keeps_the_mean():
    """beta2 = 0.999 moves v by less than a hundredth of a grid step; over many
    elements the mean follows the exact recursion.  An element's rounding adds at
    most a variance of f (1 - f) step^2 with step = v/8, f = 0.001 v / step: over
    300 steps a relative deviation below sqrt(300 * 0.008) / 8 = 0.19, over
    2^17 elements 5.4e-4; five of them are allowed."""
    cg = _cg()
    n = 1 << 17
    p = [torch.zeros(n, device="cuda")]
    opt = cg.AdamW(p, lr=0.0, betas=(0.9, 0.999), weight_decay=0.0, state_bits=8, seed=9)
    g = torch.full((n,), 0.37, device="cuda")
    g[::256] = 3.0  # the block's exponent comes from another element
    exact = 0.0
    for _ in range(300):
        opt.step([g])
        exact = 0.999 * exact + 0.001 * 0.37 ** 2
    v = opt.state_values(F32)[1].view(-1, 256)[:, 1:].double()
    assert abs(v.mean().item() / exact - 1) < 5 * 5.4e-4


def test_adamw_8bit_range_and_non_finite_blocks():
    cg = _cg()
    p = [torch.zeros(1024, device="cuda")]
    opt = cg.AdamW(p, betas=(0.9, 0.99), state_bits=8)
    g = torch.zeros(1024, device="cuda")
    g[0], g[1], g[2] = 1.0, 1e-12, 1e-30  # far below the block's largest
    g[256:512] = 1e-38
    g[513] = float("inf")
    g[768:] = torch.randn(256, device="cuda") * 1e-3
    opt.step([g])
    m, v = opt.state_values(F32)
    assert (v[:256] > 0).sum() == 2  # 1e-60 is zero in fp32, 1e-24 is not
    assert torch.isfinite(p[0][:513]).all() and torch.isfinite(p[0][768:]).all()
    assert p[0][1].abs() <= 1e-3 * 1.1  # bounded by the step's size
    assert torch.isnan(v[512:768]).all() and torch.isnan(m[512:768]).all()
    assert torch.isfinite(m[:512]).all() and torch.isfinite(v[:512]).all()
    assert torch.isfinite(m[768:]).all() and (v[768:] > 0).all()


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("copy", [BF16, F16], ids=name)
def test_adamw_16bit_copies(bits, copy):
    cg = _cg()
    params, grads = _params((300, 64, 1000), F32, F32)
    opt = cg.AdamW(params, state_bits=bits, copy_dtype=copy, **HYPER)
    for p, c in zip(params, opt.copies):
        assert torch.equal(p.to(copy), c)
    for gs in grads:
        opt.step(gs)
        for p, c in zip(params, opt.copies):
            assert torch.equal(p.to(copy), c)


def test_adamw_states_resume_to_the_bit():
    cg = _cg()
    for bits in (8, 32):
        a, grads = _params((300, 77), F32, F32)
        one = cg.AdamW(a, state_bits=bits, seed=3, **HYPER)
        one.step(grads[0])
        b = [p.clone() for p in a]
        two = cg.AdamW(b, state_bits=bits, seed=3, **HYPER)
        for x, y in ((two.m, one.m), (two.v, one.v), (two.m_exp, one.m_exp), (two.v_exp, one.v_exp)):
            if x is not None:
                x.copy_(y)
        two.step_count = one.step_count
        for opt, ps in ((one, a), (two, b)):
            opt.step(grads[1])
        assert all(torch.equal(x, y) for x, y in zip(a, b)) and torch.equal(one.m, two.m)


# ---------------------------------------------- past 2^31 and 2^32 elements --


def _room(gb):
    if torch.cuda.mem_get_info()[0] < gb * 2 ** 30:
        pytest.skip(f"needs {gb} GB of device memory")


def test_embed_past_32_bit_offsets():
    cg = _cg()
    _room(24)
    n, v, d = 2_200_000, 9, 1000  # 2.2e9 elements of bfloat16
    idx = torch.arange(n, device="cuda", dtype=torch.int32) % v
    table = torch.randn(v, d, device="cuda").bfloat16()
    out = cg.embed_forward(idx, table)
    for at in (0, n // 2, n - 3):
        assert torch.equal(out[at:at + 3], table[idx[at:at + 3].long()])
    out.zero_()
    out[-5:] = table[:5]  # only the last rows count
    got = cg.embed_backward(idx, out, v)
    ref = torch.zeros_like(table)
    ref[idx[-5:].long()] = table[:5]
    assert torch.equal(got, ref)


def test_norm_past_32_bit_offsets():
    cg = _cg()
    _room(40)
    irreps, n = "8x0e+8x1o", 70_000_000  # 2.24e9 elements of bfloat16
    norm = cg.IrrepsNorm(irreps, dtype=BF16)
    x = torch.zeros(n, 32, dtype=BF16, device="cuda")
    x[-4:] = torch.randn(4, 32, device="cuda")
    y = norm.forward(x)
    R.assert_rounded(y[-4:], R.norm(x[-4:].cpu().double(), None, irreps, 1e-5), BF16, "y")
    assert (y[:1000] == 0).all()
    g = torch.zeros_like(x)
    g[-4:] = torch.randn(4, 32, device="cuda")
    gx, gw = norm.backward(x, g)
    leaf = x[-4:].cpu().double().requires_grad_()
    w = torch.ones(16, dtype=F64, requires_grad=True)
    rx, rw = torch.autograd.grad(R.norm(leaf, w, irreps, 1e-5), (leaf, w), g[-4:].cpu().double())
    R.assert_rounded(gx[-4:], rx, BF16, "grad_x")
    R.assert_rounded(gw, rw, F32, "grad_weight")


def test_adamw_past_32_bit_offsets():
    """More than 2^32 elements in one tensor: the last block's codes, whose hash
    takes the element's upper half too."""
    cg = _cg()
    _room(48)
    n = 2 ** 32 + 300
    p = torch.zeros(n, dtype=BF16, device="cuda")
    g = torch.zeros(n, dtype=BF16, device="cuda")
    g[-300:] = torch.randn(300, device="cuda")
    opt = cg.AdamW([p], state_bits=8, seed=11, **HYPER)
    opt.step([g])
    gs = _np(g[-300:]).astype(np.float32)
    f = np.float32
    m, v = gs * f(1 - 0.9), (gs * gs) * f(1 - 0.99)
    key = R.mix32(R.mix32(R.mix32(11) ^ 0) + 1)
    key = R.mix32(R.mix32(key + 0) + 1)  # of tensor 0, upper half 1
    h = [R.mix32(k ^ key) for k in range(300)]
    um = np.array([(x >> 16) + 0.5 for x in h]) / 65536
    uv = np.array([(x & 0xFFFF) + 0.5 for x in h]) / 65536
    cm, xm = R.encode(R.pad256(m), 4, R.pad256(um))
    cv, xv = R.encode(R.pad256(v), 5, R.pad256(uv))
    assert np.array_equal(opt.m[-512:].cpu().numpy(), cm)
    assert np.array_equal(opt.v[-512:].cpu().numpy(), cv)
    assert np.array_equal(opt.m_exp[-2:].cpu().numpy(), xm)
    assert np.array_equal(opt.v_exp[-2:].cpu().numpy(), xv)
    assert (p[:1000] == 0).all() and (p[-300:] != 0).all()


# --------------------------------------------------------- captured graphs --


def test_calls_in_a_captured_graph():
    """Chained launches and workspaces from the graph's pool: replays follow their
    inputs."""
    cg = _cg()
    gen = torch.Generator().manual_seed(4)
    norm = cg.IrrepsNorm("16x0e+16x1o")
    idx = _index(5000, 60, torch.int32, 3)
    x, b, gh, gy = (_rows(gen, 500, 64, F32) for _ in range(4))
    table, g = _rows(gen, 60, 40, F32), _rows(gen, 5000, 40, F32)

    def work():
        h, y = norm.residual_forward(x, b)
        return [cg.embed_forward(idx, table), cg.embed_backward(idx, g, 60), h, y,
                *(t for t in norm.residual_backward(b, h, gh, gy) if t is not None)]

    work()  # kernels load before the capture
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for k in range(3):
        for t in (x, b, gh, gy, table, g):
            t.copy_(torch.randn(t.shape, generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, e) for a, e in zip(got, work())), k


# ------------------------------------------------------- streams, refusals --

def test_calls_follow_the_current_stream():
    """Work queued before the call on the same side stream is seen by it."""
    cg = _cg()
    gen = torch.Generator().manual_seed(1)
    table = _rows(gen, 50, 64, F32)
    norm = cg.IrrepsNorm("64x0e")
    idx = _index(4000, 50, torch.int32, 1)
    ref = norm.forward(cg.embed_forward(idx, table, 2.0))
    gref = cg.embed_backward(idx, ref, 50)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        late = torch.zeros_like(table)
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(5):
            big = big @ big * 1e-2
        late.copy_(table)
        out = norm.forward(cg.embed_forward(idx, late, 2.0))
        g = cg.embed_backward(idx, out, 50)
    side.synchronize()
    assert torch.equal(out, ref) and torch.equal(g, gref)


def test_binding_refusals():
    cg = _cg()
    idx = torch.zeros(4, dtype=torch.int32, device="cuda")
    t = torch.zeros(5, 8, device="cuda")
    bad = [
        lambda: cg.embed_forward(idx.float(), t), lambda: cg.embed_forward(idx[::2], t),
        lambda: cg.embed_forward(idx, t.t()), lambda: cg.embed_forward(idx, t.int()),
        lambda: cg.embed_forward(idx, t, out=torch.zeros(4, 7, device="cuda")),
        lambda: cg.embed_forward(idx, t, out=torch.zeros(4, 8, device="cuda", dtype=F64)),
        lambda: cg.embed_forward(idx, t, out=torch.zeros(8, 4, device="cuda").t()),
        lambda: cg.embed_backward(idx, t, 5), lambda: cg.embed_backward(idx.cpu(), t[:4], 5),
        lambda: cg.embed_backward(idx, t[:4], 5, out=torch.zeros(5, 7, device="cuda")),
        lambda: cg.embed_backward(idx.repeat(800), t[:1].expand(3200, 8), 5,
                                  workspace=torch.zeros(16, device="cuda")),
    ]
    norm = cg.IrrepsNorm("8x0e")
    w = torch.ones(8, device="cuda")
    bad += [
        lambda: norm.forward(t.double()), lambda: norm.forward(t[:, :7]),
        lambda: norm.forward(t, w.double()), lambda: norm.forward(t, w[:7]),
        lambda: norm.backward(t, t[:4]),
        lambda: norm.residual_forward(t, t, out=(t, t)),
        lambda: norm.residual_backward(t, None, None),
        lambda: norm.residual_backward(t, None, t, t),
        lambda: norm.residual_forward(None, t, gate=w.expand(4, 8)),
        lambda: norm.forward(t, out=torch.zeros(1, 8, device="cuda").expand(5, 8)),
    ]
    p = [torch.zeros(10, device="cuda")]
    opt = cg.AdamW(p)
    bad += [
        lambda: opt.step([]), lambda: opt.step([torch.zeros(9, device="cuda")]),
        lambda: opt.step([torch.zeros(20, device="cuda")[::2]]),
        lambda: opt.step([torch.zeros(10, device="cuda", dtype=F64)]),
        lambda: opt.step([torch.zeros(10)]), lambda: opt.state_values(),
        lambda: opt.step([torch.zeros(10, device="cuda")], lr=float("nan")),
        lambda: cg.AdamW([]), lambda: cg.AdamW(p, state_bits=16),
        lambda: cg.AdamW([p[0].double()], state_bits=8), lambda: cg.AdamW([p[0].int()]),
        lambda: cg.AdamW([p[0], p[0].double()]), lambda: cg.AdamW(p, copy_dtype=F64),
    ]
    for k, f in enumerate(bad):
        with pytest.raises(cg.CgtpError):
            f()
            pytest.fail(f"call {k} was not refused")
    assert opt.step_count == 0


# ------------------------------------------ rows of every width of access --

ACCESS_EMBED = [  # n, v, d, pad, shift: accesses of 16, 8, 4 and 2 bytes in both directions
    (2500, 30, 1004, 0, 0), (2500, 30, 1002, 0, 0), (2500, 30, 1001, 0, 0), (2100, 500, 34, 0, 0),
    (1500, 40, 36, 8, 4), (1500, 40, 40, 6, 2), (400, 10, 78, 2, 0), (400, 10, 140, 4, 0),
    (400, 10, 140, 4, 2), (1, 3, 2, 0, 0), (33, 9, 514, 0, 0),
]


@pytest.mark.parametrize("dtype", TYPES, ids=name)
@pytest.mark.parametrize("case", ACCESS_EMBED, ids=lambda c: "-".join(map(str, c)))
def test_embed_rows_of_every_alignment(case, dtype):
    test_embed_forward(case, dtype)
    test_embed_backward(case, dtype)


ACCESS_NORM = [  # n, irreps, pad, shift: single elements, groups of each size
    (37, "65x0e", 0, 0), (3000, "101x0e", 0, 0), (37, "131x0e", 0, 0), (2100, "257x0e", 0, 0),
    (700, "777x0e", 0, 0), (300, "1501x0e", 0, 0), (9, "3001x0e", 0, 0), (200, "4001x0e", 0, 0),
    (9, "8001x0e", 0, 0), (9, "8192x0e", 3, 1), (600, "128x0e", 3, 1), (9, "33x0e+101x0o", 0, 0),
    (9, "3001x0e+5x0o", 0, 0), (900, "67x0e+67x1o+67x2e", 0, 0), (9, "128x0e+65x1o+97x3o", 0, 0),
    (9, "67x0e+33x1o", 0, 0), (9, "67x0e+9001x0o", 0, 0), (9, "67x0e+300x1o", 0, 0),
]


@pytest.mark.parametrize("dtype", TYPES, ids=name)
@pytest.mark.parametrize("case", ACCESS_NORM, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}-{c[3]}")
def test_norm_rows_of_every_group_size(case, dtype):
    test_norm(case, dtype)
    test_residual(case, dtype)
