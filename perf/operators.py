"""Cases of the training operators around the tensor product.

Four operators of a training step: the embedding that makes a network's first
features (and its gradient), the per-irrep RMS norm before a block, the norm,
gate, residual scale and next norm after one (each with its gradient), and the
AdamW step over all of a network's parameters.

``listed()`` and ``draw()`` give the cases, ``prepare()`` makes the tensors a
training program holds before the call, ``run()`` makes one pass, in elementary
torch operations or, where ``own`` is true, through the library, and
``exact()`` evaluates the operators' definitions in 64 bits.
"""
import math

import torch
import torch.nn.functional as F

own = False

BLOCK = 256  # elements of one tensor that share the two exponents of 8-bit states
ADAM = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
SEED, STEP0 = 20240531, 10  # the rounding seed and the steps taken before the first pass

CLOUD = "64x0e+64x1o+64x2e"  # 10,000-atom cloud
MACE = "128x0e+128x1o+128x2e"  # 200,000-sample product
TFN = "32x0e+32x1o+32x2e+32x3o"  # small molecules


def listed():
    return [
        # one molecule's atoms by element, into the scalar block of its feature rows
        dict(name="embed_molecule", op="embed", rows=29, vocab=119, width=32, extra=480,
             type="float32", index="int32", skew="species"),
        # a long batch over a word-sized vocabulary, 16-bit rows
        dict(name="embed_words", op="embed", rows=131072, vocab=32000, width=1024, extra=0,
             type="bfloat16", index="int64", skew="words"),
        # the gradient of 1000 molecules' element embedding: five elements share all rows
        dict(name="embed_grad_species", op="embed_grad", rows=19310, vocab=119, width=64, extra=0,
             type="float32", index="int32", skew="species"),
        # the gradient over a word-sized vocabulary, frequencies as in text
        dict(name="embed_grad_words", op="embed_grad", rows=131072, vocab=32000, width=1024,
             extra=0, type="bfloat16", index="int64", skew="words"),
        # norm before the block, one molecule: the call's latency
        dict(name="norm_molecule", op="norm", rows=29, irreps=TFN, extra=0, type="float32"),
        # norm, gate, residual and next norm after a block of 128 channels, 200,000 rows
        dict(name="residual_mace", op="residual", rows=200000, irreps=MACE, extra=0,
             type="float32"),
        # the same over wide scalar rows in 16 bits
        dict(name="residual_wide", op="residual", rows=16384, irreps="4096x0e", extra=0,
             type="bfloat16"),
        # its gradient at the 10,000-atom cloud's sizes
        dict(name="residual_grad_cloud", op="residual_grad", rows=10000, irreps=CLOUD, extra=0,
             type="float32"),
        # its gradient over wide scalar rows in 16 bits
        dict(name="residual_grad_wide", op="residual_grad", rows=16384, irreps="4096x0e", extra=0,
             type="bfloat16"),
        # every parameter of a two-layer network of 64 channels: latency
        dict(name="adamw_small", op="adamw", layers=2, channels=64, bits=32, type="float32",
             copies=False),
        # eight layers of 1024 channels, 32-bit states: bandwidth
        dict(name="adamw_large", op="adamw", layers=8, channels=1024, bits=32, type="float32",
             copies=False),
        # the same with 8-bit states and the 16-bit copies that 16-bit weight plans read
        dict(name="adamw_large_8bit", op="adamw", layers=8, channels=1024, bits=8,
             type="float32", copies=True),
    ]


def draw(rng):
    span = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
    op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "residual", "residual_grad",
                     "adamw", "adamw"])
    kind = rng.choice(["float32", "float32", "bfloat16", "float16"])
    if op in ("embed", "embed_grad"):
        species = rng.random() < 0.5
        width = span(8, 2048)
        width -= width % 8 if rng.random() < 0.7 else 0
        rows = span(1, 262144)
        rows = min(rows, (1 << 27) // width)
        return dict(op=op, rows=rows, vocab=119 if species else span(200, 50000), width=width,
                    extra=rng.choice([0, 0, 8 * width, 5]), type=kind,
                    index=rng.choice(["int32", "int64"]), skew="species" if species else "words")
    if op == "adamw":
        return dict(op=op, layers=rng.randint(1, 8), channels=span(16, 1023),
                    bits=rng.choice([8, 32]), type=rng.choice(["float32", "float32", "bfloat16"]),
                    copies=False)
    if rng.random() < 0.35:  # scalar rows, as in a plain residual network
        width = span(64, 8192)
        width -= width % 8 if rng.random() < 0.7 else 0
        irreps = "%dx0e" % width
    else:
        mul = span(4, 256)
        mul -= mul % 4 if rng.random() < 0.7 else 0
        irreps = "+".join("%dx%d%s" % (mul, l, "eo"[l % 2]) for l in range(rng.randint(1, 4)))
    width = sum(m * (2 * l + 1) for m, l in parse(irreps))
    rows = min(span(1, 200000), (1 << 27) // width)
    return dict(op=op, rows=rows, irreps=irreps, extra=rng.choice([0, 0, 64, 3]), type=kind)


def parse(irreps):
    """[(multiplicity, l)] of an irreps string."""
    return [(int(t.split("x")[0]), int(t.split("x")[1][:-1])) for t in irreps.split("+")]


def shapes_of(case):
    """The parameters of a network of `layers` interaction blocks: the radial
    network, the two norms' weights, the residual scale, the channel mixing
    before the product and one matrix per path after it; the embedding first."""
    c = case["channels"]
    layer = [(8, 64), (64, 24 * c), (3 * c,), (3 * c,), (3 * c,), (3 * c * c,), (24, c, c)]
    return [(119, c)] + layer * case["layers"]


def layout(case):
    """Each parameter's first element in the flat states, and their length:
    every tensor starts on a block of its own."""
    at, end = [], 0
    for s in shapes_of(case):
        at.append(end)
        end += -(-math.prod(s) // BLOCK) * BLOCK
    return at, end


# ------------------------------------------------------------------ inputs --


def indices(case, gen):
    n, v = case["rows"], case["vocab"]
    if case["skew"] == "species":  # H C N O F as in small organic molecules
        share = torch.zeros(v, device="cuda")
        share[[1, 6, 7, 8, 9]] = torch.tensor([0.51, 0.35, 0.06, 0.079, 0.001], device="cuda")
        idx = torch.multinomial(share, n, replacement=True, generator=gen)
    else:  # frequency falls as one over the rank; ranks in random order
        u = torch.rand(n, device="cuda", dtype=torch.float64, generator=gen)
        rank = (float(v) ** u).long().clamp_(1, v) - 1
        idx = torch.randperm(v, device="cuda", generator=gen)[rank]
    idx[torch.rand(n, device="cuda", generator=gen) < 0.02] = -1  # padding
    return idx.to(getattr(torch, case["index"]))


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    kind = getattr(torch, case["type"])

    def normal(*shape, dtype=kind, extra=0):
        t = torch.randn(*shape[:-1], shape[-1] + extra, device="cuda", generator=gen)
        return t.to(dtype)[..., :shape[-1]]  # rows of a wider tensor where extra > 0

    s = dict(case=case, op=case["op"])
    if case["op"] in ("embed", "embed_grad"):
        s["index"], s["scale"] = indices(case, gen), math.sqrt(case["width"])
        if case["op"] == "embed":
            s["table"] = normal(case["vocab"], case["width"])
            s["out"] = torch.zeros(case["rows"], case["width"] + case["extra"], dtype=kind,
                                   device="cuda")[:, :case["width"]]
        else:
            s["grad"] = normal(case["rows"], case["width"], extra=case["extra"])
    elif case["op"] == "adamw":
        shapes, (at, end) = shapes_of(case), layout(case)
        s["params"] = [(0.05 * torch.randn(x, device="cuda", generator=gen)).to(kind)
                       for x in shapes]
        # gradients of one tensor span a few octaves; tensors differ by more
        size = 10 ** (-1 - 3 * torch.rand(len(shapes), generator=gen, device="cuda"))
        s["grads"] = [(torch.randn(x, device="cuda", generator=gen) * size[k]
                       * torch.exp2(2 * torch.randn(x, device="cuda", generator=gen))).to(kind)
                      for k, x in enumerate(shapes)]
        # the states of a program that has taken STEP0 steps
        m, v = torch.zeros(end, device="cuda"), torch.zeros(end, device="cuda")
        for k, (g, a) in enumerate(zip(s["grads"], at)):
            g = g.reshape(-1).float()
            m[a:a + g.numel()] = 0.4 * g + 0.3 * size[k] * torch.randn(
                g.numel(), device="cuda", generator=gen)
            v[a:a + g.numel()] = 0.01 * (g * g + size[k] ** 2 * torch.rand(
                g.numel(), device="cuda", generator=gen))
        s["step"] = STEP0
        if case["bits"] == 8:
            s["m"], s["m_exp"] = encode(m, 4, 1 << 19)
            s["v"], s["v_exp"] = encode(v, 5, 1 << 19)
            at_block = torch.tensor(at + [end], device="cuda") // BLOCK
            s["tensor"] = torch.repeat_interleave(torch.arange(len(at), device="cuda"),
                                                  at_block.diff())
            s["place"] = torch.arange(end, device="cuda") - BLOCK * at_block[s["tensor"]] \
                .repeat_interleave(BLOCK)
        else:
            s["m"], s["v"] = m, v
        if case["copies"]:
            s["copy"] = torch.zeros(end, dtype=torch.bfloat16, device="cuda")
        if own:
            import clebsch_gordan_tensor_gb300 as cg
            opt = cg.AdamW(s["params"], lr=ADAM["lr"], betas=(ADAM["beta1"], ADAM["beta2"]),
                           eps=ADAM["eps"], weight_decay=ADAM["weight_decay"],
                           state_bits=case["bits"], seed=SEED,
                           copy_dtype=torch.bfloat16 if case["copies"] else None)
            opt.step_count = STEP0
            opt.m.copy_(s["m"])
            opt.v.copy_(s["v"])
            if case["bits"] == 8:
                opt.m_exp.copy_(s["m_exp"])
                opt.v_exp.copy_(s["v_exp"])
            s["opt"] = opt
    else:
        blocks = parse(case["irreps"])
        n, chans = case["rows"], sum(m for m, _ in blocks)
        width = sum(m * (2 * l + 1) for m, l in blocks)
        wide = lambda: normal(n, width, extra=case["extra"])  # noqa: E731
        weight = lambda: 1 + 0.1 * normal(chans, dtype=torch.float32)  # noqa: E731
        s["b"], s["weight"] = wide(), weight()
        if case["op"] == "norm_grad":
            s["grad_y"] = wide()
        if case["op"] in ("residual", "residual_grad"):
            s["x"], s["gate"] = wide(), normal(n, chans)
            s["scale"], s["next_weight"] = 0.3 * weight(), weight()
        if case["op"] == "residual_grad":
            s["grad_h"], s["grad_y"] = wide(), wide()
            s["h"] = Plain(s).residual(s["b"], s["x"])[0]  # kept by the forward pass
        if own:
            import clebsch_gordan_tensor_gb300 as cg
            s["norm"] = cg.IrrepsNorm(case["irreps"], eps=1e-5, dtype=kind)
    return s


# ------------------------------------------------------------ plain forms --


class Plain:
    """The norm and the gated residual in 32 bits.  A feature row holds its
    irreps one after another, [2l+1, channels] each; rows of weights and gates
    hold one value per irrep and channel."""

    def __init__(self, s):
        self.blocks = parse(s["case"]["irreps"])
        self.s, self.kind = s, getattr(torch, s["case"]["type"])

    def split(self, t):
        return torch.split(t.float(), [m * (2 * l + 1) for m, l in self.blocks], 1)

    def wide(self, t):
        """A value per channel, over the 2l+1 components."""
        parts = torch.split(t.float(), [m for m, _ in self.blocks], -1)
        return torch.cat([p.repeat(*([1] * (p.dim() - 1)), 2 * l + 1)
                          for p, (_, l) in zip(parts, self.blocks)], -1)

    def narrow(self, t):
        """The sum over the 2l+1 components."""
        return torch.cat([p.unflatten(1, (2 * l + 1, m)).sum(1)
                          for p, (m, l) in zip(self.split(t), self.blocks)], 1)

    def mean(self, t):
        """Each irrep's mean, at each of its elements."""
        return torch.cat([p.mean(1, keepdim=True).expand_as(p) for p in self.split(t)], 1)

    def rsqrt(self, t):
        return torch.rsqrt(self.mean(t * t) + 1e-5)

    def norm(self, t, weight):
        t = t.float()
        return t * self.rsqrt(t) * self.wide(weight)

    def norm_grad(self, t, weight, g):
        t, g = t.float(), g.float()
        r = self.rsqrt(t)
        t = t * r
        gw = g * self.wide(weight)
        return r * (gw - t * self.mean(gw * t)), self.narrow(g * t)

    def residual(self, b, x):
        s = self.s
        gate = self.wide(torch.sigmoid(s["gate"].float()) * s["scale"])
        h = (x.float() + gate * self.norm(b, s["weight"])).to(self.kind)
        return h, self.norm(h, s["next_weight"]).to(self.kind)

    def residual_grad(self):
        s = self.s
        gx, g_next = self.norm_grad(s["h"], s["next_weight"], s["grad_y"])
        gx = gx + s["grad_h"].float()
        sig = torch.sigmoid(s["gate"].float())
        gb, dot = self.norm_grad(s["b"], s["weight"], gx * self.wide(sig * s["scale"]))
        b = s["b"].float()
        dot = self.narrow(gx * b * self.rsqrt(b))
        return dict(grad_x=gx.to(self.kind), grad_b=gb.to(self.kind),
                    grad_gate=(dot * s["scale"] * s["weight"] * sig * (1 - sig)).to(self.kind),
                    grad_weight=(dot * s["scale"] * sig).sum(0),
                    grad_scale=(dot * s["weight"] * sig).sum(0), grad_next_weight=g_next.sum(0))


def mix32(h):
    """The 32-bit finaliser of MurmurHash3 (A. Appleby, public domain), on
    Python integers or int64 tensors."""
    h = ((h ^ (h >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    h = ((h ^ (h >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


def random_bits(s):
    """The 32 random bits of every state element at the current step."""
    key = mix32(mix32(mix32(SEED & 0xFFFFFFFF) ^ (SEED >> 32)) + s["step"] & 0xFFFFFFFF)
    keys = [mix32(mix32(key + k & 0xFFFFFFFF)) for k in range(len(s["params"]))]
    keys = torch.tensor(keys, device="cuda")[s["tensor"]].repeat_interleave(BLOCK)
    return mix32(s["place"] ^ keys)  # places stay below 2^32


def bits_of(t):
    return t.view(torch.int32)


def power2(e):
    """2^e for integer tensors -126 <= e <= 126, exactly."""
    return ((e.int() + 127) << 23).view(torch.float32)


def encode(t, ebits, noise):
    """8-bit floats of `ebits` exponent and 3 fraction bits (a sign where that
    leaves one), under one power of two per block of 256: (codes, exponents).
    noise: 20 random bits per value, added below the last bit kept."""
    t = t.view(-1, BLOCK)
    top = bits_of(t.abs()).amax(1, keepdim=True)
    e = ((top >> 23) - 126).clamp(-80, 126)
    y = t.abs() * power2(-e) * 2.0 ** (-127 + 2 ** ebits)
    most = 2 ** (ebits + 3) - 1
    noise = noise.view(-1, BLOCK) if isinstance(noise, torch.Tensor) else noise
    c = (bits_of(y) + noise >> 20).clamp(max=most)
    if ebits == 5:
        c = torch.where(t > 0, c.clamp(min=1), c)  # a second moment never rounds to nothing
    else:
        c = c | (bits_of(t) >> 24 & 0x80)
    return c.to(torch.uint8).view(-1), (e + 128).to(torch.uint8).view(-1)


def decode(codes, exps, ebits):
    c = codes.view(-1, BLOCK).int()
    most = 2 ** (ebits + 3) - 1
    t = (c.bitwise_and(most) << 20).view(torch.float32) * 2.0 ** (127 - 2 ** ebits)
    t = t * power2(exps.int().view(-1, 1) - 128)
    return (torch.where(c > most, -t, t) if most < 255 else t).view(-1)


def flat(tensors):
    return torch.cat([F.pad(t.reshape(-1).float(), (0, -t.numel() % BLOCK)) for t in tensors])


def adamw(s):
    case, a = s["case"], ADAM
    s["step"] += 1
    t = s["step"]
    keep = 1 - a["lr"] * a["weight_decay"]
    rate = a["lr"] / (1 - a["beta1"] ** t)
    root = 1 / math.sqrt(1 - a["beta2"] ** t)
    g, p = flat(s["grads"]), flat(s["params"])
    eight = case["bits"] == 8
    m = decode(s["m"], s["m_exp"], 4) if eight else s["m"]
    v = decode(s["v"], s["v_exp"], 5) if eight else s["v"]
    m = m * a["beta1"] + g * (1 - a["beta1"])
    v = v * a["beta2"] + g * g * (1 - a["beta2"])
    p = p * keep - rate * m / (v.sqrt() * root + a["eps"])
    parts = [x[:q.numel()].view(q.shape) for x, q in zip(torch.split(
        p, [-(-q.numel() // BLOCK) * BLOCK for q in s["params"]]), s["params"])]
    torch._foreach_copy_(s["params"], parts)
    out = dict(params=s["params"])
    if case["copies"]:
        s["copy"].copy_(p)
        out["copy"] = s["copy"]
    if eight:
        r = random_bits(s)
        codes, exps = encode(m, 4, ((r >> 16 << 4) + 8).int())
        s["m"].copy_(codes), s["m_exp"].copy_(exps)
        codes, exps = encode(v, 5, ((r & 0xFFFF) << 4).int() + 8)
        s["v"].copy_(codes), s["v_exp"].copy_(exps)
        # three fraction bits and an eight-bit exponent: bfloat16 holds the values exactly
        out["m"] = decode(s["m"], s["m_exp"], 4).bfloat16()
        out["v"] = decode(s["v"], s["v_exp"], 5).bfloat16()
    else:
        s["m"].copy_(m), s["v"].copy_(v)
        out["m"], out["v"] = s["m"], s["v"]
    return out


def run(s):
    if own:
        return run_own(s)
    op, case = s["op"], s["case"]
    kind = getattr(torch, case["type"])
    if op == "embed":
        keep = (s["index"] >= 0).unsqueeze(1)
        rows = s["table"].float()[s["index"].long().clamp(min=0)] * s["scale"]
        return s["out"].copy_(torch.where(keep, rows, 0.0))
    if op == "embed_grad":
        keep = (s["index"] >= 0).unsqueeze(1)
        g = torch.where(keep, s["grad"].float() * s["scale"], 0.0)
        total = torch.zeros(case["vocab"], case["width"], device="cuda")
        return total.index_add_(0, s["index"].long().clamp(min=0), g).to(kind)
    if op == "adamw":
        return adamw(s)
    plain = Plain(s)
    if op == "norm":
        return plain.norm(s["b"], s["weight"]).to(kind)
    if op == "norm_grad":
        g, gw = plain.norm_grad(s["b"], s["weight"], s["grad_y"])
        return g.to(kind), gw.sum(0)
    if op == "residual":
        return plain.residual(s["b"], s["x"])
    return plain.residual_grad()


def run_own(s):
    import clebsch_gordan_tensor_gb300 as cg
    op = s["op"]
    if op == "embed":
        return cg.embed_forward(s["index"], s["table"], s["scale"], out=s["out"])
    if op == "embed_grad":
        return cg.embed_backward(s["index"], s["grad"], s["case"]["vocab"], s["scale"])
    if op == "adamw":
        opt = s["opt"]
        opt.step(s["grads"])
        m, v = opt.state_values() if s["case"]["bits"] == 8 else (opt.m, opt.v)
        out = dict(params=s["params"], m=m, v=v)
        return dict(out, copy=opt.copy) if s["case"]["copies"] else out
    norm = s["norm"]
    if op == "norm":
        return norm.forward(s["b"], s["weight"])
    if op == "norm_grad":
        return norm.backward(s["b"], s["grad_y"], s["weight"])
    if op == "residual":
        return norm.residual_forward(s["x"], s["b"], s["weight"], s["gate"], s["scale"],
                                     s["next_weight"])
    grads = norm.residual_backward(s["b"], s["h"], s["grad_h"], s["grad_y"], s["weight"],
                                   s["gate"], s["scale"], s["next_weight"])
    return dict(zip(("grad_x", "grad_b", "grad_gate", "grad_weight", "grad_scale",
                     "grad_next_weight"), grads))


# ---------------------------------------------------------- work and truth --


def work(case):
    size = 4 if case.get("type") == "float32" else 2
    if case["op"] in ("embed", "embed_grad"):
        n, v, d = case["rows"], case["vocab"], case["width"]
        # distinct rows: five elements, or what draws by one over the rank reach
        seen = min(n, 5) if case["skew"] == "species" else min(
            v, int(sum(1 - (1 - math.log1p(1 / k) / math.log(v)) ** n for k in range(1, v))))
        index = 4 if case["index"] == "int32" else 8
        if case["op"] == "embed":
            return dict(bytes=n * index + (n + seen) * d * size, flops=n * d)
        return dict(bytes=n * index + (n + v) * d * size, flops=2 * n * d)
    if case["op"] == "adamw":
        n = sum(math.prod(s) for s in shapes_of(case))
        # parameter in and out, gradient in; 32-bit moments in and out, or their
        # codes in and out and the values they stand for; copies out
        each = 3 * size + (2 * 2 * 4 if case["bits"] == 32 else 2 * 2 + 2 * 2)
        return dict(bytes=n * (each + (2 if case["copies"] else 0)), flops=14 * n)
    blocks = parse(case["irreps"])
    n, chans = case["rows"], sum(m for m, _ in blocks)
    width = sum(m * (2 * l + 1) for m, l in blocks)
    rows, gates, flops = {"norm": (2, 0, 4), "norm_grad": (3, 0, 10), "residual": (4, 1, 10),
                          "residual_grad": (6, 2, 24)}[case["op"]]
    return dict(bytes=n * size * (rows * width + gates * chans), flops=flops * n * width)


def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], torch.float64
    if op == "embed":
        table = torch.cat([s["table"].to(d) * s["scale"],
                           torch.zeros(1, case["width"], dtype=d, device="cuda")])
        return table[s["index"].long()]  # -1: the row of zeros
    if op == "embed_grad":
        total = torch.zeros(case["vocab"] + 1, case["width"], dtype=d, device="cuda")
        total.index_put_((s["index"].long(),), s["grad"].to(d), accumulate=True)
        return total[:-1] * s["scale"]
    if op == "adamw":
        return exact_adamw(s)

    def norm(t, weight):
        out, at, ch = [], 0, 0
        for m, l in parse(case["irreps"]):
            part = t[:, at:at + m * (2 * l + 1)].reshape(-1, 2 * l + 1, m)
            size = torch.sqrt((part ** 2).sum((1, 2), keepdim=True) / (m * (2 * l + 1)) + 1e-5)
            out.append((part / size * weight[ch:ch + m]).flatten(1))
            at, ch = at + m * (2 * l + 1), ch + m
        return torch.cat(out, 1)

    def scaled(t, by):
        out, at, ch = [], 0, 0
        for m, l in parse(case["irreps"]):
            part = t[:, at:at + m * (2 * l + 1)].reshape(-1, 2 * l + 1, m)
            out.append((part * by[:, None, ch:ch + m]).flatten(1))
            at, ch = at + m * (2 * l + 1), ch + m
        return torch.cat(out, 1)

    w = {k: s[k].to(d) for k in ("b", "x", "h", "gate", "weight", "scale", "next_weight",
                                 "grad_h", "grad_y") if k in s}
    if op == "norm":
        return norm(w["b"], w["weight"])
    if op == "norm_grad":
        leaves = [w["b"].requires_grad_(), w["weight"].requires_grad_()]
        return torch.autograd.grad(norm(*leaves), leaves, w["grad_y"])
    after = lambda: scaled(norm(w["b"], w["weight"]),  # noqa: E731
                           w["scale"] / (1 + torch.exp(-w["gate"])))
    if op == "residual":
        h = w["x"] + after()
        # the next norm takes h as it is stored
        return h, norm(h.to(getattr(torch, case["type"])).to(d), w["next_weight"])
    names = ("b", "gate", "weight", "scale", "next_weight")
    leaves = [w[k].requires_grad_() for k in names]
    h = w["h"].requires_grad_()
    gx, g_next = torch.autograd.grad(norm(h, w["next_weight"]), (h, w["next_weight"]),
                                     w["grad_y"])
    gx = gx + w["grad_h"]
    got = dict(zip(names, torch.autograd.grad(after(), leaves[:-1], gx)))
    return dict(grad_x=gx, grad_b=got["b"], grad_gate=got["gate"], grad_weight=got["weight"],
                grad_scale=got["scale"], grad_next_weight=g_next)


def exact_adamw(s):
    a, case, d = ADAM, s["case"], torch.float64
    s["step"] += 1
    t = s["step"]
    end = s["m"].numel()
    m, v = (torch.zeros(end, dtype=d, device="cuda") for _ in "mv")
    if case["bits"] == 8:  # code: sign, exponent field, three fraction bits; no hidden bit at field 0
        for to, name, ebits in ((m, "m", 4), (v, "v", 5)):
            c = s[name].to(d)
            sign = torch.ones_like(c)
            if ebits == 4:
                sign, c = torch.where(c >= 128, -1.0, 1.0), c % 128
            field, frac = torch.floor(c / 8), c % 8
            value = torch.where(field > 0, (8 + frac) * 2.0 ** (field - 1), frac)
            exps = s[name + "_exp"].to(d).repeat_interleave(BLOCK) - 128
            to.copy_(sign * value * 2.0 ** (-(2 ** ebits) - 2) * 2.0 ** exps)
    else:
        m.copy_(s["m"]), v.copy_(s["v"])
    out, copy = [], torch.zeros(end, dtype=d, device="cuda")
    for p, g, at in zip(s["params"], s["grads"], layout(case)[0]):
        w = slice(at, at + p.numel())
        g = g.to(d).reshape(-1)
        m[w] = a["beta1"] * m[w] + (1 - a["beta1"]) * g
        v[w] = a["beta2"] * v[w] + (1 - a["beta2"]) * g ** 2
        step = (m[w] / (1 - a["beta1"] ** t)) / (
            torch.sqrt(v[w] / (1 - a["beta2"] ** t)) + a["eps"])
        copy[w] = (1 - a["lr"] * a["weight_decay"]) * p.to(d).reshape(-1) - a["lr"] * step
        out.append(copy[w].view(p.shape))
    found = dict(params=out)
    if case["copies"]:
        found["copy"] = copy
    if case["bits"] == 8:
        r = random_bits(s)
        m, v = exact_round(m, 4, (r >> 16) / 65536), exact_round(v, 5, (r & 0xFFFF) / 65536)
    return dict(found, m=m, v=v)


def exact_round(t, ebits, u):
    """The 8-bit floats next to t under its block's power of two: the upper one
    where the rest below it and u (plus half a 16-bit step) reach one."""
    t, u = t.view(-1, BLOCK), u.view(-1, BLOCK) + 0.5 / 65536
    e = torch.frexp(t.abs().amax(1, keepdim=True))[1].clamp(-80, 126)
    x = t.abs() * torch.exp2(-e.double())
    low = 2 - 2 ** ebits  # the smallest exponent with a hidden bit
    step = torch.exp2(torch.frexp(x)[1].clamp(min=low).double() - 4)
    q = (torch.floor(x / step + u) * step).clamp(max=15 / 16)
    if ebits == 5:
        q = torch.where(t > 0, q.clamp(min=2.0 ** (low - 4)), q)
    return (torch.sign(t) * q * torch.exp2(e.double())).view(-1)
