"""Trains a small equivariant network on per-atom energies of random molecules,
through the library from the embedding to the optimiser step.

    python examples/train_species_energies.py [--steps 200] [--state-bits 8]

Layer:  element embedding -> norm -> [gather, CG product under the radial
network's weights, receiver sum, channel mixing -> norm, gate, residual scale and
the next block's norm] x layers -> linear readout -> squared error.  The target
is a fixed function of the elements around each atom.  Every forward, gradient
and update is a library call; torch holds the tensors, adds two gradients and
forms the loss.
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import clebsch_gordan_tensor_gb300 as cg  # noqa: E402
import workloads as W  # noqa: E402

ELEMENTS = 119  # rows of the embedding
PRESENT = (1, 6, 7, 8, 9)
CUTOFF = 10.0


def molecules(seed, count, dtype):
    """Graph, edge vectors, elements and target energies of random molecules."""
    rng = np.random.default_rng(seed)
    pos, g = W.molecules(rng, count, 5, 12)
    z = rng.choice(PRESENT, size=g.N, p=(0.5, 0.3, 0.08, 0.1, 0.02))
    r = np.linalg.norm(g.vec, axis=1)
    pair = np.cos(z[g.receiver] * 0.7 + z[g.sender] * 0.3) * np.exp(-0.3 * r)
    target = np.sin(z * 1.3) + np.bincount(g.receiver, weights=pair, minlength=g.N)
    to = lambda a: torch.from_numpy(a).to("cuda", dtype)  # noqa: E731
    return (cg.Graph.from_numpy(g), to(g.vec), torch.from_numpy(z.astype(np.int32)).cuda(),
            to(target[:, None]))


class Network:
    """Parameters and library handles; forward() keeps what backward() reads."""

    def __init__(self, channels=32, layers=2, dtype=torch.float32, seed=0):
        self.c, self.layers, self.dtype = channels, layers, dtype
        irreps = f"{channels}x0e+{channels}x1o+{channels}x2e"
        self.plan = cg.Plan(irreps, "0e+1o+2e", irreps, dtype=dtype)
        self.mix = cg.Linear(irreps, irreps, dtype=dtype)
        self.gates = cg.Linear(f"{channels}x0e", f"{3 * channels}x0e", dtype=dtype)
        self.readout = cg.Linear(f"{channels}x0e", "1x0e", dtype=dtype)
        self.norm = cg.IrrepsNorm(irreps, eps=1e-3, dtype=dtype)
        rng = np.random.default_rng(seed)
        new = lambda *s, by: torch.from_numpy(rng.standard_normal(s) * by).to("cuda", dtype)  # noqa: E731
        ones = lambda k, v=1.0: torch.full((k,), v, dtype=dtype, device="cuda")  # noqa: E731
        n_out, ch = self.plan.weight_numel, self.norm.channels
        self.params = {"embed": new(ELEMENTS, channels, by=1.0), "norm": ones(ch),
                       "readout": new(self.readout.weight_numel, by=channels ** -0.5)}
        for k in range(layers):
            self.params |= {
                f"W1.{k}": new(8, 64, by=8 ** -0.5), f"W2.{k}": new(64, n_out, by=64 ** -0.5),
                f"mix.{k}": new(self.mix.weight_numel, by=channels ** -0.5),
                f"gate.{k}": new(self.gates.weight_numel, by=channels ** -0.5),
                f"weight.{k}": ones(ch), f"scale.{k}": ones(ch, 0.5), f"next.{k}": ones(ch)}

    def scalars(self, rows):
        return rows[:, :self.c].contiguous()

    def forward(self, graph, vec, z):
        p = self.params
        self.graph, self.vec, self.z = graph, vec, z
        self.per = float(graph.N) / graph.E
        self.sh = cg.sh_forward(vec, 2)
        x = torch.zeros(graph.N, self.norm.dim, dtype=self.dtype, device="cuda")
        cg.embed_forward(z, p["embed"], out=x[:, :self.c])  # into the scalar channels
        self.x0 = x
        y = self.norm.forward(x, p["norm"])
        self.kept = []
        for k in range(self.layers):
            w = cg.radial_forward(vec, p[f"W1.{k}"], p[f"W2.{k}"], CUTOFF)
            message = self.plan.conv_forward(graph, y, self.sh, w, self.per)
            b = self.mix.forward(message, p[f"mix.{k}"])
            s = self.scalars(y)
            gate = self.gates.forward(s, p[f"gate.{k}"])
            h, y_next = self.norm.residual_forward(x, b, p[f"weight.{k}"], gate, p[f"scale.{k}"],
                                                   p[f"next.{k}"])
            self.kept.append((y, w, message, b, s, gate, h))
            x, y = h, y_next
        self.last = self.scalars(y)
        return self.readout.forward(self.last, p["readout"])

    def backward(self, grad_energy):
        """Gradients of every parameter, in the parameters' order."""
        p, g, graph = self.params, {}, self.graph
        gs, g["readout"] = self.readout.backward(self.last, p["readout"], grad_energy)
        gy = torch.zeros_like(self.x0)
        gy[:, :self.c] = gs
        gh = None
        for k in reversed(range(self.layers)):
            y, w, message, b, s, gate, h = self.kept[k]
            gh, gb, gz, g[f"weight.{k}"], g[f"scale.{k}"], g[f"next.{k}"] = \
                self.norm.residual_backward(b, h, gh, gy, p[f"weight.{k}"], gate, p[f"scale.{k}"],
                                            p[f"next.{k}"])
            gm, g[f"mix.{k}"] = self.mix.backward(message, p[f"mix.{k}"], gb)
            gs, g[f"gate.{k}"] = self.gates.backward(s, p[f"gate.{k}"], gz)
            gy, _, gw = self.plan.conv_backward(graph, y, self.sh, w, self.per, gm,
                                                need=(True, False, True))
            _, g[f"W1.{k}"], g[f"W2.{k}"] = cg.radial_backward(
                self.vec, p[f"W1.{k}"], p[f"W2.{k}"], gw, CUTOFF, need=(False, True, True))
            gy[:, :self.c] += gs
        gx, g["norm"] = self.norm.backward(self.x0, gy, p["norm"])
        gx += gh
        g["embed"] = cg.embed_backward(self.z, gx[:, :self.c], ELEMENTS)
        return [g[k] for k in p]


def train(steps, state_bits=32, channels=32, layers=2, count=64, lr=3e-3, report=None):
    """Losses of a run."""
    net = Network(channels, layers)
    opt = cg.AdamW(net.params.values(), lr=lr, weight_decay=0.01, state_bits=state_bits)
    batches = [molecules(seed, count, torch.float32) for seed in range(8)]
    losses = []
    for t in range(steps):
        graph, vec, z, target = batches[t % len(batches)]
        off = net.forward(graph, vec, z) - target
        loss = (off * off).mean()
        opt.step(net.backward(2 * off / off.numel()))
        losses.append(loss)
        if report and (t % report == 0 or t == steps - 1):
            print(f"step {t:5d}  mean squared error {loss.item():.5f}")
    return [x.item() for x in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawTextHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--state-bits", type=int, default=32, choices=(8, 32))
    ap.add_argument("--channels", type=int, default=32)
    ap.add_argument("--layers", type=int, default=2)
    a = ap.parse_args()
    train(a.steps, a.state_bits, a.channels, a.layers, report=20)
