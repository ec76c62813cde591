"""The example that runs the training operators together with the product: its
gradients against differences of its own forward in fp64, and its loss falling
with 32-bit and with 8-bit optimiser states."""
import importlib.util
import os

import pytest

from tests.gpu_util import need_gpu, torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "train_species_energies.py")


def _example():
    need_gpu()
    spec = importlib.util.spec_from_file_location("train_species_energies", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_every_gradient_against_differences():
    """Central differences with a step of 1e-5 on a loss of order one: truncation
    about 1e-10 and rounding about 1e-16 / 1e-5 relative to it."""
    ex = _example()
    net = ex.Network(channels=8, layers=2, dtype=torch.float64)
    graph, vec, z, target = ex.molecules(3, 6, torch.float64)

    def loss():
        off = net.forward(graph, vec, z) - target
        return off, (off * off).mean().item()

    off, base = loss()
    grads = dict(zip(net.params, net.backward(2 * off / off.numel())))
    gen = torch.Generator("cuda").manual_seed(0)
    for name, p in net.params.items():
        d = torch.randn(p.shape, dtype=p.dtype, device="cuda", generator=gen)
        keep = p.clone()
        ends = []
        for s in (1, -1):
            p.copy_(keep + s * 1e-5 * d)
            ends.append(loss()[1])
        p.copy_(keep)
        slope = (ends[0] - ends[1]) / 2e-5
        exact = (grads[name] * d).sum().item()
        size = (grads[name] * d).abs().sum().item()
        assert size > 0, name
        assert abs(slope - exact) <= 1e-6 * size + 1e-9 * base, (name, slope, exact)


@pytest.mark.parametrize("bits", [32, 8])
def test_loss_falls(bits):
    ex = _example()
    losses = ex.train(120, state_bits=bits, count=32)
    first, last = sum(losses[:8]) / 8, sum(losses[-8:]) / 8
    assert last < 0.25 * first, (first, last)
