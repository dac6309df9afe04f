"""The 8-bit dense layer, group norm and Muon in a run as they are used: dense layers over image patches with a norm between them,
trained by Muon and AdamW, then served in 8-bit integers; every step against torch in 64 bits."""
import math
import os
import sys

import pytest

from gpu_util import say
from layers_reference import codes64, orthogonal

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


class Plain:
    """widen, norm, mix and a readout in 64 bits under autograd, with the parameters of the library's layers."""

    def __init__(self, layers, groups):
        self.p = {n: t.detach().double().requires_grad_() for n, t in layers.items()}
        self.groups = groups

    def forward(self, x, codes=None):
        p = self.p

        def product(x, name):
            if codes is None:
                return x @ p[name + ".w"].t()
            c, s = codes64(p[name + ".w"].detach().float())
            cx, sx = codes64(x.float())
            return ((cx.double() @ c.double().t()) * sx.double()[:, None] * s.double())

        lead = x.shape[:2]
        h = (product(x.reshape(-1, x.shape[-1]), "widen") + p["widen.b"])
        B, S, C = *lead, h.shape[-1]
        X = h.view(B, S, self.groups, C // self.groups)
        hat = (X - X.mean((1, 3), keepdim=True)) / torch.sqrt(X.var((1, 3), correction=0, keepdim=True) + 1e-5)
        h = torch.nn.functional.silu(hat.reshape(B, S, C) * p["norm.w"] + p["norm.b"])
        f = torch.nn.functional.gelu(product(h.reshape(-1, C), "mix") + p["mix.b"]).view(B, S, C) + h
        return f


@pytest.mark.parametrize("B,S", [(6, 49), (3, 700)])
def test_training_and_serving(B, S):
    """Losses' gradients within 1e-4 of the largest of each tensor (32-bit sums of 4,200 rows and less: 2^-24 sqrt(4200) and a
    few factors of ten), updates within Muon's 1e-5 of their size, served values within the few codes that 32 bits may round
    otherwise: one code of 127 of an input's row, in one of 32 products."""
    from qml_gradients_amd.optim import AdamW, Muon
    from qml_gradients_amd.torch_layer import DenseInt8Layer, DenseLayer, GroupNormLayer
    torch.manual_seed(3)
    K, C, G = 16, 32, 8
    widen, norm = DenseLayer(K, C, B * S), GroupNormLayer(C, G, B * S, activation="silu")
    mix = DenseLayer(C, C, B * S, activation="gelu")
    x = torch.randn(B, S, K, device="cuda")
    target = torch.randn(B, S, C, device="cuda")
    named = {"widen.w": widen.weight, "widen.b": widen.bias, "norm.w": norm.weight, "norm.b": norm.bias, "mix.w": mix.weight,
             "mix.b": mix.bias}
    matrices = [t for t in named.values() if t.dim() == 2]
    opts = [Muon(matrices, lr=0.02, weight_decay=0.1), AdamW([t for t in named.values() if t.dim() == 1], lr=0.01)]
    for step in range(3):
        say(f"[gpu] step {step} of {B} x {S}")
        plain = Plain(named, G)
        for o in opts:
            o.zero_grad()
        h = norm(widen(x))
        loss = torch.mean((mix(h, residual=h) - target) ** 2)
        loss.backward()
        want = torch.mean((plain.forward(x.double()) - target.double()) ** 2)
        want.backward()
        assert abs(float(loss.detach()) - float(want.detach())) < 1e-5 * float(want.detach())
        for n, t in named.items():
            g = plain.p[n].grad
            assert float((t.grad.double() - g).abs().max()) < 1e-4 * float(g.abs().max()), n
        before = {n: t.detach().double().clone() for n, t in named.items()}
        held = [opts[0].state[t]["momentum"].double().clone() if step else torch.zeros_like(t, dtype=torch.float64) for t in matrices]
        for o in opts:
            o.step()
        for t, m, n in zip(matrices, held, ("widen.w", "mix.w")):
            m = 0.95 * m + 0.05 * t.grad.double()
            o = orthogonal(0.95 * m + 0.05 * t.grad.double())
            f = math.sqrt(max(1.0, t.shape[0] / t.shape[1]))
            new = before[n] * (1 - 0.02 * 0.1) - 0.02 * f * o
            assert float((t.detach().double() - new).abs().max()) < 0.02 * f * 1e-4 + 1e-6
        assert all(bool((t.detach().double() != before[n]).any()) for n, t in named.items())
    widen8, mix8 = DenseInt8Layer.of(widen), DenseInt8Layer.of(mix)
    plain = Plain(named, G)
    with torch.no_grad():
        h = norm(widen8(x))
        got = mix8(h, residual=h).double()
        served, wide = plain.forward(x.double(), codes=True), plain.forward(x.double())
    # a code of 127 more or less, times the largest weight, and what the slope (below 1.13) makes of it
    code = float(h.abs().max()) / 127 * float(mix.weight.abs().max())
    assert float((got - served).abs().max()) < 1.2 * 2 * code
    assert float((got - wide).abs().max()) < 0.1 * float(wide.abs().max())   # 8 bits serve what 32 were trained to
    # what a saved model holds
    again = DenseInt8Layer(C, C, B * S, activation="gelu")
    again.load_state_dict(mix8.state_dict())
    with torch.no_grad():
        assert torch.equal(again(h, residual=h), mix8(h, residual=h))


def test_8_bits_have_no_gradient():
    from qml_gradients_amd.torch_layer import DenseInt8Layer, DenseLayer
    layer = DenseInt8Layer.of(DenseLayer(8, 4, 6, bias=False, activation="tanh"))
    x = torch.randn(6, 8, device="cuda", requires_grad=True)
    with pytest.raises(RuntimeError, match="no gradient"):
        layer(x)
    with pytest.raises(RuntimeError, match="no gradient"):
        layer(x.detach(), residual=torch.zeros(6, 4, device="cuda", requires_grad=True))
    y = layer(x.detach())
    with torch.no_grad():
        assert torch.equal(layer(x), y)
    assert not list(layer.parameters()) and layer.bias is None and layer(x.detach().view(2, 3, 8)).shape == (2, 3, 4)


def test_example_runs_and_its_gradients():
    """It trains and serves; the encoder's gradients are those of the same computation in 64 bits."""
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import hybrid_images as e
    first, second, wide, narrow = e.train(steps=3, batch=16)
    assert len(first) == len(second) == 3 and all(math.isfinite(v) for v in first + second)
    assert wide.shape == narrow.shape == (16,) and torch.isfinite(narrow).all()
    torch.manual_seed(1)
    encoder = e.Encoder(8)
    x, _ = e.data(8, 5)
    w = torch.randn(8, e.CHANNELS, device="cuda")
    (encoder(x) * w).sum().backward()
    named = {"widen.w": encoder.widen.weight, "widen.b": encoder.widen.bias, "norm.w": encoder.norm.weight,
             "norm.b": encoder.norm.bias, "mix.w": encoder.mix.weight, "mix.b": encoder.mix.bias}
    plain = Plain(named, e.GROUPS)
    n = e.SIDE // e.PATCH
    patches = x.double().view(-1, n, e.PATCH, n, e.PATCH).permute(0, 1, 3, 2, 4).reshape(8, n * n, -1)
    (plain.forward(patches).mean(1) * w.double()).sum().backward()
    for name, t in named.items():
        g = plain.p[name].grad
        assert float((t.grad.double() - g).abs().max()) < 1e-4 * float(g.abs().max()), name
