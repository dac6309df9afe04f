"""A classifier around variational circuits: dense encoder, circuits, dense readout, AdamW.

    python examples/hybrid_readout.py [--steps 60] [--bits 8]

A sample's 64 features become the encoding angles of a 6-qubit circuit through a fixed dense
layer (pi * sigmoid); three circuits measure Z on qubit 0, Z on qubit 5 and X on qubit 2; a
dense residual readout turns their expectation values into a label in [-1, 1].  One AdamW
updates the circuits' angles and the readout's weights.  The data are synthetic: two noisy
clusters of opposite label.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from qml_gradients_amd.optim import AdamW  # noqa: E402
from qml_gradients_amd.torch_layer import DenseLayer, HEALayer  # noqa: E402

FEATURES, QUBITS, LAYERS, HIDDEN = 64, 6, 3, 32
OBSERVABLES = ((1 << 0, 0), (1 << 5, 0), (0, 1 << 2))   # (Z part, X part)


class HybridClassifier(torch.nn.Module):
    def __init__(self, max_batch):
        super().__init__()
        self.encode = DenseLayer(FEATURES, QUBITS, max_batch, activation="sigmoid", alpha=math.pi)
        self.encode.requires_grad_(False)   # the circuits' gradient goes to their angles, not to x
        self.circuits = torch.nn.ModuleList(
            HEALayer(QUBITS, LAYERS, max_batch, obs_mask=z, obs_x_mask=x) for z, x in OBSERVABLES)
        self.widen = DenseLayer(len(OBSERVABLES), HIDDEN, max_batch, activation="tanh")
        self.mix = DenseLayer(HIDDEN, HIDDEN, max_batch, activation="gelu")
        self.answer = DenseLayer(HIDDEN, 1, max_batch, activation="tanh")

    def forward(self, features):
        angles = self.encode(features)
        h = self.widen(torch.stack([c(angles) for c in self.circuits], dim=1))
        h = self.mix(h, residual=h)
        return self.answer(h)[:, 0]


def data(samples, seed):
    """Two clusters along one random direction, labels -1 and +1."""
    g = torch.Generator().manual_seed(seed)
    y = torch.randint(0, 2, (samples,), generator=g).float() * 2 - 1
    direction = torch.randn(FEATURES, generator=g)
    x = y[:, None] * direction + 0.7 * torch.randn(samples, FEATURES, generator=g)
    return x.cuda(), y.cuda()


def train(steps=60, bits=32, batch=64, seed=0, report=None):
    """The mean-squared error of every step."""
    torch.manual_seed(seed)
    model = HybridClassifier(batch)
    opt = AdamW([p for p in model.parameters() if p.requires_grad], lr=2e-2, state_bits=bits)
    x, y = data(batch, seed + 1)
    losses = []
    for k in range(steps):
        opt.zero_grad()
        loss = torch.mean((model(x) - y) ** 2)
        loss.backward()
        opt.step()
        losses.append(loss.detach())
        if report and k % 10 == 0:
            report(f"step {k}: loss {float(losses[-1]):.4f}")
    return [float(v) for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--bits", type=int, default=32, choices=(8, 32))
    a = ap.parse_args()
    got = train(a.steps, a.bits, report=lambda line: print(line, flush=True))
    print(f"loss {got[0]:.4f} -> {got[-1]:.4f}")
