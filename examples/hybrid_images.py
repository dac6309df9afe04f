"""Images into variational circuits: patches, dense and group-norm layers, circuits, readout; Muon and AdamW; served in 8 bits.

    python examples/hybrid_images.py [--steps 40]

A 28 x 28 image is cut into 7 x 7 patches of 16 pixels, channels last.  Two dense layers, each over every patch by itself,
with a group norm between them, and the mean over the patches make its features; a dense layer turns these into the
encoding angles of a 6-qubit circuit (pi * sigmoid).  Those layers are fixed for the circuits, whose gradient goes to their own
angles, so they are trained first, with an auxiliary dense readout: Muon takes their weight matrices, AdamW the biases and
the norm's parameters.  Then the circuits and their dense readout are trained on the angles.  Last, the encoder's dense
layers are served in 8-bit integers.  The data are synthetic: two blobs of opposite label at random places.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from qml_gradients_amd.optim import AdamW, Muon  # noqa: E402
from qml_gradients_amd.torch_layer import DenseInt8Layer, DenseLayer, GroupNormLayer, HEALayer  # noqa: E402

SIDE, PATCH, CHANNELS, GROUPS, QUBITS, LAYERS = 28, 4, 32, 8, 6, 2
PATCHES = (SIDE // PATCH) ** 2


class Encoder(torch.nn.Module):
    """[batch][28][28] to features [batch][CHANNELS]."""

    def __init__(self, max_batch):
        super().__init__()
        rows = max_batch * PATCHES
        self.widen = DenseLayer(PATCH * PATCH, CHANNELS, rows)
        self.norm = GroupNormLayer(CHANNELS, GROUPS, rows, activation="silu")
        self.mix = DenseLayer(CHANNELS, CHANNELS, rows, activation="gelu")

    def forward(self, images):
        n = SIDE // PATCH
        x = images.view(-1, n, PATCH, n, PATCH).permute(0, 1, 3, 2, 4).reshape(-1, n, n, PATCH * PATCH)
        x = self.norm(self.widen(x))
        return self.mix(x, residual=x).mean((1, 2))

    def served(self):
        """The same with its dense layers in 8-bit integers."""
        other = Encoder.__new__(Encoder)
        torch.nn.Module.__init__(other)
        other.widen, other.norm, other.mix = DenseInt8Layer.of(self.widen), self.norm, DenseInt8Layer.of(self.mix)
        return other


class Classifier(torch.nn.Module):
    """Features to an answer in [-1, 1] through the circuits."""

    def __init__(self, max_batch):
        super().__init__()
        self.angles = DenseLayer(CHANNELS, QUBITS, max_batch, activation="sigmoid", alpha=math.pi)
        self.angles.requires_grad_(False)   # the circuits' gradient goes to their angles, not to x
        self.circuits = torch.nn.ModuleList(HEALayer(QUBITS, LAYERS, max_batch, obs_mask=z) for z in (1, 1 << 5))
        self.answer = DenseLayer(len(self.circuits), 1, max_batch, activation="tanh")

    def forward(self, features):
        a = self.angles(features)
        return self.answer(torch.stack([c(a) for c in self.circuits], dim=1))[:, 0]


def optimisers(*modules, lr=0.02):
    """Muon for weight matrices (circuits' angles are none), AdamW for the rest."""
    p = [q for m in modules for q in m.parameters() if q.requires_grad]
    flat = [q for q in p if q.dim() != 2]
    made = [Muon([q for q in p if q.dim() == 2], lr=lr, adjust="rms")]
    return made + ([AdamW(flat, lr=lr)] if flat else [])


def data(samples, seed):
    """Blobs of brightness y at random places, in noise."""
    g = torch.Generator().manual_seed(seed)
    y = torch.randint(0, 2, (samples,), generator=g).float() * 2 - 1
    at = torch.rand(samples, 2, 1, generator=g) * 16 + 6
    grid = torch.arange(SIDE).float()
    blob = torch.exp(-0.1 * ((grid - at[:, 0])[:, :, None] ** 2 + (grid - at[:, 1])[:, None, :] ** 2))
    return (y[:, None, None] * blob + 0.2 * torch.randn(samples, SIDE, SIDE, generator=g)).cuda(), y.cuda()


def fit(model, opts, x, y, steps, report=None):
    losses = []
    for k in range(steps):
        for o in opts:
            o.zero_grad()
        loss = torch.mean((model(x) - y) ** 2)
        loss.backward()
        for o in opts:
            o.step()
        losses.append(loss.detach())
        if report and k % 10 == 0:
            report(f"step {k}: loss {float(losses[-1]):.4f}")
    return [float(v) for v in losses]


def train(steps=40, batch=64, seed=0, report=None):
    """(losses of the encoder, losses of the circuits, answers in 32 bits, answers with the encoder in 8)."""
    torch.manual_seed(seed)
    encoder, head = Encoder(batch), DenseLayer(CHANNELS, 1, batch, activation="tanh")
    x, y = data(batch, seed + 1)
    first = fit(lambda images: head(encoder(images))[:, 0], optimisers(encoder, head), x, y, steps, report)
    classifier = Classifier(batch)
    with torch.no_grad():
        features = encoder(x)
    second = fit(classifier, optimisers(classifier), features, y, steps, report)
    with torch.no_grad():
        return first, second, classifier(features), classifier(encoder.served()(x))


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=40)
    a = ap.parse_args()
    one, two, wide, narrow = train(a.steps, report=lambda line: print(line, flush=True))
    print(f"encoder {one[0]:.4f} -> {one[-1]:.4f}, circuits {two[0]:.4f} -> {two[-1]:.4f}, "
          f"answers in 8 bits off by {float((wide - narrow).abs().max()):.4f} at most")
