"""The dense layer's autograd function, without a GPU: the handle is replaced by one that computes on the CPU."""
import pytest

torch = pytest.importorskip("torch")

from qml_gradients_amd import torch_layer  # noqa: E402


class PlainDense:
    """Stands in for Dense: tanh, with a note of what was called.  Its outputs are filled from outside torch's view,
    as a kernel fills them."""

    def __init__(self, in_features, out_features, max_batch, dtype="fp32", activation="tanh", alpha=1.0, device=None):
        self.device, self.dtype, self.alpha, self.seen = torch.device("cpu"), torch.float32, alpha, []

    def _forward(self, x, w, bias, residual):
        x, w = x.detach().numpy(), w.detach().numpy()
        z = torch.from_numpy(x @ w.T) + (0.0 if bias is None else bias.detach())
        y = torch.empty(z.shape)
        y.numpy()[:] = (self.alpha * torch.tanh(z) + (0.0 if residual is None else residual.detach())).numpy()
        return y, z

    def forward(self, x, w, bias=None, residual=None):
        self.seen.append("forward")
        return self._forward(x, w, bias, residual)[0]

    def forward_train(self, x, w, bias=None, residual=None):
        self.seen.append("forward_train")
        return self._forward(x, w, bias, residual)

    def backward(self, dy, x, w, z, input=True, weight=True, bias=True):
        self.seen.append(("backward", input, weight, bias))
        dz = self.alpha * (1 - torch.tanh(z) ** 2) * dy
        return dz @ w if input else None, dz.t() @ x if weight else None, dz.sum(0) if bias else None


@pytest.fixture
def layer(monkeypatch):
    monkeypatch.setattr(torch_layer, "Dense", PlainDense)
    torch.manual_seed(0)
    return torch_layer.DenseLayer(5, 3, 16, activation="tanh", alpha=1.5)


def plain(layer, x, residual=None):
    y = 1.5 * torch.tanh(x @ layer.weight.t() + layer.bias)
    return y if residual is None else y + residual


def test_gradients_of_every_mixture_of_frozen_arguments(layer):
    for mask in range(16):
        x, r = torch.randn(2, 4, 5), torch.randn(2, 4, 3)
        args = (x, layer.weight, layer.bias, r)
        for k, t in enumerate(args):
            t.requires_grad_(bool(mask >> k & 1))
            t.grad = None
        layer.dense.seen.clear()
        y = layer(x, residual=r)
        want = plain(layer, x, r)
        assert torch.allclose(y, want, atol=1e-6) and y.requires_grad == bool(mask)
        assert layer.dense.seen == ["forward_train" if mask & 7 else "forward"]   # z only where a gradient needs it
        if not mask:
            continue
        dy = torch.randn_like(y)
        need = [t for t in args if t.requires_grad]
        for a, b in zip(torch.autograd.grad(y, need, dy), torch.autograd.grad(want, need, dy)):
            assert torch.allclose(a, b, atol=1e-5)


def test_nothing_is_kept_without_gradients(layer):
    x = torch.randn(4, 5, requires_grad=True)
    with torch.no_grad():
        y = layer(x)
    assert layer.dense.seen == ["forward"] and not y.requires_grad and torch.allclose(y, plain(layer, x), atol=1e-6)


@pytest.mark.parametrize("frozen", [False, True])
def test_a_tangent_is_refused_not_lost(layer, frozen):
    """The layer has no forward-mode derivative: never a silent zero."""
    layer.requires_grad_(not frozen)
    with torch.autograd.forward_ad.dual_level():
        x = torch.autograd.forward_ad.make_dual(torch.randn(4, 5), torch.ones(4, 5))
        with pytest.raises((RuntimeError, NotImplementedError)):
            layer(x)


def test_a_trace_holds_the_call(layer):
    """A trace of a frozen layer records its function, not an empty array that a replay would leave unfilled."""
    layer.requires_grad_(False)
    traced = torch.jit.trace(layer, torch.randn(4, 5), check_trace=False)
    x = torch.randn(4, 5)
    assert "DenseFunction" in str(traced.graph) or "PythonOp" in str(traced.graph)
    assert torch.allclose(traced(x), plain(layer, x), atol=1e-6)
