"""Infinities, NaN and magnitudes near fp32's end on the dense layer's tiles, where fp32 operands are split into bf16 planes:
results are those of fp32 products, and a layer that has diverged still runs at about its speed."""
import pytest

from gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from dense_reference import E  # noqa: E402

SHAPES = [(997, 1531, 803), (2048, 512, 1030), (5310, 1039, 24), (2584, 1112, 1984)]


def arguments(M, K, N, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, w, dy = (torch.randn(*s, generator=g, device="cuda") for s in ((M, K), (N, K), (M, N)))
    return x, torch.where(w.abs() < 0.1, torch.full_like(w, 0.5), w), torch.where(dy.abs() < 0.1, torch.ones_like(dy), dy)


def same_kind(got, want):
    """Finite, infinite or NaN where the sum is; finite ones near it."""
    got = got.double()
    for f in (torch.isnan, torch.isposinf, torch.isneginf):
        assert torch.equal(f(got), f(want)), f.__name__
    m = torch.isfinite(want)
    assert bool(((got[m] - want[m]).abs() <= 1e-3 * (1 + want[m].abs())).all())


@pytest.mark.parametrize("shape", SHAPES)
def test_infinities_and_nan_reach_what_they_meet(shape):
    import qml_gradients_amd as hq
    M, K, N = shape
    say(f"[gpu] dense non-finite {shape}")
    x, w, dy = arguments(M, K, N, 3)
    inf = float("inf")
    x[0, 5], x[20, 7] = inf, -inf
    x[30, 1], x[30, K - 1] = inf, -inf       # meets itself with either sign
    x[M - 1, K - 2] = float("nan")
    w[3, 9], w[N - 1, 0], w[7, K - 3] = inf, -inf, float("nan")
    dy[11, N - 2], dy[M - 2, 4], dy[17, 2] = inf, -inf, float("nan")
    layer = hq.Dense(K, N, M)
    y = layer.forward(x, w)
    same_kind(y, x.double() @ w.double().t().contiguous())
    dx, dw, db = layer.backward(dy, x, w)
    same_kind(dx, dy.double() @ w.double())
    same_kind(dw, dy.double().t().contiguous() @ x.double())
    same_kind(db, dy.double().sum(0))
    again = (layer.forward(x, w), *layer.backward(dy, x, w))
    for a, b in zip((y, dx, dw, db), again):
        assert torch.equal(torch.nan_to_num(a, nan=5.0), torch.nan_to_num(b, nan=5.0))


@pytest.mark.parametrize("shape", SHAPES)
def test_magnitudes_that_round_up_to_infinity(shape):
    """Finite values above bf16's largest, 3.3895e38: their sums of products stay finite and precise.  An fp32 sum of K
    products in any order is off by up to (K + 8) e of their magnitudes."""
    import qml_gradients_amd as hq
    M, K, N = shape
    x, w, _ = arguments(M, K, N, 4)
    x[5, 3], x[M - 1, K - 1], x[M // 2, 0] = 3.4e38, -3.4e38, 3.4028e38
    w = w * 1e-6
    y = hq.Dense(K, N, M).forward(x, w).double()
    want, mag = x.double() @ w.double().t().contiguous(), x.double().abs() @ w.double().abs().t().contiguous()
    assert bool(torch.isfinite(y).all()) and bool(((y - want).abs() <= (K + 8) * E * mag).all())


def fastest(call, times=6):
    best = float("inf")
    for _ in range(times):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        call()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


def test_a_diverged_layer_keeps_its_speed():
    """Nothing but NaN, one NaN among the weights, one sample of NaN: each value that is not finite was once formed anew by a
    single lane, 70 to 150 times the step; by whole blocks it is up to 4 times."""
    import qml_gradients_amd as hq
    M = K = N = 2048
    x, w, dy = arguments(M, K, N, 5)
    layer = hq.Dense(K, N, M, activation="silu")

    def times():
        _, z = layer.forward_train(x, w)
        return fastest(lambda: layer.forward_train(x, w)), fastest(lambda: layer.backward(dy, x, w, z))

    plain = times()
    x[M - 3] = float("nan")
    sample = times()
    x[M - 3] = 1.0
    w[3, K - 5] = float("nan")
    weight = times()
    x.fill_(float("nan"))
    whole = times()
    for name, got in (("one sample", sample), ("one weight", weight), ("all", whole)):
        say(f"[gpu] dense 2048^3 fp32, {name} NaN: {got[0] / plain[0]:.1f} and {got[1] / plain[1]:.1f} times the finite step")
        assert got[0] <= 12 * plain[0] and got[1] <= 12 * plain[1], name


@pytest.mark.parametrize("size", [1e-30, 1e-33, 1e-35, 1e-37, 1e-40])
def test_operands_near_the_smallest(size):
    """Planes end at bf16's smallest magnitude, 2^-133, so on tiles an operand is off by up to 2^-134: nothing to one of
    2^-109 (1.5e-33) or more, whose three planes hold all its bits."""
    import qml_gradients_amd as hq
    M, K, N = 2048, 512, 1030
    g = torch.Generator(device="cuda").manual_seed(1)
    x = (torch.rand(M, K, generator=g, device="cuda") + 0.5) * size
    w = (torch.rand(N, K, generator=g, device="cuda") - 0.5) * 1e20
    y = hq.Dense(K, N, M).forward(x, w).double()
    a, b = x.double(), w.double().t().contiguous()
    bound = (K + 8) * E * (a.abs() @ b.abs()) + (2.0 ** -134 if size < 2e-33 else 0.0) * b.abs().sum(0)
    assert bool(((y - a @ b).abs() <= bound).all())
