"""Group norm with an activation against its definition in 64 bits, within bounds that layers_reference derives."""
import pytest

from gpu_util import say
from layers_reference import ACTS, TYPES, excess, norm

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def make(B, S, C, dtype, seed, offset=0, gap=0, affine=True):
    """x and dy with positions `gap` elements apart and NaN between them; channels of unlike sizes and means."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def positions(t):
        wide = torch.full((B * S * (C + gap) + offset,), float("nan"), dtype=TYPES[dtype][0], device="cuda")
        v = wide[offset:].view(B, S, C + gap)[..., :C]
        v.copy_(t)
        return v

    x = positions(normal(B, S, C) * torch.exp(0.5 * normal(C)) + 3 * normal(C))
    dy = positions(normal(B, S, C))
    if not affine:
        return x, dy, None, None
    return x, dy, (1 + 0.3 * normal(C)).to(TYPES[dtype][0]), (0.3 * normal(C)).to(TYPES[dtype][0])


def check(B, S, C, G, dtype, act, seed=1, eps=1e-5, layer=None, **how):
    import qml_gradients_amd as hq
    say(f"[gpu] norm {B} x {S} x {C} in {G} groups, {dtype} {act}")
    x, dy, gamma, beta = make(B, S, C, dtype, seed, **how)
    layer = layer or hq.GroupNorm(C, G, B * S, dtype=dtype, activation=act, eps=eps)
    y, mean, rstd = layer.forward_train(x, gamma, beta)
    dx, dgamma, dbeta = layer.backward(dy, x, gamma, beta, mean, rstd)
    got = dict(y=y, mean=mean, rstd=rstd, dx=dx, dgamma=dgamma, dbeta=dbeta)
    want = norm(x, gamma, beta, dy, G, act, eps, dtype)
    for name, t in got.items():
        assert excess(t, want[name]) <= 0, (name, excess(t, want[name]))
    assert torch.equal(y, layer.forward(x, gamma, beta))
    again = layer.backward(dy, x, gamma, beta, mean, rstd)
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dgamma, dbeta)))
    # each gradient by itself
    assert torch.equal(layer.backward(dy, x, gamma, beta, mean, rstd, parameters=False)[0], dx)
    _, dw, db = layer.backward(dy, x, gamma, beta, mean, rstd, input=False)
    assert torch.equal(dw, dgamma) and torch.equal(db, dbeta)
    return layer


SIZES = [  # B, S, C, G: one workgroup and many, spans, chunks, one position, one channel a group, one group
    (1, 1, 1, 1), (1, 1, 2, 1), (1, 1, 8, 2), (3, 5, 7, 7), (2, 1, 784, 16), (1000, 1, 33, 11), (1, 784, 32, 8),
    (61, 49, 123, 41), (5, 49, 64, 1), (4, 17, 100, 100), (2, 3000, 16, 2), (1, 5000, 8, 8), (300, 16, 48, 3),
    (2, 600, 512, 32), (1, 40, 2048, 4), (1, 1500, 1, 1), (1, 40000, 3, 3), (700, 2, 5, 1), (2, 100, 1536, 1)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,S,C,G", SIZES)
def test_sizes(B, S, C, G, dtype):
    acts = ACTS if B * S * C < 20000 else (ACTS[(B + S) % 6], ACTS[(S + C + 3) % 6])
    for n, act in enumerate(acts):
        check(B, S, C, G, dtype, act, seed=n, affine=n != 1, offset=n % 2, gap=3 * (n % 2))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,S,C,G", [(1, 3, 4096, 1), (2, 9, 4096, 4096), (1, 30, 4096, 2), (3, 1, 4096, 64), (1, 9, 4095, 5),
                                     (2, 40, 3001, 3001), (20000, 1, 4, 2), (5000, 3, 24, 24)])
def test_widest_and_longest(B, S, C, G, dtype):
    check(B, S, C, G, dtype, "silu", offset=1, gap=1)


@pytest.mark.parametrize("B,S", [(20, 110), (2, 1100)])
def test_offsets_past_32_bits(B, S):
    """Positions 2^20 values apart: the last of 2,200 are past 2^31 values."""
    import qml_gradients_amd as hq
    C, G, gap = 24, 4, (1 << 20) - 24
    layer = check(B, S, C, G, "bf16", "silu", gap=gap)
    x, _, gamma, beta = make(B, S, C, "bf16", 2, gap=gap)
    want = layer.forward(x.contiguous(), gamma, beta)
    assert torch.equal(layer.forward(x, gamma, beta, out=x), want) and torch.equal(x, want)


def test_two_handles_at_once():
    import qml_gradients_amd as hq
    B, S, C, G = 2, 5000, 64, 8
    streams = [torch.cuda.Stream() for _ in range(2)]
    layers = [hq.GroupNorm(C, G, B * S, activation="silu", stream=s.cuda_stream) for s in streams]
    data = [make(B, S, C, "fp32", n) for n in (1, 2)]

    def run(layer, x, dy, gamma, beta):
        y, mean, rstd = layer.forward_train(x, gamma, beta)
        return (y, *layer.backward(dy, x, gamma, beta, mean, rstd))

    want = [run(hq.GroupNorm(C, G, B * S, activation="silu"), *d) for d in data]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for layer, d, s in zip(layers, data, streams):
            with torch.cuda.stream(s):
                got.append(run(layer, *d))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for i, r in enumerate(got) for a, b in zip(r, want[i % 2]))


def test_fewer_rows_than_the_handle_allows():
    """Sizes change from call to call, from one kernel to another and back."""
    import qml_gradients_amd as hq
    layer = hq.GroupNorm(96, 6, 9000, activation="tanh")
    for B, S in ((1, 9000), (9000, 1), (3, 3000), (2, 7), (40, 200), (1, 1), (3, 2999)):
        check(B, S, 96, 6, "fp32", "tanh", layer=layer)


def test_large_means_keep_the_variance():
    """The variance is formed of distances from the mean, so a mean 1,000 times as large does not cost it its bits (one of
    squares would be off by 1e6 units of 2^-24, the size of the variance's own 6 %)."""
    import qml_gradients_amd as hq
    for B, S, C, G in ((2, 100, 32, 4), (1, 30000, 32, 4)):
        g = torch.Generator(device="cuda").manual_seed(3)
        x = torch.randn(B, S, C, generator=g, device="cuda") + 1000
        layer = hq.GroupNorm(C, G, B * S)
        y, mean, rstd = layer.forward_train(x)
        X = x.double().view(B, S, G, C // G)
        want = 1 / torch.sqrt(X.var((1, 3), correction=0) + 1e-5)
        # the mean is off by at most a few units of 1000 2^-24, squared 4e-9 of the variance; sums of squares 700 2^-24
        assert float((rstd.double() / want - 1).abs().max()) < 708 * 2.0 ** -24
        got = layer.backward(torch.ones_like(x), x, None, None, mean, rstd)[0]
        assert float(got.abs().max()) < 1e-2   # a constant's gradient is 0 up to xhat's rounding


def test_layouts():
    """[samples][channels], several axes of positions, channels cut out of wider rows, a transposed array, out in place."""
    import qml_gradients_amd as hq
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(6, 5, 4, 24, generator=g, device="cuda")
    w, b = torch.randn(24, generator=g, device="cuda"), torch.randn(24, generator=g, device="cuda")
    layer = hq.GroupNorm(24, 4, 200, activation="gelu")
    y, mean, rstd = layer.forward_train(x, w, b)
    assert y.shape == x.shape and torch.equal(y.view(6, 20, 24), layer.forward(x.view(6, 20, 24), w, b))
    assert torch.equal(layer.forward(x[:, 0, 0], w, b), layer.forward(x[:, :1, 0].contiguous(), w, b)[:, 0])
    wide = torch.randn(6, 5, 4, 60, device="cuda")
    wide[..., 7:31] = x
    assert torch.equal(layer.forward(wide[..., 7:31], w, b), y)
    out = wide.clone()
    layer.forward(out[..., 7:31], w, b, out=out[..., 7:31])
    assert torch.equal(out[..., 7:31], y)
    assert torch.equal(out[..., :7], wide[..., :7]) and torch.equal(out[..., 31:], wide[..., 31:])
    turned = x.permute(3, 0, 1, 2).contiguous().permute(1, 2, 3, 0)
    assert torch.equal(layer.forward(turned, w, b), y)
    assert torch.equal(layer.forward(x.expand(6, 5, 4, 24)[:3], w, b), y[:3])
    assert torch.equal(layer.forward(x[::2], w, b), y[::2])
    one = x[:1, :1, :1].expand(1, 5, 4, 24)   # one position for all
    assert torch.equal(layer.forward(one, w, b), layer.forward(one.contiguous(), w, b))
    dy = torch.randn(6, 24, 5, 4, device="cuda").permute(0, 2, 3, 1)
    for a, c in zip(layer.backward(dy, wide[..., 7:31], w, b, mean, rstd), layer.backward(dy.contiguous(), x, w, b, mean, rstd)):
        assert torch.equal(a, c)


def test_groups_that_are_not_finite():
    """They are NaN; other groups and samples know nothing of them."""
    import qml_gradients_amd as hq
    for B, S, C, G in ((3, 10, 12, 3), (2, 4000, 48, 3)):
        x, dy, gamma, beta = make(B, S, C, "fp32", 1)
        layer = hq.GroupNorm(C, G, B * S, activation="silu")
        want, mean, rstd = layer.forward_train(x, gamma, beta)
        bad = x.clone()
        per = C // G
        bad[0, 3, 0], bad[1, S - 1, C - 1] = float("nan"), float("inf")
        y, m, r = layer.forward_train(bad, gamma, beta)
        hit = torch.zeros(B, G, dtype=torch.bool, device="cuda")
        hit[0, 0] = hit[1, G - 1] = True
        assert y.view(B, S, G, per)[:, :, :, :].permute(0, 2, 1, 3)[hit].isnan().all()
        assert torch.equal(y.view(B, S, G, per).permute(0, 2, 1, 3)[~hit], want.view(B, S, G, per).permute(0, 2, 1, 3)[~hit])
        assert torch.equal(m[~hit], mean[~hit]) and torch.equal(r[~hit], rstd[~hit])
        dx = layer.backward(dy, bad, gamma, beta, m, r)[0]
        good = layer.backward(dy, x, gamma, beta, mean, rstd)[0]
        assert torch.equal(dx.view(B, S, G, per).permute(0, 2, 1, 3)[~hit], good.view(B, S, G, per).permute(0, 2, 1, 3)[~hit])


def test_constant_groups():
    """Their variance is 0: xhat is 0 and rstd 1 / sqrt(eps)."""
    import qml_gradients_amd as hq
    layer = hq.GroupNorm(8, 2, 3000, eps=1e-4)
    for S in (5, 3000):
        x = torch.full((1, S, 8), 2.5, device="cuda")
        beta = torch.arange(8.0, device="cuda")
        y, mean, rstd = layer.forward_train(x, None, beta)
        assert torch.equal(y, beta.expand(1, S, 8)) and (mean == 2.5).all()
        assert float((rstd.double() * 1e-2 - 1).abs().max()) < 1e-6


def test_no_positions():
    import qml_gradients_amd as hq
    layer = hq.GroupNorm(8, 2, 10)
    w = torch.ones(8, device="cuda")
    for shape in ((0, 3, 8), (3, 0, 8), (0, 8)):
        x = torch.empty(shape, device="cuda")
        y, mean, rstd = layer.forward_train(x, w, w)
        assert y.shape == x.shape and mean.shape == (shape[0], 2)
        dx, dw, db = layer.backward(x, x, w, w, mean, rstd)
        assert dx.shape == x.shape and not dw.any() and not db.any()


@pytest.mark.parametrize("B,S,C,G", [(3, 20, 12, 3), (1, 3000, 24, 2)])
def test_gradient_against_differences(B, S, C, G):
    """Along one direction each: (L(+h) - L(-h)) / 2h of L = sum c y.  In 32 bits L is off by 2^-22 of its terms or so, so
    with h = 2^-6 differences are good to 2^-16 of the terms' norm, and to h^2 times the third derivative, some units of the
    slope here."""
    import qml_gradients_amd as hq
    x, c, gamma, beta = make(B, S, C, "fp32", 7)
    layer = hq.GroupNorm(C, G, B * S, activation="tanh")
    y, mean, rstd = layer.forward_train(x, gamma, beta)
    grads = layer.backward(c, x, gamma, beta, mean, rstd)
    g = torch.Generator(device="cuda").manual_seed(1)
    h = 2.0 ** -6
    for k, t in enumerate((x, gamma, beta)):
        v = torch.randn(t.shape, generator=g, device="cuda")
        sides = []
        for sign in (1, -1):
            a = [x, gamma, beta]
            a[k] = t + sign * h * v
            sides.append((layer.forward(*a).double() * c.double()))
        got = float((grads[k].double() * v.double()).sum())
        want = float((sides[0] - sides[1]).sum()) / (2 * h)
        terms = float(torch.linalg.vector_norm(((sides[0] - sides[1]) / (2 * h))))
        noise = 2.0 ** -22 / h * float(torch.linalg.vector_norm(sides[0]))
        assert abs(got - want) < 5 * (noise + 4 * h * h * terms), (k, got, want)


def test_autograd():
    """The module's gradients are the library's; what is not asked for is not formed."""
    import qml_gradients_amd as hq
    from qml_gradients_amd.torch_layer import GroupNormLayer
    torch.manual_seed(1)
    layer = GroupNormLayer(24, 3, 400, activation="gelu")
    with torch.no_grad():
        layer.weight.add_(0.3 * torch.randn(24, device="cuda"))
        layer.bias.add_(0.3 * torch.randn(24, device="cuda"))
    x = torch.randn(5, 40, 24, device="cuda", requires_grad=True)
    dy = torch.randn(5, 40, 24, device="cuda")
    y = layer(x)
    y.backward(dy)
    want = norm(x.detach(), layer.weight.detach(), layer.bias.detach(), dy, 3, "gelu", 1e-5, "fp32")
    for t, name in ((y.detach(), "y"), (x.grad, "dx"), (layer.weight.grad, "dgamma"), (layer.bias.grad, "dbeta")):
        assert excess(t, want[name]) <= 0, name
    with torch.no_grad():
        assert torch.equal(layer(x), y) and not layer(x).requires_grad
    layer.bias.requires_grad_(False)
    layer.bias.grad = layer.weight.grad = None
    layer(x.detach()).backward(dy)
    assert layer.bias.grad is None and excess(layer.weight.grad, want["dgamma"]) <= 0
    plain = GroupNormLayer(24, 3, 400, affine=False)
    x.grad = None
    plain(x).backward(dy)
    want = norm(x.detach(), None, None, dy, 3, "none", 1e-5, "fp32")
    assert excess(x.grad, want["dx"]) <= 0 and not list(plain.parameters())
    with pytest.raises(RuntimeError):   # x has changed since
        y = plain(x)
        with torch.no_grad():
            x.add_(1)
        y.backward(dy)


def test_streams_and_graphs():
    import qml_gradients_amd as hq
    own, side = torch.cuda.Stream(), torch.cuda.Stream()
    for B, S, C, G in ((4, 50, 40, 5), (2, 3000, 64, 8)):
        layer = hq.GroupNorm(C, G, B * S, activation="silu", stream=own.cuda_stream)
        x, dy, gamma, beta = make(B, S, C, "fp32", 1)
        layer.forward(x, gamma, beta)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y, mean, rstd = layer.forward_train(x, gamma, beta)
            held = (y, *layer.backward(dy, x, gamma, beta, mean, rstd))
        for seed in (2, 3, 4):
            for t, new in zip((x, dy, gamma, beta), make(B, S, C, "fp32", seed)):
                t.copy_(new)
            graph.replay()
            torch.cuda.synchronize()
            now = [t.clone() for t in held]
            y, mean, rstd = layer.forward_train(x, gamma, beta)
            assert all(torch.equal(a, b) for a, b in zip(now, (y, *layer.backward(dy, x, gamma, beta, mean, rstd))))
            torch.cuda.synchronize()


def test_refusals():
    import qml_gradients_amd as hq
    layer = hq.GroupNorm(12, 3, 20)
    x, w = torch.randn(2, 10, 12, device="cuda"), torch.ones(12, device="cuda")
    y, mean, rstd = layer.forward_train(x, w, w)
    for bad in (lambda: layer.forward(torch.randn(3, 10, 12, device="cuda")), lambda: layer.forward(x.bfloat16()),
                lambda: layer.forward(x.cpu()), lambda: layer.forward(x[..., :11]), lambda: layer.forward(w),
                lambda: layer.forward(x, w[:6]), lambda: layer.forward(x, w.double()), lambda: layer.forward(x, w, w[:1]),
                lambda: layer.backward(y[:1], x, w, w, mean, rstd), lambda: layer.backward(y, x, w, w, mean[:1], rstd),
                lambda: layer.backward(y, x, w, w, mean, rstd.double()), lambda: layer.forward(x, w, w, out=x[:, :, :6]),
                lambda: layer.forward(x, w, w, out=x.view(-1)[12:].view(19, 12)[:10].view(1, 10, 12))):
        with pytest.raises((hq.HqmlError, ValueError, TypeError)):
            bad()
    p, q = x.data_ptr(), y.data_ptr()
    m, r, g = mean.data_ptr(), rstd.data_ptr(), w.data_ptr()

    def forward(B=2, S=10, x=p, ldx=12, gamma=g, y=q, ldy=12, mean=m, rstd=r):
        hq.hqml_norm_forward(layer.handle, B, S, x, ldx, gamma, None, y, ldy, mean, rstd)

    dx = torch.empty_like(x)

    def backward(B=2, S=10, dy=q, lddy=12, x=p, mean=m, rstd=r, dx=dx.data_ptr(), lddx=12, dgamma=None):
        hq.hqml_norm_backward(layer.handle, B, S, dy, lddy, x, 12, g, None, mean, rstd, dx, lddx, dgamma, None)

    forward()
    backward()
    for bad in (dict(B=-1), dict(S=-1), dict(S=11), dict(x=None), dict(x=p + 2), dict(ldx=11), dict(ldx=1 << 21), dict(y=None),
                dict(mean=None), dict(rstd=None), dict(y=p + 48, S=9), dict(gamma=g + 1), dict(mean=q), dict(rstd=m),
                dict(y=p, ldy=13, S=5)):
        with pytest.raises(hq.HqmlError) as e:
            forward(**bad)
        assert e.value.status == hq.HQML_ERR_ARG, bad
    for bad in (dict(B=1 << 20, S=1 << 12), dict(dy=None), dict(lddy=3), dict(mean=None), dict(rstd=None), dict(dx=q), dict(dx=p),
                dict(lddx=11), dict(dgamma=g), dict(dgamma=m)):
        with pytest.raises(hq.HqmlError) as e:
            backward(**bad)
        assert e.value.status == hq.HQML_ERR_ARG, bad


@pytest.mark.parametrize("B,S,C,G,dtype", [(2500, 5, 4096, 64, "bf16"), (4200, 6, 2100, 2100, "bf16"), (1100, 20, 2048, 4, "fp32"),
                                           (2300, 700, 24, 3, "bf16"), (600, 2100, 16, 4, "fp32")])
def test_many_samples_that_are_split(B, S, C, G, dtype):
    """More samples than go together, on a handle made for exactly so many positions."""
    check(B, S, C, G, dtype, "silu")


@pytest.mark.parametrize("B,S,C,value", [(1, 1 << 28, 1, 1.8811031579971313), (1 << 20, 1, 2048, 1.0028703212738037)])
def test_long_sums(B, S, C, value):
    """Sums of 2^28 positions, and of 2^20 samples, of equal values: chains of additions stay below 400, each off by at
    most E of the sum.  One chain of a thread's 4,096 or 2,048 such values is off by 1,018 E or 485 E."""
    import qml_gradients_amd as hq
    x, dy = torch.ones(B, S, C, device="cuda"), torch.full((B, S, C), value, device="cuda")
    mean, rstd = torch.zeros(B, 1, device="cuda"), torch.ones(B, 1, device="cuda")
    layer = hq.GroupNorm(C, 1, B * S)
    _, dw, db = layer.backward(dy, x, None, None, mean, rstd, input=False)
    for t in (dw, db):
        off = float((t.double() / (value * B * S) - 1).abs().max())
        say(f"[gpu] long sums {B} x {S} x {C}: off {off:.2e}")
        assert off < 400 * 2.0 ** -24


@pytest.mark.parametrize("S", [5, 5000])
def test_least_eps_of_constant_groups(S):
    """rstd is up to 1 / sqrt(2^-149), whose square 32 bits do not hold: dx = rstd (dy - mean dy) all the same.  mean and rstd are
    given, exactly: a forward pass's variance has the square of its mean's rounding in it, (2.5 2^-24)^2 = 2.2e-14 for one
    rounding, beside which an eps of 2^-149 = 1.4e-45 does not show."""
    import qml_gradients_amd as hq
    layer = hq.GroupNorm(8, 2, S, eps=2.0 ** -149)
    x = torch.full((1, S, 8), 2.5, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    dy = torch.randn(1, S, 8, generator=g, device="cuda")
    rstd = torch.full((1, 2), 2.0 ** 74.5, device="cuda")
    size = float(rstd[0, 0].double())
    assert not layer.forward(x).any()
    dx, dw, db = layer.backward(dy, x, None, None, torch.full_like(rstd, 2.5), rstd)
    d = dy.double().view(1, S, 2, 4)
    want = size * (d - d.mean((1, 3), keepdim=True)).view(1, S, 8)
    # the mean's sum, 708 E of the magnitudes' mean, and 8 E of the terms
    assert float((dx.double() - want).abs().max()) <= size * 2.0 ** -24 * (708 + 8 * 6) and not dw.any()
    assert float((db.double() - dy.double().sum((0, 1))).abs().max()) <= 708 * 2.0 ** -24 * float(dy.abs().sum((0, 1)).max())


def test_more_samples_than_a_launch_takes():
    """Small samples whose sums of parameters take two launches."""
    check(66000, 1, 3000, 10, "fp32", "tanh")


def test_rounds_in_place_and_captured():
    """Samples in rounds: in place, and in a graph that is replayed with other data."""
    import qml_gradients_amd as hq
    B, S, C, G = 2100, 5, 4096, 8
    own, side = torch.cuda.Stream(), torch.cuda.Stream()
    layer = hq.GroupNorm(C, G, B * S, dtype="bf16", activation="gelu", stream=own.cuda_stream)
    x, dy, gamma, beta = make(B, S, C, "bf16", 1)
    y = layer.forward(x, gamma, beta)
    same = x.clone()
    assert layer.forward(same, gamma, beta, out=same) is same and torch.equal(same, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y, mean, rstd = layer.forward_train(x, gamma, beta)
        held = (y, *layer.backward(dy, x, gamma, beta, mean, rstd))
    for seed in (2, 3, 4):
        for t, new in zip((x, dy, gamma, beta), make(B, S, C, "bf16", seed)):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        now = [t.clone() for t in held]
        y, mean, rstd = layer.forward_train(x, gamma, beta)
        assert all(torch.equal(a, b) for a, b in zip(now, (y, *layer.backward(dy, x, gamma, beta, mean, rstd))))
        torch.cuda.synchronize()


@pytest.mark.parametrize("value", [1.8811031579971313, 1.0028703212738037, 1.5920419692993164])
def test_sums_of_many_samples_that_are_split(value):
    """As test_long_sums, of 180,000 samples: what they leave is added in chains below 400 too."""
    import qml_gradients_amd as hq
    B, S, C = 180000, 700, 24
    x, dy = torch.ones(B, S, C, device="cuda"), torch.full((B, S, C), value, device="cuda")
    mean, rstd = torch.zeros(B, 1, device="cuda"), torch.ones(B, 1, device="cuda")
    _, dw, db = hq.GroupNorm(C, 1, B * S).backward(dy, x, None, None, mean, rstd, input=False)
    for t in (dw, db):
        off = float((t.double() / (value * B * S) - 1).abs().max())
        say(f"[gpu] sums of {B} x {S} x {C}: off {off:.2e}")
        assert off < 400 * 2.0 ** -24
