"""The dense layer against its definition in 64 bits.

Bounds, elementwise and set before the first run.  With u the rounding unit of the arrays'
type (2^-24 fp32, 2^-8 bf16) and e = 2^-24 that of the sums:
  z:  a sum of K products and a bias in any order: (K + 2) e (|x| |w|^T + |bias|)
  y:  |alpha| (1.2 err(z) + 16 e (|act| + 1)) for the activation (slopes are below 1.13, its
      functions good to a few units), 2 e |y| for the residual's sum, u |y| for the rounding
  dz: |alpha dy| (0.8 (err(z) + u |z|) + 32 e (1 + |z|)) as |act''| < 0.8 and z is held in the arrays'
      type, and u |dz|; where z's sign is open, relu's slope is too: |alpha dy|
  dx, dw, db: err(dz) through the product's magnitudes, (terms + 2) e times the magnitudes,
      and u times the result.
"""
import math

import pytest

from gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

E = 2.0 ** -24
TYPES = {"fp32": (torch.float32, 2.0 ** -24), "bf16": (torch.bfloat16, 2.0 ** -8)}


def act64(z, act):
    f = {"none": lambda t: t, "relu": torch.nn.functional.relu, "gelu": torch.nn.functional.gelu,
         "silu": torch.nn.functional.silu, "tanh": torch.tanh, "sigmoid": torch.sigmoid}[act]
    z = z.detach().requires_grad_(True)
    a = f(z) * 1.0
    s, = torch.autograd.grad(a.sum(), z)
    return a.detach(), s


def make(M, K, N, dtype, seed, bias=True, residual=True):
    dt = TYPES[dtype][0]
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g) * scale).to(dt).cuda()

    return dict(x=normal(M, K), w=normal(N, K, scale=1.0 / math.sqrt(K)), bias=normal(N, scale=0.3) if bias else None,
                residual=normal(M, N) if residual else None, dy=normal(M, N))


def expect(d, dtype, act, alpha):
    """(value, bound) of y, dx, dw, db; in 64 bits on the CPU."""
    u = TYPES[dtype][1]
    x, w, dy = (d[k].detach().cpu().double() for k in ("x", "w", "dy"))
    b = torch.zeros(w.shape[0], dtype=torch.float64) if d["bias"] is None else d["bias"].cpu().double()
    z = x @ w.t() + b
    ez = (x.shape[1] + 2) * E * (x.abs() @ w.abs().t() + b.abs())
    a, s = act64(z, act)
    y = alpha * a
    ey = abs(alpha) * (1.2 * ez + 16 * E * (a.abs() + 1))
    if d["residual"] is not None:
        y = y + d["residual"].detach().cpu().double()
        ey = ey + 2 * E * y.abs() + 2 * E * (alpha * a).abs()
    ey = ey + u * (y.abs() + ey)
    dz = alpha * s * dy
    edz = (alpha * dy).abs() * (0.8 * (ez + u * z.abs()) + 32 * E * (1 + z.abs())) if act != "none" else 2 * E * dz.abs()
    if act == "relu":
        edz = torch.where(z.abs() <= ez, (alpha * dy).abs(), edz)
    if act != "none":
        edz = edz + u * (dz.abs() + edz)
    M, N = z.shape

    def product(A, eA, B, terms):
        v, m = A @ B, A.abs() @ B.abs()
        err = eA @ B.abs() + (terms + 2) * E * (m + eA @ B.abs())
        return v, err + u * (v.abs() + err)

    one = torch.ones(M, 1, dtype=torch.float64)
    db, edb = product(dz.t(), edz.t(), one, M)
    return {"y": (y, ey), "dx": product(dz, edz, w, N), "dw": product(dz.t(), edz.t(), x, M),
            "db": (db[:, 0], edb[:, 0])}


def check(name, got, want):
    value, bound = want
    got = got.detach().cpu().double()
    assert got.shape == value.shape, name
    off = (got - value).abs() - bound
    assert bool((off <= 0).all()), (name, float((got - value).abs().max()), float(off.max()))


def run(d, dtype, act, alpha, layer=None):
    import qml_gradients_amd as hq
    M, K = d["x"].shape
    N = d["w"].shape[0]
    layer = layer or hq.Dense(K, N, M, dtype=dtype, activation=act, alpha=alpha)
    y, z = layer.forward_train(d["x"], d["w"], d["bias"], d["residual"])
    assert torch.equal(y, layer.forward(d["x"], d["w"], d["bias"], d["residual"]))
    dx, dw, db = layer.backward(d["dy"], d["x"], d["w"], z)
    return {"y": y, "dx": dx, "dw": dw, "db": db}


SHAPES = [(1, 1, 1), (1, 64, 4), (2, 3, 5), (8, 4, 1), (1, 2048, 130), (16, 512, 96), (3, 1000, 33), (33, 5, 16),
          (64, 12, 64), (60, 784, 20), (1000, 784, 20), (17, 33, 65), (64, 64, 64), (65, 63, 129), (128, 256, 128),
          (130, 72, 136), (257, 129, 255), (333, 1021, 517), (512, 520, 264), (2049, 40, 24), (700, 4096, 12),
          (20, 48, 2000), (256, 2048, 512), (1030, 515, 770)]
ACTS = ["none", "relu", "gelu", "silu", "tanh", "sigmoid"]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_forward_and_gradients(case, dtype):
    M, K, N = SHAPES[case]
    act = ACTS[case % len(ACTS)]
    alpha = math.pi if act == "sigmoid" else 1.0 if case % 2 else -0.75
    say(f"[gpu] dense {M} x {K} -> {N} {dtype} {act}")
    d = make(M, K, N, dtype, 100 + case, bias=case % 3 != 1, residual=case % 4 != 2)
    got = run(d, dtype, act, alpha)
    for name, want in expect(d, dtype, act, alpha).items():
        check(name, got[name], want)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("act", ACTS)
def test_every_activation(act, dtype):
    say(f"[gpu] dense activation {act} {dtype}")
    d = make(96, 80, 72, dtype, 7)
    d["x"] = d["x"] * 3   # reach the activations' flat ends
    got = run(d, dtype, act, 1.5)
    for name, want in expect(d, dtype, act, 1.5).items():
        check(name, got[name], want)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", [(70, 96, 80), (257, 200, 136), (5, 640, 48), (1, 640, 48)])
@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 3), (2, 1), (4, 5)])
def test_strided_and_misaligned_rows(shape, offset, pad, dtype):
    """Slices of wider arrays, beginning `offset` elements in: used in place."""
    M, K, N = shape
    say(f"[gpu] dense strided {shape} offset {offset} pad {pad} {dtype}")
    d = make(M, K, N, dtype, 31)

    def inside(t):
        wide = torch.full((t.shape[0], offset + t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
        wide[:, offset:offset + t.shape[1]] = t
        return wide[:, offset:offset + t.shape[1]]

    want = expect(d, dtype, "gelu", 1.0)
    for k in ("x", "w", "residual", "dy"):
        d[k] = inside(d[k])
    got = run(d, dtype, "gelu", 1.0)
    for name in want:
        check(name, got[name], want[name])
    # output rows inside a wider array, whose other elements stay
    import qml_gradients_amd as hq
    out = inside(torch.zeros(M, N, dtype=d["x"].dtype, device="cuda"))
    layer = hq.Dense(K, N, M, dtype=dtype, activation="gelu")
    assert layer.forward(d["x"], d["w"], d["bias"], d["residual"], out=out) is out
    check("y", out, want["y"])
    whole = out._base if out._base is not None else out
    assert int(torch.isnan(whole).sum()) == M * (offset + pad)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", [(700, 333, 501), (333, 1021, 517), (1001, 520, 263), (515, 1029, 1024), (61, 2500, 3001)])
@pytest.mark.parametrize("pad", [0, 16])
def test_odd_lengths_of_large_products(shape, pad, dtype):
    """Odd lengths in every direction at sizes that go to the large tiles; with `pad`, rows that
    begin 16-byte aligned all the same, NaN between them."""
    M, K, N = shape
    say(f"[gpu] dense odd {shape} pad {pad} {dtype}")
    d = make(M, K, N, dtype, 37)
    want = expect(d, dtype, "silu", 1.0)
    if pad:
        for k in ("x", "w", "residual", "dy"):
            t = d[k]
            wide = torch.full((t.shape[0], (t.shape[1] + pad) // 8 * 8), float("nan"), dtype=t.dtype, device="cuda")
            wide[:, :t.shape[1]] = t
            d[k] = wide[:, :t.shape[1]]
    got = run(d, dtype, "silu", 1.0)
    for name in want:
        check(name, got[name], want[name])
    plain = expect(d, dtype, "none", 1.0)   # no activation: dy itself is an operand
    got = run(d, dtype, "none", 1.0)
    for name in plain:
        check(name, got[name], plain[name])


def test_transposed_weights_are_copied():
    d = make(40, 56, 24, "fp32", 3)
    d["w"] = d["w"].t().contiguous().t()
    d["x"] = d["x"].t().contiguous().t()
    want = expect(d, "fp32", "tanh", 1.0)
    got = run(d, "fp32", "tanh", 1.0)
    for name in want:
        check(name, got[name], want[name])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_residual_in_place_and_smaller_batches(dtype):
    import qml_gradients_amd as hq
    d = make(200, 96, 48, dtype, 11)
    layer = hq.Dense(96, 48, 200, dtype=dtype, activation="silu")
    for M in (200, 1, 37, 128):
        part = {k: v if k in ("w", "bias") else v[:M] for k, v in d.items()}
        got = run(part, dtype, "silu", 1.0, layer)
        for name, want in expect(part, dtype, "silu", 1.0).items():
            check(name, got[name], want)
    r = d["residual"].clone()
    y = layer.forward(d["x"], d["w"], d["bias"], r, out=r)
    assert y is r
    check("y", r, expect(d, dtype, "silu", 1.0)["y"])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", [(40, 24, 36), (700, 520, 1024), (513, 333, 1025)])
def test_each_gradient_alone(shape, dtype):
    """Gradients asked for one by one are the ones of the joint call, to the bounds; none is a no-op."""
    import qml_gradients_amd as hq
    M, K, N = shape
    for act in ("none", "gelu"):
        d = make(M, K, N, dtype, 23)
        want = expect(d, dtype, act, 1.25)
        layer = hq.Dense(K, N, M, dtype=dtype, activation=act, alpha=1.25)
        _, z = layer.forward_train(d["x"], d["w"], d["bias"], d["residual"])
        for k, name in enumerate(("dx", "dw", "db")):
            ask = [i == k for i in range(3)]
            got = layer.backward(d["dy"], d["x"], d["w"], z, *ask)
            assert [g is not None for g in got] == ask
            check(name, got[k], want[name])
        assert layer.backward(d["dy"], d["x"], d["w"], z, False, False, False) == (None, None, None)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 4096, 300), (24, 6766, 583), (7, 9000, 33), (64, 2111, 64), (4000, 37, 9), (9000, 24, 300)])
def test_long_and_narrow(shape, dtype):
    """Few rows or columns against a long sum: the products that are split over k."""
    M, K, N = shape
    say(f"[gpu] dense long and narrow {shape} {dtype}")
    d = make(M, K, N, dtype, 51)
    got = run(d, dtype, "tanh", 1.0)
    for name, want in expect(d, dtype, "tanh", 1.0).items():
        check(name, got[name], want)


# More than 512 tiles of 128 x 128 in every product: two workgroups share a compute unit, and in fp32 one LDS buffer
# a workgroup is read and refilled in turn.
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_products_of_many_tiles(dtype):
    import qml_gradients_amd as hq
    M, K, N = 2990, 2950, 3001
    say(f"[gpu] dense {M} x {K} -> {N} {dtype}")
    d = make(M, K, N, dtype, 77)
    layer = hq.Dense(K, N, M, dtype=dtype, activation="silu")
    got = run(d, dtype, "silu", 1.0, layer)
    for _ in range(5):
        again = run(d, dtype, "silu", 1.0, layer)
        assert all(torch.equal(got[k], again[k]) for k in got)
    for name, want in expect(d, dtype, "silu", 1.0).items():
        check(name, got[name], want)


# Forward products split over k whose tiles outnumber 64 x 64 ones, with the copies of odd rows beside their counters.
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", [(128, 256, 249), (100, 1001, 130), (64, 2047, 64), (16, 5001, 60), (240, 301, 250)])
def test_small_products_split_over_k(shape, dtype):
    import qml_gradients_amd as hq
    M, K, N = shape
    say(f"[gpu] dense {M} x {K} -> {N} {dtype}")
    d = make(M, K, N, dtype, 78)
    layer = hq.Dense(K, N, M, dtype=dtype, activation="tanh")
    got = run(d, dtype, "tanh", 1.0, layer)
    for _ in range(3):
        again = run(d, dtype, "tanh", 1.0, layer)
        assert all(torch.equal(got[k], again[k]) for k in got)
    for name, want in expect(d, dtype, "tanh", 1.0).items():
        check(name, got[name], want)


# At most 32 rows or columns against thousands, in each of the three products.
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", [(4877, 1401, 30), (31, 2500, 3001), (9000, 29, 3001), (2500, 3000, 32), (32, 3000, 2500)])
def test_narrow_products(shape, dtype):
    M, K, N = shape
    say(f"[gpu] dense {M} x {K} -> {N} {dtype}")
    d = make(M, K, N, dtype, 79)
    got = run(d, dtype, "gelu", -0.75)
    for name, want in expect(d, dtype, "gelu", -0.75).items():
        check(name, got[name], want)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_empty_batch(act, dtype):
    import qml_gradients_amd as hq
    dt = TYPES[dtype][0]
    layer = hq.Dense(24, 40, 8, dtype=dtype, activation=act)
    x, w, dy = (torch.ones(*s, dtype=dt, device="cuda") for s in ((0, 24), (40, 24), (0, 40)))
    y, z = layer.forward_train(x, w)
    assert y.shape == (0, 40)
    dx, dw, db = layer.backward(dy, x, w, z)
    assert dx.shape == (0, 24) and not dw.any() and not db.any() and dw.shape == (40, 24) and db.shape == (40,)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 256, 64), (96, 160, 64), (300, 264, 272)])
def test_infinities_and_nan_stay_in_their_rows(shape, dtype):
    """Every output is finite, infinite or NaN where the sum of its products is."""
    import qml_gradients_amd as hq
    M, K, N = shape
    d = make(M, K, N, dtype, 17, bias=False, residual=False)
    d["w"] = torch.where(d["w"] == 0, torch.ones_like(d["w"]), d["w"])
    d["w"][3, :] = 1.0
    d["x"][0, 5] = float("inf")
    if M > 50:
        d["x"][20, 7] = float("-inf")
        d["x"][30, 1], d["x"][30, 2] = float("inf"), float("-inf")
        d["x"][40, 0] = float("nan")
    y = hq.Dense(K, N, M, dtype=dtype).forward(d["x"], d["w"]).cpu().double()
    want = d["x"].cpu().double() @ d["w"].cpu().double().t()
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert torch.equal(torch.isposinf(y), torch.isposinf(want)) and torch.equal(torch.isneginf(y), torch.isneginf(want))


def test_large_and_small_magnitudes_fp32():
    """Products near both ends of the range keep 32-bit precision."""
    import qml_gradients_amd as hq
    M, K, N = 130, 200, 140
    g = torch.Generator().manual_seed(9)
    for sx, sw in ((1e18, 1e18), (1e-15, 1e-12), (1e30, 1e-30), (3e38 / 8, 1e-3)):
        x = (torch.rand(M, K, generator=g) + 0.5) * sx
        w = (torch.rand(N, K, generator=g) - 0.5) * sw
        y = hq.Dense(K, N, M).forward(x.cuda(), w.cuda()).cpu().double()
        mag = x.double() @ w.double().abs().t()
        assert bool(((y - x.double() @ w.double().t()).abs() <= (K + 2) * E * mag).all()), (sx, sw)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_results_repeat_bitwise(dtype):
    d = make(517, 2050, 130, dtype, 21)
    a, b = run(d, dtype, "gelu", 1.0), run(d, dtype, "gelu", 1.0)
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_another_stream_than_the_handles():
    """Inputs written on a side stream just before the call, outputs read there just after."""
    import qml_gradients_amd as hq
    d = make(512, 512, 512, "fp32", 5)
    want = expect(d, "fp32", "gelu", 1.0)
    layer = hq.Dense(512, 512, 512, activation="gelu")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        big = torch.ones(4096, 4096, device="cuda")
        for _ in range(8):
            big = big @ big * 1e-4     # keeps the side stream busy
        late = {k: v * (big[0, 0] * 0 + 1) for k, v in d.items()}
        got = {k: v * 1.0 for k, v in run(late, "fp32", "gelu", 1.0, layer).items()}
    side.synchronize()
    for name in want:
        check(name, got[name], want[name])


def test_offsets_past_32_bits():
    """Rows so far apart that element offsets pass 2^32."""
    import qml_gradients_amd as hq
    M, K, N = 4200, 40, 24
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("needs 24 GiB of free device memory")
    d = make(M, K, N, "bf16", 13)
    wide = torch.empty(M, 1 << 20, dtype=torch.bfloat16, device="cuda")
    assert (M - 1) << 20 > 1 << 32
    wide[:, :K] = d["x"]
    want = expect(d, "bf16", "gelu", 1.0)
    d["x"] = wide[:, :K]
    got = run(d, "bf16", "gelu", 1.0)
    for name in want:
        check(name, got[name], want[name])


@pytest.mark.parametrize("act", ["none", "gelu", "silu", "tanh", "sigmoid"])
def test_gradient_against_differences(act):
    """<gradient, v> against (L(t + h v) - L(t - h v)) / 2h of the kernel's own forward, with
    L = sum(dy y).  Third derivatives of the activations are below 2, so the difference is off by
    sum |dy| 2 h^2 |dz|^3 / 6 for the change dz = dz/dt v, and by the forward's rounding / h."""
    import qml_gradients_amd as hq
    M, K, N, h = 40, 24, 36, 2.0 ** -5
    d = make(M, K, N, "fp32", 41)
    got = run(d, "fp32", act, 1.0)
    layer = hq.Dense(K, N, M, activation=act)
    _, ey = expect(d, "fp32", act, 1.0)["y"]
    dy = d["dy"].cpu().double()
    g = torch.Generator().manual_seed(2)
    for name, grad in (("x", "dx"), ("w", "dw"), ("bias", "db")):
        v = torch.randn(d[name].shape, generator=g).sign() * 0.25   # steps and sums exact enough in fp32
        L = []
        for sign in (1, -1):
            moved = dict(d)
            moved[name] = d[name] + sign * h * v.cuda()
            y = layer.forward(moved["x"], moved["w"], moved["bias"], moved["residual"])
            L.append(float((dy * y.cpu().double()).sum()))
        change = {"x": lambda: v.double() @ d["w"].cpu().double().t(), "w": lambda: d["x"].cpu().double() @ v.double().t(),
                  "bias": lambda: v.double().expand(M, N)}[name]()
        moves = change.abs().max() * h
        assert moves < 1
        # the moved arguments round too: 2^-24 of their size, through the same linear map
        args = {"x": d["x"].abs().cpu().double() @ d["w"].abs().cpu().double().t(),
                "w": d["x"].abs().cpu().double() @ d["w"].abs().cpu().double().t(),
                "bias": d["bias"].abs().cpu().double().expand(M, N)}[name]
        bound = float((dy.abs() * (2 * h * h * change.abs() ** 3 / 6 + (2 * ey + 2 * E * (args + 1)) / h)).sum())
        inner = float((got[grad].cpu().double() * v.double()).sum())
        assert abs((L[0] - L[1]) / (2 * h) - inner) <= bound + 1e-5 * float((got[grad].cpu().double().abs() * 0.25).sum()), name


def test_graph_replays_match_eager():
    import qml_gradients_amd as hq
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        d = make(70, 300, 50, "bf16", 19)
        layer = hq.Dense(300, 50, 70, dtype="bf16", activation="gelu")
        run(d, "bf16", "gelu", 1.0, layer)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            y, z = layer.forward_train(d["x"], d["w"], d["bias"], d["residual"])
            grads = layer.backward(d["dy"], d["x"], d["w"], z)
        for seed in (1, 2, 3):
            fresh = make(70, 300, 50, "bf16", seed)
            for k in d:
                d[k].copy_(fresh[k])
            graph.replay()
            s.synchronize()
            held = [t.clone() for t in (y, *grads)]
            want = run(fresh, "bf16", "gelu", 1.0, layer)
            for a, b in zip(held, (want["y"], want["dx"], want["dw"], want["db"])):
                assert torch.equal(a, b)
            torch.cuda.synchronize()


def test_refusals():
    import qml_gradients_amd as hq
    d = make(8, 16, 12, "fp32", 1)
    layer = hq.Dense(16, 12, 8, activation="tanh")
    with pytest.raises(ValueError):
        layer.forward(d["x"], d["w"].t())
    with pytest.raises(TypeError):
        layer.forward(d["x"].bfloat16(), d["w"])
    with pytest.raises(TypeError):
        layer.forward(d["x"].cpu(), d["w"])
    with pytest.raises(ValueError):
        layer.forward(d["x"], d["w"], d["bias"][:-1])
    with pytest.raises(ValueError):
        layer.backward(d["dy"], d["x"], d["w"], None)
    with pytest.raises(hq.HqmlError) as e:
        layer.forward(torch.zeros(9, 16, device="cuda"), d["w"])
    assert e.value.status == hq.HQML_ERR_ARG
    p = d["x"].data_ptr()
    for args in ((8, None, 16, p, 16, None, None, 0, p, 12, None), (8, p, 15, p, 16, None, None, 0, p, 12, None),
                 (8, p, (1 << 20) + 1, p, 16, None, None, 0, p, 12, None), (-1, p, 16, p, 16, None, None, 0, p, 12, None),
                 (8, p + 2, 16, p, 16, None, None, 0, p, 12, None)):
        with pytest.raises(hq.HqmlError) as e:
            hq.hqml_dense_forward(layer.handle, *args)
        assert e.value.status == hq.HQML_ERR_ARG
    host = torch.zeros(8, 16)
    with pytest.raises(hq.HqmlError) as e:
        hq.hqml_dense_forward(layer.handle, 8, host.data_ptr(), 16, p, 16, None, None, 0, p, 12, None)
    assert e.value.status == hq.HQML_ERR_ARG
    with pytest.raises(hq.HqmlError) as e:
        hq.Dense(1 << 20, 1 << 20, 1 << 24, activation="gelu")   # workspace beyond the device
    assert e.value.status == hq.HQML_ERR_OOM


def test_out_must_not_be_an_operand():
    import qml_gradients_amd as hq
    layer = hq.Dense(16, 16, 16)
    x, w = torch.randn(16, 16, device="cuda"), torch.randn(16, 16, device="cuda")
    with pytest.raises(ValueError):
        layer.forward(x, w, out=x)
    with pytest.raises(ValueError):
        layer.forward(x, w, out=w)
    y = layer.forward(x, w)
    both = torch.cat((x, torch.zeros_like(x)), 1)   # neighbouring columns do not overlap
    assert torch.equal(layer.forward(both[:, :16], w, out=both[:, 16:]), y)
    assert torch.equal(both[:, :16], x)


def test_layer_gradients_reach_every_argument():
    from qml_gradients_amd.torch_layer import DenseLayer
    torch.manual_seed(4)
    layer = DenseLayer(20, 28, 64, activation="silu", alpha=0.5)
    x = torch.randn(4, 9, 20, device="cuda", requires_grad=True)
    r = torch.randn(4, 9, 28, device="cuda", requires_grad=True)
    y = layer(x, residual=r)
    assert y.shape == (4, 9, 28)
    dy = torch.randn_like(y)
    y.backward(dy)
    d = dict(x=x.detach().reshape(36, 20), w=layer.weight.detach(), bias=layer.bias.detach(),
             residual=r.detach().reshape(36, 28), dy=dy.reshape(36, 28))
    want = expect(d, "fp32", "silu", 0.5)
    for name, got in (("y", y.reshape(36, 28)), ("dx", x.grad.reshape(36, 20)), ("dw", layer.weight.grad),
                      ("db", layer.bias.grad)):
        check(name, got, want[name])
    assert torch.equal(r.grad, dy)
    with torch.no_grad():
        assert torch.equal(layer(x, residual=r), y.detach())
