"""The dense layer in 8-bit integers against its definition in 64 bits: codes have to be equal, results within bounds that
layers_reference derives."""
import math

import pytest

from gpu_util import say
from layers_reference import ACTS, TYPES, codes64, dense8, excess

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def matrix(rows, cols, dtype, seed, spread=1.0, offset=0, gap=0):
    """Rows of unlike sizes, `offset` elements into a wider array and `gap` elements apart, NaN between them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    wide = torch.full((rows * (cols + gap) + offset,), float("nan"), dtype=TYPES[dtype][0], device="cuda")
    t = wide[offset:].view(rows, cols + gap)[:, :cols]
    t.copy_(torch.randn(rows, cols, generator=g, device="cuda")
            * torch.exp(spread * torch.randn(rows, 1, generator=g, device="cuda")))
    return t


def check_codes(x):
    import qml_gradients_amd as hq
    codes, scales = hq.quantise_rows(x)
    want, size = codes64(x)
    assert torch.equal(codes, want)
    assert torch.equal(torch.nan_to_num(scales, nan=-1.0), torch.nan_to_num(size, nan=-1.0))
    whole = codes.as_strided((codes.shape[0], codes.stride(0)), (codes.stride(0), 1))
    assert not whole[:, codes.shape[1]:].any()   # rows end with zeros
    return codes, scales


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,K,offset,gap", [(1, 1, 0, 0), (3, 15, 1, 2), (5, 16, 0, 0), (257, 17, 3, 1), (7, 784, 0, 0),
                                               (9, 2047, 1, 5), (4, 2048, 0, 0), (3, 2049, 0, 7), (2, 8191, 1, 0),
                                               (2, 8193, 0, 0), (1, 70001, 1, 0), (1, 2047, 1, 0)])
def test_codes(rows, K, offset, gap, dtype):
    say(f"[gpu] codes {rows} x {K} {dtype}")
    check_codes(matrix(rows, K, dtype, rows + K, 2.0, offset, gap))


def test_codes_of_ties():
    """Quotients in the middle of two codes go to the even one, those next to it to their own side."""
    k = torch.arange(-126, 126, device="cuda", dtype=torch.float32)
    for size in (127.0, 254.0, 127.0 * 2.0 ** 100, 127.0 * 2.0 ** -90, 127.0 * 2.0 ** -100, 63.5 * 2.0 ** -100):
        mid = (k + 0.5) * (size / 127)
        up, down = torch.nextafter(mid, torch.full_like(mid, 1e38)), torch.nextafter(mid, torch.full_like(mid, -1e38))
        x = torch.stack([torch.cat([t, torch.tensor([size], device="cuda")]) for t in (mid, up, down)])
        codes, _ = check_codes(x)
        assert (codes[0, :-1] % 2 == 0).all() or size < 127 * 2.0 ** -100
    # quotients that 32 bits cannot tell from a tie: the size has 24 bits of its own
    g = torch.Generator(device="cuda").manual_seed(1)
    size = 1 + torch.rand(4000, 1, generator=g, device="cuda")
    n = torch.randint(0, 127, (4000, 30), generator=g, device="cuda").double()
    x = ((n + 0.5) * size.double() / 127).float()
    x = torch.cat([x, torch.nextafter(x, 2 * x), torch.nextafter(x, 0 * x), -x, size], 1)
    check_codes(x)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_codes_of_extreme_rows(dtype):
    dt = TYPES[dtype][0]
    top, least = torch.finfo(dt).max, torch.finfo(dt).smallest_normal
    x = torch.zeros(12, 40, device="cuda", dtype=dt)
    x[1] = least / 4                     # below the least scale
    x[2, 3] = top
    x[2, 4:20] = top / 3
    x[3, ::2], x[3, 1::2] = -top, top
    x[4] = 2.0 ** -94
    x[5, 7] = float("nan")
    x[6, 9] = float("inf")
    x[7, 0], x[7, 1] = float("-inf"), float("nan")
    x[8, 39] = -1.0
    x[9] = 1e-3
    x[10, 5] = 2.0 ** -99
    x[11] = -0.0
    codes, scales = check_codes(x)
    assert (codes[[0, 1, 5, 6, 7, 11]] == 0).all() and scales[5:8].isnan().all() and float(scales[0]) == 2.0 ** -100


CASES = [  # M, K, N: tiles of every size, splits, few rows, nothing round
    (1, 1, 1), (1, 64, 4), (1, 784, 20), (2, 15, 7), (1, 4096, 4096), (3, 4096, 1000), (16, 130, 33), (17, 2048, 64),
    (45, 1531, 803), (64, 8000, 100), (100, 97, 515), (300, 1021, 517), (1000, 784, 20), (513, 512, 769), (2048, 640, 1536),
    (1025, 2050, 2049)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("M,K,N", CASES)
def test_forward(M, K, N, dtype):
    import qml_gradients_amd as hq
    for n, act in enumerate(ACTS if M * N < 3000 else (ACTS[(M + K) % 6], ACTS[(M + N) % 6])):
        say(f"[gpu] dense8 {M} x {K} -> {N} {dtype} {act}")
        odd = n % 2
        x = matrix(M, K, dtype, 1 + n, 1.0, odd, 3 * odd)
        codes, scales = hq.quantise_rows(matrix(N, K, "fp32", 2, 0.3) / math.sqrt(K))
        bias = matrix(1, N, dtype, 3)[0] * 0.3 if n % 3 != 2 else None
        residual = matrix(M, N, dtype, 4, 1.0, odd, odd) if n % 3 != 1 else None
        alpha = math.pi if act == "sigmoid" else 1.0
        layer = hq.DenseInt8(K, N, M + 3, dtype=dtype, activation=act, alpha=alpha)
        y = layer.forward(x, codes, scales, bias, residual)
        assert y.dtype is TYPES[dtype][0] and excess(y, dense8(x, codes, scales, bias, residual, act, alpha, dtype)) <= 0
        assert torch.equal(y, layer.forward(x, codes, scales, bias, residual))
        if n == 0 and M > 1:   # fewer rows of the same handle
            y1 = layer.forward(x[:M // 2], codes, scales, bias, None if residual is None else residual[:M // 2])
            want = dense8(x[:M // 2], codes, scales, bias, None if residual is None else residual[:M // 2], act, alpha, dtype)
            assert excess(y1, want) <= 0


def test_sums_use_all_of_32_bits():
    """Rows of 127s of the largest length: 2^17 products of 127^2 are 2,114,060,288, below 2^31."""
    import qml_gradients_amd as hq
    K = 1 << 17
    x = torch.ones(3, K, device="cuda")
    x[1] = -1
    codes = torch.full((5, K), 127, dtype=torch.int8, device="cuda")
    codes[1, 0] = 126
    scales = torch.full((5,), 1.0, device="cuda")
    layer = hq.DenseInt8(K, 5, 3)
    y = layer.forward(x, codes, scales)
    assert excess(y, dense8(x, codes, scales, None, None, "none", 1.0, "fp32")) <= 0
    with pytest.raises(hq.HqmlError):
        hq.DenseInt8(K + 1, 5, 3)


def test_rows_that_are_not_finite():
    """Their outputs are NaN; the others know nothing of them."""
    import qml_gradients_amd as hq
    for M in (5, 300):
        x = matrix(M, 200, "fp32", 1)
        codes, scales = hq.quantise_rows(matrix(70, 200, "fp32", 2))
        layer = hq.DenseInt8(200, 70, M, activation="relu")
        want = layer.forward(x, codes, scales)
        bad = x.clone()
        bad[2, 3], bad[4, 0] = float("nan"), float("-inf")
        w = torch.randn(70, 200, device="cuda")
        got = layer.forward(bad, codes, scales)
        good = [i for i in range(M) if i not in (2, 4)]
        assert got[[2, 4]].isnan().all() and torch.equal(got[good], want[good])
        w[3, 5] = float("inf")
        c, s = hq.quantise_rows(w)
        y = layer.forward(x, c, s)
        assert y[:, 3].isnan().all() and not y[:, :3].isnan().any() and not y[:, 4:].isnan().any()


def test_codes_in_other_layouts():
    """Rows without padding, transposed, in the middle of an array, and padding that is not zero."""
    import qml_gradients_amd as hq
    M, K, N = 40, 100, 50
    x = matrix(M, K, "bf16", 1)
    codes, scales = hq.quantise_rows(matrix(N, K, "fp32", 2))
    layer = hq.DenseInt8(K, N, M, dtype="bf16")
    want = layer.forward(x, codes, scales)
    wide = torch.randint(-128, 128, (N + 2, 160), dtype=torch.int8, device="cuda")
    wide[1:-1, :K] = codes
    for c in (codes.contiguous(), codes.t().contiguous().t(), wide[1:-1, :K], wide.clone()[1:-1, :K]):
        assert torch.equal(layer.forward(x, c, scales), want)
    one = hq.DenseInt8(K, 1, M, dtype="bf16")
    assert torch.equal(one.forward(x, codes[:1], scales[:1]), want[:, :1])
    assert torch.equal(one.forward(x, codes.contiguous()[:1], scales[:1]), want[:, :1])
    spaced = torch.zeros(2 * N, device="cuda")
    spaced[::2] = scales
    assert torch.equal(layer.forward(x, codes, spaced[::2]), want)


def test_out_and_residual():
    import qml_gradients_amd as hq
    M, K, N = 33, 64, 48
    x, r = matrix(M, K, "fp32", 1), matrix(M, N, "fp32", 2)
    codes, scales = hq.quantise_rows(matrix(N, K, "fp32", 3))
    layer = hq.DenseInt8(K, N, M, activation="gelu")
    want = layer.forward(x, codes, scales, None, r)
    same = r.clone()
    assert layer.forward(x, codes, scales, None, same, out=same) is same and torch.equal(same, want)
    wide = torch.zeros(M + 1, N + 7, device="cuda")
    layer.forward(x, codes, scales, None, r, out=wide[:M, 3:3 + N])
    assert torch.equal(wide[:M, 3:3 + N], want)
    wide[:M, 3:3 + N] = 0
    assert not wide.any()   # rows behind the last one, and gaps, are as they were
    for out in (x[:, :N], same.view(-1)[8:8 + (M - 1) * N].view(M - 1, N)):
        with pytest.raises((hq.HqmlError, ValueError)):
            layer.forward(x[:out.shape[0]], codes, scales, None, same[:out.shape[0]], out=out)
    with pytest.raises(RuntimeError):   # a gradient through what `out` replaced
        a = torch.ones(M, N, device="cuda", requires_grad=True)
        loss = (a * same).sum()
        layer.forward(x, codes, scales, out=same)
        loss.backward()


def test_refusals():
    import qml_gradients_amd as hq
    layer = hq.DenseInt8(32, 16, 8)
    x = torch.randn(8, 32, device="cuda")
    codes, scales = hq.quantise_rows(torch.randn(16, 32, device="cuda"))
    assert layer.forward(x[:0], codes, scales).shape == (0, 16)
    for bad in (lambda: layer.forward(torch.randn(9, 32, device="cuda"), codes, scales),
                lambda: layer.forward(x.bfloat16(), codes, scales), lambda: layer.forward(x.cpu(), codes, scales),
                lambda: layer.forward(x, codes.float(), scales), lambda: layer.forward(x, codes[:8], scales),
                lambda: layer.forward(x, codes, scales.double()), lambda: layer.forward(x, codes, scales[:3]),
                lambda: layer.forward(x, codes, scales, torch.randn(15, device="cuda")),
                lambda: hq.quantise_rows(x.double()), lambda: hq.quantise_rows(x[0]), lambda: hq.quantise_rows(x[:, :0]),
                lambda: hq.quantise_rows(x.cpu())):
        with pytest.raises((hq.HqmlError, ValueError, TypeError)):
            bad()
    p = codes.data_ptr()
    y = torch.zeros(8, 16, device="cuda")

    def call(M=8, ldx=32, codes_ptr=p, ldw=32, scales_ptr=scales.data_ptr(), ldy=16):
        hq.hqml_dense8_forward(layer.handle, M, x.data_ptr(), ldx, codes_ptr, ldw, scales_ptr, None, None, 0, y.data_ptr(), ldy)

    call()
    for bad in (dict(M=-1), dict(M=9), dict(ldx=31), dict(codes_ptr=p + 1), dict(codes_ptr=None), dict(ldw=24), dict(ldw=16),
                dict(scales_ptr=None), dict(scales_ptr=scales.data_ptr() + 2), dict(ldy=15), dict(ldw=1 << 21),
                dict(scales_ptr=y.data_ptr())):
        with pytest.raises(hq.HqmlError) as e:
            call(**bad)
        assert e.value.status == hq.HQML_ERR_ARG
    dev, s = x.get_device(), 0
    for bad in (dict(rows=-1), dict(K=0), dict(dtype=2), dict(ldc=33), dict(ldc=16), dict(codes_ptr=p + 8), dict(device=-1),
                dict(codes_ptr=x.data_ptr())):
        a = dict(device=dev, dtype=0, rows=8, K=32, codes_ptr=p, ldc=32)
        a.update(bad)
        with pytest.raises(hq.HqmlError) as e:
            hq.hqml_quantise_rows(a["device"], s, a["dtype"], a["rows"], a["K"], x.data_ptr(), 32, a["codes_ptr"], a["ldc"],
                                  scales.data_ptr())
        assert e.value.status == hq.HQML_ERR_ARG


def test_another_stream_and_a_graph():
    """Calls from another stream wait and are waited for; captured ones replay as eager ones do."""
    import qml_gradients_amd as hq
    M, K, N = 130, 900, 300
    own, side = torch.cuda.Stream(), torch.cuda.Stream()
    layer = hq.DenseInt8(K, N, M, activation="silu", stream=own.cuda_stream)
    x = matrix(M, K, "fp32", 1)
    codes, scales = hq.quantise_rows(matrix(N, K, "fp32", 2))
    want = layer.forward(x, codes, scales)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        got = layer.forward(x + 0.0, codes, scales) + 0.0
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    w = matrix(N, K, "fp32", 2)
    with torch.cuda.graph(graph, stream=side):
        c, s = hq.quantise_rows(w)
        held = layer.forward(x, c, s)
    for seed in (1, 2, 3):
        x.copy_(matrix(M, K, "fp32", 10 + seed))
        w.copy_(matrix(N, K, "fp32", 20 + seed))
        graph.replay()
        torch.cuda.synchronize()
        now = held.clone()
        assert torch.equal(now, layer.forward(x, *hq.quantise_rows(w)))
        torch.cuda.synchronize()
    plain = hq.DenseInt8(K, N, M, stream=0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        twice = x * 2
        with pytest.raises(RuntimeError, match="default stream"):
            plain.forward(x, codes, scales)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(twice, x * 2)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_largest_tiles(dtype):
    import qml_gradients_amd as hq
    M, K, N = 4100, 1040, 4090
    say(f"[gpu] dense8 {M} x {K} -> {N} {dtype}")
    x = matrix(M, K, dtype, 1)
    codes, scales = hq.quantise_rows(matrix(N, K, dtype, 2, 0.3) / math.sqrt(K))
    residual = matrix(M, N, dtype, 3)
    y = hq.DenseInt8(K, N, M, dtype=dtype, activation="gelu").forward(x, codes, scales, None, residual)
    assert excess(y, dense8(x, codes, scales, None, residual, "gelu", 1.0, dtype)) <= 0


@pytest.mark.parametrize("rows", [3, 2200])
def test_offsets_past_32_bits(rows):
    """Rows of 2^20 values: of 2,200 of them the last are past 2^31 values, of x, codes, residual and y."""
    import qml_gradients_amd as hq
    K, N, ld = 40, 24, 1 << 20
    say(f"[gpu] dense8 {rows} rows {ld} apart")

    def wide(cols, dt, value):
        t = torch.zeros(rows * ld, dtype=dt, device="cuda").view(rows, ld)[:, ld - cols:]
        return t.copy_(value) if value is not None else t

    x, r = matrix(rows, K, "bf16", 1), matrix(rows, N, "bf16", 2)
    w = hq.quantise_rows(matrix(N, K, "bf16", 3))
    layer = hq.DenseInt8(K, N, rows, dtype="bf16", activation="silu")
    want = layer.forward(x, *w, None, r)
    assert excess(want, dense8(x, *w, None, r, "silu", 1.0, "bf16")) <= 0
    wide_x, wide_r = wide(K, torch.bfloat16, x), wide(N, torch.bfloat16, r)
    y = layer.forward(wide_x, *w, None, wide_r, out=wide_r)
    assert torch.equal(y, want)
    c, s = hq.quantise_rows(wide_x)
    c0, s0 = hq.quantise_rows(x)
    assert torch.equal(c, c0) and torch.equal(s, s0)
    # as many output channels, their codes as far apart
    codes = wide(K + 8, torch.int8, None)[:, :K]
    codes.copy_(c0)
    layer = hq.DenseInt8(K, rows, 3, dtype="bf16")
    x3 = matrix(3, K, "bf16", 4)
    assert torch.equal(layer.forward(x3, codes, s0), layer.forward(x3, c0, s0))


def test_two_handles_at_once():
    import qml_gradients_amd as hq
    K, N, M = 2048, 64, 17
    streams = [torch.cuda.Stream() for _ in range(2)]
    layers = [hq.DenseInt8(K, N, M, stream=s.cuda_stream) for s in streams]
    w = [hq.quantise_rows(matrix(N, K, "fp32", n)) for n in (1, 2)]
    x = [matrix(M, K, "fp32", n) for n in (3, 4)]
    want = [dense8(x[n], *w[n], None, None, "none", 1.0, "fp32") for n in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for n, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append(layers[n].forward(x[n], *w[n]))
    torch.cuda.synchronize()
    assert all(excess(y, want[i % 2]) <= 0 for i, y in enumerate(got))


def scaled_rows(rows, cols, size, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, cols, generator=g, device="cuda").double() * size).float()


@pytest.mark.parametrize("M,K,N", [(1, 784, 20), (3, 1000, 70), (45, 1531, 803), (300, 1021, 517), (2100, 640, 2060)])
@pytest.mark.parametrize("sx,sw", [(1e-20, 1e-20), (1e22, 1e22), (1e-25, 1e28), (1e30, 1e-28), (1e35, 1e-29), (1e-29, 1e35), (1e37, 1e20)])
def test_scales_of_any_size(M, K, N, sx, sw):
    """The scales' product may leave fp32's range where the result does not, or where the sum is 0.  Bounds as ever, with half a
    unit of the smallest numbers, 2^-150, for results below the normal range; infinite where the value rounded to fp32 is."""
    import qml_gradients_amd as hq
    x, w = scaled_rows(M, K, sx, 1), scaled_rows(N, K, sw, 2)
    w[0] = 0.0
    w[1] = 0.0
    w[1, 0] = 1000 * sw   # and x's first values are zero: a sum of 0 of rows that are not
    x[:, 0] = 0.0
    codes, scales = hq.quantise_rows(w)
    y = hq.DenseInt8(K, N, M).forward(x, codes, scales)
    value, bound = dense8(x, codes, scales, None, None, "none", 1.0, "fp32")
    top = torch.finfo(torch.float32).max
    above, below = value.abs() > 1.001 * top, value.abs() < 0.999 * top
    assert (y[:, :2] == 0).all() and not y.isnan().any()
    assert y[above].isinf().all() and (torch.sign(y[above]) == torch.sign(value[above])).all()
    off = (y.double() - value).abs() - bound - 2.0 ** -150
    assert float(off[below].max()) <= 0


@pytest.mark.parametrize("M,K,N", [(1, 784, 20), (45, 1531, 803), (2100, 640, 2060)])
@pytest.mark.parametrize("sx,sw", [(1e-20, 1e-20), (1e30, 1e-28), (1e22, 1e15)])
def test_scales_of_any_size_in_bf16(M, K, N, sx, sw):
    """With bias, activation and residual.  Half a unit of bf16's smallest numbers is 2^-134; results above the largest, 3.39e38, are
    infinite (1e37 times the square root of 784 is 2.8e38: some of the last sizes'), and so is, in 32 bits, a sum or a z above it
    whose residual would bring it back: where act(z) is above 0.85 of it (a bias is up to 0.13 of it here), either may be."""
    import qml_gradients_amd as hq
    x, w = scaled_rows(M, K, sx, 1).bfloat16(), scaled_rows(N, K, sw, 2)
    bias, residual = (scaled_rows(1, N, sx * sw, 3)[0]).bfloat16(), scaled_rows(M, N, sx * sw, 4).bfloat16()
    codes, scales = hq.quantise_rows(w)
    for act in ("none", "relu"):
        y = hq.DenseInt8(K, N, M, dtype="bf16", activation=act).forward(x, codes, scales, bias, residual)
        value, bound = dense8(x, codes, scales, bias, residual, act, 1.0, "bf16")
        top = torch.finfo(torch.bfloat16).max
        above, below = value.abs() > 1.01 * top, value.abs() < 0.99 * top
        assert y[above].isinf().all() and (torch.sign(y[above]) == torch.sign(value[above])).all()
        below &= (value - residual.double()).abs() < 0.85 * top
        off = (y.double() - value).abs() - bound - 2.0 ** -134
        assert float(off[below].max()) <= 0 and float(bias.abs().max()) < 0.13 * top
