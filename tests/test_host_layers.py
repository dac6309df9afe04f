"""Host side of the 8-bit dense layer, group norm and Muon: configurations refused without a GPU, workspace sizes, constants
of the binding as the header has them, the references' own pins."""
import ctypes
import math
import os

import pytest

import qml_gradients_amd as hq

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _lib():
    if not os.path.exists(hq.LIB_PATH):
        from qml_gradients_amd import build
        build.build()
    return hq.load()


@pytest.mark.parametrize("bad", [dict(in_features=0), dict(in_features=(1 << 17) + 1), dict(out_features=0),
                                 dict(out_features=(1 << 20) + 1), dict(max_batch=0), dict(max_batch=(1 << 24) + 1),
                                 dict(dtype=2), dict(dtype=-1), dict(activation=6), dict(alpha=math.inf), dict(alpha=math.nan),
                                 dict(device=-1)])
def test_dense8_configurations_refused(bad):
    _lib()
    good = dict(in_features=8, out_features=4, max_batch=2)
    assert hq.hqml_dense8_workspace_bytes(hq.make_dense_config(**good)) > 0
    cfg = hq.make_dense_config(**{**good, **bad})
    assert hq.hqml_dense8_workspace_bytes(cfg) == 0
    with pytest.raises(hq.HqmlError) as e:
        hq.hqml_dense8_create(cfg)
    assert e.value.status == hq.HQML_ERR_ARG


@pytest.mark.parametrize("bad", [dict(channels=0), dict(channels=4097, groups=1), dict(groups=0), dict(groups=3), dict(groups=-2),
                                 dict(max_rows=0), dict(max_rows=(1 << 30) + 1), dict(dtype=2), dict(activation=-1),
                                 dict(eps=0.0), dict(eps=-1.0), dict(eps=math.inf), dict(eps=math.nan), dict(device=-1)])
def test_norm_configurations_refused(bad):
    _lib()
    good = dict(channels=8, groups=2, max_rows=5)
    assert hq.hqml_norm_workspace_bytes(hq.make_norm_config(**good)) > 0
    cfg = hq.make_norm_config(**{**good, **bad})
    assert hq.hqml_norm_workspace_bytes(cfg) == 0
    with pytest.raises(hq.HqmlError) as e:
        hq.hqml_norm_create(cfg)
    assert e.value.status == hq.HQML_ERR_ARG


def _muon(**change):
    a = dict(param_dtype=0, grad_dtype=0, nesterov=1, steps=5, lr=0.1, momentum=0.9, weight_decay=0.0, eps=1e-7, a=3.4445,
             b=-4.775, c=2.0315, device=0, stream=None)
    a.update(change)
    return hq.hqml_muon_config(*a.values())


@pytest.mark.parametrize("bad", [dict(param_dtype=2), dict(grad_dtype=2), dict(steps=0), dict(steps=101), dict(lr=-1.0),
                                 dict(lr=math.nan), dict(lr=math.inf), dict(momentum=1.0), dict(momentum=-0.1),
                                 dict(momentum=math.nan), dict(weight_decay=-1.0), dict(eps=0.0), dict(eps=1e-60),
                                 dict(eps=math.inf), dict(a=17.0), dict(b=math.nan), dict(c=-math.inf), dict(device=-1)])
def test_muon_configurations_refused(bad):
    _lib()
    t = (hq.hqml_muon_tensor * 1)(hq.hqml_muon_tensor(None, None, None, 100, 100, 1.0))
    assert hq.hqml_muon_workspace_bytes(_muon(), 1, t) > 0
    assert hq.hqml_muon_workspace_bytes(_muon(**bad), 1, t) == 0
    with pytest.raises(hq.HqmlError) as e:
        hq.hqml_muon_step(_muon(**bad), 1, t, None, 0)
    assert e.value.status == hq.HQML_ERR_ARG


def test_muon_overlaps_refused():
    """By addresses alone: nothing is read, and arrays beside each other pass on to the next check."""
    import qml_gradients_amd as hq
    base, size = 1 << 30, 100 * 100 * 4
    P, G, M = base, base + size, base + 2 * size   # beside each other
    at = lambda n: base + n * size

    def step(*matrices, workspace=1 << 40):
        t = (hq.hqml_muon_tensor * len(matrices))(*[hq.hqml_muon_tensor(*m, 100, 100, 1.0) for m in matrices])
        with pytest.raises(hq.HqmlError) as e:
            hq.hqml_muon_step(_muon(), len(matrices), t, workspace, hq.hqml_muon_workspace_bytes(_muon(), len(matrices), t))
        return str(e.value)

    for bad in ([(P, P, M)], [(P, G, G)], [(P, G, P)], [(P, G, M), (at(3), at(4), M)], [(P, G, M), (P, at(4), at(5))],
                [(P, G, M), (at(3), P, at(4))], [(P, G, M - 4)], [(P, G, M), (at(3), at(4), at(5)), (at(5) + size - 4, at(7), at(8))]):
        assert "overlap" in step(*bad)
    for workspace in (P, G, M, M + size - 256):
        assert "overlap" in step((P, G, M), workspace=workspace)
    for good in ([(P, G, M)], [(P, G, M), (at(3), at(4), at(5))], [(P, G, M), (at(3), G, at(4))]):
        assert "overlap" not in step(*good)   # there is no such memory: refused for that


def test_muon_workspace():
    """Two X and two of the smaller side's square for each matrix, rounds of up to 1 GiB, and 64 MiB and 16 KiB of partial sums
    and counters; nothing for small matrices."""
    _lib()
    joins = (64 << 20) + (16 << 10)
    array = lambda *sizes: (hq.hqml_muon_tensor * len(sizes))(*[hq.hqml_muon_tensor(None, None, None, r, c, 1.0) for r, c in sizes])
    one = hq.hqml_muon_workspace_bytes(_muon(), 1, array((1024, 4096))) - joins
    assert one >= 2 * 4 * (1024 * 4096 + 1024 * 1024)
    assert hq.hqml_muon_workspace_bytes(_muon(param_dtype=1), 1, array((1024, 4096))) - joins <= one // 2 + 8192
    assert hq.hqml_muon_workspace_bytes(_muon(), 3, array((1024, 4096), (4096, 1024), (0, 7))) - joins <= 2 * one + 4096
    many = hq.hqml_muon_workspace_bytes(_muon(), 200, array(*[(1024, 4096)] * 200)) - joins
    assert one < many <= (1 << 30)
    assert hq.hqml_muon_workspace_bytes(_muon(), 1, array((0, 7))) == 0
    assert hq.hqml_muon_workspace_bytes(_muon(), 2, array((32, 64), (4, 64))) == 0
    assert hq.hqml_muon_workspace_bytes(_muon(), 0, None) == 0
    hq.hqml_muon_step(_muon(), 1, array((0, 7)), None, 0)   # no elements: nothing to do
    for bad in ((-1, 4), (4, -1), ((1 << 16) + 1, 4), (4, (1 << 16) + 1)):
        assert hq.hqml_muon_workspace_bytes(_muon(), 1, array(bad)) == 0


def test_null_arguments_refused():
    lib = _lib()
    assert lib.hqml_dense8_workspace_bytes(None) == 0 and lib.hqml_norm_workspace_bytes(None) == 0
    assert lib.hqml_muon_workspace_bytes(None, 0, None) == 0
    for create in (lib.hqml_dense8_create, lib.hqml_norm_create):
        assert create(None, None) == hq.HQML_ERR_ARG
        assert create(None, ctypes.byref(ctypes.c_void_p())) == hq.HQML_ERR_ARG
    assert lib.hqml_dense8_destroy(None) == hq.HQML_OK and lib.hqml_norm_destroy(None) == hq.HQML_OK
    assert lib.hqml_dense8_forward(None, 1, None, 1, None, 16, None, None, None, 0, None, 1) == hq.HQML_ERR_ARG
    assert lib.hqml_norm_forward(None, 1, 1, None, 1, None, None, None, 1, None, None) == hq.HQML_ERR_ARG
    assert lib.hqml_norm_backward(None, 1, 1, None, 1, None, 1, None, None, None, None, None, 1, None, None) == hq.HQML_ERR_ARG
    assert lib.hqml_muon_step(None, 0, None, None, 0) == hq.HQML_ERR_ARG
    assert lib.hqml_muon_step(ctypes.byref(_muon()), 2, None, None, 0) == hq.HQML_ERR_ARG
    assert lib.hqml_muon_step(ctypes.byref(_muon()), -1, None, None, 0) == hq.HQML_ERR_ARG


@pytest.mark.parametrize("change", [dict(device=-1), dict(dtype=2), dict(rows=-1), dict(K=0), dict(K=(1 << 20) + 1), dict(ldc=17),
                                    dict(ldc=16), dict(codes=8)])
def test_quantise_rows_refused(change):
    lib = _lib()
    a = dict(device=0, stream=None, dtype=0, rows=4, K=20, x=None, ldx=20, codes=16, ldc=32, scales=None)
    a.update(change)
    assert lib.hqml_quantise_rows(*a.values()) == hq.HQML_ERR_ARG


def test_constants_match_header():
    header = open(os.path.join(ROOT, "include", "hqml.h")).read()
    for name, text in (("DENSE8_MAX_IN", "(1 << 17)"), ("NORM_MAX_CHANNELS", "4096"), ("NORM_MAX_ROWS", "(1 << 30)"),
                       ("MUON_MAX_SIDE", "(1 << 16)"), ("MUON_MAX_STEPS", "100")):
        assert f"#define HQML_{name} {text}" in header and getattr(hq, f"HQML_{name}") == eval(text)


# ---- the references ----

def test_codes_by_hand():
    from layers_reference import codes64
    x = torch.tensor([[127.0, 0.5, 1.5, -2.5, 63.49, 0.0], [0.0] * 6, [1e-38] * 6, [math.inf, 1, 2, 3, 4, 5]])
    codes, scales = codes64(x)
    assert codes[0].tolist() == [127, 0, 2, -2, 63, 0] and float(scales[0]) == 1.0
    assert not codes[1].any() and not codes[2].any() and float(scales[2]) == 2.0 ** -100
    assert not codes[3].any() and math.isnan(float(scales[3]))


def test_norm_by_autograd():
    """The reference's gradients are those of its own forward pass."""
    from layers_reference import norm
    g = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(3, 5, 12, generator=g, dtype=torch.float64) for _ in range(2))
    w, b = (torch.randn(12, generator=g, dtype=torch.float64) for _ in range(2))
    for act in ("none", "gelu", "tanh"):
        got = norm(x, w, b, dy, 3, act, 1e-5, "fp32")
        leaves = [t.clone().requires_grad_() for t in (x, w, b)]
        X = leaves[0].view(3, 5, 3, 4)
        hat = (X - X.mean((1, 3), keepdim=True)) / torch.sqrt(X.var((1, 3), correction=0, keepdim=True) + 1e-5)
        z = hat.view(3, 5, 12) * leaves[1] + leaves[2]
        y = {"none": lambda t: t, "gelu": torch.nn.functional.gelu, "tanh": torch.tanh}[act](z)
        y.backward(dy)
        assert torch.allclose(got["y"][0], y)
        for name, leaf in zip(("dx", "dgamma", "dbeta"), leaves):
            assert torch.allclose(got[name][0], leaf.grad)


def planted(name, x, w, b, dy, G):
    """A norm with a mistake, in 64 bits: y or dx."""
    X = x.view(x.shape[0], -1, G, x.shape[-1] // G)
    mean = X.mean((1, 3), keepdim=True)
    n = X.shape[1] * X.shape[3]
    var = ((X - mean) ** 2).sum((1, 3), keepdim=True) / (n - 1 if name == "sample variance" else n)
    r = 1 / (torch.sqrt(var) + 1e-5 if name == "eps outside" else torch.sqrt(var + 1e-5))
    hat = (X - mean) * r
    gw = w.view(G, -1)
    y = torch.tanh(hat * gw + b.view(G, -1))
    dz = dy.view_as(X) * (1 - y * y)
    q = dz * (1 if name == "gamma left out" else gw)
    second = 0 if name == "second mean left out" else hat * (q * hat).mean((1, 3), keepdim=True)
    return y.reshape(x.shape), (r * (q - q.mean((1, 3), keepdim=True) - second)).reshape(x.shape)


@pytest.mark.parametrize("name", ["none", "sample variance", "eps outside", "gamma left out", "second mean left out"])
def test_norm_bounds_notice_mistakes(name):
    from layers_reference import excess, norm
    g = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(2, 400, 12, generator=g, dtype=torch.float64) for _ in range(2))
    w, b = (torch.randn(12, generator=g, dtype=torch.float64) for _ in range(2))
    x *= 0.01   # eps counts
    want = norm(x, w, b, dy, 3, "tanh", 1e-5, "fp32")
    y, dx = planted(name, x, w, b, dy, 3)
    wrong = excess(y, want["y"]) > 0 or excess(dx, want["dx"]) > 0
    assert wrong == (name != "none")


@pytest.mark.parametrize("planted_noise,wrong", [(0.0, False), (2.0 ** -21, False), (2.0 ** -16, True)])
def test_orthogonal_bounds_notice_fewer_bits(planted_noise, wrong):
    """Operands of fp32 parameters held in 16 bits would be noticed."""
    from layers_reference import orthogonal, orthogonal_bound
    g = torch.Generator().manual_seed(1)
    u = torch.randn(40, 60, generator=g, dtype=torch.float64)
    x, norm_bound, most = orthogonal_bound(u, "fp32")
    noisy = orthogonal(u, noise=lambda t: t * (1 + planted_noise * (torch.rand(t.shape, generator=g, dtype=torch.float64) * 2 - 1)))
    d = noisy - x
    assert (float(torch.linalg.vector_norm(d)) > norm_bound) == wrong
    assert (float(d.abs().max()) > most) == wrong


def test_orthogonal_is_near_orthogonal():
    from layers_reference import orthogonal
    g = torch.Generator().manual_seed(1)
    for shape in ((20, 50), (50, 20)):
        s = torch.linalg.svdvals(orthogonal(torch.randn(*shape, generator=g, dtype=torch.float64)))
        assert 0.6 < float(s.min()) and float(s.max()) < 1.3


# ---- Muon's own work: the entry point is replaced ----

@pytest.fixture
def calls(monkeypatch):
    from qml_gradients_amd import optim
    seen = []

    def record(cfg, n, tensors, work, size):
        array = (hq.hqml_muon_tensor * n).from_buffer_copy(tensors)
        seen.append((cfg, [(t.param, t.grad, t.momentum, t.rows, t.cols, t.scale) for t in array], size))

    monkeypatch.setattr(optim, "hqml_muon_step", record)
    monkeypatch.setattr(optim, "_current_stream", lambda device: 0)
    monkeypatch.setattr(optim.Muon, "_accept", staticmethod(lambda p: optim.Muon._fits(p)))   # takes host parameters
    return seen


def _parameter(rows, cols, dtype=torch.float32):
    p = torch.nn.Parameter(torch.ones(rows, cols, dtype=dtype))
    p.grad = torch.ones(rows, cols, dtype=dtype)
    return p


def test_muon_says_what_it_holds(calls, monkeypatch):
    from qml_gradients_amd import optim
    monkeypatch.setattr(optim, "hqml_muon_workspace_bytes", lambda cfg, n, t: 4096)
    a, b = _parameter(6, 4), _parameter(3, 5, torch.bfloat16)
    opt = optim.Muon([{"params": [a], "lr": 0.5}, {"params": [b], "adjust": "rms", "nesterov": False}], weight_decay=0.1)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    opt.step()
    (c1, t1, _), (c2, t2, _) = calls
    assert (c1.lr, c1.nesterov, c1.param_dtype, c1.weight_decay) == (0.5, 1, hq.HQML_DTYPE_FP32, 0.1)
    assert t1 == [(a.data_ptr(), a.grad.data_ptr(), opt.state[a]["momentum"].data_ptr(), 6, 4, math.sqrt(1.5))]
    assert (c2.lr, c2.nesterov, c2.param_dtype) == (0.02, 0, hq.HQML_DTYPE_BF16)
    assert t2[0][3:] == (3, 5, 0.2 * math.sqrt(5)) and opt.state[b]["momentum"].dtype is torch.float32


@pytest.mark.parametrize("bad", [dict(lr=-1.0), dict(momentum=1.0), dict(weight_decay=-1.0), dict(eps=0.0), dict(steps=0),
                                 dict(steps=101), dict(coefficients=(1.0, 2.0)), dict(adjust="no")])
def test_muon_arguments_refused(bad, calls):
    from qml_gradients_amd import optim
    with pytest.raises(ValueError):
        optim.Muon([_parameter(4, 4)], **bad)


def test_muon_states_that_do_not_fit_are_refused(calls):
    from qml_gradients_amd import optim
    p = _parameter(4, 6)
    opt = optim.Muon([p])
    for bad in (torch.zeros(6, 4), torch.zeros(4, 6, dtype=torch.float64), torch.zeros(6, 4).t()):
        opt.state[p]["momentum"] = bad
        with pytest.raises(ValueError):
            opt.step()
    saved = opt.state_dict()
    saved["state"] = {0: {"momentum": torch.zeros(6, 4)}}
    with pytest.raises(ValueError):
        optim.Muon([p]).load_state_dict(saved)
    p.grad = None
    opt.state[p]["momentum"] = torch.zeros(4, 6)
    opt.step()
    assert not calls


def test_muon_workspace_of_precise_products():
    """Two fp16 values for each operand of bf16 parameters take the workspace of fp32 parameters."""
    _lib()
    t = (hq.hqml_muon_tensor * 1)(hq.hqml_muon_tensor(None, None, None, 1024, 4096, 1.0))
    joins = (64 << 20) + (16 << 10)
    wide = hq.hqml_muon_workspace_bytes(_muon(), 1, t)
    precise = _muon(param_dtype=1)
    precise.precise = 1
    assert hq.hqml_muon_workspace_bytes(precise, 1, t) == wide
    assert hq.hqml_muon_workspace_bytes(_muon(param_dtype=1), 1, t) - joins < 0.6 * (wide - joins)


@pytest.mark.parametrize("C,G,dtype", [(4096, 32, "bf16"), (4096, 4096, "bf16"), (2048, 32, "bf16"), (1024, 1, "fp32"), (784, 16, "fp32"),
                                       (24, 3, "bf16"), (1, 1, "fp32")])
def test_norm_workspace_does_not_grow_with_samples(C, G, dtype):
    """Each sample that goes with others has two sums a channel, two values a group of its own and two of its chunks', and a
    counter's cache line: 2,048 samples, or more in up to 64 MiB; 2^30 positions take no more.  The kernels of small samples
    leave up to 768 rows of two sums a channel."""
    _lib()
    sizes = [hq.hqml_norm_workspace_bytes(hq.make_norm_config(C, G, rows, dtype=dtype)) for rows in (1 << 10, 1 << 20, 1 << 30)]
    most = max(2048 * (4 * (2 * C + 4 * G) + 128), 64 << 20) + 768
    assert 0 < sizes[0] <= sizes[1] <= sizes[2] <= most


def test_muon_border_of_long_matrices():
    """As the header has it: 14,336 values take no workspace with any number of steps, longer matrices of up to 64 on one side
    little with up to six of the usual steps, and a larger matrix's with more, unless a compute unit holds them."""
    _lib()

    def need(rows, cols, steps):
        t = (hq.hqml_muon_tensor * 1)(hq.hqml_muon_tensor(None, None, None, rows, cols, 1.0))
        return hq.hqml_muon_workspace_bytes(_muon(param_dtype=1, steps=steps), 1, t)

    for steps in (1, 6, 7, 100):
        assert need(64, 224, steps) == 0 and need(224, 64, steps) == 0
    for rows, cols in ((64, 5000), (5000, 50), (16, 16384)):
        assert 0 < need(rows, cols, 1) == need(rows, cols, 6) < 4 << 20
        assert need(rows, cols, 7) > 64 << 20
    assert need(40, 300, 6) > 0 and need(40, 300, 7) == 0
