"""Muon against its definition in 64 bits.  With p = 0 and lr = 1 a step leaves the orthogonalised update itself; its bounds
are layers_reference.orthogonal_bound's.  Momentum: two products and a sum of each element, 3 E of their sizes."""
import math

import pytest

from gpu_util import say
from layers_reference import COEFFICIENTS, E, TYPES, muon, orthogonal_bound

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def gradient(rows, cols, seed, dtype="fp32", few=4):
    """A few directions that stand out of noise."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    return ((normal(rows, few) @ normal(few, cols) + normal(rows, cols)) * 1e-3).to(TYPES[dtype][0])


def matrices(sizes, dtype="fp32", grad=None, seed=0, zero=False):
    params = []
    for n, (r, c) in enumerate(sizes):
        g = torch.Generator(device="cuda").manual_seed(100 + n + seed)
        p = torch.zeros(r, c, device="cuda") if zero else torch.randn(r, c, generator=g, device="cuda") * 0.05
        params.append(torch.nn.Parameter(p.to(TYPES[dtype][0])))
        params[-1].grad_dtype = None   # any
        params[-1].grad = gradient(r, c, n + seed, grad or dtype)
    return params


def check(sizes, dtype, grad=None, nesterov=True, steps=5, coefficients=COEFFICIENTS, seed=0):
    """One step from zero parameters and a momentum; returns the optimiser."""
    from qml_gradients_amd.optim import Muon
    say(f"[gpu] muon {sizes} {dtype} gradients {grad or dtype}")
    params = matrices(sizes, dtype, grad, seed, zero=True)
    opt = Muon(params, lr=1.0, nesterov=nesterov, steps=steps, coefficients=coefficients, adjust="none")
    before = []
    for n, p in enumerate(params):
        opt.state[p]["momentum"] = gradient(*p.shape, 50 + n + seed)
        before.append(opt.state[p]["momentum"].clone())
    opt.step()
    for p, m0 in zip(params, before):
        m, u = muon(p, p.grad, m0, 1.0, 0.95, 0.0, nesterov, 1.0)
        held = opt.state[p]["momentum"]
        assert bool(((held.double() - m).abs() <= 3 * E * (m0.double().abs() + p.grad.double().abs())).all())
        x, norm_bound, most = orthogonal_bound(u, dtype, steps, coefficients)
        off = -p.detach().double() - x
        rounding = TYPES[dtype][1] * x.abs()
        worst = float((off.abs() - rounding).max())
        got = float(torch.linalg.vector_norm(off))
        limit = norm_bound + float(torch.linalg.vector_norm(rounding))
        say(f"      off {got:.2e} (limit {limit:.2e}), largest {worst:.2e} ({most:.2e}), of {float(torch.linalg.vector_norm(x)):.2f}")
        assert got <= limit and worst <= most
    return opt


SIZES = [[(1, 1)], [(1, 5), (7, 1)], [(2, 3), (3, 2)], [(16, 16)], [(64, 12), (20, 64), (4, 64)], [(33, 65), (65, 33)],
         [(128, 64)], [(100, 300), (300, 100)], [(257, 129)], [(5, 2000), (2000, 5)], [(517, 803)], [(64, 784), (20, 784)],
         [(300, 300), (8, 16), (513, 40), (1, 100)], [(1000, 1030)], [(640, 2100), (2100, 640)]]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("n", range(len(SIZES)))
def test_sizes(n, dtype):
    check(SIZES[n], dtype, nesterov=n % 3 != 1, seed=n)


@pytest.mark.parametrize("dtype,grad", [("fp32", "bf16"), ("bf16", "fp32")])
def test_types_mixed(dtype, grad):
    check([(40, 70), (200, 130)], dtype, grad)


@pytest.mark.parametrize("steps,coefficients", [(1, COEFFICIENTS), (2, COEFFICIENTS), (9, COEFFICIENTS), (12, (1.5, -0.5, 0.0)),
                                                (3, (2.0, -1.5, 0.5))])
def test_steps_and_coefficients(steps, coefficients):
    check([(48, 90), (150, 60)], "fp32", steps=steps, coefficients=coefficients)


@pytest.mark.parametrize("sizes,dtype", [
    ([(3000, 3000)] * 2, "bf16"),                       # more of the largest tiles than compute units
    ([(2100, 2300)], "fp32"), ([(2400, 2100)], "fp32"),
    ([(200, 6000), (6000, 200)], "bf16"), ([(200, 6000), (6000, 200)], "fp32"),   # few tiles, split along k
    ([(64, 350), (350, 64), (64, 420), (48, 500)], "fp32"), ([(16, 2000), (2500, 16), (33, 600)], "bf16")])   # around the LDS's size
def test_cuts(sizes, dtype):
    check(sizes, dtype, seed=3)


THIN = [[(1, 30000)], [(64, 5000), (5000, 64)], [(7, 4099), (4099, 16), (17, 3000), (2049, 33)], [(48, 1300), (1300, 49)],
        [(64, 40000), (3, 65536)], [(62, 1175), (100, 90), (8, 8), (1175, 62)]]


@pytest.mark.parametrize("dtype,grad", [("fp32", "fp32"), ("bf16", "bf16"), ("fp32", "bf16"), ("bf16", "fp32")])
@pytest.mark.parametrize("n", range(len(THIN)))
def test_thin_matrices(n, dtype, grad):
    check(THIN[n], dtype, grad, nesterov=n % 2 == 0, seed=n)


@pytest.mark.parametrize("sizes", [(40, 3000), (5000, 64), (30, 40), (300, 200)])
def test_gradients_of_few_directions(sizes):
    """Two directions, and, of the roundings, all others 1e-8 as large: what comes of those is as large as in 64 bits."""
    from qml_gradients_amd.optim import Muon
    r, c = sizes
    g = torch.Generator(device="cuda").manual_seed(1)
    p = torch.nn.Parameter(torch.zeros(r, c, device="cuda"))
    p.grad = torch.randn(r, 2, generator=g, device="cuda") @ torch.randn(2, c, generator=g, device="cuda")
    opt = Muon([p], lr=1.0, adjust="none")
    opt.step()
    _, u = muon(p, p.grad, torch.zeros_like(p), 1.0, 0.95, 0.0, True, 1.0)
    x, norm_bound, most = orthogonal_bound(u, "fp32", 5, COEFFICIENTS)
    off = -p.detach().double() - x
    assert float(torch.linalg.vector_norm(off)) <= norm_bound + 2.0 ** -24 * float(torch.linalg.vector_norm(x))
    assert float((off.abs() - 2.0 ** -24 * x.abs()).max()) <= most


@pytest.mark.parametrize("steps,coefficients", [(1, COEFFICIENTS), (2, COEFFICIENTS), (6, COEFFICIENTS), (9, COEFFICIENTS),
                                                (12, (1.5, -0.5, 0.0)), (3, (2.0, -1.5, 0.5))])
def test_steps_of_thin_matrices(steps, coefficients):
    check([(50, 1500), (3000, 10)], "fp32", steps=steps, coefficients=coefficients)


def test_large_and_small_matrices_in_one_call():
    check([(70 + n, 90 + 2 * n) if n % 3 else (5 + n, 40) for n in range(45)], "bf16")
    check([(70 + n, 90 + 2 * n) for n in range(5)], "fp32")


def test_more_matrices_than_a_launch_takes():
    check([(3 + n, 70 - n) for n in range(40)], "fp32")


def test_step():
    """p (1 - lr decay) - lr f X, over several steps: E of p for each product and sum, and X's error times lr f."""
    from qml_gradients_amd.optim import Muon
    for adjust, f in (("spectral", lambda r, c: math.sqrt(max(1, r / c))), ("rms", lambda r, c: 0.2 * math.sqrt(max(r, c))),
                      ("none", lambda r, c: 1.0)):
        for dtype in ("fp32", "bf16"):
            params = matrices([(60, 40), (30, 90), (200, 220)], dtype)
            opt = Muon(params, lr=0.03, momentum=0.9, weight_decay=0.1, adjust=adjust)
            m = [torch.zeros(p.shape, dtype=torch.float64, device="cuda") for p in params]
            for step in range(3):
                before = [p.detach().double() for p in params]
                for n, p in enumerate(params):
                    p.grad = gradient(*p.shape, 10 * step + n, dtype)
                held = [opt.state[p]["momentum"].double() if step else torch.zeros_like(b) for p, b in zip(params, before)]
                opt.step()
                for n, p in enumerate(params):
                    m[n], u = muon(p, p.grad, held[n], 0, 0.9, 0, True, 0)
                    x, norm_bound, most = orthogonal_bound(u, dtype)
                    size = 0.03 * f(*p.shape)
                    want = before[n] * (1 - 0.03 * 0.1) - size * x
                    bound = size * most + 4 * E * (before[n].abs() + size * x.abs()) + TYPES[dtype][1] * want.abs() * 1.01
                    assert bool(((p.detach().double() - want).abs() <= bound).all())


def test_orthogonal():
    """The singular values end between 0.6 and 1.3 (where the polynomial leaves those that begin above 1e-3), the
    singular vectors where they were."""
    from qml_gradients_amd.optim import Muon
    p = matrices([(96, 160)], zero=True)
    Muon(p, lr=1.0, momentum=0.0, adjust="none").step()
    u, s, vh = torch.linalg.svd(p[0].grad.double(), full_matrices=False)
    x = -p[0].detach().double()
    d = u.t() @ x @ vh.t()
    assert 0.6 < float(d.diagonal().min()) and float(d.diagonal().max()) < 1.3
    assert float((d - torch.diag(d.diagonal())).abs().max()) < 1e-4


def test_sizes_of_gradients_do_not_count():
    """Only eps does: 1e-30 and 1e30 give the same update; below eps it falls with the gradient."""
    from qml_gradients_amd.optim import Muon
    got = []
    for size in (1.0, 2.0 ** 100, 2.0 ** -80):
        p = matrices([(30, 50)], zero=True)
        p[0].grad = gradient(30, 50, 1) * size
        Muon(p, lr=1.0, adjust="none", eps=1e-30).step()
        got.append(p[0].detach())
    assert torch.allclose(got[0], got[1], atol=1e-5) and torch.allclose(got[0], got[2], atol=1e-5)
    p = matrices([(30, 50)], zero=True)
    p[0].grad = torch.full((30, 50), 1e-12, device="cuda")   # norm 3.9e-11, below eps
    Muon(p, lr=1.0, momentum=0.0, adjust="none", steps=1).step()
    assert torch.allclose(-p[0], torch.full_like(p[0], 3.4445e-5), rtol=1e-3)


@pytest.mark.parametrize("sizes", [[(20, 30)], [(300, 200)], [(20, 3000)]])
def test_gradients_of_zero_and_nan(sizes):
    """Zeros: only the decay.  A NaN or an infinity: the whole matrix, and none beside it."""
    from qml_gradients_amd.optim import Muon
    sizes = sizes * 3
    params = matrices(sizes)
    before = [p.detach().clone() for p in params]
    params[0].grad.zero_()
    params[2].grad[1, 2] = float("nan")
    opt = Muon(params, lr=0.5, weight_decay=0.25)
    opt.step()
    assert torch.allclose(params[0], before[0] * 0.875, rtol=1e-6)
    assert params[2].isnan().all() and not params[1].isnan().any()
    assert not opt.state[params[0]]["momentum"].any()


def test_gradients_in_other_layouts_and_none():
    from qml_gradients_amd.optim import Muon
    a, b = matrices([(40, 60), (30, 20)]), matrices([(40, 60), (30, 20)])
    for p in b:
        p.grad = p.grad.t().contiguous().t()
    extra = torch.nn.Parameter(torch.ones(3, 4, device="cuda"))
    empty = torch.nn.Parameter(torch.ones(0, 4, device="cuda"))
    empty.grad = torch.ones(0, 4, device="cuda")
    x, y = Muon(a), Muon(b + [extra, empty])
    x.step(), y.step()
    assert all(torch.equal(p, q) for p, q in zip(a, b)) and (extra == 1).all()
    nothing = Muon([empty])
    nothing.step()


def test_same_result_whatever_else_is_in_the_call():
    """A matrix alone, and among others."""
    from qml_gradients_amd.optim import Muon
    for sizes in ([(40, 64), (64, 40)], [(300, 420), (129, 700)]):
        together = matrices(sizes)
        Muon(together).step()
        for n in range(2):
            alone = matrices(sizes)[n]
            Muon([alone]).step()
            assert torch.allclose(alone, together[n], atol=1e-6)


def test_streams_and_graphs():
    """A captured step repeats the step, with what the gradients then hold; eager ones on another stream come between."""
    from qml_gradients_amd.optim import Muon
    for sizes in ([(40, 30)], [(300, 420), (128, 200)], [(2000, 40), (10, 4000)], [(64, 2000), (20, 30), (100, 90)]):
        a, b = matrices(sizes), matrices(sizes)
        x, y = Muon(a), Muon(b)
        x.step(), y.step()
        torch.cuda.synchronize()
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=side):
            x.step()
        for seed in (1, 2, 3):
            for n, (p, q) in enumerate(zip(a, b)):
                new = gradient(*p.shape, 30 * seed + n)
                p.grad.copy_(new), q.grad.copy_(new)
            graph.replay()
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                y.step()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(a, b))
            assert all(torch.equal(x.state[p]["momentum"], y.state[q]["momentum"]) for p, q in zip(a, b))


def test_two_streams_at_once():
    """Steps of their own parameters do not disturb each other."""
    from qml_gradients_amd.optim import Muon
    sizes = [(200, 6000), (300, 200), (20, 30), (3000, 33)]
    both = [matrices(sizes, seed=n) for n in (0, 40)]
    alone = [matrices(sizes, seed=n) for n in (0, 40)]
    streams = [torch.cuda.Stream() for _ in both]
    opts = [Muon(p, lr=0.1) for p in both]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, o in zip(streams, opts):
            with torch.cuda.stream(s):
                o.step()
    torch.cuda.synchronize()
    for p in alone:
        o = Muon(p, lr=0.1)
        for _ in range(4):
            o.step()
    assert all(torch.equal(a, b) for x, y in zip(both, alone) for a, b in zip(x, y))


def test_parameters_are_marked_changed():
    from qml_gradients_amd.optim import Muon
    p = matrices([(8, 6)])
    loss = (p[0] * p[0]).sum()
    Muon(p).step()
    with pytest.raises(RuntimeError):
        loss.backward()


def test_saved_and_loaded():
    """A bf16 parameter's momentum stays in fp32."""
    import copy
    from qml_gradients_amd.optim import Muon
    a, b = matrices([(30, 20)], "bf16"), matrices([(30, 20)], "bf16")
    x, y = Muon(a, lr=0.1), Muon(b)
    x.step()
    b[0].data.copy_(a[0].data)
    y.load_state_dict(copy.deepcopy(x.state_dict()))
    assert y.state[b[0]]["momentum"].dtype is torch.float32 and y.param_groups[0]["lr"] == 0.1
    x.step(), y.step()
    assert torch.equal(a[0], b[0])


def test_refusals():
    import qml_gradients_amd as hq
    from qml_gradients_amd.optim import Muon
    p = torch.nn.Parameter(torch.randn(160, 80, device="cuda"))
    p.grad = torch.randn(160, 80, device="cuda")
    m = torch.zeros(160, 80, device="cuda")
    cfg = hq.hqml_muon_config(0, 0, 1, 5, 0.1, 0.9, 0.0, 1e-7, *COEFFICIENTS, 0, None)
    t = hq.hqml_muon_tensor(p.data_ptr(), p.grad.data_ptr(), m.data_ptr(), 160, 80, 1.0)
    need = hq.hqml_muon_workspace_bytes(cfg, 1, (hq.hqml_muon_tensor * 1)(t))
    work = torch.empty(need, dtype=torch.uint8, device="cuda")

    def call(bytes=need, ptr=work.data_ptr(), **change):
        u = hq.hqml_muon_tensor(t.param, t.grad, t.momentum, t.rows, t.cols, t.scale)
        for k, v in change.items():
            setattr(u, k, v)
        hq.hqml_muon_step(cfg, 1, (hq.hqml_muon_tensor * 1)(u), ptr, bytes)

    call()
    for bad in (dict(bytes=need - 1), dict(ptr=None), dict(ptr=work.data_ptr() + 16), dict(param=None), dict(grad=None),
                dict(momentum=None), dict(param=p.data_ptr() + 2), dict(momentum=m.data_ptr() + 1), dict(rows=-1),
                dict(rows=1 << 17), dict(cols=1 << 17), dict(scale=-1.0), dict(scale=math.inf), dict(rows=1 << 12, cols=1 << 12)):
        with pytest.raises(hq.HqmlError) as e:
            call(**bad)
        assert e.value.status == hq.HQML_ERR_ARG, bad
    for bad in (torch.randn(8, device="cuda"), torch.randn(8, 8, device="cuda", dtype=torch.float64), torch.randn(8, 8),
                torch.randn(8, 4, device="cuda").t()):
        with pytest.raises(ValueError):
            Muon([torch.nn.Parameter(bad)])
    opt = Muon([p])
    opt.state[p]["momentum"] = torch.zeros(80, 160, device="cuda")
    with pytest.raises(ValueError):
        opt.step()


def beyond_rounding(p, x):
    """How far p is from -x beyond its own type's rounding, of each element."""
    u = 2.0 ** -8 if p.dtype is torch.bfloat16 else 2.0 ** -24
    return ((-p.detach().double() - x).abs() - u * x.abs()).clamp_min(0.0)


def check_tight(grads, dtype, steps=5, **how):
    """As check, but what is left beyond the parameter's own rounding is held to the bounds of two fp16 values for each
    operand, or fp32, whatever the parameter's type."""
    from qml_gradients_amd.optim import Muon
    params = []
    for g in grads:
        params.append(torch.nn.Parameter(torch.zeros(g.shape, dtype=TYPES[dtype][0], device="cuda")))
        params[-1].grad_dtype = None
        params[-1].grad = g
    Muon(params, lr=1.0, adjust="none", steps=steps, **how).step()
    for p, g in zip(params, grads):
        _, u = muon(p, g, torch.zeros(g.shape, device="cuda"), 1.0, 0.95, 0.0, True, 1.0)
        x, norm_bound, most = orthogonal_bound(u, "fp32", steps)
        off = beyond_rounding(p, x)
        say(f"[gpu] muon {tuple(g.shape)} {g.dtype} for {dtype}: off {float(torch.linalg.vector_norm(off)):.2e} ({norm_bound:.2e}), "
            f"largest {float(off.max()):.2e} ({most:.2e})")
        assert float(torch.linalg.vector_norm(off)) <= norm_bound and float(off.max()) <= most


@pytest.mark.parametrize("grad", ["bf16", "fp32"])
@pytest.mark.parametrize("sizes", [[(300, 200), (100, 700)], [(640, 2100), (2100, 640)], [(1500, 1400)], [(200, 6000)]])
def test_updates_of_bf16_parameters(sizes, grad):
    check_tight([gradient(r, c, n, grad) for n, (r, c) in enumerate(sizes)], "bf16")


@pytest.mark.parametrize("sizes", [(512, 2048), (300, 200), (2048, 512), (64, 5000)])
def test_updates_of_bf16_parameters_from_few_directions(sizes):
    """Eight directions, as a batch of eight gives: roundings of operands would be lifted in all the others."""
    r, c = sizes
    g = torch.Generator(device="cuda").manual_seed(1)
    check_tight([torch.randn(r, 8, generator=g, device="cuda") @ torch.randn(8, c, generator=g, device="cuda")], "bf16")


@pytest.mark.parametrize("grad", ["bf16", "fp32"])
@pytest.mark.parametrize("sizes", [[(300, 200), (8, 16), (64, 2000)], [(517, 803)], [(1000, 1030)], [(640, 2100), (2100, 640)],
                                   [(3000, 3000)] * 2, [(200, 6000), (6000, 200)], [(70 + n, 90 + 2 * n) for n in range(30)]])
def test_half(sizes, grad, monkeypatch):
    """One fp16 value an operand, within the bounds of that; the largest tiles, their leftovers and parts along k."""
    from qml_gradients_amd import optim

    class Half(optim.Muon):
        def __init__(self, params, **how):
            super().__init__(params, half=True, **how)

    monkeypatch.setattr(optim, "Muon", Half)
    check(sizes, "bf16", grad, seed=3)


def test_half_is_of_bf16_parameters():
    """Parameters in 32 bits do not know it; a group has it or not."""
    from qml_gradients_amd.optim import Muon
    a, b = matrices([(100, 90)]), matrices([(100, 90)])
    Muon(a, half=True).step(), Muon(b).step()
    assert torch.equal(a[0], b[0])
    c, d, e = (matrices([(100, 90)], "bf16", "fp32", zero=True) for _ in range(3))
    Muon([dict(params=c, half=True), dict(params=d)], lr=1.0).step()
    Muon(e, lr=1.0).step()
    assert torch.equal(d[0], e[0]) and not torch.equal(c[0], e[0])


def test_states_saved_without_half():
    from qml_gradients_amd.optim import Muon
    a, b = matrices([(30, 20)], "bf16"), matrices([(30, 20)], "bf16")
    x, y = Muon(a), Muon(b, half=True)
    x.step()
    state = x.state_dict()
    for group in state["param_groups"]:
        del group["half"]
    y.load_state_dict(state)
    assert y.param_groups[0]["half"] is False
    y.step()


def test_graph_and_streams_of_bf16_parameters():
    """Both precisions: a captured step repeats the step, eager ones on another stream between its replays."""
    from qml_gradients_amd.optim import Muon
    for half in (False, True):
        sizes = [(300, 420), (128, 200), (2100, 2200)]
        a, b = matrices(sizes, "bf16"), matrices(sizes, "bf16")
        x, y = Muon(a, half=half), Muon(b, half=half)
        x.step(), y.step()
        torch.cuda.synchronize()
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=side):
            x.step()
        for seed in (1, 2, 3):
            for n, (p, q) in enumerate(zip(a, b)):
                new = gradient(*p.shape, 30 * seed + n, "bf16")
                p.grad.copy_(new), q.grad.copy_(new)
            graph.replay()
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                y.step()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("sizes", [[(20, 30)], [(300, 200)], [(20, 3000)]])
def test_least_eps(sizes, dtype):
    """The least eps there is: zeros only decay, and gradients whose norm is around 2^-118 give the update of their direction."""
    from qml_gradients_amd.optim import Muon
    params = matrices(sizes * 2, dtype)
    before = [p.detach().clone() for p in params]
    params[0].grad.zero_()
    with torch.no_grad():
        params[1].zero_()
    params[1].grad.copy_(gradient(*sizes[0], 3, dtype).double() * 2.0 ** -118)
    Muon(params, lr=1.0, momentum=0.0, weight_decay=0.125, adjust="none", eps=2.0 ** -149).step()
    assert torch.equal(params[0], before[0] * 0.875)
    x, norm_bound, most = orthogonal_bound(params[1].grad, dtype, eps=2.0 ** -149)
    off = beyond_rounding(params[1], x)
    assert float(torch.linalg.vector_norm(off)) <= norm_bound and float(off.max()) <= most


@pytest.mark.parametrize("sizes", [[(16, 128), (32, 64), (64, 17)], [(16, 129)], [(32, 65)], [(33, 33)], [(128, 20), (8, 8)], [(17, 64), (96, 32)]])
def test_small_matrices_by_few_and_many_waves(sizes):
    check(sizes, "fp32")
    check(sizes, "bf16", "fp32", nesterov=False)


@pytest.mark.parametrize("steps", [6, 7, 9])
def test_long_matrices_of_bf16_parameters_with_many_steps(steps):
    """Up to six steps by a polynomial in 64 bits, more by the large matrices' products; a matrix that a compute unit holds, in 32
    bits, whatever the steps.  half takes 11 bits in the second case alone."""
    sizes = [(64, 5000), (5000, 50), (40, 300)]
    grads = [gradient(r, c, n, "bf16") for n, (r, c) in enumerate(sizes)]
    check_tight(grads, "bf16", steps)
    if steps == 6:
        check_tight(grads, "bf16", steps, half=True)
    else:
        check_tight(grads[2:], "bf16", steps, half=True)
        with pytest.raises(AssertionError):
            check_tight(grads[:1], "bf16", steps, half=True)
