"""AdamW over many tensors against its formula in 64 bits.

Bounds, set before the first run, with e the rounding unit of the arithmetic (2^-24, 2^-53):
m and v round three times: 4 e of the sum of their terms' magnitudes.  The update divides and
multiplies five times by what carries such errors: 32 e |update| (a moment held in 64 bits by
the reference enters with its own magnitudes), and p rounds twice (2 e |p|), or once more
into bf16 (2^-8 |p|).  8-bit codes: the nearest to x / scale, half a step of e4m3 with 1e-5 of
slack for the 32-bit arithmetic before it.
"""
import math

import pytest

from gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

LR, BETAS, EPS, DECAY = 3e-3, (0.9, 0.995), 1e-8, 0.02
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp64": torch.float64}


def optimiser(params, bits=32, **kw):
    from qml_gradients_amd.optim import AdamW
    return AdamW(params, **{**dict(lr=LR, betas=BETAS, eps=EPS, weight_decay=DECAY, state_bits=bits), **kw})


def parameters(sizes, dtype, seed, grad=None):
    g = torch.Generator().manual_seed(seed)
    params = []
    for n in sizes:
        p = torch.nn.Parameter(torch.randn(n, generator=g, dtype=torch.float64).to(DTYPES[dtype]).cuda())
        p.grad_dtype = DTYPES[grad or dtype]
        p.grad = gradient(n, g).to(DTYPES[grad or dtype]).cuda()
        params.append(p)
    return params, g


def gradient(n, g):
    return torch.randn(n, generator=g, dtype=torch.float64) * torch.exp(torch.randn(n, generator=g, dtype=torch.float64) * 2 - 4)


def decode(codes, scale):
    at = torch.arange(codes.numel()) // 256
    return codes.cpu().float().double().view(-1) * scale.cpu().double()[at]


def formula(p, g, m, v, t):
    """(p, m, v, magnitudes of m's and v's terms, update)"""
    b1, b2 = BETAS
    m2, v2 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    mags = (b1 * m).abs() + ((1 - b1) * g).abs(), v2
    up = LR * (m2 / (1 - b1 ** t)) / ((v2 / (1 - b2 ** t)).sqrt() + EPS)
    room = LR * (mags[0] / (1 - b1 ** t)) / ((v2 / (1 - b2 ** t)).sqrt() + EPS)
    return p - LR * DECAY * p - up, m2, v2, mags, room


SIZES = [[1], [255, 256, 257], [24, 4096, 1, 4097, 60000], [12345, 8192, 3], [0, 5, 0]]


@pytest.mark.parametrize("dtype,grad", [("fp32", None), ("bf16", None), ("fp64", None), ("fp32", "bf16"), ("bf16", "fp32")])
@pytest.mark.parametrize("case", range(len(SIZES)))
def test_step_matches_formula(case, dtype, grad):
    say(f"[gpu] adamw {SIZES[case]} {dtype} gradients {grad or dtype}")
    params, g = parameters(SIZES[case], dtype, 50 + case, grad)
    opt = optimiser(params)
    e = 2.0 ** -53 if dtype == "fp64" else 2.0 ** -24
    for t in (1, 2, 3):
        before = [(p.detach().cpu().double(), p.grad.cpu().double(),
                   *(opt.state[p][k].cpu().double() if opt.state[p] else torch.zeros(p.shape, dtype=torch.float64)
                     for k in ("exp_avg", "exp_avg_sq"))) for p in params]
        opt.step()
        for p, b in zip(params, before):
            want, m, v, mags, room = formula(*b, t)
            s = opt.state[p]
            assert s["step"] == t and s["exp_avg"].dtype == (torch.float64 if dtype == "fp64" else torch.float32)
            assert bool(((s["exp_avg"].cpu().double() - m).abs() <= 4 * e * mags[0]).all())
            assert bool(((s["exp_avg_sq"].cpu().double() - v).abs() <= 4 * e * mags[1]).all())
            bound = 32 * e * room + 2 * e * (want.abs() + room)
            if dtype == "bf16":
                bound = bound + 2.0 ** -8 * (want.abs() + bound)
            assert bool(((p.detach().cpu().double() - want).abs() <= bound).all())
        for p in params:
            p.grad = gradient(p.numel(), g).to(p.grad.dtype).cuda()


def half_step(u):
    """Half the distance of neighbouring e4m3 values at magnitude u."""
    return torch.exp2(torch.floor(torch.log2(u.abs().clamp_min(2.0 ** -6))) - 4)


@pytest.mark.parametrize("dtype,grad", [("fp32", None), ("bf16", None), ("fp32", "bf16"), ("bf16", "fp32")])
@pytest.mark.parametrize("case", range(len(SIZES)))
def test_eight_bit_moments(case, dtype, grad):
    say(f"[gpu] adamw 8-bit {SIZES[case]} {dtype} gradients {grad or dtype}")
    params, g = parameters(SIZES[case], dtype, 80 + case, grad)
    opt = optimiser(params, 8)
    e = 2.0 ** -24
    for t in (1, 2, 3):
        before = []
        for p in params:
            s = opt.state[p]
            m, r = ((decode(s[k], s[k + "_scale"]) for k in ("exp_avg", "exp_avg_sq_root")) if s
                    else (torch.zeros(p.numel(), dtype=torch.float64),) * 2)
            before.append((p.detach().cpu().double(), p.grad.cpu().double(), m, r * r))
        opt.step()
        for p, b in zip(params, before):
            want, m, v, mags, room = formula(*b, t)
            s = opt.state[p]
            bound = 40 * e * room + 2 * e * (want.abs() + room)
            if dtype == "bf16":
                bound = bound + 2.0 ** -8 * (want.abs() + bound)
            assert bool(((p.detach().cpu().double() - want).abs() <= bound).all())
            for name, x, mag in (("exp_avg", m, mags[0]), ("exp_avg_sq_root", v.sqrt(), v.sqrt())):
                assert s[name].dtype == torch.float8_e4m3fn and s[name].shape == p.shape
                codes, scale = s[name].cpu().float().double().view(-1), s[name + "_scale"].cpu().double()
                blocks = -(-p.numel() // 256)
                assert scale.shape == (blocks,)
                for k in range(blocks):
                    part = slice(256 * k, min(256 * k + 256, p.numel()))
                    amax = float(x[part].abs().max())
                    assert abs(float(scale[k]) - max(amax / 448, 2.0 ** -100)) <= 8 * e * (float(mag[part].max()) / 448 + 2.0 ** -100)
                u = x / scale[torch.arange(p.numel()) // 256]
                slack = 1e-5 * (mag / scale[torch.arange(p.numel()) // 256])
                near = (codes - u).abs() <= half_step(u) + slack
                raised = (codes.abs() == 2.0 ** -9) & (u.abs() < 2.0 ** -9) & (u != 0)   # never becomes zero
                assert bool((near | raised).all())
                # not zero where the terms do not cancel within their own rounding
                assert bool((codes[x.abs() > 4 * e * mag] != 0).all()) and bool((codes[mag == 0] == 0).all())
        for p in params:
            p.grad = gradient(p.numel(), g).to(p.grad.dtype).cuda()


def test_e4m3_codes_match_torch():
    """Codes over the whole range, subnormal ones and ties among them, bit for bit as torch's
    conversion: the gradient reaches the moment alone when beta1 is 0."""
    edges = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mids = (edges[1:] + edges[:-1]) / 2
    x = torch.cat([edges, mids, mids * (1 + 2.0 ** -20), mids * (1 - 2.0 ** -20)])
    x = torch.cat([x, -x])
    rows = -(-x.numel() // 255)
    x = torch.cat([x, torch.zeros(rows * 255 - x.numel())]).view(rows, 255)
    x = torch.cat([torch.full((rows, 1), 448.0), x], dim=1).contiguous()   # every block's scale is 1
    p = torch.nn.Parameter(torch.zeros(x.numel(), device="cuda"))
    p.grad = x.view(-1).cuda()
    opt = optimiser([p], 8, betas=(0.0, 0.5))
    opt.step()
    s = opt.state[p]
    assert bool((s["exp_avg_scale"] == 1.0).all())
    held = torch.where(x.view(-1).abs() < 2.0 ** -9, torch.sign(x.view(-1)) * 2.0 ** -9, x.view(-1))
    want = held.to(torch.float8_e4m3fn).float()
    got = s["exp_avg"].cpu().float()
    assert torch.equal(got, want)


def test_many_tensors_of_odd_sizes_and_alignments():
    """More tensors than one launch takes, as slices of one buffer at odd offsets."""
    say("[gpu] adamw 131 slices")
    for dtype, bits in (("fp32", 32), ("bf16", 32), ("bf16", 8), ("fp32", 8)):
        g = torch.Generator().manual_seed(6)
        sizes = [1 + (37 * i * i) % 900 for i in range(131)]
        flat = torch.randn(sum(sizes) + 200, generator=g).to(DTYPES[dtype]).cuda()
        grads = torch.randn(sum(sizes) + 200, generator=g).to(DTYPES[dtype]).cuda()
        whole, params, at = flat.clone(), [], 1
        for n in sizes:
            p = torch.nn.Parameter(flat[at:at + n])
            p.grad = grads[at:at + n]
            params.append(p)
            at += n + 1
        alone = []
        for p in params:   # each tensor by itself, in arrays of its own
            q = torch.nn.Parameter(p.detach().clone())
            q.grad = p.grad.clone()
            o = optimiser([q], bits)
            o.step()
            o.step()
            alone.append(q.detach())
        opt = optimiser(params, bits)
        opt.step()
        opt.step()
        touched = torch.zeros(flat.numel(), dtype=torch.bool)
        at = 1
        for n, p, q in zip(sizes, params, alone):
            assert torch.equal(p.detach(), q)
            touched[at:at + n] = True
            at += n + 1
        assert torch.equal(flat.cpu()[~touched], whole.cpu()[~touched])


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_infinite_and_nan_gradients(bits):
    n = 1024
    p = torch.nn.Parameter(torch.ones(n, device="cuda"))
    p.grad = torch.zeros(n, device="cuda")
    opt = optimiser([p], bits)
    opt.step()
    want = torch.full((n,), 1 - LR * DECAY, dtype=torch.float64)
    assert bool(((p.detach().cpu().double() - want).abs() <= 2.0 ** -23).all())
    p.grad[300] = float("nan")
    p.grad[600] = float("inf")
    opt.step()
    bad = ~torch.isfinite(p.detach().cpu())
    assert bad[300] and bad[600] and int(bad.sum()) == 2    # inf / inf
    p.grad.zero_()
    opt.step()
    bad = ~torch.isfinite(p.detach().cpu())
    if bits == 32:
        assert int(bad.sum()) == 2
    else:   # a block shares its scale
        want = torch.zeros(n, dtype=torch.bool)
        want[256:768] = True
        assert torch.equal(bad, want)


def test_tiny_gradients_keep_a_root():
    """A root far below its block's largest is held as the smallest code, not as zero: the step
    stays of the size of lr."""
    p = torch.nn.Parameter(torch.zeros(256, device="cuda"))
    p.grad = torch.full((256,), 1e-7, device="cuda")
    p.grad[0] = 1.0
    opt = optimiser([p], 8, weight_decay=0.0, eps=1e-12)
    for _ in range(5):
        opt.step()
    assert float(p.detach().abs().max()) <= 5 * LR * 1.5
    assert bool((opt.state[p]["exp_avg_sq_root"].float() > 0).all())


def test_side_stream_and_large_tensor():
    """A tensor of more than 2^24 elements on a side stream, bitwise as on the main one."""
    n = (1 << 24) + 13
    g = torch.Generator(device="cuda").manual_seed(3)
    start = torch.randn(n, generator=g, device="cuda")
    grad = torch.randn(n, generator=g, device="cuda") * 1e-3
    for bits in (32, 8):
        res = []
        for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
            torch.cuda.synchronize()
            with torch.cuda.stream(stream):
                p = torch.nn.Parameter(start.clone())
                p.grad = grad * 1.0
                opt = optimiser([p], bits)
                opt.step()
                opt.step()
            stream.synchronize()
            res.append(p.detach())
        assert torch.equal(*res)
        b1, b2 = BETAS
        at = torch.tensor([0, 1, 4095, 4096, n // 2, n - 14, n - 1])
        # two equal gradients: m and v over their corrections are g and g^2
        if bits == 32:
            want = start[at].cpu().double()
            for _ in range(2):
                want = want * (1 - LR * DECAY) - LR * grad[at].cpu().double() / (grad[at].cpu().double().abs() + EPS)
            assert bool(((res[0][at].cpu().double() - want).abs() <= 1e-6).all())


@pytest.mark.parametrize("bits,dtype", [(32, "bf16"), (8, "fp32"), (32, "fp64")])
def test_state_dict_round_trip(bits, dtype):
    params, g = parameters([300, 7], dtype, 9)
    opt = optimiser(params, bits)
    opt.step()
    saved = {k: v for k, v in opt.state_dict().items()}
    copies = [torch.nn.Parameter(p.detach().clone()) for p in params]
    other = optimiser(copies, bits)
    other.load_state_dict(saved)
    for p, q in zip(params, copies):
        q.grad = p.grad.clone()
        for k, v in opt.state[p].items():
            if isinstance(v, torch.Tensor):
                assert other.state[q][k].dtype == v.dtype and other.state[q][k].data_ptr() != v.data_ptr()
    opt.step()
    other.step()
    for p, q in zip(params, copies):
        assert torch.equal(p, q)


def test_step_marks_parameters_changed():
    p = torch.nn.Parameter(torch.ones(4, device="cuda"))
    loss = (p * p).sum()
    p.grad = torch.ones(4, device="cuda")
    optimiser([p]).step()
    with pytest.raises(RuntimeError):
        loss.backward()


def test_hooks_run_once():
    p = torch.nn.Parameter(torch.ones(4, device="cuda"))
    p.grad = torch.ones(4, device="cuda")
    opt, seen = optimiser([p]), []
    opt.register_step_pre_hook(lambda o, a, k: seen.append(("before", float(p[0]))))
    opt.register_step_post_hook(lambda o, a, k: seen.append(("after", float(p[0]))))
    opt.step()
    assert [s[0] for s in seen] == ["before", "after"] and seen[0][1] == 1.0 and seen[1][1] < 1.0


def test_learning_rate_schedule_and_closure():
    p = torch.nn.Parameter(torch.ones(4, device="cuda"))
    opt = optimiser([p], weight_decay=0.0)
    schedule = torch.optim.lr_scheduler.StepLR(opt, step_size=1, gamma=0.1)

    def closure():
        opt.zero_grad()
        loss = p.sum()
        loss.backward()
        return loss

    moves = []
    for _ in range(3):
        before = float(p[0])
        assert float(opt.step(closure)) == pytest.approx(4 * before, rel=1e-6)
        moves.append(before - float(p[0]))
        schedule.step()
    for k, move in enumerate(moves):   # equal gradients: each step is lr itself
        assert move == pytest.approx(LR * 0.1 ** k, rel=1e-2)


def test_parameters_without_gradient_wait():
    a, b = (torch.nn.Parameter(torch.ones(4, device="cuda")) for _ in range(2))
    opt = optimiser([a, b])
    a.grad = torch.ones(4, device="cuda")
    opt.step()
    assert opt.state[a]["step"] == 1 and not opt.state[b] and bool((b == 1).all())
    b.grad = torch.ones(4, device="cuda")
    opt.step()
    assert opt.state[a]["step"] == 2 and opt.state[b]["step"] == 1


def test_refusals():
    import ctypes

    import qml_gradients_amd as hq
    from qml_gradients_amd.optim import AdamW
    ok = torch.nn.Parameter(torch.ones(8, device="cuda"))
    for bad in (torch.nn.Parameter(torch.ones(8)), torch.nn.Parameter(torch.ones(8, device="cuda", dtype=torch.float16)),
                torch.nn.Parameter(torch.ones(8, 8, device="cuda").t()[:, :4])):
        with pytest.raises(ValueError):
            AdamW([bad])
    with pytest.raises(ValueError):
        AdamW([torch.nn.Parameter(torch.ones(8, device="cuda", dtype=torch.float64))], state_bits=8)
    for kw in (dict(lr=-1.0), dict(betas=(1.0, 0.9)), dict(eps=-1e-8), dict(weight_decay=-1.0), dict(state_bits=4)):
        with pytest.raises(ValueError):
            AdamW([ok], **kw)
    buf = torch.zeros(64, device="cuda")
    q = buf.data_ptr()

    def call(n=8, words=None, **kw):
        f = dict(param_dtype=0, grad_dtype=0, moments=0, step=1, lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8,
                 weight_decay=0.0, device=0, stream=0)
        cfg = hq.hqml_adamw_config(**{**f, **kw})
        w = words or (q, q + 32, q + 64, q + 96, 0, 0, n)
        hq.hqml_adamw_step(cfg, 1, (ctypes.c_longlong * 7)(*w))

    for kw in (dict(step=0), dict(lr=math.nan), dict(beta1=1.0), dict(eps=-1.0), dict(param_dtype=9), dict(moments=2),
               dict(grad_dtype=2), dict(n=-1), dict(n=(1 << 40) + 1), dict(device=-1),
               dict(words=(q, 0, q + 64, q + 96, 0, 0, 8)), dict(words=(q + 2, q + 32, q + 64, q + 96, 0, 0, 8)),
               dict(moments=1), dict(n=1 << 36)):
        with pytest.raises(hq.HqmlError) as e:
            call(**kw)
        assert e.value.status == hq.HQML_ERR_ARG, kw
    with pytest.raises(hq.HqmlError) as e:
        call(param_dtype=2, grad_dtype=2, moments=1)
    assert e.value.status == hq.HQML_ERR_UNSUPPORTED
    assert not buf.any()


def test_capture_is_refused():
    import qml_gradients_amd as hq
    p = torch.nn.Parameter(torch.ones(8, device="cuda"))
    p.grad = torch.ones(8, device="cuda")
    opt = optimiser([p])
    opt.step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x = torch.ones(8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            x.mul_(2.0)
            with pytest.raises(hq.HqmlError) as e:
                opt.step()
    assert e.value.status == hq.HQML_ERR_UNSUPPORTED and opt.state[p]["step"] == 1


def test_example_trains_with_either_state():
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    try:
        import hybrid_readout
    finally:
        sys.path.pop(0)
    for bits in (32, 8):
        losses = hybrid_readout.train(steps=40, bits=bits)
        say(f"[gpu] hybrid readout, {bits}-bit moments: loss {losses[0]:.4f} -> {losses[-1]:.4f}")
        assert losses[-1] < 0.25 * losses[0]
