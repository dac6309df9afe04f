"""The optimiser's own work, without a GPU: the entry point is replaced by one that records what it is given.

What reaches it are raw pointers with the parameter's type and number of elements, so every array behind them has to be
of that type and size."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import qml_gradients_amd as hq  # noqa: E402
from qml_gradients_amd import optim  # noqa: E402

WIDE = {hq.HQML_DTYPE_FP32: 4, hq.HQML_DTYPE_BF16: 4, hq.HQML_DTYPE_FP64: 8}   # bytes of a 32-bit moment


@pytest.fixture
def calls(monkeypatch):
    """(configuration, [7 words of each tensor]) of every call."""
    seen = []

    def record(cfg, n, words):
        seen.append((cfg, [tuple(words[7 * i:7 * i + 7]) for i in range(n)]))

    monkeypatch.setattr(optim, "hqml_adamw_step", record)
    monkeypatch.setattr(optim, "_current_stream", lambda device: 0)
    monkeypatch.setattr(optim.AdamW, "add_param_group", torch.optim.Optimizer.add_param_group)   # takes host parameters
    return seen


def parameter(n=8, dtype=torch.float32):
    p = torch.nn.Parameter(torch.ones(n, dtype=dtype))
    p.grad = torch.ones(n, dtype=dtype)
    return p


def assert_in_range(opt, seen):
    """What the last call says of each tensor is what is held there."""
    cfg, tensors = seen[-1]
    at = {w[0]: w for w in tensors}
    for p, s in opt.state.items():
        w = at[p.data_ptr()]
        n = w[6]
        assert n == p.numel()
        if cfg.moments == hq.HQML_MOMENTS_32:
            held = {2: s["exp_avg"], 3: s["exp_avg_sq"]}
            need = {2: n * WIDE[cfg.param_dtype], 3: n * WIDE[cfg.param_dtype]}
        else:
            held = {2: s["exp_avg"], 3: s["exp_avg_sq_root"], 4: s["exp_avg_scale"], 5: s["exp_avg_sq_root_scale"]}
            need = {2: n, 3: n, 4: -(-n // 256) * 4, 5: -(-n // 256) * 4}
        for k, t in held.items():
            assert w[k] == t.data_ptr() and t.is_contiguous() and t.untyped_storage().nbytes() >= need[k]
        if cfg.moments == hq.HQML_MOMENTS_32:
            assert held[2].element_size() == held[3].element_size() == WIDE[cfg.param_dtype]


@pytest.mark.parametrize("saved,own", [("float32", "float64"), ("float64", "float32"), ("bfloat16", "float64"),
                                       ("float64", "bfloat16"), ("float32", "bfloat16")])
def test_moments_loaded_follow_the_parameters_type(saved, own, calls):
    a = optim.AdamW([parameter(dtype=getattr(torch, saved))])
    a.step()
    for k in ("exp_avg", "exp_avg_sq"):
        a.state[a.param_groups[0]["params"][0]][k].fill_(0.125)
    p = parameter(dtype=getattr(torch, own))
    b = optim.AdamW([p])
    b.load_state_dict(a.state_dict())
    b.step()
    assert_in_range(b, calls)
    want = torch.float64 if own == "float64" else torch.float32
    assert all(b.state[p][k].dtype is want and bool((b.state[p][k] == 0.125).all()) for k in ("exp_avg", "exp_avg_sq"))
    assert b.state[p]["step"] == 2


@pytest.mark.parametrize("before,after", [("float32", "float64"), ("float64", "float32"), ("bfloat16", "float64")])
def test_moments_follow_a_module_that_changes_its_type(before, after, calls):
    layer = torch.nn.Linear(4, 3, dtype=getattr(torch, before))
    opt = optim.AdamW(layer.parameters())
    for _ in range(2):
        for p in layer.parameters():
            p.grad = torch.ones_like(p)
        opt.step()
        assert_in_range(opt, calls)
        layer.to(getattr(torch, after))


@pytest.mark.parametrize("bits", [32, 8])
def test_moments_of_another_size_are_refused(bits, calls):
    small, large = parameter(8), parameter(1000)
    a, b = optim.AdamW([small], state_bits=bits), optim.AdamW([large], state_bits=bits)
    a.step()
    with pytest.raises(ValueError):
        b.load_state_dict(a.state_dict())
    assert not b.state                      # nothing was taken over
    b.state[large] = dict(a.state[small])   # past the loader
    with pytest.raises(ValueError):
        b.step()
    assert len(calls) == 1
    small.data = torch.ones(1000)           # a parameter that grew under its moments and gradient
    with pytest.raises(ValueError):
        a.step()
    del small.grad
    small.grad = torch.ones(1000)
    with pytest.raises(ValueError):
        a.step()
    assert len(calls) == 1


def test_moments_held_otherwise_than_the_step_takes_them_are_refused(calls):
    p = parameter(600)
    for bits, name, other in ((32, "exp_avg", torch.zeros(600, dtype=torch.int32)),
                              (32, "exp_avg_sq", torch.zeros(600, dtype=torch.bfloat16)),
                              (32, "exp_avg_sq", torch.zeros(1200)[::2]),
                              (32, "exp_avg", torch.zeros(599)),
                              (8, "exp_avg", torch.zeros(600)),
                              (8, "exp_avg_sq_root", torch.zeros(600, dtype=torch.uint8)),
                              (8, "exp_avg_scale", torch.zeros(2)),
                              (8, "exp_avg_sq_root_scale", torch.zeros(3, dtype=torch.float64)),
                              (8, "exp_avg_sq_root_scale", None)):
        opt = optim.AdamW([p], state_bits=bits)
        opt.step()
        n = len(calls)
        if other is None:
            del opt.state[p][name]
        else:
            opt.state[p][name] = other
        with pytest.raises(ValueError):
            opt.step()
        assert len(calls) == n and opt.state[p]["step"] == 1


def test_a_state_of_the_other_bits_is_refused(calls):
    p, wide = parameter(), parameter(dtype=torch.float64)
    eight = optim.AdamW([p], state_bits=8)
    eight.step()
    with pytest.raises(ValueError):   # the saved group says 8 bits: not for 64-bit parameters
        optim.AdamW([wide]).load_state_dict(eight.state_dict())
    eight.param_groups[0]["state_bits"] = 32
    with pytest.raises(ValueError):
        eight.step()


def test_parameters_that_left_the_types_are_refused(calls):
    p = parameter()
    opt = optim.AdamW([p])
    p.data = p.data.half()
    p.grad = None
    p.grad = torch.ones(8, dtype=torch.float16)
    with pytest.raises(ValueError):
        opt.step()
    assert not calls


@pytest.mark.parametrize("bits", [32, 8])
def test_plain_steps_pass_what_they_hold(bits, calls):
    params = [parameter(n) for n in (1, 256, 257, 1000)]
    opt = optim.AdamW(params, state_bits=bits)
    for t in (1, 2):
        opt.step()
        assert_in_range(opt, calls)
        assert calls[-1][0].step == t and isinstance(calls[-1][0], ctypes.Structure)
    other = optim.AdamW([parameter(p.numel()) for p in params], state_bits=bits)
    other.load_state_dict(opt.state_dict())
    other.step()
    assert_in_range(other, calls)
    assert calls[-1][0].step == 3


def test_step_hooks_are_called_as_torch_calls_them(calls):
    """Global and own hooks, in torch's order, with the step's arguments; as for one of torch's own optimisers."""
    from torch.optim.optimizer import register_optimizer_step_post_hook, register_optimizer_step_pre_hook

    def run(make):
        seen = []

        def note(name):
            return lambda o, args, kwargs: seen.append((name, args[1:] == (closure,) or kwargs == {"closure": closure}))

        def closure():
            seen.append("closure")
            return torch.tensor(2.0)

        p = parameter()
        opt = make([p])
        handles = [register_optimizer_step_pre_hook(note("global before")),
                   register_optimizer_step_post_hook(note("global after")),
                   opt.register_step_pre_hook(note("before")), opt.register_step_post_hook(note("after"))]
        try:
            assert float(opt.step(closure)) == 2.0
            opt.step()
        finally:
            for h in handles:
                h.remove()
        opt.step()
        return seen

    got = run(optim.AdamW)
    assert got == run(lambda params: torch.optim.SGD(params, lr=0.1))
    assert len(got) == 9 and got[2] == "closure" and all(e[1] for e in got[:5] if e != "closure")
    assert len(calls) == 3


def test_a_hook_may_replace_the_closure(calls):
    opt = optim.AdamW([parameter()])

    def other(o, args, kwargs):
        return (o, lambda: torch.tensor(5.0)), {}

    handle = opt.register_step_pre_hook(other)
    assert float(opt.step(lambda: torch.tensor(2.0))) == 5.0
    handle.remove()
    assert float(opt.step(lambda: torch.tensor(2.0))) == 2.0 and opt.step() is None


def test_a_profile_shows_the_step(calls):
    opt = optim.AdamW([parameter()])
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CPU]) as prof:
        opt.step()
    assert any("Optimizer.step#AdamW" in e.key for e in prof.key_averages())


def test_load_hooks_see_and_change_what_is_loaded(calls):
    a = optim.AdamW([parameter(300)], state_bits=8)
    a.step()
    p = parameter(300)
    b = optim.AdamW([p], state_bits=8)
    seen = []

    def before(o, state_dict):   # what a hook returns is loaded in its place
        changed = {**state_dict, "state": {0: {**state_dict["state"][0], "step": 41}}}
        changed["state"][0]["exp_avg_scale"] = torch.full((2,), 0.5)
        return changed

    def after(o):                # the moments are in place, in their types, and may be changed
        seen.append((o.state[p]["step"], o.state[p]["exp_avg"].dtype))
        o.state[p]["exp_avg_sq_root_scale"].fill_(0.25)

    b.register_load_state_dict_pre_hook(before)
    b.register_load_state_dict_post_hook(after)
    b.load_state_dict(a.state_dict())
    assert seen == [(41, torch.float8_e4m3fn)]
    assert bool((b.state[p]["exp_avg_scale"] == 0.5).all()) and bool((b.state[p]["exp_avg_sq_root_scale"] == 0.25).all())
    assert a.state_dict()["state"][0]["step"] == 1   # the caller's own stays
    b.step()
    assert_in_range(b, calls)
    assert calls[-1][0].step == 42


def test_saved_and_copied_optimisers_keep_their_moments(calls):
    import copy
    import io
    a = optim.AdamW([parameter(300)], state_bits=8)
    a.step()
    file = io.BytesIO()
    torch.save(a, file)
    file.seek(0)
    for b in (copy.deepcopy(a), torch.load(file, weights_only=False)):
        q = b.param_groups[0]["params"][0]
        q.grad = torch.ones(300)
        b.step()
        assert_in_range(b, calls)
        assert b.state[q]["step"] == 2 and b.state[q]["exp_avg"].dtype is torch.float8_e4m3fn
