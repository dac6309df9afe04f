"""The dense layer's bounds tell the library's precision from a lower one: mistakes planted in the reference exceed them.

The reference's own values stand in for the library's, rounded as it rounds them."""
import pytest

torch = pytest.importorskip("torch")

from dense_reference import TYPES, excess, expect, make  # noqa: E402
from test_gpu_dense_tiles import SMALL  # noqa: E402


def to_bf16(t):
    return t.to(torch.bfloat16).double()


def outputs(d, dtype, act, **kw):
    dt = TYPES[dtype][0]
    return {k: v.to(torch.float32 if k == "z" else dt) for k, (v, _) in expect(d, dtype, act, 1.0, True, **kw).items()}


@pytest.mark.parametrize("act", ["gelu", "silu", "tanh", "sigmoid"])
@pytest.mark.parametrize("case", [("bf16", 96, 80, 72, 0, 0), ("bf16", 64, 12, 64, 0, 0)])
def test_z_held_in_bf16_is_noticed(case, act):
    assert case in SMALL
    dtype, M, K, N, _, _ = case
    d = make(M, K, N, dtype, 11, device="cpu")
    want = expect(d, dtype, act, 1.0, True)
    assert all(excess(v, want[k]) <= 0 for k, v in outputs(d, dtype, act).items())
    got = outputs(d, dtype, act, held=to_bf16)
    assert any(excess(got[k], want[k]) > 0 for k in ("dx", "dw", "db"))
    assert excess(to_bf16(want["z"][0]), want["z"]) > 0


# Short sums: the bound of z grows with K, and over 1,959 terms it is wider than dz's rounding.
@pytest.mark.parametrize("case", [c for c in SMALL if c[0] == "bf16" and min(c[1:4]) >= 12 and c[2] <= 100])
def test_dz_rounded_on_the_way_to_a_small_gradient_is_noticed(case):
    dtype, M, K, N, _, _ = case
    d = make(M, K, N, dtype, 12, device="cpu")
    want = expect(d, dtype, "tanh", 1.0, True)
    dz = d["dy"].double() * (1 - torch.tanh(want["z"][0]) ** 2)
    for rounded, over in ((dz, False), (to_bf16(dz), True)):
        got = {"dx": rounded @ d["w"].double(), "dw": rounded.t() @ d["x"].double()}
        assert any(excess(v.to(torch.bfloat16), want[k]) > 0 for k, v in got.items()) == over
