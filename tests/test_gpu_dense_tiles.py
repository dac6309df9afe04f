"""Every kernel that the dense layer's choice can take, against the 64-bit definition.

TILES is chosen so that its training steps run each tile, layout pair, split and LDS form of every kernel family; a host
test compiles the choice and holds the list to that (test_host_dense_cut.py)."""
import pytest

from gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from dense_reference import excess, expect, make, run  # noqa: E402

# type, M, K, N, elements before the first row, elements between rows
TILES = [
    ("bf16", 1500, 1501, 1503, 0, 0), ("bf16", 2048, 2048, 2048, 0, 0), ("bf16", 1024, 4096, 1024, 0, 0),
    ("bf16", 1976, 5656, 3880, 0, 0), ("bf16", 829, 3058, 68, 0, 0), ("bf16", 1100, 1001, 1003, 0, 0),
    ("bf16", 1003, 1001, 1007, 1, 3), ("bf16", 2048, 2048, 2040, 1, 3), ("bf16", 2048, 2048, 2040, 2, 1),
    ("bf16", 16384, 2048, 2048, 0, 0), ("bf16", 16398, 162, 4870, 0, 0), ("bf16", 1, 80, 5493, 1, 3),
    ("bf16", 11634, 2, 668, 2, 1), ("bf16", 1, 7587, 1, 0, 0), ("bf16", 7688, 48, 8, 1, 3), ("bf16", 18, 1959, 423, 0, 0),
    ("bf16", 260, 3374, 1138, 0, 0), ("bf16", 88, 8624, 1736, 0, 0), ("bf16", 10327, 166, 4, 2, 1),
    ("bf16", 1176, 4567, 215, 0, 0), ("bf16", 1966, 70, 8881, 0, 0),
    ("fp32", 1100, 1001, 1003, 0, 0), ("fp32", 40, 1144, 656, 0, 0), ("fp32", 1003, 1001, 1007, 1, 3),
    ("fp32", 2048, 2048, 2040, 1, 3), ("fp32", 997, 1531, 803, 0, 0), ("fp32", 11733, 1, 1, 2, 1),
    ("fp32", 5310, 1039, 1, 0, 0), ("fp32", 70, 16, 8201, 1, 3), ("fp32", 18, 591, 8279, 0, 8),
    ("fp32", 2584, 1112, 1984, 1, 3), ("fp32", 1183, 1, 4383, 0, 0), ("fp32", 946, 2959, 1, 0, 0),
    ("fp32", 11223, 351, 1, 0, 0), ("fp32", 4119, 3089, 1, 0, 0), ("fp32", 4560, 928, 24, 0, 0), ("fp32", 16483, 1, 1, 0, 0),
]
# Gradients of small layers, formed in one launch with dz never rounded.
SMALL = [("bf16", 1, 7587, 1, 0, 0), ("bf16", 18, 1959, 423, 0, 0), ("fp32", 40, 1144, 656, 0, 0), ("fp32", 1183, 1, 4383, 0, 0),
         ("bf16", 64, 12, 64, 0, 0), ("fp32", 64, 12, 64, 0, 0), ("bf16", 96, 80, 72, 0, 0), ("bf16", 33, 65, 17, 1, 3)]


def step(case, act, seed):
    dtype, M, K, N, offset, gap = case
    say(f"[gpu] dense {M} x {K} -> {N} {dtype} {act}, offset {offset}, gap {gap}")
    d = make(M, K, N, dtype, seed, offset=offset, gap=gap)
    alpha = 1.25 if seed % 2 else -0.75
    got = run(d, dtype, act, alpha)
    for name, want in expect(d, dtype, act, alpha, case in SMALL).items():
        if name == "z":
            assert (got[name] is None) == (act == "none")
            if got[name] is None:
                continue
            assert got[name].dtype is torch.float32
        assert got[name].shape == want[0].shape and excess(got[name], want) <= 0, name
    again = run(d, dtype, act, alpha)
    assert all(a is None or torch.equal(a, again[k]) for k, a in got.items())


@pytest.mark.parametrize("k", range(len(TILES)))
def test_every_kernel(k):
    step(TILES[k], ("gelu", "silu", "tanh", "sigmoid")[k % 4], 300 + k)


@pytest.mark.parametrize("k", range(len(TILES)))
def test_every_kernel_without_activation(k):
    """dy itself is an operand, not dz from memory."""
    step(TILES[k], "none", 400 + k)


@pytest.mark.parametrize("act", ["relu", "gelu", "silu", "tanh", "sigmoid"])
@pytest.mark.parametrize("k", range(len(SMALL)))
def test_small_gradients(k, act):
    step(SMALL[k], act, 500 + k)
