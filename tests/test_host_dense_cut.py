"""The choice of the dense layer's kernels, compiled for the host: the sizes that the GPU tests run reach every one of them."""
import random

import pytest

import dense_cut
from test_gpu_dense_tiles import SMALL, TILES


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    return dense_cut.compile_choice(str(tmp_path_factory.mktemp("choice")))


def drawn(rng):
    """Sizes over the whole range, logarithmically, aligned and not."""
    while True:
        M, K, N = (round(2 ** rng.uniform(0, hi)) for hi in (14.3, 13.2, 13.2))
        if M * K * N <= 1.5e11:
            break
    if rng.random() < 0.4:
        M, K, N = (max(8, v // 8 * 8) for v in (M, K, N))
    return (rng.choice(("fp32", "bf16")), M, K, N, *rng.choice(((0, 0), (0, 0), (0, 8), (1, 3), (2, 1))))


def kernels(choice, case, act=True):
    dtype, M, K, N, offset, gap = case
    return dense_cut.describe(choice, M, K, N, dtype, offset, gap, act)


def test_tested_sizes_reach_every_kernel_that_sizes_reach(choice):
    tested = set().union(*(kernels(choice, c) for c in TILES))
    rng, reached = random.Random(5), {}
    for _ in range(20000):
        case, act = drawn(rng), rng.random() < 0.7
        for name in kernels(choice, case, act):
            reached.setdefault(name, case)
    missing = {name: case for name, case in reached.items() if name not in tested}
    assert not missing
    assert len(tested) > 60   # three families of tiles, small products, copies


def test_small_ones_are_small(choice):
    for case in SMALL:
        dtype = case[0]
        assert any(name.startswith(f"small gradients {dtype}") for name in kernels(choice, case)), case


@pytest.mark.parametrize("case,name", [(("bf16", 2048, 2048, 2048, 0, 0), "direct bf16 128x128 rows rows"),
                                       (("bf16", 8192, 4096, 4096, 0, 0), "direct bf16 256x256 rows cols"),
                                       (("fp32", 997, 1531, 803, 0, 0), "staged fp32 128x128 rows rows split"),
                                       (("fp32", 1, 64, 4, 0, 0), "small forward fp32 fi=1")])
def test_named_choices(choice, case, name):
    assert name in kernels(choice, case)
