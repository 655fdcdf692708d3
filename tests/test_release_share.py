"""The small release's cluster: every entry has a thread and a place in its
CTA's shared memory, and none of either is left over. The constants are read
from the source."""

import os
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "paged_kv_cache_hkv_gb300", "csrc", "tables.cu")


def constants():
    with open(SRC, encoding="utf-8") as f:
        text = f.read()
    known = {}
    for name, value in re.findall(r"^constexpr (?:int|long long) (k\w+) = ([^;]+);", text, re.M):
        if re.fullmatch(r"[\w \*]+", value):
            known[name] = eval(value, {}, known)
    return known


def cluster_ctas(c, bound):
    n = 1
    while n < c["kMaxCtas"] and bound > n * c["kTableThreads"]:
        n *= 2
    return n


def shares(c, bound, total):
    n = cluster_ctas(c, bound)
    tiles = -(-total // c["kTableThreads"])
    return [max(0, min(total, tiles * (k + 1) // n * c["kTableThreads"]) -
                tiles * k // n * c["kTableThreads"]) for k in range(n)]


def test_no_share_is_larger_than_its_place_and_the_largest_fills_it():
    c = constants()
    top = c["kSmallEntries"]
    largest = 0
    for bound in list(range(1, 3000)) + list(range(3000, top + 1, 97)) + [top - 1, top]:
        for total in {0, 1, bound // 2, bound - 1, bound}:
            s = shares(c, bound, total)
            assert sum(s) == total
            largest = max(largest, max(s))
    assert largest == c["kShare"] == c["kPerThread"] * c["kTableThreads"]


def gpu_case(rows, width, seed):
    import numpy as np

    import oracle
    from table_cases import pool_state
    from test_gpu_tables import Device, binding
    B = 8
    rng = np.random.default_rng(seed)
    tokens = np.full(rows, width * B)
    if seed:  # ragged
        tokens = rng.integers(2 * B, width * B + 1, rows)
    table, ref, queue, state = pool_state(tokens, tokens, B, width=width, prefix_blocks=2,
                                          sharers=tuple(range(0, rows, 3)), seed=seed)
    order = rng.permutation(rows)
    want = oracle.release_blocks(table, order, tokens, queue, state, ref, B)
    binding.pkv_get_device_errors(clear=True)
    d = Device(table, ref, queue, state, B)
    d.release(order, tokens)
    d.check_release(want)
    assert binding.pkv_get_device_errors(clear=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("seed", [0, 1])
@pytest.mark.parametrize("rows,width", [(1, 1024), (1, 1025), (5, 205), (2, 1024), (3, 683), (8, 512),
                                        (17, 241), (8, 1024), (9, 911), (64, 256), (4096, 4),
                                        (2, 8192), (113, 145), (1, 16384), (1, 16385), (5, 3277)])
def test_releases_around_every_cluster_size(rows, width, seed):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():  # pragma: no cover - CPU containers
        pytest.skip("needs a CUDA GPU")
    gpu_case(rows, width, seed)
