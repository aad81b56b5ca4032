"""attn_cache_reserve of more than 1,024 pages from pools of several steps of its walk (8,192 pages each): free pages
lie partly in the first step and partly in later ones, and many rows need none."""
import numpy as np
import pytest

from tests.test_gpu_cache import _reserve

pytestmark = pytest.mark.gpu


def test_the_last_page_lies_behind_the_first_step_of_the_walk():
    """1,023 pages are handed out by the second block of 1,024 slots, from what is left of the pool's first 8,192; the
    one slot after them takes the first page behind those."""
    n = 2 * 1024 - 1
    table = [[-1] * n, [8200, 8200] + [-1] * (n - 2)]     # row 1: both its slots ask, the first keeps the page
    ref = [0] * 2047 + [1] * (8192 - 2047) + [0] * 20
    ref[8200] = 2
    _reserve(table, ref, [n, 2], [n, 2], 1)


@pytest.mark.parametrize("seed", range(24))
def test_rows_that_need_pages_and_rows_that_do_not(seed):
    rng = np.random.default_rng(seed)
    rows, page, num = 8000, 4, 40000
    before = [int(rng.integers(0, 3)) * page + int(rng.integers(0, page)) for _ in range(rows)]
    new = [int(rng.choice([0, 1, 1, 1, 6], p=[0.1, 0.29, 0.29, 0.29, 0.03])) for _ in range(rows)]
    held = [-(-n // page) for n in before]
    first = int(rng.integers(300, 2400))                  # free pages among the first 8,192
    free = sorted(int(x) for x in rng.permutation(8192)[:first]) + list(range(16384 + int(rng.integers(0, 99)), num, 2))
    ref = [1] * num
    for p in free:
        ref[p] = 0
    used = iter([p for p in range(num) if ref[p]])
    table = [[next(used) for _ in range(h)] + [-1] * (6 - h) for h in held]
    _reserve(table, ref, [a + b for a, b in zip(before, new)], new, page)
