"""attn_cache_reserve where rows hold one page in very many places."""
import pytest

import scaled_dot_product_16_b200 as sdpa
from tests import serving_ref as R
from tests.test_gpu_cache import dev, guarded, status

pytestmark = pytest.mark.gpu


def _reserve(table, ref, lens, new, page, want_status, want):
    t, r, c = dev(table), dev(ref), guarded((len(table), 2))
    sdpa.attn_cache_reserve(t, r, dev(lens), dev(new), c.t, B=len(table), max_pages=len(table[0]), num_pages=len(ref),
                            page_size=page)
    status(want_status)
    c.check()
    for x, y in zip((t, r, c.t), want):
        assert x.tolist() == y


@pytest.mark.parametrize("n", [8191, 8192, 8193, 9300, 16383, 16384, 16385, 20000, 32768, 40000, 65536])
@pytest.mark.parametrize("others", [0, 7], ids=["all", "held-elsewhere"])
def test_one_row_holds_a_page_many_times(n, others):
    """A row whose every entry is the same page asks for all of them: up to 8,192 the first keeps it (or none does,
    where it is held elsewhere too) and the others get pages of their own; above, the call is refused and the
    counts are as before. A second page with two holders stands beside it."""
    if n + others > 1 << 16:
        others = 0
    table = [[3] * n, [1] * 2 + [-1] * (n - 2)]
    ref = [0] * (min(n, 8193) + 12)
    ref[3], ref[1] = n + others, 2
    lens, new = [n, 2], [n, 2]
    if n <= 8192:
        _reserve(table, ref, lens, new, 1, 0, R.reserve(table, ref, lens, new, 1))
    else:
        _reserve(table, ref, lens, new, 1, sdpa.ATTN_ERR_DATA, (table, ref, [[-1, -1]] * 2))


def test_many_rows_hold_a_page_many_times():
    """The holders of a page are spread over 600 rows of 30 entries: 18,000 ask."""
    table, ref = [[5] * 30 for _ in range(600)], [0] * 20000
    ref[5] = 18000
    _reserve(table, ref, [30] * 600, [30] * 600, 1, sdpa.ATTN_ERR_DATA, (table, ref, [[-1, -1]] * 600))
    _reserve(table, ref, [30] * 600, [10] * 600, 1, 0, R.reserve(table, ref, [30] * 600, [10] * 600, 1))
