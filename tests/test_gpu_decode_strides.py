"""attn_decode_paged: which pages the kernels with vector loads take."""
import pytest
import torch

from tests.test_gpu_decode import F32, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,page,extra", [(20, 1, 4), (20, 7, 4), (4, 3, 4), (12, 5, 8), (100, 1, 4), (124, 3, 12)])
@pytest.mark.parametrize("heads", [(4, 1), (3, 1)])
def test_float32_pages_of_an_odd_number_of_chunks(D, page, extra, heads):
    """A page of 16-byte chunks may lie any number of them apart from the next: one with an odd number has the same
    rows as one with an even number, so the same kernel takes it, with the same bits."""
    c = Case([70, 0, 333, 2000], *heads, D, F32, page=page, seed=D + page)
    want = c.check()
    q, k, v, table, lens = c.dev()
    assert (page * D + extra) % 8 != (page * D) % 8 or extra == 8
    wide = [torch.full((c.num_pages, page * D + extra), float("nan"), device="cuda") for _ in range(2)]
    for w, x in zip(wide, (k, v)):
        w[:, :page * D] = x.view(c.num_pages, -1)
    got = c.run(args=[q, *(w[:, :page * D] for w in wide), table, lens], page_stride=page * D + extra)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
