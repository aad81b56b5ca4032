"""The float32 forward at head sizes that its copies treat differently, and at the largest grid."""
import pytest
import torch

import scaled_dot_product_16_b200 as sdpa
from scaled_dot_product_16_b200 import workloads as W
from tests import gpu_util as G
from tests import serving_ref as R

pytestmark = pytest.mark.gpu

F32 = torch.float32


@pytest.mark.parametrize("Dv", [1, 3, 4, 8, 9, 0], ids=lambda x: f"Dv{x}" if x else "Dv=D")
@pytest.mark.parametrize("D", [1, 2, 3, 4, 5, 7, 8, 9, 12, 31, 32, 33])
def test_small_head_sizes(D, Dv):
    """Rows of up to 8 columns are copied together, of 9 and more one by one, whole 16-byte chunks in bulk; the value
    head size takes its own way. Both layouts, a last query and key tile that are not full, NaN behind them."""
    Dv = Dv or D
    if Dv > D:
        pytest.skip("value head sizes end at the query's")
    B, Nq, Nkv, Sq, Skv = 2, 4, 2, 45, 77
    q, k, v = W.randn((B, Nq, Sq, D), 1), W.randn((B, Nkv, Skv, D), 2), W.randn((B, Nkv, Skv, Dv), 3)
    scale = D ** -0.5
    seen = torch.ones((Sq, Skv), dtype=torch.bool)
    want = torch.stack([torch.stack([R.attend(q[b, h], k[b, h // 2], v[b, h // 2], seen, scale)[0] for h in range(Nq)])
                        for b in range(B)])
    bhsd = dict(B=B, Sq=Sq, Skv=Skv, layout=W.BHSD)
    cu = [torch.tensor([n, 2 * n], dtype=torch.int32, device="cuda") for n in (Sq, Skv)]
    tnd = dict(B=B, Sq=B * Sq, Skv=B * Skv, layout=W.TND, cu_seqlens_q=cu[0], cu_seqlens_kv=cu[1])

    def padded(x):  # NaN around the tensor
        room = torch.full((x.numel() + 512,), float("nan"), device="cuda")
        t = room[256:256 + x.numel()].view(x.shape)
        t.copy_(x)
        return t

    for kw in (bhsd, tnd):
        flat = (lambda x: x) if kw["layout"] == W.BHSD else (lambda x: x.transpose(1, 2).reshape(-1, x.shape[1], x.shape[3]))
        out = G.Guarded(tuple(flat(want).shape), F32)
        sdpa.attn_fwd_masked(padded(flat(q)), padded(flat(k)), padded(flat(v)), Nq=Nq, Nkv=Nkv, Dqk=D, Dv=Dv, scale=scale,
                             mask_mode=W.MASK_NONE, dtype=W.F32, out=out.t, **kw)
        assert sdpa.attn_get_last_error() == 0
        out.check()
        G.check_out(G.f64(out.t.cpu()), flat(want).numpy(), W.F32)


def test_more_blocks_than_one_grid_holds():
    """2^23 + 3 sequences of one query with 256 heads of one column are more than 2^31 - 1 blocks; without keys each
    of them only writes its output, 0."""
    B, Nq = 2 ** 23 + 3, 256
    free, _ = torch.cuda.mem_get_info()
    if free < 20 << 30:
        pytest.skip("needs 18 GB")
    q = torch.ones((B, Nq, 1, 1), device="cuda")
    out = torch.full_like(q, -1.0)
    sdpa.attn_fwd(q, None, None, B=B, Sq=1, Skv=0, Nq=Nq, Nkv=1, D=1, scale=1.0, mask_mode=W.MASK_NONE, dtype=W.F32,
                  layout=W.BHSD, out=out)
    assert sdpa.attn_get_last_error() == 0
    assert not out.any()
