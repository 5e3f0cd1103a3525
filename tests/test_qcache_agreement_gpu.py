"""The attention over an 8-bit cache and the one over a bf16 cache on the same rows (the 8-bit cache read back): each
element within both kernels' bounds of the other and of the float64 result."""
import pytest
import torch

from tests.qcache_cases import attend, check

pytestmark = pytest.mark.gpu

dsa = pytest.importorskip("sparse_attention_long_indexer_b200")


@pytest.mark.parametrize("n,topk", [(1, 2048), (90, 700)])
def test_both_kernels_are_within_their_bounds_of_each_other(n, topk):
    g = torch.Generator().manual_seed(95)
    cap = 3000
    dims, full = dsa.make_dims(1, n, cap), dsa.make_dims(1, cap, cap)
    ws, ws16 = dsa.Workspace.create_qcache(dims, topk), dsa.Workspace.create(dims, topk)
    cache = dsa.QCache.create(dims)
    dsa.qcache_write(full, cache, torch.randn((1, cap, 576), generator=g).to(torch.bfloat16).cuda(), None, ws)
    kv = dsa.qcache_read(full, cache, ws)
    q = torch.randn((1, n, 128, 576), generator=g).to(torch.bfloat16).cuda()
    idx = torch.randint(0, cap, (1, n, topk), generator=g, dtype=torch.int32)
    idx[0, ::7, topk // 2:] = -1
    out, lse = dsa.sparse_mla_attn_qcache(dims, q, cache, idx.cuda(), topk, ws)
    o16, l16 = dsa.sparse_mla_attn(dims, q, kv, idx.cuda(), topk, ws16)
    ws.check(), ws16.check()
    for i in range(0, n, 6):
        at = idx[0, i][idx[0, i] >= 0].long()
        ref = attend(q[0, i].double().cpu(), kv[0].cpu()[at].double(), 512, dims.softmax_scale)
        check(out[0, i], lse[0, i], ref)
        # lse of the bf16 kernel is the logarithm of the sum of the weights as rounded to bf16, each off by at most 2^-8
        # of itself, and so their sum: -ln(1 - 2^-8) < 2^-8 + 2^-16
        slack16 = 2.0 ** -8 + 2.0 ** -16
        check(o16[0, i], l16[0, i], (*ref[:3], ref[3] + slack16))
        assert ((out[0, i].double() - o16[0, i].double()).abs().cpu() <= 2 * ref[2]).all()
        assert ((lse[0, i].double() - l16[0, i].double()).abs().cpu() <= 2 * ref[3] + slack16).all()
        assert ref[2].max() <= 0.02                    # the bound itself says something: outputs are up to 0.5
