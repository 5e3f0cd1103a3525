"""A workspace made for the largest batch, in calls whose batch shrinks from step to step."""
import pytest
import torch

pytestmark = pytest.mark.gpu

dsa = pytest.importorskip("sparse_attention_long_indexer_b200")


@pytest.mark.parametrize("tree,n,batches", [(False, 1, (96, 75, 64, 40, 37, 16, 8, 3, 1)), (True, 9, (10, 4, 2, 1))])
def test_calls_of_a_shrinking_batch(tree, n, batches):
    topk, cap, g = 1024, 1500, torch.Generator().manual_seed(80)
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()             # noqa: E731
    top = batches[0]
    whole = dsa.make_dims(top, n, cap)
    ws = dsa.Workspace.create_qcache(whole, topk)
    cache = dsa.QCache.create(whole)
    dsa.qcache_write(dsa.make_dims(top, cap, cap), cache, rnd(top, cap, 576), None, ws)
    q, draft = rnd(top, n, 128, 576), rnd(top, n, 576)
    idx = torch.randint(0, cap, (top, n, topk), generator=g, dtype=torch.int32).cuda()
    parents = torch.arange(-1, n - 1, dtype=torch.int32).expand(top, n).contiguous().cuda()
    for b in batches:
        dims = dsa.make_dims(b, n, cap)
        c = dsa.QCache(cache.codes[:b], cache.scales[:b], cache.rope[:b])
        args = (dims, q[:b], c, idx[:b], topk) + ((draft[:b], parents[:b]) if tree else ())
        call = dsa.tree_mla_attn if tree else dsa.sparse_mla_attn_qcache
        out, lse = call(*args, ws)
        own = dsa.Workspace.create_qcache(dims, topk)
        want = call(*args, own)
        ws.check(), own.check()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
