"""Attention over rows of the largest magnitude that the 8-bit cache holds (448 * 2^100), with logits that rise from
block to block by less than the running maximum's slack: the unnormalised sums have to stay finite."""
import pytest
import torch

from tests.qcache_cases import attend, check, dequantised

pytestmark = pytest.mark.gpu

dsa = pytest.importorskip("sparse_attention_long_indexer_b200")

TOP = 0x7E                                             # E4M3's 448
LOG2E = 1.4426950408889634


def _cache(max_len, rise):
    """Every code 448 at scale 2^100; the RoPE part's first dim makes position s's log2 logit rise * (s // 64 % 2)
    for q = 1 there (softmax_scale 1), and the latents carry no weight in the logits (q = 0 there)."""
    dims = dict(n_heads=128, d_latent=512, d_rope=64, softmax_scale=1.0)
    cache = dsa.QCache.create(dsa.make_dims(1, 1, max_len, **dims))
    cache.codes.fill_(TOP)
    cache.scales.fill_(2.0 ** 100)
    step = (torch.arange(max_len) // 64 % 2).float() * (rise / LOG2E)
    cache.rope[0, :, 0] = step.to(torch.bfloat16).cuda()
    return dims, cache


def _rows(cache, at):
    return dequantised(cache.codes[0, at].cpu(), cache.scales[0, at].cpu(), cache.rope[0, at].cpu())


# one pair walks two blocks (one query of 128 rows), 32 blocks (more queries than pairs), or two of a range
@pytest.mark.parametrize("rise", [2.0, 6.5, 7.5, 15.0, 30.0, 31.5, 100.0])
@pytest.mark.parametrize("n,topk", [(1, 128), (1, 2048), (150, 2048)])
def test_the_largest_rows_give_finite_outputs(n, topk, rise):
    kw, cache = _cache(2048, rise)
    dims = dsa.make_dims(1, n, 2048, **kw)
    q = torch.zeros((1, n, 128, 576), dtype=torch.bfloat16)
    q[..., 512] = torch.linspace(0.25, 1, 128).to(torch.bfloat16)
    idx = torch.arange(topk, dtype=torch.int32).expand(1, n, topk).contiguous()
    ws = dsa.Workspace.create_qcache(dims, topk)
    out, lse = dsa.sparse_mla_attn_qcache(dims, q.cuda(), cache, idx.cuda(), topk, ws)
    ws.check()
    ref = attend(q[0, 0].double(), _rows(cache, idx[0, 0].long().cuda()), 512, 1.0)
    for i in {0, n // 2, n - 1}:
        check(out[0, i], lse[0, i], ref)


@pytest.mark.parametrize("quant", [True, False])
@pytest.mark.parametrize("rise", [6.5, 30.0])
def test_the_largest_rows_of_a_tree_give_finite_outputs(quant, rise):
    n, topk = 256, 2048
    kw, cache = _cache(2048, rise)
    dims = dsa.make_dims(1, n, 2048, **kw)
    ctx = cache if quant else _rows(cache, torch.arange(2048).cuda()).to(torch.bfloat16)[None].cuda()
    draft = torch.zeros((1, n, 576), dtype=torch.bfloat16)
    draft[..., :512] = 448.0 * 2.0 ** 100
    draft[..., 512] = rise / LOG2E
    parents = torch.arange(-1, n - 1, dtype=torch.int32).view(1, n)
    q = torch.zeros((1, n, 128, 576), dtype=torch.bfloat16)
    q[..., 512] = torch.linspace(0.25, 1, 128).to(torch.bfloat16)
    idx = torch.arange(topk, dtype=torch.int32).expand(1, n, topk).contiguous()
    ws = dsa.Workspace.create_qcache(dims, topk)
    out, lse = dsa.tree_mla_attn(dims, q.cuda(), ctx, idx.cuda(), topk, draft.cuda(), parents.cuda(), ws)
    ws.check()
    rows = _rows(cache, torch.arange(topk).cuda())
    for i in (0, 64, n - 1):
        check(out[0, i], lse[0, i], attend(q[0, i].double(), torch.cat([rows, draft[0, :i + 1].double()]), 512, 1.0))
