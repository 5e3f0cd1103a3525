"""Calls whose queries are split into ranges and joined, one behind the other on one workspace: the join of a
call is set up while its ranges still run, and has to read what they write, not what an earlier call left."""
import pytest
import torch

from tests.qcache_cases import attend, check, dequantised

pytestmark = pytest.mark.gpu

dsa = pytest.importorskip("sparse_attention_long_indexer_b200")


@pytest.mark.parametrize("n,topk,heads,d_latent,d_rope", [(1, 2048, 128, 512, 64), (5, 1024, 128, 512, 64),
                                                          (3, 512, 8, 64, 16), (20, 640, 37, 336, 24)])
def test_joins_of_calls_in_a_row_read_their_own_ranges(n, topk, heads, d_latent, d_rope):
    g = torch.Generator().manual_seed(70)
    dims = dsa.make_dims(1, n, 4096, n_heads=heads, d_latent=d_latent, d_rope=d_rope)
    cache = dsa.QCache.create(dims)
    codes = (torch.randn(cache.codes.shape, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    cache.codes.copy_(codes.view(torch.uint8))
    cache.scales.copy_(torch.exp2(torch.randint(-9, -5, cache.scales.shape, generator=g).float()))
    cache.rope.copy_(torch.randn(cache.rope.shape, generator=g).to(torch.bfloat16))
    ws = dsa.Workspace.create_qcache(dims, topk)
    calls = []
    for c in range(6):
        q = torch.randn((1, n, heads, d_latent + d_rope), generator=g).to(torch.bfloat16).cuda()
        idx = torch.randint(0, 4096, (1, n, topk), generator=g, dtype=torch.int32)
        if c % 3 == 1:
            idx[..., topk // 3:] = -1                  # ranges without a row, whose outputs are not written
        if c % 3 == 2:
            idx[:, n // 2] = -1                        # a query without a row
        calls.append((q, idx.cuda()))
    alone = []
    for q, idx in calls:
        ws.buf[256:].fill_(0x7F)                       # what an early read would find: huge numbers
        alone.append(dsa.sparse_mla_attn_qcache(dims, q, cache, idx, topk, ws))
        torch.cuda.synchronize()
    for i, ((q, idx), (out, lse)) in enumerate(zip(calls, alone)):
        row = idx[0, n // 2][idx[0, n // 2] >= 0].long()
        rows = dequantised(cache.codes[0, row].cpu(), cache.scales[0, row].cpu(), cache.rope[0, row].cpu())
        check(out[0, n // 2], lse[0, n // 2], attend(q[0, n // 2].double().cpu(), rows, d_latent, dims.softmax_scale))
    got = [dsa.sparse_mla_attn_qcache(dims, *calls[k % 6][:1], cache, calls[k % 6][1], topk, ws) for k in range(60)]
    ws.check()
    for k, (out, lse) in enumerate(got):
        assert torch.equal(out, alone[k % 6][0]) and torch.equal(lse, alone[k % 6][1])
