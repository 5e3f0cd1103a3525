"""More rows in a call than the cache holds (gathers of many queries' selections, padded writes), and very long caches."""
import pytest
import torch

from tests.qcache_cases import attend, check, code_values, dequantised, quantise_latent

pytestmark = pytest.mark.gpu

dsa = pytest.importorskip("sparse_attention_long_indexer_b200")


@pytest.mark.parametrize("batch,max_len,n", [(1, 100, 8 * 2048), (3, 7, 50), (2, 1, 33)])
def test_a_listed_read_of_more_rows_than_the_cache_holds(batch, max_len, n):
    g = torch.Generator().manual_seed(90)
    dims = dsa.make_dims(batch, n, max_len)
    ws = dsa.Workspace.create_qcache(dsa.make_dims(batch, 1, max_len), 1)
    cache = dsa.QCache.create(dims)
    latent = torch.randn((batch, max_len, 576), generator=g).to(torch.bfloat16).cuda()
    dsa.qcache_write(dsa.make_dims(batch, max_len, max_len), cache, latent, None, ws)
    rows = torch.randint(-2, max_len, (batch, n), generator=g, dtype=torch.int32)
    back = dsa.qcache_read(dims, cache, ws, rows=rows.cuda()).cpu().double()
    ws.check()
    want = dequantised(cache.codes.cpu(), cache.scales.cpu(), cache.rope.cpu())
    for b in range(batch):
        keep = (rows[b] >= 0)[:, None]
        assert torch.equal(back[b], torch.where(keep, want[b][rows[b].clamp(min=0).long()], torch.zeros(576).double()))


def test_a_padded_write_and_read_of_more_rows_than_the_cache_holds():
    batch, max_len, n = 3, 6, 20
    g = torch.Generator().manual_seed(91)
    dims = dsa.make_dims(batch, n, max_len)
    ws = dsa.Workspace.create_qcache(dsa.make_dims(batch, 1, max_len), 1)
    cache = dsa.QCache.create(dims)
    latent, keys = (torch.randn((batch, n, w), generator=g).to(torch.bfloat16) for w in (576, 128))
    start = torch.tensor([0, -16, 3], dtype=torch.int32)
    lengths = torch.tensor([6, 4, 5], dtype=torch.int32)
    dsa.qcache_write(dims, cache, latent.cuda(), keys.cuda(), ws, start=start.cuda(), lengths=lengths.cuda())
    back = dsa.qcache_read(dims, cache, ws, start=start.cuda(), lengths=lengths.cuda()).cpu().double()
    ws.check()
    for b in range(batch):
        for j in range(n):
            pos = int(start[b]) + j
            if not 0 <= pos < int(lengths[b]):
                assert (back[b, j] == 0).all()
                continue
            codes, scales = quantise_latent(latent[b, j], 512)
            assert torch.equal(code_values(cache.codes[b, pos].cpu()), codes)
            assert torch.equal(cache.scales[b, pos].cpu().double(), scales)
            assert torch.equal(back[b, j], dequantised(cache.codes[b, pos].cpu(), cache.scales[b, pos].cpu(),
                                                       cache.rope[b, pos].cpu()))
    # without lengths the rows past the end are reported and skipped
    dsa.qcache_write(dims, cache, latent.cuda(), None, ws)
    torch.cuda.synchronize()
    assert dsa.dsa_get_device_status(ws.buf)[0] == dsa.DSA_ERR_INDEX_RANGE


def test_the_attention_over_a_cache_longer_than_a_decode_selection():
    cap, topk = 20_000_000, 130
    g = torch.Generator().manual_seed(92)
    dims = dsa.make_dims(1, 1, cap, n_heads=2, d_latent=16, d_rope=8, idx_dim=16)
    ws = dsa.Workspace.create_qcache(dims, topk)
    cache = dsa.QCache.create(dims)
    at = torch.cat([torch.randint(0, cap, (topk - 2,), generator=g), torch.tensor([0, cap - 1])])
    cache.codes[0, at.cuda()] = torch.randint(0, 120, (topk, 16), generator=g).to(torch.uint8).cuda()
    cache.scales[0, at.cuda()] = 2.0 ** -6
    cache.rope[0, at.cuda()] = torch.randn((topk, 8), generator=g).to(torch.bfloat16).cuda()
    q = torch.randn((1, 1, 2, 24), generator=g).to(torch.bfloat16)
    out, lse = dsa.sparse_mla_attn_qcache(dims, q.cuda(), cache, at.to(torch.int32).view(1, 1, -1).cuda(), topk, ws)
    ws.check()
    rows = dequantised(cache.codes[0, at.cuda()].cpu(), cache.scales[0, at.cuda()].cpu(), cache.rope[0, at.cuda()].cpu())
    check(out[0, 0], lse[0, 0], attend(q[0, 0].double(), rows, 16, dims.softmax_scale))
