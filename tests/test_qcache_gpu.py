"""The 8-bit latent cache on B200: rows as written and as read back, bit for bit against the
definition in float64, and the padded, listed and out-of-range forms."""
import math

import pytest
import torch

from tests.qcache_cases import code_values, dequantised, quantise_latent, quantise_rows

pytestmark = pytest.mark.gpu

dsa = pytest.importorskip("sparse_attention_long_indexer_b200")

DIMS = {"prod": dict(idx_dim=128, d_latent=512, d_rope=64), "tiny": dict(idx_dim=32, d_latent=64, d_rope=16),
        "odd": dict(idx_dim=80, d_latent=336, d_rope=24), "least": dict(idx_dim=16, d_latent=16, d_rope=0)}


def _dims(name, batch, n, max_len):
    return dsa.make_dims(batch, n, max_len, **DIMS[name])


def _rows(seed, *shape):
    """bf16 rows whose magnitudes range over the whole of bf16, with zeros, subnormals and exact ties."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g, dtype=torch.float64)
    r = torch.randint(-12, 12, shape[:-1], generator=g).double()
    x = (x * torch.exp2(r)[..., None]).to(torch.bfloat16)
    flat = x.view(-1, shape[-1])
    n = flat.shape[0]
    if n > 1:
        flat[1] = 0
    if n > 2:
        flat[2] = (torch.arange(shape[-1]) % 97 - 48).to(torch.bfloat16) * 2.0 ** -133    # subnormal
    if n > 3:
        flat[3] = 3.0e38
    if n > 4:                                   # amax on the border of two scales, codes on ties
        flat[4] = (torch.arange(shape[-1]) % 57).to(torch.bfloat16) * 8
    if n > 5:
        flat[5] = flat[5].float().clamp(-2, 2).to(torch.bfloat16) * 2.0 ** -110
    return x


def _check_rows(dims, cache, at, latent, keys):
    """Cache rows at index tuple `at` hold the quantised latent and key rows."""
    codes, scales = quantise_latent(latent, dims.d_latent)
    assert torch.equal(code_values(cache.codes[at].cpu()), codes)
    assert torch.equal(cache.scales[at].cpu().double(), scales)
    assert torch.equal(cache.rope[at].cpu(), latent[..., dims.d_latent:])
    kq, ke = quantise_rows(keys.double())
    assert torch.equal(code_values(cache.k_idx[at].cpu()), kq)
    assert torch.equal(cache.k_scale[at].cpu().double(), torch.exp2(ke.double()))


@pytest.mark.parametrize("name", list(DIMS))
@pytest.mark.parametrize("batch,n", [(1, 1), (3, 7), (1, 129), (64, 1)])
def test_written_rows_are_the_definition_and_read_back_exactly(name, batch, n):
    dims = _dims(name, batch, n, n + 5)
    ws = dsa.Workspace.create_qcache(dims, 1)
    cache = dsa.QCache.create(dims)
    latent = _rows(1, batch, n, dims.d_latent + dims.d_rope)
    keys = _rows(2, batch, n, dims.idx_dim)
    start = torch.tensor([b % 6 for b in range(batch)], dtype=torch.int32)
    dsa.qcache_write(dims, cache, latent.cuda(), keys.cuda(), ws, start=start.cuda())
    back = dsa.qcache_read(dims, cache, ws, start=start.cuda())
    ws.check()
    for b in range(batch):
        at = (b, slice(int(start[b]), int(start[b]) + n))
        _check_rows(dims, cache, at, latent[b], keys[b])
        want = dequantised(cache.codes[at].cpu(), cache.scales[at].cpu(), cache.rope[at].cpu())
        assert torch.equal(back[b].cpu().double(), want)


def test_every_code_at_every_scale_reads_exactly():
    exps = list(range(-100, 101))
    dims = dsa.make_dims(1, len(exps), len(exps), idx_dim=128, d_latent=512, d_rope=8)
    ws = dsa.Workspace.create_qcache(dims, 1)
    cache = dsa.QCache.create(dims)
    codes = torch.arange(512, dtype=torch.int64) % 256
    codes[(codes & 127) == 127] = 0                          # E4M3's NaN is not a code of a cache
    cache.codes[:] = codes.to(torch.uint8).cuda()
    cache.scales[:] = torch.exp2(torch.tensor(exps, dtype=torch.float64)).float().view(1, -1, 1).cuda()
    back = dsa.qcache_read(dims, cache, ws).cpu().double()[0, :, :512]
    want = code_values(codes.to(torch.uint8))[None, :] * torch.exp2(torch.tensor(exps).double())[:, None]
    # 480 is no code, so the largest value is 448 * 2^100, a bf16; the least is 2^-109, a bf16
    assert torch.equal(back, want)


def test_infinities_saturate_and_nan_marks_its_group():
    dims = _dims("prod", 1, 4, 4)
    ws = dsa.Workspace.create_qcache(dims, 1)
    cache = dsa.QCache.create(dims)
    latent = _rows(3, 1, 4, 576)
    latent[0] = latent[0].float().clamp(-3, 3).to(torch.bfloat16)
    keys = torch.randn((1, 4, 128)).to(torch.bfloat16)
    latent[0, 0, 5] = math.inf
    latent[0, 1, 130] = -math.inf
    latent[0, 2, 300] = math.nan
    latent[0, 3, 128:256] = math.inf                        # a group without a finite value
    keys[0, 0, 3], keys[0, 1, 7], keys[0, 2, :] = math.inf, math.nan, -math.inf
    dsa.qcache_write(dims, cache, latent.cuda(), keys.cuda(), ws)
    back = dsa.qcache_read(dims, cache, ws).cpu().double()[0]
    ws.check()
    scales = cache.scales.cpu().double()[0]
    codes, want = quantise_latent(latent[0], 512)
    assert torch.equal(torch.isnan(scales), torch.isnan(want)) and torch.isnan(scales).sum() == 1
    f = torch.isfinite(want)
    assert torch.equal(scales[f], want[f])
    assert back[0, 5] == 448 * want[0, 0] and back[1, 130] == -448 * want[1, 1]
    assert torch.isnan(back[2, 256:384]).all() and torch.isfinite(back[2, :256]).all()
    assert (back[3, 128:256] == 448).all()
    kv = code_values(cache.k_idx.cpu())[0]
    assert kv[0, 3] == 448 and torch.isnan(kv[1, 7]) and torch.isfinite(kv[1, :7]).all() and (kv[2] == -448).all()
    assert torch.isfinite(cache.k_scale).all()


def test_padded_batches_leave_other_rows_as_they_were():
    batch, n, max_len = 4, 9, 20
    dims = _dims("prod", batch, n, max_len)
    ws = dsa.Workspace.create_qcache(dims, 1)
    cache = dsa.QCache.create(dims)
    for t in (cache.codes, cache.k_idx):
        t.fill_(0x55)
    cache.scales.fill_(7), cache.rope.fill_(3), cache.k_scale.fill_(5)
    before = {k: getattr(cache, k).clone() for k in ("codes", "scales", "rope", "k_idx", "k_scale")}
    latent, keys = _rows(4, batch, n, 576), _rows(5, batch, n, 128)
    # right-padded, full, left-padded (negative start), none of its rows
    start = torch.tensor([0, 11, -4, 6], dtype=torch.int32)
    lengths = torch.tensor([3, 20, 5, 6], dtype=torch.int32)
    dsa.qcache_write(dims, cache, latent.cuda(), keys.cuda(), ws, start=start.cuda(), lengths=lengths.cuda())
    ws.check()
    written = torch.zeros((batch, max_len), dtype=torch.bool)
    for b in range(batch):
        for j in range(n):
            pos = int(start[b]) + j
            if 0 <= pos < int(lengths[b]):
                written[b, pos] = True
                _check_rows(dims, cache, (b, pos), latent[b, j], keys[b, j])
    assert written.sum() == 3 + 9 + 5
    for k, t in before.items():
        assert torch.equal(getattr(cache, k).cpu()[~written], t.cpu()[~written]), k
    back = dsa.qcache_read(dims, cache, ws, start=start.cuda(), lengths=lengths.cuda()).cpu()
    for b in range(batch):
        for j in range(n):
            pos = int(start[b]) + j
            if not 0 <= pos < int(lengths[b]):
                assert (back[b, j] == 0).all()


def test_listed_sources_and_positions():
    batch, n, n_src, max_len = 3, 5, 16, 40
    dims = _dims("tiny", batch, n, max_len)
    ws = dsa.Workspace.create_qcache(dims, 1)
    cache = dsa.QCache.create(dims)
    latent, keys = _rows(6, batch, n_src, 80), _rows(7, batch, n_src, 32)
    src = torch.tensor([[0, 3, 15, -1, -1], [2, 2, 2, 2, 2], [-1, 1, -1, 4, -7]], dtype=torch.int32)
    start = torch.tensor([35, 0, 8], dtype=torch.int32)
    dsa.qcache_write(dims, cache, latent.cuda(), keys.cuda(), ws, start=start.cuda(), src_rows=src.cuda())
    ws.check()
    for b in range(batch):
        for j in range(n):
            pos = int(start[b]) + j
            if src[b, j] >= 0:
                _check_rows(dims, cache, (b, pos), latent[b, src[b, j]], keys[b, src[b, j]])
            else:
                assert (cache.codes[b, pos] == 0).all() and (cache.k_scale[b, pos] == 1).all()
    rows = torch.tensor([[35, 37, -1, 35, 0], [0, 4, 39, -5, 1], [9, 9, 9, 11, 8]], dtype=torch.int32)
    back = dsa.qcache_read(dims, cache, ws, rows=rows.cuda()).cpu().double()
    want = dequantised(cache.codes.cpu(), cache.scales.cpu(), cache.rope.cpu())
    for b in range(batch):
        for j in range(n):
            r = int(rows[b, j])
            assert torch.equal(back[b, j], want[b, r] if r >= 0 else torch.zeros(80, dtype=torch.float64))


def test_either_part_alone():
    dims = _dims("odd", 2, 3, 3)
    ws = dsa.Workspace.create_qcache(dims, 1)
    latent, keys = _rows(8, 2, 3, 360), _rows(9, 2, 3, 80)
    one, two = dsa.QCache.create(dims), dsa.QCache.create(dims)
    dsa.qcache_write(dims, one, latent.cuda(), None, ws)
    assert (one.k_idx == 0).all() and (one.k_scale == 1).all()
    dsa.qcache_write(dims, two, None, keys.cuda(), ws)
    assert (two.codes == 0).all() and (two.rope == 0).all()
    both = dsa.QCache(one.codes, one.scales, one.rope, two.k_idx, two.k_scale)
    _check_rows(dims, both, (slice(None),), latent, keys)
    ws.check()


@pytest.mark.parametrize("what", ["position", "source", "listed"])
def test_out_of_range_rows_are_reported_and_skipped(what):
    dims = _dims("prod", 2, 4, 6)
    ws = dsa.Workspace.create_qcache(dims, 1)
    cache = dsa.QCache.create(dims)
    latent, keys = _rows(10, 2, 4, 576), _rows(11, 2, 4, 128)
    start = torch.tensor([0, 4 if what == "position" else 1], dtype=torch.int32).cuda()
    src = torch.tensor([[0, 1, 2, 3], [3, 4 if what == "source" else 0, 2, 2 ** 31 - 1 if what == "source" else 1]],
                       dtype=torch.int32).cuda()
    lengths = torch.tensor([6, 2 ** 31 - 1], dtype=torch.int32).cuda()
    dsa.qcache_write(dims, cache, latent.cuda(), keys.cuda(), ws, start=start, lengths=lengths, src_rows=src)
    if what == "listed":
        ws.check()
        rows = torch.tensor([[0, 6, 1, 2 ** 31 - 1], [2, -1, 3, 4]], dtype=torch.int32).cuda()
        back = dsa.qcache_read(dims, cache, ws, rows=rows)
        assert (back[0, 1] == 0).all() and (back[0, 3] == 0).all() and (back[1, 1] == 0).all()
        _same = dequantised(cache.codes.cpu(), cache.scales.cpu(), cache.rope.cpu())
        assert torch.equal(back[1, 3].cpu().double(), _same[1, 4])
    else:
        _check_rows(dims, cache, (0, slice(0, 4)), latent[0], keys[0])
        _check_rows(dims, cache, (1, 4 if what == "position" else 1), latent[1, 3], keys[1, 3])
    torch.cuda.synchronize()
    st, _ = dsa.dsa_get_device_status(ws.buf)
    assert st == dsa.DSA_ERR_INDEX_RANGE
    ws.check()                                       # reading the status cleared it


def test_rows_past_32_bit_offsets():
    max_len = 4_300_000                              # codes past 2^31 bytes
    dims = dsa.make_dims(1, 3, max_len, idx_dim=16, d_latent=512, d_rope=8)
    ws = dsa.Workspace.create_qcache(dims, 1)
    cache = dsa.QCache.create(dims)
    latent, keys = _rows(12, 1, 3, 520), _rows(13, 1, 3, 16)
    start = torch.tensor([max_len - 3], dtype=torch.int32).cuda()
    dsa.qcache_write(dims, cache, latent.cuda(), keys.cuda(), ws, start=start)
    back = dsa.qcache_read(dims, cache, ws, start=start)
    ws.check()
    at = (0, slice(max_len - 3, max_len))
    _check_rows(dims, cache, at, latent[0], keys[0])
    assert torch.equal(back[0].cpu().double(),
                       dequantised(cache.codes[at].cpu(), cache.scales[at].cpu(), cache.rope[at].cpu()))
