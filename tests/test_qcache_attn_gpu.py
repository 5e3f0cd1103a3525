"""Attention over listed rows of the 8-bit cache, and of drafted trees, on B200, against float64."""
import math

import numpy as np
import pytest
import torch

from tests.qcache_cases import attend, check, dequantised, path_of

pytestmark = pytest.mark.gpu

dsa = pytest.importorskip("sparse_attention_long_indexer_b200")

DIMS = {"prod": dict(n_heads=128, d_latent=512, d_rope=64), "tiny": dict(n_heads=8, d_latent=64, d_rope=16),
        "odd": dict(n_heads=37, d_latent=336, d_rope=24), "least": dict(n_heads=1, d_latent=16, d_rope=0)}


def _setup(name, batch, n, max_len, topk, seed=0, scale=None):
    dims = dsa.make_dims(batch, n, max_len, softmax_scale=scale, **DIMS[name])
    g = torch.Generator().manual_seed(seed)
    cache = dsa.QCache.create(dims)
    codes = (torch.randn(cache.codes.shape, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    cache.codes.copy_(codes.view(torch.uint8))
    cache.scales.copy_(torch.exp2(torch.randint(-9, -5, cache.scales.shape, generator=g).float()))
    cache.rope.copy_(torch.randn(cache.rope.shape, generator=g).to(torch.bfloat16))
    q = torch.randn((batch, n, dims.n_heads, dims.d_latent + dims.d_rope), generator=g).to(torch.bfloat16)
    ws = dsa.Workspace.create_qcache(dims, topk)
    return dims, cache, q, ws


def _lists(seed, batch, n, topk, max_len):
    """Lists of every kind a row can be: full, short, with holes, leading padding, duplicates, empty."""
    r = np.random.default_rng(seed)
    idx = np.full((batch, n, topk), -1, dtype=np.int32)
    for t in range(batch * n):
        row = idx[t // n, t % n]
        kind = t % 6
        k = topk if kind in (0, 5) else int(r.integers(1, topk + 1))
        if kind == 4:
            continue                                                   # empty
        row[:k] = r.integers(0, max_len, k)
        if kind == 2:
            row[r.random(topk) < 0.5] = -1 - int(r.integers(0, 9))     # holes
        if kind == 3:
            row[:topk // 2] = -1                                       # leading padding
        if kind == 5:
            row[:] = row[0]                                            # one position, many times
    return torch.from_numpy(idx)


def _check_all(dims, out, lse, q, rows_of, queries=None):
    n = dims.n_q
    for t in (range(dims.batch * n) if queries is None else queries):
        b, i = divmod(t, n)
        check(out[b, i], lse[b, i], attend(q[b, i].double().cpu(), rows_of(b, i), dims.d_latent, dims.softmax_scale))


def _listed_rows(cache, b, idx_row, max_len):
    j = idx_row[(idx_row >= 0) & (idx_row < max_len)].long()
    at = j.to(cache.codes.device)
    return dequantised(cache.codes[b, at].cpu(), cache.scales[b, at].cpu(), cache.rope[b, at].cpu())


# ----------------------------------------------------------------------------- listed rows
@pytest.mark.parametrize("name,batch,n,max_len,topk", [
    ("prod", 1, 1, 1, 1), ("prod", 1, 1, 300, 64), ("prod", 1, 1, 5000, 2048), ("prod", 3, 1, 700, 65),
    ("prod", 2, 6, 900, 130), ("prod", 64, 1, 400, 320), ("prod", 1, 160, 500, 77), ("tiny", 1, 12, 90, 63),
    ("odd", 2, 7, 301, 257), ("least", 1, 6, 33, 3), ("tiny", 200, 1, 64, 200)])
def test_listed_rows(name, batch, n, max_len, topk):
    n_ok = min(n, max_len)
    dims, cache, q, ws = _setup(name, batch, n_ok, max_len, topk)
    idx = _lists(1, batch, n_ok, topk, max_len)
    out, lse = dsa.sparse_mla_attn_qcache(dims, q.cuda(), cache, idx.cuda(), topk, ws)
    ws.check()
    total = batch * n_ok
    queries = None if total <= 24 else sorted({*range(12), *range(0, total, 13), total - 1})
    _check_all(dims, out, lse, q, lambda b, i: _listed_rows(cache, b, idx[b, i], max_len), queries)


def test_agrees_with_the_bf16_kernel_on_the_read_back_cache():
    dims, cache, q, ws = _setup("prod", 1, 200, 3000, 1000, seed=3)
    idx = _lists(2, 1, 200, 1000, 3000).cuda()
    out, lse = dsa.sparse_mla_attn_qcache(dims, q.cuda(), cache, idx, 1000, ws)
    full = dsa.make_dims(1, 3000, 3000, **DIMS["prod"])
    kv = dsa.qcache_read(full, cache, ws)
    ws16 = dsa.Workspace.create(dims, 1000)
    o16, l16 = dsa.sparse_mla_attn(dims, q.cuda(), kv, idx, 1000, ws16)
    ws.check(), ws16.check()
    # each is within half a bf16 step per weight and one of the result of the same numbers
    empty = torch.isinf(l16)
    assert torch.equal(empty, torch.isinf(lse))
    assert (out.float() - o16.float()).abs().max() <= 4 * 2.0 ** -8 * max(1.0, kv.float().abs().max().item())
    assert (lse - l16)[~empty].abs().max() <= 2.0 ** -7


def test_out_of_range_positions_are_reported_and_skipped():
    dims, cache, q, ws = _setup("prod", 1, 4, 100, 200, seed=4)
    idx = torch.full((1, 4, 200), -1, dtype=torch.int32)
    idx[0, 0, :150] = torch.arange(150) % 100
    idx[0, 0, 70] = 100                                # one past the end
    idx[0, 1, 199] = 2 ** 31 - 1                       # only an invalid entry
    idx[0, 2, 3] = -2 ** 31
    idx[0, 2, 130] = 99
    idx[0, 3, 64:128] = 1000                           # a whole block
    idx[0, 3, 150] = 5
    out, lse = dsa.sparse_mla_attn_qcache(dims, q.cuda(), cache, idx.cuda(), 200, ws)
    torch.cuda.synchronize()
    assert dsa.dsa_get_device_status(ws.buf)[0] == dsa.DSA_ERR_INDEX_RANGE
    _check_all(dims, out, lse, q, lambda b, i: _listed_rows(cache, b, idx[b, i], 100))


@pytest.mark.parametrize("n", [1, 90])
def test_rows_nobody_lists_have_no_effect(n):
    dims, cache, q, ws = _setup("prod", 1, n, 256, 100, seed=5)
    idx = _lists(3, 1, n, 100, 128)                    # positions 0..127 only
    want = dsa.sparse_mla_attn_qcache(dims, q.cuda(), cache, idx.cuda(), 100, ws)
    cache.scales[:, 128:] = math.nan
    cache.rope[:, 128:] = math.inf
    got = dsa.sparse_mla_attn_qcache(dims, q.cuda(), cache, idx.cuda(), 100, ws)
    ws.check()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_a_listed_nan_reaches_its_own_query_only():
    dims, cache, q, ws = _setup("prod", 1, 3, 64, 64, seed=6)
    cache.scales[0, 7, 2] = math.nan
    idx = torch.arange(64, dtype=torch.int32).expand(1, 3, 64).clone()
    idx[0, 0, 7] = idx[0, 2, 7] = -1
    out, lse = dsa.sparse_mla_attn_qcache(dims, q.cuda(), cache, idx.cuda(), 64, ws)
    ws.check()
    assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1]).all()
    for i in (0, 2):
        check(out[0, i], lse[0, i], attend(q[0, i].double(), _listed_rows(cache, 0, idx[0, i], 64), 512,
                                           dims.softmax_scale))


@pytest.mark.parametrize("order", [1, -1])
def test_logits_that_grow_or_fall_by_hundreds_along_the_list(order):
    # row s is a multiple of one direction, so the logits are steps apart: the running max is raised
    # again and again (or never), and early blocks vanish beside late ones
    dims, cache, _, ws = _setup("prod", 1, 2, 256, 256, seed=7, scale=1.0)
    cache.codes.zero_(), cache.rope.zero_()
    cache.scales.fill_(1.0)
    cache.codes[0, :, 0] = 0x38                        # 1.0
    cache.scales[0, :, 0] = 1.0
    ramp = torch.arange(256).float() * order * 0.9
    cache.rope[0, :, 0] = ramp.to(torch.bfloat16).cuda()
    q = torch.zeros((1, 2, 128, 576), dtype=torch.bfloat16)
    q[..., 512] = torch.linspace(-2, 2, 128).to(torch.bfloat16)
    q[..., 0] = 30.0
    idx = torch.arange(256, dtype=torch.int32).expand(1, 2, 256).contiguous()
    out, lse = dsa.sparse_mla_attn_qcache(dims, q.cuda(), cache, idx.cuda(), 256, ws)
    ws.check()
    _check_all(dims, out, lse, q, lambda b, i: _listed_rows(cache, b, idx[b, i], 256))


def test_scales_over_the_whole_range():
    dims, cache, q, ws = _setup("prod", 1, 1, 64, 64, seed=8, scale=2.0 ** -60)
    exps = torch.arange(64 * 4).view(1, 64, 4) % 150 - 90             # -90 .. 59: both product forms
    cache.scales.copy_(torch.exp2(exps.float()))
    idx = torch.arange(64, dtype=torch.int32).view(1, 1, 64)
    out, lse = dsa.sparse_mla_attn_qcache(dims, q.cuda(), cache, idx.cuda(), 64, ws)
    ws.check()
    _check_all(dims, out, lse, q, lambda b, i: _listed_rows(cache, b, idx[b, i], 64))


def test_positions_past_32_bit_offsets():
    max_len = 4_300_000                                # codes past 2^31 bytes
    dims = dsa.make_dims(1, 1, max_len, n_heads=16, d_latent=512, d_rope=8, idx_dim=16)
    cache = dsa.QCache.create(dims)
    g = torch.Generator().manual_seed(9)
    hot = torch.tensor([0, 1, 2_200_000, max_len - 2, max_len - 1])
    cache.codes[0, hot.cuda()] = torch.randint(0, 120, (5, 512), generator=g).to(torch.uint8).cuda()
    cache.scales[0, hot.cuda()] = 2.0 ** -7
    cache.rope[0, hot.cuda()] = torch.randn((5, 8), generator=g).to(torch.bfloat16).cuda()
    q = torch.randn((1, 1, 16, 520), generator=g).to(torch.bfloat16)
    idx = hot.to(torch.int32).view(1, 1, 5)
    ws = dsa.Workspace.create_qcache(dims, 5)
    out, lse = dsa.sparse_mla_attn_qcache(dims, q.cuda(), cache, idx.cuda(), 5, ws)
    ws.check()
    _check_all(dims, out, lse, q, lambda b, i: _listed_rows(cache, b, idx[b, i], max_len))


# ----------------------------------------------------------------------------- drafted trees
def _tree_rows(cache, b, idx_row, draft, parents, i, max_len):
    path = path_of(parents[b].tolist(), i)
    if path is None:
        return torch.zeros((0, draft.shape[-1]), dtype=torch.float64)
    if isinstance(cache, dsa.QCache):
        ctx = _listed_rows(cache, b, idx_row, max_len)
    else:
        j = idx_row[(idx_row >= 0) & (idx_row < max_len)].long()
        ctx = cache[b, j.cuda()].double().cpu()
    return torch.cat([ctx, draft[b, path].double()])


def _parents(seed, batch, n):
    r = np.random.default_rng(seed)
    p = np.stack([[int(r.integers(-1, i)) for i in range(n)] for _ in range(batch)]).astype(np.int32)
    return torch.from_numpy(p)


@pytest.mark.parametrize("quant", [True, False])
@pytest.mark.parametrize("name,batch,n,max_len,topk", [
    ("prod", 1, 1, 50, 1), ("prod", 2, 5, 400, 200), ("prod", 1, 64, 300, 64), ("prod", 1, 65, 300, 70),
    ("prod", 3, 130, 200, 10), ("prod", 1, 16, 5000, 2048), ("odd", 2, 9, 100, 33), ("tiny", 1, 256, 300, 100)])
def test_trees(quant, name, batch, n, max_len, topk):
    dims, cache, q, ws = _setup(name, batch, n, max_len, topk, seed=10)
    g = torch.Generator().manual_seed(11)
    draft = torch.randn((batch, n, dims.d_latent + dims.d_rope), generator=g).to(torch.bfloat16)
    parents = _parents(12, batch, n)
    idx = _lists(13, batch, n, topk, max_len)
    ctx = cache
    if not quant:
        ctx = torch.randn((batch, max_len, dims.d_latent + dims.d_rope), generator=g).to(torch.bfloat16).cuda()
    out, lse = dsa.tree_mla_attn(dims, q.cuda(), ctx, idx.cuda(), topk, draft.cuda(), parents.cuda(), ws)
    ws.check()
    total = batch * n
    queries = None if total <= 24 else sorted({*range(0, total, 11), 63 % total, 64 % total, total - 1, total - 2})
    _check_all(dims, out, lse, q, lambda b, i: _tree_rows(ctx, b, idx[b, i], draft, parents, i, max_len), queries)


@pytest.mark.parametrize("n", [3, 64, 256])
def test_a_chain_is_the_causal_mask(n):
    dims, cache, q, ws = _setup("tiny", 1, n, 256, 8, seed=14)
    draft = torch.randn((1, n, 80), generator=torch.Generator().manual_seed(15)).to(torch.bfloat16)
    parents = torch.arange(-1, n - 1, dtype=torch.int32).view(1, n)
    idx = torch.full((1, n, 8), -1, dtype=torch.int32)                # no context at all
    out, lse = dsa.tree_mla_attn(dims, q.cuda(), cache, idx.cuda(), 8, draft.cuda(), parents.cuda(), ws)
    ws.check()
    _check_all(dims, out, lse, q, lambda b, i: draft[0, :i + 1].double(), sorted({0, 1, 2, n // 2, n - 1}))


def test_absent_nodes_invalid_parents_and_rows_off_the_path():
    n = 70
    dims, cache, q, ws = _setup("prod", 2, n, 100, 40, seed=16)
    draft = torch.randn((2, n, 576), generator=torch.Generator().manual_seed(17)).to(torch.bfloat16)
    parents = _parents(18, 2, n)
    parents[0, 50:] = -2                               # a padded batch
    parents[1, 4] = -9                                 # absent, and everything below it
    parents[1, 5], parents[1, 66] = 4, 5
    idx = _lists(19, 2, n, 40, 100)
    args = (dims, q.cuda(), cache, idx.cuda(), 40)
    out, lse = dsa.tree_mla_attn(*args, draft.cuda(), parents.cuda(), ws)
    ws.check()                                         # absent nodes are no error
    rows_of = lambda b, i: _tree_rows(cache, b, idx[b, i], draft, parents, i, 100)      # noqa: E731
    _check_all(dims, out, lse, q, rows_of, [0, 3, 49, 50, 69, 70, 74, 75, 76, 136, 139])
    assert (out[1, 66] == 0).all() and torch.isneginf(lse[1, 66]).all()
    # rows of absent nodes and off node 7's path may hold anything
    path = path_of(parents[1].tolist(), 7)
    bad = draft.clone()
    off = [s for s in range(n) if path is None or s not in path]
    bad[1, off] = math.nan
    out2, lse2 = dsa.tree_mla_attn(*args, bad.cuda(), parents.cuda(), ws)
    assert torch.equal(out2[1, 7], out[1, 7]) and torch.equal(lse2[1, 7], lse[1, 7])
    ws.check()
    # a parent that is not an earlier node is reported; the node and those below it are absent
    wrong = parents.clone()
    wrong[0, 2], wrong[0, 3] = 2, 2
    out3, lse3 = dsa.tree_mla_attn(*args, draft.cuda(), wrong.cuda(), ws)
    torch.cuda.synchronize()
    assert dsa.dsa_get_device_status(ws.buf)[0] == dsa.DSA_ERR_INDEX_RANGE
    assert (out3[0, 2:4] == 0).all() and torch.isneginf(lse3[0, 2:4]).all()
    assert torch.equal(out3[1], out[1])


@pytest.mark.parametrize("d_latent,d_rope,heads", [(24, 8, 3), (248, 64, 65), (504, 0, 128), (8, 24, 1), (512, 56, 64)])
def test_trees_over_a_bf16_cache_of_odd_dims(d_latent, d_rope, heads):
    dims = dsa.make_dims(2, 5, 90, n_heads=heads, d_latent=d_latent, d_rope=d_rope)
    g = torch.Generator().manual_seed(40)
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)             # noqa: E731
    q, kv, draft = rnd(2, 5, heads, d_latent + d_rope), rnd(2, 90, d_latent + d_rope).cuda(), rnd(2, 5, d_latent + d_rope)
    parents, idx = _parents(41, 2, 5), _lists(42, 2, 5, 70, 90)
    ws = dsa.Workspace.create_qcache(dims, 70)
    out, lse = dsa.tree_mla_attn(dims, q.cuda(), kv, idx.cuda(), 70, draft.cuda(), parents.cuda(), ws)
    ws.check()
    _check_all(dims, out, lse, q, lambda b, i: _tree_rows(kv, b, idx[b, i], draft, parents, i, 90))


@pytest.mark.parametrize("d_latent,d_rope,heads", [(16, 8, 2), (128, 64, 128), (240, 40, 65), (256, 64, 64),
                                                   (272, 8, 100), (496, 64, 127), (512, 0, 128)])
def test_listed_rows_of_odd_dims(d_latent, d_rope, heads):
    dims = dsa.make_dims(1, 6, 200, n_heads=heads, d_latent=d_latent, d_rope=d_rope)
    g = torch.Generator().manual_seed(43)
    cache = dsa.QCache.create(dims)
    codes = (torch.randn(cache.codes.shape, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    cache.codes.copy_(codes.view(torch.uint8))
    cache.scales.copy_(torch.exp2(torch.randint(-9, -5, cache.scales.shape, generator=g).float()))
    cache.rope.copy_(torch.randn(cache.rope.shape, generator=g).to(torch.bfloat16))
    q = torch.randn((1, 6, heads, d_latent + d_rope), generator=g).to(torch.bfloat16)
    idx = _lists(44, 1, 6, 150, 200)
    ws = dsa.Workspace.create_qcache(dims, 150)
    out, lse = dsa.sparse_mla_attn_qcache(dims, q.cuda(), cache, idx.cuda(), 150, ws)
    ws.check()
    _check_all(dims, out, lse, q, lambda b, i: _listed_rows(cache, b, idx[b, i], 200))


def test_codes_and_scales_of_another_writer():
    # E4M3's NaN codes read as NaN; a scale need not be a power of two
    dims, cache, q, ws = _setup("prod", 1, 3, 70, 70, seed=45)
    cache.scales.mul_(1.25)
    cache.codes[0, 9, 100] = 0x7F
    idx = torch.arange(70, dtype=torch.int32).expand(1, 3, 70).clone()
    idx[0, 0, 9] = idx[0, 2, 9] = -1
    out, lse = dsa.sparse_mla_attn_qcache(dims, q.cuda(), cache, idx.cuda(), 70, ws)
    ws.check()
    assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1]).all()
    back = dsa.qcache_read(dsa.make_dims(1, 70, 70, **DIMS["prod"]), cache, ws).cpu().double()[0]
    assert torch.isnan(back[9, 100]) and torch.isfinite(back[9, :100]).all()
    for i in (0, 2):                                   # the rows as read back: code * scale rounded to bf16
        check(out[0, i], lse[0, i], attend(q[0, i].double(), back[idx[0, i][idx[0, i] >= 0].long()], 512,
                                           dims.softmax_scale))


def test_many_items_of_every_length_one_after_another():
    # more queries than pairs of SMs, ranges from none to several blocks, so that consecutive items of a pair
    # meet every combination of ring stage and buffer
    n = 700
    dims, cache, q, ws = _setup("prod", 1, n, 800, 330, seed=46)
    r = np.random.default_rng(47)
    idx = np.full((1, n, 330), -1, dtype=np.int32)
    for i in range(n):
        k = int(r.integers(0, 331)) if i % 7 else 0
        idx[0, i, :k] = r.integers(0, 800, k)
    idx = torch.from_numpy(idx)
    first = None
    for _ in range(3):
        out, lse = dsa.sparse_mla_attn_qcache(dims, q.cuda(), cache, idx.cuda(), 330, ws)
        ws.check()
        if first is None:
            first = (out.clone(), lse.clone())
            _check_all(dims, out, lse, q, lambda b, i: _listed_rows(cache, b, idx[b, i], 800), range(0, n, 9))
        else:                                          # no atomics: the same bits every time
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


# ----------------------------------------------------------------------------- streams, graphs, both together
def test_a_call_on_a_given_stream():
    dims, cache, q, ws = _setup("prod", 1, 2, 500, 300, seed=48)
    idx = _lists(49, 1, 2, 300, 500).cuda()
    q = q.cuda()
    want = dsa.sparse_mla_attn_qcache(dims, q, cache, idx, 300, ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        out, lse = dsa.sparse_mla_attn_qcache(dims, q, cache, idx, 300, ws, stream=s)
        side.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    ws.check()


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_clean():
    for n, topk in ((2, 1024), (300, 130)):            # ranges with a join, and many items
        dims, cache, q, ws = _setup("prod", 1, n, 2000, topk, seed=50)
        idx = _lists(51, 1, n, topk, 2000)
        dsa.dsa_set_wait_budget_ns(1)
        try:
            dsa.sparse_mla_attn_qcache(dims, q.cuda(), cache, idx.cuda(), topk, ws)
            torch.cuda.synchronize()
            status, detail = dsa.dsa_get_device_status(ws.buf)
        finally:
            dsa.dsa_set_wait_budget_ns(0)
        assert status == dsa.DSA_ERR_DEVICE_TIMEOUT and detail >> 16 == 4
        out, lse = dsa.sparse_mla_attn_qcache(dims, q.cuda(), cache, idx.cuda(), topk, ws)
        ws.check()
        _check_all(dims, out, lse, q, lambda b, i: _listed_rows(cache, b, idx[b, i], 2000), [0, 1, n - 1])


def test_other_streams_and_replayed_graphs():
    cases = []
    for seed in (20, 21):                              # two captured graphs with a workspace each
        dims, cache, q, ws = _setup("prod", 2, 3, 3000, 1500, seed=seed)
        idx = _lists(seed, 2, 3, 1500, 3000).cuda()
        cases.append((dims, q.cuda(), cache, idx, ws))
    want = [dsa.sparse_mla_attn_qcache(d, q, c, i, 1500, w) for d, q, c, i, w in cases]
    torch.cuda.synchronize()
    graphs, got = [], []
    for d, q, c, i, w in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(dsa.sparse_mla_attn_qcache(d, q, c, i, 1500, w))
        graphs.append(g)
    side = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        for t in got:
            t[0].zero_(), t[1].zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, side):                 # both at once
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for c in cases:
        c[4].check()


def test_a_serving_step_after_another():
    """Prompt into the cache, selection by the indexer on the written keys, attention over the cache, a drafted
    tree, its accepted path committed, and the next step attending to it as to any other row."""
    batch, prompt, cap, topk, n = 2, 300, 360, 128, 6
    g = torch.Generator().manual_seed(30)
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()      # noqa: E731
    lengths = torch.tensor([300, 211], dtype=torch.int32).cuda()
    pre = dsa.make_dims(batch, prompt, cap)
    cache = dsa.QCache.create(pre)
    ws = dsa.Workspace.create_qcache(dsa.make_dims(batch, n, cap), topk)
    latent, keys = rnd(batch, prompt, 576), rnd(batch, prompt, 128)
    dsa.qcache_write(pre, cache, latent, keys, ws, lengths=lengths)

    def select(lengths):
        dec = dsa.make_dims(batch, 1, cap)
        wsi = dsa.Workspace.create(dec, topk)
        q_idx = torch.randint(0, 120, (batch, 1, 64, 128), generator=g).to(torch.uint8).cuda()
        idx = dsa.indexer_topk(dec, q_idx, rnd(batch, 1, 64), cache.k_idx, torch.ones((batch, 1)).cuda(),
                               cache.k_scale, lengths, topk, wsi)
        wsi.check()
        return idx

    draft, dkeys = rnd(batch, n, 576), rnd(batch, n, 128)
    parents = torch.tensor([[-1, 0, 0, 2, -1, 4], [-1, 0, 1, -2, -2, -2]], dtype=torch.int32)
    tree = dsa.make_dims(batch, n, cap)
    idx = torch.cat([select(lengths) for _ in range(n)], dim=1).contiguous()
    q = rnd(batch, n, 128, 576)
    out, lse = dsa.tree_mla_attn(tree, q, cache, idx, topk, draft, parents.cuda(), ws)
    _check_all(tree, out, lse, q, lambda b, i: _tree_rows(cache, b, idx[b, i].cpu(), draft.cpu(), parents, i, cap))

    # the path of node 3 of the first sequence (0, 2, 3) and of node 1 of the second (0, 1) is accepted
    src = torch.tensor([[0, 2, 3], [0, 1, -1]], dtype=torch.int32).cuda()
    commit = dsa.make_dims(batch, 3, cap)
    start, after = lengths, lengths + torch.tensor([3, 2], dtype=torch.int32).cuda()
    dsa.qcache_write(commit, cache, draft, dkeys, ws, start=start, lengths=after, src_rows=src)

    dec = dsa.make_dims(batch, 1, cap)
    idx = select(after)
    idx[0, 0, 0], idx[1, 0, 0] = 302, 212              # the committed rows among them
    q = rnd(batch, 1, 128, 576)
    out, lse = dsa.sparse_mla_attn_qcache(dec, q, cache, idx, topk, ws)
    ws.check()
    _check_all(dec, out, lse, q, lambda b, i: _listed_rows(cache, b, idx[b, i].cpu(), cap))
    rows = dsa.qcache_read(commit, cache, ws, start=start, lengths=after).cpu().double()
    assert (rows[0, 2] - draft[0, 3].double().cpu()).abs().max() <= 2.0 ** -4 * draft[0, 3].abs().max().item()
    assert (rows[1, 2] == 0).all()
