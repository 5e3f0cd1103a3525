"""Launches of the attention over caches that end early: waits that run out, then a clean call.

Each case sets a budget of 1 ns for the pipeline's waits, so that a launch's first wait which is not
already over gives up and every role ends; the status word has to hold the timeout, and calls with the
default budget that follow at once have to be right (shared memory, TMEM and barriers of the launch that
ended early are gone by then, with nothing in flight to them)."""
import pytest
import torch

from tests.qcache_cases import attend, check, dequantised, path_of

pytestmark = pytest.mark.gpu

dsa = pytest.importorskip("sparse_attention_long_indexer_b200")

H, DL, DR = 128, 512, 64


def _case(kind, n, topk, seed):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)                   # noqa: E731
    dims = dsa.make_dims(1, n, 600, n_heads=H, d_latent=DL, d_rope=DR)
    cache = dsa.QCache.create(dims)
    kv = rnd(1, 600, DL + DR).cuda()
    ws = dsa.Workspace.create_qcache(dims, topk)
    dsa.qcache_write(dsa.make_dims(1, 600, 600, n_heads=H, d_latent=DL, d_rope=DR), cache, kv, None, ws)
    q = rnd(1, n, H, DL + DR).cuda()
    idx = torch.randint(0, 600, (1, n, topk), generator=g, dtype=torch.int32).cuda()
    draft = rnd(1, n, DL + DR).cuda()
    parents = (torch.rand((1, n), generator=g) * (torch.arange(n) + 1)).floor().to(torch.int32) - 1

    def call():
        if kind == "listed":
            return dsa.sparse_mla_attn_qcache(dims, q, cache, idx, topk, ws)
        return dsa.tree_mla_attn(dims, q, cache if kind == "tree8" else kv, idx, topk, draft, parents.cuda(), ws)

    def rows(i):
        at = idx[0, i].long()
        ctx = kv[0, at].double().cpu()
        if kind != "tree16":
            ctx = dequantised(cache.codes[0, at].cpu(), cache.scales[0, at].cpu(), cache.rope[0, at].cpu())
        if kind == "listed":
            return ctx
        return torch.cat([ctx, draft[0, path_of(parents[0].tolist(), i)].double().cpu()])

    def right(out, lse):
        for i in sorted({0, n // 2, n - 1}):
            check(out[0, i], lse[0, i], attend(q[0, i].double().cpu(), rows(i), DL, dims.softmax_scale))

    return call, right, ws


# lists of one or two blocks (the control warp has nothing left to wait for behind the query's copy), one
# item per pair and several
@pytest.mark.parametrize("kind", ["listed", "tree8", "tree16"])
@pytest.mark.parametrize("n,topk", [(1, 64), (74, 128), (200, 65)])
def test_launches_that_end_early_leave_nothing_in_flight(kind, n, topk):
    call, right, ws = _case(kind, n, topk, 60)
    right(*call())
    ws.check()
    for _ in range(8):
        dsa.dsa_set_wait_budget_ns(1)
        try:
            for _ in range(3):                          # one behind the other on the same SMs
                call()
        finally:
            dsa.dsa_set_wait_budget_ns(0)
        torch.cuda.synchronize()
        assert dsa.dsa_get_device_status(ws.buf)[0] == dsa.DSA_ERR_DEVICE_TIMEOUT
        out, lse = call()
        ws.check()
    right(out, lse)


# the widest numbers of a budget, held to a minute: as signed clocks, two to the ns, those from 2^62 on would have
# passed already
@pytest.mark.parametrize("ns", [10 ** 9, 2 ** 62 - 1, 2 ** 62, 2 ** 63, 2 ** 64 - 1])
def test_a_long_budget_is_a_long_one(ns):
    call, right, ws = _case("listed", 74, 128, 61)
    dsa.dsa_set_wait_budget_ns(ns)
    try:
        out, lse = call()
        torch.cuda.synchronize()
    finally:
        dsa.dsa_set_wait_budget_ns(0)
    ws.check()
    right(out, lse)
