"""Workspace of the calls on caches: one made for the largest sizes serves every smaller call, and one that is too
small for the ranges of a split call is refused (no GPU needed: every call ends in the host's checks)."""
import ctypes
import itertools

import pytest


@pytest.fixture(scope="module")
def dsa():
    from sparse_attention_long_indexer_b200.build import build
    build()
    import sparse_attention_long_indexer_b200 as m
    return m


FAKE = 1 << 20                    # never dereferenced: q is missing in every call that has workspace enough


def _calls(dsa, dims, topk, n):
    cache = dsa.dsa_qcache(FAKE, FAKE, FAKE)
    d, c = ctypes.byref(dims), ctypes.byref(cache)
    return (dsa._lib.dsa_sparse_mla_attn_qcache(d, None, c, FAKE, topk, FAKE, FAKE, FAKE, n, None),
            dsa._lib.dsa_tree_mla_attn(d, None, FAKE, FAKE, topk, FAKE, FAKE, FAKE, FAKE, FAKE, n, None),
            dsa._lib.dsa_tree_mla_attn_qcache(d, None, c, FAKE, topk, FAKE, FAKE, FAKE, FAKE, FAKE, n, None))


@pytest.mark.parametrize("kw", [dict(), dict(n_heads=8, d_latent=64, d_rope=16)])
def test_it_never_shrinks_as_sizes_grow(dsa, kw):
    batches, ns, topks = (1, 2, 5, 16, 37, 40, 64, 75, 93, 94, 128, 300), (1, 2, 7, 64, 65, 256, 300), (1, 64, 65, 700,
                                                                                                        2048)
    size = {k: dsa.dsa_qcache_workspace_bytes(dsa.make_dims(k[0], k[1], 4096, **kw), k[2])
            for k in itertools.product(batches, ns, topks)}
    for b, n, t in size:
        for axis, values in enumerate((batches, ns, topks)):
            key = [b, n, t]
            at = values.index(key[axis])
            if at > 0:
                key[axis] = values[at - 1]
                assert size[tuple(key)] <= size[b, n, t], (key, (b, n, t))
    # at the production dims a range's outputs are 256 KB and its statistics 512 B
    if not kw:
        assert size[1, 1, 2048] <= 256 + 33 * (128 * 512 * 4 + 512) + 512
        assert max(size.values()) <= 256 + 200 * (128 * 512 * 4 + 512) + 512


@pytest.mark.parametrize("largest", [(128, 1, 2048), (40, 1, 2048), (16, 16, 2048), (4, 65, 1500)])
def test_every_smaller_call_takes_it(dsa, largest):
    n = dsa.dsa_qcache_workspace_bytes(dsa.make_dims(largest[0], largest[1], 4096), largest[2])
    for b in range(1, largest[0] + 1):
        for nq in sorted({1, (largest[1] + 1) // 2, largest[1]}):
            for topk in (1, 64, 65, largest[2] // 2, largest[2]):
                got = _calls(dsa, dsa.make_dims(b, nq, 4096), topk, n)
                assert got == (dsa.DSA_ERR_INVALID_ARG,) * 3, (b, nq, topk)       # q is missing; the workspace is not


@pytest.mark.parametrize("b,n,topk", [(1, 1, 2048), (8, 1, 2048), (37, 1, 2048), (1, 16, 2048), (1, 2, 130)])
def test_too_small_for_the_ranges_is_refused(dsa, b, n, topk):
    dims = dsa.make_dims(b, n, 4096)
    need = dsa.dsa_qcache_workspace_bytes(dims, topk)
    assert need > 256 + b * n * 2 * 128 * 512 * 4                 # split in two at least
    assert _calls(dsa, dims, topk, need) == (dsa.DSA_ERR_INVALID_ARG,) * 3
    for short in (need - 1, need // 2, 256, 0):
        assert _calls(dsa, dims, topk, short) == (dsa.DSA_ERR_WORKSPACE,) * 3, short
