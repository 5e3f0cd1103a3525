"""Refusals of the calls on an 8-bit cache and on drafted trees: everything the host can see returns
before any launch (no GPU needed)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def dsa():
    from sparse_attention_long_indexer_b200.build import build
    build()
    import sparse_attention_long_indexer_b200 as m
    return m


FAKE = 1 << 20                    # never dereferenced: every call below fails validation
ODD = FAKE + 2


def _cache(dsa, codes=FAKE, scales=FAKE, rope=FAKE):
    return dsa.dsa_qcache(codes, scales, rope)


def _write(dsa, dims, latent=FAKE, keys=FAKE, n_src=8, src=None, start=None, lengths=None, cache=None, k_idx=FAKE,
           k_scale=FAKE, ws=FAKE, n=256):
    cache = _cache(dsa) if cache is None else cache
    return dsa._lib.dsa_qcache_write(ctypes.byref(dims), latent, keys, n_src, src, start, lengths,
                                     ctypes.byref(cache) if cache else None, k_idx, k_scale, ws, n, None)


def _read(dsa, dims, cache=None, rows=None, start=None, lengths=None, out=FAKE, ws=FAKE, n=256):
    cache = _cache(dsa) if cache is None else cache
    return dsa._lib.dsa_qcache_read(ctypes.byref(dims), ctypes.byref(cache) if cache else None, rows, start, lengths,
                                    out, ws, n, None)


def _sparse(dsa, dims, topk, q=FAKE, cache=None, idx=FAKE, out=FAKE, lse=FAKE, ws=FAKE, n=None):
    cache = _cache(dsa) if cache is None else cache
    n = dsa.dsa_qcache_workspace_bytes(dims, topk) if n is None else n
    return dsa._lib.dsa_sparse_mla_attn_qcache(ctypes.byref(dims), q, ctypes.byref(cache) if cache else None, idx, topk,
                                               out, lse, ws, n, None)


def _tree(dsa, dims, topk, quant, q=FAKE, ctx=FAKE, idx=FAKE, draft=FAKE, parents=FAKE, out=FAKE, lse=FAKE, ws=FAKE,
          n=None):
    n = dsa.dsa_qcache_workspace_bytes(dims, topk) if n is None else n
    if quant:
        cache = _cache(dsa) if ctx == FAKE else ctx
        return dsa._lib.dsa_tree_mla_attn_qcache(ctypes.byref(dims), q, ctypes.byref(cache) if cache else None, idx, topk,
                                                 draft, parents, out, lse, ws, n, None)
    return dsa._lib.dsa_tree_mla_attn(ctypes.byref(dims), q, ctx, idx, topk, draft, parents, out, lse, ws, n, None)


def test_write_refuses(dsa):
    d = dsa.make_dims(2, 8, 16)
    inv, uns = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED
    assert _write(dsa, dsa.make_dims(2, 8, 16, d_latent=24)) == uns             # half a 16-byte chunk of codes
    assert _write(dsa, dsa.make_dims(2, 8, 16, d_latent=528)) == uns
    assert _write(dsa, dsa.make_dims(2, 17, 16)) == inv                         # more rows than the cache holds
    assert _write(dsa, d, latent=None, keys=None) == inv
    assert _write(dsa, d, n_src=7) == inv                                       # fewer sources than rows
    assert _write(dsa, d, n_src=-1, src=FAKE) == inv
    assert _write(dsa, d, cache=False) == inv
    assert _write(dsa, d, cache=_cache(dsa, codes=None)) == inv
    assert _write(dsa, d, cache=_cache(dsa, scales=None)) == inv
    assert _write(dsa, d, cache=_cache(dsa, rope=None)) == inv
    assert _write(dsa, d, cache=_cache(dsa, codes=FAKE + 8)) == inv
    assert _write(dsa, d, cache=_cache(dsa, scales=ODD)) == inv
    assert _write(dsa, d, k_idx=None) == inv and _write(dsa, d, k_scale=None) == inv
    for name in ("latent", "keys", "src", "start", "lengths", "k_idx", "k_scale"):
        assert _write(dsa, d, **{name: ODD}) == inv, name
    for ws, n in ((None, 256), (FAKE + 8, 256), (FAKE, 255)):
        assert _write(dsa, d, ws=ws, n=n) == dsa.DSA_ERR_WORKSPACE
    assert _write(dsa, dsa.make_dims(0, 8, 16), latent=None, keys=None) == dsa.DSA_OK       # nothing to do
    assert _write(dsa, dsa.make_dims(2, 0, 16)) == dsa.DSA_OK


def test_read_refuses(dsa):
    d = dsa.make_dims(2, 8, 16)
    inv = dsa.DSA_ERR_INVALID_ARG
    assert _read(dsa, dsa.make_dims(2, 8, 16, d_latent=40)) == dsa.DSA_ERR_UNSUPPORTED
    assert _read(dsa, d, cache=False) == inv and _read(dsa, d, cache=_cache(dsa, rope=ODD)) == inv
    assert _read(dsa, d, out=None) == inv
    for name in ("rows", "start", "lengths", "out"):
        assert _read(dsa, d, **{name: ODD}) == inv, name
    assert _read(dsa, d, n=0) == dsa.DSA_ERR_WORKSPACE
    assert _read(dsa, dsa.make_dims(2, 0, 16), out=None) == dsa.DSA_OK


def test_attention_refuses(dsa):
    inv, uns = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED
    d = dsa.make_dims(2, 8, 16)
    assert _sparse(dsa, dsa.make_dims(2, 8, 16, d_latent=24), 4) == uns
    assert _sparse(dsa, d, 0, n=1 << 20) == inv and _sparse(dsa, d, 2049, n=1 << 20) == uns
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert _sparse(dsa, dsa.make_dims(2, 8, 16, softmax_scale=scale), 4, n=1 << 20) == inv
        assert _tree(dsa, dsa.make_dims(2, 8, 16, softmax_scale=scale), 4, False, n=1 << 20) == inv
    for name in ("q", "idx", "out", "lse"):
        assert _sparse(dsa, d, 4, **{name: None}) == inv, name
        assert _sparse(dsa, d, 4, **{name: ODD}) == inv, name
    assert _sparse(dsa, d, 4, cache=False) == inv and _sparse(dsa, d, 4, cache=_cache(dsa, codes=None)) == inv
    need = dsa.dsa_qcache_workspace_bytes(d, 4)
    assert need >= 256 and _sparse(dsa, d, 4, n=need - 1) == dsa.DSA_ERR_WORKSPACE
    assert _sparse(dsa, d, 4, ws=None) == dsa.DSA_ERR_WORKSPACE
    for quant in (True, False):
        for name in ("q", "idx", "draft", "parents", "out", "lse"):
            assert _tree(dsa, d, 4, quant, **{name: None}) == inv, name
            assert _tree(dsa, d, 4, quant, **{name: ODD}) == inv, name
        assert _tree(dsa, dsa.make_dims(1, 257, 300), 4, quant, n=1 << 30) == uns        # more nodes than a tree holds
        assert _tree(dsa, d, 4, quant, n=255) == dsa.DSA_ERR_WORKSPACE
        assert _tree(dsa, dsa.make_dims(0, 8, 16), 4, quant, q=None, draft=None) == dsa.DSA_OK
    assert _tree(dsa, d, 4, True, ctx=False) == inv and _tree(dsa, d, 4, False, ctx=None) == inv
    assert _tree(dsa, d, 4, False, ctx=ODD) == inv
    # an odd latent width is a bf16 cache's alone
    assert _tree(dsa, dsa.make_dims(2, 8, 16, d_latent=24), 4, True, n=1 << 30) == uns


def test_workspace_covers_both_forms(dsa):
    for args, topk in (((1, 1, 4096), 2048), ((1, 16, 4096), 2048), ((3, 200, 4096), 77), ((1, 256, 256), 1)):
        d = dsa.make_dims(*args)
        n = dsa.dsa_qcache_workspace_bytes(d, topk)
        assert n >= 256 and n % 256 == 0
        # never more than a fp32 output for each of a few hundred ranges
        assert n <= 256 + (args[0] * args[1] + 512) * 32 * 128 * 513 * 4
    assert dsa.dsa_qcache_workspace_bytes(dsa.make_dims(1, 8, 4), 4) == 0
    assert dsa.dsa_qcache_workspace_bytes(dsa.make_dims(1, 1, 4), 0) == 0


def test_binding_checks_what_the_library_cannot_see(dsa):
    """Sizes, types and devices of tensors: the wrappers raise before the call."""
    d = dsa.make_dims(1, 4, 8, 4, 32, 8, 64, 16)
    cache = dsa.QCache.create(d, device="cpu")
    assert cache.codes.shape == (1, 8, 64) and cache.scales.shape == (1, 8, 1) and cache.rope.shape == (1, 8, 16)
    latent = torch.zeros((1, 4, 80), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="current device"):
        dsa.qcache_write(d, cache, latent, None, None)
    with pytest.raises(ValueError, match="neither"):
        dsa.qcache_write(d, cache, None, None, None)
    with pytest.raises(ValueError, match="current device"):
        dsa.qcache_read(d, cache, None)
    q = torch.zeros((1, 4, 8, 80), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="current device"):
        dsa.sparse_mla_attn_qcache(d, q, cache, torch.zeros((1, 4, 3), dtype=torch.int32), 3, None)
    for t, kind in ((latent.float(), TypeError), (latent[:, :3], ValueError)):
        with pytest.raises(kind, match="latent"):
            dsa._same("latent", t, torch.bfloat16, 4 * 80, -1)
    with pytest.raises(ValueError, match="contiguous"):
        dsa._ptr(torch.zeros((4, 8)).t())
