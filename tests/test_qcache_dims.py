"""Dims of the calls on caches: what each of them does not use is not checked, and what it uses is (no GPU needed: a
call whose dims pass ends at a missing pointer)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def dsa():
    from sparse_attention_long_indexer_b200.build import build
    build()
    import sparse_attention_long_indexer_b200 as m
    return m


FAKE = 1 << 20                    # never dereferenced: a pointer is missing in every call


def _write(dsa, dims, keys=FAKE, n_src=None):
    c = dsa.dsa_qcache(None, FAKE, FAKE)                                        # no codes
    return dsa._lib.dsa_qcache_write(ctypes.byref(dims), FAKE, keys, dims.n_q if n_src is None else n_src, None, None,
                                     FAKE, ctypes.byref(c), FAKE, FAKE, FAKE, 256, None)


def _read(dsa, dims):
    c = dsa.dsa_qcache(FAKE, FAKE, FAKE)
    return dsa._lib.dsa_qcache_read(ctypes.byref(dims), ctypes.byref(c), FAKE, None, None, None, FAKE, 256, None)


def _sparse(dsa, dims, topk=64):
    c = dsa.dsa_qcache(FAKE, FAKE, FAKE)
    return dsa._lib.dsa_sparse_mla_attn_qcache(ctypes.byref(dims), None, ctypes.byref(c), FAKE, topk, FAKE, FAKE, FAKE,
                                               1 << 34, None)


# a missing pointer and refused dims give the same status where a size is negative: the dims that are allowed are told
# from those by UNSUPPORTED ones beside them (d_latent of half a chunk is looked at behind the sizes)
def _passes(call, dsa, *args, **kw):
    ok = call(dsa, dsa.make_dims(*args, **kw)) == dsa.DSA_ERR_INVALID_ARG
    return ok and call(dsa, dsa.make_dims(*args, **{**kw, "d_latent": 24})) == dsa.DSA_ERR_UNSUPPORTED


@pytest.mark.parametrize("args", [(1, 16384, 8192), (3, 9, 4), (2, 5, 0), (1, 1, 20_000_000)])
def test_rows_and_cache_length_are_independent(dsa, args):
    assert _passes(_read, dsa, *args) and _passes(_write, dsa, *args)


def test_what_the_row_calls_do_not_use_is_not_checked(dsa):
    kw = dict(n_idx_heads=200, n_heads=500, softmax_scale=float("nan"))
    assert _passes(_read, dsa, 1, 4, 8, idx_dim=24, **kw)
    assert _passes(_write, dsa, 1, 4, 8, **kw)
    assert _passes(lambda m, d: _write(m, d, keys=None), dsa, 1, 4, 8, idx_dim=24, **kw)
    for idx_dim in (8, 24, 144):
        assert _write(dsa, dsa.make_dims(1, 4, 8, idx_dim=idx_dim)) == dsa.DSA_ERR_UNSUPPORTED
    assert _write(dsa, dsa.make_dims(1, 4, 8, idx_dim=0)) == dsa.DSA_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [_write, _read])
def test_what_the_row_calls_use_is(dsa, call):
    uns, inv = dsa.DSA_ERR_UNSUPPORTED, dsa.DSA_ERR_INVALID_ARG
    for kw in (dict(d_latent=24), dict(d_latent=528), dict(d_rope=12), dict(d_rope=72)):
        assert call(dsa, dsa.make_dims(1, 4, 8, **kw)) == uns, kw
    for args in ((-1, 4, 8), (1, -4, 8), (1, 4, -8)):
        assert call(dsa, dsa.make_dims(*args, d_latent=24)) == inv, args            # before what is unsupported
    assert call(dsa, dsa.make_dims(1, 4, 8, d_latent=0)) == inv
    assert call(dsa, dsa.make_dims(1, 4, 8, d_rope=-8)) == inv
    assert call(dsa, dsa.make_dims(1 << 16, 4, 1 << 16)) == uns                       # rows of a cache
    assert call(dsa, dsa.make_dims(1 << 16, 1 << 16, 4)) == uns                       # rows of a call


def test_the_attention_takes_a_cache_longer_than_a_decode_selection(dsa):
    assert _passes(_sparse, dsa, 1, 1, 20_000_000) and _passes(_sparse, dsa, 1, 2, 20_000_000)
    assert dsa.dsa_qcache_workspace_bytes(dsa.make_dims(1, 1, 20_000_000), 64) > 0
    # the selection itself does not, nor the calls that may run it
    assert dsa.dsa_workspace_bytes(dsa.make_dims(1, 1, 20_000_000), 64) == 0
    # queries are of positions of the cache, and drafted nodes keep to the same rule
    assert _sparse(dsa, dsa.make_dims(1, 8, 4, d_latent=24)) == dsa.DSA_ERR_INVALID_ARG
