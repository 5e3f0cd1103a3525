"""Workspaces that the calls on caches refuse before any launch (no GPU needed)."""
import pytest
import torch


@pytest.fixture(scope="module")
def dsa():
    from sparse_attention_long_indexer_b200.build import build
    build()
    import sparse_attention_long_indexer_b200 as m
    return m


def _calls(dsa, ws):
    d = dsa.make_dims(1, 2, 4, 4, 32, 8, 64, 16)
    cache = dsa.QCache.create(d, device="cpu")
    rows, q = torch.zeros((1, 2, 80), dtype=torch.bfloat16), torch.zeros((1, 2, 8, 80), dtype=torch.bfloat16)
    idx, par = torch.zeros((1, 2, 3), dtype=torch.int32), torch.full((1, 2), -1, dtype=torch.int32)
    return (lambda: dsa.qcache_write(d, cache, rows, None, ws), lambda: dsa.qcache_read(d, cache, ws),
            lambda: dsa.sparse_mla_attn_qcache(d, q, cache, idx, 3, ws),
            lambda: dsa.tree_mla_attn(d, q, cache, idx, 3, rows, par, ws),
            lambda: dsa.tree_mla_attn(d, q, torch.zeros((1, 4, 80), dtype=torch.bfloat16), idx, 3, rows, par, ws))


def _refused(dsa, monkeypatch, device, ws, kind, match):
    # the inputs pass for those of a call on `device`; the library is not to be reached
    monkeypatch.setattr(dsa, "_call_device", lambda t: device)
    monkeypatch.setattr(dsa, "_same", lambda *a: None)

    class NotReached:
        def __getattr__(self, name):
            raise AssertionError(f"{name} was called")
    monkeypatch.setattr(dsa, "_lib", NotReached())
    for call in _calls(dsa, ws):
        with pytest.raises(kind, match=match):
            call()


def test_a_workspace_elsewhere_is_refused(dsa, monkeypatch):
    # host memory, for a call on a GPU
    ws = dsa.Workspace(None, 1, torch.zeros(1024, dtype=torch.uint8))
    _refused(dsa, monkeypatch, 0, ws, ValueError, "workspace")


def test_a_workspace_of_another_type_is_refused(dsa, monkeypatch):
    # its size is counted in elements
    ws = dsa.Workspace(None, 1, torch.zeros(1024, dtype=torch.float32))
    _refused(dsa, monkeypatch, -1, ws, TypeError, "workspace")
