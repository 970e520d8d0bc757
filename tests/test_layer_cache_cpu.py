"""What LayerCache passes on, seen without a GPU."""
import pytest
import torch


@pytest.fixture
def m():
    import token_eviction_b200
    return token_eviction_b200


def test_budgets_per_head_reach_the_eviction(m, monkeypatch):
    seen = []
    monkeypatch.setattr(m._kvp_binding, "append", lambda *a: 0)
    monkeypatch.setattr(m._kvp_binding, "attend", lambda *a: 0)
    monkeypatch.setattr(m._kvp_binding, "evict", lambda *a: seen.append(a[10]) or 0)
    budgets = torch.tensor([[20, 12]], dtype=torch.int32)
    cache = m.LayerCache(1, 4, 2, 64, 64, 16, m.make_evict(32, 2, 4), device="cpu", budgets=budgets)
    cache.step(None, None, None)
    cache.evict()
    assert len(seen) == 2 and all(x is budgets for x in seen)
    cache = m.LayerCache(1, 4, 2, 64, 64, 16, m.make_evict(32, 2, 4), device="cpu")
    cache.step(None, None, None)
    assert seen[-1] is None


def test_budgets_without_a_policy_are_refused(m):
    with pytest.raises(ValueError, match="polic"):
        m.LayerCache(1, 4, 2, 64, 64, 16, device="cpu", budgets=torch.tensor([[20, 12]], dtype=torch.int32))


def test_evicting_without_a_policy_is_refused(m):
    with pytest.raises(ValueError, match="without an eviction policy"):
        m.LayerCache(1, 4, 2, 64, 64, 16, device="cpu").evict()
