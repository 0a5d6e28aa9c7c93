"""Refusals of the expert sort through the binding (no GPU needed)."""
import pytest
import torch

from dense_fp8_gemm_b200 import spense

SHAPE = 2


def test_a_refused_sort_says_why_every_time(monkeypatch):
    """The same bad shape twice, with another refusal in between."""
    monkeypatch.setattr(spense, "_device_index", lambda: 0)
    ids = torch.zeros(4, 2, dtype=torch.int64)
    for _ in range(2):
        with pytest.raises(spense.SpenseError, match="E = 2000") as e:
            spense.expert_sort(ids, 2000)
        assert e.value.code == SHAPE
        with pytest.raises(spense.SpenseError):
            spense.plan_shapes([(0, 256, 64)], 1)
