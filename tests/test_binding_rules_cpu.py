"""The binding's descriptor of logit rules, on host tensors (which count as
device -1; no GPU needed)."""
import pytest
import torch

import quantized_moe_q4_b200 as m


def words(n, V):
    return torch.zeros(n, (V + 31) // 32, dtype=torch.int32)


def test_no_masks_at_all_are_refused_not_ignored():
    """An empty tensor has no address, and no mask means that all is allowed."""
    V, T = 100, 4
    rows = torch.zeros(T, dtype=torch.int32)
    m.LogitRules(mask=words(1, V), mask_row=rows).struct(T, V, -1)
    with pytest.raises(ValueError):
        m.LogitRules(mask=words(0, V), mask_row=rows).struct(T, V, -1)
    with pytest.raises(ValueError):
        m.LogitRules(mask=words(0, V)).struct(T, V, -1)
    m.LogitRules(mask=words(0, V)).struct(0, V, -1)   # a mask a row, and no rows
