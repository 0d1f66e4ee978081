"""The gated recurrence and the 8-bit projection without a GPU: layouts of
results, sizes at the ends of the index types, and the kernels' tables of a
tile replayed."""
import numpy as np
import pytest
import torch

from scan_gated_rnns_b200 import _abi, gated, ops


@pytest.fixture
def launches(monkeypatch):
    """CPU tensors stand for the GPU's; what would be launched is recorded."""
    calls = []
    monkeypatch.setattr(ops, "_need_cuda", lambda t, name: None)
    monkeypatch.setattr(gated, "_launch", lambda fn, device, *args: calls.append((fn.__name__, args)) or 0)
    return calls


# ------------------------------------------------------------ results
def row_dense(t):
    return t.is_contiguous()


@pytest.mark.parametrize("shape", [(3, 8), (7, 8), (2, 5)])
def test_results_of_a_sliding_window_have_dense_rows(launches, shape):
    """Rows that overlap (x.unfold): the kernels write rows of D elements one
    behind another, so that is how the results have to lie."""
    rows, D = shape
    f = torch.zeros(rows + D - 1).unfold(0, D, 1)
    assert f.shape == shape and f.stride() == (1, 1)
    v = torch.zeros(rows, D)
    h, last, states = gated.gated_scan(f, v, save_states=True)
    assert row_dense(h)
    df, dv, _ = gated.gated_scan_backward(f, f, None, states, v)
    assert row_dense(df) and row_dense(dv)
    assert row_dense(gated.gated_step(f, v, torch.zeros(rows, D)))
    h, _ = gated.gated_scan_fn(f.requires_grad_(True), v)
    assert row_dense(h)
    assert [name for name, _ in launches] == ["gated_scan", "gated_scan_backward", "gated_step", "gated_scan"]
