"""The gated recurrence and the 8-bit projection without a GPU: layouts of
results, sizes at the ends of the index types, and the kernels' tables of a
tile replayed."""
import numpy as np
import pytest
import torch

from scan_gated_rnns_b200 import _abi, gated, ops

from test_abi import fake_addresses


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


# -------------------------------------------------------------- sizes
def project(rows, K, N, x_rs, w_rs):
    return _abi.lib().int8_projection(1 << 40, x_rs, _abi.SGR_I8, 2 << 40, 3 << 40, w_rs, 4 << 40, None, 5 << 40, N,
                                      _abi.SGR_F32, rows, K, N, None, 0, None)


@fake_addresses
def test_projection_of_many_rows_at_any_alignment():
    """Rows of 100 bytes: nothing refuses their number (no device is here, so
    the launch is what fails)."""
    for rows in (64 * 65535, 64 * 65535 + 1, 10 ** 7):
        assert project(rows, 100, 8, 100, 100) == _abi.SGR_ERR_CUDA
    assert project(1 << 30, 100, 1 << 14, 100, 100) == _abi.SGR_ERR_UNSUPPORTED      # tiles past 2^31 - 1


@fake_addresses
def test_scan_of_the_most_sequences():
    """The bounds' search counts sequences in 32 bits, 32 at a time."""
    def scan(n):
        return _abi.lib().gated_scan(1 << 40, 8, 2 << 40, 8, None, 0, 3 << 40, 4, n, 4 << 40, 8, None, None, 400, 8,
                                     _abi.SGR_GATE_LOG, _abi.SGR_F32, 1, 5 << 40, 1 << 30, None)

    assert scan(2 ** 31 - 1) == _abi.SGR_ERR_UNSUPPORTED and scan(2 ** 31 - 32) == _abi.SGR_ERR_UNSUPPORTED
    assert scan(2 ** 31 - 64) == _abi.SGR_ERR_CUDA
