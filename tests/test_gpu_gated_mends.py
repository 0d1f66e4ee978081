"""The gated recurrence on the GPU where its inputs are hard: rows that
overlap, gates far on either side, decays next to 1, infinities beside a gate
without gradient, and waits that run out."""
import numpy as np
import pytest
import torch

import scan_gated_rnns_b200 as sgr

from gated_reference import check, grad64, scan64

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

DEV = torch.device("cuda:0")
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,D", [(3, 8), (5, 7), (200, 256)])
def test_sliding_window(rows, D, dtype):
    rng = np.random.default_rng(rows)
    f = torch.from_numpy(rng.normal(size=rows + D - 1)).to(dtype).to(DEV).unfold(0, D, 1)
    v = torch.from_numpy(rng.normal(size=(rows, D))).to(dtype).to(DEV)
    dh = torch.from_numpy(rng.normal(size=(rows, D))).to(dtype).to(DEV)
    f64, v64, dh64 = (x.double().cpu().numpy() for x in (f, v, dh))
    zero = np.zeros((1, D))
    h, _, states = sgr.gated_scan(f, v, save_states=True)
    want, _, b, _ = scan64(f64, v64, zero, [0, rows], "sigmoid", dtype)
    check(h, want, b, dtype, "h")
    df, dv, _ = sgr.gated_scan_backward(f, v, None, states, dh)
    wf, wv, _, bf, bv, _ = grad64(f64, v64, zero, [0, rows], "sigmoid", dh64, None, dtype)
    check(df, wf, bf, dtype, "df")
    check(dv, wv, bv, dtype, "dv")
    state = torch.zeros(rows, D, device=DEV)
    y = sgr.gated_step(f, v, state)
    want, _, b, _ = scan64(f64, v64, np.zeros((rows, D)), list(range(rows + 1)), "sigmoid", dtype)
    check(y, want, b, dtype, "step")
