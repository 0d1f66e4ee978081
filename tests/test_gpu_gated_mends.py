"""The gated recurrence on the GPU where its inputs are hard: rows that
overlap, gates far on either side, decays next to 1, infinities beside a gate
without gradient, and waits that run out."""
import numpy as np
import pytest
import torch

import scan_gated_rnns_b200 as sgr
from scan_gated_rnns_b200 import _abi

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


# --------------------------------------------------- gates far on one side
#
# 16-bit I/O has to keep both probabilities to their own precision as fp32 I/O
# does (an fp32 state holds them, and bf16 holds dv = z g down to 2^-126), so
# its bounds are those of the fp32 evaluation and the rounding of its type.
def operands(dtype, f, seed, n=1):
    rng = np.random.default_rng(seed)
    rows, D = f.shape
    f = torch.from_numpy(f).to(dtype)
    v, dh = (torch.from_numpy(rng.normal(size=(rows, D))).to(dtype) for _ in range(2))
    h0, dl = (torch.from_numpy(rng.normal(size=(n, D))).float() for _ in range(2))
    return [x.to(DEV) for x in (f, v, dh, h0, dl)], [x.double().numpy() for x in (f, v, dh, h0, dl)]


def both_directions(dtype, gate, f, cu, seed=0):
    (f, v, dh, h0, dl), (f64, v64, dh64, h64, l64) = operands(dtype, f, seed, len(cu) - 1)
    cu_d = torch.tensor(cu, device=DEV)
    h, last, states = sgr.gated_scan(f, v, h0, cu_d, gate, save_states=True)
    want, wl, bh, bl = scan64(f64, v64, h64, cu, gate)
    check(h, want, bh, dtype, "h")
    check(last, wl, bl, F32, "h_last")
    df, dv, d0 = sgr.gated_scan_backward(f, v, h0, states, dh, dl, cu_d, gate)
    wf, wv, w0, bf, bv, b0 = grad64(f64, v64, h64, cu, gate, dh64, l64)
    check(df, wf, bf, dtype, "df")
    check(dv, wv, bv, dtype, "dv")
    check(d0, w0, b0, F32, "dh0")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,D,layout", [(3000, 64, "mixed"), (600, 37, "mixed"), (2000, 64, "open"), (150, 64, "closed")])
def test_gates_far_on_either_side(rows, D, layout, dtype):
    """f up to 20 on either side: 1 - a down to 2e-9, where an fp32 a is 1."""
    rng = np.random.default_rng(rows + D)
    f = rng.uniform(-20, 20, size=(rows, D))
    if layout == "open":
        f = rng.uniform(8, 20, size=(rows, D))
    elif layout == "closed":
        f = rng.uniform(-20, -5, size=(rows, D))
    both_directions(dtype, "sigmoid", f, [0, rows // 3, rows])


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_long_memory_of_open_gates(dtype):
    """The state follows v by 1 - a a row over tens of thousands of rows."""
    f = np.broadcast_to(np.array([8.0, 10.0, 12.0, 13.0, 14.0, 15.0, 16.0, 18.0]), (40000, 8)).copy()
    both_directions(dtype, "sigmoid", f, [0, 40000])


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_tokens_continue_a_scan_of_open_gates(dtype):
    """A prompt in one call and the same tokens one by one end in one state."""
    f = np.random.default_rng(7).uniform(6, 17, size=(300, 40))
    (f, v, _, h0, _), (f64, v64, _, h64, _) = operands(dtype, f, 1)
    _, last = sgr.gated_scan(f, v, h0)
    state = h0.clone()
    for t in range(f.shape[0]):
        sgr.gated_step(f[t:t + 1], v[t:t + 1], state)
    _, want, _, bound = scan64(f64, v64, h64, [0, f.shape[0]], "sigmoid")
    check(last, want, bound, F32, "scan")
    check(state, want, bound, F32, "steps")


# ------------------------------------------------------ decays next to 1
#
# With v = 0, h0 = 1 and one row the fp32 state is the decay itself.  For
# -1/4 < f <= 0 its series ends in p = 1 + x (...) and 1 + x p: p is off by
# less than 2^-24 (a rounding below 1 is 2^-25, those before it come in times
# |x| / 2), so x p by less than 2^-26, and the last rounding is 2^-25; the terms
# left out are below 2^-31.  Together less than 2^-24.
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_decays_next_to_one_are_rounded_once(dtype):
    x = torch.cat([torch.linspace(-0.2499, 0, 4000), -torch.logspace(-7, -0.61, 4000)])
    f = x.to(dtype).to(DEV).view(-1, 8)
    zero, one = torch.zeros_like(f), torch.ones(f.shape[0], 8, device=DEV)
    want = np.exp(f.double().cpu().numpy())
    _, last = sgr.gated_scan(f, zero, one, torch.arange(f.shape[0] + 1, device=DEV), "log")
    state = one.clone()
    sgr.gated_step(f, zero, state, gate="log")
    for got in (last, state):
        assert np.abs(got.double().cpu().numpy() - want).max() < 2.0 ** -24


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_long_memory_of_log_gates(dtype):
    f = np.broadcast_to(-np.exp2(-np.arange(2.0, 18.0, 2.0)), (40000, 8)).copy()
    both_directions(dtype, "log", f, [0, 40000])


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,D", [(3000, 64), (600, 37)])
def test_log_gates_of_many_sizes(rows, D, dtype):
    rng = np.random.default_rng(rows)
    f = -np.exp(rng.uniform(-10, 4, size=(rows, D))) * np.where(rng.random((rows, D)) < 0.1, -1, 1)
    both_directions(dtype, "log", f, [0, rows // 3, rows])


# --------------------------------------- a gate without gradient (f > 0)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows", [5, 500])
def test_no_gradient_where_the_log_gate_is_clamped(rows, dtype):
    """df = [f <= 0] a h g is 0 where f > 0, also beside a state or an
    upstream gradient that is infinite or NaN."""
    torch.manual_seed(rows)
    f = torch.randn(rows, 6, device=DEV).abs().neg()
    f[::3] = 0.5
    v, dh = torch.randn(rows, 6, device=DEV), torch.randn(rows, 6, device=DEV)
    inf, nan = float("inf"), float("nan")
    last = rows - rows % 3 - (3 if rows % 3 == 0 else 0)      # the last clamped row
    v[0, 1], v[0, 2] = inf, nan                               # in the state from there on
    dh[last, 3], dh[last, 4], dh[last, 5] = inf, nan, -inf    # in the flow up to there
    f, v, dh = f.to(dtype), v.to(dtype), dh.to(dtype)
    _, _, states = sgr.gated_scan(f, v, gate="log", save_states=True)
    df, dv, _ = sgr.gated_scan_backward(f, v, None, states, dh, gate="log")
    assert bool((df[f > 0] == 0).all())
    # with no clamped row the same infinities do reach df
    g = torch.minimum(f, torch.zeros_like(f))
    _, _, states = sgr.gated_scan(g, v, gate="log", save_states=True)
    df0, dv0, _ = sgr.gated_scan_backward(g, v, None, states, dh, gate="log")
    assert bool((~torch.isfinite(df0[1:last + 1, 1:])).any(0).all()) and torch.equal(dv.isnan(), dv0.isnan())
    bad = torch.full_like(f, nan)                             # a gate that is NaN itself
    df, _, _ = sgr.gated_scan_backward(bad, v, None, states, dh, gate="log")
    assert bool(df[1:].isnan().all())


# ------------------------------------------------------ waits that run out
@pytest.fixture
def hooks():
    lib = _abi.lib()
    yield lib
    lib.sgr_set_wait_limit(0)
    lib.sgr_set_block_wait_limit(0)
    lib.sgr_set_drop_publish(-1)


def compare(got, want, clean, name):
    """NaN outside `clean` (a mask of rows and channels), the same bits in it."""
    got, want = (x.reshape(clean.shape) for x in (got, want))
    assert bool(got[~clean].isnan().all()) and torch.equal(got[clean], want[clean]), name


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", ["sigmoid", "log"])
def test_a_tile_that_hands_nothing_on(gate, dtype, hooks):
    """The first tile of the first channels is mute: the tiles behind it give
    up, say so and give NaN up to the next sequence; the rest is as it was, and
    so is the next call."""
    rows, D, cu, strip = 2000, 160, [0, 500, 2000], 128 // dtype.itemsize
    rng = np.random.default_rng(1)
    f = rng.normal(size=(rows, D)) + 1 if gate == "sigmoid" else -np.exp(rng.normal(size=(rows, D)))
    (f, v, dh, h0, dl), _ = operands(dtype, f, 2, 2)
    cu_d = torch.tensor(cu, device=DEV)
    ws = sgr.Workspace(sgr.workspace_size("gated", 1, rows, D, dtype), DEV)
    clean = sgr.gated_scan(f, v, h0, cu_d, gate, save_states=True, workspace=ws)
    back = sgr.gated_scan_backward(f, v, h0, clean[2], dh, dl, cu_d, gate, workspace=ws)
    assert ws.status() == 0
    hooks.sgr_set_wait_limit(500)
    hooks.sgr_set_drop_publish(0)
    h, last = sgr.gated_scan(f, v, h0, cu_d, gate, workspace=ws)
    assert ws.status(clear=False) == _abi.SGR_ERR_TIMEOUT
    ok = torch.ones(rows, D, dtype=torch.bool, device=DEV)
    ok[192:500, :strip] = False
    compare(h, clean[0], ok, "h")
    ok = torch.ones(2, D, dtype=torch.bool, device=DEV)
    ok[0, :strip] = False
    compare(last, clean[1], ok, "h_last")
    df, dv, d0 = sgr.gated_scan_backward(f, v, h0, clean[2], dh, dl, cu_d, gate, workspace=ws)
    assert ws.status() == _abi.SGR_ERR_TIMEOUT and ws.status() == 0
    ok = torch.ones(rows, D, dtype=torch.bool, device=DEV)
    ok[500:1920, :strip] = False                             # 96 rows a tile: the last of them begins at 1920
    compare(df, back[0], ok, "df")
    compare(dv, back[1], ok, "dv")
    ok = torch.ones(2, D, dtype=torch.bool, device=DEV)
    ok[1, :strip] = False
    compare(d0, back[2], ok, "dh0")
    hooks.sgr_set_drop_publish(-1)
    hooks.sgr_set_wait_limit(0)
    for a, b in zip(sgr.gated_scan(f, v, h0, cu_d, gate, workspace=ws), clean):
        assert torch.equal(a, b)
    for a, b in zip(sgr.gated_scan_backward(f, v, h0, clean[2], dh, dl, cu_d, gate, workspace=ws), back):
        assert torch.equal(a, b)
    assert ws.status() == 0


def test_workspaces_that_do_not_fit():
    f = torch.zeros(1000, 64, device=DEV)
    need = sgr.workspace_size("gated", 1, 1000, 64, F32)
    assert need == sgr.workspace_size("gated", 10, 100, 64, F32)
    with pytest.raises(ValueError, match="workspace"):
        sgr.gated_scan(f, f, workspace=sgr.Workspace(need - 16, DEV))
    with pytest.raises(ValueError, match="workspace"):
        sgr.gated_scan(f, f, workspace=sgr.Workspace(need, "cpu"))
    assert torch.equal(sgr.gated_scan(f[:50], f[:50], workspace=sgr.Workspace(16, DEV))[0], f[:50])   # needs none


def right_or_nan(got, want):
    """Every value has the clean call's bits or is NaN; whether one is NaN."""
    odd = got != want
    assert bool(got[odd].isnan().all())
    return bool(odd.any())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,D,n,layout", [(30000, 320, 7, "plain"), (9000, 160, 40, "odd"), (60, 64, 3, "plain"),
                                             (180, 33, 1, "odd"), (40000, 64, 1, "plain")])
def test_blocks_that_give_up(rows, D, n, layout, dtype, hooks):
    """Waits between a block's warps so short that some run out: every value is
    right or NaN, what lies beside the sequences stays, and the call says so."""
    rng = np.random.default_rng(rows)
    (f, v, dh, h0, dl), _ = operands(dtype, rng.normal(size=(rows, D)), 3, n)
    if layout == "odd":
        f, v, dh = (torch.cat([x[:, :1], x], 1)[:, 1:] for x in (f, v, dh))
    cu = torch.tensor([2, *sorted(rng.integers(2, rows - 5, n - 1).tolist()), rows - 5], device=DEV)
    ws = sgr.Workspace(max(16, sgr.workspace_size("gated", 1, rows, D, dtype)), DEV)

    def forward():
        out = torch.full((rows, D), 7.0, dtype=dtype, device=DEV)
        return sgr.gated_scan(f, v, h0, cu, out=out, save_states=True, workspace=ws)

    def backward():
        return sgr.gated_scan_backward(f, v, h0, states, dh, dl, cu, workspace=ws)

    *clean, states = forward()
    back = backward()
    assert ws.status() == 0
    lost = 0
    for polls in (1, 1, 1, 2, 3):
        hooks.sgr_set_block_wait_limit(polls)
        for call, want in ((forward, clean), (backward, back)):
            got = call()
            said = ws.status()
            bad = [right_or_nan(a, b) for a, b in zip(got, want)]
            lost += any(bad)
            assert said == _abi.SGR_ERR_TIMEOUT or not any(bad) or rows <= 192
            assert bool((got[0][:2] == want[0][:2]).all()) and bool((got[0][rows - 5:] == want[0][rows - 5:]).all())
        hooks.sgr_set_block_wait_limit(0)
        for a, b in zip([*forward()[:2], *backward()], [*clean, *back]):
            assert torch.equal(a, b)
        assert ws.status() == 0
    assert lost or rows < 30000


@pytest.mark.parametrize("K", [300, 12000])
def test_projection_whose_epilogue_gives_up(K, hooks):
    """Many tokens, several tiles a pair of SMs: warps that give up waiting for
    their sums must not hand accumulators on that others still read.  A poll
    takes some 4 us, a tile of the longer rows 40."""
    M, N = 5000, 4096
    x = torch.randint(-127, 128, (M, -(-K // 16) * 16), dtype=torch.int8, device=DEV)[:, :K]
    w = torch.randint(-127, 128, (N, -(-K // 16) * 16), dtype=torch.int8, device=DEV)[:, :K]
    sx, sw = torch.rand(M, device=DEV) + 0.5, torch.rand(N, device=DEV) + 0.5
    want = sgr.int8_projection(x, w, sw, x_scale=sx)
    lost = 0
    for polls in (1, 2, 3):
        hooks.sgr_set_block_wait_limit(polls)
        lost += right_or_nan(sgr.int8_projection(x, w, sw, x_scale=sx), want)
        hooks.sgr_set_block_wait_limit(0)
        assert torch.equal(sgr.int8_projection(x, w, sw, x_scale=sx), want)
    assert lost or K < 12000


def test_many_tokens_of_few_channels_quantised_within():
    """The product is set up while a million rows are quantised and waits for
    them: the same bits as in two calls."""
    x = torch.randn(1 << 20, 256, device=DEV, dtype=BF16)
    wq, ws = sgr.int8_quantize(torch.randn(96, 256, device=DEV))
    y = sgr.int8_projection(x, wq, ws)
    q, s = sgr.int8_quantize(x)
    assert torch.equal(y, sgr.int8_projection(q, wq, ws, x_scale=s, out_dtype=BF16))


def test_projection_of_many_rows_at_any_alignment():
    """More tiles of 64 rows than a grid has rows, on rows of an odd length."""
    M, K, N = 64 * 65536 + 1, 3, 2
    x = torch.randint(-127, 128, (M, K), dtype=torch.int8, device=DEV)
    w = torch.randint(-127, 128, (N, K), dtype=torch.int8, device=DEV)
    one = torch.ones(M, device=DEV)
    y = sgr.int8_projection(x, w, one[:N], x_scale=one)
    assert torch.equal(y, (x.int()[:, None, :] * w.int()[None]).sum(-1).float())


@pytest.mark.parametrize("step", [16, 48, 128, 8])
@pytest.mark.parametrize("rows", [5, 300, 3000])
def test_projection_of_a_sliding_window(rows, step):
    """8-bit rows that overlap one another, as tokens and as channels."""
    K, N = 128, 600
    g = torch.Generator(device=DEV).manual_seed(rows + step)
    x = torch.randint(-127, 128, (step * rows + K,), dtype=torch.int8, device=DEV, generator=g).unfold(0, K, step)[:rows]
    w = torch.randint(-127, 128, (step * N + K,), dtype=torch.int8, device=DEV, generator=g).unfold(0, K, step)[:N]
    one = torch.ones(max(rows, N), device=DEV)
    y = sgr.int8_projection(x, w, one[:N], x_scale=one[:rows])
    assert torch.equal(y, (x.double() @ w.double().t()).float())


# ------------------------------------------------------------- many bounds
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_sequences_in_many_segments(dtype):
    """More bounds than a block keeps in shared memory, and enough rows that they
    are cut into segments."""
    rng = np.random.default_rng(11)
    rows, D, n = 60000, 24, 5000
    cu = [4, *sorted(rng.integers(4, rows - 100, n - 1).tolist()), rows - 100]
    both_directions(dtype, "sigmoid", rng.normal(size=(rows, D)) * 4, cu)
