"""gated_scan, gated_scan_backward, gated_step and gated_scan_fn on the GPU
against the recurrence in 64 bits, token by token (gated_reference.py holds
the error bounds and their derivation)."""
import concurrent.futures

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


def gates(rng, gate, shape):
    x = rng.normal(size=shape)
    return 2.0 * x + 1.0 if gate == "sigmoid" else np.where(rng.random(shape) < 0.05, np.abs(x), -np.exp(2 * x - 3))


def make(rng, gate, rows, D, dtype, layout="plain"):
    """f, v (rows, D) on the GPU in the given layout, and their values in float64."""
    f, v = torch.from_numpy(gates(rng, gate, (rows, D))).to(dtype), torch.from_numpy(rng.normal(size=(rows, D))).to(dtype)
    if layout == "halves":
        both = torch.cat([f, v], 1).to(DEV)
        fd, vd = both[:, :D], both[:, D:]
    elif layout == "odd":                    # rows an odd number of elements apart, bases unaligned
        buf = torch.zeros(rows, 2 * D + 3, dtype=dtype, device=DEV)
        fd, vd = buf[:, 1:D + 1], buf[:, D + 2:2 * D + 2]
        fd.copy_(f)
        vd.copy_(v)
    else:
        fd, vd = f.to(DEV), v.to(DEV)
    return fd, vd, f.double().numpy(), v.double().numpy()


def bounds_of(rng, rows, kind):
    if kind == "one":
        return [0, rows]
    if kind == "tiny":                       # sequences of one token and empty ones
        return sorted([0, rows, *range(0, rows, 1), *rng.integers(0, rows + 1, 9).tolist()])
    if kind == "padded":
        lo, hi = min(3, rows), max(min(3, rows), rows - 5)
        return [lo, *sorted(rng.integers(lo, hi + 1, 4).tolist()), hi]
    return [0, *sorted(rng.integers(0, rows + 1, 6).tolist()), rows]


def run_case(rows, D, dtype, gate, kind, layout, init, seed=0):
    rng = np.random.default_rng(seed + rows * 7 + D)
    f, v, f64, v64 = make(rng, gate, rows, D, dtype, layout)
    cu = bounds_of(rng, rows, kind)
    n = len(cu) - 1
    cu_d = torch.tensor(cu, dtype=torch.int64 if rows % 2 else torch.int32, device=DEV)
    h0 = {"none": None, "each": rng.normal(size=(n, D)).astype(np.float32),
          "one": rng.normal(size=D).astype(np.float32)}[init]
    h0_64 = np.zeros((n, D)) if h0 is None else np.broadcast_to(h0.astype(np.float64), (n, D)).copy()
    h0_d = None if h0 is None else torch.from_numpy(h0).to(DEV)
    h, last, states = sgr.gated_scan(f, v, h0_d, cu_d, gate, save_states=True)
    want_h, want_l, bh, bl = scan64(f64, v64, h0_64, cu, gate, dtype)
    check(h, want_h, bh, dtype, "h")
    check(last, want_l, bl, F32, "h_last")
    dh = torch.from_numpy(rng.normal(size=(rows, D))).to(dtype)
    dl = torch.from_numpy(rng.normal(size=(n, D)).astype(np.float32)) if seed % 2 == 0 else None
    df, dv, d0 = sgr.gated_scan_backward(f, v, h0_d, states, dh.to(DEV), None if dl is None else dl.to(DEV), cu_d, gate)
    wf, wv, w0, bf, bv, b0 = grad64(f64, v64, h0_64, cu, gate, dh.double().numpy(),
                                    None if dl is None else dl.double().numpy(), dtype)
    check(df, wf, bf, dtype, "df")
    check(dv, wv, bv, dtype, "dv")
    check(d0, w0, b0, F32, "dh0")


@pytest.mark.parametrize("gate", ["sigmoid", "log"])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,D", [(1, 1), (1, 64), (3, 33), (111, 2), (112, 64), (113, 66), (224, 31), (450, 130),
                                    (1200, 96)])
@pytest.mark.parametrize("kind", ["one", "some", "tiny", "padded"])
def test_packed_rows(rows, D, dtype, gate, kind):
    run_case(rows, D, dtype, gate, kind, "plain", ["none", "each", "one"][(rows + D) % 3], rows % 2)


@pytest.mark.parametrize("gate", ["sigmoid", "log"])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("layout", ["halves", "odd"])
@pytest.mark.parametrize("rows,D", [(5, 7), (300, 48), (500, 192), (700, 65)])
def test_row_spacings(rows, D, dtype, gate, layout):
    run_case(rows, D, dtype, gate, "some", layout, "each")


@pytest.mark.parametrize("gate", ["sigmoid", "log"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_long_sequence(dtype, gate):
    run_case(20011, 40, dtype, gate, "one", "plain", "each")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shape", [(1, 1, 8), (3, 1, 40), (5, 37, 64), (2, 300, 96), (4, 224, 32), (40, 113, 8)])
def test_dense_batches(shape, dtype):
    rng = np.random.default_rng(11)
    B, T, D = shape
    f, v, f64, v64 = make(rng, "sigmoid", B * T, D, dtype)
    h0 = rng.normal(size=(B, D)).astype(np.float32)
    h, last = sgr.gated_scan(f.view(shape), v.view(shape), torch.from_numpy(h0).to(DEV))
    cu = [i * T for i in range(B + 1)]
    want, wl, bh, bl = scan64(f64, v64, h0.astype(np.float64), cu, "sigmoid", dtype)
    assert h.shape == shape and last.shape == (B, D) and last.dtype == F32
    check(h, want, bh, dtype, "h")
    check(last, wl, bl, F32, "h_last")


@pytest.mark.parametrize("gate", ["sigmoid", "log"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_wide_batch(dtype, gate):
    run_case(2500, 1024, dtype, gate, "some", "halves", "each")


def test_no_rows_and_no_channels():
    h0 = torch.randn(3, 8, device=DEV)
    e = torch.zeros(0, 8, device=DEV)
    h, last = sgr.gated_scan(e, e, h0, torch.zeros(4, dtype=torch.int32, device=DEV))
    assert h.shape == (0, 8) and torch.equal(last, h0)
    h, last = sgr.gated_scan(e.view(3, 0, 8), e.view(3, 0, 8), h0)
    assert h.shape == (3, 0, 8) and torch.equal(last, h0)
    h, last = sgr.gated_scan(e.view(3, 0, 8), e.view(3, 0, 8))
    assert torch.equal(last, torch.zeros_like(h0))
    z = torch.zeros(4, 0, device=DEV)
    assert sgr.gated_scan(z, z)[0].shape == (4, 0)
    rows = torch.randn(5, 8, device=DEV)                     # no sequences at all: every row is padding
    h, last = sgr.gated_scan(rows, rows, None, torch.zeros(1, dtype=torch.int64, device=DEV))
    assert torch.equal(h, torch.zeros_like(rows)) and last.shape == (0, 8)
    f = e.clone().requires_grad_(True)
    g0 = h0.clone().requires_grad_(True)
    h, last = sgr.gated_scan_fn(f, e, g0, torch.zeros(4, dtype=torch.int32, device=DEV))
    last.backward(2 * torch.ones_like(last))
    assert torch.equal(g0.grad, torch.full_like(h0, 2.0))


@pytest.mark.parametrize("gate", ["sigmoid", "log"])
def test_nan_and_infinity_stay_in_their_sequence(gate):
    rng = np.random.default_rng(2)
    rows, D = 700, 70
    f, v, _, _ = make(rng, gate, rows, D, F32)
    cu = [0, 100, 101, 230, 500, 700]
    h0 = rng.normal(size=(5, D)).astype(np.float32)
    dh = rng.normal(size=(rows, D))
    f[150, 3] = float("nan")
    v[40, 5] = float("inf")
    v[300, 6] = float("nan")
    h0[3, 7] = np.inf
    dh[210, 8] = np.inf
    dh[480, 9] = np.nan
    cu_d = torch.tensor(cu, device=DEV)
    h0_d, dh_d = torch.from_numpy(h0).to(DEV), torch.from_numpy(dh).to(DEV, F32)
    h, last, states = sgr.gated_scan(f, v, h0_d, cu_d, gate, save_states=True)
    f64, v64, h64 = (x.double().cpu().numpy() for x in (f, v, h0_d))
    want, wl, bh, bl = scan64(f64, v64, h64, cu, gate)
    check(h, want, bh, F32, "h")
    check(last, wl, bl, F32, "h_last")
    df, dv, d0 = sgr.gated_scan_backward(f, v, h0_d, states, dh_d, None, cu_d, gate)
    # a column is touched only in the sequences that hold one of its odd values
    touched = {(1, 5): 0, (2, 3): 1, (2, 8): 1, (3, 6): 1, (3, 7): 1, (3, 9): 1, (0, 5): 1}
    for s, (lo, hi) in enumerate(zip(cu, cu[1:])):
        for name, x in (("df", df[lo:hi]), ("dv", dv[lo:hi]), ("dh0", d0[s:s + 1])):
            ok = torch.isfinite(x).all(0)
            for col in torch.nonzero(~ok).flatten().tolist():
                assert touched.get((s, col)) == 1, (name, s, col)


def test_closed_and_open_gates():
    """f at the infinities and at the types' ends: exact limits."""
    D = 8
    v = torch.randn(6, D, device=DEV)
    h0 = torch.randn(1, D, device=DEV)
    inf = float("inf")
    for big in (inf, 3.0e38, 200.0):
        h, _ = sgr.gated_scan(torch.full_like(v, big), v, h0)
        assert torch.equal(h, h0.expand(6, D))               # everything kept
        h, _ = sgr.gated_scan(torch.full_like(v, -big), v, h0)
        assert torch.equal(h, v)                              # nothing kept
        h, _ = sgr.gated_scan(torch.full_like(v, -big), v, h0, gate="log")
        assert torch.equal(h, v)
        h, _ = sgr.gated_scan(torch.full_like(v, big), torch.zeros_like(v), h0, gate="log")
        assert torch.equal(h, h0.expand(6, D))
    low = torch.finfo(torch.bfloat16).min
    vb = v.to(BF16)
    assert torch.equal(sgr.gated_scan(torch.full_like(vb, low), vb)[0], vb)


def test_a_given_output_keeps_its_padding_rows():
    rng = np.random.default_rng(4)
    for rows, D in ((40, 24), (400, 24)):
        f, v, f64, v64 = make(rng, "sigmoid", rows, D, BF16)
        cu = [2, 17, rows - 9]
        out = torch.full((rows, D), 7.0, dtype=BF16, device=DEV)
        f[rows - 9:] = float("nan")                           # what padding holds does not matter
        got, _ = sgr.gated_scan(f, v, None, torch.tensor(cu, device=DEV), out=out)
        assert got.data_ptr() == out.data_ptr()
        want, _, b, _ = scan64(f64, v64, np.zeros((2, D)), cu, "sigmoid", BF16)
        check(out[2:rows - 9], want[2:rows - 9], b[2:rows - 9], BF16, "h")
        assert bool((out[:2] == 7).all()) and bool((out[rows - 9:] == 7).all())
        fresh, _, st = sgr.gated_scan(f, v, None, torch.tensor(cu, device=DEV), save_states=True)
        assert bool((fresh[:2] == 0).all()) and bool((fresh[rows - 9:] == 0).all())
        df, dv, _ = sgr.gated_scan_backward(f, v, None, st, torch.ones_like(v), None, torch.tensor(cu, device=DEV))
        for x in (df, dv):
            assert bool((x[:2] == 0).all()) and bool((x[rows - 9:] == 0).all()) and bool(torch.isfinite(x).all())


def test_bounds_in_no_order_touch_nothing_else():
    """Not a valid call: the values are unspecified, the memory around the
    arrays stays as it was (the search is replayed on the CPU first)."""
    rng = np.random.default_rng(6)
    rows, D = 500, 48
    buf = torch.full((rows + 64, D), 3.0, device=DEV)
    f, v, _, _ = make(rng, "sigmoid", rows, D, F32)
    for cu in ([0, 400, 100, 500], [300, 200, 100, 0], [0, 900, -7, 500], [-50, 20, 10 ** 6, 2 ** 30]):
        out = buf[32:32 + rows]
        sgr.gated_scan(f, v, None, torch.tensor(cu, device=DEV), out=out)
        torch.cuda.synchronize()
        assert bool((buf[:32] == 3).all()) and bool((buf[32 + rows:] == 3).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_equal_calls_give_equal_bits(dtype):
    rng = np.random.default_rng(8)
    f, v, _, _ = make(rng, "log", 30000, 320, dtype)
    cu = torch.tensor([0, 9, 11000, 30000], device=DEV)
    dh = torch.randn(30000, 320, device=DEV).to(dtype)
    first = None
    for _ in range(6):
        h, last, st = sgr.gated_scan(f, v, None, cu, "log", save_states=True)
        got = [h, last, *sgr.gated_scan_backward(f, v, None, st, dh, None, cu, "log")]
        if first is None:
            first = got
        assert all(torch.equal(a, b) for a, b in zip(got, first))


# ------------------------------------------------------------- autograd
@pytest.mark.parametrize("gate", ["sigmoid", "log"])
@pytest.mark.parametrize("packed", [False, True])
def test_autograd_matches_the_formulas(gate, packed):
    rng = np.random.default_rng(12)
    B, T, D = 3, 150, 36
    f, v, f64, v64 = make(rng, gate, B * T, D, F32)
    cu = [0, 10, 10, B * T] if packed else [0, T, 2 * T, 3 * T]
    n = len(cu) - 1
    h0 = torch.randn(D, device=DEV)                          # one state for every sequence: its gradient is a sum
    if not packed:
        f, v = f.view(B, T, D), v.view(B, T, D)
    leaves = [x.clone().requires_grad_(True) for x in (f, v, h0)]
    h, last = sgr.gated_scan_fn(*leaves, torch.tensor(cu, device=DEV) if packed else None, gate)
    dh, dl = torch.randn_like(h), torch.randn_like(last)
    torch.autograd.backward([h, last], [dh, dl])
    wf, wv, w0, bf, bv, b0 = grad64(f64, v64, np.broadcast_to(h0.double().cpu().numpy(), (n, D)).copy(), cu, gate,
                                    dh.double().cpu().numpy().reshape(B * T, D), dl.double().cpu().numpy())
    check(leaves[0].grad, wf, bf, F32, "df")
    check(leaves[1].grad, wv, bv, F32, "dv")
    check(leaves[2].grad, w0.sum(0), b0.sum(0) + 2.0 ** -22 * np.abs(w0).sum(0), F32, "dh0")


@pytest.mark.parametrize("gate", ["sigmoid", "log"])
def test_gradients_against_differences(gate):
    """Along one direction, at a size of several tiles: with step e the
    quotient has a truncation error of order e^2 and a rounding error of
    2^-24 sum |h dh| / e; both are below 1 % of the norms for e = 2^-6."""
    torch.manual_seed(3)
    T, D = 260, 16
    f = torch.randn(1, T, D, device=DEV) + 1 if gate == "sigmoid" else -torch.rand(1, T, D, device=DEV) - 0.1
    v, h0, dh = torch.randn(1, T, D, device=DEV), torch.randn(1, D, device=DEV), torch.randn(1, T, D, device=DEV)
    ds = [torch.randn_like(x) for x in (f, v, h0)]
    leaves = [x.clone().requires_grad_(True) for x in (f, v, h0)]
    h, _ = sgr.gated_scan_fn(*leaves, None, gate)
    grads = torch.autograd.grad(h, leaves, dh)
    e = 2.0 ** -6

    def loss(k, s):
        args = [f, v, h0]
        args[k] = args[k] + s * e * ds[k]
        return (sgr.gated_scan(*args, None, gate)[0].double() * dh.double()).sum()

    for k in range(3):
        quotient = float((loss(k, 1) - loss(k, -1)) / (2 * e))
        along = float((grads[k].double() * ds[k].double()).sum())
        assert abs(quotient - along) <= 0.01 * float(grads[k].double().norm() * ds[k].double().norm())


def test_autograd_shapes_unused_results_and_no_second_derivative():
    f = torch.randn(2, 130, 8, device=DEV, requires_grad=True)
    v = torch.randn(2, 130, 8, device=DEV)
    h, last = sgr.gated_scan_fn(f, v)
    last.sum().backward()                                    # only the last states used, no h0
    assert f.grad.shape == f.shape and bool(torch.isfinite(f.grad).all())
    h, _ = sgr.gated_scan_fn(f, v)
    h.sum().backward()                                       # an expanded gradient
    (g,) = torch.autograd.grad(sgr.gated_scan_fn(f, v)[0].square().sum(), f, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


# -------------------------------------------------------- streams, graphs
def test_other_stream_and_two_at_once():
    rng = np.random.default_rng(21)
    f, v, _, _ = make(rng, "sigmoid", 4000, 128, BF16)
    ref = sgr.gated_scan(f, v)[0]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for i in range(12):
        with torch.cuda.stream(streams[i % 3]):
            outs.append(sgr.gated_scan(f, v)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)


def test_two_captured_graphs_replayed_at_once():
    rng = np.random.default_rng(22)
    f, v, _, _ = make(rng, "log", 5000, 96, F32)
    f2, v2, _, _ = make(rng, "log", 5000, 96, F32)
    dh = torch.randn_like(f)

    def step(f, v):
        h, last, st = sgr.gated_scan(f, v, None, None, "log", save_states=True)
        return [h, last, *sgr.gated_scan_backward(f, v, None, st, dh, None, None, "log")]

    want = [step(f, v), step(f2, v2)]
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for a, b in ((f, v), (f2, v2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(step(a, b))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got, ref in zip(outs, want):
        assert all(torch.equal(x, y) for x, y in zip(got, ref))
    f.copy_(f2)                                               # the replay reads what is there then
    v.copy_(v2)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs[0], want[1]))


# ------------------------------------------------------------------ step
@pytest.mark.parametrize("gate", ["sigmoid", "log"])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("M,D,pool", [(1, 1, 1), (8, 1024, 8), (3, 33, 10), (300, 130, 511), (64, 4096, 70)])
def test_step(M, D, pool, dtype, gate):
    rng = np.random.default_rng(M + D)
    f, v, f64, v64 = make(rng, gate, M, D, dtype, "halves" if D % 2 == 0 else "odd")
    state = torch.randn(pool, D, device=DEV)
    before = state.double().cpu().numpy()
    slots = torch.from_numpy(rng.permutation(pool)[:M]).to(DEV, torch.int32 if M % 2 else torch.int64)
    h = sgr.gated_step(f, v, state, slots, gate)
    s = slots.cpu().numpy()
    want, _, b, _ = scan64(f64, v64, before[s], list(range(M + 1)), gate, dtype)
    check(h, want, b, dtype, "h")
    check(state[slots.long()], want, b, F32, "state")
    rest = np.setdiff1d(np.arange(pool), s)
    assert np.array_equal(state.double().cpu().numpy()[rest], before[rest])
    # without slots: row i on state i
    state2 = torch.from_numpy(before).to(DEV, F32)
    h2 = sgr.gated_step(f, v, state2, gate=gate)
    want2, _, b2, _ = scan64(f64, v64, before[:M], list(range(M + 1)), gate, dtype)
    check(h2, want2, b2, dtype, "h")


@pytest.mark.parametrize("D", [32, 37])
def test_step_slots_twice_and_padding(D):
    rng = np.random.default_rng(1)
    M, pool = 70, 9
    f, v, f64, v64 = make(rng, "sigmoid", M, D, F32)
    state = torch.randn(pool, D, device=DEV)
    st = state.double().cpu().numpy()
    slots = rng.integers(-2, pool + 2, M)
    want = np.full((M, D), 7.0)
    bound = np.zeros((M, D))
    err = np.zeros_like(st)
    for i, s in enumerate(slots):
        if 0 <= s < pool:
            w, _, b, _ = scan64(f64[i:i + 1], v64[i:i + 1], st[s:s + 1], [0, 1], "sigmoid")
            st[s], err[s] = w[0], err[s] + b[0]
            want[i], bound[i] = st[s], err[s]
    out = torch.full((M, D), 7.0, device=DEV)
    fresh_state = state.clone()
    sgr.gated_step(f, v, state, torch.from_numpy(slots).to(DEV), out=out)
    check(out, want, bound, F32, "h")
    check(state, st, err, F32, "state")
    fresh = sgr.gated_step(f, v, fresh_state, torch.from_numpy(slots).to(DEV))
    pad = (slots < 0) | (slots >= pool)
    assert bool((fresh[torch.from_numpy(pad).to(DEV)] == 0).all()) and torch.equal(fresh_state, state)


def test_steps_continue_a_scan():
    torch.manual_seed(0)
    B, T, D = 4, 137, 64
    f, v = (torch.randn(B, T, D, device=DEV) for _ in range(2))
    whole, last = sgr.gated_scan(f, v)
    h, state = sgr.gated_scan(f[:, :130].contiguous(), v[:, :130].contiguous())
    for t in range(130, T):
        y = sgr.gated_step(f[:, t], v[:, t], state)
        assert torch.allclose(y, whole[:, t], rtol=1e-5, atol=1e-6)
    assert torch.allclose(state, last, rtol=1e-5, atol=1e-6)


def test_step_captured():
    torch.manual_seed(5)
    f, v, state = torch.randn(6, 96, device=DEV), torch.randn(6, 96, device=DEV), torch.randn(6, 96, device=DEV)
    want = state.clone()
    for _ in range(4):
        sgr.gated_step(f, v, want)
    g = torch.cuda.CUDAGraph()
    warm = state.clone()
    sgr.gated_step(f, v, warm)
    with torch.cuda.graph(g):
        sgr.gated_step(f, v, state)
    for _ in range(4):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(state, want)


# ------------------------------------------------------------- segments
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bounds", [
    [0, 4000, 4001, 9000, 9000, 15000, 16001],              # many segments, at uneven bounds
    [0, 16001],                                             # one sequence: one segment's worth
    [5, 100, 15900],                                        # a short first sequence, padding at both ends
    list(range(0, 16002, 127)) + [16001],                   # sequences shorter than a tile
])
def test_rows_cut_into_segments(bounds, dtype):
    rng = np.random.default_rng(len(bounds))
    rows, D, n = 16001, 24, len(bounds) - 1
    f, v, f64, v64 = make(rng, "sigmoid", rows, D, dtype)
    h0 = rng.normal(size=(n, D)).astype(np.float32)
    h0_d, cu = torch.from_numpy(h0).to(DEV), torch.tensor(bounds, device=DEV)
    h, last, states = sgr.gated_scan(f, v, h0_d, cu, save_states=True)
    want, wl, bh, bl = scan64(f64, v64, h0.astype(np.float64), bounds, "sigmoid", dtype)
    check(h, want, bh, dtype, "h")
    check(last, wl, bl, F32, "h_last")
    dh = torch.from_numpy(rng.normal(size=(rows, D))).to(dtype)
    df, dv, d0 = sgr.gated_scan_backward(f, v, h0_d, states, dh.to(DEV), None, cu)
    wf, wv, w0, bf, bv, b0 = grad64(f64, v64, h0.astype(np.float64), bounds, "sigmoid", dh.double().numpy(), None, dtype)
    check(df, wf, bf, dtype, "df")
    check(dv, wv, bv, dtype, "dv")
    check(d0, w0, b0, F32, "dh0")
    # an upstream gradient on unaligned rows takes another path than the forward did: the same places of the states
    odd = torch.zeros(rows, D + 1, dtype=dtype, device=DEV)[:, 1:]
    odd.copy_(dh)
    for a, b in zip(sgr.gated_scan_backward(f, v, h0_d, states, odd, None, cu), (df, dv, d0)):
        assert torch.equal(a, b) or torch.allclose(a.float(), b.float(), rtol=0.02, atol=1e-4)


def test_offsets_past_32_bits():
    """Arrays of more than 2^31 elements: the last channels and rows against
    the same columns in a call of their own (one sequence, so the rows are cut
    into the same tiles and the bits are equal)."""
    rows, D = 70016, 31360                                   # 2.2e9 elements, 4.4 GB each in bf16
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs 20 GB of device memory")
    g = torch.Generator(device=DEV).manual_seed(1)
    f = torch.empty(rows, D, dtype=BF16, device=DEV).normal_(generator=g)
    v = torch.empty(rows, D, dtype=BF16, device=DEV).normal_(generator=g)
    h, last, states = sgr.gated_scan(f, v, save_states=True)
    cols = slice(D - 64, D)
    h1, last1, states1 = sgr.gated_scan(f[:, cols].contiguous(), v[:, cols].contiguous(), save_states=True)
    assert torch.equal(h[:, cols], h1) and torch.equal(last[:, cols], last1)
    df, dv, _ = sgr.gated_scan_backward(f, v, None, states, h)
    df1, dv1, _ = sgr.gated_scan_backward(f[:, cols].contiguous(), v[:, cols].contiguous(), None, states1, h1)
    assert torch.equal(df[:, cols], df1) and torch.equal(dv[:, cols], dv1)


def test_autograd_captured_forward_and_backward():
    torch.manual_seed(7)
    shape = (2, 500, 64)
    f, v, dh = (torch.randn(shape, device=DEV) for _ in range(3))
    f.requires_grad_(True)
    v.requires_grad_(True)

    def step():
        h, _ = sgr.gated_scan_fn(f, v)
        return torch.autograd.grad(h, [f, v], dh)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            want = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_saved_tensors_laid_out_anew():
    """Hooks that move what is saved to the host and back give other strides."""
    torch.manual_seed(9)
    both = torch.randn(300, 96, device=DEV)
    states = torch.randn(3, 96, device=DEV)
    cu = torch.tensor([0, 10, 200, 300], device=DEV)
    dh = torch.randn(300, 48, device=DEV)
    got = []
    for hooks in (False, True):
        f, v = both[:, :48].detach().requires_grad_(True), both[:, 48:].detach().requires_grad_(True)
        h0 = states[:, 5:53].detach().requires_grad_(True)
        if hooks:
            with torch.autograd.graph.save_on_cpu():
                h, _ = sgr.gated_scan_fn(f, v, h0, cu)
        else:
            h, _ = sgr.gated_scan_fn(f, v, h0, cu)
        got.append(torch.autograd.grad(h, [f, v, h0], dh))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_broadcast_operands_and_their_gradients():
    """One row of values for every token (row stride 0): read in place, its
    gradient the sum over the rows; a batch dimension of stride 0 is refused."""
    torch.manual_seed(4)
    T, D = 250, 40
    f = torch.randn(T, D, device=DEV, requires_grad=True)
    row = torch.randn(1, D, device=DEV, requires_grad=True)
    dh = torch.randn(T, D, device=DEV)
    h, _ = sgr.gated_scan_fn(f, row.expand(T, D))
    got = torch.autograd.grad(h, [f, row], dh)
    f64 = f.detach().double().cpu().numpy()
    v64 = row.detach().double().cpu().numpy().repeat(T, 0)
    want, _, b, _ = scan64(f64, v64, np.zeros((1, D)), [0, T], "sigmoid")
    check(h, want, b, F32, "h")
    wf, wv, _, bf, bv, _ = grad64(f64, v64, np.zeros((1, D)), [0, T], "sigmoid", dh.double().cpu().numpy(), None)
    check(got[0], wf, bf, F32, "df")
    check(got[1], wv.sum(0, keepdims=True), (bv + T * 2.0 ** -24 * np.abs(wv)).sum(0, keepdims=True), F32, "row")
    with pytest.raises(ValueError, match="evenly spaced"):
        sgr.gated_scan(f[None].expand(2, T, D), f[None].expand(2, T, D))


def test_many_sequences_most_of_them_empty():
    rng = np.random.default_rng(3)
    rows, D, n = 900, 20, 30000
    bounds = np.sort(rng.integers(0, rows + 1, n - 1)).tolist()
    cu = [0, *bounds, rows]
    f, v, f64, v64 = make(rng, "log", rows, D, F32)
    h0 = rng.normal(size=(n, D)).astype(np.float32)
    h0_d, cu_d = torch.from_numpy(h0).to(DEV), torch.tensor(cu, dtype=torch.int32, device=DEV)
    h, last, states = sgr.gated_scan(f, v, h0_d, cu_d, "log", save_states=True)
    want, wl, bh, bl = scan64(f64, v64, h0.astype(np.float64), cu, "log")
    check(h, want, bh, F32, "h")
    check(last, wl, bl, F32, "h_last")
    dh = torch.randn(rows, D, device=DEV)
    dl = torch.randn(n, D, device=DEV)
    df, dv, d0 = sgr.gated_scan_backward(f, v, h0_d, states, dh, dl, cu_d, "log")
    wf, wv, w0, bf, bv, b0 = grad64(f64, v64, h0.astype(np.float64), cu, "log", dh.double().cpu().numpy(),
                                    dl.double().cpu().numpy())
    check(df, wf, bf, F32, "df")
    check(dv, wv, bv, F32, "dv")
    check(d0, w0, b0, F32, "dh0")


def in_new_thread(work):
    with concurrent.futures.ThreadPoolExecutor(1) as pool:
        return pool.submit(work).result(timeout=60)


@pytest.mark.parametrize("dtype", [F32, torch.bfloat16, torch.float16])
def test_first_call_of_a_thread(dtype):
    """A thread that has launched nothing yet, with memory at hand: short
    scans (one tile, no workspace to clear first) in both directions."""
    f = torch.randn(2, 24, 64, device=DEV).to(dtype)
    v, dh = torch.randn_like(f), torch.randn_like(f)
    *want, states = sgr.gated_scan(f, v, save_states=True)
    back = sgr.gated_scan_backward(f, v, None, states, dh)
    torch.cuda.synchronize()
    got = in_new_thread(lambda: sgr.gated_scan(f, v))
    grads = in_new_thread(lambda: sgr.gated_scan_backward(f, v, None, states, dh))
    torch.cuda.synchronize()
    for a, b in zip([*got, *grads], [*want, *back]):
        assert (a is None and b is None) or torch.equal(a, b)
