"""int8_quantize and int8_projection on the GPU against whole-number and
64-bit arithmetic, and the layer's path: projection, scan, steps.

Tolerances: the sum is exact; float(sum) rounds once (2^-24), then one product
and one fma round once each, so y is within 3 2^-24 (|s_x s_w sum| + |bias|)
before the half step of its type."""
import concurrent.futures

import numpy as np
import pytest
import torch

import scan_gated_rnns_b200 as sgr

from gated_reference import check, quantize64, scan64

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

DEV = torch.device("cuda:0")
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


# ------------------------------------------------------------- quantise
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 15), (8, 16), (5, 127), (70, 1000), (33, 4096), (2, 20001), (3000, 64)])
def test_quantize_is_exact(rows, K, dtype):
    rng = np.random.default_rng(rows + K)
    x = torch.from_numpy(rng.normal(size=(rows, K)) * np.exp(rng.normal(size=(rows, 1)) * 3)).to(dtype)
    x[rows // 2, K // 2] = 0
    q, s = sgr.int8_quantize(x.to(DEV))
    wq, ws = quantize64(x.double().numpy())
    assert q.stride(0) % 16 == 0 and q.data_ptr() % 16 == 0
    assert np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(q.cpu().numpy().astype(np.int64), wq)


def test_quantize_ties_zeros_and_odd_rows():
    # quotients exactly on a half: scale 1 (largest value 127), values k + 1/2
    ties = torch.arange(-126, 127, dtype=F32) + 0.5
    x = torch.cat([ties, torch.tensor([127.0])])
    # and next to a half, one step of the type to either side, with a scale that is no power of two
    s = np.float32(np.float32(5.3) * (np.float32(1) / np.float32(127)))
    near = torch.from_numpy((np.arange(-126, 127) + 0.5).astype(np.float32) * s)
    rows = torch.stack([x, torch.cat([near, torch.tensor([5.3])]),
                        torch.cat([torch.nextafter(near, torch.tensor(1e9)), torch.tensor([5.3])]),
                        torch.cat([torch.nextafter(near, torch.tensor(-1e9)), torch.tensor([5.3])]),
                        torch.zeros(254), torch.full((254,), 1e-40), torch.full((254,), -3e38),
                        torch.full((254,), 2.0 ** -99)])
    q, sc = sgr.int8_quantize(rows.to(DEV))
    wq, ws = quantize64(rows.double().numpy())
    assert np.array_equal(sc.cpu().numpy(), ws) and np.array_equal(q.cpu().numpy().astype(np.int64), wq)
    bad = torch.randn(4, 40)
    bad[1, 3], bad[2, 39], bad[3, 0] = float("nan"), float("inf"), float("-inf")
    q, sc = sgr.int8_quantize(bad.to(DEV))
    assert torch.isfinite(sc).tolist() == [True, False, False, False] and bool(torch.isnan(sc[1:]).all())
    assert bool((q[1:] == 0).all()) and int(q[0].abs().max()) == 127


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_scales_of_many_magnitudes(dtype):
    """|x| times 1/127 over all exponents; q is then 127 or -127."""
    rng = np.random.default_rng(5)
    x = rng.normal(size=300000) * np.exp2(rng.integers(-120, 120, 300000).astype(np.float64) * (0.1 if dtype == F16 else 1))
    x = torch.from_numpy(x).to(dtype)[:, None]
    q, s = sgr.int8_quantize(x.to(DEV))
    wq, ws = quantize64(x.double().numpy())
    assert np.array_equal(s.cpu().numpy(), ws, equal_nan=True)
    assert np.array_equal(q.cpu().numpy().astype(np.int64), wq)


def test_quantize_layouts():
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.normal(size=(4, 6, 50))).to(BF16).to(DEV)
    for view in (x, x[..., 1:40], x[:, :1], x[0, 0], x[:, :, :0]):
        q, s = sgr.int8_quantize(view)
        assert q.shape == view.shape and s.shape == view.shape[:-1]
        if view.numel():
            wq, ws = quantize64(view.double().cpu().numpy().reshape(-1, view.shape[-1]))
            assert np.array_equal(q.cpu().numpy().reshape(wq.shape), wq)
            assert np.array_equal(s.cpu().numpy().reshape(-1), ws)


# ----------------------------------------------------------- projection
def whole(rng, rows, K, lo=-127, hi=127):
    return rng.integers(lo, hi + 1, (rows, K)).astype(np.int8)


def on_gpu(q, layout):
    rows, K = q.shape
    t = torch.from_numpy(q)
    if layout == "padded":
        buf = torch.full((rows, -(-K // 16) * 16 + 16), 99, dtype=torch.int8, device=DEV)
        buf[:, :K] = t.to(DEV)
        return buf[:, :K]
    if layout == "odd":
        buf = torch.full((rows, K + 5), 99, dtype=torch.int8, device=DEV)
        buf[:, 3:3 + K] = t.to(DEV)
        return buf[:, 3:3 + K]
    return t.to(DEV)


def product_case(M, K, N, out, x_layout, w_layout, bias, seed=0, lo=-127):
    rng = np.random.default_rng(seed + M + K + N)
    xq, wq = whole(rng, M, K, lo), whole(rng, N, K, lo)
    xs, ws = np.exp(rng.normal(size=M)).astype(np.float32) / 100, np.exp(rng.normal(size=N)).astype(np.float32) / 100
    b = rng.normal(size=N).astype(np.float32) if bias else None
    y = sgr.int8_projection(on_gpu(xq, x_layout), on_gpu(wq, w_layout), torch.from_numpy(ws).to(DEV),
                            x_scale=torch.from_numpy(xs).to(DEV),
                            bias=torch.from_numpy(b).to(DEV) if bias else None, out_dtype=out)
    acc = np.rint(xq.astype(np.float64) @ wq.astype(np.float64).T)
    prod = acc * xs.astype(np.float64)[:, None] * ws.astype(np.float64)
    want = prod + (b.astype(np.float64) if bias else 0.0)
    check(y, want, 3 * 2.0 ** -24 * (np.abs(prod) + (np.abs(b) if bias else 0.0)), out, "y")


@pytest.mark.parametrize("out", [F32, BF16, F16])
@pytest.mark.parametrize("layouts", [("plain", "plain"), ("padded", "padded"), ("odd", "padded"), ("padded", "odd")])
@pytest.mark.parametrize("M,K,N", [(1, 1, 1), (1, 16, 128), (2, 31, 5), (8, 1024, 256), (16, 64, 130), (17, 200, 257),
                                   (100, 1000, 301), (129, 128, 128), (257, 528, 129), (300, 2080, 640)])
def test_products(M, K, N, layouts, out):
    product_case(M, K, N, out, *layouts, bias=(M + N) % 2 == 0)


@pytest.mark.parametrize("M", [1, 3, 7, 9, 15, 31, 32, 33, 63, 64, 65, 127, 128, 200, 256, 511, 1030])
@pytest.mark.parametrize("K,N", [(1024, 384), (4096, 2048)])
def test_products_of_every_height(M, K, N):
    product_case(M, K, N, BF16, "padded", "padded", bias=False, seed=5)


def test_product_of_extreme_values():
    """All -128: the largest sums, up to the longest rows."""
    for K in (4096, (1 << 17) - 1):
        x = torch.full((3, K + 1 if K % 16 else K), -128, dtype=torch.int8, device=DEV)[:, :K]
        w = torch.full((130, K + 1 if K % 16 else K), -128, dtype=torch.int8, device=DEV)[:, :K]
        y = sgr.int8_projection(x, w, torch.ones(130, device=DEV), x_scale=torch.ones(3, device=DEV))
        assert y.dtype == F32 and bool((y == float(np.float32(K * 128 * 128))).all())


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("M,K,N", [(1, 40, 33), (8, 1024, 512), (12, 1000, 300), (40, 260, 200), (600, 1024, 640)])
def test_products_quantised_within_the_call(M, K, N, dtype):
    rng = np.random.default_rng(M)
    x = torch.from_numpy(rng.normal(size=(M, K)) * np.exp(rng.normal(size=(M, 1)))).to(dtype).to(DEV)
    w = torch.from_numpy(rng.normal(size=(N, K))).float().to(DEV)
    wq, ws = sgr.int8_quantize(w)
    y = sgr.int8_projection(x, wq, ws)
    assert y.dtype == dtype and y.shape == (M, N)
    q, s = quantize64(x.double().cpu().numpy())
    prod = (q @ wq.cpu().numpy().astype(np.int64).T) * s.astype(np.float64)[:, None] * ws.double().cpu().numpy()
    check(y, prod, 3 * 2.0 ** -24 * np.abs(prod), dtype, "y")
    xq, xs = sgr.int8_quantize(x)                             # the two-step form: the same bits
    assert torch.equal(sgr.int8_projection(xq, wq, ws, x_scale=xs, out_dtype=dtype), y)


def test_bad_tokens_poison_their_rows_only():
    torch.manual_seed(0)
    for M in (4, 40, 300):
        x = torch.randn(M, 256, device=DEV)
        wq, ws = sgr.int8_quantize(torch.randn(192, 256, device=DEV))
        clean = sgr.int8_projection(x, wq, ws)
        x[1, 7], x[3, 0] = float("nan"), float("inf")
        y = sgr.int8_projection(x, wq, ws)
        keep = [i for i in range(M) if i not in (1, 3)]
        assert bool(torch.isnan(y[[1, 3]]).all()) and torch.equal(y[keep], clean[keep])


def test_outputs_in_place_of_others():
    """Leading dimensions, a given output with spaced rows, and what lies between them."""
    torch.manual_seed(1)
    for N in (96, 130):
        x = torch.randn(3, 50, 128, device=DEV, dtype=BF16)
        wq, ws = sgr.int8_quantize(torch.randn(N, 128, device=DEV))
        y = sgr.int8_projection(x, wq, ws)
        buf = torch.full((3, 50, N + 7), 5.0, dtype=BF16, device=DEV)
        got = sgr.int8_projection(x, wq, ws, out=buf[..., 2:2 + N])
        assert torch.equal(got, y) and bool((buf[..., :2] == 5).all()) and bool((buf[..., 2 + N:] == 5).all())
        assert sgr.int8_projection(x[:0], wq, ws).shape == (0, 50, N)


def test_streams_and_graphs():
    torch.manual_seed(2)
    wq, ws = sgr.int8_quantize(torch.randn(512, 1024, device=DEV))
    for M in (4, 40, 700):
        x, x2 = torch.randn(M, 1024, device=DEV, dtype=BF16), torch.randn(M, 1024, device=DEV, dtype=BF16)
        want, want2 = sgr.int8_projection(x, wq, ws), sgr.int8_projection(x2, wq, ws)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        graphs, outs = [], []
        for a in (x, x2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                outs.append(sgr.int8_projection(a, wq, ws))
            graphs.append(g)
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for _ in range(6):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want2)


# ------------------------------------------------------------- together
@pytest.mark.parametrize("gate", ["sigmoid", "log"])
def test_projection_scan_and_steps(gate):
    """A recurrent layer as it is served: prompts of several requests through
    the 8-bit projection, gates and values scanned in place of its output,
    then tokens one by one on the states left behind."""
    rng = np.random.default_rng(0)
    d_in, D, lens = 192, 96, [70, 1, 0, 200, 33]
    N = sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    wq, ws = sgr.int8_quantize(torch.from_numpy(rng.normal(size=(2 * D, d_in)) / 10).float().to(DEV))
    bias = torch.zeros(2 * D, device=DEV)
    bias[:D] = 1.0 if gate == "sigmoid" else -2.0
    x = torch.from_numpy(rng.normal(size=(N, d_in))).to(BF16).to(DEV)
    y = sgr.int8_projection(x, wq, ws, bias=bias)
    h, state = sgr.gated_scan(y[:, :D], y[:, D:], None, torch.tensor(cu, device=DEV), gate)
    y64 = y.double().cpu().numpy()
    want, wl, bh, bl = scan64(y64[:, :D], y64[:, D:], np.zeros((5, D)), cu, gate, BF16)
    check(h, want, bh, BF16, "h")
    check(state, wl, bl, F32, "states")
    slots = torch.tensor([4, 0, 2], device=DEV)
    for _ in range(3):
        tok = torch.from_numpy(rng.normal(size=(3, d_in))).to(BF16).to(DEV)
        y = sgr.int8_projection(tok, wq, ws, bias=bias)
        before = state.double().cpu().numpy()
        out = sgr.gated_step(y[:, :D], y[:, D:], state, slots, gate)
        y64 = y.double().cpu().numpy()
        want, _, b, _ = scan64(y64[:, :D], y64[:, D:], before[[4, 0, 2]], [0, 1, 2, 3], gate, BF16)
        check(out, want, b, BF16, "token")


@pytest.mark.parametrize("M", [4, 300])
def test_first_call_of_a_thread(M):
    """A thread that has launched nothing yet, with memory at hand."""
    rng = np.random.default_rng(M)
    x, w = (torch.from_numpy(whole(rng, rows, 256).astype(np.int8)).to(DEV) for rows in (M, 384))
    sx, sw = torch.rand(M, device=DEV), torch.rand(384, device=DEV)
    want = sgr.int8_projection(x, w, sw, x_scale=sx)
    torch.cuda.synchronize()
    with concurrent.futures.ThreadPoolExecutor(1) as pool:
        got = pool.submit(lambda: sgr.int8_projection(x, w, sw, x_scale=sx)).result(timeout=60)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
