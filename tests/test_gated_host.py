"""The gated recurrence and the 8-bit projection without a GPU: the 64-bit
reference against finite differences, the refusals of the C ABI and of the
Python binding, and the kernels' search for sequence bounds replayed on the
CPU, for bounds in order and for any others."""
import numpy as np
import pytest
import torch

from scan_gated_rnns_b200 import _abi, gated, int8, ops

from gated_reference import grad64, scan64
from test_abi import fake_addresses

TR = 96                                     # rows per tile of the kernels


# ------------------------------------------------------------- reference
@pytest.mark.parametrize("gate", ["sigmoid", "log"])
def test_reference_gradients_against_differences(gate):
    rng = np.random.default_rng(3)
    rows, D, cu = 13, 5, [0, 4, 4, 9, 13]
    f, v = rng.normal(size=(rows, D)), rng.normal(size=(rows, D))
    f = f if gate == "sigmoid" else -np.abs(f) - 0.01
    h0, dh, dl = rng.normal(size=(4, D)), rng.normal(size=(rows, D)), rng.normal(size=(4, D))

    def loss(f, v, h0):
        h, last, _, _ = scan64(f, v, h0, cu, gate)
        return (h * dh).sum() + (last * dl).sum()

    grads = grad64(f, v, h0, cu, gate, dh, dl)[:3]
    for i, x in enumerate((f, v, h0)):
        for _ in range(12):
            at = tuple(rng.integers(n) for n in x.shape)
            step = np.zeros_like(x)
            step[at] = 1e-5
            args = [f, v, h0]
            up, down = list(args), list(args)
            up[i], down[i] = x + step, x - step
            assert (loss(*up) - loss(*down)) / 2e-5 == pytest.approx(grads[i][at], rel=1e-6, abs=1e-8)


# ------------------------------------------------- bounds search, replayed
def fill_info(cu, rows, row0, row_end=None):
    """The table of a tile, lane by lane as the kernel fills it; every index is
    checked against its array."""
    n_seqs = len(cu) - 1
    start, end = [-1] * TR, [-1] * TR
    row_end = min(row0 + TR, rows) if row_end is None else row_end

    def at(i):
        assert 0 <= i <= n_seqs
        return cu[i]

    lo, hi, rounds = 0, n_seqs + 1, 0
    while lo < hi:
        rounds += 1
        assert rounds <= 16
        step = (hi - lo + 31) // 32
        probes = [lo + (lane + 1) * step - 1 for lane in range(32)]
        n = sum(i < hi and at(i) <= row0 for i in probes)
        nxt, top = lo + n * step, lo + (n + 1) * step - 1
        lo, hi = min(nxt, hi), min(top, hi)
    base = lo - 1 if lo > 0 else 0
    while True:
        more = False
        for s in range(base, base + 32):
            if s < n_seqs:
                b, e = at(s), at(s + 1)
                more |= b < row_end
                if b < e:
                    if row0 <= b < row_end:
                        start[b - row0] = s
                    if row0 < e <= row_end:
                        end[e - 1 - row0] = s
        base += 32
        if not more:
            return start, end


@pytest.mark.parametrize("seqs", [1, 2, 31, 32, 33, 40, 1000, 1100, 5000])
def test_bounds_search_finds_every_start_and_end(seqs):
    rng = np.random.default_rng(seqs)
    rows = 1500
    for trial in range(4):
        inner = np.sort(rng.integers(0, rows + 1, seqs - 1))
        cu = [0, *inner.tolist(), rows] if trial < 3 else [7, *np.clip(inner, 7, 1400).tolist(), 1400]
        want_s, want_e = {}, {}
        for s, (b, e) in enumerate(zip(cu, cu[1:])):
            if b < e:
                want_s[b], want_e[e - 1] = s, s
        got_s, got_e = {}, {}
        for row0 in range(0, rows, TR):
            start, end = fill_info(cu, rows, row0)
            got_s.update({row0 + r: s for r, s in enumerate(start) if s >= 0})
            got_e.update({row0 + r: s for r, s in enumerate(end) if s >= 0})
        assert got_s == want_s and got_e == want_e


def test_bounds_in_no_order_stay_inside_the_arrays():
    rng = np.random.default_rng(9)
    for seqs in (1, 3, 40, 200):
        for _ in range(20):
            cu = rng.integers(-5000, 5000, seqs + 1).tolist()
            for row0 in range(0, 700, TR):
                start, end = fill_info(cu, 700, row0)
                assert all(-1 <= s < seqs for s in start + end)


def segments(cu, rows, n_segs, tr):
    """(start, length, chunks, place of the first) of each segment, as the
    feeding warp finds them from any bounds."""
    n_seqs = len(cu) - 1
    clamp = [max(-1, min(rows + 1, b)) for b in cu]
    at = [0]
    for g in range(1, n_segs):
        ideal = rows // n_segs * g
        lo, hi = 0, n_seqs + 1
        while lo < hi:
            mid = (lo + hi) // 2
            if clamp[mid] <= ideal:
                lo = mid + 1
            else:
                hi = mid
        up = clamp[lo] if lo <= n_seqs else clamp[n_seqs]
        down = clamp[lo - 1] if lo > 0 else up
        x = down if ideal - down <= up - ideal else up
        at.append(max(at[-1], min(rows, max(0, x))))
    lens = [b - a for a, b in zip(at, at[1:] + [rows])]
    chunks = [-(-n // tr) for n in lens]
    return at, lens, chunks, [sum(chunks[:g]) for g in range(n_segs)]


def tiles_in_order(chunks):
    """(segment, place) of each chunk in processing order, by the kernel's stepping."""
    c = below = 0
    for k in range(sum(chunks)):
        live = [n > c for n in chunks]
        while k >= below + sum(live):
            steps = min((k - below) // sum(live), min(n for n in chunks if n > c) - c)
            c, below = c + steps, below + steps * sum(live)
            live = [n > c for n in chunks]
        yield [g for g, on in enumerate(live) if on][k - below], c


@pytest.mark.parametrize("n_segs", [1, 2, 5, 17, 32])
def test_segments_cover_the_rows_once_and_wait_for_earlier_tiles_only(n_segs):
    rng = np.random.default_rng(n_segs)
    for rows in (1, 500, 9001):
        for tr in (TR, 2 * TR):
            for trial in range(6):
                cu = np.sort(rng.integers(0, rows + 1, rng.integers(1, 60))).tolist()
                if trial == 4:
                    cu = [0, rows]
                if trial == 5:                          # in no order, out of range
                    cu = rng.integers(-rows, 3 * rows, 20).tolist()
                at, lens, chunks, first = segments(cu, rows, n_segs, tr)
                assert at[0] == 0 and sum(lens) == rows and min(lens) >= 0
                assert sum(chunks) <= -(-rows // tr) + n_segs - 1
                assert sum(-(-n // TR) for n in lens) <= _abi.lib().sgr_gated_chunks(rows) or n_segs > 1 and rows <= TR
                if trial < 5:                           # a segment never begins inside a sequence
                    inside = {r for b, e in zip(cu, cu[1:]) for r in range(b + 1, e)}
                    assert not inside & {a for a, n in zip(at, lens) if n}
                order = list(tiles_in_order(chunks))
                assert sorted(order) == sorted((g, c) for g, n in enumerate(chunks) for c in range(n))
                seen = set()
                for g, c in order:                      # the place before it in its segment came first
                    assert c == 0 or (g, c - 1) in seen
                    seen.add((g, c))


def test_chunks_and_workspace_sizes():
    lib = _abi.lib()
    assert [lib.sgr_gated_chunks(n) for n in (-1, 0, 1, TR, TR + 1, 10 * TR)] == [0, 0, 1, 1, 33, 41]
    assert lib.sgr_gated_workspace_size(TR, 4096) == 0
    need = lib.sgr_gated_workspace_size(1000, 100)
    assert need >= 256 + 11 * 128 * 8
    assert lib.sgr_gated_workspace_size(1 << 40, 4096) == 0
    assert lib.sgr_int8_workspace_size(10, 100, _abi.SGR_I8) == 0
    assert lib.sgr_int8_workspace_size(10, 100, _abi.SGR_F32) >= 10 * 112 + 40
    assert lib.sgr_int8_workspace_size(10, 1 << 17, _abi.SGR_F32) == 0


# ------------------------------------------------------------ C refusals
A, B, C, D_, E_ = (i << 32 for i in range(1, 6))
INVALID, UNSUPPORTED, WORKSPACE = _abi.SGR_ERR_INVALID_ARG, _abi.SGR_ERR_UNSUPPORTED, _abi.SGR_ERR_WORKSPACE


def scan_call(**kw):
    a = dict(f=A, f_rs=8, v=B, v_rs=8, h0=None, h0_ss=0, cu=None, cu_bytes=0, n=2, h=C, h_rs=8, last=None, states=None,
             rows=400, D=8, gate=0, dtype=0, zero=1, ws=D_, wn=1 << 30, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return _abi.lib().gated_scan(*a.values())


@fake_addresses
@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), INVALID), (dict(dtype=9), INVALID), (dict(gate=2), INVALID), (dict(rows=-1), INVALID),
    (dict(D=-1), INVALID), (dict(n=-1), INVALID), (dict(n=0), INVALID), (dict(n=3), INVALID),
    (dict(cu=E_, cu_bytes=2), INVALID), (dict(f=None), INVALID), (dict(v=None), INVALID), (dict(h=None), INVALID),
    (dict(f_rs=-8), INVALID), (dict(h_rs=7), INVALID), (dict(h=A), INVALID), (dict(h=B + 400 * 32 - 4), INVALID),
    (dict(last=A), INVALID), (dict(states=B), INVALID), (dict(ws=A), INVALID), (dict(h0=C, h0_ss=8), INVALID),
    (dict(ws=None), WORKSPACE), (dict(wn=100), WORKSPACE), (dict(ws=D_ + 4), WORKSPACE),
    (dict(rows=1 << 40), UNSUPPORTED), (dict(rows=1 << 20, D=1 << 44, f_rs=1 << 44, v_rs=1 << 44, h_rs=1 << 44), UNSUPPORTED),
    (dict(rows=0, n=0), 0), (dict(D=0), 0),
])
def test_scan_refusals(kw, code):
    assert scan_call(**kw) == code


@fake_addresses
@pytest.mark.parametrize("kw,code", [
    (dict(), None), (dict(states=None), INVALID), (dict(dh=None), INVALID), (dict(df=None), INVALID),
    (dict(dv=None), INVALID), (dict(df_rs=7), INVALID), (dict(dv_rs=7), INVALID), (dict(df=A), INVALID),
    (dict(dv=6 << 32), INVALID), (dict(dh0=A), INVALID), (dict(ws=None), WORKSPACE),
])
def test_backward_refusals(kw, code):
    a = dict(f=A, f_rs=8, v=B, v_rs=8, h0=None, h0_ss=0, cu=None, cu_bytes=0, n=2, states=C, dh=D_, dh_rs=8, dl=None,
             df=E_, df_rs=8, dv=7 << 32, dv_rs=8, dh0=None, rows=400, D=8, gate=0, dtype=0, ws=6 << 32, wn=1 << 30,
             stream=None)
    if code is None:
        return
    a.update(kw)
    assert _abi.lib().gated_scan_backward(*a.values()) == code


@fake_addresses
@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), INVALID), (dict(gate=5), INVALID), (dict(rows=-1), INVALID), (dict(n=3), INVALID),
    (dict(slots=D_, sb=2), INVALID), (dict(h=A), INVALID), (dict(h=C), INVALID), (dict(state=A), INVALID),
    (dict(srs=7), INVALID), (dict(h_rs=7), INVALID), (dict(f=None), INVALID), (dict(state=None), INVALID),
    (dict(rows=0), 0), (dict(D=0), 0),
])
def test_step_refusals(kw, code):
    a = dict(f=A, f_rs=8, v=B, v_rs=8, state=C, srs=8, n=4, slots=None, sb=0, h=E_, h_rs=8, rows=4, D=8, gate=0,
             dtype=0, zero=1, stream=None)
    a.update(kw)
    assert _abi.lib().gated_step(*a.values()) == code


@fake_addresses
@pytest.mark.parametrize("kw,code", [
    (dict(xdt=5), INVALID), (dict(ydt=3), INVALID), (dict(xs=None), INVALID), (dict(xdt=0), INVALID),
    (dict(K=0), INVALID), (dict(rows=-1), INVALID), (dict(y_rs=7), INVALID), (dict(y=A), INVALID),
    (dict(w=None), INVALID), (dict(ws_=None), INVALID), (dict(K=1 << 17, x_rs=1 << 17, w_rs=1 << 17), UNSUPPORTED),
    (dict(xdt=0, xs=None, ws=None, wn=0), WORKSPACE), (dict(xdt=0, xs=None, wn=16), WORKSPACE),
    (dict(rows=0), 0), (dict(N=0), 0),
])
def test_projection_refusals(kw, code):
    a = dict(x=A, x_rs=16, xdt=3, xs=B, w=C, w_rs=16, ws_=D_, bias=None, y=E_, y_rs=8, ydt=0, rows=4, K=16, N=8,
             ws=6 << 32, wn=1 << 20, stream=None)
    a.update(kw)
    assert _abi.lib().int8_projection(*a.values()) == code


@fake_addresses
def test_quantize_refusals():
    q = _abi.lib().int8_quantize
    assert q(A, 8, B, 8, C, 4, 8, 3, None) == INVALID
    assert q(A, 8, B, 7, C, 4, 8, 0, None) == INVALID
    assert q(A, 8, A, 8, C, 4, 8, 0, None) == INVALID
    assert q(A, 8, B, 8, None, 4, 8, 0, None) == INVALID
    assert q(A, 8, B, 8, C, -4, 8, 0, None) == INVALID
    assert q(None, 8, None, 8, C, 0, 8, 0, None) == 0


def test_other_entry_points_refuse_the_new_types():
    lib = _abi.lib()
    for dt in (_abi.SGR_F16, _abi.SGR_I8):
        assert lib.mingru_scan(A, B, None, 0, C, 2, 4, 8, dt, D_, 1 << 20, None) == INVALID
        assert lib.mingru_step(A, 8, B, 8, None, 0, C, 8, 2, 8, dt, None) == INVALID


# ------------------------------------------------------- Python refusals
@pytest.fixture
def cpu_tensors(monkeypatch):
    monkeypatch.setattr(ops, "_need_cuda", lambda t, name: None)


def test_row_strides():
    x = torch.zeros(4, 6, 16)
    assert gated._row_stride(x, "x") == 16
    assert gated._row_stride(x[..., 8:], "x") == 16
    assert gated._row_stride(x[:, :1], "x") == 96
    assert gated._row_stride(x[:1, :3], "x") == 16
    assert gated._row_stride(torch.zeros(16), "x") == 16
    assert gated._row_stride(torch.zeros(2, 3, 4, 5), "x") == 5
    assert gated._row_stride(torch.zeros(3, 1).expand(3, 1), "x") == 1
    assert gated._row_stride(torch.zeros(1, 8).expand(5, 8), "x") == 0
    for bad in (x[:, :3], x.transpose(0, 1), x.transpose(1, 2), x[..., ::2]):
        with pytest.raises(ValueError):
            gated._row_stride(bad, "x")


def test_scan_argument_errors(cpu_tensors):
    f = torch.zeros(2, 3, 8)
    rows = torch.zeros(6, 8)
    cu = torch.tensor([0, 2, 6])
    bad = [
        (ValueError, lambda: gated.gated_scan(f, f, gate="tanh")),
        (ValueError, lambda: gated.gated_scan(f, f, gate=None)),
        (TypeError, lambda: gated.gated_scan(f.double(), f.double())),
        (ValueError, lambda: gated.gated_scan(f, f.half())),
        (ValueError, lambda: gated.gated_scan(f, f[:1])),
        (ValueError, lambda: gated.gated_scan(f, f, cu_seqlens=cu)),
        (ValueError, lambda: gated.gated_scan(rows, rows, cu_seqlens=cu.float())),
        (ValueError, lambda: gated.gated_scan(rows, rows, cu_seqlens=cu[None])),
        (ValueError, lambda: gated.gated_scan(rows, rows, cu_seqlens=cu[:0])),
        (ValueError, lambda: gated.gated_scan(f, f, h0=torch.zeros(3, 8))),
        (ValueError, lambda: gated.gated_scan(f, f, h0=torch.zeros(2, 8).half())),
        (ValueError, lambda: gated.gated_scan(f, f, h0=torch.zeros(7))),
        (ValueError, lambda: gated.gated_scan(f, f, out=torch.zeros(2, 3, 9))),
        (ValueError, lambda: gated.gated_scan(torch.zeros(8), torch.zeros(8))),
        (ValueError, lambda: gated.gated_scan_backward(f, f, None, None, f)),
        (ValueError, lambda: gated.gated_scan_backward(f, f, None, torch.zeros(2, 8), f)),
        (ValueError, lambda: gated.gated_scan_backward(f, f, None, torch.zeros(1, 8), f[:1])),
        (ValueError, lambda: gated.gated_scan_backward(f, f, None, torch.zeros(1, 8), f, torch.zeros(8))),
        (ValueError, lambda: gated.gated_step(rows, rows, torch.zeros(6, 7))),
        (ValueError, lambda: gated.gated_step(rows, rows, torch.zeros(5, 8))),
        (ValueError, lambda: gated.gated_step(f, f, torch.zeros(6, 8))),
        (ValueError, lambda: gated.gated_step(rows, rows, torch.zeros(6, 8).double())),
        (ValueError, lambda: gated.gated_step(rows, rows, torch.zeros(6, 8), torch.zeros(5, dtype=torch.int32))),
        (ValueError, lambda: gated.gated_step(rows, rows, torch.zeros(6, 8), torch.zeros(6))),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()


def test_projection_argument_errors(cpu_tensors):
    x, w, s = torch.zeros(4, 16), torch.zeros(8, 16, dtype=torch.int8), torch.zeros(8)
    xq = torch.zeros(4, 16, dtype=torch.int8)
    bad = [
        (ValueError, lambda: int8.int8_projection(x, w, s, x_scale=torch.zeros(4))),
        (ValueError, lambda: int8.int8_projection(xq, w, s)),
        (TypeError, lambda: int8.int8_projection(x.double(), w, s)),
        (ValueError, lambda: int8.int8_projection(x, w.float(), s)),
        (ValueError, lambda: int8.int8_projection(x, w[:, :8], s)),
        (ValueError, lambda: int8.int8_projection(x, w, s[:7])),
        (ValueError, lambda: int8.int8_projection(x, w, s.half())),
        (ValueError, lambda: int8.int8_projection(x, w, s, bias=torch.zeros(9))),
        (ValueError, lambda: int8.int8_projection(xq, w, s, x_scale=torch.zeros(3))),
        (TypeError, lambda: int8.int8_projection(x, w, s, out_dtype=torch.float64)),
        (ValueError, lambda: int8.int8_projection(x, w, s, out=torch.zeros(4, 9))),
        (ValueError, lambda: int8.int8_projection(x, w, s, out=torch.zeros(4, 8), out_dtype=torch.float16)),
        (ValueError, lambda: int8.int8_projection(x[:, :0], w[:, :0], s)),
        (TypeError, lambda: int8.int8_quantize(x.double())),
        (ValueError, lambda: int8.int8_quantize(x.t())),
        (ValueError, lambda: int8.int8_quantize(torch.zeros(()))),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()


def test_cpu_tensors_are_refused():
    x = torch.zeros(2, 3, 8)
    for call in (lambda: gated.gated_scan(x, x), lambda: gated.gated_step(x[0], x[0], x[0]),
                 lambda: int8.int8_quantize(x), lambda: int8.int8_projection(x, x[0].to(torch.int8), x[0, :, 0])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
