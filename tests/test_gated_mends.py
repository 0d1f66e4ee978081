"""The gated recurrence and the 8-bit projection without a GPU: layouts of
results, sizes at the ends of the index types, and the kernels' tables of a
tile replayed."""
import numpy as np
import pytest
import torch

from scan_gated_rnns_b200 import _abi, gated, ops

from test_abi import fake_addresses
from test_gated_host import segments


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


# ------------------------------------------------- the table of a tile
WARPS, LANES = 12, 32


def tile_table(rows, row0, row_end, tr, cu=None, seq_rows=None):
    """(masks, cut, start, end) of a tile as the feeding warp writes them, by its
    own steps; entries it leaves as they were are None."""
    R = tr // WARPS
    full = (1 << R) - 1
    start, end = [None] * tr, [None] * tr
    lo_row, hi_row = 0, rows

    def plain():
        start[0] = end[tr - 1] = -1
        return [(0, 0, full, 1)] * WARPS, 0, start, end

    if cu is None:
        s0 = row0 // seq_rows
        k0 = row0 - s0 * seq_rows
        if k0 > 0 and k0 + tr < seq_rows:
            return plain()
        for lane in range(LANES):
            s, k = divmod(row0 + lane, seq_rows)
            for r in range(lane, tr, LANES):
                inside = row0 + r < row_end
                start[r] = s if inside and k == 0 else -1
                end[r] = s if inside and k + 1 == seq_rows else -1
                k += LANES
                if k >= seq_rows:
                    s, k = s + k // seq_rows, k % seq_rows
    else:
        n_seqs = len(cu) - 1

        def at(i):
            assert 0 <= i <= n_seqs
            return max(-1, min(rows + 1, cu[i]))

        lo, hi = 0, n_seqs + 1
        while lo < hi:
            step = (hi - lo + 31) // 32
            n = sum(i < hi and at(i) <= row0 for i in (lo + (lane + 1) * step - 1 for lane in range(LANES)))
            lo, hi = min(lo + n * step, hi), min(lo + (n + 1) * step - 1, hi)
        if 0 < lo <= n_seqs and at(lo - 1) < row0 and at(lo) > row0 + tr and row0 + tr <= row_end:
            return plain()
        lo_row, hi_row = at(0), min(at(n_seqs), rows)
        start, end = [-1] * tr, [-1] * tr
        base, more = max(lo - 1, 0), True
        while more:
            more = False
            for s in range(base, min(base + LANES, n_seqs)):
                b, e = at(s), at(s + 1)
                more |= b < row_end
                if b < e:
                    if row0 <= b < row_end:
                        start[b - row0] = s
                    if row0 < e <= row_end:
                        end[e - 1 - row0] = s
            base += LANES
    masks = [None] * WARPS
    cut = 0
    for r0 in range(0, tr, LANES):
        word = [0, 0, 0]
        for lane in range(LANES):
            r = r0 + lane
            if r < tr:
                word[0] |= (start[r] >= 0) << lane
                word[1] |= (end[r] >= 0) << lane
                word[2] |= (lo_row <= row0 + r < hi_row and row0 + r < row_end) << lane
        cut |= (1 if word[0] else 0) | (2 if word[1] else 0)
        for lane in range(LANES // R):
            if r0 // R + lane < WARPS:
                a, b, c = (w >> (lane * R) & full for w in word)
                masks[r0 // R + lane] = (a, b, c, int(a == 0 and b == 0 and c == full))
    return masks, cut, start, end


def check_tables(rows, bounds, tr, cut_at, **kind):
    """Every tile of the segments that begin at cut_at against a direct count."""
    starts = {b: s for s, (b, e) in enumerate(zip(bounds, bounds[1:])) if b < e}
    ends = {e - 1: s for s, (b, e) in enumerate(zip(bounds, bounds[1:])) if b < e}
    R, seen_plain = tr // WARPS, 0
    for lo, hi in zip(cut_at, cut_at[1:] + [rows]):
        for row0 in range(lo, hi, tr):
            row_end = min(row0 + tr, hi)
            masks, cut, start, end = tile_table(rows, row0, row_end, tr, **kind)
            inside = range(row0, row_end)
            assert cut == (1 if any(r in starts for r in inside) else 0) | (2 if any(r in ends for r in inside) else 0)
            for w in range(WARPS):
                mine = [row0 + w * R + i for i in range(R)]
                a, b, c = (sum((r < row_end and test(r)) << i for i, r in enumerate(mine))
                           for test in (starts.__contains__, ends.__contains__, lambda r: bounds[0] <= r < bounds[-1]))
                assert masks[w] == (a, b, c, int(a == 0 and b == 0 and c == (1 << R) - 1)), (row0, w)
                for i, r in enumerate(mine):              # sequences are read where the masks say so
                    assert not a >> i & 1 or start[r - row0] == starts[r]
                    assert not b >> i & 1 or end[r - row0] == ends[r]
            # the carry's view: does the tile begin (end) with a sequence
            assert (start[0] >= 0) == (row0 in starts)
            assert (end[tr - 1] >= 0) == (row0 + tr <= row_end and row0 + tr - 1 in ends)
            seen_plain += start[1] is None
    return seen_plain


@pytest.mark.parametrize("tr", [96, 192])
def test_tables_of_packed_sequences(tr):
    rng = np.random.default_rng(tr)
    rows, plain = 2500, 0
    for trial in range(30):
        n = int(rng.integers(1, [3, 8, 60, 1500][trial % 4]))
        bounds = sorted(rng.integers(0, rows + 1, n - 1).tolist())
        bounds = [[0, *bounds, rows], [3, *[max(3, min(b, 2400)) for b in bounds], 2400]][trial % 2]
        if trial >= 20:                                   # at and next to the tiles' ends
            bounds = sorted({0, rows, *(tr * int(k) + int(d) for k, d in zip(rng.integers(1, 12, 5), rng.integers(-1, 2, 5)))})
            bounds = [b for b in bounds if b <= rows]
        for n_segs in (1, 4, 32):
            at, lens, _, _ = segments(bounds, rows, n_segs, tr)
            plain += check_tables(rows, bounds, tr, sorted(set(a for a, m in zip(at, lens) if m)), cu=bounds)
    assert plain > 100


@pytest.mark.parametrize("tr", [96, 192])
@pytest.mark.parametrize("seq_rows,n", [(1, 400), (5, 100), (96, 7), (97, 9), (191, 5), (192, 5), (193, 5), (1000, 3),
                                        (288, 8)])
def test_tables_of_sequences_of_one_length(seq_rows, n, tr):
    rows = seq_rows * n
    bounds = [i * seq_rows for i in range(n + 1)]
    for n_segs in (1, 3, 32):
        cut_at = sorted({(rows // n_segs * g + seq_rows // 2) // seq_rows * seq_rows for g in range(n_segs)} - {rows} | {0})
        check_tables(rows, bounds, tr, cut_at, seq_rows=seq_rows)


def test_bounds_out_of_order_or_range_stay_inside_both_tables():
    rng = np.random.default_rng(5)
    for tr in (96, 192):
        for n in (1, 3, 40, 200):
            for _ in range(10):
                cu = rng.integers(-(1 << 40), 1 << 40, n + 1).tolist() if n == 40 else rng.integers(-900, 2000, n + 1).tolist()
                for row0 in range(0, 700, tr):
                    _, _, start, end = tile_table(700, row0, min(row0 + tr, 700), tr, cu=cu)
                    assert all(x is None or -1 <= x < n for x in start + end)


# ---------------------------------------------------------- whole calls
@fake_addresses
def test_backward_arguments_that_pass_every_check():
    """The call that the refusals vary: only the launch fails (no device)."""
    A, B, C, D_, E_ = (i << 32 for i in range(1, 6))
    assert _abi.lib().gated_scan_backward(A, 8, B, 8, None, 0, None, 0, 2, C, D_, 8, None, E_, 8, 7 << 32, 8, None, 400, 8,
                                          0, 0, 6 << 32, 1 << 30, None) == _abi.SGR_ERR_CUDA
