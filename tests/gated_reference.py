"""The gated linear recurrence and the 8-bit projection in 64 bits, token by
token, with bounds on the error an fp32 evaluation may have.

The bounds are a running error analysis: the error e of a state obeys the
recurrence itself, e_t = a_t e_{t-1} + d_t, where d_t is what step t adds:
the error of a_t (times the largest state |h| could be), that of b_t, and two
fp32 roundings.  Errors of the gates (fp32 evaluation by the hardware's 2^x
and 1/x, relative error 2^-22 and 2^-23 each, after a product f log2(e) whose
rounding is |f| 2^-24 in the exponent):
  sigmoid: both a and 1 - a to (2^-21 + |f| 2^-23) min(a, 1 - a), and a
           rounding 2^-24 of the larger one;
  log:     a to 2^-23 a where f > -1/4 (series), else (2^-21 + |f| 2^-23) a;
  16-bit I/O, log: 2^-21 + |f| 2^-23 everywhere.
  16-bit I/O, sigmoid: a = 1 / (1 + 2^x), the sum rounded (2^-24) and the
           reciprocal off by 2^-23, so 2^-22 a on top of the above, and 1 - a
           is off by as much and its own rounding, 2^-24; the same in the
           gradients.
The hardware's 2^x gives 0 for results below 2^-126, the smallest normal
number, so a probability or decay is off by at most 2^-126 there whatever its
relative error: that much is added to each.
The factor 4 covers the tile-wise evaluation (a run of rows folded into one
map, maps applied in turn: each operation of the sequential form appears at
most a few times).  Outputs add half a step of their type."""
import numpy as np
import torch

TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24}


def gate64(f, v, gate, precise):
    """a, b (of a h + b), z, and the errors of a and b."""
    with np.errstate(all="ignore"):
        rel = 2.0 ** -21 + np.abs(f) * 2.0 ** -23
        if gate == "sigmoid":
            e = np.exp(-np.abs(f))
            small, big = e / (1 + e), 1 / (1 + e)
            a, z = np.where(f >= 0, big, small), np.where(f >= 0, small, big)
            err = np.where(small == 0, 0.0, rel * small + 2.0 ** -126)
            a, z = np.where(np.isnan(f), np.nan, a), np.where(np.isnan(f), np.nan, z)
            if not precise:
                err = err + 2.0 ** -22 * a
                return a, z * v, z, err, (err + 2.0 ** -24 + 2.0 ** -23 * z) * np.abs(v)
            return a, z * v, z, err + 2.0 ** -24 * a, (err + 2.0 ** -23 * z) * np.abs(v)
        x = np.where(f > 0, 0.0, f)
        a = np.exp(x)
        near = 2.0 ** -23 if precise else rel
        ea = np.where(a == 0, 0.0, np.where(x > -0.25, near, rel) * a + 2.0 ** -126)
        return a, v, np.ones_like(a), ea, np.zeros_like(a)


def scan64(f, v, h0, cu, gate, dtype=torch.float32):
    """h, h_last and their error bounds (before the rounding to dtype); float64
    arrays (rows, D); h0 (S, D); cu a list of bounds."""
    precise = dtype == torch.float32
    a, b, _, ea, eb = gate64(f, v, gate, precise)
    h, bound = np.zeros_like(a), np.zeros_like(a)
    last, last_bound = h0.copy(), np.zeros_like(h0)
    with np.errstate(all="ignore"):
        for s, (lo, hi) in enumerate(zip(cu, cu[1:])):
            st, major, e = h0[s].copy(), np.abs(h0[s]), np.zeros(f.shape[1])
            for t in range(lo, hi):
                e = a[t] * e + ea[t] * major + eb[t]
                st = a[t] * st + b[t]
                major = a[t] * major + np.abs(b[t])
                e = e + 2.0 ** -23 * major
                h[t], bound[t] = st, e
            if hi > lo:
                last[s], last_bound[s] = st, e
    return h, last, 4 * bound, 4 * last_bound


def grad64(f, v, h0, cu, gate, dh, dh_last, dtype=torch.float32):
    """df, dv, dh0 and their error bounds (before rounding)."""
    precise = dtype == torch.float32
    a, b, z, ea, eb = gate64(f, v, gate, precise)
    h, _, hb, _ = scan64(f, v, h0, cu, gate, dtype)
    hm = scan64(f, np.abs(v), np.abs(h0), cu, gate, dtype)[0]
    df, dv, d0 = np.zeros_like(a), np.zeros_like(a), np.zeros_like(h0)
    bf, bv, b0 = np.zeros_like(a), np.zeros_like(a), np.zeros_like(h0)
    eps = 2.0 ** -22
    for s, (lo, hi) in enumerate(zip(cu, cu[1:])):
        r = dh_last[s].copy() if dh_last is not None else np.zeros(f.shape[1])
        rm, re = np.abs(r), np.zeros_like(r)
        for t in range(hi - 1, lo - 1, -1):
            g, gm = dh[t] + r, np.abs(dh[t]) + rm
            ge = re + eps * gm
            prev, pm, pe = (h[t - 1], hm[t - 1], hb[t - 1]) if t > lo else (h0[s], np.abs(h0[s]), 0.0)
            if gate == "sigmoid":
                # fp32: 1 - a to its own relative precision; 16-bit: to that of a, and a rounding
                ez = (2.0 ** -20 + np.abs(f[t]) * 2.0 ** -22) * z[t] if precise else ea[t] + 2.0 ** -24
                c, cm = a[t] * z[t] * (prev - v[t]), a[t] * z[t] * (pm + np.abs(v[t]))
                ce = a[t] * z[t] * pe + (a[t] * ez + ea[t] * z[t]) * (pm + np.abs(v[t])) + 4 * eps * cm
                dv[t], bv[t] = z[t] * g, z[t] * ge + ez * gm + 2 * eps * z[t] * gm
            else:
                keep = np.where(f[t] <= 0, 1.0, 0.0)
                c, cm = keep * a[t] * prev, keep * a[t] * pm
                ce = keep * (a[t] * pe + ea[t] * pm) + 4 * eps * cm
                dv[t], bv[t] = g, ge
            df[t] = c * g
            bf[t] = cm * ge + ce * gm + 2 * eps * cm * gm
            r, rm, re = a[t] * g, a[t] * gm, a[t] * ge + ea[t] * gm + eps * a[t] * gm
        d0[s], b0[s] = r, re
    return df, dv, d0, 4 * bf, 4 * bv, 4 * b0


def check(got, want, bound, dtype, name):
    """got (a tensor of dtype) within bound plus the rounding of its type."""
    x = got.detach().double().cpu().numpy().reshape(want.shape)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(x), np.isnan(want)), f"{name}: NaN in other places"
    assert np.array_equal(x[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), f"{name}: infinities"
    half = torch.finfo(dtype).eps / 2
    lim = bound + half * (np.abs(want) + bound) + TINY[dtype]
    off = np.abs(x - want)
    bad = fine & ~(off <= lim)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, off / lim, 0)), want.shape)
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} outside; at {i}: got {x[i]}, want {want[i]}, "
                             f"off {off[i]:.3e}, allowed {lim[i]:.3e}")


def quantize64(x):
    """q, scale (fp32) of float64 rows holding values of a narrower type."""
    with np.errstate(all="ignore"):
        m = np.abs(x).max(axis=1, initial=0.0).astype(np.float32)
        s = np.maximum(m * (np.float32(1.0) / np.float32(127.0)), np.float32(2.0 ** -100))
        ok = np.isfinite(np.abs(x).sum(axis=1)) | np.isfinite(np.abs(x).max(axis=1, initial=0.0))
        q = np.where(ok[:, None], np.rint(x / s.astype(np.float64)[:, None]), 0)
    return q.astype(np.int64), np.where(ok, s, np.float32("nan"))
