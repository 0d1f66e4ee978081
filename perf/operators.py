"""The operators of a gated recurrent layer, measured: the gated linear
recurrence over long and packed sequences (forward, and forward with its
gradients), its single-token step on a pool of states, and the layer's
projection as a product of 8-bit integers with a scale for each token and
channel.

    gate "sigmoid":  a_t = sigmoid(f_t),       h_t = a_t h_{t-1} + (1 - a_t) v_t
    gate "log":      a_t = exp(min(f_t, 0)),   h_t = a_t h_{t-1} + v_t
    projection:      y[m, n] = s_x[m] s_w[n] sum_k q_x[m, k] q_w[n, k] + bias[n],
                     q = x / s to the nearest whole number (ties to even),
                     s = largest |x| of the row / 127

`run` computes the plain form of an operator or, where `own` is true, makes
the calls of scan_gated_rnns_b200.
"""
import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
SCALE_FLOOR = 2.0 ** -100          # the smallest scale of a row

# ------------------------------------------------------------------ cases


def _scan(name, rows, width, dtype, gate, seqs, packed, pad=0, init="each", halves=False, op="scan"):
    return {"name": name, "op": op, "rows": rows, "width": width, "dtype": dtype, "gate": gate, "seqs": seqs,
            "packed": packed, "pad": pad, "init": init, "halves": halves}


def _step(name, rows, width, dtype, gate, pool):
    return {"name": name, "op": "step", "rows": rows, "width": width, "dtype": dtype, "gate": gate, "pool": pool}


def _project(name, rows, inner, width, source, out, bias):
    return {"name": name, "op": "project", "rows": rows, "inner": inner, "width": width, "source": source,
            "out": out, "bias": bias}


def listed():
    return [
        # prompts of 23 requests packed one behind another, gates and values the two halves of the
        # projection's output, states carried in: serving, the throughput workload's rows and width
        _scan("scan_prompts_bf16", 32768, 4096, "bf16", "sigmoid", 23, True, halves=True),
        # one long document, the long-sequence workload's length and width
        _scan("scan_long_f32", 131072, 512, "f32", "log", 1, False),
        # a few short requests of an odd width: latency
        _scan("scan_short_f16", 61, 1001, "f16", "sigmoid", 3, True),
        # training on the carried-state workload's shape, one learnt initial state for every sequence
        _scan("train_f32", 8 * 4096, 1024, "f32", "log", 8, False, init="one", op="train"),
        # training on packed documents, the batch padded behind the last of them
        _scan("train_packed_bf16", 16384, 2048, "bf16", "sigmoid", 11, True, pad=357, op="train"),
        # the smallest batch of the repository's configurations
        _scan("train_small_f32", 2 * 1024, 512, "f32", "sigmoid", 2, False, init="none", op="train"),
        # one token for each of 8 running requests: latency
        _step("step_8_f32", 8, 1024, "f32", "sigmoid", 8),
        # one token for each request of a full batch, states scattered over a pool
        _step("step_512_bf16", 509, 4096, "bf16", "log", 1024),
        # the projection of one token for each of 8 requests: latency
        _project("project_8_bf16", 8, 1024, 2048, "bf16", "bf16", False),
        # a batch of tokens against a wide layer: the weights' bytes
        _project("project_batch_bf16", 120, 4096, 8192, "bf16", "bf16", False),
        # a prompt through a wide layer: the product's rate
        _project("project_prompt_bf16", 8192, 4096, 8192, "bf16", "bf16", False),
        # tokens quantised before, odd sizes, full-precision output
        _project("project_odd_int8", 1111, 1000, 1502, "int8", "f32", True),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "train", "train", "step", "project", "project"])
    if op in ("scan", "train"):
        most = 1 << (27 if op == "scan" else 25)
        width = _log_uniform(rng, 1, 4096)
        if rng.random() < 0.6:
            width = -(-width // 16) * 16
        rows = _log_uniform(rng, 1, min(131072, most // width))
        packed = rng.random() < 0.6
        seqs = _log_uniform(rng, 1, min(rows, 64))
        pad = 0
        if packed:
            pad = rng.choice([0, 0, rng.randrange(0, 1 + rows // 8)])
        else:
            rows = rows // seqs * seqs
        c = _scan("", rows, width, rng.choice(["f32", "bf16", "bf16", "f16"]), rng.choice(["sigmoid", "log"]), seqs,
                  packed, pad, rng.choice(["each", "one", "none"]), rng.random() < 0.4, op)
    elif op == "step":
        rows = _log_uniform(rng, 1, 512)
        c = _step("", rows, _log_uniform(rng, 1, 4096), rng.choice(["f32", "bf16", "f16"]),
                  rng.choice(["sigmoid", "log"]), rows + rng.randrange(0, 513))
    else:
        c = _project("", _log_uniform(rng, 1, 8192), _log_uniform(rng, 16, 4096), _log_uniform(rng, 16, 8192),
                     rng.choice(["f32", "bf16", "f16", "int8"]), rng.choice(["f32", "bf16", "f16"]),
                     rng.random() < 0.5)
    del c["name"]
    return c


def work(case):
    n, w = case["rows"], case["width"]
    if case["op"] == "project":
        k = case["inner"]
        source = n * (k + 4) if case["source"] == "int8" else n * k * SIZE[case["source"]]
        return {"bytes": source + w * (k + 4) + (4 * w if case["bias"] else 0) + n * w * SIZE[case["out"]],
                "flops": 2.0 * n * k * w}
    e = SIZE[case["dtype"]]
    if case["op"] == "step":      # gates, values and outputs of the rows; their states in and out; their slots
        return {"bytes": 3 * n * w * e + 2 * 4 * n * w + 4 * n, "flops": 4.0 * n * w}
    states = {"each": case["seqs"], "one": 1, "none": 0}[case["init"]] * w * 4 + case["seqs"] * w * 4
    live = n - case["pad"]
    if case["op"] == "scan":      # f and v in, h out
        return {"bytes": 3 * live * w * e + case["pad"] * w * e + states, "flops": 4.0 * live * w}
    # f, v and dh in; h, df and dv out
    return {"bytes": 6 * live * w * e + 3 * case["pad"] * w * e + 2 * states, "flops": 14.0 * live * w}


# ----------------------------------------------------------------- inputs


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEVICE, dtype=torch.float32)


def _gates(gen, gate, *shape):
    """Pre-activations around 2 (gates mostly kept), or log-decays between
    about -0.3 and -0.005: memories of tens of tokens."""
    x = _normal(gen, *shape)
    return x + 2.0 if gate == "sigmoid" else -torch.log1p(torch.exp(-3.0 - x))


def _rows_in_whole_words(q):
    """The same 8-bit rows, each of them starting at a 16-byte boundary (the
    layout a program keeps its weights in)."""
    n, k = q.shape
    buf = torch.zeros((n, -(-k // 16) * 16), dtype=torch.int8, device=q.device)
    buf[:, :k] = q
    return buf[:, :k]


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    n, w = case["rows"], case["width"]
    st = {"case": dict(case)}
    if case["op"] == "project":
        k = case["inner"]
        weights = _normal(gen, w, k) * (1.0 + _normal(gen, w, 1).abs()) / math.sqrt(k)
        st["w_q"], st["w_scale"] = _quantize(weights)
        st["w_q"] = _rows_in_whole_words(st["w_q"].to(torch.int8))
        x = _normal(gen, n, k) * (0.5 + _normal(gen, n, 1).abs())
        if case["source"] == "int8":
            q, st["x_scale"] = _quantize(x)
            st["x"] = _rows_in_whole_words(q.to(torch.int8))
        else:
            st["x"], st["x_scale"] = x.to(TYPES[case["source"]]), None
        st["bias"] = _normal(gen, w) if case["bias"] else None
        return st
    dt = TYPES[case["dtype"]]
    if case["op"] == "step":
        st["f"], st["v"] = _gates(gen, case["gate"], n, w).to(dt), _normal(gen, n, w).to(dt)
        st["pool"] = _normal(gen, case["pool"], w)
        st["slots"] = torch.randperm(case["pool"], generator=gen, device=DEVICE)[:n].to(torch.int32)
        return st
    if case["halves"]:            # the projection's output: gates, then values, of each token
        both = torch.cat([_gates(gen, case["gate"], n, w), _normal(gen, n, w)], 1).to(dt)
        f, v = both[:, :w], both[:, w:]
    else:
        f, v = _gates(gen, case["gate"], n, w).to(dt), _normal(gen, n, w).to(dt)
    seqs = case["seqs"]
    if case["packed"]:
        cuts = torch.randint(0, n - case["pad"] + 1, (seqs - 1,), generator=gen, device=DEVICE).sort().values
        ends = torch.tensor([n - case["pad"]], device=DEVICE)
        st["cu"] = torch.cat([torch.zeros_like(ends), cuts, ends]).to(torch.int32)
    else:
        st["cu"] = None
        f, v = f.unflatten(0, (seqs, n // seqs)), v.unflatten(0, (seqs, n // seqs))
    st["f"], st["v"] = f, v
    st["h0"] = {"each": lambda: _normal(gen, seqs, w), "one": lambda: _normal(gen, w), "none": lambda: None}[case["init"]]()
    if case["op"] == "train":
        st["dh"] = _normal(gen, n, w).to(dt).reshape(f.shape)
        st["f"].requires_grad_(True)
        st["v"].requires_grad_(True)
        if st["h0"] is not None:
            st["h0"].requires_grad_(True)
    return st


# ------------------------------------------------------------- plain forms


def _quantize(x):
    """Whole numbers and the scale of each row; the quotients in 64 bits, for
    those next to a half."""
    x = x.float()
    scale = (x.abs().amax(1) / 127.0).clamp_min(SCALE_FLOOR)
    return torch.round(x.double() / scale.double()[:, None]), scale


def _plain_project(st):
    case = st["case"]
    if case["source"] == "int8":
        q, scale = st["x"], st["x_scale"]
    else:
        q, scale = _quantize(st["x"])
    y = (q.float() @ st["w_q"].float().t()) * scale[:, None] * st["w_scale"][None, :]
    if st["bias"] is not None:
        y = y + st["bias"]
    return y.to(TYPES[case["out"]])


def _gate(f, v, gate):
    """Decays and what each step adds, in 32 bits."""
    f, v = f.float(), v.float()
    if gate == "sigmoid":
        return torch.sigmoid(f), torch.sigmoid(-f) * v
    return torch.exp(f.clamp(max=0.0)), v


def _prefix(a, b):
    """h_t = a_t h_{t-1} + b_t down the rows, by halves: the steps in twos,
    the states behind every second row, then the rows between."""
    n = a.shape[0]
    if n == 1:
        return b
    m = n // 2 * 2
    behind = _prefix(a[0:m:2] * a[1:m:2], a[1:m:2] * b[0:m:2] + b[1:m:2])
    h = torch.empty_like(b)
    h[0] = b[0]
    h[1:m:2] = behind
    h[2::2] = a[2::2] * behind[: (n - 1) // 2] + b[2::2]
    return h


def _rows_of(st):
    """First and last row, and the number, of the sequences that have rows."""
    case = st["case"]
    if st["cu"] is None:
        cu = torch.arange(case["seqs"] + 1, device=DEVICE) * (case["rows"] // case["seqs"])
    else:
        cu = st["cu"].long()
    live = (cu[1:] > cu[:-1]).nonzero().flatten()
    return cu[:-1][live], cu[1:][live] - 1, live


def _states_in(st):
    case, h0 = st["case"], st["h0"]
    shape = (case["seqs"], case["width"])
    return torch.zeros(shape, device=DEVICE) if h0 is None else h0.detach().expand(shape)


def _plain_scan(st):
    """h, the last states, and what the gradients use again."""
    case = st["case"]
    live = case["rows"] - case["pad"]
    first, last, seq = _rows_of(st)
    f, v = (st[k].detach().reshape(case["rows"], case["width"])[:live] for k in ("f", "v"))
    a, b = _gate(f, v, case["gate"])
    init = _states_in(st)
    h_last = init.clone()
    out = torch.zeros((case["rows"], case["width"]), device=DEVICE)
    if live:
        cut, add = a.clone(), b.clone()
        add[first] += a[first] * init[seq]
        cut[first] = 0.0
        out[:live] = _prefix(cut, add)
        h_last[seq] = out[last]
    return out, h_last, (a, init, first, last, seq, live)


def _plain_step(st):
    a, b = _gate(st["f"], st["v"], st["case"]["gate"])
    slots = st["slots"].long()
    h = a * st["pool"][slots] + b
    st["pool"][slots] = h
    return h.to(st["f"].dtype), st["pool"]


def _plain_train(st):
    case = st["case"]
    h, h_last, (a, init, first, last, seq, live) = _plain_scan(st)
    shape, dt = st["f"].shape, st["f"].dtype
    df = torch.zeros((case["rows"], case["width"]), device=DEVICE)
    dv, dinit = torch.zeros_like(df), torch.zeros_like(init)
    if live:
        f, v, dh = (st[k].detach().reshape(case["rows"], case["width"])[:live].float() for k in ("f", "v", "dh"))
        # g_t = dh_t + a_{t+1} g_{t+1} within a sequence: the same recurrence from the last row on
        carry = torch.zeros_like(a)
        carry[:-1] = a[1:]
        carry[last] = 0.0
        g = _prefix(carry.flip(0), dh.flip(0)).flip(0)
        before = torch.empty_like(a)
        before[1:] = h[: live - 1]
        before[first] = init[seq]
        if case["gate"] == "sigmoid":
            z = torch.sigmoid(-f)
            df[:live], dv[:live] = a * z * (before - v) * g, z * g
        else:
            df[:live], dv[:live] = torch.where(f <= 0.0, a * before * g, 0.0), g
        dinit[seq] = a[first] * g[first]
    grads = [df.to(dt).reshape(shape), dv.to(dt).reshape(shape)]
    if st["h0"] is not None:
        grads.append(dinit if st["h0"].dim() == 2 else dinit.sum(0))
    return [h.to(dt).reshape(shape), h_last] + grads


# -------------------------------------------------------------------- run


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import scan_gated_rnns_b200 as sgr
        if op == "project":
            return sgr.int8_projection(state["x"], state["w_q"], state["w_scale"], x_scale=state["x_scale"],
                                       bias=state["bias"], out_dtype=TYPES[case["out"]])
        if op == "step":
            return sgr.gated_step(state["f"], state["v"], state["pool"], state["slots"], gate=case["gate"]), state["pool"]
        if op == "scan":
            return sgr.gated_scan(state["f"], state["v"], state["h0"], state["cu"], gate=case["gate"])
        h, h_last = sgr.gated_scan_fn(state["f"], state["v"], state["h0"], state["cu"], gate=case["gate"])
        leaves = [state["f"], state["v"]] + ([] if state["h0"] is None else [state["h0"]])
        return [h.detach(), h_last.detach()] + list(torch.autograd.grad(h, leaves, state["dh"]))
    with torch.no_grad():
        if op == "project":
            return _plain_project(state)
        if op == "step":
            return _plain_step(state)
        if op == "scan":
            h, h_last, _ = _plain_scan(state)
            return h.to(state["f"].dtype).reshape(state["f"].shape), h_last
        return _plain_train(state)


# ------------------------------------------------------------------ exact


def exact(case, seed):
    def walk(decay, add, start, h):
        """The recurrence token by token, as it is defined."""
        for t in range(decay.shape[0]):
            start = decay[t] * start + add[t]
            h[t] = start
        return start

    st = prepare(case, seed)
    for k in ("f", "v", "h0"):
        if st.get(k) is not None:
            st[k] = st[k].detach()
    n, w = case["rows"], case["width"]
    if case["op"] == "project":
        if case["source"] == "int8":
            x = st["x"].double() * st["x_scale"].double()[:, None]
        else:
            s = torch.clamp(torch.max(torch.abs(st["x"].float()), 1).values / 127.0, min=SCALE_FLOOR).double()[:, None]
            x = torch.round(st["x"].double() / s) * s
        y = x @ (st["w_q"].double() * st["w_scale"].double()[:, None]).T
        return y if st["bias"] is None else y + st["bias"].double()
    if case["op"] == "step":
        f, v, pool = st["f"].double(), st["v"].double(), st["pool"].double()
        prev = pool[st["slots"].long()]
        if case["gate"] == "sigmoid":
            a = 1.0 / (1.0 + torch.exp(-f))
            h = a * prev + (1.0 - a) * v
        else:
            h = torch.exp(torch.minimum(f, torch.zeros_like(f))) * prev + v
        pool[st["slots"].long()] = h
        return h, pool
    bounds = [i * (n // case["seqs"]) for i in range(case["seqs"] + 1)] if st["cu"] is None else st["cu"].tolist()
    f, v = st["f"].reshape(n, w).double(), st["v"].reshape(n, w).double()
    if case["gate"] == "sigmoid":
        a = 1.0 / (1.0 + torch.exp(-f))
        z = 1.0 / (1.0 + torch.exp(f))
        b = z * v
    else:
        a, b = torch.exp(torch.minimum(f, torch.zeros_like(f))), v
    h0 = torch.zeros((case["seqs"], w), dtype=torch.float64, device=DEVICE)
    if st["h0"] is not None:
        h0 += st["h0"].double()
    h, last = torch.zeros_like(a), h0.clone()
    for s, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        last[s] = walk(a[lo:hi], b[lo:hi], h0[s], h[lo:hi])
    if case["op"] == "scan":
        return h.reshape(st["f"].shape), last
    df, dv, d0 = torch.zeros_like(a), torch.zeros_like(a), torch.zeros_like(h0)
    dh = st["dh"].reshape(n, w).double()
    for s, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        flow = d0[s]
        for t in range(hi - 1, lo - 1, -1):
            dv[t] = dh[t] + flow
            flow = a[t] * dv[t]
        d0[s] = flow
        if hi > lo:
            prev = torch.cat([h0[s][None], h[lo : hi - 1]])
            if case["gate"] == "sigmoid":
                df[lo:hi] = a[lo:hi] * z[lo:hi] * (prev - v[lo:hi]) * dv[lo:hi]
                dv[lo:hi] *= z[lo:hi]
            else:
                df[lo:hi] = torch.where(f[lo:hi] > 0.0, torch.zeros_like(prev), a[lo:hi] * prev * dv[lo:hi])
    out = [h.reshape(st["f"].shape), last, df.reshape(st["f"].shape), dv.reshape(st["f"].shape)]
    if st["h0"] is not None:
        out.append(d0 if st["h0"].dim() == 2 else d0.sum(0))
    return out
