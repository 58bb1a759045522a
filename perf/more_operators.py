"""Measured cases of the 8-bit products and the routed experts.

A router scores E experts for every token, picks k of them and sorts the
(token, choice) pairs by expert.  An expert is two linear maps with a gated
activation between them,

    y_t = sum_j w_tj  W_out[e]^T a,   a = silu(g) * u,   [g | u] = W_in[e]^T h_t,

whose operands are e4m3 codes: activations with one power-of-two scale per
128 channels of a row, weights with one per block of 128 x 128.  The same
product without experts serves the projections of an attention block.

``run`` computes an operator in elementary torch operations, or, where
``own`` is true, by the framework's calls.  ``exact`` restates each definition
in 64 bits.
"""

import math

import torch

own = False

GROUP = 128            # channels that share one scale
E_MIN, E_MAX = -117, 119
TINY = 1e-20           # keeps the sum of a token's scores from zero

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def _route(tokens, experts, top_k, *, score="sigmoid", groups=1, top_groups=1, bias=True,
           renormalise=True, align=1, padded=0, dtype="fp32", back=False, name=None):
    c = dict(op="route", tokens=tokens, experts=experts, top_k=top_k, score=score, groups=groups,
             top_groups=top_groups, bias=bias, renormalise=renormalise, align=align,
             padded=padded, dtype=dtype, back=back)
    if name:
        c["name"] = name
    return c


def _linear(tokens, k, n, *, experts=0, top_k=1, spread=False, back=False, pack=False, align=1,
            dtype="bf16", name=None):
    c = dict(op="linear", tokens=tokens, k=k, n=n, experts=experts, top_k=top_k, spread=spread,
             back=back, pack=pack, align=align, dtype=dtype)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one token's choice in a decoding step: launches and their latency
        _route(1, 256, 8, groups=8, top_groups=4, name="route_token"),
        # a 16384-token training step with some padding tokens: choice, row order and gradient
        _route(16384, 256, 8, groups=8, top_groups=4, align=128, padded=100, back=True,
               name="route_train_16k"),
        # a decoding step of two tokens through 32 experts' first product: the weights' bytes
        _linear(2, 7168, 4096, experts=32, top_k=8, spread=True, name="experts_token"),
        # the query projection of 8 heads of 192, 16384 tokens, weights packed in the step
        _linear(16384, 7168, 1536, pack=True, name="linear_q_16k"),
        # first product of 32 experts for 16384 rows, taken from their tokens
        _linear(2048, 7168, 4096, experts=32, top_k=8, spread=True, align=128,
                name="experts_in_16k"),
        # input gradient of a small layer of odd widths
        _linear(333, 1001, 577, experts=5, top_k=2, back=True, dtype="fp32",
                name="experts_dx_odd"),
        # weight gradient of 8 experts' second product, 16384 rows
        dict(name="dw_experts_16k", op="dw", tokens=8192, top_k=2, experts=8, d=2048, n=7168,
             dtype="bf16"),
        # the same for a small layer with an fp32 gradient
        dict(name="dw_experts_small", op="dw", tokens=111, top_k=3, experts=7, d=384, n=200,
             dtype="fp32"),
        # the experts' rows back to 4096 tokens
        dict(name="combine_4k", op="combine", tokens=4096, top_k=8, experts=32, d=7168,
             dtype="bf16", back=False, align=128),
        # its backward
        dict(name="combine_bwd_2k", op="combine", tokens=2048, top_k=8, experts=32, d=7168,
             dtype="bf16", back=True, align=128),
        # gated activation of 16384 rows into 8 bits
        dict(name="swiglu_16k", op="swiglu", rows=16384, f=2048, dtype="bf16", back=False),
        # its backward, ragged rows
        dict(name="swiglu_bwd_4k", op="swiglu", rows=4097, f=2048, dtype="bf16", back=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    d = _log_int(rng, lo, hi)
    return max(lo, d // 64 * 64) if rng.random() < 0.6 else d   # model widths and odd ones


def draw(rng):
    op = rng.choice(["route", "linear", "linear", "dw", "combine", "swiglu"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    back, align = rng.random() < 0.5, rng.choice([1, 128])
    tokens, top_k, experts = _log_int(rng, 1, 2048), rng.randint(1, 8), _log_int(rng, 8, 32)
    if op == "route":
        experts = rng.choice([8, 16, 24, 40, 64, 100, 128, 160, 256])
        groups = rng.choice([g for g in (1, 2, 4, 8) if experts % g == 0])
        top_groups = rng.randint(1, groups)
        top_k = rng.randint(1, min(8, experts // groups * top_groups))
        tokens = _log_int(rng, 1, 16384)
        return _route(tokens, experts, top_k, score=rng.choice(["sigmoid", "softmax"]),
                      groups=groups, top_groups=top_groups, bias=rng.random() < 0.5,
                      renormalise=rng.random() < 0.7, align=align,
                      padded=rng.choice([0, tokens // 5]), dtype=dtype, back=back)
    if op == "linear" and rng.random() < 0.4:
        return _linear(_log_int(rng, 1, 16384), _width(rng, 64, 7168), _width(rng, 64, 1536),
                       back=back, pack=rng.random() < 0.3, dtype=dtype)
    if op == "linear":
        return _linear(tokens, _width(rng, 64, 7168), _width(rng, 64, 4096), experts=experts,
                       top_k=top_k, spread=rng.random() < 0.5 and not back, back=back,
                       align=align, dtype=dtype)
    if op == "dw":
        return dict(op=op, tokens=tokens, top_k=top_k, experts=experts, d=_width(rng, 64, 2048),
                    n=_width(rng, 64, 2048), dtype=dtype)
    if op == "combine":
        return dict(op=op, tokens=tokens, top_k=top_k, experts=experts, d=_width(rng, 64, 7168),
                    dtype=dtype, back=back, align=align)
    return dict(op=op, rows=_log_int(rng, 1, 16384), f=_width(rng, 64, 2048), dtype=dtype,
                back=back)


# ------------------------------------------------------------------ 8-bit rows
def _pitch(d):
    """(code bytes, bytes) of a row: codes padded to whole groups, scale bytes
    padded to 16."""
    codes = -(-d // GROUP) * GROUP
    return codes, codes + -(-(codes // GROUP) // 16) * 16


def _exponent(top):
    """The smallest e with top <= 448 * 2^e, within its range (448 = 0.875 * 2^9)."""
    m, x = torch.frexp(top)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(top > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


def _codes(v, e):
    """e4m3 bytes of fp32 values times 2^-e (two factors: each in range)."""
    t = torch.ldexp(v, -e).clamp(-448.0, 448.0)
    return t.to(torch.float8_e4m3fn).view(torch.uint8)


def _pack_rows(v):
    """Rows of fp32 values as codes and one scale byte per 128 channels."""
    rows, d = v.shape
    cols, pitch = _pitch(d)
    g = v.new_zeros(rows, cols)
    g[:, :d] = v
    g = g.view(rows, -1, GROUP)
    e = _exponent(g.abs().amax(dim=2))
    out = torch.zeros(rows, pitch, dtype=torch.uint8, device=v.device)
    out[:, :cols] = _codes(g, e[:, :, None]).view(rows, cols)
    out[:, cols:cols + cols // GROUP] = (e + 127).to(torch.uint8)
    return out


def _pack_weight(w):
    """w [E, K, N] fp32 as rows of its columns [E N, .] and of its rows [E K, .],
    with one scale per 128 x 128 block."""
    fwd, bwd = [], []
    for m in w:
        K, N = m.shape
        ck, pk = _pitch(K)
        cn, pn = _pitch(N)
        g = m.new_zeros(ck, cn)
        g[:K, :N] = m
        g = g.view(ck // GROUP, GROUP, cn // GROUP, GROUP)
        e = _exponent(g.abs().amax(dim=(1, 3)))
        codes = _codes(g, e[:, None, :, None]).view(ck, cn)
        byte = (e + 127).to(torch.uint8)
        f = torch.zeros(N, pk, dtype=torch.uint8, device=w.device)
        f[:, :ck] = codes[:, :N].t()
        f[:, ck:ck + ck // GROUP] = byte.t().repeat_interleave(GROUP, dim=0)[:N]
        b = torch.zeros(K, pn, dtype=torch.uint8, device=w.device)
        b[:, :cn] = codes[:K]
        b[:, cn:cn + cn // GROUP] = byte.repeat_interleave(GROUP, dim=0)[:K]
        fwd.append(f)
        bwd.append(b)
    return torch.cat(fwd), torch.cat(bwd)


def _values(buf, d):
    """fp32 values of rows of codes."""
    cols, _ = _pitch(d)
    v = buf[:, :cols].contiguous().view(torch.float8_e4m3fn).float()
    e = buf[:, cols:cols + cols // GROUP].to(torch.int32) - 127
    v = torch.ldexp(v.view(len(buf), -1, GROUP), e[:, :, None])
    return v.view(len(buf), cols)[:, :d]


# ------------------------------------------------------------------ row order
def _order(expert, n_experts, align, cap):
    """Pairs (t, j), numbered t k + j, sorted by expert, every expert's rows from
    a multiple of ``align``: (row [T, k], pair [cap], start [E + 1])."""
    flat = expert.reshape(-1).long()
    count = torch.bincount(flat[flat >= 0], minlength=n_experts)
    room = (count + align - 1) // align * align
    start = torch.cat([room.new_zeros(1), room.cumsum(0)])
    before = torch.cat([count.new_zeros(1), count.cumsum(0)])
    by = torch.argsort(torch.where(flat >= 0, flat, torch.full_like(flat, n_experts)), stable=True)
    by = by[:int(before[-1])]
    e = flat[by]
    at = start[e] + torch.arange(len(by), device=by.device) - before[e]
    row = torch.full_like(flat, -1)
    row[by] = at
    pair = torch.full((cap,), -1, dtype=torch.int64, device=by.device)
    pair[at] = by
    return row.view(expert.shape).int(), pair.int(), start.int()


def _capacity(tokens, top_k, experts, align):
    p = tokens * top_k
    return (p + min(experts, p) * (align - 1)) // align * align


def _plan(case, gen, dev):
    """A batch's choices, some experts liked better than others, in rows without
    spare ones at the end; what a program keeps of its routing.  The seed says
    which tokens go where; how many rows an expert gets is the case's."""
    T, k, E = case["tokens"], case["top_k"], case["experts"]
    own_gen = torch.Generator(dev).manual_seed(E)
    like = torch.softmax(0.5 * torch.randn(E, generator=own_gen, device=dev), dim=0)
    expert = torch.multinomial(like.expand(T, E), min(k, E), generator=own_gen).int()
    expert = expert[torch.randperm(T, generator=gen, device=dev)]
    cap = _capacity(T, expert.shape[1], E, case.get("align", 128))
    row, pair, start = _order(expert, E, case.get("align", 128), cap)
    bounds = start.tolist()
    weight = torch.rand(expert.shape, generator=gen, device=dev) + 0.05
    weight /= weight.sum(dim=1, keepdim=True)
    return dict(expert=expert, weight=weight, row=row, pair=pair[:bounds[-1]].clone(),
                start=start), bounds


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)
    dt = _DT[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    st = {"case": case}
    op = case["op"]
    if op == "route":
        T, E = case["tokens"], case["experts"]
        st["logits"] = (1.5 * normal(T, E)).to(dt)
        if case["padded"]:
            at = torch.randperm(T, generator=gen, device=dev)[:case["padded"]]
            st["logits"][at] = -math.inf
        st["bias"] = 0.1 * normal(E) if case["bias"] else None
        st["dweight"] = normal(T, case["top_k"])
        if own:
            import sequence_latent_norm_gb300 as laga
            st["router"] = laga.Router(
                E, case["top_k"], score=case["score"], groups=case["groups"],
                top_groups=case["top_groups"], renormalise=case["renormalise"], scale=2.5,
                align=case["align"], io_dtype=case["dtype"])
        return st
    if op == "swiglu":
        R, f = case["rows"], case["f"]
        st["gu"] = (1.5 * normal(R, 2 * f)).to(dt)
        if case["back"]:
            st["da"] = normal(R, f).to(dt)
        return st
    if case["experts"]:
        st["plan"], st["bounds"] = _plan(case, gen, dev)
        rows = len(st["plan"]["pair"])
        live = (st["plan"]["pair"] >= 0)[:, None]
    else:
        rows, live = case["tokens"], torch.ones(case["tokens"], 1, dtype=torch.bool, device=dev)
    if op == "linear":
        E, K, N = max(case["experts"], 1), case["k"], case["n"]
        w = torch.empty(E, K, N, device=dev).normal_(0.0, K ** -0.5, generator=gen)
        if case["pack"]:
            st["w"] = w[0].to(torch.bfloat16)
        else:
            st["fwd"], st["bwd"] = _pack_weight(w)
        del w
        lead = case["tokens"] if case["spread"] else rows
        x = normal(lead, N if case["back"] else K)
        st["x"] = _pack_rows(x if case["spread"] else x * live)
    elif op == "dw":
        a = normal(rows, case["d"])
        st["ck"] = _pack_rows(a * torch.sigmoid(a) * live)
        st["dy"] = (normal(rows, case["n"]) * live).to(dt)
    else:
        st["y"] = (normal(rows, case["d"]) * live).to(dt)
        if case["back"]:
            st["dout"] = normal(case["tokens"], case["d"]).to(dt)
    if own:
        import sequence_latent_norm_gb300 as laga
        if "plan" in st:
            p = st["plan"]
            st["routes"] = laga.Routes(p["expert"], p["weight"], p["row"], p["pair"], p["start"],
                                       case.get("align", 128))
        else:
            st["routes"] = None
        if op == "linear":
            st["x8"] = laga.Checkpoint8(st["x"], case["n"] if case["back"] else case["k"])
            if not case["pack"]:
                shape = (K, N) if not case["experts"] else (E, K, N)
                st["w8"] = laga.Weight8(shape, st["fwd"], st["bwd"])
        elif op == "dw":
            st["ck8"] = laga.Checkpoint8(st["ck"], case["d"])
    return st


# ------------------------------------------------------------------ plain and own passes
def _scores(x, score):
    return torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, dim=1).nan_to_num(nan=0.0)


def _run_route(st):
    case = st["case"]
    T, E, k, G = case["tokens"], case["experts"], case["top_k"], case["groups"]
    s = _scores(st["logits"].double(), case["score"])     # the choice in 64 bits: close scores
    c = s if st["bias"] is None else s + st["bias"].double()
    c = torch.where(st["logits"].isinf(), torch.full_like(c, -math.inf), c)
    if case["top_groups"] < G:
        best = c.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :2]
        total = best[:, :, 0] + (best[:, :, 1:].sum(dim=2)
                                 if best.shape[2] > 1 else 0.0)
        total = torch.where(best[:, :, -1].isinf(), best[:, :, 0], total)
        order = total.sort(dim=1, descending=True, stable=True).indices
        keep = torch.zeros(T, G, dtype=torch.bool, device=c.device)
        keep.scatter_(1, order[:, :case["top_groups"]], True)
        c = torch.where(keep.repeat_interleave(E // G, dim=1), c, torch.full_like(c, -math.inf))
    top = c.sort(dim=1, descending=True, stable=True)
    off = top.values[:, :k].isinf()
    idx = top.indices[:, :k]
    w = torch.where(off, torch.zeros((), device=c.device), s.float().gather(1, idx))
    total = w.sum(dim=1, keepdim=True) + TINY
    weight = 2.5 * (w / total if case["renormalise"] else w)
    expert = torch.where(off, torch.full_like(idx, -1), idx).int()
    cap = _capacity(T, k, E, case["align"])
    row, pair, start = _order(expert, E, case["align"], cap)
    out = dict(expert=expert, weight=weight, row=row, pair=pair, start=start)
    if case["back"]:
        g = 2.5 * st["dweight"].masked_fill(off, 0.0)
        if case["renormalise"]:
            g = (g - (g * w).sum(dim=1, keepdim=True) / total) / total
        g = torch.zeros_like(s, dtype=torch.float32).scatter_(1, idx, g.masked_fill(off, 0.0))
        s32 = s.float()
        if case["score"] == "sigmoid":
            d = g * s32 * torch.sigmoid(-st["logits"].float())
        else:
            d = s32 * (g - (g * s32).sum(dim=1, keepdim=True))
        out["dlogits"] = d.to(_DT[case["dtype"]])
    return out


def _segments(st, rows):
    """(expert, first row, last row + 1) of every piece of the rows."""
    if "plan" not in st:
        return [(0, 0, rows)]
    b = st["bounds"]
    return [(e, b[e], b[e + 1]) for e in range(len(b) - 1) if b[e + 1] > b[e]]


def _run_linear(st):
    case = st["case"]
    K, N = case["k"], case["n"]
    if case["pack"]:
        fwd, bwd = _pack_weight(st["w"].float()[None])
    else:
        fwd, bwd = st["fwd"], st["bwd"]
    x = _values(st["x"], N if case["back"] else K)
    if case["spread"]:
        pair = st["plan"]["pair"].long()
        x = torch.where((pair >= 0)[:, None], x[pair.clamp(min=0) // st["plan"]["row"].shape[1]],
                        torch.zeros((), device=x.device))
    out = torch.empty(len(x), K if case["back"] else N, dtype=_DT[case["dtype"]], device=x.device)
    for e, a, b in _segments(st, len(x)):
        w = _values(bwd[e * K:(e + 1) * K], N) if case["back"] else _values(
            fwd[e * N:(e + 1) * N], K)
        out[a:b] = x[a:b] @ w.t()
    return {"y": out}


def _run_dw(st):
    case = st["case"]
    v = _values(st["ck"], case["d"])
    dw = torch.zeros(case["experts"], case["d"], case["n"], device=v.device)
    for e, a, b in _segments(st, len(v)):
        dw[e] = v[a:b].t() @ st["dy"][a:b].float()
    return {"dw": dw}


def _run_combine(st):
    case, p = st["case"], st["plan"]
    y = st["y"].float()
    rows = y[p["row"].long()]                               # [T, k, d]
    if not case["back"]:
        return {"out": (p["weight"][:, :, None] * rows).sum(dim=1).to(st["y"].dtype)}
    dout = st["dout"].float()
    pair = p["pair"].long()
    at = pair.clamp(min=0)
    w = p["weight"].reshape(-1)[at].masked_fill(pair < 0, 0.0)
    dy = w[:, None] * dout[at // p["row"].shape[1]]
    return {"dy": dy.to(st["y"].dtype), "dweight": (rows * dout[:, None, :]).sum(dim=2)}


def _run_swiglu(st):
    f = st["case"]["f"]
    g, u = st["gu"][:, :f].float(), st["gu"][:, f:].float()
    sig = torch.sigmoid(g)
    if not st["case"]["back"]:
        return {"a8": _values(_pack_rows(g * sig * u), f).to(torch.bfloat16)}
    da = st["da"].float()
    dg = da * u * sig * (1.0 + g * torch.sigmoid(-g))
    return {"dgu": torch.cat([dg, da * g * sig], dim=1).to(st["gu"].dtype)}


def _run_own(st):
    import sequence_latent_norm_gb300 as laga
    case = st["case"]
    if case["op"] == "route":
        r = st["router"].forward(st["logits"], st["bias"])
        out = dict(expert=r.expert, weight=r.weight, row=r.row, pair=r.pair, start=r.start)
        if case["back"]:
            out["dlogits"] = st["router"].backward(st["logits"], r, st["dweight"])
        return out
    if case["op"] == "linear":
        w8 = laga.pack_weight8(st["w"]) if case["pack"] else st["w8"]
        x8 = laga.spread8(st["x8"], st["routes"]) if case["spread"] else st["x8"]
        f = laga.linear8_dx if case["back"] else laga.linear8
        return {"y": f(x8, w8, routes=st["routes"], dtype=_DT[case["dtype"]])}
    if case["op"] == "dw":
        return {"dw": laga.weight_grad8(st["ck8"], st["dy"], routes=st["routes"])}
    if case["op"] == "combine":
        if not case["back"]:
            return {"out": laga.combine(st["y"], st["routes"])}
        dy, dweight = laga.combine_grad(st["dout"], st["routes"], y=st["y"])
        return {"dy": dy, "dweight": dweight}
    if case["back"]:
        return {"dgu": laga.swiglu8_grad(st["gu"], st["da"])}
    return {"a8": laga.swiglu8(st["gu"]).unpack()}


def run(state):
    if own:
        return _run_own(state)
    return {"route": _run_route, "linear": _run_linear, "dw": _run_dw, "combine": _run_combine,
            "swiglu": _run_swiglu}[state["case"]["op"]](state)


# ------------------------------------------------------------------ work
def _used(experts, rows):
    """Experts that get a row, on average."""
    return experts * (1.0 - (1.0 - 1.0 / experts) ** rows)


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "swiglu":
        n = case["rows"] * case["f"]
        if case["back"]:
            return {"bytes": 5 * n * size, "flops": 14 * n}
        return {"bytes": 2 * n * size + 1.008 * n + 2 * n, "flops": 8 * n}
    T, k = case["tokens"], case["top_k"]
    if op == "route":
        n = T * case["experts"]
        b = n * size + 16 * T * k
        return {"bytes": b + (n * size + 4 * T * k if case["back"] else 0),
                "flops": (20 if case["back"] else 12) * n}
    rows = T * min(k, case["experts"]) if case["experts"] else T
    if op == "linear":
        K, N = case["k"], case["n"]
        a, b = (N, K) if case["back"] else (K, N)
        wbytes = K * N * (2 if case["pack"] else _used(case["experts"], rows)
                          if case["experts"] else 1)
        return {"bytes": (T if case["spread"] else rows) * a + wbytes + rows * b * size,
                "flops": 2 * rows * K * N}
    if op == "dw":
        d, n = case["d"], case["n"]
        return {"bytes": rows * (d + n * size) + 4 * case["experts"] * d * n,
                "flops": 2 * rows * d * n}
    d = case["d"]
    if case["back"]:
        return {"bytes": (2 * rows + T) * d * size + 12 * rows, "flops": 3 * rows * d}
    return {"bytes": (rows + T) * d * size + 8 * rows, "flops": 2 * rows * d}


# ------------------------------------------------------------------ in 64 bits
def _exact_kept(buf, d):
    """float64 values of rows of codes, from their bits."""
    cols, _ = _pitch(d)
    b = buf[:, :cols].to(torch.int64)
    expo, frac = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(expo > 0, (1.0 + frac / 8.0) * torch.exp2((expo - 7).double()),
                      frac / 8.0 * 2.0 ** -6)
    v = torch.where(b >= 128, -mag, mag)
    scale = torch.exp2(buf[:, cols:cols + cols // GROUP].double() - 127.0)
    return (v * scale.repeat_interleave(GROUP, dim=1))[:, :d]


def _exact_round8(g):
    """float64 values of one group, all under one scale, rounded to its codes."""
    top = float(g.abs().max())
    e = math.ceil(math.log2(top / 448.0)) if top > 0 else E_MIN
    while top > 448.0 * 2.0 ** e:
        e += 1
    while e > E_MIN and top <= 448.0 * 2.0 ** (e - 1):
        e -= 1
    unit = 2.0 ** max(E_MIN, min(E_MAX, e))
    t = (g / unit).clamp(-448.0, 448.0)
    binade = torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(binade - 3.0)
    return torch.round(t / step) * step * unit


def _exact_rows8(v):
    """The same for every 128 channels of every row at once."""
    out = torch.empty_like(v)
    for c in range(0, v.shape[1], GROUP):
        g = v[:, c:c + GROUP]
        top = g.abs().amax(dim=1, keepdim=True)
        e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.full_like(top, 2.0 ** -120))
                                  / 448.0))
        for _ in range(2):     # log2 may be a unit off next to a border
            e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
            e = torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e)
        unit = torch.exp2(e.clamp(E_MIN, E_MAX))
        t = (g / unit).clamp(-448.0, 448.0)
        binade = torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6)))
        step = torch.exp2(binade - 3.0)
        out[:, c:c + GROUP] = torch.round(t / step) * step * unit
    return out


def _exact_route(case, st):
    T, E, k, G = case["tokens"], case["experts"], case["top_k"], case["groups"]
    l = st["logits"].double()
    dev = l.device
    if case["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        m = l.amax(dim=1, keepdim=True)
        p = torch.exp(l - torch.where(m > -math.inf, m, torch.zeros_like(m)))
        s = p / p.sum(dim=1, keepdim=True).clamp(min=1e-300)
    c = s + (0.0 if st["bias"] is None else st["bias"].double())
    c = c.masked_fill(l == -math.inf, -math.inf)

    def first_best(v):
        """Index of each row's largest value, the lowest of equal ones, and the value."""
        top = v.amax(dim=1, keepdim=True)
        n = torch.arange(v.shape[1], device=dev).expand_as(v)
        return torch.where(v == top, n, v.shape[1]).amin(dim=1, keepdim=True), top

    if case["top_groups"] < G:
        per = c.reshape(T * G, E // G)
        i, a = first_best(per)
        _, b = first_best(per.scatter(1, i, -math.inf))
        score = (a + b.clamp(min=-1e300).where(b > -math.inf, torch.zeros_like(b))).view(T, G)
        keep = torch.zeros(T, G, dtype=torch.bool, device=dev)
        for _ in range(case["top_groups"]):
            i, _ = first_best(score.masked_fill(keep, -math.inf))
            keep.scatter_(1, i, True)
        c = c.masked_fill(~keep.repeat_interleave(E // G, dim=1), -math.inf)
    expert, val = [], []
    for _ in range(k):
        i, top = first_best(c)
        on = top > -math.inf
        expert.append(torch.where(on, i, -1))
        val.append(torch.where(on, s.gather(1, i), 0.0))
        c = c.scatter(1, i, -math.inf)
    expert, val = torch.cat(expert, dim=1), torch.cat(val, dim=1)
    total = val.sum(dim=1, keepdim=True) + TINY
    weight = 2.5 * (val / total if case["renormalise"] else val)

    flat = expert.reshape(-1).tolist()
    members = [[] for _ in range(E)]
    for p, e in enumerate(flat):
        if e >= 0:
            members[e].append(p)
    cap = _capacity(T, k, E, case["align"])
    row, pair, start = [-1] * len(flat), [-1] * cap, [0]
    for e in range(E):
        for i, p in enumerate(members[e]):
            row[p] = start[e] + i
            pair[start[e] + i] = p
        start.append(start[e] + -(-len(members[e]) // case["align"]) * case["align"])

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    out = dict(expert=expert.int(), weight=weight, row=ints(row).view(T, k), pair=ints(pair),
               start=ints(start))
    if case["back"]:
        # gradient of each score, then of the logits, from the quotient's derivative
        gw = 2.5 * st["dweight"].double() * (expert >= 0)
        if case["renormalise"]:
            gs = gw / total - (gw * val).sum(dim=1, keepdim=True) / total.square()
        else:
            gs = gw
        gs = gs * (expert >= 0)
        g = torch.zeros(T, E + 1, dtype=torch.float64, device=dev)
        g.scatter_(1, torch.where(expert >= 0, expert, E).long(), gs)
        g = g[:, :E]
        if case["score"] == "sigmoid":
            out["dlogits"] = g * s / (1.0 + torch.exp(l))
        else:
            out["dlogits"] = g * s - s * (g * s).sum(dim=1, keepdim=True)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(case, st)
    if op == "swiglu":
        f = case["f"]
        g, u = st["gu"].double().split(f, dim=1)
        if not case["back"]:
            return {"a8": _exact_rows8(g * u / (1.0 + torch.exp(-g)))}
        da, den = st["da"].double(), 1.0 + torch.exp(-g)
        slope = 1.0 / den + g * torch.exp(-g) / den.square()
        return {"dgu": torch.cat([da * u * slope, da * g / den], dim=1)}
    pieces = [(0, 0, None)]
    if case["experts"]:
        b = st["plan"]["start"].tolist()
        pieces = [(e, b[e], b[e + 1]) for e in range(case["experts"])]
        pair = st["plan"]["pair"].long()
        token = torch.div(pair, st["plan"]["row"].shape[1], rounding_mode="floor")
    if op == "linear":
        K, N = case["k"], case["n"]
        a = _exact_kept(st["x"], N if case["back"] else K)
        if case["spread"]:
            a = torch.where((pair >= 0)[:, None], a[token.clamp(min=0)],
                            torch.zeros((), dtype=a.dtype, device=a.device))
        out = []
        for e, lo, hi in pieces:
            if case["pack"]:
                w = st["w"].double()
                for i in range(0, K, GROUP):
                    for j in range(0, N, GROUP):
                        w[i:i + GROUP, j:j + GROUP] = _exact_round8(
                            w[i:i + GROUP, j:j + GROUP])
            else:
                w = _exact_kept(st["bwd"][e * K:(e + 1) * K], N)
            out.append(torch.einsum("rn,kn->rk" if case["back"] else "rk,kn->rn", a[lo:hi], w))
        return {"y": torch.cat(out)}
    if op == "dw":
        a = _exact_kept(st["ck"], case["d"])
        return {"dw": torch.stack([torch.einsum("td,tn->dn", a[lo:hi], st["dy"][lo:hi].double())
                                   for _, lo, hi in pieces])}
    y, w, row = st["y"].double(), st["plan"]["weight"].double(), st["plan"]["row"].long()
    if not case["back"]:
        return {"out": sum(w[:, j:j + 1] * y[row[:, j]] for j in range(row.shape[1]))}
    dout = st["dout"].double()
    dy = torch.zeros_like(y)
    for j in range(row.shape[1]):
        dy[row[:, j]] = w[:, j:j + 1] * dout
    return {"dy": dy, "dweight": torch.stack([torch.einsum("td,td->t", dout, y[row[:, j]])
                                              for j in range(row.shape[1])], dim=1)}
