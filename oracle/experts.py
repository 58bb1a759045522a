"""fp64 oracle of routing, 8-bit products by expert, and the gated activation.

Plain NumPy, written from the definitions in include/laga.h; shares no code
with the CUDA path.  Test infrastructure only.
"""

import numpy as np

from .residual import E_MAX, E_MIN, GROUP, e4m3_values, pack, row_layout, unpack

TINY = 1e-20


# ------------------------------------------------------------------ routing
def scores(logits, score):
    """Scores of fp64 logits [T, E]; a token all of whose experts are off has zeros."""
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-logits))
    m = logits.max(axis=1, keepdims=True)
    p = np.exp(logits - np.where(np.isfinite(m), m, 0.0))
    z = p.sum(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        return np.divide(p, z, out=np.zeros_like(p), where=z != 0)


def best(v, n):
    """Indices of the n largest of v, best first, the lowest of equal ones first;
    -inf does not count."""
    order = sorted(range(len(v)), key=lambda i: (-v[i], i))
    return [i for i in order[:n] if v[i] > -np.inf]


def choose(logits, bias, *, top_k, groups=1, top_groups=1, score="sigmoid", renormalise=True,
           scale=1.0):
    """(expert [T, k], weight [T, k]) of fp64 logits [T, E]."""
    T, E = logits.shape
    b = np.zeros(E) if bias is None else bias
    nan = np.isnan(logits) | np.isnan(b)
    if score == "softmax":
        nan = nan | (logits == np.inf)
    l = np.where(nan, -np.inf, logits)
    s = scores(l, score)
    c = np.where(l == -np.inf, -np.inf, s + np.where(np.isnan(b), 0.0, b))
    expert, weight = np.full((T, top_k), -1, np.int32), np.zeros((T, top_k))
    size = E // groups
    for t in range(T):
        row = c[t].copy()
        if top_groups < groups:
            total = []
            for g in range(groups):
                two = best(row[g * size:(g + 1) * size], 2)
                total.append(sum(row[g * size + i] for i in two) if two else -np.inf)
            keep = best(total, top_groups)
            for g in range(groups):
                if g not in keep:
                    row[g * size:(g + 1) * size] = -np.inf
        e = best(row, top_k)
        expert[t, :len(e)] = e
        w = s[t, e]
        weight[t, :len(e)] = scale * (w / (w.sum() + TINY) if renormalise else w)
        if nan[t].any():
            weight[t] = np.nan
    return expert, weight


def order(expert, *, first=0, local, align, rows, weight=None):
    """(row, pair, start) of the choices: pairs of the local experts, by expert.  A
    choice without an expert whose weight is a NaN has row -2."""
    T, k = expert.shape
    row, pair = np.full(T * k, -1, np.int32), np.full(rows, -1, np.int32)
    if weight is not None:
        row[((expert < 0) & np.isnan(weight)).reshape(-1)] = -2
    start = [0]
    flat = expert.reshape(-1)
    for e in range(first, first + local):
        p = np.flatnonzero(flat == e)
        at = start[-1] + np.arange(len(p))
        row[p], pair[at] = at, p
        start.append(start[-1] + -(-len(p) // align) * align)
    return row.reshape(T, k), pair, np.array(start, np.int32)


def route_bwd(logits, expert, dweight, *, score="sigmoid", renormalise=True, scale=1.0):
    """Gradient of fp64 logits for the weights' dweight at fixed choice."""
    s = scores(logits, score)
    out = np.zeros_like(logits)
    for t in range(len(logits)):
        on = np.flatnonzero(expert[t] >= 0)
        e, dw = expert[t, on], scale * dweight[t, on]
        v = s[t, e]
        if renormalise:
            D = v.sum() + TINY
            dv = dw / D - (dw * v).sum() / D ** 2
        else:
            dv = dw
        ds = np.zeros(logits.shape[1])
        np.add.at(ds, e, dv)
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                out[t] = ds * s[t] / (1.0 + np.exp(logits[t]))
        else:
            out[t] = s[t] * (ds - (ds * s[t]).sum())
    return out


# ------------------------------------------------------------------ 8 bits
def pack_weight(w):
    """(fwd, bwd) bytes of fp64 weights [E, K, N], one scale per 128 x 128 block."""
    E, K, N = w.shape
    ck, pk = row_layout(K)
    cn, pn = row_layout(N)
    g = np.zeros((E, ck, cn))
    g[:, :K, :N] = w
    blocks = g.reshape(E, ck // GROUP, GROUP, cn // GROUP, GROUP)
    bad = ~np.isfinite(blocks).all(axis=(2, 4))
    m, x = np.frexp(np.where(bad[:, :, None, :, None], 0.0, np.abs(blocks)).max(axis=(2, 4)))
    x = np.where(m <= 448.0 / 512.0, x - 9, x - 8)          # m 2^x <= 448 2^e
    x = np.where(m == 0, E_MIN, np.clip(x, E_MIN, E_MAX))
    t = np.where(bad[:, :, None, :, None], 0.0, blocks) / 2.0 ** x[:, :, None, :, None]
    t = np.clip(t, -448.0, 448.0).reshape(E, ck, cn)
    size = np.abs(t)
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(size, 2.0 ** -7))), -6.0) - 3.0)
    size = np.rint(size / step) * step                      # ties to even
    table = e4m3_values()[:0x7f]
    code = np.searchsorted(table, size)
    assert (table[code] == size).all()
    code = (code + np.where(np.signbit(t), 128, 0)).astype(np.uint8)
    byte = np.where(bad, 255, x + 127).astype(np.uint8)
    fwd, bwd = np.zeros((E, N, pk), np.uint8), np.zeros((E, K, pn), np.uint8)
    fwd[:, :, :ck] = code[:, :, :N].transpose(0, 2, 1)
    fwd[:, :, ck:ck + ck // GROUP] = np.repeat(byte.transpose(0, 2, 1), GROUP, axis=1)[:, :N]
    bwd[:, :, :cn] = code[:, :K]
    bwd[:, :, cn:cn + cn // GROUP] = np.repeat(byte, GROUP, axis=1)[:, :K]
    return fwd.reshape(E * N, pk), bwd.reshape(E * K, pn)


def mm8(a, b, k, n, start=None):
    """y[r] = a[r] b_e^T of 8-bit rows, and the sum of the terms' magnitudes;
    rows behind the last one in use are zero here."""
    va, vb = unpack(a, k), unpack(b, k)
    y, mag = np.zeros((len(a), n)), np.zeros((len(a), n))
    for e in range(len(b) // n):
        lo, hi = (0, len(a)) if start is None else (start[e], start[e + 1])
        w = vb[e * n:(e + 1) * n]
        y[lo:hi], mag[lo:hi] = va[lo:hi] @ w.T, np.abs(va[lo:hi]) @ np.abs(w).T
    return y, mag


def spread(buf, pair, top_k):
    out = np.zeros((len(pair), buf.shape[1]), np.uint8)
    out[pair >= 0] = buf[pair[pair >= 0] // top_k]
    return out


def weight_grad(buf, d, dy, start, gamma=None):
    """dw [E, d, n], and the sum of the terms' magnitudes."""
    v = unpack(buf, d) * (1.0 if gamma is None else gamma)
    seg = [(start[e], start[e + 1]) for e in range(len(start) - 1)]
    return (np.stack([v[a:b].T @ dy[a:b] for a, b in seg]),
            np.stack([np.abs(v[a:b]).T @ np.abs(dy[a:b]) for a, b in seg]))


# ------------------------------------------------------------------ rows back
def combine(y, weight, row):
    """out [T, d], and the sum of the terms' magnitudes."""
    out, mag = (np.zeros((len(row), y.shape[1])) for _ in range(2))
    for t in range(len(row)):
        for j, r in enumerate(row[t]):
            if r >= 0:
                out[t] += weight[t, j] * y[r]
                mag[t] += np.abs(weight[t, j] * y[r])
            elif r == -2:
                out[t] = np.nan
    return out, mag


def combine_bwd(dout, y, weight, row):
    """(dy, dweight, sum of dweight's terms' magnitudes)."""
    dy = np.zeros_like(y)
    dw, mag = np.zeros(row.shape), np.zeros(row.shape)
    for t in range(len(row)):
        for j, r in enumerate(row[t]):
            if r >= 0:
                dy[r] = weight[t, j] * dout[t]
                dw[t, j] = (dout[t] * y[r]).sum()
                mag[t, j] = np.abs(dout[t] * y[r]).sum()
    return dy, dw, mag


# ------------------------------------------------------------------ activation
def swiglu(gu):
    f = gu.shape[1] // 2
    with np.errstate(over="ignore"):
        return gu[:, :f] / (1.0 + np.exp(-gu[:, :f])) * gu[:, f:]


def swiglu_bwd(gu, da):
    f = gu.shape[1] // 2
    g, u = gu[:, :f], gu[:, f:]
    with np.errstate(over="ignore"):
        s, r = 1.0 / (1.0 + np.exp(-g)), 1.0 / (1.0 + np.exp(g))
    return np.concatenate([da * u * s * (1.0 + g * r), da * g * s], axis=1)


# ------------------------------------------------------------------ the block
def bf16(v):
    """fp64 values rounded to bf16 (8 significand bits, nearest even)."""
    m, e = np.frexp(v)
    return np.ldexp(np.rint(m * 256.0) / 256.0, e)


def quantised(v):
    return unpack(pack(v), v.shape[1])


def quantised_weight(w):
    """[E, K, N] as its 128 x 128 blocks' codes hold it."""
    _, bwd = pack_weight(w)
    return unpack(bwd, w.shape[2]).reshape(w.shape)


def block_fwd(h, w_router, bias, w_in, w_out, *, exact=False, io="bf16", **route):
    """(y, state) of routed experts over tokens h [T, d]: the block's 8-bit
    roundings and those of bf16 (``io``), or none with ``exact``."""
    q, qw, r = ((lambda v: v,) * 3) if exact else (quantised, quantised_weight, bf16)
    if io == "fp32":
        r = lambda v: v      # noqa: E731  (fp32's roundings are far below the others)
    logits = h @ w_router
    expert, weight = choose(logits, bias, **route)
    row, pair, start = order(expert, local=w_in.shape[0], align=1, rows=int((expert >= 0).sum()))
    h8, wi, wo = q(h), qw(w_in), qw(w_out)
    x = h8[pair // expert.shape[1]]
    seg = [(e, start[e], start[e + 1]) for e in range(len(wi)) if start[e + 1] > start[e]]
    gu = np.concatenate([r(x[a:b] @ wi[e]) for e, a, b in seg])
    act = q(swiglu(gu))
    rows = np.concatenate([r(act[a:b] @ wo[e]) for e, a, b in seg])
    y, _ = combine(rows, weight, row)
    return r(y), dict(h=h, h8=h8, x=x, wi=wi, wo=wo, gu=gu, act=act, rows=rows, logits=logits,
                      expert=expert, weight=weight, row=row, seg=seg, w_router=w_router,
                      fns=(q, r), route=route)


def block_bwd(st, dy):
    q, r = st["fns"]
    d_rows, dweight, _ = combine_bwd(dy, st["rows"], st["weight"], st["row"])
    d_rows = r(d_rows)
    d8 = q(d_rows)
    n, d = len(st["wi"]), dy.shape[1]
    da = np.concatenate([r(d8[a:b] @ st["wo"][e].T) for e, a, b in st["seg"]])
    dgu = r(swiglu_bwd(st["gu"], da))
    dgu8 = q(dgu)
    dx = np.concatenate([r(dgu8[a:b] @ st["wi"][e].T) for e, a, b in st["seg"]])
    dw_in, dw_out = np.zeros(st["wi"].shape), np.zeros(st["wo"].shape)
    for e, a, b in st["seg"]:
        dw_in[e], dw_out[e] = st["x"][a:b].T @ dgu[a:b], st["act"][a:b].T @ d_rows[a:b]
    kw = {k: v for k, v in st["route"].items() if k in ("score", "renormalise", "scale")}
    dlogits = route_bwd(st["logits"], st["expert"], dweight, **kw)
    back, _ = combine(dx, np.ones_like(st["weight"]), st["row"])
    return dict(dh=r(r(back) + r(dlogits @ st["w_router"].T)), dw_router=st["h8"].T @ dlogits,
                dw_in=dw_in, dw_out=dw_out)
