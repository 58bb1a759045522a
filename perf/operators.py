"""Measured cases of the residual-stream operators and the 8-bit checkpoints.

Around an attention block the residual stream runs

    x' = x + alpha * sigmoid(a) * N_post(y) * gamma_post
    h  = N_pre(x') * gamma_pre

(N: LayerNorm, RMS norm or, behind the block, none; a: gate logits per
element or per token, or no gate).  What its backward needs of the
activations, the normalised y^ and x^, is kept in the I/O type or as an 8-bit
checkpoint: e4m3 codes with one power-of-two scale per 128 channels.  A
weight gradient behind the norm is taken from the same checkpoint.

``run`` computes an operator in elementary torch operations in 32 bits, or,
where ``own`` is true, by the framework's calls.  ``exact`` restates each
definition in 64 bits.
"""

import math

import torch

own = False

GROUP = 128            # channels that share one scale
E_MIN, E_MAX = -117, 119
EPS = 1e-5

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def _res(op, rows, d, *, post=True, pre=True, norm_post="rms", norm_pre="rms", gate="none",
         ckpt=False, dtype="bf16", name=None):
    c = dict(op=op, rows=rows, d=d, post=post, pre=pre, norm_post=norm_post, norm_pre=norm_pre,
             gate=gate, ckpt=ckpt, dtype=dtype)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one token in front of a block (decoding): a launch and its latency
        _res("res_fwd", 1, 7168, post=False, name="pre_fwd_token"),
        # between two blocks of a 16384-token step at d_model 7168, activations kept in bf16
        _res("res_fwd", 16384, 7168, gate="full", name="junction_fwd_16k"),
        # the same with a token gate, LayerNorm and both activations kept in 8 bits
        _res("res_fwd", 4096, 7168, norm_post="layer", norm_pre="layer", gate="token", ckpt=True,
             name="junction_fwd_ckpt_4k"),
        # behind the last block, fp32, a ragged batch and an odd width
        _res("res_fwd", 333, 1001, pre=False, norm_post="layer", gate="full", dtype="fp32",
             name="post_fwd_fp32_odd"),
        # backward of the 16384-token step from 8-bit checkpoints
        _res("res_bwd", 16384, 7168, gate="full", ckpt=True, name="junction_bwd_ckpt_16k"),
        # backward in fp32 from the kept activations, residual add without a post norm
        _res("res_bwd", 2047, 2048, norm_post="none", norm_pre="layer", gate="token",
             dtype="fp32", name="junction_bwd_fp32"),
        # backward of a small block's first norm
        _res("res_bwd", 129, 512, post=False, norm_pre="layer", name="pre_bwd_small"),
        # an activation of the 16384-token step into 8 bits and back
        dict(name="pack_16k", op="pack", rows=16384, d=7168, dtype="bf16"),
        # a ragged fp32 activation of odd width
        dict(name="pack_fp32_odd", op="pack", rows=257, d=1001, dtype="fp32"),
        # gradient of W_kv_a (512 + 64 columns) from the fp32 latent gradient
        dict(name="dw_kva_16k", op="dw", rows=16384, d=7168, n=576, dtype="fp32", gain=True),
        # gradient of W_q for 8 heads of 192
        dict(name="dw_q_16k", op="dw", rows=16384, d=7168, n=1536, dtype="bf16", gain=True),
        # a small block's weight gradient over a ragged chunk
        dict(name="dw_small", op="dw", rows=333, d=384, n=200, dtype="bf16", gain=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["res_fwd", "res_bwd", "pack", "dw"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    rows, d = _log_int(rng, 1, 16384), _log_int(rng, 64, 7168)
    if rng.random() < 0.6:
        d = max(64, d // 8 * 8)        # model widths; the rest are odd ones
    if op == "pack":
        return dict(op=op, rows=rows, d=d, dtype=dtype)
    if op == "dw":
        return dict(op=op, rows=rows, d=d, n=_log_int(rng, 8, 1536), dtype=dtype,
                    gain=rng.random() < 0.5)
    post, pre = rng.choice([(True, True), (True, True), (True, False), (False, True)])
    return _res(op, rows, d, post=post, pre=pre, norm_post=rng.choice(["rms", "layer", "none"]),
                norm_pre=rng.choice(["rms", "layer"]), gate=rng.choice(["none", "token", "full"]),
                ckpt=rng.random() < 0.5, dtype=dtype)


# ------------------------------------------------------------------ 8-bit rows
def _pitch(d):
    """(code bytes, bytes) of a checkpoint row: codes padded to whole groups,
    scale bytes padded to 16."""
    codes = -(-d // GROUP) * GROUP
    return codes, codes + -(-(codes // GROUP) // 16) * 16


def _groups(v):
    rows, d = v.shape
    g = v.new_zeros(rows, _pitch(d)[0])
    g[:, :d] = v
    return g.reshape(rows, -1, GROUP)


def _quantise(v):
    """Codes (e4m3), exponents and whole-group NaN marks of fp32 values."""
    g = _groups(v)
    bad = ~torch.isfinite(g).all(dim=2)
    g = torch.where(bad[:, :, None], torch.zeros_like(g), g)
    m, k = torch.frexp(g.abs().amax(dim=2))          # amax = m 2^k, m in [0.5, 1)
    e = torch.where(m <= 0.875, k - 9, k - 8).clamp(E_MIN, E_MAX)
    t = torch.ldexp(g, -e[:, :, None]).clamp(-448.0, 448.0)
    return t.to(torch.float8_e4m3fn), e, bad


def _values(codes, e, bad, d):
    v = torch.ldexp(codes.float(), e[:, :, None])
    v = torch.where(bad[:, :, None], torch.full_like(v, float("nan")), v)
    return v.reshape(v.shape[0], -1)[:, :d]


def _buffer(v):
    """The checkpoint rows (uint8) of fp32 values."""
    codes, e, bad = _quantise(v)
    cols, pitch = _pitch(v.shape[1])
    buf = torch.zeros(v.shape[0], pitch, dtype=torch.uint8, device=v.device)
    buf[:, :cols] = codes.reshape(v.shape[0], cols).view(torch.uint8)
    buf[:, cols:cols + e.shape[1]] = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
    return buf


def _decode(buf, d):
    cols, _ = _pitch(d)
    n = cols // GROUP
    codes = buf[:, :cols].contiguous().view(torch.float8_e4m3fn).reshape(buf.shape[0], n, GROUP)
    s = buf[:, cols:cols + n].int()
    return _values(codes, s - 127, s == 255, d)


# ------------------------------------------------------------------ inputs
def _gain(d, gen):
    return 1.0 + 0.1 * torch.randn(d, device="cuda", generator=gen)


def _stream(rows, d, gen):
    """A residual stream: unit channels, a few of them large, a small offset."""
    x = torch.randn(rows, d, device="cuda", generator=gen)
    big = torch.rand(d, device="cuda", generator=gen) < 0.005
    return x * torch.where(big, 20.0, 1.0) + 0.05


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    rows, d, dt = case["rows"], case["d"], _DT[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    st = dict(case=case)
    if case["op"] == "pack":
        st["x"] = _stream(rows, d, gen).to(dt)
        return st
    if case["op"] == "dw":
        st["ck"] = _buffer(randn(rows, d))
        st["dy"] = (0.02 * randn(rows, case["n"])).to(dt)
        st["gamma"] = _gain(d, gen) if case["gain"] else None
        return st
    x, y = _stream(rows, d, gen).to(dt), randn(rows, d).to(dt)
    if case["post"]:
        st["alpha"] = 0.5 + torch.rand(1, device="cuda", generator=gen)
        if case["norm_post"] != "none":
            st["gamma_post"] = _gain(d, gen)
        if case["gate"] != "none":
            st["gate"] = randn(rows, d if case["gate"] == "full" else 1).to(dt)
    if case["pre"]:
        st["gamma_pre"] = _gain(d, gen)
    if case["op"] == "res_fwd":
        st["x"] = x
        if case["post"]:
            st["y"] = y
        return st
    # the backward's inputs: what the forward kept, and the incoming gradients
    if case["post"]:
        hat, st["stat_post"] = _hat(y.float(), case["norm_post"])
        st["y"] = _buffer(hat) if case["ckpt"] else y
    if case["pre"]:
        hat, st["stat_pre"] = _hat(x.float(), case["norm_pre"])
        st["x"] = _buffer(hat) if case["ckpt"] else x
        st["dh"] = randn(rows, d).to(dt)
    # a gradient of the stream that has something to do with the block's output
    st["dx_out"] = (randn(rows, d) + 0.1 * y.float()).to(dt)
    return st


# ------------------------------------------------------------------ plain form
def _hat(v, norm):
    """Normalised rows and their [mean, 1/std]."""
    if norm == "none":
        return v, torch.stack([torch.zeros_like(v[:, 0]), torch.ones_like(v[:, 0])], dim=1)
    mean = v.mean(dim=1, keepdim=True) if norm == "layer" else torch.zeros_like(v[:, :1])
    c = v - mean
    rstd = 1.0 / torch.sqrt((c * c).mean(dim=1, keepdim=True) + EPS)
    return c * rstd, torch.cat([mean, rstd], dim=1)


def _sigmoid(a):
    return 1.0 / (1.0 + torch.exp(-a))


def _plain_fwd(st):
    c, dt = st["case"], _DT[st["case"]["dtype"]]
    out = {}
    x = st["x"].float()
    if c["post"]:
        hat, out["stat_post"] = _hat(st["y"].float(), c["norm_post"])
        z = hat * st["gamma_post"] if "gamma_post" in st else hat
        if "gate" in st:
            z = z * _sigmoid(st["gate"].float())
        x = x + st["alpha"] * z
        out["x"] = x.to(dt)
        if c["ckpt"]:
            out["y8"] = _values(*_quantise(hat), c["d"]).to(torch.bfloat16)
    if c["pre"]:
        hat, out["stat_pre"] = _hat(x, c["norm_pre"])
        out["h"] = (hat * st["gamma_pre"]).to(dt)
        if c["ckpt"]:
            out["x8"] = _values(*_quantise(hat), c["d"]).to(torch.bfloat16)
    return out


def _norm_bwd(f, hat, rstd, norm):
    if norm == "none":
        return f
    m = (f * hat).mean(dim=1, keepdim=True)
    g = f - hat * m
    if norm == "layer":
        g = g - f.mean(dim=1, keepdim=True)
    return rstd * g


def _plain_bwd(st):
    c, dt = st["case"], _DT[st["case"]["dtype"]]

    def kept(v, stat):
        if c["ckpt"]:
            return _decode(v, c["d"])
        return (v.float() - stat[:, :1]) * stat[:, 1:]

    out = {}
    D = st["dx_out"].float()
    if c["pre"]:
        hat, dh = kept(st["x"], st["stat_pre"]), st["dh"].float()
        out["dgamma_pre"] = (dh * hat).sum(dim=0)
        D = D + _norm_bwd(dh * st["gamma_pre"], hat, st["stat_pre"][:, 1:], c["norm_pre"])
        out["dx"] = D.to(dt)
    if c["post"]:
        hat = kept(st["y"], st["stat_post"])
        z = hat * st["gamma_post"] if "gamma_post" in st else hat
        alpha = st["alpha"]
        dz = alpha * D
        u = z
        if "gate" in st:
            s = _sigmoid(st["gate"].float())
            da = dz * z * s * (1.0 - s)
            out["dgate"] = (da if c["gate"] == "full" else da.sum(dim=1, keepdim=True)).to(dt)
            u, dz = z * s, dz * s
        out["dalpha"] = (D * u).sum().reshape(1)
        if "gamma_post" in st:
            out["dgamma_post"] = (dz * hat).sum(dim=0)
            dz = dz * st["gamma_post"]
        out["dy"] = _norm_bwd(dz, hat, st["stat_post"][:, 1:], c["norm_post"]).to(dt)
    return out


def _plain(st):
    c = st["case"]
    if c["op"] == "res_fwd":
        return _plain_fwd(st)
    if c["op"] == "res_bwd":
        return _plain_bwd(st)
    if c["op"] == "pack":
        return {"x8": _values(*_quantise(st["x"].float()), c["d"]).to(_DT[c["dtype"]])}
    dw = _decode(st["ck"], c["d"]).t() @ st["dy"].float()
    return {"dw": dw * st["gamma"][:, None] if c["gain"] else dw}


# ------------------------------------------------------------------ the framework's calls
def _own(st):
    import sequence_latent_norm_gb300 as laga
    c = st["case"]
    if c["op"] == "pack":
        return {"x8": laga.pack8(st["x"]).unpack(st["x"].dtype)}
    if c["op"] == "dw":
        return {"dw": laga.weight_grad8(laga.Checkpoint8(st["ck"], c["d"]), st["dy"],
                                        gamma=st["gamma"])}
    if "plan" not in st:
        st["plan"] = laga.ResidualNorm(c["d"], post=c["post"], pre=c["pre"],
                                       norm_post=c["norm_post"], norm_pre=c["norm_pre"],
                                       gate=c["gate"], ckpt=c["ckpt"], io_dtype=c["dtype"],
                                       eps=EPS, device="cuda")
    plan = st["plan"]
    gains = dict(gate=st.get("gate"), alpha=st.get("alpha"), gamma_post=st.get("gamma_post"),
                 gamma_pre=st.get("gamma_pre"))
    if c["op"] == "res_fwd":
        r = plan.forward(st["x"], st.get("y"), **gains)
        out = {}
        if c["post"]:
            out["stat_post"], out["x"] = r.saved.stat_post, r.x
            if c["ckpt"]:
                out["y8"] = r.saved.y.unpack(torch.bfloat16)
        if c["pre"]:
            out["stat_pre"], out["h"] = r.saved.stat_pre, r.h
            if c["ckpt"]:
                out["x8"] = r.saved.x.unpack(torch.bfloat16)
        return out
    keep = (lambda v: laga.Checkpoint8(v, c["d"])) if c["ckpt"] else (lambda v: v)
    saved = laga.ResidualSaved(y=keep(st["y"]) if c["post"] else None,
                               x=keep(st["x"]) if c["pre"] else None,
                               stat_post=st.get("stat_post"), stat_pre=st.get("stat_pre"), **gains)
    g = plan.backward(saved, st["dx_out"], st.get("dh"))
    out = {}
    if c["pre"]:
        out["dgamma_pre"], out["dx"] = g.dgamma_pre, g.dx
    if c["post"]:
        if c["gate"] != "none":
            out["dgate"] = g.dgate
        out["dalpha"] = g.dalpha
        if c["norm_post"] != "none":
            out["dgamma_post"] = g.dgamma_post
        out["dy"] = g.dy
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work
def work(case):
    rows, d = case["rows"], case["d"]
    b = 2 if case["dtype"] == "bf16" else 4
    n, row8 = rows * d, _pitch(d)[1]
    if case["op"] == "pack":                 # the activation in, the values it stands for out
        return {"bytes": 2 * n * b, "flops": 4 * n}
    if case["op"] == "dw":
        out = 4 * d * case["n"] + (4 * d if case["gain"] else 0)
        return {"bytes": rows * row8 + rows * case["n"] * b + out, "flops": 2 * n * case["n"]}
    post, pre, fwd = case["post"], case["pre"], case["op"] == "res_fwd"
    gate = 0 if not post else {"none": 0, "token": rows * b, "full": n * b}[case["gate"]]
    total = gate + (4 * d if pre else 0) + (4 * d if post and case["norm_post"] != "none" else 0)
    stats = 8 * rows * (int(post) + int(pre))
    if fwd:
        total += n * b * (3 if post else 1)              # x, y, x'
        total += n * b if pre else 0                     # h
        total += 2 * n * (int(post) + int(pre)) if case["ckpt"] else 0
        return {"bytes": total + stats, "flops": n * (12 * int(post) + 8 * int(pre))}
    kept = rows * row8 if case["ckpt"] else n * b
    total += stats + gate + kept * (int(post) + int(pre)) + n * b     # and dgate, D
    total += 2 * n * b + 4 * d if pre else 0             # dh, dx, dgamma_pre
    total += n * b + 4 if post else 0                    # dy, dalpha
    total += 4 * d if post and case["norm_post"] != "none" else 0
    return {"bytes": total, "flops": n * (20 * int(post) + 10 * int(pre))}


# ------------------------------------------------------------------ 64 bits
def _exact_round8(v):
    """What the 8-bit form of float64 values stands for, by the definition:
    per group the smallest power of two 2^e with max|v| <= 448 2^e, then the
    nearest multiple of the e4m3 step at |v| 2^-e (ties to even)."""
    rows, d = v.shape
    out = torch.empty_like(v)
    for c0 in range(0, d, GROUP):
        g = v[:, c0:c0 + GROUP]
        top = g.abs().max(dim=1, keepdim=True).values
        e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 448.0))
        for _ in range(2):     # log2 may be a unit off next to a border
            e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
            e = torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e)
        unit = torch.exp2(e.clamp(E_MIN, E_MAX))
        t = (g / unit).clamp(-448.0, 448.0)
        binade = torch.full_like(t, -6.0)
        for k in range(-5, 9):
            binade = torch.where(t.abs() >= 2.0 ** k, torch.full_like(t, float(k)), binade)
        step = torch.exp2(binade - 3.0)
        r = torch.round(t / step) * step * unit
        out[:, c0:c0 + GROUP] = torch.where(torch.isfinite(g).all(dim=1, keepdim=True), r,
                                            torch.full_like(r, float("nan")))
    return out


def _exact_kept(buf, d):
    """float64 values of checkpoint rows, from the bits of the codes."""
    cols, _ = _pitch(d)
    b = buf[:, :cols].to(torch.int64)
    expo, frac = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(expo > 0, (1.0 + frac / 8.0) * torch.exp2((expo - 7).double()),
                      frac / 8.0 * 2.0 ** -6)
    v = torch.where(b >= 128, -mag, mag)
    scale = torch.exp2(buf[:, cols:cols + cols // GROUP].double() - 127.0)
    return (v * scale.repeat_interleave(GROUP, dim=1))[:, :d]


def _exact_stat(v, norm):
    if norm == "none":
        return torch.zeros(len(v), 1, device=v.device, dtype=v.dtype), torch.ones(
            len(v), 1, device=v.device, dtype=v.dtype)
    if norm == "rms":
        mu = torch.zeros(len(v), 1, device=v.device, dtype=v.dtype)
        return mu, (v.square().sum(dim=1, keepdim=True) / v.shape[1] + EPS).rsqrt()
    var, mu = torch.var_mean(v, dim=1, keepdim=True, correction=0)
    return mu, (var + EPS).rsqrt()


def exact(case, seed):
    st = prepare(case, seed)
    d = case["d"]
    f = {k: v.double() for k, v in st.items()
         if isinstance(v, torch.Tensor) and v.dtype != torch.uint8}
    if case["op"] == "pack":
        return {"x8": _exact_round8(f["x"])}
    if case["op"] == "dw":
        left = _exact_kept(st["ck"], d)
        if case["gain"]:
            left = left * f["gamma"]
        return {"dw": torch.einsum("tc,tn->cn", left, f["dy"])}
    sig = torch.sigmoid(f["gate"]) if "gate" in f else 1.0
    gp = f.get("gamma_post", 1.0)
    out = {}
    if case["op"] == "res_fwd":
        x = f["x"]
        if case["post"]:
            mu, r = _exact_stat(f["y"], case["norm_post"])
            out["stat_post"] = torch.cat([mu, r], dim=1)
            hat = (f["y"] - mu) * r
            x = x + f["alpha"] * sig * (gp * hat)
            out["x"] = x
            if case["ckpt"]:
                out["y8"] = _exact_round8(hat)
        if case["pre"]:
            mu, r = _exact_stat(x, case["norm_pre"])
            out["stat_pre"] = torch.cat([mu, r], dim=1)
            hat = (x - mu) * r
            out["h"] = hat * f["gamma_pre"]
            if case["ckpt"]:
                out["x8"] = _exact_round8(hat)
        return out

    def back(g, hat, r, norm):
        # transpose of v -> (v - mean) r at fixed data: r (I - P) with P the
        # projection on the row of ones (LayerNorm) and on hat
        if norm == "none":
            return g
        proj = hat * (g * hat).sum(dim=1, keepdim=True) / d
        if norm == "layer":
            proj = proj + g.sum(dim=1, keepdim=True) / d
        return r * (g - proj)

    def kept(name, stat):
        if case["ckpt"]:
            return _exact_kept(st[name], d)
        return (f[name] - f[stat][:, :1]) * f[stat][:, 1:]

    D = f["dx_out"]
    if case["pre"]:
        hat = kept("x", "stat_pre")
        out["dgamma_pre"] = torch.einsum("td,td->d", f["dh"], hat)
        D = D + back(f["dh"] * f["gamma_pre"], hat, f["stat_pre"][:, 1:], case["norm_pre"])
        out["dx"] = D
    if case["post"]:
        hat = kept("y", "stat_post")
        if "gate" in f:
            da = f["alpha"] * D * (gp * hat) * sig * torch.sigmoid(-f["gate"])
            out["dgate"] = da if case["gate"] == "full" else da.sum(dim=1, keepdim=True)
        out["dalpha"] = (D * sig * gp * hat).sum().reshape(1)
        du = f["alpha"] * D * sig
        if "gamma_post" in f:
            out["dgamma_post"] = torch.einsum("td,td->d", du, hat)
        out["dy"] = back(du * gp, hat, f["stat_post"][:, 1:], case["norm_post"])
    return out
