"""Cases, plain forms and 64-bit values of the experts' products in 8-bit floating point and of their
training: a product with a scale for each block of 128, products grouped by expert with both of
their gradients, and 8-bit checkpoints of the SwiGLU activations.

    f8       tokens in 8-bit floating point (a scale per row and 128 channels) times their experts'
             8-bit weights (a scale per 128 x 128 block)
    product  each expert's rows times its weight matrix, ragged row counts
    dx       gradient of the rows: dy W, or dg W1 + du W3 of a SwiGLU layer in one call
    dw       gradient of each expert's weights: dy^T x over its rows, x as it is or from an 8-bit checkpoint
    ckpt     h = silu(g) u keeping g and u in 8 bits, and its backward pass from what was kept
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
BLOCK = 128


def listed():
    return [
        # the up product of a decode batch: two or three rows an expert, the weights are the work
        dict(name="f8 decode", op="f8", T=64, K=6, E=160, n_in=5120, n_out=1536, dtype="bf16", pow2=0),
        # a ragged batch over a few wide experts
        dict(name="f8 wide ragged", op="f8", T=1001, K=2, E=8, n_in=4096, n_out=14336, dtype="f32", pow2=1),
        # prefill over many small experts
        dict(name="f8 prefill", op="f8", T=16384, K=8, E=128, n_in=2048, n_out=768, dtype="bf16", pow2=1),
        # fp32 weights, odd sizes, a handful of rows an expert
        dict(name="product f32 13", op="product", T=13, K=3, E=24, n_in=1000, n_out=1416, dtype="f32"),
        # the down product of a training batch over many experts
        dict(name="product train", op="product", T=8192, K=6, E=160, n_in=1536, n_out=5120, dtype="bf16"),
        # the smallest layer's gradient, gate and up together
        dict(name="dx f32 tiny", op="dx", T=64, K=2, E=8, n_in=128, n_out=256, dtype="f32", pair=True),
        # wide experts, gate and up together: the largest contraction
        dict(name="dx wide pair", op="dx", T=4096, K=2, E=8, n_in=4096, n_out=14336, dtype="bf16", pair=True),
        # fp32, odd sizes, experts with few rows or none
        dict(name="dw f32 ragged", op="dw", T=301, K=3, E=24, n_in=1000, n_out=1416, dtype="f32",
             x8=False, add=False),
        # many experts' weight gradient from the layer's input kept in 8 bits, in token order
        dict(name="dw train kept x", op="dw", T=8192, K=6, E=160, n_in=5120, n_out=1536, dtype="bf16",
             x8=True, add=False),
        # small experts, many rows each, added to the gradient of the batches before
        dict(name="dw accumulated", op="dw", T=16384, K=8, E=128, n_in=2048, n_out=768, dtype="bf16",
             x8=False, add=True),
        # a short batch's activations: latency
        dict(name="ckpt short", op="ckpt", rows=384, F=1536, dtype="bf16"),
        # all rows of a training batch over small experts
        dict(name="ckpt train", op="ckpt", rows=131072, F=768, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, step):
    return max(lo, _log(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(["f8", "f8", "product", "dx", "dw", "ckpt"])
    if op == "ckpt":
        while True:
            c = dict(op=op, rows=_log(rng, 1, 131072), F=_mult(rng, 16, 14336, 16),
                     dtype=rng.choice(["bf16", "bf16", "f32"]))
            if c["rows"] * c["F"] <= 1e8:
                return c
    while True:
        E = _log(rng, 1, 160)
        c = dict(op=op, T=_log(rng, 1, 16384), K=rng.randint(1, min(8, E)), E=E,
                 n_in=_mult(rng, 64, 5120, 16 if op in ("f8", "dw") else 8),
                 n_out=_mult(rng, 64, 5120, 8), dtype=rng.choice(["bf16", "bf16", "f32"]))
        if op == "f8":
            c |= dict(pow2=rng.choice([0, 1]))
        if op == "dx":
            c |= dict(pair=rng.random() < 0.5)
        if op == "dw":
            c |= dict(x8=rng.random() < 0.5, add=rng.random() < 0.4)
        macs, weights = c["T"] * c["K"] * c["n_in"] * c["n_out"], E * c["n_in"] * c["n_out"]
        small = c["dtype"] == "f32" and op != "f8"
        if macs <= (2e10 if small else 2e11) and weights <= (2e8 if small else 1.2e9):
            return c


def _touched(E, n):
    """Experts that n independent draws out of E are expected to meet."""
    return E * (1.0 - (1.0 - 1.0 / E) ** n)


def work(case):
    c = case
    b = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "ckpt":
        # forward: g and u in, h and both in 8 bits out; backward: dh and both in, dg, du and h out
        n, s = c["rows"] * c["F"], c["rows"] * -(-c["F"] // BLOCK)
        return {"bytes": n * (3 * b + 2 + 2 + 4 * b) + 16 * s, "flops": 20 * n}
    rows, n_in, n_out, E = c["T"] * c["K"], c["n_in"], c["n_out"], c["E"]
    act = _touched(E, rows)
    flops = 2 * rows * n_in * n_out
    if c["op"] == "f8":
        kb = -(-n_in // BLOCK)
        return {"bytes": act * (n_out * n_in + 4 * -(-n_out // BLOCK) * kb) + c["T"] * (n_in * b + 4 * kb)
                + rows * (4 + n_out * b) + 4 * E, "flops": flops}
    if c["op"] == "product":
        return {"bytes": b * (act * n_out * n_in + rows * (n_in + n_out)) + 4 * E, "flops": flops}
    if c["op"] == "dx":
        n = 2 if c["pair"] else 1
        return {"bytes": b * (n * act * n_out * n_in + rows * (n * n_out + n_in)) + 4 * E, "flops": n * flops}
    x = c["T"] * (n_in + 4 * -(-n_in // BLOCK)) + 4 * rows if c["x8"] else rows * n_in * b
    return {"bytes": rows * n_out * b + x + E * n_out * n_in * (8 if c["add"] else 4) + 4 * E, "flops": flops}


# ---------------------------------------------------------------- inputs
def _gen(seed, salt=0):
    g = torch.Generator(device=DEV)
    g.manual_seed((int(seed) * 1000003 + salt) & ((1 << 62) - 1))
    return g


def _randn(shape, std, dtype, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype).mul_(std)


def _tokens(T, d, g):
    """Rows of a clustered embedding with noise, as decoder states of related tokens are, with a
    few channels of large activations."""
    cent = torch.randn(64, d, generator=g, device=DEV)
    pick = torch.randint(0, 64, (T,), generator=g, device=DEV)
    loud = torch.rand(d, generator=g, device=DEV) < 0.005
    return (cent[pick] + 0.5 * torch.randn(T, d, generator=g, device=DEV)) * torch.where(loud, 6.0, 1.0)


def _routes(T, K, E, seed):
    """Dispatched rows of T tokens with K experts each, some experts busier than others: the
    token of each row in expert order, the experts' row offsets, the most rows of one expert."""
    rng = np.random.RandomState(int(seed) % (1 << 31))
    p = (1.0 + rng.permutation(E)) ** -0.3
    idx = rng.choice(E, size=T * K, p=p / p.sum())
    order = np.argsort(idx, kind="stable")
    n = np.bincount(idx, minlength=E)
    off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    return (torch.as_tensor((order // K).astype(np.int32), device=DEV),
            torch.as_tensor(off, device=DEV), int(n.max()))


def _blocks(n):
    return -(-n // BLOCK)


def _weights_f8(E, n_out, n_in, g):
    """Weights N(0, 1/n_in) in 8-bit floating point with a scale per 128 x 128 block."""
    nb, kb = _blocks(n_out), _blocks(n_in)
    q = torch.empty(E, n_out, n_in, dtype=F8, device=DEV)
    s = torch.empty(E, nb, kb, device=DEV)
    step = max(1, (1 << 27) // (nb * kb * BLOCK * BLOCK))
    for e in range(0, E, step):
        n = min(step, E - e)
        w = torch.zeros(n, nb * BLOCK, kb * BLOCK, device=DEV)
        w[:, :n_out, :n_in] = torch.randn(n, n_out, n_in, generator=g, device=DEV).mul_(1.0 / math.sqrt(n_in))
        v = w.view(n, nb, BLOCK, kb, BLOCK)
        s[e:e + n] = v.abs().amax((2, 4)) / F8_MAX
        v = v / s[e:e + n, :, None, :, None]
        q[e:e + n] = v.reshape(n, nb * BLOCK, kb * BLOCK)[:, :n_out, :n_in].to(F8)
    return q, s


def _block_scale(x, pow2):
    """The scale of each row's 128-blocks: the largest magnitude over 448, or the power of two
    that is not below it."""
    T, d = x.shape
    pad = torch.zeros(T, _blocks(d) * BLOCK, dtype=x.dtype, device=x.device)
    pad[:, :d] = x.abs()
    s = pad.view(T, -1, BLOCK).amax(-1)
    s = s / torch.full_like(s, F8_MAX)  # (by a number torch would multiply with its inverse)
    if pow2:
        m, e = torch.frexp(s)
        s = torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e))
    return s


def _spread(s, d):
    return s.repeat_interleave(BLOCK, -1)[..., :d]


def _quantise(x, pow2):
    s = _block_scale(x, pow2)
    return (x / _spread(s, x.shape[1])).to(F8), s


def prepare(case, seed):
    c, g = case, _gen(seed)
    st, dt = {"case": dict(c)}, TYPES[case["dtype"]]
    if c["op"] == "ckpt":
        rows, F = c["rows"], c["F"]
        st["g"], st["u"] = _randn((rows, F), 1.2, dt, g), _randn((rows, F), 1.0, dt, g)
        st["dh"] = _randn((rows, F), 0.02, dt, g)
    else:
        T, K, E, n_in, n_out = (c[k] for k in ("T", "K", "E", "n_in", "n_out"))
        st["row_src"], st["off"], st["cap"] = _routes(T, K, E, seed)
        R = T * K
        if c["op"] == "f8":
            st["x"] = _tokens(T, n_in, g).to(dt)
            st["wq"], st["ws"] = _weights_f8(E, n_out, n_in, g)
        elif c["op"] == "product":
            st["x"] = _tokens(T, n_in, g).to(dt)[st["row_src"].long()]
            st["w"] = _randn((E, n_out, n_in), 1.0 / math.sqrt(n_in), dt, g)
        elif c["op"] == "dx":
            for k in ("", "2") if c["pair"] else ("",):
                st["dy" + k] = _randn((R, n_out), 0.02, dt, g)
                st["w" + k] = _randn((E, n_out, n_in), 1.0 / math.sqrt(n_in), dt, g)
        else:
            st["dy"] = _randn((R, n_out), 0.02, dt, g)
            x = _tokens(T, n_in, g).to(dt)
            if c["x8"]:
                st["xq"], st["xs"] = _quantise(x.float(), 1)
            else:
                st["x"] = x[st["row_src"].long()]
            if c["add"]:
                st["before"] = _randn((E, n_out, n_in), 0.1, torch.float32, g)
    if own:
        _own_state(st)
    return st


# ---------------------------------------------------------------- the framework's calls
def _own_state(st):
    import routing_token_shuffle_gb300 as smoe

    c, dt = st["case"], TYPES[st["case"]["dtype"]]
    st["smoe"] = smoe
    new = lambda *s, dtype=dt: torch.empty(*s, dtype=dtype, device=DEV)  # noqa: E731
    if c["op"] == "ckpt":
        rows, F = c["rows"], c["F"]
        st["desc"] = smoe.make_desc(rows, F, 1, 1, 1, F, 0, 1, 1, c["dtype"])
        for k in ("g8", "u8"):
            st[k], st[k + "s"] = new(rows, F, dtype=F8), new(rows, _blocks(F), dtype=torch.float32)
        for k in ("h", "h_again", "dg", "du"):
            st[k] = new(rows, F)
        return
    T, K, E, n_in, n_out = (c[k] for k in ("T", "K", "E", "n_in", "n_out"))
    st["desc"] = smoe.make_desc(T, n_in, E, K, 1, n_out, 0, 1, 1, c["dtype"])
    st["work"] = smoe.workspace_products(st["desc"])
    if c["op"] == "f8":
        st["xq"], st["xs"] = new(T, n_in, dtype=F8), new(T, _blocks(n_in), dtype=torch.float32)
    st["out"] = new(E, n_out, n_in, dtype=torch.float32) if c["op"] == "dw" else \
        new(T * K, n_in if c["op"] == "dx" else n_out)


def _run_own(st):
    c, smoe = st["case"], st["smoe"]
    if c["op"] == "ckpt":
        smoe.smoe_swiglu_f8(st["desc"], st["g"], st["u"], h=st["h"], g8=st["g8"], g8_scale=st["g8s"],
                            u8=st["u8"], u8_scale=st["u8s"], pow2=1)
        smoe.smoe_swiglu_grad_f8(st["desc"], st["dh"], st["g8"], st["g8s"], st["u8"], st["u8s"],
                                 st["dg"], st["du"], h=st["h_again"])
        return {k: st[k] for k in ("h", "g8s", "u8s", "dg", "du", "h_again")}
    if c["op"] == "f8":
        smoe.smoe_rows_f8(st["desc"], st["x"], st["xq"], st["xs"], pow2=c["pow2"])
        smoe.smoe_expert_matmul_f8(st["desc"], st["xq"], st["xs"], st["off"], st["wq"], st["ws"],
                                   st["out"], st["work"], row_src=st["row_src"])
        return {"y": st["out"], "scale": st["xs"]}
    if c["op"] == "product":
        smoe.smoe_expert_matmul(st["desc"], st["x"], st["off"], st["w"], st["out"], st["work"])
    elif c["op"] == "dx":
        smoe.smoe_expert_matmul_dx(st["desc"], st["dy"], st["w"], st["off"], st["out"], st["work"],
                                   dy2=st.get("dy2"), w2=st.get("w2"))
    elif c["x8"]:
        smoe.smoe_expert_matmul_dw_f8(st["desc"], st["dy"], st["xq"], st["xs"], st["off"], st["out"],
                                      st["work"], row_src=st["row_src"], add=st.get("before"))
    else:
        smoe.smoe_expert_matmul_dw(st["desc"], st["dy"], st["x"], st["off"], st["out"], st["work"],
                                   add=st.get("before"))
    return st["out"]


# ---------------------------------------------------------------- plain forms
def _places(st):
    """Each row's expert and its place among that expert's rows."""
    r = torch.arange(st["case"]["T"] * st["case"]["K"], device=DEV)
    e = torch.bucketize(r, st["off"][1:].long(), right=True)
    return e, r - st["off"].long()[e]


def _padded(st, rows, e, pos):
    """[E, most rows of one expert, channels], zeros behind each expert's rows."""
    x = torch.zeros(st["case"]["E"], st["cap"], rows.shape[1], device=DEV)
    x[e, pos] = rows.float()
    return x


def _plain_f8(st):
    c = st["case"]
    xq, s = _quantise(st["x"].float(), c["pow2"])
    x = xq.float() * _spread(s, c["n_in"])
    w = st["wq"].float()
    w *= _spread(st["ws"], c["n_in"]).repeat_interleave(BLOCK, 1)[:, :c["n_out"]]
    e, pos = _places(st)
    y = torch.bmm(_padded(st, x[st["row_src"].long()], e, pos), w.transpose(1, 2))[e, pos]
    return {"y": y.to(TYPES[c["dtype"]]), "scale": s}


def _plain_product(st):
    e, pos = _places(st)
    y = torch.bmm(_padded(st, st["x"], e, pos), st["w"].float().transpose(1, 2))[e, pos]
    return y.to(TYPES[st["case"]["dtype"]])


def _plain_dx(st):
    e, pos = _places(st)
    d = torch.bmm(_padded(st, st["dy"], e, pos), st["w"].float())
    if st["case"]["pair"]:
        d = torch.baddbmm(d, _padded(st, st["dy2"], e, pos), st["w2"].float())
    return d[e, pos].to(TYPES[st["case"]["dtype"]])


def _plain_dw(st):
    c = st["case"]
    e, pos = _places(st)
    x = (st["xq"].float() * _spread(st["xs"], c["n_in"]))[st["row_src"].long()] if c["x8"] else st["x"]
    dw = torch.bmm(_padded(st, st["dy"], e, pos).transpose(1, 2), _padded(st, x, e, pos))
    return dw + st["before"] if c["add"] else dw


def _plain_ckpt(st):
    dt, F = TYPES[st["case"]["dtype"]], st["case"]["F"]
    g, u, dh = st["g"].float(), st["u"].float(), st["dh"].float()
    h = g / (1.0 + torch.exp(-g)) * u
    (g8, gs), (u8, us) = _quantise(g, 1), _quantise(u, 1)
    g, u = g8.float() * _spread(gs, F), u8.float() * _spread(us, F)
    sig = 1.0 / (1.0 + torch.exp(-g))
    silu = g * sig
    return {"h": h.to(dt), "g8s": gs, "u8s": us, "dg": (dh * u * (sig * (1.0 + g * (1.0 - sig)))).to(dt),
            "du": (dh * silu).to(dt), "h_again": (silu * u).to(dt)}


def run(state):
    if own:
        return _run_own(state)
    return {"f8": _plain_f8, "product": _plain_product, "dx": _plain_dx, "dw": _plain_dw,
            "ckpt": _plain_ckpt}[state["case"]["op"]](state)


# ---------------------------------------------------------------- 64 bits
def _held(x, pow2):
    """What x stands for once it is held in 8 bits, and the scales: block by block."""
    T, d = x.shape
    out, scales = torch.empty_like(x), []
    for k in range(0, d, BLOCK):
        b = x[:, k:k + BLOCK]
        s = b.abs().max(dim=1).values / 448
        if pow2:
            near = torch.exp2(torch.round(torch.log2(s)))
            s = torch.where(near < s, 2 * near, near)
        # three bits behind the leading one, and steps of 2^-9 for the smallest
        v = b / s[:, None]
        step = torch.exp2(torch.clamp(torch.floor(torch.log2(v.abs().clamp_min(1e-30))), min=-6) - 3)
        out[:, k:k + BLOCK] = torch.round(v / step) * step * s[:, None]
        scales.append(s)
    return out, torch.stack(scales, 1)


def exact(case, seed):
    c, st, f64 = case, prepare(case, seed), torch.float64
    if c["op"] == "ckpt":
        g, u, dh = (st[k].to(f64) for k in ("g", "u", "dh"))
        h = g * torch.sigmoid(g) * u
        (g, gs), (u, us) = _held(g, 1), _held(u, 1)
        s = torch.sigmoid(g)
        return {"h": h, "g8s": gs, "u8s": us, "dg": dh * u * (s + g * s * (1 - s)), "du": dh * g * s,
                "h_again": g * s * u}
    off, src = st["off"].tolist(), st["row_src"].long()
    E, n_in, n_out, R = c["E"], c["n_in"], c["n_out"], c["T"] * c["K"]
    seg = lambda e: slice(off[e], off[e + 1])  # noqa: E731
    if c["op"] == "f8":
        x, scale = _held(st["x"].to(f64), c["pow2"])
        y = torch.empty(R, n_out, dtype=f64, device=DEV)
        for e in range(E):
            if off[e + 1] > off[e]:
                s = st["ws"][e].to(f64).repeat_interleave(BLOCK, 0)[:n_out].repeat_interleave(BLOCK, 1)[:, :n_in]
                y[seg(e)] = x[src[seg(e)]] @ (st["wq"][e].to(f64) * s).T
        return {"y": y, "scale": scale}
    if c["op"] in ("product", "dx"):
        out = torch.zeros(R, n_out if c["op"] == "product" else n_in, dtype=f64, device=DEV)
        for e in range(E):
            if off[e + 1] == off[e]:
                continue
            if c["op"] == "product":
                out[seg(e)] = st["x"][seg(e)].to(f64) @ st["w"][e].to(f64).T
            else:
                for k in ("", "2") if c["pair"] else ("",):
                    out[seg(e)] += st["dy" + k][seg(e)].to(f64) @ st["w" + k][e].to(f64)
        return out
    out = st["before"].to(f64) if c["add"] else torch.zeros(E, n_out, n_in, dtype=f64, device=DEV)
    for e in range(E):
        if c["x8"]:
            t = src[seg(e)]
            x = st["xq"][t].to(f64) * st["xs"][t].to(f64).repeat_interleave(BLOCK, 1)[:, :n_in]
        else:
            x = st["x"][seg(e)].to(f64)
        out[e] += st["dy"][seg(e)].to(f64).T @ x
    return out
