"""Cases, plain forms and 64-bit values of the serving operators around the MoE layer.

    add_rmsnorm    r + y, its root-mean-square norm, and the norm in 8 bits with a scale per row
    moe_few        a whole MoE layer (gate, top-K, SwiGLU experts, weighted sum) for 1 to 64 tokens
    matmul_i8      rows of 8-bit integers times their experts' 8-bit weights, a scale per row and channel
    ffn_i8         the experts' SwiGLU FFN on 8-bit integers, the hidden rows requantised in between
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the norm in front of a router while one token is decoded
        dict(name="norm decode 1", op="norm", T=1, d=5120, dtype="bf16", y=True, x=True, q=False),
        # an fp32 layer's ragged batch: norm, and the 8-bit rows of an 8-bit FFN
        dict(name="norm ragged f32", op="norm", T=1001, d=4096, dtype="f32", y=True, x=True, q=True),
        # prefill: every output at once
        dict(name="norm prefill", op="norm", T=8192, d=5120, dtype="bf16", y=True, x=True, q=True),
        # one decoded token on the grouped router of small experts: latency
        dict(name="few grouped 1", op="few", T=1, d=2048, E=128, K=8, H=8, F=768, n_shared=0,
             dtype="bf16", renorm=1),
        # a few wide experts, three tokens (a short speculative draft)
        dict(name="few wide 3", op="few", T=3, d=4096, E=8, K=2, H=1, F=14336, n_shared=0,
             dtype="bf16", renorm=0),
        # many experts and two shared ones: the decode step's whole batch
        dict(name="few shared 64", op="few", T=64, d=5120, E=160, K=6, H=1, F=1536, n_shared=2,
             dtype="bf16", renorm=0),
        # fp32 weights, odd sizes
        dict(name="few f32 13", op="few", T=13, d=1000, E=24, K=3, H=1, F=1416, n_shared=1,
             dtype="f32", renorm=1),
        # 8-bit up product of a decode batch: few rows an expert, the weights are the work
        dict(name="matmul decode", op="matmul", T=64, K=6, E=160, n_in=5120, n_out=1536,
             dtype="bf16"),
        # 8-bit product of a prefill batch over small experts
        dict(name="matmul prefill", op="matmul", T=16384, K=8, E=128, n_in=2048, n_out=768,
             dtype="f32"),
        # 8-bit FFN while 5 tokens are decoded, shared experts included
        dict(name="ffn decode 5", op="ffn", T=5, d=5120, E=160, K=6, F=1536, n_shared=2),
        # ragged batch over wide experts
        dict(name="ffn wide ragged", op="ffn", T=1001, d=4096, E=8, K=2, F=14336, n_shared=0),
        # prefill over many experts and two shared ones
        dict(name="ffn prefill", op="ffn", T=8192, d=5120, E=160, K=6, F=1536, n_shared=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, step):
    return max(lo, _log(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(["norm", "few", "few", "matmul", "ffn"])
    while True:
        if op == "norm":
            c = dict(op=op, T=_log(rng, 1, 8192), d=_mult(rng, 64, 8192, 8),
                     dtype=rng.choice(["bf16", "bf16", "f32"]), y=rng.random() < 0.75,
                     x=True, q=rng.random() < 0.6)
            if c["T"] * c["d"] <= 8192 * 5120:
                return c
        elif op == "few":
            E = _log(rng, 4, 160)
            H = rng.choice([h for h in (1, 1, 2, 4, 8) if E % h == 0])
            K = H * min(rng.choice([1, 2, 3]), E // H)
            c = dict(op=op, T=_log(rng, 1, 64), d=_mult(rng, 256, 5120, 8), E=E, K=K, H=H,
                     F=_mult(rng, 64, 8192, 8), n_shared=rng.choice([0, 0, 1, 2]),
                     dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), renorm=rng.choice([0, 1]))
            size = 4 if c["dtype"] == "f32" else 2
            if (E + 2) * 3 * c["d"] * c["F"] * size <= 6.4e9 // (1 if size == 2 else 4) and K <= 24:
                return c
        elif op == "matmul":
            E = _log(rng, 1, 160)
            c = dict(op=op, T=_log(rng, 1, 8192), K=rng.randint(1, min(8, E)), E=E,
                     n_in=_mult(rng, 64, 5120, 16), n_out=_mult(rng, 64, 5120, 8),
                     dtype=rng.choice(["bf16", "f32"]))
            if c["T"] * c["K"] * c["n_in"] * c["n_out"] <= 2e11 and E * c["n_in"] * c["n_out"] <= 1.2e9:
                return c
        else:
            E = _log(rng, 1, 160)
            c = dict(op=op, T=_log(rng, 1, 4096), d=_mult(rng, 64, 5120, 16), E=E,
                     K=rng.randint(1, min(8, E)), F=_mult(rng, 64, 4096, 16),
                     n_shared=rng.choice([0, 0, 1, 2]))
            rows = c["T"] * (c["K"] + c["n_shared"])
            if rows * c["d"] * c["F"] <= 2e11 and (E + 2) * c["d"] * c["F"] <= 1.2e9:
                return c


def _touched(E, n):
    """Experts that n independent draws out of E are expected to meet."""
    return E * (1.0 - (1.0 - 1.0 / E) ** n)


def work(case):
    c = case
    if c["op"] == "norm":
        b = 4 if c["dtype"] == "f32" else 2
        per = 4 + (b + 4 if c["y"] else 0) + (b if c["x"] else 0) + (1 if c["q"] else 0)
        return {"bytes": c["T"] * c["d"] * per + 4 * c["d"] + (4 * c["T"] if c["q"] else 0),
                "flops": 4 * c["T"] * c["d"]}
    if c["op"] == "few":
        b = 4 if c["dtype"] == "f32" else 2
        act = c["E"] * (1.0 - (1.0 - c["K"] / c["E"]) ** c["T"]) + c["n_shared"]
        pairs = c["T"] * (c["K"] + c["n_shared"])
        return {"bytes": b * (3 * act * c["d"] * c["F"] + c["E"] * c["d"] + 2 * c["T"] * c["d"])
                + 8 * c["T"] * c["K"],
                "flops": 6 * pairs * c["d"] * c["F"] + 2 * c["T"] * c["E"] * c["d"]}
    if c["op"] == "matmul":
        rows, b = c["T"] * c["K"], 4 if c["dtype"] == "f32" else 2
        act = _touched(c["E"], rows)
        return {"bytes": act * c["n_out"] * (c["n_in"] + 4) + c["T"] * (c["n_in"] + 4)
                + rows * (4 + c["n_out"] * b) + 4 * c["E"],
                "flops": 2 * rows * c["n_in"] * c["n_out"]}
    rows = c["T"] * (c["K"] + c["n_shared"])
    act = _touched(c["E"], c["T"] * c["K"]) + c["n_shared"]
    return {"bytes": act * (3 * c["d"] * c["F"] + 8 * c["F"] + 4 * c["d"])
            + c["T"] * (c["d"] + 4) + rows * 2 * c["d"] + 4 * c["T"] * c["K"],
            "flops": 6 * rows * c["d"] * c["F"]}


# ---------------------------------------------------------------- inputs
def _gen(seed, salt=0):
    g = torch.Generator(device=DEV)
    g.manual_seed((int(seed) * 1000003 + salt) & ((1 << 62) - 1))
    return g


def _randn(shape, std, dtype, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype).mul_(std)


def _tokens(T, d, g):
    """Rows of a clustered embedding with noise, as decoder states of related tokens are."""
    cent = torch.randn(64, d, generator=g, device=DEV)
    pick = torch.randint(0, 64, (T,), generator=g, device=DEV)
    return cent[pick] + 0.5 * torch.randn(T, d, generator=g, device=DEV)


def _quantised(shape, g):
    """Weights N(0, 1/n_in) in 8 bits with a scale per output channel."""
    E, n, k = shape
    q = torch.empty(shape, dtype=torch.int8, device=DEV)
    s = torch.empty((E, n), dtype=torch.float32, device=DEV)
    step = max(1, (1 << 27) // (n * k))
    for e in range(0, E, step):
        w = torch.randn(min(step, E - e), n, k, generator=g, device=DEV).mul_(1.0 / math.sqrt(k))
        sc = w.abs().amax(-1) / 127.0
        s[e:e + step] = sc
        q[e:e + step] = torch.round(w / sc[..., None]).to(torch.int8)
    return q, s


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


def _rows_i8(T, d, g):
    """Normalised rows in 8 bits with a scale per row."""
    x = _tokens(T, d, g)
    s = x.abs().amax(-1) / 127.0
    return torch.round(x / s[:, None]).to(torch.int8), s.contiguous()


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = {"case": dict(c)}
    if own:
        import routing_token_shuffle_gb300 as smoe
        st["smoe"] = smoe
    if c["op"] == "norm":
        T, d, dt = c["T"], c["d"], TYPES[c["dtype"]]
        st["r"] = torch.randn(T, d, generator=g, device=DEV)
        loud = torch.rand(d, generator=g, device=DEV) < 0.005  # channels of large activations
        st["r"] *= torch.where(loud, 6.0, 1.0)
        st["y"] = _randn((T, d), 0.5, dt, g) if c["y"] else None
        st["gamma"] = 1.0 + 0.1 * torch.randn(d, generator=g, device=DEV)
        if own:
            st["desc"] = smoe.make_desc(T, d, 1, 1, 1, 8, 0, 1, 1, c["dtype"])
            st["r_out"] = torch.empty_like(st["r"]) if c["y"] else None
            st["x_out"] = torch.empty(T, d, dtype=dt, device=DEV) if c["x"] else None
            st["q"] = torch.empty(T, d, dtype=torch.int8, device=DEV) if c["q"] else None
            st["qs"] = torch.empty(T, device=DEV) if c["q"] else None
            st["deq"] = torch.empty(T, d, dtype=torch.bfloat16, device=DEV) if c["q"] else None
    elif c["op"] == "few":
        T, d, E, F, dt = c["T"], c["d"], c["E"], c["F"], TYPES[c["dtype"]]
        n = E + c["n_shared"]
        st["x"] = _tokens(T, d, g).to(dt)
        st["w_gate"] = _randn((E, d), 1.0 / math.sqrt(d), dt, g)
        st["w1"] = _randn((n, F, d), 1.0 / math.sqrt(d), dt, g)
        st["w3"] = _randn((n, F, d), 1.0 / math.sqrt(d), dt, g)
        st["w2"] = _randn((n, d, F), 1.0 / math.sqrt(F), dt, g)
        if own:
            st["desc"] = smoe.make_desc(T, d, E, c["K"], c["H"], F, c["n_shared"], 1, 1,
                                        c["dtype"], c["renorm"])
            st["ws"] = smoe.workspace_few(st["desc"])
            st["out"] = torch.empty(T, d, dtype=dt, device=DEV)
            st["idx"] = torch.empty(T, c["K"], dtype=torch.int32, device=DEV)
            st["w"] = torch.empty(T, c["K"], device=DEV)
    elif c["op"] == "matmul":
        T, K, E, dt = c["T"], c["K"], c["E"], TYPES[c["dtype"]]
        st["row_src"], st["off"], st["cap"] = _routes(T, K, E, seed)
        st["xq"], st["xs"] = _rows_i8(T, c["n_in"], g)
        st["wq"], st["ws_"] = _quantised((E, c["n_out"], c["n_in"]), g)
        if own:
            st["desc"] = smoe.make_desc(T, c["n_in"], E, K, 1, c["n_out"], 0, 1, 1, c["dtype"])
            st["ws"] = smoe.workspace_i8(st["desc"])
            st["out"] = torch.empty(T * K, c["n_out"], dtype=dt, device=DEV)
    else:
        T, d, K, E, F, S = c["T"], c["d"], c["K"], c["E"], c["F"], c["n_shared"]
        st["row_src"], st["off"], st["cap"] = _routes(T, K, E, seed)
        st["xq"], st["xs"] = _rows_i8(T, d, g)
        st["w1"], st["s1"] = _quantised((E + S, F, d), g)
        st["w3"], st["s3"] = _quantised((E + S, F, d), g)
        st["w2"], st["s2"] = _quantised((E + S, d, F), g)
        if own:
            st["desc"] = smoe.make_desc(T, d, E, K, 1, F, S, 1, 1, "bf16")
            st["ws"] = smoe.workspace_i8(st["desc"])
            st["W"] = smoe.i8_weights(*(st[k] for k in ("w1", "s1", "w3", "s3", "w2", "s2")))
            st["out"] = torch.empty(T * K, d, dtype=torch.bfloat16, device=DEV)
            st["out_sh"] = torch.empty(S, T, d, dtype=torch.bfloat16, device=DEV) if S else None
    return st


# ---------------------------------------------------------------- the framework's calls
def _run_own(st):
    c, smoe = st["case"], st["smoe"]
    if c["op"] == "norm":
        smoe.smoe_add_rmsnorm(st["desc"], st["r"], st["gamma"], y=st["y"], r_out=st["r_out"],
                              x_out=st["x_out"], q_out=st["q"], q_scale=st["qs"], eps=EPS)
        if c["q"]:
            torch.mul(st["q"], st["qs"][:, None], out=st["deq"])
        return {"r": st["r_out"], "x": st["x_out"], "q": st["deq"], "scale": st["qs"]}
    if c["op"] == "few":
        smoe.smoe_moe_forward_few(st["desc"], st["x"], st["w_gate"], st["w1"], st["w3"], st["w2"],
                                  st["out"], st["ws"], topk_idx=st["idx"], topk_w=st["w"])
        return {"y": st["out"], "idx": st["idx"], "w": st["w"]}
    if c["op"] == "matmul":
        smoe.smoe_expert_matmul_i8(st["desc"], st["xq"], st["xs"], st["off"], st["wq"], st["ws_"],
                                   st["out"], st["ws"], row_src=st["row_src"])
        return st["out"]
    smoe.smoe_expert_ffn_i8(st["desc"], st["xq"], st["xs"], st["off"], st["W"], st["out"], st["ws"],
                            row_src=st["row_src"], y_shared=st["out_sh"])
    return {"rows": st["out"], "shared": st["out_sh"]}


# ---------------------------------------------------------------- plain forms
def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _plain_norm(st):
    c = st["case"]
    h = st["r"] + st["y"].float() if c["y"] else st["r"]
    n = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * st["gamma"]
    out = {"r": h if c["y"] else None, "x": n.to(TYPES[c["dtype"]]) if c["x"] else None}
    if c["q"]:
        s = n.abs().amax(-1) / 127.0
        q = torch.round(n / s[:, None])
        out |= {"q": (q * s[:, None]).to(torch.bfloat16), "scale": s}
    return out


def _pick(logits, K, H):
    """The K/H largest of each of H groups; the lower index first where logits are equal."""
    T, E = logits.shape
    order = torch.sort(logits.view(T, H, E // H), dim=-1, descending=True, stable=True).indices
    base = torch.arange(H, device=logits.device)[None, :, None] * (E // H)
    return (order[..., :K // H] + base).reshape(T, K)


def _plain_few(st):
    c = st["case"]
    T, E, K, S = c["T"], c["E"], c["K"], c["n_shared"]
    x = st["x"].float()
    logits = st["x"].double() @ st["w_gate"].double().T  # the selection compares them
    idx = _pick(logits, K, c["H"])
    w = torch.softmax(logits, -1).gather(1, idx)
    w = (w / w.sum(-1, keepdim=True) if c["renorm"] else w).float()
    if T * K >= E:  # every expert on every token
        w1, w3, w2 = (st[k].float() for k in ("w1", "w3", "w2"))
        h = _silu(torch.matmul(x, w1.transpose(1, 2))) * torch.matmul(x, w3.transpose(1, 2))
        dense = torch.zeros(T, E + S, device=x.device)
        dense.scatter_(1, idx, w)
        dense[:, E:] = 1.0
        y = torch.bmm(h * dense.T[:, :, None], w2.transpose(1, 2)).sum(0)
    else:
        sh = torch.arange(E, E + S, device=x.device).expand(T, S)
        e, wk = torch.cat([idx, sh], 1), torch.cat([w, torch.ones_like(w[:, :1]).expand(T, S)], 1)
        h = (_silu((st["w1"][e].float() @ x[:, None, :, None]).squeeze(-1))
             * (st["w3"][e].float() @ x[:, None, :, None]).squeeze(-1)) * wk[..., None]
        y = (st["w2"][e].float() @ h[..., None]).squeeze(-1).sum(1)
    return {"y": y.to(TYPES[c["dtype"]]), "idx": idx.to(torch.int32), "w": w}


def _places(st, rows):
    """Each row's expert and its place among that expert's rows."""
    r = torch.arange(rows, device=DEV)
    e = torch.bucketize(r, st["off"][1:].long(), right=True)
    return e, r - st["off"].long()[e]


def _product(rows_q, e, pos, wq, cap):
    """Whole-number sums of each row with its expert's weights (below 2^24: exact in fp32)."""
    x = torch.zeros(wq.shape[0], cap, wq.shape[2], device=DEV)
    x[e, pos] = rows_q
    return torch.bmm(x, wq.float().transpose(1, 2))[e, pos]


def _plain_matmul(st):
    c = st["case"]
    src = st["row_src"].long()
    e, pos = _places(st, c["T"] * c["K"])
    acc = _product(st["xq"][src].float(), e, pos, st["wq"], st["cap"])
    return (acc * st["xs"][src][:, None] * st["ws_"][e]).to(TYPES[c["dtype"]])


def _plain_ffn(st):
    c = st["case"]
    E, S, T, R = c["E"], c["n_shared"], c["T"], c["T"] * c["K"]
    src = st["row_src"].long()
    e, pos = _places(st, R)

    def rows(xr, xs, e, pos, w1, w3, w2, s1, s3, s2, cap):
        g = _product(xr, e, pos, w1, cap) * xs[:, None] * s1[e]
        u = _product(xr, e, pos, w3, cap) * xs[:, None] * s3[e]
        h = _silu(g) * u
        hs = h.abs().amax(-1) / 127.0
        hq = torch.round(h / hs[:, None])
        return (_product(hq, e, pos, w2, cap) * hs[:, None] * s2[e]).to(torch.bfloat16)

    W = [st[k] for k in ("w1", "w3", "w2", "s1", "s3", "s2")]
    out = {"rows": rows(st["xq"][src].float(), st["xs"][src], e, pos, *(w[:E] for w in W), st["cap"]),
           "shared": None}
    if S:
        es = torch.arange(S, device=DEV).repeat_interleave(T)
        ts = torch.arange(T, device=DEV).repeat(S)
        out["shared"] = rows(st["xq"][ts].float(), st["xs"][ts], es, ts, *(w[E:] for w in W),
                             T).view(S, T, c["d"])
    return out


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _plain_norm, "few": _plain_few, "matmul": _plain_matmul,
            "ffn": _plain_ffn}[state["case"]["op"]](state)


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    c, st = case, prepare(case, seed)
    f64 = torch.float64
    if c["op"] == "norm":
        h = st["r"].to(f64) + (st["y"].to(f64) if c["y"] else 0.0)
        n = h / torch.sqrt((h * h).sum(-1, keepdim=True) / c["d"] + EPS) * st["gamma"].to(f64)
        out = {"r": h if c["y"] else None, "x": n}
        if c["q"]:
            s = n.abs().max(dim=-1).values / 127
            out |= {"q": torch.round(n / s[:, None]) * s[:, None], "scale": s}
        return out
    if c["op"] == "few":
        T, E, K, H, S = c["T"], c["E"], c["K"], c["H"], c["n_shared"]
        x = st["x"].to(f64)
        logits = x @ st["w_gate"].to(f64).T
        per = E // H
        idx = torch.stack([torch.argsort(-logits[:, h * per:(h + 1) * per], dim=1, stable=True)
                           [:, :K // H] + h * per for h in range(H)], 1).reshape(T, K)
        z = torch.exp(logits - logits.max(1, keepdim=True).values)
        w = torch.take_along_dim(z, idx, 1) / (torch.take_along_dim(z, idx, 1).sum(1, keepdim=True)
                                               if c["renorm"] else z.sum(1, keepdim=True))
        y = torch.zeros(T, c["d"], dtype=f64, device=DEV)
        for e in range(E + S):
            t, k = torch.nonzero(idx == e, as_tuple=True) if e < E else (torch.arange(T, device=DEV), None)
            if not len(t):
                continue
            g, u = x[t] @ st["w1"][e].to(f64).T, x[t] @ st["w3"][e].to(f64).T
            o = (g * u * torch.sigmoid(g)) @ st["w2"][e].to(f64).T
            y.index_add_(0, t, o if k is None else o * w[t, k][:, None])
        return {"y": y, "idx": idx.to(torch.int32), "w": w}
    off = st["off"].tolist()
    src = st["row_src"].long()
    if c["op"] == "matmul":
        out = torch.zeros(c["T"] * c["K"], c["n_out"], dtype=f64, device=DEV)
        for e in range(c["E"]):
            t = src[off[e]:off[e + 1]]
            out[off[e]:off[e + 1]] = (st["xq"][t].to(f64) @ st["wq"][e].to(f64).T
                                      * st["xs"][t].to(f64)[:, None] * st["ws_"][e].to(f64))
        return out

    def ffn(t, e):
        x, xs = st["xq"][t].to(f64), st["xs"][t].to(f64)[:, None]
        g = x @ st["w1"][e].to(f64).T * xs * st["s1"][e].to(f64)
        u = x @ st["w3"][e].to(f64).T * xs * st["s3"][e].to(f64)
        h = g * u * torch.sigmoid(g)
        hs = h.abs().max(dim=-1, keepdim=True).values / 127
        return torch.round(h / hs) @ st["w2"][e].to(f64).T * hs * st["s2"][e].to(f64)

    rows = torch.zeros(c["T"] * c["K"], c["d"], dtype=f64, device=DEV)
    for e in range(c["E"]):
        if off[e + 1] > off[e]:
            rows[off[e]:off[e + 1]] = ffn(src[off[e]:off[e + 1]], e)
    every = torch.arange(c["T"], device=DEV)
    shared = [ffn(every, c["E"] + j) for j in range(c["n_shared"])]
    return {"rows": rows, "shared": torch.stack(shared) if shared else None}
