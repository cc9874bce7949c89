"""The serving operators on the GPU against plain formulas in 64 bits: the RMS norm with
8-bit rows, the few-token layer, the 8-bit expert products, and a run of them together.

Tolerances count roundings: half a step of the type (bf16 2^-8, fp32 2^-24, relative to the
value), and for a contraction whose operands were rounded, six standard deviations of
independent roundings, sqrt(sum of squared terms) x step / sqrt(3)."""
import math

import pytest
import torch

import routing_token_shuffle_gb300 as smoe

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def i32(*shape):
    return torch.empty(*shape, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ RMS norm
def norm_ref(r, y, gamma, eps):
    h = r.double() + (y.double() if y is not None else 0.0)
    return h, h * gamma.double() / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)


def norm_buffers(T, d, dt, r=True, x=True, q=True):
    return dict(r_out=torch.full((T, d), 7.0, device="cuda") if r else None,
                x_out=torch.full((T, d), 7.0, device="cuda", dtype=DT[dt]) if x else None,
                q_out=torch.full((T, d), 7, device="cuda", dtype=torch.int8) if q else None,
                q_scale=torch.full((T,), 7.0, device="cuda") if q else None)


def norm_desc(T, d, dt):
    return smoe.make_desc(T, d, 1, 1, 1, 8, 0, 1, 1, dt)


# fp32: one thread adds at most 32 squares, then a tree of 5 shuffles and at most 32 warp
# sums: under 70 roundings in the sum, half of that in its root, a few more around it
NORM_F32 = 48 * 2.0 ** -24


def check_norm(n, out, dt):
    tol = NORM_F32 + (HALF["bf16"] if dt == "bf16" else 0.0)
    if out["x_out"] is not None:
        assert ((out["x_out"].double() - n).abs() <= tol * n.abs() + 1e-37).all()
    if out["q_out"] is not None:
        s = out["q_scale"].double()
        ref = n.abs().amax(-1) / 127
        assert ((s - ref).abs() <= NORM_F32 * ref).all()
        err = (out["q_out"].double() * s[:, None] - n).abs()
        assert (err <= s[:, None] * (0.5 + 128 * 2 * NORM_F32)).all()
        top = out["q_out"].abs().amax(-1)
        assert ((top == 127) | (ref == 0)).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 8), (3, 64), (1, 256), (9, 264), (257, 1024), (5, 1032),
                                 (1, 5120), (77, 4096), (33, 8192), (4, 8200), (2, 16384),
                                 (1000, 40), (2049, 2048)])
def test_add_rmsnorm(T, d, dt):
    g = gen(T * 31 + d)
    r, y = randn(g, T, d) * 3, randn(g, T, d).to(DT[dt])
    gamma = 1 + 0.3 * randn(g, d)
    for with_y in (True, False):
        out = norm_buffers(T, d, dt)
        smoe.smoe_add_rmsnorm(norm_desc(T, d, dt), r, gamma, y=y if with_y else None, eps=1e-5, **out)
        h, n = norm_ref(r, y if with_y else None, gamma, 1e-5)
        assert torch.equal(out["r_out"], r + y.float() if with_y else r)
        check_norm(norm_ref(out["r_out"], None, gamma, 1e-5)[1], out, dt)


@pytest.mark.parametrize("r,x,q", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1)])
def test_add_rmsnorm_each_output_alone(r, x, q):
    g = gen(5)
    R, y, gamma = randn(g, 19, 1544), randn(g, 19, 1544).bfloat16(), randn(g, 1544)
    out = norm_buffers(19, 1544, "bf16", r, x, q)
    smoe.smoe_add_rmsnorm(norm_desc(19, 1544, "bf16"), R, gamma, y=y, **out)
    full = norm_buffers(19, 1544, "bf16")
    smoe.smoe_add_rmsnorm(norm_desc(19, 1544, "bf16"), R, gamma, y=y, **full)
    for k, v in out.items():
        assert v is None or torch.equal(v, full[k]), k


def test_add_rmsnorm_in_place():
    """r_out over r and x_out over y."""
    g = gen(6)
    r, y, gamma = randn(g, 65, 2056), randn(g, 65, 2056).bfloat16(), randn(g, 2056)
    a = norm_buffers(65, 2056, "bf16")
    smoe.smoe_add_rmsnorm(norm_desc(65, 2056, "bf16"), r, gamma, y=y, **a)
    smoe.smoe_add_rmsnorm(norm_desc(65, 2056, "bf16"), r, gamma, y=y, r_out=r, x_out=y)
    assert torch.equal(r, a["r_out"]) and torch.equal(y, a["x_out"])


@pytest.mark.parametrize("eps", [0.0, 1e-38, 1e-31, 1e-29])
@pytest.mark.parametrize("d", [128, 1000, 5120, 8200])
def test_add_rmsnorm_tiny_rows(d, eps):
    """Rows whose squares fp32 does not hold, with an eps of zero or as small: the norm all the
    same; a row of zeros gives zeros. Each combination of outputs, and r_out over r."""
    g = gen(16)
    r = randn(g, 7, d)
    r[1] = 0.0
    for i, s in ((2, 1e-15), (3, 1e-20), (4, 1e-30), (5, 3e-41)):
        r[i] *= s
    r[6] *= 1e-30
    r[6, 5] = 1e-19
    gamma = 1 + 0.3 * randn(g, d)
    n = norm_ref(r, None, gamma, eps)[1]
    if eps == 0:
        n[1] = 0.0
    desc = norm_desc(7, d, "f32")
    first = norm_buffers(7, d, "f32")
    smoe.smoe_add_rmsnorm(desc, r, gamma, eps=eps, **first)
    # above eps = 2^-100 h gamma is not scaled: row 5's products are below fp32's normal numbers
    good = [0, 1, 2, 3, 4, 6] + ([5] if eps < 2.0 ** -100 else [])
    check_norm(n[good], {k: v[good] for k, v in first.items()}, "f32")
    assert first["q_scale"][1] == 0 and (first["q_out"][1] == 0).all() and (first["x_out"][1] == 0).all()
    out = norm_buffers(7, d, "f32", r=False)
    smoe.smoe_add_rmsnorm(desc, r, gamma, eps=eps, **out)
    y = r * 0.5  # r / 2 + r / 2 is r, but for the smallest values' last bit
    keep = [0, 1, 2, 3, 4, 6]
    summed = norm_buffers(7, d, "f32", r=False)
    smoe.smoe_add_rmsnorm(desc, r - y, gamma, y=y, eps=eps, **summed)
    for k in ("x_out", "q_out", "q_scale"):
        assert torch.equal(out[k], first[k]) and torch.equal(summed[k][keep], first[k][keep]), k
    x = torch.empty_like(r)
    r2 = r.clone()
    smoe.smoe_add_rmsnorm(desc, r2, gamma, r_out=r2, x_out=x, eps=eps)
    assert torch.equal(r2, r) and torch.equal(x, first["x_out"])


@pytest.mark.parametrize("d", [128, 5120])
def test_add_rmsnorm_overflowing_row(d):
    """A finite row whose squares overflow: n is 0 and the scale says so; its neighbour stays."""
    g = gen(8)
    r = randn(g, 2, d)
    r[0] = 1e30
    gamma = torch.ones(d, device="cuda")
    out = norm_buffers(2, d, "f32")
    smoe.smoe_add_rmsnorm(norm_desc(2, d, "f32"), r, gamma, eps=1e-6, **out)
    assert (out["x_out"][0] == 0).all() and out["q_scale"][0].isnan() and (out["q_out"][0] == 0).all()
    check_norm(norm_ref(r, None, gamma, 1e-6)[1][1:], {k: v[1:] for k, v in out.items()}, "f32")


@pytest.mark.parametrize("d", [128, 5120])
def test_add_rmsnorm_odd_rows(d):
    """Zero rows, tiny rows, rows with an infinity or a NaN; the rows beside them."""
    g = gen(7)
    r = randn(g, 8, d)
    r[1] = 0.0
    r[2] *= 1e-30
    r[3, 5] = math.inf
    r[4, d - 1] = math.nan
    r[5] *= 1e15
    r[6] = 0.0
    r[6, 3] = 1.0
    gamma = torch.ones(d, device="cuda")
    out = norm_buffers(8, d, "f32")
    smoe.smoe_add_rmsnorm(norm_desc(8, d, "f32"), r, gamma, eps=0.0 if d == 128 else 1e-6, **out)
    good = [0, 5, 6, 7]
    n = norm_ref(r, None, gamma, 0.0 if d == 128 else 1e-6)[1]
    check_norm(n[good], {k: v[good] for k, v in out.items()}, "f32")
    s, q = out["q_scale"], out["q_out"]
    assert s[3].isnan() and s[4].isnan() and (q[3:5] == 0).all()
    if d == 5120:  # eps > 0: a zero row is zeros
        assert s[1] == 0 and (q[1] == 0).all() and (out["x_out"][1] == 0).all()
        check_norm(n[2:3], {k: v[2:3] for k, v in out.items()}, "f32")


# ------------------------------------------------------------------ few-token layer
class Few:
    def __init__(self, T, d, E, K, H, F, S, dt, renorm=0, seed=0):
        g = gen(seed + T + d + E + F)
        self.T, self.d, self.E, self.K, self.H, self.F, self.S = T, d, E, K, H, F, S
        self.dt, self.renorm = dt, renorm
        t, n = DT[dt], E + S
        self.x = randn(g, T, d).to(t)
        self.w_gate = (randn(g, E, d) / math.sqrt(d)).to(t)
        self.w1 = (randn(g, n, F, d) / math.sqrt(d)).to(t)
        self.w3 = (randn(g, n, F, d) / math.sqrt(d)).to(t)
        self.w2 = (randn(g, n, d, F) / math.sqrt(F)).to(t)
        self.desc = smoe.make_desc(T, d, E, K, H, F, S, 1, 1, dt, renorm)
        self.ws = smoe.workspace_few(self.desc)
        self.y = torch.full((T, d), 7.0, dtype=t, device="cuda")
        self.logits = torch.empty(T, E, device="cuda")
        self.idx, self.w = i32(T, K), torch.empty(T, K, device="cuda")

    def run(self, **kw):
        smoe.smoe_moe_forward_few(self.desc, self.x, self.w_gate, self.w1, self.w3, self.w2, self.y,
                                  self.ws, logits=self.logits, topk_idx=self.idx, topk_w=self.w, **kw)

    def routes(self, logits):
        T, E, K, H = self.T, self.E, self.K, self.H
        o = torch.sort(logits.view(T, H, E // H), dim=-1, descending=True, stable=True).indices
        idx = (o[..., :K // H] + torch.arange(H, device="cuda")[None, :, None] * (E // H)).reshape(T, K)
        w = torch.softmax(logits.double(), -1).gather(1, idx)
        return idx, w / w.sum(-1, keepdim=True) if self.renorm else w

    def reference(self, idx, w):
        """(y, the square sum of the down product's terms) in float64."""
        x = self.x.double()
        y, sq = torch.zeros(self.T, self.d, dtype=torch.float64, device="cuda"), 0.0
        sq = torch.zeros_like(y)
        for e in range(self.E + self.S):
            if e < self.E:
                t, k = torch.nonzero(idx == e, as_tuple=True)
                wk = w[t, k].double()[:, None]
            else:
                t, wk = torch.arange(self.T, device="cuda"), 1.0
            if not len(t):
                continue
            g, u = x[t] @ self.w1[e].double().T, x[t] @ self.w3[e].double().T
            h = g * torch.sigmoid(g) * u * wk
            w2 = self.w2[e].double()
            y.index_add_(0, t, h @ w2.T)
            sq.index_add_(0, t, h.square() @ w2.square().T)
        return y, sq

    def check(self):
        smoe.smoe_get_status(self.ws)
        ref_l = self.x.double() @ self.w_gate.double().T
        # an fp32 sum of d products, added in blocks: sqrt(d) roundings of the typical sum
        assert (self.logits.double() - ref_l).abs().max() <= 8 * math.sqrt(self.d) * 2.0 ** -24 * ref_l.abs().max()
        idx, w = self.routes(self.logits)
        assert torch.equal(self.idx.long(), idx)
        assert ((self.w.double() - w).abs() <= 2e-6 * w + 1e-37).all()
        y, sq = self.reference(idx, self.w)
        err = (self.y.double() - y).abs()
        rms = sq.sqrt()
        if self.dt == "bf16":
            # y rounded once; h as two bf16 values (2^-8 of 2^-8); the fp32 sums are below both
            tol = HALF["bf16"] * y.abs() + (6 / math.sqrt(3) * HALF["bf16"] ** 2 + 1e-4) * rms
        else:
            # three chained fp32 contractions of d, d and F (K F) terms: each
            # sqrt(n) 2^-24 / sqrt(3) of the typical sum, six standard deviations
            n = math.sqrt(2 * self.d + self.F * (self.K + self.S))
            tol = 6 / math.sqrt(3) * n * 2.0 ** -24 * rms + 2 * HALF["f32"] * y.abs()
        assert (err <= tol + 1e-30).all(), (err / tol).max()


FEW = [
    # T, d, E, K, H, F, S, renorm
    (1, 2048, 128, 8, 8, 768, 0, 1), (1, 256, 8, 2, 1, 512, 0, 0), (2, 1024, 16, 2, 1, 1000, 1, 0),
    (5, 5120, 40, 6, 1, 1536, 2, 0), (16, 512, 32, 4, 2, 264, 0, 1), (17, 520, 32, 4, 1, 136, 1, 1),
    (32, 768, 8, 8, 1, 200, 0, 0), (33, 1000, 24, 3, 3, 1416, 1, 0), (64, 1024, 160, 6, 1, 384, 2, 1),
    (64, 136, 4, 1, 1, 72, 0, 0), (3, 4096, 8, 2, 1, 1792, 0, 0), (1, 8, 1, 1, 1, 8, 0, 0),
    (7, 8, 512, 32, 1, 8, 8, 1), (64, 64, 512, 32, 32, 64, 0, 0), (1, 128, 4, 1, 1, 128, 0, 0),
    (64, 72, 2, 1, 1, 4096, 0, 0), (13, 4096, 33, 3, 1, 24, 0, 0), (8, 768, 20, 2, 1, 448, 1, 0),
    (9, 768, 20, 2, 1, 448, 1, 0), (10, 264, 300, 5, 1, 64, 0, 1), (11, 264, 130, 13, 13, 72, 0, 0),
]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,E,K,H,F,S,renorm", FEW)
def test_moe_few(T, d, E, K, H, F, S, renorm, dt):
    c = Few(T, d, E, K, H, F, S, dt, renorm)
    c.run()
    c.check()
    first = c.y.clone()
    for _ in range(3):  # the same bits again, the workspace as the last call left it
        c.y.fill_(3.0)
        c.run()
        assert torch.equal(c.y, first)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_moe_few_all_tokens_on_the_same_experts(dt):
    c = Few(48, 512, 64, 3, 1, 320, 1, dt)
    c.x[:] = c.x[0]
    c.run()
    c.check()
    assert (c.idx == c.idx[0]).all() and (c.y == c.y[0]).all()


def test_moe_few_ties_take_the_lower_index():
    c = Few(9, 64, 96, 6, 2, 64, 0, "f32")
    c.w_gate[:] = 0.0  # every logit is zero
    c.run()
    want = torch.tensor([0, 1, 2, 48, 49, 50], device="cuda", dtype=torch.int32)
    assert (c.idx == want).all()
    assert torch.allclose(c.w, torch.full_like(c.w, 1 / 96), rtol=1e-6)
    c.check()


def test_moe_few_over_its_input():
    c = Few(6, 640, 12, 2, 1, 192, 1, "bf16")
    c.run()
    smoe.smoe_moe_forward_few(c.desc, c.x, c.w_gate, c.w1, c.w3, c.w2, c.x, c.ws)
    assert torch.equal(c.x, c.y)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 30, 64])
def test_moe_few_over_its_input_again(T, dt):
    """The layer applied to its own output, call after call, as with separate buffers."""
    c = Few(T, 640, 12, 2, 1, 192, 1, dt)
    x = c.x.clone()
    for _ in range(8):
        c.run()
        smoe.smoe_moe_forward_few(c.desc, x, c.w_gate, c.w1, c.w3, c.w2, x, c.ws)
        assert torch.equal(x, c.y)
        c.x.copy_(c.y)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [5, 20])
def test_moe_few_weights_that_are_not_finite(T, dt):
    """A weight of W2 that is not finite: its expert's tokens get it at its channel; the other
    channels keep their bits, and an expert that no token is routed to changes nothing."""
    c = Few(T, 256, 64, 2, 1, 96, 0, dt)
    c.run()
    clean = c.y.clone()
    touched = sorted(set(c.idx.flatten().tolist()))
    e, other = touched[1], next(i for i in range(64) if i not in touched)
    c.w2[other] = math.nan
    c.run()
    assert torch.equal(c.y, clean)
    c.w2[e, 77, 5] = math.inf
    c.run()
    keep = [i for i in range(256) if i != 77]
    assert torch.equal(c.y[:, keep], clean[:, keep])
    routed = (c.idx == e).any(1)
    assert not c.y[routed, 77].isfinite().any()
    smoe.smoe_get_status(c.ws)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 16, 32, 64])
def test_moe_few_most_experts(T, dt):
    """512 experts of which each token takes 32, 8 shared ones: the largest tables in shared memory."""
    c = Few(T, 72, 512, 32, 4, 40, 8, dt, renorm=1)
    c.run()
    c.check()


def test_moe_few_keeps_other_tokens_out():
    """A token whose states overflow its experts does not reach the other tokens."""
    c = Few(4, 256, 8, 2, 1, 128, 1, "bf16")
    c.run()
    clean = c.y.clone()
    c.x[2] = 1e30
    c.run()
    keep = [0, 1, 3]
    assert torch.equal(c.y[keep], clean[keep])


def test_moe_few_matches_the_layer():
    """The staged layer on the same inputs, within its own roundings (h, expert rows, y)."""
    c = Few(24, 1024, 32, 4, 1, 512, 1, "bf16")
    c.run()
    ws = smoe.workspace(c.desc)
    y = torch.empty_like(c.y)
    smoe.smoe_moe_forward_routed(c.desc, c.x, c.idx, c.w, c.w1, c.w3, c.w2, y, ws)
    smoe.smoe_get_status(ws)
    _, sq = c.reference(c.idx.long(), c.w)
    tol = 4 * HALF["bf16"] * c.y.double().abs() + 16 * HALF["bf16"] * sq.sqrt()
    assert ((y.double() - c.y.double()).abs() <= tol).all()


def test_moe_few_graphs_share_a_workspace_and_streams():
    """Two captured graphs on one workspace, replayed in turn with new inputs, and eager calls
    on another stream between them."""
    a = Few(5, 512, 16, 2, 1, 256, 1, "bf16", seed=1)
    b = Few(5, 512, 16, 2, 1, 256, 1, "bf16", seed=2)
    b.ws = a.ws
    side = torch.cuda.Stream()
    graphs = []
    for c in (a, b):
        c.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    for i in range(3):
        for c, g in zip((a, b), graphs):
            c.x.copy_(torch.randn(5, 512, device="cuda"))
            c.y.fill_(9.0)
            g.replay()
            torch.cuda.synchronize()
            c.check()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            a.y.fill_(9.0)
            a.run()
        side.synchronize()
        a.check()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_moe_few_reads_nothing_of_an_old_workspace(dt):
    """Only a workspace's first 256 bytes have to be zero; one buffer serves several shapes."""
    big = Few(40, 640, 48, 4, 1, 320, 1, dt)
    ws = torch.full((2 * big.ws.numel(),), 0xFF, dtype=torch.uint8, device="cuda")
    ws[:256] = 0
    small = Few(2, 320, 8, 2, 2, 96, 0, dt)
    for c in (big, small, big):
        c.ws = ws
        c.run()
        c.check()
        assert (ws[:256] == 0).all()  # as it was, for the next call


# shapes whose shared memory would fit an odd number of stages
@pytest.mark.parametrize("T,d,E,K,F", [(64, 1000, 24, 3, 712), (40, 520, 8, 2, 264), (24, 1000, 8, 2, 712),
                                       (32, 264, 24, 3, 136), (13, 512, 160, 6, 264), (7, 256, 128, 8, 136)])
def test_moe_few_fp32_repeats_its_bits(T, d, E, K, F):
    """Two inputs in turn, a few hundred calls: the first call's bits every time."""
    c = Few(T, d, E, K, 1, F, 1, "f32")
    xs, want = [c.x, c.x.flip(1).contiguous() * 2], []
    for c.x in xs:
        c.run()
        c.check()
        want.append(c.y.clone())
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(400):
        c.x = xs[i & 1]
        c.run()
        wrong += (c.y != want[i & 1]).sum()
    assert wrong.item() == 0


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,counter", [(4, 0), (4, 1), (24, 0), (24, 1), (24, 2)])
def test_moe_few_a_wait_that_runs_out(T, counter, dt):
    """A counter of the kernel's (first barrier, second barrier, selected tokens) that starts one
    short: every wait for it runs into its limit, the status says so, and the workspace serves
    the next call as before."""
    c = Few(T, 512, 16, 2, 1, 320, 1, dt)
    c.run()
    c.check()
    want = c.y.clone()
    words = c.ws[:256].view(torch.int32)
    words[32 + counter] = -1
    c.run()
    with pytest.raises(smoe.SmoeError) as e:
        smoe.smoe_get_status(c.ws)
    assert e.value.code == -7
    assert (words == 0).all()
    for _ in range(3):
        c.y.fill_(3.0)
        c.run()
        smoe.smoe_get_status(c.ws)
        assert torch.equal(c.y, want)


def test_moe_few_two_streams_at_once():
    """Two calls with their own workspaces on two streams."""
    cs = [Few(3 + i, 768, 16, 2, 1, 384, i, "bf16", seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(cs, streams):
            c.run(stream=s)
    torch.cuda.synchronize()
    for c in cs:
        c.check()


# ------------------------------------------------------------------ 8-bit products
def rows_of(T, K, E, seed, empty=()):
    """(row_src, expert_off) of T tokens with K picks each; the experts in `empty` get none."""
    g = torch.Generator().manual_seed(seed)
    p = torch.rand(E, generator=g) + 0.1
    for e in empty:
        p[e] = 0.0
    e = torch.multinomial(p, T * K, replacement=True, generator=g)
    order = torch.argsort(e, stable=True)
    off = torch.zeros(E + 1, dtype=torch.int64)
    off[1:] = torch.cumsum(torch.bincount(e, minlength=E), 0)
    return (order // K).int().cuda(), off.int().cuda()


def int8(g, *shape, lo=-127):
    return torch.randint(lo, 128, shape, generator=g, device="cuda").to(torch.int8)


def matmul_ref(xq, xs, src, off, wq, sw):
    """(out in float64, its integer sums)."""
    off = off.tolist()
    out = torch.zeros(len(src), wq.shape[1], dtype=torch.float64, device="cuda")
    acc = torch.zeros_like(out)
    for e in range(wq.shape[0]):
        t = src[off[e]:off[e + 1]].long()
        a = xq[t].double() @ wq[e].double().T
        acc[off[e]:off[e + 1]] = a
        out[off[e]:off[e + 1]] = a * xs[t].double()[:, None] * sw[e].double()
    return out, acc


MM = [
    # T, K, E, n_in, n_out
    (1, 1, 1, 16, 8), (1, 6, 40, 5120, 1536), (2, 2, 8, 64, 8), (3, 1, 2, 48, 72),
    (64, 6, 160, 1024, 264), (100, 8, 16, 2048, 768), (257, 2, 5, 272, 136), (7, 2, 3, 4096, 1032),
    (1000, 4, 8, 512, 640), (2000, 2, 4, 128, 256), (130, 1, 1, 1040, 3000), (513, 3, 31, 96, 200),
    (39, 1, 1, 80, 24), (40, 1, 1, 80, 24), (193, 1, 1, 208, 520), (385, 1, 1, 64, 8),
    (900, 1, 2, 64, 1544),
]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,E,n_in,n_out", MM)
def test_expert_matmul_i8(T, K, E, n_in, n_out, dt):
    g = gen(T + n_in)
    src, off = rows_of(T, K, E, T + E, empty=(1,) if E > 4 else ())
    xq, wq = int8(g, T, n_in), int8(g, E, n_out, n_in, lo=-128)
    xs, sw = torch.rand(T, generator=g, device="cuda") + 0.01, torch.rand(E, n_out, generator=g, device="cuda")
    desc = smoe.make_desc(T, n_in, E, min(K, E), 1, max(8, n_out), 0, 1, 1, dt)
    ref, acc = matmul_ref(xq, xs, src, off, wq, sw)
    assert acc.abs().max() < 2 ** 24
    tol = (2 * HALF["f32"] + (HALF["bf16"] if dt == "bf16" else 0.0)) * 1.01 * ref.abs()
    for gathered in (True, False):
        ws = smoe.workspace_i8(desc)
        out = torch.full((T * K, n_out), 7.0, dtype=DT[dt], device="cuda")
        if gathered:
            smoe.smoe_expert_matmul_i8(desc, xq, xs, off, wq, sw, out, ws, row_src=src)
        else:
            smoe.smoe_expert_matmul_i8(desc, xq[src.long()], xs[src.long()], off, wq, sw, out, ws)
        smoe.smoe_get_status(ws)
        assert ((out.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("T,n_out", [(20, 40), (90, 40), (90, 1552)])
@pytest.mark.parametrize("n_in", [1024, 5120])
def test_expert_matmul_i8_largest_values(n_in, T, n_out):
    """Every product 127 x 127 (exact to n_in = 1024; beyond 2^24 fp32 roundings of the sum)."""
    E = 2
    xq = torch.full((T, n_in), 127, dtype=torch.int8, device="cuda")
    xq[1::2] = -127
    wq = torch.full((E, n_out, n_in), 127, dtype=torch.int8, device="cuda")
    wq[:, 3] = -128
    src, off = rows_of(T, 1, E, 3)
    xs, sw = torch.ones(T, device="cuda"), torch.ones(E, n_out, device="cuda")
    desc = smoe.make_desc(T, n_in, E, 1, 1, 64, 0, 1, 1, "f32")
    ws, out = smoe.workspace_i8(desc), torch.empty(T, n_out, device="cuda")
    smoe.smoe_expert_matmul_i8(desc, xq, xs, off, wq, sw, out, ws, row_src=src)
    ref, acc = matmul_ref(xq, xs, src, off, wq, sw)
    # past 2^24 each of the n_in / 16 additions may lose one unit in the last place
    tol = 0.0 if n_in <= 1024 else n_in / 16 * 2.0 ** -23
    assert ((out.double() - ref).abs() <= tol * ref.abs()).all()


def test_expert_matmul_i8_leaves_other_rows():
    """Segments that end before T K: the rows behind them stay as they were; empty experts at
    both ends."""
    g = gen(1)
    T, K, E, n_in, n_out = 40, 3, 6, 160, 88
    xq, wq = int8(g, T, n_in), int8(g, E, n_out, n_in)
    src = torch.randint(0, T, (T * K,), generator=g, device="cuda", dtype=torch.int32)
    off = torch.tensor([0, 0, 17, 17, 80, 90, 90], dtype=torch.int32, device="cuda")
    xs, sw = torch.rand(T, generator=g, device="cuda"), torch.rand(E, n_out, generator=g, device="cuda")
    desc = smoe.make_desc(T, 160, E, K, 1, 88, 0, 1, 1, "f32")
    ws = smoe.workspace_i8(desc)
    out = torch.full((T * K, n_out), 7.0, device="cuda")
    smoe.smoe_expert_matmul_i8(desc, xq, xs, off, wq, sw, out, ws, row_src=src)
    smoe.smoe_get_status(ws)
    assert (out[90:] == 7.0).all()
    ref, _ = matmul_ref(xq, xs, src, off, wq, sw)
    assert ((out[:90].double() - ref[:90]).abs() <= 2.1 * HALF["f32"] * ref[:90].abs()).all()


@pytest.mark.parametrize("T,n_out", [(16, 264), (64, 264), (64, 1600)])
def test_expert_matmul_i8_padded_batch(T, n_out):
    """Rows outside the segments may name no token: they are neither read nor written."""
    g = gen(9)
    K, E, n_in = 2, 3, 192
    xq, wq = int8(g, T, n_in), int8(g, E, n_out, n_in)
    src, off = rows_of(T // 2, K, E, 4)
    lead = 5  # rows in front of the first segment
    src = torch.cat([torch.full((lead,), T, dtype=torch.int32, device="cuda"), src,
                     torch.full((T * K - len(src) - lead,), -1, dtype=torch.int32, device="cuda")])
    off = off + lead
    xs, sw = torch.rand(T, generator=g, device="cuda"), torch.rand(E, n_out, generator=g, device="cuda")
    desc = smoe.make_desc(T, n_in, E, K, 1, n_out, 0, 1, 1, "f32")
    ws = smoe.workspace_i8(desc)
    ws[256:] = 0xFF
    out = torch.full((T * K, n_out), 7.0, device="cuda")
    smoe.smoe_expert_matmul_i8(desc, xq, xs, off, wq, sw, out, ws, row_src=src)
    smoe.smoe_get_status(ws)
    n = int(off[-1])
    ref, _ = matmul_ref(xq, xs, src, off, wq, sw)
    assert ((out[lead:n].double() - ref[lead:n]).abs() <= 2.1 * HALF["f32"] * ref[lead:n].abs()).all()
    assert (out[n:] == 7.0).all() and (out[:lead] == 7.0).all()


@pytest.mark.parametrize("T,n_out", [(12, 136), (50, 136), (50, 1608)])
def test_expert_matmul_i8_scales_that_are_not_finite(T, n_out):
    """A NaN channel scale gives NaN in that channel of that expert, a NaN row scale in that
    token's rows, nowhere else."""
    g = gen(10)
    K, E, n_in = 2, 2, 128
    xq, wq = int8(g, T, n_in), int8(g, E, n_out, n_in)
    src, off = rows_of(T, K, E, 5)
    xs, sw = torch.rand(T, generator=g, device="cuda"), torch.rand(E, n_out, generator=g, device="cuda")
    xs[11], sw[1, 77] = math.nan, math.nan
    desc = smoe.make_desc(T, n_in, E, K, 1, n_out, 0, 1, 1, "bf16")
    ws, out = smoe.workspace_i8(desc), torch.empty(T * K, n_out, dtype=torch.bfloat16, device="cuda")
    smoe.smoe_expert_matmul_i8(desc, xq, xs, off, wq, sw, out, ws, row_src=src)
    want = torch.zeros(T * K, n_out, dtype=torch.bool, device="cuda")
    want[src == 11] = True
    want[int(off[1]):, 77] = True
    assert torch.equal(out.isnan(), want)


@pytest.mark.parametrize("T,n_out", [(6000, 1552), (2200, 1552)])
def test_expert_matmul_i8_queued_in_place(T, n_out):
    """Many calls queued one behind the other whose rows a kernel puts in place while the pairs of
    the product behind it start (192 and 160 row tiles)."""
    g = gen(14)
    K, E, n_in = 8, 64, 1024
    xq, wq = int8(g, T, n_in), int8(g, E, n_out, n_in)
    src, off = rows_of(T, K, E, 3)
    xs, sw = torch.rand(T, generator=g, device="cuda"), torch.rand(E, n_out, generator=g, device="cuda")
    desc = smoe.make_desc(T, n_in, E, K, 1, n_out, 0, 1, 1, "f32")
    ws, out = smoe.workspace_i8(desc), torch.empty(T * K, n_out, device="cuda")
    for _ in range(4):
        for _ in range(500):
            smoe.smoe_expert_matmul_i8(desc, xq, xs, off, wq, sw, out, ws, row_src=src)
        smoe.smoe_get_status(ws)
    ref, acc = matmul_ref(xq, xs, src, off, wq, sw)
    assert acc.abs().max() < 2 ** 24
    assert ((out.double() - ref).abs() <= 2.1 * HALF["f32"] * ref.abs()).all()


@pytest.mark.parametrize("T,K,E,n_in,n_out", [(4000, 4, 8, 1024, 256), (700, 6, 20, 4096, 264),
                                              (97, 2, 3, 272, 1536)])
def test_expert_matmul_i8_gathered_rows_on_one_workspace(T, K, E, n_in, n_out):
    """Calls with other rows and scales queued one behind the other on one workspace, the rows
    gathered by pairs of CTAs: each call's output is what the call alone gives."""
    g = gen(13)
    wq, sw = int8(g, E, n_out, n_in), torch.rand(E, n_out, generator=g, device="cuda")
    desc = smoe.make_desc(T, n_in, E, K, 1, n_out, 0, 1, 1, "f32")
    calls = []
    for i in range(3):
        src, off = rows_of(T, K, E, i)
        xs = torch.rand(T, generator=g, device="cuda") * 10.0 ** i
        calls.append((int8(g, T, n_in), xs, src, off, torch.empty(T * K, n_out, device="cuda")))
    ws = smoe.workspace_i8(desc)
    for _ in range(60):
        for xq, xs, src, off, out in calls:
            out.fill_(7.0)
        for xq, xs, src, off, out in calls:
            smoe.smoe_expert_matmul_i8(desc, xq, xs, off, wq, sw, out, ws, row_src=src)
    smoe.smoe_get_status(ws)
    for xq, xs, src, off, out in calls:
        ref, acc = matmul_ref(xq, xs, src, off, wq, sw)
        assert acc.abs().max() < 2 ** 24
        assert ((out.double() - ref).abs() <= 2.1 * HALF["f32"] * ref.abs()).all()


def test_expert_matmul_i8_two_streams_at_once():
    g = gen(11)
    cs = []
    for i in range(2):
        T, K, E, n_in, n_out = 300 + 7 * i, 2, 4, 512, 264
        xq, wq = int8(g, T, n_in), int8(g, E, n_out, n_in)
        src, off = rows_of(T, K, E, i)
        xs, sw = torch.rand(T, generator=g, device="cuda"), torch.rand(E, n_out, generator=g, device="cuda")
        desc = smoe.make_desc(T, n_in, E, K, 1, n_out, 0, 1, 1, "f32")
        cs.append((desc, xq, xs, src, off, wq, sw, smoe.workspace_i8(desc), torch.empty(T * K, n_out, device="cuda"),
                   torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for desc, xq, xs, src, off, wq, sw, ws, out, stream in cs:
            smoe.smoe_expert_matmul_i8(desc, xq, xs, off, wq, sw, out, ws, row_src=src, stream=stream)
    torch.cuda.synchronize()
    for desc, xq, xs, src, off, wq, sw, ws, out, _ in cs:
        ref, _ = matmul_ref(xq, xs, src, off, wq, sw)
        assert ((out.double() - ref).abs() <= 2.1 * HALF["f32"] * ref.abs()).all()


# tokens and channels that take the narrow tiles, the wide ones that gather their rows, and
# the wide ones whose rows are put in place (160 and 192 rows high)
TILES = [(30, 32), (200, 32), (200, 1544), (600, 1544), (900, 1544)]


@pytest.mark.parametrize("T,n_out", TILES)
def test_expert_matmul_i8_reports_bad_rows(T, n_out):
    """A row_src entry out of range: a zero row and SMOE_ERR_DATA; a bad expert_off: nothing."""
    g = gen(2)
    E, n_in = 2, 64
    xq, wq = int8(g, T, n_in), int8(g, E, n_out, n_in)
    src, off = rows_of(T, 1, E, 1)
    src[4], src[9] = T, -1
    xs, sw = torch.ones(T, device="cuda"), torch.ones(E, n_out, device="cuda")
    desc = smoe.make_desc(T, n_in, E, 1, 1, n_out, 0, 1, 1, "f32")
    ws, out = smoe.workspace_i8(desc), torch.full((T, n_out), 7.0, device="cuda")
    smoe.smoe_expert_matmul_i8(desc, xq, xs, off, wq, sw, out, ws, row_src=src)
    with pytest.raises(smoe.SmoeError) as e:
        smoe.smoe_get_status(ws)
    assert e.value.code == -6
    assert (out[4] == 0).all() and (out[9] == 0).all() and (out[5] != 0).any()
    out.fill_(7.0)
    bad = off.clone()
    bad[1] = T + 5
    smoe.smoe_expert_matmul_i8(desc, xq, xs, bad, wq, sw, out, ws, row_src=rows_of(T, 1, E, 1)[0])
    with pytest.raises(smoe.SmoeError):
        smoe.smoe_get_status(ws)
    assert (out == 7.0).all()


# ------------------------------------------------------------------ 8-bit FFN
class Ffn8:
    def __init__(self, T, d, E, K, F, S, dt, seed=0, empty=()):
        g = gen(seed + T + d)
        self.T, self.E, self.K, self.S, self.dt, self.F, self.d = T, E, K, S, dt, F, d
        n = E + S
        self.src, self.off = rows_of(T, K, E, T + E + seed, empty)
        x = randn(g, T, d)
        self.xs = (x.abs().amax(-1) / 127).contiguous()
        self.xq = torch.round(x / self.xs[:, None]).to(torch.int8)
        self.q = {}
        for name, shape in (("1", (n, F, d)), ("3", (n, F, d)), ("2", (n, d, F))):
            w = randn(g, *shape) / math.sqrt(shape[-1])
            s = (w.abs().amax(-1) / 127).contiguous()
            self.q["w" + name], self.q["s" + name] = torch.round(w / s[..., None]).to(torch.int8), s
        self.W = smoe.i8_weights(*(self.q[k] for k in ("w1", "s1", "w3", "s3", "w2", "s2")))
        self.desc = smoe.make_desc(T, d, E, K, 1, F, S, 1, 1, dt)
        self.ws = smoe.workspace_i8(self.desc)
        self.y = torch.full((T * K, d), 7.0, dtype=DT[dt], device="cuda")
        self.ysh = torch.full((S, T, d), 7.0, dtype=DT[dt], device="cuda") if S else None

    def run(self, **kw):
        smoe.smoe_expert_ffn_i8(self.desc, self.xq, self.xs, self.off, self.W, self.y, self.ws,
                                row_src=self.src, y_shared=self.ysh, **kw)

    def expert(self, t, e):
        """(out, how far it may be off) in float64. The hidden values are computed in fp32: one
        whose place between two integers is within 1e-3 of the middle may go either way."""
        q = {k: v[e].double() for k, v in self.q.items()}
        x, xs = self.xq[t].double(), self.xs[t].double()[:, None]
        g, u = x @ q["w1"].T * xs * q["s1"], x @ q["w3"].T * xs * q["s3"]
        h = g * torch.sigmoid(g) * u
        hs = h.abs().amax(-1, keepdim=True) / 127
        v = h / hs
        hq = torch.round(v)
        edge = ((v - hq).abs() > 0.5 - 1e-3).double()
        out = hq @ q["w2"].T * hs * q["s2"]
        half = HALF["f32"] * 16 + (HALF["bf16"] if self.dt == "bf16" else 0.0)
        return out, half * out.abs() + 1.01 * (edge @ q["w2"].abs().T) * hs * q["s2"] + 1e-30

    def check(self):
        smoe.smoe_get_status(self.ws)
        off = self.off.tolist()
        for e in range(self.E):
            if off[e + 1] > off[e]:
                out, tol = self.expert(self.src[off[e]:off[e + 1]].long(), e)
                assert ((self.y[off[e]:off[e + 1]].double() - out).abs() <= tol).all(), e
        for j in range(self.S):
            out, tol = self.expert(torch.arange(self.T, device="cuda"), self.E + j)
            assert ((self.ysh[j].double() - out).abs() <= tol).all(), j


FFN = [
    # T, d, E, K, F, S
    (1, 16, 1, 1, 16, 0), (1, 512, 8, 2, 768, 0), (5, 1024, 40, 6, 512, 2), (64, 640, 160, 6, 96, 2),
    (33, 272, 4, 3, 144, 1), (500, 256, 8, 2, 1040, 0), (300, 2048, 16, 8, 768, 0),
    (1000, 512, 4, 2, 256, 1), (193, 64, 1, 1, 48, 1), (65, 32, 2, 1, 16, 8), (150, 96, 3, 2, 784, 2),
    (700, 128, 2, 1, 800, 0), (900, 128, 2, 1, 800, 1),
]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,E,K,F,S", FFN)
def test_expert_ffn_i8(T, d, E, K, F, S, dt):
    c = Ffn8(T, d, E, K, F, S, dt, empty=(0, 3) if E > 4 else ())
    c.run()
    c.check()
    first = c.y.clone()
    c.y.fill_(3.0)
    c.run()
    assert torch.equal(first, c.y)


# tokens (of 2 experts each, of 3) and hidden channels that take the narrow tiles, the wide ones
# that gather their rows, and the wide ones whose rows are put in place (160 and 192 rows high)
@pytest.mark.parametrize("S", [0, 1])
@pytest.mark.parametrize("T,F", [(20, 64), (300, 64), (300, 800), (1000, 800)])
def test_expert_ffn_i8_padded_batch(T, F, S):
    """Rows in front of the first segment and behind the last one name no token: they are neither
    read nor written, whatever an old workspace holds."""
    c = Ffn8(T, 128, 3, 2, F, S, "f32")
    n, lead = T * 2, 7
    e = torch.sort(torch.randint(0, 3, (n - lead - 11,), generator=torch.Generator().manual_seed(T))).values
    src = torch.randint(0, T, (len(e),), generator=torch.Generator().manual_seed(T + 1)).int().cuda()
    c.src = torch.cat([torch.full((lead,), T, dtype=torch.int32, device="cuda"), src,
                       torch.full((11,), -1, dtype=torch.int32, device="cuda")])
    off = torch.zeros(4, dtype=torch.int64)
    off[1:] = torch.cumsum(torch.bincount(e, minlength=3), 0)
    c.off = (off + lead).int().cuda()
    c.ws[256:] = 0xFF
    for _ in range(2):  # the second call on what the first one left
        c.y.fill_(7.0)
        c.run()
        c.check()
        assert (c.y[:lead] == 7.0).all() and (c.y[n - 11:] == 7.0).all()


@pytest.mark.parametrize("T,K", [(9, 4), (300, 32), (700, 32), (6400, 32)])
def test_expert_ffn_i8_most_experts(T, K):
    """512 experts and 8 shared ones, in each tile form."""
    c = Ffn8(T, 32, 512, K, 16, 8, "f32", empty=(0, 200, 511))
    c.run()
    smoe.smoe_get_status(c.ws)
    off = c.off.tolist()
    for e in range(0, 512, 37):
        if off[e + 1] > off[e]:
            out, tol = c.expert(c.src[off[e]:off[e + 1]].long(), e)
            assert ((c.y[off[e]:off[e + 1]].double() - out).abs() <= tol).all(), e
    assert not (c.y == 7.0).all(1).any()
    for j in range(8):
        out, tol = c.expert(torch.arange(T, device="cuda"), 512 + j)
        assert ((c.ysh[j].double() - out).abs() <= tol).all(), j


def test_expert_ffn_i8_rows_in_dispatched_order():
    c = Ffn8(70, 256, 8, 2, 160, 0, "bf16")
    c.run()
    want = c.y.clone()
    c.y.fill_(7.0)
    src = c.src.long()
    smoe.smoe_expert_ffn_i8(c.desc, c.xq[src].contiguous(), c.xs[src].contiguous(), c.off, c.W, c.y, c.ws)
    assert torch.equal(c.y, want)


def test_expert_ffn_i8_zero_and_non_finite_rows():
    """A zero token gives zeros, a NaN scale gives NaN in its own rows only."""
    c = Ffn8(40, 128, 4, 2, 64, 1, "f32")
    c.run()
    clean, clean_sh = c.y.clone(), c.ysh.clone()
    c.xq[3] = 0
    c.xs[7] = math.nan
    c.run()
    src = c.src.long()
    z, n = src == 3, src == 7
    assert (c.y[z] == 0).all() and (c.ysh[0, 3] == 0).all()
    assert c.y[n].isnan().all() and c.ysh[0, 7].isnan().all()
    assert torch.equal(c.y[~(z | n)], clean[~(z | n)])


def test_expert_ffn_i8_captured_graphs_share_a_workspace():
    a, b = (Ffn8(20, 256, 8, 2, 160, 1, "bf16", seed=s) for s in (1, 2))
    b.ws = a.ws
    graphs = []
    for c in (a, b):
        c.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    for _ in range(2):
        for c, g in zip((a, b), graphs):
            c.y.fill_(9.0)
            g.replay()
            torch.cuda.synchronize()
            c.check()


# ------------------------------------------------------------------ together
def test_norm_route_dispatch_ffn_combine():
    """An 8-bit layer as it is served: residual add and norm, route on the norm, dispatch, 8-bit
    FFN on the norm's 8-bit rows, combine; against the same steps in float64 on its routes."""
    T, d, E, K, F, S = 200, 512, 16, 4, 320, 1
    c = Ffn8(T, d, E, K, F, S, "bf16")
    g = gen(3)
    r, y = randn(g, T, d) * 2, randn(g, T, d).bfloat16()
    gamma = 1 + 0.1 * randn(g, d)
    w_gate = (randn(g, E, d) / math.sqrt(d)).bfloat16()
    ws = smoe.workspace(c.desc)
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    c.xq, c.xs = torch.empty(T, d, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    idx, w = i32(T, K), torch.empty(T, K, device="cuda")
    pair_row, c.src, c.off = i32(T, K), i32(T * K), i32(E + 1)
    out = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    smoe.smoe_add_rmsnorm(c.desc, r, gamma, y=y, r_out=r, x_out=x, q_out=c.xq, q_scale=c.xs)
    smoe.smoe_route(c.desc, x, w_gate, idx, w, ws=ws)
    smoe.smoe_dispatch(c.desc, idx, c.off, pair_row, c.src, ws)
    c.run()
    smoe.smoe_combine(c.desc, c.y, pair_row, w, out, ws, y_shared=c.ysh)
    smoe.smoe_get_status(ws)
    n = norm_ref(r, None, gamma, 1e-6)[1]
    check_norm(n, dict(x_out=x, q_out=c.xq, q_scale=c.xs), "bf16")
    c.check()
    ref = c.ysh[0].double() + (w.double()[..., None] * c.y[pair_row.long()].double()).sum(1)
    mag = c.ysh[0].double().abs() + (w.double()[..., None] * c.y[pair_row.long()].double().abs()).sum(1)
    assert ((out.double() - ref).abs() <= HALF["bf16"] * ref.abs() + 8 * HALF["f32"] * mag).all()


@pytest.mark.parametrize("T,n_out", [(40, 264), (900, 264), (900, 1608)])
def test_norm_then_product_queued(T, n_out):
    """Norms and the products of their rows queued one behind the other on the same buffers, two
    inputs in turn: each product is that of its own norm's rows."""
    g = gen(15)
    K, E, d = 2, 3, 1024
    wq, sw = int8(g, E, n_out, d), torch.rand(E, n_out, generator=g, device="cuda")
    src, off = rows_of(T, K, E, 6)
    desc = smoe.make_desc(T, d, E, K, 1, n_out, 0, 1, 1, "f32")
    rs, gamma = [randn(g, T, d), 50 * randn(g, T, d)], 1 + 0.1 * randn(g, d)
    q, qs = torch.empty(T, d, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    qd, qsd = torch.empty(T * K, d, dtype=torch.int8, device="cuda"), torch.empty(T * K, device="cuda")
    ddesc = smoe.make_desc(T * K, d, E, 1, 1, n_out, 0, 1, 1, "f32")
    ws, outs = smoe.workspace_i8(desc), torch.empty(20, 2, T * K, n_out, device="cuda")
    rd = [r[src.long()].contiguous() for r in rs]
    for i in range(20):
        r = i & 1
        smoe.smoe_add_rmsnorm(desc, rs[r], gamma, q_out=q, q_scale=qs)
        smoe.smoe_expert_matmul_i8(desc, q, qs, off, wq, sw, outs[i, 0], ws, row_src=src)
        smoe.smoe_add_rmsnorm(ddesc, rd[r], gamma, q_out=qd, q_scale=qsd)
        smoe.smoe_expert_matmul_i8(desc, qd, qsd, off, wq, sw, outs[i, 1], ws)
    smoe.smoe_get_status(ws)
    for r in (0, 1):
        smoe.smoe_add_rmsnorm(desc, rs[r], gamma, q_out=q, q_scale=qs)
        ref, _ = matmul_ref(q, qs, src, off, wq, sw)
        assert ((outs[r::2].double() - ref).abs() <= 2.1 * HALF["f32"] * ref.abs()).all()


def test_the_8bit_layer_captured():
    """The same run captured into a graph and replayed on new inputs, equal to the eager run."""
    T, d, E, K, F, S = 120, 256, 8, 2, 192, 1
    c = Ffn8(T, d, E, K, F, S, "bf16")
    g = gen(8)
    r0 = randn(g, T, d)
    r, y = r0.clone(), randn(g, T, d).bfloat16()
    gamma, w_gate = 1 + 0.1 * randn(g, d), (randn(g, E, d) / math.sqrt(d)).bfloat16()
    ws = smoe.workspace(c.desc)
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    c.xq, c.xs = torch.empty(T, d, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    idx, w = i32(T, K), torch.empty(T, K, device="cuda")
    pair_row, c.src, c.off = i32(T, K), i32(T * K), i32(E + 1)
    out = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")

    def layer():
        smoe.smoe_add_rmsnorm(c.desc, r, gamma, y=y, r_out=r, x_out=x, q_out=c.xq, q_scale=c.xs)
        smoe.smoe_route(c.desc, x, w_gate, idx, w, ws=ws)
        smoe.smoe_dispatch(c.desc, idx, c.off, pair_row, c.src, ws)
        c.run()
        smoe.smoe_combine(c.desc, c.y, pair_row, w, out, ws, y_shared=c.ysh)

    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for i in range(3):
        y.copy_(randn(g, T, d).bfloat16())
        r.copy_(r0 * (i + 1))
        layer()
        want = out.clone()
        r.copy_(r0 * (i + 1))
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        c.check()
    smoe.smoe_get_status(ws)


def test_few_beside_the_8bit_products():
    """The cooperative few-token kernel and the 8-bit FFN's pairs on two streams at once."""
    a, b = Few(6, 1024, 16, 2, 1, 512, 1, "bf16"), Ffn8(400, 512, 8, 2, 320, 1, "bf16")
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        a.run(stream=streams[0])
        b.run(stream=streams[1])
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_decode_steps_captured():
    """Norm, few-token layer and norm in one graph, step after step on the residual it updates."""
    c = Few(3, 512, 16, 2, 1, 256, 1, "bf16")
    g = gen(12)
    r, gamma = randn(g, 3, 512), 1 + 0.1 * randn(g, 512)
    eager = r.clone()

    def step(res):
        smoe.smoe_add_rmsnorm(c.desc, res, gamma, x_out=c.x)
        c.run()
        smoe.smoe_add_rmsnorm(c.desc, res, gamma, y=c.y, r_out=res)

    for _ in range(4):
        step(eager)
    torch.cuda.synchronize()
    graph, res = torch.cuda.CUDAGraph(), r.clone()
    with torch.cuda.graph(graph):
        step(res)
    res.copy_(r)
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    smoe.smoe_get_status(c.ws)
    assert torch.equal(res, eager)


def test_norm_then_few():
    """A decode step: the norm's output is the few-token layer's input, its output the next
    norm's addend."""
    c = Few(8, 768, 24, 3, 1, 320, 1, "bf16")
    g = gen(4)
    r, gamma = randn(g, 8, 768), 1 + 0.1 * randn(g, 768)
    smoe.smoe_add_rmsnorm(c.desc, r, gamma, x_out=c.x)
    c.run()
    out = norm_buffers(8, 768, "bf16")
    smoe.smoe_add_rmsnorm(c.desc, r, gamma, y=c.y, **out)
    c.check()
    assert torch.equal(out["r_out"], r + c.y.float())
    check_norm(norm_ref(out["r_out"], None, gamma, 1e-6)[1], out, "bf16")
