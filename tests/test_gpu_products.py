"""The 8-bit floating-point rows and products, the grouped products with their gradients and the
8-bit activation checkpoints on the GPU, against plain formulas in 64 bits.

Tolerances. A rounding is off by at most half a step of its type (bf16 2^-8, fp32 2^-24, e4m3
2^-4, relative to the value). A sum of n products in fp32, each addition off by at most a step of
the running sum (2^-23: a tensor core may cut off instead of rounding), is off by at most n 2^-23
sum |a b|; a tensor core adds 16 (32) products at once, so n is the count of its additions."""
import math

import pytest
import torch

import routing_token_shuffle_gb300 as smoe

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
F8 = torch.float8_e4m3fn
F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def within(x, ref, tol):
    """|x - ref| <= tol everywhere (a NaN is not)."""
    err = (x.double() - ref.double()).abs()
    bad = ~(err <= tol)
    n = int(bad.sum())
    assert n == 0, (n, float(err[bad].max()), bad.nonzero()[0].tolist())


def same(a, b):
    n = int((a != b).sum())
    assert n == 0, (n, a.numel(), (a != b).nonzero()[0].tolist())


def f8(x):
    """e4m3, with zeros for values past the largest (only magnitudes up to 448 are passed)."""
    return x.to(F8)


def blocks(n):
    return -(-n // 128)


def spread(s, n):
    return s.double().repeat_interleave(128, -1)[..., :n]


# ------------------------------------------------------------------ rows in 8 bits
def rows_desc(dt):
    return smoe.make_desc(1, 8, 1, 1, 1, 8, 0, 1, 1, dt)


def rows_ref(x, pow2):
    """(scale, x / scale) by block, in fp32 as it is documented."""
    T, d = x.shape
    pad = torch.zeros(T, blocks(d) * 128, device=x.device)
    pad[:, :d] = x.float().abs()
    s = pad.view(T, -1, 128).amax(-1)
    s = s / torch.full_like(s, 448.0)  # (by a number torch would multiply with its inverse)
    if pow2:
        m, e = torch.frexp(s)
        s = torch.where(s > 0, torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e)), s)
    return s, x.float() / s.repeat_interleave(128, 1)[:, :d]


@pytest.mark.parametrize("pow2", [0, 1])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 8), (3, 128), (1, 136), (17, 120), (64, 5120), (2049, 2048),
                                 (33, 8200), (700, 1000), (40000, 128)])
def test_rows_f8(T, d, dt, pow2):
    x = (randn(gen(T + d), T, d) * 3).to(DT[dt])
    q = torch.full((T, d), 7, dtype=torch.uint8, device="cuda")
    s = torch.full((T, blocks(d)), 7.0, device="cuda")
    smoe.smoe_rows_f8(rows_desc(dt), x, q, s, pow2=pow2)
    rs, v = rows_ref(x, pow2)
    same(s, rs)
    same(q, f8(v).view(torch.uint8))
    # half a step of e4m3, and half of its smallest step (2^-9) for magnitudes near zero
    within(q.view(F8).double() * spread(s, d), x, x.double().abs() * 2.0 ** -4 + spread(s, d) * 2.0 ** -10)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("pow2", [0, 1])
def test_rows_f8_odd_blocks(dt, pow2):
    """Zero blocks, tiny blocks, exact powers of two, blocks with an infinity or a NaN; the blocks
    beside them and the largest values."""
    x = randn(gen(3), 9, 300).to(DT[dt])
    x[1, :128] = 0.0
    x[2, 128:256] *= 1e-37          # 4e-37 / 448: below the smallest normal number
    x[3, 5], x[4, 299], x[5, 130] = math.inf, math.nan, -math.inf
    x[6] = 0.0
    x[6, ::128] = 3.5               # 448 x 2^-7
    x[7] = torch.finfo(DT[dt]).max
    x[8, :128] *= 1e-30
    q = torch.full((9, 300), 7, dtype=torch.uint8, device="cuda")
    s = torch.full((9, 3), 7.0, device="cuda")
    # 300 is no multiple of 8: the first 296 channels
    x, q = x[:, :296].contiguous(), q[:, :296].contiguous()
    x[4, 295] = math.nan
    smoe.smoe_rows_f8(rows_desc(dt), x, q, s, pow2=pow2)
    bad = torch.zeros(9, 3, dtype=torch.bool, device="cuda")
    bad[3, 0] = bad[4, 2] = bad[5, 1] = True
    zero = torch.zeros_like(bad)
    zero[1, 0] = zero[2, 1] = True
    assert s[bad].isnan().all() and (s[zero] == 0).all()
    off = (bad | zero).repeat_interleave(128, 1)[:, :296]
    assert (q[off] == 0).all()
    rs, v = rows_ref(torch.where(off, torch.zeros_like(x), x), pow2)
    same(s[~(bad | zero)], rs[~(bad | zero)])
    same(q[~off], f8(torch.where(off, torch.zeros_like(v), v)).view(torch.uint8)[~off])
    assert (s[6] == 2.0 ** -7).all() and (q[6, ::128] == 0x7e).all()


# ------------------------------------------------------------------ SwiGLU, kept in 8 bits
def swiglu_tol(dt):
    """exp, a division and three products around them in fp32 (under 2^-20 with the fast forms of
    bf16 layers, 2^-21 with the accurate ones), and the result's rounding."""
    return HALF[dt] + (2.0 ** -20 if dt == "bf16" else 2.0 ** -21)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 8), (5, 128), (384, 1536), (37, 1000), (3001, 768), (9, 14336)])
def test_swiglu_f8(T, d, dt):
    g_ = gen(T * 7 + d)
    g, u, dh = ((randn(g_, T, d) * s).to(DT[dt]) for s in (2.0, 1.0, 0.1))
    if d >= 128:
        g[0, :8] = torch.tensor([-200.0, -90, -20, -1e-6, 0, 1e-6, 60, 300], device="cuda").to(DT[dt])
    new = lambda: (torch.full((T, d), 7, dtype=torch.uint8, device="cuda"),  # noqa: E731
                   torch.full((T, blocks(d)), 7.0, device="cuda"))
    (h8, hs), (g8, gs), (u8, us) = new(), new(), new()
    h = torch.full_like(g, 7.0)
    desc = rows_desc(dt)
    smoe.smoe_swiglu_f8(desc, g, u, h=h, h8=h8, h8_scale=hs, g8=g8, g8_scale=gs, u8=u8, u8_scale=us)
    for x, q, s in ((g, g8, gs), (u, u8, us)):
        rs, v = rows_ref(x, 1)
        same(s, rs)
        same(q, f8(v).view(torch.uint8))
    G, U = g.double(), u.double()
    ref = G * torch.sigmoid(G) * U
    # sig below 2^-126 is zero in fp32: 1e-37 |g u|
    within(h, ref, swiglu_tol(dt) * ref.abs() + 1e-37 * (G * U).abs() + 1e-38)
    back = h8.view(F8).double() * spread(hs, d)
    within(back, ref, ref.abs() * (2.0 ** -4 + 2.0 ** -19) + spread(hs, d) * 2.0 ** -9)
    # each output alone, h over g and over u
    for k in ("h8", "g8", "u8"):
        q, s = new()
        smoe.smoe_swiglu_f8(desc, g, u, **{k: q, k + "_scale": s})
        want = {"h8": (h8, hs), "g8": (g8, gs), "u8": (u8, us)}[k]
        same(q, want[0])
        same(s, want[1])
    for over in (0, 1):
        a = [g.clone(), u.clone()]
        smoe.smoe_swiglu_f8(desc, *a, h=a[over])
        same(a[over], h)
    # backward, from what was kept
    G, U, D = g8.view(F8).double() * spread(gs, d), u8.view(F8).double() * spread(us, d), dh.double()
    sig = torch.sigmoid(G)
    dg, du, h2 = (torch.full_like(g, 7.0) for _ in range(3))
    smoe.smoe_swiglu_grad_f8(desc, dh, g8, gs, u8, us, dg, du, h=h2)
    tol = swiglu_tol(dt)
    small = 1e-37 * (1 + (G * U * D).abs() + (G * D).abs() + (G * U).abs()) + 1e-38
    # 1 + g (1 - sig) has a root near g = -1.28: what its terms lose is relative to them
    terms = (D * U * sig).abs() * (1 + G.abs() * (1 - sig))
    ref = D * U * sig * (1 + G * (1 - sig))
    # (1 - sig is off by a step of 1 where sig is near it: 2^-23 |g|)
    within(dg, ref, HALF[dt] * ref.abs() + 2 * (tol - HALF[dt]) * terms + 2.0 ** -23 * (D * U * sig * G).abs() + small)
    within(du, D * G * sig, tol * (D * G * sig).abs() + small)
    within(h2, G * sig * U, tol * (G * sig * U).abs() + small)
    dg2 = dh.clone()
    smoe.smoe_swiglu_grad_f8(desc, dg2, g8, gs, u8, us, dg2, torch.empty_like(du))
    same(dg2, dg)


def test_swiglu_gradient_against_differences():
    """dg and du of sum(h dh), by central differences in 64 bits of the kept values."""
    g_ = gen(11)
    desc, dh = rows_desc("f32"), randn(g_, 4, 128)
    g, u = randn(g_, 4, 128) * 2, randn(g_, 4, 128)
    q = [torch.empty(4, 128, dtype=torch.uint8, device="cuda") for _ in range(2)]
    s = [torch.empty(4, 1, device="cuda") for _ in range(2)]
    smoe.smoe_swiglu_f8(desc, g, u, g8=q[0], g8_scale=s[0], u8=q[1], u8_scale=s[1])
    dg, du = torch.empty_like(g), torch.empty_like(g)
    smoe.smoe_swiglu_grad_f8(desc, dh, q[0], s[0], q[1], s[1], dg, du)
    G, U = (a.view(F8).double() * spread(b, 128) for a, b in zip(q, s))
    f = lambda g, u: g * torch.sigmoid(g) * u * dh.double()  # noqa: E731
    e = 1e-5
    # the differences' own error: e^2 |h'''| / 6, and 2^-52 / e of the values
    num = (f(G + e, U) - f(G - e, U)) / (2 * e)
    within(dg, num, 1e-6 * (1 + num.abs()))
    num = (f(G, U + e) - f(G, U - e)) / (2 * e)
    within(du, num, 1e-6 * (1 + num.abs()))


def test_swiglu_kept_block_that_is_not_finite():
    """A kept block with a NaN scale gives NaN gradients there, and nowhere else."""
    g = randn(gen(2), 3, 384)
    u, dh = torch.ones_like(g), torch.ones_like(g)
    g[1, 200] = math.inf
    q = [torch.empty(3, 384, dtype=torch.uint8, device="cuda") for _ in range(2)]
    s = [torch.empty(3, 3, device="cuda") for _ in range(2)]
    smoe.smoe_swiglu_f8(rows_desc("f32"), g, u, g8=q[0], g8_scale=s[0], u8=q[1], u8_scale=s[1])
    dg, du = torch.empty_like(g), torch.empty_like(g)
    smoe.smoe_swiglu_grad_f8(rows_desc("f32"), dh, q[0], s[0], q[1], s[1], dg, du)
    bad = torch.zeros(3, 384, dtype=torch.bool, device="cuda")
    bad[1, 128:256] = True
    assert torch.equal(dg.isnan(), bad) and torch.equal(du.isnan(), bad)


# ------------------------------------------------------------------ products
def offsets(kind, R, E, seed):
    """expert_off of R rows: even; skewed with empty experts; all on one expert; the last rows
    (and the first) on nobody."""
    rng = torch.Generator().manual_seed(seed)
    if kind == "one":
        n = torch.zeros(E, dtype=torch.long)
        n[E // 2] = R
    elif kind == "even":
        n = torch.full((E,), R // E)
        n[: R - int(n.sum())] += 1
    else:
        p = torch.rand(E, generator=rng) ** 3
        p[torch.rand(E, generator=rng) < 0.3] = 0.0
        if float(p.sum()) == 0:
            p[0] = 1.0
        used = R if kind == "skew" else max(1, R - R // 5)
        n = torch.bincount(torch.multinomial(p, used, replacement=True, generator=rng), minlength=E)
    first = R // 10 if kind == "gaps" else 0
    off = torch.cat([torch.zeros(1, dtype=torch.long), n.cumsum(0)]) + first
    return off.to(torch.int32).cuda().clamp_(max=R)


class Case:
    def __init__(self, T, K, E, n_in, n_out, dt, kind, seed=0):
        self.T, self.K, self.E, self.n_in, self.n_out, self.dt = T, K, E, n_in, n_out, dt
        self.R = T * K
        self.off = offsets(kind, self.R, E, seed + T)
        o = self.off.tolist()
        self.seg = [slice(o[e], o[e + 1]) for e in range(E)]
        self.inside = torch.zeros(self.R, dtype=torch.bool, device="cuda")
        self.inside[o[0]:o[E]] = True
        self.desc = smoe.make_desc(T, n_in, E, K, 1, n_out, 0, 1, 1, dt)
        self.ws = smoe.workspace_products(self.desc)
        self.g = gen(seed + T * 31 + n_in + n_out)

    def rows(self, n, scale=1.0):
        """Rows with NaN outside the segments."""
        x = (randn(self.g, self.R, n) * scale).to(DT[self.dt])
        x[~self.inside] = math.nan
        return x

    def weights(self):
        return (randn(self.g, self.E, self.n_out, self.n_in) / math.sqrt(self.n_in)).to(DT[self.dt])

    def out(self, n):
        return torch.full((self.R, n), 7.0, dtype=DT[self.dt], device="cuda")

    def check_rows(self, out, ref, mag, adds):
        smoe.smoe_get_status(self.ws)
        assert (out[~self.inside] == 7.0).all()
        i = self.inside
        within(out[i], ref[i], HALF[self.dt] * ref[i].abs() + adds * 2.0 ** -23 * mag[i] + 1e-37)


SHAPES = [
    # T, K, E, n_in, n_out, kind
    (1, 1, 1, 16, 8, "even"), (5, 2, 3, 8, 8, "skew"), (600, 1, 2, 16, 8, "skew"), (1, 2, 4, 64, 72, "even"), (3, 2, 8, 272, 136, "skew"),
    (64, 6, 160, 256, 384, "skew"), (40, 2, 3, 1008, 520, "gaps"), (129, 1, 1, 128, 256, "one"),
    (64, 1, 1, 144, 264, "one"), (301, 3, 24, 1008, 200, "skew"), (400, 2, 2, 128, 1416, "gaps"),
    (1000, 1, 3, 512, 512, "skew"), (777, 4, 16, 80, 776, "gaps"), (2048, 2, 8, 384, 640, "even"),
    (95, 2, 512, 64, 64, "skew"), (950, 2, 7, 520, 264, "gaps"),
    (1500, 1, 1, 640, 72, "gaps"), (3000, 1, 2, 128, 136, "skew"), (2600, 1, 1, 1040, 264, "one"), (17, 1, 1, 5120, 64, "one"), (700, 2, 5, 2064, 24, "skew"),
]


def adds16(n):
    return n / 16 + 24  # the tensor core's additions, and a few around them


def adds1(n):
    return n + 4


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,E,n_in,n_out,kind", SHAPES)
def test_expert_matmul(T, K, E, n_in, n_out, kind, dt):
    c = Case(T, K, E, n_in, n_out, dt, kind)
    x, w, out = c.rows(n_in), c.weights(), c.out(n_out)
    smoe.smoe_expert_matmul(c.desc, x, c.off, w, out, c.ws)
    ref, mag = torch.zeros(2, c.R, n_out, dtype=F64, device="cuda")
    for e, s in enumerate(c.seg):
        ref[s] = x[s].double() @ w[e].double().T
        mag[s] = x[s].double().abs() @ w[e].double().abs().T
    c.check_rows(out, ref, mag, adds16(n_in) if dt == "bf16" else adds1(n_in))
    again = c.out(n_out)
    smoe.smoe_expert_matmul(c.desc, x, c.off, w, again, c.ws)
    same(again, out)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,E,n_in,n_out,kind", SHAPES)
def test_expert_matmul_dx(T, K, E, n_in, n_out, kind, dt):
    c = Case(T, K, E, n_in, n_out, dt, kind, seed=1)
    dy, w, dy2, w2 = c.rows(n_out), c.weights(), c.rows(n_out), c.weights()
    for two in (False, True):
        dx = c.out(n_in)
        smoe.smoe_expert_matmul_dx(c.desc, dy, w, c.off, dx, c.ws, **(dict(dy2=dy2, w2=w2) if two else {}))
        ref, mag = torch.zeros(2, c.R, n_in, dtype=F64, device="cuda")
        for e, s in enumerate(c.seg):
            for a, b in ((dy, w), (dy2, w2))[: 1 + two]:
                ref[s] += a[s].double() @ b[e].double()
                mag[s] += a[s].double().abs() @ b[e].double().abs()
        n = n_out * (1 + two)
        c.check_rows(dx, ref, mag, adds16(n) if dt == "bf16" else adds1(n))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,E,n_in,n_out,kind", SHAPES)
def test_expert_matmul_dw(T, K, E, n_in, n_out, kind, dt):
    c = Case(T, K, E, n_in, n_out, dt, kind, seed=2)
    dy, x = c.rows(n_out), c.rows(n_in)
    ref, mag = torch.zeros(2, E, n_out, n_in, dtype=F64, device="cuda")
    most = 0
    for e, s in enumerate(c.seg):
        ref[e] = dy[s].double().T @ x[s].double()
        mag[e] = dy[s].double().abs().T @ x[s].double().abs()
        most = max(most, s.stop - s.start)
    adds = adds16(most) if dt == "bf16" else adds1(most)
    dw = torch.full((E, n_out, n_in), 7.0, device="cuda")
    smoe.smoe_expert_matmul_dw(c.desc, dy, x, c.off, dw, c.ws)
    smoe.smoe_get_status(c.ws)
    within(dw, ref, adds * 2.0 ** -23 * mag)
    # added to an earlier gradient, in a buffer of its own and in place
    before = randn(c.g, E, n_out, n_in)
    want = dw + before
    both = torch.full_like(dw, 7.0)
    smoe.smoe_expert_matmul_dw(c.desc, dy, x, c.off, both, c.ws, add=before)
    same(both, want)
    smoe.smoe_expert_matmul_dw(c.desc, dy, x, c.off, before, c.ws, add=before)
    same(before, want)


@pytest.mark.parametrize("pow2", [0, 1])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,E,n_in,n_out,kind", [s for s in SHAPES if s[3] % 16 == 0])
def test_expert_matmul_dw_f8(T, K, E, n_in, n_out, kind, dt, pow2):
    """From token rows kept in 8 bits through row_src, and from dispatched ones: what the product of
    the widened rows gives, to the bit."""
    c = Case(T, K, E, n_in, n_out, dt, kind, seed=3)
    dy = c.rows(n_out)
    x = (randn(c.g, T, n_in) * 2).to(DT[dt])
    q, s = torch.empty(T, n_in, dtype=F8, device="cuda"), torch.empty(T, blocks(n_in), device="cuda")
    smoe.smoe_rows_f8(c.desc, x, q, s, pow2=pow2)
    src = torch.randint(0, T, (c.R,), generator=c.g, device="cuda", dtype=torch.int32)
    wide = (q.float() * s.repeat_interleave(128, 1)[:, :n_in]).to(DT[dt])
    if pow2:
        same(wide.double(), q.double() * spread(s, n_in))
    rows = wide[src.long()]
    want, got = (torch.full((E, n_out, n_in), 7.0, device="cuda") for _ in range(2))
    smoe.smoe_expert_matmul_dw(c.desc, dy, rows, c.off, want, c.ws)
    src[~c.inside] = -5  # rows of nobody are not looked up
    smoe.smoe_expert_matmul_dw_f8(c.desc, dy, q, s, c.off, got, c.ws, row_src=src)
    smoe.smoe_get_status(c.ws)
    same(got, want)
    got.fill_(7.0)
    src = src.long().clamp(min=0)
    smoe.smoe_expert_matmul_dw_f8(c.desc, dy, q.view(torch.uint8)[src], s[src], c.off, got, c.ws, add=want)
    same(got, want + want)


class F8Case(Case):
    def __init__(self, *a, pow2=0, seed=4):
        super().__init__(*a, seed=seed)
        T, E, n_in, n_out = self.T, self.E, self.n_in, self.n_out
        self.x = randn(self.g, T, n_in).to(DT[self.dt])
        self.q = torch.empty(T, n_in, dtype=F8, device="cuda")
        self.s = torch.empty(T, blocks(n_in), device="cuda")
        smoe.smoe_rows_f8(self.desc, self.x, self.q, self.s, pow2=pow2)
        self.wq = f8(randn(self.g, E, n_out, n_in) * 60)
        self.sw = torch.rand(E, blocks(n_out), blocks(n_in), generator=self.g, device="cuda") * 1e-3 + 1e-4
        self.src = torch.randint(0, T, (self.R,), generator=self.g, device="cuda", dtype=torch.int32)

    def run(self, src=True, **kw):
        out = self.out(self.n_out)
        q, s = (self.q, self.s) if src else (self.q.view(torch.uint8)[self.src.long()].view(F8),
                                              self.s[self.src.long()])
        smoe.smoe_expert_matmul_f8(self.desc, q, s, self.off, self.wq, self.sw, out, self.ws,
                                   row_src=self.src if src else None, **kw)
        return out

    def reference(self):
        x = (self.q.double() * spread(self.s, self.n_in))[self.src.long()]
        ref, mag = torch.zeros(2, self.R, self.n_out, dtype=F64, device="cuda")
        for e, s in enumerate(self.seg):
            w = self.wq[e].double() * spread(self.sw[e].repeat_interleave(128, 0)[:self.n_out], self.n_in)
            ref[s], mag[s] = x[s] @ w.T, x[s].abs() @ w.abs().T
        return ref, mag

    def check(self, out):
        # additions of 32 products each, one more a block for its scaled sum
        self.check_rows(out, *self.reference(), self.n_in / 32 + blocks(self.n_in) + 8)


@pytest.mark.parametrize("pow2", [0, 1])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,E,n_in,n_out,kind", [s for s in SHAPES if s[3] % 16 == 0])
def test_expert_matmul_f8(T, K, E, n_in, n_out, kind, dt, pow2):
    c = F8Case(T, K, E, n_in, n_out, dt, kind, pow2=pow2)
    out = c.run()
    c.check(out)
    same(c.run(src=False), out)


# ------------------------------------------------------------------ what the tiles must keep apart
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,n_in,n_out", [(200, 136, 72), (700, 520, 264), (40, 1000, 104), (4200, 520, 264)])
def test_an_expert_that_is_not_finite_stays_alone(T, n_in, n_out, dt):
    """Infinities and NaN in one expert's rows or weights reach no other expert's results."""
    c = Case(T, 1, 5, n_in, n_out, dt, "skew", seed=9)
    c.off = torch.tensor([0, T // 4 + 3, T // 2 + 1, T // 2 + 8, T - 5, T], dtype=torch.int32, device="cuda")
    o = c.off.tolist()
    c.inside[:] = True
    x, dy, w = c.rows(n_in), c.rows(n_out), c.weights()
    clean = c.out(n_out), c.out(n_in), torch.empty(5, n_out, n_in, device="cuda")
    dirty = c.out(n_out), c.out(n_in), torch.empty(5, n_out, n_in, device="cuda")
    for bad in range(5):
        s = slice(o[bad], o[bad + 1])
        for out, spoil in ((clean, False), (dirty, True)):
            x_, dy_, w_ = x.clone(), dy.clone(), w.clone()
            if spoil:
                for t in (x_[s], dy_[s], w_[bad]):
                    t[...] = math.nan
                    t.view(-1)[::3] = math.inf
            smoe.smoe_expert_matmul(c.desc, x_, c.off, w_, out[0], c.ws)
            smoe.smoe_expert_matmul_dx(c.desc, dy_, w_, c.off, out[1], c.ws)
            smoe.smoe_expert_matmul_dw(c.desc, dy_, x_, c.off, out[2], c.ws)
        keep = torch.ones(T, dtype=torch.bool, device="cuda")
        keep[s] = False
        same(dirty[0][keep], clean[0][keep])
        same(dirty[1][keep], clean[1][keep])
        others = [e for e in range(5) if e != bad]
        same(dirty[2][others], clean[2][others])
        assert not dirty[0][s].isfinite().any() and not dirty[2][bad].isfinite().any()


@pytest.mark.parametrize("T", [60, 900])
def test_f8_expert_that_is_not_finite_stays_alone(T):
    c = F8Case(T, 1, 5, 272, 200, "f32", "skew", seed=9)
    clean, o = c.run(), c.off.tolist()
    bad = max(range(5), key=lambda e: o[e + 1] - o[e])
    c.wq.view(torch.uint8)[bad] = 0x7f      # NaN
    c.sw[bad] = math.inf
    dirty = c.run()
    keep = torch.ones(c.R, dtype=torch.bool, device="cuda")
    keep[o[bad]:o[bad + 1]] = False
    same(dirty[keep], clean[keep])
    # a token whose scale is NaN: its rows alone
    c = F8Case(T, 1, 5, 272, 200, "f32", "skew", seed=9)
    c.s[3, 1] = math.nan
    dirty = c.run()
    hit = c.src == 3
    same(dirty[~hit], clean[~hit])
    assert dirty[hit & c.inside].isnan().all()


# ------------------------------------------------------------------ bad data, empty batches
def test_bad_offsets_write_nothing():
    for dt in ("bf16", "f32"):
        for bad in ([0, 40, 30, 60], [0, 20, 40, 61], [-1, 20, 40, 60]):
            c = Case(60, 1, 3, 64, 128, dt, "even")
            x, dy, w = c.rows(64), c.rows(128), c.weights()
            off = torch.tensor(bad, dtype=torch.int32, device="cuda")
            out, dx, dw = c.out(128), c.out(64), torch.full((3, 128, 64), 7.0, device="cuda")
            for call in (lambda: smoe.smoe_expert_matmul(c.desc, x, off, w, out, c.ws),
                         lambda: smoe.smoe_expert_matmul_dx(c.desc, dy, w, off, dx, c.ws),
                         lambda: smoe.smoe_expert_matmul_dw(c.desc, dy, x, off, dw, c.ws)):
                call()
                with pytest.raises(smoe.SmoeError, match="SMOE_ERR_DATA"):
                    smoe.smoe_get_status(c.ws)
            assert (out == 7).all() and (dx == 7).all() and (dw == 7).all()
    f = F8Case(60, 1, 3, 64, 128, "bf16", "even")
    f.off = torch.tensor([0, 40, 30, 60], dtype=torch.int32, device="cuda")
    assert (f.run() == 7).all()
    with pytest.raises(smoe.SmoeError, match="SMOE_ERR_DATA"):
        smoe.smoe_get_status(f.ws)


@pytest.mark.parametrize("T", [30, 600])
def test_bad_row_src(T):
    """An entry out of range gives a zero row and an error in the status; the others stay."""
    f = F8Case(T, 2, 4, 256, 264, "bf16", "even")
    good = f.run()
    smoe.smoe_get_status(f.ws)
    keep = f.src.clone()
    f.src[[5, 11, 2 * T - 1]] = torch.tensor([-1, T, 1 << 30], dtype=torch.int32, device="cuda")
    hit = f.src != keep
    bad = f.run()
    with pytest.raises(smoe.SmoeError, match="SMOE_ERR_DATA"):
        smoe.smoe_get_status(f.ws)
    same(bad[~hit], good[~hit])
    assert (bad[hit] == 0).all()
    for dt in ("bf16", "f32"):
        c = Case(T, 2, 4, 256, 264, dt, "even")
        dy, dw, want = c.rows(264), torch.empty(4, 264, 256, device="cuda"), torch.empty(4, 264, 256, device="cuda")
        smoe.smoe_expert_matmul_dw_f8(c.desc, dy, f.q, f.s, c.off, dw, c.ws, row_src=f.src)
        with pytest.raises(smoe.SmoeError, match="SMOE_ERR_DATA"):
            smoe.smoe_get_status(c.ws)
        dy[hit] = 0.0
        smoe.smoe_expert_matmul_dw_f8(c.desc, dy, f.q, f.s, c.off, want, c.ws, row_src=keep)
        same(dw, want)


def test_empty_batches():
    for dt in ("bf16", "f32"):
        d0 = smoe.make_desc(0, 64, 3, 1, 1, 128, 0, 1, 1, dt)
        ws, e = smoe.workspace_products(d0), torch.empty(0, 64, dtype=DT[dt], device="cuda")
        y, w = torch.empty(0, 128, dtype=DT[dt], device="cuda"), torch.ones(3, 128, 64, dtype=DT[dt], device="cuda")
        off = torch.zeros(4, dtype=torch.int32, device="cuda")
        smoe.smoe_expert_matmul(d0, e, off, w, y, ws)
        smoe.smoe_expert_matmul_dx(d0, y, w, off, e, ws)
        dw, add = torch.full((3, 128, 64), 7.0, device="cuda"), torch.rand(3, 128, 64, device="cuda")
        smoe.smoe_expert_matmul_dw(d0, y, e, off, dw, ws)
        assert (dw == 0).all()
        smoe.smoe_expert_matmul_dw(d0, y, e, off, dw, ws, add=add)
        same(dw, add)
        q, s = torch.empty(0, 64, dtype=F8, device="cuda"), torch.empty(0, 1, device="cuda")
        smoe.smoe_rows_f8(d0, e, q, s)
        smoe.smoe_expert_matmul_dw_f8(d0, y, q, s, off, dw, ws, row_src=off)
        assert (dw == 0).all()
        smoe.smoe_swiglu_f8(d0, e, e, h=e, g8=q, g8_scale=s)
        smoe.smoe_swiglu_grad_f8(d0, e, q, s, q, s, e, e)
        # tokens, and none of their rows on any expert
        c = Case(9, 1, 3, 64, 128, dt, "even")
        x, dy = c.rows(64), c.rows(128)
        x[:] = math.nan
        dy[:] = math.nan
        out = c.out(128)
        smoe.smoe_expert_matmul(c.desc, x, off, w, out, c.ws)
        assert (out == 7).all()
        smoe.smoe_expert_matmul_dw(c.desc, dy, x, off, dw, c.ws, add=add)
        same(dw, add)
        smoe.smoe_get_status(c.ws)


# ------------------------------------------------------------------ streams, graphs, long offsets
class Step:
    """A training step of the experts' FFN from a batch of tokens, as a program runs it: dispatch, up
    products, SwiGLU kept in 8 bits, down product, combine; and back, with every gradient."""

    def __init__(self, T, d, E, K, F, dt, seed=0):
        g = gen(seed + T + d + F)
        t = DT[dt]
        self.T, self.d, self.E, self.K, self.F, self.dt = T, d, E, K, F, dt
        R = T * K
        self.desc = smoe.make_desc(T, d, E, K, 1, F, 0, 1, 1, dt)
        self.ws, self.wp = smoe.workspace(self.desc), smoe.workspace_products(self.desc)
        self.x = randn(g, T, d).to(t)
        self.idx = torch.stack([torch.randperm(E, generator=g, device="cuda")[:K] for _ in range(T)]).int()
        self.w = torch.softmax(randn(g, T, K), -1)
        self.w1, self.w3 = ((randn(g, E, F, d) / math.sqrt(d)).to(t) for _ in range(2))
        self.w2 = (randn(g, E, d, F) / math.sqrt(F)).to(t)
        self.dout = (randn(g, T, d) * 0.1).to(t)
        i = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        n = lambda *s, dtype=t: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        self.off, self.pair, self.tok = i(E + 1), i(T, K), i(R)
        self.xd, self.y, self.dyd = n(R, d), n(R, d), n(R, d)
        self.g, self.u, self.h, self.dh, self.dg, self.du, self.h2 = (n(R, F) for _ in range(7))
        self.x8, self.xs = n(T, d, dtype=F8), n(T, blocks(d), dtype=torch.float32)
        self.g8, self.u8 = n(R, F, dtype=F8), n(R, F, dtype=F8)
        self.gs, self.us = (n(R, blocks(F), dtype=torch.float32) for _ in range(2))
        self.out, self.dxd = n(T, d), n(R, d)
        self.dw1, self.dw3 = (n(E, F, d, dtype=torch.float32) for _ in range(2))
        self.dw2 = n(E, d, F, dtype=torch.float32)

    def forward(self):
        smoe.smoe_dispatch(self.desc, self.idx, self.off, self.pair, self.tok, self.ws, x_src=self.x, x_disp=self.xd)
        smoe.smoe_rows_f8(self.desc, self.x, self.x8, self.xs, pow2=1)
        smoe.smoe_expert_matmul(self.desc, self.xd, self.off, self.w1, self.g, self.wp)
        smoe.smoe_expert_matmul(self.desc, self.xd, self.off, self.w3, self.u, self.wp)
        smoe.smoe_swiglu_f8(self.desc, self.g, self.u, h=self.h, g8=self.g8, g8_scale=self.gs, u8=self.u8,
                            u8_scale=self.us)
        smoe.smoe_expert_matmul(self.desc, self.h, self.off, self.w2, self.y, self.wp)
        smoe.smoe_combine(self.desc, self.y, self.pair, self.w, self.out, self.ws)

    def backward(self):
        """dy of each row is its token's gradient times its weight."""
        wr = torch.empty(self.T * self.K, device="cuda")
        wr[self.pair.view(-1).long()] = self.w.view(-1)
        self.dyd.copy_((self.dout.float()[self.tok.long()] * wr[:, None]))
        smoe.smoe_expert_matmul_dx(self.desc, self.dyd, self.w2, self.off, self.dh, self.wp)
        smoe.smoe_swiglu_grad_f8(self.desc, self.dh, self.g8, self.gs, self.u8, self.us, self.dg, self.du, h=self.h2)
        smoe.smoe_expert_matmul_dw(self.desc, self.dyd, self.h2, self.off, self.dw2, self.wp)
        smoe.smoe_expert_matmul_dw_f8(self.desc, self.dg, self.x8, self.xs, self.off, self.dw1, self.wp, row_src=self.tok)
        smoe.smoe_expert_matmul_dw_f8(self.desc, self.du, self.x8, self.xs, self.off, self.dw3, self.wp, row_src=self.tok)
        smoe.smoe_expert_matmul_dx(self.desc, self.dg, self.w1, self.off, self.dxd, self.wp, dy2=self.du, w2=self.w3)

    def outputs(self):
        return [self.out, self.dw1, self.dw3, self.dw2, self.dxd]

    def check(self):
        """Against autograd in 64 bits: the 8-bit values are off by up to 2^-4, so a sum of n terms that
        carry independent such errors is off by about 2^-4 / sqrt(3) of its terms' root sum of
        squares; five of those (the largest of 10^5 values lies at 4.4)."""
        T, K, E = self.T, self.K, self.E
        x, w1, w3, w2 = (t.double().requires_grad_() for t in (self.x, self.w1, self.w3, self.w2))
        out = torch.zeros(T, self.d, dtype=F64, device="cuda")
        for e in range(E):
            t, k = torch.nonzero(self.idx == e, as_tuple=True)
            if len(t):
                g, u = x[t] @ w1[e].T, x[t] @ w3[e].T
                out = out.index_add(0, t, ((g * torch.sigmoid(g) * u) @ w2[e].T) * self.w[t, k].double()[:, None])
        out.backward(self.dout.double())
        rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
        step = 2.0 ** -8 if self.dt == "bf16" else 2.0 ** -20
        assert rel(self.out, out.detach()) <= 4 * step
        # each term of a gradient carries the relative errors of at most three 8-bit values (x, g and
        # u; dg carries g twice): their norm is within 4 x 2^-4 / sqrt(3) of the gradient's own
        tol = 4 * 2.0 ** -4 / math.sqrt(3) + 8 * step
        assert rel(self.dw1, w1.grad) <= tol and rel(self.dw3, w3.grad) <= tol
        assert rel(self.dw2, w2.grad) <= tol
        dx = torch.zeros_like(x).index_add(0, self.tok.long(), self.dxd.double())
        assert rel(dx, x.grad) <= tol
        smoe.smoe_get_status(self.wp)
        smoe.smoe_get_status(self.ws)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,E,K,F", [(64, 128, 8, 2, 256), (300, 272, 24, 3, 144), (1024, 512, 4, 2, 384)])
def test_training_step(T, d, E, K, F, dt):
    c = Step(T, d, E, K, F, dt)
    c.forward()
    c.backward()
    c.check()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_captured_step_and_two_streams(dt):
    """Both passes replayed from a graph on new inputs, and two steps on two streams at once, each
    with its own workspaces, give the eager step's bits."""
    a, b = Step(300, 256, 12, 2, 272, dt), Step(280, 256, 12, 2, 272, dt, seed=5)
    want = []
    for c in (a, b):
        c.forward()
        c.backward()
        want.append([o.clone() for o in c.outputs()])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for c, s in zip((a, b), streams):
            for o in c.outputs():
                o.fill_(3.0)
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                c.forward()
                c.backward()
        torch.cuda.synchronize()
        for c, w in zip((a, b), want):
            for o, v in zip(c.outputs(), w):
                same(o, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.forward()
        a.backward()
    for o in a.outputs():
        o.fill_(3.0)
    graph.replay()
    for o, v in zip(a.outputs(), want[0]):
        same(o, v)
    a.x.copy_(a.x.flip(0))
    a.idx.copy_(a.idx.flip(0))
    graph.replay()
    got = [o.clone() for o in a.outputs()]
    a.forward()
    a.backward()
    for o, v in zip(a.outputs(), got):
        same(o, v)
    smoe.smoe_get_status(a.wp)


def test_f8_ffn_from_its_parts():
    """Tokens in 8 bits, gate and up products, SwiGLU to 8 bits, down product: the forward pass on
    8-bit weights, against 64 bits of the same quantised values."""
    T, d, E, K, F = 200, 384, 6, 2, 272
    up, down = F8Case(T, K, E, d, F, "bf16", "even"), F8Case(T, K, E, F, d, "bf16", "even")
    g, u = up.run(), None
    wq, sw = f8(randn(up.g, E, F, d) * 60), up.sw * 0.7
    u = up.out(F)
    smoe.smoe_expert_matmul_f8(up.desc, up.q, up.s, up.off, wq, sw, u, up.ws, row_src=up.src)
    h8 = torch.empty(T * K, F, dtype=F8, device="cuda")
    hs = torch.empty(T * K, blocks(F), device="cuda")
    smoe.smoe_swiglu_f8(up.desc, g, u, h8=h8, h8_scale=hs, pow2=0)
    y = down.out(d)
    smoe.smoe_expert_matmul_f8(down.desc, h8, hs, down.off, down.wq, down.sw, y, down.ws)
    h = h8.double() * spread(hs, F)
    ref, mag = torch.zeros(2, T * K, d, dtype=F64, device="cuda")
    for e, s in enumerate(down.seg):
        w = down.wq[e].double() * spread(down.sw[e].repeat_interleave(128, 0)[:d], F)
        ref[s], mag[s] = h[s] @ w.T, h[s].abs() @ w.abs().T
    down.check_rows(y, ref, mag, F / 32 + blocks(F) + 8)
    G, U = g.double(), u.double()
    hr = G * torch.sigmoid(G) * U
    within(h, hr, hr.abs() * (2.0 ** -4 + 2.0 ** -19) + spread(hs, F) * 2.0 ** -9)


def test_offsets_past_32_bits():
    """Rows and weights whose elements pass 2^31, and bytes 2^32."""
    d, T = 8192, 270000  # 2.2e9 elements of a matrix of rows
    desc = smoe.make_desc(T, d, 2, 1, 1, 16, 0, 1, 1, "bf16")
    g = gen(3)
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    q, s = torch.empty(T, d, dtype=F8, device="cuda"), torch.empty(T, blocks(d), device="cuda")
    smoe.smoe_rows_f8(desc, x, q, s, pow2=1)
    rows = torch.tensor([0, 1, 131071, 262143, 262144, T - 2, T - 1], device="cuda")
    rs, v = rows_ref(x[rows], 1)
    same(s[rows], rs)
    same(q[rows].view(torch.uint8), f8(v).view(torch.uint8))
    off = torch.tensor([0, 150001, T], dtype=torch.int32, device="cuda")
    w = (randn(g, 2, 16, d) / math.sqrt(d)).bfloat16()
    ws, y = smoe.workspace_products(desc), torch.empty(T, 16, dtype=torch.bfloat16, device="cuda")
    e = (rows >= 150001).long()
    smoe.smoe_expert_matmul(desc, x, off, w, y, ws)
    ref = torch.einsum("rd,rnd->rn", x[rows].double(), w[e].double())
    mag = torch.einsum("rd,rnd->rn", x[rows].double().abs(), w[e].double().abs())
    within(y[rows], ref, HALF["bf16"] * ref.abs() + adds16(d) * 2.0 ** -23 * mag)
    wq, sw = f8(randn(g, 2, 16, d) * 60), torch.rand(2, 1, blocks(d), generator=g, device="cuda") * 1e-3
    smoe.smoe_expert_matmul_f8(desc, q, s, off, wq, sw, y, ws)
    ww = wq.double() * spread(sw.expand(2, 16, -1), d)
    xx = q[rows].double() * spread(s[rows], d)
    ref = torch.einsum("rd,rnd->rn", xx, ww[e])
    mag = torch.einsum("rd,rnd->rn", xx.abs(), ww[e].abs())
    within(y[rows], ref, HALF["bf16"] * ref.abs() + (d / 32 + blocks(d) + 8) * 2.0 ** -23 * mag)
    dx = torch.empty_like(x)
    smoe.smoe_expert_matmul_dx(desc, y, w, off, dx, ws)
    ref = torch.einsum("rn,rnd->rd", y[rows].double(), w[e].double())
    mag = torch.einsum("rn,rnd->rd", y[rows].double().abs(), w[e].double().abs())
    within(dx[rows], ref, HALF["bf16"] * ref.abs() + adds16(16) * 2.0 ** -23 * mag)
    dw = torch.empty(2, 16, d, device="cuda")
    smoe.smoe_expert_matmul_dw(desc, y, x, off, dw, ws)
    got = dw.clone()
    for i, sl in enumerate((slice(0, 150001), slice(150001, T))):
        ref, mag = torch.zeros(2, 16, d, dtype=F64, device="cuda")
        for a in range(sl.start, sl.stop, 20000):
            b = min(a + 20000, sl.stop)
            ref += y[a:b].double().T @ x[a:b].double()
            mag += y[a:b].double().abs().T @ x[a:b].double().abs()
        # within a chunk of 1024 rows 64 additions of the tensor core, and the chunks' own
        n = 1024 / 16 + 150000 / 1024 + 24
        within(got[i], ref, n * 2.0 ** -23 * mag)
    smoe.smoe_expert_matmul_dw_f8(desc, y, q, s, off, dw, ws)
    h = torch.empty_like(x)
    smoe.smoe_swiglu_f8(desc, x, dx, h=h, g8=q, g8_scale=s, pow2=1)
    G, U = x[rows].double(), dx[rows].double()
    ref = G * torch.sigmoid(G) * U
    within(h[rows], ref, swiglu_tol("bf16") * ref.abs() + 1e-38)
    smoe.smoe_get_status(ws)


@pytest.mark.parametrize("rows", [5000, 40000])
def test_long_sums_do_not_drift(rows):
    """One expert with many rows: the error stays that of its chunks (1024 rows, 64 additions
    cut off at 24 bits: 64 x 2^-24 of the running sum on average) and of their rounded sum."""
    c = Case(rows, 1, 2, 128, 136, "bf16", "one")
    dy, x = c.rows(136), c.rows(128)
    dw = torch.empty(2, 136, 128, device="cuda")
    smoe.smoe_expert_matmul_dw(c.desc, dy, x, c.off, dw, c.ws)
    ref = dy.double().T @ x.double()
    assert float((dw[1].double() - ref).norm() / ref.norm()) <= 64 * 2.0 ** -24
    assert (dw[0] == 0).all()
    f = Case(rows, 1, 2, 128, 136, "f32", "one")
    dy, x = f.rows(136), f.rows(128)
    smoe.smoe_expert_matmul_dw(f.desc, dy, x, f.off, dw, f.ws)
    ref = dy.double().T @ x.double()
    assert float((dw[1].double() - ref).norm() / ref.norm()) <= 64 * 2.0 ** -24


def test_weight_gradient_wider_than_the_descriptor():
    """n_out above the descriptor's d and F: no room is kept for its planes, and none is needed."""
    T, E, n_in, n_out = 512, 2, 512, 1024
    c = Case(T, 1, E, n_in, n_out, "f32", "even")
    desc = smoe.make_desc(T, n_in, E, 1, 1, 64, 0, 1, 1, "f32")
    ws = smoe.workspace_products(desc)
    dy, x, w = c.rows(n_out), c.rows(n_in), c.weights()
    dw, out, dx = torch.empty(E, n_out, n_in, device="cuda"), c.out(n_out), c.out(n_in)
    smoe.smoe_expert_matmul_dw(desc, dy, x, c.off, dw, ws)
    smoe.smoe_expert_matmul(desc, x, c.off, w, out, ws)
    smoe.smoe_expert_matmul_dx(desc, dy, w, c.off, dx, ws)
    smoe.smoe_get_status(ws)
    for e, s in enumerate(c.seg):
        d = lambda a, b: (a.double() @ b.double(), a.double().abs() @ b.double().abs())  # noqa: E731
        for got, (ref, mag), n in ((dw[e], d(dy[s].T, x[s]), T), (out[s], d(x[s], w[e].T), n_in),
                                   (dx[s], d(dy[s], w[e]), n_out)):
            within(got, ref, adds1(n) * 2.0 ** -23 * mag)


def test_two_graphs_in_turn():
    """Two captured steps, each with its own workspaces, replayed in turn on one stream."""
    a, b = Step(200, 128, 6, 2, 144, "bf16"), Step(90, 128, 6, 2, 144, "f32", seed=3)
    want, graphs = [], []
    for c in (a, b):
        c.forward()
        c.backward()
        torch.cuda.synchronize()
        want.append([o.clone() for o in c.outputs()])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.forward()
            c.backward()
        graphs.append(g)
    for _ in range(3):
        for c in (a, b):
            for o in c.outputs():
                o.fill_(3.0)
        for g in graphs + graphs[::-1]:
            g.replay()
        for c, w in zip((a, b), want):
            for o, v in zip(c.outputs(), w):
                same(o, v)


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e30])
def test_fp32_products_over_the_range(scale):
    """Rows far from one: the planes of an fp32 operand keep its 24 bits (to 1e-33)."""
    c = Case(2048, 1, 4, 384, 264, "f32", "even", seed=6)
    x, dy, w = c.rows(384) * scale, c.rows(264) * scale, c.weights()
    x[::7] = x[::7].bfloat16().float()  # rows whose lower planes are zero
    out, dx, dw = c.out(264), c.out(384), torch.empty(4, 264, 384, device="cuda")
    smoe.smoe_expert_matmul(c.desc, x, c.off, w, out, c.ws)
    smoe.smoe_expert_matmul_dx(c.desc, dy, w, c.off, dx, c.ws)
    smoe.smoe_expert_matmul_dw(c.desc, dy / scale, x, c.off, dw, c.ws)
    smoe.smoe_get_status(c.ws)
    for e, s in enumerate(c.seg):
        d = lambda a, b: (a.double() @ b.double(), a.double().abs() @ b.double().abs())  # noqa: E731
        for got, (ref, mag) in ((out[s], d(x[s], w[e].T)), (dx[s], d(dy[s], w[e])), (dw[e], d((dy / scale)[s].T, x[s]))):
            # six products of planes, each with a dropped rest of 2^-24 of its term, and chunks of
            # 128 with 48 additions cut off at 24 bits
            within(got, ref, 64 * 2.0 ** -23 * mag)
            assert float((got.double() - ref).norm() / ref.norm()) <= 2e-6


# ------------------------------------------------------------------ long contractions in bf16
def dropped_terms(n, rows, cols):
    """Rows and weights whose exact products lie a little above the middle of two bf16 numbers:
    1 + 2^-8 - 2^-14 at the front and n - 16 terms of 2^-28 behind it, 2^-13.2 in all. Every one
    of those is below half a step of a running sum near 1, whether it is rounded or cut off, sixteen
    at once too. (rows, cols: powers of two that the rows and columns are scaled by.)"""
    x, w = torch.full((n,), 2.0 ** -14, device="cuda"), torch.full((n,), 2.0 ** -14, device="cuda")
    x[:16], w[:16] = 0.0, 0.0
    x[:3], w[:3] = torch.tensor([1.0, 2.0 ** -8, -2.0 ** -14], device="cuda"), 1.0
    return (rows[:, None] * x).bfloat16(), (cols[:, None] * w).bfloat16()


@pytest.mark.parametrize("T", [100, 300, 512])
def test_long_sums_keep_small_terms(T):
    """Products and row gradients over 28672 channels (100 rows: tiles of one SM; 300: a tile of 256
    and a remainder with its operands swapped; 512: whole tiles): a sum in one accumulator loses what
    lies behind its first terms, sums over chunks do not."""
    n, m = 28672, 264
    rows = 2.0 ** (torch.arange(T, device="cuda") % 5 - 2)
    cols = 2.0 ** (torch.arange(m, device="cuda") % 3)
    x, w = dropped_terms(n, rows, cols)
    want = (rows[:, None] * cols * (1 + 2.0 ** -7)).bfloat16()
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    desc = smoe.make_desc(T, n, 1, 1, 1, m, 0, 1, 1, "bf16")
    ws, out = smoe.workspace_products(desc), torch.full((T, m), 7.0, dtype=torch.bfloat16, device="cuda")
    smoe.smoe_expert_matmul(desc, x, off, w[None].contiguous(), out, ws)
    same(out, want)
    wt = w.T.contiguous()  # [n_out, n_in] of a gradient over n_out = n channels
    out.fill_(7.0)
    smoe.smoe_expert_matmul_dx(desc, x, wt[None], off, out, ws)
    same(out, want)
    out.fill_(7.0)
    h = n // 2
    smoe.smoe_expert_matmul_dx(desc, x[:, :h].contiguous(), wt[None, :h].contiguous(), off, out, ws,
                               dy2=x[:, h:].contiguous(), w2=wt[None, h:].contiguous())
    same(out, want)
    smoe.smoe_get_status(ws)


@pytest.mark.parametrize("T", [100, 300, 512])
def test_long_sums_are_not_biased(T):
    """Positive terms: 64 additions to a chunk of 1024, each cut off by about 2^-23 of a running sum
    that is half of the chunk's on average: about 2^-18 of the result, and as much again for cuts above
    one step and for the noise of the values that this moves across the middle of two bf16 numbers
    (2^-8 sqrt(2^-10 / N), N > 25000: below 2^-20). One accumulator over 28672 channels loses 2^-13."""
    n, m = 28672, 256
    g = gen(T)
    x = (torch.rand(T, n, generator=g, device="cuda") * (1 + torch.rand(T, 1, generator=g, device="cuda"))).bfloat16()
    w = (torch.rand(m, n, generator=g, device="cuda") * (1 + torch.rand(m, 1, generator=g, device="cuda"))).bfloat16()
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    desc = smoe.make_desc(T, n, 1, 1, 1, m, 0, 1, 1, "bf16")
    ws, out = smoe.workspace_products(desc), torch.empty(T, m, dtype=torch.bfloat16, device="cuda")
    ref = x.double() @ w.double().T
    near = ref.float().bfloat16().double()  # (the first rounding moves a value by 2^-24 at most)
    for call in (lambda: smoe.smoe_expert_matmul(desc, x, off, w[None], out, ws),
                 lambda: smoe.smoe_expert_matmul_dx(desc, x, w.T.contiguous()[None], off, out, ws)):
        call()
        assert float(((out.double() - near) / ref).mean().abs()) <= 2.0 ** -17
        within(out, ref, HALF["bf16"] * ref * (1 + 2.0 ** -8))


@pytest.mark.parametrize("T,K,E,n_in,n_out,kind", [
    (100, 1, 1, 4168, 136, "one"), (700, 2, 3, 2056, 1032, "skew"), (512, 1, 1, 1024, 2048, "one"),
    (64, 2, 6, 1032, 2056, "gaps"), (1024, 1, 2, 5128, 520, "even"), (450, 1, 1, 136, 9000, "one"),
])
def test_long_products(T, K, E, n_in, n_out, kind):
    """bf16 products and row gradients whose contractions end in, at and behind a chunk, both
    pairs' too: 64 additions a chunk, one more for each."""
    c = Case(T, K, E, n_in, n_out, "bf16", kind, seed=8)
    x, dy, w, dy2, w2 = c.rows(n_in), c.rows(n_out), c.weights(), c.rows(n_out), c.weights()
    for call, n, pairs, width in (
            (lambda o: smoe.smoe_expert_matmul(c.desc, x, c.off, w, o, c.ws), n_in, [(x, w.transpose(1, 2))], n_out),
            (lambda o: smoe.smoe_expert_matmul_dx(c.desc, dy, w, c.off, o, c.ws), n_out, [(dy, w)], n_in),
            (lambda o: smoe.smoe_expert_matmul_dx(c.desc, dy, w, c.off, o, c.ws, dy2=dy2, w2=w2), 2 * n_out,
             [(dy, w), (dy2, w2)], n_in)):
        out, again = c.out(width), c.out(width)
        call(out)
        ref, mag = torch.zeros(2, c.R, width, dtype=F64, device="cuda")
        for e, s in enumerate(c.seg):
            for a, b in pairs:
                ref[s] += a[s].double() @ b[e].double()
                mag[s] += a[s].double().abs() @ b[e].double().abs()
        c.check_rows(out, ref, mag, 64 + n / 1024 + 8)
        call(again)
        same(again, out)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [30, 600])
def test_bad_row_src_beside_weights_that_are_not_finite(T, dt):
    """An entry out of range gives a row of zeros whatever its expert's weights and scales are."""
    f = F8Case(T, 2, 4, 256, 264, dt, "even")
    o, keep = f.off.tolist(), f.src.clone()
    f.wq.view(torch.uint8)[0] = 0x7f       # NaN
    f.sw[1], f.sw[2] = math.inf, math.nan
    rows = [s for e in range(4) for s in (o[e], (o[e] + o[e + 1]) // 2, o[e + 1] - 1)]
    f.src[rows] = torch.tensor([-1, T, 1 << 30] * 4, dtype=torch.int32, device="cuda")
    out = f.run()
    with pytest.raises(smoe.SmoeError, match="SMOE_ERR_DATA"):
        smoe.smoe_get_status(f.ws)
    hit = f.src != keep
    assert int(hit.sum()) == 12 and (out[hit] == 0).all()
    assert not out[:o[3]][~hit[:o[3]]].isfinite().any() and out[o[3]:].isfinite().all()


# ------------------------------------------------------------------ products in fp32, not in fewer bits
# T, K, E, n_in, n_out, kind: few rows an expert (streamed weights), 64-row tiles, whole and
# in slices, planes on the tensor cores, whole and in slices
FP32_SHAPES = [
    (40, 2, 24, 1000, 1416, "skew"), (9, 1, 2, 1416, 200, "even"), (4096, 1, 1, 64, 512, "one"), (256, 2, 4, 264, 256, "skew"),
    (300, 1, 1, 1416, 136, "gaps"), (2048, 2, 4, 1000, 2056, "skew"), (512, 1, 4, 1032, 1000, "even"), (700, 1, 1, 1416, 264, "one"),
]


@pytest.mark.parametrize("T,K,E,n_in,n_out,kind", FP32_SHAPES)
def test_fp32_products_keep_24_bits(T, K, E, n_in, n_out, kind):
    """Relative error in the Frobenius norm. On the CUDA cores each of n additions is off by at most
    2^-24 of a running sum whose square grows evenly: 2^-24 sqrt(n / 2) of the result, below 2e-6 up to
    2200 additions in a row (a sum over 2 x 2056 is split over eight warps or slices). On the tensor cores
    chunks of 128: 48 additions, each cut off by half of 2^-23 on average of a running sum that is 2/3 of the
    chunk's, 1.9e-6. Operands of 11 bits (tf32) give 3e-4, without the three smallest plane products
    5e-6."""
    c = Case(T, K, E, n_in, n_out, "f32", kind, seed=12)
    x, dy, w, dy2, w2 = c.rows(n_in), c.rows(n_out), c.weights(), c.rows(n_out), c.weights()
    out, dx, dx2, dw = c.out(n_out), c.out(n_in), c.out(n_in), torch.empty(E, n_out, n_in, device="cuda")
    smoe.smoe_expert_matmul(c.desc, x, c.off, w, out, c.ws)
    smoe.smoe_expert_matmul_dx(c.desc, dy, w, c.off, dx, c.ws)
    smoe.smoe_expert_matmul_dx(c.desc, dy, w, c.off, dx2, c.ws, dy2=dy2, w2=w2)
    smoe.smoe_expert_matmul_dw(c.desc, dy, x, c.off, dw, c.ws)
    smoe.smoe_get_status(c.ws)
    refs = [torch.zeros_like(t, dtype=F64) for t in (out, dx, dx2, dw)]
    for e, s in enumerate(c.seg):
        refs[0][s] = x[s].double() @ w[e].double().T
        refs[1][s] = dy[s].double() @ w[e].double()
        refs[2][s] = refs[1][s] + dy2[s].double() @ w2[e].double()
        refs[3][e] = dy[s].double().T @ x[s].double()
    for got, ref in zip((out, dx, dx2), refs):
        assert (got[~c.inside] == 7).all()
        assert float((got.double() - ref)[c.inside].norm() / ref.norm()) <= 2e-6
    assert float((dw.double() - refs[3]).norm() / refs[3].norm()) <= 2e-6


@pytest.mark.parametrize("T", [60, 900])
def test_f8_token_whose_scale_is_nan(T):
    """The rows of a token with a NaN scale are NaN, and no others (rows of that token among them)."""
    c = F8Case(T, 1, 5, 272, 200, "f32", "skew", seed=9)
    o = c.off.tolist()
    c.src[c.src == 3] = 4
    c.src[[o[0], o[5] - 1, (o[0] + o[5]) // 2]] = 3
    clean = c.run()
    c.s[3, 1] = math.nan
    dirty = c.run()
    hit = (c.src == 3) & c.inside
    assert int(hit.sum()) == 3
    same(dirty[~hit], clean[~hit])
    assert dirty[hit].isnan().all()


def test_swiglu_far_from_zero():
    """bf16 layers take sig from a fast exponential that is off by (2 + 1.2 |g|) steps of 2^-23, and a
    division and sums off by two more: (4 + 1.2 |g|) 2^-23 of the result, beside its rounding. Below
    g = -87 sig is under 2^-126 and may be zero."""
    g = torch.linspace(-100, 100, 4096, device="cuda").bfloat16().view(32, 128)
    u, dh = torch.full_like(g, 0.75), torch.full_like(g, 1.5)
    q, s = [torch.empty(32, 128, dtype=F8, device="cuda") for _ in range(2)], [torch.empty(32, 1, device="cuda") for _ in range(2)]
    h, h2, dg, du = (torch.full_like(g, 7.0) for _ in range(4))
    smoe.smoe_swiglu_f8(rows_desc("bf16"), g, u, h=h, g8=q[0], g8_scale=s[0], u8=q[1], u8_scale=s[1])
    smoe.smoe_swiglu_grad_f8(rows_desc("bf16"), dh, q[0], s[0], q[1], s[1], dg, du, h=h2)
    err = lambda g: (4 + 1.2 * g.abs()) * 2.0 ** -23  # noqa: E731
    G, U, D = g.double(), u.double(), dh.double()
    ref = G * torch.sigmoid(G) * U
    within(h, ref, (HALF["bf16"] + err(G) + 2.0 ** -22) * ref.abs() + 2.0 ** -126 * (G * U).abs() + 1e-38)
    G, U = (a.double() * spread(b, 128) for a, b in zip(q, s))
    sig = torch.sigmoid(G)
    tiny = 2.0 ** -126 * (1 + (G * U * D).abs() + (G * D).abs()) * (1 + G.abs())
    within(h2, G * sig * U, (HALF["bf16"] + err(G) + 2.0 ** -22) * (G * sig * U).abs() + tiny)
    within(du, D * G * sig, (HALF["bf16"] + err(G) + 2.0 ** -22) * (D * G * sig).abs() + tiny)
    # 1 + g (1 - sig): its terms' errors are relative to them, and 1 - sig is off by a step of 1
    terms = (D * U * sig).abs() * (1 + G.abs() * (1 - sig))
    ref = D * U * sig * (1 + G * (1 - sig))
    within(dg, ref, HALF["bf16"] * ref.abs() + 2 * (err(G) + 2.0 ** -22) * terms + 2.0 ** -23 * (D * U * sig * G).abs() + tiny)


@pytest.mark.parametrize("T", [90, 700])
def test_long_products_captured_and_on_two_streams(T):
    """Contractions of several chunks on two streams at once, each with its own workspace, and replayed
    from a graph on new rows, give the eager calls' bits."""
    cases = [Case(T, 2, 2, 2568, 4104, "bf16", kind, seed=s) for kind, s in (("skew", 20), ("gaps", 21))]
    for c in cases:
        c.x, c.dy, c.w, c.dy2, c.w2 = c.rows(2568), c.rows(4104), c.weights(), c.rows(4104), c.weights()
        c.y, c.dx = c.out(4104), c.out(2568)

    def run(c):
        smoe.smoe_expert_matmul(c.desc, c.x, c.off, c.w, c.y, c.ws)
        smoe.smoe_expert_matmul_dx(c.desc, c.dy, c.w, c.off, c.dx, c.ws, dy2=c.dy2, w2=c.w2)

    want = []
    for c in cases:
        run(c)
        want.append((c.y.clone(), c.dx.clone()))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for c, s in zip(cases, streams):
            c.y.fill_(7.0)
            c.dx.fill_(7.0)
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                run(c)
        torch.cuda.synchronize()
        for c, (y, dx) in zip(cases, want):
            same(c.y, y)
            same(c.dx, dx)
    c = cases[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(c)
    for t in (c.x, c.dy, c.dy2):
        t.neg_()
    c.y.fill_(7.0)
    c.dx.fill_(7.0)
    graph.replay()
    for got, was in ((c.y, want[0][0]), (c.dx, want[0][1])):
        same(got[c.inside], -was[c.inside])
        assert (got[~c.inside] == 7.0).all()
    smoe.smoe_get_status(c.ws)
