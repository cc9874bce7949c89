"""The product, gradient and 8-bit row entry points refuse bad arguments on the host, before any
CUDA call."""
import ctypes

import pytest

from routing_token_shuffle_gb300 import binding as B
from routing_token_shuffle_gb300 import build as build_mod


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.lib()


def desc(**kw):
    d = dict(T=16, d=128, E=8, K=2, H=1, F=256, n_shared=0, P=1, vocab=1, dtype="bf16")
    d.update(kw)
    return B.make_desc(**d)


def ref(d):
    return ctypes.byref(d)


# name, pointer arguments in order (True: required)
PRODUCTS = {
    "smoe_expert_matmul_f8": ((1, 1, 0, 1, 1, 1, 1), 16),  # xq, x_scale, row_src, off, wq, w_scale, out
    "smoe_expert_matmul": ((1, 1, 1, 1), 8),               # x, off, w, out
    "smoe_expert_matmul_dx": ((1, 1, 0, 0, 1, 1), 8),      # dy, w, dy2, w2, off, dx
    "smoe_expert_matmul_dw": ((1, 1, 1, 0, 1), 8),         # dy, x, off, add, dw
    "smoe_expert_matmul_dw_f8": ((1, 1, 1, 0, 1, 0, 1), 16),  # dy, xq, x_scale, row_src, off, add, dw
}


@pytest.mark.parametrize("name", PRODUCTS)
def test_product_refusals(lib, name):
    f, (need, step) = getattr(lib, name), PRODUCTS[name]
    d = desc()
    n = lib.smoe_product_workspace_size(ref(d))
    assert n >= 256
    ok = [16] * len(need)
    for k, required in enumerate(need):
        a = list(ok)
        a[k] = 16 + 8
        assert f(ref(d), 256, 128, *a, 256, n, None) == -3, k
        if required:
            a[k] = None
            assert f(ref(d), 256, 128, *a, 256, n, None) == -1, k
    for n_out, n_in in ((256, 0), (256, -16), (256, 4), (256, 128 + step // 2), (0, 128), (12, 128),
                        (-8, 128), (1 << 30, 128), (1 << 27, 1 << 20)):
        assert f(ref(d), n_out, n_in, *ok, 256, n, None) == -2, (n_out, n_in)
    assert f(None, 256, 128, *ok, 256, n, None) == -1
    assert f(ref(d), 256, 128, *ok, None, n, None) == -4
    assert f(ref(d), 256, 128, *ok, 256, n - 1, None) == -4
    assert f(ref(d), 256, 128, *ok, 256 + 16, n, None) == -3
    bad = desc(K=9)
    assert lib.smoe_product_workspace_size(ref(bad)) == 0
    assert f(ref(bad), 256, 128, *ok, 256, n, None) == -2


def test_second_pair_goes_together(lib):
    f, d = lib.smoe_expert_matmul_dx, desc()
    n = lib.smoe_product_workspace_size(ref(d))
    assert f(ref(d), 256, 128, 16, 16, 16, None, 16, 16, 256, n, None) == -1
    assert f(ref(d), 256, 128, 16, 16, None, 16, 16, 16, 256, n, None) == -1
    assert b"go together" in lib.smoe_last_error()


def test_kept_rows_fit_the_workspace(lib):
    f, d = lib.smoe_expert_matmul_dw_f8, desc()
    n = lib.smoe_product_workspace_size(ref(d))
    assert f(ref(d), 256, 272, 16, 16, 16, None, 16, None, 16, 256, n, None) == -2
    assert b"max(d, F)" in lib.smoe_last_error()


def test_product_workspace_holds_the_widened_rows(lib):
    size = lambda **kw: lib.smoe_product_workspace_size(ref(desc(**kw)))  # noqa: E731
    assert size(T=32) - size(T=16) == 16 * 2 * 256 * 2
    # fp32: rows of twice the size, and three bf16 planes of either operand of a weight gradient
    assert size(dtype="f32") - size() == 16 * 2 * 256 * (2 + 2 * 6)
    assert size(T=0) > 0


def test_rows_f8_refusals(lib):
    f, d = lib.smoe_rows_f8, desc()  # desc, rows, cols, x, pow2, q, scale, stream
    assert f(None, 4, 128, 16, 0, 16, 16, None) == -1
    for k in range(3):
        a = [16, 16, 16]
        a[k] = None
        assert f(ref(d), 4, 128, a[0], 0, a[1], a[2], None) == -1
        a[k] = 24
        assert f(ref(d), 4, 128, a[0], 0, a[1], a[2], None) == -3
    for rows, cols in ((-1, 128), (4, 0), (4, 12), (4, -8), (1 << 30, 256)):
        assert f(ref(d), rows, cols, 16, 0, 16, 16, None) == -2
    for pow2 in (-1, 2):
        assert f(ref(d), 4, 128, 16, pow2, 16, 16, None) == -1
    assert f(ref(d), 0, 128, 16, 0, 16, 16, None) == 0


def test_swiglu_refusals(lib):
    f, d = lib.smoe_swiglu_f8, desc()  # desc, rows, cols, g, u, pow2, h, h8, hs, g8, gs, u8, us, stream
    ok = [16, 16, 1] + [16] * 7
    for k in (0, 1):
        a = list(ok)
        a[k] = None
        assert f(ref(d), 4, 128, *a, None) == -1
    for k in (0, 1, 3, 4, 5, 6, 7, 8, 9):
        a = list(ok)
        a[k] = 24
        assert f(ref(d), 4, 128, *a, None) == -3
    for k in (4, 5, 6, 7, 8, 9):
        a = list(ok)
        a[k] = None
        assert f(ref(d), 4, 128, *a, None) == -1 and b"go together" in lib.smoe_last_error()
    assert f(ref(d), 4, 128, 16, 16, 1, *[None] * 7, None) == -1
    assert f(ref(d), 4, 128, 16, 16, 2, *ok[3:], None) == -1
    assert f(ref(d), 4, 100, *ok, None) == -2
    assert f(ref(d), 0, 128, *ok, None) == 0


def test_swiglu_grad_refusals(lib):
    f, d = lib.smoe_swiglu_grad_f8, desc()  # desc, rows, cols, dh, g8, gs, u8, us, dg, du, h, stream
    ok = [16] * 8
    for k in range(8):
        a = list(ok)
        a[k] = 24
        assert f(ref(d), 4, 128, *a, None) == -3
        if k < 7:
            a[k] = None
            assert f(ref(d), 4, 128, *a, None) == -1
    assert f(ref(d), 4, 100, *ok, None) == -2
    assert f(ref(d), 0, 128, *ok, None) == 0


def test_binding_refuses_other_shapes(lib):
    import torch
    z, w = torch.zeros(16), torch.zeros(7, 16, 16)
    with pytest.raises(ValueError, match="7 experts"):
        B.smoe_expert_matmul(desc(), z, z, w, z, z, stream=0)
    with pytest.raises(ValueError, match="not contiguous"):
        B.smoe_expert_matmul(desc(), z, z, torch.zeros(8, 16, 32).transpose(1, 2), z, z, stream=0)
    with pytest.raises(ValueError, match="w2 has shape"):
        B.smoe_expert_matmul_dx(desc(), z, torch.zeros(8, 16, 16), z, z, z, dy2=z, w2=torch.zeros(8, 16, 8),
                                stream=0)
    with pytest.raises(ValueError, match="add has shape"):
        B.smoe_expert_matmul_dw(desc(), z, z, z, torch.zeros(8, 16, 16), z, add=w, stream=0)
    with pytest.raises(ValueError, match="u8 has shape"):
        B.smoe_swiglu_f8(desc(), torch.zeros(2, 16), torch.zeros(2, 16), u8=z, u8_scale=z, stream=0)


def test_binding_refuses_buffers_that_are_too_small(lib):
    """Each buffer's type and room, before any call: a call of [T K] = 32 rows on 8 experts of 256 x 128."""
    import torch
    bf, f4, f8, i4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32
    z = lambda t, *s: torch.zeros(*s, dtype=t)  # noqa: E731
    d, R = desc(), 32
    ws = z(torch.uint8, 16)
    w, w8, off, src = z(bf, 8, 256, 128), z(f8, 8, 256, 128), z(i4, 9), z(i4, R)
    x, y, dw = z(bf, R, 128), z(bf, R, 256), z(f4, 8, 256, 128)
    x8, xs, wsc = z(f8, 16, 128), z(f4, 16, 1), z(f4, 8, 2, 1)
    g, g8, gs = z(bf, R, 136), z(f8, R, 136), z(f4, R, 2)
    calls = {
        B.smoe_rows_f8: dict(x=g, q=g8, scale=gs),
        B.smoe_expert_matmul_f8: dict(xq=x8, x_scale=xs, expert_off=off, wq=w8, w_scale=wsc, out=y, row_src=src),
        B.smoe_expert_matmul: dict(x=x, expert_off=off, w=w, out=y),
        B.smoe_expert_matmul_dx: dict(dy=y, w=w, expert_off=off, dx=x, dy2=y, w2=w),
        B.smoe_expert_matmul_dw: dict(dy=y, x=x, expert_off=off, dw=dw, add=dw),
        B.smoe_expert_matmul_dw_f8: dict(dy=y, xq=x8, x_scale=xs, expert_off=off, dw=dw, row_src=src, add=dw),
        B.smoe_swiglu_f8: dict(g=g, u=g, h=g, h8=g8, h8_scale=gs, g8=g8, g8_scale=gs, u8=g8, u8_scale=gs),
        B.smoe_swiglu_grad_f8: dict(dh=g, g8=g8, g8_scale=gs, u8=g8, u8_scale=gs, dg=g, du=g, h=g),
    }
    for f, kw in calls.items():
        more = {} if "swiglu" in f.__name__ or "rows" in f.__name__ else dict(ws=ws)
        # whole buffers pass the binding: the C side refuses the workspace, or goes on to the device
        if more:
            with pytest.raises(B.SmoeError, match="workspace"):
                f(d, **kw, **more, stream=0)
        for name, t in kw.items():
            short = t.reshape(-1)[:-1] if t.dim() == 1 else t[:-1]
            other = t.to({bf: f4, f4: bf, f8: bf, i4: torch.int64}[t.dtype])
            for bad in (short, other):
                with pytest.raises(ValueError, match="has shape|holds 7 experts"):
                    f(d, **{**kw, name: bad}, **more, stream=0)
    # longer buffers are taken, as of a larger batch; matrices that are another's transpose are not
    with pytest.raises(B.SmoeError):
        B.smoe_expert_matmul(d, z(bf, 40, 128), z(i4, 12), w, z(bf, 40, 256), ws, stream=0)
    with pytest.raises(ValueError, match="w2 has shape"):
        B.smoe_expert_matmul_dx(d, y, w, off, x, ws, dy2=y, w2=z(bf, 8, 128, 256), stream=0)
    with pytest.raises(ValueError, match="add has shape"):
        B.smoe_expert_matmul_dw(d, y, x, off, dw, ws, add=z(f4, 8, 128, 256), stream=0)
    # rows in dispatched order, not token rows
    with pytest.raises(ValueError, match="xq has shape"):
        B.smoe_expert_matmul_f8(d, x8, z(f4, R, 1), off, w8, wsc, y, ws, stream=0)
    with pytest.raises(ValueError, match="x_scale has shape"):
        B.smoe_expert_matmul_dw_f8(d, y, z(f8, R, 128), xs, off, dw, ws, stream=0)
