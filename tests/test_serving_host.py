"""The serving entry points refuse bad arguments on the host, before any CUDA call."""
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


def test_norm_refusals(lib):
    f = lib.smoe_add_rmsnorm   # desc, r, y, gamma, eps, r_out, x_out, q_out, q_scale, stream
    d = desc()
    assert f(None, 16, None, 16, 1e-6, 16, None, None, None, None) == -1
    assert f(ref(d), None, None, 16, 1e-6, 16, None, None, None, None) == -1
    assert f(ref(d), 16, None, None, 1e-6, 16, None, None, None, None) == -1
    assert f(ref(d), 16, None, 16, 1e-6, None, None, None, None, None) == -1    # no output
    assert f(ref(d), 16, None, 16, 1e-6, None, None, 16, None, None) == -1      # q without scale
    assert f(ref(d), 16, None, 16, 1e-6, 16, None, None, 16, None) == -1        # scale without q
    assert f(ref(d), 16, None, 16, -1.0, 16, None, None, None, None) == -1
    assert f(ref(d), 16, None, 16, float("nan"), 16, None, None, None, None) == -1
    for k in range(7):                                                          # alignment
        a = [16, 16, 16, 16, 16, 16, 16]
        a[k] = 16 + 8
        assert f(ref(d), a[0], a[1], a[2], 1e-6, a[3], a[4], a[5], a[6], None) == -3
    assert f(ref(desc(d=16392)), 16, None, 16, 1e-6, 16, None, None, None, None) == -2
    assert b"16384" in lib.smoe_last_error()
    assert f(ref(desc(d=100)), 16, None, 16, 1e-6, 16, None, None, None, None) == -2
    assert f(ref(desc(T=0)), 16, None, 16, 1e-6, 16, None, None, None, None) == 0


def test_few_refusals(lib):
    f = lib.smoe_moe_forward_few  # desc, x, w_gate, w1, w3, w2, y, logits, idx, w, ws, bytes, stream
    d = desc()
    n = lib.smoe_few_workspace_size(ref(d))
    assert n > 0
    ok = [16] * 6 + [None] * 3
    for k in range(6):
        a = list(ok)
        a[k] = None
        assert f(ref(d), *a, 256, n, None) == -1
    for k in range(9):
        a = list(ok)
        a[k] = 16 + 4
        assert f(ref(d), *a, 256, n, None) == -3
    assert f(ref(d), *ok, None, n, None) == -4
    assert f(ref(d), *ok, 256, n - 1, None) == -4
    assert f(ref(d), *ok, 256 + 16, n, None) == -3
    big = desc(T=65)
    assert lib.smoe_few_workspace_size(ref(big)) == 0
    assert f(ref(big), *ok, 256, n, None) == -2 and b"64" in lib.smoe_last_error()
    assert lib.smoe_few_workspace_size(ref(desc(T=64))) > 0
    assert f(ref(desc(E=512, F=1 << 23, d=8)), *ok, 256, 1 << 60, None) == -2
    with pytest.raises(B.SmoeError):
        B.workspace_few(big, device="cpu")


def test_few_workspace_grows_with_the_batch(lib):
    sizes = [lib.smoe_few_workspace_size(ref(desc(T=t, E=64, K=4))) for t in (1, 2, 16, 17, 64)]
    assert sizes == sorted(sizes)


def test_matmul_i8_refusals(lib):
    f = lib.smoe_expert_matmul_i8  # desc, n_out, n_in, xq, xs, src, off, wq, sw, out, ws, bytes, stream
    d = desc()
    n = lib.smoe_i8_workspace_size(ref(d))
    ok = [16, 16, None, 16, 16, 16, 16]
    for k in (0, 1, 3, 4, 5, 6):
        a = list(ok)
        a[k] = None
        assert f(ref(d), 256, 128, *a, 256, n, None) == -1
    for k in range(7):
        a = list(ok)
        a[k] = 16 + 4
        assert f(ref(d), 256, 128, *a, 256, n, None) == -3
    for n_out, n_in in ((256, 0), (256, -16), (256, 120), (256, 272), (0, 128), (12, 128), (-8, 128),
                        (1 << 30, 128)):
        assert f(ref(d), n_out, n_in, *ok, 256, n, None) == -2, (n_out, n_in)
    assert f(ref(d), 256, 128, *ok, None, n, None) == -4
    assert f(ref(d), 256, 128, *ok, 256, n - 1, None) == -4
    assert lib.smoe_i8_workspace_size(ref(desc(K=9))) == 0


def test_ffn_i8_refusals(lib):
    f = lib.smoe_expert_ffn_i8  # desc, xq, xs, src, off, weights, y, y_sh, ws, bytes, stream
    d = desc(n_shared=1)
    n = lib.smoe_i8_workspace_size(ref(d))
    W = lambda **kw: ctypes.byref(B.I8Weights(**{**{k: 16 for k in ("w1", "s1", "w3", "s3", "w2", "s2")}, **kw}))  # noqa: E731
    ok = [16, 16, 16, 16]
    for k in range(4):
        a = list(ok)
        a[k] = None  # row_src (k = 2) is needed with shared experts
        assert f(ref(d), *a, W(), 16, 16, 256, n, None) == -1
    assert f(ref(d), *ok, None, 16, 16, 256, n, None) == -1
    assert f(ref(d), *ok, W(), None, 16, 256, n, None) == -1
    assert f(ref(d), *ok, W(), 16, None, 256, n, None) == -1
    for k in ("w1", "s1", "w3", "s3", "w2", "s2"):
        assert f(ref(d), *ok, W(**{k: None}), 16, 16, 256, n, None) == -1
        assert f(ref(d), *ok, W(**{k: 20}), 16, 16, 256, n, None) == -3
    assert f(ref(d), *ok, W(), 16, 16, 256, n - 1, None) == -4
    assert f(ref(desc(d=136)), *ok, W(), 16, 16, 256, 1 << 40, None) == -2
    assert f(ref(desc(F=264)), *ok, W(), 16, 16, 256, 1 << 40, None) == -2


def test_binding_refuses_strided_rows(lib):
    import torch
    d = desc()
    with pytest.raises(ValueError, match="not contiguous"):
        B.smoe_add_rmsnorm(d, torch.zeros(16, 256)[:, ::2], torch.ones(128), r_out=torch.zeros(16, 128),
                           stream=0)
    with pytest.raises(ValueError, match="not contiguous"):
        B.smoe_moe_forward_few(d, torch.zeros(128, 16).t(), *[torch.zeros(1)] * 6, stream=0)
    with pytest.raises(ValueError, match="not contiguous"):
        B.i8_weights(torch.zeros(8, 128, 256).transpose(1, 2), *[torch.zeros(8, 256)] * 5)


def test_binding_refuses_weights_of_another_expert_count(lib):
    import torch
    z = torch.zeros(16)
    with pytest.raises(ValueError, match="7 experts"):
        B.smoe_expert_matmul_i8(desc(), z, z, z, torch.zeros(7, 16, 16, dtype=torch.int8), z, z, z, stream=0)


def test_norm_eps_is_at_most_one(lib):
    f, d = lib.smoe_add_rmsnorm, desc(T=0)
    for eps, code in ((0.0, 0), (1.0, 0), (1.5, -1), (float("inf"), -1)):
        assert f(ref(d), 16, None, 16, eps, 16, None, None, None, None) == code, eps
