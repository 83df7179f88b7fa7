"""Cross and shared-prefix attention without a GPU: refusals on the host, before any launch, and the
64-bit reference and its bounds against differences and a simulated bf16 kernel (CPU only)."""
import ctypes

import pytest
import torch

import dense_ref
from block_sparse_spherical_b200 import abi, api, build

A = 4096          # an address that is never used: validation comes first


@pytest.fixture(scope="module")
def lib():
    build.build()
    return abi.load()


def cross_cfg(**over):
    c = abi.BsaCrossConfig(2, 8, 4, 100, 300, 64, abi.BSA_BF16, 0.0)
    for k, v in over.items():
        setattr(c, k, v)
    return c


def prefix_cfg(**over):
    c = abi.BsaPrefixConfig(6, 2, 8, 4, 3, 300, 40, 64, abi.BSA_BF16, 0.0)
    for k, v in over.items():
        setattr(c, k, v)
    return c


COMMON = [(dict(batch=0), 1), (dict(heads=0), 1), (dict(kv_heads=0), 1), (dict(kv_heads=3), 1), (dict(n_q=0), 1),
          (dict(head_dim=0), 1), (dict(dtype=9), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
          (dict(scale=float("inf")), 1), (dict(dtype=0), 2), (dict(head_dim=32), 2), (dict(head_dim=96), 2),
          (dict(n_q=2147483647), 2)]


@pytest.mark.parametrize("over,code", COMMON + [(dict(n_k=0), 1), (dict(n_k=2147483647), 2)])
def test_cross_config_refusals(lib, over, code):
    n = ctypes.c_size_t(0)
    c = ctypes.byref(cross_cfg(**over))
    assert lib.bsa_cross_workspace_size(c, ctypes.byref(n)) == code
    assert lib.bsa_cross_backward_workspace_size(c, ctypes.byref(n)) == code
    assert lib.bsa_cross_attention(c, A, 2 * A, 3 * A, None, 4 * A, None, None, A, 1 << 40, None, None) == code


@pytest.mark.parametrize("over,code", COMMON + [(dict(n_prefix=0), 1), (dict(n_own=0), 1), (dict(groups=0), 1),
                                                (dict(groups=4), 1), (dict(n_own=2147483647), 2)])
def test_prefix_config_refusals(lib, over, code):
    n = ctypes.c_size_t(0)
    c = ctypes.byref(prefix_cfg(**over))
    assert lib.bsa_prefix_workspace_size(c, ctypes.byref(n)) == code
    assert lib.bsa_prefix_attention(c, A, 2 * A, 3 * A, None, 4 * A, 5 * A, None, 6 * A, A, 1 << 40, None,
                                    None) == code


def test_cross_pointer_refusals(lib):
    c = ctypes.byref(cross_cfg())
    ok = [A, 2 * A, 3 * A, None, 4 * A, None, None]
    call = lambda a, ws=A, n=1 << 40, st=None: lib.bsa_cross_attention(c, *a, ws, n, st, None)
    for i in (0, 1, 2, 4):                                   # q, k, v, out
        assert call(ok[:i] + [None] + ok[i + 1:]) == 1
        assert call(ok[:i] + [ok[i] + 8] + ok[i + 1:]) == 3
    assert call(ok[:3] + [A + 2] + ok[4:]) == 3 and call(ok[:5] + [A + 2, None]) == 3 and call(ok[:6] + [A + 8]) == 3 and call(ok, st=A + 1) == 3
    assert call(ok[:4] + [A, None, None]) == 1               # out is q
    assert call(ok[:6] + [4 * A]) == 1 and call(ok[:6] + [2 * A]) == 1   # out_low is out, k
    assert lib.bsa_cross_workspace_size(c, None) == 1 and lib.bsa_cross_workspace_size(None, None) == 1


def test_backward_pointer_refusals(lib):
    c = ctypes.byref(cross_cfg())
    ok = [A, 2 * A, 3 * A, None, 4 * A, 5 * A, 10 * A, 6 * A, 7 * A, 8 * A, 9 * A]   # q k v len out lse low dout dq dk dv
    call = lambda a, ws=A, n=1 << 40: lib.bsa_cross_attention_backward(c, *a, ws, n, None, None)
    for i in (0, 1, 2, 4, 5, 7, 8, 9, 10):
        assert call(ok[:i] + [None] + ok[i + 1:]) == 1
    for i in (0, 1, 2, 4, 6, 7, 8, 9, 10):
        assert call(ok[:i] + [ok[i] + 8] + ok[i + 1:]) == 3
    assert call(ok[:8] + [8 * A, 8 * A, 9 * A]) == 1         # dq is dk
    assert call(ok[:10] + [6 * A]) == 1                      # dv is dout
    assert call(ok[:10] + [10 * A]) == 1                     # dv is out_low


def test_prefix_pointer_refusals(lib):
    c = ctypes.byref(prefix_cfg())
    ok = [A, 2 * A, 3 * A, None, 4 * A, 5 * A, None, 6 * A]  # q kp vp len ko vo len out
    call = lambda a, st=None: lib.bsa_prefix_attention(c, *a, A, 1 << 40, st, None)
    for i in (0, 1, 2, 4, 5, 7):
        assert call(ok[:i] + [None] + ok[i + 1:]) == 1
        assert call(ok[:i] + [ok[i] + 8] + ok[i + 1:]) == 3
    assert call(ok[:7] + [A]) == 1 and call(ok, st=A + 1) == 3


def test_workspace_refusals(lib):
    """Sizes whose key axis is split need a workspace, of the stated size and alignment."""
    n = ctypes.c_size_t(0)
    c = ctypes.byref(cross_cfg(batch=1, heads=1, kv_heads=1, n_q=1, n_k=100000))
    args = [A, 2 * A, 3 * A, None, 4 * A, None, None]
    assert lib.bsa_cross_workspace_size(c, ctypes.byref(n)) == 0
    if n.value:
        assert lib.bsa_cross_attention(c, *args, None, n.value, None, None) == 6
        assert lib.bsa_cross_attention(c, *args, A, n.value - 1, None, None) == 6
        assert lib.bsa_cross_attention(c, *args, A + 16, n.value, None, None) == 3
    c = ctypes.byref(prefix_cfg())
    args = [A, 2 * A, 3 * A, None, 4 * A, 5 * A, None, 6 * A]
    assert lib.bsa_prefix_workspace_size(c, ctypes.byref(n)) == 0
    if n.value:
        assert lib.bsa_prefix_attention(c, *args, None, n.value, None, None) == 6
        assert lib.bsa_prefix_attention(c, *args, A, n.value - 1, None, None) == 6
        assert lib.bsa_prefix_attention(c, *args, A + 16, n.value, None, None) == 3


def test_layers_need_a_gpu_and_a_known_dtype():
    with pytest.raises(TypeError):
        api.CrossAttention(1, 1, 1, 1, 64, dtype=torch.float16, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        api.CrossAttention(1, 1, 1, 1, 64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        api.PrefixAttention(2, 1, 1, 1, 1, 64, device="cpu")


def test_reference_gradients_are_differences():
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)
    q, k, v, g = r(2, 4, 3, 8), r(2, 2, 5, 8), r(2, 2, 5, 8), r(2, 4, 3, 8)
    lens = [5, 2]
    ref = dense_ref.cross(q, k, v, lens, dout=g)
    f = lambda: float((dense_ref.cross(q, k, v, lens)["out"] * g).sum())
    for x, grad in ((q, ref["dq"]), (k, ref["dk"]), (v, ref["dv"])):
        for i in torch.randperm(x.numel(), generator=gen)[:24].tolist():
            at, h = x.view(-1), 1e-5
            x0 = float(at[i])
            at[i] = x0 + h
            up = f()
            at[i] = x0 - h
            diff = (up - f()) / (2 * h)
            at[i] = x0
            assert abs(diff - float(grad.reshape(-1)[i])) <= 1e-8


def test_bounds_hold_for_a_simulated_kernel_and_catch_mistakes():
    """bf16 roundings where the kernel makes them stay inside the bounds; a dropped key, an
    unscaled gradient and a missing D do not."""
    gen = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16)
    q, k, v, g = r(1, 1, 40, 64), r(1, 1, 70, 64), r(1, 1, 70, 64), r(1, 1, 40, 64)
    ref = dense_ref.cross(q, k, v, dout=g)
    bf = lambda x: x.to(torch.bfloat16).float()
    qf, kf, vf, gf = (x.float()[0, 0] for x in (q, k, v, g))
    s = qf @ kf.T / 8
    m = s.amax(-1, keepdim=True)
    w = torch.exp(s - m)
    z = w.sum(-1, keepdim=True)
    exact = bf(w) @ vf / z
    out = bf(exact)
    p = w / z
    dterm = (gf * (out + bf(exact - out))).sum(-1, keepdim=True)
    full = p * (gf @ vf.T - dterm)
    ds = bf(full)
    got = dict(out=out, dv=bf(bf(p).T @ gf), dq=bf((ds + bf(full - ds)) @ kf / 8), dk=bf(ds.T @ qf / 8))
    for name, x in got.items():
        dense_ref.check(x[None, None], ref, name)
    wrong = dict(out=bf(bf(w[:, 1:]) @ vf[1:] / z), dq=bf(ds @ kf), dk=bf(bf(p * (gf @ vf.T)).T @ qf / 8))
    for name, x in wrong.items():
        with pytest.raises(AssertionError):
            dense_ref.check(x[None, None], ref, name)
