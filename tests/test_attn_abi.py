"""Refusals of the attention calls, before the device is touched (no GPU: the
pointers are never followed)."""
import ctypes
import math

import pytest
import torch

import rank_latent_attention_flare_b200 as fl
from rank_latent_attention_flare_b200 import _lib

OK, INVALID, UNSUPPORTED, WORKSPACE, CUDA = 0, 1, 2, 3, 4
F = 0x7F0000000000
no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                                 reason="fake-pointer validation tests run on CPU-only hosts")


@pytest.fixture(scope="module")
def lib():
    from rank_latent_attention_flare_b200 import build
    build.build()
    return fl.load()


def strides(*triples):
    arr = (_lib.FlareStrides * len(triples))()
    for i, t in enumerate(triples):
        arr[i] = _lib.FlareStrides(*t)
    return arr


def attn_fwd(lib, B=2, Hq=4, Hk=2, Nq=30, Nk=50, D=64, dt=1, scale=0.125, q=F, k=F, v=F, y=F,
             st=None, ql=None, kl=None, lse=None, low=None, ws=F, wsb=None):
    if wsb is None:
        wsb = lib.flare_attn_workspace_size(0, B, Hq, Hk, Nq, Nk, D, dt) or (1 << 30)
    return lib.flare_attn_fwd(q, k, v, y, st, ql, kl, B, Hq, Hk, Nq, Nk, D, dt, scale, 0, lse,
                              low, ws, wsb, None)


def attn_bwd(lib, B=2, Hq=4, Hk=2, Nq=30, Nk=50, D=64, dt=1, scale=0.125, lse=F, dq=F, dk=F, dv=F,
             low=None, st=None, ws=F, wsb=None):
    if wsb is None:
        wsb = lib.flare_attn_workspace_size(1, B, Hq, Hk, Nq, Nk, D, dt) or (1 << 30)
    return lib.flare_attn_bwd(F, F, F, F, low, F, lse, dq, dk, dv, st, None, None, B, Hq, Hk, Nq,
                              Nk, D, dt, scale, 0, ws, wsb, None)


@no_gpu_only
@pytest.mark.parametrize("call", [attn_fwd, attn_bwd], ids=["fwd", "bwd"])
def test_attn_sizes(lib, call):
    assert call(lib) == CUDA                        # valid: fails only at the launch
    assert call(lib, dt=0) == CUDA
    for bad in (dict(B=0), dict(Hq=0), dict(Hk=0), dict(Nq=0), dict(Nk=-1), dict(D=0), dict(dt=2),
                dict(Hq=5), dict(B=1 << 21), dict(Hq=1 << 17, Hk=1)):
        assert call(lib, **bad) == INVALID, bad
    for s in (0.0, -1.0, math.nan, math.inf):
        assert call(lib, scale=s) == INVALID
    for bad in (dict(D=4), dict(D=20), dict(D=136), dict(Nk=(1 << 30) + 1),
                dict(B=1 << 20, Hq=32)):
        assert call(lib, **bad) == UNSUPPORTED, bad


@no_gpu_only
def test_attn_pointers_and_workspace(lib):
    for name in ("q", "k", "v", "y"):
        assert attn_fwd(lib, **{name: None}) == INVALID
        assert attn_fwd(lib, **{name: F + 8}) == INVALID
    assert attn_fwd(lib, lse=F + 4) == INVALID and attn_fwd(lib, low=F + 2) == INVALID
    assert attn_fwd(lib, low=F) == CUDA and attn_bwd(lib, low=F) == CUDA
    assert attn_bwd(lib, low=F + 8) == INVALID
    assert attn_fwd(lib, ql=F + 2) == INVALID and attn_fwd(lib, kl=F + 1) == INVALID
    assert attn_fwd(lib, ql=F + 4, kl=F + 8) == CUDA
    assert attn_bwd(lib, lse=None) == INVALID
    assert attn_bwd(lib, dq=None) == CUDA            # dk and dv alone
    assert attn_bwd(lib, dk=None, dv=None) == CUDA   # dq alone
    assert attn_bwd(lib, dk=None) == INVALID and attn_bwd(lib, dv=None) == INVALID
    assert attn_bwd(lib, dq=None, dk=None, dv=None) == INVALID
    for call, back in ((attn_fwd, 0), (attn_bwd, 1)):
        need = lib.flare_attn_workspace_size(back, 2, 4, 2, 30, 50, 64, 1)
        assert need > 0
        assert call(lib, wsb=need - 1) == WORKSPACE
        assert call(lib, ws=None) == WORKSPACE
        assert call(lib, ws=F + 16) == WORKSPACE
    assert lib.flare_attn_workspace_size(0, 2, 4, 3, 30, 50, 64, 1) == 0
    assert lib.flare_attn_workspace_size(1, 2, 4, 2, 30, 50, 60, 1) == 0


@no_gpu_only
def test_attn_strides(lib):
    q, k = (4 * 30 * 64, 30 * 64, 64), (2 * 50 * 64, 50 * 64, 64)
    tok = (30 * 4 * 64, 64, 4 * 64)
    assert attn_fwd(lib, st=strides(q, k, k, tok)) == CUDA
    assert attn_fwd(lib, st=strides((0, 0, 64), (0, 0, 64), (0, 50 * 64, 64), q)) == CUDA
    assert attn_fwd(lib, st=strides((0, 0, 0), k, k, q)) == INVALID      # all queries one row
    assert attn_fwd(lib, st=strides(q, (-64, 64, 64), k, q)) == INVALID
    assert attn_fwd(lib, st=strides(q, k, (50 * 64, 64, 68), q)) == UNSUPPORTED
    assert attn_fwd(lib, st=strides(q, k, k, (0, 30 * 64, 64))) == INVALID   # output rows coincide
    assert attn_fwd(lib, st=strides(q, k, k, (4 * 30 * 64, 29 * 64, 64))) == INVALID
    # a dimension of one entry has no stride
    assert attn_fwd(lib, Nq=1, st=strides((256, 64, 7), k, k, (256, 64, 3))) == CUDA
    back = [q, k, k, q, q, q, k, k]
    assert attn_bwd(lib, st=strides(*back)) == CUDA
    back[6] = (0, 50 * 64, 64)
    assert attn_bwd(lib, st=strides(*back)) == INVALID
    assert attn_bwd(lib, st=strides(*back), dk=None, dv=None) == CUDA    # dk is not written


def norm_fwd(lib, B=2, Hq=4, Hk=2, N=30, D=64, R=64, dt=1, eps=1e-6, q=F, k=F, wq=F, wk=F, cos=F,
             sin=F, sb=0, qo=F, ko=F, st=None):
    return lib.flare_qk_norm_rope_fwd(q, k, wq, wk, cos, sin, sb, qo, ko, st, B, Hq, Hk, N, D, R, 0,
                                      dt, eps, None)


def norm_bwd(lib, B=2, Hq=4, Hk=2, N=30, D=64, R=64, dt=1, eps=1e-6, cos=F, sin=F, sb=0, dq=F,
             dwq=F, ws=F, wsb=None, st=None):
    if wsb is None:
        wsb = lib.flare_qk_norm_rope_workspace_size(B, Hq, Hk, N, D, dt) or (1 << 30)
    return lib.flare_qk_norm_rope_bwd(F, F, F, F, cos, sin, sb, F, F, dq, F, dwq, F, st, B, Hq, Hk,
                                      N, D, R, 0, dt, eps, ws, wsb, None)


@no_gpu_only
@pytest.mark.parametrize("call", [norm_fwd, norm_bwd], ids=["fwd", "bwd"])
def test_norm_rope_sizes(lib, call):
    assert call(lib) == CUDA and call(lib, dt=0) == CUDA
    assert call(lib, Hq=5, Hk=3) == CUDA            # heads need not divide here
    for bad in (dict(B=0), dict(N=0), dict(Hq=0), dict(Hk=0), dict(D=0), dict(dt=7), dict(R=80),
                dict(R=-16), dict(eps=0.0), dict(eps=math.nan), dict(eps=-1.0), dict(cos=None),
                dict(sin=F + 4), dict(sb=10)):
        assert call(lib, **bad) == INVALID, bad
    for bad in (dict(D=136, R=0), dict(D=60, R=0), dict(R=8), dict(N=(1 << 30) + 1),
                dict(sb=30 * 32 + 2)):
        assert call(lib, **bad) == UNSUPPORTED, bad
    assert call(lib, R=0, cos=None, sin=None) == CUDA
    assert call(lib, sb=30 * 32) == CUDA


@no_gpu_only
def test_norm_rope_pointers(lib):
    for name in ("q", "k", "qo", "ko"):
        assert norm_fwd(lib, **{name: None}) == INVALID
    assert norm_fwd(lib, wq=None, wk=None) == CUDA
    assert norm_fwd(lib, wq=F + 2) == INVALID
    assert norm_bwd(lib, dq=None) == INVALID
    assert norm_bwd(lib, dwq=None) == CUDA
    need = lib.flare_qk_norm_rope_workspace_size(2, 4, 2, 30, 64, 1)
    assert need > 0 and norm_bwd(lib, wsb=need - 1) == WORKSPACE
    assert norm_bwd(lib, ws=F + 128) == WORKSPACE
    assert lib.flare_qk_norm_rope_workspace_size(2, 4, 2, 30, 62, 1) == 0
    q, k = (4 * 30 * 64, 30 * 64, 64), (2 * 30 * 64, 30 * 64, 64)
    assert norm_fwd(lib, st=strides(q, k, q, k)) == CUDA
    assert norm_fwd(lib, st=strides((0, 30 * 64, 64), k, q, k)) == CUDA
    assert norm_fwd(lib, st=strides(q, k, (0, 30 * 64, 64), k)) == INVALID
    assert norm_fwd(lib, st=strides(q, (2 * 30 * 64, 30 * 64, 66), q, k)) == UNSUPPORTED


def test_binding_refuses_host_tensors():
    x = torch.zeros(1, 2, 8, 16)
    for call in (lambda: fl.attn_fwd(x, x, x), lambda: fl.attn(x, x, x),
                 lambda: fl.attn_bwd(x, x, x, x, x, x[..., 0]),
                 lambda: fl.qk_norm_rope_fwd(x, x), lambda: fl.qk_norm_rope(x, x)):
        with pytest.raises(ValueError):
            call()


def test_signatures_take_integers(lib):
    assert ctypes.sizeof(ctypes.c_size_t) == 8
    assert lib.flare_attn_workspace_size(0, 1, 1, 1, 1, 1, 8, 0) > 0


@pytest.mark.gpu
def test_binding_refuses_wrong_shapes():
    """Checks of the binding and of the library that need device tensors."""
    q, k = torch.zeros(2, 4, 5, 16, device="cuda"), torch.zeros(2, 3, 6, 16, device="cuda")
    with pytest.raises(ValueError):
        fl.attn_fwd(q, k, k)                                    # 4 heads over 3
    k = torch.zeros(2, 2, 6, 16, device="cuda")
    with pytest.raises(ValueError):
        fl.attn_fwd(q, k, k[:, :, :5])
    with pytest.raises(ValueError):
        fl.attn_fwd(q, k, k.double())
    with pytest.raises(TypeError):
        fl.attn_fwd(q.half(), k.half(), k.half())
    with pytest.raises(ValueError):
        fl.attn_fwd(q, k, k, k_lens=torch.tensor([6, 6], device="cuda"))   # int64
    with pytest.raises(fl.FlareError):
        fl.attn_fwd(q[..., :12], k[..., :12], k[..., :12])
    with pytest.raises(ValueError):
        fl.qk_norm_rope_fwd(q, k)                               # 5 and 6 tokens
    with pytest.raises(ValueError):
        fl.qk_norm_rope_fwd(q, q, torch.ones(8, device="cuda"))
    with pytest.raises(ValueError):
        fl.qk_norm_rope_fwd(q, q, None, None, torch.zeros(5, 8, device="cuda"))
    with pytest.raises(ValueError):
        fl.qk_norm_rope_fwd(q, q, None, None, torch.zeros(4, 8, device="cuda"),
                            torch.zeros(4, 8, device="cuda"))
