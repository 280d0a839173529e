"""Refusals of the token-major entry points (layer norm, gated delta rule) on
a machine without a GPU: checked on the host, nothing is launched."""
import ctypes

import pytest

from structured_state_space_dplr_b200 import _lib
from structured_state_space_dplr_b200 import build as s4build

FAKE = 0x7f0000000000          # 256-byte aligned, never dereferenced
FAKE2 = 0x7f1000000000


@pytest.fixture(scope="module")
def lib():
    s4build.build()
    return _lib.lib()


def p(v):
    return ctypes.c_void_p(v)


def test_norm_entries_reject_bad_arguments(lib):
    x, ga, be, z, mu, rs, ws = (p(FAKE + 0x1000000 * i) for i in range(7))
    eps = ctypes.c_float(1e-5)
    f = lambda dt=0, x=x, ga=ga, eps=eps, rows=8, D=64, z=z, mu=mu: lib.s4_layernorm(  # noqa: E731
        dt, x, ga, be, eps, rows, D, z, mu, rs, p(0))
    assert f(dt=3) == f(rows=-1) == f(D=0) == _lib.S4_ERR_INVALID_ARG
    assert f(D=8193) == f(rows=1 << 31) == _lib.S4_ERR_UNSUPPORTED
    assert f(x=p(0)) == f(mu=p(0)) == f(eps=ctypes.c_float(0.0)) == f(eps=ctypes.c_float(float("nan"))) == \
        _lib.S4_ERR_INVALID_ARG
    assert f(x=p(FAKE + 2)) == _lib.S4_ERR_INVALID_ARG                    # not aligned to a float
    assert f(z=p(FAKE + 1024)) == f(z=ga) == f(mu=z) == _lib.S4_ERR_INVALID_ARG   # overlaps
    assert f(rows=0, x=p(0)) == _lib.S4_OK                                 # nothing to do
    n = ctypes.c_size_t()
    assert lib.s4_layernorm_backward_workspace_size(64, ctypes.byref(n)) == 0 and n.value > 0
    assert lib.s4_layernorm_backward_workspace_size(8193, ctypes.byref(n)) == _lib.S4_ERR_UNSUPPORTED
    assert lib.s4_layernorm_backward_workspace_size(0, ctypes.byref(n)) == _lib.S4_ERR_INVALID_ARG
    lib.s4_layernorm_backward_workspace_size(64, ctypes.byref(n))
    dz, dx, dg, db = (p(FAKE2 + 0x1000000 * i) for i in range(4))
    g = lambda dz=dz, dx=dx, dg=dg, ws=ws, nb=n.value, rows=8: lib.s4_layernorm_backward(  # noqa: E731
        0, dz, x, ga, mu, rs, rows, 64, dx, dg, db, ws, nb, p(0))
    assert g(dz=p(0)) == g(dg=p(0)) == g(dx=x) == g(dg=db) == _lib.S4_ERR_INVALID_ARG
    assert g(ws=p(0)) == g(nb=n.value - 1) == g(ws=p(FAKE + 0x6000010)) == _lib.S4_ERR_WORKSPACE
    c = lambda H=64, L=64, dz=dz, nb=n.value, eps=eps: lib.s4_layernorm_channels_backward(  # noqa: E731
        dz, x, ga, eps, 2, H, L, dx, dg, db, ws, nb, p(0))
    assert c(L=100) == c(L=8) == c(L=131072) == _lib.S4_ERR_UNSUPPORTED
    assert c(H=0) == c(H=8193) == c(dz=p(0)) == c(dz=dx) == c(dz=p(FAKE2 + 8)) == _lib.S4_ERR_INVALID_ARG
    assert c(nb=16) == _lib.S4_ERR_WORKSPACE


def test_gated_delta_scan_rejects_bad_arguments(lib):
    q, k, v, g, be, st, o = (p(FAKE + 0x1000000 * i) for i in range(7))

    def f(dt=1, q=q, sq=256, sk=256, sv=512, scale=1.0, st=st, Bt=2, T=3, Hk=2, Hv=4, Dk=128, Dv=128, o=o):
        return lib.s4_gated_delta_scan(dt, q, sq, k, sk, v, sv, g, be, ctypes.c_float(scale), st, Bt, T, Hk, Hv, Dk,
                                       Dv, o, p(0))
    bad = _lib.S4_ERR_INVALID_ARG
    assert f(dt=7) == f(q=p(0)) == f(st=p(0)) == f(Bt=0) == f(T=-1) == f(Hk=0) == f(Hv=3) == f(Dk=0) == bad
    assert f(Dk=100) == f(Dv=136) == f(Dv=4) == _lib.S4_ERR_UNSUPPORTED
    assert f(sq=255) == f(sq=248) == f(sv=504) == f(sk=260) == f(scale=float("inf")) == bad
    assert f(q=p(FAKE + 8)) == f(o=v) == f(st=o) == f(o=q) == bad
    assert f(T=0, q=p(0)) == _lib.S4_OK


def test_gated_delta_chunks_reject_bad_arguments(lib):
    q, k, v, g, be, st, o, ws, fs, do, dq, dk, dv, dg, db = (p(FAKE + 0x10000000 * i) for i in range(15))
    n = ctypes.c_size_t()
    size = lambda dt=1, Bt=2, tok=200, Hk=2, Hv=4, Dk=128, Dv=128, keep=1: lib.s4_gated_delta_workspace_size(  # noqa: E731
        dt, Bt, tok, Hk, Hv, Dk, Dv, keep, ctypes.byref(n))
    bad, no = _lib.S4_ERR_INVALID_ARG, _lib.S4_ERR_UNSUPPORTED
    assert size(dt=5) == size(Bt=0) == size(tok=-1) == size(Hv=3) == bad
    assert size(Dk=12) == size(Dv=256) == size(tok=1 << 31) == size(tok=(1 << 31) - 1, Hv=128, Hk=128) == no
    assert lib.s4_gated_delta_workspace_size(1, 2, 200, 2, 4, 128, 128, 1, None) == bad
    assert size(keep=0) == 0
    small = n.value
    assert size() == 0 and n.value > small and n.value % 256 == 0
    need = n.value

    def f(dt=1, q=q, sq=256, st=st, cu=0, Bt=2, tok=200, Dk=128, o=o, fs=fs, keep=1, ws=ws, nb=need, scale=1.0):
        return lib.s4_gated_delta_forward(dt, q, sq, k, 256, v, 512, g, be, ctypes.c_float(scale), st, p(cu), Bt, tok, 2,
                                          4, Dk, 128, o, fs, keep, ws, nb, p(0), p(0))
    assert f(dt=9) == f(q=p(0)) == f(o=p(0)) == f(sq=128) == f(tok=201) == f(scale=float("inf")) == bad
    assert f(o=v) == f(fs=o) == f(o=ws) == f(st=p(FAKE + 0x50000000 + 8)) == f(fs=ws) == bad
    assert f(Dk=130) == f(Dk=136) == no
    assert f(ws=p(0)) == f(nb=need - 1) == f(ws=p(FAKE + 0x70000010)) == _lib.S4_ERR_WORKSPACE

    def b(do=do, dq=dq, dv=dv, dg=dg, tok=200, Bt=2, ws=ws, nb=need):
        return lib.s4_gated_delta_backward(1, g, be, ctypes.c_float(1.0), p(0), Bt, tok, 2, 4, 128, 128, do, p(0), dq, dk,
                                           dv, dg, db, p(0), ws, nb, p(0), p(0))
    assert b(do=p(0)) == b(dq=p(0)) == b(dg=p(0)) == b(tok=201) == b(Bt=0) == bad
    assert b(dv=do) == b(dq=dk) == b(dg=db) == b(dv=ws) == bad
    assert b(ws=p(0)) == b(nb=small) == _lib.S4_ERR_WORKSPACE


@pytest.mark.parametrize("Bt,Hk,Hv,Dk,Dv", [(1, 4, 8, 128, 128), (1, 1, 1, 64, 64), (1, 1, 2, 8, 128), (2, 2, 4, 128, 96),
                                            (4, 4, 8, 128, 128), (3, 1, 3, 72, 40), (8, 8, 16, 128, 128),
                                            (13, 8, 16, 128, 128), (5, 2, 6, 96, 80), (1, 32, 32, 128, 128)])
@pytest.mark.parametrize("keep", [0, 1])
def test_gated_delta_workspace_for_more_tokens_serves_fewer(lib, Bt, Hk, Hv, Dk, Dv, keep):
    n = ctypes.c_size_t()
    last = 0
    for tokens in [*range(0, 3000, 7), *range(3000, 80000, 64), *range(80000, 1000000, 640)]:
        assert lib.s4_gated_delta_workspace_size(1, Bt, tokens, Hk, Hv, Dk, Dv, keep, ctypes.byref(n)) == 0
        assert n.value >= last, tokens
        last = n.value
