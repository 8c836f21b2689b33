"""Refusals of moe_add_rmsnorm, moe_linear and moe_route_scored: every check below fails on the host
before anything is enqueued, so no GPU is needed; and the binding's own checks."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from bit_moe_expert_top_amd import _lib

    return _lib


P = 4096  # a 16-byte aligned address that is never dereferenced


def norm(L, x=P, xd=1, r=P, rd=2, w=P, eps=1e-6, T=4, H=64, ro=P, y=P, q=P, qs=P):
    return L.lib.moe_add_rmsnorm(x, xd, r, rd, w, eps, T, H, ro, y, q, qs, None)


@pytest.mark.parametrize("bad,want", [
    (dict(T=-1), -1), (dict(H=0), -1), (dict(H=-8), -1), (dict(xd=3), -1), (dict(xd=0), -1), (dict(rd=3), -1),
    (dict(eps=0.0), -1), (dict(eps=-1.0), -1), (dict(eps=math.inf), -1), (dict(eps=math.nan), -1), (dict(eps=1e-40), -1),
    (dict(H=72), -1),                             # MXFP8 of part of a block
    (dict(H=68, q=None, qs=None), -2), (dict(H=16392, q=None, qs=None), -2),
    (dict(x=None), -1), (dict(w=None), -1), (dict(y=None, q=None, qs=None), -1), (dict(qs=None), -1), (dict(q=None), -1),
    (dict(r=None), -1),                           # residual_out without a residual
    (dict(x=P + 4), -1), (dict(r=P + 2), -1), (dict(ro=P + 8), -1), (dict(w=P + 2), -1), (dict(y=P + 8), -1),
    (dict(q=P + 4), -1),
])
def test_norm_refusals(L, bad, want):
    assert norm(L, **bad) == want


def test_norm_of_no_rows(L):
    assert norm(L, T=0) == 0
    assert norm(L, T=0, x=None, w=None, y=None, q=None, qs=None) == 0


def linear(L, x=P, xs=None, w=P, ws=None, dt=2, T=4, N=64, K=64, bias=P, act=0, r=P, rd=1, out=P, od=1):
    return L.lib.moe_linear(x, xs, w, ws, dt, T, N, K, bias, act, r, rd, out, od, None)


@pytest.mark.parametrize("bad,want", [
    (dict(T=-1), -1), (dict(N=0), -1), (dict(K=0), -1), (dict(dt=1), -1), (dict(dt=4), -1), (dict(act=-1), -1),
    (dict(act=5), -1), (dict(rd=3), -1), (dict(od=3), -1), (dict(od=0), -1), (dict(act=4, N=63), -1),
    (dict(K=60), -2), (dict(K=(1 << 20) + 8), -2), (dict(N=(1 << 20) + 1), -2), (dict(T=(1 << 26) + 1), -2),
    (dict(x=None), -1), (dict(w=None), -1), (dict(out=None), -1), (dict(x=P + 8), -1), (dict(w=P + 2), -1),
    (dict(out=P + 2), -1), (dict(out=P + 1, od=2), -1), (dict(r=P + 2), -1), (dict(bias=P + 2), -1),
    (dict(dt=3, xs=P, ws=P, K=72, od=2), -1),     # MXFP8: part of a block
    (dict(dt=3, xs=P, ws=P, od=1), -2),           # MXFP8 to fp32
    (dict(dt=3, xs=None, ws=P, od=2), -1), (dict(dt=3, xs=P, ws=None, od=2), -1),
])
def test_linear_refusals(L, bad, want):
    assert linear(L, **bad) == want


def test_linear_of_no_rows(L):
    assert linear(L, T=0) == 0


def route(L, lg=P, bias=P, T=4, E=32, k=4, score=1, G=4, keep=2, top=2, renorm=1, scale=1.0, ids=P, w=P):
    return L.lib.moe_route_scored(lg, bias, T, E, k, score, G, keep, top, renorm, scale, ids, w, None)


@pytest.mark.parametrize("bad,want", [
    (dict(T=-1), -1), (dict(E=0), -1), (dict(E=1028), -1), (dict(k=0), -1), (dict(k=33, G=1, keep=1), -1),
    (dict(E=128, k=65, G=1, keep=1), -1), (dict(score=0), -1), (dict(score=3), -1), (dict(G=0), -1), (dict(G=5), -1),
    (dict(keep=0), -1), (dict(keep=5), -1), (dict(top=0), -1), (dict(top=3), -1), (dict(k=17), -1),
    (dict(scale=math.inf), -1), (dict(scale=math.nan), -1), (dict(E=130, G=65, keep=4), -2),
    (dict(lg=None), -1), (dict(ids=None), -1), (dict(w=None), -1),
])
def test_route_refusals(L, bad, want):
    assert route(L, **bad) == want


def test_route_of_no_tokens(L):
    assert route(L, T=0, lg=None, ids=None, w=None) == 0


def test_the_binding_refuses_what_the_kernels_do_not_read(L):
    x, w = torch.zeros(4, 64), torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="on the GPU"):
        L.moe_add_rmsnorm(x, w, 1e-6)                       # CPU tensors
    with pytest.raises(ValueError, match="x"):
        L.moe_add_rmsnorm(x.double(), w, 1e-6)
    with pytest.raises(ValueError, match="x"):
        L.moe_add_rmsnorm(torch.zeros(64, 4).t(), w, 1e-6)  # strides
    with pytest.raises(ValueError, match="weight"):
        L.moe_add_rmsnorm(x, w[:32], 1e-6)
    with pytest.raises(ValueError, match="go together"):
        L.moe_add_rmsnorm(x, w, 1e-6, q=torch.zeros(4, 64, dtype=torch.uint8))
    with pytest.raises(ValueError, match="without a residual"):
        L.moe_add_rmsnorm(x, w, 1e-6, residual_out=x)
    with pytest.raises(ValueError, match="residual_out"):   # another type than the residual's
        L.moe_add_rmsnorm(x, w, 1e-6, residual=x, residual_out=x.bfloat16())
    xb, wb = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="on the GPU"):
        L.moe_linear(xb, wb)
    with pytest.raises(ValueError, match="w: expected"):
        L.moe_linear(xb, wb[:, :32])
    with pytest.raises(ValueError, match="act"):
        L.moe_linear(xb, wb, act="tanh")
    with pytest.raises(ValueError, match="go together"):
        L.moe_linear(xb, wb, x_scales=torch.zeros(4, 2, dtype=torch.uint8))
    with pytest.raises(ValueError, match="residual"):
        L.moe_linear(xb, wb, residual=torch.zeros(4, 9))
    with pytest.raises(ValueError, match="out"):
        L.moe_linear(xb, wb, act="swiglu", out=torch.zeros(4, 8))
    with pytest.raises(ValueError, match="on the GPU"):
        L.moe_route_scored(x, 4)
    with pytest.raises(ValueError, match="logits"):
        L.moe_route_scored(xb, 4)
    with pytest.raises(ValueError, match="bias"):
        L.moe_route_scored(x, 4, bias=torch.zeros(63))
    with pytest.raises(ValueError, match="score"):
        L.moe_route_scored(x, 4, score="tanh")
    assert ctypes.sizeof(ctypes.c_void_p) == 8


def test_header_and_binding_agree(L):
    import os
    import re

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "bitmoe.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for name in ("moe_add_rmsnorm", "moe_linear", "moe_route_scored"):
        args = re.search(name + r"\(([^)]*)\)", text).group(1).split(",")
        got = [ctypes.c_void_p if "*" in a else ctypes.c_float if a.split()[0] == "float" else ctypes.c_int32 for a in args]
        assert got == getattr(L.lib, name).argtypes, name
    for enum, table in (("MOE_ACT_", L.ACTS), ("MOE_SCORE_", L.SCORES)):
        for key, value in table.items():
            assert re.search(rf"{enum}{key.upper()} = {value}\b", text), key
