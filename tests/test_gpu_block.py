"""GPU: the operators around the expert FFN (moe_add_rmsnorm, moe_linear, moe_route_scored) against
the fp64 oracle, at the sizes, types and masks where they can go wrong; the block that runs them
together; captured and replayed calls, another stream, in-place and offset buffers.

Tolerances.  A rounding to bf16 is off by at most 2^-8 of the value, to fp32 by 2^-24."""
import numpy as np
import pytest
import torch

from oracle import block as OB
from oracle import formats as OF
from oracle import moe as OM

from _helpers import KAPPA, device_layer, host, oracle_layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_moe_expert_top_amd import _lib

    return _lib


def values(t):
    """fp64 values of a float tensor, of bf16 bits (int16) as bf16."""
    if t.dtype == torch.int16:
        t = t.view(torch.bfloat16)
    return host(t.float()).astype(np.float64)


def cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


DT = {"f32": torch.float32, "bf16": torch.bfloat16}
GUARD = 64  # values behind an output that have to stay as they are


def guarded(shape, dtype):
    """An output tensor and the buffer around it, filled with a pattern."""
    n = int(np.prod(shape))
    buf = torch.full((n + GUARD,), 0x5A, dtype=torch.uint8, device="cuda").repeat_interleave(dtype.itemsize).view(dtype)
    return buf[:n].view(shape), buf


def guard_kept(buf):
    return bool((buf.view(torch.uint8)[-GUARD * buf.element_size():] == 0x5A).all())


# ------------------------------------------------------------------ residual + RMS norm
def norm_case(T, H, x, res, seed=0, big=1.0):
    r = np.random.default_rng([seed, T, H])
    xv = cuda((r.normal(size=(T, H)) * big).astype(np.float32), DT[x])
    rv = None if res is None else cuda((r.normal(size=(T, H)) * np.exp(r.normal(size=H)) * big).astype(np.float32), DT[res])
    wv = cuda((1 + 0.3 * r.normal(size=H)).astype(np.float32), torch.bfloat16)
    return xv, rv, wv


def check_norm(L, xv, rv, wv, eps, q=True, in_place=False):
    T, H = xv.shape
    y, ybuf = guarded((T, H), torch.bfloat16)
    qe, qbuf = guarded((T, H), torch.uint8) if q else (None, None)
    qs, sbuf = guarded((T, H // 32), torch.uint8) if q else (None, None)
    want_s, want_y = OB.add_rmsnorm(values(xv), None if rv is None else values(rv), values(wv), eps,
                                    rv is not None and rv.dtype == torch.bfloat16)
    ro = None if rv is None else (rv if in_place else torch.empty_like(rv))
    L.moe_add_rmsnorm(xv, wv, eps, residual=rv, residual_out=ro, y=y, q=qe, q_scales=qs)
    torch.cuda.synchronize()
    if ro is not None:
        np.testing.assert_array_equal(values(ro), want_s.astype(np.float64))
    # sum of squares: each thread sums at most 64 values one after another, then at most 6 + 8
    # additions join them: (64 + 14) 2^-24, half of it under the root; mean, eps, rsqrt (2 ulp) and
    # two products: 6 more roundings.  Then one rounding to bf16.
    rel = (39 + 8) * 2.0**-24
    np.testing.assert_array_less(np.abs(values(y) - want_y), np.abs(want_y) * (2.0**-8 + rel) * 1.0001 + 1e-37)
    assert guard_kept(ybuf)
    if q:
        we, ws = L.moe_mxfp8_quantize(y)
        np.testing.assert_array_equal(host(qe), host(we))
        np.testing.assert_array_equal(host(qs), host(ws))
        oe, osc = OF.mxfp8_quantize(values(y))
        np.testing.assert_array_equal(host(qe), oe)
        np.testing.assert_array_equal(host(qs), osc)
        assert guard_kept(qbuf) and guard_kept(sbuf)


@pytest.mark.parametrize("H", [8, 32, 72, 96, 256, 512, 520, 1024, 1056, 2016, 2048, 2080, 4096, 4128, 8192, 8224, 16384])
def test_norm_widths(L, H):
    for T, x, res in ((1, "f32", "bf16"), (5, "bf16", "f32")):
        xv, rv, wv = norm_case(T, H, x, res)
        check_norm(L, xv, rv, wv, 1e-6, q=H % 32 == 0)


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("res", [None, "f32", "bf16"])
@pytest.mark.parametrize("T,H", [(1, 256), (3, 4096), (4097, 64), (1031, 512)])
def test_norm_types(L, x, res, T, H):
    xv, rv, wv = norm_case(T, H, x, res)
    check_norm(L, xv, rv, wv, 1e-5, in_place=T % 2 == 1)


def test_norm_extreme_rows(L):
    """Rows of zeros, of one value, of very small and very large values; a residual that cancels x."""
    H = 256
    r = np.random.default_rng(5)
    x = r.normal(size=(8, H)).astype(np.float32)
    x[0] = 0
    x[1] = 0
    x[1, 77] = 3
    x[2] *= 1e-30
    x[3] *= 1e15
    x[4] = -0.0
    x[5, 32:64] = 0
    x[6] = 1e-40
    w = cuda(np.ones(H, np.float32), torch.bfloat16)
    check_norm(L, cuda(x), None, w, 1e-6)
    check_norm(L, cuda(x), None, w, 1.2e-38)
    check_norm(L, cuda(x), cuda(-x), w, 1e-6)


def test_norm_rows_are_independent(L):
    """A NaN or infinite row leaves the others as they are; a row has the same bits alone."""
    xv, rv, wv = norm_case(9, 4096, "f32", "bf16")
    y0 = L.moe_add_rmsnorm(xv, wv, 1e-6, residual=rv).clone()
    one = L.moe_add_rmsnorm(xv[4:5].clone(), wv, 1e-6, residual=rv[4:5].clone())
    assert torch.equal(one[0], y0[4])
    xv[2, 5] = float("nan")
    xv[7, 9] = float("inf")
    y1 = L.moe_add_rmsnorm(xv, wv, 1e-6, residual=rv)
    keep = [0, 1, 3, 4, 5, 6, 8]
    assert torch.equal(y0[keep], y1[keep])


def test_norm_broken_rows_quantise_alike(L):
    """NaN and infinities in a row: q and its scales are what moe_mxfp8_quantize makes of y."""
    xv, _, wv = norm_case(6, 256, "f32", None)
    xv[1, 3] = float("nan")
    xv[2, 40] = float("inf")
    xv[4, 200] = -float("inf")
    y = torch.empty((6, 256), dtype=torch.int16, device="cuda")
    q, qs = torch.empty((6, 256), dtype=torch.uint8, device="cuda"), torch.empty((6, 8), dtype=torch.uint8, device="cuda")
    L.moe_add_rmsnorm(xv, wv, 1e-6, y=y, q=q, q_scales=qs)
    q2, qs2 = L.moe_mxfp8_quantize(y)
    assert torch.equal(q, q2) and torch.equal(qs, qs2)


def test_norm_many_rows(L):
    """More rows than the tests of the widths have: every row is computed."""
    T, H = 70001, 64
    xv, rv, wv = norm_case(T, H, "bf16", "bf16")
    check_norm(L, xv, rv, wv, 1e-6)


def test_norm_equals_addition_then_norm(L):
    xv, rv, wv = norm_case(33, 2048, "f32", "bf16")
    ro = torch.empty_like(rv)
    y = L.moe_add_rmsnorm(xv, wv, 1e-6, residual=rv, residual_out=ro)
    assert torch.equal(y, L.moe_add_rmsnorm(ro, wv, 1e-6))


# ------------------------------------------------------------------ dense product
def mx_pair(L, v):
    e, s = L.moe_mxfp8_quantize(v.view(torch.int16))
    return e, s, OF.dequant_fp8(host(e), host(s))


def check_linear(L, T, N, K, act="none", bias=False, res=None, out="f32", mx=False, seed=0, offset=0, in_place=False,
                 scale=1.0):
    r = np.random.default_rng([seed, T, N, K])
    cols = N // 2 if act == "swiglu" else N
    xb = cuda((r.normal(size=(T, K)) * scale).astype(np.float32), torch.bfloat16)
    wb = cuda((r.normal(size=(N, K)) / np.sqrt(K)).astype(np.float32), torch.bfloat16)
    kw = {}
    if mx:
        x, kw["x_scales"], xv = mx_pair(L, xb)
        w, kw["w_scales"], wv = mx_pair(L, wb)
    else:
        x, w, xv, wv = xb, wb, values(xb), values(wb)
    bv = r.normal(size=N).astype(np.float32) if bias else None
    o, buf = guarded((T * cols + offset,), DT[out])
    o = o[offset:].view(T, cols)
    rv = rw = None
    if res:
        rv = cuda(r.normal(size=(T, cols)).astype(np.float32), DT[res])
        rw = values(rv)
        if in_place:
            o.copy_(rv)
            rv = o
    want = OB.linear(xv, wv, bv, act, rw)
    L.moe_linear(x, w, bias=None if bv is None else cuda(bv), act=act, residual=rv, out=o, **kw)
    torch.cuda.synchronize()
    got = values(o)
    # the sums' error: bf16 products are exact in fp32 and each of the K additions rounds a partial
    # sum, twice the bound of rounding to nearest (2^-24 of at most sum |x w|); the FP8 matrix cores'
    # is KAPPA times the root of the sum of squared products
    mag = np.abs(xv) @ np.abs(wv).T
    dev = KAPPA * np.sqrt((xv * xv) @ (wv * wv).T) if mx else np.minimum(K * 2.0**-23, 1e-3) * mag
    a = OB.linear(xv, wv, bv)
    dev = dev + np.abs(a) * 2.0**-23
    # through the activation: slopes of at most 1.13 (gelu) and 1.1 (silu), and the exponential's
    # relative error, (3 |a| + 8) 2^-23 with its argument's rounding and the quotient
    if act == "swiglu":
        g, u, dg, du = a[:, :cols], a[:, cols:], dev[:, :cols], dev[:, cols:]
        s = np.abs(OB.act(g, "silu"))
        dev = 1.1 * dg * (np.abs(u) + du) + (s + 1.1 * dg) * du + s * np.abs(u) * (3 * np.abs(g) + 8) * 2.0**-23
    elif act in ("gelu", "silu"):
        size = np.abs(a) + (0.1 * np.abs(a) ** 3 if act == "gelu" else 0)
        dev = 1.13 * dev + np.abs(OB.act(a, act)) * (3 * size + 8) * 2.0**-23
    half = 2.0**-8 if out == "bf16" else 2.0**-24
    dev = dev + (np.abs(want) + dev) * (half + (2.0**-24 if res else 0)) + 1e-37
    np.testing.assert_array_less(np.abs(got - want), dev * 1.0001)
    if not mx and out == "f32" and act == "none" and T * N >= 64:
        # in the root mean square: K independent roundings of partial sums no larger than the result
        err = np.linalg.norm(got - want) / np.linalg.norm(want)
        assert err <= 2 * 2.0**-24 * (np.sqrt(K) + 2), err
    assert guard_kept(buf)


@pytest.mark.parametrize("T", [1, 2, 7, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 200, 255, 256, 257, 300, 513])
@pytest.mark.parametrize("mx", [False, True])
def test_linear_rows(L, T, mx):
    check_linear(L, T, 200, 320, bias=True, res="f32", out="bf16", mx=mx)
    check_linear(L, T, 528, 2048, act="swiglu", out="bf16", mx=mx)


@pytest.mark.parametrize("N", [1, 2, 3, 31, 33, 60, 64, 127, 129, 255, 384, 513])
def test_linear_columns(L, N):
    for T in (3, 70, 400):
        check_linear(L, T, N, 256, bias=True, out="f32", res="bf16")
        check_linear(L, T, 2 * N, 256, act="swiglu", bias=True, out="bf16", mx=True)


@pytest.mark.parametrize("K", [8, 16, 24, 32, 40, 56, 64, 72, 96, 120, 128, 136, 248, 256, 264, 504, 512, 520, 1000, 1032,
                               2016, 4096, 5000, 16384])
def test_linear_depths(L, K):
    for T in (1, 20, 90, 260):
        check_linear(L, T, 96, K)
    if K % 32 == 0:
        for T in (1, 20, 90, 260):
            check_linear(L, T, 96, K, out="bf16", mx=True)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu", "swiglu"])
@pytest.mark.parametrize("mx", [False, True])
def test_linear_epilogue(L, act, mx):
    for T in (1, 40, 300):
        for bias in (False, True):
            for res, out in ((None, "bf16"), ("f32", "bf16"), ("bf16", "bf16"), (None, "f32"), ("bf16", "f32")):
                if mx and out == "f32":
                    continue
                check_linear(L, T, 264, 256, act=act, bias=bias, res=res, out=out, mx=mx)


@pytest.mark.parametrize("T,N,K", [(1024, 1024, 512), (777, 1288, 1056), (2048, 512, 4096), (4100, 256, 256), (300, 4096, 128)])
@pytest.mark.parametrize("mx", [False, True])
def test_linear_large(L, T, N, K, mx):
    check_linear(L, T, N, K, out="bf16" if mx else "f32", mx=mx)
    check_linear(L, T, N, K, act="swiglu", bias=True, res="bf16", out="bf16", mx=mx)


@pytest.mark.parametrize("T,N,K", [  # the kernels of moe_linear and their edges: few steps and many, ragged rows and columns
    (5, 4096, 1032), (30, 4090, 520), (61, 4096, 200), (200, 1000, 1032), (512, 4096, 200), (500, 4090, 1032),
    (1001, 4096, 136), (1001, 4090, 1032), (2048, 4096, 264), (4096, 4096, 72), (4001, 4090, 328)])
def test_linear_kernels_bf16(L, T, N, K):
    check_linear(L, T, N, K, bias=True, res="bf16", out="f32")
    check_linear(L, T, N, K, act="swiglu", out="bf16")


@pytest.mark.parametrize("T,N,K", [
    (5, 4096, 2080), (30, 4090, 544), (61, 4096, 416), (200, 1000, 2080), (256, 1000, 96), (2048, 1000, 160),
    (2047, 1001, 2080), (1001, 4096, 288), (2048, 4096, 128), (1990, 4090, 1184)])
def test_linear_kernels_mxfp8(L, T, N, K):
    check_linear(L, T, N, K, bias=True, res="f32", out="bf16", mx=True)
    if N % 2 == 0:
        check_linear(L, T, N, K, act="swiglu", out="bf16", mx=True)


@pytest.mark.parametrize("T,N,K", [(2048, 1000, 32), (2048, 1000, 160), (2047, 1004, 2080), (1001, 4096, 288),
                                   (2048, 4096, 128), (1990, 4090, 1184), (4090, 2048, 544), (2048, 512, 4096)])
def test_linear_mxfp8_bf16_residual(L, T, N, K):
    check_linear(L, T, N, K, bias=True, res="bf16", out="bf16", mx=True)
    check_linear(L, T, N, K, act="silu", res="bf16", out="bf16", mx=True, in_place=True)
    if N % 8 == 0:
        check_linear(L, T, N, K, act="swiglu", res="bf16", out="bf16", mx=True, in_place=True)


def test_linear_rows_do_not_touch_each_other(L):
    """A NaN in a token row stays in that row, also in the rows the kernels fill up with."""
    for T, N in ((3, 64), (20, 64), (60, 96), (100, 4096), (700, 4096)):
        x, w = torch.randn(T, 256, device="cuda").bfloat16(), torch.randn(N, 256, device="cuda").bfloat16()
        a = L.moe_linear(x, w, out_dtype=torch.float32)
        x[T // 2, 17] = float("nan")
        b = L.moe_linear(x, w, out_dtype=torch.float32)
        keep = [t for t in range(T) if t != T // 2]
        assert torch.equal(a[keep], b[keep]) and bool(torch.isnan(b[T // 2]).all())


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu", "swiglu"])
@pytest.mark.parametrize("T,N", [(3, 64), (60, 96), (300, 512)])
def test_linear_carries_nan_and_infinities(L, act, T, N):
    """A NaN or an infinite sum comes out as the definition has it, through every activation."""
    r = np.random.default_rng([T, N])
    x = cuda(r.normal(size=(T, 64)).astype(np.float32), torch.bfloat16)
    w = cuda(np.abs(r.normal(size=(N, 64))).astype(np.float32) + 0.1, torch.bfloat16)
    for t, v in ((0, float("nan")), (1, float("inf")), (2, -float("inf"))):
        x[t, 5] = v
    got = values(L.moe_linear(x, w, act=act, out_dtype=torch.float32))[:3]
    with np.errstate(invalid="ignore", over="ignore"):
        want = OB.linear(values(x)[:3], values(w), act_name=act)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    np.testing.assert_array_equal(got[np.isinf(want)], want[np.isinf(want)])
    assert np.isinf(got).sum() == np.isinf(want).sum()


def test_linear_large_values(L):
    """Activations far from zero: the exponential overflows on one side, the result is its limit."""
    for act in ("gelu", "silu", "swiglu"):
        check_linear(L, 40, 64, 64, act=act, scale=300.0)


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_linear_offset_and_in_place_outputs(L, out):
    """An output that starts at any element, and one that is its own residual."""
    for T in (3, 50, 300):
        for offset in (1, 2, 4):
            check_linear(L, T, 128, 256, res=out, out=out, offset=offset, in_place=True)
        check_linear(L, T, 131, 256, res=out, out=out, offset=3, in_place=True)


def test_linear_mxfp8_extreme_scales(L):
    """Zero blocks (scale byte 0) and large and small block exponents."""
    r = np.random.default_rng(9)
    T, N, K = 40, 64, 256
    x = r.normal(size=(T, K)) * np.repeat(np.exp2(r.integers(-20, 20, size=(T, K // 32))), 32, axis=1)
    x[3] = 0
    x[:, 64:96] = 0
    w = r.normal(size=(N, K))
    w[5, 32:64] = 0
    (xe, xs, xv), (we, ws, wv) = (mx_pair(L, cuda(v.astype(np.float32), torch.bfloat16)) for v in (x, w))
    got = values(L.moe_linear(xe, we, x_scales=xs, w_scales=ws))
    want = OB.linear(xv, wv)
    dev = KAPPA * np.sqrt((xv * xv) @ (wv * wv).T)
    np.testing.assert_array_less(np.abs(got - want), dev + (np.abs(want) + dev) * 2.0**-8 + 1e-30)


# ------------------------------------------------------------------ scored routing
def check_route(L, logits, k, **kw):
    bias = kw.pop("bias", None)
    T, E = logits.shape
    ids, ibuf = guarded((T, k), torch.int32)
    gates, gbuf = guarded((T, k), torch.float32)
    L.moe_route_scored(cuda(logits), k, bias=None if bias is None else cuda(bias), topk_ids=ids, topk_w=gates, **kw)
    torch.cuda.synchronize()
    want, gw = OB.route_scored(logits, k, bias=bias, **kw)
    np.testing.assert_array_equal(host(ids), want)
    # exp with an argument rounded in fp32: (|l - max| + 8) 2^-23 of the gate; the sum over the
    # experts, a quotient and a product: 16 more roundings of 2^-24
    lg = np.where(np.isfinite(logits), logits, 0.0)
    spread = np.abs(lg).max(axis=1, keepdims=True) * 2
    assert not np.isnan(host(gates)).any()
    np.testing.assert_array_less(np.abs(host(gates) - gw), np.abs(gw) * (spread + 16) * 2.0**-23 + 1e-38)
    assert guard_kept(ibuf) and guard_kept(gbuf)


ROUTES = [  # E, k, n_group, topk_group
    (1, 1, 1, 1), (2, 2, 1, 1), (8, 2, 1, 1), (8, 8, 2, 2), (12, 4, 4, 2), (60, 4, 1, 1), (64, 6, 8, 3), (65, 3, 5, 1),
    (100, 10, 4, 2), (127, 5, 1, 1), (128, 8, 64, 32), (160, 6, 8, 3), (256, 8, 8, 4), (384, 8, 8, 4), (384, 8, 1, 1),
    (512, 10, 16, 3), (513, 1, 3, 1), (1024, 64, 8, 2), (1024, 8, 64, 8),
]


@pytest.mark.parametrize("E,k,G,keep", ROUTES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_shapes(L, E, k, G, keep, score):
    r = np.random.default_rng([E, k, G])
    for T, top, biased, renorm in ((1, 1, False, True), (3, 2, True, True), (70, 1, True, False), (70, 2, False, False)):
        lg = (r.normal(size=(T, E)) * 2).astype(np.float32)
        bias = (r.normal(size=E) * 0.1).astype(np.float32) if biased else None
        check_route(L, lg, k, score=score, bias=bias, n_group=G, topk_group=keep, group_top=top, renormalize=renorm,
                    scale=2.5 if renorm else 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties(L, score):
    """Logits and biases on a few levels, so that experts and groups tie everywhere."""
    r = np.random.default_rng(11)
    for E, k, G, keep in ((16, 4, 4, 2), (64, 8, 8, 4), (384, 8, 8, 4), (1000, 20, 10, 3)):
        lg = r.integers(-1, 2, size=(50, E)).astype(np.float32)
        lg[0] = 0.0
        lg[1] = np.where(r.random(E) < 0.5, 0.0, -0.0)
        bias = (r.integers(-1, 2, size=E) * 0.25).astype(np.float32)
        for b in (None, bias, np.zeros(E, np.float32)):
            for top in (1, 2):
                check_route(L, lg, k, score=score, bias=b, n_group=G, topk_group=keep, group_top=top, renormalize=True)
                check_route(L, lg, k, score=score, bias=b)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_scores_next_to_each_other(L, score):
    """Logits that differ in their last bits, with biases that undo the difference: the order is that
    of 64-bit scores, far below what fp32 tells apart."""
    r = np.random.default_rng(12)
    E = 256
    base = r.normal(size=(60, 8)).astype(np.float32)
    lg = np.repeat(base, E // 8, axis=1)
    lg = np.nextafter(lg, np.where(r.random(lg.shape) < 0.5, np.inf, -np.inf).astype(np.float32))
    bias = (r.integers(-3, 4, size=E) * 2.0**-24).astype(np.float32)
    for b in (None, bias):
        check_route(L, lg, 8, score=score, bias=b, renormalize=True)
        check_route(L, lg, 8, score=score, bias=b, n_group=8, topk_group=4, group_top=2, renormalize=True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_out_of_service(L, score):
    """A bias of -inf: taken last, gate 0, nothing for the group; groups with one expert left or none."""
    r = np.random.default_rng(13)
    E = 32
    lg = r.normal(size=(40, E)).astype(np.float32)
    for dead in (range(0), range(8), range(1, 8), range(2, 32), range(1, 32), range(32)):
        bias = (r.normal(size=E) * 0.1 - 1.0).astype(np.float32)
        bias[list(dead)] = -np.inf
        for top in (1, 2):
            check_route(L, lg, 6, score=score, bias=bias, n_group=4, topk_group=2, group_top=top, renormalize=True)
        check_route(L, lg, 6, score=score, bias=bias, renormalize=True)
        check_route(L, lg, 6, score=score, bias=bias)


def test_route_broken_bias(L):
    """A NaN bias takes an expert out of service like one of -inf; huge biases order by themselves."""
    lg = np.random.default_rng(18).normal(size=(30, 64)).astype(np.float32)
    bias = np.zeros(64, np.float32)
    bias[[3, 17, 40]] = np.nan
    bias[[5, 60]] = 1e30
    bias[9] = -1e30
    for G, keep in ((1, 1), (4, 2), (8, 8)):
        for score in ("sigmoid", "softmax"):
            for top in (1, 2):
                check_route(L, lg, 8, score=score, bias=bias, n_group=G, topk_group=keep, group_top=top)


def test_route_equal_rows(L):
    """Padding rows: every logit the same, the experts in order."""
    for E, G, keep in ((64, 1, 1), (384, 8, 4), (1000, 10, 2)):
        lg = np.zeros((9, E), np.float32)
        lg[1], lg[2] = 5.0, -300.0
        for score in ("sigmoid", "softmax"):
            check_route(L, lg, 8, score=score, n_group=G, topk_group=keep, group_top=2, renormalize=True)


def test_route_masked_and_broken_logits(L):
    r = np.random.default_rng(14)
    lg = r.normal(size=(12, 40)).astype(np.float32)
    lg[0, :30] = -np.inf
    lg[1, 1:] = -np.inf
    lg[2] = -np.inf
    lg[3, 7] = np.nan
    lg[4] = np.nan
    lg[5] = np.finfo(np.float32).min
    lg[6, 3] = np.finfo(np.float32).min
    lg[7] = 80.0
    lg[8] = -120.0
    for score in ("sigmoid", "softmax"):
        for bias in (None, np.zeros(40, np.float32)):
            for G, keep in ((1, 1), (4, 2)):
                kw = dict(score=score, bias=None if bias is None else cuda(bias), n_group=G, topk_group=keep, group_top=2,
                          renormalize=True)
                ids, gates = L.moe_route_scored(cuda(lg), 6, **kw)
                ids, gates = host(ids), host(gates)
                assert ((ids >= 0) & (ids < 40)).all() and np.isfinite(gates).all()
                assert all(len(set(row)) == 6 for row in ids)
                want, gw = OB.route_scored(lg, 6, **{**kw, "bias": bias})
                np.testing.assert_array_equal(ids, want)
                np.testing.assert_allclose(gates, gw, rtol=3e-5, atol=1e-30)


@pytest.mark.parametrize("E,k,G,keep", [
    (4, 4, 1, 1), (64, 6, 8, 3), (100, 10, 4, 2), (128, 16, 16, 8), (160, 6, 8, 3), (256, 8, 8, 4), (260, 3, 13, 5),
    (384, 8, 8, 4), (384, 8, 1, 1), (384, 16, 3, 1), (512, 10, 16, 3), (512, 16, 1, 1), (508, 5, 2, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_batches(L, E, k, G, keep, score):
    """Batches that fill the GPU: several tokens to a wave, tokens that have to be routed again among them."""
    r = np.random.default_rng([E, k, G, 3])
    T = 8197
    lg = (r.normal(size=(T, E)) * 2).astype(np.float32)
    lg[::7] = np.round(lg[::7])                       # ties
    lg[5::50, : E // 2] = lg[5::50, E // 2 : E // 2 * 2]
    lg[11::97] = 0.0
    lg[13::97, : max(1, E // 3)] = -np.inf
    lg[17::97] = -200.0
    lg[T - 2] = np.round(lg[T - 2])
    bias = (r.normal(size=E) * 0.1).astype(np.float32)
    bias[r.permutation(E)[: E // 8]] = -np.inf
    some = np.r_[np.arange(0, 260), np.arange(T - 60, T), np.arange(260, T, 29)]
    for top, b, renorm in ((1, None, True), (2, bias, True), (1, bias, False), (2, None, False)):
        kw = dict(score=score, n_group=G, topk_group=keep, group_top=top, renormalize=renorm, scale=1.5)
        ids, gates = L.moe_route_scored(cuda(lg), k, bias=None if b is None else cuda(b), **kw)
        ids, gates = host(ids), host(gates)
        want, gw = OB.route_scored(lg[some], k, bias=b, **kw)
        np.testing.assert_array_equal(ids[some], want)
        spread = np.abs(np.where(np.isfinite(lg[some]), lg[some], 0)).max(axis=1, keepdims=True) * 2
        np.testing.assert_array_less(np.abs(gates[some] - gw), np.abs(gw) * (spread + 16) * 2.0**-23 + 1e-38)
        # the other tokens by the small batches' kernel
        for t in range(0, T, 500):
            i2, g2 = L.moe_route_scored(cuda(lg[t:t + 500]), k, bias=None if b is None else cuda(b), **kw)
            np.testing.assert_array_equal(host(i2), ids[t:t + 500])
            np.testing.assert_allclose(host(g2), gates[t:t + 500], rtol=1e-4, atol=1e-38)


@pytest.mark.parametrize("E,k,G,keep", [(64, 6, 4, 2), (256, 8, 8, 4), (384, 16, 1, 1), (512, 10, 1, 1), (512, 8, 16, 5)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_batches_close(L, E, k, G, keep, score):
    """Large batches whose scores are a few fp32 steps of the logit apart, within and across groups: the order is the
    64-bit one, wherever it is found."""
    r = np.random.default_rng([E, k, G, 5])
    T = 8200
    levels = np.linspace(-1.0, 2.0, 40)
    flat = levels[r.integers(0, 40, size=(T, E))].astype(np.float32)
    steps = r.integers(0, 4, size=(T, E)) * 10.0 ** r.integers(-8, -3, size=(T, 1))
    lg = (flat * (1.0 + steps)).astype(np.float32)
    # a token in eight: one level for all its larger logits, a few steps apart
    lg[::8] = np.minimum(lg[::8], np.float32(0.5) + r.integers(0, 6, size=lg[::8].shape).astype(np.float32) * 2.0**-24)
    some = np.r_[np.arange(0, 300), np.arange(T - 12, T), np.arange(300, T, 37)]
    same = np.full(E, 0.25, np.float32)                       # the scores' order is the logits'
    mixed = (r.integers(-2, 3, size=E) * 0.03125).astype(np.float32)
    # Sums of two scores only of the levels themselves: p(l + d) + p(l - d) is 2 p(l) to within d^2, which 64
    # bits do not hold apart for steps as small as these.
    for top, b, x in ((1, same, lg), (1, mixed, lg), (1, None, lg), (2, same, flat)):
        kw = dict(score=score, n_group=G, topk_group=keep, group_top=top, renormalize=True, scale=2.5)
        ids, _ = L.moe_route_scored(cuda(x), k, bias=None if b is None else cuda(b), **kw)
        want, _ = OB.route_scored(x[some], k, bias=b, **kw)
        np.testing.assert_array_equal(host(ids)[some], want)


def test_route_batches_replayed_and_off_alignment(L):
    """A large batch in a captured graph, and from logits that start at any float."""
    r = np.random.default_rng(31)
    T, E = 9000, 256
    lg = np.round(r.normal(size=(T, E)) * 8).astype(np.float32) / 8
    bias = cuda((r.normal(size=E) * 0.1).astype(np.float32))
    kw = dict(score="sigmoid", bias=bias, n_group=8, topk_group=3, group_top=2, renormalize=True)
    buf = torch.zeros(T * E + 1, device="cuda")
    off = buf[1:].view(T, E)
    off.copy_(cuda(lg))
    on = cuda(lg)
    i0, g0 = L.moe_route_scored(on, 8, **kw)
    i1, g1 = L.moe_route_scored(off, 8, **kw)
    assert torch.equal(i0, i1)
    np.testing.assert_allclose(host(g0), host(g1), rtol=1e-5)
    ids, gates = torch.zeros_like(i0), torch.zeros_like(g0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.moe_route_scored(on, 8, topk_ids=ids, topk_w=gates, **kw)
    for turn in range(3):
        on.copy_(cuda(np.roll(lg, turn, axis=0)))
        graph.replay()
        torch.cuda.synchronize()
        want = L.moe_route_scored(on, 8, **kw)
        assert torch.equal(ids, want[0]) and torch.equal(gates, want[1])


def test_offsets_past_32_bits(L):
    """More than 2^31 elements in an array: the last rows are those of a small call."""
    last = 40
    x = torch.zeros((1_050_000, 2056), dtype=torch.bfloat16, device="cuda")
    w = torch.randn(2056, device="cuda").bfloat16()
    x[-last:] = torch.randn(last, 2056, device="cuda").bfloat16()
    y = L.moe_add_rmsnorm(x, w, 1e-6)
    assert torch.equal(y[-last:], L.moe_add_rmsnorm(x[-last:].clone(), w, 1e-6)) and not bool(y[:1000].view(torch.bfloat16).any())
    del x, y
    x = torch.zeros((530_000, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.randn(4096, 64, device="cuda").bfloat16()
    x[-last:] = torch.randn(last, 64, device="cuda").bfloat16()
    out = L.moe_linear(x, w)
    small = values(L.moe_linear(x[-last:].clone(), w))
    # sums of 64 products in two orders, each rounded to bf16
    np.testing.assert_allclose(values(out[-last:]), small, rtol=2.0**-7, atol=64 * 2.0**-22)
    assert not bool(out[:1000].view(torch.bfloat16).any())
    del x, out
    lg = torch.zeros((5_600_000, 384), device="cuda")
    lg[-last:] = torch.randn(last, 384, device="cuda")
    ids, gates = L.moe_route_scored(lg, 4, n_group=8, topk_group=2, renormalize=True)
    i2, g2 = L.moe_route_scored(lg[-last:].clone(), 4, n_group=8, topk_group=2, renormalize=True)
    assert torch.equal(ids[-last:], i2) and bool((ids[:1000] == torch.arange(4, device="cuda")).all())
    np.testing.assert_allclose(host(gates[-last:]), host(g2), rtol=1e-5)
    del lg
    torch.cuda.empty_cache()


def test_route_long(L):
    lg = np.random.default_rng(15).normal(size=(3001, 384)).astype(np.float32)
    bias = (np.random.default_rng(16).normal(size=384) * 0.05).astype(np.float32)
    check_route(L, lg, 8, score="sigmoid", bias=bias, n_group=8, topk_group=4, group_top=2, renormalize=True, scale=2.5)


def test_route_agrees_with_moe_route(L):
    """Softmax without a bias, renormalised: the ids of moe_route, and its gates to fp32 rounding."""
    lg = cuda(np.random.default_rng(17).normal(size=(500, 384)).astype(np.float32))
    a, ga = L.moe_route(lg, 8)
    b, gb = L.moe_route_scored(lg, 8, renormalize=True)
    assert torch.equal(a, b)
    np.testing.assert_allclose(host(ga), host(gb), rtol=1e-5)


# ------------------------------------------------------------------ streams, capture, empty batches
def test_no_rows(L):
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")
    assert L.moe_add_rmsnorm(z(0, 64), z(64, dt=torch.bfloat16), 1e-6).shape == (0, 64)
    assert L.moe_linear(z(0, 64, dt=torch.bfloat16), z(8, 64, dt=torch.bfloat16)).shape == (0, 8)
    assert L.moe_route_scored(z(0, 16), 2)[0].shape == (0, 2)


def all_three(L, s):
    L.moe_add_rmsnorm(s["x"], s["wn"], 1e-6, residual=s["res"], residual_out=s["ro"], y=s["y"], q=s["q"], q_scales=s["qs"])
    L.moe_linear(s["y"], s["wr"], out=s["lg"])
    L.moe_route_scored(s["lg"], 4, score="sigmoid", bias=s["b"], n_group=4, topk_group=2, group_top=2, renormalize=True,
                       topk_ids=s["ids"], topk_w=s["gates"])
    L.moe_linear(s["q"], s["w1"], x_scales=s["qs"], w_scales=s["w1s"], act="swiglu", out=s["h"])
    return [s[k].clone() for k in ("ro", "y", "q", "qs", "lg", "ids", "gates", "h")]


def state(L, T, H=512, E=32, I=256, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device="cuda")
    w1, w1s = L.moe_mxfp8_quantize((n(2 * I, H) / 16).bfloat16().view(torch.int16))
    return dict(x=n(T, H), res=n(T, H).bfloat16(), ro=e(T, H), wn=n(H).bfloat16(), y=e(T, H), q=e(T, H, dt=torch.uint8),
                qs=e(T, H // 32, dt=torch.uint8), wr=(n(E, H) / 16).bfloat16(), lg=e(T, E, dt=torch.float32),
                b=0.1 * n(E), ids=e(T, 4, dt=torch.int32), gates=e(T, 4, dt=torch.float32), w1=w1, w1s=w1s, h=e(T, I))


@pytest.mark.parametrize("T", [1, 48, 700])
def test_captured_calls_replay(L, T):
    """The calls in a HIP graph, replayed on changing inputs with eager work between the replays."""
    s = state(L, T)
    all_three(L, s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = all_three(L, s)
    for seed in range(1, 5):
        new = state(L, T, seed=seed)
        for k in ("x", "res", "wr", "b", "w1", "w1s", "wn"):
            s[k].copy_(new[k])
        g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        want = all_three(L, new)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_two_streams_at_once(L):
    """Calls on two streams at the same time do not share anything."""
    a, b = state(L, 300, seed=1), state(L, 300, seed=2)
    want = [all_three(L, a), all_three(L, b)]
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(sa):
            ga = all_three(L, a)
        with torch.cuda.stream(sb):
            gb = all_three(L, b)
        torch.cuda.synchronize()
        for x, y in zip(ga + gb, want[0] + want[1]):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_results_do_not_change_from_call_to_call(L):
    s = state(L, 257)
    want = all_three(L, s)
    for _ in range(5):
        for x, y in zip(all_three(L, s), want):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


# ------------------------------------------------------------------ the block
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [1, 16, 130])
def test_block(L, T, mx):
    """Norm, router, scored routing, experts and a shared expert together, each step against the
    oracle's on the step's own input, and the block's output against the whole."""
    sp, dw = device_layer("tiny")
    H, E, k, Is = sp["H"], sp["E"], sp["k"], 256
    r = np.random.default_rng([T, 21])
    wn = cuda((1 + 0.1 * r.normal(size=H)).astype(np.float32), torch.bfloat16)
    wr = cuda((r.normal(size=(E, H)) / 16).astype(np.float32), torch.bfloat16)
    rb = (r.normal(size=E) * 0.05).astype(np.float32)
    w1, w2 = (cuda((r.normal(size=s) / np.sqrt(s[1])).astype(np.float32), torch.bfloat16) for s in ((2 * Is, H), (H, Is)))
    ws = [w1, w2]
    if mx:
        ws = [L.moe_mxfp8_quantize(v.view(torch.int16)) for v in ws]
    route = dict(score="sigmoid", n_group=4, topk_group=2, group_top=1, renormalize=True, scale=1.5)
    blk = L.MoeBlock(dw, k, wn, wr, router_bias=cuda(rb), route=route, ws1=ws[0], ws2=ws[1])
    x, res = cuda(r.normal(size=(T, H)).astype(np.float32)), cuda(r.normal(size=(T, H)).astype(np.float32), torch.bfloat16)
    s0, y0 = OB.add_rmsnorm(values(x), values(res), values(wn), 1e-6, True)
    o = L.block_forward(blk, x, res)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(values(res), s0.astype(np.float64))
    y = values(o["y"])
    np.testing.assert_array_less(np.abs(y - y0), np.abs(y0) * (2.0**-8 + 1e-5) + 1e-37)
    np.testing.assert_allclose(values(o["logits"]), OB.linear(y, values(wr)), atol=H * 2.0**-23 * 40)
    ids, gates = OB.route_scored(host(o["logits"]), k, bias=rb, **route)
    np.testing.assert_array_equal(host(o["ids"]), ids)
    np.testing.assert_allclose(host(o["gates"]), gates, rtol=1e-5)
    lay = oracle_layer("tiny")
    _, offsets, perm, inv = OM.permute(ids, E)
    yp = OM.expert_ffn(lay, host(o["y"]).view(np.uint16), k, offsets, perm)
    routed = OM.combine(yp, inv, gates, T, k)
    rms = np.sqrt(np.mean(routed**2))
    assert np.abs(values(o["routed"]) - routed).max() <= 2e-2 * rms
    if mx:
        deq = lambda p: OF.dequant_fp8(host(p[0]), host(p[1]))
        h = OB.linear(deq((o["q"], o["q_scales"])), deq(ws[0]), act_name="swiglu")
        hv = values(o["h"])
        assert np.abs(hv - h).max() <= 2.0**-8 * np.abs(h).max() + 1e-2 * np.sqrt(np.mean(h * h))
        he, hs = OF.mxfp8_quantize(hv)
        out = OB.linear(OF.dequant_fp8(he, hs), deq(ws[1]), residual=values(o["routed"]))
    else:
        h = OB.linear(y, values(w1), act_name="swiglu")
        hv = values(o["h"])
        assert np.abs(hv - h).max() <= 2.0**-8 * np.abs(h).max() + 1e-4
        out = OB.linear(hv, values(w2), residual=values(o["routed"]))
    tol = 2.0**-8 * np.abs(out).max() + KAPPA * np.abs(out).max() if mx else 1e-4
    assert np.abs(values(o["out"]) - out).max() <= tol
