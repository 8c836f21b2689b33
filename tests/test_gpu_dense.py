"""GPU: FP8 with a scale per block of 128 and products of it, the gated projection, the gradients of both,
against the fp64 oracle, at the sizes, types and values where they can go wrong; a shared expert's pass through them
together; captured and replayed calls, another stream, rows behind the last one.

Tolerances.  A rounding to bf16 is off by at most 2^-8 of the value, to fp32 by 2^-24.  Products of bf16 values are exact in
fp32 and each of n additions rounds a partial sum, twice the bound of rounding to nearest (2^-24 of at most the sum
of magnitudes).  The FP8 matrix cores' sums are off by at most KAPPA times the root of the sum of squared products."""
import numpy as np
import pytest
import torch

from oracle import block as OB
from oracle import dense as OD

from _helpers import KAPPA, device_layer, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_moe_expert_top_amd import _lib

    return _lib


DT = {"f32": torch.float32, "bf16": torch.bfloat16}
GUARD = 64  # values behind an output that have to stay as they are
ACTS = ["none", "relu", "gelu", "silu"]


def values(t):
    """fp64 values of a float tensor, of bf16 bits (int16) as bf16."""
    if t.dtype == torch.int16:
        t = t.view(torch.bfloat16)
    return host(t.float()).astype(np.float64)


def cuda(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(dtype)


def guarded(shape, dtype):
    """An output tensor and the buffer around it, filled with a pattern."""
    n = int(np.prod(shape))
    buf = torch.full((n + GUARD,), 0x5A, dtype=torch.uint8, device="cuda").repeat_interleave(dtype.itemsize).view(dtype)
    return buf[:n].view(shape), buf


def guard_kept(buf):
    return bool((buf.view(torch.uint8)[-GUARD * buf.element_size():] == 0x5A).all())


def bf16(r, *shape, scale=1.0):
    return cuda(r.normal(size=shape) * scale, torch.bfloat16)


# ------------------------------------------------------------------ quantisation
def check_quantize(L, x, by):
    rows, K = x.shape
    q, qbuf = guarded((rows, K), torch.uint8)
    s, sbuf = guarded((OD.up(rows, by), OD.up(K)), torch.float32)
    L.moe_fp8_quantize(x, block_rows=by, q=q, scales=s)
    torch.cuda.synchronize()
    want_q, want_s = OD.fp8_quantize(host(x.float()), by)
    np.testing.assert_array_equal(host(s), want_s)  # NaN counts as equal
    got = host(q)
    # a zero's sign has a test of its own
    np.testing.assert_array_equal(np.where(got == 0x80, 0, got), np.where(want_q == 0x80, 0, want_q))
    assert guard_kept(qbuf) and guard_kept(sbuf)


@pytest.mark.parametrize("by", [1, 128])
@pytest.mark.parametrize("rows,K", [(1, 16), (1, 4096), (3, 112), (7, 128), (64, 144), (127, 2016), (128, 256), (129, 272),
                                    (300, 1040), (1000, 512)])
def test_quantize_shapes(L, rows, K, by):
    r = np.random.default_rng([rows, K, by])
    size = np.exp(2 * r.normal(size=(rows, 1)))
    for dtype in (torch.float32, torch.bfloat16):
        check_quantize(L, cuda(size * r.normal(size=(rows, K)), dtype), by)


@pytest.mark.parametrize("by", [1, 128])
def test_quantize_many_blocks(L, by):
    """More blocks than workgroups of a launch."""
    x = torch.randn(1 << 20, 2048, device="cuda", dtype=torch.bfloat16) if by == 1 else torch.randn(
        1 << 19, 512, device="cuda", dtype=torch.bfloat16)
    q, s = L.moe_fp8_quantize(x, block_rows=by)
    rows = torch.cat([torch.arange(256), torch.arange(x.shape[0] - 256, x.shape[0])])
    want_q, want_s = OD.fp8_quantize(host(x[rows.cuda()].float()), by)
    np.testing.assert_array_equal(host(q[rows.cuda()]), want_q)
    blocks = torch.unique(rows // by).cuda()
    np.testing.assert_array_equal(host(s[blocks]), want_s)


@pytest.mark.parametrize("rows,K,by,dtype", [
    ((1 << 25) + 77, 16, 1, torch.bfloat16),   # workgroups that take two turns: from 2^25 blocks on
    (1 << 26, 16, 1, torch.bfloat16),          # all of them do, and the largest number of rows
    ((1 << 24) + 33, 144, 1, torch.float32),
    (128 * 16384 + 5, 144, 128, torch.bfloat16),
])
def test_quantize_large_is_its_slices(L, rows, K, by, dtype):
    """A call of many blocks has the bits of calls of 2^20 rows each."""
    x = torch.randn(rows, K, device="cuda", dtype=dtype)
    q, s = L.moe_fp8_quantize(x, block_rows=by)
    for i in range(0, rows, 1 << 20):
        part = x[i:i + (1 << 20)]
        pq, ps = L.moe_fp8_quantize(part, block_rows=by)
        assert torch.equal(q[i:i + (1 << 20)], pq) and torch.equal(s[i // by:i // by + len(ps)], ps), i


@pytest.mark.parametrize("by", [1, 128])
def test_quantize_extremes(L, by):
    """Zeros, subnormal and huge values, ties, infinities and NaN, each in a block of its own."""
    r = np.random.default_rng(3)
    for dtype in (torch.float32, torch.bfloat16):
        rows = []
        for size in (0.0, 1e-45, 3e-44, 1e-41, 1e-38, 1e-30, 2.0**-60, 2.0**-59, 1.0, 2.0**99, 2.0**101, 3e38):
            rows.append(np.clip(size * r.uniform(-1, 1, size=128), -3.38e38, 3.38e38))
        ties = np.concatenate([np.arange(1, 64) / 32 * 1.75, np.arange(1, 66) * 0.4375])  # multiples of an element step's half
        ties[-1] = 448.0
        rows += [ties, -ties, 3 * ties]
        for bad in (np.inf, -np.inf, np.nan):
            v = r.normal(size=128)
            v[77] = bad
            rows.append(v)
        x = np.stack(rows).astype(np.float32)
        if by == 128:
            x = np.repeat(x, 128, axis=0)
            x[1::128] *= 0.5
        check_quantize(L, cuda(x, dtype), by)


@pytest.mark.parametrize("by", [1, 128])
@pytest.mark.parametrize("top", [2.0**-100, 1.0, 2.0**110])
def test_quantize_signed_zeros(L, by, top):
    """-0 and negative values that round to zero are 0x80, with the short division and with the plain one."""
    v = np.tile([0.0, -0.0, 2.0**-20, -(2.0**-20)], (4, 32))
    v[:, 5] = 1.0
    x = cuda(v * top)
    q, _ = L.moe_fp8_quantize(x, block_rows=by)
    want = np.tile([0x00, 0x80, 0x00, 0x80], (4, 32))
    want[:, 5] = 0x7E  # 448
    np.testing.assert_array_equal(host(q), want)


# ------------------------------------------------------------------ FP8 product
def fp8_operand(L, v, by, gated=False):
    """Elements, scales and fp64 values of bf16 rows v."""
    parts = [L.moe_fp8_quantize(p.contiguous(), block_rows=by) for p in (v.chunk(2) if gated else (v,))]
    q, s = torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
    return q, s, OD.fp8_values(host(q), host(s), by, gated)


def act_deviation(a, dev, act, cols):
    """How far act(a) (with the gate's product for swiglu) is off where a is off by dev: slopes of at most 1.13
    (gelu) and 1.1 (silu), and the exponential's relative error, (3 |z| + 8) 2^-23 with its argument's rounding and
    the quotient."""
    if act in ("gelu", "silu"):
        size = np.abs(a) + (0.1 * np.abs(a) ** 3 if act == "gelu" else 0)
        return 1.13 * dev + np.abs(OB.act(a, act)) * (3 * size + 8) * 2.0**-23
    if act == "swiglu":
        return gate_deviation(a, dev, "silu", cols)
    return dev


def gate_deviation(a, dev, act, cols):
    """The same for act(g) * u."""
    g, u, dg, du = a[:, :cols], a[:, cols:], dev[:, :cols], dev[:, cols:]
    v = np.abs(OB.act(g, act))
    dv = act_deviation(g, dg, act, cols)
    return dv * (np.abs(u) + du) + v * du + v * np.abs(u) * 2.0**-23


def check_fp8(L, T, N, K, act="none", bias=False, res=None, seed=0, offset=0, in_place=False, operands=None):
    r = np.random.default_rng([seed, T, N, K])
    gated = act == "swiglu"
    cols = N // 2 if gated else N
    x, xs, xv = operands[0] if operands else fp8_operand(L, bf16(r, T, K) * cuda(np.exp(r.normal(size=K)), torch.bfloat16), 1)
    w, ws, wv = operands[1] if operands else fp8_operand(
        L, bf16(r, N, K, scale=K**-0.5) * cuda(np.exp(0.5 * r.normal(size=(N, 1))), torch.bfloat16), 128, gated)
    bv = r.normal(size=N).astype(np.float32) if bias else None
    o, buf = guarded((T * cols + offset,), torch.bfloat16)
    o = o[offset:].view(T, cols)
    rv = rw = None
    if res:
        rv = cuda(r.normal(size=(T, cols)), DT[res])
        rw = values(rv)
        if in_place:
            o.copy_(rv)
            rv = o
    want = OB.linear(xv, wv, bv, act, rw)
    L.moe_linear_fp8(x, xs, w, ws, bias=None if bv is None else cuda(bv), act=act, residual=rv, out=o)
    torch.cuda.synchronize()
    a = OB.linear(xv, wv, bv)
    # a block's sum as the FP8 cores make it (KAPPA), three roundings of its two scales, the blocks' fp32 sum
    dev = KAPPA * np.sqrt((xv * xv) @ (wv * wv).T) + (OD.up(K) + 3) * 2.0**-23 * (np.abs(xv) @ np.abs(wv).T) + np.abs(a) * 2.0**-23
    dev = act_deviation(a, dev, act, cols)
    dev = dev + (np.abs(want) + dev) * (2.0**-8 + (2.0**-24 if res else 0)) + 1e-37
    np.testing.assert_array_less(np.abs(values(o) - want), dev * 1.0001)
    assert guard_kept(buf)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 32, 33, 63, 64, 65, 100, 128, 129, 200, 255, 256, 257, 513])
def test_fp8_rows(L, T):
    check_fp8(L, T, 200, 336, bias=True, res="f32")
    check_fp8(L, T, 528, 2048, act="swiglu")


@pytest.mark.parametrize("N", [1, 2, 3, 31, 60, 127, 128, 129, 130, 255, 257, 384, 513])
def test_fp8_columns(L, N):
    """Block rows that end early, gate and up blocks that start off 128."""
    for T in (3, 70, 400):
        check_fp8(L, T, N, 256, bias=True, res="bf16")
        check_fp8(L, T, 2 * N, 256, act="swiglu", bias=True)


@pytest.mark.parametrize("K", [16, 32, 48, 112, 128, 144, 240, 256, 272, 384, 496, 512, 528, 640, 1008, 1040, 2016, 4096, 16384])
def test_fp8_depths(L, K):
    for T in (1, 20, 90, 260):
        check_fp8(L, T, 96, K)


@pytest.mark.parametrize("act", ACTS + ["swiglu"])
def test_fp8_epilogue(L, act):
    for T in (1, 40, 300):
        for bias in (False, True):
            for res in (None, "f32", "bf16"):
                check_fp8(L, T, 264, 256, act=act, bias=bias, res=res)


@pytest.mark.parametrize("T,N,K", [(1024, 1024, 512), (777, 1288, 1056), (2048, 512, 4096), (4100, 256, 256), (300, 4096, 128),
                                   (1990, 4090, 1168), (4001, 4090, 336), (2048, 4096, 272), (2300, 2304, 2320)])
def test_fp8_large(L, T, N, K):
    check_fp8(L, T, N, K, bias=True, res="f32")
    check_fp8(L, T, N, K, act="swiglu", res="bf16", in_place=True)


def test_fp8_offset_and_in_place_outputs(L):
    for T in (3, 50, 300):
        for offset in (1, 2, 4):
            check_fp8(L, T, 136, 128, res="bf16", offset=offset, in_place=True)
            check_fp8(L, T, 137, 128, res="f32", offset=offset)


def test_fp8_scales_of_very_different_size(L):
    """Neighbouring blocks whose scales differ by 2^60, blocks of zeros (scale 0) and zero rows."""
    r = np.random.default_rng(9)
    for T, N in ((5, 64), (70, 300), (400, 512)):
        x, w = r.normal(size=(T, 512)), r.normal(size=(N, 512))
        x[:, :128] *= 2.0**-30
        x[:, 256:384] *= 2.0**30
        w[:, 256:384] *= 2.0**-60
        x[0], w[:, 384:], x[1, 128:256] = 0, 0, 0
        ops = (fp8_operand(L, cuda(x, torch.bfloat16), 1), fp8_operand(L, cuda(w, torch.bfloat16), 128))
        check_fp8(L, T, N, 512, operands=ops)


def test_fp8_rows_do_not_touch_each_other(L):
    """A NaN in a token row, as an element or as a scale, stays in that row, also in the rows the kernels fill up with."""
    for T, N in ((3, 64), (20, 64), (60, 96), (100, 4096), (700, 4096)):
        r = np.random.default_rng(T)
        (x, xs, _), (w, ws, _) = fp8_operand(L, bf16(r, T, 272), 1), fp8_operand(L, bf16(r, N, 272), 128)
        a = L.moe_linear_fp8(x, xs, w, ws).view(torch.bfloat16)
        keep = [t for t in range(T) if t != T // 2]
        for target in (x, xs):
            old = target[T // 2].clone()
            target[T // 2, 1] = 0x7F if target is x else float("nan")
            b = L.moe_linear_fp8(x, xs, w, ws).view(torch.bfloat16)
            assert torch.equal(a[keep], b[keep]) and bool(torch.isnan(b[T // 2]).all())
            target[T // 2] = old


# token rows and weight rows, one for each kernel of the product (few rows: 8, 16, 32 and 64 to a slot; tiles of 64, of 128
# with one and two workgroups to a CU, of 256)
FP8_KERNELS = [(1, 96), (12, 96), (30, 4090), (60, 4096), (200, 2050), (520, 4090), (1100, 4090), (2100, 4090)]


@pytest.mark.parametrize("T,N", FP8_KERNELS)
@pytest.mark.parametrize("size,power", [("small", 132), ("large", -145), ("large", -153)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_fp8_scales_whose_product_leaves_fp32(L, T, N, size, power, act):
    """x_scale * w_scale is about 2^power, beyond the range of fp32 or where it has few bits left; the results are not.
    With SwiGLU so for the up rows, and gates near 1."""
    r = np.random.default_rng([T, abs(power)])
    K, kb = 4 * 128 + 48, 5

    def elements(n):
        # of both signs: the smallest magnitude and zeros, or the largest magnitudes
        q = r.integers(0, 2, size=(n, K)) if size == "small" else r.integers(0x78, 0x7F, size=(n, K))
        return (q | 0x80 * r.integers(0, 2, size=(n, K))).astype(np.uint8)

    def scales(n, e):
        return (r.uniform(1, 2, size=(n, kb)) * 2.0**e).astype(np.float32)

    # the blocks share the power between the sides differently, with subnormal scales among them
    ex = 66 + np.array([0, 20, -10, 10, 7]) if power > 0 else -75 + np.array([0, 20, -15, -60, 7])
    x, xs, w = elements(T), scales(T, ex), elements(N)
    if act == "swiglu":
        near = 15 if size == "small" else -20  # the sums of products are about 2^-near
        ws = np.concatenate([scales(OD.up(N // 2), near - ex), scales(OD.up(N // 2), power - ex)])
    else:
        ws = scales(OD.up(N), power - ex)
    xv, wv = OD.fp8_values(x, xs, 1), OD.fp8_values(w, ws, 128, act == "swiglu")
    want = OB.linear(xv, wv, act_name=act)
    got = values(L.moe_linear_fp8(*(torch.from_numpy(t).cuda() for t in (x, xs, w, ws)), act=act))
    # as in check_fp8; where results are subnormal, half a step of bf16 there, and a step of fp32 for each operation before
    a = OB.linear(xv, wv)
    dev = KAPPA * np.sqrt((xv * xv) @ (wv * wv).T) + (kb + 3) * 2.0**-23 * (np.abs(xv) @ np.abs(wv).T) + 4 * kb * 2.0**-149
    dev = act_deviation(a, dev, act, N // 2)
    dev = dev + (np.abs(want) + dev) * 2.0**-8 + 2.0**-134 + 2.0**-148
    assert 2.0**-133 < np.abs(want).max() < 2.0**127
    np.testing.assert_array_less(np.abs(got - want), dev * 1.0001)


@pytest.mark.parametrize("T,N", FP8_KERNELS)
def test_fp8_zero_sums_under_huge_scales(L, T, N):
    """A block whose products are all zero adds nothing, however large the (finite) scales of both sides are."""
    r = np.random.default_rng(T)
    x, w = r.integers(0, 0x7F, size=(T, 272)).astype(np.uint8), r.integers(0, 0x7F, size=(N, 272)).astype(np.uint8)
    x[:, :128], w[:, 128:] = 0, 0
    xs, ws = np.full((T, 3), 2.0**100, dtype=np.float32), np.full((OD.up(N), 3), 2.0**100, dtype=np.float32)
    got = L.moe_linear_fp8(*(torch.from_numpy(t).cuda() for t in (x, xs, w, ws)))
    assert not got.view(torch.bfloat16).float().abs().max().item()


@pytest.mark.parametrize("T,N", FP8_KERNELS)
def test_fp8_far_scale_of_one_row(L, T, N):
    """A token row with a scale of 2^70 or 2^-70 changes no bit of the other rows, which are summed beside it."""
    r = np.random.default_rng(T)
    (x, xs, _), (w, ws, _) = fp8_operand(L, bf16(r, T, 272), 1), fp8_operand(L, bf16(r, N, 272), 128)
    a = L.moe_linear_fp8(x, xs, w, ws)
    keep = [t for t in range(T) if t != T // 2]
    for power in (70, -70):
        xs[T // 2] = 2.0**power
        b = L.moe_linear_fp8(x, xs, w, ws)
        assert torch.equal(a[keep], b[keep]) and not torch.equal(a[T // 2], b[T // 2])


# ------------------------------------------------------------------ gated projection
def check_glu(L, T, I, K, act, keep=True, scale=1.0):
    r = np.random.default_rng([T, I, K])
    x, w = bf16(r, T, K, scale=scale), bf16(r, 2 * I, K, scale=K**-0.5)
    h, hbuf = guarded((T, I), torch.bfloat16)
    a, abuf = guarded((T, 2 * I), torch.bfloat16) if keep else (None, None)
    L.moe_glu(x, w, act=act, a=a, out=h)
    torch.cuda.synchronize()
    want_h, want_a = OD.glu(values(x), values(w), act)
    dev = min(K * 2.0**-23, 1e-3) * (np.abs(values(x)) @ np.abs(values(w)).T)
    dh = gate_deviation(want_a, dev, act, I)
    np.testing.assert_array_less(np.abs(values(h) - want_h), (dh + (np.abs(want_h) + dh) * 2.0**-8) * 1.0001 + 1e-37)
    assert guard_kept(hbuf)
    if keep:
        np.testing.assert_array_less(np.abs(values(a) - want_a), (dev + (np.abs(want_a) + dev) * 2.0**-8) * 1.0001 + 1e-37)
        assert guard_kept(abuf)


@pytest.mark.parametrize("T", [1, 2, 8, 9, 17, 33, 64, 65, 129, 257, 300])
def test_glu_rows(L, T):
    for act in ACTS:
        check_glu(L, T, 104, 328, act)
    check_glu(L, T, 264, 2048, "silu", keep=False)


@pytest.mark.parametrize("T,I,K", [(5, 8, 8), (3, 16, 40), (70, 24, 72), (400, 8, 136), (1001, 2048, 136), (1001, 504, 1032),
                                   (4096, 2048, 72), (4001, 2040, 328), (512, 2048, 200), (2048, 256, 4096), (300, 40, 5000)])
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_glu_shapes(L, T, I, K, act):
    check_glu(L, T, I, K, act)


def test_glu_far_from_zero(L):
    """The exponential overflows on one side, the result is its limit."""
    for act in ACTS:
        check_glu(L, 40, 64, 64, act, scale=300.0)


def test_glu_is_the_swiglu_product(L):
    """The same sums as moe_linear's, and the kept pre-activations change nothing."""
    r = np.random.default_rng(2)
    for T in (1, 40, 300, 1001):
        x, w = bf16(r, T, 256), bf16(r, 512, 256, scale=1 / 16)
        h = L.moe_glu(x, w)
        assert torch.equal(h, L.moe_linear(x, w, act="swiglu"))
        assert torch.equal(h, L.moe_glu(x, w, a=torch.empty(T, 512, dtype=torch.bfloat16, device="cuda")))


# ------------------------------------------------------------------ gradients
def check_grads(got, want, dev, half, what):
    np.testing.assert_array_less(np.abs(got - want), (dev + (np.abs(want) + dev) * half) * 1.0001 + 1e-37, err_msg=what)


def check_linear_backward(L, T, N, K, dx="bf16", dw="f32", accumulate=False, seed=0):
    r = np.random.default_rng([seed, T, N, K])
    dy, x, w = bf16(r, T, N, scale=0.01), bf16(r, T, K), bf16(r, N, K, scale=K**-0.5)
    gx, xbuf = guarded((T, K), DT[dx])
    gw, wbuf = guarded((N, K), DT[dw])
    before = 0.0
    if accumulate:
        gw.copy_(cuda(r.normal(size=(N, K)) * 0.1, DT[dw]))
        before = values(gw)
    got = L.moe_linear_backward(dy, x, w, dx=gx, dw=gw, accumulate=accumulate)
    torch.cuda.synchronize()
    assert got[0] is gx and got[1] is gw
    y, xv, wv = values(dy), values(x), values(w)
    want_x, want_w = OD.linear_grad(y, xv, wv)
    half = {"f32": 2.0**-24, "bf16": 2.0**-8}
    check_grads(values(gx), want_x, min(N * 2.0**-23, 1e-3) * (np.abs(y) @ np.abs(wv)), half[dx], "dx")
    dev = min((T + 8) * 2.0**-23, 1e-3) * (np.abs(y).T @ np.abs(xv)) + (2.0**-23 * np.abs(before + want_w) if accumulate else 0)
    check_grads(values(gw), before + want_w, dev, half[dw], "dw")
    for name, g, want, n in (("dx", gx, want_x, N), ("dw", gw, want_w, T)):
        if g.dtype == torch.float32 and want.size >= 64 and not accumulate:
            # in the root mean square: n independent roundings of partial sums no larger than the result
            err = np.linalg.norm(values(g) - want) / np.linalg.norm(want)
            assert err <= 2 * 2.0**-24 * (np.sqrt(n) + 2), (name, err)
    assert guard_kept(xbuf) and guard_kept(wbuf)


@pytest.mark.parametrize("T", [1, 2, 3, 7, 8, 15, 16, 17, 31, 63, 64, 65, 127, 129, 200, 255, 257, 513, 1000])
def test_linear_backward_rows(L, T):
    check_linear_backward(L, T, 72, 136, dx="f32")
    check_linear_backward(L, T, 256, 128, dw="bf16")


@pytest.mark.parametrize("N,K", [(8, 8), (8, 256), (16, 24), (40, 1000), (128, 64), (136, 520), (264, 264), (520, 72), (1000, 40),
                                 (2056, 96), (96, 2056), (1024, 1024)])
def test_linear_backward_shapes(L, N, K):
    for T in (5, 130, 700):
        check_linear_backward(L, T, N, K)


@pytest.mark.parametrize("T,N,K", [(4099, 512, 264), (20001, 64, 48), (70000, 8, 16), (300, 4096, 4096), (8192, 1024, 256),
                                   (2048, 2048, 2048), (33, 4104, 136)])
def test_linear_backward_large(L, T, N, K):
    check_linear_backward(L, T, N, K, dx="f32")


@pytest.mark.parametrize("dx", ["f32", "bf16"])
@pytest.mark.parametrize("dw", ["f32", "bf16"])
def test_linear_backward_types_and_accumulation(L, dx, dw):
    for T, N, K in ((3, 64, 64), (300, 264, 136), (4099, 128, 72)):
        for accumulate in (False, True):
            check_linear_backward(L, T, N, K, dx=dx, dw=dw, accumulate=accumulate)


# sizes off every tile for each layout of a gradient call: gradients wanted, tile of dx, whether the sums of dx and of dw are
# split, whether dw's workgroups come first
GRAD_LAYOUTS = [
    ((1001, 1008, 2016), "both", (128, 128), False, False, False),
    ((471, 32, 3600), "both", (128, 128), False, False, True),
    ((3426, 200, 384), "both", (128, 128), False, True, False),
    ((7258, 32, 200), "both", (128, 128), False, True, True),
    ((238, 3400, 328), "both", (128, 128), True, False, False),
    ((260, 3984, 264), "both", (128, 128), True, False, True),
    ((5845, 1752, 72), "both", (128, 128), True, True, False),
    ((8214, 1024, 80), "both", (128, 128), True, True, True),
    ((8243, 32, 216), "dx", (128, 128), False, False, False),
    ((205, 720, 2696), "dw", (128, 128), False, False, True),
    ((5131, 72, 2240), "dw", (128, 128), False, True, True),
    ((341, 664, 3632), "both", (128, 256), False, False, False),
    ((520, 416, 3832), "both", (128, 256), False, False, True),
    ((3721, 200, 648), "both", (128, 256), False, True, False),
    ((7308, 32, 464), "both", (128, 256), False, True, True),
    ((206, 3792, 760), "both", (128, 256), True, False, False),
    ((467, 3416, 728), "both", (128, 256), True, False, True),
    ((8557, 920, 144), "both", (128, 256), True, True, True),
    ((8490, 32, 416), "dx", (128, 256), False, False, False),
    ((8191, 4088, 2040), "dw", (128, 256), False, False, True),
    ((8580, 1480, 648), "dw", (128, 256), False, True, True),
    ((919, 1088, 3984), "both", (256, 256), False, False, False),
    ((8191, 4088, 2040), "both", (256, 256), False, False, True),
    ((16381, 2040, 504), "both", (256, 256), False, True, False),
    ((3408, 32, 2056), "both", (256, 256), False, True, True),
    ((496, 3992, 1304), "both", (256, 256), True, False, False),
    ((8631, 32, 800), "dx", (256, 256), False, False, False),
    ((202, 3384, 2408), "dw", (256, 256), False, False, True),
]


@pytest.mark.parametrize("sizes,need,tile,split_dx,split_dw,dw_first", GRAD_LAYOUTS)
def test_linear_backward_layouts(L, sizes, need, tile, split_dx, split_dw, dw_first):
    """Every layout with tiles wider than 64, of both types and with accumulation, against fp64 products on the GPU."""
    T, N, K = sizes
    nx, nw = need != "dw", need != "dx"
    lay = L.moe_debug_grad_tiles(T, N, K, nx, nw)
    assert (lay["tile"], lay["splits_dx"] > 1, lay["splits_dw"] > 1, lay["dw_first"]) == (tile, split_dx, split_dw, dw_first)
    gen = torch.Generator(device="cuda").manual_seed(T + N + K)
    normal = lambda *shape, scale: (scale * torch.randn(*shape, generator=gen, device="cuda")).bfloat16()
    dy, x, w = normal(T, N, scale=0.01), normal(T, K, scale=1.0), normal(N, K, scale=K**-0.5)
    y64, x64, w64 = dy.double(), x.double(), w.double()
    yt = y64.t().contiguous()
    half = {"f32": 2.0**-24, "bf16": 2.0**-8}

    def check(got, want, dev, dtype):
        dev = (dev + (want.abs() + dev) * half[dtype]) * 1.0001 + 1e-37
        assert bool(((got.double() - want).abs() <= dev).all()), (dtype, float(((got.double() - want).abs() / dev).max()))

    if nx:
        want_x, dev_x = y64 @ w64, min(N * 2.0**-23, 1e-3) * (y64.abs() @ w64.abs())
    if nw:
        want_w, dev_w = yt @ x64, min((T + 8) * 2.0**-23, 1e-3) * (yt.abs() @ x64.abs())
    for tx, tw, accumulate in (("bf16", "bf16", False), ("f32", "f32", True), ("bf16", "f32", False), ("f32", "bf16", True)):
        gx, xbuf = guarded((T, K), DT[tx]) if nx else (None, None)
        gw, wbuf = guarded((N, K), DT[tw]) if nw else (None, None)
        before = normal(N, K, scale=0.1)
        if nw and accumulate:
            gw.copy_(before)
        L.moe_linear_backward(dy, x if nw else None, w if nx else None, dx=gx, dw=gw, need_dx=nx, need_dw=nw,
                              accumulate=accumulate and nw)
        torch.cuda.synchronize()
        if nx:
            check(gx, want_x, dev_x, tx)
            assert guard_kept(xbuf)
        if nw:
            total = want_w + before.double() if accumulate else want_w
            check(gw, total, dev_w + 2.0**-23 * total.abs() if accumulate else dev_w, tw)
            assert guard_kept(wbuf)


@pytest.mark.parametrize("T,I,K,tile", [(1001, 504, 2016, (128, 128)), (341, 336, 3632, (128, 256)), (919, 544, 3984, (256, 256))])
def test_glu_backward_wide_tiles(L, T, I, K, tile):
    assert L.moe_debug_grad_tiles(T, 2 * I, K)["tile"] == tile
    for dw, accumulate in (("bf16", False), ("f32", True)):
        check_glu_backward(L, T, I, K, "gelu", dw=dw, accumulate=accumulate)


def test_calls_of_no_rows(L):
    e = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        dw = torch.full((24, 40), 3.0, dtype=dtype, device="cuda")
        L.moe_linear_backward(e(0, 24), e(0, 40), e(24, 40), dw=dw, accumulate=True)
        assert bool((dw == 3).all())
        L.moe_linear_backward(e(0, 24), e(0, 40), e(24, 40), dw=dw)
        assert not bool(dw.any())
        dw.fill_(3.0)
        dx, _ = L.moe_glu_backward(e(0, 12 * 8), e(0, 24 * 8), e(0, 40), e(24 * 8, 40), dw=torch.ones(24 * 8, 40, device="cuda"))
        assert dx.shape == (0, 40)
    # dx alone: nothing to do
    assert L.moe_linear_backward(e(0, 24), None, e(24, 40), need_dw=False)[0].shape == (0, 40)
    assert L.moe_glu_backward(e(0, 24), e(0, 48), None, e(48, 40), need_dw=False)[0].shape == (0, 40)
    for act in ACTS:
        assert L.moe_glu(e(0, 64), e(48, 64), act=act).shape == (0, 24)
    q, s = L.moe_fp8_quantize(e(0, 272))
    w, ws = L.moe_fp8_quantize(torch.randn(40, 272, device="cuda"), 128)
    assert q.shape == (0, 272) and s.shape == (0, 3) and L.moe_linear_fp8(q, s, w, ws).shape == (0, 40)
    q, s = L.moe_fp8_quantize(e(0, 272), block_rows=128)
    assert q.shape == (0, 272) and s.shape == (0, 3)


def test_linear_backward_needs(L):
    """One gradient alone, without the operand that only the other reads, and the same bits."""
    r = np.random.default_rng(4)
    dy, x, w = bf16(r, 300, 72), bf16(r, 300, 136), bf16(r, 72, 136)
    dx, dw = L.moe_linear_backward(dy, x, w)
    assert L.moe_linear_backward(dy, None, w, need_dw=False)[1] is None
    assert torch.equal(L.moe_linear_backward(dy, None, w, need_dw=False)[0], dx)
    assert torch.equal(L.moe_linear_backward(dy, x, None, need_dx=False)[1], dw)


def check_glu_backward(L, T, I, K, act, dw="bf16", scale=1.0, accumulate=False):
    r = np.random.default_rng([T, I, K])
    dh, a = bf16(r, T, I, scale=0.01), bf16(r, T, 2 * I, scale=scale)
    x, w = bf16(r, T, K), bf16(r, 2 * I, K, scale=K**-0.5)
    gx, xbuf = guarded((T, K), torch.bfloat16)
    gw, wbuf = guarded((2 * I, K), DT[dw])
    gw.copy_(cuda(r.normal(size=(2 * I, K)) * 0.1, DT[dw]))
    before = values(gw) if accumulate else 0.0
    L.moe_glu_backward(dh, a, x, w, act=act, dx=gx, dw=gw, accumulate=accumulate)
    torch.cuda.synchronize()
    d, av, xv, wv = values(dh), values(a), values(x), values(w)
    da = OD.glu_grad(d, av, act)
    want_x, want_w = OD.linear_grad(da, xv, wv)
    # the slope p + g p (1 - p) z': p's relative error (3 |z| + 8) 2^-23 acts on both terms, the second's size is at most
    # |g| z' p; then da's three products and its rounding to bf16, and the sums
    g, u = av[:, :I], av[:, I:]
    size = np.abs(g) + (0.1 * np.abs(g) ** 3 if act == "gelu" else 0)
    dz = 1.6 * (1 + 0.1342 * g * g) if act == "gelu" else 1.0
    e = (3 * size + 12) * 2.0**-23 if act in ("gelu", "silu") else 0.0
    p_far = np.where(g < -15, 0.0, 1.0)  # p |g|^3 < 1e-3 there, nothing is left of it
    dda = np.concatenate([np.abs(d * u) * e * (1 + np.abs(g) * dz) * np.maximum(p_far, 1e-3), np.abs(da[:, I:]) * e], axis=1)
    dda = dda + np.abs(da) * (2.0**-8 + 2.0**-22) + 1e-40
    mag = np.abs(da) + dda
    check_grads(values(gx), want_x, dda @ np.abs(wv) + min(2 * I * 2.0**-23, 1e-3) * (mag @ np.abs(wv)), 2.0**-8, "dx")
    dev = dda.T @ np.abs(xv) + min((T + 8) * 2.0**-23, 1e-3) * (mag.T @ np.abs(xv))
    if accumulate:
        dev = dev + 2.0**-23 * np.abs(before + want_w)
    check_grads(values(gw), before + want_w, dev, 2.0**-24 if dw == "f32" else 2.0**-8, "dw")
    if not accumulate:
        # in the root mean square: the rounding of da (2^-8 at most, independent from value to value), then of the result
        for name, got, want in (("dx", gx, want_x), ("dw", gw, want_w)):
            if want.size >= 64:
                err = np.linalg.norm(values(got) - want) / np.linalg.norm(want)
                assert err <= 1.5 * 2.0**-8, (name, err)
    assert guard_kept(xbuf) and guard_kept(wbuf)


@pytest.mark.parametrize("T,I,K", [(1, 8, 8), (1, 512, 2048), (3, 24, 40), (17, 64, 128), (64, 104, 72), (257, 40, 264), (1001, 504, 136),
                                   (700, 136, 1032), (4099, 64, 64), (2048, 1024, 256)])
@pytest.mark.parametrize("act", ACTS)
def test_glu_backward(L, T, I, K, act):
    check_glu_backward(L, T, I, K, act)


def test_glu_backward_accumulates(L):
    for dw in ("f32", "bf16"):
        check_glu_backward(L, 300, 64, 72, "silu", dw=dw, accumulate=True)
        check_glu_backward(L, 300, 64, 72, "gelu", dw=dw)


@pytest.mark.parametrize("act", ACTS)
def test_glu_backward_far_from_zero(L, act):
    check_glu_backward(L, 130, 64, 72, act, scale=60.0)


def test_glu_backward_extreme_activations(L):
    """Gates as large as bf16 has them: the slopes are their limits, nothing is NaN."""
    g = torch.tensor([-3.0e38, -1e30, -1e19, -100.0, 0.0, 100.0, 1e19, 1e30, 3.0e38] + [1.0] * 7, device="cuda")
    a = torch.cat([g, torch.full((16,), 0.5, device="cuda")])[None].bfloat16()
    dh = torch.full((1, 16), 1e-3, device="cuda").bfloat16()
    x, w = torch.ones(1, 8, device="cuda").bfloat16(), torch.ones(32, 8, device="cuda").bfloat16()
    for act in ACTS:
        dw = L.moe_glu_backward(dh, a, x, w, act=act, need_dx=False, dw=torch.empty(32, 8, device="cuda"))[1]
        with np.errstate(all="ignore"):
            av = values(a)
            want = OD.glu_grad(values(dh), np.clip(av, -1e4, 1e4), act)[0]  # the slopes' limits
            want[16:] = values(dh)[0] * OB.act(np.where(av[0, :16] < -1e4, -1e4 if act != "none" else av[0, :16], av[0, :16]), act) \
                if act != "gelu" else values(dh)[0] * np.where(np.abs(av[0, :16]) > 50, np.maximum(av[0, :16], 0), OB.act(av[0, :16], act))
        got = values(dw)[:, 0]
        assert np.isfinite(got).all(), act
        np.testing.assert_allclose(got, want, rtol=2.0**-8 + 1e-5, atol=1e-12)


# ------------------------------------------------------------------ together, graphs, streams
def test_shared_expert_in_fp8(L):
    """The shared expert as it is served: quantised weights and activations, FC1 with SwiGLU, FC2 with the routed output."""
    r = np.random.default_rng(11)
    H, I = 512, 384
    w1, w2 = fp8_operand(L, bf16(r, 2 * I, H, scale=H**-0.5), 128, True), fp8_operand(L, bf16(r, H, I, scale=I**-0.5), 128)
    for T in (1, 50, 300):
        y, routed = bf16(r, T, H), cuda(r.normal(size=(T, H)))
        q, s = L.moe_fp8_quantize(y)
        h = L.moe_linear_fp8(q, s, w1[0], w1[1], act="swiglu")
        hq, hs = L.moe_fp8_quantize(h)
        out = L.moe_linear_fp8(hq, hs, w2[0], w2[1], residual=routed)
        torch.cuda.synchronize()
        # each call on what the one before gave
        want_h = OB.linear(OD.fp8_values(host(q), host(s), 1), w1[2], act_name="swiglu")
        assert np.linalg.norm(values(h) - want_h) <= (2.0**-8 + 3 * KAPPA) * np.linalg.norm(want_h)
        wq, wsc = OD.fp8_quantize(values(h), 1)
        assert np.array_equal(host(hs), wsc) and np.array_equal(host(hq) & 0x7F, wq & 0x7F)
        want = OB.linear(OD.fp8_values(host(hq), host(hs), 1), w2[2], residual=values(routed))
        assert np.linalg.norm(values(out) - want) <= (2.0**-8 + KAPPA) * np.linalg.norm(want)
        # and the whole against the unquantised expert: e4m3 steps of 2^-4, at most half of them everywhere
        full = OB.linear(OB.linear(values(y), w1[2], act_name="swiglu"), w2[2], residual=values(routed))
        assert np.linalg.norm(values(out) - full) <= 2.0**-4 * np.linalg.norm(full)


def expert_step(L, x, w1, w2, dout, bufs):
    """Forward and backward of a shared expert in bf16: what a training step does with it."""
    L.moe_glu(x, w1, a=bufs["a"], out=bufs["h"])
    L.moe_linear(bufs["h"], w2, out=bufs["y"])
    L.moe_linear_backward(dout, bufs["h"], w2, dx=bufs["dh"], dw=bufs["dw2"])
    L.moe_glu_backward(bufs["dh"], bufs["a"], x, w1, dx=bufs["dx"], dw=bufs["dw1"])


def expert_buffers(T, H, I):
    e = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device="cuda")
    return dict(a=e(T, 2 * I), h=e(T, I), y=e(T, H), dh=e(T, I), dx=e(T, H), dw1=e(2 * I, H, dtype=torch.float32),
                dw2=e(H, I, dtype=torch.float32))


def test_shared_expert_training_step(L):
    r = np.random.default_rng(12)
    T, H, I = 300, 264, 136
    x, w1, w2, dout = bf16(r, T, H), bf16(r, 2 * I, H, scale=H**-0.5), bf16(r, H, I, scale=I**-0.5), bf16(r, T, H, scale=0.01)
    b = expert_buffers(T, H, I)
    expert_step(L, x, w1, w2, dout, b)
    torch.cuda.synchronize()
    h, a = OD.glu(values(x), values(w1), "silu")
    dh, dw2 = OD.linear_grad(values(dout), h, values(w2))
    dx, dw1 = OD.linear_grad(OD.glu_grad(dh, a, "silu"), values(x), values(w1))
    # every link rounds its result to bf16 (2^-8 of the value at most) and no gradient has more than four such links
    for name, want in (("y", OB.linear(h, values(w2))), ("dw2", dw2), ("dx", dx), ("dw1", dw1)):
        err = np.linalg.norm(values(b[name]) - want) / np.linalg.norm(want)
        assert err <= 4 * 2.0**-8, (name, err)


def all_calls(L, T=150, seed=0):
    """A call of every operator, and its outputs."""
    r = np.random.default_rng(seed)
    H, I = 272, 136
    x, w1, w2 = bf16(r, T, H), bf16(r, 2 * I, H, scale=H**-0.5), bf16(r, H, I, scale=I**-0.5)
    dout = bf16(r, T, H, scale=0.01)
    (q1, s1, _), b = fp8_operand(L, w1, 128, True), expert_buffers(T, H, I)
    b.update(q=torch.empty(T, H, dtype=torch.uint8, device="cuda"), s=torch.empty(T, 3, device="cuda"),
             o=torch.empty(T, I, dtype=torch.bfloat16, device="cuda"))

    def run():
        L.moe_fp8_quantize(x, q=b["q"], scales=b["s"])
        L.moe_linear_fp8(b["q"], b["s"], q1, s1, act="swiglu", out=b["o"])
        expert_step(L, x, w1, w2, dout, b)

    return run, b, x


def test_captured_calls(L):
    """Captured once and replayed on new inputs, with eager work and synchronisation between the replays."""
    for T in (1, 40, 300):
        run, b, x = all_calls(L, T)
        run()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            run()
        for i in range(4):
            x.copy_(bf16(np.random.default_rng(100 + i), *x.shape))
            for t in b.values():
                t.fill_(7)
            graph.replay()
            torch.cuda.synchronize()
            got = {k: t.clone() for k, t in b.items()}
            run()
            torch.cuda.synchronize()
            for k in b:
                assert torch.equal(got[k], b[k]), (T, i, k)


def test_two_graphs_and_another_stream(L):
    """Two captured graphs replayed on two streams at once, each with workspaces of its own."""
    runs = [all_calls(L, T, seed) for T, seed in ((200, 1), (333, 2))]
    graphs, streams, want = [], [torch.cuda.Stream(), torch.cuda.Stream()], []
    for (run, b, _), stream in zip(runs, streams):
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            run()
        stream.synchronize()
        want.append({k: t.clone() for k, t in b.items()})
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            run()
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for _, b, _ in runs:
            for t in b.values():
                t.fill_(7)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (_, b, _), w in zip(runs, want):
            for k in b:
                assert torch.equal(b[k], w[k]), k


def test_split_sums_captured(L):
    """Gradients whose parts lie in a workspace, captured with one of their own and with a given one that holds NaN."""
    r = np.random.default_rng(21)
    for T, N, K in ((3426, 200, 384), (206, 3792, 760), (8214, 1024, 80)):
        lay = L.moe_debug_grad_tiles(T, N, K)
        assert lay["splits_dx"] > 1 or lay["splits_dw"] > 1
        dy, x, w = bf16(r, T, N, scale=0.01), bf16(r, T, K), bf16(r, N, K, scale=K**-0.5)
        dx, dw = torch.empty(T, K, device="cuda"), torch.zeros(N, K, device="cuda")
        ws = torch.empty(L.lib.moe_linear_backward_ws_bytes(T, N, K) + 4096, dtype=torch.uint8, device="cuda")
        graphs = []
        for given in (None, ws):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                L.moe_linear_backward(dy, x, w, dx=dx, dw=dw, accumulate=True, ws=given)
            graphs.append(g)
        for i in range(3):
            dy.copy_(bf16(r, T, N, scale=0.01))
            want = L.moe_linear_backward(dy, x, w, dx=torch.empty_like(dx), dw=torch.ones_like(dw), accumulate=True)
            torch.cuda.synchronize()
            for g in graphs:
                ws.fill_(0xFF)
                dx.fill_(7)
                dw.fill_(1)
                g.replay()
                torch.cuda.synchronize()
                assert torch.equal(dx, want[0]) and torch.equal(dw, want[1]), (T, N, K, i)


def test_gradients_of_one_tensor_twice(L):
    """dy, x and w may be one array, or parts of one that overlap."""
    r = np.random.default_rng(22)
    big = bf16(r, 1000, 136)
    for a, x, w in ((big[8:144], big[8:144], big[8:144]), (big[:700], big[16:716], big[3:139])):
        dx, dw = L.moe_linear_backward(a, x, w)
        ex, ew = L.moe_linear_backward(a.clone(), x.clone(), w.clone())
        assert torch.equal(dx, ex) and torch.equal(dw, ew)


def test_same_bits_on_every_call(L):
    for T in (3, 150, 700):
        run, b, _ = all_calls(L, T)
        run()
        first = {k: t.clone() for k, t in b.items()}
        for _ in range(3):
            run()
            for k in b:
                assert torch.equal(b[k], first[k]), (T, k)


# ------------------------------------------------------------------ the block with a block-scaled FP8 shared expert
def block_fp8(L, Is=144):
    sp, dw = device_layer("tiny")
    H, E = sp["H"], sp["E"]
    r = np.random.default_rng(43)
    w1, w2 = fp8_operand(L, bf16(r, 2 * Is, H, scale=H**-0.5), 128, True), fp8_operand(L, bf16(r, H, Is, scale=Is**-0.5), 128)
    wn, wr = cuda(1 + 0.1 * r.normal(size=H), torch.bfloat16), bf16(r, E, H, scale=1 / 16)
    blk = L.MoeBlock(dw, sp["k"], wn, wr, route=dict(score="sigmoid"), ws1=w1[:2], ws2=w2[:2])
    return H, blk, L.MoeBlock(dw, sp["k"], wn, wr, route=dict(score="sigmoid")), w1[2], w2[2]


@pytest.mark.parametrize("T", [0, 1, 16, 130])
@pytest.mark.parametrize("Is", [144, 256])
def test_block(L, T, Is):
    """The shared expert's part on the block's own norm and routed sum; the rest as without one."""
    H, blk, bare, v1, v2 = block_fp8(L, Is)
    r = np.random.default_rng(T)
    x, res = cuda(r.normal(size=(T, H))), bf16(r, T, H)
    res2 = res.clone()
    o, plain = L.block_forward(blk, x, res), L.block_forward(bare, x, res2)
    torch.cuda.synchronize()
    for k in ("y", "logits", "ids", "gates", "perm", "routed"):
        assert torch.equal(o[k], plain[k]), k
    assert torch.equal(res, res2) and o["out"].shape == (T, H)
    if T == 0:
        return
    q, s = OD.fp8_quantize(values(o["y"]), 1)
    np.testing.assert_array_equal(host(o["q_scales"]), s)
    h = OB.linear(OD.fp8_values(q, s, 1), v1, act_name="swiglu")
    hv = values(o["h"])
    # a rounding to bf16, and the FP8 cores' sums through the gate (their KAPPA on both halves)
    assert np.linalg.norm(hv - h) <= (2.0**-8 + 3 * KAPPA) * np.linalg.norm(h)
    out = OB.linear(OD.fp8_values(*OD.fp8_quantize(hv, 1), 1), v2, residual=values(o["routed"]))
    assert np.linalg.norm(values(o["out"]) - out) <= (2.0**-8 + KAPPA) * np.linalg.norm(out)


def test_block_captured(L):
    H, blk, _, _, _ = block_fp8(L)
    x, res = torch.randn(40, H, device="cuda"), torch.randn(40, H, device="cuda").bfloat16()
    L.block_forward(blk, x.clone(), res.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = L.block_forward(blk, x, res)
    for i in range(4):
        x.copy_(torch.randn(40, H, device="cuda"))
        res.copy_(torch.randn(40, H, device="cuda").bfloat16())
        eager = res.clone()
        graph.replay()
        torch.cuda.synchronize()
        got = captured["out"].clone()
        want = L.block_forward(blk, x, eager)
        torch.cuda.synchronize()
        assert torch.equal(got, want["out"]) and torch.equal(res, eager)


# ------------------------------------------------------------------ types, differences
def test_types_of_the_tensors(L):
    """bf16 as its bits and e4m3 elements as that type: the same bits."""
    r = np.random.default_rng(5)
    x, w = bf16(r, 70, 144), bf16(r, 2 * 40, 144, scale=1 / 12)
    q, s = L.moe_fp8_quantize(x)
    q2, s2 = L.moe_fp8_quantize(x.view(torch.int16), q=torch.empty(70, 144, dtype=torch.float8_e4m3fn, device="cuda"))
    assert torch.equal(q, q2.view(torch.uint8)) and torch.equal(s, s2)
    wq, ws = L.moe_fp8_quantize(w, 128)
    out = L.moe_linear_fp8(q, s, wq, ws)
    same = L.moe_linear_fp8(q2, s, wq.view(torch.float8_e4m3fn), ws, out=torch.empty(70, 80, dtype=torch.bfloat16, device="cuda"))
    assert out.dtype == torch.int16 and torch.equal(out, same.view(torch.int16))
    a = torch.empty(70, 80, dtype=torch.int16, device="cuda")
    h = L.moe_glu(x.view(torch.int16), w, a=a)
    a2 = torch.empty(70, 80, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(h, L.moe_glu(x, w.view(torch.int16), a=a2)) and torch.equal(a, a2.view(torch.int16))
    dx, dw = L.moe_glu_backward(h, a, x, w)
    ex, ew = L.moe_glu_backward(h.view(torch.bfloat16), a2, x.view(torch.int16), w.view(torch.int16),
                                dx=torch.empty(70, 144, dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(dx, ex.view(torch.int16)) and torch.equal(dw, ew)


@pytest.mark.parametrize("T,I,K", [(9, 24, 40), (130, 72, 136)])
def test_glu_gradient_against_differences(L, T, I, K):
    """Without an activation h is quadratic in x and in w, so central differences have no error of their own: the
    change of sum(dh h) along a direction is the gradient's product with it."""
    r = np.random.default_rng([T, I])
    grid = lambda *s: cuda(r.integers(-8, 9, size=s) / 8.0, torch.bfloat16)  # sums and differences are bf16 values again
    x, w, ex, ew, dh = grid(T, K), grid(2 * I, K), grid(T, K), grid(2 * I, K), grid(T, I)
    a = torch.empty(T, 2 * I, dtype=torch.bfloat16, device="cuda")
    L.moe_glu(x, w, act="none", a=a)
    dx, dw = L.moe_glu_backward(dh, a, x, w, act="none", dx=torch.empty(T, K, device="cuda"),
                                dw=torch.empty(2 * I, K, device="cuda"))
    d = values(dh)
    for grad, e, of in ((dx, ex, lambda s: L.moe_glu(x + s * ex, w, act="none")),
                        (dw, ew, lambda s: L.moe_glu(x, w + s * ew, act="none"))):
        hi, lo = values(of(1)), values(of(-1))
        want, got = float(((hi - lo) * d).sum()) / 2, float((values(grad) * values(e)).sum())
        # h is rounded to bf16, the kept a and the gradient of a too: a 2^-8 of each term of the sums
        av, ev = values(a), values(e)
        if e is ex:
            moved = np.abs(ev) @ np.abs(values(w)).T
        else:
            moved = np.abs(values(x)) @ np.abs(ev).T
        terms = np.abs(d) * (np.abs(av[:, I:]) * moved[:, :I] + np.abs(av[:, :I]) * moved[:, I:])
        bound = 2.0**-8 * ((np.abs(hi) + np.abs(lo)) * np.abs(d)).sum() / 2 + 2 * 2.0**-8 * terms.sum() * 1.01
        assert abs(want - got) <= bound
        # and much nearer where the roundings, being independent, cancel
        assert abs(want - got) <= 8 * 2.0**-8 * (np.sqrt((((np.abs(hi) + np.abs(lo)) * d) ** 2).sum()) + np.sqrt((terms**2).sum()))
