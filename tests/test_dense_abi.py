"""Refusals of the FP8 block-scaled product and its quantiser, the gated projection and the gradient calls: every
check fails on the host before anything is enqueued, so no GPU is needed; and the binding's own checks."""
import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from bit_moe_expert_top_amd import _lib

    return _lib


def at(i):
    """A 4096-byte aligned address that is never dereferenced, 16 MiB from the others."""
    return (i + 1) << 24


X, XS, W, WS, B, R, O, A, D, DX, DW, S = (at(i) for i in range(12))


def quantize(L, x=X, dt=2, rows=4, K=64, by=1, q=O, s=XS):
    return L.lib.moe_fp8_quantize(x, dt, rows, K, by, q, s, None)


@pytest.mark.parametrize("bad,want", [
    (dict(rows=-1), -1), (dict(K=0), -1), (dict(dt=3), -1), (dict(dt=0), -1), (dict(by=0), -1), (dict(by=64), -1),
    (dict(K=72), -2), (dict(K=(1 << 20) + 16), -2), (dict(rows=(1 << 26) + 1), -2), (dict(rows=1 << 26, K=4096), -2), (dict(x=None), -1), (dict(q=None), -1),
    (dict(s=None), -1), (dict(x=X + 8), -1), (dict(q=O + 4), -1), (dict(s=XS + 2), -1),
    (dict(q=X), -1), (dict(q=X + 504), -1), (dict(s=X + 4), -1), (dict(s=O + 252), -1),
])
def test_quantize_refusals(L, bad, want):
    assert quantize(L, **bad) == want


@pytest.mark.parametrize("rows,by,want", [(1 << 18, 1, -2), ((1 << 18) - 1, 128, -2), ((1 << 18) - 127, 128, -2),
                                          ((1 << 18) - 128, 128, -1), ((1 << 18) - 1, 1, -1)])
def test_quantize_block_counts(L, rows, by, want):
    """The largest counts of blocks: below them the call gets as far as the missing arrays."""
    assert quantize(L, x=None, rows=rows, K=1 << 20, by=by) == want


def fp8(L, x=X, xs=XS, w=W, ws=WS, T=4, N=64, K=64, bias=B, act=0, r=R, rd=1, out=O):
    return L.lib.moe_linear_fp8(x, xs, w, ws, T, N, K, bias, act, r, rd, out, None)


@pytest.mark.parametrize("bad,want", [
    (dict(T=-1), -1), (dict(N=0), -1), (dict(K=0), -1), (dict(act=-1), -1), (dict(act=5), -1), (dict(rd=3), -1),
    (dict(act=4, N=63), -1), (dict(K=72), -2), (dict(K=(1 << 20) + 16), -2), (dict(N=(1 << 20) + 1), -2),
    (dict(T=(1 << 26) + 1), -2), (dict(x=None), -1), (dict(xs=None), -1), (dict(w=None), -1), (dict(ws=None), -1),
    (dict(out=None), -1), (dict(x=X + 8), -1), (dict(w=W + 4), -1), (dict(xs=XS + 2), -1), (dict(ws=WS + 1), -1),
    (dict(bias=B + 2), -1), (dict(out=O + 1), -1), (dict(r=R + 2), -1), (dict(r=O), -1), (dict(r=O + 2, rd=2), -1),
    (dict(out=X), -1), (dict(out=W + 4094), -1), (dict(out=XS + 14), -1), (dict(out=WS), -1), (dict(out=B + 254), -1),
])
def test_fp8_product_refusals(L, bad, want):
    assert fp8(L, **bad) == want


def glu(L, x=X, w=W, T=4, I=64, K=64, act=3, a=A, h=O):
    return L.lib.moe_glu(x, w, T, I, K, act, a, h, None)


@pytest.mark.parametrize("bad,want", [
    (dict(T=-1), -1), (dict(I=0), -1), (dict(K=-8), -1), (dict(act=4), -1), (dict(act=-1), -1), (dict(K=60), -2),
    (dict(I=60), -2), (dict(K=(1 << 20) + 8), -2), (dict(I=(1 << 19) + 8), -2), (dict(T=(1 << 26) + 1), -2),
    (dict(x=None), -1), (dict(w=None), -1), (dict(h=None), -1), (dict(x=X + 8), -1), (dict(w=W + 8), -1),
    (dict(h=O + 8), -1), (dict(a=A + 8), -1), (dict(a=X), -1), (dict(h=X), -1), (dict(h=A + 128), -1), (dict(h=W + 64), -1),
])
def test_glu_refusals(L, bad, want):
    assert glu(L, **bad) == want


def linear_backward(L, dy=D, x=X, w=W, T=4, N=64, K=64, dx=DX, dxt=2, dw=DW, dwt=1, acc=0, ws=S, n=1 << 22):
    return L.lib.moe_linear_backward(dy, x, w, T, N, K, dx, dxt, dw, dwt, acc, ws, n, None)


def glu_backward(L, dh=D, a=A, x=X, w=W, T=4, I=64, K=64, act=3, dx=DX, dxt=2, dw=DW, dwt=1, acc=0, ws=S, n=1 << 22):
    return L.lib.moe_glu_backward(dh, a, x, w, T, I, K, act, dx, dxt, dw, dwt, acc, ws, n, None)


GRAD_BAD = [
    (dict(T=-1), -1), (dict(K=0), -1), (dict(K=60), -2), (dict(K=(1 << 20) + 8), -2), (dict(T=1 << 30), -2), (dict(dxt=3), -1),
    (dict(dwt=0), -1), (dict(dx=None, dw=None), -1), (dict(x=None), -1), (dict(w=None), -1), (dict(x=X + 8), -1),
    (dict(w=W + 2), -1), (dict(dx=DX + 8), -1), (dict(dw=DW + 8), -1), (dict(dx=X), -1), (dict(dx=W), -1), (dict(dw=W + 64), -1), (dict(dx=D), -1), (dict(dw=DX + 16), -1),
    (dict(dw=S), -1), (dict(dx=S + 4096), -1),
]


@pytest.mark.parametrize("bad,want", GRAD_BAD + [(dict(N=0), -1), (dict(N=60), -2), (dict(N=(1 << 20) + 8), -2),
                                                 (dict(dy=None), -1), (dict(dy=D + 8), -1)])
def test_linear_backward_refusals(L, bad, want):
    assert linear_backward(L, **bad) == want


@pytest.mark.parametrize("bad,want", GRAD_BAD + [
    (dict(I=0), -1), (dict(I=60), -2), (dict(I=(1 << 19) + 8), -2), (dict(act=4), -1), (dict(act=-1), -1), (dict(dh=None), -1),
    (dict(a=None), -1), (dict(dh=D + 8), -1), (dict(a=A + 8), -1), (dict(dw=A), -1), (dict(ws=A), -1), (dict(ws=D), -1),
    (dict(ws=S + 8), -1), (dict(ws=None), -1), (dict(n=16), -3)])
def test_glu_backward_refusals(L, bad, want):
    assert glu_backward(L, **bad) == want


@pytest.mark.parametrize("call", [linear_backward, glu_backward])
@pytest.mark.parametrize("ws", [X, W, D, X + 256, W - (1 << 21), DX, DW])
def test_workspace_apart(L, call, ws):
    """The workspace is written before or while the inputs are read: it may share bytes with no array."""
    assert call(L, ws=ws) == -1


def test_of_no_rows(L):
    assert quantize(L, rows=0, x=None, q=None, s=None) == 0
    assert fp8(L, T=0, x=None, xs=None, w=None, ws=None, out=None) == 0
    assert glu(L, T=0, x=None, w=None, h=None) == 0
    assert linear_backward(L, T=0, dy=None, x=None, w=None, dx=None, dw=None, ws=None, n=0) == 0
    assert glu_backward(L, T=0, dh=None, a=None, x=None, w=None, dx=None, dw=None, ws=None, n=0) == 0


def test_workspace_sizes(L):
    """A byte less than the call needs is refused; long sums of few outputs are split and need one, whole tiles do not."""
    n = L.lib.moe_linear_backward_ws_bytes(16384, 512, 256)
    assert n > 0 and L.lib.moe_linear_backward_ws_bytes(8192, 4096, 4096) == 0
    far = dict(dy=at(100), x=at(200), w=at(300), dx=at(400), dw=at(500), ws=at(600))
    assert linear_backward(L, T=16384, N=512, K=256, n=n - 1, **far) == -3
    assert linear_backward(L, T=16384, N=512, K=256, n=n, **{**far, "ws": at(600) + 8}) == -1
    for T, I, K in ((1, 64, 64), (4099, 1024, 512), (16384, 256, 256)):
        n = L.lib.moe_glu_backward_ws_bytes(T, I, K)
        assert n >= 4 * T * I + L.lib.moe_linear_backward_ws_bytes(T, 2 * I, K)
        assert glu_backward(L, T=T, I=I, K=K, n=n - 1, dh=at(100), x=at(200), w=at(300), dx=at(400), dw=at(500), ws=at(600),
                            a=at(700)) == -3
    assert L.lib.moe_glu_backward_ws_bytes(0, 64, 64) == 0
    for bad in ((-1, 8, 8), (4, 12, 8), (4, 8, 12), (4, 0, 8), (4, 8, 1 << 21)):
        assert L.lib.moe_linear_backward_ws_bytes(*bad) == 0
    for bad in ((-1, 8, 8), (4, 12, 8), (4, 8, 12), (4, 1 << 30, 8)):
        assert L.lib.moe_glu_backward_ws_bytes(*bad) == 0


@pytest.mark.parametrize("bad,want", [((0, 8, 8, 3), -1), ((4, 0, 8, 3), -1), ((4, 8, -8, 3), -1), ((4, 8, 8, 0), -1),
                                      ((4, 8, 8, 4), -1), ((4, 12, 8, 3), -2), ((4, 8, 1 << 21, 3), -2)])
def test_grad_tiles_refusals(L, bad, want):
    import ctypes

    v = (ctypes.c_int32 * 5)()
    assert L.lib.moe_debug_grad_tiles(*bad, v) == want
    assert L.lib.moe_debug_grad_tiles(4, 8, 8, 3, None) == -1


def test_grad_tiles(L):
    """What the layout says of the workspace: fp32 parts of the split sums, none without."""
    assert L.moe_debug_grad_tiles(8192, 4096, 4096) == dict(tile=(256, 256), splits_dx=1, splits_dw=1, dw_first=True)
    for T, N, K in ((16384, 512, 256), (3426, 200, 384), (1, 4096, 4096)):
        parts = 0
        for dx, dw in ((True, True), (True, False), (False, True)):
            lay = L.moe_debug_grad_tiles(T, N, K, dx, dw)
            n = (lay["splits_dx"] * T * K if lay["splits_dx"] > 1 else 0) + (lay["splits_dw"] * N * K if lay["splits_dw"] > 1 else 0)
            parts = max(parts, 4 * n)
        assert L.lib.moe_linear_backward_ws_bytes(T, N, K) == parts


def test_given_workspace_is_not_sized(L):
    ws = torch.empty(64, dtype=torch.uint8)
    asked = []
    size = lambda *sizes: asked.append(sizes) or 32
    assert L._grad_ws(ws, size, ws.device, 1, 2, 3) == (ws, ws.data_ptr(), 64) and not asked
    got = L._grad_ws(None, size, ws.device, 1, 2, 3)
    assert got[0].shape == (32,) and got[1:] == (got[0].data_ptr(), 32) and asked == [(1, 2, 3)]
    assert L._grad_ws(None, lambda: 0, ws.device) == (None, None, 0)


BF = torch.bfloat16


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("call", [
    lambda L: L.moe_fp8_quantize(z(4, 64)),                                   # not on the GPU
    lambda L: L.moe_fp8_quantize(z(4, 64, dtype=torch.float16)),
    lambda L: L.moe_fp8_quantize(z(64)),
    lambda L: L.moe_fp8_quantize(z(4, 64), block_rows=32),
    lambda L: L.moe_fp8_quantize(z(4, 64), scales=z(4, 2, dtype=torch.float32)),
    lambda L: L.moe_linear_fp8(z(4, 64, dtype=torch.uint8), z(4, 1, dtype=torch.float32), z(8, 64, dtype=torch.uint8),
                               z(8, 1, dtype=torch.float32)),                 # a scale per row instead of per block
    lambda L: L.moe_linear_fp8(z(4, 64, dtype=torch.uint8), z(4, 1, dtype=torch.float32), z(8, 64, dtype=torch.uint8),
                               z(1, 1, dtype=torch.float32), act="swiglu"),   # gate and up have blocks of their own
    lambda L: L.moe_linear_fp8(z(4, 64), z(4, 1, dtype=torch.float32), z(8, 64, dtype=torch.uint8),
                               z(1, 1, dtype=torch.float32)),
    lambda L: L.moe_linear_fp8(z(4, 64, dtype=torch.uint8), z(4, 1, dtype=torch.float32), z(8, 64, dtype=torch.uint8),
                               z(1, 1, dtype=torch.float32), act="tanh"),
    lambda L: L.moe_glu(z(4, 64), z(15, 64)),
    lambda L: L.moe_glu(z(4, 64), z(16, 64), act="swiglu"),
    lambda L: L.moe_glu(z(4, 64), z(16, 32)),
    lambda L: L.moe_glu(z(4, 64), z(16, 64), a=z(4, 8)),
    lambda L: L.moe_glu(z(4, 128)[:, ::2], z(16, 64)),
    lambda L: L.moe_linear_backward(z(4, 8), None, z(8, 64)),
    lambda L: L.moe_linear_backward(z(4, 8), z(4, 64), None),
    lambda L: L.moe_linear_backward(z(4, 8), z(4, 64), z(8, 64), need_dx=False, need_dw=False),
    lambda L: L.moe_linear_backward(z(4, 8), z(4, 64), z(8, 64), accumulate=True),
    lambda L: L.moe_linear_backward(z(4, 8), z(4, 64), z(8, 64), dx=z(4, 64, dtype=torch.float16)),
    lambda L: L.moe_linear_backward(z(4, 8), z(4, 64), z(8, 64), dw=z(64, 8)),
    lambda L: L.moe_linear_backward(z(4, 8), z(5, 64), z(8, 64)),
    lambda L: L.moe_linear_backward(z(4, 8), z(4, 64), z(8, 64), ws=z(4, 4, dtype=torch.uint8)),
    lambda L: L.moe_glu_backward(z(4, 8), z(4, 8), z(4, 64), z(16, 64)),
    lambda L: L.moe_glu_backward(z(4, 8), z(4, 16), z(4, 64), z(8, 64)),
    lambda L: L.moe_glu_backward(z(4, 8), z(4, 16), z(4, 64), z(16, 64), act="swiglu"),
])
def test_binding_refusals(L, call):
    with pytest.raises(ValueError):
        call(L)


# ------------------------------------------------------------------ the block's shared expert in FP8
@pytest.fixture(scope="module")
def layer(L):
    from _helpers import FMT, layer_arrays

    sp, arrays = layer_arrays("tiny")
    return sp, L.DeviceWeights(FMT[sp["fmt"]], sp["E"], sp["H"], sp["I"], arrays, device="cpu")


def fp8_pair(rows, cols, parts=1):
    return (torch.zeros(rows, cols, dtype=torch.uint8),
            torch.zeros(parts * ((rows // parts + 127) // 128), (cols + 127) // 128))


def fp8_block(L, layer, ws1, ws2):
    sp, dw = layer
    return L.MoeBlock(dw, sp["k"], z(sp["H"]), z(sp["E"], sp["H"]), ws1=ws1, ws2=ws2)


@pytest.mark.parametrize("Is", [16, 128, 144, 256])
def test_block_takes_block_scaled_shared_experts(L, layer, Is):
    H = layer[0]["H"]
    fp8_block(L, layer, fp8_pair(2 * Is, H, 2), list(fp8_pair(H, Is)))


@pytest.mark.parametrize("ws1,ws2,match", [
    (lambda H: fp8_pair(288, H), lambda H: fp8_pair(H, 144), "ws1"),                 # gate and up have block rows of their own
    (lambda H: fp8_pair(288, H, 2), lambda H: fp8_pair(H, 160), "ws2"),
    (lambda H: fp8_pair(16, H, 2), lambda H: fp8_pair(H, 8), "ws2"),                 # rows of 8 values
    (lambda H: fp8_pair(288, H, 2), lambda H: z(H, 144), "ws2"),                     # FP8 and bf16 mixed
    (lambda H: fp8_pair(256, H, 2), lambda H: (fp8_pair(H, 128)[0], torch.zeros(H, 4, dtype=torch.uint8)), "ws2"),  # and MXFP8
    (lambda H: fp8_pair(288, H, 2) + (None,), lambda H: fp8_pair(H, 144), "pairs"),
])
def test_block_refuses_other_shared_experts(L, layer, ws1, ws2, match):
    H = layer[0]["H"]
    with pytest.raises(ValueError, match=match):
        fp8_block(L, layer, ws1(H), ws2(H))
