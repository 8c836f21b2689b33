"""block_forward refuses operands that do not fit the layer's experts before it changes anything: an expert id
past the layer's experts has no row in moe_combine's input, rows shorter than H would be read past their end, and a call that fails
later would leave the residual stream with x already added.  CPU tensors: nothing is launched."""
import pytest
import torch

from _helpers import FMT, layer_arrays


@pytest.fixture(scope="module")
def L():
    from bit_moe_expert_top_amd import _lib

    return _lib


@pytest.fixture(scope="module")
def layer(L):
    sp, arrays = layer_arrays("tiny")
    return sp, L.DeviceWeights(FMT[sp["fmt"]], sp["E"], sp["H"], sp["I"], arrays, device="cpu")


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def mx(n, k):
    return torch.zeros(n, k, dtype=torch.uint8), torch.zeros(n, k // 32, dtype=torch.uint8)


def block(L, layer, **change):
    sp, dw = layer
    H, E = sp["H"], sp["E"]
    args = dict(k=sp["k"], norm_weight=bf16(H), router_weight=bf16(E, H), router_bias=torch.zeros(E),
                route=dict(score="sigmoid", n_group=4, topk_group=2), ws1=bf16(512, H), ws2=bf16(H, 256))
    args.update({key: v(H, E) if callable(v) else v for key, v in change.items()})
    return L.MoeBlock(dw, **args)


def test_fitting_operands(L, layer):
    block(L, layer)
    block(L, layer, ws1=None, ws2=None, router_bias=None)
    block(L, layer, router_weight=lambda H, E: bf16(E - 4, H), router_bias=lambda H, E: torch.zeros(E - 4))
    block(L, layer, ws1=lambda H, E: mx(512, H), ws2=lambda H, E: mx(H, 256))
    block(L, layer, ws1=lambda H, E: list(mx(512, H)), ws2=lambda H, E: list(mx(H, 256)))


@pytest.mark.parametrize("change,match", [
    (dict(router_weight=lambda H, E: bf16(E + 8, H)), "router_weight"),   # ids past the layer's experts
    (dict(router_weight=lambda H, E: bf16(E - 4, H)), "router_bias"),
    (dict(router_weight=lambda H, E: bf16(E, H // 2)), "router_weight"),
    (dict(norm_weight=lambda H, E: bf16(H // 2)), "norm_weight"),
    (dict(router_bias=lambda H, E: torch.zeros(E + 1)), "router_bias"),
    (dict(ws1=lambda H, E: bf16(512, H // 2)), "ws1"),
    (dict(ws1=lambda H, E: bf16(511, H)), "ws1"),
    (dict(ws2=lambda H, E: bf16(H, 128)), "ws2"),
    (dict(ws2=lambda H, E: bf16(H // 2, 256)), "ws2"),
    (dict(ws2=lambda H, E: mx(H, 256)), "ws2"),                          # bf16 and MXFP8 mixed
    (dict(ws1=lambda H, E: (mx(512, H)[0], mx(512, H // 2)[1]), ws2=lambda H, E: mx(H, 256)), "ws1"),
    (dict(ws1=lambda H, E: bf16(8, H), ws2=lambda H, E: bf16(H, 4)), "ws2"),   # rows of 4 values
    (dict(ws1=None), "together"),
    (dict(k=0), "k"),
    (dict(k=lambda H, E: E + 1), "k"),
    (dict(route=dict(n_group=5)), "route"),
    (dict(route=dict(n_group=4, topk_group=5)), "route"),
    (dict(route=dict(score="tanh")), "route"),
    (dict(route=dict(groups=4)), "route"),
    (dict(route=dict(scale=float("inf"))), "route"),
    (dict(eps=0.0), "eps"),
])
def test_refused_when_made(L, layer, change, match):
    with pytest.raises(ValueError, match=match):
        block(L, layer, **change)


def test_refused_when_changed_afterwards(L, layer):
    sp, _ = layer
    H, E = sp["H"], sp["E"]
    blk = block(L, layer)
    blk.router_weight = bf16(E + 8, H)
    with pytest.raises(ValueError, match="router_weight"):
        L.block_forward(blk, bf16(4, H), bf16(4, H))


@pytest.mark.parametrize("x,res,match", [
    (lambda H: bf16(4, H // 2), lambda H: bf16(4, H // 2), "x: expected"),       # rows shorter than the experts'
    (lambda H: bf16(4, 2 * H), lambda H: bf16(4, 2 * H), "x: expected"),
    (lambda H: bf16(4 * H), lambda H: bf16(4, H), "x: expected"),
    (lambda H: bf16(4, H).double(), lambda H: bf16(4, H), "x: expected"),
    (lambda H: bf16(4, H), lambda H: bf16(3, H), "residual: expected"),
    (lambda H: bf16(4, H), lambda H: bf16(4, H).double(), "residual: expected"),
    (lambda H: bf16(4 * H + 1)[1:].view(4, H), lambda H: bf16(4, H), "x: expected"),           # alignment
    # more tokens than the experts take (memory that is never touched)
    (lambda H: torch.empty((1 << 31) // H, H, dtype=torch.bfloat16), lambda H: bf16(4, H), "fewer tokens"),
    (lambda H: torch.empty(4, H, dtype=torch.bfloat16, device="meta"), lambda H: bf16(4, H), "x: expected"),
])
def test_inputs_refused(L, layer, x, res, match):
    H = layer[0]["H"]
    with pytest.raises(ValueError, match=match):
        L.block_forward(block(L, layer), x(H), res(H))
