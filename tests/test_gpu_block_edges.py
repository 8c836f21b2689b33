"""GPU: edges of the operators around the expert FFN, against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import block as OB
from oracle import moe as OM

from _helpers import device_layer, host, oracle_layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_moe_expert_top_amd import _lib

    return _lib


def cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


# ------------------------------------------------------------------ the block
def tiny_block(L, rows=None, mx=False):
    sp, dw = device_layer("tiny")
    H, E, Is = sp["H"], rows or sp["E"], 256
    r = np.random.default_rng(41)
    bf = lambda *s: cuda((r.normal(size=s) / np.sqrt(s[-1])).astype(np.float32), torch.bfloat16)
    ws = [bf(2 * Is, H), bf(H, Is)]
    if mx:
        ws = [L.moe_mxfp8_quantize(v.view(torch.int16)) for v in ws]
    return sp, L.MoeBlock(dw, sp["k"], 1 + bf(1, H)[0], bf(E, H), route=dict(score="sigmoid"), ws1=ws[0], ws2=ws[1])


@pytest.mark.parametrize("mx", [False, True])
def test_block_of_no_tokens(L, mx):
    sp, blk = tiny_block(L, mx=mx)
    o = L.block_forward(blk, torch.empty(0, sp["H"], device="cuda"), torch.empty(0, sp["H"], device="cuda"))
    torch.cuda.synchronize()
    assert o["out"].shape == (0, sp["H"]) and not bool(o["counts"].any()) and not bool(o["offsets"].any())


def test_block_with_experts_that_are_not_routed_to(L):
    sp, blk = tiny_block(L, rows=5)
    x = torch.randn(33, sp["H"], device="cuda")
    o = L.block_forward(blk, x, None)  # without a residual stream
    torch.cuda.synchronize()
    ids, _ = OB.route_scored(host(o["logits"]), sp["k"], score="sigmoid")
    np.testing.assert_array_equal(host(o["ids"]), ids)
    _, offsets, perm, inv = OM.permute(ids, sp["E"])
    yp = OM.expert_ffn(oracle_layer("tiny"), host(o["y"]).view(np.uint16), sp["k"], offsets, perm)
    want = OM.combine(yp, inv, host(o["gates"]).astype(np.float64), 33, sp["k"])
    # the layer's bar for experts computed in bf16
    assert np.abs(host(o["routed"]) - want).max() <= 2e-2 * np.sqrt(np.mean(want**2))


# ------------------------------------------------------------------ the binding
def test_calls_with_the_public_stream_queries(L, monkeypatch):
    """As on a torch without the private ones: the call is enqueued on the current stream."""
    monkeypatch.setattr(L, "_raw_device", torch.cuda.current_device)
    monkeypatch.setattr(L, "_raw_stream", lambda index: torch.cuda.current_stream(index).cuda_stream)
    lg = torch.randn(50, 64, device="cuda")
    want = L.moe_route_scored(lg, 4)
    torch.cuda.synchronize()
    ids, gates = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        L.moe_route_scored(lg, 4, topk_ids=ids, topk_w=gates)
        got = ids.clone(), gates.clone()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
