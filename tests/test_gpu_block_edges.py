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


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [1, 40])
def test_block_captured_and_on_another_stream(L, T, mx):
    """The whole block in a HIP graph, replayed on changing inputs with eager work between the replays, and on a stream of
    its own: the bits of the eager call, the residual stream updated by each."""
    sp, blk = tiny_block(L, mx=mx)
    H = sp["H"]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)
    new = lambda: (torch.randn(T, H, generator=gen, device="cuda"), torch.randn(T, H, generator=gen, device="cuda").bfloat16())
    x, res = new()
    L.block_forward(blk, x.clone(), res.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = L.block_forward(blk, x, res)
    side = torch.cuda.Stream()
    for _ in range(4):
        nx, nres = new()
        x.copy_(nx)
        res.copy_(nres)
        graph.replay()
        torch.cuda.synchronize()
        got, got_res = captured["out"].clone(), res.clone()
        eager_res, side_res = nres.clone(), nres.clone()
        want = L.block_forward(blk, nx, eager_res)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            beside = L.block_forward(blk, nx, side_res)
        torch.cuda.synchronize()
        for out, r in ((got, got_res), (beside["out"], side_res)):
            assert torch.equal(out.view(torch.uint8), want["out"].view(torch.uint8))
            assert torch.equal(r.view(torch.uint8), eager_res.view(torch.uint8))


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


# ------------------------------------------------------------------ routing
def check_route(L, lg, k, some=None, **kw):
    bias = kw.pop("bias", None)
    ids, gates = L.moe_route_scored(cuda(lg), k, bias=None if bias is None else cuda(bias), **kw)
    ids, gates = host(ids), host(gates)
    some = np.arange(len(lg)) if some is None else some
    want, gw = OB.route_scored(lg[some], k, bias=bias, **kw)
    np.testing.assert_array_equal(ids[some], want)
    # exp with an argument rounded in fp32: (|l - max| + 8) 2^-23 of the gate; sums, a quotient and a product: 16 more
    # roundings of 2^-24
    finite = np.where(np.isfinite(lg[some]), lg[some], 0.0)
    spread = np.abs(finite).max(axis=1, keepdims=True) * 2
    assert np.isfinite(gates).all()
    np.testing.assert_array_less(np.abs(gates[some] - gw), np.abs(gw) * (spread + 16) * 2.0**-23 + 1e-38)
    return ids


def microseconds(call, n=10):
    """The time of a call on the GPU: the median replay of a graph of n of them."""
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(n):
            call()
    times = []
    for _ in range(9):
        start, end = torch.cuda.Event(True), torch.cuda.Event(True)
        start.record()
        graph.replay()
        end.record()
        torch.cuda.synchronize()
        times.append(start.elapsed_time(end) * 1e3 / n)
    return sorted(times)[4]


def route_time(L, lg, k, bias=None, **kw):
    lg, bias = cuda(lg), None if bias is None else cuda(bias)
    ids = torch.empty(len(lg), k, dtype=torch.int32, device="cuda")
    gates = torch.empty(len(lg), k, device="cuda")
    return microseconds(lambda: L.moe_route_scored(lg, k, bias=bias, topk_ids=ids, topk_w=gates, **kw))


def rows_of(T):
    """The rows that the oracle checks of a large batch."""
    return np.r_[np.arange(0, min(T, 300)), np.arange(300, T, 41)]


@pytest.mark.parametrize("T", [50, 8200])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,keep,k", [(64, 8, 4, 6), (256, 8, 3, 8), (384, 4, 2, 16), (512, 16, 5, 8)])
def test_groups_out_of_service(L, T, score, E, G, keep, k):
    """Whole groups with a bias of -inf or NaN: one, as many as leave fewer than stay, one left, none left."""
    r = np.random.default_rng([T, E, 51])
    lg = (r.normal(size=(T, E)) * 2).astype(np.float32)
    lg[::9] = np.round(lg[::9])  # ties
    gs = E // G
    some = rows_of(T)[::4]
    for dead in (1, G - keep + 1, G - 1, G):
        bias = (r.normal(size=E) * 0.1).astype(np.float32)
        for g in r.permutation(G)[:dead]:
            bias[g * gs:(g + 1) * gs] = -np.inf if g % 2 else np.nan
        for top in (1, 2):
            check_route(L, lg, k, some, score=score, bias=bias, n_group=G, topk_group=keep, group_top=top, renormalize=True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_time_with_a_group_out_of_service(L, score):
    """A group out of service leaves the others' choice to fp32: the call takes no more than twice its time."""
    r = np.random.default_rng(52)
    lg = r.normal(size=(32768, 384)).astype(np.float32)
    bias = (r.normal(size=384) * 0.05).astype(np.float32)
    dead = bias.copy()
    dead[48:96] = -np.inf
    kw = dict(score=score, n_group=8, topk_group=4, group_top=2, renormalize=True)
    plain, less = route_time(L, lg, 8, bias, **kw), route_time(L, lg, 8, dead, **kw)
    assert less < 2 * plain, (plain, less)


def masked_logits(T, E, G, seed):
    """Masks of -inf: a quarter of the logits, one expert, all but a few, all but one group, all; some rows
    without one, and ties among what is left."""
    r = np.random.default_rng([T, E, seed])
    lg = (r.normal(size=(T, E)) * 2).astype(np.float32)
    lg[::5] = np.round(lg[::5])
    gs = E // G
    for t in range(T):
        kind = t % 16
        if kind < 8:
            lg[t, r.random(E) < 0.25] = -np.inf
        elif kind == 8:
            lg[t, r.integers(E)] = -np.inf
        elif kind == 9:
            lg[t, r.permutation(E)[int(r.integers(1, 20)):]] = -np.inf
        elif kind == 10:
            g = int(r.integers(G))
            lg[t, :g * gs] = lg[t, (g + 1) * gs:] = -np.inf
        elif kind == 11:
            lg[t, r.permutation(E)[1:]] = -np.inf
        elif kind == 12:
            lg[t] = -np.inf
    return lg


@pytest.mark.parametrize("T", [61, 8200])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,keep,k", [(64, 8, 4, 6), (256, 1, 1, 8), (384, 8, 3, 16), (510, 1, 1, 10), (512, 16, 5, 8)])
def test_masked_logits(L, T, score, E, G, keep, k):
    lg = masked_logits(T, E, G, 53)
    r = np.random.default_rng([E, 54])
    bias = (r.normal(size=E) * 0.1).astype(np.float32)
    level = np.full(E, 0.25, np.float32)  # masked experts tie with one another
    some = rows_of(T)
    for b, top, renorm in ((None, 1, True), (bias, 2, True), (level, 1, False), (None, 2, False)):
        check_route(L, lg, k, some, score=score, bias=b, n_group=G, topk_group=keep, group_top=top, renormalize=renorm)


@pytest.mark.parametrize("score,groups,biased", [("softmax", (1, 1), False), ("sigmoid", (8, 4), True)])
def test_time_of_masked_logits(L, score, groups, biased):
    """A quarter of each row masked: no more than twice the time of the rows without the mask."""
    r = np.random.default_rng(55)
    lg = r.normal(size=(32768, 384)).astype(np.float32)
    bias = (r.normal(size=384) * 0.05).astype(np.float32) if biased else None
    masked = np.where(r.random(lg.shape) < 0.25, np.float32(-np.inf), lg)
    kw = dict(score=score, n_group=groups[0], topk_group=groups[1], renormalize=True)
    plain, less = route_time(L, lg, 8, bias, **kw), route_time(L, masked, 8, bias, **kw)
    assert less < 2 * plain, (plain, less)
    small, few = route_time(L, lg[:64], 8, bias, **kw), route_time(L, masked[:64], 8, bias, **kw)
    assert few < 2 * small, (small, few)


@pytest.mark.parametrize("T", [70, 8200])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,keep,k", [(1, 1, 1, 1), (60, 5, 2, 24), (64, 8, 8, 6), (256, 1, 1, 8), (384, 8, 4, 8),
                                        (384, 8, 4, 16), (512, 16, 5, 8), (1000, 10, 2, 30)])
def test_padding_rows(L, T, score, E, G, keep, k):
    """Rows of one value (0, +-large, -inf, +inf and NaN among them) between others, rows that differ in one logit
    only; without a bias, with equal ones, with all out of service, with one that differs."""
    r = np.random.default_rng([T, E, k, 56])
    lg = (r.normal(size=(T, E)) * 2).astype(np.float32)
    for i, v in enumerate((0.0, -0.0, 3.0, -300.0, 1e30, -np.inf, np.inf, np.nan)):
        lg[i::16] = v
    lg[8::16] = 1.0
    lg[8::16, E // 2] = np.nextafter(np.float32(1.0), np.float32(2.0))
    lg[9::16] = np.where(r.random(lg[9::16].shape) < 0.5, 0.0, -0.0)
    level = np.full(E, -0.5, np.float32)
    odd = level.copy()
    odd[E - 1] = 0.25
    some = rows_of(T)[::2]
    for b, top, renorm in ((None, 1, True), (None, 2, False), (level, 2, True), (0 * level, 1, False), (odd, 1, True),
                           (np.full(E, -np.inf, np.float32), 2, True), (np.full(E, np.nan, np.float32), 1, True)):
        kw = dict(score=score, n_group=G, topk_group=keep, group_top=top, renormalize=renorm, scale=1.5)
        ids, gates = L.moe_route_scored(cuda(lg), k, bias=None if b is None else cuda(b), **kw)
        with np.errstate(invalid="ignore"):
            want, gw = OB.route_scored(lg[some], k, bias=b, **kw)
        ids, gates = host(ids)[some], host(gates)[some]
        np.testing.assert_array_equal(ids, want)
        # the same bound as check_route's; e^-300 and its kind are 0 in fp32
        finite = np.where(np.isfinite(lg[some]) & (np.abs(lg[some]) < 1e4), lg[some], 0.0)
        spread = np.abs(finite).max(axis=1, keepdims=True) * 2
        np.testing.assert_array_less(np.abs(gates - gw), np.abs(gw) * (spread + 16) * 2.0**-23 + 1e-38)


@pytest.mark.parametrize("score,groups,biased,value", [
    ("softmax", (1, 1), False, 0.0), ("sigmoid", (1, 1), False, 0.0), ("softmax", (8, 4), True, 0.0), ("sigmoid", (8, 4), True, 0.0),
    ("softmax", (1, 1), False, -np.inf), ("sigmoid", (1, 1), False, -np.inf), ("sigmoid", (8, 4), True, -np.inf)])
def test_time_of_padding_rows(L, score, groups, biased, value):
    """Half of the batch padding, its logits all 0 or all masked, the biases (if any) not trained yet: no more than three
    times the time of a full batch (up to 2.3 measured; 4 to 10 where such rows are routed plainly in 64 bits)."""
    r = np.random.default_rng(57)
    for T in (64, 32768):
        lg = r.normal(size=(T, 384)).astype(np.float32)
        bias = np.zeros(384, np.float32) if biased else None
        padded = lg.copy()
        padded[T // 2:] = value
        kw = dict(score=score, n_group=groups[0], topk_group=groups[1], renormalize=True)
        plain, less = route_time(L, lg, 8, bias, **kw), route_time(L, padded, 8, bias, **kw)
        assert less < 3 * plain, (T, plain, less)


@pytest.mark.parametrize("T", [60, 8200])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biases_of_very_different_size(L, T, score):
    """Scores a few 1e-6 apart in groups whose biases are around 0, 1e3 and -1e3, 1e6: each score is rounded by its own
    size, and the order is that of 64 bits."""
    r = np.random.default_rng([T, 58])
    E, G = 32, 8
    lg = (1e-5 * r.normal(size=(T, E))).astype(np.float32)
    bias = np.zeros(E, np.float32)
    bias[4:8] = (1000.0, -1000.0, 0.0, 0.0)
    bias[8:12] = (1000.0, -1000.0, -1000.0, -1000.0)
    bias[20:24] = (1e6, -1e6, -1e6, -1e6)
    some = rows_of(T)
    for keep in (1, 2, 3, 5):
        for top in (1, 2):
            check_route(L, lg, 3, some, score=score, bias=bias, n_group=G, topk_group=keep, group_top=top, renormalize=True)
    check_route(L, lg, 12, some, score=score, bias=bias)
