"""The dense feed-forward operators beside the routed experts, as a user's program calls them: quantisation to
FP8 with a scale for each block of 128, the product of such operands with its epilogue, and the gated
feed-forward projection of a shared expert with its gradients and those of a plain product.

``own`` selects the library's kernels; otherwise ``run`` computes the plain form in torch."""
import math

import torch

own = False

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
BLOCK = 128


# ---------------------------------------------------------------------------- the cases
def listed():
    return [
        # quantisation
        # the activations of a serving batch in front of an FP8 product
        dict(name="quantize batch", op="quantize", rows=64, K=4096, x="bf16", by=1),
        # the weights of a shared expert's FC1, once, from the fp32 master copy
        dict(name="quantize weights", op="quantize", rows=4096, K=4096, x="f32", by=128),
        # FP8 products
        # shared expert of one decoded token: FC1 with SwiGLU, bound by reading the weights
        dict(name="fp8 token", op="linear", T=1, N=4096, K=4096, act="swiglu", bias=False, res="none"),
        # shared expert of a serving batch: FC2 with the routed output added
        dict(name="fp8 batch", op="linear", T=64, N=4096, K=2048, act="none", bias=False, res="f32"),
        # a ragged middle-sized batch with every part of the epilogue, blocks that end early
        dict(name="fp8 ragged", op="linear", T=1001, N=1000, K=2016, act="gelu", bias=True, res="f32"),
        # shared expert of a prefill: FC1 with SwiGLU
        dict(name="fp8 prefill", op="linear", T=8192, N=4096, K=4096, act="swiglu", bias=False, res="none"),
        # gated projection
        # the shared expert of the smaller layer for one token
        dict(name="glu token", op="glu", T=1, I=512, K=2048, act="silu", keep=False),
        # a training batch's forward pass, which keeps what the backward pass reads
        dict(name="glu train", op="glu", T=8192, I=2048, K=4096, act="silu", keep=True),
        # its gradients
        # a short ragged batch
        dict(name="glu backward ragged", op="glu_backward", T=1001, I=504, K=2016, act="gelu"),
        # a training batch
        dict(name="glu backward train", op="glu_backward", T=8192, I=2048, K=4096, act="silu"),
        # gradients of the down projection
        # the smaller layer, long batch: few weights, long sums over the tokens, fp32 weight gradient
        dict(name="linear backward small", op="linear_backward", T=16384, N=2048, K=512, dw="f32"),
        # the larger layer's training batch
        dict(name="linear backward train", op="linear_backward", T=8192, N=4096, K=2048, dw="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "linear", "linear", "glu", "glu_backward", "linear_backward"))
    if op == "quantize":
        K = 16 * _log(rng, 4, 512)
        return dict(op=op, rows=_log(rng, 1, min(65536, (1 << 26) // K)), K=K, x=rng.choice(("bf16", "f32")),
                    by=rng.choice((1, 128)))
    T = _log(rng, 1, 8192)
    if op == "linear":
        act = rng.choice(("none", "relu", "gelu", "silu", "swiglu"))
        N = _log(rng, 8, 4096)
        return dict(op=op, T=T, N=N + (N % 2 if act == "swiglu" else 0), K=16 * _log(rng, 4, 256), act=act,
                    bias=rng.random() < 0.5, res=rng.choice(("none", "bf16", "f32")))
    if op == "linear_backward":
        return dict(op=op, T=T, N=8 * _log(rng, 2, 512), K=8 * _log(rng, 2, 512), dw=rng.choice(("bf16", "f32")))
    case = dict(op=op, T=T, I=8 * _log(rng, 2, 256), K=8 * _log(rng, 4, 512),
                act=rng.choice(("none", "relu", "gelu", "silu")))
    if op == "glu":
        case["keep"] = rng.random() < 0.5
    return case


# ---------------------------------------------------------------------------- inputs
def _type(name):
    return {"f32": F32, "bf16": BF16}[name]


def _up(n):
    return (n + BLOCK - 1) // BLOCK


def _blocks(v, by):
    """v [rows][K] in whole blocks of by x 128, padded with zeros: [row blocks][by][K blocks][128]."""
    rows, K = v.shape
    v = torch.nn.functional.pad(v, (0, _up(K) * BLOCK - K, 0, -rows % by))
    return v.reshape(-1, by, _up(K), BLOCK)


def _quantize(v, by):
    """e4m3 elements and fp32 scales (amax / 448) of fp32 values, a scale for each block of by x 128."""
    rows, K = v.shape
    b = _blocks(v, by)
    top = b.abs().amax((1, 3))
    scales = top / torch.full_like(top, 448.0)  # a division: by a plain number torch multiplies with 1/448
    s = scales[:, None, :, None]
    q = torch.where(s > 0, b / s, 0.0).clamp(-448.0, 448.0).to(E4M3)
    return q.reshape(-1, b.shape[2] * BLOCK)[:rows, :K].contiguous(), scales


def _values(q, scales, by, dtype):
    """The values of e4m3 elements with a scale for each block of by x 128."""
    rows, K = q.shape
    s = scales.to(dtype).repeat_interleave(by, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :K]
    return q.to(dtype) * s


def _halves(w, gated):
    """The matrices that weight rows belong to: gate and up have block rows of their own."""
    return w.chunk(2) if gated else (w,)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 29)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def activations(T, K):
        # what a norm leaves: a few channels are larger than the others
        size = torch.exp(0.4 * normal(K)) + 12.0 * (torch.rand(K, generator=g, device="cuda") < 0.004)
        return size * normal(T, K)

    def empty(shape, dtype):
        return torch.empty(shape, dtype=dtype, device="cuda")

    s = dict(case=case)
    K = case["K"]
    if case["op"] == "quantize":
        rows, by = case["rows"], case["by"]
        x = activations(rows, K) if by == 1 else normal(rows, K) / math.sqrt(K)
        s["x"] = x.to(_type(case["x"]))
        s["q"] = empty((rows, K), torch.uint8)
        s["scales"] = empty(((rows + by - 1) // by, _up(K)), F32)
        return s
    T = case["T"]
    if case["op"] == "linear":
        N, gated = case["N"], case["act"] == "swiglu"
        n_out = N // 2 if gated else N
        s["x"], s["xs"] = _quantize(activations(T, K).to(BF16).float(), 1)
        # rows of different size, as trained weights have them
        w = torch.exp(0.3 * normal(N, 1)) * normal(N, K) / math.sqrt(K)
        parts = [_quantize(p, 128) for p in _halves(w, gated)]
        s["w"], s["ws"] = torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
        s["bias"] = 0.3 * normal(N) if case["bias"] else None
        s["res"] = normal(T, n_out).to(_type(case["res"])) if case["res"] != "none" else None
        s["out"] = empty((T, n_out), BF16)
        return s
    rows = case["N"] if case["op"] == "linear_backward" else 2 * case["I"]
    s["x"] = activations(T, K).to(BF16)
    s["w"] = (normal(rows, K) / math.sqrt(K)).to(BF16)
    if case["op"] == "glu":
        s["h"] = empty((T, case["I"]), BF16)
        s["a"] = empty((T, rows), BF16) if case["keep"] else None
        return s
    if case["op"] == "glu_backward":
        s["a"] = (1.3 * normal(T, rows)).to(BF16)
        s["dh"] = (1e-3 * normal(T, case["I"])).to(BF16)
    else:
        s["dy"] = (1e-3 * normal(T, rows)).to(BF16)
    s["dx"] = empty((T, K), BF16)
    s["dw"] = empty((rows, K), _type(case.get("dw", "bf16")))
    return s


# ---------------------------------------------------------------------------- one pass
def run(s):
    if own:
        from bit_moe_expert_top_amd import ops

        return _own(s, ops)
    return {"quantize": _run_quantize, "linear": _run_linear, "glu": _run_glu, "glu_backward": _run_glu_backward,
            "linear_backward": _run_linear_backward}[s["case"]["op"]](s)


def _own(s, ops):
    c = s["case"]
    if c["op"] == "quantize":
        ops.moe_fp8_quantize(s["x"], block_rows=c["by"], q=s["q"], scales=s["scales"])
        return {"q": s["q"].view(E4M3), "scales": s["scales"]}
    if c["op"] == "linear":
        ops.moe_linear_fp8(s["x"], s["xs"], s["w"], s["ws"], bias=s["bias"], act=c["act"], residual=s["res"],
                           out=s["out"])
        return {"out": s["out"]}
    if c["op"] == "glu":
        ops.moe_glu(s["x"], s["w"], act=c["act"], a=s["a"], out=s["h"])
        return {"h": s["h"]} if s["a"] is None else {"h": s["h"], "a": s["a"]}
    if c["op"] == "glu_backward":
        ops.moe_glu_backward(s["dh"], s["a"], s["x"], s["w"], act=c["act"], dx=s["dx"], dw=s["dw"])
    else:
        ops.moe_linear_backward(s["dy"], s["x"], s["w"], dx=s["dx"], dw=s["dw"])
    return {"dx": s["dx"], "dw": s["dw"]}


def _run_quantize(s):
    q, scales = _quantize(s["x"].float(), s["case"]["by"])
    return {"q": q, "scales": scales}


def _act(a, act):
    if act == "relu":
        return torch.clamp(a, min=0.0)
    if act == "gelu":
        return 0.5 * a * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (a + 0.044715 * a * a * a)))
    if act == "silu":
        return a / (1.0 + torch.exp(-a))
    return a


def _slope(a, act):
    if act == "relu":
        return (a > 0).to(a.dtype)
    if act == "gelu":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (a + 0.044715 * a * a * a))
        return 0.5 * (1.0 + t) + 0.5 * a * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * a * a)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-a))
        return p * (1.0 + a * (1.0 - p))
    return torch.ones_like(a)


def _run_linear(s):
    c = s["case"]
    gated = c["act"] == "swiglu"
    x = _values(s["x"], s["xs"], 1, F32)
    w = torch.cat([_values(q, b, 128, F32) for q, b in zip(_halves(s["w"], gated), _halves(s["ws"], gated))])
    a = x @ w.t()
    if s["bias"] is not None:
        a = a + s["bias"]
    if gated:
        gate, up = a.chunk(2, 1)
        a = _act(gate, "silu") * up
    else:
        a = _act(a, c["act"])
    if s["res"] is not None:
        a = a + s["res"].float()
    return {"out": a.to(BF16)}


def _run_glu(s):
    a = s["x"].float() @ s["w"].float().t()
    gate, up = a.chunk(2, 1)
    h = (_act(gate, s["case"]["act"]) * up).to(BF16)
    return {"h": h} if s["a"] is None else {"h": h, "a": a.to(BF16)}


def _run_glu_backward(s):
    act = s["case"]["act"]
    gate, up = s["a"].float().chunk(2, 1)
    dh = s["dh"].float()
    da = torch.cat([dh * up * _slope(gate, act), dh * _act(gate, act)], 1)
    return {"dx": (da @ s["w"].float()).to(BF16), "dw": (da.t() @ s["x"].float()).to(s["dw"].dtype)}


def _run_linear_backward(s):
    dy = s["dy"].float()
    return {"dx": (dy @ s["w"].float()).to(BF16), "dw": (dy.t() @ s["x"].float()).to(s["dw"].dtype)}


# ---------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    size = {"f32": 4, "bf16": 2, "none": 0}
    K = case["K"]
    if case["op"] == "quantize":
        rows, by = case["rows"], case["by"]
        return {"bytes": rows * K * (size[case["x"]] + 1) + 4 * ((rows + by - 1) // by) * _up(K), "flops": 3 * rows * K}
    T = case["T"]
    if case["op"] == "linear":
        N, gated = case["N"], case["act"] == "swiglu"
        n_out = N // 2 if gated else N
        scales = 4 * _up(K) * (T + (2 * _up(n_out) if gated else _up(N)))
        return {"bytes": (T + N) * K + scales + T * n_out * (size[case["res"]] + 2) + (4 * N if case["bias"] else 0),
                "flops": 2 * T * N * K}
    if case["op"] == "glu":
        I = case["I"]
        return {"bytes": 2 * (T * K + 2 * I * K + T * I * (3 if case["keep"] else 1)), "flops": 4 * T * I * K}
    if case["op"] == "glu_backward":
        I = case["I"]
        return {"bytes": 2 * (3 * T * I + 2 * T * K + 4 * I * K), "flops": 8 * T * I * K}
    N = case["N"]
    return {"bytes": 2 * (T * N + 2 * T * K + N * K) + size[case["dw"]] * N * K, "flops": 4 * T * N * K}


# ---------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"quantize": _exact_quantize, "linear": _exact_linear, "glu": _exact_glu, "glu_backward": _exact_glu_backward,
            "linear_backward": _exact_linear_backward}[case["op"]](case, s)


def _exact_quantize(case, s):
    rows, K, by = case["rows"], case["K"], case["by"]
    q = torch.empty(rows, K, dtype=torch.float64, device="cuda")
    scales = torch.empty_like(s["scales"], dtype=torch.float64)
    step = by * max(1, (1 << 24) // (by * K))
    for i in range(0, rows, step):
        x = s["x"][i:i + step].double()
        for j in range(_up(K)):
            part = x[:, j * BLOCK:(j + 1) * BLOCK]
            top = part.abs().amax(1)
            top = torch.stack([t.amax() for t in top.split(by)]) if by > 1 else top
            scales[i // by:i // by + len(top), j] = top / 448
            # the block's values with the largest brought to 448 (by the unrounded scale: 3/8 of the largest lies half
            # way between two elements)
            top = top.repeat_interleave(by)[:len(x), None]
            v = torch.where(top > 0, part * 448 / top, 0.0)
            # e4m3: steps of 2^-3 of the value's own power of two, of 2^-9 below 2^-6, no value above 448
            unit = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
            q[i:i + step, j * BLOCK:(j + 1) * BLOCK] = (torch.round(v / unit) * unit).clamp(-448, 448)
    return {"q": q, "scales": scales}


def _exact_act(a, act):
    """The activation and its slope."""
    if act == "relu":
        return torch.where(a > 0, a, 0.0), torch.where(a > 0, 1.0, 0.0).to(a.dtype)
    if act == "none":
        return a, torch.ones_like(a)
    # a sigma(z): z = a (silu), or 2 sqrt(2/pi) (a + 0.044715 a^3) (gelu)
    if act == "silu":
        z, dz = a, 1.0
    else:
        z = 2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)
        dz = 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * a ** 2)
    p = torch.sigmoid(z)
    return a * p, p + a * p * torch.sigmoid(-z) * dz


def _exact_linear(case, s):
    K, N, T = case["K"], case["N"], case["T"]
    gated = case["act"] == "swiglu"
    first = N // 2 if gated else N  # rows of a matrix of its own
    row = torch.arange(N, device="cuda")
    block_row = row // BLOCK if not gated else torch.where(row < first, row // BLOCK, _up(first) + (row - first) // BLOCK)
    a = torch.zeros(T, N, dtype=torch.float64, device="cuda")
    for j in range(_up(K)):
        k = slice(j * BLOCK, min(K, (j + 1) * BLOCK))
        xk = s["x"][:, k].double() * s["xs"][:, j, None].double()
        wk = s["w"][:, k].double() * s["ws"][block_row, j, None].double()
        a += torch.matmul(xk, wk.t().contiguous())
    if s["bias"] is not None:
        a += s["bias"].double()
    if gated:
        a = _exact_act(a[:, :first], "silu")[0] * a[:, first:]
    else:
        a = _exact_act(a, case["act"])[0]
    if s["res"] is not None:
        a = a + s["res"].double()
    return {"out": a}


def _exact_glu(case, s):
    a = torch.matmul(s["x"].double(), s["w"].double().t().contiguous())
    h = _exact_act(a[:, :case["I"]], case["act"])[0] * a[:, case["I"]:]
    return {"h": h, "a": a} if case["keep"] else {"h": h}


def _exact_gradients(da, s):
    return {"dx": torch.matmul(da, s["w"].double()), "dw": torch.matmul(da.t().contiguous(), s["x"].double())}


def _exact_glu_backward(case, s):
    I = case["I"]
    a, dh = s["a"].double(), s["dh"].double()
    value, slope = _exact_act(a[:, :I], case["act"])
    da = torch.empty_like(a)
    da[:, :I] = dh * a[:, I:] * slope
    da[:, I:] = dh * value
    return _exact_gradients(da, s)


def _exact_linear_backward(case, s):
    return _exact_gradients(s["dy"].double(), s)
