"""The operators around the expert FFN, as a user's program calls them: residual + RMS norm with an
MXFP8 output, the dense matrix product with its epilogue, and scored routing.

``own`` selects the library's kernels; otherwise ``run`` computes the plain form in torch."""
import math

import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-6


# ---------------------------------------------------------------------------- the cases
def listed():
    return [
        # residual + norm
        # one decoded token: the routed experts' fp32 sum joins a bf16 residual stream
        dict(name="norm token", op="norm", T=1, H=4096, x="f32", res="bf16", y=True, q=True),
        # a serving batch in front of the router and an FP8 product
        dict(name="norm batch", op="norm", T=64, H=4096, x="f32", res="bf16", y=True, q=True),
        # a prompt chunk of a long context, ragged token count, bf16 experts only
        dict(name="norm prompt", op="norm", T=16381, H=2048, x="bf16", res="bf16", y=True, q=False),
        # a large prefill in front of FP8 products, fp32 residual stream
        dict(name="norm prefill", op="norm", T=32768, H=4096, x="bf16", res="f32", y=True, q=True),
        # scored routing
        # one decode step of the 384-expert layer: sigmoid scores, balance bias, 4 of 8 groups
        dict(name="route batch", op="route", T=64, E=384, k=8, score="sigmoid", bias=True, groups=8, keep=4, top=2,
             renorm=True, scale=2.5, off=0),
        # a prefill of the 512-expert layer: softmax over all experts, some of them out of service
        dict(name="route prompt", op="route", T=4099, E=512, k=10, score="softmax", bias=True, groups=1, keep=1, top=1,
             renorm=False, scale=1.0, off=16),
        # the largest prefill of the 384-expert layer
        dict(name="route prefill", op="route", T=65536, E=384, k=8, score="sigmoid", bias=True, groups=8, keep=4, top=2,
             renorm=True, scale=2.5, off=0),
        # dense products
        # router logits of a serving batch: few rows, few columns, all of K
        dict(name="linear router", op="linear", T=64, N=384, K=4096, kind="bf16", act="none", bias=False, res="none",
             out="f32"),
        # shared expert of one decoded token: FC1 with SwiGLU, bound by reading the weights
        dict(name="linear token", op="linear", T=1, N=4096, K=4096, kind="bf16", act="swiglu", bias=False, res="none",
             out="bf16"),
        # a ragged middle-sized batch with every part of the epilogue
        dict(name="linear ragged", op="linear", T=1001, N=1000, K=2016, kind="bf16", act="gelu", bias=True, res="f32",
             out="f32"),
        # shared expert of a prefill: FC1 with SwiGLU
        dict(name="linear prefill", op="linear", T=8192, N=4096, K=4096, kind="bf16", act="swiglu", bias=False,
             res="none", out="bf16"),
        # shared expert of a prefill in MXFP8: FC2 with the routed output added
        dict(name="linear mxfp8", op="linear", T=8192, N=4096, K=2048, kind="mxfp8", act="none", bias=False, res="bf16",
             out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "route", "linear", "linear"))
    if op == "norm":
        q = rng.random() < 0.5
        H = 32 * _log(rng, 8, 256) if q else 8 * _log(rng, 8, 1024)
        T = _log(rng, 1, min(65536, 32768 * 4096 // H))
        return dict(op=op, T=T, H=H, x=rng.choice(("f32", "bf16")), res=rng.choice(("none", "bf16", "f32")),
                    y=not q or rng.random() < 0.7, q=q)
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        E = groups * max(2, _log(rng, 8, 1024) // groups)
        keep = rng.randint(1, groups)
        k = rng.randint(1, min(16, keep * (E // groups)))
        return dict(op=op, T=_log(rng, 1, 65536 * 384 // max(E, 384)), E=E, k=k, score=rng.choice(("softmax", "sigmoid")),
                    bias=rng.random() < 0.6, groups=groups, keep=keep, top=rng.choice((1, 2)), renorm=rng.random() < 0.6,
                    scale=rng.choice((1.0, 2.5)), off=0)
    kind = rng.choice(("bf16", "bf16", "mxfp8"))
    act = rng.choice(("none", "relu", "gelu", "silu", "swiglu"))
    K = 32 * _log(rng, 4, 128) if kind == "mxfp8" else 8 * _log(rng, 16, 512)
    N = _log(rng, 8, 4096)
    N += N % 2 if act == "swiglu" else 0
    res = rng.choice(("none", "bf16", "f32"))
    return dict(op=op, T=_log(rng, 1, 8192), N=N, K=K, kind=kind, act=act, bias=rng.random() < 0.5, res=res,
                out="bf16" if kind == "mxfp8" else rng.choice(("bf16", "f32")))


# ---------------------------------------------------------------------------- inputs
def _type(name):
    return {"f32": F32, "bf16": BF16}[name]


def _quantize(v):
    """MXFP8 of values [rows][K]: e4m3 elements and e8m0 scales, as tensors of those types."""
    rows, K = v.shape
    b = v.reshape(rows, K // 32, 32)
    amax = b.abs().amax(-1, keepdim=True)
    _, e = torch.frexp(amax.double())  # amax = m * 2^e with m in [0.5, 1)
    shared = torch.where(amax > 0, e - 9, -127).clamp(-127, 127)
    scaled = torch.ldexp(b.double(), -shared).clamp(-448.0, 448.0).float()
    elems = scaled.to(torch.float8_e4m3fn).reshape(rows, K)
    return elems, (shared + 127).to(torch.uint8).reshape(rows, K // 32).view(torch.float8_e8m0fnu)


def _values(elems, scales, dtype):
    """The values an MXFP8 matrix stands for."""
    rows, K = elems.shape
    s = torch.exp2(scales.view(torch.uint8).to(dtype) - 127.0)
    return (elems.to(dtype).reshape(rows, K // 32, 32) * s[..., None]).reshape(rows, K)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = dict(case=case)
    T = case["T"]
    if case["op"] == "norm":
        H = case["H"]
        s["x"] = (0.5 * normal(T, H)).to(_type(case["x"]))
        s["weight"] = (1.0 + 0.2 * normal(H)).to(BF16)
        s["res"] = None
        if case["res"] != "none":
            # a residual stream grows with depth and has a few large channels
            size = torch.exp(normal(H)) + 40.0 * (torch.rand(H, generator=g, device="cuda") < 0.004)
            s["res"] = (size * normal(T, H)).to(_type(case["res"]))
            s["res_out"] = torch.empty_like(s["res"])
        s["y"] = torch.empty(T, H, dtype=BF16, device="cuda") if case["y"] else None
        s["q"] = torch.empty(T, H, dtype=torch.uint8, device="cuda") if case["q"] else None
        s["qs"] = torch.empty(T, H // 32, dtype=torch.uint8, device="cuda") if case["q"] else None
    elif case["op"] == "route":
        E, k = case["E"], case["k"]
        rank = torch.randperm(E, generator=g, device="cuda") + 1
        s["logits"] = normal(T, E) - 1.1 * torch.log(rank.float())
        s["bias"] = None
        if case["bias"]:
            # what balancing leaves: popular experts pushed down
            s["bias"] = 0.02 * torch.log(rank.float()) + 0.01 * normal(E)
            if case["off"]:
                s["bias"][torch.randperm(E, generator=g, device="cuda")[:case["off"]]] = -math.inf
        s["ids"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        s["gates"] = torch.empty(T, k, dtype=F32, device="cuda")
    else:
        N, K = case["N"], case["K"]
        n_out = N // 2 if case["act"] == "swiglu" else N
        x, w = normal(T, K).to(BF16), (normal(N, K) / math.sqrt(K)).to(BF16)
        if case["kind"] == "mxfp8":
            (s["x"], s["xs"]), (s["w"], s["ws"]) = _quantize(x.float()), _quantize(w.float())
        else:
            s["x"], s["w"], s["xs"], s["ws"] = x, w, None, None
        s["bias"] = 0.3 * normal(N) if case["bias"] else None
        s["res"] = normal(T, n_out).to(_type(case["res"])) if case["res"] != "none" else None
        s["out"] = torch.empty(T, n_out, dtype=_type(case["out"]), device="cuda")
    return s


# ---------------------------------------------------------------------------- one pass
def run(s):
    if own:
        from bit_moe_expert_top_amd import ops

        return _own(s, ops)
    return {"norm": _norm, "route": _route, "linear": _linear}[s["case"]["op"]](s)


def _own(s, ops):
    c = s["case"]
    if c["op"] == "norm":
        ops.moe_add_rmsnorm(s["x"], s["weight"], EPS, residual=s["res"], residual_out=s.get("res_out"), y=s["y"],
                            q=s["q"], q_scales=s["qs"])
        return _norm_outputs(s.get("res_out"), s["y"],
                             None if s["q"] is None else s["q"].view(torch.float8_e4m3fn),
                             None if s["qs"] is None else s["qs"].view(torch.float8_e8m0fnu))
    if c["op"] == "route":
        ops.moe_route_scored(s["logits"], c["k"], score=c["score"], bias=s["bias"], n_group=c["groups"],
                             topk_group=c["keep"], group_top=c["top"], renormalize=c["renorm"], scale=c["scale"],
                             topk_ids=s["ids"], topk_w=s["gates"])
        return {"ids": s["ids"], "gates": s["gates"]}
    ops.moe_linear(s["x"], s["w"], x_scales=s["xs"], w_scales=s["ws"], bias=s["bias"], act=c["act"], residual=s["res"],
                   out=s["out"])
    return {"out": s["out"]}


def _norm_outputs(res, y, q, qs):
    return {k: v for k, v in (("res", res), ("y", y), ("q", q), ("scales", qs)) if v is not None}


def _norm(s):
    c = s["case"]
    v, res = s["x"].float(), None
    if s["res"] is not None:
        res = (v + s["res"].float()).to(s["res"].dtype)  # the residual stream as it is kept
        v = res.float()
    y = (v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * s["weight"].float()).to(BF16)
    q, qs = _quantize(y.float()) if c["q"] else (None, None)
    return _norm_outputs(res, y if c["y"] else None, q, qs)


def _route(s):
    # in 64 bits: the choice of experts hangs on scores that lie next to each other
    c = s["case"]
    T, E, G = c["T"], c["E"], c["groups"]
    logits = s["logits"].double()
    score = torch.sigmoid(logits) if c["score"] == "sigmoid" else torch.softmax(logits, -1)
    choice = score if s["bias"] is None else score + s["bias"].double()
    dead = choice == -math.inf
    key = logits if s["bias"] is None else choice
    key = torch.where(dead, -1e300, key)  # taken last
    if G > 1:
        by_group = torch.sort(choice.reshape(T, G, E // G), dim=-1, descending=True).values[..., :c["top"]]
        total = torch.where(by_group == -math.inf, 0.0, by_group).sum(-1)
        total = torch.where(by_group[..., 0] == -math.inf, -math.inf, total)
        kept = torch.sort(total, dim=-1, descending=True, stable=True).indices[:, :c["keep"]]
        mask = torch.zeros(T, G, dtype=torch.bool, device=logits.device).scatter_(1, kept, True)
        key = torch.where(mask[..., None].expand(T, G, E // G).reshape(T, E), key, -math.inf)
    ids = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :c["k"]]
    gates = torch.where(dead, 0.0, score).gather(1, ids)
    if c["renorm"]:
        total = gates.sum(-1, keepdim=True)
        gates = torch.where(total > 0, gates / total, 0.0)
    return {"ids": ids.int(), "gates": (gates * c["scale"]).float()}


def _act(a, act):
    if act == "relu":
        return torch.clamp(a, min=0.0)
    if act == "gelu":
        return 0.5 * a * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (a + 0.044715 * a * a * a)))
    if act == "silu":
        return a / (1.0 + torch.exp(-a))
    if act == "swiglu":
        n = a.shape[1] // 2
        return a[:, :n] / (1.0 + torch.exp(-a[:, :n])) * a[:, n:]
    return a


def _linear(s):
    c = s["case"]
    mx = c["kind"] == "mxfp8"
    x = _values(s["x"], s["xs"], F32) if mx else s["x"].float()
    w = _values(s["w"], s["ws"], F32) if mx else s["w"].float()
    a = x @ w.t()
    if s["bias"] is not None:
        a = a + s["bias"]
    a = _act(a, c["act"])
    if s["res"] is not None:
        a = a + s["res"].float()
    return {"out": a.to(s["out"].dtype)}


# ---------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    size = {"f32": 4, "bf16": 2, "none": 0}
    T = case["T"]
    if case["op"] == "norm":
        per = size[case["x"]] + 2 * size[case["res"]] + (2 if case["y"] else 0) + (33 / 32 if case["q"] else 0)
        return {"bytes": T * case["H"] * per + 2 * case["H"], "flops": 5 * T * case["H"]}
    if case["op"] == "route":
        return {"bytes": 4 * T * case["E"] + 8 * T * case["k"], "flops": 8 * T * case["E"]}
    N, K = case["N"], case["K"]
    n_out = N // 2 if case["act"] == "swiglu" else N
    element = 33 / 32 if case["kind"] == "mxfp8" else 2
    return {"bytes": (T + N) * K * element + T * n_out * (size[case["res"]] + size[case["out"]]) + (4 * N if case["bias"] else 0),
            "flops": 2 * T * N * K}


# ---------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "route": _exact_route, "linear": _exact_linear}[case["op"]](case, s)


def _exact_norm(case, s):
    outs = dict(res=[], y=[], q=[], scales=[])
    step = max(1, (1 << 26) // case["H"])
    for i in range(0, case["T"], step):
        v = s["x"][i:i + step].double()
        if s["res"] is not None:
            v = (v + s["res"][i:i + step].double()).to(s["res"].dtype).double()
            outs["res"].append(v)
        y = v / torch.sqrt(v.square().mean(1, keepdim=True) + EPS) * s["weight"].double()
        outs["y"].append(y)
        if case["q"]:
            # the quantised values are those of y as a bf16 tensor
            b = y.to(BF16).double().unflatten(1, (-1, 32))
            amax = b.abs().amax(2, keepdim=True)
            power = torch.where(amax > 0, torch.floor(torch.log2(amax)) - 8, -127.0).clamp(-127, 127)
            # e4m3: steps of 2^-3 of the value's own power of two, of 2^-9 below 2^-6
            v = (b * torch.exp2(-power)).clamp(-448, 448)
            unit = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
            outs["q"].append((torch.round(v / unit) * unit).flatten(1))
            outs["scales"].append(torch.exp2(power)[..., 0])
    cat = {k: torch.cat(v) if v else None for k, v in outs.items()}
    return _norm_outputs(cat["res"], cat["y"] if case["y"] else None, cat["q"], cat["scales"])


def _exact_route(case, s):
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    l = s["logits"].double()
    if case["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-l))
    else:
        z = torch.exp(l - l.amax(1, keepdim=True))
        p = z / z.sum(1, keepdim=True)
    c = p.clone() if s["bias"] is None else p + s["bias"].double()
    live = c > -math.inf
    left = torch.ones(T, E, dtype=torch.bool, device=l.device)
    if G > 1:
        each = torch.where(live, c, -math.inf).view(T, G, E // G)
        best = each.amax(2)
        if case["top"] == 2:
            first = each.argmax(2, keepdim=True)
            second = each.scatter(2, first, -math.inf).amax(2)
            best = best + torch.where(second > -math.inf, second, 0.0)
        allowed = torch.zeros(T, G, dtype=torch.bool, device=l.device)
        for _ in range(case["keep"]):
            g = torch.where(allowed, -math.inf, best)
            # the first of the largest among the groups not taken yet
            g = ((g == g.amax(1, keepdim=True)) & ~allowed).int().argmax(1, keepdim=True)
            allowed.scatter_(1, g, True)
        left = allowed.repeat_interleave(E // G, 1)
    order = l if s["bias"] is None else c
    ids, gates = [], []
    for _ in range(k):
        # among the live ones first, then among the others: the largest, the lowest id on ties
        live_left = left & live
        some = live_left.any(1, keepdim=True)
        pool = torch.where(some, live_left, left)
        v = torch.where(pool, torch.where(live, order, 0.0), -math.inf)
        i = (pool & (v == v.amax(1, keepdim=True))).int().argmax(1, keepdim=True)
        ids.append(i)
        gates.append(torch.where(live.gather(1, i), p.gather(1, i), 0.0))
        left = left.scatter(1, i, False)
    ids, gates = torch.cat(ids, 1), torch.cat(gates, 1)
    if case["renorm"]:
        total = gates.sum(1, keepdim=True)
        gates = torch.where(total > 0, gates / total, 0.0)
    return {"ids": ids.int(), "gates": gates * case["scale"]}


def _exact_linear(case, s):
    def wide(elems, scales):
        if scales is None:
            return elems.double()
        power = scales.view(torch.uint8).double() - 127
        return elems.double() * torch.exp2(power).repeat_interleave(32, 1)

    a = torch.matmul(wide(s["x"], s["xs"]), wide(s["w"], s["ws"]).t().contiguous())
    if s["bias"] is not None:
        a += s["bias"].double()
    act = case["act"]
    if act == "relu":
        a = torch.where(a > 0, a, 0.0)
    elif act == "silu":
        a = a * torch.sigmoid(a)
    elif act == "gelu":
        a = a * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3))
    elif act == "swiglu":
        gate, up = a.chunk(2, 1)
        a = gate * torch.sigmoid(gate) * up
    if s["res"] is not None:
        a = a + s["res"].double()
    return {"out": a}
