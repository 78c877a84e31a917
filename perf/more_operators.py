"""The operators around the experts' products as cases to measure.

Each case is one call (or the two calls that always follow one another) on data as a routed-expert model meets it: the
norm in front of the layer with the residual's addition and an 8-bit output, its gradient; the router's selection with a
bias for balance and limited to groups of experts, its gradient; the experts' products in 8 bits; the weighted sum of
the experts' results, its gradient.  Layer sizes are this repository's: its tiny layer (H 256, F 512, 8 experts, top-2),
the Mixtral-shaped layer (H 4096, F 14336, 8 experts, top-2) and the DeepSeek-V3-shaped layer (H 7168, F 2048, 256
experts, top-8).
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
E4M3 = torch.float8_e4m3fn
EPS = 1e-6


def norm(name, T, H, dtype, residual, gain, out, eight):
    """x [T, H]; residual: the residual's type or ""; out: the type of the normalised output or "" for none; eight: 8 bits too."""
    return dict(name=name, op="norm", T=T, H=H, dtype=dtype, residual=residual, gain=gain, out=out, eight=eight)


def route(name, T, E, top, groups, keep, kind, group_score, bias, renorm, scale, dtype, op="route"):
    return dict(name=name, op=op, T=T, E=E, top=top, groups=groups, keep=keep, kind=kind, group_score=group_score, bias=bias,
                renorm=renorm, scale=scale, dtype=dtype)


def product(name, T, E, top, n, k, act, gather, quantise, out):
    return dict(name=name, op="product8", T=T, E=E, top=top, n=n, k=k, act=act, gather=gather, quantise=quantise, out=out)


def listed():
    return [
        # decode of one token: the router reads 16 bits, the experts 8; the call's latency is what counts
        norm("norm, 1 token", 1, 7168, "bf16", "bf16", "bf16", "bf16", True),
        # a long prompt in front of 8-bit experts
        norm("norm to 8 bits, 8192 tokens", 8192, 7168, "bf16", "bf16", "bf16", "", True),
        # a fine-tuning step of odd length whose residual stream is kept in 32 bits: the norm's gradient and the gain's
        dict(name="norm gradient, 8191 tokens", op="norm_grad", T=8191, H=4096, dtype="bf16", h="fp32", gain="fp32", dsum=True),
        # routing of one token, groups of experts limited; latency
        route("balanced route, 1 token", 1, 256, 8, 8, 4, 1, "top2", True, True, 2.5, "fp32"),
        # routing of a long prompt from logits in the model's own type
        route("balanced route, 16384 tokens", 16384, 256, 8, 8, 4, 1, "top2", True, True, 2.5, "bf16"),
        # the routing's gradient of a training step, softmax over all experts
        route("route gradient, 16384 tokens", 16384, 160, 6, 8, 3, 0, "max", False, False, 16.0, "fp32", op="route_grad"),
        # a draft-verify pass: four tokens' experts summed
        dict(name="combine, 4 tokens", op="combine", T=4, H=7168, top=8, dtype="bf16", out="bf16", residual=True, places=True),
        # an uneven prompt of many experts a token, added to the shared expert's result
        dict(name="combine, 2049 tokens", op="combine", T=2049, H=7168, top=8, dtype="bf16", out="bf16", residual=True, places=True),
        # a fine-tuning step of the Mixtral-shaped layer
        dict(name="combine gradient, 8192 tokens", op="combine_grad", T=8192, H=4096, top=2, dtype="bf16", places=True),
        # a draft-verify pass in 8 bits: the rows quantised, then the down projection; the weights' bytes are what counts
        product("8-bit down, 4 tokens", 4, 256, 8, 7168, 2048, False, False, True, "bf16"),
        # an uneven prompt of odd length: gate/up with SwiGLU from the norm's 8-bit rows
        product("8-bit gate/up, 1001 tokens", 1001, 8, 2, 14336, 4096, True, True, False, "bf16"),
        # a long prompt: the rows quantised, then the down projection
        product("8-bit down, 8192 tokens", 8192, 8, 2, 4096, 14336, False, False, True, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "quantise", "route", "route", "route_grad", "combine", "combine_grad", "product8",
                     "product8"])
    types = ["bf16", "bf16", "fp16", "fp32"]
    if op in ("norm", "norm_grad", "quantise"):
        step = rng.choice([1, 8, 64])                # odd widths among them
        H = max(step, _log(rng, 64, 16384) // step * step)
        T = min(_log(rng, 1, 16384), 58_000_000 // H)
        if op == "norm":
            out, eight = rng.choice([("bf16", False), ("fp16", False), ("fp32", False), ("", True), ("bf16", True)])
            return norm("", T, H, rng.choice(types), rng.choice(["", "bf16", "fp32", "fp16"]), rng.choice(["", "bf16", "fp32"]), out,
                        eight)
        if op == "norm_grad":
            return dict(op=op, T=T, H=H, dtype=rng.choice(types), h=rng.choice(types), gain=rng.choice(["", "bf16", "fp32"]),
                        dsum=rng.random() < 0.6)
        return dict(op=op, T=T, H=H, dtype=rng.choice(types))
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 4, 8, rng.randint(2, 16)])
        size = _log(rng, 8, 64)
        E = groups * size if groups > 1 else rng.randint(8, 512)
        keep = rng.randint(max(1, groups // 2), groups)
        top = rng.randint(1, min(16, keep * (E // groups)))
        return route("", _log(rng, 1, 16384), E, top, groups, keep, rng.randint(0, 1), rng.choice(["top2", "max"]),
                     op == "route" and rng.random() < 0.7, rng.random() < 0.6, rng.choice([1.0, 2.5]), rng.choice(types), op=op)
    if op in ("combine", "combine_grad"):
        H, top = _log(rng, 64, 8192), rng.randint(1, 16)
        if rng.random() < 0.7:
            H = max(8, H // 8 * 8)
        c = dict(op=op, T=min(_log(rng, 1, 8192), 110_000_000 // (H * top)), H=H, top=top, dtype=rng.choice(types),
                 places=rng.random() < 0.7)
        return c if op == "combine_grad" else dict(c, out=rng.choice(types), residual=rng.random() < 0.5)
    while True:
        E = _log(rng, 4, 256)
        top = rng.randint(1, min(8, E))
        T = _log(rng, 1, 8192)
        n, k = (max(16, _log(rng, 96, 14336) // 16 * 16) for _ in range(2))
        n -= rng.choice([0, 0, 0, 2, 5])             # widths of the results may be odd, rows in 8 bits are whole 16s
        act = rng.random() < 0.4
        if T * top * n * (2 if act else 1) * k <= 0.9e12 and E * n * (2 if act else 1) * k <= 2e9:
            break
    return product("", T, E, top, n, k, act, rng.random() < 0.5, rng.random() < 0.3, rng.choice(["bf16", "fp16", "fp32"]))


def _places(T, top, E, gen):
    """A routed batch: each token takes `top` different experts, some more liked than others.  (pairs in sorted order, counts)"""
    liked = 0.5 * torch.randn(E, generator=gen, device="cuda")
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=gen, device="cuda").clamp_(1e-9, 1 - 1e-7)))
    e, pairs = torch.sort((liked + noise).topk(top, dim=1).indices.reshape(-1), stable=True)
    return pairs, torch.bincount(e, minlength=E)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, T = case["op"], case["T"]
    s = dict(case=case)

    def normal(*shape, dtype="fp32", scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=TYPES[dtype]).mul_(scale)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if op == "norm":
        H = case["H"]
        s["x"] = normal(T, H, dtype=case["dtype"])
        s["residual"] = normal(T, H, dtype=case["residual"], scale=2.0) if case["residual"] else None
        s["gain"] = normal(H, dtype=case["gain"], scale=0.2).add_(1.0) if case["gain"] else None
        s["want"] = (("out",) if case["out"] else ()) + (("out8",) if case["eight"] else ())
    elif op == "norm_grad":
        H = case["H"]
        s["dy"] = normal(T, H, dtype=case["dtype"])
        s["h"] = normal(T, H, dtype=case["h"], scale=2.0)
        s["rstd"] = (1 / torch.sqrt(s["h"].double().square().mean(1) + EPS)).float()
        s["gain"] = normal(H, dtype=case["gain"], scale=0.2).add_(1.0) if case["gain"] else None
        s["dsum"] = normal(T, H, dtype=case["h"]) if case["dsum"] else None
    elif op == "quantise":
        s["x"] = normal(T, case["H"], dtype=case["dtype"])
    elif op in ("route", "route_grad"):
        E, k = case["E"], case["top"]
        s["logits"] = normal(T, E, dtype=case["dtype"], scale=1.5)
        s["bias"] = normal(E, scale=0.05) if case["bias"] else None
        if op == "route_grad":
            s["idx"] = uniform(T, E).topk(k, dim=1).indices.to(torch.int32)
            s["dweights"] = normal(T, k)
    elif op in ("combine", "combine_grad"):
        H, k = case["H"], case["top"]
        s["y"] = normal(T * k, H, dtype=case["dtype"])
        s["weights"] = torch.softmax(normal(T, k), 1)
        s["places"] = None
        if case["places"]:
            pairs, _ = _places(T, k, max(2 * k, 8), gen)
            s["places"] = torch.empty(T * k, dtype=torch.int32, device="cuda")
            s["places"][pairs] = torch.arange(T * k, dtype=torch.int32, device="cuda")
            s["places"] = s["places"].view(T, k)
        if op == "combine":
            s["residual"] = normal(T, H, dtype=case["out"]) if case["residual"] else None
        else:
            s["dout"] = normal(T, H, dtype=case["dtype"])
    else:
        E, k, top = case["E"], case["k"], case["top"]
        n = case["n"] * (2 if case["act"] else 1)
        pairs, counts = _places(T, top, E, gen)
        s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        s["offsets"][1:] = counts.cumsum(0)
        s["rows"] = (pairs // top).to(torch.int32) if case["gather"] else None
        x = normal(T if case["gather"] else T * top, k, dtype="bf16")
        if case["quantise"]:
            s["x"] = x
        else:
            s["xs"] = x.float().abs().amax(1) / 448
            s["x8"] = (x.float() / s["xs"][:, None]).to(E4M3)
        s["w8"] = torch.empty(E, n, k, dtype=E4M3, device="cuda")
        for e in range(E):
            s["w8"][e] = normal(n, k, dtype="bf16", scale=100.0).clamp_(-448, 448).to(E4M3)
        s["ws"] = (uniform(E, n) + 0.5) * (0.01 * k ** -0.5)
        # the plain form's plan: which experts have rows, and the most that one has
        s["active"] = counts.nonzero()[:, 0]
        s["most"] = int(counts.max())
        s["out"] = empty(T * top, case["n"], dtype=TYPES[case["out"]])
    return s


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import routed_expert_ffn_03_gb300 as M
        if op == "norm":
            return M.rms_norm(s["x"], gain=s["gain"], residual=s["residual"], eps=EPS, want=s["want"],
                              out_dtype=TYPES.get(case["out"]))._asdict()
        if op == "norm_grad":
            return M.rms_norm_backward(s["dy"], s["h"], s["rstd"], gain=s["gain"], dsum=s["dsum"])
        if op == "quantise":
            return M.quantize_rows(s["x"])
        if op == "route":
            return M.balanced_route(s["logits"], case["top"], bias=s["bias"], router=case["kind"], groups=case["groups"],
                                    keep=case["keep"], group_score=case["group_score"], renormalize=case["renorm"],
                                    scale=case["scale"])
        if op == "route_grad":
            return M.balanced_route_backward(s["dweights"], s["logits"], s["idx"], router=case["kind"], renormalize=case["renorm"],
                                             scale=case["scale"])
        if op == "combine":
            return M.combine_rows(s["y"], s["weights"], places=s["places"], residual=s["residual"], out_dtype=TYPES[case["out"]])
        if op == "combine_grad":
            return M.combine_rows_backward(s["dout"], s["y"], s["weights"], places=s["places"])
        x8, xs = M.quantize_rows(s["x"]) if case["quantise"] else (s["x8"], s["xs"])
        return M.grouped_matmul8(x8, xs, s["w8"], s["ws"], s["offsets"], rows=s["rows"], act="swiglu" if case["act"] else None,
                                 out=s["out"])
    return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "quantise": _plain_quantise, "route": _plain_route,
            "route_grad": _plain_route_grad, "combine": _plain_combine, "combine_grad": _plain_combine_grad,
            "product8": _plain_product}[op](s)


def _eight(y):
    scale = (y.abs().amax(1) / 448).clamp(min=2.0 ** -100)
    return (y / scale[:, None]).to(E4M3), scale


def _plain_norm(s):
    case = s["case"]
    h = s["x"].float()
    out = dict(out=None, sum=None, rstd=None, out8=None, scale=None)
    if s["residual"] is not None:   # what is stored is what is normalised
        out["sum"] = (h + s["residual"].float()).to(s["residual"].dtype)
        h = out["sum"].float()
    y = h * (1 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS))
    if s["gain"] is not None:
        y = y * s["gain"].float()
    if case["out"]:
        out["out"] = y.to(TYPES[case["out"]])
    if case["eight"]:
        out["out8"], out["scale"] = _eight(y)
    return out


def _plain_norm_grad(s):
    dy, n = s["dy"].float(), s["h"].float() * s["rstd"][:, None]
    d = dy if s["gain"] is None else dy * s["gain"].float()
    dh = s["rstd"][:, None] * (d - n * (d * n).mean(1, keepdim=True))
    if s["dsum"] is not None:
        dh = dh + s["dsum"].float()
    dgain = None if s["gain"] is None else (dy * n).sum(0, dtype=torch.float64).float()   # 64 bits: a sum over all tokens
    return dh.to(s["h"].dtype), dgain


def _plain_quantise(s):
    return _eight(s["x"].float())


def _plain_scores(l, kind):
    if kind == 1:
        return 1 / (1 + torch.exp(-l))
    p = torch.exp(l - l.amax(1, keepdim=True))
    return p / p.sum(1, keepdim=True)


def _plain_route(s):
    # 64 bits: experts are chosen by comparing scores
    case = s["case"]
    T, E, k, G = case["T"], case["E"], case["top"], case["groups"]
    sc = _plain_scores(s["logits"].double(), case["kind"])
    c = sc if s["bias"] is None else sc + s["bias"].double()
    if case["keep"] < G:
        best = torch.sort(c.view(T, G, E // G), dim=2, descending=True).values
        g = best[:, :, :2].sum(2) if case["group_score"] == "top2" else best[:, :, 0]
        order = torch.sort(g, dim=1, descending=True, stable=True).indices[:, case["keep"]:]
        out = torch.zeros(T, G, dtype=torch.bool, device="cuda").scatter_(1, order, True)
        c = torch.where(out.repeat_interleave(E // G, 1), -torch.inf, c)
    idx = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(sc, 1, idx)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    e, pairs = torch.sort(idx.reshape(-1), stable=True)
    offsets = torch.cat([e.new_zeros(1), torch.bincount(e, minlength=E).cumsum(0)])
    places = torch.empty_like(pairs).scatter_(0, pairs, torch.arange(T * k, device="cuda"))
    i32 = torch.int32
    return (idx.to(i32), (w * case["scale"]).float(), offsets.to(i32), (pairs // k).to(i32), pairs.to(i32),
            places.view(T, k).to(i32))


def _plain_route_grad(s):
    case = s["case"]
    l, idx = s["logits"].float(), s["idx"].long()
    v = s["dweights"] * case["scale"]
    p = _plain_scores(l, case["kind"])
    ps = torch.gather(p, 1, idx)
    if case["renorm"]:
        r = ps / ps.sum(1, keepdim=True)
        d = r * (v - (r * v).sum(1, keepdim=True))
        if case["kind"] == 1:
            d = d * (1 - ps)
    elif case["kind"] == 1:
        d = v * ps * (1 - ps)
    else:
        return (torch.zeros_like(p).scatter_(1, idx, v * ps) - p * (v * ps).sum(1, keepdim=True)).to(s["logits"].dtype)
    return torch.zeros_like(p).scatter_(1, idx, d).to(s["logits"].dtype)


def _plain_rows(s):
    case = s["case"]
    y = s["y"] if s["places"] is None else s["y"][s["places"].reshape(-1).long()]
    return y.view(case["T"], case["top"], case["H"]).float()


def _plain_combine(s):
    out = (_plain_rows(s) * s["weights"][:, :, None]).sum(1)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return out.to(TYPES[s["case"]["out"]])


def _plain_combine_grad(s):
    case = s["case"]
    dout = s["dout"].float()[:, None, :]
    dweights = (_plain_rows(s) * dout).sum(2)
    d = (dout * s["weights"][:, :, None]).to(s["y"].dtype).view(-1, case["H"])
    dy = d
    if s["places"] is not None:
        dy = torch.empty_like(d)
        dy[s["places"].reshape(-1).long()] = d
    return dy, dweights


def _plain_product(s):
    case = s["case"]
    x8, xs = _eight(s["x"].float()) if case["quantise"] else (s["x8"], s["xs"])
    x = x8.float()
    if s["rows"] is not None:
        x, xs = x[s["rows"].long()], xs[s["rows"].long()]
    M, a, o = x.shape[0], s["active"], s["offsets"].long()
    at = o[a][:, None] + torch.arange(s["most"], device="cuda")       # rows of the groups that have any, padded to the longest
    at = torch.where(at < o[a + 1][:, None], at, M)
    x, xs = torch.cat([x, x.new_zeros(1, x.shape[1])]), torch.cat([xs, xs.new_zeros(1)])
    w = s["w8"].view(torch.uint8)[a].view(E4M3).float()
    y = (x[at] @ w.transpose(1, 2)) * xs[at][:, :, None] * s["ws"][a][:, None, :]
    if case["act"]:
        g, u = y[..., : case["n"]], y[..., case["n"]:]
        y = g / (1 + torch.exp(-g)) * u
    out = y.new_empty(M + 1, case["n"], dtype=TYPES[case["out"]])
    out[at.reshape(-1)] = y.reshape(-1, case["n"]).to(out.dtype)
    return out[:M]


def work(case):
    op, T = case["op"], case["T"]
    if op == "norm":
        H = case["H"]
        r = SIZE[case["residual"]] * 2 if case["residual"] else 0
        g = SIZE[case["gain"]] if case["gain"] else 0
        o = (SIZE[case["out"]] if case["out"] else 0) + (1 if case["eight"] else 0)
        return {"bytes": T * H * (SIZE[case["dtype"]] + r + o) + H * g + (4 * T if case["eight"] else 0), "flops": 0.0}
    if op == "norm_grad":
        H, h = case["H"], SIZE[case["h"]]
        g = SIZE[case["gain"]] + 4 if case["gain"] else 0
        return {"bytes": T * H * (SIZE[case["dtype"]] + h * (3 if case["dsum"] else 2)) + 4 * T + H * g, "flops": 0.0}
    if op == "quantise":
        return {"bytes": T * case["H"] * (SIZE[case["dtype"]] + 1) + 4 * T, "flops": 0.0}
    if op == "route":
        E, k = case["E"], case["top"]
        return {"bytes": T * E * SIZE[case["dtype"]] + 20 * T * k + 4 * (E + 1) + (4 * E if case["bias"] else 0), "flops": 0.0}
    if op == "route_grad":
        E, k, el = case["E"], case["top"], SIZE[case["dtype"]]
        dense = case["kind"] == 0 and not case["renorm"]
        return {"bytes": T * (E * el + 8 * k + (E if dense else k) * el), "flops": 0.0}
    if op == "combine":
        H, k = case["H"], case["top"]
        o = SIZE[case["out"]] * (2 if case["residual"] else 1)
        return {"bytes": T * H * (k * SIZE[case["dtype"]] + o) + T * k * (8 if case["places"] else 4), "flops": 0.0}
    if op == "combine_grad":
        H, k, el = case["H"], case["top"], SIZE[case["dtype"]]
        return {"bytes": T * H * el * (2 * k + 1) + T * k * (12 if case["places"] else 8), "flops": 0.0}
    M, n, k = T * case["top"], case["n"], case["k"]
    nw = n * (2 if case["act"] else 1)
    active = case["E"] * (1 - (1 - case["top"] / case["E"]) ** T)   # experts that have rows, on average
    x = (T if case["gather"] else M) * ((2 if case["quantise"] else 1) * k + (0 if case["quantise"] else 4))
    return {"bytes": active * nw * (k + 4) + x + 4 * (case["E"] + 1) + (4 * M if case["gather"] else 0) + M * n * SIZE[case["out"]],
            "flops": 2.0 * M * nw * k}


def _nearest_e4m3(v):
    """Magnitudes of e4m3 numbers are m 2^e: 3 bits behind the leading one down to 2^-6, steps of 2^-9 below, 448 at most."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h, total = s["x"].double(), None
        if s["residual"] is not None:
            total = (h + s["residual"].double()).to(s["residual"].dtype).double()
            h = total
        y = h * torch.rsqrt(h.square().sum(1) / case["H"] + EPS)[:, None]
        y = y if s["gain"] is None else y * s["gain"].double()
        scale = (y.abs().amax(1) / 448).clamp(min=2.0 ** -100)
        return dict(out=y if case["out"] else None, sum=total, rstd=None, out8=y / scale[:, None] if case["eight"] else None,
                    scale=scale if case["eight"] else None)
    if op == "norm_grad":
        # d/dh of h_i r g_i, r = (mean h^2 + eps)^-1/2 as it was stored
        dy, h, r = s["dy"].double(), s["h"].double(), s["rstd"].double()
        c = dy if s["gain"] is None else dy * s["gain"].double()
        dh = torch.addcmul(c * r[:, None], h, (-(c * h).sum(1) * r ** 3 / case["H"])[:, None])
        dh = dh if s["dsum"] is None else dh + s["dsum"].double()
        return dh, None if s["gain"] is None else torch.einsum("th,th,t->h", dy, h, r)
    if op == "quantise":
        x = s["x"].double()
        scale = (x.abs().amax(1) / 448).clamp(min=2.0 ** -100)
        return x / scale[:, None], scale
    if op in ("route", "route_grad"):
        T, E, k = case["T"], case["E"], case["top"]
        l = s["logits"].double()
        logp = -torch.log1p(torch.exp(-l)) if case["kind"] == 1 else l - torch.logsumexp(l, 1, keepdim=True)
        if op == "route_grad":
            idx, v = s["idx"].long(), s["dweights"].double() * case["scale"]
            with torch.enable_grad():
                q = l.clone().requires_grad_(True)
                lp = torch.nn.functional.logsigmoid(q) if case["kind"] == 1 else torch.log_softmax(q, 1)
                sel = lp.gather(1, idx)
                w = torch.softmax(sel, 1) if case["renorm"] else torch.exp(sel)
                return torch.autograd.grad((w * v).sum(), q)[0]
        sc = torch.exp(logp)
        c = sc if s["bias"] is None else sc + s["bias"].double()
        if case["keep"] < case["groups"]:
            two = c.view(T, case["groups"], -1).topk(min(2, E // case["groups"]), dim=2).values
            g = two.sum(2) if case["group_score"] == "top2" else two[..., 0]
            kept = torch.zeros_like(g).scatter_(1, g.topk(case["keep"], dim=1).indices, 1.0)
            c = c.masked_fill(kept.repeat_interleave(E // case["groups"], 1) == 0, -torch.inf)
        # equal scores (of equal 16-bit logits): the lower expert first, by its place among its token's
        place = torch.empty(T, E, dtype=torch.int64, device="cuda")
        low = torch.ones(E, E, dtype=torch.bool, device="cuda").tril(-1)
        for t in range(0, T, 64):
            a, b = c[t:t + 64, None, :], c[t:t + 64, :, None]
            place[t:t + 64] = ((a > b) | ((a == b) & low)).sum(2)
        idx = place.argsort(1)[:, :k]
        w = sc.gather(1, idx)
        w = (w / w.sum(1, keepdim=True) if case["renorm"] else w) * case["scale"]
        return None, w, None, None, None, None
    if op in ("combine", "combine_grad"):
        T, k, H = case["T"], case["top"], case["H"]
        places = torch.arange(T * k, device="cuda").view(T, k) if s["places"] is None else s["places"].long()
        out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        dy, dw = torch.empty(T * k if op == "combine_grad" else 0, H, dtype=torch.float64, device="cuda"), []
        for j in range(k):
            y, w = s["y"].index_select(0, places[:, j]).double(), s["weights"][:, j, None].double()
            if op == "combine":
                out.addcmul_(y, w)
            else:
                dw.append((y * s["dout"].double()).sum(1))
                dy[places[:, j]] = w * s["dout"].double()
        if op == "combine_grad":
            return dy, torch.stack(dw, 1)
        return out if s["residual"] is None else out + s["residual"].double()
    if case["quantise"]:
        x = s["x"].double()
        scale = (s["x"].float().abs().amax(1) / 448).clamp(min=2.0 ** -100)   # kept in 32 bits
        x = _nearest_e4m3(x / scale.double()[:, None]) * scale.double()[:, None]
    else:
        x = s["x8"].double() * s["xs"].double()[:, None]
    o = s["offsets"].tolist()
    out = torch.zeros(case["T"] * case["top"], case["n"], dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        a, z = o[e], o[e + 1]
        if a == z:
            continue
        xe = x[a:z] if s["rows"] is None else x.index_select(0, s["rows"][a:z])
        y = xe.mm(s["w8"][e].double().T) * s["ws"][e].double()
        if case["act"]:
            g = y[:, : case["n"]]
            y = g * torch.sigmoid(g) * y[:, case["n"]:]
        out[a:z] = y
    return out
