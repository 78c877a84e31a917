"""The grouped-expert and draft-verify operators as cases to measure.

Each case is one call of one operator on data as a routed-expert model meets it: the router's selection for a
batch with its rows grouped by expert, the products of ragged groups with their experts' 16-bit weights (forward,
fused SwiGLU, the inputs' and the weights' gradients), and the verification of drafted tokens.  Layer sizes are this
repository's: its tiny layer (H 256, F 512, 8 experts, top-2), the Mixtral-shaped layer (H 4096, F 14336, 8
experts, top-2) and the DeepSeek-V3-shaped layer (H 7168, F 2048, 256 experts, top-8).  Vocabulary sizes are generic.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def matmul(name, T, E, top, n, k, dtype, act=False, layout="nk", gather=True, out="same"):
    """One grouped product: T tokens routed to `top` of E experts, k inputs, n outputs (of each of gate and up with act)."""
    return dict(name=name, op="matmul", T=T, E=E, top=top, n=n, k=k, dtype=dtype, act=act, layout=layout, gather=gather,
                out=dtype if out == "same" else out)


def listed():
    return [
        # the smallest batch: four tokens of the tiny layer, gate/up with SwiGLU; the call's latency is what counts
        matmul("tiny gate/up, 4 tokens", 4, 8, 2, 512, 256, "bf16", act=True),
        # decode of one token: 8 experts of 256, one row each; the weights' bytes are what counts
        matmul("dsv3 gate/up, 1 token", 1, 256, 8, 2048, 7168, "bf16", act=True),
        # a draft-verify pass (3 drafted tokens and one): about 30 experts with one or two rows, the down projection
        matmul("dsv3 down, 4 tokens", 4, 256, 8, 7168, 2048, "fp16", gather=False),
        # an uneven prompt of odd length over few large experts: about 250 rows an expert
        matmul("mixtral gate/up, 1001 tokens", 1001, 8, 2, 14336, 4096, "bf16", act=True),
        # a long prompt: 2048 rows an expert, the down projection
        matmul("mixtral down, 8192 tokens", 8192, 8, 2, 4096, 14336, "bf16", gather=False),
        # the input's gradient of the gate projection in fine-tuning: the weights are read across their rows
        matmul("mixtral input grad, 4096 tokens", 4096, 8, 2, 4096, 14336, "bf16", layout="kn", gather=False),
        # the weights' gradient of the same step, kept in 32 bits as the sum that an optimiser adds up
        dict(name="mixtral weight grad, 4096 tokens", op="wgrad", T=4096, E=8, top=2, n=14336, k=4096, dtype="bf16",
             gather=True, out="fp32"),
        # many small experts: about 100 rows an expert, the gradient's bytes outweigh its products
        dict(name="dsv3 weight grad, 777 tokens", op="wgrad", T=777, E=64, top=8, n=2048, k=7168, dtype="fp16",
             gather=True, out="fp16"),
        # routing of one token's logits as the router writes them; the call's latency is what counts
        dict(name="route, 1 token", op="route", T=1, E=256, top=8, kind=1, dtype="fp32"),
        # routing of a long batch in the model's own type: equal logits occur, the lower expert goes first
        dict(name="route, 16384 tokens", op="route", T=16384, E=256, top=8, kind=0, dtype="bf16"),
        # one sequence's three drafted tokens over a small vocabulary
        dict(name="verify, 1 sequence", op="verify", B=1, D=3, V=32000, dtype="fp32", q=True),
        # a serving batch with up to five drafts each over a large, odd vocabulary
        dict(name="verify, 256 sequences", op="verify", B=256, D=5, V=129281, dtype="bf16", q=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["matmul", "matmul", "matmul", "wgrad", "wgrad", "route", "verify"])
    if op in ("matmul", "wgrad"):
        while True:
            E = _log(rng, 4, 256)
            top = rng.randint(1, min(8, E))
            T = _log(rng, 1, 8192)
            step = rng.choice([1, 8, 16, 64, 64])          # odd widths among them
            n = max(step, _log(rng, 96, 14336) // step * step)
            k = max(step, _log(rng, 96, 14336) // step * step)
            act = op == "matmul" and rng.random() < 0.4
            if T * top * n * (2 if act else 1) * k <= 0.96e12 and E * n * (2 if act else 1) * k <= 4e9:
                break
        dtype = rng.choice(["bf16", "fp16"])
        out = rng.choice([dtype, "fp32"])
        if op == "wgrad":
            return dict(op=op, T=T, E=E, top=top, n=n, k=k, dtype=dtype, gather=rng.random() < 0.5, out=out)
        layout = "nk" if act else rng.choice(["nk", "kn"])
        return dict(op=op, T=T, E=E, top=top, n=n, k=k, dtype=dtype, act=act, layout=layout, gather=rng.random() < 0.5, out=out)
    if op == "route":
        E = _log(rng, 4, 1024)
        return dict(op=op, T=_log(rng, 1, 16384), E=E, top=rng.randint(1, min(16, E)), kind=rng.randint(0, 1),
                    dtype=rng.choice(["fp32", "bf16", "fp16"]))
    return dict(op=op, B=_log(rng, 1, 256), D=rng.randint(1, 8), V=_log(rng, 1000, 150000), dtype=rng.choice(["fp32", "bf16", "fp16"]),
                q=rng.random() < 0.7)


def _groups(case, gen):
    """Routed pairs sorted by expert: each token takes `top` different experts, some experts more liked than others."""
    T, E, top = case["T"], case["E"], case["top"]
    liked = 0.5 * torch.randn(E, generator=gen, device="cuda")
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=gen, device="cuda").clamp_(1e-9, 1 - 1e-7)))
    idx = (liked + noise).topk(top, dim=1).indices
    e, pairs = torch.sort(idx.reshape(-1), stable=True)
    counts = torch.bincount(e, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return (pairs // top).to(torch.int32), offsets, counts


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = case["op"], TYPES[case["dtype"]]
    s = dict(case=case)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dt).mul_(scale)

    if op in ("matmul", "wgrad"):
        rows, s["offsets"], counts = _groups(case, gen)
        M = case["T"] * case["top"]
        s["rows"] = rows if case["gather"] else None
        s["x"] = normal(case["T"] if case["gather"] else M, case["k"])
        # the plain form's plan: which experts have rows, and the most that one has
        s["active"] = counts.nonzero()[:, 0]
        s["most"] = int(counts.max())
        if op == "matmul":
            n = case["n"] * (2 if case["act"] else 1)
            shape = (case["E"], n, case["k"]) if case["layout"] == "nk" else (case["E"], case["k"], n)
            s["w"] = normal(*shape, scale=case["k"] ** -0.5)
            s["out"] = torch.empty(M, case["n"], dtype=TYPES[case["out"]], device="cuda")
        else:
            s["dy"] = normal(M, case["n"])
            s["out"] = torch.empty(case["E"], case["n"], case["k"], dtype=TYPES[case["out"]], device="cuda")
    elif op == "route":
        T, E, k = case["T"], case["E"], case["top"]
        s["logits"] = normal(T, E, scale=1.5)
        s["out"] = (torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda"),
                    torch.empty(E + 1, dtype=torch.int32, device="cuda"),
                    torch.empty(T * k, dtype=torch.int32, device="cuda"), torch.empty(T * k, dtype=torch.int32, device="cuda"))
    else:
        B, D, V = case["B"], case["D"], case["V"]
        target = 2.5 * torch.randn(B, D + 1, V, generator=gen, device="cuda")
        if case["q"]:  # a draft model that is mostly right
            q = torch.softmax(target[:, :D] + 0.6 * torch.randn(B, D, V, generator=gen, device="cuda"), -1)
        else:          # drafts taken from earlier text: given without probabilities
            q = torch.softmax(target[:, :D], -1)
        pick = q / torch.empty_like(q).exponential_(generator=gen)
        s["draft"] = pick.argmax(-1).to(torch.int32)
        s["p"] = torch.softmax(target, -1).to(dt)
        s["q"] = q.to(dt) if case["q"] else None
        s["u"] = torch.rand(B, D + 1, generator=gen, device="cuda")
        s["lengths"] = torch.randint(max(0, D - 2), D + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        s["lengths"][: max(1, B // 2)] = D
        s["out"] = (torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, D + 1, dtype=torch.int32, device="cuda"))
    return s


def run(s):
    case = s["case"]
    if own:
        import routed_expert_ffn_03_gb300 as M
        if case["op"] == "matmul":
            return M.grouped_matmul(s["x"], s["w"], s["offsets"], rows=s["rows"], w_layout=case["layout"],
                                    act="swiglu" if case["act"] else None, out=s["out"])
        if case["op"] == "wgrad":
            return M.grouped_wgrad(s["dy"], s["x"], s["offsets"], x_rows=s["rows"], out=s["out"])
        if case["op"] == "route":
            return M.group_route(s["logits"], case["top"], router=case["kind"], out=s["out"])
        return M.verify_draft(s["p"], s["draft"], s["u"], q=s["q"], lengths=s["lengths"], out=s["out"])
    return {"matmul": _plain_matmul, "wgrad": _plain_wgrad, "route": _plain_route, "verify": _plain_verify}[case["op"]](s)


def _padded(s, v, M):
    """Rows of the groups that have any, each padded with zero rows to the longest, in 32 bits; and where each row stands."""
    a, o = s["active"], s["offsets"].long()
    at = o[a][:, None] + torch.arange(s["most"], device="cuda")
    inside = at < o[a + 1][:, None]
    at = torch.where(inside, at, M)
    v = torch.cat([v, v.new_zeros(1, v.shape[1])])
    return v[at].float(), at


def _plain_matmul(s):
    case = s["case"]
    x = s["x"] if s["rows"] is None else s["x"][s["rows"].long()]
    M = x.shape[0]
    xp, at = _padded(s, x, M)
    w = s["w"][s["active"]].float()
    y = xp @ (w.transpose(1, 2) if case["layout"] == "nk" else w)
    if case["act"]:
        g, u = y[..., : case["n"]], y[..., case["n"]:]
        y = g / (1 + torch.exp(-g)) * u
    out = y.new_empty(M + 1, case["n"], dtype=TYPES[case["out"]])
    out[at.reshape(-1)] = y.reshape(-1, case["n"]).to(out.dtype)
    return out[:M]


def _plain_wgrad(s):
    case = s["case"]
    x = s["x"] if s["rows"] is None else s["x"][s["rows"].long()]
    M = x.shape[0]
    dyp, xp = _padded(s, s["dy"], M)[0], _padded(s, x, M)[0]
    out = torch.zeros(case["E"], case["n"], case["k"], dtype=TYPES[case["out"]], device="cuda")
    out[s["active"]] = (dyp.transpose(1, 2) @ xp).to(out.dtype)
    return out


def _plain_route(s):
    case = s["case"]
    T, E, k = case["T"], case["E"], case["top"]
    l, idx = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True)
    l, idx = l[:, :k], idx[:, :k]
    z = torch.minimum(l, torch.zeros_like(l)) - torch.log1p(torch.exp(-l.abs())) if case["kind"] == 1 else l
    w = torch.exp(z - z[:, :1])
    w = w / w.sum(1, keepdim=True)
    e, pairs = torch.sort(idx.reshape(-1), stable=True)
    offsets = (e[None, :] < torch.arange(E + 1, device="cuda")[:, None]).sum(1) if T * k < 4096 else \
        torch.cat([e.new_zeros(1), torch.bincount(e, minlength=E).cumsum(0)])
    i32 = torch.int32
    return idx.to(i32), w, offsets.to(i32), (pairs // k).to(i32), pairs.to(i32)


def _plain_verify(s):
    # 64 bits: the token is found by comparing long sums with a border
    case = s["case"]
    B, D, V = case["B"], case["D"], case["V"]
    b = torch.arange(B, device="cuda")
    draft, length = s["draft"].long(), s["lengths"].long()
    pd = torch.gather(s["p"][:, :D], 2, draft[..., None])[..., 0].double()
    qd = torch.gather(s["q"], 2, draft[..., None])[..., 0].double() if case["q"] else torch.ones_like(pd)
    i = torch.arange(D, device="cuda")
    reject = ~(s["u"][:, :D].double() * qd < pd) & (i < length[:, None])
    r = torch.where(reject, i, length[:, None]).min(1).values          # the first rejected draft, or the length
    rejected = r < length
    p = s["p"][b, r].double()
    if case["q"]:
        q = s["q"][b, r.clamp(max=D - 1)].double()
    else:
        q = torch.zeros_like(p).scatter_(1, draft[b, r.clamp(max=D - 1)][:, None], 1.0)
    w = torch.where(rejected[:, None], (p - q).clamp(min=0), p)
    w = torch.where((w.sum(1) > 0)[:, None], w, p)
    c = w.cumsum(1)
    token = (c <= s["u"][:, D:].double() * c[:, -1:]).sum(1)
    j = torch.arange(D + 1, device="cuda")
    tokens = torch.cat([draft, draft.new_zeros(B, 1)], 1)
    tokens = torch.where(j < r[:, None], tokens, torch.where(j == r[:, None], token[:, None], -1))
    return r.to(torch.int32), tokens.to(torch.int32)


def _active(case):
    """Experts that have rows, on average, when each token takes `top` of E."""
    return case["E"] * (1 - (1 - case["top"] / case["E"]) ** case["T"])


def work(case):
    op = case["op"]
    if op in ("matmul", "wgrad"):
        M, n, k = case["T"] * case["top"], case["n"], case["k"]
        x = (case["T"] if case["gather"] else M) * k * 2
        index = 4 * (case["E"] + 1) + (4 * M if case["gather"] else 0)
        if op == "matmul":
            nw = n * (2 if case["act"] else 1)
            return {"bytes": _active(case) * nw * k * 2 + x + index + M * n * SIZE[case["out"]], "flops": 2.0 * M * nw * k}
        return {"bytes": x + index + M * n * 2 + case["E"] * n * k * SIZE[case["out"]], "flops": 2.0 * M * n * k}
    if op == "route":
        T, E, k = case["T"], case["E"], case["top"]
        return {"bytes": T * E * SIZE[case["dtype"]] + 16 * T * k + 4 * (E + 1), "flops": 0.0}
    # one row of p for each sequence, and one of q where a draft is rejected (about three of four)
    B, D, V = case["B"], case["D"], case["V"]
    return {"bytes": B * V * SIZE[case["dtype"]] * (1.75 if case["q"] else 1.0) + B * (4 * (D + 1) * 3 + 8), "flops": 0.0}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("matmul", "wgrad"):
        o = s["offsets"].tolist()
        if op == "matmul":
            out = torch.zeros(case["T"] * case["top"], case["n"], dtype=torch.float64, device="cuda")
        else:
            out = torch.zeros(case["E"], case["n"], case["k"], dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            a, z = o[e], o[e + 1]
            if a == z:
                continue
            x = (s["x"][a:z] if s["rows"] is None else s["x"].index_select(0, s["rows"][a:z])).double()
            if op == "wgrad":
                out[e] = s["dy"][a:z].double().T.mm(x)
                continue
            w = s["w"][e].double()
            if case["layout"] == "nk":
                w = w.T
            if case["act"]:
                g = x.mm(w[:, : case["n"]])
                out[a:z] = g * torch.sigmoid(g) * x.mm(w[:, case["n"]:])
            else:
                out[a:z] = x.mm(w)
        return out
    if op == "route":
        T, E, k = case["T"], case["E"], case["top"]
        l = s["logits"].double()
        # the expert's place among its token's: those above it, and equal ones with a lower id
        place = torch.empty(T, E, dtype=torch.int64, device="cuda")
        low = torch.ones(E, E, dtype=torch.bool, device="cuda").tril(-1)
        for t in range(0, T, 64):
            v = l[t:t + 64]
            a, c = v[:, None, :], v[:, :, None]
            place[t:t + 64] = ((a > c) | ((a == c) & low)).sum(2)
        idx = place.argsort(1)[:, :k]
        chosen = l.gather(1, idx)
        if case["kind"] == 1:
            chosen = -torch.log1p(torch.exp(-chosen))
        w = torch.softmax(chosen, 1)
        flat = idx.reshape(-1)
        pairs = (flat * (T * k) + torch.arange(T * k, device="cuda")).argsort()
        offsets = torch.searchsorted(flat[pairs].contiguous(), torch.arange(E + 1, device="cuda"))
        return idx, w, offsets, pairs // k, pairs
    count, rows = [], []
    draft, length, u = s["draft"].tolist(), s["lengths"].tolist(), s["u"].double().tolist()
    for b in range(case["B"]):
        out, p, w = [], None, None
        for i in range(length[b]):
            p, t = s["p"][b, i].double(), draft[b][i]
            q = s["q"][b, i].double() if case["q"] else torch.zeros_like(p).index_fill_(0, torch.tensor([t], device="cuda"), 1.0)
            if u[b][i] * float(q[t]) < float(p[t]):
                out.append(t)
                continue
            w = torch.relu(p - q)
            break
        if w is None:
            w = s["p"][b, length[b]].double()
        elif not float(w.sum()) > 0:
            w = p
        c = w.cumsum(0)
        count.append(len(out))
        out.append(int(torch.searchsorted(c, u[b][-1] * c[-1:], right=True)))
        rows.append(out + [-1] * (case["D"] + 1 - len(out)))
    return torch.tensor(count), torch.tensor(rows)
