"""Measured cases of the 4-bit group-scale products and the mixture-of-experts operators.

Four operators of a decoder whose linear layers are kept in 4 bits with one scale (and
perhaps one zero point) per group of consecutive inputs, w[n][k] = s[n][k/G] (q[n][k] - z[n][k/G]):

  matmul   y [M, N] = x [M, K] . W^T: the dense linears, from one token to a prompt
  route    a router's logits [T, E] -> the top-k experts of each token, their weights, and
           the token slots sorted by expert (offsets, order)
  gate_up  h [T, k, F] = silu(x . Wg_e^T) * (x . Wu_e^T) for each token's k experts e
  down     y [T, N] = sum_j weight[t][j] (h[t][j] . Wd_e^T)

`own = False` computes each in elementary torch operations in 32 bits; `own = True` calls the
framework.  Tensors are laid out as checkpoints hold them: codes two to a byte (even k in the
low nibble), scales f16 or bf16 [.., N, K/G], zero points uint8 [.., N, K/G] or none (8).
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one token through the smallest square linear of a 135M decoder: launch latency
        dict(name="matmul 1x576x576 f32 g32", op="matmul", M=1, N=576, K=576, G=32, zeros=False, dt="f32"),
        # one token, the attention projections of an 8B decoder
        dict(name="matmul 1x4096x4096 bf16 g128", op="matmul", M=1, N=4096, K=4096, G=128, zeros=True, dt="bf16"),
        # one token, the widest linear of a 70B decoder: the weight stream
        dict(name="matmul 1x28672x8192 f16 g64", op="matmul", M=1, N=28672, K=8192, G=64, zeros=False, dt="f16"),
        # eight sequences decoded together, an 8B decoder's MLP
        dict(name="matmul 8x14336x4096 bf16 g128", op="matmul", M=8, N=14336, K=4096, G=128, zeros=True, dt="bf16"),
        # a short odd prompt with f32 activations
        dict(name="matmul 37x14336x4096 f32 g32", op="matmul", M=37, N=14336, K=4096, G=32, zeros=True, dt="f32"),
        # a prompt of 1024 tokens
        dict(name="matmul 1024x14336x4096 f16 g128", op="matmul", M=1024, N=14336, K=4096, G=128, zeros=True, dt="f16"),
        # one decode step's routing
        dict(name="route 1x64 softmax", op="route", T=1, E=64, k=6, score="softmax", bias=False, groups=1, top_groups=1, renorm=True, dt="f32"),
        # a prompt's routing with balance bias and expert groups
        dict(name="route 4096x256 sigmoid groups", op="route", T=4096, E=256, k=8, score="sigmoid", bias=True, groups=8, top_groups=4, renorm=True, dt="bf16"),
        # one token's experts
        dict(name="gate_up 1 of 64 bf16", op="gate_up", T=1, E=64, k=8, K=2048, F=1024, G=128, zeros=True, dt="bf16"),
        # a prompt's experts
        dict(name="gate_up 2048 of 64 bf16", op="gate_up", T=2048, E=64, k=8, K=2048, F=1024, G=128, zeros=True, dt="bf16"),
        # sixteen sequences decoded together, many small experts
        dict(name="down 16 of 128 f16", op="down", T=16, E=128, k=8, F=768, N=2048, G=32, zeros=False, dt="f16"),
        # a prompt's experts, back to the residual stream
        dict(name="down 2048 of 64 f16", op="down", T=2048, E=64, k=8, F=1024, N=2048, G=128, zeros=True, dt="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _inputs(rng, lo, hi, G):
    """A row length: a multiple of the group."""
    v = max(G, _log(rng, lo, hi) // G * G)
    return v + G if v == 3072 else v


def draw(rng):
    op = rng.choice(["matmul", "matmul", "route", "gate_up", "down"])
    dt = rng.choice(["f32", "f16", "bf16"])
    G, zeros = rng.choice([32, 64, 128]), rng.random() < 0.5
    if op == "matmul":
        K = _inputs(rng, 256, 14336, G)
        N = _log(rng, 64, 28672)
        N += N == 3072
        return dict(op=op, M=_log(rng, 1, 1024), N=min(N, 28672 * 4096 // K), K=K, G=G, zeros=zeros, dt=dt)
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * max(2, _log(rng, 8, 256) // groups)
        score = rng.choice(["softmax", "sigmoid"])
        top_groups = max(1, groups // 2)
        k = min(rng.randint(1, 8), top_groups * (E // groups))
        return dict(op=op, T=_log(rng, 1, 4096), E=E, k=k, score=score, bias=score == "sigmoid" and rng.random() < 0.7,
                    groups=groups, top_groups=top_groups, renorm=rng.random() < 0.7, dt=dt)
    E = _log(rng, 8, 64)
    k = rng.randint(1, min(8, E))
    T = _log(rng, 1, 2048)
    if op == "gate_up":
        F = _log(rng, 128, 1024)
        return dict(op=op, T=T, E=E, k=k, K=_inputs(rng, 256, 2048, G), F=F, G=G, zeros=zeros, dt=dt)
    return dict(op=op, T=T, E=E, k=k, F=_inputs(rng, 128, 1024, G), N=_log(rng, 256, 2048), G=G, zeros=zeros, dt=dt)


def _weights(gen, E, N, K, G, zeros, dt):
    """Codes, scales and zero points: bell-shaped codes, scales that differ by row and group."""
    def nibble():
        a = torch.randint(0, 8, (E, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
        return a + torch.randint(0, 9, (E, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    codes = nibble() | (nibble() << 4)
    s = 0.004 + 0.008 * torch.rand((E, N, K // G), generator=gen, device="cuda")
    scales = s.to(torch.bfloat16 if dt == "bf16" else torch.float16)
    z = torch.randint(6, 10, (E, N, K // G), generator=gen, device="cuda", dtype=torch.uint8) if zeros else None
    return codes, scales, z


def _routed(gen, T, E, k):
    """A finished routing: ids, weights, offsets, order."""
    logits = torch.randn((T, E), generator=gen, device="cuda") + 0.5 * torch.randn(E, generator=gen, device="cuda")
    v, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    return _plan(ids[:, :k].to(torch.int32).contiguous(), torch.softmax(v[:, :k], 1).contiguous(), E)


def _plan(ids, weights, E):
    by_expert, order = torch.sort(ids.reshape(-1), stable=True)
    offsets = torch.searchsorted(by_expert, torch.arange(E + 1, device=ids.device, dtype=ids.dtype))
    return ids, weights, offsets.to(torch.int32), order.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c, dt = case, DT[case["dt"]]
    if c["op"] == "route":
        s = dict(case=c, logits=(1.5 * torch.randn((c["T"], c["E"]), generator=gen, device="cuda")).to(dt), bias=None)
        if c["bias"]:  # balance biases move in fixed small steps
            s["bias"] = 0.001 * torch.randint(-100, 101, (c["E"],), generator=gen, device="cuda").float()
        return s
    if c["op"] == "matmul":
        E, N, K, rows = 1, c["N"], c["K"], (c["M"],)
    elif c["op"] == "gate_up":
        E, N, K, rows = c["E"], 2 * c["F"], c["K"], (c["T"],)
    else:
        E, N, K, rows = c["E"], c["N"], c["F"], (c["T"], c["k"])
    codes, scales, zeros = _weights(gen, E, N, K, c["G"], c["zeros"], c["dt"])
    s = dict(case=c, x=torch.randn(rows + (K,), generator=gen, device="cuda").to(dt))
    if c["op"] != "matmul":
        s["route"] = _routed(gen, c["T"], E, c["k"])
    if own:  # laid out once, as a program does when it loads its weights
        import gguf_block_quantized_qmatmul_gb300 as q
        s["q"] = q
        s["w"] = q.q4g_pack(codes, scales, zeros, gate_up=c["op"] == "gate_up")
        if c["op"] != "matmul":
            s["route"] = q.Route(*s["route"])
    else:
        s["w"] = (codes, scales, zeros)
    return s


# ------------------------------------------------------------------ plain forms, 32 bits


def _dequantize(w):
    codes, scales, zeros = w
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float()
    c = c.unflatten(-1, (scales.shape[-1], -1))
    z = 8.0 if zeros is None else zeros.float().unsqueeze(-1)
    return ((c - z) * scales.float().unsqueeze(-1)).flatten(-2)


def _some(w, ids):
    return tuple(None if t is None else t[ids] for t in w)


def _plain_matmul(s):
    return (s["x"].float() @ _dequantize(s["w"])[0].T).to(s["x"].dtype)


def _plain_route(s):
    c, l = s["case"], s["logits"].float()
    if c["score"] == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
        pick = l if s["bias"] is None else score + s["bias"]
    else:
        score = 1.0 / (1.0 + torch.exp(-l))
        pick = score if s["bias"] is None else score + s["bias"]
    if c["groups"] > 1:
        by = pick.unflatten(1, (c["groups"], -1))
        best = torch.sort(by, dim=2, descending=True).values
        best = best[..., :2].sum(2) if s["bias"] is not None else best[..., 0]
        keep = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        kept = torch.zeros_like(best, dtype=torch.bool).scatter_(1, keep, True)
        pick = by.masked_fill(~kept.unsqueeze(2), -math.inf).flatten(1)
    ids = torch.sort(pick, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return _plan(ids.to(torch.int32), w, c["E"])


def _plain_gate_up(s):
    c, x, ids = s["case"], s["x"].float(), s["route"][0].long()
    if c["T"] * c["k"] <= c["E"]:  # few slots: each with its own expert's weights
        both = (_dequantize(_some(s["w"], ids)) @ x[:, None, :, None])[..., 0]
    else:  # every expert for every token, then the chosen ones
        both = (x @ _dequantize(s["w"]).flatten(0, 1).T).unflatten(1, (c["E"], -1))
        both = both.gather(1, ids[..., None].expand(-1, -1, both.shape[2]))
    g, u = both[..., :c["F"]], both[..., c["F"]:]
    return (g / (1.0 + torch.exp(-g)) * u).to(s["x"].dtype)


def _plain_down(s):
    c, h, ids, wt = s["case"], s["x"].float(), s["route"][0].long(), s["route"][1]
    if c["T"] * c["k"] <= c["E"]:
        y = (_dequantize(_some(s["w"], ids)) @ h[..., None])[..., 0]
        return (y * wt[..., None]).sum(1).to(s["x"].dtype)
    every = torch.zeros((c["T"], c["E"], c["F"]), device=h.device)  # zero where an expert is not chosen
    every.scatter_(1, ids[..., None].expand(-1, -1, c["F"]), h * wt[..., None])
    return (every.flatten(1) @ _dequantize(s["w"]).transpose(1, 2).flatten(0, 1)).to(s["x"].dtype)


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"matmul": _plain_matmul, "route": _plain_route, "gate_up": _plain_gate_up, "down": _plain_down}[op](s)
    if op == "matmul":
        return s["q"].q4g_matmul(s["w"], s["x"])
    if op == "gate_up":
        return s["q"].moe_gate_up(s["w"], s["x"], s["route"])
    if op == "down":
        return s["q"].moe_down(s["w"], s["x"], s["route"])
    import gguf_block_quantized_qmatmul_gb300 as q
    c = s["case"]
    return tuple(q.moe_route(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"], top_groups=c["top_groups"],
                             group_score="top2" if c["bias"] else "max", renorm=c["renorm"]))


# ------------------------------------------------------------------ 64 bits


def _exact_rows(codes, scales, zeros, x):
    """x . W^T of one weight matrix in 64 bits, 4096 rows at a time: s (q - z) summed in two parts, even and odd k."""
    out = []
    for n in range(0, codes.shape[0], 4096):
        b, sc = codes[n:n + 4096], scales[n:n + 4096].double()
        z = torch.full_like(sc, 8.0) if zeros is None else zeros[n:n + 4096].double()
        half = codes.shape[1] // sc.shape[1]  # bytes per group
        sc, z = sc.repeat_interleave(half, 1), z.repeat_interleave(half, 1)
        lo, hi = (b & 15).double(), (b >> 4).double()
        out.append(x[:, 0::2] @ (sc * lo - sc * z).T + x[:, 1::2] @ (sc * hi - sc * z).T)
    return torch.cat(out, 1)


def _exact_route(s):
    """Which experts are chosen is decided on 32-bit values, as the operator is defined; their weights are computed in 64 bits."""
    c, l = s["case"], s["logits"].float()
    pick = l if c["score"] == "softmax" else torch.reciprocal(torch.exp(-l) + 1.0)
    if s["bias"] is not None:
        pick = pick + s["bias"]
    pick = pick.cpu().double()
    if c["groups"] > 1:
        for t in range(c["T"]):
            part = pick[t].view(c["groups"], -1)
            best = part.topk(2, 1).values.float().sum(1) if s["bias"] is not None else part.amax(1)
            chosen = sorted(range(c["groups"]), key=lambda g: (-float(best[g]), g))[:c["top_groups"]]
            for g in set(range(c["groups"])) - set(chosen):
                part[g] = -math.inf
    ids = torch.argsort(pick, dim=1, descending=True, stable=True)[:, :c["k"]]
    d = l.cpu().double()
    w = torch.sigmoid(d) if c["score"] == "sigmoid" else torch.softmax(d, 1)
    w = w.gather(1, ids)
    return None, (w / w.sum(1, keepdim=True) if c["renorm"] else w), None, None


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c = case
    if c["op"] == "route":
        return _exact_route(s)
    codes, scales, zeros = s["w"]
    x = s["x"].double()
    if c["op"] == "matmul":
        return _exact_rows(codes[0], scales[0], None if zeros is None else zeros[0], x)
    ids, wt, offsets, order = s["route"]
    at, slots = offsets.tolist(), order.long()
    rows = x.repeat_interleave(c["k"], 0) if c["op"] == "gate_up" else x.flatten(0, 1)
    out = torch.zeros((c["T"] * c["k"], c["F"] if c["op"] == "gate_up" else c["N"]), device="cuda", dtype=torch.float64)
    for e in range(c["E"]):
        mine = slots[at[e]:at[e + 1]]
        if not mine.numel():
            continue
        y = _exact_rows(codes[e], scales[e], None if zeros is None else zeros[e], rows[mine])
        if c["op"] == "gate_up":
            g, u = y.split(c["F"], 1)
            y = g * torch.sigmoid(g) * u
        out[mine] = y
    out = out.unflatten(0, (c["T"], c["k"]))
    return out if c["op"] == "gate_up" else (out * wt.double()[..., None]).sum(1)


def work(case):
    c, b = case, SIZE[case["dt"]]
    if c["op"] == "route":  # logits in; ids, weights, order and offsets out
        return {"bytes": c["T"] * c["E"] * b + c["T"] * c["k"] * 12 + 4 * (c["E"] + 1), "flops": 4.0 * c["T"] * c["E"]}
    per = 0.5 + (2.5 if c["zeros"] else 2.0) / c["G"]  # bytes a weight: code, scale, 4-bit zero point
    if c["op"] == "matmul":
        return {"bytes": c["N"] * c["K"] * per + c["M"] * (c["N"] + c["K"]) * b, "flops": 2.0 * c["M"] * c["N"] * c["K"]}
    used = c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** c["T"])  # experts that some token chose, under even routing
    slots = c["T"] * c["k"]
    if c["op"] == "gate_up":
        return {"bytes": used * 2 * c["F"] * c["K"] * per + (c["T"] * c["K"] + slots * c["F"]) * b + 8 * slots, "flops": 4.0 * slots * c["F"] * c["K"]}
    return {"bytes": used * c["N"] * c["F"] * per + (slots * c["F"] + c["T"] * c["N"]) * b + 12 * slots, "flops": 2.0 * slots * c["N"] * c["F"]}
