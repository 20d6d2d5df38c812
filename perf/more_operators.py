"""Measured cases of the 8-bit products, the norms around a block and the whole mixture-of-experts layer.

A decoder block on quantized weights, between the products that are there already:

  linear       y [M, N] = x [M, K] . W^T in 8-bit integers: codes of W with a scale per output channel,
               codes of x with a scale per row (token), made in the call:
               d = max|x| / 127, code = round(x (1 / d)) (half away from zero, 32 bits)
  norm         what stands between two blocks: the block's output is normed, gated, scaled and added
               to the residual stream, and the sum is normed for the next block:
               r' = r + scale gate (y / rms(y)) w_post,  h = (r' / rms(r')) w_pre
  norm_linear  the same with h as 8-bit codes and a scale per row, and the 8-bit product that takes them
  moe          a whole mixture-of-experts layer for a few tokens: router product, top-k, SwiGLU of the
               chosen experts' 4-bit products, weighted sum

`own = False` computes each in elementary torch operations in 32 bits; `own = True` calls the
framework.  Tensors are laid out as checkpoints hold them: 8-bit codes int8 [N, K] with f32 scales
[N]; 4-bit codes two to a byte (even k in the low nibble), scales f16 or bf16 [.., N, K/G], zero
points uint8 of that shape or none (8).
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6


def listed():
    return [
        # one token through the smallest square linear of a 135M decoder: launch latency
        dict(name="linear 1x576x576 f32", op="linear", M=1, N=576, K=576, dt="f32"),
        # one token, the widest linear of a 70B decoder: the weight stream
        dict(name="linear 1x28672x8192 bf16", op="linear", M=1, N=28672, K=8192, dt="bf16"),
        # eight sequences decoded together, an 8B decoder's MLP
        dict(name="linear 8x14336x4096 f16", op="linear", M=8, N=14336, K=4096, dt="f16"),
        # a short odd prompt back to the residual stream: few outputs, long rows
        dict(name="linear 37x4096x14336 f32", op="linear", M=37, N=4096, K=14336, dt="f32"),
        # a prompt of 1024 tokens
        dict(name="linear 1024x14336x4096 bf16", op="linear", M=1024, N=14336, K=4096, dt="bf16"),
        # one decode step of a 135M decoder, norms before the next block only
        dict(name="norm 1x576 f32", op="norm", T=1, K=576, post=False, gate="none", scale=1.0, dt="f32"),
        # a prompt, norms on both sides of the block, a learned gate per channel
        dict(name="norm 4096x4096 bf16", op="norm", T=4096, K=4096, post=True, gate="channel", scale=0.7, dt="bf16"),
        # sixteen sequences decoded together: norms, then an attention projection in 8 bits
        dict(name="norm_linear 16x4096x4096 bf16", op="norm_linear", T=16, N=4096, K=4096, post=True, gate="none", scale=1.0, dt="bf16"),
        # an odd prompt through the same, gated per token and channel
        dict(name="norm_linear 611x1536x576 f16", op="norm_linear", T=611, N=1536, K=576, post=True, gate="token", scale=0.5, dt="f16"),
        # one token's mixture-of-experts layer
        dict(name="moe 1 of 64 bf16", op="moe", T=1, E=64, k=8, K=2048, F=1024, G=128, zeros=True, score="softmax", bias=False, dt="bf16"),
        # three sequences with f32 activations, many small experts, balance bias
        dict(name="moe 3 of 128 f32", op="moe", T=3, E=128, k=6, K=2048, F=768, G=32, zeros=False, score="sigmoid", bias=True, dt="f32"),
        # sixteen sequences decoded together
        dict(name="moe 16 of 64 f16", op="moe", T=16, E=64, k=8, K=2048, F=1024, G=64, zeros=True, score="softmax", bias=False, dt="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _whole(rng, lo, hi, G):
    """A row length: a multiple of the group."""
    return max(G, _log(rng, lo, hi) // G * G)


def draw(rng):
    op = rng.choice(["linear", "linear", "norm", "norm_linear", "moe", "moe"])
    dt = rng.choice(["f32", "f16", "bf16"])
    if op == "linear":
        K = _log(rng, 64, 14336)
        K = K if rng.random() < 0.2 else max(64, K // 32 * 32)  # rows of any length, mostly of whole blocks
        return dict(op=op, M=_log(rng, 1, 1024), N=min(_log(rng, 64, 28672), 14336 * 4096 // K), K=K, dt=dt)
    if op == "moe":
        E, G = _log(rng, 8, 128), rng.choice([32, 64, 128])
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op=op, T=_log(rng, 1, 16), E=E, k=rng.randint(1, min(8, E)), K=_whole(rng, 256, 2048, G), F=_whole(rng, 128, 1024, G), G=G,
                    zeros=rng.random() < 0.5, score=score, bias=score == "sigmoid" and rng.random() < 0.7, dt=dt)
    K = _log(rng, 64, 8192)
    T = min(_log(rng, 1, 4096), 4096 * 4096 // K)
    c = dict(op=op, T=T, K=K, post=rng.random() < 0.6, gate=rng.choice(["none", "channel", "token"]), scale=rng.choice([1.0, 0.5, 0.22]), dt=dt)
    if op == "norm_linear":
        c["T"], c["N"], c["dt"] = min(T, 1024), _log(rng, 64, 8192), rng.choice(["f16", "bf16"])
    return c


def _rand(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _weights8(gen, N, K):
    """Codes as a checkpoint's per-channel quantization leaves them, scales that differ by channel."""
    codes = torch.clamp(torch.round(30.0 * _rand(gen, N, K)), -127, 127).to(torch.int8)
    return codes, (0.5 + torch.rand(N, generator=gen, device="cuda")) * (0.03 / K ** 0.5)


def _weights4(gen, E, N, K, G, zeros, dt):
    """Codes, scales and zero points: bell-shaped codes, scales that differ by row and group."""
    def nibble():
        a = torch.randint(0, 8, (E, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
        return a + torch.randint(0, 9, (E, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    codes = nibble() | (nibble() << 4)
    s = (0.5 + torch.rand((E, N, K // G), generator=gen, device="cuda")) * (0.3 / K ** 0.5)
    z = torch.randint(6, 10, (E, N, K // G), generator=gen, device="cuda", dtype=torch.uint8) if zeros else None
    return codes, s.to(torch.bfloat16 if dt == "bf16" else torch.float16), z


def _activations(gen, M, K):
    """Bell-shaped, with a few channels far larger than the others, as a residual stream has them."""
    x = _rand(gen, M, K)
    x[:, torch.randint(0, K, (4,), generator=gen, device="cuda")] *= 8.0
    return x


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c, dt = case, DT[case["dt"]]
    s = dict(case=c, gate=None, post=None)
    if c["op"] == "moe":
        s["x"] = _rand(gen, c["T"], c["K"]).to(dt)
        s["router"] = (_rand(gen, c["E"], c["K"]) * (1.5 / c["K"] ** 0.5)).to(dt)
        # balance biases move in fixed small steps
        s["bias"] = 0.001 * torch.randint(-100, 101, (c["E"],), generator=gen, device="cuda").float() if c["bias"] else None
        s["w"] = [_weights4(gen, c["E"], 2 * c["F"], c["K"], c["G"], c["zeros"], c["dt"]),
                  _weights4(gen, c["E"], c["K"], c["F"], c["G"], c["zeros"], c["dt"])]
    elif c["op"] == "linear":
        s["x"] = _activations(gen, c["M"], c["K"]).to(dt)
    else:
        T, K = c["T"], c["K"]
        s["y"] = (0.3 * _rand(gen, T, K)).to(dt)
        s["r"] = _activations(gen, T, K).to(dt)
        if c["gate"] != "none":
            s["gate"] = torch.sigmoid(_rand(gen, *((K,) if c["gate"] == "channel" else (T, K)))).to(dt)
        if c["post"]:
            s["post"] = (1.0 + 0.2 * _rand(gen, K)).to(dt)
        s["pre"] = (1.0 + 0.2 * _rand(gen, K)).to(dt)
    if "N" in c:
        s["w"] = [_weights8(gen, c["N"], c["K"])]
    if own:  # laid out once, as a program does when it loads its weights
        import gguf_block_quantized_qmatmul_gb300 as q
        s["q"] = q
        if c["op"] == "moe":
            s["w"] = [q.q4g_pack(*s["w"][0], gate_up=True), q.q4g_pack(*s["w"][1])]
        elif "N" in c:
            s["w"] = [q.q8c_pack(*s["w"][0])]
    return s


# ------------------------------------------------------------------ plain forms, 32 bits


def _codes(x):
    """Codes (as 32-bit values) and scales of the rows of x."""
    d = x.abs().amax(1, keepdim=True) / 127.0
    v = x * torch.where(d != 0, 1.0 / d, 0.0)
    q = torch.trunc(v)
    q = q + torch.where((v - q).abs() >= 0.5, torch.sign(v), 0.0)
    return torch.clamp(q, -127, 127), d


def _product(q, d, w, dt):
    codes, scales = w
    return (q @ codes.float().T * scales * d).to(dt)


def _norm(x, w):
    return x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * w.float()


def _plain_norm(s):
    v = s["y"].float()
    if s["post"] is not None:
        v = _norm(v, s["post"])
    if s["gate"] is not None:
        v = v * s["gate"].float()
    r = s["r"].float() + s["case"]["scale"] * v
    return r, _norm(r, s["pre"])


def _dequantize(w):
    codes, scales, zeros = w
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float()
    c = c.unflatten(-1, (scales.shape[-1], -1))
    z = 8.0 if zeros is None else zeros.float().unsqueeze(-1)
    return ((c - z) * scales.float().unsqueeze(-1)).flatten(-2)


def _some(w, ids):
    return tuple(None if t is None else t[ids] for t in w)


def _plain_moe(s):
    c, x = s["case"], s["x"].float()
    l = x @ s["router"].float().T
    if c["score"] == "softmax":
        score = torch.exp(l - l.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
        pick = l
    else:
        score = 1.0 / (1.0 + torch.exp(-l))
        pick = score if s["bias"] is None else score + s["bias"]
    ids = torch.sort(pick, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    wt = score.gather(1, ids)
    wt = wt / wt.sum(1, keepdim=True)
    up, down = s["w"]
    few = c["T"] * c["k"] <= c["E"]  # few slots: each with its own expert's weights
    if few:
        both = (_dequantize(_some(up, ids)) @ x[:, None, :, None])[..., 0]
    else:  # every expert for every token, then the chosen ones
        both = (x @ _dequantize(up).flatten(0, 1).T).unflatten(1, (c["E"], -1))
        both = both.gather(1, ids[..., None].expand(-1, -1, both.shape[2]))
    g, u = both[..., :c["F"]], both[..., c["F"]:]
    h = g / (1.0 + torch.exp(-g)) * u
    if few:
        y = ((_dequantize(_some(down, ids)) @ h[..., None])[..., 0] * wt[..., None]).sum(1)
    else:
        every = torch.zeros((c["T"], c["E"], c["F"]), device=h.device)  # zero where an expert is not chosen
        every.scatter_(1, ids[..., None].expand(-1, -1, c["F"]), h * wt[..., None])
        y = every.flatten(1) @ _dequantize(down).transpose(1, 2).flatten(0, 1)
    return y.to(s["x"].dtype)


def _plain(s):
    c, dt = s["case"], DT[s["case"]["dt"]]
    if c["op"] == "moe":
        return _plain_moe(s)
    if c["op"] == "linear":
        return _product(*_codes(s["x"].float()), s["w"][0], dt)
    r, h = _plain_norm(s)
    if c["op"] == "norm":
        return r.to(dt), h.to(dt)
    return r.to(dt), _product(*_codes(h), s["w"][0], dt)


def run(s):
    if not own:
        return _plain(s)
    c, q = s["case"], s["q"]
    if c["op"] == "moe":
        return q.moe_layer(s["w"][0], s["w"][1], s["router"], s["x"], c["k"], score=c["score"], bias=s["bias"])
    if c["op"] == "linear":
        return q.q8c_matmul(s["w"][0], s["x"])
    if c["op"] == "norm":
        return q.block_norm(s["y"], s["pre"], residual=s["r"], post_weight=s["post"], gate=s["gate"], scale=c["scale"], eps=EPS)
    r, h = q.block_norm(s["y"], s["pre"], residual=s["r"], post_weight=s["post"], gate=s["gate"], scale=c["scale"], eps=EPS, quantize=True)
    return r, q.q8c_matmul(s["w"][0], h, dtype=s["y"].dtype)


# ------------------------------------------------------------------ 64 bits


def _exact_codes(x):
    """Codes are decided on 32-bit values, as the operator is defined: the scale and its reciprocal are rounded to 32 bits."""
    top = x.abs().max(1).values
    d = torch.div(top, torch.full_like(top, 127.0))
    v = (x * torch.nan_to_num(d.reciprocal(), posinf=0.0)[:, None]).double()
    q = torch.sign(v) * torch.floor(v.abs() + 0.5)
    return q.clamp(-127.0, 127.0), d.double()


def _exact_product(x, w):
    """Integer sums of two halves of the rows in 64 bits, scaled."""
    q, d = _exact_codes(x)
    codes, scales = w
    at = codes.shape[1] // 2
    out = torch.empty((x.shape[0], codes.shape[0]), dtype=torch.float64, device=x.device)
    for n in range(0, codes.shape[0], 4096):
        b = codes[n:n + 4096].double()
        out[:, n:n + 4096] = (torch.mm(q[:, :at], b[:, :at].T) + torch.mm(q[:, at:], b[:, at:].T)) * scales[n:n + 4096].double()
    return out * d[:, None]


def _exact_scaled(x, w):
    return x * torch.rsqrt(x.square().sum(1) / x.shape[1] + EPS)[:, None] * w.double()


def _exact_norm(s):
    v = s["y"].double()
    if s["post"] is not None:
        v = _exact_scaled(v, s["post"])
    if s["gate"] is not None:
        v = torch.mul(s["gate"].double(), v)
    r = torch.add(s["r"].double(), v, alpha=s["case"]["scale"])
    return r, _exact_scaled(r, s["pre"])


def _exact_expert(w, e):
    """One expert's weights in 64 bits, even and odd inputs put in their places."""
    codes, scales, zeros = (None if t is None else t[e] for t in w)
    out = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.float64, device=codes.device)
    half = codes.shape[1] // scales.shape[1]  # bytes per group
    sc = scales.double().repeat_interleave(half, 1)
    z = 8.0 if zeros is None else zeros.double().repeat_interleave(half, 1)
    out[:, 0::2] = sc * ((codes & 15).double() - z)
    out[:, 1::2] = sc * ((codes >> 4).double() - z)
    return out


def _exact_moe(s):
    c, x = s["case"], s["x"].double()
    l = torch.einsum("tk,ek->te", x, s["router"].double())
    score = torch.softmax(l, 1) if c["score"] == "softmax" else torch.sigmoid(l)
    pick = l if c["score"] == "softmax" else score if s["bias"] is None else score + s["bias"].double()
    ids = torch.argsort(pick, dim=1, descending=True, stable=True)[:, :c["k"]]
    wt = torch.nn.functional.normalize(score.gather(1, ids), p=1.0, dim=1)
    y = torch.zeros_like(x)
    for e in sorted(set(ids.flatten().tolist())):
        t, j = (ids == e).nonzero(as_tuple=True)
        both = torch.mm(x[t], _exact_expert(s["w"][0], e).T)
        h = torch.nn.functional.silu(both[:, :c["F"]]).mul(both[:, c["F"]:])
        y.index_add_(0, t, torch.mm(h, _exact_expert(s["w"][1], e).T) * wt[t, j][:, None])
    return y


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "moe":
        return _exact_moe(s)
    if case["op"] == "linear":
        return _exact_product(s["x"].float(), s["w"][0])
    r, h = _exact_norm(s)
    if case["op"] == "norm":
        return r, h
    return r, _exact_product(h.float(), s["w"][0])


def work(case):
    c, b = case, SIZE[case["dt"]]
    if c["op"] == "linear":
        return {"bytes": c["N"] * (c["K"] + 4.0) + c["M"] * (c["N"] + c["K"]) * b, "flops": 2.0 * c["M"] * c["N"] * c["K"]}
    if c["op"] == "moe":
        per = 0.5 + (2.5 if c["zeros"] else 2.0) / c["G"]  # bytes a weight: code, scale, 4-bit zero point
        used = c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** c["T"])  # experts that some token chose, under even routing
        return {"bytes": used * 3 * c["F"] * c["K"] * per + (c["E"] + 2 * c["T"]) * c["K"] * b,
                "flops": c["T"] * (6.0 * c["k"] * c["F"] + 2.0 * c["E"]) * c["K"]}
    rows = {"none": 0, "channel": 1, "token": c["T"]}[c["gate"]] + 1 + c["post"]  # gate and weights
    if c["op"] == "norm":  # block's output and residual in, residual and norm out
        return {"bytes": (4 * c["T"] + rows) * c["K"] * b, "flops": 10.0 * c["T"] * c["K"]}
    return {"bytes": (3 * c["T"] + rows) * c["K"] * b + c["N"] * (c["K"] + 4.0) + c["T"] * c["N"] * b,
            "flops": 2.0 * c["T"] * c["N"] * c["K"] + 14.0 * c["T"] * c["K"]}
