"""The operators around the FP8 linear layers of a transformer block: cases, plain forms and exact values.

Four operators, named by a case's "op":

  rmsnorm   z = x + residual; v = z * rsqrt(mean(z^2) + eps) * weight; v quantized per token in
            groups of `block` channels (e4m3 codes and float32 or UE8M0 scales), the new residual
            bf16(z), and on request bf16(v)
  silu_mul  v = silu(gate) * up, quantized in the same way (the input of a down projection)
  route     softmax over a token's expert logits, its k largest in falling order (ties: the lowest
            index), weights renormalized over the chosen ones
  moe       a mixture-of-experts layer for few tokens on e4m3 expert weights with 128 x 128 block
            scales: x quantized per token, gate and up products, silu(gate) * up quantized, down
            product, the weighted sum over the token's experts

`own` false: elementary torch operations in float32.  `own` true: the calls that a user makes of
fine_grained_fp8_act_b200.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
FLOOR = 2.0 ** -126


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one token of a decoder block, hidden 7168: latency
        {"name": "norm decode 1x7168", "op": "rmsnorm", "M": 1, "K": 7168, "fmt": "float", "block": 128,
         "residual": True, "y": True},
        # an odd batch of rows of a shared step, scales for the block-scaled tensor core path
        {"name": "norm ragged 517x4096", "op": "rmsnorm", "M": 517, "K": 4096, "fmt": "ue8m0", "block": 32,
         "residual": False, "y": False},
        # a long prompt at the largest hidden size of the benchmark
        {"name": "norm prompt 16384x12288", "op": "rmsnorm", "M": 16384, "K": 12288, "fmt": "float", "block": 128,
         "residual": True, "y": False},
        # sixteen tokens between the gate/up and the down projection (Llama-3-8B widths)
        {"name": "silu decode 16x14336", "op": "silu_mul", "M": 16, "K": 14336, "fmt": "float", "block": 128,
         "y": False},
        # the dense MLP of the benchmark, 8192 tokens, width 18432
        {"name": "silu prompt 8192x18432", "op": "silu_mul", "M": 8192, "K": 18432, "fmt": "ue8m0", "block": 128,
         "y": False},
        # routing of one decoded token; of a prompt; of many tokens over few experts with bf16 logits (ties)
        {"name": "route decode 1x256", "op": "route", "T": 1, "E": 256, "k": 8, "dtype": "float32"},
        {"name": "route prompt 16384x256", "op": "route", "T": 16384, "E": 256, "k": 8, "dtype": "float32"},
        {"name": "route bf16 5001x60", "op": "route", "T": 5001, "E": 60, "k": 4, "dtype": "bfloat16"},
        # one decoded token through the benchmark's expert layer: 8 of 256 experts are read
        {"name": "moe decode 1 of 256", "op": "moe", "T": 1, "E": 256, "k": 8, "H": 7168, "I": 2048, "fmt": "ue8m0",
         "local": 1.0},
        # a batch of sequences on a few wide experts, most of them read by several tokens
        {"name": "moe batch 24 of 8", "op": "moe", "T": 24, "E": 8, "k": 2, "H": 4096, "I": 14336, "fmt": "float",
         "local": 1.0},
        # one rank of an expert-parallel group: only some of the slots are its own; odd widths
        {"name": "moe shard 37 of 64", "op": "moe", "T": 37, "E": 64, "k": 6, "H": 2064, "I": 1424, "fmt": "ue8m0",
         "local": 0.4},
        # a batch of 64 sequences through the benchmark's expert layer: nearly every expert is read
        {"name": "moe batch 64 of 256", "op": "moe", "T": 64, "E": 256, "k": 8, "H": 7168, "I": 2048, "fmt": "float",
         "local": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rmsnorm", "silu_mul", "route", "moe", "moe"])
    fmt = rng.choice(["float", "ue8m0"])
    if op in ("rmsnorm", "silu_mul"):
        K = 16 * _log(rng, 8, 1152 if op == "silu_mul" else 768)
        M = _log(rng, 1, min(16384, 150000000 // K))
        c = {"op": op, "M": M, "K": K, "fmt": fmt, "block": rng.choice([128, 128, 64, 32]), "y": rng.random() < 0.3}
        if op == "rmsnorm":
            c["residual"] = rng.random() < 0.7
        return c
    if op == "route":
        E = rng.choice([8, 16, 60, 64, 128, 160, 256, 384, 512])
        return {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, min(E, 12)),
                "dtype": rng.choice(["float32", "bfloat16"])}
    E = rng.choice([8, 16, 40, 64, 128])
    return {"op": op, "T": _log(rng, 1, 64), "E": E, "k": rng.randint(1, min(E, 8)), "H": 16 * _log(rng, 16, 320),
            "I": 16 * _log(rng, 8, 96), "fmt": fmt, "local": rng.choice([1.0, 1.0, 0.5])}


# ----------------------------------------------------------------- inputs --
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _bf16(shape, g, std=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(0.0, std, generator=g)


def _activations(M, K, g, std=1.0):
    """Normal rows with a hundredth of the channels twenty times as large, as a residual stream has them."""
    x = _bf16((M, K), g, std)
    x[:, torch.randperm(K, generator=g, device=DEV)[:max(1, K // 100)]] *= 20.0
    return x


def _experts(E, N, K, g, fmt):
    """e4m3 codes [E, N, K] of normal weights (each block's largest value near 448) and their block scales."""
    wq = torch.empty((E, N, K), dtype=E4M3, device=DEV)
    step = max(1, (1 << 28) // (N * K))
    for e in range(0, E, step):
        n = min(step, E - e)
        wq[e:e + n] = _bf16((n, N, K), g, 448.0 / 4.2).clamp_(-448.0, 448.0).to(E4M3)
    s = torch.empty((E, -(-N // 128), -(-K // 128)), dtype=torch.float32, device=DEV)
    s.normal_(0.0, 0.4, generator=g).exp_().mul_(0.02 * 4.2 / 448.0)
    if fmt == "ue8m0":
        s = torch.exp2(torch.round(torch.log2(s))).to(E8M0)
    return wq, s


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"case": c}
    if c["op"] == "rmsnorm":
        s["x"] = _activations(c["M"], c["K"], g)
        s["weight"] = (1.0 + 0.2 * torch.randn(c["K"], generator=g, device=DEV)).to(torch.bfloat16)
        s["residual"] = _activations(c["M"], c["K"], g, 2.0) if c["residual"] else None
        s["eps"] = 1e-6
    elif c["op"] == "silu_mul":
        s["gate_up"] = _bf16((c["M"], 2 * c["K"]), g, 1.5)  # the two halves of one projection's output
    elif c["op"] == "route":
        s["logits"] = torch.randn((c["T"], c["E"]), generator=g, device=DEV).mul_(2.0).to(getattr(torch, c["dtype"]))
    else:
        T, E, k = c["T"], c["E"], c["k"]
        s["x"] = _activations(T, c["H"], g)
        popular = torch.randn(E, generator=g, device=DEV) * 0.5
        noise = torch.rand((T, E), generator=g, device=DEV).clamp_min_(1e-30)
        ids = torch.sort(popular - torch.log(-torch.log(noise)), dim=1, descending=True).indices[:, :k]
        away = torch.rand((T, k), generator=g, device=DEV) >= c["local"]
        s["ids"] = ids.masked_fill(away, -1).to(torch.int32)  # -1: another rank's expert
        w = torch.rand((T, k), generator=g, device=DEV) + 0.1
        s["weights"] = w / w.sum(1, keepdim=True)
        s["w13"], s["s13"] = _experts(E, 2 * c["I"], c["H"], g, c["fmt"])
        s["w2"], s["s2"] = _experts(E, c["H"], c["I"], g, c["fmt"])
    if own and c["op"] == "moe":
        import fine_grained_fp8_act_b200 as fg8
        # the workspace that a serving program allocates once per layer shape
        n = fg8.fg8_moe_mlp_workspace_bytes(c["T"], c["k"], c["E"], c["H"], c["I"], fg8.scale_fmt_code(c["fmt"]))
        s["workspace"] = torch.zeros(n, dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------ plain forms --
def _ceil_pow2(s):
    m, e = torch.frexp(s)
    return torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e))


def _quantize(v, block, fmt):
    """float32 [..., K] -> (e4m3 codes [..., K], scales [..., ceil(K / block)] float32)."""
    K = v.shape[-1]
    n = -(-K // block)
    g = torch.nn.functional.pad(v, (0, n * block - K)).unflatten(-1, (n, block))
    amax = g.abs().amax(-1)
    s = (amax / torch.full_like(amax, 448.0)).clamp_min(FLOOR)  # by a tensor: a true division on every device
    if fmt == "ue8m0":
        s = _ceil_pow2(s)
    q = (g / s[..., None]).clamp(-448.0, 448.0).to(E4M3)
    return q.flatten(-2)[..., :K].contiguous(), s


def _scales_out(s, fmt):
    return s.to(E8M0) if fmt == "ue8m0" else s


def _dequantize(q, s, block=128):
    """e4m3 [..., N, K] with block scales [..., ceil(N/block), ceil(K/block)] -> float32."""
    n, k = q.shape[-2:]
    s = s.float().repeat_interleave(block, -2)[..., :n, :].repeat_interleave(block, -1)[..., :k]
    return q.float().mul_(s)


def _act_values(v, fmt):
    q, s = _quantize(v, 128, fmt)
    return q.float() * s.repeat_interleave(128, -1)[..., :q.shape[-1]]


def _silu_mul(g, u):
    return g / (1.0 + torch.exp(-g)) * u


def _pick(t, i):
    return t.view(torch.uint8)[i].view(t.dtype) if t.element_size() == 1 else t[i]


def _plain(s):
    c = s["case"]
    if c["op"] == "rmsnorm":
        z = s["x"].float()
        if s["residual"] is not None:
            z = z + s["residual"].float()
        v = z * (1.0 / torch.sqrt(z.square().mean(-1, keepdim=True) + s["eps"])) * s["weight"].float()
        q, sc = _quantize(v, c["block"], c["fmt"])
        return {"codes": q, "scales": _scales_out(sc, c["fmt"]),
                "residual": z.to(torch.bfloat16) if s["residual"] is not None else None,
                "y": v.to(torch.bfloat16) if c["y"] else None}
    if c["op"] == "silu_mul":
        v = _silu_mul(s["gate_up"][:, :c["K"]].float(), s["gate_up"][:, c["K"]:].float())
        q, sc = _quantize(v, c["block"], c["fmt"])
        return {"codes": q, "scales": _scales_out(sc, c["fmt"]), "y": v.to(torch.bfloat16) if c["y"] else None}
    if c["op"] == "route":
        l = s["logits"].float()
        top, ids = torch.sort(l, dim=1, descending=True, stable=True)
        top, ids = top[:, :c["k"]], ids[:, :c["k"]]
        w = torch.exp(top - top[:, :1])
        return {"ids": ids.to(torch.int32), "weights": w / w.sum(1, keepdim=True)}
    T, E, k, I = c["T"], c["E"], c["k"], c["I"]
    x = _act_values(s["x"].float(), c["fmt"])
    live = s["ids"] >= 0
    if T * k <= E:  # few pairs: the chosen experts' matrices, one per pair
        e = s["ids"].clamp_min(0).flatten().long()
        h = torch.bmm(_dequantize(_pick(s["w13"], e), _pick(s["s13"], e)), x.repeat_interleave(k, 0)[:, :, None])[..., 0]
        h = _act_values(_silu_mul(h[:, :I], h[:, I:]), c["fmt"])
        o = torch.bmm(_dequantize(_pick(s["w2"], e), _pick(s["s2"], e)), h[:, :, None])[..., 0]
        return {"y": (o.unflatten(0, (T, k)) * (s["weights"] * live)[..., None]).sum(1).to(torch.bfloat16)}
    # many pairs: every token through every expert, then the chosen ones' weighted sum
    h = torch.matmul(x, _dequantize(s["w13"], s["s13"]).transpose(1, 2))
    h = _act_values(_silu_mul(h[..., :I], h[..., I:]), c["fmt"])
    o = torch.matmul(h, _dequantize(s["w2"], s["s2"]).transpose(1, 2))
    chosen = s["ids"][..., None] == torch.arange(E, dtype=torch.int32, device=DEV)
    w = (chosen * s["weights"][..., None]).sum(1)
    return {"y": (o * w.t()[..., None]).sum(0).to(torch.bfloat16)}


def _own(s):
    import fine_grained_fp8_act_b200 as fg8
    c = s["case"]
    if c["op"] == "rmsnorm":
        q, sc, r, y = fg8.rmsnorm_quant(s["x"], s["weight"], s["eps"], s["residual"], c["fmt"], block=c["block"],
                                        return_y=c["y"])
        return {"codes": q, "scales": sc, "residual": r, "y": y}
    if c["op"] == "silu_mul":
        q, sc, y = fg8.silu_mul_quant(s["gate_up"][:, :c["K"]], s["gate_up"][:, c["K"]:], c["fmt"], block=c["block"],
                                      return_y=c["y"])
        return {"codes": q, "scales": sc, "y": y}
    if c["op"] == "route":
        ids, w = fg8.moe_route(s["logits"], c["k"])
        return {"ids": ids, "weights": w}
    return {"y": fg8.moe_mlp(s["x"], s["ids"], s["weights"], s["w13"], s["s13"], s["w2"], s["s2"], c["fmt"],
                             workspace=s["workspace"])}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- work --
def work(case):
    c = case
    if c["op"] in ("rmsnorm", "silu_mul"):
        n = c["M"] * c["K"]
        scales = c["M"] * -(-c["K"] // c["block"]) * (4 if c["fmt"] == "float" else 1)
        extra = 2 * n if c["y"] else 0
        if c["op"] == "silu_mul":
            return {"bytes": 5 * n + scales + extra, "flops": 8 * n}
        return {"bytes": (7 if c["residual"] else 3) * n + 2 * c["K"] + scales + extra, "flops": 8 * n}
    if c["op"] == "route":
        n = c["T"] * c["E"]
        return {"bytes": n * (4 if c["dtype"] == "float32" else 2) + 8 * c["T"] * c["k"], "flops": 4 * n}
    # the experts that random routing is expected to reach, each read once
    pairs = c["T"] * c["k"] * c["local"]
    reached = c["E"] * (1.0 - (1.0 - c["k"] * c["local"] / c["E"]) ** c["T"])
    return {"bytes": reached * 3 * c["H"] * c["I"] + 4 * c["T"] * c["H"], "flops": pairs * 6.0 * c["H"] * c["I"]}


# ------------------------------------------------------------------ exact --
def _codes64(v, group, fmt):
    """Values of the e4m3 codes, and scales, of each row's groups: the definition in 64 bits, with the two roundings that
    belong to it, the scale's and the quotient's to 32 bits (bf16 inputs often lie on a border between two codes)."""
    rows, K = v.shape
    codes, scales = [], []
    for k0 in range(0, K, group):
        part = v[:, k0:k0 + group]
        s = part.abs().max(dim=1, keepdim=True).values
        s = s / torch.full_like(s, 448.0)
        s = torch.where(s < FLOOR, torch.full_like(s, FLOOR), s).to(torch.float32).to(torch.float64)
        if fmt == "ue8m0":
            p = torch.pow(2.0, torch.floor(torch.log2(s)))
            p = torch.where(p > s, p / 2, p)
            p = torch.where(2 * p <= s, 2 * p, p)
            s = torch.where(p < s, 2 * p, p)
        a = torch.abs(part / s).to(torch.float32).to(torch.float64).clamp(max=448.0)
        # the spacing of e4m3 at a: 2^(floor(log2 a) - 3), at least 2^-9; ties to even by round()
        e = torch.floor(torch.log2(torch.where(a > 0, a, torch.ones_like(a)))).clamp(min=-6.0)
        ulp = torch.pow(2.0, e - 3.0)
        codes.append(torch.sign(part) * torch.round(a / ulp) * ulp)
        scales.append(s)
    return torch.cat(codes, 1), torch.cat(scales, 1)


def _expert64(q, s, block=128):
    w = q.to(torch.float64)
    sd = s.to(torch.float32).to(torch.float64)
    n = torch.arange(w.shape[0], device=DEV) // block
    k = torch.arange(w.shape[1], device=DEV) // block
    return w * sd[n][:, k]


def _rows64(v, fmt):
    q, s = _codes64(v, 128, fmt)
    return q * s[:, torch.arange(v.shape[1], device=DEV) // 128]


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    if c["op"] in ("rmsnorm", "silu_mul"):
        codes, scales, res, ys = [], [], [], []
        for r in range(0, c["M"], 1024):  # rows in slices, so that 64 bits fit beside the inputs
            if c["op"] == "rmsnorm":
                z = s["x"][r:r + 1024].to(torch.float64)
                if c["residual"]:
                    z = z + s["residual"][r:r + 1024].to(torch.float64)
                    res.append(z)
                norm = torch.sqrt((z * z).sum(dim=1) / c["K"] + s["eps"])
                v = z / norm[:, None] * s["weight"].to(torch.float64)
            else:
                both = s["gate_up"][r:r + 1024].to(torch.float64)
                gate, up = both[:, :c["K"]], both[:, c["K"]:]
                v = gate * up / (1.0 + torch.exp(-gate))
            q, sc = _codes64(v, c["block"], c["fmt"])
            codes.append(q.to(torch.float32))  # e4m3 values: exact in 32 bits
            scales.append(sc)
            if c["y"]:
                ys.append(v)
        out = {"codes": torch.cat(codes), "scales": torch.cat(scales), "y": torch.cat(ys) if ys else None}
        if c["op"] == "rmsnorm":
            out["residual"] = torch.cat(res).to(torch.float64) if res else None
        return out
    if c["op"] == "route":
        l = s["logits"].to(torch.float64)
        left, ids, vals = l.clone(), [], []
        for _ in range(c["k"]):
            best = left.max(dim=1, keepdim=True).values
            at = torch.where(left == best, torch.arange(c["E"], device=DEV), c["E"]).min(dim=1, keepdim=True).values
            ids.append(at)
            vals.append(best)
            left = left.scatter(1, at, float("-inf"))
        p = torch.softmax(torch.cat(vals, 1), dim=1)
        return {"ids": torch.cat(ids, 1).to(torch.int32), "weights": p}
    x = _rows64(s["x"].to(torch.float64), c["fmt"])
    y = torch.zeros_like(x)
    for e in range(c["E"]):
        t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
        if t.numel() == 0:
            continue
        h = x[t] @ _expert64(s["w13"][e], s["s13"][e]).t()
        h = _rows64(h[:, :c["I"]] / (1.0 + torch.exp(-h[:, :c["I"]])) * h[:, c["I"]:], c["fmt"])
        y.index_add_(0, t, (h @ _expert64(s["w2"][e], s["s2"][e]).t()) * s["weights"][t, j].to(torch.float64)[:, None])
    return {"y": y}
