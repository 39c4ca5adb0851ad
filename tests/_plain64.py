"""Plain 64-bit forms of the operators around the linears, and how far a
float32 kernel that follows the same formulas may be from them.

Quantized outputs are checked against what was quantized, not code for code:
with v known up to a relative error e, a code c of a group with scale s is
right when c is within half a step of e4m3 at v / s, widened by e."""
import torch

F64 = torch.float64
U = 2.0 ** -24           # half a step of float32, relative
FLOOR = 2.0 ** -126


def e4m3_half_step(q):
    """Half the spacing of e4m3 at |q| (2^-10 for subnormals)."""
    a = q.abs().clamp(min=2.0 ** -6, max=448.0)
    return torch.exp2(torch.floor(torch.log2(a)) - 4.0)


def scale_values(xs):
    return xs.float().to(F64)


def expand(s, block, K):
    return s.repeat_interleave(block, -1)[..., :K]


def check_quantized(xq, xs, v, err, fmt, block, what=""):
    """xq e4m3 [M, K] and xs [M, G] are a quantization of values within err
    (absolute, [M, K]) of v (float64 [M, K])."""
    M, K = v.shape
    G = -(-K // block)
    assert tuple(xq.shape) == (M, K) and tuple(xs.shape) == (M, G)
    s = scale_values(xs)
    pad = torch.nn.functional.pad
    hi = pad(v.abs() + err, (0, G * block - K)).unflatten(-1, (G, block)).amax(-1)
    lo = pad((v.abs() - err).clamp(min=0.0), (0, G * block - K)).unflatten(-1, (G, block)).amax(-1)
    # the scale: amax / 448, floored, rounded once to float32 (U), or the power of two above it
    hi = (hi / 448.0).clamp(min=FLOOR) * (1 + 2 * U)
    lo = (lo / 448.0).clamp(min=FLOOR) * (1 - 2 * U)
    if fmt == "float":
        bad = (s > hi) | (s < lo)
    else:
        m, _ = torch.frexp(s)
        bad = (m != 0.5) | (s < lo) | (s / 2 >= hi)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} scales off"
    sx = expand(s, block, K)
    c, q = xq.float().to(F64), v / sx
    # the quotient is rounded to float32 (U) before the cast; beyond 448 the cast saturates
    slack = err / sx + 2 * U * q.abs()
    far = (c - q.clamp(-448.0, 448.0)).abs() > e4m3_half_step(q.abs() + slack) + slack
    far |= ~torch.isfinite(c)
    assert not bool(far.any()), f"{what}: {int(far.sum())} codes off, first at {torch.nonzero(far)[0].tolist()}"


def rmsnorm(x, weight, eps, residual):
    """(v, |error| of a float32 evaluation): z, its square, the mean's division, the square root and its
    reciprocal and the two products round once each (half of what precedes the root counts), and a sum of K
    squares in which no term passes through more than 16 ceil(K / 8192) + 32 additions."""
    z = x.to(F64) if residual is None else x.to(F64) + residual.to(F64)
    K = z.shape[1]
    v = z / torch.sqrt(z.square().mean(1, keepdim=True) + eps) * weight.to(F64)
    return z, v, v.abs() * U * (16 * -(-K // 8192) + 32 + 12)


def silu_mul(g, u):
    """(v, |error|) of g / (1 + e) * u with e = exp(-g) by an exponential that is off by at most 2^-22 (4 U): 4 U and
    1 U for e, which the quotient passes on at most whole, then the sum 1 + e, its reciprocal (an ulp, 2 U) and two
    products: 9 U (11 U for a form that also multiplies by e).  Where 1 / (1 + e) is below float32's normal range,
    g < -126 ln 2 = -87.336, it may be 0: silu is then below 87.4 2^-126 < 1.03e-36 in size, and all of it is lost."""
    g, u = g.to(F64), u.to(F64)
    v = g / (1.0 + torch.exp(-g)) * u
    return v, v.abs() * (U * 11) + (g < -87.336) * u.abs() * 1.03e-36


def quantize_values(v, fmt, block=128):
    """(values the codes stand for, scales [M, G], quotients): the definition in 64 bits, the scale and the quotient
    rounded to float32 as it says."""
    M, K = v.shape
    G = -(-K // block)
    amax = torch.nn.functional.pad(v.abs(), (0, G * block - K)).unflatten(-1, (G, block)).amax(-1)
    s = (amax / 448.0).clamp(min=FLOOR).float().to(F64)
    if fmt != "float":
        m, e = torch.frexp(s)
        s = torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e))
    sx = expand(s, block, K)
    q = (v / sx).float().to(F64).clamp(-448.0, 448.0)
    step = 2 * e4m3_half_step(q)
    return torch.round(q / step) * step * sx, s, q


def dequantize(wq, ws, block=128):
    n, k = wq.shape[-2:]
    s = ws.float().to(F64).repeat_interleave(block, -2)[..., :n, :]
    return wq.float().to(F64) * expand(s, block, k)


def moe_mlp(xhat, ids, weights, w13, s13, w2, s2, fmt):
    """(y, |error|) float64 [T, H] of the expert layer on dequantized activations xhat [T, H].

    The error a float32 evaluation may have: products summed over ceil(K / 128) blocks of four tensor-core steps,
    each sum off by U of what is added (Bg, Bu: the sums of absolute values); that moves silu(gate) * up, and an
    element of h whose quotient is that near a border between two codes may take the neighbouring code; the down
    products likewise, then the sum over the slots.  y's own rounding to bf16 is half a step, 2^-8 of y."""
    T, H = xhat.shape
    E, I = w13.shape[0], w2.shape[2]
    y = torch.zeros(T, H, dtype=F64, device=xhat.device)
    err = torch.zeros_like(y)
    e_up, e_down = (20 + -(-H // 128)) * U, (20 + -(-I // 128)) * U
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel() == 0:
            continue
        W, W2 = dequantize(w13[e], s13[e]), dequantize(w2[e], s2[e])
        h, B = xhat[t] @ W.t(), xhat[t].abs() @ W.abs().t()
        g, u, Bg, Bu = h[:, :I], h[:, I:], B[:, :I], B[:, I:]
        sg = 1.0 / (1.0 + torch.exp(-g))
        v = g * sg * u
        dv = (sg + g * sg * (1 - sg)).abs() * u.abs() * Bg * e_up + (g * sg).abs() * Bu * e_up + v.abs() * 10 * U
        hq, s, q = quantize_values(v, fmt)
        # how far a quotient may move: its own error and the scale's (the largest element's)
        sx = expand(s, 128, I)
        G = s.shape[1]
        rel = torch.nn.functional.pad(dv, (0, G * 128 - I)).unflatten(-1, (G, 128)).amax(-1)
        rel = expand(rel / (448.0 * s), 128, I) + 4 * U
        dq = dv / sx + q.abs() * rel
        half = e4m3_half_step(q)
        border = half - (q - hq / sx).abs()           # distance to the nearer border of the code's interval
        dh = torch.where(border <= dq, 2 * half * sx, torch.zeros_like(dq)) + hq.abs() * (rel if fmt == "float" else 0)
        if fmt != "float":                             # a scale next to a power of two may take the other one
            m, _ = torch.frexp(torch.nn.functional.pad(v.abs(), (0, G * 128 - I)).unflatten(-1, (G, 128)).amax(-1) /
                               448.0)
            near = expand(((m - 0.5).abs() < 1e-3) | ((m - 1.0).abs() < 1e-3), 128, I)
            dh = torch.where(near, 2 * half * sx + dh, dh)
        w = weights[t, j].to(F64)[:, None]
        o = hq @ W2.t()
        y.index_add_(0, t, w * o)
        err.index_add_(0, t, w.abs() * (dh @ W2.abs().t() + (hq.abs() @ W2.abs().t()) * e_down))
    return y, err + y.abs() * 2.0 ** -8 + 1e-30
