"""The operators around the linears on the GPU, against 64-bit plain forms
(_plain64.py): RMS norm and silu(gate) * up with quantized outputs, expert
routing, and the mixture-of-experts layer for few tokens."""
import numpy as np
import pytest
import torch

import _plain64 as P
import workloads as W
from _canary import Canary

pytestmark = pytest.mark.gpu

BF16, F32, F64, U8, I32 = torch.bfloat16, torch.float32, torch.float64, torch.uint8, torch.int32
FMTS = ["float", "ue8m0"]


@pytest.fixture(scope="module")
def fg8():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import fine_grained_fp8_act_b200 as m
    m.lib()
    return m


def _s():
    return torch.cuda.current_stream().cuda_stream


def _bits(t):
    return t.view(U8) if t.element_size() == 1 else t


def _same(a, b):
    return torch.equal(_bits(a.contiguous()), _bits(b.contiguous()))


# --------------------------------------------------------------- rms norm --
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K,block,residual", [
    (1, 16, 128, True), (3, 48, 32, False), (2, 512, 128, True), (5, 528, 64, True), (7, 1024, 128, False),
    (4, 1040, 32, True), (1, 7168, 128, True), (33, 2064, 128, True), (130, 4096, 64, False), (2, 4112, 128, True),
    (3, 8208, 128, True), (600, 7168, 128, False), (1300, 4112, 64, True), (9500, 480, 32, True),
    (300, 16400, 128, True), (2, 12288, 128, True), (2, 12304, 64, True), (2, 24576, 128, False), (2, 24592, 32, True),
    (1, 60000, 128, True), (1023, 256, 128, True)])
def test_rmsnorm_quant(fg8, fmt, M, K, block, residual):
    x = W.x_outliers(M, K, seed=M + K).cuda()
    r = W.normal((M, K), 3.0, seed=M + K + 1).cuda() if residual else None
    w = (1 + W.normal((K,), 0.3, seed=K).float()).to(BF16).cuda()
    xq, xs, ro, y = fg8.rmsnorm_quant(x, w, 1e-5, r, fmt, block=block, return_y=True)
    torch.cuda.synchronize()
    z, v, err = P.rmsnorm(x, w, float(np.float32(1e-5)), r)
    P.check_quantized(xq, xs, v, err, fmt, block, "rmsnorm")
    assert bool(((y.to(F64) - v).abs() <= v.abs() * 2.0 ** -8 + err).all())
    if residual:
        assert torch.equal(ro, (x.float() + r.float()).to(BF16))
    else:
        assert ro is None


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("K,tokens", [(272, 32), (624, 16), (1024, 16), (1040, 10), (2048, 8), (2304, 6), (4096, 4),
                                      (4112, 4), (5632, 4), (6160, 3), (8192, 3), (8208, 2), (9232, 2), (12288, 2),
                                      (12304, 1), (16384, 1), (16400, 1), (24576, 1)])
def test_rmsnorm_teams(fg8, K, tokens, residual):
    """Enough rows for the streaming form at every number of tokens that a CTA works on side by side (32 down to 1,
    up to one hardware barrier each): the last rows of the grid's last turn included."""
    M = 4 * 148 * tokens + 5
    x, w = W.normal((M, K), 2.0, seed=K).cuda(), W.normal((K,), 1.0, seed=K + 2).cuda()
    r = W.normal((M, K), 2.0, seed=K + 1).cuda() if residual else None
    xq, xs, ro, y = fg8.rmsnorm_quant(x, w, 1e-6, r, "float", return_y=True)
    z, v, err = P.rmsnorm(x, w, float(np.float32(1e-6)), r)
    P.check_quantized(xq, xs, v, err, "float", 128, "rmsnorm")
    assert bool(((y.to(F64) - v).abs() <= v.abs() * 2.0 ** -8 + err).all())
    if residual:
        assert torch.equal(ro, (x.float() + r.float()).to(BF16))


@pytest.mark.parametrize("fmt", FMTS)
def test_rmsnorm_quant_of_bf16_steps(fg8, fmt):
    """Where v is exact in bf16 (rows of +-2^a with weights 2^b, so that the mean square is a power of two and
    eps vanishes beside it), the fused codes and scales are quantize_act's of v, bit for bit."""
    M, K = 9, 1024
    g = torch.Generator().manual_seed(3)
    sign = torch.randint(0, 2, (M, K), generator=g) * 2.0 - 1.0
    x = (sign * torch.exp2(torch.arange(M, dtype=F32)[:, None] - 2)).to(BF16).cuda()
    w = torch.exp2(torch.randint(-6, 7, (K,), generator=g).float()).to(BF16).cuda()
    xq, xs, _, y = fg8.rmsnorm_quant(x, w, 1e-30, None, fmt, return_y=True)
    v = (sign.cuda() * w.float()).to(BF16)
    assert torch.equal(y, v)
    q, s = fg8.quantize_act(v, fmt)
    assert _same(xq, q) and _same(xs, s)


@pytest.mark.parametrize("K", [512, 7168, 30000 // 16 * 16])
def test_rmsnorm_strides_in_place_and_zero_rows(fg8, K):
    M = 6
    x = W.normal((M, K), 1.0, seed=1).cuda()
    x[2] = 0
    big = torch.zeros(M, K + 24, dtype=BF16, device="cuda")
    xv = big[:, 8:8 + K]
    xv.copy_(x)
    r = W.normal((M, K + 8), 1.0, seed=2).cuda()
    rv = r[:, :K]
    rv[2] = 0
    w = W.normal((K,), 1.0, seed=3).cuda()
    want = fg8.rmsnorm_quant(x, w, 1e-6, rv.contiguous(), "float", return_y=True)
    tail = r[:, K:].clone()
    got = fg8.rmsnorm_quant(xv, w, 1e-6, rv, "float", return_y=True, residual_out=rv)
    assert got[2].data_ptr() == rv.data_ptr()
    for a, b in zip(got, want):
        assert _same(a, b)
    assert torch.equal(r[:, K:], tail)
    assert bool((got[0][2].float() == 0).all())                   # codes of a zero row (-0 under a negative weight)
    assert bool((got[1][2] == P.FLOOR).all()) and bool((got[3][2] == 0).all())
    # x's own buffer as the new residual
    got = fg8.rmsnorm_quant(xv, w, 1e-6, want[2], "float", residual_out=xv)
    again = fg8.rmsnorm_quant(x, w, 1e-6, want[2], "float")
    assert _same(got[0], again[0]) and torch.equal(xv, again[2])


@pytest.mark.parametrize("fmt", FMTS)
def test_rmsnorm_extremes(fg8, fmt):
    """Rows at both ends of float32's range: sums of squares stay finite up to 2^63 or so, small rows sink into eps."""
    K = 256
    rows = [torch.full((K,), 2.0 ** 59), torch.full((K,), 2.0 ** -60), torch.full((K,), 2.0 ** -130),
            torch.cat([torch.full((1,), 2.0 ** 60), torch.full((K - 1,), 2.0 ** -60)])]
    x = torch.stack(rows).to(BF16).cuda()
    w = torch.ones(K, dtype=BF16, device="cuda")
    xq, xs, _, _ = fg8.rmsnorm_quant(x, w, 1e-6, None, fmt)
    _, v, err = P.rmsnorm(x, w, float(np.float32(1e-6)), None)
    P.check_quantized(xq, xs, v, err + 2.0 ** -149, fmt, 128)


# --------------------------------------------------------------- silu_mul --
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K,block", [(1, 16, 128), (3, 144, 32), (16, 14336, 128), (129, 2048, 64), (257, 1040, 128),
                                       (5, 272, 64), (2100, 4112, 128)])
def test_silu_mul_quant(fg8, fmt, M, K, block):
    both = W.normal((M, 2 * K), 3.0, seed=M + K).cuda()
    both[:, ::37] *= 30
    g, u = both[:, :K], both[:, K:]
    xq, xs, y = fg8.silu_mul_quant(g, u, fmt, block=block, return_y=True)
    v, err = P.silu_mul(g, u)
    P.check_quantized(xq, xs, v, err, fmt, block, "silu_mul")
    assert bool(((y.to(F64) - v).abs() <= v.abs() * 2.0 ** -8 + err).all())
    a = fg8.silu_mul_quant(g.contiguous(), u.contiguous(), fmt, block=block)
    assert _same(a[0], xq) and _same(a[1], xs) and a[2] is None


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K,N", [(1, 16, 8), (5, 400, 264), (33, 7168, 136), (130, 1040, 256), (600, 528, 512),
                                   (9500, 480, 64), (1300, 4112, 72), (300, 16400, 64)])
def test_prepare_forms(fg8, fmt, M, K, N):
    """fg8_linear_prepare_rmsnorm / _silu_mul leave the stand-alone forms' codes and scales in the GEMM's layouts, and
    the linears built on them give gemm_prequant's bits where both run the tiled GEMM, and the oracle's values
    otherwise.  The workspace starts as noise behind its header: padding must not reach y."""
    from _ws_layout import decode, offsets
    code = fg8.scale_fmt_code(fmt)
    x, r = W.x_outliers(M, K, seed=M + K).cuda(), W.normal((M, K), 1.0, seed=M).cuda()
    nw = (1 + W.normal((K,), 0.3, seed=K).float()).to(BF16).cuda()
    wq, ws = fg8.quantize_weight(W.normal((N, K), 0.05, seed=N).cuda(), fmt)
    b = W.normal((N,), 0.1, seed=N + 1).cuda()
    nb = fg8.fg8_linear_workspace_bytes(M, N, K, code)
    for which in ("rmsnorm", "silu"):
        wsp = torch.full((nb,), 0xA5, dtype=U8, device="cuda")
        wsp[:1024] = 0
        if which == "rmsnorm":
            q, s, ro, _ = fg8.rmsnorm_quant(x, nw, 1e-6, r, fmt)
            y, ro2 = fg8.rmsnorm_linear(x, nw, wq, ws, b, 1e-6, r, fmt, workspace=wsp)
            assert torch.equal(ro, ro2)
        else:
            q, s, _ = fg8.silu_mul_quant(x, r, fmt)
            y = fg8.silu_mul_linear(x, r, wq, ws, b, fmt, workspace=wsp)
        torch.cuda.synchronize()
        gq, gs = decode(wsp.cpu().numpy(), M, K, code)
        assert np.array_equal(gq, q.view(U8).cpu().numpy()), which
        want = s.cpu().numpy().view(np.uint32) if code == 0 else s.view(U8).cpu().numpy()
        assert np.array_equal(gs, want), which
        if code == 1:  # the tiles' other entries are 2^0
            xs_off, Kb = offsets(M, K)[1], (K + 127) // 128
            rows, slots = (M + 127) // 128 * 128, (Kb + 3) // 4 * 4
            t = wsp[xs_off:xs_off + rows * slots].cpu().numpy()
            full = decode(np.concatenate([np.zeros(offsets(rows, slots * 128)[1], np.uint8), t]), rows, slots * 128, 1)[1]
            assert (full[M:] == 127).all() and (full[:, Kb:] == 127).all()
        if fg8.fg8_linear_plan(M, N, K, code)[0] == 0:
            assert torch.equal(y, fg8.gemm_prequant(q, s, wq, ws, b, fmt)), which
        else:
            import oracle
            from conftest import y_tolerance
            ref, bound, _ = oracle.linear_dequant(gq, s.cpu().numpy() if code == 0 else gs, wq.view(U8).cpu().numpy(),
                                                  ws.cpu().numpy() if code == 0 else ws.view(U8).cpu().numpy(),
                                                  W.bf16_bits(b), code)
            out = y.float().cpu().numpy().astype(np.float64)
            assert np.all(np.abs(out - ref) <= y_tolerance(bound, ref, out)), which
        assert fg8.fg8_check_device_status(wsp.data_ptr(), _s()) == 0


def test_silu_mul_every_gate(fg8):
    """Every finite bf16 gate up to +-100, both signs of up."""
    b = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF16)
    b = b[torch.isfinite(b) & (b.abs() <= 100)]
    n = b.numel() // 128 * 128
    g = torch.cat([b[:n], b[-128:]]).reshape(-1, 128).cuda()
    u = (W.normal(tuple(g.shape), 1.0, seed=4).cuda())
    for fmt in FMTS:
        xq, xs, y = fg8.silu_mul_quant(g, u, fmt, return_y=True)
        v, err = P.silu_mul(g, u)
        P.check_quantized(xq, xs, v, err + 2.0 ** -149, fmt, 128)
        assert bool(((y.to(F64) - v).abs() <= v.abs() * 2.0 ** -8 + err + 2.0 ** -134).all())


@pytest.mark.parametrize("M", [3, 5000])
def test_silu_mul_extreme_gates(fg8, M):
    """Finite gates up to bf16's largest: silu is the gate itself above, zero below; nothing becomes NaN.  (M 5000:
    the streaming kernel.)"""
    K = 512
    big = torch.tensor([3.3895e38, -3.3895e38, 2.4e38, -2.4e38, 1e30, -1e30, 89.0, -89.0, 88.0, -88.0, 0.0, -0.0,
                        1e-38, -1e-38, 1e-40, -1e-40], dtype=BF16).repeat(K // 16)
    g = big.repeat(M, 1).cuda()
    u = torch.full((M, K), 2.0 ** -20, dtype=BF16, device="cuda")
    for fmt in FMTS:
        xq, xs, y = fg8.silu_mul_quant(g, u, fmt, return_y=True)
        v, err = P.silu_mul(g, u)
        P.check_quantized(xq, xs, v, err + 2.0 ** -149, fmt, 128)
        assert bool(((y.to(F64) - v).abs() <= v.abs() * 2.0 ** -8 + err + 2.0 ** -134).all())


# ------------------------------------------------------------------ route --
def _route64(l, k, renormalize, scale):
    l = l.float().to(F64).cpu().numpy()
    T, E = l.shape
    ok = ~np.isnan(l) & (l != -np.inf)
    ids = np.full((T, k), -1, np.int64)
    w = np.zeros((T, k))
    for t in range(T):
        order = sorted((e for e in range(E) if ok[t, e]), key=lambda e: (-l[t, e], e))[:k]
        if not order:
            continue
        top = l[t, order[0]]
        ex = [1.0 if l[t, e] == top else float(np.exp(l[t, e] - top)) for e in range(E)]
        tot = sum(ex[e] for e in (order if renormalize else range(E)) if ok[t, e])
        ids[t, :len(order)] = order
        w[t, :len(order)] = [scale * ex[e] / tot for e in order]
    return ids, w


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E,k,renormalize", [(1, 1, 1, True), (3, 8, 2, True), (5, 8, 8, False), (130, 60, 4, True),
                                               (7, 64, 6, False), (1, 256, 8, True), (33, 160, 12, True),
                                               (65, 384, 32, True), (4, 1024, 8, False), (9, 1000, 32, True),
                                               (6, 32, 5, True), (6, 33, 5, False), (6, 96, 6, True),
                                               (6, 97, 6, False), (6, 128, 7, True), (6, 129, 7, True),
                                               (6, 192, 8, False), (6, 193, 8, True), (6, 257, 8, True),
                                               (6, 385, 9, True), (6, 512, 9, False), (6, 513, 9, True),
                                               (6, 768, 10, True), (6, 769, 10, False)])
def test_moe_route(fg8, dtype, T, E, k, renormalize):
    g = torch.Generator().manual_seed(T + E)
    l = (torch.randn(T, E, generator=g) * 3).to(dtype)
    if T > 2:
        l[0] = 0.5                                    # every logit the same
        l[1, ::2] = -float("inf")                     # masked experts
        l[2] = -float("inf")
        l[2, E // 2] = -7.0                           # one left
    if T > 4:
        l[3] = -float("inf")                          # none left
        l[4, E // 3] = float("nan")
    if T > 6:
        l[5, ::2], l[5, 1::2] = 0.0, -0.0             # one value, two signs
        l[6, 1], l[6, 3] = float("inf"), float("inf")
    ids, w = fg8.moe_route(l.cuda(), k, renormalize, 2.5)
    want_ids, want_w = _route64(l, k, renormalize, 2.5)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    # expf 2 ulp on either side of the division, a sum of at most E terms in lanes and then 5 steps, two roundings;
    # the difference l - l_max rounds once, which its exponential turns into |l - l_max| U of the value
    spread = 40.0
    tol = (8 + (k if renormalize else E) / 32 + 6 + 3 + 2 * spread) * P.U
    assert np.all(np.abs(w.cpu().numpy() - want_w) <= tol * np.abs(want_w) + 1e-37)


def test_moe_route_strided(fg8):
    big = torch.randn(50, 80, device="cuda")
    l = big[:, 3:67]
    a, b = fg8.moe_route(l, 6), fg8.moe_route(l.contiguous(), 6)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---------------------------------------------------------------- moe_mlp --
def _experts(fg8, E, N, K, fmt, seed):
    qs = [fg8.quantize_weight(W.w_row_groups(N, K, 0.02, seed=seed + e).cuda(), fmt) for e in range(E)]
    return (torch.stack([_bits(q) for q, _ in qs]).view(qs[0][0].dtype),
            torch.stack([_bits(s) for _, s in qs]).view(qs[0][1].dtype))


class Layer:
    def __init__(self, fg8, T, k, E, H, I, fmt, seed=0):
        self.fmt, self.E = fmt, E
        self.x = W.x_outliers(T, H, seed=seed + 1).cuda()
        self.w13, self.s13 = _experts(fg8, E, 2 * I, H, fmt, seed + 100)
        self.w2, self.s2 = _experts(fg8, E, H, I, fmt, seed + 500)
        g = torch.Generator().manual_seed(seed)
        self.ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(I32).cuda()
        self.w = (torch.rand(T, k, generator=g) + 0.1).cuda()

    def run(self, fg8, **kw):
        return fg8.moe_mlp(kw.pop("x", self.x), self.ids, self.w, self.w13, self.s13, self.w2, self.s2, self.fmt, **kw)

    def check(self, y):
        torch.cuda.synchronize()
        xhat, _, _ = P.quantize_values(self.x.to(F64), self.fmt)
        ids = torch.where(self.ids < self.E, self.ids, -1)
        want, err = P.moe_mlp(xhat, ids, self.w, self.w13, self.s13, self.w2, self.s2, self.fmt)
        d = (y.to(F64) - want).abs()
        assert bool((d <= err).all()), f"{int((~(d <= err)).sum())} of {d.numel()} off, worst {float((d / err).max())}"


MOE = [  # T, k, E, H, I
    (1, 1, 1, 16, 16), (1, 2, 4, 256, 128), (1, 8, 16, 1024, 256), (2, 2, 3, 272, 144), (5, 3, 7, 400, 208),
    (16, 4, 8, 512, 384), (17, 2, 2, 640, 256), (33, 1, 1, 384, 128), (40, 6, 6, 144, 400), (64, 8, 32, 256, 128),
    (100, 2, 4, 528, 272), (128, 4, 4, 256, 256), (256, 2, 3, 128, 128), (128, 32, 40, 64, 48), (3, 2, 5, 2304, 1040)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,k,E,H,I", MOE)
def test_moe_mlp(fg8, fmt, T, k, E, H, I):
    a = Layer(fg8, T, k, E, H, I, fmt, seed=T + E)
    ws = torch.zeros(fg8.fg8_moe_mlp_workspace_bytes(T, k, E, H, I, fg8.scale_fmt_code(fmt)), dtype=U8, device="cuda")
    y = a.run(fg8, workspace=ws)
    a.check(y)
    assert torch.equal(a.run(fg8, workspace=ws), y)              # the workspace's counters are back at rest
    xq, xs = fg8.quantize_act(a.x, fmt)                          # the same from codes
    assert torch.equal(a.run(fg8, x=xq, x_scale=xs), y)
    assert fg8.fg8_check_device_status(ws.data_ptr(), _s()) == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_moe_mlp_slots(fg8, fmt):
    """Skipped slots, tokens with none, the same expert in several slots, weights of zero, below zero and large."""
    T, k, E, H, I = 24, 4, 6, 400, 272
    a = Layer(fg8, T, k, E, H, I, fmt, seed=9)
    a.ids[0] = -1
    a.ids[1] = torch.tensor([-5, 2, -1, -2 ** 31], device="cuda")
    a.ids[2] = 3
    a.ids[3] = torch.tensor([0, 0, 5, 0], device="cuda")
    a.ids[20:] = 4
    a.w[4], a.w[5], a.w[6] = 0.0, -1.0, 1e4
    a.w[0] = float("nan")                                        # weights of skipped slots are not read into y
    y = a.run(fg8)
    assert bool((y[0] == 0).all())
    a.w[0] = 0.0
    a.check(y)
    a.ids[:] = -1
    assert bool((a.run(fg8) == 0).all())


def test_moe_mlp_expert_out_of_range(fg8):
    T, k, E, H, I = 5, 2, 4, 256, 128
    a = Layer(fg8, T, k, E, H, I, "float", seed=3)
    ws = torch.zeros(fg8.fg8_moe_mlp_workspace_bytes(T, k, E, H, I, 0), dtype=U8, device="cuda")
    a.ids[1, 1], a.ids[3, 0] = E, 2 ** 31 - 1
    y = a.run(fg8, workspace=ws)
    a.check(y)
    assert fg8.fg8_check_device_status(ws.data_ptr(), _s()) == fg8.FG8_ERR_INVALID_ARG
    a.ids.clamp_(max=E - 1)
    a.check(a.run(fg8, workspace=ws))
    assert fg8.fg8_check_device_status(ws.data_ptr(), _s()) == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_moe_mlp_matches_grouped_layers(fg8, fmt):
    """One token per expert through the padded grouped layers: the same weights and codes, with the products of
    gate and up rounded to bf16 in between (2^-8 each, of values whose quantization is 2^-4)."""
    T, k, E, H, I = 4, 2, 4, 512, 256
    a = Layer(fg8, T, k, E, H, I, fmt, seed=21)
    y = a.run(fg8).float()
    rows, where = [], []
    row_expert = torch.full((128 * E,), -1, dtype=I32)
    xr = torch.zeros(128 * E, H, dtype=BF16, device="cuda")
    ids = a.ids.cpu()
    at = [0] * E
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            r = 128 * e + at[e]
            at[e] += 1
            xr[r] = a.x[t]
            row_expert[r] = e
            where.append((t, j, r))
    for e in range(E):
        row_expert[128 * e] = e if at[e] else -1
    gu = fg8.grouped_linear(xr, row_expert.cuda(), a.w13, a.s13, None, fmt)
    live = torch.tensor([r for _, _, r in where], device="cuda")
    h = torch.zeros(128 * E, I, dtype=BF16, device="cuda")
    h[live] = fg8.silu_mul_quant(gu[live][:, :I], gu[live][:, I:], fmt, return_y=True)[2]
    o = fg8.grouped_linear(h, row_expert.cuda(), a.w2, a.s2, None, fmt)
    want = torch.zeros(T, H, device="cuda")
    for t, j, r in where:
        want[t] += a.w[t, j] * o[r].float()
    assert float((y - want).norm() / want.norm()) < 0.05


# ------------------------------------------------- streams, graphs, bounds --
def test_outputs_stay_in_bounds(fg8):
    M, K, I = 37, 400, 272
    x, r, w = (W.normal((M, K), 1.0, seed=s).cuda() for s in (1, 2, 3))
    cq, cs, cr, cy = (Canary(n, "cuda") for n in (M * K, M * 4 * 4, M * (K + 8) * 2, M * (K + 16) * 2))
    q, s = cq.matrix(U8, M, K, K), cs.matrix(F32, M, 4, 4)
    ro, y = cr.matrix(BF16, M, K, K + 8), cy.matrix(BF16, M, K, K + 16)
    fg8.fg8_rmsnorm_quant(x.data_ptr(), M, K, K, r.data_ptr(), K, w.data_ptr(), 1e-6, cq.ptr(), cs.ptr(), 0, 128,
                          cr.ptr(), K + 8, cy.ptr(), K + 16, _s())
    a = fg8.rmsnorm_quant(x, w[0].contiguous(), 1e-6, r, "float", return_y=True)
    assert torch.equal(q, _bits(a[0])) and torch.equal(s, a[1]) and torch.equal(ro, a[2]) and torch.equal(y, a[3])
    assert cq.intact() and cs.intact() and cr.intact() and cy.intact()
    cq, cs, cy = (Canary(n, "cuda") for n in (M * K, M * 13, M * (K + 8) * 2))
    q, s, y = cq.matrix(U8, M, K, K), cs.matrix(U8, M, 13, 13), cy.matrix(BF16, M, K, K + 8)
    fg8.fg8_silu_mul_quant(x.data_ptr(), r.data_ptr(), M, K, K, K, cq.ptr(), cs.ptr(), 1, 32, cy.ptr(), K + 8, _s())
    a = fg8.silu_mul_quant(x, r, "ue8m0", block=32, return_y=True)
    assert torch.equal(q, _bits(a[0])) and torch.equal(s, _bits(a[1])) and torch.equal(y, a[2])
    assert cq.intact() and cs.intact() and cy.intact()
    ci, cw = Canary(M * 3 * 4, "cuda"), Canary(M * 3 * 4, "cuda")
    i, wt = ci.matrix(I32, M, 3, 3), cw.matrix(F32, M, 3, 3)
    l = torch.randn(M, 50, device="cuda")
    fg8.fg8_moe_route(l.data_ptr(), 0, M, 50, 50, 3, 1, 1.0, ci.ptr(), cw.ptr(), _s())
    a = fg8.moe_route(l, 3)
    assert torch.equal(i, a[0]) and torch.equal(wt, a[1]) and ci.intact() and cw.intact()
    for fmt in (0, 1):
        b = Layer(fg8, M, 3, 5, K, I, FMTS[fmt], seed=4)
        need = fg8.fg8_moe_mlp_workspace_bytes(M, 3, 5, K, I, fmt)
        cy, cw = Canary(M * (K + 8) * 2, "cuda"), Canary(need, "cuda")
        y = cy.matrix(BF16, M, K, K + 8)
        cw.zeroed()
        for _ in range(2):
            fg8.fg8_moe_mlp(b.x.data_ptr(), 0, M, K, K, b.ids.data_ptr(), b.w.data_ptr(), 3, 5, I, b.w13.data_ptr(),
                            b.s13.data_ptr(), b.w2.data_ptr(), b.s2.data_ptr(), cy.ptr(), K + 8, fmt, cw.ptr(), need,
                            _s())
        assert torch.equal(y, b.run(fg8)) and cy.intact() and cw.intact()
        assert fg8.fg8_check_device_status(cw.ptr(), _s()) == 0


def _block(fg8, b, norm_w, gate_w, h, res, ws, k):
    """The expert half of a transformer block: norm, router, experts; returns every output."""
    xq, xs, res, y = fg8.rmsnorm_quant(h, norm_w, 1e-6, res, b.fmt, return_y=True)
    ids, w = fg8.moe_route(torch.matmul(y, gate_w).float(), k)
    return fg8.moe_mlp(xq, ids, w, b.w13, b.s13, b.w2, b.s2, b.fmt, x_scale=xs, workspace=ws), res, ids, w, xq, xs


@pytest.mark.parametrize("fmt", FMTS)
def test_expert_block_runs_together_and_in_graphs(fg8, fmt):
    T, k, E, H, I = 19, 3, 8, 512, 256
    b = Layer(fg8, T, k, E, H, I, fmt, seed=31)
    norm_w = (1 + W.normal((H,), 0.2, seed=5).float()).to(BF16).cuda()
    gate_w = W.normal((H, E), 0.05, seed=6).cuda()
    h, res = W.normal((T, H), 1.0, seed=7).cuda(), W.normal((T, H), 1.0, seed=8).cuda()
    ws = torch.zeros(fg8.fg8_moe_mlp_workspace_bytes(T, k, E, H, I, fg8.scale_fmt_code(fmt)), dtype=U8, device="cuda")
    y, new_res, ids, w, xq, xs = _block(fg8, b, norm_w, gate_w, h, res, ws, k)
    # the layer's own reference on the codes and the routing that it was given
    xhat = xq.float().to(F64) * P.expand(P.scale_values(xs), 128, H)
    want, err = P.moe_mlp(xhat, ids, w, b.w13, b.s13, b.w2, b.s2, fmt)
    assert bool(((y.to(F64) - want).abs() <= err).all())
    # two captured graphs that share the workspace, replayed in turn on a stream of their own
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        _block(fg8, b, norm_w, gate_w, h, res, ws, k)
    side.synchronize()
    for _ in range(2):
        hh = h.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = _block(fg8, b, norm_w, gate_w, hh, res, ws, k)
        graphs.append((g, hh, out))
    for trial in range(3):
        for n, (g, hh, out) in enumerate(graphs):
            hh.copy_(W.normal((T, H), 1.0 + n, seed=50 + trial).cuda())
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                g.replay()
            side.synchronize()
            eager = _block(fg8, b, norm_w, gate_w, hh, res, ws, k)
            for got, ref in zip(out, eager):
                assert _same(got, ref)
    assert fg8.fg8_check_device_status(ws.data_ptr(), _s()) == 0
    del graphs


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [3, 200])
def test_dense_block_runs_together(fg8, orc, fmt, T):
    """norm -> gate/up -> silu_mul -> down, each step's input the codes of the one before."""
    H, I = 512, 784
    code = fg8.scale_fmt_code(fmt)
    w13, s13 = fg8.quantize_weight(W.normal((2 * I, H), 0.04, seed=1).cuda(), fmt)
    w2, s2 = fg8.quantize_weight(W.normal((H, I), 0.04, seed=2).cuda(), fmt)
    norm_w = (1 + W.normal((H,), 0.2, seed=3).float()).to(BF16).cuda()
    h = W.x_outliers(T, H, seed=4).cuda()
    xq, xs, _, _ = fg8.rmsnorm_quant(h, norm_w, 1e-6, None, fmt)
    gu = fg8.gemm_prequant(xq, xs, w13, s13, None, fmt)
    aq, as_, _ = fg8.silu_mul_quant(gu[:, :I], gu[:, I:], fmt)
    y = fg8.gemm_prequant(aq, as_, w2, s2, None, fmt)
    torch.cuda.synchronize()

    def np8(t):
        return t.view(U8).cpu().numpy()

    def nps(t):
        return t.cpu().numpy() if code == 0 else np8(t)
    from conftest import y_tolerance
    for got, (q, s, wq, ws) in ((gu, (xq, xs, w13, s13)), (y, (aq, as_, w2, s2))):
        ref, bound, _ = orc.linear_dequant(np8(q), nps(s), np8(wq), nps(ws), None, code)
        out = got.float().cpu().numpy().astype(np.float64)
        assert np.all(np.abs(out - ref) <= y_tolerance(bound, ref, out))


def test_other_stream_and_concurrent_workspaces(fg8):
    """Calls on two streams at once, each with a workspace of its own, give what one call alone gives."""
    T, k, E, H, I = 12, 2, 6, 1024, 512
    b = Layer(fg8, T, k, E, H, I, "ue8m0", seed=41)
    want = b.run(fg8)
    torch.cuda.synchronize()
    n = fg8.fg8_moe_mlp_workspace_bytes(T, k, E, H, I, 1)
    streams = [torch.cuda.Stream() for _ in range(2)]
    wss = [torch.zeros(n, dtype=U8, device="cuda") for _ in streams]
    outs = [torch.empty(T, H, dtype=BF16, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, ws, o in zip(streams, wss, outs):
            with torch.cuda.stream(s):
                b.run(fg8, out=o, workspace=ws)
    torch.cuda.synchronize()
    for ws, o in zip(wss, outs):
        assert torch.equal(o, want)
        assert fg8.fg8_check_device_status(ws.data_ptr(), _s()) == 0


def test_empty_batches(fg8):
    z = torch.zeros(0, 256, dtype=BF16, device="cuda")
    w = torch.ones(256, dtype=BF16, device="cuda")
    xq, xs, r, y = fg8.rmsnorm_quant(z, w, 1e-6, z, "float", return_y=True)
    assert xq.shape == (0, 256) and xs.shape == (0, 2) and r.shape == (0, 256) and y.shape == (0, 256)
    assert fg8.silu_mul_quant(z, z, "ue8m0", block=32)[1].shape == (0, 8)
    ids, wt = fg8.moe_route(torch.zeros(0, 8, device="cuda"), 2)
    assert ids.shape == (0, 2)
    b = Layer(fg8, 1, 2, 4, 256, 128, "float", seed=1)
    assert fg8.moe_mlp(z, ids, wt, b.w13, b.s13, b.w2, b.s2, "float").shape == (0, 256)


# ------------------------------------------------ what a caller may also do --
@pytest.mark.parametrize("fmt", FMTS)
def test_moe_mlp_most_pairs_and_experts(fg8, fmt):
    """The limits on tokens x slots and on experts at once: 4096 pairs over 1024 experts, and over one."""
    a = Layer(fg8, 256, 16, 1024, 64, 32, fmt, seed=1)
    y = a.run(fg8)
    a.check(y)
    a.ids[:] = 1023
    a.check(a.run(fg8))


def test_moe_mlp_one_workspace_for_many_shapes(fg8):
    """Layers of several shapes, and a dense linear, on one workspace in turn: its header is at rest between them."""
    shapes = [(1, 2, 4, 256, 128, "float"), (60, 4, 8, 1040, 272, "ue8m0"), (7, 1, 3, 4096, 48, "float")]
    layers = [Layer(fg8, *s, seed=11 + i) for i, s in enumerate(shapes)]
    x = W.x_normal(16, 4096, seed=3).cuda()
    wq, ws = fg8.quantize_weight(W.normal((1024, 4096), 0.02, seed=4).cuda(), "float")
    n = max(fg8.fg8_moe_mlp_workspace_bytes(*s[:5], fg8.scale_fmt_code(s[5])) for s in shapes)
    wsp = torch.zeros(max(n, fg8.fg8_linear_workspace_bytes(16, 1024, 4096, 0)), dtype=U8, device="cuda")
    want = [a.run(fg8) for a in layers] + [fg8.linear(x, wq, ws)]
    for _ in range(3):
        for a, w in zip(layers, want):
            assert torch.equal(a.run(fg8, workspace=wsp), w)
            assert torch.equal(fg8.linear(x, wq, ws, workspace=wsp), want[-1])
    assert fg8.fg8_check_device_status(wsp.data_ptr(), _s()) == 0


@pytest.mark.parametrize("codes", [False, True])
def test_moe_mlp_tokens_do_not_mix(fg8, codes):
    """NaN in one token's input stays in that token's output; a token without a slot does not read its own."""
    T, k, E, H, I = 20, 2, 3, 400, 272
    a = Layer(fg8, T, k, E, H, I, "float", seed=8)
    a.ids[11] = -1
    y = a.run(fg8)
    x = a.x.clone()
    x[5], x[11] = float("nan"), float("inf")
    kw = dict(x=x)
    if codes:
        xq, xs = fg8.quantize_act(a.x, "float")
        xq = xq.clone()
        xq.view(U8)[5], xq.view(U8)[11] = 0x7F, 0x7F
        kw = dict(x=xq, x_scale=xs)
    z = a.run(fg8, **kw)
    keep = [t for t in range(T) if t != 5]
    assert torch.equal(z[keep], y[keep]) and bool((z[11] == 0).all()) and bool(torch.isnan(z[5]).all())


def test_moe_mlp_strided_rows(fg8):
    T, k, E, H, I = 9, 2, 4, 272, 144
    a = Layer(fg8, T, k, E, H, I, "ue8m0", seed=6)
    want = a.run(fg8)
    big = torch.zeros(T, H + 40, dtype=BF16, device="cuda")
    xv = big[:, 24:24 + H]
    xv.copy_(a.x)
    out = torch.full((T, H + 8), 7.0, dtype=BF16, device="cuda")
    y = a.run(fg8, x=xv, out=out[:, :H])
    assert torch.equal(y, want) and bool((out[:, H:] == 7).all())


def test_norm_rows_do_not_mix(fg8):
    for M, K in ((6, 1040), (5000, 512), (1300, 4096)):
        x, r = W.normal((M, K), 1.0, seed=1).cuda(), W.normal((M, K), 1.0, seed=2).cuda()
        w = torch.ones(K, dtype=BF16, device="cuda")
        want = fg8.rmsnorm_quant(x, w, 1e-6, r, "float")
        x[M // 2, 3] = float("nan")
        got = fg8.rmsnorm_quant(x, w, 1e-6, r, "float")
        keep = torch.arange(M, device="cuda") != M // 2
        for g, e in zip(got[:3], want[:3]):
            assert _same(_bits(g)[keep], _bits(e)[keep])


def test_norm_and_silu_past_32_bit_offsets(fg8):
    """2.2e9 elements: the last rows' outputs lie past 2^31 elements and 2^32 bytes."""
    M, K = 270000, 8192
    x = torch.empty(M, K, dtype=BF16, device="cuda")
    x[:-8] = 1.0
    x[-8:] = W.x_outliers(8, K, seed=5).cuda()
    w = (1 + W.normal((K,), 0.3, seed=6).float()).to(BF16).cuda()
    xq, xs, _, _ = fg8.rmsnorm_quant(x, w, 1e-6, None, "float")
    _, v, err = P.rmsnorm(x[-8:], w, float(np.float32(1e-6)), None)
    P.check_quantized(xq[-8:], xs[-8:], v, err, "float", 128)
    del xq, xs
    xq, xs, _ = fg8.silu_mul_quant(x, x, "ue8m0", block=64)
    v, err = P.silu_mul(x[-8:], x[-8:])
    P.check_quantized(xq[-8:], xs[-8:], v, err, "ue8m0", 64)


def test_moe_mlp_weights_past_32_bit_offsets(fg8):
    """160 experts, 4.7e9 bytes of gate and up weights: the last ones' results are those of a layer of just them."""
    E, H, I = 160, 7168, 2048
    a = Layer(fg8, 3, 2, 3, H, I, "float", seed=9)
    at = torch.tensor([0, E - 2, E - 1], device="cuda")
    b = Layer.__new__(Layer)
    b.fmt, b.E, b.x, b.w, b.ids = a.fmt, E, a.x, a.w, at[a.ids.long()].to(I32)
    for name in ("w13", "s13", "w2", "s2"):
        few = getattr(a, name)
        many = torch.zeros((E, *few.shape[1:]), dtype=U8 if few.element_size() == 1 else few.dtype, device="cuda")
        many[at] = _bits(few)
        setattr(b, name, many.view(few.dtype))
    y = a.run(fg8)
    a.check(y)
    assert torch.equal(b.run(fg8), y)


def test_unaligned_views_are_refused(fg8):
    x = W.normal((8, 528), 1.0, seed=1).cuda()
    w = torch.ones(512, dtype=BF16, device="cuda")
    for call in (lambda: fg8.rmsnorm_quant(x[:, 4:516], w), lambda: fg8.silu_mul_quant(x[:, 4:516], x[:, :512]),
                 lambda: fg8.rmsnorm_quant(x[:, :520], torch.ones(520, dtype=BF16, device="cuda"))):
        with pytest.raises(fg8.FG8Error) as e:
            call()
        assert e.value.status == fg8.FG8_ERR_ALIGNMENT
