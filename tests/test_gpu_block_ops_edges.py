"""The operators around the linears where their formulas meet the edges of
float32 and of torch's strides: overflow of finite inputs, one-row views,
the streaming form of silu(gate) * up.  64-bit plain forms as in
test_gpu_block_ops.py."""
import numpy as np
import pytest
import torch

import _plain64 as P
import workloads as W
from test_gpu_block_ops import FMTS, Layer, _bits, _s, _same

pytestmark = pytest.mark.gpu

BF16, F32, F64, U8, I32 = torch.bfloat16, torch.float32, torch.float64, torch.uint8, torch.int32


@pytest.fixture(scope="module")
def fg8():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import fine_grained_fp8_act_b200 as m
    m.lib()
    return m


# ---------------------------------------- finite inputs, an infinite value --
def _check_overflowed(fg8, fmt, got, clean, y, m, block):
    """Row m's group 0 holds a value past float32: its scale is the one that quantize_act gives such a group (inf, or
    the UE8M0 NaN), the value does not come back finite, and no other group is touched."""
    xq, xs = got[0], got[1]
    assert bool(torch.isinf(y[m, 5]))
    q, s = fg8.quantize_act(y, fmt, block)
    assert _same(xs[m:m + 1, :1], s[m:m + 1, :1])
    assert not bool(torch.isfinite(xq[m, 5].float() * xs[m, 0].float()))
    keep = torch.ones_like(_bits(xs), dtype=torch.bool)
    keep[m, 0] = False
    assert torch.equal(_bits(xs)[keep], _bits(clean[1])[keep])
    cols = P.expand(keep, block, xq.shape[1])
    assert torch.equal(_bits(xq)[cols], _bits(clean[0])[cols])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,block", [(3, 128), (3, 32), (29000, 128), (29000, 64)])
def test_silu_mul_product_past_float32(fg8, fmt, M, block):
    """silu(8) * 3e38 is 2.4e39.  (M 29000: the streaming kernel.)"""
    K = 512
    g, u = W.normal((M, K), 2.0, seed=1).cuda(), W.normal((M, K), 2.0, seed=2).cuda()
    clean = fg8.silu_mul_quant(g, u, fmt, block=block)
    m = M - 2
    g[m, 5], u[m, 5] = 8.0, 3e38
    got = fg8.silu_mul_quant(g, u, fmt, block=block, return_y=True)
    _check_overflowed(fg8, fmt, got, clean, got[2], m, block)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K,block", [(3, 512, 128), (10000, 512, 64), (1200, 4112, 128)])
def test_rmsnorm_value_past_float32(fg8, fmt, M, K, block):
    """A row whose one large element is sqrt(K) times its rms, under a weight of 3e38."""
    x, w = W.normal((M, K), 1.0, seed=3).cuda(), W.normal((K,), 1.0, seed=4).cuda()
    m = M - 2
    x[m] = 0
    x[m, 5], w[5] = 1000.0, 3e38
    x[:m, 5] = 0
    x[m + 1:, 5] = 0
    clean = fg8.rmsnorm_quant(x * (torch.arange(M, device="cuda") != m)[:, None], w, 1e-6, None, fmt, block=block)
    got = fg8.rmsnorm_quant(x, w, 1e-6, None, fmt, block=block, return_y=True)
    _check_overflowed(fg8, fmt, got, clean, got[3], m, block)


# ----------------------------------- rows whose squares are past float32 ----
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,K", [(6, 256), (6, 16400), (6, 30000), (10000, 256), (1300, 4112), (2500, 4096),
                                 (700, 16400)])
def test_rmsnorm_squares_past_float32(fg8, fmt, residual, M, K):
    """Finite rows whose sum of squares overflows float32 are normalized like all others: the mean square is then
    taken of z 2^-80.  1 / rms may be subnormal there, 4 U off instead of its rounding's 1 U."""
    x = W.normal((M, K), 1.0, seed=M + K).float().cuda()
    top = 3.3e38 if not residual else 1.6e38
    m = torch.arange(M, device="cuda")
    x[m % 5 == 1] *= 2.0 ** 64                                     # squares alone reach 2^128
    x[m % 5 == 2] = x[m % 5 == 2].sign() * top                     # nothing larger exists
    x[m % 5 == 3] = 0
    x[m % 5 == 3, 7] = 2.0 ** 100                                  # one element
    x[m % 5 == 4] *= 2.0 ** 61                                     # the sum, not its terms
    x = x.to(BF16)
    r = x.clone() if residual else None
    w = (1 + W.normal((K,), 0.3, seed=K).float()).to(BF16).cuda()
    xq, xs, ro, y = fg8.rmsnorm_quant(x, w, 1e-6, r, fmt, return_y=True)
    z, v, err = P.rmsnorm(x, w, float(np.float32(1e-6)), r)
    err = err + v.abs() * 4 * P.U
    P.check_quantized(xq, xs, v, err, fmt, 128, "rmsnorm")
    assert bool(((y.to(F64) - v).abs() <= v.abs() * 2.0 ** -8 + err).all())
    if residual:
        assert torch.equal(ro, (x.float() + r.float()).to(BF16))


def test_rmsnorm_large_eps(fg8):
    """mean square + eps past float32 although both are finite."""
    x = torch.full((4, 256), 1.5e19, dtype=BF16, device="cuda")
    w = torch.ones(256, dtype=BF16, device="cuda")
    eps = 2.5e38
    xq, xs, _, _ = fg8.rmsnorm_quant(x, w, eps, None, "float")
    _, v, err = P.rmsnorm(x, w, float(np.float32(eps)), None)
    P.check_quantized(xq, xs, v, err + v.abs() * 4 * P.U, "float", 128)


# ----------------------------------------------------------- one-row views --
def _one_rows(K):
    """One row at strides that are not its length: hidden[:, -1] of a batch of one, a buffer whose width is no
    multiple of 8, a column's transpose."""
    a = torch.zeros(3, 2 * K, dtype=BF16, device="cuda")[1:2, :K]
    b = torch.zeros(1, K + 4, dtype=BF16, device="cuda")[:, :K]
    c = torch.zeros(K, 1, dtype=BF16, device="cuda").t()
    return [a, b, c]


@pytest.mark.parametrize("which", range(3))
@pytest.mark.parametrize("fmt", FMTS)
def test_one_row_views(fg8, fmt, which):
    """norm -> experts -> norm on one decoded token out of a larger tensor, as for the token alone."""
    H, I, E, k = 512, 256, 4, 2
    b = Layer(fg8, 1, k, E, H, I, fmt, seed=3)
    x = _one_rows(H)[which]
    x.copy_(b.x)
    r = _one_rows(H)[which]
    r.copy_(W.normal((1, H), 1.0, seed=9))
    w = (1 + W.normal((H,), 0.3, seed=H).float()).to(BF16).cuda()

    def chain(x, r):
        q, s, ro, y = fg8.rmsnorm_quant(x, w, 1e-6, r, fmt, return_y=True)
        o = b.run(fg8, x=q, x_scale=s)
        o2 = b.run(fg8, x=x)
        q2, s2, ro2, _ = fg8.rmsnorm_quant(o, w, 1e-6, ro, fmt)
        a, c, v = fg8.silu_mul_quant(x, r, fmt, return_y=True)
        return q, s, ro, y, o, o2, q2, s2, ro2, a, c, v
    got, want = chain(x, r), chain(x.clone(memory_format=torch.contiguous_format).reshape(-1).reshape(1, H),
                                   r.reshape(-1).clone().reshape(1, H))
    for g, e in zip(got, want):
        assert g.stride() == (g.shape[1], 1) and _same(g, e)


@pytest.mark.parametrize("which", range(3))
def test_one_row_outputs_and_linears(fg8, which):
    H, I, E, k = 512, 256, 4, 2
    b = Layer(fg8, 1, k, E, H, I, "float", seed=3)
    x, out, ro = (_one_rows(H)[which] for _ in range(3))
    x.copy_(b.x)
    w = torch.ones(H, dtype=BF16, device="cuda")
    assert torch.equal(b.run(fg8, out=out), b.run(fg8)) and torch.equal(out, b.run(fg8))
    wq, ws = fg8.quantize_weight(W.normal((H, H), 0.05, seed=2).cuda(), "float")
    y, _ = fg8.rmsnorm_linear(x, w, wq, ws, None, 1e-6, x, residual_out=ro, out=out)
    want, want_r = fg8.rmsnorm_linear(b.x, w, wq, ws, None, 1e-6, b.x)
    assert torch.equal(y, want) and torch.equal(ro, want_r)
    fg8.silu_mul_linear(x, x, wq, ws, out=out)
    assert torch.equal(out, fg8.silu_mul_linear(b.x, b.x, wq, ws))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_route_of_one_row_view(fg8, dtype):
    l = torch.randn(64, 1, device="cuda").to(dtype).t()
    a, b = fg8.moe_route(l, 6), fg8.moe_route(l.reshape(-1).clone().reshape(1, 64), 6)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# -------------------------------------- silu(gate) * up, its streaming form --
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K,block", [(30001, 480, 128), (3300, 4112, 64), (1700, 8208, 32), (28500, 16, 128)])
def test_silu_mul_stream(fg8, fmt, M, K, block):
    """Sizes past the few-token kernel's (six items of 512 channels a warp of the whole GPU)."""
    both = W.normal((M, 2 * K), 3.0, seed=M + K).cuda()
    both[:, ::37] *= 30
    g, u = both[:, :K], both[:, K:]
    xq, xs, y = fg8.silu_mul_quant(g, u, fmt, block=block, return_y=True)
    v, err = P.silu_mul(g, u)
    P.check_quantized(xq, xs, v, err, fmt, block, "silu_mul")
    # gates of -90 and below leave v under 2^-126, where bf16's steps are all 2^-133: half of one beside the 2^-8
    assert bool(((y.to(F64) - v).abs() <= v.abs() * 2.0 ** -8 + err + 2.0 ** -134).all())
    # a row's results do not depend on how many rows there are: the few-token kernel's bits
    few = fg8.silu_mul_quant(g[-9:], u[-9:], fmt, block=block, return_y=True)
    for a, b in zip((xq, xs, y), few):
        assert _same(a[-9:], b)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K,N", [(30001, 480, 64), (3300, 4112, 72), (10007, 1040, 64)])
def test_prepare_forms_streamed(fg8, fmt, M, K, N):
    """The streaming kernels with their scales in the GEMM's layouts, against gemm_prequant on the row-major ones."""
    code = fg8.scale_fmt_code(fmt)
    x, r = W.x_outliers(M, K, seed=M + K).cuda(), W.normal((M, K), 1.0, seed=M).cuda()
    nw = (1 + W.normal((K,), 0.3, seed=K).float()).to(BF16).cuda()
    wq, ws = fg8.quantize_weight(W.normal((N, K), 0.05, seed=N).cuda(), fmt)
    wsp = torch.full((fg8.fg8_linear_workspace_bytes(M, N, K, code),), 0xA5, dtype=U8, device="cuda")
    wsp[:1024] = 0
    q, s, ro, _ = fg8.rmsnorm_quant(x, nw, 1e-6, r, fmt)
    y, ro2 = fg8.rmsnorm_linear(x, nw, wq, ws, None, 1e-6, r, fmt, workspace=wsp)
    assert torch.equal(ro, ro2) and torch.equal(y, fg8.gemm_prequant(q, s, wq, ws, None, fmt))
    q, s, ro, _ = fg8.rmsnorm_quant(x, nw, 1e-6, None, fmt)
    y, _ = fg8.rmsnorm_linear(x, nw, wq, ws, None, 1e-6, None, fmt, workspace=wsp)
    assert torch.equal(y, fg8.gemm_prequant(q, s, wq, ws, None, fmt))
    q, s, _ = fg8.silu_mul_quant(x, r, fmt)
    y = fg8.silu_mul_linear(x, r, wq, ws, None, fmt, workspace=wsp)
    assert torch.equal(y, fg8.gemm_prequant(q, s, wq, ws, None, fmt))
    assert fg8.fg8_check_device_status(wsp.data_ptr(), _s()) == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_silu_mul_extreme_gates_streamed(fg8, fmt):
    """Finite gates up to bf16's largest in the streaming kernel: zeros below, the gate itself above, no NaN."""
    M, K = 29000, 512
    big = torch.tensor([3.3895e38, -3.3895e38, 2.4e38, -2.4e38, 1e30, -1e30, 89.0, -89.0, 88.0, -88.0, 0.0, -0.0,
                        1e-38, -1e-38, 1e-40, -1e-40], dtype=BF16).repeat(K // 16)
    g = big.repeat(M, 1).cuda()
    u = torch.full((M, K), 2.0 ** -20, dtype=BF16, device="cuda")
    xq, xs, y = fg8.silu_mul_quant(g, u, fmt, return_y=True)
    v, err = P.silu_mul(g, u)
    P.check_quantized(xq, xs, v, err + 2.0 ** -149, fmt, 128)
    assert bool(((y.to(F64) - v).abs() <= v.abs() * 2.0 ** -8 + err + 2.0 ** -134).all())


# --------------------------------------------- workspaces made for the call --
def _leave_noise(n):
    """n bytes of 0xA5 left behind in the caching allocator, for the next allocation of this size."""
    for _ in range(2):
        t = torch.full((n,), 0xA5, dtype=U8, device="cuda")
        torch.cuda.synchronize()
        del t


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,k,E,H,I", [(1, 2, 4, 256, 128), (40, 4, 8, 2064, 1424), (100, 2, 4, 528, 272)])
def test_moe_mlp_on_used_memory(fg8, fmt, T, k, E, H, I):
    """Without a workspace argument the layer runs on memory that held something else."""
    a = Layer(fg8, T, k, E, H, I, fmt, seed=T)
    a.ids[T // 2] = -1
    a.w[T // 2] = float("nan")
    n = fg8.fg8_moe_mlp_workspace_bytes(T, k, E, H, I, fg8.scale_fmt_code(fmt))
    want = a.run(fg8, workspace=torch.zeros(n, dtype=U8, device="cuda"))
    for _ in range(3):
        _leave_noise(n)
        assert torch.equal(a.run(fg8), want)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K,N", [(5, 400, 264), (130, 1040, 256), (256, 8192, 1024), (3, 2064, 40000)])
def test_linears_on_used_memory(fg8, fmt, M, K, N):
    x, r = W.x_outliers(M, K, seed=M).cuda(), W.normal((M, K), 1.0, seed=K).cuda()
    nw = torch.ones(K, dtype=BF16, device="cuda")
    wq, ws = fg8.quantize_weight(W.normal((N, K), 0.05, seed=N).cuda(), fmt)
    n = fg8.fg8_linear_workspace_bytes(M, N, K, fg8.scale_fmt_code(fmt))
    wsp = torch.zeros(n, dtype=U8, device="cuda")
    want = (fg8.rmsnorm_linear(x, nw, wq, ws, None, 1e-6, r, fmt, workspace=wsp)[0],
            fg8.silu_mul_linear(x, r, wq, ws, None, fmt, workspace=wsp))
    for _ in range(3):
        _leave_noise(n)
        assert torch.equal(fg8.rmsnorm_linear(x, nw, wq, ws, None, 1e-6, r, fmt)[0], want[0])
        _leave_noise(n)
        assert torch.equal(fg8.silu_mul_linear(x, r, wq, ws, None, fmt), want[1])
