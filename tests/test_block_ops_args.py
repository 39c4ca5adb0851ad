"""The host-side checks of the operators around the linears, without a GPU:
what the C entry points refuse before any launch, and which operand the
Python wrappers name."""
import pytest
import torch

import fine_grained_fp8_act_b200 as fg8

FAKE = 0x10000  # a 256-byte aligned non-null "device" address; never dereferenced on these paths
BIG = 1 << 40
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.fixture(scope="module")
def raw():
    from fine_grained_fp8_act_b200 import build
    build.build()
    return fg8.lib()


def _caller(f, order, defaults):
    def call(**kw):
        assert set(kw) <= set(order), kw
        return f(*[{**defaults, **kw}[n] for n in order])
    return call


def _gpu():
    return 0 if torch.cuda.is_available() else 3


def test_rmsnorm_refusals(raw):
    c = _caller(raw.fg8_rmsnorm_quant,
                "x M K ld_x r ld_r w eps q s fmt block ro ld_ro y ld_y stream".split(),
                dict(x=FAKE, M=4, K=256, ld_x=256, r=FAKE, ld_r=256, w=FAKE, eps=1e-6, q=FAKE, s=FAKE, fmt=0,
                     block=128, ro=FAKE, ld_ro=256, y=FAKE, ld_y=256, stream=None))
    for bad in (dict(fmt=2), dict(block=16), dict(M=-1), dict(K=0), dict(K=(1 << 30) + 16, ld_x=1 << 31), dict(ld_x=248),
                dict(ld_r=248), dict(ld_ro=248), dict(ld_y=248), dict(eps=0.0), dict(eps=-1e-6),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(w=None), dict(q=None), dict(s=None),
                dict(r=None), dict(ro=None), dict(M=1 << 31)):
        assert c(**bad) == 1, bad
    for bad in (dict(K=200, ld_x=200, ld_r=200, ld_ro=200, ld_y=200), dict(ld_x=260), dict(ld_r=260), dict(ld_ro=260),
                dict(ld_y=260), dict(x=FAKE + 8), dict(w=FAKE + 2), dict(q=FAKE + 4), dict(s=FAKE + 2),
                dict(r=FAKE + 8), dict(ro=FAKE + 8), dict(y=FAKE + 8)):
        assert c(**bad) == 2, bad
    assert c(M=0, x=None, w=None, q=None, s=None) == 0
    if not torch.cuda.is_available():
        assert c() == 3 and c(r=None, ro=None, y=None, fmt=1, s=FAKE + 1, block=32) == 3


def test_silu_mul_refusals(raw):
    c = _caller(raw.fg8_silu_mul_quant, "g u M K ld_g ld_u q s fmt block y ld_y stream".split(),
                dict(g=FAKE, u=FAKE, M=4, K=256, ld_g=512, ld_u=512, q=FAKE, s=FAKE, fmt=1, block=64, y=None, ld_y=0,
                     stream=None))
    for bad in (dict(fmt=-1), dict(block=96), dict(M=-1), dict(K=0), dict(ld_g=128), dict(ld_u=128),
                dict(y=FAKE, ld_y=128), dict(g=None), dict(u=None), dict(q=None), dict(s=None)):
        assert c(**bad) == 1, bad
    for bad in (dict(K=248), dict(ld_g=516), dict(ld_u=516), dict(g=FAKE + 8), dict(u=FAKE + 2), dict(q=FAKE + 8),
                dict(y=FAKE + 8, ld_y=256), dict(y=FAKE, ld_y=260), dict(fmt=0, s=FAKE + 2)):
        assert c(**bad) == 2, bad
    assert c(M=0, g=None) == 0


def test_prepare_refusals(raw):
    c = _caller(raw.fg8_linear_prepare_rmsnorm,
                "x M N K ld_x r ld_r w eps ro ld_ro y ld_y ws fmt wsp nb stream".split(),
                dict(x=FAKE, M=40, N=256, K=256, ld_x=256, r=None, ld_r=0, w=FAKE, eps=1e-6, ro=None, ld_ro=0, y=None,
                     ld_y=0, ws=FAKE, fmt=1, wsp=FAKE, nb=BIG, stream=None))
    for bad in (dict(fmt=3), dict(M=-1), dict(M=(1 << 31) - 1), dict(N=0), dict(ld_x=128), dict(eps=0.0), dict(x=None),
                dict(w=None), dict(ws=None), dict(r=FAKE, ld_r=256), dict(y=FAKE, ld_y=128)):
        assert c(**bad) == 1, bad
    for bad in (dict(N=252), dict(K=200), dict(x=FAKE + 8), dict(w=FAKE + 8), dict(y=FAKE + 8, ld_y=256)):
        assert c(**bad) == 2, bad
    for bad in (dict(wsp=None), dict(wsp=FAKE + 64), dict(nb=1024)):
        assert c(**bad) == 4, bad
    assert c(M=0, x=None, wsp=None) == 0
    d = _caller(raw.fg8_linear_prepare_silu_mul, "g u M N K ld_g ld_u ws fmt wsp nb stream".split(),
                dict(g=FAKE, u=FAKE, M=40, N=256, K=256, ld_g=512, ld_u=512, ws=FAKE, fmt=0, wsp=FAKE, nb=BIG,
                     stream=None))
    for bad in (dict(fmt=-1), dict(g=None), dict(u=None), dict(ws=None), dict(ld_u=128), dict(K=0)):
        assert d(**bad) == 1, bad
    for bad in (dict(N=4), dict(K=248), dict(ld_g=516), dict(u=FAKE + 8)):
        assert d(**bad) == 2, bad
    assert d(nb=2048) == 4 and d(M=0, g=None) == 0
    if not torch.cuda.is_available():
        assert c() == 3 and d() == 3


def test_route_refusals(raw):
    c = _caller(raw.fg8_moe_route, "l bf16 T E ld k renorm scale ids w stream".split(),
                dict(l=FAKE, bf16=0, T=4, E=64, ld=64, k=8, renorm=1, scale=1.0, ids=FAKE, w=FAKE, stream=None))
    for bad in (dict(T=-1), dict(T=1 << 31), dict(E=0), dict(E=1025, ld=1025), dict(k=0), dict(k=33), dict(E=4, k=5),
                dict(ld=63), dict(scale=float("nan")), dict(scale=float("inf")), dict(l=None), dict(ids=None),
                dict(w=None)):
        assert c(**bad) == 1, bad
    for bad in (dict(l=FAKE + 2), dict(bf16=1, l=FAKE + 1), dict(ids=FAKE + 2), dict(w=FAKE + 2)):
        assert c(**bad) == 2, bad
    assert c(T=0, l=None) == 0
    if not torch.cuda.is_available():
        assert c(bf16=1, l=FAKE + 2) == 3


def test_moe_mlp_refusals(raw):
    order = "x xs T H ld_x ids w k E I w13 s13 w2 s2 y ld_y fmt ws nb stream".split()
    c = _caller(raw.fg8_moe_mlp, order,
                dict(x=FAKE, xs=None, T=4, H=256, ld_x=256, ids=FAKE, w=FAKE, k=2, E=8, I=128, w13=FAKE, s13=FAKE,
                     w2=FAKE, s2=FAKE, y=FAKE, ld_y=256, fmt=1, ws=FAKE, nb=BIG, stream=None))
    for bad in (dict(T=-1), dict(T=257), dict(k=0), dict(k=33), dict(T=256, k=17), dict(E=0), dict(E=1025), dict(H=0),
                dict(H=16400, ld_x=16400, ld_y=16400), dict(I=0), dict(E=1024, I=1 << 21), dict(fmt=2), dict(ld_x=240),
                dict(ld_y=240), dict(xs=FAKE, ld_x=272), dict(x=None), dict(ids=None), dict(w=None), dict(w13=None),
                dict(s13=None), dict(w2=None), dict(s2=None), dict(y=None)):
        assert c(**bad) == 1, bad
    for bad in (dict(H=264, ld_x=264, ld_y=264), dict(I=136), dict(ld_x=260), dict(ld_y=260), dict(x=FAKE + 8),
                dict(xs=FAKE + 2, fmt=0), dict(ids=FAKE + 2), dict(w=FAKE + 2), dict(w13=FAKE + 8), dict(s13=FAKE + 4),
                dict(w2=FAKE + 8), dict(s2=FAKE + 4), dict(y=FAKE + 8)):
        assert c(**bad) == 2, bad
    for bad in (dict(ws=None), dict(ws=FAKE + 64), dict(nb=1024)):
        assert c(**bad) == 4, bad
    assert c(T=0, x=None, ws=None, nb=0) == 0
    f = raw.fg8_moe_mlp_workspace_bytes
    need = f(4, 2, 8, 256, 128, 1)
    assert need > 1024 and need % 256 == 0 and f(4, 2, 8, 264, 128, 1) == 0 and f(257, 2, 8, 256, 128, 1) == 0
    assert f(8, 2, 8, 256, 128, 1) > need
    assert c(nb=need - 1) == 4
    if not torch.cuda.is_available():
        assert c(nb=need) == 3 and c(xs=FAKE + 1, fmt=1) == 3


def _raises(match, fn, *a, **k):
    with pytest.raises(ValueError, match=match):
        fn(*a, **k)


def test_wrappers_name_the_operand():
    x, w = torch.zeros(4, 256, dtype=BF16), torch.zeros(256, dtype=BF16)
    n = fg8.rmsnorm_quant
    _raises("x must be a CUDA tensor", n, x, w, 1e-6, x)
    _raises("x must be a 2-D bf16", n, x.float(), w)
    _raises("weight must have shape", n, x, w[:128].contiguous())
    _raises("weight must be", n, x, w.float())
    _raises("residual must be", n, x, w, 1e-6, x[:3])
    _raises("residual_out needs", n, x, w, residual_out=x)
    _raises("residual_out must be", n, x, w, 1e-6, x, residual_out=torch.zeros(4, 128, dtype=BF16))
    _raises("scale_fmt", n, x, w, 1e-6, None, "fp8")
    wq, ws = torch.zeros(64, 256, dtype=E4M3), torch.zeros(1, 2)
    _raises("x must be a CUDA tensor", fg8.rmsnorm_linear, x, w, wq, ws)
    _raises("wq must have shape", fg8.rmsnorm_linear, x, w, wq[:, :128].contiguous(), ws)
    _raises("weight must have shape", fg8.rmsnorm_linear, x, w[:8], wq, ws)
    _raises("residual_out needs", fg8.rmsnorm_linear, x, w, wq, ws, residual_out=x)
    _raises("x must be a CUDA tensor", fg8.silu_mul_linear, x, x, wq, ws)
    _raises("up must be", fg8.silu_mul_linear, x, x[:2], wq, ws)
    _raises("bias must have shape", fg8.silu_mul_linear, x, x, wq, ws, w)
    s = fg8.silu_mul_quant
    _raises("gate must be a CUDA tensor", s, x, x)
    _raises("up must be", s, x, x[:, :128])
    _raises("gate must have unit stride", s, x.t(), x.t())
    r = fg8.moe_route
    _raises("logits must be a CUDA tensor", r, torch.zeros(3, 8), 2)
    _raises("logits must be a 2-D", r, torch.zeros(3, 8, dtype=torch.float16), 2)
    _raises("unit stride", r, torch.zeros(8, 3).t(), 2)
    _raises("k must be", r, torch.zeros(3, 8), 9)
    T, H, I, E, k = 4, 256, 144, 3, 2
    ids, wt = torch.zeros(T, k, dtype=I32), torch.zeros(T, k)
    w13, s13 = torch.zeros(E, 2 * I, H, dtype=E4M3), torch.zeros(E, 3, 2, dtype=F32)
    w2, s2 = torch.zeros(E, H, I, dtype=E4M3), torch.zeros(E, 2, 2, dtype=F32)
    xs = torch.zeros(T, 2)
    m = fg8.moe_mlp
    _raises("x must be a CUDA tensor", m, x, ids, wt, w13, s13, w2, s2, "float")
    _raises("x must be a CUDA tensor", m, x.to(E4M3), ids, wt, w13, s13, w2, s2, "float", x_scale=xs)
    _raises("x must be", m, x, ids, wt, w13, s13, w2, s2, "float", x_scale=xs)
    _raises("x must be a 2-D bf16", m, x.to(E4M3), ids, wt, w13, s13, w2, s2, "float")
    _raises("x_scale must have shape", m, x.to(E4M3), ids, wt, w13, s13, w2, s2, "float", x_scale=xs[:, :1].contiguous())
    _raises("ids must be", m, x, ids.long(), wt, w13, s13, w2, s2, "float")
    _raises("ids must have shape", m, x, ids[:3].contiguous(), wt, w13, s13, w2, s2, "float")
    _raises("weights must be", m, x, ids, wt.to(BF16), w13, s13, w2, s2, "float")
    _raises("w13 must have shape", m, x, ids, wt, w13[:, :I].contiguous(), s13, w2, s2, "float")
    _raises("w13_scale_inv must be", m, x, ids, wt, w13, s13, w2, s2, "ue8m0")
    _raises("w2 must have shape", m, x, ids, wt, w13, s13, w2[:2].contiguous(), s2, "float")
    _raises("w2_scale_inv must have shape", m, x, ids, wt, w13, s13, w2, s2[:, :, :1].contiguous(), "float")
    _raises("out must be", m, x, ids, wt, w13, s13, w2, s2, "float", out=torch.zeros(T, H + 8, dtype=BF16))


def test_plain_forms_agree_with_themselves():
    """The tests' 64-bit forms: a quantization made by the definition passes its own check, and one that is a step
    or a scale off does not."""
    import _plain64 as P
    g = torch.Generator().manual_seed(1)
    v = torch.randn(5, 200, generator=g, dtype=torch.float64) * 3
    for fmt in ("float", "ue8m0"):
        for block in (128, 64, 32):
            hat, s, q = P.quantize_values(v, fmt, block)
            codes = (hat / P.expand(s, block, 200)).float().to(E4M3)
            scales = s.float() if fmt == "float" else s.float().to(E8M0)
            P.check_quantized(codes, scales, v, v.abs() * 1e-6, fmt, block)
            wrong = codes.clone().view(torch.uint8)
            wrong[2, 77] += 1
            with pytest.raises(AssertionError, match="codes off"):
                P.check_quantized(wrong.view(E4M3), scales, v, v.abs() * 1e-6, fmt, block)
            other = scales.clone().view(torch.uint8) if fmt != "float" else scales.clone()
            other[1, 0] += 1 if fmt != "float" else float(scales[1, 0]) * 1e-5
            with pytest.raises(AssertionError, match="off"):
                P.check_quantized(codes, other.view(scales.dtype), v, v.abs() * 1e-6, fmt, block)
