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
