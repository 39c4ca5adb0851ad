"""The few-token expert layer's bounded waits: with the test hook on, its MMA
thread waits on a barrier that nothing completes; after the wait limit (1 ms
here) the kernels record FG8_ERR_TIMEOUT, drain their copies and return, and
the same workspace gives right results again once the status was read."""
import pytest
import torch

from test_gpu_block_ops import Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fg8():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import fine_grained_fp8_act_b200 as m
    m.lib()
    return m


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("T,k,E,H,I,fmt", [(1, 2, 4, 512, 256, "float"), (40, 4, 8, 2048, 640, "ue8m0")])
def test_moe_wait_limit_reports_timeout(fg8, T, k, E, H, I, fmt, codes):
    a = Layer(fg8, T, k, E, H, I, fmt, seed=5)
    kw = {}
    if codes:
        xq, xs = fg8.quantize_act(a.x, fmt)
        kw = dict(x=xq, x_scale=xs)
    n = fg8.fg8_moe_mlp_workspace_bytes(T, k, E, H, I, fg8.scale_fmt_code(fmt))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    want = a.run(fg8, **dict(kw))
    torch.cuda.synchronize()
    try:
        fg8.fg8_set_wait_limit_ns(1_000_000)
        fg8.fg8_set_test_stall(True)
        a.run(fg8, workspace=ws, **dict(kw))
        torch.cuda.synchronize()
        assert fg8.fg8_check_device_status(ws.data_ptr(), s) == fg8.FG8_ERR_TIMEOUT
    finally:
        fg8.fg8_set_test_stall(False)
        fg8.fg8_set_wait_limit_ns(2_000_000_000)
    y = a.run(fg8, workspace=ws, **dict(kw))
    assert fg8.fg8_check_device_status(ws.data_ptr(), s) == fg8.FG8_OK
    assert torch.equal(y, want)
    a.check(y)
