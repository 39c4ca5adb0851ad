"""What the few-token expert layer's two kernels report while they overlap:
the second one's wait limit counts its own waits, not the first one's time."""
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


def _workspace(fg8, T, k, E, H, I, fmt):
    return torch.zeros(fg8.fg8_moe_mlp_workspace_bytes(T, k, E, H, I, fg8.scale_fmt_code(fmt)), dtype=torch.uint8,
                       device="cuda")


@pytest.mark.parametrize("T,k,E,H,I,fmt", [(1, 2, 4, 512, 256, "float"), (40, 4, 8, 2048, 640, "ue8m0"),
                                           (24, 2, 8, 4096, 1024, "float")])
def test_second_kernel_sits_out_a_slow_first(fg8, T, k, E, H, I, fmt):
    """One CTA of the first kernel is three wait limits late: the second kernel, whose other CTAs started long before,
    waits for it without a timeout, and neither adds to sums nor counts arrivals that are still the first one's."""
    a = Layer(fg8, T, k, E, H, I, fmt, seed=5)
    ws = _workspace(fg8, T, k, E, H, I, fmt)
    s = torch.cuda.current_stream().cuda_stream
    want = a.run(fg8, workspace=ws)
    torch.cuda.synchronize()
    try:
        fg8.fg8_set_wait_limit_ns(20_000_000)
        fg8.fg8_set_test_stall(2)
        y = a.run(fg8, workspace=ws)
        torch.cuda.synchronize()
        assert fg8.fg8_check_device_status(ws.data_ptr(), s) == fg8.FG8_OK
    finally:
        fg8.fg8_set_test_stall(0)
        fg8.fg8_set_wait_limit_ns(2_000_000_000)
    assert torch.equal(y, want)
    assert bool((ws[:1024] == 0).all())                          # status word and counters at rest
    assert torch.equal(a.run(fg8, workspace=ws), want)


@pytest.mark.parametrize("T,k,E,H,I,fmt", [(5, 2, 4, 512, 256, "float"), (40, 4, 8, 2048, 640, "ue8m0")])
def test_timeout_outlives_a_bad_expert(fg8, T, k, E, H, I, fmt):
    """The first kernel times out on routing that also names an expert out of range: y is unspecified then, and the
    status says so, rather than that some slots were skipped."""
    a = Layer(fg8, T, k, E, H, I, fmt, seed=6)
    ws = _workspace(fg8, T, k, E, H, I, fmt)
    s = torch.cuda.current_stream().cuda_stream
    good = a.ids.clone()
    a.ids[1, 0] = E
    try:
        fg8.fg8_set_wait_limit_ns(40_000_000)
        fg8.fg8_set_test_stall(3)
        a.run(fg8, workspace=ws)
        torch.cuda.synchronize()
        assert fg8.fg8_check_device_status(ws.data_ptr(), s) == fg8.FG8_ERR_TIMEOUT
    finally:
        fg8.fg8_set_test_stall(0)
        fg8.fg8_set_wait_limit_ns(2_000_000_000)
    a.run(fg8, workspace=ws)
    assert fg8.fg8_check_device_status(ws.data_ptr(), s) == fg8.FG8_ERR_INVALID_ARG
    a.ids.copy_(good)
    a.check(a.run(fg8, workspace=ws))
    assert fg8.fg8_check_device_status(ws.data_ptr(), s) == fg8.FG8_OK
