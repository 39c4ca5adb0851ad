"""The workspace that the wrappers around the linears make for a call of their
own: only its header starts at zero (host side)."""
import pytest
import torch

from fine_grained_fp8_act_b200 import layer

U8 = torch.uint8


@pytest.fixture
def dirty(monkeypatch):
    """torch.empty on memory that was used before."""
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: torch.full((n,), 0xA5, dtype=dtype, device=device))


@pytest.mark.parametrize("nbytes", [0, 512, 1024, 5000])
def test_only_the_header_is_zeroed(dirty, nbytes):
    ws = layer._workspace_behind_header(nbytes, torch.device("cpu"), None)
    assert ws.dtype is U8 and ws.numel() == max(nbytes, 1024)
    assert bool((ws[:1024] == 0).all()) and bool((ws[1024:] == 0xA5).all())


def test_a_given_workspace_stays_as_it_is():
    ws = torch.full((4096,), 7, dtype=U8)
    assert layer._workspace_behind_header(4000, ws.device, ws) is ws and bool((ws == 7).all())
    with pytest.raises(ValueError, match="too small"):
        layer._workspace_behind_header(4097, ws.device, ws)
