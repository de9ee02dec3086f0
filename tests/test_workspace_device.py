"""Which device a workspace is allocated on."""
import pytest
import torch

import kimi_delta_attention_12_gb300 as kda


@pytest.mark.parametrize("device,on", [(None, "cuda"), (0, 0), (1, 1), ("cpu", "cpu")])
def test_workspace_on_the_device_that_is_named(monkeypatch, device, on):
    """Device 0 is device 0, whichever is the current one."""
    from kimi_delta_attention_12_gb300 import build
    build.build()
    seen = []
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: seen.append(device))
    kda.alloc_workspace(2, 128, 4, 128, 128, torch.bfloat16, device=device)
    assert seen == [on]
