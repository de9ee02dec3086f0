"""The stream of a call and its tensors' device, with a stand-in for a stream of a device that
this machine does not have."""
import types

import pytest
import torch

import kimi_delta_attention_12_gb300 as kda

OTHER = types.SimpleNamespace(device=torch.device("cuda", 7))


def test_a_stream_of_another_device_is_refused():
    with pytest.raises(ValueError, match="stream is of cuda:7"):
        kda._on(OTHER, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["prefill", "batch", "decode", "backward", "norm",
                                  "norm_backward"])
def test_every_call_refuses_it(call):
    x = torch.zeros(4, 2, 32, device="cuda")
    g = torch.zeros(2, device="cuda")
    y, w = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    calls = dict(
        prefill=lambda: kda.kda_lin_prefill(x, x, x, g, stream=OTHER),
        batch=lambda: kda.kda_lin_prefill(x[None], x[None], x[None], g, stream=OTHER),
        decode=lambda: kda.kda_lin_decode_step(x, x, x, g, torch.zeros(4, 2, 32, 32,
                                                                       device="cuda"),
                                               stream=OTHER),
        backward=lambda: kda.kda_lin_backward(x, x, x, g, x, stream=OTHER),
        norm=lambda: kda.kda_block_norm(y, w, stream=OTHER),
        norm_backward=lambda: kda.kda_block_norm_backward(y, w, y, stream=OTHER))
    with pytest.raises(ValueError, match="stream is of cuda:7"):
        calls[call]()
