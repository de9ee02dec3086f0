"""4-D batches of the decayed linear attention: strided ones on the caller's stream, and
shapes that do not go together."""
import pytest
import torch

import kimi_delta_attention_12_gb300 as kda

pytestmark = pytest.mark.gpu


def batch(dtype, d, B=3, T=200, H=2):
    """q, k, v as a [B, H, T, d] projection gives them, seen as [B, T, H, d]."""
    gen = torch.Generator(device="cuda").manual_seed(d)
    x = [torch.randn(B, H, T, d, generator=gen, device="cuda").mul(d ** -0.5).to(dtype)
         .transpose(1, 2) for _ in range(3)]
    return x, -torch.rand(H, generator=gen, device="cuda")


@pytest.mark.parametrize("dtype,d", [(torch.float32, 64), (torch.bfloat16, 128)])
def test_strided_batch_on_a_side_stream(dtype, d):
    """The rows are laid out on the stream that reads them: a current stream that is busy
    holds nothing up, and nothing of its work is waited for or missed."""
    x, g = batch(dtype, d)
    want = kda.kda_lin_prefill(*(t.contiguous() for t in x), g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(100_000_000)                 # some 50 ms of the current stream
    got = kda.kda_lin_prefill(*x, g, stream=side)
    side.synchronize()
    with torch.cuda.stream(side):
        same = [bool(torch.equal(a, b)) for a, b in zip(got, want)]
    assert all(same)
    torch.cuda.synchronize()


def test_batches_of_other_shapes_are_refused():
    (q, k, v), g = batch(torch.float32, 32)
    swapped = k.transpose(0, 1).contiguous()       # [T, B, H, d] beside [B, T, H, d]
    with pytest.raises(ValueError):
        kda.kda_lin_prefill(q, swapped, v, g)
    with pytest.raises(ValueError):
        kda.kda_lin_prefill(q, k, v.transpose(0, 1), g)
    with pytest.raises(ValueError):
        kda.kda_lin_prefill(q, k[0], v, g)


def test_host_batches_are_refused():
    x = [torch.zeros(2, 4, 1, 32) for _ in range(3)]
    with pytest.raises(ValueError):
        kda.kda_lin_prefill(*x, torch.zeros(1))


@pytest.mark.parametrize("dtype,d", [(torch.float32, 32), (torch.bfloat16, 128)])
def test_status_after_calls_of_no_tokens(dtype, d):
    """A workspace with leftovers of another use reports no timeout."""
    q = torch.empty(0, 2, d, dtype=dtype, device="cuda")
    g = torch.zeros(2, device="cuda")
    cu = torch.zeros(4, dtype=torch.int32)
    need = max(kda.lin_prefill_workspace_bytes(3, 0, 2, d, d, dtype),
               kda.lin_backward_workspace_bytes(3, 0, 2, d, d, dtype))
    for final in (False, True):
        w = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        kda.kda_lin_prefill(q, q, q, g, None, cu.cuda(), cu, output_final_state=final,
                            workspace=w)
        assert kda.workspace_status(w) == kda.KDA_OK
    w = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    kda.kda_lin_backward(q, q, q, g, q, None, cu.cuda(), cu, workspace=w)
    assert kda.workspace_status(w) == kda.KDA_OK
