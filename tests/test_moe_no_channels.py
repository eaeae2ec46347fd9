"""The combine's gradient of rows without channels: the weights' gradients are sums
of nothing, and still written."""
import pytest
import torch

import fp8_fine_grained_quant_b200 as fq

A16 = 0x10000


@pytest.mark.parametrize("args,status", [
    ((None, None, 256, 0, A16, A16, 4, 2, None, None, 0, None, None, None), fq.ERR_NULL),    # no dweights
    ((None, None, 256, 0, None, A16, 4, 2, None, None, 0, None, A16, None), fq.ERR_NULL),    # no slots
    ((None, None, 256, 0, A16, None, 4, 2, None, None, 0, None, A16, None), fq.ERR_NULL),    # no weights
    ((None, None, 256, 0, A16, A16, 4, 2, None, None, 0, None, A16 + 1, None), fq.ERR_ALIGN),
    ((None, None, 256, 0, A16, A16, 0, 2, None, None, 0, None, None, None), fq.OK),          # no tokens either
])
def test_argument_checks_without_channels(args, status):
    assert fq.lib().fp8_moe_combine_bwd(*args) == status


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [0, 128])
@pytest.mark.parametrize("k", [1, 2, 9, 32])
@pytest.mark.parametrize("pads", [False, True])
def test_weight_gradients_without_channels_are_zero(rows, k, pads):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev = torch.device("cuda:0")
    T = 300

    def bf16(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device=dev)

    slots = torch.randint(-1, 128, (T, k), dtype=torch.int32, device=dev)
    layout = dict(m_indices=torch.zeros(rows // 128, dtype=torch.int32, device=dev),
                  counts=torch.full((4,), 70, dtype=torch.int32, device=dev)) if pads else {}
    dw = torch.full((T, k), 7.0, device=dev)
    dy, got = fq.fp8_moe_combine_bwd(bf16(T, 0), bf16(rows, 0), slots, torch.full((T, k), float("nan"), device=dev),
                                     dweights=dw, **layout)
    assert dy.shape == (rows, 0) and got is not None and bool((dw == 0).all())
    assert fq.fp8_moe_combine(bf16(rows, 0), slots).shape == (T, 0)
