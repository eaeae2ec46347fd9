"""Outputs that share memory with an input other threads still read are refused
before anything is launched; neighbours in one buffer are not."""
import pytest
import torch

import fp8_fine_grained_quant_b200 as fq

pytestmark = pytest.mark.gpu
T, ROWS, D, I = 128, 256, 256, 128
bf16, u8 = torch.bfloat16, torch.uint8


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def _views(dev, elements, other, dtype, starts):
    """(buffer of `elements` at the front, one of `other` from each start)."""
    buf = torch.zeros(max(starts) + elements + other, dtype=dtype, device=dev)
    return buf[:elements], [buf[s:s + other] for s in starts]


def _refused(call, match):
    n = fq.launch_count()
    with pytest.raises(ValueError, match=match):
        call()
    assert fq.launch_count() == n


def test_combine_into_its_rows(dev):
    slots = torch.arange(T, dtype=torch.int32, device=dev)[:, None]
    y, outs = _views(dev, ROWS * D, T * D, bf16, [0, 128, ROWS * D - 128, ROWS * D])
    y.fill_(1.0)
    for out in outs[:-1]:
        _refused(lambda: fq.fp8_moe_combine(y.view(ROWS, D), slots, out=out.view(T, D)), "out may not be y")
    assert bool((fq.fp8_moe_combine(y.view(ROWS, D), slots, out=outs[-1].view(T, D)) == 1).all())
    out, ys = _views(dev, T * D, ROWS * D, bf16, [128, T * D])
    _refused(lambda: fq.fp8_moe_combine(ys[0].view(ROWS, D), slots, out=out.view(T, D)), "out may not be y")
    fq.fp8_moe_combine(ys[1].view(ROWS, D), slots, out=out.view(T, D))


def test_combine_gradient_into_its_rows(dev):
    slots = torch.arange(T, dtype=torch.int32, device=dev)[:, None]
    w = torch.ones((T, 1), device=dev)
    dout, y0 = torch.ones((T, D), dtype=bf16, device=dev), torch.ones((ROWS, D), dtype=bf16, device=dev)
    y, dys = _views(dev, ROWS * D, ROWS * D, bf16, [0, D, ROWS * D - 128, ROWS * D])
    for dy in dys[:-1]:
        _refused(lambda: fq.fp8_moe_combine_bwd(dout, y.view(ROWS, D), slots, w, dy=dy.view(ROWS, D)), "dy may not be y")
    got, _ = fq.fp8_moe_combine_bwd(dout, y.view(ROWS, D), slots, w, dy=dys[-1].view(ROWS, D))
    assert bool((got[:T] == 1).all())
    do, dys = _views(dev, T * D, ROWS * D, bf16, [0, T * D - 128])
    for dy in dys:
        _refused(lambda: fq.fp8_moe_combine_bwd(do.view(T, D), y0, slots, w, dy=dy.view(ROWS, D)), "dy may not be dout")


def test_swiglu_gradient_into_its_checkpoint(dev):
    dh = torch.ones((T, I), dtype=bf16, device=dev)
    n, ns = T * 2 * I, T * 2 * I // 128
    sc = torch.ones((T, ns // T), device=dev)
    qc, qs = _views(dev, n, n, u8, [0, 128, n - 16, n])
    for q in qs[:-1]:
        _refused(lambda: fq.fp8_swiglu_bwd_1x128(dh, qc.view(T, 2 * I), sc, q=q.view(T, 2 * I)), "q may not be qc")
    fq.fp8_swiglu_bwd_1x128(dh, qc.view(T, 2 * I), sc, q=qs[-1].view(T, 2 * I))
    sc, ss = _views(dev, ns, ns, torch.float32, [0, 1, ns - 1, ns])
    for s in ss[:-1]:
        _refused(lambda: fq.fp8_swiglu_bwd_1x128(dh, qc.view(T, 2 * I), sc, s=s), "s may not be sc")
    fq.fp8_swiglu_bwd_1x128(dh, qc.view(T, 2 * I), sc, s=ss[-1])
    dh, dcs = _views(dev, T * I, n, bf16, [0, T * I - 128])
    for dc in dcs:
        _refused(lambda: fq.fp8_swiglu_bwd_1x128(dh.view(T, I), qc.view(T, 2 * I), sc, dc=dc.view(T, 2 * I)),
                 "dc may not be dh")
