"""A contiguous layout cut off at a block: a user's buffers hold fewer rows than the
layout needs, and end inside an expert's run.  The entries whose rows are left keep
them: only rows past an expert's count are padding."""
import numpy as np
import pytest
import torch

import oracle
import fp8_fine_grained_quant_b200 as fq
from oracle import moe
from parity import bf16_bits_of, to_torch_bf16

pytestmark = pytest.mark.gpu
D = 256
COUNTS = [200, 0, 128, 1, 384, 0, 257]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def _layout(rng, dev):
    ids = rng.permutation(np.repeat(np.arange(len(COUNTS)), COUNTS)).astype(np.int32)[:, None]
    slots, m, counts = fq.fp8_moe_layout_contiguous(torch.from_numpy(ids).to(dev), len(COUNTS))
    osl, om, oc = moe.layout_contiguous(ids, len(COUNTS))
    assert np.array_equal(slots.cpu().numpy(), osl) and oc.tolist() == COUNTS
    return slots, m, counts, osl, om, oc


def _bf16(rng, shape):
    return moe.f32_to_bf16(rng.standard_normal(shape).astype(np.float32))


BLOCKS = list(range(1, 1 + sum(-(-c // 128) for c in COUNTS))) + [12]   # 12: past the last used block


@pytest.mark.parametrize("blocks", BLOCKS)
def test_dispatch_into_a_cut_layout(dev, blocks):
    rng = np.random.default_rng(blocks)
    slots, m, counts, osl, om, oc = _layout(rng, dev)
    rows = blocks * 128
    x = _bf16(rng, (sum(COUNTS), D))
    q = torch.full((rows, D), 0x5A, dtype=torch.uint8, device=dev)
    s = torch.full((rows, D // 128), -3.0, device=dev)
    fq.fp8_moe_dispatch_1x128(to_torch_bf16(x, dev), slots, rows, m_indices=m[:blocks].contiguous(), counts=counts,
                              q=q, s=s)
    oq, os_ = oracle.quant_act_1x128(x)
    eq, es = np.full((rows, D), 0x5A, np.uint8), np.full((rows, D // 128), -3.0, np.float32)
    pad = moe.pad_rows(om, oc)[:rows]
    eq[pad], es[pad] = 0, 1.0
    kept = osl[:, 0] < rows
    eq[osl[kept, 0]], es[osl[kept, 0]] = oq[kept], os_[kept]
    assert np.array_equal(q.cpu().numpy(), eq) and np.array_equal(s.cpu().numpy(), es)


@pytest.mark.parametrize("blocks", BLOCKS)
def test_combine_gradient_of_a_cut_layout(dev, blocks):
    rng = np.random.default_rng(100 + blocks)
    slots, m, counts, osl, om, oc = _layout(rng, dev)
    rows, T = blocks * 128, sum(COUNTS)
    y, do = _bf16(rng, (rows, D)), _bf16(rng, (T, D))
    w = rng.random((T, 1)).astype(np.float32)
    dy = torch.full((rows, D), -7.0, dtype=torch.bfloat16, device=dev)
    _, dw = fq.fp8_moe_combine_bwd(to_torch_bf16(do, dev), to_torch_bf16(y, dev), slots, torch.from_numpy(w).to(dev),
                                   m_indices=m[:blocks].contiguous(), counts=counts, dy=dy)
    ref = np.full((rows, D), moe.f32_to_bf16(np.float32([-7.0]))[0], np.uint16)
    ref[moe.pad_rows(om, oc)[:rows]] = 0
    kept = osl[:, 0] < rows
    ref[osl[kept, 0]] = moe.f32_to_bf16(moe.bf16_to_f32(do)[kept] * w[kept])   # one FP32 product, one rounding
    assert np.array_equal(bf16_bits_of(dy), ref)
    rw, mag = moe.combine_dweights(moe.bf16_to_f32(do).astype(np.float64), moe.bf16_to_f32(y).astype(np.float64), osl)
    # two products in one lane's chain of eight channels, 8 chains and their joins: below 32 roundings
    assert np.all(np.abs(dw.cpu().numpy() - rw) <= 32 * 2.0 ** -24 * mag)
    assert np.all(dw.cpu().numpy()[~kept] == 0)
