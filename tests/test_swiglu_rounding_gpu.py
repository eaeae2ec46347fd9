"""Every bf16 of the SwiGLU with its checkpoint, made visible.

h is known outside only through its tile's codes and scale.  In a tile whose other
127 elements are far smaller, the scale fl32(|h| / 448) names |h| (bf16 values differ
by 2^-9 at least, scales by 2^-24) and the code's sign bit its sign.  The sweep takes
every finite bf16 gate from -110 to the largest with every mantissa of up, scaled so
that |h| is near 1: the relative error of the FP32 evaluation does not depend on up's
exponent, so a bracket that is anywhere too narrow gives a wrong bf16 here.
"""
import numpy as np
import pytest
import torch

import oracle
import fp8_fine_grained_quant_b200 as fq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def _pairs(gate_bits, dev):
    """(gate, up) bf16 for every gate and every mantissa of up, |silu(gate) up| in [1/2, 4) where up can reach it."""
    g = gate_bits.to(torch.int16).to(dev).view(torch.bfloat16)
    gd = g.double()
    silu = gd * torch.sigmoid(gd)
    _, e = torch.frexp(silu)
    man = 1.0 + torch.arange(128, device=dev, dtype=torch.float64) / 128.0
    u = torch.ldexp(man[None, :].expand(g.numel(), 128).clone(), (-e).clamp(-126, 127)[:, None])
    u = u * torch.where(torch.arange(128, device=dev) % 3 == 0, -1.0, 1.0)[None, :]
    ub = u.to(torch.bfloat16)
    assert torch.equal(ub.double(), u)
    return g[:, None].expand(-1, 128).contiguous().view(-1), ub.view(-1)


def _seen(g, u, fill_up, dev):
    """(scale, sign) of each pair's tile, the pair at a place that moves from tile to tile."""
    n = g.numel()
    c1 = torch.empty((n, 2, 128), dtype=torch.bfloat16, device=dev)
    c1[:, 0] = 1.0
    c1[:, 1] = fill_up
    tile = torch.arange(n, device=dev)
    at = (tile * 37 + tile // 128) % 128
    c1[tile, 0, at] = g
    c1[tile, 1, at] = u
    (qh, sh), _ = fq.fp8_swiglu_ckpt_1x128(c1.view(n, 256))
    code = qh.view(torch.uint8)[tile, at]
    assert bool(((code & 0x7F) == 0x7E).all())               # it is its tile's largest
    return sh.view(-1).cpu().numpy(), (code >> 7).cpu().numpy()


# In a lane of 16 elements the others decide which way the kernel goes: all inside its FP32 range, or one below it.
@pytest.mark.parametrize("fill_up", [2.0 ** -60, 2.0 ** -110])
def test_every_gate_with_every_mantissa_of_up(dev, fill_up):
    positive = torch.arange(0x0001, 0x7F80, dtype=torch.int32)                       # finite
    negative = torch.arange(0x0001, 0x42DD, dtype=torch.int32) - 0x8000              # to -110
    gates = torch.cat([positive, negative])
    wrong = 0
    for part in gates.split(1 << 13):
        g, u = _pairs(part, dev)
        s, sign = _seen(g, u, fill_up, dev)
        bits = torch.stack([g, u], 1).view(torch.int16).cpu().numpy().view(np.uint16)
        h = oracle.swiglu_bf16(bits)[:, 0]
        mag = ((h & 0x7FFF).astype(np.uint32) << 16).view(np.float32)
        wrong += int(((s != mag / np.float32(448.0)) | (sign != h >> 15)).sum())
    assert wrong == 0, wrong
