"""8-bit activation checkpoints on the GPU: the SwiGLU's checkpoint, its backward
from there, the weight-gradient operand, and a training step of the expert MLP
made of them.

Bounds (u = 2^-24): exp(-|g|) is the square of an ex2.approx (4u, so 8u, and 0.6u
of roundings), rcp.approx is within 2u, sums and products within 1u each.  Of p and
1 - p the larger, r = 1 / (1 + e), is off by at most 4.3u + 3u = 7.3u relative, the
smaller, e r, by 8.6u + 4u = 12.6u (an error of e reaches them as e / (1 + e) and
1 / (1 + e) of it).  With three products and the sum 1 + g (1 - p), d is within 17u
of the magnitudes that the oracle returns (|dh u| p (|g| (1 - p) + |1 + g (1 - p)|)
and |dh g p|); the tests allow 32u = 2^-19, and 2^-8 for the bf16 rounding.
"""
import numpy as np
import pytest
import torch

import oracle
import fp8_fine_grained_quant_b200 as fq
from oracle import moe
from parity import assert_gemm_close, bf16_bits_of, bytes_of, to_torch_bf16
from test_chain_gpu import _c1

pytestmark = pytest.mark.gpu
TINY = 1e-35


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def _bf16(rng, shape, scale=1.0):
    return moe.f32_to_bf16((scale * rng.standard_normal(shape)).astype(np.float32))


@pytest.mark.parametrize("rows,inter", [(1, 128), (3, 384), (300, 256), (64, 2048), (777, 640)])
def test_swiglu_checkpoint(dev, rows, inter):
    rng = np.random.default_rng(rows + inter)
    c1 = _c1(rng, rows, inter)
    t = to_torch_bf16(c1, dev)
    (qh, sh), (qc, sc) = fq.fp8_swiglu_ckpt_1x128(t)
    torch.cuda.synchronize(dev)
    oq, os_ = oracle.quant_act_1x128(oracle.swiglu_bf16(c1))
    assert np.array_equal(bytes_of(qh), oq) and np.array_equal(sh.cpu().numpy(), os_)
    oq, os_ = oracle.quant_act_1x128(c1)
    assert np.array_equal(bytes_of(qc), oq) and np.array_equal(sc.cpu().numpy(), os_)
    # the bytes of the separate kernels
    q2, s2 = fq.fp8_swiglu_quant_1x128(t)
    q3, s3 = fq.fp8_quant_act_1x128(t)
    assert torch.equal(qh.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(sh, s2)
    assert torch.equal(qc.view(torch.uint8), q3.view(torch.uint8)) and torch.equal(sc, s3)


def test_swiglu_checkpoint_beside_rows_that_are_not_finite(dev):
    """Rows of NaN and infinities (blocks that nobody wrote) do not touch their
    neighbours' tiles."""
    rng = np.random.default_rng(8)
    c1 = _c1(rng, 40, 256)
    bad = c1.copy()
    bad[5] = 0x7FC0
    bad[17, ::3] = 0x7F80
    bad[39] = 0xFF80
    good = [r for r in range(40) if r not in (5, 17, 39)]
    (qh, sh), (qc, sc) = fq.fp8_swiglu_ckpt_1x128(to_torch_bf16(bad, dev))
    torch.cuda.synchronize(dev)
    oq, os_ = oracle.quant_act_1x128(oracle.swiglu_bf16(c1))
    assert np.array_equal(bytes_of(qh)[good], oq[good]) and np.array_equal(sh.cpu().numpy()[good], os_[good])
    oq, os_ = oracle.quant_act_1x128(c1)
    assert np.array_equal(bytes_of(qc)[good], oq[good]) and np.array_equal(sc.cpu().numpy()[good], os_[good])


def _check_tiles(q, s, d, err):
    """q, s quantize values within err of d (float64): s within the error of the tile's amax (and its own
    rounding), every code that of a value within err."""
    rows, n = d.shape
    s = s.reshape(rows, n // 128, 1)
    dt, et = d.reshape(rows, -1, 128), err.reshape(rows, -1, 128)
    amax, ea = np.abs(dt).max(axis=2, keepdims=True), et.max(axis=2, keepdims=True)
    zero = amax == 0
    assert np.all(np.abs(s - amax / 448)[~zero] <= ((ea + amax * 2.0 ** -23) / 448 + TINY)[~zero])
    assert np.all(s[zero] == 1)
    dec = oracle.e4m3_decode_table()

    def value(v):
        return dec[oracle.e4m3_encode_array(np.clip(v, -500, 500).astype(np.float32).reshape(-1))].reshape(v.shape)

    wide = 2.0 ** -22     # the quotient's rounding and the float32 conversions here
    x = dt / s
    got = dec[q].reshape(rows, -1, 128)
    assert np.all(got >= value(x - et / s - wide * np.abs(x)))
    assert np.all(got <= value(x + et / s + wide * np.abs(x)))


@pytest.mark.parametrize("rows,inter", [(1, 128), (5, 384), (130, 256), (64, 2048), (333, 640)])
def test_swiglu_gradient_from_the_checkpoint(dev, rows, inter):
    rng = np.random.default_rng(rows + inter)
    qc, sc = oracle.quant_act_1x128(_c1(rng, rows, inter))
    dh = _bf16(rng, (rows, inter), 0.1)
    dh[0, :128] = 0                                              # a tile without gradient
    tq, ts = torch.from_numpy(qc).to(dev), torch.from_numpy(sc).to(dev)
    # the huge magnitudes of the SwiGLU's edge values overflow a gradient: keep their products finite
    big = np.abs(moe.dequant_1x128(qc, sc)) > 1e30
    dh[(big[:, :inter] | big[:, inter:])] = 0
    dc, (q, s) = fq.fp8_swiglu_bwd_1x128(to_torch_bf16(dh, dev), tq, ts)
    torch.cuda.synchronize(dev)
    ref, mag = moe.swiglu_bwd(moe.bf16_to_f32(dh).astype(np.float64), qc, sc)
    err = 2.0 ** -19 * mag + TINY
    got = moe.bf16_to_f32(bf16_bits_of(dc)).astype(np.float64)
    assert np.all(np.abs(got - ref) <= err + 2.0 ** -8 * (np.abs(ref) + err))
    _check_tiles(bytes_of(q), s.cpu().numpy().astype(np.float64), ref, err)


def test_swiglu_gradient_of_extreme_gates(dev):
    """Gates where exp overflows or 1 - p vanishes, and gates of both zeros."""
    g = np.array([-448.0, -100.0, -90.0, -88.0, -1.28125, -0.0, 0.0, 1.0, 20.0, 90.0, 448.0], dtype=np.float32)
    codes = oracle.e4m3_encode_array(np.resize(g, 128))
    qc = np.concatenate([codes, np.full(128, oracle.e4m3_encode(1.5), np.uint8)])[None]
    sc = np.ones((1, 2), np.float32)
    dh = np.full((1, 128), moe.f32_to_bf16(np.float32([-2.0]))[0], np.uint16)
    dc, (q, s) = fq.fp8_swiglu_bwd_1x128(to_torch_bf16(dh, dev), torch.from_numpy(qc).to(dev), torch.from_numpy(sc).to(dev))
    ref, mag = moe.swiglu_bwd(np.full((1, 128), -2.0), qc, sc)
    err = 2.0 ** -19 * mag + TINY
    got = dc.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= err + 2.0 ** -8 * (np.abs(ref) + err))
    _check_tiles(bytes_of(q), s.cpu().numpy().astype(np.float64), ref, err)


@pytest.mark.parametrize("M,K,Mp", [(1, 128, None), (128, 128, 128), (200, 256, None), (200, 384, 256), (1000, 640, None),
                                    (512, 1152, None), (0, 128, 512), (3, 7168, 128)])
def test_token_axis_operand(dev, M, K, Mp):
    rng = np.random.default_rng(M + K)
    x = _bf16(rng, (M, K))
    x = moe.f32_to_bf16(moe.bf16_to_f32(x) * np.exp(rng.standard_normal((M, 1)) * 2).astype(np.float32))
    if M > 2:
        x[1] = 0                                                  # a token of zeros (scale 1)
        x[:, 5] = 0                                               # a channel of zeros
        x[2, :64] = moe.f32_to_bf16(np.float32([1e-39]))[0]       # subnormal values and scales
    q, s = oracle.quant_act_1x128(x) if M else (np.zeros((0, K), np.uint8), np.zeros((0, K // 128), np.float32))
    qt, st = fq.fp8_ckpt_128x1_t(torch.from_numpy(q).to(dev), torch.from_numpy(s).to(dev), Mp)
    torch.cuda.synchronize(dev)
    oqt, ost = moe.ckpt_128x1_t(q, s, qt.shape[1])
    assert np.array_equal(st.cpu().numpy(), ost)
    assert np.array_equal(bytes_of(qt), oqt)


def test_token_axis_operand_near_ties_and_scale_range(dev):
    """Scales that put quotients on and next to E4M3 midpoints, tiny scales (the
    division path) and large ones."""
    rng = np.random.default_rng(77)
    M, K = 384, 256
    q = rng.integers(0, 0x7F, (M, K)).astype(np.uint8) | (rng.integers(0, 2, (M, K)) << 7).astype(np.uint8)
    s = np.ones((M, K // 128), np.float32)
    s[128:256] = np.float32(2.0) ** rng.integers(-40, 40, (128, K // 128)).astype(np.float32)
    s[256:320] = np.float32(1e-40) * rng.integers(1, 50, (64, K // 128)).astype(np.float32)
    s[320:] = np.nextafter(np.float32(1.0), np.float32(2.0)) * rng.choice(np.float32([1, 0.5, 1.25, 1.5]), (64, K // 128))
    for lo, hi in ((0, 128), (128, 256), (256, 320), (320, 384), (0, 384)):
        qt, st = fq.fp8_ckpt_128x1_t(torch.from_numpy(q[lo:hi].copy()).to(dev), torch.from_numpy(s[lo:hi].copy()).to(dev))
        oqt, ost = moe.ckpt_128x1_t(q[lo:hi], s[lo:hi], qt.shape[1])
        assert np.array_equal(st.cpu().numpy(), ost)
        assert np.array_equal(bytes_of(qt), oqt)


def test_wgrad_from_a_checkpoint(dev):
    """dW = dY^T X with X kept as the codes that the forward pass multiplied."""
    rng = np.random.default_rng(5)
    M, N, K = 700, 256, 384
    x, dy = _bf16(rng, (M, K)), _bf16(rng, (M, N))
    qx, sx = fq.fp8_quant_act_1x128(to_torch_bf16(x, dev))
    qxt, sxt = fq.fp8_ckpt_128x1_t(qx, sx)
    qdt, sdt = fq.fp8_quant_act_128x1_t(to_torch_bf16(dy, dev))
    dw = fq.fp8_gemm_wgrad(qdt, sdt, qxt, sxt)
    torch.cuda.synchronize(dev)
    assert fq.get_device_error(device=dev) == fq.OK
    oqt, ost = moe.ckpt_128x1_t(bytes_of(qx), sx.cpu().numpy(), 1024)
    ref = oracle.gemm_1d1d(bytes_of(qdt), sdt.cpu().numpy().T.copy(), oqt, ost.T.copy())
    assert_gemm_close(bf16_bits_of(dw), ref, "wgrad from a checkpoint")


def test_expert_mlp_training_step(dev):
    """Route -> layout -> dispatch -> GEMM1 -> SwiGLU with checkpoint -> GEMM2 ->
    combine, and back: combine gradient -> Dgrad2 -> SwiGLU gradient from the
    checkpoint -> Dgrad1 -> dispatch gradient and routing gradient, with Wgrad
    operands of one expert from its saved rows.  Every step is compared with the
    oracle on that step's own inputs, so errors do not pile up."""
    rng = np.random.default_rng(6)
    T, E, k, D, I = 200, 4, 2, 256, 128
    x, do = _bf16(rng, (T, D)), _bf16(rng, (T, D), 0.1)
    l = rng.standard_normal((T, E)).astype(np.float32)
    w1, w2 = _bf16(rng, (E, 2 * I, D), 0.06), _bf16(rng, (E, D, I), 0.09)
    logits = torch.from_numpy(l).to(dev)
    ids, w = fq.fp8_moe_route(logits, k, score="sigmoid")
    slots, m, counts = fq.fp8_moe_layout_contiguous(ids, E)
    rows = m.numel() * 128
    qx, sx = fq.fp8_moe_dispatch_1x128(to_torch_bf16(x, dev), slots, rows, m_indices=m, counts=counts,
                                       q=torch.zeros((rows, D), dtype=torch.uint8, device=dev),
                                       s=torch.ones((rows, D // 128), device=dev))
    qw1, sw1 = fq.fp8_quant_w_128x128(to_torch_bf16(w1, dev))
    qw2, sw2 = fq.fp8_quant_w_128x128(to_torch_bf16(w2, dev))
    c1 = torch.zeros((rows, 2 * I), dtype=torch.bfloat16, device=dev)
    fq.fp8_grouped_gemm_contiguous(qx, sx, qw1, sw1, m, out=c1)
    (qh, sh), (qc, sc) = fq.fp8_swiglu_ckpt_1x128(c1)
    y = torch.zeros((rows, D), dtype=torch.bfloat16, device=dev)
    fq.fp8_grouped_gemm_contiguous(qh, sh, qw2, sw2, m, out=y)
    out = fq.fp8_moe_combine(y, slots, w)
    # backward
    dy, dw = fq.fp8_moe_combine_bwd(to_torch_bf16(do, dev), y, slots, w, m_indices=m, counts=counts,
                                    dy=torch.zeros_like(y))
    qdy, sdy = fq.fp8_quant_act_1x128(dy)
    qw2t, sw2t = fq.fp8_transpose_w_128x128(qw2, sw2)
    dh = torch.zeros((rows, I), dtype=torch.bfloat16, device=dev)
    fq.fp8_grouped_gemm_contiguous(qdy, sdy, qw2t, sw2t, m, out=dh)
    dc, (qd, sd) = fq.fp8_swiglu_bwd_1x128(dh, qc, sc)
    qw1t, sw1t = fq.fp8_transpose_w_128x128(qw1, sw1)
    dxr = torch.zeros((rows, D), dtype=torch.bfloat16, device=dev)
    fq.fp8_grouped_gemm_contiguous(qd, sd, qw1t, sw1t, m, out=dxr)
    dx = fq.fp8_moe_combine(dxr, slots)
    dl = fq.fp8_moe_route_bwd(logits, ids, dw, score="sigmoid")
    torch.cuda.synchronize(dev)
    assert fq.get_device_error(device=dev) == fq.OK

    oi, ow = moe.route(l, k, score="sigmoid")
    osl, om, oc = moe.layout_contiguous(oi, E)
    assert np.array_equal(ids.cpu().numpy(), oi) and np.array_equal(slots.cpu().numpy(), osl)
    used = np.repeat(om >= 0, 128)

    def grouped(q, s, qw, sw):
        return oracle.grouped_contiguous(bytes_of(q), s.cpu().numpy(), bytes_of(qw), sw.cpu().numpy(), om)[used]

    assert_gemm_close(bf16_bits_of(c1)[used], grouped(qx, sx, qw1, sw1), "GEMM1")
    assert_gemm_close(bf16_bits_of(y)[used], grouped(qh, sh, qw2, sw2), "GEMM2")
    assert_gemm_close(bf16_bits_of(dh)[used], grouped(qdy, sdy, qw2t, sw2t), "Dgrad2")
    assert_gemm_close(bf16_bits_of(dxr)[used], grouped(qd, sd, qw1t, sw1t), "Dgrad1")

    def f64(t):
        return moe.bf16_to_f32(bf16_bits_of(t)).astype(np.float64)

    def close(got, ref, mag, n):
        acc = n * 2.0 ** -24 * mag
        assert np.all(np.abs(got - ref) <= acc + 2.0 ** -8 * (np.abs(ref) + acc) + TINY)

    wv = w.double().cpu().numpy()
    close(f64(out), *moe.combine(f64(y), osl, wv), 2)
    close(f64(dx), *moe.combine(f64(dxr), osl), 2)
    rw, mag = moe.combine_dweights(moe.bf16_to_f32(do).astype(np.float64), f64(y), osl)
    assert np.all(np.abs(dw.cpu().numpy() - rw) <= 32 * 2.0 ** -24 * mag)
    ref, mag = moe.swiglu_bwd(f64(dh), bytes_of(qc), sc.cpu().numpy())
    err = 2.0 ** -19 * mag + TINY
    assert np.all(np.abs(f64(dc) - ref) <= err + 2.0 ** -8 * (np.abs(ref) + err))
    rl, mag = moe.route_bwd(l, oi, dw.cpu().numpy(), score="sigmoid")
    assert np.all(np.abs(dl.cpu().numpy() - rl) <= 2 * (2 * np.abs(l).max() + 64) * 2.0 ** -24 * mag + TINY)

    # Wgrad of the busiest expert from its saved rows: its run of the layout, padded by whole zero rows
    e = int(np.argmax(oc))
    at = np.flatnonzero(om == e)
    r0, r1 = int(at[0]) * 128, int(at[-1] + 1) * 128
    qxt, sxt = fq.fp8_ckpt_128x1_t(qx[r0:r1], sx[r0:r1])
    qdt, sdt = fq.fp8_quant_act_128x1_t(dc[r0:r1])
    dw1 = fq.fp8_gemm_wgrad(qdt, sdt, qxt, sxt)
    torch.cuda.synchronize(dev)
    oqt, ost = moe.ckpt_128x1_t(bytes_of(qx)[r0:r1], sx.cpu().numpy()[r0:r1], qxt.shape[1])
    assert np.array_equal(bytes_of(qxt), oqt) and np.array_equal(sxt.cpu().numpy(), ost)
    ref = oracle.gemm_1d1d(bytes_of(qdt), sdt.cpu().numpy().T.copy(), oqt, ost.T.copy())
    assert_gemm_close(bf16_bits_of(dw1), ref, "Wgrad1")


def test_offsets_beyond_32_bits(dev):
    """Element offsets that pass 2^32: the last rows of large operands give what
    the same rows give alone."""
    inter, n = 7168, 512
    rows = 300_544                       # rows * 2 * inter > 2^32
    assert (rows - n) * 2 * inter > 1 << 32
    c1 = torch.zeros((rows, 2 * inter), dtype=torch.bfloat16, device=dev)
    c1[-n:] = torch.randn((n, 2 * inter), dtype=torch.bfloat16, device=dev)
    (qh, sh), (qc, sc) = fq.fp8_swiglu_ckpt_1x128(c1)
    (qhn, shn), (qcn, scn) = fq.fp8_swiglu_ckpt_1x128(c1[-n:])
    del c1
    for big, small in ((qh, qhn), (sh, shn), (qc, qcn), (sc, scn)):
        assert torch.equal(big[-n:].view(torch.uint8), small.view(torch.uint8))
    assert int(qc[:-n].view(torch.uint8).count_nonzero()) == 0 and bool((sc[:-n] == 1).all())
    dh = torch.randn((rows, inter), dtype=torch.bfloat16, device=dev)
    dc, (q, s) = fq.fp8_swiglu_bwd_1x128(dh, qc, sc)
    dcn, (qn, sn) = fq.fp8_swiglu_bwd_1x128(dh[-n:], qcn, scn)
    assert torch.equal(dc[-n:], dcn) and torch.equal(q[-n:].view(torch.uint8), qn.view(torch.uint8))
    assert torch.equal(s[-n:], sn)
    del dc, dh
    qt, st = fq.fp8_ckpt_128x1_t(q, s, Mp=rows)
    qtn, stn = fq.fp8_ckpt_128x1_t(qn, sn, Mp=n)
    assert torch.equal(qt[:, -n:].contiguous().view(torch.uint8), qtn.view(torch.uint8))
    assert torch.equal(st[-(n // 128):], stn)
