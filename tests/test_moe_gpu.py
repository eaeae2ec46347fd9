"""Routing, layouts, dispatch and combine on the GPU, against the float64
oracle (oracle/moe.py) and the C oracle's quantizer.

Bounds (u = 2^-24, half an ulp of FP32 relative to the value; a bf16 rounding is
off by at most 2^-8):
* expf and the divisions are within 2 ulp (4u) and the argument l - m of an exp
  is rounded once (u |l - m|), so a weight is off by at most
  (2 R + 64) u relative, R the largest |l - m| (|l| for the sigmoid) of the row
  and 64 an upper count of the roundings of sums, quotients and products;
* a gradient r (g - <g, r>) (1 - p) adds the errors of its terms, bounded by the
  same factor times the sum of the magnitudes that the oracle returns, twice
  (r enters the mean too);
* a sum of k products in order: k u times the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

import oracle
import fp8_fine_grained_quant_b200 as fq
from oracle import moe
from parity import assert_gemm_close, bf16_bits_of, bytes_of, to_torch_bf16

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TINY = 1e-35   # results below FP32's normal range


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def _logits(rng, T, E, dtype, dev, sigma=1.5):
    t = torch.from_numpy((sigma * rng.standard_normal((T, E))).astype(np.float32)).to(dtype)
    return t.to(dev), t.double().numpy()


def _spread(l, score):
    f = np.where(np.isfinite(l), l, 0.0)
    return float(f.max() - f.min()) if score == "softmax" else float(np.abs(f).max())


def _check_route(dev, logits, host, k, **kw):
    bias = kw.get("bias")
    args = dict(kw, bias=None if bias is None else torch.tensor(bias, dtype=torch.float32, device=dev))
    ids, w = fq.fp8_moe_route(logits, k, **args)
    torch.cuda.synchronize(dev)
    oi, ow = moe.route(host, k, **dict(kw, bias=None if bias is None else np.float32(bias)))
    assert np.array_equal(ids.cpu().numpy(), oi)
    rows = min(_spread(host, kw.get("score", "softmax")), 400.0)
    tol = (2 * rows + 64) * U
    assert np.all(np.abs(w.cpu().numpy() - ow) <= tol * np.abs(ow) + TINY), np.abs(w.cpu().numpy() - ow).max()
    return ids, w


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (3, 2, 2), (130, 8, 2), (77, 7, 3), (65, 33, 5), (64, 60, 4),
                                   (9, 64, 32), (257, 32, 8), (50, 100, 6), (33, 160, 6), (40, 256, 8), (20, 320, 8),
                                   (6, 1000, 10), (5, 1024, 32), (30, 512, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route(dev, T, E, k, dtype, score):
    rng = np.random.default_rng(T * 1000 + E + k)
    logits, host = _logits(rng, T, E, dtype, dev)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    _check_route(dev, logits, host, k, score=score)
    _check_route(dev, logits, host, k, score=score, renorm=False, scale=2.5)
    _check_route(dev, logits, host, k, score=score, bias=bias, scale=0.5)
    _check_route(dev, logits, host, k, score=score, bias=bias, renorm=False)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,G,KG,GT,k", [(256, 8, 4, 2, 8), (160, 8, 3, 1, 6), (64, 8, 1, 2, 8), (64, 32, 5, 2, 6),
                                         (60, 5, 2, 2, 7), (60, 3, 2, 1, 8), (32, 32, 4, 1, 4), (512, 16, 16, 2, 8),
                                         (96, 2, 1, 2, 8), (1024, 4, 2, 2, 8), (8, 4, 2, 2, 4), (320, 10, 3, 2, 10),
                                         (1020, 17, 5, 2, 8), (990, 30, 10, 1, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_groups(dev, E, G, KG, GT, k, dtype, score, biased):
    rng = np.random.default_rng(E + G + KG)
    logits, host = _logits(rng, 61, E, dtype, dev)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32) if biased else None
    _check_route(dev, logits, host, k, score=score, bias=bias, n_group=G, topk_group=KG, group_top=GT)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G,KG", [(1, 1), (4, 2)])
@pytest.mark.parametrize("biased", [False, True])
def test_route_masks_and_special_logits(dev, score, G, KG, biased):
    """Rows that a mask empties or nearly empties, masks of -inf, of NaN and of
    the type's lowest value, +inf, and experts barred by their bias."""
    E, k = 64, 6
    rng = np.random.default_rng(3)
    l = (1.5 * rng.standard_normal((12, E))).astype(np.float32)
    l[0] = -np.inf
    l[1] = np.nan
    l[2, 5:] = -np.inf
    l[3, :-1] = np.nan
    l[4] = np.finfo(np.float32).min
    l[5, 2:] = np.finfo(np.float32).min
    l[6, ::3] = -np.inf
    l[7, 40] = np.inf
    l[8, 16:] = -np.inf             # only the first group of four has experts left
    l[9, ::2] = np.nan
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32) if biased else None
    if biased:
        bias[[1, 17, 33]] = -np.inf
        bias[2] = np.nan
    for renorm in (True, False):
        _check_route(dev, torch.from_numpy(l).to(dev), l.astype(np.float64), k, score=score, bias=bias, n_group=G,
                     topk_group=KG, group_top=2, renorm=renorm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("G,KG", [(1, 1), (8, 4), (5, 2)])
def test_route_ties_go_to_the_lower_index(dev, score, biased, G, KG):
    rng = np.random.default_rng(11)
    E = 160
    l = np.round(rng.standard_normal((64, E)) * 2).astype(np.float32) / 2    # few distinct values, -0 among the zeros
    l[:8] = 0.0
    l[3, ::2] = -0.0
    bias = np.zeros(E, np.float32) if biased else None
    _check_route(dev, torch.from_numpy(l).to(dev), l.astype(np.float64), 8, score=score, bias=bias, n_group=G,
                 topk_group=KG, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G,KG", [(1, 1), (8, 2)])
def test_route_keys_closer_than_fp32(dev, score, G, KG):
    """Keys that differ by less than an FP32 evaluation of them is off: the
    choice must still be that of the exact keys."""
    rng = np.random.default_rng(12)
    E = 256
    base = (np.abs(rng.standard_normal((64, 1))) + 2.0).astype(np.float32)
    l = np.repeat(base, E, axis=1)
    ulps = rng.permuted(np.tile(np.arange(E), (64, 1)), axis=1)
    l = (l.view(np.int32) + ulps.astype(np.int32)).view(np.float32)          # all distinct, all within 256 ulp
    l[32:, ::2] -= 3.0
    for bias in (None, np.zeros(E, np.float32), np.full(E, 0.25, np.float32)):
        _check_route(dev, torch.from_numpy(l).to(dev), l.astype(np.float64), 8, score=score, bias=bias, n_group=G,
                     topk_group=KG, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,KG,GT", [(256, 1, 1, 1), (256, 8, 4, 2), (64, 8, 3, 2), (64, 4, 2, 1), (60, 5, 2, 2),
                                       (384, 8, 4, 2), (8, 1, 1, 1)])
@pytest.mark.parametrize("biased", [False, True])
def test_route_settles_single_close_comparisons(dev, score, E, G, KG, GT, biased):
    """A few keys of a row an ulp apart, next to the choice's border or inside it,
    and pairs of groups whose best keys differ by an ulp: the comparisons that FP32
    leaves open are settled by the exact keys, the others kept."""
    rng = np.random.default_rng(E + G + KG)
    T, k, size = 400, min(6, E // 2), E // G
    l = (1.5 * rng.standard_normal((T, E))).astype(np.float32)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32) if biased else None
    if biased and G > 1:
        bias[size:2 * size] = bias[:size]                 # groups 0 and 1 can be twins
    elif biased:
        bias[E // 2:] = bias[:E // 2]
    step = np.where(rng.random((T, E)) < 0.5, np.float32(np.inf), np.float32(-np.inf))
    for t in range(T):
        if G > 1 and t % 2:
            l[t, size:2 * size] = l[t, :size]
            e = rng.integers(0, size)
            l[t, size + e] = np.nextafter(l[t, e], step[t, e])
        else:
            for e in rng.choice(E // 2, min(4, E // 2), replace=False):   # e and e + E/2, an ulp apart or equal
                l[t, e + E // 2] = np.nextafter(l[t, e], step[t, e]) if rng.random() < 0.8 else l[t, e]
            order = np.argsort(-l[t, :E // 2])
            e = order[min(k // 2, E // 2 - 1)]
            l[t, e + E // 2] = np.nextafter(l[t, e], step[t, e])
    for renorm in (True, False):
        _check_route(dev, torch.from_numpy(l).to(dev), l.astype(np.float64), k, score=score, bias=bias, n_group=G,
                     topk_group=KG, group_top=GT, renorm=renorm)


def test_route_settles_keys_of_different_experts_with_different_biases(dev):
    """p_i + b_i and p_j + b_j equal to FP32's last digits for unequal logits and
    biases, at the border of the choice."""
    rng = np.random.default_rng(31)
    T, E, k = 600, 128, 8
    l = (1.5 * rng.standard_normal((T, E))).astype(np.float32)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    for t in range(T):
        key = 1 / (1 + np.exp(-l[t].astype(np.float64))) + bias
        order = np.argsort(-key)
        for place in (k - 1, 2):                           # the last that counts, and one inside
            i, j = order[place], order[rng.integers(40, E)]
            p = key[i] - bias[j]
            if 0.01 < p < 0.99:
                l[t, j] = np.float32(np.log(p / (1 - p)))
    _check_route(dev, torch.from_numpy(l).to(dev), l.astype(np.float64), k, score="sigmoid", bias=bias)


@pytest.mark.parametrize("l0", [-120.0, -80.0, 60.0])
def test_route_sigmoid_ratios_survive_underflow(dev, l0):
    rng = np.random.default_rng(13)
    l = (l0 + rng.standard_normal((9, 32))).astype(np.float32)
    ids, w = _check_route(dev, torch.from_numpy(l).to(dev), l.astype(np.float64), 4, score="sigmoid")
    assert torch.allclose(w.sum(1), torch.ones(9, device=dev), rtol=1e-5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (70, 60, 4), (33, 256, 8), (129, 7, 7), (10, 1024, 32), (64, 160, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient(dev, T, E, k, dtype, score, renorm):
    rng = np.random.default_rng(T + E + k)
    logits, host = _logits(rng, T, E, dtype, dev)
    host = host.copy()
    if E > k and T > 4:
        logits[2, 0] = float("-inf")
        host[2, 0] = -np.inf
    ids, _ = moe.route(host, k, score=score)
    if T > 8:
        ids[3, 0] = -1            # a place without an expert
        ids[4, :] = -1
        ids[5, -1] = ids[5, 0]    # an id twice (k == 1: the same entry)
        ids[6, 0] = E + 7         # outside the experts
        ids[7, 0] = 0 if E > k else ids[7, 0]
    g = rng.standard_normal((T, k)).astype(np.float32)
    dl = fq.fp8_moe_route_bwd(logits, torch.from_numpy(ids).to(dev), torch.from_numpy(g).to(dev), score=score,
                              renorm=renorm, scale=1.5)
    torch.cuda.synchronize(dev)
    ref, mag = moe.route_bwd(host, ids, g, score=score, renorm=renorm, scale=1.5)
    tol = 2 * (2 * _spread(host, score) + 64) * U * mag + TINY
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert dl.dtype == dtype
    assert np.all(np.abs(dl.double().cpu().numpy() - ref) <= tol)


def test_route_gradient_of_empty_rows_is_zero(dev):
    l = torch.full((3, 16), float("-inf"), device=dev)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            ids, w = fq.fp8_moe_route(l, 4, score=score, renorm=renorm)
            assert torch.all(ids == -1) and torch.all(w == 0)
            out = torch.full_like(l, 7.0)
            fq.fp8_moe_route_bwd(l, ids, torch.ones_like(w), score=score, renorm=renorm, dlogits=out)
            assert torch.all(out == 0)


def _ids(rng, T, E, k, idle=0.1):
    """Distinct experts per token (repeated ones where k > E), unevenly popular, some tokens without any."""
    pop = rng.standard_normal(E) * 1.5
    ids = np.argsort(-(pop + rng.gumbel(size=(T, E))), axis=1)[:, :k].astype(np.int32)
    if k > E:
        ids = rng.integers(0, E, (T, k)).astype(np.int32)
    ids[rng.random((T, k)) < idle] = -1
    return ids


LAYOUTS = [(0, 8, 2), (1, 1, 1), (1, 32, 8), (5, 3, 2), (128, 1, 1), (129, 2, 1), (1000, 32, 8), (4097, 7, 3),
           (513, 1024, 2), (3000, 256, 8), (40, 4, 32), (2048, 60, 5), (4096, 32, 8), (4097, 32, 8),
           (32769, 1024, 1), (9000, 300, 6)]


@pytest.mark.parametrize("T,E,k", LAYOUTS)
def test_layouts(dev, T, E, k):
    rng = np.random.default_rng(T + E + k)
    ids = _ids(rng, T, E, k) if T else np.zeros((0, k), np.int32)
    if T > 3:
        ids[2, 0] = E             # just outside
        ids[3, 0] = -(1 << 31)
    t = torch.from_numpy(ids).to(dev)
    slots, m, counts = fq.fp8_moe_layout_contiguous(t, E)
    os_, om, oc = moe.layout_contiguous(ids, E)
    assert np.array_equal(slots.cpu().numpy(), os_) and np.array_equal(m.cpu().numpy(), om)
    assert np.array_equal(counts.cpu().numpy(), oc)
    for cap in (128, 256):
        slots, mm = fq.fp8_moe_layout_masked(t, E, cap)
        os_, om = moe.layout_masked(ids, E, cap)
        assert np.array_equal(slots.cpu().numpy(), os_) and np.array_equal(mm.cpu().numpy(), om)


def test_layout_of_many_entries(dev):
    """More entries than one wave of CTAs, one expert holding most of them."""
    rng = np.random.default_rng(1)
    ids = np.where(rng.random((40000, 8)) < 0.7, 3, rng.integers(0, 200, (40000, 8))).astype(np.int32)
    t = torch.from_numpy(ids).to(dev)
    for _ in range(2):   # the same layout every time
        slots, m, counts = fq.fp8_moe_layout_contiguous(t, 200)
        os_, om, oc = moe.layout_contiguous(ids, 200)
        assert np.array_equal(slots.cpu().numpy(), os_) and np.array_equal(m.cpu().numpy(), om)
        assert np.array_equal(counts.cpu().numpy(), oc)


@pytest.mark.parametrize("T,k,E", [(606208, 1, 40), (606209, 1, 1), (75777, 8, 1024), (200001, 8, 33)])
def test_layout_of_more_entries_than_a_chunk_an_sm(dev, T, k, E):
    """From 148 chunks of 4096 entries on the chunks grow; the last may be short or empty."""
    rng = np.random.default_rng(T)
    ids = rng.integers(-1, E, (T, k)).astype(np.int32)
    t = torch.from_numpy(ids).to(dev)
    slots, m, counts = fq.fp8_moe_layout_contiguous(t, E)
    os_, om, oc = moe.layout_contiguous(ids, E)
    assert np.array_equal(slots.cpu().numpy(), os_) and np.array_equal(m.cpu().numpy(), om)
    assert np.array_equal(counts.cpu().numpy(), oc)
    cap = (T * k // (E + 1)) // 128 * 128 + 128
    slots, mm = fq.fp8_moe_layout_masked(t, E, cap)
    os_, om = moe.layout_masked(ids, E, cap)
    assert np.array_equal(slots.cpu().numpy(), os_) and np.array_equal(mm.cpu().numpy(), om)


def test_large_layout_on_another_stream(dev):
    """The workspace of a large layout belongs to the stream the call names: two
    streams at once, each with its own entries, repeated."""
    rng = np.random.default_rng(4)
    hosts = [_ids(rng, 6000, 64, 8), _ids(rng, 7000, 64, 8)]
    devs = [torch.from_numpy(h).to(dev) for h in hosts]
    side = torch.cuda.Stream(dev)
    torch.cuda.synchronize(dev)
    got = []
    for _ in range(8):
        got.append([fq.fp8_moe_layout_contiguous(devs[0], 64), fq.fp8_moe_layout_contiguous(devs[1], 64, stream=side)])
    torch.cuda.synchronize(dev)
    for pair in got:
        for host, (slots, m, counts) in zip(hosts, pair):
            os_, om, oc = moe.layout_contiguous(host, 64)
            assert np.array_equal(slots.cpu().numpy(), os_) and np.array_equal(m.cpu().numpy(), om)
            assert np.array_equal(counts.cpu().numpy(), oc)


def _bf16(rng, shape, scale=1.0):
    return moe.f32_to_bf16((scale * rng.standard_normal(shape)).astype(np.float32))


@pytest.mark.parametrize("T,E,k,D", [(1, 8, 2, 128), (1, 32, 8, 7168), (61, 32, 8, 1152), (300, 5, 3, 256), (7, 4, 1, 384),
                                     (130, 64, 32, 128)])
@pytest.mark.parametrize("layout", ["contiguous", "masked"])
def test_dispatch(dev, T, E, k, D, layout):
    rng = np.random.default_rng(T + D)
    x = _bf16(rng, (T, D), 3.0)
    x[0, :128] = 0
    ids = _ids(rng, T, E, k)
    t = torch.from_numpy(ids).to(dev)
    if layout == "contiguous":
        slots, m, counts = fq.fp8_moe_layout_contiguous(t, E)
        rows, pads = m.numel() * 128, dict(m_indices=m, counts=counts)
        osl, om, oc = moe.layout_contiguous(ids, E)
        pad = moe.pad_rows(om, oc)
    else:
        slots, _ = fq.fp8_moe_layout_masked(t, E, 128)
        rows, pads = E * 128, {}
        osl = moe.layout_masked(ids, E, 128)[0]
        pad = np.zeros(rows, dtype=bool)
    q = torch.full((rows, D), 0x5A, dtype=torch.uint8, device=dev)
    s = torch.full((rows, D // 128), -3.0, device=dev)
    fq.fp8_moe_dispatch_1x128(to_torch_bf16(x, dev), slots, rows, q=q, s=s, **pads)
    torch.cuda.synchronize(dev)
    oq, os_ = oracle.quant_act_1x128(x)
    eq, es = np.full((rows, D), 0x5A, np.uint8), np.full((rows, D // 128), -3.0, np.float32)
    eq[pad], es[pad] = 0, 1.0
    tok, j = np.nonzero(osl >= 0)
    eq[osl[tok, j]], es[osl[tok, j]] = oq[tok], os_[tok]
    assert np.array_equal(q.cpu().numpy(), eq)                    # rows behind the last entry as they were
    assert np.array_equal(s.cpu().numpy(), es)


def test_dispatch_skips_slots_outside_the_rows(dev):
    rng = np.random.default_rng(2)
    x = to_torch_bf16(_bf16(rng, (4, 256)), dev)
    slots = torch.tensor([[0, 128], [1 << 30, -5], [127, -1], [-(1 << 31), 64]], dtype=torch.int32, device=dev)
    q, s = torch.zeros((128, 256), dtype=torch.uint8, device=dev), torch.zeros((128, 2), device=dev)
    fq.fp8_moe_dispatch_1x128(x, slots, 128, q=q, s=s)
    assert torch.nonzero(s[:, 0]).flatten().tolist() == [0, 64, 127]


@pytest.mark.parametrize("T,E,k,D", [(1, 8, 2, 128), (1, 32, 8, 7168), (61, 32, 8, 1152), (300, 5, 3, 256), (130, 64, 32, 128),
                                     (9, 4, 1, 384)])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("layout", ["contiguous", "masked"])
def test_combine(dev, T, E, k, D, weighted, layout):
    rng = np.random.default_rng(T + D)
    ids = _ids(rng, T, E, k)
    slots = moe.layout_contiguous(ids, E)[0] if layout == "contiguous" else moe.layout_masked(ids, E, 128)[0]
    rows = len(moe.layout_contiguous(ids, E)[1]) * 128 if layout == "contiguous" else E * 128
    y = _bf16(rng, (rows, D))
    used = np.zeros(rows, dtype=bool)
    used[slots[slots >= 0]] = True
    y[~used] = 0x7FC0                                              # NaN in rows that no entry names
    w = rng.random((T, k)).astype(np.float32)
    w[slots < 0] = np.nan                                          # and in weights without a row
    yt = to_torch_bf16(y, dev)
    out = fq.fp8_moe_combine(yt.view(E, 128, D) if layout == "masked" else yt, torch.from_numpy(slots).to(dev),
                             torch.from_numpy(w).to(dev) if weighted else None)
    torch.cuda.synchronize(dev)
    ref, mag = moe.combine(moe.bf16_to_f32(y).astype(np.float64), slots, w if weighted else None)
    err = np.abs(moe.bf16_to_f32(bf16_bits_of(out)).astype(np.float64) - ref)
    acc = k * U * mag
    assert np.all(err <= acc + 2.0 ** -8 * (np.abs(ref) + acc) + TINY)
    assert np.all(bf16_bits_of(out)[(slots < 0).all(axis=1)] == 0)


def test_combine_of_no_rows_is_zero(dev):
    out = fq.fp8_moe_combine(torch.empty((0, 256), dtype=torch.bfloat16, device=dev),
                             torch.full((3, 2), -1, dtype=torch.int32, device=dev))
    assert torch.all(out == 0)


@pytest.mark.parametrize("T,E,k,D", [(1, 8, 2, 128), (3, 32, 8, 7168), (61, 32, 8, 1152), (300, 5, 3, 256), (130, 64, 32, 128),
                                     (9, 4, 1, 2176), (40, 16, 9, 4224)])
@pytest.mark.parametrize("layout", ["contiguous", "masked"])
def test_combine_gradient(dev, T, E, k, D, layout):
    rng = np.random.default_rng(T + D)
    ids = _ids(rng, T, E, k)
    if layout == "contiguous":
        slots, m, c = moe.layout_contiguous(ids, E)
        rows, pad = len(m) * 128, moe.pad_rows(m, c)
        pads = dict(m_indices=torch.from_numpy(m).to(dev), counts=torch.from_numpy(c).to(dev))
    else:
        slots, _ = moe.layout_masked(ids, E, 128)
        rows, pads = E * 128, {}
        pad = np.zeros(rows, dtype=bool)
    y, do = _bf16(rng, (rows, D)), _bf16(rng, (T, D))
    w = rng.random((T, k)).astype(np.float32)
    dy = torch.full((rows, D), -7.0, dtype=torch.bfloat16, device=dev)
    _, dw = fq.fp8_moe_combine_bwd(to_torch_bf16(do, dev), to_torch_bf16(y, dev), torch.from_numpy(slots).to(dev),
                                   torch.from_numpy(w).to(dev), dy=dy, **pads)
    torch.cuda.synchronize(dev)
    do32 = moe.bf16_to_f32(do)
    ref = np.full((rows, D), moe.f32_to_bf16(np.float32([-7.0]))[0], np.uint16)
    ref[pad] = 0
    tok, j = np.nonzero(slots >= 0)
    ref[slots[tok, j]] = moe.f32_to_bf16(do32[tok] * w[tok, j][:, None])   # one FP32 product, one rounding
    assert np.array_equal(bf16_bits_of(dy), ref)
    rw, mag = moe.combine_dweights(do32.astype(np.float64), moe.bf16_to_f32(y).astype(np.float64), slots)
    # at most D / 128 products in one thread's chain or one lane's, and 16 additions joining them
    assert np.all(np.abs(dw.cpu().numpy() - rw) <= (D // 128 + 16 + 8) * U * mag + TINY)
    assert np.all(dw.cpu().numpy()[slots < 0] == 0)


def test_streams_and_graph_replay(dev):
    """The serving calls on a side stream, and captured once and replayed on new
    tokens: no host step, the layout recomputed on the device each time."""
    rng = np.random.default_rng(21)
    T, E, k, D, cap = 33, 16, 4, 256, 128
    logits = torch.zeros((T, E), device=dev)
    x = torch.zeros((T, D), dtype=torch.bfloat16, device=dev)
    q, s = torch.zeros((E * cap, D), dtype=torch.uint8, device=dev), torch.zeros((E * cap, D // 128), device=dev)
    y = torch.zeros((E * cap, D), dtype=torch.bfloat16, device=dev)
    hold = {}

    def step():
        hold["ids"], hold["w"] = fq.fp8_moe_route(logits, k, score="sigmoid")
        hold["slots"], hold["m"] = fq.fp8_moe_layout_masked(hold["ids"], E, cap)
        fq.fp8_moe_dispatch_1x128(x, hold["slots"], E * cap, q=q, s=s)
        hold["out"] = fq.fp8_moe_combine(y, hold["slots"], hold["w"])

    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream(dev).wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for r in range(3):
        l = rng.standard_normal((T, E)).astype(np.float32)
        xb, yb = _bf16(rng, (T, D)), _bf16(rng, (E * cap, D))
        logits.copy_(torch.from_numpy(l))
        x.copy_(to_torch_bf16(xb, dev))
        y.copy_(to_torch_bf16(yb, dev))
        graph.replay()
        torch.cuda.synchronize(dev)
        oi, ow = moe.route(l, k, score="sigmoid")
        osl, om = moe.layout_masked(oi, E, cap)
        assert np.array_equal(hold["ids"].cpu().numpy(), oi) and np.array_equal(hold["m"].cpu().numpy(), om)
        oq, _ = oracle.quant_act_1x128(xb)
        tok, j = np.nonzero(osl >= 0)
        assert np.array_equal(q.cpu().numpy()[osl[tok, j]], oq[tok])
        ref, mag = moe.combine(moe.bf16_to_f32(yb).astype(np.float64), osl, ow)
        err = np.abs(moe.bf16_to_f32(bf16_bits_of(hold["out"])).astype(np.float64) - ref)
        assert np.all(err <= 100 * U * mag + 2.0 ** -8 * (np.abs(ref) + mag * 100 * U) + TINY)


def test_masked_layer(dev):
    """A serving layer from logits to output: route -> masked layout -> dispatch ->
    GEMM1 -> SwiGLU -> GEMM2 -> combine, captured in a graph and replayed, each step
    against the oracle on its own inputs.  One expert runs out of capacity."""
    rng = np.random.default_rng(41)
    T, E, k, D, I, cap = 200, 6, 2, 256, 128, 128
    l = rng.standard_normal((T, E)).astype(np.float32)
    l[:, 2] += 2.0                                                  # over 128 tokens choose expert 2
    x = _bf16(rng, (T, D))
    logits, xt = torch.from_numpy(l).to(dev), to_torch_bf16(x, dev)
    qw1, sw1 = fq.fp8_quant_w_128x128(to_torch_bf16(_bf16(rng, (E, 2 * I, D), 0.06), dev))
    qw2, sw2 = fq.fp8_quant_w_128x128(to_torch_bf16(_bf16(rng, (E, D, I), 0.09), dev))
    q = torch.zeros((E, cap, D), dtype=torch.uint8, device=dev)
    s = torch.ones((E, cap, D // 128), device=dev)
    c1 = torch.zeros((E, cap, 2 * I), dtype=torch.bfloat16, device=dev)
    y = torch.zeros((E, cap, D), dtype=torch.bfloat16, device=dev)
    r = {}

    def layer():
        r["ids"], r["w"] = fq.fp8_moe_route(logits, k)
        r["slots"], r["m"] = fq.fp8_moe_layout_masked(r["ids"], E, cap)
        fq.fp8_moe_dispatch_1x128(xt, r["slots"], E * cap, q=q, s=s)
        fq.fp8_grouped_gemm_masked(q, s, qw1, sw1, r["m"], out=c1)
        r["qh"], r["sh"] = fq.fp8_swiglu_quant_1x128(c1, masked_m=r["m"])
        fq.fp8_grouped_gemm_masked(r["qh"], r["sh"], qw2, sw2, r["m"], out=y)
        r["out"] = fq.fp8_moe_combine(y, r["slots"], r["w"])

    layer()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    graph.replay()
    torch.cuda.synchronize(dev)
    assert fq.get_device_error(device=dev) == fq.OK
    oi, ow = moe.route(l, k)
    osl, om = moe.layout_masked(oi, E, cap)
    assert om[2] == cap and (osl < 0).any()
    assert np.array_equal(r["slots"].cpu().numpy(), osl) and np.array_equal(r["m"].cpu().numpy(), om)
    oq, _ = oracle.quant_act_1x128(x)
    tok, j = np.nonzero(osl >= 0)
    assert np.array_equal(q.cpu().numpy().reshape(E * cap, D)[osl[tok, j]], oq[tok])
    ref1 = oracle.grouped_masked(bytes_of(q), s.cpu().numpy(), bytes_of(qw1), sw1.cpu().numpy(), om)
    ref2 = oracle.grouped_masked(bytes_of(r["qh"]), r["sh"].cpu().numpy(), bytes_of(qw2), sw2.cpu().numpy(), om)
    for e in range(E):
        m = int(om[e])
        assert_gemm_close(bf16_bits_of(c1)[e, :m], ref1[e, :m], "GEMM1")
        assert_gemm_close(bf16_bits_of(y)[e, :m], ref2[e, :m], "GEMM2")
    yf = moe.bf16_to_f32(bf16_bits_of(y)).astype(np.float64).reshape(E * cap, D)
    ref, mag = moe.combine(yf, osl, r["w"].double().cpu().numpy())
    err = np.abs(moe.bf16_to_f32(bf16_bits_of(r["out"])).astype(np.float64) - ref)
    assert np.all(err <= k * U * mag + 2.0 ** -8 * (np.abs(ref) + k * U * mag) + TINY)


def test_empty_calls(dev):
    """No tokens, no rows, no channels: nothing is launched or written, the counts
    are still set."""
    e = torch.empty((0, 16), device=dev)
    ids, w = fq.fp8_moe_route(e, 4)
    assert ids.shape == w.shape == (0, 4)
    assert fq.fp8_moe_route_bwd(e, ids, w).shape == (0, 16)
    counts = torch.full((16,), 7, dtype=torch.int32, device=dev)
    slots, m, _ = fq.fp8_moe_layout_contiguous(ids, 16, counts=counts)
    assert slots.shape == (0, 4) and m.numel() == 0 and torch.all(counts == 0)
    _, mm = fq.fp8_moe_layout_masked(ids, 16, 128)
    assert torch.all(mm == 0)
    x = torch.empty((0, 256), dtype=torch.bfloat16, device=dev)
    q, s = fq.fp8_moe_dispatch_1x128(x, slots, 0, m_indices=m, counts=counts)
    assert q.shape == (0, 256) and s.shape == (0, 2)
    keep = torch.full((128, 256), 3.0, dtype=torch.bfloat16, device=dev)
    assert fq.fp8_moe_combine(keep, slots).shape == (0, 256)
    dy, dw = fq.fp8_moe_combine_bwd(x, torch.zeros_like(keep), slots, w, dy=keep)
    assert torch.all(keep == 3.0) and dw.shape == (0, 4)
    none = torch.empty((3, 0), dtype=torch.bfloat16, device=dev)
    assert fq.fp8_moe_dispatch_1x128(none, torch.zeros((3, 1), dtype=torch.int32, device=dev), 128)[0].shape == (128, 0)
    (qh, _), (qc, _) = fq.fp8_swiglu_ckpt_1x128(torch.empty((0, 512), dtype=torch.bfloat16, device=dev))
    assert qh.shape == (0, 256) and qc.shape == (0, 512)
    dc, (qd, _) = fq.fp8_swiglu_bwd_1x128(x, torch.empty((0, 512), dtype=torch.uint8, device=dev),
                                          torch.empty((0, 4), device=dev))
    assert dc.shape == qd.shape == (0, 512)
    torch.cuda.synchronize(dev)


def test_misaligned_tensors_are_refused(dev):
    """A contiguous view that starts off the alignment raises the library's error,
    and the next call works."""
    x = torch.zeros(4 * 256 + 8, dtype=torch.bfloat16, device=dev)[8:].view(4, 256)      # 16 bytes in: 32 needed
    slots = torch.zeros((4, 2), dtype=torch.int32, device=dev)
    with pytest.raises(fq.Fp8qError) as e:
        fq.fp8_moe_dispatch_1x128(x, slots, 128)
    assert e.value.status == fq.ERR_ALIGN
    with pytest.raises(fq.Fp8qError):
        fq.fp8_moe_combine(torch.zeros(128 * 128 + 4, dtype=torch.bfloat16, device=dev)[4:].view(128, 128), slots)
    assert torch.all(fq.fp8_moe_combine(torch.zeros((128, 128), dtype=torch.bfloat16, device=dev), slots) == 0)
    with pytest.raises(ValueError, match="dy may not be y"):
        y = torch.zeros((128, 128), dtype=torch.bfloat16, device=dev)
        fq.fp8_moe_combine_bwd(torch.zeros((4, 128), dtype=torch.bfloat16, device=dev), y, slots,
                               torch.zeros((4, 2), device=dev), dy=y)


def test_results_do_not_depend_on_the_run(dev):
    rng = np.random.default_rng(22)
    T, E, k, D = 500, 32, 8, 1024
    ids = torch.from_numpy(_ids(rng, T, E, k)).to(dev)
    slots, m, c = fq.fp8_moe_layout_contiguous(ids, E)
    rows = m.numel() * 128
    y, do = to_torch_bf16(_bf16(rng, (rows, D)), dev), to_torch_bf16(_bf16(rng, (T, D)), dev)
    w = torch.rand((T, k), device=dev)
    first = None
    for _ in range(3):
        dy, dw = fq.fp8_moe_combine_bwd(do, y, slots, w, m_indices=m, counts=c, dy=torch.zeros_like(y))
        got = (bytes_of(dy), bytes_of(dw), bytes_of(fq.fp8_moe_combine(y, slots, w)))
        first = first or got
        assert all(np.array_equal(a, b) for a, b in zip(first, got))


def test_offsets_beyond_32_bits(dev):
    """Rows whose byte and element offsets pass 2^32: the last rows of large buffers get
    what the same rows give in small ones."""
    T, k, D = 40, 2, 7168
    rows = 600_064                       # rows * D > 2^32
    assert (rows - 128) * D > 1 << 32
    rng = np.random.default_rng(5)
    slots = torch.from_numpy(rng.permutation(T * k).astype(np.int32).reshape(T, k)).to(dev)   # in the last 128 rows
    far = slots + (rows - 128)
    x = torch.randn((T, D), dtype=torch.bfloat16, device=dev)
    q, s = torch.zeros((rows, D), dtype=torch.uint8, device=dev), torch.zeros((rows, D // 128), device=dev)
    fq.fp8_moe_dispatch_1x128(x, far, rows, q=q, s=s)
    qn, sn = torch.zeros((128, D), dtype=torch.uint8, device=dev), torch.zeros((128, D // 128), device=dev)
    fq.fp8_moe_dispatch_1x128(x, slots, 128, q=qn, s=sn)
    assert torch.equal(q[-128:], qn) and torch.equal(s[-128:], sn)
    assert int(q[:-128].count_nonzero()) == 0 and int(s[:-128].count_nonzero()) == 0
    del q, s
    y = torch.zeros((rows, D), dtype=torch.bfloat16, device=dev)
    y[-128:] = torch.randn((128, D), dtype=torch.bfloat16, device=dev)
    w = torch.rand((T, k), device=dev)
    assert torch.equal(fq.fp8_moe_combine(y, far, w), fq.fp8_moe_combine(y[-128:], slots, w))
    dy, dyn = torch.zeros_like(y), torch.zeros((128, D), dtype=torch.bfloat16, device=dev)
    _, dw = fq.fp8_moe_combine_bwd(x, y, far, w, dy=dy)
    _, dwn = fq.fp8_moe_combine_bwd(x, y[-128:], slots, w, dy=dyn)
    assert torch.equal(dw, dwn) and torch.equal(dy[-128:], dyn) and int(dy[:-128].count_nonzero()) == 0


def test_logits_beyond_32_bits(dev):
    """T * E passes 2^32: the last rows' choice, weights and gradients."""
    E, k = 1024, 8
    T = (1 << 22) + 300
    logits = torch.zeros((T, E), dtype=torch.bfloat16, device=dev)
    logits[-300:] = torch.randn((300, E), dtype=torch.bfloat16, device=dev)
    ids, w = fq.fp8_moe_route(logits, k)
    ids0, w0 = fq.fp8_moe_route(logits[-300:], k)
    assert torch.equal(ids[-300:], ids0) and torch.equal(w[-300:], w0)
    assert bool((ids[:-300] == torch.arange(k, dtype=torch.int32, device=dev)).all())   # ties: the lower index
    g = torch.randn((T, k), device=dev)
    d = fq.fp8_moe_route_bwd(logits, ids, g, renorm=False)
    assert torch.equal(d[-300:], fq.fp8_moe_route_bwd(logits[-300:], ids0, g[-300:], renorm=False))
