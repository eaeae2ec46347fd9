"""CPU pins of the routing, layout, combine and checkpoint oracle (none retypes
the oracle's own formulas): hand-worked cases, finite differences, library
softmax, and the existing C oracle's quantizers."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl
from oracle import moe


def test_route_hand_case():
    l = np.array([[0.0, 3.0, 1.0, 2.0]])
    ids, w = moe.route(l, 2)
    assert ids.tolist() == [[1, 3]]
    assert np.allclose(w, [[1 / (1 + np.exp(-1.0)), 1 / (1 + np.exp(1.0))]], rtol=1e-14)
    ids, w = moe.route(l, 2, renorm=False, scale=2.0)
    assert np.allclose(w[0], 2.0 * torch.softmax(torch.tensor(l), 1).numpy()[0, [1, 3]], rtol=1e-14)
    # the bias moves the choice (expert 0 first), not the weights
    ids, w = moe.route(l, 2, bias=[5.0, 0, 0, 0], score="sigmoid", renorm=False)
    assert ids.tolist() == [[0, 1]]
    assert np.allclose(w[0], torch.sigmoid(torch.tensor([0.0, 3.0], dtype=torch.float64)).numpy(), rtol=1e-14)


def test_route_groups_ties_and_masks():
    # groups {0,1} {2,3} {4,5}: best pair sums 4, 5, 5 -> with two groups kept, group 1 before group 2, then both
    key = np.array([[3.0, 1.0, 5.0, 0.0, 2.5, 2.5]])
    ids, _ = moe.route(np.zeros((1, 6)), 2, bias=key[0], score="sigmoid", n_group=3, topk_group=1, group_top=2)
    assert ids.tolist() == [[2, 3]]
    ids, _ = moe.route(np.zeros((1, 6)), 3, bias=key[0], score="sigmoid", n_group=3, topk_group=2, group_top=2)
    assert ids.tolist() == [[2, 4, 5]]
    ids, w = moe.route(np.full((1, 6), -np.inf), 2)
    assert ids.tolist() == [[-1, -1]] and np.all(w == 0)
    ids, w = moe.route(np.array([[np.nan, -np.inf, 0.0]]), 2)
    assert ids.tolist() == [[2, -1]] and w.tolist() == [[1.0, 0.0]]
    ids, _ = moe.route(np.array([[1.0, 1.0, 1.0]]), 3)
    assert ids.tolist() == [[0, 1, 2]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(5)
    l = rng.standard_normal((3, 7))
    ids, _ = moe.route(l, 3, score=score, renorm=renorm, scale=1.5)
    g = rng.standard_normal((3, 3))

    def loss(x):   # the choice held at `ids`
        x = torch.tensor(x)
        p = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)
        w = torch.gather(p, 1, torch.tensor(ids.astype(np.int64)))
        if renorm:
            w = w / w.sum(1, keepdim=True)
        return float((1.5 * w * torch.tensor(g)).sum())

    got, mag = moe.route_bwd(l, ids, g, score=score, renorm=renorm, scale=1.5)
    h = 1e-6
    for t in range(3):
        for e in range(7):
            a, b = l.copy(), l.copy()
            a[t, e] += h
            b[t, e] -= h
            # central differences: h^2/6 |f'''| + eps |f| / h, below 1e-9 for these O(1) values
            assert abs((loss(a) - loss(b)) / (2 * h) - got[t, e]) < 1e-8
    assert np.all(mag >= np.abs(got) * (1 - 1e-12))


def test_route_gradient_of_a_repeated_id_is_the_sum():
    l = np.array([[0.3, -0.4, 1.0]])
    one, _ = moe.route_bwd(l, np.array([[2, -1]]), np.array([[1.25, 9.0]]), score="sigmoid", renorm=False)
    two, _ = moe.route_bwd(l, np.array([[2, 2]]), np.array([[1.0, 0.25]]), score="sigmoid", renorm=False)
    assert np.allclose(one, two, rtol=1e-15) and one[0, 0] == 0


def test_layouts_hand_case():
    ids = np.array([[2, 0], [2, -1], [0, 5], [2, 0]], dtype=np.int32)   # 5 is no expert of 3
    slots, m, counts = moe.layout_contiguous(ids, 3)
    assert counts.tolist() == [3, 0, 3]
    assert slots.tolist() == [[128, 0], [129, -1], [1, -1], [130, 2]]
    assert m.tolist() == [0, 2, -1]            # (8 + 127 * 3) // 128 blocks
    pad = moe.pad_rows(m, counts)
    assert np.flatnonzero(~pad).tolist() == [0, 1, 2, 128, 129, 130] + list(range(256, 384))
    slots, mm = moe.layout_masked(np.full((130, 1), 1), 2, 128)
    assert mm.tolist() == [0, 128] and slots[127, 0] == 255 and slots[128:, 0].tolist() == [-1, -1]


def test_block_bound_is_reached_and_never_passed():
    for n, E in [(1, 1), (5, 9), (128, 1), (129, 1), (1000, 4), (4096 * 8, 32), (7, 3)]:
        B = (n + 127 * min(n, E)) // 128
        m = min(n, E)
        worst = np.ones(m, dtype=int)          # one entry each, the rest stacked so that every remainder is 1
        worst[0] += n - m
        assert sum(-(-c // 128) for c in worst) <= B
        rng = np.random.default_rng(n)
        for _ in range(50):
            c = rng.multinomial(n, np.full(E, 1 / E))
            assert sum(-(-v // 128) for v in c) <= B


def test_combine_and_its_gradient():
    rng = np.random.default_rng(2)
    y, w, do = rng.standard_normal((5, 4)), rng.random((2, 3)), rng.standard_normal((2, 4))
    slots = np.array([[4, 0, -1], [2, 99, 3]])
    out, _ = moe.combine(y, slots, w)
    assert np.allclose(out[0], w[0, 0] * y[4] + w[0, 1] * y[0]) and np.allclose(out[1], w[1, 0] * y[2] + w[1, 2] * y[3])
    dw, _ = moe.combine_dweights(do, y, slots)
    for t in range(2):
        for j in range(3):
            a = w.copy()
            a[t, j] += 1.0                       # linear in w: the difference is the derivative
            assert abs(((moe.combine(y, slots, a)[0] - out) * do).sum() - dw[t, j]) < 1e-12


def test_f32_quantization_equals_the_bf16_oracle_on_bf16_values():
    rng = np.random.default_rng(8)
    bits = wl.bf16_bits((rng.standard_normal((6, 384)) * 3).astype(np.float32))
    oq, os_ = oracle.quant_act_1x128(bits)
    q, s = moe.quant_f32(moe.bf16_to_f32(bits).reshape(6, 3, 128))
    assert np.array_equal(q.reshape(6, 384), oq) and np.array_equal(s, os_)


def test_regrouping_exact_values_equals_the_token_axis_oracle():
    """Where every 1x128 tile has scale 1 the checkpoint holds E4M3 values, which
    bf16 holds too: regrouping must equal the token-axis oracle of those values."""
    rng = np.random.default_rng(9)
    q = rng.integers(0, 0x7F, (300, 128)).astype(np.uint8) | (rng.integers(0, 2, (300, 128)) << 7).astype(np.uint8)
    v = oracle.e4m3_decode_table()[q]
    qt, st = moe.ckpt_128x1_t(q, np.ones((300, 1), np.float32), 512)
    oq, os_ = oracle.quant_act_128x1(wl.bf16_bits(v.astype(np.float32)))
    assert np.array_equal(qt[:, :300], oq.T) and np.all(qt[:, 300:] == 0)
    assert np.array_equal(st[:3], os_) and np.all(st[3:] == 1)


def test_swiglu_gradient_against_differences():
    rng = np.random.default_rng(4)
    q = rng.integers(0, 0x40, (2, 256)).astype(np.uint8) | (rng.integers(0, 2, (2, 256)) << 7).astype(np.uint8)
    s = np.full((2, 2), 0.75, np.float32)
    dh = rng.standard_normal((2, 128))
    d, mag = moe.swiglu_bwd(dh, q, s)
    v = moe.dequant_1x128(q, s).astype(np.float64)

    def f(x):
        g, u = torch.tensor(x[:, :128]), torch.tensor(x[:, 128:])
        return float((torch.nn.functional.silu(g) * u * torch.tensor(dh)).sum())

    h = 1e-5
    for at in [(0, 0), (0, 127), (0, 128), (1, 40), (1, 255)]:
        a, b = v.copy(), v.copy()
        a[at] += h
        b[at] -= h
        assert abs((f(a) - f(b)) / (2 * h) - d[at]) < 1e-8 * (1 + abs(f(v)))
    assert np.all(mag >= np.abs(d) * (1 - 1e-12))


def test_bf16_rounding_helper():
    v = np.array([1.0, 1.00390625, 1.01171875, -2.5e-3, 3e38], dtype=np.float32)   # two ties among them
    assert np.array_equal(moe.f32_to_bf16(v), torch.tensor(v).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16))
