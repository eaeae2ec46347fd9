"""Calls that name a stream other than the current one: what they allocate belongs
to that stream, so that no work queued on the current stream can still use it, and
outputs outlive the current stream's work on them."""
import numpy as np
import pytest
import torch

import fp8_fine_grained_quant_b200 as fq
from oracle import moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


@pytest.fixture
def side(dev):
    torch.cuda.synchronize(dev)
    return torch.cuda.Stream(dev)


def _busy(dev, n=40):
    """Queues some tens of milliseconds of products on the current stream."""
    a = torch.ones((8192, 8192), dtype=torch.bfloat16, device=dev)
    b = torch.empty_like(a)
    torch.mm(a, a, out=b)
    for _ in range(n):
        torch.mm(a, a, out=b)
    return a, b


def _stream_of(t):
    """The stream whose pool holds t."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no segment holds the tensor")


def _moe_calls(dev):
    """name -> call(stream): every call marshalled in C++, with fresh outputs."""
    T, E, k, D, I = 64, 16, 4, 256, 256
    g = torch.Generator(device=dev).manual_seed(3)
    logits = torch.randn((T, E), generator=g, device=dev)
    x = torch.randn((T, D), generator=g, device=dev).bfloat16()
    ids, w = fq.fp8_moe_route(logits, k)
    slots, m, counts = fq.fp8_moe_layout_contiguous(ids, E)
    rows = m.numel() * 128
    y = torch.randn((rows, D), generator=g, device=dev).bfloat16()
    c1 = torch.randn((T, 2 * I), generator=g, device=dev).bfloat16()
    (_, _), (qc, sc) = fq.fp8_swiglu_ckpt_1x128(c1)
    dh = torch.randn((T, I), generator=g, device=dev).bfloat16()
    torch.cuda.synchronize(dev)
    return {
        "route": lambda s: fq.fp8_moe_route(logits, k, stream=s),
        "route_bwd": lambda s: [fq.fp8_moe_route_bwd(logits, ids, w, stream=s)],
        "layout_contiguous": lambda s: fq.fp8_moe_layout_contiguous(ids, E, stream=s),
        "layout_masked": lambda s: fq.fp8_moe_layout_masked(ids, E, 128, stream=s),
        "dispatch": lambda s: fq.fp8_moe_dispatch_1x128(x, slots, rows, stream=s),
        "combine": lambda s: [fq.fp8_moe_combine(y, slots, w, stream=s)],
        "combine_bwd": lambda s: fq.fp8_moe_combine_bwd(x, y, slots, w, m_indices=m, counts=counts, stream=s),
        "swiglu_ckpt": lambda s: [t for p in fq.fp8_swiglu_ckpt_1x128(c1, stream=s) for t in p],
        "swiglu_bwd": lambda s: (lambda r: [r[0], *r[1]])(fq.fp8_swiglu_bwd_1x128(dh, qc, sc, stream=s)),
        "ckpt_128x1_t": lambda s: fq.fp8_ckpt_128x1_t(qc, sc, stream=s),
    }


@pytest.mark.parametrize("how", ["stream", "handle"])
def test_outputs_belong_to_the_named_stream(dev, side, how):
    for name, call in _moe_calls(dev).items():
        mine = call(None)
        torch.cuda.synchronize(dev)
        theirs = call(side if how == "stream" else side.cuda_stream)
        torch.cuda.synchronize(dev)
        for a, b in zip(mine, theirs):
            assert _stream_of(a) == 0, name
            assert _stream_of(b) == side.cuda_stream, name
        if name not in ("dispatch", "combine_bwd"):            # those leave rows unwritten
            for a, b in zip(mine, theirs):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name


def test_naming_the_current_stream_changes_nothing(dev, side):
    calls = _moe_calls(dev)
    for stream in (0, 1, torch.cuda.default_stream(dev)):       # 1: the legacy default stream's own handle
        for name, call in calls.items():
            assert all(_stream_of(t) == 0 for t in call(stream)), name
    with torch.cuda.stream(side):
        for name, call in calls.items():
            assert all(_stream_of(t) == side.cuda_stream for t in call(side)), name
            assert all(_stream_of(t) == 0 for t in call(0)), name
            assert all(_stream_of(t) == 0 for t in call(1)), name
    torch.cuda.synchronize(dev)


@pytest.mark.parametrize("layout", ["contiguous", "masked"])
def test_workspace_belongs_to_the_named_stream(dev, side, layout):
    T, E, k = 6000, 64, 8
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, device=dev)
    n = fq.lib().fp8_moe_layout_workspace(T, k, E) * 4
    assert n > 0
    slots, counts = torch.empty_like(ids), torch.empty(E, dtype=torch.int32, device=dev)
    m = torch.empty(fq.moe_contiguous_blocks(T, k, E), dtype=torch.int32, device=dev)

    def sizes():
        out = {}
        for seg in torch.cuda.memory_snapshot():
            out[seg["stream"]] = out.get(seg["stream"], 0) + seg["total_size"]
        return out

    torch.cuda.synchronize(dev)
    torch.cuda.empty_cache()
    before = sizes()
    assert side.cuda_stream not in before
    if layout == "contiguous":
        fq.fp8_moe_layout_contiguous(ids, E, slots=slots, m_indices=m, counts=counts, stream=side)
    else:
        fq.fp8_moe_layout_masked(ids, E, 1024, slots=slots, masked_m=counts, stream=side)
    after = sizes()
    assert after.pop(side.cuda_stream) >= n
    assert after == before
    torch.cuda.synchronize(dev)
    ref = moe.layout_contiguous(ids.cpu().numpy(), E) if layout == "contiguous" else \
        moe.layout_masked(ids.cpu().numpy(), E, 1024)
    assert np.array_equal(slots.cpu().numpy(), ref[0]) and np.array_equal(counts.cpu().numpy(), ref[-1])


def test_layouts_on_two_streams_behind_other_work(dev, side):
    """Equal sizes, so that a shared pool would give both the same workspace."""
    rng = np.random.default_rng(4)
    hosts = [rng.integers(0, 64, (6000, 8)).astype(np.int32) for _ in range(2)]
    devs = [torch.from_numpy(h).to(dev) for h in hosts]
    torch.cuda.synchronize(dev)
    got, hold = [], []
    for _ in range(3):
        hold.append(_busy(dev, 5))
        for _ in range(4):
            got.append([fq.fp8_moe_layout_contiguous(devs[0], 64),
                        fq.fp8_moe_layout_contiguous(devs[1], 64, stream=side)])
    torch.cuda.synchronize(dev)
    refs = [moe.layout_contiguous(h, 64) for h in hosts]
    for pair in got:
        for ref, out in zip(refs, pair):
            assert all(np.array_equal(a, b.cpu().numpy()) for a, b in zip(ref, out))


def _freed_block_is_left_alone(dev, call):
    """Memory that the current stream has freed, with a copy of it still queued, is
    not written by the call on another stream."""
    sizes = {t.untyped_storage().nbytes() for t in call(None)}
    torch.cuda.synchronize(dev)
    torch.cuda.empty_cache()
    old = [torch.full((n,), 5, dtype=torch.uint8, device=dev) for n in sizes]
    new = [torch.empty_like(t) for t in old]
    hold = _busy(dev)
    for a, b in zip(old, new):
        b.copy_(a)
    del old, a
    out = call(torch.cuda.Stream(dev))
    torch.cuda.synchronize(dev)
    assert all(bool((t == 5).all()) for t in new)
    del hold, out


def _output_outlives_queued_work(dev, side, first, second):
    """An output dropped while the current stream still reads it is not given to the
    named stream's next call."""
    with torch.cuda.stream(side):
        want = [t.clone() for t in first(None)]
    torch.cuda.synchronize(dev)
    out = first(side)
    torch.cuda.current_stream(dev).wait_stream(side)
    got = [torch.empty_like(t) for t in out]
    hold = _busy(dev)
    for a, b in zip(out, got):
        b.copy_(a)
    del out, a
    again = second(side)
    torch.cuda.synchronize(dev)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(want, got))
    del hold, again


def test_memory_of_other_streams_is_left_alone(dev, side):
    T, E = 8192, 256
    l1, l2 = torch.randn((T, E), device=dev), torch.randn((T, E), device=dev)
    c1 = torch.randn((2048, 1024), device=dev).bfloat16()
    _freed_block_is_left_alone(dev, lambda s: fq.fp8_moe_route(l1, 8, stream=s))
    _freed_block_is_left_alone(dev, lambda s: [t for p in fq.fp8_swiglu_ckpt_1x128(c1, stream=s) for t in p])
    _output_outlives_queued_work(dev, side, lambda s: fq.fp8_moe_route(l1, 8, stream=s),
                                 lambda s: fq.fp8_moe_route(l2, 8, stream=s))


def test_named_stream_inside_a_captured_graph(dev, side):
    """A stream that joins a capture: the workspace and outputs of its calls stay the
    graph's, whatever is allocated between replays."""
    T, E, k = 6000, 64, 8
    ids = torch.zeros((T, k), dtype=torch.int32, device=dev)
    fq.fp8_moe_layout_contiguous(ids, E)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream(dev)
        side.wait_stream(here)
        a = fq.fp8_moe_layout_contiguous(ids, E, stream=side)
        b = fq.fp8_moe_layout_masked(ids, E, 1024)
        here.wait_stream(side)
    rng = np.random.default_rng(9)
    for _ in range(3):
        host = rng.integers(0, E, (T, k)).astype(np.int32)
        ids.copy_(torch.from_numpy(host))
        with torch.cuda.stream(side):
            junk = [torch.full((1 << 16,), 7, dtype=torch.int32, device=dev) for _ in range(8)]
        junk += [torch.full((1 << 16,), 7, dtype=torch.int32, device=dev) for _ in range(8)]
        torch.cuda.synchronize(dev)
        graph.replay()
        torch.cuda.synchronize(dev)
        assert all(bool((t == 7).all()) for t in junk)
        for ref, out in ((moe.layout_contiguous(host, E), a), (moe.layout_masked(host, E, 1024), b)):
            assert all(np.array_equal(x, y.cpu().numpy()) for x, y in zip(ref, out))


def _gemm_and_quantizer_calls(dev):
    """name -> call(stream): the calls marshalled in Python, with fresh outputs."""
    g = torch.Generator(device=dev).manual_seed(4)

    def bf16(*shape):
        return torch.randn(shape, generator=g, device=dev).bfloat16()

    x, w, wg, c1 = bf16(256, 512), bf16(128, 512), bf16(2, 128, 512), bf16(256, 512)
    qa, sa = fq.fp8_quant_act_1x128(x)
    qw, sw = fq.fp8_quant_w_128x128(w)
    qg, sg = fq.fp8_quant_w_128x128(wg)
    pa, ta = fq.fp8_quant_act_1x128_ue8m0(x)
    pw, tw = fq.fp8_quant_w_128x128_ue8m0(w)
    pg, tg = fq.fp8_quant_w_128x128_ue8m0(wg)
    xt, st = fq.fp8_quant_act_128x1_t(x)
    ma, mw, mg = fq.fp8_mx_scales_act(ta), fq.fp8_mx_scales_w(tw), fq.fp8_mx_scales_w(tg)
    ta3 = ta.view(2, 128, 4)
    ma3 = torch.cat([fq.fp8_mx_scales_act(ta3[e]) for e in range(2)])
    m_indices = torch.tensor([1, 0], dtype=torch.int32, device=dev)
    masked_m = torch.tensor([128, 128], dtype=torch.int32, device=dev)
    qa3, sa3, pa3 = qa.view(2, 128, 512), sa.view(2, 128, 4), pa.view(2, 128, 512)
    torch.cuda.synchronize(dev)
    return {
        "quant_act": lambda s: fq.fp8_quant_act_1x128(x, stream=s),
        "quant_w": lambda s: fq.fp8_quant_w_128x128(w, stream=s),
        "quant_act_w": lambda s: [t for p in fq.fp8_quant_act_w(x, w, stream=s) for t in p],
        "quant_act_ue8m0": lambda s: fq.fp8_quant_act_1x128_ue8m0(x, stream=s),
        "quant_w_ue8m0": lambda s: fq.fp8_quant_w_128x128_ue8m0(w, stream=s),
        "quant_act_128x1": lambda s: fq.fp8_quant_act_128x1(x, stream=s),
        "quant_act_128x1_t": lambda s: fq.fp8_quant_act_128x1_t(x, stream=s),
        "transpose": lambda s: fq.fp8_transpose_w_128x128(qw, sw, stream=s),
        "swiglu": lambda s: fq.fp8_swiglu_quant_1x128(c1, stream=s),
        "gemm": lambda s: [fq.fp8_gemm_blockscaled(qa, sa, qw, sw, stream=s)],
        "gemm_unpromoted": lambda s: [fq.fp8_gemm_unpromoted_diag(qa, sa, qw, sw, stream=s)],
        "wgrad": lambda s: [fq.fp8_gemm_wgrad(xt, st, xt, st, stream=s)],
        "grouped": lambda s: [fq.fp8_grouped_gemm_contiguous(qa, sa, qg, sg, m_indices, stream=s)],
        "masked": lambda s: [fq.fp8_grouped_gemm_masked(qa3, sa3, qg, sg, masked_m, stream=s)],
        "mx_scales_act": lambda s: [fq.fp8_mx_scales_act(ta, stream=s)],
        "mx_scales_w": lambda s: [fq.fp8_mx_scales_w(tw, stream=s)],
        "gemm_mx": lambda s: [fq.fp8_gemm_mx(pa, ma, pw, mw, stream=s)],
        "grouped_mx": lambda s: [fq.fp8_grouped_gemm_mx_contiguous(pa, ma, pg, mg, m_indices, stream=s)],
        "masked_mx": lambda s: [fq.fp8_grouped_gemm_mx_masked(pa3, ma3, pg, mg, masked_m, stream=s)],
    }


@pytest.mark.parametrize("how", ["stream", "handle"])
def test_outputs_of_gemms_and_quantizers_belong_to_the_named_stream(dev, side, how):
    for name, call in _gemm_and_quantizer_calls(dev).items():
        mine = call(None)
        torch.cuda.synchronize(dev)
        theirs = call(side if how == "stream" else side.cuda_stream)
        torch.cuda.synchronize(dev)
        for a, b in zip(mine, theirs):
            assert _stream_of(a) == 0, name
            assert _stream_of(b) == side.cuda_stream, name
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name
    assert fq.get_device_error(device=dev) == fq.OK


def test_gemms_and_quantizers_on_the_current_stream_by_name(dev, side):
    calls = _gemm_and_quantizer_calls(dev)
    for stream in (0, 1, torch.cuda.default_stream(dev)):
        for name, call in calls.items():
            assert all(_stream_of(t) == 0 for t in call(stream)), name
    with torch.cuda.stream(side):
        for name, call in calls.items():
            assert all(_stream_of(t) == side.cuda_stream for t in call(side)), name
            assert all(_stream_of(t) == 0 for t in call(0)), name
            assert all(_stream_of(t) == 0 for t in call(1)), name
    torch.cuda.synchronize(dev)
    assert fq.get_device_error(device=dev) == fq.OK


def test_quantizers_leave_memory_of_other_streams_alone(dev, side):
    x1, x2 = (torch.randn((4096, 1024), device=dev).bfloat16() for _ in range(2))
    _freed_block_is_left_alone(dev, lambda s: fq.fp8_quant_act_1x128(x1, stream=s))
    _output_outlives_queued_work(dev, side, lambda s: fq.fp8_quant_act_1x128(x1, stream=s),
                                 lambda s: fq.fp8_quant_act_1x128(x2, stream=s))
