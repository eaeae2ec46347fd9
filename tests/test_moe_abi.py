"""Refusals of the routing, layout, dispatch, combine and checkpoint entry
points (CPU only): the C layer's statuses before any launch, the binding's
messages before any call, and one NVTX range per call."""
import json
import os
import subprocess
import sys

import pytest
import torch

import fp8_fine_grained_quant_b200 as fq
from test_nvtx_ranges import ROOT, recorder  # noqa: F401  (a fixture)

A16, A4, A1, A2 = 0x10000, 0x10004, 0x10001, 0x10002
BIG = 1 << 31
u8, f32, bf16, i32 = torch.uint8, torch.float32, torch.bfloat16, torch.int32


def z(*shape, dtype=u8):
    return torch.zeros(shape, dtype=dtype)


def _route(T=4, E=8, k=2, G=1, KG=1, GT=1, logits=A16, bf=0, bias=None, ids=A16, w=A16):
    return (logits, bf, T, E, bias, 0, k, G, KG, GT, 1, 1.0, ids, w, None)


CASES = [
    ("fp8_moe_route", _route(T=-1), fq.ERR_SHAPE),
    ("fp8_moe_route", _route(T=BIG), fq.ERR_SHAPE),
    ("fp8_moe_route", _route(E=0), fq.ERR_SHAPE),
    ("fp8_moe_route", _route(E=1025), fq.ERR_SHAPE),
    ("fp8_moe_route", _route(k=0), fq.ERR_SHAPE),
    ("fp8_moe_route", _route(k=9), fq.ERR_SHAPE),                       # more places than experts
    ("fp8_moe_route", _route(E=64, k=33), fq.ERR_SHAPE),
    ("fp8_moe_route", _route(G=3), fq.ERR_SHAPE),                       # does not divide E
    ("fp8_moe_route", _route(E=64, G=64), fq.ERR_SHAPE),
    ("fp8_moe_route", _route(G=2, KG=3), fq.ERR_SHAPE),
    ("fp8_moe_route", _route(k=5, G=2, KG=1), fq.ERR_SHAPE),            # more places than the kept groups' experts
    ("fp8_moe_route", _route(GT=3), fq.ERR_SHAPE),
    ("fp8_moe_route", _route(T=0, logits=None, ids=None, w=None), fq.OK),
    ("fp8_moe_route", _route(logits=None), fq.ERR_NULL),
    ("fp8_moe_route", _route(ids=None), fq.ERR_NULL),
    ("fp8_moe_route", _route(w=None), fq.ERR_NULL),
    ("fp8_moe_route", _route(logits=A2), fq.ERR_ALIGN),
    ("fp8_moe_route", _route(logits=A1, bf=1), fq.ERR_ALIGN),
    ("fp8_moe_route", _route(bias=A1), fq.ERR_ALIGN),
    ("fp8_moe_route_bwd", (A16, 0, 4, 2000, A16, A16, 0, 2, 1, 1.0, A16, None), fq.ERR_SHAPE),
    ("fp8_moe_route_bwd", (A16, 0, 4, 8, A16, A16, 0, 33, 1, 1.0, A16, None), fq.ERR_SHAPE),
    ("fp8_moe_route_bwd", (A16, 0, 0, 8, None, None, 0, 2, 1, 1.0, None, None), fq.OK),
    ("fp8_moe_route_bwd", (A16, 0, 4, 8, None, A16, 0, 2, 1, 1.0, A16, None), fq.ERR_NULL),
    ("fp8_moe_route_bwd", (A16, 0, 4, 8, A16, A16, 0, 2, 1, 1.0, A2, None), fq.ERR_ALIGN),
    ("fp8_moe_layout_contiguous", (A16, 4, 0, 8, A16, A16, A16, A16, None), fq.ERR_SHAPE),
    ("fp8_moe_layout_contiguous", (A16, 4, 2, 1025, A16, A16, A16, A16, None), fq.ERR_SHAPE),
    ("fp8_moe_layout_contiguous", (A16, BIG - 1, 2, 8, A16, A16, A16, A16, None), fq.ERR_SHAPE),   # 2^32 rows
    ("fp8_moe_layout_contiguous", (A16, 4, 2, 8, A16, A16, None, A16, None), fq.ERR_NULL),
    ("fp8_moe_layout_contiguous", (A16, 4, 2, 8, None, A16, A16, A16, None), fq.ERR_NULL),
    ("fp8_moe_layout_contiguous", (A16, 0, 2, 8, None, None, None, A16, None), fq.ERR_NULL),       # counts are written
    ("fp8_moe_layout_contiguous", (A1, 4, 2, 8, A16, A16, A16, A16, None), fq.ERR_ALIGN),
    ("fp8_moe_layout_masked", (A16, 4, 2, 8, 100, A16, A16, A16, None), fq.ERR_SHAPE),
    ("fp8_moe_layout_masked", (A16, 4, 2, 8, 0, A16, A16, A16, None), fq.ERR_SHAPE),
    ("fp8_moe_layout_masked", (A16, 4, 2, 1024, 1 << 21, A16, A16, A16, None), fq.ERR_SHAPE),      # E * cap = 2^31
    ("fp8_moe_layout_masked", (A16, 4, 2, 8, 128, A16, None, A16, None), fq.ERR_NULL),
    ("fp8_moe_layout_masked", (A16, 4, 2, 8, 128, A1, A16, A16, None), fq.ERR_ALIGN),
    ("fp8_moe_layout_masked", (A16, 10000, 8, 8, 128, A16, A16, None, None), fq.ERR_NULL),    # needs a workspace
    ("fp8_moe_layout_contiguous", (A16, 10000, 8, 8, A16, A16, A16, A1, None), fq.ERR_ALIGN),
    ("fp8_moe_dispatch_1x128", (A16, 4, 100, A16, 2, 256, None, None, 0, A16, A16, None), fq.ERR_SHAPE),
    ("fp8_moe_dispatch_1x128", (A16, 4, 128, A16, 2, -1, None, None, 0, A16, A16, None), fq.ERR_SHAPE),
    ("fp8_moe_dispatch_1x128", (A16, BIG - 1, 256, A16, 2, 256, None, None, 0, A16, A16, None), fq.ERR_SHAPE),
    ("fp8_moe_dispatch_1x128", (A16, 4, 128, A16, 2, 200, A16, A16, 8, A16, A16, None), fq.ERR_SHAPE),
    ("fp8_moe_dispatch_1x128", (A16, 4, 128, A16, 2, 256, A16, A16, 0, A16, A16, None), fq.ERR_SHAPE),
    ("fp8_moe_dispatch_1x128", (A16, 4, 128, A16, 2, 256, A16, None, 8, A16, A16, None), fq.ERR_NULL),
    ("fp8_moe_dispatch_1x128", (A16, 0, 128, None, 2, 0, None, A16, 8, None, None, None), fq.OK),  # an empty layout
    ("fp8_moe_combine_bwd", (A16, None, 0, 128, A16, A16, 0, 2, None, A16, 8, None, A16, None), fq.OK),
    ("fp8_moe_dispatch_1x128", (A16, 0, 128, None, 2, 256, None, None, 0, None, None, None), fq.OK),
    ("fp8_moe_dispatch_1x128", (A16, 4, 128, A16, 2, 0, None, None, 0, None, None, None), fq.OK),
    ("fp8_moe_dispatch_1x128", (A16, 4, 128, None, 2, 256, None, None, 0, A16, A16, None), fq.ERR_NULL),
    ("fp8_moe_dispatch_1x128", (A16 + 16, 4, 128, A16, 2, 256, None, None, 0, A16, A16, None), fq.ERR_ALIGN),
    ("fp8_moe_dispatch_1x128", (A16, 4, 128, A16, 2, 256, None, None, 0, A4, A16, None), fq.ERR_ALIGN),
    ("fp8_moe_combine", (A16, 256, 100, A16, A16, 4, 2, A16, None), fq.ERR_SHAPE),
    ("fp8_moe_combine", (A16, 256, 128, A16, A16, 4, 0, A16, None), fq.ERR_SHAPE),
    ("fp8_moe_combine", (None, 256, 128, A16, A16, 4, 2, A16, None), fq.ERR_NULL),
    ("fp8_moe_combine", (A16, 256, 128, A16, None, 0, 2, A16, None), fq.OK),
    ("fp8_moe_combine", (A4, 256, 128, A16, A16, 4, 2, A16, None), fq.ERR_ALIGN),
    ("fp8_moe_combine", (A16, 256, 128, A16, A1, 4, 2, A16, None), fq.ERR_ALIGN),
    ("fp8_moe_combine_bwd", (A16, A16, 256, 100, A16, A16, 4, 2, None, None, 0, A16, A16, None), fq.ERR_SHAPE),
    ("fp8_moe_combine_bwd", (A16, A16, 256, 128, A16, None, 4, 2, None, None, 0, A16, A16, None), fq.ERR_NULL),
    ("fp8_moe_combine_bwd", (A16, A16, 256, 128, A16, A16, 4, 2, None, A16, 8, A16, A16, None), fq.ERR_NULL),
    ("fp8_moe_combine_bwd", (A16, A16, 256, 128, A16, A16, 0, 2, None, None, 0, A16, A16, None), fq.OK),
    ("fp8_moe_combine_bwd", (A16, A16, 256, 128, A16, A16, 4, 2, None, None, 0, A4, A16, None), fq.ERR_ALIGN),
    ("fp8_swiglu_ckpt_1x128", (A16, 4, 100, A16, A16, A16, A16, None), fq.ERR_SHAPE),
    ("fp8_swiglu_ckpt_1x128", (A16, BIG - 1, 256, A16, A16, A16, A16, None), fq.ERR_SHAPE),
    ("fp8_swiglu_ckpt_1x128", (A16, 0, 128, A16, A16, A16, A16, None), fq.OK),
    ("fp8_swiglu_ckpt_1x128", (A16, 4, 128, A16, A16, None, A16, None), fq.ERR_NULL),
    ("fp8_swiglu_ckpt_1x128", (A16 + 16, 4, 128, A16, A16, A16, A16, None), fq.ERR_ALIGN),
    ("fp8_swiglu_ckpt_1x128", (A16, 4, 128, A16, A16, A4, A16, None), fq.ERR_ALIGN),
    ("fp8_swiglu_bwd_1x128", (A16, A16, A16, 4, 100, A16, A16, A16, None), fq.ERR_SHAPE),
    ("fp8_swiglu_bwd_1x128", (A16, A16, A16, 4, 128, None, A16, A16, None), fq.ERR_NULL),
    ("fp8_swiglu_bwd_1x128", (A16, A16, A16, 4, 0, A16, A16, A16, None), fq.OK),
    ("fp8_swiglu_bwd_1x128", (A16, A4, A16, 4, 128, A16, A16, A16, None), fq.ERR_ALIGN),
    ("fp8_ckpt_128x1_t", (A16, A16, 4, 100, 128, A16, A16, None), fq.ERR_SHAPE),
    ("fp8_ckpt_128x1_t", (A16, A16, 200, 128, 128, A16, A16, None), fq.ERR_SHAPE),   # fewer padded tokens than tokens
    ("fp8_ckpt_128x1_t", (A16, A16, 4, 128, 200, A16, A16, None), fq.ERR_SHAPE),
    ("fp8_ckpt_128x1_t", (A16, A16, 0, 128, 0, A16, A16, None), fq.OK),
    ("fp8_ckpt_128x1_t", (None, A16, 4, 128, 128, A16, A16, None), fq.ERR_NULL),
    ("fp8_ckpt_128x1_t", (A16, A16, 4, 128, 128, A16, A4, None), fq.ERR_ALIGN),
]


@pytest.mark.parametrize("name,args,expect", CASES)
def test_c_layer_refuses(name, args, expect):
    assert getattr(fq.lib(), name)(*args) == expect


NVTX_CHILD = r"""
import ctypes, json, sys
sys.path.insert(0, sys.argv[1])
sys.path.insert(0, sys.argv[1] + "/tests")
import fp8_fine_grained_quant_b200 as fq
from test_moe_abi import CASES
rec = ctypes.CDLL(sys.argv[2])
rec.rec_log.restype = ctypes.c_char_p
out = []
for name, args, expect in CASES:
    rec.rec_clear()
    rc = getattr(fq.lib(), name)(*args)
    out.append({"name": name, "rc": rc, "log": rec.rec_log().decode(), "depth": rec.rec_depth()})
print(json.dumps(out))
"""


def test_every_call_opens_and_closes_its_range(recorder):  # noqa: F811
    env = dict(os.environ, NVTX_INJECTION64_PATH=str(recorder), CUDA_VISIBLE_DEVICES="")
    res = subprocess.run([sys.executable, "-c", NVTX_CHILD, str(ROOT), str(recorder)], env=env, capture_output=True,
                         text=True, timeout=300, check=True)
    rows = json.loads(res.stdout.strip().splitlines()[-1])
    assert len(rows) == len(CASES) and len({r["name"] for r in rows}) == 10
    for r in rows:
        assert r["log"] == "push %s\npop\n" % r["name"] and r["depth"] == 0, r


def lg(T=4, E=8, dtype=f32):
    return z(T, E, dtype=dtype)


@pytest.mark.parametrize("kw,match", [
    (dict(top_k=0), "top_k = 0"),
    (dict(top_k=9), "top_k = 9"),
    (dict(top_k=2, score="relu"), "score must be"),
    (dict(top_k=2, n_group=3), "n_group = 3"),
    (dict(top_k=2, n_group=2, topk_group=3), "topk_group = 3"),
    (dict(top_k=2, group_top=3), "group_top = 3"),
    (dict(top_k=5, n_group=2, topk_group=1), "exceeds the 4 experts"),
    (dict(top_k=2, bias=z(7, dtype=f32)), "bias holds 7"),
    (dict(top_k=2, ids=z(7, dtype=i32)), "ids holds 7"),
    (dict(top_k=2, weights=z(9, dtype=f32)), "weights holds 9"),
    (dict(top_k=2, bias=z(8, dtype=bf16)), "bias: dtype"),
    (dict(top_k=2), "CUDA tensor"),
])
def test_route_arguments(kw, match):
    with pytest.raises((ValueError, TypeError), match=match):
        fq.fp8_moe_route(lg(), **kw)


def test_route_logits():
    with pytest.raises(TypeError, match="logits: dtype"):
        fq.fp8_moe_route(lg(dtype=torch.float16), 2)
    with pytest.raises(ValueError, match="logits must be contiguous"):
        fq.fp8_moe_route(lg(4, 16)[:, ::2], 2)
    with pytest.raises(ValueError, match="1025 experts"):
        fq.fp8_moe_route(lg(1, 1025), 2)


def test_route_bwd_arguments():
    ids, g = z(4, 2, dtype=i32), z(4, 2, dtype=f32)
    with pytest.raises(ValueError, match="ids holds 6"):
        fq.fp8_moe_route_bwd(lg(), z(3, 2, dtype=i32), g)
    with pytest.raises(ValueError, match="dweights holds 4"):
        fq.fp8_moe_route_bwd(lg(), ids, z(4, 1, dtype=f32))
    with pytest.raises(TypeError, match="dlogits: dtype"):
        fq.fp8_moe_route_bwd(lg(dtype=bf16), ids, g, dlogits=lg())
    with pytest.raises(TypeError, match="ids: dtype"):
        fq.fp8_moe_route_bwd(lg(), ids.long(), g)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fq.fp8_moe_route_bwd(lg(), ids, g)


def test_layout_workspace_size():
    ws = fq.lib().fp8_moe_layout_workspace
    assert ws(4096, 8, 32) == 0                       # one cluster
    assert ws(4097, 8, 32) == 9 * 32                  # 32776 entries: nine chunks of 4096
    assert ws(1 << 20, 8, 256) == 148 * 256           # no more chunks than SMs
    assert ws(-1, 8, 32) == ws(4097, 33, 32) == ws(4097, 8, 1025) == 0


def test_layout_arguments():
    ids = z(4, 2, dtype=i32)
    assert fq.moe_contiguous_blocks(4, 2, 3) == (8 + 127 * 3) // 128
    with pytest.raises(ValueError, match="E = 0"):
        fq.fp8_moe_layout_contiguous(ids, 0)
    with pytest.raises(ValueError, match="m_indices holds 4"):
        fq.fp8_moe_layout_contiguous(ids, 3, m_indices=z(4, dtype=i32))
    with pytest.raises(ValueError, match="counts holds 4"):
        fq.fp8_moe_layout_contiguous(ids, 3, counts=z(4, dtype=i32))
    with pytest.raises(ValueError, match="cap = 100"):
        fq.fp8_moe_layout_masked(ids, 3, 100)
    with pytest.raises(ValueError, match="cap = 200"):
        fq.fp8_moe_layout_masked(ids, 3, 200)
    with pytest.raises(ValueError, match="masked_m holds 2"):
        fq.fp8_moe_layout_masked(ids, 3, 128, masked_m=z(2, dtype=i32))
    with pytest.raises(ValueError, match="33 columns"):
        fq.fp8_moe_layout_masked(z(4, 33, dtype=i32), 3, 128)
    for call in (lambda: fq.fp8_moe_layout_contiguous(ids, 3), lambda: fq.fp8_moe_layout_masked(ids, 3, 128)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_dispatch_arguments():
    x, sl = z(4, 256, dtype=bf16), z(4, 2, dtype=i32)
    m, c = z(2, dtype=i32), z(3, dtype=i32)
    with pytest.raises(ValueError, match="slots are for 3 tokens"):
        fq.fp8_moe_dispatch_1x128(x, z(3, 2, dtype=i32), 256)
    with pytest.raises(ValueError, match="go together"):
        fq.fp8_moe_dispatch_1x128(x, sl, 256, m_indices=m)
    with pytest.raises(ValueError, match="m_indices holds 2 elements, the call needs 3"):
        fq.fp8_moe_dispatch_1x128(x, sl, 384, m_indices=m, counts=c)
    with pytest.raises(ValueError, match="q holds 256"):
        fq.fp8_moe_dispatch_1x128(x, sl, 256, q=z(1, 256))
    with pytest.raises(ValueError, match="D = 200"):
        fq.fp8_moe_dispatch_1x128(z(4, 200, dtype=bf16), sl, 256)
    with pytest.raises(ValueError, match="negative"):
        fq.fp8_moe_dispatch_1x128(x, sl, -128)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fq.fp8_moe_dispatch_1x128(x, sl, 256, m_indices=m, counts=c)


def test_combine_arguments():
    y, sl, w, g = z(256, 128, dtype=bf16), z(4, 2, dtype=i32), z(4, 2, dtype=f32), z(4, 128, dtype=bf16)
    with pytest.raises(ValueError, match="weights holds 6"):
        fq.fp8_moe_combine(y, sl, z(3, 2, dtype=f32))
    with pytest.raises(ValueError, match="out holds 128"):
        fq.fp8_moe_combine(y, sl, w, out=z(1, 128, dtype=bf16))
    with pytest.raises(ValueError, match="differ in D"):
        fq.fp8_moe_combine_bwd(z(4, 256, dtype=bf16), y, sl, w)
    with pytest.raises(TypeError, match="weights must be"):
        fq.fp8_moe_combine_bwd(g, y, sl, None)
    with pytest.raises(ValueError, match="dy holds 128"):
        fq.fp8_moe_combine_bwd(g, y, sl, w, dy=z(1, 128, dtype=bf16))
    with pytest.raises(ValueError, match="slots are for 3"):
        fq.fp8_moe_combine_bwd(g, y, z(3, 2, dtype=i32), w)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fq.fp8_moe_combine(y.view(2, 128, 128), sl, w)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fq.fp8_moe_combine_bwd(g, y, sl, w)


def test_checkpoint_arguments():
    c1 = z(4, 512, dtype=bf16)
    with pytest.raises(ValueError, match="not 2 x a multiple"):
        fq.fp8_swiglu_ckpt_1x128(z(4, 384, dtype=bf16))
    with pytest.raises(ValueError, match="qc holds 1024"):
        fq.fp8_swiglu_ckpt_1x128(c1, qc=z(4, 256))
    with pytest.raises(ValueError, match="sc holds 8 elements, the call needs 16"):
        fq.fp8_swiglu_ckpt_1x128(c1, sc=z(4, 2, dtype=f32))
    with pytest.raises(ValueError, match="CUDA tensor"):
        fq.fp8_swiglu_ckpt_1x128(c1)
    dh, qc, sc = z(4, 256, dtype=bf16), z(4, 512), z(4, 4, dtype=f32)
    with pytest.raises(ValueError, match=r"needs \[4, 512\]"):
        fq.fp8_swiglu_bwd_1x128(dh, z(4, 256), sc)
    with pytest.raises(ValueError, match="sc holds 8"):
        fq.fp8_swiglu_bwd_1x128(dh, qc, z(4, 2, dtype=f32))
    with pytest.raises(ValueError, match="dc holds 1024"):
        fq.fp8_swiglu_bwd_1x128(dh, qc, sc, dc=z(4, 256, dtype=bf16))
    with pytest.raises(ValueError, match="CUDA tensor"):
        fq.fp8_swiglu_bwd_1x128(dh, qc, sc)
    with pytest.raises(ValueError, match="s holds 4"):
        fq.fp8_ckpt_128x1_t(z(4, 256), z(4, 1, dtype=f32))
    with pytest.raises(ValueError, match="below the token count"):
        fq.fp8_ckpt_128x1_t(z(200, 256), z(200, 2, dtype=f32), Mp=128)
    with pytest.raises(ValueError, match="qt holds"):
        fq.fp8_ckpt_128x1_t(z(200, 256), z(200, 2, dtype=f32), qt=z(256, 256))
    with pytest.raises(ValueError, match="CUDA tensor"):
        fq.fp8_ckpt_128x1_t(z(200, 256), z(200, 2, dtype=f32))
