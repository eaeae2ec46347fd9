"""Measured cases of the mixture-of-experts and activation-checkpoint operators.

Three operators around the grouped and dense FP8 GEMMs:

* routing      -- expert choice from router logits (and its gradient);
* dispatch     -- the grouped GEMMs' row layouts, the tokens quantized into them,
                  the weighted sum of the experts' outputs (and its gradient);
* checkpoints  -- what the backward pass keeps in 8 bits: the SwiGLU input saved
                  as 1x128 E4M3 tiles, the SwiGLU backward that reads it, and the
                  weight-gradient operand made from a saved 1x128 activation.

``run`` computes a case in plain torch operations (``own`` false) or through
the library's entry points (``own`` true), on the same inputs.  ``exact`` gives
the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

TILE = 128
DEV = "cuda"
NEG = float("-inf")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the router of one decoded token: 256 experts in 8 groups, 4 groups kept, sigmoid scores with a balance bias
        dict(name="route_one_token", op="route", T=1, E=256, k=8, score="sigmoid", bias=True, groups=8, kept=4,
             group_top=2, renorm=True, dtype="f32", masks=False),
        # the router of a 4096-token prompt over 32 experts, top-8 (the MoE workloads' routing), bf16 logits
        dict(name="route_prompt", op="route", T=4096, E=32, k=8, score="softmax", bias=False, groups=1, kept=1,
             group_top=1, renorm=True, dtype="bf16", masks=False),
        # a long batch through the grouped, biased router, with masked experts and one row that has none left
        dict(name="route_long", op="route", T=32768, E=256, k=8, score="sigmoid", bias=True, groups=8, kept=4,
             group_top=2, renorm=True, dtype="f32", masks=True),
        # the router's gradient in training: plain softmax probabilities (every logit gets a gradient)
        dict(name="route_grad", op="route_bwd", T=16384, E=160, k=6, score="softmax", renorm=False, dtype="f32"),
        # decode: 61 tokens of a running batch quantized into the masked layout's expert slots
        dict(name="dispatch_decode", op="dispatch", T=61, E=32, k=8, D=7168, layout="masked", cap=256, idle=3),
        # the 4096-token MoE layer of the contiguous workload: layout, quantization, padding
        dict(name="dispatch_prompt", op="dispatch", T=4096, E=32, k=8, D=7168, layout="contiguous", cap=0, idle=0),
        # decode: the weighted sum of 61 tokens' expert outputs
        dict(name="combine_decode", op="combine", T=61, E=32, k=8, D=7168, layout="masked", cap=256, idle=3,
             weighted=True),
        # training: the gradient of that sum with respect to the experts' outputs and the routing weights
        dict(name="combine_grad", op="combine_bwd", T=4096, E=32, k=8, D=7168, layout="contiguous", cap=0, idle=0),
        # a short, odd micro-batch: SwiGLU output and its 8-bit checkpoint
        dict(name="ckpt_store_short", op="ckpt_store", rows=333, inter=2048),
        # the contiguous workload's rows: SwiGLU output and its 8-bit checkpoint
        dict(name="ckpt_store", op="ckpt_store", rows=35072, inter=2048),
        # SwiGLU backward from the checkpoint, same rows
        dict(name="ckpt_swiglu_grad", op="ckpt_bwd", rows=35072, inter=2048),
        # the weight-gradient operand of a dense layer from the activation its forward pass quantized
        dict(name="ckpt_wgrad_operand", op="ckpt_t", rows=4096, K=7168),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_bwd", "dispatch", "combine", "combine_bwd", "ckpt_store", "ckpt_bwd", "ckpt_t"])
    if op == "route":
        E = rng.choice([8, 16, 32, 60, 64, 128, 160, 256, 320, 512])
        groups = rng.choice([g for g in (1, 1, 2, 4, 5, 8, 16) if E % g == 0 and E // g >= 4])
        kept = rng.randint(1, groups)
        k = min(rng.choice([1, 2, 4, 6, 8, 10]), kept * (E // groups))
        return dict(op=op, T=_log(rng, 1, 16384), E=E, k=k, score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.6, groups=groups, kept=kept, group_top=rng.choice([1, 2]),
                    renorm=k > 1 and rng.random() < 0.7, dtype=rng.choice(["f32", "bf16"]),
                    masks=rng.random() < 0.4)
    if op == "route_bwd":
        E = rng.choice([8, 16, 32, 60, 64, 128, 160, 256, 320, 512])
        return dict(op=op, T=_log(rng, 16, 16384), E=E, k=rng.choice([2, 4, 6, 8]),
                    score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.6,
                    dtype=rng.choice(["f32", "bf16"]))
    if op in ("dispatch", "combine", "combine_bwd"):
        E, k = rng.choice([8, 16, 32, 64, 128]), rng.choice([1, 2, 4, 6, 8])
        D = 128 * rng.randint(4, 56)
        T = min(_log(rng, 1, 8192), max(1, 200_000_000 // (k * D)))
        c = dict(op=op, T=T, E=E, k=k, D=D, layout="contiguous" if op == "combine_bwd" else
                 rng.choice(["contiguous", "masked"]), cap=0, idle=rng.choice([0, 0, T // 5]))
        if c["layout"] == "masked":
            c["T"] = min(T, 512)
            c["idle"] = min(c["idle"], c["T"] // 5)
            c["cap"] = rng.choice([128, 256])   # experts past their capacity drop their last tokens
        if op == "combine":
            c["weighted"] = rng.random() < 0.7  # unweighted: the gradient of the dispatch
        return c
    if op == "ckpt_t":
        K = 128 * rng.randint(2, 56)
        return dict(op=op, rows=min(_log(rng, 1, 8192), 32_000_000 // K), K=K)
    inter = 128 * rng.randint(2, 32)
    return dict(op=op, rows=min(_log(rng, 1, 32768), 64_000_000 // inter), inter=inter)


def work(c):
    """Bytes each input is read and each output written once; arithmetic in FP32 operations (no matrix products)."""
    op = c["op"]
    if op == "route":
        n = c["T"] * c["E"]
        return {"bytes": n * (2 if c["dtype"] == "bf16" else 4) + 8 * c["T"] * c["k"] + 4 * c["E"] * c["bias"],
                "flops": 12 * n}
    if op == "route_bwd":
        n, b = c["T"] * c["E"], 2 if c["dtype"] == "bf16" else 4
        # softmax probabilities need every logit, the other forms the chosen ones only
        read = n * b if c["score"] == "softmax" and not c["renorm"] else c["T"] * c["k"] * b
        return {"bytes": read + n * b + 8 * c["T"] * c["k"], "flops": 6 * n}
    if op in ("dispatch", "combine", "combine_bwd"):
        T = c["T"] - c["idle"]
        n, D = T * c["k"], c["D"]
        if op == "dispatch":
            return {"bytes": 2 * T * D + n * (D + D // 32) + 8 * c["T"] * c["k"], "flops": 4 * T * D}
        if op == "combine":
            return {"bytes": 2 * n * D + 2 * c["T"] * D + 8 * c["T"] * c["k"], "flops": 2 * n * D}
        return {"bytes": 4 * n * D + 2 * T * D + 12 * c["T"] * c["k"], "flops": 3 * n * D}
    if op == "ckpt_t":
        n, Mp = c["rows"] * c["K"], -(-c["rows"] // 512) * 512
        return {"bytes": n + n // 32 + Mp * c["K"] + Mp // 32 * c["K"], "flops": 4 * n}
    n = c["rows"] * c["inter"]
    if op == "ckpt_store":
        return {"bytes": 4 * n + 3 * n + 3 * n // 32, "flops": 30 * n}
    return {"bytes": 2 * n + 2 * n + 2 * n // 32 + 4 * n + 2 * n + 2 * n // 32, "flops": 40 * n}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _routing_ids(c, g):
    """Distinct experts for each token, unevenly popular (Zipf 1.1 over a random ranking, Gumbel top-k); idle tokens
    (padding of a batch) have none."""
    T, E, k = c["T"], c["E"], c["k"]
    rank = torch.randperm(E, generator=g, device=DEV)
    pop = -1.1 * torch.log(rank.float() + 1.0)
    u = torch.rand((T, E), generator=g, device=DEV).clamp_(1e-7, 1 - 1e-7)
    ids = torch.topk(pop - torch.log(-torch.log(u)), k, dim=1).indices.to(torch.int32)
    if c["idle"]:
        ids[T - c["idle"]:] = -1
    return ids.contiguous()


def _rows(c):
    """Rows of the expert-major buffers: the masked layout's slots, or the contiguous layout's bound on whole blocks."""
    if c["layout"] == "masked":
        return c["E"] * c["cap"]
    n = c["T"] * c["k"]
    return (n + (TILE - 1) * min(c["E"], n)) // TILE * TILE


def prepare(c, seed):
    g = _gen(seed)
    op = c["op"]
    s = {"c": dict(c)}
    if op in ("route", "route_bwd"):
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        T, E = c["T"], c["E"]
        l = 1.5 * torch.randn((T, E), generator=g, device=DEV) + 0.5 * torch.randn((E,), generator=g, device=DEV)
        if c.get("masks"):
            gone = torch.rand((T, E), generator=g, device=DEV) < 0.3 * (torch.rand((T, 1), generator=g, device=DEV) < 0.25)
            l = l.masked_fill(gone, NEG)
            if T >= 8:
                l[T - 2] = NEG
        s["logits"] = l.to(dt).contiguous()
        if op == "route":
            s["bias"] = 0.1 * torch.randn((E,), generator=g, device=DEV) if c["bias"] else None
        else:
            u = torch.rand((T, E), generator=g, device=DEV)
            s["ids"] = torch.topk(l + 0.3 * u, c["k"], dim=1).indices.to(torch.int32).contiguous()
            s["dw"] = torch.randn((T, c["k"]), generator=g, device=DEV)
        return s
    if op in ("dispatch", "combine", "combine_bwd"):
        T, k, D, rows = c["T"], c["k"], c["D"], _rows(c)
        s["ids"] = _routing_ids(c, g)
        if op == "dispatch":
            chan = torch.exp(0.7 * torch.randn((D,), generator=g, device=DEV))
            s["x"] = (torch.randn((T, D), generator=g, device=DEV) * chan).to(torch.bfloat16)
            # one row more than the layout has: a place for entries without a slot in the plain form
            s["q"] = torch.zeros((rows + 1, D), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
            s["s"] = torch.zeros((rows + 1, D // TILE), dtype=torch.float32, device=DEV)
            return s
        lay = _layout_contiguous(s["ids"], c["E"], rows) if c["layout"] == "contiguous" else \
            _layout_masked(s["ids"], c["E"], c["cap"])
        s["slots"] = lay[0]
        if c["layout"] == "contiguous":
            s["m_indices"], s["counts"] = lay[1], lay[2]
        s["y"] = torch.randn((rows, D), generator=g, device=DEV).to(torch.bfloat16)
        w = torch.rand((T, k), generator=g, device=DEV) + 0.05
        s["w"] = w / w.sum(1, keepdim=True)
        if op == "combine_bwd":
            s["dout"] = torch.randn((T, D), generator=g, device=DEV).to(torch.bfloat16)
            s["dy"] = torch.zeros((rows + 1, D), dtype=torch.bfloat16, device=DEV)
        elif not c["weighted"]:
            s["w"] = None
        return s
    if op == "ckpt_t":
        M, K = c["rows"], c["K"]
        chan = torch.exp(0.7 * torch.randn((K,), generator=g, device=DEV))
        x = (torch.randn((M, K), generator=g, device=DEV) * chan).to(torch.bfloat16)
        s["q"], s["s"] = _quant_1x128(x)
        return s
    M, inter = c["rows"], c["inter"]
    chan = torch.exp(0.4 * torch.randn((2 * inter,), generator=g, device=DEV))
    c1 = (torch.randn((M, 2 * inter), generator=g, device=DEV) * chan).to(torch.bfloat16)
    if op == "ckpt_store":
        s["c1"] = c1
        return s
    s["qc"], s["sc"] = _quant_1x128(c1)
    s["dh"] = (0.1 * torch.randn((M, inter), generator=g, device=DEV)).to(torch.bfloat16)
    return s


# ------------------------------------------------------------------ plain forms
def _e4m3(v):
    """FP32 -> E4M3, round to nearest even, saturating."""
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _scale(amax):
    """fl32(amax / 448), 1 for a group of zeros (the divisor as a tensor: a true division)."""
    s = amax / torch.full((), 448.0, device=amax.device)
    return torch.where(s == 0, torch.ones_like(s), s)


def _quant_1x128(x):
    """1x128 tiles of a 2-D tensor of bf16 or FP32 values: codes and scales."""
    v = x.float().view(x.shape[0], -1, TILE)
    s = _scale(v.abs().amax(dim=2))
    return _e4m3(v / s[:, :, None]).view(x.shape), s


def _round_bf16(v):
    """64-bit values to bf16 with one rounding: the FP32 step of the conversion is moved off a bf16 midpoint that it
    only reached by rounding."""
    f = v.float()
    bits = f.view(torch.int32)
    d = v - f.double()
    step = torch.sign(d) * torch.sign(f.double())
    mid = (bits & 0xFFFF) == 0x8000
    bits = torch.where(mid, bits + step.to(torch.int32), bits)
    return bits.view(torch.float32).to(torch.bfloat16)


def _route(s):
    """Selection in 64 bits: scores next to each other decide whole numbers."""
    c, l = s["c"], s["logits"].double()
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    ok = l > NEG
    l = torch.where(ok, l, torch.full_like(l, NEG))
    if c["score"] == "softmax":
        m = l.amax(dim=1, keepdim=True)
        e = torch.exp(l - torch.where(m > NEG, m, torch.zeros_like(m)))
        p = e / e.sum(dim=1, keepdim=True).clamp_min(1e-300)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    none = torch.full_like(p, NEG)
    key = torch.where(ok, p + s["bias"].double() if s["bias"] is not None else p, none)
    order = key if s["bias"] is not None else l
    if G > 1:
        best = torch.sort(key.view(T, G, E // G), dim=2, descending=True).values[:, :, :c["group_top"]]
        some = best[:, :, 0] > NEG
        total = torch.where(best > NEG, best, torch.zeros_like(best)).sum(dim=2)
        total = torch.where(some, total, torch.full_like(total, NEG))
        kept = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :c["kept"]]
        keep = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        order = torch.where(keep[:, :, None].expand(T, G, E // G).reshape(T, E), order, none)
    top = torch.sort(order, dim=1, descending=True, stable=True)
    ids, found = top.indices[:, :k], top.values[:, :k] > NEG
    w = torch.where(found, torch.gather(p, 1, ids), torch.zeros_like(p[:, :k]))
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True).clamp_min(1e-300)
    return torch.where(found, ids, torch.full_like(ids, -1)).to(torch.int32), (2.5 * w).float()


def _route_bwd(s):
    c, l, dw = s["c"], s["logits"].float(), s["dw"]
    at = s["ids"].long()
    if c["score"] == "softmax" and not c["renorm"]:
        e = torch.exp(l - l.amax(dim=1, keepdim=True))
        p = e / e.sum(dim=1, keepdim=True)
        d = torch.zeros_like(l).scatter_add_(1, at, dw)
        dl = 2.5 * p * (d - (d * p).sum(dim=1, keepdim=True))
        return dl.to(s["logits"].dtype)
    ls = torch.gather(l, 1, at)
    if c["score"] == "softmax":
        e = torch.exp(ls - ls.amax(dim=1, keepdim=True))
        p = e / e.sum(dim=1, keepdim=True)
        ds = 2.5 * p * (dw - (dw * p).sum(dim=1, keepdim=True))
    else:
        p = 1.0 / (1.0 + torch.exp(-ls))
        not_p = 1.0 / (1.0 + torch.exp(ls))
        if c["renorm"]:
            r = p / p.sum(dim=1, keepdim=True)
            ds = 2.5 * r * (dw - (dw * r).sum(dim=1, keepdim=True)) * not_p
        else:
            ds = 2.5 * dw * p * not_p
    return torch.zeros_like(l).scatter_add_(1, at, ds).to(s["logits"].dtype)


def _ranks(ids, E):
    """For each entry its expert (E where it has none), and its rank among the expert's entries in order."""
    e = ids.reshape(-1).long()
    e = torch.where((e >= 0) & (e < E), e, torch.full_like(e, E))
    counts = torch.zeros(E + 1, dtype=torch.int64, device=e.device).scatter_add_(0, e, torch.ones_like(e))
    order = torch.sort(e, stable=True).indices
    start = torch.cumsum(counts, 0) - counts
    rank = torch.empty_like(e)
    rank[order] = torch.arange(e.numel(), device=e.device) - start[e[order]]
    return e, rank, counts[:E]


def _layout_contiguous(ids, E, rows):
    e, rank, counts = _ranks(ids, E)
    blocks = (counts + TILE - 1) // TILE
    end = torch.cumsum(blocks, 0)
    first = torch.cat([end - blocks, end[-1:]])
    slot = torch.where(e < E, first[e] * TILE + rank, torch.full_like(e, -1))
    b = torch.arange(rows // TILE, device=ids.device)
    owner = (b[:, None] >= end[None, :]).sum(dim=1)
    m_indices = torch.where(owner < E, owner, torch.full_like(owner, -1))
    return slot.view(ids.shape).to(torch.int32), m_indices.to(torch.int32), counts.to(torch.int32)


def _layout_masked(ids, E, cap):
    e, rank, counts = _ranks(ids, E)
    slot = torch.where((e < E) & (rank < cap), e * cap + rank, torch.full_like(e, -1))
    return slot.view(ids.shape).to(torch.int32), counts.clamp_max(cap).to(torch.int32)


def _pad_rows(c, m_indices, slot, rows):
    """The contiguous layout's rows inside used blocks that no entry fills."""
    pad = (m_indices >= 0).repeat_interleave(TILE)
    pad = torch.cat([pad, torch.zeros(1, dtype=torch.bool, device=pad.device)])
    pad[slot] = False
    return pad


def _dispatch(s):
    c, x = s["c"], s["x"]
    rows, k = _rows(c), c["k"]
    if c["layout"] == "contiguous":
        lay = _layout_contiguous(s["ids"], c["E"], rows)
    else:
        lay = _layout_masked(s["ids"], c["E"], c["cap"])
    slot = lay[0].reshape(-1).long()
    slot = torch.where(slot >= 0, slot, torch.full_like(slot, rows))
    q, sc = _quant_1x128(x)
    tok = torch.arange(c["T"], device=x.device).repeat_interleave(k)
    s["q"].view(torch.uint8)[slot] = q.view(torch.uint8)[tok]
    s["s"][slot] = sc[tok]
    if c["layout"] == "contiguous":
        pad = _pad_rows(c, lay[1], slot, rows)
        s["q"].view(torch.uint8).masked_fill_(pad[:, None], 0)
        s["s"].masked_fill_(pad[:, None], 1.0)
    return list(lay) + [s["q"][:rows], s["s"][:rows]]


def _combine(s):
    slot, y, w = s["slots"].long(), s["y"], s["w"]
    v = torch.where((slot >= 0)[:, :, None], y[slot.clamp_min(0)].float(), torch.zeros((), device=y.device))
    if w is not None:
        v = v * w[:, :, None]
    return v.sum(dim=1).to(torch.bfloat16)


def _combine_bwd(s):
    c, slot, y, w, dout = s["c"], s["slots"].long(), s["y"], s["w"], s["dout"].float()
    rows = _rows(c)
    has = slot >= 0
    g = dout[:, None, :] * w[:, :, None]
    flat = torch.where(has, slot, torch.full_like(slot, rows)).reshape(-1)
    s["dy"][flat] = g.to(torch.bfloat16).view(-1, c["D"])
    s["dy"].masked_fill_(_pad_rows(c, s["m_indices"], flat, rows)[:, None], 0)
    dw = (y[slot.clamp_min(0)].float() * dout[:, None, :]).sum(dim=2)
    return s["dy"][:rows], torch.where(has, dw, torch.zeros_like(dw))


def _ckpt_store(s):
    """h is the correctly rounded bf16 of silu(gate) * up: 64 bits decide next to a rounding border."""
    c1, n = s["c1"], s["c"]["inter"]
    g, u = c1[:, :n].double(), c1[:, n:].double()
    h = _round_bf16(g / (1.0 + torch.exp(-g)) * u)
    return list(_quant_1x128(h)) + list(_quant_1x128(c1))


def _dequant(q, s):
    return (q.float().view(q.shape[0], -1, TILE) * s[:, :, None]).view(q.shape)


def _ckpt_bwd(s):
    n = s["c"]["inter"]
    c1, dh = _dequant(s["qc"], s["sc"]), s["dh"].float()
    g, u = c1[:, :n], c1[:, n:]
    p = 1.0 / (1.0 + torch.exp(-g))
    dg = dh * u * (p * (1.0 + g * (1.0 - p)))
    du = dh * (g * p)
    dc = torch.cat([dg, du], dim=1)
    return [dc.to(torch.bfloat16)] + list(_quant_1x128(dc))


def _ckpt_t(s):
    q, sc = s["q"], s["s"]
    M, K = q.shape
    Mp = -(-M // 512) * 512
    v = torch.zeros((Mp, K), device=q.device)
    v[:M] = _dequant(q, sc)
    v = v.view(Mp // TILE, TILE, K)
    st = _scale(v.abs().amax(dim=1))
    qt = _e4m3(v / st[:, None, :]).view(Mp, K)
    return qt.view(torch.uint8).t().contiguous().view(torch.float8_e4m3fn), st


_PLAIN = {"route": _route, "route_bwd": _route_bwd, "dispatch": _dispatch, "combine": _combine,
          "combine_bwd": _combine_bwd, "ckpt_store": _ckpt_store, "ckpt_bwd": _ckpt_bwd, "ckpt_t": _ckpt_t}


# ------------------------------------------------------------------ the library's calls
def _own(s):
    import fp8_fine_grained_quant_b200 as fq
    c = s["c"]
    op = c["op"]
    if op == "route":
        return fq.fp8_moe_route(s["logits"], c["k"], bias=s["bias"], score=c["score"], n_group=c["groups"],
                                topk_group=c["kept"], group_top=c["group_top"], renorm=c["renorm"], scale=2.5)
    if op == "route_bwd":
        return fq.fp8_moe_route_bwd(s["logits"], s["ids"], s["dw"], score=c["score"], renorm=c["renorm"], scale=2.5)
    if op == "dispatch":
        rows = _rows(c)
        q, sc = s["q"][:rows], s["s"][:rows]
        if c["layout"] == "contiguous":
            slots, m_indices, counts = fq.fp8_moe_layout_contiguous(s["ids"], c["E"])
            fq.fp8_moe_dispatch_1x128(s["x"], slots, rows, m_indices=m_indices, counts=counts, q=q, s=sc)
            return slots, m_indices, counts, q, sc
        slots, masked_m = fq.fp8_moe_layout_masked(s["ids"], c["E"], c["cap"])
        fq.fp8_moe_dispatch_1x128(s["x"], slots, rows, q=q, s=sc)
        return slots, masked_m, q, sc
    if op == "combine":
        return fq.fp8_moe_combine(s["y"], s["slots"], s["w"])
    if op == "combine_bwd":
        dy = s["dy"][:_rows(c)]
        return fq.fp8_moe_combine_bwd(s["dout"], s["y"], s["slots"], s["w"], m_indices=s["m_indices"],
                                      counts=s["counts"], dy=dy)
    if op == "ckpt_store":
        (qh, sh), (qc, sc) = fq.fp8_swiglu_ckpt_1x128(s["c1"])
        return qh, sh, qc, sc
    if op == "ckpt_bwd":
        dc, (q, sc) = fq.fp8_swiglu_bwd_1x128(s["dh"], s["qc"], s["sc"])
        return dc, q, sc
    return fq.fp8_ckpt_128x1_t(s["q"], s["s"])


def run(s):
    return _own(s) if own else _PLAIN[s["c"]["op"]](s)


# ------------------------------------------------------------------ the definitions in 64 bits
def _x_e4m3(v):
    """Nearest E4M3 value (ties to even) of 64-bit values, from the format: 3 mantissa bits, least exponent -6."""
    a = v.abs().clamp_max(448.0)
    _, e = torch.frexp(a)
    step = torch.ldexp(torch.ones_like(a), torch.clamp(e - 1, min=-6) - 3)
    return torch.sign(v) * torch.round(a / step) * step


def _x_groups(v):
    """Values and scales of groups along the last axis: s = fl32(amax / 448), q = E4M3(fl32(x / s))."""
    s = (v.abs().amax(dim=-1, keepdim=True) / 448.0).float().double()
    s = torch.where(s > 0, s, torch.ones_like(s))
    return _x_e4m3((v / s).float().double()), s.squeeze(-1)


def _x_quant(x):
    q, s = _x_groups(x.view(x.shape[0], -1, TILE))
    return q.view(x.shape), s


def _x_route(s):
    c = s["c"]
    l = s["logits"].double()
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    if c["score"] == "softmax":
        p = torch.nan_to_num(torch.exp(torch.log_softmax(l, dim=1)), nan=0.0)
    else:
        p = torch.sigmoid(l)
    key = p if s["bias"] is None else p + s["bias"].double()
    key = key.masked_fill(l == NEG, NEG)
    if G > 1:
        first = torch.topk(key.view(T, G, E // G), c["group_top"], dim=2).values
        total = first.masked_fill(first == NEG, 0.0).sum(dim=2).masked_fill(first[:, :, 0] == NEG, NEG)
        a, b = total[:, :, None], total[:, None, :]
        lower = torch.tril(torch.ones((G, G), dtype=torch.bool, device=l.device), diagonal=-1)
        place = ((b > a) | ((b == a) & lower)).sum(dim=2)  # groups ahead of this one
        key = key.view(T, G, E // G).masked_fill((place >= c["kept"])[:, :, None], NEG).view(T, E)
    got = torch.topk(key, k, dim=1)
    w = torch.gather(p, 1, got.indices) * (got.values > NEG)
    if c["renorm"]:
        w = torch.nan_to_num(w / w.sum(dim=1, keepdim=True))
    return [None, 2.5 * w]


def _x_route_bwd(s):
    """Jacobian-vector products by automatic differentiation of the forward formulas in 64 bits."""
    c = s["c"]
    l = s["logits"].double().requires_grad_(True)
    p = torch.softmax(l, dim=1) if c["score"] == "softmax" else torch.sigmoid(l)
    w = torch.gather(p, 1, s["ids"].long())
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return torch.autograd.grad((2.5 * w * s["dw"].double()).sum(), l)[0]


def _x_slots(s):
    """The layouts by counting, on the host."""
    import numpy as np
    c = s["c"]
    ids = s["ids"].cpu().numpy().reshape(-1)
    E = c["E"]
    slot = np.full(ids.size, -1, dtype=np.int64)
    at = 0
    rows = _rows(c)
    pad = np.zeros(rows, dtype=bool)
    for e in range(E):
        mine = np.flatnonzero(ids == e)
        if c["layout"] == "masked":
            mine = mine[:c["cap"]]
            slot[mine] = e * c["cap"] + np.arange(mine.size)
        else:
            slot[mine] = at + np.arange(mine.size)
            end = at + -(-mine.size // TILE) * TILE
            pad[at + mine.size:end] = True
            at = end
    return torch.from_numpy(slot).to(DEV), torch.from_numpy(pad).to(DEV)


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op == "route":
        return _x_route(s)
    if op == "route_bwd":
        return _x_route_bwd(s)
    if op in ("dispatch", "combine", "combine_bwd"):
        slot, pad = _x_slots(s)
        got = torch.nonzero(slot >= 0).squeeze(1)
        tok, row = got // c["k"], slot[got]
        rows, D = _rows(c), c["D"]
        if op == "dispatch":
            qx, sx = _x_quant(s["x"].double())
            q = torch.zeros((rows, D), dtype=torch.float64, device=DEV)
            sc = torch.zeros((rows, D // TILE), dtype=torch.float64, device=DEV)
            q[row], sc[row] = qx[tok], sx[tok]
            sc[pad] = 1.0
            return [None] * (3 if c["layout"] == "contiguous" else 2) + [q, sc]
        w = s["w"].double().view(-1)[got] if s["w"] is not None else torch.ones(got.numel(), dtype=torch.float64, device=DEV)
        if op == "combine":
            out = torch.zeros((c["T"], D), dtype=torch.float64, device=DEV)
            return out.index_add_(0, tok, s["y"][row].double() * w[:, None])
        dy = torch.zeros((rows, D), dtype=torch.float64, device=DEV)
        do = s["dout"].double()[tok]
        dy[row] = do * w[:, None]
        dw = torch.zeros(c["T"] * c["k"], dtype=torch.float64, device=DEV)
        dw[got] = (do * s["y"][row].double()).sum(dim=1)
        return dy, dw.view(c["T"], c["k"])
    if op == "ckpt_store":
        v, n = s["c1"].double(), c["inter"]
        h = v[:, :n] * torch.sigmoid(v[:, :n]) * v[:, n:]
        # one rounding to 8 significant bits (the values are far from bf16's least exponent)
        m, e = torch.frexp(h)
        h = torch.ldexp(torch.round(m * 256.0), e - 8)
        return list(_x_quant(h)) + list(_x_quant(v))
    if op == "ckpt_bwd":
        n = c["inter"]
        v = (s["qc"].double().view(c["rows"], -1, TILE) * s["sc"].double()[:, :, None]).float().double()
        v = v.view(c["rows"], 2 * n)
        g, u, dh = v[:, :n], v[:, n:], s["dh"].double()
        p = torch.sigmoid(g)
        dc = torch.cat([dh * u * p * (1.0 + g * torch.sigmoid(-g)), dh * g * p], dim=1)
        return [dc] + list(_x_quant(dc))
    M, K = c["rows"], c["K"]
    Mp = -(-M // 512) * 512
    v = torch.zeros((Mp, K), dtype=torch.float64, device=DEV)
    v[:M] = (s["q"].double().view(M, -1, TILE) * s["s"].double()[:, :, None]).float().double().view(M, K)
    q, st = _x_groups(v.t().contiguous().view(K, Mp // TILE, TILE))
    return q.view(K, Mp), st.t().contiguous()
