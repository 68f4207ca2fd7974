"""What stands between the FP8 products of a transformer block with experts, as
measured cases: each operator's plain form in elementary torch operations, the
same call through the library (``own``), and its value in 64 bits.

Operators
  norm      RMSNorm with the residual's addition, e4m3 codes with 1 x 128
            scales (and bf16), and its gradient
  gate      experts and routing weights of every token from the gate's logits
  balance   per-expert counts and the balance loss of every sequence, and the
            gradient of the loss and of the routing weights by the logits
  swiglu    silu(gate) * up between the grouped products, e4m3 codes with
            1 x 128 scales, and its gradient
  combine   the gradient of the weighted sum of the experts' rows

Shapes are those of the pages' configurations: 7168 wide, 256 experts in 8
groups of which 4 are kept, 8 experts a token, 2048 wide experts; and 2048
wide, 64 experts without groups, 6 a token.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 128
EPS = 1e-6
FP8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one user's token in front of an attention block: latency
        dict(op="norm", name="norm 1 x 7168 ue8m0", rows=1, width=7168, ld=7168, res="bf16", fmt="ue8m0", y=False),
        # a prefill in front of the expert block: codes for the shared expert, bf16 for the gate and the dispatch
        dict(op="norm", name="norm 4096 x 7168", rows=4096, width=7168, ld=7168, res="bf16", fmt="fp32", y=True),
        # the same norm in a training step, with the gradient that goes past the block
        dict(op="norm_bwd", name="norm gradient 4096 x 7168", rows=4096, width=7168, h="bf16", dres=True),
        # a decode batch's gate: latency
        dict(op="gate", name="gate 32 x 256", rows=32, experts=256, topk=8, groups=8, keep=4, bias=True,
             score="sigmoid", dtype="f32", masked=False),
        # a prefill's gate
        dict(op="gate", name="gate 4096 x 256", rows=4096, experts=256, topk=8, groups=8, keep=4, bias=True,
             score="sigmoid", dtype="f32", masked=False),
        # a training batch of several packed sequences, both gradients into the logits
        dict(op="balance", name="balance 4096 x 256, 5 sequences", rows=4096, experts=256, topk=8, score="sigmoid",
             dtype="f32", seqs=5, weights=True),
        # one sequence of an odd length in the small model, the loss alone
        dict(op="balance", name="balance 999 x 64", rows=999, experts=64, topk=6, score="softmax", dtype="bf16",
             seqs=1, weights=False),
        # one token's 8 experts: latency
        dict(op="swiglu", name="swiglu 8 x 2048 ue8m0", rows=8, used=8, width=2048, fmt="ue8m0", y=False),
        # a prefill's routed rows
        dict(op="swiglu", name="swiglu 32768 x 2048", rows=32768, used=32768, width=2048, fmt="fp32", y=False),
        # a training step's routed rows in a buffer for more of them
        dict(op="swiglu_bwd", name="swiglu gradient 29999 x 2048", rows=32768, used=29999, width=2048),
        # the small model's combine, an odd number of tokens, some pairs on no expert
        dict(op="combine", name="combine gradient 999 x 6 x 2048", rows=999, topk=6, width=2048, dropped=0.05,
             dtype="f32"),
        # a training step's combine
        dict(op="combine", name="combine gradient 4096 x 8 x 7168", rows=4096, topk=8, width=7168, dropped=0.0,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "gate", "gate", "balance", "balance", "swiglu", "swiglu_bwd",
                     "combine"])
    c = dict(op=op)
    if op in ("norm", "norm_bwd"):
        c["width"] = BLOCK * _log(rng, 1, 144)
        c["rows"] = _log(rng, 1, min(16384, 2 * 4096 * 7168 // c["width"]))
        if op == "norm":
            # power-of-two scales in serving batches; larger ones may meet a border in 32 bits
            c["fmt"] = rng.choice(["fp32", "ue8m0", "none"]) if c["rows"] * c["width"] < 1 << 21 else rng.choice(
                ["fp32", "none"])
            c["y"] = c["fmt"] == "none" or rng.random() < 0.4
            c["res"] = rng.choice(["none", "bf16", "f32"])
            c["ld"] = c["width"] + rng.choice([0, 0, 8, 576])
        else:
            c["h"] = rng.choice(["bf16", "f32"])
            c["dres"] = rng.random() < 0.6
        return c
    if op in ("gate", "balance"):
        c["experts"] = rng.choice([5, 8, 16, 60, 64, 72, 128, 160, 256, 256, 384, 512])
        c["topk"] = min(c["experts"], rng.choice([1, 2, 4, 6, 8, 8, 9]))
        c["rows"] = _log(rng, 1, min(30000, 8 * 4096 * 256 // c["experts"]))
        c["score"] = rng.choice(["sigmoid", "softmax"])
        c["dtype"] = rng.choice(["f32", "f32", "bf16"])
        if op == "gate":
            c["groups"] = rng.choice([g for g in (1, 1, 2, 4, 8, 8) if c["experts"] % g == 0])
            c["keep"] = rng.randint(max(1, c["groups"] // 2), c["groups"])
            c["topk"] = min(c["topk"], c["experts"] // c["groups"] * c["keep"])
            c["bias"] = rng.random() < 0.6
            c["masked"] = rng.random() < 0.3
        else:
            c["seqs"] = _log(rng, 1, 64)
            c["weights"] = rng.random() < 0.7
        return c
    if op in ("swiglu", "swiglu_bwd"):
        c["width"] = BLOCK * _log(rng, 2, 144)
        c["rows"] = _log(rng, 1, 32768 * 2048 // c["width"])
        c["used"] = c["rows"] if rng.random() < 0.5 else rng.randint(1, c["rows"])
        if op == "swiglu":
            c["fmt"] = rng.choice(["fp32", "ue8m0", "none"]) if c["rows"] * c["width"] < 1 << 21 else rng.choice(
                ["fp32", "none"])
            c["y"] = c["fmt"] == "none" or rng.random() < 0.3
        return c
    c["topk"] = rng.choice([1, 2, 4, 6, 8, 8])
    c["width"] = rng.choice([BLOCK * _log(rng, 1, 56), BLOCK * _log(rng, 1, 56), rng.randint(1, 4000)])
    c["rows"] = _log(rng, 1, min(8192, 4096 * 8 * 7168 // (c["width"] * c["topk"])))
    c["dropped"] = rng.choice([0.0, 0.0, 0.1])
    c["dtype"] = rng.choice(["bf16", "f32"])
    return c


# ----------------------------------------------------------------- the inputs

def _f32(shape, gen, std=1.0):
    return torch.randn(shape, dtype=torch.float32, device=DEV, generator=gen).mul_(std)


def _typed(t, name):
    return t.to(torch.bfloat16) if name == "bf16" else t


def _bounds(case, seed):
    """Boundaries of the packed sequences: the case's lengths, in an order of the seed's."""
    r = random.Random("%d %d" % (case["rows"], case["seqs"]))
    cuts = sorted(r.randint(0, case["rows"]) for _ in range(case["seqs"] - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [case["rows"]])]
    random.Random(seed * 7919 + 17).shuffle(lens)
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def _routed(case):
    pairs = case["rows"] * case["topk"]
    return pairs - int(pairs * case["dropped"])


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, n = case["op"], case["rows"]
    s = dict(case)
    if op in ("norm", "norm_bwd"):
        K = case["width"]
        s["w"] = _typed(torch.rand(K, device=DEV, generator=gen) + 0.5, "bf16")
        if op == "norm":
            # the norm's input may be a slice of a wider product's output
            s["x"] = _typed(_f32((n, case["ld"]), gen), "bf16")[:, :K]
            s["r"] = None if case["res"] == "none" else _typed(_f32((n, K), gen, 3.0), case["res"])
        else:
            s["dy"] = _typed(_f32((n, K), gen, 0.1), "bf16")
            s["x"] = _typed(_f32((n, K), gen, 3.0), case["h"])
            s["r"] = _typed(_f32((n, K), gen, 0.1), case["h"]) if case["dres"] else None
        return s
    if op in ("gate", "balance"):
        E = case["experts"]
        # experts differ in how much they are asked for
        z = _f32((n, E), gen, 1.2) + _f32((E,), gen, 0.5)
        if op == "gate":
            if case["masked"]:
                z.masked_fill_(torch.rand((n, E), device=DEV, generator=gen) < 0.2, -math.inf)
            s["b"] = _f32((E,), gen, 0.1) if case["bias"] else None
            s["z"] = _typed(z, case["dtype"])
            return s
        s["z"] = _typed(z, case["dtype"])
        s["idx"] = s["z"].float().sort(dim=-1, descending=True, stable=True)[1][:, :case["topk"]].to(torch.int32).contiguous()
        at = _bounds(case, seed)
        s["cu"] = torch.tensor(at, dtype=torch.int32, device=DEV)
        s["d_loss"] = torch.rand(case["seqs"], device=DEV, generator=gen) + 0.5
        s["dw"] = _f32((n, case["topk"]), gen, 0.01) if case["weights"] else None
        return s
    if op in ("swiglu", "swiglu_bwd"):
        N = case["width"]
        s["gu"] = _typed(_f32((n, 2 * N), gen, 1.5), "bf16")
        s["count"] = torch.tensor([case["used"]], dtype=torch.int32, device=DEV)
        if op == "swiglu_bwd":
            s["dy"] = _typed(_f32((n, N), gen, 0.1), "bf16")
            s["dgu"] = torch.zeros((n, 2 * N), dtype=torch.bfloat16, device=DEV)
            return s
        s["out"] = torch.zeros((n, N), dtype=torch.bfloat16, device=DEV) if case["y"] else None
        s["q"] = s["s"] = None
        if case["fmt"] != "none":
            s["q"] = torch.zeros((n, N), dtype=torch.uint8, device=DEV).view(FP8)
            s["s"] = torch.zeros((n, N // BLOCK), dtype=torch.float32, device=DEV)
        return s
    k, N = case["topk"], case["width"]
    R = _routed(case)
    # rows lie by expert: a token's pairs are far from one another
    order = torch.randperm(n * k, device=DEV, generator=gen)[:R]
    row_of = torch.full((n * k,), -1, dtype=torch.int32, device=DEV)
    row_of[order] = torch.arange(R, dtype=torch.int32, device=DEV)
    s["row_of"] = row_of.view(n, k)
    s["dy"] = _typed(_f32((n, N), gen, 0.1), case["dtype"])
    s["out"] = _typed(_f32((R, N), gen), "bf16")
    w = torch.rand((n, k), device=DEV, generator=gen) + 0.05
    s["w"] = w / w.sum(-1, keepdim=True)
    return s


# ------------------------------------------------------------ the plain forms

def _quantised(c, fmt):
    """(codes, scales) of each 128 values, as act_quant makes them."""
    b = c.view(c.shape[0], -1, BLOCK)
    k = b.abs().amax(-1).clamp(min=1e-4) / 448
    if fmt == "ue8m0":
        m, e = torch.frexp(k)
        k = torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e))
    return (b / k[..., None]).clamp(-448, 448).to(FP8).view(c.shape), k


def _plain_norm(s):
    t = s["x"].float()
    if s["r"] is not None:
        t = t + s["r"].float()
    c = t * (1 / (t.square().mean(-1, keepdim=True) + EPS).sqrt()) * s["w"].float()
    got = [] if s["fmt"] == "none" else list(_quantised(c, s["fmt"]))
    if s["y"]:
        got.append(c.to(torch.bfloat16))
    if s["r"] is not None:
        got.append(t.to(s["r"].dtype))
    return got


def _plain_norm_bwd(s):
    h, dy = s["x"].float(), s["dy"].float()
    r = 1 / (h.square().mean(-1, keepdim=True) + EPS).sqrt()
    g = dy * s["w"].float()
    dx = r * (g - h * (r.square() * (g * h).mean(-1, keepdim=True)))
    if s["r"] is not None:
        dx = dx + s["r"].float()
    return [dx.to(s["x"].dtype), (dy * h * r).sum(0)]


def _scores(z, kind):
    """Scores in 64 bits: those next to each other decide who is chosen."""
    z = z.double()
    if kind == "sigmoid":
        return 1 / (1 + (-z).exp())
    top = z.amax(-1, keepdim=True)
    e = (z - torch.where(top == -math.inf, torch.zeros_like(top), top)).exp()
    tot = e.sum(-1, keepdim=True)
    return torch.where(tot > 0, e / tot, torch.zeros_like(e))


def _plain_gate(s):
    z = s["z"].float()
    T, E = z.shape
    score = _scores(z, s["score"]).float()
    key = z
    if s["b"] is not None:
        key = torch.where(z > -math.inf, score + s["b"], z)
    if s["groups"] > 1:
        by = key.view(T, s["groups"], -1)
        if s["b"] is None:
            val = by.amax(-1)
        else:
            two = by.sort(-1, descending=True)[0][..., :2]
            val = torch.where(two > -math.inf, two, torch.zeros_like(two)).sum(-1)
            val = torch.where(two[..., 0] > -math.inf, val, two[..., 0])
        best = val.sort(dim=-1, descending=True, stable=True)[1][:, :s["keep"]]
        kept = torch.zeros((T, s["groups"]), dtype=torch.bool, device=DEV)
        kept[torch.arange(T, device=DEV)[:, None], best] = True
        key = torch.where(kept[..., None], by, torch.full_like(by, -math.inf)).view(T, E)
    top, idx = key.sort(dim=-1, descending=True, stable=True)
    top, idx = top[:, :s["topk"]], idx[:, :s["topk"]]
    w = torch.where(top > -math.inf, score.gather(1, idx), torch.zeros_like(top))
    tot = w.sum(-1, keepdim=True)
    w = torch.where(tot > 0, w / tot, torch.zeros_like(w)) * 2.5
    return [torch.where(top > -math.inf, idx, -1).to(torch.int32), w]


def _plain_balance(s):
    z, idx, S, k = s["z"].float(), s["idx"].long(), s["seqs"], s["topk"]
    T, E = z.shape
    score = _scores(z, s["score"]).float()
    cu = s["cu"].long()
    seq = torch.searchsorted(cu, torch.arange(T, device=DEV), right=True) - 1
    n = (cu[1:] - cu[:-1]).float()
    some = n.clamp(min=1)
    hit = torch.zeros((T, E), device=DEV)
    hit.scatter_(1, idx, 1.0)
    tot = score.sum(-1, keepdim=True)
    share = score / tot
    member = seq == torch.arange(S, device=DEV)[:, None]
    counts = torch.matmul(member.float(), hit)
    probs = torch.matmul(member.double(), share.double()).float() / some[:, None]
    loss = (counts * probs).sum(-1) * (E / (k * some))
    g = (counts * (s["d_loss"] * E / (k * some * some))[:, None])[seq]
    d = (g - (g * share).sum(-1, keepdim=True)) / tot            # by the scores
    if s["dw"] is not None:
        w = score.gather(1, idx)
        all_w = w.sum(-1, keepdim=True)
        dw = 2.5 / all_w * (s["dw"] - (s["dw"] * w).sum(-1, keepdim=True) / all_w)
        d = d.scatter_add(1, idx, dw)
    if s["score"] == "sigmoid":
        dz = d * score * (1 - score)
    else:
        dz = score * (d - (d * score).sum(-1, keepdim=True))
    return [loss, counts.to(torch.int32), probs, dz.to(s["z"].dtype)]


def _plain_swiglu(s):
    N = s["width"]
    g, u = s["gu"][:, :N].float(), s["gu"][:, N:].float()
    a = g * (1 / (1 + (-g).exp())) * u
    live = torch.arange(s["rows"], device=DEV)[:, None] < s["count"]
    got = []
    if s["q"] is not None:
        q, k = _quantised(a, s["fmt"])
        b = s["q"].view(torch.uint8)
        b.copy_(torch.where(live, q.view(torch.uint8), b))
        s["s"].copy_(torch.where(live, k, s["s"]))
        got += [s["q"], s["s"]]
    if s["out"] is not None:
        s["out"].copy_(torch.where(live, a.to(torch.bfloat16), s["out"]))
        got.append(s["out"])
    return got


def _plain_swiglu_bwd(s):
    N = s["width"]
    g, u, dy = s["gu"][:, :N].float(), s["gu"][:, N:].float(), s["dy"].float()
    sig = 1 / (1 + (-g).exp())
    live = torch.arange(s["rows"], device=DEV)[:, None] < s["count"]
    d = torch.cat((dy * u * sig * (1 + g * (1 - sig)), dy * g * sig), 1).to(torch.bfloat16)
    s["dgu"].copy_(torch.where(live, d, s["dgu"]))
    return [s["dgu"]]


def _plain_combine(s):
    rows = s["row_of"].long()
    dy, w, out = s["dy"].float(), s["w"], s["out"]
    d_out = torch.zeros((out.shape[0] + 1, out.shape[1]), dtype=torch.bfloat16, device=DEV)
    d_w = []
    for k in range(s["topk"]):
        r = rows[:, k]
        on = r >= 0
        d_w.append(torch.where(on, (dy * out[r.clamp(min=0)].float()).sum(-1), torch.zeros_like(w[:, k])))
        d_out[torch.where(on, r, out.shape[0])] = (w[:, k, None] * dy).to(torch.bfloat16)
    return [d_out[:-1], torch.stack(d_w, 1)]


# ---------------------------------------------------------------- the library

def _own(s):
    import block_scaled_fp8_03_amd as fp8bs
    op = s["op"]
    if op == "norm":
        if s["fmt"] == "none":
            got = fp8bs.rmsnorm(s["x"], s["w"], EPS, s["r"])
            return [got] if s["r"] is None else list(got)
        return list(fp8bs.rmsnorm_quant(s["x"], s["w"], EPS, s["r"], s["fmt"], return_y=s["y"]))
    if op == "norm_bwd":
        return list(fp8bs.rmsnorm_bwd(s["dy"], s["x"], s["w"], EPS, s["r"]))
    if op == "gate":
        return list(fp8bs.moe_gate(s["z"], s["topk"], s["b"], s["groups"], s["keep"], s["score"], route_scale=2.5))
    if op == "balance":
        loss, counts, probs = fp8bs.moe_balance(s["z"], s["idx"], s["cu"], s["score"])
        dz = fp8bs.moe_gate_bwd(s["z"], s["idx"], s["dw"], s["score"], route_scale=2.5, cu_seq=s["cu"], counts=counts,
                                d_loss=s["d_loss"], out_dtype=s["z"].dtype)
        return [loss, counts, probs, dz]
    if op in ("swiglu", "swiglu_bwd"):
        N = s["width"]
        g, u = s["gu"][:, :N], s["gu"][:, N:]
        if op == "swiglu_bwd":
            fp8bs.fp8bs_swiglu_bwd(s["dy"], g, u, s["dgu"][:, :N], s["dgu"][:, N:], s["count"])
            return [s["dgu"]]
        fp8bs.fp8bs_swiglu(g, u, s["out"], s["q"], s["s"], "fp32" if s["fmt"] == "none" else s["fmt"], s["count"])
        return [t for t in (s["q"], s["s"], s["out"]) if t is not None]
    return list(fp8bs.moe_combine_bwd(s["dy"], s["out"], s["w"], s["row_of"]))


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "gate": _plain_gate, "balance": _plain_balance,
            "swiglu": _plain_swiglu, "swiglu_bwd": _plain_swiglu_bwd, "combine": _plain_combine}[state["op"]](state)


# ------------------------------------------------------------------- the work

def work(case):
    op, n = case["op"], case["rows"]
    size = {"bf16": 2, "f32": 4, "none": 0}
    if op == "norm":
        K = case["width"]
        per = 2 + 2 * size[case["res"]] + 2 * case["y"] + (case["fmt"] != "none") * (1 + 4 / BLOCK)
        return {"bytes": n * K * per + 2 * K, "flops": 10 * n * K}
    if op == "norm_bwd":
        K = case["width"]
        return {"bytes": n * K * (2 + size[case["h"]] * (2 + case["dres"])) + 6 * K, "flops": 14 * n * K}
    if op in ("gate", "balance"):
        E, k, b = case["experts"], case["topk"], size[case["dtype"]]
        if op == "gate":
            return {"bytes": n * (E * b + 8 * k) + 4 * E, "flops": 12 * n * E}
        return {"bytes": n * (2 * E * b + k * (8 if case["weights"] else 4)) + 8 * case["seqs"] * E, "flops": 30 * n * E}
    if op == "swiglu":
        per = 4 + 2 * case["y"] + (case["fmt"] != "none") * (1 + 4 / BLOCK)
        return {"bytes": case["used"] * case["width"] * per + 4, "flops": 10 * case["used"] * case["width"]}
    if op == "swiglu_bwd":
        return {"bytes": 10 * case["used"] * case["width"] + 4, "flops": 16 * case["used"] * case["width"]}
    k, N, b = case["topk"], case["width"], size[case["dtype"]]
    rows = _routed(case)
    return {"bytes": rows * 4 * N + n * N * b + 12 * n * k, "flops": 3 * rows * N}


# ------------------------------------------------------------ values in 64 bits

def _exact_codes(c, fmt):
    g = c.unflatten(-1, (-1, BLOCK))
    k = g.abs().amax(-1).clamp(min=1e-4) / 448
    if fmt == "ue8m0":
        k = torch.exp2(torch.ceil(torch.log2(k)))
    return [(g / k[..., None]).flatten(-2), k]


def _exact_norm(s):
    t = s["x"].double() if s["r"] is None else s["x"].double() + s["r"].double()
    c = t / torch.linalg.vector_norm(t, dim=-1, keepdim=True).square().div(s["width"]).add(EPS).sqrt() * s["w"].double()
    got = [] if s["fmt"] == "none" else _exact_codes(c, s["fmt"])
    return got + ([c] if s["y"] else []) + ([] if s["r"] is None else [t])


def _exact_norm_bwd(s):
    h, w = s["x"].double().requires_grad_(), s["w"].double().requires_grad_()
    y = h / (h.pow(2).sum(-1, keepdim=True) / s["width"] + EPS).sqrt() * w
    dh, dw = torch.autograd.grad(y, (h, w), s["dy"].double())
    return [dh if s["r"] is None else dh + s["r"].double(), dw]


def _exact_gate(s):
    """Token by token in the order of the definition: float32 keys, lowest index first among equals."""
    z = s["z"].double().cpu().numpy()
    T, E = z.shape
    if s["score"] == "sigmoid":
        p = 1 / (1 + np.exp(-z))
    else:
        e = np.exp(z - np.maximum(z.max(1, keepdims=True), -1e300))
        p = e / np.maximum(e.sum(1, keepdims=True), 1e-300)
    key = z.astype(np.float32)
    if s["b"] is not None:
        key = np.where(np.isinf(z), np.float32(-np.inf), p.astype(np.float32) + s["b"].cpu().numpy())
    G = s["groups"]
    idx, w = np.full((T, s["topk"]), -1, np.int32), np.zeros((T, s["topk"]))
    for t in range(T):
        row = key[t]
        if G > 1:
            parts = np.sort(row.reshape(G, -1), 1)[:, ::-1]
            val = parts[:, 0].copy()
            if s["b"] is not None and parts.shape[1] > 1:
                val = np.where(np.isinf(parts[:, 1]), val, val + parts[:, 1])
            out = np.argsort(-val, kind="stable")[s["keep"]:]
            row = row.reshape(G, -1).copy()
            row[out] = -np.inf
            row = row.ravel()
        at = [i for i in np.argsort(-row, kind="stable")[:s["topk"]] if row[i] > -np.inf]
        idx[t, :len(at)], w[t, :len(at)] = at, p[t, at]
    tot = w.sum(1, keepdims=True)
    return [torch.from_numpy(idx), torch.from_numpy(2.5 * w / np.where(tot > 0, tot, 1))]


def _exact_balance(s):
    z = s["z"].double().requires_grad_()
    idx, k, E, at = s["idx"].long(), s["topk"], s["experts"], s["cu"].tolist()
    p = torch.special.expit(z) if s["score"] == "sigmoid" else torch.softmax(z, -1)
    share = p / p.sum(-1, keepdim=True)
    loss, counts, probs = [], [], []
    for a, b in zip(at, at[1:]):
        n = torch.bincount(idx[a:b].flatten(), minlength=E)
        m = share[a:b].sum(0) / max(1, b - a)
        loss.append((n.double() * m).sum() * E / (k * max(1, b - a)))
        counts.append(n)
        probs.append(m)
    loss = torch.stack(loss)
    aim = (loss * s["d_loss"].double()).sum()
    if s["dw"] is not None:
        c = p.gather(1, idx)
        aim = aim + (c / c.sum(-1, keepdim=True) * 2.5 * s["dw"].double()).sum()
    dz, = torch.autograd.grad(aim, z)
    return [loss.detach(), torch.stack(counts), torch.stack(probs).detach(), dz]


def _exact_swiglu(s):
    n, N = s["used"], s["width"]
    gu = s["gu"][:n].double()
    a = torch.zeros((s["rows"], N), dtype=torch.float64, device=DEV)
    a[:n] = torch.nn.functional.silu(gu[:, :N]) * gu[:, N:]
    got = []
    if s["q"] is not None:
        q, k = _exact_codes(a, s["fmt"])
        k[n:] = 0
        got += [q, k]
    return got + ([] if s["out"] is None else [a])


def _exact_swiglu_bwd(s):
    n, N = s["used"], s["width"]
    gu = s["gu"][:n].double().requires_grad_()
    d, = torch.autograd.grad(torch.nn.functional.silu(gu[:, :N]) * gu[:, N:], gu, s["dy"][:n].double())
    return [torch.nn.functional.pad(d, (0, 0, 0, s["rows"] - n))]


def _exact_combine(s):
    rows, w = s["row_of"].long().flatten(), s["w"].double().flatten()
    pair = torch.nonzero(rows >= 0)[:, 0]
    d_out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    d_w = torch.zeros_like(w)
    for a in range(0, pair.shape[0], 4096):
        p = pair[a:a + 4096]
        dy = s["dy"][p // s["topk"]].double()
        d_out[rows[p]] = dy * w[p, None]
        d_w[p] = (dy * s["out"][rows[p]].double()).sum(-1)
    return [d_out, d_w.view(s["w"].shape)]


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_bwd": _exact_norm_bwd, "gate": _exact_gate, "balance": _exact_balance,
            "swiglu": _exact_swiglu, "swiglu_bwd": _exact_swiglu_bwd, "combine": _exact_combine}[case["op"]](s)
