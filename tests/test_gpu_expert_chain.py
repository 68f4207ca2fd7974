"""A block with experts, forward and backward, through the library alone: norm with
codes, gate, route, expert products around SwiGLU, combine; then the gradients back
to the residual stream.  Each operator's result is compared with the value in 64 bits
of the very inputs it got; the whole is run in a captured graph, on other streams and
on two at once, and has to give the eager result bit by bit."""
import pytest
import torch

import block_scaled_fp8_03_amd as fp8bs
import expert_util as eu

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
EPS, SCALE = 1e-6, 2.5
T, K, I, E, TOPK, GROUPS, KEEP = 75, 256, 128, 128, 4, 8, 3
CU = [0, 31, 31, 70]                              # the last tokens are in no sequence


class Layer:
    """Weights, as a program keeps them: FP8 both ways round."""

    def __init__(self, seed):
        self.norm_w = (eu.normal((K,), seed, 0.1) + 1).to(DEV)
        self.bias = eu.normal((E,), seed + 1, 0.05, F32).to(DEV)
        self.gate = self._both(eu.normal((E, K), seed + 2, 0.1))
        self.up = self._experts(2 * I, K, seed + 3)
        self.down = self._experts(K, I, seed + 4)
        self.cu = torch.tensor(CU, dtype=torch.int32, device=DEV)
        self.ones = torch.ones((T, TOPK), device=DEV)

    @staticmethod
    def _both(w):
        q, s = fp8bs.weight_quant(w.to(DEV))
        turn = lambda t: t.transpose(-1, -2).contiguous()  # noqa: E731
        return q, s, turn(q.view(torch.uint8)).view(eu.FP8), turn(s)

    def _experts(self, n, k, seed):
        each = [self._both(eu.normal((n, k), 1000 * seed + e, 0.06)) for e in range(E)]
        return tuple(torch.stack([x[i].view(torch.uint8) if i % 2 == 0 else x[i] for x in each]).contiguous()
                     for i in range(4))

    @staticmethod
    def fp8(t):
        return t.view(eu.FP8)

    def forward(self, x, res):
        f = {}
        f["q"], f["s"], f["y"], f["h"] = fp8bs.rmsnorm_quant(x, self.norm_w, EPS, res, return_y=True)
        f["logits"] = fp8bs.w8a16_gemm(f["y"], self.gate[0], self.gate[1], F32)
        f["idx"], f["w"] = fp8bs.moe_gate(f["logits"], TOPK, self.bias, GROUPS, KEEP, route_scale=SCALE)
        f["loss"], f["counts"], f["probs"] = fp8bs.moe_balance(f["logits"], f["idx"], self.cu)
        f["offsets"], _, f["row_of"] = fp8bs.moe_route(f["idx"], E)
        R = T * TOPK
        f["n"] = f["offsets"][-1:]
        xq, xs = fp8bs.moe_quant_scatter(f["y"], f["row_of"], R)
        f["gu"] = fp8bs.moe_gemm(xq, xs, self.fp8(self.up[0]), self.up[1], f["offsets"])
        f["a_q"], f["a_s"], f["a"] = fp8bs.swiglu_quant(f["gu"][:, :I], f["gu"][:, I:], n_rows=f["n"], return_y=True)
        f["out"] = fp8bs.moe_gemm(f["a_q"], f["a_s"], self.fp8(self.down[0]), self.down[1], f["offsets"])
        f["moe"] = fp8bs.moe_combine(f["out"], f["w"], f["row_of"])
        return f

    def backward(self, f, d_moe, d_h, d_loss):
        b = {}
        b["d_out"], b["d_w"] = fp8bs.moe_combine_bwd(d_moe, f["out"], f["w"], f["row_of"])
        q, s = fp8bs.act_quant(b["d_out"])
        b["d_a"] = fp8bs.moe_gemm(q, s, self.fp8(self.down[2]), self.down[3], f["offsets"])
        b["d_gu"] = torch.zeros_like(f["gu"])
        fp8bs.fp8bs_swiglu_bwd(b["d_a"], f["gu"][:, :I], f["gu"][:, I:], b["d_gu"][:, :I], b["d_gu"][:, I:], f["n"])
        q, s = fp8bs.act_quant(b["d_gu"])
        rows = fp8bs.moe_gemm(q, s, self.fp8(self.up[2]), self.up[3], f["offsets"])
        b["d_y"] = fp8bs.moe_combine(rows, self.ones, f["row_of"], F32)
        b["d_logits"] = fp8bs.moe_gate_bwd(f["logits"], f["idx"], b["d_w"], route_scale=SCALE, cu_seq=self.cu,
                                           counts=f["counts"], d_loss=d_loss, out_dtype=BF16)
        b["d_y"] = (b["d_y"] + fp8bs.w8a16_gemm(b["d_logits"], self.gate[2], self.gate[3], F32)).to(BF16)
        b["d_x"], b["d_norm_w"] = fp8bs.rmsnorm_bwd(b["d_y"], f["h"], self.norm_w, EPS, d_h)
        return b


def _inputs(seed):
    return (eu.normal((T, K), seed).to(DEV), eu.normal((T, K), seed + 1, 2.0).to(DEV),
            eu.normal((T, K), seed + 2, 0.1).to(DEV), eu.normal((T, K), seed + 3, 0.1).to(DEV),
            torch.tensor([0.01, 0.02, -0.03], device=DEV))


def _run(layer, x, res, d_moe, d_h, d_loss):
    f = layer.forward(x, res)
    b = layer.backward(f, d_moe, d_h, d_loss)
    n = int(f["n"]) if not torch.cuda.is_current_stream_capturing() else None
    return f, b, n


KEPT = ("q", "s", "y", "h", "logits", "idx", "w", "loss", "counts", "probs", "moe")
GRADS = ("d_w", "d_y", "d_logits", "d_x", "d_norm_w")


def _results(f, b):
    return [f[k].view(torch.uint8) if f[k].dtype == eu.FP8 else f[k] for k in KEPT] + [b[k] for k in GRADS]


@pytest.fixture(scope="module")
def layer():
    return Layer(5)


def test_each_step(layer):
    x, res, d_moe, d_h, d_loss = _inputs(1)
    f, b, n = _run(layer, x, res, d_moe, d_h, d_loss)
    c = {k: v.cpu() for k, v in f.items() if isinstance(v, torch.Tensor)}
    rel = eu.norm_rel(K)
    _, norm = eu.norm(x.cpu(), res.cpu(), layer.norm_w.cpu(), EPS)
    assert torch.equal(c["h"], (x.float() + res.float()).to(BF16).cpu())
    eu.inside(c["y"], norm, norm.abs() * (eu.H_BF16 + rel), "y")
    eu.check_codes(f["q"], f["s"], norm, rel, False, "codes")
    idx, w = eu.gate(c["logits"], TOPK, layer.bias.cpu(), GROUPS, KEEP, "sigmoid", True, SCALE)
    assert torch.equal(c["idx"], idx)
    srel = eu.score_rel(c["logits"], E)
    eu.inside(c["w"], w, w * (2 * srel + TOPK * eu.H_F32), "w")
    loss, counts, probs = eu.balance(c["logits"], c["idx"], CU, "sigmoid")
    assert torch.equal(c["counts"], counts) and n == T * TOPK
    eu.inside(c["loss"], loss, loss * (srel + (T + 64 + E) * eu.H_F32), "loss")
    eu.inside(c["probs"], probs, probs * (srel + (T + 64) * eu.H_F32), "probs")
    a = eu.swiglu(c["gu"][:, :I], c["gu"][:, I:])
    eu.inside(c["a"], a, a.abs() * (eu.H_BF16 + eu.SILU_REL) + 1e-36, "a")
    eu.check_codes(f["a_q"], f["a_s"], a, eu.SILU_REL, False, "a's codes")
    d_out, d_w, size = eu.combine_bwd(d_moe.cpu(), c["out"], c["w"], c["row_of"])
    eu.inside(b["d_out"], d_out, d_out.abs() * (eu.H_BF16 + 2 * eu.H_F32), "d_out")
    eu.inside(b["d_w"], d_w, size * (K / 64 + 16) * eu.H_F32, "d_w")
    dg, dsize, du = eu.swiglu_bwd(b["d_a"].cpu(), c["gu"][:, :I], c["gu"][:, I:])
    eu.inside(b["d_gu"][:, :I], dg, dg.abs() * eu.H_BF16 + dsize * 2 * eu.SILU_REL + 1e-36, "d_gate")
    eu.inside(b["d_gu"][:, I:], du, du.abs() * (eu.H_BF16 + eu.SILU_REL) + 1e-36, "d_up")
    dz, zsize = eu.gate_bwd(c["logits"], c["idx"], b["d_w"].cpu(), "sigmoid", True, SCALE, CU, d_loss.cpu())
    eu.inside(b["d_logits"], dz, dz.abs() * eu.H_BF16 + zsize * (4 * srel + TOPK * eu.H_F32) * 1.01 + 1e-37, "d_logits")
    dx, bound, dw, dw_bound = eu.norm_bwd(b["d_y"].cpu(), c["h"], layer.norm_w.cpu(), EPS, d_h.cpu())
    eu.inside(b["d_x"], dx, dx.abs() * eu.H_BF16 + bound * 1.01, "d_x")
    eu.inside(b["d_norm_w"], dw, dw_bound, "d_norm_w")


def test_captured_and_replayed(layer):
    """Two graphs of the layer, replayed in turn on new inputs, with eager work between."""
    graphs = []
    for seed in (10, 20):
        held = _inputs(seed)
        for _ in range(2):
            _run(layer, *held)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f, b, _ = _run(layer, *held)
            out = _results(f, b)
        graphs.append((g, held, out))
    for turn in range(3):
        for n, (g, held, out) in enumerate(graphs):
            new = _inputs(100 + 10 * turn + n)
            for a, v in zip(held, new):
                a.copy_(v)
            g.replay()
            got = [t.clone() for t in out]
            f, b, _ = _run(layer, *new)
            for k, a, v in zip(KEPT + GRADS, got, _results(f, b)):
                assert torch.equal(a, v), (turn, n, k)


def test_two_streams_at_once(layer):
    """Two runs on streams of their own, launched without a wait between, on tensors of another stream."""
    sets = [_inputs(30), _inputs(40)]
    want = []
    for held in sets:
        f, b, _ = _run(layer, *held)
        want.append([t.clone() for t in _results(f, b)])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s, held in zip(streams, sets):
            with torch.cuda.stream(s):
                f = layer.forward(held[0], held[1])
                got.append((f, layer.backward(f, *held[2:])))
        torch.cuda.synchronize()
        for (f, b), ref in zip(got, want):
            for k, a, v in zip(KEPT + GRADS, _results(f, b), ref):
                assert torch.equal(a, v), k


def test_tokens_without_experts(layer):
    """A token whose logits are all masked takes no row, adds nothing to the output and gets no gradient."""
    x, res, d_moe, d_h, d_loss = _inputs(50)
    f = layer.forward(x, res)
    z = f["logits"].clone()
    z[3], z[7, 2:] = float("-inf"), float("-inf")
    idx, w = fp8bs.moe_gate(z, TOPK, layer.bias, GROUPS, KEEP, route_scale=SCALE)
    offsets, _, row_of = fp8bs.moe_route(idx, E)
    n = int(offsets[-1])
    assert n == T * TOPK - TOPK - 2 and (row_of[3] == -1).all() and (row_of[7] >= 0).sum() == 2
    gu = torch.full((T * TOPK, 2 * I), float("nan"), dtype=BF16, device=DEV)
    xq, xs = fp8bs.moe_quant_scatter(f["y"], row_of, T * TOPK)
    fp8bs.fp8bs_moe_gemm(xq, xs, layer.fp8(layer.up[0]), layer.up[1], offsets, gu)
    q, s = fp8bs.swiglu_quant(gu[:, :I], gu[:, I:], n_rows=offsets[-1:])
    out = torch.full((T * TOPK, K), float("nan"), dtype=BF16, device=DEV)
    fp8bs.fp8bs_moe_gemm(q, s, layer.fp8(layer.down[0]), layer.down[1], offsets, out)
    y = fp8bs.moe_combine(out, w, row_of)
    assert torch.isfinite(y).all() and (y[3] == 0).all()
    d_out, d_w = fp8bs.moe_combine_bwd(d_moe, out, w, row_of)
    assert torch.isfinite(d_out[:n]).all() and (d_w[3] == 0).all() and (d_w[7, 2:] == 0).all()
    d = fp8bs.moe_gate_bwd(z, idx, d_w, route_scale=SCALE)
    assert torch.isfinite(d).all() and (d[3] == 0).all() and (d[7, 2:] == 0).all()
