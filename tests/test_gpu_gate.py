"""fp8bs_moe_gate, fp8bs_moe_balance and fp8bs_moe_gate_bwd against values in 64
bits: the experts exactly, the rest within bounds of float32 arithmetic."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_03_amd as fp8bs
import expert_util as eu

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")
EXPERTS = [1, 2, 5, 8, 60, 64, 65, 100, 128, 160, 256, 257, 384, 512, 1000, 1024]


def _groups(E):
    return [g for g in (1, 2, 4, 8, 16, 64) if E % g == 0]


def _check(z, topk, bias=None, groups=1, keep=None, kind="sigmoid", normalize=True, scale=1.0, zd=None):
    idx, w = fp8bs.moe_gate(z.to(DEV) if zd is None else zd, topk, None if bias is None else bias.to(DEV), groups, keep,
                            kind, normalize, scale)
    ri, rw = eu.gate(z, topk, bias, groups, keep or groups, kind, normalize, scale)
    assert torch.equal(idx.cpu(), ri), (z.shape, topk, groups, keep, kind)
    # float32's smallest numbers keep no relative precision
    eu.inside(w, rw, rw.abs() * (2 * eu.score_rel(z, z.shape[1]) + topk * eu.H_F32) + 1e-37 * abs(scale), "weights")
    return idx, w


@pytest.mark.parametrize("E", EXPERTS)
@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_gate(E, kind, with_bias):
    for n, groups in enumerate(_groups(E)):
        T = [1, 3, 130, 37, 5, 4][n % 6]
        keep = max(1, groups // 2)
        topk = min(E // groups * keep, [8, 1, 6, 64, 9, 3][n % 6])
        z = eu.normal((T, E), E + n, 2.0, BF16 if n % 2 else F32)
        bias = eu.normal((E,), 99 + E, 0.3, F32) if with_bias else None
        _check(z, topk, bias, groups, keep, kind, n % 3 != 2, 2.5 if n % 2 else 1.0)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_gate_many_tokens_choose_exactly(kind, with_bias):
    """Every near tie of 20000 tokens goes as in 64 bits."""
    z = eu.normal((20000, 256), 5, 1.2, F32)
    _check(z, 8, eu.normal((256,), 6, 0.05, F32) if with_bias else None, 8, 4, kind, True, 2.5)


def _near_ties(kind):
    """Tokens with two experts at the border of the top 4 whose logits are neighbours in float32: their scores are the same
    number or the next one, decided within 1/20 of a step (but not 1/500) of a rounding's border."""
    E, topk, many = 64, 4, 400000
    g = eu.gen(7)
    lo = (1.0 + 2.5 * torch.rand(many, generator=g)) if kind == "sigmoid" else (0.26 + 0.2 * torch.rand(many, generator=g))
    lo = lo.numpy().astype(np.float32)
    hi = np.nextafter(lo, np.float32(10))
    z = np.full((many, E), -5.0, np.float32) + torch.rand((many, E), generator=g).numpy()
    z[:, 5:8] = 6.0, 7.0, 8.0
    z[:, 5:8] -= 0 if kind == "sigmoid" else 5.0
    z[:, 20], z[:, 41] = lo, hi
    p = eu.scores(z, kind)[:, [20, 41]]
    step = np.spacing(p.astype(np.float32)).astype(np.float64)
    off = np.abs(np.mod(p / step, 1.0) - 0.5)          # from the middle of two float32 numbers, in steps
    near = (off.min(1) < 0.05) & (off.min(1) > 0.002)
    z = torch.from_numpy(z[near][:4000])
    assert z.shape[0] == 4000
    return z, topk


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("shift", [0.0, -0.5])
def test_gate_near_ties_choose_exactly(kind, shift):
    """With a bias the choice goes by scores in 64 bits, rounded once: float32 arithmetic gives hundreds of these tokens another expert."""
    z, topk = _near_ties(kind)
    bias = torch.zeros(64)
    bias[[20, 41]] = shift * (1.0 if kind == "sigmoid" else 0.06)   # key = score + shift is exact
    sloppy = torch.sigmoid(z) if kind == "sigmoid" else torch.softmax(z, -1)
    pair = lambda p: (p[:, 41] > p[:, 20])  # noqa: E731
    exact = torch.from_numpy(eu.scores(z.numpy(), kind)).float()
    assert pair(exact).any() and not pair(exact).all() and (pair(sloppy) != pair(exact)).sum() > 100
    idx, _ = _check(z, topk, bias, kind=kind)
    assert set(idx[:, 3].tolist()) == {20, 41} and torch.equal(idx[:, 3].cpu() == 41, pair(exact))


def test_gate_ties_go_to_the_lowest_index():
    for E in (8, 64, 200, 512):
        z = torch.zeros((3, E))
        z[1, ::2] = -0.0
        z[2] = torch.arange(E) // 7 % 3
        for bias in (None, torch.zeros(E)):
            for groups in (1, 4):
                _check(z, min(8, E // 2), bias, groups, max(1, groups // 2))
    # saturated sigmoids: without a bias by the logits, with one the scores tie
    z = torch.linspace(20, 40, 64)[None].float()
    _check(z, 4)
    _check(z, 4, torch.zeros(64))


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("groups", [1, 8])
def test_gate_masks(kind, with_bias, groups):
    E, topk = 64, 6
    z = eu.normal((12, E), 3, 2.0, F32)
    z[0] = -INF                                   # nothing left
    z[1] = NAN
    z[2, 3:] = -INF                               # fewer than topk, in one group
    z[3, 1::2] = -INF
    z[4, 5] = INF
    z[5, 5], z[5, 40] = INF, INF
    z[6, 9] = NAN
    z[7, 8:56] = -INF                             # whole groups
    z[8] = -3.0e38
    z[9] = -100.0
    z[9, 0] = -INF
    z[10] = torch.where(torch.arange(E) % 8 == 0, 1.0, -INF)   # one expert a group
    z[11, 0] = 3.0e38
    bias = None
    if with_bias:
        bias = eu.normal((E,), 4, 0.3, F32)
        bias[13] = -INF
        bias[20] = NAN
        bias[21] = INF
    idx, w = _check(z, topk, bias, groups, max(1, groups // 2), kind)
    assert (idx[:2] == -1).all() and (w[:2] == 0).all()
    assert ((idx >= 0) | (w == 0)).all()


def test_gate_strides_and_one_value():
    z = eu.normal((20, 300), 3, 2.0, BF16)
    zd = z.to(DEV)
    _check(z[:, 7:167], 6, None, 4, 2, zd=zd[:, 7:167])
    one = zd[:1, :64].expand(9, 64)
    _check(z[:1, :64].expand(9, 64), 6, zd=one)
    _check(torch.zeros((2, 1)), 1)
    idx, w = fp8bs.moe_gate(torch.empty((0, 64), device=DEV), 6)
    assert idx.shape == (0, 6) and w.shape == (0, 6)


def _cu(T, S, seed):
    r = np.random.default_rng(seed)
    return [0] + sorted(int(v) for v in r.integers(0, T + 1, S - 1)) + [T] if S > 0 else [0]


def _balance(z, idx, cu, kind, zd=None):
    dev = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    loss, counts, probs = fp8bs.moe_balance(z.to(DEV) if zd is None else zd, idx.to(DEV), dev(cu), kind)
    at = cu or [0, z.shape[0]]
    rl, rc, rp = eu.balance(z, idx, at, kind)
    assert torch.equal(counts.cpu(), rc)
    most = max(b - a for a, b in zip(at, at[1:]))
    rel = eu.score_rel(z, z.shape[1]) + (most + 64) * eu.H_F32
    eu.inside(probs, rp, rp * rel + 1e-37, "probs")
    eu.inside(loss, rl, rl * (rel + z.shape[1] * eu.H_F32) + 1e-36, "loss")
    return loss, counts, probs


@pytest.mark.parametrize("E", EXPERTS)
@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
def test_balance(E, kind):
    for n, (T, S) in enumerate([(1, 1), (7, 3), (64, 1), (129, 1), (700, 5), (40, 64)]):
        z = eu.normal((T, E), E + n, 2.0, BF16 if n % 2 else F32)
        topk = min(E, [8, 1, 6, 64][n % 4])
        idx = torch.randint(-1, E + 1, (T, topk), generator=eu.gen(n), dtype=torch.int32)   # some on no expert
        cu = None if S == 1 and n % 2 == 0 else _cu(T, S, n)
        loss, counts, probs = _balance(z, idx, cu, kind)
        again = _balance(z, idx, cu, kind)
        assert all(torch.equal(a, b) for a, b in zip(again, (loss, counts, probs)))
        d_loss = eu.normal((S,), 50 + n, 1.0, F32)
        dw = eu.normal((T, topk), 60 + n, 0.1, F32)
        for use_w, use_l in ((True, True), (False, True), (True, False), (False, False)):
            _gate_bwd(z, idx, dw if use_w else None, kind, n % 2 == 0, 2.5, cu, counts, d_loss if use_l else None,
                      BF16 if n % 3 == 2 else F32)


def _gate_bwd(z, idx, dw, kind, normalize, scale, cu, counts, d_loss, out_dtype, zd=None):
    dev = lambda v: None if v is None else v.to(DEV)  # noqa: E731
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
    got = fp8bs.moe_gate_bwd(dev(z) if zd is None else zd, dev(idx), dev(dw), kind, normalize, scale, cud,
                             counts, dev(d_loss), out_dtype)
    ref, size = eu.gate_bwd(z, idx, dw, kind, normalize, scale, cu or [0, z.shape[0]], d_loss)
    rel = 4 * eu.score_rel(z, z.shape[1]) + idx.shape[1] * eu.H_F32
    half = eu.H_BF16 if out_dtype == BF16 else eu.H_F32
    eu.inside(got, ref, ref.abs() * half + size * rel * (1 + half) + 1e-37, "d_logits")
    return got


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
def test_masks_in_the_loss_and_gradients(kind):
    T, E, topk = 10, 60, 6
    z = eu.normal((T, E), 3, 2.0, F32)
    z[0] = -INF
    z[1, 5:] = -INF
    z[2, 4] = NAN
    z[3] = -120.0                                  # scores that underflow
    z[4] = -95.0
    z[5] = 90.0
    z[6, 3] = 60.0
    idx, _ = fp8bs.moe_gate(z.to(DEV), topk, score=kind)
    idx = idx.cpu()
    idx[7] = idx[7, 0]                             # the same expert in every slot
    idx[8, 1::2] = idx[8, 0]
    dw, d_loss = eu.normal((T, topk), 5, 1.0, F32), torch.tensor([1.0, -2.0, 3.0])
    cu = [0, 3, 3, 9]                              # the last token is in none
    got = fp8bs.moe_balance(z.to(DEV), idx.to(DEV), torch.tensor(cu, dtype=torch.int32, device=DEV), kind)
    rl, rc, rp = eu.balance(z, idx, cu, kind)
    assert torch.equal(got[1].cpu(), rc) and got[0][1] == 0
    ok = [0, 1] if kind == "sigmoid" else [0, 1, 2]   # sums of denormal scores carry no precision
    eu.inside(got[2][ok], rp[ok], rp[ok] * (2 * eu.score_rel(z[:3], E) + 100 * eu.H_F32), "probs")
    assert torch.isfinite(got[2]).all() and torch.isfinite(got[0]).all()
    for normalize in (True, False):
        g = fp8bs.moe_gate_bwd(z.to(DEV), idx.to(DEV), dw.to(DEV), kind, normalize, 2.0,
                               torch.tensor(cu, dtype=torch.int32, device=DEV), got[1], d_loss.to(DEV))
        ref, size = eu.gate_bwd(z, idx, dw, kind, normalize, 2.0, cu, d_loss)
        assert torch.isfinite(g).all()
        assert (g.cpu()[~(z > -INF)] == 0).all()
        rows = [t for t in range(T) if not (kind == "sigmoid" and t in (3, 4))]
        eu.inside(g[rows], ref[rows], (size * (4 * eu.score_rel(z[[0, 1, 2, 5, 6, 7, 8, 9]], E) + 100 * eu.H_F32)
                                       + ref.abs() * eu.H_F32 + 1e-37)[rows], "d_logits")


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
def test_losses_with_masks(kind):
    """Losses and mean shares of sequences with masked, NaN, infinite and saturated logits, and experts named twice."""
    T, E, topk = 14, 60, 6
    z = eu.normal((T, E), 13, 2.0, F32)
    z[0] = -INF
    z[1, 5:] = -INF
    z[2, 4], z[2, 50:] = NAN, -INF
    z[4] = -120.0                                  # scores that underflow: a sequence of their own
    z[5] = -95.0
    z[6] = 90.0
    z[7, 3] = 60.0
    z[8, 2], z[8, 9] = INF, INF
    z[9, ::2] = NAN
    idx, _ = fp8bs.moe_gate(z.to(DEV), topk, score=kind)
    idx = idx.cpu()
    idx[7] = idx[7, 0]
    idx[10, 1::2] = idx[10, 0]
    cu = [0, 4, 6, 6, 12, 13]                      # the last token is in none
    loss, counts, probs = fp8bs.moe_balance(z.to(DEV), idx.to(DEV), torch.tensor(cu, dtype=torch.int32, device=DEV), kind)
    rl, rc, rp = eu.balance(z, idx, cu, kind)
    assert torch.equal(counts.cpu(), rc)
    assert (probs >= 0).all() and torch.isfinite(probs).all() and torch.isfinite(loss).all()
    rel = 2 * eu.score_rel(z, E) + 100 * eu.H_F32
    ok = [0, 2, 3, 4] if kind == "sigmoid" else [0, 1, 2, 3, 4]   # sums of denormal scores carry no precision
    eu.inside(probs[ok], rp[ok], rp[ok] * rel + 1e-37, "probs")
    eu.inside(loss[ok], rl[ok], rl[ok] * (rel + E * eu.H_F32) + 1e-36, "loss")
    assert (rl[[0, 3, 4]] > 0).all() and loss[2] == 0
    dl = torch.tensor([1.0, 0.0, 5.0, -2.0, 3.0])
    dev = torch.tensor(cu, dtype=torch.int32, device=DEV)
    d = fp8bs.moe_gate_bwd(z.to(DEV), idx.to(DEV), None, kind, cu_seq=dev, counts=counts, d_loss=dl.to(DEV))
    ref, size = eu.gate_bwd(z, idx, None, kind, True, 1.0, cu, dl)
    assert (d.cpu()[~(z > -INF)] == 0).all() and (d[13] == 0).all()
    rows = [r for r in range(T) if r not in (4, 5)]
    eu.inside(d[rows], ref[rows], (size * 2 * rel + ref.abs() * eu.H_F32 + 1e-37)[rows], "d_logits")


def test_bounds_that_are_wrong_stay_inside():
    """Boundaries out of range or falling: nothing outside the buffers is written."""
    E, guard = 64, 4096
    z, idx = eu.normal((500, E), 1, 1.0, F32).to(DEV), torch.zeros((500, 2), dtype=torch.int32, device=DEV)
    for cu in ([-5, 300, 10, 999], [400, 300, 200, 100], [1 << 30, -(1 << 30), 1 << 30, 0], [7, 7, 7, 7], [600, 700, 800, 900]):
        cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
        need = fp8bs.lib().fp8bs_moe_balance_workspace_size(500, 3, E)
        buf = torch.zeros(need + 2 * guard, dtype=torch.uint8, device=DEV)
        out = torch.full((3 * E * 2 + 3 + 200,), -7, dtype=torch.int32, device=DEV)
        counts, probs = out[50:50 + 3 * E].view(3, E), out[100 + 3 * E:100 + 6 * E].view(F32).view(3, E)
        loss = out[150 + 6 * E:153 + 6 * E].view(F32)
        buf[:guard], buf[-guard:] = 1, 1
        fp8bs.fp8bs_moe_balance(z, idx, cu, "sigmoid", counts, probs, loss, buf[guard:-guard])
        assert (buf[:guard] == 1).all() and (buf[-guard:] == 1).all()
        for part in (out[:50], out[50 + 3 * E:100 + 3 * E], out[100 + 6 * E:150 + 6 * E], out[153 + 6 * E:]):
            assert (part == -7).all()
        fp8bs.moe_gate_bwd(z, idx, None, cu_seq=cu, counts=counts, d_loss=torch.ones(3, device=DEV))
    torch.cuda.synchronize()


def test_balance_many_sequences_and_long_ones():
    """More sequences than probes of a wave, of no, one and many tokens; more tokens than two a wave."""
    E, topk = 32, 4
    T = 20000
    lens = ([0, 1, 2, 0, 0, 17, 3] * 800)[:5000]
    lens[77] = 0
    lens[77] = T - sum(lens)
    cu = [0] + np.cumsum(lens).tolist()
    z = eu.normal((T, E), 1, 2.0, F32)
    idx = torch.randint(0, E, (T, topk), generator=eu.gen(2), dtype=torch.int32)
    _, counts, _ = _balance(z, idx, cu, "sigmoid")
    _gate_bwd(z, idx, None, "sigmoid", True, 1.0, cu, counts, eu.normal((len(lens),), 3, 1.0, F32), F32)
    _balance(z, idx, None, "softmax")


@pytest.mark.parametrize("runs", [1, 2, 3, 4, 200, 70000])
def test_balance_runs_of_empty_sequences(runs):
    """Empty sequences between a workgroup's tokens, before the first and behind the last."""
    E, topk = 24, 3
    lens = [0] * runs + [5] + [0] * runs + [1, 1] + [0] * runs + [60, 0, 2] + [0] * runs
    cu = [0] + np.cumsum(lens).tolist()
    T = cu[-1] + 7                                 # the last tokens are in none
    z = eu.normal((T, E), runs, 2.0, F32)
    idx = torch.randint(0, E, (T, topk), generator=eu.gen(2), dtype=torch.int32)
    dev = torch.tensor(cu, dtype=torch.int32, device=DEV)
    loss, counts, probs = (t.cpu() for t in fp8bs.moe_balance(z.to(DEV), idx.to(DEV), dev))
    has = [n for n, v in enumerate(lens) if v]
    rl, rc, rp = eu.balance(z, idx, [0] + [cu[n + 1] for n in has], "sigmoid")
    assert torch.equal(counts[has], rc) and int(counts.sum()) == topk * cu[-1]
    eu.inside(probs[has], rp, rp * (eu.score_rel(z, E) + 128 * eu.H_F32), "probs")
    eu.inside(loss[has], rl, rl * (eu.score_rel(z, E) + (128 + E) * eu.H_F32), "loss")
    assert int((probs != 0).any(1).sum()) == int((loss != 0).sum()) == len(has)


def test_balance_no_tokens_and_no_sequences():
    z, idx = torch.empty((0, 64), device=DEV), torch.empty((0, 4), dtype=torch.int32, device=DEV)
    loss, counts, probs = fp8bs.moe_balance(z, idx, torch.zeros(4, dtype=torch.int32, device=DEV))
    assert loss.tolist() == [0, 0, 0] and not counts.any() and not probs.any()
    assert fp8bs.moe_gate_bwd(z, idx).shape == (0, 64)
    loss, _, _ = fp8bs.moe_balance(z, idx, torch.zeros(1, dtype=torch.int32, device=DEV))
    assert loss.shape == (0,)


def test_even_use_costs_one():
    """All experts used alike and scored alike: a loss of 1."""
    E, topk = 64, 4
    idx = torch.arange(E * 3, dtype=torch.int32).view(-1, topk) % E
    z = torch.zeros((idx.shape[0], E))
    for kind in ("sigmoid", "softmax"):
        loss, _, _ = fp8bs.moe_balance(z.to(DEV), idx.to(DEV), None, kind)
        assert abs(float(loss) - 1) < 64 * eu.H_F32


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_differences(kind, normalize):
    """Along directions, against differences of the formula in 64 bits (ids and counts held)."""
    T, E, topk, cu = 40, 96, 6, [0, 11, 40]
    z = eu.normal((T, E), 1, 1.5, F32)
    idx, _ = fp8bs.moe_gate(z.to(DEV), topk, score=kind)
    _, counts, _ = fp8bs.moe_balance(z.to(DEV), idx, torch.tensor(cu, dtype=torch.int32, device=DEV), kind)
    dw, dl = eu.normal((T, topk), 2, 1.0, F32), torch.tensor([20.0, -30.0])
    d = _gate_bwd(z, idx.cpu(), dw, kind, normalize, 2.5, cu, counts, dl, F32)
    c = counts.double().cpu()

    def f(zz):
        p = torch.special.expit(zz) if kind == "sigmoid" else torch.softmax(zz, -1)
        w = p.gather(1, idx.cpu().long())
        w = w / w.sum(-1, keepdim=True) if normalize else w
        share = p / p.sum(-1, keepdim=True)
        loss = [E / (topk * (b - a)) * (c[s] * share[a:b].mean(0)).sum() for s, (a, b) in enumerate(zip(cu, cu[1:]))]
        return (2.5 * w * dw.double()).sum() + (torch.stack(loss) * dl.double()).sum()

    _, size = eu.gate_bwd(z, idx.cpu(), dw, kind, normalize, 2.5, cu, dl)
    for seed in range(3):
        v = eu.normal((T, E), 30 + seed, 1.0, F32).double()
        step = 1e-5
        diff = (f(z.double() + step * v) - f(z.double() - step * v)) / (2 * step)
        bound = (size * (4 * eu.score_rel(z, E) + 8 * eu.H_F32) * v.abs()).sum() + 1e-6
        eu.inside((d.double().cpu() * v).sum(), diff, bound, "along a direction")


def test_most_tokens():
    """As many tokens as one launch has; all alike, read by a stride of 0."""
    T, E, topk = (1 << 24) - 1, 8, 2
    one = eu.normal((1, E), 1, 1.0, F32).to(DEV)
    z = one.expand(T, E)
    idx, w = fp8bs.moe_gate(z, topk)
    i1, w1 = fp8bs.moe_gate(one, topk)
    assert (idx == i1).all() and (w == w1).all()
    cu = torch.tensor([0, 5, T - 1, T], dtype=torch.int32, device=DEV)
    loss, counts, probs = fp8bs.moe_balance(z, idx, cu)
    n = [5, T - 6, 1]
    for s in range(3):
        assert counts[s, i1[0].long()].tolist() == [n[s]] * topk and int(counts[s].sum()) == topk * n[s]
    share = torch.sigmoid(one.double())
    share = (share / share.sum()).expand(3, E)
    # a wave of a workgroup adds 4096 tokens up one by one, and 512 workgroups' sums follow
    eu.inside(probs, share, share.cpu() * (eu.score_rel(one.cpu(), E) + (4096 + 600) * eu.H_F32), "probs")
    d = fp8bs.moe_gate_bwd(z, idx, None, cu_seq=cu, counts=counts, d_loss=torch.ones(3, device=DEV))
    lone = fp8bs.moe_gate_bwd(one, i1, None, counts=counts[2:], d_loss=torch.ones(1, device=DEV))
    assert torch.equal(d[T - 1:], lone) and torch.equal(d[5:6], d[T - 2:T - 1])
