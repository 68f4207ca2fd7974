"""Helpers of the paged MLA cache's tests: random batches, and the operators in
64 bits on the CPU (plain loops over sequences and rows, torch float64)."""
import math

import numpy as np
import torch

import block_scaled_fp8_03_amd as fp8bs

R, D = fp8bs.MLA_RANK, fp8bs.MLA_ROPE
BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn
U8 = 2.0 ** -8      # half a step of bf16, relative


def pow2_scale(amax):
    """The smallest power of two >= max(amax, 1e-4) / 448 (float32 division, as act_quant's ue8m0 rule)."""
    m, e = torch.frexp(amax.float().clamp(min=1e-4) / 448)
    return torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e))


def make_cache(P, ps, dtype, gen):
    rope = torch.randn((P, ps, D), generator=gen).to(BF16)
    x = torch.randn((P, ps, R), generator=gen)
    if dtype == BF16:
        return fp8bs.MlaCache(x.to(BF16), rope, None)
    g = x.view(P, ps, R // 128, 128)
    s = pow2_scale(g.abs().amax(-1))
    return fp8bs.MlaCache((g / s[..., None]).clamp(-448, 448).to(FP8).view(P, ps, R), rope, s)


def latent64(cache):
    """The values that the cached latents stand for."""
    x = cache.latent.to(torch.float64) if cache.latent.dtype == BF16 else cache.latent.float().double()
    if cache.scale is not None:
        x = x * cache.scale.double().repeat_interleave(128, -1)
    return x


def to_dev(cache, dev="cuda"):
    return fp8bs.MlaCache(*(None if t is None else t.to(dev) for t in cache))


def make_table(lens, ps, P, gen, behind=-1, W=None):
    """Distinct random pages per row; `behind` fills the entries after a row's last page."""
    need = [-(-n // ps) for n in lens]
    W = W or max(1, max(need, default=1))
    order = torch.randperm(P, generator=gen).tolist()
    table = torch.full((len(lens), W), behind, dtype=torch.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = torch.tensor(order[at:at + k], dtype=torch.int32)
        at += k
    assert at <= P
    return table


def cu_of(nq):
    return torch.tensor(np.concatenate([[0], np.cumsum(nq)]), dtype=torch.int32)


def seq_rows(cache, table, b, n):
    """(latent, rope) in float64 of a sequence's first n tokens."""
    ps = cache.latent.shape[1]
    ids = table[b, :-(-n // ps)].long()
    one = fp8bs.MlaCache(*(None if t is None else t[ids] for t in cache))
    return latent64(one).reshape(-1, R)[:n], one.rope.double().reshape(-1, D)[:n]


def attention64(q_lat, q_rope, cache, table, cu, lens, scale, causal):
    """out, lse, and two scales of the error: A = softmax-weighted |c| [T, H, R] and the
    largest sum of |products| of a row's visible scores [T, H]."""
    T, H, _ = q_lat.shape
    out = torch.zeros((T, H, R), dtype=torch.float64)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64)
    A, S = torch.zeros_like(out), torch.zeros((T, H), dtype=torch.float64)
    for b in range(table.shape[0]):
        n = int(lens[b])
        if n == 0:
            continue
        c, k = seq_rows(cache, table, b, n)
        lo, hi = int(cu[b]), int(cu[b + 1])
        for t in range(lo, hi):
            end = max(0, n - (hi - lo) + (t - lo) + 1) if causal else n
            if end == 0:
                continue
            ql, qr = q_lat[t].double(), q_rope[t].double()
            s = scale * (ql @ c[:end].T + qr @ k[:end].T)
            S[t] = abs(scale) * (ql.abs() @ c[:end].abs().T + qr.abs() @ k[:end].abs().T).amax(-1)
            lse[t] = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[t][:, None])
            out[t] = p @ c[:end]
            A[t] = p @ c[:end].abs()
    return out, lse, A, S


def check_attention(out, lse, ref, lens_max, what):
    """A score is a float32 sum of exact products in 18 matrix steps of 32 (each step's own
    sum, its addition and the scale: within 32 * 2^-24 = 2^-19 of the sum of |products|, S).
    The probabilities take that error e twice (numerator and sum) and a rounding to bf16
    (2^-8); the sums over the tokens add at most one 2^-24 per token.  A bf16 result is
    rounded once more."""
    r, rl, A, S = ref
    e = 2.0 ** -19 * S
    n = 2.0 ** -24 * (lens_max + 64)
    bar = A * (U8 + 2 * e[..., None] + 2 * n + 2.0 ** -20) + (U8 * r.abs() if out.dtype == BF16 else 0) + 1e-30
    err = (out.double().cpu() - r).abs()
    bad = ~(err <= bar)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, first {bad.nonzero()[:4].tolist()}, worst {(err / bar).max():.3g}"
    if lse is not None:
        got = lse.double().cpu()
        assert torch.equal(torch.isinf(got), torch.isinf(rl)), f"{what}: lse of empty rows"
        ok = ~torch.isinf(rl)
        bar = e + n + 2.0 ** -20 + 2.0 ** -22 * rl.abs()
        bad = ((got - rl).abs() > bar) & ok | torch.isnan(got)
        assert not bad.any(), f"{what}: lse, {int(bad.sum())} outside, first {bad.nonzero()[:4].tolist()}"


def update_plain(table, lens, parent, want, P, ps):
    """cache_update by its definition: (table, lens, copies) with copies = (from page, to page, tokens)."""
    tab, ln, par, want = table.tolist(), lens.tolist(), parent.tolist(), want.tolist()
    W = table.shape[1]
    used = {g for r, n in zip(tab, ln) for g in r[:-(-n // ps)]}
    free = [g for g in range(P) if g not in used]
    rows = []
    for p, w in zip(par, want):
        ok = 0 <= p < len(tab)
        w = min(max(w, 0), W * ps)
        keep = min(w, ln[p]) if ok else 0
        rows.append((tab[p][:-(-keep // ps)] if ok else [], keep, w, w > keep and keep % ps != 0))
    held = {}
    for i, (pages, keep, w, grows) in enumerate(rows):
        for j, g in enumerate(pages):
            held.setdefault(g, []).append((min(ps, keep - j * ps), grows and j == len(pages) - 1, i))
    out, lens_out, copies, at = [], [], [], 0
    for i, (pages, keep, w, grows) in enumerate(rows):
        own = False
        if grows:
            most = max(n for n, _, _ in held[pages[-1]])
            own = i != min([r for n, gr, r in held[pages[-1]] if n == most and gr], default=-1)
        need = -(-w // ps) - len(pages) + own if w > keep else 0
        take, at = free[at:at + need], at + need
        if need and at > len(free):
            w, take, own = keep, [], False
        if own:
            copies.append((pages[-1], take[0], keep % ps))
        row = (pages[:-1] if own else pages) + take
        out.append(row + [-1] * (W - len(row)))
        lens_out.append(w)
    return torch.tensor(out, dtype=torch.int32).view(-1, W), torch.tensor(lens_out, dtype=torch.int32), copies


def write64(q_rope, kv, w, eps, cs, pos):
    """c, rotated key and rotated queries of tokens at the given positions."""
    x = kv.double()
    c = x[:, :R] / torch.sqrt(x[:, :R].square().mean(-1, keepdim=True) + eps) * w.double()
    z = torch.view_as_complex(cs[pos].double())

    def turn(v, z):
        v = torch.view_as_complex(v.double().unflatten(-1, (-1, 2)).contiguous())
        return torch.view_as_real(v * z).flatten(-2)

    return c, turn(x[:, R:], z), turn(q_rope, z[:, None])


def rope_table(n, gen=None):
    ang = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    return torch.stack((ang.cos(), ang.sin()), -1).float()
