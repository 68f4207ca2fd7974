"""Plain values in 64 bits of an expert block's operators, and the bounds that the
library's results are held to, for the tests.

H(t) is half a step of type t relative to the value: 2^-8 for bf16, 2^-24 for
float32, 2^-4 for e4m3."""
import numpy as np
import torch

DEV = "cuda"
H_BF16, H_F32, H_E4M3 = 2.0 ** -8, 2.0 ** -24, 2.0 ** -4
E4M3_LOW = 2.0 ** -10            # half of e4m3's smallest step
FP8 = torch.float8_e4m3fn


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(shape, seed, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen(seed), dtype=torch.float32) * std).to(dtype)


def inside(got, ref, bound, what):
    """|got - ref| <= bound, element by element; the same infinities and NaN."""
    got, ref = got.double().cpu(), ref.double().cpu()
    bound = torch.as_tensor(bound, dtype=torch.float64).cpu().expand(ref.shape)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~((got - ref).abs() <= bound) & ~(got == ref) & ~(got.isnan() & ref.isnan())
    if bad.any():
        at = bad.nonzero()[:5].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; (index, got, ref, bound): "
                             f"{[(i, float(got[tuple(i)]), float(ref[tuple(i)]), float(bound[tuple(i)])) for i in at]}")


def check_codes(q, s, c, rel, ue8m0, what):
    """Codes and scales of the 128-blocks of c, whose float32 value is within rel of it."""
    M, K = c.shape
    q, s = q.float().double().cpu(), s.double().cpu()
    c = c.double().cpu()
    want = c.view(M, -1, 128).abs().amax(-1).clamp(min=1e-4) / 448
    if ue8m0:
        m, _ = torch.frexp(s)
        assert (m == 0.5).all(), what + ": scales are powers of two"
        assert (s >= want * (1 - 2 * rel)).all() and (s < 2 * want * (1 + 2 * rel)).all(), what + ": scale"
    else:
        inside(s, want, want * (rel + 2 * H_F32), what + ": scale")
    # the code's half step (of the quotient, whose own error is rel), or half of the smallest step; 448 is the largest
    each = s.repeat_interleave(128, 1)
    inside(q * each, c, c.abs() * (H_E4M3 + 2 * rel) * (1 + rel) + E4M3_LOW * each + 448 * each * 2 * rel, what + ": codes")


def check_special_codes(q, s, c, rel, ue8m0, what):
    """As check_codes, with infinities and NaN in c: the scale is that of a block's numbers, infinite if one of them is; the
    code of a NaN, and of infinity over infinity, is NaN; a finite value over infinity gives 0."""
    M, K = c.shape
    b = c.double().cpu().view(M, -1, 128)
    top = torch.where(b.isnan(), 0.0, b).abs().amax(-1)
    codes, s = q.cpu().float().view(M, -1, 128), s.cpu()
    assert torch.equal(s.isinf(), top.isinf()) and (s > 0).all(), what + ": scales of infinite blocks"
    inf = top.isinf()[..., None].expand_as(b)
    nan = b.isnan() | (b.isinf() & inf)
    assert torch.equal(codes.isnan(), nan), what + ": NaN codes"
    assert (codes[inf & ~nan] == 0).all(), what + ": finite values of infinite blocks"
    keep = ~(inf | nan)
    put = lambda t, v: torch.where(keep, t, v).view(M, K)  # noqa: E731
    check_codes(put(codes, 0.0), torch.where(top.isinf(), 2.0 ** -22 if ue8m0 else 1e-4 / 448, s), put(b, 0.0), rel, ue8m0, what)


# ------------------------------------------------------------------------ norm

def norm_rel(K):
    """Of the float32 norm: the sum's additions (8 of a vector, up to 4 vectors a lane, 6 in a wave, 16 waves), halved
    by the root, and a handful of roundings after it."""
    return (32 + 6 + 16 + 12) * H_F32


def norm(x, res, w, eps):
    t = x.double() + (0 if res is None else res.double())
    return t, t / (t.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()


def norm_bwd(dy, h, w, eps, dres):
    """(dx, its bound, dw, its bound) without the outputs' rounding."""
    dy, h, w = dy.double(), h.double(), w.double()
    r = 1 / (h.square().mean(-1, keepdim=True) + eps).sqrt()
    g = dy * w
    dot, size = (g * h).mean(-1, keepdim=True), (g * h).abs().mean(-1, keepdim=True)
    dx = r * (g - h * r * r * dot)
    # three factors r: 3 norm_rel of each part, and the sums' own additions
    bound = r * (g.abs() + h.abs() * r * r * size) * 4 * norm_rel(h.shape[1])
    if dres is not None:
        dx = dx + dres.double()
        bound = bound + dx.abs() * H_F32
    each = dy * h * r
    return dx, bound, each.sum(0), each.abs().sum(0) * (norm_rel(h.shape[1]) + (h.shape[0] + 32) * H_F32)


# ------------------------------------------------------------------------ gate

def scores(z, kind):
    """z float32 -> scores in 64 bits; masked experts 0."""
    z = np.where(np.isnan(z), -np.inf, z.astype(np.float64))
    with np.errstate(over="ignore"):
        if kind == "sigmoid":
            p = 1 / (1 + np.exp(-z))
            return np.where(p < 2.0 ** -150, 0, p)       # float32 has none so small
    top = z.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.where(z == top, 1.0, np.exp(z - top))
    e = np.where(z == -np.inf, 0.0, e)
    return e / np.maximum(e.sum(1, keepdims=True), 1e-300)


def gate(z, topk, bias=None, groups=1, keep=None, kind="sigmoid", normalize=True, scale=1.0):
    """(indices, weights in 64 bits), token by token."""
    z = z.float().cpu().numpy()
    T, E = z.shape
    p = scores(z, kind)
    with np.errstate(invalid="ignore"):
        key = z if bias is None else p.astype(np.float32) + bias.cpu().numpy()
        key = np.where((z > -np.inf) & (key > -np.inf), key, np.float32(-np.inf))
    idx, w = np.full((T, topk), -1, np.int32), np.zeros((T, topk))
    for t in range(T):
        row = key[t].reshape(groups, -1).copy()
        if groups > 1:
            top = -np.sort(-row, 1)
            val = top[:, 0].copy()
            if bias is not None and top.shape[1] > 1:
                val = np.where(top[:, 1] > -np.inf, top[:, 0] + np.where(top[:, 1] > -np.inf, top[:, 1], 0), val)
            row[np.argsort(-val, kind="stable")[keep:]] = -np.inf
        row = row.ravel()
        at = [i for i in np.argsort(-row, kind="stable")[:topk] if row[i] > -np.inf]
        idx[t, :len(at)], w[t, :len(at)] = at, p[t, at]
    if normalize:
        tot = w.sum(1, keepdims=True)
        w = w / np.where(tot > 0, tot, 1)
    return torch.from_numpy(idx), torch.from_numpy(w * scale)


def score_rel(z, E):
    """Of a float32 score and of its share: the exponential's argument (up to the logits' spread, rounded) and value,
    sums of E of them, a few quotients."""
    f = z.float()
    f = f[torch.isfinite(f)]
    # scores of logits further apart than float32's exponents reach are 0
    spread = min(float(f.max() - f.min()), 104.0) if f.numel() else 0.0
    return (spread + E / 64 + 6 + 16) * 2 * H_F32


def balance(z, idx, cu, kind):
    """(loss, counts, probs) of each sequence."""
    p = scores(z.float().cpu().numpy(), kind)
    E, topk, idx = p.shape[1], idx.shape[1], idx.cpu().numpy()
    tot = p.sum(1, keepdims=True)
    share = p / np.where(tot > 0, tot, 1)
    loss, counts, probs = [], [], []
    for a, b in zip(cu, cu[1:]):
        n = b - a
        i = idx[a:b].ravel()
        c = np.bincount(i[(i >= 0) & (i < E)], minlength=E)
        m = share[a:b].sum(0) / max(n, 1)
        counts.append(c)
        probs.append(m)
        loss.append((c * m).sum() * E / (topk * max(n, 1)))
    return (torch.tensor(np.array(loss)), torch.from_numpy(np.array(counts).astype(np.int32)),
            torch.from_numpy(np.array(probs)))


def gate_bwd(z, idx, dw, kind, normalize, scale, cu, d_loss):
    """(d_logits, sum of the absolute parts of it)."""
    p = scores(z.float().cpu().numpy(), kind)
    T, E = p.shape
    idx = idx.cpu().numpy()
    topk = idx.shape[1]
    u, size = np.zeros((T, E)), np.zeros((T, E))
    tot = p.sum(1, keepdims=True)
    share = p / np.where(tot > 0, tot, 1)
    if d_loss is not None:
        for s, (a, b) in enumerate(zip(cu, cu[1:])):
            if b <= a:
                continue
            i = idx[a:b].ravel()
            c = np.bincount(i[(i >= 0) & (i < E)], minlength=E)
            g = float(d_loss[s]) * E / (topk * (b - a) ** 2) * c
            m = (g * share[a:b]).sum(1, keepdims=True)
            u[a:b] += (g - m) * share[a:b]
            size[a:b] += (np.abs(g) + np.abs(m)) * share[a:b]
    if dw is not None:
        dw = dw.double().cpu().numpy()
        for t in range(T):
            ok = [(k, e) for k, e in enumerate(idx[t]) if 0 <= e < E]
            if not ok:
                continue
            ks, es = zip(*ok)
            own = p[t, list(es)]
            d = dw[t, list(ks)]
            if normalize:
                S = own.sum()
                own = own / S if S > 0 else own * 0
                m, am = (d * own).sum(), (np.abs(d) * own).sum()
                np.add.at(size[t], list(es), scale * (np.abs(d) + am) * own)
                np.add.at(u[t], list(es), scale * (d - m) * own)
            else:
                np.add.at(size[t], list(es), scale * np.abs(d) * own)
                np.add.at(u[t], list(es), scale * d * own)
    if kind == "sigmoid":
        zz = np.where(np.isnan(z.float().cpu().numpy()), -np.inf, z.float().cpu().numpy().astype(np.float64))
        with np.errstate(over="ignore"):
            f = 1 / (1 + np.exp(zz))
        return torch.from_numpy(u * f), torch.from_numpy(size * f)
    return (torch.from_numpy(u - p * u.sum(1, keepdims=True)),
            torch.from_numpy(size + p * size.sum(1, keepdims=True)))


# ------------------------------------------------------------------ activation

SILU_REL = 24 * H_F32            # the exponential, a quotient, three products


def swiglu(g, u):
    g, u = g.double(), u.double()
    return g * torch.special.expit(g) * u


def swiglu_bwd(dy, g, u):
    """(dgate, its size, dup)."""
    dy, g, u = dy.double(), g.double(), u.double()
    s, c = torch.special.expit(g), torch.special.expit(-g)
    return dy * u * s * (1 + g * c), (dy * u * s).abs() * (1 + g.abs()), dy * g * s


# ------------------------------------------------------------------- combine

def combine_bwd(dy, out, w, row_of):
    """(d_out with NaN in rows that no pair maps to, d_w, sum of |dy * out|)."""
    dy, out, w = dy.double(), out.double(), w.double()
    R = out.shape[0]
    d_out = torch.full(out.shape, float("nan"), dtype=torch.float64)
    d_w, size = torch.zeros(w.shape, dtype=torch.float64), torch.zeros(w.shape, dtype=torch.float64)
    for t in range(w.shape[0]):
        for k in range(w.shape[1]):
            r = int(row_of[t, k])
            if 0 <= r < R:
                d_out[r] = w[t, k] * dy[t]
                d_w[t, k] = (dy[t] * out[r]).sum()
                size[t, k] = (dy[t] * out[r]).abs().sum()
    return d_out, d_w, size
