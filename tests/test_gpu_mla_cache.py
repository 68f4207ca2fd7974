"""GPU parity of the paged MLA cache's operators: fp8bs_mla_cache_write (norm,
rotation, store) within derived bars of 64-bit values; fp8bs_cache_update and
fp8bs_cache_compact exactly, against their definitions in plain Python and by
the properties that a user relies on."""
import math

import pytest
import torch

import block_scaled_fp8_03_amd as fp8bs
from mla_util import (BF16, D, FP8, R, U8, cu_of, latent64, make_cache, make_table, pow2_scale, rope_table, to_dev,
                      update_plain, write64)

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def bits(t):
    return t.contiguous().view(torch.uint8).cpu()


# ---------------------------------------------------------------------- write

def write_case(H, nq, lens, ps, dtype, wdt, seed, spare=1):
    g = torch.Generator().manual_seed(seed)
    P = sum(-(-n // ps) for n in lens) + spare
    cache = make_cache(P, ps, dtype, g)
    table = make_table(lens, ps, P, g)
    T = sum(nq)
    q = torch.randn((T, H, 128 + D), generator=g).to(BF16)
    kv = (3 * torch.randn((T, R + D), generator=g)).to(BF16)
    w = (torch.rand(R, generator=g) + 0.5).to(wdt)
    return q, kv, w, rope_table(max(lens) + 1), cache, table, cu_of(nq), torch.tensor(lens, dtype=torch.int32)


def slots(nq, lens, table, ps):
    """(token, position, page, offset) of the new tokens that have a place."""
    t, out = 0, []
    for b, (n, ln) in enumerate(zip(nq, lens)):
        for i in range(n):
            p = ln - n + i
            if p >= 0:
                out.append((t, p, int(table[b, p // ps]), p % ps))
            t += 1
    return out


@pytest.mark.parametrize("dtype", [BF16, FP8], ids=["bf16", "fp8"])
@pytest.mark.parametrize("H,nq,lens,ps,wdt", [
    (1, [1], [1], 1, BF16),
    (16, [1, 1, 1], [5, 64, 65], 64, torch.float32),
    (128, [1, 0, 2], [100, 3, 31], 16, BF16),
    (3, [40, 7], [40, 90], 7, torch.float32),
    (25, [0, 9, 0], [4, 9, 0], 100, BF16),
    (0, [3], [3], 16, BF16),
    (4, [6, 1], [4, 1], 4, BF16),               # two tokens at positions below 0
])
def test_write(H, nq, lens, ps, wdt, dtype):
    q, kv, w, cs, cache, table, cu, ln = write_case(H, nq, lens, ps, dtype, wdt, 100 + H + sum(lens))
    dev = to_dev(cache)
    q_out = torch.full((q.shape[0], H, D), 9.0, dtype=BF16, device=DEV)
    fp8bs.fp8bs_mla_cache_write(q.to(DEV)[..., 128:], kv.to(DEV), w.to(DEV), 1e-6, cs.to(DEV), q_out, dev,
                                table.to(DEV), cu.to(DEV), ln.to(DEV))
    torch.cuda.synchronize()
    where = slots(nq, lens, table, ps)
    tok = torch.tensor([x[0] for x in where])
    pos = torch.tensor([x[1] for x in where])
    pg, off = torch.tensor([x[2] for x in where]), torch.tensor([x[3] for x in where])
    c, k, qr = write64(q[..., 128:], kv, w, 1e-6, cs, torch.zeros(q.shape[0], dtype=torch.long).index_put((tok,), pos))
    got = fp8bs.MlaCache(*(None if t is None else t.cpu() for t in dev))

    # norm: the mean's 2^-20, halved by the root, and four roundings: within 2^-20; then one rounding to bf16
    # or to e4m3, 2^-4 of the value or half a subnormal step of 2^-9 units
    x, ref = latent64(got)[pg, off], c[tok]
    if dtype == BF16:
        bar = (U8 + 2.0 ** -20) * ref.abs()
    else:
        amax = ref.view(-1, R // 128, 128).abs().amax(-1)
        s, want = got.scale[pg, off], pow2_scale(amax)
        edge = torch.minimum(torch.frexp(amax / 448)[0] - 0.5, 1 - torch.frexp(amax / 448)[0]) < 2.0 ** -18
        assert ((s == want) | edge).all()
        step = s.double().repeat_interleave(128, -1)
        bar = torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -10 * step) + 2.0 ** -20 * ref.abs()
    assert ((x - ref).abs() <= bar).all()
    # rotation: two products and a sum in float32, rounded to bf16
    for a, b, src in ((got.rope[pg, off].double(), k[tok], kv[tok, R:].double()),
                      (q_out.double().cpu()[tok], qr[tok], q[tok][..., 128:].double())):
        size = src.unflatten(-1, (-1, 2)).abs().sum(-1).repeat_interleave(2, -1)
        assert ((a - b).abs() <= U8 * b.abs() + 2.0 ** -22 * size).all()

    # everything else as it was
    rest = torch.ones(cache.latent.shape[:2], dtype=torch.bool)
    rest[pg, off] = False
    for a, b in zip(got, cache):
        assert a is None or torch.equal(bits(a[rest]), bits(b[rest]))
    skipped = torch.ones(q.shape[0], dtype=torch.bool)
    skipped[tok] = False
    assert (q_out.cpu()[skipped] == 9).all()


def test_write_skips_what_has_no_place():
    """Rows behind the last sequence, positions beyond the rope table and pages
    that do not exist."""
    q, kv, w, cs, cache, table, cu, ln = write_case(8, [2, 2, 2], [20, 40, 10], 8, BF16, BF16, 7)
    cs = cs[:39]                                  # sequence 1's second token is at 39
    table[2, 1] = 10 ** 6                         # sequence 2's tokens at 8 and 9
    qk, kvk = torch.cat([q, q[:2]]), torch.cat([kv, kv[:2]])
    dev = to_dev(cache)
    q_out = torch.full((8, 8, D), 9.0, dtype=BF16, device=DEV)
    fp8bs.fp8bs_mla_cache_write(qk.to(DEV)[..., 128:], kvk.to(DEV), w.to(DEV), 1e-6, cs.to(DEV), q_out, dev,
                                table.to(DEV), cu.to(DEV), ln.to(DEV))
    torch.cuda.synchronize()
    changed = (dev.latent.cpu() != cache.latent).any(-1)
    want = torch.zeros_like(changed)
    for b, p in ((0, 18), (0, 19), (1, 38)):
        want[table[b, p // 8], p % 8] = True
    assert torch.equal(changed, want)
    assert (q_out[[3, 6, 7]] == 9).all() and not (q_out[[0, 1, 2, 4, 5]] == 9).all(-1).any()


@pytest.mark.parametrize("B", [64, 65, 300, 5000])
def test_write_many_sequences(B):
    """The sequence of a token among many, some without new tokens."""
    g = torch.Generator().manual_seed(B)
    nq = torch.randint(0, 3, (B,), generator=g).tolist()
    lens = [n + int(x) for n, x in zip(nq, torch.randint(0, 5, (B,), generator=g))]
    q, kv, w, cs, cache, table, cu, ln = write_case(1, nq, lens, 4, BF16, BF16, B)
    dev = to_dev(cache)
    q_out = fp8bs.mla_cache_write(q.to(DEV)[..., 128:], kv.to(DEV), w.to(DEV), 1e-6, cs.to(DEV), dev, table.to(DEV),
                                  cu.to(DEV), ln.to(DEV))
    tok, pos, pg, off = (torch.tensor(x) for x in zip(*slots(nq, lens, table, 4)))
    c, k, qr = write64(q[tok][..., 128:], kv[tok], w, 1e-6, cs, pos)
    x = latent64(fp8bs.MlaCache(*(None if t is None else t.cpu() for t in dev)))[pg, off]
    assert ((x - c).abs() <= (U8 + 2.0 ** -20) * c.abs()).all()
    size = q[tok][..., 128:].double().unflatten(-1, (-1, 2)).abs().sum(-1).repeat_interleave(2, -1)
    assert ((q_out.double().cpu()[tok] - qr).abs() <= U8 * qr.abs() + 2.0 ** -22 * size).all()


@pytest.mark.parametrize("cu", [[0, 10, 2, 3], [0, 10, 2, 20], [0, 20, 0, 20], [-3, 4, -7, 6], [0, -(2 ** 31), 5, 2 ** 31 - 1],
                                [20, 10, 5, 0], [7, 7, 3, 3]])
@pytest.mark.parametrize("dtype", [BF16, FP8], ids=["bf16", "fp8"])
def test_write_boundaries_that_decrease(cu, dtype):
    """cu_q out of order is outside the contract, but nothing is written but tokens
    below a sequence's length, in its own pages: not to the page that the entries
    behind the table name, nor to another row's."""
    T, ps, W, B = 20, 4, 3, 3
    for lens in ([12, 12, 12], [5, 12, 7], [0, 3, 2 ** 31 - 1]):
        cache = make_cache(12, ps, dtype, torch.Generator().manual_seed(17))
        entries = torch.full((64, W), 11, dtype=torch.int32)         # page 11 is no sequence's
        entries[:B] = torch.tensor([[4, 0, 7], [2, 9, 5], [8, 1, 3]])
        g = torch.Generator().manual_seed(18)
        q, kv = torch.randn((T, 4, D), generator=g).to(BF16), torch.randn((T, R + D), generator=g).to(BF16)
        dev = to_dev(cache)
        fp8bs.mla_cache_write(q.to(DEV), kv.to(DEV), torch.ones(R, device=DEV), 1e-6, rope_table(64).to(DEV), dev,
                              entries.to(DEV)[:B], torch.tensor(cu, dtype=torch.int32, device=DEV),
                              torch.tensor(lens, dtype=torch.int32, device=DEV))
        torch.cuda.synchronize()
        own = torch.zeros(cache.latent.shape[:2], dtype=torch.bool)
        for b in range(B):
            for p in range(min(lens[b], W * ps)):
                own[entries[b, p // ps], p % ps] = True
        for a, b in zip(dev, cache):
            assert a is None or torch.equal(bits(a.cpu()[~own]), bits(b[~own])), (cu, lens)


def test_write_quantises_as_act_quant():
    """With the norm switched off (unit-size rows, weight 1) the 8-bit cache
    holds exactly act_quant's ue8m0 codes and scales of the bf16 latents."""
    T = 33
    x = torch.randint(0, 2, (T, R), generator=torch.Generator().manual_seed(3)) * 2.0 - 1
    x = x.view(T, 2, 256)
    x[:, 0] *= 1.25
    x[:, 1] *= math.sqrt(2 - 1.25 ** 2)           # not representable: the mean is near 1, not at it
    x = x.view(T, R).to(BF16)
    kv = torch.cat([x, torch.zeros(T, D, dtype=BF16)], 1).to(DEV)
    cache = fp8bs.mla_cache_alloc(T, 1, DEV, FP8)
    inv = 1 / torch.sqrt(x.double().square().mean(-1))
    assert ((inv - 1).abs() < 2e-3).all()
    table = torch.arange(T, dtype=torch.int32, device=DEV).view(1, T)
    fp8bs.mla_cache_write(torch.zeros(T, 1, D, dtype=BF16, device=DEV), kv, torch.ones(R, device=DEV), 0.0,
                          rope_table(T).to(DEV), cache, table, torch.tensor([0, T], dtype=torch.int32, device=DEV),
                          torch.tensor([T], dtype=torch.int32, device=DEV))
    normed = (x.double() * inv[:, None])
    q, s = fp8bs.act_quant(normed.to(BF16).to(DEV), "ue8m0")
    assert torch.equal(s.cpu(), cache.scale.view(T, -1).cpu())
    # the two differ where rounding to bf16 first crosses a code's edge; values of one block are all alike here
    assert torch.equal(bits(q), bits(cache.latent.view(T, R)))


# --------------------------------------------------------------- update, compact

def random_rows(seed, B, N, ps, P, ctx, W):
    g = torch.Generator().manual_seed(seed)
    lens, left = [], P
    for _ in range(B):
        n = int(torch.randint(0, ctx + 1, (1,), generator=g))
        if -(-n // ps) > min(left, W):
            n = 0
        left -= -(-n // ps)
        lens.append(n)
    table = make_table(lens, ps, P, g, W=W)
    # rows that share pages already: a row continues another's prefix
    for b in range(1, B):
        if torch.rand(1, generator=g) < 0.4 and lens[b - 1]:
            lens[b] = int(torch.randint(1, lens[b - 1] + 1, (1,), generator=g))
            table[b] = -1
            k = -(-lens[b] // ps)
            table[b, :k] = table[b - 1, :k]
    parent = torch.randint(-1, B + 1, (N,), generator=g).to(torch.int32)
    have = torch.tensor([lens[p] if 0 <= p < B else 0 for p in parent.tolist()])
    want = (have + torch.randint(-3, 4 + ps, (N,), generator=g)).to(torch.int32)
    same = torch.rand(N, generator=g) < 0.3
    want[same] = have[same].to(torch.int32)
    return table, torch.tensor(lens, dtype=torch.int32), parent, want


def run_update(cache, table, lens, parent, want):
    dev = to_dev(cache)
    out = fp8bs.cache_update(dev, *(t.to(DEV) for t in (table, lens, parent, want)))
    again = fp8bs.cache_update(dev, *(t.to(DEV) for t in (table, lens, parent, want)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, again))
    return out[0].cpu(), out[1].cpu(), fp8bs.MlaCache(*(None if t is None else t.cpu() for t in dev))


@pytest.mark.parametrize("dtype", [BF16, FP8], ids=["bf16", "fp8"])
@pytest.mark.parametrize("B,N,ps,P,ctx,W", [
    (1, 1, 16, 8, 40, 6), (4, 9, 8, 60, 50, 8), (7, 3, 1, 90, 12, 20), (3, 20, 64, 40, 200, 5),
    (30, 40, 16, 400, 100, 9), (5, 12, 7, 33, 60, 12),          # the last runs out of pages
    (40, 300, 4, 3000, 60, 70), (6, 1500, 16, 70000, 300, 24), (2, 5, 4096, 6, 5000, 3),
    (20, 30, 16, 300, 100, 6000), (3, 2500, 4, 9000, 60, 16),   # wide tables, many rows: not one launch
])
def test_update(B, N, ps, P, ctx, W, dtype):
    table, lens, parent, want = random_rows(B * 100 + N, B, N, ps, P, ctx, W)
    if P * ps > 10 ** 5 and dtype == FP8:
        pytest.skip("one type is enough at this size")
    cache = make_cache(P, ps, dtype, torch.Generator().manual_seed(5)) if P * ps < 10 ** 5 else fp8bs.MlaCache(
        torch.zeros((P, ps, R), dtype=BF16), torch.zeros((P, ps, D), dtype=BF16), None)
    t_ref, l_ref, copies = update_plain(table, lens, parent, want, P, ps)
    t, l, got = run_update(cache, table, lens, parent, want)
    assert torch.equal(l, l_ref) and torch.equal(t, t_ref)
    expect = [None if x is None else x.clone() for x in cache]
    for a, b, n in copies:
        for x in expect:
            if x is not None:
                x.view(torch.uint8)[b, :n] = x.view(torch.uint8)[a, :n]
    for x, y in zip(got, expect):
        assert x is None or torch.equal(bits(x), bits(y))
    # what a user relies on: a row holds its parent's kept tokens, and no one else has a page that it will write into
    users = {}
    for i in range(N):
        for j in range(-(-int(l[i]) // ps)):
            users.setdefault(int(t[i, j]), []).append((i, j))
    for i in range(N):
        p = int(parent[i])
        keep = min(int(lens[p]), max(0, int(want[i]))) if 0 <= p < B else 0
        for j in range(-(-keep // ps)):
            n = min(ps, keep - j * ps)
            for x, y in zip(got, cache):
                assert x is None or torch.equal(bits(x[t[i, j], :n]), bits(y[table[p, j], :n]))
        for j in range(keep // ps, -(-int(l[i]) // ps) if int(l[i]) > keep else 0):
            for r, slot in users[int(t[i, j])]:
                if r == i:
                    continue
                q = int(parent[r])
                other = min(int(lens[q]), max(0, int(want[r]))) if 0 <= q < B else 0
                # a sharer only reads what was there before this row's new tokens, and does not grow there
                assert slot == j and other - j * ps <= keep - j * ps and int(l[r]) == other


def test_update_beam_search_steps():
    """Ten steps of beam search: rows forked, dropped and grown by a token that
    is then written; every row must read back its own history."""
    ps, P, W, N = 4, 64, 8, 6
    g = torch.Generator().manual_seed(9)
    cache = fp8bs.mla_cache_alloc(P, ps, DEV)
    for t in cache:
        if t is not None:
            t.zero_()
    table = torch.full((1, W), -1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(1, dtype=torch.int32, device=DEV)
    history = [[]]
    for step in range(20):
        par = torch.randint(0, len(history), (N,), generator=g)
        parent = par.to(torch.int32).to(DEV)
        table, lens = fp8bs.cache_update(cache, table, lens, parent, lens[parent.long()] + 1)
        history = [history[p] + [100.0 * step + i] for i, p in enumerate(par.tolist())]
        n = step + 1
        assert lens.tolist() == [n] * N
        for i in range(N):                       # the new token's row
            cache.latent[table[i, (n - 1) // ps], (n - 1) % ps] = history[i][-1]
        for i in range(N):
            got = [float(cache.latent[table[i, j // ps], j % ps, 0]) for j in range(n)]
            assert got == [float(torch.tensor(h).to(BF16)) for h in history[i]]


@pytest.mark.parametrize("dtype", [BF16, FP8], ids=["bf16", "fp8"])
@pytest.mark.parametrize("B,ps,P,ctx,W", [(1, 16, 40, 100, 9), (9, 8, 333, 100, 14), (20, 1, 500, 30, 30),
                                          (5, 64, 31, 400, 8), (0, 16, 9, 10, 3), (3, 16, 6, 32, 2), (50, 4, 40000, 90, 30),
                                          (30, 8, 700, 100, 9000)])
def test_compact(B, ps, P, ctx, W, dtype):
    table, lens, _, _ = random_rows(300 + B + P, B, 1, ps, P, ctx, W) if B else (
        torch.zeros((0, W), dtype=torch.int32), torch.zeros(0, dtype=torch.int32), None, None)
    if dtype == FP8 and P > 10000:
        pytest.skip("one type is enough at this size")
    cache = make_cache(P, ps, dtype, torch.Generator().manual_seed(6))
    used = sorted({int(table[b, j]) for b in range(B) for j in range(-(-int(lens[b]) // ps))})
    n = len(used)
    to = dict(zip([g for g in used if g >= n], [g for g in range(n) if g not in set(used)]))
    dev = to_dev(cache)
    for _ in range(2):                            # twice on the same inputs: the same
        t, count = fp8bs.cache_compact(dev, table.to(DEV), lens.to(DEV))
    torch.cuda.synchronize()
    t = t.cpu()
    assert int(count) == n
    want = torch.full_like(table, -1)
    for b in range(B):
        for j in range(-(-int(lens[b]) // ps)):
            want[b, j] = to.get(int(table[b, j]), int(table[b, j]))
    assert torch.equal(t, want)
    for x, y in zip(dev, cache):
        if x is None:
            continue
        y = y.clone().view(torch.uint8)
        for a, b in to.items():
            y[b] = y[a]
        assert torch.equal(x.view(torch.uint8).cpu(), y)


def test_bad_tables_stay_inside():
    """Entries that name no page, lengths beyond the table: nothing outside is touched, good rows are right."""
    ps, P, W = 8, 20, 3
    cache = make_cache(P, ps, BF16, torch.Generator().manual_seed(8))
    table = torch.tensor([[3, 4, 5], [-7, 2 ** 31 - 1, 99], [6, 7, 8]], dtype=torch.int32)
    lens = torch.tensor([20, 2 ** 31 - 1, -4], dtype=torch.int32)
    dev = to_dev(cache)
    t, count = fp8bs.cache_compact(dev, table.to(DEV), lens.to(DEV))
    assert int(count) == 3 and t.tolist() == [[0, 1, 2], [-1, -1, -1], [-1, -1, -1]]
    dev = to_dev(cache)
    t, l = fp8bs.cache_update(dev, table.to(DEV), lens.to(DEV), torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV),
                              torch.tensor([25, 5, 2 ** 31 - 1], dtype=torch.int32, device=DEV))
    assert l.tolist() == [24, 5, 24] and t[0].tolist() == [3, 4, 5] and t[2].tolist() == [0, 1, 2]


def test_update_rows_that_ask_for_more_than_int32():
    """1024 rows that ask for 2^21 pages each, 2^31 together: none is grown, nor
    is the row behind them, whose turn comes after theirs."""
    W, N = 1 << 21, 1100
    cache = fp8bs.mla_cache_alloc(64, 1, DEV)
    want = torch.full((N,), W, dtype=torch.int32)
    want[0], want[-1] = 3, 1
    none = torch.full((N,), -1, dtype=torch.int32, device=DEV)
    t, l = fp8bs.cache_update(cache, torch.full((1, W), -1, dtype=torch.int32, device=DEV),
                              torch.zeros(1, dtype=torch.int32, device=DEV), none, want.to(DEV))
    assert l[0] == 3 and (l[1:] == 0).all()
    assert t[0, :4].tolist() == [0, 1, 2, -1] and (t[0, 3:] == -1).all()
    assert all((part == -1).all() for part in t[1:].split(128))
