"""The paged MLA cache's operators together, as a model's layer uses them:
cache_update -> mla_absorb_key -> mla_cache_write -> mla_attention ->
mla_absorb_value, over steps of several tokens and of one, with forks between.
Each stage is checked against its formula in 64 bits on the stage before's own
output, and what the cache holds against the tokens that were put in, so a page
that went wrong in any step shows.  Then the same steps captured into a graph,
on other streams and two at a time, and a cache longer than 32-bit offsets."""

import pytest
import torch

import block_scaled_fp8_03_amd as fp8bs
from mla_util import (BF16, D, FP8, R, U8, attention64, check_attention, cu_of, latent64, make_cache, pow2_scale,
                      rope_table, to_dev, write64)

pytestmark = pytest.mark.gpu
DEV = "cuda"
DN = DV = 128
SCALE = (DN + D) ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def layer_weights(H, gen):
    w = (0.05 * torch.randn((H * (DN + DV), R), generator=gen)).to(BF16).to(DEV)
    q, s = fp8bs.weight_quant(w)
    return q, s, (torch.rand(R, generator=gen) + 0.5).to(BF16).to(DEV), rope_table(512).to(DEV)


def layer(weights, q, kv, cache, table, cu, lens, out=None):
    """One layer's step: (q_lat, q_rope, attention, lse, result)."""
    wq, ws, norm, cs = weights
    q_lat = fp8bs.mla_absorb_key(q[..., :DN], wq, ws, DN, DV)
    q_rope = fp8bs.mla_cache_write(q[..., DN:], kv, norm, 1e-6, cs, cache, table, cu, lens)
    x, lse = fp8bs.mla_attention(q_lat, q_rope, cache, table, cu, lens, SCALE, return_lse=True)
    return q_lat, q_rope, x, lse, fp8bs.mla_absorb_value(x, wq, ws, DN, DV)


def on_cpu(cache):
    return fp8bs.MlaCache(*(None if t is None else t.cpu() for t in cache))


def check_absorb(got, x, w, what):
    """Bar of the bf16 path: 2^-13 of the sum of |products|, and the bf16 result's half step."""
    x, w = x.double().cpu(), w.double().cpu()
    ref, size = torch.einsum("thi,hij->thj", x, w), torch.einsum("thi,hij->thj", x.abs(), w.abs())
    assert ((got.double().cpu() - ref).abs() <= 2.0 ** -13 * size + U8 * ref.abs() + 1e-30).all(), what


@pytest.mark.parametrize("dtype", [BF16, FP8], ids=["bf16", "fp8"])
@pytest.mark.parametrize("H,ps", [(16, 16), (128, 5), (8, 64)])
def test_layer_over_steps(H, ps, dtype):
    g = torch.Generator().manual_seed(H + ps)
    weights = layer_weights(H, g)
    w = fp8bs.weight_dequant(weights[0], weights[1]).view(H, DN + DV, R)
    P, W = 400 // ps + 40, 200 // ps + 2
    cache = fp8bs.mla_cache_alloc(P, ps, DEV, dtype)
    table, lens = torch.full((1, W), -1, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    rows = [[]]                                            # each row's (kv, position)
    # (parents, tokens kept of each, new tokens of each): two prompts, a chunk beside a single token, forks, a
    # truncated row (rejected drafts), a row dropped, single tokens
    steps = [([-1, -1], [0, 0], [37, 5]), ([0, 1], [37, 5], [1, 29]), ([0, 0, 1, 1], [38, 38, 34, 20], [1, 1, 1, 1]),
             ([0, 1, 2], [39, 39, 33], [4, 0, 3]), ([0, 2, 2], [41, 36, 36], [1, 1, 1]), ([2, 0], [37, 42], [1, 1])]
    for n, (parent, keep, new) in enumerate(steps):
        total = [k + m for k, m in zip(keep, new)]
        # a row that keeps less than its parent has and grows again: first cut, then grown
        table, lens = fp8bs.cache_update(cache, table, lens, i32(parent).to(DEV), i32(keep).to(DEV))
        same = torch.arange(len(parent), dtype=torch.int32, device=DEV)
        table, lens = fp8bs.cache_update(cache, table, lens, same, i32(total).to(DEV))
        assert lens.tolist() == total
        T = sum(new)
        q = torch.randn((T, H, DN + D), generator=g).to(BF16)
        kv = torch.randn((T, R + D), generator=g).to(BF16)
        cu = cu_of(new)
        got = layer(weights, q.to(DEV), kv.to(DEV), cache, table, cu.to(DEV), lens)
        torch.cuda.synchronize()
        what = f"step {n}"
        rows = [(rows[p] if 0 <= p < len(rows) else [])[:k] + [(kv[t], k + t - int(cu[i])) for t in range(int(cu[i]), int(cu[i + 1]))]
                for i, (p, k) in enumerate(zip(parent, keep))]
        # every row's cache holds its own tokens
        host, tab = on_cpu(cache), table.cpu()
        for i, row in enumerate(rows):
            pos = torch.tensor([p for _, p in row])
            assert pos.tolist() == list(range(total[i]))
            c, k, _ = write64(torch.zeros((len(row), 1, D)), torch.stack([x for x, _ in row]), weights[2].cpu(), 1e-6,
                              weights[3].cpu(), pos)
            pg, off = tab[i, pos // ps].long(), pos % ps
            bar = (U8 + 2.0 ** -20) * c.abs()
            if dtype == FP8:
                step = pow2_scale(c.view(-1, R // 128, 128).abs().amax(-1)).double().repeat_interleave(128, -1)
                # twice the scale where the largest value lies at the edge of two scales
                bar = torch.maximum(2.0 ** -4 * c.abs(), 2.0 ** -9 * step) + 2.0 ** -20 * c.abs()
            assert ((latent64(host)[pg, off] - c).abs() <= bar).all(), what
            size = torch.stack([x for x, _ in row])[:, R:].double().unflatten(-1, (-1, 2)).abs().sum(-1).repeat_interleave(2, -1)
            assert ((host.rope[pg, off].double() - k).abs() <= U8 * k.abs() + 2.0 ** -22 * size).all(), what
        q_lat, q_rope, x, lse, y = got
        check_absorb(q_lat, q[..., :DN], w[:, :DN], what)
        ref = attention64(q_lat.cpu(), q_rope.cpu(), host, tab, cu, lens.cpu(), SCALE, True)
        check_attention(x, lse, ref, max(total), what)
        check_absorb(y, x, w[:, DN:].transpose(1, 2), what)


def decode_state(H, N, ps, dtype, seed, ctx=150):
    """A cache holding N rows of random lengths and room for 20 more tokens each."""
    g = torch.Generator().manual_seed(seed)
    W = -(-(ctx + 20) // ps)
    P = 2 * N * W
    cache = to_dev(make_cache(P, ps, dtype, g))
    lens = torch.randint(1, ctx + 1, (N,), generator=g).to(torch.int32)
    table, lens = fp8bs.cache_update(cache, torch.full((1, W), -1, dtype=torch.int32, device=DEV),
                                     i32([0]).to(DEV), torch.full((N,), -1, dtype=torch.int32, device=DEV), lens.to(DEV))
    return cache, table, lens, g


@pytest.mark.parametrize("dtype", [BF16, FP8], ids=["bf16", "fp8"])
@pytest.mark.parametrize("H,N,ps", [(16, 12, 16), (128, 3, 64)])
def test_captured_steps(H, N, ps, dtype):
    """Beam-search steps replayed from one graph, with eager calls of the same
    operators on other tensors between, against the same steps run eagerly."""
    cache, table, lens, g = decode_state(H, N, ps, dtype, 3 * H + N)
    weights = layer_weights(H, g)
    mirror = fp8bs.MlaCache(*(None if t is None else t.clone() for t in cache))
    t_eager, l_eager = table.clone(), lens.clone()
    cu = torch.arange(N + 1, dtype=torch.int32, device=DEV)
    parent = torch.arange(N, dtype=torch.int32, device=DEV)
    q, kv = torch.zeros((N, H, DN + D), dtype=BF16, device=DEV), torch.zeros((N, R + D), dtype=BF16, device=DEV)
    result = torch.zeros((N, H, DV), dtype=BF16, device=DEV)

    def step(cache, table, lens):
        want = lens[parent.long()] + 1
        t, l = fp8bs.cache_update(cache, table, lens, parent, want)
        y = layer(weights, q, kv, cache, t, cu, l)[-1]
        compacted, count = fp8bs.cache_compact(cache, t, l)
        table.copy_(compacted)
        lens.copy_(l)
        return y

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                       # a warm-up on copies: the captured state stays
        step(fp8bs.MlaCache(*(None if t is None else t.clone() for t in cache)), table.clone(), lens.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        result.copy_(step(cache, table, lens))
    for n in range(5):
        q.copy_(torch.randn(q.shape, generator=g).to(BF16))
        kv.copy_(torch.randn(kv.shape, generator=g).to(BF16))
        parent.copy_(torch.randint(0, N, (N,), generator=g).to(torch.int32))
        graph.replay()
        y = step(mirror, t_eager, l_eager)
        torch.cuda.synchronize()
        assert torch.equal(result, y) and result.float().abs().max() > 0, f"replay {n}"
        assert torch.equal(table, t_eager) and torch.equal(lens, l_eager), f"replay {n}"
        used = torch.unique(table[table >= 0]).long()
        for i in range(N):
            last = int(lens[i]) - 1
            for a, b in zip(cache, mirror):
                assert a is None or torch.equal(a[table[i, last // ps].long(), last % ps].view(torch.uint8),
                                                b[table[i, last // ps].long(), last % ps].view(torch.uint8)), f"replay {n}"
        assert int(used.max()) == len(used) - 1


def test_two_streams_at_once():
    """Two batches on two streams, each call with a workspace of its own, beside
    each other several times: the bytes of the calls made alone."""
    cases, alone, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, (H, N, dtype, ctx) in enumerate([(16, 40, FP8, 3000), (128, 8, BF16, 2000)]):
        cache, table, lens, g = decode_state(H, N, 64, dtype, 50 + i, ctx)
        q_lat = torch.randn((N, H, R), generator=g).to(BF16).to(DEV)
        q_rope = torch.randn((N, H, D), generator=g).to(BF16).to(DEV)
        cu = torch.arange(N + 1, dtype=torch.int32, device=DEV)
        cases.append((q_lat, q_rope, cache, table, cu, lens, SCALE, True, True))
        alone.append(fp8bs.mla_attention(*cases[-1]))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(fp8bs.mla_attention(*cases[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, alone[i][0]) and torch.equal(lse, alone[i][1])


def test_inputs_made_on_the_callers_stream():
    """A call on a stream of its own takes what that stream made right before,
    and what follows there sees the whole result."""
    cache, table, lens, g = decode_state(16, 8, 16, BF16, 77)
    q_lat = torch.randn((8, 16, R), generator=g).to(BF16).to(DEV)
    q_rope = torch.randn((8, 16, D), generator=g).to(BF16).to(DEV)
    cu = torch.arange(9, dtype=torch.int32, device=DEV)
    want = fp8bs.mla_attention(q_lat, q_rope, cache, table, cu, lens, SCALE)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(3):
            late = torch.full_like(q_lat, float("nan"))
            late.copy_(q_lat)
            z = fp8bs.mla_attention(late, q_rope, cache, table, cu, lens, SCALE) * 2
    s.synchronize()
    assert torch.equal(z, want * 2)


@pytest.mark.parametrize("dtype", [BF16, FP8], ids=["bf16", "fp8"])
def test_cache_beyond_32_bit_offsets(dtype):
    """Pages at both ends of a cache of 2^24 tokens (16 GiB of bf16 latents, more
    than 2^32 elements; 8 GiB of codes): write, attend, fork with a copy, and
    compact, against the same steps in a small cache."""
    ps, P, small_P, H, n = 64, 2 ** 18, 64, 16, 300
    g = torch.Generator().manual_seed(13)
    small = to_dev(make_cache(small_P, ps, dtype, g))
    big = fp8bs.mla_cache_alloc(P, ps, DEV, dtype)
    W = 6
    here = i32([[3, 9, 20, 1, 40, -1], [5, 60, 8, 33, 2, -1]])
    there = torch.where(here >= 0, P - small_P + here, here)
    there[0, 1] = 7                                        # and one at the front
    for a, b in zip(here.flatten().tolist(), there.flatten().tolist()):
        if a >= 0:
            for x, y in zip(small, big):
                if x is not None:
                    y[b] = x[a]
    lens = i32([n, n - 10]).to(DEV)
    q = torch.randn((6, H, DN + D), generator=g).to(BF16).to(DEV)
    kv = torch.randn((6, R + D), generator=g).to(BF16).to(DEV)
    cu = i32([0, 4, 6]).to(DEV)
    weights = layer_weights(H, g)
    a = layer(weights, q, kv, small, here.to(DEV), cu, lens)
    b = layer(weights, q, kv, big, there.to(DEV), cu, lens)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    parent, want = i32([0, 0, 1]).to(DEV), i32([n + 1, n + 1, n - 5]).to(DEV)
    ta, la = fp8bs.cache_update(small, here.to(DEV), lens, parent, want)
    tb, lb = fp8bs.cache_update(big, there.to(DEV), lens, parent, want)
    tc, count = fp8bs.cache_compact(big, tb, lb)
    torch.cuda.synchronize()
    used = torch.unique(tb[tb >= 0])
    assert torch.equal(la, lb) and int(count) == len(used) == int(tc.max()) + 1 and int(tb.max()) >= P - small_P
    for i, par in enumerate(parent.tolist()):
        keep = min(int(lens[par]), int(want[i]))
        for j in range(-(-keep // ps)):
            m = min(ps, keep - j * ps)
            for x, y in zip(small, big):
                assert x is None or torch.equal(x[ta[i, j].long(), :m].view(torch.uint8),
                                                y[tc[i, j].long(), :m].view(torch.uint8)), (i, j)
