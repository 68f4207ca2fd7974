"""GPU parity of fp8bs_mla_attention (new tokens over a paged MLA cache) against
the formula in 64 bits: row tiles of every kind, both cache types, lengths from
none to many pages, odd page sizes, strided queries, masks that leave rows
empty, and garbage wherever the operator must not look.

The library takes larger row tiles (up to what a sequence's rows fill) the more
work the table's width lets it expect, so every case runs twice, with a table
as wide as its sequences ("narrow") and with one for a million tokens ("wide")."""
import math

import pytest
import torch

import block_scaled_fp8_03_amd as fp8bs
from mla_util import (BF16, D, FP8, R, U8, attention64, check_attention, cu_of, make_cache, make_table, to_dev)

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 192.0 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.fixture(params=["narrow", "wide"])
def width(request):
    return request.param


def columns(width, lens, ps):
    return None if width == "narrow" else max((1 << 20) // ps, -(-max(lens) // ps))


def batch(H, nq, lens, ps, dtype, seed, spare=2, W=None, behind=-1):
    g = torch.Generator().manual_seed(seed)
    P = sum(-(-n // ps) for n in lens) + spare
    cache = make_cache(P, ps, dtype, g)
    table = make_table(lens, ps, P, g, behind, W)
    T = sum(nq)
    q_lat = torch.randn((T, H, R), generator=g).to(BF16)
    q_rope = torch.randn((T, H, D), generator=g).to(BF16)
    return q_lat, q_rope, cache, table, cu_of(nq), torch.tensor(lens, dtype=torch.int32)


def run(args, causal=True, dt=BF16, lse=True, scale=SCALE):
    q_lat, q_rope, cache, table, cu, lens = args
    got = fp8bs.mla_attention(q_lat.to(DEV), q_rope.to(DEV), to_dev(cache), table.to(DEV), cu.to(DEV), lens.to(DEV),
                              scale, causal, lse, dt)
    torch.cuda.synchronize()
    return got if lse else (got, None)


def compare(args, what, causal=True, dt=BF16, scale=SCALE):
    q_lat, q_rope, cache, table, cu, lens = args
    out, lse = run(args, causal, dt, True, scale)
    ref = attention64(q_lat, q_rope, cache, table, cu, lens, scale, causal)
    check_attention(out, lse, ref, int(lens.max()), what)
    return out, lse


@pytest.mark.parametrize("dtype", [BF16, FP8], ids=["bf16", "fp8"])
@pytest.mark.parametrize("H,nq,lens,ps", [
    (1, [1], [1], 1),
    (16, [1], [31], 16),
    (16, [1, 1, 1], [32, 33, 500], 64),
    (5, [1, 2, 0, 1], [7, 40, 90, 129], 7),
    (17, [1, 1], [64, 65], 32),               # a second row tile of one row
    (32, [1, 1], [257, 100], 48),
    (48, [1], [300], 64),
    (64, [1, 1], [130, 1], 64),
    (128, [1, 1, 1], [1, 257, 700], 64),
    (100, [1], [95], 64),                     # ragged 128-row tile
    (16, [9, 40], [9, 300], 16),              # chunks: eight tokens a tile
    (128, [5], [261], 64),
    (3, [50, 1, 17], [50, 200, 60], 100),
    (24, [3, 3], [3, 1000], 1),
    (8, [4, 4, 4, 4], [4, 40, 400, 401], 4096),
])
def test_attention(H, nq, lens, ps, dtype, width):
    args = batch(H, nq, lens, ps, dtype, 7 * H + sum(lens), W=columns(width, lens, ps))
    compare(args, f"H {H} nq {nq} lens {lens} ps {ps}")


@pytest.mark.parametrize("dt", [BF16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("H,nq", [(16, [1, 7, 30]), (128, [1, 2, 3])])
def test_causal_and_output_types(H, nq, causal, dt, width):
    lens = [70, 33, 200]
    compare(batch(H, nq, lens, 32, BF16, 11 + H, W=columns(width, lens, 32)), f"H {H} causal {causal} {dt}", causal, dt)


@pytest.mark.parametrize("H", [1, 16, 40, 128])
@pytest.mark.parametrize("dtype", [BF16, FP8], ids=["bf16", "fp8"])
def test_rows_that_see_nothing(H, dtype, width):
    """A sequence of no tokens, and more new tokens than the cache holds: those
    at positions below 0 see nothing, and give zeros and -inf."""
    lens = [0, 3, 40, 0]
    args = batch(H, [2, 5, 3, 1], lens, 16, dtype, 21 + H, W=columns(width, lens, 16))
    out, lse = compare(args, f"empty rows, H {H}")
    empty = torch.tensor([0, 1, 2, 3, 10])
    assert (out[empty] == 0).all() and (lse[empty] == -math.inf).all()
    assert not torch.isinf(lse[4:10]).any()


@pytest.mark.parametrize("H,nq", [(16, [1, 1]), (64, [1, 1]), (128, [1, 3]), (32, [1, 1])])
def test_garbage_out_of_sight(H, nq, width):
    """NaN in every unused cache row and page and beside the table's used part
    indices of no page at all: nothing behind a sequence is looked at."""
    args = batch(H, nq, [45, 130], 32, BF16, 31 + H, W=9 if width == "narrow" else 1 << 15, behind=2 ** 30)
    q_lat, q_rope, cache, table, cu, lens = args
    used = torch.zeros(cache.latent.shape[:2], dtype=torch.bool)
    for b, n in enumerate(lens.tolist()):
        for j in range(n):
            used[table[b, j // 32], j % 32] = True
    lat, rope = cache.latent.clone(), cache.rope.clone()
    lat[~used], rope[~used] = math.nan, math.nan
    dirty = (q_lat, q_rope, fp8bs.MlaCache(lat, rope, None), table, cu, lens)
    a, la = run(args)
    b, lb = run(dirty)
    assert torch.equal(a, b) and torch.equal(la, lb)
    compare(args, "clean")


@pytest.mark.parametrize("H,nq", [(16, [3, 40]), (4, [30, 9]), (2, [16, 12]), (1, [12, 7]), (128, [3, 2])])
@pytest.mark.parametrize("dtype", [BF16, FP8], ids=["bf16", "fp8"])
def test_not_finite_where_masked(H, nq, dtype, width):
    """NaN (and in bf16 infinities) in tokens that only a chunk's later rows see:
    the rows before them are what they are without, those that see a NaN are NaN."""
    lens = [70, 131]
    args = batch(H, nq, lens, 16, dtype, 61 + H, W=columns(width, lens, 16))
    q_lat, q_rope, cache, table, cu, ln = args
    for b, (n, m) in enumerate(zip(lens, nq)):
        first = n - m + (m + 1) // 2                 # the first bad token
        for at, kind in ((first, math.nan), (first + 1, math.inf), (first + 2, math.nan)):
            if at < n:
                page = cache.latent[table[b, at // 16], at % 16]
                if dtype == FP8:
                    page.view(torch.uint8)[7 * b + 3] = 0x7F
                    page.view(torch.uint8)[500] = 0xFF
                else:
                    page[7 * b + 3], page[500] = kind, -kind
        cache.rope[table[b, first // 16], first % 16, 9] = math.inf
    out, lse = run(args)
    ref = attention64(q_lat, q_rope, cache, table, cu, ln, SCALE, True)
    clean = ~torch.isnan(ref[1]).any(1)
    sees = torch.cat([torch.arange(m) >= (m + 1) // 2 for m in nq])
    assert torch.equal(clean, ~sees)
    check_attention(out[clean.to(DEV)], lse[clean.to(DEV)], tuple(x[clean] for x in ref), 131, "rows that do not see it")
    assert torch.isnan(out[sees.to(DEV)]).all() and torch.isnan(lse[sees.to(DEV)]).all()


def compare_not_finite(args, what, scale=SCALE):
    """Element by element what the formula gives where cached tokens hold infinities: NaN in a channel where a
    weight of 0 (a score of -inf) meets an infinity, in all of a row with a score of +inf or NaN, and the others
    within the bars, whose size of a score is that of the tokens with finite ones.  Calls repeated give the same bytes."""
    q_lat, q_rope, cache, table, cu, lens = args
    ref, ref_lse, A, _ = attention64(*args, scale, True)
    tame = fp8bs.MlaCache(*(None if t is None else t.clone() for t in cache))
    for t in (tame.latent, tame.rope):
        if t.dtype == BF16:
            t[torch.isinf(t)] = 0
    S = attention64(q_lat, q_rope, tame, table, cu, lens, scale, True)[3]
    runs = [run(args, dt=torch.float32, scale=scale) for _ in range(3)]
    out, lse = (t.cpu() for t in runs[0])
    for a, b in runs[1:]:
        assert torch.equal(a.cpu().view(torch.int32), out.view(torch.int32))
        assert torch.equal(b.cpu().view(torch.int32), lse.view(torch.int32))
    nan = torch.isnan(ref)
    assert nan.any() and not nan.all(-1).all()
    got = torch.isnan(out)
    assert torch.equal(got, nan), f"{what}: NaN differs in {(got != nan).sum()} of {nan.sum()}, first {(got != nan).nonzero()[:4].tolist()}"
    lost = nan.all(-1)
    assert torch.isnan(lse[lost]).all()
    fill = [torch.where(nan, 0.0, t.double()) for t in (out, ref, A)]
    ok = ~lost
    check_attention(fill[0][ok].float(), lse[ok], (fill[1][ok], ref_lse[ok], fill[2][ok], S[ok]), int(lens.max()), what)


@pytest.mark.parametrize("H,nq", [(16, [3, 40]), (4, [30, 9]), (2, [16, 12]), (1, [12, 7]), (3, [7, 14]), (40, [4, 7]),
                                  (128, [3, 2])])
@pytest.mark.parametrize("scale", [SCALE, -SCALE], ids=["plus", "minus"])
@pytest.mark.parametrize("where", ["later", "all", "both"])
def test_infinities_that_rows_see(H, nq, scale, where, width):
    """One infinite latent in a token that a chunk's later rows see, one in a token that all see right before
    the chunk, or both beside one that the last row sees: about half of a row's scores of it are -inf."""
    lens = [70, 131]
    args = batch(H, nq, lens, 16, BF16, 67 + H, W=columns(width, lens, 16))
    q_lat, q_rope, cache, table, cu, ln = args
    for b, (n, m) in enumerate(zip(lens, nq)):
        spots = {"later": [(n - m + (m + 1) // 2, 7 + 8 * b)], "all": [(n - m - 1, 130 + b)],
                 "both": [(n - m - 1, 64 + b), (n - m + (m + 1) // 2, 511 - b), (n - 1, 300)]}[where]
        for at, channel in spots:
            cache.latent[table[b, at // 16], at % 16, channel] = -math.inf if (at + H) % 2 else math.inf
    compare_not_finite(args, f"H {H} nq {nq} {where}", scale)


@pytest.mark.parametrize("H,nq", [(16, [9, 40]), (2, [16, 12]), (1, [12, 7]), (128, [3, 2])])
@pytest.mark.parametrize("dtype", [BF16, FP8], ids=["bf16", "fp8"])
def test_infinite_keys(H, nq, dtype, width):
    """Infinities in the rotated part alone: a score of -inf takes its token out, with nothing to spread."""
    lens = [70, 131]
    args = batch(H, nq, lens, 16, dtype, 73 + H, W=columns(width, lens, 16))
    cache, table = args[2], args[3]
    for b, (n, m) in enumerate(zip(lens, nq)):
        for at, d in ((n - m - 2, 5), (n - m + m // 2, 40)):
            cache.rope[table[b, at // 16], at % 16, d] = math.inf
    compare_not_finite(args, f"H {H} nq {nq}")


@pytest.mark.parametrize("H", [16, 128])
def test_boundaries_that_decrease(H, width):
    """cu_q out of order is outside the contract, but writes only rows of the
    call; sequences laid over each other many times are left undone."""
    lens = [40] * 5
    q_lat, q_rope, cache, table, _, ln = batch(H, [40], lens, 16, BF16, 71, W=columns(width, lens, 16))
    for cu, undone in (([0, 30, 10, 40, 40, 40], False), ([0, 40, 0, 40, 0, 40], True)):
        out = torch.full((48, H, R), 3.0, dtype=BF16, device=DEV)
        ws = torch.empty(fp8bs.lib().fp8bs_mla_attention_workspace_size(40, H, 5), dtype=torch.uint8, device=DEV)
        fp8bs.fp8bs_mla_attention(q_lat.to(DEV), q_rope.to(DEV), to_dev(cache), table.to(DEV),
                                  torch.tensor(cu, dtype=torch.int32, device=DEV), ln.to(DEV), SCALE, out[4:44], None, ws)
        torch.cuda.synchronize()
        assert (out[:4] == 3).all() and (out[44:] == 3).all()
        assert not undone or (out == 3).all()


@pytest.mark.parametrize("H", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", [BF16, FP8], ids=["bf16", "fp8"])
def test_pages_outside_the_cache_do_not_fault(H, dtype, width):
    """Entries that name no page: the sequence's result is unspecified, the others' is not touched by it."""
    lens = [100, 64, 90]
    args = batch(H, [1, 1, 1], lens, 32, dtype, 41, W=columns(width, lens, 32))
    q_lat, q_rope, cache, table, cu, lens = args
    ref = attention64(q_lat, q_rope, cache, table, cu, lens, SCALE, True)
    bad = table.clone()
    bad[1, :4] = torch.tensor([-5, 2 ** 31 - 1, 12345678, -2 ** 31])
    out, lse = run((q_lat, q_rope, cache, bad, cu, lens))
    keep = torch.tensor([0, 2])
    check_attention(out[keep], lse[keep], tuple(x[keep] for x in ref), 100, "beside bad pages")


@pytest.mark.parametrize("H", [6, 12, 24, 48])
def test_strided_queries_and_rows_behind(H, width):
    """Queries as slices (token and head strides of their own), and rows behind
    the last sequence, which keep what they held."""
    nq, lens = [3, 2], [50, 77]
    args = batch(H, nq, lens, 32, FP8, 51, W=columns(width, lens, 32))
    q_lat, q_rope, cache, table, cu, lens = args
    wide = torch.full((7, H + 1, R + 64), 5.0, dtype=BF16)
    wide[:5, :H, :R], wide[:5, 1:, R:] = q_lat, q_rope
    wide = wide.to(DEV)
    ql, qr = wide[:, :H, :R], wide[:, 1:, R:]
    out = torch.full((7, H, R), 3.0, dtype=BF16, device=DEV)
    lse = torch.full((7, H), 3.0, device=DEV)
    need = fp8bs.lib().fp8bs_mla_attention_workspace_size(7, H, 2)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    fp8bs.fp8bs_mla_attention(ql, qr, to_dev(cache), table.to(DEV), cu.to(DEV), lens.to(DEV), SCALE, out, lse, ws)
    torch.cuda.synchronize()
    ref = attention64(q_lat, q_rope, cache, table, cu, lens, SCALE, True)
    check_attention(out[:5], lse[:5], ref, 77, "strided")
    assert (out[5:] == 3).all() and (lse[5:] == 3).all()


@pytest.mark.parametrize("H", [16, 32, 64, 128])
def test_late_maximum(H, width):
    """Scores that grow along the sequence by far more than the lazy rescale's
    margin, then fall: the running maximum moves many times."""
    args = batch(H, [1 if H < 100 else 2], [400], 64, BF16, 61, W=columns(width, [400], 64))
    q_lat, q_rope, cache, table, cu, lens = args
    size = torch.linspace(0.1, 6.0, 400)
    size[300:] = torch.linspace(6.0, 0.1, 100)
    lat = cache.latent.float()
    for j in range(400):
        lat[table[0, j // 64], j % 64] *= size[j]
    cache = fp8bs.MlaCache(lat.to(BF16), cache.rope, None)
    compare((q_lat, q_rope, cache, table, cu, lens), "growing scores")


@pytest.mark.parametrize("scale", [-0.05, 0.0, 1.0])
def test_any_scale(scale, width):
    lens = [60, 99]
    compare(batch(96, [2, 1], lens, 32, BF16, 71, W=columns(width, lens, 32)), f"scale {scale}", scale=scale)


@pytest.mark.parametrize("scale", [2.3e38, -2.3e38])
def test_largest_scale(scale, width):
    """Queries of zero: every score is 0, whatever the scale, and the output the mean."""
    lens = [60, 99]
    q_lat, q_rope, *rest = batch(96, [2, 1], lens, 32, BF16, 72, W=columns(width, lens, 32))
    compare((q_lat * 0, q_rope * 0, *rest), f"scale {scale}", scale=scale)


@pytest.mark.parametrize("dtype", [BF16, FP8], ids=["bf16", "fp8"])
def test_many_sequences(dtype, width):
    """300 sequences of odd lengths, none, one or a few new tokens each."""
    g = torch.Generator().manual_seed(81)
    nq = torch.randint(0, 4, (300,), generator=g).tolist()
    lens = torch.randint(0, 90, (300,), generator=g).tolist()
    compare(batch(8, nq, lens, 16, dtype, 82, W=columns(width, lens, 16)), "300 sequences")


@pytest.mark.parametrize("H,B", [(2, 8192), (48, 1500), (128, 1100)])
def test_as_many_sequences_as_there_may_be(H, B, width):
    """Up to the limit of 8192 sequences, some empty, some without new tokens."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 12, (B,), generator=g).tolist()
    nq = torch.randint(0, 3, (B,), generator=g).tolist()
    args = batch(H, nq, lens, 4, BF16, 91 + H, W=max(3, columns(width, lens, 64 * 4) or 0) if width == "wide" else None)
    compare(args, f"{B} sequences")


@pytest.mark.parametrize("dtype", [BF16, FP8], ids=["bf16", "fp8"])
@pytest.mark.parametrize("H,B,n", [(16, 1, 20000), (128, 2, 5000), (16, 3, 5000), (64, 1, 7000), (32, 2, 6000)])
def test_long_sequences(H, B, n, dtype, width):
    """Few rows over a long cache: the token axis is split, and joined from a few parts or from many."""
    lens = [n - 37 * b for b in range(B)]
    args = batch(H, [1] * B, lens, 64, dtype, 91 + n, W=columns(width, lens, 64))
    compare(args, f"long {H} {B} {n}")


@pytest.mark.parametrize("dtype", [BF16, FP8], ids=["bf16", "fp8"])
def test_chunk_over_many_tiles(dtype, width):
    """More row tiles than one workgroup takes, whole and split, in sequences of several lengths."""
    nq, lens = [70, 3, 90, 1], [300, 800, 90, 1000]
    compare(batch(40, nq, lens, 48, dtype, 96, W=columns(width, lens, 48)), "chunk over many tiles")


def test_longest_sequence():
    """A length beyond the limit: 2^31 - 4096 tokens, all one page of one token's
    copies, so that the output is its latent and the sum counts the tokens."""
    n, W = 2 ** 31 - 4096, 2 ** 31 // 4096
    q_lat, q_rope, cache, _, cu, _ = batch(4, [1], [1], 4096, BF16, 81, spare=0)
    cache.latent[:], cache.rope[:] = cache.latent[0, 0].clone(), cache.rope[0, 0].clone()
    args = (q_lat, q_rope, cache, torch.zeros((1, W), dtype=torch.int32), cu, torch.tensor([2 ** 31 - 1], dtype=torch.int32))
    out, lse = run(args)
    c, k = cache.latent[0, 0].double(), cache.rope[0, 0].double()
    s = SCALE * (q_lat[0].double() @ c + q_rope[0].double() @ k)
    # each probability is 1 but for its exponent's rounding (2^-19); a wave adds 2^31 / (256 * 4 * 32) = 2^16 times
    # to its accumulators (2^-24 each); the output's bf16
    assert ((out[0].double().cpu() - c).abs() <= (U8 + 2.0 ** -8 + 2.0 ** -19) * c.abs()).all()
    size = SCALE * (q_lat[0].double().abs() @ c.abs() + q_rope[0].double().abs() @ k.abs())
    assert ((lse[0].double().cpu() - s - math.log(n)).abs() <= 2.0 ** -19 * size + 2.0 ** -18).all()


def test_no_new_tokens_and_no_sequences():
    args = batch(16, [0, 0], [10, 20], 16, BF16, 95)
    out, lse = run(args)
    assert out.shape == (0, 16, R) and lse.shape == (0, 16)
