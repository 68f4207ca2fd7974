"""fp8bs_swiglu, fp8bs_swiglu_bwd and fp8bs_moe_combine_bwd against values in 64 bits."""
import pytest
import torch

import block_scaled_fp8_03_amd as fp8bs
import expert_util as eu

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")
SIZES = [(1, 128), (3, 256), (17, 384), (5, 1920), (33, 2048), (2, 18432), (260, 128), (1, 65536)]
TINY = 1e-36                     # of products with denormal sigmoids, which carry no relative precision


def _inputs(M, N, seed, std=3.0):
    gu = eu.normal((M, 2 * N), seed, std)
    gu[0, :4] = torch.tensor([0.0, -0.0, -100.0, 90.0])
    return gu, gu.to(DEV)


@pytest.mark.parametrize("M,N", SIZES)
@pytest.mark.parametrize("fmt", ["fp32", "ue8m0"])
def test_swiglu(M, N, fmt):
    gu, d = _inputs(M, N, M + N)
    a = eu.swiglu(gu[:, :N], gu[:, N:])
    q, s, y = fp8bs.swiglu_quant(d[:, :N], d[:, N:], fmt, return_y=True)
    eu.inside(y, a, a.abs() * (eu.H_BF16 + eu.SILU_REL) + TINY, "y")
    eu.check_codes(q, s, a, eu.SILU_REL, fmt == "ue8m0", "codes")
    # two tensors, and the outputs apart
    q2, s2 = fp8bs.swiglu_quant(d[:, :N].contiguous(), d[:, N:].contiguous(), fmt)
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s)
    assert torch.equal(fp8bs.swiglu(d[:, :N], d[:, N:]), y)


@pytest.mark.parametrize("M,N", SIZES)
def test_swiglu_bwd(M, N):
    gu, d = _inputs(M, N, 7 * M + N)
    dy = eu.normal((M, N), 9, 0.5)
    dg, size, du = eu.swiglu_bwd(dy, gu[:, :N], gu[:, N:])
    got = torch.full((M, 2 * N + 64), NAN, dtype=BF16, device=DEV)
    fp8bs.fp8bs_swiglu_bwd(dy.to(DEV), d[:, :N], d[:, N:], got[:, :N], got[:, N + 64:])
    assert got[:, N:N + 64].isnan().all()
    eu.inside(got[:, :N], dg, dg.abs() * eu.H_BF16 + size * 2 * eu.SILU_REL + TINY, "dgate")
    eu.inside(got[:, N + 64:], du, du.abs() * (eu.H_BF16 + eu.SILU_REL) + TINY, "dup")
    a, b = fp8bs.swiglu_bwd(dy.to(DEV), d[:, :N].contiguous(), d[:, N:].contiguous())
    assert torch.equal(a, got[:, :N]) and torch.equal(b, got[:, N + 64:])


@pytest.mark.parametrize("count", [-3, 0, 1, 37, 64, 99])
def test_rows_behind_the_count_stay(count):
    """They are neither read (NaN there) nor written."""
    M, N = 64, 1280
    n = min(max(count, 0), M)
    gu, d = _inputs(M, N, 3)
    d[n:] = NAN
    dy = eu.normal((M, N), 4).to(DEV)
    c = torch.tensor([count], dtype=torch.int32, device=DEV)
    q = torch.full((M, N), 0x5A, dtype=torch.uint8, device=DEV)
    s, y = torch.full((M, N // 128), -7.0, device=DEV), torch.full((M, N), 9.0, dtype=BF16, device=DEV)
    fp8bs.fp8bs_swiglu(d[:, :N], d[:, N:], y, q, s, "fp32", c)
    assert (q[n:] == 0x5A).all() and (s[n:] == -7).all() and (y[n:] == 9).all()
    dg, du = torch.full((M, N), 8.0, dtype=BF16, device=DEV), torch.full((M, N), 9.0, dtype=BF16, device=DEV)
    fp8bs.fp8bs_swiglu_bwd(dy, d[:, :N], d[:, N:], dg, du, c[0])
    assert (dg[n:] == 8).all() and (du[n:] == 9).all()
    if n:
        g, u = d[:n, :N].contiguous(), d[:n, N:].contiguous()
        q2, s2, y2 = fp8bs.swiglu_quant(g, u, return_y=True)
        assert torch.equal(q[:n], q2.view(torch.uint8)) and torch.equal(s[:n], s2) and torch.equal(y[:n], y2)
        dg2, du2 = fp8bs.swiglu_bwd(dy[:n].contiguous(), g, u)
        assert torch.equal(dg[:n], dg2) and torch.equal(du[:n], du2)


def test_swiglu_differences():
    """The gradient along directions against differences in 64 bits."""
    M, N = 6, 256
    gu, d = _inputs(M, N, 5)
    dy = eu.normal((M, N), 6)
    dg, du = fp8bs.swiglu_bwd(dy.to(DEV), d[:, :N], d[:, N:])
    g, u = gu[:, :N].double(), gu[:, N:].double()
    for seed in range(3):
        v, w = eu.normal((M, N), 10 + seed).double(), eu.normal((M, N), 20 + seed).double()
        f = lambda k: (eu.swiglu(g + k * v, u + k * w) * dy.double()).sum()  # noqa: E731
        diff = (f(1e-5) - f(-1e-5)) / 2e-5
        a, b = dg.double().cpu(), du.double().cpu()
        _, size, _ = eu.swiglu_bwd(dy, g, u)
        bound = ((a.abs() * eu.H_BF16 + size * 2 * eu.SILU_REL) * v.abs() + b.abs() * eu.H_BF16 * w.abs()).sum() + 1e-5
        eu.inside((a * v + b * w).sum(), diff, bound, "along a direction")


def test_sigmoids_below_float32s_range():
    """Gates down to -170, whose sigmoid is 2^-245: no allowance but half of bf16's smallest step, 2^-134."""
    M, N = 64, 1280
    g = -170 * torch.rand((M, N), generator=eu.gen(1))
    g[:, :128] = torch.linspace(-86, -105, 128)
    # up to the size that leaves the product within float32
    size = 2.0 ** (torch.rand((M, N), generator=eu.gen(2)) * 240 - 120)
    u = torch.where(torch.rand((M, N), generator=eu.gen(3)) < 0.5, size, -size)
    g, u, dy = g.to(BF16), u.to(BF16), eu.normal((M, N), 4, 1.0)
    a = eu.swiglu(g, u)
    low = 2.0 ** -134 * (1 + eu.H_BF16)
    # the outputs that the allowance elsewhere passes over are most of these
    assert ((a.abs() > 2.0 ** -126) & (g < -88)).sum() > 1000
    eu.inside(fp8bs.swiglu(g.to(DEV), u.to(DEV)), a, a.abs() * (eu.H_BF16 + eu.SILU_REL) + low, "y")
    q, s = fp8bs.swiglu_quant(g.to(DEV), u.to(DEV), "ue8m0")
    eu.check_codes(q, s, a, eu.SILU_REL, True, "codes")
    dg, part, du = eu.swiglu_bwd(dy, g, u)
    got_g, got_u = fp8bs.swiglu_bwd(dy.to(DEV), g.to(DEV), u.to(DEV))
    eu.inside(got_g, dg, dg.abs() * eu.H_BF16 + part * 2 * eu.SILU_REL + low, "dgate")
    eu.inside(got_u, du, du.abs() * (eu.H_BF16 + eu.SILU_REL) + low, "dup")


@pytest.mark.parametrize("fmt", ["fp32", "ue8m0"])
def test_infinities_and_nan_stay_in_their_blocks(fmt):
    """Products beyond float32, infinite and NaN inputs: values as the formula has them, codes as c / s has them."""
    M, N = 20, 640
    gu = eu.normal((M, 2 * N), 11, 3.0)
    clean = fp8bs.swiglu_quant(gu.to(DEV)[:, :N], gu.to(DEV)[:, N:], fmt, return_y=True)
    for row, col, g, u in ((3, 5, 1e30, -1e30), (3, 130, 3e38, 3e38), (7, 300, INF, 2.0), (9, 639, NAN, 1.0), (9, 2, 1.0, NAN),
                           (9, 4, 1.0, 1e30), (12, 250, 1.0, -INF), (15, 400, INF, 0.0)):
        gu[row, col], gu[row, N + col] = g, u
    a = eu.swiglu(gu[:, :N], gu[:, N:]).float()   # beyond float32: infinite
    q, s, y = fp8bs.swiglu_quant(gu.to(DEV)[:, :N], gu.to(DEV)[:, N:], fmt, return_y=True)
    eu.inside(y, a.double(), a.double().abs().nan_to_num(0, 0) * (eu.H_BF16 + eu.SILU_REL) + TINY, "y")
    eu.check_special_codes(q, s, a, eu.SILU_REL, fmt == "ue8m0", "codes")
    for got, want in zip((q.view(torch.uint8), s, y), (clean[0].view(torch.uint8), clean[1], clean[2])):
        rest = [r for r in range(M) if r not in (3, 7, 9, 12, 15)]
        assert torch.equal(got[rest], want[rest])


@pytest.mark.parametrize("M,N", [(8001, 2048), (32768, 2048), (30001, 384), (120001, 384)])
def test_many_rows_as_few(M, N):
    """More than 8 workgroups a CU (a thread takes rows in turn), below and above 160 MB (where inputs are read with a hint),
    counts that end inside a thread's rows: bit by bit what a few rows at a time give, and nothing behind the count."""
    g = torch.Generator(DEV)
    g.manual_seed(M)
    gu = (torch.randn((M, 2 * N), device=DEV, generator=g) * 2).to(BF16)
    dy = torch.randn((M, N), device=DEV, generator=g).to(BF16)
    few = 2000 if N == 2048 else 10000
    same = lambda a, b: torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))  # noqa: E731
    for n in (M, (M - 2768) | 1, (M // 4 - 1) | 1):
        gu[n:], dy[n:] = NAN, NAN
        count = torch.tensor([n], dtype=torch.int32, device=DEV)
        q = torch.full((M, N), 0x5A, dtype=torch.uint8, device=DEV)
        s, y = torch.full((M, N // 128), -7.0, device=DEV), torch.full((M, N), 9.0, dtype=BF16, device=DEV)
        d = torch.full((M, 2 * N), 8.0, dtype=BF16, device=DEV)
        fp8bs.fp8bs_swiglu(gu[:, :N], gu[:, N:], y, q.view(eu.FP8), s, "fp32", None if n == M else count)
        fp8bs.fp8bs_swiglu_bwd(dy, gu[:, :N], gu[:, N:], d[:, :N], d[:, N:], None if n == M else count)
        assert (q[n:] == 0x5A).all() and (s[n:] == -7).all() and (y[n:] == 9).all() and (d[n:] == 8).all()
        for a in range(0, n, few):
            b = min(a + few, n)
            part = gu[a:b]
            q2, s2, y2 = fp8bs.swiglu_quant(part[:, :N], part[:, N:], return_y=True)
            dg2, du2 = fp8bs.swiglu_bwd(dy[a:b], part[:, :N], part[:, N:])
            assert same(q[a:b], q2) and same(s[a:b], s2) and same(y[a:b], y2), (n, a)
            assert same(d[a:b, :N], dg2) and same(d[a:b, N:], du2), (n, a)


def test_swiglu_last_rows_beyond_32_bits():
    M, N, ld = 40000, 256, 1 << 16
    buf = torch.zeros(M * ld, dtype=BF16, device=DEV)
    g, u = buf.view(M, ld)[:, :N], buf.view(M, ld)[:, ld - N:]
    some = eu.normal((2, 2 * N), 1).to(DEV)
    g[M - 2:], u[M - 2:] = some[:, :N], some[:, N:]
    y = fp8bs.swiglu(g, u)
    assert torch.equal(y[M - 2:], fp8bs.swiglu(some[:, :N], some[:, N:])) and (y[:M - 2] == 0).all()


# ------------------------------------------------------- the combine's gradient

@pytest.mark.parametrize("T,topk,N", [(1, 1, 8), (1, 8, 7168), (5, 6, 2048), (33, 2, 136), (7, 3, 1), (4, 20, 1003),
                                      (9, 9, 4096), (130, 8, 520), (2, 8, 65536 + 8)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dropped", [False, True])
def test_combine_bwd(T, topk, N, dtype, dropped):
    P = T * topk
    R = P + 3                                     # rows that no pair maps to
    order = torch.randperm(R, generator=eu.gen(1))[:P].to(torch.int32)
    if dropped:
        order[::3] = torch.tensor([-1, R, -(1 << 31), (1 << 31) - 1, R + 7]).repeat(P)[:order[::3].shape[0]].to(torch.int32)
    row_of = order.view(T, topk)
    dy, out = eu.normal((T, N), 2, 0.5, dtype), eu.normal((R, N), 3)
    w = torch.rand((T, topk), generator=eu.gen(4)) - 0.3
    ref, d_w, size = eu.combine_bwd(dy, out, w, row_of)
    got, got_w = torch.full((R, N), NAN, dtype=BF16, device=DEV), torch.full((T, topk), NAN, device=DEV)
    fp8bs.fp8bs_moe_combine_bwd(dy.to(DEV), out.to(DEV), w.to(DEV), row_of.to(DEV), got, got_w)
    eu.inside(got, ref, ref.abs() * (eu.H_BF16 + 2 * eu.H_F32) + 1e-38, "d_out")
    eu.inside(got_w, d_w, size * (N / 64 + 16) * eu.H_F32, "d_w")
    a, b = fp8bs.moe_combine_bwd(dy.to(DEV), out.to(DEV), w.to(DEV), row_of.to(DEV))
    used = ~ref.isnan()[:, 0]
    assert torch.equal(a.cpu()[used], got.cpu()[used]) and torch.equal(b, got_w)


def test_combine_bwd_nothing():
    e = lambda *s, dtype=BF16: torch.empty(s, dtype=dtype, device=DEV)  # noqa: E731
    d_out, d_w = fp8bs.moe_combine_bwd(e(0, 64), e(5, 64), e(0, 2, dtype=F32), e(0, 2, dtype=torch.int32))
    assert d_out.shape == (5, 64) and d_w.shape == (0, 2)
    _, d_w = fp8bs.moe_combine_bwd(torch.ones((3, 64), dtype=BF16, device=DEV), e(0, 64), torch.ones((3, 2), device=DEV),
                                   torch.zeros((3, 2), dtype=torch.int32, device=DEV))
    assert (d_w == 0).all()
    _, d_w = fp8bs.moe_combine_bwd(e(3, 0), e(4, 0), torch.ones((3, 2), device=DEV),
                                   torch.zeros((3, 2), dtype=torch.int32, device=DEV))
    assert (d_w == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_combine_bwd_many_rows_as_few(dtype):
    """196 MB of rows, read with a hint: bit by bit what a few tokens at a time give."""
    T, topk, N = 1500, 8, 4096
    R = T * topk + 3
    g = torch.Generator(DEV)
    g.manual_seed(1)
    row_of = torch.randperm(R, device=DEV, generator=g)[:T * topk].to(torch.int32)
    row_of[::50] = -1
    row_of = row_of.view(T, topk)
    dy, out = torch.randn((T, N), device=DEV, generator=g).to(dtype), torch.randn((R, N), device=DEV, generator=g).to(BF16)
    w = torch.rand((T, topk), device=DEV, generator=g)
    both = [(torch.full((R, N), 9.0, dtype=BF16, device=DEV), torch.full((T, topk), NAN, device=DEV)) for _ in range(2)]
    fp8bs.fp8bs_moe_combine_bwd(dy, out, w, row_of, *both[0])
    for a in range(0, T, 100):
        d_w = torch.full((100, topk), NAN, device=DEV)
        fp8bs.fp8bs_moe_combine_bwd(dy[a:a + 100], out, w[a:a + 100], row_of[a:a + 100], both[1][0], d_w)
        both[1][1][a:a + 100] = d_w
    for one, many in zip(*both):
        assert torch.equal(one, many)
    used = torch.zeros(R, dtype=torch.bool, device=DEV)
    used[row_of[row_of >= 0].long()] = True
    assert (both[0][0][~used] == 9).all() and int((~used).sum()) == 3 + T * topk // 50


@pytest.mark.parametrize("N", [1536, 1003])
def test_combine_bwd_two_pairs_of_one_row(N):
    """Each element of the row receives one of the two products; both pairs' weights their gradients."""
    T, topk, R = 6, 2, 5
    row_of = torch.tensor([[0, 0], [1, 2], [2, 3], [-1, 4], [4, -1], [R, -1]], dtype=torch.int32)
    dy, out = eu.normal((T, N), 1, 0.5), eu.normal((R, N), 2)
    w = torch.rand((T, topk), generator=eu.gen(3)) + 0.1
    d_out, d_w = fp8bs.moe_combine_bwd(dy.to(DEV), out.to(DEV), w.to(DEV), row_of.to(DEV))
    _, ref_w, size = eu.combine_bwd(dy, out, w, row_of)
    eu.inside(d_w, ref_w, size * (N / 64 + 16) * eu.H_F32, "d_w")
    for row in range(R):
        each = [(w[t, k] * dy[t].float()).to(BF16) for t in range(T) for k in range(topk) if row_of[t, k] == row]
        assert torch.stack([d_out[row].cpu() == e for e in each]).any(0).all(), row


def test_combine_bwd_beyond_32_bits():
    """Rows past 2^31 elements of out and d_out."""
    R, N = 300000, 7168
    out = torch.zeros((R, N), dtype=BF16, device=DEV)
    row_of = torch.tensor([[R - 1, 5], [R - 2, 0]], dtype=torch.int32, device=DEV)
    out[R - 1] = 1.0
    dy = torch.ones((2, N), dtype=BF16, device=DEV)
    d_out, d_w = torch.zeros_like(out), torch.zeros((2, 2), device=DEV)
    fp8bs.fp8bs_moe_combine_bwd(dy, out, torch.tensor([[2.0, 3.0], [4.0, 5.0]], device=DEV), row_of, d_out, d_w)
    assert d_w.tolist() == [[7168.0, 0.0], [0.0, 0.0]]
    assert [float(d_out[r, N - 1]) for r in (R - 1, R - 2, R - 3, 0, 5)] == [2.0, 4.0, 0.0, 5.0, 3.0]
