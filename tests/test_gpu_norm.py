"""fp8bs_rmsnorm and fp8bs_rmsnorm_bwd against values in 64 bits."""
import pytest
import torch

import block_scaled_fp8_03_amd as fp8bs
import expert_util as eu

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6
# every layout of a row: 16, 32 and 64 lanes (full and not), a workgroup with 1, 2 and 4 vectors a lane
WIDTHS = [128, 256, 384, 512, 640, 1536, 2048, 4096, 4224, 7168, 16384, 18432, 32768]


def _poisoned(shape, dtype):
    if dtype == eu.FP8:
        return torch.full(shape, 0x7F, dtype=torch.uint8, device=DEV).view(eu.FP8)
    return torch.full(shape, float("nan"), dtype=dtype, device=DEV)


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("res,w_type,fmt,pad,M", [
    (None, BF16, "fp32", 0, 1), (BF16, BF16, "ue8m0", 8, 3), (F32, F32, "fp32", 576, 17), (BF16, F32, "fp32", 0, 33),
])
def test_norm(K, res, w_type, fmt, pad, M):
    x = eu.normal((M, K + pad), 1, 2.0)[:, :K]
    r = None if res is None else eu.normal((M, K), 2, 3.0, res)
    w = eu.normal((K,), 3, 1.0, w_type)
    t, c = eu.norm(x, r, w, EPS)
    rel = eu.norm_rel(K)
    xd = eu.normal((M, K + pad), 1, 2.0).to(DEV)[:, :K]
    rd = None if r is None else r.to(DEV)
    q, s = _poisoned((M, K), eu.FP8), _poisoned((M, K // 128), F32)
    y, h = _poisoned((M, K), BF16), None if r is None else _poisoned((M, K), res)
    fp8bs.fp8bs_rmsnorm(xd, rd, h, w.to(DEV), EPS, y, q, s, fmt)
    eu.inside(y, c, c.abs() * (eu.H_BF16 + rel), "y")
    eu.check_codes(q, s, c, rel, fmt == "ue8m0", "codes")
    if r is not None:
        assert torch.equal(h.cpu(), (x.float() + r.float()).to(res)), "the sum is float32, rounded once"
    # the outputs apart are the same ones
    y2 = fp8bs.rmsnorm(xd, w.to(DEV), EPS, rd)
    q2 = fp8bs.rmsnorm_quant(xd, w.to(DEV), EPS, rd, fmt)
    assert torch.equal(y2 if r is None else y2[0], y)
    assert torch.equal(q2[0].view(torch.uint8), q.view(torch.uint8)) and torch.equal(q2[1], s)
    if r is not None:
        assert torch.equal(y2[1], h) and torch.equal(q2[2], h)
        # in place
        again = rd.clone()
        y3 = torch.empty_like(y)
        fp8bs.fp8bs_rmsnorm(xd, again, again, w.to(DEV), EPS, y3, None, None)
        assert torch.equal(again, h) and torch.equal(y3, y)


def test_norm_rows_of_their_own():
    """Rows of zeros, of one value, of large and small ones, next to each other; and broadcast rows."""
    K = 1536
    x = torch.zeros((6, K), dtype=BF16)
    x[1] = 5.0
    x[2] = 1e15
    x[3] = 1e-15
    x[4, 7] = 3e4
    x[5, ::2] = -2.0
    w = eu.normal((K,), 3, 1.0)
    _, c = eu.norm(x, None, w, EPS)
    q, s, y = fp8bs.rmsnorm_quant(x.to(DEV), w.to(DEV), EPS, return_y=True)
    eu.inside(y, c, c.abs() * (eu.H_BF16 + eu.norm_rel(K)), "y")
    eu.check_codes(q, s, c, eu.norm_rel(K), False, "codes")
    one = eu.normal((1, K), 4).to(DEV)
    many = fp8bs.rmsnorm(one.expand(5, K), w.to(DEV), EPS)
    assert torch.equal(many, fp8bs.rmsnorm(one, w.to(DEV), EPS).expand(5, K))
    # squares beyond float32: zeros
    assert (fp8bs.rmsnorm(torch.full((1, K), 1e30, dtype=BF16, device=DEV), w.to(DEV), EPS) == 0).all()


@pytest.mark.parametrize("K", [512, 1536])
@pytest.mark.parametrize("fmt", ["fp32", "ue8m0"])
def test_infinities_and_nan_stay_in_their_rows(K, fmt):
    """A weight beyond what float32 holds of its column, one that is NaN; a row with an infinity, one with a NaN."""
    M, inf, nan = 12, float("inf"), float("nan")
    x, w = eu.normal((M, K), 1, 2.0), eu.normal((K,), 2, 1.0)
    x[4, 7], x[6, 300], x[9, 5] = inf, nan, -inf
    w[130], w[200], w[400] = 3e38, nan, inf
    _, c = eu.norm(x, None, w, EPS)
    # the row's squares are infinite: zeros, and NaN where an infinity is divided by their root
    c = torch.where(x.isinf().any(1, keepdim=True), x.double() * 0 * w.double(), c).float()
    q, s, y = fp8bs.rmsnorm_quant(x.to(DEV), w.to(DEV), EPS, None, fmt, return_y=True)
    eu.inside(y, c.double(), c.double().abs().nan_to_num(0, 0) * (eu.H_BF16 + eu.norm_rel(K)), "y")
    eu.check_special_codes(q, s, c, eu.norm_rel(K), fmt == "ue8m0", "codes")
    assert c.isinf().any() and s.isinf().any()


def test_norm_no_rows():
    w = torch.ones(256, dtype=BF16, device=DEV)
    q, s, y = fp8bs.rmsnorm_quant(torch.empty((0, 256), dtype=BF16, device=DEV), w, EPS, return_y=True)
    assert q.shape == (0, 256) and s.shape == (0, 2) and y.shape == (0, 256)


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("h_type,w_type,dres,pad,M", [
    (BF16, BF16, True, 0, 1), (F32, BF16, False, 8, 33), (BF16, F32, True, 64, 7), (F32, F32, True, 0, 1200),
])
def test_norm_bwd(K, h_type, w_type, dres, pad, M):
    M = min(M, 1 + (4 << 20) // K)
    dy, hp = eu.normal((M, K), 5, 0.5), eu.normal((M, K + pad), 6, 2.0, h_type)
    w, dr = eu.normal((K,), 7, 1.0, w_type), eu.normal((M, K), 8, 0.5, h_type) if dres else None
    dx, bound, dw, dw_bound = eu.norm_bwd(dy, hp[:, :K], w, EPS, dr)
    half = eu.H_BF16 if h_type == BF16 else eu.H_F32
    drd = dr.to(DEV) if dres else None
    hd = hp.to(DEV)[:, :K]
    got, got_w = fp8bs.rmsnorm_bwd(dy.to(DEV), hd, w.to(DEV), EPS, drd)
    assert got.dtype == h_type
    eu.inside(got, dx, dx.abs() * half + bound * (1 + half), "dx")
    eu.inside(got_w, dw, dw_bound, "dw")
    # without dw, and onto dres itself
    onto = drd.clone() if dres else torch.empty_like(got)
    fp8bs.fp8bs_rmsnorm_bwd(dy.to(DEV), hd, w.to(DEV), EPS, onto if dres else None, onto, None, None)
    assert torch.equal(onto, got)
    for _ in range(3):
        a, b = fp8bs.rmsnorm_bwd(dy.to(DEV), hd, w.to(DEV), EPS, drd)
        assert torch.equal(a, got) and torch.equal(b, got_w), "the same from call to call"


@pytest.mark.parametrize("K", [256, 1536, 32768])
def test_norm_bwd_rows_beyond_float32(K):
    """A row whose squares sum to infinity, forward a constant 0: dres goes through, nothing to the weight; its neighbours are
    as without it.  A row of zeros likewise has its own eps."""
    M = 9
    dy, h, dres = eu.normal((M, K), 1, 0.5), eu.normal((M, K), 2, 2.0), eu.normal((M, K), 3, 0.5)
    w = eu.normal((K,), 4)
    h[2], h[5] = 1e25, 0.0
    h[7, 3] = -1e30
    dx, dw = fp8bs.rmsnorm_bwd(dy.to(DEV), h.to(DEV), w.to(DEV), EPS, dres.to(DEV))
    ref, bound, _, _ = eu.norm_bwd(dy, h, w, EPS, dres)
    big = [2, 7]
    assert torch.equal(dx[big].cpu(), dres[big])
    rest = [r for r in range(M) if r not in big]
    eu.inside(dx[rest], ref[rest], ref[rest].abs() * eu.H_BF16 + bound[rest] * 1.01, "dx")
    _, _, ref_w, bound_w = eu.norm_bwd(dy[rest], h[rest], w, EPS, None)
    eu.inside(dw, ref_w, bound_w, "dw")


def test_norm_bwd_no_rows():
    w = torch.ones(256, dtype=BF16, device=DEV)
    e = torch.empty((0, 256), dtype=BF16, device=DEV)
    dx, dw = fp8bs.rmsnorm_bwd(e, e, w, EPS)
    assert dx.shape == (0, 256) and (dw == 0).all()


@pytest.mark.parametrize("M,K", [(5, 512), (9, 1536)])
def test_norm_bwd_differences(M, K):
    """Along directions, against differences of the forward formula in 64 bits."""
    dy, h, w = eu.normal((M, K), 1), eu.normal((M, K), 2, 2.0, F32), eu.normal((K,), 3, 1.0, F32)
    dx, dw = fp8bs.rmsnorm_bwd(dy.to(DEV), h.to(DEV), w.to(DEV), EPS)
    f = lambda hh, ww: (eu.norm(hh, None, ww, EPS)[1] * dy.double()).sum()  # noqa: E731
    step = 1e-5
    for seed in range(3):
        v, u = eu.normal((M, K), 10 + seed, 1.0, F32).double(), eu.normal((K,), 20 + seed, 1.0, F32).double()
        by_h = (f(h.double() + step * v, w) - f(h.double() - step * v, w)) / (2 * step)
        by_w = (f(h.double(), w.double() + step * u) - f(h.double(), w.double() - step * u)) / (2 * step)
        _, bound, _, dw_bound = eu.norm_bwd(dy, h, w, EPS, None)
        # the gradient's own bound along the direction, its rounding, and a difference of step^2
        eu.inside((dx.double().cpu() * v).sum(), by_h, ((bound + dx.double().cpu().abs() * eu.H_F32) * v.abs()).sum()
                  + 1e-6, "by h")
        eu.inside((dw.double().cpu() * u).sum(), by_w, (dw_bound * u.abs()).sum() + 1e-6, "by w")


def _on_device(shape, gen, std, dtype):
    return (torch.randn(shape, device=DEV, generator=gen) * std).to(dtype)


@pytest.mark.parametrize("M,K,res", [(4096, 7168, BF16), (4096, 7168, F32), (8001, 7168, None), (60001, 384, BF16),
                                     (70001, 256, F32), (3000, 16384, BF16), (1200, 32768, None)])
def test_norm_many_rows_as_few(M, K, res):
    """More than 160 MB, where inputs are read with a hint: bit by bit what a few rows at a time give."""
    g = torch.Generator(DEV)
    g.manual_seed(K)
    x, w = _on_device((M, K), g, 2.0, BF16), _on_device((K,), g, 1.0, BF16)
    r = None if res is None else _on_device((M, K), g, 3.0, res)
    assert M * K * (5 + {None: 0, BF16: 4, F32: 8}[res]) > 160 << 20
    got = fp8bs.rmsnorm_quant(x, w, EPS, r, return_y=True)
    few = (24 << 20) // (K * 13)
    for a in range(0, M, few):
        rows = slice(a, min(a + few, M))
        part = fp8bs.rmsnorm_quant(x[rows], w, EPS, None if r is None else r[rows], return_y=True)
        for one, many in zip(part, got):
            assert torch.equal(one.view(torch.uint8), many[rows].view(torch.uint8)), a


@pytest.mark.parametrize("M,K,h_type,w_type", [(4096, 7168, BF16, BF16), (2001, 7168, F32, F32), (60001, 384, BF16, F32),
                                               (90001, 256, BF16, BF16), (200001, 128, BF16, BF16), (11001, 2048, BF16, BF16),
                                               (1700, 16384, BF16, BF16), (1500, 18432, BF16, BF16), (900, 32768, F32, BF16)])
def test_norm_bwd_many_rows_as_few(M, K, h_type, w_type):
    """The same of the gradient by the rows; the weight's against its sum in 64 bits."""
    g = torch.Generator(DEV)
    g.manual_seed(K)
    dy, h = _on_device((M, K), g, 0.5, BF16), _on_device((M, K), g, 2.0, h_type)
    dres, w = _on_device((M, K), g, 0.5, h_type), _on_device((K,), g, 1.0, w_type)
    assert M * K * (8 if h_type == BF16 else 14) > 160 << 20
    dx, dw = fp8bs.rmsnorm_bwd(dy, h, w, EPS, dres)
    few = (24 << 20) // (K * 14)
    for a in range(0, M, few):
        rows = slice(a, min(a + few, M))
        part, _ = fp8bs.rmsnorm_bwd(dy[rows], h[rows], w, EPS, dres[rows])
        assert torch.equal(part, dx[rows]), a
    each = dy.double() * h.double() / (h.double().square().mean(-1, keepdim=True) + EPS).sqrt()
    eu.inside(dw, each.sum(0), each.abs().sum(0) * (eu.norm_rel(K) + (M + 32) * eu.H_F32), "dw")
    again, dw2 = fp8bs.rmsnorm_bwd(dy, h, w, EPS, dres)
    assert torch.equal(again, dx) and torch.equal(dw2, dw)


def test_norm_last_rows_beyond_32_bits():
    """Offsets past 2^31 elements: the last rows of a strided input and of large outputs."""
    K, ld, M = 7168, 1 << 16, 40000
    buf = torch.zeros(M * ld, dtype=BF16, device=DEV)          # 2.6e9 elements
    x = buf.view(M, ld)[:, :K]
    some = eu.normal((3, K), 1)
    x[M - 3:] = some.to(DEV)
    w = eu.normal((K,), 2).to(DEV)
    y = fp8bs.rmsnorm(x, w, EPS)
    assert torch.equal(y[M - 3:], fp8bs.rmsnorm(some.to(DEV), w, EPS)) and (y[:M - 3] == 0).all()


@pytest.mark.parametrize("M,K", [(67108860, 128), (4194303, 640)])
def test_norm_most_rows(M, K):
    """As many rows as one launch has; all alike, read by a stride of 0."""
    one, w = eu.normal((1, K), 1).to(DEV), eu.normal((K,), 2).to(DEV)
    y = fp8bs.rmsnorm(one.expand(M, K), w, EPS)
    want = fp8bs.rmsnorm(one, w, EPS)
    for at in (0, M // 2, M - 5):
        assert torch.equal(y[at:at + 5], want.expand(5, K))
    assert torch.equal(y[::4099], want.expand(y[::4099].shape[0], K))
