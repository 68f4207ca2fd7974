"""Host checks of the expert block's entry points (norm, gate, balance, activation,
their gradients, the combine's): bad arguments are refused before any HIP call
(the addresses below are never touched), and the binding refuses tensors that
do not fit."""
import os
import re

import pytest
import torch

import block_scaled_fp8_03_amd as fp8bs

OK, NULL, SHAPE, ALIGN, ENUM, HIP, ALIAS = 0, 1, 2, 3, 4, 5, 6
A = [0x100000000 * (i + 1) for i in range(16)]
INF, NAN = float("inf"), float("nan")

NORM = dict(x=A[0], ld=256, res=A[1], res_out=A[2], res_type=0, w=A[3], w_f32=0, eps=1e-6, y=A[4], q=A[5], s=A[6], fmt=0,
            M=4, K=256, stream=None)
NORM_BWD = dict(dy=A[0], h=A[1], ld=256, h_type=0, w=A[2], w_f32=0, eps=1e-6, dres=A[3], dx=A[4], dw=A[5], M=4000, K=256,
                ws=A[6], nws=1 << 40, stream=None)
GATE = dict(z=A[0], ld=64, z_type=1, bias=A[1], T=4, E=64, topk=6, groups=4, keep=2, score=0, norm=1, scale=1.0, idx=A[2],
            w=A[3], stream=None)
BALANCE = dict(z=A[0], ld=64, z_type=1, idx=A[1], cu=A[2], T=4000, S=2, E=64, topk=6, score=0, counts=A[3], probs=A[4],
               loss=A[5], ws=A[6], nws=1 << 40, stream=None)
GATE_BWD = dict(z=A[0], ld=64, z_type=1, idx=A[1], dw=A[2], score=0, norm=1, scale=1.0, cu=A[3], counts=A[4], dl=A[5], T=4,
                S=2, E=64, topk=6, out=A[6], out_type=1, stream=None)
SWIGLU = dict(g=A[0], ld_g=256, u=A[1], ld_u=256, n=A[2], y=A[3], q=A[4], s=A[5], fmt=0, M=4, N=256, stream=None)
SWIGLU_BWD = dict(dy=A[0], g=A[1], ld_g=256, u=A[2], ld_u=256, n=A[3], dg=A[4], ld_dg=256, du=A[5], ld_du=256, M=4, N=256,
                  stream=None)
COMBINE_BWD = dict(dy=A[0], dy_type=0, out=A[1], w=A[2], row_of=A[3], d_out=A[4], d_w=A[5], T=4, topk=2, R=8, N=64,
                   stream=None)
ALL = {"fp8bs_rmsnorm": NORM, "fp8bs_rmsnorm_bwd": NORM_BWD, "fp8bs_moe_gate": GATE, "fp8bs_moe_balance": BALANCE,
       "fp8bs_moe_gate_bwd": GATE_BWD, "fp8bs_swiglu": SWIGLU, "fp8bs_swiglu_bwd": SWIGLU_BWD,
       "fp8bs_moe_combine_bwd": COMBINE_BWD}

# (entry point, status): changes of one argument or more that give it
REFUSED = [
    ("fp8bs_rmsnorm", SHAPE, [dict(M=-1), dict(K=-128), dict(K=200), dict(K=32768 + 128), dict(M=1 << 22, K=640), dict(M=1 << 26),
                              dict(ld=-8), dict(eps=-1.0), dict(eps=INF), dict(eps=NAN), dict(ld=1 << 62)]),
    ("fp8bs_rmsnorm", ENUM, [dict(res_type=2), dict(fmt=2), dict(fmt=-1)]),
    ("fp8bs_rmsnorm", NULL, [dict(x=None), dict(w=None), dict(res=None), dict(res_out=None), dict(q=None), dict(s=None),
                             dict(y=None, q=None, s=None)]),
    ("fp8bs_rmsnorm", ALIGN, [dict(ld=260), dict(x=A[0] + 8), dict(w=A[3] + 2), dict(res=A[1] + 8), dict(res_out=A[2] + 8),
                              dict(y=A[4] + 8), dict(q=A[5] + 8), dict(s=A[6] + 2)]),
    ("fp8bs_rmsnorm", ALIAS, [dict(y=A[0]), dict(q=A[0] + 16), dict(res_out=A[1] + 16), dict(y=A[1] + 512), dict(res_out=A[0]),
                              dict(q=A[4] + 1024), dict(s=A[5] + 512), dict(y=A[3] + 256), dict(y=A[2]),
                              dict(res=A[0], res_out=A[0])]),
    ("fp8bs_rmsnorm_bwd", SHAPE, [dict(M=-1), dict(K=100), dict(ld=-8), dict(eps=NAN), dict(nws=0), dict(K=1 << 16)]),
    ("fp8bs_rmsnorm_bwd", ENUM, [dict(h_type=2)]),
    ("fp8bs_rmsnorm_bwd", NULL, [dict(dy=None), dict(h=None), dict(w=None), dict(dx=None), dict(ws=None)]),
    ("fp8bs_rmsnorm_bwd", ALIGN, [dict(ld=257), dict(dy=A[0] + 8), dict(h=A[1] + 8), dict(w=A[2] + 8), dict(dres=A[3] + 8),
                                  dict(dx=A[4] + 8), dict(dw=A[5] + 4), dict(ws=A[6] + 8)]),
    ("fp8bs_rmsnorm_bwd", ALIAS, [dict(dx=A[0]), dict(dx=A[1]), dict(dx=A[3] + 16), dict(dw=A[2]), dict(ws=A[4]),
                                  dict(dw=A[4] + 1024), dict(ws=A[1])]),
    ("fp8bs_moe_gate", SHAPE, [dict(T=-1), dict(T=1 << 24), dict(E=0), dict(E=1025, groups=1), dict(topk=0), dict(topk=65, E=128),
                               dict(topk=9, E=8), dict(groups=3), dict(groups=0), dict(keep=0), dict(keep=5), dict(ld=-1),
                               dict(groups=128, E=128, keep=1), dict(scale=INF), dict(scale=NAN), dict(ld=1 << 62)]),
    ("fp8bs_moe_gate", ENUM, [dict(z_type=2), dict(score=2), dict(score=-1)]),
    ("fp8bs_moe_gate", NULL, [dict(z=None), dict(idx=None), dict(w=None)]),
    ("fp8bs_moe_gate", ALIGN, [dict(z=A[0] + 2), dict(z=A[0] + 1, z_type=0), dict(bias=A[1] + 2), dict(idx=A[2] + 1),
                               dict(w=A[3] + 2)]),
    ("fp8bs_moe_gate", ALIAS, [dict(idx=A[0] + 64), dict(w=A[2] + 16), dict(w=A[1])]),
    ("fp8bs_moe_balance", SHAPE, [dict(T=-1), dict(S=-1), dict(S=1 << 22), dict(E=1025), dict(topk=65), dict(nws=0),
                                  dict(cu=None), dict(ld=-1)]),
    ("fp8bs_moe_balance", ENUM, [dict(z_type=3), dict(score=7)]),
    ("fp8bs_moe_balance", NULL, [dict(z=None), dict(idx=None), dict(counts=None), dict(probs=None), dict(loss=None),
                                 dict(ws=None)]),
    ("fp8bs_moe_balance", ALIGN, [dict(z=A[0] + 2), dict(idx=A[1] + 2), dict(cu=A[2] + 2), dict(counts=A[3] + 1),
                                  dict(probs=A[4] + 2), dict(loss=A[5] + 2), dict(ws=A[6] + 8)]),
    ("fp8bs_moe_balance", ALIAS, [dict(counts=A[1]), dict(probs=A[3] + 256), dict(loss=A[2] + 4), dict(ws=A[0] + 16),
                                  dict(ws=A[4])]),
    ("fp8bs_moe_gate_bwd", SHAPE, [dict(T=-1), dict(S=0), dict(S=-1), dict(cu=None), dict(E=2000), dict(scale=-INF), dict(ld=-4)]),
    ("fp8bs_moe_gate_bwd", ENUM, [dict(z_type=2), dict(score=2), dict(out_type=2)]),
    ("fp8bs_moe_gate_bwd", NULL, [dict(z=None), dict(idx=None), dict(counts=None), dict(out=None)]),
    ("fp8bs_moe_gate_bwd", ALIGN, [dict(z=A[0] + 2), dict(idx=A[1] + 2), dict(dw=A[2] + 2), dict(cu=A[3] + 2),
                                   dict(counts=A[4] + 2), dict(dl=A[5] + 2), dict(out=A[6] + 8)]),
    ("fp8bs_moe_gate_bwd", ALIAS, [dict(out=A[0]), dict(out=A[1] + 16), dict(out=A[2]), dict(out=A[4] + 256), dict(out=A[5])]),
    ("fp8bs_swiglu", SHAPE, [dict(M=-1), dict(N=-128), dict(N=192), dict(ld_g=-8), dict(ld_u=-8), dict(M=1 << 40),
                             dict(ld_g=1 << 62), dict(N=1 << 31)]),
    ("fp8bs_swiglu", ENUM, [dict(fmt=5)]),
    ("fp8bs_swiglu", NULL, [dict(g=None), dict(u=None), dict(q=None), dict(s=None), dict(y=None, q=None, s=None)]),
    ("fp8bs_swiglu", ALIGN, [dict(ld_g=260), dict(ld_u=4), dict(g=A[0] + 8), dict(u=A[1] + 2), dict(n=A[2] + 2),
                             dict(y=A[3] + 8), dict(q=A[4] + 8), dict(s=A[5] + 1)]),
    ("fp8bs_swiglu", ALIAS, [dict(y=A[0]), dict(q=A[1] + 16), dict(s=A[4]), dict(s=A[2]), dict(y=A[4] - 1024)]),
    ("fp8bs_swiglu_bwd", SHAPE, [dict(M=-1), dict(N=64), dict(ld_dg=128), dict(ld_du=248), dict(ld_g=-8), dict(ld_du=-256)]),
    ("fp8bs_swiglu_bwd", NULL, [dict(dy=None), dict(g=None), dict(u=None), dict(dg=None), dict(du=None)]),
    ("fp8bs_swiglu_bwd", ALIGN, [dict(ld_g=4), dict(ld_u=4), dict(ld_dg=260), dict(ld_du=260), dict(dy=A[0] + 8),
                                 dict(g=A[1] + 8), dict(u=A[2] + 8), dict(n=A[3] + 1), dict(dg=A[4] + 8), dict(du=A[5] + 8)]),
    ("fp8bs_swiglu_bwd", ALIAS, [dict(dg=A[1]), dict(du=A[0] + 16), dict(du=A[4]), dict(du=A[4] + 512, ld_dg=320, ld_du=320),
                                 dict(du=A[4] + 256, ld_dg=512, ld_du=512), dict(du=A[4] + 512, ld_dg=512, ld_du=1024),
                                 dict(du=A[4] + 768, ld_dg=512, ld_du=512), dict(dg=A[3] - 64)]),
    ("fp8bs_moe_combine_bwd", SHAPE, [dict(T=-1), dict(T=1 << 23), dict(topk=0), dict(R=-1), dict(N=-1), dict(R=1 << 31),
                                      dict(N=1 << 61)]),
    ("fp8bs_moe_combine_bwd", ENUM, [dict(dy_type=2)]),
    ("fp8bs_moe_combine_bwd", NULL, [dict(dy=None), dict(out=None), dict(w=None), dict(row_of=None), dict(d_out=None),
                                     dict(d_w=None)]),
    ("fp8bs_moe_combine_bwd", ALIGN, [dict(dy=A[0] + 8), dict(out=A[1] + 2), dict(w=A[2] + 2), dict(row_of=A[3] + 2),
                                      dict(d_out=A[4] + 8), dict(d_w=A[5] + 2)]),
    ("fp8bs_moe_combine_bwd", ALIAS, [dict(d_out=A[1]), dict(d_out=A[0] + 16), dict(d_w=A[2]), dict(d_w=A[4] + 4),
                                      dict(d_w=A[3] + 16)]),
]

# calls that do nothing: no pointer is looked at
NOTHING = [("fp8bs_rmsnorm", dict(M=0)), ("fp8bs_rmsnorm", dict(K=0)), ("fp8bs_rmsnorm_bwd", dict(M=0, dw=None)),
           ("fp8bs_rmsnorm_bwd", dict(K=0)), ("fp8bs_moe_gate", dict(T=0)), ("fp8bs_moe_balance", dict(S=0)),
           ("fp8bs_moe_gate_bwd", dict(T=0)), ("fp8bs_swiglu", dict(M=0)), ("fp8bs_swiglu", dict(N=0)),
           ("fp8bs_swiglu_bwd", dict(M=0)), ("fp8bs_swiglu_bwd", dict(N=0)), ("fp8bs_moe_combine_bwd", dict(T=0))]


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(fp8bs.library_path):
        from block_scaled_fp8_03_amd import build
        build.build()
    return fp8bs.lib()


def call(L, name, **kw):
    base = ALL[name]
    assert set(kw) <= set(base)
    return getattr(L, name)(*{**base, **kw}.values())


@pytest.mark.parametrize("name,status,changes", REFUSED, ids=[f"{n}-{s}" for n, s, _ in REFUSED])
def test_refusals(L, name, status, changes):
    for kw in changes:
        assert call(L, name, **kw) == status, kw


@pytest.mark.parametrize("name,kw", NOTHING)
def test_nothing_to_do(L, name, kw):
    assert call(L, name, **kw) == OK
    pointers = {k: None for k, v in ALL[name].items() if v in A and k not in kw and k != "cu" and k != "dl"}
    assert call(L, name, **{**pointers, **kw}) == OK


def test_workspace_sizes(L):
    f, g = L.fp8bs_rmsnorm_bwd_workspace_size, L.fp8bs_moe_balance_workspace_size
    assert f(0, 256) == 0 and f(1, 7168) == 0 and f(4096, 7168) > 0
    assert f(-1, 256) == f(1, 100) == f(1, 1 << 16) == f(1 << 22, 1024) == f(1 << 26, 128) == -1
    assert g(0, 1, 64) == g(100, 0, 64) == 0 and g(4096, 1, 256) > 0
    assert g(-1, 1, 64) == g(1 << 24, 1, 64) == g(1, -1, 64) == g(1, 1, 0) == g(1, 1, 1025) == g(1, 1 << 22, 64) == -1


def test_float32_sums_stay_in_32_bits(tmp_path):
    """The balance and the gate's gradient sum floats over a wave: by DPP steps, with no 64-bit additions and no exchanges
    through LDS, which a sum in 64 bits that takes a float's place would bring."""
    from block_scaled_fp8_03_amd import build
    out = str(tmp_path / "gate.s")
    build._run([build.HIPCC, *build.COMMON_FLAGS, *build.HIP_FLAGS, *build.VGPR_FORM, "-x", "hip", "-S", "--cuda-device-only",
                os.path.join(build.CSRC, "gate.hip"), "-o", out])
    with open(out) as f:
        text = f.read()
    kernels = re.findall(r"^(_ZN5fp8bs\d+moe_(?:balance|balance_join|gate_bwd)_kernel\w*):.*?$(.*?)^\s+s_endpgm$", text, re.M | re.S)
    assert len(kernels) == 9 * 3 + 1              # 1 to 16 experts a lane, loads wide or not; the balance twice
    for name, body in kernels:
        found = re.findall(r"v_add_f64\w*|ds_bpermute_b32|ds_swizzle_b32", body)
        assert not found, (name, found)


# --------------------------------------------------------------- the binding

def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def f32(*s):
    return torch.zeros(s)


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def test_cpu_tensors_are_refused(L):
    w = bf(256)
    for f in (lambda: fp8bs.rmsnorm(bf(2, 256), w, 1e-6), lambda: fp8bs.rmsnorm_bwd(bf(2, 256), bf(2, 256), w, 1e-6),
              lambda: fp8bs.moe_gate(f32(2, 64), 6), lambda: fp8bs.moe_balance(f32(2, 64), i32(2, 6)),
              lambda: fp8bs.moe_gate_bwd(f32(2, 64), i32(2, 6), f32(2, 6)), lambda: fp8bs.swiglu(bf(2, 256), bf(2, 256)),
              lambda: fp8bs.swiglu_bwd(bf(2, 256), bf(2, 256), bf(2, 256)),
              lambda: fp8bs.moe_combine_bwd(bf(2, 64), bf(4, 64), f32(2, 2), i32(2, 2))):
        with pytest.raises(ValueError, match="must be a device tensor"):
            f()


def test_tensors_that_do_not_fit(L):
    w = bf(256)
    bad = [
        (TypeError, lambda: fp8bs.rmsnorm([1.0], w, 1e-6)), (ValueError, lambda: fp8bs.rmsnorm(bf(256), w, 1e-6)),
        (TypeError, lambda: fp8bs.rmsnorm(f32(2, 256), w, 1e-6)), (ValueError, lambda: fp8bs.rmsnorm(bf(2, 256), bf(128), 1e-6)),
        (ValueError, lambda: fp8bs.rmsnorm(bf(256, 2).t(), w, 1e-6)),
        (ValueError, lambda: fp8bs.rmsnorm(bf(2, 256), w, 1e-6, bf(3, 256))),
        (TypeError, lambda: fp8bs.rmsnorm(bf(2, 256), w, 1e-6, bf(2, 256).half())),
        (TypeError, lambda: fp8bs.fp8bs_rmsnorm(bf(2, 256), bf(2, 256), f32(2, 256), w, 1e-6, bf(2, 256), None, None)),
        (ValueError, lambda: fp8bs.rmsnorm_quant(bf(2, 256), w, 1e-6, scale_fmt="e5m2")),
        (TypeError, lambda: fp8bs.rmsnorm_bwd(f32(2, 256), bf(2, 256), w, 1e-6)),
        (TypeError, lambda: fp8bs.rmsnorm_bwd(bf(2, 256), bf(2, 256), w, 1e-6, f32(2, 256))),
        (ValueError, lambda: fp8bs.rmsnorm_bwd(bf(2, 256), bf(2, 250), bf(250), 1e-6)),
        (ValueError, lambda: fp8bs.moe_gate(f32(64), 6)), (TypeError, lambda: fp8bs.moe_gate(f32(2, 64).double(), 6)),
        (ValueError, lambda: fp8bs.moe_gate(f32(2, 64), 6, score="tanh")),
        (ValueError, lambda: fp8bs.moe_gate(f32(2, 64), 6, f32(63))), (TypeError, lambda: fp8bs.moe_gate(f32(2, 64), 6, bf(64))),
        (ValueError, lambda: fp8bs.moe_balance(f32(2, 64), i32(3, 6))),
        (TypeError, lambda: fp8bs.moe_balance(f32(2, 64), f32(2, 6))),
        (ValueError, lambda: fp8bs.moe_balance(f32(2, 64), i32(2, 6), i32(2, 2))),
        (TypeError, lambda: fp8bs.moe_balance(f32(2, 64), i32(2, 6), [0, 2])),
        (TypeError, lambda: fp8bs.moe_balance(f32(2, 64), i32(2, 6), i32(2).long())),
        (ValueError, lambda: fp8bs.moe_balance(f32(2, 2000), i32(2, 6))),
        (ValueError, lambda: fp8bs.moe_gate_bwd(f32(2, 64), i32(2, 6), f32(2, 5))),
        (ValueError, lambda: fp8bs.moe_gate_bwd(f32(2, 64), i32(2, 6), counts=i32(2, 64), d_loss=f32(2))),
        (TypeError, lambda: fp8bs.moe_gate_bwd(f32(2, 64), i32(2, 6), out_dtype=torch.float16)),
        (ValueError, lambda: fp8bs.swiglu(bf(2, 256), bf(2, 128))), (TypeError, lambda: fp8bs.swiglu(bf(2, 256), f32(2, 256))),
        (ValueError, lambda: fp8bs.swiglu(bf(2, 256), bf(2, 256), i32(2))),
        (TypeError, lambda: fp8bs.swiglu(bf(2, 256), bf(2, 256), 2)),
        (TypeError, lambda: fp8bs.swiglu(bf(2, 256), bf(2, 256), f32(1))),
        (ValueError, lambda: fp8bs.swiglu_bwd(bf(2, 128), bf(2, 256), bf(2, 256))),
        (ValueError, lambda: fp8bs.moe_combine_bwd(bf(3, 64), bf(4, 64), f32(2, 2), i32(2, 2))),
        (TypeError, lambda: fp8bs.moe_combine_bwd(bf(2, 64), f32(4, 64), f32(2, 2), i32(2, 2))),
        (TypeError, lambda: fp8bs.moe_combine_bwd(bf(2, 64), bf(4, 64), f32(2, 2), i32(2, 2).long())),
    ]
    for n, (kind, f) in enumerate(bad):
        with pytest.raises(kind):
            f()
            pytest.fail(f"call {n} was taken")
