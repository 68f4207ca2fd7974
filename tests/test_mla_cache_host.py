"""Host checks of the paged MLA cache's entry points: bad arguments are refused
before any HIP call (the addresses below are never touched), and the binding
refuses tensors that do not fit.  Also that the attention kernel's listing
leaves the accumulator registers to the kernel."""
import os

import pytest
import torch

import block_scaled_fp8_03_amd as fp8bs

OK, NULL, SHAPE, ALIGN, ENUM, HIP, ALIAS = 0, 1, 2, 3, 4, 5, 6
A = [0x10000000 * (i + 1) for i in range(16)]
INF = float("inf")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(fp8bs.library_path):
        from block_scaled_fp8_03_amd import build
        build.build()
    return fp8bs.lib()


WRITE = dict(q=A[0], ldq_t=768, ldq_h=192, kv=A[1], ld_kv=576, w=A[2], w_f32=0, eps=1e-6, cs=A[3], n_pos=100, q_out=A[4],
             latent=A[5], scale=None, rope=A[6], fmt=0, table=A[7], cu=A[8], lens=A[9], T=4, H=4, B=2, W=3, P=10, ps=16,
             R=512, dr=64, stream=None)
ATTN = dict(q=A[0], ldq_t=2048, ldq_h=512, qr=A[1], ldr_t=256, ldr_h=64, latent=A[2], scale=None, rope=A[3], fmt=0,
            table=A[4], cu=A[5], lens=A[6], sm=0.1, causal=1, out=A[7], dt=0, lse=A[8], T=4, H=4, B=2, W=3, P=10, ps=16,
            R=512, dr=64, ws=A[9], nws=1 << 40, stream=None)
UPDATE = dict(latent=A[0], scale=None, rope=A[1], fmt=0, table=A[2], lens=A[3], parent=A[4], new=A[5], tout=A[6], lout=A[7],
              B=2, N=3, W=3, P=20000, ps=1, R=512, dr=64, ws=A[8], nws=1 << 40, stream=None)
COMPACT = dict(latent=A[0], scale=None, rope=A[1], fmt=0, table=A[2], lens=A[3], tout=A[4], count=A[5], B=2, W=3, P=140000,
               ps=1, R=512, dr=64, ws=A[6], nws=1 << 40, stream=None)


def call(f, base, **kw):
    assert set(kw) <= set(base)
    return f(*{**base, **kw}.values())


@pytest.mark.parametrize("name,base,floats", [
    ("fp8bs_mla_cache_write", WRITE, ["kv", "q", "q_out", "latent", "rope"]),
    ("fp8bs_mla_attention", ATTN, ["q", "qr", "latent", "rope", "out", "ws"]),
    ("fp8bs_cache_update", UPDATE, ["latent", "rope", "ws"]),
    ("fp8bs_cache_compact", COMPACT, ["latent", "rope", "ws"]),
])
def test_shared_refusals(L, name, base, floats):
    f = getattr(L, name)
    for kw in (dict(R=256), dict(dr=32), dict(B=-1), dict(W=0), dict(P=0), dict(ps=0), dict(ps=4097),
               dict(P=1 << 31), dict(P=1 << 20, ps=4096), dict(W=-3), dict(W=(1 << 30) + 1)):
        assert call(f, base, **kw) == SHAPE, kw
    for kw in (dict(fmt=2), dict(fmt=-1)):
        assert call(f, base, **kw) == ENUM, kw
    assert call(f, base, fmt=1) == NULL                       # codes without scales
    assert call(f, base, fmt=1, scale=A[15] + 4) == ALIGN
    for k in floats:
        assert call(f, base, **{k: None}) == NULL, k
        assert call(f, base, **{k: base[k] + 8}) == ALIGN, k
    for k in ("table", "lens"):
        assert call(f, base, **{k: None}) == NULL, k
        assert call(f, base, **{k: base[k] + 2}) == ALIGN, k


def test_write_refusals(L):
    f = L.fp8bs_mla_cache_write
    for kw in (dict(T=-1), dict(H=-1), dict(n_pos=-1), dict(eps=-1.0), dict(eps=INF), dict(eps=float("nan")),
               dict(ldq_t=-8), dict(ld_kv=-8), dict(T=1 << 31), dict(ldq_t=1 << 62, T=1 << 20)):
        assert call(f, WRITE, **kw) == SHAPE, kw
    for kw in (dict(ldq_t=4), dict(ldq_h=12), dict(ld_kv=577), dict(w=A[2] + 1), dict(w=A[2] + 2, w_f32=1),
               dict(cs=A[3] + 2), dict(cu=A[8] + 1)):
        assert call(f, WRITE, **kw) == ALIGN, kw
    for k in ("w", "cs", "cu"):
        assert call(f, WRITE, **{k: None}) == NULL, k
    for kw in (dict(q_out=A[0]), dict(q_out=A[1] + 16), dict(q_out=A[5] + 1024), dict(kv=A[5]), dict(table=A[6] + 128),
               dict(q_out=A[9])):
        assert call(f, WRITE, **kw) == ALIAS, kw
    assert call(f, WRITE, T=0, kv=None, q=None, q_out=None, w=None) == OK
    assert call(f, WRITE, B=0) == OK


def test_attention_refusals(L):
    f, ws = L.fp8bs_mla_attention, L.fp8bs_mla_attention_workspace_size
    for kw in (dict(T=-1), dict(H=0), dict(T=1 << 24, H=128), dict(B=8193), dict(sm=INF), dict(sm=float("nan")),
               dict(ldq_h=-8), dict(ldr_t=-8)):
        assert call(f, ATTN, **kw) == SHAPE, kw
    for kw in (dict(ldq_t=4), dict(ldr_h=12), dict(lse=A[8] + 2), dict(cu=A[5] + 3)):
        assert call(f, ATTN, **kw) == ALIGN, kw
    assert call(f, ATTN, dt=2) == ENUM
    assert call(f, ATTN, cu=None) == NULL
    need = ws(4, 4, 2)
    for kw in (dict(out=A[0] + 64), dict(lse=A[1]), dict(out=A[2]), dict(lse=A[7] + 16), dict(out=A[4]),
               dict(ws=A[7]), dict(ws=A[3] + 16)):
        assert call(f, ATTN, **kw) == ALIAS, kw
    assert call(f, ATTN, T=0, q=None, out=None) == OK
    assert call(f, ATTN, B=0) == OK
    assert ws(-1, 4, 2) == ws(4, 0, 2) == ws(4, 4, -1) == ws(1 << 24, 128, 2) == ws(4, 4, 8193) == -1
    assert ws(0, 4, 2) == ws(4, 4, 0) == 0
    assert call(f, ATTN, nws=need - 1) == SHAPE


def test_attention_scale_limit(L):
    """|scale| log2(e) has to be a float32: beyond, a score of 0 would be NaN."""
    for sm in (2.31e38, -2.31e38, 3.0e38):
        assert call(L.fp8bs_mla_attention, ATTN, sm=sm) == SHAPE, sm
    for sm in (2.3e38, -2.3e38):                              # accepted: the next check's answer
        assert call(L.fp8bs_mla_attention, ATTN, sm=sm, ldq_t=4) == ALIGN, sm


def test_update_and_compact_refusals(L):
    f, g = L.fp8bs_cache_update, L.fp8bs_cache_compact
    for kw in (dict(N=-1), dict(N=1 << 18), dict(nws=L.fp8bs_cache_update_workspace_size(2, 3, 3, 20000) - 1)):
        assert call(f, UPDATE, **kw) == SHAPE, kw
    for k in ("parent", "new", "tout", "lout"):
        assert call(f, UPDATE, **{k: None}) == NULL, k
        assert call(f, UPDATE, **{k: UPDATE[k] + 2}) == ALIGN, k
    for kw in (dict(tout=A[2]), dict(lout=A[3] + 4), dict(tout=A[0]), dict(ws=A[1] + 16), dict(lout=A[6] + 4), dict(ws=A[4]),
               dict(table=A[0])):
        assert call(f, UPDATE, **kw) == ALIAS, kw
    assert call(f, UPDATE, N=0, parent=None, tout=None) == OK
    assert call(g, COMPACT, nws=L.fp8bs_cache_compact_workspace_size(2, 3, 140000) - 1) == SHAPE
    for k in ("tout", "count"):
        assert call(g, COMPACT, **{k: None}) == NULL, k
        assert call(g, COMPACT, **{k: COMPACT[k] + 2}) == ALIGN, k
    for kw in (dict(tout=A[2]), dict(count=A[3]), dict(tout=A[0]), dict(ws=A[1] + 16), dict(count=A[4] + 4)):
        assert call(g, COMPACT, **kw) == ALIAS, kw
    for sizes in ((2, 3, 3, 0), (2, 1 << 18, 3, 10), (2, -1, 3, 10), (-1, 3, 3, 10), (2, 3, 0, 10), (1 << 24, 3, 3, 10)):
        assert L.fp8bs_cache_update_workspace_size(*sizes) == -1, sizes
    for sizes in ((2, 3, 0), (-1, 3, 10), (2, 0, 10), (1 << 24, 3, 10)):
        assert L.fp8bs_cache_compact_workspace_size(*sizes) == -1, sizes
    assert L.fp8bs_cache_update_workspace_size(2, 0, 3, 20000) == 0
    # small tables need none
    assert L.fp8bs_cache_update_workspace_size(2, 3, 3, 10) == L.fp8bs_cache_compact_workspace_size(2, 3, 10) == 0


def test_update_leaves_one_launch_where_four_are_faster(L):
    """Where four launches win in a graph (50,000 table entries and more) they are taken: they need a workspace."""
    size = L.fp8bs_cache_update_workspace_size
    for B, N, W in ((64, 256, 100), (128, 128, 125), (256, 256, 64)):
        assert size(B, N, W, 16000) == 0, (B, N, W)
    for B, N, W in ((64, 256, 158), (64, 256, 189), (16, 512, 95), (4, 500, 110)):
        assert size(B, N, W, 16000) > 0, (B, N, W)


def test_sizes_beyond_one_launch(L):
    """A workgroup of 256 threads a token or row: 2^24 of them is one too many."""
    assert call(L.fp8bs_mla_cache_write, WRITE, T=1 << 24) == SHAPE
    assert call(L.fp8bs_cache_update, UPDATE, B=(1 << 24) - 3) == SHAPE
    assert call(L.fp8bs_cache_compact, COMPACT, B=1 << 24) == SHAPE


def test_write_number_of_sequences(L):
    """The kernel's search looks at places up to 64 behind the last boundary, in 32 bits."""
    for B in ((1 << 30) + 1, (1 << 31) - 1):
        assert call(L.fp8bs_mla_cache_write, WRITE, B=B, W=1, H=0, table=1 << 44, cu=1 << 45, lens=1 << 46) == SHAPE


def test_cache_arrays_that_overlap(L):
    """The writing entry points refuse a cache whose arrays lie over each other."""
    for name, base in (("fp8bs_mla_cache_write", WRITE), ("fp8bs_cache_update", UPDATE), ("fp8bs_cache_compact", COMPACT)):
        f, tokens = getattr(L, name), base["P"] * base["ps"]
        codes = dict(fmt=1, scale=A[15])
        for kw in (dict(rope=base["latent"]), dict(rope=base["latent"] + tokens * 1024 - 16),
                   dict(latent=base["rope"] + tokens * 128 - 16), dict(codes, rope=base["latent"] + tokens * 512 - 16),
                   dict(codes, scale=base["latent"] + 16), dict(codes, scale=base["rope"] + tokens * 128 - 16)):
            assert call(f, base, **kw) == ALIAS, (name, kw)


def test_binding_refusals():
    """Shapes and types are refused before anything is asked of a device."""
    bf, i32 = torch.bfloat16, torch.int32
    cache = fp8bs.mla_cache_alloc(4, 16, "cpu")
    table, cu, lens = torch.zeros((2, 2), dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32)
    q, qr = torch.zeros((3, 4, 512), dtype=bf), torch.zeros((3, 4, 64), dtype=bf)
    kv, w, cs = torch.zeros((3, 576), dtype=bf), torch.zeros(512), torch.zeros((9, 32, 2))
    with pytest.raises(TypeError):
        fp8bs.mla_cache_alloc(4, 16, "cpu", torch.float16)
    for bad in (dict(q=q[..., :256]), dict(q=q[0]), dict(qr=qr[:2]), dict(qr=qr[:, :3]), dict(cache=fp8bs.MlaCache(
            cache.latent[..., :256], cache.rope)), dict(cache=fp8bs.MlaCache(cache.latent, cache.rope[:3])),
            dict(cache=fp8bs.MlaCache(cache.latent.view(torch.uint8)[..., :512], cache.rope)),
            dict(cache=cache._replace(scale=torch.zeros(4, 16, 4))), dict(q=q), dict(table=table[0])):
        a = {**dict(q=q, qr=qr, cache=cache, table=table, cu=cu, lens=lens), **bad}
        with pytest.raises((ValueError, TypeError)):
            out = torch.empty((3, 4, 512), dtype=bf)
            fp8bs.fp8bs_mla_attention(a["q"], a["qr"], a["cache"], a["table"], a["cu"], a["lens"], 0.1, out, None, out)
    for bad in (dict(kv=kv[:, :512]), dict(kv=kv[:2]), dict(w=w[:8]), dict(cs=cs[..., :1]), dict(qr=qr[..., :32])):
        a = {**dict(qr=qr, kv=kv, w=w, cs=cs), **bad}
        with pytest.raises((ValueError, TypeError)):
            fp8bs.mla_cache_write(a["qr"], a["kv"], a["w"], 1e-6, a["cs"], cache, table, cu, lens)
    with pytest.raises((ValueError, TypeError)):
        fp8bs.cache_update(cache, table, lens, torch.zeros(3, dtype=i32), torch.zeros(3, dtype=i32))
    with pytest.raises((ValueError, TypeError)):
        fp8bs.cache_compact(cache, table, lens)


def test_binding_refuses_what_is_no_tensor():
    """None, numbers and arrays in a tensor's place: a TypeError that names the argument."""
    i32 = torch.int32
    cache = fp8bs.mla_cache_alloc(4, 16, "cpu")
    table, cu, lens = torch.zeros((2, 2), dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32)
    q, qr = torch.zeros((3, 4, 512), dtype=torch.bfloat16), torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    kv, w, cs = torch.zeros((3, 576), dtype=torch.bfloat16), torch.zeros(512), torch.zeros((9, 32, 2))
    out = torch.empty((3, 4, 512), dtype=torch.bfloat16)
    calls = {
        "attention": (fp8bs.fp8bs_mla_attention, dict(q_lat=q, q_rope=qr, cache=cache, table=table, cu_q=cu, lens=lens,
                                                      scale=0.1, out=out, lse=None, workspace=None)),
        "write": (fp8bs.fp8bs_mla_cache_write, dict(q_rope=qr, kv=kv, norm_w=w, eps=1e-6, rope_cs=cs, q_out=qr.clone(),
                                                    cache=cache, table=table, cu_q=cu, lens=lens)),
        "update": (fp8bs.fp8bs_cache_update, dict(cache=cache, table=table, lens=lens, parent=lens, new_lens=lens,
                                                  table_out=table.clone(), lens_out=lens.clone(), workspace=None)),
        "compact": (fp8bs.fp8bs_cache_compact, dict(cache=cache, table=table, lens=lens, table_out=table.clone(),
                                                    count=torch.zeros((), dtype=i32), workspace=None)),
    }
    for what, (f, args) in calls.items():
        for name, value in args.items():
            if isinstance(value, torch.Tensor):
                for bad in (None, 3, [1, 2], value.float().numpy()):
                    with pytest.raises(TypeError, match=name):
                        f(**{**args, name: bad})
        for bad in (None, cache.latent, (cache.latent, cache.rope), cache._replace(latent=None), cache._replace(rope=None)):
            with pytest.raises(TypeError, match="cache"):
                f(**{**args, "cache": bad})
    for f, args in ((fp8bs.mla_attention, (None, qr, cache, table, cu, lens, 0.1)),
                    (fp8bs.mla_attention, (q, qr, None, table, cu, lens, 0.1)),
                    (fp8bs.mla_attention, (q, qr, cache, None, cu, lens, 0.1)),
                    (fp8bs.mla_cache_write, (None, kv, w, 1e-6, cs, cache, table, cu, lens)),
                    (fp8bs.cache_update, (cache, None, lens, lens, lens)), (fp8bs.cache_update, (cache, table, lens, None, lens)),
                    (fp8bs.cache_update, (None, table, lens, lens, lens)), (fp8bs.cache_compact, (None, table, lens)),
                    (fp8bs.cache_compact, (cache, None, lens))):
        with pytest.raises(TypeError):
            f(*args)


def test_listing_check():
    """The build refuses an attention kernel whose compiler-made instructions
    touch AGPRs (the accumulators live there, named in inline assembly) or spill."""
    from block_scaled_fp8_03_amd import build
    asm = "\t;;#ASMSTART\n\tv_accvgpr_read_b32 v1, a[0x41]\n\t;;#ASMEND\n"
    build.check_listing("x", asm + "\tv_add_f32_e32 v1, v2, v3\n\ts_add_i32 s1, s2, s3\n")
    for line in ("\tv_accvgpr_write_b32 a3, v1", "\tv_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]",
                 "\tscratch_store_dword off, v1, s0", "\tds_read_b128 a[4:7], v1"):
        with pytest.raises(RuntimeError):
            build.check_listing("x", asm + line + "\n")
    mfma = "\t;;#ASMSTART\n\tv_mfma_f32_32x32x16_bf16 a[0x10:0x1f], v[8:11], v[12:15], a[0x10:0x1f]\n\t;;#ASMEND\n"
    build.check_listing("x", "\tv_mov_b32_e32 v9, v1\n\ts_nop 1\n" + mfma)
    build.check_listing("x", "\tv_mov_b32_e32 v9, v1\n\ts_nop 0\n\tds_read_b128 v[8:11], v1\n" + mfma)
    for line in ("\tv_mov_b32_e32 v9, v1\n", "\tv_cvt_pk_bf16_f32 v15, v1, v2\n\ts_nop 0\n"):
        with pytest.raises(RuntimeError):
            build.check_listing("x", line + mfma)
    assert "mla_attention.hip" in build.OWN_AGPR_SOURCES


def test_listing_check_across_branches():
    """What runs before an MFMA is not always what stands above it: the end of a
    loop comes before its start, a jump's source before its target, and nothing falls
    out of a jump that is always taken."""
    from block_scaled_fp8_03_amd import build
    mfma = "\t;;#ASMSTART\n\tv_mfma_f32_32x32x16_bf16 a[0x10:0x1f], v[8:11], v[12:15], a[0x10:0x1f]\n\t;;#ASMEND\n"
    write, other = "\tv_mov_b32_e32 v9, v1\n", "\tv_mov_b32_e32 v30, v1\n"
    loop = ".LBB0_1:\n" + mfma + "{}\ts_cbranch_scc1 .LBB0_1\n; %bb.2:\n\ts_endpgm\n"
    jump = "{}\ts_cbranch_execz .LBB0_3\n" + 3 * other + "\ts_branch .LBB0_4\n.LBB0_3:\n" + mfma + ".LBB0_4:\n\ts_endpgm\n"
    past = "\ts_cbranch_scc0 .LBB0_6\n; %bb.5:\n{}\ts_branch .LBB0_7\n.LBB0_6:\n" + mfma + ".LBB0_7:\n\ts_endpgm\n"
    chain = "{}\ts_branch .LBB0_9\n.LBB0_8:\n" + 2 * other + ".LBB0_9:\n" + mfma
    swap = "\tv_swap_b32 v30, v9\n"
    for text in (loop.format(write), loop.format(swap), jump.format(write), chain.format(write)):
        with pytest.raises(RuntimeError):
            build.check_listing("x", text)
    for text in (loop.format(write + "\ts_nop 1\n"), loop.format(write + 2 * other), loop.format(other),
                 jump.format(write + 2 * other), jump.format(other), past.format(write), chain.format(other)):
        build.check_listing("x", text)
    # each kernel stands for itself
    build.check_listing("x", "one:\n" + write + "\ts_endpgm\ntwo:\n" + mfma + "\ts_endpgm\n")


def test_the_listing_checked_is_that_of_the_object(tmp_path):
    """The object and its listing come from one compilation."""
    from block_scaled_fp8_03_amd import build
    src = tmp_path / "small.hip"
    src.write_text("#include <hip/hip_runtime.h>\n__global__ void k(int* p) { p[threadIdx.x] += 1; }\n")
    obj, text = build.compile_listed([build.HIPCC, "--offload-arch=gfx950", "-x", "hip"], str(src), str(tmp_path))
    assert os.path.exists(obj) and "s_endpgm" in text
    listing, = [f for f in os.listdir(tmp_path) if f.endswith("gfx950.s")]
    assert (tmp_path / listing).read_text() == text
