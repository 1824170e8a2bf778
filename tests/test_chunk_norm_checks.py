"""CPU checks of the refusals of fp8_attn_chunk, fp8_rms_norm_group_quant and
fp8_silu_mul_group_quant: the library's host checks (nothing is enqueued) and the binding's checks
of shapes, which run before any pointer is handed on."""
import ctypes

import pytest
import torch

import fp8_e4m3_quantization_amd as fq

EINVAL, ENULL, EALIGN = -1, -2, -3
FAKE = 0x100000  # an aligned, never-dereferenced address: the checks return first
NAN, INF = float("nan"), float("inf")
BF16 = torch.bfloat16


def _chunk(**over):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, tab=FAKE, lens=FAKE, cu=FAKE, out=FAKE, lse=None, n=3, tq=9, mb=8,
             ts=8, hq=8, hkv=2, d=128, bs=16, nb=64, ks=1.0, vs=1.0, scale=0.1, causal=1, qs=1024,
             os=1024, cs=16 * 256, ws=FAKE, wb=1 << 40)
    a.update(over)
    return fq.load().fp8_attn_chunk(*[a[x] for x in (
        "q", "kc", "vc", "tab", "lens", "cu", "out", "lse", "n", "tq", "mb", "ts", "hq", "hkv", "d", "bs",
        "nb", "ks", "vs", "scale", "causal", "qs", "os", "cs", "ws", "wb")], None)


def test_chunk_refusals():
    for over in [dict(n=-1), dict(n=(1 << 16) + 1), dict(tq=-1), dict(tq=1 << 28), dict(mb=-1),
                 dict(ts=7), dict(hq=0), dict(hq=7), dict(hkv=0), dict(d=80), dict(bs=0), dict(nb=0),
                 dict(mb=1 << 20, ts=1 << 20, bs=2048, cs=2048 * 256), dict(ks=0.0), dict(vs=-1.0),
                 dict(ks=NAN), dict(scale=0.0), dict(scale=NAN), dict(scale=INF), dict(qs=1000),
                 dict(os=8), dict(cs=16 * 255), dict(cs=1 << 32), dict(nb=1 << 62), dict(wb=16),
                 dict(qs=(1 << 30) + 8), dict(os=(1 << 30) + 8), dict(ts=(1 << 40) + 1)]:
        assert _chunk(**over) == EINVAL, over
    for name in ("q", "kc", "vc", "tab", "lens", "cu", "out", "ws"):
        assert _chunk(**{name: None}) == ENULL, name
    for over in [dict(q=FAKE + 8), dict(kc=FAKE + 8), dict(vc=FAKE + 4), dict(out=FAKE + 8),
                 dict(ws=FAKE + 128), dict(qs=1028), dict(os=1028), dict(cs=16 * 256 + 8),
                 dict(lens=FAKE + 2), dict(cu=FAKE + 1), dict(lse=FAKE + 2)]:
        assert _chunk(**over) == EALIGN, over
    assert _chunk(n=0, q=None) == 0
    assert _chunk(tq=0, q=None) == 0


def test_chunk_workspace_size():
    b = ctypes.c_uint64(7)
    lib = fq.load()
    assert lib.fp8_attn_chunk_workspace_size(2, 8, 8, 2, 128, None) == ENULL
    for bad in [(-1, 8, 8, 2, 128), (2, -1, 8, 2, 128), (2, 8, 7, 2, 128), (2, 8, 8, 2, 100),
                (2, 8, 8, 0, 128), ((1 << 16) + 1, 8, 8, 2, 128), (2, 1 << 28, 8, 2, 128)]:
        assert lib.fp8_attn_chunk_workspace_size(*bad, ctypes.byref(b)) == EINVAL, bad
        assert b.value == 0
    assert fq.fp8_attn_chunk_workspace_size(0, 8, 8, 2, 128) == 0
    assert fq.fp8_attn_chunk_workspace_size(1, 5, 40, 4, 128) > 0
    assert fq.fp8_attn_chunk_workspace_size(300, 300, 40, 4, 128) == 0  # so many are not cut
    assert fq.fp8_attn_chunk_workspace_size(1, 1 << 17, 40, 4, 128) == 0  # nor where queries suffice
    most = 64 << 20
    for seqs, tq, hq, hkv, d in [(1, 1, 1, 1, 64), (16, 64, 40, 4, 128), (3, 900, 32, 8, 256),
                                 (256, 5000, 64, 64, 256), (1, 1 << 20, 1, 1, 256)]:
        assert fq.fp8_attn_chunk_workspace_size(seqs, tq, hq, hkv, d) <= most


def _norm(**over):
    a = dict(x=FAKE, res=FAKE, w=FAKE, eps=1e-6, ro=FAKE, no=FAKE, q=FAKE, s=FAKE, m=4, k=256, xs=256,
             rs=256, ros=256, nos=256)
    a.update(over)
    return fq.load().fp8_rms_norm_group_quant(*[a[x] for x in (
        "x", "res", "w", "eps", "ro", "no", "q", "s", "m", "k", "xs", "rs", "ros", "nos")], None)


def test_norm_refusals():
    for over in [dict(m=-1), dict(k=0), dict(k=-128), dict(k=200), dict(m=1 << 31), dict(m=1 << 62),
                 dict(eps=-1e-6), dict(eps=2.0), dict(eps=NAN), dict(xs=248), dict(rs=0), dict(ros=128),
                 dict(nos=255), dict(xs=1 << 41), dict(res=None)]:
        assert _norm(**over) == EINVAL, over
    for over in [dict(x=None), dict(q=None), dict(s=None), dict(ro=None)]:
        assert _norm(**over) == ENULL, over
    for over in [dict(x=FAKE + 2), dict(res=FAKE + 8), dict(w=FAKE + 8), dict(ro=FAKE + 4),
                 dict(no=FAKE + 8), dict(q=FAKE + 8), dict(s=FAKE + 2), dict(xs=260), dict(rs=260),
                 dict(ros=260), dict(nos=260)]:
        assert _norm(**over) == EALIGN, over
    assert _norm(m=0, x=None, q=None) == 0


def _silu(**over):
    a = dict(g=FAKE, u=FAKE, o=FAKE, q=FAKE, s=FAKE, m=4, k=256, gs=512, us=512, os=256)
    a.update(over)
    return fq.load().fp8_silu_mul_group_quant(*[a[x] for x in ("g", "u", "o", "q", "s", "m", "k", "gs",
                                                               "us", "os")], None)


def test_silu_refusals():
    for over in [dict(m=-1), dict(k=0), dict(k=130), dict(m=1 << 31), dict(gs=248), dict(us=128),
                 dict(os=0), dict(us=1 << 41)]:
        assert _silu(**over) == EINVAL, over
    for over in [dict(g=None), dict(u=None), dict(q=None), dict(s=None)]:
        assert _silu(**over) == ENULL, over
    for over in [dict(g=FAKE + 2), dict(u=FAKE + 8), dict(o=FAKE + 8), dict(q=FAKE + 8), dict(s=FAKE + 1),
                 dict(gs=516), dict(us=516), dict(os=260)]:
        assert _silu(**over) == EALIGN, over
    assert _silu(m=0, g=None) == 0


# ------------------------------------------------------------------------- the binding


def test_binding_refuses_chunk_shapes():
    q, pool = torch.zeros((9, 1024), dtype=BF16), torch.zeros(8 * 16 * 256, dtype=torch.uint8)
    tab, lens = torch.zeros((3, 4), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    cu = torch.tensor([0, 2, 5, 9], dtype=torch.int32)

    def call(*a, **kw):
        return fq.fp8_attn_chunk(*a, 8, 2, 128, 16, 1.0, 1.0, **kw)

    for bad in [(q, pool, pool, tab[:2], lens, cu), (q, pool, pool, tab, lens[:2], cu),
                (q, pool, pool, tab, lens, cu[:3]), (q, pool, pool, tab[0], lens, cu)]:
        with pytest.raises(ValueError, match="block_tables must"):
            call(*bad)
    with pytest.raises(ValueError, match="pools"):
        call(q, pool, pool[:100], tab, lens, cu)
    with pytest.raises(ValueError, match="q must be"):
        call(q[:, :100], pool, pool, tab, lens, cu)
    with pytest.raises(ValueError, match="out has"):
        call(q, pool, pool, tab, lens, cu, out=q[:2])
    with pytest.raises(ValueError, match="lse must"):
        call(q, pool, pool, tab, lens, cu, out=q, lse=torch.zeros((8, 9)))
    with pytest.raises(ValueError, match="rows must be packed"):
        call(q, pool, pool, torch.zeros((3, 8), dtype=torch.int32)[:, ::2], lens, cu)
    with pytest.raises(ValueError, match="too wide"):  # (32 bits of it would pass for a width of 4)
        call(q, pool, pool, torch.empty((3, (1 << 32) + 4), dtype=torch.int32, device="meta"), lens, cu)
    with pytest.raises(ValueError, match="GPU memory"):
        call(q, pool, pool, tab, lens, cu)


def test_binding_refuses_norm_and_silu_shapes():
    x, w = torch.zeros((4, 256), dtype=BF16), torch.zeros(256, dtype=BF16)
    norm, silu = fq.fp8_rms_norm_group_quant, fq.fp8_silu_mul_group_quant
    with pytest.raises(ValueError, match="x must be"):
        norm(x[0], w)
    with pytest.raises(ValueError, match="weight must"):
        norm(x, w[:100])
    with pytest.raises(ValueError, match="residual must"):
        norm(x, w, residual=x[:3])
    with pytest.raises(ValueError, match="goes with"):
        norm(x, w, residual_out=x)
    with pytest.raises(ValueError, match="norm_out must"):
        norm(x, w, norm_out=x[:, :128])
    with pytest.raises(ValueError, match="packed"):
        norm(torch.zeros((4, 512), dtype=BF16)[:, ::2], w)
    with pytest.raises(ValueError, match="q must be"):
        norm(x, w, q=torch.zeros((4, 128), dtype=torch.uint8))
    with pytest.raises(ValueError, match="scales"):
        silu(x, x, scales=torch.zeros((4, 3)))
    with pytest.raises(ValueError, match="up must be"):
        silu(x, x[:, :128])
    with pytest.raises(ValueError, match="out must be"):
        silu(x, x, out=x[:2])
    wide = torch.empty((1, (1 << 32) + 128), dtype=BF16, device="meta")
    for call in (lambda: norm(wide, None), lambda: silu(wide, wide)):
        with pytest.raises(ValueError, match="too many"):
            call()
    for call in (lambda: norm(x, w), lambda: silu(x, x)):
        with pytest.raises(ValueError, match="GPU memory"):
            call()
