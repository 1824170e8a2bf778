"""CPU checks of the attention operators' refusals: the library's host checks (nothing is
enqueued) and the binding's checks of shapes, which run before any pointer is handed on."""
import ctypes

import pytest
import torch

import fp8_e4m3_quantization_amd as fq

EINVAL, ENULL, EALIGN = -1, -2, -3
FAKE = 0x100000  # an aligned, never-dereferenced address: the checks return first
NAN, INF = float("nan"), float("inf")


def _rope(write=False, **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, qw=FAKE, kw=FAKE, eps=1e-6, pos=FAKE, cs=FAKE, npos=64, rot=64,
             inter=0, kc=FAKE, vc=FAKE, slots=FAKE, t=4, hq=8, hkv=2, d=128, bs=16, nb=8, ks=1.0,
             vs=1.0, qs=1024, kst=256, vst=256, cst=16 * 256, qo=FAKE, ko=FAKE, qos=1024, kos=256)
    a.update(over)
    head = (a["qw"], a["kw"], a["eps"], a["pos"], a["cs"], a["npos"], a["rot"], a["inter"])
    if not write:
        return fq.load().qk_norm_rope(a["q"], a["k"], *head, a["t"], a["hq"], a["hkv"], a["d"],
                                      a["qs"], a["kst"], a["qo"], a["ko"], a["qos"], a["kos"], None)
    return fq.load().fp8_qk_norm_rope_kv_write(
        a["q"], a["k"], a["v"], *head, a["kc"], a["vc"], a["slots"], a["t"], a["hq"], a["hkv"],
        a["d"], a["bs"], a["nb"], a["ks"], a["vs"], a["qs"], a["kst"], a["vst"], a["cst"], a["qo"],
        a["ko"], a["qos"], a["kos"], None)


@pytest.mark.parametrize("write", [False, True])
def test_norm_rope_refusals(write):
    for over in [dict(t=-1), dict(hq=0), dict(hkv=-1), dict(d=0), dict(d=65537), dict(rot=-2),
                 dict(rot=63), dict(rot=130), dict(npos=0), dict(eps=-1e-6), dict(eps=NAN),
                 dict(eps=INF), dict(qs=1023), dict(kst=255), dict(qos=1000), dict(kos=0),
                 dict(qs=2 ** 31), dict(qos=2 ** 40)]:
        assert _rope(write, **over) == EINVAL, over
    for name in ("q", "k", "qo", "pos", "cs"):
        assert _rope(write, **{name: None}) == ENULL, name
    for over in [dict(q=FAKE + 1), dict(ko=FAKE + 1), dict(qw=FAKE + 1), dict(pos=FAKE + 4),
                 dict(cs=FAKE + 2)]:
        assert _rope(write, **over) == EALIGN, over
    assert _rope(write, t=0, q=None, k=None) == 0


def test_norm_rope_write_refusals():
    for over in [dict(bs=0), dict(nb=0), dict(ks=0.0), dict(vs=NAN), dict(ks=2.0 ** 65),
                 dict(vst=255), dict(vst=2 ** 31), dict(cst=16 * 256 - 1), dict(nb=1 << 62)]:
        assert _rope(True, **over) == EINVAL, over
    for name in ("v", "kc", "vc", "slots"):
        assert _rope(True, **{name: None}) == ENULL, name
    assert _rope(False, ko=None) == ENULL  # without a cache the keys need somewhere to go
    assert _rope(True, slots=FAKE + 4) == EALIGN


def _prefill(**over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, cq=FAKE, ck=FAKE, out=FAKE, lse=FAKE, n=2, tq=64, tk=64, hq=8,
             hkv=2, d=128, scale=0.1, causal=1, qs=1024, ks=256, vs=256, os=1024, ws=None, wb=0)
    a.update(over)
    return fq.load().attn_prefill(*[a[x] for x in ("q", "k", "v", "cq", "ck", "out", "lse", "n", "tq",
                                                   "tk", "hq", "hkv", "d", "scale", "causal", "qs",
                                                   "ks", "vs", "os", "ws", "wb")],
                                    None)


def test_prefill_refusals():
    for over in [dict(n=-1), dict(tq=-1), dict(tk=-1), dict(tq=(1 << 30) + 1), dict(hq=0),
                 dict(hkv=0), dict(hq=9), dict(d=96), dict(d=0), dict(scale=0.0), dict(scale=-1.0),
                 dict(scale=NAN), dict(scale=INF), dict(qs=1023), dict(ks=255), dict(vs=128),
                 dict(os=1016), dict(ks=(1 << 23) + 8)]:
        assert _prefill(**over) == EINVAL, over
    for name in ("q", "k", "v", "cq", "ck", "out"):
        assert _prefill(**{name: None}) == ENULL, name
    for over in [dict(q=FAKE + 8), dict(k=FAKE + 2), dict(v=FAKE + 8), dict(out=FAKE + 8),
                 dict(qs=1028), dict(ks=260), dict(vs=260), dict(os=1028), dict(cq=FAKE + 2),
                 dict(lse=FAKE + 1)]:
        assert _prefill(**over) == EALIGN, over
    assert _prefill(n=0, q=None) == 0
    assert _prefill(tq=0, q=None) == 0
    split = dict(n=1, tq=64, tk=100000)  # few queries over long keys: a workspace is needed
    need = fq.attn_prefill_workspace_size(1, 64, 100000, 8, 2, 128)
    assert need > 0 and fq.attn_prefill_workspace_size(1, 100000, 100000, 8, 2, 128) == 0
    assert _prefill(**split) == ENULL
    assert _prefill(**split, ws=FAKE, wb=need - 1) == EINVAL
    assert _prefill(**split, ws=FAKE + 16, wb=need) == EALIGN
    b = ctypes.c_uint64(7)
    lib = fq.load()
    assert lib.attn_prefill_workspace_size(1, 64, 64, 8, 2, 128, None) == ENULL
    for bad in [(-1, 64, 64, 8, 2, 128), (1, -1, 64, 8, 2, 128), (1, 64, 64, 8, 3, 128),
                (1, 64, 64, 8, 2, 96)]:
        assert lib.attn_prefill_workspace_size(*bad, ctypes.byref(b)) == EINVAL and b.value == 0


def _decode(**over):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, tab=FAKE, lens=FAKE, out=FAKE, lse=None, n=3, mb=8, ts=8, hq=8,
             hkv=2, d=128, bs=16, nb=64, ks=1.0, vs=1.0, scale=0.1, qs=1024, os=1024, cs=16 * 256,
             ws=FAKE, wb=1 << 40)
    a.update(over)
    return fq.load().fp8_attn_decode(*[a[x] for x in ("q", "kc", "vc", "tab", "lens", "out", "lse",
                                                      "n", "mb", "ts", "hq", "hkv", "d", "bs", "nb",
                                                      "ks", "vs", "scale", "qs", "os", "cs", "ws",
                                                      "wb")], None)


def test_decode_refusals():
    for over in [dict(n=-1), dict(mb=-1), dict(ts=7), dict(hq=0), dict(hq=7), dict(hkv=0),
                 dict(d=80), dict(bs=0), dict(nb=0), dict(mb=1 << 20, ts=1 << 20, bs=2048,
                                                          cs=2048 * 256),
                 dict(ks=0.0), dict(vs=-1.0), dict(scale=0.0), dict(scale=NAN), dict(qs=1000),
                 dict(os=8), dict(cs=16 * 255), dict(nb=1 << 62), dict(wb=16)]:
        assert _decode(**over) == EINVAL, over
    for name in ("q", "kc", "vc", "tab", "lens", "out", "ws"):
        assert _decode(**{name: None}) == ENULL, name
    for over in [dict(q=FAKE + 8), dict(kc=FAKE + 8), dict(vc=FAKE + 4), dict(out=FAKE + 8),
                 dict(ws=FAKE + 128), dict(qs=1028), dict(cs=16 * 256 + 8), dict(lens=FAKE + 2)]:
        assert _decode(**over) == EALIGN, over
    assert _decode(n=0, q=None) == 0


def test_decode_workspace_size():
    b = ctypes.c_uint64(7)
    lib = fq.load()
    assert lib.fp8_attn_decode_workspace_size(2, 8, 2, 128, None) == ENULL
    for bad in [(-1, 8, 2, 128), (2, 7, 2, 128), (2, 8, 2, 100), (2, 8, 0, 128)]:
        assert lib.fp8_attn_decode_workspace_size(*bad, ctypes.byref(b)) == EINVAL
        assert b.value == 0
    assert fq.fp8_attn_decode_workspace_size(0, 40, 4, 128) == 0
    assert fq.fp8_attn_decode_workspace_size(1, 40, 4, 128) > 0


# ------------------------------------------------------------------------- the binding


def _rows(t, e):
    return torch.zeros((t, e), dtype=torch.bfloat16)


def test_binding_refuses_rope_shapes():
    q, k = _rows(4, 8 * 128), _rows(4, 256)
    pos, cs = torch.zeros(4, dtype=torch.int64), torch.zeros((64, 128))
    with pytest.raises(ValueError, match="q must be"):
        fq.qk_norm_rope(q[:, :100], k, pos, cs, 8, 2, 128)
    with pytest.raises(ValueError, match="k has"):
        fq.qk_norm_rope(q, k[:3], pos, cs, 8, 2, 128)
    with pytest.raises(ValueError, match="positions has"):
        fq.qk_norm_rope(q, k, pos[:2], cs, 8, 2, 128)
    with pytest.raises(ValueError, match="both positions"):
        fq.qk_norm_rope(q, k, pos, None, 8, 2, 128)
    with pytest.raises(ValueError, match="q_weight"):
        fq.qk_norm_rope(q, k, pos, cs, 8, 2, 128, q_weight=torch.zeros(64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="packed"):
        fq.qk_norm_rope(_rows(4, 2048)[:, ::2], k, pos, cs, 8, 2, 128)
    pool = torch.zeros(8 * 16 * 256, dtype=torch.uint8)
    slots = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="slot_mapping has"):
        fq.fp8_qk_norm_rope_kv_write(q, k, k, pos, cs, pool, pool, slots[:3], 8, 2, 128, 16, 1.0, 1.0)
    with pytest.raises(ValueError, match="pools"):
        fq.fp8_qk_norm_rope_kv_write(q, k, k, pos, cs, pool, pool[:-1], slots, 8, 2, 128, 16, 1.0, 1.0)
    with pytest.raises(ValueError, match="GPU memory"):
        fq.qk_norm_rope(q, k, pos, cs, 8, 2, 128)


def test_binding_refuses_prefill_shapes():
    q, k = _rows(64, 1024), _rows(64, 256)
    cu = torch.tensor([0, 30, 64], dtype=torch.int32)
    with pytest.raises(ValueError, match="v has"):
        fq.attn_prefill(q, k, k[:60], cu, 8, 2, 128)
    with pytest.raises(ValueError, match="cu_seqlens"):
        fq.attn_prefill(q, k, k, cu, 8, 2, 128, cu_seqlens_k=cu[:2])
    with pytest.raises(ValueError, match="out has"):
        fq.attn_prefill(q, k, k, cu, 8, 2, 128, out=q[:10])
    with pytest.raises(ValueError, match="lse must"):
        fq.attn_prefill(q, k, k, cu, 8, 2, 128, out=q, lse=torch.zeros((8, 64)))
    with pytest.raises(ValueError, match="GPU memory"):
        fq.attn_prefill(q, k, k, cu, 8, 2, 128)


def test_binding_refuses_decode_shapes():
    q, pool = _rows(3, 1024), torch.zeros(8 * 16 * 256, dtype=torch.uint8)
    tab, lens = torch.zeros((3, 4), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)

    def call(*a, **kw):
        return fq.fp8_attn_decode(*a, 8, 2, 128, 16, 1.0, 1.0, **kw)

    with pytest.raises(ValueError, match="block_tables must"):
        call(q, pool, pool, tab[:2], lens)
    with pytest.raises(ValueError, match="block_tables must"):
        call(q, pool, pool, tab, lens[:2])
    with pytest.raises(ValueError, match="pools"):
        call(q, pool, pool[:100], tab, lens)
    with pytest.raises(ValueError, match="out has"):
        call(q, pool, pool, tab, lens, out=q[:2])
    with pytest.raises(ValueError, match="rows must be packed"):
        call(q, pool, pool, torch.zeros((3, 8), dtype=torch.int32)[:, ::2], lens)
    with pytest.raises(ValueError, match="GPU memory"):
        call(q, pool, pool, tab, lens)
