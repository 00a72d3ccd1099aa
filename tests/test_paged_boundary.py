"""The paged cache's calls without a GPU: every bad argument is refused on the host before
anything is enqueued, and the binding checks types, shapes and devices."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def s5():
    import block_sparse_attention_step5_gb300 as s5
    s5.build()
    s5.load()
    return s5


FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: the calls below end on the host
ODD = ctypes.c_void_p(0x10008)


def append(s5, e4m3=True, geom=None, pages=(8, 64, 4), N=1, B=1, rot=128, t_cap=64, q=FAKE, qs=4096, k=FAKE, ks=512,
           v=FAKE, vs=512, seq=FAKE, pos=FAKE, cos=FAKE, sin=FAKE, q_out=FAKE, kp=FAKE, vp=FAKE, ksc=FAKE, vsc=FAKE,
           table=FAKE):
    geom = geom or s5.STEP5_GEOMETRY
    fn = s5.load().step5_kv_append_e4m3 if e4m3 else s5.load().step5_kv_append
    pg = None if pages is None else ctypes.byref(s5.Pages(*pages))
    scales = (ksc, vsc) if e4m3 else ()
    return fn(ctypes.byref(geom), pg, N, B, rot, t_cap, q, qs, k, ks, v, vs, seq, pos, cos, sin, q_out, kp, vp,
              *scales, table, None)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("bad, want", [
    (dict(pages=None), 1), (dict(pages=(0, 64, 4)), 1), (dict(pages=(8, 60, 4)), 1), (dict(pages=(8, 64, 0)), 1),
    (dict(pages=(8, 0, 4)), 1),
    (dict(pages=(1 << 24, 64, 4)), 1),          # 2^24 * 4 * 64 pool rows
    (dict(pages=(8, 64, 1 << 26)), 1),          # 2^32 tokens a sequence
    (dict(table=None), 1),                      # no table: a sequence is one page
    (dict(table=None, pages=(8, 64, 1), B=9), 1),
    (dict(N=0), 1), (dict(N=-1), 1), (dict(N=(1 << 24) + 1), 2), (dict(B=0), 1), (dict(t_cap=0), 1),
    (dict(rot=24), 2), (dict(rot=144), 2), (dict(rot=-16), 2),
    (dict(k=None), 1), (dict(v=None), 1), (dict(seq=None), 1), (dict(pos=None), 1), (dict(kp=None), 1),
    (dict(vp=None), 1), (dict(q=None), 1), (dict(q_out=None), 1), (dict(cos=None), 1), (dict(sin=None), 1),
    (dict(k=ODD), 1), (dict(v=ODD), 1), (dict(q=ODD), 1), (dict(q_out=ODD), 1), (dict(kp=ODD), 1), (dict(vp=ODD), 1),
    (dict(cos=ODD), 1), (dict(sin=ODD), 1),
    (dict(ks=504), 1), (dict(vs=508), 1), (dict(ks=516), 1), (dict(qs=4095), 1), (dict(qs=4088), 1),
])
def test_append_refusals(s5, e4m3, bad, want):
    assert append(s5, e4m3, **bad) == want


def test_append_e4m3_needs_scales(s5):
    assert append(s5, True, ksc=None) == 1
    assert append(s5, True, vsc=None) == 1


def attend(s5, sparse, geom=None, pages=(8, 64, 4), N=1, B=1, window=0, q=FAKE, kp=FAKE, vp=FAKE, ksc=FAKE, vsc=FAKE,
           table=FAKE, seq=FAKE, pos=FAKE, ids=FAKE, cnt=FAKE, gate=None, out=FAKE, ws=FAKE, nbytes=None):
    geom = geom or s5.STEP5_GEOMETRY
    pg = None if pages is None else ctypes.byref(s5.Pages(*pages))
    nbytes = s5.step5_paged_workspace_bytes(geom) if nbytes is None else nbytes
    g = ctypes.byref(geom)
    if sparse:
        return s5.load().step5_sparse_attn_e4m3(g, pg, N, B, q, kp, vp, ksc, vsc, table, seq, pos, ids, cnt, gate, out,
                                                ws, nbytes, None)
    return s5.load().step5_paged_attn_e4m3(g, pg, N, B, window, q, kp, vp, ksc, vsc, table, seq, pos, gate, out, ws,
                                           nbytes, None)


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("bad, want", [
    (dict(pages=None), 1), (dict(pages=(8, 12, 4)), 1), (dict(pages=(-1, 64, 4)), 1),
    (dict(pages=(1 << 24, 64, 4)), 1), (dict(pages=(8, 64, 1 << 26)), 1), (dict(table=None), 1),
    (dict(N=0), 1), (dict(B=0), 1), (dict(N=65536), 2),
    (dict(q=None), 1), (dict(kp=None), 1), (dict(vp=None), 1), (dict(ksc=None), 1), (dict(vsc=None), 1),
    (dict(seq=None), 1), (dict(pos=None), 1), (dict(out=None), 1),
    (dict(q=ODD), 1), (dict(kp=ODD), 1), (dict(vp=ODD), 1), (dict(out=ODD), 1), (dict(ws=ODD), 1),
    (dict(ws=None), 3), (dict(nbytes=0), 3), (dict(nbytes=16), 3),
])
def test_attention_refusals(s5, sparse, bad, want):
    assert attend(s5, sparse, **bad) == want


def test_attention_refuses_bad_masks_and_geometry(s5):
    assert attend(s5, False, window=-1) == 1
    assert attend(s5, True, ids=None) == 1
    assert attend(s5, True, cnt=None) == 1
    for sparse in (False, True):
        assert attend(s5, sparse, geom=s5.Geometry.step5(num_q_heads=24), nbytes=1 << 30) == 2
        assert attend(s5, sparse, geom=s5.Geometry.step5(head_dim=64), nbytes=1 << 30) == 2


def test_workspace_bytes(s5):
    assert s5.step5_paged_workspace_bytes(s5.STEP5_GEOMETRY) > 0
    assert s5.step5_paged_workspace_bytes(s5.Geometry.step5(head_dim=64)) == 0


def test_paged_cache_checks(s5):
    u8, bf = (torch.zeros((2, 4, 16, 128), dtype=d) for d in (torch.uint8, torch.bfloat16))
    sc = torch.ones((2, 4, 2))
    tab = torch.zeros((1, 2), dtype=torch.int32)
    s5.PagedCache(bf, bf)
    assert s5.PagedCache(bf, bf).B == 2 and s5.PagedCache(u8, u8, tab, sc, sc).B == 1
    for args in ((u8, bf), (u8, u8), (u8, u8, tab, sc), (bf, bf, tab, sc, sc), (u8, u8, tab.long(), sc, sc),
                 (u8, u8, tab[0], sc, sc), (u8, u8, tab, sc[:1], sc), (u8, u8, tab, sc.double(), sc), (u8[0], u8[0]),
                 (u8.int(), u8.int(), tab, sc, sc)):
        with pytest.raises(ValueError):
            s5.PagedCache(*args)


def test_paged_cache_follows_its_tensors(s5):
    """An assigned tensor is checked and used from then on; a refused one changes nothing."""
    u8, sc = torch.zeros((4, 2, 16, 128), dtype=torch.uint8), torch.ones((4, 2, 2))
    tab = torch.zeros((1, 2), dtype=torch.int32)
    tensors = dict(k=u8, v=u8.clone(), block_table=tab, k_scales=sc, v_scales=sc.clone())
    cache = s5.PagedCache(**tensors)
    order = ("k", "v", "k_scales", "v_scales", "block_table")
    for name in order:
        tensors[name] = tensors[name].clone()
        setattr(cache, name, tensors[name])
        assert getattr(cache, name) is tensors[name]
        assert cache._pools == tuple(tensors[n].data_ptr() for n in order)
    cache.block_table = tensors["block_table"] = torch.zeros((3, 5), dtype=torch.int32)
    assert cache.B == 3 and cache.pages.table_len == 5
    before = dict(cache.__dict__)
    for name, bad in (("block_table", tab.long()), ("block_table", torch.zeros((2, 3), dtype=torch.int32).t()), ("k", u8[:2]), ("k", u8.bfloat16()),
                      ("k_scales", None), ("v_scales", sc.double()), ("v", u8.transpose(0, 1))):
        with pytest.raises(ValueError):
            setattr(cache, name, bad)
    for name in ("B", "pages", "e4m3", "groups", "head_dim", "device"):
        with pytest.raises(AttributeError):
            setattr(cache, name, 7)
    cache.pages.num_pages = 1 << 20
    assert cache.__dict__ == before and cache.pages.num_pages == 4


def test_binding_refuses_cpu_tensors(s5):
    """No tensor of a call may lie elsewhere than on the current GPU."""
    g = s5.STEP5_GEOMETRY
    u8 = torch.zeros((2, 4, 16, 128), dtype=torch.uint8)
    sc = torch.ones((2, 4, 2))
    tab = torch.zeros((1, 2), dtype=torch.int32)
    row = torch.zeros(1, dtype=torch.int32)
    kv = torch.zeros((1, 4, 128), dtype=torch.bfloat16)
    with pytest.raises((ValueError, RuntimeError)):
        s5.step5_kv_append_e4m3(g, kv, kv, s5.PagedCache(u8, u8, tab, sc, sc), row, row)
