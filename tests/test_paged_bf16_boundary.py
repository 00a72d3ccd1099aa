"""The bf16 paged cache's attention and the step's plan without a GPU: every bad argument is refused on the
host before anything is enqueued, and the binding checks types, shapes and devices."""
import ctypes

import pytest
import torch

from test_paged_boundary import FAKE, ODD, s5  # noqa: F401


def attend(s5, sparse, geom=None, pages=(8, 64, 4), N=1, B=1, window=0, q=FAKE, qs=4096, kp=FAKE, vp=FAKE, table=FAKE,  # noqa: F811
           seq=FAKE, pos=FAKE, ids=FAKE, cnt=FAKE, gate=None, out=FAKE, ws=FAKE, nbytes=None):
    geom = geom or s5.STEP5_GEOMETRY
    pg = None if pages is None else ctypes.byref(s5.Pages(*pages))
    nbytes = s5.step5_paged_workspace_bytes(geom) if nbytes is None else nbytes
    g = ctypes.byref(geom)
    if sparse:
        return s5.load().step5_sparse_attn_paged(g, pg, N, B, q, qs, kp, vp, table, seq, pos, ids, cnt, gate, out, ws, nbytes, None)
    return s5.load().step5_paged_attn(g, pg, N, B, window, q, qs, kp, vp, table, seq, pos, gate, out, ws, nbytes, None)


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("bad, want", [
    (dict(pages=None), 1), (dict(pages=(8, 12, 4)), 1), (dict(pages=(-1, 64, 4)), 1),
    (dict(pages=(1 << 24, 64, 4)), 1), (dict(pages=(8, 64, 1 << 26)), 1), (dict(table=None), 1),
    (dict(N=0), 1), (dict(B=0), 1), (dict(N=65536), 2),
    (dict(q=None), 1), (dict(kp=None), 1), (dict(vp=None), 1), (dict(seq=None), 1), (dict(pos=None), 1), (dict(out=None), 1),
    (dict(q=ODD), 1), (dict(kp=ODD), 1), (dict(vp=ODD), 1), (dict(out=ODD), 1), (dict(ws=ODD), 1),
    (dict(qs=4088), 1), (dict(qs=4100), 1), (dict(qs=0), 1), (dict(qs=-4096), 1),
    (dict(ws=None), 3), (dict(nbytes=0), 3), (dict(nbytes=16), 3),
])
def test_attention_refusals(s5, sparse, bad, want):  # noqa: F811
    assert attend(s5, sparse, **bad) == want


def test_more_refusals(s5):  # noqa: F811
    assert attend(s5, False, window=-1) == 1
    assert attend(s5, True, ids=None) == 1 and attend(s5, True, cnt=None) == 1
    bad = s5.Geometry.step5(head_dim=64)
    assert attend(s5, False, geom=bad, nbytes=1 << 30) == 2 and attend(s5, True, geom=bad, nbytes=1 << 30) == 2
    assert s5.load().step5_paged_attn(None, None, 1, 1, 0, *[None] * 1, 0, *[None] * 8, 0, None) == 1


PLAN = ("lengths", "new", "table", "held", "free_pages", "free_count", "row_seq", "row_pos", "row_start", "ends", "granted",
        "region_begin", "region_end")


def plan(s5, geom=None, pages=(8, 64, 4), N=4, B=2, **over):  # noqa: F811
    pg = None if pages is None else ctypes.byref(s5.Pages(*pages))
    return s5.load().step5_paged_plan(ctypes.byref(geom or s5.STEP5_GEOMETRY), pg, N, B, *(over.get(n, FAKE) for n in PLAN), None)


@pytest.mark.parametrize("bad, want", [(dict(pages=None), 1), (dict(pages=(0, 64, 4)), 1), (dict(pages=(8, 60, 4)), 1),
                                       (dict(pages=(8, 64, 1 << 26)), 1), (dict(N=0), 1), (dict(B=0), 1),
                                       (dict(N=(1 << 24) + 1), 2), (dict(B=8193), 2)] + [({n: None}, 1) for n in PLAN])
def test_plan_refusals(s5, bad, want):  # noqa: F811
    assert plan(s5, **bad) == want


def test_plan_without_a_table_is_refused(s5):  # noqa: F811
    assert plan(s5, table=None, pages=(8, 64, 1)) == 1


def test_the_binding_checks_kinds_and_devices(s5):  # noqa: F811
    geom = s5.STEP5_GEOMETRY
    k = torch.zeros((2, 4, 64, 128), dtype=torch.bfloat16)
    cache = s5.PagedCache(k, k.clone())
    q, out = (torch.zeros((1, 32, 128), dtype=torch.bfloat16) for _ in range(2))
    row = torch.zeros(1, dtype=torch.int32)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        s5.step5_paged_attn(geom, q, cache, row, row, out, None)
    table = s5.PagedTable.create(4, 64, 2, 1, device="cpu")
    rows = s5.PagedRows.create(1, 4, device="cpu")
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        s5.step5_paged_plan(table, rows, row, row)
    assert table.free_pages.tolist() == [3, 2, 1, 0] and table.free_count.tolist() == [4]
    assert rows.row_start.shape == (2,) and rows.row_seq.shape == (4,)


def test_handles_check_what_is_assigned(s5):  # noqa: F811
    i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32)
    table = s5.PagedTable(i32(3, 4), i32(3), i32(20), i32(1), 16)
    assert table.B == 3 and table.page_tokens == 16
    for name, bad in (("held", i32(4)), ("held", torch.zeros(3)), ("free_count", i32(2)), ("block_table", i32(2, 4)),
                      ("block_table", i32(3, 8)[:, ::2]), ("free_pages", i32(2, 2)), ("held", None)):
        with pytest.raises(ValueError):
            setattr(table, name, bad)
    for name in ("B", "page_tokens", "device"):
        with pytest.raises(AttributeError):
            setattr(table, name, 1)
    longer = i32(40)
    table.free_pages = longer
    assert table.free_pages is longer and table._shape.num_pages == 40 and table._args[2] == longer.data_ptr()
    rows = s5.PagedRows.create(3, 10, device="cpu")
    with pytest.raises(ValueError):
        rows.ends = i32(4)
    with pytest.raises(ValueError):
        rows.row_pos = i32(11)
    lengths = i32(3)
    rows.ends = lengths
    assert rows.ends is lengths and rows.B == 3 and rows.N == 10


def test_a_step_whose_plan_does_not_fit_moves_nothing(s5, monkeypatch):  # noqa: F811
    """Other rows than q's, another table than the cache's, or other pages: refused before the plan runs."""
    ran = []
    monkeypatch.setattr(s5, "step5_paged_plan", lambda *a, **kw: ran.append(1))
    geom = s5.STEP5_GEOMETRY
    table = s5.PagedTable.create(6, 64, 2, 1, device="cpu")
    row = torch.zeros(1, dtype=torch.int32)

    def step(N, cache):
        t = {"q": torch.zeros((2, 32, 128), dtype=torch.bfloat16)}
        rows = s5.PagedRows.create(1, N, device="cpu")
        s5.decode_step_paged(geom, t, cache, *[None] * 8, max_regions_per_seq=16, plan=(table, rows, row, row))

    create = lambda pages, tokens, of: s5.PagedCache.create(geom, pages, tokens, of, e4m3=False, device="cpu")
    with pytest.raises(ValueError, match="rows"):
        step(3, create(6, 64, table.block_table))
    own = s5.PagedCache(*(torch.zeros((6, 4, 64, 128), dtype=torch.bfloat16) for _ in range(2)))
    for cache in (create(6, 64, table.block_table.clone()), create(7, 64, table.block_table), create(6, 32, table.block_table), own):
        with pytest.raises(ValueError, match="table"):
            step(2, cache)
    assert not ran


def test_a_plan_of_other_sequences_than_the_caches_moves_nothing(s5, monkeypatch):  # noqa: F811
    """A cache over the first rows of the plan's table has its address and its length, and fewer sequences: refused."""
    ran = []
    monkeypatch.setattr(s5, "step5_paged_plan", lambda *a, **kw: ran.append(1))
    geom = s5.STEP5_GEOMETRY
    table = s5.PagedTable.create(6, 64, 2, 3, device="cpu")
    rows = s5.PagedRows.create(3, 2, device="cpu")
    cache = s5.PagedCache.create(geom, 6, 64, table.block_table[:2], e4m3=False, device="cpu")
    t = {"q": torch.zeros((2, 32, 128), dtype=torch.bfloat16)}
    with pytest.raises(ValueError, match="table"):
        s5.decode_step_paged(geom, t, cache, *[None] * 8, max_regions_per_seq=16, plan=(table, rows, *[torch.zeros(3).int()] * 2))
    assert not ran


@pytest.mark.parametrize("planned", [False, True])
@pytest.mark.parametrize("name, shape", [("idx_q", (3, 16, 64)), ("w", (1, 16)), ("idx_k", (3, 4, 128, 64)), ("idx_z", (2, 4, 64, 64)),
                                         ("summaries", (1, 4, 16, 64)), ("summaries", (2, 4, 16)), ("idx_k", None), ("sum_end", (1,)), ("sum_begin", "bf16"), ("w", "bf16"),
                                         ("cos", (100, 16)), ("sin", (128, 8))])
def test_a_step_of_other_rows_or_sequences_than_its_indexers_is_refused(s5, monkeypatch, planned, name, shape):  # noqa: F811
    """The scoring takes its rows from idx_q, the summaries their sequences from idx_k: more of them than there are rows and
    regions to summarise would be read past their ends."""
    ran = []
    monkeypatch.setattr(s5, "step5_paged_plan", lambda *a, **kw: ran.append("plan"))
    monkeypatch.setattr(s5, "step5_kv_append", lambda *a, **kw: ran.append("append"))
    geom = s5.STEP5_GEOMETRY
    table = s5.PagedTable.create(6, 64, 2, 2, device="cpu")
    cache = s5.PagedCache.create(geom, 6, 64, table.block_table, e4m3=False, device="cpu")
    bf16 = lambda *of: torch.zeros(of, dtype=torch.bfloat16)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)
    t = {"q": bf16(2, 32, 128), "idx_q": bf16(2, 16, 64), "w": torch.zeros(2, 16), "idx_k": bf16(2, 4, 128, 64), "idx_z": bf16(2, 4, 128, 64),
         "summaries": torch.zeros((2, 4, 16, 64), dtype=torch.uint8), "cos": bf16(128, 16), "sin": bf16(128, 16),
         "row_seq": i32(2), "row_pos": i32(2), "sum_begin": i32(2), "sum_end": i32(2)}
    t[name] = None if shape is None else t[name].bfloat16() if shape == "bf16" else torch.zeros(shape, dtype=t[name].dtype)
    if planned and name.startswith("sum_"):
        return  # (the plan's own)
    plan = (table, s5.PagedRows.create(2, 2, device="cpu"), i32(2), i32(2)) if planned else None
    with pytest.raises(ValueError, match=name):
        s5.decode_step_paged(geom, t, cache, None, None, bf16(2, 4, 128), bf16(2, 4, 128), *[None] * 4, max_regions_per_seq=16, plan=plan)
    assert not ran


def test_calls_that_only_check(s5):  # noqa: F811
    """While a thread's checks alone are on, its calls of a paged step refuse what they refuse, and enqueue nothing (without a GPU
    a call that went on would fail); another thread's are not touched."""
    import threading

    if torch.cuda.is_available():
        pytest.skip("addresses that no GPU may see")

    from test_paged_boundary import append
    from test_paged_boundary import attend as attend_e4m3
    lib, g = s5.load(), ctypes.byref(s5.STEP5_GEOMETRY)
    summarize = lambda span=4, k=FAKE: lib.step5_region_summarize(g, 2, 64, 8, span, k, FAKE, None, None, FAKE, FAKE, FAKE, None, None)
    score = lambda N=2, q=FAKE: lib.step5_index_score_topk(g, N, 2, 64, 8, q, FAKE, FAKE, FAKE, None, None, FAKE, FAKE, FAKE, None, None, FAKE, 1 << 40, None)
    assert s5.step5_set_check_only(1) == 0
    try:
        assert [plan(s5), append(s5), append(s5, e4m3=False), attend(s5, False), attend(s5, True), attend_e4m3(s5, False),
                attend_e4m3(s5, True), summarize(), score()] == [0] * 9
        assert [plan(s5, N=0), append(s5, k=ODD), append(s5, e4m3=False, rot=24), attend(s5, False, qs=4100), attend(s5, True, ws=None),
                attend_e4m3(s5, False, out=None), attend_e4m3(s5, True, N=65536), summarize(k=ODD), summarize(-1), score(0), score(q=None)] \
            == [1, 1, 2, 1, 3, 1, 2, 1, 1, 1, 1]
        assert s5.step5_set_check_only(2) == 1 and s5.step5_set_check_only(1) == 1
        seen = []
        other = threading.Thread(target=lambda: seen.append(s5.step5_set_check_only(0)))
        other.start()
        other.join()
        assert seen == [0]
    finally:
        assert s5.step5_set_check_only(0) == 1
    assert plan(s5) == 4


def test_what_the_other_calls_of_a_planned_step_refuse_is_refused_before_it(s5, monkeypatch):  # noqa: F811
    """The plan runs behind the checks of every call: here the first of them finds its tensors on the CPU."""
    ran, geom = [], s5.STEP5_GEOMETRY
    monkeypatch.setattr(s5, "step5_paged_plan", lambda *a, **kw: ran.append(1))
    table = s5.PagedTable.create(6, 64, 2, 2, device="cpu")
    cache = s5.PagedCache.create(geom, 6, 64, table.block_table, e4m3=False, device="cpu")
    bf16 = lambda *of: torch.zeros(of, dtype=torch.bfloat16)
    t = {"q": bf16(2, 32, 128), "idx_q": bf16(2, 16, 64), "w": torch.zeros(2, 16), "idx_k": bf16(2, 4, 128, 64), "idx_z": bf16(2, 4, 128, 64),
         "summaries": torch.zeros((2, 4, 16, 64), dtype=torch.uint8), "cos": None, "sin": None}
    rows, of = s5.PagedRows.create(2, 2, device="cpu"), torch.zeros(2, dtype=torch.int32)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        s5.decode_step_paged(geom, t, cache, None, None, bf16(2, 4, 128), bf16(2, 4, 128), *[None] * 4, max_regions_per_seq=1, plan=(table, rows, of, of))
    assert not ran and s5.step5_set_check_only(0) == 0
