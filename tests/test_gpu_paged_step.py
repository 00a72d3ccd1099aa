"""decode_step_paged with a plan on the GPU: what it refuses moves nothing, padded steps, either kind of pool, and a step
captured in a graph and replayed."""
import pytest
import torch

import paged_bf16_reference as B16
import paged_reference as R
from test_gpu_paged import dev, geometry, normal, s5, status  # noqa: F401

pytestmark = pytest.mark.gpu


class Step:
    """Three sequences in a table of six with a planned step of one or two tokens each: everything that decode_step_paged takes.
    The indexer's tensors have random values (finite, as the front end writes them)."""

    def __init__(self, s5, N=6, e4m3=False, lengths=(300, 0, 77, 0, 1001, 0), new=(1, 0, 2, 0, 1, 0), pt=64, seed=1, cap=2048):  # noqa: F811
        gen = torch.Generator().manual_seed(seed)
        self.s5, self.gen, self.N, self.pt, self.e4m3 = s5, gen, N, pt, e4m3
        self.geom = g = geometry(s5, top_k=32)
        B = self.B = len(lengths)
        self.table = s5.PagedTable.create(B * cap // pt, pt, cap // pt, B)
        self.rows = s5.PagedRows.create(B, N)
        self.cache = s5.PagedCache.create(g, B * cap // pt, pt, self.table.block_table, e4m3=e4m3)
        self.lengths, self.new = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (lengths, new))
        # the tokens that are there
        start = s5.PagedRows.create(B, sum(lengths))
        s5.step5_paged_plan(self.table, start, torch.zeros_like(self.lengths), self.lengths)
        k, v = (normal(gen, sum(lengths), 4, 128).cuda() for _ in "kv")
        (s5.step5_kv_append_e4m3 if e4m3 else s5.step5_kv_append)(g, k, v, self.cache, start.row_seq, start.row_pos)
        self.t = {"q": normal(gen, N, 32, 128, scale=1.5).cuda(), "idx_q": normal(gen, N, 16, 64).cuda(), "w": torch.rand(N, 16, generator=gen).cuda(),
                  "idx_k": normal(gen, B, 4, cap, 64).cuda(), "idx_z": normal(gen, B, 4, cap, 64).cuda(), "cos": None, "sin": None,
                  "summaries": torch.zeros((B, 4, cap // 8, 64), dtype=torch.uint8, device="cuda")}
        s5.step5_region_summarize(g, self.t["idx_k"], self.t["idx_z"], None, None, torch.zeros_like(self.lengths), self.lengths // 8,
                                  self.t["summaries"])
        half = normal(gen, cap, 64).cuda()
        i32 = lambda *shape: torch.full(shape, 55, dtype=torch.int32, device="cuda")
        self.args = {"k": normal(gen, N, 4, 128).cuda(), "v": normal(gen, N, 4, 128).cuda(), "sel_ids": i32(N, 4, 32), "sel_count": i32(N, 4),
                     "q_rot": torch.full_like(self.t["q"], 5.0), "out": torch.full_like(self.t["q"], 5.0),
                     "ws": s5.Workspace.create(g, N, cap // 8), "paged_ws": s5.PagedWorkspace.create(g), "cos": half, "sin": half,
                     "gate": normal(gen, N, 32).cuda(), "max_regions_per_seq": 1}
        assert status(s5) == 0

    def run(self, **over):
        t = {**self.t, **{k[2:]: over.pop(k) for k in list(over) if k.startswith("t_")}}
        a = {**self.args, **over}
        self.s5.decode_step_paged(self.geom, t, self.cache, plan=(self.table, self.rows, self.lengths, self.new), **a)

    def state(self):
        names = ("block_table", "held", "free_pages", "free_count")
        return [getattr(self.table, n).clone() for n in names] + [self.lengths.clone(), self.cache.k.clone()]


def test_what_a_planned_step_refuses_moves_nothing(s5):  # noqa: F811
    """Every argument of the calls behind the plan is checked before it runs: with lengths the plan's own ends, as a captured
    step has them, a step that moved pages and then failed would grow the sequences twice when it is called again."""
    c = Step(s5, N=4)
    c.rows.ends = c.lengths
    before = c.state()
    a, t = c.args, c.t
    off = lambda x: torch.zeros(x.numel() + 4, dtype=x.dtype, device="cuda")[4:].view(x.shape)  # (8 bytes past an alignment of 16)
    for bad in (dict(k=a["k"][:3]), dict(k=a["k"].float()), dict(v=a["v"].cpu()), dict(v=a["v"][:, :2]), dict(k=off(a["k"])), dict(q_rot=a["q_rot"][:2]),
                dict(q_rot=None), dict(cos=a["cos"][:, :20]), dict(cos=a["cos"], sin=None), dict(cos=a["cos"][:, :12].contiguous(), sin=a["sin"][:, :12].contiguous()),
                dict(sel_ids=a["sel_ids"][..., :16]), dict(sel_ids=a["sel_ids"].long()), dict(sel_count=a["sel_count"][:3]), dict(sel_ids=None),
                dict(out=a["out"][:3]), dict(out=off(a["out"])), dict(out=None), dict(gate=a["gate"].float()), dict(gate=a["gate"][:, :8]),
                dict(paged_ws=None), dict(paged_ws=torch.zeros(64, dtype=torch.uint8, device="cuda")), dict(ws=None), dict(max_regions_per_seq=-1),
                dict(t_idx_q=off(t["idx_q"])), dict(t_idx_k=off(t["idx_k"])), dict(t_summaries=t["summaries"][..., :32]),
                dict(t_summaries=t["summaries"].cpu()), dict(t_q=off(t["q"])), dict(t_cos=a["cos"][:, :16].contiguous())):
        with pytest.raises((ValueError, s5.Step5Error, AttributeError, TypeError)):
            c.run(**bad)
        assert all(torch.equal(x, y) for x, y in zip(before, c.state())), list(bad)
        assert status(s5) == 0 and bool((a["out"] == 5.0).all())
    c.run()  # (none of them left the checks on)
    assert status(s5) == 0
    assert c.lengths.tolist() == [301, 0, 79, 0, 1002, 0] and not bool((a["out"] == 5.0).all())


@pytest.mark.parametrize("path", [0, 1, 2, 3])
@pytest.mark.parametrize("noalloc", [False, True])
def test_scoring_of_padding(s5, path, noalloc):  # noqa: F811
    """Rows of sequence -1 have no picks and raise no flag, on every selection path; the other rows' picks are what they
    are without them, and a row out of range is still told."""
    g = geometry(s5, top_k=64)
    gen = torch.Generator().manual_seed(path)
    B, t_cap = 3, 4096
    summ = torch.randint(0, 120, (B, 4, t_cap // 8, 64), generator=gen).to(torch.uint8).cuda()
    N = 24
    seq = torch.tensor([0, -1, 1, -1, -1, 2, 2, -1] * 3, dtype=torch.int32)
    pos = torch.where(seq >= 0, torch.randint(0, t_cap, (N,), generator=gen), torch.tensor([-1, 7, 1 << 30] * 8)).int()
    q, w = normal(gen, N, 16, 64).cuda(), torch.rand(N, 16, generator=gen).cuda()

    def score(keep, seq=seq, pos=pos):
        n = int(keep.sum())
        out = [torch.full((n, 4, 64), 99, dtype=torch.int32, device="cuda"), torch.full((n, 4), 99, dtype=torch.int32, device="cuda"),
               torch.full((n, 4, 64), 99.0, device="cuda")]
        at = (g, q[keep].contiguous(), w[keep].contiguous(), *dev(seq[keep], pos[keep]), None, None, summ, *out[:2])
        prev = s5.step5_set_select_path(path)
        try:
            if noalloc:
                s5.step5_index_score_topk_noalloc(*at, t_cap=t_cap, sel_scores=out[2])
            else:
                s5.step5_index_score_topk(*at, s5.Workspace.create(g, n, t_cap // 8).tensor, t_cap=t_cap, sel_scores=out[2])
        finally:
            s5.step5_set_select_path(prev)
        return out
    real = seq >= 0
    got = score(torch.ones(N, dtype=torch.bool))
    assert status(s5) == 0
    pad = [x[~real] for x in got]
    assert bool((pad[0] == -1).all()) and bool((pad[1] == 0).all()) and bool((pad[2] == float("-inf")).all())
    alone = score(real)
    assert status(s5) == 0 and all(torch.equal(x[real], y) for x, y in zip(got, alone))
    none = score(~real)
    assert status(s5) == 0 and all(torch.equal(x, y) for x, y in zip(none, pad))
    for b, p in ((-2, 0), (B, 0), (0, t_cap), (0, -1)):
        seq2, pos2 = seq.clone(), pos.clone()
        seq2[5], pos2[5] = b, p
        got2 = score(torch.ones(N, dtype=torch.bool), seq2, pos2)
        assert status(s5) == s5.DEV_RANGE, (b, p)
        keep = real & (torch.arange(N) != 5)
        assert all(torch.equal(x[keep], y[keep]) for x, y in zip(got2, got))


def check_step(s5, c):  # noqa: F811
    """A step's outputs against the attention over what the cache holds, and its picks against the scoring of its rows alone."""
    real = c.rows.row_seq >= 0
    seq, pos = c.rows.row_seq[real], c.rows.row_pos[real]
    a = c.args
    for x, left in (("q_rot", 5.0), ("out", 5.0), ("sel_ids", -1), ("sel_count", 0)):
        assert bool((a[x][~real] == left).all()), x
    if not bool(real.any()):
        return
    half = a["cos"].cpu(), a["sin"].cpu()
    q_rot, ids, cnt, out, gate = (a[x][real].cpu() for x in ("q_rot", "sel_ids", "sel_count", "out", "gate"))
    assert torch.equal(q_rot.double(), R.rotate(c.t["q"][real].cpu().double(), *half, pos.cpu().long()))
    n = int(real.sum())
    ids2, cnt2 = torch.empty_like(a["sel_ids"][:n]), torch.empty_like(a["sel_count"][:n])
    s5.step5_index_score_topk(c.geom, c.t["idx_q"][real], c.t["w"][real], seq, pos, None, None, c.t["summaries"], ids2, cnt2,
                              s5.Workspace.create(c.geom, n, c.t["summaries"].shape[2]).tensor, t_cap=c.t["idx_k"].shape[2])
    assert torch.equal(ids2.cpu(), ids) and torch.equal(cnt2.cpu(), cnt)
    args = (c.table.block_table.cpu(), seq.cpu(), pos.cpu(), c.geom.softmax_scale)
    if c.e4m3:
        want = R.attend(q_rot, R.decode(c.cache.k), R.decode(c.cache.v), c.cache.k_scales.cpu(), c.cache.v_scales.cpu(), *args,
                        ids=ids, counts=cnt, gate=gate)
        assert R.off(out, *want) <= 1.0
    else:
        want = B16.attend(q_rot, c.cache.k.cpu(), c.cache.v.cpu(), *args, ids=ids, counts=cnt, gate=gate)
        assert B16.off(out, *want, False) <= 1.0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("pt", [16, 64])
def test_padded_steps(s5, e4m3, pt):  # noqa: F811
    """Steps of six rows of which sequences take one, two or none, with sequences that start, pause, are rolled back and find no
    pages: nothing is flagged, padding is left alone, and every output is right."""
    c = Step(s5, e4m3=e4m3, pt=pt, seed=pt)
    for new in ([1, 0, 2, 0, 1, 0], [0, 0, 0, 0, 0, 0], [0, 1, 2, 0, 3, 0], [1, 0, 0, 0, 0, 0], [1, 1, 1, 1, 1, 1]):
        c.new.copy_(torch.tensor(new))
        for x, left in (("q_rot", 5.0), ("out", 5.0), ("sel_ids", 55), ("sel_count", 55)):
            c.args[x].fill_(left)
        c.run()
        assert status(s5) == 0 and c.rows.granted.tolist() == new
        check_step(s5, c)
        c.lengths = c.rows.ends.clone()
    # no page left for the second, third and fourth sequence, whose next tokens need one
    c.table.free_count.zero_()
    held = c.table.held.tolist()
    c.lengths.copy_(torch.tensor([c.lengths[0].item(), held[1] * pt, held[2] * pt, held[3] * pt, 100, 1]))
    c.new.copy_(torch.tensor([1, 1, 1, 2, 1, 0]))
    c.table.held[4] = -(-101 // pt)
    for x, left in (("q_rot", 5.0), ("out", 5.0)):
        c.args[x].fill_(left)
    c.run()
    assert status(s5) == 0 and c.rows.granted.tolist() == [1, 0, 0, 0, 1, 0]
    check_step(s5, c)


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_captured_planned_step(s5, e4m3):  # noqa: F811
    """The whole step in a graph that goes on from the one before, replayed past the ends of pages and regions, against the
    same steps called one after another: the same bits."""
    steps = [Step(s5, e4m3=e4m3, pt=16, seed=3) for _ in range(2)]
    for c in steps:
        c.rows.ends = c.lengths
        c.run()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        steps[0].run()
    for i in range(20):
        for c in steps:
            c.t["q"].copy_(normal(torch.Generator().manual_seed(i), *c.t["q"].shape))
            c.new.copy_(torch.tensor([1, i % 2, 2, 0, 1, 0]))
        graph.replay()
        steps[1].run()
        for x in ("q_rot", "out", "sel_ids", "sel_count"):
            assert torch.equal(*(c.args[x] for c in steps)), (i, x)
        assert all(torch.equal(x, y) for x, y in zip(*(c.state() for c in steps)))
        assert torch.equal(*(c.t["summaries"] for c in steps))
    assert status(s5) == 0
    assert steps[0].lengths.tolist() == [321, 10, 119, 0, 1022, 0]
    check_step(s5, steps[0])


def test_front_end_of_padding(s5):  # noqa: F811
    """The front end of a planned step's rows: padding raises no flag and writes nothing but its normalised q; a row out of range
    is still told."""
    c = Step(s5)
    c.run()
    g, N, t = c.geom, c.N, c.t
    pre = [normal(c.gen, N, h, 64).cuda() for h in (16, 4, 4)]
    norm = [normal(c.gen, 64).cuda() for _ in range(3)]
    real = c.rows.row_seq >= 0

    def front(rows, seq, pos):
        q, k, z, summ = torch.full_like(pre[0][rows], 5.0), t["idx_k"].clone(), t["idx_z"].clone(), t["summaries"].clone()
        s5.step5_indexer_front(g, *(x[rows].contiguous() for x in pre), *norm, 1e-6, seq[rows].contiguous(), pos[rows].contiguous(), None, None,
                               q, k, z, summ)
        return q, k, z, summ
    every = torch.ones_like(real)
    got = front(every, c.rows.row_seq, c.rows.row_pos)
    assert status(s5) == 0 and bool(real.any()) and not bool(real.all())
    alone = front(real, c.rows.row_seq, c.rows.row_pos)
    assert status(s5) == 0 and torch.equal(got[0][real], alone[0]) and all(torch.equal(x, y) for x, y in zip(got[1:], alone[1:]))
    for b, p in ((-2, 0), (c.B, 0), (0, -1), (0, 2048)):
        seq, pos = c.rows.row_seq.clone(), c.rows.row_pos.clone()
        seq[-1], pos[-1] = b, p
        bad = front(every, seq, pos)
        assert status(s5) == s5.DEV_RANGE and all(torch.equal(x, y) for x, y in zip(got, bad)), (b, p)
