"""Attention over the bf16 pages on the GPU against its definition in 64 bits: rows on their own and rows
that share tiles, windows, picks, what lies outside the keys, and a run of plan, append and attention."""
import numpy as np
import pytest
import torch

import paged_bf16_reference as B16
import paged_reference as R
import synthetic as S
from test_gpu_paged import ROWS, SHAPES, dev, geometry, normal, rows_of, s5, status, tables  # noqa: F401

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


class Case:
    """bf16 pools, their table and rows at (row_seq, row_pos), and the 64-bit answer."""

    def __init__(self, s5, runs, G=4, hq=8, pt=64, seed=1, q_scale=1.5, extra=0, apart=False, B=None, **geom):  # noqa: F811
        self.s5, self.gen = s5, torch.Generator().manual_seed(seed)
        self.geom = geometry(s5, G, hq, **geom)
        self.G, self.hq, self.pt = G, hq, pt
        self.seq, self.pos = rows_of(*runs)
        self.N, self.B = len(self.seq), B or int(self.seq.max()) + 1
        length = -(-(int(self.pos.max()) + 1 + extra) // pt)
        self.table = tables(self.gen, self.B, length)
        P = self.B * length + 3
        self.k, self.v = (normal(self.gen, P, G, pt, 128) for _ in "kv")
        qkv = normal(self.gen, self.N, G * (hq + 2), 128, scale=q_scale)
        self.q = qkv[:, :G * hq] if apart else qkv[:, :G * hq].contiguous()
        self.ws = s5.PagedWorkspace.create(self.geom)
        self.ids = self.cnt = self.gate = None

    def gated(self):
        self.gate = normal(self.gen, self.N, self.G * self.hq, scale=2.0)
        return self

    def pick(self, at_most=None):
        top_k = self.geom.top_k
        self.ids = torch.full((self.N, self.G, top_k), -1, dtype=torch.int32)
        self.cnt = torch.zeros((self.N, self.G), dtype=torch.int32)
        for n in range(self.N):
            own = max(int(self.pos[n]), 0) // 8
            for g in range(self.G):
                c = min(top_k, own, at_most(n, g) if at_most else own)
                self.ids[n, g, :c] = torch.randperm(max(own, 1), generator=self.gen)[:c].int()
                self.cnt[n, g] = c
        return self

    def cache(self):
        return self.s5.PagedCache(*dev(self.k, self.v, self.table))

    def q_on_gpu(self):
        """As the rows lie on the host: dense, or a slice of the projection's rows."""
        base = self.q._base if self.q._base is not None else self.q
        return base.cuda()[:, :self.G * self.hq]

    def run(self, window=0, cache=None, out=None, ws=None, stream=None):
        if out is None:
            out = torch.full((self.N, self.G * self.hq, 128), 5.0, dtype=torch.bfloat16, device="cuda")
        seq, pos, ids, cnt, gate = dev(self.seq, self.pos, self.ids, self.cnt, self.gate)
        cache, ws, q = cache or self.cache(), ws or self.ws, self.q_on_gpu()
        if ids is None:
            self.s5.step5_paged_attn(self.geom, q, cache, seq, pos, out, ws, window=window, gate=gate, stream=stream)
        else:
            self.s5.step5_sparse_attn_paged(self.geom, q, cache, seq, pos, ids, cnt, out, ws, gate=gate, stream=stream)
        return out

    @property
    def shared(self):
        return self.ids is None and B16.shares(self.N, self.hq, self.B)

    def want(self, window=0, **kw):
        return B16.attend(self.q, self.k, self.v, self.table, self.seq, self.pos, self.geom.softmax_scale, window, self.ids,
                          self.cnt, self.gate, **kw)

    def check(self, window=0):
        got = self.run(window).cpu()
        assert status(self.s5) == 0
        self.near(got, *self.want(window))

    def near(self, got, out, mass):
        real = self.seq >= 0
        assert bool((got[~real] == 5.0).all())
        assert B16.off(got[real], out[real], mass[real], self.shared) <= 1.0

    def unseen(self, window=0):
        """Pool tokens [P][pt] that no row sees (in any group: windows only)."""
        mask = torch.ones((self.k.shape[0], self.pt), dtype=torch.bool)
        for b, p in zip(self.seq.tolist(), self.pos.tolist()):
            if b >= 0:
                for t in B16.keys_of(p, window, None, 0):
                    page, slot = R.place(self.table, b, int(t), self.pt)
                    mask[page, slot] = False
        return mask


LONGER = {
    "drafts": [(b, 100 + 37 * b, 4) for b in range(5)],
    "two_chunks": [(1, 333, 70), (0, 0, 75)],
    "one_chunk": [(0, 517, 130)],
    "prompt": [(0, 0, 300)],
    "with_padding": [(0, 40, 33), (-1, 0, 7), (1, 250, 60), (-1, 0, 40)],
    "scattered": [(0, 700, 1), (1, 5, 20), (0, 20, 1), (1, 600, 40), (0, 333, 3), (1, 100, 2)],
}


@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("G, hq, pt", SHAPES)
def test_rows(s5, rows, G, hq, pt):  # noqa: F811
    Case(s5, ROWS[rows], G, hq, pt, seed=len(rows) + pt).check()


@pytest.mark.parametrize("rows", list(LONGER))
@pytest.mark.parametrize("G, hq, pt, window", [(4, 8, 64, 0), (1, 16, 128, 0), (2, 4, 24, 0), (2, 8, 8, 100),
                                               (2, 16, 200, 33), (1, 4, 256, 128)])
def test_longer_rows(s5, rows, G, hq, pt, window):  # noqa: F811
    Case(s5, LONGER[rows], G, hq, pt, seed=len(rows) + pt, apart=True).gated().check(window)


@pytest.mark.parametrize("rows", ["odd", "ragged", "chunk_on", "draft"])
@pytest.mark.parametrize("window", [1, 2, 8, 127, 128, 129, 1000, 2 ** 31 - 1, 2 ** 40])
def test_windows(s5, rows, window):  # noqa: F811
    Case(s5, ROWS[rows], pt=16, seed=window % 97).check(window)


@pytest.mark.parametrize("tokens", [1, 2, 127, 128, 129, 1023, 4096, 6001])
@pytest.mark.parametrize("rows", [1, 3, 40])
def test_lengths(s5, tokens, rows):  # noqa: F811
    Case(s5, [(0, max(0, tokens - rows), rows)], G=2, seed=tokens).check()


DRAFTS = {
    "two": [(b, 90 + 61 * b, 2) for b in range(6)], "three": [(b, 300 + 7 * b, 3) for b in range(5)],
    "four": [(b, 1000 - 37 * b, 4) for b in range(4)], "seven": [(0, 2040, 7), (1, 3, 7)],
    "mixed": [(0, 500, 1), (1, 33, 4), (-1, 0, 2), (2, 900, 2), (3, 0, 3), (-1, 0, 1), (4, 127, 3)],
    "woven": [(0, 500, 1), (1, 433, 1), (0, 501, 1), (1, 434, 1), (2, 60, 1), (0, 20, 1), (2, 61, 1), (2, 700, 2)],
}


@pytest.mark.parametrize("rows", list(DRAFTS))
@pytest.mark.parametrize("G, hq, pt, window", [(4, 8, 64, 0), (2, 16, 24, 0), (3, 4, 16, 0), (2, 8, 8, 45), (1, 16, 128, 130), (4, 4, 40, 9)])
def test_drafts(s5, rows, G, hq, pt, window):  # noqa: F811
    """A few rows of each sequence, which read its keys together where the table holds enough of them."""
    Case(s5, DRAFTS[rows], G, hq, pt, seed=len(rows) + window, apart=True, extra=24000 // (G * len(DRAFTS[rows]))).gated().check(window)


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("window", [0, 70])
def test_values_of_a_later_draft_stay_with_it(s5, window, bad):  # noqa: F811
    """Four drafts of each of three sequences: a value that is not finite, at one draft's token, reaches that draft
    and those behind it, and no row before it or of another sequence."""
    c = Case(s5, [(0, 300, 4), (1, 77, 4), (2, 1500, 4)], G=4, pt=16, seed=4, extra=20000)
    clean = c.want(window)
    page, slot = R.place(c.table, 1, 78, c.pt)
    c.v[page, 2, slot, 100], c.k[R.place(c.table, 0, 302, c.pt)[0], 1, 302 % 16, 9] = bad, NAN
    got = c.run(window).cpu().float()
    assert status(s5) == 0
    hit = got[5:8, 16:24, 100]
    assert bool(torch.isnan(hit).all() if bad != bad else (hit == bad).all())
    got[5:8, 16:24, 100] = clean[0][5:8, 16:24, 100].float()
    assert bool(torch.isnan(got[2:4, 8:16]).all())
    got[2:4, 8:16] = clean[0][2:4, 8:16].float()
    c.near(got.bfloat16(), *clean)


@pytest.mark.parametrize("bad", [NAN, INF])
def test_drafts_of_windows_that_lie_apart(s5, bad):  # noqa: F811
    """What lies between the windows of rows of one item is not touched, whatever its pages and table entries hold."""
    c = Case(s5, [(0, 5000, 2), (0, 40, 2), (1, 900, 3), (1, 8, 1)], G=4, pt=16, seed=8, extra=9000)
    want = c.want(30)
    mask = c.unseen(30)[:, None, :, None]
    c.k.masked_fill_(mask, bad)
    c.v.masked_fill_(mask, bad)
    c.table[0, 4:300], c.table[1, 3:50] = -1, 10 ** 7
    got = c.run(30).cpu()
    assert status(s5) == 0
    c.near(got, *want)


@pytest.mark.parametrize("G, hq, pt", [(8, 4, 16), (8, 8, 64), (8, 16, 40)])
def test_drafts_in_long_windows(s5, G, hq, pt):  # noqa: F811
    """Windows long enough for rows to read their keys together, their first tokens inside tiles."""
    Case(s5, [(b, 3000 + 137 * b, 4) for b in range(3)] + [(3, 500, 2), (-1, 0, 1), (4, 2222, 3)], G, hq, pt, seed=hq).check(1100)


@pytest.mark.parametrize("bad", [NAN, INF])
def test_long_windows_of_one_item_that_lie_apart(s5, bad):  # noqa: F811
    """As above, and with a gap between the windows of an item's rows: what lies there is not touched."""
    c = Case(s5, [(0, 9000, 2), (0, 1300, 2), (1, 7000, 3), (1, 40, 1), (2, 5000, 8)], G=8, hq=8, pt=16, seed=8)
    want = c.want(1100)
    mask = c.unseen(1100)[:, None, :, None]
    c.k.masked_fill_(mask, bad)
    c.v.masked_fill_(mask, bad)
    c.table[0, 100:480], c.table[1, 10:350] = -1, 10 ** 7
    got = c.run(1100).cpu()
    assert status(s5) == 0
    c.near(got, *want)


def test_drafts_on_bad_pages_and_out_of_range(s5):  # noqa: F811
    c = Case(s5, [(0, 500, 4), (1, 90, 4), (2, 33, 4)], G=4, pt=32, seed=6, extra=20000)
    c.table[0, 3], c.table[2, 0], c.table[2, 1] = -1, 10 ** 6, -9
    c.seq[5], c.pos[6], c.seq[7] = 77, c.table.shape[1] * 32, -1
    got = c.run().cpu()
    assert status(s5) == 1
    assert bool((got[5:7] == 0).all()) and bool((got[7] == 5.0).all()) and bool((got[8:12] == 0).all())
    c.seq[5:7] = -1
    want = c.want(bad_pages=(-1, 10 ** 6, -9))
    ok = [0, 1, 2, 3, 4, 8, 9, 10, 11]
    assert B16.off(got[ok], want[0][ok], want[1][ok], c.shared) <= 1.0


def test_scores_of_minus_infinity(s5):  # noqa: F811
    """Keys whose scores overflow to -infinity weigh nothing, wherever they stand; a row with no others gets zeros."""
    for runs in ([(0, 600, 1)], [(0, 600, 4), (1, 5000, 1)], [(0, 600, 40)]):
        c = Case(s5, runs, G=1, hq=16, pt=64, seed=2)
        c.q = c.q.contiguous()
        c.q[0, :, 0], c.q[0, 3, 1] = 3.0e38, 0
        lows = torch.rand(601, generator=c.gen) < 0.5
        lows[:200] = True
        for t in range(601):
            page, slot = R.place(c.table, 0, t, c.pt)
            c.k[page, :, slot, 0] = -3.0e38 if lows[t] else 0.0
        got = c.run().cpu()[:1]
        assert status(s5) == 0
        out, mass = torch.zeros((1, 16, 128), dtype=torch.float64), torch.zeros((1, 16, 128), dtype=torch.float64)
        tok = torch.nonzero(~lows)[:, 0]
        page, slot = (torch.tensor(x) for x in zip(*[R.place(c.table, 0, int(t), c.pt) for t in tok]))
        w = torch.softmax(c.q[0].double() @ c.k[page, 0, slot].double().T * c.geom.softmax_scale, -1)
        out[0], mass[0] = w @ c.v[page, 0, slot].double(), w @ c.v[page, 0, slot].double().abs()
        assert B16.off(got, out, mass, c.shared) <= 1.0
        for t in range(601):
            page, slot = R.place(c.table, 0, t, c.pt)
            c.k[page, :, slot, 0] = -3.0e38
        assert bool((c.run().cpu()[0] == 0).all()) and status(s5) == 0


@pytest.mark.parametrize("runs", [[(b, 97 * b, 1) for b in range(40)], [(0, 900, 1), (1, 9000, 1), (2, 17, 1)],
                                  [(0, 30, 200), (1, 4000, 200)]])
def test_ragged_batches(s5, runs):  # noqa: F811
    Case(s5, runs, G=2, hq=8, seed=9).check()


@pytest.mark.parametrize("G, hq, pt", SHAPES)
@pytest.mark.parametrize("top_k", [1, 40, 512])
def test_picks(s5, top_k, G, hq, pt):  # noqa: F811
    runs = [(0, 1500, 2), (1, 7, 1), (1, 8, 1), (-1, 0, 1), (2, 5000, 1), (0, 333, 3)]
    Case(s5, runs, G, hq, pt, seed=top_k, apart=True, top_k=top_k).gated().pick(lambda n, g: 7 * n + 300 * g + 1).check()


def test_picks_of_many_rows(s5):  # noqa: F811
    Case(s5, [(0, 900, 100), (1, 3000, 90)], G=4, hq=8, seed=3, top_k=60).pick().check()


def test_peaked_scores(s5):  # noqa: F811
    """Large scores: the running maximum moves by more than the slack, tile after tile."""
    for runs in ([(0, 2000, 1), (1, 777, 1)], [(0, 1500, 40)]):
        c = Case(s5, runs, G=2, seed=5)
        c.q = c.q.contiguous()
        # each row's scores climb along its sequence, up to 16 in log2 units
        for b in range(c.B):
            u = torch.randn(128, generator=c.gen)
            u = u / u.norm()
            for t in range(int(c.pos.max()) + 1):
                at = R.place(c.table, b, t, c.pt)
                c.k[at[0], :, at[1]] = (u * (t / 150.0)).bfloat16()
            c.q[c.seq == b] = (u * 10.0).bfloat16()
        c.check()


# ------------------------------------------------------------------------------ what lies outside the keys

@pytest.mark.parametrize("bad", [NAN, INF, -INF, torch.finfo(torch.bfloat16).min])
@pytest.mark.parametrize("runs, window", [([(0, 101, 1), (1, 300, 1)], 0), ([(0, 300, 1)], 50), ([(0, 131, 40)], 0),
                                          ([(0, 700, 50), (1, 10, 20)], 90), ([(0, 5, 1), (0, 900, 1), (0, 450, 40)], 30)])
def test_tokens_outside_never_reach_the_result(s5, runs, window, bad):  # noqa: F811
    c = Case(s5, runs, G=2, pt=24, seed=8, extra=200)
    want = c.want(window)
    mask = c.unseen(window)[:, None, :, None]
    c.k.masked_fill_(mask, bad)
    c.v.masked_fill_(mask, bad)
    got = c.run(window).cpu()
    assert status(s5) == 0
    c.near(got, *want)


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("first, rows, window", [(100, 40, 0), (300, 64, 70), (0, 33, 0), (511, 2, 0)])
def test_values_of_a_later_row_stay_with_it(s5, first, rows, window, bad):  # noqa: F811
    """A token that some rows of a chunk see and others do not: its infinite value reaches the rows that see it, in its
    dimension, and none of the others."""
    c = Case(s5, [(0, first, rows)], G=2, pt=16, seed=4)
    clean = c.want(window)
    tok = first + rows // 2
    page, slot = R.place(c.table, 0, tok, c.pt)
    c.v[page, 1, slot, 77] = bad
    got = c.run(window).cpu().float()
    assert status(s5) == 0
    sees = (c.pos >= tok) & ((c.pos - tok < window) if window else True)
    hit = got[:, c.hq:, 77]
    assert bool(torch.isnan(hit[sees]).all() if bad != bad else (hit[sees] == bad).all())
    got[:, c.hq:, 77] = clean[0][:, c.hq:, 77].float()
    c.near(got.bfloat16(), *clean)


def test_both_infinities_of_later_rows(s5):  # noqa: F811
    """Values of both signs in one dimension: the rows that see both get NaN."""
    c = Case(s5, [(0, 200, 40)], G=1, pt=16, seed=4)
    for tok, x in ((210, INF), (220, -INF)):
        page, slot = R.place(c.table, 0, tok, c.pt)
        c.v[page, 0, slot, 3] = x
    got = c.run().cpu().float()[:, :, 3]
    pos = c.pos
    assert bool(torch.isfinite(got[pos < 210]).all())
    assert bool((got[(pos >= 210) & (pos < 220)] == INF).all()) and bool(torch.isnan(got[pos >= 220]).all())


def test_nan_key_of_a_later_row_stays_with_it(s5):  # noqa: F811
    for rows in (3, 40):
        c = Case(s5, [(0, 200, rows)], G=1, pt=16, seed=4)
        clean = c.want()
        page, slot = R.place(c.table, 0, 202, c.pt)
        c.k[page, 0, slot, 5] = NAN
        got = c.run().cpu()
        assert bool(torch.isnan(got[2:]).all())
        assert B16.off(got[:2], clean[0][:2], clean[1][:2], c.shared) <= 1.0


@pytest.mark.parametrize("runs", [[(0, 500, 1), (1, 90, 1)], [(0, 400, 60), (1, 20, 60)]])
def test_bad_pages_and_rows(s5, runs):  # noqa: F811
    c = Case(s5, runs, G=2, hq=8, pt=32, seed=6)
    c.table[0, 3], c.table[1, 0] = -1, 10 ** 6
    got = c.run().cpu()
    assert status(s5) == 1
    c.near(got, *c.want(bad_pages=(-1, 10 ** 6)))
    # a row whose every key is on a bad page, rows out of range, padding
    c = Case(s5, [(0, 40, 1), (1, 9, 1), (2, 3, 1), (1, 5, 1), (0, 7, 1), (1, 2, 40)] if len(runs[0]) and runs[0][2] > 1 else
             [(0, 40, 1), (1, 9, 1), (2, 3, 1), (1, 5, 1), (0, 7, 1)], G=2, hq=8, pt=32, seed=6)
    c.table[2, 0] = -7
    c.seq[1], c.pos[3], c.seq[4] = 99, 64, -1
    c.pos[3] = c.table.shape[1] * 32
    got = c.run().cpu()
    assert status(s5) == 1
    assert bool((got[1:4] == 0).all()) and bool((got[4] == 5.0).all())
    ok = torch.ones(c.N, dtype=torch.bool)
    ok[1:5] = False
    c.seq[1:4] = -1
    want = c.want()
    assert B16.off(got[ok], want[0][ok], want[1][ok], c.shared) <= 1.0


def test_bad_picks(s5):  # noqa: F811
    c = Case(s5, [(0, 700, 1), (0, 90, 1)], G=2, seed=2, top_k=16).pick()
    want = c.want()
    ids, cnt = c.ids, c.cnt
    good = c.run().cpu()
    assert status(s5) == 0
    c.near(good, *want)
    # an id at or past the row's own region, a negative one, and a count past top_k
    c.ids, c.cnt = ids.clone(), cnt.clone()
    c.ids[0, 0, 3], c.ids[0, 0, 4], c.cnt[1, 1] = 700 // 8, -1, 99
    got = c.run().cpu()
    assert status(s5) == 1
    assert torch.equal(got[0, c.hq:], good[0, c.hq:])
    keep = [i for i in range(16) if i not in (3, 4)]
    c.ids[0, 0, :14], c.cnt[0, 0] = ids[0, 0, keep], 14
    c.ids[1], c.cnt[1] = ids[1], cnt[1]
    want = c.want()
    assert B16.off(got[0, :c.hq], want[0][0, :c.hq], want[1][0, :c.hq], False) <= 1.0


# ------------------------------------------------------------------------------ buffers, streams, graphs

@pytest.mark.parametrize("runs", [[(0, 300, 1), (1, 40, 1)], [(0, 150, 48)]])
def test_buffers_of_the_smallest_alignment(s5, runs):  # noqa: F811
    """Every buffer 16 bytes past a larger alignment."""
    c = Case(s5, runs, G=2, seed=3)
    def odd(t):
        flat = torch.zeros(t.numel() * t.element_size() + 272, dtype=torch.uint8, device="cuda")
        at = -flat.data_ptr() % 256 + 16
        return flat[at:at + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
    k, v, q, out = (odd(t) for t in (c.k, c.v, c.q, c.q))
    for d, s in ((k, c.k), (v, c.v), (q, c.q)):
        d.copy_(s)
    ws = odd(torch.empty(s5.step5_paged_workspace_bytes(c.geom), dtype=torch.uint8))
    s5.step5_paged_attn(c.geom, q, s5.PagedCache(k, v, c.table.cuda()), *dev(c.seq, c.pos), out, ws)
    assert status(s5) == 0
    c.near(out.cpu(), *c.want())


@pytest.mark.parametrize("runs, picks", [([(0, 3000, 1), (1, 500, 1)], False), ([(0, 600, 100), (1, 9, 100)], False),
                                         ([(0, 3000, 1), (1, 500, 1)], True)])
def test_the_same_bits_again_and_in_graphs(s5, runs, picks):  # noqa: F811
    """Repeated, captured and replayed, with the workspace overwritten in between and two graphs on one workspace."""
    c = Case(s5, runs, G=4, seed=7, top_k=64)
    c = c.pick() if picks else c
    first = c.run()
    cache, (seq, pos, ids, cnt), q = c.cache(), dev(c.seq, c.pos, c.ids, c.cnt), c.q.cuda()

    def call(out):
        if picks:
            s5.step5_sparse_attn_paged(c.geom, q, cache, seq, pos, ids, cnt, out, c.ws)
        else:
            s5.step5_paged_attn(c.geom, q, cache, seq, pos, out, c.ws)
    outs = [torch.zeros_like(first) for _ in range(2)]
    graphs = []
    for o in outs:
        call(o)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            call(o)
        graphs.append(gr)
    for _ in range(3):
        c.ws.tensor.fill_(255)
        for o, gr in zip(outs, graphs):
            o.zero_()
            gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, first) for o in outs)
    # other rows in the same graph
    q.copy_(normal(c.gen, *c.q.shape))
    graphs[0].replay()
    call(outs[1])
    assert torch.equal(*outs) and not torch.equal(outs[0], first)
    assert status(s5) == 0


def test_two_streams_at_once(s5):  # noqa: F811
    cases = [Case(s5, [(0, 3000, 1), (1, 800, 1)], seed=1), Case(s5, [(0, 700, 90)], seed=2)]
    want = [c.run() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[torch.zeros_like(w) for _ in range(8)] for w in want]
    caches = [c.cache() for c in cases]
    torch.cuda.synchronize()
    for i in range(8):
        for c, st, o, cache in zip(cases, streams, outs, caches):
            with torch.cuda.stream(st):
                c.run(cache=cache, out=o[i])
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for w, os in zip(want, outs) for o in os)


@pytest.mark.parametrize("runs, picks", [([(0, 1000, 1)], False), ([(0, 900, 40)], False), ([(0, 1000, 2)], True)])
def test_pools_past_32_bit_offsets(s5, runs, picks):  # noqa: F811
    """A pool of 2^24 + 512 token rows and groups (4.3 GB), the sequence's pages at its end."""
    c = Case(s5, runs, G=2, pt=64, seed=3, top_k=32)
    c = c.pick() if picks else c
    want = c.want()
    P = (1 << 24) // 128 + 40
    k, v = (torch.zeros((P, 2, 64, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[P - c.k.shape[0]:], v[P - c.v.shape[0]:] = c.k.cuda(), c.v.cuda()
    got = c.run(cache=s5.PagedCache(k, v, (c.table + (P - c.k.shape[0])).cuda()))
    assert status(s5) == 0
    c.near(got.cpu(), *want)


@pytest.mark.parametrize("N, hq, window", [(1, 8, 0), (1, 4, 700), (2, 16, 5000), (4, 4, 0), (4, 8, 5000), (40, 4, 0), (40, 8, 700), (40, 16, 133)])
def test_the_last_positions_of_all(s5, N, hq, window):  # noqa: F811
    """Rows at the end of a table of 2^31 - 32 tokens.  All its entries but the last name one page, whose
    keys' scores lie so far below the last page's that their weights are zero."""
    gen = torch.Generator().manual_seed(N + hq)
    pt, length = 65528, 32772
    cap = pt * length
    assert cap == 2 ** 31 - 32
    geom = geometry(s5, 1, hq)
    k, v = (normal(gen, 2, 1, pt, 128) for _ in "kv")
    q = normal(gen, N, hq, 128)
    q[..., 0] = 8.0
    k[0, ..., 0], k[1, ..., 0] = -400.0, 0.0
    table = torch.zeros((1, length), dtype=torch.int32)
    table[0, -1] = 1
    seq, pos = torch.zeros(N, dtype=torch.int32), torch.arange(cap - N, cap).int()
    out = torch.full((N, hq, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    kg, vg, tg, qg, sg, pg = dev(k, v, table, q, seq, pos)
    s5.step5_paged_attn(geom, qg, s5.PagedCache(kg, vg, tg), sg, pg, out, s5.PagedWorkspace.create(geom), window=window)
    assert status(s5) == 0
    first = cap - pt
    want, mass = B16.attend(q, k[1:], v[1:], torch.zeros((1, 1), dtype=torch.int32), seq, (pos - first).int(), geom.softmax_scale, window)
    assert B16.off(out, want, mass, B16.shares(N, hq, 1)) <= 1.0


def test_contiguous_caches_as_pages(s5):  # noqa: F811
    """A cache without a table, a page a sequence, against step5_sparse_attn over the same picks."""
    c = Case(s5, [(0, 900, 1), (1, 77, 1)], G=4, pt=1024, seed=5, top_k=64).pick()
    c.k, c.v, c.table = c.k[:2].contiguous(), c.v[:2].contiguous(), None
    got = c.run(cache=s5.PagedCache(*dev(c.k, c.v)))
    assert status(s5) == 0
    c.near(got.cpu(), *c.want())
    other = torch.empty_like(got)
    s5.step5_sparse_attn(c.geom, *dev(c.q, c.k, c.v, c.seq, c.pos, c.ids, c.cnt), other, None)
    out, mass = c.want()
    assert float(((got.double() - other.double()).cpu().abs() / (2 * B16.tolerance(out, mass, True))).max()) <= 1.0


@pytest.mark.parametrize("n", [1, 5, 200])
def test_padding_alone(s5, n):  # noqa: F811
    """Calls whose every row is padding write nothing."""
    for picks in (False, True):
        c = Case(s5, [(-1, 0, n)], G=2, B=1, top_k=8)
        c = c.pick() if picks else c
        assert bool((c.run() == 5.0).all()) and status(s5) == 0


@pytest.mark.parametrize("runs", [[(0, 900, 1), (1, 77, 1)], [(0, 700, 3), (1, 9, 4)], [(0, 650, 60), (1, 0, 60)]])
def test_dense_over_contiguous_caches(s5, runs):  # noqa: F811
    c = Case(s5, runs, G=2, pt=2048, seed=5)
    c.k, c.v, c.table = c.k[:2].contiguous(), c.v[:2].contiguous(), None
    got = c.run(100, cache=s5.PagedCache(*dev(c.k, c.v)))
    assert status(s5) == 0
    c.near(got.cpu(), *c.want(100))


def test_most_rows_of_a_call(s5):  # noqa: F811
    """65,535 rows, on their own and sharing tiles, against a few of them alone."""
    for B, runs in ((65535, [(b, b % 40, 1) for b in range(65535)]), (1, [(0, 0, 65535)])):
        c = Case(s5, [(0, 0, 1)], G=1, hq=4, pt=64, B=1, seed=3)
        seq, pos = rows_of(*runs)
        length = -(-(int(pos.max()) + 1) // 64)
        k, v = (torch.randn((2 * length, 1, 64, 128), generator=torch.Generator("cuda").manual_seed(i), device="cuda").bfloat16() for i in (1, 2))
        table = torch.arange(2 * length, device="cuda").int()[:length].expand(B, length).contiguous()
        cache = s5.PagedCache(k, v, table)
        q = torch.randn((65535, 4, 128), generator=torch.Generator("cuda").manual_seed(3), device="cuda").bfloat16()
        out = torch.full_like(q, 5.0)
        s5.step5_paged_attn(c.geom, q, cache, *dev(seq, pos), out, c.ws, window=300)
        assert status(s5) == 0
        some = torch.tensor([0, 1, 17, 31, 32, 33, 40000, 65533, 65534])
        want = B16.attend(q[some].cpu(), k.cpu(), v.cpu(), table[:1].cpu(), torch.zeros(9, dtype=torch.int32), pos[some],
                          c.geom.softmax_scale, 300)
        assert B16.off(out[some], *want, B == 1) <= 1.0
        assert not bool((out == 5.0).all(-1).any())


def test_run_together(s5):  # noqa: F811
    """Prompts planned, appended and attended in chunks, then decode steps of the whole path with their plan, drafts
    rolled back, over bf16 pages: every output is the attention over what the cache holds."""
    w = S.workload({"positions": [4300, 4170], "B": 2}, seed=41)
    t = S.materialize(w, device="cuda")
    geom, pt, B, N = s5.STEP5_GEOMETRY, 32, 2, 700
    length = -(-4400 // pt)
    slots = s5.PagedTable.create(2 * length, pt, length, B)
    rows = s5.PagedRows.create(B, N)
    cache = s5.PagedCache.create(geom, 2 * length, pt, slots.block_table, e4m3=False)
    pws = s5.PagedWorkspace.create(geom)
    cos, sin = dev(*S.rope_tables(length * pt, 64))
    gen = torch.Generator().manual_seed(2)
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    q = normal(gen, N, 32, 128).cuda()
    q_rot = torch.zeros_like(q)
    out = torch.zeros_like(q)
    at = [0, 0]
    goal = [int(p) for p in w.row_pos]
    while at != goal:
        more = [min(goal[0] - at[0], 400), min(goal[1] - at[1], 300)]
        s5.step5_paged_plan(slots, rows, lengths, torch.tensor(more, dtype=torch.int32, device="cuda"))
        k, v = (torch.zeros((N, 4, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        for b, n0 in ((0, 0), (1, more[0])):
            for dst, src in ((k, t["k_cache"]), (v, t["v_cache"])):
                dst[n0:n0 + more[b]] = src[b, :, at[b]:at[b] + more[b]].transpose(0, 1)
        s5.step5_kv_append(geom, k, v, cache, rows.row_seq, rows.row_pos, cos, sin, q=q, q_out=q_rot)
        s5.step5_paged_attn(geom, q_rot, cache, rows.row_seq, rows.row_pos, out, pws, window=200)
        lengths = rows.ends.clone()
        at = [a + m for a, m in zip(at, more)]
        assert lengths.tolist() == at and status(s5) == 0
    last = rows.row_seq >= 0
    pick = torch.nonzero(last)[:, 0][::37]
    host = [x[pick].cpu() for x in (q_rot, rows.row_seq, rows.row_pos)]
    want = B16.attend(host[0], cache.k.cpu(), cache.v.cpu(), slots.block_table.cpu(), host[1], host[2], geom.softmax_scale, 200)
    assert B16.off(out[pick], *want, True) <= 1.0
    # three drafted tokens each, taken back
    before = [x.clone() for x in (slots.free_pages, slots.free_count, slots.held)]
    for more in (3, 0):
        s5.step5_paged_plan(slots, rows, lengths, torch.full((B,), more, dtype=torch.int32, device="cuda"))
    assert all(torch.equal(a, b) for a, b in zip(before, (slots.free_pages, slots.free_count, slots.held)))
    # the whole path, planned
    ws = s5.Workspace.create(geom, 2, w.r_cap)
    rows = s5.PagedRows.create(B, 2)
    ids = torch.empty((2, 4, 512), dtype=torch.int32, device="cuda")
    cnt = torch.empty((2, 4), dtype=torch.int32, device="cuda")
    out, q_rot = (torch.empty((2, 32, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, v = (torch.stack([t[x][b, :, goal[b]] for b in range(2)]) for x in ("k_cache", "v_cache"))
    one = torch.ones(B, dtype=torch.int32, device="cuda")
    # (the regions before the step's are summarised at once)
    s5.step5_region_summarize(geom, t["idx_k"], t["idx_z"], t["cos"], t["sin"], torch.zeros_like(lengths), lengths // 8, t["summaries"])
    s5.decode_step_paged(geom, t, cache, ws, pws, k, v, ids, cnt, q_rot, out, 1, cos, sin, plan=(slots, rows, lengths, one))
    assert status(s5) == 0
    assert rows.row_pos.tolist() == goal and rows.row_seq.tolist() == [0, 1]
    assert rows.region_end.tolist() == [(p + 1) // 8 for p in goal]
    want = B16.attend(q_rot.cpu(), cache.k.cpu(), cache.v.cpu(), slots.block_table.cpu(), rows.row_seq.cpu(), rows.row_pos.cpu(),
                      geom.softmax_scale, ids=ids.cpu(), counts=cnt.cpu())
    assert B16.off(out, *want, False) <= 1.0
    # the same picks as the bf16 path's over contiguous caches
    ids2, cnt2 = torch.empty_like(ids), torch.empty_like(cnt)
    s5.step5_index_score_topk(geom, t["idx_q"], t["w"], t["row_seq"], t["row_pos"], t["cos"], t["sin"], t["summaries"], ids2,
                              cnt2, ws.tensor, t_cap=t["idx_k"].shape[2])
    assert torch.equal(ids, ids2) and torch.equal(cnt, cnt2)


# ------------------------------------------------------------------------------ what one row's values leave behind

def test_bad_pages_behind_values_that_are_not_finite(s5):  # noqa: F811
    """Blocks of two sequences in turn, so that each CTA takes some of either: one's values are all NaN, the other's first
    pages are bad.  What the first leaves in shared memory does not reach the second, whose rows all see those pages."""
    for bad in (NAN, INF):
        c = Case(s5, [(b, 255, 32) for _ in range(160) for b in range(2)], G=1, hq=8, pt=16, seed=11)
        assert c.shared
        c.v[c.table[0].long()] = bad
        c.table[1, 1:3], c.table[1, 9] = -1, 10 ** 6
        got = c.run().cpu()
        assert status(s5) == 1
        hit = got[c.seq == 0].float()
        assert bool(torch.isnan(hit).all() if bad != bad else (hit == bad).all())
        assert bool(torch.isfinite(got[c.seq == 1]).all())
        some = torch.nonzero(c.seq == 1)[::97, 0]
        want = B16.attend(c.q[some], c.k, c.v, c.table, c.seq[some], c.pos[some], c.geom.softmax_scale, bad_pages=(-1, 10 ** 6))
        assert B16.off(got[some], *want, True) <= 1.0


def milliseconds(fn):
    """The least of five calls."""
    times = []
    for _ in range(6):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        fn()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    return min(times[1:])


@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("block, window", [([(0, 73, 12), (1, 16000, 4)], 0), ([(0, 16001, 16)], 8000)])
def test_values_that_no_row_sees_take_no_time(s5, block, window, bad):  # noqa: F811
    """Blocks with rows of two sequences, and windows, enough of them for whole items: what lies behind the last tokens and
    before the windows is not finite.  It changes no bit and costs about nothing (the tiles that it is cleared from)."""
    c = Case(s5, block * 304, G=1, hq=16, pt=64, seed=12)
    assert c.shared
    clean, cache, q = c.run(window), c.cache(), c.q_on_gpu()
    out, (seq, pos) = torch.zeros_like(clean), dev(c.seq, c.pos)
    call = lambda: s5.step5_paged_attn(c.geom, q, cache, seq, pos, out, c.ws, window=window)
    before = milliseconds(call)
    c.seq, c.pos = c.seq[:16], c.pos[:16]  # (the others see the same)
    cache.v.masked_fill_(c.unseen(window)[:, None, :, None].cuda(), bad)
    after = milliseconds(call)
    assert torch.equal(out, clean) and status(s5) == 0
    assert after <= 1.5 * before + 0.1, (before, after)


def test_values_that_are_seen_far_apart(s5):  # noqa: F811
    """As above, blocks with rows of two sequences: what is not finite at the first tokens and at the last reaches the rows that
    see it, in its dimension, and nothing else changes a bit; the call takes no search of all that lies between."""
    c = Case(s5, [(0, 73, 12), (1, 16000, 4)] * 304, G=1, hq=16, pt=64, seed=13)
    clean, cache, q = c.run(), c.cache(), c.q_on_gpu()
    out, (seq, pos) = torch.zeros_like(clean), dev(c.seq, c.pos)
    call = lambda: s5.step5_paged_attn(c.geom, q, cache, seq, pos, out, c.ws)
    before = milliseconds(call)
    want = clean.clone()
    for b, tok, d, x in ((0, 3, 5, NAN), (0, 80, 6, INF), (1, 2, 7, -INF), (1, 16000, 9, INF), (1, 16001, 20, -INF),
                         (1, 16002, 30, INF), (1, 9000, 30, -INF)):
        page, slot = R.place(c.table, b, tok, c.pt)
        cache.v[page, 0, slot, d] = x
        hit = ((seq == b) & (pos >= tok))[:, None] & (torch.arange(128, device="cuda") == d)
        hit = hit[:, None, :].expand(want.shape)
        want[hit] = x if d != 30 or tok == 16002 else torch.where(want[hit] == INF, NAN, x).bfloat16()
    after = milliseconds(call)
    assert status(s5) == 0
    assert torch.equal(out.nan_to_num(-1e30, 2e30, -2e30), want.nan_to_num(-1e30, 2e30, -2e30))
    assert after <= 4 * before + 0.1, (before, after)


@pytest.mark.parametrize("bad", [NAN, -INF])
@pytest.mark.parametrize("dims", [slice(0, 128), slice(70, 71)])
def test_values_that_are_not_finite_throughout(s5, dims, bad):  # noqa: F811
    """The same where a sequence has them at every token, in every dimension or in one."""
    c = Case(s5, [(0, 73, 12), (1, 16000, 4)] * 304, G=1, hq=16, pt=64, seed=13)
    clean, cache, q = c.run(), c.cache(), c.q_on_gpu()
    out, (seq, pos) = torch.zeros_like(clean), dev(c.seq, c.pos)
    call = lambda: s5.step5_paged_attn(c.geom, q, cache, seq, pos, out, c.ws)
    before = milliseconds(call)
    cache.v[c.table[1].long().cuda(), :, :, dims] = bad
    after = milliseconds(call)
    assert status(s5) == 0
    hit = out[seq == 1][:, :, dims].float()
    assert bool(torch.isnan(hit).all() if bad != bad else (hit == bad).all())
    out[:, :, dims] = torch.where((seq == 1)[:, None, None], clean[:, :, dims], out[:, :, dims])
    assert torch.equal(out, clean)
    assert after <= 20 * before + 0.1, (before, after)


def test_values_that_two_drafts_see_far_apart(s5):  # noqa: F811
    """Rows of two sequences that read their keys together, 304 such items: values that are not finite at the first tokens and at
    the last reach the rows that see them, and the call takes no search of all that lies between."""
    c = Case(s5, [(0, 16000, 1), (1, 15998, 1)], G=1, hq=8, pt=64, seed=14)
    c.table = c.table.repeat(304, 1)
    c.B, c.N, c.seq, c.pos = 608, 1216, torch.arange(608).int().repeat_interleave(2).view(304, 2, 2).transpose(1, 2).reshape(-1).contiguous(), c.pos.repeat(608)
    c.q = normal(c.gen, c.N, 8, 128)
    clean, cache, q = c.run(), c.cache(), c.q_on_gpu()
    out, (seq, pos) = torch.zeros_like(clean), dev(c.seq, c.pos)
    call = lambda: s5.step5_paged_attn(c.geom, q, cache, seq, pos, out, c.ws)
    before = milliseconds(call)
    want = clean.clone()
    for b, tok, d, x in ((0, 3, 5, NAN), (0, 15999, 6, INF), (1, 2, 7, -INF), (1, 15998, 9, INF)):
        page, slot = R.place(c.table, b, tok, c.pt)
        cache.v[page, 0, slot, d] = x
        want[(seq % 2 == b), :, d] = x
    after = milliseconds(call)
    assert status(s5) == 0
    assert torch.equal(out.nan_to_num(-1e30, 2e30, -2e30), want.nan_to_num(-1e30, 2e30, -2e30))
    assert after <= 1.5 * before + 0.1, (before, after)
